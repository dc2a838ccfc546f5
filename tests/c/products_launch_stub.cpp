// Host stand-ins for the launchers of the unit's products and 8-bit codes, for
// the sanitizer build: every launch reports that no device is present.
#include "products.hpp"
#include "quant.hpp"

namespace fsdp {

hipError_t launch_product(const ProductArgs&, ProductType, int32_t, const ProductRule&,
                          const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_gather_quantize(const QuantItem*, int64_t, const void*, int, const QuantBuffers&,
                                  bool, const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_dequantize(const QuantItem*, int64_t, const QuantBuffers&, int, const PtrArray&,
                             int, const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_quantize_rows(const QuantizeRows&, int, const Sink&) {
  return hipErrorNoDevice;
}

}  // namespace fsdp
