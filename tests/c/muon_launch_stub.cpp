// Host stand-ins for the Muon kernel launchers, beside launch_stub.cpp, for
// the sanitizer build: every launch reports that no device is present.
#include "muon.hpp"

namespace fsdp {

hipError_t launch_muon_momentum(const MuonItem*, int64_t, const PtrArray&, int, int, bool, float*,
                                void*, int, const MuonScalars&, bool, const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_muon_apply(const MuonItem*, int64_t, const MuonScale*, const void*, int, float*,
                             void*, int, const MuonScalars&, bool, const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_muon_norm(const MuonArgs&, const MuonChunk*, int64_t, const void*, int,
                            const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_muon_convert(const MuonArgs&, const MuonConvertTile*, int64_t, const void*, int,
                               double, const double (&)[3], const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_muon_gram(const MuonArgs&, const MuonTiles&, const MuonTiles&, int,
                            const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_muon_poly(const MuonArgs&, const MuonTiles&, bool, const double (&)[3],
                            const Sink&) {
  return hipErrorNoDevice;
}
hipError_t launch_muon_step(const MuonArgs&, const MuonTiles&, int, bool, bool,
                            const double (&)[3], void*, int, const Sink&) {
  return hipErrorNoDevice;
}

}  // namespace fsdp
