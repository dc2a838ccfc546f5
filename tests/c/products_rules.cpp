// What the host side does with a product (no GPU; launches report that there
// is no device).  Every line of the input is one, "op type groups rows n k lda
// ldb ldc aligned" (type 0 fp32, 1 bf16, 2 codes; a pitch of 0: the row's length;
// aligned 0: operands half a word off); every line of the output "tile direct
// n_parts status" of its rule and its call.
#include <cstdio>

#include "products.hpp"

int main() {
  fsdp_matmul m{};
  int type, aligned;
  long long rows, n, k, lda, ldb, ldc;
  while (std::scanf("%d %d %d %lld %lld %lld %lld %lld %lld %d", &m.op, &type, &m.groups, &rows,
                    &n, &k, &lda, &ldb, &ldc, &aligned) == 10) {
    const bool tn = m.op == FSDP_MATMUL_TN, nt = m.op == FSDP_MATMUL_NT, codes = type == 2;
    auto pitch = [&](long long x) { return codes ? (x + 15) / 16 * 16 : x; };
    m.rows = rows;
    m.n = n;
    m.k = k;
    m.lda = lda ? lda : pitch(tn ? n : k);
    m.ldb = ldb ? ldb : pitch(nt || tn ? k : n);
    m.ldc = ldc ? ldc : tn ? k : n;
    m.group_stride = m.groups > 1 ? (tn ? n * m.ldc : (nt ? n : k) * m.ldb) : 0;
    // far-apart addresses that nothing reads
    auto at = [&](int i, int off = 0) {
      return reinterpret_cast<void*>((uintptr_t(1) << 45) + i * (uintptr_t(1) << 42) + off);
    };
    const int32_t* offsets = static_cast<const int32_t*>(at(0));
    const int off = aligned ? 0 : type == 1 ? 2 : 4;
    int32_t status;
    if (codes)
      status = fsdp_grouped_matmul_i8(&m, offsets, static_cast<const int8_t*>(at(1)),
                                      static_cast<const float*>(at(4)),
                                      static_cast<const int8_t*>(at(2)), nullptr, 0, at(3),
                                      FSDP_F32, nullptr);
    else
      status = fsdp_grouped_matmul(&m, offsets, at(1, off), at(2, off), type, at(3), FSDP_F32,
                                   at(5), int64_t(1) << 40, nullptr);
    // (as the call finds it: pieces of 16 bytes that are aligned and whole)
    const bool direct = codes || (type == 1 && aligned && (tn ? n : k) % 8 == 0 &&
                                  (nt || tn ? k : n) % 8 == 0 && m.lda % 8 == 0 && m.ldb % 8 == 0);
    const fsdp::ProductRule r =
        fsdp::product_rule(m, static_cast<fsdp::ProductType>(type), direct);
    std::printf("%d %d %d %d\n", r.tile, int(r.direct), r.n_parts, status);
  }
  return 0;
}
