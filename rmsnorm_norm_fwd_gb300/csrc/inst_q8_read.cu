// Kernels that read 8-bit rows back.
#include "q8_any_kernels.cuh"
#include "q8_read_kernels.cuh"

namespace gbn {
#define GBN_READ(F, NRM, PR)                                                                             \
    {(const void *)&q8_read_vec<F, NRM, PR, kF32>, (const void *)&q8_read_vec<F, NRM, PR, kF16>, \
     (const void *)&q8_read_vec<F, NRM, PR, kBF16>}
#define GBN_READ2(F) \
    {{GBN_READ(F, false, false), GBN_READ(F, false, true)}, {GBN_READ(F, true, false), GBN_READ(F, true, true)}}
const void *const kQ8Read[2][2][2][3] = {GBN_READ2(kE4M3), GBN_READ2(kI8)};
const void *const kQ8ReadAny[2] = {(const void *)&q8_read_any<false>, (const void *)&q8_read_any<true>};
const int kQ8ReadCTA = kReadCTA, kQ8ReadRows = kReadRows;
}  // namespace gbn
