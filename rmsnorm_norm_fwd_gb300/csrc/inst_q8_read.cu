// Vector kernels that read 8-bit rows back: [format][norm][type of y].
#include "q8_read_kernels.cuh"

namespace gbn {
#define GBN_READ(F, NRM) \
    {(const void *)&q8_read_vec<F, NRM, kF32>, (const void *)&q8_read_vec<F, NRM, kF16>, (const void *)&q8_read_vec<F, NRM, kBF16>}
const void *const kQ8Read[2][2][3] = {{GBN_READ(kE4M3, false), GBN_READ(kE4M3, true)},
                                      {GBN_READ(kI8, false), GBN_READ(kI8, true)}};
const int kQ8ReadCTA = kReadCTA, kQ8ReadRows = kReadRows;
}  // namespace gbn
