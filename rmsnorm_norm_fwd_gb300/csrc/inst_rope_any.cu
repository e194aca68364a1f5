// Head operators element by element.
#include "rope_any_kernels.cuh"

namespace gbn {
#define GBN_FWD(MODE) \
    {(const void *)&rope_fwd_any<MODE, 1>, (const void *)&rope_fwd_any<MODE, 2>, (const void *)&rope_fwd_any<MODE, 4>, \
     (const void *)&rope_fwd_any<MODE, 8>, (const void *)&rope_fwd_any<MODE, 16>}
#define GBN_BWD(LN) \
    {(const void *)&rope_bwd_any<LN, 1>, (const void *)&rope_bwd_any<LN, 2>, (const void *)&rope_bwd_any<LN, 4>, \
     (const void *)&rope_bwd_any<LN, 8>, (const void *)&rope_bwd_any<LN, 16>}
const void *const kRopeFwdAny[3][kRopeAnySizes] = {GBN_FWD(kRopeOnly), GBN_FWD(kRopeRms), GBN_FWD(kRopeLn)};
const void *const kRopeBwdAny[2][kRopeAnySizes] = {GBN_BWD(false), GBN_BWD(true)};
}  // namespace gbn
