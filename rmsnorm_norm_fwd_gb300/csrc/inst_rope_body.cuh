// Vector kernels of the head operators: GBN_MODE, a RopeMode, or -1 - is_layernorm for the backward; GBN_XT, GBN_V, the
// type and elements of a vector.  Defines kRopeVec_<GBN_NAME>[], by lanes a head (4, 8, 16, 32).
#include "rope_vec_kernels.cuh"

namespace gbn {
#ifndef GBN_CAT
#define GBN_CAT2(a, b) a##b
#define GBN_CAT(a, b) GBN_CAT2(a, b)
#endif
const void *const GBN_CAT(kRopeVec_, GBN_NAME)[kRopeVecLanes] = {
#if GBN_MODE >= 0
    (const void *)&rope_fwd_vec<GBN_MODE, GBN_XT, GBN_V, 4, 2>, (const void *)&rope_fwd_vec<GBN_MODE, GBN_XT, GBN_V, 8, 2>,
    (const void *)&rope_fwd_vec<GBN_MODE, GBN_XT, GBN_V, 16, 2>, (const void *)&rope_fwd_vec<GBN_MODE, GBN_XT, GBN_V, 32, 2>
#else
    (const void *)&rope_bwd_vec<GBN_MODE == -2, GBN_XT, GBN_V, 4, 2>,
    (const void *)&rope_bwd_vec<GBN_MODE == -2, GBN_XT, GBN_V, 8, 2>,
    (const void *)&rope_bwd_vec<GBN_MODE == -2, GBN_XT, GBN_V, 16, 2>,
    (const void *)&rope_bwd_vec<GBN_MODE == -2, GBN_XT, GBN_V, 32, 2>
#endif
};
}  // namespace gbn
#undef GBN_MODE
#undef GBN_XT
#undef GBN_V
#undef GBN_NAME
