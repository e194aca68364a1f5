// Vector kernels of the head operators: GBN_MODE, a RopeMode, or -1 - is_layernorm for the backward; GBN_XT, GBN_V, the
// type and elements of a vector.  Defines kRopeVec_<GBN_NAME>[kind][lanes a head].  Whole heads rotated as halves or as
// neighbours have kernels of their own on 16-byte vectors up to 16 lanes, where they measured faster; the rest runs
// on the kernels for any rotation.
#include "rope_vec_kernels.cuh"

#ifndef GBN_CAT
#define GBN_CAT2(a, b) a##b
#define GBN_CAT(a, b) GBN_CAT2(a, b)
#define GBN_STR2(a) #a
#define GBN_STR(a) GBN_STR2(a)
#endif
#if GBN_MODE >= 0
#define GBN_K(L, KIND, S) \
    {(const void *)&rope_fwd_vec<GBN_MODE, GBN_XT, GBN_V, L, KIND, GBN_FU(KIND), 2>, "vec" GBN_STR(GBN_V) "x" #L S, \
     rope_fwd_smem(GBN_V, GBN_XT == kF32 ? 4 : 2, L, GBN_FU(KIND)), GBN_FU(KIND)}
#else
#define GBN_K(L, KIND, S) \
    {(const void *)&rope_bwd_vec<GBN_MODE == -2, GBN_XT, GBN_V, L, KIND, GBN_BU(KIND), 2>, "vec" GBN_STR(GBN_V) "x" #L S, \
     rope_bwd_smem(GBN_V, GBN_XT == kF32 ? 4 : 2, L, GBN_BU(KIND)), GBN_BU(KIND)}
#endif
#define GBN_FU(KIND) (GBN_MODE == 0 && KIND != kRopeSome ? 2 : 1)
#define GBN_BU(KIND) 1
#define GBN_ANY {GBN_K(4, kRopeSome, ""), GBN_K(8, kRopeSome, ""), GBN_K(16, kRopeSome, ""), GBN_K(32, kRopeSome, "")}

namespace gbn {
const RopeVariant GBN_CAT(kRopeVec_, GBN_NAME)[kRopeVecKinds][kRopeVecLanes] = {
#if GBN_WHOLE
    {GBN_K(4, kRopeHalves, "h"), GBN_K(8, kRopeHalves, "h"), GBN_K(16, kRopeHalves, "h"), GBN_K(32, kRopeSome, "")},
    {GBN_K(4, kRopeNeighbours, "n"), GBN_K(8, kRopeNeighbours, "n"), GBN_K(16, kRopeNeighbours, "n"),
     GBN_K(32, kRopeSome, "")},
#else
    GBN_ANY, GBN_ANY,
#endif
    GBN_ANY};
}  // namespace gbn
#undef GBN_K
#undef GBN_FU
#undef GBN_BU
#undef GBN_ANY
#undef GBN_MODE
#undef GBN_XT
#undef GBN_V
#undef GBN_WHOLE
#undef GBN_NAME
