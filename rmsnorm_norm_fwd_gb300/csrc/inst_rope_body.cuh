// Vector kernels of the head operators: GBN_MODE, a RopeMode, or -1 - is_layernorm for the backward; GBN_XT, GBN_V,
// GBN_C, the type and elements of a vector and the vectors of half a lane's elements.  Defines
// kRopeVec_<GBN_NAME>[kind][lanes a head].  GBN_WHOLE: whole heads rotated as halves (1) and as neighbours (2) have
// kernels of their own up to 16 lanes (prefill of 16384 tokens of 32 heads of 72, 8-byte vectors, 38 us against 45 us, their
// rotation 33 us against 37 us; not the backward on 8-byte vectors, 64.3 us against 65.8 us); what is rarer runs on the
// kernels for any rotation.  GBN_ODD: heads on 5, 6 and 10 lanes too (heads of 80 16.4 us against 19.0 us).
#include "rope_vec_kernels.cuh"

#ifndef GBN_CAT
#define GBN_CAT2(a, b) a##b
#define GBN_CAT(a, b) GBN_CAT2(a, b)
#define GBN_STR2(a) #a
#define GBN_STR(a) GBN_STR2(a)
#endif
// Heads a lane and pass: two for the rotation alone (26520 tokens of 80 heads 179 us, 194 us with one), one for the
// norms (prefill of 16384 tokens 57.8 us, 64.7 us with two; backward 98 us, 108 us with two).
#define GBN_U(KIND) (GBN_MODE == 0 && KIND != kRopeSome ? 2 : 1)
#define GBN_VECTOR (int)sizeof(RopeRaw<GBN_XT, GBN_V>), GBN_C, GBN_C *GBN_V
#define GBN_NAMED(L, S) "vec" GBN_STR(GBN_V) "x" #L S
#if GBN_MODE >= 0
#define GBN_K(L, KIND, S) \
    {(const void *)&rope_fwd_vec<GBN_MODE, GBN_XT, GBN_V, GBN_C, L, KIND, GBN_U(KIND), 2>, GBN_NAMED(L, S), \
     rope_fwd_smem(GBN_VECTOR, L, GBN_U(KIND)), GBN_U(KIND), L}
#else
#define GBN_K(L, KIND, S) \
    {(const void *)&rope_bwd_vec<GBN_MODE == -2, GBN_XT, GBN_V, GBN_C, L, KIND, 2>, GBN_NAMED(L, S), \
     rope_bwd_smem(GBN_VECTOR, L, GBN_MODE == -2), 1, L}
#endif
#if GBN_ODD
#define GBN_LANES(KIND, S) \
    {GBN_K(4, KIND, S), GBN_K(5, KIND, S), GBN_K(6, KIND, S), GBN_K(8, KIND, S), GBN_K(10, KIND, S), \
     GBN_K(16, KIND, S), GBN_K(32, kRopeSome, "")}
#else
#define GBN_LANES(KIND, S) \
    {GBN_K(4, KIND, S), GBN_K(8, KIND, S), GBN_K(8, KIND, S), GBN_K(8, KIND, S), GBN_K(16, KIND, S), \
     GBN_K(16, KIND, S), GBN_K(32, kRopeSome, "")}
#endif

namespace gbn {
const RopeVariant GBN_CAT(kRopeVec_, GBN_NAME)[kRopeVecKinds][kRopeVecLanes] = {
#if GBN_WHOLE >= 1
    GBN_LANES(kRopeHalves, "h"),
#else
    GBN_LANES(kRopeSome, ""),
#endif
#if GBN_WHOLE >= 2
    GBN_LANES(kRopeNeighbours, "n"),
#else
    GBN_LANES(kRopeSome, ""),
#endif
    GBN_LANES(kRopeSome, "")};
}  // namespace gbn
#undef GBN_LANES
#undef GBN_K
#undef GBN_U
#undef GBN_VECTOR
#undef GBN_NAMED
#undef GBN_MODE
#undef GBN_XT
#undef GBN_V
#undef GBN_C
#undef GBN_WHOLE
#undef GBN_ODD
#undef GBN_NAME
