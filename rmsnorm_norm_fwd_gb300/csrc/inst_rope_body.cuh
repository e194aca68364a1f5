// Vector kernels of the head operators: GBN_MODE, a RopeMode, or -1 - is_layernorm for the backward; GBN_XT, GBN_V,
// GBN_C, the type and elements of a vector and the vectors of half a lane's elements.  Defines
// kRopeVec_<GBN_NAME>[kind][lanes a head].  GBN_WHOLE 2: whole heads rotated as halves or as neighbours have kernels of
// their own up to 16 lanes (prefill of 16384 tokens of 32 heads of 72, 8-byte vectors, 38 us against 45 us, their
// rotation 33 us against 37 us).  1: all run on the kernels for any rotation, as the backward on 8-byte vectors (64.3 us
// against 65.8 us); 0: and on powers of two.
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
#define GBN_ANY(L) GBN_K(L, kRopeSome, "")
#if GBN_WHOLE
#define GBN_SOME {GBN_ANY(4), GBN_ANY(5), GBN_ANY(6), GBN_ANY(8), GBN_ANY(10), GBN_ANY(16), GBN_ANY(32)}
#else
#define GBN_SOME {GBN_ANY(4), GBN_ANY(8), GBN_ANY(8), GBN_ANY(8), GBN_ANY(16), GBN_ANY(16), GBN_ANY(32)}
#endif

namespace gbn {
const RopeVariant GBN_CAT(kRopeVec_, GBN_NAME)[kRopeVecKinds][kRopeVecLanes] = {
#if GBN_WHOLE == 2
    {GBN_K(4, kRopeHalves, "h"), GBN_K(5, kRopeHalves, "h"), GBN_K(6, kRopeHalves, "h"), GBN_K(8, kRopeHalves, "h"),
     GBN_K(10, kRopeHalves, "h"), GBN_K(16, kRopeHalves, "h"), GBN_ANY(32)},
    {GBN_K(4, kRopeNeighbours, "n"), GBN_K(5, kRopeNeighbours, "n"), GBN_K(6, kRopeNeighbours, "n"),
     GBN_K(8, kRopeNeighbours, "n"), GBN_K(10, kRopeNeighbours, "n"), GBN_K(16, kRopeNeighbours, "n"), GBN_ANY(32)},
#else
    GBN_SOME, GBN_SOME,
#endif
    GBN_SOME};
}  // namespace gbn
#undef GBN_SOME
#undef GBN_K
#undef GBN_U
#undef GBN_VECTOR
#undef GBN_NAMED
#undef GBN_ANY
#undef GBN_MODE
#undef GBN_XT
#undef GBN_V
#undef GBN_C
#undef GBN_WHOLE
#undef GBN_NAME
