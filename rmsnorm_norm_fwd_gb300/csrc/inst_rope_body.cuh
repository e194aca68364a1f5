// Vector kernels of the head operators: GBN_MODE, a RopeMode, or -1 - is_layernorm for the backward; GBN_XT, GBN_V,
// GBN_C, the type and elements of a vector and the vectors of half a lane's elements.  Defines
// kRopeVec_<GBN_NAME>[kind][lanes a head].
//
// GBN_WHOLE: whole heads rotated as halves (1) and as neighbours (2) have kernels of their own up to 16 lanes; what is
// rarer runs on the kernels for any rotation.  With them and without, bf16, 16384 tokens of 32 + 8 heads as halves
// (heads of 256: 8192), us:
//     head   RMSNorm, LayerNorm      backward of each        rotation
//      64    30.9 33.1  35.5 40.7    44.8 45.6  54.2 57.2    28.2 30.4
//      96    46.9 50.0  53.8 62.0    67.1 69.5  82.3 85.1    41.3 45.8
//     128    54.3 56.0  58.8 66.8    81.9 80.8  89.1 92.3    57.2 53.6
//     256    56.3 56.5  58.5 63.4    88.0 83.3  88.1 90.1    57.2 55.2
// (the rotation of 26520 tokens of 80 heads of 128: 170 us, 179 us).  Neighbours the same within 1% where they have
// kernels; fp32, at 90% of the copy rate either way, within 1% (rotation of heads of 64: 55.2 us, 53.0 us).  On 8-byte
// vectors heads of 72 37.8 us against 45 us, their rotation 33 us against 37 us, not the backward: 64.3 us, 65.8 us.
//
// GBN_ODD: heads on 5, 6 and 10 lanes too, else on the next power of two.  With them and without, 16384 tokens of
// 16 + 16 heads as halves, us (80, 96, 160: bf16 on 16-byte vectors; 72, 88, 152: fp16 on 8-byte ones):
//     head lanes  RMSNorm, LayerNorm      backward of each          rotation
//      80    5    35.9 41.8  42.5 51.0    54.6  63.6   65.1  79.1   35.1 32.6
//      96    6    41.3 42.4  49.8 51.4    61.0  63.6   75.6  79.2   34.5 34.0
//     160   10    60.5 70.2  72.1 88.2    93.7 113.1  115.5 143.2   57.6 54.4
//      72    5    37.8 43.4  46.8 54.8    65.8  75.7   83.3  90.7   33.8 32.2
//      88    6    43.3 43.7  54.7 55.1    76.1  76.0   99.2  91.2   35.2 34.8
//     152   10    62.2 72.0  81.8 98.1   118.4 133.2  158.0 168.6   54.8 58.4
// Heads of 112 and 192 leave an eighth and a quarter of 8 and 16 lanes without work: 44.1 us and 74.4 us forward (78%
// and 80% of the copy rate), 65.5 us and 113 us backward.
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
