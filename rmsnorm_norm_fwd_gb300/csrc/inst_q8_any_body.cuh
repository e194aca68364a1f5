// inst_q8_any_body.cuh -- kernels for rows without 16-byte vectors, one norm
// (the including unit defines GBN_Q8_LN and GBN_Q8_NAME).
#include "q8_any_kernels.cuh"

namespace gbn {

// (TPR, VB, NT, MINB, CL) by row capacity TPR * VB * CL * 8.  Four CTAs an SM
// against three: 8192 x 4001 bf16 RMSNorm 32 us against 34 us; four blocks a
// thread on fewer threads 49 us.
#define GBN_Q8A_GEOMS(X)   \
    X(32, 1, 256, 4, 1)    \
    X(32, 2, 256, 4, 1)    \
    X(64, 2, 256, 4, 1)    \
    X(128, 2, 256, 4, 1)   \
    X(256, 2, 256, 4, 1)   \
    X(512, 2, 512, 2, 1)   \
    X(512, 2, 512, 2, 2)   \
    X(512, 2, 512, 2, 4)   \
    X(512, 2, 512, 2, 8)   \
    X(1024, 2, 1024, 1, 8)
// The backward holds dy, xhat and one or two column sums per element.
#define GBN_Q8AB_GEOMS(X)  \
    X(32, 1, 256, 3, 1)    \
    X(32, 2, 256, 2, 1)    \
    X(64, 2, 256, 2, 1)    \
    X(128, 2, 256, 2, 1)   \
    X(256, 2, 256, 2, 1)   \
    X(512, 2, 512, 1, 1)   \
    X(512, 2, 512, 1, 2)   \
    X(512, 2, 512, 1, 4)   \
    X(512, 2, 512, 1, 8)   \
    X(1024, 2, 1024, 1, 8)
#define GBN_STR2(x) #x
#define GBN_STR(x) GBN_STR2(x)
#define GBN_Q8A_FWD(T, V, N, B, C, OUT, CK)                                                                 \
    {"any" GBN_STR(T) "x" GBN_STR(V) "c" GBN_STR(C),                                                        \
     (const void *)&q8_fwd_any<GBN_Q8_LN, T, V, N, B, C, OUT, CK>, T, V, N, C, N * V * 32 * (GBN_Q8_LN ? 2 : 1)},
#define GBN_Q8A_Y(T, V, N, B, C) GBN_Q8A_FWD(T, V, N, B, C, kOutY, true)
#define GBN_Q8A_R(T, V, N, B, C) GBN_Q8A_FWD(T, V, N, B, C, kOutRow, false)
#define GBN_Q8A_G(T, V, N, B, C) GBN_Q8A_FWD(T, V, N, B, C, kOutGroup, false)
#define GBN_Q8A_RC(T, V, N, B, C) GBN_Q8A_FWD(T, V, N, B, C, kOutRow, true)
#define GBN_Q8A_GC(T, V, N, B, C) GBN_Q8A_FWD(T, V, N, B, C, kOutGroup, true)
#define GBN_Q8A_BWD(T, V, N, B, C)                                                                           \
    {"any" GBN_STR(T) "x" GBN_STR(V) "c" GBN_STR(C), (const void *)&q8_bwd_any<GBN_Q8_LN, T, V, N, B, C>, T, V, N, C, \
     N * V * 32},

static const Q8Variant kY[] = {GBN_Q8A_GEOMS(GBN_Q8A_Y)};
static const Q8Variant kR[] = {GBN_Q8A_GEOMS(GBN_Q8A_R)};
static const Q8Variant kG[] = {GBN_Q8A_GEOMS(GBN_Q8A_G)};
static const Q8Variant kRC[] = {GBN_Q8A_GEOMS(GBN_Q8A_RC)};
static const Q8Variant kGC[] = {GBN_Q8A_GEOMS(GBN_Q8A_GC)};
static const Q8Variant kB[] = {GBN_Q8AB_GEOMS(GBN_Q8A_BWD)};
constexpr int kGeoms = (int)(sizeof(kY) / sizeof(kY[0]));
static_assert(kGeoms <= kQ8MaxVariants, "occupancy slots");
const Q8Table GBN_Q8_NAME[kQ8FwdKinds + 1] = {{kY, kGeoms},  {kR, kGeoms},  {kG, kGeoms},
                                              {kRC, kGeoms}, {kGC, kGeoms}, {kB, kGeoms}};

}  // namespace gbn
