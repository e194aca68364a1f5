// inst_q8_fwd_body.cuh -- row-resident forward kernels of the 8-bit operators
// for one storage type of the rows and one norm (the including unit defines
// GBN_Q8_XT, GBN_Q8_LN, GBN_Q8_PRAW and GBN_Q8_NAME).
#include "q8_rows_kernels.cuh"

namespace gbn {

// (TPR, VPT, NT, MINB, CL) by row capacity TPR * VPT * CL * 8; MINB CTAs per SM
// of the launch bound (as many as registers and the parameters in shared memory
// allow).  Measured for bf16 LayerNorm with group scales, 16384 x 8192: 256 x 4
// at four CTAs 82 us, three 88 us, two 99 us; 512 x 2 at two 112 us.  160 x 4
// fills rows of 5120 (16384 x 5120: 62 us against 75 us on 256 x 3); RMSNorm is
// faster there with more CTAs' rows in flight (46 us on 256 x 3, 49 us).  Wide
// LayerNorm rows: clusters of 256-thread CTAs (2048 x 32768: 59 us against 61
// us with 512 threads, 93 us with 1024); RMSNorm is level, on half the CTAs.
#if GBN_Q8_LN
// raw 16-bit gamma and beta leave room for a fourth CTA
#if GBN_Q8_PRAW
#define GBN_Q8_B4 4
#define GBN_Q8_B2 2
#else
#define GBN_Q8_B4 3
#define GBN_Q8_B2 1
#endif
#define GBN_Q8F_GEOMS(X)         \
    X(32, 1, 256, 4, 1)          \
    X(32, 2, 256, 4, 1)          \
    X(32, 4, 256, GBN_Q8_B4, 1)  \
    X(64, 4, 256, GBN_Q8_B4, 1)  \
    X(128, 4, 256, GBN_Q8_B4, 1) \
    X(160, 4, 160, 5, 1)         \
    X(256, 3, 256, GBN_Q8_B4, 1) \
    X(256, 4, 256, GBN_Q8_B4, 1) \
    X(512, 3, 512, GBN_Q8_B2, 1) \
    X(512, 4, 512, GBN_Q8_B2, 1) \
    X(256, 3, 256, GBN_Q8_B4, 4) \
    X(256, 4, 256, GBN_Q8_B4, 4) \
    X(256, 3, 256, GBN_Q8_B4, 8) \
    X(256, 4, 256, GBN_Q8_B4, 8) \
    X(512, 3, 512, GBN_Q8_B2, 8) \
    X(512, 4, 512, GBN_Q8_B2, 8)
#else
#define GBN_Q8F_GEOMS(X) \
    X(32, 1, 256, 4, 1)  \
    X(32, 2, 256, 4, 1)  \
    X(32, 4, 256, 4, 1)  \
    X(64, 4, 256, 4, 1)  \
    X(128, 4, 256, 4, 1) \
    X(256, 3, 256, 4, 1) \
    X(256, 4, 256, 4, 1) \
    X(512, 3, 512, 2, 1) \
    X(512, 4, 512, 2, 1) \
    X(512, 3, 512, 2, 2) \
    X(512, 4, 512, 2, 2) \
    X(512, 3, 512, 2, 4) \
    X(512, 4, 512, 2, 4) \
    X(512, 3, 512, 2, 8) \
    X(512, 4, 512, 2, 8)
#endif

#define GBN_STR2(x) #x
#define GBN_STR(x) GBN_STR2(x)
#define GBN_Q8F_ENTRY(TPR, VPT, NT, MINB, CL, OUT, CK)                                                       \
    {"rows" GBN_STR(TPR) "x" GBN_STR(VPT) "c" GBN_STR(CL),                                                     \
     (const void *)&q8_fwd_rows<GBN_Q8_LN, GBN_Q8_XT, GBN_Q8_PRAW, TPR, VPT, NT, MINB, CL, OUT, CK>, TPR, VPT, \
     NT, CL, q8_fwd_smem(GBN_Q8_LN, GBN_Q8_PRAW, VPT, NT)},
#define GBN_Q8F_Y(T, V, N, B, C) GBN_Q8F_ENTRY(T, V, N, B, C, kOutY, true)
#define GBN_Q8F_R(T, V, N, B, C) GBN_Q8F_ENTRY(T, V, N, B, C, kOutRow, false)
#define GBN_Q8F_G(T, V, N, B, C) GBN_Q8F_ENTRY(T, V, N, B, C, kOutGroup, false)
#define GBN_Q8F_RC(T, V, N, B, C) GBN_Q8F_ENTRY(T, V, N, B, C, kOutRow, true)
#define GBN_Q8F_GC(T, V, N, B, C) GBN_Q8F_ENTRY(T, V, N, B, C, kOutGroup, true)

static const Q8Variant kY[] = {GBN_Q8F_GEOMS(GBN_Q8F_Y)};
static const Q8Variant kR[] = {GBN_Q8F_GEOMS(GBN_Q8F_R)};
static const Q8Variant kG[] = {GBN_Q8F_GEOMS(GBN_Q8F_G)};
static const Q8Variant kRC[] = {GBN_Q8F_GEOMS(GBN_Q8F_RC)};
static const Q8Variant kGC[] = {GBN_Q8F_GEOMS(GBN_Q8F_GC)};
constexpr int kGeoms = (int)(sizeof(kY) / sizeof(kY[0]));
static_assert(kGeoms <= kQ8MaxVariants, "occupancy slots");
const Q8Table GBN_Q8_NAME[5] = {{kY, kGeoms}, {kR, kGeoms}, {kG, kGeoms}, {kRC, kGeoms}, {kGC, kGeoms}};

}  // namespace gbn
