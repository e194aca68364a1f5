// inst_q8_bwd_body.cuh -- row-resident backward kernels from the 8-bit
// checkpoint for one norm (the including unit defines GBN_Q8_LN and
// GBN_Q8_NAME): dy, dres and dx of one type (fp32, fp16, bf16), or of any.
#include "q8_bwd_kernels.cuh"

namespace gbn {

// (TPR, VPT, R, NT, MINB, CL) by row capacity TPR * VPT * CL * 8.  LayerNorm
// holds two column sums per element: fewer elements a thread, but two rows at a
// time (bf16 16384 x 8192: 145 us against 173 us one at a time).  RMSNorm with
// its one sum is faster with twice the elements and one row (163 us against 177
// us with a residual's gradient).  Wide rows go to clusters of 256-thread CTAs,
// two an SM, as far as they hold them (RMSNorm 2048 x 65536: 154 us against 162
// us with 512-thread CTAs; LayerNorm 2048 x 32768: 99 us against 106 us).
#if GBN_Q8_LN
#define GBN_Q8B_GEOMS(X, XT)    \
    X(32, 1, 2, 256, 2, 1, XT)  \
    X(32, 2, 2, 256, 2, 1, XT)  \
    X(64, 2, 2, 256, 2, 1, XT)  \
    X(128, 2, 2, 512, 1, 1, XT) \
    X(256, 2, 2, 256, 2, 1, XT) \
    X(320, 2, 1, 320, 2, 1, XT) \
    X(512, 2, 2, 512, 1, 1, XT) \
    X(256, 2, 2, 256, 2, 4, XT) \
    X(256, 2, 2, 256, 2, 8, XT) \
    X(512, 2, 2, 512, 1, 8, XT) \
    X(512, 4, 1, 512, 1, 8, XT)
#else
#define GBN_Q8B_GEOMS(X, XT)    \
    X(32, 1, 2, 256, 3, 1, XT)  \
    X(32, 2, 2, 256, 2, 1, XT)  \
    X(32, 4, 1, 256, 2, 1, XT)  \
    X(64, 4, 1, 256, 2, 1, XT)  \
    X(128, 4, 1, 256, 2, 1, XT) \
    X(160, 4, 1, 160, 3, 1, XT) \
    X(256, 3, 1, 256, 2, 1, XT) \
    X(256, 4, 1, 256, 2, 1, XT) \
    X(512, 3, 1, 512, 1, 1, XT) \
    X(512, 4, 1, 512, 1, 1, XT) \
    X(256, 3, 1, 256, 2, 4, XT) \
    X(256, 4, 1, 256, 2, 4, XT) \
    X(256, 3, 1, 256, 2, 8, XT) \
    X(256, 4, 1, 256, 2, 8, XT) \
    X(512, 4, 1, 512, 1, 8, XT)
#endif
#define GBN_STR2(x) #x
#define GBN_STR(x) GBN_STR2(x)
#define GBN_Q8B_ENTRY(TPR, VPT, R, NT, MINB, CL, XT)                                    \
    {"rows" GBN_STR(TPR) "x" GBN_STR(VPT) "c" GBN_STR(CL) "r" GBN_STR(R),               \
     (const void *)&q8_bwd_rows<GBN_Q8_LN, XT, TPR, VPT, R, NT, MINB, CL>, TPR, VPT, NT, CL, NT * VPT * 32},

static const Q8Variant kB0[] = {GBN_Q8B_GEOMS(GBN_Q8B_ENTRY, kF32)};
static const Q8Variant kB1[] = {GBN_Q8B_GEOMS(GBN_Q8B_ENTRY, kF16)};
static const Q8Variant kB2[] = {GBN_Q8B_GEOMS(GBN_Q8B_ENTRY, kBF16)};
static const Q8Variant kB3[] = {GBN_Q8B_GEOMS(GBN_Q8B_ENTRY, -1)};
constexpr int kGeoms = (int)(sizeof(kB0) / sizeof(kB0[0]));
static_assert(kGeoms <= kQ8MaxVariants, "occupancy slots");
const Q8Table GBN_Q8_NAME[4] = {{kB0, kGeoms}, {kB1, kGeoms}, {kB2, kGeoms}, {kB3, kGeoms}};

}  // namespace gbn
