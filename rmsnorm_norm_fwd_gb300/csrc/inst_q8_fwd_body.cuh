// inst_q8_fwd_body.cuh -- row-resident forward kernels of the 8-bit operators
// for one storage type of the rows (the including unit defines GBN_Q8_XT and
// GBN_Q8_SUFFIX).
#include "q8_rows_kernels.cuh"

namespace gbn {

// (TPR, VPT, NT, MINB), by row capacity TPR * VPT * 8; MINB CTAs per SM of
// the launch bound.
#define GBN_Q8F_GEOMS(X) \
    X(32, 1, 256, 4)     \
    X(32, 2, 256, 4)     \
    X(32, 4, 256, 4)     \
    X(64, 4, 256, 4)     \
    X(128, 4, 256, 4)    \
    X(256, 3, 256, 4)    \
    X(256, 4, 256, 4)    \
    X(512, 3, 512, 2)    \
    X(512, 4, 512, 2)

#define GBN_STR2(x) #x
#define GBN_STR(x) GBN_STR2(x)
#define GBN_CAT2(a, b) a##b
#define GBN_CAT(a, b) GBN_CAT2(a, b)
#define GBN_Q8F_ENTRY(TPR, VPT, NT, MINB) \
    {"rows" GBN_STR(TPR) "x" GBN_STR(VPT), \
     (const void *)&q8_fwd_rows<GBN_Q8_LN, GBN_Q8_XT, TPR, VPT, NT, MINB, GBN_Q8_OUT, GBN_Q8_CK>, TPR, VPT, NT},

#define GBN_Q8_LN false
#define GBN_Q8_OUT 0
#define GBN_Q8_CK true
static const Q8Variant kRmsY[] = {GBN_Q8F_GEOMS(GBN_Q8F_ENTRY)};
#undef GBN_Q8_OUT
#undef GBN_Q8_CK
#define GBN_Q8_OUT 1
#define GBN_Q8_CK false
static const Q8Variant kRmsQ[] = {GBN_Q8F_GEOMS(GBN_Q8F_ENTRY)};
#undef GBN_Q8_CK
#define GBN_Q8_CK true
static const Q8Variant kRmsQC[] = {GBN_Q8F_GEOMS(GBN_Q8F_ENTRY)};
#undef GBN_Q8_LN
#undef GBN_Q8_OUT
#undef GBN_Q8_CK
#define GBN_Q8_LN true
#define GBN_Q8_OUT 0
#define GBN_Q8_CK true
static const Q8Variant kLnY[] = {GBN_Q8F_GEOMS(GBN_Q8F_ENTRY)};
#undef GBN_Q8_OUT
#undef GBN_Q8_CK
#define GBN_Q8_OUT 1
#define GBN_Q8_CK false
static const Q8Variant kLnQ[] = {GBN_Q8F_GEOMS(GBN_Q8F_ENTRY)};
#undef GBN_Q8_CK
#define GBN_Q8_CK true
static const Q8Variant kLnQC[] = {GBN_Q8F_GEOMS(GBN_Q8F_ENTRY)};

#define GBN_Q8_TABLE(a) {a, (int)(sizeof(a) / sizeof(a[0]))}
const Q8Table GBN_CAT(kQ8Fwd_, GBN_Q8_SUFFIX)[2][3] = {
    {GBN_Q8_TABLE(kRmsY), GBN_Q8_TABLE(kRmsQ), GBN_Q8_TABLE(kRmsQC)},
    {GBN_Q8_TABLE(kLnY), GBN_Q8_TABLE(kLnQ), GBN_Q8_TABLE(kLnQC)}};

}  // namespace gbn
