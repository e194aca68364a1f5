// Head operators element by element.
#include "rope_any_kernels.cuh"

namespace gbn {
namespace {
template <int M, int L, int C, int B> constexpr RopeVariant fwd(const char *name) {
    return {(const void *)&rope_fwd_any<M, L, C, B>, name, (int)sizeof(RopeAnySmem<L, C>), 1, L};
}
template <bool LN, int L, int C, int B> constexpr RopeVariant bwd(const char *name) {
    return {(const void *)&rope_bwd_any<LN, L, C, B>, name, (int)sizeof(RopeAnyBwdSmem<LN, L, C>), 1, L};
}
}  // namespace
#define GBN_SIZES(F, M) \
    {F<M, 4, 8, 2>("any4x8"), F<M, 8, 8, 2>("any8x8"), F<M, 16, 8, 2>("any16x8"), F<M, 32, 8, 2>("any32x8"), \
     F<M, 32, 16, 1>("any32x16")}
const RopeVariant kRopeFwdAny[3][kRopeAnySizes] = {GBN_SIZES(fwd, kRopeOnly), GBN_SIZES(fwd, kRopeRms),
                                                   GBN_SIZES(fwd, kRopeLn)};
const RopeVariant kRopeBwdAny[2][kRopeAnySizes] = {GBN_SIZES(bwd, false), GBN_SIZES(bwd, true)};
const void *const kRopeColumns = (const void *)&rope_columns;
}  // namespace gbn
