// Head operators element by element.
#include "rope_any_kernels.cuh"

namespace gbn {
#define GBN_K(F, M, L, C, B) {(const void *)&F<M, L, C, B>, "any" #L "x" #C, (int)sizeof(RopeAnySmem<L, C>), 1, L}
#define GBN_SIZES(F, M) {GBN_K(F, M, 4, 8, 2), GBN_K(F, M, 8, 8, 2), GBN_K(F, M, 16, 8, 2), GBN_K(F, M, 32, 8, 2), GBN_K(F, M, 32, 16, 1)}
const RopeVariant kRopeFwdAny[3][kRopeAnySizes] = {GBN_SIZES(rope_fwd_any, kRopeOnly), GBN_SIZES(rope_fwd_any, kRopeRms),
                                                   GBN_SIZES(rope_fwd_any, kRopeLn)};
const RopeVariant kRopeBwdAny[2][kRopeAnySizes] = {GBN_SIZES(rope_bwd_any, false), GBN_SIZES(rope_bwd_any, true)};
}  // namespace gbn
