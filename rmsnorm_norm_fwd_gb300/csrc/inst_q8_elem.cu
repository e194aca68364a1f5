// Element-wise kernels of the 8-bit operators.
#include "q8_elem_kernels.cuh"

namespace gbn {
const void *const kQ8FwdElem[2] = {(const void *)&q8_fwd_elem<false>, (const void *)&q8_fwd_elem<true>};
const void *const kQ8BwdElem[2] = {(const void *)&q8_bwd_elem<false>, (const void *)&q8_bwd_elem<true>};
}  // namespace gbn
