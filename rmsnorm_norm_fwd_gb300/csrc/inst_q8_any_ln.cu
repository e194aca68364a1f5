// 8-bit operators on rows without 16-byte vectors: LayerNorm.
#define GBN_Q8_LN 1
#define GBN_Q8_NAME kQ8Any_ln
#include "inst_q8_any_body.cuh"
