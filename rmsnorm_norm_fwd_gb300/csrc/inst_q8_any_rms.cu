// 8-bit operators on rows without 16-byte vectors: RMSNorm.
#define GBN_Q8_LN 0
#define GBN_Q8_NAME kQ8Any_rms
#include "inst_q8_any_body.cuh"
