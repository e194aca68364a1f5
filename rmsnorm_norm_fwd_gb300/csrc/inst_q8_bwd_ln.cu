// Row-resident backward from the 8-bit checkpoint: LayerNorm.
#define GBN_Q8_LN 1
#define GBN_Q8_NAME kQ8Bwd_ln
#include "inst_q8_bwd_body.cuh"
