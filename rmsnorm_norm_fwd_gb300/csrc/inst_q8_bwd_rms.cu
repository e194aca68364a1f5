// Row-resident backward from the 8-bit checkpoint: RMSNorm.
#define GBN_Q8_LN 0
#define GBN_Q8_NAME kQ8Bwd_rms
#include "inst_q8_bwd_body.cuh"
