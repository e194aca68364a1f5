// Row-resident forward of the 8-bit operators: LayerNorm, bf16 rows, gamma and beta of the same type.
#define GBN_Q8_XT 2
#define GBN_Q8_LN 1
#define GBN_Q8_PRAW 1
#define GBN_Q8_NAME kQ8Fwd_ln_bf16_raw
#include "inst_q8_fwd_body.cuh"
