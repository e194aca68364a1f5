// Row-resident forward of the 8-bit operators: LayerNorm, f16 rows.
#define GBN_Q8_XT 1
#define GBN_Q8_LN 1
#define GBN_Q8_PRAW 0
#define GBN_Q8_NAME kQ8Fwd_ln_f16
#include "inst_q8_fwd_body.cuh"
