// Row-resident forward of the 8-bit operators: RMSNorm, f32 rows.
#define GBN_Q8_XT 0
#define GBN_Q8_LN 0
#define GBN_Q8_PRAW 0
#define GBN_Q8_NAME kQ8Fwd_rms_f32
#include "inst_q8_fwd_body.cuh"
