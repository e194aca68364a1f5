// Row-resident forward of the 8-bit operators, bf16 rows.
#define GBN_Q8_XT 2
#define GBN_Q8_SUFFIX bf16
#include "inst_q8_fwd_body.cuh"
