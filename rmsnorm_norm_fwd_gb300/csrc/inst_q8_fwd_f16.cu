// Row-resident forward of the 8-bit operators, f16 rows.
#define GBN_Q8_XT 1
#define GBN_Q8_SUFFIX f16
#include "inst_q8_fwd_body.cuh"
