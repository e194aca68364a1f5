// Row-resident forward of the 8-bit operators, f32 rows.
#define GBN_Q8_XT 0
#define GBN_Q8_SUFFIX f32
#include "inst_q8_fwd_body.cuh"
