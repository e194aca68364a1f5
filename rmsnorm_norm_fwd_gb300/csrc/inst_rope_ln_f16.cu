// Head operators on vectors: one direction and norm, these types.
#define GBN_MODE 2
#define GBN_XT kF16
#define GBN_V 8
#define GBN_C 1
#define GBN_WHOLE 2
#define GBN_ODD 1
#define GBN_NAME ln_f16v8
#include "inst_rope_body.cuh"
