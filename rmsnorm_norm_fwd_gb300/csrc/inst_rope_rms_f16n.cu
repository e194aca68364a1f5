// Head operators on vectors: one direction and norm, these types.
#define GBN_MODE 1
#define GBN_XT kF16
#define GBN_V 4
#define GBN_C 2
#define GBN_WHOLE 1
#define GBN_ODD 1
#define GBN_NAME rms_f16v4
#include "inst_rope_body.cuh"
#define GBN_MODE 1
#define GBN_XT kF16
#define GBN_V 2
#define GBN_C 4
#define GBN_WHOLE 0
#define GBN_ODD 0
#define GBN_NAME rms_f16v2
#include "inst_rope_body.cuh"
