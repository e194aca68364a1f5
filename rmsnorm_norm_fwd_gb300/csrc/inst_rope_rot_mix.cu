// Head operators on vectors: one direction and norm, these types.
#define GBN_MODE 0
#define GBN_XT kF32
#define GBN_V 2
#define GBN_C 2
#define GBN_WHOLE 0
#define GBN_ODD 0
#define GBN_NAME rot_f32v2
#include "inst_rope_body.cuh"
#define GBN_MODE 0
#define GBN_XT kMixed
#define GBN_V 4
#define GBN_C 2
#define GBN_WHOLE 0
#define GBN_ODD 0
#define GBN_NAME rot_mixv4
#include "inst_rope_body.cuh"
