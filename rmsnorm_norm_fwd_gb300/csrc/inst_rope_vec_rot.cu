// Head operators on vectors, one direction and norm.
#define GBN_MODE 0
#define GBN_XT kBF16
#define GBN_V 8
#define GBN_NAME rot_bf16v8
#include "inst_rope_body.cuh"
#define GBN_MODE 0
#define GBN_XT kF16
#define GBN_V 8
#define GBN_NAME rot_f16v8
#include "inst_rope_body.cuh"
#define GBN_MODE 0
#define GBN_XT kBF16
#define GBN_V 4
#define GBN_NAME rot_bf16v4
#include "inst_rope_body.cuh"
#define GBN_MODE 0
#define GBN_XT kF16
#define GBN_V 4
#define GBN_NAME rot_f16v4
#include "inst_rope_body.cuh"
#define GBN_MODE 0
#define GBN_XT kF32
#define GBN_V 4
#define GBN_NAME rot_f32v4
#include "inst_rope_body.cuh"
