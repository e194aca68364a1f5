// rope_params.h -- argument block and launch limits of the head operators:
// norms of queries and keys for each head with the position rotation, their
// backward, the rotation alone (include/gbnorm.h).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gbn {

constexpr int kRopeMaxDim = 1024;  // largest head (GBNORM_MAX_HEAD_DIM)
constexpr int kRopeMaxAxes = 4;    // GBNORM_MAX_AXES (two bits a pair in RopeParams::axis)
constexpr int kRopeCTA = 256;      // threads of a CTA
constexpr int kRopeWarps = kRopeCTA / 32;

// Heads of one tensor: element i of head h of token (b, s) at
// p + (b * batch + s * token + h * head + i) elements (for the kernels on
// vectors the strides are in vectors).
struct RopeHeads {
    void *p;
    int64_t batch, token, head;
};

// Index 0: queries, 1: keys.
struct RopeParams {
    RopeHeads x[2];        // forward: input; backward: the input of the forward
    RopeHeads y[2];        // forward: output; backward: dx
    RopeHeads g[2];        // backward: gradient of the forward's output
    const void *gamma[2];  // [D] pdt, or null (1)
    const void *beta[2];   // [D] pdt, or null (0; LayerNorm only)
    float *mean, *rstd;    // [B * S, H0 + H1] or null; the backward reads them
    float *ws;             // backward: [2][P][2 D] partial rows (second block: dbeta)
    const void *pos;       // positions, strides in elements
    const float *inv_freq; // [rot / 2]
    int64_t pos_axis, pos_batch, pos_token;
    int64_t B, S;
    int64_t units;         // passes over all tokens (a pass: the heads one warp works on at once)
    int64_t warps;         // warps of the grid that take them
    int passes[2];         // of a token
    int rounds;            // whole tokens a warp
    int step_b, step_s;    // warps tokens on, in batches and tokens
    int heads[2];
    int D, rot;
    int inter;             // pairs (2j, 2j + 1), else (j, j + rot / 2)
    int pos64, axes;
    int xdt, ydt, pdt;
    float eps, sign;       // sign -1: the rotation's transpose
    uint32_t axis[kRopeMaxDim / 2 / 16];  // the axis of pair j: bits 2 (j mod 16) of word j / 16
};

enum RopeMode : int { kRopeOnly = 0, kRopeRms = 1, kRopeLn = 2 };

struct RopeVariant {
    const void *f;
    const char *name;
    int smem;  // without parameters (vectors) or column sums (element by element)
    int u;     // heads a lane and pass
    int lanes; // a head
};

// Element by element, any alignment, strides, types and size: [mode][by pairs a head: 32, 64, 128, 256, 512].
constexpr int kRopeAnySizes = 5;
extern const RopeVariant kRopeFwdAny[3][kRopeAnySizes];
extern const RopeVariant kRopeBwdAny[2][kRopeAnySizes];  // RMSNorm, LayerNorm
// The backward's second stage: (ws, int P, int N, dgamma, dbeta), CTAs of 1024 for 32 columns each.
extern const void *const kRopeColumns;

// On vectors of `vector` bytes, c of them for each half of a lane's 2 * half
// elements, l lanes a head, u heads a lane and pass (backward: one): passes in flight a warp, and
// dynamic shared memory without the parameters (rings, tables of cosines and
// sines, frequencies, the backward's sums of the other tensor; its column sums
// take the place of the rings).
// Two passes: forward of 16384 tokens of 40 heads of 128 54.5 us, 56.9 us with
// three, 58.6 us with four; backward 85.0, 88.3 and 89.2 us then.
constexpr int kRopeFwdDepth = 2, kRopeBwdDepth = 2;
constexpr int rope_fwd_smem(int vector, int c, int half, int l, int u) {
    return kRopeWarps * (kRopeFwdDepth * u * 64 * c * vector + 8 * half * l) + 12 * half * l;
}
constexpr int rope_bwd_smem(int vector, int c, int half, int l, bool ln) {
    return kRopeWarps * (kRopeBwdDepth * (128 * c * vector + 256) + 8 * half * l + half * (ln ? 512 : 256)) +
           12 * half * l;
}

constexpr int kRopeVecLanes = 7;
constexpr int kRopeLaneCounts[kRopeVecLanes] = {4, 5, 6, 8, 10, 16, 32};  // lanes a head
constexpr int kRopeVecKinds = 3;  // RopeKind
// For each direction and norm (rot: the rotation alone; b: backward) and vector.
#define GBN_ROPE_VEC(M) \
    extern const RopeVariant kRopeVec_##M##_bf16v8[kRopeVecKinds][kRopeVecLanes], \
        kRopeVec_##M##_f16v8[kRopeVecKinds][kRopeVecLanes], kRopeVec_##M##_bf16v4[kRopeVecKinds][kRopeVecLanes], \
        kRopeVec_##M##_f16v4[kRopeVecKinds][kRopeVecLanes], kRopeVec_##M##_bf16v2[kRopeVecKinds][kRopeVecLanes], \
        kRopeVec_##M##_f16v2[kRopeVecKinds][kRopeVecLanes], kRopeVec_##M##_f32v4[kRopeVecKinds][kRopeVecLanes], \
        kRopeVec_##M##_f32v2[kRopeVecKinds][kRopeVecLanes], kRopeVec_##M##_mixv4[kRopeVecKinds][kRopeVecLanes]
GBN_ROPE_VEC(rot);
GBN_ROPE_VEC(rms);
GBN_ROPE_VEC(ln);
GBN_ROPE_VEC(brms);
GBN_ROPE_VEC(bln);
#undef GBN_ROPE_VEC

}  // namespace gbn
