// q8_params.h -- argument blocks and kernel tables of the 8-bit operators
// (8-bit norm output, 8-bit checkpoint, backward from it, reading back),
// shared by their instantiation units and their host code (q8_api.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "params.h"

namespace gbn {

// Storage formats of 8-bit rows (gbnorm_q8_t).
constexpr int kE4M3 = 0, kI8 = 1;

// Row strides (ld*) are in elements of their tensor.  A group is 2^g
// consecutive columns (the last one of a row may be shorter); qg = -1: one
// scale per row.
struct Q8FwdParams {
    const void *x;      // [M, ldx] xdt
    const void *res;    // [M, ldr] xdt, or null (no residual add)
    void *h;            // [M, ldh] xdt: x + res as normalised, or null (not stored)
    const void *gamma;  // [N] pdt, or null (1)
    const void *beta;   // [N] pdt, or null (0; LayerNorm only)
    void *y;            // [M, ldy] ydt, or null (8-bit output instead)
    uint8_t *q;         // [M, ldq] 8-bit output, or null
    float *qs;          // its scales: row i, group g at i * qs_row + g * qs_grp
    uint8_t *c;         // [M, ldc] checkpoint codes, or null
    float *cs;          // [M, ldcs] (scale, mid) pairs of the checkpoint's groups
    float *mean;        // [M] or null (LayerNorm only)
    float *rstd;        // [M] or null
    int64_t ldx, ldr, ldh, ldy, ldq, qs_row, qs_grp, ldc, ldcs;
    int64_t M, N;
    float eps;
    int xdt, pdt, ydt;
    int qfmt, qg, cg;
    float one;          // 1, not known at compile time (codes8_i8)
};

struct Q8BwdParams {
    const void *dy;     // [M, lddy] ydt
    const uint8_t *c;   // [M, ldc] checkpoint codes
    const float *cs;    // [M, ldcs] (scale, mid) pairs
    const void *dres;   // [M, lddres] xdt added into dx, or null
    const void *gamma;  // [N] pdt, or null (1)
    const float *mean;  // [M] (LayerNorm only)
    const float *rstd;  // [M]
    void *dx;           // [M, lddx] xdt
    float *ws;          // [2][P][N] float partial rows (second block: dbeta)
    int64_t lddy, ldc, ldcs, lddres, lddx;
    int64_t M, N;
    int xdt, pdt, ydt;
    int cg;
};

struct Q8ReadParams {
    const uint8_t *q;   // [M, ldq] 8-bit rows
    const float *scale; // row i, group g at i * s_row + g * s_grp
    const float *mid;   // same layout, or null (0)
    const float *mean;  // [M] or null (0)
    const float *rstd;  // [M] or null (1)
    const void *gamma;  // [N] pdt, or null (1)
    const void *beta;   // [N] pdt, or null (0)
    void *y;            // [M, ldy] ydt
    int64_t ldq, s_row, s_grp, ldy;
    int64_t M, N;
    int pdt, ydt;
    int qfmt, qg;
};

// A compiled kernel with rows in registers: capacity tpr * vpt * cl * 8 elements.
struct Q8Variant {
    const char *name;
    const void *kernel;
    int tpr, vpt, cta;
    int cl;    // CTAs of the cluster that shares a row
    int smem;  // dynamic shared memory
};
struct Q8Table {
    const Q8Variant *v;  // by capacity
    int count;
};
constexpr int kQ8MaxVariants = 24;  // entries per table
// Forward: y and checkpoint; 8-bit rows with a scale per row, with group
// scales; the same two with the checkpoint.
constexpr int kQ8FwdKinds = 5;
extern const Q8Table kQ8Fwd_rms_f32[kQ8FwdKinds], kQ8Fwd_rms_f16[kQ8FwdKinds], kQ8Fwd_rms_bf16[kQ8FwdKinds];
extern const Q8Table kQ8Fwd_ln_f32[kQ8FwdKinds], kQ8Fwd_ln_f16[kQ8FwdKinds], kQ8Fwd_ln_bf16[kQ8FwdKinds];
// LayerNorm with 16-bit gamma and beta of the rows' type, kept so in shared memory.
extern const Q8Table kQ8Fwd_ln_f16_raw[kQ8FwdKinds], kQ8Fwd_ln_bf16_raw[kQ8FwdKinds];

// Backward: dy, dres and dx all fp32, fp16, bf16; any combination.
extern const Q8Table kQ8Bwd_rms[4], kQ8Bwd_ln[4];
// Rows without 16-byte vectors, any types: the forward's kinds, then the backward.
extern const Q8Table kQ8Any_rms[kQ8FwdKinds + 1], kQ8Any_ln[kQ8FwdKinds + 1];
// Reading back: [format][with the norm on top][scale and mid as pairs][type of y]; a second kernel
// argument (int) is the chunks of a row side by side in a CTA.
extern const void *const kQ8Read[2][2][2][3];
extern const int kQ8ReadCTA, kQ8ReadRows;
// Without vectors: [with the norm on top]; a second argument, the blocks of 256
// columns side by side in a CTA.
extern const void *const kQ8ReadAny[2];

// Element-wise kernels, [is_ln].
extern const void *const kQ8FwdElem[2];
extern const void *const kQ8BwdElem[2];

}  // namespace gbn
