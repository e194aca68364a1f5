// q8_api.cu -- the C ABI of the 8-bit operators (include/gbnorm.h): argument
// checks, the choice of a kernel, launches.  As in api.cu nothing here
// allocates device memory or synchronises.
#include <atomic>
#include <cmath>
#include <cstdio>
#include <initializer_list>

#include <cuda_runtime.h>

#include "../../include/gbnorm.h"
#include "host_shared.h"
#include "q8_params.h"

namespace gbn {
namespace {

int elem_size(int dtype) { return dtype == GBNORM_F32 ? 4 : 2; }
bool valid_dtype(int d) { return d == GBNORM_F32 || d == GBNORM_F16 || d == GBNORM_BF16; }
bool aligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool valid_shape(int64_t M, int64_t N) {
    if (M < 0 || N < 1 || N > GBNORM_MAX_N) return false;
    return M == 0 || M <= (INT64_MAX / 16) / N;  // byte offsets fit comfortably in int64
}
bool valid_ld(int64_t ld, int64_t N, int64_t M) { return ld >= N && (M == 0 || ld <= (INT64_MAX / 16) / M); }

// log2 of a group size, -1 for one scale per row, -2 if not supported.
int group_log2(int group) {
    switch (group) {
        case 0: return -1;
        case 32: return 5;
        case 64: return 6;
        case 128: return 7;
        case 256: return 8;
        default: return -2;
    }
}
int64_t groups_of(int64_t N, int lg) { return lg < 0 ? 1 : (N + ((int64_t)1 << lg) - 1) >> lg; }

// A tensor as the aliasing check sees it: the bytes [p, p + bytes), and what
// has to agree for an output to be exactly an input (in place).
struct Span {
    const void *p;
    size_t bytes;
    int64_t ld;   // row stride in elements; 0: not a row tensor
    int es;       // element size
    bool inplace; // outputs: may be exactly a row tensor among the inputs (inputs: may be overwritten so)
};
Span rows(const void *p, int64_t M, int64_t N, int64_t ld, int es, bool inplace) {
    return {p, p && M > 0 ? ((size_t)(M - 1) * (size_t)ld + (size_t)N) * (size_t)es : 0, ld, es, inplace};
}
Span flat(const void *p, int64_t n, int es) { return {p, p ? (size_t)n * (size_t)es : 0, 0, es, false}; }

// Every pointer of these is aligned to its elements (NULL is).
struct Typed {
    const void *p;
    int es;
};
bool elements_aligned(std::initializer_list<Typed> l) {
    for (const Typed &t : l)
        if (!aligned(t.p, (unsigned)t.es)) return false;
    return true;
}

// 16-byte vectors for a row tensor: aligned base and row stride.
bool vec_rows(const void *p, int64_t ld, int es) { return !p || (aligned(p, 16) && (ld * es) % 16 == 0); }

bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
bool bad_aliasing(const Span *outs, int no, const Span *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j) {
            const Span &o = outs[i], &s = ins[j];
            if (o.inplace && s.inplace && o.p == s.p && o.ld == s.ld && o.es == s.es && o.bytes == s.bytes) continue;
            if (overlap(o, s)) return true;
        }
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

// Scales of [M, G] groups at i * row + g * grp: positive strides that put no
// two of them in one place.  The floats they span, 0 if invalid.
int64_t scale_span(int64_t M, int64_t G, int64_t row, int64_t grp) {
    if (M == 0) return 1;
    const int64_t most = INT64_MAX / 64;
    if ((M > 1 && (row < 1 || row > most / M)) || (G > 1 && (grp < 1 || grp > most / G))) return 0;
    const int64_t rs = M > 1 ? (M - 1) * row : 0, gs = G > 1 ? (G - 1) * grp : 0;
    if (M > 1 && G > 1 && row <= gs && grp <= rs) return 0;
    return rs + gs + 1;
}

// Name of the kernel the calling thread's last call launched: forward,
// backward, read.
thread_local const char *t_last[3] = {"", "", ""};

int launch(const void *kernel, int64_t grid, int cta, size_t dyn, void *params, cudaStream_t s) {
    void *args[1] = {params};
    if (cudaLaunchKernel(kernel, dim3((unsigned)grid), dim3((unsigned)cta), args, dyn, s) != cudaSuccess)
        return GBNORM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? GBNORM_OK : GBNORM_ERR_CUDA;
}

// Persistent grid of `units` pieces of work at `per_sm` CTAs an SM.
int64_t grid_of(int64_t units, int64_t per_sm, const HostDevice &d) {
    int64_t cap = per_sm * d.sms;
    const int64_t limit = host_grid_limit();
    if (limit > 0 && limit < cap) cap = limit;
    return units < cap ? units : cap;
}

// Kernels with rows in registers: how many row groups (CTAs, or clusters) run
// at once on the device, measured once per device and slot.
constexpr int kBwdSlots = 3 * 3 * kQ8FwdKinds * kQ8MaxVariants, kAnySlots = kBwdSlots + 2 * 4 * kQ8MaxVariants,
              kSlots = kAnySlots + 2 * (kQ8FwdKinds + 1) * kQ8MaxVariants;
std::atomic<int> g_resident[kHostMaxDev][kSlots];

int cluster_launch(const Q8Variant &v, int64_t units, void *params, cudaStream_t s, cudaLaunchConfig_t *cfg,
                   cudaLaunchAttribute *attr) {
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)v.cl;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    *cfg = {};
    cfg->gridDim = dim3((unsigned)(units * v.cl));
    cfg->blockDim = dim3((unsigned)v.cta);
    cfg->dynamicSmemBytes = (size_t)v.smem;
    cfg->stream = s;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
    if (!params) return GBNORM_OK;
    void *args[1] = {params};
    if (cudaLaunchKernelExC(cfg, v.kernel, args) != cudaSuccess) return GBNORM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? GBNORM_OK : GBNORM_ERR_CUDA;
}

int resident(const Q8Variant &v, int slot, const HostDevice &d, int *out) {
    std::atomic<int> &c = g_resident[d.dev][slot];
    int o = c.load(std::memory_order_relaxed);
    if (o == 0) {
        if (cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess)
            return GBNORM_ERR_CUDA;
        if (v.cl == 1) {
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, v.kernel, v.cta, (size_t)v.smem) != cudaSuccess)
                return GBNORM_ERR_CUDA;
            o *= d.sms;
        } else {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute attr;
            cluster_launch(v, 1, nullptr, nullptr, &cfg, &attr);
            if (cudaOccupancyMaxActiveClusters(&o, v.kernel, &cfg) != cudaSuccess) return GBNORM_ERR_CUDA;
        }
        if (o <= 0) return GBNORM_ERR_UNSUPPORTED;
        c.store(o, std::memory_order_relaxed);
    }
    *out = o;
    return GBNORM_OK;
}

// CTAs (clusters) of variant v over M rows.
int row_units(const Q8Variant &v, int slot, int64_t M, const HostDevice &d, int64_t *units) {
    int o;
    const int st = resident(v, slot, d, &o);
    if (st != GBNORM_OK) return st;
    const int64_t rpc = v.cta / v.tpr, want = (M + rpc - 1) / rpc;
    int64_t cap = o;
    const int64_t limit = host_grid_limit();
    if (limit > 0 && limit / v.cl < cap) cap = limit / v.cl > 0 ? limit / v.cl : 1;
    *units = want < cap ? want : cap;
    return GBNORM_OK;
}

int launch_rows(const Q8Variant &v, int64_t units, void *params, cudaStream_t s) {
    if (v.cl == 1) return launch(v.kernel, units, v.cta, (size_t)v.smem, params, s);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    return cluster_launch(v, units, params, s, &cfg, &attr);
}

// The first variant of the table that holds N elements, -1 if none does.
int find_rows(const Q8Table &t, int64_t N) {
    for (int i = 0; i < t.count; ++i)
        if ((int64_t)t.v[i].tpr * t.v[i].vpt * t.v[i].cl * 8 >= N) return i;
    return -1;
}

// Checks shared by the two forwards; fills the spans of what every forward has.
struct FwdArgs {
    int is_ln;
    Q8FwdParams p;
    int qgroup, cgroup;
};

int do_fwd(FwdArgs &a, cudaStream_t stream) {
    Q8FwdParams &p = a.p;
    if ((a.is_ln != 0 && a.is_ln != 1) || !valid_dtype(p.xdt) || !valid_dtype(p.pdt) || !valid_dtype(p.ydt))
        return GBNORM_ERR_INVALID_ARG;
    if (!valid_shape(p.M, p.N) || !std::isfinite(p.eps) || p.eps < 0.f) return GBNORM_ERR_INVALID_ARG;
    if (p.qfmt != GBNORM_E4M3 && p.qfmt != GBNORM_INT8) return GBNORM_ERR_INVALID_ARG;
    p.qg = group_log2(a.qgroup);
    p.cg = group_log2(a.cgroup);
    const int64_t M = p.M, N = p.N;
    if (!a.is_ln) {
        p.beta = nullptr;
        p.mean = nullptr;
    }
    if (!p.res && p.h) return GBNORM_ERR_INVALID_ARG;
    if (!p.res) p.ldr = N;
    if (!p.h) p.ldh = N;
    if (!p.y) p.ldy = N;
    if (!p.q) p.ldq = N;
    if (!p.c) p.ldc = N;
    const int xs = elem_size(p.xdt), ps = elem_size(p.pdt);
    if (!elements_aligned({{p.x, xs}, {p.res, xs}, {p.h, xs}, {p.y, elem_size(p.ydt)}, {p.gamma, ps}, {p.beta, ps},
                           {p.mean, 4}, {p.rstd, 4}}))
        return GBNORM_ERR_INVALID_ARG;
    int64_t qspan = 0, cspan = 0;
    for (int64_t ld : {p.ldx, p.ldr, p.ldh, p.ldy, p.ldq, p.ldc})
        if (M > 0 && !valid_ld(ld, N, M)) return GBNORM_ERR_INVALID_ARG;
    if (p.q) {
        if (p.qg == -2 || !p.qs || !aligned(p.qs, 4)) return GBNORM_ERR_INVALID_ARG;
        qspan = scale_span(M, groups_of(N, p.qg), p.qs_row, p.qs_grp);
        if (qspan == 0) return GBNORM_ERR_INVALID_ARG;
    }
    if (p.c) {
        const int64_t pairs = 2 * groups_of(N, p.cg);
        if (p.cg < 0 || !p.cs || !aligned(p.cs, 8) || (M > 0 && !valid_ld(p.ldcs, pairs, M)) || p.ldcs % 2 != 0)
            return GBNORM_ERR_INVALID_ARG;
        cspan = M > 0 ? (M - 1) * p.ldcs + pairs : 0;
    }
    if (M > 0 && (!p.x || (!p.y && !p.q))) return GBNORM_ERR_INVALID_ARG;
    const Span outs[8] = {rows(p.y, M, N, p.ldy, elem_size(p.ydt), true), rows(p.h, M, N, p.ldh, xs, true),
                          rows(p.q, M, N, p.ldq, 1, false), rows(p.c, M, N, p.ldc, 1, false),
                          flat(p.qs, p.q && M > 0 ? qspan : 0, 4), flat(p.cs, p.c ? cspan : 0, 4),
                          flat(p.rstd, M, 4), flat(p.mean, M, 4)};
    const Span ins[4] = {rows(p.x, M, N, p.ldx, xs, true), rows(p.res, M, N, p.ldr, xs, true),
                         flat(p.gamma, N, ps), flat(p.beta, N, ps)};
    if (bad_aliasing(outs, 8, ins, 4)) return GBNORM_ERR_INVALID_ARG;
    HostDevice d;
    const int s = host_device(&d);
    if (s != GBNORM_OK) return s;
    t_last[0] = "";
    if (M == 0) return GBNORM_OK;
    const bool vec = N % 8 == 0 && vec_rows(p.x, p.ldx, xs) && vec_rows(p.res, p.ldr, xs) && vec_rows(p.h, p.ldh, xs) &&
                     vec_rows(p.y, p.ldy, elem_size(p.ydt)) && aligned(p.gamma, 16) && aligned(p.beta, 16) &&
                     aligned(p.q, 8) && p.ldq % 8 == 0 && aligned(p.c, 8) && p.ldc % 8 == 0;
    // rows: RMSNorm, LayerNorm, LayerNorm with gamma and beta of the rows' type
    static const Q8Table *const tables[3][3] = {{kQ8Fwd_rms_f32, kQ8Fwd_rms_f16, kQ8Fwd_rms_bf16},
                                                {kQ8Fwd_ln_f32, kQ8Fwd_ln_f16, kQ8Fwd_ln_bf16},
                                                {kQ8Fwd_ln_f32, kQ8Fwd_ln_f16_raw, kQ8Fwd_ln_bf16_raw}};
    const int op = a.is_ln && p.pdt == p.xdt ? 2 : a.is_ln;
    const int kind = p.y ? 0 : (p.qg < 0 ? 1 : 2) + (p.c ? 2 : 0);
    const Q8Table &t = vec ? tables[op][p.xdt][kind] : (a.is_ln ? kQ8Any_ln : kQ8Any_rms)[kind];
    const int i = find_rows(t, N);
    if (i >= 0) {
        const int slot = (vec ? ((p.xdt * 3 + op) * kQ8FwdKinds + kind) * kQ8MaxVariants
                              : kAnySlots + (a.is_ln * (kQ8FwdKinds + 1) + kind) * kQ8MaxVariants) + i;
        int64_t units;
        const int st = row_units(t.v[i], slot, M, d, &units);
        if (st == GBNORM_OK) {
            t_last[0] = t.v[i].name;
            return launch_rows(t.v[i], units, &p, stream);
        }
        if (st != GBNORM_ERR_UNSUPPORTED) return st;  // else this device holds no such CTA or cluster
    }
    t_last[0] = "elem";
    return launch(kQ8FwdElem[a.is_ln], grid_of(M, 8, d), kElemCTA, 0, &p, stream);
}

// The backward's kernel for rows of these storage types (x_dtype == y_dtype: that
// type, else 3; without vectors 4) and its partial rows; v NULL: element by
// element, one CTA per SM.
struct BwdPlan {
    const Q8Variant *v;
    int64_t P;
};
int bwd_plan(int is_ln, int types, int64_t M, int64_t N, const HostDevice &d, BwdPlan *pl) {
    const Q8Table &t = types < 4 ? (is_ln ? kQ8Bwd_ln : kQ8Bwd_rms)[types] : (is_ln ? kQ8Any_ln : kQ8Any_rms)[kQ8FwdKinds];
    const int i = find_rows(t, N);
    if (i >= 0) {
        const int slot = (types < 4 ? kBwdSlots + (is_ln * 4 + types) * kQ8MaxVariants
                                    : kAnySlots + (is_ln * (kQ8FwdKinds + 1) + kQ8FwdKinds) * kQ8MaxVariants) + i;
        const int st = row_units(t.v[i], slot, M, d, &pl->P);
        pl->v = &t.v[i];
        if (st != GBNORM_ERR_UNSUPPORTED) return st;
    }
    *pl = BwdPlan{nullptr, grid_of(M, 1, d)};
    return GBNORM_OK;
}
// Workspace: the most partial rows that any types and alignment need for this
// shape, so that it depends on the shape alone.
int bwd_ws_bytes(int is_ln, int64_t M, int64_t N, const HostDevice &d, size_t *bytes) {
    int64_t P = 0;
    for (int types = N % 8 == 0 ? 0 : 4; types <= 4 && M > 0; ++types) {
        BwdPlan pl;
        const int st = bwd_plan(is_ln, types, M, N, d, &pl);
        if (st != GBNORM_OK) return st;
        if (pl.P > P) P = pl.P;
    }
    *bytes = ((size_t)P * (size_t)N * 4u * (is_ln ? 2u : 1u) + 255u) & ~(size_t)255u;
    return GBNORM_OK;
}

}  // namespace
}  // namespace gbn

using namespace gbn;

extern "C" {

int norm_fwd_q8(int is_layernorm, int64_t M, int64_t N, float eps, const void *x, int64_t ldx, int x_dtype,
                const void *residual, int64_t ldr, void *h, int64_t ldh, const void *gamma, const void *beta,
                int param_dtype, void *q, int64_t ldq, int q_format, int q_group, float *q_scale, int64_t qs_row,
                int64_t qs_group, int8_t *codes, int64_t ldc, int c_group, float *c_scale, int64_t ldcs, float *mean,
                float *rstd, gbnorm_stream_t stream) {
    if (M > 0 && !q) return GBNORM_ERR_INVALID_ARG;
    FwdArgs a{is_layernorm, {}, q_group, codes ? c_group : 128};
    a.p = Q8FwdParams{x, residual, h, gamma, beta, nullptr, static_cast<uint8_t *>(q), q_scale,
                      reinterpret_cast<uint8_t *>(codes), c_scale, mean, rstd, ldx, ldr, ldh, N, ldq, qs_row, qs_group,
                      ldc, ldcs, M, N, eps, x_dtype, param_dtype, x_dtype, q_format, 0, 0, 1.f};
    return do_fwd(a, stream);
}

int norm_fwd_ck8(int is_layernorm, int64_t M, int64_t N, float eps, const void *x, int64_t ldx, int x_dtype,
                 const void *residual, int64_t ldr, void *h, int64_t ldh, const void *gamma, const void *beta,
                 int param_dtype, void *y, int64_t ldy, int y_dtype, int8_t *codes, int64_t ldc, int c_group,
                 float *c_scale, int64_t ldcs, float *mean, float *rstd, gbnorm_stream_t stream) {
    if (M > 0 && (!y || !codes)) return GBNORM_ERR_INVALID_ARG;
    FwdArgs a{is_layernorm, {}, 0, c_group};
    a.p = Q8FwdParams{x, residual, h, gamma, beta, y, nullptr, nullptr, reinterpret_cast<uint8_t *>(codes), c_scale,
                      mean, rstd, ldx, ldr, ldh, ldy, N, 1, 1, ldc, ldcs, M, N, eps, x_dtype, param_dtype, y_dtype,
                      GBNORM_E4M3, 0, 0, 1.f};
    return do_fwd(a, stream);
}

size_t norm_bwd_ck8_workspace_size(int is_layernorm, int64_t M, int64_t N) {
    if ((is_layernorm != 0 && is_layernorm != 1) || !valid_shape(M, N)) return 0;
    HostDevice d;
    size_t need = 0;
    if (host_device(&d) != GBNORM_OK || bwd_ws_bytes(is_layernorm, M, N, d, &need) != GBNORM_OK) return 0;
    return need > 0 ? need : 256;  // M = 0: nothing is used; 0 means an error
}

int norm_bwd_ck8(int is_layernorm, int64_t M, int64_t N, const void *dy, int64_t lddy, int y_dtype,
                 const int8_t *codes, int64_t ldc, int c_group, const float *c_scale, int64_t ldcs, const void *dres,
                 int64_t lddres, const void *gamma, int param_dtype, const float *mean, const float *rstd, void *dx,
                 int64_t lddx, int x_dtype, float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes,
                 gbnorm_stream_t stream) {
    const int cg = group_log2(c_group);
    if ((is_layernorm != 0 && is_layernorm != 1) || !valid_dtype(x_dtype) || !valid_dtype(param_dtype) ||
        !valid_dtype(y_dtype) || !valid_shape(M, N) || cg < 0)
        return GBNORM_ERR_INVALID_ARG;
    if (!is_layernorm) {
        dbeta = nullptr;
        mean = nullptr;
    }
    if (!dres) lddres = N;
    const int64_t pairs = 2 * groups_of(N, cg);
    if (M > 0) {
        if (!dy || !codes || !c_scale || !rstd || !dx || (is_layernorm && !mean)) return GBNORM_ERR_INVALID_ARG;
        for (int64_t ld : {lddy, ldc, lddres, lddx})
            if (!valid_ld(ld, N, M)) return GBNORM_ERR_INVALID_ARG;
        if (!valid_ld(ldcs, pairs, M) || ldcs % 2 != 0 || !aligned(c_scale, 8)) return GBNORM_ERR_INVALID_ARG;
    }
    const int xs = elem_size(x_dtype);
    if (!elements_aligned({{dy, elem_size(y_dtype)}, {dres, xs}, {dx, xs}, {gamma, elem_size(param_dtype)}, {mean, 4},
                           {rstd, 4}, {dgamma, 4}, {dbeta, 4}}))
        return GBNORM_ERR_INVALID_ARG;
    HostDevice d;
    int s = host_device(&d);
    size_t need = 0;
    if (s == GBNORM_OK) s = bwd_ws_bytes(is_layernorm, M, N, d, &need);
    const Span outs[4] = {rows(dx, M, N, lddx, xs, true), flat(dgamma, N, 4), flat(dbeta, N, 4),
                          flat(M > 0 ? workspace : nullptr, (int64_t)need, 1)};
    const Span ins[7] = {rows(dy, M, N, lddy, elem_size(y_dtype), true), rows(dres, M, N, lddres, xs, true),
                         rows(codes, M, N, ldc, 1, false), flat(c_scale, M > 0 ? (M - 1) * ldcs + pairs : 0, 4),
                         flat(gamma, N, elem_size(param_dtype)), flat(rstd, M, 4), flat(mean, M, 4)};
    if (bad_aliasing(outs, 4, ins, 7)) return GBNORM_ERR_INVALID_ARG;
    if (s != GBNORM_OK) return s;
    t_last[1] = "";
    int64_t P = 0;
    if (M > 0) {
        if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return GBNORM_ERR_WORKSPACE;
        Q8BwdParams p{dy, reinterpret_cast<const uint8_t *>(codes), c_scale, dres, gamma, mean, rstd, dx,
                      static_cast<float *>(workspace), lddy, ldc, ldcs, lddres, lddx, M, N, x_dtype, param_dtype,
                      y_dtype, cg};
        const int ys = elem_size(y_dtype);
        const bool vec = N % 8 == 0 && vec_rows(dy, lddy, ys) && vec_rows(dres, lddres, xs) && vec_rows(dx, lddx, xs) &&
                         aligned(gamma, 16) && aligned(codes, 8) && ldc % 8 == 0;
        BwdPlan pl;
        int st = bwd_plan(is_layernorm, !vec ? 4 : x_dtype == y_dtype ? x_dtype : 3, M, N, d, &pl);
        if (st != GBNORM_OK) return st;
        P = pl.P;
        t_last[1] = pl.v ? pl.v->name : "elem";
        st = pl.v ? launch_rows(*pl.v, P, &p, stream)
                  : launch(kQ8BwdElem[is_layernorm], P, kElemCTA, 0, &p, stream);
        if (st != GBNORM_OK) return st;
    }
    return host_colreduce(is_layernorm, static_cast<const float *>(workspace), P, N, dgamma, dbeta, M > 0, stream);
}

int q8_read(int64_t M, int64_t N, const void *q, int64_t ldq, int q_format, int q_group, const float *scale,
            const float *mid, int64_t s_row, int64_t s_group, const float *mean, const float *rstd, const void *gamma,
            const void *beta, int param_dtype, void *y, int64_t ldy, int y_dtype, gbnorm_stream_t stream) {
    const int qg = group_log2(q_group);
    if (!valid_shape(M, N) || qg == -2 || !valid_dtype(param_dtype) || !valid_dtype(y_dtype) ||
        (q_format != GBNORM_E4M3 && q_format != GBNORM_INT8))
        return GBNORM_ERR_INVALID_ARG;
    int64_t sspan = 0;
    if (M > 0) {
        if (!q || !scale || !y || !aligned(scale, 4) || !aligned(mid, 4) || !valid_ld(ldq, N, M) ||
            !valid_ld(ldy, N, M))
            return GBNORM_ERR_INVALID_ARG;
        sspan = scale_span(M, groups_of(N, qg), s_row, s_group);
        if (sspan == 0) return GBNORM_ERR_INVALID_ARG;
    }
    const int ps = elem_size(param_dtype);
    if (!elements_aligned({{y, elem_size(y_dtype)}, {gamma, ps}, {beta, ps}, {mean, 4}, {rstd, 4}}))
        return GBNORM_ERR_INVALID_ARG;
    const Span outs[1] = {rows(y, M, N, ldy, elem_size(y_dtype), false)};
    const Span ins[7] = {rows(q, M, N, ldq, 1, false), flat(scale, sspan, 4), flat(mid, sspan, 4), flat(mean, M, 4),
                         flat(rstd, M, 4), flat(gamma, N, ps), flat(beta, N, ps)};
    if (bad_aliasing(outs, 1, ins, 7)) return GBNORM_ERR_INVALID_ARG;
    HostDevice d;
    const int s = host_device(&d);
    if (s != GBNORM_OK) return s;
    t_last[2] = "";
    if (M == 0) return GBNORM_OK;
    Q8ReadParams p{static_cast<const uint8_t *>(q), scale, mid, mean, rstd, gamma, beta, y, ldq, s_row, s_group, ldy,
                   M, N, param_dtype, y_dtype, q_format, qg};
    const bool norm = mean || rstd || gamma || beta;
    const bool vec = N % 8 == 0 && aligned(q, 8) && ldq % 8 == 0 && vec_rows(y, ldy, elem_size(y_dtype)) &&
                     aligned(gamma, 16) && aligned(beta, 16);
    // column blocks of equal width, as many rows side by side as fit
    const int64_t nc = vec ? N / 8 : (N + 255) / 256, most = vec ? kQ8ReadCTA : kElemCTA / 32;
    const int64_t gx = (nc + most - 1) / most;
    int wide = (int)((nc + gx - 1) / gx);
    const int64_t ry = most / wide, rows = ry * (vec ? kQ8ReadRows : 1);
    int64_t gy = grid_of((M + rows - 1) / rows * gx, 8, d) / gx;
    gy = gy < 1 ? 1 : gy > 65535 ? 65535 : gy;
    const bool pair = mid == scale + 1 && s_row % 2 == 0 && s_group % 2 == 0 && aligned(scale, 8);
    const void *kernel = vec ? kQ8Read[q_format][norm][pair][y_dtype] : kQ8ReadAny[norm];
    void *args[2] = {&p, &wide};
    t_last[2] = vec ? "vec" : "any";
    if (cudaLaunchKernel(kernel, dim3((unsigned)gx, (unsigned)gy), dim3((unsigned)(wide * ry * (vec ? 1 : 32))), args, 0,
                         stream) != cudaSuccess)
        return GBNORM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? GBNORM_OK : GBNORM_ERR_CUDA;
}

int gbnorm_q8_last_variant(int what, char *buf, size_t len) {
    if (what < 0 || what > 2 || !buf || len == 0) return GBNORM_ERR_INVALID_ARG;
    std::snprintf(buf, len, "%s", t_last[what]);
    return GBNORM_OK;
}

}  // extern "C"
