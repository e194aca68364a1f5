// rope_api.cu -- the C ABI of the head operators (include/gbnorm.h): argument
// checks, the choice of a kernel, launches.  As in api.cu nothing here
// allocates device memory or synchronises.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>

#include <cuda_runtime.h>

#include "../../include/gbnorm.h"
#include "host_shared.h"
#include "rope_params.h"

namespace gbn {
namespace {

int elem_size(int dtype) { return dtype == GBNORM_F32 ? 4 : 2; }
bool valid_dtype(int d) { return d == GBNORM_F32 || d == GBNORM_F16 || d == GBNORM_BF16; }
bool aligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Most CTAs an SM of the backward: bounds its partial rows, so that the
// workspace depends on the shape alone.
constexpr int64_t kBwdPerSm = 2;

// A tensor of heads as the aliasing check sees it, in bytes: runs of `run`
// bytes at p + i0 st[0] + i1 st[1] + i2 st[2], i < n; extents of one element
// have stride 0.
struct Box {
    uintptr_t p;
    int64_t run, n[3], st[3];
    int es;
    int64_t span() const {
        int64_t s = run;
        for (int i = 0; i < 3; ++i) s += (n[i] - 1) * st[i];
        return s;
    }
};

constexpr int64_t kMostBytes = INT64_MAX / 16;

// False if a stride is negative or the tensor's bytes do not fit.
bool make_box(const gbnorm_heads_t &h, int64_t B, int64_t S, int64_t H, int64_t D, int dtype, Box *out) {
    const int es = elem_size(dtype);
    *out = Box{reinterpret_cast<uintptr_t>(h.p), D * es, {B, S, H}, {h.batch, h.token, h.head}, es};
    int64_t left = kMostBytes - out->run;
    for (int i = 0; i < 3; ++i) {
        if (out->n[i] <= 1) {
            out->st[i] = 0;
            continue;
        }
        if (out->st[i] < 0 || out->st[i] > left / es / (out->n[i] - 1)) return false;
        out->st[i] *= es;
        left -= (out->n[i] - 1) * out->st[i];
    }
    return true;
}

bool same(const Box &a, const Box &b) {
    return a.p == b.p && a.es == b.es && a.run == b.run && !std::memcmp(a.st, b.st, sizeof a.st) &&
           !std::memcmp(a.n, b.n, sizeof a.n);
}

// No two elements in one place: each stride passes all that the smaller ones span.
bool injective(const Box &a) {
    int o[3] = {0, 1, 2};
    std::sort(o, o + 3, [&](int i, int j) { return a.st[i] < a.st[j]; });
    int64_t inner = a.run;
    for (int i : o) {
        if (a.n[i] <= 1) continue;
        if (a.st[i] < inner) return false;
        inner += (a.n[i] - 1) * a.st[i];
    }
    return true;
}

// The bytes a box covers in each period of `per` bytes, 0 if it does not repeat with that period.
int64_t window(const Box &a, int64_t per) {
    int64_t w = a.run;
    for (int i = 0; i < 3; ++i)
        if (a.n[i] > 1 && a.st[i] % per != 0) w += (a.n[i] - 1) * a.st[i];
    return w <= per ? w : 0;
}

// May the two share a byte?  Spans apart: no.  Else both may be parts of one
// larger tensor (queries and keys within a packed projection): if they repeat
// with a common period and cover different parts of it, no.
bool may_overlap(const Box &a, const Box &b) {
    if (!a.p || !b.p) return false;
    if (a.p + (uintptr_t)a.span() <= b.p || b.p + (uintptr_t)b.span() <= a.p) return false;
    for (const Box *x : {&a, &b})
        for (int i = 0; i < 3; ++i) {
            const int64_t per = x->st[i];
            if (x->n[i] <= 1 || per <= 0) continue;
            const int64_t wa = window(a, per), wb = window(b, per);
            if (!wa || !wb) continue;
            const uintptr_t u = (uintptr_t)per;
            const int64_t d = (int64_t)((b.p % u + u - a.p % u) % u);
            if (d >= wa && per - d >= wb) return false;
        }
    return true;
}

Box flat(const void *p, int64_t bytes) {
    return Box{bytes > 0 ? reinterpret_cast<uintptr_t>(p) : 0, bytes, {1, 1, 1}, {0, 0, 0}, 1};
}

struct Shape {
    int64_t B, S, H[2], D;
    int64_t tokens() const { return B * S; }
    int tensors() const { return H[1] > 0 ? 2 : 1; }
};

constexpr int64_t kMostTokens = (int64_t)1 << 40;

bool valid_heads(const Shape &s) {
    return s.H[0] >= 1 && s.H[1] >= 0 && s.H[0] <= GBNORM_MAX_HEADS && s.H[1] <= GBNORM_MAX_HEADS && s.D >= 1 &&
           s.D <= kRopeMaxDim;
}
bool valid_shape(const Shape &s) {
    if (!valid_heads(s) || s.B < 0 || s.S < 0) return false;
    return s.B <= INT32_MAX && s.S <= INT32_MAX && s.tokens() <= kMostTokens;
}

// Checks what every call has and fills the parameters that do not depend on the direction.
int common(const gbnorm_rope_t *r, bool need_rotation, Shape *s, RopeParams *p) {
    if (!r) return GBNORM_ERR_INVALID_ARG;
    *s = Shape{r->batches, r->tokens, {r->heads[0], r->heads[1]}, r->dim};
    if (!valid_shape(*s) || !valid_dtype(r->x_dtype) || !valid_dtype(r->y_dtype) || !valid_dtype(r->param_dtype))
        return GBNORM_ERR_INVALID_ARG;
    if (r->rot < (need_rotation ? 2 : 0) || r->rot > s->D || r->rot % 2 != 0 ||
        (r->interleaved != 0 && r->interleaved != 1))
        return GBNORM_ERR_INVALID_ARG;
    std::memset(p, 0, sizeof *p);
    p->B = s->B;
    p->S = s->S;
    p->heads[0] = (int)s->H[0];
    p->heads[1] = (int)s->H[1];
    p->D = (int)s->D;
    p->rot = r->rot;
    p->inter = r->interleaved;
    p->xdt = r->x_dtype;
    p->ydt = r->y_dtype;
    p->pdt = r->param_dtype;
    p->sign = 1.f;
    if (r->rot == 0) return GBNORM_OK;
    if (r->axes < 1 || r->axes > kRopeMaxAxes || (r->pos_dtype != GBNORM_I32 && r->pos_dtype != GBNORM_I64) ||
        (r->axes > 1 && !r->pair_axis) || !r->inv_freq || !aligned(r->inv_freq, 4))
        return GBNORM_ERR_INVALID_ARG;
    const int ps = r->pos_dtype == GBNORM_I64 ? 8 : 4;
    if (s->tokens() > 0 && (!r->positions || !aligned(r->positions, ps))) return GBNORM_ERR_INVALID_ARG;
    const int64_t n[3] = {r->axes, s->B, s->S}, st[3] = {r->pos_axis, r->pos_batch, r->pos_token};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] < 0 || st[i] > kMostBytes / 64 / n[i])) return GBNORM_ERR_INVALID_ARG;
    p->pos = r->positions;
    p->pos64 = ps == 8;
    p->axes = r->axes;
    p->pos_axis = r->axes > 1 ? r->pos_axis : 0;
    p->pos_batch = s->B > 1 ? r->pos_batch : 0;
    p->pos_token = s->S > 1 ? r->pos_token : 0;
    p->inv_freq = r->inv_freq;
    if (r->pair_axis)
        for (int j = 0; j < r->rot / 2; ++j) {
            if (r->pair_axis[j] >= r->axes) return GBNORM_ERR_INVALID_ARG;
            p->axis[j / 16] |= (uint32_t)r->pair_axis[j] << (2 * (j % 16));
        }
    return GBNORM_OK;
}

// The rows of heads of one side of a call (x, y or dy): checked and stored.
int take(const gbnorm_heads_t *h, const Shape &s, int dtype, bool out, RopeHeads *to, Box *box) {
    for (int i = 0; i < 2; ++i) {
        box[i] = flat(nullptr, 0);
        to[i] = RopeHeads{nullptr, 0, 0, 0};
        if (i >= s.tensors() || s.tokens() == 0) continue;
        if (!h || !h[i].p || !aligned(h[i].p, (unsigned)elem_size(dtype)) ||
            !make_box(h[i], s.B, s.S, s.H[i], s.D, dtype, &box[i]) || (out && !injective(box[i])))
            return GBNORM_ERR_INVALID_ARG;
        const int es = elem_size(dtype);
        to[i] = RopeHeads{h[i].p, box[i].st[0] / es, box[i].st[1] / es, box[i].st[2] / es};
    }
    return GBNORM_OK;
}

// Bytes that the positions span.
int64_t pos_bytes(const RopeParams &p) {
    if (!p.pos || p.B * p.S == 0) return 0;
    return ((p.axes - 1) * p.pos_axis + (p.B - 1) * p.pos_batch + (p.S - 1) * p.pos_token + 1) * (p.pos64 ? 8 : 4);
}

// outs may overlap nothing, except that outs[i] may be exactly ins[i] for i < same_n.
bool bad_aliasing(const Box *outs, int no, const Box *ins, int ni, int same_n) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j) {
            if (i == j && i < same_n && same(outs[i], ins[j])) continue;
            if (may_overlap(outs[i], ins[j])) return true;
        }
        for (int j = i + 1; j < no; ++j)
            if (may_overlap(outs[i], outs[j])) return true;
    }
    return false;
}

thread_local const char *t_last[3] = {"", "", ""};

// Passes of `at_once` heads, shared out over a grid of at most per_sm CTAs an
// SM: one pass a warp where that is few enough.  Returns the CTAs, -1 if a
// warp's passes do not fit its counter.
int64_t share(RopeParams *p, const Shape &s, int64_t at_once, int64_t per_sm, const HostDevice &d) {
    int64_t cap = per_sm * d.sms;
    const int64_t limit = host_grid_limit();
    if (limit > 0 && limit < cap) cap = limit;
    p->units = 0;
    for (int i = 0; i < 2; ++i) {
        p->passes[i] = (int)((s.H[i] + at_once - 1) / at_once);
        p->units += s.tokens() * p->passes[i];
    }
    p->warps = std::min(p->units, cap * kRopeWarps);
    if (p->units / p->warps >= INT32_MAX) return -1;
    // whole tokens as a front (prefill of 16384 tokens 62 -> 57 us, backward 97 -> 88 us) where a warp has four or
    // more; below, the uneven rest costs more than the order gives (8192 tokens rotated: 21.7 us without, 23.0 us with)
    const int64_t rounds = s.tokens() / p->warps;
    p->rounds = rounds < 4 ? 0 : (int)rounds;
    p->step_b = (int)(p->warps / s.S);
    p->step_s = (int)(p->warps % s.S);
    return (p->warps + kRopeWarps - 1) / kRopeWarps;
}

int launch(const void *kernel, int64_t grid, size_t dyn, RopeParams *p, cudaStream_t st) {
    void *args[1] = {p};
    if (cudaLaunchKernel(kernel, dim3((unsigned)grid), dim3(kRopeCTA), args, dyn, st) != cudaSuccess)
        return GBNORM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? GBNORM_OK : GBNORM_ERR_CUDA;
}

// A kernel of a call.
struct Kernel {
    const void *f;
    const char *name;
    int heads;  // of a pass
    int smem;
    int slot;   // its place in the cache of what a device holds
};

// Column sums of the P partial rows into dgamma and dbeta (0 rows: zeros).  The
// launch may begin while the rows' kernel drains; it waits for that before it reads.
int columns(int is_ln, const float *ws, int P, int N, float *dgamma, float *dbeta, cudaStream_t st) {
    if (!dgamma && !dbeta) return GBNORM_OK;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)((N + 31) / 32), is_ln ? 2u : 1u);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = P > 0 ? 1 : 0;
    void *args[5] = {&ws, &P, &N, &dgamma, &dbeta};
    if (cudaLaunchKernelExC(&cfg, kRopeColumns, args) != cudaSuccess) return GBNORM_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? GBNORM_OK : GBNORM_ERR_CUDA;
}

int any_size(int D, int rot) {  // 32 << that pairs hold a head
    const int pairs = rot / 2 + (D - rot + 1) / 2;
    int lg = 0;
    while (32 << lg < pairs) ++lg;
    return lg;
}

constexpr int kVecTypes = 9;  // fp32, fp16, bf16 by two, by four, differing types by four, fp16, bf16 by eight

// Elements of the vectors that all tensors of a call move as: every head and
// chunk starts on a vector, the rotated part holds whole ones.  0: none.
int vector_of(const RopeParams &p, bool back) {
    const int xs = elem_size(p.xdt), ys = elem_size(p.ydt);
    const struct {
        const RopeHeads *t;
        int es;
    } all[3] = {{p.x, xs}, {p.y, back ? xs : ys}, {back ? p.g : p.x, back ? ys : xs}};
    for (int v = p.xdt == p.ydt && xs == 2 ? 8 : 4; v >= (p.xdt == p.ydt ? 2 : 4); v /= 2) {
        bool ok = p.D % v == 0 && (p.inter ? p.rot % v : p.rot / 2 % v) == 0;
        for (const auto &a : all)
            for (int i = 0; i < 2; ++i) {
                const RopeHeads &t = a.t[i];
                ok = ok && aligned(t.p, (unsigned)(v * a.es)) && (t.batch | t.token | t.head) % v == 0 &&
                     ((t.batch | t.token | t.head) / v) >> 32 == 0;
            }
        if (ok) return v;
    }
    return 0;
}

// mode: a RopeMode, or -1 - is_layernorm for the backward.  Strides become those of the kernel's kind.
Kernel pick(int mode, RopeParams &p) {
#define GBN_T(M) \
    {kRopeVec_##M##_f32v2, kRopeVec_##M##_f16v2, kRopeVec_##M##_bf16v2, kRopeVec_##M##_f32v4, kRopeVec_##M##_f16v4, \
     kRopeVec_##M##_bf16v4, kRopeVec_##M##_mixv4, kRopeVec_##M##_f16v8, kRopeVec_##M##_bf16v8}
    static const RopeVariant(*const tables[5][kVecTypes])[kRopeVecLanes] = {GBN_T(rot), GBN_T(rms), GBN_T(ln),
                                                                            GBN_T(brms), GBN_T(bln)};
#undef GBN_T
    const int v = vector_of(p, mode < 0), m = mode < 0 ? 2 - mode : mode;
    if (v) {
        const int chunks = p.D / v, rot = p.rot / v;
        const int slots = p.inter ? (chunks + 1) / 2 : rot / 2 + (chunks - rot + 1) / 2;
        const int kind = p.rot == p.D ? p.inter : 2;  // as RopeKind
        const int t = p.xdt != p.ydt ? 6 : p.xdt + (v == 2 ? 0 : v == 4 ? 3 : 6);
        const int c = p.xdt == p.ydt && p.xdt == GBNORM_F32 ? 4 / v : 8 / v;  // slots a lane
        for (int l = 0; l < kRopeVecLanes; ++l)
            if (slots <= kRopeLaneCounts[l] * c) {
                const RopeVariant &k = tables[m][t][kind][l];
                for (RopeHeads *h : {p.x, p.y, p.g})
                    for (int i = 0; i < 2; ++i) {
                        h[i].batch /= v;
                        h[i].token /= v;
                        h[i].head /= v;
                    }
                // gamma (and beta) of both tensors as fp32 behind the rings
                const int par = mode == kRopeOnly ? 0 : mode == kRopeLn ? 16 * p.D : 8 * p.D;
                return {k.f, k.name, 32 / k.lanes * k.u, k.smem + par,
                        ((m * kVecTypes + t) * kRopeVecKinds + kind) * kRopeVecLanes + l};
            }
    }
    const int n = any_size(p.D, p.rot), slot = 5 * kVecTypes * kRopeVecKinds * kRopeVecLanes + m * kRopeAnySizes + n;
    const RopeVariant &k = mode < 0 ? kRopeBwdAny[-1 - mode][n] : kRopeFwdAny[mode][n];
    return {k.f, k.name, 32 / k.lanes, k.smem + (mode < 0 ? kRopeWarps * p.D * 4 : 0), slot};
}
constexpr int kSlots = 5 * kVecTypes * kRopeVecKinds * kRopeVecLanes + 5 * kRopeAnySizes;
std::atomic<int> g_resident[kHostMaxDev][kSlots];

// CTAs of a kernel that an SM holds, measured once per device.
int resident(const Kernel &k, const HostDevice &d, int *out) {
    std::atomic<int> &c = g_resident[d.dev][k.slot];
    int o = c.load(std::memory_order_relaxed);
    if (o == 0) {
        // heads of several sizes share a kernel: allow for the parameters (8 KB) or column sums (32 KB) of any
        if (cudaFuncSetAttribute(k.f, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem + 32 * 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, k.f, kRopeCTA, (size_t)k.smem) != cudaSuccess)
            return GBNORM_ERR_CUDA;
        if (o <= 0) return GBNORM_ERR_UNSUPPORTED;
        c.store(o, std::memory_order_relaxed);
    }
    *out = o;
    return GBNORM_OK;
}

// Forward kernels: the norm with the rotation (mode kRopeRms, kRopeLn), the rotation alone.
int run_fwd(int mode, RopeParams *p, const Shape &s, cudaStream_t st) {
    const int what = mode == kRopeOnly ? 2 : 0;
    HostDevice d;
    const int e = host_device(&d);
    if (e != GBNORM_OK) return e;
    t_last[what] = "";
    if (s.tokens() == 0) return GBNORM_OK;
    const Kernel k = pick(mode, *p);
    int per_sm;
    const int o = resident(k, d, &per_sm);
    if (o != GBNORM_OK) return o;
    const int64_t grid = share(p, s, k.heads, per_sm, d);
    if (grid < 0) return GBNORM_ERR_UNSUPPORTED;
    t_last[what] = k.name;
    return launch(k.f, grid, (size_t)k.smem, p, st);
}

int64_t bwd_rows(const Shape &s, const HostDevice &d) {  // most partial rows of any kernel
    const int64_t units = s.tokens() * (s.H[0] + s.H[1]), cap = kBwdPerSm * d.sms;
    return std::min(cap, (units + kRopeWarps - 1) / kRopeWarps);
}
size_t bwd_ws(int is_ln, const Shape &s, const HostDevice &d) {
    const size_t b = (size_t)bwd_rows(s, d) * (size_t)s.D * (size_t)s.tensors() * 4u * (is_ln ? 2u : 1u);
    return (b + 255u) & ~(size_t)255u;
}

int rotate(const gbnorm_rope_t *r, const gbnorm_heads_t *x, const gbnorm_heads_t *y, bool back, cudaStream_t stream) {
    Shape s;
    RopeParams p;
    int e = common(r, true, &s, &p);
    if (e != GBNORM_OK) return e;
    if (back) {
        std::swap(p.xdt, p.ydt);
        p.sign = -1.f;
    }
    Box in[4], out[2];
    if ((e = take(x, s, p.xdt, false, p.x, in)) != GBNORM_OK) return e;
    if ((e = take(y, s, p.ydt, true, p.y, out)) != GBNORM_OK) return e;
    in[2] = flat(p.pos, pos_bytes(p));
    in[3] = flat(p.inv_freq, 2 * p.rot);
    if (bad_aliasing(out, 2, in, 4, 2)) return GBNORM_ERR_INVALID_ARG;
    return run_fwd(kRopeOnly, &p, s, stream);
}

}  // namespace
}  // namespace gbn

using namespace gbn;

extern "C" {

int qk_norm_rope_fwd(int is_layernorm, float eps, const gbnorm_rope_t *r, const gbnorm_heads_t *x,
                     const gbnorm_heads_t *y, const void *const *gamma, const void *const *beta, float *mean,
                     float *rstd, gbnorm_stream_t stream) {
    Shape s;
    RopeParams p;
    if ((is_layernorm != 0 && is_layernorm != 1) || !std::isfinite(eps) || eps < 0.f) return GBNORM_ERR_INVALID_ARG;
    int e = common(r, false, &s, &p);
    if (e != GBNORM_OK) return e;
    if (!is_layernorm) {
        beta = nullptr;
        mean = nullptr;
    }
    Box in[8], out[4];
    if ((e = take(x, s, p.xdt, false, p.x, in)) != GBNORM_OK) return e;
    if ((e = take(y, s, p.ydt, true, p.y, out)) != GBNORM_OK) return e;
    const int ps = elem_size(p.pdt);
    for (int i = 0; i < 2; ++i) {
        p.gamma[i] = gamma && i < s.tensors() ? gamma[i] : nullptr;
        p.beta[i] = beta && i < s.tensors() ? beta[i] : nullptr;
        if (!aligned(p.gamma[i], (unsigned)ps) || !aligned(p.beta[i], (unsigned)ps)) return GBNORM_ERR_INVALID_ARG;
        in[4 + i] = flat(p.gamma[i], s.D * ps);
        in[6 + i] = flat(p.beta[i], s.D * ps);
    }
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return GBNORM_ERR_INVALID_ARG;
    in[2] = flat(p.pos, pos_bytes(p));
    in[3] = flat(p.inv_freq, 2 * p.rot);
    const int64_t stats = s.tokens() * (s.H[0] + s.H[1]) * 4;
    out[2] = flat(mean, stats);
    out[3] = flat(rstd, stats);
    if (bad_aliasing(out, 4, in, 8, 2)) return GBNORM_ERR_INVALID_ARG;
    p.mean = mean;
    p.rstd = rstd;
    p.eps = eps;
    return run_fwd(is_layernorm ? kRopeLn : kRopeRms, &p, s, stream);
}

size_t qk_norm_rope_bwd_workspace_size(int is_layernorm, int64_t tokens, int64_t heads_q, int64_t heads_k,
                                       int64_t dim) {
    const Shape s{1, tokens, {heads_q, heads_k}, dim};  // of all batches: more than one may hold
    HostDevice d;
    if ((is_layernorm != 0 && is_layernorm != 1) || !valid_heads(s) || tokens < 0 || tokens > kMostTokens ||
        host_device(&d) != GBNORM_OK)
        return 0;
    const size_t need = bwd_ws(is_layernorm, s, d);
    return need > 0 ? need : 256;  // no tokens: nothing is used; 0 means an error
}

int qk_norm_rope_bwd(int is_layernorm, const gbnorm_rope_t *r, const gbnorm_heads_t *dy, const gbnorm_heads_t *x,
                     const gbnorm_heads_t *dx, const void *const *gamma, const float *mean, const float *rstd,
                     float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes, gbnorm_stream_t stream) {
    Shape s;
    RopeParams p;
    if (is_layernorm != 0 && is_layernorm != 1) return GBNORM_ERR_INVALID_ARG;
    int e = common(r, false, &s, &p);
    if (e != GBNORM_OK) return e;
    if (!is_layernorm) {
        dbeta = nullptr;
        mean = nullptr;
    }
    Box in[10], out[5];
    if ((e = take(dy, s, p.ydt, false, p.g, in)) != GBNORM_OK) return e;
    if ((e = take(x, s, p.xdt, false, p.x, in + 2)) != GBNORM_OK) return e;
    if ((e = take(dx, s, p.xdt, true, p.y, out)) != GBNORM_OK) return e;
    if (s.tokens() > 0 && (!rstd || (is_layernorm && !mean))) return GBNORM_ERR_INVALID_ARG;
    const int ps = elem_size(p.pdt);
    for (int i = 0; i < 2; ++i) {
        p.gamma[i] = gamma && i < s.tensors() ? gamma[i] : nullptr;
        if (!aligned(p.gamma[i], (unsigned)ps)) return GBNORM_ERR_INVALID_ARG;
        in[4 + i] = flat(p.gamma[i], s.D * ps);
    }
    for (const void *v : {(const void *)mean, (const void *)rstd, (const void *)dgamma, (const void *)dbeta})
        if (!aligned(v, 4)) return GBNORM_ERR_INVALID_ARG;
    const int64_t stats = s.tokens() * (s.H[0] + s.H[1]) * 4, N = s.D * s.tensors();
    in[6] = flat(mean, stats);
    in[7] = flat(rstd, stats);
    in[8] = flat(p.pos, pos_bytes(p));
    in[9] = flat(p.inv_freq, 2 * p.rot);
    HostDevice d;
    e = host_device(&d);
    const size_t need = e == GBNORM_OK ? bwd_ws(is_layernorm, s, d) : 0;
    out[2] = flat(dgamma, N * 4);
    out[3] = flat(dbeta, N * 4);
    out[4] = flat(workspace, (int64_t)need);
    if (bad_aliasing(out, 5, in, 10, 2)) return GBNORM_ERR_INVALID_ARG;
    if (e != GBNORM_OK) return e;
    t_last[1] = "";
    int64_t P = 0;
    if (s.tokens() > 0) {
        if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return GBNORM_ERR_WORKSPACE;
        p.mean = const_cast<float *>(mean);
        p.rstd = const_cast<float *>(rstd);
        p.ws = static_cast<float *>(workspace);
        p.sign = -1.f;
        const Kernel k = pick(-1 - is_layernorm, p);
        int per_sm;
        if ((e = resident(k, d, &per_sm)) != GBNORM_OK) return e;
        P = share(&p, s, k.heads, std::min<int64_t>(per_sm, kBwdPerSm), d);
        if (P < 0) return GBNORM_ERR_UNSUPPORTED;
        t_last[1] = k.name;
        e = launch(k.f, P, (size_t)k.smem, &p, stream);
        if (e != GBNORM_OK) return e;
    }
    return columns(is_layernorm, static_cast<const float *>(workspace), (int)P, (int)N, dgamma, dbeta, stream);
}

int rope_fwd(const gbnorm_rope_t *r, const gbnorm_heads_t *x, const gbnorm_heads_t *y, gbnorm_stream_t stream) {
    return rotate(r, x, y, false, stream);
}

int rope_bwd(const gbnorm_rope_t *r, const gbnorm_heads_t *dy, const gbnorm_heads_t *dx, gbnorm_stream_t stream) {
    return rotate(r, dy, dx, true, stream);
}

int gbnorm_rope_last_variant(int what, char *buf, size_t len) {
    if (what < 0 || what > 2 || !buf || len == 0) return GBNORM_ERR_INVALID_ARG;
    std::snprintf(buf, len, "%s", t_last[what]);
    return GBNORM_OK;
}

}  // extern "C"
