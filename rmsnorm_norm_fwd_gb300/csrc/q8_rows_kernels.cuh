// q8_rows_kernels.cuh -- forward of the 8-bit operators with rows in
// registers: a row group of TPR threads holds one row, each thread VPT chunks
// of 8 consecutive elements, chunk k * TPR + t.
//
// What bounds it: DRAM.  A row is read once and written once (bf16: 2 + 1
// bytes an element, 7 with a residual sum); per element the arithmetic is a
// few operations on fp32 pairs.  Measured, bf16, share of the copy rate's time:
// RMSNorm 16384 x 8192 with a residual 150 us (92%), without 65 us (91%), group
// scales 16384 x 4096 36 us (84%); fp32 rows of 8192 102 us (97%).  LayerNorm
// 16384 x 8192 with group scales 82 us (73%): 15.6 instructions an element
// against 10.4, issue at 61% and DRAM at 39%, so latency too: a row group waits
// for its own loads and two exchanges with nothing of its next row in flight but
// the prefetch.  The same for clusters: 1024 x 65536 49 us (61%), issue at 44%.
//
//   - A chunk is 16 bytes of a 16-bit type in and 8 codes out, so a group of
//     32..256 columns is 4..32 consecutive lanes of a warp: its maxima are a
//     lane butterfly, without shared memory.
//   - RMSNorm's codes are those of h * gamma (rstd cancels): with group scales
//     they are written before the row's sum is known, with row scales the sum
//     and the maximum are one reduction with one barrier.
//   - The checkpoint's codes need h alone and are written before the
//     statistics too.
//   - A thread holds 8 to 32 elements, so that four 256-thread CTAs share an SM
//     (three where LayerNorm keeps gamma and beta as fp32) and their phases overlap.
//   - Rows longer than one CTA holds are split over a cluster of 2 to 8 CTAs,
//     which exchange the row's sums through distributed shared memory.
//   - Every thread keeps gamma (beta) of its own columns in its own slots of
//     shared memory, as fp32: no conversion, no branch on the parameter type and
//     no barrier in the loop.  LayerNorm with 16-bit gamma and beta of the rows'
//     type keeps them so and widens them at each use: that leaves room for the
//     fourth CTA (16384 x 8192: 82 us against 90 us with fp32 ones).
#pragma once

#include <type_traits>

#include "q8_common.cuh"

namespace gbn {

// Element type by code, for conversions resolved at compile time.
template <int XT> struct TypeOf;
template <> struct TypeOf<kF32> { using T = float; };
template <> struct TypeOf<kF16> { using T = __half; };
template <> struct TypeOf<kBF16> { using T = __nv_bfloat16; };

// A chunk of 8 elements as it is stored.
template <int XT> struct Raw8 {
    uint4 v[XT == kF32 ? 2 : 1];
};
// Chunk c of a row that nothing of this launch writes to the same place
// before it is read (rows may be overwritten in place, by the thread that
// read them), through L2 only: no row is read twice.
template <int XT> __device__ __forceinline__ Raw8<XT> ld_raw8(const void *row, int64_t c) {
    constexpr int W = XT == kF32 ? 2 : 1;
    Raw8<XT> r;
    const uint4 *p = static_cast<const uint4 *>(row) + c * W;
#pragma unroll
    for (int w = 0; w < W; ++w)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.v[w].x), "=r"(r.v[w].y), "=r"(r.v[w].z), "=r"(r.v[w].w)
                     : "l"(p + w));
    return r;
}
template <int XT> __device__ __forceinline__ void unpack8(const Raw8<XT> &r, float2 (&f)[4]) {
    using T = typename TypeOf<XT>::T;
    constexpr int PW = XT == kF32 ? 2 : 4;  // pairs per 16 bytes
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = vpair<T>(r.v[i / PW], i % PW);
}
// Bytes (a multiple of 16, 16-byte aligned) brought to L2; nothing waits for them.
__device__ __forceinline__ void prefetch_l2(const void *p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// Chunk c of a parameter row (read-only, kept in L1), or the constant an
// absent one stands for.
__device__ __forceinline__ void par8g(const void *row, int64_t c, int dt, float absent, float2 (&f)[4]) {
    if (row == nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f2s(absent);
    } else if (dt == kF32) {
        const uint4 a = ld_vec(row, 2 * c), b = ld_vec(row, 2 * c + 1);
        f[0] = vpair<float>(a, 0), f[1] = vpair<float>(a, 1);
        f[2] = vpair<float>(b, 0), f[3] = vpair<float>(b, 1);
    } else {
        const uint4 a = ld_vec(row, c);
        if (dt == kBF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = vpair<__nv_bfloat16>(a, i);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = vpair<__half>(a, i);
        }
    }
}

template <int XT> __device__ __forceinline__ Raw8<XT> pack8(const float2 (&f)[4]) {
    using T = typename TypeOf<XT>::T;
    Raw8<XT> r;
    r.v[0] = vpack2<T>(f);
    if constexpr (XT == kF32) r.v[1] = vpack2<T>(f + 2);
    return r;
}
template <int XT> __device__ __forceinline__ void st_raw8(void *row, int64_t c, const Raw8<XT> &r) {
    constexpr int W = XT == kF32 ? 2 : 1;
#pragma unroll
    for (int w = 0; w < W; ++w) st_vec(row, c * W + w, r.v[w]);
}

// max(|a|, |b|, m) and max / min of three, NaN kept.
__device__ __forceinline__ float amax3(float m, float2 f) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(f.x), "f"(f.y));
    return r;
}
__device__ __forceinline__ float amax8(const float2 (&f)[4]) {
    return fmax_nan(amax3(amax3(0.f, f[0]), f[1]), amax3(amax3(0.f, f[2]), f[3]));
}
// Eight int8 codes of u as two words: rint(u) is the low byte of u + 1.5 *
// 2^23.  The sum is written as u * one + magic with `one` = 1 from the kernel's
// arguments: a plain addition was seen fused with the product that made u, and
// next to a tie the fused form rounds u differently from the two steps that
// define the codes.
__device__ __forceinline__ uint2 codes8_i8(const float2 (&u)[4], float one) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 magic = f2s(12582912.f);
        const float2 a = f2fma(u[2 * i], f2s(one), magic), b = f2fma(u[2 * i + 1], f2s(one), magic);
        const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
        w[i] = __byte_perm(lo, hi, 0x5410);
    }
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint32_t e4m3_quad(float2 a, float2 b) {
    uint32_t w;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(w)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return w;
}
__device__ __forceinline__ uint2 codes8(const float2 (&u)[4], int fmt, float one) {
    if (fmt == kI8) return codes8_i8(u, one);
    return make_uint2(e4m3_quad(u[0], u[1]), e4m3_quad(u[2], u[3]));
}

// Lanes that combine WPR warps' partials in a butterfly (a power of two; the
// same on every warp and, each step being commutative, the same bits on every
// lane).
__host__ __device__ constexpr int pow2_at_least(int v) { return v <= 1 ? 1 : 2 * pow2_at_least((v + 1) / 2); }

// What a row group of TPR threads (CL > 1: in each of the CL CTAs of a cluster)
// reduces through: its scratch of [2][WPR] float4 and, for a cluster, a buffer
// of [2][CL] in every CTA.  Two copies, so that one barrier a reduction
// suffices: it proves that every reader of the copy before last is done.
template <int TPR, int CL> struct RowReduce {
    static constexpr int WPR = TPR / 32, SCRATCH = 2 * WPR + (CL > 1 ? 2 * CL : 0);
    float4 *scratch;
    int parity, bar_id;

    // The partial v of this thread's warp; every thread gets that of warp
    // `lane` modulo the next power of two (zeros past the last warp).
    __device__ __forceinline__ float4 warps(float4 v) {
        constexpr int L = pow2_at_least(WPR);
        const int wig = (threadIdx.x % TPR) >> 5, lane = threadIdx.x & 31;
        float4 *buf = scratch + parity * WPR;
        if (lane == 0) buf[wig] = v;
        named_sync(bar_id, TPR);
        const int w = lane & (L - 1);
        const float4 b = w < WPR ? buf[w] : make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (CL == 1) parity ^= 1;
        return b;
    }
    // The same over the CTAs of the cluster (CL a power of two): each CTA
    // stores its value into every CTA's buffer; that of CTA lane mod CL.
    __device__ __forceinline__ float4 ctas(float4 v) {
        float4 *buf = scratch + 2 * WPR + parity * CL;
        if (threadIdx.x < CL)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                             map_to_rank(smem_u32(buf + cluster_ctarank()), threadIdx.x)),
                         "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                         : "memory");
        cluster_sync_all();
        parity ^= 1;
        return buf[threadIdx.x & (CL - 1)];
    }
};

// Sum over a row group of `s` and maximum (NaN kept) of `m`; the same bits on
// every thread.  Maxima are of magnitudes.
template <int TPR, int CL, bool MAX>
__device__ __forceinline__ void group_sum_max(float &s, float &m, RowReduce<TPR, CL> &rr) {
    auto step = [&](int o) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if constexpr (MAX) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) step(o);
    if constexpr (TPR > 32) {
        const float4 b = rr.warps(make_float4(s, MAX ? m : 0.f, 0.f, 0.f));
        s = b.x;
        if constexpr (MAX) m = b.y;
#pragma unroll
        for (int o = pow2_at_least(TPR / 32) / 2; o > 0; o >>= 1) step(o);
    }
    if constexpr (CL > 1) {
        const float4 b = rr.ctas(make_float4(s, MAX ? m : 0.f, 0.f, 0.f));
        s = b.x;
        if constexpr (MAX) m = b.y;
#pragma unroll
        for (int o = CL / 2; o > 0; o >>= 1) step(o);
    }
}

// Elements that a thread, its warp and its CTA hold of a row: the same for every
// row, so taken once.
struct RowCounts {
    float thread, inv_thread, warp, inv_warp, cta, inv_cta;
};
__device__ __forceinline__ float inv_or_0(float c) { return c > 0.f ? 1.f / c : 0.f; }
__device__ __forceinline__ RowCounts row_counts(int thread, float cta) {
    float w = (float)thread;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return RowCounts{(float)thread, inv_or_0((float)thread), w, inv_or_0(w), cta, inv_or_0(cta)};
}

// Mean and sum of squared deviations of a row from its threads' own (the
// update of Chan, Golub and LeVeque in its group form: over a warp's lanes, the
// warps, the CTAs).  inv_n: 1 / N.  Squares beyond fp32 leave m2 infinite (rstd 0)
// and the mean finite, as long as the sum of the row's magnitudes is inside fp32;
// past that means become infinite and m2 NaN.
template <int TPR, int CL>
__device__ __forceinline__ void group_meanvar(float &mean, float &m2, const RowCounts &cnt, float inv_n,
                                              RowReduce<TPR, CL> &rr) {
    float s = mean * cnt.thread;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mw = s * cnt.inv_warp;
    const float d = mean - mw;
    float q = cnt.thread > 0.f ? m2 + cnt.thread * (d * d) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    mean = mw;
    m2 = q;
    // the parts' (mean, m2, count), one a lane, over L lanes
    auto join = [&](float4 b, int L, float inv) {
        s = b.x * b.z;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < L) s += __shfl_xor_sync(0xffffffffu, s, o);
        mean = s * inv;
        const float dd = b.x - mean;
        m2 = b.z > 0.f ? b.y + b.z * (dd * dd) : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < L) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
    };
    if constexpr (TPR > 32)
        join(rr.warps(make_float4(mean, m2, cnt.warp, 0.f)), pow2_at_least(TPR / 32), CL == 1 ? inv_n : cnt.inv_cta);
    if constexpr (CL > 1) join(rr.ctas(make_float4(mean, m2, cnt.cta, 0.f)), CL, inv_n);
}

// h = x + r rounded once to the storage type.
template <int XT> __device__ __forceinline__ void add8(Raw8<XT> &h, const Raw8<XT> &r) {
    if constexpr (XT == kF32) {
        float2 a[4], b[4];
        unpack8<XT>(h, a);
        unpack8<XT>(r, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = f2add(a[i], b[i]);
        h = pack8<XT>(a);
    } else {
        using T2 = typename std::conditional<XT == kBF16, __nv_bfloat162, __half2>::type;
        T2 *a = reinterpret_cast<T2 *>(&h.v[0]);
        const T2 *b = reinterpret_cast<const T2 *>(&r.v[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = __hadd2_rn(a[i], b[i]);
    }
}

// Each lane has a value for its chunk of VPT groups side by side (chunk k of
// the 2^lg lanes of a group forms one).  max_of_own reduces all VPT at once: in
// the first two steps partner lanes trade halves, so that lane l goes on with
// chunk l mod 4 alone (own_chunk), 5 shuffles for 4 groups of 16 lanes instead
// of 16.  What follows from a maximum (a division) is then done once a lane, and
// the lanes of a group (at least four) fetch the results from one another.
template <int VPT> __device__ __forceinline__ int own_chunk(int lane) {
    return VPT == 1 ? 0 : VPT == 2 ? lane & 1 : lane & 3;
}
template <int VPT, typename V, typename Max>
__device__ __forceinline__ V max_of_own(const V (&a)[VPT], V none, int lane, int lg, Max &&mx) {
    V r;
    int done = 0;  // steps taken
    if constexpr (VPT == 1) {
        r = a[0];
    } else {
        const bool b0 = lane & 1, b1 = lane & 2;
        auto trade = [&](V even, V odd, bool bit, int o) {
            return mx(bit ? odd : even, __shfl_xor_sync(0xffffffffu, bit ? even : odd, o));
        };
        r = trade(a[0], a[1], b0, 1);
        done = 1;
        if constexpr (VPT > 2) {
            V hi;
            if constexpr (VPT == 4) hi = trade(a[2], a[3], b0, 1);
            else hi = trade(a[2], none, b0, 1);
            r = trade(r, hi, b1, 2);
            done = 2;
        }
    }
#pragma unroll
    for (int o = 0; o < 5; ++o)
        if (o >= done && o < lg) r = mx(r, __shfl_xor_sync(0xffffffffu, r, 1 << o));
    return r;
}
template <int VPT> __device__ __forceinline__ float fetch(float own, int lane, int k) {
    return VPT == 1 ? own : __shfl_sync(0xffffffffu, own, (lane & ~(VPT == 2 ? 1 : 3)) | k);
}

// Maximum and minimum over the groups of a lane's own chunk (max_of_own) of
// stored values; has(k) false: no chunk k here.
template <int XT, int VPT, typename Has>
__device__ __forceinline__ void range_of_own(const Raw8<XT> (&h)[VPT], Has &&has, int lane, int lg, float &top,
                                             float &low) {
    if constexpr (XT == kF32) {
        float hi[VPT], lo[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float2 f[4];
            unpack8<XT>(h[k], f);
            float a = -INFINITY, b = -INFINITY;  // max, -min
            if (has(k)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a = fmax_nan(a, fmax_nan(f[i].x, f[i].y));
                    b = fmax_nan(b, fmax_nan(-f[i].x, -f[i].y));
                }
            }
            hi[k] = a;
            lo[k] = b;
        }
        top = max_of_own<VPT>(hi, -INFINITY, lane, lg, fmax_nan);
        low = -max_of_own<VPT>(lo, -INFINITY, lane, lg, fmax_nan);
    } else {
        // on pairs of the stored type, then (max, -min) as one pair, so that a
        // butterfly step is one shuffle and one maximum
        using T2 = typename std::conditional<XT == kBF16, __nv_bfloat162, __half2>::type;
        constexpr uint32_t kLowest = XT == kBF16 ? 0xff80ff80u : 0xfc00fc00u;  // (-inf, -inf)
        uint32_t w[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const T2 *p = reinterpret_cast<const T2 *>(&h[k].v[0]);
            const T2 hi = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
            const T2 lo = __hmin2_nan(__hmin2_nan(p[0], p[1]), __hmin2_nan(p[2], p[3]));
            T2 m;
            m.x = __hmax_nan(hi.x, hi.y);
            m.y = __hneg(__hmin_nan(lo.x, lo.y));
            w[k] = has(k) ? *reinterpret_cast<const uint32_t *>(&m) : kLowest;
        }
        const uint32_t r = max_of_own<VPT>(w, kLowest, lane, lg, [](uint32_t a, uint32_t b) {
            const T2 n = __hmax2_nan(*reinterpret_cast<const T2 *>(&a), *reinterpret_cast<const T2 *>(&b));
            return *reinterpret_cast<const uint32_t *>(&n);
        });
        const T2 n = *reinterpret_cast<const T2 *>(&r);
        top = to_f(n.x);
        low = -to_f(n.y);
    }
}

constexpr int kOutY = 0, kOutRow = 1, kOutGroup = 2;  // y in ydt; 8-bit rows with a scale per row; per group

// Bytes of shared memory for the threads' own parameters: as fp32, or (PRAW)
// in the rows' own 16-bit type.
__host__ __device__ constexpr int q8_fwd_smem(bool ln, bool praw, int vpt, int nt) {
    return nt * vpt * (praw ? 16 : 32) * (ln ? 2 : 1);
}

// Chunks of a row of nc that each of CL CTAs holds: a multiple of a warp's
// lanes, so that groups stay inside a warp.
template <int CL> __device__ __forceinline__ int cta_slice(int nc) {
    return CL == 1 ? nc : ((nc + CL - 1) / CL + 31) & ~31;
}

// FULL: every thread holds VPT chunks.  CL > 1: a row is split over the CTAs
// of a cluster.
template <bool LN, int XT, bool PRAW, int TPR, int VPT, int NT, int CL, int OUT, bool CK, bool FULL>
__device__ __forceinline__ void q8_fwd_body(const Q8FwdParams &p, float4 *par, float4 *scratch_all) {
    constexpr int RPC = NT / TPR;
    static_assert(CL == 1 || RPC == 1, "a cluster shares one row");
    constexpr int xes = XT == kF32 ? 4 : 2;
    constexpr bool RQ = !LN && OUT != kOutY;  // codes of h * gamma
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, lane = threadIdx.x & 31;
    RowReduce<TPR, CL> rr{scratch_all + grp * RowReduce<TPR, CL>::SCRATCH, 0, 1 + grp};
    // this CTA's part of a row: chunks [c0, c0 + nc)
    const int slice = cta_slice<CL>((int)(p.N / 8)), c0 = CL == 1 ? 0 : (int)cluster_ctarank() * slice;
    const int nc = CL == 1 ? slice : max(0, min(slice, (int)(p.N / 8) - c0));
    const float inv_n = 1.f / (float)p.N;
    const float qmax = q8_max(p.qfmt), inv_qmax = q8_inv_max(p.qfmt);
    const int qlg = p.qg - 3, clg = p.cg - 3;  // log2 of the lanes of a group
    const int own = own_chunk<VPT>(lane);
    auto has = [&](int k) { return FULL || k * TPR + t < nc; };
    constexpr int PW = PRAW ? 1 : 2;  // 16-byte words of a parameter chunk
    float4 *gp = par + threadIdx.x, *bp = par + PW * VPT * NT + threadIdx.x;
    auto param = [&](const float4 *q, int k, float2 (&f)[4]) {
        if constexpr (PRAW) {
            Raw8<XT> r;
            r.v[0] = *reinterpret_cast<const uint4 *>(q + k * NT);
            unpack8<XT>(r, f);
        } else {
            const float4 a = q[2 * k * NT], b = q[(2 * k + 1) * NT];
            f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
            f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
        }
    };
    auto keep = [&](float4 *q, int k, const float2 (&f)[4]) {
        if constexpr (PRAW) {
            *reinterpret_cast<uint4 *>(q + k * NT) = pack8<XT>(f).v[0];
        } else {
            q[2 * k * NT] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            q[(2 * k + 1) * NT] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
        }
    };
    RowCounts cnt;
    if constexpr (LN) {
        int mine = 0;
#pragma unroll
        for (int k = 0; k < VPT; ++k) mine += has(k) ? 8 : 0;
        cnt = row_counts(mine, (float)(8 * nc));
    }
    bool first = true;
    const int64_t stride = (int64_t)(gridDim.x / CL) * RPC;
    for (int64_t row = (int64_t)(blockIdx.x / CL) * RPC + grp; row < p.M; row += stride) {
        Raw8<XT> h[VPT];
        const unsigned char *xr = static_cast<const unsigned char *>(p.x) + (row * p.ldx + 8 * c0) * xes;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            h[k] = Raw8<XT>{};
            if (has(k)) h[k] = ld_raw8<XT>(xr, k * TPR + t);
        }
        if (p.res) {
            const unsigned char *rr = static_cast<const unsigned char *>(p.res) + (row * p.ldr + 8 * c0) * xes;
            Raw8<XT> r[VPT];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                r[k] = Raw8<XT>{};
                if (has(k)) r[k] = ld_raw8<XT>(rr, k * TPR + t);
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) add8<XT>(h[k], r[k]);
            if (p.h) {
                unsigned char *hr = static_cast<unsigned char *>(p.h) + (row * p.ldh + 8 * c0) * xes;
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (has(k)) st_raw8<XT>(hr, k * TPR + t, h[k]);
            }
        }
        // The next row on its way to L2 while this one is worked on; with a
        // residual the loads of a row alone keep DRAM busy (16384 x 8192:
        // 149 us without, 158 us with the prefetch).
        if (t == 0 && p.res == nullptr) {
            const int64_t next = row + stride;
            if (next < p.M && nc > 0)
                prefetch_l2(static_cast<const unsigned char *>(p.x) + (next * p.ldx + 8 * c0) * xes, nc * 8 * xes);
        }
        if (first) {  // behind the first row's loads
            first = false;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float2 f[4];
                par8g(has(k) ? p.gamma : nullptr, c0 + k * TPR + t, p.pdt, 1.f, f);
                keep(gp, k, f);
                if constexpr (LN) {
                    par8g(has(k) ? p.beta : nullptr, c0 + k * TPR + t, p.pdt, 0.f, f);
                    keep(bp, k, f);
                }
            }
        }
        if constexpr (CK) {
            uint8_t *cr = p.c + row * p.ldc + 8 * c0;
            float top, low;
            range_of_own<XT, VPT>(h, has, lane, clg, top, low);
            const CkGroup g = ck_group(top, low);
            // the first lanes of a group write its pairs, lane k of it chunk k's
            const int at = own * TPR + (t & ~((1 << clg) - 1));
            if ((lane & ((1 << clg) - 1)) < VPT && (FULL || at < nc))
                *reinterpret_cast<float2 *>(p.cs + row * p.ldcs + 2 * ((c0 + at) >> clg)) = make_float2(g.scale, g.mid);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const float2 nm = f2s(-fetch<VPT>(g.mid, lane, k)), inv = f2s(fetch<VPT>(g.inv, lane, k));
                float2 u[4];
                unpack8<XT>(h[k], u);
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = f2mul(f2add(u[i], nm), inv);
                if (has(k)) *reinterpret_cast<uint2 *>(cr + 8 * (k * TPR + t)) = codes8_i8(u, p.one);
            }
        }

        // ---------------------------------------------------------------- sums of the row
        uint8_t *qr = p.q + row * p.ldq + 8 * c0;
        float *qs = p.qs + row * p.qs_row;
        float acc, mean = 0.f, m = 0.f, unused = 0.f;
        // codes of o (chunk k), scaled by inv
        auto put = [&](int k, float2 (&o)[4], float inv) {
            const float2 i2 = f2s(inv);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = f2mul(o[i], i2);
            if (has(k)) *reinterpret_cast<uint2 *>(qr + 8 * (k * TPR + t)) = codes8(o, p.qfmt, p.one);
        };
        float2 o[VPT][4];    // h, then what is stored of it: h * gamma or y
#pragma unroll
        for (int k = 0; k < VPT; ++k) unpack8<XT>(h[k], o[k]);
        float gscale = 0.f;  // the maximum of this lane's own group
        auto put_groups = [&]() {
            float am[VPT];
#pragma unroll
            for (int k = 0; k < VPT; ++k) am[k] = amax8(o[k]);
            gscale = max_of_own<VPT>(am, 0.f, lane, qlg, fmax_nan);
            const float inv = q8_inv(gscale, qmax);
#pragma unroll
            for (int k = 0; k < VPT; ++k) put(k, o[k], fetch<VPT>(inv, lane, k));
        };
        if constexpr (LN) {
            // The thread's mean, then the deviations from it: nothing
            // cancels.  (Sum and squares about the thread's first element in
            // one pass are as many operations and level in time, but cancel
            // where that element is an outlier: 8191 x 1003 rows of N(0.5, 1)
            // with single values of 60, rstd off by up to 35 * 2^-24 against
            // 3 * 2^-24 this way.)
            float2 s2 = f2s(0.f), q2 = f2s(0.f);
#pragma unroll
            for (int k = 0; k < VPT; ++k)  // zeros past the row's end
#pragma unroll
                for (int i = 0; i < 4; ++i) s2 = f2add(s2, o[k][i]);
            mean = (s2.x + s2.y) * cnt.inv_thread;
            const float2 nt = f2s(-mean);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!has(k)) continue;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 d = f2add(o[k][i], nt);
                    q2 = f2fma(d, d, q2);
                }
            }
            acc = q2.x + q2.y;
            group_meanvar<TPR, CL>(mean, acc, cnt, inv_n, rr);
        } else {
            float2 a2 = f2s(0.f);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) a2 = f2fma(o[k][i], o[k][i], a2);
                if constexpr (RQ) {
                    float2 g8[4];
                    param(gp, k, g8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[k][i] = f2mul(o[k][i], g8[i]);
                    if constexpr (OUT == kOutRow) m = fmax_nan(m, amax8(o[k]));
                }
            }
            acc = a2.x + a2.y;
            if constexpr (OUT == kOutGroup) put_groups();
            group_sum_max<TPR, CL, OUT == kOutRow>(acc, m, rr);
        }
        const float rstd = rsqrtf(acc * inv_n + p.eps);
        if (t == 0 && c0 == 0) {
            if (p.rstd) p.rstd[row] = rstd;
            if (LN && p.mean) p.mean[row] = mean;
        }

        // ---------------------------------------------------------------- output
        const float2 nm = f2s(-mean), rs = f2s(rstd);
        if constexpr (!RQ) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {  // y; zeros past the row's end
                float2 g8[4], b8[4];
                param(gp, k, g8);
                if constexpr (LN) {
                    param(bp, k, b8);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[k][i] = has(k) ? f2fma(f2mul(f2add(o[k][i], nm), rs), g8[i], b8[i]) : f2s(0.f);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[k][i] = f2mul(f2mul(o[k][i], rs), g8[i]);
                }
                if constexpr (OUT == kOutY) {
                    if (has(k)) st8p(row_ptr(p.y, row, p.ldy, p.ydt), 8 * (int64_t)(c0 + k * TPR + t), p.ydt, o[k]);
                } else if constexpr (OUT == kOutRow) {
                    m = fmax_nan(m, amax8(o[k]));
                }
            }
        }
        if constexpr (OUT == kOutGroup) {
            if constexpr (!RQ) put_groups();
            const int at = own * TPR + (t & ~((1 << qlg) - 1));
            if ((lane & ((1 << qlg) - 1)) < VPT && (FULL || at < nc))
                qs[((c0 + at) >> qlg) * p.qs_grp] = q8_scale(gscale, RQ ? rstd : 1.f, qmax, inv_qmax);
        } else if constexpr (OUT == kOutRow) {
            if constexpr (!RQ) group_sum_max<TPR, CL, true>(unused, m, rr);
            const float inv = q8_inv(m, qmax);
#pragma unroll
            for (int k = 0; k < VPT; ++k) put(k, o[k], inv);
            if (t == 0 && c0 == 0) qs[0] = q8_scale(m, RQ ? rstd : 1.f, qmax, inv_qmax);
        }
    }
}

template <bool LN, int XT, bool PRAW, int TPR, int VPT, int NT, int MINB, int CL, int OUT, bool CK>
__global__ void __launch_bounds__(NT, MINB) q8_fwd_rows(const Q8FwdParams p) {
    static_assert(NT % TPR == 0 && TPR % 32 == 0 && VPT <= 4, "row groups");
    static_assert(TPR == 32 || NT / TPR < 16, "named barriers");
    extern __shared__ __align__(16) float4 q8_par[];
    __shared__ float4 scratch[NT / TPR * RowReduce<TPR, CL>::SCRATCH];
    if constexpr (CL > 1) cluster_sync_all();  // every CTA runs before another writes to its shared memory
    if (p.N == (int64_t)CL * TPR * VPT * 8)
        q8_fwd_body<LN, XT, PRAW, TPR, VPT, NT, CL, OUT, CK, true>(p, q8_par, scratch);
    else
        q8_fwd_body<LN, XT, PRAW, TPR, VPT, NT, CL, OUT, CK, false>(p, q8_par, scratch);
}

}  // namespace gbn
