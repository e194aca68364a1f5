// q8_bwd_kernels.cuh -- backward of the norms from the 8-bit checkpoint, rows
// in registers: a row group of TPR threads holds one row of codes and dy, each
// thread VPT chunks of 8 consecutive elements, chunk k * TPR + t, always the
// same columns, so that its dgamma (dbeta) sums stay in registers.
//
// With the group's (scale, mid) and the row's statistics xhat is one
// multiply-add of the code: xhat = code * (scale * rstd) + (mid - mean) * rstd.
// Two passes over the registers: sum g xhat (and sum g), one barrier, then dx
// and the column sums; codes and dy are widened again in the second pass.
//
// Rows longer than one CTA holds are split over a cluster, as in the forward.
//
// What bounds it: DRAM, 5 bytes an element (bf16 dy and dx, 1.06 bytes of
// checkpoint), 7 with a residual's gradient.  The next row is prefetched to L2
// while one is worked on (copying it to shared memory asynchronously instead
// measured 251 us against 163 us).  Measured, bf16: RMSNorm 16384 x 8192 117 us,
// 163 us with a residual's gradient (86% of the copy rate's time); LayerNorm
// 16384 x 8192 145 us (69%), 16384 x 4096 77 us (65%): 19 instructions an element
// at 16 warps an SM, which is what two column sums in registers leave; issue at
// 47%, so latency more than instructions.
#pragma once

#include "q8_rows_kernels.cuh"

namespace gbn {

// Eight int8 codes as fp32 (exact): the code with its sign bit flipped as the
// low byte of 2^23 is 2^23 + 128 + code.
__device__ __forceinline__ void i8_pairs(uint2 w, float2 (&f)[4]) {
    const uint32_t a = w.x ^ 0x80808080u, b = w.y ^ 0x80808080u;
    const float2 off = f2s(-8388736.f);
    auto at = [](uint32_t v, int i) { return __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7650 | i)); };
    f[0] = f2add(make_float2(at(a, 0), at(a, 1)), off);
    f[1] = f2add(make_float2(at(a, 2), at(a, 3)), off);
    f[2] = f2add(make_float2(at(b, 0), at(b, 1)), off);
    f[3] = f2add(make_float2(at(b, 2), at(b, 3)), off);
}
__device__ __forceinline__ uint2 ld_codes8(const uint8_t *row, int c) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(row + 8 * c));
    return v;
}

// NV (1, 2, 4) sums over a row group; the same bits on every thread.  Partner
// lanes trade values first, so that each lane goes on with one of them (value
// lane mod NV): 6 shuffles for four sums over a warp instead of 20.
template <int TPR, int CL, int NV>
__device__ __forceinline__ void group_sums(float (&v)[NV], RowReduce<TPR, CL> &rr) {
    static_assert(NV == 1 || NV == 2 || NV == 4, "values");
    const int lane = threadIdx.x & 31;
    auto trade = [&](float even, float odd, int o) {
        const bool b = lane & o;
        return (b ? odd : even) + __shfl_xor_sync(0xffffffffu, b ? even : odd, o);
    };
    float r = v[0];
    if constexpr (NV == 2) r = trade(v[0], v[1], 1);
    if constexpr (NV == 4) r = trade(trade(v[0], v[1], 1), trade(v[2], v[3], 1), 2);
#pragma unroll
    for (int o = NV; o < 32; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if constexpr (TPR > 32) {
        constexpr int WPR = TPR / 32, MOST = 32 / NV, L = pow2_at_least(WPR), AT_ONCE = L < MOST ? L : MOST;
        float *buf = reinterpret_cast<float *>(rr.scratch + rr.parity * WPR);
        if (lane < NV) buf[((threadIdx.x % TPR) >> 5) * NV + lane] = r;
        named_sync(rr.bar_id, TPR);
        r = 0.f;
#pragma unroll
        for (int w0 = 0; w0 < WPR; w0 += AT_ONCE) {
            const int w = w0 + ((lane / NV) & (AT_ONCE - 1));
            if (w < WPR) r += buf[w * NV + (lane & (NV - 1))];
        }
#pragma unroll
        for (int o = NV; o < NV * AT_ONCE; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        if constexpr (CL == 1) rr.parity ^= 1;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = NV == 1 ? r : __shfl_sync(0xffffffffu, r, i);
    if constexpr (CL > 1) {
        float4 b = rr.ctas(make_float4(v[0], NV > 1 ? v[1] : 0.f, NV > 2 ? v[2] : 0.f, NV > 2 ? v[3] : 0.f));
        float *f = &b.x;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int o = CL / 2; o > 0; o >>= 1) f[i] += __shfl_xor_sync(0xffffffffu, f[i], o);
            v[i] = f[i];
        }
    }
}

// Eight elements as read: a type fixed at compile time stays as stored, an
// unknown one (XT -1) is widened at once.
template <int XT> struct Row8 {
    Raw8<XT> r;
    __device__ __forceinline__ void load(const void *row, int c, int) { r = ld_raw8<XT>(row, c); }
    __device__ __forceinline__ void zero() { r = Raw8<XT>{}; }
    __device__ __forceinline__ void get(float2 (&f)[4]) const { unpack8<XT>(r, f); }
};
template <> struct Row8<-1> {
    float2 v[4];
    __device__ __forceinline__ void load(const void *row, int c, int dt) {
        if (dt == kF32) unpack8<kF32>(ld_raw8<kF32>(row, c), v);
        else if (dt == kBF16) unpack8<kBF16>(ld_raw8<kBF16>(row, c), v);
        else unpack8<kF16>(ld_raw8<kF16>(row, c), v);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f2s(0.f);
    }
    __device__ __forceinline__ void get(float2 (&f)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = v[i];
    }
};

// The 16-byte-aligned part of [p, p + bytes) brought to L2.
__device__ __forceinline__ void prefetch_l2_inner(const void *p, int bytes) {
    const uintptr_t a = (reinterpret_cast<uintptr_t>(p) + 15) & ~(uintptr_t)15;
    const uintptr_t e = (reinterpret_cast<uintptr_t>(p) + bytes) & ~(uintptr_t)15;
    if (e > a) prefetch_l2(reinterpret_cast<const void *>(a), (int)(e - a));
}

__device__ __forceinline__ const void *at_chunk(const void *row, int c, int dt) {
    return static_cast<const unsigned char *>(row) + (int64_t)c * 8 * esize(dt);
}

// XT: storage type of dy, dres and dx, or -1 for any combination.  R: rows a
// row group works on at a time (their sums share one barrier).
template <bool LN, int XT, int TPR, int VPT, int R, int NT, int MINB, int CL>
__global__ void __launch_bounds__(NT, MINB) q8_bwd_rows(const Q8BwdParams p) {
    static_assert(NT % TPR == 0 && TPR % 32 == 0, "row groups");
    static_assert(TPR == 32 || NT / TPR < 16, "named barriers");
    pdl_launch_dependents();  // the column reduce waits for this grid's completion
    constexpr int RPC = NT / TPR, NS = LN ? 2 : 1;
    static_assert(CL == 1 || RPC == 1, "a cluster shares one row");
    extern __shared__ __align__(16) float4 q8_par[];  // own gamma, then the row groups' column sums
    __shared__ float4 scratch_all[RPC * RowReduce<TPR, CL>::SCRATCH];
    if constexpr (CL > 1) cluster_sync_all();  // every CTA runs before another writes to its shared memory
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    RowReduce<TPR, CL> rr{scratch_all + grp * RowReduce<TPR, CL>::SCRATCH, 0, 1 + grp};
    // this CTA's part of a row: chunks [c0, c0 + nc)
    const int slice = cta_slice<CL>((int)(p.N / 8)), c0 = CL == 1 ? 0 : (int)cluster_ctarank() * slice;
    const int nc = CL == 1 ? slice : max(0, min(slice, (int)(p.N / 8) - c0));
    const int clg = p.cg - 3;
    const int xdt = XT >= 0 ? XT : p.xdt, ydt = XT >= 0 ? XT : p.ydt;
    const float inv_n = 1.f / (float)p.N;
    auto has = [&](int k) { return k * TPR + t < nc; };
    float4 *gp = q8_par + threadIdx.x;
    float2 accg[VPT][4], accb[LN ? VPT : 1][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            accg[k][i] = f2s(0.f);
            if constexpr (LN) accb[k][i] = f2s(0.f);
        }
    bool first = true;
    const int64_t stride = (int64_t)(gridDim.x / CL) * RPC;
    for (int64_t row0 = (int64_t)(blockIdx.x / CL) * RPC + grp; row0 < p.M; row0 += R * stride) {
        Row8<XT> dy[R][VPT];
        uint2 code[R][VPT];
        float2 ab[R][VPT];  // (scale, mid), then xhat = code * a + b
        float rstd[R], mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * stride;
            const bool ok = R == 1 || row < p.M;
            rstd[r] = mean[r] = 0.f;
            if (ok) {
                rstd[r] = __ldg(p.rstd + row);
                if constexpr (LN) mean[r] = __ldg(p.mean + row);
            }
            const void *dyr = at_chunk(row_ptr(p.dy, row, p.lddy, ydt), c0, ydt);
            const uint8_t *cr = p.c + row * p.ldc + 8 * c0;
            const float2 *cs = reinterpret_cast<const float2 *>(p.cs + row * p.ldcs);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                dy[r][k].zero();
                code[r][k] = make_uint2(0, 0);
                ab[r][k] = make_float2(0.f, 0.f);
                if (ok && has(k)) {
                    dy[r][k].load(dyr, k * TPR + t, ydt);
                    code[r][k] = ld_codes8(cr, k * TPR + t);
                    ab[r][k] = __ldg(cs + ((c0 + k * TPR + t) >> clg));
                }
            }
        }
        if (t < R) {
            const int64_t next = row0 + (R + t) * stride;
            if (next < p.M && nc > 0) {
                prefetch_l2(at_chunk(row_ptr(p.dy, next, p.lddy, ydt), c0, ydt), nc * 8 * esize(ydt));
                prefetch_l2_inner(p.c + next * p.ldc + 8 * c0, nc * 8);
                prefetch_l2_inner(p.cs + next * p.ldcs + 2 * (c0 >> clg), (((nc - 1) >> clg) + 1) * 8);
                if (p.dres)
                    prefetch_l2(at_chunk(row_ptr(p.dres, next, p.lddres, xdt), c0, xdt), nc * 8 * esize(xdt));
            }
        }
        if (first) {  // behind the first rows' loads
            first = false;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float2 f[4];
                par8g(has(k) ? p.gamma : nullptr, c0 + k * TPR + t, p.pdt, 1.f, f);
                gp[2 * k * NT] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
                gp[(2 * k + 1) * NT] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
            }
        }
        // g and xhat of chunk k
        auto values = [&](int r, int k, const float4 &a, const float4 &b, float2 (&d)[4], float2 (&g)[4], float2 (&xh)[4]) {
            dy[r][k].get(d);
            i8_pairs(code[r][k], xh);
            g[0] = f2mul(d[0], make_float2(a.x, a.y)), g[1] = f2mul(d[1], make_float2(a.z, a.w));
            g[2] = f2mul(d[2], make_float2(b.x, b.y)), g[3] = f2mul(d[3], make_float2(b.z, b.w));
#pragma unroll
            for (int i = 0; i < 4; ++i) xh[i] = f2fma(xh[i], f2s(ab[r][k].x), f2s(ab[r][k].y));
        };
        float2 s2[R], s1[R];
#pragma unroll
        for (int r = 0; r < R; ++r) s2[r] = s1[r] = f2s(0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const float4 ga = gp[2 * k * NT], gb = gp[(2 * k + 1) * NT];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                ab[r][k] = make_float2(ab[r][k].x * rstd[r], (ab[r][k].y - mean[r]) * rstd[r]);
                float2 d[4], g[4], xh[4];
                values(r, k, ga, gb, d, g, xh);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s2[r] = f2fma(g[i], xh[i], s2[r]);
                    if constexpr (LN) s1[r] = f2add(s1[r], g[i]);
                }
            }
        }
        float sum[R * NS];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sum[r * NS] = s2[r].x + s2[r].y;
            if constexpr (LN) sum[r * NS + 1] = s1[r].x + s1[r].y;
        }
        group_sums<TPR, CL, R * NS>(sum, rr);
        // dx = rstd (g - c1 - xhat c2) + dres
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if (!has(k)) continue;
            const float4 ga = gp[2 * k * NT], gb = gp[(2 * k + 1) * NT];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t row = row0 + r * stride;
                if (R > 1 && row >= p.M) continue;
                const float2 r2 = f2s(rstd[r]), nrc2 = f2s(-rstd[r] * (sum[r * NS] * inv_n)),
                             nrc1 = f2s(LN ? -rstd[r] * (sum[r * NS + NS - 1] * inv_n) : 0.f);
                Row8<XT> dr;
                if (p.dres) dr.load(at_chunk(row_ptr(p.dres, row, p.lddres, xdt), c0, xdt), k * TPR + t, xdt);
                float2 d[4], g[4], xh[4], o[4];
                values(r, k, ga, gb, d, g, xh);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[i] = f2fma(nrc2, xh[i], LN ? f2fma(r2, g[i], nrc1) : f2mul(r2, g[i]));
                    accg[k][i] = f2fma(d[i], xh[i], accg[k][i]);
                    if constexpr (LN) accb[k][i] = f2add(accb[k][i], d[i]);
                }
                if (p.dres) {
                    float2 q[4];
                    dr.get(q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = f2add(o[i], q[i]);
                }
                st8p(row_ptr(p.dx, row, p.lddx, xdt), 8 * (int64_t)(c0 + k * TPR + t), xdt, o);
            }
        }
    }

    // This CTA's (cluster's) partial row: the row groups' sums of the same columns are
    // added in group order through shared memory.
    auto store = [&](float2 (&acc)[VPT][4], float *ws) {
        if constexpr (RPC > 1) {
            __syncthreads();  // gp, or the other sum, is no longer needed
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                gp[2 * k * NT] = make_float4(acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y);
                gp[(2 * k + 1) * NT] = make_float4(acc[k][2].x, acc[k][2].y, acc[k][3].x, acc[k][3].y);
            }
            __syncthreads();
            for (int s = threadIdx.x; s < 2 * VPT * TPR; s += NT) {
                const int kh = s / TPR, tt = s % TPR;  // half chunk kh of thread tt
                const int64_t col = 8 * (int64_t)((kh >> 1) * TPR + tt) + 4 * (kh & 1);
                if (col >= p.N) continue;
                float4 a = q8_par[kh * NT + tt];
#pragma unroll
                for (int g = 1; g < RPC; ++g) {
                    const float4 b = q8_par[kh * NT + g * TPR + tt];
                    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
                }
                *reinterpret_cast<float4 *>(ws + col) = a;
            }
        } else {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (!has(k)) continue;
                float4 *o = reinterpret_cast<float4 *>(ws + 8 * (int64_t)(c0 + k * TPR + t));
                o[0] = make_float4(acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y);
                o[1] = make_float4(acc[k][2].x, acc[k][2].y, acc[k][3].x, acc[k][3].y);
            }
        }
    };
    const int64_t P = gridDim.x / CL, part = blockIdx.x / CL;
    store(accg, p.ws + part * p.N);
    if constexpr (LN) store(accb, p.ws + (P + part) * p.N);
}

}  // namespace gbn
