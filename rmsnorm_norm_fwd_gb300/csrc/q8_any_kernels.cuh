// q8_any_kernels.cuh -- forward and backward of the 8-bit operators for rows
// without 16-byte vectors (any length, stride, alignment and types), rows in
// registers.
//
// A warp holds VB blocks of 256 consecutive elements, each lane 8 of a block, 32
// apart, so that every access of a warp is 32 consecutive elements whatever
// their alignment, and a group of 32..256 columns is 1..8 of a lane's elements
// across the warp.  Apart from that the steps are those of the vector kernels.
// What bounds it: the load and store instructions, one an element (8192 x 4001
// bf16 RMSNorm 32 us, 45% of the copy rate's time, 23 instructions an element,
// with group scales 43 us, 34%; 8191 x 1003 fp32 LayerNorm 18 us, 33%; backward
// 8192 x 4001 72 us, 34%).
#pragma once

#include "q8_bwd_kernels.cuh"

namespace gbn {

// Where a lane's 8 elements of a block are in every row: from element `at`, 32
// apart, those below `rem` of 32 i there.
struct Block {
    int64_t at;
    int rem;
    bool full;  // all 256 elements there (uniform over the warp)
    __device__ __forceinline__ bool has(int i) const { return 32 * i < rem; }
};
__device__ __forceinline__ Block block_at(int64_t base, int64_t n) {
    const int lane = threadIdx.x & 31;
    const int64_t rem = n - base - lane;
    return Block{base + lane, (int)(rem < 0 ? 0 : rem > 256 ? 256 : rem), base + 256 <= n};
}
// Calls f(i) for the elements that are there.
template <typename F> __device__ __forceinline__ void each(const Block &b, F &&f) {
    if (b.full) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f(i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (b.has(i)) f(i);
    }
}
// The block's elements of a row as stored, zero past its end: loads alone, so
// that several blocks' are in flight before the first is waited for.
struct RawBlock {
    uint32_t w[8];
};
__device__ __forceinline__ void ld_raw_block(const void *row, const Block &b, int dt, RawBlock &r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = 0;
    if (dt == kF32) {
        const uint32_t *p = static_cast<const uint32_t *>(row) + b.at;
        each(b, [&](int i) { r.w[i] = p[32 * i]; });
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(row) + b.at;
        each(b, [&](int i) { r.w[i] = p[32 * i]; });
    }
}
__device__ __forceinline__ void widen_block(const RawBlock &r, int dt, float (&v)[8]) {
    if (dt == kF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
    } else if (dt == kBF16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __half2float(__ushort_as_half((unsigned short)r.w[i]));
    }
}
__device__ __forceinline__ void ld_block(const void *row, const Block &b, int dt, float (&v)[8]) {
    RawBlock r;
    ld_raw_block(row, b, dt, r);
    widen_block(r, dt, v);
}
// Copies what was read for the first of a group's 2^lg neighbouring elements
// of a lane to the others.
template <typename T> __device__ __forceinline__ void spread_groups(T (&v)[8], int lg) {
#pragma unroll
    for (int i = 1; i < 8; ++i)
        if (lg >= 3 || (i & ((1 << lg) - 1))) v[i] = v[i - 1];
}
__device__ __forceinline__ bool leads_group(int i, int lg) { return lg >= 3 ? i == 0 : (i & ((1 << lg) - 1)) == 0; }
__device__ __forceinline__ void st_block(void *row, const Block &b, int dt, const float (&v)[8]) {
    auto all = [&](auto *p) {
        using T = typename std::remove_pointer<decltype(p)>::type;
        each(b, [&](int i) { p[b.at + 32 * i] = from_f<T>(v[i]); });
    };
    if (dt == kF32) all(static_cast<float *>(row));
    else if (dt == kBF16) all(static_cast<__nv_bfloat16 *>(row));
    else all(static_cast<__half *>(row));
}
__device__ __forceinline__ void st_bytes(uint8_t *row, const Block &b, const uint32_t (&v)[8]) {
    each(b, [&](int i) { row[b.at + 32 * i] = (uint8_t)v[i]; });
}

// A thread's own parameters of a block in shared memory, as fp32: `absent` for a
// null row, else zero past the row's end (what they multiply is zero there too).
template <int NT> __device__ __forceinline__ void keep_block(float4 *own, const void *row, const Block &b, int dt, float absent) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = absent;
    if (row) ld_block(row, b, dt, g);
    own[0] = make_float4(g[0], g[1], g[2], g[3]);
    own[NT] = make_float4(g[4], g[5], g[6], g[7]);
}
template <int NT> __device__ __forceinline__ void own_block(const float4 *own, float (&g)[8]) {
    const float4 a = own[0], b = own[NT];
    g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
    g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
}

// Maxima over the groups of a block: m[i] joined with its 2^lg - 1 neighbours
// of the same group, then over the warp's lanes, all 8 side by side (partner
// lanes trade halves in the first three steps): lane l gets that of i = l mod 8.
__device__ __forceinline__ float block_max(float (&m)[8], int lg) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
        if (o < (1 << lg)) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = fmax_nan(m[i], m[i ^ o]);
#pragma unroll
            for (int i = 0; i < 8; ++i) m[i] = t[i];
        }
    auto trade = [&](float even, float odd, int o) {
        const bool b = lane & o;
        return fmax_nan(b ? odd : even, __shfl_xor_sync(0xffffffffu, b ? even : odd, o));
    };
    const float a0 = trade(m[0], m[1], 1), a1 = trade(m[2], m[3], 1), a2 = trade(m[4], m[5], 1), a3 = trade(m[6], m[7], 1);
    float r = trade(trade(a0, a1, 2), trade(a2, a3, 2), 4);
    r = fmax_nan(r, __shfl_xor_sync(0xffffffffu, r, 8));
    return fmax_nan(r, __shfl_xor_sync(0xffffffffu, r, 16));
}
__device__ __forceinline__ float from_lane(float v, int i) { return __shfl_sync(0xffffffffu, v, i); }

// Elements of a row that each of CL CTAs holds: whole blocks.
template <int CL> __device__ __forceinline__ int64_t cta_columns(int64_t n) {
    return CL == 1 ? n : ((n + CL - 1) / CL + 255) & ~(int64_t)255;
}

template <bool LN, int TPR, int VB, int NT, int MINB, int CL, int OUT, bool CK>
__global__ void __launch_bounds__(NT, MINB) q8_fwd_any(const Q8FwdParams p) {
    static_assert(TPR == 32 || NT / TPR < 16, "named barriers");
    constexpr int RPC = NT / TPR, WPR = TPR / 32;
    constexpr bool RQ = !LN && OUT != kOutY;  // codes of h * gamma
    extern __shared__ __align__(16) float4 q8_par[];  // own gamma, then own beta
    __shared__ float4 scratch_all[RPC * RowReduce<TPR, CL>::SCRATCH];
    if constexpr (CL > 1) cluster_sync_all();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, lane = threadIdx.x & 31, warp = t >> 5;
    float4 *gp = q8_par + threadIdx.x, *bp = gp + 2 * VB * NT;
    RowReduce<TPR, CL> rr{scratch_all + grp * RowReduce<TPR, CL>::SCRATCH, 0, 1 + grp};
    // this CTA's part of a row: elements [j0, n)
    const int64_t cols = cta_columns<CL>(p.N), j0 = CL == 1 ? 0 : (int64_t)cluster_ctarank() * cols;
    const int64_t n = CL == 1 ? p.N : (j0 + cols < p.N ? j0 + cols : p.N);
    const float inv_n = 1.f / (float)p.N;
    const float qmax = q8_max(p.qfmt), inv_qmax = q8_inv_max(p.qfmt);
    const int qlg = p.qg - 5, clg = p.cg - 5;  // log2 of a lane's elements of a group in a block
    Block blk[VB];
#pragma unroll
    for (int k = 0; k < VB; ++k) blk[k] = block_at(j0 + 256 * (int64_t)(k * WPR + warp), n);
    auto base = [&](int k) { return blk[k].at - lane; };
    auto has = [&](int k, int i) { return blk[k].has(i); };
    RowCounts cnt;
    if constexpr (LN) {
        int mine = 0;
#pragma unroll
        for (int k = 0; k < VB; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) mine += has(k, i) ? 1 : 0;
        cnt = row_counts(mine, n > j0 ? (float)(n - j0) : 0.f);
    }
    bool first = true;
    const int64_t stride = (int64_t)(gridDim.x / CL) * RPC;
    for (int64_t row = (int64_t)(blockIdx.x / CL) * RPC + grp; row < p.M; row += stride) {
        float v[VB][8];  // h, then what is stored of it: h * gamma or y
        const void *xr = row_ptr(p.x, row, p.ldx, p.xdt);
        RawBlock xw[VB], rw[VB];
#pragma unroll
        for (int k = 0; k < VB; ++k) ld_raw_block(xr, blk[k], p.xdt, xw[k]);
        if (p.res) {
            const void *rrow = row_ptr(p.res, row, p.ldr, p.xdt);
#pragma unroll
            for (int k = 0; k < VB; ++k) ld_raw_block(rrow, blk[k], p.xdt, rw[k]);
        }
        if (t == 0 && n > j0) {
            const int64_t next = row + stride;
            if (next < p.M)
                prefetch_l2_inner(static_cast<const unsigned char *>(row_ptr(p.x, next, p.ldx, p.xdt)) + j0 * esize(p.xdt),
                                  (int)(n - j0) * esize(p.xdt));
        }
#pragma unroll
        for (int k = 0; k < VB; ++k) widen_block(xw[k], p.xdt, v[k]);
        if (p.res) {
#pragma unroll
            for (int k = 0; k < VB; ++k) {
                float r[8];
                widen_block(rw[k], p.xdt, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = round_to(v[k][i] + r[i], p.xdt);
            }
            if (p.h) {
                void *hr = row_ptr(p.h, row, p.ldh, p.xdt);
#pragma unroll
                for (int k = 0; k < VB; ++k) st_block(hr, blk[k], p.xdt, v[k]);
            }
        }
        if (first) {  // behind the first row's loads
            first = false;
#pragma unroll
            for (int k = 0; k < VB; ++k) {
                keep_block<NT>(gp + 2 * k * NT, p.gamma, blk[k], p.pdt, 1.f);
                if constexpr (LN) keep_block<NT>(bp + 2 * k * NT, p.beta, blk[k], p.pdt, 0.f);
            }
        }
        if constexpr (CK) {
            uint8_t *cr = p.c + row * p.ldc;
            float *cs = p.cs + row * p.ldcs;
#pragma unroll
            for (int k = 0; k < VB; ++k) {
                float hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    hi[i] = has(k, i) ? v[k][i] : -INFINITY;
                    lo[i] = has(k, i) ? -v[k][i] : -INFINITY;
                }
                const CkGroup g = ck_group(block_max(hi, clg), -block_max(lo, clg));
                const int64_t first = base(k) + 32 * lane;  // lane i < 8: first element of i
                if (lane < 8 && (lane & ((1 << clg) - 1)) == 0 && first < n) {
                    cs[2 * (first >> p.cg)] = g.scale;
                    cs[2 * (first >> p.cg) + 1] = g.mid;
                }
                uint32_t code[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    code[i] = i8_code(__fmul_rn(__fsub_rn(v[k][i], from_lane(g.mid, i)), from_lane(g.inv, i)));
                st_bytes(cr, blk[k], code);
            }
        }

        // ---------------------------------------------------------------- sums of the row
        uint8_t *qr = p.q + row * p.ldq;
        float *qs = p.qs + row * p.qs_row;
        float acc = 0.f, mean = 0.f, m = 0.f, unused = 0.f;
        float gmax[VB];  // lane l: the maximum of the group of i = l mod 8
        auto put = [&](int k, auto &&inv) {
            uint32_t code[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) code[i] = q8_code(__fmul_rn(v[k][i], inv(i)), p.qfmt);
            st_bytes(qr, blk[k], code);
        };
        auto put_groups = [&]() {
#pragma unroll
            for (int k = 0; k < VB; ++k) {
                float a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] = fabsf(v[k][i]);
                gmax[k] = block_max(a, qlg);
                const float inv = q8_inv(gmax[k], qmax);
                put(k, [&](int i) { return from_lane(inv, i); });
            }
        };
        if constexpr (LN) {
            // the thread's mean, then the deviations from it, as the vector kernels
#pragma unroll
            for (int k = 0; k < VB; ++k)  // zeros past the row's end
#pragma unroll
                for (int i = 0; i < 8; ++i) mean += v[k][i];
            mean *= cnt.inv_thread;
#pragma unroll
            for (int k = 0; k < VB; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (has(k, i)) {
                        const float d = v[k][i] - mean;
                        acc = fmaf(d, d, acc);
                    }
            group_meanvar<TPR, CL>(mean, acc, cnt, inv_n, rr);
        } else {
#pragma unroll
            for (int k = 0; k < VB; ++k) {
#pragma unroll
                for (int i = 0; i < 8; ++i) acc = fmaf(v[k][i], v[k][i], acc);
                if constexpr (RQ) {
                    float g[8];
                    own_block<NT>(gp + 2 * k * NT, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[k][i] *= g[i];
                        m = fmax_nan(m, fabsf(v[k][i]));
                    }
                }
            }
            if constexpr (OUT == kOutGroup) put_groups();
            group_sum_max<TPR, CL, OUT == kOutRow>(acc, m, rr);
        }
        const float rstd = rsqrtf(acc * inv_n + p.eps);
        if (t == 0 && j0 == 0) {
            if (p.rstd) p.rstd[row] = rstd;
            if (LN && p.mean) p.mean[row] = mean;
        }

        // ---------------------------------------------------------------- output
        if constexpr (!RQ) {
#pragma unroll
            for (int k = 0; k < VB; ++k) {  // y; zeros past the row's end
                float g[8];
                own_block<NT>(gp + 2 * k * NT, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = has(k, i) ? (v[k][i] - mean) * rstd * g[i] : 0.f;
                if constexpr (LN) {
                    own_block<NT>(bp + 2 * k * NT, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[k][i] += g[i];
                }
                if constexpr (OUT == kOutY) {
                    st_block(row_ptr(p.y, row, p.ldy, p.ydt), blk[k], p.ydt, v[k]);
                } else if constexpr (OUT == kOutRow) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = fmax_nan(m, fabsf(v[k][i]));
                }
            }
        }
        if constexpr (OUT == kOutGroup) {
            if constexpr (!RQ) put_groups();
            // lanes 8 k to 8 k + 7 write block k's (block_max leaves i's maximum on every lane l mod 8 = i)
            static_assert(VB <= 4, "eight lanes a block");
            float top = gmax[0];
            int64_t first = base(0);
#pragma unroll
            for (int k = 1; k < VB; ++k)
                if (lane >> 3 == k) top = gmax[k], first = base(k);
            first += 32 * (lane & 7);
            if (lane < 8 * VB && (lane & 7 & ((1 << qlg) - 1)) == 0 && first < n)
                qs[(first >> p.qg) * p.qs_grp] = q8_scale(top, RQ ? rstd : 1.f, qmax, inv_qmax);
        } else if constexpr (OUT == kOutRow) {
            if constexpr (!RQ) group_sum_max<TPR, CL, true>(unused, m, rr);
            const float inv = q8_inv(m, qmax);
#pragma unroll
            for (int k = 0; k < VB; ++k) put(k, [&](int) { return inv; });
            if (t == 0 && j0 == 0) qs[0] = q8_scale(m, RQ ? rstd : 1.f, qmax, inv_qmax);
        }
    }
}

template <bool LN, int TPR, int VB, int NT, int MINB, int CL>
__global__ void __launch_bounds__(NT, MINB) q8_bwd_any(const Q8BwdParams p) {
    static_assert(TPR == 32 || NT / TPR < 16, "named barriers");
    pdl_launch_dependents();  // the column reduce waits for this grid's completion
    constexpr int RPC = NT / TPR, WPR = TPR / 32;
    extern __shared__ __align__(16) float4 q8_par[];  // own gamma, then the row groups' column sums, [VB][8][NT]
    __shared__ float4 scratch_all[RPC * RowReduce<TPR, CL>::SCRATCH];
    if constexpr (CL > 1) cluster_sync_all();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR, warp = t >> 5;
    RowReduce<TPR, CL> rr{scratch_all + grp * RowReduce<TPR, CL>::SCRATCH, 0, 1 + grp};
    float4 *gp = q8_par + threadIdx.x;
    const int64_t cols = cta_columns<CL>(p.N), j0 = CL == 1 ? 0 : (int64_t)cluster_ctarank() * cols;
    const int64_t n = CL == 1 ? p.N : (j0 + cols < p.N ? j0 + cols : p.N);
    const float inv_n = 1.f / (float)p.N;
    Block blk[VB];
#pragma unroll
    for (int k = 0; k < VB; ++k) blk[k] = block_at(j0 + 256 * (int64_t)(k * WPR + warp), n);
    float accg[VB][8], accb[LN ? VB : 1][8];
#pragma unroll
    for (int k = 0; k < VB; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            accg[k][i] = 0.f;
            if constexpr (LN) accb[k][i] = 0.f;
        }
    bool first = true;
    const int64_t stride = (int64_t)(gridDim.x / CL) * RPC;
    for (int64_t row = (int64_t)(blockIdx.x / CL) * RPC + grp; row < p.M; row += stride) {
        const void *dyr = row_ptr(p.dy, row, p.lddy, p.ydt);
        const uint8_t *cr = p.c + row * p.ldc;
        const float *cs = p.cs + row * p.ldcs;
        const float rstd = __ldg(p.rstd + row);
        const float mean = LN ? __ldg(p.mean + row) : 0.f;
        RawBlock dw[VB];
        uint8_t code[VB][8];
        float2 sm[VB][8];  // (scale, mid)
#pragma unroll
        for (int k = 0; k < VB; ++k) {
            ld_raw_block(dyr, blk[k], p.ydt, dw[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) code[k][i] = 0, sm[k][i] = make_float2(0.f, mean);
            each(blk[k], [&](int i) { code[k][i] = cr[blk[k].at + 32 * i]; });
            each(blk[k], [&](int i) {
                if (leads_group(i, p.cg - 5))
                    sm[k][i] = __ldg(reinterpret_cast<const float2 *>(cs) + ((blk[k].at + 32 * i) >> p.cg));
            });
        }
        if (t == 0 && n > j0) {
            const int64_t next = row + stride;
            if (next < p.M) {
                prefetch_l2_inner(static_cast<const unsigned char *>(row_ptr(p.dy, next, p.lddy, p.ydt)) + j0 * esize(p.ydt),
                                  (int)(n - j0) * esize(p.ydt));
                prefetch_l2_inner(p.c + next * p.ldc + j0, (int)(n - j0));
            }
        }
        if (first) {  // behind the first row's loads
            first = false;
#pragma unroll
            for (int k = 0; k < VB; ++k) keep_block<NT>(gp + 2 * k * NT, p.gamma, blk[k], p.pdt, 1.f);
        }
        float d[VB][8], xh[VB][8];
#pragma unroll
        for (int k = 0; k < VB; ++k) {
            widen_block(dw[k], p.ydt, d[k]);
            spread_groups(sm[k], p.cg - 5);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                xh[k][i] = blk[k].has(i) ? fmaf((float)(int8_t)code[k][i], sm[k][i].x * rstd, (sm[k][i].y - mean) * rstd) : 0.f;
        }
        float sum[LN ? 2 : 1] = {};
#pragma unroll
        for (int k = 0; k < VB; ++k) {
            float g[8];
            own_block<NT>(gp + 2 * k * NT, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dg = d[k][i] * g[i];
                sum[0] = fmaf(dg, xh[k][i], sum[0]);
                if constexpr (LN) sum[LN ? 1 : 0] += dg;
            }
        }
        group_sums<TPR, CL, LN ? 2 : 1>(sum, rr);
        const float nrc2 = -rstd * (sum[0] * inv_n), nrc1 = LN ? -rstd * (sum[LN ? 1 : 0] * inv_n) : 0.f;
        void *dxr = row_ptr(p.dx, row, p.lddx, p.xdt);
        const void *drr = p.dres ? row_ptr(p.dres, row, p.lddres, p.xdt) : nullptr;
#pragma unroll
        for (int k = 0; k < VB; ++k) {
            float g[8], o[8];
            own_block<NT>(gp + 2 * k * NT, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dg = d[k][i] * g[i];
                o[i] = fmaf(nrc2, xh[k][i], fmaf(rstd, dg, nrc1));
                accg[k][i] = fmaf(d[k][i], xh[k][i], accg[k][i]);
                if constexpr (LN) accb[k][i] += d[k][i];
            }
            if (drr) {
                float r[8];
                ld_block(drr, blk[k], p.xdt, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] += r[i];
            }
            st_block(dxr, blk[k], p.xdt, o);
        }
    }
    // this CTA's (cluster's) partial row; several row groups are added in group order
    auto store = [&](float (&acc)[VB][8], float *ws) {
        if constexpr (RPC > 1) {
            float *q8_sums = reinterpret_cast<float *>(q8_par);
            __syncthreads();
#pragma unroll
            for (int k = 0; k < VB; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) q8_sums[(8 * k + i) * NT + threadIdx.x] = acc[k][i];
            __syncthreads();
            for (int s = threadIdx.x; s < 8 * VB * TPR; s += NT) {
                const int ki = s / TPR, tt = s % TPR;
                const int64_t j = 256 * (int64_t)((ki >> 3) * WPR + (tt >> 5)) + 32 * (ki & 7) + (tt & 31);
                if (j >= p.N) continue;
                float a = q8_sums[ki * NT + tt];
#pragma unroll
                for (int g = 1; g < RPC; ++g) a += q8_sums[ki * NT + g * TPR + tt];
                ws[j] = a;
            }
        } else {
#pragma unroll
            for (int k = 0; k < VB; ++k) st_block(ws, blk[k], kF32, acc[k]);
        }
    };
    const int64_t P = gridDim.x / CL, part = blockIdx.x / CL;
    store(accg, p.ws + part * p.N);
    if constexpr (LN) store(accb, p.ws + (P + part) * p.N);
}

// 8-bit rows read back: a warp keeps one block of columns, with gamma and beta
// of it in registers, and walks down the rows.  blockDim.x = 32 wx ry threads:
// wx blocks of the columns (blockIdx.x), ry rows side by side.
template <bool NORM>
__global__ void __launch_bounds__(kElemCTA) q8_read_any(const Q8ReadParams p, int wx) {
    constexpr int U = 2;  // rows in flight
    const int warp = threadIdx.x >> 5, ry = blockDim.x / (32 * wx);
    const Block b = block_at(256 * ((int64_t)blockIdx.x * wx + warp % wx), p.N);
    if (b.at - (threadIdx.x & 31) >= p.N) return;
    float g[8], be[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f, be[i] = 0.f;
    if constexpr (NORM) {
        if (p.gamma) ld_block(p.gamma, b, p.pdt, g);
        if (p.beta) ld_block(p.beta, b, p.pdt, be);
    }
    const int glg = p.qg < 0 ? 3 : p.qg - 5;  // log2 of a lane's elements of a group
    const int64_t step = (int64_t)gridDim.y * ry;
    for (int64_t row0 = (int64_t)blockIdx.y * ry + warp / wx; row0 < p.M; row0 += U * step) {
        uint8_t code[U][8];
        float a[U][8], m[U][8], mean[U], rstd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step;
            mean[u] = 0.f, rstd[u] = 1.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) code[u][i] = 0, a[u][i] = m[u][i] = 0.f;
            if (row >= p.M) continue;
            const uint8_t *q = p.q + row * p.ldq + b.at;
            each(b, [&](int i) { code[u][i] = q[32 * i]; });
            each(b, [&](int i) {
                if (leads_group(i, glg)) {
                    const int64_t at = row * p.s_row + (p.qg < 0 ? 0 : (b.at + 32 * i) >> p.qg) * p.s_grp;
                    a[u][i] = __ldg(p.scale + at);
                    if (p.mid) m[u][i] = __ldg(p.mid + at);
                }
            });
            if constexpr (NORM) {
                if (p.mean) mean[u] = __ldg(p.mean + row);
                if (p.rstd) rstd[u] = __ldg(p.rstd + row);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * step;
            if (row >= p.M) break;
            spread_groups(a[u], glg);
            spread_groups(m[u], glg);
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = fmaf(a[u][i], q8_value(code[u][i], p.qfmt), m[u][i]);
                if constexpr (NORM) v[i] = fmaf((v[i] - mean[u]) * rstd[u], g[i], be[i]);
            }
            st_block(row_ptr(p.y, row, p.ldy, p.ydt), b, p.ydt, v);
        }
    }
}

}  // namespace gbn
