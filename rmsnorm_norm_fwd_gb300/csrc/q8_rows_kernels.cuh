// q8_rows_kernels.cuh -- forward of the 8-bit operators with rows in
// registers: a row group of TPR threads holds one row, each thread VPT chunks
// of 8 consecutive elements, chunk k * TPR + t.
//
// What bounds it: DRAM.  A row is read once and written once (bf16: 2 + 1
// bytes an element, 7 with a residual sum); per element the arithmetic is a
// few operations on fp32 pairs.
//
//   - A chunk is 16 bytes of a 16-bit type in and 8 codes out, so a group of
//     32..256 columns is 4..32 consecutive lanes of a warp: its maxima are a
//     lane butterfly, without shared memory.
//   - RMSNorm's codes are those of h * gamma (rstd cancels): with group scales
//     they are written before the row's sum is known, with row scales the sum
//     and the maximum are one reduction with one barrier.
//   - The checkpoint's codes need h alone and are written before the
//     statistics too.
#pragma once

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
template <int XT> __device__ __forceinline__ float2 round2(float2 v) {
    if constexpr (XT == kF32) return v;
    return make_float2(round_to(v.x, XT), round_to(v.y, XT));
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

__device__ __forceinline__ float amax8(const float2 (&f)[4]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmax_nan(m, fmax_nan(fabsf(f[i].x), fabsf(f[i].y)));
    return m;
}
// Maximum over the aligned 2^lg lanes of a group (lg <= 5, uniform).
__device__ __forceinline__ float lanes_max(float v, int lg) {
#pragma unroll
    for (int o = 0; o < 5; ++o)
        if (o < lg) v = fmax_nan(v, __shfl_xor_sync(0xffffffffu, v, 1 << o));
    return v;
}
__device__ __forceinline__ float lanes_min(float v, int lg) {
#pragma unroll
    for (int o = 0; o < 5; ++o)
        if (o < lg) v = fmin_nan(v, __shfl_xor_sync(0xffffffffu, v, 1 << o));
    return v;
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
__device__ __forceinline__ uint2 codes8(const float2 (&u)[4], int fmt, float one) {
    if (fmt == kI8) return codes8_i8(u, one);
    return make_uint2(e4m3_pair(u[0].x, u[0].y) | e4m3_pair(u[1].x, u[1].y) << 16,
                      e4m3_pair(u[2].x, u[2].y) | e4m3_pair(u[3].x, u[3].y) << 16);
}

// Sum over a row group of `s` and maximum (NaN kept) of `m`, through this
// group's scratch of [2][2][WPR] floats under its named barrier; the same bits
// on every thread.
template <int TPR, bool MAX>
__device__ __forceinline__ void group_sum_max(float &s, float &m, float *scratch, int &parity, int bar_id) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if constexpr (MAX) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if constexpr (TPR > 32) {
        constexpr int WPR = TPR / 32;
        const int wig = (threadIdx.x % TPR) >> 5, lane = threadIdx.x & 31;
        float2 *buf = reinterpret_cast<float2 *>(scratch) + parity * WPR;
        if (lane == 0) buf[wig] = make_float2(s, MAX ? m : 0.f);
        named_sync(bar_id, TPR);
        s = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float2 b = buf[w];
            s += b.x;
            if constexpr (MAX) m = fmax_nan(m, b.y);
        }
        parity ^= 1;
    }
}

// OUT 0: y in ydt; 1: 8-bit rows.  CK: the checkpoint too.
template <bool LN, int XT, int TPR, int VPT, int NT, int MINB, int OUT, bool CK>
__global__ void __launch_bounds__(NT, MINB) q8_fwd_rows(const Q8FwdParams p) {
    static_assert(NT % TPR == 0 && TPR % 32 == 0 && NT / TPR < 16, "row groups");
    constexpr int RPC = NT / TPR, WPR = TPR / 32;
    __shared__ __align__(16) float scratch_all[RPC * 4 * WPR];
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    float *scratch = scratch_all + grp * 4 * WPR;
    const int64_t nc = p.N / 8;
    const float n = (float)p.N;
    const bool full = nc == (int64_t)TPR * VPT;  // every thread holds VPT chunks (uniform)
    const int xes = XT == kF32 ? 4 : 2;
    const float qmax = q8_max(p.qfmt);
    const int qlg = p.qg - 3, clg = p.cg - 3;  // log2 of the lanes of a group
    int parity = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPC + grp; row < p.M; row += (int64_t)gridDim.x * RPC) {
        const unsigned char *xr = static_cast<const unsigned char *>(p.x) + row * p.ldx * xes;
        float2 v[VPT][4];  // h; RMSNorm's 8-bit output: h * gamma
        {
            Raw8<XT> xw[VPT], rw[VPT];
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (k * TPR + t < nc) xw[k] = ld_raw8<XT>(xr, k * TPR + t);
            if (p.res) {
                const unsigned char *rr = static_cast<const unsigned char *>(p.res) + row * p.ldr * xes;
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (k * TPR + t < nc) rw[k] = ld_raw8<XT>(rr, k * TPR + t);
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (k * TPR + t < nc) {
                    unpack8<XT>(xw[k], v[k]);
                    if (p.res) {
                        float2 r8[4];
                        unpack8<XT>(rw[k], r8);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[k][i] = round2<XT>(f2add(v[k][i], r8[i]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[k][i] = f2s(0.f);
                }
            }
        }
        if (p.h) {
            unsigned char *hr = static_cast<unsigned char *>(p.h) + row * p.ldh * xes;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (k * TPR + t < nc) st8p(hr, 8 * (int64_t)(k * TPR + t), XT, v[k]);
        }
        if constexpr (CK) {
            uint8_t *cr = p.c + row * p.ldc;
            float *cs = p.cs + row * p.ldcs;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = k * TPR + t;
                float top = -INFINITY, low = INFINITY;
                if (c < nc) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        top = fmax_nan(top, fmax_nan(v[k][i].x, v[k][i].y));
                        low = fmin_nan(low, fmin_nan(v[k][i].x, v[k][i].y));
                    }
                }
                const CkGroup g = ck_group(lanes_max(top, clg), lanes_min(low, clg));
                if (c < nc) {
                    const float2 nm = f2s(-g.mid), inv = f2s(g.inv);
                    float2 u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = f2mul(f2add(v[k][i], nm), inv);
                    *reinterpret_cast<uint2 *>(cr + 8 * c) = codes8_i8(u, p.one);
                    if ((c & ((1 << clg) - 1)) == 0)
                        *reinterpret_cast<float2 *>(cs + 2 * (c >> clg)) = make_float2(g.scale, g.mid);
                }
            }
        }
        float2 a2 = f2s(0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) a2 = LN ? f2add(a2, v[k][i]) : f2fma(v[k][i], v[k][i], a2);
        float acc = a2.x + a2.y, unused = 0.f;

        if constexpr (!LN && OUT == 1) {
            // t = h * gamma
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (k * TPR + t < nc) {
                    float2 g8[4];
                    par8g(p.gamma, k * TPR + t, p.pdt, 1.f, g8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[k][i] = f2mul(v[k][i], g8[i]);
                }
            uint8_t *qr = p.q + row * p.ldq;
            float amax[VPT];
#pragma unroll
            for (int k = 0; k < VPT; ++k) amax[k] = amax8(v[k]);
            if (p.qg >= 0) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    amax[k] = lanes_max(amax[k], qlg);
                    const float2 inv = f2s(q8_inv(amax[k], qmax));
                    float2 u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = f2mul(v[k][i], inv);
                    if (k * TPR + t < nc) *reinterpret_cast<uint2 *>(qr + 8 * (k * TPR + t)) = codes8(u, p.qfmt, p.one);
                }
                group_sum_max<TPR, false>(acc, unused, scratch, parity, 1 + grp);
                const float rstd = rsqrtf(acc / n + p.eps);
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int c = k * TPR + t;
                    if (c < nc && (c & ((1 << qlg) - 1)) == 0)
                        p.qs[row * p.qs_row + (c >> qlg) * p.qs_grp] = q8_scale(amax[k], rstd, qmax);
                }
                if (t == 0 && p.rstd) p.rstd[row] = rstd;
            } else {
                float m = amax[0];
#pragma unroll
                for (int k = 1; k < VPT; ++k) m = fmax_nan(m, amax[k]);
                group_sum_max<TPR, true>(acc, m, scratch, parity, 1 + grp);
                const float rstd = rsqrtf(acc / n + p.eps);
                const float2 inv = f2s(q8_inv(m, qmax));
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    float2 u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = f2mul(v[k][i], inv);
                    if (k * TPR + t < nc) *reinterpret_cast<uint2 *>(qr + 8 * (k * TPR + t)) = codes8(u, p.qfmt, p.one);
                }
                if (t == 0) {
                    p.qs[row * p.qs_row] = q8_scale(m, rstd, qmax);
                    if (p.rstd) p.rstd[row] = rstd;
                }
            }
            continue;
        }

        float mean = 0.f;
        if constexpr (LN) {
            if (full) {
                constexpr float kC = (float)(VPT * 8);
                mean = acc * (1.f / kC);
                const float2 nm = f2s(-mean);
                float2 q2 = f2s(0.f);
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 d = f2add(v[k][i], nm);
                        q2 = f2fma(d, d, q2);
                    }
                acc = q2.x + q2.y;
                group_meanvar_equal<TPR>(mean, acc, kC, scratch, parity, 1 + grp);
            } else {
                group_sum_max<TPR, false>(acc, unused, scratch, parity, 1 + grp);
                mean = acc / n;
                const float2 nm = f2s(-mean);
                float2 q2 = f2s(0.f);
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (k * TPR + t >= nc) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 d = f2add(v[k][i], nm);
                        q2 = f2fma(d, d, q2);
                    }
                }
                acc = q2.x + q2.y;
                group_sum_max<TPR, false>(acc, unused, scratch, parity, 1 + grp);
            }
        } else {
            group_sum_max<TPR, false>(acc, unused, scratch, parity, 1 + grp);
        }
        const float rstd = rsqrtf(acc / n + p.eps);
        if (t == 0) {
            if (p.rstd) p.rstd[row] = rstd;
            if (LN && p.mean) p.mean[row] = mean;
        }
        const float2 nm = f2s(-mean), rs = f2s(rstd);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = k * TPR + t;
            float2 o[4];
            if (c < nc) {
                float2 g8[4];
                par8g(p.gamma, c, p.pdt, 1.f, g8);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = f2mul(f2mul(LN ? f2add(v[k][i], nm) : v[k][i], rs), g8[i]);
                if (LN && p.beta) {
                    float2 b8[4];
                    par8g(p.beta, c, p.pdt, 0.f, b8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = f2add(o[i], b8[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = f2s(0.f);
            }
            if constexpr (OUT == 0) {
                if (c < nc) st8p(row_ptr(p.y, row, p.ldy, p.ydt), 8 * (int64_t)c, p.ydt, o);
            } else if (p.qg >= 0) {
                const float amax = lanes_max(amax8(o), qlg);
                const float2 inv = f2s(q8_inv(amax, qmax));
                if (c < nc) {
                    float2 u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = f2mul(o[i], inv);
                    *reinterpret_cast<uint2 *>(p.q + row * p.ldq + 8 * c) = codes8(u, p.qfmt, p.one);
                    if ((c & ((1 << qlg) - 1)) == 0)
                        p.qs[row * p.qs_row + (c >> qlg) * p.qs_grp] = q8_scale(amax, 1.f, qmax);
                }
            } else {
                m = fmax_nan(m, amax8(o));
#pragma unroll
                for (int i = 0; i < 4; ++i) v[k][i] = o[i];
            }
        }
        if constexpr (OUT == 1) {
            if (p.qg < 0) {
                group_sum_max<TPR, true>(unused, m, scratch, parity, 1 + grp);
                const float2 inv = f2s(q8_inv(m, qmax));
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    float2 u[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = f2mul(v[k][i], inv);
                    if (k * TPR + t < nc)
                        *reinterpret_cast<uint2 *>(p.q + row * p.ldq + 8 * (k * TPR + t)) = codes8(u, p.qfmt, p.one);
                }
                if (t == 0) p.qs[row * p.qs_row] = q8_scale(m, 1.f, qmax);
            }
        }
    }
}

}  // namespace gbn
