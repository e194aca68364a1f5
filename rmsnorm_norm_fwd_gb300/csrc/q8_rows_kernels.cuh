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

// Maximum and minimum of the chunks of a group, one chunk a lane, over its
// 2^lg lanes; `ok` false: no chunk here.
template <int XT>
__device__ __forceinline__ void lanes_range(const Raw8<XT> &r, bool ok, int lg, float &top, float &low) {
    if constexpr (XT == kF32) {
        float2 f[4];
        unpack8<XT>(r, f);
        top = -INFINITY, low = INFINITY;
        if (ok) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                top = fmax_nan(top, fmax_nan(f[i].x, f[i].y));
                low = fmin_nan(low, fmin_nan(f[i].x, f[i].y));
            }
        }
        top = lanes_max(top, lg);
        low = lanes_min(low, lg);
    } else {
        // on pairs of the stored type, then (max, -min) as one pair, so that a
        // butterfly step is one shuffle and one maximum
        using T2 = typename std::conditional<XT == kBF16, __nv_bfloat162, __half2>::type;
        const T2 *p = reinterpret_cast<const T2 *>(&r.v[0]);
        const T2 hi = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
        const T2 lo = __hmin2_nan(__hmin2_nan(p[0], p[1]), __hmin2_nan(p[2], p[3]));
        T2 m;
        m.x = __hmax_nan(hi.x, hi.y);
        m.y = __hneg(__hmin_nan(lo.x, lo.y));
        uint32_t w = *reinterpret_cast<const uint32_t *>(&m);
        constexpr uint32_t kLowest = XT == kBF16 ? 0xff80ff80u : 0xfc00fc00u;  // (-inf, -inf)
        if (!ok) w = kLowest;
#pragma unroll
        for (int o = 0; o < 5; ++o)
            if (o < lg) {
                const uint32_t v = __shfl_xor_sync(0xffffffffu, w, 1 << o);
                const T2 n = __hmax2_nan(*reinterpret_cast<const T2 *>(&w), *reinterpret_cast<const T2 *>(&v));
                w = *reinterpret_cast<const uint32_t *>(&n);
            }
        const T2 n = *reinterpret_cast<const T2 *>(&w);
        top = to_f(n.x);
        low = -to_f(n.y);
    }
}

// OUT 0: y in ydt; 1: 8-bit rows.  CK: the checkpoint too.
//
// A row stays in its storage type between the passes (half the registers of
// fp32 for 16-bit types, so that more rows are in flight) and is widened, and
// RMSNorm's product with gamma formed, again in each.
template <bool LN, int XT, int TPR, int VPT, int NT, int MINB, int OUT, bool CK>
__global__ void __launch_bounds__(NT, MINB) q8_fwd_rows(const Q8FwdParams p) {
    static_assert(NT % TPR == 0 && TPR % 32 == 0 && NT / TPR < 16, "row groups");
    constexpr int RPC = NT / TPR, WPR = TPR / 32;
    __shared__ __align__(16) float scratch_all[RPC * 4 * WPR];
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    float *scratch = scratch_all + grp * 4 * WPR;
    const int nc = (int)(p.N / 8);
    const float n = (float)p.N;
    const bool full = nc == TPR * VPT;  // every thread holds VPT chunks (uniform)
    constexpr int xes = XT == kF32 ? 4 : 2;
    const float qmax = q8_max(p.qfmt);
    const int qlg = p.qg - 3, clg = p.cg - 3;  // log2 of the lanes of a group
    int parity = 0;
    for (int64_t row = (int64_t)blockIdx.x * RPC + grp; row < p.M; row += (int64_t)gridDim.x * RPC) {
        Raw8<XT> h[VPT];
        const unsigned char *xr = static_cast<const unsigned char *>(p.x) + row * p.ldx * xes;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            h[k] = Raw8<XT>{};
            if (k * TPR + t < nc) h[k] = ld_raw8<XT>(xr, k * TPR + t);
        }
        if (p.res) {
            const unsigned char *rr = static_cast<const unsigned char *>(p.res) + row * p.ldr * xes;
            Raw8<XT> r[VPT];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                r[k] = Raw8<XT>{};
                if (k * TPR + t < nc) r[k] = ld_raw8<XT>(rr, k * TPR + t);
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float2 a[4], b[4];
                unpack8<XT>(h[k], a);
                unpack8<XT>(r[k], b);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = f2add(a[i], b[i]);
                h[k] = pack8<XT>(a);  // the sum rounded once to the storage type
            }
            if (p.h) {
                unsigned char *hr = static_cast<unsigned char *>(p.h) + row * p.ldh * xes;
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    if (k * TPR + t < nc) st_raw8<XT>(hr, k * TPR + t, h[k]);
            }
        }
        if constexpr (CK) {
            uint8_t *cr = p.c + row * p.ldc;
            float *cs = p.cs + row * p.ldcs;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = k * TPR + t;
                float top, low;
                lanes_range<XT>(h[k], c < nc, clg, top, low);
                const CkGroup g = ck_group(top, low);
                if (c < nc) {
                    const float2 nm = f2s(-g.mid), inv = f2s(g.inv);
                    float2 u[4];
                    unpack8<XT>(h[k], u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[i] = f2mul(f2add(u[i], nm), inv);
                    *reinterpret_cast<uint2 *>(cr + 8 * c) = codes8_i8(u, p.one);
                    if ((c & ((1 << clg) - 1)) == 0)
                        *reinterpret_cast<float2 *>(cs + 2 * (c >> clg)) = make_float2(g.scale, g.mid);
                }
            }
        }

        // ---------------------------------------------------------------- sums of the row
        uint8_t *qr = p.q + row * p.ldq;
        float *qs = p.qs + row * p.qs_row;
        float2 a2 = f2s(0.f);
        float m = 0.f, unused = 0.f;
        constexpr bool RQ = !LN && OUT == 1;  // codes of h * gamma
        float amax[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = k * TPR + t;
            float2 v[4];
            unpack8<XT>(h[k], v);
#pragma unroll
            for (int i = 0; i < 4; ++i) a2 = LN ? f2add(a2, v[i]) : f2fma(v[i], v[i], a2);
            if constexpr (RQ) {
                if (c < nc && p.gamma) {
                    float2 g8[4];
                    par8g(p.gamma, c, p.pdt, 1.f, g8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = f2mul(v[i], g8[i]);
                }
                amax[k] = amax8(v);
                if (p.qg >= 0) {
                    amax[k] = lanes_max(amax[k], qlg);
                    const float2 inv = f2s(q8_inv(amax[k], qmax));
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = f2mul(v[i], inv);
                    if (c < nc) *reinterpret_cast<uint2 *>(qr + 8 * c) = codes8(v, p.qfmt, p.one);
                } else {
                    m = fmax_nan(m, amax[k]);
                }
            }
        }
        float acc = a2.x + a2.y, mean = 0.f;
        if constexpr (LN) {
            float2 q2 = f2s(0.f);
            if (full) {
                constexpr float kC = (float)(VPT * 8);
                mean = acc * (1.f / kC);
            } else {
                group_sum_max<TPR, false>(acc, unused, scratch, parity, 1 + grp);
                mean = acc / n;
            }
            const float2 nm = f2s(-mean);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (k * TPR + t >= nc) continue;
                float2 v[4];
                unpack8<XT>(h[k], v);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 d = f2add(v[i], nm);
                    q2 = f2fma(d, d, q2);
                }
            }
            acc = q2.x + q2.y;
            if (full) group_meanvar_equal<TPR>(mean, acc, (float)(VPT * 8), scratch, parity, 1 + grp);
            else group_sum_max<TPR, false>(acc, unused, scratch, parity, 1 + grp);
        } else {
            group_sum_max<TPR, RQ>(acc, m, scratch, parity, 1 + grp);
        }
        const float rstd = rsqrtf(acc / n + p.eps);
        if (t == 0) {
            if (p.rstd) p.rstd[row] = rstd;
            if (LN && p.mean) p.mean[row] = mean;
        }

        // ---------------------------------------------------------------- output
        const float2 nm = f2s(-mean), rs = f2s(rstd);
        // chunk k of y (RQ: of h * gamma); zeros past the row's end
        auto out8 = [&](int k, float2 (&o)[4]) {
            const int c = k * TPR + t;
            unpack8<XT>(h[k], o);
            if (c < nc) {
                if constexpr (LN) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = f2mul(f2add(o[i], nm), rs);
                } else if constexpr (!RQ) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = f2mul(o[i], rs);
                }
                if (p.gamma) {
                    float2 g8[4];
                    par8g(p.gamma, c, p.pdt, 1.f, g8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = f2mul(o[i], g8[i]);
                }
                if (LN && p.beta) {
                    float2 b8[4];
                    par8g(p.beta, c, p.pdt, 0.f, b8);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = f2add(o[i], b8[i]);
                }
            }
        };
        if constexpr (OUT == 0) {
            void *yr = row_ptr(p.y, row, p.ldy, p.ydt);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float2 o[4];
                out8(k, o);
                if (k * TPR + t < nc) st8p(yr, 8 * (int64_t)(k * TPR + t), p.ydt, o);
            }
        } else if (p.qg >= 0) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = k * TPR + t;
                if constexpr (!RQ) {
                    float2 o[4];
                    out8(k, o);
                    amax[k] = lanes_max(amax8(o), qlg);
                    const float2 inv = f2s(q8_inv(amax[k], qmax));
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[i] = f2mul(o[i], inv);
                    if (c < nc) *reinterpret_cast<uint2 *>(qr + 8 * c) = codes8(o, p.qfmt, p.one);
                }
                if (c < nc && (c & ((1 << qlg) - 1)) == 0)
                    qs[(c >> qlg) * p.qs_grp] = q8_scale(amax[k], RQ ? rstd : 1.f, qmax);
            }
        } else {
            if constexpr (!RQ) {
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    float2 o[4];
                    out8(k, o);
                    m = fmax_nan(m, amax8(o));
                }
                group_sum_max<TPR, true>(unused, m, scratch, parity, 1 + grp);
            }
            const float2 inv = f2s(q8_inv(m, qmax));
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float2 o[4];
                out8(k, o);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = f2mul(o[i], inv);
                if (k * TPR + t < nc) *reinterpret_cast<uint2 *>(qr + 8 * (k * TPR + t)) = codes8(o, p.qfmt, p.one);
            }
            if (t == 0) qs[0] = q8_scale(m, RQ ? rstd : 1.f, qmax);
        }
    }
}

}  // namespace gbn
