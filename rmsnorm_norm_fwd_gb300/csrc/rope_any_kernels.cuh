// rope_any_kernels.cuh -- the head operators element by element: any head
// size up to 1024, alignment, strides and types.
//
// L lanes hold a head, each C slots of two elements, slot i of lane l being
// number j = i L + l of the head: the elements of rotated pair j, or behind the
// rotated pairs two elements that are not (rot + u and rot + rest + u, the last
// of which may be missing).  So the rotation needs no exchange here either, and
// the lanes' loads of a slot are side by side.  Cosines, sines and parameters
// lie in shared memory in the order of the lanes' slots.
//
// What bounds it: instructions, 35 an element in the forward (16384 tokens of 40
// heads of 98 bf16 106 us, 36% of the copy rate's time) and 61 in the backward (161
// us): a load, a store and a conversion for each element, where the kernels on
// vectors take one of each for four to eight, and register spills: 16 elements a
// lane with coefficients or sums, and three types in one kernel, are more than 128
// registers (bytes of stores and loads: rotation 36, 72; RMSNorm 72, 144, its
// backward 104, 144; LayerNorm 148, 360, its backward 372, 620; with 16 slots three
// of the five spill at 255 registers).  A warp a head, without the next pass ahead,
// measured 319 and 837 us.
#pragma once

#include "rope_vec_kernels.cuh"

namespace gbn {

template <int L, int C> struct RopeSlots {
    static constexpr int N = L * C;
    uint32_t at[C];           // the two elements, 16 bits each
    uint32_t has_a, has_b, turned;  // one bit a slot
    __device__ __forceinline__ RopeSlots(const RopeParams &p, int sl) {
        has_a = has_b = turned = 0;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int j = i * L + sl, a = first(p, j), b = second(p, j);
            at[i] = (uint32_t)(a < 0 ? 0 : a) | (uint32_t)(b < 0 ? 0 : b) << 16;
            has_a |= (uint32_t)(a >= 0) << i;
            has_b |= (uint32_t)(b >= 0) << i;
            turned |= (uint32_t)(2 * j < p.rot) << i;
        }
    }
    // The elements of slot j of a head, -1 where there is none.
    static __device__ __forceinline__ int first(const RopeParams &p, int j) {
        const int half = p.rot / 2, rest = (p.D - p.rot + 1) / 2;
        return j < half ? (p.inter ? 2 * j : j) : j < half + rest ? p.rot + j - half : -1;
    }
    static __device__ __forceinline__ int second(const RopeParams &p, int j) {
        const int half = p.rot / 2, rest = (p.D - p.rot + 1) / 2;
        if (j < half) return p.inter ? 2 * j + 1 : j + half;
        return j < half + rest && p.rot + rest + j - half < p.D ? p.rot + rest + j - half : -1;
    }
    // Where a value of slot j lies in shared memory: planes of four slots of a lane.
    static __device__ __forceinline__ int place(int j) {
        const int i = j / L, sl = j % L;
        return (i >> 2) * (4 * L) + sl * 4 + (i & 3);
    }
    static __device__ __forceinline__ void get(const float *from, int sl, float2 (&f)[C / 2]) {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(from + i * (4 * L) + sl * 4);
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    }
    __device__ __forceinline__ int a(int i) const { return (int)(at[i] & 0xffffu); }
    __device__ __forceinline__ int b(int i) const { return (int)(at[i] >> 16); }

    // A head's elements as stored (`in`: it is there), zeros where there are none.
    __device__ __forceinline__ void load(const char *q, int dt, bool in, uint32_t (&ra)[C], uint32_t (&rb)[C]) const {
#pragma unroll
        for (int i = 0; i < C; ++i) ra[i] = rb[i] = 0;
        if (!in) return;
        if (dt == kF32) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if ((has_a >> i) & 1u) ra[i] = *reinterpret_cast<const uint32_t *>(q + a(i) * 4);
                if ((has_b >> i) & 1u) rb[i] = *reinterpret_cast<const uint32_t *>(q + b(i) * 4);
            }
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if ((has_a >> i) & 1u) ra[i] = *reinterpret_cast<const uint16_t *>(q + a(i) * 2);
                if ((has_b >> i) & 1u) rb[i] = *reinterpret_cast<const uint16_t *>(q + b(i) * 2);
            }
        }
    }
    static __device__ __forceinline__ void widen(const uint32_t (&r)[C], int dt, float2 (&f)[C / 2]) {
        if (dt == kF32) {
#pragma unroll
            for (int i = 0; i < C / 2; ++i)
                f[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        } else if (dt == kBF16) {
#pragma unroll
            for (int i = 0; i < C / 2; ++i)
                f[i] = make_float2(__uint_as_float(r[2 * i] << 16), __uint_as_float(r[2 * i + 1] << 16));
        } else {
#pragma unroll
            for (int i = 0; i < C / 2; ++i)
                f[i] = make_float2(__half2float(__ushort_as_half((unsigned short)r[2 * i])),
                                   __half2float(__ushort_as_half((unsigned short)r[2 * i + 1])));
        }
    }
    __device__ __forceinline__ void store(char *q, int dt, const float2 (&fa)[C / 2], const float2 (&fb)[C / 2]) const {
        auto one = [&](int e, float v) {
            if (dt == kF32) *reinterpret_cast<float *>(q + e * 4) = v;
            else if (dt == kBF16) *reinterpret_cast<__nv_bfloat16 *>(q + e * 2) = __float2bfloat16_rn(v);
            else *reinterpret_cast<__half *>(q + e * 2) = __float2half_rn(v);
        };
        auto all = [&] {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if ((has_a >> i) & 1u) one(a(i), i & 1 ? fa[i / 2].y : fa[i / 2].x);
                if ((has_b >> i) & 1u) one(b(i), i & 1 ? fb[i / 2].y : fb[i / 2].x);
            }
        };
        if (dt == kF32) all();
        else if (dt == kBF16) all();
        else all();
    }
    // v, zero in the slots that a mask does not have.
    static __device__ __forceinline__ void keep(uint32_t mask, float2 (&v)[C / 2]) {
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            v[i].x = (mask >> (2 * i)) & 1u ? v[i].x : 0.f;
            v[i].y = (mask >> (2 * i + 1)) & 1u ? v[i].y : 0.f;
        }
    }
    // Parameters of both tensors in the order of the slots: [a, b][N].
    static __device__ __forceinline__ void parameters(const RopeParams &p, float *to, const void *row, float none) {
        for (int j = threadIdx.x; j < N; j += kRopeCTA) {
            const int a = first(p, j), b = second(p, j);
            to[place(j)] = row && a >= 0 ? ld1(row, a, p.pdt) : none;
            to[N + place(j)] = row && b >= 0 ? ld1(row, b, p.pdt) : none;
        }
    }
};

// Cosines and sines of a warp's token, in the order of the slots; the frequencies of the call.
template <int L, int C> struct RopeSlotTable {
    static constexpr int N = L * C, PER = (N + 31) / 32;
    float c[N], s[N];
    __device__ __forceinline__ void ones(int lane, int rot) {
        for (int j = rot / 2 + lane; j < N; j += 32) {
            c[RopeSlots<L, C>::place(j)] = 1.f;
            s[RopeSlots<L, C>::place(j)] = 0.f;
        }
    }
    __device__ __forceinline__ void put(const uint64_t *turns, const float *bad, const RopeParams &p, int64_t pos,
                                        int lane) {
        // sixteen at once are more code than the loop bears: backward of heads of 602 160 us, 130 us with two
        constexpr int AT_ONCE = PER > 8 ? 2 : PER;
        __syncwarp();  // the last token's have been read
#pragma unroll AT_ONCE
        for (int i = 0; i < PER; ++i) {
            const int j = lane + 32 * i;
            const bool in = 2 * j < p.rot;
            const int64_t at = __shfl_sync(0xffffffffu, (long long)pos, in ? (int)rope_axis(p, j) : 0);
            if (in) {
                float cs, sn;
                rope_sincos((uint64_t)at * turns[j], p.sign, &cs, &sn);
                c[RopeSlots<L, C>::place(j)] = cs + bad[j];
                s[RopeSlots<L, C>::place(j)] = sn + bad[j];
            }
        }
        __syncwarp();
    }
};

// Dynamic shared memory of a CTA: tables, frequencies, then parameters ([queries, keys][gamma, beta][a, b][N]).
template <int L, int C> struct RopeAnySmem {
    RopeSlotTable<L, C> tables[kRopeWarps];
    uint64_t turns[L * C];
    float bad[L * C];
    float par[8 * L * C];
    __device__ __forceinline__ void fill(const RopeParams &p) {
        for (int j = threadIdx.x; 2 * j < p.rot; j += kRopeCTA) {
            bool b;
            turns[j] = rope_turns<false>(__ldg(p.inv_freq + j), &b);
            bad[j] = b ? __int_as_float(0x7fffffff) : 0.f;
        }
    }
};

template <bool LN, int L, int C> struct RopeAnyBwdSmem {
    RopeAnySmem<L, C> sm;
    RopeAside<C / 2 * (LN ? 2 : 1)> asides[kRopeWarps];
};

template <int MODE, int L, int C, int MINB>
__global__ void __launch_bounds__(kRopeCTA, MINB) rope_fwd_any(const __grid_constant__ RopeParams p) {
    constexpr int G = 32 / L, H = C / 2, N = L * C;
    using Slots = RopeSlots<L, C>;
    extern __shared__ __align__(16) unsigned char rope_smem[];
    RopeAnySmem<L, C> &sm = *reinterpret_cast<RopeAnySmem<L, C> *>(rope_smem);
    const int lane = threadIdx.x & 31, sl = lane % L, grp = lane / L;
    RopeSlotTable<L, C> &tab = sm.tables[threadIdx.x >> 5];
    RopeCursor<G> w(p, grp);
    const Slots ch(p, sl);
    const int xes = esize(p.xdt), yes = esize(p.ydt);
    auto at = [&](const RopeCursor<G> &c, const RopeHeads &t, int es) {
        return static_cast<char *>(t.p) + (c.b * t.batch + c.s * t.token + c.head(p) * t.head) * es;
    };
    uint32_t ra[C], rb[C];
    if (w.left) ch.load(at(w, p.x[w.r], xes), p.xdt, w.hl > 0, ra, rb);
    int64_t pos = w.left ? rope_position(p, w, lane) : 0;
    sm.fill(p);
    tab.ones(lane, p.rot);
    if constexpr (MODE != kRopeOnly) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            Slots::parameters(p, sm.par + r * 4 * N, p.gamma[r], 1.f);
            if constexpr (MODE == kRopeLn) Slots::parameters(p, sm.par + r * 4 * N + 2 * N, p.beta[r], 0.f);
        }
    }
    __syncthreads();
    if (!w.left) return;
    const float inv = 1.f / (float)p.D;
    int turn = 2;  // 2: another token's angles, 1: another tensor's coefficients
    float2 ca[H], sa[H], cb[H], sb[H], ba[H], bb[H];
    while (true) {
        float2 va[H], vb[H];
        Slots::widen(ra, p.xdt, va);
        Slots::widen(rb, p.xdt, vb);
        if (turn == 2) tab.put(sm.turns, sm.bad, p, pos, lane);
        if (turn) {
            const float *par = sm.par + w.r * 4 * N;
            float2 ga[H], gb[H], c[H], s[H];
            Slots::get(tab.c, sl, c);
            Slots::get(tab.s, sl, s);
            if constexpr (MODE != kRopeOnly) {
                Slots::get(par, sl, ga);
                Slots::get(par + N, sl, gb);
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) ga[i] = gb[i] = f2s(1.f);
            }
            if constexpr (MODE == kRopeLn) {
                Slots::get(par + 2 * N, sl, ba);
                Slots::get(par + 3 * N, sl, bb);
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                ca[i] = f2mul(ga[i], c[i]);
                cb[i] = f2mul(gb[i], c[i]);
                sa[i] = f2mul(gb[i], make_float2(-s[i].x, -s[i].y));
                sb[i] = f2mul(ga[i], s[i]);
                if constexpr (MODE == kRopeLn) {
                    // beta turned; where there is no partner it takes nothing from another, as x below
                    const float2 va = ba[i], vb = bb[i];
                    auto turned = [&](float own, float other, float cc, float ss, int slot) {
                        return (ch.turned >> slot) & 1u ? own * cc + other * ss : own;
                    };
                    ba[i].x = turned(va.x, vb.x, c[i].x, -s[i].x, 2 * i);
                    ba[i].y = turned(va.y, vb.y, c[i].y, -s[i].y, 2 * i + 1);
                    bb[i].x = turned(vb.x, va.x, c[i].x, s[i].x, 2 * i);
                    bb[i].y = turned(vb.y, va.y, c[i].y, s[i].y, 2 * i + 1);
                }
            }
            Slots::keep(ch.turned, sa);
            Slots::keep(ch.turned, sb);
        }
        const bool in = w.hl > 0;
        char *y = at(w, p.y[w.r], yes);
        const int64_t stat = w.stat(p);
        turn = w.next(p, grp);
        if (w.left) {
            ch.load(at(w, p.x[w.r], xes), p.xdt, w.hl > 0, ra, rb);
            if (turn == 2) pos = rope_position(p, w, lane);
        }
        if constexpr (MODE != kRopeOnly) {
            float mean = 0.f;
            if constexpr (MODE == kRopeLn) {
                float2 t = f2s(0.f);
#pragma unroll
                for (int i = 0; i < H; ++i) t = f2add(t, f2add(va[i], vb[i]));
                float sum[1] = {t.x + t.y};
                group_sum<L, 1>(sum);
                mean = sum[0] * inv;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    va[i] = f2add(va[i], f2s(-mean));
                    vb[i] = f2add(vb[i], f2s(-mean));
                }
                Slots::keep(ch.has_a, va);
                Slots::keep(ch.has_b, vb);
            }
            float2 t = f2s(0.f);
#pragma unroll
            for (int i = 0; i < H; ++i) t = f2fma(va[i], va[i], f2fma(vb[i], vb[i], t));
            float sq[1] = {t.x + t.y};
            group_sum<L, 1>(sq);
            const float rstd = rsqrtf(sq[0] * inv + p.eps);
            if (sl == 0 && in) {
                if (p.rstd) p.rstd[stat] = rstd;
                if (MODE == kRopeLn && p.mean) p.mean[stat] = mean;
            }
#pragma unroll
            for (int i = 0; i < H; ++i) {
                va[i] = f2mul(va[i], f2s(rstd));
                vb[i] = f2mul(vb[i], f2s(rstd));
            }
        }
        float2 ta[H], tb[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            ta[i] = vb[i];
            tb[i] = va[i];
        }
        if (p.rot < p.D) {  // an element that is not rotated takes nothing from another, not even a NaN
            Slots::keep(ch.turned, ta);
            Slots::keep(ch.turned, tb);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) {
            va[i] = f2fma(va[i], ca[i], MODE == kRopeLn ? f2fma(ta[i], sa[i], ba[i]) : f2mul(ta[i], sa[i]));
            vb[i] = f2fma(vb[i], cb[i], MODE == kRopeLn ? f2fma(tb[i], sb[i], bb[i]) : f2mul(tb[i], sb[i]));
        }
        if (in) ch.store(y, p.ydt, va, vb);
        if (!w.left) return;
    }
}

template <bool LN, int L, int C, int MINB>
__global__ void __launch_bounds__(kRopeCTA, MINB) rope_bwd_any(const __grid_constant__ RopeParams p) {
    pdl_launch_dependents();  // the column reduce waits for this grid's completion
    constexpr int G = 32 / L, H = C / 2, N = L * C;
    using Slots = RopeSlots<L, C>;
    using Aside = RopeAside<H * (LN ? 2 : 1)>;
    extern __shared__ __align__(16) unsigned char rope_smem[];  // RopeAnyBwdSmem, then the column sums [kRopeWarps][D]
    RopeAnyBwdSmem<LN, L, C> &both = *reinterpret_cast<RopeAnyBwdSmem<LN, L, C> *>(rope_smem);
    RopeAnySmem<L, C> &sm = both.sm;
    float *acc = reinterpret_cast<float *>(&both + 1);
    const int lane = threadIdx.x & 31, sl = lane % L, grp = lane / L, warp = threadIdx.x >> 5;
    RopeSlotTable<L, C> &tab = sm.tables[warp];
    Aside &aside = both.asides[warp];
    RopeCursor<G> w(p, grp);
    const Slots ch(p, sl);
    const int xes = esize(p.xdt), ges = esize(p.ydt);
    auto at = [&](const RopeHeads &t, int es) {
        return static_cast<char *>(t.p) + (w.b * t.batch + w.s * t.token + w.head(p) * t.head) * es;
    };
    uint32_t xa[C], xb[C], ga[C], gb[C];
    float rstd = 0.f, mean = 0.f;
    auto load = [&] {
        ch.load(at(p.x[w.r], xes), p.xdt, w.hl > 0, xa, xb);
        ch.load(at(p.g[w.r], ges), p.ydt, w.hl > 0, ga, gb);
        rstd = __ldg(p.rstd + w.stat(p));
        if constexpr (LN) mean = __ldg(p.mean + w.stat(p));
    };
    if (w.left) load();
    int64_t pos = w.left ? rope_position(p, w, lane) : 0;
    sm.fill(p);
    tab.ones(lane, p.rot);
#pragma unroll
    for (int i = 0; i < 2; ++i) Slots::parameters(p, sm.par + i * 4 * N, p.gamma[i], 1.f);
    __syncthreads();
    float2 da[H], db[H], ea[H], eb[H];
#pragma unroll
    for (int i = 0; i < H; ++i) da[i] = db[i] = ea[i] = eb[i] = f2s(0.f);
    aside.clear(lane);
    auto swap = [&] {
        aside.template swap<H / 2>(da, 0, lane);
        aside.template swap<H / 2>(db, H / 2, lane);
        if constexpr (LN) {
            aside.template swap<H / 2>(ea, H, lane);
            aside.template swap<H / 2>(eb, H + H / 2, lane);
        }
    };
    if (w.left) {
        const float inv = 1.f / (float)p.D;
        int turn = 2;
        while (true) {
            float2 va[H], vb[H], ta[H], tb[H];
            const int r = w.r;
            const float *par = sm.par + r * 4 * N;
            if (turn == 2) tab.put(sm.turns, sm.bad, p, pos, lane);
            Slots::widen(ga, p.ydt, va);
            Slots::widen(gb, p.ydt, vb);
            {  // the gradient turned back (the sign of s is the transpose's)
                float2 c[H], s[H];
                Slots::get(tab.c, sl, c);
                Slots::get(tab.s, sl, s);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    ta[i] = vb[i];
                    tb[i] = va[i];
                }
                if (p.rot < p.D) {
                    Slots::keep(ch.turned, ta);
                    Slots::keep(ch.turned, tb);
                }
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    ta[i] = f2fma(va[i], c[i], f2mul(make_float2(-ta[i].x, -ta[i].y), s[i]));
                    tb[i] = f2fma(vb[i], c[i], f2mul(tb[i], s[i]));
                }
            }
            Slots::widen(xa, p.xdt, va);
            Slots::widen(xb, p.xdt, vb);
            const float rs = rstd, mu = mean;
            const bool in = w.hl > 0;
            char *y = at(p.y[r], xes);
            turn = w.next(p, grp);
            if (w.left) {
                load();
                if (turn == 2) pos = rope_position(p, w, lane);
            }
            float2 dot = f2s(0.f), sum = f2s(0.f), wa[H], wb[H];
            Slots::get(par, sl, wa);
            Slots::get(par + N, sl, wb);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if constexpr (LN) {
                    va[i] = f2add(va[i], f2s(-mu));
                    vb[i] = f2add(vb[i], f2s(-mu));
                    ea[i] = f2add(ea[i], ta[i]);
                    eb[i] = f2add(eb[i], tb[i]);
                }
                va[i] = f2mul(va[i], f2s(rs));
                vb[i] = f2mul(vb[i], f2s(rs));
                if (in) {  // zeros times another head's infinite statistics are NaN
                    da[i] = f2fma(ta[i], va[i], da[i]);
                    db[i] = f2fma(tb[i], vb[i], db[i]);
                }
                ta[i] = f2mul(ta[i], wa[i]);
                tb[i] = f2mul(tb[i], wb[i]);
                dot = f2fma(ta[i], va[i], f2fma(tb[i], vb[i], dot));
                if constexpr (LN) sum = f2add(sum, f2add(ta[i], tb[i]));
            }
            float v[LN ? 2 : 1];
            v[0] = dot.x + dot.y;
            if constexpr (LN) v[1] = sum.x + sum.y;
            group_sum<L, LN ? 2 : 1>(v);
            const float2 c2 = f2s(-v[0] * inv * rs), c1 = f2s(LN ? -v[LN ? 1 : 0] * inv * rs : 0.f);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                ta[i] = f2fma(va[i], c2, LN ? f2fma(ta[i], f2s(rs), c1) : f2mul(ta[i], f2s(rs)));
                tb[i] = f2fma(vb[i], c2, LN ? f2fma(tb[i], f2s(rs), c1) : f2mul(tb[i], f2s(rs)));
            }
            if (in) ch.store(y, p.xdt, ta, tb);
            if (w.left ? w.r != r : r) swap();  // at the end the queries' are in the registers
            if (!w.left) break;
        }
    }
    // the sums of the groups of lanes of a warp, then of the CTA's warps
    char *mine = reinterpret_cast<char *>(acc + warp * p.D);
    auto columns = [&](float2 (&u)[H], float2 (&v)[H]) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < H; ++i) {
                u[i].x += __shfl_xor_sync(0xffffffffu, u[i].x, o);
                u[i].y += __shfl_xor_sync(0xffffffffu, u[i].y, o);
                v[i].x += __shfl_xor_sync(0xffffffffu, v[i].x, o);
                v[i].y += __shfl_xor_sync(0xffffffffu, v[i].y, o);
            }
        if (grp == 0) ch.store(mine, kF32, u, v);
    };
    for (int r = 0; r < (p.heads[1] ? 2 : 1); ++r) {
        if (r) swap();
        columns(da, db);
        rope_partial(p, acc, 0, r);
        if constexpr (LN) {
            columns(ea, eb);
            rope_partial(p, acc, 1, r);
        }
    }
}

// out[c] = sum over the P partial rows of ws [2][P][N] (block blockIdx.y), 32
// columns a CTA, warp w the rows w, w + 32, ..., then the warps in order.  A head
// has few columns, so one CTA for all of them (as for long rows) would read the
// rows one latency after another.  __ldcg: ws is written while this grid may
// already be resident, and the read-only path (__ldg) is for memory that nobody
// writes meanwhile.
constexpr int kRopeColumnsCTA = 1024;
__global__ void __launch_bounds__(kRopeColumnsCTA)
    rope_columns(const float *ws, int P, int N, float *out0, float *out1) {
    __shared__ float part[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float *out = blockIdx.y ? out1 : out0;
    pdl_wait_primary();  // launched right behind the kernel that writes ws
    if (!out) return;
    const float *from = ws + (int64_t)blockIdx.y * P * N + col;
    float v = 0.f;
    if (col < N) {
        constexpr int AT_ONCE = 10;  // 304 rows (two CTAs an SM) are one round
        for (int p0 = warp; p0 < P; p0 += 32 * AT_ONCE) {
            float a[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) a[i] = p0 + 32 * i < P ? __ldcg(from + (int64_t)(p0 + 32 * i) * N) : 0.f;
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) v += a[i];
        }
    }
    part[warp][lane] = v;
    __syncthreads();
    if (warp || col >= N) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) v += part[i][lane];
    out[col] = v;
}

}  // namespace gbn
