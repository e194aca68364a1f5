// rope_vec_kernels.cuh -- the head operators on vectors.
//
// A group of L lanes holds one head, 32 / L heads a warp and pass; a lane holds
// two chunks of V consecutive elements, one 8- or 16-byte vector each.  Where
// pair j is (j, j + rot / 2) the two chunks are partners (j..j+V-1 and the same
// behind rot / 2), where pairs are neighbours every chunk holds whole pairs; so
// the rotation needs no exchange, and a row sum is log2 L shuffles.
//
// The lanes of a warp share out the pairs of a token, put their cosines and
// sines into the warp's part of shared memory, and each lane takes those of its
// chunks: once a token, for all its heads.  gamma is folded into them,
//     y_a = n_a (gamma_a cos) - n_b (gamma_b sin),   y_b = n_b (gamma_b cos) + n_a (gamma_a sin),
// with n the values before gamma, so that an element costs a product with rstd
// and two with coefficients.
#pragma once

#include "rope_common.cuh"

namespace gbn {

// V elements as stored.
template <int XT, int V> struct RopeRaw;
template <> struct RopeRaw<kF32, 4> { uint4 v; };
template <> struct RopeRaw<kF16, 8> { uint4 v; };
template <> struct RopeRaw<kBF16, 8> { uint4 v; };
template <> struct RopeRaw<kF16, 4> { uint2 v; };
template <> struct RopeRaw<kBF16, 4> { uint2 v; };

__device__ __forceinline__ void rope_ld(const void *p, uint4 &v) { v = *static_cast<const uint4 *>(p); }
__device__ __forceinline__ void rope_ld(const void *p, uint2 &v) { v = *static_cast<const uint2 *>(p); }
__device__ __forceinline__ void rope_st(void *p, const uint4 &v) { *static_cast<uint4 *>(p) = v; }
__device__ __forceinline__ void rope_st(void *p, const uint2 &v) { *static_cast<uint2 *>(p) = v; }

template <int XT> __device__ __forceinline__ float2 rope_pair(uint32_t w) {
    if constexpr (XT == kBF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <int XT> __device__ __forceinline__ uint32_t rope_word(float2 f) {
    if constexpr (XT == kBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <int XT, int V> __device__ __forceinline__ void rope_unpack(const RopeRaw<XT, V> &r, float2 (&f)[V / 2]) {
    if constexpr (XT == kF32) {
        f[0] = make_float2(__uint_as_float(r.v.x), __uint_as_float(r.v.y));
        f[1] = make_float2(__uint_as_float(r.v.z), __uint_as_float(r.v.w));
    } else {
        f[0] = rope_pair<XT>(r.v.x);
        f[1] = rope_pair<XT>(r.v.y);
        if constexpr (V == 8) {
            f[2] = rope_pair<XT>(r.v.z);
            f[3] = rope_pair<XT>(r.v.w);
        }
    }
}
template <int XT, int V> __device__ __forceinline__ RopeRaw<XT, V> rope_pack(const float2 (&f)[V / 2]) {
    RopeRaw<XT, V> r;
    if constexpr (XT == kF32) {
        r.v = make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                         __float_as_uint(f[1].y));
    } else {
        r.v.x = rope_word<XT>(f[0]);
        r.v.y = rope_word<XT>(f[1]);
        if constexpr (V == 8) {
            r.v.z = rope_word<XT>(f[2]);
            r.v.w = rope_word<XT>(f[3]);
        }
    }
    return r;
}

// Asynchronous copies into the lane's own places of the ring: no other thread
// reads them, so that waiting for the lane's own groups is enough.  Lanes
// without an element fill with zeros (`from` is then any valid address).
__device__ __forceinline__ void rope_cp(void *to, const void *from, bool in, const uint4 &) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void rope_cp(void *to, const void *from, bool in, const uint2 &) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 8 : 0) : "memory");
}
__device__ __forceinline__ void rope_cp(void *to, const void *from, bool in, float) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ void rope_cp_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void rope_cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Row `row` of D parameters widened to fp32 into shared memory, a null row as `none`; every thread takes its share.
__device__ __forceinline__ void rope_param(float *to, const void *row, int D, int dt, float none) {
    for (int c = threadIdx.x; c < D; c += kRopeCTA) to[c] = row ? ld1(row, c, dt) : none;
}
// V values from shared memory.
template <int V> __device__ __forceinline__ void rope_get(const float *from, float2 (&f)[V / 2]) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const float4 v = reinterpret_cast<const float4 *>(from)[i];
        f[2 * i] = make_float2(v.x, v.y);
        f[2 * i + 1] = make_float2(v.z, v.w);
    }
}

// What is rotated, fixed at compile time where it is common: the whole head, as
// halves or as neighbours, or anything (read from the call, through selects).
enum RopeKind : int { kRopeHalves = 0, kRopeNeighbours = 1, kRopeSome = 2 };

// The two chunks of a lane: first elements, whether they are there, whether they are rotated, and their first pair.
template <int V, int L, int KIND> struct RopeChunks {
    int a, b, pa, pb;
    bool oka, okb, ra, rb;
    __device__ __forceinline__ RopeChunks(const RopeParams &p, int sl) {
        const int n = p.D / V, nr = p.rot / V;
        int ca, cb;
        if (KIND == kRopeNeighbours || (KIND == kRopeSome && p.inter)) {
            const int ns = (n + 1) / 2;
            ca = sl;
            cb = ns + sl;
            oka = sl < ns;
            okb = oka && cb < n;
            pa = ca * (V / 2);
            pb = cb * (V / 2);
        } else {
            const int half = nr / 2;
            ca = sl < half ? sl : nr + 2 * (sl - half);
            cb = sl < half ? sl + half : ca + 1;
            oka = ca < n;
            okb = cb < n;
            pa = pb = sl * V;
        }
        a = ca * V;
        b = cb * V;
        ra = oka && ca < nr;
        rb = okb && cb < nr;
        if (!oka) a = 0;  // lanes without a chunk stay inside the head
        if (!okb) b = 0;
        if (!ra) pa = V * L;
        if (!rb) pb = V * L;
    }
};

// The frequencies of a call in turns, once a CTA.
template <int V, int L> struct RopeTurns {
    static constexpr int N = V * L;
    static_assert(N <= kRopeCTA, "a pair a thread");
    uint64_t f[N];
    float bad[N];  // 0, or NaN where the frequency is not a number of turns
    __device__ __forceinline__ void fill(const RopeParams &p) {
        const int j = threadIdx.x;
        if (2 * j >= p.rot) return;
        bool b;
        f[j] = rope_turns(__ldg(p.inv_freq + j), &b);
        bad[j] = b ? __int_as_float(0x7fffffff) : 0.f;
    }
};
// A warp's cosines and sines: written by the lane that computed the pair, read by those whose chunks hold it.
template <int V, int L> struct RopeTable {
    static constexpr int N = V * L, PER = N / 32 > 0 ? N / 32 : 1;
    float c[N + V], s[N + V];  // the last V: what is not rotated
    __device__ __forceinline__ void ones(int lane) {
        if (lane < V) {
            c[N + lane] = 1.f;
            s[N + lane] = 0.f;
        }
    }
    // pos: lane a holds the position on axis a; axis: two bits for each of the lane's pairs lane, lane + 32, ...
    __device__ __forceinline__ void put(const RopeTurns<V, L> &turns, const RopeParams &p, int64_t pos, uint32_t axis,
                                        int lane) {
        __syncwarp();  // the last token's have been read
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = lane + 32 * i;
            const int64_t at = __shfl_sync(0xffffffffu, (long long)pos, (axis >> (2 * i)) & 3u);
            if (2 * j < p.rot) {
                float cs, sn;
                rope_sincos((uint64_t)at * turns.f[j], p.sign, &cs, &sn);
                c[j] = cs + turns.bad[j];
                s[j] = sn + turns.bad[j];
            }
        }
        __syncwarp();
    }
    static __device__ __forceinline__ uint32_t axes(const RopeParams &p, int lane) {
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (2 * (lane + 32 * i) < p.rot) a |= rope_axis(p, lane + 32 * i) << (2 * i);
        return a;
    }
};
// Lane a's position of the token at the walk, on axis a.
template <typename W> __device__ __forceinline__ int64_t rope_position(const RopeParams &p, const W &w, int lane) {
    if (lane >= p.axes) return 0;
    const int64_t q = w.b * p.pos_batch + w.s * p.pos_token + lane * p.pos_axis;
    return p.pos64 ? (int64_t)__ldg(static_cast<const long long *>(p.pos) + q)
                   : (int64_t)__ldg(static_cast<const int *>(p.pos) + q);
}

__device__ __forceinline__ float2 f2swap(float2 v) { return make_float2(v.y, v.x); }

template <int MODE, int XT, int V, int L, int KIND, int U, int MINB>
__global__ void __launch_bounds__(kRopeCTA, MINB) rope_fwd_vec(const __grid_constant__ RopeParams p) {
    constexpr int G = 32 / L, H = V / 2, ES = XT == kF32 ? 4 : 2, DEPTH = kRopeFwdDepth;
    using Table = RopeTable<V, L>;
    using Raw = RopeRaw<XT, V>;
    // rings, tables, frequencies, then gamma (and beta) of the queries and of the keys
    extern __shared__ __align__(16) unsigned char rope_smem[];
    const int lane = threadIdx.x & 31, sl = lane % L, grp = lane / L, warp = threadIdx.x >> 5;
    Raw(*ring)[U][2][32] = reinterpret_cast<Raw(*)[U][2][32]>(rope_smem) + warp * DEPTH;
    Table *tables = reinterpret_cast<Table *>(rope_smem + sizeof(Raw) * 64 * U * DEPTH * kRopeWarps);
    RopeTurns<V, L> &turns = *reinterpret_cast<RopeTurns<V, L> *>(tables + kRopeWarps);
    float *par = reinterpret_cast<float *>(&turns + 1);
    Table &tab = tables[warp];
    RopeTokens w(p), ahead = w;  // the pass worked on, the pass to load
    const RopeChunks<V, L, KIND> ch(p, sl);
    const int nq = p.passes[0];
    const bool fill_a = ch.oka, fill_b = ch.okb;
    // head of this lane's in a pass; past the last one it repeats that, unstored
    auto head = [&](int blk, int r, int u) { return (blk - (r ? nq : 0)) * (G * U) + u * G + grp; };
    auto load = [&](int slot) {
        if (ahead.left) {
            const int r = ahead.blk >= nq, last = p.heads[r] - 1;
            const char *x = static_cast<const char *>(p.x[r].p) + ahead.at(p.x[r]) * ES;
            const int64_t step = p.x[r].head * ES;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = head(ahead.blk, r, u);
                const char *q = x + (h < last ? h : last) * step;
                rope_cp(&ring[slot][u][0][lane], q + ch.a * ES, fill_a, Raw{}.v);
                rope_cp(&ring[slot][u][1][lane], q + ch.b * ES, fill_b, Raw{}.v);
            }
            ahead.next(p);
        }
        rope_cp_end();
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(i);
    int64_t pos = w.left ? rope_position(p, w, lane) : 0;
    const uint32_t axis = Table::axes(p, lane);
    turns.fill(p);
    tab.ones(lane);
    if constexpr (MODE != kRopeOnly) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            rope_param(par + r * p.D, p.gamma[r], p.D, p.pdt, 1.f);
            if constexpr (MODE == kRopeLn) rope_param(par + (2 + r) * p.D, p.beta[r], p.D, p.pdt, 0.f);
        }
    }
    __syncthreads();
    if (!w.left) return;
    const float inv = 1.f / (float)p.D;
    const bool inter = KIND == kRopeNeighbours || (KIND == kRopeSome && p.inter);
    float2 ca[H], sa[H], cb[H], sb[H], ba[H], bb[H];
    bool fresh = true, turn = true;  // another token's angles, another tensor's coefficients
    for (int slot = 0;; slot = slot == DEPTH - 1 ? 0 : slot + 1) {
        const int r = w.blk >= nq, h0 = head(w.blk, r, 0), heads = p.heads[r];
        char *y = static_cast<char *>(p.y[r].p) + w.at(p.y[r]) * ES;
        const int64_t stat = (w.b * p.S + w.s) * (p.heads[0] + p.heads[1]) + (r ? p.heads[0] : 0);
        const bool nf = w.next(p);
        if (fresh) tab.put(turns, p, pos, axis, lane);
        if (turn) {
            float2 ga[H], gb[H];
            if constexpr (MODE != kRopeOnly) {
                rope_get<V>(par + r * p.D + ch.a, ga);
                rope_get<V>(par + r * p.D + ch.b, gb);
            } else {
#pragma unroll
                for (int i = 0; i < H; ++i) ga[i] = gb[i] = f2s(1.f);
            }
            if constexpr (MODE == kRopeLn) {
                rope_get<V>(par + (2 + r) * p.D + ch.a, ba);
                rope_get<V>(par + (2 + r) * p.D + ch.b, bb);
            }
            if (inter) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    {
                        const float c = tab.c[ch.pa + i], s = tab.s[ch.pa + i];
                        ca[i] = make_float2(ga[i].x * c, ga[i].y * c);
                        sa[i] = make_float2(-ga[i].y * s, ga[i].x * s);
                        if constexpr (MODE == kRopeLn)
                            ba[i] = make_float2(ba[i].x * c - ba[i].y * s, ba[i].y * c + ba[i].x * s);
                    }
                    {
                        const float c = tab.c[ch.pb + i], s = tab.s[ch.pb + i];
                        cb[i] = make_float2(gb[i].x * c, gb[i].y * c);
                        sb[i] = make_float2(-gb[i].y * s, gb[i].x * s);
                        if constexpr (MODE == kRopeLn)
                            bb[i] = make_float2(bb[i].x * c - bb[i].y * s, bb[i].y * c + bb[i].x * s);
                    }
                }
            } else {
                float2 c[H], s[H];
                rope_get<V>(tab.c + ch.pa, c);
                rope_get<V>(tab.s + ch.pa, s);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    ca[i] = f2mul(ga[i], c[i]);
                    sa[i] = f2mul(gb[i], make_float2(-s[i].x, -s[i].y));
                    cb[i] = f2mul(gb[i], c[i]);
                    sb[i] = f2mul(ga[i], s[i]);
                    if constexpr (MODE == kRopeLn) {
                        const float2 v = ba[i];
                        ba[i] = make_float2(v.x * c[i].x - bb[i].x * s[i].x, v.y * c[i].y - bb[i].y * s[i].y);
                        bb[i] = make_float2(bb[i].x * c[i].x + v.x * s[i].x, bb[i].y * c[i].y + v.y * s[i].y);
                    }
                }
            }
            if constexpr (KIND == kRopeSome) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    sa[i] = ch.ra ? sa[i] : f2s(0.f);
                    sb[i] = ch.rb ? sb[i] : f2s(0.f);
                }
            }
        }
        if (w.left && nf) pos = rope_position(p, w, lane);
        rope_cp_wait<DEPTH - 1>();
        Raw ra[U], rb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            ra[u] = ring[slot][u][0][lane];
            rb[u] = ring[slot][u][1][lane];
        }
        load(slot);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * G;
            float2 va[H], vb[H];
            rope_unpack<XT, V>(ra[u], va);
            rope_unpack<XT, V>(rb[u], vb);
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
                        va[i] = ch.oka ? f2add(va[i], f2s(-mean)) : f2s(0.f);
                        vb[i] = ch.okb ? f2add(vb[i], f2s(-mean)) : f2s(0.f);
                    }
                }
                float2 t = f2s(0.f);
#pragma unroll
                for (int i = 0; i < H; ++i) t = f2fma(va[i], va[i], f2fma(vb[i], vb[i], t));
                float sq[1] = {t.x + t.y};
                group_sum<L, 1>(sq);
                const float rstd = rsqrtf(sq[0] * inv + p.eps);
                if (p.rstd && sl == 0 && h < heads) p.rstd[stat + h] = rstd;
                if (MODE == kRopeLn && p.mean && sl == 0 && h < heads) p.mean[stat + h] = mean;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    va[i] = f2mul(va[i], f2s(rstd));
                    vb[i] = f2mul(vb[i], f2s(rstd));
                }
            }
            float2 ua[H], ub[H];
#pragma unroll
            for (int i = 0; i < H; ++i) {
                float2 ta = inter ? f2swap(va[i]) : vb[i], tb = inter ? f2swap(vb[i]) : va[i];
                if constexpr (KIND == kRopeSome) {  // an element that is not rotated takes nothing from another, not even a NaN
                    ta = ch.ra ? ta : f2s(0.f);
                    tb = ch.rb ? tb : f2s(0.f);
                }
                ua[i] = f2fma(va[i], ca[i], f2mul(ta, sa[i]));
                ub[i] = f2fma(vb[i], cb[i], f2mul(tb, sb[i]));
                if constexpr (MODE == kRopeLn) {
                    ua[i] = f2add(ua[i], ba[i]);
                    ub[i] = f2add(ub[i], bb[i]);
                }
            }
            char *q = y + h * (p.y[r].head * ES);
            if (h < heads && ch.oka) rope_st(q + ch.a * ES, rope_pack<XT, V>(ua).v);
            if (h < heads && ch.okb) rope_st(q + ch.b * ES, rope_pack<XT, V>(ub).v);
        }
        if (!w.left) return;
        fresh = nf;
        turn = nf || w.blk == nq;
    }
}

template <bool LN, int XT, int V, int L, int KIND, int U, int MINB>
__global__ void __launch_bounds__(kRopeCTA, MINB) rope_bwd_vec(const __grid_constant__ RopeParams p) {
    pdl_launch_dependents();  // the column reduce waits for this grid's completion
    constexpr int G = 32 / L, H = V / 2, ES = XT == kF32 ? 4 : 2, DEPTH = kRopeBwdDepth;
    using Table = RopeTable<V, L>;
    using Raw = RopeRaw<XT, V>;
    struct Slot {
        Raw x[U][2][32], g[U][2][32];
        float mean[U][32], rstd[U][32];
    };
    // rings, tables, frequencies, gamma of the queries and of the keys; at the end the column sums [kRopeWarps][D] over the rings
    extern __shared__ __align__(16) unsigned char rope_smem[];
    const int lane = threadIdx.x & 31, sl = lane % L, grp = lane / L, warp = threadIdx.x >> 5;
    Slot *ring = reinterpret_cast<Slot *>(rope_smem) + warp * DEPTH;
    Table *tables = reinterpret_cast<Table *>(rope_smem + sizeof(Slot) * DEPTH * kRopeWarps);
    RopeTurns<V, L> &turns = *reinterpret_cast<RopeTurns<V, L> *>(tables + kRopeWarps);
    float *par = reinterpret_cast<float *>(&turns + 1), *rope_acc = reinterpret_cast<float *>(rope_smem);
    Table &tab = tables[warp];
    RopeWalk w(p), ahead = w;  // the pass worked on, the pass to load
    const RopeChunks<V, L, KIND> ch(p, sl);
    const int r = w.r, heads = p.heads[r];
    auto load = [&](int slot) {
        if (ahead.left) {
            const char *x = static_cast<const char *>(p.x[r].p) + ahead.at(p.x[r]) * ES,
                       *g = static_cast<const char *>(p.g[r].p) + ahead.at(p.g[r]) * ES;
            const int64_t stat = ahead.stat(p), xs = p.x[r].head * ES, gs = p.g[r].head * ES;
            Slot &to = ring[slot];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // past the last head a lane repeats that with a gradient of zeros, unstored
                const int h0 = ahead.blk * (G * U) + u * G + grp, h = h0 < heads ? h0 : heads - 1;
                const bool in = h0 < heads;
                rope_cp(&to.x[u][0][lane], x + h * xs + ch.a * ES, ch.oka, Raw{}.v);
                rope_cp(&to.x[u][1][lane], x + h * xs + ch.b * ES, ch.okb, Raw{}.v);
                rope_cp(&to.g[u][0][lane], g + h * gs + ch.a * ES, in && ch.oka, Raw{}.v);
                rope_cp(&to.g[u][1][lane], g + h * gs + ch.b * ES, in && ch.okb, Raw{}.v);
                rope_cp(&to.rstd[u][lane], p.rstd + stat + h, true, 0.f);
                if constexpr (LN) rope_cp(&to.mean[u][lane], p.mean + stat + h, true, 0.f);
            }
            ahead.next(p);
        }
        rope_cp_end();
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(i);
    int64_t pos = w.left ? rope_position(p, w, lane) : 0;
    const uint32_t axis = Table::axes(p, lane);
    turns.fill(p);
    tab.ones(lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) rope_param(par + i * p.D, p.gamma[i], p.D, p.pdt, 1.f);
    __syncthreads();
    float2 da[H], db[H], ea[H], eb[H];
#pragma unroll
    for (int i = 0; i < H; ++i) da[i] = db[i] = ea[i] = eb[i] = f2s(0.f);
    if (w.left) {
        const float inv = 1.f / (float)p.D;
        const bool inter = KIND == kRopeNeighbours || (KIND == kRopeSome && p.inter);
        bool fresh = true;
        for (int slot = 0;; slot = slot == DEPTH - 1 ? 0 : slot + 1) {
            char *y = static_cast<char *>(p.y[r].p) + w.at(p.y[r]) * ES;
            const int h0 = w.blk * (G * U) + grp;
            const bool nf = w.next(p);
            if (fresh) tab.put(turns, p, pos, axis, lane);
            if (w.left && nf) pos = rope_position(p, w, lane);
            rope_cp_wait<DEPTH - 1>();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // the gradient turned back (the sign of s is the transpose's)
                float2 ta[H], tb[H];
                {
                    float2 c[H], s[H], ga[H], gb[H];  // c, s: of the chunks' pairs (neighbours: first a's, then b's)
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const int at = inter ? (2 * i < H ? ch.pa + 2 * i : ch.pb + 2 * i - H) : ch.pa + 2 * i;
                        c[i] = *reinterpret_cast<const float2 *>(tab.c + at);
                        s[i] = *reinterpret_cast<const float2 *>(tab.s + at);
                    }
                    rope_unpack<XT, V>(ring[slot].g[u][0][lane], ga);
                    rope_unpack<XT, V>(ring[slot].g[u][1][lane], gb);
                    if (inter) {
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const float ci = i & 1 ? c[i / 2].y : c[i / 2].x, si = i & 1 ? s[i / 2].y : s[i / 2].x;
                            const float cj = i & 1 ? c[H / 2 + i / 2].y : c[H / 2 + i / 2].x,
                                        sj = i & 1 ? s[H / 2 + i / 2].y : s[H / 2 + i / 2].x;
                            float2 m = f2swap(ga[i]), n = f2swap(gb[i]);
                            if constexpr (KIND == kRopeSome) {
                                m = ch.ra ? m : f2s(0.f);
                                n = ch.rb ? n : f2s(0.f);
                            }
                            ta[i] = make_float2(ga[i].x * ci - m.x * si, ga[i].y * ci + m.y * si);
                            tb[i] = make_float2(gb[i].x * cj - n.x * sj, gb[i].y * cj + n.y * sj);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            float2 m = gb[i], n = ga[i];
                            if constexpr (KIND == kRopeSome) {
                                m = ch.ra ? m : f2s(0.f);
                                n = ch.ra ? n : f2s(0.f);
                            }
                            ta[i] = f2fma(ga[i], c[i], f2mul(make_float2(-m.x, -m.y), s[i]));
                            tb[i] = f2fma(gb[i], c[i], f2mul(n, s[i]));
                        }
                    }
                }
                float2 xa[H], xb[H];
                rope_unpack<XT, V>(ring[slot].x[u][0][lane], xa);
                rope_unpack<XT, V>(ring[slot].x[u][1][lane], xb);
                const float rstd = ring[slot].rstd[u][lane], mean = LN ? ring[slot].mean[u][lane] : 0.f;
                if (u == U - 1) load(slot);
                float2 dot = f2s(0.f), sum = f2s(0.f);
                float2 wa[H], wb[H];
                rope_get<V>(par + r * p.D + ch.a, wa);
                rope_get<V>(par + r * p.D + ch.b, wb);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if constexpr (LN) {
                        xa[i] = f2add(xa[i], f2s(-mean));
                        xb[i] = f2add(xb[i], f2s(-mean));
                        ea[i] = f2add(ea[i], ta[i]);
                        eb[i] = f2add(eb[i], tb[i]);
                    }
                    xa[i] = f2mul(xa[i], f2s(rstd));
                    xb[i] = f2mul(xb[i], f2s(rstd));
                    da[i] = f2fma(ta[i], xa[i], da[i]);
                    db[i] = f2fma(tb[i], xb[i], db[i]);
                    ta[i] = f2mul(ta[i], wa[i]);
                    tb[i] = f2mul(tb[i], wb[i]);
                    dot = f2fma(ta[i], xa[i], f2fma(tb[i], xb[i], dot));
                    if constexpr (LN) sum = f2add(sum, f2add(ta[i], tb[i]));
                }
                float v[LN ? 2 : 1];
                v[0] = dot.x + dot.y;
                if constexpr (LN) v[1] = sum.x + sum.y;
                group_sum<L, LN ? 2 : 1>(v);
                const float2 c2 = f2s(-v[0] * inv), c1 = f2s(LN ? -v[LN ? 1 : 0] * inv : 0.f);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if constexpr (LN) {
                        ta[i] = f2add(ta[i], c1);
                        tb[i] = f2add(tb[i], c1);
                    }
                    ta[i] = f2mul(f2fma(xa[i], c2, ta[i]), f2s(rstd));
                    tb[i] = f2mul(f2fma(xb[i], c2, tb[i]), f2s(rstd));
                }
                const int h = h0 + u * G;
                char *q = y + h * (p.y[r].head * ES);
                if (h < heads && ch.oka) rope_st(q + ch.a * ES, rope_pack<XT, V>(ta).v);
                if (h < heads && ch.okb) rope_st(q + ch.b * ES, rope_pack<XT, V>(tb).v);
            }
            if (!w.left) break;
            fresh = nf;
        }
    }
    __syncthreads();  // the rings of all warps have been read
    // the sums of the groups of lanes (the same columns) of a warp, then of the CTA's warps
    float *mine = rope_acc + warp * p.D;
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
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if (ch.oka) *reinterpret_cast<float2 *>(mine + ch.a + 2 * i) = u[i];
                if (ch.okb) *reinterpret_cast<float2 *>(mine + ch.b + 2 * i) = v[i];
            }
        }
    };
    columns(da, db);
    rope_partial(p, rope_acc, 0);
    if constexpr (LN) {
        columns(ea, eb);
        rope_partial(p, rope_acc, 1);
    }
}

}  // namespace gbn
