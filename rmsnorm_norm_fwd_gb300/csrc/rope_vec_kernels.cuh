// rope_vec_kernels.cuh -- the head operators on vectors.
//
// A group of L lanes holds one head, 32 / L heads a warp and pass; a lane holds C
// times two chunks of V consecutive elements, each moved as one vector of 4, 8 or
// 16 bytes (C V = 8 for 16-bit types, so that a lane has 16 elements).  Where
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
//
// What bounds it: DRAM for the rotation alone (26520 tokens of 80 heads of 128
// bf16 170 us, 94% of the copy rate's time) and RMSNorm (16384 tokens of 40 heads:
// forward 54.6 us, 91%, 13 instructions an element; backward 80.2 us, 93%, 19);
// with LayerNorm (60 and 90 us, 83%) and heads that leave lanes or vectors unused,
// instruction issue and latency at 16 warps an SM.  That is what 16 elements of a
// lane with their coefficients or sums leave (106 to 128 registers): capped at 80
// registers for 24 warps the kernels spill, forward 81 us and backward 142 us.
// At 128 registers some of LayerNorm's spill too: the backward on vectors below
// 16 bytes, for differing types and in fp16 on 10 and 32 lanes by 4 to 108 bytes,
// the forward on 8-byte vectors and for differing types by 4 to 32.
// Copies straight into registers, one pass ahead, in place of the rings: forward
// 98 us, backward 147 us.
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
template <> struct RopeRaw<kF32, 2> { uint2 v; };
template <> struct RopeRaw<kF16, 2> { uint32_t v; };
template <> struct RopeRaw<kBF16, 2> { uint32_t v; };
// Types that differ within a call, read from it: 16 bytes hold four elements of any.
constexpr int kMixed = 3;
template <> struct RopeRaw<kMixed, 4> { uint4 v; };
template <int XT> __device__ __forceinline__ int rope_esize(int dt) {
    return XT == kMixed ? esize(dt) : XT == kF32 ? 4 : 2;
}

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
template <int XT, int V>
__device__ __forceinline__ void rope_unpack(const RopeRaw<XT, V> &r, int dt, float2 *f) {
    if constexpr (V == 2) {
        if constexpr (XT == kF32) f[0] = make_float2(__uint_as_float(r.v.x), __uint_as_float(r.v.y));
        else f[0] = rope_pair<XT>(r.v);
    } else if constexpr (XT == kMixed) {
        if (dt == kF32) {
            f[0] = make_float2(__uint_as_float(r.v.x), __uint_as_float(r.v.y));
            f[1] = make_float2(__uint_as_float(r.v.z), __uint_as_float(r.v.w));
        } else if (dt == kBF16) {
            f[0] = rope_pair<kBF16>(r.v.x);
            f[1] = rope_pair<kBF16>(r.v.y);
        } else {
            f[0] = rope_pair<kF16>(r.v.x);
            f[1] = rope_pair<kF16>(r.v.y);
        }
    } else if constexpr (XT == kF32) {
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
// V elements rounded to their type and stored.
template <int XT, int V> __device__ __forceinline__ void rope_store(char *p, int dt, const float2 *f) {
    if constexpr (V == 2) {
        if constexpr (XT == kF32) *reinterpret_cast<float2 *>(p) = f[0];
        else *reinterpret_cast<uint32_t *>(p) = rope_word<XT>(f[0]);
    } else if (XT == kF32 || (XT == kMixed && dt == kF32)) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    } else if constexpr (V == 8) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(rope_word<XT>(f[0]), rope_word<XT>(f[1]), rope_word<XT>(f[2]), rope_word<XT>(f[3]));
    } else if (XT == kBF16 || (XT == kMixed && dt == kBF16)) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(rope_word<kBF16>(f[0]), rope_word<kBF16>(f[1]));
    } else {
        *reinterpret_cast<uint2 *>(p) = make_uint2(rope_word<kF16>(f[0]), rope_word<kF16>(f[1]));
    }
}

// Asynchronous copies into the lane's own places of the ring: no other thread
// reads them, so that waiting for the lane's own groups is enough.  Lanes
// without an element fill with zeros (`from` is then any valid address).
template <int BYTES> __device__ __forceinline__ void rope_cp_bytes(void *to, const void *from, bool in) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(in ? 16 : 0)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(smem_u32(to)), "l"(from),
                     "r"(in ? BYTES : 0), "n"(BYTES)
                     : "memory");
}
template <int XT, int V>
__device__ __forceinline__ void rope_cp(RopeRaw<XT, V> *to, const char *from, bool in, int dt) {
    if constexpr (XT == kMixed) {
        if (dt == kF32) rope_cp_bytes<16>(to, from, in);
        else rope_cp_bytes<8>(to, from, in);
    } else {
        rope_cp_bytes<(int)sizeof(RopeRaw<XT, V>)>(to, from, in);
    }
}
__device__ __forceinline__ void rope_cp_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void rope_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Values that a lane reads V at a time lie in shared memory as planes of four
// (element 8 c + 4 h + i at h n / 2 + 4 c + i of n), so that the lanes' 16-byte
// reads are side by side; with V = 4 they are so as they are.
template <int V> __device__ __forceinline__ int rope_place(int e, int n) {
    return V == 8 ? ((e >> 2) & 1) * (n / 2) + (e >> 3) * 4 + (e & 3) : e;
}
// Row `row` of D parameters widened to fp32 into shared memory, a null row as `none`; every thread takes its share.
template <int V> __device__ __forceinline__ void rope_param(float *to, const void *row, int D, int dt, float none) {
    for (int c = threadIdx.x; c < D; c += kRopeCTA) to[rope_place<V>(c, D)] = row ? ld1(row, c, dt) : none;
}
// The V values from e (a multiple of V) on, of n.
template <int V> __device__ __forceinline__ void rope_get(const float *from, int e, int n, float2 *f) {
    if constexpr (V == 2) {
        f[0] = *reinterpret_cast<const float2 *>(from + e);
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 v = *reinterpret_cast<const float4 *>(from + e / (V / 4) + i * (n / 2));
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    }
}

// What is rotated, fixed at compile time where it is common: the whole head, as
// halves or as neighbours, or anything (read from the call, through selects).
enum RopeKind : int { kRopeHalves = 0, kRopeNeighbours = 1, kRopeSome = 2 };

// The chunks of a lane: first elements, whether they are there, whether they are rotated.  Slot i of lane sl is number
// i L + sl of the head.
template <int V, int C, int L, int KIND> struct RopeChunks {
    int a[C], b[C];
    bool oka[C], okb[C], ra[C], rb[C];
    __device__ __forceinline__ RopeChunks(const RopeParams &p, int sl, bool used) {
        const int n = p.D / V, nr = p.rot / V;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int j = i * L + sl;
            int ca, cb;
            if (KIND == kRopeNeighbours || (KIND == kRopeSome && p.inter)) {
                const int ns = (n + 1) / 2;
                ca = j;
                cb = ns + j;
                oka[i] = j < ns;
            } else {
                const int half = nr / 2, rest = (n - nr + 1) / 2;
                ca = j < half ? j : nr + (j - half);
                cb = j < half ? j + half : ca + rest;
                oka[i] = j < half + rest;
            }
            oka[i] = oka[i] && used;
            okb[i] = oka[i] && cb < n;
            ra[i] = oka[i] && ca < nr;
            rb[i] = okb[i] && cb < nr;
            a[i] = oka[i] ? ca * V : 0;  // lanes without a chunk stay inside the head
            b[i] = okb[i] ? cb * V : 0;
        }
    }
};

// Sums over the L lanes of a head.  Powers of two by a butterfly.  Else by
// rotations within the group, whose order of additions differs between lanes:
// halves first where L is even, then sums of 3 by two rotations, of 5 by a chain
// of 2, 4 and 5.  (Heads of 80 on five lanes instead of eight: 16.4 us against 19.0
// us for 4099 tokens of 32, LayerNorm.)
template <int L> struct RopeLanes {
    static constexpr bool POW2 = (L & (L - 1)) == 0;
    int sl, base;
    __device__ __forceinline__ RopeLanes(int lane) : sl(lane % L), base(lane - lane % L) {}
    __device__ __forceinline__ float from(float v, int by) const {
        const int at = sl + by;
        return __shfl_sync(0xffffffffu, v, base + (at >= L ? at - L : at));
    }
    template <int R> __device__ __forceinline__ void sum(float (&v)[R]) const {
        if constexpr (POW2) {
            group_sum<L, R>(v);
        } else {
            static_assert(L == 5 || L == 6 || L == 10, "lanes a head");
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float t = v[i];
                if constexpr (L == 6) t += from(t, 3);
                if constexpr (L == 10) t += from(t, 5);
                if constexpr (L == 6) {
                    const float a = from(t, 1), b = from(t, 2);
                    v[i] = t + (a + b);
                } else {
                    float u = t + from(t, 1);
                    u += from(u, 2);
                    v[i] = u + from(t, 4);
                }
            }
        }
    }
};

// The frequencies of a call in turns, once a CTA.
template <int N> struct RopeTurns {
    static_assert(N <= kRopeCTA, "a pair a thread");
    uint64_t f[N];
    float bad[N];  // 0, or NaN where the frequency is not a number of turns
    template <bool LOCAL> __device__ __forceinline__ void fill(const RopeParams &p) {
        const int j = threadIdx.x;
        if (2 * j >= p.rot) return;
        bool b;
        f[j] = rope_turns<LOCAL>(__ldg(p.inv_freq + j), &b);
        bad[j] = b ? __int_as_float(0x7fffffff) : 0.f;
    }
};
// A warp's cosines and sines: written by the lane that computed the pair, read by those whose chunks hold it.
// As halves, a chunk's V pairs are read at once, and lie as rope_place says.
template <int V, int N> struct RopeTable {
    static constexpr int PER = (N + 31) / 32;
    float c[N], s[N];
    // Behind the rotated pairs: cosine 1 and sine 0, for the chunks that are not.
    __device__ __forceinline__ void ones(int lane, int rot, bool inter) {
        for (int j = rot / 2 + lane; j < N; j += 32) {
            const int at = inter ? j : rope_place<V>(j, N);
            c[at] = 1.f;
            s[at] = 0.f;
        }
    }
    // pos: lane a holds the position on axis a; axis: two bits for each of the lane's pairs lane, lane + 32, ...
    __device__ __forceinline__ void put(const RopeTurns<N> &turns, const RopeParams &p, int64_t pos, uint32_t axis,
                                        int lane, bool inter) {
        __syncwarp();  // the last token's have been read
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = lane + 32 * i;
            const int64_t at = __shfl_sync(0xffffffffu, (long long)pos, (axis >> (2 * i)) & 3u);
            if (2 * j < p.rot) {
                float cs, sn;
                rope_sincos((uint64_t)at * turns.f[j], p.sign, &cs, &sn);
                const int to = inter ? j : rope_place<V>(j, N);
                c[to] = cs + turns.bad[j];
                s[to] = sn + turns.bad[j];
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

constexpr int kRopeNoHead = 1 << 20;  // the group of lanes beyond the last whole one: never has a head

__device__ __forceinline__ float2 f2swap(float2 v) { return make_float2(v.y, v.x); }

template <int MODE, int XT, int V, int C, int L, int KIND, int U, int MINB>
__global__ void __launch_bounds__(kRopeCTA, MINB) rope_fwd_vec(const __grid_constant__ RopeParams p) {
    constexpr int G = 32 / L, HV = V / 2, H = C * HV, N = C * V * L, DEPTH = kRopeFwdDepth;
    // Where an element is not rotated, its beta stays as it is and takes nothing from another's, not even a NaN's
    // product with 0: left out of the fold, or, where that takes registers the kernel does not have, read again.
    // (LayerNorm of heads of 98 on 16-bit vectors of two: 92.7 us read again, 99.7 us left out, 92.3 us without either;
    // of 80 on vectors of eight 16.3 us read again, 15.9 us left out; fp32 of 98 56.3 us and 55.3 us.)
    constexpr bool AGAIN = MODE == kRopeLn && KIND == kRopeSome && C == 4;
    constexpr bool SELECT = MODE == kRopeLn && KIND == kRopeSome && C != 4;
    using Table = RopeTable<V, N>;
    using Raw = RopeRaw<XT, V>;
    // rings, tables, frequencies, then gamma (and beta) of the queries and of the keys
    extern __shared__ __align__(16) unsigned char rope_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const RopeLanes<L> lanes(lane);
    const int sl = lanes.sl, grp = lane < G * L ? lane / L : kRopeNoHead;
    Raw(*ring)[U][2 * C][32] = reinterpret_cast<Raw(*)[U][2 * C][32]>(rope_smem) + warp * DEPTH;
    Table *tables = reinterpret_cast<Table *>(rope_smem + sizeof(Raw) * 64 * C * U * DEPTH * kRopeWarps);
    RopeTurns<N> &turns = *reinterpret_cast<RopeTurns<N> *>(tables + kRopeWarps);
    float *par = reinterpret_cast<float *>(&turns + 1);
    Table &tab = tables[warp];
    RopeCursor<G * U> w(p, grp), ahead = w;  // the pass worked on, the pass to load
    const RopeChunks<V, C, L, KIND> ch(p, sl, lane < G * L);
    const bool inter = KIND == kRopeNeighbours || (KIND == kRopeSome && p.inter);
    const int xes = rope_esize<XT>(p.xdt), yes = rope_esize<XT>(p.ydt);
    const char *x = ahead.at(p, p.x[ahead.r], V * xes);
    int64_t xs = p.x[ahead.r].head * (G * V * xes);
    auto load = [&](int slot) {
        if (ahead.left) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // a lane without a head in the pass reads another, and stores nothing
                const char *q = u == 0 ? x : x + (ahead.hl > u * G ? u * xs : 0);
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    rope_cp(&ring[slot][u][2 * i][lane], q + ch.a[i] * xes, ch.oka[i], p.xdt);
                    rope_cp(&ring[slot][u][2 * i + 1][lane], q + ch.b[i] * xes, ch.okb[i], p.xdt);
                }
            }
            if (ahead.next(p, grp)) {
                x = ahead.at(p, p.x[ahead.r], V * xes);
                xs = p.x[ahead.r].head * (G * V * xes);
            } else if (ahead.hl > 0) {
                x += U * xs;
            }
        }
        rope_cp_end();
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(i);
    int64_t pos = w.left ? rope_position(p, w, lane) : 0;
    const uint32_t axis = Table::axes(p, lane);
    turns.template fill<C == 4>(p);
    tab.ones(lane, p.rot, inter);
    if constexpr (MODE != kRopeOnly) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            rope_param<V>(par + r * p.D, p.gamma[r], p.D, p.pdt, 1.f);
            if constexpr (MODE == kRopeLn) rope_param<V>(par + (2 + r) * p.D, p.beta[r], p.D, p.pdt, 0.f);
        }
    }
    __syncthreads();
    if (!w.left) return;
    const float inv = 1.f / (float)p.D;
    char *y = w.at(p, p.y[w.r], V * yes);
    int64_t ys = p.y[w.r].head * (G * V * yes), stat = w.stat(p);
    float2 ca[H], sa[H], cb[H], sb[H], ba[H], bb[H];
    int turn = 2;  // 2: another token's angles, 1: another tensor's coefficients
    for (int slot = 0;; slot = slot == DEPTH - 1 ? 0 : slot + 1) {
        const int r = w.r, hl = w.hl;
        if (turn == 2) tab.put(turns, p, pos, axis, lane, inter);
        if (turn) {
            float2 ga[H], gb[H];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if constexpr (MODE != kRopeOnly) {
                    rope_get<V>(par + r * p.D, ch.a[i], p.D, ga + i * HV);
                    rope_get<V>(par + r * p.D, ch.b[i], p.D, gb + i * HV);
                } else {
#pragma unroll
                    for (int k = 0; k < HV; ++k) ga[i * HV + k] = gb[i * HV + k] = f2s(1.f);
                }
                if constexpr (MODE == kRopeLn) {
                    rope_get<V>(par + (2 + r) * p.D, ch.a[i], p.D, ba + i * HV);
                    rope_get<V>(par + (2 + r) * p.D, ch.b[i], p.D, bb + i * HV);
                }
            }
            if (inter) {  // pairs of a chunk from element e on: from e / 2 on
                auto fold = [&](const float2 &g, int at, bool rotated, float2 &cc, float2 &ss, float2 &bias) {
                    const float c = tab.c[at], s = tab.s[at];
                    cc = make_float2(g.x * c, g.y * c);
                    ss = make_float2(-g.y * s, g.x * s);
                    if constexpr (MODE == kRopeLn) {
                        if (!SELECT || rotated)
                            bias = make_float2(bias.x * c - bias.y * s, bias.y * c + bias.x * s);
                    }
                };
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    fold(ga[i], ch.a[i / HV] / 2 + i % HV, ch.ra[i / HV], ca[i], sa[i], ba[i]);
                    fold(gb[i], ch.b[i / HV] / 2 + i % HV, ch.rb[i / HV], cb[i], sb[i], bb[i]);
                }
            } else {
                float2 c[H], s[H];
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    rope_get<V>(tab.c, (i * L + sl) * V, N, c + i * HV);
                    rope_get<V>(tab.s, (i * L + sl) * V, N, s + i * HV);
                }
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    ca[i] = f2mul(ga[i], c[i]);
                    sa[i] = f2mul(gb[i], make_float2(-s[i].x, -s[i].y));
                    cb[i] = f2mul(gb[i], c[i]);
                    sb[i] = f2mul(ga[i], s[i]);
                    if constexpr (MODE == kRopeLn) {
                        const float2 v = ba[i], u = bb[i];
                        ba[i] = make_float2(v.x * c[i].x - u.x * s[i].x, v.y * c[i].y - u.y * s[i].y);
                        bb[i] = make_float2(u.x * c[i].x + v.x * s[i].x, u.y * c[i].y + v.y * s[i].y);
                        if constexpr (SELECT) {
                            ba[i] = ch.ra[i / HV] ? ba[i] : v;
                            bb[i] = ch.ra[i / HV] ? bb[i] : u;
                        }
                    }
                }
            }
            if constexpr (AGAIN) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    if (!ch.ra[i]) rope_get<V>(par + (2 + r) * p.D, ch.a[i], p.D, ba + i * HV);
                    if (!ch.rb[i]) rope_get<V>(par + (2 + r) * p.D, ch.b[i], p.D, bb + i * HV);
                }
            }
            if constexpr (KIND == kRopeSome) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    sa[i] = ch.ra[i / HV] ? sa[i] : f2s(0.f);
                    sb[i] = ch.rb[i / HV] ? sb[i] : f2s(0.f);
                }
            }
        }
        turn = w.next(p, grp);
        if (w.left && turn == 2) pos = rope_position(p, w, lane);
        rope_cp_wait<DEPTH - 1>();
        Raw raw[U][2 * C];
#pragma unroll
        for (int i = 0; i < U * 2 * C; ++i) raw[i / (2 * C)][i % (2 * C)] = ring[slot][i / (2 * C)][i % (2 * C)][lane];
        load(slot);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = hl > u * G;
            float2 va[H], vb[H];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                rope_unpack<XT, V>(raw[u][2 * i], p.xdt, va + i * HV);
                rope_unpack<XT, V>(raw[u][2 * i + 1], p.xdt, vb + i * HV);
            }
            if constexpr (MODE != kRopeOnly) {
                float mean = 0.f;
                if constexpr (MODE == kRopeLn) {
                    float2 t = f2s(0.f);
#pragma unroll
                    for (int i = 0; i < H; ++i) t = f2add(t, f2add(va[i], vb[i]));
                    float sum[1] = {t.x + t.y};
                    lanes.sum(sum);
                    mean = sum[0] * inv;
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        va[i] = f2add(va[i], f2s(-mean));
                        vb[i] = f2add(vb[i], f2s(-mean));
                    }
                }
                float sq[1] = {0.f};
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    float2 ta = f2s(0.f), tb = f2s(0.f);
#pragma unroll
                    for (int k = i * HV; k < (i + 1) * HV; ++k) {
                        ta = f2fma(va[k], va[k], ta);
                        tb = f2fma(vb[k], vb[k], tb);
                    }
                    // a chunk that is not there holds zeros, with the mean off it no longer
                    const bool ka = MODE != kRopeLn || ch.oka[i], kb = MODE != kRopeLn || ch.okb[i];
                    sq[0] += (ka ? ta.x + ta.y : 0.f) + (kb ? tb.x + tb.y : 0.f);
                }
                lanes.sum(sq);
                const float rstd = rsqrtf(sq[0] * inv + p.eps);
                if (p.rstd && sl == 0 && in) p.rstd[stat + u * G] = rstd;
                if (MODE == kRopeLn && p.mean && sl == 0 && in) p.mean[stat + u * G] = mean;
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
                if constexpr (KIND == kRopeSome) {  // what is not rotated takes nothing from another, not even a NaN
                    ta = ch.ra[i / HV] ? ta : f2s(0.f);
                    tb = ch.rb[i / HV] ? tb : f2s(0.f);
                }
                ua[i] = f2fma(va[i], ca[i], MODE == kRopeLn ? f2fma(ta, sa[i], ba[i]) : f2mul(ta, sa[i]));
                ub[i] = f2fma(vb[i], cb[i], MODE == kRopeLn ? f2fma(tb, sb[i], bb[i]) : f2mul(tb, sb[i]));
            }
            char *q = u == 0 ? y : y + u * ys;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (in && ch.oka[i]) rope_store<XT, V>(q + ch.a[i] * yes, p.ydt, ua + i * HV);
                if (in && ch.okb[i]) rope_store<XT, V>(q + ch.b[i] * yes, p.ydt, ub + i * HV);
            }
        }
        if (!w.left) return;
        if (turn) {
            y = w.at(p, p.y[w.r], V * yes);
            ys = p.y[w.r].head * (G * V * yes);
            stat = w.stat(p);
        } else {
            y += U * ys;
            stat += U * G;
        }
    }
}

template <bool LN, int XT, int V, int C, int L, int KIND, int MINB>
__global__ void __launch_bounds__(kRopeCTA, MINB) rope_bwd_vec(const __grid_constant__ RopeParams p) {
    pdl_launch_dependents();  // the column reduce waits for this grid's completion
    constexpr int G = 32 / L, HV = V / 2, H = C * HV, N = C * V * L, DEPTH = kRopeBwdDepth;
    // A gradient of zeros times another head's infinity is a NaN, so that lanes without a head either have zeros for x
    // and its statistics too or leave the column sums out.  (Zeros, leaving out: heads of 98 as neighbours 106.7 us,
    // 110.7 us; on vectors of eight LayerNorm of heads of 256 51.9 us, 50.0 us, of 192 145 us, 142 us; bf16 rows with
    // an fp32 gradient 120 us, 113 us.)
    constexpr bool ZEROS = V == 2;
    using Table = RopeTable<V, N>;
    using Raw = RopeRaw<XT, V>;
    struct Slot {
        Raw x[2 * C][32], g[2 * C][32];
        float mean[32], rstd[32];
    };
    // rings, sums aside, tables, frequencies, gamma of the queries and of the keys; at the end the column sums
    // [kRopeWarps][D] over the rings
    using Aside = RopeAside<H * (LN ? 2 : 1)>;
    extern __shared__ __align__(16) unsigned char rope_smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const RopeLanes<L> lanes(lane);
    const int sl = lanes.sl, grp = lane < G * L ? lane / L : kRopeNoHead;
    Slot *ring = reinterpret_cast<Slot *>(rope_smem) + warp * DEPTH;
    Aside *asides = reinterpret_cast<Aside *>(rope_smem + sizeof(Slot) * DEPTH * kRopeWarps), &aside = asides[warp];
    Table *tables = reinterpret_cast<Table *>(asides + kRopeWarps);
    RopeTurns<N> &turns = *reinterpret_cast<RopeTurns<N> *>(tables + kRopeWarps);
    float *par = reinterpret_cast<float *>(&turns + 1), *rope_acc = reinterpret_cast<float *>(rope_smem);
    Table &tab = tables[warp];
    RopeCursor<G> w(p, grp), ahead = w;  // the pass worked on, the pass to load
    const RopeChunks<V, C, L, KIND> ch(p, sl, lane < G * L);
    const bool inter = KIND == kRopeNeighbours || (KIND == kRopeSome && p.inter);
    const int xes = rope_esize<XT>(p.xdt), ges = rope_esize<XT>(p.ydt);
    const char *x = ahead.at(p, p.x[ahead.r], V * xes), *g = ahead.at(p, p.g[ahead.r], V * ges);
    int64_t xs = p.x[ahead.r].head * (G * V * xes), gs = p.g[ahead.r].head * (G * V * ges);
    int64_t stat = ahead.stat(p);
    auto load = [&](int slot) {
        if (ahead.left) {
            Slot &to = ring[slot];
            // a lane without a head in the pass reads another (or zeros) with a gradient of zeros, and stores nothing
            const bool in = ahead.hl > 0, at = in || !ZEROS;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                rope_cp(&to.x[2 * i][lane], x + ch.a[i] * xes, at && ch.oka[i], p.xdt);
                rope_cp(&to.x[2 * i + 1][lane], x + ch.b[i] * xes, at && ch.okb[i], p.xdt);
                rope_cp(&to.g[2 * i][lane], g + ch.a[i] * ges, in && ch.oka[i], p.ydt);
                rope_cp(&to.g[2 * i + 1][lane], g + ch.b[i] * ges, in && ch.okb[i], p.ydt);
            }
            rope_cp_bytes<4>(&to.rstd[lane], p.rstd + stat, at);
            if constexpr (LN) rope_cp_bytes<4>(&to.mean[lane], p.mean + stat, at);
            if (ahead.next(p, grp)) {
                x = ahead.at(p, p.x[ahead.r], V * xes);
                g = ahead.at(p, p.g[ahead.r], V * ges);
                xs = p.x[ahead.r].head * (G * V * xes);
                gs = p.g[ahead.r].head * (G * V * ges);
                stat = ahead.stat(p);
            } else if (ahead.hl > 0) {
                x += xs;
                g += gs;
                stat += G;
            }
        }
        rope_cp_end();
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(i);
    int64_t pos = w.left ? rope_position(p, w, lane) : 0;
    const uint32_t axis = Table::axes(p, lane);
    turns.template fill<C == 4>(p);
    tab.ones(lane, p.rot, inter);
#pragma unroll
    for (int i = 0; i < 2; ++i) rope_param<V>(par + i * p.D, p.gamma[i], p.D, p.pdt, 1.f);
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
        char *y = w.at(p, p.y[w.r], V * xes);
        int64_t ys = p.y[w.r].head * (G * V * xes);
        int turn = 2;
        for (int slot = 0;; slot = slot == DEPTH - 1 ? 0 : slot + 1) {
            const int r = w.r;
            const bool in = w.hl > 0;
            if (turn == 2) tab.put(turns, p, pos, axis, lane, inter);
            turn = w.next(p, grp);
            if (w.left && turn == 2) pos = rope_position(p, w, lane);
            rope_cp_wait<DEPTH - 1>();
            // the gradient turned back (the sign of s is the transpose's)
            float2 ta[H], tb[H];
            {
                float2 ga[H], gb[H];
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    rope_unpack<XT, V>(ring[slot].g[2 * i][lane], p.ydt, ga + i * HV);
                    rope_unpack<XT, V>(ring[slot].g[2 * i + 1][lane], p.ydt, gb + i * HV);
                }
                if (inter) {
                    auto turned = [&](float2 d, int at, bool rotated) {
                        const float c = tab.c[at], s = tab.s[at];
                        float2 m = f2swap(d);
                        if constexpr (KIND == kRopeSome) m = rotated ? m : f2s(0.f);
                        return make_float2(d.x * c - m.x * s, d.y * c + m.y * s);
                    };
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        ta[i] = turned(ga[i], ch.a[i / HV] / 2 + i % HV, ch.ra[i / HV]);
                        tb[i] = turned(gb[i], ch.b[i / HV] / 2 + i % HV, ch.rb[i / HV]);
                    }
                } else {
                    float2 c[H], s[H];
#pragma unroll
                    for (int i = 0; i < C; ++i) {
                        rope_get<V>(tab.c, (i * L + sl) * V, N, c + i * HV);
                        rope_get<V>(tab.s, (i * L + sl) * V, N, s + i * HV);
                    }
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        float2 m = gb[i], n = ga[i];
                        if constexpr (KIND == kRopeSome) {
                            m = ch.ra[i / HV] ? m : f2s(0.f);
                            n = ch.ra[i / HV] ? n : f2s(0.f);
                        }
                        ta[i] = f2fma(ga[i], c[i], f2mul(make_float2(-m.x, -m.y), s[i]));
                        tb[i] = f2fma(gb[i], c[i], f2mul(n, s[i]));
                    }
                }
            }
            float2 xa[H], xb[H];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                rope_unpack<XT, V>(ring[slot].x[2 * i][lane], p.xdt, xa + i * HV);
                rope_unpack<XT, V>(ring[slot].x[2 * i + 1][lane], p.xdt, xb + i * HV);
            }
            const float rstd = ring[slot].rstd[lane], mean = LN ? ring[slot].mean[lane] : 0.f;
            load(slot);
            float2 dot = f2s(0.f), sum = f2s(0.f);
            float2 wa[H], wb[H];
#pragma unroll
            for (int i = 0; i < C; ++i) {
                rope_get<V>(par + r * p.D, ch.a[i], p.D, wa + i * HV);
                rope_get<V>(par + r * p.D, ch.b[i], p.D, wb + i * HV);
            }
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
                if (ZEROS || in) {
                    da[i] = f2fma(ta[i], xa[i], da[i]);
                    db[i] = f2fma(tb[i], xb[i], db[i]);
                }
                ta[i] = f2mul(ta[i], wa[i]);
                tb[i] = f2mul(tb[i], wb[i]);
                dot = f2fma(ta[i], xa[i], f2fma(tb[i], xb[i], dot));
                if constexpr (LN) sum = f2add(sum, f2add(ta[i], tb[i]));
            }
            float v[LN ? 2 : 1];
            v[0] = dot.x + dot.y;
            if constexpr (LN) v[1] = sum.x + sum.y;
            lanes.sum(v);
            // dx = rstd g - rstd c1 - xhat (rstd c2)
            const float2 c2 = f2s(-v[0] * inv * rstd), c1 = f2s(LN ? -v[LN ? 1 : 0] * inv * rstd : 0.f);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                ta[i] = f2fma(xa[i], c2, LN ? f2fma(ta[i], f2s(rstd), c1) : f2mul(ta[i], f2s(rstd)));
                tb[i] = f2fma(xb[i], c2, LN ? f2fma(tb[i], f2s(rstd), c1) : f2mul(tb[i], f2s(rstd)));
            }
#pragma unroll
            for (int i = 0; i < C; ++i) {
                if (in && ch.oka[i]) rope_store<XT, V>(y + ch.a[i] * xes, p.xdt, ta + i * HV);
                if (in && ch.okb[i]) rope_store<XT, V>(y + ch.b[i] * xes, p.xdt, tb + i * HV);
            }
            if (!w.left) {
                if (r) swap();
                break;
            }
            if (turn) {
                y = w.at(p, p.y[w.r], V * xes);
                ys = p.y[w.r].head * (G * V * xes);
                if (w.r != r) swap();
            } else {
                y += ys;
            }
        }
    }
    __syncthreads();  // the rings of all warps have been read
    // the sums of the groups of lanes (the same columns) of a warp, then of the CTA's warps
    float *mine = rope_acc + warp * p.D;
    auto columns = [&](float2 (&u)[H], float2 (&v)[H]) {
        if constexpr (RopeLanes<L>::POW2) {
#pragma unroll
            for (int o = L; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    u[i].x += __shfl_xor_sync(0xffffffffu, u[i].x, o);
                    u[i].y += __shfl_xor_sync(0xffffffffu, u[i].y, o);
                    v[i].x += __shfl_xor_sync(0xffffffffu, v[i].x, o);
                    v[i].y += __shfl_xor_sync(0xffffffffu, v[i].y, o);
                }
        } else {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 a = u[i], b = v[i];
#pragma unroll
                for (int o = L; o < G * L; o += L) {
                    u[i].x += __shfl_down_sync(0xffffffffu, a.x, o);
                    u[i].y += __shfl_down_sync(0xffffffffu, a.y, o);
                    v[i].x += __shfl_down_sync(0xffffffffu, b.x, o);
                    v[i].y += __shfl_down_sync(0xffffffffu, b.y, o);
                }
            }
        }
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if (ch.oka[i / HV]) *reinterpret_cast<float2 *>(mine + ch.a[i / HV] + 2 * (i % HV)) = u[i];
                if (ch.okb[i / HV]) *reinterpret_cast<float2 *>(mine + ch.b[i / HV] + 2 * (i % HV)) = v[i];
            }
        }
    };
    // the queries' sums are in the registers, the keys' aside
    for (int r = 0; r < (p.heads[1] ? 2 : 1); ++r) {
        if (r) swap();
        columns(da, db);
        rope_partial(p, rope_acc, 0, r);
        if constexpr (LN) {
            columns(ea, eb);
            rope_partial(p, rope_acc, 1, r);
        }
    }
}

}  // namespace gbn
