// rope_common.cuh -- what the kernels of the head operators share: angles, the
// share of the work that a warp takes, the backward's partial rows.
#pragma once

#include "ex_kernels.cuh"
#include "rope_params.h"

namespace gbn {

// Angles.  Position times frequency is taken modulo one turn without rounding
// either the product or the reduction: a frequency becomes F = f / (2 pi) in
// units of 2^-64 turns, modulo one turn, and p F in 64-bit integers wraps
// exactly where the angle does.  F is within half a unit, so the angle of
// position p is within |p| 2^-65 turns of the product's (a product of fp32
// values would be off by up to 2^-24 of the whole angle, 0.06 radians at position
// 10^6).  1 / (2 pi) enters with 192 bits: what is cut off below them is less than
// 2^-40 of a unit for every frequency below 2^87 (128 bits would cut off 28 units
// at 2^70).  Frequencies from there on, like infinities and NaN, give NaN.
//
// LOCAL: the words come from an array indexed at run time, in local memory, else
// by selects, to the same bits.  Selects start a kernel sooner (a single token
// 3.45 us, 3.65 us from the array); 16-bit vectors of two, whose kernels use every
// register, run on fewer of them with the array (16384 tokens of 32 + 8 heads of 98
// as neighbours 72.7 us, 75.5 us with selects).
constexpr uint64_t kTurnHi = 0x28be60db9391054aull, kTurnMid = 0x7f09d5f47d4d3770ull,
                   kTurnLo = 0x36d8a5664f10e410ull;  // 2^192 / (2 pi)

template <bool LOCAL> __device__ __forceinline__ uint64_t rope_turns(float f, bool *bad) {
    const uint32_t bits = __float_as_uint(f), ex = (bits >> 23) & 0xffu;
    const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    *bad = ex >= 127 + 87;
    // m 2^128 / (2 pi) as three words; |f| / (2 pi) turns = that * 2^(e - 128), F = that >> (64 - e)
    const uint64_t b = __umul64hi(m, kTurnLo), lo = m * kTurnMid + b, c = __umul64hi(m, kTurnMid) + (lo < b ? 1u : 0u),
                   mid = m * kTurnHi + c, hi = __umul64hi(m, kTurnHi) + (mid < c ? 1u : 0u);
    const int sh = 64 - ((ex ? (int)ex : 1) - 150);  // 1 .. 213 for frequencies below 2^87
    uint64_t r;
    if constexpr (LOCAL) {
        auto from = [&](int at) -> uint64_t {  // bits at .. at + 63 of (hi, mid, lo)
            const uint64_t w[4] = {lo, mid, hi, 0};
            uint64_t x = 0, y = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (at >> 6 == i) {
                    x = w[i];
                    y = w[i + 1];
                }
            const int k = at & 63;
            return k ? (x >> k) | (y << (64 - k)) : x;
        };
        r = from(sh) + (from(sh - 1) & 1u);  // to nearest
    } else {
        const int at = sh - 1, k = at & 63;
        uint64_t x = at < 64 ? lo : mid, y = at < 64 ? mid : hi;
        if (at >= 128) {
            x = at < 192 ? hi : 0;
            y = 0;
        }
        const uint64_t t = (x >> k) | (y << 1 << (63 - k));  // one bit more than r, and the one above it in y
        r = (t >> 1) + ((y >> k) << 63) + (t & 1u);
    }
    return (bits >> 31) ? 0 - r : r;
}

__device__ __forceinline__ uint32_t rope_axis(const RopeParams &p, int j) {
    return (p.axis[j >> 4] >> (2 * (j & 15))) & 3u;
}
// cos and sign * sin of u 2^-64 turns.  The nearest quarter turn comes off in the
// integer, so that the one rounding of the angle, of what is left to fp32, is of
// at most an eighth of a turn: pi 2^-27 radians.  (Of up to half a turn it would
// be pi 2^-25, more than sincospif's own error.)
__device__ __forceinline__ void rope_sincos(uint64_t u, float sign, float *c, float *s) {
    const uint32_t h = (uint32_t)(u >> 32) + (1u << 29);  // its top bits: the quarter
    const uint64_t left = (uint64_t)((h & 0x3fffffffu) - (1u << 29)) << 32 | (uint32_t)u;
    float sn, cs;
    sincospif(__ll2float_rn((long long)left) * 1.0842021724855044e-19f, &sn, &cs);  // half turns: 2^-63
    const uint32_t a = __float_as_uint(h & 0x40000000u ? sn : cs), b = __float_as_uint(h & 0x40000000u ? cs : sn);
    *c = __uint_as_float(a ^ ((h + 0x40000000u) & 0x80000000u));
    *s = __uint_as_float(b ^ (h & 0x80000000u)) * sign;
}

// a / n of numbers that mostly fit 32 bits (a division in 64 is some hundred instructions).
__device__ __forceinline__ int64_t rope_div(int64_t a, int64_t n) {
    return ((a | n) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)n) : a / n;
}

// A warp's share of the passes over the tokens, each with its queries' heads and
// then its keys', so that both take the token's angles.  A pass takes GU heads,
// lane group `grp` one of them (and every 32 / L-th).  Passes over one tensor of
// a token are a segment: within one a step is an addition.
//
// A warp takes every W-th token as long as all W warps have one, so that the
// grid moves through memory as a front, and then its share of the passes over
// the tokens that are left.
template <int GU> struct RopeCursor {
    int left;    // passes to go, this one included
    int cnt;     // of the segment
    int hl;      // heads of the segment from this lane's on
    int b, s;    // token
    int r;       // 0 queries, 1 keys
    int rounds;  // whole tokens to go
    __device__ __forceinline__ RopeCursor(const RopeParams &p, int grp) {
        const int64_t w = warp();
        left = cnt = hl = b = s = r = rounds = 0;
        if (w >= p.warps) return;
        const int np = p.passes[0] + p.passes[1];
        int64_t first, count;
        rest(p, w, np, &first, &count);
        rounds = p.rounds;
        left = rounds * np + (int)count;
        start(p, grp, rounds > 0 ? w * np : first, np);
    }
    static __device__ __forceinline__ int64_t warp() {
        return (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    }
    // The share of warp w in the passes over the tokens behind the whole rounds.
    static __device__ __forceinline__ void rest(const RopeParams &p, int64_t w, int np, int64_t *first,
                                                int64_t *count) {
        const int64_t W = p.warps, done = p.rounds * W * np, U = p.units - done, each = rope_div(U, W);
        const int64_t more = U - each * W;
        *first = done + each * w + (w < more ? w : more);
        *count = each + (w < more ? 1 : 0);
    }
    __device__ __forceinline__ void start(const RopeParams &p, int grp, int64_t u, int np) {
        const int64_t t = rope_div(u, np);
        int blk = (int)(u - t * np);
        r = blk >= p.passes[0];
        if (r) blk -= p.passes[0];
        cnt = p.passes[r] - blk;
        hl = p.heads[r] - blk * GU - grp;
        b = (int)rope_div(t, p.S);
        s = (int)(t - b * p.S);
    }
    // To the next pass: 0 of the same segment, 1 of the keys of the token, 2 of another token.
    __device__ __forceinline__ int next(const RopeParams &p, int grp) {
        --left;
        if (--cnt) {
            hl -= GU;
            return 0;
        }
        const bool keys = r == 0 && p.passes[1] > 0;
        r = keys;
        cnt = p.passes[r];
        hl = p.heads[r] - grp;
        if (keys) return 1;
        --rounds;
        const bool far = rounds > 0;
        b += far ? p.step_b : 0;
        const uint32_t to = (uint32_t)s + (far ? p.step_s : 1), S = (uint32_t)p.S;  // below 2^32
        s = (int)(to >= S ? to - S : to);
        b += to >= S;
        if (rounds == 0) {
            int64_t first, count;
            const int np = p.passes[0] + p.passes[1];
            rest(p, warp(), np, &first, &count);
            start(p, grp, first, np);
        }
        return 2;
    }
    // This lane's head of the pass, the last one if it has none.
    __device__ __forceinline__ int head(const RopeParams &p) const { return p.heads[r] - (hl > 0 ? hl : 1); }
    // Address of that head in t, whose strides are in vectors of `size` bytes and below 2^32.
    __device__ __forceinline__ char *at(const RopeParams &p, const RopeHeads &t, int size) const {
        auto times = [](int i, int64_t stride) { return (uint64_t)(uint32_t)i * (uint32_t)stride; };
        return static_cast<char *>(t.p) + (times(b, t.batch) + times(s, t.token) + times(head(p), t.head)) * size;
    }
    __device__ __forceinline__ int64_t stat(const RopeParams &p) const {
        return (b * p.S + s) * (p.heads[0] + p.heads[1]) + (r ? p.heads[0] : 0) + head(p);
    }
};

// The backward's column sums of a CTA: acc[warp][D] in shared memory, each
// warp's own row filled with its sums of tensor r, added in the order of the
// warps into the CTA's partial row [2][D] (or [1][D] without keys) of block
// `which`.
__device__ __forceinline__ void rope_partial(const RopeParams &p, const float *acc, int which, int r) {
    const int n = p.D * (p.heads[1] ? 2 : 1);
    float *row = p.ws + ((int64_t)which * gridDim.x + blockIdx.x) * n + r * p.D;
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += kRopeCTA) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRopeWarps; ++w) v += acc[w * p.D + c];
        row[c] = v;
    }
    __syncthreads();  // acc may be filled again
}

// The sums of the tensor that a warp is not working on: N float4 a lane.
template <int N> struct RopeAside {
    float4 v[N][32];
    __device__ __forceinline__ void clear(int lane) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    // Changes places with f[0 .. 2 M - 1], kept from entry `at` on.
    template <int M> __device__ __forceinline__ void swap(float2 (&f)[2 * M], int at, int lane) {
#pragma unroll
        for (int i = 0; i < M; ++i) {
            const float4 t = v[at + i][lane];
            v[at + i][lane] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
            f[2 * i] = make_float2(t.x, t.y);
            f[2 * i + 1] = make_float2(t.z, t.w);
        }
    }
};

}  // namespace gbn
