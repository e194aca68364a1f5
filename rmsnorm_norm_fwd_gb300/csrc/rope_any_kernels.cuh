// rope_any_kernels.cuh -- the head operators element by element: any head
// size up to 1024, alignment, strides and types.
//
// A warp takes one head at a time.  A lane holds N pairs: rotated pair j =
// lane + 32 i, behind the rotated ones the rest of the head in pairs that are
// not rotated (elements rot + u and rot + rest + u, the last of which may be
// missing), so that rotation needs no exchange and a lane computes the cosines
// of its own pairs, once a token.
//
// What bounds it: an element a load and a store, latency.  It serves what the
// vector kernels cannot (heads without vectors of 8 bytes, mixed types).
#pragma once

#include "rope_common.cuh"

namespace gbn {

// Element indexes of a lane's pairs; second -1 where there is none, both where the pair is not there.
template <int N> struct RopeSlots {
    int a[N], b[N];
    uint32_t turned;  // one bit a pair
    __device__ __forceinline__ RopeSlots(const RopeParams &p, int lane) {
        const int half = p.rot / 2, rest = (p.D - p.rot + 1) / 2;
        turned = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int j = lane + 32 * i, u = j - half;
            if (u < 0) {
                a[i] = p.inter ? 2 * j : j;
                b[i] = p.inter ? 2 * j + 1 : j + half;
                turned |= 1u << i;
            } else {
                a[i] = u < rest ? p.rot + u : -1;
                b[i] = u < rest && p.rot + rest + u < p.D ? p.rot + rest + u : -1;
            }
        }
    }
};

template <int N>
__device__ __forceinline__ void rope_any_load(const RopeSlots<N> &sl, const void *p, int64_t at, int dt, float (&a)[N],
                                              float (&b)[N], float none = 0.f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        a[i] = sl.a[i] >= 0 ? (p ? ld1(p, at + sl.a[i], dt) : 1.f) : none;
        b[i] = sl.b[i] >= 0 ? (p ? ld1(p, at + sl.b[i], dt) : 1.f) : none;
    }
}
template <int N>
__device__ __forceinline__ void rope_any_store(const RopeSlots<N> &sl, void *p, int64_t at, int dt, const float (&a)[N],
                                               const float (&b)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (sl.a[i] >= 0) st1(p, at + sl.a[i], dt, a[i]);
        if (sl.b[i] >= 0) st1(p, at + sl.b[i], dt, b[i]);
    }
}

template <int MODE, int N>
__global__ void __launch_bounds__(kRopeCTA) rope_fwd_any(const RopeParams p) {
    const int lane = threadIdx.x & 31;
    RopeWalk w(p);
    if (!w.left) return;
    const RopeSlots<N> sl(p, lane);
    RopeAngles<N> ang;
    ang.init(p, lane);
    float ga[N], gb[N], ba[N], bb[N], c[N], s[N];
    if constexpr (MODE != kRopeOnly) rope_any_load(sl, p.gamma[w.r], 0, p.pdt, ga, gb);
#pragma unroll
    for (int i = 0; i < N; ++i) ba[i] = bb[i] = 0.f;
    if constexpr (MODE == kRopeLn)
        if (p.beta[w.r]) rope_any_load(sl, p.beta[w.r], 0, p.pdt, ba, bb);
    const float inv = 1.f / (float)p.D;
    const RopeHeads x = p.x[w.r], y = p.y[w.r];
    for (bool fresh = true; w.left; fresh = w.next(p)) {
        if (fresh)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((sl.turned >> i) & 1u) ang.get(p, w.b * p.pos_batch + w.s * p.pos_token, i, c + i, s + i);
        float a[N], b[N];
        rope_any_load(sl, x.p, w.at(x) + w.blk * x.head, p.xdt, a, b);
        if constexpr (MODE != kRopeOnly) {
            float sum[1] = {0.f};
            if constexpr (MODE == kRopeLn) {
#pragma unroll
                for (int i = 0; i < N; ++i) sum[0] += a[i] + b[i];
                group_sum<32, 1>(sum);
                sum[0] *= inv;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    a[i] = sl.a[i] >= 0 ? a[i] - sum[0] : 0.f;
                    b[i] = sl.b[i] >= 0 ? b[i] - sum[0] : 0.f;
                }
            }
            float sq[1] = {0.f};
#pragma unroll
            for (int i = 0; i < N; ++i) sq[0] += a[i] * a[i] + b[i] * b[i];
            group_sum<32, 1>(sq);
            const float rstd = rsqrtf(sq[0] * inv + p.eps);
            if (lane == 0) {
                const int64_t at = w.stat(p) + w.blk;
                if (p.rstd) p.rstd[at] = rstd;
                if (MODE == kRopeLn && p.mean) p.mean[at] = sum[0];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                a[i] = a[i] * rstd * ga[i] + ba[i];
                b[i] = b[i] * rstd * gb[i] + bb[i];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((sl.turned >> i) & 1u) {
                const float v = a[i];
                a[i] = v * c[i] - b[i] * s[i];
                b[i] = b[i] * c[i] + v * s[i];
            }
        rope_any_store(sl, y.p, w.at(y) + w.blk * y.head, p.ydt, a, b);
    }
}

template <bool LN, int N>
__global__ void __launch_bounds__(kRopeCTA) rope_bwd_any(const RopeParams p) {
    pdl_launch_dependents();  // the column reduce waits for this grid's completion
    extern __shared__ __align__(16) float rope_acc[];  // [kRopeWarps][D]
    const int lane = threadIdx.x & 31;
    RopeWalk w(p);
    const RopeSlots<N> sl(p, lane);
    float ga[N], gb[N], c[N], s[N], da[N], db[N], ea[N], eb[N];
    RopeAngles<N> ang;
    if (w.left) {
        ang.init(p, lane);
        rope_any_load(sl, p.gamma[w.r], 0, p.pdt, ga, gb);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) da[i] = db[i] = ea[i] = eb[i] = 0.f;
    const float inv = 1.f / (float)p.D;
    const RopeHeads x = p.x[w.r], g = p.g[w.r], y = p.y[w.r];
    for (bool fresh = true; w.left; fresh = w.next(p)) {
        if (fresh)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((sl.turned >> i) & 1u) ang.get(p, w.b * p.pos_batch + w.s * p.pos_token, i, c + i, s + i);
        float a[N], b[N], u[N], v[N];
        rope_any_load(sl, x.p, w.at(x) + w.blk * x.head, p.xdt, a, b);
        rope_any_load(sl, g.p, w.at(g) + w.blk * g.head, p.ydt, u, v);
        const int64_t at = w.stat(p) + w.blk;
        const float rstd = p.rstd[at], mean = LN ? p.mean[at] : 0.f;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if ((sl.turned >> i) & 1u) {  // the transpose: sign is -1 in the angles
                const float t = u[i];
                u[i] = t * c[i] - v[i] * s[i];
                v[i] = v[i] * c[i] + t * s[i];
            }
            a[i] = sl.a[i] >= 0 ? (a[i] - mean) * rstd : 0.f;
            b[i] = sl.b[i] >= 0 ? (b[i] - mean) * rstd : 0.f;
            da[i] += u[i] * a[i];
            db[i] += v[i] * b[i];
            if constexpr (LN) {
                ea[i] += u[i];
                eb[i] += v[i];
            }
            u[i] *= ga[i];
            v[i] *= gb[i];
            sum[0] += u[i] * a[i] + v[i] * b[i];
            if constexpr (LN) sum[1] += u[i] + v[i];
        }
        group_sum<32, 2>(sum);
        const float c2 = sum[0] * inv, c1 = sum[1] * inv;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] = rstd * (u[i] - c1 - a[i] * c2);
            b[i] = rstd * (v[i] - c1 - b[i] * c2);
        }
        rope_any_store(sl, y.p, w.at(y) + w.blk * y.head, p.xdt, a, b);
    }
    float *mine = rope_acc + (threadIdx.x >> 5) * p.D;
    rope_any_store(sl, mine, 0, kF32, da, db);
    rope_partial(p, rope_acc, 0);
    if constexpr (LN) {
        rope_any_store(sl, mine, 0, kF32, ea, eb);
        rope_partial(p, rope_acc, 1);
    }
}

}  // namespace gbn
