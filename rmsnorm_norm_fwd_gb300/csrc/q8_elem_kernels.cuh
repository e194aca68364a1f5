// q8_elem_kernels.cuh -- forward and backward of the 8-bit operators one element
// at a time: one CTA per row, any row length, stride, alignment and combination
// of types.  They read a row two to four times (from L2 after the first) and
// serve rows longer than a cluster holds (131072 elements), which they only get
// right: an element a load and a CTA a row bound them.  512 x 262144 bf16, group
// scales: RMSNorm 1.3 ms, LayerNorm 2.1 ms (5% and 3% of the copy rate's time);
// backward 10.6 and 12.6 ms (1%), its column sums read and written for every row.
#pragma once

#include "q8_common.cuh"

namespace gbn {

// Maximum over a warp, NaN kept.
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_min_nan(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmin_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Forward.  Order of the passes: statistics (h is stored in the first and
// read from there on), checkpoint, then the output, so that h over x or r, or
// y over x or r, may be in place: every pass is over before the output's
// pass writes, and there each element is read by the thread that writes it.
template <bool LN>
__global__ void __launch_bounds__(kElemCTA) q8_fwd_elem(const Q8FwdParams p) {
    constexpr int W = kElemCTA / 32;
    __shared__ float red[2 * W];
    __shared__ float red_max[W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float n = (float)p.N;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const void *xr = row_ptr(p.x, row, p.ldx, p.xdt);
        const void *rr = p.res ? row_ptr(p.res, row, p.ldr, p.xdt) : nullptr;
        void *hr = p.h ? row_ptr(p.h, row, p.ldh, p.xdt) : nullptr;
        auto sum = [&](int64_t j) {
            const float x = ld1(xr, j, p.xdt);
            return rr ? round_to(x + ld1(rr, j, p.xdt), p.xdt) : x;
        };
        auto hval = [&](int64_t j) { return hr ? ld1(hr, j, p.xdt) : sum(j); };
        float s[1] = {0.f};
        for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA) {
            const float v = sum(j);
            if (hr) st1(hr, j, p.xdt, v);
            s[0] += LN ? v : v * v;
        }
        cta_allreduce<kElemCTA, 1>(s, red, parity);  // its barrier also makes h visible to the CTA
        float mean = 0.f;
        if constexpr (LN) {
            mean = s[0] / n;
            s[0] = 0.f;
            for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA) {
                const float d = hval(j) - mean;
                s[0] += d * d;
            }
            cta_allreduce<kElemCTA, 1>(s, red, parity);
        }
        const float rstd = rsqrtf(s[0] / n + p.eps);
        if (threadIdx.x == 0) {
            if (p.rstd) p.rstd[row] = rstd;
            if (LN && p.mean) p.mean[row] = mean;
        }
        if (p.c) {  // a warp per group
            const int64_t gn = (int64_t)1 << p.cg, groups = (p.N + gn - 1) >> p.cg;
            uint8_t *cr = p.c + row * p.ldc;
            for (int64_t g = warp; g < groups; g += W) {
                const int64_t j0 = g << p.cg, j1 = j0 + gn < p.N ? j0 + gn : p.N;
                float top = hval(j0), low = top;
                for (int64_t j = j0 + lane; j < j1; j += 32) {
                    const float v = hval(j);
                    top = fmax_nan(top, v);
                    low = fmin_nan(low, v);
                }
                const CkGroup k = ck_group(warp_max_nan(top), warp_min_nan(low));
                for (int64_t j = j0 + lane; j < j1; j += 32) cr[j] = (uint8_t)ck_code(hval(j), k);
                if (lane == 0) {
                    p.cs[row * p.ldcs + 2 * g] = k.scale;
                    p.cs[row * p.ldcs + 2 * g + 1] = k.mid;
                }
            }
            if (p.y) __syncthreads();  // y may be written over what the groups read
        }
        auto gam = [&](int64_t j) { return p.gamma ? ld1(p.gamma, j, p.pdt) : 1.f; };
        // RMSNorm's codes do not depend on rstd (it cancels in y / max|y|):
        // they are taken of h * gamma, and rstd enters the scale alone.
        auto out = [&](int64_t j) {
            if constexpr (!LN) return hval(j) * gam(j);
            return ((hval(j) - mean) * rstd) * gam(j) + (p.beta ? ld1(p.beta, j, p.pdt) : 0.f);
        };
        if (p.y) {
            void *yr = row_ptr(p.y, row, p.ldy, p.ydt);
            for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA)
                st1(yr, j, p.ydt, LN ? out(j) : (hval(j) * rstd) * gam(j));
            continue;
        }
        const float qmax = q8_max(p.qfmt), mul = LN ? 1.f : rstd;
        uint8_t *qr = p.q + row * p.ldq;
        if (p.qg >= 0) {  // a warp per group
            const int64_t gn = (int64_t)1 << p.qg, groups = (p.N + gn - 1) >> p.qg;
            for (int64_t g = warp; g < groups; g += W) {
                const int64_t j0 = g << p.qg, j1 = j0 + gn < p.N ? j0 + gn : p.N;
                float amax = 0.f;
                for (int64_t j = j0 + lane; j < j1; j += 32) amax = fmax_nan(amax, fabsf(out(j)));
                amax = warp_max_nan(amax);
                const float inv = q8_inv(amax, qmax);
                for (int64_t j = j0 + lane; j < j1; j += 32) qr[j] = q8_code(out(j) * inv, p.qfmt);
                if (lane == 0) p.qs[row * p.qs_row + g * p.qs_grp] = q8_scale(amax, mul, qmax, q8_inv_max(p.qfmt));
            }
        } else {
            float amax = 0.f;
            for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA) amax = fmax_nan(amax, fabsf(out(j)));
            amax = warp_max_nan(amax);
            __syncthreads();  // the previous row's readers of red_max are done
            if (lane == 0) red_max[warp] = amax;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < W; ++w) amax = fmax_nan(amax, red_max[w]);
            const float inv = q8_inv(amax, qmax);
            for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA) qr[j] = q8_code(out(j) * inv, p.qfmt);
            if (threadIdx.x == 0) p.qs[row * p.qs_row] = q8_scale(amax, mul, qmax, q8_inv_max(p.qfmt));
        }
    }
}

// Backward from the checkpoint; each CTA accumulates its partial dgamma/dbeta
// row in its own workspace row.
template <bool LN>
__global__ void __launch_bounds__(kElemCTA) q8_bwd_elem(const Q8BwdParams p) {
    pdl_launch_dependents();
    __shared__ float red[2 * 2 * (kElemCTA / 32)];
    const float n = (float)p.N;
    const int64_t P = gridDim.x;
    float *wsg = p.ws + (int64_t)blockIdx.x * p.N;
    float *wsb = p.ws + (P + blockIdx.x) * p.N;
    for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA) {
        wsg[j] = 0.f;
        if constexpr (LN) wsb[j] = 0.f;
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const void *dyr = row_ptr(p.dy, row, p.lddy, p.ydt);
        const uint8_t *cr = p.c + row * p.ldc;
        const float *cs = p.cs + row * p.ldcs;
        const float rstd = __ldg(p.rstd + row);
        const float mean = LN ? __ldg(p.mean + row) : 0.f;
        auto gam = [&](int64_t j) { return p.gamma ? ld1(p.gamma, j, p.pdt) : 1.f; };
        auto xhat = [&](int64_t j) {
            const int64_t g = j >> p.cg;
            return (fmaf(__ldg(cs + 2 * g), (float)(int8_t)cr[j], __ldg(cs + 2 * g + 1)) - mean) * rstd;
        };
        float s[2] = {0.f, 0.f};
        for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA) {
            const float g = ld1(dyr, j, p.ydt) * gam(j);
            s[0] += g * xhat(j);
            s[1] += g;
        }
        cta_allreduce<kElemCTA, 2>(s, red, parity);
        const float c2 = s[0] / n;
        const float c1 = LN ? s[1] / n : 0.f;
        void *dxr = row_ptr(p.dx, row, p.lddx, p.xdt);
        const void *drr = p.dres ? row_ptr(p.dres, row, p.lddres, p.xdt) : nullptr;
        for (int64_t j = threadIdx.x; j < p.N; j += kElemCTA) {
            const float xh = xhat(j), dyv = ld1(dyr, j, p.ydt);
            float o = rstd * (dyv * gam(j) - c1 - xh * c2);
            if (drr) o += ld1(drr, j, p.xdt);
            st1(dxr, j, p.xdt, o);
            wsg[j] += dyv * xh;
            if constexpr (LN) wsb[j] += dyv;
        }
    }
}

}  // namespace gbn
