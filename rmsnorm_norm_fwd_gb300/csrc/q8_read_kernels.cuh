// q8_read_kernels.cuh -- 8-bit rows read back.
//
// Nothing is reduced: a thread keeps one chunk of 8 columns, with gamma and
// beta of it in registers, and walks down the rows, four at a time so that
// enough loads are in flight.  What bounds it: DRAM, 1 byte in and 2 (4) out an
// element.
#pragma once

#include "q8_bwd_kernels.cuh"

namespace gbn {

constexpr int kReadCTA = 256, kReadRows = 4;

// blockDim.x = tx * ry threads: tx chunks of a column block (blockIdx.x), ry
// rows side by side.  NORM: statistics, gamma or beta are given.
template <int FMT, bool NORM, int YT>
__global__ void __launch_bounds__(kReadCTA) q8_read_vec(const Q8ReadParams p, int tx) {
    constexpr int yes = YT == kF32 ? 4 : 2;
    const int ry = blockDim.x / tx, r = threadIdx.x / tx;
    const int c = blockIdx.x * tx + threadIdx.x % tx;
    if (c >= (int)(p.N / 8) || r >= ry) return;
    float2 g8[4], b8[4];
    if constexpr (NORM) {
        par8g(p.gamma, c, p.pdt, 1.f, g8);
        par8g(p.beta, c, p.pdt, 0.f, b8);
    }
    const int64_t group = p.qg >= 0 ? c >> (p.qg - 3) : 0;
    const int64_t step = (int64_t)gridDim.y * ry;
    for (int64_t row0 = (int64_t)blockIdx.y * ry + r; row0 < p.M; row0 += kReadRows * step) {
        uint2 w[kReadRows];
        float scale[kReadRows], mid[kReadRows], mean[kReadRows], rstd[kReadRows];
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            const int64_t row = row0 + i * step;
            w[i] = make_uint2(0, 0);
            scale[i] = mid[i] = mean[i] = 0.f;
            rstd[i] = 1.f;
            if (row < p.M) {
                w[i] = ld_codes8(p.q + row * p.ldq, c);
                const int64_t at = row * p.s_row + group * p.s_grp;
                scale[i] = __ldg(p.scale + at);
                if (p.mid) mid[i] = __ldg(p.mid + at);
                if constexpr (NORM) {
                    if (p.mean) mean[i] = __ldg(p.mean + row);
                    if (p.rstd) rstd[i] = __ldg(p.rstd + row);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            const int64_t row = row0 + i * step;
            if (row >= p.M) break;
            float2 v[4];
            if constexpr (FMT == kI8) {
                i8_pairs(w[i], v);
            } else {
                v[0] = e4m3_to_f2(w[i].x & 0xffffu), v[1] = e4m3_to_f2(w[i].x >> 16);
                v[2] = e4m3_to_f2(w[i].y & 0xffffu), v[3] = e4m3_to_f2(w[i].y >> 16);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = f2fma(v[j], f2s(scale[i]), f2s(mid[i]));
                if constexpr (NORM)
                    v[j] = f2add(f2mul(f2mul(f2add(v[j], f2s(-mean[i])), f2s(rstd[i])), g8[j]), b8[j]);
            }
            st_raw8<YT>(static_cast<unsigned char *>(p.y) + row * p.ldy * yes, c, pack8<YT>(v));
        }
    }
}

}  // namespace gbn
