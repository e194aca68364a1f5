// q8_read_kernels.cuh -- 8-bit rows read back.
//
// Nothing is reduced: a thread keeps one chunk of 8 columns, with gamma and
// beta of it in registers, and walks down the rows, kReadRows at a time so that
// enough loads are in flight.  With the statistics folded into the group's
// (scale, mid) a value is one multiply-add of its code, a second one with the
// norm on top.  What bounds it: DRAM, 1 byte in and 2 (4) out an element.
// Measured: 65536 x 2048 with the norm 65 us (93% of the copy rate's time); with
// the statistics folded in as they were loaded the loads waited for one another
// (92 us).
#pragma once

#include "q8_bwd_kernels.cuh"

namespace gbn {

constexpr int kReadCTA = 256, kReadRows = 4;

// blockDim.x = tx * ry threads: tx chunks of a column block (blockIdx.x), ry
// rows side by side.  NORM: statistics, gamma or beta are given.  PAIR: scale
// and mid side by side, 8-byte aligned (a checkpoint).
template <int FMT, bool NORM, bool PAIR, int YT>
__global__ void __launch_bounds__(kReadCTA, 4) q8_read_vec(const Q8ReadParams p, int tx) {
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
    const int64_t rq = ry * p.ldq, rs = ry * p.s_row, ryb = ry * p.ldy * yes;  // from one of a thread's rows to the next
    const int64_t step = (int64_t)gridDim.y * ry * kReadRows;
    const int width = min(tx, (int)(p.N / 8) - (int)blockIdx.x * tx) * 8;
    // kReadRows * ry consecutive rows at a time
    for (int64_t row0 = (int64_t)blockIdx.y * ry * kReadRows + r; row0 < p.M; row0 += step) {
        if (threadIdx.x % tx < kReadRows) {  // the next rows' codes on their way to L2
            const int64_t next = row0 + step + (threadIdx.x % tx) * ry;
            if (next < p.M) prefetch_l2_inner(p.q + next * p.ldq + 8 * (int64_t)blockIdx.x * tx, width);
        }
        const uint8_t *q = p.q + row0 * p.ldq;
        const int64_t at0 = row0 * p.s_row + group * p.s_grp;
        unsigned char *y = static_cast<unsigned char *>(p.y) + row0 * p.ldy * yes;
        uint2 w[kReadRows];
        float a[kReadRows], b[kReadRows], mean[kReadRows], rstd[kReadRows];  // a, b: scale, mid
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            const int64_t row = row0 + i * ry, at = at0 + i * rs;
            w[i] = make_uint2(0, 0);
            a[i] = b[i] = mean[i] = 0.f;
            rstd[i] = 1.f;
            if (row < p.M) {
                w[i] = ld_codes8(q + i * rq, c);
                if constexpr (PAIR) {
                    const float2 sm = __ldg(reinterpret_cast<const float2 *>(p.scale + at));
                    a[i] = sm.x, b[i] = sm.y;
                } else {
                    a[i] = __ldg(p.scale + at);
                    if (p.mid) b[i] = __ldg(p.mid + at);
                }
                if constexpr (NORM) {
                    if (p.mean) mean[i] = __ldg(p.mean + row);
                    if (p.rstd) rstd[i] = __ldg(p.rstd + row);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kReadRows; ++i) {
            float2 v[4];
            if constexpr (NORM) {  // value = code * a + b
                a[i] *= rstd[i];
                b[i] = (b[i] - mean[i]) * rstd[i];
            }
            if constexpr (FMT == kI8) {
                i8_pairs(w[i], v);
            } else {
                v[0] = e4m3_to_f2(w[i].x & 0xffffu), v[1] = e4m3_to_f2(w[i].x >> 16);
                v[2] = e4m3_to_f2(w[i].y & 0xffffu), v[3] = e4m3_to_f2(w[i].y >> 16);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = f2fma(v[j], f2s(a[i]), f2s(b[i]));
                if constexpr (NORM) v[j] = f2fma(v[j], g8[j], b8[j]);
            }
            if (row0 + i * ry < p.M) st_raw8<YT>(y + i * ryb, c, pack8<YT>(v));
        }
    }
}

}  // namespace gbn
