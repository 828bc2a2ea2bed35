// Column sums: of fp32 partials, the second half of the weight gradients that are
// sums over rows (layer norm's dgamma and dbeta, linear's dbias), or of the rows
// themselves (dbias without an activation).
#pragma once

#include "elem16.h"
#include "token_internal.h"

namespace c3d {

// Floats of LDS that column_sum_block needs.
constexpr int column_sum_lds(int threads) { return threads / 4 * 17; }

// Block b takes 16 columns: THREADS / 4 threads per 4 columns add every
// (THREADS / 4)-th row, then 16 threads per column add those sums in a fixed
// order.  (64 bytes of each row per block, many rows in flight: 2048 columns of
// 1024 partials take 4.4 us, one row at a time took 20 us.)
template <typename E, int THREADS>
__device__ __forceinline__ void column_sum_block(const ColumnSumParams &p, int b, float *lds) {
    constexpr int LANES = THREADS / 4, PER = LANES / 16;
    const int tc = threadIdx.x & 3, tr = threadIdx.x >> 2;
    b = xcd_range(b, (p.cols + 15) / 16);  // the blocks that share cache lines on one XCD
    const int c = b * 16 + tc * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < p.cols && p.in16) {
#pragma unroll 8
        for (int r = tr; r < p.rows; r += LANES) {
            const e16x4_t u = *reinterpret_cast<const e16x4_t *>(p.in16 + r * p.stride + c);
            v.x += to_f32<E>(u[0]);
            v.y += to_f32<E>(u[1]);
            v.z += to_f32<E>(u[2]);
            v.w += to_f32<E>(u[3]);
        }
    } else if (c < p.cols) {
#pragma unroll 8
        for (int r = tr; r < p.rows; r += LANES) {
            const float4 u = *reinterpret_cast<const float4 *>(p.part + (int64_t)r * p.cols + c);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
    }
    float *row = lds + tr * 17 + tc * 4;
    row[0] = v.x;
    row[1] = v.y;
    row[2] = v.z;
    row[3] = v.w;
    __syncthreads();
    if (threadIdx.x >= 256) return;
    const int col = threadIdx.x >> 4, q = threadIdx.x & 15;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) t += lds[(q * PER + i) * 17 + col];
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) t += __shfl_xor(t, off);
    const int oc = b * 16 + col;
    if (q == 0 && oc < p.cols) {
        _Float16 *o = oc < p.split ? p.out0 : p.out1;
        if (o) o[oc < p.split ? oc : oc - p.split] = from_f32<E>(t);
    }
}

}  // namespace c3d
