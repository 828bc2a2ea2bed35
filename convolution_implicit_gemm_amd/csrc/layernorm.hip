// Layer norm over the channels of token rows, forward and backward, gfx950.
//
//   forward:  mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//             y = (x - mu) r gamma + beta
//   backward: g = dy gamma, xh = (x - mu) r,
//             dx = r (g - mean(g) - xh mean(g xh)) (+ dres),
//             dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
//
// Both are streams over HBM (2 reads and writes of a row forward, 3 or 4
// backward), so a row is read once and stays in registers: a team of WPR waves
// holds one row as NV 16-byte vectors per lane, and the second moment is taken
// about the mean in a second sweep over the registers (no cancellation, at no
// traffic).  Sums are fp32; y, dx and the weight gradients are rounded once.
// The weights' gradients: every team walks rows blockwise and keeps its
// columns' sums in registers, the block adds its teams through LDS and writes
// one fp32 partial, and a second kernel adds the blocks in a fixed order (no
// atomics: the result does not depend on the order blocks finish in).  Up to
// 2048 rows other blocks of the same launch take 16 columns each and walk all
// rows, whose statistics are known, instead: dy and x are read twice, from L2,
// but nothing has to be joined.
//
// Measured, bf16: 36864 x 2048 forward 54-57 us, 5.3-5.6 TB/s (copies: 4.9 to 6.0);
// its gradient with a residual's 120 us, 5.0 TB/s.  Few rows are bound by latency: 1
// x 1024 2.4 us, the gradients of 1543 x 1032 5.1 us.
#include "column_sum.h"

namespace c3d {

namespace {

constexpr int64_t kLnWideRows = 512, kLnColumnRows = 2048;

// Sum over the wave, the same in every lane: shifted adds within rows of 16
// lanes, then the rows' last lanes into the next rows, all in vector
// registers (a shuffle through LDS per step doubles a small row's latency).
__device__ __forceinline__ float wave_sum(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
#define C3D_DPP_ADD(ctrl, rows)                                                                                    \
    v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), ctrl, rows, 0xf, false))
    C3D_DPP_ADD(0x111, 0xf);  // row_shr:1
    C3D_DPP_ADD(0x112, 0xf);  // row_shr:2
    C3D_DPP_ADD(0x114, 0xf);  // row_shr:4
    C3D_DPP_ADD(0x118, 0xf);  // row_shr:8: lane 15 of each row holds the row's sum
    C3D_DPP_ADD(0x142, 0xa);  // row_bcast:15 into rows 1 and 3
    C3D_DPP_ADD(0x143, 0xc);  // row_bcast:31 into rows 2 and 3: lane 63 holds the sum
#undef C3D_DPP_ADD
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
#else
    return v;
#endif
}

// Sum over the WPR waves of a row's team.  slot: this team's 2 x WPR floats of
// LDS; `turn` alternates, so that one barrier per sum is enough.
template <int WPR>
__device__ __forceinline__ float team_sum(float v, float *slot, int wave_in_team, int turn) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        float *s = slot + turn * WPR;
        if ((threadIdx.x & 63) == 0) s[wave_in_team] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < WPR; ++i) v += s[i];
    }
    return v;
}

template <typename E>
__device__ __forceinline__ e16x8_t load_vec(const _Float16 *p) {
    return *reinterpret_cast<const e16x8_t *>(p);
}

// Threads of a block: one row's team, or four one-wave teams.
template <int WPR>
constexpr int ln_threads() {
    return (WPR > 4 ? WPR : 4) * 64;
}

template <typename E, int NV, int WPR>
__global__ __launch_bounds__(ln_threads<WPR>()) void layernorm_kernel(LnParams p) {
    constexpr int TEAMS = ln_threads<WPR>() / 64 / WPR;
    __shared__ float red[TEAMS * 2 * WPR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int team = wave / WPR, wt = wave % WPR;
    const int first = (wt * 64 + lane) * 8;
    float *slot = red + team * 2 * WPR;
    const float inv_c = 1.0f / (float)p.c;
    for (int64_t row0 = (int64_t)blockIdx.x * TEAMS; row0 < p.rows; row0 += (int64_t)gridDim.x * TEAMS) {
        const int64_t row = row0 + team;
        const bool live = row < p.rows;  // a team past the end keeps the barriers' count
        e16x8_t v[NV];
        const _Float16 *xr = p.x + row * p.x_stride;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = first + i * WPR * 512;
            v[i] = live && c < p.c ? load_vec<E>(xr + c) : e16x8_t{};
#pragma unroll
            for (int e = 0; e < 8; ++e) s += to_f32<E>(v[i][e]);
        }
        const float mean = team_sum<WPR>(s, slot, wt, 0) * inv_c;
        float s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * WPR * 512 < p.c)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float d = to_f32<E>(v[i][e]) - mean;
                    s2 = fmaf(d, d, s2);
                }
        const float rstd = 1.0f / sqrtf(team_sum<WPR>(s2, slot, wt, 1) * inv_c + p.eps);
        if (!live) continue;
        _Float16 *yr = p.y + row * p.y_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = first + i * WPR * 512;
            if (c >= p.c) continue;
            const e16x8_t ga = p.gamma ? load_vec<E>(p.gamma + c) : e16x8_t{};
            const e16x8_t be = p.beta ? load_vec<E>(p.beta + c) : e16x8_t{};
            e16x8_t o;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float a = p.gamma ? rstd * to_f32<E>(ga[e]) : rstd;
                o[e] = from_f32<E>(fmaf(to_f32<E>(v[i][e]) - mean, a, to_f32<E>(be[e])));
            }
            *reinterpret_cast<e16x8_t *>(yr + c) = o;
        }
        if (p.stats && wt == 0 && lane == 0) p.stats[row] = make_float2(mean, rstd);
    }
}

// dx of the rows that workgroup `block` of `blocks` walks and, with SUMS, its
// partial of the weights' gradients.
template <typename E, int NV, int WPR, bool SUMS>
__device__ __forceinline__ void ln_grad_rows(const LnGradParams &p, int block, int blocks, float *join) {
    constexpr int TEAMS = ln_threads<WPR>() / 64 / WPR;
    constexpr int SPAN = NV * WPR * 512;  // columns a team covers
    __shared__ float red[TEAMS * 2 * WPR];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int team = wave / WPR, wt = wave % WPR;
    const int first = (wt * 64 + lane) * 8;
    float *slot = red + team * 2 * WPR;
    const float inv_c = 1.0f / (float)p.c;
    e16x8_t ga[NV];
    float dg[SUMS ? NV : 1][8], db[SUMS ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = first + i * WPR * 512;
        ga[i] = p.gamma && c < p.c ? load_vec<E>(p.gamma + c) : e16x8_t{};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!p.gamma) ga[i][e] = from_f32<E>(1.0f);
            if constexpr (SUMS) dg[i][e] = db[i][e] = 0.0f;
        }
    }
    // The next row's loads are issued before the current row is worked on (a
    // block of 16 waves has no registers to spare for that).
    constexpr bool AHEAD = WPR < 16;
    struct Row {
        e16x8_t x[NV], dy[NV], dres[NV];
        float2 st;
    };
    const int64_t step = (int64_t)blocks * TEAMS;
    auto fetch = [&](int64_t row, Row &r) {
        const bool live = row < p.rows;
        r.st = live ? p.stats[row] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = first + i * WPR * 512;
            const bool in = live && c < p.c;
            r.x[i] = in ? load_vec<E>(p.x + row * p.x_stride + c) : e16x8_t{};
            r.dy[i] = in ? load_vec<E>(p.dy + row * p.y_stride + c) : e16x8_t{};
            r.dres[i] = in && p.dres ? load_vec<E>(p.dres + row * p.x_stride + c) : e16x8_t{};
        }
    };
    Row cur, next;
    int64_t row = (int64_t)block * TEAMS + team;
    const int64_t rounds = (p.rows - (int64_t)block * TEAMS + step - 1) / step;  // the same for all teams
    if (AHEAD) fetch(row, cur);
    for (int64_t k = 0; k < rounds; ++k, row += step) {
        if (!AHEAD)
            fetch(row, cur);
        else if (k + 1 < rounds)
            fetch(row + step, next);
        float s1 = 0.0f, s2 = 0.0f;
        // columns past the end and rows past the end read zeros with zero
        // statistics: they add nothing
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (first + i * WPR * 512 < p.c)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = (to_f32<E>(cur.x[i][e]) - cur.st.x) * cur.st.y, d = to_f32<E>(cur.dy[i][e]);
                    const float g = d * to_f32<E>(ga[i][e]);
                    s1 += g;
                    s2 = fmaf(g, xh, s2);
                    if constexpr (SUMS) {
                        dg[i][e] = fmaf(d, xh, dg[i][e]);
                        db[i][e] += d;
                    }
                }
        s1 = team_sum<WPR>(s1, slot, wt, 0) * inv_c;
        s2 = team_sum<WPR>(s2, slot, wt, 1) * inv_c;
        if (row < p.rows)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = first + i * WPR * 512;
                if (c >= p.c) continue;
                e16x8_t o;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float xh = (to_f32<E>(cur.x[i][e]) - cur.st.x) * cur.st.y;
                    const float g = to_f32<E>(cur.dy[i][e]) * to_f32<E>(ga[i][e]);
                    o[e] = from_f32<E>(fmaf(cur.st.y, g - s1 - xh * s2, to_f32<E>(cur.dres[i][e])));
                }
                *reinterpret_cast<e16x8_t *>(p.dx + row * p.x_stride + c) = o;
            }
        if (AHEAD) cur = next;
    }
    if constexpr (SUMS) {
        float *out = p.part + (int64_t)block * 2 * p.c;
        auto put = [&](float *to, const float (&v)[8]) {
            *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
        };
    #pragma unroll
        for (int which = 0; which < 2; ++which) {
    #pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = first + i * WPR * 512;
                if constexpr (TEAMS > 1)
                    put(join + team * SPAN + c, which ? db[i] : dg[i]);
                else if (c < p.c)
                    put(out + which * p.c + c, which ? db[i] : dg[i]);
            }
            if constexpr (TEAMS > 1) {  // add the teams in turn
                __syncthreads();
                for (int c = threadIdx.x * 4; c < p.c; c += ln_threads<WPR>() * 4) {
                    float4 t = *reinterpret_cast<const float4 *>(join + c);
    #pragma unroll
                    for (int k = 1; k < TEAMS; ++k) {
                        const float4 u = *reinterpret_cast<const float4 *>(join + k * SPAN + c);
                        t.x += u.x;
                        t.y += u.y;
                        t.z += u.z;
                        t.w += u.w;
                    }
                    *reinterpret_cast<float4 *>(out + which * p.c + c) = t;
                }
                __syncthreads();
            }
        }
    }
}

// dgamma and dbeta of 16 columns, straight from dy, x and the rows' statistics:
// two threads per row, THREADS / 2 rows at once, their sums through LDS in a
// fixed order.  Bound by the latency of a thread's rows.  The column blocks that
// share cache lines run on one XCD (dealt out in turn: 1543 x 1032 8.1 us, so
// 5.1); 8 or 32 columns, or 8 rows ahead instead of 4, are within 20% either way.
constexpr int kLnCols = 16;
constexpr int ln_cols_lds(int threads) { return threads * 8 / kLnCols * (2 * kLnCols + 1); }
template <typename E, int THREADS>
__device__ __forceinline__ void ln_grad_cols(const LnGradParams &p, int block, float *lds) {
    constexpr int PER_ROW = kLnCols / 8, ROWS = THREADS / PER_ROW, OUT = 2 * kLnCols, PARTS = THREADS / OUT;
    const int tc = threadIdx.x % PER_ROW, tr = threadIdx.x / PER_ROW;
    const int c = block * kLnCols + tc * 8;
    float dg[8] = {}, db[8] = {};
    if (c < p.c)
#pragma unroll 4
        for (int64_t r = tr; r < p.rows; r += ROWS) {
            const float2 st = p.stats[r];
            const e16x8_t x = load_vec<E>(p.x + r * p.x_stride + c), dy = load_vec<E>(p.dy + r * p.y_stride + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = to_f32<E>(dy[e]);
                dg[e] = fmaf(d, (to_f32<E>(x[e]) - st.x) * st.y, dg[e]);
                db[e] += d;
            }
        }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        lds[tr * (OUT + 1) + tc * 8 + e] = dg[e];
        lds[tr * (OUT + 1) + kLnCols + tc * 8 + e] = db[e];
    }
    __syncthreads();
    const int o = threadIdx.x % OUT, part = threadIdx.x / OUT;
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < ROWS / PARTS; ++i) t += lds[(part * (ROWS / PARTS) + i) * (OUT + 1) + o];
    __syncthreads();
    lds[part * OUT + o] = t;
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int i = 1; i < PARTS; ++i) t += lds[i * OUT + o];
    const int oc = block * kLnCols + o % kLnCols;
    _Float16 *out = o < kLnCols ? p.dgamma : p.dbeta;
    if (out && oc < p.c) out[oc] = from_f32<E>(t);
}

template <typename E, int NV, int WPR>
__global__ __launch_bounds__(ln_threads<WPR>()) void layernorm_grad_kernel(LnGradParams p) {
    constexpr int TEAMS = ln_threads<WPR>() / 64 / WPR;
    __shared__ __attribute__((aligned(16))) float join[TEAMS > 1 ? TEAMS * NV * WPR * 512 : 4];
    ln_grad_rows<E, NV, WPR, true>(p, blockIdx.x, gridDim.x, join);
}

// Blocks [0, col_blocks) own columns of the weights' gradients, the others rows of dx.
template <typename E, int NV, int WPR>
__global__ __launch_bounds__(ln_threads<WPR>()) void layernorm_grad_split_kernel(LnGradParams p, int col_blocks) {
    __shared__ float lds[ln_cols_lds(ln_threads<WPR>())];
    const int b = blockIdx.x;
    if (b < col_blocks)
        ln_grad_cols<E, ln_threads<WPR>()>(p, xcd_range(b, col_blocks), lds);
    else
        ln_grad_rows<E, NV, WPR, false>(p, b - col_blocks, gridDim.x - col_blocks, nullptr);
}

template <typename E>
__global__ __launch_bounds__(256) void column_sum_kernel(ColumnSumParams p) {
    __shared__ float lds[column_sum_lds(256)];
    column_sum_block<E, 256>(p, blockIdx.x, lds);
}

__global__ __launch_bounds__(256) void zero_rows_kernel(_Float16 *y, int64_t rows, int width, int64_t stride) {
    const int64_t total = rows * width;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256)
        y[i / width * stride + i % width] = (_Float16)0.0f;
}

// (vectors per lane, waves per row) of a channel count.  `wide`: one row per
// block of four waves also where a wave could hold it.
template <typename F>
hipError_t ln_dispatch(int c, bool wide, F &&f) {
    using std::integral_constant;
    if (c <= 512) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
    if (wide && c <= 2048) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
    if (c <= 1024) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
    if (c <= 2048) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
    if (c <= 4096) return f(integral_constant<int, 2>{}, integral_constant<int, 4>{});
    if (c <= 8192) return f(integral_constant<int, 2>{}, integral_constant<int, 8>{});
    return f(integral_constant<int, 2>{}, integral_constant<int, 16>{});
}

// Few rows: a row's latency counts, not the stream's rate.  (200 x 1032: forward
// 3.9 -> 3.2 us, gradient 9.6 -> 7.0; 36864 x 1024: gradient 44 -> 85 us.)
bool ln_wide(int64_t rows) { return rows <= kLnWideRows; }
int ln_teams(int64_t rows, int c) { return c <= (ln_wide(rows) ? 512 : 2048) ? 4 : 1; }

}  // namespace

hipError_t launch_layernorm(const LnParams &p, hipStream_t s) {
    const int64_t want = (p.rows + ln_teams(p.rows, p.c) - 1) / ln_teams(p.rows, p.c);
    const unsigned grid = (unsigned)(want < 65536 ? want : 65536);
    return ln_dispatch(p.c, ln_wide(p.rows), [&](auto nv, auto wpr) {
        constexpr int NV = decltype(nv)::value, WPR = decltype(wpr)::value;
        if (p.bf16)
            hipLaunchKernelGGL((layernorm_kernel<__bf16, NV, WPR>), dim3(grid), dim3(ln_threads<WPR>()), 0, s, p);
        else
            hipLaunchKernelGGL((layernorm_kernel<_Float16, NV, WPR>), dim3(grid), dim3(ln_threads<WPR>()), 0, s, p);
        return hipGetLastError();
    });
}

int32_t ln_grad_blocks(int64_t rows, int32_t c) {
    // two rows per team and more: a block's partial is written and read again, as
    // much traffic as two or three rows.  Up to four, while 256 blocks are left.
    const int64_t passes = (rows + ln_teams(rows, c) - 1) / ln_teams(rows, c);
    int64_t rounds = (passes + 255) / 256;
    if (rounds > 4) rounds = (passes + 511) / 512 < 4 ? 4 : (passes + 511) / 512;
    if (rounds < 2 && passes > 1) rounds = 2;
    return (int32_t)((passes + rounds - 1) / rounds);
}

hipError_t launch_layernorm_grad(const LnGradParams &p, hipStream_t s) {
    const bool wide = ln_wide(p.rows);
    // One launch for few rows (all gradients, bf16: 1 x 1024 4.6 -> 2.6 us, 613 x 2048
    // 9.8 -> 5.0, 1543 x 1032 9.8 -> 5.1, 2000 x 1024 9.8 -> 6.6, 2000 x 8192 40 -> 28,
    // 513 x 16384 level, 2048 x 16384 56 -> 63;
    // 3000 x 2048 14.7 -> 15.7, 4097 x 1024 13.0 -> 16.3) and for dx alone (36864 x 2048
    // 92 -> 78).  dx in place of dy or x would change what the columns' blocks read.
    const bool in_place = p.dx == p.dy || p.dx == p.x;
    if (!p.part || (!in_place && p.rows <= kLnColumnRows)) {
        const int cols = p.part ? (p.c + kLnCols - 1) / kLnCols : 0;
        const int64_t want = (p.rows + ln_teams(p.rows, p.c) - 1) / ln_teams(p.rows, p.c);
        const unsigned grid = (unsigned)(cols + (want < 65536 ? want : 65536));
        return ln_dispatch(p.c, wide, [&](auto nv, auto wpr) {
            constexpr int NV = decltype(nv)::value, WPR = decltype(wpr)::value;
            const auto go = [&](auto *kernel) {
                hipLaunchKernelGGL(kernel, dim3(grid), dim3(ln_threads<WPR>()), 0, s, p, cols);
            };
            if (p.bf16)
                go(layernorm_grad_split_kernel<__bf16, NV, WPR>);
            else
                go(layernorm_grad_split_kernel<_Float16, NV, WPR>);
            return hipGetLastError();
        });
    }
    const unsigned grid = (unsigned)ln_grad_blocks(p.rows, p.c);
    hipError_t e = ln_dispatch(p.c, wide, [&](auto nv, auto wpr) {
        constexpr int NV = decltype(nv)::value, WPR = decltype(wpr)::value;
        const auto go = [&](auto *kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(ln_threads<WPR>()), 0, s, p); };
        if (p.bf16)
            go(layernorm_grad_kernel<__bf16, NV, WPR>);
        else
            go(layernorm_grad_kernel<_Float16, NV, WPR>);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    ColumnSumParams cs = {};
    cs.part = p.part;
    cs.out0 = p.dgamma;
    cs.out1 = p.dbeta;
    cs.rows = (int32_t)grid;
    cs.cols = 2 * p.c;
    cs.split = p.c;
    cs.bf16 = p.bf16;
    return launch_column_sum(cs, s);
}

hipError_t launch_column_sum(const ColumnSumParams &p, hipStream_t s) {
    const dim3 grid((unsigned)((p.cols + 15) / 16));
    if (p.bf16)
        hipLaunchKernelGGL((column_sum_kernel<__bf16>), grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((column_sum_kernel<_Float16>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_zero_rows(_Float16 *y, int64_t rows, int32_t width, int64_t stride, hipStream_t s) {
    const int64_t blocks = (rows * width + 1023) / 1024;
    hipLaunchKernelGGL(zero_rows_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, y, rows,
                       width, stride);
    return hipGetLastError();
}

}  // namespace c3d
