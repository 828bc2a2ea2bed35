// Device helpers of the matrix-product kernels (linear.hip): operand tiles in
// LDS for both storage orders, their MFMA fragments, activations, and the
// epilogue.
#pragma once

#include "igemm_common.h"
#include "token_internal.h"

namespace c3d {

constexpr int kGemmBK = 64;                 // contraction per stage
constexpr int kGemmRow = kGemmBK * 2;       // bytes of one LDS row, contraction contiguous

// z -> act(z) and act'(z), fp32, two transcendental instructions each.
// GELU (erf form) as max(z, 0) - |z| Phi(-|z|); the tanh form as z * sigmoid(2u),
// u = sqrt(2 / pi) (z + 0.044715 z^3).
// Defined for every z: the kept z is rounded to 16 bits and a finite one of fp16's
// product may be infinite there.  act(+inf) = +inf, act(-inf) = 0, the slopes 1
// and 0; a NaN stays one.
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGeluA = 0.797884560802865356f, kGeluB = 0.044715f;

__device__ __forceinline__ float sigmoid_f(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * v));
}
// sigmoid(2u) of the tanh form: 1 / (1 + 2^(z (k + k B z^2)))
__device__ __forceinline__ float sigmoid_2u(float z) {
    constexpr float k = -2.0f * kLog2e * kGeluA;
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * fmaf(k * kGeluB, z * z, k)));
}
// Phi(-|z|) of the standard normal distribution; ex: exp(-z^2 / 2).  Phi(-z)
// exp(z^2 / 2) falls from 1/2 like 1 / (z sqrt(2 pi)), so it is fitted by a
// polynomial in t = 1 / (1 + 0.362 z): seven terms by least squares, reweighted
// towards the least relative error over 0 <= z <= 14, 8e-7 (1e-6 as evaluated in
// fp32).  The error is relative, so that z Phi(z) far below 0 keeps the digits of
// its type (a formula for erf of absolute error 1.5e-7 is off by half an fp16 ulp at
// z = -4 and by two bf16 ulps at -8).
__device__ __forceinline__ float normal_tail(float z, float &ex) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.362f, fabsf(z), 1.0f));
    ex = __builtin_amdgcn_exp2f(z * (-0.5f * kLog2e * z));
    float q = fmaf(t, 0.047938287f, -0.180009678f);
    q = fmaf(t, q, 0.176617280f);
    q = fmaf(t, q, 0.028831471f);
    q = fmaf(t, q, 0.139429703f);
    q = fmaf(t, q, 0.142689303f);
    q = fmaf(t, q, 0.144503906f);
    return q * t * ex;
}
// z bounded to +-1e4, where every activation has its limit's value to the last
// bit: the factor of a term that tends to 0 (which an infinite z would make NaN).
// The exponentials take z itself, so that a NaN comes through.
__device__ __forceinline__ float bounded(float z) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_fmed3f(z, -1e4f, 1e4f);
#else
    return z;
#endif
}
// z bounded below (and max(z, 0)) the same way: one v_med3 with an upper bound that
// the compiler cannot see is infinite (its own maximum first quiets z, one
// instruction more: 1% of a product with SiLU).
__device__ __forceinline__ float bounded_below(float z, float low) {
#if defined(__HIP_DEVICE_COMPILE__)
    float inf = __builtin_inff();
    asm("" : "+v"(inf));
    return __builtin_amdgcn_fmed3f(z, low, inf);
#else
    return z < low ? low : z;
#endif
}
template <int ACT>
__device__ __forceinline__ float act_f(float z) {
    if constexpr (ACT == CONV3D_ACT_SILU) return bounded_below(z, -1e4f) * sigmoid_f(z);
    if constexpr (ACT == CONV3D_ACT_GELU) {
        float ex;
        return fmaf(-fabsf(bounded(z)), normal_tail(z, ex), bounded_below(z, 0.0f));  // z Phi(z) for either sign
    }
    if constexpr (ACT == CONV3D_ACT_GELU_TANH) return bounded_below(z, -1e4f) * sigmoid_2u(z);
    return z;
}
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == CONV3D_ACT_NONE) return 1.0f;
    const float b = bounded(z);
    if constexpr (ACT == CONV3D_ACT_SILU) {
        const float s = sigmoid_f(z);
        return s * fmaf(b, 1.0f - s, 1.0f);
    }
    if constexpr (ACT == CONV3D_ACT_GELU) {
        float ex;
        const float tail = normal_tail(z, ex);
        return fmaf(b * 0.398942280401432678f, ex, z < 0.0f ? tail : 1.0f - tail);
    }
    const float s = sigmoid_2u(z);
    return s * fmaf(b * (1.0f - s), fmaf(6.0f * kGeluA * kGeluB * b, b, 2.0f * kGeluA), 1.0f);
}

// Calls f(std::integral_constant<int, ACT>) for the activation chosen at run time.
template <typename F>
__device__ __forceinline__ void act_switch(int act, F &&f) {
    switch (act) {
        case CONV3D_ACT_SILU: f(std::integral_constant<int, CONV3D_ACT_SILU>{}); break;
        case CONV3D_ACT_GELU: f(std::integral_constant<int, CONV3D_ACT_GELU>{}); break;
        case CONV3D_ACT_GELU_TANH: f(std::integral_constant<int, CONV3D_ACT_GELU_TANH>{}); break;
        default: f(std::integral_constant<int, CONV3D_ACT_NONE>{}); break;
    }
}

// ---- operand tiles in LDS.  An operand tile is ROWS output rows (or columns)
// x 64 of the contraction, ROWS x 128 bytes in either order (a whole cache line
// of every row per stage: with 32 of the contraction and half lines the forward
// product of 8192^3 ran at 1130 TFLOP/s, with whole ones at 1320 to 1410):
//   contraction contiguous (TR = false): ROWS rows of 128 bytes; 16-byte chunk
//     c of row r sits at chunk c ^ swz<64>(r);
//   transposed (TR = true): 64 rows (one per contraction index) of 2 ROWS
//     bytes; chunk c of row r sits at chunk c ^ tr_swz(r), so that the 4 rows x
//     64 bytes that a half-wave's transposing reads take fill all banks.
// Loads are 16 bytes per lane, 1 KiB per instruction, straight into LDS; the
// swizzle is applied to the global side.

// CH: 16-byte chunks of a row.  A row of 16 chunks spans all banks, one of 8
// half of them; rows that repeat the same banks exchange their 64-byte pieces.
template <int CH>
__device__ __forceinline__ int tr_swz(int row) {
    return CH >= 16 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
}

// One operand as a workgroup reads it: a moving buffer resource and the lane's
// offsets for its NI load instructions per stage.
template <bool TR, int ROWS, int NI>
struct Operand {
    const _Float16 *base;   // TR: the stage's first row, at the tile's columns; else the tile's first row
    int64_t stride;
    int left;               // contraction not yet loaded, from the current stage on
    int ncols;              // TR: columns of the tile inside the matrix
    uint32_t records, soff;
    uint32_t voff[NI];
    int kc[NI];             // !TR: the contraction index of the lane's chunk within the stage

    // instruction ids: first, first + step, ... (NI of them)
    __device__ __forceinline__ void init(const _Float16 *m, int64_t stride_, int row0, int rows_total, int k0, int kend,
                                         int first, int step, int lane) {
        stride = stride_;
        left = kend - k0;
        soff = 0;
        const int rows = rows_total - row0 < ROWS ? rows_total - row0 : ROWS;
        ncols = rows;
        if constexpr (TR) {
            base = m + (int64_t)k0 * stride + row0;
            constexpr unsigned CH = ROWS / 8;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const unsigned lin = (unsigned)((first + j * step) * 64 + lane);
                const int r = (int)(lin / CH), c = (int)(lin % CH) ^ tr_swz<(int)CH>(r);
                voff[j] = c * 8 < ncols ? (uint32_t)(r * (int)stride + c * 8) * 2u : kOOB;
                kc[j] = 0;
            }
        } else {
            base = m + (int64_t)row0 * stride + k0;
            records = (uint32_t)((rows - 1) * (int)stride + (left > 0 ? left : 0)) * 2u;
#pragma unroll
            for (int j = 0; j < NI; ++j) {
                const int lin = (first + j * step) * 64 + lane;
                const int r = lin >> 3, c = (lin & 7) ^ swz<kGemmBK>(r);
                kc[j] = c * 8;
                voff[j] = r < rows ? (uint32_t)(r * (int)stride + c * 8) * 2u : kOOB;
            }
        }
    }
    // The current stage into `lds` (the operand's stage buffer), then on by STEP
    // stages; the contraction past its end reads as zeros.
    template <int STEP>
    __device__ __forceinline__ void load(char *lds, int first, int step) {
        if constexpr (TR) {
            // past the end: no record, so every offset is out of range
            const int rows = left < kGemmBK ? left : kGemmBK;
            const int rec = ((rows - 1) * (int)stride + ncols) * 2;
            const buf_rsrc r = make_rsrc(base, (uint32_t)(rec < 0 || left <= 0 ? 0 : rec));
#pragma unroll
            for (int j = 0; j < NI; ++j) dma16(r, lds + (first + j * step) * 1024, voff[j], 0u);
            base += STEP * kGemmBK * stride;
        } else {
            const buf_rsrc r = make_rsrc(base, records);
#pragma unroll
            for (int j = 0; j < NI; ++j)
                dma16(r, lds + (first + j * step) * 1024, kc[j] < left ? voff[j] : kOOB, soff);
            soff += STEP * kGemmRow;
        }
        left -= STEP * kGemmBK;
    }
};

// The transposing LDS reads.  Within 16 lanes, lane j reads 8 bytes of row j / 4
// and lane i receives column i of those 4 rows; two reads, 4 rows apart, make
// one lane's 8 contraction values.  Written as assembly that waits for its own
// results: for the compiler's own form of the read it waits for every load into
// LDS still in flight, stages ahead included.  ROW: bytes of one LDS row; K0: the first row.
#define C3D_TR(d, a, o) "ds_read_b64_tr_b16 %" #d ", %" #a " offset:%" #o "\n\t"
template <int ROW, int K0>
__device__ __forceinline__ void tr_read2(const uint32_t (&a)[2], uint64_t (&v)[8]) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile(C3D_TR(0, 8, 10) C3D_TR(1, 8, 11) C3D_TR(2, 9, 10) C3D_TR(3, 9, 11) C3D_TR(4, 8, 12) C3D_TR(5, 8, 13)
                     C3D_TR(6, 9, 12) C3D_TR(7, 9, 13) "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]),
                   "=&v"(v[7])
                 : "v"(a[0]), "v"(a[1]), "n"(K0 * ROW), "n"((K0 + 4) * ROW), "n"((K0 + 16) * ROW), "n"((K0 + 20) * ROW)
                 : "memory");
#endif
}
template <int ROW, int K0>
__device__ __forceinline__ void tr_read1(const uint32_t (&a)[1], uint64_t (&v)[4]) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile(C3D_TR(0, 4, 5) C3D_TR(1, 4, 6) C3D_TR(2, 4, 7) C3D_TR(3, 4, 8) "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
                 : "v"(a[0]), "n"(K0 * ROW), "n"((K0 + 4) * ROW), "n"((K0 + 16) * ROW), "n"((K0 + 20) * ROW)
                 : "memory");
#endif
}
template <int ROW, int K0>
__device__ __forceinline__ void tr_read4(const uint32_t (&a)[4], uint64_t (&v)[16]) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile(C3D_TR(0, 16, 20) C3D_TR(1, 16, 21) C3D_TR(2, 17, 20) C3D_TR(3, 17, 21) C3D_TR(4, 18, 20)
                     C3D_TR(5, 18, 21) C3D_TR(6, 19, 20) C3D_TR(7, 19, 21) C3D_TR(8, 16, 22) C3D_TR(9, 16, 23)
                         C3D_TR(10, 17, 22) C3D_TR(11, 17, 23) C3D_TR(12, 18, 22) C3D_TR(13, 18, 23)
                             C3D_TR(14, 19, 22) C3D_TR(15, 19, 23) "s_waitcnt lgkmcnt(0)"
                 : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]),
                   "=&v"(v[7]), "=&v"(v[8]), "=&v"(v[9]), "=&v"(v[10]), "=&v"(v[11]), "=&v"(v[12]), "=&v"(v[13]),
                   "=&v"(v[14]), "=&v"(v[15])
                 : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(K0 * ROW), "n"((K0 + 4) * ROW),
                   "n"((K0 + 16) * ROW), "n"((K0 + 20) * ROW)
                 : "memory");
#endif
}
#undef C3D_TR

// Byte offsets of a lane's MFMA fragments within an operand's stage buffer.
// A fragment covers 32 output rows (from row0, a multiple of 32) x 16 of the
// contraction: lane l holds output row l % 32, contraction 8 (l / 32) .. + 7.
template <bool TR, int ROWS, int NF>
struct Fragments {
    uint32_t off[TR ? NF : 4];
    __device__ __forceinline__ void init(int row0, int lane) {
        if constexpr (TR) {
            const int j = lane & 15, g = (lane >> 4) & 1, r = (lane >> 5) * 8 + (j >> 2);
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const int chunk = ((row0 + i * 32 + 16 * g) >> 3) + ((j & 3) >> 1);
                off[i] = r * ROWS * 2 + ((chunk ^ tr_swz<ROWS / 8>(j >> 2)) << 4) + (j & 1) * 8;
            }
        } else {
            const int r = lane & 31, hi = lane >> 5;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) off[kk] = (row0 + r) * kGemmRow + (((2 * kk + hi) ^ swz<kGemmBK>(r)) * 16);
        }
    }
    // the fragments of k-steps KK0 and KK0 + 1 of a stage
    template <int KK0>
    __device__ __forceinline__ void read(const char *lds, half8_t (&f)[2][NF]) const {
        if constexpr (TR) {
            static_assert(NF == 1 || NF == 2 || NF == 4, "one assembly block per operand");
            const uint32_t base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)lds;
            uint32_t a[NF];
            uint64_t v[4 * NF];
#pragma unroll
            for (int i = 0; i < NF; ++i) a[i] = base + off[i];
            if constexpr (NF == 1)
                tr_read1<ROWS * 2, KK0 * 16>(a, v);
            else if constexpr (NF == 2)
                tr_read2<ROWS * 2, KK0 * 16>(a, v);
            else
                tr_read4<ROWS * 2, KK0 * 16>(a, v);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < NF; ++i)
                    f[kk][i] = __builtin_shufflevector(__builtin_bit_cast(half4_t, v[(kk * NF + i) * 2]),
                                                       __builtin_bit_cast(half4_t, v[(kk * NF + i) * 2 + 1]), 0, 1, 2,
                                                       3, 4, 5, 6, 7);
        } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < NF; ++i)
                    f[kk][i] = *reinterpret_cast<const half8_t *>(lds + off[KK0 + kk] + i * 32 * kGemmRow);
        }
    }
};

// 2-byte buffer load; out-of-range loads read zero.
__device__ __forceinline__ _Float16 load2(buf_rsrc r, uint32_t off) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_bit_cast(_Float16, __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0));
#else
    (void)r;
    (void)off;
    return (_Float16)0.0f;
#endif
}

// 16-byte buffer store; out-of-range stores are dropped.
__device__ __forceinline__ void gemm_store16(buf_rsrc r, uint32_t off, half8_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 0);
#else
    (void)r;
    (void)off;
    (void)v;
#endif
}

__device__ __forceinline__ void gemm_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
template <int N>
__device__ __forceinline__ void gemm_wait_loads() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// A 16-bit output tile in LDS, rows of BN elements: 16-byte chunk c of row v at
// chunk c ^ (v mod chunks), and rows with bit 4 set keep the two 8-byte halves
// of a chunk swapped, so that both the fragments' 8-byte accesses (32 rows at
// one chunk) and the rows' 16-byte accesses spread over all banks.
template <int BN>
__device__ __forceinline__ int tile_chunk(int v, int c) {
    return v * BN * 2 + ((c ^ (v & (BN / 8 - 1))) << 4);
}

// Tile rows between LDS and global memory in whole rows, 16 bytes per lane: a
// thread takes one chunk of every RP-th row.  Rows past the matrix lie past the
// records; a column past it is out of range itself.
template <int BM, int BN, int THREADS>
__device__ __forceinline__ void store_rows(const char *smem, _Float16 *out, int64_t stride, int rows, int cols) {
    constexpr int CH = BN / 8, RP = THREADS / CH;
    static_assert(RP % CH == 0, "a thread's rows share one swizzle");
    const buf_rsrc r = make_rsrc(out, (uint32_t)((rows - 1) * (int)stride + cols) * 2u);
    const int v0 = (int)threadIdx.x / CH, c = (int)threadIdx.x % CH;
    const uint32_t off = c * 8 < cols ? (uint32_t)(v0 * (int)stride + c * 8) * 2u : kOOB;
    const char *at = smem + tile_chunk<BN>(v0, c);
#pragma unroll
    for (int k = 0; k < BM / RP; ++k) {
        half8_t h = *reinterpret_cast<const half8_t *>(at + k * RP * BN * 2);
        if ((v0 + k * RP) & 16) h = __builtin_shufflevector(h, h, 4, 5, 6, 7, 0, 1, 2, 3);
        gemm_store16(r, off + (uint32_t)(k * RP * 2) * (uint32_t)stride, h);
    }
}
// The residual's rows into the same places.  The 8-byte halves are not swapped
// (they arrive as they are); the fragments read them so.
template <int BM, int BN, int THREADS>
__device__ __forceinline__ void load_rows(char *smem, const _Float16 *in, int64_t stride, int rows, int cols) {
    constexpr int CH = BN / 8, RP = THREADS / CH;
    const buf_rsrc r = make_rsrc(in, (uint32_t)((rows - 1) * (int)stride + cols) * 2u);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int v0 = (int)threadIdx.x / CH, c = ((int)threadIdx.x % CH) ^ (v0 & (CH - 1));
    const uint32_t off = c * 8 < cols ? (uint32_t)(v0 * (int)stride + c * 8) * 2u : kOOB;
#pragma unroll
    for (int k = 0; k < BM / RP; ++k)
        dma16(r, smem + (k * THREADS + wave * 64) * 16, off + (uint32_t)(k * RP * 2) * (uint32_t)stride, 0u);
}

// Epilogue of a whole tile: z = acc (the bias is in it), stored when asked
// for; y = act(z) + residual; each rounded once.  Staged through LDS so that it
// leaves in whole rows.  Lane's register 4g + e of fragment (i, j): column
// WN * wni + 32 i + 8 g + 4 (lane / 32) + e, row WM * wmi + 32 j + lane % 32.
// Every LDS buffer of the K loop is free, and every wave is past it.
template <typename E, int BM, int BN, int WM, int WN, int THREADS>
__device__ __forceinline__ void gemm_store_tile(const GemmParams &p, const f32x16 (&acc)[WN / 32][WM / 32], char *smem,
                                                int m0, int n0, int wmi, int wni, int lane) {
    constexpr int TN = WN / 32, TM = WM / 32;
    const int rows = p.M - m0 < BM ? p.M - m0 : BM, cols = p.N - n0 < BN ? p.N - n0 : BN;
    const int rrow = lane & 31, rhi = lane >> 5;
    auto stage = [&](auto actc, auto resc) {
        constexpr int ACT = decltype(actc)::value;
        constexpr bool RES = decltype(resc)::value;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int j = 0; j < TM; ++j) {
                    const int v = wmi * WM + j * 32 + rrow;
                    char *chunk = smem + tile_chunk<BN>(v, wni * (WN / 8) + i * 4 + g);
                    half4_t h;
                    if constexpr (RES) {
                        const half4_t r = *reinterpret_cast<const half4_t *>(chunk + rhi * 8);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            h[e] = from_f32<E>(act_f<ACT>(acc[i][j][4 * g + e]) + to_f32<E>(r[e]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = from_f32<E>(act_f<ACT>(acc[i][j][4 * g + e]));
                    }
                    *reinterpret_cast<half4_t *>(chunk + ((rhi ^ ((v >> 4) & 1)) << 3)) = h;
                }
        gemm_barrier();
    };
    if (p.z) {
        stage(std::integral_constant<int, CONV3D_ACT_NONE>{}, std::false_type{});
        store_rows<BM, BN, THREADS>(smem, p.z + (int64_t)m0 * p.N + n0, p.N, rows, cols);
        gemm_barrier();
    }
    if (p.res) {
        load_rows<BM, BN, THREADS>(smem, p.res + (int64_t)m0 * p.res_stride + n0, p.res_stride, rows, cols);
        gemm_wait_loads<0>();
        gemm_barrier();
        act_switch(p.act, [&](auto ac) { stage(ac, std::true_type{}); });
    } else {
        act_switch(p.act, [&](auto ac) { stage(ac, std::false_type{}); });
    }
    store_rows<BM, BN, THREADS>(smem, p.y + (int64_t)m0 * p.y_stride + n0, p.y_stride, rows, cols);
}

// The bias of a lane's columns: element 4g + e of [i] is column col0 + 32 i + 8 g + 4 (lane / 32) + e.
template <int TN>
__device__ __forceinline__ void gemm_load_bias(const GemmParams &p, half4_t (&b)[TN][4], bool bias, int col0,
                                               int lane) {
    const buf_rsrc rb = make_rsrc(bias ? p.bias : p.p, bias ? (uint32_t)p.N * 2u : 0u);
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int co = col0 + i * 32 + 8 * g + 4 * (lane >> 5);
            b[i][g] = load8(rb, bias && co < p.N ? (uint32_t)co * 2u : kOOB);
        }
}

// Epilogue of one wave's 64 x 128 part of a tile, through 8 KiB of LDS that no
// other wave touches (no barrier), 64 columns at a time: rows of 128 bytes,
// 16-byte chunk c of row v at chunk c ^ ((v >> 1) & 7), rows with bit 4 set
// with the 8-byte halves of a chunk swapped, so that both the fragments' 8-byte
// accesses (32 rows at one chunk) and the rows' 16-byte accesses spread over all
// banks.  It leaves in whole cache lines.  row0, col0: the wave's first row and
// column; rows, cols: how many of its 64 and 128 are inside the matrix (may be
// none).
template <typename E>
__device__ __forceinline__ void gemm_store_wave(const GemmParams &p, const f32x16 (&acc)[4][2], char *lds, int row0,
                                                int col0, int rows, int cols, int lane) {
    if (rows <= 0 || cols <= 0) return;
    const int rrow = lane & 31, rhi = lane >> 5;
    const int vr = lane >> 3, vc = lane & 7;  // row accesses: 8 rows of 8 chunks per instruction
    // Byte offset of the lane's chunk c in rows vr, vr + 8, ... of columns
    // [64 h, 64 h + 64): rows past the matrix lie past the records, a column past
    // it is out of range itself (and stays so with a multiple of the stride on top).
    auto first_off = [&](int c, int64_t stride, int h) {
        return h * 64 + c * 8 < cols ? (uint32_t)(vr * (int)stride + h * 64 + c * 8) * 2u : kOOB;
    };
    const int key = (vr >> 1) & 3;  // ((8 k + vr) >> 1) & 7 is key, with bit 2 set for odd k
    auto fragments = [&](auto actc, auto resc, int h) {
        constexpr int ACT = decltype(actc)::value;
        constexpr bool RES = decltype(resc)::value;
#pragma unroll
        for (int ii = 0; ii < 2; ++ii)
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int v = j * 32 + rrow, c = ii * 4 + g;
                    char *chunk = lds + v * 128 + ((c ^ ((v >> 1) & 7)) << 4);
                    half4_t r = {}, o;
                    if constexpr (RES) r = *reinterpret_cast<const half4_t *>(chunk + rhi * 8);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = h ? acc[2 + ii][j][4 * g + e] : acc[ii][j][4 * g + e];
                        o[e] = from_f32<E>(RES ? act_f<ACT>(z) + to_f32<E>(r[e]) : act_f<ACT>(z));
                    }
                    *reinterpret_cast<half4_t *>(chunk + ((rhi ^ ((v >> 4) & 1)) << 3)) = o;
                }
    };
    auto rows_out = [&](_Float16 *out, int64_t stride, int h) {
        const buf_rsrc r = make_rsrc(out, (uint32_t)((rows - 1) * (int)stride + cols) * 2u);
        const uint32_t off = first_off(vc, stride, h);
        const char *at[2] = {lds + vr * 128 + ((vc ^ key) << 4), lds + vr * 128 + ((vc ^ key ^ 4) << 4)};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            half8_t t = *reinterpret_cast<const half8_t *>(at[k & 1] + k * 1024);
            if (k & 2) t = __builtin_shufflevector(t, t, 4, 5, 6, 7, 0, 1, 2, 3);  // row & 16
            gemm_store16(r, off + (uint32_t)(k * 16) * (uint32_t)stride, t);
        }
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (p.z) {
            fragments(std::integral_constant<int, CONV3D_ACT_NONE>{}, std::false_type{}, h);
            rows_out(p.z + (int64_t)row0 * p.N + col0, p.N, h);
        }
        if (p.res) {
            const buf_rsrc r = make_rsrc(p.res + (int64_t)row0 * p.res_stride + col0,
                                         (uint32_t)((rows - 1) * (int)p.res_stride + cols) * 2u);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the rows before have left the LDS
            const uint32_t off[2] = {first_off(vc ^ key, p.res_stride, h), first_off(vc ^ key ^ 4, p.res_stride, h)};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                dma16(r, lds + k * 1024, off[k & 1] + (uint32_t)(k * 16) * (uint32_t)p.res_stride, 0u);
            gemm_wait_loads<0>();
            act_switch(p.act, [&](auto ac) { fragments(ac, std::true_type{}, h); });
        } else {
            act_switch(p.act, [&](auto ac) { fragments(ac, std::false_type{}, h); });
        }
        rows_out(p.y + (int64_t)row0 * p.y_stride + col0, p.y_stride, h);
    }
}

// The bias of a lane's columns as the accumulators' start value.
template <typename E, int WM, int WN>
__device__ __forceinline__ void gemm_init_acc(const GemmParams &p, f32x16 (&acc)[WN / 32][WM / 32], bool bias, int col0,
                                              int lane) {
    half4_t b[WN / 32][4];
    gemm_load_bias<WN / 32>(p, b, bias, col0, lane);
#pragma unroll
    for (int i = 0; i < WN / 32; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int j = 0; j < WM / 32; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][4 * g + e] = to_f32<E>(b[i][g][e]);
}

// A K-piece's fp32 partial tile, in fragment order.
template <int BM, int BN, int WM, int WN>
__device__ __forceinline__ void gemm_store_partial(const GemmParams &p, const f32x16 (&acc)[WN / 32][WM / 32], int slot,
                                                   int wave, int lane) {
    constexpr int TN = WN / 32, TM = WM / 32;
    f32x4 *pp = reinterpret_cast<f32x4 *>(p.partial + (size_t)slot * (BM * BN));
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
                pp[(((wave * TN + i) * TM + j) * 4 + g) * 64 + lane] = v;
            }
}

// Work unit u: a whole tile (slot < 0) or K-piece `slot` of a split tile, and
// its range of stages.  Tiles are walked in groups of kGemmGroup rows of tiles,
// down the rows first: the workgroups that an XCD runs at once (a contiguous
// range of units) then share both operands' tiles in its L2.  Pieces are walked
// range of the contraction by range, so that an XCD reads its ranges of both
// operands and not all of them.
constexpr int kGemmGroup = 4;
__device__ __forceinline__ void gemm_unit(const GemmParams &p, int u, int &m_tile, int &n_tile, int &it0, int &it1,
                                          int &slot) {
    it0 = 0;
    it1 = p.niter;
    slot = -1;
    int tile = u;
    if (u >= p.dp_tiles) {
        slot = u - p.dp_tiles;
        const int piece = slot / p.sk_tiles;
        tile = p.dp_tiles + slot % p.sk_tiles;
        it0 = (int)((int64_t)p.niter * piece / p.sk_pieces);
        it1 = (int)((int64_t)p.niter * (piece + 1) / p.sk_pieces);
    }
    const int per_group = kGemmGroup * p.n_tiles;
    const int g0 = tile / per_group * kGemmGroup;
    const int rows = p.m_tiles - g0 < kGemmGroup ? p.m_tiles - g0 : kGemmGroup;
    const int r = tile - g0 * p.n_tiles;
    m_tile = g0 + r % rows;
    n_tile = r / rows;
}

}  // namespace c3d
