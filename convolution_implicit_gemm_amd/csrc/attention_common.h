// Device helpers of the attention kernels (attention.hip, attention_grad.hip):
// which keys a query sees, tiles of rows in LDS and their MFMA fragments, and
// exchanges between the halves of a wave.
#pragma once

#include "igemm_common.h"
#include "token_internal.h"

namespace c3d {

// ---- rows.  The query heads that share a key head are rows of one problem:
// row r of a (sample, key head) is query token r / group, query head r % group of
// the key head's group.  Keys and values are then read once for all of them.

// What a sample has and where its queries stand.
struct AttnSample {
    int queries, keys;  // of this sample
    int64_t offset;     // position of query 0
};
__device__ __forceinline__ AttnSample attn_sample(const AttnParams &p, int b) {
    AttnSample s{p.tq, p.tk, p.q_offset};
    if (p.lengths) {
        const int ql = p.lengths[2 * b], kl = p.lengths[2 * b + 1];
        s.queries = ql < 0 ? 0 : ql < p.tq ? ql : p.tq;
        s.keys = kl < 0 ? 0 : kl < p.tk ? kl : p.tk;
    }
    if (p.tail) s.offset += s.keys - s.queries;
    return s;
}

// The keys [lo, hi) that query token i sees (lo <= hi): those up to the end of its own
// frame, from `window` frames back.  Both ends grow with i.  Positions are below
// 2^32 (the host checks).
struct AttnRange {
    int lo, hi;
};
__device__ __forceinline__ AttnRange attn_range(const AttnParams &p, const AttnSample &s, int i) {
    if (!p.frame) return {0, s.keys};
    const int64_t pos = s.offset + i;
    if (pos < 0) return {0, 0};
    const uint32_t f = (uint32_t)pos / (uint32_t)p.frame;
    const uint64_t end = ((uint64_t)f + 1) * (uint32_t)p.frame;
    const int hi = end < (uint64_t)s.keys ? (int)end : s.keys;
    int lo = 0;
    if (p.window && (uint64_t)f + 1 > (uint32_t)p.window) {
        const uint64_t from = ((uint64_t)f + 1 - (uint32_t)p.window) * (uint32_t)p.frame;
        lo = from < (uint64_t)s.keys ? (int)from : s.keys;
    }
    return {lo, hi};
}

// The other way round: the query tokens [lo, hi) that see a key of the sample.
__device__ __forceinline__ AttnRange attn_seen_by(const AttnParams &p, const AttnSample &s, int key) {
    if (!p.frame) return {0, s.queries};
    const int64_t f = (uint32_t)key / (uint32_t)p.frame, q = s.queries;
    const int64_t from = f * p.frame - s.offset;
    const int64_t to = p.window ? (f + p.window) * p.frame - s.offset : q;
    const int lo = (int)(from < 0 ? 0 : from < q ? from : q), hi = (int)(to < 0 ? 0 : to < q ? to : q);
    return {lo, hi < lo ? lo : hi};
}

// ---- tiles in LDS: rows of DP elements (the head's, then zeros), 2 DP bytes.
// 16-byte chunk c of row r sits at chunk c ^ attn_swz(r): the 16 rows that a read of
// one chunk touches at a time, and the 4 rows x 64 bytes of a transposing read, each
// lie in different banks (16 chunks fill all of them once).
template <int DP>
__device__ __forceinline__ int attn_swz(int r) {
    static_assert(DP == 32 || DP == 64 || DP == 96 || DP == 128, "padded head sizes");
    if constexpr (DP == 128) return (r & 3) << 2 | ((r >> 2) & 3);
    if constexpr (DP == 64) return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
    return (r >> 2) & 3;
}

// The lane as the compiler cannot see through it: what is worked out of it is worked out where it
// is used, and not kept in registers across a kernel's loop.
__device__ __forceinline__ int opaque(int v) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(v));
#endif
    return v;
}

// Rows of a tensor straight into LDS tiles of ROWS rows, by WAVES waves.  LEAN: one offset
// for all of a lane's loads, each with a resource of its own (a dozen scalar instructions), where
// the rows between them swizzle alike: for kernels short of registers.
template <int DP, int ROWS, int WAVES, bool LEAN = false>
struct AttnTile {
    static constexpr int CH = DP / 8, LOADS = ROWS * CH / 64, NI = (LOADS + WAVES - 1) / WAVES;
    static constexpr int STEP = WAVES * 64 / CH;  // rows from one of a lane's loads to the next
    static constexpr bool ONE = LEAN && WAVES * 64 % CH == 0 && STEP % 16 == 0;
    const _Float16 *base;  // row 0
    int64_t stride;
    int rows, dim;
    uint32_t voff[ONE ? 1 : NI];

    __device__ __forceinline__ AttnTile(const _Float16 *base_, int64_t stride_, int rows_, int dim_, int wave, int lane)
        : base(base_), stride(stride_), rows(rows_), dim(dim_) {
#pragma unroll
        for (int j = 0; j < (ONE ? 1 : NI); ++j) {
            const int lin = (wave + j * WAVES) * 64 + lane;
            const int r = lin / CH, c = (lin % CH) ^ attn_swz<DP>(r);
            voff[j] = c * 8 < dim ? (uint32_t)(r * (int)stride + c * 8) * 2u : kOOB;
        }
    }
    // rows [row0, row0 + ROWS) into lds; those past the end, and elements past the head, as zeros
    __device__ __forceinline__ void load(char *lds, int row0, int wave) const {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int first = row0 + (ONE ? j * STEP : 0), most = ONE && STEP < ROWS ? STEP : ROWS;
            const int left = rows - first, n = left < most ? left : most;
            const buf_rsrc rs = make_rsrc(base + first * stride, n > 0 ? (uint32_t)((n - 1) * (int)stride + dim) * 2u : 0u);
            if (LOADS % WAVES == 0 || wave + j * WAVES < LOADS)
                dma16(rs, lds + (wave + j * WAVES) * 1024, voff[ONE ? 0 : j], 0u);
        }
    }
};

__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p;
}

// The MFMA fragment of 32 rows x 16 elements, contraction along the row: lane l
// holds row l % 32, elements 16 kk + 8 (l / 32) .. + 7.
template <int DP>
struct AttnRows {
    // chunk bits that the swizzle changes: the others are added
    static constexpr int XOR = DP == 128 ? 7 : DP == 64 ? 3 : 1;
    uint32_t off;  // of kk = 0
    __device__ __forceinline__ void init(int lane) {
        const int r = lane & 31;
        off = r * DP * 2 + (((lane >> 5) ^ attn_swz<DP>(r)) << 4);
    }
    // tile + off of a tile (which lies on 256 bytes), and row0 of its rows
    static __device__ __forceinline__ half8_t read(uint32_t at, int row0, int kk) {
#if defined(__HIP_DEVICE_COMPILE__)
        typedef const __attribute__((address_space(3))) half8_t lds_half8;
        return *(lds_half8 *)((at ^ ((kk & XOR) << 5)) + (uint32_t)((kk & ~XOR) * 32 + row0 * DP * 2));
#else
        return half8_t{};
#endif
    }
};

// Fragments with the rows as contraction: lane l holds column (element) l % 32 of
// each group of 32, and of the 16 rows of a step rows 4 h .. + 3 and 8 + 4 h .. + 3,
// h = l / 32: the order in which a 32 x 32 accumulator holds its rows, so that
// probabilities go from one MFMA's result into the next one's operand in place.
// ds_read_b64_tr_b16: within 16 lanes, lane j gives the address of 8 bytes of row
// j / 4 and lane i receives column i of the 4 rows.  In assembly that waits for itself:
// for the compiler's own form it would wait for every load into LDS still in flight.
#define C3D_TR(d, a, o) "ds_read_b64_tr_b16 %" #d ", %" #a " offset:%" #o "\n\t"
template <int DP>
struct AttnCols {
    static constexpr int NT = DP / 32, ROW = DP * 2;
    static constexpr bool XOR = DP == 128 || DP == 64;  // the column group's bits are swizzled
    uint32_t off0, off1;  // rows 4 h .. and 8 + 4 h .. of a step, column group 0
    __device__ __forceinline__ void init(int lane) {
        const int j = lane & 15, g = (lane >> 4) & 1, h = lane >> 5;
        const int r0 = 4 * h + (j >> 2), r1 = r0 + 8, c = 2 * g + ((j & 3) >> 1);
        off0 = r0 * ROW + ((c ^ attn_swz<DP>(r0)) << 4) + (j & 1) * 8;
        off1 = r1 * ROW + ((c ^ attn_swz<DP>(r1)) << 4) + (j & 1) * 8;
    }
    static __device__ __forceinline__ uint32_t group(uint32_t at, int t) { return XOR ? at ^ (t << 6) : at + (t << 6); }
    // One fragment in the compiler's own form, which it moves and waits for by itself (and for the wave's
    // loads into LDS too: the caller sees to it that they have had their time).  b0, b1: the
    // tile's address + off0, off1.
    template <int S>
    static __device__ __forceinline__ half8_t fragment(uint32_t b0, uint32_t b1, int t) {
#if defined(__HIP_DEVICE_COMPILE__)
        typedef __fp16 v4 __attribute__((__vector_size__(8)));
        typedef __attribute__((address_space(3))) v4 lds_v4;
        const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_v4 *)(group(b0, t) + S * 16 * ROW));
        const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_v4 *)(group(b1, t) + S * 16 * ROW));
        return __builtin_shufflevector(__builtin_bit_cast(half4_t, lo), __builtin_bit_cast(half4_t, hi), 0, 1, 2, 3, 4, 5,
                                       6, 7);
#else
        return half8_t{};
#endif
    }
    // the fragments of rows [16 S, 16 S + 16) of the tile
    template <int S>
    __device__ __forceinline__ void read(const char *tile, half8_t (&f)[NT]) const {
#if defined(__HIP_DEVICE_COMPILE__)
        const uint32_t b0 = lds_address(tile) + off0, b1 = lds_address(tile) + off1;
        uint64_t lo[NT], hi[NT];
        if constexpr (NT == 4) {
            asm volatile(C3D_TR(0, 8, 16) C3D_TR(4, 12, 16) C3D_TR(1, 9, 16) C3D_TR(5, 13, 16) C3D_TR(2, 10, 16)
                             C3D_TR(6, 14, 16) C3D_TR(3, 11, 16) C3D_TR(7, 15, 16) "s_waitcnt lgkmcnt(0)"
                         : "=&v"(lo[0]), "=&v"(lo[1]), "=&v"(lo[2]), "=&v"(lo[3]), "=&v"(hi[0]), "=&v"(hi[1]), "=&v"(hi[2]),
                           "=&v"(hi[3])
                         : "v"(group(b0, 0)), "v"(group(b0, 1)), "v"(group(b0, 2)), "v"(group(b0, 3)), "v"(group(b1, 0)),
                           "v"(group(b1, 1)), "v"(group(b1, 2)), "v"(group(b1, 3)), "n"(S * 16 * ROW)
                         : "memory");
        } else if constexpr (NT == 3) {
            asm volatile(C3D_TR(0, 6, 12) C3D_TR(3, 9, 12) C3D_TR(1, 7, 12) C3D_TR(4, 10, 12) C3D_TR(2, 8, 12)
                             C3D_TR(5, 11, 12) "s_waitcnt lgkmcnt(0)"
                         : "=&v"(lo[0]), "=&v"(lo[1]), "=&v"(lo[2]), "=&v"(hi[0]), "=&v"(hi[1]), "=&v"(hi[2])
                         : "v"(group(b0, 0)), "v"(group(b0, 1)), "v"(group(b0, 2)), "v"(group(b1, 0)), "v"(group(b1, 1)),
                           "v"(group(b1, 2)), "n"(S * 16 * ROW)
                         : "memory");
        } else if constexpr (NT == 2) {
            asm volatile(C3D_TR(0, 4, 8) C3D_TR(2, 6, 8) C3D_TR(1, 5, 8) C3D_TR(3, 7, 8) "s_waitcnt lgkmcnt(0)"
                         : "=&v"(lo[0]), "=&v"(lo[1]), "=&v"(hi[0]), "=&v"(hi[1])
                         : "v"(group(b0, 0)), "v"(group(b0, 1)), "v"(group(b1, 0)), "v"(group(b1, 1)), "n"(S * 16 * ROW)
                         : "memory");
        } else {
            asm volatile(C3D_TR(0, 2, 4) C3D_TR(1, 3, 4) "s_waitcnt lgkmcnt(0)"
                         : "=&v"(lo[0]), "=&v"(hi[0])
                         : "v"(b0), "v"(b1), "n"(S * 16 * ROW)
                         : "memory");
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
            f[t] = __builtin_shufflevector(__builtin_bit_cast(half4_t, lo[t]), __builtin_bit_cast(half4_t, hi[t]), 0, 1,
                                           2, 3, 4, 5, 6, 7);
#endif
    }
};
#undef C3D_TR

// The values that lanes l % 32 and l % 32 + 32 hold, to both.
struct Halves {
    float low, high;
    __device__ __forceinline__ explicit Halves(float v) : low(v), high(v) {
#if defined(__HIP_DEVICE_COMPILE__)
        uint32_t a = __builtin_bit_cast(uint32_t, v), b = a;
        asm("" : "+v"(b));  // a swap of one value with itself: the compiler takes both results for the same
        const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        low = __builtin_bit_cast(float, (uint32_t)r[0]);
        high = __builtin_bit_cast(float, (uint32_t)r[1]);
#endif
    }
};
// fp16 has 5 bits of exponent: in the gradients, probabilities (at most 1, 5e-5 in even rows of 20000
// keys) are 2^15 times as large as operands, so that they stay normal numbers, and what is
// summed of them is divided by that at the end.  (The forward pass knows no lse yet and lifts by less:
// see kAttnLift.)
template <typename E>
constexpr float kLift = std::is_same_v<E, __bf16> ? 0.0f : 15.0f;
template <typename E>
constexpr float kDrop = std::is_same_v<E, __bf16> ? 1.0f : 0x1p-15f;

template <int NT>
__device__ __forceinline__ void acc_scale(f32x16 (&acc)[NT], float f) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[t][e] *= f;
}

// dS = P (dP - delta) is as large as the gradients make it.  Lifted with P it may not fit fp16: then
// its column (a query in dq, a key in dk: one per lane, sums and all) is scaled down by a power
// of two, for good.  bf16 has fp32's exponents and needs none of this.
template <typename E>
struct ColumnScale {
    float f = 1.0f;
    // the column's 16 new values here and its 16 in the other half of the wave, and its sums so far
    template <int NT>
    __device__ __forceinline__ void apply(f32x16 &x, f32x16 (&acc)[NT]) {
#if defined(__HIP_DEVICE_COMPILE__)
        if constexpr (!std::is_same_v<E, __bf16>) {
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
            if (__builtin_amdgcn_ballot_w64(top * f > 32768.0f)) {
                const Halves h(top);
                const float most = fmaxf(h.low, h.high);
                // the power of two that brings the largest value to 2^13 .. 2^14
                const int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23) - 127;
                const float to = __builtin_bit_cast(float, (uint32_t)(13 - e + 127) << 23);
                const float now = most * f > 32768.0f ? to : f, by = now / f;
                f = now;
                acc_scale<NT>(acc, by);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= f;
        }
#endif
    }
};

// Row (of a 32 x 32 accumulator) that register i of a lane in half h holds.
__device__ __forceinline__ constexpr int acc_row(int i, int h) { return (i & 3) + 8 * (i >> 2) + 4 * h; }

__device__ __forceinline__ float both_max(float v) {
    const Halves x(v);
    return fmaxf(x.low, x.high);
}
__device__ __forceinline__ float both_sum(float v) {
    const Halves x(v);
    return x.low + x.high;
}

// One wave's accumulators to another one that holds the same rows and columns, through LDS:
// 16 bytes per lane at a time, lane by lane.
template <int NT>
__device__ __forceinline__ void acc_put(float *to, const f32x16 (&acc)[NT], int lane) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<f32x4 *>(to + ((t * 4 + (e >> 2)) * 64 + lane) * 4) =
                f32x4{acc[t][e], acc[t][e + 1], acc[t][e + 2], acc[t][e + 3]};
}
// acc = acc * own + other * f
template <int NT>
__device__ __forceinline__ void acc_join(const float *from, f32x16 (&acc)[NT], float own, float f, int lane) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const f32x4 o = *reinterpret_cast<const f32x4 *>(from + ((t * 4 + (e >> 2)) * 64 + lane) * 4);
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[t][e + m] = fmaf(acc[t][e + m], own, o[m] * f);
        }
}

// Eight consecutive accumulator registers as an operand's fragment.
template <typename E>
__device__ __forceinline__ half8_t pack8(const f32x16 &v, int first) {
    half8_t f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = from_f32<E>(v[first + e]);
    return f;
}

// A column of an accumulator (32 elements of one output row, times `mul`) to
// memory: lane l holds row l % 32's elements acc_row(i, l / 32); the halves swap so
// that each writes 16 bytes at a time.  out: the row's element 0 of this tile; left: elements
// of the head from there on.
template <typename E>
__device__ __forceinline__ void store_column(_Float16 *out, const f32x16 &v, float mul, int left, int lane, bool on) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int h = lane >> 5;
#pragma unroll
    for (int g = 0; g < 4; g += 2) {  // elements 8 g .. 8 g + 15
        uint32_t w[2][2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                h2 t;
                t[0] = from_f32<E>(v[4 * (g + q) + 2 * x] * mul);
                t[1] = from_f32<E>(v[4 * (g + q) + 2 * x + 1] * mul);
                w[q][x] = __builtin_bit_cast(uint32_t, t);
            }
        // half 0 takes elements 8 g .. + 7 (its own first four, the other's), half 1 the next eight
        const auto r0 = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
        const auto r1 = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
        typedef uint32_t u4 __attribute__((ext_vector_type(4)));
        const u4 q = {r0[0], r1[0], r0[1], r1[1]};
        const int e0 = 8 * (g + h);
        if (on && e0 < left) *reinterpret_cast<u4 *>(out + e0) = q;
    }
#endif
}

}  // namespace c3d
