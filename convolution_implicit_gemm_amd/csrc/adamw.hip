// The AdamW step over many tensors in one launch: each element's weight, gradient and
// states are read once and written once, in fp32 between.
#include <climits>

#include "elem16.h"
#include "token_internal.h"

namespace c3d {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// The largest of 16 adjacent lanes' values, to all of them.
__device__ __forceinline__ float max16(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto step = [&](auto ctrl) {
        const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false);
        v = fmaxf(v, __builtin_bit_cast(float, o));
    };
    step(std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
    step(std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
    step(std::integral_constant<int, 0x141>{});  // row_half_mirror
    step(std::integral_constant<int, 0x140>{});  // row_mirror
#endif
    return v;
}

__device__ __forceinline__ float power_of_two(int e) { return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23); }

// 8 codes -> values times `unit`
__device__ __forceinline__ void decode8(u32x2_t c, float unit, float (&x)[8]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], true);
        x[4 * w] = a[0] * unit;
        x[4 * w + 1] = a[1] * unit;
        x[4 * w + 2] = b[0] * unit;
        x[4 * w + 3] = b[1] * unit;
    }
#endif
}

// The block's power e: the least from -126 on with its largest finite value at most
// 448 * 2^e (448 = 7/8 * 2^9, the largest e4m3 number).  The block is 16 lanes' 8 values.
__device__ __forceinline__ int block_power(const float (&x)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = fabsf(x[i]);
        top = fmaxf(top, a < __builtin_inff() ? a : 0.0f);
    }
    top = max16(top);
    const uint32_t bits = __builtin_bit_cast(uint32_t, top);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);  // 1.75 * 2^8 = 448
    return e < -126 ? -126 : e;
}
template <bool ROOT>
__device__ __forceinline__ u32x2_t encode8(const float (&x)[8], int e) {
    u32x2_t c = {};
#if defined(__HIP_DEVICE_COMPILE__)
    const float inv = power_of_two(-e);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = x[i] * inv;
        if (ROOT) y[i] = x[i] > 0.0f ? fmaxf(y[i], 0x1p-9f) : y[i];  // the least code but 0
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w], y[4 * w + 1], 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w + 2], y[4 * w + 3], v, true);
        c[w] = (uint32_t)v;
    }
#endif
    return c;
}

// 8 elements, or the `left` first of them, as vectors or one by one.
template <typename T>
__device__ __forceinline__ void load_f32(const T *p, int left, float (&x)[8]) {
    if (left >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t *>(p + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * h + i] = v[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < left ? p[i] : 0.0f;
    }
}
__device__ __forceinline__ void store_f32(float *p, int left, const float (&x)[8]) {
    if (left >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<f32x4_t *>(p + 4 * h) = f32x4_t{x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = x[i];
    }
}
template <typename E>
__device__ __forceinline__ void load_16(const _Float16 *p, int left, float (&x)[8]) {
    if (left >= 8) {
        const e16x8_t v = *reinterpret_cast<const e16x8_t *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32<E>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < left ? to_f32<E>(p[i]) : 0.0f;
    }
}
template <typename E>
__device__ __forceinline__ void store_16(_Float16 *p, int left, const float (&x)[8]) {
    if (left >= 8) {
        e16x8_t v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = from_f32<E>(x[i]);
        *reinterpret_cast<e16x8_t *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) p[i] = from_f32<E>(x[i]);
    }
}
__device__ __forceinline__ u32x2_t load_codes(const uint8_t *p, int left) {
    if (left >= 8) return *reinterpret_cast<const u32x2_t *>(p);
    u32x2_t c = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) c[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return c;
}
__device__ __forceinline__ void store_codes(uint8_t *p, int left, u32x2_t c) {
    if (left >= 8) {
        *reinterpret_cast<u32x2_t *>(p) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
}

// A lane takes 8 elements at a time, 16 lanes a block of 128, whose scale they find by
// themselves; a workgroup p.units times 2048 elements of one tensor.
template <typename E, bool STATE8, bool GRAD32>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwParams p) {
    const int lane = threadIdx.x & 63;
    // the tensor: the last one whose first workgroup is not behind this one
    const int mine = lane < kAdamwTensors ? p.first[lane] : INT_MAX;
    const int at = __popcll(__builtin_amdgcn_ballot_w64(mine <= (int)blockIdx.x)) - 1;
    const AdamwTensor &t = p.t[__builtin_amdgcn_readfirstlane(at)];
    const AdamwHyper h = p.device_hyper ? *p.device_hyper : p.hyper;
    const float keep = 1.0f - h.lr_decay * t.decay;
    const int64_t first = (int64_t)((int)blockIdx.x - p.first[__builtin_amdgcn_readfirstlane(at)]) * p.units * kAdamwUnit;
    for (int u = 0; u < p.units; ++u) {
        const int64_t base = first + (int64_t)u * kAdamwUnit + threadIdx.x * 8;
        if (first + (int64_t)u * kAdamwUnit >= t.count) break;
        const int64_t rest = t.count - base;
        const int left = rest <= 0 ? 0 : rest < 8 ? (int)rest : 8;
        float g[8], m[8], v[8], w[8];
        const int64_t block = base / kAdamwBlock;
        const bool scaled = left > 0;
        if (GRAD32)
            load_f32(static_cast<const float *>(t.grad) + base, left, g);
        else
            load_16<E>(static_cast<const _Float16 *>(t.grad) + base, left, g);
        if (t.master)
            load_f32(t.master + base, left, w);
        else
            load_16<E>(t.param + base, left, w);
        if constexpr (STATE8) {
            const u32x2_t cm = load_codes(static_cast<const uint8_t *>(t.m) + base, left);
            const u32x2_t cv = load_codes(static_cast<const uint8_t *>(t.v) + base, left);
            const int em = scaled ? t.m_scale[block] : 0, ev = scaled ? t.v_scale[block] : 0;
            decode8(cm, ldexpf(1.0f, em - 127), m);
            decode8(cv, ldexpf(1.0f, ev - 127), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= v[i];
        } else {
            load_f32(static_cast<const float *>(t.m) + base, left, m);
            load_f32(static_cast<const float *>(t.v) + base, left, v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = g[i] * h.grad_scale;
            m[i] = fmaf(m[i], h.beta1, x * h.rest1);
            v[i] = fmaf(v[i], h.beta2, x * x * h.rest2);
            const float root = sqrtf(v[i]);
            w[i] = fmaf(w[i], keep, -h.lr1 * (m[i] / fmaf(root, h.root2, h.eps)));
            if (STATE8) v[i] = root;
        }
        if (t.master) store_f32(t.master + base, left, w);
        if (t.param) store_16<E>(t.param + base, left, w);
        if constexpr (STATE8) {
            const int em = block_power(m), ev = block_power(v);
            store_codes(static_cast<uint8_t *>(t.m) + base, left, encode8<false>(m, em));
            store_codes(static_cast<uint8_t *>(t.v) + base, left, encode8<true>(v, ev));
            if (scaled && (threadIdx.x & 15) == 0) {
                t.m_scale[block] = (uint8_t)(em + 127);
                t.v_scale[block] = (uint8_t)(ev + 127);
            }
        } else {
            store_f32(static_cast<float *>(t.m) + base, left, m);
            store_f32(static_cast<float *>(t.v) + base, left, v);
        }
    }
}

template <typename E>
static void launch(const AdamwParams &p, int64_t blocks, bool state8, bool grad32, hipStream_t s) {
    const dim3 g((uint32_t)blocks), b(256);
    if (state8 && grad32)
        adamw_kernel<E, true, true><<<g, b, 0, s>>>(p);
    else if (state8)
        adamw_kernel<E, true, false><<<g, b, 0, s>>>(p);
    else if (grad32)
        adamw_kernel<E, false, true><<<g, b, 0, s>>>(p);
    else
        adamw_kernel<E, false, false><<<g, b, 0, s>>>(p);
}

hipError_t launch_adamw(const AdamwParams &p, int64_t blocks, bool bf16, bool state8, bool grad32, hipStream_t s) {
    if (bf16)
        launch<__bf16>(p, blocks, state8, grad32, s);
    else
        launch<_Float16>(p, blocks, state8, grad32, s);
    return hipGetLastError();
}

}  // namespace c3d
