// The AdamW step over many tensors in one launch: each element's weight, gradient and
// states are read once and written once, in fp32 between.
#include <climits>

#include "elem16.h"
#include "token_internal.h"

namespace c3d {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// The largest of the values of lanes 32 h .. 32 h + 31, to all of them.
__device__ __forceinline__ float max32(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto step = [&](auto ctrl) {
        const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false);
        v = fmaxf(v, __builtin_bit_cast(float, o));
    };
    step(std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
    step(std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
    step(std::integral_constant<int, 0x141>{});  // row_half_mirror
    step(std::integral_constant<int, 0x140>{});  // row_mirror
    uint32_t x = __builtin_bit_cast(uint32_t, v), y = x;
    asm("" : "+v"(y));  // a swap of one value with itself: the compiler takes both results for the same
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    v = fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
#endif
    return v;
}

// 4 codes -> values times `unit`
__device__ __forceinline__ void decode4(uint32_t c, float unit, float (&x)[4]) {
#if defined(__HIP_DEVICE_COMPILE__)
    const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
    x[0] = a[0] * unit;
    x[1] = a[1] * unit;
    x[2] = b[0] * unit;
    x[3] = b[1] * unit;
#endif
}

// The block's power e: the least from -126 on with its largest finite value at most
// 448 * 2^e (448 = 7/8 * 2^9, the largest e4m3 number).  The block is 32 lanes' 4 values.
__device__ __forceinline__ int block_power(const float (&x)[4]) {
    float top = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    if (!(top < __builtin_inff())) {  // rare: infinities, and NaN in all four
        top = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fabsf(x[i]) < __builtin_inff() ? fmaxf(top, fabsf(x[i])) : top;
    }
    const uint32_t bits = __builtin_bit_cast(uint32_t, max32(top));
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);  // 1.75 * 2^8 = 448
    return e < -126 ? -126 : e;
}
// 2^-e of N blocks to a half wave, whose lanes all hold them: the first wave of the workgroup works
// out those of all.  By powf, as a program that scales its states elementwise (ldexp of a tensor
// is a product with its powf) takes it: powf is half an ulp off for a sixth of the powers, which decides
// where values go that lie exactly on the border between two codes, both equally near, and with gradients of
// 8 bits and betas of few digits one in 250 does.  Codes are then that program's to the bit, and weights
// follow its weights; with 2^-e exact, one code in 250 is the other neighbour, and its weight a step later off by up to a
// tenth of a step.  The price is time: 61 tensors of 14 million 39.8 us (2^-e exact: 35.2), 201 million weights 542 (534).
// Against the definition in 64 bits neither is ahead by much: 1.28% of m's codes are the other neighbour (exact 1.16%), most
// of them from the rounding of beta m + (1 - beta) g itself.
template <int N>
__device__ __forceinline__ void inverse_powers(const int (&e)[N], float (&inv)[N]) {
    static_assert(8 * N <= 64, "one wave for all");
    __shared__ int powers[8 * N];
    __shared__ float inverses[8 * N];
    const auto meet = [] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    const int half = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) powers[half * N + k] = e[k];
    }
    meet();
    if (threadIdx.x < 8 * N) {
        float two = 2.0f;
#if defined(__HIP_DEVICE_COMPILE__)
        asm("" : "+v"(two));
#endif
        inverses[threadIdx.x] = powf(two, (float)-powers[threadIdx.x]);
    }
    meet();
#pragma unroll
    for (int k = 0; k < N; ++k) inv[k] = inverses[half * N + k];
}
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], float inv) {
#if defined(__HIP_DEVICE_COMPILE__)
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, v, true);
    uint32_t c = (uint32_t)v;
    if (ROOT && ((c - 0x01010101u) & ~c & 0x80808080u)) {  // a byte of 0: the least code but 0 for what is not 0
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(c >> (8 * i) & 0xffu) && x[i] > 0.0f) c |= 1u << (8 * i);
    }
    return c;
#else
    return 0;
#endif
}

// FAR: past the caches, for steps whose tensors would only push each other out.
template <bool FAR, typename T>
__device__ __forceinline__ T load_of(const void *p) {
    if constexpr (FAR)
        return __builtin_nontemporal_load(static_cast<const T *>(p));
    else
        return *static_cast<const T *>(p);
}
template <bool FAR, typename T>
__device__ __forceinline__ void store_to(void *p, T v) {
    if constexpr (FAR)
        __builtin_nontemporal_store(v, static_cast<T *>(p));
    else
        *static_cast<T *>(p) = v;
}

// 4 elements, or the `left` first of them, as vectors or one by one.
template <bool FAR>
__device__ __forceinline__ void load_f32(const float *p, int left, float (&x)[4]) {
    if (left >= 4) {
        const f32x4_t v = load_of<FAR, f32x4_t>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i < left ? p[i] : 0.0f;
    }
}
template <bool FAR>
__device__ __forceinline__ void store_f32(float *p, int left, const float (&x)[4]) {
    if (left >= 4) {
        store_to<FAR>(p, f32x4_t{x[0], x[1], x[2], x[3]});
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = x[i];
    }
}
template <typename E, bool FAR>
__device__ __forceinline__ void load_16(const _Float16 *p, int left, float (&x)[4]) {
    if (left >= 4) {
        const e16x4_t v = load_of<FAR, e16x4_t>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = to_f32<E>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i < left ? to_f32<E>(p[i]) : 0.0f;
    }
}
template <typename E, bool FAR>
__device__ __forceinline__ void store_16(_Float16 *p, int left, const float (&x)[4]) {
    if (left >= 4) {
        e16x4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = from_f32<E>(x[i]);
        store_to<FAR>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = from_f32<E>(x[i]);
    }
}
template <bool FAR>
__device__ __forceinline__ uint32_t load_codes(const uint8_t *p, int left) {
    if (left >= 4) return load_of<FAR, uint32_t>(p);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) c |= (uint32_t)p[i] << (8 * i);
    return c;
}
template <bool FAR>
__device__ __forceinline__ void store_codes(uint8_t *p, int left, uint32_t c) {
    if (left >= 4) {
        store_to<FAR>(p, c);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = (uint8_t)(c >> (8 * i));
}

// m and v as the formulas read, each product and sum rounded by itself, and v's root to the nearest: a
// program that evaluates them in fp32 gets the same bits, so that 8-bit codes next to a border between
// two of them do not differ between the two (contracted, one in 10^6 did, and their weights by
// up to a step's size one step later).
__device__ __forceinline__ void new_states(const AdamwHyper &h, float x, float &m, float &v, float &root) {
#pragma clang fp contract(off)
    m = m * h.beta1 + x * h.rest1;
    v = v * h.beta2 + (x * x) * h.rest2;
    root = sqrtf(v);
}

// A lane takes 4 adjacent elements at a time (one access of up to 16 bytes to each array, whole
// lines of it to a wave), half a wave a block of 128, whose largest value it finds by itself; a
// workgroup adamw_unit() adjacent elements of one tensor, all of them on their way at once, so that
// workgroups that run together read and write adjacent memory: 201 million weights, 8-bit
// states 537-542 us, 6.0 TB/s, bound by memory (with 24 times the elements to a workgroup, one after the
// other, a fifth more); fp32 states 1024-1031 us, 5.5 TB/s.
template <typename E, bool STATE8, bool GRAD32, bool FAR>
__global__ __launch_bounds__(256) void adamw_kernel(AdamwParams p) {
    constexpr int PARTS = adamw_unit(FAR) / 1024;
    const int lane = threadIdx.x & 63;
    // the tensor: the last one whose first workgroup is not behind this one
    const int mine = lane < kAdamwTensors ? p.first[lane] : INT_MAX;
    const int at = __builtin_amdgcn_readfirstlane(__popcll(__builtin_amdgcn_ballot_w64(mine <= (int)blockIdx.x)) - 1);
    const AdamwTensor &t = p.t[at];
    const AdamwHyper h = p.device_hyper ? *p.device_hyper : p.hyper;
    const float keep = 1.0f - h.lr_decay * t.decay;
    const int64_t unit = (int64_t)((int)blockIdx.x - p.first[at]) * adamw_unit(FAR);
    float g[PARTS][4], m[PARTS][4], v[PARTS][4], w[PARTS][4];
    uint32_t cm[PARTS], cv[PARTS];
    int em[PARTS], ev[PARTS], left[PARTS];
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        const int64_t base = unit + k * 1024 + threadIdx.x * 4, rest = t.count - base;
        left[k] = rest <= 0 ? 0 : rest < 4 ? (int)rest : 4;
        if (GRAD32)
            load_f32<FAR>(static_cast<const float *>(t.grad) + base, left[k], g[k]);
        else
            load_16<E, FAR>(static_cast<const _Float16 *>(t.grad) + base, left[k], g[k]);
        if (t.master)
            load_f32<FAR>(t.master + base, left[k], w[k]);
        else
            load_16<E, FAR>(t.param + base, left[k], w[k]);
        if constexpr (STATE8) {
            cm[k] = load_codes<FAR>(static_cast<const uint8_t *>(t.m) + base, left[k]);
            cv[k] = load_codes<FAR>(static_cast<const uint8_t *>(t.v) + base, left[k]);
            em[k] = left[k] ? t.m_scale[base / kAdamwBlock] : 0;
            ev[k] = left[k] ? t.v_scale[base / kAdamwBlock] : 0;
        } else {
            load_f32<FAR>(static_cast<const float *>(t.m) + base, left[k], m[k]);
            load_f32<FAR>(static_cast<const float *>(t.v) + base, left[k], v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < PARTS; ++k) {
        const int64_t base = unit + k * 1024 + threadIdx.x * 4;
        if constexpr (STATE8) {
            decode4(cm[k], ldexpf(1.0f, em[k] - 127), m[k]);
            decode4(cv[k], ldexpf(1.0f, ev[k] - 127), v[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] *= v[k][i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = g[k][i] * h.grad_scale;
            float root;
            new_states(h, x, m[k][i], v[k][i], root);
            // the instruction's reciprocal, an ulp off at most: 2^-23 of the step, not of the weight; the
            // denominator is 0 or at least a root of 2^-149 or eps, never a subnormal (hyper_of refuses such an eps)
            w[k][i] = fmaf(w[k][i], keep, -h.lr1 * m[k][i] * __builtin_amdgcn_rcpf(fmaf(root, h.root2, h.eps)));
            if (STATE8) v[k][i] = root;
        }
        if (t.master) store_f32<FAR>(t.master + base, left[k], w[k]);
        if (t.param) store_16<E, FAR>(t.param + base, left[k], w[k]);
        if constexpr (!STATE8) {
            store_f32<FAR>(static_cast<float *>(t.m) + base, left[k], m[k]);
            store_f32<FAR>(static_cast<float *>(t.v) + base, left[k], v[k]);
        }
    }
    if constexpr (STATE8) {
        int e[2 * PARTS];
        float inv[2 * PARTS];
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            e[2 * k] = block_power(m[k]);
            e[2 * k + 1] = block_power(v[k]);
        }
        inverse_powers<2 * PARTS>(e, inv);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            const int64_t base = unit + k * 1024 + threadIdx.x * 4;
            store_codes<FAR>(static_cast<uint8_t *>(t.m) + base, left[k], encode4<false>(m[k], inv[2 * k]));
            store_codes<FAR>(static_cast<uint8_t *>(t.v) + base, left[k], encode4<true>(v[k], inv[2 * k + 1]));
            if (left[k] && (threadIdx.x & 31) == 0) {
                t.m_scale[base / kAdamwBlock] = (uint8_t)(e[2 * k] + 127);
                t.v_scale[base / kAdamwBlock] = (uint8_t)(e[2 * k + 1] + 127);
            }
        }
    }
}

template <typename E, bool FAR>
static void launch(const AdamwParams &p, int64_t blocks, bool state8, bool grad32, hipStream_t s) {
    const dim3 g((uint32_t)blocks), b(256);
    if (state8 && grad32)
        adamw_kernel<E, true, true, FAR><<<g, b, 0, s>>>(p);
    else if (state8)
        adamw_kernel<E, true, false, FAR><<<g, b, 0, s>>>(p);
    else if (grad32)
        adamw_kernel<E, false, true, FAR><<<g, b, 0, s>>>(p);
    else
        adamw_kernel<E, false, false, FAR><<<g, b, 0, s>>>(p);
}

hipError_t launch_adamw(const AdamwParams &p, int64_t blocks, bool far, bool bf16, bool state8, bool grad32, hipStream_t s) {
    if (bf16 && far)
        launch<__bf16, true>(p, blocks, state8, grad32, s);
    else if (bf16)
        launch<__bf16, false>(p, blocks, state8, grad32, s);
    else if (far)
        launch<_Float16, true>(p, blocks, state8, grad32, s);
    else
        launch<_Float16, false>(p, blocks, state8, grad32, s);
    return hipGetLastError();
}

}  // namespace c3d
