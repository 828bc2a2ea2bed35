// Attention over the tokens of a latent grid, forward:
//   o_i = sum_j exp(s_ij - lse_i) v_j,  s_ij = scale q_i . k_j,  lse_i = log sum_j exp(s_ij)
// over the keys j that query i sees.
//
// One pass over the keys with a running maximum and sum per query (in the
// exponent of 2, fp32).  Scores are computed transposed, S^T = K Q^T: an MFMA's
// result then holds one query per lane, so that the maximum, the sum and the
// rescaling of a query's output are a lane's own business (one exchange between
// the halves of the wave for the maximum), and its registers are, as they stand, the operand
// P^T of O^T = V^T P^T.  Probabilities are rounded to the element type for that
// product, one rounding of each, half an ulp as the tensors themselves have; their sum is taken
// of the fp32 values.  fp16 has few exponents for that: there they are lifted (kAttnLift), so that only
// those below 2^-25 of a row's largest are held in fewer bits, in steps of 2^-35.
#include "attention_common.h"

namespace c3d {

constexpr float kAttnLog2e = 1.44269504088896341f, kAttnLn2 = 0.693147180559945309f;

// Exponentials are taken against the running maximum less kAttnLift, in units of log2, and the maximum
// follows a step only where it would be passed by more than kAttnRise: they are then at most 2^15 in
// fp16, which has few exponents and could not hold small ones otherwise (2^16 would be too large: the rounding of
// scores may add 1 to the exponent from 2^24 on, in units of log2, where they tell keys apart no more).  Where many weak keys
// stand beside a strong one whose value is next to nothing, the weak ones are the result: 36863 of
// them 17.5 nats below lost a third of it without a lift, and lose at most 6e-4 with 2^11.  A maximum that follows at once
// (lifts of 12 to 14) rescales the sums more often: 613 keys in heads of 80 7 to 8% more time, this rise 2%,
// a rise of 8 (a lift of 7) none; 20480 keys in heads of 64 1 to 3%, none and none.
// bf16 has fp32's exponents: no lift, and a maximum that seldom follows.
template <typename E>
constexpr float kAttnLift = std::is_same_v<E, __bf16> ? 0.0f : 11.0f;
template <typename E>
constexpr float kAttnRise = std::is_same_v<E, __bf16> ? 8.0f : 4.0f;

// The running softmax of one query per lane, scores in units of log2.
struct AttnSoftmax {
    float max, use;  // the running maximum, less the lift; the same where there is one, else 0
    float sum;       // of the lane's own half of the keys
    __device__ __forceinline__ void init() {
        max = -__builtin_inff();
        use = 0.0f;
        sum = 0.0f;
    }
    // the maximum up to m; the factor of what was summed before
    __device__ __forceinline__ float raise(float m) {
        const float before = max;
        max = fmaxf(max, m);
        use = max == -__builtin_inff() ? 0.0f : max;
        const float f = __builtin_amdgcn_exp2f(before - use);
        sum *= f;
        return f;
    }
};

// The logarithm of a row's sum, the lift taken off where it is exact.
template <typename E>
__device__ __forceinline__ float attn_lse(float use, float sum) {
    return ((use + kAttnLift<E>) + __builtin_amdgcn_logf(sum * __builtin_exp2f(-kAttnLift<E>))) * kAttnLn2;
}

// 1 / sum; 0 for a row that saw no key.
__device__ __forceinline__ float attn_inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

// ---- tiles of 32 RG rows and BN KG keys, 8 waves: wave (rg, kg) holds rows 32 rg .. + 31,
// every lane one of them, and takes the kg-th BN keys of each step; the kg waves of the same rows
// meet in LDS at the end.  Two steps' K and V are in LDS in turn, loaded straight into it while
// the step before is computed.  More rows to a tile read K and V less often, more waves to a
// row shorten the way through its keys: where the rows alone do not fill the card.  What is left
// is the latency of a step: score products, softmax and output products of a wave depend on each other, and
// the other wave of its SIMD fills only part of the gaps (1024 tokens, 8 heads of 128: 16 us in tiles of 64 rows, 272
// TFLOP/s; 4096 tokens, token by token, 16 heads of 128: 78 us in tiles of 128, 880 TFLOP/s).  Deeper rings do not
// help: 3 and 4 steps in LDS were level to slower.  Heads up to 64 are held to 128 registers, two workgroups to a
// CU; 128 rows of heads of 64 spill 6 of them.
template <typename E, int DP, int RG, int KG, int BN>
__global__ __launch_bounds__(512, DP <= 64 ? 4 : 2) void attention_tile_kernel(AttnParams p) {
    constexpr int NT = DP / 32, KK = DP / 16, XN = BN / 32, STEP = KG * BN, TILE = STEP * DP * 2;
    static_assert(RG * KG == 8, "eight waves");
    __shared__ __attribute__((aligned(1024))) char smem[4 * TILE];
    static_assert((KG - 1) * RG * (NT * 4096 + 512) <= (int)sizeof(smem), "the waves' sums fit the buffers");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rg = wave % RG, kg = wave / RG;
    // the longest tiles of a masked problem first, heads side by side
    const int heads = p.n * p.hk, tiles = (int)gridDim.x / heads;
    const int head = blockIdx.x % heads, tile = tiles - 1 - blockIdx.x / heads;
    const int b = head / p.hk, hk = head % p.hk;
    const AttnSample s = attn_sample(p, b);
    const int r0 = tile * RG * 32, d = p.d, last = s.queries - 1;

    int lo = 0, hi = 0;  // the keys that the tile's rows see
    {
        const int t_first = r0 / p.group, t_last = (r0 + RG * 32 - 1) / p.group;
        if (t_first <= last) {
            lo = attn_range(p, s, t_first).lo & ~(BN - 1);
            hi = attn_range(p, s, t_last < last ? t_last : last).hi;
        }
    }
    if (p.splits > 1) {
        lo += blockIdx.y * p.pieces * STEP;
        const int end = lo + p.pieces * STEP;
        hi = hi < end ? hi : end;
    }
    // keys behind hi come as zeros, whatever a cache holds there
    const AttnTile<DP, STEP, 8> tk(p.k + b * p.ks[0] + hk * p.ks[2], p.ks[1], hi, d, wave, lane),
        tv(p.v + b * p.vs[0] + hk * p.vs[2], p.vs[1], hi, d, wave, lane);
    if (lo < hi) {
        tk.load(smem, lo, wave);
        tv.load(smem + TILE, lo, wave);
    }
    // this lane's row; rows past the sample's last query take that one's place
    const int r = r0 + rg * 32 + (lane & 31);
    const int i = r / p.group, g = r - i * p.group;
    const bool alive = i < s.queries;
    half8_t q[KK];
    {
        const _Float16 *row = p.q + b * p.qs[0] + i * p.qs[1] + (int64_t)(hk * p.group + g) * p.qs[2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int e = 16 * kk + 8 * (lane >> 5);
            half8_t z = {};
            q[kk] = alive && e < d ? *reinterpret_cast<const half8_t *>(row + e) : z;
        }
    }
    const AttnRange seen = last < 0 ? AttnRange{0, 0} : attn_range(p, s, i < last ? i : last);
    const int wave_lo = __builtin_amdgcn_readfirstlane(seen.lo), wave_hi_all = __builtin_amdgcn_readfirstlane(seen.hi);
    const int wave_lo_all = __builtin_amdgcn_readlane(seen.lo, 31), wave_hi = __builtin_amdgcn_readlane(seen.hi, 31);
    AttnRows<DP> fk;
    AttnCols<DP> fv;
    fk.init(lane);
    fv.init(lane);

    const float c = p.scale * kAttnLog2e;
    AttnSoftmax sm;
    sm.init();
    f32x16 acc[NT] = {};
    int buf = 0;
    for (int at = lo; at < hi; at += STEP) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const char *ks = smem + buf * 2 * TILE + kg * BN * DP * 2, *vs = ks + TILE;
        buf ^= 1;
        auto next = [&]() {
            if (at + STEP < hi) {
                char *to = smem + buf * 2 * TILE;
                tk.load(to, at + STEP, wave);
                tv.load(to + TILE, at + STEP, wave);
            }
        };
        const int j0 = at + kg * BN;
        if (j0 + BN <= wave_lo || j0 >= wave_hi) {
            next();
            continue;
        }
        const uint32_t kr = lds_address(ks) + fk.off;
        f32x16 x[XN] = {};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int t = 0; t < XN; ++t) x[t] = mfma_32x32x16<E>(fk.read(kr, 32 * t, kk), q[kk], x[t]);
        // behind the products, which these then do not hold up: the next step's loads, and the first of v's
        // fragments, whose wait the products cover
        half8_t ahead[2][NT];
        fv.template read<0>(vs, ahead[0]);
        fv.template read<1>(vs, ahead[1]);
        next();
        if (j0 < wave_lo_all || j0 + BN > wave_hi_all) {
            const int from = seen.lo - j0, to = seen.hi - j0;
#pragma unroll
            for (int t = 0; t < XN; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = 32 * t + acc_row(e, lane >> 5);
                    x[t][e] = j >= from && j < to ? x[t][e] : -__builtin_inff();
                }
        }
        float mx = x[0][0];
#pragma unroll
        for (int t = 0; t < XN; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[t][e]);
        mx = both_max(mx) * c;
        if (__builtin_amdgcn_ballot_w64(mx > sm.max + (kAttnLift<E> + kAttnRise<E>))) {
            const float f = sm.raise(mx - kAttnLift<E>);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[t][e] *= f;
        }
#pragma unroll
        for (int t = 0; t < XN; ++t)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[t][e] = __builtin_amdgcn_exp2f(fmaf(x[t][e], c, -sm.use));
                sm.sum += x[t][e];
            }
        static_for<2 * XN>([&](auto step) {
            constexpr int S = decltype(step)::value;
            half8_t f[NT];
            if constexpr (S > 1) fv.template read<S>(vs, f);
            const half8_t w = pack8<E>(x[S / 2], (S & 1) * 8);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = mfma_32x32x16<E>(S > 1 ? f[t] : ahead[S & 1][t], w, acc[t]);
        });
    }
    if constexpr (KG > 1) {
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the buffers are free
        float *sums = reinterpret_cast<float *>(smem);
        float2 *ml = reinterpret_cast<float2 *>(sums + (KG - 1) * RG * NT * 1024);
        if (kg > 0) {
            const int at = (kg - 1) * RG + rg;
            acc_put<NT>(sums + at * NT * 1024, acc, lane);
            ml[at * 64 + lane] = make_float2(sm.max, sm.sum);
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll 1
        for (int o = 0; o < KG - 1; ++o) {
            const int at = o * RG + rg;
            const float2 x = ml[at * 64 + lane];
            const float own = sm.raise(x.x), f = __builtin_amdgcn_exp2f(x.x - sm.use);
            sm.sum = fmaf(x.y, f, sm.sum);
            acc_join<NT>(sums + at * NT * 1024, acc, own, f, lane);
        }
    }
    const float sum = both_sum(sm.sum);
    if (r >= p.rows) return;
    if (p.splits > 1) {
        const int64_t at = ((int64_t)blockIdx.y * heads + head) * p.rows + r;
        if (lane < 32) p.part_ml[at] = make_float2(sm.max, sum);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int e0 = 32 * t + acc_row(e, lane >> 5);
                if (e0 < d)
                    *reinterpret_cast<f32x4 *>(p.part_o + at * d + e0) =
                        f32x4{acc[t][e], acc[t][e + 1], acc[t][e + 2], acc[t][e + 3]};
            }
        return;
    }
    if (!alive) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x16{};
    }
    const float inv = attn_inverse(sum);
    const int h = hk * p.group + g;
    if (p.lse && lane < 32)
        p.lse[((int64_t)b * p.hq + h) * p.tq + i] =
            alive ? attn_lse<E>(sm.use, sum) : -__builtin_inff();
    _Float16 *out = p.o + b * p.os[0] + i * p.os[1] + h * p.os[2];
#pragma unroll
    for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, acc[t], inv, d - 32 * t, lane, true);
}

// ---- 256 rows, 64 keys to a step, for problems that fill the card: the same computation with
// the two waves of each SIMD (w and w + 4) one phase apart.  A phase is either a step's
// softmax, on the vector units, or the products around it (the next step's scores and this
// step's share of the output), on the matrix core, so that each SIMD's matrix core always has
// one of its two waves.  One barrier per phase.  K and V are in LDS three steps deep: in the
// softmax of step t a wave issues its share of K(t + 2) and V(t + 1), which take the places of
// K(t - 1) and V(t - 2), whose last readers were one phase and two phases ago, and sees that they have landed
// at the end of the products that follow; the other group's first reads of them are two phases later.
// 20480 tokens causal by frames of 4096, 16 heads of 128: 1709-1760 us, 1170-1205 TFLOP/s (the tile kernel 1904),
// matrix cores busy 65% at the 1.7-1.8 GHz that power leaves.  9 frames of 1024 tokens, 16 heads of 128: 101-108 us,
// 710-764 TFLOP/s, busy 48%: 576 equal tiles on 256 CUs are 2.25 rounds, and take three.  At heads of 64 a
// score costs as many cycles of the vector units as at 128 for half the products (4096 rows on 20480 keys 392-405 us,
// 850-880 TFLOP/s, vector units busy 63%, matrix cores 40%).  Heads up to 64 are held to 128 registers, which
// leaves room for two workgroups to a CU and spills 8 of them at 64, 2 at 32: with 256 registers and no spills the same
// case, one workgroup to a CU, takes 394 us for 392.
template <typename E, int DP>
__global__ __launch_bounds__(512, DP <= 64 ? 4 : 2) void attention_phase_kernel(AttnParams p) {
    constexpr int BN = 64, NT = DP / 32, KK = DP / 16, TILE = BN * DP * 2;
    __shared__ __attribute__((aligned(1024))) char smem[6 * TILE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = p.n * p.hk, tiles = (int)gridDim.x / heads;
    const int head = blockIdx.x % heads, tile = tiles - 1 - blockIdx.x / heads;
    const int b = head / p.hk, hk = head % p.hk;
    const AttnSample s = attn_sample(p, b);
    const int r0 = tile * 256, d = p.d, last = s.queries - 1;
    int lo = 0, hi = 0;
    {
        const int t_first = r0 / p.group, t_last = (r0 + 255) / p.group;
        if (t_first <= last) {
            lo = attn_range(p, s, t_first).lo & ~(BN - 1);
            hi = attn_range(p, s, t_last < last ? t_last : last).hi;
        }
    }
    if (p.splits > 1) {
        lo += blockIdx.y * p.pieces * BN;
        const int end = lo + p.pieces * BN;
        hi = hi < end ? hi : end;
    }
    const AttnTile<DP, BN, 8> tk(p.k + b * p.ks[0] + hk * p.ks[2], p.ks[1], hi, d, wave, lane),
        tv(p.v + b * p.vs[0] + hk * p.vs[2], p.vs[1], hi, d, wave, lane);
    char *const vbuf = smem + 3 * TILE;
    const bool any = lo < hi;
    if (any) {
        tk.load(smem, lo, wave);
        tv.load(vbuf, lo, wave);
        tk.load(smem + TILE, lo + BN, wave);  // behind the last key: zeros
    }
    const int r = r0 + wave * 32 + (lane & 31);
    const int i = r / p.group, g = r - i * p.group;
    const bool alive = i < s.queries;
    half8_t q[KK];
    {
        const _Float16 *row = p.q + b * p.qs[0] + i * p.qs[1] + (int64_t)(hk * p.group + g) * p.qs[2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int e = 16 * kk + 8 * (lane >> 5);
            half8_t z = {};
            q[kk] = alive && e < d ? *reinterpret_cast<const half8_t *>(row + e) : z;
        }
    }
    const AttnRange seen = last < 0 ? AttnRange{0, 0} : attn_range(p, s, i < last ? i : last);
    const int all_lo = __builtin_amdgcn_readlane(seen.lo, 31), all_hi = __builtin_amdgcn_readfirstlane(seen.hi);
    AttnRows<DP> fk;
    AttnCols<DP> fv;
    fk.init(lane);
    fv.init(lane);
    const float c = p.scale * kAttnLog2e;
    AttnSoftmax sm;
    sm.init();
    f32x16 acc[NT] = {};
    if (any) {
        auto phase_end = [&]() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
        f32x16 x[2];
        half8_t w[4];
        auto scores = [&](const char *ks) {
            const uint32_t kr = lds_address(ks) + fk.off;
            x[0] = x[1] = f32x16{};
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int t = 0; t < 2; ++t) x[t] = mfma_32x32x16<E>(fk.read(kr, 32 * t, kk), q[kk], x[t]);
        };
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (wave >= 4) phase_end();
        scores(smem);
        phase_end();
        int k1 = 1, v0 = 0;  // the places of K(t + 1) and V(t)
        for (int j0 = lo; j0 < hi; j0 += BN) {
            const int k2 = k1 == 2 ? 0 : k1 + 1, v1 = v0 == 2 ? 0 : v0 + 1;
            tk.load(smem + k2 * TILE, j0 + 2 * BN, wave);
            tv.load(vbuf + v1 * TILE, j0 + BN, wave);
            if (j0 < all_lo || j0 + BN > all_hi) {
                const int from = seen.lo - j0, to = seen.hi - j0;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = 32 * t + acc_row(e, lane >> 5);
                        x[t][e] = j >= from && j < to ? x[t][e] : -__builtin_inff();
                    }
            }
            float mx = x[0][0];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[t][e]);
            mx = both_max(mx) * c;
            if (__builtin_amdgcn_ballot_w64(mx > sm.max + (kAttnLift<E> + kAttnRise<E>))) {
                const float f = sm.raise(mx - kAttnLift<E>);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[t][e] *= f;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[t][e] = __builtin_amdgcn_exp2f(fmaf(x[t][e], c, -sm.use));
                    sm.sum += x[t][e];
                }
#pragma unroll
            for (int t = 0; t < 4; ++t) w[t] = pack8<E>(x[t / 2], (t & 1) * 8);
            __builtin_amdgcn_sched_barrier(0);
            phase_end();
            __builtin_amdgcn_s_setprio(2);
            scores(smem + k1 * TILE);
            const uint32_t b0 = lds_address(vbuf + v0 * TILE) + fv.off0, b1 = lds_address(vbuf + v0 * TILE) + fv.off1;
            static_for<4>([&](auto step) {
                constexpr int S = decltype(step)::value;
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] = mfma_32x32x16<E>(fv.template fragment<S>(b0, b1, t), w[S], acc[t]);
            });
            __builtin_amdgcn_s_setprio(0);
            k1 = k2;
            v0 = v1;
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        if (wave < 4) phase_end();  // as many barriers as the other group
    }
    const float sum = both_sum(sm.sum);
    if (r >= p.rows) return;
    if (p.splits > 1) {
        const int64_t at = ((int64_t)blockIdx.y * heads + head) * p.rows + r;
        if (lane < 32) p.part_ml[at] = make_float2(sm.max, sum);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int e0 = 32 * t + acc_row(e, lane >> 5);
                if (e0 < d)
                    *reinterpret_cast<f32x4 *>(p.part_o + at * d + e0) =
                        f32x4{acc[t][e], acc[t][e + 1], acc[t][e + 2], acc[t][e + 3]};
            }
        return;
    }
    if (!alive) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x16{};
    }
    const float inv = attn_inverse(sum);
    const int h = hk * p.group + g;
    if (p.lse && lane < 32)
        p.lse[((int64_t)b * p.hq + h) * p.tq + i] =
            alive ? attn_lse<E>(sm.use, sum) : -__builtin_inff();
    _Float16 *out = p.o + b * p.os[0] + i * p.os[1] + h * p.os[2];
#pragma unroll
    for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, acc[t], inv, d - 32 * t, lane, true);
}

// ---- few rows (at most 32 to a key head: single tokens): the time is that of reading
// K and V once.  Every wave takes 32 keys at a time, in turn with the other waves, through
// LDS buffers of its own, so that no barrier ties the waves' loads together; their sums
// meet in LDS at the end.  16 samples of one token, 16 heads over 4 key heads of 128, up to 36864
// keys: 170 us and 4.3 for the join, 5.5 TB/s, bound by memory (matrix cores busy 10%).
template <typename E, int DP>
__global__ __launch_bounds__(256) void attention_few_kernel(AttnParams p) {
    constexpr int WAVES = 4, BN = 32, NT = DP / 32, KK = DP / 16, TILE = BN * DP * 2, NL = 2 * AttnTile<DP, BN, 1>::LOADS;
    static_assert(WAVES * BN == attn_tile(kAttnFew).keys, "keys of a step");
    __shared__ __attribute__((aligned(1024))) char smem[WAVES * 4 * TILE];
    static_assert(WAVES * (32 * DP + 64) * 4 <= (int)sizeof(smem), "the waves' sums fit the buffers");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = p.n * p.hk, head = blockIdx.x % heads, split = blockIdx.x / heads;
    const int b = head / p.hk, hk = head % p.hk;
    const AttnSample s = attn_sample(p, b);
    const int r = lane & 31;
    const int i = r / p.group, g = r - i * p.group;
    const bool alive = r < p.rows && i < s.queries;
    const int last = s.queries - 1;
    const AttnRange seen = last < 0 ? AttnRange{0, 0} : attn_range(p, s, i < last ? i : last);
    const int lo_all = __builtin_amdgcn_readlane(seen.lo, 31), hi_all = __builtin_amdgcn_readfirstlane(seen.hi);
    int lo = __builtin_amdgcn_readfirstlane(seen.lo) & ~(BN - 1), hi = __builtin_amdgcn_readlane(seen.hi, 31);
    if (p.splits > 1) {
        lo += split * p.pieces * WAVES * BN;
        const int end = lo + p.pieces * WAVES * BN;
        hi = hi < end ? hi : end;
    }
    const int d = p.d;
    const AttnTile<DP, BN, 1> tk(p.k + b * p.ks[0] + hk * p.ks[2], p.ks[1], hi, d, 0, lane),
        tv(p.v + b * p.vs[0] + hk * p.vs[2], p.vs[1], hi, d, 0, lane);
    char *mine = smem + wave * 4 * TILE;
    int buf = 0;
    int j0 = lo + wave * BN;
    // rows past the last key load zeros, so every step has the same number of loads
    tk.load(mine, j0, 0);
    tv.load(mine + TILE, j0, 0);
    half8_t q[KK];
    {
        const _Float16 *row = p.q + b * p.qs[0] + i * p.qs[1] + (int64_t)(hk * p.group + g) * p.qs[2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int e = 16 * kk + 8 * (lane >> 5);
            half8_t z = {};
            q[kk] = alive && e < d ? *reinterpret_cast<const half8_t *>(row + e) : z;
        }
    }
    AttnRows<DP> fk;
    AttnCols<DP> fv;
    fk.init(lane);
    fv.init(lane);
    const float c = p.scale * kAttnLog2e;
    AttnSoftmax sm;
    sm.init();
    f32x16 acc[NT] = {};
    for (; j0 < hi; j0 += WAVES * BN) {
        char *next = mine + (buf ^ 1) * 2 * TILE;
        tk.load(next, j0 + WAVES * BN, 0);
        tv.load(next + TILE, j0 + WAVES * BN, 0);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NL) : "memory");
        const char *ks = mine + buf * 2 * TILE, *vs = ks + TILE;
        buf ^= 1;
        const uint32_t kr = lds_address(ks) + fk.off;
        f32x16 x = {};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) x = mfma_32x32x16<E>(fk.read(kr, 0, kk), q[kk], x);
        if (j0 < lo_all || j0 + BN > hi_all) {
            const int from = seen.lo - j0, to = seen.hi - j0;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int j = acc_row(e, lane >> 5);
                x[e] = j >= from && j < to ? x[e] : -__builtin_inff();
            }
        }
        float mx = x[0];
#pragma unroll
        for (int e = 1; e < 16; ++e) mx = fmaxf(mx, x[e]);
        mx = both_max(mx) * c;
        if (__builtin_amdgcn_ballot_w64(mx > sm.max + (kAttnLift<E> + kAttnRise<E>))) {
            const float f = sm.raise(mx - kAttnLift<E>);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[t][e] *= f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            x[e] = __builtin_amdgcn_exp2f(fmaf(x[e], c, -sm.use));
            sm.sum += x[e];
        }
        static_for<2>([&](auto step) {
            constexpr int S = decltype(step)::value;
            half8_t f[NT];
            fv.template read<S>(vs, f);
            const half8_t w = pack8<E>(x, S * 8);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = mfma_32x32x16<E>(f[t], w, acc[t]);
        });
    }
    // the waves' results meet: [wave][row][element] sums, then [wave][row] (maximum, sum)
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    float *sums = reinterpret_cast<float *>(smem);
    float2 *ml = reinterpret_cast<float2 *>(sums + WAVES * 32 * DP);
    const float total = both_sum(sm.sum);
    if (lane < 32) ml[wave * 32 + r] = make_float2(sm.max, total);
    // 16-byte pieces exchange places so that the rows' equal elements lie in different banks
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const int piece = (32 * t + acc_row(e, lane >> 5)) >> 2;
            *reinterpret_cast<f32x4 *>(sums + (wave * 32 + r) * DP + ((piece ^ (r & 7)) << 2)) =
                f32x4{acc[t][e], acc[t][e + 1], acc[t][e + 2], acc[t][e + 3]};
        }
    __syncthreads();
    const int pieces = d >> 2;
    for (int at = threadIdx.x; at < p.rows * pieces; at += 256) {
        const int row = at / pieces, e = (at - row * pieces) * 4;
        float m = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) m = fmaxf(m, ml[w * 32 + row].x);
        const float use = m == -__builtin_inff() ? 0.0f : m;
        float sum = 0.0f;
        f32x4 v = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float2 x = ml[w * 32 + row];
            const float f = __builtin_amdgcn_exp2f(x.x - use);
            sum = fmaf(x.y, f, sum);
            const f32x4 a = *reinterpret_cast<const f32x4 *>(sums + (w * 32 + row) * DP + (((e >> 2) ^ (row & 7)) << 2));
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = fmaf(a[k], f, v[k]);
        }
        if (p.splits > 1) {
            const int64_t to = ((int64_t)split * heads + head) * p.rows + row;
            *reinterpret_cast<f32x4 *>(p.part_o + to * d + e) = v;
            if (e == 0) p.part_ml[to] = make_float2(m, sum);
            continue;
        }
        const int ti = row / p.group, h = hk * p.group + row - ti * p.group;
        const bool live = ti < s.queries;
        const float inv = attn_inverse(sum);
        if (e == 0 && p.lse)
            p.lse[((int64_t)b * p.hq + h) * p.tq + ti] =
                live ? attn_lse<E>(use, sum) : -__builtin_inff();
        half4_t o;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = live ? from_f32<E>(v[k] * inv) : (_Float16)0.0f;
        *reinterpret_cast<half4_t *>(p.o + b * p.os[0] + ti * p.os[1] + h * p.os[2] + e) = o;
    }
}

// The pieces of each row's keys joined, in a fixed order: a workgroup per row, LANES lanes of four
// elements to a piece, the pieces in turn over the workgroup, whose sums meet in LDS.  (With a wave per
// row, one token of 16 heads on 36864 keys of 4 key heads, 128 pieces, took 38 us instead of 20.)
template <typename E, int LANES>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnParams p) {
    constexpr int SETS = 256 / LANES;
    __shared__ __attribute__((aligned(16))) float sums[256 * 4];
    __shared__ float2 ml[SETS];
    const int heads = p.n * p.hk, set = threadIdx.x / LANES, l = threadIdx.x % LANES, e = 4 * l;
    const int64_t unit = blockIdx.x, count = (int64_t)heads * p.rows;
    const int head = (int)(unit / p.rows), row = (int)(unit - (int64_t)head * p.rows);
    float m = -__builtin_inff(), sum = 0.0f;
    f32x4 v = {};
#pragma unroll 2
    for (int k = set; k < p.splits; k += SETS) {
        const float2 x = p.part_ml[k * count + unit];
        f32x4 a = {};
        if (e < p.d) a = *reinterpret_cast<const f32x4 *>(p.part_o + (k * count + unit) * p.d + e);
        const float top = fmaxf(m, x.x), use = top == -__builtin_inff() ? 0.0f : top;
        const float own = __builtin_amdgcn_exp2f(m - use), f = __builtin_amdgcn_exp2f(x.x - use);
        m = top;
        sum = fmaf(sum, own, x.y * f);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = fmaf(v[c], own, a[c] * f);
    }
    *reinterpret_cast<f32x4 *>(sums + threadIdx.x * 4) = v;
    if (l == 0) ml[set] = make_float2(m, sum);
    __syncthreads();
    if (set > 0) return;
#pragma unroll
    for (int k = 1; k < SETS; ++k) m = fmaxf(m, ml[k].x);
    const float use = m == -__builtin_inff() ? 0.0f : m;
    v = f32x4{};
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
        const float2 x = ml[k];
        const float f = __builtin_amdgcn_exp2f(x.x - use);
        sum = fmaf(x.y, f, sum);
        const f32x4 a = *reinterpret_cast<const f32x4 *>(sums + (k * LANES + l) * 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = fmaf(a[c], f, v[c]);
    }
    const int b = head / p.hk, hk = head - b * p.hk;
    const int ti = row / p.group, h = hk * p.group + row - ti * p.group;
    const bool live = ti < attn_sample(p, b).queries;
    const float inv = attn_inverse(sum);
    if (l == 0 && p.lse)
        p.lse[((int64_t)b * p.hq + h) * p.tq + ti] =
            live ? attn_lse<E>(use, sum) : -__builtin_inff();
    if (e < p.d) {
        half4_t o;
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = live ? from_f32<E>(v[c] * inv) : (_Float16)0.0f;
        *reinterpret_cast<half4_t *>(p.o + b * p.os[0] + ti * p.os[1] + h * p.os[2] + e) = o;
    }
}

template <typename E, int DP>
static void launch_forward(const AttnParams &p, AttnTileKind kind, hipStream_t s) {
    const int heads = p.n * p.hk, rows = attn_tile(kind).rows;
    const dim3 grid((uint32_t)(heads * ((p.rows + rows - 1) / rows)), (uint32_t)p.splits), block(512);
    switch (kind) {
        case kAttnFew: attention_few_kernel<E, DP><<<dim3(heads * p.splits), dim3(256), 0, s>>>(p); break;
        case kAttn64: attention_tile_kernel<E, DP, 2, 4, 32><<<grid, block, 0, s>>>(p); break;
        case kAttn128: attention_tile_kernel<E, DP, 4, 2, 64><<<grid, block, 0, s>>>(p); break;
        default: attention_phase_kernel<E, DP><<<grid, block, 0, s>>>(p); break;
    }
    if (p.splits > 1) {
        attention_join_kernel<E, (DP > 64 ? 32 : DP / 4)><<<dim3((uint32_t)(heads * p.rows)), dim3(256), 0, s>>>(p);
    }
}

template <typename E>
static void launch_forward_dim(const AttnParams &p, AttnTileKind kind, hipStream_t s) {
    if (p.d <= 32)
        launch_forward<E, 32>(p, kind, s);
    else if (p.d <= 64)
        launch_forward<E, 64>(p, kind, s);
    else if (p.d <= 96)
        launch_forward<E, 96>(p, kind, s);
    else
        launch_forward<E, 128>(p, kind, s);
}

hipError_t launch_attention(const AttnParams &p, AttnTileKind kind, hipStream_t s) {
    if (p.bf16)
        launch_forward_dim<__bf16>(p, kind, s);
    else
        launch_forward_dim<_Float16>(p, kind, s);
    return hipGetLastError();
}

}  // namespace c3d
