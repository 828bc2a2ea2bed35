// Attention's gradients.  With P = exp(s - lse) computed again from q, k and the
// forward pass's lse, and delta_i = dout_i . o_i:
//   dP_ij = dout_i . v_j,  dS_ij = P_ij (dP_ij - delta_i)
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dout_i
// One kernel holds query rows and runs over the keys (dq), another holds keys and runs over the
// query rows (dk, dv); a third is both in one launch.  S and dP are computed in both, seven products for
// the five of the formula, so that a sum is one workgroup's own: its waves' parts meet in LDS, in a fixed order.
// Where few keys meet many queries, a key tile's steps are split over workgroups, which leave fp32 partials of dk
// and dv in the workspace; a join kernel adds them in their order.  No atomics: the same result in every call.
#include "attention_common.h"

namespace c3d {

constexpr float kAttnLog2e = 1.44269504088896341f;

// What the kernels read of a query row besides its vectors, from the forward pass's lse and the
// row sum dout . o: -lse / scale and -delta, the values that the accumulators of S and dP start
// from (0 for rows that see no key, whose probabilities are never used).
__device__ __forceinline__ float start_of_scores(float lse, float scale) {
    return lse == -__builtin_inff() ? 0.0f : -lse / scale;
}

template <typename E>
__device__ __forceinline__ float dot8(half8_t a, half8_t b) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(to_f32<E>(a[e]), to_f32<E>(b[e]), s);
    return s;
}

// ---- dq: tiles of 32 RG rows and BN KG keys as in the forward pass.  S^T = K Q^T and dP^T = V dout^T
// hold one query per lane; dS^T is, as it stands, the operand of dq^T = K^T dS^T.
//
// delta_i = sum_j P_ij dP_ij is dout_i . o_i, but o is rounded, and where a query sees few keys
// that rounding is as large as those of dS and dq together (one key: dS is 0, and would be
// nothing but it).  Tiles whose first query sees fewer than kFewKeys keys therefore take the
// sum itself, in a pass over the keys of its own, as long as there are at most kFewSpan of them: for 64
// tokens, causal, the error of dq falls from 1.72 to 1.43 times that of the plain form.
constexpr int kFewKeys = 160, kFewSpan = 512;
//
// Three products for two of the forward pass, and the exponentials once more; K and V of a step are in LDS,
// read as they lie and transposed.  20480 tokens causal by frames of 4096, 16 heads of 128: 2502 us, 1236 TFLOP/s,
// matrix cores busy 65%, power-bound as the forward pass; 3 samples of 1543 tokens, 12 heads of 80 on 4: 38 us, busy 27%: a
// step of 128 rows is 2.1 us, 1.9 of it products (of 96 elements for 80), but a workgroup has about five, and 6.5 us of
// its own around them (the first loads, the waves' join, the stores) that no other one on its CU covers.
//
// READY: nlse and ndelta are there, from a launch of this kernel without dq.
template <int DP, int RG, int KG, int BN>
constexpr int dq_lds() {
    static_assert(RG * KG == 8, "eight waves");
    static_assert((KG - 1) * RG * (DP / 32) * 4096 <= 4 * KG * BN * DP * 2, "the waves' sums fit the buffers");
    return 4 * KG * BN * DP * 2 + (KG > 1 ? 2048 : 0);
}
template <typename E, int DP, int RG, int KG, int BN, bool READY>
__device__ __forceinline__ void dq_tile(const AttnParams &p, int block, int tiles, char *smem) {
    constexpr int NT = DP / 32, KK = DP / 16, XN = BN / 32, STEP = KG * BN, TILE = STEP * DP * 2;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rg = wave % RG, kg = wave / RG;
    const int heads = p.n * p.hk;
    const int head = block % heads, tile = tiles - 1 - block / heads;
    const int b = head / p.hk, hk = head % p.hk;
    const AttnSample s = attn_sample(p, b);
    const int r0 = tile * RG * 32, d = p.d, last = s.queries - 1;
    int lo = 0, hi = 0;
    bool few = false;
    {
        const int t_first = r0 / p.group, t_last = (r0 + RG * 32 - 1) / p.group;
        if (t_first <= last) {
            const AttnRange first = attn_range(p, s, t_first);
            lo = first.lo & ~(BN - 1);
            hi = attn_range(p, s, t_last < last ? t_last : last).hi;
            few = !READY && first.hi - first.lo < kFewKeys && hi - lo <= kFewSpan;
        }
        if (!p.dq && !few) hi = lo;  // the rows' sums alone are asked for
    }
    const AttnTile<DP, STEP, 8> tk(p.k + b * p.ks[0] + hk * p.ks[2], p.ks[1], s.keys, d, wave, lane),
        tv(p.v + b * p.vs[0] + hk * p.vs[2], p.vs[1], s.keys, d, wave, lane);
    if (lo < hi) {
        tk.load(smem, lo, wave);
        tv.load(smem + TILE, lo, wave);
    }
    const int r = r0 + rg * 32 + (lane & 31);
    const int i = r / p.group, g = r - i * p.group, h = hk * p.group + g;
    const bool alive = i < s.queries;
    half8_t q[KK], go[KK];
    float delta = 0.0f, lse = -__builtin_inff();
    {
        const _Float16 *rq = p.q + b * p.qs[0] + i * p.qs[1] + h * p.qs[2];
        const int64_t at = b * p.os[0] + i * p.os[1] + h * p.os[2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int e = 16 * kk + 8 * (lane >> 5);
            half8_t z = {}, o = {};
            q[kk] = go[kk] = z;
            if (alive && e < d) {
                q[kk] = *reinterpret_cast<const half8_t *>(rq + e);
                go[kk] = *reinterpret_cast<const half8_t *>(p.dout + at + e);
                if (!READY) o = *reinterpret_cast<const half8_t *>(p.o + at + e);
            }
            if (!READY) delta += dot8<E>(go[kk], o);
        }
        if (!READY) delta = both_sum(delta);
        const int64_t row = ((int64_t)b * p.hq + h) * p.tq + i;
        if (alive) lse = p.lse[row];
        if (READY && alive) delta = -p.ndelta[row];
    }
    const AttnRange seen = last < 0 ? AttnRange{0, 0} : attn_range(p, s, i < last ? i : last);
    const int wave_lo = __builtin_amdgcn_readfirstlane(seen.lo), wave_hi_all = __builtin_amdgcn_readfirstlane(seen.hi);
    const int wave_lo_all = __builtin_amdgcn_readlane(seen.lo, 31), wave_hi = __builtin_amdgcn_readlane(seen.hi, 31);
    AttnRows<DP> fr;
    AttnCols<DP> fc;
    fr.init(lane);
    fc.init(lane);
    const float c = p.scale * kAttnLog2e, lse2 = (lse == -__builtin_inff() ? 0.0f : lse * kAttnLog2e) - kLift<E>;
    f32x16 acc[NT] = {};
    ColumnScale<E> scale;
    float sum = 0.0f;  // of P dP, this lane's keys
    int buf = 0;
    // one pass over the keys: the sum of P dP (SUM), or dq; the first step's tiles are on their way
    auto pass = [&](auto which) {
        constexpr bool SUM = decltype(which)::value;
        for (int at = lo; at < hi; at += STEP) {
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const char *ks = smem + buf * 2 * TILE + kg * BN * DP * 2;
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
            const bool edge = j0 < wave_lo_all || j0 + BN > wave_hi_all;
            const uint32_t kr = lds_address(ks) + fr.off;
            static_for<XN>([&](auto sub) {
                constexpr int T = decltype(sub)::value;
                f32x16 x = {}, y;
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = SUM ? 0.0f : -delta;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    x = mfma_32x32x16<E>(fr.read(kr, 32 * T, kk), q[kk], x);
                    y = mfma_32x32x16<E>(fr.read(kr, STEP + 32 * T, kk), go[kk], y);
                }
                if constexpr (T == 0) next();  // behind the products, which it then does not hold up
                if (edge) {
                    const int from = seen.lo - j0, to = seen.hi - j0;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = 32 * T + acc_row(e, lane >> 5);
                        x[e] = j >= from && j < to ? x[e] : -__builtin_inff();
                    }
                }
                if constexpr (SUM) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        sum = fmaf(__builtin_amdgcn_exp2f(fmaf(x[e], c, -lse2 - kLift<E>)), y[e], sum);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(x[e], c, -lse2)) * y[e];
                    scale.template apply<NT>(x, acc);
                    static_for<2>([&](auto step) {
                        constexpr int S = decltype(step)::value;
                        half8_t f[NT];
                        fc.template read<2 * T + S>(ks, f);
                        const half8_t w = pack8<E>(x, S * 8);
#pragma unroll
                        for (int t = 0; t < NT; ++t) acc[t] = mfma_32x32x16<E>(f[t], w, acc[t]);
                    });
                }
            });
        }
    };
    if (few) {
        pass(std::true_type{});
        sum = both_sum(sum);
        if constexpr (KG > 1) {
            float *parts = reinterpret_cast<float *>(smem + 4 * TILE);
            parts[threadIdx.x] = sum;
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int k = 0; k < KG; ++k) sum += parts[(k * RG + rg) * 64 + lane];
        }
        delta = sum;
        buf = 0;
        if (p.dq && hi - lo > STEP) {  // a single step is still there
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the buffers are free
            tk.load(smem, lo, wave);
            tv.load(smem + TILE, lo, wave);
        }
    }
    if (!READY && r < p.rows && lane < 32 && kg == 0) {
        const int64_t row = ((int64_t)b * p.hq + h) * p.tq + i;
        p.nlse[row] = start_of_scores(lse, p.scale);
        p.ndelta[row] = alive ? -delta : 0.0f;
    }
    if (!p.dq) return;
    pass(std::false_type{});
    if constexpr (KG > 1) {
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the buffers are free
        float *sums = reinterpret_cast<float *>(smem);
        if constexpr (!std::is_same_v<E, __bf16>) acc_scale<NT>(acc, 1.0f / scale.f);
        scale.f = 1.0f;
        if (kg > 0) acc_put<NT>(sums + ((kg - 1) * RG + rg) * NT * 1024, acc, lane);
        __syncthreads();
        if (kg > 0) return;
#pragma unroll 1
        for (int o = 0; o < KG - 1; ++o) acc_join<NT>(sums + (o * RG + rg) * NT * 1024, acc, 1.0f, 1.0f, lane);
    }
    if (r >= p.rows) return;
    if (!alive) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x16{};
    }
    _Float16 *out = p.dq + b * p.qs[0] + i * p.qs[1] + h * p.qs[2];
#pragma unroll
    for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, acc[t], p.scale * kDrop<E> / scale.f, d - 32 * t, lane, true);
}
template <typename E, int DP, int RG, int KG, int BN>
__global__ __launch_bounds__(512) void attention_dq_kernel(AttnParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[dq_lds<DP, RG, KG, BN>()];
    dq_tile<E, DP, RG, KG, BN, false>(p, blockIdx.x, (int)gridDim.x / (p.n * p.hk), smem);
}

// ---- dk, dv: tiles of 32 KW keys and BM QG query tokens, 8 waves: wave (kw, qg) holds keys
// 32 kw .. + 31 (one key per lane of every result) and takes the qg-th BM tokens of each step; the
// query heads of the key head are taken one after the other.  S = Q K^T and dP = dout V^T; P
// and dS are, as they stand, the operands of dv^T = dout^T P and dk^T = Q^T dS.  The qg waves of
// the same keys meet in LDS at the end.
//
// 20480 tokens causal by frames of 4096, 16 heads of 128: 3566 us, 1155 TFLOP/s over its four products, matrix cores
// busy 55%, LDS 41%: a SIMD's two waves hold 256 accumulators, and what a wave reads of Q and dout
// feeds only its 32 keys.  At heads of 128 the 256 registers do not hold all: 18 to 32 are spilled, and one of them,
// the lane's offset of the rows' numbers, is reloaded in every step behind the next tiles' loads, for which the first two
// waves then wait too.  One wave per SIMD with 64 keys, its steps pipelined, reads half of that
// and took 4686 us: nothing fills its softmax.  3 samples of 1543 tokens, 12 heads of 80 on 4: 50 us and 6 for the join.
template <int DP, int KW, int QG, int BM>
constexpr int dkv_lds() {
    constexpr int bytes = (DP > 64 ? KW * 32 * DP * 2 : 0) + 4 * QG * BM * DP * 2 + 4 * QG * BM * 4;
    static_assert(KW * QG == 8, "eight waves");
    static_assert(bytes <= 160 * 1024, "LDS is 160 KiB per CU");
    static_assert((QG - 1) * KW * (DP / 32) * 4096 <= bytes, "the waves' sums fit the buffers");
    return bytes;
}
template <typename E, int DP, int KW, int QG, int BM>
__device__ __forceinline__ void dkv_tile(const AttnParams &p, int block, int piece, char *smem) {
    constexpr int NT = DP / 32, KK = DP / 16, XN = BM / 32, STEP = QG * BM, TILE = STEP * DP * 2, BN = KW * 32;
    constexpr bool KLDS = DP > 64;  // k in LDS: with both in registers two waves would not fit a SIMD
    constexpr int KBYTES = KLDS ? BN * DP * 2 : 0;
    char *tiles = smem + KBYTES;
    float *rows_at = reinterpret_cast<float *>(tiles + 4 * TILE);  // [2][nlse, ndelta][STEP]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kw = wave % KW, qg = wave / KW;
    const int heads = p.n * p.hk;
    const int head = block % heads, tile = block / heads;  // the longest of a masked problem first
    const int b = head / p.hk, hk = head % p.hk;
    const AttnSample s = attn_sample(p, b);
    const int j0 = tile * BN, j = j0 + kw * 32 + (lane & 31), last = s.keys - 1, d = p.d;
    const bool alive = j < s.keys;
    // the sequence of steps: the tokens that see the tile's keys, for one query head after the other
    int lo = 0, hi = 0;
    if (j0 <= last) {
        lo = attn_seen_by(p, s, j0).lo & ~(BM - 1);
        hi = attn_seen_by(p, s, j0 + BN - 1 < last ? j0 + BN - 1 : last).hi;
    }
    const int steps = hi > lo ? (hi - lo + STEP - 1) / STEP : 0;
    int first = 0, total = steps * p.group;
    if (p.grad_splits > 1) {
        first = piece * p.grad_pieces;
        if (first >= total && piece) return;  // the join counts the pieces the same way
        total = total < first + p.grad_pieces ? total : first + p.grad_pieces;
    }
    int load_g = steps ? first / steps : 0, load_step = first - load_g * steps;
    int step = load_step;
    if constexpr (KLDS) {
        const AttnTile<DP, BN, 8> tk(p.k + b * p.ks[0] + hk * p.ks[2], p.ks[1], s.keys, d, wave, lane);
        tk.load(smem, j0, wave);
    }
    AttnTile<DP, STEP, 8, true> tq(nullptr, p.qs[1], s.queries, d, wave, lane), tg(nullptr, p.os[1], s.queries, d, wave, lane);
    auto load = [&](int at) {  // the next step of the sequence
        const int h = hk * p.group + load_g, i0 = lo + load_step * STEP;
        char *to = tiles + at * 2 * TILE;
        tq.base = p.q + b * p.qs[0] + h * p.qs[2];
        tg.base = p.dout + b * p.os[0] + h * p.os[2];
        tq.load(to, i0, wave);
        tg.load(to + TILE, i0, wave);
        // a row's two numbers: one row per lane of the first waves
        constexpr int WAVES = STEP / 64;
        if (wave < 2 * WAVES) {
            const int part = wave % WAVES * 64, which = wave / WAVES;
            const float *from = (which ? p.ndelta : p.nlse) + ((int64_t)b * p.hq + h) * p.tq + i0 + part;
            const int left = s.queries - i0 - part;
            const buf_rsrc rs = make_rsrc(from, left > 0 ? (uint32_t)(left < 64 ? left : 64) * 4u : 0u);
#if defined(__HIP_DEVICE_COMPILE__)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(rows_at + (at * 2 + which) * STEP + part), 4, lane * 4,
                                                     0, 0, 0);
#endif
        }
        if (++load_step == steps) {
            load_step = 0;
            ++load_g;
        }
    };
    if (first < total) load(0);
    half8_t k[KLDS ? 1 : KK], v[KK];
    {
        const _Float16 *rk = p.k + b * p.ks[0] + j * p.ks[1] + hk * p.ks[2];
        const _Float16 *rv = p.v + b * p.vs[0] + j * p.vs[1] + hk * p.vs[2];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int e = 16 * kk + 8 * (lane >> 5);
            half8_t z = {};
            if constexpr (!KLDS) k[kk] = alive && e < d ? *reinterpret_cast<const half8_t *>(rk + e) : z;
            v[kk] = alive && e < d ? *reinterpret_cast<const half8_t *>(rv + e) : z;
        }
    }
    // keys past the sample's last take that one's place
    const AttnRange seen = last < 0 ? AttnRange{0, 0} : attn_seen_by(p, s, j < last ? j : last);
    const int wave_lo = __builtin_amdgcn_readfirstlane(seen.lo), wave_hi_all = __builtin_amdgcn_readfirstlane(seen.hi);
    const int wave_lo_all = __builtin_amdgcn_readlane(seen.lo, 31), wave_hi = __builtin_amdgcn_readlane(seen.hi, 31);
    AttnRows<DP> fr;
    AttnCols<DP> fc;
    fr.init(lane);
    fc.init(lane);
    const float c = p.scale * kAttnLog2e;
    f32x16 ak[NT] = {}, av[NT] = {};
    ColumnScale<E> scale;
    int buf = 0;
    for (int n = first; n < total; ++n) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const char *qs = tiles + buf * 2 * TILE + qg * BM * DP * 2, *gs = qs + TILE;
        const float *starts = rows_at + buf * 2 * STEP + qg * BM;
        const int i0 = lo + step * STEP + qg * BM;
        buf ^= 1;
        if (++step == steps) step = 0;
        if (i0 + BM <= wave_lo || i0 >= wave_hi) {
            if (n + 1 < total) load(buf);
            continue;
        }
        const bool edge = i0 < wave_lo_all || i0 + BM > wave_hi_all;
        const uint32_t qr = lds_address(qs) + fr.off;
        const uint32_t kr = opaque(lds_address(smem) + kw * 32 * DP * 2 + fr.off);
        static_for<XN>([&](auto sub) {
            constexpr int T = decltype(sub)::value;
            f32x16 x, y;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const f32x4 sx = *reinterpret_cast<const f32x4 *>(starts + 32 * T + acc_row(e, lane >> 5));
                const f32x4 sy = *reinterpret_cast<const f32x4 *>(starts + STEP + 32 * T + acc_row(e, lane >> 5));
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    x[e + m] = sx[m];
                    y[e + m] = sy[m];
                }
            }
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                if constexpr (KLDS)
                    x = mfma_32x32x16<E>(fr.read(qr, 32 * T, kk), fr.read(kr, 0, kk), x);
                else
                    x = mfma_32x32x16<E>(fr.read(qr, 32 * T, kk), k[kk], x);
                y = mfma_32x32x16<E>(fr.read(qr, STEP + 32 * T, kk), v[kk], y);
            }
            if constexpr (T == 0) {
                if (n + 1 < total) load(buf);  // behind the products, which it then does not hold up
            }
            if (edge) {
                const int from = seen.lo - i0, to = seen.hi - i0;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int m = 32 * T + acc_row(e, lane >> 5);
                    x[e] = m >= from && m < to ? x[e] : -__builtin_inff();
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                x[e] = __builtin_amdgcn_exp2f(kLift<E> == 0.0f ? x[e] * c : fmaf(x[e], c, kLift<E>));
                y[e] *= x[e];
            }
            const half8_t w[2] = {pack8<E>(x, 0), pack8<E>(x, 8)};
            scale.template apply<NT>(y, ak);
            static_for<2>([&](auto half) {
                constexpr int S = decltype(half)::value;
                half8_t f[NT];
                fc.template read<2 * T + S>(gs, f);
#pragma unroll
                for (int t = 0; t < NT; ++t) av[t] = mfma_32x32x16<E>(f[t], w[S], av[t]);
                fc.template read<2 * T + S>(qs, f);
                const half8_t u = pack8<E>(y, S * 8);
#pragma unroll
                for (int t = 0; t < NT; ++t) ak[t] = mfma_32x32x16<E>(f[t], u, ak[t]);
            });
        });
    }
    // without a step, k is still on its way into LDS
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if constexpr (!std::is_same_v<E, __bf16>) acc_scale<NT>(ak, 1.0f / scale.f);
    if constexpr (QG > 1) {
        float *sums = reinterpret_cast<float *>(smem);
        static_for<2>([&](auto w) {
            auto &acc = decltype(w)::value ? av : ak;
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the buffers are free
            if (qg > 0) acc_put<NT>(sums + ((qg - 1) * KW + kw) * NT * 1024, acc, lane);
            __syncthreads();
            if (qg == 0) {
#pragma unroll 1
                for (int o = 0; o < QG - 1; ++o) acc_join<NT>(sums + (o * KW + kw) * NT * 1024, acc, 1.0f, 1.0f, lane);
            }
        });
        if (qg > 0) return;
    }
    if (j >= p.tk) return;
    if (p.grad_splits > 1) {
        const int64_t at = (((int64_t)piece * heads + head) * p.tk + j) * d;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int e0 = 32 * t + acc_row(e, lane >> 5);
                if (e0 < d) {
                    *reinterpret_cast<f32x4 *>(p.part_dk + at + e0) = f32x4{ak[t][e], ak[t][e + 1], ak[t][e + 2], ak[t][e + 3]};
                    *reinterpret_cast<f32x4 *>(p.part_dv + at + e0) = f32x4{av[t][e], av[t][e + 1], av[t][e + 2], av[t][e + 3]};
                }
            }
        return;
    }
    if (!alive) {
#pragma unroll
        for (int t = 0; t < NT; ++t) ak[t] = av[t] = f32x16{};
    }
    if (p.dk) {
        _Float16 *out = p.dk + b * p.ks[0] + j * p.ks[1] + hk * p.ks[2];
#pragma unroll
        for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, ak[t], p.scale * kDrop<E>, d - 32 * t, lane, true);
    }
    if (p.dv) {
        _Float16 *out = p.dv + b * p.vs[0] + j * p.vs[1] + hk * p.vs[2];
#pragma unroll
        for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, av[t], kDrop<E>, d - 32 * t, lane, true);
    }
}
template <typename E, int DP, int KW, int QG, int BM>
__global__ __launch_bounds__(512, 2) void attention_dkv_kernel(AttnParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[dkv_lds<DP, KW, QG, BM>()];
    dkv_tile<E, DP, KW, QG, BM>(p, blockIdx.x, blockIdx.y, smem);
}

// Both in one launch, where neither fills the card: blocks [0, kv_units) dk and dv, piece by piece, the
// others dq, with the rows' numbers from a launch before.  1024 tokens, 8 heads of 128: all gradients 46 -> 35 us.
template <typename E, int DP, int W, int G, int BN, int BM>
__global__ __launch_bounds__(512, 2) void attention_grads_kernel(AttnParams p, int kv_units, int kv_tiles, int q_tiles) {
    constexpr int A = dq_lds<DP, W, G, BN>(), B = dkv_lds<DP, W, G, BM>();
    __shared__ __attribute__((aligned(1024))) char smem[A > B ? A : B];
    const int b = blockIdx.x;
    if (b < kv_units)
        dkv_tile<E, DP, W, G, BM>(p, b % kv_tiles, b / kv_tiles, smem);
    else
        dq_tile<E, DP, W, G, BN, true>(p, b - kv_units, q_tiles, smem);
}

// The pieces of each key's steps added in their order: four elements per lane.
template <typename E>
__global__ __launch_bounds__(256) void attention_dkv_join_kernel(AttnParams p, int tile_keys, int tile_tokens, int align) {
    const int heads = p.n * p.hk, quads = p.d >> 2;
    const int64_t unit = (int64_t)blockIdx.x * 256 + threadIdx.x, keys = (int64_t)heads * p.tk;
    if (unit >= keys * quads) return;
    const int64_t key = unit / quads;
    const int e = (int)(unit - key * quads) * 4, head = (int)(key / p.tk), j = (int)(key - (int64_t)head * p.tk);
    const int b = head / p.hk, hk = head - b * p.hk;
    const AttnSample s = attn_sample(p, b);
    int pieces = 0;  // of this key's tile
    if (j < s.keys) {
        const int j0 = j / tile_keys * tile_keys, jl = j0 + tile_keys - 1;
        const int lo = attn_seen_by(p, s, j0).lo & ~(align - 1), hi = attn_seen_by(p, s, jl < s.keys ? jl : s.keys - 1).hi;
        const int total = hi > lo ? (hi - lo + tile_tokens - 1) / tile_tokens * p.group : 0;
        pieces = (total + p.grad_pieces - 1) / p.grad_pieces;
    }
    f32x4 ak = {}, av = {};
    for (int z = 0; z < pieces; ++z) {
        const int64_t at = (z * keys + key) * p.d + e;
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p.part_dk + at), c = *reinterpret_cast<const f32x4 *>(p.part_dv + at);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            ak[m] += a[m];
            av[m] += c[m];
        }
    }
    half4_t ok, ov;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        ok[m] = from_f32<E>(ak[m] * (p.scale * kDrop<E>));
        ov[m] = from_f32<E>(av[m] * kDrop<E>);
    }
    if (p.dk) *reinterpret_cast<half4_t *>(p.dk + b * p.ks[0] + j * p.ks[1] + hk * p.ks[2] + e) = ok;
    if (p.dv) *reinterpret_cast<half4_t *>(p.dv + b * p.vs[0] + j * p.vs[1] + hk * p.vs[2] + e) = ov;
}

template <typename E, int DP>
static void launch_grad(const AttnParams &p, const AttnGradKinds &k, hipStream_t s) {
    const int heads = p.n * p.hk, rows = attn_tile(k.q).rows, keys = attn_tile(k.kv).rows;
    const int q_tiles = (p.rows + rows - 1) / rows, kv_tiles = heads * ((p.tk + keys - 1) / keys);
    const dim3 block(512);
    const bool kv = p.tk > 0 && (p.dk || p.dv), together = k.together && kv && p.dq && p.tq > 0;
    if (p.tq > 0) {
        AttnParams r = p;
        if (together) r.dq = nullptr;  // the rows' numbers alone
        const dim3 grid((uint32_t)(heads * q_tiles));
        switch (k.q) {
            case kAttn64: attention_dq_kernel<E, DP, 2, 4, 32><<<grid, block, 0, s>>>(r); break;
            case kAttn128: attention_dq_kernel<E, DP, 4, 2, 64><<<grid, block, 0, s>>>(r); break;
            default: attention_dq_kernel<E, DP, 8, 1, 64><<<grid, block, 0, s>>>(r); break;
        }
    }
    if (!kv) return;
    if (together) {
        const int kv_units = kv_tiles * p.grad_splits;
        const dim3 grid((uint32_t)(kv_units + heads * q_tiles));
        if (k.kv == kAttn64)
            attention_grads_kernel<E, DP, 2, 4, 32, 32><<<grid, block, 0, s>>>(p, kv_units, kv_tiles, q_tiles);
        else
            attention_grads_kernel<E, DP, 4, 2, 64, 32><<<grid, block, 0, s>>>(p, kv_units, kv_tiles, q_tiles);
    } else {
        const dim3 grid((uint32_t)kv_tiles, (uint32_t)p.grad_splits);
        switch (k.kv) {
            case kAttn64: attention_dkv_kernel<E, DP, 2, 4, 32><<<grid, block, 0, s>>>(p); break;
            case kAttn128: attention_dkv_kernel<E, DP, 4, 2, 32><<<grid, block, 0, s>>>(p); break;
            default: attention_dkv_kernel<E, DP, 8, 1, 64><<<grid, block, 0, s>>>(p); break;
        }
    }
    if (p.grad_splits > 1) {
        const int64_t count = (int64_t)heads * p.tk * (p.d / 4);
        attention_dkv_join_kernel<E><<<dim3((uint32_t)((count + 255) / 256)), dim3(256), 0, s>>>(
            p, keys, attn_grad_step(k.kv), k.kv == kAttn256 ? 64 : 32);
    }
}

template <typename E>
static void launch_grad_dim(const AttnParams &p, const AttnGradKinds &k, hipStream_t s) {
    if (p.d <= 32)
        launch_grad<E, 32>(p, k, s);
    else if (p.d <= 64)
        launch_grad<E, 64>(p, k, s);
    else if (p.d <= 96)
        launch_grad<E, 96>(p, k, s);
    else
        launch_grad<E, 128>(p, k, s);
}

hipError_t launch_attention_grad(const AttnParams &p, const AttnGradKinds &k, hipStream_t s) {
    if (p.bf16)
        launch_grad_dim<__bf16>(p, k, s);
    else
        launch_grad_dim<_Float16>(p, k, s);
    return hipGetLastError();
}

}  // namespace c3d
