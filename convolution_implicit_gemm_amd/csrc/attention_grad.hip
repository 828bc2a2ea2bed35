// Attention's gradients.  With P = exp(s - lse) computed again from q, k and the
// forward pass's lse, and delta_i = dout_i . o_i:
//   dP_ij = dout_i . v_j,  dS_ij = P_ij (dP_ij - delta_i)
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dout_i
// Two kernels: one holds query rows and runs over the keys (dq), the other holds keys
// and runs over the query rows (dk, dv).  S and dP are computed in both, seven products for
// the five of the formula, so that every sum stays in the registers of one wave: no
// atomics, no partial sums in memory, the same result in every call.
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

// ---- dq: tiles of WAVES x 32 rows as in the forward pass.  S^T = K Q^T and dP^T = V dout^T
// hold one query per lane; dS^T is, as it stands, the operand of dq^T = K^T dS^T.
template <typename E, int DP, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void attention_dq_kernel(AttnParams p) {
    constexpr int BN = kAttnTileKeys, NT = DP / 32, KK = DP / 16, TILE = BN * DP * 2;
    __shared__ __attribute__((aligned(1024))) char smem[4 * TILE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = p.n * p.hk, tiles = (int)gridDim.x / heads;
    const int head = blockIdx.x % heads, tile = tiles - 1 - blockIdx.x / heads;
    const int b = head / p.hk, hk = head % p.hk;
    const AttnSample s = attn_sample(p, b);
    const int r0 = tile * WAVES * 32;
    const int r = r0 + wave * 32 + (lane & 31);
    const int i = r / p.group, g = r - i * p.group, h = hk * p.group + g;
    const bool alive = i < s.queries;
    const int last = s.queries - 1;
    const AttnRange seen = last < 0 ? AttnRange{0, 0} : attn_range(p, s, i < last ? i : last);
    const int t_first = r0 / p.group, t_last = (r0 + WAVES * 32 - 1) / p.group;
    int lo = 0, hi = 0;
    if (t_first <= last) {
        lo = attn_range(p, s, t_first).lo;
        hi = attn_range(p, s, t_last < last ? t_last : last).hi;
    }
    lo &= ~(BN - 1);
    const int wave_lo = __builtin_amdgcn_readfirstlane(seen.lo), wave_hi_all = __builtin_amdgcn_readfirstlane(seen.hi);
    const int wave_lo_all = __builtin_amdgcn_readlane(seen.lo, 31), wave_hi = __builtin_amdgcn_readlane(seen.hi, 31);

    const int d = p.d;
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
                o = *reinterpret_cast<const half8_t *>(p.o + at + e);
            }
            delta += dot8<E>(go[kk], o);
        }
        delta = both_sum(delta);
        const int64_t row = ((int64_t)b * p.hq + h) * p.tq + i;
        if (alive) lse = p.lse[row];
        if (r < p.rows && lane < 32) {
            p.nlse[row] = start_of_scores(lse, p.scale);
            p.ndelta[row] = -delta;
        }
    }
    if (!p.dq) return;  // only the rows' sums were asked for
    const AttnTile<DP, BN, WAVES> tk(p.k + b * p.ks[0] + hk * p.ks[2], p.ks[1], s.keys, d, wave, lane), tv(p.v + b * p.vs[0] + hk * p.vs[2], p.vs[1], s.keys, d, wave, lane);
    AttnRows<DP> fr;
    AttnCols<DP> fc;
    fr.init(lane);
    fc.init(lane);
    const float c = p.scale * kAttnLog2e, lse2 = lse == -__builtin_inff() ? 0.0f : lse * kAttnLog2e;
    f32x16 acc[NT] = {};
    int buf = 0;
    if (lo < hi) {
        tk.load(smem, lo, wave);
        tv.load(smem + TILE, lo, wave);
    }
    for (int j0 = lo; j0 < hi; j0 += BN) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const char *ks = smem + buf * 2 * TILE;
        buf ^= 1;
        if (j0 + BN < hi) {
            char *next = smem + buf * 2 * TILE;
            tk.load(next, j0 + BN, wave);
            tv.load(next + TILE, j0 + BN, wave);
        }
        if (j0 + BN <= wave_lo || j0 >= wave_hi) continue;
        const bool edge = j0 < wave_lo_all || j0 + BN > wave_hi_all;
        const uint32_t kr = lds_address(ks) + fr.off;
        static_for<2>([&](auto sub) {
            constexpr int T = decltype(sub)::value;
            f32x16 x = {}, y;
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = -delta;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                x = mfma_32x32x16<E>(fr.read(kr, 32 * T, kk), q[kk], x);
                y = mfma_32x32x16<E>(fr.read(kr, BN + 32 * T, kk), go[kk], y);
            }
            if (edge) {
                const int from = seen.lo - j0, to = seen.hi - j0;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = 32 * T + acc_row(e, lane >> 5);
                    x[e] = j >= from && j < to ? x[e] : -__builtin_inff();
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(x[e], c, -lse2)) * y[e];
            static_for<2>([&](auto step) {
                constexpr int S = decltype(step)::value;
                half8_t f[NT];
                fc.template read<2 * T + S>(ks, f);
                const half8_t w = pack8<E>(x, S * 8);
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] = mfma_32x32x16<E>(f[t], w, acc[t]);
            });
        });
    }
    if (r >= p.rows) return;
    if (!alive) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x16{};
    }
    _Float16 *out = p.dq + b * p.qs[0] + i * p.qs[1] + h * p.qs[2];
#pragma unroll
    for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, acc[t], p.scale, d - 32 * t, lane, true);
}

// ---- dk, dv: WAVES x 32 keys, wave w holds keys 32 w .. + 31 (one key per lane of every
// result) and all waves share the tile of 64 query tokens in LDS; the query heads of the
// key head are taken one after the other.  S = Q K^T and dP = dout V^T; P and dS are,
// as they stand, the operands of dv^T = dout^T P and dk^T = Q^T dS.
template <typename E, int DP, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void attention_dkv_kernel(AttnParams p) {
    constexpr int BM = 64, NT = DP / 32, KK = DP / 16, TILE = BM * DP * 2, BN = WAVES * 32;
    constexpr bool KLDS = DP > 64;  // k in LDS: with both in registers two waves would not fit a SIMD
    constexpr int KBYTES = KLDS ? BN * DP * 2 : 0;
    __shared__ __attribute__((aligned(1024))) char smem[KBYTES + 4 * TILE + 4 * BM * 4];
    char *tiles = smem + KBYTES;
    float *rows_at = reinterpret_cast<float *>(tiles + 4 * TILE);  // [2][nlse, ndelta][BM]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = p.n * p.hk;
    const int head = blockIdx.x % heads, tile = blockIdx.x / heads;  // the longest of a masked problem first
    const int b = head / p.hk, hk = head % p.hk;
    const AttnSample s = attn_sample(p, b);
    const int j0 = tile * BN, j = j0 + wave * 32 + (lane & 31);
    const bool alive = j < s.keys;
    // the query tokens [lo, hi) that see a key
    auto seen_by = [&](int key) -> AttnRange {
        if (!p.frame) return {0, s.queries};
        const int64_t f = (uint32_t)key / (uint32_t)p.frame;
        const int64_t from = f * p.frame - s.offset;
        const int64_t to = p.window ? (f + p.window) * p.frame - s.offset : (int64_t)s.queries;
        const int64_t q = s.queries;
        const int a = (int)(from < 0 ? 0 : from < q ? from : q), z = (int)(to < 0 ? 0 : to < q ? to : q);
        return {a, z < a ? a : z};
    };
    const int last = s.keys - 1;
    // keys past the sample's last take that one's place
    const AttnRange seen = last < 0 ? AttnRange{0, 0} : seen_by(j < last ? j : last);
    int lo = 0, hi = 0;
    if (j0 <= last) {
        lo = seen_by(j0).lo & ~(BM - 1);
        const int jl = j0 + BN - 1;
        hi = seen_by(jl < last ? jl : last).hi;
    }
    const int wave_lo = __builtin_amdgcn_readfirstlane(seen.lo), wave_hi_all = __builtin_amdgcn_readfirstlane(seen.hi);
    const int wave_lo_all = __builtin_amdgcn_readlane(seen.lo, 31), wave_hi = __builtin_amdgcn_readlane(seen.hi, 31);
    const int d = p.d;
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
    if constexpr (KLDS) {
        const AttnTile<DP, BN, WAVES> tk(p.k + b * p.ks[0] + hk * p.ks[2], p.ks[1], s.keys, d, wave, lane);
        tk.load(smem, j0, wave);
    }
    AttnRows<DP> fr;
    AttnCols<DP> fc;
    fr.init(lane);
    fc.init(lane);
    const float c = p.scale * kAttnLog2e;
    f32x16 ak[NT] = {}, av[NT] = {};
    AttnTile<DP, BM, WAVES> tq(nullptr, p.qs[1], s.queries, d, wave, lane), tg(nullptr, p.os[1], s.queries, d, wave, lane);
    const int steps = hi > lo ? (hi - lo + BM - 1) / BM : 0, total = steps * p.group;
    int load_g = 0, load_step = 0;
    auto load = [&](int at) {  // the next tile of the sequence
        const int h = hk * p.group + load_g, i0 = lo + load_step * BM;
        char *to = tiles + at * 2 * TILE;
        tq.base = p.q + b * p.qs[0] + h * p.qs[2];
        tg.base = p.dout + b * p.os[0] + h * p.os[2];
        tq.load(to, i0, wave);
        tg.load(to + TILE, i0, wave);
        // a row's two numbers: waves 0 and 1, one row per lane
        if (wave < 2) {
            const float *from = (wave ? p.ndelta : p.nlse) + ((int64_t)b * p.hq + h) * p.tq + i0;
            const int left = s.queries - i0;
            const buf_rsrc rs = make_rsrc(from, left > 0 ? (uint32_t)(left < BM ? left : BM) * 4u : 0u);
#if defined(__HIP_DEVICE_COMPILE__)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(rows_at + (at * 2 + wave) * BM), 4, lane * 4, 0, 0, 0);
#endif
        }
        if (++load_step == steps) {
            load_step = 0;
            ++load_g;
        }
    };
    int buf = 0, step = 0;
    if (total) load(0);
    for (int n = 0; n < total; ++n) {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const char *qs = tiles + buf * 2 * TILE, *gs = qs + TILE;
        const float *starts = rows_at + buf * 2 * BM;
        const int i0 = lo + step * BM;
        buf ^= 1;
        if (++step == steps) step = 0;
        if (n + 1 < total) load(buf);
        if (i0 + BM <= wave_lo || i0 >= wave_hi) continue;
        const bool edge = i0 < wave_lo_all || i0 + BM > wave_hi_all;
        const uint32_t qr = lds_address(qs) + fr.off;
        const uint32_t kr = opaque(lds_address(smem) + wave * 32 * DP * 2 + fr.off);
        static_for<2>([&](auto sub) {
            constexpr int T = decltype(sub)::value;
            f32x16 x, y;
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const f32x4 sx = *reinterpret_cast<const f32x4 *>(starts + 32 * T + acc_row(e, lane >> 5));
                const f32x4 sy = *reinterpret_cast<const f32x4 *>(starts + BM + 32 * T + acc_row(e, lane >> 5));
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
                y = mfma_32x32x16<E>(fr.read(qr, BM + 32 * T, kk), v[kk], y);
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
                x[e] = __builtin_amdgcn_exp2f(x[e] * c);
                y[e] *= x[e];
            }
            static_for<2>([&](auto half) {
                constexpr int S = decltype(half)::value;
                half8_t f[NT];
                fc.template read<2 * T + S>(gs, f);
                const half8_t w = pack8<E>(x, S * 8);
#pragma unroll
                for (int t = 0; t < NT; ++t) av[t] = mfma_32x32x16<E>(f[t], w, av[t]);
                fc.template read<2 * T + S>(qs, f);
                const half8_t u = pack8<E>(y, S * 8);
#pragma unroll
                for (int t = 0; t < NT; ++t) ak[t] = mfma_32x32x16<E>(f[t], u, ak[t]);
            });
        });
    }
    if (j >= p.tk) return;
    if (!alive) {
#pragma unroll
        for (int t = 0; t < NT; ++t) ak[t] = av[t] = f32x16{};
    }
    if (p.dk) {
        _Float16 *out = p.dk + b * p.ks[0] + j * p.ks[1] + hk * p.ks[2];
#pragma unroll
        for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, ak[t], p.scale, d - 32 * t, lane, true);
    }
    if (p.dv) {
        _Float16 *out = p.dv + b * p.vs[0] + j * p.vs[1] + hk * p.vs[2];
#pragma unroll
        for (int t = 0; t < NT; ++t) store_column<E>(out + 32 * t, av[t], 1.0f, d - 32 * t, lane, true);
    }
}

template <typename E, int DP>
static void launch_grad(const AttnParams &p, hipStream_t s) {
    const int heads = p.n * p.hk;
    if (p.tq > 0) {
        const int tiles = (p.rows + kAttnTileRows - 1) / kAttnTileRows;
        attention_dq_kernel<E, DP, kAttnTileRows / 32><<<dim3(heads * tiles), dim3(kAttnTileRows * 2), 0, s>>>(p);
    }
    if (p.tk > 0 && (p.dk || p.dv))
        attention_dkv_kernel<E, DP, 8><<<dim3(heads * ((p.tk + 255) / 256)), dim3(512), 0, s>>>(p);
}

template <typename E>
static void launch_grad_dim(const AttnParams &p, hipStream_t s) {
    if (p.d <= 32)
        launch_grad<E, 32>(p, s);
    else if (p.d <= 64)
        launch_grad<E, 64>(p, s);
    else if (p.d <= 96)
        launch_grad<E, 96>(p, s);
    else
        launch_grad<E, 128>(p, s);
}

hipError_t launch_attention_grad(const AttnParams &p, hipStream_t s) {
    if (p.bf16)
        launch_grad_dim<__bf16>(p, s);
    else
        launch_grad_dim<_Float16>(p, s);
    return hipGetLastError();
}

}  // namespace c3d
