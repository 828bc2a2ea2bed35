// The matrix product behind `linear` and its gradients, for gfx950.
//
//   forward  y  = act(x w^T + bias) + residual     columns: w  [n][k], rows: x  [m][k]
//   dx       dx = dz w                             columns: w^T,       rows: dz [m][n]
//   dw       dw = dz^T x                           columns: x^T,       rows: dz^T
//
// One kernel template serves all three: each operand tile is staged through
// LDS in the order it is stored in, and the operands whose contraction is not
// contiguous are read back through the transposing LDS read, so that no
// transposed copy of a tensor is ever made.
//
// The MFMA's A operand is the output's columns, so a lane's accumulators hold 4
// adjacent columns of one row.  Sums are fp32; y and z are rounded once.
#include "column_sum.h"
#include "gemm_common.h"

namespace c3d {

namespace {

// Work unit number b of the launch.  Workgroups are dealt to the XCDs in turn;
// the whole tiles and the pieces are each dealt out in contiguous ranges per XCD.
__device__ __forceinline__ void gemm_my_unit(const GemmParams &p, int b, int &m_tile, int &n_tile, int &it0, int &it1,
                                             int &slot) {
    const int u = b < p.dp_tiles ? xcd_range(b, p.dp_tiles)
                                 : p.dp_tiles + xcd_range(b - p.dp_tiles, p.sk_tiles * p.sk_pieces);
    gemm_unit(p, u, m_tile, n_tile, it0, it1, slot);
}

// ---- ring kernel: KG groups of 4 waves, each with a ring of NS stages, one
// barrier per stage.  The groups take the tile's stages in turn (a long
// contraction over few tiles then needs no second launch to join its pieces);
// their sums meet in LDS, in group order.  Bound by what L2 delivers: 16 to 20
// TB/s over the card, so the tile is the largest that still fills it.  Forward,
// bf16: 64 x 64 tiles 613 x 2048 x 2048 14 us; 128 x 128 with two groups 2048^3
// 23.5 us (730 TFLOP/s; one group 26.7); 64 x 64 with four 64 x 2048 x 2048 8.6 us.
template <int BM_, int BN_, int WM_, int WN_, int NS_, int KG_>
struct RingTile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_, KG = KG_;
    static constexpr int THREADS = 256 * KG, STAGE = (BM + BN) * kGemmRow, LDS = KG * NS * STAGE;
    static_assert((BM / WM) * (BN / WN) == 4, "4 waves per group");
    static_assert(LDS >= BM * BN * 2 && LDS >= (KG - 1) * BM * BN * 4 && LDS <= 160 * 1024, "epilogue, sums, LDS");
};
using Ring128 = RingTile<128, 128, 64, 64, 2, 1>;
using Ring64 = RingTile<64, 64, 32, 32, 4, 1>;
using Ring64G4 = RingTile<64, 64, 32, 32, 2, 4>;
using Ring128G2 = RingTile<128, 128, 64, 64, 2, 2>;

// Work unit b of one product.
template <typename E, bool PT, bool QT, typename T>
__device__ __forceinline__ void gemm_ring_unit(const GemmParams &p, int b, char *smem) {
    constexpr int BM = T::BM, BN = T::BN, WM = T::WM, WN = T::WN, NS = T::NS, KG = T::KG;
    constexpr int TN = WN / 32, TM = WM / 32, WAVES = 4;
    constexpr int PB = BN * kGemmRow, QB = BM * kGemmRow, STAGE = PB + QB;
    constexpr int NP = PB / 1024 / WAVES, NQ = QB / 1024 / WAVES;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3;
    const int kg = KG > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) : 0;
    const int wmi = wave / (BN / WN), wni = wave % (BN / WN);
    int mt, nt, it0, it1, slot;
    gemm_my_unit(p, b, mt, nt, it0, it1, slot);
    const int m0 = mt * BM, n0 = nt * BN;
    const int kend = it1 * kGemmBK < p.K ? it1 * kGemmBK : p.K;
    char *ring = smem + kg * NS * STAGE;

    Operand<PT, BN, NP> op;
    Operand<QT, BM, NQ> oq;
    op.init(p.p, p.p_stride, n0, p.N, (it0 + kg) * kGemmBK, kend, wave, WAVES, lane);
    oq.init(p.q, p.q_stride, m0, p.M, (it0 + kg) * kGemmBK, kend, wave, WAVES, lane);
    int wbuf = 0;
    auto fire = [&]() {
        char *s = ring + wbuf * STAGE;
        op.template load<KG>(s, wave, WAVES);
        oq.template load<KG>(s + PB, wave, WAVES);
        wbuf = wbuf + 1 == NS ? 0 : wbuf + 1;
    };
    Fragments<PT, BN, TN> fp;
    Fragments<QT, BM, TM> fq;
    fp.init(wni * WN, lane);
    fq.init(wmi * WM, lane);

    // stages past the end load zeros (their reads are out of range), so that
    // every wave's load count stays the same
    f32x16 acc[TN][TM];
    gemm_init_acc<E, WM, WN>(p, acc, slot < 0 && kg == 0 && p.bias, n0 + wni * WN, lane);
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) fire();
    int rbuf = 0;
    for (int it = it0; it < it1; it += KG) {
        gemm_wait_loads<(NS - 2) * (NP + NQ)>();
        gemm_barrier();  // the stage has landed, and everyone is done with the one before it
        fire();
        const char *s = ring + rbuf * STAGE;
        static_for<2>([&](auto hc) {
            constexpr int KK0 = 2 * decltype(hc)::value;
            half8_t a[2][TN], bq[2][TM];
            fp.template read<KK0>(s, a);
            fq.template read<KK0>(s + PB, bq);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int j = 0; j < TM; ++j) acc[i][j] = mfma_32x32x16<E>(a[kk][i], bq[kk][j], acc[i][j]);
        });
        rbuf = rbuf + 1 == NS ? 0 : rbuf + 1;
    }
    gemm_wait_loads<0>();
    if constexpr (KG > 1) {
        gemm_barrier();
        constexpr int QUADS = BM * BN / 4;
        f32x4 *sums = reinterpret_cast<f32x4 *>(smem);
        auto at = [&](int g, int i, int j, int q) -> f32x4 & {
            return sums[(g - 1) * QUADS + (((wave * TN + i) * TM + j) * 4 + q) * 64 + lane];
        };
        if (kg)
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f32x4 v;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
                        at(kg, i, j, q) = v;
                    }
        gemm_barrier();
        if (kg) return;  // a wave that has ended counts as arrived at later barriers
#pragma unroll
        for (int g = 1; g < KG; ++g)
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x4 v = at(g, i, j, q);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += v[e];
                    }
    }
    if (slot >= 0) {
        gemm_store_partial<BM, BN, WM, WN>(p, acc, slot, wave, lane);
        return;
    }
    gemm_barrier();
    gemm_store_tile<E, BM, BN, WM, WN, 256>(p, acc, smem, m0, n0, wmi, wni, lane);
}

template <typename E, bool PT, bool QT, typename T>
__global__ __launch_bounds__(T::THREADS) void gemm_ring_kernel(GemmParams p) {
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
    gemm_ring_unit<E, PT, QT, T>(p, blockIdx.x, smem);
}

// Both gradients' products and the columns' sums behind dbias in one launch:
// blocks [0, x_units) dx, [x_units, x_units + w_units) dw, then the sums.  Where
// neither product fills the card they share it, and a small backward pass is
// three launches, two without an activation.  4097 x 2048 x 512 with its activation
// 44 us, dx and dw in launches of their own 54; 2048^3 without one 40 and 56.
template <typename E, typename T>
__global__ __launch_bounds__(T::THREADS) void gemm_pair_kernel(GemmParams px, GemmParams pw, ColumnSumParams cs,
                                                               int x_units, int w_units) {
    __shared__ __attribute__((aligned(1024))) char smem[T::LDS];
    const int b = blockIdx.x;
    if (b < x_units)
        gemm_ring_unit<E, true, false, T>(px, b, smem);
    else if (b < x_units + w_units)
        gemm_ring_unit<E, true, true, T>(pw, b - x_units, smem);
    else
        column_sum_block<E, T::THREADS>(cs, b - x_units - w_units, reinterpret_cast<float *>(smem));
}

// ---- ping-pong kernel: 8 waves in two groups of 4, one wave of each on every
// SIMD (waves w and w + 4 share one).  Group g owns half of the tile's columns
// and alternates between a memory phase (the MFMA fragments of two k-steps from
// LDS into registers, its share of the loads of a later stage) and a compute
// phase (those MFMAs, at raised priority); the groups run one phase apart with
// one workgroup barrier per phase, so that each SIMD's matrix core is fed by
// one wave while the other reads LDS.
//
// Stage s (64 of the contraction) is read by group g in phases 4s + g (k-steps
// 0-1) and 4s + 2 + g (k-steps 2-3).  LDS is a ring of five operand buffers
// that hold, in turn, p(0), q(0), p(1), q(1), ...: while stage s is computed
// the two buffers of stage s - 1 are refilled, with q(s + 1) from the first
// memory phase and p(s + 2) from the second, so that a load has at least two
// and a half phases (p: six) to land.  All but p(s + 2) have to have landed
// before phase 4s + 4: both groups wait for their own in phase 4s + 3.
//
// A workgroup runs work units until none is left (one workgroup per CU), and
// the ring runs on across them: the last stages of a unit load the first of the
// next.  At its end the two buffers of the last stage are free and serve the
// epilogue, 8 KiB per wave, so that its stores drain under the next unit's
// stages (2 to 3% less time than one workgroup per unit).  Bound by power: the
// matrix cores are busy 80% of the cycles on dw and 71% with a contraction of
// 2048, an activation and 600 MB of output, at the clock that leaves.  In TFLOP/s:
// 8192^3 bf16 1320-1400 forward, 1375 dx and dw, fp16 1290, 1270 and 1280; 36864 x
// 8192 x 2048 bf16 1310 (945 us), 1345 and 1390, fp16 1235, 1250 and 1310; with bf16
// tanh GELU 1000-1030 us.
template <typename E, bool PT, bool QT>
__global__ __launch_bounds__(512) void gemm_pp_kernel(GemmParams p0) {
    constexpr int BM = 256, BN = 256, WM = BM / 4, WN = BN / 2, TN = WN / 32, TM = WM / 32, WAVES = 8;
    constexpr int BUF = BN * kGemmRow, NP = BUF / 1024 / WAVES, NQ = NP;
    __shared__ __attribute__((aligned(1024))) char smem[5 * BUF];
    static_assert(sizeof(smem) <= 160 * 1024, "LDS is 160 KiB per CU");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = wave >> 2, wmi = wave & 3, wni = grp;
    // The lane and the parameters as the compiler cannot see through them: what
    // the once-per-unit code needs is worked out and read again there instead of
    // being kept in registers (and spilled) across the loop over stages.
    auto opaque_lane = [&]() {
        int l = lane;
#if defined(__HIP_DEVICE_COMPILE__)
        asm volatile("" : "+v"(l));
#endif
        return l;
    };
#if defined(__HIP_DEVICE_COMPILE__)
    const uint64_t kaddr = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
#endif
    auto params = [&]() -> GemmParams {
#if defined(__HIP_DEVICE_COMPILE__)
        uint64_t ka = kaddr;
        asm volatile("" : "+s"(ka));
        return *reinterpret_cast<const GemmParams __attribute__((address_space(4))) *>(ka);
#else
        return p0;
#endif
    };
    struct Unit {
        int mt, nt, it0, it1, slot;
    };
    auto unit_of = [&](const GemmParams &p, int u) {
        Unit r;
        gemm_my_unit(p, u, r.mt, r.nt, r.it0, r.it1, r.slot);
        return r;
    };

    Operand<PT, BN, NP> op;
    Operand<QT, BM, NQ> oq;
    auto aim_p = [&](const GemmParams &p, const Unit &u) {
        const int kend = u.it1 * kGemmBK < p.K ? u.it1 * kGemmBK : p.K;
        op.init(p.p, p.p_stride, u.nt * BN, p.N, u.it0 * kGemmBK, kend, wave, WAVES, opaque_lane());
    };
    auto aim_q = [&](const GemmParams &p, const Unit &u) {
        const int kend = u.it1 * kGemmBK < p.K ? u.it1 * kGemmBK : p.K;
        oq.init(p.q, p.q_stride, u.mt * BM, p.M, u.it0 * kGemmBK, kend, wave, WAVES, opaque_lane());
    };
    Fragments<PT, BN, TN> fp;
    Fragments<QT, BM, TM> fq;
    fp.init(wni * WN, lane);
    fq.init(wmi * WM, lane);

    int u = blockIdx.x;
    Unit cur, next;
    {
        const GemmParams p = params();
        cur = unit_of(p, u);
        aim_p(p, cur);
        aim_q(p, cur);
    }
    op.template load<1>(smem, wave, WAVES);
    oq.template load<1>(smem + BUF, wave, WAVES);
    op.template load<1>(smem + 2 * BUF, wave, WAVES);
    gemm_wait_loads<NP>();
    gemm_barrier();
    int pbuf = 0;  // p(s); q(s) and the refills follow it in the ring
    auto ring = [&](int d) {
        const int i = pbuf + d;
        return smem + (i >= 5 ? i - 5 : i) * BUF;
    };
    for (;;) {
        f32x16 acc[TN][TM] = {};
        _Float16 bias[TN];
        half8_t a[2][TN], bq[2][TM];
        auto compute = [&]() {
            __builtin_amdgcn_s_setprio(2);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int j = 0; j < TM; ++j) acc[i][j] = mfma_32x32x16<E>(a[kk][i], bq[kk][j], acc[i][j]);
            __builtin_amdgcn_s_setprio(0);
        };
        auto stage = [&](auto lastc) {
            constexpr bool LAST = decltype(lastc)::value;
            const char *ps = ring(0), *qs = ring(1);
            auto memory = [&](auto hc) {
                constexpr int H = decltype(hc)::value;
                auto refill = [&]() {
                    if constexpr (H == 0)
                        oq.template load<1>(ring(3), wave, WAVES);
                    else
                        op.template load<1>(ring(4), wave, WAVES);
                };
                // the bias goes ahead of the stage's loads, so that the wait
                // for those covers it
                if constexpr (LAST && H == 0) {
                    const GemmParams p = params();
                    const bool has = cur.slot < 0 && p.bias != nullptr;
                    const buf_rsrc rb = make_rsrc(has ? p.bias : p.p, has ? (uint32_t)p.N * 2u : 0u);
                    const int l = opaque_lane(), co = cur.nt * BN + wni * WN + l;
#pragma unroll
                    for (int i = 0; i < TN; ++i)
                        bias[i] = load2(rb, l < 32 && co + i * 32 < p.N ? (uint32_t)(co + i * 32) * 2u : kOOB);
                }
                if constexpr (PT || QT) refill();  // the transposing reads wait for themselves
                fq.template read<2 * H>(qs, bq);
                fp.template read<2 * H>(ps, a);
                if constexpr (!PT && !QT) refill();
            };
            memory(std::integral_constant<int, 0>{});
            gemm_barrier();
            compute();
            gemm_barrier();
            memory(std::integral_constant<int, 1>{});
            if (grp) gemm_wait_loads<NP>();
            gemm_barrier();
            compute();
            if (!grp) gemm_wait_loads<NP>();
            if (!(LAST && grp)) gemm_barrier();  // group 1's last would pair with nothing
            if constexpr (!LAST) pbuf = pbuf + 2 >= 5 ? pbuf - 3 : pbuf + 2;
        };
        if (grp) gemm_barrier();  // group 1 runs one phase behind
        for (int it = cur.it0; it + 2 < cur.it1; ++it) stage(std::false_type{});
        // two stages are left (there are at least two): p is loaded to its end
        // and goes on to the next unit, then q; without one, both load zeros, so
        // that every wave's load count stays the same
        u += gridDim.x;
        bool more;
        {
            const GemmParams p = params();
            more = u < p.dp_tiles + p.sk_tiles * p.sk_pieces;
            if (more) {
                next = unit_of(p, u);
                aim_p(p, next);
            } else {
                op.left = 0;
            }
        }
        stage(std::false_type{});
        if (more)
            aim_q(params(), next);
        else
            oq.left = 0;
        stage(std::true_type{});
        __builtin_amdgcn_sched_barrier(0);
        // the bias is one more step of the contraction, times one: exact, and 8
        // MFMAs instead of 192 vector instructions
        half8_t one = {};
        one[0] = opaque_lane() < 32 ? from_f32<E>(1.0f) : (_Float16)0.0f;
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            half8_t b = {};
            b[0] = bias[i];
#pragma unroll
            for (int j = 0; j < TM; ++j) acc[i][j] = mfma_32x32x16<E>(b, one, acc[i][j]);
        }
        __builtin_amdgcn_sched_barrier(0);
        // every wave is past its reads of the last stage (group 0 passed the
        // barrier after them, group 1 made them)
        {
            const GemmParams p = params();
            const int m0 = cur.mt * BM + wmi * WM, n0 = cur.nt * BN + wni * WN;  // this wave's part
            if (cur.slot >= 0)
                gemm_store_partial<BM, BN, WM, WN>(p, acc, cur.slot, wmi * 2 + wni, opaque_lane());
            else
                gemm_store_wave<E>(p, acc, ring(grp) + wmi * 8192, m0, n0, p.M - m0 < WM ? p.M - m0 : WM,
                                   p.N - n0 < WN ? p.N - n0 : WN, opaque_lane());
        }
        if (!more) break;
        pbuf = pbuf + 2 >= 5 ? pbuf - 3 : pbuf + 2;
        cur = next;
        gemm_barrier();  // the epilogue's buffers are free again
    }
    gemm_wait_loads<0>();
}

// ---- few rows (m <= 16): the product is the stream of w from HBM.  A block
// takes 16 columns and splits the contraction over its WAVES waves; every lane
// reads w's rows straight into the MFMA's A fragment (16x16x32: 16 columns, 64
// contiguous bytes of each), several in flight, and the rows of x (which stay
// in cache) into B.  The waves' sums meet in LDS, in wave order; one wave runs the
// epilogue.  No LDS staging, no second launch.  Launches one after the other, w from
// the caches and from HBM: 1 x 4096 x 1024 3.2 and 4.4 us, of which the launch is
// about 2 (64 x 64 tiles 6.3 and 7.4).  A CU draws 32 bytes a nanosecond this way,
// whatever its waves (4, 8 and 16 measured level), so few columns of a long
// contraction go to the tiles that split it: 512 x 8192 8.7 and 10.4 us, here 10.4
// and 11.5.
template <typename E>
__device__ __forceinline__ f32x4 mfma_16x16x32(half8_t a, half8_t b, f32x4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (std::is_same_v<E, __bf16>)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                       c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
#else
    (void)a;
    (void)b;
    return c;
#endif
}

// The epilogue of 4 adjacent columns of one row (v: the full sums, without bias).
template <typename E>
__device__ __forceinline__ void gemm_finish_quad(const GemmParams &p, f32x4 v, int m, int n) {
    if (p.bias) {
        const half4_t bv = *reinterpret_cast<const half4_t *>(p.bias + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += to_f32<E>(bv[e]);
    }
    half4_t h;
    if (p.z) {
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = from_f32<E>(v[e]);
        *reinterpret_cast<half4_t *>(p.z + (int64_t)m * p.N + n) = h;
    }
    act_switch(p.act, [&](auto ac) {
        constexpr int ACT = decltype(ac)::value;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_f<ACT>(v[e]);
    });
    if (p.res) {
        const half4_t rv = *reinterpret_cast<const half4_t *>(p.res + (int64_t)m * p.res_stride + n);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += to_f32<E>(rv[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = from_f32<E>(v[e]);
    *reinterpret_cast<half4_t *>(p.y + (int64_t)m * p.y_stride + n) = h;
}

constexpr int kRowsWaves = 8, kRowsAhead = 8;
template <typename E>
__global__ __launch_bounds__(kRowsWaves * 64) void gemm_rows_kernel(GemmParams p) {
    __shared__ f32x4 sums[kRowsWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, kq = (lane >> 4) * 8;
    const int n0 = blockIdx.x * 16;
    // columns and rows past the end read the last one; their sums are dropped
    const int nr = n0 + r16 < p.N ? n0 + r16 : p.N - 1, mr = r16 < p.M ? r16 : p.M - 1;
    const _Float16 *wp = p.p + (int64_t)nr * p.p_stride + kq;
    const _Float16 *xp = p.q + (int64_t)mr * p.q_stride + kq;
    // this wave's steps of 32
    const int steps = (p.K + 31) / 32;
    const int s0 = steps * wave / kRowsWaves, s1 = steps * (wave + 1) / kRowsWaves;
    f32x4 acc = {};
    for (int s = s0; s < s1; s += kRowsAhead) {
        half8_t a[kRowsAhead], b[kRowsAhead];
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) {
            const int k = (s + u) * 32;
            const bool in = s + u < s1 && k + kq < p.K;
            a[u] = in ? *reinterpret_cast<const half8_t *>(wp + k) : half8_t{};
            b[u] = in ? *reinterpret_cast<const half8_t *>(xp + k) : half8_t{};
        }
#pragma unroll
        for (int u = 0; u < kRowsAhead; ++u) acc = mfma_16x16x32<E>(a[u], b[u], acc);
    }
    sums[wave][lane] = acc;
    __syncthreads();
    const int n = n0 + 4 * (lane >> 4);
    if (wave != 0 || r16 >= p.M || n >= p.N) return;
#pragma unroll
    for (int i = 1; i < kRowsWaves; ++i) acc += sums[i][lane];
    gemm_finish_quad<E>(p, acc, r16, n);
}

// ---- the pieces of the split tiles, added in order, then the epilogue.  One
// thread per 4 adjacent columns; blocks of the tile's fragment order.  A stream
// over the fp32 partials: 128 tiles of 256 x 256 in 2 pieces (67 MB) 15 us, 4.4 TB/s.
template <typename E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void gemm_join_block(const GemmParams &p, int b) {
    constexpr int TN = WN / 32, TM = WM / 32, QUADS = BM * BN / 4;
    const int st = b / (QUADS / 256), qd = b % (QUADS / 256) * 256 + threadIdx.x;
    int mt, nt, it0, it1, slot;
    gemm_unit(p, p.dp_tiles + st, mt, nt, it0, it1, slot);
    const int lane = qd & 63;
    int r = qd >> 6;
    const int g = r & 3;
    r >>= 2;
    const int j = r % TM;
    r /= TM;
    const int i = r % TN, wave = r / TN;
    const int wmi = wave / (BN / WN), wni = wave % (BN / WN);
    const int m = mt * BM + wmi * WM + j * 32 + (lane & 31);
    const int n = nt * BN + wni * WN + i * 32 + 8 * g + 4 * (lane >> 5);
    if (m >= p.M || n >= p.N) return;
    const f32x4 *pp = reinterpret_cast<const f32x4 *>(p.partial) + (size_t)st * QUADS + qd;
    const size_t piece = (size_t)p.sk_tiles * QUADS;
    f32x4 v = pp[0];
#pragma unroll 8
    for (int k = 1; k < p.sk_pieces; ++k) v += pp[k * piece];
    gemm_finish_quad<E>(p, v, m, n);
}

// Blocks [0, x_blocks) join the first product's tiles, the others the second's.
template <typename E, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmParams p, GemmParams p2, int x_blocks) {
    const int b = blockIdx.x;
    if (b < x_blocks)
        gemm_join_block<E, BM, BN, WM, WN>(p, b);
    else
        gemm_join_block<E, BM, BN, WM, WN>(p2, b - x_blocks);
}

// ---- dz = dy act'(z) and its column sums.  A block walks a strip of rows for
// 256 groups of 8 columns (or, where there are fewer, several rows at once) and
// writes the strip's fp32 sums, of dz before its rounding.  A separate pass, because
// both products read dz (dx every column panel, dw every row panel, through loads
// that go straight to LDS).  A stream: 36864 x 8192 bf16 360 us, 5.0 TB/s; 4097 x 2048
// fp16 13 us, half of it the activation's arithmetic.
//
// dz is rounded once to the element type, as the matrix cores' operand.  Its
// rounding error adds to that of rounding dx and dw themselves, in their L2 norms
// 2.08e-4 -> 2.93e-4 in fp16 and 1.66e-3 -> 2.35e-3 in bf16 (against 64-bit products of
// the rounded dz the error is the results' rounding alone).  The matrix cores have
// no product of a wider operand with a 16-bit one: to keep what the rounding drops,
// dz would have to go in as two 16-bit terms, which doubles both products, 1.8 of the
// 2.2 ms that the gradients of 36864 x 8192 x 2048 take.
template <typename E, int ACT, bool DZ>
__global__ __launch_bounds__(256) void act_grad_kernel(ActGradParams p, int groups, int rows_at_once) {
    __shared__ float s[256 * 8];
    const int gl = threadIdx.x % groups, rl = threadIdx.x / groups;
    const int c = (blockIdx.x * groups + gl) * 8;
    float sum[8] = {};
    if (rl < rows_at_once && c < p.n) {
        const int64_t r0 = p.m * blockIdx.y / p.strips, r1 = p.m * (blockIdx.y + 1) / p.strips;
#pragma unroll 4
        for (int64_t r = r0 + rl; r < r1; r += rows_at_once) {
            const half8_t d = *reinterpret_cast<const half8_t *>(p.dy + r * p.dy_stride + c);
            half8_t o;
            if constexpr (DZ) {
                const half8_t zv = *reinterpret_cast<const half8_t *>(p.z + r * p.n + c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float v = to_f32<E>(d[e]) * act_slope<ACT>(to_f32<E>(zv[e]));
                    sum[e] += v;
                    o[e] = from_f32<E>(v);
                }
                *reinterpret_cast<half8_t *>(p.dz + r * p.n + c) = o;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += to_f32<E>(d[e]);
            }
        }
    }
    if (!p.colpart) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[threadIdx.x * 8 + e] = sum[e];
    __syncthreads();
    for (int i = threadIdx.x; i < groups * 8; i += 256) {
        const int col = blockIdx.x * groups * 8 + i;
        if (col >= p.n) break;
        float t = 0.0f;
        for (int q = 0; q < rows_at_once; ++q) t += s[q * groups * 8 + i];
        p.colpart[(int64_t)blockIdx.y * p.n + col] = t;
    }
}

// The cost model, in microseconds and for each layout: a step (a stage of 64 per
// group of waves) with few workgroups on the card and operands in L2, a step with
// per_cu workgroups on every CU, the share that operands outside the L2s add to
// the first, what the launch costs, and what each round of workgroups adds
// before and after its steps.  Fitted to the times of 4500 products of 300 random
// sizes (1..36864 rows, 64..8192 columns) with each kernel in turn: within 10%
// rms, and on 150 other sizes the kernel it picks takes 1.1% longer than the
// fastest on average, 10% at the 95th percentile.
const GemmTile kTiles[] = {
    {"m256n256k64", 256, 256, kGemmBK, 512, 1, 1, {0.53, 0.61, 0.77}, {1.59, 1.62, 1.30}, 1.0, 0.0, 6.9},
    {"m128n128k64", 128, 128, kGemmBK, 256, 2, 1, {0.41, 0.47, 0.52}, {1.27, 1.16, 1.19}, 0.65, 1.5, 2.8},
    {"m64n64k64", 64, 64, kGemmBK, 256, 2, 1, {0.16, 0.21, 0.23}, {0.47, 0.49, 0.56}, 1.2, 2.1, 1.7},
    {"m64n64k64g4", 64, 64, kGemmBK, 1024, 1, 4, {0.49, 0.54, 0.69}, {1.05, 1.21, 1.31}, 0.95, 2.3, 2.3},
    {"m128n128k64g2", 128, 128, kGemmBK, 512, 1, 2, {0.69, 0.80, 0.84}, {1.34, 1.30, 1.24}, 0.33, 1.7, 3.4},
    {"m16n16k32", 16, 16, 32, kRowsWaves * 64, 4, 1, {}, {}, 0.0, 0.0, 0.0},  // few rows: rows_us
};

unsigned units_of(const GemmParams &p) { return (unsigned)(p.dp_tiles + p.sk_tiles * p.sk_pieces); }

unsigned join_blocks(const GemmParams &p, int tile) {
    return (unsigned)((int64_t)p.sk_tiles * (kTiles[tile].bm * kTiles[tile].bn / 4) / 256);
}

// The split tiles of p (and of p2, or null).
template <typename E>
hipError_t launch_join(const GemmParams &p, const GemmParams *p2, int tile, hipStream_t s) {
    const unsigned jx = join_blocks(p, tile), jw = p2 ? join_blocks(*p2, tile) : 0;
    if (jx + jw == 0) return hipSuccess;
    const GemmParams &q = p2 ? *p2 : p;
    const dim3 grid(jx + jw);
    const auto go = [&](auto *kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p, q, (int)jx); };
    switch (tile) {
        case 0: go(gemm_join_kernel<E, 256, 256, 64, 128>); break;
        case 1:
        case 4: go(gemm_join_kernel<E, 128, 128, 64, 64>); break;
        default: go(gemm_join_kernel<E, 64, 64, 32, 32>); break;
    }
    return hipGetLastError();
}

template <typename E, bool PT, bool QT>
hipError_t launch_tile(const GemmParams &p, int tile, hipStream_t s) {
    const dim3 grid(units_of(p)), block((unsigned)kTiles[tile].threads);
    switch (tile) {
        case 0: {
            GemmParams q = p;
            if (q.niter < 2) q.niter = 2;  // a stage past the contraction's end is one of zeros
            const dim3 cus(grid.x < (unsigned)kGemmCUs ? grid.x : (unsigned)kGemmCUs);
            hipLaunchKernelGGL((gemm_pp_kernel<E, PT, QT>), cus, block, 0, s, q);
            break;
        }
        case 1: hipLaunchKernelGGL((gemm_ring_kernel<E, PT, QT, Ring128>), grid, block, 0, s, p); break;
        case 2: hipLaunchKernelGGL((gemm_ring_kernel<E, PT, QT, Ring64>), grid, block, 0, s, p); break;
        case 3: hipLaunchKernelGGL((gemm_ring_kernel<E, PT, QT, Ring64G4>), grid, block, 0, s, p); break;
        default: hipLaunchKernelGGL((gemm_ring_kernel<E, PT, QT, Ring128G2>), grid, block, 0, s, p); break;
    }
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_join<E>(p, nullptr, tile, s);
}

template <typename E>
hipError_t launch_pair(const GemmParams &px, const GemmParams &pw, int tile, const ColumnSumParams &cs,
                       hipStream_t s) {
    const int xu = (int)units_of(px), wu = (int)units_of(pw);
    const dim3 grid((unsigned)(xu + wu + (cs.out0 ? (cs.cols + 15) / 16 : 0))), block((unsigned)kTiles[tile].threads);
    switch (tile) {
        case 1: hipLaunchKernelGGL((gemm_pair_kernel<E, Ring128>), grid, block, 0, s, px, pw, cs, xu, wu); break;
        case 2: hipLaunchKernelGGL((gemm_pair_kernel<E, Ring64>), grid, block, 0, s, px, pw, cs, xu, wu); break;
        case 3: hipLaunchKernelGGL((gemm_pair_kernel<E, Ring64G4>), grid, block, 0, s, px, pw, cs, xu, wu); break;
        default: return hipErrorInvalidValue;
    }
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : launch_join<E>(px, &pw, tile, s);
}

}  // namespace

const GemmTile *gemm_tiles(int *count) {
    *count = (int)(sizeof(kTiles) / sizeof(kTiles[0]));
    return kTiles;
}

hipError_t launch_gemm(const GemmParams &p, int tile, GemmLayout layout, hipStream_t s) {
    if (tile == kGemmRowsTile) {
        const dim3 grid((unsigned)((p.N + 15) / 16));
        if (p.bf16)
            hipLaunchKernelGGL((gemm_rows_kernel<__bf16>), grid, dim3(kRowsWaves * 64), 0, s, p);
        else
            hipLaunchKernelGGL((gemm_rows_kernel<_Float16>), grid, dim3(kRowsWaves * 64), 0, s, p);
        return hipGetLastError();
    }
    switch (layout) {
        case kGemmForward:
            return p.bf16 ? launch_tile<__bf16, false, false>(p, tile, s)
                          : launch_tile<_Float16, false, false>(p, tile, s);
        case kGemmDx:
            return p.bf16 ? launch_tile<__bf16, true, false>(p, tile, s)
                          : launch_tile<_Float16, true, false>(p, tile, s);
        default:
            return p.bf16 ? launch_tile<__bf16, true, true>(p, tile, s) : launch_tile<_Float16, true, true>(p, tile, s);
    }
}

hipError_t launch_gemm_pair(const GemmParams &dx, const GemmParams &dw, int tile, const ColumnSumParams &cs,
                            hipStream_t s) {
    return dx.bf16 ? launch_pair<__bf16>(dx, dw, tile, cs, s) : launch_pair<_Float16>(dx, dw, tile, cs, s);
}

namespace {
int act_groups(int32_t n) { return n / 8 < 256 ? n / 8 : 256; }
}  // namespace

int32_t act_grad_strips(int64_t m, int32_t n) {
    const int g = act_groups(n), at_once = 256 / g;
    const int64_t col_blocks = (n / 8 + g - 1) / g;
    int64_t strips = (1024 + col_blocks - 1) / col_blocks;
    const int64_t most = (m + 4 * at_once - 1) / (4 * at_once);  // at least 4 steps each
    if (strips > most) strips = most;
    return (int32_t)(strips < 1 ? 1 : strips);
}

hipError_t launch_act_grad(const ActGradParams &p, hipStream_t s) {
    const int g = act_groups(p.n), at_once = 256 / g;
    const dim3 grid((unsigned)((p.n / 8 + g - 1) / g), (unsigned)p.strips);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p, g, at_once);
        return hipGetLastError();
    };
#define C3D_ACT_GRAD(ACT, DZ)                                       \
    (p.bf16 ? go(act_grad_kernel<__bf16, ACT, DZ>) : go(act_grad_kernel<_Float16, ACT, DZ>))
    switch (p.act) {
        case CONV3D_ACT_SILU: return C3D_ACT_GRAD(CONV3D_ACT_SILU, true);
        case CONV3D_ACT_GELU: return C3D_ACT_GRAD(CONV3D_ACT_GELU, true);
        case CONV3D_ACT_GELU_TANH: return C3D_ACT_GRAD(CONV3D_ACT_GELU_TANH, true);
        default: return C3D_ACT_GRAD(CONV3D_ACT_NONE, false);
    }
#undef C3D_ACT_GRAD
}

}  // namespace c3d
