// Rotary positions over (time, height, width) on query and key heads, gfx950.
//
// Pair p of a head, on axis a at position s, is turned by s * base^(-2 i / dim_a),
// i being p's index within its axis:  (u, v) -> (u cos - v sin, u sin + v cos).
// The gradient is the turn by the negative angle.
//
// A stream over HBM: each element is read and written once (in place, if the
// caller wants), so the rest has to hide behind that.  A block takes some
// tokens: first its threads work out the sines and cosines of (token, pair), once
// for all heads, into LDS; whole turns are dropped from the angle in 64 bits
// (positions of any size keep their accuracy), the rest goes through fp32
// sincospi.  Then they walk the tokens' heads in memory order, one task per
// thread and step (a task: 8 adjacent elements, or 8 + 8 of the two halves), so
// that a wave reads and writes whole runs of a token's row.  No table, no extra
// launch, no extra traffic.  36864 tokens of 16 + 16 heads of 128 inside fused rows:
// 122 us, 4.9 TB/s (one thread per token and group of pairs, walking the heads: 145
// us); 16 single tokens 4.3 us.
#include "elem16.h"
#include "token_internal.h"

namespace c3d {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;       // tasks of a thread whose loads are in flight at once
constexpr int kRopeMaxTokens = 16;  // tokens of a block

// a / b for 0 <= a < 2^22: the float quotient is off by at most one
__device__ __forceinline__ int small_div(int a, int b, float rcp_b) {
    int q = (int)((float)a * rcp_b);
    const int r = a - q * b;
    q += r >= b ? 1 : 0;
    q -= r < 0 ? 1 : 0;
    return q;
}

// The block's tokens from `first` on.  HALVES: the pair is (p, p + pairs) instead of
// (2p, 2p + 1).  turn: [token][pair] (cos, sin); place: a token's offsets in q, q's
// output, k, k's output.
template <typename E, bool HALVES>
__device__ __forceinline__ void rope3d_tokens(const RopeParams &p, int64_t first, int tasks, int tokens_per_block,
                                              float2 *turn, int64_t (*place)[4]) {
    const int64_t left = p.tokens * p.n - first;
    const int ntok = left < tokens_per_block ? (int)left : tokens_per_block;
    const int64_t ns0 = first / p.tokens, tok0 = first - ns0 * p.tokens;  // the first token's sample and index

    if (threadIdx.x < ntok * 4) {
        const int t = threadIdx.x >> 2, which = threadIdx.x & 3;
        const int64_t over = tok0 + t, dn = over / p.tokens;
        const RopeTensor &x = which < 2 ? p.q : p.k;
        const int64_t *st = which & 1 ? x.out_stride : x.in_stride;
        place[t][which] = (ns0 + dn) * st[0] + (over - dn * p.tokens) * st[1];
    }
    const float rcp_pairs = 1.0f / (float)p.pairs;
    for (int i = threadIdx.x; i < ntok * p.pairs; i += kRopeThreads) {
        const int t = small_div(i, p.pairs, rcp_pairs), pr = i - t * p.pairs;
        const int axis = pr < p.end_t ? 0 : pr < p.end_h ? 1 : 2;
        double pos;
        if (p.positions) {
            pos = (double)p.positions[(first + t) * 3 + axis];
        } else {
            const int64_t tok = (tok0 + t) % p.tokens;
            const int64_t hw = (int64_t)p.h * p.w;
            const int64_t frame = tok / hw;
            const int r = (int)(tok - frame * hw);
            pos = axis == 0 ? (double)(frame + p.t_offset) : (double)(axis == 1 ? r / p.w : r % p.w);
        }
        double turns = pos * p.turns[pr];
        turns -= rint(turns);
        float sn, cs;
        sincospif(2.0f * (float)turns, &sn, &cs);
        turn[i] = make_float2(cs, p.inverse ? -sn : sn);
    }
    __syncthreads();

    const int heads = p.q.heads + p.k.heads;
    const int per_token = heads * tasks, items = ntok * per_token;
    const int turning = HALVES ? p.pairs / 8 : (p.pairs + 3) / 4;  // tasks that turn pairs
    const float rcp_token = 1.0f / (float)per_token, rcp_tasks = 1.0f / (float)tasks;
    struct Item {
        const _Float16 *in;
        _Float16 *out;
        const float2 *cs;
        bool turns;
        int np;
    };
    auto item = [&](int i) {
        const int t = small_div(i, per_token, rcp_token), r = i - t * per_token;
        const int hh = small_div(r, tasks, rcp_tasks), task = r - hh * tasks;
        const bool isq = hh < p.q.heads;
        const int head = isq ? hh : hh - p.q.heads;
        Item m;
        m.turns = task < turning;
        const int e0 = HALVES && !m.turns ? 2 * p.pairs + (task - turning) * 8 : task * 8;
        m.in = (isq ? p.q.in : p.k.in) + place[t][isq ? 0 : 2] +
               head * (isq ? p.q.in_stride[2] : p.k.in_stride[2]) + e0;
        m.out = (isq ? p.q.out : p.k.out) + place[t][isq ? 1 : 3] +
                head * (isq ? p.q.out_stride[2] : p.k.out_stride[2]) + e0;
        const int p0 = task * (HALVES ? 8 : 4);
        m.cs = turn + t * p.pairs + p0;
        m.np = p.pairs - p0;
        return m;
    };
    // The batch's loads go first: an output may be its input, so the compiler
    // cannot move a load above an earlier store itself.
    for (int base = threadIdx.x; base < items; base += kRopeThreads * kRopeBatch) {
        Item m[kRopeBatch];
        e16x8_t a[kRopeBatch], b[kRopeBatch];
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            const int i = base + k * kRopeThreads;
            if (i >= items) continue;
            m[k] = item(i);
            a[k] = *reinterpret_cast<const e16x8_t *>(m[k].in);
            if (HALVES && m[k].turns) b[k] = *reinterpret_cast<const e16x8_t *>(m[k].in + p.pairs);
        }
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            if (base + k * kRopeThreads >= items) continue;
            if (m[k].turns) {
                if constexpr (HALVES) {
                    e16x8_t oa, ob;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 c = m[k].cs[i];
                        const float u = to_f32<E>(a[k][i]), v = to_f32<E>(b[k][i]);
                        oa[i] = from_f32<E>(fmaf(u, c.x, -v * c.y));
                        ob[i] = from_f32<E>(fmaf(u, c.y, v * c.x));
                    }
                    *reinterpret_cast<e16x8_t *>(m[k].out + p.pairs) = ob;
                    a[k] = oa;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < m[k].np) {  // a pair that does not turn keeps its bits
                            const float2 c = m[k].cs[i];
                            const float u = to_f32<E>(a[k][2 * i]), v = to_f32<E>(a[k][2 * i + 1]);
                            a[k][2 * i] = from_f32<E>(fmaf(u, c.x, -v * c.y));
                            a[k][2 * i + 1] = from_f32<E>(fmaf(u, c.y, v * c.x));
                        }
                }
            }
            *reinterpret_cast<e16x8_t *>(m[k].out) = a[k];
        }
    }
}

template <typename E, bool HALVES>
__global__ __launch_bounds__(kRopeThreads) void rope3d_kernel(RopeParams p, int tasks, int tokens_per_block) {
    extern __shared__ float2 turn[];
    __shared__ int64_t place[kRopeMaxTokens][4];
    const int64_t all = p.tokens * p.n, step = (int64_t)gridDim.x * tokens_per_block;
    for (int64_t first = (int64_t)blockIdx.x * tokens_per_block; first < all; first += step) {
        rope3d_tokens<E, HALVES>(p, first, tasks, tokens_per_block, turn, place);
        __syncthreads();  // the next tokens' sines overwrite these
    }
}

}  // namespace

hipError_t launch_rope3d(const RopeParams &p, hipStream_t s) {
    const int tasks = p.halves ? p.pairs / 8 + (p.head_dim - 2 * p.pairs) / 8 : p.head_dim / 8;
    const int64_t total = p.tokens * p.n;
    // one token per block where that leaves CUs idle otherwise, else enough
    // tokens that a thread has a few batches
    const int per_token = (p.q.heads + p.k.heads) * tasks;
    int tpb = (4 * kRopeBatch * kRopeThreads + per_token - 1) / per_token;
    if (tpb > kRopeMaxTokens) tpb = kRopeMaxTokens;
    while (tpb > 1 && (int64_t)tpb * per_token >= 1 << 22) --tpb;  // small_div's range
    while (tpb > 1 && (total + tpb - 1) / tpb < 1024) --tpb;
    const int64_t blocks = (total + tpb - 1) / tpb;
    const dim3 grid((unsigned)(blocks < 1 << 22 ? blocks : 1 << 22));  // a launch holds fewer than 2^32 threads
    const size_t lds = (size_t)tpb * p.pairs * sizeof(float2);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kRopeThreads), lds, s, p, tasks, tpb);
        return hipGetLastError();
    };
    if (p.halves) return p.bf16 ? go(rope3d_kernel<__bf16, true>) : go(rope3d_kernel<_Float16, true>);
    return p.bf16 ? go(rope3d_kernel<__bf16, false>) : go(rope3d_kernel<_Float16, false>);
}

}  // namespace c3d
