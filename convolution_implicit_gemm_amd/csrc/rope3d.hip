// Rotary positions over (time, height, width) on query and key heads, gfx950.
//
// Pair p of a head, on axis a at position s, is turned by s * base^(-2 i / dim_a),
// i being p's index within its axis:  (u, v) -> (u cos - v sin, u sin + v cos).
// The gradient is the turn by the negative angle.
//
// A stream over HBM: each element is read and written once (in place, if the
// caller wants), so the rest has to hide behind that.  A thread owns one group
// of pairs of one token (8 adjacent elements, or 8 + 8 of the two halves) and
// walks a range of the token's query and key heads with the same sines and
// cosines, which it computes itself: whole turns are dropped from the angle in
// 64 bits (positions of any size keep their accuracy), the rest goes through
// fp32 sincospi.  No table, no extra launch, no extra traffic.
#include "elem16.h"
#include "token_internal.h"

namespace c3d {

namespace {

constexpr int kRopeThreads = 256;

// HALVES: the pair is (p, p + pairs) instead of (2p, 2p + 1).
template <typename E, bool HALVES>
__global__ __launch_bounds__(kRopeThreads) void rope3d_kernel(RopeParams p, int tasks, int tokens_per_block,
                                                              int heads_per_block) {
    constexpr int NP = HALVES ? 8 : 4;  // pairs of a rotating task
    const int slot = threadIdx.x / tasks, task = threadIdx.x - slot * tasks;
    const int64_t idx = (int64_t)blockIdx.x * tokens_per_block + slot;  // flattened (sample, token)
    if (slot >= tokens_per_block || idx >= p.tokens * p.n) return;
    const int ns = (int)(idx / p.tokens);
    const int64_t tok = idx - (int64_t)ns * p.tokens;

    // the task's elements: group e0 (and e1 = e0 + pairs), turned for pairs p0 .. p0 + NP - 1
    const int turning = p.pairs / NP;  // tasks of whole groups of pairs
    int e0, np, p0;
    if (HALVES) {
        const bool turn = task < turning;
        e0 = turn ? task * 8 : 2 * p.pairs + (task - turning) * 8;
        np = turn ? 8 : 0;
        p0 = task * 8;
    } else {
        e0 = task * 8;
        p0 = task * 4;
        np = p.pairs - p0;
        np = np < 0 ? 0 : (np > 4 ? 4 : np);
    }
    float cs[NP], sn[NP];
    {
        double pos[3];
        if (p.positions) {
            const int32_t *pp = p.positions + idx * 3;
            for (int a = 0; a < 3; ++a) pos[a] = (double)pp[a];
        } else {
            const int64_t hw = (int64_t)p.h * p.w;
            const int64_t t = tok / hw;
            const int r = (int)(tok - t * hw);
            pos[0] = (double)(t + p.t_offset);
            pos[1] = (double)(r / p.w);
            pos[2] = (double)(r % p.w);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            cs[i] = 1.0f;
            sn[i] = 0.0f;
            if (i < np) {
                const int pr = p0 + i;
                double turns = (pr < p.end_t ? pos[0] : pr < p.end_h ? pos[1] : pos[2]) * p.turns[pr];
                turns -= rint(turns);
                sincospif(2.0f * (float)turns, &sn[i], &cs[i]);
                if (p.inverse) sn[i] = -sn[i];
            }
        }
    }

    const int heads = p.q.heads + p.k.heads;
    const int h0 = blockIdx.y * heads_per_block;
    const int h1 = h0 + heads_per_block < heads ? h0 + heads_per_block : heads;
    for (int hh = h0; hh < h1; ++hh) {
        const bool isq = hh < p.q.heads;
        const RopeTensor &t = isq ? p.q : p.k;
        const int head = isq ? hh : hh - p.q.heads;
        const _Float16 *in = t.in + ns * t.in_stride[0] + tok * t.in_stride[1] + head * t.in_stride[2] + e0;
        _Float16 *out = t.out + ns * t.out_stride[0] + tok * t.out_stride[1] + head * t.out_stride[2] + e0;
        e16x8_t a = *reinterpret_cast<const e16x8_t *>(in);
        if constexpr (HALVES) {
            if (np) {
                e16x8_t b = *reinterpret_cast<const e16x8_t *>(in + p.pairs);
                e16x8_t oa, ob;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = to_f32<E>(a[i]), v = to_f32<E>(b[i]);
                    oa[i] = from_f32<E>(fmaf(u, cs[i], -v * sn[i]));
                    ob[i] = from_f32<E>(fmaf(u, sn[i], v * cs[i]));
                }
                *reinterpret_cast<e16x8_t *>(out + p.pairs) = ob;
                a = oa;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < np) {  // a pair that does not turn keeps its bits
                    const float u = to_f32<E>(a[2 * i]), v = to_f32<E>(a[2 * i + 1]);
                    a[2 * i] = from_f32<E>(fmaf(u, cs[i], -v * sn[i]));
                    a[2 * i + 1] = from_f32<E>(fmaf(u, sn[i], v * cs[i]));
                }
        }
        *reinterpret_cast<e16x8_t *>(out) = a;
    }
}

}  // namespace

hipError_t launch_rope3d(const RopeParams &p, hipStream_t s) {
    const int tasks = p.halves ? p.pairs / 8 + (p.head_dim - 2 * p.pairs) / 8 : p.head_dim / 8;
    const int tpb = kRopeThreads / tasks;
    const int64_t blocks = (p.tokens * p.n + tpb - 1) / tpb;
    const int heads = p.q.heads + p.k.heads;
    const int hpb = 8;
    const dim3 grid((unsigned)blocks, (unsigned)((heads + hpb - 1) / hpb));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(kRopeThreads), 0, s, p, tasks, tpb, hpb);
        return hipGetLastError();
    };
    if (p.halves) return p.bf16 ? go(rope3d_kernel<__bf16, true>) : go(rope3d_kernel<_Float16, true>);
    return p.bf16 ? go(rope3d_kernel<__bf16, false>) : go(rope3d_kernel<_Float16, false>);
}

}  // namespace c3d
