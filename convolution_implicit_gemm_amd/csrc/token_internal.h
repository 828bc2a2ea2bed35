// Internal interfaces of the token operators (linear, layernorm, rope3d):
// their host-side entry points (token_api.cpp) and their gfx950 kernels.  Not
// installed; not part of the public ABI.
#pragma once

#include "c3d_internal.h"
#include "conv3d.h"

namespace c3d {

// Status helpers shared with api.cpp: set the thread's message and return the
// status; clear it; check that the current device is a gfx950.
conv3d_status api_fail(conv3d_status s, const char *fmt, ...);
conv3d_status api_ok();
conv3d_status api_check_device();

// ---- linear: out[m][n] = epilogue(sum_k q[m][k] p[n][k]).
// One matrix product as the kernels execute it.  p is the operand of the
// output's columns (contiguous in memory), q the operand of its rows.  Each is
// stored with the contraction contiguous ([n][k], [m][k]) or, transposed, as
// its rows ([k][n], [k][m]).
struct GemmParams {
    const _Float16 *p, *q;         // 16-bit storage: fp16, or bf16 when bf16 is set
    int64_t p_stride, q_stride;    // elements between rows of the stored matrices
    const _Float16 *bias;          // [N] or null
    const _Float16 *res;           // [M][N] or null, res_stride
    _Float16 *z;                   // [M][N] contiguous or null: the value before the activation
    _Float16 *y;                   // [M][N], y_stride
    int64_t y_stride, res_stride;
    int32_t M, N, K;
    int32_t act;                   // conv3d_act
    int32_t bf16;
    int32_t m_tiles, n_tiles;
    int32_t niter;                 // K stages of one tile
    int32_t dp_tiles;              // tiles [0, dp_tiles) run whole, one workgroup each
    int32_t sk_tiles, sk_pieces;   // the other tiles run as sk_pieces K-pieces each
    float *partial;                // [sk_tiles * sk_pieces][tile_m * tile_n] fp32 (workspace)
};


enum GemmLayout { kGemmForward = 0, kGemmDx = 1, kGemmDw = 2 };  // (p, q): (k, k), (T, k), (T, T)

struct GemmTile {
    const char *name;
    int bm, bn, bk, threads;
    int per_cu;    // workgroups that share a CU
    int groups;    // groups of waves that take the stages in turn
    double step_us_few[3], step_us_full[3], cold, launch_us, round_us;  // cost model (linear.hip)
};
constexpr int kGemmCUs = 256;
constexpr int kGemmMaxPieces = 32;
// The kernel of few rows, an index into gemm_tiles: forward products of at most kGemmRowsMax rows.
constexpr int kGemmRowsTile = 5, kGemmRowsMax = 16;
const GemmTile *gemm_tiles(int *count);
hipError_t launch_gemm(const GemmParams &p, int tile, GemmLayout layout, hipStream_t s);
// dx, dw and the column sums (cs.out0 null: none) in one launch, with one tile
// of kGemmPairFirst .. kGemmPairLast for both.
constexpr int kGemmPairFirst = 1, kGemmPairLast = 3;
struct ColumnSumParams;
hipError_t launch_gemm_pair(const GemmParams &dx, const GemmParams &dw, int tile, const ColumnSumParams &cs,
                            hipStream_t s);

// dz = dy * act'(z) (dz may be null: no activation) and the column sums of dz
// as `strips` fp32 partials [strips][n] (colpart may be null).
struct ActGradParams {
    const _Float16 *dy, *z;
    int64_t dy_stride;
    _Float16 *dz;     // contiguous [m][n]
    float *colpart;
    int64_t m;
    int32_t n, act, bf16, strips;
};
int32_t act_grad_strips(int64_t m, int32_t n);
hipError_t launch_act_grad(const ActGradParams &p, hipStream_t s);
// The sums over the rows of part [rows][cols] (cols a multiple of 8), or of in16's
// rows of elements, `stride` apart, rounded to the element type: columns below
// split into out0, the others into out1 (either may be null).
struct ColumnSumParams {
    const float *part;
    const _Float16 *in16;
    int64_t stride;
    _Float16 *out0, *out1;
    int32_t rows, cols, split, bf16;
};
// Rows of elements are summed by whole columns up to 6144 rows and 6144 x 8192
// elements, else by strips of rows, whose sums need a launch more but take all CUs
// for any shape.  bf16 dbias without an activation, strips against whole columns, in
// us, alone and in one pass with dx and dw (k = 512):
//   64 x 64 7.0 and 4.8, 8.1 and 6.3;        6144 x 64 6.9 and 5.1, 17.2 and 14.3
//   4000 x 2048 13.6 and 5.2, 37 and 31;     6144 x 8192 20.8 and 21.5, 124 and 114
//   2000 x 16384 16.8 and 15.3, 95 and 89;   512 x 65536 17.9 and 12.4, 125 and 114
// and beyond: 8192 x 8192 25 and 28, 155 and 148;  12288 x 2048 15 and 21, 75 and 75;
//   4000 x 16384 26 and 28, 175 and 176;     6144 x 65536 144 and 209, 843 and 908.
constexpr int64_t kColumnRows = 6144, kColumnElements = kColumnRows * 8192;
inline bool sum_whole_columns(int64_t rows, int32_t cols) {
    return rows <= kColumnRows && rows * cols <= kColumnElements;
}
hipError_t launch_column_sum(const ColumnSumParams &p, hipStream_t s);
// Zeros into rows of `width` elements, `stride` apart.
hipError_t launch_zero_rows(_Float16 *y, int64_t rows, int32_t width, int64_t stride, hipStream_t s);

// ---- layernorm
constexpr int kLnMaxC = 16384;
struct LnParams {
    const _Float16 *x, *gamma, *beta;
    _Float16 *y;
    float2 *stats;  // [rows] (mean, 1 / sqrt(var + eps)) or null
    int64_t rows, x_stride, y_stride;
    int32_t c;
    float eps;
    int32_t bf16;
};
hipError_t launch_layernorm(const LnParams &p, hipStream_t s);
struct LnGradParams {
    const _Float16 *dy, *x, *gamma, *dres;
    const float2 *stats;
    _Float16 *dx, *dgamma, *dbeta;
    float *part;    // [blocks][2][c] (workspace), or null when neither weight gradient is asked for
    int64_t rows, x_stride, y_stride;
    int32_t c, bf16;
};
int32_t ln_grad_blocks(int64_t rows, int32_t c);
hipError_t launch_layernorm_grad(const LnGradParams &p, hipStream_t s);

// ---- rope3d
constexpr int kRopeMaxPairs = 128;
struct RopeTensor {
    const _Float16 *in;
    _Float16 *out;
    int64_t in_stride[3], out_stride[3];  // sample, token, head, in elements
    int32_t heads;
};
struct RopeParams {
    RopeTensor q, k;
    const int32_t *positions;  // [n][tokens][3] or null: the grid's own
    int64_t tokens;            // per sample
    int32_t n, h, w, t_offset;
    int32_t head_dim, pairs;   // rotated pairs: pairs [0, end_t) turn with time, [end_t, end_h) height, the rest width
    int32_t end_t, end_h;
    int32_t halves, bf16, inverse;
    double turns[kRopeMaxPairs];  // whole turns per position of each pair
};
hipError_t launch_rope3d(const RopeParams &p, hipStream_t s);

// ---- attention
constexpr int kAttnMaxDim = 128, kAttnFewRows = 32;
struct AttnParams {
    const _Float16 *q, *k, *v;
    _Float16 *o;                 // backward: read
    float *lse;                  // [n][heads_q][tq], forward: or null
    const int32_t *lengths;      // [n][2] (queries, keys) or null
    int64_t qs[3], ks[3], vs[3], os[3];  // sample, token, head, in elements
    int64_t q_offset;
    int32_t n, hq, hk, group, d, tq, tk;
    int32_t rows;                // tq * group: the rows of one (sample, key head)
    int32_t frame, window, tail, bf16;
    float scale;
    // forward: `splits` pieces of each row's keys; more than one leave partials
    int32_t splits, pieces;      // pieces: keys of a piece, in tiles of the kernel
    float *part_o;               // [splits][n * hk][rows][d] sums of unnormalised values
    float2 *part_ml;             // [splits][n * hk][rows] (maximum, sum), in the exponent of 2
    // backward
    const _Float16 *dout;
    _Float16 *dq, *dk, *dv;
    float *nlse, *ndelta;        // [n][hq][tq] in the workspace: see attention_grad.hip
    // dk and dv: `grad_splits` pieces of each key tile's steps, of grad_pieces steps each; more than
    // one leave partials, [grad_splits][n * hk][tk][d]
    int32_t grad_splits, grad_pieces;
    float *part_dk, *part_dv;
};
// Tiles of the kernels: rows (query tokens times the query heads of a key head) and
// keys of a step.  kAttnFew: all rows of a key head in one tile.
enum AttnTileKind { kAttnFew = 0, kAttn64 = 1, kAttn128 = 2, kAttn256 = 3 };
struct AttnTileSize {
    const char *name;
    int rows, keys, threads;
};
constexpr AttnTileSize attn_tile(AttnTileKind k) {
    return k == kAttnFew ? AttnTileSize{"attention_few", 32, 128, 256}
         : k == kAttn64  ? AttnTileSize{"attention_64x128", 64, 128, 512}
         : k == kAttn128 ? AttnTileSize{"attention_128x128", 128, 128, 512}
                         : AttnTileSize{"attention_256x64", 256, 64, 512};
}
hipError_t launch_attention(const AttnParams &p, AttnTileKind kind, hipStream_t s);
// dq by tiles of kind_q; dk and dv by tiles of as many keys as kind_kv has rows, and 64
// query tokens (kAttn64: 128) to a step.
constexpr int attn_grad_step(AttnTileKind kind) { return kind == kAttn64 ? 128 : 64; }
struct AttnGradKinds {
    AttnTileKind q, kv;
    bool together;  // in one launch: both kAttn64 or both kAttn128
};
hipError_t launch_attention_grad(const AttnParams &p, const AttnGradKinds &k, hipStream_t s);

// ---- adamw
constexpr int kAdamwBlock = 128;    // elements that share a scale
constexpr int kAdamwTensors = 48;   // of a launch: their table travels in the kernel's arguments (4 KiB)
// Elements of a workgroup.  far: the step's tensors are larger than the last-level cache (256 MB)
// and go past the caches.  201 million weights, 8-bit states, 3.2 GB: 537-542 us, through the caches
// 7% more; 14 million in 61 tensors, 133 MB: past the caches 15% more than 38-40 us.
constexpr int adamw_unit(bool far) { return far ? 2048 : 1024; }
constexpr int64_t kAdamwCached = (int64_t)256 << 20;
struct AdamwTensor {
    _Float16 *param;
    float *master;
    const void *grad;
    void *m, *v;
    uint8_t *m_scale, *v_scale;
    int64_t count;
    float decay;
};
struct AdamwHyper {
    float grad_scale, beta1, rest1, beta2, rest2;  // rest: 1 - beta
    float lr1;          // lr / (1 - beta1^step)
    float root2;        // 1 / sqrt(1 - beta2^step)
    float eps, lr_decay;  // lr * weight_decay
};
struct AdamwParams {
    AdamwTensor t[kAdamwTensors];
    int32_t first[kAdamwTensors];  // of each tensor's workgroups; INT32_MAX behind the last tensor
    const AdamwHyper *device_hyper;
    AdamwHyper hyper;
};
static_assert(sizeof(AdamwParams) <= 4096, "kernel arguments");
hipError_t launch_adamw(const AdamwParams &p, int64_t blocks, bool far, bool bf16, bool state8, bool grad32, hipStream_t s);

}  // namespace c3d
