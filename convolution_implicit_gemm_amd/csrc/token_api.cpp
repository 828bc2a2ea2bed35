// Host side of the token operators declared in include/conv3d.h (linear,
// layernorm, rope3d): validation, planning, and launches on the caller's
// stream.  Nothing here synchronises the device or allocates device memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <utility>

#include "token_internal.h"

using c3d::api_check_device;
using c3d::api_fail;
using c3d::api_ok;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 20;
constexpr int kMaxWidth = 65536;
constexpr double kMaxElements = 281474976710656.0;  // 2^48, from a tensor's first element to its last
constexpr int kCUs = 256;

bool misaligned(const void *p, uintptr_t bytes = 16) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Device memory [p, p + bytes) of a matrix, for overlap checks.
struct Span {
    uintptr_t lo, hi;
    Span(const void *p, int64_t rows, int64_t cols, int64_t stride, int64_t elem = 2)
        : lo(reinterpret_cast<uintptr_t>(p)),
          hi(p && rows > 0 ? lo + (uintptr_t)(((rows - 1) * stride + cols) * elem) : lo) {}
    Span(const void *p, size_t bytes) : lo(reinterpret_cast<uintptr_t>(p)), hi(p ? lo + bytes : lo) {}
    // nothing meets an empty one
    bool meets(const Span &o) const { return lo < o.hi && o.lo < hi && lo < hi && o.lo < o.hi; }
};

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// One matrix product's kernel and how its tiles are run.
struct GemmPlan {
    int tile = 0;
    int m_tiles = 0, n_tiles = 0, niter = 0;
    int dp = 0, sk = 0, pieces = 0;
    size_t partial_bytes = 0;
};

constexpr double kJoinBytesPerUs = 9e6;
constexpr double kJoinLaunchUs = 4.5;
// One launch of dx and dw is taken up to this much above the sum of their own
// best estimates, which are the more optimistic ones: over 300 sizes the slower
// way is then taken at a mean loss of 0.6%, at 1.0 of 1.8%.
constexpr double kPairMargin = 1.2;
constexpr double kL2Bytes = 32e6;  // all eight
constexpr size_t kMaxPartial = (size_t)256 << 20;

// What steps of a product cost in a tile's kernel.  `missed` is how much of its
// operands the L2s (4 MB on each of the 8 dies) cannot hold.
struct TileCost {
    const c3d::GemmTile &t;
    double few, full;
    int64_t slots;
    TileCost(const c3d::GemmTile &tile, c3d::GemmLayout l, double operand_bytes) : t(tile) {
        full = t.step_us_full[l];
        slots = (int64_t)kCUs * t.per_cu;
        const double missed = operand_bytes < kL2Bytes ? operand_bytes / kL2Bytes : 1.0;
        few = t.step_us_few[l] * (1.0 + t.cold * missed);
        if (few > full) few = full;
    }
    // Steps of a card with `units` workgroups on it: as much faster as they are
    // fewer (the L2s serve the operands of all of them), down to the time of a few.
    double step(int64_t units) const {
        const double s = units < slots ? full * units / slots : full;
        return s > few ? s : few;
    }
    // `units` workgroups of `steps` steps each: rounds of as many as fit the card.
    double rounds(int64_t units, double steps) const {
        const int64_t rem = units % slots;
        return units / slots * (steps * full + t.round_us) + (rem ? steps * step(rem) + t.round_us : 0.0);
    }
};

// The kernel of few rows: every workgroup streams its 16 columns of w at what one
// CU draws, 32 bytes per nanosecond, less for the rows of x read beside them
// (measured over n and k from 256 to 16384, m = 1, 4, 16), and all of them at
// 6.4 TB/s.
double rows_us(int64_t m, int n, int64_t k) {
    const double rounds = n > 16 * kCUs ? n / (16.0 * kCUs) : 1.0;
    const double draw = rounds * (double)k * 1e-3 * (1.0 + 0.041 * m), stream = 2.0 * n * k / 6.4e6;
    return 2.3 + (draw > stream ? draw : stream);
}

// CONV3D_LINEAR_TILE: a kernel's name, or its name + "+pair", which also makes
// a backward pass run dx and dw in one launch of it.
struct Forced {
    const char *v = getenv("CONV3D_LINEAR_TILE");
    const size_t len = v ? strcspn(v, "+") : 0;
    bool is(const char *name) const { return v && strlen(name) == len && strncmp(v, name, len) == 0; }
    bool pair() const { return v && strcmp(v + len, "+pair") == 0; }
};

// Launches hold fewer than 2^32 threads; the first tile's kernel launches at
// most one workgroup per CU and only counts its units.
bool runnable(int tile, const c3d::GemmTile &t, int64_t units) {
    return tile == 0 ? units < (int64_t)1 << 30 : units * t.threads < (int64_t)1 << 31;
}

// The kernel and decomposition with the least time by the measured rates.  A
// last partial round of tiles can be run as pieces of the contraction instead,
// which costs writing and adding fp32 partials in a second launch.
GemmPlan plan_gemm(int64_t m, int n, int64_t k, c3d::GemmLayout layout, double *us) {
    int count = 0;
    const c3d::GemmTile *tiles = c3d::gemm_tiles(&count);
    const Forced force;
    GemmPlan best;
    double best_s = -1.0;
    if (layout == c3d::kGemmForward && m <= c3d::kGemmRowsMax &&
        (!force.v || force.is(tiles[c3d::kGemmRowsTile].name))) {
        best.tile = c3d::kGemmRowsTile;
        best.m_tiles = 1;
        best.n_tiles = best.dp = (n + 15) / 16;
        best_s = rows_us(m, n, k);
        if (force.v) {
            *us = best_s;
            return best;
        }
    }
    bool found = false;
    for (int pass = force.v ? 0 : 1; pass < 2 && !found; ++pass)
        for (int i = 0; i < count; ++i) {
            const c3d::GemmTile &t = tiles[i];
            if (i == c3d::kGemmRowsTile) continue;
            if (pass == 0 && !force.is(t.name)) continue;
            GemmPlan g;
            g.tile = i;
            g.m_tiles = (int)((m + t.bm - 1) / t.bm);
            g.n_tiles = (n + t.bn - 1) / t.bn;
            g.niter = (int)((k + t.bk - 1) / t.bk);
            const int64_t all = (int64_t)g.m_tiles * g.n_tiles;
            const int64_t slots = (int64_t)kCUs * t.per_cu;
            if (!runnable(i, t, all)) continue;
            g.dp = (int)all;
            auto steps = [&](int pieces) {
                return (double)(((g.niter + pieces - 1) / pieces + t.groups - 1) / t.groups);
            };
            const TileCost cost(t, layout, 2.0 * ((double)m * k + (double)n * k));
            double sec = t.launch_us + cost.rounds(all, steps(1));
            const int64_t full = all / slots, rem = all % slots;
            GemmPlan pick = g;
            for (int pc = 2; rem && pc <= c3d::kGemmMaxPieces && pc * 4 <= g.niter; ++pc) {
                const size_t bytes = (size_t)rem * pc * t.bm * t.bn * 4;
                if (bytes > kMaxPartial) break;
                const double s2 = t.launch_us + cost.rounds(full * slots, steps(1)) +
                                  cost.rounds(rem * pc, steps(pc)) + 2.0 * bytes / kJoinBytesPerUs + kJoinLaunchUs;
                if (s2 < sec * 0.97) {
                    sec = s2;
                    pick.dp = (int)(full * slots);
                    pick.sk = (int)rem;
                    pick.pieces = pc;
                    pick.partial_bytes = bytes;
                }
            }
            found = true;
            // both operands and the output once, as fast as the tiles stream them
            const double stream = 2.0 + 2.0 * ((double)m * k + (double)n * k + (double)m * n) / 6.0e6;
            if (sec < stream) sec = stream;
            if (best_s < 0.0 || sec < best_s) {
                best_s = sec;
                best = pick;
            }
        }
    *us = best_s;
    return best;
}

// Tiles of one product, all split into `pieces` (1: none).
GemmPlan even_split(int tile, const c3d::GemmTile &t, int64_t m, int n, int64_t k, int pieces) {
    GemmPlan g;
    g.tile = tile;
    g.m_tiles = (int)((m + t.bm - 1) / t.bm);
    g.n_tiles = (n + t.bn - 1) / t.bn;
    g.niter = (int)((k + t.bk - 1) / t.bk);
    const int all = g.m_tiles * g.n_tiles;
    if (pieces > 1) {
        g.sk = all;
        g.pieces = pieces;
        g.partial_bytes = (size_t)all * pieces * t.bm * t.bn * 4;
    } else {
        g.dp = all;
    }
    return g;
}

// dx and dw in one launch, sharing the card: the tile and the pieces of each
// with the least time, and that time.  Units that fit the card at once take as
// long as the longest, at the rate of all of them; more take the sum of their
// steps at the full card's rate and a part of the longest, when the card drains.
// (Fitted with the tiles' rates: within 10% rms of 900 pairs' times.)
double plan_pair(int64_t m, int n, int k, GemmPlan *dx, GemmPlan *dw) {
    int count = 0;
    const c3d::GemmTile *tiles = c3d::gemm_tiles(&count);
    const Forced force;
    double best = -1.0;
    for (int i = c3d::kGemmPairFirst; i <= c3d::kGemmPairLast; ++i) {
        const c3d::GemmTile &t = tiles[i];
        if (force.v && !force.is(t.name)) continue;
        auto tiles_of = [&](int64_t rows, int64_t cols) {
            return ((rows + t.bm - 1) / t.bm) * ((cols + t.bn - 1) / t.bn);
        };
        if (!runnable(i, t, (tiles_of(m, k) + tiles_of(n, k)) * 2)) continue;
        const double operands = 2.0 * ((double)m * k + (double)n * k + (double)m * n);
        const TileCost cost_x(t, c3d::kGemmDx, operands), cost_w(t, c3d::kGemmDw, operands);
        const int64_t slots = cost_x.slots;
        auto steps = [&](const GemmPlan &g) {
            const int per = g.pieces ? (g.niter + g.pieces - 1) / g.pieces : g.niter;
            return (double)((per + t.groups - 1) / t.groups);
        };
        auto units = [](const GemmPlan &g) { return (int64_t)g.dp + (int64_t)g.sk * g.pieces; };
        for (int px : {1, 2, 3, 4, 6, 8})
            for (int pw : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
                const GemmPlan x = even_split(i, t, m, k, n, px), w = even_split(i, t, n, k, m, pw);
                if ((px > 1 && px * 4 > x.niter) || (pw > 1 && pw * 4 > w.niter)) continue;
                const size_t bytes = x.partial_bytes + w.partial_bytes;
                if (bytes > kMaxPartial) continue;
                const int64_t all = units(x) + units(w);
                const double tx = steps(x) * cost_x.step(all) + t.round_us;
                const double tw = steps(w) * cost_w.step(all) + t.round_us;
                double us = tx > tw ? tx : tw;
                const double sum = (units(x) * tx + units(w) * tw) / slots;
                if (all > slots) us = sum + 0.3 * us;
                us += t.launch_us;
                if (bytes) us += 2.0 * bytes / kJoinBytesPerUs + kJoinLaunchUs;
                if (best < 0.0 || us < best) {
                    best = us;
                    *dx = x;
                    *dw = w;
                }
            }
    }
    return best;
}

void fill(c3d::GemmParams &q, const GemmPlan &g, int64_t m, int n, int64_t k, int bf16, void *partial) {
    q.M = (int32_t)m;
    q.N = n;
    q.K = (int32_t)k;
    q.bf16 = bf16;
    q.m_tiles = g.m_tiles;
    q.n_tiles = g.n_tiles;
    q.niter = g.niter;
    q.dp_tiles = g.dp;
    q.sk_tiles = g.sk;
    q.sk_pieces = g.pieces;
    q.partial = static_cast<float *>(partial);
}

const _Float16 *in16(const void *p) { return static_cast<const _Float16 *>(p); }
_Float16 *out16(void *p) { return static_cast<_Float16 *>(p); }

// A row stride: 0 means contiguous.  Returns a status, *out the stride.
conv3d_status row_stride(int64_t given, int64_t width, const char *what, int64_t *out) {
    *out = given ? given : width;
    if (given < 0 || (given && given < width) || given % 8)
        return api_fail(CONV3D_ERR_INVALID_ARG, "%s (%lld) must be 0 or a multiple of 8 of at least %lld", what,
                        (long long)given, (long long)width);
    if (given > kMaxStride)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "%s (%lld) is above %lld", what, (long long)given,
                        (long long)kMaxStride);
    return CONV3D_OK;
}

conv3d_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (misaligned(ws)) return api_fail(CONV3D_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    if (need && (!ws || bytes < need))
        return api_fail(CONV3D_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? bytes : (size_t)0);
    return CONV3D_OK;
}

conv3d_status launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return api_fail(CONV3D_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return api_ok();
}

}  // namespace

// ---------------------------------------------------------------- linear

struct linear_plan_s {
    linear_desc d;
    int64_t xs, ys, rs;
    GemmPlan fwd, dx, dw;
    GemmPlan pair_dx, pair_dw;  // dx and dw in one launch, when both are asked for
    bool pair;
    int strips;               // partial sums of dbias
    size_t off_col, off_part; // backward workspace: [dz][column sums][partial tiles]
    size_t back_bytes;
};

extern "C" {

conv3d_status linear_plan(const linear_desc *d, linear_plan_t *out, size_t *workspace_bytes) {
    if (!d || !out || !workspace_bytes)
        return api_fail(CONV3D_ERR_INVALID_ARG, "desc, out and workspace_bytes are required");
    if (d->m < 0 || d->n < 1 || d->k < 1) return api_fail(CONV3D_ERR_INVALID_ARG, "m >= 0, n >= 1 and k >= 1 needed");
    if (d->act < CONV3D_ACT_NONE || d->act > CONV3D_ACT_GELU_TANH)
        return api_fail(CONV3D_ERR_INVALID_ARG, "unknown activation %d", d->act);
    const uint32_t known = CONV3D_F_BIAS | CONV3D_F_RESIDUAL | CONV3D_F_PREACT | CONV3D_F_BF16;
    if (d->flags & ~known) return api_fail(CONV3D_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags & ~known);
    if (d->n % 8 || d->k % 8 || d->n > kMaxWidth || d->k > kMaxWidth)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "n (%d) and k (%d) must be multiples of 8 up to %d", d->n, d->k,
                        kMaxWidth);
    if (d->m >= kMaxRows) return api_fail(CONV3D_ERR_UNSUPPORTED, "m (%lld) is too large", (long long)d->m);
    int64_t xs, ys, rs;
    conv3d_status st = row_stride(d->x_stride, d->k, "x_stride", &xs);
    if (st == CONV3D_OK) st = row_stride(d->y_stride, d->n, "y_stride", &ys);
    if (st == CONV3D_OK) st = row_stride(d->residual_stride, d->n, "residual_stride", &rs);
    if (st != CONV3D_OK) return st;
    linear_plan_s *p = new (std::nothrow) linear_plan_s();
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "out of host memory");
    p->d = *d;
    p->xs = xs;
    p->ys = ys;
    p->rs = rs;
    p->strips = c3d::act_grad_strips(d->m, d->n);
    p->off_col = p->off_part = p->back_bytes = 0;
    if (d->m > 0) {
        double us_f, us_x, us_w;
        p->fwd = plan_gemm(d->m, d->n, d->k, c3d::kGemmForward, &us_f);
        p->dx = plan_gemm(d->m, d->k, d->n, c3d::kGemmDx, &us_x);
        p->dw = plan_gemm(d->n, d->k, d->m, c3d::kGemmDw, &us_w);
        for (const GemmPlan *g : {&p->fwd, &p->dx, &p->dw})
            if (g->dp + g->sk == 0) {
                delete p;
                return api_fail(CONV3D_ERR_UNSUPPORTED, "the product has too many tiles");
            }
        const Forced force;
        const double us_pair = plan_pair(d->m, d->n, d->k, &p->pair_dx, &p->pair_dw);
        // one launch less, and neither product's tail leaves the card idle
        p->pair = us_pair >= 0.0 &&
                  (force.v ? force.pair() : us_pair < kPairMargin * (us_x + us_w));
        const size_t dz = d->act != CONV3D_ACT_NONE ? align256((size_t)d->m * d->n * 2) : 0;
        size_t part = p->dx.partial_bytes > p->dw.partial_bytes ? p->dx.partial_bytes : p->dw.partial_bytes;
        const size_t both = p->pair ? p->pair_dx.partial_bytes + p->pair_dw.partial_bytes : 0;
        if (both > part) part = both;
        p->off_col = dz;
        p->off_part = dz + align256((size_t)p->strips * d->n * 4);
        p->back_bytes = p->off_part + part;
    }
    *out = p;
    *workspace_bytes = p->fwd.partial_bytes;
    return api_ok();
}

conv3d_status linear_plan_query(linear_plan_t p, linear_plan_info *info) {
    if (!p || !info) return api_fail(CONV3D_ERR_INVALID_ARG, "plan and info are required");
    memset(info, 0, sizeof(*info));
    int count = 0;
    const c3d::GemmTile &t = c3d::gemm_tiles(&count)[p->fwd.tile];
    info->tile_m = t.bm;
    info->tile_n = t.bn;
    info->tile_k = t.bk;
    info->threads = t.threads;
    info->grid = p->fwd.dp + (int64_t)p->fwd.sk * p->fwd.pieces;
    info->split_tiles = p->fwd.sk;
    info->split_pieces = p->fwd.pieces;
    info->workspace_bytes = p->fwd.partial_bytes;
    info->backward_workspace_bytes = p->back_bytes;
    snprintf(info->kernel_name, sizeof(info->kernel_name), "%s", t.name);
    return api_ok();
}

void linear_plan_destroy(linear_plan_t p) { delete p; }

conv3d_status linear_forward(linear_plan_t p, const void *x, const void *w, const void *bias, const void *residual,
                             void *y, void *preact, void *workspace, size_t workspace_bytes, void *stream) {
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "plan is null");
    const linear_desc &d = p->d;
    if (!(d.flags & CONV3D_F_BIAS)) bias = nullptr;
    else if (!bias) return api_fail(CONV3D_ERR_INVALID_ARG, "the plan needs a bias");
    if (!(d.flags & CONV3D_F_RESIDUAL)) residual = nullptr;
    else if (!residual && d.m) return api_fail(CONV3D_ERR_INVALID_ARG, "the plan needs a residual");
    if (!(d.flags & CONV3D_F_PREACT)) preact = nullptr;
    else if (!preact && d.m) return api_fail(CONV3D_ERR_INVALID_ARG, "the plan needs preact");
    if (!w || (d.m && (!x || !y))) return api_fail(CONV3D_ERR_INVALID_ARG, "x, w and y are required");
    if (misaligned(x) || misaligned(w) || misaligned(bias) || misaligned(residual) || misaligned(y) ||
        misaligned(preact))
        return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    conv3d_status st = check_workspace(workspace, workspace_bytes, p->fwd.partial_bytes);
    if (st != CONV3D_OK) return st;
    const Span sx(x, d.m, d.k, p->xs), sw(w, d.n, d.k, d.k), sb(bias, 1, d.n, d.n), sr(residual, d.m, d.n, p->rs),
        sy(y, d.m, d.n, p->ys), sz(preact, d.m, d.n, d.n), sws(workspace, p->fwd.partial_bytes);
    for (const Span *o : {&sy, &sz, &sws})
        if (o->meets(sx) || o->meets(sw) || o->meets(sb) || o->meets(sr))
            return api_fail(CONV3D_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
    if (sy.meets(sz) || sws.meets(sy) || sws.meets(sz))
        return api_fail(CONV3D_ERR_INVALID_ARG, "y, preact and the workspace overlap");
    if (d.m == 0) return api_ok();
    st = api_check_device();
    if (st != CONV3D_OK) return st;
    c3d::GemmParams q = {};
    fill(q, p->fwd, d.m, d.n, d.k, (d.flags & CONV3D_F_BF16) ? 1 : 0, workspace);
    q.p = in16(w);
    q.p_stride = d.k;
    q.q = in16(x);
    q.q_stride = p->xs;
    q.bias = in16(bias);
    q.res = in16(residual);
    q.res_stride = p->rs;
    q.z = out16(preact);
    q.y = out16(y);
    q.y_stride = p->ys;
    q.act = d.act;
    return launched(c3d::launch_gemm(q, p->fwd.tile, c3d::kGemmForward, static_cast<hipStream_t>(stream)), "linear");
}

size_t linear_backward_workspace(linear_plan_t p) { return p ? p->back_bytes : 0; }

conv3d_status linear_backward(linear_plan_t p, const void *dy, const void *x, const void *w, const void *preact,
                              void *dx, void *dw, void *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "plan is null");
    const linear_desc &d = p->d;
    const bool act = d.act != CONV3D_ACT_NONE;
    if (!dx && !dw && !dbias) return api_fail(CONV3D_ERR_INVALID_ARG, "no gradient is asked for");
    if (!dw) x = nullptr;
    if (!dx) w = nullptr;
    if (!act) preact = nullptr;
    if ((dx && !w) || (d.m && (!dy || (dw && !x) || (act && !preact))))
        return api_fail(CONV3D_ERR_INVALID_ARG, "dy is required, w for dx, x for dw, and preact for an activation");
    if (misaligned(dy) || misaligned(x) || misaligned(w) || misaligned(preact) || misaligned(dx) || misaligned(dw) ||
        misaligned(dbias))
        return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
    conv3d_status st = check_workspace(workspace, workspace_bytes, p->back_bytes);
    if (st != CONV3D_OK) return st;
    const Span in[] = {Span(dy, d.m, d.n, p->ys), Span(x, d.m, d.k, p->xs), Span(w, d.n, d.k, d.k),
                       Span(preact, d.m, d.n, d.n)};
    const Span res[] = {Span(dx, d.m, d.k, p->xs), Span(dw, d.n, d.k, d.k), Span(dbias, 1, d.n, d.n),
                        Span(workspace, p->back_bytes)};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : in)
            if (res[i].meets(s))
                return api_fail(CONV3D_ERR_INVALID_ARG, "a gradient or the workspace overlaps an input");
        for (int j = 0; j < i; ++j)
            if (res[i].meets(res[j]))
                return api_fail(CONV3D_ERR_INVALID_ARG, "the gradients and the workspace overlap");
    }
    st = api_check_device();
    if (st != CONV3D_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int bf16 = (d.flags & CONV3D_F_BF16) ? 1 : 0;
    hipError_t e = hipSuccess;
    if (d.m == 0) {  // sums over no rows
        if (dw) e = c3d::launch_zero_rows(out16(dw), d.n, d.k, d.k, s);
        if (e == hipSuccess && dbias) e = c3d::launch_zero_rows(out16(dbias), 1, d.n, d.n, s);
        return launched(e, "linear_backward");
    }
    char *ws = static_cast<char *>(workspace);
    const _Float16 *dz = in16(dy);
    int64_t dz_stride = p->ys;
    c3d::ColumnSumParams cs = {};
    // without an activation dbias can come straight from dy
    const bool direct = !act && dbias && c3d::sum_whole_columns(d.m, d.n);
    if (dbias) {
        cs.part = reinterpret_cast<float *>(ws + p->off_col);
        cs.in16 = direct ? in16(dy) : nullptr;
        cs.stride = p->ys;
        cs.out0 = out16(dbias);
        cs.rows = direct ? (int32_t)d.m : p->strips;
        cs.cols = cs.split = d.n;
        cs.bf16 = bf16;
    }
    if (act || (dbias && !direct)) {
        c3d::ActGradParams a = {};
        a.dy = in16(dy);
        a.dy_stride = p->ys;
        a.z = in16(preact);
        a.dz = act ? reinterpret_cast<_Float16 *>(ws) : nullptr;
        a.colpart = dbias ? const_cast<float *>(cs.part) : nullptr;
        a.m = d.m;
        a.n = d.n;
        a.act = d.act;
        a.bf16 = bf16;
        a.strips = p->strips;
        e = c3d::launch_act_grad(a, s);
        if (act) {
            dz = a.dz;
            dz_stride = d.n;
        }
    }
    const bool pair = dx && dw && p->pair;
    if (e == hipSuccess && dbias && !pair) e = c3d::launch_column_sum(cs, s);
    c3d::GemmParams qx = {}, qw = {};
    char *part = ws + p->off_part;
    if (dx) {
        fill(qx, pair ? p->pair_dx : p->dx, d.m, d.k, d.n, bf16, part);
        qx.p = in16(w);
        qx.p_stride = d.k;
        qx.q = dz;
        qx.q_stride = dz_stride;
        qx.y = out16(dx);
        qx.y_stride = p->xs;
    }
    if (dw) {
        fill(qw, pair ? p->pair_dw : p->dw, d.n, d.k, d.m, bf16, pair ? part + p->pair_dx.partial_bytes : part);
        qw.p = in16(x);
        qw.p_stride = p->xs;
        qw.q = dz;
        qw.q_stride = dz_stride;
        qw.y = out16(dw);
        qw.y_stride = d.k;
    }
    if (pair) {
        if (e == hipSuccess) e = c3d::launch_gemm_pair(qx, qw, p->pair_dx.tile, cs, s);
    } else {
        if (e == hipSuccess && dx) e = c3d::launch_gemm(qx, p->dx.tile, c3d::kGemmDx, s);
        if (e == hipSuccess && dw) e = c3d::launch_gemm(qw, p->dw.tile, c3d::kGemmDw, s);
    }
    return launched(e, "linear_backward");
}

// -------------------------------------------------------------- layernorm

static conv3d_status ln_sizes(int64_t rows, int32_t c, int64_t x_stride, int64_t y_stride, int64_t *xs, int64_t *ys) {
    if (rows < 0 || c < 1) return api_fail(CONV3D_ERR_INVALID_ARG, "rows >= 0 and c >= 1 needed");
    if (c % 8 || c > c3d::kLnMaxC)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "c (%d) must be a multiple of 8 up to %d", c, c3d::kLnMaxC);
    if (rows >= (int64_t)1 << 40) return api_fail(CONV3D_ERR_UNSUPPORTED, "too many rows");
    conv3d_status st = row_stride(x_stride, c, "x_stride", xs);
    if (st == CONV3D_OK) st = row_stride(y_stride, c, "y_stride", ys);
    return st;
}

static conv3d_status ln_entry(const void *x, const void *gamma, const void *beta, void *y, void *stats, int64_t rows,
                              int32_t c, int64_t x_stride, int64_t y_stride, float eps, void *stream, int bf16) {
    int64_t xs, ys;
    conv3d_status st = ln_sizes(rows, c, x_stride, y_stride, &xs, &ys);
    if (st != CONV3D_OK) return st;
    if (!(eps >= 0.0f)) return api_fail(CONV3D_ERR_INVALID_ARG, "eps must be non-negative");
    if (rows && (!x || !y)) return api_fail(CONV3D_ERR_INVALID_ARG, "x and y are required");
    if (misaligned(x) || misaligned(y) || misaligned(gamma) || misaligned(beta) || misaligned(stats, 8))
        return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned (stats: 8)");
    const Span sx(x, rows, c, xs), sy(y, rows, c, ys), ss(stats, rows, 2, 2, 4), sg(gamma, 1, c, c), sb(beta, 1, c, c);
    if ((sy.meets(sx) && !(x == y && xs == ys)) || sy.meets(sg) || sy.meets(sb))
        return api_fail(CONV3D_ERR_INVALID_ARG, "y overlaps an input");
    if (ss.meets(sx) || ss.meets(sy) || ss.meets(sg) || ss.meets(sb))
        return api_fail(CONV3D_ERR_INVALID_ARG, "stats overlaps a tensor");
    if (rows == 0) return api_ok();
    st = api_check_device();
    if (st != CONV3D_OK) return st;
    c3d::LnParams q = {};
    q.x = in16(x);
    q.gamma = in16(gamma);
    q.beta = in16(beta);
    q.y = out16(y);
    q.stats = static_cast<float2 *>(stats);
    q.rows = rows;
    q.x_stride = xs;
    q.y_stride = ys;
    q.c = c;
    q.eps = eps;
    q.bf16 = bf16;
    return launched(c3d::launch_layernorm(q, static_cast<hipStream_t>(stream)), "layernorm");
}

conv3d_status layernorm(const void *x, const void *gamma, const void *beta, void *y, void *stats, int64_t rows,
                        int32_t c, int64_t x_stride, int64_t y_stride, float eps, void *stream) {
    return ln_entry(x, gamma, beta, y, stats, rows, c, x_stride, y_stride, eps, stream, 0);
}

conv3d_status layernorm_bf16(const void *x, const void *gamma, const void *beta, void *y, void *stats, int64_t rows,
                             int32_t c, int64_t x_stride, int64_t y_stride, float eps, void *stream) {
    return ln_entry(x, gamma, beta, y, stats, rows, c, x_stride, y_stride, eps, stream, 1);
}

size_t layernorm_backward_workspace(int64_t rows, int32_t c) {
    if (rows < 1 || c < 1 || c % 8 || c > c3d::kLnMaxC || rows >= (int64_t)1 << 40) return 0;
    return (size_t)c3d::ln_grad_blocks(rows, c) * 2 * c * 4;
}

static conv3d_status ln_back_entry(const void *dy, const void *x, const void *gamma, const void *stats,
                                   const void *dres, void *dx, void *dgamma, void *dbeta, int64_t rows, int32_t c,
                                   int64_t x_stride, int64_t y_stride, void *workspace, size_t workspace_bytes,
                                   void *stream, int bf16) {
    int64_t xs, ys;
    conv3d_status st = ln_sizes(rows, c, x_stride, y_stride, &xs, &ys);
    if (st != CONV3D_OK) return st;
    if (rows && (!dy || !x || !stats || !dx))
        return api_fail(CONV3D_ERR_INVALID_ARG, "dy, x, stats and dx are required");
    if (misaligned(dy) || misaligned(x) || misaligned(gamma) || misaligned(stats, 8) || misaligned(dres) ||
        misaligned(dx) || misaligned(dgamma, 2) || misaligned(dbeta, 2))
        return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned (stats: 8)");
    const size_t need = dgamma || dbeta ? layernorm_backward_workspace(rows, c) : 0;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != CONV3D_OK) return st;
    const Span sdy(dy, rows, c, ys), sx(x, rows, c, xs), sdr(dres, rows, c, xs), sg(gamma, 1, c, c),
        ss(stats, rows, 2, 2, 4), sdx(dx, rows, c, xs);
    if ((sdx.meets(sdy) && !(dx == dy && xs == ys)) || (sdx.meets(sx) && dx != x) || (sdx.meets(sdr) && dx != dres) ||
        sdx.meets(sg) || sdx.meets(ss))
        return api_fail(CONV3D_ERR_INVALID_ARG, "dx overlaps an input");
    const Span res[] = {sdx, Span(dgamma, 1, c, c), Span(dbeta, 1, c, c), Span(workspace, need)};
    for (int i = 1; i < 4; ++i) {
        for (const Span *s : {&sdy, &sx, &sdr, &sg, &ss})
            if (res[i].meets(*s))
                return api_fail(CONV3D_ERR_INVALID_ARG, "a gradient or the workspace overlaps an input");
        for (int j = 0; j < i; ++j)
            if (res[i].meets(res[j]))
                return api_fail(CONV3D_ERR_INVALID_ARG, "the gradients and the workspace overlap");
    }
    st = api_check_device();
    if (st != CONV3D_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (rows == 0) {  // sums over no rows
        hipError_t e = hipSuccess;
        if (dgamma) e = c3d::launch_zero_rows(out16(dgamma), 1, c, c, s);
        if (e == hipSuccess && dbeta) e = c3d::launch_zero_rows(out16(dbeta), 1, c, c, s);
        return launched(e, "layernorm_backward");
    }
    c3d::LnGradParams q = {};
    q.dy = in16(dy);
    q.x = in16(x);
    q.gamma = in16(gamma);
    q.dres = in16(dres);
    q.stats = static_cast<const float2 *>(stats);
    q.dx = out16(dx);
    q.dgamma = out16(dgamma);
    q.dbeta = out16(dbeta);
    q.part = need ? static_cast<float *>(workspace) : nullptr;
    q.rows = rows;
    q.x_stride = xs;
    q.y_stride = ys;
    q.c = c;
    q.bf16 = bf16;
    return launched(c3d::launch_layernorm_grad(q, s), "layernorm_backward");
}

conv3d_status layernorm_backward(const void *dy, const void *x, const void *gamma, const void *stats,
                                 const void *dres, void *dx, void *dgamma, void *dbeta, int64_t rows, int32_t c,
                                 int64_t x_stride, int64_t y_stride, void *workspace, size_t workspace_bytes,
                                 void *stream) {
    return ln_back_entry(dy, x, gamma, stats, dres, dx, dgamma, dbeta, rows, c, x_stride, y_stride, workspace,
                         workspace_bytes, stream, 0);
}

conv3d_status layernorm_backward_bf16(const void *dy, const void *x, const void *gamma, const void *stats,
                                      const void *dres, void *dx, void *dgamma, void *dbeta, int64_t rows,
                                      int32_t c, int64_t x_stride, int64_t y_stride, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    return ln_back_entry(dy, x, gamma, stats, dres, dx, dgamma, dbeta, rows, c, x_stride, y_stride, workspace,
                         workspace_bytes, stream, 1);
}

// ----------------------------------------------------------------- rope3d

}  // extern "C"

struct rope3d_plan_s {
    rope3d_desc d;
    int64_t tokens;
    int64_t qs[3], ks[3], qos[3], kos[3];
    bool folds_in, folds_out;  // the inputs' or the outputs' strides put different elements on one address
    c3d::RopeParams prm;  // pointers, strides and direction filled per call
};

namespace {

conv3d_status rope_strides(const int64_t *given, int64_t tokens, int heads, int dim, const char *what, int64_t *out) {
    if (!given[0] && !given[1] && !given[2]) {
        out[2] = dim;
        out[1] = (int64_t)heads * dim;
        out[0] = tokens * out[1];
        return CONV3D_OK;
    }
    for (int i = 0; i < 3; ++i) {
        if (given[i] < 0 || given[i] % 8)
            return api_fail(CONV3D_ERR_INVALID_ARG, "%s (%lld) must be a non-negative multiple of 8", what,
                            (long long)given[i]);
        if (given[i] >= (int64_t)1 << 40) return api_fail(CONV3D_ERR_UNSUPPORTED, "%s is too large", what);
        out[i] = given[i];
    }
    return CONV3D_OK;
}

Span rope_span(const void *p, const int64_t *s, int64_t n, int64_t tokens, int heads, int dim) {
    if (n < 1 || tokens < 1 || heads < 1) return Span(nullptr, (size_t)0);
    return Span(p, (size_t)((n - 1) * s[0] + (tokens - 1) * s[1] + (heads - 1) * s[2] + dim) * 2);
}

bool same3(const int64_t *a, const int64_t *b) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

// Heads of dim elements at base + (sample, token, head) . strides: whether two of
// them share an element, by search over the differences of their indices.  A
// term of the search is a stride and the range of its index (or of the difference
// of two); from the largest stride down, only such indices are followed as the
// smaller ones can still bring back, a handful for layouts whose strides nest.
class HeadSearch {
    struct Term {
        int64_t stride, lo, hi;
    };
    Term t_[6];
    int64_t below_[7], above_[7];  // how far the terms from i on reach down and up
    int n_ = 0;
    const int64_t dim_;
    const bool itself_;   // one tensor: different indices only
    bool twice_ = false;  // two of its indices step by the same stride
    int64_t left_ = 1 << 16;       // steps until the search counts as unanswered

    bool search(int i, int64_t at, bool same) {
        if (i == n_) return at > -dim_ && at < dim_ && !(itself_ && same);
        const Term &t = t_[i];
        if (t.stride == 0) return search(i + 1, at, false);
        // at + c stride + rest in (-dim, dim), rest in [-below, above]
        const int64_t from = -dim_ + 1 - above_[i + 1] - at, to = dim_ - 1 + below_[i + 1] - at;
        int64_t c = from > 0 ? (from + t.stride - 1) / t.stride : -(-from / t.stride);
        int64_t last = to >= 0 ? to / t.stride : -((-to + t.stride - 1) / t.stride);
        if (c < t.lo) c = t.lo;
        if (last > t.hi) last = t.hi;
        for (; c <= last && left_ > 0; ++c) {
            --left_;
            if (search(i + 1, at + c * t.stride, same && c == 0)) return true;
        }
        return false;
    }

public:
    HeadSearch(int64_t dim, bool itself) : dim_(dim), itself_(itself) {}
    // lo <= 0 <= hi; terms of one stride are one
    void add(int64_t stride, int64_t lo, int64_t hi) {
        if (lo == hi) return;
        int i = 0;
        while (i < n_ && t_[i].stride > stride) ++i;
        if (i < n_ && t_[i].stride == stride) {
            t_[i].lo += lo;
            t_[i].hi += hi;
            twice_ = true;
            return;
        }
        for (int j = n_++; j > i; --j) t_[j] = t_[j - 1];
        t_[i] = {stride, lo, hi};
    }
    bool found(int64_t offset) {
        below_[n_] = above_[n_] = 0;
        for (int i = n_ - 1; i >= 0; --i) {
            below_[i] = below_[i + 1] - t_[i].lo * t_[i].stride;
            above_[i] = above_[i + 1] + t_[i].hi * t_[i].stride;
        }
        return (itself_ && twice_) || search(0, offset, true);
    }
    bool unanswered() const { return left_ <= 0; }
};

// Whether heads of one tensor share an element (or cannot be shown not to).
bool rope_folds(const rope3d_desc &d, int64_t tokens, const int64_t *s, int heads) {
    if (d.n < 1 || tokens < 1 || heads < 1) return false;
    const int64_t ext[3] = {d.n, tokens, heads};
    HeadSearch h(d.head_dim, true);
    for (int i = 0; i < 3; ++i) h.add(s[i], -(ext[i] - 1), ext[i] - 1);
    return h.found(0) || h.unanswered();
}

// Whether heads of two tensors share an element.
bool rope_share(const rope3d_desc &d, int64_t tokens, const void *a, const int64_t *sa, int ha, const void *b,
                const int64_t *sb, int hb) {
    if (!rope_span(a, sa, d.n, tokens, ha, d.head_dim).meets(rope_span(b, sb, d.n, tokens, hb, d.head_dim)))
        return false;
    const int64_t ea[3] = {d.n, tokens, ha}, eb[3] = {d.n, tokens, hb};
    HeadSearch h(d.head_dim, false);
    for (int i = 0; i < 3; ++i) {
        h.add(sa[i], -(ea[i] - 1), 0);
        h.add(sb[i], 0, eb[i] - 1);
    }
    const int64_t bytes = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    return h.found(bytes / 2);  // both are 16-byte aligned
}

conv3d_status rope_run(rope3d_plan_t p, const void *q, const void *k, void *qo, void *ko, const void *positions,
                       int32_t t_offset, void *stream, bool inverse) {
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "plan is null");
    const rope3d_desc &d = p->d;
    const bool given = (d.flags & CONV3D_F_POSITIONS) != 0;
    if (!d.heads_k) k = ko = nullptr;
    if (!given) positions = nullptr;
    const bool any = d.n > 0 && p->tokens > 0;
    if (any && (!q || !qo || (d.heads_k && (!k || !ko)) || (given && !positions)))
        return api_fail(CONV3D_ERR_INVALID_ARG, "q and its output are required, k and its output with heads_k, and "
                                                "positions with CONV3D_F_POSITIONS");
    if (misaligned(q) || misaligned(k) || misaligned(qo) || misaligned(ko) || misaligned(positions, 4))
        return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned (positions: 4)");
    const int64_t *qi = inverse ? p->qos : p->qs, *qj = inverse ? p->qs : p->qos;
    const int64_t *ki = inverse ? p->kos : p->ks, *kj = inverse ? p->ks : p->kos;
    auto clash = [&](const void *in, const int64_t *si, const void *out, const int64_t *so, int heads) {
        if (in == out && same3(si, so)) return false;
        return rope_span(in, si, d.n, p->tokens, heads, d.head_dim)
            .meets(rope_span(out, so, d.n, p->tokens, heads, d.head_dim));
    };
    if (clash(q, qi, qo, qj, d.heads_q) || clash(k, ki, ko, kj, d.heads_k))
        return api_fail(CONV3D_ERR_INVALID_ARG, "an output overlaps its input without being it");
    if (!any) return api_ok();
    if (inverse ? p->folds_in : p->folds_out)
        return api_fail(CONV3D_ERR_INVALID_ARG, "different elements of an output overlap");
    if (d.heads_k && (rope_share(d, p->tokens, qo, qj, d.heads_q, ko, kj, d.heads_k) ||
                      rope_share(d, p->tokens, qo, qj, d.heads_q, k, ki, d.heads_k) ||
                      rope_share(d, p->tokens, ko, kj, d.heads_k, q, qi, d.heads_q)))
        return api_fail(CONV3D_ERR_INVALID_ARG, "an output overlaps the other output or its input");
    const Span pos(positions, positions ? (size_t)d.n * p->tokens * 12 : 0);
    if (pos.meets(rope_span(qo, qj, d.n, p->tokens, d.heads_q, d.head_dim)) ||
        pos.meets(rope_span(ko, kj, d.n, p->tokens, d.heads_k, d.head_dim)))
        return api_fail(CONV3D_ERR_INVALID_ARG, "an output overlaps the positions");
    conv3d_status st = api_check_device();
    if (st != CONV3D_OK) return st;
    c3d::RopeParams r = p->prm;
    r.q.in = in16(q);
    r.q.out = out16(qo);
    r.k.in = in16(k);
    r.k.out = out16(ko);
    for (int i = 0; i < 3; ++i) {
        r.q.in_stride[i] = qi[i];
        r.q.out_stride[i] = qj[i];
        r.k.in_stride[i] = ki[i];
        r.k.out_stride[i] = kj[i];
    }
    r.positions = static_cast<const int32_t *>(positions);
    r.t_offset = t_offset;
    r.inverse = inverse ? 1 : 0;
    return launched(c3d::launch_rope3d(r, static_cast<hipStream_t>(stream)), "rope3d");
}

}  // namespace

extern "C" {

conv3d_status rope3d_plan(const rope3d_desc *d, rope3d_plan_t *out) {
    if (!d || !out) return api_fail(CONV3D_ERR_INVALID_ARG, "desc and out are required");
    if (d->n < 0 || d->t < 0 || d->h < 0 || d->w < 0)
        return api_fail(CONV3D_ERR_INVALID_ARG, "n, t, h and w must not be negative");
    if (d->heads_q < 1 || d->heads_k < 0 || d->head_dim < 1)
        return api_fail(CONV3D_ERR_INVALID_ARG, "heads_q and head_dim must be positive, heads_k not negative");
    if (d->pairing != ROPE3D_PAIR_ADJACENT && d->pairing != ROPE3D_PAIR_HALVES)
        return api_fail(CONV3D_ERR_INVALID_ARG, "unknown pairing %d", d->pairing);
    const uint32_t known = CONV3D_F_POSITIONS | CONV3D_F_BF16;
    if (d->flags & ~known) return api_fail(CONV3D_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags & ~known);
    const int dims[3] = {d->dim_t, d->dim_h, d->dim_w};
    int64_t sum = 0;
    for (int v : dims) {
        if (v < 0 || v % 2) return api_fail(CONV3D_ERR_INVALID_ARG, "dim_t, dim_h and dim_w must be even and >= 0");
        sum += v;
    }
    if (sum < 2 || sum > d->head_dim)
        return api_fail(CONV3D_ERR_INVALID_ARG, "dim_t + dim_h + dim_w must be 2 .. head_dim (%d)", d->head_dim);
    if (!(d->base > 0.0) || !std::isfinite(d->base))
        return api_fail(CONV3D_ERR_INVALID_ARG, "base must be positive and finite");
    if (d->head_dim % 8 || d->head_dim > 512 || sum > 2 * c3d::kRopeMaxPairs)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 up to 512, the dims up to %d together",
                        2 * c3d::kRopeMaxPairs);
    if (d->pairing == ROPE3D_PAIR_HALVES && sum % 16)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "ROPE3D_PAIR_HALVES needs dims that are a multiple of 16 together");
    if (d->heads_q > 16384 || d->heads_k > 16384) return api_fail(CONV3D_ERR_UNSUPPORTED, "too many heads");
    const double per_sample = (double)d->t * d->h * d->w, total = per_sample * d->n;
    if (per_sample >= 2147483648.0 || total >= 2147483648.0 || (double)d->h * d->w >= 2147483648.0)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "2^31 tokens or more");
    rope3d_plan_s *p = new (std::nothrow) rope3d_plan_s();
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "out of host memory");
    p->d = *d;
    p->tokens = (int64_t)d->t * d->h * d->w;
    conv3d_status st = rope_strides(d->q_stride, p->tokens, d->heads_q, d->head_dim, "q_stride", p->qs);
    if (st == CONV3D_OK) st = rope_strides(d->k_stride, p->tokens, d->heads_k, d->head_dim, "k_stride", p->ks);
    if (st == CONV3D_OK)
        st = rope_strides(d->q_out_stride, p->tokens, d->heads_q, d->head_dim, "q_out_stride", p->qos);
    if (st == CONV3D_OK)
        st = rope_strides(d->k_out_stride, p->tokens, d->heads_k, d->head_dim, "k_out_stride", p->kos);
    // every offset within a tensor, in bytes, fits 64 bits
    const auto length = [&](const int64_t *s, int heads) {
        return d->n && p->tokens && heads
                   ? (double)(d->n - 1) * s[0] + (double)(p->tokens - 1) * s[1] + (double)(heads - 1) * s[2]
                   : 0.0;
    };
    if (st == CONV3D_OK)
        for (const auto &t : {std::pair<const int64_t *, int>{p->qs, d->heads_q}, {p->qos, d->heads_q},
                              {p->ks, d->heads_k}, {p->kos, d->heads_k}})
            if (length(t.first, t.second) >= kMaxElements)
                st = api_fail(CONV3D_ERR_UNSUPPORTED, "a tensor is 2^48 elements long or longer");
    if (st != CONV3D_OK) {
        delete p;
        return st;
    }
    p->folds_in = rope_folds(*d, p->tokens, p->qs, d->heads_q) || rope_folds(*d, p->tokens, p->ks, d->heads_k);
    p->folds_out = rope_folds(*d, p->tokens, p->qos, d->heads_q) || rope_folds(*d, p->tokens, p->kos, d->heads_k);
    c3d::RopeParams &r = p->prm;
    r.tokens = p->tokens;
    r.n = d->n;
    r.h = d->h;
    r.w = d->w;
    r.head_dim = d->head_dim;
    r.pairs = (int32_t)(sum / 2);
    r.end_t = d->dim_t / 2;
    r.end_h = (d->dim_t + d->dim_h) / 2;
    r.halves = d->pairing == ROPE3D_PAIR_HALVES;
    r.bf16 = (d->flags & CONV3D_F_BF16) ? 1 : 0;
    r.q.heads = d->heads_q;
    r.k.heads = d->heads_k;
    int pr = 0;
    for (int v : dims)
        for (int i = 0; i < v / 2; ++i)
            r.turns[pr++] = std::pow(d->base, -2.0 * i / v) / 6.283185307179586476925286766559;
    *out = p;
    return api_ok();
}

void rope3d_plan_destroy(rope3d_plan_t p) { delete p; }

conv3d_status rope3d_forward(rope3d_plan_t p, const void *q, const void *k, void *q_out, void *k_out,
                             const void *positions, int32_t t_offset, void *stream) {
    return rope_run(p, q, k, q_out, k_out, positions, t_offset, stream, false);
}

conv3d_status rope3d_backward(rope3d_plan_t p, const void *dq_out, const void *dk_out, void *dq, void *dk,
                              const void *positions, int32_t t_offset, void *stream) {
    return rope_run(p, dq_out, dk_out, dq, dk, positions, t_offset, stream, true);
}

}  // extern "C"
