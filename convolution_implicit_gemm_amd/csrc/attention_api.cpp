// Host side of attention as declared in include/conv3d.h: validation, planning, and
// launches on the caller's stream.  Nothing here synchronises the device or
// allocates device memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>

#include "token_checks.h"

using namespace c3d;

struct attention_plan_s {
    attention_desc d;
    int64_t qs[3], ks[3], vs[3], os[3];
    bool folds_q, folds_k, folds_v, folds_o;  // strides that put different elements on one address
    AttnTileKind kind;
    AttnGradKinds grad;
    int64_t grid;
    size_t off_ml, fwd_bytes, off_delta, off_dk, off_dv, back_bytes;
    AttnParams prm;  // pointers filled per call
};

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxOffset = (int64_t)1 << 30;
constexpr int kAttnCUs = 256, kMaxPieces = 128;

conv3d_status attn_strides(const int64_t *given, int64_t tokens, int heads, int dim, const char *what, int64_t *out) {
    if (!given[0] && !given[1] && !given[2]) {
        out[2] = dim;
        out[1] = (int64_t)heads * dim;
        out[0] = tokens * out[1];
    } else {
        for (int i = 0; i < 3; ++i) {
            if (given[i] < 0 || given[i] % 8)
                return api_fail(CONV3D_ERR_INVALID_ARG, "%s (%lld) must be a non-negative multiple of 8", what,
                                (long long)given[i]);
            if (given[i] >= (int64_t)1 << 40) return api_fail(CONV3D_ERR_UNSUPPORTED, "%s is too large", what);
            out[i] = given[i];
        }
        if (tokens > 1 && out[1] < dim)
            return api_fail(CONV3D_ERR_INVALID_ARG, "%s: tokens (%lld) overlap within a head of %d", what,
                            (long long)out[1], dim);
    }
    if (tokens > 1 && out[1] > (int64_t)1 << 20)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "%s between tokens (%lld) is above 2^20", what, (long long)out[1]);
    if (tokens <= 1) out[1] = dim;  // never used to move
    return CONV3D_OK;
}

// ---- which kernel, and how many pieces.  Times in us, from the kernels' measured steps.

// One operator's problem: `heads` independent ones of `rows` rows, each of which walks `most` elements
// of the other side, `mean` on average.
struct Problem {
    int64_t heads, rows;
    double most, mean;
    int dim;
};
struct Choice {
    AttnTileKind kind;
    int pieces;
    double us;
};

enum Pass { kForward, kDq, kDkv };

// Fitted to 3700 timed calls (heads of 32, 64, 96 and 128, 64 to 9216 tokens, 2 to 48 heads, with and
// without a mask, 1 to 16 pieces): over those calls the choice was 1 to 3% off the fastest kernel on average.
// Per pass: the time of a call besides its steps (kDkv: with that of the row sums), of a
// workgroup besides its steps, what joining the waves adds to that, the share of the longest workgroup
// that the end of unequal ones waits for, a second launch to join pieces, and the partials' us per 2^20 or so values.
struct PassCost {
    double call, group, joined, tail, join, part;
};
constexpr PassCost kPass[3] = {
    {4.6, 1.4, 0.0, 0.29, 3.9, 2.4}, {1.0, 4.5, 2.0, 0.2, 3.0, 2.0}, {9.7, 0.0, 1.4, 0.28, 3.4, 2.7}};
// A step of a workgroup by pass, tile (64, 128, 256 rows) and padded head (32, 64, 96, 128).
constexpr double kStepUs[3][3][4] = {
    {{0.48, 0.73, 1.26, 1.47}, {0.89, 1.20, 1.60, 2.00}, {1.02, 1.17, 1.43, 1.53}},
    {{0.33, 0.84, 1.40, 1.70}, {0.92, 1.48, 2.07, 2.63}, {1.02, 1.50, 1.93, 2.27}},
    {{0.69, 1.49, 2.03, 3.05}, {0.72, 1.21, 1.71, 2.21}, {1.45, 2.03, 2.81, 3.95}}};
// Pieces are taken where they save a tenth: their join is a launch more.
constexpr double kPieceMargin = 1.1;

AttnTileKind forced_kind(AttnTileKind otherwise, bool few) {
    const char *v = getenv("CONV3D_ATTENTION_TILE");
    if (!v) return otherwise;
    for (AttnTileKind k : {kAttnFew, kAttn64, kAttn128, kAttn256})
        if ((k != kAttnFew || few) && strcmp(v, attn_tile(k).name) == 0) return k;
    return otherwise;
}
int forced_pieces(int otherwise) {
    const char *v = getenv("CONV3D_ATTENTION_SPLITS");
    const int k = v ? atoi(v) : 0;
    return k < 1 ? otherwise : k > kMaxPieces ? kMaxPieces : k;
}

Choice choose(Pass pass, const Problem &w, bool splits) {
    Choice best = {kAttn256, 1, -1.0};
    const bool few = pass == kForward && w.rows <= kAttnFewRows;
    const AttnTileKind only = forced_kind(few ? kAttnFew : kAttn256, few);
    const bool forced = getenv("CONV3D_ATTENTION_TILE") != nullptr;
    for (AttnTileKind kind : {kAttn256, kAttn128, kAttn64, kAttnFew}) {
        if (forced ? kind != only : (kind == kAttnFew) != few) continue;
        const AttnTileSize t = attn_tile(kind);
        const int64_t tiles = w.heads * ((w.rows + t.rows - 1) / t.rows);
        const double keys = pass == kDkv ? attn_grad_step(kind) : t.keys;
        for (int z = 1; z <= kMaxPieces; z += z < 8 ? 1 : z < 16 ? 2 : z < 32 ? 4 : 16) {
            const int pieces = forced_pieces(z);
            const double most = std::ceil(std::ceil(w.most / keys) / pieces), mean = w.mean / keys / pieces;
            if (z > 1 && (!splits || z > w.most / keys || tiles * z > (few ? 1 : 4) * kAttnCUs)) break;
            const double units = (double)tiles * pieces, rounds = units / kAttnCUs;
            double us;
            if (kind == kAttnFew) {
                // a step's latency (from the last-level cache or from memory), the first ones' longer, or all
                // workgroups' shares of the memory's rate
                const bool cached = 4.0 * w.heads * w.most * w.dim < 2e8;
                const double least = w.dim > 64 ? (cached ? 0.87 : 1.45) : (cached ? 0.61 : 0.8);
                const double share = (units < kAttnCUs ? units : kAttnCUs) * 512.0 * w.dim / 5.8e6;
                const double step = std::sqrt(std::hypot(least * least, share * share));
                us = 3.6 + std::ceil(rounds) * most * step + 0.4 * least * (most < 5 ? most : 5) +
                     (pieces > 1 ? 2.2 + 0.02 * pieces : 0.0);
            } else {
                const PassCost &k = kPass[pass];
                const double c = kStepUs[pass][kind - kAttn64][(w.dim - 1) / 32], fixed = k.group + (kind == kAttn256 ? 0.0 : k.joined);
                // equal workgroups run in whole rounds; unequal ones, longest first, fill up
                const double even = std::ceil(rounds) * (most * c + fixed);
                const double fill = rounds * (mean * c + fixed) + k.tail * most * c, longest = most * c + fixed;
                us = k.call + (w.mean > 0.95 * w.most ? even : fill > longest ? fill : longest);
            }
            if (pieces > 1 && kind != kAttnFew)
                us = kPieceMargin * (us + kPass[pass].join + (double)w.heads * w.rows * w.dim * pieces * kPass[pass].part / 1e6);
            if (best.us < 0.0 || us < best.us) best = {kind, pieces, us};
            if (pieces != z) break;  // forced
        }
    }
    return best;
}

// dq beside dk and dv in one launch of tiles of one kind, after a launch for the rows' numbers.  That is
// worth it where either alone leaves CUs idle: 1024 tokens, 8 heads of 128 46 -> 35 us, 256
// tokens 26 -> 22; 2048 tokens, 256 workgroups each, 81 and 82.
double together_us(AttnTileKind kind, const Problem &q, const Problem &kv, int pieces) {
    const PassCost &kq = kPass[kDq], &kk = kPass[kDkv];
    const int rows = attn_tile(kind).rows, column = (q.dim - 1) / 32;
    const double cq = kStepUs[kDq][kind - kAttn64][column], ck = kStepUs[kDkv][kind - kAttn64][column];
    const double units_q = (double)q.heads * ((q.rows + rows - 1) / rows),
                 units_k = (double)kv.heads * ((kv.rows + rows - 1) / rows) * pieces;
    const double keys = attn_tile(kind).keys, tokens = attn_grad_step(kind);
    const double fq = kq.group + kq.joined, fk = kk.group + kk.joined;
    const double longest_q = std::ceil(q.most / keys) * cq + fq, longest_k = std::ceil(std::ceil(kv.most / tokens) / pieces) * ck + fk;
    const double longest = longest_q > longest_k ? longest_q : longest_k;
    const double share = (units_q * (q.mean / keys * cq + fq) + units_k * (kv.mean / tokens / pieces * ck + fk)) / kAttnCUs;
    const double work = units_q + units_k <= kAttnCUs ? longest : share + 0.3 * longest;
    // four waves to a row meet at the end of the 64-row tiles, two in the others: 64 tokens, heads of 64 and
    // 128, 13.7 and 20.6 us against 11.4 and 15.9
    double us = 5.5 + (work > longest ? work : longest) + (kind == kAttn64 ? 0.037 * q.dim : 0.0);
    if (pieces > 1) us += kk.join + (double)kv.heads * kv.rows * kv.dim * pieces * kk.part / 1e6;
    return us;
}
// Of kPass[kDkv].call, the launch for the rows' numbers that dk and dv were timed with.
constexpr double kRowsUs = 5.0;

// The tensors of a call.
struct Tensors {
    const attention_plan_s &p;
    Span span(const void *ptr, const int64_t *s, bool query) const {
        return heads_span(ptr, s, p.d.n, query ? p.d.tq : p.d.tk, query ? p.d.heads_q : p.d.heads_k, p.d.head_dim);
    }
    bool share(const void *a, const int64_t *sa, bool qa, const void *b, const int64_t *sb, bool qb) const {
        if (!a || !b) return false;
        const attention_desc &d = p.d;
        return heads_share(a, sa, qa ? d.tq : d.tk, qa ? d.heads_q : d.heads_k, b, sb, qb ? d.tq : d.tk,
                           qb ? d.heads_q : d.heads_k, d.n, d.head_dim, true);
    }
};

struct Operand {
    const void *ptr;
    const int64_t *s;
    bool query;
};

conv3d_status common_checks(const attention_plan_s &p, const void *lengths, int64_t q_offset) {
    if (q_offset > kMaxOffset || q_offset < -kMaxOffset)
        return api_fail(CONV3D_ERR_INVALID_ARG, "q_offset (%lld) is outside -2^30 .. 2^30", (long long)q_offset);
    if ((p.d.flags & CONV3D_F_LENGTHS) && !lengths && p.d.n > 0)
        return api_fail(CONV3D_ERR_INVALID_ARG, "lengths are required with CONV3D_F_LENGTHS");
    return CONV3D_OK;
}

}  // namespace

extern "C" {

conv3d_status attention_plan(const attention_desc *d, attention_plan_t *out, size_t *workspace_bytes) {
    if (!d || !out || !workspace_bytes)
        return api_fail(CONV3D_ERR_INVALID_ARG, "desc, out and workspace_bytes are required");
    if (d->n < 0 || d->tq < 0 || d->tk < 0) return api_fail(CONV3D_ERR_INVALID_ARG, "n, tq and tk must not be negative");
    if (d->frame < 0 || d->window < 0) return api_fail(CONV3D_ERR_INVALID_ARG, "frame and window must not be negative");
    if (d->window && !d->frame) return api_fail(CONV3D_ERR_INVALID_ARG, "a window needs a frame");
    if (d->heads_q < 1 || d->heads_k < 1 || d->heads_q % d->heads_k)
        return api_fail(CONV3D_ERR_INVALID_ARG, "heads_q (%d) must be a positive multiple of heads_k (%d)", d->heads_q,
                        d->heads_k);
    if (d->head_dim < 1) return api_fail(CONV3D_ERR_INVALID_ARG, "head_dim must be positive");
    if (!(d->scale >= 0.0f) || !std::isfinite(d->scale))
        return api_fail(CONV3D_ERR_INVALID_ARG, "scale must be positive and finite, or 0");
    // the backward pass starts its scores from -lse / scale
    if (d->scale > 0.0f && (d->scale < 0x1p-64f || d->scale > 0x1p64f))
        return api_fail(CONV3D_ERR_UNSUPPORTED, "scale is outside 2^-64 .. 2^64");
    const uint32_t known = CONV3D_F_BF16 | CONV3D_F_LENGTHS | CONV3D_F_TAIL;
    if (d->flags & ~known) return api_fail(CONV3D_ERR_INVALID_ARG, "unknown flag bits 0x%x", d->flags & ~known);
    if (d->head_dim % 8 || d->head_dim > kAttnMaxDim)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 up to %d", kAttnMaxDim);
    if (d->heads_q > 16384) return api_fail(CONV3D_ERR_UNSUPPORTED, "too many heads");
    const int group = d->heads_q / d->heads_k;
    if (d->tk >= kMaxTokens || (int64_t)d->tq * group >= kMaxTokens)
        return api_fail(CONV3D_ERR_UNSUPPORTED, "2^30 tokens or more");
    attention_plan_s *p = new (std::nothrow) attention_plan_s();
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "out of host memory");
    p->d = *d;
    struct {
        const int64_t *given;
        int64_t *to;
        int tokens, heads;
        const char *name;
        bool *folds;
    } const ts[4] = {{d->q_stride, p->qs, d->tq, d->heads_q, "q_stride", &p->folds_q},
                     {d->k_stride, p->ks, d->tk, d->heads_k, "k_stride", &p->folds_k},
                     {d->v_stride, p->vs, d->tk, d->heads_k, "v_stride", &p->folds_v},
                     {d->o_stride, p->os, d->tq, d->heads_q, "o_stride", &p->folds_o}};
    conv3d_status st = CONV3D_OK;
    for (const auto &t : ts) {
        st = attn_strides(t.given, t.tokens, t.heads, d->head_dim, t.name, t.to);
        const double length = d->n && t.tokens ? (double)(d->n - 1) * t.to[0] + (double)(t.tokens - 1) * t.to[1] +
                                                     (double)(t.heads - 1) * t.to[2]
                                               : 0.0;
        if (st == CONV3D_OK && length >= kMaxElements)
            st = api_fail(CONV3D_ERR_UNSUPPORTED, "a tensor is 2^48 elements long or longer");
        if (st != CONV3D_OK) {
            delete p;
            return st;
        }
        *t.folds = heads_fold(d->n, t.tokens, t.heads, d->head_dim, t.to);
    }
    AttnParams &r = p->prm;
    for (int i = 0; i < 3; ++i) {
        r.qs[i] = p->qs[i];
        r.ks[i] = p->ks[i];
        r.vs[i] = p->vs[i];
        r.os[i] = p->os[i];
    }
    r.n = d->n;
    r.hq = d->heads_q;
    r.hk = d->heads_k;
    r.group = group;
    r.d = d->head_dim;
    r.tq = d->tq;
    r.tk = d->tk;
    r.rows = d->tq * group;
    r.frame = d->frame;
    r.window = d->window;
    r.tail = (d->flags & CONV3D_F_TAIL) ? 1 : 0;
    r.bf16 = (d->flags & CONV3D_F_BF16) ? 1 : 0;
    r.scale = d->scale > 0.0f ? d->scale : (float)(1.0 / std::sqrt((double)d->head_dim));

    const int64_t heads = (int64_t)d->n * d->heads_k;
    // what a query sees of the keys, and a key of the queries: offsets and lengths are the calls', so the
    // queries are taken as the last tokens of whole samples
    double most = d->tk, mean = d->tk, back = d->tq, back_mean = d->tq;
    if (d->frame) {
        const double offset = d->tk > d->tq ? (double)(d->tk - d->tq) : 0.0, window = (double)d->window * d->frame;
        if (d->window && window + d->frame < most) most = window + d->frame;
        mean = offset + 0.5 * (d->tq + (d->frame < d->tq ? d->frame : d->tq));
        mean = mean < most ? mean : most;
        if (d->window && window + d->frame < back) back = window + d->frame;
        back_mean = d->tk ? mean * d->tq / d->tk : 0.0;
        back_mean = back_mean < back ? back_mean : back;
    }
    const Problem of_q = {heads, r.rows, most, mean, d->head_dim},
                  of_kv = {heads, d->tk, back * group, back_mean * group, d->head_dim};
    const Choice fwd = choose(kForward, of_q, true), dq = choose(kDq, of_q, false);
    Choice dkv = choose(kDkv, of_kv, true);
    p->kind = fwd.kind;
    p->grad = {dq.kind, dkv.kind, false};
    if (heads > 0 && d->tq > 0 && d->tk > 0) {
        const char *force = getenv("CONV3D_ATTENTION_TOGETHER");
        double us = dq.us + dkv.us - kRowsUs;
        for (AttnTileKind kind : {kAttn64, kAttn128}) {
            if (forced_kind(kind, false) != kind) continue;
            const int pieces = forced_pieces(dkv.kind == kind ? dkv.pieces : 1);
            double both = together_us(kind, of_q, of_kv, pieces);
            // unequal tiles fill the card well enough by themselves, and their first ones see few keys, whose
            // numbers take a pass of their own
            if (mean < 0.95 * most) both = 1.1 * both + 3.0;
            if (force ? force[0] == '1' : both < us) {
                us = both;
                p->grad = {kind, kind, true};
                dkv.kind = kind;
                dkv.pieces = pieces;
            }
        }
    }
    const AttnTileSize tile = attn_tile(fwd.kind);
    const int64_t units = heads * ((r.rows + tile.rows - 1) / tile.rows),
                  units64 = heads * (((int64_t)(r.rows > d->tk ? r.rows : d->tk) + 63) / 64);
    if (units64 >= (int64_t)1 << 22) {
        delete p;
        return api_fail(CONV3D_ERR_UNSUPPORTED, "the call has too many tiles");
    }
    // all of a row's keys, whatever the call's offset (a range may start inside a step)
    int64_t span = d->tk;
    if (d->window) {
        const int64_t tokens = tile.rows / group + 2;
        const int64_t seen = ((int64_t)d->window + tokens / d->frame + 1) * d->frame;
        if (seen < span) span = seen;
    }
    const int64_t steps = (span + tile.keys - 1) / tile.keys + 1;
    r.splits = fwd.pieces < steps ? fwd.pieces : (int32_t)steps;
    r.pieces = (int32_t)((steps + r.splits - 1) / r.splits);
    p->grid = units * r.splits;
    p->off_ml = p->fwd_bytes = 0;
    if (r.splits > 1) {
        p->off_ml = align256((size_t)r.splits * heads * r.rows * r.d * 4);
        p->fwd_bytes = p->off_ml + (size_t)r.splits * heads * r.rows * 8;
    }
    // the same for a key's queries: steps of one query head, for all of them
    const int grad_keys = attn_tile(dkv.kind).rows, grad_step = attn_grad_step(dkv.kind);
    int64_t back_span = d->tq;
    if (d->window) {
        const int64_t seen = ((int64_t)d->window + grad_keys / d->frame + 1) * d->frame;
        if (seen < back_span) back_span = seen;
    }
    const int64_t back_steps = ((back_span + grad_step - 1) / grad_step + 1) * group;
    r.grad_splits = dkv.pieces < back_steps ? dkv.pieces : (int32_t)back_steps;
    r.grad_pieces = (int32_t)((back_steps + r.grad_splits - 1) / r.grad_splits);
    p->off_delta = align256((size_t)d->n * d->heads_q * d->tq * 4);
    p->off_dk = p->off_dv = p->back_bytes = 2 * p->off_delta;
    if (r.grad_splits > 1) {
        p->off_dv = p->off_dk + align256((size_t)r.grad_splits * heads * d->tk * r.d * 4);
        p->back_bytes = p->off_dv + (size_t)r.grad_splits * heads * d->tk * r.d * 4;
    }
    *out = p;
    *workspace_bytes = p->fwd_bytes;
    return api_ok();
}

conv3d_status attention_plan_query(attention_plan_t p, attention_plan_info *info) {
    if (!p || !info) return api_fail(CONV3D_ERR_INVALID_ARG, "plan and info are required");
    memset(info, 0, sizeof(*info));
    const AttnTileSize t = attn_tile(p->kind);
    info->tile_rows = t.rows;
    info->tile_keys = t.keys;
    info->threads = t.threads;
    info->splits = p->prm.splits;
    info->grid = p->grid;
    info->workspace_bytes = p->fwd_bytes;
    info->backward_workspace_bytes = p->back_bytes;
    snprintf(info->kernel_name, sizeof(info->kernel_name), "%s", t.name);
    return api_ok();
}

void attention_plan_destroy(attention_plan_t p) { delete p; }

conv3d_status attention_forward(attention_plan_t p, const void *q, const void *k, const void *v, void *o, void *lse,
                                const void *lengths, int64_t q_offset, void *workspace, size_t workspace_bytes,
                                void *stream) {
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "plan is null");
    const attention_desc &d = p->d;
    if (!(d.flags & CONV3D_F_LENGTHS)) lengths = nullptr;
    const bool any = d.n > 0 && d.tq > 0, keys = any && d.tk > 0;
    if ((any && (!q || !o)) || (keys && (!k || !v)))
        return api_fail(CONV3D_ERR_INVALID_ARG, "q, k, v and o are required");
    if (misaligned(q) || misaligned(k) || misaligned(v) || misaligned(o) || misaligned(lse, 4) || misaligned(lengths, 4))
        return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned (lse, lengths: 4)");
    conv3d_status st = common_checks(*p, lengths, q_offset);
    if (st == CONV3D_OK) st = check_workspace(workspace, workspace_bytes, p->fwd_bytes);
    if (st != CONV3D_OK || !any) return st != CONV3D_OK ? st : api_ok();
    if (p->folds_o) return api_fail(CONV3D_ERR_INVALID_ARG, "different elements of o overlap");
    const Tensors t{*p};
    const Operand ins[] = {{q, p->qs, true}, {k, p->ks, false}, {v, p->vs, false}};
    const Span so = t.span(o, p->os, true), sl(lse, lse ? (size_t)d.n * d.heads_q * d.tq * 4 : 0),
               sn(lengths, lengths ? (size_t)d.n * 8 : 0), sw(workspace, p->fwd_bytes);
    for (const Operand &x : ins) {
        const Span sx = t.span(x.ptr, x.s, x.query);
        if (t.share(o, p->os, true, x.ptr, x.s, x.query) || sl.meets(sx) || sw.meets(sx))
            return api_fail(CONV3D_ERR_INVALID_ARG, "o, lse or the workspace overlaps an input");
    }
    if (so.meets(sl) || so.meets(sn) || so.meets(sw) || sl.meets(sn) || sl.meets(sw) || sw.meets(sn))
        return api_fail(CONV3D_ERR_INVALID_ARG, "o, lse, lengths and the workspace overlap");
    st = api_check_device();
    if (st != CONV3D_OK) return st;
    AttnParams r = p->prm;
    r.q = in16(q);
    r.k = in16(k);
    r.v = in16(v);
    r.o = out16(o);
    r.lse = static_cast<float *>(lse);
    r.lengths = static_cast<const int32_t *>(lengths);
    r.q_offset = q_offset;
    r.part_o = static_cast<float *>(workspace);
    r.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + p->off_ml);
    return launched(launch_attention(r, p->kind, static_cast<hipStream_t>(stream)), "attention");
}

size_t attention_backward_workspace(attention_plan_t p) { return p ? p->back_bytes : 0; }

conv3d_status attention_backward(attention_plan_t p, const void *dout, const void *q, const void *k, const void *v,
                                 const void *o, const void *lse, void *dq, void *dk, void *dv, const void *lengths,
                                 int64_t q_offset, void *workspace, size_t workspace_bytes, void *stream) {
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "plan is null");
    const attention_desc &d = p->d;
    if (!(d.flags & CONV3D_F_LENGTHS)) lengths = nullptr;
    const bool any = d.n > 0 && (d.tq > 0 || d.tk > 0);
    if (any && !dq && !dk && !dv) return api_fail(CONV3D_ERR_INVALID_ARG, "no gradient is asked for");
    if ((any && d.tq > 0 && (!dout || !q || !o || !lse)) || (any && d.tk > 0 && (!k || !v)))
        return api_fail(CONV3D_ERR_INVALID_ARG, "dout, q, k, v, o and lse are required");
    for (const void *x : {dout, q, k, v, o, (const void *)dq, (const void *)dk, (const void *)dv})
        if (misaligned(x)) return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned (lse, lengths: 4)");
    if (misaligned(lse, 4) || misaligned(lengths, 4))
        return api_fail(CONV3D_ERR_INVALID_ARG, "pointers must be 16-byte aligned (lse, lengths: 4)");
    conv3d_status st = common_checks(*p, lengths, q_offset);
    if (st == CONV3D_OK) st = check_workspace(workspace, workspace_bytes, p->back_bytes);
    if (st != CONV3D_OK || !any) return st != CONV3D_OK ? st : api_ok();
    if ((dq && p->folds_q) || (dk && p->folds_k) || (dv && p->folds_v))
        return api_fail(CONV3D_ERR_INVALID_ARG, "different elements of a gradient overlap");
    const Tensors t{*p};
    const Operand ins[] = {{dout, p->os, true}, {q, p->qs, true}, {k, p->ks, false}, {v, p->vs, false}, {o, p->os, true}};
    const Operand outs[] = {{dq, p->qs, true}, {dk, p->ks, false}, {dv, p->vs, false}};
    const Span sl(lse, (size_t)d.n * d.heads_q * d.tq * 4), sn(lengths, lengths ? (size_t)d.n * 8 : 0),
        sw(workspace, p->back_bytes);
    for (int i = 0; i < 3; ++i) {
        const Operand &y = outs[i];
        if (!y.ptr) continue;
        const Span sy = t.span(y.ptr, y.s, y.query);
        for (const Operand &x : ins)
            if (t.share(y.ptr, y.s, y.query, x.ptr, x.s, x.query))
                return api_fail(CONV3D_ERR_INVALID_ARG, "a gradient overlaps an input");
        for (int j = 0; j < i; ++j)
            if (t.share(y.ptr, y.s, y.query, outs[j].ptr, outs[j].s, outs[j].query))
                return api_fail(CONV3D_ERR_INVALID_ARG, "the gradients overlap");
        if (sy.meets(sl) || sy.meets(sn) || sy.meets(sw))
            return api_fail(CONV3D_ERR_INVALID_ARG, "a gradient overlaps lse, lengths or the workspace");
    }
    for (const Operand &x : ins)
        if (sw.meets(t.span(x.ptr, x.s, x.query)))
            return api_fail(CONV3D_ERR_INVALID_ARG, "the workspace overlaps an input");
    if (sw.meets(sl) || sw.meets(sn)) return api_fail(CONV3D_ERR_INVALID_ARG, "the workspace overlaps an input");
    st = api_check_device();
    if (st != CONV3D_OK) return st;
    AttnParams r = p->prm;
    r.q = in16(q);
    r.k = in16(k);
    r.v = in16(v);
    r.o = const_cast<_Float16 *>(in16(o));
    r.lse = const_cast<float *>(static_cast<const float *>(lse));
    r.dout = in16(dout);
    r.dq = out16(dq);
    r.dk = out16(dk);
    r.dv = out16(dv);
    r.lengths = static_cast<const int32_t *>(lengths);
    r.q_offset = q_offset;
    r.nlse = static_cast<float *>(workspace);
    char *ws = static_cast<char *>(workspace);
    r.ndelta = reinterpret_cast<float *>(ws + p->off_delta);
    r.part_dk = reinterpret_cast<float *>(ws + p->off_dk);
    r.part_dv = reinterpret_cast<float *>(ws + p->off_dv);
    return launched(launch_attention_grad(r, p->grad, static_cast<hipStream_t>(stream)), "attention_backward");
}

}  // extern "C"
