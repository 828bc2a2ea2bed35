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
    bool few;
    int64_t grid;
    size_t off_ml, fwd_bytes, off_delta, back_bytes;
    AttnParams prm;  // pointers filled per call
};

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxOffset = (int64_t)1 << 30;
constexpr int kAttnCUs = 256;

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

// How many pieces to split the keys into.  `units` workgroups take `steps` steps each.
int attn_splits(int64_t units, int64_t steps, bool few) {
    if (const char *v = getenv("CONV3D_ATTENTION_SPLITS")) {
        const int k = atoi(v);
        return k < 1 ? 1 : k > steps ? (int)steps : k;
    }
    const int64_t least = few ? 2 : 8;  // steps worth a piece
    int64_t want = units > 0 ? kAttnCUs / units : 1;
    if (want > steps / least) want = steps / least;
    if (want > 256) want = 256;
    return want < 1 ? 1 : (int)want;
}

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
    p->few = r.rows <= kAttnFewRows;
    const int64_t tiles = p->few ? 1 : (r.rows + kAttnTileRows - 1) / kAttnTileRows;
    const int64_t units = heads * tiles, key_tiles = heads * (((int64_t)d->tk + 127) / 128);
    if (units >= (int64_t)1 << 22 || key_tiles >= (int64_t)1 << 22) {
        delete p;
        return api_fail(CONV3D_ERR_UNSUPPORTED, "the call has too many tiles");
    }
    // the keys that one tile's rows see together
    int64_t span = d->tk;
    if (d->window) {
        const int64_t tokens = p->few ? d->tq : kAttnTileRows / group + 2;
        const int64_t seen = ((int64_t)d->window + tokens / d->frame + 1) * d->frame;
        if (seen < span) span = seen;
    }
    const int step = p->few ? kAttnFewKeys : kAttnTileKeys;
    const int64_t steps = (span + step - 1) / step + 1;  // one more: a range may start inside a tile
    r.splits = units ? attn_splits(units, steps, p->few) : 1;
    r.pieces = (int32_t)((steps + r.splits - 1) / r.splits);
    p->grid = units * r.splits;
    p->off_ml = p->fwd_bytes = 0;
    if (r.splits > 1) {
        p->off_ml = align256((size_t)r.splits * heads * r.rows * r.d * 4);
        p->fwd_bytes = p->off_ml + (size_t)r.splits * heads * r.rows * 8;
    }
    p->off_delta = align256((size_t)d->n * d->heads_q * d->tq * 4);
    p->back_bytes = 2 * p->off_delta;
    *out = p;
    *workspace_bytes = p->fwd_bytes;
    return api_ok();
}

conv3d_status attention_plan_query(attention_plan_t p, attention_plan_info *info) {
    if (!p || !info) return api_fail(CONV3D_ERR_INVALID_ARG, "plan and info are required");
    memset(info, 0, sizeof(*info));
    info->tile_rows = p->few ? kAttnFewRows : kAttnTileRows;
    info->tile_keys = p->few ? kAttnFewKeys : kAttnTileKeys;
    info->threads = p->few ? 256 : kAttnTileRows * 2;
    info->splits = p->prm.splits;
    info->grid = p->grid;
    info->workspace_bytes = p->fwd_bytes;
    info->backward_workspace_bytes = p->back_bytes;
    snprintf(info->kernel_name, sizeof(info->kernel_name), "%s", p->few ? "attention_few" : "attention_tile");
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
    return launched(launch_attention(r, p->few, static_cast<hipStream_t>(stream)), "attention");
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
    r.ndelta = reinterpret_cast<float *>(static_cast<char *>(workspace) + p->off_delta);
    return launched(launch_attention_grad(r, static_cast<hipStream_t>(stream)), "attention_backward");
}

}  // extern "C"
