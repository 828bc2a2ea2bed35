// Checks that the token operators' entry points share (token_api.cpp,
// attention_api.cpp, adamw_api.cpp): alignment, overlaps of matrices and of heads with strides,
// workspaces and launches.  Host only.
#pragma once

#include <hip/hip_runtime.h>

#include "token_internal.h"

namespace c3d {

constexpr double kMaxElements = 281474976710656.0;  // 2^48, from a tensor's first element to its last

inline bool misaligned(const void *p, uintptr_t bytes = 16) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

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

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

inline const _Float16 *in16(const void *p) { return static_cast<const _Float16 *>(p); }
inline _Float16 *out16(void *p) { return static_cast<_Float16 *>(p); }

inline conv3d_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (misaligned(ws)) return api_fail(CONV3D_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    if (need && (!ws || bytes < need))
        return api_fail(CONV3D_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? bytes : (size_t)0);
    return CONV3D_OK;
}

inline conv3d_status launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return api_fail(CONV3D_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return api_ok();
}

inline bool same3(const int64_t *a, const int64_t *b) { return a[0] == b[0] && a[1] == b[1] && a[2] == b[2]; }

inline Span heads_span(const void *p, const int64_t *s, int64_t n, int64_t tokens, int heads, int dim) {
    if (n < 1 || tokens < 1 || heads < 1) return Span(nullptr, (size_t)0);
    return Span(p, (size_t)((n - 1) * s[0] + (tokens - 1) * s[1] + (heads - 1) * s[2] + dim) * 2);
}

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
inline bool heads_fold(int64_t n, int64_t tokens, int heads, int dim, const int64_t *s) {
    if (n < 1 || tokens < 1 || heads < 1) return false;
    const int64_t ext[3] = {n, tokens, heads};
    HeadSearch h(dim, true);
    for (int i = 0; i < 3; ++i) h.add(s[i], -(ext[i] - 1), ext[i] - 1);
    return h.found(0) || h.unanswered();
}

// Whether heads of two tensors share an element; cautious: or cannot be shown not to.
inline bool heads_share(const void *a, const int64_t *sa, int64_t ta, int ha, const void *b, const int64_t *sb,
                        int64_t tb, int hb, int64_t n, int dim, bool cautious) {
    if (!heads_span(a, sa, n, ta, ha, dim).meets(heads_span(b, sb, n, tb, hb, dim))) return false;
    const int64_t ea[3] = {n, ta, ha}, eb[3] = {n, tb, hb};
    HeadSearch h(dim, false);
    for (int i = 0; i < 3; ++i) {
        h.add(sa[i], -(ea[i] - 1), 0);
        h.add(sb[i], 0, eb[i] - 1);
    }
    const int64_t bytes = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    return h.found(bytes / 2) || (cautious && h.unanswered());  // both are 16-byte aligned
}

}  // namespace c3d
