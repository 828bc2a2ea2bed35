// Host side of adamw_step as declared in include/conv3d.h: validation, the
// launches' tables, and launches on the caller's stream.  Nothing here
// synchronises the device or allocates device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <new>
#include <vector>

#include "token_checks.h"

using namespace c3d;

struct adamw_plan_s {
    struct Launch {
        AdamwParams prm;
        int64_t blocks;
    };
    std::vector<Launch> launches;
    std::vector<std::pair<uintptr_t, uintptr_t>> written;  // in order, disjoint
    uint32_t flags;
    bool far;
};

namespace {

struct Range {
    uintptr_t lo, hi;
    bool write;
};

conv3d_status hyper_of(const adamw_hyper *h, AdamwHyper *out) {
    if (!h) return api_fail(CONV3D_ERR_INVALID_ARG, "hyper is required");
    if (!(h->lr >= 0.0) || !(h->eps >= 0.0) || !(h->weight_decay >= 0.0) || !std::isfinite(h->lr) ||
        !std::isfinite(h->eps) || !std::isfinite(h->weight_decay) || !std::isfinite(h->grad_scale))
        return api_fail(CONV3D_ERR_INVALID_ARG, "lr, eps and weight_decay must be finite and not negative, grad_scale finite");
    if (!(h->beta1 >= 0.0 && h->beta1 < 1.0 && h->beta2 >= 0.0 && h->beta2 < 1.0))
        return api_fail(CONV3D_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
    if (h->step < 1) return api_fail(CONV3D_ERR_INVALID_ARG, "step (%lld) counts from 1", (long long)h->step);
    // 1 - beta^step without the cancellation of a beta next to 1
    const double t = (double)h->step;
    const auto rest = [&](double b) { return b > 0.0 ? -std::expm1(t * std::log(b)) : 1.0; };
    out->grad_scale = (float)h->grad_scale;
    out->beta1 = (float)h->beta1;
    out->rest1 = (float)(1.0 - h->beta1);
    out->beta2 = (float)h->beta2;
    out->rest2 = (float)(1.0 - h->beta2);
    out->lr1 = (float)(h->lr / rest(h->beta1));
    out->root2 = (float)(1.0 / std::sqrt(rest(h->beta2)));
    out->eps = (float)h->eps;
    out->lr_decay = (float)(h->lr * h->weight_decay);
    for (float x : {out->grad_scale, out->lr1, out->root2, out->eps, out->lr_decay})
        if (!std::isfinite(x)) return api_fail(CONV3D_ERR_INVALID_ARG, "a hyperparameter is past the range of fp32");
    // the kernel's reciprocal of a subnormal is infinite, and 0 times that no number
    if (h->eps > 0.0 && out->eps < FLT_MIN) return api_fail(CONV3D_ERR_INVALID_ARG, "eps is below 2^-126 and not 0");
    return CONV3D_OK;
}
static_assert(sizeof(AdamwHyper) == ADAMW_DEVICE_HYPER * sizeof(float), "the numbers in device memory");

// The plan's tables; throws std::bad_alloc.
conv3d_status build(const adamw_tensor *tensors, int32_t count, uint32_t flags, adamw_plan_s *p) {
    const bool state8 = (flags & CONV3D_F_STATE8) != 0;
    const int64_t grad_bytes = flags & CONV3D_F_GRAD32 ? 4 : 2, state_bytes = state8 ? 1 : 4;
    std::vector<Range> all;
    std::vector<const adamw_tensor *> used;
    int64_t total = 0;
    for (int32_t i = 0; i < count; ++i) {
        const adamw_tensor &t = tensors[i];
        if (t.count < 0) return api_fail(CONV3D_ERR_INVALID_ARG, "tensor %d: a negative count", i);
        if (!(t.decay >= 0.0f) || !std::isfinite(t.decay))
            return api_fail(CONV3D_ERR_INVALID_ARG, "tensor %d: decay must be finite and not negative", i);
        if (t.count == 0) continue;
        if (t.count >= (int64_t)1 << 40 || (total += t.count) >= (int64_t)1 << 40)
            return api_fail(CONV3D_ERR_UNSUPPORTED, "2^40 elements or more");
        if ((!t.param && !t.master) || !t.grad || !t.m || !t.v || (state8 && (!t.m_scale || !t.v_scale)))
            return api_fail(CONV3D_ERR_INVALID_ARG, "tensor %d: param or master, grad, m and v (and their scales) are required", i);
        for (const void *x : {(const void *)t.param, (const void *)t.master, t.grad, (const void *)t.m, (const void *)t.v})
            if (misaligned(x)) return api_fail(CONV3D_ERR_INVALID_ARG, "tensor %d: pointers must be 16-byte aligned", i);
        const auto add = [&](const void *ptr, int64_t bytes, bool write) {
            const uintptr_t lo = reinterpret_cast<uintptr_t>(ptr);
            if (ptr) all.push_back({lo, lo + (uintptr_t)bytes, write});
        };
        add(t.param, t.count * 2, true);
        add(t.master, t.count * 4, true);
        add(t.grad, t.count * grad_bytes, false);
        add(t.m, t.count * state_bytes, true);
        add(t.v, t.count * state_bytes, true);
        if (state8) {
            add(t.m_scale, (t.count + kAdamwBlock - 1) / kAdamwBlock, true);
            add(t.v_scale, (t.count + kAdamwBlock - 1) / kAdamwBlock, true);
        }
        used.push_back(&t);
    }
    std::sort(all.begin(), all.end(), [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t any = 0, write = 0;  // ends so far of all ranges and of the written ones
    for (const Range &r : all) {
        if (r.lo < write || (r.write && r.lo < any)) return api_fail(CONV3D_ERR_INVALID_ARG, "tensors overlap");
        any = std::max(any, r.hi);
        if (r.write) {
            write = std::max(write, r.hi);
            p->written.push_back({r.lo, r.hi});
        }
    }
    p->flags = flags;
    int64_t bytes = 0;
    for (const Range &r : all) bytes += (int64_t)(r.hi - r.lo);
    p->far = bytes > kAdamwCached;
    const int64_t unit = adamw_unit(p->far);
    for (size_t at = 0; at < used.size();) {
        p->launches.push_back({});
        adamw_plan_s::Launch &l = p->launches.back();
        const size_t end = std::min(used.size(), at + kAdamwTensors);
        int64_t block = 0;
        for (size_t i = at; i < end; ++i) {
            const adamw_tensor &t = *used[i];
            AdamwTensor &d = l.prm.t[i - at];
            d.param = out16(t.param);
            d.master = static_cast<float *>(t.master);
            d.grad = t.grad;
            d.m = t.m;
            d.v = t.v;
            d.m_scale = static_cast<uint8_t *>(t.m_scale);
            d.v_scale = static_cast<uint8_t *>(t.v_scale);
            d.count = t.count;
            d.decay = t.decay;
            l.prm.first[i - at] = (int32_t)block;
            block += (t.count + unit - 1) / unit;
            if (block >= (int64_t)1 << 22) return api_fail(CONV3D_ERR_UNSUPPORTED, "too many elements in one launch");
        }
        for (size_t i = end - at; i < (size_t)kAdamwTensors; ++i) l.prm.first[i] = INT_MAX;
        l.blocks = block;
        at = end;
    }
    return CONV3D_OK;
}

}  // namespace

extern "C" {

conv3d_status adamw_plan(const adamw_tensor *tensors, int32_t count, uint32_t flags, adamw_plan_t *out) {
    if (!out || (count > 0 && !tensors)) return api_fail(CONV3D_ERR_INVALID_ARG, "tensors and out are required");
    if (count < 0) return api_fail(CONV3D_ERR_INVALID_ARG, "count must not be negative");
    const uint32_t known = CONV3D_F_BF16 | CONV3D_F_STATE8 | CONV3D_F_GRAD32;
    if (flags & ~known) return api_fail(CONV3D_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags & ~known);
    adamw_plan_s *p = new (std::nothrow) adamw_plan_s();
    conv3d_status st = CONV3D_ERR_INVALID_ARG;
    try {
        if (p) st = build(tensors, count, flags, p);
        else api_fail(st, "out of host memory");
    } catch (const std::bad_alloc &) {
        st = api_fail(CONV3D_ERR_INVALID_ARG, "out of host memory");
    }
    if (st != CONV3D_OK) {
        delete p;
        return st;
    }
    *out = p;
    return api_ok();
}

void adamw_plan_destroy(adamw_plan_t p) { delete p; }

conv3d_status adamw_hyper_pack(const adamw_hyper *h, float *out) {
    AdamwHyper x;
    const conv3d_status st = hyper_of(h, &x);
    if (st != CONV3D_OK) return st;
    if (!out) return api_fail(CONV3D_ERR_INVALID_ARG, "out is required");
    const float v[ADAMW_DEVICE_HYPER] = {x.grad_scale, x.beta1, x.rest1, x.beta2, x.rest2, x.lr1, x.root2, x.eps, x.lr_decay};
    for (int i = 0; i < ADAMW_DEVICE_HYPER; ++i) out[i] = v[i];
    return api_ok();
}

conv3d_status adamw_step(adamw_plan_t p, const adamw_hyper *hyper, const void *device_hyper, void *stream) {
    if (!p) return api_fail(CONV3D_ERR_INVALID_ARG, "plan is null");
    AdamwHyper h = {};
    if (device_hyper) {
        if (misaligned(device_hyper, 4)) return api_fail(CONV3D_ERR_INVALID_ARG, "device_hyper must be 4-byte aligned");
        const uintptr_t lo = reinterpret_cast<uintptr_t>(device_hyper), hi = lo + sizeof(AdamwHyper);
        // the first written range that ends behind lo
        const auto at = std::upper_bound(p->written.begin(), p->written.end(), lo,
                                         [](uintptr_t v, const std::pair<uintptr_t, uintptr_t> &r) { return v < r.second; });
        if (at != p->written.end() && at->first < hi)
            return api_fail(CONV3D_ERR_INVALID_ARG, "device_hyper overlaps a tensor that is written");
    } else {
        const conv3d_status st = hyper_of(hyper, &h);
        if (st != CONV3D_OK) return st;
    }
    if (p->launches.empty()) return api_ok();
    const conv3d_status st = api_check_device();
    if (st != CONV3D_OK) return st;
    for (const adamw_plan_s::Launch &l : p->launches) {
        AdamwParams q = l.prm;
        q.hyper = h;
        q.device_hyper = static_cast<const AdamwHyper *>(device_hyper);
        const hipError_t e = launch_adamw(q, l.blocks, p->far, (p->flags & CONV3D_F_BF16) != 0, (p->flags & CONV3D_F_STATE8) != 0,
                                          (p->flags & CONV3D_F_GRAD32) != 0, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return launched(e, "adamw_step");
    }
    return api_ok();
}

}  // extern "C"
