// Host checks of rows of heads (tq_rows), shared by the calls that take them.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <utility>

#include "tq.h"

namespace tq {

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline tq_status check_rows(const tq_rows* r, int elem) {
    if (!r || !r->data || !aligned(r->data, 16)) return TQ_ERR_INVALID_ARG;
    if (r->stride_batch * elem % 16 != 0 || r->stride_head * elem % 16 != 0 || r->stride_token * elem % 16 != 0)
        return TQ_ERR_INVALID_ARG;
    return TQ_OK;
}

// The axes of rows of heads, in elements, the largest stride first; an axis of one element has none.
struct Axes {
    int64_t stride[3], n[3];
    Axes(const tq_rows* r, int64_t nb, int64_t nh, int64_t nt) : stride{r->stride_batch, r->stride_head, r->stride_token}, n{nb, nh, nt} {
        for (int i = 0; i < 3; ++i) stride[i] = n[i] > 1 ? std::abs(stride[i]) : 0;
        for (int i = 0; i < 2; ++i)
            for (int k = 0; k < 2 - i; ++k)
                if (stride[k] < stride[k + 1]) std::swap(stride[k], stride[k + 1]), std::swap(n[k], n[k + 1]);
    }
    // Whether two rows whose starts differ by a sum of steps along axes k.. lie within D elements of being `delta` apart. A
    // yes has such rows to show; a no is sure where each stride is as long as what the smaller ones span.
    bool meet(int64_t delta, int k, int D) const {
        if (k == 3 || stride[k] == 0) return std::abs(delta) < D;
        const int64_t d = delta / stride[k];
        for (int64_t i = d - 1; i <= d + 1; ++i)
            if (std::abs(i) < n[k] && meet(delta - i * stride[k], k + 1, D)) return true;
        return false;
    }
    // Whether the rows share memory with each other.
    bool meets_itself(int D) const {
        for (int k = 0; k < 3; ++k)
            if ((stride[k] > 0 && meet(stride[k], k + 1, D)) || (stride[k] == 0 && n[k] > 1)) return true;
        return false;
    }
};

// Whether two sets of rows lie alike: equal strides along every axis of more than one element.
inline bool same_layout(const tq_rows* a, const tq_rows* b, int64_t nb, int64_t nh, int64_t nt) {
    return (nb <= 1 || a->stride_batch == b->stride_batch) && (nh <= 1 || a->stride_head == b->stride_head) &&
           (nt <= 1 || a->stride_token == b->stride_token);
}

// What one set of rows spans, in elements from its data pointer: [first, last + D).
inline void rows_span(const tq_rows* r, int64_t nb, int64_t nh, int64_t nt, int D, int64_t& lo, int64_t& hi) {
    lo = 0, hi = D;
    const int64_t reach[3] = {nb > 1 ? r->stride_batch * (nb - 1) : 0, nh > 1 ? r->stride_head * (nh - 1) : 0, nt > 1 ? r->stride_token * (nt - 1) : 0};
    for (int64_t x : reach) (x < 0 ? lo : hi) += x;
}

// Whether a row of a ([nb][ha][nt] of them) shares memory with a row of b ([nb][hb][nt]). Sets in different layouts share where
// their spans do; of sets that lie alike, a yes has two such rows to show, and a no is sure as in Axes::meet.
inline bool rows_meet(const tq_rows* a, int64_t ha, const tq_rows* b, int64_t hb, int64_t nb, int64_t nt, int D, int elem) {
    int64_t alo, ahi, blo, bhi;
    rows_span(a, nb, ha, nt, D, alo, ahi);
    rows_span(b, nb, hb, nt, D, blo, bhi);
    const int64_t apart = (reinterpret_cast<intptr_t>(b->data) - reinterpret_cast<intptr_t>(a->data)) / elem;
    if (apart + blo >= ahi || alo >= apart + bhi) return false;
    if (!same_layout(a, b, nb, std::min(ha, hb), nt)) return true;   // (the stride of a single head says nothing)
    // steps (a's index less b's) along each axis, the largest stride first
    struct { int64_t stride, lo, hi; } axis[3] = {{nb > 1 ? a->stride_batch : 0, 1 - nb, nb - 1},
                                                  {ha > 1 ? a->stride_head : hb > 1 ? b->stride_head : 0, 1 - hb, ha - 1},
                                                  {nt > 1 ? a->stride_token : 0, 1 - nt, nt - 1}};
    for (auto& x : axis)
        if (x.stride < 0) x = {-x.stride, -x.hi, -x.lo};
    for (int i = 0; i < 2; ++i)
        for (int k = 0; k < 2 - i; ++k)
            if (axis[k].stride < axis[k + 1].stride) std::swap(axis[k], axis[k + 1]);
    auto meet = [&](auto&& self, int64_t delta, int k) -> bool {
        if (k == 3 || axis[k].stride == 0) return std::abs(delta) < D;
        const int64_t d = delta / axis[k].stride;
        for (int64_t i = d - 1; i <= d + 1; ++i)
            if (i >= axis[k].lo && i <= axis[k].hi && self(self, delta - i * axis[k].stride, k + 1)) return true;
        return false;
    };
    return meet(meet, apart, 0);
}

}  // namespace tq
