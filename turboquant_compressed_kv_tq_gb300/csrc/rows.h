// Host checks of rows of heads (tq_rows), shared by the calls that take them.
#pragma once

#include <algorithm>
#include <cstddef>
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

// Sums of steps along three axes: lo .. hi of each stride, the largest stride first.
struct Steps {
    int64_t stride[3], lo[3], hi[3];
    int looks = 1 << 20;   // at most; a few where each stride is as long as what the smaller ones span
    void sort() {
        for (int i = 0; i < 3; ++i)
            if (stride[i] < 0) stride[i] = -stride[i], std::swap(lo[i], hi[i]), lo[i] = -lo[i], hi[i] = -hi[i];
        for (int i = 0; i < 2; ++i)
            for (int k = 0; k < 2 - i; ++k)
                if (stride[k] < stride[k + 1]) std::swap(stride[k], stride[k + 1]), std::swap(lo[k], lo[k + 1]), std::swap(hi[k], hi[k + 1]);
    }
    // Whether a sum along axes k.. lies within D elements of `delta`: exact, and yes where it cannot be told in so many looks.
    bool meet(int64_t delta, int k, int64_t D) {
        if (k == 3 || stride[k] == 0) return std::abs(delta) < D;
        int64_t least = delta - D + 1, most = delta + D - 1;   // of the steps along axis k
        for (int j = k + 1; j < 3; ++j) least -= stride[j] * hi[j], most -= stride[j] * lo[j];
        auto down = [&](int64_t x) { return x / stride[k] - (x % stride[k] < 0); };
        const int64_t end = std::min(hi[k], down(most));
        for (int64_t i = std::max(lo[k], down(least + stride[k] - 1)); i <= end; ++i)
            if (--looks < 0 || meet(delta - i * stride[k], k + 1, D)) return true;
        return false;
    }
};

// The axes of rows of heads, in elements; an axis of one element has none.
struct Axes {
    Steps steps;
    Axes(const tq_rows* r, int64_t nb, int64_t nh, int64_t nt) {
        const int64_t stride[3] = {r->stride_batch, r->stride_head, r->stride_token}, n[3] = {nb, nh, nt};
        for (int i = 0; i < 3; ++i) steps.stride[i] = n[i] > 1 ? stride[i] : 0, steps.lo[i] = 1 - n[i], steps.hi[i] = n[i] - 1;
        steps.sort();
    }
    // Whether two rows lie within D elements of being `delta` apart.
    bool meet(int64_t delta, int D) const { return Steps(steps).meet(delta, 0, D); }
    // Whether the rows share memory with each other.
    bool meets_itself(int D) const {
        Steps s = steps;
        for (int k = 0; k < 3; ++k) {
            s.lo[k] = 1;   // the first axis along which two rows lie apart
            if (s.stride[k] == 0 ? s.hi[k] > 0 : s.meet(0, k, D)) return true;
        }
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
// their spans do; sets that lie alike, where two rows do.
inline bool rows_meet(const tq_rows* a, int64_t ha, const tq_rows* b, int64_t hb, int64_t nb, int64_t nt, int D, int elem) {
    int64_t alo, ahi, blo, bhi;
    rows_span(a, nb, ha, nt, D, alo, ahi);
    rows_span(b, nb, hb, nt, D, blo, bhi);
    const int64_t apart = (reinterpret_cast<intptr_t>(b->data) - reinterpret_cast<intptr_t>(a->data)) / elem;
    if (apart + blo >= ahi || alo >= apart + bhi) return false;
    if (!same_layout(a, b, nb, std::min(ha, hb), nt)) return true;   // (the stride of a single head says nothing)
    // steps: a's index less b's
    Steps s{{nb > 1 ? a->stride_batch : 0, ha > 1 ? a->stride_head : hb > 1 ? b->stride_head : 0, nt > 1 ? a->stride_token : 0},
            {1 - nb, 1 - hb, 1 - nt},
            {nb - 1, ha - 1, nt - 1}};
    s.sort();
    return s.meet(apart, 0, D);
}

// The bytes of an array (none of a null pointer's).
struct Span {
    intptr_t lo = 0, hi = 0;
    Span(const void* p, int64_t bytes) {
        if (p && bytes > 0) lo = reinterpret_cast<intptr_t>(p), hi = lo + bytes;
    }
    bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
    // A row of `bytes` of p + b * stride_b + r * stride_r (bytes), b < nb, r < nr.
    bool meets_rows(const void* p, int64_t stride_b, int64_t nb, int64_t stride_r, int64_t nr, int64_t bytes) const {
        if (!p || nb <= 0 || nr <= 0 || lo == hi) return false;
        const intptr_t first = reinterpret_cast<intptr_t>(p);
        const int64_t b = stride_b * (nb - 1), r = stride_r * (nr - 1);
        if (first + std::min<int64_t>(b, 0) + std::min<int64_t>(r, 0) >= hi || first + std::max<int64_t>(b, 0) + std::max<int64_t>(r, 0) + bytes <= lo) return false;
        // a row's start lies in (lo - bytes, hi): twice that, about its middle
        Steps s{{nb > 1 ? 2 * stride_b : 0, nr > 1 ? 2 * stride_r : 0, 0}, {0, 0, 0}, {nb - 1, nr - 1, 0}};
        s.sort();
        return s.meet(lo + hi - bytes - 2 * first, 0, hi - lo + bytes);
    }
};
// Whether any of `written` shares memory with another, or with one of `read`.
template <size_t W, size_t R>
bool spans_meet(const Span (&written)[W], const Span (&read)[R]) {
    for (size_t i = 0; i < W; ++i) {
        for (size_t j = i + 1; j < W; ++j)
            if (written[i].meets(written[j])) return true;
        for (const Span& r : read)
            if (written[i].meets(r)) return true;
    }
    return false;
}

}  // namespace tq
