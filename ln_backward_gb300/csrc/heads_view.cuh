// heads_view.cuh -- strided tensors of heads on the host: their extents, and which of them share elements.
#pragma once

#include <algorithm>

#include "tb_common.cuh"

namespace tb {
namespace {

// ---------------------------------------------------------------- host: strided buffers
struct View {
    const char* p;
    int64_t n[3];        // batch, seq, heads
    int64_t s[3];        // strides in elements (0 where the size is 1)
};

inline View view_of(const tb_heads* t, int64_t batch, int64_t seq) {
    View v{static_cast<const char*>(t->data), {batch, seq, t->heads},
           {t->stride_batch, t->stride_seq, t->stride_head}};
    for (int i = 0; i < 3; ++i)
        if (v.n[i] <= 1) v.s[i] = 0;
    return v;
}

// Elements from the first to behind the last one; false when that leaves 2^60.
inline bool extent(const View& v, int64_t dim, int64_t* out) {
    __int128 e = dim;
    for (int i = 0; i < 3; ++i) e += (__int128)(v.n[i] - 1) * v.s[i];
    if (e > ((__int128)1 << 60)) return false;
    *out = (int64_t)e;
    return true;
}

// Whether no two (batch, seq, head) rows of `dim` elements share one, decided by
// nesting: each stride reaches over everything that the smaller strides span.  `order`
// receives the sizes above 1, by falling stride.
inline bool nested(const View& v, int64_t dim, int (&order)[3], int* count) {
    int n = 0;
    for (int i = 0; i < 3; ++i)
        if (v.n[i] > 1) order[n++] = i;
    std::sort(order, order + n, [&](int x, int y) { return v.s[x] > v.s[y]; });
    *count = n;
    int64_t inner = dim;
    for (int i = n - 1; i >= 0; --i) {
        if (v.s[order[i]] < inner) return false;
        inner += (v.n[order[i]] - 1) * v.s[order[i]];
    }
    return true;
}

inline bool meet(const View& a, const View& b, const int64_t (&s)[3], const int* order, int count, int at,
          int64_t delta, int64_t dim) {
    if (at == count) return delta > -dim && delta < dim;
    const int i = order[at];
    const int64_t step = s[i];
    // (row of b) - (row of a) = k with -(a.n - 1) <= k <= b.n - 1; what the inner strides
    // add is below one step in size
    int64_t k = -delta / step;
    for (int64_t c = k - 1; c <= k + 1; ++c)
        if (c >= -(a.n[i] - 1) && c <= b.n[i] - 1 &&
            meet(a, b, s, order, count, at + 1, delta + c * step, dim))
            return true;
    return false;
}

// Whether an output view shares an element with another view.  Exact where both walk
// memory by the same strides (slices of one buffer); otherwise any common address range
// counts as shared.
inline bool shares(const View& out, const View& other, int64_t dim, size_t es) {
    int64_t ea = 0, eb = 0;
    if (!extent(out, dim, &ea) || !extent(other, dim, &eb)) return true;
    if (!overlap(range_of(out.p, ea, es), range_of(other.p, eb, es))) return false;
    View both = out;
    for (int i = 0; i < 3; ++i) {
        if (out.n[i] > 1 && other.n[i] > 1 && out.s[i] != other.s[i]) return true;
        both.s[i] = out.n[i] > 1 ? out.s[i] : other.s[i];
        both.n[i] = std::max(out.n[i], other.n[i]);
    }
    int order[3], count = 0;
    if (!nested(both, dim, order, &count)) return true;
    const int64_t delta = (int64_t)(reinterpret_cast<uintptr_t>(other.p) -
                                    reinterpret_cast<uintptr_t>(out.p)) / (int64_t)es;
    return meet(out, other, both.s, order, count, 0, delta, dim);
}

// The very same rows: a call in place.
inline bool same(const View& a, const View& b) {
    return a.p == b.p && a.n[0] == b.n[0] && a.n[1] == b.n[1] && a.n[2] == b.n[2] &&
           a.s[0] == b.s[0] && a.s[1] == b.s[1] && a.s[2] == b.s[2];
}

inline tb_status check_view(const tb_heads* t, int64_t batch, int64_t seq, int64_t dim, size_t es, View* v) {
    if (t->heads < 0 || t->stride_batch < 0 || t->stride_seq < 0 || t->stride_head < 0)
        return TB_ERR_INVALID_VALUE;
    *v = view_of(t, batch, seq);
    if (batch == 0 || seq == 0 || t->heads == 0) return TB_OK;
    if (!t->data) return TB_ERR_INVALID_VALUE;
    int64_t e = 0;
    if (t->heads > (1 << 20) || !extent(*v, dim, &e)) return TB_ERR_INVALID_VALUE;
    return aligned_to(t->data, es) ? TB_OK : TB_ERR_MISALIGNED;
}

}  // namespace
}  // namespace tb
