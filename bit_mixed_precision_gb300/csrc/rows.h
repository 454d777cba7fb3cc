// Host only: whether the rows that two tensors consist of share memory.
#pragma once

#include <stdint.h>

#include <utility>

namespace kvq {

// Rows of `row` bytes at at + i_0 stride[0] + i_1 stride[1] + .., 0 <= i_a < size[a]: axes of one entry and of stride 0 left
// out, by ascending stride, dense ones joined to the row.  size[a] and stride[a] >= 0, in bytes.
struct Rows {
    int64_t at = 0, row = 0, size[3] = {0, 0, 0}, stride[3] = {0, 0, 0};
    int n = 0;

    Rows() = default;
    Rows(const void* p, int64_t bytes) : at((int64_t)reinterpret_cast<uintptr_t>(p)), row(bytes) {}
    Rows(const void* p, int64_t bytes, const int64_t (&sizes)[3], const int64_t (&strides)[3]) : Rows(p, bytes) {
        for (int i = 0; i < 3; ++i) {
            if (sizes[i] == 1 || strides[i] == 0) continue;
            int j = n++;
            for (; j > 0 && stride[j - 1] > strides[i]; --j) size[j] = size[j - 1], stride[j] = stride[j - 1];
            size[j] = sizes[i], stride[j] = strides[i];
        }
        while (n > 0 && stride[0] == row) {
            row *= size[0];
            for (int i = 1; i < n; ++i) size[i - 1] = size[i], stride[i - 1] = stride[i];
            --n;
        }
    }
    // from the first byte of the rows of the first m axes to behind the last
    int64_t extent(int m) const {
        int64_t e = row;
        for (int i = 0; i < m; ++i) e += (size[i] - 1) * stride[i];
        return e;
    }
    // No two rows share a byte, as in every view that slicing and transposing give: each axis steps over all the axes of
    // smaller strides together.
    bool nested() const {
        for (int i = 0; i < n; ++i)
            if (stride[i] < extent(i)) return false;
        return true;
    }
};

// The whole numbers i of [first, last] with lo < i s < hi (s > 0).
inline void steps_between(int64_t lo, int64_t hi, int64_t s, int64_t& first, int64_t& last) {
    auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
    const int64_t a = floor_div(lo, s) + 1, b = -floor_div(-hi, s) - 1;
    if (a > first) first = a;
    if (b < last) last = b;
}

// Do rows of a's first na axes, from a_at on, share a byte with those of b?  Exact for views of one array; true where a
// decision would take more than a few steps an axis.
inline bool rows_meet(const Rows& a, int na, int64_t a_at, const Rows& b, int nb, int64_t b_at) {
    if (a_at + a.extent(na) <= b_at || b_at + b.extent(nb) <= a_at) return false;
    if (na == 0 && nb == 0) return true;
    constexpr int64_t kMost = 8;
    if (na > 0 && nb > 0 && a.stride[na - 1] == b.stride[nb - 1]) {
        // entries i of a and j of b are shifted by (j - i) strides: one comparison for each difference that is close enough
        const int64_t s = a.stride[na - 1], d = b_at - a_at;
        int64_t first = 1 - a.size[na - 1], last = b.size[nb - 1] - 1;
        steps_between(-d - b.extent(nb - 1), a.extent(na - 1) - d, s, first, last);
        if (last - first >= kMost) return true;
        for (int64_t k = first; k <= last; ++k)
            if (rows_meet(a, na - 1, a_at, b, nb - 1, b_at + k * s)) return true;
        return false;
    }
    if (na == 0 || (nb > 0 && b.stride[nb - 1] > a.stride[na - 1])) return rows_meet(b, nb, b_at, a, na, a_at);
    // the entries of a's widest axis that reach into b
    const int64_t s = a.stride[na - 1], e = a.extent(na - 1), d = b_at - a_at;
    int64_t first = 0, last = a.size[na - 1] - 1;
    steps_between(d - e, d + b.extent(nb), s, first, last);
    if (last - first >= 2 && nb == 0 && s >= e) return true;        // those in the middle lie within b's one row
    if (last - first >= kMost) return true;
    for (int64_t i = first; i <= last; ++i)
        if (rows_meet(a, na - 1, a_at + i * s, b, nb, b_at)) return true;
    return false;
}

inline bool rows_meet(const Rows& a, const Rows& b) { return rows_meet(a, a.n, a.at, b, b.n, b.at); }

}  // namespace kvq
