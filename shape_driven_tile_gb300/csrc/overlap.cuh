// overlap.cuh -- whether two strided tensors share a byte (host side), so that a call can refuse
// outputs that lie over its inputs or over each other, and take slices of the same rows.
#pragma once

#include <algorithm>
#include <cstdint>
#include <utility>

namespace sdt {

// n0 x n1 stretches of `len` bytes, step0 and step1 bytes apart (not negative; a dimension of one never steps).
struct Stretches {
    const void *p;
    int64_t n0, step0, n1, step1, len;
};

namespace overlap_detail {

// n stretches of `len` bytes, `step` bytes apart.
struct Row {
    uintptr_t p;
    int64_t n, step, len;
    int64_t extent() const {
        int64_t e;
        return __builtin_mul_overflow(n - 1, step, &e) || __builtin_add_overflow(e, len, &e) ? INT64_MAX : e;
    }
};

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0

inline bool apart(uintptr_t a, int64_t a_len, uintptr_t b, int64_t b_len) {
    return a <= b ? b - a >= uint64_t(a_len) : a - b >= uint64_t(b_len);
}

inline bool rows_share(Row x, Row y) {
    if (apart(x.p, x.extent(), y.p, y.extent())) return false;
    if (x.n > y.n) std::swap(x, y);
    const auto d = [](uintptr_t to, uintptr_t from) { return static_cast<int64_t>(to - from); };
    if (y.n == 1) return true;  // two single stretches that are not apart
    // stretch i of y begins at y.p + i * y.step: those that reach into [at, at + len) have -y.len < y_i - at < len
    const auto reach = [&](int64_t off, int64_t len, int64_t lo, int64_t hi) {  // off = y.p - at; i in lo .. hi
        return std::max(lo, floor_div(-y.len - off, y.step) + 1) <= std::min(hi, -floor_div(off - len, y.step) - 1);
    };
    if (x.n == 1 || x.step == y.step) return reach(d(y.p, x.p), x.len, 1 - x.n, y.n - 1);
    for (int64_t i = 0; i < x.n; ++i)
        if (reach(d(y.p, x.p + uintptr_t(i) * uintptr_t(x.step)), x.len, 0, y.n - 1)) return true;
    return false;
}

// Neighbouring stretches joined; then few in the second dimension.
inline Stretches joined(Stretches s) {
    if (s.n0 == 1) s.step0 = 0;
    if (s.n1 == 1) s.step1 = 0;
    for (int turn = 0; turn < 2; ++turn) {
        if (s.step1 <= s.len) {
            s.len += (s.n1 - 1) * s.step1;
            s.n1 = 1;
            s.step1 = 0;
        }
        std::swap(s.n0, s.n1);
        std::swap(s.step0, s.step1);
    }
    if (s.step1 <= s.len) {  // (again: what the other dimension joined may reach further now)
        s.len += (s.n1 - 1) * s.step1;
        s.n1 = 1;
        s.step1 = 0;
    }
    if (s.n1 > s.n0) {
        std::swap(s.n0, s.n1);
        std::swap(s.step0, s.step1);
    }
    return s;
}

}  // namespace overlap_detail

// Whether a and b share a byte.  Exact; a few comparisons where they lie apart as a whole or have the same row stride.
inline bool overlap(const Stretches &a, const Stretches &b) {
    using namespace overlap_detail;
    if (!a.p || !b.p || a.n0 < 1 || a.n1 < 1 || a.len < 1 || b.n0 < 1 || b.n1 < 1 || b.len < 1) return false;
    const auto extent = [](const Stretches &s) { return Row{0, s.n1, s.step1, Row{0, s.n0, s.step0, s.len}.extent()}.extent(); };
    if (apart(reinterpret_cast<uintptr_t>(a.p), extent(a), reinterpret_cast<uintptr_t>(b.p), extent(b))) return false;
    const Stretches x = joined(a), y = joined(b);
    const auto row = [](const Stretches &s, int64_t i) {
        return Row{reinterpret_cast<uintptr_t>(s.p) + uintptr_t(i) * uintptr_t(s.step1), s.n0, s.step0, s.len};
    };
    for (int64_t i = 0; i < x.n1; ++i)
        for (int64_t j = 0; j < y.n1; ++j)
            if (rows_share(row(x, i), row(y, j))) return true;
    return false;
}

// Bytes from one to the next of n elements `stride` apart (a dimension of one never steps: its stride may be anything).
inline int64_t step_bytes(int64_t n, int64_t stride, int64_t size) { return n > 1 ? stride * size : 0; }

// Rows of `len` bytes.
inline Stretches rows_of(const void *p, int64_t rows, int64_t step, int64_t len) { return {p, rows, step, 1, 0, len}; }

}  // namespace sdt
