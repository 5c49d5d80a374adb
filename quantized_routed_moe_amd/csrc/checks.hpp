// Host-side checks that the operators' entry points share.
#pragma once

#include <cstdint>

#include "../../include/moe.h"
#include "grouped.hpp"

namespace qrmoe {

constexpr int64_t kMaxFeatures = 65536, kMaxStride = 1 << 21;

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
inline bool known_dtype(int dt) { return dt == MOE_DT_F32 || dt == MOE_DT_BF16 || dt == MOE_DT_F16; }

// A matrix of `rows` rows of `cols` elements at a row stride (both in elements of `bytes` bytes).
struct Mat {
    const void *p;
    int64_t rows, cols, stride;
    int bytes;
    uintptr_t begin() const { return (uintptr_t)p; }
    uintptr_t end() const { return rows > 0 ? begin() + (uintptr_t)(((rows - 1) * stride + cols) * bytes) : begin(); }
};

// Present, 16-byte aligned rows that do not overlap each other and end within the address space (what is computed from
// the row count afterwards does not wrap).
inline int check_mat(const Mat &m) {
    if (m.rows > 0 && (!m.p || !aligned16(m.p))) return MOE_ERR_INVALID_ARG;
    if (m.stride < m.cols || m.stride > INT64_MAX / m.bytes || m.stride * m.bytes % 16 != 0) return MOE_ERR_INVALID_ARG;
    if (m.stride > kMaxStride) return MOE_ERR_UNSUPPORTED;
    if (m.rows > INT64_MAX / (m.stride * m.bytes) || m.end() < m.begin()) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}
// Whether a byte belongs to both: not where their spans are apart, nor where rows of the same stride lie side by side
// (columns of one wide matrix).
inline bool overlap(const Mat &a, const Mat &b) {
    if (a.begin() >= b.end() || b.begin() >= a.end() || a.begin() == a.end() || b.begin() == b.end()) return false;
    const uintptr_t step = (uintptr_t)(a.stride * a.bytes);
    if (step != (uintptr_t)(b.stride * b.bytes)) return true;
    const uintptr_t wa = (uintptr_t)(a.cols * a.bytes), wb = (uintptr_t)(b.cols * b.bytes);
    // where b's rows begin in those of a
    const uintptr_t at = b.begin() >= a.begin() ? (b.begin() - a.begin()) % step
                                                : (step - (a.begin() - b.begin()) % step) % step;
    return at < wa || at + wb > step;
}

}  // namespace qrmoe

#define MOE_TRY(expr)                      \
    do {                                   \
        const int st_ = (expr);            \
        if (st_ != MOE_OK) return st_;     \
    } while (0)
