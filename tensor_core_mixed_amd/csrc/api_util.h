// Argument checks shared by the C entries: extents of matrices, overlap,
// alignment, statuses.
#pragma once
#include <cstdint>
#include <exception>

#include "../../include/tcm.h"

namespace tcm {

constexpr int64_t kDim = (int64_t)1 << 31;

// bytes of a rows x cols matrix of leading dimension ld; -1 past 2^62
inline int64_t span_of(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
    if (rows == 0 || cols == 0) return 0;
    if (rows > 1 && ld > (((int64_t)1 << 60) - cols) / (rows - 1)) return -1;
    const int64_t n = (rows - 1) * ld + cols;
    return n > ((int64_t)1 << 62) / es ? -1 : n * es;
}

struct Region {
    const void* p;
    int64_t bytes;
};
inline bool cross(const Region& a, const Region& b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const char *x = (const char*)a.p, *y = (const char*)b.p;
    return x < y + b.bytes && y < x + a.bytes;
}
// no output crosses another output or an input
template <int NO, int NI>
bool disjoint(const Region (&out)[NO], const Region (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (cross(out[i], out[j])) return false;
        for (const Region& r : in)
            if (cross(out[i], r)) return false;
    }
    return true;
}
inline bool word_aligned(const void* p) { return ((uintptr_t)p & 3) == 0; }

inline int done(int hip_status) { return hip_status == 0 ? TCM_OK : TCM_ERR_HIP; }

// nothing thrown on the host (memory, a lock) leaves a C entry
template <class F>
int guarded(F f) {
    try {
        return f();
    } catch (const std::exception&) {
        return TCM_ERR_ALLOC;
    }
}

}  // namespace tcm
