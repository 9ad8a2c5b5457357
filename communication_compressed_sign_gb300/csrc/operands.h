// operands.h -- what the C entries of the operators share: predicates on the
// matrices that a caller passes, environment hooks, trace ranges.
#pragma once

#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include <cstdlib>

#include "embed.h"

namespace lc {

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

inline int64_t env_index(const char* name)
{
    const char* v = std::getenv(name);
    if (!v || !*v)
        return 0;
    char* end = nullptr;
    const long long x = std::strtoll(v, &end, 10);
    return (*end == '\0' && x > 0) ? static_cast<int64_t>(x) : 0;
}

inline size_t element_size(int type) { return type == LIONCUB_ROWS_BF16 ? 2 : 4; }

// Rows of `width` bytes, `step` bytes apart.
struct Span {
    uintptr_t at;
    uintptr_t step, width;
    int64_t rows;
};

inline Span span_of(const lioncub_rows& m, int64_t rows, int64_t cols)
{
    const uintptr_t size = element_size(m.type);
    return {reinterpret_cast<uintptr_t>(m.data), m.stride * size, cols * size, rows};
}

// Whether two spans may have bytes in common: their ranges do, and they are
// not disjoint columns of rows that lie the same distance apart.
inline bool overlap(const Span& a, const Span& b)
{
    if (a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0)
        return false;
    const uintptr_t a1 = a.at + (a.rows - 1) * a.step + a.width;
    const uintptr_t b1 = b.at + (b.rows - 1) * b.step + b.width;
    if (a.at >= b1 || b.at >= a1)
        return false;
    const uintptr_t step = a.step;
    if (step != b.step)
        return true;
    const uintptr_t ahead = b.at >= a.at ? (b.at - a.at) % step : step - 1 - (a.at - b.at - 1) % step;  // (b - a) mod step
    return ahead < a.width || ahead + b.width > step;
}

inline bool overlap(const lioncub_rows& a, int64_t arows, const lioncub_rows& b, int64_t brows, int64_t cols)
{
    return overlap(span_of(a, arows, cols), span_of(b, brows, cols));
}

inline bool same_matrix(const lioncub_rows& a, const lioncub_rows& b)
{
    return a.data == b.data && a.stride == b.stride && a.type == b.type;
}

// Rows that start on 16-byte boundaries.
inline bool aligned_rows(const lioncub_rows* m)
{
    return !m || (reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && m->stride * element_size(m->type) % 16 == 0);
}

inline Rows rows_of(const lioncub_rows* m) { return m ? Rows{m->data, m->stride} : Rows{nullptr, 0}; }

}  // namespace lc
