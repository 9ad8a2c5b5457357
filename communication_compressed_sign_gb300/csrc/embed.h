// embed.h -- shared declarations of the input-layer operators (embedding
// lookup, its gradient, dropout); the public C ABI is include/lioncub_embed.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "lioncub_embed.h"

namespace lc {

constexpr int kStatusIndex = 8;

// Dropout as a kernel sees it.  An element's 16 random bits, placed in the top
// half of a word, stay when that word is above `limit` = T * 65536 - 1; T is
// in [1, 65536], so T == 65536 keeps nothing without a case of its own (T == 0
// is a launch without dropout).
struct DropArgs {
    uint64_t first;     // the generator's state for output 0
    uint64_t row_step;  // from a row's states to the next row's (a width that is a multiple of 4)
    uint32_t limit;
    float rescale;
};

// A matrix: row i at data + i * stride elements.
struct Rows {
    void* data;
    int64_t stride;
};

// The places of a batch (see lioncub_token_batch).
struct Places {
    const void* tokens;
    const void* positions;
    int64_t seq_len;
    int64_t first;
    int32_t n;
    int32_t wide;  // ids are int64, else int32
    int32_t vocab;
    int32_t npos;  // rows of the position table
};

// Slabs of columns that warps take a row by: 256 wide where matrices allow
// 16-byte moves, else 224.
inline int32_t slabs_of(int64_t cols, bool vec) { return static_cast<int32_t>(vec ? (cols + 255) / 256 : (cols + 223) / 224); }

struct LookupArgs {
    Places at;
    Rows table, pos_table, out;  // pos_table.data may be null
    DropArgs drop;
    float scale;
    int32_t dim;
    int32_t slabs, span;  // set by launch_lookup; span: places of a sequence
    uint32_t rounds;      // likewise
    int* status;
};

// Which number a place is sorted by.
enum KeyKind { kKeyToken = 0, kKeyPosition = 1 };

// Places a warp of the row sums takes; segments longer than this are summed in
// pieces.  At most 16, so that a stretch and a short segment's overhang fit 32
// lanes.  Less in a batch whose walks then still fit three of the four blocks
// that an SM holds, the fourth left to fills: a walk is bound by latency, so its
// places cost time while SMs are idle (16384 places of 768 columns, added in
// place: 16 a warp 25.8 us, 11 to 14 21 to 24; with the fills of a whole table
// 11 took 53 us and 14 or 16 48.6).
constexpr int kMaxPiece = 16, kMinPiece = 4, kWalkSlots = 152 * 3;
inline int64_t grad_stretches(int64_t n, int piece) { return (n + piece - 1) / piece; }
inline int grad_piece(int64_t n, int64_t slabs)
{
    for (int piece = kMinPiece; piece < kMaxPiece; ++piece)
        if ((grad_stretches(n, piece) + 7) / 8 * slabs <= kWalkSlots)
            return piece;
    return kMaxPiece;
}
// The most that a batch of up to n places has.
inline int64_t grad_max_stretches(int64_t n, int64_t slabs)
{
    const int64_t few = kWalkSlots * 8 / slabs, many = grad_stretches(n, kMaxPiece);
    const int64_t most = few > many ? few : many;
    return most < grad_stretches(n, kMinPiece) ? most : grad_stretches(n, kMinPiece);
}
// Blocks of 8 stretches, each of which may leave two partials.
inline int64_t grad_partial_rows(int64_t stretches) { return (stretches + 7) / 8 * 2; }

// The sort of a batch's places by key.  order has an entry for each place that
// has a key, grouped by key and ascending within one: (place, key, begin and end
// of the key's entries), so that what a walk needs comes with one load.
// segment[key] holds begin and end too, for every key; total counts the entries.
struct SortTask {
    Places at;
    int32_t kind;      // KeyKind
    int32_t keys;      // key values: [0, keys)
    int32_t capacity;  // entries of order (checked builds)
    int32_t log_blocks;  // set by launch_sort
    int4* order;
    int2* segment;
    int32_t* total;
};

struct SortArgs {
    SortTask task[2];
    int32_t tasks;
    uint64_t* arrived[2];  // the row sums' counters, zeroed here
    int64_t arrived_count;
    uint32_t* begun;  // set to `call` once the launches before the sort are done
    uint32_t call;    // a number of this call's own, not 0
    int* status;
};

// Row sums of dout over the segments.
struct RowSumArgs {
    Rows dout, base, grad;  // base.data null: zeros
    const int4* order;
    const int2* segment;
    const int32_t* total;
    float* partial;          // two fp32 rows for each block of stretches
    int64_t partial_stride;  // 256 for each slab
    int64_t partial_rows;
    uint64_t* arrived;       // arrivals, for each (row of partial, slab)
    DropArgs drop;
    float factor;
    int32_t rows;  // rows of grad
    int32_t dim;
    int32_t slabs, piece;  // set by launch_row_sums
    int32_t n;      // rows of dout
    uint32_t* begun;  // as in SortArgs
    uint32_t call;
    int* status;
};

struct DropoutArgs {
    Rows x, residual, out;  // residual.data may be null
    DropArgs drop;
    int64_t rows;
    int64_t cols;
};

// vec: the matrices allow 16-byte moves of 8 columns (launch_dropout: their
// starts and strides do); drop: dropout is on.
cudaError_t launch_lookup(const LookupArgs& a, int table_type, int out_type, bool vec, bool drop, cudaStream_t s);
cudaError_t launch_sort(SortArgs a, cudaStream_t s);
// Row sums of a table whose places are sorted and, in the same launch, of
// `positions` (null: none): sorted too, or running with its places `at`.  Starts
// before the launch before it, the sort of the same `call`, has ended, and waits
// for it; running positions, which do not use it, wait only until `begun` tells
// that what came before the sort is done, and leave `begun` at 0.
enum PositionKind { kNoPositions = 0, kRunningPositions = 1, kSortedPositions = 2 };
cudaError_t launch_row_sums(RowSumArgs a, const RowSumArgs* positions, PositionKind kind, const Places& at, int dout_type,
                            int grad_type, bool vec, bool drop, cudaStream_t s);
cudaError_t launch_dropout(const DropoutArgs& a, int x_type, int out_type, bool vec, bool drop, cudaStream_t s);

}  // namespace lc
