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
    uint64_t key;
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

struct LookupArgs {
    Places at;
    Rows table, pos_table, out;  // pos_table.data may be null
    DropArgs drop;
    float scale;
    int32_t dim;
    int32_t groups;  // column groups of the kernel's vector width in a row
    int* status;
};

// Which number a place is sorted by.
enum KeyKind { kKeyToken = 0, kKeyPosition = 1 };

// Segments longer than this are summed in pieces, cut at its multiples.
constexpr int kGradPiece = 64;
inline int64_t grad_stretches(int64_t n) { return (n + kGradPiece - 1) / kGradPiece; }

// The sort of a batch's places by key: order holds the places grouped by key,
// ascending within a key, sorted_key their keys; segment[key] is the key's
// range in order, total the number of places that have a key.
struct SortArgs {
    Places at;
    int32_t keys;      // key values: [0, keys)
    int32_t capacity;  // entries of order (checked builds)
    int32_t* order;
    int32_t* sorted_key;
    int2* segment;
    int32_t* total;
    int* status;
};

// Row sums of dout over the segments.
struct RowSumArgs {
    Rows dout, base, grad;  // base.data null: zeros
    const int32_t* order;
    const int32_t* sorted_key;
    const int2* segment;
    const int32_t* total;
    float* partial;          // two fp32 rows a stretch of kGradPiece places
    int64_t partial_stride;  // dim rounded up to 16 bytes
    int64_t partial_rows;
    DropArgs drop;
    float factor;
    int32_t rows;    // rows of grad
    int32_t dim;
    int32_t groups;
    int32_t n;       // rows of dout
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
cudaError_t launch_sort(const SortArgs& a, KeyKind kind, cudaStream_t s);
cudaError_t launch_row_sums(const RowSumArgs& a, int dout_type, int grad_type, bool vec, bool drop, cudaStream_t s);
cudaError_t launch_dropout(const DropoutArgs& a, int x_type, int out_type, bool vec, bool drop, cudaStream_t s);

// Column groups of a row -> thread blocks: TX threads along a row, TY rows a
// block, so that a thread's row and columns need no division and nearly every
// thread of a block has work whatever the width.
struct RowGrid {
    dim3 block, grid;
};
inline RowGrid row_grid(int64_t rows, int64_t groups, int threads)
{
    const int64_t slabs = (groups + threads - 1) / threads;
    const int64_t tx = (groups + slabs - 1) / slabs;
    const int64_t ty = threads / tx;
    RowGrid g;
    g.block = dim3(static_cast<unsigned>(tx), static_cast<unsigned>(ty));
    g.grid = dim3(static_cast<unsigned>((rows + ty - 1) / ty), static_cast<unsigned>(slabs));
    return g;
}

}  // namespace lc
