// block.h -- shared declarations of the block operators (norm, 8-bit
// checkpoints, activation, rotary positions); the public C ABI is
// include/lioncub_block.h.
#pragma once

#include "embed.h"
#include "lioncub_block.h"

namespace lc {

// A matrix with the type of its elements (LIONCUB_ROWS_*); data may be null.
struct TypedRows {
    void* data;
    int64_t stride;
    int32_t type;
#ifdef LIONCUB_BOUNDS_CHECK
    int64_t rows, cols;
#endif
};

// A matrix in 8 bits; codes may be null.  Groups are 1 << log_group columns, or
// the whole row (kRowGroup).
constexpr int kRowGroup = 62;
struct PackedRows {
    uint8_t* codes;
    float* scales;
    int64_t stride, scale_stride;
    int64_t cols;
    int32_t log_group;
    int32_t e4m3;  // else whole numbers
    float one;     // 1 (see codes8)
#ifdef LIONCUB_BOUNDS_CHECK
    int64_t rows;
#endif
};

struct NormArgs {
    TypedRows x, residual, weight, summed, out;
    PackedRows saved, packed;  // the sum's and the result's codes
    float* rstd;
    int64_t n;
    int32_t dim;
    int32_t warps;  // of a row; set by launch_norm, per_column too
    float eps;
    float per_column;  // 1 / dim
};

struct NormGradArgs {
    TypedRows dout, saved, residual_grad, dx, weight, again;
    PackedRows packed;
    const float* rstd;
    float* partial;  // a row of dim for each block, null: no weight gradient
    int64_t partial_rows;
    int64_t n;
    int32_t dim;
    // set by launch_norm_grad: warps of a row, rows at once in a block, rows in flight for each
    // of those, bytes of such a row and where its parts begin, 1 / dim
    int32_t warps, teams, slots, slot_bytes, at_saved, at_residual;
    float per_column;
    uint32_t first_wait_polls;  // fault injection: >0 caps the first wait for copies at this many polls
    int* status;
};

struct WeightGradArgs {
    const float* partial;
    int32_t rows;  // of partial
    TypedRows base, grad;
    int32_t dim;
};

struct ActivationArgs {
    TypedRows x, up, out;           // forward; backward: x and up null where packed
    TypedRows dout, dx, dup, again;  // backward
    PackedRows saved, saved_up;     // forward: written; backward: read
    int64_t rows, cols;
};

struct HeadsArgs {
    const void* in;
    void* out;
    int64_t in_batch, in_place, in_head, out_batch, out_place, out_head;
#ifdef LIONCUB_BOUNDS_CHECK
    const char *in_end, *out_end;
#endif
};

struct RotaryArgs {
    HeadsArgs side[2];
    int32_t heads[2];
    const uint64_t* turns;  // of each pair: turns a position, in units of 2^-64
    const void* positions;
    int64_t first;
    int64_t places;  // of all sequences
    int32_t seq;
    int32_t wide;  // positions are int64, else int32
    int32_t head_dim, pairs;
    int32_t copy;  // columns behind the rotated ones are copied
    float cos_factor, sin_factor;
};

// vec: the matrices allow 16-byte moves.
cudaError_t launch_norm(NormArgs a, bool vec, cudaStream_t s);
// Its blocks, one for each multiprocessor at most, leave a row of partial sums each.
int norm_grad_blocks(int64_t n, int dim, int multiprocessors);
cudaError_t launch_norm_grad(NormGradArgs a, int blocks, bool vec, cudaStream_t s);
cudaError_t launch_weight_grad(const WeightGradArgs& a, cudaStream_t s);
// Codes with one scale a row (forward norms without the norm).
cudaError_t launch_pack_rows(const TypedRows& x, const PackedRows& out, int64_t rows, int dim, bool vec, cudaStream_t s);
// kind: LIONCUB_ACTIVATION_*, or kIdentity (out may then be null: x is only packed).
constexpr int kIdentity = -1;
cudaError_t launch_activation(const ActivationArgs& a, int kind, bool vec, cudaStream_t s);
cudaError_t launch_activation_grad(const ActivationArgs& a, int kind, bool vec, cudaStream_t s);
cudaError_t launch_unpack(const PackedRows& x, const TypedRows& out, int64_t rows, int64_t cols, bool vec, cudaStream_t s);
// move: elements at a time, 8 (then 16-byte aligned, and whole halves of 8 pairs), 4, 2 or 1.
// copy_by_four: columns that are copied may be moved four at a time.
cudaError_t launch_rotary(const RotaryArgs& a, int type, bool interleaved, int move, bool copy_by_four, cudaStream_t s);

#ifdef LIONCUB_BOUNDS_CHECK
// Checked builds: each file of kernels has a word that they set bits of (kStatusOutOfBounds)
// for an access that lies outside, which is left out.  Reads and clears it; synchronizes.
cudaError_t take_norm_word(int* word);
cudaError_t take_norm_grad_word(int* word);
cudaError_t take_activation_word(int* word);
cudaError_t take_rotary_word(int* word);
#endif

}  // namespace lc
