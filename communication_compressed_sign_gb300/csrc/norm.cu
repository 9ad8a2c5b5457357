// norm.cu -- the root-mean-square norm of rows, with the residual added before
// and 8-bit codes of the sum and of the result after:
//   h = x + residual,  out = h * rstd * weight,  rstd = 1 / sqrt(mean(h^2) + eps).
//
// Memory-bound.  A row stays in the registers of one or more warps from its only
// reading to its writing; one sum over the row stands between (a cluster or a
// second reading is not needed: 16384 columns are 16 warps of 32 elements a lane;
// above 8192 columns fp32 rows spill 108 bytes a thread, scalar moves 308).
// Measured: 65536 x 2048 bf16 with a residual into e4m3 134.8 us (7.0 TB/s, above a
// measured copy's rate), 8192 x 768 onto an fp32 residual 12.7 us (5.9 TB/s), 4907
// x 771 fp32 11.1 us (5.5 TB/s, scalar moves), 8 rows 1.5 us.  Rows of 3905 bf16
// with one scale each, by scalar moves, take 161 us for 41152 (3.0 TB/s): about 30
// instructions an element, half of them a warp's overhead, and two barriers a row.
// With the sum kept in bf16 and in int8 for the backward pass, 65536 x 2048 bf16 175
// us (6.9 TB/s); 4096 x 16384 bf16 60.0 us (6.7 TB/s), fp32 128 us (6.3 TB/s).
#include <climits>

#include "block_device.cuh"

namespace lc {
namespace {

constexpr int kMaxWarps = 16;  // of a row
constexpr int kRowsOfWarps = 8;  // rows of a block, where a row is one warp's

// The sum over a row of what each of its warps has, and likewise the largest.
__device__ __forceinline__ float row_sum(float v, float* shared, int warps, int warp, int lane)
{
    v = warp_sum(v);
    if (warps > 1) {
        if (lane == 0)
            shared[warp] = v;
        __syncthreads();
        v = sum_of_warps(shared, warps, lane);
    }
    return v;
}

__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* shared, int warps, int warp, int lane)
{
    v = __reduce_max_sync(kAll, v);
    if (warps > 1) {
        if (lane == 0)
            shared[warp] = v;
        __syncthreads();
        v = __reduce_max_sync(kAll, lane < warps ? shared[lane] : 0);
    }
    return v;
}

// The codes of a row whose chunks are in x.
template <int C, bool VEC>
__device__ __forceinline__ void pack_row(const PackedRows& p, const Columns<VEC> (&cols)[C], int64_t row, const float (&x)[C][8],
                                         uint32_t* shared, int warps, int warp, int lane)
{
    if (p.log_group != kRowGroup) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            pack_chunk<VEC>(p, cols[c], row, x[c], largest_of(x[c]), lane);
        return;
    }
    uint32_t largest = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
        largest = max(largest, largest_of(x[c]));
    const GroupScale s(row_max(largest, shared, warps, warp, lane), p.e4m3);
#pragma unroll
    for (int c = 0; c < C; ++c)
        pack_chunk_of_row<VEC>(p, cols[c], row, x[c], s);
    if (warp == 0 && lane == 0 && scale_inside(p, row, 0))
        p.scales[row * p.scale_stride] = s.scale;
}

// A row is that of `warps` warps, C neighbouring chunks each.  Registers are capped
// for three blocks of 16 warps an SM: 41152 rows of 3905 bf16, whose scalar moves are
// 64 bytes a warp, took 202 us with the 64 of before, 161 so.
template <typename XT, typename RT, int C, bool VEC, bool WARP_ROWS>
__global__ void __launch_bounds__(kMaxWarps * 32, C <= 2 ? 3 : 2) k_norm(const __grid_constant__ NormArgs a)
{
    __shared__ float sums[kMaxWarps];
    __shared__ uint32_t maxima[2][kMaxWarps];
    const int lane = threadIdx.x & 31, in_block = threadIdx.x >> 5;
    const int warps = WARP_ROWS ? 1 : a.warps, warp = WARP_ROWS ? 0 : in_block;
    const int64_t row = WARP_ROWS ? static_cast<int64_t>(blockIdx.x) * kRowsOfWarps + in_block : blockIdx.x;
    wait_for_launch_before();
    if (WARP_ROWS && row >= a.n)
        return;
    Columns<VEC> cols[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        cols[c] = Columns<VEC>((warp * C + c) * kChunk, lane, a.dim);

    float h[C][8];
    {
        Chunk<XT, VEC> x[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            load_row(x[c], cols[c], a.x, row);
        if (a.residual.data) {
            Chunk<RT, VEC> r[C];
#pragma unroll
            for (int c = 0; c < C; ++c)
                load_row(r[c], cols[c], a.residual, row);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float y[8];
                x[c].unpack(h[c]);
                r[c].unpack(y);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    set_pair(h[c], k, add2(pair_of(h[c], k), pair_of(y, k)));
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                x[c].unpack(h[c]);
        }
    }
    if (a.summed.data)
#pragma unroll
        for (int c = 0; c < C; ++c)
            store_typed<VEC>(cols[c], a.summed, row, h[c]);

    float2 squares = both(0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            squares = fma2(pair_of(h[c], k), pair_of(h[c], k), squares);
    float sum = __fadd_rn(squares.x, squares.y);
    sum = row_sum(sum, sums, warps, warp, lane);
    const float rstd = rsqrtf(fmaf(sum, a.per_column, a.eps));
    if (a.rstd && warp == 0 && lane == 0 && access_ok(row < a.n))
        a.rstd[row] = rstd;
    if (a.saved.codes)
        pack_row<C, VEC>(a.saved, cols, row, h, maxima[0], warps, warp, lane);

#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            set_pair(h[c], k, mul2(pair_of(h[c], k), both(rstd)));
        if (a.weight.data) {
            float w[8];
            load_typed<VEC>(cols[c], a.weight, 0, w);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                set_pair(h[c], k, mul2(pair_of(h[c], k), pair_of(w, k)));
        }
    }
    if (a.packed.codes) {
        pack_row<C, VEC>(a.packed, cols, row, h, maxima[1], warps, warp, lane);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            store_typed<VEC>(cols[c], a.out, row, h[c]);
    }
}

// The codes of rows that have one scale each.
template <typename XT, int C, bool VEC>
__global__ void __launch_bounds__(kMaxWarps * 32) k_pack_rows(const TypedRows x, const PackedRows out, const int64_t rows, const int dim,
                                                              const int warps)
{
    __shared__ uint32_t maxima[kMaxWarps];
    const int lane = threadIdx.x & 31, in_block = threadIdx.x >> 5, warp = warps == 1 ? 0 : in_block;
    const int64_t row = warps == 1 ? static_cast<int64_t>(blockIdx.x) * kRowsOfWarps + in_block : blockIdx.x;
    wait_for_launch_before();
    if (row >= rows)
        return;
    Columns<VEC> cols[C];
    Chunk<XT, VEC> v[C];
    float h[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        cols[c] = Columns<VEC>((warp * C + c) * kChunk, lane, dim);
        load_row(v[c], cols[c], x, row);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        v[c].unpack(h[c]);
    pack_row<C, VEC>(out, cols, row, h, maxima, warps, warp, lane);
}

// How a row of `dim` columns is spread: C chunks for each of `warps` warps.  Two,
// but one while there are few chunks in all, whose rows are then done sooner (8
// rows of 768: 1.5 us, with two 2.0, with three 2.9; 8192 rows onto an fp32
// residual 12.8, 13.6, 14.0), though not of wide rows, whose barriers then cost more
// (2048 rows of 2048: 6.6 and 6.2; 65536: 170 and 139).
struct Spread {
    int c, warps;
    Spread(int64_t rows, int dim)
    {
        const int chunks = (dim + kChunk - 1) / kChunk;
        const int64_t all = rows * chunks;
        c = chunks <= kMaxWarps && (all <= 4096 || (chunks <= 4 && all <= 32768)) ? 1 : chunks <= 2 * kMaxWarps ? 2 : 4;
        c = c < chunks ? c : chunks;
        warps = (chunks + c - 1) / c;
    }
};

// f(integral constant C) for the spread's C
template <typename F>
cudaError_t with_chunks(int c, F&& f)
{
    switch (c) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    default: return f(std::integral_constant<int, 4>());
    }
}

unsigned row_blocks(int64_t rows, int warps) { return static_cast<unsigned>(warps == 1 ? (rows + kRowsOfWarps - 1) / kRowsOfWarps : rows); }
int row_threads(int warps) { return 32 * (warps == 1 ? kRowsOfWarps : warps); }

template <typename XT, typename RT, bool VEC>
cudaError_t launch_t(const NormArgs& a, int c, cudaStream_t s)
{
    return with_chunks(c, [&](auto n) {
        constexpr int C = decltype(n)::value;
        if constexpr (C <= 2)
            if (a.warps == 1)
                return launch_programmatic(k_norm<XT, RT, C, VEC, true>, row_blocks(a.n, 1), row_threads(1), 0, s, a);
        return launch_programmatic(k_norm<XT, RT, C, VEC, false>, row_blocks(a.n, a.warps), row_threads(a.warps), 0, s, a);
    });
}

}  // namespace

#ifdef LIONCUB_BOUNDS_CHECK
cudaError_t take_norm_word(int* word) { return take_word(word); }
#endif

cudaError_t launch_norm(NormArgs a, bool vec, cudaStream_t s)
{
    if (a.n == 0)
        return cudaSuccess;
    const Spread spread(a.n, a.dim);
    a.warps = spread.warps;
    a.per_column = 1.0f / static_cast<float>(a.dim);
    if (!vec)
        return launch_t<float, float, false>(a, spread.c, s);
    const bool xb = a.x.type == LIONCUB_ROWS_BF16, rb = a.residual.type == LIONCUB_ROWS_BF16;
    if (xb)
        return rb ? launch_t<__nv_bfloat16, __nv_bfloat16, true>(a, spread.c, s) : launch_t<__nv_bfloat16, float, true>(a, spread.c, s);
    return rb ? launch_t<float, __nv_bfloat16, true>(a, spread.c, s) : launch_t<float, float, true>(a, spread.c, s);
}

cudaError_t launch_pack_rows(const TypedRows& x, const PackedRows& out, int64_t rows, int dim, bool vec, cudaStream_t s)
{
    const Spread spread(rows, dim);
    return with_chunks(spread.c, [&](auto n) {
        constexpr int C = decltype(n)::value;
        const unsigned blocks = row_blocks(rows, spread.warps);
        const int threads = row_threads(spread.warps);
        if (!vec)
            return launch_programmatic(k_pack_rows<float, C, false>, blocks, threads, 0, s, x, out, rows, dim, spread.warps);
        return x.type == LIONCUB_ROWS_BF16
                   ? launch_programmatic(k_pack_rows<__nv_bfloat16, C, true>, blocks, threads, 0, s, x, out, rows, dim, spread.warps)
                   : launch_programmatic(k_pack_rows<float, C, true>, blocks, threads, 0, s, x, out, rows, dim, spread.warps);
    });
}

}  // namespace lc
