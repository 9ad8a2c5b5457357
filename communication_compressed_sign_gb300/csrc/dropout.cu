// dropout.cu -- dropout over a matrix, with an optional residual added:
//   out[e] = (keep(e) ? RN(r * x[e]) : 0) (+ residual[e]).
// The backward pass is the same map of the gradient, with the mask drawn again
// from the same counters.
//
// Memory-bound: each element is read and written once and no mask exists in
// memory.  One thread takes a group of 8 elements (one where rows are apart and
// not 16-byte aligned).
#include "embed_device.cuh"

namespace lc {
namespace {

constexpr int kDropoutThreads = 256;

// Elements [e, e + V) of a matrix whose rows start at these element offsets.
template <typename XT, typename OT, int V, bool DROP>
__device__ __forceinline__ void drop_group(const DropoutArgs& a, int64_t e, int64_t ex, int64_t er, int64_t eo)
{
    float x[V];
    load_row<XT, V>(a.x.data, ex, x);
    if constexpr (DROP) {
        auto scale = [&](int k, bool keep) { x[k] = keep ? __fmul_rn(a.drop.rescale, x[k]) : 0.0f; };
        if constexpr (V == 8)
            for_kept8(a.drop, a.drop.first + (static_cast<uint64_t>(e) >> 2) * kSplitMix64Step, scale);
        else
            scale(0, stays1(a.drop, e));
    }
    if (a.residual.data) {
        float y[V];
        load_row<OT, V>(a.residual.data, er, y);
#pragma unroll
        for (int k = 0; k < V; ++k)
            x[k] = __fadd_rn(x[k], y[k]);
    }
    store_row<OT, V>(a.out.data, eo, x);
}

// Dense matrices: one flat vector, whatever the width, the last group ragged.
template <typename XT, typename OT, bool DROP>
__global__ void __launch_bounds__(kDropoutThreads) k_dropout_flat(const DropoutArgs a)
{
    const int64_t n = a.rows * a.cols;
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * kDropoutThreads + threadIdx.x) * 8;
    if (e + 8 <= n)
        drop_group<XT, OT, 8, DROP>(a, e, e, e, e);
    else
        for (int64_t k = e; k < n; ++k)
            drop_group<XT, OT, 1, DROP>(a, k, k, k, k);
}

// Rows apart from one another (or not 16-byte aligned).
template <typename XT, typename OT, int V, bool DROP>
__global__ void __launch_bounds__(kDropoutThreads) k_dropout_rows(const DropoutArgs a)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t j = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * V;
    if (i < a.rows && j < a.cols)
        drop_group<XT, OT, V, DROP>(a, i * a.cols + j, i * a.x.stride + j, i * a.residual.stride + j,
                                    i * a.out.stride + j);
}

template <typename XT, typename OT, bool DROP>
cudaError_t launch_t(const DropoutArgs& a, bool vec, cudaStream_t s)
{
    const bool dense = a.x.stride == a.cols && a.out.stride == a.cols && (!a.residual.data || a.residual.stride == a.cols);
    if (vec && dense) {
        const int64_t blocks = (a.rows * a.cols + kDropoutThreads * 8 - 1) / (kDropoutThreads * 8);
        k_dropout_flat<XT, OT, DROP><<<static_cast<unsigned>(blocks), kDropoutThreads, 0, s>>>(a);
    } else if (vec && a.cols % 8 == 0) {
        const RowGrid g = row_grid(a.rows, a.cols / 8, kDropoutThreads);
        k_dropout_rows<XT, OT, 8, DROP><<<g.grid, g.block, 0, s>>>(a);
    } else {
        const RowGrid g = row_grid(a.rows, a.cols, kDropoutThreads);
        k_dropout_rows<XT, OT, 1, DROP><<<g.grid, g.block, 0, s>>>(a);
    }
    return cudaGetLastError();
}

template <typename XT, typename OT>
cudaError_t launch_d(const DropoutArgs& a, bool vec, bool drop, cudaStream_t s)
{
    return drop ? launch_t<XT, OT, true>(a, vec, s) : launch_t<XT, OT, false>(a, vec, s);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int x_type, int out_type, bool vec, bool drop, cudaStream_t s)
{
    if (a.rows == 0 || a.cols == 0)
        return cudaSuccess;
    if (x_type == LIONCUB_ROWS_BF16)
        return out_type == LIONCUB_ROWS_BF16 ? launch_d<__nv_bfloat16, __nv_bfloat16>(a, vec, drop, s)
                                             : launch_d<__nv_bfloat16, float>(a, vec, drop, s);
    return out_type == LIONCUB_ROWS_BF16 ? launch_d<float, __nv_bfloat16>(a, vec, drop, s)
                                         : launch_d<float, float>(a, vec, drop, s);
}

}  // namespace lc
