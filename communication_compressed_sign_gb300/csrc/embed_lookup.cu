// embed_lookup.cu -- embedding lookup with scaling, position rows and dropout:
//   out[i,j] = keep(i*D+j) ? RN(r * RN(RN(scale * table[t_i,j]) + pos_table[q_i,j])) : 0.
//
// Memory-bound: a table row is read and an output row written once per place
// (repeated tokens hit L2), the mask costs integer instructions only.  One
// thread takes one group of 8 columns (one column where the width or the
// alignment does not allow 16-byte moves) of one place; see row_grid for how
// threads map to rows.
#include "embed_device.cuh"

namespace lc {
namespace {

constexpr int kLookupThreads = 256;

template <typename TT, typename OT, int V, bool DROP>
__global__ void __launch_bounds__(kLookupThreads) k_lookup(const LookupArgs a)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int32_t g = blockIdx.y * blockDim.x + threadIdx.x;
    if (i >= a.at.n || g >= a.groups)
        return;
    const int32_t j = g * V;
    const int32_t t = token_at(a.at, i, a.status);
    float y[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
        y[k] = 0.0f;
    if (t >= 0) {
        load_row<TT, V>(a.table.data, t * a.table.stride + j, y);
#pragma unroll
        for (int k = 0; k < V; ++k)
            y[k] = __fmul_rn(a.scale, y[k]);
        const int32_t q = a.pos_table.data ? position_at(a.at, i, a.status) : -1;
        if (q >= 0) {
            float p[V];
            load_row<TT, V>(a.pos_table.data, q * a.pos_table.stride + j, p);
#pragma unroll
            for (int k = 0; k < V; ++k)
                y[k] = __fadd_rn(y[k], p[k]);
        }
        if constexpr (DROP) {
            const uint32_t keep = keep_bits<V>(a.drop, static_cast<uint64_t>(i) * a.dim + j);
#pragma unroll
            for (int k = 0; k < V; ++k)
                y[k] = (keep >> k & 1u) ? __fmul_rn(a.drop.rescale, y[k]) : 0.0f;
        }
    }
    store_row<OT, V>(a.out.data, i * a.out.stride + j, y);
}

template <typename TT, typename OT, int V>
cudaError_t launch_v(const LookupArgs& a, bool drop, cudaStream_t s)
{
    const RowGrid g = row_grid(a.at.n, a.groups, kLookupThreads);
    if (drop)
        k_lookup<TT, OT, V, true><<<g.grid, g.block, 0, s>>>(a);
    else
        k_lookup<TT, OT, V, false><<<g.grid, g.block, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename TT, typename OT>
cudaError_t launch_t(LookupArgs a, bool vec, bool drop, cudaStream_t s)
{
    a.groups = vec ? a.dim / 8 : a.dim;
    return vec ? launch_v<TT, OT, 8>(a, drop, s) : launch_v<TT, OT, 1>(a, drop, s);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, int table_type, int out_type, bool vec, bool drop, cudaStream_t s)
{
    if (a.at.n == 0)
        return cudaSuccess;
    if (table_type == LIONCUB_ROWS_BF16)
        return out_type == LIONCUB_ROWS_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, vec, drop, s)
                                             : launch_t<__nv_bfloat16, float>(a, vec, drop, s);
    return out_type == LIONCUB_ROWS_BF16 ? launch_t<float, __nv_bfloat16>(a, vec, drop, s)
                                         : launch_t<float, float>(a, vec, drop, s);
}

}  // namespace lc
