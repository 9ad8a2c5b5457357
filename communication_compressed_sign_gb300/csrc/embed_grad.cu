// embed_grad.cu -- gradient of the embedding lookup:
//   grad[v,:] = base[v,:] + f * sum over places i with key_i == v of keep * dout[i,:].
//
// Two launches: a sort of the places by key, then one thread per (row, column
// group) that adds the rows of dout of its key's places in ascending order and
// writes the row once -- rows without a place as zeros (or base), so the dense
// gradient needs no clearing pass and no atomics, and the order of every sum
// depends on the batch alone.
#include "embed_device.cuh"

namespace lc {
namespace {

// --- sort ------------------------------------------------------------------------
//
// Counting sort without communication between blocks: block r owns the keys
// with key % R == r (interleaved, so that frequent low ids spread over the
// blocks) and reads all keys itself: it counts those of lower blocks, which
// gives the base of its part of `order`, and its own per key and warp.  After
// a scan it reads the keys again and places its own.  Each warp takes a
// contiguous slice of the places in order, so places stay ascending within a
// key.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortKeys = kSortThreads;  // keys a block can own: one per thread in the scan

template <int KIND>
__device__ __forceinline__ int32_t sort_key(const SortArgs& a, int64_t i, int* status)
{
    const int32_t t = token_at(a.at, i, status);
    if (KIND == kKeyToken || t < 0)
        return t;
    return position_at(a.at, i, status);
}

template <int KIND>
__global__ void __launch_bounds__(kSortThreads) k_sort(const SortArgs a, int log_blocks)
{
    __shared__ int cnt[kSortWarps][kSortKeys];
    __shared__ int part[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int mask = (1 << log_blocks) - 1;
    const int mine = blockIdx.x;
    const int owned = mine < a.keys ? ((a.keys - 1 - mine) >> log_blocks) + 1 : 0;
    for (int k = tid; k < kSortWarps * kSortKeys; k += kSortThreads)
        (&cnt[0][0])[k] = 0;
    __syncthreads();

    const int64_t slice = (a.at.n + kSortThreads - 1) / kSortThreads * 32;
    const int64_t lo = warp * slice, hi = min(lo + slice, static_cast<int64_t>(a.at.n));
    int below = 0;
    int* status = mine == 0 ? a.status : nullptr;
    for (int64_t i = lo + lane; i < hi; i += 32) {
        const int32_t key = sort_key<KIND>(a, i, status);
        if (key < 0)
            continue;
        const int b = key & mask;
        below += b < mine ? 1 : 0;
        if (b == mine)
            atomicAdd(&cnt[warp][key >> log_blocks], 1);
    }
    below = __reduce_add_sync(0xffffffffu, below);
    if (lane == 0)
        part[warp] = below;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w)
        base += part[w];
    __syncthreads();

    // thread k: key k's total, then its start, then a start for each warp
    int total = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w)
        total += cnt[w][tid];
    int run = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, run, o);
        run += lane >= o ? up : 0;
    }
    if (lane == 31)
        part[warp] = run;
    __syncthreads();
    int start = base + run - total;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w)
        start += w < warp ? part[w] : 0;
    if (tid < owned) {
        const int32_t key = (tid << log_blocks) | mine;
        if (index_ok(a.status, key < a.keys && start + total <= a.capacity))
            a.segment[key] = make_int2(start, start + total);
    }
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w][tid];
        cnt[w][tid] = start;
        start += c;
    }
    __syncthreads();

    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const int64_t i = i0 + lane;
        const int32_t key = i < hi ? sort_key<KIND>(a, i, nullptr) : -1;
        const bool take = key >= 0 && (key & mask) == mine;
        const unsigned takers = __ballot_sync(0xffffffffu, take);
        if (take) {
            const int k = key >> log_blocks;
            const unsigned same = __match_any_sync(takers, k);
            const int at = cnt[warp][k] + __popc(same & ((1u << lane) - 1));
            __syncwarp(takers);
            if ((same >> lane) == 1u)  // the last lane with this key
                cnt[warp][k] = at + 1;
            __syncwarp(takers);
            if (index_ok(a.status, at >= 0 && at < a.capacity))
                a.order[at] = static_cast<int32_t>(i);
        }
        __syncwarp();
    }
}

// --- row sums ----------------------------------------------------------------------

constexpr int kSumThreads = 256;

template <typename DT, typename GT, int V, bool DROP>
__global__ void __launch_bounds__(kSumThreads) k_row_sums(const RowSumArgs a)
{
    const int64_t v = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int32_t g = blockIdx.y * blockDim.x + threadIdx.x;
    if (v >= a.rows || g >= a.groups)
        return;
    const int32_t j = g * V;
    const int2 seg = a.segment[v];
    if (seg.x == seg.y && a.base.data == a.grad.data)
        return;
    float sum[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
        sum[k] = 0.0f;
    for (int p = seg.x; p < seg.y; ++p) {
        const int64_t i = a.order[p];
        if (!index_ok(a.status, i >= 0 && i < a.n))
            continue;
        float x[V];
        load_row<DT, V>(a.dout.data, i * a.dout.stride + j, x);
        const uint32_t keep = DROP ? keep_bits<V>(a.drop, static_cast<uint64_t>(i) * a.dim + j) : 0xffu;
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (keep >> k & 1u)
                sum[k] = __fadd_rn(sum[k], x[k]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
        sum[k] = __fmul_rn(a.factor, sum[k]);
    if (a.base.data) {
        float b[V];
        load_row<GT, V>(a.base.data, v * a.base.stride + j, b);
#pragma unroll
        for (int k = 0; k < V; ++k)
            sum[k] = __fadd_rn(b[k], sum[k]);
    }
    store_row<GT, V>(a.grad.data, v * a.grad.stride + j, sum);
}

template <typename DT, typename GT, int V>
cudaError_t launch_v(const RowSumArgs& a, bool drop, cudaStream_t s)
{
    const RowGrid g = row_grid(a.rows, a.groups, kSumThreads);
    if (drop)
        k_row_sums<DT, GT, V, true><<<g.grid, g.block, 0, s>>>(a);
    else
        k_row_sums<DT, GT, V, false><<<g.grid, g.block, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename DT, typename GT>
cudaError_t launch_t(RowSumArgs a, bool vec, bool drop, cudaStream_t s)
{
    a.groups = vec ? a.dim / 8 : a.dim;
    return vec ? launch_v<DT, GT, 8>(a, drop, s) : launch_v<DT, GT, 1>(a, drop, s);
}

}  // namespace

cudaError_t launch_sort(const SortArgs& a, KeyKind kind, cudaStream_t s)
{
    int log_blocks = 8;
    while ((static_cast<int64_t>(kSortKeys) << log_blocks) < a.keys)
        ++log_blocks;
    const int blocks = 1 << log_blocks;
    if (kind == kKeyToken)
        k_sort<kKeyToken><<<blocks, kSortThreads, 0, s>>>(a, log_blocks);
    else
        k_sort<kKeyPosition><<<blocks, kSortThreads, 0, s>>>(a, log_blocks);
    return cudaGetLastError();
}

cudaError_t launch_row_sums(const RowSumArgs& a, int dout_type, int grad_type, bool vec, bool drop, cudaStream_t s)
{
    if (dout_type == LIONCUB_ROWS_BF16)
        return grad_type == LIONCUB_ROWS_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, vec, drop, s)
                                              : launch_t<__nv_bfloat16, float>(a, vec, drop, s);
    return grad_type == LIONCUB_ROWS_BF16 ? launch_t<float, __nv_bfloat16>(a, vec, drop, s)
                                          : launch_t<float, float>(a, vec, drop, s);
}

}  // namespace lc
