// embed_grad.cu -- gradient of the embedding lookup:
//   grad[v,:] = base[v,:] + f * sum over places i with key_i == v of keep * dout[i,:].
//
// A sort of the places by key, then one thread per (row, column group) that adds
// the rows of dout of its key's places in ascending order and writes the row
// once -- rows without a place as zeros (or base), so the dense gradient needs
// no clearing pass and no atomics, and the order of every sum depends on the
// batch alone.
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
    if (mine == (1 << log_blocks) - 1 && tid == kSortThreads - 1)
        *a.total = start + total;
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
            if (index_ok(a.status, at >= 0 && at < a.capacity)) {
                a.order[at] = static_cast<int32_t>(i);
                a.sorted_key[at] = key;
            }
        }
        __syncwarp();
    }
}

// --- row sums ----------------------------------------------------------------------
//
// Rows of up to kLong places are added by the threads of their row.  Longer
// segments would leave a few threads adding thousands of rows (token
// frequencies follow a power law), so they are cut at the multiples of kLong
// of `order`: each piece is summed by a row of threads of its own into an fp32
// partial, and a second launch adds a segment's partials in order.  A stretch
// of kLong entries holds at most two pieces of long segments: the end of one
// that began before it (slot 0) and the begin of one that goes on (slot 1).
constexpr int kSumThreads = 256;
constexpr int kLong = kGradPiece;
constexpr int kInFlight = 4;  // rows of dout a thread loads before it adds them

// Adds the rows of dout of the places order[lo..hi) to sum, in order.
template <typename DT, int V, bool DROP>
__device__ __forceinline__ void add_places(const RowSumArgs& a, int lo, int hi, int32_t j, float (&sum)[V])
{
    for (int p = lo; p < hi; p += kInFlight) {
        Group<DT, V> x[kInFlight];
        int64_t i[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            i[u] = p + u < hi ? a.order[p + u] : -1;
            if (!index_ok(a.status, i[u] < a.n && (i[u] >= 0 || p + u >= hi)))
                i[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (i[u] >= 0)
                x[u].load(a.dout.data, i[u] * a.dout.stride + j);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            if (i[u] < 0)
                continue;
            const uint32_t keep = DROP ? keep_bits<V>(a.drop, static_cast<uint64_t>(i[u]) * a.dim + j) : 0xffu;
            float y[V];
            x[u].unpack(y);
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (keep >> k & 1u)
                    sum[k] = __fadd_rn(sum[k], y[k]);
        }
    }
}

// grad[v, j..j+V) = base + factor * sum.
template <typename GT, int V>
__device__ __forceinline__ void finish_row(const RowSumArgs& a, int64_t v, int32_t j, float (&sum)[V])
{
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

// The pieces of long segments in entries [c * kLong, (c + 1) * kLong) of
// order: [lo[s], hi[s]) for slot s, empty when there is none.  key[s]: whose.
__device__ __forceinline__ void pieces_of(const RowSumArgs& a, int64_t c, int total, int (&lo)[2], int (&hi)[2], int (&key)[2])
{
    const int begin = static_cast<int>(c * kLong), end = static_cast<int>(min((c + 1) * kLong, static_cast<int64_t>(total)));
    lo[0] = hi[0] = lo[1] = hi[1] = 0;
    key[0] = key[1] = -1;
    if (begin >= end)
        return;
    const int first = a.sorted_key[begin], last = a.sorted_key[end - 1];
    const int2 f = a.segment[first], l = a.segment[last];
    if (f.x < begin && f.y - f.x > kLong) {
        lo[0] = begin;
        hi[0] = min(f.y, end);
        key[0] = first;
    }
    if (l.x >= begin && l.y - l.x > kLong) {
        lo[1] = l.x;
        hi[1] = end;
        key[1] = last;
    }
}

// Blocks [0, piece_blocks) of a column slab sum pieces, the others rows.
template <typename DT, typename GT, int V, bool DROP>
__global__ void __launch_bounds__(kSumThreads) k_row_sums(const RowSumArgs a, unsigned piece_blocks)
{
    const int32_t g = blockIdx.y * blockDim.x + threadIdx.x;
    if (g >= a.groups)
        return;
    const int32_t j = g * V;
    if (blockIdx.x < piece_blocks) {
        const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
        int lo[2], hi[2], key[2];
        pieces_of(a, c, *a.total, lo, hi, key);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (lo[s] == hi[s])
                continue;
            float sum[V];
#pragma unroll
            for (int k = 0; k < V; ++k)
                sum[k] = 0.0f;
            add_places<DT, V, DROP>(a, lo[s], hi[s], j, sum);
            if (index_ok(a.status, 2 * c + s < a.partial_rows))
                store_row<float, V>(a.partial, (2 * c + s) * a.partial_stride + j, sum);
        }
        return;
    }
    const int64_t v = static_cast<int64_t>(blockIdx.x - piece_blocks) * blockDim.y + threadIdx.y;
    if (v >= a.rows)
        return;
    const int2 seg = a.segment[v];
    if (seg.y - seg.x > kLong || (seg.x == seg.y && a.base.data == a.grad.data))
        return;
    float sum[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
        sum[k] = 0.0f;
    add_places<DT, V, DROP>(a, seg.x, seg.y, j, sum);
    finish_row<GT, V>(a, v, j, sum);
}

// Adds the partials of the long segment that begins in stretch c, if one does:
// a block's 8 warps each add a contiguous share of its pieces in order, warp 0
// the shares in order.
constexpr int kJoinWarps = 8;
template <typename GT, int V>
__global__ void __launch_bounds__(kJoinWarps * 32) k_join_pieces(const RowSumArgs a)
{
    __shared__ float share[kJoinWarps][32][V + 1];
    const int64_t c = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int total = *a.total;
    int lo[2], hi[2], key[2];
    pieces_of(a, c, total, lo, hi, key);
    // a segment that begins exactly at a stretch, or inside it
    if (key[1] < 0)
        return;
    const int2 seg = a.segment[key[1]];
    const int64_t pieces = (seg.y - 1) / kLong - c + 1;
    const int64_t each = (pieces + kJoinWarps - 1) / kJoinWarps;
    const int64_t from = min(warp * each, pieces), to = min(from + each, pieces);
    const int32_t g = blockIdx.y * 32 + lane;
    float sum[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
        sum[k] = 0.0f;
    if (g < a.groups) {
        for (int64_t q = from; q < to; q += kInFlight) {
            float x[kInFlight][V];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                // slot 1 of the stretch it begins in, slot 0 of the later ones
                const int64_t row = 2 * (c + q + u) + (q + u == 0 ? 1 : 0);
                if (q + u < to && index_ok(a.status, row < a.partial_rows))
                    load_row<float, V>(a.partial, row * a.partial_stride + g * V, x[u]);
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                if (q + u < to)
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        sum[k] = __fadd_rn(sum[k], x[u][k]);
        }
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
        share[warp][lane][k] = sum[k];
    __syncthreads();
    if (warp != 0 || g >= a.groups)
        return;
    for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
        for (int k = 0; k < V; ++k)
            sum[k] = __fadd_rn(sum[k], share[w][lane][k]);
    finish_row<GT, V>(a, key[1], g * V, sum);
}

template <typename DT, typename GT, int V>
cudaError_t launch_v(const RowSumArgs& a, bool drop, cudaStream_t s)
{
    RowGrid g = row_grid(a.rows, a.groups, kSumThreads);
    const int64_t stretches = a.n > kLong ? grad_stretches(a.n) : 0;  // no segment is long otherwise
    const unsigned piece_blocks = static_cast<unsigned>((stretches + g.block.y - 1) / g.block.y);
    g.grid.x += piece_blocks;
    if (drop)
        k_row_sums<DT, GT, V, true><<<g.grid, g.block, 0, s>>>(a, piece_blocks);
    else
        k_row_sums<DT, GT, V, false><<<g.grid, g.block, 0, s>>>(a, piece_blocks);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && stretches > 0) {
        const dim3 grid(static_cast<unsigned>(stretches), static_cast<unsigned>((a.groups + 31) / 32));
        k_join_pieces<GT, V><<<grid, kJoinWarps * 32, 0, s>>>(a);
        e = cudaGetLastError();
    }
    return e;
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
