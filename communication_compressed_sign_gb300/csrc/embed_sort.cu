// embed_sort.cu -- stable sort of a batch's places by key (token or position).
//
// Keys are spread over R buckets by their low bits (interleaved, so that the
// frequent low ids of a vocabulary do not meet in one), and a block sorts one
// bucket by counting.  No block waits for another.  Two ways into the buckets:
//
//   direct   every bucket's block reads all keys: it takes its own and counts
//            those of lower buckets, which gives its base.  One launch, R * n
//            key reads from L2.
//   tiled    count (tile x bucket), scatter into buckets, then a block per
//            bucket: three launches, 4 n key reads.
//
// Direct up to kDirectPlaces places.  A sort is bound by latency (dependent
// loads, launches), not by the few bytes it moves.
//
// Stability: a warp takes a contiguous slice of its block's places in order,
// counts per (warp, key), and after the scan places its keys 32 at a time,
// ranked among equal keys of the 32 by a warp match.
#include "embed_device.cuh"

namespace lc {
namespace {

constexpr int kThreads1 = 256;
constexpr int kWarps = kThreads1 / 32;
constexpr int kMaxOwn = 1024;     // keys of one bucket
constexpr int kMaxBuckets = 1024;
constexpr int kBatch = 4;         // groups of 32 keys a warp loads at once
constexpr unsigned kAll = 0xffffffffu;

// Where a sort's keys come from: the places themselves, or a bucket's pairs.
enum Source { kTokens = kKeyToken, kPositions = kKeyPosition, kPairs = 2 };

template <int SRC>
__device__ __forceinline__ int32_t key_of(const SortArgs& a, int64_t i, int* status)
{
    const int32_t t = token_at(a.at, i, status);
    if (SRC == kTokens || t < 0)
        return t;
    return position_at(a.at, i, status);
}

__device__ __forceinline__ int warp_inclusive(int x, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kAll, x, o);
        x += lane >= o ? up : 0;
    }
    return x;
}

// Exclusive prefix of x over the block's threads; the block's total in `sum`.
__device__ __forceinline__ int block_exclusive(int x, int* part, int& sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int inc = warp_inclusive(x, lane);
    __syncthreads();  // part may still be read from an earlier use
    if (lane == 31)
        part[warp] = inc;
    __syncthreads();
    int before = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? part[w] : 0;
        sum += part[w];
    }
    return before + inc - x;
}

// The rank of this lane among lower lanes with the same digit, and whether it
// is the last of them; lanes outside `takers` take no part.
__device__ __forceinline__ int rank_of(unsigned takers, int digit, int lane, bool& last)
{
    const unsigned same = __match_any_sync(takers, digit);
    last = (same >> lane) == 1u;
    return __popc(same & ((1u << lane) - 1));
}

// Zeroes the arrival counters of the row sums, spread over the grid.
__device__ __forceinline__ void clear_arrived(const SortArgs& a)
{
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; k < a.arrived_count;
         k += static_cast<int64_t>(gridDim.x) * blockDim.x)
        a.arrived[k] = 0;
}

// --- tiled, first: keys of each (tile, bucket) ----------------------------------------

template <int SRC>
__global__ void __launch_bounds__(kThreads1) k_sort_count(const SortArgs a)
{
    __shared__ int hist[kMaxBuckets];
    const int buckets = 1 << a.log_buckets;
    for (int k = threadIdx.x; k < buckets; k += kThreads1)
        hist[k] = 0;
    clear_arrived(a);
    __syncthreads();
    const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.tile, hi = min(lo + a.tile, static_cast<int64_t>(a.at.n));
    for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += kBatch * kThreads1) {
        int32_t key[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            key[u] = i0 + u * kThreads1 < hi ? key_of<SRC>(a, i0 + u * kThreads1, a.status) : -1;
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (key[u] >= 0)
                atomicAdd(&hist[key[u] & (buckets - 1)], 1);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < buckets; k += kThreads1)
        a.tile_count[static_cast<int64_t>(blockIdx.x) * buckets + k] = hist[k];
}

// --- tiled, second: (key, place) pairs into buckets -------------------------------------

template <int SRC>
__global__ void __launch_bounds__(kThreads1) k_sort_scatter(const SortArgs a)
{
    __shared__ int cnt[kWarps][kMaxBuckets];
    __shared__ int part[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int buckets = 1 << a.log_buckets, tiles = gridDim.x, mine = blockIdx.x;
    for (int k = tid; k < buckets; k += kThreads1)
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            cnt[w][k] = 0;
    __syncthreads();

    const int64_t begin = static_cast<int64_t>(mine) * a.tile, end = min(begin + a.tile, static_cast<int64_t>(a.at.n));
    const int64_t slice = a.tile / kWarps;  // a multiple of 32
    const int64_t lo = begin + warp * slice, hi = min(lo + slice, end);
    for (int64_t i0 = lo + lane; i0 < hi; i0 += 32) {
        const int32_t key = key_of<SRC>(a, i0, nullptr);
        if (key >= 0)
            atomicAdd(&cnt[warp][key & (buckets - 1)], 1);
    }
    __syncthreads();

    // thread t: bases of buckets t, t + 256, ...: everything in lower buckets,
    // then the same bucket's keys in lower tiles, then in lower warps
    int carried = 0;
    for (int k0 = 0; k0 < buckets; k0 += kThreads1) {
        const int k = k0 + tid;
        int total = 0, lower = 0;
#pragma unroll 8
        for (int t = 0; t < tiles; ++t) {
            const int c = a.tile_count[static_cast<int64_t>(t) * buckets + k];
            total += c;
            lower += t < mine ? c : 0;
        }
        int sum;
        const int start = carried + block_exclusive(total, part, sum);
        carried += sum;
        if (mine == 0)
            a.bucket_start[k] = start;
        int at = start + lower;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int c = cnt[w][k];
            cnt[w][k] = at;
            at += c;
        }
    }
    if (mine == 0 && tid == 0) {
        a.bucket_start[buckets] = carried;
        *a.total = carried;
    }
    __syncthreads();

    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const int64_t i = i0 + lane;
        const int32_t key = i < hi ? key_of<SRC>(a, i, nullptr) : -1;
        const unsigned takers = __ballot_sync(kAll, key >= 0);
        if (key >= 0) {
            const int b = key & (buckets - 1);
            bool last;
            const int at = cnt[warp][b] + rank_of(takers, b, lane, last);
            __syncwarp(takers);
            if (last)
                cnt[warp][b] = at + 1;
            if (index_ok(a.status, at >= 0 && at < a.capacity))
                a.pairs[at] = make_int2(key, static_cast<int32_t>(i));
        }
        __syncwarp();
    }
}

// --- a bucket's keys, sorted -------------------------------------------------------------

template <int SRC>
__global__ void __launch_bounds__(kThreads1) k_sort_bucket(const SortArgs a)
{
    __shared__ int cnt[kWarps][kMaxOwn];
    __shared__ int part[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int shift = a.log_buckets, mask = (1 << shift) - 1;
    const int mine = blockIdx.x;
    const int own = mine < a.keys ? ((a.keys - 1 - mine) >> shift) + 1 : 0;  // keys of this bucket
    for (int k = tid; k < own; k += kThreads1)
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            cnt[w][k] = 0;
    if (SRC != kPairs)
        clear_arrived(a);
    __syncthreads();

    int64_t begin = 0, end = a.at.n;
    if (SRC == kPairs) {
        begin = a.bucket_start[mine];
        end = a.bucket_start[mine + 1];
    }
    const int64_t slice = (end - begin + kThreads1 - 1) / kThreads1 * 32;
    const int64_t lo = begin + warp * slice, hi = min(lo + slice, end);
    int* status = SRC != kPairs && mine == 0 ? a.status : nullptr;
    int below = 0;
    for (int64_t i0 = lo + lane; i0 < hi; i0 += kBatch * 32) {
        int32_t key[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            key[u] = -1;
            if (i0 + u * 32 < hi)
                key[u] = SRC == kPairs ? a.pairs[i0 + u * 32].x : key_of<SRC>(a, i0 + u * 32, status);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (key[u] < 0)
                continue;
            if (SRC == kPairs || (key[u] & mask) == mine)
                atomicAdd(&cnt[warp][key[u] >> shift], 1);
            else
                below += (key[u] & mask) < mine ? 1 : 0;
        }
    }
    int base = static_cast<int>(begin);
    if (SRC != kPairs)
        block_exclusive(below, part, base);
    __syncthreads();

    for (int k0 = 0; k0 < own; k0 += kThreads1) {
        const int k = k0 + tid;
        int count[kWarps], total = 0, sum;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            count[w] = k < own ? cnt[w][k] : 0;
            total += count[w];
        }
        int at = base + block_exclusive(total, part, sum);
        base += sum;
        if (k < own) {
            const int32_t key = (k << shift) | mine;
            if (index_ok(a.status, key < a.keys && at >= 0 && at + total <= a.capacity))
                a.segment[key] = make_int2(at, at + total);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                cnt[w][k] = at;
                at += count[w];
            }
        }
    }
    if (SRC != kPairs && mine == mask && tid == 0)
        *a.total = base;
    __syncthreads();

    for (int64_t i0 = lo; i0 < hi; i0 += kBatch * 32) {
        int32_t key[kBatch], place[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32 + lane;
            key[u] = -1;
            place[u] = static_cast<int32_t>(i);
            if (i < hi) {
                if (SRC == kPairs) {
                    const int2 p = a.pairs[i];
                    key[u] = p.x;
                    place[u] = p.y;
                } else {
                    key[u] = key_of<SRC>(a, i, nullptr);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const bool take = key[u] >= 0 && (key[u] & mask) == mine;
            const unsigned takers = __ballot_sync(kAll, take);
            if (take) {
                const int k = key[u] >> shift;
                bool last;
                const int at = cnt[warp][k] + rank_of(takers, k, lane, last);
                __syncwarp(takers);
                if (last)
                    cnt[warp][k] = at + 1;
                if (index_ok(a.status, at >= 0 && at < a.capacity)) {
                    a.order[at] = place[u];
                    a.sorted_key[at] = key[u];
                }
            }
            __syncwarp();
        }
    }
}

template <int SRC>
cudaError_t launch_from(const SortArgs& a, cudaStream_t s)
{
    const int buckets = 1 << a.log_buckets;
    if (a.at.n <= kDirectPlaces) {
        k_sort_bucket<SRC><<<buckets, kThreads1, 0, s>>>(a);
        return cudaGetLastError();
    }
    const unsigned tiles = static_cast<unsigned>((a.at.n + a.tile - 1) / a.tile);
    k_sort_count<SRC><<<tiles, kThreads1, 0, s>>>(a);
    k_sort_scatter<SRC><<<tiles, kThreads1, 0, s>>>(a);
    k_sort_bucket<kPairs><<<buckets, kThreads1, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sort(SortArgs a, KeyKind kind, cudaStream_t s)
{
    a.log_buckets = sort_log_buckets(a.keys);
    a.tile = sort_tile(a.at.n);
    return kind == kKeyToken ? launch_from<kTokens>(a, s) : launch_from<kPositions>(a, s);
}

}  // namespace lc
