// embed_sort.cu -- the stable sort of a batch's places by key (token or
// position), the first launch of an embedding gradient.
//
// By counting.  Block b of C owns the keys with key % C == b (interleaved, so
// that the frequent low ids of a vocabulary spread over the blocks).  It counts
// the keys of lower blocks, which gives the base of its part of `order`, and its
// own for each warp and key.  Each warp takes a contiguous slice of the places,
// so a scan over warps keeps places ascending within a key.  What a warp finds
// of its block's keys it keeps in a list in shared memory, and only that list is
// placed, ranked among equal keys by ballots (a ballot a key bit; the match
// instruction took about 150 cycles).
//
// Small batches are bound by latency, and every block reads all keys.  In large
// ones that is bound by L2 (67 MB of reads for 65536 places), so there a cluster
// of blocks reads each key once, a part a block, lists those of its own blocks
// in shared memory, and each block takes its own from the cluster's lists.  (64
// to 256 blocks measured, 128 the best; clusters of 2, 4 and 8: two sorts of
// 65536 places and the gradient of 768 columns 94, 87 and 91 us against 98
// without.  A radix sort of two passes in one cluster read each key once too,
// but its barriers and passes took 38 us for 65536 places.)
#include <cooperative_groups.h>

#include <type_traits>

#include "embed_device.cuh"

namespace lc {
namespace {

// Threads of a block: 1024, or 512 for small batches, whose scan over warps and
// barriers are shorter (launches back to back, 512 and 1024 threads: 1024 places
// 3.6 and 4.6 us, 8192 4.5 and 4.9, 16384 6.1 and 6.0, 65536 15.4 and 12.5).
constexpr int kBlock = 1024, kSmallBlock = 512;
constexpr int64_t kSmallBatch = 8192;
constexpr int kMaxOwned = 1024;    // keys of a block
constexpr int kBatch = 8;          // groups of 32 keys a warp loads at once
constexpr int kList = 256;         // a warp's list; a slice with more is read again
constexpr int kCluster = 4;        // blocks that share their reading
constexpr int kShared = 256;       // a warp's list of its cluster's keys
// Places, over the tables, above which blocks read in clusters, and up to which
// (whole gradients of 768 columns, microseconds without and with clusters: one
// table 9216 places 23.5 and 24.0, 16384 27.8 and 28.4, 32768 40.5 and 39.3, 65536
// 57.7 and 54.1, 131072 92 and 84, 262144 204 and 212, where slices hold so much
// of a frequent token that they are read again; two tables 9216 34.2 and 33.3,
// 65536 81 and 75).
constexpr int64_t kClusterAbove = 16384, kClusterUpTo = 131072;

// The key of a place from its token (and position, where that is the key), or
// -1.  IT: the type of ids and positions.
template <int KIND, typename IT>
__device__ __forceinline__ int32_t key_of(const Places& at, IT token, IT position, int* status)
{
    using U = typename std::make_unsigned<IT>::type;
    const bool there = static_cast<U>(token) < static_cast<U>(at.vocab);
    const IT key = KIND == kKeyToken ? token : position;
    const bool good = static_cast<U>(key) < static_cast<U>(KIND == kKeyToken ? at.vocab : at.npos);
    if ((!there && token >= 0) || (there && !good))
        flag(status, kStatusIndex);
    return there && good ? static_cast<int32_t>(key) : -1;
}

// Tokens (and positions) of places i0 + 32 u + lane below hi: the loads before
// any use, so that they are in flight together.
template <int KIND, typename IT>
struct RawKeys {
    IT token[kBatch], position[KIND == kKeyPosition ? kBatch : 1];
    template <bool WHOLE>
    __device__ __forceinline__ void load(const Places& at, int64_t i0, int64_t hi, int lane)
    {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int64_t i = i0 + u * 32 + lane;
            token[u] = -1;
            if (WHOLE || i < hi) {
                token[u] = static_cast<const IT*>(at.tokens)[i];
                if (KIND == kKeyPosition)
                    position[KIND == kKeyPosition ? u : 0] =
                        at.positions ? static_cast<const IT*>(at.positions)[i]
                                     : static_cast<IT>(at.first + static_cast<uint32_t>(i) % static_cast<uint32_t>(at.seq_len));
            }
        }
    }
    __device__ __forceinline__ int32_t key(const Places& at, int u, int* status) const
    {
        return key_of<KIND, IT>(at, token[u], position[KIND == kKeyPosition ? u : 0], status);
    }
};

// Places one key of each lane that has one: the lane's rank among equal keys
// of the warp, after those its warp placed before.
__device__ __forceinline__ void place_keys(const SortTask& t, int* next, const int2* range, int owned, bool has, int owned_key, int key_bits,
                                           int32_t key, int32_t place, int lane, int* status)
{
    unsigned same = __ballot_sync(kAll, has);
    for (int b = 0; b < key_bits; ++b) {
        const bool bit = owned_key >> b & 1;
        const unsigned ones = __ballot_sync(kAll, bit);
        same &= bit ? ones : ~ones;
    }
    has = index_ok(status, !has || owned_key < owned) && has;
    int at = 0;
    if (has)
        at = next[owned_key] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (has) {
        if ((same >> lane) == 1u)  // the last lane with this key
            next[owned_key] = at + 1;
        if (index_ok(status, at >= 0 && at < t.capacity))
            t.order[at] = make_int4(place, key, range[owned_key].x, range[owned_key].y);
    }
    __syncwarp();
}

// Keys a block owns at most, rounded to 16 bytes of counts.
__host__ __device__ constexpr int owned_width(int keys, int shift)
{
    return (((keys + (1 << shift) - 1) >> shift) + 3) / 4 * 4;
}

template <int KIND, typename IT, int BLOCK, bool CLUSTERED>
__device__ void sort_task(const SortTask& t, int mine, int* memory, int* all_status, uint32_t* begun, uint32_t call)
{
    namespace cg = cooperative_groups;
    constexpr int kWarps = BLOCK / 32;
    __shared__ int part[kWarps];
    __shared__ int2 reads[CLUSTERED ? kWarps : 1];  // of what a warp read: the cluster's keys, and those below the cluster's
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int shift = t.log_blocks, mask = (1 << shift) - 1;
    const int owned = mine < t.keys ? ((t.keys - 1 - mine) >> shift) + 1 : 0;
    const int width = owned_width(t.keys, shift);  // of the rows of count
    int* count = memory;                           // kWarps x width: keys of each (warp, key), then where the next goes
    uint32_t* list = reinterpret_cast<uint32_t*>(memory + kWarps * width) + warp * kList;  // place in slice | owned key << 16
    int2* range = reinterpret_cast<int2*>(memory + kWarps * (width + kList));  // the block's segments
    // CLUSTERED, kWarps x kShared: place in what the warp reads | (owned key, block of the cluster) << 16
    uint32_t* lists = reinterpret_cast<uint32_t*>(range + width);
    int* status = mine == 0 ? all_status : nullptr;
    for (int k = tid; k < kWarps * width / 4; k += BLOCK)
        reinterpret_cast<int4*>(count)[k] = make_int4(0, 0, 0, 0);
    count += warp * width;
    // what came before in the stream is done; then the row sums may start beside this,
    // and running positions may read it as soon as the one thread has told so
    wait_for_launch_before();
    if (begun && tid == 0)
        tell_begun(begun, call);
    let_next_launch_start();

    const int64_t n = t.at.n;
    const int64_t slice = (n + BLOCK - 1) / BLOCK * 32;
    const int64_t lo = warp * slice, hi = min(lo + slice, n);
    int found = 0, below = 0;
    // counts and lists the block's among 32 keys (-1: none)
    auto count_keys = [&](int32_t key, int place_in_slice) {
        const int b = key & mask;
        below += key >= 0 && b < mine ? 1 : 0;
        const bool take = key >= 0 && b == mine;
        const unsigned takers = __ballot_sync(kAll, take);
        if (takers == 0)
            return;
        if (take) {
            const int k = key >> shift, at = found + __popc(takers & ((1u << lane) - 1));
            const bool good = index_ok(all_status, k < owned && place_in_slice >= 0 && place_in_slice < slice);
            if (good)
                atomicAdd(&count[k], 1);
            if (good && at < kList)
                list[at] = static_cast<uint32_t>(place_in_slice) | static_cast<uint32_t>(k) << 16;
        }
        found += __popc(takers);
    };
    RawKeys<KIND, IT> raw;
    bool all = true;  // the block reads all places
    if constexpr (CLUSTERED) {
        // the block reads kWarps / kCluster slices for the cluster, kCluster of its warps each of them
        const cg::cluster_group cluster = cg::this_cluster();
        const int rank = mine & (kCluster - 1), first = mine - rank;
        const int64_t fine = (slice / 32 + kCluster - 1) / kCluster * 32;
        const int64_t lo0 = (rank * (kWarps / kCluster) + warp / kCluster) * slice;
        const int64_t flo = min(lo0 + warp % kCluster * fine, n), fhi = min(min(flo + fine, lo0 + slice), n);
        int kept = 0, lower = 0;
        for (int64_t i0 = flo; i0 < fhi; i0 += kBatch * 32) {
            raw.template load<false>(t.at, i0, fhi, lane);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int32_t key = raw.key(t.at, u, first == 0 ? all_status : nullptr);
                const int b = (key & mask) - first;
                lower += key >= 0 && b < 0 ? 1 : 0;
                const bool take = key >= 0 && b >= 0 && b < kCluster;
                const unsigned takers = __ballot_sync(kAll, take);
                const int at = kept + __popc(takers & ((1u << lane) - 1));
                if (take && at < kShared)
                    lists[warp * kShared + at] = static_cast<uint32_t>(i0 - flo + u * 32 + lane) |
                                                 static_cast<uint32_t>((key >> shift) * kCluster + b) << 16;
                kept += __popc(takers);
            }
        }
        lower = __reduce_add_sync(kAll, lower);
        if (lane == 0)
            reads[warp] = make_int2(kept, lower);
        cluster.sync();
        const int2 theirs = warp < kCluster ? *cluster.map_shared_rank(&reads[lane], warp) : make_int2(0, 0);
        // the lists of the warp's slice
        const int owner = warp / (kWarps / kCluster), part0 = warp % (kWarps / kCluster) * kCluster;
        const int length = lane < kCluster ? cluster.map_shared_rank(&reads[part0], owner)[lane].x : 0;
        all = __syncthreads_or(theirs.x > kShared);  // a list did not suffice
        if (!all) {
            below = theirs.y;
            int before = length;  // items in the lists before lane l's
#pragma unroll
            for (int o = 1; o < kCluster; o <<= 1) {
                const int up = __shfl_up_sync(kAll, before, o);
                before += lane >= o ? up : 0;
            }
            const int items = __shfl_sync(kAll, before, kCluster - 1);
            before -= length;
            const uint32_t* their_lists = cluster.map_shared_rank(lists + part0 * kShared, owner);
            for (int q = 0; q < items; q += 32) {
                int l = 0, start = 0;  // the item's list and where that starts
#pragma unroll
                for (int j = 1; j < kCluster; ++j) {
                    const int at = __shfl_sync(kAll, before, j);
                    if (q + lane >= at) {
                        l = j;
                        start = at;
                    }
                }
                int32_t key = -1;
                int place_in_slice = 0;
                if (q + lane < items) {
                    const int in_list = q + lane - start;
                    const uint32_t item = index_ok(all_status, in_list >= 0 && in_list < kShared) ? their_lists[l * kShared + in_list] : 0,
                                   k = item >> 16;
                    key = static_cast<int32_t>(k / kCluster) << shift | (first + static_cast<int>(k % kCluster));
                    place_in_slice = l * static_cast<int>(fine) + static_cast<int>(item & 0xffff);
                }
                count_keys(key, place_in_slice);
            }
        }
    } else {
        __syncthreads();  // count is zero
    }
    if (all) {
        auto count_batch = [&](int64_t i0) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                count_keys(raw.key(t.at, u, CLUSTERED ? nullptr : status), static_cast<int>(i0 - lo) + u * 32 + lane);
        };
        int64_t i0 = lo;
        for (; i0 + kBatch * 32 <= hi; i0 += kBatch * 32) {
            raw.template load<true>(t.at, i0, hi, lane);
            count_batch(i0);
        }
        if (i0 < hi) {
            raw.template load<false>(t.at, i0, hi, lane);
            count_batch(i0);
        }
    }
    if constexpr (CLUSTERED)
        cg::this_cluster().barrier_arrive();  // nothing of another block is read from here on
    below = __reduce_add_sync(kAll, below);
    if (lane == 0)
        part[warp] = below;
    __syncthreads();
    int base = __reduce_add_sync(kAll, lane < kWarps ? part[lane] : 0);

    // thread: one of the block's keys, over the warps
    for (int k0 = 0; k0 < owned; k0 += BLOCK) {
        const int k = k0 + tid;
        int total = 0;
        if (k < owned) {
#pragma unroll 8
            for (int w = 0; w < kWarps; ++w)
                total += memory[w * width + k];
        }
        int inc = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(kAll, inc, o);
            inc += lane >= o ? up : 0;
        }
        __syncthreads();  // part is read above and in the round before
        if (lane == 31)
            part[warp] = inc;
        __syncthreads();
        const int others = lane < kWarps ? part[lane] : 0;
        const int start = base + __reduce_add_sync(kAll, lane < warp ? others : 0) + inc - total;
        base += __reduce_add_sync(kAll, others);
        if (k < owned) {
            const int32_t key = (k << shift) | mine;
            if (index_ok(all_status, key < t.keys && start >= 0 && start + total <= t.capacity))
                t.segment[key] = make_int2(start, start + total);
            range[k] = make_int2(start, start + total);
            int at = start;
            for (int w0 = 0; w0 < kWarps; w0 += 8) {  // 8 loads at a time: a store between two keeps them apart
                int each[8];
#pragma unroll
                for (int w = 0; w < 8; ++w)
                    each[w] = memory[(w0 + w) * width + k];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    memory[(w0 + w) * width + k] = at;
                    at += each[w];
                }
            }
        }
    }
    if (mine == mask && tid == 0)
        *t.total = base;
    __syncthreads();

    const int key_bits = 32 - __clz(width - 1);
    auto place_list = [&](int items, int64_t first_place) {
        for (int q = 0; q < items; q += 32) {
            const bool has = q + lane < items;
            const uint32_t item = has ? list[q + lane] : 0;
            const int k = static_cast<int>(item >> 16);
            place_keys(t, count, range, owned, has, k, key_bits, (k << shift) | mine, static_cast<int32_t>(first_place + (item & 0xffff)),
                       lane, all_status);
        }
    };
    if (found <= kList && slice <= 65536) {
        place_list(found, lo);
    } else {  // read again, a list at a time
        int items = 0;
        int64_t first_place = lo;
        for (int64_t i1 = lo; i1 < hi;) {
            if (items > kList - 32 || i1 + kBatch * 32 - first_place > 65536) {
                __syncwarp();
                place_list(items, first_place);
                items = 0;
                first_place = i1;
            }
            raw.template load<false>(t.at, i1, hi, lane);
            int groups = 0;  // until the list may be full
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (items > kList - 32)
                    continue;
                const int32_t key = raw.key(t.at, u, nullptr);
                const bool has = key >= 0 && (key & mask) == mine;
                const unsigned takers = __ballot_sync(kAll, has);
                if (has && index_ok(all_status, items + __popc(takers) <= kList))
                    list[items + __popc(takers & ((1u << lane) - 1))] =
                        static_cast<uint32_t>(i1 - first_place + u * 32 + lane) | static_cast<uint32_t>(key >> shift) << 16;
                items += __popc(takers);
                groups = u + 1;
            }
            i1 += groups * 32;
        }
        __syncwarp();
        place_list(items, first_place);
    }
    if constexpr (CLUSTERED)
        cg::cluster_group::barrier_wait(cg::cluster_group::arrival_token{});
}

template <int BLOCK, bool CLUSTERED>
__global__ void __launch_bounds__(BLOCK) k_sort(const __grid_constant__ SortArgs a)
{
    extern __shared__ __align__(16) int memory[];
    int block = blockIdx.x;
    uint32_t* const begun = block == 0 ? a.begun : nullptr;  // one block tells
    for (int k = 0; k < a.tasks; ++k) {
        const int sorters = 1 << a.task[k].log_blocks;
        if (block < sorters) {
            const SortTask& t = a.task[k];
            if (t.kind == kKeyToken)
                t.at.wide ? sort_task<kKeyToken, int64_t, BLOCK, CLUSTERED>(t, block, memory, a.status, begun, a.call)
                          : sort_task<kKeyToken, int32_t, BLOCK, CLUSTERED>(t, block, memory, a.status, begun, a.call);
            else
                t.at.wide ? sort_task<kKeyPosition, int64_t, BLOCK, CLUSTERED>(t, block, memory, a.status, begun, a.call)
                          : sort_task<kKeyPosition, int32_t, BLOCK, CLUSTERED>(t, block, memory, a.status, begun, a.call);
            break;
        }
        block -= sorters;
    }
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * BLOCK + threadIdx.x; k < a.arrived_count;
         k += static_cast<int64_t>(gridDim.x) * BLOCK)
        a.arrived[0][k] = a.arrived[1][k] = 0;
}

template <int BLOCK, bool CLUSTERED>
cudaError_t launch_block(const SortArgs& a, int blocks, int width, cudaStream_t s)
{
    constexpr int kWarps = BLOCK / 32;
    constexpr size_t kLists = sizeof(int) * kWarps * kList + (CLUSTERED ? sizeof(uint32_t) * kWarps * kShared : 0);
    const size_t shared = sizeof(int) * kWarps * width + kLists + sizeof(int2) * width;
    constexpr size_t kMost = sizeof(int) * kWarps * kMaxOwned + kLists + sizeof(int2) * kMaxOwned;
    static_assert(kMost <= 220 * 1024, "a block fits an SM");
    if (shared > 48 * 1024) {
        // the kernel's limit, the same for every call: calls of other threads launch by it too
        const cudaError_t e =
            cudaFuncSetAttribute(k_sort<BLOCK, CLUSTERED>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost));
        if (e != cudaSuccess)
            return e;
    }
    return launch_programmatic_clusters(k_sort<BLOCK, CLUSTERED>, static_cast<unsigned>(blocks), BLOCK, CLUSTERED ? kCluster : 1, shared, s, a);
}

}  // namespace

cudaError_t launch_sort(SortArgs a, cudaStream_t s)
{
    int width = 1, sorters = 0;
    bool clustered = static_cast<int64_t>(a.task[0].at.n) * a.tasks > kClusterAbove && a.task[0].at.n <= kClusterUpTo;
    for (int k = 0; k < a.tasks; ++k) {
        SortTask& t = a.task[k];
        // One wave of blocks, each with a key at least.  So a table of few rows is
        // sorted by few blocks, whose lists overflow and are read again (whole
        // gradients of 65536 places of 768 columns, microseconds: of 1 row 80.7, 2 rows
        // 75.0, 8 65.0, 37 60.8, 100 44.9, 1000 44.8).
        while (t.log_blocks < (a.tasks > 1 ? 6 : 7) && t.keys >> (t.log_blocks + 1) > 0)
            ++t.log_blocks;
        while ((static_cast<int64_t>(kMaxOwned) << t.log_blocks) < t.keys)
            ++t.log_blocks;
        const int w = owned_width(t.keys, t.log_blocks);
        width = width < w ? w : width;
        sorters += 1 << t.log_blocks;
        // evenly spread keys put places / 32 / blocks on a list: a quarter of it at most
        clustered = clustered && 1 << t.log_blocks >= kCluster && t.at.n <= (int64_t(kShared) * 8) << t.log_blocks;
    }
    if (clustered)
        return launch_block<kBlock, true>(a, sorters, width, s);
    return a.task[0].at.n <= kSmallBatch ? launch_block<kSmallBlock, false>(a, sorters, width, s)
                                         : launch_block<kBlock, false>(a, sorters, width, s);
}

}  // namespace lc
