// embed_sort.cu -- the stable sort of a batch's places by key (token or
// position), the first launch of an embedding gradient.
//
// By counting, without communication between blocks.  Block b of C owns
// the keys with key % C == b (interleaved, so that the frequent low ids of a
// vocabulary spread over the blocks) and reads all keys itself: it counts those
// of lower blocks, which gives the base of its part of `order`, and its own for
// each warp and key.  Each warp takes a contiguous slice of the places, so a
// scan over warps keeps places ascending within a key.  What a warp finds of
// its block's keys it keeps in a list in shared memory, and only that list is
// placed, ranked among equal keys by ballots (a ballot a key bit; the match
// instruction took about 150 cycles).  A sort moves few bytes: it is bound by
// latency in small batches, and by each block's reads of all keys from L2 in
// large ones (8 bytes a place; 64 to 256 blocks measured, 128 the best).  A
// radix sort of two passes in one thread-block cluster read each key once, but
// its barriers and passes took 23 us for 1024 places and 38 us for 65536.
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
__device__ __forceinline__ void place_keys(const SortTask& t, int* next, const int2* range, bool has, int owned_key, int key_bits,
                                           int32_t key, int32_t place, int lane, int* status)
{
    unsigned same = __ballot_sync(kAll, has);
    for (int b = 0; b < key_bits; ++b) {
        const bool bit = owned_key >> b & 1;
        const unsigned ones = __ballot_sync(kAll, bit);
        same &= bit ? ones : ~ones;
    }
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

template <int KIND, typename IT, int BLOCK>
__device__ void sort_task(const SortTask& t, int mine, int* memory, int* all_status)
{
    constexpr int kWarps = BLOCK / 32;
    __shared__ int part[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int shift = t.log_blocks, mask = (1 << shift) - 1;
    const int owned = mine < t.keys ? ((t.keys - 1 - mine) >> shift) + 1 : 0;
    const int width = owned_width(t.keys, shift);  // of the rows of count
    int* count = memory;                         // kWarps x width: keys of each (warp, key), then where the next goes
    uint32_t* list = reinterpret_cast<uint32_t*>(memory + kWarps * width) + warp * kList;  // place in slice | owned key << 16
    int2* range = reinterpret_cast<int2*>(memory + kWarps * (width + kList));  // the block's segments
    int* status = mine == 0 ? all_status : nullptr;
    for (int k = tid; k < kWarps * width / 4; k += BLOCK)
        reinterpret_cast<int4*>(count)[k] = make_int4(0, 0, 0, 0);
    count += warp * width;
    // what came before in the stream is done; then the row sums may start beside this, and rely on that
    wait_for_launch_before();
    let_next_launch_start();

    const int64_t n = t.at.n;
    const int64_t slice = (n + BLOCK - 1) / BLOCK * 32;
    const int64_t lo = warp * slice, hi = min(lo + slice, n);
    int found = 0, below = 0;
    __syncthreads();  // count is zero
    RawKeys<KIND, IT> raw;
    auto count_keys = [&](int64_t i0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int32_t key = raw.key(t.at, u, status);
            const int b = key & mask;
            below += key >= 0 && b < mine ? 1 : 0;
            const bool take = key >= 0 && b == mine;
            const unsigned takers = __ballot_sync(kAll, take);
            if (takers == 0)
                continue;
            if (take) {
                const int k = key >> shift, at = found + __popc(takers & ((1u << lane) - 1));
                atomicAdd(&count[k], 1);
                if (at < kList)
                    list[at] = static_cast<uint32_t>(i0 - lo + u * 32 + lane) | static_cast<uint32_t>(k) << 16;
            }
            found += __popc(takers);
        }
    };
    int64_t i0 = lo;
    for (; i0 + kBatch * 32 <= hi; i0 += kBatch * 32) {
        raw.template load<true>(t.at, i0, hi, lane);
        count_keys(i0);
    }
    if (i0 < hi) {
        raw.template load<false>(t.at, i0, hi, lane);
        count_keys(i0);
    }
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
    if (found <= kList && slice <= 65536) {
        for (int q = 0; q < found; q += 32) {
            const bool has = q + lane < found;
            const uint32_t item = has ? list[q + lane] : 0;
            const int k = static_cast<int>(item >> 16);
            place_keys(t, count, range, has, k, key_bits, (k << shift) | mine, static_cast<int32_t>(lo + (item & 0xffff)), lane, all_status);
        }
    } else {
        for (int64_t i1 = lo; i1 < hi; i1 += kBatch * 32) {
            raw.template load<false>(t.at, i1, hi, lane);
            for (int u = 0; u < kBatch; ++u) {
                const int32_t key = raw.key(t.at, u, nullptr);
                const bool has = key >= 0 && (key & mask) == mine;
                if (__ballot_sync(kAll, has))
                    place_keys(t, count, range, has, has ? key >> shift : 0, key_bits, key, static_cast<int32_t>(i1 + u * 32 + lane),
                               lane, all_status);
            }
        }
    }
}

template <int BLOCK>
__global__ void __launch_bounds__(BLOCK) k_sort(const __grid_constant__ SortArgs a)
{
    extern __shared__ __align__(16) int memory[];
    int block = blockIdx.x;
    for (int k = 0; k < a.tasks; ++k) {
        const int sorters = 1 << a.task[k].log_blocks;
        if (block < sorters) {
            const SortTask& t = a.task[k];
            if (t.kind == kKeyToken)
                t.at.wide ? sort_task<kKeyToken, int64_t, BLOCK>(t, block, memory, a.status)
                          : sort_task<kKeyToken, int32_t, BLOCK>(t, block, memory, a.status);
            else
                t.at.wide ? sort_task<kKeyPosition, int64_t, BLOCK>(t, block, memory, a.status)
                          : sort_task<kKeyPosition, int32_t, BLOCK>(t, block, memory, a.status);
            break;
        }
        block -= sorters;
    }
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * BLOCK + threadIdx.x; k < a.arrived_count;
         k += static_cast<int64_t>(gridDim.x) * BLOCK)
        a.arrived[0][k] = a.arrived[1][k] = 0;
}

template <int BLOCK>
cudaError_t launch_block(const SortArgs& a, int blocks, int width, cudaStream_t s)
{
    const size_t shared = sizeof(int) * (BLOCK / 32) * (width + kList) + sizeof(int2) * width;
    static_assert(sizeof(int) * (BLOCK / 32) * (kMaxOwned + kList) + sizeof(int2) * kMaxOwned <= 220 * 1024, "a block fits an SM");
    if (shared > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k_sort<BLOCK>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(shared));
        if (e != cudaSuccess)
            return e;
    }
    return launch_programmatic(k_sort<BLOCK>, static_cast<unsigned>(blocks), BLOCK, shared, s, a);
}

}  // namespace

cudaError_t launch_sort(SortArgs a, cudaStream_t s)
{
    int width = 1, sorters = 0;
    for (int k = 0; k < a.tasks; ++k) {
        SortTask& t = a.task[k];
        // one wave of blocks, each with a key at least
        while (t.log_blocks < (a.tasks > 1 ? 6 : 7) && t.keys >> (t.log_blocks + 1) > 0)
            ++t.log_blocks;
        while ((static_cast<int64_t>(kMaxOwned) << t.log_blocks) < t.keys)
            ++t.log_blocks;
        const int w = owned_width(t.keys, t.log_blocks);
        width = width < w ? w : width;
        sorters += 1 << t.log_blocks;
    }
    return a.task[0].at.n <= kSmallBatch ? launch_block<kSmallBlock>(a, sorters, width, s)
                                         : launch_block<kBlock>(a, sorters, width, s);
}

}  // namespace lc
