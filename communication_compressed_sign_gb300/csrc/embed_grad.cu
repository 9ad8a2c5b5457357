// embed_grad.cu -- gradient of the embedding lookup from the sorted places:
//   grad[v,:] = base[v,:] + factor * sum over places i with key_i == v of keep * dout[i,:].
//
// Every row of the dense gradient is written once -- rows without a place as
// zeros (or base) -- so there is no clearing pass, and no float atomics: the
// order of every sum depends on the call's arguments (how the pieces below are
// cut: the places, the width, 16-byte moves or not), never on the schedule.
//
// The unit of work is one warp on a slab of columns.
//   walk   a stretch of `piece` entries of `order`: the warp adds the rows of
//          dout of the segments that begin there, several rows in flight
//          whatever the segments' lengths, and writes a row of grad at each
//          segment's end.  A segment of up to `piece` places belongs to the
//          stretch it begins in.  A longer one is cut at the stretches' bounds: a
//          block's warps take consecutive stretches and add their pieces in
//          shared memory, blocks leave an fp32 partial, and the last of a group of
//          blocks to arrive (an integer counter) adds the partials in order.  So
//          units are alike in size however skewed the tokens are.
//   fill   rows without a place.
// Large gradients without dropout are bound by memory (dout is read and grad
// written once), small ones by the walks' latency, and those with dropout by the
// integer instructions of the mask: about 86 a row and slab, of which drawing
// takes 40.  Running positions read dout, and draw the mask, a second time.
// Measured (bf16, 50257 rows): 16 x 1024 places of 1024 columns 32 us (137 MB),
// 64 x 1024 of 2048 with positions and dropout 164 us (750 MB).
#include <algorithm>
#include <type_traits>

#include "embed_device.cuh"

namespace lc {
namespace {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;
constexpr int kInFlight = 4;           // rows of dout a warp loads before it adds them
constexpr int kFillRows = 8;           // rows of grad a fill warp looks at
constexpr unsigned kLead = 152 * 4;    // blocks the SMs hold: how many of a kind go ahead of the mix
// A running position of more sequences than kWay is shared by up to eight warps
// of a block, while all of them fit the SMs at once: its places are added one
// after the other by a warp.  (Whole gradients of 768 columns, microseconds: 128
// sequences of 64 by one warp 38.4, shared above 8, 16, 32 and 64 sequences 26.1,
// 26.1, 24.7 and 25.2; 64 of 16 23.1, then 19.6, 18.0, 18.0 and 23.6.  128 of 1024,
// which fill the SMs, 121, and 124 if shared all the same.)
constexpr int64_t kWay = 32;
constexpr int kJoinLog = 4, kJoin = 1 << kJoinLog;  // partials of a group of the gathering tree
constexpr int kJoinBits = kJoinLog + 1;             // counter bits of a level: 12 levels, 2^30 places need 6

// Adds rows of dout to a running sum and writes it where the key changes.
template <typename DT, typename GT, bool VEC, bool DROP>
struct Walker {
    static constexpr int N = kLaneCols<VEC>;
    const RowSumArgs& a;
    const Slab<VEC> cols;
    SlabMask<VEC> mask;
    float sum[N];

    __device__ __forceinline__ Walker(const RowSumArgs& args, int slab, int lane, typename SlabMask<VEC>::Shared* shared)
        : a(args), cols(slab, lane, args.dim), mask(args.drop, slab, lane, args.dim, shared)
    {
        clear();
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < N; ++k)
            sum[k] = 0.0f;
    }
    __device__ __forceinline__ void add(const SlabGroup<DT, VEC>& x, int u, uint32_t i)
    {
        if constexpr (DROP && sizeof(DT) == 2) {
            mask.add(u, i, x, sum);
        } else if constexpr (VEC && sizeof(DT) == 2) {
            const uint32_t w[4] = {x.g.raw.x, x.g.raw.y, x.g.raw.z, x.g.raw.w};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                add_bf16(sum[k], k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xffff);
        } else if constexpr (sizeof(DT) == 2) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                add_bf16(sum[k], __bfloat16_as_ushort(x.x[k]));
        } else {
            float y[N];
            x.unpack(y);
            if constexpr (DROP) {
                mask.row(u, i, [&](int k, bool keep) {
                    if (keep)
                        sum[k] = __fadd_rn(sum[k], y[k]);
                });
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    sum[k] = __fadd_rn(sum[k], y[k]);
            }
        }
    }
    // grad[v] = base[v] + factor * sum
    __device__ __forceinline__ void finish(int64_t v)
    {
        if (!index_ok(a.status, v >= 0 && v < a.rows))
            return;
#pragma unroll
        for (int k = 0; k < N; ++k)
            sum[k] = __fmul_rn(a.factor, sum[k]);
        if (a.base.data) {
            SlabGroup<GT, VEC> b;
            b.load(cols, a.base.data, v * a.base.stride);
            float y[N];
            b.unpack(y);
#pragma unroll
            for (int k = 0; k < N; ++k)
                sum[k] = __fadd_rn(y[k], sum[k]);
        }
        store_slab<GT, VEC>(cols, a.grad.data, v * a.grad.stride, sum);
    }
    // Adds up the blocks' sums of a long segment [begin, end): a tree of groups of
    // kJoin, in which the last of a group to arrive adds the group's partials in
    // order and goes on as one block of the next level.  True where the whole
    // sum has come together.
    __device__ __forceinline__ bool gather(int begin, int end, int block, int slab, int lane)
    {
        const int first = begin / a.piece / kWarps;
        int node = block - first, nodes = (end - 1) / a.piece / kWarps - first + 1;
        const int64_t column = slab * 256 + lane * 8;  // partial rows are whole slabs
        // the r-th block's partial and counter: slot 1 of the block the segment begins in, slot 0 of the later ones
        auto slot = [&](int r) { return 2 * static_cast<int64_t>(first + r) + (r == 0 ? 1 : 0); };
        auto partial = [&](int r) { return a.partial + slot(r) * a.partial_stride + column; };
        // every slot used lies between this segment's first and last
        if (!index_ok(a.status, first >= 0 && node >= 0 && node < nodes && slot(nodes - 1) < a.partial_rows && slab < a.slabs &&
                                    column + 8 <= a.partial_stride))
            return false;
#pragma unroll 1
        for (int level = 0; nodes > 1; ++level) {
            const int group = node / kJoin, members = min(kJoin, nodes - group * kJoin), scale = kJoinLog * level;
            store_partial(partial(node << scale));
            __syncwarp();
            uint64_t before = 0;
            if (lane == 0)
                before = arrive(&a.arrived[slot(group << scale << kJoinLog) * a.slabs + slab], 1ull << (kJoinBits * level));
            __syncwarp();  // what lane 0's arrival acquired is the other lanes' too
            before = __shfl_sync(kAll, before, 0);
            if ((before >> (kJoinBits * level) & ((1u << kJoinBits) - 1)) != members - 1)
                return false;
            clear();
#pragma unroll 4
            for (int m = 0; m < members; ++m)
                add_partial(partial((group * kJoin + m) << scale));
            node = group;
            nodes = (nodes + kJoin - 1) / kJoin;
        }
        return true;
    }
    // Counts an arrival, by one lane between two barriers of its warp: what the
    // warp wrote before the first is visible to whom the counter tells of it
    // (release), and what it tells of is visible to the warp after the second
    // (acquire).  A shuffle would hand on the count, not the order of memory.
    static __device__ __forceinline__ uint64_t arrive(uint64_t* counter, uint64_t one)
    {
        uint64_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], %2;" : "=l"(before) : "l"(counter), "l"(one) : "memory");
        return before;
    }
    __device__ __forceinline__ void put(float4 (&to)[2][32], int lane) const
    {
        to[0][lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        to[1][lane] = make_float4(sum[4], sum[5], sum[6], N == 8 ? sum[N - 1] : 0.0f);
    }
    // A lane's sums lie together in a partial row, whichever columns they are.
    __device__ __forceinline__ void store_partial(float* p) const
    {
        reinterpret_cast<float4*>(p)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(sum[4], sum[5], sum[6], N == 8 ? sum[N - 1] : 0.0f);
    }
    __device__ __forceinline__ void add_partial(const float* p)
    {
        add_group(__ldcg(reinterpret_cast<const float4*>(p)), __ldcg(reinterpret_cast<const float4*>(p) + 1));
    }
    __device__ __forceinline__ void add_group(const float4& x, const float4& y)
    {
        const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < N; ++k)
            sum[k] = __fadd_rn(sum[k], z[k]);
    }
};

// Row v, columns [begin, end): zeros, or base.  (16 bytes or one element a lane
// and step: a tight loop, since a fill should be bound by its stores.)
template <typename GT, bool VEC>
__device__ __forceinline__ void fill_row(const RowSumArgs& a, int64_t v, int begin, int end, int lane)
{
    if (!index_ok(a.status, v >= 0 && v < a.rows && begin >= 0 && end <= a.dim))
        return;
    constexpr int kPer = VEC ? 16 / sizeof(GT) : 1;
    using Unit = typename std::conditional<VEC, uint4, GT>::type;
    Unit* dst = reinterpret_cast<Unit*>(static_cast<GT*>(a.grad.data) + v * a.grad.stride);
    const int last = end / kPer;
    if (a.base.data) {
        const Unit* src = reinterpret_cast<const Unit*>(static_cast<const GT*>(a.base.data) + v * a.base.stride);
#pragma unroll 4
        for (int k = begin / kPer + lane; k < last; k += 32)
            dst[k] = src[k];
    } else {
        const Unit zero{};
#pragma unroll 4
        for (int k = begin / kPer + lane; k < last; k += 32)
            dst[k] = zero;
    }
}

// Those of rows [row0, row0 + kFillRows) that have no place.
template <typename GT, bool VEC>
__device__ __forceinline__ void fill_rows(const RowSumArgs& a, int64_t row0, int lane)
{
    bool empty = false;
    if (lane < kFillRows && row0 + lane < a.rows) {
        const int2 seg = a.segment[row0 + lane];
        empty = seg.x == seg.y;
    }
    unsigned todo = __ballot_sync(kAll, empty);
    while (todo) {
        const int64_t v = row0 + __ffs(todo) - 1;
        todo &= todo - 1;
        fill_row<GT, VEC>(a, v, 0, a.dim, lane);
    }
}

// The position of the n-th (from 0) set bit of a word that has more than n.
__device__ __forceinline__ int nth_bit(unsigned word, int n)
{
    int at = 0;
#pragma unroll
    for (int half = 16; half > 0; half >>= 1) {
        const int low = __popc(word & ((1u << half) - 1));
        if (n >= low) {
            n -= low;
            word >>= half;
            at += half;
        }
    }
    return at;
}

// What the blocks of a launch do.  Running positions need no sort, so they lead
// while it may still run; walks start next, since they take longest; the rest
// are spread evenly: walks are bound by latency or, with dropout, by integer
// instructions, and fills by memory, so they run side by side.
struct Roles {
    unsigned lead;       // position blocks at the front
    uint64_t positions;  // share of position blocks among the others, in 2^-32
    uint64_t fill;       // share of fill blocks among walks and fills, likewise
    unsigned walk_lead;       // walk blocks in front of the mix of walks and fills
    unsigned position_walks;  // sorted positions: walks before fills
    int log_ways;             // running positions: warps of a row and slab
    int64_t way;              // and the places of a warp's sequences
    __host__ __device__ __forceinline__ unsigned positions_before(unsigned block) const
    {
        return block <= lead ? block : lead + static_cast<unsigned>(((block - lead) * positions) >> 32);
    }
    __host__ __device__ __forceinline__ unsigned fills_before(unsigned block) const
    {
        return block <= walk_lead ? 0 : static_cast<unsigned>(((block - walk_lead) * fill) >> 32);
    }
};

// What a block of walks shares: the masks' draws, and its warps' sums of long
// segments, of the one that goes on from before a warp's stretch and of the one
// that begins in it.
template <bool VEC, bool DROP>
struct WalkShared {
    typename SlabMask<VEC>::Shared mask[DROP ? kWarps : 1];
    float4 sums[kWarps][2][2][32];
    bool any[kWarps];  // running positions: whether a warp's part has a place
    __device__ __forceinline__ typename SlabMask<VEC>::Shared* of(int warp) { return &mask[DROP ? warp : 0]; }
};

// A block of stretches of the sorted places, one a warp, on one slab.
template <typename DT, typename GT, bool VEC, bool DROP>
__device__ __forceinline__ void walk(const RowSumArgs& a, unsigned index, int warp, int lane, WalkShared<VEC, DROP>& shared)
{
    const int block = static_cast<int>(index / static_cast<unsigned>(a.slabs));  // places and so stretches fit 31 bits
    const int slab = static_cast<int>(index - static_cast<unsigned>(block) * a.slabs);
    const int64_t begin64 = (static_cast<int64_t>(block) * kWarps + warp) * a.piece;
    const int begin = static_cast<int>(min(begin64, static_cast<int64_t>(a.n)));
    // the stretch's entries and what a short segment can reach beyond it, not waiting for how many are set
    const int mine = min(begin + lane, a.n);  // below 2^31
    const int4 entry = mine < a.n ? a.order[mine] : make_int4(0, 0, 0, 0);
    const int total = *a.total, end = min(begin + a.piece, total);
    bool work = begin < total;
    work = __all_sync(kAll, index_ok(a.status, mine >= total || (entry.x >= 0 && entry.x < a.n && entry.y >= 0 && entry.y < a.rows))) && work;
    const int last = max(end - 1 - begin, 0);
    const int begin0 = __shfl_sync(kAll, entry.z, 0), end0 = __shfl_sync(kAll, entry.w, 0);
    const int begin1 = __shfl_sync(kAll, entry.z, last), end1 = __shfl_sync(kAll, entry.w, last);
    const bool tail = work && begin0 < begin && end0 - begin0 > a.piece;   // a long segment goes on here
    const bool head = work && begin1 >= begin && end1 - begin1 > a.piece;  // a long segment begins here
    // short segments: one that began before belongs there, one that begins here is taken to its end
    const int from = begin0 < begin ? end0 : begin, to = head ? begin1 : (begin1 < begin ? begin : end1);
    const int32_t above = __shfl_up_sync(kAll, entry.y, 1);
    const unsigned begins = __ballot_sync(kAll, lane == 0 || entry.y != above);

    Walker<DT, GT, VEC, DROP> w(a, slab, lane, shared.of(warp));
#pragma unroll 1
    for (int part = 0; part < 3; ++part) {  // the long segment's end, short segments, a long segment's begin
        if (part == 0 ? !tail : part == 1 ? !work : !head)
            continue;
        const int lo = part == 0 ? begin : part == 1 ? from : begin1;
        const int hi = part == 0 ? min(end0, end) : part == 1 ? to : end;
        if (lo >= hi)
            continue;
        w.clear();
        const int here = hi - begin;
        int32_t current = __shfl_sync(kAll, entry.y, lo - begin);
#pragma unroll 1
        for (int q = lo - begin; q < here; q += kInFlight) {
            SlabGroup<DT, VEC> x[kInFlight];
            int32_t place[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {  // past the end the last row again: no branch between the loads
                place[u] = __shfl_sync(kAll, entry.x, min(q + u, here - 1));
                x[u].load(w.cols, a.dout.data, static_cast<uint32_t>(place[u]) * a.dout.stride);
            }
            if (DROP)
                w.mask.template draw<kInFlight>(here - q, [&](int u) { return place[u]; });
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                if (q + u >= here)
                    break;
                if ((begins >> (q + u) & 1u) && q + u > lo - begin) {
                    w.finish(current);
                    w.clear();
                    current = __shfl_sync(kAll, entry.y, q + u);
                }
                w.add(x[u], u, place[u]);
            }
        }
        if (part == 1)
            w.finish(current);
        else
            w.put(shared.sums[warp][part == 0 ? 0 : 1], lane);
    }
    if (!__syncthreads_or(tail || head))
        return;

    // a long segment's pieces in this block, added in order by the warp of the
    // first of them: the one it begins in, or the block's first
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
        if (part == 0 ? !tail || warp > 0 : !head)
            continue;
        const int seg_begin = part == 0 ? begin0 : begin1, seg_end = part == 0 ? end0 : end1;
        const int until = min(kWarps - 1, (seg_end - 1) / a.piece - block * kWarps);
        w.clear();
        w.add_group(shared.sums[warp][part][0][lane], shared.sums[warp][part][1][lane]);
        for (int other = warp + 1; other <= until; ++other)
            w.add_group(shared.sums[other][0][0][lane], shared.sums[other][0][1][lane]);
        if (w.gather(seg_begin, seg_end, block, slab, lane))
            w.finish(__shfl_sync(kAll, entry.y, part == 0 ? 0 : last));
    }
}

// Positions that run with the place, first + i % seq_len: row q's places are
// q - first, q - first + seq_len, ... and need no sort.  One row on one slab,
// `ways` warps of a block a part of the sequences each.
template <typename DT, typename GT, bool VEC, bool DROP>
__device__ __forceinline__ void running_row(const RowSumArgs& a, const Places& at, const Roles& roles, int64_t unit, int warp, int lane,
                                            WalkShared<VEC, DROP>& shared)
{
    const int part = warp & ((1 << roles.log_ways) - 1);
    unit >>= roles.log_ways;
    const int64_t row = quotient(unit, a.slabs);
    const int slab = static_cast<int>(unit - row * a.slabs);
    const int64_t place0 = row - at.first, from = place0 + part * roles.way, until = min(from + roles.way, static_cast<int64_t>(at.n));
    const bool in_batch = row < a.rows && place0 >= 0 && place0 < at.seq_len;
    bool any = false;
    Walker<DT, GT, VEC, DROP> w(a, slab, lane, shared.of(warp));
    for (int64_t p0 = from; in_batch && p0 < until; p0 += 32 * at.seq_len) {
        const int64_t mine = p0 + lane * at.seq_len;
        const unsigned there = __ballot_sync(kAll, mine < until && token_at(at, mine, nullptr) >= 0);
        const int here = __popc(there);
        any |= here > 0;
        const int32_t my_place = static_cast<int32_t>(p0 + nth_bit(there, lane) * at.seq_len);  // lane l: the l-th there
        if constexpr (kBoundsCheck) {
            if (!__all_sync(kAll, index_ok(a.status, lane >= here || (my_place >= 0 && my_place < a.n))))
                continue;
        }
#pragma unroll 1
        for (int q = 0; q < here; q += kInFlight) {
            SlabGroup<DT, VEC> x[kInFlight];
            int32_t place[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                place[u] = __shfl_sync(kAll, my_place, min(q + u, here - 1));
                x[u].load(w.cols, a.dout.data, static_cast<uint32_t>(place[u]) * a.dout.stride);
            }
            if (DROP)
                w.mask.template draw<kInFlight>(here - q, [&](int u) { return place[u]; });
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                if (q + u >= here)
                    break;
                w.add(x[u], u, place[u]);
            }
        }
    }
    if (roles.log_ways > 0) {  // the parts together, in order
        if (part > 0)
            w.put(shared.sums[warp][0], lane);
        if (lane == 0)
            shared.any[warp] = any;
        __syncthreads();
        if (part > 0)
            return;
#pragma unroll 1
        for (int other = warp + 1; other < warp + (1 << roles.log_ways); ++other) {
            any |= shared.any[other];
            w.add_group(shared.sums[other][0][0][lane], shared.sums[other][0][1][lane]);
        }
    }
    if (row >= a.rows)
        return;
    if (any)
        w.finish(row);
    else if (a.base.data != a.grad.data)
        fill_row<GT, VEC>(a, row, slab * kSlabCols<VEC>, min((slab + 1) * kSlabCols<VEC>, a.dim), lane);
}

// a: the table whose places are sorted; p: the positions' table.
// The bound of 64 registers was chosen on bf16 dout; of the kernels for an aligned
// fp32 dout, whose four rows in flight take twice the room, most spill 12 to 128
// bytes (16 x 1024 places of 768 columns, microseconds: bf16 to bf16 27.8, to fp32
// 38.9; fp32 to bf16 33.6, to fp32 42.1).
template <typename DT, typename GT, bool VEC, bool DROP, int POSITIONS>
__global__ void __launch_bounds__(kBlock, VEC ? 4 : 3)
    k_row_sums(const __grid_constant__ RowSumArgs a, const __grid_constant__ RowSumArgs p, const Places at, const Roles roles)
{
    __shared__ WalkShared<VEC, DROP> shared;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned block = blockIdx.x;
    if constexpr (POSITIONS != kNoPositions) {
        const unsigned before = roles.positions_before(block);
        if (roles.positions_before(block + 1) != before) {
            const int64_t unit = static_cast<int64_t>(before) * kWarps + warp;
            // Running positions need nothing of the sort, only what the launches before
            // it left (dout, the tokens), and so run while it does.  (All after the sort:
            // 64 x 1024 places of 2048 columns 169 us instead of 164, 1024 sequences of
            // 256 of 768 299 instead of 258.)
            if constexpr (POSITIONS == kRunningPositions) {
                wait_until_begun(p.begun, p.call, lane);
                running_row<DT, GT, VEC, DROP>(p, at, roles, unit, warp, lane, shared);
            }
            wait_for_launch_before();  // the launch after this one relies on the sort's end too
            if (POSITIONS == kRunningPositions && blockIdx.x == 0 && threadIdx.x == 0)
                tell_begun(p.begun, 0);  // blocks that start from here on find the sort done
            if constexpr (POSITIONS == kSortedPositions) {
                if (before < roles.position_walks)
                    walk<DT, GT, VEC, DROP>(p, before, warp, lane, shared);
                else
                    fill_rows<GT, VEC>(p, (unit - static_cast<int64_t>(roles.position_walks) * kWarps) * kFillRows, lane);
            }
            return;
        }
        block -= before;
    }
    const unsigned fills = roles.fills_before(block);
    wait_for_launch_before();
    if (roles.fills_before(block + 1) != fills)
        fill_rows<GT, VEC>(a, (static_cast<int64_t>(fills) * kWarps + warp) * kFillRows, lane);
    else
        walk<DT, GT, VEC, DROP>(a, block - fills, warp, lane, shared);
}

unsigned blocks_for(int64_t warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

// The share of `part` among `all`, in 2^-32, rounded up: exactly part of them.
uint64_t share_of(unsigned part, unsigned all) { return all ? ((static_cast<uint64_t>(part) << 32) + all - 1) / all : 0; }

unsigned walk_blocks(const RowSumArgs& a) { return blocks_for(grad_stretches(a.n, a.piece)) * a.slabs; }
unsigned fill_blocks(const RowSumArgs& a)
{
    return a.base.data == a.grad.data ? 0 : blocks_for((a.rows + kFillRows - 1) / kFillRows);  // none in place
}

template <typename DT, typename GT, bool VEC, bool DROP, int POSITIONS>
cudaError_t launch_p(const RowSumArgs& a, const RowSumArgs& p, const Places& at, cudaStream_t s)
{
    Roles roles = {};
    const unsigned walks = walk_blocks(a);
    const unsigned fills = fill_blocks(a);
    unsigned positions = 0;
    if (POSITIONS == kRunningPositions) {
        const int64_t sequences = (at.n + at.seq_len - 1) / at.seq_len, used = std::min<int64_t>(at.seq_len, at.n) * p.slabs;
        while (roles.log_ways < 3 && sequences >> roles.log_ways > kWay && used << (roles.log_ways + 1) <= kLead * kWarps)
            ++roles.log_ways;
        roles.way = ((sequences - 1) >> roles.log_ways) * at.seq_len + at.seq_len;
        positions = blocks_for((static_cast<int64_t>(p.rows) * p.slabs) << roles.log_ways);
        roles.lead = positions < kLead ? positions : kLead;
    } else if (POSITIONS == kSortedPositions) {
        roles.position_walks = walk_blocks(p);
        positions = roles.position_walks + fill_blocks(p);
    }
    const unsigned blocks = walks + fills + positions;
    if (blocks == 0)
        return cudaSuccess;
    roles.positions = share_of(positions - roles.lead, blocks - roles.lead);
    roles.walk_lead = walks < kLead ? walks : kLead;
    roles.fill = share_of(fills, walks - roles.walk_lead + fills);
    return launch_programmatic(k_row_sums<DT, GT, VEC, DROP, POSITIONS>, blocks, kBlock, 0, s, a, p, at, roles);
}

template <typename DT, typename GT, bool VEC, bool DROP>
cudaError_t launch_k(RowSumArgs a, RowSumArgs p, PositionKind kind, const Places& at, cudaStream_t s)
{
    a.slabs = p.slabs = slabs_of(a.dim, VEC);
    a.piece = p.piece = grad_piece(a.n, a.slabs);
    if (kind == kRunningPositions)
        return launch_p<DT, GT, VEC, DROP, kRunningPositions>(a, p, at, s);
    if (kind == kSortedPositions)
        return launch_p<DT, GT, VEC, DROP, kSortedPositions>(a, p, at, s);
    return launch_p<DT, GT, VEC, DROP, kNoPositions>(a, p, at, s);
}

template <typename DT, typename GT>
cudaError_t launch_t(const RowSumArgs& a, const RowSumArgs& p, PositionKind kind, const Places& at, bool vec, bool drop,
                     cudaStream_t s)
{
    if (vec)
        return drop ? launch_k<DT, GT, true, true>(a, p, kind, at, s) : launch_k<DT, GT, true, false>(a, p, kind, at, s);
    return drop ? launch_k<DT, GT, false, true>(a, p, kind, at, s) : launch_k<DT, GT, false, false>(a, p, kind, at, s);
}

}  // namespace

cudaError_t launch_row_sums(RowSumArgs a, const RowSumArgs* positions, PositionKind kind, const Places& at, int dout_type,
                            int grad_type, bool vec, bool drop, cudaStream_t s)
{
    const RowSumArgs& p = positions ? *positions : a;
    if (dout_type == LIONCUB_ROWS_BF16)
        return grad_type == LIONCUB_ROWS_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, p, kind, at, vec, drop, s)
                                              : launch_t<__nv_bfloat16, float>(a, p, kind, at, vec, drop, s);
    return grad_type == LIONCUB_ROWS_BF16 ? launch_t<float, __nv_bfloat16>(a, p, kind, at, vec, drop, s)
                                          : launch_t<float, float>(a, p, kind, at, vec, drop, s);
}

}  // namespace lc
