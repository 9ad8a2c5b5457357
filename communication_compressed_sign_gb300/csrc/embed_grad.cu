// embed_grad.cu -- gradient of the embedding lookup from the sorted places:
//   grad[v,:] = base[v,:] + factor * sum over places i with key_i == v of keep * dout[i,:].
//
// Every row of the dense gradient is written once -- rows without a place as
// zeros (or base) -- so there is no clearing pass, and no float atomics: the
// order of every sum depends on the batch alone.
//
// The unit of work is one warp on a slab of 256 columns.
//   walk   a stretch of `piece` entries of `order`: the warp adds the rows of
//          dout of the segments that begin there, several rows in flight
//          whatever the segments' lengths, and writes a row of grad at each
//          segment's end.  A segment of up to `piece` places belongs to the
//          stretch it begins in.  A longer one is cut at the stretches' bounds:
//          each warp leaves an fp32 partial, and the last of a group of partials to
//          arrive (an integer counter) adds them in order.  So units are alike in size
//          however skewed the tokens are.
//   fill   rows without a place.
// Bound by memory: dout is read once and grad written once.
#include "embed_device.cuh"

namespace lc {
namespace {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;
constexpr int kInFlight = 4;              // rows of dout a warp loads before it adds them
constexpr int kFillRows = 8;              // rows of grad a fill warp looks at
constexpr int kScanRows = 64;             // rows of grad a scanning fill block takes
constexpr int64_t kScan = 2048;           // batches up to this many places fill by scanning
constexpr unsigned kLead = 152 * 4;       // blocks the SMs hold
constexpr unsigned kLeadScans = 152 * 2;  // scanning fills that run beside the sort

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
    __device__ __forceinline__ void add(const SlabGroup<DT, VEC>& x, uint32_t i)
    {
        if constexpr (DROP && sizeof(DT) == 2) {
            mask.add(i, x, sum);
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
                mask.row(i, [&](int k, bool keep) {
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
    // Adds up the pieces of a long segment: a tree of groups of 8, in which the
    // last of a group to arrive adds the group's partials in order and goes on
    // as one piece of the next level.  True where the whole sum has come together.
    __device__ __forceinline__ bool gather(int2 seg, int stretch, int slab, int lane)
    {
        const int first = seg.x / a.piece;
        int node = stretch - first, nodes = (seg.y - 1) / a.piece - first + 1;
        const int64_t column = slab * 256 + lane * 8;  // partial rows are whole slabs
        // piece r's partial and counter: slot 1 of the stretch the segment begins in, slot 0 of the later ones
        auto slot = [&](int r) { return 2 * static_cast<int64_t>(first + r) + (r == 0 ? 1 : 0); };
        auto partial = [&](int r) { return a.partial + slot(r) * a.partial_stride + column; };
        if (!index_ok(a.status, 2 * static_cast<int64_t>(stretch) + 1 < a.partial_rows))
            return false;
#pragma unroll 1
        for (int level = 0; nodes > 1; ++level) {
            const int group = node >> 3, members = min(8, nodes - group * 8), scale = 3 * level;
            store_partial(partial(node << scale));
            __threadfence();
            __syncwarp();
            int before = 0;
            if (lane == 0)  // four bits a level
                before = atomicAdd(&a.arrived[slot(group << scale << 3) * a.slabs + slab], 1 << (4 * level));
            before = __shfl_sync(kAll, before, 0);
            if ((before >> (4 * level) & 15) != members - 1)
                return false;
            __threadfence();
            clear();
#pragma unroll 4
            for (int m = 0; m < members; ++m)
                add_partial(partial((group * 8 + m) << scale));
            node = group;
            nodes = (nodes + 7) / 8;
        }
        return true;
    }
    // A lane's sums lie together in a partial row, whichever columns they are.
    __device__ __forceinline__ void store_partial(float* p) const
    {
        reinterpret_cast<float4*>(p)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(sum[4], sum[5], sum[6], N == 8 ? sum[N - 1] : 0.0f);
    }
    __device__ __forceinline__ void add_partial(const float* p)
    {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(p)), y = __ldcg(reinterpret_cast<const float4*>(p) + 1);
        const float z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < N; ++k)
            sum[k] = __fadd_rn(sum[k], z[k]);
    }
};

// Row v on one slab: zeros, or base.
template <typename GT, bool VEC>
__device__ __forceinline__ void fill_slab(const RowSumArgs& a, const Slab<VEC>& cols, int64_t v)
{
    if (a.base.data) {
        SlabGroup<GT, VEC> b;
        b.load(cols, a.base.data, v * a.base.stride);
        b.store(cols, a.grad.data, v * a.grad.stride);
    } else {
        const float zero[kLaneCols<VEC>] = {};
        store_slab<GT, VEC>(cols, a.grad.data, v * a.grad.stride, zero);
    }
}

// Those of rows [row0, row0 + kScanRows) that no token of the batch has, found
// without the sort: the block looks through all tokens.
template <typename GT, bool VEC>
__device__ __forceinline__ void scan_and_fill(const RowSumArgs& a, const Places& at, int64_t row0, int warp, int lane)
{
    __shared__ unsigned has[kScanRows / 32];
    if (threadIdx.x < kScanRows / 32)
        has[threadIdx.x] = 0;
    __syncthreads();
    constexpr int kTokens = 8;  // loads in flight
    for (int i0 = threadIdx.x; i0 < at.n; i0 += kTokens * kBlock) {
        int64_t t[kTokens];
#pragma unroll
        for (int u = 0; u < kTokens; ++u)
            t[u] = i0 + u * kBlock < at.n ? index_at(at.tokens, i0 + u * kBlock, at.wide) : -1;
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            const uint64_t r = static_cast<uint64_t>(t[u] - row0);
            if (t[u] >= 0 && r < kScanRows)
                atomicOr(&has[r >> 5], 1u << (r & 31));
        }
    }
    __syncthreads();
    for (int r = warp; r < kScanRows; r += kWarps) {
        if ((has[r >> 5] >> (r & 31) & 1u) || row0 + r >= a.rows)
            continue;
        for (int slab = 0; slab < a.slabs; ++slab)
            fill_slab<GT, VEC>(a, Slab<VEC>(slab, lane, a.dim), row0 + r);
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
        for (int slab = 0; slab < a.slabs; ++slab)
            fill_slab<GT, VEC>(a, Slab<VEC>(slab, lane, a.dim), v);
    }
}

// Programmatic launches: a kernel may start before the launch before it in the
// stream has ended, and waits here until all of that is done and visible.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// What the blocks of a launch do.  Blocks that need no sort lead, while it may
// still run: fills that scan the tokens (small batches), else running positions.
// The rest are spread evenly: walks are bound by latency or, with dropout, by
// integer instructions, and fills by memory, so they run side by side.
struct Roles {
    int scan;            // fills look through the tokens (kScanRows rows a block), else through the segments
    unsigned scans;      // such blocks at the front
    unsigned lead;       // position blocks at the front
    uint64_t positions;  // share of position blocks among the others, in 2^-32
    uint64_t fill;       // share of fill blocks among walks and fills, likewise
    unsigned position_walks;  // sorted positions: walks before fills
    __host__ __device__ __forceinline__ unsigned positions_before(unsigned block) const
    {
        return block <= lead ? block : lead + static_cast<unsigned>(((block - lead) * positions) >> 32);
    }
    __host__ __device__ __forceinline__ unsigned fills_before(unsigned block) const
    {
        return static_cast<unsigned>((block * fill) >> 32);
    }
};

// One stretch of the sorted places on one slab.
template <typename DT, typename GT, bool VEC, bool DROP>
__device__ __forceinline__ void walk(const RowSumArgs& a, int64_t unit, int lane, typename SlabMask<VEC>::Shared* shared)
{
    const int stretch = static_cast<int>(quotient(unit, a.slabs));  // places and so stretches fit 31 bits
    const int slab = static_cast<int>(unit - static_cast<int64_t>(stretch) * a.slabs);
    const int total = *a.total;
    if (static_cast<int64_t>(stretch) * a.piece >= total)
        return;
    const int begin = stretch * a.piece, end = min(begin + a.piece, total);
    // the stretch, and what a short segment can reach beyond it
    const int mine = begin + lane;
    const int32_t my_place = mine < total ? a.order[mine] : 0, my_key = mine < total ? a.sorted_key[mine] : 0;
    if (!__all_sync(kAll, index_ok(a.status, my_place >= 0 && my_place < a.n && my_key >= 0 && my_key < a.rows)))
        return;
    const int2 seg0 = a.segment[__shfl_sync(kAll, my_key, 0)], seg1 = a.segment[__shfl_sync(kAll, my_key, end - 1 - begin)];
    const bool tail = seg0.x < begin && seg0.y - seg0.x > a.piece;   // a long segment goes on here
    const bool head = seg1.x >= begin && seg1.y - seg1.x > a.piece;  // a long segment begins here
    // short segments: one that began before belongs there, one that begins here is taken to its end
    const int from = seg0.x < begin ? seg0.y : begin, to = head ? seg1.x : (seg1.x < begin ? begin : seg1.y);
    const int32_t above = __shfl_up_sync(kAll, my_key, 1);
    const unsigned begins = __ballot_sync(kAll, lane == 0 || my_key != above);

    Walker<DT, GT, VEC, DROP> w(a, slab, lane, shared);
#pragma unroll 1
    for (int part = 0; part < 3; ++part) {  // the long segment's end, short segments, a long segment's begin
        if (part == 0 ? !tail : part == 2 && !head)
            continue;
        const int lo = part == 0 ? begin : part == 1 ? from : seg1.x;
        const int hi = part == 0 ? min(seg0.y, end) : part == 1 ? to : end;
        if (lo >= hi)
            continue;
        w.clear();
        const int here = hi - begin;
        int32_t current = __shfl_sync(kAll, my_key, lo - begin);
#pragma unroll 1
        for (int q = lo - begin; q < here; q += kInFlight) {
            SlabGroup<DT, VEC> x[kInFlight];
            int32_t place[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {  // past the end the last row again: no branch between the loads
                place[u] = __shfl_sync(kAll, my_place, min(q + u, here - 1));
                x[u].load(w.cols, a.dout.data, static_cast<uint32_t>(place[u]) * a.dout.stride);
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                if (q + u >= here)
                    break;
                if ((begins >> (q + u) & 1u) && q + u > lo - begin) {
                    w.finish(current);
                    w.clear();
                    current = __shfl_sync(kAll, my_key, q + u);
                }
                w.add(x[u], place[u]);
            }
        }
        if (part == 1 || w.gather(part == 0 ? seg0 : seg1, stretch, slab, lane))
            w.finish(current);
    }
}

// Positions that run with the place, first + i % seq_len: row q's places are
// q - first, q - first + seq_len, ... and need no sort.  One row on one slab.
template <typename DT, typename GT, bool VEC, bool DROP>
__device__ __forceinline__ void running_row(const RowSumArgs& a, const Places& at, int64_t unit, int lane,
                                            typename SlabMask<VEC>::Shared* shared)
{
    const int64_t row = quotient(unit, a.slabs);
    const int slab = static_cast<int>(unit - row * a.slabs);
    if (row >= a.rows)
        return;
    const int64_t place0 = row - at.first;
    if (place0 < 0 || place0 >= at.seq_len || place0 >= at.n) {
        if (a.base.data != a.grad.data)
            fill_slab<GT, VEC>(a, Slab<VEC>(slab, lane, a.dim), row);
        return;
    }
    Walker<DT, GT, VEC, DROP> w(a, slab, lane, shared);
    for (int64_t p0 = place0; p0 < at.n; p0 += 32 * at.seq_len) {
        const int64_t mine = p0 + lane * at.seq_len;
        const unsigned there = __ballot_sync(kAll, mine < at.n && token_at(at, mine, nullptr) >= 0);
        const int here = __popc(there);
        const int32_t my_place = static_cast<int32_t>(p0 + nth_bit(there, lane) * at.seq_len);  // lane l: the l-th there
#pragma unroll 1
        for (int q = 0; q < here; q += kInFlight) {
            SlabGroup<DT, VEC> x[kInFlight];
            int32_t place[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                place[u] = __shfl_sync(kAll, my_place, min(q + u, here - 1));
                x[u].load(w.cols, a.dout.data, static_cast<uint32_t>(place[u]) * a.dout.stride);
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                if (q + u >= here)
                    break;
                w.add(x[u], place[u]);
            }
        }
    }
    w.finish(row);
}

// a: the table whose places are sorted; p: the positions' table.
template <typename DT, typename GT, bool VEC, bool DROP, int POSITIONS>
__global__ void __launch_bounds__(kBlock, VEC ? 4 : 3)
    k_row_sums(const __grid_constant__ RowSumArgs a, const __grid_constant__ RowSumArgs p, const Places at, const Roles roles)
{
    __shared__ typename SlabMask<VEC>::Shared buffers[DROP ? kWarps : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    typename SlabMask<VEC>::Shared* shared = &buffers[DROP ? warp : 0];
    unsigned block = blockIdx.x;
    if (block < roles.scans) {
        scan_and_fill<GT, VEC>(a, at, static_cast<int64_t>(block) * kScanRows, warp, lane);
        wait_for_launch_before();  // the launch after this one relies on it
        return;
    }
    block -= roles.scans;
    if constexpr (POSITIONS != kNoPositions) {
        const unsigned before = roles.positions_before(block);
        if (roles.positions_before(block + 1) != before) {
            const int64_t unit = static_cast<int64_t>(before) * kWarps + warp;
            if constexpr (POSITIONS == kRunningPositions)
                running_row<DT, GT, VEC, DROP>(p, at, unit, lane, shared);
            wait_for_launch_before();
            if constexpr (POSITIONS == kSortedPositions) {
                if (before < roles.position_walks)
                    walk<DT, GT, VEC, DROP>(p, unit, lane, shared);
                else
                    fill_rows<GT, VEC>(p, (unit - static_cast<int64_t>(roles.position_walks) * kWarps) * kFillRows, lane);
            }
            return;
        }
        block -= before;
    }
    const unsigned fills = roles.fills_before(block);
    const bool fill = roles.fills_before(block + 1) != fills;
    if (fill && roles.scan)
        scan_and_fill<GT, VEC>(a, at, static_cast<int64_t>(roles.scans + fills) * kScanRows, warp, lane);
    wait_for_launch_before();
    if (fill && !roles.scan)
        fill_rows<GT, VEC>(a, (static_cast<int64_t>(fills) * kWarps + warp) * kFillRows, lane);
    else if (!fill)
        walk<DT, GT, VEC, DROP>(a, static_cast<int64_t>(block - fills) * kWarps + warp, lane, shared);
}

unsigned blocks_for(int64_t warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

// The share of `part` among `all`, in 2^-32, rounded up: exactly part of them.
uint64_t share_of(unsigned part, unsigned all) { return all ? ((static_cast<uint64_t>(part) << 32) + all - 1) / all : 0; }

unsigned walk_blocks(const RowSumArgs& a) { return blocks_for(grad_stretches(a.n, a.piece) * a.slabs); }
unsigned fill_blocks(const RowSumArgs& a)
{
    return a.base.data == a.grad.data ? 0 : blocks_for((a.rows + kFillRows - 1) / kFillRows);  // none in place
}

template <typename DT, typename GT, bool VEC, bool DROP, int POSITIONS>
cudaError_t launch_p(const RowSumArgs& a, const RowSumArgs& p, const Places& at, cudaStream_t s)
{
    Roles roles = {};
    const unsigned walks = walk_blocks(a);
    unsigned fills = fill_blocks(a), positions = 0;
    if (fills > 0 && a.scan && a.n <= kScan) {
        const unsigned scans = static_cast<unsigned>((a.rows + kScanRows - 1) / kScanRows);
        roles.scan = 1;
        roles.scans = scans < kLeadScans ? scans : kLeadScans;
        fills = scans - roles.scans;
    }
    if (POSITIONS == kRunningPositions) {
        positions = blocks_for(static_cast<int64_t>(p.rows) * p.slabs);
        roles.lead = roles.scan ? 0 : positions < kLead ? positions : kLead;
    } else if (POSITIONS == kSortedPositions) {
        roles.position_walks = walk_blocks(p);
        positions = roles.position_walks + fill_blocks(p);
    }
    const unsigned blocks = walks + fills + positions;
    if (roles.scans + blocks == 0)
        return cudaSuccess;
    roles.positions = share_of(positions - roles.lead, blocks - roles.lead);
    roles.fill = share_of(fills, walks + fills);
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(roles.scans + blocks);
    c.blockDim = dim3(kBlock);
    c.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k_row_sums<DT, GT, VEC, DROP, POSITIONS>, a, p, at, roles);
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
