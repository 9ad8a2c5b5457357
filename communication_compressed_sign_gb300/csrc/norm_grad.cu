// norm_grad.cu -- the gradient of the root-mean-square norm (n = h * rstd,
// g = dout * weight):
//   dx = residual_grad + rstd * (g - n * mean(g * n)),  again = n * weight,
//   weight_grad_j = weight_base_j + sum over rows of dout * n.
//
// Memory-bound.  A team of warps takes a row at a time, with one sum over the row
// between reading and writing it.  Teams walk over rows (persistent blocks, one
// for each multiprocessor), so that a column's share of the weight's gradient
// stays in a register (up to 8192 columns); three threads of the team have the next rows brought into
// a ring in shared memory by bulk copies meanwhile, one matrix each.  A block adds its teams'
// columns in order and leaves one row of sums, and a second launch adds those of
// all blocks in order.
//
// Measured: 65536 x 2048 bf16 from int8, with the normed rows again, 181.8 us (6.7
// TB/s, 98 % of a measured copy); 8192 x 768 onto fp32 18.0 us (4.9 TB/s; some 6
// of them are the two launches' beginnings and ends, 2.6 the second launch); 4907
// x 771 bf16 13.8 us (2.2 TB/s, scalar reads of the ring; 16.7 with one thread
// starting the copies of all matrices).  Above 8192 columns a lane has 32 elements
// of a row, and of what it keeps for them (the weight's sums, dout, h, the residual)
// 236 to 636 bytes a thread are spilled: 4096 x 16384 bf16 153 us (3.5 TB/s), from
// int8 150 (3.1 TB/s).  65536 x 2048 with its rows loaded ahead into registers, 16
// warps an SM: 241 us (too few loads in flight); with each thread's elements copied
// ahead by itself (cp.async): 246 us (as many instructions for the load-store unit as
// bytes allow).
//
// A row of any alignment comes by bulk copies: of the 16-byte pieces that it
// touches, as far as they lie within the matrix; the ends of the first and the last
// row that do not are copied by the thread that starts the copy.
#include "block_device.cuh"

namespace lc {
namespace {

constexpr int kBlockWarps = 16;
// Rows of a team in flight: as many as fit kRingWanted, two where that is one and
// kRingBytes has room.  More only let reads run further ahead of the writes: 8192
// fp32 rows of 768 took 14.9 us with two, 15.8 with three, 17.1 with five; 16384
// rows of 2048 from 8 bits 51.0, 51.8 and 53.2.
constexpr int kMaxSlots = 8;
constexpr int kRingWanted = 72 * 1024, kRingBytes = 208 * 1024;
constexpr uint32_t kWaitLimit = 1u << 20;  // polls

// Where h comes from; scalar reads go by the type that the launch gives.
enum Source { kFromBf16, kFromF32, kFromCodes };

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Waits for a phase of a barrier, for a bounded time; false when it gave up.
__device__ __forceinline__ bool wait_phase(uint32_t barrier, uint32_t parity)
{
    uint32_t ok = 0;
    for (uint32_t i = 0; i < kWaitLimit && !ok; ++i)
        asm volatile("{\n .reg .pred P;\n mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2;\n selp.u32 %0, 1, 0, P;\n}"
                     : "=r"(ok) : "r"(barrier), "r"(parity) : "memory");
    return ok != 0;
}
// The same with at most `polls` tests that return at once: the stand-in for a wait
// that runs out, and all that is left after one did.
__device__ __forceinline__ bool test_phase(uint32_t barrier, uint32_t parity, uint32_t polls)
{
    uint32_t ok = 0;
    for (uint32_t i = 0; i < polls && !ok; ++i)
        asm volatile("{\n .reg .pred P;\n mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n selp.u32 %0, 1, 0, P;\n}"
                     : "=r"(ok) : "r"(barrier), "r"(parity) : "memory");
    return ok != 0;
}

// Meets the warps of a team, whose earlier reads and writes of shared memory are then done.
__device__ __forceinline__ void team_barrier(int team, int warps)
{
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

// A matrix whose rows are brought into shared memory: those of a slot start `at`
// bytes behind the slot's start, on a 16-byte boundary of memory.
struct Stream {
    const char* base;
    int64_t step;  // bytes between rows
    int32_t bytes;  // of a row; 0: no such matrix
    int32_t at;
};

#ifdef LIONCUB_BOUNDS_CHECK
// Where the room of a matrix ends in a slot.
__device__ __forceinline__ int32_t room_end(const NormGradArgs& a, const Stream& m)
{
    return m.at == 0 ? a.at_saved : m.at == a.at_saved ? a.at_residual : a.slot_bytes;
}
__device__ __forceinline__ uint32_t ring_bytes()
{
    uint32_t n;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(n));
    return n;
}
#endif

// Checked builds: whether the bytes [begin, end) of a slot are in the room of a matrix there.
__device__ __forceinline__ bool room_ok(const NormGradArgs& a, const Stream& m, const char* slot, int64_t begin, int64_t end)
{
#ifdef LIONCUB_BOUNDS_CHECK
    extern __shared__ __align__(16) char shared[];
    const int64_t at = slot - shared;
    return access_ok(begin >= m.at && begin <= end && end <= room_end(a, m) && at >= 0 && at % a.slot_bytes == 0 && at + end <= ring_bytes());
#else
    return true;
#endif
}

// Checked builds: whether a row is one of a matrix, and whether a copy starts and ends at
// 16-byte boundaries, between the first and the last of its elements.
__device__ __forceinline__ bool row_ok(const NormGradArgs& a, const Stream& m, int64_t row)
{
#ifdef LIONCUB_BOUNDS_CHECK
    const int64_t rows = m.at == 0 ? a.dout.rows : m.at != a.at_saved ? a.residual_grad.rows : a.packed.codes ? a.packed.rows : a.saved.rows;
    return access_ok(row >= 0 && row < rows && row < a.n);
#else
    return true;
#endif
}
__device__ __forceinline__ bool copy_ok(const NormGradArgs& a, const Stream& m, const char* from, const char* to, uint32_t bytes)
{
#ifdef LIONCUB_BOUNDS_CHECK
    return access_ok(((reinterpret_cast<uintptr_t>(from) | shared_address(to) | bytes) & 15) == 0 && from >= m.base &&
                     from + bytes <= m.base + (a.n - 1) * m.step + m.bytes);
#else
    return true;
#endif
}

// The slot of a row that starts `shift` bytes behind a boundary has it `shift`
// bytes behind its own start.
__device__ __forceinline__ uint32_t shift_of(const Stream& m, int64_t row)
{
    return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(m.base)) + static_cast<uint32_t>(row) * static_cast<uint32_t>(m.step)) & 15;
}

// Bytes that the copies of a row bring: whole 16-byte pieces, but none that lies
// partly before the matrix's first or behind its last element.
struct Window {
    const char *row, *from, *to;
    __device__ __forceinline__ Window(const Stream& m, int64_t i, int64_t n)
    {
        constexpr uintptr_t kPiece = 15;
        row = m.base + i * m.step;
        const uintptr_t a = reinterpret_cast<uintptr_t>(row), first = reinterpret_cast<uintptr_t>(m.base);
        const uintptr_t last = first + (n - 1) * m.step + m.bytes;
        const uintptr_t low = max(a & ~kPiece, (first + kPiece) & ~kPiece), high = min((a + m.bytes + kPiece) & ~kPiece, last & ~kPiece);
        from = reinterpret_cast<const char*>(low);
        to = reinterpret_cast<const char*>(max(low, high));
    }
    __device__ __forceinline__ uint32_t bytes() const { return static_cast<uint32_t>(to - from); }
};

// One thread for each stream: starts the copy of its row i into a slot.
template <bool VEC>
__device__ __forceinline__ void start_row(const NormGradArgs& a, const Stream& m, int64_t i, char* slot, uint32_t barrier)
{
    const char* from = m.base + i * m.step;
    uint32_t bytes = m.bytes;
    char* to = slot + m.at;
    // what was read and written in the slot by ordinary accesses comes before the copy
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    if constexpr (!VEC) {
        const Window w(m, i, a.n);
        to += shift_of(m, i);
        // what lies outside, in the first and the last rows
        const char* end = w.row + m.bytes;
        if (row_ok(a, m, i) && room_ok(a, m, slot, to - slot, to - slot + m.bytes)) {
            for (const char* p = w.row; p < w.from && p < end; ++p)
                to[p - w.row] = *p;
            for (const char* p = w.to > w.row ? w.to : w.row; p < end; ++p)
                to[p - w.row] = *p;
        }
        to += w.from - w.row;
        from = w.from;
        bytes = w.bytes();
    }
    if (bytes && !(row_ok(a, m, i) && room_ok(a, m, slot, to - slot, to - slot + bytes) && copy_ok(a, m, from, to, bytes)))
        bytes = 0;
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(barrier), "r"(bytes) : "memory");
    if (bytes)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(shared_address(to)),
                     "l"(from), "r"(bytes), "r"(barrier)
                     : "memory");
}

// A lane's elements of a chunk, from a row in shared memory.
template <typename T, bool VEC>
__device__ __forceinline__ void read_chunk(Chunk<T, VEC>& v, const Columns<VEC>& c, const char* row, int type)
{
    if constexpr (VEC) {
        if constexpr (sizeof(T) == 2) {
            v.g.raw = c.count ? *reinterpret_cast<const uint4*>(row + c.at * 2) : make_uint4(0, 0, 0, 0);
        } else {
            const float4* p = reinterpret_cast<const float4*>(row + c.at * 4);
            v.g.a = c.count ? p[0] : make_float4(0, 0, 0, 0);
            v.g.b = c.count ? p[1] : make_float4(0, 0, 0, 0);
        }
    } else {
        v.load(c, row, 0, type);
    }
}
template <bool VEC>
__device__ __forceinline__ void read_codes(CodeChunk<VEC>& v, const Columns<VEC>& c, const char* row)
{
    if constexpr (VEC) {
        v.w = c.count ? *reinterpret_cast<const uint2*>(row + c.at) : make_uint2(0, 0);
    } else {
        const uint8_t* codes = reinterpret_cast<const uint8_t*>(row) + c.at;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v.code[k] = k < c.count ? codes[32 * k] : 0;
    }
}

// Checked builds: whether a column of a team has a place among the block's sums.
__device__ __forceinline__ bool sums_ok(const NormGradArgs& a, int team, int64_t column)
{
#ifdef LIONCUB_BOUNDS_CHECK
    return access_ok(team < a.teams && column < a.dim && (int64_t(team) * a.dim + column + 1) * int64_t(sizeof(float)) <= ring_bytes());
#else
    return true;
#endif
}

template <bool VEC>
__device__ __forceinline__ void load_weight(const NormGradArgs& a, const Columns<VEC>& c, float (&w)[8])
{
    if (a.weight.data) {
        load_typed<VEC>(c, a.weight, 0, w);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = 1.0f;
    }
}

template <typename DT, typename GT, int SOURCE, int C, bool VEC>
__global__ void __launch_bounds__(kBlockWarps * 32, 1) k_norm_grad(const __grid_constant__ NormGradArgs a)
{
    constexpr bool kKeepWeight = C <= 2;  // else it is read again from cache, for the registers
    constexpr bool kCodes = SOURCE == kFromCodes;
    extern __shared__ __align__(16) char shared[];  // the ring; in the end the block's sums of its columns
    __shared__ float sums[2][kBlockWarps];
    __shared__ int gave_up[kBlockWarps];  // a team's wait ran out
    __shared__ __align__(8) uint64_t barriers[kBlockWarps * kMaxSlots];
    const int lane = threadIdx.x & 31, in_block = threadIdx.x >> 5;
    const int warps = a.warps, team = in_block / warps, warp = in_block - team * warps;
    Columns<VEC> cols[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        cols[c] = Columns<VEC>((warp * C + c) * kChunk, lane, a.dim);
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + team;
    const int size_d = VEC ? sizeof(DT) : a.dout.type == LIONCUB_ROWS_BF16 ? 2 : 4;
    const int size_h = kCodes ? 1 : VEC ? (SOURCE == kFromBf16 ? 2 : 4) : a.saved.type == LIONCUB_ROWS_BF16 ? 2 : 4;
    const int size_g = VEC ? sizeof(GT) : a.residual_grad.type == LIONCUB_ROWS_BF16 ? 2 : 4;
    const Stream streams[3] = {
        {static_cast<const char*>(a.dout.data), a.dout.stride * size_d, a.dim * size_d, 0},
        {kCodes ? reinterpret_cast<const char*>(a.packed.codes) : static_cast<const char*>(a.saved.data),
         kCodes ? a.packed.stride : a.saved.stride * size_h, a.dim * size_h, a.at_saved},
        {static_cast<const char*>(a.residual_grad.data), a.residual_grad.stride * size_g, a.residual_grad.data ? a.dim * size_g : 0,
         a.at_residual}};
    char* ring = shared + static_cast<int64_t>(team) * a.slots * a.slot_bytes;
    const uint32_t full = shared_address(barriers + team * kMaxSlots);
    // the first lanes of a team start the copies, one stream each
    const Stream mine = lane == 0 ? streams[0] : lane == 1 ? streams[1] : streams[2];
    const bool starts = warp == 0 && lane < 3 && mine.bytes;
    if (warp == 0 && lane == 0) {
        gave_up[team] = 0;
        for (int k = 0; k < a.slots; ++k)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(full + 8 * k), "r"(a.residual_grad.data ? 3 : 2) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    team_barrier(team, warps);
    let_next_launch_start();
    wait_for_launch_before();
    uint32_t started = 0, last_parity = 0;  // of the slots, a bit each
    if (starts)
        for (int k = 0; k < a.slots && row + k * step < a.n; ++k) {
            start_row<VEC>(a, mine, row + k * step, ring + k * a.slot_bytes, full + 8 * k);
            started |= 1u << k;
        }

    // what is small is loaded a row ahead
    float rstd = 0.0f, scale[C] = {};
    const auto load_small = [&](int64_t i) {
        rstd = access_ok(i >= 0 && i < a.n) ? a.rstd[i] : 0.0f;
        if constexpr (kCodes) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int64_t at = VEC ? cols[c].at : cols[c].at - lane + 32 * (lane & 7);
                scale[c] = at < a.dim && scale_inside(a.packed, i, at >> a.packed.log_group) ? a.packed.scales[i * a.packed.scale_stride + (at >> a.packed.log_group)] : 0.0f;
            }
        }
    };
    if (row < a.n)
        load_small(row);
    float weight[kKeepWeight ? C : 1][8], grad[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            grad[c][k] = 0.0f;
        if constexpr (kKeepWeight)
            load_weight<VEC>(a, cols[c], weight[c]);
    }
    uint32_t parity = 0, polls = a.first_wait_polls;  // polls: 0 for the ordinary wait
    bool failed = false;
    int turn = 0, slot = 0;
    for (; row < a.n; row += step) {
        if (!(polls ? test_phase(full + 8 * slot, parity, polls) : wait_phase(full + 8 * slot, parity))) {
            gave_up[team] = 1;
            flag(a.status, kStatusWaitTimeout);
        }
        // dout, then g = dout * weight; n = h * rstd
        float g[C][8], n[C][8];
        float2 sums2 = both(0.0f);
        Chunk<GT, VEC> residual[C];
        const float r = rstd;
        const char* in = ring + slot * a.slot_bytes;
        // checked builds: none of a lane's columns where they are not in the matrix's room of the slot
        const auto in_slot = [&](const Stream& m, const Columns<VEC>& c, int size) {
            const int64_t at = m.at + (VEC ? 0 : shift_of(m, row));
            return !c.count || (access_ok(c.last() < a.dim) && room_ok(a, m, in, at + c.at * size, at + (c.last() + 1) * size)) ? c : c.none();
        };
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float w[8];
            if constexpr (!kKeepWeight)
                load_weight<VEC>(a, cols[c], w);
            Chunk<DT, VEC> d;
            read_chunk(d, in_slot(streams[0], cols[c], size_d), in + (VEC ? 0 : shift_of(streams[0], row)), a.dout.type);
            d.unpack(g[c]);
            const char* h = in + a.at_saved + (VEC ? 0 : shift_of(streams[1], row));
            const Columns<VEC> from = in_slot(streams[1], cols[c], size_h);
            if constexpr (kCodes) {
                CodeChunk<VEC> v;
                read_codes(v, from, h);
                v.scale = scale[c];
                v.unpack(a.packed, n[c]);
            } else {
                Chunk<std::conditional_t<SOURCE == kFromBf16, __nv_bfloat16, float>, VEC> v;
                read_chunk(v, from, h, a.saved.type);
                v.unpack(n[c]);
            }
            if (a.residual_grad.data)
                read_chunk(residual[c], in_slot(streams[2], cols[c], size_g), in + a.at_residual + (VEC ? 0 : shift_of(streams[2], row)),
                           a.residual_grad.type);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 nk = mul2(pair_of(n[c], k), both(r)), dk = pair_of(g[c], k);
                const float2 gk = mul2(dk, pair_of(kKeepWeight ? weight[kKeepWeight ? c : 0] : w, k));
                set_pair(grad[c], k, fma2(dk, nk, pair_of(grad[c], k)));
                sums2 = fma2(gk, nk, sums2);
                set_pair(n[c], k, nk);
                set_pair(g[c], k, gk);
            }
        }
        if (row + step < a.n)
            load_small(row + step);
        float sum = warp_sum(__fadd_rn(sums2.x, sums2.y));
        if (warps > 1 && lane == 0)  // sums of two rows take turns, so one barrier a row is enough
            sums[turn][in_block] = sum;
        team_barrier(team, warps);
        // What follows a wait that ran out is not what it should be, but ends soon: the team
        // starts no row and has no long wait any more.
        failed = gave_up[team];
        polls = failed ? 1 : 0;
        if (starts && !failed && row + a.slots * step < a.n) {  // the slot has been read
            start_row<VEC>(a, mine, row + a.slots * step, ring + slot * a.slot_bytes, full + 8 * slot);
            last_parity ^= 1u << slot;
        }
        if (++slot == a.slots) {
            slot = 0;
            parity ^= 1;
        }
        if (warps > 1) {
            sum = 0.0f;
            for (int k = 0; k < warps; ++k)
                sum = __fadd_rn(sum, sums[turn][team * warps + k]);
            turn ^= 1;
        }
        const float mean = __fmul_rn(sum, a.per_column);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.again.data) {
                float y[8], w[8];
                if constexpr (!kKeepWeight)
                    load_weight<VEC>(a, cols[c], w);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    set_pair(y, k, mul2(pair_of(n[c], k), pair_of(kKeepWeight ? weight[kKeepWeight ? c : 0] : w, k)));
                store_typed<VEC>(cols[c], a.again, row, y);
            }
            float rest[8] = {};
            if (a.residual_grad.data)
                residual[c].unpack(rest);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                set_pair(g[c], k, fma2(both(r), fma2(pair_of(n[c], k), both(-mean), pair_of(g[c], k)), pair_of(rest, k)));
            store_typed<VEC>(cols[c], a.dx, row, g[c]);
        }
    }
    if (failed)  // no copy may still be under way when the block ends
        for (int k = 0; k < a.slots; ++k)
            if (started >> k & 1)
                wait_phase(full + 8 * k, last_parity >> k & 1);
    if (!a.partial)
        return;
    float* columns = reinterpret_cast<float*>(shared);  // a row for each team
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float* mine = columns + team * a.dim + cols[c].at;
        if (cols[c].count && !sums_ok(a, team, cols[c].last()))
            continue;
        if (VEC) {
            if (cols[c].count) {
                Group8<float> v;
                v.pack(grad[c]);
                v.store(mine, 0);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < cols[c].count)
                    mine[32 * k] = grad[c][k];
        }
    }
    __syncthreads();
    float* to = a.partial + static_cast<int64_t>(blockIdx.x) * a.dim;
    if (index_ok(a.status, static_cast<int64_t>(blockIdx.x) < a.partial_rows))
        for (int j = threadIdx.x; j < a.dim; j += blockDim.x) {
            float sum = columns[j];
            for (int t = 1; t < a.teams; ++t)
                sum = __fadd_rn(sum, columns[t * a.dim + j]);
            to[j] = sum;
        }
}

// The blocks' rows, added in a fixed order: a warp adds every 32nd row of 32
// columns, all of its loads in flight at once, and then takes one of the columns.
constexpr int kJoinWarps = 32, kJoinLoads = 5;

// Checked builds: whether a column is one of a row's.
__device__ __forceinline__ bool one_row_ok(const TypedRows& m, int column)
{
#ifdef LIONCUB_BOUNDS_CHECK
    return access_ok(m.rows == 1 && column >= 0 && column < m.cols);
#else
    return true;
#endif
}

__global__ void __launch_bounds__(kJoinWarps * 32) k_weight_grad(const __grid_constant__ WeightGradArgs a)
{
    __shared__ float sums[kJoinWarps][33];  // a column of it touches every bank once
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.x * 32;
    let_next_launch_start();
    wait_for_launch_before();
    float sum = 0.0f;
    if (first + lane < a.dim)
        for (int row = warp; row < a.rows; row += kJoinLoads * kJoinWarps) {
            float v[kJoinLoads];
#pragma unroll
            for (int u = 0; u < kJoinLoads; ++u) {
                const int i = row + u * kJoinWarps;
                v[u] = i < a.rows && access_ok(first + lane < a.dim) ? a.partial[static_cast<int64_t>(i) * a.dim + first + lane] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < kJoinLoads; ++u)
                sum = __fadd_rn(sum, v[u]);
        }
    sums[warp][lane] = sum;
    __syncthreads();
    const int j = first + warp;
    sum = warp_sum(sums[lane][warp]);
    if (lane || j >= a.dim || !one_row_ok(a.grad, j) || (a.base.data && !one_row_ok(a.base, j)))
        return;
    if (a.base.data)
        sum = __fadd_rn(sum, a.base.type == LIONCUB_ROWS_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.base.data)[j])
                                                               : static_cast<const float*>(a.base.data)[j]);
    if (a.grad.type == LIONCUB_ROWS_BF16)
        static_cast<__nv_bfloat16*>(a.grad.data)[j] = __float2bfloat16_rn(sum);
    else
        static_cast<float*>(a.grad.data)[j] = sum;
}

// How a row is spread over a team, and how many teams a block has.
struct Spread {
    int c, warps, teams;
    explicit Spread(int dim)
    {
        const int chunks = (dim + kChunk - 1) / kChunk;
        c = chunks == 1 ? 1 : chunks <= 2 * kBlockWarps ? 2 : 4;
        warps = (chunks + c - 1) / c;
        teams = kBlockWarps / warps;
    }
};

template <typename DT, typename GT, int SOURCE, int C, bool VEC>
cudaError_t launch_c(const NormGradArgs& a, int blocks, cudaStream_t s)
{
    const auto kernel = k_norm_grad<DT, GT, SOURCE, C, VEC>;
    const int ring = a.slots * a.slot_bytes * a.teams, columns = a.partial ? a.teams * a.dim * static_cast<int>(sizeof(float)) : 0;
    // the kernel's limit, the same for every call: calls of other threads launch by it too
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess)
        return e;
    return launch_programmatic(kernel, static_cast<unsigned>(blocks), a.warps * a.teams * 32, ring > columns ? ring : columns, s, a);
}

template <typename DT, typename GT, int SOURCE, bool VEC>
cudaError_t launch_s(const NormGradArgs& a, int c, int blocks, cudaStream_t s)
{
    switch (c) {
    case 1: return launch_c<DT, GT, SOURCE, 1, VEC>(a, blocks, s);
    case 2: return launch_c<DT, GT, SOURCE, 2, VEC>(a, blocks, s);
    default: return launch_c<DT, GT, SOURCE, 4, VEC>(a, blocks, s);
    }
}

template <typename DT, typename GT, bool VEC>
cudaError_t launch_t(const NormGradArgs& a, int c, int blocks, cudaStream_t s)
{
    if (a.packed.codes)
        return launch_s<DT, GT, kFromCodes, VEC>(a, c, blocks, s);
    if (!VEC || a.saved.type == LIONCUB_ROWS_F32)  // scalar moves go by the type that the launch gives
        return launch_s<DT, GT, kFromF32, VEC>(a, c, blocks, s);
    return launch_s<DT, GT, kFromBf16, VEC>(a, c, blocks, s);
}

}  // namespace

#ifdef LIONCUB_BOUNDS_CHECK
cudaError_t take_norm_grad_word(int* word) { return take_word(word); }
#endif

int norm_grad_blocks(int64_t n, int dim, int multiprocessors)
{
    const Spread spread(dim);
    const int64_t all = (n + spread.teams - 1) / spread.teams;
    return static_cast<int>(all < multiprocessors ? all : multiprocessors);
}

cudaError_t launch_norm_grad(NormGradArgs a, int blocks, bool vec, cudaStream_t s)
{
    if (a.n == 0)
        return cudaSuccess;
    const Spread spread(a.dim);
    a.warps = spread.warps;
    a.teams = spread.teams;
    // a slot: a row of each matrix, from a 16-byte boundary to one
    const auto room = [&](int size) { return (a.dim * size + 15 + 15) / 16 * 16; };
    const auto size_of = [](const TypedRows& m) { return m.type == LIONCUB_ROWS_BF16 ? 2 : 4; };
    a.at_saved = room(size_of(a.dout));
    a.at_residual = a.at_saved + room(a.packed.codes ? 1 : size_of(a.saved));
    a.slot_bytes = a.at_residual + (a.residual_grad.data ? room(size_of(a.residual_grad)) : 0);
    const int all = a.slot_bytes * a.teams, most = kRingBytes / all;
    a.slots = kRingWanted / all < 2 ? 2 : kRingWanted / all;
    a.slots = a.slots > most ? most : a.slots > kMaxSlots ? kMaxSlots : a.slots;
    static_assert(3 * (LIONCUB_NORM_MAX_DIM * 4 + 30) <= kRingBytes, "a row of every width has a slot");
    a.per_column = 1.0f / static_cast<float>(a.dim);
    if (!vec)
        return launch_t<float, float, false>(a, spread.c, blocks, s);
    const bool db = a.dout.type == LIONCUB_ROWS_BF16, gb = a.residual_grad.type == LIONCUB_ROWS_BF16;
    if (db)
        return gb ? launch_t<__nv_bfloat16, __nv_bfloat16, true>(a, spread.c, blocks, s) : launch_t<__nv_bfloat16, float, true>(a, spread.c, blocks, s);
    return gb ? launch_t<float, __nv_bfloat16, true>(a, spread.c, blocks, s) : launch_t<float, float, true>(a, spread.c, blocks, s);
}

cudaError_t launch_weight_grad(const WeightGradArgs& a, cudaStream_t s)
{
    return launch_programmatic(k_weight_grad, (a.dim + 31) / 32, kJoinWarps * 32, 0, s, a);
}

}  // namespace lc
