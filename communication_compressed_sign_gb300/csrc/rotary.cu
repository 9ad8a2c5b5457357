// rotary.cu -- rotary positions: each pair of columns (a, b) of a head turns by
// position * frequency,
//   (a, b) -> m * (a cos - b sin, a sin + b cos).
//
// Memory-bound.  The angle is the same for all heads of a place, so a block takes
// a few places, works out their cosines and sines once into shared memory, and
// then walks over the places' heads in the order of memory.  (A thread with the
// same columns of several heads keeps its angles in registers, but then all blocks
// read the same few heads of every place at a time: 192 to 275 us by how many
// heads, where this took 196 whatever the layout.  The first items loaded before
// the angles are worked out: 202, and nothing gained by small calls.)  Queries and
// keys are one list of heads, so that a block waits for memory as seldom as it can: one
// after the other 8 places took 2.4 us, 45708 x 12 heads of 80 60 us.
// Measured: 65536 places, 40 heads of 128 bf16 193 us (6.95 TB/s); 8192 places, 24
// heads of 64 out of a fused product 10.9 us (4.6 TB/s; two waves); 8 places 1.8 us.
// Heads of 80 with 40 interleaved columns, 4 elements at a time, 7.0 us for 8192 x
// 10 (3.7 TB/s); with 20, 45708 x 12 heads: halves, 2 at a time, 38 us (4.6 TB/s), and
// interleaved, 4 at a time, 35.6.
// Angles are turns in 64-bit fixed point: position * turns-a-position wraps
// around by itself, which is the exact reduction that far positions need (in
// fp32 the angle of position 100000 would be off by 0.004).
#include <algorithm>
#include <climits>

#include "block_device.cuh"

namespace lc {
namespace {

// Threads of a block, and its places: as many as make up kBytes of heads, kMaxPlaces at most.
// By 9, 12 and 16 KB: 8192 places of 24 x 64 bf16 12.0, 10.9, 12.4 us, fp32 17.0, 17.0, 18.1;
// 65536 of 40 x 128 bf16 202, 193, 193.  Blocks of 192 threads 11.0, 17.3, 195; of 256 11.7,
// 16.9, 195 (4 places each).
constexpr int kBlock = 128;
constexpr int kMaxPlaces = 8;
constexpr int kBytes = 12288;

// cos and sin of a position's angle.  The nearest quarter turn is taken off in
// whole numbers, so what is left is at most an eighth of a turn.
__device__ __forceinline__ void angle_of(uint64_t position, uint64_t turns, const RotaryArgs& a, float& c, float& s)
{
    const int32_t phase = static_cast<int32_t>((position * turns) >> 32);  // of a turn, in units of 2^-32
    const int32_t quarter = static_cast<int32_t>(static_cast<uint32_t>(phase) + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(phase) - (static_cast<uint32_t>(quarter) << 30));
    float rs, rc;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &rs, &rc);
    c = quarter & 1 ? rs : rc;
    s = quarter & 1 ? rc : rs;
    // quarters 0, 1, 2, 3: (c, s), (-s, c), (-c, -s), (s, -c)
    if ((quarter + 1) & 2)
        c = -c;
    if (quarter & 2)
        s = -s;
    c = __fmul_rn(c, a.cos_factor);
    s = __fmul_rn(s, a.sin_factor);
}

// What a thread moves at once.  16-byte moves: twice 8 columns, half of the rotated
// ones apart, or 8 columns that are copied.
template <typename T, bool INTERLEAVED>
struct WideItem {
    static constexpr int kPairs = 8, kCopied = 8;
    Group8<T> g[2];
    int first, second;  // columns; second < 0: to be copied

    __device__ __forceinline__ void place(const RotaryArgs& a, int item, int turning)
    {
        first = item < turning ? item * 8 : 2 * a.pairs + (item - turning) * 8;
        second = item < turning ? first + a.pairs : -1;
    }
    // checked builds: whether move k (of two) is within a head (unless there is none), and where it begins
    static constexpr int kMoves = 2, kMove = 8;
    __device__ __forceinline__ int move_at(const RotaryArgs&, int k) const { return k ? second : first; }
    __device__ __forceinline__ bool has_move(int k) const { return !k || second >= 0; }
    // ... and the last of its pairs' angles, or -1
    __device__ __forceinline__ int last_pair(const RotaryArgs& a, int item) const
    {
        return second < 0 ? -1 : INTERLEAVED ? item * 4 + a.pairs / 2 + 3 : item * 8 + 7;
    }
    __device__ __forceinline__ void load(const RotaryArgs&, const T* in)
    {
        load(g[0], in + first);
        if (second >= 0)
            load(g[1], in + second);
    }
    __device__ __forceinline__ void turn(const float* cosines, const float* sines, int item, int pairs)
    {
        if (second < 0)
            return;
        float u[8], v[8];
        g[0].unpack(u);
        g[1].unpack(v);
        // four pairs a round: of either move (interleaved), or half of both
        const int at = INTERLEAVED ? item * 4 : item * 8, next = INTERLEAVED ? pairs / 2 : 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 c = *reinterpret_cast<const float4*>(cosines + at + h * next), s = *reinterpret_cast<const float4*>(sines + at + h * next);
            if constexpr (INTERLEAVED) {  // (x c - y s, y c + x s)
                float(&y)[8] = h ? v : u;
                const float ck[4] = {c.x, c.y, c.z, c.w}, sk[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 w = pair_of(y, k);
                    set_pair(y, k, fma2(make_float2(w.y, w.x), make_float2(-sk[k], sk[k]), mul2(w, both(ck[k]))));
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 ck = k ? make_float2(c.z, c.w) : make_float2(c.x, c.y), sk = k ? make_float2(s.z, s.w) : make_float2(s.x, s.y);
                    const float2 p = pair_of(u, 2 * h + k), q = pair_of(v, 2 * h + k);
                    set_pair(u, 2 * h + k, fma2(q, make_float2(-sk.x, -sk.y), mul2(p, ck)));
                    set_pair(v, 2 * h + k, fma2(p, sk, mul2(q, ck)));
                }
            }
        }
        g[0].pack(u);
        g[1].pack(v);
    }
    __device__ __forceinline__ void store(const RotaryArgs&, T* out) const
    {
        store(g[0], out + first);
        if (second >= 0)
            store(g[1], out + second);
    }
    // fp32 by 32 bytes where they allow: 1024 places of 24 x 64 3.0 us by 16, 2.65 so
    static __device__ __forceinline__ void load(Group8<T>& v, const T* p)
    {
        if constexpr (sizeof(T) == 4)
            load8(p, v);
        else
            v.load(p, 0);
    }
    static __device__ __forceinline__ void store(const Group8<T>& v, T* p)
    {
        if constexpr (sizeof(T) == 4) {
            float x[8];
            v.unpack(x);
            store8(p, x);
        } else {
            v.store(p, 0);
        }
    }
};

// Other alignments: four pairs, or eight columns that are copied, MOVE elements at a time.
template <typename T, bool INTERLEAVED, int MOVE>
struct NarrowItem {
    static constexpr int kPairs = 4, kCopied = 8;
    struct alignas(MOVE * sizeof(T)) Move {
        T x[MOVE];
    };
    Move m[8 / MOVE];  // elements in the order of columns: pairs lie 4 apart, or side by side
    int first, count;  // a column, or a pair, and how many are left from it
    bool copied;

    __device__ __forceinline__ void place(const RotaryArgs& a, int item, int turning)
    {
        copied = item >= turning;
        first = copied ? 2 * a.pairs + (item - turning) * 8 : item * 4;
        count = copied ? a.head_dim - first : a.pairs - first;
    }
    __device__ __forceinline__ int column(const RotaryArgs& a, int k) const
    {
        return copied ? first + k : INTERLEAVED ? 2 * first + k : first + (k & 3) + (k >> 2) * a.pairs;
    }
    __device__ __forceinline__ bool has(int k) const { return (copied ? k : INTERLEAVED ? k >> 1 : k & 3) < count; }
    static constexpr int kMoves = 8 / MOVE, kMove = MOVE;
    __device__ __forceinline__ int move_at(const RotaryArgs& a, int k) const { return column(a, k * MOVE); }
    __device__ __forceinline__ bool has_move(int k) const { return has(k * MOVE); }
    __device__ __forceinline__ int last_pair(const RotaryArgs&, int item) const { return copied ? -1 : item * 4 + min(count, 4) - 1; }
    __device__ __forceinline__ T& element(int k) { return m[k / MOVE].x[k % MOVE]; }
    __device__ __forceinline__ void load(const RotaryArgs& a, const T* in)
    {
#pragma unroll
        for (int k = 0; k < 8; k += MOVE)
            if (has(k))
                m[k / MOVE] = *reinterpret_cast<const Move*>(in + column(a, k));
    }
    __device__ __forceinline__ void turn(const float* cosines, const float* sines, int item, int)
    {
        if (copied)
            return;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < count) {
                T &one = element(INTERLEAVED ? 2 * k : k), &two = element(INTERLEAVED ? 2 * k + 1 : k + 4);
                const float u = static_cast<float>(one), v = static_cast<float>(two), c = cosines[item * 4 + k], s = sines[item * 4 + k];
                one = static_cast<T>(fmaf(u, c, -__fmul_rn(v, s)));
                two = static_cast<T>(fmaf(v, c, __fmul_rn(u, s)));
            }
    }
    __device__ __forceinline__ void store(const RotaryArgs& a, T* out) const
    {
#pragma unroll
        for (int k = 0; k < 8; k += MOVE)
            if (has(k))
                *reinterpret_cast<Move*>(out + column(a, k)) = m[k / MOVE];
    }
};

// Eight columns that are copied, four at a time.
template <typename T>
struct CopiedItem {
    struct alignas(4 * sizeof(T)) Move {
        T x[4];
    };
    Move m[2];
    int first, count;

    __device__ __forceinline__ void place(const RotaryArgs& a, int item, int)
    {
        first = 2 * a.pairs + item * 8;
        count = a.head_dim - first;
    }
    static constexpr int kMoves = 2, kMove = 4;
    __device__ __forceinline__ int move_at(const RotaryArgs&, int k) const { return first + 4 * k; }
    __device__ __forceinline__ bool has_move(int k) const { return 4 * k < count; }
    __device__ __forceinline__ int last_pair(const RotaryArgs&, int) const { return -1; }
    __device__ __forceinline__ void load(const RotaryArgs&, const T* in)
    {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (4 * k < count)
                m[k] = *reinterpret_cast<const Move*>(in + first + 4 * k);
    }
    __device__ __forceinline__ void turn(const float*, const float*, int, int) {}
    __device__ __forceinline__ void store(const RotaryArgs&, T* out) const
    {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (4 * k < count)
                *reinterpret_cast<Move*>(out + first + 4 * k) = m[k];
    }
};

template <typename T, bool INTERLEAVED, int MOVE>
using ItemOf = std::conditional_t<MOVE == 8, WideItem<T, INTERLEAVED>, NarrowItem<T, INTERLEAVED, MOVE>>;

// n / d by a product, for n * d < 2^32; a block whose numbers are larger divides.
struct Divisor {
    uint32_t d, magic;  // magic 0: divide
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return magic ? __umulhi(n, magic) : n / d; }
};
Divisor divisor(uint32_t d, uint64_t largest) { return {d, d > 1 && largest * d < (1ull << 32) ? static_cast<uint32_t>((1ull << 32) / d + 1) : 0}; }

// Where the heads of a place are, of either side.
template <typename T>
struct Place {
    const T* in[2];
    T* out[2];
};

// Checked builds: whether an item's moves of a head lie in it and in its matrices, on boundaries
// of their size, and its pairs have angles.
template <typename Item, typename T>
__device__ __forceinline__ bool item_ok(const RotaryArgs& a, const Item& x, int item, int place, int places, int side, int head, const T* in,
                                        const T* out)
{
#ifdef LIONCUB_BOUNDS_CHECK
    const HeadsArgs& s = a.side[side];
    bool ok = place < places && places <= kMaxPlaces && head >= 0 && head < a.heads[side] && x.last_pair(a, item) < a.pairs;
    for (int k = 0; k < Item::kMoves; ++k)
        if (x.has_move(k)) {
            const int at = x.move_at(a, k);
            constexpr uintptr_t kAlign = Item::kMove == 8 ? 16 : Item::kMove * sizeof(T);
            ok = ok && at >= 0 && at + Item::kMove <= a.head_dim && in >= s.in && out >= s.out &&
                 reinterpret_cast<const char*>(in + at + Item::kMove) <= s.in_end &&
                 reinterpret_cast<const char*>(out + at + Item::kMove) <= s.out_end && reinterpret_cast<uintptr_t>(in + at) % kAlign == 0 &&
                 reinterpret_cast<uintptr_t>(out + at) % kAlign == 0;
        }
    return access_ok(ok);
#else
    return true;
#endif
}

// The items of the heads of some places, of both sides, over the block's threads.
template <typename Item, typename T>
__device__ __forceinline__ void walk(const RotaryArgs& a, int places, const Place<T>* at, const float* cosines, const float* sines,
                                     const Divisor& items, const Divisor& heads, int turning)
{
    constexpr int kUnits = 2;  // items of a thread, whose loads are in flight together
    const uint32_t units = places * heads.d * items.d;
    for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kUnits * kBlock) {
        Item x[kUnits];
        uint32_t item[kUnits], p[kUnits];
        T* out[kUnits];
        bool ok[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const uint32_t unit = u0 + u * kBlock;
            if (unit < units) {
                const uint32_t head = items.of(unit);  // of all places
                item[u] = unit - head * items.d;
                p[u] = heads.of(head);
                uint32_t h = head - p[u] * heads.d;
                const bool side = h >= a.heads[0];
                h -= side ? a.heads[0] : 0;
                out[u] = at[p[u]].out[side] + h * (side ? a.side[1].out_head : a.side[0].out_head);
                x[u].place(a, item[u], turning);
                const T* in = at[p[u]].in[side] + h * (side ? a.side[1].in_head : a.side[0].in_head);
                ok[u] = item_ok(a, x[u], item[u], p[u], places, side, h, in, out[u]);
                if (ok[u])
                    x[u].load(a, in);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            if (u0 + u * kBlock < units && (!kBoundsCheck || ok[u])) {
                x[u].turn(cosines + p[u] * a.pairs, sines + p[u] * a.pairs, item[u], a.pairs);
                x[u].store(a, out[u]);
            }
    }
}

// Checked builds: whether a place's pair has its cosine and sine in shared memory.
__device__ __forceinline__ bool angles_ok(int all, int i)
{
#ifdef LIONCUB_BOUNDS_CHECK
    uint32_t bytes;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(bytes));
    return access_ok(i < all && 2 * all * sizeof(float) <= bytes);
#else
    return true;
#endif
}

// APART: columns that are copied are walked over by themselves (copied: their items).
template <typename T, bool INTERLEAVED, int MOVE, bool APART>
__global__ void __launch_bounds__(kBlock, 8) k_rotary(const __grid_constant__ RotaryArgs a, const int turning, const Divisor items,
                                                   const Divisor copied, const Divisor heads, const int block_places)
{
    using Item = ItemOf<T, INTERLEAVED, MOVE>;
    extern __shared__ __align__(16) float cosines[];  // of each place and pair; then the sines
    __shared__ Place<T> at[kMaxPlaces];
    __shared__ int64_t positions[kMaxPlaces];
    float* sines = cosines + block_places * a.pairs;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * block_places;
    const int places = static_cast<int>(min(a.places - first, static_cast<int64_t>(block_places)));
    if (a.positions)
        wait_for_launch_before();
    if (threadIdx.x < places && access_ok(places <= kMaxPlaces && first + places <= a.places)) {
        const int64_t place = first + threadIdx.x, b = quotient(place, a.seq), s = place - b * a.seq;
        positions[threadIdx.x] = a.positions ? index_at(a.positions, place, a.wide) : a.first + s;
        for (int k = 0; k < 2; ++k) {
            at[threadIdx.x].in[k] = static_cast<const T*>(a.side[k].in) + (b * a.side[k].in_batch + s * a.side[k].in_place);
            at[threadIdx.x].out[k] = static_cast<T*>(a.side[k].out) + (b * a.side[k].out_batch + s * a.side[k].out_place);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < places * a.pairs; i += kBlock) {
        const int p = i / a.pairs;
        if (!angles_ok(block_places * a.pairs, i))
            continue;
        angle_of(static_cast<uint64_t>(positions[p]), a.turns[i - p * a.pairs], a, cosines[i], sines[i]);
    }
    if (!a.positions)  // the angles need nothing of the launches before
        wait_for_launch_before();
    __syncthreads();
    walk<Item, T>(a, places, at, cosines, sines, items, heads, turning);
    if constexpr (APART)
        walk<CopiedItem<T>, T>(a, places, at, cosines, sines, copied, heads, 0);
}

template <typename T, bool INTERLEAVED, int MOVE, bool APART = false>
cudaError_t launch_t(const RotaryArgs& a, cudaStream_t s)
{
    const int rest = a.copy ? a.head_dim - 2 * a.pairs : 0;
    using Item = ItemOf<T, INTERLEAVED, MOVE>;
    const int turning = (a.pairs + Item::kPairs - 1) / Item::kPairs, copied = (rest + Item::kCopied - 1) / Item::kCopied;
    const int items = turning + copied;
    // Places of a block: kBytes of heads, but fewer while that leaves less than four blocks a
    // multiprocessor.
    const int64_t heads = int64_t(a.heads[0]) + a.heads[1], of_place = heads * a.head_dim * sizeof(T);
    int64_t places = std::min<int64_t>(kMaxPlaces, (kBytes + of_place - 1) / of_place);
    places = std::max<int64_t>(1, std::min<int64_t>(places, a.places / (152 * 4)));
    const int64_t blocks = (a.places + places - 1) / places;
    const int64_t most = places * heads * items;
    if (blocks > INT_MAX || most > INT_MAX)
        return cudaErrorInvalidConfiguration;
    return launch_programmatic(k_rotary<T, INTERLEAVED, MOVE, APART>, static_cast<unsigned>(blocks), kBlock,
                               places * a.pairs * 2 * sizeof(float), s, a, turning, divisor(APART ? turning : items, most),
                               divisor(copied, most), divisor(static_cast<uint32_t>(heads), most), static_cast<int>(places));
}

template <typename T, bool INTERLEAVED>
cudaError_t launch_l(const RotaryArgs& a, int move, bool copy_by_four, cudaStream_t s)
{
    // Columns that are copied go by themselves, four at a time, unless all are moved by eight:
    // warps whose lanes do either do both.  45708 x 12 heads of 80, 20 columns in halves 66.6 us
    // among one another, 60.5 apart; interleaved 52.5, 36.5.
    if (copy_by_four && a.copy && a.head_dim > 2 * a.pairs) {
        if (move == 4)
            return launch_t<T, INTERLEAVED, 4, true>(a, s);
        if constexpr (!INTERLEAVED)
            if (move == 2)
                return launch_t<T, INTERLEAVED, 2, true>(a, s);
    }
    switch (move) {
    case 8: return launch_t<T, INTERLEAVED, 8>(a, s);
    case 4: return launch_t<T, INTERLEAVED, 4>(a, s);
    case 2: return launch_t<T, INTERLEAVED, 2>(a, s);
    default: return launch_t<T, INTERLEAVED, 1>(a, s);
    }
}

}  // namespace

#ifdef LIONCUB_BOUNDS_CHECK
cudaError_t take_rotary_word(int* word) { return take_word(word); }
#endif

cudaError_t launch_rotary(const RotaryArgs& a, int type, bool interleaved, int move, bool copy_by_four, cudaStream_t s)
{
    if (a.places == 0 || a.heads[0] + a.heads[1] == 0)
        return cudaSuccess;
    if (type == LIONCUB_ROWS_BF16)
        return interleaved ? launch_l<__nv_bfloat16, true>(a, move, copy_by_four, s) : launch_l<__nv_bfloat16, false>(a, move, copy_by_four, s);
    return interleaved ? launch_l<float, true>(a, move, copy_by_four, s) : launch_l<float, false>(a, move, copy_by_four, s);
}

}  // namespace lc
