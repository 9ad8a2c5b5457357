// rotary.cu -- rotary positions: each pair of columns (a, b) of a head turns by
// position * frequency,
//   (a, b) -> m * (a cos - b sin, a sin + b cos).
//
// Memory-bound.  The angle is the same for all heads of a place, so a block takes
// a few places, works out their cosines and sines once into shared memory, and
// then walks over the places' heads in the order of memory.  (A thread with the
// same columns of several heads keeps its angles in registers, but then all blocks
// read the same few heads of every place at a time: 192 to 275 us by how many
// heads, where this takes 196 whatever the layout.  The first items loaded before
// the angles are worked out: 202, and nothing gained by small calls.)
// Measured: 65536 places, 40 heads of 128 bf16 196 us (6.8 TB/s); 8192 places, 24
// heads of 64 out of a fused product 11.3 us (4.5 TB/s; two waves); 8 places 2.4 us.
// Heads of 80 with 40 interleaved columns, 4 elements at a time, 8.4 us for 8192 x
// 10 (3.0 TB/s); with 20, 45708 x 12 heads: halves, 2 at a time, 67 us (2.6 TB/s), and
// interleaved, 4 at a time, 58 (3.0 TB/s).
// Angles are turns in 64-bit fixed point: position * turns-a-position wraps
// around by itself, which is the exact reduction that far positions need (in
// fp32 the angle of position 100000 would be off by 0.004).
#include <algorithm>
#include <climits>

#include "block_device.cuh"

namespace lc {
namespace {

// Threads and places of a block.  8192 places of 24 x 64 and 65536 of 40 x 128: blocks of
// 256 with 2, 4, 6, 8 and 14 places 19.8, 14.2, 13.0, 11.6 and 14.5 us (fewer repeat the
// start, more leave SMs idle) and 215, 196, 195, 196 and 195; of 128 with 4 11.3 and 196,
// with 8 14.5 and 196.
constexpr int kBlock = 128;
constexpr int kMaxPlaces = 4;
constexpr int kItems = 8;      // of a thread, about, where there are many places

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
    __device__ __forceinline__ void load(const RotaryArgs&, const T* in)
    {
        g[0].load(in, first);
        if (second >= 0)
            g[1].load(in, second);
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
        g[0].store(out, first);
        if (second >= 0)
            g[1].store(out, second);
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

template <typename T, bool INTERLEAVED, int MOVE>
using ItemOf = std::conditional_t<MOVE == 8, WideItem<T, INTERLEAVED>, NarrowItem<T, INTERLEAVED, MOVE>>;

// n / d by a product, for n * d < 2^32; a block whose numbers are larger divides.
struct Divisor {
    uint32_t d, magic;  // magic 0: divide
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return magic ? __umulhi(n, magic) : n / d; }
};
Divisor divisor(uint32_t d, uint64_t largest) { return {d, d > 1 && largest * d < (1ull << 32) ? static_cast<uint32_t>((1ull << 32) / d + 1) : 0}; }

template <typename T, bool INTERLEAVED, int MOVE>
__global__ void __launch_bounds__(kBlock, 8) k_rotary(const __grid_constant__ RotaryArgs a, const int turning, const Divisor items,
                                                   const Divisor heads0, const Divisor heads1, const int block_places)
{
    constexpr int kUnits = 2;  // items of a thread, whose loads are in flight together
    using Item = ItemOf<T, INTERLEAVED, MOVE>;
    extern __shared__ __align__(16) float cosines[];  // of each place and pair; then the sines
    __shared__ int64_t starts[kMaxPlaces][4];         // of a place: elements to its in and out of either side
    __shared__ int64_t positions[kMaxPlaces];
    float* sines = cosines + block_places * a.pairs;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * block_places;
    const int places = static_cast<int>(min(a.places - first, static_cast<int64_t>(block_places)));
    if (a.positions)
        wait_for_launch_before();
    if (threadIdx.x < places) {
        const int64_t place = first + threadIdx.x, b = quotient(place, a.seq), s = place - b * a.seq;
        positions[threadIdx.x] = a.positions ? index_at(a.positions, place, a.wide) : a.first + s;
        for (int k = 0; k < 2; ++k) {
            starts[threadIdx.x][2 * k] = b * a.side[k].in_batch + s * a.side[k].in_place;
            starts[threadIdx.x][2 * k + 1] = b * a.side[k].out_batch + s * a.side[k].out_place;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < places * a.pairs; i += kBlock) {
        const int p = i / a.pairs;
        angle_of(static_cast<uint64_t>(positions[p]), a.turns[i - p * a.pairs], a, cosines[i], sines[i]);
    }
    if (!a.positions)  // the angles need nothing of the launches before
        wait_for_launch_before();
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const Divisor heads = k ? heads1 : heads0;
        const uint32_t units = places * heads.d * items.d;
        const T* in = static_cast<const T*>(a.side[k].in);
        T* out = static_cast<T*>(a.side[k].out);
        const int64_t in_head = a.side[k].in_head, out_head = a.side[k].out_head;
        for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kUnits * kBlock) {
            Item x[kUnits];
            uint32_t item[kUnits], p[kUnits], h[kUnits];
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const uint32_t unit = u0 + u * kBlock;
                if (unit < units) {
                    const uint32_t head = items.of(unit);  // of all places
                    item[u] = unit - head * items.d;
                    p[u] = heads.of(head);
                    h[u] = head - p[u] * heads.d;
                    x[u].place(a, item[u], turning);
                    x[u].load(a, in + (starts[p[u]][2 * k] + h[u] * in_head));
                }
            }
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
                if (u0 + u * kBlock < units) {
                    x[u].turn(cosines + p[u] * a.pairs, sines + p[u] * a.pairs, item[u], a.pairs);
                    x[u].store(a, out + (starts[p[u]][2 * k + 1] + h[u] * out_head));
                }
        }
    }
}

template <typename T, bool INTERLEAVED, int MOVE>
cudaError_t launch_t(const RotaryArgs& a, cudaStream_t s)
{
    const int rest = a.copy ? a.head_dim - 2 * a.pairs : 0;
    using Item = ItemOf<T, INTERLEAVED, MOVE>;
    const int turning = (a.pairs + Item::kPairs - 1) / Item::kPairs, items = turning + (rest + Item::kCopied - 1) / Item::kCopied;
    // Places of a block: about kItems items for each of its threads, fewer while that leaves
    // less than four blocks a multiprocessor.
    const int64_t of_place = int64_t(a.heads[0] + a.heads[1]) * items;
    int64_t places = std::min<int64_t>(kMaxPlaces, (kItems * kBlock + of_place - 1) / of_place);
    places = std::max<int64_t>(1, std::min<int64_t>(places, a.places / (152 * 4)));
    const int64_t blocks = (a.places + places - 1) / places;
    const int64_t most = places * std::max(a.heads[0], a.heads[1]) * items;
    if (blocks > INT_MAX || most > INT_MAX)
        return cudaErrorInvalidConfiguration;
    return launch_programmatic(k_rotary<T, INTERLEAVED, MOVE>, static_cast<unsigned>(blocks), kBlock, places * a.pairs * 2 * sizeof(float), s, a,
                               turning, divisor(items, most), divisor(a.heads[0], most), divisor(a.heads[1], most), static_cast<int>(places));
}

template <typename T, bool INTERLEAVED>
cudaError_t launch_l(const RotaryArgs& a, int move, cudaStream_t s)
{
    switch (move) {
    case 8: return launch_t<T, INTERLEAVED, 8>(a, s);
    case 4: return launch_t<T, INTERLEAVED, 4>(a, s);
    case 2: return launch_t<T, INTERLEAVED, 2>(a, s);
    default: return launch_t<T, INTERLEAVED, 1>(a, s);
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int type, bool interleaved, int move, cudaStream_t s)
{
    if (a.places == 0 || a.heads[0] + a.heads[1] == 0)
        return cudaSuccess;
    if (type == LIONCUB_ROWS_BF16)
        return interleaved ? launch_l<__nv_bfloat16, true>(a, move, s) : launch_l<__nv_bfloat16, false>(a, move, s);
    return interleaved ? launch_l<float, true>(a, move, s) : launch_l<float, false>(a, move, s);
}

}  // namespace lc
