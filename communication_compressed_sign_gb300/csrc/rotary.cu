// rotary.cu -- rotary positions: each pair of columns (a, b) of a head turns by
// position * frequency,
//   (a, b) -> m * (a cos - b sin, a sin + b cos).
//
// Memory-bound.  The angle is the same for all heads of a place, so a thread
// takes the same columns of several heads and computes sines and cosines once.
// Angles are turns in 64-bit fixed point: position * turns-a-position wraps
// around by itself, which is the exact reduction that far positions need (in
// fp32 the angle of position 100000 would be off by 0.004).
#include <climits>

#include "block_device.cuh"

namespace lc {
namespace {

constexpr int kBlock = 256;

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

__device__ __forceinline__ float first_turned(float x, float y, float c, float s) { return fmaf(x, c, -__fmul_rn(y, s)); }
__device__ __forceinline__ float second_turned(float x, float y, float c, float s) { return fmaf(y, c, __fmul_rn(x, s)); }

// A thread's place, the item of each head that it has, and its share of heads.
struct Share {
    int64_t place, b;
    int item, group, s;
    bool on;
    __device__ __forceinline__ Share(const RotaryArgs& a, int items)
    {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
        const int64_t rest = quotient(t, items);
        item = static_cast<int>(t - rest * items);
        place = quotient(rest, a.groups);
        group = static_cast<int>(rest - place * a.groups);
        on = place < a.places;
        b = quotient(place, a.seq);
        s = static_cast<int>(place - b * a.seq);
    }
    __device__ __forceinline__ uint64_t position(const RotaryArgs& a) const
    {
        return static_cast<uint64_t>(a.positions ? index_at(a.positions, place, a.wide) : a.first + s);
    }
};

struct Head {
    int64_t in, out;
    const HeadsArgs* side;
    __device__ __forceinline__ Head(const RotaryArgs& a, const Share& t, int h)
    {
        const int second = h >= a.heads[0];
        side = &a.side[second];
        const int at = second ? h - a.heads[0] : h;
        in = t.b * side->in_batch + t.s * side->in_place + at * side->in_head;
        out = t.b * side->out_batch + t.s * side->out_place + at * side->out_head;
    }
};

// 8 columns a move.  Items: halves: pairs / 8 of two groups of 8 columns that
// turn together; interleaved: pairs / 4 of one group; then groups that are copied.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kBlock) k_rotary(const __grid_constant__ RotaryArgs a, const int turning, const int items)
{
    const Share t(a, items);
    wait_for_launch_before();
    if (!t.on)
        return;
    const int heads = a.heads[0] + a.heads[1];
    if (t.item >= turning) {
        const int col = 2 * a.pairs + (t.item - turning) * 8;
        for (int h = t.group; h < heads; h += a.groups) {
            const Head at(a, t, h);
            Group8<T> x;
            x.load(at.side->in, at.in + col);
            x.store(at.side->out, at.out + col);
        }
        return;
    }
    constexpr int N = INTERLEAVED ? 4 : 8;  // pairs
    const uint64_t position = t.position(a);
    float c[N], s[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
        angle_of(position, a.turns[t.item * N + k], a, c[k], s[k]);
    for (int h = t.group; h < heads; h += a.groups) {
        const Head at(a, t, h);
        if constexpr (INTERLEAVED) {
            const int col = t.item * 8;
            Group8<T> g;
            g.load(at.side->in, at.in + col);
            float x[8], y[8];
            g.unpack(x);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[2 * k] = first_turned(x[2 * k], x[2 * k + 1], c[k], s[k]);
                y[2 * k + 1] = second_turned(x[2 * k], x[2 * k + 1], c[k], s[k]);
            }
            g.pack(y);
            g.store(at.side->out, at.out + col);
        } else {
            const int col = t.item * 8;
            Group8<T> g, o;
            g.load(at.side->in, at.in + col);
            o.load(at.side->in, at.in + col + a.pairs);
            float x[8], y[8], u[8], v[8];
            g.unpack(x);
            o.unpack(y);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                u[k] = first_turned(x[k], y[k], c[k], s[k]);
                v[k] = second_turned(x[k], y[k], c[k], s[k]);
            }
            g.pack(u);
            o.pack(v);
            g.store(at.side->out, at.out + col);
            o.store(at.side->out, at.out + col + a.pairs);
        }
    }
}

// Any alignment: an item is a pair, or a column that is copied.
template <typename T>
__global__ void __launch_bounds__(kBlock) k_rotary_scalar(const __grid_constant__ RotaryArgs a, const int interleaved, const int items)
{
    const Share t(a, items);
    wait_for_launch_before();
    if (!t.on)
        return;
    const int heads = a.heads[0] + a.heads[1];
    if (t.item >= a.pairs) {
        const int col = a.pairs + t.item;
        for (int h = t.group; h < heads; h += a.groups) {
            const Head at(a, t, h);
            static_cast<T*>(at.side->out)[at.out + col] = static_cast<const T*>(at.side->in)[at.in + col];
        }
        return;
    }
    float c, s;
    angle_of(t.position(a), a.turns[t.item], a, c, s);
    const int one = interleaved ? 2 * t.item : t.item, two = interleaved ? one + 1 : one + a.pairs;
    for (int h = t.group; h < heads; h += a.groups) {
        const Head at(a, t, h);
        const T* in = static_cast<const T*>(at.side->in) + at.in;
        T* out = static_cast<T*>(at.side->out) + at.out;
        const float x = static_cast<float>(in[one]), y = static_cast<float>(in[two]);
        out[one] = static_cast<T>(first_turned(x, y, c, s));
        out[two] = static_cast<T>(second_turned(x, y, c, s));
    }
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, int type, bool interleaved, bool vec, cudaStream_t s)
{
    const int heads = a.heads[0] + a.heads[1];
    if (a.places == 0 || heads == 0)
        return cudaSuccess;
    const int rest = a.copy ? a.head_dim - 2 * a.pairs : 0;
    const int turning = vec ? (interleaved ? a.pairs / 4 : a.pairs / 8) : a.pairs;
    const int items = turning + (vec ? rest / 8 : rest);
    // About four heads a thread, fewer while threads are too few for all multiprocessors.
    const int64_t lanes = a.places * items;
    int64_t groups = (heads + 3) / 4;
    const int64_t wanted = (int64_t(152) * 1024 + lanes - 1) / lanes;
    groups = groups < wanted ? wanted : groups;
    a.groups = static_cast<int32_t>(groups < heads ? groups : heads);
    const int64_t blocks = (lanes * a.groups + kBlock - 1) / kBlock;
    if (blocks > INT_MAX)
        return cudaErrorInvalidConfiguration;
    const unsigned n = static_cast<unsigned>(blocks);
    if (!vec)
        return type == LIONCUB_ROWS_BF16 ? launch_programmatic(k_rotary_scalar<__nv_bfloat16>, n, kBlock, 0, s, a, int(interleaved), items)
                                         : launch_programmatic(k_rotary_scalar<float>, n, kBlock, 0, s, a, int(interleaved), items);
    if (type == LIONCUB_ROWS_BF16)
        return interleaved ? launch_programmatic(k_rotary<__nv_bfloat16, true>, n, kBlock, 0, s, a, turning, items)
                           : launch_programmatic(k_rotary<__nv_bfloat16, false>, n, kBlock, 0, s, a, turning, items);
    return interleaved ? launch_programmatic(k_rotary<float, true>, n, kBlock, 0, s, a, turning, items)
                       : launch_programmatic(k_rotary<float, false>, n, kBlock, 0, s, a, turning, items);
}

}  // namespace lc
