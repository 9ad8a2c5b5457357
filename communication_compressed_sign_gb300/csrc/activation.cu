// activation.cu -- f(x) (* up) and its gradient, 8-bit codes of matrices, and
// what codes stand for:
//   f(x) = x * s(z), s(z) = 1 / (1 + exp(-z)), z = x or 2 sqrt(2 / pi) (x + 0.044715 x^3),
//   f'(x) = s + x * s * (1 - s) * z'.
//
// Memory-bound: each element is read and written once; groups of columns that
// share a scale lie inside a warp's chunk of 256 columns, so their maxima need
// shuffles only.  Dense matrices whose rows are whole groups are one long row.
// Measured: SiLU, gated, 16384 x 8192 bf16, saved in int8, forward and backward 366
// us (6.6 TB/s, 98 % of a measured copy; the forward pass issues 78 % of its
// cycles), GELU without a gate 204 us (6.6 TB/s); 16384 x 4096 bf16 packed and
// unpacked 63.5 us (6.4 TB/s; packing issues 75 %); 4925 x 771 fp32 out of rows of
// 776 9.1 us (3.4 TB/s, scalar moves).
#include <algorithm>
#include <climits>

#include "block_device.cuh"

namespace lc {
namespace {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;
// Chunks of a warp, whose loads are in flight together.  An activation by scalar
// moves has too few registers for two (4907 x 771 bf16 with two inputs saved in 8
// bits, both ways: 28.4 us, 27.0 with one); packing by them has not (9.9 with one, 9.4).
template <int KIND, bool VEC>
constexpr int kUnitsOf = VEC || KIND == kIdentity ? 2 : 1;

// Blocks that an SM should have room for, which caps the registers.  bf16 both ways, by 4, 5
// and 6 blocks: SiLU, gated, 16384 x 8192 387, 370, 382 us; GELU 218, 205, 199; by
// scalar moves 4907 x 771 x 2 (1, 5, 6) 28.6, 26.1, 24.2, 8192 x 3905 x 2 163, 155, 145.
// The caps hold for fp32 too, whose gradient from matrices spills 240 to 312 bytes a
// thread by them (it was not measured by others): SiLU, gated, 8192 x 8192 226 us,
// 6.0 TB/s; GELU 116 us, 6.9 TB/s.
template <bool VEC>
constexpr int kBlocks = VEC ? 5 : 6;

__device__ __forceinline__ float exp2_approx(float x)  // off by at most 2 units in the last place
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_approx(float x)  // off by at most one unit; 0 for x above 2^126
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// f(x) and, where it is wanted, f'(x), of a pair.  s = 1 / (1 + 2^w) with w = -z log2(e).
template <int KIND, bool SLOPE>
__device__ __forceinline__ void value_and_slope(float2 x, float2& f, float2& slope)
{
    constexpr double kLog2e = 1.4426950408889634, kTwice = 1.5957691216057308, kCube = 0.044715;  // kTwice: 2 sqrt(2 / pi)
    float2 w, square;
    if constexpr (KIND == LIONCUB_ACTIVATION_GELU) {
        square = mul2(x, x);
        w = mul2(x, fma2(square, both(static_cast<float>(-kTwice * kCube * kLog2e)), both(static_cast<float>(-kTwice * kLog2e))));
    } else {
        w = mul2(x, both(static_cast<float>(-kLog2e)));
    }
    const float2 below = add2(make_float2(exp2_approx(w.x), exp2_approx(w.y)), both(1.0f));
    const float2 s = make_float2(reciprocal_approx(below.x), reciprocal_approx(below.y));
    f = mul2(x, s);
    if constexpr (SLOPE) {
        const float2 t = mul2(f, fma2(s, both(-1.0f), both(1.0f)));
        if constexpr (KIND == LIONCUB_ACTIVATION_GELU) {
            // s is 0 or 1 long before the square could overflow, and t is then 0
            square = make_float2(fminf(square.x, 1e30f), fminf(square.y, 1e30f));
            slope = fma2(t, fma2(square, both(static_cast<float>(3 * kTwice * kCube)), both(static_cast<float>(kTwice))), s);
        } else {
            slope = add2(t, s);
        }
    }
}

// How the work is cut.  A warp has kUnits neighbouring chunks of a row, which has
// `spans` times as many; or, where that would leave lanes idle, each lane has groups
// of 8 columns by itself, of which a row has `lanes` (0: not), so that a warp
// may have several rows.
struct Cut {
    int64_t spans;
    int32_t lanes;
};

template <int kUnits, bool VEC, bool LANES>
struct Units {
    int64_t row[kUnits];
    Columns<VEC> cols[kUnits];
    bool on[kUnits];  // the warp has something to do
    __device__ __forceinline__ Units(int64_t rows, int64_t width, const Cut& cut)
    {
        const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
        const int lane = threadIdx.x & 31;
        if constexpr (LANES) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int64_t first = (unit * kUnits + u) * 32;
                row[u] = quotient(first + lane, cut.lanes);
                const bool there = row[u] < rows;
                cols[u].at = there ? (first + lane - row[u] * cut.lanes) * 8 : 0;
                cols[u].count = there ? 8 : 0;
                row[u] = there ? row[u] : 0;
                on[u] = first < rows * cut.lanes;
            }
        } else {
            const int64_t r = rows == 1 ? 0 : quotient(unit, static_cast<int>(cut.spans));
            const int64_t first = r < rows ? (unit - r * cut.spans) * (kUnits * kChunk) : width;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                row[u] = r;
                cols[u] = Columns<VEC>(first + u * kChunk, lane, width);
                on[u] = first + u * kChunk < width;
            }
        }
    }
};

// The scales of up to four groups that a lane belongs to, one of each of its chunks
// and matrices: a group has four lanes at least, so each works out one (a quotient is
// most of the work) and the others take it from there.  Each lane by itself: the
// gated 16384 x 8192 above 371.7 us (366.2 so), 16384 x 4096 packed only, by two chunks
// a warp, 67.3 (66.6).
template <int N>
struct SharedScales {
    float inv[N];  // negative: the group stands for NaN
    float scale;   // of number lane % N
    __device__ __forceinline__ SharedScales(const uint32_t (&largest)[N], const PackedRows* const (&to)[N], int lane)
    {
        static_assert(N == 1 || N == 2 || N == 4, "a power of two, and no more than a group's lanes");
        const int pick = lane & (N - 1);
        uint32_t m = largest[0];
        int e4m3 = to[0]->e4m3;
#pragma unroll
        for (int k = 1; k < N; ++k) {
            m = pick == k ? largest[k] : m;
            e4m3 = pick == k ? to[k]->e4m3 : e4m3;
        }
        const GroupScale s(m, e4m3);
        scale = s.scale;
        const float mine = s.bad ? -1.0f : s.inv;
#pragma unroll
        for (int k = 0; k < N; ++k)
            inv[k] = __shfl_sync(kAll, mine, (lane & ~(N - 1)) | k);
    }
};

template <typename T, int KIND, bool VEC, bool LANES, int kUnits = kUnitsOf<KIND, VEC>>
__global__ void __launch_bounds__(kBlock, kBlocks<VEC>) k_activation(const __grid_constant__ ActivationArgs a, const Cut cut)
{
    const Units<kUnits, VEC, LANES> u(a.rows, a.cols, cut);
    const int lane = threadIdx.x & 31;
    wait_for_launch_before();
    if (!u.on[0])
        return;
    Chunk<T, VEC> vx[kUnits], vup[kUnits];
    const bool gated = KIND != kIdentity && a.up.data;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        load_row(vx[i], u.cols[i], a.x, u.row[i]);
        if (gated)
            load_row(vup[i], u.cols[i], a.up, u.row[i]);
    }
    // codes of a chunk, number k of the shared scales (VEC)
    constexpr int N = KIND == kIdentity ? kUnits : 2 * kUnits;
    float inv[N] = {}, scale = 0.0f;
    const auto pack = [&](const PackedRows& p, int i, const float(&x)[8], int k) {
        if constexpr (VEC) {
            const Columns<VEC>& c = u.cols[i];
            const uint2 w = codes8(x, inv[k], inv[k] < 0.0f, p);
            if (c.count && inside(p, c, u.row[i]))
                *reinterpret_cast<uint2*>(p.codes + u.row[i] * p.stride + c.at) = w;
            // lane k of a group has its scale, and columns or not
            const int64_t group = c.at >> p.log_group;
            if ((lane & ((1 << (p.log_group - 3)) - 1)) == k && (LANES ? c.count != 0 : group << p.log_group < a.cols) &&
                scale_inside(p, u.row[i], group))
                p.scales[u.row[i] * p.scale_stride + group] = scale;
        }
    };
    if constexpr (VEC)
        if (a.saved.codes || (gated && a.saved_up.codes)) {
            uint32_t largest[N];
            const PackedRows* to[N];
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                largest[i] = a.saved.codes ? lanes_max(vx[i].largest(), a.saved.log_group - 3) : 0;
                to[i] = &a.saved;
                if constexpr (KIND != kIdentity) {
                    largest[kUnits + i] = gated && a.saved_up.codes ? lanes_max(vup[i].largest(), a.saved_up.log_group - 3) : 0;
                    to[kUnits + i] = &a.saved_up;
                }
            }
            const SharedScales<N> s(largest, to, lane);
            scale = s.scale;
#pragma unroll
            for (int k = 0; k < N; ++k)
                inv[k] = s.inv[k];
        }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (!u.on[i])
            continue;
        float x[8];
        vx[i].unpack(x);
        if (a.saved.codes) {
            if constexpr (VEC)
                pack(a.saved, i, x, i);
            else
                pack_chunk<VEC>(a.saved, u.cols[i], u.row[i], x, 0, lane);
        }
        if constexpr (KIND != kIdentity) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 f, unused;
                value_and_slope<KIND, false>(pair_of(x, k), f, unused);
                set_pair(x, k, f);
            }
            if (gated) {
                float y[8];
                vup[i].unpack(y);
                if (a.saved_up.codes) {
                    if constexpr (VEC)
                        pack(a.saved_up, i, y, kUnits + i);
                    else
                        pack_chunk<VEC>(a.saved_up, u.cols[i], u.row[i], y, 0, lane);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    set_pair(x, k, mul2(pair_of(x, k), pair_of(y, k)));
            }
            store_typed<VEC>(u.cols[i], a.out, u.row[i], x);
        }
    }
}

template <typename T, int KIND, bool PACKED, bool VEC, bool LANES>
__global__ void __launch_bounds__(kBlock, kBlocks<VEC>) k_activation_grad(const __grid_constant__ ActivationArgs a, const Cut cut)
{
    constexpr int kUnits = kUnitsOf<KIND, VEC>;
    const Units<kUnits, VEC, LANES> u(a.rows, a.cols, cut);
    const int lane = threadIdx.x & 31;
    wait_for_launch_before();
    if (!u.on[0])
        return;
    const bool gated = PACKED ? a.saved_up.codes != nullptr : a.up.data != nullptr;
    using Saved = std::conditional_t<PACKED, CodeChunk<VEC>, Chunk<T, VEC>>;
    Chunk<T, VEC> vd[kUnits];
    Saved vx[kUnits], vup[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        load_row(vd[i], u.cols[i], a.dout, u.row[i]);
        if constexpr (PACKED) {
            vx[i].load(a.saved, u.cols[i], u.row[i], lane);
            if (gated)
                vup[i].load(a.saved_up, u.cols[i], u.row[i], lane);
        } else {
            load_row(vx[i], u.cols[i], a.x, u.row[i]);
            if (gated)
                load_row(vup[i], u.cols[i], a.up, u.row[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (!u.on[i])
            continue;
        float x[8], up[8], d[8];
        vd[i].unpack(d);
        if constexpr (PACKED) {
            vx[i].unpack(a.saved, x);
            if (gated)
                vup[i].unpack(a.saved_up, up);
        } else {
            vx[i].unpack(x);
            if (gated)
                vup[i].unpack(up);
        }
        float y[8], dup[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 f, slope;
            value_and_slope<KIND, true>(pair_of(x, k), f, slope);
            float2 g = pair_of(d, k);
            set_pair(dup, k, mul2(g, f));
            if (gated) {
                g = mul2(g, pair_of(up, k));
                f = mul2(f, pair_of(up, k));
            }
            set_pair(y, k, f);
            set_pair(x, k, mul2(g, slope));
        }
        store_typed<VEC>(u.cols[i], a.dx, u.row[i], x);
        if (gated && a.dup.data)
            store_typed<VEC>(u.cols[i], a.dup, u.row[i], dup);
        if (a.again.data)
            store_typed<VEC>(u.cols[i], a.again, u.row[i], y);
    }
}

template <bool VEC, bool LANES, int kUnits = kUnitsOf<kIdentity, VEC>>
__global__ void __launch_bounds__(kBlock) k_unpack(const PackedRows x, const TypedRows out, const int64_t rows, const int64_t cols,
                                                   const Cut cut)
{
    const Units<kUnits, VEC, LANES> u(rows, cols, cut);
    wait_for_launch_before();
    if (!u.on[0])
        return;
    CodeChunk<VEC> v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
        v[i].load(x, u.cols[i], u.row[i], threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        float y[8];
        v[i].unpack(x, y);
        store_typed<VEC>(u.cols[i], out, u.row[i], y);
    }
}

// group: the most columns that share a scale.
struct Grid {
    Cut cut;
    int64_t blocks;
    Grid(int64_t rows, int64_t cols, int units, bool vec, int group)
    {
        const int64_t width = int64_t(units) * kChunk;
        cut.spans = (cols + width - 1) / width;
        int64_t all = rows * cut.spans;  // warps
        cut.lanes = 0;
        // By lanes where more than a quarter of the chunks' lanes had no columns, if groups are then
        // whole (and so lie within a warp).  Forward and backward, two inputs saved in 8 bits out
        // of wider rows: 13131 rows of 128 41.7 us by chunks, 7.2 by lanes; 16384 of 768 41.9 and 42.7.
        if (vec && rows > 1 && cols % std::max(group, 8) == 0 && cut.spans * width * 3 > cols * 4 && cols / 8 <= INT_MAX) {
            cut.lanes = static_cast<int32_t>(cols / 8);
            all = (rows * cut.lanes + 32 * units - 1) / (32 * units);
        }
        blocks = (all + kWarps - 1) / kWarps;
    }
    bool fits() const { return blocks <= INT_MAX && cut.spans <= INT_MAX; }
    // bf16 packed or unpacked only, by four chunks a warp, which then share one quotient, and not two
    // (that is g): where it leaves hardly more chunks without columns and there is a block for each
    // place of 152 SMs.  Packed by two and by four: 8192 x 4096 20.1, 19.0 us, 8192 rows of 768 out of
    // 776 5.0, 4.5, 4096 x 2048 5.27, 5.03; but 3060 x 2048 4.19, 4.27, 788 x 768 1.5, 1.9, 16384 rows
    // of 1536 16.2, 17.5; 8192 x 4096 fp32 25.5, 26.1.  Unpacked as well 16384 x 4096 takes 1 us less.
    bool better_than(const Grid& g) const
    {
        return !cut.lanes && !g.cut.lanes && cut.spans * 30 <= g.cut.spans * 16 && blocks >= 6 * 152;
    }
};

int group_of(const PackedRows& p) { return !p.codes ? 1 : p.log_group == kRowGroup ? 8 : 1 << p.log_group; }

template <typename T, bool VEC, int KIND>
cudaError_t forward_t(const ActivationArgs& a, cudaStream_t s)
{
    const Grid g(a.rows, a.cols, kUnitsOf<KIND, VEC>, VEC, std::max(group_of(a.saved), group_of(a.saved_up)));
    if (!g.fits())
        return cudaErrorInvalidConfiguration;
    const auto go = [&](auto kernel) { return launch_programmatic(kernel, static_cast<unsigned>(g.blocks), kBlock, 0, s, a, g.cut); };
    if constexpr (VEC)
        if (g.cut.lanes)
            return go(k_activation<T, KIND, VEC, true>);
    if constexpr (VEC && KIND == kIdentity && std::is_same_v<T, __nv_bfloat16>) {
        const Grid wide(a.rows, a.cols, 4, VEC, group_of(a.saved));
        if (wide.better_than(g))
            return launch_programmatic(k_activation<T, KIND, VEC, false, 4>, static_cast<unsigned>(wide.blocks), kBlock, 0, s, a, wide.cut);
    }
    return go(k_activation<T, KIND, VEC, false>);
}

template <typename T, bool VEC>
cudaError_t forward_k(const ActivationArgs& a, int kind, cudaStream_t s)
{
    switch (kind) {
    case LIONCUB_ACTIVATION_SILU: return forward_t<T, VEC, LIONCUB_ACTIVATION_SILU>(a, s);
    case LIONCUB_ACTIVATION_GELU: return forward_t<T, VEC, LIONCUB_ACTIVATION_GELU>(a, s);
    default: return forward_t<T, VEC, kIdentity>(a, s);
    }
}

template <typename T, bool VEC, bool PACKED, int KIND>
cudaError_t backward_k(const ActivationArgs& a, cudaStream_t s)
{
    const Grid g(a.rows, a.cols, kUnitsOf<KIND, VEC>, VEC, 8);
    if (!g.fits())
        return cudaErrorInvalidConfiguration;
    const auto go = [&](auto kernel) { return launch_programmatic(kernel, static_cast<unsigned>(g.blocks), kBlock, 0, s, a, g.cut); };
    if constexpr (VEC)
        if (g.cut.lanes)
            return go(k_activation_grad<T, KIND, PACKED, VEC, true>);
    return go(k_activation_grad<T, KIND, PACKED, VEC, false>);
}

template <typename T, bool VEC, bool PACKED>
cudaError_t backward_t(const ActivationArgs& a, int kind, cudaStream_t s)
{
    return kind == LIONCUB_ACTIVATION_SILU ? backward_k<T, VEC, PACKED, LIONCUB_ACTIVATION_SILU>(a, s)
                                           : backward_k<T, VEC, PACKED, LIONCUB_ACTIVATION_GELU>(a, s);
}

template <bool PACKED>
cudaError_t backward_p(const ActivationArgs& a, int kind, bool vec, cudaStream_t s)
{
    if (!vec)
        return backward_t<float, false, PACKED>(a, kind, s);
    return a.dout.type == LIONCUB_ROWS_BF16 ? backward_t<__nv_bfloat16, true, PACKED>(a, kind, s) : backward_t<float, true, PACKED>(a, kind, s);
}

}  // namespace

#ifdef LIONCUB_BOUNDS_CHECK
cudaError_t take_activation_word(int* word) { return take_word(word); }
#endif

cudaError_t launch_activation(const ActivationArgs& a, int kind, bool vec, cudaStream_t s)
{
    if (a.rows == 0 || a.cols == 0)
        return cudaSuccess;
    if (!vec)
        return forward_k<float, false>(a, kind, s);
    return a.x.type == LIONCUB_ROWS_BF16 ? forward_k<__nv_bfloat16, true>(a, kind, s) : forward_k<float, true>(a, kind, s);
}

cudaError_t launch_activation_grad(const ActivationArgs& a, int kind, bool vec, cudaStream_t s)
{
    if (a.rows == 0 || a.cols == 0)
        return cudaSuccess;
    return a.saved.codes ? backward_p<true>(a, kind, vec, s) : backward_p<false>(a, kind, vec, s);
}

cudaError_t launch_unpack(const PackedRows& x, const TypedRows& out, int64_t rows, int64_t cols, bool vec, cudaStream_t s)
{
    if (rows == 0 || cols == 0)
        return cudaSuccess;
    const Grid g(rows, cols, vec ? kUnitsOf<kIdentity, true> : kUnitsOf<kIdentity, false>, vec, 8);
    if (!g.fits())
        return cudaErrorInvalidConfiguration;
    const Grid wide(rows, cols, 4, vec, 8);
    if (vec && out.type == LIONCUB_ROWS_BF16 && wide.better_than(g))
        return launch_programmatic(k_unpack<true, false, 4>, static_cast<unsigned>(wide.blocks), kBlock, 0, s, x, out, rows, cols, wide.cut);
    const auto go = [&](auto kernel) { return launch_programmatic(kernel, static_cast<unsigned>(g.blocks), kBlock, 0, s, x, out, rows, cols, g.cut); };
    return !vec ? go(k_unpack<false, false>) : g.cut.lanes ? go(k_unpack<true, true>) : go(k_unpack<true, false>);
}

}  // namespace lc
