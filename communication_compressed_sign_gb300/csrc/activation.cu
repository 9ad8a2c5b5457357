// activation.cu -- f(x) (* up) and its gradient, 8-bit codes of matrices, and
// what codes stand for:
//   f(x) = x * s(z), s(z) = 1 / (1 + exp(-z)), z = x or 2 sqrt(2 / pi) (x + 0.044715 x^3),
//   f'(x) = s + x * s * (1 - s) * z'.
//
// Memory-bound: each element is read and written once; groups of columns that
// share a scale lie inside a warp's chunk of 256 columns, so their maxima need
// shuffles only.  Dense matrices whose rows are whole groups are one long row.
#include <climits>

#include "block_device.cuh"

namespace lc {
namespace {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;
constexpr int kUnits = 2;  // chunks of a warp, whose loads are in flight together

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

// The chunks of a warp: kUnits neighbours in a row, of which it has `spans` times as many.
template <bool VEC>
struct Units {
    int64_t row, first, width;
    Columns<VEC> cols[kUnits];
    __device__ __forceinline__ Units(int64_t rows, int64_t w, int64_t spans) : width(w)
    {
        const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
        row = rows == 1 ? 0 : quotient(unit, static_cast<int>(spans));
        first = (unit - row * spans) * (kUnits * kChunk);
        if (row >= rows)  // behind the last
            first = width;
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            cols[u] = Columns<VEC>(first + u * kChunk, threadIdx.x & 31, width);
    }
    __device__ __forceinline__ bool none() const { return first >= width; }
    __device__ __forceinline__ bool on(int u) const { return first + u * kChunk < width; }
};

template <typename T, int KIND, bool VEC>
__global__ void __launch_bounds__(kBlock) k_activation(const __grid_constant__ ActivationArgs a, const int64_t spans)
{
    const Units<VEC> u(a.rows, a.cols, spans);
    const int lane = threadIdx.x & 31;
    wait_for_launch_before();
    if (u.none())
        return;
    Chunk<T, VEC> vx[kUnits], vup[kUnits];
    const bool gated = KIND != kIdentity && a.up.data;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        vx[i].load(u.cols[i], a.x.data, u.row * a.x.stride, a.x.type);
        if (gated)
            vup[i].load(u.cols[i], a.up.data, u.row * a.up.stride, a.up.type);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (!u.on(i))
            continue;
        float x[8];
        vx[i].unpack(x);
        if (a.saved.codes)
            pack_chunk<VEC>(a.saved, u.cols[i], u.row, x, vx[i].largest(), lane);
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
                if (a.saved_up.codes)
                    pack_chunk<VEC>(a.saved_up, u.cols[i], u.row, y, vup[i].largest(), lane);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    set_pair(x, k, mul2(pair_of(x, k), pair_of(y, k)));
            }
            store_typed<VEC>(u.cols[i], a.out.data, u.row * a.out.stride, a.out.type, x);
        }
    }
}

template <typename T, int KIND, bool PACKED, bool VEC>
__global__ void __launch_bounds__(kBlock) k_activation_grad(const __grid_constant__ ActivationArgs a, const int64_t spans)
{
    const Units<VEC> u(a.rows, a.cols, spans);
    const int lane = threadIdx.x & 31;
    wait_for_launch_before();
    if (u.none())
        return;
    const bool gated = PACKED ? a.saved_up.codes != nullptr : a.up.data != nullptr;
    using Saved = std::conditional_t<PACKED, CodeChunk<VEC>, Chunk<T, VEC>>;
    Chunk<T, VEC> vd[kUnits];
    Saved vx[kUnits], vup[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        vd[i].load(u.cols[i], a.dout.data, u.row * a.dout.stride, a.dout.type);
        if constexpr (PACKED) {
            vx[i].load(a.saved, u.cols[i], u.row, lane);
            if (gated)
                vup[i].load(a.saved_up, u.cols[i], u.row, lane);
        } else {
            vx[i].load(u.cols[i], a.x.data, u.row * a.x.stride, a.x.type);
            if (gated)
                vup[i].load(u.cols[i], a.up.data, u.row * a.up.stride, a.up.type);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (!u.on(i))
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
        store_typed<VEC>(u.cols[i], a.dx.data, u.row * a.dx.stride, a.dx.type, x);
        if (gated && a.dup.data)
            store_typed<VEC>(u.cols[i], a.dup.data, u.row * a.dup.stride, a.dup.type, dup);
        if (a.again.data)
            store_typed<VEC>(u.cols[i], a.again.data, u.row * a.again.stride, a.again.type, y);
    }
}

template <bool VEC>
__global__ void __launch_bounds__(kBlock) k_unpack(const PackedRows x, const TypedRows out, const int64_t rows, const int64_t cols,
                                                   const int64_t spans)
{
    const Units<VEC> u(rows, cols, spans);
    wait_for_launch_before();
    if (u.none())
        return;
    CodeChunk<VEC> v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
        v[i].load(x, u.cols[i], u.row, threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        float y[8];
        v[i].unpack(x, y);
        store_typed<VEC>(u.cols[i], out.data, u.row * out.stride, out.type, y);
    }
}

struct Grid {
    int64_t spans, blocks;
    Grid(int64_t rows, int64_t cols)
    {
        spans = (cols + kUnits * kChunk - 1) / (kUnits * kChunk);
        blocks = (rows * spans + kWarps - 1) / kWarps;
    }
    bool fits(int64_t rows) const { return blocks <= INT_MAX && (rows == 1 || spans <= INT_MAX); }
};

template <typename T, bool VEC>
cudaError_t forward_t(const ActivationArgs& a, int kind, cudaStream_t s)
{
    const Grid g(a.rows, a.cols);
    if (!g.fits(a.rows))
        return cudaErrorInvalidConfiguration;
    const unsigned blocks = static_cast<unsigned>(g.blocks);
    switch (kind) {
    case LIONCUB_ACTIVATION_SILU: return launch_programmatic(k_activation<T, LIONCUB_ACTIVATION_SILU, VEC>, blocks, kBlock, 0, s, a, g.spans);
    case LIONCUB_ACTIVATION_GELU: return launch_programmatic(k_activation<T, LIONCUB_ACTIVATION_GELU, VEC>, blocks, kBlock, 0, s, a, g.spans);
    default: return launch_programmatic(k_activation<T, kIdentity, VEC>, blocks, kBlock, 0, s, a, g.spans);
    }
}

template <typename T, bool VEC, bool PACKED>
cudaError_t backward_t(const ActivationArgs& a, int kind, cudaStream_t s)
{
    const Grid g(a.rows, a.cols);
    if (!g.fits(a.rows))
        return cudaErrorInvalidConfiguration;
    const unsigned blocks = static_cast<unsigned>(g.blocks);
    return kind == LIONCUB_ACTIVATION_SILU
               ? launch_programmatic(k_activation_grad<T, LIONCUB_ACTIVATION_SILU, PACKED, VEC>, blocks, kBlock, 0, s, a, g.spans)
               : launch_programmatic(k_activation_grad<T, LIONCUB_ACTIVATION_GELU, PACKED, VEC>, blocks, kBlock, 0, s, a, g.spans);
}

template <bool PACKED>
cudaError_t backward_p(const ActivationArgs& a, int kind, bool vec, cudaStream_t s)
{
    if (!vec)
        return backward_t<float, false, PACKED>(a, kind, s);
    return a.dout.type == LIONCUB_ROWS_BF16 ? backward_t<__nv_bfloat16, true, PACKED>(a, kind, s) : backward_t<float, true, PACKED>(a, kind, s);
}

}  // namespace

cudaError_t launch_activation(const ActivationArgs& a, int kind, bool vec, cudaStream_t s)
{
    if (a.rows == 0 || a.cols == 0)
        return cudaSuccess;
    if (!vec)
        return forward_t<float, false>(a, kind, s);
    return a.x.type == LIONCUB_ROWS_BF16 ? forward_t<__nv_bfloat16, true>(a, kind, s) : forward_t<float, true>(a, kind, s);
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
    const Grid g(rows, cols);
    if (!g.fits(rows))
        return cudaErrorInvalidConfiguration;
    const unsigned blocks = static_cast<unsigned>(g.blocks);
    return vec ? launch_programmatic(k_unpack<true>, blocks, kBlock, 0, s, x, out, rows, cols, g.spans)
               : launch_programmatic(k_unpack<false>, blocks, kBlock, 0, s, x, out, rows, cols, g.spans);
}

}  // namespace lc
