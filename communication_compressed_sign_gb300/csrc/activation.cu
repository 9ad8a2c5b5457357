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

// f(x) and, where it is wanted, f'(x).  |x| > 30 is beyond where s changes: the
// bound keeps powers of x finite.
template <int KIND, bool SLOPE>
__device__ __forceinline__ void value_and_slope(float x, float& f, float& slope)
{
    constexpr float kTwice = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float y = KIND == LIONCUB_ACTIVATION_GELU ? fminf(fmaxf(x, -30.0f), 30.0f) : x;
    const float square = __fmul_rn(y, y);
    const float z = KIND == LIONCUB_ACTIVATION_GELU ? __fmul_rn(kTwice, __fmul_rn(y, fmaf(0.044715f, square, 1.0f))) : x;
    const float s = __fdividef(1.0f, __fadd_rn(1.0f, expf(-z)));
    f = __fmul_rn(x, s);
    if (SLOPE) {
        const float dz = KIND == LIONCUB_ACTIVATION_GELU ? fmaf(kTwice * 3 * 0.044715f, square, kTwice) : 1.0f;
        slope = fmaf(__fmul_rn(f, __fsub_rn(1.0f, s)), dz, s);
    }
}

// A row and the chunk of it that a warp has.
template <bool VEC>
struct Unit {
    int64_t row;
    Columns<VEC> cols;
    bool on;
    __device__ __forceinline__ Unit(int64_t rows, int64_t width, int64_t chunks) : row(0)
    {
        const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
        row = rows == 1 ? 0 : quotient(unit, static_cast<int>(chunks));
        const int64_t chunk = unit - row * chunks;
        on = row < rows && chunk < chunks;
        cols = Columns<VEC>(chunk * kChunk, threadIdx.x & 31, width);
    }
};

template <typename T, int KIND, bool VEC>
__global__ void __launch_bounds__(kBlock) k_activation(const __grid_constant__ ActivationArgs a, const int64_t chunks)
{
    const Unit<VEC> u(a.rows, a.cols, chunks);
    const int lane = threadIdx.x & 31;
    wait_for_launch_before();
    if (!u.on)
        return;
    Chunk<T, VEC> vx, vup;
    vx.load(u.cols, a.x.data, u.row * a.x.stride, a.x.type);
    if (KIND != kIdentity && a.up.data)
        vup.load(u.cols, a.up.data, u.row * a.up.stride, a.up.type);
    float x[8];
    vx.unpack(x);
    if (a.saved.codes)
        pack_chunk<VEC>(a.saved, u.cols, u.row, x, lane);
    if constexpr (KIND != kIdentity) {
        float unused;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            value_and_slope<KIND, false>(x[k], x[k], unused);
        if (a.up.data) {
            float y[8];
            vup.unpack(y);
            if (a.saved_up.codes)
                pack_chunk<VEC>(a.saved_up, u.cols, u.row, y, lane);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = __fmul_rn(x[k], y[k]);
        }
        store_typed<VEC>(u.cols, a.out.data, u.row * a.out.stride, a.out.type, x);
    }
}

template <typename T, int KIND, bool PACKED, bool VEC>
__global__ void __launch_bounds__(kBlock) k_activation_grad(const __grid_constant__ ActivationArgs a, const int64_t chunks)
{
    const Unit<VEC> u(a.rows, a.cols, chunks);
    wait_for_launch_before();
    if (!u.on)
        return;
    const bool gated = PACKED ? a.saved_up.codes != nullptr : a.up.data != nullptr;
    Chunk<T, VEC> vd;
    vd.load(u.cols, a.dout.data, u.row * a.dout.stride, a.dout.type);
    float x[8], up[8], d[8];
    if constexpr (PACKED) {
        CodeChunk<VEC> vx, vup;
        vx.load(a.saved, u.cols, u.row);
        if (gated)
            vup.load(a.saved_up, u.cols, u.row);
        vx.unpack(a.saved, x);
        if (gated)
            vup.unpack(a.saved_up, up);
    } else {
        Chunk<T, VEC> vx, vup;
        vx.load(u.cols, a.x.data, u.row * a.x.stride, a.x.type);
        if (gated)
            vup.load(u.cols, a.up.data, u.row * a.up.stride, a.up.type);
        vx.unpack(x);
        if (gated)
            vup.unpack(up);
    }
    vd.unpack(d);
    float y[8], dup[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float f, slope;
        value_and_slope<KIND, true>(x[k], f, slope);
        dup[k] = __fmul_rn(d[k], f);
        y[k] = gated ? __fmul_rn(f, up[k]) : f;
        x[k] = __fmul_rn(gated ? __fmul_rn(d[k], up[k]) : d[k], slope);
    }
    store_typed<VEC>(u.cols, a.dx.data, u.row * a.dx.stride, a.dx.type, x);
    if (gated && a.dup.data)
        store_typed<VEC>(u.cols, a.dup.data, u.row * a.dup.stride, a.dup.type, dup);
    if (a.again.data)
        store_typed<VEC>(u.cols, a.again.data, u.row * a.again.stride, a.again.type, y);
}

template <bool VEC>
__global__ void __launch_bounds__(kBlock) k_unpack(const PackedRows x, const TypedRows out, const int64_t rows, const int64_t cols,
                                                   const int64_t chunks)
{
    const Unit<VEC> u(rows, cols, chunks);
    wait_for_launch_before();
    if (!u.on)
        return;
    CodeChunk<VEC> v;
    v.load(x, u.cols, u.row);
    float y[8];
    v.unpack(x, y);
    store_typed<VEC>(u.cols, out.data, u.row * out.stride, out.type, y);
}

struct Grid {
    int64_t chunks, blocks;
    Grid(int64_t rows, int64_t cols)
    {
        chunks = (cols + kChunk - 1) / kChunk;
        blocks = (rows * chunks + kWarps - 1) / kWarps;
    }
    bool fits(int64_t rows) const { return blocks <= INT_MAX && (rows == 1 || chunks <= INT_MAX); }
};

template <typename T, bool VEC>
cudaError_t forward_t(const ActivationArgs& a, int kind, cudaStream_t s)
{
    const Grid g(a.rows, a.cols);
    if (!g.fits(a.rows))
        return cudaErrorInvalidConfiguration;
    const unsigned blocks = static_cast<unsigned>(g.blocks);
    switch (kind) {
    case LIONCUB_ACTIVATION_SILU: return launch_programmatic(k_activation<T, LIONCUB_ACTIVATION_SILU, VEC>, blocks, kBlock, 0, s, a, g.chunks);
    case LIONCUB_ACTIVATION_GELU: return launch_programmatic(k_activation<T, LIONCUB_ACTIVATION_GELU, VEC>, blocks, kBlock, 0, s, a, g.chunks);
    default: return launch_programmatic(k_activation<T, kIdentity, VEC>, blocks, kBlock, 0, s, a, g.chunks);
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
               ? launch_programmatic(k_activation_grad<T, LIONCUB_ACTIVATION_SILU, PACKED, VEC>, blocks, kBlock, 0, s, a, g.chunks)
               : launch_programmatic(k_activation_grad<T, LIONCUB_ACTIVATION_GELU, PACKED, VEC>, blocks, kBlock, 0, s, a, g.chunks);
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
    return vec ? launch_programmatic(k_unpack<true>, blocks, kBlock, 0, s, x, out, rows, cols, g.chunks)
               : launch_programmatic(k_unpack<false>, blocks, kBlock, 0, s, x, out, rows, cols, g.chunks);
}

}  // namespace lc
