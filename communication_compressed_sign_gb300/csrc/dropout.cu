// dropout.cu -- dropout over a matrix, with an optional residual added:
//   out[e] = (keep(e) ? RN(r * x[e]) : 0) (+ residual[e]).
// The backward pass is the same map of the gradient, with the mask drawn again
// from the same counters.
//
// Memory-bound: each element is read and written once and no mask exists in
// memory.  Dense, aligned matrices are one flat vector, 8 elements a thread;
// others are taken by rows, a warp on a slab of columns.  Measured: 65536 x 2048
// bf16 81 us (6.6 TB/s, 98 % of a measured copy), 8192 x 768 bf16 onto an fp32
// residual 10.4 us (6.0 TB/s); rows of 771 bf16, 776 apart, 16384 of them 15.6 us
// (3.2 TB/s: scalar moves).
#include <climits>

#include "embed_device.cuh"

namespace lc {
namespace {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;

// x = keep ? r x : 0 (+ residual)
__device__ __forceinline__ float dropped(const DropArgs& d, float x, bool keep)
{
    return keep ? __fmul_rn(d.rescale, x) : 0.0f;
}

// The last elements of a flat vector, one by one.
template <typename XT, typename OT, bool DROP>
__device__ __forceinline__ void drop_one(const DropoutArgs& a, int64_t e)
{
    float x = static_cast<float>(static_cast<const XT*>(a.x.data)[e]);
    if constexpr (DROP) {
        const uint64_t u = splitmix64_mix(a.drop.first + (static_cast<uint64_t>(e) >> 2) * kSplitMix64Step);
        x = dropped(a.drop, x, lower_stays(a.drop, static_cast<uint32_t>(u >> (16 * (e & 3)))));
    }
    if (a.residual.data)
        x = __fadd_rn(x, static_cast<float>(static_cast<const OT*>(a.residual.data)[e]));
    static_cast<OT*>(a.out.data)[e] = static_cast<OT>(x);
}

template <typename XT, typename OT, bool DROP>
__global__ void __launch_bounds__(kBlock) k_dropout_flat(const DropoutArgs a)
{
    wait_for_launch_before();
    const int64_t n = a.rows * a.cols;
    const int64_t e = (static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x) * 8;
    if (e + 8 > n) {
        for (int64_t k = e; k < n; ++k)
            drop_one<XT, OT, DROP>(a, k);
        return;
    }
    Group8<XT> in;
    Group8<OT> res, out;
    in.load(a.x.data, e);
    if (a.residual.data)
        res.load(a.residual.data, e);
    float x[8];
    in.unpack(x);
    if constexpr (DROP)
        for_kept8(a.drop, a.drop.first + (static_cast<uint64_t>(e) >> 2) * kSplitMix64Step,
                  [&](int k, bool keep) { x[k] = dropped(a.drop, x[k], keep); });
    if (a.residual.data) {
        float y[8];
        res.unpack(y);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = __fadd_rn(x[k], y[k]);
    }
    out.pack(x);
    out.store(a.out.data, e);
}

constexpr int kRows = 4;  // rows a warp loads before it works on them

template <typename XT, typename OT, bool VEC, bool DROP>
__global__ void __launch_bounds__(kBlock) k_dropout_rows(const DropoutArgs a, const int slabs)
{
    constexpr int N = kLaneCols<VEC>;
    __shared__ typename SlabMask<VEC>::Shared shared[DROP ? kWarps : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t row0 = quotient(unit, slabs) * kRows;
    const int slab = static_cast<int>(unit - row0 / kRows * slabs);
    wait_for_launch_before();
    if (row0 >= a.rows)
        return;
    const Slab<VEC> cols(slab, lane, static_cast<int>(a.cols));
    SlabMask<VEC> mask(a.drop, slab, lane, static_cast<int>(a.cols), &shared[DROP ? warp : 0]);
    SlabGroup<XT, VEC> in[kRows];
    SlabGroup<OT, VEC> res[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int64_t i = min(row0 + u, a.rows - 1);
        in[u].load(cols, a.x.data, i * a.x.stride);
        if (a.residual.data)
            res[u].load(cols, a.residual.data, i * a.residual.stride);
    }
    if (DROP)
        mask.template draw<kRows>(static_cast<int>(min(a.rows - row0, static_cast<int64_t>(kRows))), [&](int u) { return row0 + u; });
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int64_t i = row0 + u;
        if (i >= a.rows)
            break;
        float x[N];
        in[u].unpack(x);
        if constexpr (DROP)
            mask.row(u, static_cast<uint32_t>(i), [&](int k, bool keep) { x[k] = dropped(a.drop, x[k], keep); });
        if (a.residual.data) {
            float y[N];
            res[u].unpack(y);
#pragma unroll
            for (int k = 0; k < N; ++k)
                x[k] = __fadd_rn(x[k], y[k]);
        }
        store_slab<OT, VEC>(cols, a.out.data, i * a.out.stride, x);
    }
}

template <typename XT, typename OT, bool DROP>
cudaError_t launch_t(const DropoutArgs& a, bool vec, cudaStream_t s)
{
    const bool dense = a.x.stride == a.cols && a.out.stride == a.cols && (!a.residual.data || a.residual.stride == a.cols);
    if (vec && dense) {
        const int64_t blocks = (a.rows * a.cols + kBlock * 8 - 1) / (kBlock * 8);
        return launch_programmatic(k_dropout_flat<XT, OT, DROP>, static_cast<unsigned>(blocks), kBlock, 0, s, a);
    }
    const bool wide = vec && a.cols % 8 == 0;
    const int slabs = slabs_of(a.cols, wide);
    const int64_t blocks = ((a.rows + kRows - 1) / kRows * slabs + kWarps - 1) / kWarps;
    if (blocks > INT_MAX)
        return cudaErrorInvalidConfiguration;
    return wide ? launch_programmatic(k_dropout_rows<XT, OT, true, DROP>, static_cast<unsigned>(blocks), kBlock, 0, s, a, slabs)
                : launch_programmatic(k_dropout_rows<XT, OT, false, DROP>, static_cast<unsigned>(blocks), kBlock, 0, s, a, slabs);
}

template <typename XT, typename OT>
cudaError_t launch_d(const DropoutArgs& a, bool vec, bool drop, cudaStream_t s)
{
    return drop ? launch_t<XT, OT, true>(a, vec, s) : launch_t<XT, OT, false>(a, vec, s);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, int x_type, int out_type, bool vec, bool drop, cudaStream_t s)
{
    if (a.rows == 0 || a.cols == 0)
        return cudaSuccess;
    if (x_type == LIONCUB_ROWS_BF16)
        return out_type == LIONCUB_ROWS_BF16 ? launch_d<__nv_bfloat16, __nv_bfloat16>(a, vec, drop, s)
                                             : launch_d<__nv_bfloat16, float>(a, vec, drop, s);
    return out_type == LIONCUB_ROWS_BF16 ? launch_d<float, __nv_bfloat16>(a, vec, drop, s)
                                         : launch_d<float, float>(a, vec, drop, s);
}

}  // namespace lc
