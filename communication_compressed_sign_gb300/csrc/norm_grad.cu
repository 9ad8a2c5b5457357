// norm_grad.cu -- the gradient of the root-mean-square norm (n = h * rstd,
// g = dout * weight):
//   dx = residual_grad + rstd * (g - n * mean(g * n)),  again = n * weight,
//   weight_grad_j = weight_base_j + sum over rows of dout * n.
//
// Memory-bound.  A team of warps takes a row, whose chunks stay in registers
// across the one sum over the row.  Teams walk over rows (persistent blocks, one
// for each multiprocessor), so that a column's share of the weight's gradient
// stays in registers too; a block adds its teams' in order and leaves one row of
// sums, and a second launch adds those of all blocks in order.
#include "block_device.cuh"

namespace lc {
namespace {

constexpr int kMaxWarps = 16;    // of a row
constexpr int kBlockWarps = 16;  // of a block

// Where h comes from.
enum Source { kFromBf16, kFromF32, kFromCodes };

template <int SOURCE, bool VEC>
struct SavedChunk {
    std::conditional_t<SOURCE == kFromCodes, CodeChunk<VEC>, Chunk<std::conditional_t<SOURCE == kFromBf16, __nv_bfloat16, float>, VEC>> v;
    __device__ __forceinline__ void load(const NormGradArgs& a, const Columns<VEC>& c, int64_t row)
    {
        if constexpr (SOURCE == kFromCodes)
            v.load(a.packed, c, row);
        else
            v.load(c, a.saved.data, row * a.saved.stride, a.saved.type);
    }
    __device__ __forceinline__ void unpack(const NormGradArgs& a, float (&x)[8]) const
    {
        if constexpr (SOURCE == kFromCodes)
            v.unpack(a.packed, x);
        else
            v.unpack(x);
    }
};

// What a team reads of a row.
template <typename DT, typename GT, int SOURCE, int C, bool VEC>
struct RowInputs {
    Chunk<DT, VEC> dout[C];
    SavedChunk<SOURCE, VEC> saved[C];
    Chunk<GT, VEC> residual[C];
    float rstd;
    __device__ __forceinline__ void load(const NormGradArgs& a, const Columns<VEC> (&cols)[C], int64_t row)
    {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            dout[c].load(cols[c], a.dout.data, row * a.dout.stride, a.dout.type);
            saved[c].load(a, cols[c], row);
        }
        rstd = a.rstd[row];
        if (a.residual_grad.data)
#pragma unroll
            for (int c = 0; c < C; ++c)
                residual[c].load(cols[c], a.residual_grad.data, row * a.residual_grad.stride, a.residual_grad.type);
    }
};

__device__ __forceinline__ void team_barrier(int team, int warps)
{
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

template <bool VEC>
__device__ __forceinline__ void load_weight(const NormGradArgs& a, const Columns<VEC>& c, float (&w)[8])
{
    if (a.weight.data) {
        load_typed<VEC>(c, a.weight.data, 0, a.weight.type, w);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = 1.0f;
    }
}

template <typename DT, typename GT, int SOURCE, int C, bool VEC>
__global__ void __launch_bounds__(kBlockWarps * 32) k_norm_grad(const __grid_constant__ NormGradArgs a)
{
    // Wide rows need their registers for one row: the next one is then not loaded
    // ahead, and the widest read the weight again from cache.
    constexpr bool kAhead = C == 1;
    constexpr int kKept = C < 4 ? C : 1;
    extern __shared__ float columns[];  // the block's sums of its columns
    __shared__ float sums[2][kBlockWarps];
    const int lane = threadIdx.x & 31, in_block = threadIdx.x >> 5;
    const int warps = a.warps, team = in_block / warps, warp = in_block - team * warps;
    Columns<VEC> cols[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
        cols[c] = Columns<VEC>((warp + c * warps) * kChunk, lane, a.dim);
    wait_for_launch_before();

    float weight[kKept][8], grad[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            grad[c][k] = 0.0f;
#pragma unroll
    for (int c = 0; c < kKept; ++c)
        load_weight<VEC>(a, cols[c], weight[c]);
    const float size = static_cast<float>(a.dim);
    const int64_t step = static_cast<int64_t>(gridDim.x) * a.teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + team;
    int turn = 0;
    RowInputs<DT, GT, SOURCE, C, VEC> in;
    if (kAhead && row < a.n)
        in.load(a, cols, row);
    for (; row < a.n; row += step) {
        if (!kAhead)
            in.load(a, cols, row);
        // dout, then g = dout * weight; n = h * rstd
        float g[C][8], n[C][8], sum = 0.0f;
        const float rstd = in.rstd;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            in.dout[c].unpack(g[c]);
            in.saved[c].unpack(a, n[c]);
            float w[8];
            if (kKept < C)
                load_weight<VEC>(a, cols[c], w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                n[c][k] = __fmul_rn(n[c][k], rstd);
                grad[c][k] = fmaf(g[c][k], n[c][k], grad[c][k]);
                g[c][k] = __fmul_rn(g[c][k], kKept < C ? w[k] : weight[c % kKept][k]);
                sum = fmaf(g[c][k], n[c][k], sum);
            }
        }
        Chunk<GT, VEC> residual[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            residual[c] = in.residual[c];
        if (kAhead && row + step < a.n)
            in.load(a, cols, row + step);
        sum = warp_sum(sum);
        if (warps > 1) {  // sums of two rows take turns, so one barrier a row is enough
            if (lane == 0)
                sums[turn][in_block] = sum;
            team_barrier(team, warps);
            sum = 0.0f;
            for (int k = 0; k < warps; ++k)
                sum = __fadd_rn(sum, sums[turn][team * warps + k]);
            turn ^= 1;
        }
        const float mean = __fdiv_rn(sum, size);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.again.data) {
                float y[8], w[8];
                if (kKept < C)
                    load_weight<VEC>(a, cols[c], w);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    y[k] = __fmul_rn(n[c][k], kKept < C ? w[k] : weight[c % kKept][k]);
                store_typed<VEC>(cols[c], a.again.data, row * a.again.stride, a.again.type, y);
            }
            float rest[8];
            if (a.residual_grad.data)
                residual[c].unpack(rest);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float d = __fmul_rn(rstd, fmaf(-n[c][k], mean, g[c][k]));
                g[c][k] = a.residual_grad.data ? __fadd_rn(d, rest[k]) : d;
            }
            store_typed<VEC>(cols[c], a.dx.data, row * a.dx.stride, a.dx.type, g[c]);
        }
    }
    if (!a.partial)
        return;
    for (int t = 0; t < a.teams; ++t) {  // a column is one lane's in every team
        if (team == t) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < cols[c].count) {
                        const int j = static_cast<int>(cols[c].at) + (VEC ? k : 32 * k);
                        columns[j] = t ? __fadd_rn(columns[j], grad[c][k]) : grad[c][k];
                    }
        }
        __syncthreads();
    }
    float* to = a.partial + static_cast<int64_t>(blockIdx.x) * a.dim;
    if (index_ok(a.status, static_cast<int64_t>(blockIdx.x) < a.partial_rows))
        for (int j = threadIdx.x; j < a.dim; j += blockDim.x)
            to[j] = columns[j];
}

// The blocks' rows, added in order: a warp adds every eighth row of 32 columns,
// and one of them the eight sums.
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(kJoinWarps * 32) k_weight_grad(const __grid_constant__ WeightGradArgs a)
{
    __shared__ float sums[kJoinWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    wait_for_launch_before();
    float sum = 0.0f;
    if (j < a.dim)
#pragma unroll 4
        for (int64_t i = warp; i < a.rows; i += kJoinWarps)
            sum = __fadd_rn(sum, a.partial[i * a.dim + j]);
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp || j >= a.dim)
        return;
    for (int k = 1; k < kJoinWarps; ++k)
        sum = __fadd_rn(sum, sums[k][lane]);
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
        c = chunks <= kMaxWarps ? 1 : chunks <= 2 * kMaxWarps ? 2 : 4;
        warps = (chunks + c - 1) / c;
        teams = kBlockWarps / warps;
    }
};

template <typename DT, typename GT, int SOURCE, int C, bool VEC>
cudaError_t launch_c(const NormGradArgs& a, int blocks, cudaStream_t s)
{
    const auto kernel = k_norm_grad<DT, GT, SOURCE, C, VEC>;
    const size_t shared = a.partial ? a.dim * sizeof(float) : 0;
    if (shared > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, LIONCUB_NORM_MAX_DIM * sizeof(float));
        if (e != cudaSuccess)
            return e;
    }
    return launch_programmatic(kernel, static_cast<unsigned>(blocks), a.warps * a.teams * 32, shared, s, a);
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
