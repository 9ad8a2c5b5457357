// embed_lookup.cu -- embedding lookup with scaling, position rows and dropout:
//   out[i,j] = keep(i*D+j) ? RN(r * RN(RN(scale * table[t_i,j]) + pos_table[q_i,j])) : 0.
//
// A table row is read and an output row written once for each place (repeated
// tokens hit L2).  One warp takes several places on a slab of columns, so that
// their rows are in flight together and the index arithmetic is shared.  Wide
// rows with dropout are bound by instructions about as much as by memory, so
// sums and rescalings are done two at a time (fp32 pairs).
#include "embed_device.cuh"

namespace lc {
namespace {

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;

// y += q and y *= r, in pairs.  Pairs are used for a sum whose result is
// rescaled, never for a product that is then summed: the assembler fuses a
// paired product and sum, whatever their rounding modifiers.
template <int N>
__device__ __forceinline__ void add_pairs(float (&y)[N], const float (&q)[N])
{
#pragma unroll
    for (int k = 0; k + 1 < N; k += 2)
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "+f"(y[k]), "+f"(y[k + 1]) : "f"(q[k]), "f"(q[k + 1]));
    if constexpr (N % 2)
        y[N - 1] = __fadd_rn(y[N - 1], q[N - 1]);
}
template <int N>
__device__ __forceinline__ void scale_pairs(float (&y)[N], float r)
{
#pragma unroll
    for (int k = 0; k + 1 < N; k += 2)
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
            : "+f"(y[k]), "+f"(y[k + 1]) : "f"(r));
    if constexpr (N % 2)
        y[N - 1] = __fmul_rn(y[N - 1], r);
}

// One warp: PLACES places on a slab of columns.  With running positions they
// are the same place of that many sequences, so its position row is read once;
// otherwise neighbours.
template <typename TT, typename OT, bool VEC, bool DROP, int PLACES, bool RUNNING>
__global__ void __launch_bounds__(kBlock) k_lookup(const LookupArgs a)
{
    constexpr int N = kLaneCols<VEC>;
    __shared__ typename SlabMask<VEC>::Shared shared[DROP ? kWarps : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const int64_t group = quotient(unit, a.slabs);
    const int slab = static_cast<int>(unit - group * a.slabs);
    const int span = static_cast<int>(a.span);
    int64_t place0 = group * PLACES, step = 1, in_sequence = 0;
    if constexpr (RUNNING) {
        const int64_t sequences = quotient(group, span);  // PLACES sequences each
        step = span;
        in_sequence = group - sequences * span;
        place0 = sequences * PLACES * step + in_sequence;
    }
    if (place0 >= a.at.n)
        return;

    // lane u: the token and position of place u
    int my_token = -1, my_position = -1;
    if (lane < PLACES && place0 + lane * step < a.at.n) {
        my_token = token_at(a.at, place0 + lane * step, a.status);
        if (a.pos_table.data)
            my_position = RUNNING ? static_cast<int>(a.at.first + in_sequence) : position_at(a.at, place0 + lane * step, a.status);
    }
    const Slab<VEC> cols(slab, lane, a.dim);
    SlabMask<VEC> mask(a.drop, slab, lane, a.dim, &shared[DROP ? warp : 0]);
    SlabGroup<TT, VEC> x[PLACES], p[RUNNING ? 1 : PLACES];
    int token[PLACES], position[PLACES];
#pragma unroll
    for (int u = 0; u < PLACES; ++u) {
        token[u] = __shfl_sync(kAll, my_token, u);
        x[u].load(cols, a.table.data, static_cast<uint32_t>(max(token[u], 0)) * a.table.stride);
    }
    if (a.pos_table.data) {
#pragma unroll
        for (int u = 0; u < PLACES; ++u) {
            position[u] = __shfl_sync(kAll, my_position, u);
            if (u == 0 || !RUNNING)
                p[u].load(cols, a.pos_table.data, static_cast<uint32_t>(max(position[u], 0)) * a.pos_table.stride);
        }
    }
#pragma unroll
    for (int u = 0; u < PLACES; ++u) {
        const int64_t place = place0 + u * step;
        if (place >= a.at.n)
            break;
        const uint32_t i = static_cast<uint32_t>(place);
        float y[N];
        if (token[u] < 0) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                y[k] = 0.0f;
            store_slab<OT, VEC>(cols, a.out.data, i * a.out.stride, y);
            continue;
        }
        x[u].unpack(y);
        if (a.scale != 1.0f) {
#pragma unroll
            for (int k = 0; k < N; ++k)
                y[k] = __fmul_rn(a.scale, y[k]);
        }
        if (a.pos_table.data && position[u] >= 0) {
            float q[N];
            p[RUNNING ? 0 : u].unpack(q);
            add_pairs(y, q);
        }
        if constexpr (DROP) {
            scale_pairs(y, a.drop.rescale);
            mask.row(i, [&](int k, bool keep) { y[k] = keep ? y[k] : 0.0f; });
        }
        store_slab<OT, VEC>(cols, a.out.data, i * a.out.stride, y);
    }
}

// Four places a warp keep enough bytes in flight and share a position row;
// fewer warps than the SMs hold run one place each, for the latency.
constexpr int kPlaces = 4;
constexpr int64_t kFewWarps = 152 * kWarps;

template <typename TT, typename OT, bool VEC, bool DROP>
cudaError_t launch_k(LookupArgs a, cudaStream_t s)
{
    a.slabs = slabs_of(a.dim, VEC);
    a.span = a.at.seq_len < a.at.n ? a.at.seq_len : a.at.n;
    const bool few = a.at.n * static_cast<int64_t>(a.slabs) <= kFewWarps;
    const bool running = a.pos_table.data && !a.at.positions && !few;
    const int64_t places = few ? 1 : kPlaces;
    int64_t groups = (a.at.n + places - 1) / places;
    if (running) {
        const int64_t sequences = (a.at.n + a.span - 1) / a.span;
        groups = (sequences + places - 1) / places * a.span;
    }
    const unsigned blocks = static_cast<unsigned>((groups * a.slabs + kWarps - 1) / kWarps);
    if (few)
        k_lookup<TT, OT, VEC, DROP, 1, false><<<blocks, kBlock, 0, s>>>(a);
    else if (running)
        k_lookup<TT, OT, VEC, DROP, kPlaces, true><<<blocks, kBlock, 0, s>>>(a);
    else
        k_lookup<TT, OT, VEC, DROP, kPlaces, false><<<blocks, kBlock, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename TT, typename OT>
cudaError_t launch_t(const LookupArgs& a, bool vec, bool drop, cudaStream_t s)
{
    if (vec)
        return drop ? launch_k<TT, OT, true, true>(a, s) : launch_k<TT, OT, true, false>(a, s);
    return drop ? launch_k<TT, OT, false, true>(a, s) : launch_k<TT, OT, false, false>(a, s);
}

}  // namespace

cudaError_t launch_lookup(const LookupArgs& a, int table_type, int out_type, bool vec, bool drop, cudaStream_t s)
{
    if (a.at.n == 0)
        return cudaSuccess;
    if (table_type == LIONCUB_ROWS_BF16)
        return out_type == LIONCUB_ROWS_BF16 ? launch_t<__nv_bfloat16, __nv_bfloat16>(a, vec, drop, s)
                                             : launch_t<__nv_bfloat16, float>(a, vec, drop, s);
    return out_type == LIONCUB_ROWS_BF16 ? launch_t<float, __nv_bfloat16>(a, vec, drop, s)
                                         : launch_t<float, float>(a, vec, drop, s);
}

}  // namespace lc
