// embed_lookup.cu -- embedding lookup with scaling, position rows and dropout:
//   out[i,j] = keep(i*D+j) ? RN(r * RN(RN(scale * table[t_i,j]) + pos_table[q_i,j])) : 0.
//
// A table row is read and an output row written once for each place (repeated
// tokens hit L2).  One warp takes several places on a slab of columns, so that
// their rows are in flight together and the index arithmetic is shared.  Wide
// rows with dropout are bound by instructions about as much as by memory, so
// sums and rescalings are done two at a time (fp32 pairs).  Measured (fp32 rows
// of 2048 columns to bf16, 64 x 1024 places, 413 MB at least): 87 us with
// dropout, 77 without; 8 x 1024 of 768 (27 MB): 7.2 and 5.0 us.
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

// Which position row a place adds.
enum Positions { kNone, kRunning, kGiven };

// One warp: a.rounds times PLACES places on a slab of columns, PLACES in flight
// and the tokens of the next round on their way.  With running positions they
// are the same place of that many sequences, so its position row is read once;
// otherwise neighbours.
template <typename TT, typename OT, bool VEC, bool DROP, int PLACES, int POSITIONS>
__global__ void __launch_bounds__(kBlock) k_lookup(const LookupArgs a)
{
    constexpr int N = kLaneCols<VEC>;
    constexpr int kRows = POSITIONS == kGiven ? PLACES : 1;  // position rows in flight
    __shared__ typename SlabMask<VEC>::Shared shared[DROP ? kWarps : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    const uint32_t group = static_cast<uint32_t>(quotient(unit, a.slabs));
    const int slab = static_cast<int>(unit - static_cast<int64_t>(group) * a.slabs);
    const uint32_t places = PLACES * a.rounds, n = a.at.n;
    uint32_t step = 1, first = group * places, in_sequence = 0;
    if constexpr (POSITIONS == kRunning) {
        const uint32_t sequences = group / static_cast<uint32_t>(a.span);
        step = a.span;
        in_sequence = group - sequences * step;
        first = sequences * places * step + in_sequence;
    }
    wait_for_launch_before();
    if (first >= n)
        return;
    const Slab<VEC> cols(slab, lane, a.dim);
    SlabMask<VEC> mask(a.drop, slab, lane, a.dim, &shared[DROP ? warp : 0]);
    SlabGroup<TT, VEC> x[PLACES], p[kRows];
    // lane u: the token (and position) of place u of the round
    int next_token = -1, next_position = -1;
    auto fetch = [&](uint32_t round) {
        const uint64_t place = first + static_cast<uint64_t>(round * PLACES + lane) * step;
        next_token = next_position = -1;
        if (lane < PLACES && place < n) {
            next_token = token_at(a.at, place, a.status);
            if (POSITIONS == kGiven)  // an empty place's is loaded beside its token, but never an error
                next_position = position_at(a.at, place, next_token >= 0 ? a.status : nullptr);
        }
    };
    fetch(0);
    if (POSITIONS == kRunning && index_ok(a.status, a.at.first + in_sequence < a.at.npos))
        p[0].load(cols, a.pos_table.data, (a.at.first + in_sequence) * a.pos_table.stride);
    for (uint32_t round = 0; round < a.rounds; ++round) {
        int token[PLACES], position[PLACES];
#pragma unroll
        for (int u = 0; u < PLACES; ++u) {
            token[u] = __shfl_sync(kAll, next_token, u);
            if (!index_ok(a.status, token[u] < a.at.vocab))
                return;
            x[u].load(cols, a.table.data, static_cast<uint32_t>(max(token[u], 0)) * a.table.stride);
        }
        if (POSITIONS == kGiven) {
#pragma unroll
            for (int u = 0; u < PLACES; ++u) {
                position[u] = __shfl_sync(kAll, next_position, u);
                if (!index_ok(a.status, position[u] < a.at.npos))
                    return;
                p[kRows > u ? u : 0].load(cols, a.pos_table.data, static_cast<uint32_t>(max(position[u], 0)) * a.pos_table.stride);
            }
        }
        if (round + 1 < a.rounds)
            fetch(round + 1);
        if (DROP)
            mask.template draw<PLACES>(PLACES, [&](int u) { return first + (round * PLACES + u) * step; });
#pragma unroll
        for (int u = 0; u < PLACES; ++u) {
            const uint64_t place = first + static_cast<uint64_t>(round * PLACES + u) * step;
            if (place >= n)
                return;
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
            if (POSITIONS == kRunning || (POSITIONS == kGiven && position[u] >= 0)) {
                float q[N];
                p[kRows > u ? u : 0].unpack(q);
                add_pairs(y, q);
            }
            if constexpr (DROP) {
                scale_pairs(y, a.drop.rescale);
                mask.row(u, i, [&](int k, bool keep) { y[k] = keep ? y[k] : 0.0f; });
            }
            store_slab<OT, VEC>(cols, a.out.data, i * a.out.stride, y);
        }
    }
}

// Places in flight keep the memory busy (4; 2 where each has a position row of
// its own, for the registers); rounds of them hide the tokens' loads and share
// the index arithmetic and a position row, while there are warps for the SMs
// nearly once over: 64 x 1024 places of 2048 columns 101 -> 88 us with 8 rounds,
// 8 x 1024 of 768 7.5 -> 7.2 us with 2; 4907 of 771 lost by them (6.1 -> 7.0 us).
// Fewer warps than the SMs hold run one place each, for the latency.
constexpr int64_t kFewWarps = 152 * kWarps;
constexpr int64_t kManyWarps = 152 * 36;
constexpr uint32_t kMaxRounds = 8;

template <typename TT, typename OT, bool VEC, bool DROP, int PLACES, int POSITIONS>
cudaError_t launch_p(LookupArgs a, cudaStream_t s)
{
    const int64_t warps = a.at.n * static_cast<int64_t>(a.slabs), sequences = (a.at.n + a.span - 1) / a.span;
    a.rounds = 1;
    while (PLACES > 1 && a.rounds < kMaxRounds && warps > kManyWarps * PLACES * a.rounds &&
           (POSITIONS != kRunning || sequences > PLACES * a.rounds))
        a.rounds *= 2;
    const int64_t places = PLACES * a.rounds;
    const int64_t groups = POSITIONS == kRunning ? (sequences + places - 1) / places * a.span : (a.at.n + places - 1) / places;
    return launch_programmatic(k_lookup<TT, OT, VEC, DROP, PLACES, POSITIONS>,
                               static_cast<unsigned>((groups * a.slabs + kWarps - 1) / kWarps), kBlock, 0, s, a);
}

template <typename TT, typename OT, bool VEC, bool DROP>
cudaError_t launch_k(LookupArgs a, cudaStream_t s)
{
    a.slabs = slabs_of(a.dim, VEC);
    a.span = static_cast<int32_t>(a.at.seq_len < a.at.n ? a.at.seq_len : a.at.n);
    if (!a.pos_table.data)
        return a.at.n * static_cast<int64_t>(a.slabs) <= kFewWarps ? launch_p<TT, OT, VEC, DROP, 1, kNone>(a, s)
                                                                    : launch_p<TT, OT, VEC, DROP, 4, kNone>(a, s);
    if (a.at.n * static_cast<int64_t>(a.slabs) <= kFewWarps)
        return launch_p<TT, OT, VEC, DROP, 1, kGiven>(a, s);
    return a.at.positions ? launch_p<TT, OT, VEC, DROP, 2, kGiven>(a, s) : launch_p<TT, OT, VEC, DROP, 4, kRunning>(a, s);
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
