// embed_device.cuh -- element moves, the dropout mask and place lookups shared
// by the input-layer kernels.  As in device_common.cuh, every float operation
// rounds once to nearest and no product is fused with a sum.
#pragma once

#include "device_common.cuh"
#include "embed.h"
#include "splitmix64.cuh"

namespace lc {

constexpr unsigned kAll = 0xffffffffu;

// --- programmatic launches -------------------------------------------------------------
//
// The operators' kernels may start before the launch before them in the stream
// has ended (the gap between two launches is a good part of a small one's
// time: a decoding step's lookup 1.9 -> 1.6 us).  They touch no memory that
// others use until wait_for_launch_before() returns: all of that launch, and of
// what it waited for, is then done and visible.  (A gradient's running positions
// need nothing of the launch before theirs, only what was there before that: see
// wait_until_begun.)  let_next_launch_start() lets
// the blocks of the next launch start beside this one's, which only the sort
// wants (the lookup and dropout gained nothing or lost).
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A launch may hand on before it ends that those before it are done.  One of its
// threads, which has waited and so sees what they wrote, stores the call's number
// in a word (release); a warp of the next launch that reads that number there
// (acquire) comes after the thread, and so after all that the thread had waited
// for.  That the next launch was let start says nothing of memory.  A warp that
// does not find the number waits like any other, so none ever waits for the word.
__device__ __forceinline__ void tell_begun(uint32_t* begun, uint32_t call)
{
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(begun), "r"(call) : "memory");
}
__device__ __forceinline__ void wait_until_begun(const uint32_t* begun, uint32_t call, int lane)
{
    uint32_t found = 0;
    if (lane == 0)
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(found) : "l"(begun) : "memory");
    __syncwarp();  // what lane 0 acquired is the other lanes' too
    if (__shfl_sync(kAll, found, 0) != call)
        wait_for_launch_before();
}

template <typename Kernel, typename... Args>
cudaError_t launch_programmatic_clusters(Kernel kernel, unsigned blocks, int threads, unsigned cluster, size_t shared, cudaStream_t s,
                                         const Args&... args)
{
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(blocks);
    c.blockDim = dim3(static_cast<unsigned>(threads));
    c.dynamicSmemBytes = shared;
    c.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

template <typename Kernel, typename... Args>
cudaError_t launch_programmatic(Kernel kernel, unsigned blocks, int threads, size_t shared, cudaStream_t s, const Args&... args)
{
    return launch_programmatic_clusters(kernel, blocks, threads, 1, shared, s, args...);
}

// --- 8 consecutive, 16-byte aligned elements ------------------------------------------

// The elements as they lie in memory, so that groups waiting in registers take
// no more room than they did there.
template <typename T>
struct Group8;

template <>
struct Group8<__nv_bfloat16> {
    uint4 raw;
    __device__ __forceinline__ void load(const void* base, int64_t e)
    {
        raw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + e);
    }
    __device__ __forceinline__ void store(void* base, int64_t e) const
    {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e) = raw;
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const
    {
        x[0] = bf16_bits_lo(raw.x); x[1] = bf16_bits_hi(raw.x);
        x[2] = bf16_bits_lo(raw.y); x[3] = bf16_bits_hi(raw.y);
        x[4] = bf16_bits_lo(raw.z); x[5] = bf16_bits_hi(raw.z);
        x[6] = bf16_bits_lo(raw.w); x[7] = bf16_bits_hi(raw.w);
    }
    static __device__ __forceinline__ uint32_t pair(float lo, float hi)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    __device__ __forceinline__ void pack(const float (&x)[8])
    {
        raw = make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7]));
    }
};

template <>
struct Group8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t e)
    {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + e);
        a = p[0];
        b = p[1];
    }
    __device__ __forceinline__ void store(void* base, int64_t e) const
    {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e);
        p[0] = a;
        p[1] = b;
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void pack(const float (&x)[8])
    {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// --- a warp on a slab of a row --------------------------------------------------------
//
// Where the matrices allow 16-byte moves (VEC) a slab is 256 columns, 8 in a
// row for each lane.  Else it is 224, every 32nd from a lane's own, so that a
// warp's scalar moves are contiguous; 224 rather than 256 because its elements
// then touch 57 outputs of the generator at most, two for each lane.

template <bool VEC>
constexpr int kLaneCols = VEC ? 8 : 7;
template <bool VEC>
constexpr int kSlabCols = 32 * kLaneCols<VEC>;

template <bool VEC>
struct Slab;

template <>
struct Slab<true> {
    int col;
    bool on;
    __device__ __forceinline__ Slab(int slab, int lane, int dim) : col(slab * 256 + lane * 8), on(col < dim) {}
};

template <>
struct Slab<false> {
    int col;
    int count;  // columns of this lane: col, col + 32, ...
    __device__ __forceinline__ Slab(int slab, int lane, int dim) : col(slab * 224 + lane)
    {
        const int left = dim - col;
        count = left <= 0 ? 0 : (left > 192 ? 7 : (left + 31) / 32);
    }
};

// A lane's elements of the row that starts at element e.
template <typename T, bool VEC>
struct SlabGroup;

template <typename T>
struct SlabGroup<T, true> {
    Group8<T> g;
    __device__ __forceinline__ void load(const Slab<true>& c, const void* base, int64_t e)
    {
        if (c.on)
            g.load(base, e + c.col);
        else
            g = Group8<T>{};
    }
    __device__ __forceinline__ void store(const Slab<true>& c, void* base, int64_t e) const
    {
        if (c.on)
            g.store(base, e + c.col);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const { g.unpack(x); }
    __device__ __forceinline__ void pack(const float (&x)[8]) { g.pack(x); }
};

template <typename T>
struct SlabGroup<T, false> {
    T x[7];
    __device__ __forceinline__ void load(const Slab<false>& c, const void* base, int64_t e)
    {
        const T* p = static_cast<const T*>(base) + e + c.col;
        if (c.count == 7) {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                x[k] = p[32 * k];
        } else {
#pragma unroll
            for (int k = 0; k < 7; ++k)
                x[k] = k < c.count ? p[32 * k] : T(0.0f);
        }
    }
    __device__ __forceinline__ void store(const Slab<false>& c, void* base, int64_t e) const
    {
        T* p = static_cast<T*>(base) + e + c.col;
#pragma unroll
        for (int k = 0; k < 7; ++k)
            if (k < c.count)
                p[32 * k] = x[k];
    }
    __device__ __forceinline__ void unpack(float (&y)[7]) const
    {
#pragma unroll
        for (int k = 0; k < 7; ++k)
            y[k] = static_cast<float>(x[k]);
    }
    __device__ __forceinline__ void pack(const float (&y)[7])
    {
#pragma unroll
        for (int k = 0; k < 7; ++k) {
            if constexpr (sizeof(T) == 2)
                x[k] = __float2bfloat16_rn(y[k]);
            else
                x[k] = y[k];
        }
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_slab(const Slab<VEC>& c, void* base, int64_t e, const float (&x)[kLaneCols<VEC>])
{
    SlabGroup<T, VEC> g;
    g.pack(x);
    g.store(c, base, e);
}

// --- the dropout mask -------------------------------------------------------------
//
// One output of the generator serves 4 elements, 16 bits each: a draw per
// element would make bf16 streams bound by integer instructions instead of
// memory.  Output k comes from the state key + (k + 1) * gamma, so states are
// stepped by additions and the product with gamma is paid once a row or thread.

// Whether the two 16-bit fields of a word stay.  The upper one decides the
// comparison of the whole word by itself, the lower one is moved up.  (The
// two-halves maximum instruction that also gives both comparisons measured 12 %
// slower on a bf16 dropout.)
__device__ __forceinline__ bool lower_stays(const DropArgs& d, uint32_t w) { return w << 16 > d.limit; }
__device__ __forceinline__ bool upper_stays(const DropArgs& d, uint32_t w) { return w > d.limit; }

// f(k, whether element k stays) for 8 elements whose first output has the
// state z (the element number is a multiple of 4).
template <typename F>
__device__ __forceinline__ void for_kept8(const DropArgs& d, uint64_t z, F&& f)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint64_t u = splitmix64_mix(z + h * kSplitMix64Step);
        const uint32_t lo = static_cast<uint32_t>(u), hi = static_cast<uint32_t>(u >> 32);
        f(4 * h, lower_stays(d, lo));
        f(4 * h + 1, upper_stays(d, lo));
        f(4 * h + 2, lower_stays(d, hi));
        f(4 * h + 3, upper_stays(d, hi));
    }
}

// fp32 additions that take one operand in bf16 (exact: the operand is widened,
// the sum rounded once), so that elements need no unpacking; with a mask, one
// comparison and one predicated addition an element.  10 % fewer instructions
// than unpacking in a pass that integer instructions bound.
__device__ __forceinline__ void add_bf16(float& sum, uint32_t x)
{
    asm("add.rn.f32.bf16 %0, %1, %0;" : "+f"(sum) : "h"(static_cast<unsigned short>(x)));
}
// the same where word > limit
__device__ __forceinline__ void add_bf16_where(float& sum, uint32_t x, uint32_t word, uint32_t limit)
{
    asm("{\n\t.reg .pred p;\n\tsetp.gt.u32 p, %2, %3;\n\t@p add.rn.f32.bf16 %0, %1, %0;\n\t}"
        : "+f"(sum) : "h"(static_cast<unsigned short>(x)), "r"(word), "r"(limit));
}

// The mask of a lane's columns of a slab, row by row.
template <bool VEC>
struct SlabMask;

// dim is a multiple of 4 here, so a row's first output is a whole step from
// the next row's: state = first + row * d.row_step + column / 4 * gamma.
template <>
struct SlabMask<true> {
    struct Shared {};
    const DropArgs& d;
    uint64_t z;
    __device__ __forceinline__ SlabMask(const DropArgs& args, int slab, int lane, int, Shared*)
        : d(args), z(args.first + static_cast<uint64_t>(slab * 64 + lane * 2) * kSplitMix64Step)
    {
    }
    template <int ROWS, typename Row>
    __device__ __forceinline__ void draw(int, Row&&)
    {
    }
    template <typename F>
    __device__ __forceinline__ void row(int, uint32_t i, F&& f)
    {
        for_kept8(d, z + i * d.row_step, f);
    }
    __device__ __forceinline__ void add(int, uint32_t i, const SlabGroup<__nv_bfloat16, true>& x, float (&sum)[8])
    {
        const uint64_t at = z + i * d.row_step;
        const uint32_t w[4] = {x.g.raw.x, x.g.raw.y, x.g.raw.z, x.g.raw.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint64_t u = splitmix64_mix(at + h * kSplitMix64Step);
            const uint32_t lo = static_cast<uint32_t>(u), hi = static_cast<uint32_t>(u >> 32);
            add_bf16_where(sum[4 * h], w[2 * h] & 0xffff, lo << 16, d.limit);
            add_bf16_where(sum[4 * h + 1], w[2 * h] >> 16, lo, d.limit);
            add_bf16_where(sum[4 * h + 2], w[2 * h + 1] & 0xffff, hi << 16, d.limit);
            add_bf16_where(sum[4 * h + 3], w[2 * h + 1] >> 16, hi, d.limit);
        }
    }
};

// A row may begin inside an output's four elements.  The warp draws the outputs
// that a slab's 224 elements can touch once, into shared memory; there the
// elements' fields lie one after the other, 16 bits each.  Rows are drawn a few
// at a time: 16384 rows of 771 bf16 elements, 776 apart, 15.6 us, and 18.9 drawn
// one by one.
template <>
struct SlabMask<false> {
    struct Shared {
        uint64_t outputs[4][64];
    };
    const DropArgs& d;
    Shared* shared;
    uint32_t dim, first_col, lane;
    __device__ __forceinline__ SlabMask(const DropArgs& args, int slab, int l, int width, Shared* buffers)
        : d(args), shared(buffers), dim(width), first_col(slab * 224), lane(l)
    {
    }
    // draws for rows row(0) .. row(count - 1), ROWS of them at most, whose latencies overlap
    template <int ROWS, typename Row>
    __device__ __forceinline__ void draw(int count, Row&& row)
    {
        static_assert(ROWS <= 4, "rows of outputs");
        __syncwarp();  // what was drawn before is used
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            if (u >= count)
                break;
            const uint64_t e = static_cast<uint64_t>(static_cast<uint32_t>(row(u))) * dim + first_col;
            const uint64_t z = d.first + ((e >> 2) + lane) * kSplitMix64Step;
            shared->outputs[u][lane] = splitmix64_mix(z);
            shared->outputs[u][lane + 32] = splitmix64_mix(z + 32 * kSplitMix64Step);
        }
        __syncwarp();
    }
    // the lane's fields of the u-th row drawn, row i: of its column k at [32 k]
    __device__ __forceinline__ const uint16_t* fields(int u, uint32_t i) const
    {
        return reinterpret_cast<const uint16_t*>(shared->outputs[u]) + ((i * dim + first_col) & 3) + lane;
    }
    template <typename F>
    __device__ __forceinline__ void row(int u, uint32_t i, F&& f)
    {
        const uint16_t* field = fields(u, i);
#pragma unroll
        for (int k = 0; k < 7; ++k)
            f(k, field[32 * k] > d.limit >> 16);
    }
    __device__ __forceinline__ void add(int u, uint32_t i, const SlabGroup<__nv_bfloat16, false>& x, float (&sum)[7])
    {
        const uint16_t* field = fields(u, i);
#pragma unroll
        for (int k = 0; k < 7; ++k)
            add_bf16_where(sum[k], __bfloat16_as_ushort(x.x[k]), field[32 * k], d.limit >> 16);
    }
};

// --- places --------------------------------------------------------------------------

// a / b for a >= 0: 64-bit division takes about five times the instructions of a
// 32-bit one, which is nearly always enough.
__device__ __forceinline__ int64_t quotient(int64_t a, int b)
{
    return a <= 0xffffffffll ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

__device__ __forceinline__ int64_t index_at(const void* p, int64_t i, int wide)
{
    return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

__device__ __forceinline__ void flag(int* status, int bit)
{
    if (status)
        atomicOr(status, bit);
}

// The token of place i, or -1 for an empty place (an id beyond the table
// counts as one and is recorded).
__device__ __forceinline__ int32_t token_at(const Places& at, int64_t i, int* status)
{
    const int64_t t = index_at(at.tokens, i, at.wide);
    if (t >= at.vocab) {
        flag(status, kStatusIndex);
        return -1;
    }
    return t < 0 ? -1 : static_cast<int32_t>(t);
}

// The position row of place i, or -1 when it is outside the table (recorded).
__device__ __forceinline__ int32_t position_at(const Places& at, int64_t i, int* status)
{
    const int64_t q = at.positions ? index_at(at.positions, i, at.wide)
                                   : at.first + static_cast<uint32_t>(i) % static_cast<uint32_t>(at.seq_len);
    if (q < 0 || q >= at.npos) {
        flag(status, kStatusIndex);
        return -1;
    }
    return static_cast<int32_t>(q);
}

// Checked builds: records an index outside its buffer; the access is skipped.
__device__ __forceinline__ bool index_ok(int* status, bool ok)
{
    if constexpr (kBoundsCheck) {
        if (!ok)
            flag(status, kStatusOutOfBounds);
        return ok;
    }
    return true;
}

}  // namespace lc
