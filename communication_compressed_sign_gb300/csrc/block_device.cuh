// block_device.cuh -- element moves, 8-bit codes and sums over a row, shared by
// the block operators' kernels.  A warp works on chunks of 256 columns, 8 for
// each lane: consecutive ones where the matrices allow 16-byte moves (VEC), else
// every 32nd, so that a warp's scalar moves are contiguous.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "block.h"
#include "embed_device.cuh"

namespace lc {

constexpr int kChunk = 256;

// A lane's columns of the chunk that starts at column `first`: value k is
// column at + k (VEC) or at + 32 k, for k < count.
template <bool VEC>
struct Columns {
    int64_t at;
    int count;
    bool whole;  // all of the chunk's columns are there
    Columns() = default;
    __device__ __forceinline__ Columns(int64_t first, int lane, int64_t cols)
    {
        at = first + (VEC ? lane * 8 : lane);
        const int64_t left = cols - at;
        whole = cols - first >= kChunk;
        if (VEC)
            count = left > 0 ? 8 : 0;
        else
            count = left <= 0 ? 0 : left > 224 ? 8 : static_cast<int>((left + 31) >> 5);
    }
    __device__ __forceinline__ int64_t last() const { return VEC ? at + 7 : at + 32 * (count - 1); }
    __device__ __forceinline__ Columns none() const
    {
        Columns c = *this;
        c.count = 0;
        c.whole = false;
        return c;
    }
};

// --- checked builds ----------------------------------------------------------------------
//
// With -DLIONCUB_BOUNDS_CHECK the rows, columns, groups and moves of every access, of
// memory and of rings in shared memory, are compared with the matrices' sizes; one
// that lies outside is recorded and left out.  Elsewhere all of this is true and gone.
#ifdef LIONCUB_BOUNDS_CHECK
namespace {
__device__ int t_word;

cudaError_t take_word(int* word)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess)
        e = cudaMemcpyFromSymbol(word, t_word, sizeof *word);
    const int none = 0;
    return e == cudaSuccess ? cudaMemcpyToSymbol(t_word, &none, sizeof none) : e;
}
}  // namespace
#endif

__device__ __forceinline__ bool access_ok(bool ok)
{
#ifdef LIONCUB_BOUNDS_CHECK
    return index_ok(&t_word, ok);
#else
    return true;
#endif
}

// A lane's columns of a row.
template <bool VEC>
__device__ __forceinline__ bool inside(const TypedRows& m, const Columns<VEC>& c, int64_t row)
{
#ifdef LIONCUB_BOUNDS_CHECK
    const int64_t size = m.type == LIONCUB_ROWS_BF16 ? 2 : 4;
    const uintptr_t at = reinterpret_cast<uintptr_t>(m.data) + (row * m.stride + c.at) * size;
    return !c.count || access_ok(row >= 0 && row < m.rows && c.at >= 0 && c.last() < m.cols && at % (VEC ? 16 : size) == 0);
#else
    return true;
#endif
}
// The same of codes.
template <bool VEC>
__device__ __forceinline__ bool inside(const PackedRows& p, const Columns<VEC>& c, int64_t row)
{
#ifdef LIONCUB_BOUNDS_CHECK
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.codes) + row * p.stride + c.at;
    return !c.count || access_ok(row >= 0 && row < p.rows && c.at >= 0 && c.last() < p.cols && at % (VEC ? 8 : 1) == 0);
#else
    return true;
#endif
}
__device__ __forceinline__ bool scale_inside(const PackedRows& p, int64_t row, int64_t group)
{
#ifdef LIONCUB_BOUNDS_CHECK
    return access_ok(row >= 0 && row < p.rows && group >= 0 && group <= (p.cols - 1) >> p.log_group);
#else
    return true;
#endif
}

// --- fp32 pairs ---------------------------------------------------------------------------
//
// These kernels move so few bytes an element that instructions bound them before
// memory does, so arithmetic is done two elements an instruction (with that, maxima
// on bf16 pairs and approximate exponentials the gated activation of 16384 x 8192,
// both ways, went from 503 to 369 us).  The assembler fuses a paired product with
// a paired sum that takes it, whatever their rounding says: where the product must
// be rounded first, the sum is an fma whose other factor only the host knows.
__device__ __forceinline__ float2 add2(float2 x, float2 y) { return __fadd2_rn(x, y); }
__device__ __forceinline__ float2 mul2(float2 x, float2 y) { return __fmul2_rn(x, y); }
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) { return __ffma2_rn(x, y, z); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair_of(const float (&x)[8], int k) { return make_float2(x[2 * k], x[2 * k + 1]); }
__device__ __forceinline__ void set_pair(float (&x)[8], int k, float2 v)
{
    x[2 * k] = v.x;
    x[2 * k + 1] = v.y;
}

// --- sums and maxima over a row -------------------------------------------------------------

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int by = 16; by; by >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kAll, v, by));
    return v;
}

// The sum of what up to 16 warps left in shared memory, in every lane.
__device__ __forceinline__ float sum_of_warps(const float* part, int warps, int lane)
{
    if (warps <= 4) {  // fewer instructions and less latency than by shuffles
        float v = 0.0f;
        for (int k = 0; k < warps; ++k)
            v = __fadd_rn(v, part[k]);
        return v;
    }
    float v = (lane & 15) < warps ? part[lane & 15] : 0.0f;
#pragma unroll
    for (int by = 8; by; by >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kAll, v, by));
    return v;
}

// The largest magnitude of 8 elements, as the bits of a float: infinities come after all
// finite ones and NaN after those, so a maximum of these numbers keeps them.
__device__ __forceinline__ uint32_t largest_of(const float (&x)[8])
{
    float a, b, c;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(x[0]), "f"(x[1]), "f"(x[2]));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(b) : "f"(x[3]), "f"(x[4]), "f"(x[5]));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(c) : "f"(x[6]), "f"(x[7]), "f"(a));
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(b), "f"(c), "f"(c));
    return __float_as_uint(a);
}

// The largest over each group of 2^log_lanes lanes, at least 4.  (Masked warp
// reductions run once for each group: 32 columns a group took 31 M warp
// instructions on 8192 x 4096 elements, these 15 M.)
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int log_lanes)
{
    v = max(v, __shfl_xor_sync(kAll, v, 1));
    v = max(v, __shfl_xor_sync(kAll, v, 2));
    if (log_lanes >= 3)
        v = max(v, __shfl_xor_sync(kAll, v, 4));
    if (log_lanes >= 4)
        v = max(v, __shfl_xor_sync(kAll, v, 8));
    if (log_lanes >= 5)
        v = max(v, __shfl_xor_sync(kAll, v, 16));
    return v;
}

// --- a lane's 8 elements ----------------------------------------------------------------

// Of one type known to the compiler; missing ones read as 0.
template <typename T, bool VEC>
struct Chunk;

// Eight fp32 numbers by one move of 32 bytes where their place allows (rows of which
// do all lanes or none), so that a store fills whole sectors of memory: 8192 x 4096
// fp32 packed and unpacked 59.8 us by moves of 16 bytes, 51.5 by stores of 32; GELU of
// 788 x 768 fp32, both ways, 3.59, 3.76, and 3.57 by loads of 32 too.
__device__ __forceinline__ void load8(const float* p, Group8<float>& g)
{
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(g.a.x), "=f"(g.a.y), "=f"(g.a.z), "=f"(g.a.w), "=f"(g.b.x), "=f"(g.b.y), "=f"(g.b.z), "=f"(g.b.w)
                     : "l"(p) : "memory");
    } else {
        g.a = reinterpret_cast<const float4*>(p)[0];
        g.b = reinterpret_cast<const float4*>(p)[1];
    }
}

template <typename T>
struct Chunk<T, true> {
    Group8<T> g;
    __device__ __forceinline__ void load(const Columns<true>& c, const void* base, int64_t e, int)
    {
        if (!c.count)
            g = Group8<T>{};
        else if constexpr (sizeof(T) == 4)
            load8(static_cast<const float*>(base) + e + c.at, g);
        else
            g.load(base, e + c.at);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const { g.unpack(x); }
    // the bits of the largest magnitude (see largest_of)
    __device__ __forceinline__ uint32_t largest() const
    {
        if constexpr (sizeof(T) == 2) {
            uint32_t a, b;
            asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(g.raw.x), "r"(g.raw.y));
            asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(g.raw.z), "r"(g.raw.w));
            asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
            return max(a << 16 & 0x7fffffffu, a & 0x7fff0000u);
        } else {
            float x[8];
            g.unpack(x);
            return largest_of(x);
        }
    }
};

// Scalar moves are of a type that the launch gives: their widening is no burden.
template <typename T>
struct Chunk<T, false> {
    float x[8];
    template <typename E>
    __device__ __forceinline__ void load_of(const Columns<false>& c, const E* p)
    {
        if (c.whole) {  // without a comparison for each
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = static_cast<float>(p[32 * k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < c.count ? static_cast<float>(p[32 * k]) : 0.0f;
        }
    }
    __device__ __forceinline__ void load(const Columns<false>& c, const void* base, int64_t e, int type)
    {
        if (type == LIONCUB_ROWS_BF16)
            load_of(c, static_cast<const __nv_bfloat16*>(base) + e + c.at);
        else
            load_of(c, static_cast<const float*>(base) + e + c.at);
    }
    __device__ __forceinline__ void unpack(float (&y)[8]) const
    {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = x[k];
    }
    __device__ __forceinline__ uint32_t largest() const { return 0; }  // not used
};

// A lane's columns of a row of a matrix.
template <typename T, bool VEC>
__device__ __forceinline__ void load_row(Chunk<T, VEC>& v, const Columns<VEC>& c, const TypedRows& m, int64_t row)
{
    v.load(inside(m, c, row) ? c : c.none(), m.data, row * m.stride, m.type);
}

// Loads and stores of a type that the launch gives.
template <bool VEC>
__device__ __forceinline__ void load_typed(const Columns<VEC>& c, const TypedRows& m, int64_t row, float (&x)[8])
{
    if (VEC && m.type == LIONCUB_ROWS_F32) {
        Chunk<float, VEC> v;
        load_row(v, c, m, row);
        v.unpack(x);
    } else {
        Chunk<__nv_bfloat16, VEC> v;
        load_row(v, c, m, row);
        v.unpack(x);
    }
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8])
{
    if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store_typed(const Columns<VEC>& c, const TypedRows& m, int64_t row, const float (&x)[8])
{
    if (!inside(m, c, row))
        return;
    const int64_t e = row * m.stride;
    if constexpr (VEC) {
        if (!c.count)
            return;
        if (m.type == LIONCUB_ROWS_BF16) {
            Group8<__nv_bfloat16> g;
            g.pack(x);
            g.store(m.data, e + c.at);
        } else {
            store8(static_cast<float*>(m.data) + e + c.at, x);
        }
    } else {
        const auto store = [&](auto* p) {
            using E = std::remove_pointer_t<decltype(p)>;
            if (c.whole) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    p[32 * k] = static_cast<E>(x[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < c.count)
                        p[32 * k] = static_cast<E>(x[k]);
            }
        };
        if (m.type == LIONCUB_ROWS_BF16)
            store(static_cast<__nv_bfloat16*>(m.data) + e + c.at);
        else
            store(static_cast<float*>(m.data) + e + c.at);
    }
}

// --- codes of 8 bits --------------------------------------------------------------------------

// What a group's largest magnitude gives (see the header).
struct GroupScale {
    float inv, scale;
    bool bad;
    __device__ __forceinline__ GroupScale(uint32_t largest, bool e4m3)
    {
        constexpr uint32_t kSmallest = 0x0d800000u, kInfinity = 0x7f800000u;  // 2^-100
        const float a = __uint_as_float(largest);
        const bool some = largest - kSmallest < kInfinity - kSmallest;
        bad = largest >= kInfinity;
        inv = some ? __fdiv_rn(e4m3 ? 448.0f : 127.0f, a) : 0.0f;
        scale = some ? __fmul_rn(a, e4m3 ? 1.0f / 448.0f : 1.0f / 127.0f) : __uint_as_float(bad ? 0x7fffffffu : 0u);
    }
};

// Eight codes, the first in the lowest byte.  The paths are kept apart by asm
// that may not be moved: computing both and choosing costs more than the branch.
__device__ __forceinline__ uint32_t e4m3_pairs(float2 a, float2 b)
{
    uint32_t w;
    asm volatile("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
                 "mov.b32 %0, {lo, hi};\n\t}" : "=r"(w) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return w;
}
// 1.5 * 2^23 more is rounded to a whole number, whose two's complement is then the
// lowest bits.  `one` is 1, which only the host knows: the products stay rounded.
__device__ __forceinline__ uint32_t int8_pairs(float2 a, float2 b, float one)
{
    const float2 magic = both(12582912.0f);
    a = fma2(a, both(one), magic);
    b = fma2(b, both(one), magic);
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv, bool bad, const PackedRows& p)
{
    uint2 w;
    float2 y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        y[k] = mul2(pair_of(x, k), both(inv));
    if (p.e4m3)
        w = make_uint2(e4m3_pairs(y[0], y[1]), e4m3_pairs(y[2], y[3]));
    else
        w = make_uint2(int8_pairs(y[0], y[1], p.one), int8_pairs(y[2], y[3], p.one));
    if (bad)
        w = make_uint2(0, 0);
    return w;
}

// Two codes, in the lowest bytes of either number.
__device__ __forceinline__ void codes2(float2 x, float inv, const PackedRows& p, uint32_t& a, uint32_t& b)
{
    x = mul2(x, both(inv));
    if (p.e4m3) {
        uint16_t w;
        asm volatile("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(w) : "f"(x.x), "f"(x.y));
        a = w;
        b = w >> 8;
    } else {
        x = fma2(x, both(p.one), both(12582912.0f));
        a = __float_as_uint(x.x);
        b = __float_as_uint(x.y);
    }
}

// What eight codes stand for.
__device__ __forceinline__ void restore4(uint32_t w, bool e4m3, float scale, float2& a, float2& b)
{
    if (e4m3) {
        a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffff), __NV_E4M3)));
        b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3)));
    } else {  // the byte + 128 as the lowest bits of 2^23 + it
        w ^= 0x80808080u;
        const float2 off = both(-8388736.0f);
        a = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)), __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))), off);
        b = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)), __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443))), off);
    }
    a = mul2(a, both(scale));
    b = mul2(b, both(scale));
}
__device__ __forceinline__ void restore8(uint2 w, bool e4m3, float scale, float (&x)[8])
{
    float2 a, b;
    restore4(w.x, e4m3, scale, a, b);
    set_pair(x, 0, a);
    set_pair(x, 1, b);
    restore4(w.y, e4m3, scale, a, b);
    set_pair(x, 2, a);
    set_pair(x, 3, b);
}

// What one code stands for.
__device__ __forceinline__ float restore1(uint32_t code, bool e4m3, float scale)
{
    const float v = e4m3 ? __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)))
                         : __fsub_rn(__uint_as_float((code ^ 0x80u) | 0x4b000000u), 8388736.0f);
    return __fmul_rn(v, scale);
}

// Codes and scales of a chunk of a row whose groups lie inside chunks; x holds
// zeros where there are no columns.  largest: of x (VEC).
template <bool VEC>
__device__ __forceinline__ void pack_chunk(const PackedRows& p, const Columns<VEC>& c, int64_t row, const float (&x)[8], uint32_t largest,
                                           int lane)
{
    float* scales = p.scales + row * p.scale_stride;
    uint8_t* codes = p.codes + row * p.stride + c.at;
    const bool e4m3 = p.e4m3;
    if constexpr (VEC) {
        const int log_lanes = p.log_group - 3;  // of a group
        const GroupScale s(lanes_max(largest, log_lanes), e4m3);
        const uint2 w = codes8(x, s.inv, s.bad, p);
        if (c.count && inside(p, c, row)) {
            *reinterpret_cast<uint2*>(codes) = w;
            if ((lane & ((1 << log_lanes) - 1)) == 0 && scale_inside(p, row, c.at >> p.log_group))
                scales[c.at >> p.log_group] = s.scale;
        }
    } else {
        // a group is 32 lanes wide and 1 to 8 values deep
        const auto pack = [&](auto d) {
            constexpr int kDeep = decltype(d)::value, kGroups = 8 / kDeep;
            uint32_t m = 0;  // lane g: the largest of group g
            const int mine = lane & (kGroups - 1);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float v = x[g * kDeep];
#pragma unroll
                for (int k = 1; k < kDeep; k += 2)  // three at a time
                    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(v) : "f"(x[g * kDeep + k]), "f"(x[g * kDeep + (k + 1 < kDeep ? k + 1 : k)]));
                const uint32_t all = __reduce_max_sync(kAll, __float_as_uint(v) & 0x7fffffffu);
                m = mine == g ? all : m;
            }
            const GroupScale s(m, e4m3);
            const int64_t at = c.at - lane + 32 * kDeep * mine;  // the group's first column
            if (lane < kGroups && at < p.cols && scale_inside(p, row, at >> p.log_group))
                scales[at >> p.log_group] = s.scale;
            const bool ok = inside(p, c, row);
            if (c.whole && (!kBoundsCheck || __all_sync(kAll, ok)) && !__any_sync(kAll, s.bad)) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const float inv = __shfl_sync(kAll, s.inv, g);
                    if constexpr (kDeep == 1) {
                        uint32_t code, unused;
                        codes2(make_float2(x[g], 0.0f), inv, p, code, unused);
                        codes[32 * g] = static_cast<uint8_t>(code);
                    } else {
#pragma unroll
                        for (int k = g * kDeep; k < (g + 1) * kDeep; k += 2) {
                            uint32_t a, b;
                            codes2(make_float2(x[k], x[k + 1]), inv, p, a, b);
                            codes[32 * k] = static_cast<uint8_t>(a);
                            codes[32 * k + 32] = static_cast<uint8_t>(b);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const float inv = __shfl_sync(kAll, s.inv, g);
                    const bool none = __shfl_sync(kAll, s.bad, g);
#pragma unroll
                    for (int k = g * kDeep; k < (g + 1) * kDeep; ++k)
                        if (k < c.count && ok) {
                            uint32_t code, unused;
                            codes2(make_float2(x[k], 0.0f), inv, p, code, unused);
                            codes[32 * k] = none ? 0 : static_cast<uint8_t>(code);
                        }
                }
            }
        };
        switch (p.log_group) {
        case 5: pack(std::integral_constant<int, 1>()); break;
        case 6: pack(std::integral_constant<int, 2>()); break;
        case 7: pack(std::integral_constant<int, 4>()); break;
        default: pack(std::integral_constant<int, 8>()); break;
        }
    }
}

// The same with one scale for the whole row.
template <bool VEC>
__device__ __forceinline__ void pack_chunk_of_row(const PackedRows& p, const Columns<VEC>& c, int64_t row, const float (&x)[8],
                                                  const GroupScale& s)
{
    uint8_t* codes = p.codes + row * p.stride + c.at;
    if (!inside(p, c, row))
        return;
    if constexpr (VEC) {
        if (c.count)
            *reinterpret_cast<uint2*>(codes) = codes8(x, s.inv, s.bad, p);
    } else {
        const bool plain = c.whole && !s.bad;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            uint32_t a, b;
            codes2(make_float2(x[k], x[k + 1]), s.inv, p, a, b);
            if (plain) {
                codes[32 * k] = static_cast<uint8_t>(a);
                codes[32 * k + 32] = static_cast<uint8_t>(b);
            } else {
                if (k < c.count)
                    codes[32 * k] = s.bad ? 0 : static_cast<uint8_t>(a);
                if (k + 1 < c.count)
                    codes[32 * k + 32] = s.bad ? 0 : static_cast<uint8_t>(b);
            }
        }
    }
}

// A lane's 8 codes of a chunk and their scales.
template <bool VEC>
struct CodeChunk;

template <>
struct CodeChunk<true> {
    uint2 w;
    float scale;
    __device__ __forceinline__ void load(const PackedRows& p, const Columns<true>& c, int64_t row, int)
    {
        w = make_uint2(0, 0);
        scale = 0.0f;
        if (c.count && inside(p, c, row) && scale_inside(p, row, c.at >> p.log_group)) {
            w = *reinterpret_cast<const uint2*>(p.codes + row * p.stride + c.at);
            scale = p.scales[row * p.scale_stride + (c.at >> p.log_group)];
        }
    }
    __device__ __forceinline__ void unpack(const PackedRows& p, float (&x)[8]) const { restore8(w, p.e4m3, scale, x); }
};

template <>
struct CodeChunk<false> {
    uint32_t code[8];
    float scale;  // of value lane % 8
    __device__ __forceinline__ void load(const PackedRows& p, const Columns<false>& c, int64_t row, int lane)
    {
        const uint8_t* codes = p.codes + row * p.stride + c.at;
        const int64_t at = c.at - lane + 32 * (lane & 7);
        scale = at < p.cols && scale_inside(p, row, at >> p.log_group) ? p.scales[row * p.scale_stride + (at >> p.log_group)] : 0.0f;
        const bool ok = inside(p, c, row);
        if (c.whole && ok) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                code[k] = codes[32 * k];
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                code[k] = k < c.count && ok ? codes[32 * k] : 0;
        }
    }
    __device__ __forceinline__ void unpack(const PackedRows& p, float (&y)[8]) const
    {
        if (p.e4m3) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                y[k] = restore1(code[k], true, __shfl_sync(kAll, scale, k));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                y[k] = restore1(code[k], false, __shfl_sync(kAll, scale, k));
        }
    }
};

}  // namespace lc
