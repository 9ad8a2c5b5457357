// block_device.cuh -- element moves, 8-bit codes and sums over a row, shared by
// the block operators' kernels.  A warp works on chunks of 256 columns, 8 for
// each lane: consecutive ones where the matrices allow 16-byte moves (VEC), else
// every 32nd, so that a warp's scalar moves are contiguous.
#pragma once

#include <cuda_fp8.h>

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
    Columns() = default;
    __device__ __forceinline__ Columns(int64_t first, int lane, int64_t cols)
    {
        at = first + (VEC ? lane * 8 : lane);
        const int64_t left = cols - at;
        if (VEC)
            count = left > 0 ? 8 : 0;
        else
            count = left <= 0 ? 0 : left > 224 ? 8 : static_cast<int>((left + 31) >> 5);
    }
};

// --- a lane's 8 elements ----------------------------------------------------------------

// Of one type known to the compiler; missing ones read as 0.
template <typename T, bool VEC>
struct Chunk;

template <typename T>
struct Chunk<T, true> {
    Group8<T> g;
    __device__ __forceinline__ void load(const Columns<true>& c, const void* base, int64_t e, int)
    {
        if (c.count)
            g.load(base, e + c.at);
        else
            g = Group8<T>{};
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const { g.unpack(x); }
};

// Scalar moves are of a type that the launch gives: their widening is no burden.
template <typename T>
struct Chunk<T, false> {
    float x[8];
    __device__ __forceinline__ void load(const Columns<false>& c, const void* base, int64_t e, int type)
    {
        if (type == LIONCUB_ROWS_BF16) {
            const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + e + c.at;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < c.count ? __bfloat162float(p[32 * k]) : 0.0f;
        } else {
            const float* p = static_cast<const float*>(base) + e + c.at;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < c.count ? p[32 * k] : 0.0f;
        }
    }
    __device__ __forceinline__ void unpack(float (&y)[8]) const
    {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = x[k];
    }
};

// Loads and stores of a type that the launch gives.
template <bool VEC>
__device__ __forceinline__ void load_typed(const Columns<VEC>& c, const void* base, int64_t e, int type, float (&x)[8])
{
    if (VEC && type == LIONCUB_ROWS_F32) {
        Chunk<float, VEC> v;
        v.load(c, base, e, type);
        v.unpack(x);
    } else {
        Chunk<__nv_bfloat16, VEC> v;
        v.load(c, base, e, type);
        v.unpack(x);
    }
}

template <bool VEC>
__device__ __forceinline__ void store_typed(const Columns<VEC>& c, void* base, int64_t e, int type, const float (&x)[8])
{
    if constexpr (VEC) {
        if (!c.count)
            return;
        if (type == LIONCUB_ROWS_BF16) {
            Group8<__nv_bfloat16> g;
            g.pack(x);
            g.store(base, e + c.at);
        } else {
            Group8<float> g;
            g.pack(x);
            g.store(base, e + c.at);
        }
    } else if (type == LIONCUB_ROWS_BF16) {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + e + c.at;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < c.count)
                p[32 * k] = __float2bfloat16_rn(x[k]);
    } else {
        float* p = static_cast<float*>(base) + e + c.at;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < c.count)
                p[32 * k] = x[k];
    }
}

// --- sums and maxima over a row -------------------------------------------------------------

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int by = 16; by; by >>= 1)
        v = __fadd_rn(v, __shfl_xor_sync(kAll, v, by));
    return v;
}

// Magnitudes are compared as the numbers that their bits are: infinities come
// after all finite ones and NaN after those, so a maximum keeps them.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// --- codes of 8 bits --------------------------------------------------------------------------

// What a group's largest magnitude gives (see the header).
struct GroupScale {
    float inv, scale;
    bool bad;
    __device__ __forceinline__ GroupScale(uint32_t largest, bool e4m3)
    {
        const float a = __uint_as_float(largest);
        bad = largest >= 0x7f800000u;
        const bool none = bad || a < 0x1p-100f;
        inv = none ? 0.0f : __fdiv_rn(e4m3 ? 448.0f : 127.0f, a);
        scale = bad ? __uint_as_float(0x7fffffffu) : none ? 0.0f : __fmul_rn(a, e4m3 ? 1.0f / 448.0f : 1.0f / 127.0f);
    }
};

// Four codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const GroupScale& s, bool e4m3)
{
    a = __fmul_rn(a, s.inv);
    b = __fmul_rn(b, s.inv);
    c = __fmul_rn(c, s.inv);
    d = __fmul_rn(d, s.inv);
    uint32_t w;
    if (e4m3) {
        w = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
            static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
    } else {  // adding 1.5 * 2^23 rounds to a whole number, whose two's complement is then the lowest bits
        const float magic = 12582912.0f;
        const uint32_t ab = __byte_perm(__float_as_uint(__fadd_rn(a, magic)), __float_as_uint(__fadd_rn(b, magic)), 0x0040);
        const uint32_t cd = __byte_perm(__float_as_uint(__fadd_rn(c, magic)), __float_as_uint(__fadd_rn(d, magic)), 0x0040);
        w = __byte_perm(ab, cd, 0x5410);
    }
    return s.bad ? 0 : w;
}

// What four codes are, without their scale.
__device__ __forceinline__ void numbers4(uint32_t w, bool e4m3, float& a, float& b, float& c, float& d)
{
    if (e4m3) {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffff), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
        const float2 p = __half22float2(__half2(lo)), q = __half22float2(__half2(hi));
        a = p.x; b = p.y; c = q.x; d = q.y;
    } else {  // the byte + 128 as the lowest bits of 2^23 + it
        w ^= 0x80808080u;
        const float off = 8388736.0f;
        a = __fsub_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)), off);
        b = __fsub_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441)), off);
        c = __fsub_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)), off);
        d = __fsub_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443)), off);
    }
}

// Codes and scales of a chunk of a row whose groups lie inside chunks; x holds
// zeros where there are no columns.
template <bool VEC>
__device__ __forceinline__ void pack_chunk(const PackedRows& p, const Columns<VEC>& c, int64_t row, const float (&x)[8], int lane)
{
    float* scales = p.scales + row * p.scale_stride;
    uint8_t* codes = p.codes + row * p.stride + c.at;
    const bool e4m3 = p.e4m3;
    uint32_t m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        m[k] = magnitude(x[k]);
    if constexpr (VEC) {
        uint32_t largest = max(max(max(m[0], m[1]), max(m[2], m[3])), max(max(m[4], m[5]), max(m[6], m[7])));
        const int lanes = 1 << (p.log_group - 3);  // of a group
        for (int by = lanes >> 1; by; by >>= 1)
            largest = max(largest, __shfl_xor_sync(kAll, largest, by));
        const GroupScale s(largest, e4m3);
        if (c.count) {
            *reinterpret_cast<uint2*>(codes) = make_uint2(codes4(x[0], x[1], x[2], x[3], s, e4m3), codes4(x[4], x[5], x[6], x[7], s, e4m3));
            if ((lane & (lanes - 1)) == 0)
                scales[c.at >> p.log_group] = s.scale;
        }
    } else {  // a group is 32 lanes wide and 1 to 8 values deep
        const int deep = 1 << (p.log_group - 5);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            m[k] = __reduce_max_sync(kAll, m[k]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t largest = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((j ^ k) < deep)  // deep is a power of two: the same group
                    largest = max(largest, m[j]);
            const GroupScale s(largest, e4m3);
            if (k < c.count) {
                codes[32 * k] = static_cast<uint8_t>(codes4(x[k], 0.0f, 0.0f, 0.0f, s, e4m3));
                if (lane == 0 && (k & (deep - 1)) == 0)
                    scales[(c.at + 32 * k) >> p.log_group] = s.scale;
            }
        }
    }
}

// The same with one scale for the whole row.
template <bool VEC>
__device__ __forceinline__ void pack_chunk_of_row(const PackedRows& p, const Columns<VEC>& c, int64_t row, const float (&x)[8],
                                                  const GroupScale& s)
{
    uint8_t* codes = p.codes + row * p.stride + c.at;
    const bool e4m3 = p.e4m3;
    if constexpr (VEC) {
        if (c.count)
            *reinterpret_cast<uint2*>(codes) = make_uint2(codes4(x[0], x[1], x[2], x[3], s, e4m3), codes4(x[4], x[5], x[6], x[7], s, e4m3));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < c.count)
                codes[32 * k] = static_cast<uint8_t>(codes4(x[k], 0.0f, 0.0f, 0.0f, s, e4m3));
    }
}

// A lane's 8 codes of a chunk and their scales, as they lie in memory.
template <bool VEC>
struct CodeChunk;

template <>
struct CodeChunk<true> {
    uint2 w;
    float scale;
    __device__ __forceinline__ void load(const PackedRows& p, const Columns<true>& c, int64_t row)
    {
        w = make_uint2(0, 0);
        scale = 0.0f;
        if (c.count) {
            w = *reinterpret_cast<const uint2*>(p.codes + row * p.stride + c.at);
            scale = p.scales[row * p.scale_stride + (c.at >> p.log_group)];
        }
    }
    __device__ __forceinline__ void unpack(const PackedRows& p, float (&x)[8]) const
    {
        numbers4(w.x, p.e4m3, x[0], x[1], x[2], x[3]);
        numbers4(w.y, p.e4m3, x[4], x[5], x[6], x[7]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] = __fmul_rn(x[k], scale);
    }
};

template <>
struct CodeChunk<false> {
    float x[8];
    __device__ __forceinline__ void load(const PackedRows& p, const Columns<false>& c, int64_t row)
    {
        const uint8_t* codes = p.codes + row * p.stride + c.at;
        const float* scales = p.scales + row * p.scale_stride;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            x[k] = 0.0f;
            if (k < c.count) {
                float v, unused;
                numbers4(codes[32 * k], p.e4m3, v, unused, unused, unused);
                x[k] = __fmul_rn(v, scales[(c.at + 32 * k) >> p.log_group]);
            }
        }
    }
    __device__ __forceinline__ void unpack(const PackedRows&, float (&y)[8]) const
    {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            y[k] = x[k];
    }
};

}  // namespace lc
