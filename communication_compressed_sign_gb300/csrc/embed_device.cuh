// embed_device.cuh -- element moves, the dropout mask and place lookups shared
// by the input-layer kernels.  As in device_common.cuh, every float operation
// is an explicit round-to-nearest intrinsic.
#pragma once

#include "device_common.cuh"
#include "embed.h"
#include "splitmix64.cuh"

namespace lc {

// --- V consecutive elements of a row <-> floats ---------------------------------

// The elements as they lie in memory, so that groups waiting in registers take
// no more room than they did there.
template <typename T, int V>
struct Group {
    static_assert(V == 1, "one element or a 16-byte aligned group of 8");
    T raw;
    __device__ __forceinline__ void load(const void* base, int64_t e) { raw = static_cast<const T*>(base)[e]; }
    __device__ __forceinline__ void unpack(float (&x)[1]) const { x[0] = static_cast<float>(raw); }
};

template <>
struct Group<__nv_bfloat16, 8> {
    uint4 raw;
    __device__ __forceinline__ void load(const void* base, int64_t e)
    {
        raw = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + e);
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const
    {
        x[0] = bf16_bits_lo(raw.x); x[1] = bf16_bits_hi(raw.x);
        x[2] = bf16_bits_lo(raw.y); x[3] = bf16_bits_hi(raw.y);
        x[4] = bf16_bits_lo(raw.z); x[5] = bf16_bits_hi(raw.z);
        x[6] = bf16_bits_lo(raw.w); x[7] = bf16_bits_hi(raw.w);
    }
};

template <>
struct Group<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* base, int64_t e)
    {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + e);
        a = p[0];
        b = p[1];
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

template <typename T, int V>
__device__ __forceinline__ void load_row(const void* base, int64_t e, float (&x)[V])
{
    Group<T, V> g;
    g.load(base, e);
    g.unpack(x);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T, int V>
__device__ __forceinline__ void store_row(void* base, int64_t e, const float (&x)[V])
{
    if constexpr (V == 8 && sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e) =
            make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
    } else if constexpr (V == 8) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + e);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else if constexpr (sizeof(T) == 2) {
        static_cast<__nv_bfloat16*>(base)[e] = __float2bfloat16_rn(x[0]);
    } else {
        static_cast<float*>(base)[e] = x[0];
    }
}

// --- the dropout mask -------------------------------------------------------------

// Bit j set: element e + j stays (e a multiple of 8 when V == 8).  One output
// of the generator serves 4 elements, 16 bits each: two 64-bit products for 4
// elements, where a draw per element would make bf16 streams bound by integer
// instructions instead of memory.
template <int V>
__device__ __forceinline__ uint32_t keep_bits(const DropArgs& d, uint64_t e)
{
    if constexpr (V == 8) {
        uint32_t keep = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint64_t u = splitmix64(d.key, (e >> 2) + h);
            const uint32_t lo = static_cast<uint32_t>(u), hi = static_cast<uint32_t>(u >> 32);
            keep |= (lo << 16 > d.limit ? 1u : 0u) << (4 * h);
            keep |= (lo > d.limit ? 2u : 0u) << (4 * h);
            keep |= (hi << 16 > d.limit ? 4u : 0u) << (4 * h);
            keep |= (hi > d.limit ? 8u : 0u) << (4 * h);
        }
        return keep;
    } else {
        const uint64_t u = splitmix64(d.key, e >> 2);
        const uint32_t f = static_cast<uint32_t>(u >> (16 * (e & 3)));
        return f << 16 > d.limit ? 1u : 0u;
    }
}

// --- places --------------------------------------------------------------------------

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
    const int64_t q = at.positions ? index_at(at.positions, i, at.wide) : at.first + i % at.seq_len;
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
