// token_logprobs.cuh - what both forms of token_logprobs use: vectors of a row, powers of two, keys that order logits. Internal header.
#pragma once

#include <type_traits>

#include "decode_api.h"

namespace moe {

#ifdef __CUDACC__

constexpr float kFar = -1000.0f;  // an exponent whose power of two is 0
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 16 bytes of a row.
template <int TYPE>
struct Vec16 {
    static constexpr int W = 16 / static_cast<int>(sizeof(typename Elem<TYPE>::T));
    uint32_t w[4];
    __device__ __forceinline__ void load(const typename Elem<TYPE>::T* p) {
        const uint4 v = gload(reinterpret_cast<const uint4*>(p));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
    __device__ __forceinline__ float get(int e) const {
        if (TYPE == MOE_F32) return __uint_as_float(w[e & 3]);
        const uint32_t x = w[(e >> 1) & 3];
        if (TYPE == MOE_BF16) return __uint_as_float(e & 1 ? x & 0xffff0000u : x << 16);
        return __half2float(__ushort_as_half(static_cast<unsigned short>(e & 1 ? x >> 16 : x & 0xffffu)));
    }
};

// Larger for larger values, 0 for NaN (-0 counts as 0).
__device__ __forceinline__ uint32_t order(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x == x ? b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float unorder(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
__device__ __forceinline__ unsigned long long key_of(float x, uint32_t index) {
    const uint32_t o = order(x);
    return o ? static_cast<unsigned long long>(o) << 32 | ~index : 0ull;
}

// Keys (32 or 64 bits) in descending order over the lanes. U: unrolled so many times.
template <typename K>
__device__ __forceinline__ K other_key(K k, int o, bool more) {
    const K y = __shfl_xor_sync(0xffffffffu, k, o);
    return (k > y) == more ? k : y;
}
template <int U, typename K>
__device__ __forceinline__ K sorted_keys(K k, int lane) {
#pragma unroll U
    for (int n = 2; n <= 32; n <<= 1)
#pragma unroll U
        for (int o = n >> 1; o > 0; o >>= 1) k = other_key(k, o, !(lane & o) == !(lane & n));
    return k;
}
// The 32 largest of two such lists (y's from the end).
template <int U, typename K>
__device__ __forceinline__ K merged_keys(K k, K y, int lane) {
    k = k > y ? k : y;
#pragma unroll U
    for (int o = 16; o > 0; o >>= 1) k = other_key(k, o, !(lane & o));
    return k;
}

#endif

}  // namespace moe
