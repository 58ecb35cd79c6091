// kv8.cuh - the 8-bit key/value cache's record layout and the dense rows' element types, shared by
// the cache, attention and norm kernels. Internal header (not part of the C ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "moe_kv8.h"

namespace moe {

// These kernels may start before the one they follow has ended (they wait for it before they touch
// memory), so what they read is not constant over their lifetime: plain loads, not the read-only path.
template <typename T>
__device__ __forceinline__ T gload(const T* p) {
    return *p;
}

constexpr int kKvBlock = 32;                  // tokens of a record
constexpr int kKvNoWindow = 0x7fffffff - 63;  // a window of as many positions is none (and a position less it fits in 32 bits)
constexpr int kKvHead = 16;                   // record header: f32 k_scale, f32 v_scale, 8 unused
constexpr float kKvTiny = 7.888609052210118e-31f;  // 2^-100: a block below it is stored as zeros

__host__ __device__ constexpr int kv8_record_bytes(int D) { return kKvHead + 2 * kKvBlock * D; }

// byte of the key code (token t, dim d) and of the value code in a record
__device__ __forceinline__ int kv8_k_at(int D, int t, int d) {
    return kKvHead + ((((t >> 1) & 3) * (D >> 5) + (d >> 5)) * 8 + 2 * (t >> 3) + (t & 1)) * 32 + (d & 31);
}
__device__ __forceinline__ int kv8_v_at(int D, int t, int d) { return kKvHead + kKvBlock * D + d * kKvBlock + t; }

template <int TYPE>
struct Elem;
template <>
struct Elem<MOE_F32> {
    using T = float;
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<MOE_F16> {
    using T = __half;
    static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<MOE_BF16> {
    using T = __nv_bfloat16;
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// Eight consecutive elements; vec: p is 16-byte aligned.
template <int TYPE>
__device__ __forceinline__ void load8(const typename Elem<TYPE>::T* p, bool vec, float (&v)[8]) {
    using E = Elem<TYPE>;
    constexpr int kB = 8 * sizeof(typename E::T);
    union {
        typename E::T e[8];
        uint4 w[kB / 16];
    } u;
    if (vec) {
#pragma unroll
        for (int i = 0; i < kB / 16; ++i) u.w[i] = gload(reinterpret_cast<const uint4*>(p) + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) u.e[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = E::get(u.e[i]);
}

template <int TYPE>
__device__ __forceinline__ void store8(typename Elem<TYPE>::T* p, bool vec, const float (&v)[8]) {
    using E = Elem<TYPE>;
    constexpr int kB = 8 * sizeof(typename E::T);
    union U {
        typename E::T e[8];
        uint4 w[kB / 16];
        __device__ U() {}
    } u;
#pragma unroll
    for (int i = 0; i < 8; ++i) u.e[i] = E::put(v[i]);
    if (vec) {
#pragma unroll
        for (int i = 0; i < kB / 16; ++i) reinterpret_cast<uint4*>(p)[i] = u.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = u.e[i];
    }
}

// store8, where `on`, by a whole warp in which lanes l and l ^ X (the one without bit X first) store neighbouring
// eights of one row, both or neither. In fp32 a lane's two vectors lie 32 bytes from the next lane's, so that each store would fill
// half of every sector; the lanes exchange halves first, and each store fills whole ones.
template <int TYPE, int X>
__device__ __forceinline__ void store8_pair(typename Elem<TYPE>::T* p, bool vec, const float (&v)[8], bool on) {
    if constexpr (TYPE == MOE_F32) {
        if (vec) {
            const bool second = threadIdx.x & X;
            float r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __shfl_xor_sync(0xffffffffu, second ? v[i] : v[4 + i], X);
            if (!on) return;
            float* at = second ? p - 4 : p;
            *reinterpret_cast<float4*>(at) = second ? make_float4(r[0], r[1], r[2], r[3]) : make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(at + 8) = second ? make_float4(v[4], v[5], v[6], v[7]) : make_float4(r[0], r[1], r[2], r[3]);
            return;
        }
    }
    if (on) store8<TYPE>(p, vec, v);
}

// max of non-negative values that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Eight consecutive elements as they lie in memory.
template <int TYPE>
struct Raw8 {
    static constexpr int kWords = 2 * static_cast<int>(sizeof(typename Elem<TYPE>::T));
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const typename Elem<TYPE>::T* p, bool vec) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = gload(reinterpret_cast<const uint4*>(p) + i);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else if (TYPE == MOE_F32) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = gload(reinterpret_cast<const uint32_t*>(p) + i);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = gload(reinterpret_cast<const uint16_t*>(p) + 2 * i) |
                       static_cast<uint32_t>(gload(reinterpret_cast<const uint16_t*>(p) + 2 * i + 1)) << 16;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int e) const {
        if (TYPE == MOE_F32) return __uint_as_float(w[e & (kWords - 1)]);
        const uint32_t x = w[(e >> 1) & (kWords - 1)];
        return TYPE == MOE_BF16 ? __uint_as_float(e & 1 ? x & 0xffff0000u : x << 16) : half(e);
    }
    __device__ __forceinline__ float half(int e) const {  // of 16-bit words that hold fp16
        const uint32_t x = w[(e >> 1) & (kWords - 1)];
        return __half2float(__ushort_as_half(static_cast<unsigned short>(e & 1 ? x >> 16 : x & 0xffffu)));
    }
    // The running maximum of magnitudes, as bits (a NaN is above all): of one value, or of two 16-bit halves.
    __device__ __forceinline__ uint32_t amax(uint32_t m) const {
        if constexpr (TYPE == MOE_F32) {
            float f = __uint_as_float(m);
#pragma unroll
            for (int i = 0; i < kWords; ++i) f = max_nan(f, fabsf(__uint_as_float(w[i])));
            return __float_as_uint(f);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            return m;
        }
    }
    static __device__ __forceinline__ uint32_t float_bits(uint32_t m) {  // of amax(), as fp32
        if (TYPE == MOE_F32) return m;
        const uint32_t h = max(m >> 16, m & 0xffffu);
        return TYPE == MOE_BF16 ? h << 16 : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
    }
};

// Packed fp32 pairs.
__device__ __forceinline__ unsigned long long pk2(float x, float y) {
    return (static_cast<unsigned long long>(__float_as_uint(y)) << 32) | __float_as_uint(x);
}
__device__ __forceinline__ float2 up2(unsigned long long v) {
    return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t lo2(unsigned long long v) { return static_cast<uint32_t>(v); }
__device__ __forceinline__ uint32_t hi2(unsigned long long v) { return static_cast<uint32_t>(v >> 32); }

// the low bytes of four words
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return prmt(prmt(a, b, 0x0040u), prmt(c, d, 0x0040u), 0x5410u);
}

// Device copy of moe_kv8_cache.
struct KvCache {
    uint8_t* pool;
    const int32_t* table;
    int64_t table_stride;
    int64_t n_pages;
    int n_kv, D, page_blocks, max_pages, n_seqs, rec;
};

// The record of (sequence b, block j, head h), or nullptr (*err gets MOE_ERR_PAGE).
__device__ __forceinline__ uint8_t* kv8_record(const KvCache& c, int b, int j, int h, int32_t* err) {
    const int pi = j / c.page_blocks, pb = j - pi * c.page_blocks;
    if (pi < c.max_pages) {
        const int32_t pg = gload(c.table + b * c.table_stride + pi);
        if (pg >= 0 && pg < c.n_pages)
            return c.pool + ((static_cast<int64_t>(pg) * c.n_kv + h) * c.page_blocks + pb) * c.rec;
    }
    set_err(err, MOE_ERR_PAGE);
    return nullptr;
}

// The blocks that ragged rows touch, as a flat list with gaps: sequence b's first block has index
// floor(cu[b] / 32) + 2 b. A sequence of n tokens touches at most floor((n + 30) / 32) + 1 blocks,
// which is no more than the distance to the next sequence's index, and all indices lie below
// floor(n_tokens / 32) + 2 n_seqs.
__host__ __device__ inline int64_t kv8_slots(int64_t n_tokens, int n_seqs) { return n_tokens / 32 + 2LL * n_seqs; }

struct KvSlot {
    int b;             // sequence, -1: none
    int blk;           // block of the sequence
    int t0, t1;        // the block's tokens in the range: t0 <= t < t1
    int64_t row;       // dense row of token t: row + t
};

// Find slot `s`. All threads of a warp call it with the same s; the sequence is found by a 32-way
// search over its lanes (one round of loads per factor of 32 in n_seqs).
__device__ __forceinline__ KvSlot kv8_slot(int64_t s, const int32_t* cu, const int32_t* start,
                                           int n_seqs, int64_t n_tokens, int32_t* err) {
    KvSlot r;
    r.b = -1;
    r.blk = r.t0 = r.t1 = 0;
    r.row = 0;
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seqs;  // the last b in [lo, lo + n) whose first index is <= s
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool ok = lane * step < n && (static_cast<int64_t>(gload(cu + i)) >> 5) + 2LL * i <= s;
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        const int k = m ? 31 - __clz(m) : 0;
        n = min(step, n - k * step);
        lo += k * step;
    }
    const int64_t c0 = gload(cu + lo), c1 = gload(cu + lo + 1), p0 = gload(start + lo);
    if (c0 < 0 || c1 < c0 || c1 > n_tokens || p0 < 0 || p0 + (c1 - c0) > 0x7fffffff) {
        set_err(err, MOE_ERR_LEN);
        return r;
    }
    const int64_t k = s - ((c0 >> 5) + 2LL * lo);
    const int64_t blk = (p0 >> 5) + k, p1 = p0 + (c1 - c0);
    if (k < 0 || c1 == c0 || blk * 32 >= p1) return r;
    r.b = lo;
    r.blk = static_cast<int>(blk);
    r.t0 = static_cast<int>(p0 > blk * 32 ? p0 - blk * 32 : 0);
    r.t1 = static_cast<int>(p1 < blk * 32 + 32 ? p1 - blk * 32 : 32);
    r.row = c0 + blk * 32 - p0;
    return r;
}

// Dense rows of one of keys or values.
template <typename T>
struct KvRows {
    T* p;
    int64_t ts, hs;
    bool vec;  // 16-byte vectors
};

}  // namespace moe
