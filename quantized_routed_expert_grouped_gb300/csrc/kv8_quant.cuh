// kv8_quant.cuh - codes and scales of a block of 32 tokens of one key/value head, by a CTA of 128 threads: what the kernels
// that write the cache share (kv8_cache.cu says how, and what it costs). Internal header (not part of the C ABI).
#pragma once

#include <type_traits>

#include "kv8.cuh"

namespace moe {

constexpr int kKvThreads = 128;
constexpr int kKvTurn = 36;  // bytes of a dim's 32 tokens in shared memory, padded

// x * inv rounded to an integer (ties to even) in the low byte of the result, plus 128: |x * inv| <= 127
// up to two roundings, so adding 1.5 * 2^23 + 128 leaves the integer in the low bits.
__device__ __forceinline__ uint32_t code_word(float x, float inv) {
    return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f + 128.0f));
}
__device__ __forceinline__ unsigned long long code_words(float x, float y, float inv) {
    // (single products: the assembler joins a packed product and a packed addition into one rounding)
    return add2(pk2(__fmul_rn(x, inv), __fmul_rn(y, inv)), pk2(12582912.0f + 128.0f, 12582912.0f + 128.0f));
}
// byte i of w, a code, as code - 128
__device__ __forceinline__ float code_value(uint32_t w, int i) {
    return __fadd_rn(__uint_as_float(prmt(w, 0x4b000000u, 0x7440u + i)), -8388736.0f);  // 2^23 + 128
}

struct Scales {
    float scale, inv, ratio;
    bool grew;
};
__device__ __forceinline__ Scales block_scale(float amax, float old, bool kept) {
    Scales s;
    s.scale = max_nan(old, amax < kKvTiny ? 0.0f : __fdiv_rn(amax, 127.0f));
    if (!(s.scale <= 3.4028234e38f)) s.scale = __int_as_float(0x7fffffff);
    const bool some = s.scale > 0.0f;
    s.inv = some ? __fdiv_rn(1.0f, s.scale) : 0.0f;
    s.ratio = some && kept ? __fdiv_rn(old, s.scale) : 0.0f;
    s.grew = s.scale != old;
    return s;
}
// four codes under a larger scale (a block without one holds zeros)
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
    return pack4(code_word(code_value(w, 0), ratio), code_word(code_value(w, 1), ratio), code_word(code_value(w, 2), ratio),
                 code_word(code_value(w, 3), ratio));
}

// A thread's kept key codes under the larger scale (kr: its token and eight dims of each 32).
template <int NB>
__device__ __forceinline__ void rescale_keys(uint2* kr, const Scales& s) {
    const bool some = s.inv > 0.0f;
    uint2 q[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) q[n] = kr[n * 32];
#pragma unroll
    for (int n = 0; n < NB; ++n)
        kr[n * 32] = some ? make_uint2(rescale4(q[n].x, s.ratio), rescale4(q[n].y, s.ratio)) : make_uint2(0x80808080u, 0x80808080u);
}

// The CTA's kept value codes, tokens 0 .. t0, under the larger scale (vr: the record's values).
template <int NB>
__device__ __forceinline__ void rescale_values(uint8_t* vr, int t0, const Scales& s) {
    constexpr int D = NB * 32;
    const bool some = s.inv > 0.0f;
    const int words = (t0 + 3) / 4;  // of a dim's 32 bytes: D words / 128 <= 2 NB a thread
    uint32_t q[2 * NB];
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
        const int i = n * kKvThreads + threadIdx.x, d = i / words;
        if (d < D) q[n] = *(reinterpret_cast<const uint32_t*>(vr + d * 32) + i - d * words);
    }
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
        const int i = n * kKvThreads + threadIdx.x, d = i / words, x = i - d * words;
        if (d >= D) continue;
        uint32_t* at = reinterpret_cast<uint32_t*>(vr + d * 32) + x;
        const uint32_t w = some ? rescale4(q[n], s.ratio) : 0x80808080u;
        if (4 * x + 4 <= t0) {
            *at = w;
        } else {  // the word's last bytes belong to new tokens
            for (int e = 0; 4 * x + e < t0; ++e) reinterpret_cast<uint8_t*>(at)[e] = static_cast<uint8_t>(w >> (8 * e));
        }
    }
}

// The CTA's new values: a thread's are of token vt, eight dims of each 32. A whole block is turned in shared memory (turn: D *
// kKvTurn bytes) and leaves by vectors, part of one by single bytes. (All threads of the CTA; where `whole`, a barrier.)
template <int TYPE, int NB>
__device__ __forceinline__ void write_values(uint8_t* vr, uint8_t* turn, const Raw8<TYPE> (&v)[NB], int vt, bool vin, bool whole, const Scales& s) {
    constexpr int D = NB * 32;
    const bool some = s.inv > 0.0f;
    const int lane = threadIdx.x & 31;
    if (vin) {
        auto put = [&](uint8_t* at, auto step) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const unsigned long long x = some ? code_words(v[n].get(2 * e), v[n].get(2 * e + 1), s.inv) : (128ull << 32 | 128);
                    at[(n * 32 + 2 * e) * step.value] = static_cast<uint8_t>(lo2(x));
                    at[(n * 32 + 2 * e + 1) * step.value] = static_cast<uint8_t>(hi2(x));
                }
        };
        if (whole) put(turn + (lane & 3) * 8 * kKvTurn + vt, std::integral_constant<int, kKvTurn>{});
        else put(vr + (lane & 3) * 8 * 32 + vt, std::integral_constant<int, 32>{});  // part of a block: single bytes
    }
    if (!whole) return;
    __syncthreads();
    for (int i = threadIdx.x; i < D * 2; i += kKvThreads) {  // 16 tokens of a dim
        const uint32_t* at = reinterpret_cast<const uint32_t*>(turn + (i >> 1) * kKvTurn + (i & 1) * 16);
        reinterpret_cast<uint4*>(vr)[i] = make_uint4(at[0], at[1], at[2], at[3]);
    }
}

}  // namespace moe
