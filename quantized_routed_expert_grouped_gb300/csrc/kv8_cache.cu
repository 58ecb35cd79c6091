// kv8_cache.cu - quantising keys and values into the paged 8-bit cache, and reading them back.
//
// Write: scale = max |x| / 127 over a block's tokens and dims, code = rint(x * (1 / scale)) + 128; where a
// block keeps earlier tokens, scale = max(old, new) and their codes become rint((c - 128) * (old / scale)) + 128.
// Read: (code - 128) * scale. Every step is one fp32 operation, so the results are the same bits for any
// layout of the work.
//
// Both are bound by memory; a value costs its own size and one byte, and a few operations (a product, an
// addition that rounds and moves the code into the low byte, a byte permute). Write: one CTA per
// (block, head) holds all of the block's new keys and values in registers between the maximum and the
// codes, so they are read once, with D / 16 vectors per thread in flight. Read: one warp per (block, head)
// and keys or values. A warp takes eight tokens by 32 dims, 64 or 128 bytes of each row: of the keys
// that is a tile of the record, 256 bytes; the values are stored by dim, so the write turns them in shared
// memory (rows of 36 bytes: no two lanes of a store share a bank), and the read turns blocks of eight
// dims and four tokens in registers.
// Measured (GB300, of 6787 GB/s that a copy reaches; bf16, 8 heads of 128): writing 26k tokens of seven
// prompts, 33 us for 105 MB of rows and 53 MB of records (4.8 TB/s; the instructions fill 67 % of the
// issue slots; from fp32 rows 43 us for 209 MB and 53 MB, 6.1 TB/s), reading them back 31 us (into fp32 48 us). Reading 87k tokens of five prefixes: 86 us for 179 MB and 355 MB
// (6.2 TB/s, memory); 100k tokens into fp32 162 us (6.3 TB/s; 201 with stores that fill half sectors). Small calls (64 windows of 4 tokens) take 6 us each, launch and latency.
#include <type_traits>

#include "internal.h"
#include "kv8.cuh"
#include "kv8_api.h"

namespace moe {

namespace {

constexpr int kThreads = 128;

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

// NB = D / 32.
// CTAs per SM: the more, the more rows in flight and the shorter the last wave (prompts of 25k tokens, 8 heads of
// 128: 34 us at eight, 37 at the six that the compiler's own choice of registers leaves).
constexpr int write_ctas(int type, int nb) { return type != MOE_F32 && nb <= 4 ? 8 : type != MOE_F32 || nb <= 4 ? 5 : 3; }

template <int TYPE, int NB>
__global__ void __launch_bounds__(kThreads, write_ctas(TYPE, NB)) kv8_write_kernel(KvCache c, KvRows<const typename Elem<TYPE>::T> K,
                                                             KvRows<const typename Elem<TYPE>::T> V,
                                                             int64_t n_tokens, const int32_t* cu, const int32_t* start,
                                                             int32_t* err) {
    constexpr int D = NB * 32, kTurn = 36;  // bytes of a dim's 32 tokens in shared memory, padded
    __shared__ uint32_t red[2][4];
    __shared__ __align__(16) uint8_t turn[D * kTurn];
    const int h = blockIdx.x % c.n_kv, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const KvSlot s = kv8_slot(blockIdx.x / c.n_kv, cu, start, c.n_seqs, n_tokens, err);
    if (s.b < 0) return;
    uint8_t* rec = kv8_record(c, s.b, s.blk, h, err);
    if (!rec) return;
    auto* kb = K.p + s.row * K.ts + h * K.hs + (lane & 3) * 8;
    auto* vb = V.p + s.row * V.ts + h * V.hs + (lane & 3) * 8;
    const float2 old2 = s.t0 > 0 ? *reinterpret_cast<const float2*>(rec) : make_float2(0.0f, 0.0f);

    // A lane's values are of one token: of the keys, the warp's group of the record; of the values, eight
    // tokens a warp. Dims 32 n + 8 (lane & 3) ..
    const int g = lane >> 2, kt = 8 * (g >> 1) + 2 * wid + (g & 1), vt = wid * 8 + g;
    const bool kin = kt >= s.t0 && kt < s.t1, vin = vt >= s.t0 && vt < s.t1;
    Raw8<TYPE> k[NB], v[NB];
    kb += kt * K.ts;
    vb += vt * V.ts;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        k[n].clear();
        v[n].clear();
        if (kin) k[n].load(kb + n * 32, K.vec);
        if (vin) v[n].load(vb + n * 32, V.vec);
    }
    uint32_t ak = 0, av = 0;  // magnitudes order as their bits do
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        ak = k[n].amax(ak);
        av = v[n].amax(av);
    }
    ak = __reduce_max_sync(0xffffffffu, Raw8<TYPE>::float_bits(ak));
    av = __reduce_max_sync(0xffffffffu, Raw8<TYPE>::float_bits(av));
    if (lane == 0) {
        red[0][wid] = ak;
        red[1][wid] = av;
    }
    __syncthreads();  // also: every thread has read the old scales
    ak = max(max(red[0][0], red[0][1]), max(red[0][2], red[0][3]));
    av = max(max(red[1][0], red[1][1]), max(red[1][2], red[1][3]));
    const Scales sk = block_scale(__uint_as_float(ak), old2.x, s.t0 > 0), sv = block_scale(__uint_as_float(av), old2.y, s.t0 > 0);
    if (threadIdx.x == 0) *reinterpret_cast<float2*>(rec) = make_float2(sk.scale, sv.scale);

    // a block without a scale (zeros, or not finite) holds codes 128
    const bool some_k = sk.inv > 0.0f, some_v = sv.inv > 0.0f;
    uint2* kr = reinterpret_cast<uint2*>(rec + kKvHead) + wid * NB * 32 + lane;
    uint8_t* vr = rec + kKvHead + kKvBlock * D;
    if (kt < s.t0 && sk.grew) {  // kept tokens under the larger scale
        uint2 q[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) q[n] = kr[n * 32];
#pragma unroll
        for (int n = 0; n < NB; ++n)
            kr[n * 32] = some_k ? make_uint2(rescale4(q[n].x, sk.ratio), rescale4(q[n].y, sk.ratio)) : make_uint2(0x80808080u, 0x80808080u);
    }
    if (s.t0 > 0 && sv.grew) {
        const int words = (s.t0 + 3) / 4;  // of a dim's 32 bytes: D words / 128 <= 2 NB a thread
        uint32_t q[2 * NB];
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n) {
            const int i = n * kThreads + threadIdx.x, d = i / words;
            if (d < D) q[n] = *(reinterpret_cast<const uint32_t*>(vr + d * 32) + i - d * words);
        }
#pragma unroll
        for (int n = 0; n < 2 * NB; ++n) {
            const int i = n * kThreads + threadIdx.x, d = i / words, x = i - d * words;
            if (d >= D) continue;
            uint32_t* at = reinterpret_cast<uint32_t*>(vr + d * 32) + x;
            const uint32_t w = some_v ? rescale4(q[n], sv.ratio) : 0x80808080u;
            if (4 * x + 4 <= s.t0) {
                *at = w;
            } else {  // the word's last bytes belong to new tokens
                for (int e = 0; 4 * x + e < s.t0; ++e) reinterpret_cast<uint8_t*>(at)[e] = static_cast<uint8_t>(w >> (8 * e));
            }
        }
    }
    if (kin) {
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            uint2 q = make_uint2(0x80808080u, 0x80808080u);
            if (some_k) {
                unsigned long long x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = code_words(k[n].get(2 * e), k[n].get(2 * e + 1), sk.inv);
                q.x = pack4(lo2(x[0]), hi2(x[0]), lo2(x[1]), hi2(x[1]));
                q.y = pack4(lo2(x[2]), hi2(x[2]), lo2(x[3]), hi2(x[3]));
            }
            kr[n * 32] = q;
        }
    }
    const bool whole = s.t0 == 0 && s.t1 == 32;
    if (vin) {
        auto put = [&](uint8_t* at, auto step) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const unsigned long long x = some_v ? code_words(v[n].get(2 * e), v[n].get(2 * e + 1), sv.inv) : (128ull << 32 | 128);
                    at[(n * 32 + 2 * e) * step.value] = static_cast<uint8_t>(lo2(x));
                    at[(n * 32 + 2 * e + 1) * step.value] = static_cast<uint8_t>(hi2(x));
                }
        };
        if (whole) put(turn + (lane & 3) * 8 * kTurn + vt, std::integral_constant<int, kTurn>{});
        else put(vr + (lane & 3) * 8 * 32 + vt, std::integral_constant<int, 32>{});  // part of a block: single bytes
    }
    if (!whole) return;
    __syncthreads();
    for (int i = threadIdx.x; i < D * 2; i += kThreads) {  // 16 tokens of a dim
        const uint32_t* at = reinterpret_cast<const uint32_t*>(turn + (i >> 1) * kTurn + (i & 1) * 16);
        reinterpret_cast<uint4*>(vr)[i] = make_uint4(at[0], at[1], at[2], at[3]);
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(KvCache c, KvRows<typename Elem<TYPE>::T> K,
                                                            KvRows<typename Elem<TYPE>::T> V, int64_t n_tokens, int64_t n_work,
                                                            const int32_t* cu, const int32_t* start, int32_t* err) {
    const int lane = threadIdx.x & 31;
    int64_t work = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (work >= n_work) return;
    pdl_wait();
    pdl_trigger();
    const bool values = work & 1;
    work >>= 1;
    const int h = static_cast<int>(work % c.n_kv);
    const KvSlot s = kv8_slot(work / c.n_kv, cu, start, c.n_seqs, n_tokens, err);
    if (s.b < 0) return;
    const uint8_t* rec = kv8_record(c, s.b, s.blk, h, err);
    if (!rec) return;
    auto* kb = K.p + s.row * K.ts + h * K.hs;
    auto* vb = V.p + s.row * V.ts + h * V.hs;
    const int NB = c.D / 32;
    const float2 sc = gload(reinterpret_cast<const float2*>(rec));
    const int g = lane >> 2;
    const uint2* kr = reinterpret_cast<const uint2*>(rec + kKvHead);
#pragma unroll 1
    for (int i = 0; i < NB && !values; ++i) {
        uint2 q[4];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) q[jj] = gload(kr + (jj * NB + i) * 32 + lane);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const int t = 8 * (g >> 1) + 2 * jj + (g & 1);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(code_value(e < 4 ? q[jj].x : q[jj].y, e & 3), sc.x);
            store8_pair<TYPE, 1>(kb + t * K.ts + i * 32 + (lane & 3) * 8, K.vec, x, t >= s.t0 && t < s.t1);
        }
    }
    // lane (dims 8 dg .., tokens 4 tq ..) of 32 dims
    const int tq = lane & 7, dg = lane >> 3;
    const uint32_t* vr = reinterpret_cast<const uint32_t*>(rec + kKvHead + kKvBlock * c.D);
#pragma unroll 1
    for (int i = 0; i < NB && values; ++i) {
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = gload(vr + (i * 32 + dg * 8 + e) * 8 + tq);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * tq + j;
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(code_value(q[e], j), sc.y);
            store8_pair<TYPE, 8>(vb + t * V.ts + i * 32 + dg * 8, V.vec, x, t >= s.t0 && t < s.t1);
        }
    }
}

template <int TYPE>
cudaError_t write_t(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start, int32_t* err,
                    bool kvec, bool vvec, unsigned grid, cudaStream_t st) {
    using T = typename Elem<TYPE>::T;
    const KvRows<const T> K{static_cast<const T*>(r.k), r.k_token_stride, r.k_head_stride, kvec};
    const KvRows<const T> V{static_cast<const T*>(r.v), r.v_token_stride, r.v_head_stride, vvec};
    switch (c.D / 32) {
#define MOE_KV8_CASE(NB) \
    case NB: return launch_kernel(kv8_write_kernel<TYPE, NB>, dim3(grid), dim3(kThreads), 0, st, true, c, K, V, r.n_tokens, cu, start, err);
        MOE_KV8_CASE(1)
        MOE_KV8_CASE(2)
        MOE_KV8_CASE(3)
        MOE_KV8_CASE(4)
        MOE_KV8_CASE(5)
        MOE_KV8_CASE(6)
        MOE_KV8_CASE(7)
        MOE_KV8_CASE(8)
#undef MOE_KV8_CASE
    }
    return cudaErrorInvalidValue;
}

template <int TYPE>
cudaError_t read_t(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start, int32_t* err,
                   bool kvec, bool vvec, int64_t work, cudaStream_t st) {
    using T = typename Elem<TYPE>::T;
    const KvRows<T> K{static_cast<T*>(r.k), r.k_token_stride, r.k_head_stride, kvec};
    const KvRows<T> V{static_cast<T*>(r.v), r.v_token_stride, r.v_head_stride, vvec};
    const unsigned grid = static_cast<unsigned>((work + kThreads / 32 - 1) / (kThreads / 32));
    return launch_kernel(kv8_read_kernel<TYPE>, dim3(grid), dim3(kThreads), 0, st, true, c, K, V, r.n_tokens, work, cu, start, err);
}

}  // namespace

cudaError_t launch_kv8_write(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start,
                             int32_t* err, bool kvec, bool vvec, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(kv8_slots(r.n_tokens, c.n_seqs) * c.n_kv);
    if (r.type == MOE_F32) return write_t<MOE_F32>(c, r, cu, start, err, kvec, vvec, grid, st);
    if (r.type == MOE_F16) return write_t<MOE_F16>(c, r, cu, start, err, kvec, vvec, grid, st);
    return write_t<MOE_BF16>(c, r, cu, start, err, kvec, vvec, grid, st);
}

cudaError_t launch_kv8_read(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start,
                            int32_t* err, bool kvec, bool vvec, cudaStream_t st) {
    const int64_t work = kv8_slots(r.n_tokens, c.n_seqs) * c.n_kv * 2;
    if (r.type == MOE_F32) return read_t<MOE_F32>(c, r, cu, start, err, kvec, vvec, work, st);
    if (r.type == MOE_F16) return read_t<MOE_F16>(c, r, cu, start, err, kvec, vvec, work, st);
    return read_t<MOE_BF16>(c, r, cu, start, err, kvec, vvec, work, st);
}

}  // namespace moe
