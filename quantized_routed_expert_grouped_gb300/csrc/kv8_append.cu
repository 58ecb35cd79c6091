// kv8_append.cu - new keys, normed and rotated on the way, and values into the paged 8-bit cache, and the same tokens' queries
// normed and rotated beside them, in one launch. The codes and scales are those of kv8_cache.cu, of the fp32 keys that
// the norm and the rotation give (they are not rounded to the rows' type first: one rounding less).
//
// The list is kv8_slots' blocks of 32 positions; a CTA takes one block for some key/value heads, or for some query heads, as
// head_rope.cu does. For keys a token is four lanes, which hold D / 16 pairs of vectors of eight dims between them (NU = D / 64
// rounded up each, as RopeUnit pairs them), so that the norm is two shuffles and a pair is a lane's own. The block's
// angles are computed once a CTA, a (token, pair) a thread, into shared memory, and serve its heads.
#include "decode_api.h"
#include "kv8_quant.cuh"

namespace moe {

namespace {

constexpr int kThreads = kKvThreads;

// The angles of a block: a token's row (put_angle) is an odd multiple of 64 bytes, so that the eight lanes of an access (two
// tokens) share no bank.
__host__ __device__ inline int angle_row(int rot) { return rot / 4 + (rot / 16 % 2 ? 0 : 4); }  // in float4

// What token t of the block turns by.
__device__ __forceinline__ int turn_at(const AppendArgs& a, const KvSlot& s, int t) {
    return a.positions ? gload(a.positions + s.row + t) : s.blk * kKvBlock + t;
}

// the largest magnitude (a NaN stays)
__device__ __forceinline__ float amax3(float m, float a, float b) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(a), "f"(b));
    return d;
}

template <int TYPE, int NB>
__device__ __forceinline__ void append_block(const AppendArgs& a, const KvSlot& s, int h0, int h1, float4* angles) {
    constexpr int D = NB * 32, NU = (NB + 1) / 2, kUnits = D / 16;
    using T = typename Elem<TYPE>::T;
    __shared__ uint32_t red[2][4];
    __shared__ __align__(16) uint8_t turn[D * kKvTurn];
    __shared__ __align__(16) float weights[D];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int g = lane >> 2, kt = 8 * (g >> 1) + 2 * wid + (g & 1), vt = wid * 8 + g;
    const bool kin = kt >= s.t0 && kt < s.t1, vin = vt >= s.t0 && vt < s.t1;
    const int row4 = angle_row(a.r.rot), turning = a.r.rot / 16;
    uint8_t* rec = kv8_record(a.c, s.b, s.blk, h0, a.err);
    if (!rec) return;  // (the CTA's heads share the page)
    if (a.r.rot) put_angles<8>(reinterpret_cast<float*>(angles + s.t0 * row4), a.r, s.t1 - s.t0, row4 * 4, [&](int t) { return turn_at(a, s, s.t0 + t); });
    if (a.k_weight) put_weights<8>(weights, a.r, D, a.k_weight, a.w_type);
    if (a.r.rot || a.k_weight) __syncthreads();
    int e0[NU], e1[NU];  // a lane's units of its token, -1: none
#pragma unroll
    for (int n = 0; n < NU; ++n) {
        const RopeUnit u(a.r, D, 8, 4 * n + (lane & 3));
        e0[n] = u.in ? u.e0 : -1;
        e1[n] = u.e1;
    }
    const T* kb = static_cast<const T*>(a.k) + (s.row + kt) * a.kt + h0 * a.kh;
    const T* vb = static_cast<const T*>(a.v) + (s.row + vt) * a.vt + h0 * a.vh + (lane & 3) * 8;
#pragma unroll 1
    for (int h = h0; h < h1; ++h, kb += a.kh, vb += a.vh, rec += static_cast<int64_t>(a.c.page_blocks) * a.c.rec) {
        const float2 old2 = s.t0 > 0 ? *reinterpret_cast<const float2*>(rec) : make_float2(0.0f, 0.0f);
        Raw8<TYPE> k[NU][2], v[NB];
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            k[n][0].clear();
            k[n][1].clear();
            if (kin && e0[n] >= 0) {
                k[n][0].load(kb + e0[n], a.kvec);
                k[n][1].load(kb + e1[n], a.kvec);
            }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            v[n].clear();
            if (vin) v[n].load(vb + n * 32, a.vvec);
        }
        // ---- keys: norm, rotation
        unsigned long long x[NU][2][4];
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][w][e] = pk2(k[n][w].get(2 * e), k[n][w].get(2 * e + 1));
        if (a.k_weight) {
            unsigned long long s2 = 0;
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s2 = fma2(x[n][w][e], x[n][w][e], s2);
            const float2 f = up2(s2);
            float ss = f.x + f.y;
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            const float inv = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
            const unsigned long long ii = pk2(inv, inv);
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                if (e0[n] < 0) continue;
                const float4* ww = reinterpret_cast<const float4*>(weights) + 4 * n + (lane & 3);
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 y = ww[(2 * w + e) * kUnits];
                        x[n][w][2 * e] = mul2(mul2(x[n][w][2 * e], ii), pk2(y.x, y.y));
                        x[n][w][2 * e + 1] = mul2(mul2(x[n][w][2 * e + 1], ii), pk2(y.z, y.w));
                    }
            }
        }
        float mk = 0.0f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int u = 4 * n + (lane & 3);
            if (kin && u < turning) rope_turn<8>(x[n][0], x[n][1], angles + kt * row4 + u, turning, a.r.inter);
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = up2(x[n][w][e]);
                    mk = amax3(mk, f.x, f.y);
                }
        }
        uint32_t ak = __float_as_uint(mk), av = 0;  // magnitudes order as their bits do (a NaN is above all)
#pragma unroll
        for (int n = 0; n < NB; ++n) av = v[n].amax(av);
        ak = __reduce_max_sync(0xffffffffu, ak);
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
        uint8_t* vr = rec + kKvHead + kKvBlock * D;
        if (kt < s.t0 && sk.grew) rescale_keys<NB>(reinterpret_cast<uint2*>(rec + kKvHead) + wid * NB * 32 + lane, sk);
        if (s.t0 > 0 && sv.grew) rescale_values<NB>(vr, s.t0, sv);
        if (kin) {
#pragma unroll
            for (int n = 0; n < NU; ++n) {
                if (e0[n] < 0) continue;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    uint2 q = make_uint2(0x80808080u, 0x80808080u);  // a block without a scale (zeros, or not finite)
                    if (sk.inv > 0.0f) {
                        unsigned long long y[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = up2(x[n][w][e]);
                            y[e] = code_words(f.x, f.y, sk.inv);
                        }
                        q.x = pack4(lo2(y[0]), hi2(y[0]), lo2(y[1]), hi2(y[1]));
                        q.y = pack4(lo2(y[2]), hi2(y[2]), lo2(y[3]), hi2(y[3]));
                    }
                    *reinterpret_cast<uint2*>(rec + kv8_k_at(D, kt, w ? e1[n] : e0[n])) = q;
                }
            }
        }
        write_values<TYPE, NB>(vr, turn, v, vt, vin, s.t0 == 0 && s.t1 == 32, sv);
        if (h + 1 < h1) __syncthreads();  // red and turn are written again
    }
}

constexpr int lanes_of(int type, int nb) {
    const int n = nb * 32 * (type == MOE_F32 ? 4 : 2) / 32;
    return n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : 32;
}

template <int TYPE, int NB, bool VEC>
__device__ __forceinline__ void append_queries(const AppendArgs& a, const KvSlot& s, int h0, int h1, float* sm) {
    using Warp = RopeWarp<TYPE, lanes_of(TYPE, NB), VEC>;
    const int n = s.t1 - s.t0, first = s.t0 + (threadIdx.x >> 5);
    float* qw = sm + n * a.r.rot;
    Warp w(a.r, NB * 32);
    if (first < s.t1) w.start(a.q, s.row + first, h0, h1);
    if (a.r.rot) put_angles<Warp::W>(sm, a.r, n, a.r.rot, [&](int t) { return turn_at(a, s, s.t0 + t); });
    if (a.q.weight) put_weights<Warp::W>(qw, a.r, NB * 32, a.q.weight, a.w_type);
    __syncthreads();
#pragma unroll 1
    for (int t = first; t < s.t1; t += kThreads / 32) {
        if (t != first) w.start(a.q, s.row + t, h0, h1);
        w.run(a.q, a.r, NB * 32, a.eps, sm + (t - s.t0) * a.r.rot, qw, s.row + t, h0, h1);
    }
}

// CTAs an SM, by the registers that a thread's keys and values need (prompts of 25k tokens, 8 heads of 128, 32 query heads, bf16: seven
// 117 us, six 122, without a limit 149).
constexpr int append_ctas(int type, int nb) { return nb <= 4 ? type == MOE_F32 ? 5 : 7 : nb <= 6 ? 4 : 3; }

template <int TYPE, int NB>
__global__ void __launch_bounds__(kThreads, append_ctas(TYPE, NB)) kv8_append_kernel(const AppendArgs a) {
    extern __shared__ __align__(16) float4 angles[];
    const int parts = a.kparts + a.qparts;
    const int slot = blockIdx.x / parts, part = blockIdx.x - slot * parts;
    pdl_wait();
    pdl_trigger();
    const KvSlot s = kv8_slot(slot, a.cu, a.start, a.c.n_seqs, a.n_tokens, a.err);
    if (s.b < 0) return;
    if (part < a.kparts) {
        append_block<TYPE, NB>(a, s, part * a.kheads, min(a.c.n_kv, (part + 1) * a.kheads), angles);
        return;
    }
    const int h0 = (part - a.kparts) * a.qheads, h1 = min(a.q.n, h0 + a.qheads);
    if (a.q.xvec && a.q.ovec) append_queries<TYPE, NB, true>(a, s, h0, h1, reinterpret_cast<float*>(angles));
    else append_queries<TYPE, NB, false>(a, s, h0, h1, reinterpret_cast<float*>(angles));
}

template <int TYPE>
cudaError_t append_t(AppendArgs& a, cudaStream_t st) {
    const int64_t slots = kv8_slots(a.n_tokens, a.c.n_seqs);
    // Heads of a CTA: one of the keys, a round or two of the queries, where there are few blocks; with many, four and 16, which
    // the block's angles serve (the same prompts: four 117 us, two 123, eight 125, one 160).
    const bool many = slots * a.c.n_kv > 152 * 16;
    a.kheads = many ? 4 : 1;
    a.qheads = many ? 16 : 8;
    a.kparts = (a.c.n_kv + a.kheads - 1) / a.kheads;
    a.qparts = (a.q.n + a.qheads - 1) / a.qheads;
    const unsigned grid = static_cast<unsigned>(slots * (a.kparts + a.qparts));
    const int keys = 32 * angle_row(a.r.rot) * static_cast<int>(sizeof(float4)), queries = rope_smem(a.r.rot, a.c.D, 32);
    const size_t smem = a.q.n && queries > keys ? queries : keys;
    switch (a.c.D / 32) {
#define MOE_KV8_CASE(NB) \
    case NB: return launch_kernel(kv8_append_kernel<TYPE, NB>, dim3(grid), dim3(kThreads), smem, st, true, a);
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

}  // namespace

cudaError_t launch_kv8_append(AppendArgs a, int type, cudaStream_t st) {
    if (type == MOE_F32) return append_t<MOE_F32>(a, st);
    if (type == MOE_F16) return append_t<MOE_F16>(a, st);
    return append_t<MOE_BF16>(a, st);
}

}  // namespace moe
