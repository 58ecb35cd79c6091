// kv8_append.cu - new keys, normed and rotated on the way, and values into the paged 8-bit cache, and the same tokens' queries
// normed and rotated beside them, in one launch. The codes and scales are those of kv8_cache.cu, of the fp32 keys that
// the norm and the rotation give (they are not rounded to the rows' type first: one rounding less).
//
// The list is kv8_slots' blocks of 32 positions; a CTA takes a block for the keys, or the values, of some key/value heads, or for some
// query heads, as head_rope.cu does. (Keys and values apart need fewer registers, and angles and weights are the keys' alone.) For keys a
// token is four lanes, which hold D / 16 pairs of vectors of eight dims between them (NU = D / 64 rounded up each, as
// RopeUnit pairs them), so that the norm is two shuffles and a pair is a lane's own. The block's angles are computed once a
// CTA into shared memory, a pair a thread, and serve its heads. A record's two scales are written by the two CTAs.
//
// Bound by memory and by its instructions together. Measured (GB300, bf16): 25.5k tokens of seven prompts, 8 heads of 128 and
// 32 query heads: 108 us for 575 MB (5.3 TB/s of the copy's 6.7; issue slots 58 %); keys and values alone 48 us, of which the rotation
// takes 7 and the norm 4 (moe_kv8_write 31: its keys stay packed). 64 windows of four: 8.4 us; one token: 3.5 us.
#include "decode_api.h"
#include "kv8_quant.cuh"

namespace moe {

namespace {

constexpr int kThreads = kKvThreads;

// The angles of a block: a token's row (put_angles) is an odd multiple of 64 bytes, so that the eight lanes of an access (two
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

// The block's largest magnitude, from the threads' (as bits: they order as magnitudes do, a NaN above all).
__device__ __forceinline__ float block_max(uint32_t (&red)[4], uint32_t m) {
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();  // also: every thread has read the old scale
    return __uint_as_float(max(max(red[0], red[1]), max(red[2], red[3])));
}

template <int TYPE, int NB>
__device__ __forceinline__ void append_keys(const AppendArgs& a, const KvSlot& s, int h0, int h1, uint8_t* rec, uint32_t (&red)[4], float* weights, float4* angles) {
    constexpr int D = NB * 32, NU = (NB + 1) / 2, kUnits = D / 16;
    using T = typename Elem<TYPE>::T;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, kt = 8 * (g >> 1) + 2 * wid + (g & 1);
    const bool kin = kt >= s.t0 && kt < s.t1;
    const int row4 = angle_row(a.r.rot), turning = a.r.rot / 16;
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
#pragma unroll 1
    for (int h = h0; h < h1; ++h, kb += a.kh, rec += static_cast<int64_t>(a.c.page_blocks) * a.c.rec) {
        const float old = s.t0 > 0 ? *reinterpret_cast<const float*>(rec) : 0.0f;
        Raw8<TYPE> k[NU][2];
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            k[n][0].clear();
            k[n][1].clear();
            if (kin && e0[n] >= 0) {
                k[n][0].load(kb + e0[n], a.kvec);
                k[n][1].load(kb + e1[n], a.kvec);
            }
        }
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
                if (e0[n] < 0 || !kin) continue;  // (no token there: zeros, which 1 / sqrt(0) would make NaN)
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
        const Scales sk = block_scale(block_max(red, __float_as_uint(mk)), old, s.t0 > 0);
        if (threadIdx.x == 0) *reinterpret_cast<float*>(rec) = sk.scale;
        if (kt < s.t0 && sk.grew) rescale_keys<NB>(reinterpret_cast<uint2*>(rec + kKvHead) + wid * NB * 32 + lane, sk);
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
        if (h + 1 < h1) __syncthreads();  // red is written again
    }
}

template <int TYPE, int NB>
__device__ __forceinline__ void append_values(const AppendArgs& a, const KvSlot& s, int h0, int h1, uint8_t* rec, uint32_t (&red)[4], uint8_t* turn) {
    constexpr int D = NB * 32;
    using T = typename Elem<TYPE>::T;
    const int lane = threadIdx.x & 31, vt = (threadIdx.x >> 5) * 8 + (lane >> 2);
    const bool vin = vt >= s.t0 && vt < s.t1;
    const T* vb = static_cast<const T*>(a.v) + (s.row + vt) * a.vt + h0 * a.vh + (lane & 3) * 8;
#pragma unroll 1
    for (int h = h0; h < h1; ++h, vb += a.vh, rec += static_cast<int64_t>(a.c.page_blocks) * a.c.rec) {
        const float old = s.t0 > 0 ? *reinterpret_cast<const float*>(rec + 4) : 0.0f;
        Raw8<TYPE> v[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            v[n].clear();
            if (vin) v[n].load(vb + n * 32, a.vvec);
        }
        uint32_t av = 0;
#pragma unroll
        for (int n = 0; n < NB; ++n) av = v[n].amax(av);
        const Scales sv = block_scale(block_max(red, Raw8<TYPE>::float_bits(av)), old, s.t0 > 0);
        if (threadIdx.x == 0) *reinterpret_cast<float*>(rec + 4) = sv.scale;
        uint8_t* vr = rec + kKvHead + kKvBlock * D;
        if (s.t0 > 0 && sv.grew) rescale_values<NB>(vr, s.t0, sv);
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

// CTAs an SM, by the registers that a thread's keys need (prompts of 25k tokens, 8 heads of 128, 32 query heads, bf16: eight 108 us,
// seven 112; 4 and 16 heads of 256: five 125, three 153, six, which spill, 125; 192, fp32: six 130, four 155; three tokens of 192: 4.5 and 4.3).
constexpr int append_ctas(int type, int nb) { return nb <= 4 ? type == MOE_F32 ? 5 : 8 : nb <= 6 ? 6 : 5; }

template <int TYPE, int NB>
__global__ void __launch_bounds__(kThreads, append_ctas(TYPE, NB)) kv8_append_kernel(const AppendArgs a) {
    extern __shared__ __align__(16) float4 angles[];
    constexpr int D = NB * 32;
    __shared__ uint32_t red[4];
    __shared__ __align__(16) uint8_t turn[D * kKvTurn];
    __shared__ __align__(16) float weights[D];
    const int parts = a.kparts + a.vparts + a.qparts;
    const int slot = blockIdx.x / parts, part = blockIdx.x - slot * parts;
    pdl_wait();
    pdl_trigger();
    KvSlot s = kv8_slot(slot, a.cu, a.start, a.c.n_seqs, a.n_tokens, a.err);
    if (s.b < 0) return;
    if (part < a.kparts + a.vparts) {
        const bool values = part >= a.kparts;
        const int each = values ? a.vheads : a.kheads, h0 = (values ? part - a.kparts : part) * each, h1 = min(a.c.n_kv, h0 + each);
        uint8_t* rec = kv8_record(a.c, s.b, s.blk, h0, a.err);
        if (!rec) return;  // (the heads share the page)
        if (values) append_values<TYPE, NB>(a, s, h0, h1, rec, red, turn);
        else append_keys<TYPE, NB>(a, s, h0, h1, rec, red, weights, angles);
        return;
    }
    const int qpart = part - a.kparts - a.vparts, h0 = (qpart >> a.qshift) * a.qheads, h1 = min(a.q.n, h0 + a.qheads);
    if (a.qshift) {  // these tokens of the block alone
        const int split = 1 << a.qshift, each = (s.t1 - s.t0 + split - 1) >> a.qshift;
        s.t0 += (qpart & (split - 1)) * each;
        s.t1 = min(s.t1, s.t0 + each);
        if (s.t0 >= s.t1) return;
    }
    if (a.q.xvec && a.q.ovec) append_queries<TYPE, NB, true>(a, s, h0, h1, reinterpret_cast<float*>(angles));
    else append_queries<TYPE, NB, false>(a, s, h0, h1, reinterpret_cast<float*>(angles));
}

template <int TYPE>
cudaError_t append_t(AppendArgs& a, cudaStream_t st) {
    const int64_t slots = kv8_slots(a.n_tokens, a.c.n_seqs);
    // Heads of a CTA. Keys: one where there are few blocks, with many eight, which the block's angles serve (the same prompts:
    // eight 108 us, four 112; keys and values in one CTA, four heads each, 117). Values: two (64 windows of four: two 8.4 us, one 9.0, four 8.7).
    const bool many = slots * a.c.n_kv > 152 * 16;
    a.kheads = many ? 8 : 1;
    a.vheads = 2;
    // Queries: two rounds of a warp, eight heads at most; where that makes many CTAs four rounds, 32 heads (the prompts: half as many
    // 2 % longer, twice 6 %; 16 heads of 192, fp32: 4 155 us, 16 180; 26 prompts of 495 to 657, 32 heads of 160 and 4 key heads: 4 102, 2 120).
    // Else a block of several tokens over two or four CTAs (12 prompts of 286 to 621, 16 query heads of 128, fp16: 13.9 us, undivided 19.9; four of 1200,
    // 32 heads: 27.5 and 39; 51 windows of 1 to 22, 20 of 256: two 12.7, four 15.1, undivided 14.1).
    const int round = 32 / lanes_of(TYPE, a.c.D / 32);
    a.qheads = round > 4 ? 8 : 2 * round;
    const bool many_q = many || slots * ((a.q.n + a.qheads - 1) / a.qheads) > 152 * 16;
    if (many_q) a.qheads = round > 8 ? 32 : 4 * round;
    a.qshift = many_q || a.n_tokens <= 4 * a.c.n_seqs ? 0 : a.n_tokens <= 16 * a.c.n_seqs ? 1 : 2;
    a.kparts = (a.c.n_kv + a.kheads - 1) / a.kheads;
    a.vparts = (a.c.n_kv + a.vheads - 1) / a.vheads;
    a.qparts = (a.q.n + a.qheads - 1) / a.qheads << a.qshift;
    const unsigned grid = static_cast<unsigned>(slots * (a.kparts + a.vparts + a.qparts));
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
