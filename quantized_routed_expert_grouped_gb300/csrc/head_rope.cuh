// head_rope.cuh - norm and rotation of the heads of dense rows, a warp for heads of one token: what the kernels of
// head_rope.cu and kv8_append.cu share. Internal header (not part of the C ABI).
//
//   y = x / sqrt(mean x^2 + eps) * w;   (a, b) -> factor (a cos t - b sin t, a sin t + b cos t),  t = position * f
//
// A head is D / W vectors of 16 bytes (W = 8 elements of 16 bits, 4 of fp32). A lane holds two of them: s and
// s + rot / 2W of the rotated dims, so that in both layouts a lane has whole pairs and a warp's accesses fill whole
// sectors; the dims that stay follow, paired in the same way. L = a power of two >= D / 2W lanes hold a head, and the
// 32 / L groups of a warp take heads of one token in turn. The angles of a CTA's tokens and the weights lie in shared memory, in
// the order in which lanes read them (chunks of 16 bytes, one after another over the lanes of a head): held in registers they
// left a third of the warps.
//
// Angles. turns = f / 2 pi in units of 2^-64; position * turns, in 64 bits, drops whole turns by itself, so the angle of a
// far position is as exact as that of a near one. The nearest quarter of a turn is taken off in whole numbers too; the rest, up
// to pi / 4, goes to fp32 and into the Taylor polynomials of sine and cosine to the 9th and 10th power (what they leave out is below
// 2^-29). No table of positions is read, and none limits them.
#pragma once

#include "internal.h"
#include "kv8.cuh"
#include "moe_decode.h"

namespace moe {

// The rotation as the kernels take it (rot = 0: none).
struct RopeArgs {
    const uint64_t* turns;
    int rot, start, inter;
    float factor;
};

// One set of heads (queries or keys).
struct HeadSet {
    const void* x;
    void* out;
    const void* weight;
    int64_t xt, xh, ot, oh;  // strides in elements: token, head
    int n;
    bool xvec, ovec;  // 16-byte vectors
};

#ifdef __CUDACC__

// 16 bytes as they lie in memory; VEC: they are aligned.
template <int TYPE, bool VEC>
struct RawVec {
    using T = typename Elem<TYPE>::T;
    static constexpr int W = 16 / static_cast<int>(sizeof(T));
    uint32_t w[4];
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC) {
            const uint4 v = gload(reinterpret_cast<const uint4*>(p));
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else if constexpr (TYPE == MOE_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = gload(reinterpret_cast<const uint32_t*>(p) + i);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = gload(reinterpret_cast<const uint16_t*>(p) + 2 * i) |
                       static_cast<uint32_t>(gload(reinterpret_cast<const uint16_t*>(p) + 2 * i + 1)) << 16;
        }
    }
    __device__ __forceinline__ float get(int e) const {
        if (TYPE == MOE_F32) return __uint_as_float(w[e & 3]);
        const uint32_t x = w[(e >> 1) & 3];
        if (TYPE == MOE_BF16) return __uint_as_float(e & 1 ? x & 0xffff0000u : x << 16);
        return __half2float(__ushort_as_half(static_cast<unsigned short>(e & 1 ? x >> 16 : x & 0xffffu)));
    }
    // of packed pairs of fp32
    __device__ __forceinline__ void put(const unsigned long long (&v)[W / 2]) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const float2 f = up2(v[i]);
            if constexpr (TYPE == MOE_F32) {
                w[2 * i] = __float_as_uint(f.x);
                w[2 * i + 1] = __float_as_uint(f.y);
            } else if constexpr (TYPE == MOE_F16) {
                const __half2 h = __floats2half2_rn(f.x, f.y);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (VEC) {
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (TYPE == MOE_F32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                reinterpret_cast<uint16_t*>(p)[2 * i] = static_cast<uint16_t>(w[i]);
                reinterpret_cast<uint16_t*>(p)[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
            }
        }
    }
};

// The two vectors of lane s of a head (W elements each), by their first dims, and the pairs that they hold.
struct RopeUnit {
    int e0, e1;
    bool in, turn;  // the head has them; they are rotated
    __device__ __forceinline__ RopeUnit(const RopeArgs& r, int D, int W, int s) {
        const int pairs = r.rot / (2 * W), rest = (D - r.rot) / (2 * W);
        in = s < pairs + rest;
        turn = s < pairs;
        if (turn) {
            e0 = r.start + s * W;
            e1 = e0 + r.rot / 2;
        } else {  // the dims that stay, counted without the rotated ones
            e0 = (s - pairs) * W;
            e1 = e0 + rest * W;
            if (e0 >= r.start) e0 += r.rot;
            if (e1 >= r.start) e1 += r.rot;
        }
    }
};
// The pair that slot j (of W) of rotated lane s is: of the halves layout elements j of both vectors, of the interleaved
// one elements 2j, 2j + 1 of the first vector, then of the second.
__device__ __forceinline__ int rope_pair(const RopeArgs& r, int W, int s, int j) {
    if (!r.inter) return s * W + j;
    return j < W / 2 ? s * (W / 2) + j : r.rot / 4 + s * (W / 2) + j - W / 2;
}

// factor * (cos, sin) of position * turns.
__device__ __forceinline__ float2 rope_angle(uint64_t turns, int position, float factor) {
    const uint64_t at = turns * static_cast<uint64_t>(static_cast<int64_t>(position));
    const uint32_t quarter = static_cast<uint32_t>((at + (1ull << 61)) >> 62);
    const float t = static_cast<float>(static_cast<int64_t>(at - (static_cast<uint64_t>(quarter) << 62))) * 3.4061215800086834e-19f;  // 2 pi / 2^64
    const float z = t * t;
    const float s = t * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), 1.0f) * factor;
    const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f) * factor;
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;  // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
    return make_float2((quarter + 1) & 2 ? -x : x, quarter & 2 ? -y : y);
}

// The rotation of a lane's two vectors, in place, as packed pairs of fp32; at: its angles' chunks, `lanes` apart.
template <int W>
__device__ __forceinline__ void rope_turn(unsigned long long (&a)[W / 2], unsigned long long (&b)[W / 2], const float4* at, int lanes, int inter) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        const float4 f = at[i * lanes];
        if (!inter) {
            const unsigned long long c = pk2(f.x, f.y), s = pk2(f.z, f.w), neg = mul2(b[i], pk2(-1.0f, -1.0f));
            const unsigned long long x = fma2(neg, s, mul2(a[i], c));
            b[i] = fma2(a[i], s, mul2(b[i], c));
            a[i] = x;
        } else {  // two pairs of the first vector, or of the second
            auto one = [](unsigned long long& v, float c, float s) {
                const float2 x = up2(v);
                v = pk2(fmaf(-x.y, s, x.x * c), fmaf(x.x, s, x.y * c));
            };
            one(i < W / 4 ? a[2 * i] : b[2 * i - W / 2], f.x, f.z);
            one(i < W / 4 ? a[2 * i + 1] : b[2 * i + 1 - W / 2], f.y, f.w);
        }
    }
}

// The shared memory of a CTA: angles of up to T tokens, then the weights of queries and of keys.
__host__ __device__ inline int rope_smem(int rot, int D, int T) { return (T * rot + 2 * D) * 4; }

// The angles of n tokens, by the CTA. A token's are rot / 4 chunks of two pairs (both cosines, both sines, as packed arithmetic takes
// them), chunk j / 2 of lane s at (j / 2) * lanes + s; tokens lie `row` floats apart. A thread has one pair of every
// so many tokens. place(t): the token's position.
template <int W, typename F>
__device__ __forceinline__ void put_angles(float* to, const RopeArgs& r, int n, int row, F place) {
    const int half = r.rot / 2, lanes = r.rot / (2 * W), each = max(1, static_cast<int>(blockDim.x) / half);
    const int first = threadIdx.x / half;  // (half <= blockDim.x)
    if (first >= each) return;
    const int i = threadIdx.x - first * half, s = i / W, j = i - s * W;
    const uint64_t turns = gload(r.turns + rope_pair(r, W, s, j));
    to += ((j >> 1) * lanes + s) * 4 + (j & 1) + first * row;
    for (int t = first; t < n; t += each, to += each * row) {
        const float2 f = rope_angle(turns, place(t), r.factor);
        to[0] = f.x;
        to[2] = f.y;
    }
}
// A set's weights as fp32: chunk c (of four) of lane s at c * lanes + s; the second vector's after all of the first's.
template <int W>
__device__ __forceinline__ void put_weights(float* to, const RopeArgs& r, int D, const void* weight, int w_type) {
    const int lanes = D / (2 * W);
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
        const int s = i / (2 * W), e = i - s * 2 * W, v = e / W, j = e - v * W;
        const RopeUnit u(r, D, W, s);
        const int at = (v ? u.e1 : u.e0) + j;
        const float w = w_type == MOE_F32 ? gload(static_cast<const float*>(weight) + at) : w_type == MOE_F16 ? __half2float(gload(static_cast<const __half*>(weight) + at))
                                                                                                              : __bfloat162float(gload(static_cast<const __nv_bfloat16*>(weight) + at));
        to[((v * (W / 4) + (j >> 2)) * lanes + s) * 4 + (j & 3)] = w;
    }
}

// Heads h0 .. h1 of a row by the whole warp: start() sends for the first ones, run() does them. L lanes a head; angles: the
// token's; weights: the set's.
template <int TYPE, int L, bool VEC>
struct RopeWarp {
    using Raw = RawVec<TYPE, VEC>;
    using T = typename Elem<TYPE>::T;
    static constexpr int W = Raw::W, G = 32 / L;  // elements of a vector, heads of a round
    const RopeUnit u;
    const int s, g;
    Raw ra, rb;

    __device__ __forceinline__ RopeWarp(const RopeArgs& r, int D) : u(r, D, W, threadIdx.x & (L - 1)), s(threadIdx.x & (L - 1)), g((threadIdx.x & 31) / L) {
        ra.clear();  // (a lane without dims adds zeros to its head's sum)
        rb.clear();
    }
    __device__ __forceinline__ void start(const HeadSet& set, int64_t row, int h0, int h1) {
        if (!u.in || h0 + g >= h1) return;
        const T* x = static_cast<const T*>(set.x) + row * set.xt + (h0 + g) * set.xh + u.e0;
        ra.load(x);
        rb.load(x + u.e1 - u.e0);
    }
    __device__ __forceinline__ void run(const HeadSet& set, const RopeArgs& r, int D, float eps, const float* angles, const float* weights, int64_t row, int h0, int h1) {
        const T* x = static_cast<const T*>(set.x) + row * set.xt + (h0 + g) * set.xh + u.e0;
        T* out = static_cast<T*>(set.out) + row * set.ot + (h0 + g) * set.oh + u.e0;
        const int64_t xs = G * set.xh, os = G * set.oh;
        const int second = u.e1 - u.e0, lanes = D / (2 * W), turning = r.rot / (2 * W);
        const float4* aw = reinterpret_cast<const float4*>(angles) + s;
        const float4* ww = reinterpret_cast<const float4*>(weights) + s;
        int left = u.in ? h1 - h0 - g : 0;  // heads from the lane's on
#pragma unroll 1
        for (int n = h1 - h0; n > 0; n -= G, left -= G) {  // (a warp's lanes stay together)
            unsigned long long a[W / 2], b[W / 2];
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                a[e] = pk2(ra.get(2 * e), ra.get(2 * e + 1));
                b[e] = pk2(rb.get(2 * e), rb.get(2 * e + 1));
            }
            x += xs;
            if (left > G) {
                ra.load(x);
                rb.load(x + second);
            }
            if (set.weight) {
                unsigned long long s2 = mul2(a[0], a[0]);
#pragma unroll
                for (int e = 1; e < W / 2; ++e) s2 = fma2(a[e], a[e], s2);
#pragma unroll
                for (int e = 0; e < W / 2; ++e) s2 = fma2(b[e], b[e], s2);
                const float2 f = up2(s2);
                float ss = f.x + f.y;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(fmaf(ss, 1.0f / static_cast<float>(D), eps));
                const unsigned long long ii = pk2(inv, inv);
                if (u.in) {
#pragma unroll
                    for (int c = 0; c < W / 4; ++c) {
                        const float4 p = ww[c * lanes], q = ww[(W / 4 + c) * lanes];
                        a[2 * c] = mul2(mul2(a[2 * c], ii), pk2(p.x, p.y));
                        a[2 * c + 1] = mul2(mul2(a[2 * c + 1], ii), pk2(p.z, p.w));
                        b[2 * c] = mul2(mul2(b[2 * c], ii), pk2(q.x, q.y));
                        b[2 * c + 1] = mul2(mul2(b[2 * c + 1], ii), pk2(q.z, q.w));
                    }
                }
            }
            if (u.turn) rope_turn<W>(a, b, aw, turning, r.inter);
            if (left > 0) {
                Raw y;
                y.put(a);
                y.store(out);
                y.put(b);
                y.store(out + second);
            }
            out += os;
        }
    }
};

#endif

}  // namespace moe
