// head_rope.cuh - norm and rotation of the heads of dense rows, a warp for heads of one token: what the kernels of
// head_rope.cu and kv8_append.cu share. Internal header (not part of the C ABI).
//
//   y = x / sqrt(mean x^2 + eps) * w;   (a, b) -> factor (a cos t - b sin t, a sin t + b cos t),  t = position * f
//
// A head is D / W vectors of 16 bytes (W = 8 elements of 16 bits, 4 of fp32). A lane holds two of them: s and
// s + rot / 2W of the rotated dims, so that in both layouts a lane has whole pairs and a warp's accesses fill whole
// sectors; the dims that stay follow, paired in the same way. L = a power of two >= D / 2W lanes hold a head, and the
// 32 / L groups of a warp take heads of one token in turn: the W angles of a lane are the same for all of them, each group
// computes its share, and they are exchanged by shuffles.
//
// Angles. turns = f / 2 pi in units of 2^-64; position * turns, in 64 bits, drops whole turns by itself, so the angle of a
// far position is as exact as that of a near one (what is left is the rounding to fp32: 9e-8 at half a turn). No table of
// positions is read, and none limits them.
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

// A vector of 16 bytes as it lies in memory.
template <int TYPE>
struct RawVec {
    using T = typename Elem<TYPE>::T;
    static constexpr int W = 16 / static_cast<int>(sizeof(T));
    uint32_t w[4];
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
    __device__ __forceinline__ void load(const T* p, bool vec) {
        if (vec) {
            const uint4 v = gload(reinterpret_cast<const uint4*>(p));
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else if (TYPE == MOE_F32) {
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
};

template <int TYPE>
__device__ __forceinline__ void store_vec(typename Elem<TYPE>::T* p, bool vec, const unsigned long long (&v)[RawVec<TYPE>::W / 2]) {
    using E = Elem<TYPE>;
    constexpr int W = RawVec<TYPE>::W;
    uint32_t w[4];
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
    if (vec) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (TYPE == MOE_F32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            reinterpret_cast<uint16_t*>(p)[2 * i] = static_cast<uint16_t>(w[i]);
            reinterpret_cast<uint16_t*>(p)[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
        }
    }
}

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

// factor * (cos, sin) of the pair's angle at a position.
__device__ __forceinline__ float2 rope_angle(const RopeArgs& r, int position, int pair) {
    const uint64_t at = gload(r.turns + pair) * static_cast<uint64_t>(static_cast<int64_t>(position));
    float s, c;
    sincospif(static_cast<float>(static_cast<int64_t>(at)) * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns, in [-1, 1]
    return make_float2(c * r.factor, s * r.factor);
}

// The rotation of a lane's two vectors, in place, as packed pairs of fp32.
template <int W>
__device__ __forceinline__ void rope_turn(unsigned long long (&a)[W / 2], unsigned long long (&b)[W / 2], const float (&c)[W], const float (&s)[W], int inter) {
    if (!inter) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const unsigned long long cc = pk2(c[2 * i], c[2 * i + 1]), ss = pk2(s[2 * i], s[2 * i + 1]), neg = pk2(-s[2 * i], -s[2 * i + 1]);
            const unsigned long long x = fma2(b[i], neg, mul2(a[i], cc));
            b[i] = fma2(a[i], ss, mul2(b[i], cc));
            a[i] = x;
        }
    } else {
        auto one = [](unsigned long long& v, float c, float s) {
            const float2 f = up2(v);
            v = pk2(fmaf(-f.y, s, f.x * c), fmaf(f.x, s, f.y * c));
        };
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            one(a[i], c[i], s[i]);
            one(b[i], c[W / 2 + i], s[W / 2 + i]);
        }
    }
}

template <int W>
__device__ __forceinline__ void weight_vec(const void* w, int w_type, int at, unsigned long long (&v)[W / 2]) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        float x, y;
        if (w_type == MOE_F32) {
            const float2 f = gload(reinterpret_cast<const float2*>(static_cast<const float*>(w) + at) + i);
            x = f.x;
            y = f.y;
        } else {
            const uint32_t u = gload(reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(w) + at) + i);
            if (w_type == MOE_BF16) {
                x = __uint_as_float(u << 16);
                y = __uint_as_float(u & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
                x = f.x;
                y = f.y;
            }
        }
        v[i] = pk2(x, y);
    }
}

// Heads h0 .. h1 of one row by the whole warp. L lanes a head, two rounds of 32 / L heads with their loads in flight.
template <int TYPE, int L>
__device__ __forceinline__ void rope_heads(const HeadSet& set, const RopeArgs& r, int D, int w_type, float eps, int64_t row, const int32_t* position, int at,
                                           int h0, int h1) {
    using Raw = RawVec<TYPE>;
    using T = typename Elem<TYPE>::T;
    constexpr int W = Raw::W, G = 32 / L, kAhead = 2;
    const int lane = threadIdx.x & 31, s = lane & (L - 1), g = lane / L;
    const RopeUnit u(r, D, W, s);
    const T* x = static_cast<const T*>(set.x) + row * set.xt;
    T* out = static_cast<T*>(set.out) + row * set.ot;
    Raw raw[kAhead][2];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            raw[i][0].clear();
            raw[i][1].clear();
            if (u.in && h + i * G < h1) {
                const T* p = x + (h + i * G) * set.xh;
                raw[i][0].load(p + u.e0, set.xvec);
                raw[i][1].load(p + u.e1, set.xvec);
            }
        }
    };
    load(h0 + g);
    float c[W], sn[W];
    if (r.rot) {  // each group computes P of the lane's W angles
        constexpr int P = G < W ? W / G : 1;
        const int pos = position ? gload(position) : at;
        float2 mine[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            mine[i] = make_float2(1.0f, 0.0f);
            if (u.turn && g * P + i < W) mine[i] = rope_angle(r, pos, rope_pair(r, W, s, g * P + i));
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
            c[j] = __shfl_sync(0xffffffffu, mine[j % P].x, j / P * L + s);
            sn[j] = __shfl_sync(0xffffffffu, mine[j % P].y, j / P * L + s);
        }
    }
    unsigned long long w0[W / 2], w1[W / 2];
    if (set.weight && u.in) {
        weight_vec<W>(set.weight, w_type, u.e0, w0);
        weight_vec<W>(set.weight, w_type, u.e1, w1);
    }
    const float mean = 1.0f / static_cast<float>(D);
    for (int h = h0 + g; h - g < h1; h += kAhead * G) {  // (a warp's lanes stay together)
        unsigned long long a[kAhead][W / 2], b[kAhead][W / 2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                a[i][e] = pk2(raw[i][0].get(2 * e), raw[i][0].get(2 * e + 1));
                b[i][e] = pk2(raw[i][1].get(2 * e), raw[i][1].get(2 * e + 1));
            }
        load(h + kAhead * G);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (set.weight) {
                unsigned long long s2 = 0;
#pragma unroll
                for (int e = 0; e < W / 2; ++e) s2 = fma2(b[i][e], b[i][e], fma2(a[i][e], a[i][e], s2));
                const float2 f = up2(s2);
                float ss = f.x + f.y;
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(fmaf(ss, mean, eps));
                const unsigned long long ii = pk2(inv, inv);
#pragma unroll
                for (int e = 0; e < W / 2; ++e) {
                    a[i][e] = mul2(mul2(a[i][e], ii), w0[e]);
                    b[i][e] = mul2(mul2(b[i][e], ii), w1[e]);
                }
            }
            if (u.turn) rope_turn<W>(a[i], b[i], c, sn, r.inter);
            if (u.in && h + i * G < h1) {
                T* p = out + (h + i * G) * set.oh;
                store_vec<TYPE>(p + u.e0, set.ovec, a[i]);
                store_vec<TYPE>(p + u.e1, set.ovec, b[i]);
            }
        }
    }
}

#endif

}  // namespace moe
