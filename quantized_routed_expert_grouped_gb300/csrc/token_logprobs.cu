// token_logprobs.cu - log probabilities of given tokens, the most likely tokens, entropy and log-sum-exp of rows of logits,
// in one pass over them.
//
//   t_j = scale (x_j - m),  s = sum e^t_j,  u = sum t_j e^t_j;   lse = scale m + log s,  log p_j = t_j - log s,
//   entropy = log s - u / s
//
// m is a thread's running maximum, moved once a tile (s and u are rescaled where it grows); threads, then the CTAs of a row,
// join theirs. Differences come before the product with the scale, so that x_j = m gives 0 exactly and masks of the type's
// lowest value overflow to -inf at most. In base 2: e^t = 2^((x - m) scale log2 e).
//
// The most likely tokens. A logit and its index are one 64-bit key, larger for a larger logit and among equal ones for
// the lower index, so that every order is strict and the result does not depend on timing. A CTA keeps its best `top` keys, the
// last of which is the bar that a later tile's logit must pass (strictly: its index is higher); a tile with few threads above
// the bar appends their keys and ranks the list anew. Where many are above it (a row's first tile), the bar first rises to the
// top-th best of the maxima of 128 pairs of threads: at least `top` keys pass, and no more than 2 `top` threads have any, whatever the
// logits are. Ranks are counts of larger keys.
//
// A row is read by a cluster of C CTAs (C a power of two up to 8, where rows are few), which join through distributed
// shared memory: one launch, no workspace. Rows need no alignment: the elements before a row's first 16-byte boundary and after
// its last one are taken singly, in its first and last tile.
#include <cooperative_groups.h>

#include "decode_api.h"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kUnroll = 4, kTile = kThreads * kUnroll;  // vectors of a tile
constexpr int kTop = 32, kMaxCluster = 8;
constexpr int kGroups = kThreads / 2;
constexpr int kHot = 64;  // threads whose keys a list takes at once
constexpr int kCap = kTop + kHot * (kUnroll * 8 + 1);
constexpr float kFar = -1000.0f;  // an exponent whose power of two is 0
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

// Sums of e^t and t e^t (in base 2) next to a maximum.
struct Stats {
    float m, s, u;
    __device__ __forceinline__ void move(float m1, float c) {  // m1 >= m
        const float d = fmaxf((m - (m1 == -INFINITY ? 0.0f : m1)) * c, kFar), f = ex2(d);
        u = fmaf(s, d, u) * f;
        s *= f;
        m = m1;
    }
    __device__ __forceinline__ void join(Stats o, float c) {
        const float m1 = fmaxf(m, o.m);
        move(m1, c);
        o.move(m1, c);
        s += o.s;
        u += o.u;
    }
};

template <int TYPE>
__device__ __forceinline__ float max_of(const RawVec<TYPE>& v, float mx) {  // (a NaN does not count)
    if constexpr (TYPE == MOE_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, v.get(e));
        return mx;
    } else {
        using H = typename std::conditional<TYPE == MOE_F16, __half2, __nv_bfloat162>::type;
        const H* h = reinterpret_cast<const H*>(v.w);
        const H a = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        const float2 f = TYPE == MOE_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&a)) : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&a));
        return fmaxf(mx, fmaxf(f.x, f.y));
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 4) token_logprobs_kernel(const LogprobArgs a) {
    using Raw = RawVec<TYPE>;
    using T = typename Elem<TYPE>::T;
    constexpr int W = Raw::W;
    constexpr uint32_t kNone = TYPE == MOE_F32 ? 0xff800000u : TYPE == MOE_F16 ? 0xfc00fc00u : 0xff80ff80u;  // -inf
    __shared__ unsigned long long list[kCap];                // the best keys in order, then new ones
    __shared__ __align__(16) unsigned long long work[kMaxCluster * kTop];
    __shared__ unsigned long long bar;                       // a raised bar
    __shared__ Stats stat[kThreads / 32 + 1];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31;
    const int C = a.cluster, rank = blockIdx.x % C, row = blockIdx.x / C;
    if (tid == 0) count = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const T* x = static_cast<const T*>(a.x) + row * a.stride;
    // a given token's logit, on its way meanwhile
    int id = -1;
    float given = 0.0f;
    if (rank == 0 && tid < a.n_ids) {
        id = gload(a.ids + static_cast<int64_t>(row) * a.n_ids + tid);
        if (id >= 0 && id < a.V) given = Elem<TYPE>::get(gload(x + id));
    }
    const int head = min(a.V, static_cast<int>((-reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T)));
    const int nv = (a.V - head) / W, tail = a.V - head - nv * W;
    const int v0 = static_cast<int>(static_cast<int64_t>(nv) * rank / C), v1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / C);
    const T* xv = x + head;
    Raw next[kUnroll];
    auto load = [&](int at) {
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int v = at + i * kThreads + tid;
            if (v < v1) {
                next[i].load(xv + static_cast<int64_t>(v) * W, true);
            } else {
                next[i].w[0] = next[i].w[1] = next[i].w[2] = next[i].w[3] = kNone;
            }
        }
    };
    load(v0);
    Stats st{-INFINITY, 0.0f, 0.0f};
    unsigned long long best = 0;  // the bar: the list's last key, 0 while it is not full
    int at = v0;
    do {
        Raw cur[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) cur[i] = next[i];
        // singles: of the row's start thread 0 .., of its end thread 32 ..
        int single = -1;
        if (rank == 0 && at == v0 && tid < head) single = tid;
        if (rank == C - 1 && at + kTile >= v1 && tid >= 32 && tid < 32 + tail) single = head + nv * W + tid - 32;
        const float alone = single >= 0 ? Elem<TYPE>::get(gload(x + single)) : -INFINITY;
        load(at + kTile);
        // ---- statistics
        float mx = alone == alone ? alone : -INFINITY;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) mx = max_of<TYPE>(cur[i], mx);
        if (mx > st.m) st.move(mx, a.c);
        const float mr = st.m == -INFINITY ? 0.0f : st.m;
        const unsigned long long mm = pk2(-mr, -mr), cc = pk2(a.c, a.c);
        unsigned long long s2 = 0, u2 = 0;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                const float2 t = up2(mul2(add2(pk2(cur[i].get(2 * e), cur[i].get(2 * e + 1)), mm), cc));
                const unsigned long long p = pk2(ex2(t.x), ex2(t.y));
                s2 = add2(s2, p);
                u2 = fma2(p, pk2(fmaxf(t.x, kFar), fmaxf(t.y, kFar)), u2);
            }
        const float2 sf = up2(s2), uf = up2(u2);
        st.s += sf.x + sf.y;
        st.u += uf.x + uf.y;
        if (single >= 0) {
            const float t = (alone - mr) * a.c, p = ex2(t);
            st.s += p;
            st.u = fmaf(p, fmaxf(t, kFar), st.u);
        }
        // ---- the best keys
        if (a.top) {
            const bool hot = order(mx) > static_cast<uint32_t>(best >> 32);
            const int n_hot = __syncthreads_count(hot);
            if (n_hot) {
                auto each = [&](auto f) {
                    if (!hot) return;
                    if (single >= 0) f(key_of(alone, static_cast<uint32_t>(single)));
#pragma unroll
                    for (int i = 0; i < kUnroll; ++i) {
                        const int v = at + i * kThreads + tid;
                        if (v >= v1) continue;
#pragma unroll
                        for (int e = 0; e < W; ++e) f(key_of(cur[i].get(e), static_cast<uint32_t>(head + v * W + e)));
                    }
                };
                unsigned long long least = best + 1;
                if (n_hot > kHot) {
                    unsigned long long k = 0;
                    each([&](unsigned long long y) { k = y > k ? y : k; });
                    const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, 1);
                    if (!(tid & 1)) work[tid >> 1] = k > o ? k : o;
                    if (tid == 0) bar = 0;
                    __syncthreads();
                    if (tid < kGroups) {
                        const unsigned long long mine = work[tid];
                        int above = 0;
#pragma unroll 16
                        for (int j = 0; j < kGroups; ++j) above += work[j] > mine;
                        if (above == a.top - 1 && mine) bar = mine;
                    }
                    __syncthreads();
                    least = bar > least ? bar : least;
                }
                each([&](unsigned long long y) {
                    if (y >= least) list[atomicAdd(&count, 1)] = y;
                });
                __syncthreads();
                const int n = count, keep = min(n, a.top);
                for (int i = tid; i < n; i += kThreads) {
                    const unsigned long long mine = list[i];
                    int above = 0;
#pragma unroll 4
                    for (int j = 0; j < n; ++j) above += list[j] > mine;
                    if (above < a.top) work[above] = mine;
                }
                __syncthreads();
                if (tid < keep) list[tid] = work[tid];
                if (tid == 0) count = keep;
                best = n >= a.top ? work[a.top - 1] : 0;
                __syncthreads();
            }
        }
        at += kTile;
    } while (at < v1);

    // ---- the CTA's, then the row's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stats y;
        y.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        y.s = __shfl_xor_sync(0xffffffffu, st.s, o);
        y.u = __shfl_xor_sync(0xffffffffu, st.u, o);
        // (the lower lane's first in both lanes, so that they agree)
        if (lane & o) {
            const Stats z = st;
            st = y;
            y = z;
        }
        st.join(y, a.c);
    }
    if (lane == 0) stat[tid >> 5] = st;
    __syncthreads();
    st = stat[0];
    for (int w = 1; w < kThreads / 32; ++w) st.join(stat[w], a.c);
    if (C > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        if (tid == 0) stat[kThreads / 32] = st;
        cluster.sync();
        if (rank == 0) {
            const int from = tid / kTop, i = tid % kTop;  // (kMaxCluster * kTop threads)
            unsigned long long mine = 0;
            if (a.top && from < C && i < *cluster.map_shared_rank(&count, from)) mine = cluster.map_shared_rank(list, from)[i];
            work[tid] = mine;
            for (int r = 1; r < C; ++r) st.join(*cluster.map_shared_rank(stat + kThreads / 32, r), a.c);
            __syncthreads();
            if (a.top) {
                int above = 0, some = __syncthreads_count(mine != 0);
#pragma unroll 16
                for (int j = 0; j < C * kTop; ++j) above += work[j] > mine;
                if (mine && above < a.top) list[above] = mine;
                if (tid == 0) count = min(some, a.top);
                __syncthreads();
            }
        }
        cluster.sync();
    }
    if (rank != 0) return;
    const bool none = st.s == 0.0f;
    const float ls = logf(st.s);
    auto logprob = [&](float v) { return none ? -INFINITY : (v - st.m) * a.scale - ls; };
    for (int i = tid; i < a.n_ids; i += kThreads) {
        const int64_t to = static_cast<int64_t>(row) * a.n_ids + i;
        if (i >= kThreads) {
            id = gload(a.ids + to);
            if (id >= 0 && id < a.V) given = Elem<TYPE>::get(gload(x + id));
        }
        a.logprobs[to] = id >= 0 && id < a.V ? logprob(given) : -INFINITY;
    }
    if (tid < a.top) {
        const int64_t to = static_cast<int64_t>(row) * a.top + tid;
        const bool has = tid < count;
        const unsigned long long k = has ? list[tid] : 0;
        a.top_ids[to] = has ? static_cast<int32_t>(~static_cast<uint32_t>(k)) : -1;
        a.top_logprobs[to] = has ? logprob(unorder(static_cast<uint32_t>(k >> 32))) : NAN;
    }
    if (tid == 0) {
        if (a.entropy) a.entropy[row] = none ? 0.0f : ls - st.u * kLn2 / st.s;
        if (a.lse) a.lse[row] = none ? -INFINITY : fmaf(st.m, a.scale, ls);
    }
}

template <int TYPE>
cudaError_t logprobs_t(LogprobArgs a, cudaStream_t st) {
    constexpr int W = RawVec<TYPE>::W;
    // CTAs of a row: until every SM has two, and while each still has a whole tile
    a.cluster = 1;
    while (a.cluster < kMaxCluster && static_cast<int64_t>(a.rows) * a.cluster < 304 && a.V / W / a.cluster > kTile) a.cluster *= 2;
    a.c = a.scale * kLog2e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<TYPE>, a);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, int type, cudaStream_t st) {
    if (type == MOE_F32) return logprobs_t<MOE_F32>(a, st);
    if (type == MOE_F16) return logprobs_t<MOE_F16>(a, st);
    return logprobs_t<MOE_BF16>(a, st);
}

}  // namespace moe
