// token_logprobs.cu - log probabilities of given tokens, the most likely tokens, entropy and log-sum-exp of rows of logits,
// in one pass over them. (Short rows: token_logprobs_short.cu.)
//
//   t_j = c x_j - r,  s = sum 2^t_j,  u = sum t_j 2^t_j   (c = scale log2 e);
//   log p_j = scale (x_j - m) - l,  l = ln 2 (log2 s - (c m - r)),  lse = scale m + l,  entropy = ln 2 (log2 s - u / s)
//
// m is the row's largest logit. r is a whole number near c times the largest that a thread has seen (kSlack below it at most), so that a
// logit's exponent is one fused product, rounded once, and what r is does not matter to the result; s and u are rescaled where r
// moves, which few tiles need. (It is above -2^24: what lies below has a power of 0 there, and nothing but such logits is a row for the second pass.) Threads join theirs, then the CTAs of a row, always in the same order. t 2^t of a logit of -inf has to be 0: 16-bit logits
// are clamped in pairs before they are converted, fp32's t one by one. Where that or c m leaves the range (rows masked by their type's lowest value,
// scales near 0 or far above 1) the row's sums are taken a second time, differences first. Powers are the hardware's (2^-22 of
// themselves); sums are fp32: a thread's terms of a tile in two halves (of eight in fp32, of sixteen in 16 bits), which are then added to its two
// running ones; the second pass, which few rows need, adds them to those one by one. Joined sums are not next to the row's largest logit, so what
// cannot be below 0 is held there at the end.
//
// The most likely tokens. A logit and its index are one 64-bit key, larger for a larger logit and among equal ones for
// the lower index: every order is strict, and nothing depends on timing. A CTA keeps its best `top` keys in order; the
// last one's logit is the bar. Every span of two tiles the threads whose maximum is above it are noted (an equal logit comes later, and
// loses); kHot of them, or the row's end, are looked through at once: of many only those that reach the top-th best of
// their maxima and the list, a warp for a span, read again (from L2: kept in registers they cost a quarter of the warps).
// While the list is not full, or more threads than kHot are above it, a new bar comes first: the least of the warps' maxima of
// rank top / warps, which `top` threads reach; and where more than kHot reach that (ties: masked rows), the top-th best of
// the threads' best keys, by sorting networks over lanes and merging over warps, so that never more than kHot spans are looked through,
// whatever the logits are. Ranks are counts of larger keys.
//
// A row is read by a cluster of C CTAs (a power of two up to 8, where rows are few); each sends its sums to all, and its list to the first,
// through distributed shared memory, behind one barrier: one launch, no workspace. Rows need no alignment: what lies before a
// row's first 16-byte boundary and after its last one is taken singly, at the end.
//
// Bound by memory while it only sums (2047 rows of 131,075, bf16, 537 MB: 86 us, 6.2 TB/s of a copy's 6.7; fp32 1024 rows of
// 131,072: 78 us, 6.8 TB/s); picking the best keys costs a barrier a span and a chain of latencies a row: top 1 104 us, top 5
// 107, top 20 127 (issue slots 58 %). 192 rows of 65,537, fp32, top 20: 24 us; one row of 32,768: 7.3 us, of which 3 are picking
// and 2 joining the cluster.
#include <cooperative_groups.h>
#include <type_traits>

#include "token_logprobs.cuh"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kUnroll = 4;  // vectors of a thread's tile
constexpr int kSpan = 2;    // tiles between two looks for the best keys: one is added while the next is on its way
constexpr int NT = 256;     // threads of a CTA
constexpr int kTop = 32, kMaxCluster = 8;
constexpr float kSlack = 8.0f;    // powers of two above its reference that a thread's maximum may rise
constexpr float kReach = 16777216.0f;  // 2^24: c x and the whole number next to it differ by a half at most


// Sums of 2^t and t 2^t, t = c x - r, next to a whole number r (at most kSlack below
// the largest c x); and the largest x.
struct Stats {
    float r, s, u, m;
    __device__ __forceinline__ void move(float to) {  // to >= r, and above -inf
        const float d = fmaxf(r - to, kFar), f = ex2(d);
        u = fmaf(s, d, u) * f;
        s *= f;
        r = to;
    }
    // of N lanes, the sums in lane 0
    template <int N>
    __device__ __forceinline__ void join() {
        float to = r;
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1) {
            to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        if (to > -INFINITY) move(to);
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            u += __shfl_xor_sync(0xffffffffu, u, o);
        }
    }
};

// The largest of a thread's tile. (A NaN does not count.)
template <int TYPE>
__device__ __forceinline__ float max_of(const Vec16<TYPE> (&v)[kUnroll]) {
    if constexpr (TYPE == MOE_F32) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, v[i].get(e));
        return mx;
    } else {
        using H = typename std::conditional<TYPE == MOE_F16, __half2, __nv_bfloat162>::type;
        H a = *reinterpret_cast<const H*>(v[0].w);
#pragma unroll
        for (int i = 1; i < 4 * kUnroll; ++i) a = __hmax2(a, *reinterpret_cast<const H*>(&v[i >> 2].w[i & 3]));
        const float2 f = TYPE == MOE_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&a)) : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&a));
        return fmaxf(fmaxf(f.x, f.y), -INFINITY);
    }
}

// A value far below any logit next to which it matters, and logits below it moved there (a NaN stays).
template <int TYPE>
constexpr float kLow = TYPE == MOE_F16 ? -65504.0f : -1.329227995784916e36f;  // -2^120
template <int TYPE>
__device__ __forceinline__ void clamp_low(Vec16<TYPE>& v) {
    if constexpr (TYPE != MOE_F32) {
        using H = typename std::conditional<TYPE == MOE_F16, __half2, __nv_bfloat162>::type;
        const uint32_t low = TYPE == MOE_F16 ? 0xfbfffbffu : 0xfb80fb80u;
        H* h = reinterpret_cast<H*>(v.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __hmax2_nan(h[i], *reinterpret_cast<const H*>(&low));
    }
}

__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();  // (the aligned form takes a warp's lanes together)
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

template <int TYPE>
__global__ void __launch_bounds__(NT, 4) token_logprobs_kernel(const LogprobArgs a) {
    using Raw = Vec16<TYPE>;
    using T = typename Elem<TYPE>::T;
    constexpr int W = Raw::W, kTile = NT * kUnroll;  // vectors of a tile
    constexpr int kHot = 64, kCap = kTop + kHot * kSpan * kUnroll * W;  // threads' spans to be looked through at once, and their keys
    constexpr int kFew = 2 * (NT / 32);  // spans that are looked through sooner than sifted
    constexpr uint32_t kNone = TYPE == MOE_F32 ? 0xff800000u : TYPE == MOE_F16 ? 0xfc00fc00u : 0xff80ff80u;  // -inf
    __shared__ __align__(16) unsigned long long list[kCap];  // the best keys in order, then new ones
    __shared__ __align__(16) unsigned long long work[kMaxCluster * kTop];
    __shared__ unsigned long long bar;  // a raised bar: a key, order() of a value
    __shared__ uint32_t raised;
    __shared__ uint32_t hot_max[kHot];  // spans of threads with logits above the bar: their maxima and first vectors
    __shared__ int hot_at[kHot], hots, listed;  // (listed: keys in order)
    __shared__ Stats stat[NT / 32];                           // of the warps
    __shared__ Stats all[2][kMaxCluster];                     // of the row's CTAs; once more
    __shared__ unsigned long long best_of[kMaxCluster * kTop];  // their best keys
    __shared__ int ids[NT];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 31;
    const int C = a.cluster, rank = blockIdx.x % C, row = blockIdx.x / C;
    if (tid == 0) count = hots = listed = 0;
    __syncthreads();
    if (C > 1) cluster_arrive();
    pdl_wait();
    pdl_trigger();
    const T* x = static_cast<const T*>(a.x) + row * a.stride;
    const int head = min(a.V, static_cast<int>((-reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T)));
    const int nv = (a.V - head) / W, tail = a.V - head - nv * W;
    const int v0 = static_cast<int>(static_cast<int64_t>(nv) * rank / C), v1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / C);
    const T* xv = x + head;
    Stats st{-INFINITY, 0.0f, 0.0f, -INFINITY};
    uint32_t best = 0;  // the bar: order() of the list's last logit, 0 while the list is not full
    int pending = 0;    // hots at most, as all threads know it
    // Spans of threads (their first vectors; the second may be none, -1) by a warp, a word or two a lane of each: keys of values of at
    // least `least`, and of at least `low`.
    auto look = [&](int first, int second, float least, unsigned long long low) {
        constexpr int kWords = kSpan * kUnroll * 4, kEach = (kWords + 31) / 32;
        uint32_t w[2][kEach];
        auto fetch = [&](int v, uint32_t (&w)[kEach]) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (i * 32 + lane < kWords && v + i * 8 * NT < v1) w[i] = gload(reinterpret_cast<const uint32_t*>(xv + static_cast<int64_t>(v + i * 8 * NT) * W) + (lane & 3));
        };
        auto put = [&](float y, uint32_t index) {
            if (y >= least) {
                const unsigned long long k = key_of(y, index);
                if (k >= low) list[atomicAdd(&count, 1)] = k;
            }
        };
        auto sift = [&](int v, const uint32_t (&w)[kEach]) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (i * 32 + lane >= kWords || v + i * 8 * NT >= v1) continue;
                const uint32_t index = head + (v + i * 8 * NT) * W + (lane & 3) * (W / 4);
                if (TYPE == MOE_F32) {
                    put(__uint_as_float(w[i]), index);
                } else {
                    Raw r;
                    r.w[0] = w[i];
                    put(r.get(0), index);
                    put(r.get(1), index + 1);
                }
            }
        };
        const int mine = (lane >> 2) * NT;
        fetch(first + mine, w[0]);
        if (second >= 0) fetch(second + mine, w[1]);
        sift(first + mine, w[0]);
        if (second >= 0) sift(second + mine, w[1]);
    };
    // The spans that wait are looked through (of many, those that reach the top-th best of their maxima and the list); then the list is put in order.
    // (What was appended before is visible. Keys below `low`, and values
    // below `base`, an order(), do not count.)
    auto flush = [&](unsigned long long low, uint32_t base) {
        const int n = hots, keys = listed;
        if (n) {
            if (tid == 0) raised = base;
            if (n > kFew) {
                uint32_t* v = reinterpret_cast<uint32_t*>(work);
                for (int i = tid; i < (n + keys + 3) / 4 * 4; i += NT) v[i] = i < n ? hot_max[i] : i < n + keys ? static_cast<uint32_t>(list[i - n] >> 32) : 0;
                __syncthreads();
                for (int i = tid; i < n + keys; i += NT) {
                    const uint32_t mine = v[i];
                    int above = 0, same = 0;
#pragma unroll 4
                    for (int j = 0; j < (n + keys + 3) / 4; ++j) {
                        const uint4 y = reinterpret_cast<const uint4*>(v)[j];
                        above += (y.x > mine) + (y.y > mine) + (y.z > mine) + (y.w > mine);
                        same += (y.x == mine) + (y.y == mine) + (y.z == mine) + (y.w == mine);
                    }
                    if (above < a.top && above + same >= a.top && mine > base) raised = mine;
                }
            }
            __syncthreads();
            const uint32_t least = max(raised, best ? best + 1 : 0);  // (of a full list, what equals its last comes later)
            const int mine = (tid >> 5) + lane * (NT / 32);
            unsigned on = __ballot_sync(0xffffffffu, mine < n && hot_max[mine < n ? mine : 0] >= least);
            while (on) {
                const int first = __ffs(on) - 1;
                on &= on - 1;
                const int second = __ffs(on) - 1;
                on &= on - 1;
                look(hot_at[(tid >> 5) + first * (NT / 32)], second < 0 ? -1 : hot_at[(tid >> 5) + second * (NT / 32)], unorder(least), low);
            }
            __syncthreads();
        }
        const int m = count, keep = min(m, a.top);
        for (int i = tid; i < m; i += NT) {
            const unsigned long long mine = list[i];
            int above = 0;
#pragma unroll 4
            for (int j = 0; j < m / 2; ++j) {
                const ulonglong2 y = reinterpret_cast<const ulonglong2*>(list)[j];
                above += (y.x > mine) + (y.y > mine);
            }
            if (m & 1) above += list[m - 1] > mine;
            if (above < a.top) work[above] = mine;
        }
        __syncthreads();
        if (tid < keep) list[tid] = work[tid];
        if (tid == 0) {
            count = listed = keep;
            hots = 0;
        }
        best = m >= a.top ? static_cast<uint32_t>(work[a.top - 1] >> 32) : 0;
        pending = 0;
        __syncthreads();
    };
    // The 32 largest keys of the first n warps (a power of two), whose lanes have theirs in order; in the first warp.
    auto merged_lists = [&](unsigned long long k, int n) {
        const int wid = tid >> 5;
#pragma unroll 1
        for (int half = n / 2; half > 0; half >>= 1) {
            if (wid >= half && wid < 2 * half) work[tid - 32 * half] = k;
            __syncthreads();
            if (wid < half) k = merged_keys<1>(k, work[tid ^ 31], lane);
            __syncthreads();
        }
        return k;
    };
    int at = v0;
    auto load = [&](Raw (&raw)[kUnroll], int from) {
        const T* p = xv + static_cast<int64_t>(from + tid) * W;
        if (from + kTile <= v1) {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) raw[i].load(p + i * NT * W);
        } else {
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (from + i * NT + tid < v1) raw[i].load(p + i * NT * W);
                else raw[i].w[0] = raw[i].w[1] = raw[i].w[2] = raw[i].w[3] = kNone;
            }
        }
    };
    float most;  // of a span
    auto add = [&](Raw (&raw)[kUnroll]) {
        const float mx = max_of<TYPE>(raw);
        most = fmaxf(most, mx);
        // (2^kSlack is far from fp32's range: few tiles move the reference)
        if (mx * a.c > fmaxf(st.r + kSlack, -kReach)) st.move(ceilf(mx * a.c));
        const float r = st.r == -INFINITY ? 0.0f : st.r;
        const unsigned long long rr = pk2(-r, -r), cc = pk2(a.c, a.c);
        unsigned long long s2 = 0, u2 = 0;
        // (t 2^t of a logit of -inf is 0: 16-bit logits are clamped in pairs before the conversion, fp32's t one by one)
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            clamp_low<TYPE>(raw[i]);
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                unsigned long long t = fma2(pk2(raw[i].get(2 * e), raw[i].get(2 * e + 1)), cc, rr);
                const float2 f = up2(t);
                const unsigned long long p = pk2(ex2(f.x), ex2(f.y));
                if (TYPE == MOE_F32) t = pk2(fmaxf(f.x, kFar), fmaxf(f.y, kFar));
                s2 = add2(s2, p);
                u2 = fma2(p, t, u2);
            }
        }
        const float2 sf = up2(s2), uf = up2(u2);
        st.s += sf.x + sf.y;
        st.u += uf.x + uf.y;
    };
    Raw even[kUnroll], odd[kUnroll];
    load(even, at);
    if (rank == 0 && tid < a.n_ids) ids[tid] = gload(a.ids + static_cast<int64_t>(row) * a.n_ids + tid);
    for (;;) {
        const bool last = at >= v1;
        if (last && !pending) break;
        most = -INFINITY;
        if (!last) {
            load(odd, at + kTile);
            add(even);
            load(even, at + 2 * kTile);
            if (at + kTile < v1) add(odd);
            st.m = fmaxf(st.m, most);
        }
        // ---- the best keys
        if (a.top) {
            const uint32_t mine = at + tid < v1 ? order(most) : 0;
            bool hot = mine > best;
            const int n_hot = __syncthreads_count(hot);
            const bool few = best && n_hot <= kHot;
            auto wait = [&]() {  // the span is looked through later
                if (!hot) return;
                const int i = atomicAdd(&hots, 1);
                hot_max[i] = mine;
                hot_at[i] = at + tid;
            };
            // what is to be done, step by step (one place for each, since this code is fetched anew for a CTA's few passes)
            enum { kNothing, kWait, kRaise, kTies, kFlush };
            int now = kNothing, then = kNothing;
            unsigned long long low = 0;
            uint32_t base = order(-INFINITY);
            if (last) {
                now = kFlush;
            } else if (n_hot && few && pending + n_hot <= kHot) {
                wait();
                pending += n_hot;
            } else if (n_hot) {
                now = few ? kWait : kRaise;
                if (pending) {
                    then = now;
                    now = kFlush;
                }
            }
            while (now != kNothing) {
                if (now == kFlush) {
                    flush(low, base);
                    hot = mine > best;
                    now = then;
                    then = kNothing;
                    continue;
                }
                if (now == kRaise) {  // a bar: a maximum that `top` threads reach, as many in each warp
                    uint32_t m = mine, r = 0;
                    for (int i = 0; i < a.top; i += NT / 32) {
                        r = __reduce_max_sync(0xffffffffu, m);
                        if (m == r) m = 0;
                    }
                    uint32_t* low32 = reinterpret_cast<uint32_t*>(work);
                    if (lane == 0) low32[tid >> 5] = r;
                    __syncthreads();
                    uint32_t least = low32[0];
#pragma unroll
                    for (int w = 1; w < NT / 32; ++w) least = min(least, low32[w]);
                    base = max(base, least);  // (0: fewer threads than that have any)
                    hot = mine >= base;
                    if (__syncthreads_count(hot) > kHot) {
                        now = kTies;
                        continue;
                    }
                }
                if (now == kTies) {  // the top-th best of the threads' best keys
                    unsigned long long mine_key = 0;
                    if (mine) {
#pragma unroll 4
                        for (int i = 0; i < kSpan * kUnroll; ++i) {
                            const int v = at + i * NT + tid;
                            if (v >= v1) break;
                            Raw y;
                            y.load(xv + static_cast<int64_t>(v) * W);
#pragma unroll
                            for (int e = 0; e < W; ++e) {
                                const unsigned long long z = key_of(y.get(e), static_cast<uint32_t>(head + v * W + e));
                                mine_key = z > mine_key ? z : mine_key;
                            }
                        }
                    }
                    const unsigned long long k = merged_lists(sorted_keys<1>(mine_key, lane), NT / 32);
                    if (tid == a.top - 1) bar = k;  // (0: fewer threads than that have any)
                    __syncthreads();
                    low = bar;
                    base = order(-INFINITY);
                    hot = mine_key && mine_key >= low;
                }
                wait();
                pending += now == kWait ? n_hot : kHot;
                if (now != kWait) {
                    __syncthreads();
                    now = kFlush;
                } else {
                    now = kNothing;
                }
            }
        }
        if (last) break;
        at += kSpan * kTile;
    }
    // a given token's logit, on its way meanwhile
    int id = -1;
    float given = 0.0f;
    if (rank == 0 && tid < a.n_ids) {
        id = ids[tid];
        if (id >= 0 && id < a.V) given = Elem<TYPE>::get(gload(x + id));
    }
    // single logits: of the row's start threads 0 .., of its end threads 8 ..
    int single = -1;
    if (rank == 0 && tid < head) single = tid;
    if (rank == C - 1 && tid >= 8 && tid < 8 + tail) single = head + nv * W + tid - 8;
    if (a.top && (C == 1 ? head + tail : rank == 0 ? head : rank == C - 1 ? tail : 0)) {
        unsigned long long k = 0;
        if (single >= 0) k = key_of(Elem<TYPE>::get(gload(x + single)), static_cast<uint32_t>(single));
        const bool more = k && (!best || k > list[a.top - 1]);
        if (__syncthreads_count(more)) {  // into its place (their keys are few)
            if (more) list[atomicAdd(&count, 1)] = k;
            __syncthreads();
            const int m = count;
            for (int i = tid; i < m; i += NT) {
                const unsigned long long mine = list[i];
                int above = 0;
                for (int j = 0; j < m; ++j) above += list[j] > mine;
                if (above < a.top) work[above] = mine;
            }
            __syncthreads();
            if (tid < min(m, a.top)) list[tid] = work[tid];
            if (tid == 0) count = min(m, a.top);
            __syncthreads();
        }
    }
    if (single >= 0) {
        const float y = Elem<TYPE>::get(gload(x + single));
        st.m = fmaxf(st.m, y);
        if (y * a.c > fmaxf(st.r + kSlack, -kReach)) st.move(ceilf(y * a.c));
        const float t = fmaf(y, a.c, st.r == -INFINITY ? 0.0f : -st.r), p = ex2(t);
        st.s += p;
        st.u = fmaf(p, fmaxf(t, kFar), st.u);
    }

    // ---- the CTA's sums, then the row's
    auto join = [&](int pass) {
        st.template join<32>();
        if (lane == 0) stat[tid >> 5] = st;
        __syncthreads();
        if (tid < 32) {  // to every CTA of the row, and the best keys to the first
            st = stat[lane & (NT / 32 - 1)];
            st.template join<NT / 32>();
            st.r = __shfl_sync(0xffffffffu, st.r, 0);
            st.s = __shfl_sync(0xffffffffu, st.s, 0);
            st.u = __shfl_sync(0xffffffffu, st.u, 0);
            st.m = __shfl_sync(0xffffffffu, st.m, 0);
        }
        if (C > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            if (!pass) cluster_wait();  // (they have all started)
            if (tid < C) *cluster.map_shared_rank(&all[pass][rank], tid) = st;
            if (!pass && tid < a.top) *cluster.map_shared_rank(best_of + rank * a.top + tid, 0) = tid < count ? list[tid] : 0;
            cluster_arrive();
            cluster_wait();
            if (tid < 32) {
                st = all[pass][lane & (kMaxCluster - 1)];
                if ((lane & (kMaxCluster - 1)) >= C) st = Stats{-INFINITY, 0.0f, 0.0f, -INFINITY};
                st.template join<kMaxCluster>();
            }
            __syncthreads();
        }
        if (tid == 0) all[pass][0] = st;
        __syncthreads();
        st = all[pass][0];
    };
    join(0);
    // Where c times the row's largest logit is too large to subtract, or a clamped logit would count next to it (rows that are masked by
    // their type's lowest value; scales near 0 or far above 1): once more, with differences first.
    const bool ends = fabsf(st.m) < INFINITY && !(fabsf(st.m * a.c) < kReach && (TYPE == MOE_F32 || ((st.m - kLow<TYPE>) * a.c > 250.0f && -kLow<TYPE> * a.c < 1e38f)));
    if (ends) {
        const float m = st.m;
        st = Stats{0.0f, 0.0f, 0.0f, m};
        auto one = [&](float y) {
            const float t = (y - m) * a.c, p = ex2(t);
            st.s += p;
            st.u = fmaf(p, fmaxf(t, kFar), st.u);
        };
        for (int v = v0 + tid; v < v1; v += NT) {
            Raw y;
            y.load(xv + static_cast<int64_t>(v) * W);
#pragma unroll
            for (int e = 0; e < W; ++e) one(y.get(e));
        }
        if (rank == 0 && tid < head) one(Elem<TYPE>::get(gload(x + tid)));
        if (rank == C - 1 && tid < tail) one(Elem<TYPE>::get(gload(x + head + nv * W + tid)));
        __syncthreads();
        join(1);
    }
    if (rank != 0) return;
    if (C > 1 && a.top) {
        const unsigned long long k = merged_lists(tid >> 5 < C && lane < a.top ? best_of[(tid >> 5) * a.top + lane] : 0, C);
        if (tid < a.top) list[tid] = k;
        __syncthreads();
    }
    const bool none = st.m == -INFINITY && st.s == st.s;  // (a row of NaN is none of -inf)
    // The log of the sum of e^(scale (x - m)), and the entropy: of at least 0, but each a difference of numbers of up to kSlack and a half, whose
    // rounding falls on either side where one token has all of the probability.
    auto above0 = [](float v) { return v < 0.0f ? 0.0f : v; };  // (a NaN stays)
    const float l2 = log2f(st.s), ls = above0((l2 - (ends ? 0.0f : fmaf(st.m, a.c, -st.r))) * kLn2);
    auto logprob = [&](float v) { return none ? -INFINITY : (v - st.m) * a.scale - ls; };
    for (int i = tid; i < a.n_ids; i += NT) {
        const int64_t to = static_cast<int64_t>(row) * a.n_ids + i;
        if (i >= NT) {
            id = gload(a.ids + to);
            if (id >= 0 && id < a.V) given = Elem<TYPE>::get(gload(x + id));
        }
        a.logprobs[to] = id >= 0 && id < a.V ? logprob(given) : -INFINITY;
    }
    if (tid < a.top) {
        const int64_t to = static_cast<int64_t>(row) * a.top + tid;
        const unsigned long long k = C > 1 || tid < count ? list[tid] : 0;
        const bool has = k != 0;
        a.top_ids[to] = has ? static_cast<int32_t>(~static_cast<uint32_t>(k)) : -1;
        a.top_logprobs[to] = has ? logprob(unorder(static_cast<uint32_t>(k >> 32))) : NAN;
    }
    if (tid == 0) {
        if (a.entropy) a.entropy[row] = none ? 0.0f : above0((l2 - st.u / st.s) * kLn2);
        if (a.lse) a.lse[row] = none ? -INFINITY : fmaf(st.m, a.scale, ls);
    }
}

template <int TYPE>
cudaError_t logprobs_t(LogprobArgs a, cudaStream_t st) {
    constexpr int W = Vec16<TYPE>::W, kTile = NT * kUnroll;
    // CTAs of a row: until there are two for every SM, and while each has more than a tile (192 rows of 65,537, fp32, top 20: two of a row 23 us,
    // four 31, as the keys are picked in each)
    a.cluster = 1;
    while (a.cluster < kMaxCluster && static_cast<int64_t>(a.rows) * a.cluster < 304 && a.V / W / a.cluster > kTile) a.cluster *= 2;
    a.c = a.scale * kLog2e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows) * a.cluster);
    cfg.blockDim = dim3(NT);
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
    if (logprobs_short(a, type)) return launch_token_logprobs_short(a, type, st);
    if (type == MOE_F32) return logprobs_t<MOE_F32>(a, st);
    if (type == MOE_F16) return logprobs_t<MOE_F16>(a, st);
    return logprobs_t<MOE_BF16>(a, st);
}

}  // namespace moe
