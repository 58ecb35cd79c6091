// token_logprobs_short.cu - token_logprobs of rows that fit in shared memory: a warp a row, or two or four.
//
//   t_j = (x_j - m) c,  s = sum 2^t_j,  u = sum t_j 2^t_j   (m the row's largest logit, c = scale log2 e);
//   log p_j = scale (x_j - m) - ln 2 log2 s,  lse = scale m + ln 2 log2 s,  entropy = ln 2 (log2 s - u / s)
//
// The row comes by asynchronous copies, all in flight at once, and a thread reads what it has copied itself, for m and then for
// the sums. Meanwhile it picks what can be among the most likely tokens: each thread has had the maxima of two halves of its logits, and
// the top-th largest of all of those (in order by sorting networks over the lanes, merged over the warps) is a bar that `top` logits reach, and
// seldom many more. These, as keys of value and index (larger for a larger value, and among equal ones for the lower index), are
// appended to a list, and put in order 32 at a time by the same networks: their order in the list does not matter. Where more reach the bar than
// the list holds (ties, masked rows), the top-th best value is found by halving, and of those that equal it the first are taken,
// in the order of their indices: never more work than a pass over the row for each bit of a value.
//
// Bound by its instructions (17.7 a lane and logit of 16,000 in bf16, top 20, 71 % of the issue slots: 13.6 are the copies and the two passes, which
// a row without the best tokens takes too, 2.3 the bar and the first key, 1.8 the other nineteen; the other kernel's one pass takes 8.6 in all. Fused
// products and clamps in pairs, as there, take as long), a row of its own by 3 us of latencies. Measured (GB300): bf16, top 20: 2000 rows of 2000 8.3 us (by
// the other kernel 24), of 16,000 28.9 (39); fp32: 8000 of 19 10 us (37), of 1000 15.8 (66), of 4000 39 us for 128 MB (97).
#include "token_logprobs.cuh"

namespace moe {

namespace {

constexpr int kRows = 4, kCap = 128;  // rows of a CTA at most; keys of a list
// Bytes of a row at most: a rule on the bytes alone. Measured, bf16, us by the other kernel / here:
//   rows, KB      top 0          top 1          top 5          top 20
//   1 of 32       3.0 / 4.6      5.3 / 5.9      5.4 / 6.0      6.6 / 6.4
//   4 of 43       3.0 / 5.4      5.5 / 6.8      6.4 / 7.0      8.4 / 7.5
//   64 of 43      3.7 / 5.6      6.4 / 7.0      7.4 / 7.2      9.9 / 7.7
//   192 of 43     6.1 / 6.6      9.4 / 7.9      9.6 / 8.2      14.1 / 8.6
//   608 of 32     5.5 / 8.7      8.1 / 10.5     9.1 / 10.9     14.6 / 11.6
//   2000 of 32    20.7 / 21.1    29.5 / 25.5    29.6 / 26.2    37.7 / 27.6
//   2000 of 43    24.2 / 31.7    34.7 / 37.3    38.0 / 38.2    48.9 / 40.1
// It gains with many of the best tokens and with hundreds of rows; few rows near the limit lose by it up to 1.3 us with the best token or five, and calls without
// the best tokens up to 2.6, thousands of rows 7.5: there a rule on `top` too would choose the other kernel.
constexpr int kRowBytes = 48 * 1024;

__device__ __forceinline__ void copy16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

// G: warps of a row. One: a CTA has several rows, whose warps go on their own; else a row.
template <int TYPE, int G>
__global__ void __launch_bounds__(G == 1 ? kRows * 32 : G * 32, G == 1 ? 8 : 4) token_logprobs_short_kernel(const LogprobArgs a) {
    using Raw = Vec16<TYPE>;
    using T = typename Elem<TYPE>::T;
    constexpr int W = Raw::W, kThreads = G * 32;
    extern __shared__ __align__(16) uint4 rows[];
    __shared__ unsigned long long lists[G == 1 ? kRows : 1][kCap];
    __shared__ int counts[G == 1 ? kRows : 1];
    __shared__ uint32_t bins[G][32], tops[G];  // of the warps
    __shared__ float2 sums[G];
    const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31, mine = G == 1 ? wid : 0;  // (mine: the row's place in the CTA)
    const int tid = G == 1 ? lane : threadIdx.x;                                        // of the row
    const int row = G == 1 ? blockIdx.x * (blockDim.x >> 5) + wid : blockIdx.x;
    pdl_wait();
    pdl_trigger();
    if (row >= a.rows) return;  // (of a CTA of several rows: the warp)
    const T* x = static_cast<const T*>(a.x) + row * a.stride;
    const int head = min(a.V, static_cast<int>((-reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T)));
    const int nv = (a.V - head) / W, tail = a.V - head - nv * W;
    uint4* held = rows + mine * (a.V / W);
    unsigned long long* list = lists[mine];
    int& count = counts[mine];
    for (int v = tid; v < nv; v += kThreads) copy16(held + v, x + head + v * W);
    // single logits, before the row's first 16-byte boundary and after its last: threads 0 .. and 8 ..
    const int single = tid < head ? tid : tid >= 8 && tid < 8 + tail ? head + nv * W + tid - 8 : -1;
    const float alone = single < 0 ? -INFINITY : Elem<TYPE>::get(gload(x + single));
    const int64_t id0 = static_cast<int64_t>(row) * a.n_ids;
    int id = tid < a.n_ids ? gload(a.ids + id0 + tid) : -1;
    float given = id >= 0 && id < a.V ? Elem<TYPE>::get(gload(x + id)) : -INFINITY;
    if (tid == 0) count = 0;
    asm volatile("cp.async.wait_all;" ::: "memory");
    auto vec = [&](int v) {
        Raw r;
        *reinterpret_cast<uint4*>(r.w) = held[v];
        return r;
    };

    // ---- the largest logits of the thread's halves (even and odd elements; a NaN does not count), and of the row
    float m0 = -INFINITY, m1 = -INFINITY;
    if constexpr (TYPE == MOE_F32) {
#pragma unroll 2
        for (int v = tid; v < nv; v += kThreads) {
            const Raw r = vec(v);
            m0 = fmaxf(m0, fmaxf(r.get(0), r.get(2)));
            m1 = fmaxf(m1, fmaxf(r.get(1), r.get(3)));
        }
    } else {
        using H = typename std::conditional<TYPE == MOE_F16, __half2, __nv_bfloat162>::type;
        uint32_t none = TYPE == MOE_F16 ? 0xfc00fc00u : 0xff80ff80u;  // -inf
        H h = *reinterpret_cast<const H*>(&none);
#pragma unroll 2
        for (int v = tid; v < nv; v += kThreads) {
            const Raw r = vec(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) h = __hmax2(h, *reinterpret_cast<const H*>(&r.w[i]));
        }
        const float2 f = TYPE == MOE_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&h)) : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&h));
        m0 = f.x;
        m1 = f.y;
    }
    m0 = fmaxf(m0, alone);
    uint32_t most = __reduce_max_sync(0xffffffffu, order(fmaxf(m0, m1))), bar = 0;
    auto reversed = [&](auto k) { return __shfl_xor_sync(0xffffffffu, k, 31); };
    if (a.top) bar = merged_keys<5>(sorted_keys<5>(order(m0), lane), reversed(sorted_keys<5>(order(m1), lane)), lane);
    if (G > 1) {
        bins[wid][lane] = bar;
        if (lane == 0) tops[wid] = most;
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < G; ++w) {
            most = max(most, tops[w]);
            if (a.top && w != wid) bar = merged_keys<5>(bar, bins[w][31 - lane], lane);
        }
    }
    __syncwarp();
    const float m = unorder(most);
    bar = __shfl_sync(0xffffffffu, bar, max(a.top - 1, 0));
    // bits of a vector's logits of at least `least`
    auto reach = [&](const Raw& r, float least) {
        uint32_t hits = 0;
        float y = fmaxf(r.get(0), r.get(1));
#pragma unroll
        for (int e = 2; e < W; ++e) y = fmaxf(y, r.get(e));
        if (y >= least) {
#pragma unroll
            for (int e = 0; e < W; ++e) hits |= r.get(e) >= least ? 1u << e : 0u;
        }
        return hits;
    };
    // keys of some logits of vectors v, v + step, .. (W bits each) are appended, as many as there is place for
    auto append = [&](uint32_t hits, int v, int step) {
        if (!hits) return;
        int at = atomicAdd(&count, __popc(hits));
        for (; hits && at < kCap; hits &= hits - 1, ++at) {
            const int b = __ffs(hits) - 1, i = (v + b / W * step) * W + b % W;
            list[at] = key_of(Elem<TYPE>::get(reinterpret_cast<const T*>(held)[i]), static_cast<uint32_t>(head + i));
        }
    };
    auto append_single = [&]() {
        const int at = atomicAdd(&count, 1);
        if (at < kCap) list[at] = key_of(alone, static_cast<uint32_t>(single));
    };

    // ---- the sums (t 2^t of a logit of -inf is 0), and what reaches the bar
    const bool low = bar == order(-INFINITY);  // (which only counts where too few are above it)
    const float base = m == -INFINITY ? 0.0f : m, least = a.top ? unorder(low ? bar + 1 : bar) : NAN;
    float s = 0.0f, u = 0.0f;
    const unsigned long long mm = pk2(-base, -base), cc = pk2(a.c, a.c);
    uint32_t hits = 0;
    int n_hits = 0;  // vectors whose bits are in it
    int v = tid;
    for (; v < nv; v += kThreads) {
        const Raw r = vec(v);
        unsigned long long s2 = 0, u2 = 0;
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            const float2 t = up2(mul2(add2(pk2(r.get(2 * e), r.get(2 * e + 1)), mm), cc));
            const unsigned long long p = pk2(ex2(t.x), ex2(t.y));
            s2 = add2(s2, p);
            u2 = fma2(p, pk2(fmaxf(t.x, kFar), fmaxf(t.y, kFar)), u2);
        }
        const float2 sf = up2(s2), uf = up2(u2);
        s += sf.x + sf.y;
        u += uf.x + uf.y;
        hits |= reach(r, least) << n_hits * W;
        if (++n_hits == 32 / W) {
            append(hits, v - (n_hits - 1) * kThreads, kThreads);
            hits = n_hits = 0;
        }
    }
    append(hits, v - n_hits * kThreads, kThreads);
    if (single >= 0) {
        const float t = (alone - base) * a.c, p = ex2(t);
        s += p;
        u = fmaf(p, fmaxf(t, kFar), u);
        if (alone >= least) append_single();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {  // (the same in every lane)
        s += __shfl_xor_sync(0xffffffffu, s, o);
        u += __shfl_xor_sync(0xffffffffu, u, o);
    }
    if (G > 1) {
        if (lane == 0) sums[wid] = make_float2(s, u);
        __syncthreads();
        s = u = 0.0f;
#pragma unroll
        for (int w = 0; w < G; ++w) {
            s += sums[w].x;
            u += sums[w].y;
        }
    }
    __syncwarp();
    const bool none = m == -INFINITY && s == s;  // (a row of NaN is none of -inf)
    const float l2 = log2f(s), ls = l2 * kLn2;   // log of the sum of e^(scale (x - m))
    auto logprob = [&](float v) { return none ? -INFINITY : (v - m) * a.scale - ls; };
    for (int i = tid; i < a.n_ids; i += kThreads) {
        if (i >= kThreads) {
            id = gload(a.ids + id0 + i);
            if (id >= 0 && id < a.V) given = Elem<TYPE>::get(gload(x + id));
        }
        a.logprobs[id0 + i] = id >= 0 && id < a.V ? logprob(given) : -INFINITY;
    }
    if (tid == 0) {
        if (a.entropy) a.entropy[row] = none ? 0.0f : (l2 - u / s) * kLn2;
        if (a.lse) a.lse[row] = none ? -INFINITY : fmaf(m, a.scale, ls);
    }
    if (!a.top || tid >= 32) return;

    // ---- the best keys, by a warp
    int n = count;
    if (low || n > kCap) {
        // Too many reach the bar (ties; or it is -inf): those above it; where those are too many, the top-th best value
        // instead, and those above that; and, as far as places are left, the first that equal it.
        auto above = [&](uint32_t o) {
            __syncwarp();
            if (lane == 0) count = 0;
            __syncwarp();
            const float y = unorder(o + 1);
#pragma unroll 1
            for (int v = lane; v < nv; v += 32) append(reach(vec(v), y), v, 0);
            if (single >= 0 && alone >= y) append_single();
            __syncwarp();
            return count;
        };
        if (!low) n = above(bar);
        if (n > kCap) {
            uint32_t over = most + 1;  // (which none reach; the bar is reached by `top` at least)
#pragma unroll 1
            while (over - bar > 1) {
                const uint32_t mid = bar + (over - bar) / 2;
                const float y = unorder(mid);
                int c = alone >= y;
#pragma unroll 1
                for (int v = lane; v < nv; v += 32) {
                    const Raw r = vec(v);
#pragma unroll
                    for (int e = 0; e < W; ++e) c += r.get(e) >= y;
                }
                (static_cast<int>(__reduce_add_sync(0xffffffffu, c)) >= a.top ? bar : over) = mid;
            }
            n = above(bar);
        }
        // hits: a bit for each of a lane's logits (all of the same value) from `first` on, in order over the lanes
        const float same = unorder(bar);
        auto level = [&](uint32_t hits, int first) {
            const int c = __popc(hits);
            int upto = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            for (int at = n + upto - c; hits && at < a.top; hits &= hits - 1, ++at) list[at] = key_of(same, static_cast<uint32_t>(first + __ffs(hits) - 1));
            n += __shfl_sync(0xffffffffu, upto, 31);
        };
        if (n < a.top) {
            level(lane < head && alone == same, lane);
#pragma unroll 1
            for (int v = lane; v - lane < nv && n < a.top; v += 32) {
                uint32_t hits = 0;
                if (v < nv) {
                    const Raw r = vec(v);
#pragma unroll
                    for (int e = 0; e < W; ++e) hits |= r.get(e) == same ? 1u << e : 0u;
                }
                level(hits, head + v * W);
            }
            level(lane >= 8 && single >= 0 && alone == same, single);
            n = min(n, a.top);
        }
        __syncwarp();
    }
    unsigned long long best = 0;
#pragma unroll 1
    for (int i = 0; i < n; i += 32) {
        const unsigned long long k = sorted_keys<5>(i + lane < n ? list[i + lane] : 0ull, lane);
        best = i ? merged_keys<5>(best, reversed(k), lane) : k;
    }
    if (lane < a.top) {
        const int64_t to = static_cast<int64_t>(row) * a.top + lane;
        a.top_ids[to] = best ? static_cast<int32_t>(~static_cast<uint32_t>(best)) : -1;
        a.top_logprobs[to] = best ? logprob(unorder(static_cast<uint32_t>(best >> 32))) : NAN;
    }
}

// Whether rows are so many that a CTA each leaves none idle: then fewer warps a row.
bool many(const LogprobArgs& a) { return a.rows > 152 * 4; }
int64_t row_bytes(const LogprobArgs& a, int type) { return static_cast<int64_t>(a.V / (type == MOE_F32 ? 4 : 8)) * 16; }

template <int TYPE, int G>
cudaError_t short_g(LogprobArgs a, cudaStream_t st) {
    const int bytes = static_cast<int>(row_bytes(a, TYPE));
    a.c = a.scale * kLog2e;
    if (G == 1) return launch_kernel(token_logprobs_short_kernel<TYPE, G>, dim3((a.rows + kRows - 1) / kRows), dim3(kRows * 32), kRows * bytes, st, true, a);
    if (bytes > 44 * 1024) {  // (with the rest above what every launch may have)
        const cudaError_t e = cudaFuncSetAttribute(token_logprobs_short_kernel<TYPE, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowBytes);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(token_logprobs_short_kernel<TYPE, G>, dim3(a.rows), dim3(G * 32), bytes, st, true, a);
}

// Warps of a row, measured with bf16, top 5, by one, two and four: 2000 rows of 4 KB 7.7, 8.7, 10.9 us; of 16 KB 21.7, 16.0, 16.1; of 32 KB
// 45.7, 35.1, 27.4; 300 rows of 8 KB 7.3, 6.1, 5.9; one of 200 bytes 4.7, 4.9, 5.5.
template <int TYPE>
cudaError_t short_t(const LogprobArgs& a, cudaStream_t st) {
    const int64_t bytes = row_bytes(a, TYPE);
    if (bytes <= (many(a) ? 4096 : 1024)) return short_g<TYPE, 1>(a, st);
    return many(a) && bytes <= 16 * 1024 ? short_g<TYPE, 2>(a, st) : short_g<TYPE, 4>(a, st);
}

}  // namespace

bool logprobs_short(const LogprobArgs& a, int type) { return row_bytes(a, type) <= kRowBytes; }

cudaError_t launch_token_logprobs_short(const LogprobArgs& a, int type, cudaStream_t st) {
    if (type == MOE_F32) return short_t<MOE_F32>(a, st);
    if (type == MOE_F16) return short_t<MOE_F16>(a, st);
    return short_t<MOE_BF16>(a, st);
}

}  // namespace moe
