// kv8_attention.cu - planning the attention call, and the kernel that joins the parts of sequences
// that several CTAs worked on.
#include <algorithm>

#include "kv8_attention.cuh"

namespace moe {

namespace {

// A row's place in the list: its parts i0 .. i0 + cnt (cnt 1: one CTA held the row's segment whole, it is in
// out already), each in its CTA's first slot but a first one that is not at the CTA's start.
struct RowParts {
    const float* parts;
    int64_t pf, ml;  // floats of a part; its m, RP floats before its l
    int i0, cnt, rr;
    bool head;
    __device__ __forceinline__ RowParts(const AttnPlan& p, int row) {
        const AttnArgs& a = p.a;
        const int bt = row / a.n_heads, h = row - bt * a.n_heads, b = bt / a.T, t = bt - b * a.T;
        const int kv = h / a.G, r = t * a.G + h - kv * a.G, rb = r / p.g.RP;
        rr = r - rb * p.g.RP;
        const int at = p.plan[b], n = p.plan[b + 1] - at, chunk = p.plan[a.c.n_seqs + 1];
        const int s0 = at * p.segs + (kv * p.g.RB + rb) * n;  // in the list
        i0 = s0;
        cnt = n;
        head = true;
        if (n > 0 && chunk) {  // (else a CTA per part)
            i0 = (s0 + kAttnSegCost) / chunk;  // the CTA of the first block
            cnt = (s0 + n - 1) / chunk - i0 + 1;
            head = s0 <= static_cast<int64_t>(i0) * chunk;  // that CTA has no block of an earlier segment
        }
        parts = p.parts;
        pf = attn_part_floats(p.g.RP, a.c.D);
        ml = static_cast<int64_t>(p.g.RP) * a.c.D + rr;
    }
    __device__ __forceinline__ const float* part(int j) const { return parts + (2LL * (i0 + j) + (j == 0 && !head ? 1 : 0)) * pf; }
};

// (M, Ls) joined with (m, l)
__device__ __forceinline__ void join_ml(float& M, float& Ls, float m, float l) {
    const float nm = fmaxf(M, m), bs = nm == -INFINITY ? 0.0f : nm;
    Ls = Ls * ex2(M - bs) + l * ex2(m - bs);
    M = nm;
}
// The power 2^(m - M) by which a part counts, as a factor of its weight and one of its rows: fp32 may not hold it as one,
// while the rows' values are as far above the other parts'. (To the sum of the weights such a part adds nothing.)
__device__ __forceinline__ float2 part_power(float m, float M) {
    constexpr float kLeast = -120.0f;
    return make_float2(ex2(fmaxf(m - M, kLeast)), ex2(fminf(m - M - kLeast, 0.0f)));
}
__device__ __forceinline__ void axpy4(float w, const float4& y, float4& v) {
    v.x = fmaf(w, y.x, v.x);
    v.y = fmaf(w, y.y, v.y);
    v.z = fmaf(w, y.z, v.z);
    v.w = fmaf(w, y.w, v.w);
}
__device__ __forceinline__ void axpy4(float2 w, const float4& y, float4& v) {
    axpy4(w.x, make_float4(y.x * w.y, y.y * w.y, y.z * w.y, y.w * w.y), v);
}
__device__ __forceinline__ void put_out(const AttnPlan& p, int row, int d, const float4& v) {
    const int64_t at = static_cast<int64_t>(row) * p.a.c.D + d;
    if (p.out_type == MOE_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.a.out) + at) = v;
    } else if (p.out_type == MOE_F16) {
        __half2* q = reinterpret_cast<__half2*>(static_cast<__half*>(p.a.out) + at);
        q[0] = __floats2half2_rn(v.x, v.y);
        q[1] = __floats2half2_rn(v.z, v.w);
    } else {
        __nv_bfloat162* q = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.a.out) + at);
        q[0] = __floats2bfloat162_rn(v.x, v.y);
        q[1] = __floats2bfloat162_rn(v.z, v.w);
    }
}

// A part is (row / l, m, l), its weight l 2^(m - M) / L. A sequence without blocks gives zeros here.
// Bound by latency: a few MB of parts, behind a chain of two loads (the plan, the parts). Joining in the
// CTA that ends last instead, in one kernel, took longer (its fence and counter are paid by every CTA).
//
// A segment that may have more than kManyParts parts (it has at most a block a warp, and an even share of the CTAs
// where lengths are even): a CTA for 64 dims of a row. Every part's m and l are loaded at once, a thread each (two past
// 256), and the rows of 128 parts at once, sixteen threads each, before the first wait. 131k tokens of 4 heads: 31.8 us
// for the call against 34.6 with the kernel below, a million tokens of one 90.9 against 94.5; 777 tokens 10.4 against 9.8.
constexpr int kManyParts = 32;
constexpr int kSlice = 64, kSubs = 256 / (kSlice / 4), kAtOnce = 8;
static_assert(kAttnMaxCtas <= 512, "two parts a thread");
__global__ void __launch_bounds__(256) kv8_combine_parts_kernel(const AttnPlan p) {
    __shared__ float2 wt[512];
    __shared__ float wm[8];
    __shared__ float4 acc[8][kSlice / 4 + 1];
    pdl_wait();
    pdl_trigger();
    const int D = p.a.c.D, slices = (D + kSlice - 1) / kSlice, row = blockIdx.x / slices, slice = blockIdx.x - row * slices;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31, sub = tid >> 4, d = slice * kSlice + (tid & 15) * 4;
    const RowParts x(p, row);
    if (x.cnt == 1) return;
    float m[2], l[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = tid + i * 256;
        const float* q = x.part(j) + x.ml;
        m[i] = j < x.cnt ? q[0] : -INFINITY;
        l[i] = j < x.cnt ? q[p.g.RP] : 0.0f;
    }
    float4 y[kAtOnce];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int j = j0 + k * kSubs;
            if (j < x.cnt && d < D) y[k] = *reinterpret_cast<const float4*>(x.part(j) + static_cast<int64_t>(x.rr) * D + d);
        }
    };
    fetch(sub);
    float M = fmaxf(m[0], m[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) wm[wid] = M;
    __syncthreads();
    M = wm[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) M = fmaxf(M, wm[k]);
    const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (i == 0 || x.cnt > 256) {
            const float2 w = part_power(m[i], base);
            wt[tid + i * 256] = make_float2(l[i] * w.x, w.y);
        }
    __syncthreads();
    float4 v = make_float4(0, 0, 0, 0);
    float L = 0.0f;
    for (int j0 = sub; j0 < x.cnt; j0 += kSubs * kAtOnce) {
        if (j0 != sub) fetch(j0);
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (j0 + k * kSubs < x.cnt) {
                const float2 w = wt[j0 + k * kSubs];
                L += w.x;
                if (d < D) axpy4(w, y[k], v);
            }
    }
    __syncwarp();
    L += __shfl_xor_sync(0xffffffffu, L, 16);
    v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
    v.z += __shfl_xor_sync(0xffffffffu, v.z, 16);
    v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
    if (lane < 16) acc[wid][lane] = v;
    if (lane == 0) acc[wid][kSlice / 4].x = L;
    __syncthreads();
    if (tid < 16) {
#pragma unroll
        for (int k = 1; k < 8; ++k) {
            axpy4(1.0f, acc[k][tid], v);
            L += acc[k][kSlice / 4].x;
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        if (d < D) put_out(p, row, d, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        if (p.a.lse && slice == 0 && tid == 0) p.a.lse[row] = L == 0.0f ? -INFINITY : M * kLn2 + logf(L);
    }
}

// Else WPR warps a row, a run of kRun parts each at once; a warp a row where there are many, most of them of few
// parts or one (16 x 64 rows of 3 to 4 parts: 29.5 us for the call against 32.9 with eight; 4 x 128 of 14: 23.0 and 21.7).
template <int WPR>
__global__ void __launch_bounds__(256) kv8_combine_kernel(const AttnPlan p) {
    constexpr int kRun = 4;
    __shared__ float acc[WPR > 1 ? 8 : 1][256];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, w = wid % WPR, D = p.a.c.D;
    const int row = blockIdx.x * (8 / WPR) + wid / WPR;
    if (row >= p.a.c.n_seqs * p.a.T * p.a.n_heads) return;  // WPR == 1 where more than one row shares the CTA
    const RowParts x(p, row);
    if (x.cnt == 1) return;
    float4 y[kRun][2];
    float ym[kRun], yl[kRun];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const int j = j0 + k * WPR;
            ym[k] = -INFINITY;
            yl[k] = 0.0f;
            if (j >= x.cnt) continue;
            const float* q = x.part(j);
            ym[k] = q[x.ml];
            yl[k] = q[x.ml + p.g.RP];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i * 128 + lane * 4 < D) y[k][i] = *reinterpret_cast<const float4*>(q + static_cast<int64_t>(x.rr) * D + i * 128 + lane * 4);
        }
    };
    fetch(w);  // with the loads of all parts' m and l below
    float M = -INFINITY, Ls = 0.0f;
    for (int j = lane; j < x.cnt; j += 32)  // (a lane's running sum, for its running maximum)
        join_ml(M, Ls, x.part(j)[x.ml], x.part(j)[x.ml + p.g.RP]);
    __syncwarp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m = __shfl_xor_sync(0xffffffffu, M, o), l = __shfl_xor_sync(0xffffffffu, Ls, o);
        join_ml(M, Ls, m, l);
    }
    const float base = M == -INFINITY ? 0.0f : M, inv = Ls == 0.0f ? 0.0f : 1.0f / Ls;
    float4 v[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
    for (int j0 = w; j0 < x.cnt; j0 += WPR * kRun) {
        if (j0 != w) fetch(j0);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if (j0 + k * WPR >= x.cnt) continue;
            float2 wt = part_power(ym[k], base);
            wt.x *= yl[k] * inv;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i * 128 + lane * 4 < D) axpy4(wt, y[k][i], v[i]);
        }
    }
    if (WPR > 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i * 128 + lane * 4 < D) *reinterpret_cast<float4*>(&acc[wid][i * 128 + lane * 4]) = v[i];
        __syncthreads();
        if (w) return;
        for (int k = 1; k < WPR; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i * 128 + lane * 4 < D) axpy4(1.0f, *reinterpret_cast<const float4*>(&acc[wid + k][i * 128 + lane * 4]), v[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (i * 128 + lane * 4 < D) put_out(p, row, i * 128 + lane * 4, v[i]);
    if (p.a.lse && lane == 0) p.a.lse[row] = Ls == 0.0f ? -INFINITY : M * kLn2 + logf(Ls);
}
constexpr int kFewRows = 768;

}  // namespace

int64_t attn_workspace_bytes(int n_seqs, int T, int n_heads, int n_kv, int D) {
    // (as much as any smaller head_dim asks for, so that a workspace serves smaller calls too)
    const int R = T * (n_heads / n_kv), one = attn_geom(R, false).RP, two = attn_geom(R, true).RP;
    const int64_t floats = std::max(attn_part_floats(one, D), attn_part_floats(two, std::min(D, 128)));
    return attn_plan_bytes(n_seqs) + 2LL * kAttnMaxCtas * floats * 4;
}

// The list of blocks, with the segments' fixed parts, is counted in 32 bits.
bool attn_list_fits(const AttnArgs& a) {
    const double most = 1.0 * a.c.n_seqs * a.c.n_kv * attn_geom(a.T * a.G, false).RB * (1.0 * a.c.max_pages * a.c.page_blocks + kAttnSegCost);
    return most < 2147483647.0 - 2 * kAttnMaxCtas;
}

cudaError_t launch_attn_combine(const AttnPlan& p, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(p.a.c.n_seqs) * p.a.T * p.a.n_heads;
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(kv8_combine_parts_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kv8_combine_kernel<8>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kv8_combine_kernel<1>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_relaxed);
    }
    const int64_t blocks = static_cast<int64_t>(p.a.c.max_pages) * p.a.c.page_blocks;
    if (blocks > kManyParts * kAttnWarps && static_cast<int64_t>(p.a.c.n_seqs) * p.segs * kManyParts < kAttnMaxCtas) {
        const int64_t slices = rows * ((p.a.c.D + kSlice - 1) / kSlice);
        return launch_kernel(kv8_combine_parts_kernel, dim3(static_cast<unsigned>(slices)), dim3(256), 0, st, true, p);
    }
    if (rows <= kFewRows)
        return launch_kernel(kv8_combine_kernel<8>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, true, p);
    return launch_kernel(kv8_combine_kernel<1>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, st, true, p);
}

cudaError_t launch_kv8_attention(const AttnArgs& a, int type, cudaStream_t st) {
    AttnPlan p{};
    p.a = a;
    p.R = a.T * a.G;
    const int64_t blocks = static_cast<int64_t>(a.c.n_seqs) * a.c.n_kv * a.c.max_pages * a.c.page_blocks;
    p.g = attn_geom(p.R, type != MOE_F32 && a.c.D <= 128 && p.R > 16 && blocks >= kAttnLong);
    p.prec = type == MOE_F32 ? kAttnSplit : type == MOE_F16 && (p.R <= 16 || blocks < kAttnShort) ? kAttnWeights : kAttnPlain;
    p.segs = a.c.n_kv * p.g.RB;
    p.out_type = type;
    p.plan = static_cast<int*>(a.workspace);
    p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + attn_plan_bytes(a.c.n_seqs));
    const cudaError_t e = type == MOE_F32 ? launch_attn_f32(p, st) : type == MOE_F16 ? launch_attn_f16(p, st) : launch_attn_bf16(p, st);
    return e == cudaSuccess ? launch_attn_combine(p, st) : e;
}

}  // namespace moe
