// kv8_attention.cu - planning the attention call, and the kernel that joins the parts of sequences
// that several CTAs worked on.
#include <algorithm>

#include "kv8_attention.cuh"

namespace moe {

namespace {

// WPR warps take one output row's parts in turn; a part is (row / l, m, l), its weight l 2^(m - M) / L.
// Rows of a segment that one CTA held whole are in out already; a sequence without blocks gives
// zeros here.
// Bound by latency (2.5 MB of parts and a chain of two loads: 2 to 4 us behind the attention kernel).
// The loads of a run of parts are in flight together with those of every part's m and l; several
// warps a row where the rows are few. Joining in the CTA that ends last instead, in one kernel, took
// longer (its fence and counter are paid by every CTA).
template <int WPR>
__global__ void __launch_bounds__(256) kv8_combine_kernel(const AttnPlan p) {
    constexpr int kRows = 8 / WPR;
    __shared__ float acc[WPR > 1 ? 8 : 1][256];
    pdl_wait();
    pdl_trigger();
    const AttnArgs& a = p.a;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, sub = wid / WPR, w = wid - sub * WPR, D = a.c.D;
    const int row = blockIdx.x * kRows + sub, rows = a.c.n_seqs * a.T * a.n_heads;
    if (row >= rows) return;  // WPR == 1 where more than one row shares the CTA
    const int bt = row / a.n_heads, h = row - bt * a.n_heads, b = bt / a.T, t = bt - b * a.T;
    const int kv = h / a.G, r = t * a.G + h - kv * a.G, rb = r / p.g.RP, rr = r - rb * p.g.RP;
    const int at = p.plan[b], n = p.plan[b + 1] - at, chunk = p.plan[a.c.n_seqs + 1];
    const int s0 = at * p.segs + (kv * p.g.RB + rb) * n;  // in the list
    int i0 = 0, cnt = 0;
    bool head = false;
    if (n > 0) {
        if (chunk) {
            i0 = (s0 + kAttnSegCost) / chunk;  // the CTA of the first block
            cnt = (s0 + n - 1) / chunk - i0 + 1;
            head = s0 <= static_cast<int64_t>(i0) * chunk;  // that CTA has no block of an earlier segment
        } else {  // a CTA per part
            i0 = s0;
            cnt = n;
            head = true;
        }
        if (cnt == 1) return;
    }
    const int64_t pf = attn_part_floats(p.g.RP, D), ml = static_cast<int64_t>(p.g.RP) * D + rr;
    auto part = [&](int j) { return p.parts + (2LL * (i0 + j) + (j == 0 && !head ? 1 : 0)) * pf; };
    constexpr int kRun = 4;
    float4 y[kRun][2];
    float ym[kRun], yl[kRun];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const int j = j0 + k * WPR;
            ym[k] = -INFINITY;
            yl[k] = 0.0f;
            if (j >= cnt) continue;
            const float* q = part(j);
            ym[k] = q[ml];
            yl[k] = q[ml + p.g.RP];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i * 128 + lane * 4 < D) y[k][i] = *reinterpret_cast<const float4*>(q + static_cast<int64_t>(rr) * D + i * 128 + lane * 4);
        }
    };
    fetch(w);  // with the loads of all parts' m and l below
    float M = -INFINITY, Ls = 0.0f;
    for (int j = lane; j < cnt; j += 32) {  // (a lane's running sum, for its running maximum)
        const float m = part(j)[ml], l = part(j)[ml + p.g.RP], nm = fmaxf(M, m), bs = nm == -INFINITY ? 0.0f : nm;
        Ls = Ls * ex2(M - bs) + l * ex2(m - bs);
        M = nm;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m = __shfl_xor_sync(0xffffffffu, M, o), l = __shfl_xor_sync(0xffffffffu, Ls, o);
        const float nm = fmaxf(M, m), bs = nm == -INFINITY ? 0.0f : nm;
        Ls = Ls * ex2(M - bs) + l * ex2(m - bs);
        M = nm;
    }
    const float base = M == -INFINITY ? 0.0f : M, inv = Ls == 0.0f ? 0.0f : 1.0f / Ls;
    float4 v[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
    for (int j0 = w; j0 < cnt; j0 += WPR * kRun) {
        if (j0 != w) fetch(j0);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if (j0 + k * WPR >= cnt) continue;
            const float wt = yl[k] * ex2(ym[k] - base) * inv;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (i * 128 + lane * 4 < D) {
                    v[i].x = fmaf(wt, y[k][i].x, v[i].x);
                    v[i].y = fmaf(wt, y[k][i].y, v[i].y);
                    v[i].z = fmaf(wt, y[k][i].z, v[i].z);
                    v[i].w = fmaf(wt, y[k][i].w, v[i].w);
                }
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
                if (i * 128 + lane * 4 < D) {
                    const float4 y = *reinterpret_cast<const float4*>(&acc[wid + k][i * 128 + lane * 4]);
                    v[i].x += y.x;
                    v[i].y += y.y;
                    v[i].z += y.z;
                    v[i].w += y.w;
                }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = i * 128 + lane * 4;
        if (d >= D) continue;
        if (p.out_type == MOE_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + static_cast<int64_t>(row) * D + d) = v[i];
        } else if (p.out_type == MOE_F16) {
            __half2* q = reinterpret_cast<__half2*>(static_cast<__half*>(a.out) + static_cast<int64_t>(row) * D + d);
            q[0] = __floats2half2_rn(v[i].x, v[i].y);
            q[1] = __floats2half2_rn(v[i].z, v[i].w);
        } else {
            __nv_bfloat162* q = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + static_cast<int64_t>(row) * D + d);
            q[0] = __floats2bfloat162_rn(v[i].x, v[i].y);
            q[1] = __floats2bfloat162_rn(v[i].z, v[i].w);
        }
    }
    if (a.lse && lane == 0) a.lse[row] = Ls == 0.0f ? -INFINITY : M * kLn2 + logf(Ls);
}

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
        e = cudaFuncSetAttribute(kv8_combine_kernel<8>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kv8_combine_kernel<1>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_relaxed);
    }
    // few rows have many parts each
    if (rows <= 1024)
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
