// kv8_attention.cu - attention of a verify window over the 8-bit cache.
//
// For a row (query token t, head h) and the positions j it sees: s_j = scale * q . k_j,
// m = max s_j, out = sum e^(s_j - m) v_j / sum e^(s_j - m), kept as a running maximum, sum and
// weighted row that are rescaled when the maximum grows.
#include "internal.h"
#include "kv8.cuh"
#include "kv8_api.h"

namespace moe {

namespace {

constexpr int kWarps = 4;

// One CTA per (sequence, query token, head); a warp takes every fourth block of 32 tokens, lane =
// token for the scores and lane = dims lane, lane + 32, .. for the weighted values.
template <int TYPE>
__global__ void __launch_bounds__(kWarps * 32) kv8_attention_kernel(AttnArgs a) {
    using E = Elem<TYPE>;
    extern __shared__ float sm[];
    const int D = a.c.D, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int h = blockIdx.x % a.n_heads, t = blockIdx.x / a.n_heads % a.T, b = blockIdx.x / a.n_heads / a.T;
    float* qs = sm;               // [D]
    float* part = sm + D;         // [kWarps][D + 2]
    const typename E::T* q = static_cast<const typename E::T*>(a.q) + b * a.qs + t * a.qt + h * a.qh;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) qs[d] = E::get(q[d]);
    __syncthreads();
    int len = a.lens[b];
    const int64_t cap = static_cast<int64_t>(a.c.max_pages) * a.c.page_blocks * 32;
    if (len < 0) {
        set_err(a.err, MOE_ERR_LEN);
        len = 0;
    }
    if (len > cap) {
        set_err(a.err, MOE_ERR_PAGE);
        len = static_cast<int>(cap);
    }
    const int pos = len - a.T + t;
    const uint32_t bits = a.tree ? static_cast<uint32_t>(a.tree[b * a.T + t]) : 0u;
    float m = -INFINITY, l = 0.0f, o[8];
    for (int i = 0; i < 8; ++i) o[i] = 0.0f;
    const int nblk = pos < 0 ? 0 : (len + 31) / 32;
    for (int j = wid; j < nblk; j += kWarps) {
        const uint8_t* rec = kv8_record(a.c, b, j, h / a.G, a.err);
        if (!rec) continue;
        const float ks = reinterpret_cast<const float*>(rec)[0], vs = reinterpret_cast<const float*>(rec)[1];
        const int key = j * 32 + lane;
        float dot = 0.0f;
        for (int d = 0; d < D; ++d) dot += qs[d] * (rec[kv8_k_at(D, lane, d)] - 128);
        float s = dot * ks * a.scale;
        const int w = key - (len - a.T);
        const bool see = key < len && (a.tree ? (w < 0 || (bits >> w & 1u)) : key <= pos) &&
                         (a.window == 0 || key > pos - a.window);
        if (!see) s = -INFINITY;
        float bm = s;
        for (int x = 16; x > 0; x >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, x));
        if (!__any_sync(0xffffffffu, see)) continue;
        const float nm = fmaxf(m, bm), base = nm == -INFINITY ? 0.0f : nm;
        const float al = expf(m - base);
        const float p = see ? expf(s - base) : 0.0f;
        float sum = p;
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = l * al + sum;
        m = nm;
        for (int i = 0; i < D / 32; ++i) {
            float acc = 0.0f;
            for (int x = 0; x < 32; ++x) {
                const float px = __shfl_sync(0xffffffffu, p, x);
                if (px != 0.0f) acc += px * (rec[kv8_v_at(D, x, i * 32 + lane)] - 128);
            }
            o[i] = o[i] * al + acc * vs;
        }
    }
    float* mine = part + wid * (D + 2);
    for (int i = 0; i < D / 32; ++i) mine[i * 32 + lane] = o[i];
    if (lane == 0) {
        mine[D] = m;
        mine[D + 1] = l;
    }
    __syncthreads();
    float mx = -INFINITY, total = 0.0f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, part[w * (D + 2) + D]);
    const float base = mx == -INFINITY ? 0.0f : mx;
    for (int w = 0; w < kWarps; ++w) total += part[w * (D + 2) + D + 1] * expf(part[w * (D + 2) + D] - base);
    const int64_t row = (static_cast<int64_t>(b) * a.T + t) * a.n_heads + h;
    typename E::T* out = static_cast<typename E::T*>(a.out) + row * D;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float acc = 0.0f;
        for (int w = 0; w < kWarps; ++w) acc += part[w * (D + 2) + d] * expf(part[w * (D + 2) + D] - base);
        out[d] = E::put(total == 0.0f ? 0.0f : acc / total);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = base + logf(total);
}

}  // namespace

cudaError_t launch_kv8_attention(const AttnArgs& a, int type, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(a.c.n_seqs * a.T * a.n_heads);
    const int smem = (a.c.D + kWarps * (a.c.D + 2)) * 4;
    if (type == MOE_F32) kv8_attention_kernel<MOE_F32><<<grid, kWarps * 32, smem, st>>>(a);
    else if (type == MOE_F16) kv8_attention_kernel<MOE_F16><<<grid, kWarps * 32, smem, st>>>(a);
    else kv8_attention_kernel<MOE_BF16><<<grid, kWarps * 32, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
