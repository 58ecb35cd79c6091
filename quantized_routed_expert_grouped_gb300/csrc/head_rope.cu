// head_rope.cu - norm and rotation of the heads of query and key rows in one pass (the mathematics and a lane's share are
// in head_rope.cuh).
//
// A CTA takes up to four tokens. Its warps compute the tokens' angles and lay out the weights in shared memory while
// each one's first heads are on their way; then a warp takes a token's heads, round after round, with the next round's loads in flight.
// Bound by memory where there are many rows, else by its chain of latencies. Measured (GB300, of 6703 GB/s that a copy
// reaches): 8191 tokens of 72 heads of 128 dims, bf16, normed and rotated: 51.7 us for 302 MB read and written (5.8 TB/s; 54 % of
// the issue slots, 24 warps an SM at 72 registers). With angles and weights in registers, 118 a thread, it took 63; without a limit on registers
// 59. 256 tokens of 40 heads, fp32: 3.2 us; one token: 2.3 us.
#include "decode_api.h"

namespace moe {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32, kMaxTokens = 4;

template <int TYPE, int L, bool VEC>
__global__ void __launch_bounds__(kThreads, 7) head_norm_rope_kernel(const HeadRopeArgs a) {
    extern __shared__ __align__(16) float sm[];
    using Warp = RopeWarp<TYPE, L, VEC>;
    constexpr int W = Warp::W, G = Warp::G;
    // the CTA's tokens t0 .. t0 + n; this warp's first one, and its rounds r0 .. r1 of a token's (queries', then keys')
    const int wid = threadIdx.x >> 5, tile = blockIdx.x / a.splits, split = blockIdx.x - tile * a.splits;
    const int64_t t0 = static_cast<int64_t>(tile) * a.tokens;
    const int n = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.n - t0));
    const int first = wid / a.warps, rq = (a.q.n + G - 1) / G, rounds = rq + (a.k.n + G - 1) / G;
    const int part = split * a.warps + wid - first * a.warps, parts = a.splits * a.warps;
    const int r0 = rounds * part / parts, r1 = rounds * (part + 1) / parts;
    const int q0 = r0 * G, q1 = min(a.q.n, r1 * G), k0 = max(r0 - rq, 0) * G, k1 = min(a.k.n, (r1 - rq) * G);
    float *qw = sm + n * a.r.rot, *kw = qw + a.D;
    Warp w(a.r, a.D);
    pdl_wait();
    pdl_trigger();
    if (first < n) {
        if (q0 < q1) w.start(a.q, t0 + first, q0, q1);
        else if (k0 < k1) w.start(a.k, t0 + first, k0, k1);
    }
    if (a.r.rot) put_angles<W>(sm, a.r, n, a.r.rot, [&](int t) { return gload(a.positions + t0 + t); });
    if (a.q.weight) put_weights<W>(qw, a.r, a.D, a.q.weight, a.w_type);
    if (a.k.weight) put_weights<W>(kw, a.r, a.D, a.k.weight, a.w_type);
    __syncthreads();
    for (int t = first; t < n; t += kWarps / a.warps) {
        const float* angles = sm + t * a.r.rot;
        if (q0 < q1) {
            if (t != first) w.start(a.q, t0 + t, q0, q1);
            w.run(a.q, a.r, a.D, a.eps, angles, qw, t0 + t, q0, q1);
        }
        if (k0 < k1) {
            if (t != first || q0 < q1) w.start(a.k, t0 + t, k0, k1);
            w.run(a.k, a.r, a.D, a.eps, angles, kw, t0 + t, k0, k1);
        }
    }
}

template <int TYPE, int L, bool VEC>
cudaError_t rope_l(HeadRopeArgs& a, cudaStream_t st) {
    constexpr int G = 32 / L;
    // Many tokens: up to four a CTA, so that weights and setting up serve several (8191 tokens of 72 heads of 128: 51.7 us, with
    // eight 52.1, with sixteen 57); few: a token's rounds over the CTA's warps, and over several CTAs. Three a CTA (2736 to 3647 tokens) leave a warp in
    // four without any: 3000 tokens take 22.5 us, 3400, a second wave of CTAs, 32.0, 4000, four a CTA, 26.7.
    const int rounds = (a.q.n + G - 1) / G + (a.k.n + G - 1) / G;
    const int64_t each = a.n / (152 * 6);
    a.tokens = static_cast<int>(each < 1 ? 1 : each > kMaxTokens ? kMaxTokens : each);
    a.warps = a.tokens >= kWarps ? 1 : kWarps / a.tokens;  // of a token in a CTA
    a.splits = 1;
    while (a.n * a.splits < 152 * 2 && a.splits * a.warps < rounds) ++a.splits;
    const int64_t grid = (a.n + a.tokens - 1) / a.tokens * a.splits;
    return launch_kernel(head_norm_rope_kernel<TYPE, L, VEC>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), rope_smem(a.r.rot, a.D, a.tokens), st, true, a);
}

template <int TYPE, bool VEC>
cudaError_t rope_v(HeadRopeArgs& a, cudaStream_t st) {
    const int lanes = a.D / (2 * RawVec<TYPE, VEC>::W);
    if (lanes <= 2) return rope_l<TYPE, 2, VEC>(a, st);
    if (lanes <= 4) return rope_l<TYPE, 4, VEC>(a, st);
    if (lanes <= 8) return rope_l<TYPE, 8, VEC>(a, st);
    if (lanes <= 16) return rope_l<TYPE, 16, VEC>(a, st);
    if constexpr (TYPE == MOE_F32) return rope_l<TYPE, 32, VEC>(a, st);
    return cudaErrorInvalidValue;
}

template <int TYPE>
cudaError_t rope_t(HeadRopeArgs& a, cudaStream_t st) {
    const bool vec = (a.q.n == 0 || (a.q.xvec && a.q.ovec)) && (a.k.n == 0 || (a.k.xvec && a.k.ovec));
    return vec ? rope_v<TYPE, true>(a, st) : rope_v<TYPE, false>(a, st);
}

}  // namespace

cudaError_t launch_head_norm_rope(HeadRopeArgs a, int type, cudaStream_t st) {
    if (type == MOE_F32) return rope_t<MOE_F32>(a, st);
    if (type == MOE_F16) return rope_t<MOE_F16>(a, st);
    return rope_t<MOE_BF16>(a, st);
}

}  // namespace moe
