// head_rope.cu - norm and rotation of the heads of query and key rows in one pass (the mathematics and a lane's share are
// in head_rope.cuh).
//
// Bound by memory: a value is read once and written once, with five instructions. A warp takes up to kHeadsOfWarp rounds of heads of
// one token's queries or keys, so that its angles and weights serve several heads.
#include "decode_api.h"

namespace moe {

namespace {

constexpr int kThreads = 128;

template <int TYPE, int L>
__global__ void __launch_bounds__(kThreads) head_norm_rope_kernel(const HeadRopeArgs a) {
    const uint32_t id = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), per = a.qw + a.kw;
    const uint32_t token = id / per;
    const int part = static_cast<int>(id - token * per);
    if (token >= a.n) return;
    pdl_wait();
    pdl_trigger();
    const bool keys = part >= a.qw;
    const HeadSet& set = keys ? a.k : a.q;
    const int each = keys ? a.kh : a.qh, h0 = (keys ? part - a.qw : part) * each;
    rope_heads<TYPE, L>(set, a.r, a.D, a.w_type, a.eps, token, a.positions + token, 0, h0, min(set.n, h0 + each));
}

template <int TYPE, int L>
cudaError_t rope_l(HeadRopeArgs& a, cudaStream_t st) {
    constexpr int G = 32 / L;
    // rounds of heads of a warp: as few as give the device 16 warps an SM, 8 at most
    const int64_t rounds = a.n * ((a.q.n + G - 1) / G + (a.k.n + G - 1) / G);
    const int each = static_cast<int>(rounds / (152 * 16) < 1 ? 1 : rounds / (152 * 16) > 8 ? 8 : rounds / (152 * 16));
    a.qh = a.kh = each * G;
    a.qw = (a.q.n + a.qh - 1) / a.qh;
    a.kw = (a.k.n + a.kh - 1) / a.kh;
    const int64_t warps = a.n * (a.qw + a.kw);
    return launch_kernel(head_norm_rope_kernel<TYPE, L>, dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32))), dim3(kThreads), 0, st, true, a);
}

template <int TYPE>
cudaError_t rope_t(HeadRopeArgs& a, cudaStream_t st) {
    const int lanes = a.D / (2 * RawVec<TYPE>::W);
    if (lanes <= 2) return rope_l<TYPE, 2>(a, st);
    if (lanes <= 4) return rope_l<TYPE, 4>(a, st);
    if (lanes <= 8) return rope_l<TYPE, 8>(a, st);
    if (lanes <= 16) return rope_l<TYPE, 16>(a, st);
    if constexpr (TYPE == MOE_F32) return rope_l<TYPE, 32>(a, st);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_head_norm_rope(HeadRopeArgs a, int type, cudaStream_t st) {
    if (type == MOE_F32) return rope_t<MOE_F32>(a, st);
    if (type == MOE_F16) return rope_t<MOE_F16>(a, st);
    return rope_t<MOE_BF16>(a, st);
}

}  // namespace moe
