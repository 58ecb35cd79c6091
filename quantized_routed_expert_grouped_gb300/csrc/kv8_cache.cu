// kv8_cache.cu - quantising keys and values into the paged 8-bit cache, and reading them back.
#include "internal.h"
#include "kv8.cuh"
#include "kv8_api.h"

namespace moe {

namespace {

constexpr int kThreads = 128;

// max of non-negative values that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) kv8_write_kernel(KvCache c, KvRows<const typename Elem<TYPE>::T> K,
                                                             KvRows<const typename Elem<TYPE>::T> V,
                                                             int64_t n_tokens, const int32_t* cu, const int32_t* start,
                                                             int32_t* err) {
    __shared__ float red[4];
    const int h = blockIdx.y, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const KvSlot s = kv8_slot(blockIdx.x, cu, start, c.n_seqs, n_tokens, err);
    if (s.b < 0) return;
    uint8_t* rec = kv8_record(c, s.b, s.blk, h, err);
    if (!rec) return;
    const int pieces = c.D / 8;
    for (int w = 0; w < 2; ++w) {  // keys, then values
        const auto& R = w ? V : K;
        const auto* base = R.p + s.row * R.ts + h * R.hs;
        float amax = 0.0f, v[8];
        for (int i = s.t0 * pieces + threadIdx.x; i < s.t1 * pieces; i += kThreads) {
            const int t = i / pieces, d = (i - t * pieces) * 8;
            load8<TYPE>(base + t * R.ts + d, R.vec, v);
            for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v[e]));
        }
        for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (lane == 0) red[wid] = amax;
        __syncthreads();
        amax = max_nan(max_nan(red[0], red[1]), max_nan(red[2], red[3]));
        float* sp = reinterpret_cast<float*>(rec) + w;
        const float old = s.t0 > 0 ? *sp : 0.0f;
        __syncthreads();
        float scale = amax < kKvTiny ? 0.0f : __fdiv_rn(amax, 127.0f);
        scale = max_nan(old, scale);
        if (!(scale <= 3.4028234e38f)) scale = __int_as_float(0x7fffffff);
        const bool some = scale > 0.0f;
        const float inv = some ? __fdiv_rn(1.0f, scale) : 0.0f, ratio = some ? __fdiv_rn(old, scale) : 0.0f;
        for (int i = s.t0 * pieces + threadIdx.x; i < s.t1 * pieces; i += kThreads) {
            const int t = i / pieces, d = (i - t * pieces) * 8;
            load8<TYPE>(base + t * R.ts + d, R.vec, v);
            for (int e = 0; e < 8; ++e) {
                const int q = some ? __float2int_rn(fminf(fmaxf(__fmul_rn(v[e], inv), -127.0f), 127.0f)) : 0;
                rec[w ? kv8_v_at(c.D, t, d + e) : kv8_k_at(c.D, t, d + e)] = static_cast<uint8_t>(q + 128);
            }
        }
        if (s.t0 > 0 && scale != old)
            for (int i = threadIdx.x; i < s.t0 * c.D; i += kThreads) {
                const int t = i / c.D, d = i - t * c.D;
                uint8_t* p = rec + (w ? kv8_v_at(c.D, t, d) : kv8_k_at(c.D, t, d));
                const int q = some ? __float2int_rn(__fmul_rn(static_cast<float>(*p - 128), ratio)) : 0;
                *p = static_cast<uint8_t>(q + 128);
            }
        if (threadIdx.x == 0) *sp = scale;
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads) kv8_read_kernel(KvCache c, KvRows<typename Elem<TYPE>::T> K,
                                                            KvRows<typename Elem<TYPE>::T> V, int64_t n_tokens,
                                                            const int32_t* cu, const int32_t* start, int32_t* err) {
    const int h = blockIdx.y;
    const KvSlot s = kv8_slot(blockIdx.x, cu, start, c.n_seqs, n_tokens, err);
    if (s.b < 0) return;
    const uint8_t* rec = kv8_record(c, s.b, s.blk, h, err);
    if (!rec) return;
    const int pieces = c.D / 8;
    for (int w = 0; w < 2; ++w) {
        const auto& R = w ? V : K;
        auto* base = R.p + s.row * R.ts + h * R.hs;
        const float scale = reinterpret_cast<const float*>(rec)[w];
        for (int i = s.t0 * pieces + threadIdx.x; i < s.t1 * pieces; i += kThreads) {
            const int t = i / pieces, d = (i - t * pieces) * 8;
            float v[8];
            for (int e = 0; e < 8; ++e)
                v[e] = (rec[w ? kv8_v_at(c.D, t, d + e) : kv8_k_at(c.D, t, d + e)] - 128) * scale;
            store8<TYPE>(base + t * R.ts + d, R.vec, v);
        }
    }
}

template <int TYPE>
cudaError_t write_t(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start, int32_t* err,
                    bool kvec, bool vvec, dim3 grid, cudaStream_t st) {
    using T = typename Elem<TYPE>::T;
    const KvRows<const T> K{static_cast<const T*>(r.k), r.k_token_stride, r.k_head_stride, kvec};
    const KvRows<const T> V{static_cast<const T*>(r.v), r.v_token_stride, r.v_head_stride, vvec};
    kv8_write_kernel<TYPE><<<grid, kThreads, 0, st>>>(c, K, V, r.n_tokens, cu, start, err);
    return cudaGetLastError();
}

template <int TYPE>
cudaError_t read_t(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start, int32_t* err,
                   bool kvec, bool vvec, dim3 grid, cudaStream_t st) {
    using T = typename Elem<TYPE>::T;
    const KvRows<T> K{static_cast<T*>(r.k), r.k_token_stride, r.k_head_stride, kvec};
    const KvRows<T> V{static_cast<T*>(r.v), r.v_token_stride, r.v_head_stride, vvec};
    kv8_read_kernel<TYPE><<<grid, kThreads, 0, st>>>(c, K, V, r.n_tokens, cu, start, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_write(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start,
                             int32_t* err, bool kvec, bool vvec, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(kv8_slots(r.n_tokens, c.n_seqs)), c.n_kv);
    if (r.type == MOE_F32) return write_t<MOE_F32>(c, r, cu, start, err, kvec, vvec, grid, st);
    if (r.type == MOE_F16) return write_t<MOE_F16>(c, r, cu, start, err, kvec, vvec, grid, st);
    return write_t<MOE_BF16>(c, r, cu, start, err, kvec, vvec, grid, st);
}

cudaError_t launch_kv8_read(const KvCache& c, const moe_kv8_rows& r, const int32_t* cu, const int32_t* start,
                            int32_t* err, bool kvec, bool vvec, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(kv8_slots(r.n_tokens, c.n_seqs)), c.n_kv);
    if (r.type == MOE_F32) return read_t<MOE_F32>(c, r, cu, start, err, kvec, vvec, grid, st);
    if (r.type == MOE_F16) return read_t<MOE_F16>(c, r, cu, start, err, kvec, vvec, grid, st);
    return read_t<MOE_BF16>(c, r, cu, start, err, kvec, vvec, grid, st);
}

}  // namespace moe
