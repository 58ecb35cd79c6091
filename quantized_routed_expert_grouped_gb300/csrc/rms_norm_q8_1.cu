// rms_norm_q8_1.cu - residual addition, root-mean-square norm and the experts' q8_1 rows in one
// pass, and reading q8_1 rows back.
//
//   h = x + residual;  y = h * (1 / sqrt(mean(h^2) + eps)) * weight;  xq = q8_1(y)
//
// One CTA per row; a thread holds eight consecutive values of C chunks in registers, so the row is
// read once and the outputs may overwrite the inputs. A q8_1 block of 32 values is four
// neighbouring threads. The sum of squares is fp32: per thread, then over the warp's lanes, then
// over the warps in order.
//
// Bound by memory where there are many rows; what the kernel adds is latency (a row's loads, one barrier,
// its stores), which other rows' CTAs cover, and the arithmetic, kept to a dozen instructions a value by
// packed pairs and by codes that are divided out only next to a tie.
// Measured (GB300, of 6787 GB/s that a copy reaches): 8191 rows of 4096, bf16, with the residual, the sum,
// y and q8_1 rows: 47 us for 134 MB read and 172 MB written (6.4 TB/s, issue slots 74 % full), fp32 85 us for 575 MB
// (6.8 TB/s; in fp32 half as many CTAs an SM, as at 32 registers the row spilled: 118 us; 16-bit rows at 32 spill 24 bytes, fp32 ones of more than 16,384 columns
// 200); reading the q8_1 rows
// back 14 us for 38 MB and 67 MB (much of it still in L2 at the end). Four rows: 1 to 3 us each.
#include "internal.h"
#include "kv8.cuh"
#include "kv8_api.h"

namespace moe {

namespace {

// the q8_1 block of four neighbouring lanes' values (32 in all): the lane's codes and header word
__device__ __forceinline__ void quad_q8_1(const float (&y)[8], uint32_t (&code)[2], uint32_t& hdr) {
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(y[e]));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float d = __fdiv_rn(amax, 127.0f);
    // Candidates: y * (1 / d) is within 2^-15 of the quotient, and adding 1.5 * 2^23 rounds it to an
    // integer, in the low bits. Where one lies that near a tie (or 1 / d is not a normal number), the
    // lane's codes are taken from the quotients.
    const float inv = d > 1.1754944e-38f && d < 3.4028234e38f ? __fdiv_rn(1.0f, d) : 0.0f;
    const unsigned long long vv = pk2(inv, inv), up = pk2(12582912.0f, 12582912.0f), down = pk2(-12582912.0f, -12582912.0f);
    unsigned long long x[4], sum = 0;
    float far = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const unsigned long long r = mul2(pk2(y[2 * e], y[2 * e + 1]), vv);
        x[e] = add2(r, up);
        const unsigned long long n = add2(x[e], down);
        const float2 rr = up2(r), nn = up2(n);
        far = fmaxf(far, fmaxf(fabsf(rr.x - nn.x), fabsf(rr.y - nn.y)));
        sum = add2(sum, n);
    }
    const float2 s2 = up2(sum);
    float S = s2.x + s2.y;
    code[0] = pack4(lo2(x[0]), hi2(x[0]), lo2(x[1]), hi2(x[1]));
    code[1] = pack4(lo2(x[2]), hi2(x[2]), lo2(x[3]), hi2(x[3]));
    if (!(far < 0.5f - 3.0517578125e-5f) || inv == 0.0f) {
        int sum_i = 0;
        code[0] = code[1] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int q = d == 0.0f ? 0 : static_cast<int>(roundf(__fdiv_rn(y[e], d)));
            sum_i += q;
            code[e >> 2] |= static_cast<uint32_t>(q & 255) << (8 * (e & 3));
        }
        S = static_cast<float>(sum_i);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    hdr = __half_as_ushort(__float2half_rn(d)) | static_cast<uint32_t>(__half_as_ushort(__float2half_rn(__fmul_rn(d, S)))) << 16;
}

__device__ __forceinline__ void weight8(const void* w, int w_type, int col, float (&v)[8]) {
    if (w_type == MOE_F32) load8<MOE_F32>(static_cast<const float*>(w) + col, true, v);
    else if (w_type == MOE_F16) load8<MOE_F16>(static_cast<const __half*>(w) + col, true, v);
    else load8<MOE_BF16>(static_cast<const __nv_bfloat16*>(w) + col, true, v);
}

template <int TYPE, int C>
__global__ void __launch_bounds__(1024, C == 2 && TYPE != MOE_F32 ? 2 : 1) add_rms_norm_q8_1_kernel(const moe_norm_call c) {
    using E = Elem<TYPE>;
    using T = typename E::T;
    __shared__ float red[32];
    pdl_wait();
    pdl_trigger();
    const int64_t row = blockIdx.x;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const T* x = static_cast<const T*>(c.x) + row * c.x_stride;
    const T* r = c.residual ? static_cast<const T*>(c.residual) + row * c.residual_stride : nullptr;
    Raw8<TYPE> rx[C], rr[C];
#pragma unroll
    for (int k = 0; k < C; ++k) {  // all of the row's loads before the arithmetic
        const int col = (k * blockDim.x + threadIdx.x) * 8;
        rx[k].clear();
        rr[k].clear();
        if (col < c.cols) {
            rx[k].load(x + col, true);
            if (r) rr[k].load(r + col, true);
        }
    }
    unsigned long long h[C][4], s2 = 0;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[k][e] = add2(pk2(rx[k].get(2 * e), rx[k].get(2 * e + 1)), pk2(rr[k].get(2 * e), rr[k].get(2 * e + 1)));
            s2 = fma2(h[k][e], h[k][e], s2);
        }
    const float2 ss2 = up2(s2);
    float ss = ss2.x + ss2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) red[wid] = ss;
    __syncthreads();  // also: every thread's reads of the row lie before the writes below
    ss = 0.0f;
    for (int w = 0; w < nw; ++w) ss += red[w];
    auto put8 = [&](T* to, const float (&v)[8], bool on) {
        if (C > 1) store8_pair<TYPE, 1>(to, true, v, on);
        else if (on) store8<TYPE>(to, true, v);  // (few rows: the exchange would add to the chain)
    };
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, static_cast<float>(c.cols)) + c.eps));
#pragma unroll
    for (int k = 0; k < C; ++k) {
        // a warp's columns are whole q8_1 blocks, and lanes past the row carry zeros into its shuffles
        const int col = (k * blockDim.x + threadIdx.x) * 8;
        const bool in = col < c.cols;
        if (!__any_sync(0xffffffffu, in)) continue;
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (c.sum) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = up2(h[k][e]);
                y[2 * e] = v.x;
                y[2 * e + 1] = v.y;
            }
            put8(static_cast<T*>(c.sum) + row * c.cols + col, y, in);
        }
        if (in) {
            weight8(c.weight, c.w_type, col, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = up2(mul2(mul2(h[k][e], pk2(inv, inv)), pk2(y[2 * e], y[2 * e + 1])));
                y[2 * e] = v.x;
                y[2 * e + 1] = v.y;
            }
        }
        if (c.y) put8(static_cast<T*>(c.y) + row * c.cols + col, y, in);
        if (c.xq) {
            uint32_t code[2], hdr;
            quad_q8_1(y, code, hdr);
            if (in) {
                uint32_t* blk = reinterpret_cast<uint32_t*>(c.xq + row * (c.cols / 32) + col / 32);
                const int part = (col >> 3) & 3;
                blk[1 + 2 * part] = code[0];
                blk[2 + 2 * part] = code[1];
                if (part == 0) blk[0] = hdr;
            }
        }
    }
}

// N pieces of eight values a thread, all loaded first: with one the loads in flight do not cover memory's
// latency where there are many rows.
template <int TYPE, int N>
__global__ void __launch_bounds__(256) dequantize_q8_1_kernel(const moe_q8_1* xq, int64_t n_blocks,
                                                              typename Elem<TYPE>::T* out) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (256 * N) + threadIdx.x, n = n_blocks * 4;
    pdl_wait();
    pdl_trigger();
    uint32_t hdr[N], w[N][2];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t i = i0 + k * 256;
        hdr[k] = w[k][0] = w[k][1] = 0;
        if (i >= n) continue;
        const uint32_t* blk = reinterpret_cast<const uint32_t*>(xq + (i >> 2));
        const int part = static_cast<int>(i & 3);
        hdr[k] = gload(blk);
        w[k][0] = gload(blk + 1 + 2 * part);
        w[k][1] = gload(blk + 2 + 2 * part);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t i = i0 + k * 256;
        const float d = h2f_bits(hdr[k]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)  // code + 128 in the low bits of 2^23
            v[e] = d * __fadd_rn(__uint_as_float(prmt(w[k][e >> 2] ^ 0x80808080u, 0x4b000000u, 0x7440u + (e & 3))), -8388736.0f);
        store8_pair<TYPE, 1>(out + i * 8, true, v, i < n);
    }
}

}  // namespace

namespace {

template <int TYPE>
cudaError_t norm_t(const moe_norm_call& c, cudaStream_t st) {
    const int pieces = c.cols / 8;
    const unsigned grid = static_cast<unsigned>(c.rows);
    // few rows: as many threads as the row has pieces, for the shortest chain; many, or long ones: two pieces a
    // thread, and four where a CTA's threads do not reach (6169 rows of 10720: two 97 us, four 120; fp32 217, 250)
    const int chunks = pieces > 2048 ? 4 : pieces > 1024 || (c.rows > 304 && pieces >= 64) ? 2 : 1;
    const int threads = ((pieces + chunks - 1) / chunks + 31) / 32 * 32;
    if (chunks == 1) return launch_kernel(add_rms_norm_q8_1_kernel<TYPE, 1>, dim3(grid), dim3(threads), 0, st, true, c);
    if (chunks == 2) return launch_kernel(add_rms_norm_q8_1_kernel<TYPE, 2>, dim3(grid), dim3(threads), 0, st, true, c);
    return launch_kernel(add_rms_norm_q8_1_kernel<TYPE, 4>, dim3(grid), dim3(threads), 0, st, true, c);
}

template <int TYPE>
cudaError_t dequantize_t(const moe_q8_1* xq, int64_t n_blocks, typename Elem<TYPE>::T* out, cudaStream_t st) {
    constexpr int kMany = 2;
    const int64_t pieces = n_blocks * 4;
    if (pieces <= 304 * 2048)  // at most two rounds of the device's threads
        return launch_kernel(dequantize_q8_1_kernel<TYPE, 1>, dim3(static_cast<unsigned>((pieces + 255) / 256)), dim3(256), 0, st, true, xq, n_blocks, out);
    constexpr int kCta = 256 * kMany;
    return launch_kernel(dequantize_q8_1_kernel<TYPE, kMany>, dim3(static_cast<unsigned>((pieces + kCta - 1) / kCta)), dim3(256), 0, st, true, xq,
                         n_blocks, out);
}

}  // namespace

cudaError_t launch_add_rms_norm_q8_1(const moe_norm_call& c, cudaStream_t st) {
    if (c.rows == 0) return cudaSuccess;
    if (c.type == MOE_F32) return norm_t<MOE_F32>(c, st);
    if (c.type == MOE_F16) return norm_t<MOE_F16>(c, st);
    return norm_t<MOE_BF16>(c, st);
}

cudaError_t launch_dequantize_q8_1(const moe_q8_1* xq, int64_t n_blocks, void* out, int type, cudaStream_t st) {
    if (n_blocks == 0) return cudaSuccess;
    if (type == MOE_F32) return dequantize_t<MOE_F32>(xq, n_blocks, static_cast<float*>(out), st);
    if (type == MOE_F16) return dequantize_t<MOE_F16>(xq, n_blocks, static_cast<__half*>(out), st);
    return dequantize_t<MOE_BF16>(xq, n_blocks, static_cast<__nv_bfloat16*>(out), st);
}

}  // namespace moe
