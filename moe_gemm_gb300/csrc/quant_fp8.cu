// Quantizers to FP8 (e4m3) with one scale per block of 128, on sm_103a: activations per
// token and 128 K, weights per [128, 128] block ("Running DeepSeek-V4-Flash-Vision on
// 4xA800", §一: FP8 weights in [128, 128] blocks, power-of-two scales).
//
//   s = amax / 448, or the smallest power of two that is no smaller;
//   q = e4m3(x / s), the quotient rounded to FP32 and then to e4m3, ties to even.
//
// What bounds the activations': instructions: 4096 x 8192 take 23 us (4.4 TB/s), with powers of two,
// which are multiplied by their reciprocal, 18.5 (5.5 TB/s); with one unit per thread 29 and 25. (The
// 4.5 us between them are one IEEE division per value. A product with the reciprocal that is
// divided only next to a tie, as the INT8 quantizers have it, would give the same codes.)
// The weights': reads, 28672 x 8192 214 us (5.5 TB/s), 8192 x 8192 72 us (4.7 TB/s); a block's rows are
// read twice, the second time from L2.
//
// 448 is the largest e4m3 number. Of a block of zeros, or below 225 * 2^-149, the scale is 0 (power of
// two: 2^-127) and the codes are 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "quant_math.cuh"

namespace w8a8 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kTop = 448.0f;
constexpr int kActThreads = 256;

// Two e4m3 codes, the first in the low byte (round to nearest even, 448 at most: values are larger only
// where amax / 448 is a few 2^-149 and was rounded down, 667 at most).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The smallest 2^e >= amax / 448 (decided exactly: amax <= 448 * 2^e), e clamped to
// [-127, 127]. 448 = 1.75 * 2^8, so for a normal amax in [2^E, 2^(E+1)) e is E - 8 or
// E - 7.
__device__ __forceinline__ float pow2_scale_fp8(float amax) {
    const int bexp = static_cast<int>(__float_as_uint(amax) >> 23);
    if (bexp == 0) return pow2_from_exponent(-127);
    int e = max(bexp - 127 - 8, -127);
    if (!(amax <= kTop * pow2_from_exponent(e))) ++e;
    return pow2_from_exponent(e);
}

__device__ __forceinline__ float scale_of(float amax, bool pow2) {
    return pow2 ? pow2_scale_fp8(amax) : __fdiv_rn(amax, kTop);
}

// The codes of 8 values under scale s. Powers of two divide exactly, by their
// reciprocal where that is a normal number.
__device__ __forceinline__ uint2 codes8_fp8(const float (&x)[8], float s, bool pow2) {
    float y[8];
    if (s == 0.0f) return make_uint2(0u, 0u);
    if (pow2 && s <= 0x1p126f && s >= 0x1p-126f) {
        const float r = __frcp_rn(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j] * r;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(x[j], s);
    }
    return make_uint2(e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16,
                      e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16);
}

// 16 lanes per (token, group), 8 values each; a thread takes kUnits of them, one block's width
// apart, all loaded before the first is worked on.
template <bool kPow2, bool kVec, int kUnits>
__global__ void __launch_bounds__(kActThreads)
quant_act_fp8_kernel(const uint16_t *a, int64_t lda, int units, int G, int chained, uint8_t *qa,
                     float *sa) {
    griddep_wait();
    // (behind the wait: when the product starts, all before this kernel is done, writers of weights too)
    if (chained) griddep_launch_dependents();
    constexpr int kPerBlock = kActThreads / 16;
    const int first = blockIdx.x * kPerBlock * kUnits + (threadIdx.x >> 4);
    const int c = threadIdx.x & 15;
    uint4 v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int u = min(first + i * kPerBlock, units - 1);
        const int m = static_cast<unsigned>(u) / static_cast<unsigned>(G);
        const uint16_t *src = a + m * lda + (u - m * G) * 128 + c * 8;
        if (kVec) {
            v[i] = __ldcs(reinterpret_cast<const uint4 *>(src));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = src[2 * j] | static_cast<uint32_t>(src[2 * j + 1]) << 16;
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        // (behind the last unit: that one again, the same values, so that every lane is at every shuffle)
        const int u = min(first + i * kPerBlock, units - 1);
        uint32_t mx = amax_bits8(v[i]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(kFull, mx, o));
        const float s = scale_of(bf16_bits_to_f32(mx), kPow2);
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
            x[2 * j + 1] = bf16_bits_to_f32(w[j] >> 16);
        }
        reinterpret_cast<uint2 *>(qa)[static_cast<int64_t>(u) * 16 + c] = codes8_fp8(x, s, kPow2);
        if (c == 0) sa[u] = s;
    }
}

// One CTA per block: 8 warps, a row of 128 values per warp at a time.
__global__ void __launch_bounds__(256)
quant_weight_fp8_kernel(const float *w, int N, int K, int pow2, uint8_t *qw, float *sw) {
    griddep_wait();
    __shared__ float s_max[8];
    const int g = blockIdx.x, b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = min(128, N - b * 128);
    const float *src = w + static_cast<int64_t>(b) * 128 * K + g * 128 + lane * 4;
    float m = 0.0f;
    for (int r = warp; r < rows; r += 8) {
        const float4 v = *reinterpret_cast<const float4 *>(src + static_cast<int64_t>(r) * K);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    m = s_max[lane & 7];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float s = scale_of(m, pow2 != 0);
    if (threadIdx.x == 0) sw[static_cast<int64_t>(b) * gridDim.x + g] = s;
    uint8_t *dst = qw + static_cast<int64_t>(b) * 128 * K + g * 128 + lane * 4;
    for (int r = warp; r < rows; r += 8) {
        const float4 v = *reinterpret_cast<const float4 *>(src + static_cast<int64_t>(r) * K);
        uint32_t q = 0;
        if (s != 0.0f)
            q = e4m3x2(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s)) |
                e4m3x2(__fdiv_rn(v.z, s), __fdiv_rn(v.w, s)) << 16;
        *reinterpret_cast<uint32_t *>(dst + static_cast<int64_t>(r) * K) = q;
    }
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream,
                   Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_act_fp8(const uint16_t *a, int64_t M, int64_t K, int64_t lda, void *qa,
                                 float *sa, bool pow2, bool chained, cudaStream_t stream) {
    // (units are below 2^31 / 128.) A long call takes four units per thread, for more loads
    // in flight; a decode step has SMs to fill.
    const int G = static_cast<int>(K >> 7);
    const int units = static_cast<int>(M * G);
    const bool many = units >= 1 << 15;
    const int per = kActThreads / 16 * (many ? 4 : 1);
    const dim3 grid(static_cast<unsigned>((units + per - 1) / per));
    const bool vec = lda % 8 == 0 && (reinterpret_cast<uintptr_t>(a) & 15) == 0;
    auto *kernel = quant_act_fp8_kernel<false, false, 1>;
    if (many)
        kernel = pow2 ? (vec ? quant_act_fp8_kernel<true, true, 4> : quant_act_fp8_kernel<true, false, 4>)
                      : (vec ? quant_act_fp8_kernel<false, true, 4> : quant_act_fp8_kernel<false, false, 4>);
    else
        kernel = pow2 ? (vec ? quant_act_fp8_kernel<true, true, 1> : quant_act_fp8_kernel<true, false, 1>)
                      : (vec ? quant_act_fp8_kernel<false, true, 1> : quant_act_fp8_kernel<false, false, 1>);
    return launch(kernel, grid, kActThreads, stream, a, lda, units, G, chained ? 1 : 0,
                  static_cast<uint8_t *>(qa), sa);
}

cudaError_t launch_quant_weight_fp8(const float *w, int64_t N, int64_t K, bool pow2, void *qw,
                                    float *sw, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(K >> 7), static_cast<unsigned>((N + 127) >> 7));
    return launch(quant_weight_fp8_kernel, grid, 256, stream, w, static_cast<int>(N),
                  static_cast<int>(K), pow2 ? 1 : 0, static_cast<uint8_t *>(qw), sw);
}

}  // namespace w8a8
