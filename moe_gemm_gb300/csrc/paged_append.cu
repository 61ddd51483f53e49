// Append to the paged KV cache with the position rotation on the way, on sm_103a:
// queries and keys of new tokens are turned by their positions, the queries go
// to the caller's rows, keys and values into their slots ("Deploying Hunyuan
// 770B in INT8 on domestic accelerators", §3.4: every key and value vector gets
// its own scale when it is written). The slots and positions are those of
// paged_kv.cu's plan.
//
//   angle  of a token at position p, pair i: p * inv_freq[i], i < rot / 2;
//   turn   (a, b) -> (a cos - b sin, b cos + a sin), (a, b) the elements i and
//          rot / 2 + i of a head, or its neighbours 2 i and 2 i + 1; elements
//          rot .. 127 stay;
//   write  q rounded to BF16; k and v to BF16 pages, or to INT8 with amax / 127.
//
// The angle is needed modulo a full turn, and p * inv_freq passes 2^20 radians, where
// binary32 has no fraction left of a turn's 2^-4. So it is kept in turns, as a 64-bit
// fraction: F = inv_freq / 2 pi modulo 1, times 2^64 (one FP64 product), and p * F
// wraps by itself, exactly. F is off by 2^-55 of a turn (inv_freq up to 1), p * F by
// 2^-24 at the largest position; its nearest quarter is taken off as integers, so that what
// goes to sine and cosine is at most pi / 4 and a binary32 number of full precision.
//
// One CTA per token and run of heads. Its first rot / 2 threads make the sines
// and cosines once, in shared memory; then 16 lanes take a head's vector, 8 values
// each. A lane's partners are in the lane rot / 16 further (one shuffle of
// its 16 bytes), or its own.
//
// What bounds it: a prompt's tokens with INT8 pages (8192 x 64 + 8 + 8 heads, 319 MB) take 69 us,
// 4.6 TB/s, with 68 % of the issue slots used; BF16 pages (4097 x 32 + 8 + 8, half a head turned,
// 101 MB) 15.8 us, 6.4 TB/s of a measured 6.7. 256 threads per token: 77 and 17.3 us (a CTA's
// chain of position, sine and barrier in front of half the work), three vectors in flight 75
// and 17. 32 tokens take 3.7 us, launch and that chain; there a token's heads are
// divided among CTAs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "quant_math.cuh"

namespace w8a8 {
namespace {

constexpr int kThreads = 128;
constexpr int kPerPass = kThreads / 16;      // vectors that a CTA takes at a time
constexpr unsigned kFull = 0xFFFFFFFFu;

struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t qt, qh, kt, kh, vt, vh, ot, oh;
    const int32_t *positions, *slots;
    const float *inv_freq;
    int half;                                // rot / 2
    float amplitude;
    int Hq, Hkv, page, n_slots;
    int run;                                 // vectors of a CTA
    uint16_t *q_out;
    void *kc, *vc;
    float *ks, *vs;
};

// cos and sin of 2 pi * (phase / 2^64).
__device__ __forceinline__ float2 cos_sin_of(uint64_t phase) {
    const int32_t h = static_cast<int32_t>(phase >> 32);     // turns * 2^32
    const int32_t quarter = (h >> 30) + ((h >> 29) & 1);     // the nearest
    const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(h) -
                                              (static_cast<uint32_t>(quarter) << 30));
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a : a, quarter & 2 ? -b : b);
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// The codes of 8 values of magnitude at most amax, s = amax / 127.
__device__ __forceinline__ uint2 quantize8_f32(const float (&x)[8], float s) {
    const bool fast = s >= 1.17549435e-38f;       // a normal scale: 1 / s is finite
    const float r = fast ? __frcp_rn(s) : 0.0f;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = code_plus_round(x[j], s, r, fast);
    return make_uint2(pack_code_bytes(f[0], f[1], f[2], f[3]),
                      pack_code_bytes(f[4], f[5], f[6], f[7]));
}

template <bool kInt8, bool kPairs, int U>
__global__ void __launch_bounds__(kThreads)
paged_kv_append_kernel(const AppendArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ float2 s_turn[64];
    const int64_t t = blockIdx.x;
    const int p = a.positions[t];
    if (p < 0) return;                       // (a refused request's token: nothing is written)
    const int c = threadIdx.x & 15;
    const int end = min(a.Hq + 2 * a.Hkv, static_cast<int>(blockIdx.y + 1) * a.run);
    const int first = blockIdx.y * a.run + (threadIdx.x >> 4);
    auto load = [&](int n) {
        const uint16_t *src = n < a.Hq           ? a.q + t * a.qt + n * a.qh
                              : n < a.Hq + a.Hkv ? a.k + t * a.kt + (n - a.Hq) * a.kh
                                                 : a.v + t * a.vt + (n - a.Hq - a.Hkv) * a.vh;
        return __ldcs(reinterpret_cast<const uint4 *>(src) + c);
    };
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        x[u] = first + u * kPerPass < end ? load(first + u * kPerPass) : make_uint4(0, 0, 0, 0);
    const int slot = a.slots[t];
    if (threadIdx.x < a.half) {
        const double turns = static_cast<double>(a.inv_freq[threadIdx.x]) * 0.15915494309189533577;
        const int64_t f = __double2ll_rn((turns - rint(turns)) * 0x1p64);
        const float2 cs = cos_sin_of(static_cast<uint64_t>(f) * static_cast<uint32_t>(p));
        s_turn[threadIdx.x] = make_float2(cs.x * a.amplitude, cs.y * a.amplitude);
    }
    __syncthreads();
    // a lane's cosines and sines: of its 8 elements, or of its 4 pairs
    constexpr int kMine = kPairs ? 4 : 8;
    float cs[kMine], sn[kMine];
    const int lanes = a.half >> 3;           // half the lanes that turn
    const bool turns = c < 2 * lanes;
    const bool upper = !kPairs && c >= lanes;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int i = kPairs ? 4 * c + j : 8 * (upper ? c - lanes : c) + j;
        const float2 v = turns ? s_turn[i] : make_float2(1.0f, 0.0f);
        cs[j] = v.x;
        sn[j] = upper ? v.y : -v.y;          // of the partner's share
    }
    const int partner = (threadIdx.x & 16) + (!turns ? c : upper ? c - lanes : c + lanes);
    const int page_of = slot / a.page;
    const bool has_slot = slot >= 0 && slot < a.n_slots;
    for (int n0 = blockIdx.y * a.run; n0 < end; n0 += U * kPerPass) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (n0 + u * kPerPass >= end) break;             // (the same for the CTA)
            const int n = n0 + u * kPerPass + (threadIdx.x >> 4);
            uint4 w = x[u];
            const int next = n + U * kPerPass;
            if (next < end) x[u] = load(next);
            float y[8];
            uint32_t *ww = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[2 * j] = bf16_bits_to_f32(ww[j] & 0xFFFFu);
                y[2 * j + 1] = bf16_bits_to_f32(ww[j] >> 16);
            }
            const bool rotated = n < a.Hq + a.Hkv;
            if (kPairs) {
                if (rotated && turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float e = y[2 * j], o = y[2 * j + 1];
                        y[2 * j] = fmaf(e, cs[j], o * sn[j]);
                        y[2 * j + 1] = fmaf(o, cs[j], -(e * sn[j]));
                    }
                }
            } else {
                uint4 z;
                z.x = __shfl_sync(kFull, w.x, partner);
                z.y = __shfl_sync(kFull, w.y, partner);
                z.z = __shfl_sync(kFull, w.z, partner);
                z.w = __shfl_sync(kFull, w.w, partner);
                const uint32_t *zz = reinterpret_cast<const uint32_t *>(&z);
                if (rotated && turns) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[2 * j] = fmaf(y[2 * j], cs[2 * j],
                                        bf16_bits_to_f32(zz[j] & 0xFFFFu) * sn[2 * j]);
                        y[2 * j + 1] = fmaf(y[2 * j + 1], cs[2 * j + 1],
                                            bf16_bits_to_f32(zz[j] >> 16) * sn[2 * j + 1]);
                    }
                }
            }
            // an INT8 vector's largest magnitude (shuffles of all lanes, where any has one)
            float m = 0.0f;
            if (kInt8 && __any_sync(kFull, n >= a.Hq)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(y[j]));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
            }
            if (n >= end) continue;
            if (kInt8 && n >= a.Hq) {
                if (!has_slot) continue;
                const bool is_v = !rotated;
                const int h = n - a.Hq - (is_v ? a.Hkv : 0);
                const int64_t row = (static_cast<int64_t>(page_of) * a.Hkv + h) * a.page +
                                    (slot - page_of * a.page);
                const float s = __fdiv_rn(m, 127.0f);
                reinterpret_cast<uint2 *>(is_v ? a.vc : a.kc)[row * 16 + c] = quantize8_f32(y, s);
                if (c == 0) (is_v ? a.vs : a.ks)[row] = s;
                continue;
            }
            uint4 out = w;
            if (rotated && turns)
                out = make_uint4(bf16x2_bits(y[0], y[1]), bf16x2_bits(y[2], y[3]),
                                 bf16x2_bits(y[4], y[5]), bf16x2_bits(y[6], y[7]));
            if (n < a.Hq) {
                reinterpret_cast<uint4 *>(a.q_out + t * a.ot + n * a.oh)[c] = out;
            } else if (has_slot) {
                const bool is_v = !rotated;
                const int h = n - a.Hq - (is_v ? a.Hkv : 0);
                const int64_t row = (static_cast<int64_t>(page_of) * a.Hkv + h) * a.page +
                                    (slot - page_of * a.page);
                reinterpret_cast<uint4 *>(is_v ? a.vc : a.kc)[row * 16 + c] = out;
            }
        }
    }
}

template <bool kInt8, bool kPairs>
cudaError_t launch_as(const AppendArgs &a, int64_t T, int runs, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(T), static_cast<unsigned>(runs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_kv_append_kernel<kInt8, kPairs, 2>, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_kv_append(const PagedAppendProblem &p, int num_sms, cudaStream_t stream) {
    AppendArgs a;
    a.q = p.q;
    a.k = p.w.k;
    a.v = p.w.v;
    a.qt = p.qt;
    a.qh = p.qh;
    a.kt = p.w.kt;
    a.kh = p.w.kh;
    a.vt = p.w.vt;
    a.vh = p.w.vh;
    a.ot = p.ot;
    a.oh = p.oh;
    a.positions = p.positions;
    a.slots = p.w.slots;
    a.inv_freq = p.inv_freq;
    a.half = static_cast<int>(p.rot / 2);
    a.amplitude = p.amplitude;
    a.Hq = static_cast<int>(p.Hq);
    a.Hkv = static_cast<int>(p.w.Hkv);
    a.page = static_cast<int>(p.w.page);
    a.n_slots = static_cast<int>(p.w.P * p.w.page);
    a.q_out = p.q_out;
    a.kc = p.w.kc;
    a.vc = p.w.vc;
    a.ks = p.w.ks;
    a.vs = p.w.vs;
    // a token's heads are divided among CTAs, a pass each, while that leaves SMs idle
    const int vectors = a.Hq + 2 * a.Hkv;
    const int passes = (vectors + kPerPass - 1) / kPerPass;
    int runs = static_cast<int>(p.w.T >= 2 * num_sms ? 1 : (2 * num_sms + p.w.T - 1) / p.w.T);
    runs = runs < passes ? runs : passes;
    const int per = (passes + runs - 1) / runs;
    a.run = per * kPerPass;
    runs = (passes + per - 1) / per;
    if (p.w.int8)
        return p.interleaved ? launch_as<true, true>(a, p.w.T, runs, stream)
                             : launch_as<true, false>(a, p.w.T, runs, stream);
    return p.interleaved ? launch_as<false, true>(a, p.w.T, runs, stream)
                         : launch_as<false, false>(a, p.w.T, runs, stream);
}

}  // namespace w8a8
