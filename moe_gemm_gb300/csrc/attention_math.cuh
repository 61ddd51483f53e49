// Register-level parts of the decode attention kernels (mma.sync m16n8k16):
// the fragments of 32 positions of K and V per warp, the scores, the online
// softmax and the output product. Shared by the contiguous-cache and the paged
// forms, which differ in how the rows reach shared memory and in which
// (position, query) pairs are masked.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace w8a8 {

constexpr int kHeadDim = 128;

// ------------------------------------------------------- tensor-core helpers
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held one 32-bit pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&x));
}

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t x) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x));
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
    return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The magnitudes of a pair of BF16 values, as bits. For INT8 caches q goes to fp16 scaled
// by one power of two for neighbouring rows, from the largest of these. What is no finite
// number makes its own row none, and would turn all others into zeros if it set the
// scale: it counts as 0.
__device__ __forceinline__ uint32_t finite_bits2(uint32_t bf16_pair) {
    const uint32_t m = bf16_pair & 0x7FFF7FFFu;
    return m & ~__vcmpgeu2(m, 0x7F807F80u);
}

// One chunk's operands in registers: K rows pw + 16 mt + gid (+ 8), dims
// [32 t, 32 t + 32); V rows pw + 16 mt + 2 t + {0, 1, 8, 9}, dims [16 gid,
// 16 gid + 16); the K and V scales of the K rows (zero past the sequence).
template <bool kInt8>
struct ChunkRegs {
    static constexpr int kRowBytes = kInt8 ? kHeadDim : 2 * kHeadDim;
    static constexpr int KV = kRowBytes / 4 / 16;   // 16-byte vectors of a lane's 32 K dims
    static constexpr int VV = kRowBytes / 8 / 16;   // 16-byte vectors of a lane's 16 V dims
    uint4 k[2][2][KV];
    uint4 v[2][4][VV];
    float ks[2][2], vs[2][2];
};

// Running state of one warp over the chunks it has seen: per head its max
// score, the lane's share of sum exp(s - max), and the unnormalised output
// (in units of 2^-se: the fp16 range scaling of the INT8 cache).
template <int NT>
struct WarpState {
    float m[NT][2];
    float l[NT][2];
    float o[8][NT][4];
    int se, low;    // low: the smallest se so far (its start: 100)
};

// One chunk into the warp's running state (online softmax: the state is
// rescaled by exp(m_old - m_new) when a larger score arrives). valid(row, nt,
// j) tells whether query row 8 nt + 2 t + j sees the chunk's position `row`;
// the V scales of positions that no query sees are zero. values(r) is called once
// the scores are done and may fill in V's part of r (which then need not be held
// beside K's). kLog2: scale takes the scores to log2 units, and the exponentials
// are powers of two by the hardware's approximation (2 ulp) instead of expf.
template <int NT, bool kInt8, bool kLog2 = false, typename Valid, typename Values>
__device__ __forceinline__ void attend_chunk(WarpState<NT> &st, ChunkRegs<kInt8> &r,
                                             const uint32_t (&qf)[NT][16], Valid valid,
                                             Values values, float scale, float qinv, int pw, int gid,
                                             int t) {
    auto power = [](float v) {
        if constexpr (kLog2) return ex2_approx(v);
        else return expf(v);
    };
    // ---- scores: k-step kb covers dims 32 t + 4 kb + {0..3} of each lane
    float sacc[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) sacc[mt][nt][i] = 0.0f;
#pragma unroll
    for (int kb = 0; kb < 8; ++kb) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
            uint32_t a[4];
            if constexpr (kInt8) {
                // codes widened exactly to fp16; q is in fp16 too (scaled)
                i8x4_to_f16x4(word_of(r.k[mt][0][kb >> 2], kb & 3), a[0], a[2]);
                i8x4_to_f16x4(word_of(r.k[mt][1][kb >> 2], kb & 3), a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16(sacc[mt][nt], a, qf[nt][2 * kb], qf[nt][2 * kb + 1]);
            } else {
                a[0] = word_of(r.k[mt][0][kb >> 1], (2 * kb) & 3);
                a[2] = word_of(r.k[mt][0][kb >> 1], (2 * kb + 1) & 3);
                a[1] = word_of(r.k[mt][1][kb >> 1], (2 * kb) & 3);
                a[3] = word_of(r.k[mt][1][kb >> 1], (2 * kb + 1) & 3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_bf16(sacc[mt][nt], a, qf[nt][2 * kb], qf[nt][2 * kb + 1]);
            }
        }
    }
    // scaled scores (fragment i: row gid + 8 (i >> 1), head 8 nt + 2 t + (i & 1))
    // and the chunk's max per head over the warp
    float mc[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mc[nt][0] = mc[nt][1] = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int hf = i >> 1;
                const int row = pw + 16 * mt + gid + 8 * hf;
                // (the fp16 q carries the power of two 1/qinv: scaling back is exact)
                const float sv =
                    valid(row, nt, i & 1)
                        ? (sacc[mt][nt][i] * (r.ks[mt][hf] * scale)) * qinv
                        : -INFINITY;
                sacc[mt][nt][i] = sv;
                mc[nt][i & 1] = fmaxf(mc[nt][i & 1], sv);
            }
    float mu[NT][2], alpha[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float m = mc[nt][j];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float m_new = fmaxf(st.m[nt][j], m);
            mu[nt][j] = m_new == -INFINITY ? 0.0f : m_new;   // no valid score yet
            alpha[nt][j] = power(st.m[nt][j] - mu[nt][j]);    // 0 while the state is empty
            st.m[nt][j] = m_new;
            st.l[nt][j] *= alpha[nt][j];
        }
    values(r);
    // the warp's largest V scale of the chunk sets the power of two that keeps
    // P' in fp16's normal range (INT8 cache); rows of other lanes t are the same
    int se = st.se;
    if constexpr (kInt8) {
        float vmax = fmaxf(fmaxf(r.vs[0][0], r.vs[0][1]), fmaxf(r.vs[1][0], r.vs[1][1]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xFFFFFFFFu, vmax, o));
        const int bexp = static_cast<int>((__float_as_uint(vmax) >> 23) & 0xFFu);
        // (at most 2^60 finer than the coarsest unit so far: the FP32 sums in it stay finite)
        if (bexp != 0) se = max(-100, min(min(100, st.low + 60), 14 - (bexp - 127)));
        st.low = min(st.low, se);
    }
    // rescale the state's output: exp(m_old - m_new) and the change of units (at most
    // 2^100 finer, from the start's; coarser by more than binary32 has: nothing is left)
    const float ratio =
        se - st.se < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(se - st.se + 127) << 23);
    st.se = se;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) st.o[i][nt][k] *= alpha[nt][k & 1] * ratio;
    const float pscale = __uint_as_float(static_cast<uint32_t>(se + 127) << 23);
    // probabilities, their sums, and the B fragments of the output product
    constexpr int NS = kInt8 ? 2 : 3;   // hi, lo (fp16) or hi, mid, lo (bf16)
    uint32_t bp[2][NT][NS][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float pp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float pr = power(sacc[mt][nt][i] - mu[nt][i & 1]);
                st.l[nt][i & 1] += pr;
                pp[i] = (pr * r.vs[mt][i >> 1]) * pscale;
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float x0 = pp[2 * hf], x1 = pp[2 * hf + 1];
                if constexpr (kInt8) {
                    const uint32_t hi = pack_f16x2(x0, x1);
                    const float2 hv = unpack_f16x2(hi);
                    const uint32_t lo = pack_f16x2(x0 - hv.x, x1 - hv.y);
                    bp[mt][nt][0][hf] = movmatrix_trans(hi);
                    bp[mt][nt][1][hf] = movmatrix_trans(lo);
                } else {
                    const uint32_t hi = pack_bf16x2(x0, x1);
                    const float2 hv = unpack_bf16x2(hi);
                    const float r0 = x0 - hv.x, r1 = x1 - hv.y;
                    const uint32_t mid = pack_bf16x2(r0, r1);
                    const float2 mv = unpack_bf16x2(mid);
                    const uint32_t lo = pack_bf16x2(r0 - mv.x, r1 - mv.y);
                    bp[mt][nt][0][hf] = movmatrix_trans(hi);
                    bp[mt][nt][1][hf] = movmatrix_trans(mid);
                    bp[mt][nt][2][hf] = movmatrix_trans(lo);
                }
            }
        }
    // ---- unnormalised output: m-tile i holds dims 16 gid + 2 i (row gid) and
    // 16 gid + 2 i + 1 (row gid + 8)
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t a[4];
            if constexpr (kInt8) {
                // bytes 2i, 2i + 1 of the four positions' 16-byte vectors, as
                // fp16 pairs over positions (1024 + biased byte, minus 1152)
                const int w = i >> 1;
                const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                const uint32_t g01 = prmt(word_of(r.v[mt][0][0], w) ^ 0x80808080u,
                                          word_of(r.v[mt][1][0], w) ^ 0x80808080u, sel);
                const uint32_t g23 = prmt(word_of(r.v[mt][2][0], w) ^ 0x80808080u,
                                          word_of(r.v[mt][3][0], w) ^ 0x80808080u, sel);
                const uint32_t x[4] = {prmt(g01, 0x64646464u, 0x4140u),
                                       prmt(g01, 0x64646464u, 0x4342u),
                                       prmt(g23, 0x64646464u, 0x4140u),
                                       prmt(g23, 0x64646464u, 0x4342u)};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a[k]) : "r"(x[k]), "r"(0x64806480u));
            } else {
                const uint32_t w0 = word_of(r.v[mt][0][i >> 2], i & 3);
                const uint32_t w1 = word_of(r.v[mt][1][i >> 2], i & 3);
                const uint32_t w2 = word_of(r.v[mt][2][i >> 2], i & 3);
                const uint32_t w3 = word_of(r.v[mt][3][i >> 2], i & 3);
                a[0] = prmt(w0, w1, 0x5410u);
                a[1] = prmt(w0, w1, 0x7632u);
                a[2] = prmt(w2, w3, 0x5410u);
                a[3] = prmt(w2, w3, 0x7632u);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int sp = 0; sp < NS; ++sp) {
                    if constexpr (kInt8)
                        mma_f16(st.o[i][nt], a, bp[mt][nt][sp][0], bp[mt][nt][sp][1]);
                    else
                        mma_bf16(st.o[i][nt], a, bp[mt][nt][sp][0], bp[mt][nt][sp][1]);
                }
        }
    }
}

}  // namespace w8a8
