// Product of FP8 (e4m3) activations and weights with a scale for each block of 128, on the
// tcgen05 tensor cores of sm_103a ("Running DeepSeek-V4-Flash-Vision on 4xA800", §一:
// FP8 weights in [128, 128] blocks):
//
//   y[m, n] = sum_g (sa[m, g] sw[n / 128, g]) P_g[m, n],  P_g = sum over k in group g of
//   qa[m, k] qw[n, k]
//
// The scales change every 128 K, so a group's products are summed by themselves in tensor
// memory (kind::f8f6f4, FP32), and the groups are added up in registers, acc = fma(P_g,
// sa sw, acc), in K order. A token is a lane of tensor memory, so a thread has one token and
// its scale is one number per group and block.
//
// A tile is 128 tokens (the M of an instruction) by a slice of w <= 256 weight rows, over
// all of K. A step is a group: 128 bytes of every row, one 128-byte swizzle atom
// wide, four instructions of 32 K. The slices are as wide as makes the waves of
// tiles fullest: a decode step's weights then divide evenly among the SMs with no split of K.
//
// Warps: 0 loads (TMA), 1 issues the products, 4-7 and 8-11 add up a half of the slice
// each (128 lanes), 2 and 3 only give up their registers.
//
// What bounds it. Up to 32 tokens (gemm_fp8_rows_kernel): HBM (8 tokens x 28672 x 8192, 235 MB:
// 38.0 us, 6.2 TB/s). Some tens to hundreds: the steps, which take some 400 cycles to hand a
// stage and a buffer on, whatever they hold, so those of narrow slices hold 2 or 4 groups (64 x
// 8192 x 4096: 12.4 us). Many tokens (gemm_fp8_pair_kernel):
// tensor memory, which the products' sums and the reads of a group's sums share: 4096
// x 8192 x 8192 take 209 us, 2.63 PFLOP/s; a form that reads an eighth of the sums takes 170,
// one that reads half of them 183, and adding costs nothing beside reading. Tried
// and slower: 16 warps that add up (254 us), reads of 32 columns with two in flight (spills,
// 449), scales through cp.async (221).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "quant_math.cuh"
#include "tensor_map.h"

namespace w8a8 {
namespace {

constexpr int kThreads = 384;
constexpr int kTokens = 128;
constexpr int kMaxSlice = 256;
constexpr int kMaxStages = 16, kMaxBufs = 8, kMaxPerStep = 4;
constexpr int kSmemBytes = 227 * 1024;
constexpr int kOffStages = 1024;           // barriers and flags before them
constexpr int kStagedBytes = 8 * 32 * 17 * 4;   // outputs on their way, at the end
constexpr int kTmemCols = 512;
// 384 threads are launched with 168 registers; the 256 that add up get 232, the others 40
// (216 and 72: 221 -> 216 us at 4096 x 8192 x 8192).
constexpr uint32_t kSumRegs = 232, kOtherRegs = 40;
static_assert(256 * kSumRegs + 128 * kOtherRegs == kThreads * 168);

struct Fp8Args {
    const float *sa, *sw;
    void *y;
    int M, N, G;
    int w, half;               // rows of a slice, and of the first half of it
    int a_bytes, b_bytes;      // of a stage
    int a_box, b_box;          // bytes that a copy brings
    int stages, bufs, buf_cols;
    int per_step;              // groups of a step: of a stage, of a buffer
    int m_tiles, tiles;
    int n_mma;                 // the slice in an instruction's N
    int out_fp32, wide_store;  // rows of y allow 32-byte stores
    int words;                 // ... or 4-byte stores
    int early;                 // the kernel before is the quantizer of the same call
    unsigned long long *err;
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages], d_full[kMaxBufs], d_empty[kMaxBufs], drain;
    uint32_t tmem;
    volatile int abort_flag;
};
static_assert(sizeof(Bars) <= kOffStages);

struct Ring {
    uint32_t idx = 0, phase = 0;
    __device__ __forceinline__ void advance(uint32_t n) {
        if (++idx == n) {
            idx = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// Instruction descriptor, kind::f8f6f4: e4m3 operands (format 0), FP32 sums, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// Upper word of a K-major operand's descriptor with the 128-byte swizzle, 8-row groups
// 1024 bytes apart; the lower word is the address in units of 16 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }

template <bool kAccumulate>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "n"(kAccumulate ? 1 : 0), "n"(kDescHi)
        : "memory");
}

// 32 columns of the warp's 32 lanes; the registers are valid after tmem_wait32 on them.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// A load that stays where it is written (an ordinary one: the kernel before may have
// written the scales while this one had started).
__device__ __forceinline__ float ld_now(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ unsigned long long f2_fma(unsigned long long a, unsigned long long b,
                                                     unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One thread's outputs: kCols consecutive columns of a row, `cols` of them in the matrix (a
// multiple of what a store of 32 bytes holds).
template <int kCols>
__device__ __forceinline__ void store_row(const Fp8Args &a, int64_t at, int cols,
                                          const unsigned long long (&acc)[kCols / 2]) {
#pragma unroll
    for (int i = 0; i < kCols / 16; ++i) {
        if (16 * i >= cols) break;
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) f2_split(acc[8 * i + j], v[2 * j], v[2 * j + 1]);
        uint32_t u[8];
        if (a.out_fp32) {
            float *y = static_cast<float *>(a.y) + at + 16 * i;
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[j]);
            store32(y, u);
            if (16 * i + 8 < cols) {
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[8 + j]);
                store32(y + 8, u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
            store32(static_cast<__nv_bfloat16 *>(a.y) + at + 16 * i, u);
        }
    }
}

// The same for a warp's 32 rows where rows of y do not allow that: through shared memory, so that
// a store covers 64 bytes of a row instead of one value in each of 32.
template <int kCols>
__device__ __forceinline__ void store_staged(const Fp8Args &a, uint32_t *buf, int m0, int c0,
                                             int cols,
                                             const unsigned long long (&acc)[kCols / 2]) {
    const int lane = threadIdx.x & 31;
    const int per = a.out_fp32 ? 16 : 32;         // columns of 64 bytes
    const int rows = min(32, a.M - m0);
#pragma unroll
    for (int i = 0; i < kCols / 16; ++i) {
        if (!a.out_fp32 && (i & 1)) continue;
        if (16 * i >= cols) break;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float x, y;
            f2_split(acc[8 * i + j], x, y);
            if (a.out_fp32) {
                buf[lane * 17 + 2 * j] = __float_as_uint(x);
                buf[lane * 17 + 2 * j + 1] = __float_as_uint(y);
            } else {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
                buf[lane * 17 + j] = *reinterpret_cast<const uint32_t *>(&b);
                if (i + 1 < kCols / 16) {
                    f2_split(acc[8 * (i + 1 < kCols / 16 ? i + 1 : i) + j], x, y);
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(x, y);
                    buf[lane * 17 + 8 + j] = *reinterpret_cast<const uint32_t *>(&b2);
                }
            }
        }
        __syncwarp();
        const int left = cols - 16 * i;           // columns from here on
        if (a.words) {
            const int w = lane & 15;
            const bool mine = (a.out_fp32 ? w : 2 * w) < min(left, per);
            for (int r = lane >> 4; r < rows; r += 2) {
                const int64_t at = static_cast<int64_t>(m0 + r) * a.N + c0 + 16 * i;
                uint32_t *row = a.out_fp32 ? static_cast<uint32_t *>(a.y) + at
                                           : reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.y) + at);
                if (mine) row[w] = buf[r * 17 + w];
            }
        } else {                                  // BF16, rows at odd places
            for (int r = 0; r < rows; ++r) {
                const int64_t at = static_cast<int64_t>(m0 + r) * a.N + c0 + 16 * i;
                if (lane < min(left, per))
                    static_cast<uint16_t *>(a.y)[at + lane] =
                        reinterpret_cast<const uint16_t *>(buf + r * 17)[lane];
            }
        }
    }
}

// kCols: columns of a half of the slice, rounded up to 32 (what is read past the half is not
// stored, and lies within tensor memory: launch_gemm_fp8). Slices of more than 128 rows have one
// group per step.
template <int kCols>
__global__ void __launch_bounds__(kThreads, 1)
gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmap_a,
                const __grid_constant__ CUtensorMap tmap_b, const Fp8Args a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    Bars &s = *reinterpret_cast<Bars *>(smem_raw + (base - raw));
    const uint32_t sA = base + kOffStages;
    const uint32_t sB = sA + a.stages * a.per_step * a.a_bytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        for (int i = 0; i < a.bufs; ++i) {
            mbar_init(smem_u32(&s.d_full[i]), 1);
            mbar_init(smem_u32(&s.d_empty[i]), 8);
        }
        mbar_init(smem_u32(&s.drain), 1);
        s.abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmap_a);
        tma_prefetch_desc(&tmap_b);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s.tmem), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *abort_flag = &s.abort_flag;
    if (!a.early) griddep_wait();    // (Fp8Problem::chained)
    griddep_launch_dependents();

    if (warp < 4) {
        setmaxnreg_dec<kOtherRegs>();
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------- TMA producer
            Ring r;
            uint32_t issued = 0;
            bool ok = true;
            // The first weights are asked for while the call's quantizer, which writes the tokens'
            // codes and scales, still runs.
            const int steps = (a.G + a.per_step - 1) / a.per_step;
            const int ahead = a.stages < steps ? a.stages : steps;
            auto load = [&](const void *map, uint32_t to, int bytes, int step, int row,
                            uint32_t bar) {
                const int groups = min(a.per_step, a.G - step * a.per_step);
                for (int i = 0; i < groups; ++i)
                    tma_load_2d(to + i * bytes, map, (step * a.per_step + i) * 128, row, bar);
            };
            auto expect = [&](int step, uint32_t bar) {
                mbar_arrive_expect_tx(bar, min(a.per_step, a.G - step * a.per_step) *
                                               (a.a_box + a.b_box));
            };
            {
                const int n = blockIdx.x / a.m_tiles;
                for (int i = 0; i < ahead; ++i) {
                    const uint32_t bar = smem_u32(&s.full[i]);
                    expect(i, bar);
                    load(&tmap_b, sB + i * a.per_step * a.b_bytes, a.b_bytes, i, n * a.w, bar);
                }
                griddep_wait();
                const int m0 = (blockIdx.x - n * a.m_tiles) * kTokens;
                for (int i = 0; i < ahead; ++i)
                    load(&tmap_a, sA + i * a.per_step * a.a_bytes, a.a_bytes, i, m0,
                         smem_u32(&s.full[i]));
                issued = ahead;
                r.idx = ahead == a.stages ? 0 : ahead;
                r.phase = ahead == a.stages ? 1 : 0;
            }
            for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
                const int n = t / a.m_tiles;
                const int m0 = (t - n * a.m_tiles) * kTokens, n0 = n * a.w;
                for (int i = t == blockIdx.x ? ahead : 0; i < steps; ++i) {
                    if (!mbar_wait(smem_u32(&s.empty[r.idx]), r.phase ^ 1u, abort_flag, a.err,
                                   ROLE_PRODUCER, 0, kWaitLimitNs, KID_FP8)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_u32(&s.full[r.idx]);
                    expect(i, bar);
                    load(&tmap_b, sB + r.idx * a.per_step * a.b_bytes, a.b_bytes, i, n0, bar);
                    load(&tmap_a, sA + r.idx * a.per_step * a.a_bytes, a.a_bytes, i, m0, bar);
                    r.advance(a.stages);
                    ++issued;
                }
            }
            if (!ok) {       // the copies in flight land before the CTA goes
                const uint32_t n = a.stages;
                for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i) {
                    const unsigned long long t0 = globaltimer_ns();
                    while (!mbar_try_wait(smem_u32(&s.full[i % n]), (i / n) & 1u) &&
                           globaltimer_ns() - t0 < kWaitLimitNs) {
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------- products
            Ring r, d;
            bool ok = true;
            const uint32_t idesc = idesc_e4m3(kTokens, a.n_mma);
            for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
                for (int g = 0; g < a.G; g += a.per_step) {
                    ok = mbar_wait(smem_u32(&s.d_empty[d.idx]), d.phase ^ 1u, abort_flag, a.err,
                                   ROLE_MMA, 0, kWaitLimitNs, KID_FP8) &&
                         mbar_wait(smem_u32(&s.full[r.idx]), r.phase, abort_flag, a.err, ROLE_MMA,
                                   1, kWaitLimitNs, KID_FP8);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const int groups = min(a.per_step, a.G - g);
                    const uint32_t da = desc_lo(sA + r.idx * a.per_step * a.a_bytes);
                    const uint32_t db = desc_lo(sB + r.idx * a.per_step * a.b_bytes);
                    const uint32_t dt = tmem + d.idx * a.per_step * a.buf_cols;
                    const uint32_t ka = a.a_bytes >> 4, kb = a.b_bytes >> 4, kd = a.buf_cols;
                    if (elect_one()) {
                        // (the groups' instructions take turns: one that adds to what the one
                        // before it wrote waits for it)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
#pragma unroll
                            for (int i = 0; i < kMaxPerStep; ++i) {
                                if (i >= groups) break;
                                if (k == 0) mma_e4m3<false>(dt + i * kd, da + i * ka, db + i * kb, idesc);
                                else mma_e4m3<true>(dt + i * kd, da + i * ka + 2 * k, db + i * kb + 2 * k, idesc);
                            }
                        }
                        mma_commit(smem_u32(&s.empty[r.idx]));
                        mma_commit(smem_u32(&s.d_full[d.idx]));
                    }
                    __syncwarp();
                    r.advance(a.stages);
                    d.advance(a.bufs);
                }
            }
            if (elect_one()) mma_commit(smem_u32(&s.drain));
            __syncwarp();
            const unsigned long long t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&s.drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else {
        // ----------------------------------------------------------- sums of groups
        setmaxnreg_inc<kSumRegs>();
        griddep_wait();
        const int h = (warp >> 2) - 1, q = warp & 3;
        const uint32_t my_tmem = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * a.half;
        uint32_t *stage_buf = reinterpret_cast<uint32_t *>(smem_raw + kSmemBytes - kStagedBytes) +
                              (warp - 4) * 32 * 17;
        Ring d;
        bool ok = true;
        for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
            const int n = t / a.m_tiles;
            const int m0 = (t - n * a.m_tiles) * kTokens;
            const int c0 = n * a.w + h * a.half;
            const int cols = min(h == 0 ? a.half : a.w - a.half, a.N - c0);
            const bool on = m0 + q * 32 < a.M && cols > 0;   // the same for the warp
            const int m = m0 + q * 32 + lane;
            // columns before `edge` have the scale of block c0 / 128, the others of the next
            const int edge = 128 - (c0 & 127);
            const float *sa = a.sa + static_cast<int64_t>(min(m, a.M - 1)) * a.G;
            const float *sw0 = a.sw + static_cast<int64_t>(on ? c0 >> 7 : 0) * a.G;
            const float *sw1 = on && cols > edge ? sw0 + a.G : sw0;
            unsigned long long acc[kCols / 2];
#pragma unroll
            for (int j = 0; j < kCols / 2; ++j) acc[j] = 0ull;
            uint32_t at = 0;
            if (!on) {                               // (only hands the buffers on)
                for (int g = 0; g < a.G; g += a.per_step) {
                    ok = mbar_wait(smem_u32(&s.d_full[d.idx]), d.phase, abort_flag, a.err,
                                   ROLE_EPILOGUE, 1, kWaitLimitNs, KID_FP8);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_relaxed(smem_u32(&s.d_empty[d.idx]));
                    d.advance(a.bufs);
                }
                continue;
            }
            float fa = ld_now(sa), f0 = ld_now(sw0), f1 = ld_now(sw1);
            int left = 0;                            // groups of the step
            for (int g = 0; g < a.G; ++g) {
                const float s0 = fa * f0, s1 = fa * f1;
                if (g + 1 < a.G) {
                    fa = ld_now(sa + g + 1);
                    f0 = ld_now(sw0 + g + 1);
                    f1 = ld_now(sw1 + g + 1);
                }
                if (kCols > 64 || left == 0) {
                    ok = mbar_wait(smem_u32(&s.d_full[d.idx]), d.phase, abort_flag, a.err,
                                   ROLE_EPILOGUE, 0, kWaitLimitNs, KID_FP8);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    if (kCols <= 64) left = min(a.per_step, a.G - g);
                    at = my_tmem + d.idx * a.per_step * a.buf_cols;
                }
                uint32_t v[2][32];
                tmem_ld32(at, v[0]);
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    tmem_wait32(v[c & 1]);
                    if (c + 1 < kCols / 32)
                        tmem_ld32(at + 32 * c + 32, v[(c + 1) & 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float f = 32 * c + 8 * i < edge ? s0 : s1;
                        const unsigned long long f2 = f2_bits(f, f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            unsigned long long &o = acc[16 * c + 4 * i + j];
                            o = f2_fma(f2_bits(__uint_as_float(v[c & 1][8 * i + 2 * j]),
                                               __uint_as_float(v[c & 1][8 * i + 2 * j + 1])),
                                       f2, o);
                        }
                    }
                }
                at += a.buf_cols;
                if (kCols > 64 || --left == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed(smem_u32(&s.d_empty[d.idx]));
                    d.advance(a.bufs);
                }
            }
            if (ok) {
                if (a.wide_store) {
                    if (m < a.M) store_row<kCols>(a, static_cast<int64_t>(m) * a.N + c0, cols, acc);
                } else {
                    store_staged<kCols>(a, stage_buf, m - lane, c0, cols, acc);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ pairs of CTAs
// The same product for many tokens, where shared memory's bandwidth bounds the form
// above: a group's instructions read 48 KB of operands in the 512 cycles that they take, and as
// much is written. Two CTAs on neighbouring SMs take a tile of 256 tokens x 256 weight
// rows together (cta_group::2): each holds its 128 tokens and half of the weights, so a
// group reads and writes 32 KB per SM, and each adds up its own tokens. One thread of the
// first CTA issues for both; its barriers collect the copies of both and the releases
// of both CTAs' tensor memory (4096 x 8192 x 8192: 319 us with single CTAs, 209 with pairs).
constexpr int kPairTokens = 256, kPairRows = 256;
constexpr int kPairStageBytes = 2 * 128 * 128;
constexpr int kPairStages = (kSmemBytes - 1024 - kOffStages - kStagedBytes) / kPairStageBytes;
constexpr int kPairBand = 8;              // token tiles that share weights in L2

constexpr int kPairCols = kPairRows / 2;  // columns of a warp

struct PairTile {
    int m0, n0;
};
// Tiles in bands of kPairBand token tiles, the weights' tiles one after the other.
__device__ __forceinline__ PairTile pair_tile(int t, int m_tiles, int n_tiles) {
    const int band = t / (kPairBand * n_tiles);
    const int in = t - band * kPairBand * n_tiles;
    const int rows = min(kPairBand, m_tiles - band * kPairBand);
    const int n = in / rows;
    return {(band * kPairBand + in - n * rows) * kPairTokens, n * kPairRows};
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the same shared memory in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first(uint32_t saddr) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(saddr));
    return r;
}
// (Relaxed, and waited for with the CTA's scope: what the barrier guards is tensor memory, whose
// reads have completed before. A release or an acquire over the cluster would wait for
// the thread's outstanding loads and drop what L1 holds, twice per group: 546 us instead of 226
// at 4096 x 8192 x 8192.)
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A load into this CTA whose bytes count at a barrier of the pair's first.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void *tmap, int x, int y,
                                              uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <bool kAccumulate>
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "n"(kAccumulate ? 1 : 0), "n"(kDescHi)
        : "memory");
}
// An arrival at the barrier of both CTAs when what was issued is done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_b, const Fp8Args a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    Bars &s = *reinterpret_cast<Bars *>(smem_raw + (base - raw));
    const uint32_t sA = base + kOffStages;
    const uint32_t sB = sA + kPairStages * 128 * 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s.d_full[i]), 1);
            mbar_init(smem_u32(&s.d_empty[i]), 16);
        }
        mbar_init(smem_u32(&s.drain), 1);
        s.abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmap_a);
        tma_prefetch_desc(&tmap_b);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)),
                     "r"(static_cast<uint32_t>(kTmemCols))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *abort_flag = &s.abort_flag;
    const int pairs = gridDim.x >> 1, first = blockIdx.x >> 1;
    const int n_tiles = (a.N + kPairRows - 1) / kPairRows;
    griddep_launch_dependents();
    griddep_wait();

    if (warp < 4) {
        setmaxnreg_dec<kOtherRegs>();
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------- TMA producer
            Ring r;
            uint32_t issued = 0;
            bool ok = true;
            for (int t = first; t < a.tiles && ok; t += pairs) {
                const PairTile p = pair_tile(t, a.m_tiles, n_tiles);
                for (int g = 0; g < a.G; ++g) {
                    if (!mbar_wait(smem_u32(&s.empty[r.idx]), r.phase ^ 1u, abort_flag, a.err,
                                   ROLE_PRODUCER, 10, kWaitLimitNs, KID_FP8)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = in_first(smem_u32(&s.full[r.idx]));
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&s.full[r.idx]), 2 * kPairStageBytes);
                    tma_load_pair(sB + r.idx * 128 * 128, &tmap_b, g * 128, p.n0 + 128 * rank, bar);
                    tma_load_pair(sA + r.idx * 128 * 128, &tmap_a, g * 128, p.m0 + 128 * rank, bar);
                    r.advance(kPairStages);
                    ++issued;
                }
            }
            if (!ok) {       // the copies in flight land before the CTA goes
                if (rank == 0) {
                    const uint32_t n = kPairStages;
                    for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i) {
                        const unsigned long long t0 = globaltimer_ns();
                        while (!mbar_try_wait(smem_u32(&s.full[i % n]), (i / n) & 1u) &&
                               globaltimer_ns() - t0 < kWaitLimitNs) {
                        }
                    }
                } else {     // (counted at the other CTA: a time that no copy takes)
                    const unsigned long long t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < 10000000ull) {
                    }
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ------------------------------------------------------- products
            Ring r, d;
            bool ok = true;
            const uint32_t idesc = idesc_e4m3(kPairTokens, kPairRows);
            for (int t = first; t < a.tiles && ok; t += pairs) {
                for (int g = 0; g < a.G; ++g) {
                    ok = mbar_wait(smem_u32(&s.d_empty[d.idx]), d.phase ^ 1u, abort_flag, a.err,
                                   ROLE_MMA, 10, kWaitLimitNs, KID_FP8) &&
                         mbar_wait(smem_u32(&s.full[r.idx]), r.phase, abort_flag, a.err, ROLE_MMA,
                                   11, kWaitLimitNs, KID_FP8);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t da = desc_lo(sA + r.idx * 128 * 128);
                    const uint32_t db = desc_lo(sB + r.idx * 128 * 128);
                    const uint32_t dt = tmem + d.idx * 256;
                    if (elect_one()) {
                        mma_pair<false>(dt, da, db, idesc);
                        mma_pair<true>(dt, da + 2, db + 2, idesc);
                        mma_pair<true>(dt, da + 4, db + 4, idesc);
                        mma_pair<true>(dt, da + 6, db + 6, idesc);
                        commit_pair(smem_u32(&s.empty[r.idx]));
                        commit_pair(smem_u32(&s.d_full[d.idx]));
                    }
                    __syncwarp();
                    r.advance(kPairStages);
                    d.advance(2);
                }
            }
            if (elect_one()) commit_pair(smem_u32(&s.drain));
            __syncwarp();
        }
        if (warp == 1) {     // both CTAs: no product and no arrival is left on its way
            const unsigned long long t0 = globaltimer_ns();
            while (!mbar_try_wait(smem_u32(&s.drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
            }
        }
    } else {
        // ----------------------------------------------------------- sums of groups
        setmaxnreg_inc<kSumRegs>();
        const int h = (warp >> 2) - 1, q = warp & 3;
        const uint32_t my_tmem = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * kPairCols;
        uint32_t *stage_buf = reinterpret_cast<uint32_t *>(smem_raw + kSmemBytes - kStagedBytes) +
                              (warp - 4) * 32 * 17;
        Ring d;
        bool ok = true;
        for (int t = first; t < a.tiles && ok; t += pairs) {
            const PairTile p = pair_tile(t, a.m_tiles, n_tiles);
            const int c0 = p.n0 + h * kPairCols;
            const int cols = min(kPairCols, a.N - c0);
            const int m0 = p.m0 + 128 * static_cast<int>(rank) + q * 32;
            const bool on = m0 < a.M && cols > 0;            // the same for the warp
            const int m = m0 + lane;
            const float *sa = a.sa + static_cast<int64_t>(min(m, a.M - 1)) * a.G;
            const float *sw = a.sw + static_cast<int64_t>(on ? c0 >> 7 : 0) * a.G;
            unsigned long long acc[kPairCols / 2];
#pragma unroll
            for (int j = 0; j < kPairCols / 2; ++j) acc[j] = 0ull;
            float fa = ld_now(sa), fw = ld_now(sw);
            for (int g = 0; g < a.G; ++g) {
                const float f = fa * fw;
                if (g + 1 < a.G) {
                    fa = ld_now(sa + g + 1);
                    fw = ld_now(sw + g + 1);
                }
                ok = mbar_wait(smem_u32(&s.d_full[d.idx]), d.phase, abort_flag, a.err,
                               ROLE_EPILOGUE, 10, kWaitLimitNs, KID_FP8);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = my_tmem + d.idx * 256;
                const unsigned long long f2 = f2_bits(f, f);
                uint32_t v[2][16];
                tmem_ld_16cols(at, v[0]);
#pragma unroll
                for (int c = 0; c < kPairCols / 16; ++c) {
                    tmem_wait_ld_dep16(v[c & 1]);
                    if (c < kPairCols / 16 - 1) {
                        tmem_ld_16cols(at + 16 * c + 16, v[(c + 1) & 1]);
                    } else {                                 // all is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_remote(in_first(smem_u32(&s.d_empty[d.idx])));
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[8 * c + j] = f2_fma(f2_bits(__uint_as_float(v[c & 1][2 * j]),
                                                        __uint_as_float(v[c & 1][2 * j + 1])),
                                                f2, acc[8 * c + j]);
                }
                d.advance(2);
            }
            if (ok && on) {
                if (a.wide_store) {
                    if (m < a.M) store_row<kPairCols>(a, static_cast<int64_t>(m) * a.N + c0, cols, acc);
                } else {
                    store_staged<kPairCols>(a, stage_buf, m0, c0, cols, acc);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();      // (nobody leaves while the other may still reach its memory)
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(static_cast<uint32_t>(kTmemCols))
                     : "memory");
    }
}

// ------------------------------------------------------------------ few tokens
// The same product for up to 32 tokens, with the operands the other way round: 128 weight rows, a
// block of scales, are the lanes, kTok tokens the columns. An instruction reads what it needs
// and no more, a group's sums are kTok columns, and a store of y is 32 neighbours of a row. Against
// slices: 1 x 10240 x 8192 25.7 -> 16.8 us, 16 x 1024 x 1024 5.1 -> 3.8, 1 x 4096 x 4096 9.6 ->
// 7.2, 32 x 16384 x 4096 16.5 -> 15.0, 8 x 28672 x 8192 41.7 -> 38.0; level at 32 x 8192 x
// 4096. What bounds it: HBM from some 100 tiles on (80 take 5.0 TB/s, 112 6.2); with fewer, what an
// SM takes in, 64 KB of weights a step in 0.55 us (one tile's 2, 8 and 16 steps: 3.8, 7.2 and
// 11.6 us).
constexpr int kRowsMaxTokens = 32;
constexpr int kRowsThreads = 256;
constexpr int kRowsTmemCols = 256;

// Groups of a step: 4 with 16 tokens (1 x 4096 x 4096: 7.2 us, with 2 8.9), 2 with 32, whose stages are
// larger (32 x 16384 x 4096: 15.0, with 4 16.2; 32 x 8192 x 4096: 11.0 and 10.5).
template <int kTok>
struct RowsShape {
    static constexpr int kPerStep = kTok == 16 ? 4 : 2;
    static constexpr int kBufs = kRowsTmemCols / (kPerStep * kTok);
    static constexpr int kW = 128 * 128, kT = kTok * 128;
    static constexpr int kStage = kPerStep * (kW + kT);
    static constexpr int kStages = (kSmemBytes - 1024 - kOffStages) / kStage;
    static_assert(kStages >= 2 && kStages <= kMaxStages && kBufs >= 2 && kBufs <= kMaxBufs);
};

template <int kTok>
__global__ void __launch_bounds__(kRowsThreads, 1)
gemm_fp8_rows_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_b, const Fp8Args a) {
    using Shape = RowsShape<kTok>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    Bars &s = *reinterpret_cast<Bars *>(smem_raw + (base - raw));
    const uint32_t sW = base + kOffStages;
    const uint32_t sT = sW + Shape::kStages * Shape::kPerStep * Shape::kW;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Shape::kStages; ++i) {
            mbar_init(smem_u32(&s.full[i]), 1);
            mbar_init(smem_u32(&s.empty[i]), 1);
        }
        for (int i = 0; i < Shape::kBufs; ++i) {
            mbar_init(smem_u32(&s.d_full[i]), 1);
            mbar_init(smem_u32(&s.d_empty[i]), 4);
        }
        mbar_init(smem_u32(&s.drain), 1);
        s.abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmap_a);
        tma_prefetch_desc(&tmap_b);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s.tmem), kRowsTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem;
    volatile int *abort_flag = &s.abort_flag;
    const int steps = (a.G + Shape::kPerStep - 1) / Shape::kPerStep;
    if (!a.early) griddep_wait();    // (Fp8Problem::chained)
    griddep_launch_dependents();

    if (warp == 0 && lane == 0) {
        // ----------------------------------------------------------- TMA producer
        Ring r;
        uint32_t issued = 0;
        bool ok = true;
        auto groups_of = [&](int step) { return min(Shape::kPerStep, a.G - step * Shape::kPerStep); };
        auto load_weights = [&](int stage, int step, int n0) {
            const uint32_t bar = smem_u32(&s.full[stage]);
            mbar_arrive_expect_tx(bar, groups_of(step) * (Shape::kW + Shape::kT));
            for (int i = 0; i < groups_of(step); ++i)
                tma_load_2d(sW + (stage * Shape::kPerStep + i) * Shape::kW, &tmap_b,
                            (step * Shape::kPerStep + i) * 128, n0, bar);
        };
        auto load_tokens = [&](int stage, int step) {
            for (int i = 0; i < groups_of(step); ++i)
                tma_load_2d(sT + (stage * Shape::kPerStep + i) * Shape::kT, &tmap_a,
                            (step * Shape::kPerStep + i) * 128, 0, smem_u32(&s.full[stage]));
        };
        // (the first weights before the call's quantizer has written the tokens' codes)
        const int ahead = min(Shape::kStages, steps);
        for (int i = 0; i < ahead; ++i) load_weights(i, i, blockIdx.x * 128);
        griddep_wait();
        for (int i = 0; i < ahead; ++i) load_tokens(i, i);
        issued = ahead;
        r.idx = ahead == Shape::kStages ? 0 : ahead;
        r.phase = ahead == Shape::kStages ? 1 : 0;
        for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
            for (int i = t == blockIdx.x ? ahead : 0; i < steps; ++i) {
                if (!mbar_wait(smem_u32(&s.empty[r.idx]), r.phase ^ 1u, abort_flag, a.err,
                               ROLE_PRODUCER, 20, kWaitLimitNs, KID_FP8)) {
                    ok = false;
                    break;
                }
                load_weights(r.idx, i, t * 128);
                load_tokens(r.idx, i);
                r.advance(Shape::kStages);
                ++issued;
            }
        }
        if (!ok) {           // the copies in flight land before the CTA goes
            const uint32_t n = Shape::kStages;
            for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i) {
                const unsigned long long t0 = globaltimer_ns();
                while (!mbar_try_wait(smem_u32(&s.full[i % n]), (i / n) & 1u) &&
                       globaltimer_ns() - t0 < kWaitLimitNs) {
                }
            }
        }
    } else if (warp == 1) {
        // --------------------------------------------------------------- products
        Ring r, d;
        bool ok = true;
        const uint32_t idesc = idesc_e4m3(128, kTok);
        for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
            for (int i = 0; i < steps; ++i) {
                ok = mbar_wait(smem_u32(&s.d_empty[d.idx]), d.phase ^ 1u, abort_flag, a.err,
                               ROLE_MMA, 20, kWaitLimitNs, KID_FP8) &&
                     mbar_wait(smem_u32(&s.full[r.idx]), r.phase, abort_flag, a.err, ROLE_MMA, 21,
                               kWaitLimitNs, KID_FP8);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t dw = desc_lo(sW + r.idx * Shape::kPerStep * Shape::kW);
                const uint32_t dk = desc_lo(sT + r.idx * Shape::kPerStep * Shape::kT);
                const uint32_t dt = tmem + d.idx * Shape::kPerStep * kTok;
                const int groups = a.G - i * Shape::kPerStep;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int j = 0; j < Shape::kPerStep; ++j) {
                            if (j >= groups) break;
                            const uint32_t w = dw + j * (Shape::kW >> 4) + 2 * k;
                            const uint32_t x = dk + j * (Shape::kT >> 4) + 2 * k;
                            if (k == 0) mma_e4m3<false>(dt + j * kTok, w, x, idesc);
                            else mma_e4m3<true>(dt + j * kTok, w, x, idesc);
                        }
                    }
                    mma_commit(smem_u32(&s.empty[r.idx]));
                    mma_commit(smem_u32(&s.d_full[d.idx]));
                }
                __syncwarp();
                r.advance(Shape::kStages);
                d.advance(Shape::kBufs);
            }
        }
        if (elect_one()) mma_commit(smem_u32(&s.drain));
        __syncwarp();
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&s.drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------- sums of groups
        griddep_wait();
        const int q = warp & 3;
        const uint32_t my_tmem = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const bool mine = lane < a.M;        // a lane brings the scales of token `lane`
        const float *sa = a.sa + static_cast<int64_t>(mine ? lane : 0) * a.G;
        Ring d;
        bool ok = true;
        for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
            const float *sw = a.sw + static_cast<int64_t>(t) * a.G;
            float acc[kTok];
#pragma unroll
            for (int j = 0; j < kTok; ++j) acc[j] = 0.0f;
            float fa[Shape::kPerStep], fw[Shape::kPerStep];
            auto ask = [&](int g) {
#pragma unroll
                for (int i = 0; i < Shape::kPerStep; ++i) {
                    const int at = min(g + i, a.G - 1);
                    fa[i] = ld_now(sa + at);
                    fw[i] = ld_now(sw + at);
                }
            };
            ask(0);
            for (int g = 0; g < a.G; g += Shape::kPerStep) {
                float f[Shape::kPerStep];
#pragma unroll
                for (int i = 0; i < Shape::kPerStep; ++i) f[i] = fa[i] * fw[i];
                ask(g + Shape::kPerStep);
                ok = mbar_wait(smem_u32(&s.d_full[d.idx]), d.phase, abort_flag, a.err,
                               ROLE_EPILOGUE, 20, kWaitLimitNs, KID_FP8);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                uint32_t v[Shape::kPerStep][kTok / 16][16];
#pragma unroll
                for (int i = 0; i < Shape::kPerStep; ++i)
#pragma unroll
                    for (int c = 0; c < kTok / 16; ++c)
                        tmem_ld_16cols(my_tmem + (d.idx * Shape::kPerStep + i) * kTok + 16 * c, v[i][c]);
#pragma unroll
                for (int i = 0; i < Shape::kPerStep; ++i)
#pragma unroll
                    for (int c = 0; c < kTok / 16; ++c) tmem_wait_ld_dep16(v[i][c]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(smem_u32(&s.d_empty[d.idx]));
                d.advance(Shape::kBufs);
#pragma unroll
                for (int i = 0; i < Shape::kPerStep; ++i) {
                    if (g + i >= a.G) break;         // (an odd last step: what it read is of an older one)
#pragma unroll
                    for (int j = 0; j < kTok; ++j)
                        acc[j] = fmaf(__uint_as_float(v[i][j / 16][j % 16]),
                                      __shfl_sync(0xFFFFFFFFu, f[i], j), acc[j]);
                }
            }
            const int n = t * 128 + q * 32 + lane;
            if (!ok || n >= a.N) continue;
#pragma unroll
            for (int j = 0; j < kTok; ++j) {
                if (j >= a.M) break;
                const int64_t at = static_cast<int64_t>(j) * a.N + n;
                if (a.out_fp32)
                    static_cast<float *>(a.y)[at] = acc[j];
                else
                    static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(acc[j]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kRowsTmemCols);
    }
}

// A matrix of bytes [rows, K] in boxes of box_rows rows x 128 K.
bool encode(CUtensorMap *map, const void *ptr, int64_t K, int64_t rows, int box_rows) {
    auto fn = tensor_map_encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
    cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <auto kernel, int kCtaThreads = kThreads>
cudaError_t launch_as(const CUtensorMap &ta, const CUtensorMap &tb, const Fp8Args &a, int grid,
                      cudaStream_t stream) {
    static int attr_done[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        // setmaxnreg.inc can only take registers that the CTA was launched with
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
        if (kCtaThreads == kThreads &&
            fa.numRegs * kThreads < static_cast<int>(256 * kSumRegs + 128 * kOtherRegs))
            return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (e != cudaSuccess) return e;
        attr_done[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kCtaThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, ta, tb, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8Problem &p, int num_sms, cudaStream_t stream) {
    Fp8Args a;
    a.sa = p.sa;
    a.sw = p.sw;
    a.y = p.y;
    a.M = static_cast<int>(p.M);
    a.N = static_cast<int>(p.N);
    a.G = static_cast<int>(p.K >> 7);
    a.m_tiles = (a.M + kTokens - 1) / kTokens;
    // The slice's width: the least waves x width (a wave takes as long as its tiles are
    // wide, and the 16 stand for its ends), the wider where two are level (fewer reads of
    // the tokens).
    int64_t best = INT64_MAX;
    a.w = 8;
    for (int w = 8; w <= kMaxSlice; w += w < 32 ? 8 : 16) {
        const int64_t tiles = static_cast<int64_t>(a.m_tiles) * ((a.N + w - 1) / w);
        const int64_t cost = (tiles + num_sms - 1) / num_sms * (w + 16);
        if (cost <= best) {
            best = cost;
            a.w = w;
        }
    }
    a.out_fp32 = p.out_fp32;
    a.early = p.chained;
    const int per32 = p.out_fp32 ? 8 : 16;
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    a.words = p.out_fp32 || (a.N % 2 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 3) == 0);
    CUtensorMap ta, tb;
    if (a.M <= kRowsMaxTokens) {
        a.tiles = (a.N + 127) / 128;
        const int tok = a.M <= 16 ? 16 : 32;
        if (!encode(&ta, p.qa, p.K, p.M, tok) || !encode(&tb, p.qw, p.K, p.N, 128))
            return cudaErrorInvalidValue;
        // As many CTAs as have the same number of tiles each: some SMs' second tiles alone do
        // not take what HBM gives (against a CTA on every SM: 8 x 28672 x 8192, 112 CTAs, 38.0 / 40.7
        // us; 1 x 20480 x 4096, 80, 16.5 / 19.2; 32 x 40000 x 4096, 105, 30.9 / 35.3; 8 x 65536 x 2048,
        // 128, 24.0 / 24.2).
        const int waves = (a.tiles + num_sms - 1) / num_sms;
        const int grid = (a.tiles + waves - 1) / waves;
        return tok == 16
                   ? launch_as<gemm_fp8_rows_kernel<16>, kRowsThreads>(ta, tb, a, grid, stream)
                   : launch_as<gemm_fp8_rows_kernel<32>, kRowsThreads>(ta, tb, a, grid, stream);
    }
    // Pairs of CTAs, where their waves of tiles take less: a tile of theirs takes as long as one of
    // w = 164 (single CTAs / pairs: 512 x 4096 x 4096, w = 112, 15.8 / 18.5 us; 8192 x 256 x
    // 2048, w = 128, 9.9 / 11.6; 777 x 4200 x 2048, w = 208, 19.1 / 15.2; 8192 x 512 x 2048, w =
    // 256, 16.0 / 12.5; 4096 x 8192 x 8192 319 / 209).
    const int64_t m2 = (a.M + kPairTokens - 1) / kPairTokens, n2 = (a.N + kPairRows - 1) / kPairRows;
    const int64_t pairs = num_sms / 2;
    if ((m2 * n2 + pairs - 1) / pairs * (164 + 16) < best && m2 * n2 <= INT32_MAX - 4096) {
        a.m_tiles = static_cast<int>(m2);
        a.tiles = static_cast<int>(m2 * n2);
        a.wide_store = (reinterpret_cast<uintptr_t>(p.y) & 31) == 0 && a.N % per32 == 0;
        if (!encode(&ta, p.qa, p.K, p.M, 128) || !encode(&tb, p.qw, p.K, p.N, 128))
            return cudaErrorInvalidValue;
        const int grid = 2 * static_cast<int>(a.tiles < pairs ? a.tiles : pairs);
        return launch_as<gemm_fp8_pair_kernel>(ta, tb, a, grid, stream);
    }
    a.n_mma = (a.w + 15) / 16 * 16;
    a.half = a.w <= 32 ? a.w : (a.w / 2 + 15) / 16 * 16;
    const int a_rows = a.M >= kTokens ? kTokens : (a.M + 7) / 8 * 8;
    a.a_box = a_rows * 128;
    a.b_box = a.w * 128;
    a.a_bytes = a.a_box;
    a.b_bytes = a.n_mma * 128;
    // An instruction reads 128 rows of tokens, past the last stage's where they are fewer:
    // into the weights' stages and the outputs' place behind them, 16 KB at least. (Those
    // lanes of tensor memory are never read.)
    static_assert(kStagedBytes >= 128 * 128);
    const int room = kSmemBytes - 1024 - kOffStages - kStagedBytes;
    a.buf_cols = (a.w + 31) / 32 * 32;
    // Groups of a step. Handing a stage and a buffer on takes some 400 cycles a step, more than the
    // weights of a narrow slice: as many as leave two buffers and four stages.
    a.per_step = kMaxPerStep;
    while (a.per_step > 1 && (2 * a.per_step * a.buf_cols > kTmemCols ||
                              4 * a.per_step * (a.a_bytes + a.b_bytes) > room || a.per_step > a.G))
        a.per_step /= 2;
    a.stages = room / (a.per_step * (a.a_bytes + a.b_bytes));
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    a.bufs = kTmemCols / (a.per_step * a.buf_cols);
    if (a.bufs > kMaxBufs) a.bufs = kMaxBufs;
    // (the second half's columns are read up to a multiple of 32)
    const int last = (a.bufs * a.per_step - 1) * a.buf_cols + (a.w > a.half ? a.half : 0);
    if (last + (a.half + 31) / 32 * 32 > kTmemCols || (a.half > 64 && a.per_step != 1))
        return cudaErrorInvalidValue;
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * ((a.N + a.w - 1) / a.w);
    if (tiles > INT32_MAX - 4096) return cudaErrorInvalidValue;
    a.tiles = static_cast<int>(tiles);
    a.wide_store = (reinterpret_cast<uintptr_t>(p.y) & 31) == 0 && a.N % per32 == 0 && a.w % per32 == 0;
    if (!encode(&ta, p.qa, p.K, p.M, a_rows) || !encode(&tb, p.qw, p.K, p.N, a.w))
        return cudaErrorInvalidValue;
    const int grid = a.tiles < num_sms ? a.tiles : num_sms;
    if (a.half <= 32) return launch_as<gemm_fp8_kernel<32>>(ta, tb, a, grid, stream);
    if (a.half <= 64) return launch_as<gemm_fp8_kernel<64>>(ta, tb, a, grid, stream);
    if (a.half <= 96) return launch_as<gemm_fp8_kernel<96>>(ta, tb, a, grid, stream);
    return launch_as<gemm_fp8_kernel<128>>(ta, tb, a, grid, stream);
}

}  // namespace w8a8
