// A whole mixture-of-experts layer for a few tokens, on sm_103a: the experts that the
// gate picked (gate.cu) for T <= 32 tokens, in one kernel ("Deploying Hunyuan
// 770B in INT8 on domestic accelerators", §1.3 and §4.1). With few tokens the layer
// is a stream of the picked experts' weights, read once; the six kernels that
// moe_ffn takes for many tokens cost more than the stream.
//
//   u = (x's codes . W_gate_up[e]) in exact group sums, scaled in group order
//   h = silu(gate) * up, quantized per (token, expert)
//   d = (h's codes . W_down[e]), y[t] = sum_j w[t, j] d[t, j]
//
// Every step is that of moe_ffn, rounding for rounding, so y is the same bits.
//
// The grid is one CTA per SM, launched cooperatively, since its parts wait on one
// another three times: for the tokens' codes, for h (its scale needs whole
// rows), and for h's codes.
//
// Work. The rows of all picked experts form a line, and every warp of the grid takes
// an equal stretch of it, whatever the routing: rows of gate and up in pairs for
// the first product; for the second a CTA has the same output rows of every
// expert, so that it adds up its tokens' experts by itself, and its warps share
// those. A warp takes its rows 16 at a time (8 pairs), one K group of 128 per
// step, through a ring of its own in shared memory (cp.async, no barrier with other
// warps). The ring runs on through the waits: the first weights of a product are
// asked for before what they are multiplied with is there.
//
// A step is eight mma.sync m16n8k16 on fp16 (weights' rows x tokens x 128 K): codes are
// exact in fp16 and a group's sum in FP32, as in the other products here. K is permuted
// alike on both sides, so that a lane has 32 consecutive codes of its rows, and of its
// token's codes, which are kept as fp16.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "moe_math.cuh"
#include "quant_math.cuh"

namespace w8a8 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;
constexpr int kStageBytes = 16 * 128;
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kSyncs = 3;                    // grid-wide waits
constexpr unsigned kFull = 0xFFFFFFFFu;

struct LayerArgs {
    const uint16_t *x;
    int64_t ldx;
    int vec;                                 // rows of x may be read 16 bytes at a time
    const int32_t *ids;
    const float *w;
    int T, k, E, H, I;
    const int8_t *qw_up, *qw_down;
    const float *sw_up, *sw_down;
    void *y;
    int out_fp32;
    unsigned *sync;                          // [kSyncs], zeros
    unsigned *hmax;                          // [T k], zeros: largest |h| as bits
    float *sx;                               // [T]
    __half *xq;                              // [T, H] codes
    float *h;                                // [T k, I]
    __half *hq;                              // [T k, I] codes
    float *d;                                // [T k, H]
    unsigned long long *err;
};

// What the gate picked, by expert: those with tokens, in order of their index, and the
// (token, choice) pairs of each.
struct Routes {
    int count[kMaxExperts];                  // then the expert's first pair
    int expert[kMoeFewMaxPairs];
    int first[kMoeFewMaxPairs + 1];
    int pair[kMoeFewMaxPairs];
    int part[kWarps];
    int n;
    int abort;
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 operands, FP32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Waits until every CTA of the grid has come here. A CTA whose wait gives up says so
// and leaves, and so do the others, each by its own limit.
__device__ __forceinline__ bool grid_wait(unsigned *counter, int *abort, unsigned long long *err,
                                          unsigned site) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        unsigned seen;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                     : "=r"(seen) : "l"(counter) : "memory");
        const unsigned long long t0 = globaltimer_ns();
        unsigned i = 0;
        ++seen;
        while (seen < gridDim.x) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                         : "=r"(seen) : "l"(counter) : "memory");
            if ((++i & 255u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                record_device_error(err, KID_MOE, ROLE_EPILOGUE, site);
                break;
            }
        }
        __threadfence();
    }
    __syncthreads();
    return *abort == 0;
}

// Exclusive sum over the block's threads.
__device__ __forceinline__ int block_scan(int v, int *part, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    const int mine = lane < kWarps ? part[lane] : 0;
    const int before = __reduce_add_sync(kFull, lane < warp ? mine : 0);
    total = __reduce_add_sync(kFull, mine);
    __syncthreads();
    return before + incl - v;
}

// The routes, from the ids: every CTA makes them for itself (at most 512 ids).
__device__ __forceinline__ void make_routes(const LayerArgs &a, Routes &r) {
    const int n = a.T * a.k;                 // <= kThreads
    for (int e = threadIdx.x; e < a.E; e += kThreads) r.count[e] = 0;
    if (threadIdx.x == 0) r.abort = 0;
    __syncthreads();
    int id = -1, place = 0;
    if (threadIdx.x < n) {
        id = a.ids[threadIdx.x];
        if (id < 0 || id >= a.E) id = -1;
        // (an expert's pairs come in any order: each is a column of its own)
        if (id >= 0) place = atomicAdd(&r.count[id], 1);
    }
    __syncthreads();
    // two experts per thread; experts with tokens and pairs are counted together
    const int e0 = 2 * threadIdx.x;
    const int c0 = e0 < a.E ? r.count[e0] : 0, c1 = e0 + 1 < a.E ? r.count[e0 + 1] : 0;
    int total;
    const int at = block_scan(((c0 > 0) + (c1 > 0)) << 16 | (c0 + c1), r.part, total);
    int slot = at >> 16, pairs = at & 0xFFFF;
    if (c0 > 0) {
        r.expert[slot] = e0;
        r.first[slot++] = pairs;
        r.count[e0] = pairs;
        pairs += c0;
    }
    if (c1 > 0) {
        r.expert[slot] = e0 + 1;
        r.first[slot] = pairs;
        r.count[e0 + 1] = pairs;
    }
    if (threadIdx.x == 0) {
        r.n = total >> 16;
        r.first[total >> 16] = total & 0xFFFF;
    }
    __syncthreads();
    if (id >= 0) r.pair[r.count[id] + place] = threadIdx.x;
    __syncthreads();
}

// A warp's stretch of the line of rows: units (experts) of L rows, of which a tile takes
// up to kMost from one unit; `steps` groups of K per tile.
struct Cursor {
    int pos, end;            // in rows of the line
    int unit, at;            // the unit that pos lies in, and its row there
    __device__ __forceinline__ Cursor(int64_t units, int L, int part, int parts) {
        const int64_t total = units * L;
        pos = static_cast<int>(total * part / parts);
        end = static_cast<int>(total * (part + 1) / parts);
        unit = pos / L;
        at = pos - unit * L;
    }
    __device__ __forceinline__ int rows(int L, int most) const {
        return min(min(most, end - pos), L - at);
    }
    __device__ __forceinline__ void next(int n, int L) {
        pos += n;
        at += n;
        if (at == L) {
            at = 0;
            ++unit;
        }
    }
};

// The weights' side of a product: kUp, pairs of rows (i, I + i) of W_gate_up, else rows
// [r0, r0 + L) of W_down.
template <bool kUp>
struct Feed {
    static constexpr int kMost = kUp ? 8 : 16;
    Cursor c;
    int step, rows;
    uint32_t dst;            // the lane's piece of the stage that the next copy goes to
    const int8_t *src;       // the lane's piece of the tile's first row, at that step

    __device__ __forceinline__ Feed(const LayerArgs &a, const Routes &r, uint32_t ring, int r0,
                                    int L, int part, int parts)
        : c(r.n, L, part, parts), step(0), rows(0), src(nullptr) {
        const int lane = threadIdx.x & 31;
        dst = ring + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
        open(a, r, r0, L);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(a, r, ring, r0, L);
    }
    __device__ __forceinline__ void open(const LayerArgs &a, const Routes &r, int r0, int L) {
        if (c.pos >= c.end) return;
        const int lane = threadIdx.x & 31;
        rows = c.rows(L, kMost) - (lane >> 3);       // rows from the lane's first on
        const int64_t e = r.expert[c.unit];
        src = kUp ? a.qw_up + (e * 2 * a.I + c.at + (lane >> 3)) * a.H
                  : a.qw_down + (e * a.H + r0 + c.at + (lane >> 3)) * a.I;
        src += (lane & 7) * 16;
    }
    // Asks for the next step's weights.
    __device__ __forceinline__ void issue(const LayerArgs &a, const Routes &r, uint32_t ring,
                                          int r0, int L) {
        if (c.pos < c.end) {
            // rows 0-3, 4-7 (whose swizzle differs in bit 2), 8-11, 12-15
            const int K = kUp ? a.H : a.I;
            const int64_t third = kUp ? static_cast<int64_t>(a.I) * a.H : 8 * K;
            if (rows > 0) cp_async_16(dst, src);
            if (rows > 4) cp_async_16((dst ^ 64) + 512, src + 4 * K);
            if (rows > (kUp ? 0 : 8)) cp_async_16(dst + 1024, src + third);
            if (rows > (kUp ? 4 : 12)) cp_async_16((dst ^ 64) + 1536, src + third + 4 * K);
            src += 128;
            if (++step == K >> 7) {
                step = 0;
                c.next(c.rows(L, kMost), L);
                open(a, r, r0, L);
            }
        }
        cp_async_commit();
        dst += kStageBytes;
        if (dst - ring >= kStages * kStageBytes) dst -= kStages * kStageBytes;
    }
};

// One tile: 16 rows of weights by up to 8 NT tokens, over all of K. acc: [token tile][the
// lane's outputs: rows g and g + 8, tokens 2 c and 2 c + 1], g = lane / 4, c = lane % 4.
template <int NT, bool kUp>
__device__ __forceinline__ void tile_product(const LayerArgs &a, const Routes &r, Feed<kUp> &f,
                                             uint32_t ring, int r0, int L, uint32_t &read,
                                             const __half *codes, const int (&tok)[NT],
                                             const float *sw0, const float *sw1,
                                             float (&acc)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
    const int steps = (kUp ? a.H : a.I) >> 7;
    for (int s = 0; s < steps; ++s) {
        uint4 b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = reinterpret_cast<const uint4 *>(codes + tok[0] + s * 128)[i];
        const float w0 = sw0[s], w1 = sw1[s];
        cp_async_wait<kStages - 2>();
        __syncwarp();                        // the stage is there; the one before is read
        f.issue(a, r, ring, r0, L);
        const uint32_t at = read;
        read += kStageBytes;
        if (read - ring >= kStages * kStageBytes) read -= kStages * kStageBytes;
        uint4 q[4] = {lds128(at), lds128(at ^ 16), lds128(at + 1024), lds128((at ^ 16) + 1024)};
        uint32_t lo[2][8], hi[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t word[8] = {q[2 * i].x,     q[2 * i].y,     q[2 * i].z,     q[2 * i].w,
                                      q[2 * i + 1].x, q[2 * i + 1].y, q[2 * i + 1].z, q[2 * i + 1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) i8x4_to_f16x4(word[j], lo[i][j], hi[i][j]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n > 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    b[i] = reinterpret_cast<const uint4 *>(codes + tok[n] + s * 128)[i];
            }
            float p[2][4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma_16816(p[0], lo[0][2 * j], lo[1][2 * j], hi[0][2 * j], hi[1][2 * j], b[j].x, b[j].y);
                mma_16816(p[1], lo[0][2 * j + 1], lo[1][2 * j + 1], hi[0][2 * j + 1],
                          hi[1][2 * j + 1], b[j].z, b[j].w);
            }
            // (sums of integers below 2^24: exact in any order)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[n][j] = fmaf(p[0][j] + p[1][j], j < 2 ? w0 : w1, acc[n][j]);
        }
    }
}

template <int NT, bool kUp>
__device__ __forceinline__ void take_tile(const LayerArgs &a, const Routes &r, Feed<kUp> &f,
                                          const Cursor &c, int rows, uint32_t ring, int r0, int L,
                                          uint32_t &read, int p0, int n_tok) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int64_t e = r.expert[c.unit];
    const int K = kUp ? a.H : a.I;
    int tok[NT];                             // where the lane's tokens' codes are
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        // (columns past the last token repeat it and are not stored)
        const int pair = r.pair[p0 + min(8 * n + g, n_tok - 1)];
        tok[n] = (kUp ? pair / a.k : pair) * K + q * 32;
    }
    const int groups = K >> 7;
    const float *sw0, *sw1;
    if (kUp) {
        sw0 = a.sw_up + (e * 2 * a.I + c.at + min(g, rows - 1)) * groups;
        sw1 = sw0 + static_cast<int64_t>(a.I) * groups;
    } else {
        sw0 = a.sw_down + (e * a.H + r0 + c.at + min(g, rows - 1)) * groups;
        sw1 = a.sw_down + (e * a.H + r0 + c.at + min(g + 8, rows - 1)) * groups;
    }
    float acc[NT][4];
    tile_product<NT, kUp>(a, r, f, ring, r0, L, read, kUp ? a.xq : a.hq, tok, sw0, sw1, acc);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = 8 * n + 2 * q + j;
            const int pair = r.pair[p0 + min(col, n_tok - 1)];
            if (kUp) {
                float h = 0.0f;
                if (col < n_tok && g < rows) {
                    const float s = a.sx[pair / a.k];
                    h = swiglu_f32(__fmul_rn(acc[n][j], s), __fmul_rn(acc[n][j + 2], s));
                    a.h[static_cast<int64_t>(pair) * a.I + c.at + g] = h;
                }
                unsigned m = __float_as_uint(fabsf(h));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
                if (g == 0 && col < n_tok) atomicMax(a.hmax + pair, m);
            } else if (col < n_tok) {
                const float s = __fdiv_rn(__uint_as_float(a.hmax[pair]), 127.0f);
                float *d = a.d + static_cast<int64_t>(pair) * a.H + r0 + c.at;
                if (g < rows) d[g] = __fmul_rn(acc[n][j], s);
                if (g + 8 < rows) d[g + 8] = __fmul_rn(acc[n][j + 2], s);
            }
        }
    }
}

// The warp's share of a product.
template <bool kUp>
__device__ __forceinline__ void product(const LayerArgs &a, const Routes &r, Feed<kUp> &f,
                                        Cursor c, uint32_t ring, int L, int r0) {
    // the lane's first piece of a stage: row lane / 4, 16-byte pieces 2 (lane % 4) and the
    // next, swizzled by the row
    const int lane = threadIdx.x & 31;
    uint32_t read = ring + (lane >> 2) * 128 + (((2 * (lane & 3)) ^ (lane >> 2)) << 4);
    while (c.pos < c.end) {
        const int rows = c.rows(L, Feed<kUp>::kMost);
        const int p0 = r.first[c.unit], n_tok = r.first[c.unit + 1] - p0;
        if (n_tok <= 8)
            take_tile<1, kUp>(a, r, f, c, rows, ring, r0, L, read, p0, n_tok);
        else if (n_tok <= 16)
            take_tile<2, kUp>(a, r, f, c, rows, ring, r0, L, read, p0, n_tok);
        else
            take_tile<4, kUp>(a, r, f, c, rows, ring, r0, L, read, p0, n_tok);
        c.next(rows, L);
    }
    cp_async_wait<0>();
}

// Codes and scales of the tokens blockIdx.x, + gridDim.x, ...
__device__ __forceinline__ void quantize_tokens(const LayerArgs &a, int *red) {
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const uint16_t *row = a.x + t * a.ldx;
        auto load8 = [&](int i) {
            if (a.vec) return reinterpret_cast<const uint4 *>(row)[i];
            uint4 v;
            uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = row[8 * i + 2 * j] | static_cast<uint32_t>(row[8 * i + 2 * j + 1]) << 16;
            return v;
        };
        unsigned m = 0;
        for (int i = threadIdx.x; i < a.H >> 3; i += kThreads) m = max(m, amax_bits8(load8(i)));
        m = __reduce_max_sync(kFull, m);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        m = __reduce_max_sync(kFull, (threadIdx.x & 31) < kWarps ? red[threadIdx.x & 31] : 0u);
        const float s = __fdiv_rn(bf16_bits_to_f32(m), 127.0f);
        const bool fast = s >= 1.17549435e-38f;      // a normal scale: 1 / s is finite
        const float rcp = fast ? __frcp_rn(s) : 0.0f;
        if (threadIdx.x == 0) a.sx[t] = s;
        for (int i = threadIdx.x; i < a.H >> 3; i += kThreads)
            reinterpret_cast<uint4 *>(a.xq + static_cast<int64_t>(t) * a.H)[i] =
                quantize8_f16(load8(i), s, rcp, fast);
    }
}

// Codes of h, 8 values per thread at a time, spread over the grid. (By the pairs' own
// index: their order within an expert is each CTA's own. Pairs that are not routed
// have no largest h, and zeros.)
__device__ __forceinline__ void quantize_h(const LayerArgs &a) {
    const int per = a.I >> 3;
    const int n = a.T * a.k * per;
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads) {
        const int pair = i / per;
        const int64_t at = static_cast<int64_t>(i) * 8;
        const float s = __fdiv_rn(__uint_as_float(__ldcg(a.hmax + pair)), 127.0f);
        const bool fast = s >= 1.17549435e-38f;
        const float rcp = fast ? __frcp_rn(s) : 0.0f;
        const float4 u = __ldcg(reinterpret_cast<const float4 *>(a.h + at));
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.h + at) + 1);
        const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 p =
                __floats2half2_rn(code_plus_round(x[2 * j], s, rcp, fast) - kRoundAdd,
                                  code_plus_round(x[2 * j + 1], s, rcp, fast) - kRoundAdd);
            o[j] = *reinterpret_cast<const uint32_t *>(&p);
        }
        *reinterpret_cast<uint4 *>(a.hq + at) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
moe_layer_kernel(const LayerArgs a) {
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ Routes r;
    __shared__ int s_red[kWarps];
    griddep_wait();
    make_routes(a, r);
    const int warp = threadIdx.x >> 5;
    const uint32_t ring = smem_u32(s_ring) + warp * kStages * kStageBytes;
    const int part = blockIdx.x * kWarps + warp, parts = gridDim.x * kWarps;
    {
        Feed<true> f(a, r, ring, 0, a.I, part, parts);
        const Cursor c(r.n, a.I, part, parts);
        quantize_tokens(a, s_red);
        if (!grid_wait(a.sync + 0, &r.abort, a.err, 0)) {
            cp_async_wait<0>();
            return;
        }
        product<true>(a, r, f, c, ring, a.I, 0);
    }
    // the CTA's output rows
    const int r0 = static_cast<int>(static_cast<int64_t>(a.H) * blockIdx.x / gridDim.x);
    const int L = static_cast<int>(static_cast<int64_t>(a.H) * (blockIdx.x + 1) / gridDim.x) - r0;
    if (L > 0) {
        __syncwarp();
        Feed<false> f(a, r, ring, r0, L, warp, kWarps);
        const Cursor c(r.n, L, warp, kWarps);
        bool ok = grid_wait(a.sync + 1, &r.abort, a.err, 1);
        if (ok) {
            quantize_h(a);
            ok = grid_wait(a.sync + 2, &r.abort, a.err, 2);
        }
        griddep_launch_dependents();
        if (!ok) {
            cp_async_wait<0>();
            return;
        }
        product<false>(a, r, f, c, ring, L, r0);
    } else {
        if (!grid_wait(a.sync + 1, &r.abort, a.err, 1)) return;
        quantize_h(a);
        grid_wait(a.sync + 2, &r.abort, a.err, 2);
        return;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * L; i += kThreads) {
        const int t = i / L, n = r0 + i - t * L;
        float acc = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int id = a.ids[t * a.k + j];
            if (id < 0 || id >= a.E) continue;
            acc = fmaf(a.w[t * a.k + j], a.d[static_cast<int64_t>(t * a.k + j) * a.H + n], acc);
        }
        const int64_t at = static_cast<int64_t>(t) * a.H + n;
        if (a.out_fp32)
            static_cast<float *>(a.y)[at] = acc;
        else
            static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(acc);
    }
}

struct FewLayout {
    size_t sync, hmax, sx, xq, h, hq, d, total;
};
FewLayout few_layout(int64_t T, int64_t k, int64_t H, int64_t I) {
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t at = off;
        off += (n + 255) / 256 * 256;
        return at;
    };
    const size_t n = static_cast<size_t>(T * k);
    FewLayout l;
    l.sync = take((kSyncs + n) * 4);
    l.hmax = l.sync + kSyncs * 4;
    l.sx = take(T * 4);
    l.xq = take(static_cast<size_t>(T) * H * 2);
    l.h = take(n * I * 4);
    l.hq = take(n * I * 2);
    l.d = take(n * H * 4);
    l.total = off;
    return l;
}

}  // namespace

size_t moe_few_workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I) {
    return few_layout(T, k, H, I).total;
}

void moe_few_zeroes(const MoeFewProblem &p, uint32_t **words, int *n) {
    const FewLayout l = few_layout(p.T, p.k, p.H, p.I);
    *words = reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.workspace) + l.sync);
    *n = static_cast<int>(kSyncs + p.T * p.k);
}

cudaError_t launch_moe_few(const MoeFewProblem &p, int num_sms, cudaStream_t stream) {
    const FewLayout l = few_layout(p.T, p.k, p.H, p.I);
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    LayerArgs a;
    a.x = p.x;
    a.ldx = p.ldx;
    a.vec = p.ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 15) == 0;
    a.ids = p.ids;
    a.w = p.w;
    a.T = static_cast<int>(p.T);
    a.k = static_cast<int>(p.k);
    a.E = static_cast<int>(p.E);
    a.H = static_cast<int>(p.H);
    a.I = static_cast<int>(p.I);
    a.qw_up = p.qw_up;
    a.qw_down = p.qw_down;
    a.sw_up = p.sw_up;
    a.sw_down = p.sw_down;
    a.y = p.y;
    a.out_fp32 = p.out_fp32;
    a.sync = reinterpret_cast<unsigned *>(ws + l.sync);
    a.hmax = reinterpret_cast<unsigned *>(ws + l.hmax);
    a.sx = reinterpret_cast<float *>(ws + l.sx);
    a.xq = reinterpret_cast<__half *>(ws + l.xq);
    a.h = reinterpret_cast<float *>(ws + l.h);
    a.hq = reinterpret_cast<__half *>(ws + l.hq);
    a.d = reinterpret_cast<float *>(ws + l.d);
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    static int attr_done[64] = {0};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        e = cudaFuncSetAttribute(moe_layer_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kRingBytes);
        if (e != cudaSuccess) return e;
        attr_done[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRingBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, moe_layer_kernel, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace w8a8
