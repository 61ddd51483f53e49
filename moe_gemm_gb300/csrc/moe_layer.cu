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
// Every step is that of moe_ffn, rounding for rounding, so y is the same bits. The tokens'
// codes come from the gate's launch.
//
// The grid is one CTA per SM, launched cooperatively, since its parts wait on one
// another twice: for h (its scale needs whole rows), and for h's codes.
//
// Work. The rows of all picked experts form a line, which is cut into stretches of equal
// cost for the warps of the grid. Of the second product a CTA has the same output rows
// of every expert, so that it adds up its tokens' experts by itself, and its warps cut
// that line. A warp takes its rows 16 at a time (of the first product 8 rows of gate and the
// 8 of up that belong to them), one K group of 128 per step, through a ring of its own in
// shared memory (cp.async, no barrier with other warps). The ring runs on through the waits.
//
// A step of an expert with three and more tokens is four mma.sync m16n8k32 on the int8 codes
// (weights' rows x tokens x 128 K), of one with one or two tokens dp4a: a group's sum is an
// exact integer either way. K is permuted alike on both sides, so that a lane has 32
// consecutive codes of its rows, and of its token's codes.
//
// What bounds it. 16 tokens, 8 of 64 experts (H 4096, I 1536, 1.1 GB): 221 us with the gate, 5.0
// TB/s; 24 tokens of 256 experts (H 2048, I 640, 554 MB): 100 us, 5.6 TB/s; there the SMs that
// end their stretch last, 10 % after the mean (L1 at 52 % of its peak, issue slots 36 %). 32 tokens of
// 64 experts (1.2 GB): 302 us, 4.1 TB/s: most experts have three tokens and more, whose steps ask for
// the tokens' codes and use them at once (L1 35 %, issue slots 28 %: latency). One token (156 MB):
// 45 us, 3.4 TB/s: the streams take 28, the
// rest are the gate and two launches (4), the routes and the first loads (3), two waits of the
// grid with h's codes between them (6) and the ends of the streams. Measured on the way (16 tokens):
// operands widened to fp16, as moe_ffn has them, 246 us; dp4a for up to 8 tokens 435; even
// stretches instead of equal costs 232; a fifth to a half of the line taken in pieces by warps
// that are done 240 to 223, but 57 instead of 46 for one token; L2 prefetches during the
// waits, h's codes made by every CTA, 3 or 6 stages: no gain.
#include <cuda_bf16.h>
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
constexpr int kMaxOutputBytes = 64 << 10;   // d of a CTA's rows, in shared memory
constexpr int kSyncs = 2;                    // grid-wide waits
constexpr int kQueue = 8;                    // tiles that a ring is ahead at most
constexpr unsigned kFull = 0xFFFFFFFFu;
// What a row of an expert costs, by its tokens: stretches of one length took 190, 222 and 255
// thousand cycles where all their experts had one, two and more tokens.
constexpr int kCostOne = 6, kCostTwo = 7, kCostMore = 8;

struct LayerArgs {
    const int32_t *ids;
    const float *w;
    int T, k, E, H, I;
    const int8_t *qw_up, *qw_down;
    const float *sw_up, *sw_down;
    void *y;
    int out_fp32;
    unsigned *sync;                          // [kSyncs], zeros
    unsigned *hmax;                          // [T k], zeros: largest |h| as bits
    const float *sx;                         // [T]
    const int8_t *xq;                        // [T, H] codes
    float *h;                                // [T k, I]
    int8_t *hq;                              // [T k, I] codes
    unsigned long long *err;
};

// A warp's stretch of the line of rows, and the tiles it has been cut into.
struct Stretch {
    int pos, end;            // rows of the line
    int unit, at;            // the unit that pos lies in, and its row there
    int opened;              // tiles so far
    int2 tile[kQueue];       // the last of them: {unit << 8 | rows, first row}
};

// What the gate picked, by expert: those with tokens, in order of their index, and the
// (token, choice) pairs of each.
struct Routes {
    int count[kMaxExperts];                  // then the expert's first pair
    int expert[kMoeFewMaxPairs];
    int first[kMoeFewMaxPairs + 1];
    int cost[kMoeFewMaxPairs + 1];           // of a row of all experts before
    int pair[kMoeFewMaxPairs];
    int part[kWarps];
    Stretch stretch[2][kWarps];              // of both products
    float w[kMoeFewMaxPairs];                // of the pairs
    bool routed[kMoeFewMaxPairs];            // whether they have an expert
    int n;
    int abort;
};

static_assert(kRingBytes + kMaxOutputBytes + sizeof(Routes) <= 227 * 1024);

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

// D[16 x 8] += A[16 x 32] B[32 x 8], int8 operands, int32 sums.
__device__ __forceinline__ void mma_16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Waits until every CTA of the grid has come here. A CTA whose wait gives up says so
// and leaves, and so do the others, each by its own limit.
__device__ __forceinline__ bool grid_wait(unsigned *counter, int *abort, unsigned long long *err,
                                          unsigned site) {
    __syncthreads();
    if (threadIdx.x == 0) {
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
    griddep_wait();                          // (the ids, and the tokens' codes)
    int id = -1, place = 0;
    if (threadIdx.x < n) {
        id = a.ids[threadIdx.x];
        if (id < 0 || id >= a.E) id = -1;
        r.w[threadIdx.x] = a.w[threadIdx.x];
        r.routed[threadIdx.x] = id >= 0;
        // (an expert's pairs come in any order: each is a column of its own)
        if (id >= 0) place = atomicAdd(&r.count[id], 1);
    }
    __syncthreads();
    // two experts per thread; experts with tokens (10 bits), pairs (10 bits) and what a row costs
    // beyond the least (at most 512 * (kCostMore - kCostOne)) are summed together
    static_assert(kCostMore - kCostOne <= 4 && kMoeFewMaxPairs <= 512);
    const int e0 = 2 * threadIdx.x;
    const int c0 = e0 < a.E ? r.count[e0] : 0, c1 = e0 + 1 < a.E ? r.count[e0 + 1] : 0;
    auto more = [](int n) { return n <= 1 ? 0 : n == 2 ? kCostTwo - kCostOne : kCostMore - kCostOne; };
    int total;
    const int at = block_scan(((c0 > 0) + (c1 > 0)) | (c0 + c1) << 10 | (more(c0) + more(c1)) << 20,
                              r.part, total);
    int slot = at & 1023, pairs = at >> 10 & 1023, cost = slot * kCostOne + (at >> 20);
    if (c0 > 0) {
        r.expert[slot] = e0;
        r.first[slot] = pairs;
        r.cost[slot++] = cost;
        r.count[e0] = pairs;
        pairs += c0;
        cost += kCostOne + more(c0);
    }
    if (c1 > 0) {
        r.expert[slot] = e0 + 1;
        r.first[slot] = pairs;
        r.cost[slot] = cost;
        r.count[e0 + 1] = pairs;
    }
    if (threadIdx.x == 0) {
        r.n = total & 1023;
        r.first[r.n] = total >> 10 & 1023;
        r.cost[r.n] = r.n * kCostOne + (total >> 20);
    }
    __syncthreads();
    if (id >= 0) r.pair[r.count[id] + place] = threadIdx.x;
    __syncthreads();
}

// Groups of K that a step of a tile takes: tiles that are not full, of experts with one or two
// tokens, take 2 or 4 so that the ring still has as many bytes on their way (a step lasts a
// third of HBM's latency, whatever it holds).
template <bool kUp>
__device__ __forceinline__ int tile_groups(int rows, int n_tok, int K) {
    const int full = (kUp ? 8 : 16) / rows;
    if (n_tok > 2 || full < 2 || K % 256 != 0) return 1;
    return full >= 4 && K % 512 == 0 ? 4 : 2;
}
// Where a 16-byte piece of a row of a stage lies, such that what eight lanes read at once
// (take_tile, take_tile_dot) is in different banks.
__device__ __forceinline__ int swizzled(int piece, int row, int wide) {
    return wide == 1   ? piece ^ (row & 7)
           : wide == 2 ? piece ^ ((row & 1) | (piece >> 3 << 1))
                       : piece ^ (piece >> 3);
}

// Where part `part` of `parts` equal parts of n begins. (n * part / parts in 32 bits: a 64-bit
// division takes a microsecond.)
__device__ __forceinline__ int share(int n, int part, int parts) {
    const unsigned q = static_cast<unsigned>(n) / parts, rest = n - q * parts;
    return q * part + rest * part / parts;
}

// The warp's stretches of both lines, of units of L rows (part of parts) and of R rows (the warp's of
// the CTA's): four borders, a lane each.
__device__ __forceinline__ void cut_line(Routes &r, int L, int part, int parts, int R) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool second = lane & 2;
    const int rows = second ? R : L;
    const int at = second ? share(r.cost[r.n] * rows, warp + (lane & 1), kWarps)
                          : share(r.cost[r.n] * rows, part + (lane & 1), parts);  // <= 512 * 8 * 8192
    int lo = 0, hi = r.n;                    // cost[lo] rows <= at < cost[hi] rows
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (r.cost[mid] * rows <= at) lo = mid; else hi = mid;
    }
    int row = 0;
    if (r.n > 0 && rows > 0) row = min(rows, (at - r.cost[lo] * rows) / (r.cost[lo + 1] - r.cost[lo]));
    const int pos = lo * rows + row, end = __shfl_down_sync(kFull, pos, 1);
    if (lane == 0 || lane == 2) {
        Stretch &w = r.stretch[lane >> 1][warp];
        w.pos = pos;
        w.end = end;
        w.unit = row == rows ? lo + 1 : lo;  // (a border at a unit's end)
        w.at = row == rows ? 0 : row;
        w.opened = 0;
    }
    __syncwarp();
}

// The weights' side of a product: kUp, pairs of rows (i, I + i) of W_gate_up, else rows
// [r0, r0 + L) of W_down. The line has r.n units (experts) of L rows; the warp takes stretches
// of it, a tile of up to kMost rows of one unit at a time, K group by K group. Tiles
// are told to the other side through the queue. What a step does not need lies in
// shared memory.
template <bool kUp>
struct Feed {
    static constexpr int kMost = kUp ? 8 : 16;
    int left;                // steps of the tile that are not asked for yet; 0: no more tiles
    int rows;                // rows of the tile from the lane's first on
    int wide;                // groups of a step
    uint32_t dst, off;       // the stage that the next copy goes to, the lane's piece in it
    const int8_t *src;       // the lane's piece of the tile's first row, at that step

    // `w`: the warp's stretch (cut_line).
    __device__ __forceinline__ Feed(const LayerArgs &a, Routes &r, Stretch &w, uint32_t ring, int r0,
                                    int L)
        : left(0), rows(0), wide(1), dst(ring), off(0), src(nullptr) {
        open(a, r, w, r0, L);
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) issue(a, r, w, ring, r0, L);
        __syncwarp();
    }
    // The next tile, if there is one.
    __device__ __forceinline__ void open(const LayerArgs &a, const Routes &r, Stretch &w, int r0,
                                         int L) {
        const int lane = threadIdx.x & 31;
        int n = min(w.end - w.pos, L - w.at);
        if (n <= 0) return;
        n = (n + (n - 1) / kMost) / ((n - 1) / kMost + 1);    // tiles of even height
        const int unit = w.unit, at = w.at;
        const int n_tok = r.first[unit + 1] - r.first[unit];
        const int K = kUp ? a.H : a.I;
        // (half a tile and the rest after it take fewer steps than 5/8 or 3/4 of one)
        if (n > kMost / 2 && n <= kMost * 3 / 4 && tile_groups<kUp>(kMost / 2, n_tok, K) > 1)
            n = kMost / 2;
        __syncwarp();
        if (lane == 0) {
            w.tile[w.opened & (kQueue - 1)] = make_int2(unit << 8 | n, at);
            ++w.opened;
            w.pos += n;
            w.at = at + n == L ? 0 : at + n;
            w.unit = at + n == L ? unit + 1 : unit;
        }
        __syncwarp();
        wide = tile_groups<kUp>(n, n_tok, K);
        left = (K >> 7) / wide;
        // a stage is 16 / wide rows of 128 wide bytes; the lane's first row and piece of it
        const int row = wide == 1 ? lane >> 3 : wide == 2 ? lane >> 4 : 0;
        const int piece = lane & (8 * wide - 1);
        off = row * 128 * wide + (swizzled(piece, row, wide) << 4);
        rows = n - row;
        const int64_t e = r.expert[unit];
        src = (kUp ? a.qw_up + (e * 2 * a.I + at + row) * a.H
                   : a.qw_down + (e * a.H + r0 + at + row) * a.I) + piece * 16;
    }
    // Asks for the next step's weights.
    __device__ __forceinline__ void issue(const LayerArgs &a, const Routes &r, Stretch &w,
                                          uint32_t ring, int r0, int L) {
        if (left > 0) {
            // the lane's rows are 4 / wide apart: 512 bytes of the stage (whose swizzle differs
            // by the row's bit 2, where a group is a step); the second two of W_gate_up are up
            const int K = kUp ? a.H : a.I;
            const int apart = 4 / wide;
            const int64_t third = kUp ? static_cast<int64_t>(a.I) * a.H : 2 * apart * K;
            const uint32_t to = dst + off, odd = wide == 1 ? to ^ 64 : to;
            if (rows > 0) cp_async_16(to, src);
            if (rows > apart) cp_async_16(odd + 512, src + apart * K);
            if (rows > (kUp ? 0 : 2 * apart)) cp_async_16(to + 1024, src + third);
            if (rows > (kUp ? apart : 3 * apart)) cp_async_16(odd + 1536, src + third + apart * K);
            src += 128 * wide;
            if (--left == 0) open(a, r, w, r0, L);
        }
        cp_async_commit();
        dst += kStageBytes;
        if (dst - ring >= kStages * kStageBytes) dst -= kStages * kStageBytes;
    }
};

// One step of the ring: waits for the stage at `read`, asks for one more.
template <bool kUp>
__device__ __forceinline__ uint32_t next_stage(const LayerArgs &a, Routes &r, Feed<kUp> &f,
                                               uint32_t ring, int r0, int L, uint32_t &read) {
    cp_async_wait<kStages - 2>();
    __syncwarp();                            // the stage is there; the one before is read
    f.issue(a, r, r.stretch[kUp ? 0 : 1][threadIdx.x >> 5], ring, r0, L);
    const uint32_t at = read;
    read = read + kStageBytes - ring >= kStages * kStageBytes ? ring : read + kStageBytes;
    return at;
}

// A tile of an expert with three and more tokens: 16 rows of weights by up to 8 NT tokens, over
// all of K. acc: [token tile][the lane's outputs: rows g and g + 8, tokens 2 c and 2 c + 1],
// g = lane / 4, c = lane % 4.
template <int NT, bool kUp>
__device__ __forceinline__ void tile_product(const LayerArgs &a, Routes &r, Feed<kUp> &f,
                                             uint32_t ring, int r0, int L, uint32_t &read,
                                             const int (&tok)[NT], const float *sw0,
                                             const float *sw1, float (&acc)[NT][4]) {
    const int lane = threadIdx.x & 31;
    // row lane / 4, 16-byte pieces 2 (lane % 4) and the next, swizzled by the row
    const uint32_t mine = (lane >> 2) * 128 + (((2 * (lane & 3)) ^ (lane >> 2)) << 4);
    const int8_t *codes = kUp ? a.xq : a.hq;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
    const int steps = (kUp ? a.H : a.I) >> 7;
    for (int s = 0; s < steps; ++s) {
        uint4 b[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                b[n][i] = reinterpret_cast<const uint4 *>(codes + tok[n] + s * 128)[i];
        const float w0 = sw0[s], w1 = sw1[s];
        const uint32_t at = next_stage(a, r, f, ring, r0, L, read) + mine;
        const uint4 lo[2] = {lds128(at), lds128(at ^ 16)};                      // row g
        const uint4 hi[2] = {lds128(at + 1024), lds128((at ^ 16) + 1024)};      // row g + 8
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            int p[4] = {};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mma_16832(p, lo[i].x, hi[i].x, lo[i].y, hi[i].y, b[n][i].x, b[n][i].y);
                mma_16832(p, lo[i].z, hi[i].z, lo[i].w, hi[i].w, b[n][i].z, b[n][i].w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[n][j] = fmaf(static_cast<float>(p[j]), j < 2 ? w0 : w1, acc[n][j]);
        }
    }
}

// Row `row` of a tile: the weight row's scales, its output.
template <bool kUp>
__device__ __forceinline__ const float *scales_of(const LayerArgs &a, int64_t e, int at, int r0,
                                                  int row, int rows) {
    if (!kUp) return a.sw_down + (e * a.H + r0 + at + min(row, rows - 1)) * (a.I >> 7);
    // rows 0-7 of gate, 8-15 of up
    return a.sw_up + (e * 2 * a.I + (row & 8 ? a.I : 0) + at + min(row & 7, rows - 1)) * (a.H >> 7);
}

template <int NT, bool kUp>
__device__ __forceinline__ void take_tile(const LayerArgs &a, Routes &r, Feed<kUp> &f, int unit,
                                          int row0, int rows, uint32_t ring, int r0, int L,
                                          uint32_t &read, int p0, int n_tok, float *s_d) {
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int64_t e = r.expert[unit];
    const int K = kUp ? a.H : a.I;
    int tok[NT];                             // where the lane's tokens' codes are
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        // (columns past the last token repeat it and are not stored)
        const int pair = r.pair[p0 + min(8 * n + g, n_tok - 1)];
        tok[n] = (kUp ? pair / a.k : pair) * K + q * 32;
    }
    float acc[NT][4];
    tile_product<NT, kUp>(a, r, f, ring, r0, L, read, tok,
                          scales_of<kUp>(a, e, row0, r0, g, rows),
                          scales_of<kUp>(a, e, row0, r0, g + 8, rows), acc);
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
                    a.h[static_cast<int64_t>(pair) * a.I + row0 + g] = h;
                }
                unsigned m = __float_as_uint(fabsf(h));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
                if (g == 0 && col < n_tok) atomicMax(a.hmax + pair, m);
            } else if (col < n_tok) {
                const float s = __fdiv_rn(__uint_as_float(a.hmax[pair]), 127.0f);
                float *d = s_d + pair * L + row0;
                if (g < rows) d[g] = __fmul_rn(acc[n][j], s);
                if (g + 8 < rows) d[g + 8] = __fmul_rn(acc[n][j + 2], s);
            }
        }
    }
}

// A tile of an expert with NT = 1 or 2 tokens, kWide groups a step: 2 kWide lanes have a row, 64
// bytes of it each.
template <int NT, int kWide, bool kUp>
__device__ __forceinline__ void take_tile_dot(const LayerArgs &a, Routes &r, Feed<kUp> &f, int unit,
                                              int row0, int rows, uint32_t ring, int r0, int L,
                                              uint32_t &read, int p0, float *s_d) {
    const int lane = threadIdx.x & 31;
    constexpr int kLanes = 2 * kWide, kRows = 16 / kWide;
    const int row = lane / kLanes, part = lane % kLanes;
    const int64_t e = r.expert[unit];
    const int K = kUp ? a.H : a.I;
    const int8_t *codes = kUp ? a.xq : a.hq;
    int tok[NT], pair[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        pair[n] = r.pair[p0 + n];
        tok[n] = (kUp ? pair[n] / a.k : pair[n]) * K + part * 64;
    }
    // (gate rows, then as many of up)
    const float *sw = kUp ? scales_of<kUp>(a, e, row0, r0, row % (kRows / 2) + (row / (kRows / 2)) * 8, rows)
                          : scales_of<kUp>(a, e, row0, r0, row, rows);
    // pieces 4 part .. 4 part + 3 of the row
    const uint32_t mine = row * 128 * kWide + (swizzled(4 * part, row, kWide) << 4);
    float acc[NT] = {};
    for (int s = 0; s < K >> 7; s += kWide) {
        uint4 b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                b[n][i] = reinterpret_cast<const uint4 *>(codes + tok[n] + s * 128)[i];
        float w[kWide];
#pragma unroll
        for (int i = 0; i < kWide; ++i) w[i] = sw[s + i];
        const uint32_t at = next_stage(a, r, f, ring, r0, L, read) + mine;
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = lds128(at ^ (i << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sum = __dp4a(static_cast<int>(q[i].x), static_cast<int>(b[n][i].x), sum);
                sum = __dp4a(static_cast<int>(q[i].y), static_cast<int>(b[n][i].y), sum);
                sum = __dp4a(static_cast<int>(q[i].z), static_cast<int>(b[n][i].z), sum);
                sum = __dp4a(static_cast<int>(q[i].w), static_cast<int>(b[n][i].w), sum);
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
#pragma unroll
            for (int i = 0; i < kWide; ++i) {        // the groups in order
                const int p = kWide == 1 ? sum : __shfl_sync(kFull, sum, 2 * i, kLanes);
                acc[n] = fmaf(static_cast<float>(p), w[i], acc[n]);
            }
        }
    }
    const bool first = part == 0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (kUp) {
            const float u = __fmul_rn(acc[n], a.sx[pair[n] / a.k]);
            const float h = swiglu_f32(u, __shfl_down_sync(kFull, u, 16));   // (lanes 0-15)
            const bool gate = lane < 16 && row < rows;
            if (gate && first) a.h[static_cast<int64_t>(pair[n]) * a.I + row0 + row] = h;
            const unsigned m = __reduce_max_sync(kFull, gate ? __float_as_uint(fabsf(h)) : 0u);
            if (lane == 0) atomicMax(a.hmax + pair[n], m);
        } else if (row < rows && first) {
            s_d[pair[n] * L + row0 + row] =
                __fmul_rn(acc[n], __fdiv_rn(__uint_as_float(a.hmax[pair[n]]), 127.0f));
        }
    }
}

// The warp's share of a product.
template <bool kUp>
__device__ __forceinline__ void product(const LayerArgs &a, Routes &r, Feed<kUp> &f, uint32_t ring,
                                        int L, int r0, float *s_d) {
    uint32_t read = ring;
    volatile Stretch &w = r.stretch[kUp ? 0 : 1][threadIdx.x >> 5];
    for (int taken = 0; taken < w.opened; ++taken) {
        const int2 tile = make_int2(w.tile[taken & (kQueue - 1)].x, w.tile[taken & (kQueue - 1)].y);
        const int unit = tile.x >> 8, rows = tile.x & 255;
        const int p0 = r.first[unit], n_tok = r.first[unit + 1] - p0;
        const int wide = tile_groups<kUp>(rows, n_tok, kUp ? a.H : a.I);
        if (n_tok == 1 && wide == 1)
            take_tile_dot<1, 1, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, s_d);
        else if (n_tok == 1 && wide == 2)
            take_tile_dot<1, 2, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, s_d);
        else if (n_tok == 1)
            take_tile_dot<1, 4, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, s_d);
        else if (n_tok == 2 && wide == 1)
            take_tile_dot<2, 1, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, s_d);
        else if (n_tok == 2 && wide == 2)
            take_tile_dot<2, 2, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, s_d);
        else if (n_tok == 2)
            take_tile_dot<2, 4, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, s_d);
        else if (n_tok <= 8)
            take_tile<1, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, n_tok, s_d);
        else if (n_tok <= 16)
            take_tile<2, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, n_tok, s_d);
        else
            take_tile<4, kUp>(a, r, f, unit, tile.y, rows, ring, r0, L, read, p0, n_tok, s_d);
    }
    cp_async_wait<0>();
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
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = code_plus_round(x[j], s, rcp, fast);
        const uint2 c = make_uint2(pack_code_bytes(f[0], f[1], f[2], f[3]),
                                   pack_code_bytes(f[4], f[5], f[6], f[7]));
        *reinterpret_cast<uint2 *>(a.hq + at) = c;
    }
}

__global__ void __launch_bounds__(kThreads, 1)
moe_layer_kernel(const LayerArgs a) {
    extern __shared__ __align__(128) uint8_t s_ring[];   // the rings, then s_d
    __shared__ Routes r;
    const int warp = threadIdx.x >> 5;
    const uint32_t ring = smem_u32(s_ring) + warp * kStages * kStageBytes;
    float *s_d = reinterpret_cast<float *>(s_ring + kRingBytes);     // [T k][L]
    // the CTA's output rows
    const int r0 = share(a.H, blockIdx.x, gridDim.x);
    const int L = share(a.H, blockIdx.x + 1, gridDim.x) - r0;
    make_routes(a, r);
    cut_line(r, a.I, blockIdx.x * kWarps + warp, gridDim.x * kWarps, L);
    {
        Feed<true> f(a, r, r.stretch[0][warp], ring, 0, a.I);
        product<true>(a, r, f, ring, a.I, 0, s_d);
    }
    __syncwarp();
    Feed<false> f(a, r, r.stretch[1][warp], ring, r0, L);
    bool ok = grid_wait(a.sync + 0, &r.abort, a.err, 0);
    if (ok) {
        quantize_h(a);
        ok = grid_wait(a.sync + 1, &r.abort, a.err, 1);
    }
    griddep_launch_dependents();
    if (!ok) {
        cp_async_wait<0>();
        return;
    }
    product<false>(a, r, f, ring, L, r0, s_d);
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * L; i += kThreads) {
        const int t = i / L, n = i - t * L;
        float acc = 0.0f;
        // (s_d is not written where there is no expert; a weight of 0 counts, as its d may not be finite)
        for (int j = t * a.k; j < (t + 1) * a.k; ++j)
            if (r.routed[j]) acc = fmaf(r.w[j], s_d[j * L + n], acc);
        const int64_t at = static_cast<int64_t>(t) * a.H + r0 + n;
        if (a.out_fp32)
            static_cast<float *>(a.y)[at] = acc;
        else
            static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(acc);
    }
}

struct FewLayout {
    size_t zeros, sx, xq, h, hq, total;
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
    l.zeros = take((kSyncs + n) * 4);
    l.sx = take(T * 4);
    l.xq = take(static_cast<size_t>(T) * H);
    l.h = take(n * I * 4);
    l.hq = take(n * I);
    l.total = off;
    return l;
}

size_t few_outputs_bytes(int64_t T, int64_t k, int64_t H, int num_sms) {
    return static_cast<size_t>(T * k) * ((H + num_sms - 1) / num_sms) * sizeof(float);
}

}  // namespace

bool uses_moe_few(int64_t T, int64_t k, int64_t H, int num_sms) {
    return T <= kMoeFewMaxTokens && T * k <= kMoeFewMaxPairs &&
           few_outputs_bytes(T, k, H, num_sms) <= kMaxOutputBytes;
}

size_t moe_few_workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I) {
    return few_layout(T, k, H, I).total;
}

MoeFewTokens moe_few_tokens(const MoeFewProblem &p) {
    const FewLayout l = few_layout(p.T, p.k, p.H, p.I);
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    MoeFewTokens t;
    t.x = p.x;
    t.ldx = p.ldx;
    t.T = static_cast<int>(p.T);
    t.H = static_cast<int>(p.H);
    t.vec = p.ldx % 8 == 0 && (reinterpret_cast<uintptr_t>(p.x) & 15) == 0;
    t.sx = reinterpret_cast<float *>(ws + l.sx);
    t.xq = reinterpret_cast<int8_t *>(ws + l.xq);
    t.zeros = reinterpret_cast<uint32_t *>(ws + l.zeros);
    t.n_zeros = static_cast<int>(kSyncs + p.T * p.k);
    return t;
}

cudaError_t launch_moe_few(const MoeFewProblem &p, int num_sms, cudaStream_t stream) {
    const FewLayout l = few_layout(p.T, p.k, p.H, p.I);
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    LayerArgs a;
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
    a.sync = reinterpret_cast<unsigned *>(ws + l.zeros);
    a.hmax = a.sync + kSyncs;
    a.sx = reinterpret_cast<const float *>(ws + l.sx);
    a.xq = reinterpret_cast<const int8_t *>(ws + l.xq);
    a.h = reinterpret_cast<float *>(ws + l.h);
    a.hq = reinterpret_cast<int8_t *>(ws + l.hq);
    cudaError_t e = device_error_word(&a.err);
    if (e != cudaSuccess) return e;
    static int attr_done[64] = {0};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        e = cudaFuncSetAttribute(moe_layer_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kRingBytes + kMaxOutputBytes);
        if (e != cudaSuccess) return e;
        attr_done[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(num_sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRingBytes + few_outputs_bytes(p.T, p.k, p.H, num_sms);
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
