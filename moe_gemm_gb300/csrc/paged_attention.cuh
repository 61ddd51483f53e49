// What the paged-attention kernels share: the cache's description, the copies
// of one tile of 128 positions through the block table, the workspace of
// divided items and the place of an output row.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_math.cuh"
#include "common.cuh"
#include "internal.h"
#include "paged_schedule.cuh"

namespace w8a8 {

// ------------------------------------------------------------- cache loading
struct PagedCache {
    const int32_t *table;   // [B, W]
    const float *ks, *vs;   // INT8: [P, Hkv, page]
    int W, P, Hkv, page;
    int box;                // rows of one TMA box: gcd(page, 128)
    int page_shift;         // log2 of page, -1: not a power of two
};

__device__ __forceinline__ int page_of(const PagedCache &c, int pos) {
    return c.page_shift >= 0 ? pos >> c.page_shift : pos / c.page;
}

// One tile of 128 positions of one (request, kv head) in shared memory: K and
// V rows of 128 bytes with the 128-byte swizzle (16-byte piece c of row r at
// piece c ^ (r & 7)); BF16 rows are two such halves, 64 dimensions each.
template <bool kInt8>
struct Tile {
    static constexpr int kHalves = kInt8 ? 1 : 2;
    static constexpr int kBytes = kHalves * kTilePositions * 128;   // of K, or of V
};

// Which positions of a tile hold keys of the request: bit i of word i / 32.
// Positions outside [lo, hi), and those of pages whose table entry is not a
// page, are masked for every query and not loaded.
struct TileMask {
    uint32_t w[4];
};

// Where a tile's boxes lie in the cache: lane i of the loading warp has box i.
struct TileBoxes {
    int64_t row;            // the lane's box: its first cache row
    bool use;               // the lane's box is loaded
    int used;               // boxes that are loaded
    TileMask mask;          // the same in every lane
};

// Finds the boxes of a tile through the block table (the whole warp calls it).
__device__ __forceinline__ TileBoxes find_boxes(const PagedCache &c, int b, int h, int tile, int lo,
                                                int hi, unsigned long long *err) {
    const int lane = threadIdx.x & 31;
    const int pos = tile * kTilePositions + lane * c.box;
    const int boxes = kTilePositions / c.box;
    bool use = lane < boxes && pos < hi && pos + c.box > lo;
    int64_t row = 0;
    if (use) {
        const int pg = page_of(c, pos);
        // (an ordinary load: the kernel that writes the table may run when this one starts)
        const int id = c.table[static_cast<int64_t>(b) * c.W + pg];
        if (id < 0 || id >= c.P) {
            use = false;
            record_device_error(err, KID_ATTN, ROLE_PRODUCER, 9);
        } else {
            row = (static_cast<int64_t>(id) * c.Hkv + h) * c.page + (pos - pg * c.page);
        }
    }
    const unsigned used = __ballot_sync(0xFFFFFFFFu, use);
    // the mask: lane l answers for positions 4 l .. 4 l + 3
    uint32_t nib = 0;
    const bool page_ok = (used >> (4 * lane / c.box)) & 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int p = tile * kTilePositions + 4 * lane + i;
        if (page_ok && p >= lo && p < hi) nib |= 1u << i;
    }
    uint32_t word = nib << (4 * (lane & 7));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) word |= __shfl_xor_sync(0xFFFFFFFFu, word, o);
    TileBoxes t;
    t.row = row;
    t.use = use;
    t.used = __popc(used);
#pragma unroll
    for (int i = 0; i < 4; ++i) t.mask.w[i] = __shfl_sync(0xFFFFFFFFu, word, 8 * i);
    return t;
}

// Issues the copies of a tile's K or V rows to dst (boxes that are not loaded
// leave whatever their shared memory held). They arrive at `bar`, which the
// caller has told to expect tile_bytes().
template <bool kInt8>
__device__ __forceinline__ void copy_boxes(const PagedCache &c, const TileBoxes &t,
                                           const CUtensorMap *map, uint32_t dst, uint32_t bar) {
    if (!t.use) return;
    const uint32_t off = static_cast<uint32_t>((threadIdx.x & 31) * c.box) * 128;
#pragma unroll
    for (int half = 0; half < Tile<kInt8>::kHalves; ++half)
        tma_load_2d(dst + off + half * kTilePositions * 128, map, half * 64,
                    static_cast<int>(t.row), bar);
}

// The same of the INT8 vectors' scales.
__device__ __forceinline__ void copy_scales(const PagedCache &c, const TileBoxes &t,
                                            const float *scales, uint32_t dst, uint32_t bar) {
    if (!t.use) return;
    bulk_g2s(dst + (threadIdx.x & 31) * c.box * 4, scales + t.row, c.box * 4, bar);
}

template <bool kInt8>
__device__ __forceinline__ uint32_t tile_bytes(const PagedCache &c, const TileBoxes &t) {
    return static_cast<uint32_t>(t.used * c.box) * (kInt8 ? 128 : 256);
}
__device__ __forceinline__ uint32_t scale_bytes(const PagedCache &c, const TileBoxes &t) {
    return static_cast<uint32_t>(t.used * c.box) * 4;
}

// The positions of a request that any of its new tokens may see: nothing
// outside them is read.
__device__ __forceinline__ void request_span(const PagedSchedule &s, const PagedRequest &r, int &lo,
                                             int &hi) {
    lo = s.window > 0 ? max(max(r.base, 0) - s.window + 1, 0) : 0;
    hi = r.kv;
}

// ------------------------------------------------------------------ workspace
// Of every CTA two slots; a slot holds, of up to `rows` query rows, the sums
// sum_j 2^(t_j - m) v_j (rows x 128; t: scores in log2 units), then m, then
// sum_j 2^(t_j - m).
__device__ __forceinline__ float *slot_of(float *ws, int rows, int cta, int slot) {
    return ws + (static_cast<int64_t>(cta) * 2 + slot) * rows * (kHeadDim + 2);
}
// After the slots of `ctas` CTAs, the cuts.
__host__ __device__ inline PagedCut *cuts_of(float *ws, int rows, int ctas) {
    return reinterpret_cast<PagedCut *>(ws + static_cast<int64_t>(ctas) * 2 * rows * (kHeadDim + 2));
}

// The largest |x| of 8 BF16 values, as bits (attention_math.cuh: finite_bits2).
__device__ __forceinline__ uint32_t finite_amax8(const uint4 &v) {
    const uint32_t m = __vmaxu2(__vmaxu2(finite_bits2(v.x), finite_bits2(v.y)),
                                __vmaxu2(finite_bits2(v.z), finite_bits2(v.w)));
    return max(m & 0xFFFFu, m >> 16);
}

// The attention kernels work in log2 units.
constexpr float kLog2e = 1.4426950408889634f;

struct PagedOut {
    void *out;              // [T, Hq, 128]
    int fp32, Hq, G;
};

__device__ __forceinline__ int64_t out_row(const PagedOut &o, const PagedRequest &r, int h,
                                           int tok0, int row) {
    return (static_cast<int64_t>(r.t0) + tok0 + row / o.G) * o.Hq + h * o.G + row % o.G;
}

struct PagedSetup {
    PagedSchedule s;
    PagedCache c;
    PagedOut o;
};

// Fills the parts that depend on the call alone; `rows` query rows per item.
PagedSetup paged_setup(const PagedAttnProblem &p, int rows);

// A tensor map over the cache as rows of 128 bytes or BF16 values, a box of
// 128 bytes x `box` rows.
bool paged_encode_cache(CUtensorMap *map, const void *ptr, bool int8, const PagedAttnProblem &p,
                        int box);

// The tiles kernel (paged_attention_tiles.cu): 256 query rows per item on the
// tcgen05 tensor cores. Its workspace slots have kPagedTileRows rows and it
// runs kPagedTileCtas CTAs at most.
constexpr int kPagedTileRows = 256;
constexpr int kPagedTileCtas = 160;
cudaError_t launch_paged_tiles(const PagedAttnProblem &p, const PagedSetup &u, int ctas,
                               unsigned long long *err, cudaStream_t stream);

}  // namespace w8a8
