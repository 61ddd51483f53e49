// Attention over the paged cache for calls with many query rows, on the
// tcgen05 tensor cores of sm_103a (the operator: paged_attention.cu).
//
// An item is 256 query rows of one (request, kv head): two halves of 128 rows
// (whole tokens x the G query heads that share the kv head), whose products
// alternate on the tensor core so that one half's softmax runs beside the
// other half's products. Per tile of 128 positions and half:
//
//   S = Q K^T         128 x 128 x 128, both operands in shared memory
//   softmax           one thread per row: S from tensor memory, running
//                     maximum and sum, P back to tensor memory over S
//   O += P V          128 x 128 x 128, P from tensor memory, V as it lies
//                     (N-major), O stays in tensor memory for the whole item
//
// Tensor memory: S0, S1, O0, O1 of 128 columns each (all 512).
//
// The reference m of the exponentials p_j = 2^(t_j - m) (t: scores in log2 units)
// is a maximum that was seen, not the running one: it stays while the tile's
// sums show that no weight passes 2^8, so most tiles take no maximum at all, and
// O is rescaled a few times per item instead of at every tile (rescaling only past a
// threshold is a published method for attention on this generation). Weights above 1
// cost no accuracy. Sums and statistics are FP32.
//
// BF16 pages: P is rounded to BF16 for the product (half a step 2^-8 of each
// weight; V is BF16, and both operands have one type).
// INT8 pages: a converter warpgroup widens the codes to fp16 (exact) into
// shared memory. Scores are S * (k scale); a weight carries its v scale,
// P_j = p_j * vs_j * 2^-e, rounded to fp16 (half a step 2^-11). e follows the
// largest v scale s of the tiles, up and down, to within 2^3: P stays below 2^12, and a
// weight loses no more than 2^-25 2^e <= 2^-22 s in fp16's subnormals. So a vector
// far larger than the rest costs the other vectors of its own tile their bits, whether or
// not a row gives it weight. O is in units of 2^e.
// q goes to fp16 too, scaled by one power of two per item, which the k scales
// take back exactly.
//
// The softmax warps read S in the layout of 16 x 256 bits: a thread has 4 rows
// and 2 of every 8 columns, so the per-column scales are read from shared memory
// once for 4 rows (a row per thread reads them for one: the reads alone then
// took longer than the products).
//
// What bounds it. BF16 pages: eight prompts of up to 8192 tokens (1.45e12 operations)
// take 1.12 ms, 1.29 PFLOP/s, and 1.17 after half a second of such calls, when the power
// limit holds the SMs at 1.97 GHz instead of 2.07: 2.0 us per tile and SM, of which the products are 1.3 (an
// S of 64 columns reads as many bytes of Q as one of 128, 48 cycles for 32); the
// rest is what a half waits for the hand-over between its softmax and its products, and
// some 5 us per item for its start and end. With the scores in one part of 128 columns
// the softmax waited for whole products: 1.44 ms. INT8 pages: 2048 tokens over 30001
// positions and eight single tokens (2.08e12) take 2.01 ms, 1.04 PFLOP/s; without the
// widening of codes they would take 1.87, without the scales' part of the softmax as
// well 1.69. BF16 pages of the same call take 1.47.
//
// A wait that gives up is voted on by the warp: its lanes go on to votes and shuffles
// of all of them, so they must leave together.
//
// Warps: 0-3 and 4-7 softmax of the halves, 8 and 10 issue the halves'
// products, 9 loads, 11 walks the CTA's share, 12-15 convert (INT8).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_math.cuh"
#include "common.cuh"
#include "internal.h"
#include "paged_attention.cuh"
#include "paged_schedule.cuh"
#include "quant_math.cuh"
#include "tensor_map.h"

namespace w8a8 {
namespace {

constexpr int kThreads = 512;
constexpr int kHalfRows = 128;
constexpr int kInfo = 4;             // tiles whose mask and scales are kept
constexpr float kMaxWeight = 256.0f; // sums of a tile's weights that move the reference
constexpr int kOperandBytes = 128 * 128 * 2;
// Registers of a softmax thread and of the others: together 256 for a pair, 2 x 128
// pairs = the 512 x 128 that the block is launched with. Measured: INT8, whose
// converters want more, 2.05 ms with 160 / 96 then (2.10 with 168 / 88, 2.16 with 152 /
// 104); BF16 1.11 ms with 168 / 88 (1.13 with 160 / 96).
template <bool kInt8>
struct Regs {
    static constexpr uint32_t kSoftmax = kInt8 ? 160 : 168, kOther = 256 - kSoftmax;
};

struct TilesArgs {
    PagedSchedule s;
    PagedCache c;
    PagedOut o;
    int half_tokens;        // whole tokens of a half: 128 / G
    float scale_log2;       // softmax scale * log2(e)
    float *ws;
    unsigned long long *err;
};

// A piece of an item, as the warps take it from shared memory. Warp 11 walks the
// line ahead of the others (two 64-bit divisions and a walk step per piece: in each
// of the 15 warps, between two items, they took 2000 to 4000 cycles).
struct TilePiece {
    int b, h, t0, base, kv;             // the request: block table row, kv head, first row, ...
    int tok0, ntok, tile0, first, last; // paged_schedule.cuh: PagedPiece
    int whole, slot;
    int lo;                             // positions below it are masked for every token
    int end;                            // no piece: the share ends
};
constexpr int kPieces = 4;              // pieces that warp 11 is ahead at most
constexpr int kTakers = 15;             // warps that take them

// A tile's scores come in two halves of 64 columns, so that one is ready while the
// softmax is at the other (packed prompts of 16 thousand tokens, BF16: 1.44 -> 1.17
// ms). INT8 neither gains nor loses by it (a chunk over 30001 positions takes 2.1 ms
// either way) and has it for the one form of the products. A tile moves some 250 KB of
// operands, 100 of conversion and 130 of scales through shared memory there; leaving
// out the latter two saves 16 %, so its bandwidth alone is not the bound.
constexpr int kN = 2, kCols = kTilePositions / kN;

template <bool kInt8>
struct TilesSmem {
    // BF16 operands are copied straight into 5 slots; INT8 codes land in 3 raw
    // slots and are widened into 3.
    static constexpr int kOps = kInt8 ? 3 : 5;
    static constexpr int kRaws = 3;
    uint8_t q[2][kOperandBytes];
    uint8_t op[kOps][kOperandBytes];
    uint8_t raw[kInt8 ? kRaws : 1][kInt8 ? kOperandBytes / 2 : 16];
    float rks[kInfo][kInt8 ? 128 : 4], rvs[kInfo][kInt8 ? 128 : 4];   // scales as stored
    // of two columns: what a score is multiplied by (to log2 units), then what
    // its weight is; both 0 where the position is masked for every query
    float4 col[kInfo][kInt8 ? 64 : 1];
    float unit[kInfo];                   // 2^e
    uint32_t qmax[4];
    TileMask mask[kInfo];
    uint64_t op_full[kOps], op_empty[kOps], raw_full[kRaws], raw_empty[kRaws];
    uint64_t info_full[kInfo];
    uint64_t q_land[2], q_full[2], q_empty[2];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];   // of a half of the rows, a part of a tile
    uint64_t o_free[2];
    uint64_t q_max, fix, drain[2];
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    TilePiece piece[kPieces];
    uint32_t tmem;
    volatile int abort_flag;
};

// Shared-memory operand descriptors, all with the 128-byte swizzle and 8-row
// groups 1024 bytes apart: the upper word is one constant, the lower word the
// address and the leading offset, in units of 16 bytes. One thread issues every
// product, so what it computes per instruction counts: with whole descriptors
// built from addresses an instruction took 140 cycles to issue, against the 64
// that the tensor core needs for it.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_kmajor(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
// N-major: rows of k (128 bytes: 64 values of n); the next 64 values of n lie
// half an operand further (leading offset).
__device__ __forceinline__ uint32_t desc_nmajor(uint32_t saddr) {
    return (saddr >> 4) | (static_cast<uint32_t>(kOperandBytes / 2 / 16) << 16);
}

// D[tmem] (+)= A * B, kind::f16, cta_group::1; A from shared memory or from
// tensor memory.
template <bool kAccumulate>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "n"(kAccumulate ? 1 : 0), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n"
        " mov.b64 db, {%2, %5};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
constexpr uint32_t kBNMajor = 1u << 16;   // instruction descriptor: B is N-major

#define W8A8_O16(r)                                                                            \
    "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),         \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),              \
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
#define W8A8_IO16(r)                                                                           \
    "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),         \
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),              \
        "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
#define W8A8_I16(r, o)                                                                          \
    "r"(r[o + 0]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]),   \
        "r"(r[o + 6]), "r"(r[o + 7]), "r"(r[o + 8]), "r"(r[o + 9]), "r"(r[o + 10]),             \
        "r"(r[o + 11]), "r"(r[o + 12]), "r"(r[o + 13]), "r"(r[o + 14]), "r"(r[o + 15])

constexpr uint32_t kLane16 = 16u << 16;   // tensor-memory address of lane 16

// 32 columns of the warp's 32 lanes as two blocks of 16 lanes: lane l of the warp
// gets, of the lanes l / 4 (registers 4 i, 4 i + 1) and l / 4 + 8 (4 i + 2, 4 i +
// 3) of each block, columns 8 i + 2 (l % 4) and the one after it. Asynchronous:
// valid after tmem_wait_tile on the same registers.
__device__ __forceinline__ void tmem_ld_tile(uint32_t t, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : W8A8_O16(a)
        : "r"(t)
        : "memory");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : W8A8_O16(b)
        : "r"(t + kLane16)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_tile(uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : W8A8_IO16(a), W8A8_IO16(b) : : "memory");
}
__device__ __forceinline__ void tmem_st_tile(uint32_t t, const uint32_t (&a)[16],
                                             const uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::W8A8_I16(a, 0),
        "r"(t)
        : "memory");
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::W8A8_I16(b, 0),
        "r"(t + kLane16)
        : "memory");
}
// 16-bit pairs into 16 lanes: register 2 i + j is column 4 i + l % 4 of lane l / 4 +
// 8 j.
__device__ __forceinline__ void tmem_st_p(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::W8A8_I16(r, 0),
        "r"(t)
        : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ unsigned long long f2_fma(unsigned long long a, unsigned long long b,
                                                     unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// What hides keys of a part of a tile from a thread's rows: of row k, the
// columns 8 i + 2 (l % 4) + e with 8 i + e in [lo[k], hi[k]] are seen, and those whose
// bit in the mask (shifted by 2 (l % 4)) is set.
struct RowMask {
    int lo[4], hi[4];
    uint32_t w[2];
};

__device__ __forceinline__ bool hidden(const RowMask &m, int k, int c) {
    return c > m.hi[k] || c < m.lo[k] || !((m.w[c >> 5] >> (c & 31)) & 1u);
}

// The mask as values that only the masked form of a loop can use: the compiler
// otherwise works out all of a tile's comparisons ahead of the choice between the
// forms, for tiles without a mask too (measured: twice the time of a long chunk).
__device__ __forceinline__ RowMask here(RowMask m) {
#pragma unroll
    for (int k = 0; k < 4; ++k) asm volatile("" : "+r"(m.lo[k]), "+r"(m.hi[k]));
    asm volatile("" : "+r"(m.w[0]), "+r"(m.w[1]));
    return m;
}

// A part's weights of a thread's 4 rows (row k: lanes l / 4 + 8 (k & 1) of
// block k >> 1) against the references -nm, as P's register image, and their
// sums by row.
template <bool kInt8, bool kMasked>
__device__ __forceinline__ void weigh(uint32_t ts, const float4 *col, float c,
                                      const float (&nm)[4], const RowMask &mask,
                                      uint32_t (&pk)[2][32 / kN], float (&sum)[4]) {
    RowMask mk;
    if constexpr (kMasked) mk = here(mask);
    unsigned long long l2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) l2[k] = f2_bits(0.0f, 0.0f);
#pragma unroll
    for (int cc = 0; cc < 4 / kN; ++cc) {
        uint32_t r[2][16];
        tmem_ld_tile(ts + cc * 32, r[0], r[1]);
        tmem_wait_tile(r[0], r[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 f = make_float4(c, c, 1.0f, 1.0f);
            if constexpr (kInt8) f = col[(cc * 4 + i) * 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t(&x)[16] = r[k >> 1];
                const int o = 4 * i + 2 * (k & 1);
                float p0, p1;
                f2_split(f2_fma(f2_bits(__uint_as_float(x[o]), __uint_as_float(x[o + 1])),
                                f2_bits(f.x, f.y), f2_bits(nm[k], nm[k])),
                         p0, p1);
                if constexpr (kMasked) {
                    const int cl = cc * 32 + i * 8;
                    if (hidden(mk, k, cl)) p0 = -INFINITY;
                    if (hidden(mk, k, cl + 1)) p1 = -INFINITY;
                }
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                unsigned long long p2 = f2_bits(p0, p1);
                l2[k] = f2_add(l2[k], p2);
                uint32_t &out = pk[k >> 1][(cc * 4 + i) * 2 + (k & 1)];
                if constexpr (kInt8) {
                    f2_split(f2_mul(p2, f2_bits(f.z, f.w)), p0, p1);
                    out = pack_f16x2(p0, p1);
                } else {
                    out = pack_bf16x2(p0, p1);
                }
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, b;
        f2_split(l2[k], a, b);
        sum[k] = a + b;
    }
}

// The largest score of each of a thread's rows in a tile (log2 units; the same
// in the 4 lanes that share the rows).
template <bool kInt8, bool kMasked>
__device__ __forceinline__ void row_max(uint32_t ts, const float4 *col, float c, const RowMask &mask,
                                        float (&top)[4]) {
    RowMask mk;
    if constexpr (kMasked) mk = here(mask);
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = -INFINITY;
#pragma unroll 1
    for (int cc = 0; cc < 4 / kN; ++cc) {
        uint32_t w = 0;
        if constexpr (kMasked) w = cc == 0 ? mk.w[0] : mk.w[1];
        uint32_t r[2][16];
        tmem_ld_tile(ts + cc * 32, r[0], r[1]);
        tmem_wait_tile(r[0], r[1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 f = make_float4(c, c, 1.0f, 1.0f);
            if constexpr (kInt8) f = col[(cc * 4 + i) * 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int o = 4 * i + 2 * (k & 1);
                float p0 = __uint_as_float(r[k >> 1][o]) * f.x;
                float p1 = __uint_as_float(r[k >> 1][o + 1]) * f.y;
                if constexpr (kMasked) {
                    const int cl = i * 8;
                    const int hi = mk.hi[k] - cc * 32, lo = mk.lo[k] - cc * 32;
                    if (cl > hi || cl < lo || !((w >> cl) & 1u)) p0 = -INFINITY;
                    if (cl + 1 > hi || cl + 1 < lo || !((w >> (cl + 1)) & 1u)) p1 = -INFINITY;
                }
                top[k] = fmaxf(top[k], fmaxf(p0, p1));
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], 1));
        top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], 2));
    }
}

// 4 x 4 transpose over the four lanes of a quad: lane q's v[i] becomes lane i's
// v[q].
__device__ __forceinline__ void quad_transpose(uint32_t (&v)[4], int quad) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const bool up = (quad & o) != 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & o) continue;
            const uint32_t give = up ? v[i] : v[i | o];
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, o);
            if (up) v[i] = got;
            else v[i | o] = got;
        }
    }
}

// O (in tensor memory) times a factor per row.
__device__ __forceinline__ void scale_rows(uint32_t to, const float (&f)[4]) {
#pragma unroll 1
    for (int cc = 0; cc < 4; ++cc) {
        uint32_t r[2][16];
        tmem_ld_tile(to + cc * 32, r[0], r[1]);
        tmem_wait_tile(r[0], r[1]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                r[h][j] = __float_as_uint(__uint_as_float(r[h][j]) * f[2 * h + ((j >> 1) & 1)]);
        tmem_st_tile(to + cc * 32, r[0], r[1]);
    }
}

// 16-byte piece j of row r of q in shared memory.
__device__ __forceinline__ uint4 *q_piece(uint8_t *q, int r, int j) {
    return reinterpret_cast<uint4 *>(q + (j >> 3) * (kOperandBytes / 2) + r * 128 +
                                     (((j & 7) ^ (r & 7)) << 4));
}

// The tiles that a half of an item sees within a piece: [from, upto), in tiles
// of the request.
struct HalfTiles {
    bool exists;
    int first, last;        // positions of its first and last token
    int from, upto;
};

__device__ __forceinline__ HalfTiles half_tiles(const PagedSchedule &s, const TilePiece &p, int half,
                                                int half_tokens) {
    HalfTiles t;
    const int a = half * half_tokens, z = min(a + half_tokens, p.ntok);
    t.exists = a < p.ntok;
    t.first = p.base + p.tok0 + a;
    t.last = p.base + p.tok0 + z - 1;
    const int lo = s.window > 0 ? max(max(t.first, 0) - s.window + 1, 0) / kTilePositions : 0;
    const int hi = t.last >= 0 ? t.last / kTilePositions + 1 : 0;
    t.from = max(p.tile0 + p.first, lo);
    t.upto = t.exists ? min(p.tile0 + p.last, hi) : t.from;
    if (t.upto < t.from) t.upto = t.from;
    return t;
}

// The rows of a half that are the item's: the copy of q always brings half_tokens
// tokens, and in a request's last item those after its own are another request's, or
// nobody's, and may hold anything. They become zeros, so that what rows decide together
// (the scaling of INT8 pages' q, when references move) does not depend on them.
__device__ __forceinline__ int own_rows(const TilePiece &p, int half, int half_tokens, int G) {
    return min(p.ntok - half * half_tokens, half_tokens) * G;
}

template <bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
paged_tiles_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                   const __grid_constant__ CUtensorMap vm, const TilesArgs a) {
    extern __shared__ uint8_t smem_raw[];
    using Smem = TilesSmem<kInt8>;
    constexpr uint32_t kOps = Smem::kOps, kRaws = Smem::kRaws;
    Smem &sm = *reinterpret_cast<Smem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedSchedule &s = a.s;
    volatile int *abort = &sm.abort_flag;
    auto bar = [](uint64_t &b) { return smem_u32(&b); };
    if (tid == 0) {
        for (uint32_t i = 0; i < kOps; ++i) {
            mbar_init(bar(sm.op_full[i]), kInt8 ? 128 : 1);
            mbar_init(bar(sm.op_empty[i]), 2);   // one arrival per half
        }
        for (uint32_t i = 0; i < kRaws; ++i) {
            mbar_init(bar(sm.raw_full[i]), 1);
            mbar_init(bar(sm.raw_empty[i]), 128);
        }
        for (int i = 0; i < kInfo; ++i) mbar_init(bar(sm.info_full[i]), kInt8 ? 128 : 1);
        for (int h = 0; h < 2; ++h) {
            mbar_init(bar(sm.q_land[h]), 1);
            mbar_init(bar(sm.q_full[h]), kInt8 ? 128 : 1);
            mbar_init(bar(sm.q_empty[h]), 1 + kHalfRows);
            for (int e = 0; e < 2; ++e) {
                mbar_init(bar(sm.s_full[h][e]), 1);
                mbar_init(bar(sm.p_full[h][e]), kHalfRows);
                mbar_init(bar(sm.pv_done[h][e]), 1);
            }
            mbar_init(bar(sm.o_free[h]), kHalfRows);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(sm.piece_full[i]), 1);
            mbar_init(bar(sm.piece_empty[i]), kInt8 ? kTakers : kTakers - 4);
        }
        mbar_init(bar(sm.q_max), 128);
        mbar_init(bar(sm.fix), 1);
        mbar_init(bar(sm.drain[0]), 1);
        mbar_init(bar(sm.drain[1]), 1);
        sm.abort_flag = 0;
        fence_mbarrier_init();
    }
    // rows of q past a half's whole tokens are never written: zeros, so that
    // what is computed for them stays finite
    for (int i = tid; i < 2 * kOperandBytes / 16; i += kThreads)
        reinterpret_cast<uint4 *>(sm.q)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == 8) {
        tmem_alloc(smem_u32(&sm.tmem), 512);
        tmem_relinquish();
    }
    griddep_launch_dependents();
    griddep_wait();
    const PagedShare sh = paged_share<kThreads>(s, blockIdx.x, gridDim.x);   // (synchronises)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    PagedWalk w;
    w.start(s, sh);
    if (tid == kThreads - 1)
        paged_write_cut(s, sh, w, blockIdx.x, cuts_of(a.ws, kPagedTileRows, gridDim.x));
    const bool mine = static_cast<int>(blockIdx.x) < sh.ctas;
    // The next piece (the whole warp calls it); false: there is none, or a wait gave up.
    uint32_t taken = 0;
    auto take = [&](TilePiece &p, bool &ok, unsigned role) -> bool {
        const int i = taken % kPieces;
        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar(sm.piece_full[i]), (taken / kPieces) & 1, abort,
                                                     a.err, role, 10, kWaitLimitNs, KID_ATTN));
        if (!ok) return false;
        p = sm.piece[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.piece_empty[i]));
        ++taken;
        return p.end == 0;
    };
    uint32_t it = 0;        // tiles of the pieces before this one
    uint32_t qn[2] = {0, 0};   // pieces with the half before this one

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        setmaxnreg_inc<Regs<kInt8>::kSoftmax>();
        const int h = warp >> 2;
        const int quad = lane & 3, r4 = (warp & 3) * 32 + (lane >> 2);
        int tok4[4];        // the tokens, within the half, of the thread's rows r4 + 8 k
#pragma unroll
        for (int k = 0; k < 4; ++k) tok4[k] = (r4 + 8 * k) / a.o.G;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // lane 32 (warp % 4)
        const uint32_t ts = tmem + lanes + h * 128, to = tmem + lanes + 256 + h * 128;
        uint32_t sn = 0;            // active tiles
        bool ok = true;
        TilePiece p;
        while (mine && take(p, ok, ROLE_EPILOGUE)) {
            const bool work = p.last > p.first;
            const HalfTiles t = half_tiles(s, p, h, a.half_tokens);
            if (work && t.exists) {
                ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar(sm.q_full[h]), qn[h] & 1, abort, a.err,
                                                             ROLE_EPILOGUE, 1, kWaitLimitNs, KID_ATTN));
                mbar_arrive(bar(sm.q_empty[h]));
                ++qn[h];
            }
            float m[4], l[4];
            int pos[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m[k] = -INFINITY;
                l[k] = 0.0f;
                pos[k] = t.first + tok4[k];
            }
            float unit = 0.0f;
            bool first = true;
            for (int x = t.from; work && ok && x < t.upto; ++x, ++sn) {
                const uint32_t ti = it + static_cast<uint32_t>(x - p.tile0 - p.first);
                const int info = ti % kInfo;
#pragma unroll 1
                for (int e = 0; e < kN; ++e) {
                    // (in this order: a half that passes over tiles would not
                    // know which of two phases an earlier info slot is in)
                    ok = __all_sync(0xFFFFFFFFu,
                                    ok &&
                                        mbar_wait(bar(sm.s_full[h][e]), sn & 1, abort, a.err,
                                                  ROLE_EPILOGUE, 2, kWaitLimitNs, KID_ATTN) &&
                                        mbar_wait(bar(sm.info_full[info]), (ti / kInfo) & 1, abort,
                                                  a.err, ROLE_EPILOGUE, 3, kWaitLimitNs, KID_ATTN));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t tse = ts + e * kCols;
                    const int c0 = x * kTilePositions + e * kCols;
                    RowMask mk;
                    mk.w[0] = sm.mask[info].w[2 * e];
                    mk.w[1] = sm.mask[info].w[2 * e + 1];
                    const bool masked = c0 + kCols - 1 > t.first ||
                                        (s.window > 0 && c0 <= t.last - s.window) ||
                                        (mk.w[0] & mk.w[1]) != 0xFFFFFFFFu;
                    mk.w[0] >>= 2 * quad;
                    mk.w[1] >>= 2 * quad;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mk.hi[k] = pos[k] - c0 - 2 * quad;
                        mk.lo[k] = s.window > 0 ? mk.hi[k] - s.window + 1 : -kTilePositions;
                    }
                    const float4 *col = kInt8 ? &sm.col[info][e * (kCols / 2) + quad] : nullptr;
                    bool move = m[0] == -INFINITY || m[1] == -INFINITY || m[2] == -INFINITY ||
                                m[3] == -INFINITY;
                    float turn = 1.0f;          // change of O's unit
                    if constexpr (kInt8) {
                        const float un = sm.unit[info];
                        if (un != unit && !first) turn = unit / un;
                        unit = un;
                    }
                    // Before O is rescaled, the output product of the part before has to
                    // be done (those before that are: this part's scores came after).
                    auto settle = [&]() {
                        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar(sm.pv_done[h][e ^ 1]), (sn + e + 1) & 1,
                                                                     abort, a.err, ROLE_EPILOGUE, 5,
                                                                     kWaitLimitNs, KID_ATTN));
                        tc_fence_after();
                    };
                    uint32_t pk[2][32 / kN];
                    float sum[4];
                    for (bool again = false;; again = true) {
                        if (__any_sync(0xFFFFFFFFu, move)) {
                            // new references: the part's maxima
                            float top[4], f[4];
                            if (masked) row_max<kInt8, true>(tse, col, a.scale_log2, mk, top);
                            else row_max<kInt8, false>(tse, col, a.scale_log2, mk, top);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                f[k] = turn;
                                if (top[k] > m[k]) {
                                    const float alpha = ex2_approx(m[k] - top[k]);
                                    f[k] *= alpha;
                                    l[k] *= alpha;
                                    m[k] = top[k];
                                }
                            }
                            if (!first) {
                                settle();
                                scale_rows(to, f);
                            }
                            turn = 1.0f;
                            again = true;
                        }
                        float nm[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) nm[k] = m[k] == -INFINITY ? 0.0f : -m[k];
                        if (masked) weigh<kInt8, true>(tse, col, a.scale_log2, nm, mk, pk, sum);
                        else weigh<kInt8, false>(tse, col, a.scale_log2, nm, mk, pk, sum);
                        if (again) break;
                        move = !(fmaxf(fmaxf(sum[0], sum[1]), fmaxf(sum[2], sum[3])) <= kMaxWeight);
                        if (!__any_sync(0xFFFFFFFFu, move)) break;
                    }
                    if (turn != 1.0f) {
                        const float f[4] = {turn, turn, turn, turn};
                        settle();
                        scale_rows(to, f);
                    }
                    first = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) l[k] += sum[k];
                    tmem_st_p(tse, pk[0]);
                    tmem_st_p(tse + kLane16, pk[1]);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(bar(sm.p_full[h][e]));
                }
            }
            if (work) it += static_cast<uint32_t>(p.last - p.first);
            // ---- the item's (or the share's) result of this row
            const bool any = work && t.upto > t.from;
            if (any) {
                // the last output products (sn counts this piece's tiles already)
                ok = __all_sync(0xFFFFFFFFu, ok &&
                                                 mbar_wait(bar(sm.pv_done[h][0]), (sn - 1) & 1, abort, a.err,
                                                           ROLE_EPILOGUE, 4, kWaitLimitNs, KID_ATTN) &&
                                                 mbar_wait(bar(sm.pv_done[h][1]), (sn - 1) & 1, abort, a.err,
                                                           ROLE_EPILOGUE, 6, kWaitLimitNs, KID_ATTN));
            }
            if (!ok) break;
            tc_fence_after();
            if (t.exists) {
                float f[4];
                int64_t at[4];      // of the rows: where they go, < 0: nowhere
                float *part = slot_of(a.ws, kPagedTileRows, blockIdx.x, p.slot);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 1);
                    l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 2);
                    const int row = r4 + 8 * k, tok = tok4[k];
                    const int irow = h * a.half_tokens * a.o.G + row;   // the item's row
                    f[k] = kInt8 ? unit : 1.0f;
                    at[k] = -1;
                    if (tok >= a.half_tokens || h * a.half_tokens + tok >= p.ntok) continue;
                    if (p.whole) {
                        f[k] *= l[k] == 0.0f ? 0.0f : 1.0f / l[k];
                        at[k] = ((static_cast<int64_t>(p.t0) + p.tok0 + h * a.half_tokens + tok) * a.o.Hq +
                                 static_cast<int64_t>(p.h) * a.o.G + (row - tok * a.o.G)) * kHeadDim;
                    } else {
                        at[k] = static_cast<int64_t>(irow) * kHeadDim;
                        if (quad == 0) {
                            part[kPagedTileRows * kHeadDim + irow] = m[k];
                            part[kPagedTileRows * (kHeadDim + 1) + irow] = l[k];
                        }
                    }
                }
                const bool wide = !p.whole || a.o.fp32;
                float *base = p.whole ? static_cast<float *>(a.o.out) : part;
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t r[2][16];
                    if (any) {
                        tmem_ld_tile(to + cc * 32, r[0], r[1]);
                        tmem_wait_tile(r[0], r[1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[0][j] = r[1][j] = 0u;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x0 = __uint_as_float(r[k >> 1][4 * i + 2 * (k & 1)]) * f[k];
                            const float x1 = __uint_as_float(r[k >> 1][4 * i + 2 * (k & 1) + 1]) * f[k];
                            if (wide) {
                                if (at[k] >= 0)
                                    *reinterpret_cast<float2 *>(base + at[k] + cc * 32 + i * 8 + 2 * quad) =
                                        make_float2(x0, x1);
                            }
                            v[i] = pack_bf16x2(x0, x1);
                        }
                        // the four lanes of a row change columns 8 i + 2 q of each i
                        // for the 8 columns of i = q: 16 bytes to store
                        quad_transpose(v, quad);
                        if (!wide && at[k] >= 0)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o.out) + at[k] + cc * 32 +
                                                       quad * 8) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                    __syncwarp();
                }
                if (any) {
                    tc_fence_before();
                    mbar_arrive(bar(sm.o_free[h]));
                }
            }
        }
    } else if (warp < 12) {
        setmaxnreg_dec<Regs<kInt8>::kOther>();
        if ((warp == 8 || warp == 10) && mine) {
            // ------------------------------------------ the products of one half
            // The whole warp walks, waits and counts, on values made uniform
            // (u()), and one elected lane issues: the products' operands then
            // stay in uniform registers. A warp per half, so that neither's
            // waits hold up the other's products.
            constexpr uint32_t idesc = kInt8 ? idesc_f16_f32(128, 128) : idesc_bf16_f32(128, 128);
            constexpr uint32_t idesc_s = kInt8 ? idesc_f16_f32(128, kCols) : idesc_bf16_f32(128, kCols);
            auto u = [](auto v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
            const int h = warp == 8 ? 0 : 1;
            const uint32_t q0 = u(desc_kmajor(smem_u32(sm.q[h])));
            const uint32_t k0 = u(desc_kmajor(smem_u32(sm.op))), v0 = u(desc_nmajor(smem_u32(sm.op)));
            const uint32_t tsc = u(tmem) + h * 128, to = u(tmem) + 256 + h * 128;
            const bool leader = elect_one();
            uint32_t pn = 0, on = 0, nq = 0;
            uint32_t sk = 0, ph = 0;     // slot and phase of the next operand tile
            bool ok = true;
            auto wait = [&](uint64_t &b, uint32_t phase, unsigned site) {
                ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar(b), phase & 1, abort, a.err, ROLE_MMA,
                                                             site, kWaitLimitNs, KID_ATTN));
                tc_fence_after();
            };
            auto advance = [&]() {
                if (++sk == kOps) {
                    sk = 0;
                    ph ^= 1;
                }
            };
            TilePiece p;
            while (u(take(p, ok, ROLE_MMA))) {
                const int cb = u(p.tile0 + p.first), ce = u(p.tile0 + p.last);
                if (ce <= cb) continue;
                const HalfTiles t = half_tiles(s, p, h, a.half_tokens);
                const int from = u(t.from), upto = u(t.upto);
                if (u(t.exists)) {
                    wait(sm.q_full[h], nq++, 1);
                    if (upto == from && leader) mma_commit(bar(sm.q_empty[h]));
                }
                // scores of part e of tile x: kCols rows of K
                auto scores = [&](int x, int e, uint32_t slot) {
                    const uint32_t k = k0 + slot * (kOperandBytes / 16) + e * (kCols * 128 / 16);
                    if (leader) {
                        mma_ss<false>(tsc + e * kCols, q0, k, idesc_s);
#pragma unroll
                        for (int kk = 1; kk < 8; ++kk) {
                            const uint32_t off = (kk >> 2) * (kOperandBytes / 32) + (kk & 3) * 2;
                            mma_ss<true>(tsc + e * kCols, q0 + off, k + off, idesc_s);
                        }
                        mma_commit(bar(sm.s_full[h][e]));
                        if (e == kN - 1 && x == upto - 1) mma_commit(bar(sm.q_empty[h]));
                    }
                    __syncwarp();
                };
                // Operand tiles come as K, V of each tile. The scores of part e of tile x
                // + 1 follow the output product of part e of tile x, whose weights lay
                // in the same columns.
                wait(sm.op_full[sk], ph, 2);
                if (!ok) break;
                if (from <= cb && cb < upto) {
#pragma unroll
                    for (int e = 0; e < kN; ++e) scores(cb, e, sk);
                }
                if (leader) mma_commit(bar(sm.op_empty[sk]));
                advance();
                for (int x = cb; x < ce; ++x) {
                    const uint32_t sv = sk;
                    wait(sm.op_full[sk], ph, 3);
                    advance();
                    if (x + 1 < ce) wait(sm.op_full[sk], ph, 6);
                    if (!ok) break;
                    const bool now = from <= x && x < upto, next = x + 1 < ce && from <= x + 1 && x + 1 < upto;
#pragma unroll
                    for (int e = 0; e < kN; ++e) {
                        if (now) {
                            wait(sm.p_full[h][e], pn, 4);
                            if (e == 0 && x == from && on > 0) wait(sm.o_free[h], on - 1, 5);
                            if (!ok) break;
                            const uint32_t v = v0 + sv * (kOperandBytes / 16) + e * (kCols * 128 / 16);
                            if (leader) {
                                mma_ts(to, tsc + e * kCols, v, idesc | kBNMajor, e > 0 || x > from ? 1u : 0u);
#pragma unroll
                                for (int kk = 1; kk < kCols / 16; ++kk)
                                    mma_ts(to, tsc + e * kCols + kk * 8, v + kk * 128, idesc | kBNMajor, 1u);
                                mma_commit(bar(sm.pv_done[h][e]));
                            }
                            __syncwarp();
                        }
                        if (next) scores(x + 1, e, sk);
                    }
                    if (!ok) break;
                    if (now) {
                        ++pn;
                        if (x == upto - 1) ++on;
                    }
                    if (leader) {
                        mma_commit(bar(sm.op_empty[sv]));
                        if (x + 1 < ce) mma_commit(bar(sm.op_empty[sk]));
                    }
                    if (x + 1 < ce) advance();
                }
            }
            // nothing may be in flight when tensor memory is freed and the CTA ends
            if (leader) mma_commit(bar(sm.drain[h]));
            __syncwarp();
            int never = 0;
            mbar_wait(bar(sm.drain[h]), 0, &never, a.err, ROLE_MMA, 8, kWaitLimitNs, KID_ATTN);
        } else if (warp == 9 && mine) {
            // ---------------------------------------------------------- the loads
            bool ok = true;
            uint32_t u = 0, fixes = 0;   // operand tiles, V tiles made zero in places
            uint32_t lands[2] = {0, 0};  // q's halves with rows to be made zero
            TilePiece p;
            while (take(p, ok, ROLE_PRODUCER)) {
                if (p.last <= p.first) continue;
                const int lo = p.lo, hi = p.kv;
                TileBoxes next = find_boxes(a.c, p.b, p.h, p.tile0 + p.first, lo, hi, a.err);
                for (int x = p.first; x < p.last && ok; ++x, ++it) {
                    const TileBoxes tb = next;
                    const int info = it % kInfo;
                    const bool full = (tb.mask.w[0] & tb.mask.w[1] & tb.mask.w[2] & tb.mask.w[3]) ==
                                      0xFFFFFFFFu;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++u) {
                        constexpr uint32_t kSlots = kInt8 ? kRaws : kOps;
                        const uint32_t sl = u % kSlots;
                        uint64_t &full_bar = kInt8 ? sm.raw_full[sl] : sm.op_full[sl];
                        uint64_t &empty_bar = kInt8 ? sm.raw_empty[sl] : sm.op_empty[sl];
                        if (u >= kSlots)
                            ok = __all_sync(0xFFFFFFFFu,
                                            ok && mbar_wait(bar(empty_bar), (u / kSlots - 1) & 1, abort,
                                                            a.err, ROLE_PRODUCER, 1, kWaitLimitNs, KID_ATTN));
                        if (!ok) break;
                        const uint32_t dst = kInt8 ? smem_u32(sm.raw[sl]) : smem_u32(sm.op[sl]);
                        // A V tile with masked positions is made zero there
                        // (BF16: whatever lies in them, times a weight of zero,
                        // need not be zero) before the products may read it.
                        const bool mend = !kInt8 && kv == 1 && !full;
                        const uint32_t b = mend ? bar(sm.fix) : bar(full_bar);
                        if (lane == 0) {
                            if (kv == 0) sm.mask[info] = tb.mask;
                            mbar_arrive_expect_tx(b, tile_bytes<kInt8>(a.c, tb) +
                                                         (kInt8 && kv == 0 ? 2 * scale_bytes(a.c, tb) : 0));
                            if (!kInt8 && kv == 0) mbar_arrive(bar(sm.info_full[info]));
                        }
                        __syncwarp();
                        copy_boxes<kInt8>(a.c, tb, kv == 0 ? &km : &vm, dst, b);
                        if constexpr (kInt8) {
                            if (kv == 0) {
                                copy_scales(a.c, tb, a.c.ks, smem_u32(sm.rks[info]), b);
                                copy_scales(a.c, tb, a.c.vs, smem_u32(sm.rvs[info]), b);
                            }
                        }
                        // (the table's entries for the next tile come while V waits)
                        if (kv == 0 && x + 1 < p.last)
                            next = find_boxes(a.c, p.b, p.h, p.tile0 + x + 1, lo, hi, a.err);
                        if (mend) {
                            ok = __all_sync(0xFFFFFFFFu, mbar_wait(b, fixes & 1, abort, a.err, ROLE_PRODUCER,
                                                                   2, kWaitLimitNs, KID_ATTN));
                            ++fixes;
                            for (int i = lane; i < kOperandBytes / 16; i += 32) {
                                const int r = (i >> 3) & 127;
                                if (!((tb.mask.w[r >> 5] >> (r & 31)) & 1u))
                                    reinterpret_cast<uint4 *>(sm.op[sl])[i] = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(full_bar));
                        }
                        if (kv == 0 && x == p.first) {
                            // the item's q, once the item before is done with its own
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (h * a.half_tokens >= p.ntok) continue;
                                if (qn[h] > 0)
                                    ok = __all_sync(0xFFFFFFFFu,
                                                    ok && mbar_wait(bar(sm.q_empty[h]), (qn[h] - 1) & 1, abort,
                                                                    a.err, ROLE_PRODUCER, 3, kWaitLimitNs,
                                                                    KID_ATTN));
                                if (!ok) break;
                                ++qn[h];
                                // (INT8: the converters do what spare rows need)
                                const bool spare = !kInt8 && own_rows(p, h, a.half_tokens, a.o.G) <
                                                                 a.half_tokens * a.o.G;
                                if (lane == 0) {
                                    const uint32_t qb = bar(kInt8 || spare ? sm.q_land[h] : sm.q_full[h]);
                                    mbar_arrive_expect_tx(qb, a.half_tokens * a.o.G * kHeadDim * 2);
#pragma unroll
                                    for (int d = 0; d < 2; ++d)
                                        tma_load_3d(smem_u32(sm.q[h]) + d * (kOperandBytes / 2), &qm,
                                                    d * 64, p.h * a.o.G,
                                                    p.t0 + p.tok0 + h * a.half_tokens, qb);
                                }
                                __syncwarp();
                                if (spare) {
                                    ok = __all_sync(0xFFFFFFFFu,
                                                    mbar_wait(bar(sm.q_land[h]), lands[h]++ & 1, abort, a.err,
                                                              ROLE_PRODUCER, 6, kWaitLimitNs, KID_ATTN));
                                    for (int i = own_rows(p, h, a.half_tokens, a.o.G) * 16 + lane;
                                         i < a.half_tokens * a.o.G * 16; i += 32)
                                        *q_piece(sm.q[h], i >> 4, i & 15) = make_uint4(0, 0, 0, 0);
                                    fence_proxy_async_smem();
                                    __syncwarp();
                                    if (lane == 0) mbar_arrive(bar(sm.q_full[h]));
                                }
                            }
                        }
                    }
                }
            }
            if (!ok) {   // nothing may be in flight when the CTA ends
                int never = 0;
                constexpr uint32_t kSlots = kInt8 ? kRaws : kOps;
                for (uint32_t x = u > kSlots ? u - kSlots : 0; x < u; ++x)
                    mbar_wait(bar(kInt8 ? sm.raw_full[x % kSlots] : sm.op_full[x % kSlots]),
                              (x / kSlots) & 1, &never, a.err, ROLE_PRODUCER, 4, kWaitLimitNs, KID_ATTN);
                for (int h = 0; h < 2; ++h) {
                    if (qn[h] > 0)
                        mbar_wait(bar(kInt8 ? sm.q_land[h] : sm.q_full[h]), (qn[h] - 1) & 1, &never,
                                  a.err, ROLE_PRODUCER, 5, kWaitLimitNs, KID_ATTN);
                    if (lands[h] > 0)
                        mbar_wait(bar(sm.q_land[h]), (lands[h] - 1) & 1, &never, a.err,
                                  ROLE_PRODUCER, 7, kWaitLimitNs, KID_ATTN);
                }
            }
        } else if (warp == 11 && mine) {
            // --------------------------------------------------------- the pieces
            bool ok = true;
            for (uint32_t n = 0; ok; ++n) {
                PagedPiece p;
                bool end = w.done(s, sh.end);
                while (!end) {
                    p = paged_piece(s, w, sh.begin, sh.end);
                    if (p.last > p.first || p.whole) break;
                    w.next(s);
                    end = w.done(s, sh.end);
                }
                const int i = n % kPieces;
                if (n >= kPieces)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(sm.piece_empty[i]), (n / kPieces - 1) & 1, abort,
                                                           a.err, ROLE_PRODUCER, 11, kWaitLimitNs, KID_ATTN));
                if (!ok) break;
                if (lane == 0) {
                    TilePiece t;
                    t.end = end ? 1 : 0;
                    if (!end) {
                        int lo, hi;
                        request_span(s, w.r, lo, hi);
                        t.b = w.b;
                        t.h = w.h;
                        t.t0 = w.r.t0;
                        t.base = w.r.base;
                        t.kv = hi;
                        t.lo = lo;
                        t.tok0 = p.tok0;
                        t.ntok = p.ntok;
                        t.tile0 = p.tile0;
                        t.first = p.first;
                        t.last = p.last;
                        t.whole = p.whole ? 1 : 0;
                        t.slot = p.slot;
                    }
                    sm.piece[i] = t;
                    mbar_arrive(bar(sm.piece_full[i]));
                }
                __syncwarp();
                if (end) break;
                w.next(s);
            }
        }
    } else {
        setmaxnreg_dec<Regs<kInt8>::kOther>();
        if constexpr (kInt8) {
            // ---------------------------------------------------- INT8 to fp16
            const int ct = tid - 384;               // 0 .. 127
            const int cw = ct >> 5;
            // Eight lanes take pieces 0-3 (4-7) of rows r and r ^ 5: reads and writes
            // through the swizzle then fall in distinct banks. A lane's rows are two of
            // every eight (1024 bytes), of the warp's 32.
            uint32_t from[2], to0[2];
            {
                const int pc = (lane & 3) + ((lane >> 3) & 1) * 4;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int pi = i * 2 + (lane >> 4), r = (lane & 4) ? pi ^ 5 : pi;
                    from[i] = (cw * 32 + r) * 128 + ((pc ^ r) << 4);
                    to0[i] = (pc >> 2) * (kOperandBytes / 2) + (cw * 32 + r) * 128 + ((((pc & 3) * 2) ^ r) << 4);
                }
            }
            bool ok = true;
            uint32_t u = 0, items = 0;
            TilePiece p;
            while (mine && take(p, ok, ROLE_CONVERT)) {
                if (p.last <= p.first) continue;
                int e = -100, top = -100;           // O's unit is 2^e; the largest so far
                float unscale = 0.0f;               // of q's scaling, and to log2 units
                for (int x = p.first; x < p.last && ok; ++x, ++it) {
                    const int info = it % kInfo;
                    for (int kv = 0; kv < 2; ++kv, ++u) {
                        const uint32_t rs = u % kRaws, os = u % kOps;
                        ok = __all_sync(0xFFFFFFFFu,
                                        ok &&
                                            mbar_wait(bar(sm.raw_full[rs]), (u / kRaws) & 1, abort, a.err,
                                                      ROLE_CONVERT, 1, kWaitLimitNs, KID_ATTN) &&
                                            (u < kOps ||
                                             mbar_wait(bar(sm.op_empty[os]), (u / kOps - 1) & 1, abort,
                                                       a.err, ROLE_CONVERT, 2, kWaitLimitNs, KID_ATTN)));
                        if (!ok) break;
                        // 16 codes to 32 bytes at a time
                        const uint8_t *src = sm.raw[rs];
                        uint8_t *dst = sm.op[os];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint4 y[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                y[i] = *reinterpret_cast<const uint4 *>(src + from[i & 1] + (2 * j + (i >> 1)) * 1024);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint4 g, f;
                                i8x4_to_f16x4(y[i].x, g.x, g.y);
                                i8x4_to_f16x4(y[i].y, g.z, g.w);
                                i8x4_to_f16x4(y[i].z, f.x, f.y);
                                i8x4_to_f16x4(y[i].w, f.z, f.w);
                                uint8_t *d = dst + (2 * j + (i >> 1)) * 1024;
                                *reinterpret_cast<uint4 *>(d + to0[i & 1]) = g;
                                *reinterpret_cast<uint4 *>(d + (to0[i & 1] ^ 16)) = f;
                            }
                        }
                        fence_proxy_async_smem();
                        mbar_arrive(bar(sm.op_full[os]));
                        if (kv == 1) {
                            mbar_arrive(bar(sm.raw_empty[rs]));
                            continue;
                        }
                        if (x == p.first) {
                            // the item's q to fp16, a row of each half per thread, scaled
                            // so that the largest value lies in [2^14, 2^15). (Once per item,
                            // so kept small: unrolled, its instructions pushed the tiles' out
                            // of the cache: 2.04 -> 2.11 ms for the long chunk.)
                            const int halves = a.half_tokens < p.ntok ? 2 : 1;
                            uint32_t mq = 0;
                            for (int h = 0; h < halves; ++h) {
                                ok = __all_sync(0xFFFFFFFFu,
                                                ok && mbar_wait(bar(sm.q_land[h]), qn[h] & 1, abort, a.err,
                                                                ROLE_CONVERT, 3, kWaitLimitNs, KID_ATTN));
                                ++qn[h];
                                if (ct >= own_rows(p, h, a.half_tokens, a.o.G))
#pragma unroll 1
                                    for (int j = 0; j < 16; ++j)
                                        *q_piece(sm.q[h], ct, j) = make_uint4(0, 0, 0, 0);
#pragma unroll 4
                                for (int j = 0; j < 16; ++j)
                                    mq = max(mq, amax_bits8(*q_piece(sm.q[h], ct, j)));
                            }
                            if (mq >= 0x7F80u) {    // no finite number: those that are
                                mq = 0;
#pragma unroll 1
                                for (int j = 0; j < 16 * halves; ++j)
                                    mq = max(mq, finite_amax8(*q_piece(sm.q[j >> 4], ct, j & 15)));
                            }
                            mq = __reduce_max_sync(0xFFFFFFFFu, mq);
                            if (lane == 0) sm.qmax[cw] = mq;
                            __syncwarp();
                            mbar_arrive(bar(sm.q_max));
                            ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar(sm.q_max), items & 1, abort, a.err,
                                                                         ROLE_CONVERT, 4, kWaitLimitNs,
                                                                         KID_ATTN));
                            ++items;
                            if (!ok) break;
                            mq = max(max(sm.qmax[0], sm.qmax[1]), max(sm.qmax[2], sm.qmax[3]));
                            const int be = static_cast<int>(mq >> 7);
                            const int se = be == 0 ? 0 : max(-100, min(100, 14 - (be - 127)));
                            const float qs = __uint_as_float(static_cast<uint32_t>(se + 127) << 23);
                            unscale = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - se) << 23);
                            for (int h = 0; h < halves; ++h) {
#pragma unroll 1
                                for (int j = 0; j < 16; ++j) {
                                    uint4 y = *q_piece(sm.q[h], ct, j);
                                    y.x = pack_f16x2(__uint_as_float(y.x << 16) * qs, __uint_as_float(y.x & 0xFFFF0000u) * qs);
                                    y.y = pack_f16x2(__uint_as_float(y.y << 16) * qs, __uint_as_float(y.y & 0xFFFF0000u) * qs);
                                    y.z = pack_f16x2(__uint_as_float(y.z << 16) * qs, __uint_as_float(y.z & 0xFFFF0000u) * qs);
                                    y.w = pack_f16x2(__uint_as_float(y.w << 16) * qs, __uint_as_float(y.w & 0xFFFF0000u) * qs);
                                    *q_piece(sm.q[h], ct, j) = y;
                                }
                                fence_proxy_async_smem();
                                mbar_arrive(bar(sm.q_full[h]));
                            }
                        }
                        // what the softmax takes of the scales, one position per thread;
                        // the tile's largest v scale, by every warp for itself
                        const TileMask tm = sm.mask[info];
                        uint32_t wm = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((tm.w[i] >> lane) & 1u)
                                wm = max(wm, __float_as_uint(fabsf(sm.rvs[info][32 * i + lane])));
                        wm = __reduce_max_sync(0xFFFFFFFFu, wm);
                        const bool live = (sm.mask[info].w[cw] >> lane) & 1u;
                        const float rk = live ? sm.rks[info][ct] : 0.0f;
                        const float rv = live ? sm.rvs[info][ct] : 0.0f;
                        mbar_arrive(bar(sm.raw_empty[rs]));
                        // a new unit when the largest weight would pass 16 of it, or
                        // stay below 1/8 (not more than 2^60 below the item's largest unit:
                        // O is FP32; a tile of zero vectors needs none)
                        const int te = max(-100, min(100, static_cast<int>(wm >> 23) - 127));
                        if (static_cast<unsigned>(te - e + 3) > 6u && wm != 0) {
                            e = max(te, top - 60);
                            top = max(top, e);
                        }
                        const float un = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
                        const float ui = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                        float *c4 = reinterpret_cast<float *>(&sm.col[info][ct >> 1]) + (ct & 1);
                        c4[0] = rk * unscale;
                        c4[2] = rv * ui;
                        if (ct == 0) sm.unit[info] = un;
                        mbar_arrive(bar(sm.info_full[info]));
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// q as [T, Hq, 128]: a box is 64 dimensions x the G heads of a kv head x the
// whole tokens of a half.
bool encode_q(CUtensorMap *map, const PagedAttnProblem &p, int half_tokens) {
    auto fn = tensor_map_encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(p.Hq), static_cast<cuuint64_t>(p.T)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.qh) * 2, static_cast<cuuint64_t>(p.qt) * 2};
    cuuint32_t bx[3] = {64, static_cast<cuuint32_t>(p.Hq / p.Hkv),
                        static_cast<cuuint32_t>(half_tokens)};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p.q), dims, strides,
              bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kInt8>
cudaError_t launch_kind(const PagedAttnProblem &p, const PagedSetup &u, int ctas,
                        unsigned long long *err, cudaStream_t stream) {
    auto kernel = paged_tiles_kernel<kInt8>;
    const size_t smem = sizeof(TilesSmem<kInt8>) + 1024;
    static_assert(sizeof(TilesSmem<kInt8>) + 1024 <= 227 * 1024, "shared memory");
    static int attr_done[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        attr_done[dev] = 1;
    }
    TilesArgs a;
    a.s = u.s;
    a.c = u.c;
    a.o = u.o;
    a.half_tokens = kHalfRows / u.o.G;
    a.scale_log2 = p.scale * kLog2e;
    a.ws = static_cast<float *>(p.workspace);
    a.err = err;
    CUtensorMap qm, km, vm;
    if (!encode_q(&qm, p, a.half_tokens) || !paged_encode_cache(&km, p.kc, kInt8, p, u.c.box) ||
        !paged_encode_cache(&vm, p.vc, kInt8, p, u.c.box))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, qm, km, vm, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tiles(const PagedAttnProblem &p, const PagedSetup &u, int ctas,
                               unsigned long long *err, cudaStream_t stream) {
    return p.ks != nullptr ? launch_kind<true>(p, u, ctas, err, stream)
                           : launch_kind<false>(p, u, ctas, err, stream);
}

}  // namespace w8a8
