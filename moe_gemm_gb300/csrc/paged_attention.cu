// Attention of each request's new tokens over its pages of the KV cache, on
// sm_103a ("Deploying Hunyuan 770B in INT8 on domestic accelerators", §3.4:
// the attention kernel reads the INT8 cache and applies the vectors' scales
// itself). Query i of a request's n new tokens stands at position p = kv_len -
// n + i and sees the keys max(0, p - window + 1) .. p:
//
//   o = sum_j softmax_j(scale q . k_j) v_j.
//
// One call serves prompts, chunks of prompts over what is cached of them,
// guessed tokens and single tokens together. The query heads that share a kv
// head are rows of one product, so the cache is read once for all of them;
// the work is shared out as paged_schedule.cuh says.
//  * paged_rows_kernel: up to 16 query rows per item (mma.sync), for calls of
//    few new tokens per request: an HBM stream of the cache.
//  * paged_tiles_kernel (paged_attention_tiles.cu): up to 256 query rows per item
//    on the tcgen05 tensor cores, for calls with more.
//  * paged_combine_kernel joins the shares of items that were divided.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attention_math.cuh"
#include "common.cuh"
#include "internal.h"
#include "paged_attention.cuh"
#include "paged_schedule.cuh"
#include "tensor_map.h"

namespace w8a8 {
namespace {

constexpr int kMaxCtas = 512;        // of the rows kernel
constexpr int kRowsMax = 16;         // query rows of an item, rows kernel
constexpr int kRowWarps = 4;         // 32 positions of a tile each
constexpr int kRowThreads = kRowWarps * 32;
constexpr float kNegInf = -INFINITY;

// The kernel of a call, by the query rows that a request and kv head have on
// average: up to 16 fit one item of the rows kernel, which reads the cache
// once; more take the tiles kernel. 32 requests at 4096 positions, 8 kv heads, rows
// kernel / tiles kernel: 16 rows INT8 80 / 144 us and BF16 135 / 102, 24 rows 144 /
// 144 and 247 / 103. (BF16 pages pay for their place among the first 16: their
// probabilities keep 24 bits there, and 8 in the tiles kernel.) The lengths are on the
// device, so one kernel takes the whole call: 32 single tokens over 4096 positions
// (INT8 63 us, BF16 102) with a chunk of 512 over 4096 (118, 90) take 255 and 181 in
// one call.
bool uses_tiles(int64_t T, int64_t B, int64_t G) { return T * G > kRowsMax * B; }

// ------------------------------------------------------------ the rows kernel
struct RowsArgs {
    PagedSchedule s;
    PagedCache c;
    PagedOut o;
    const uint16_t *q;      // [T, Hq, 128], token stride qt, head stride qh
    int64_t qt, qh;
    float scale;            // to log2 units
    float *ws;
    unsigned long long *err;
};

// Tiles that a warp keeps in flight, with two CTAs of INT8 pages per SM or one of BF16
// pages (three CTAs per SM took 69 us when the decode step below took 56: their
// registers spill).
template <bool kInt8>
constexpr int kRowStages = kInt8 ? 2 : 3;

template <int NT, bool kInt8>
struct RowsSmem {
    static constexpr int kSlice = Tile<kInt8>::kBytes / kRowWarps;   // K, or V, of 32 positions
    static constexpr int kStages = kRowStages<kInt8>;
    uint4 k[kRowWarps][kStages][kSlice / 16];       // 1024-byte aligned
    uint4 v[kRowWarps][kStages][kSlice / 16];
    float ks[kRowWarps][kStages][32], vs[kRowWarps][kStages][32];
    uint32_t mask[kRowWarps][kStages];              // which positions hold keys
    float merge[8 * NT * 4][32];                    // a warp's output, as fragments
    float red_m[kRowWarps][8 * NT], red_l[kRowWarps][8 * NT];
    uint64_t kfull[kRowWarps][kStages], vfull[kRowWarps][kStages];
    volatile int abort_flag;
};

// A lane's fragments of 32 landed positions (attention_math.cuh: ChunkRegs);
// bit i of the mask: position i is a key.
__device__ __forceinline__ int slice_at(int row, int piece) {
    return ((piece >> 3) * 32 + row) * 8 + ((piece & 7) ^ (row & 7));
}

template <bool kInt8>
__device__ __forceinline__ void key_frags(ChunkRegs<kInt8> &r, const uint4 *k, const float *ks,
                                          int gid, int t) {
    using R = ChunkRegs<kInt8>;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int row = 16 * mt + gid + 8 * hf;
#pragma unroll
            for (int x = 0; x < R::KV; ++x) r.k[mt][hf][x] = k[slice_at(row, t * R::KV + x)];
            r.ks[mt][hf] = kInt8 ? ks[row] : 1.0f;
        }
}

template <bool kInt8>
__device__ __forceinline__ void value_frags(ChunkRegs<kInt8> &r, const uint4 *v, const float *vs,
                                            uint32_t mask, int gid, int t) {
    using R = ChunkRegs<kInt8>;
    auto ok = [&](int row) { return (mask >> row) & 1u; };
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int row = 16 * mt + gid + 8 * hf;
            const float s = kInt8 ? vs[row] : 1.0f;
            r.vs[mt][hf] = ok(row) ? s : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 16 * mt + 2 * t + (j < 2 ? j : j + 6);
#pragma unroll
            for (int x = 0; x < R::VV; ++x) {
                r.v[mt][j][x] = v[slice_at(row, gid * R::VV + x)];
                // what lies in a masked BF16 position may be no number at all
                if (!kInt8 && !ok(row)) r.v[mt][j][x] = make_uint4(0, 0, 0, 0);
            }
        }
    }
}

// A persistent CTA of four warps. Warp w takes positions [32 w, 32 w + 32) of
// each of its items' tiles, and loads them for itself: one to four TMA boxes of
// K and of V and the scales, kRowStages tiles ahead, so that warps wait for one
// another only when an item ends (a fifth warp that loaded for all held the
// registers of one to two CTAs per SM: a decode step of 32 requests at 4096
// positions took 62 us when this form took 56). Query row r of an item is query
// head r % G of its new token r / G. Arithmetic as in the contiguous-cache
// kernel (attention.cu): scores and outputs by mma.sync with FP32 sums, the
// probabilities split into two fp16 (three bf16) parts, running maximum and sum
// per warp.
//
// BF16 pages are an HBM stream when there is enough of one: 4 requests at 33 to 131
// thousand positions (1.34 GB) take 218 us, 6.2 TB/s. (A stage is copied into again when
// the scores are done, or V's fragments read. Both at once, or both later, took 228 to 232;
// mbarriers in place of the fences 224, and INT8 57 for 55 below.) INT8 pages halve the bytes and
// not the instructions: 32 requests at 2 to 4 thousand positions (214 MB) take 55 us,
// 3.9 TB/s, of which about 13 are the same for any length (2 until the share is known,
// 4 until the first tiles are there, 1.4 for the join, 5 for the second kernel) and the
// rest runs at 5.4 TB/s.
template <int NT, bool kInt8>
__global__ void __launch_bounds__(kRowThreads, kInt8 ? 2 : 1)
paged_rows_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                  const RowsArgs a) {
    extern __shared__ uint8_t smem_raw[];
    using Smem = RowsSmem<NT, kInt8>;
    constexpr int kStages = Smem::kStages;
    Smem &sm = *reinterpret_cast<Smem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, t = lane & 3;
    const PagedSchedule &s = a.s;
    if (tid == 0) {
        for (int i = 0; i < kRowWarps; ++i)
            for (int j = 0; j < kStages; ++j) {
                mbar_init(smem_u32(&sm.kfull[i][j]), 1);
                mbar_init(smem_u32(&sm.vfull[i][j]), 1);
            }
        sm.abort_flag = 0;
        fence_mbarrier_init();
    }
    griddep_launch_dependents();
    griddep_wait();   // lengths, tables and the cache may come from the kernel before
    const PagedShare sh = paged_share<kRowThreads>(s, blockIdx.x, gridDim.x);   // (synchronises)
    PagedWalk w;
    w.start(s, sh);
    if (tid == kRowThreads - 1)
        paged_write_cut(s, sh, w, blockIdx.x, cuts_of(a.ws, kRowsMax, gridDim.x));
    if (static_cast<int>(blockIdx.x) >= sh.ctas || w.done(s, sh.end)) return;
    uint32_t it = 0, issued = 0;   // tiles so far: stage it % kStages, phase it / kStages
    bool ok = true;
    const int box_shift = __ffs(a.c.box) - 1;

    // Where the boxes of the warp's part of the tiles from x on (of the request's, before
    // end) lie in the cache, through the block table: 2^box_shift tiles at a time, lane l
    // has box l % boxes of tile x + l / boxes (its first row; -1: not loaded).
    const int boxes_log2 = 5 - box_shift;
    auto find = [&](const PagedWalk &w, int x, int end) -> int {
        int lo, hi;
        request_span(s, w.r, lo, hi);
        x += lane >> boxes_log2;
        if (x >= end) return -1;
        const int pos = x * kTilePositions + 32 * warp + ((lane << box_shift) & 31);
        if (pos >= hi || pos + a.c.box <= lo) return -1;
        const int pg = page_of(a.c, pos);
        const int id = a.c.table[static_cast<int64_t>(w.b) * a.c.W + pg];
        if (id < 0 || id >= a.c.P) {
            record_device_error(a.err, KID_ATTN, ROLE_PRODUCER, 9);
            return -1;
        }
        return (id * a.c.Hkv + w.h) * a.c.page + pos - pg * a.c.page;   // (rows of the cache: below 2^31)
    };
    int found = -1, found_at = 0;   // from find, and its x
    // The lane's box of tile x, one of those found.
    auto place = [&](int x) -> int {
        const int row = __shfl_sync(0xFFFFFFFFu, found, (((x - found_at) << boxes_log2) + lane) & 31);
        return (lane >> boxes_log2) == 0 ? row : -1;
    };
    // Starts the copies of K, or of V, of the boxes at `row` into stage n % kStages.
    // Its last reader is this warp, every lane of which has put a fence between its reads
    // and here: the copy is another proxy's, and orders itself after nothing else. (Without,
    // copies from L2 overtook reads, mostly of BF16 pages with 16 rows per item.)
    auto copy = [&](bool v, int row, uint32_t n) {
        const int sg = n % kStages;
        const uint32_t bar = smem_u32(v ? &sm.vfull[warp][sg] : &sm.kfull[warp][sg]);
        const unsigned used = __ballot_sync(0xFFFFFFFFu, row >= 0);
        if (lane == 0)
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(used) << box_shift) *
                                           (kInt8 ? 128 + 4 : 2 * 128));
        __syncwarp();
        if (row < 0) return;
        const uint32_t dst = smem_u32(v ? sm.v[warp][sg] : sm.k[warp][sg]) +
                             static_cast<uint32_t>(lane << box_shift) * 128;
#pragma unroll
        for (int half = 0; half < Tile<kInt8>::kHalves; ++half)
            tma_load_2d(dst + half * 4096, v ? &vm : &km, half * 64, row, bar);
        if constexpr (kInt8)
            bulk_g2s(smem_u32(v ? &sm.vs[warp][sg][lane << box_shift] : &sm.ks[warp][sg][lane << box_shift]),
                     (v ? a.c.vs : a.c.ks) + row, a.c.box * 4, bar);
    };
    // Which of the 32 positions hold keys, given where the boxes lie.
    auto keys = [&](const PagedWalk &w, int x, int row) -> uint32_t {
        int lo, hi;
        request_span(s, w.r, lo, hi);
        const unsigned used = __ballot_sync(0xFFFFFFFFu, row >= 0);
        const int pos = x * kTilePositions + 32 * warp + lane;
        return __ballot_sync(0xFFFFFFFFu,
                             ((used >> (lane >> box_shift)) & 1u) && pos >= lo && pos < hi);
    };
    // (the fences of the piece before cover all its reads)
    auto begin = [&](const PagedWalk &w, const PagedPiece &p) {
        found_at = p.tile0 + p.first;
        found = find(w, found_at, p.tile0 + p.last);    // (8 tiles or more)
#pragma unroll
        for (int j = 0; j < kStages; ++j) {
            if (p.first + j >= p.last) continue;
            const int x = p.tile0 + p.first + j, row = place(x);
            copy(false, row, it + j);
            copy(true, row, it + j);
            const uint32_t mask = keys(w, x, row);
            if (lane == 0) sm.mask[warp][(it + j) % kStages] = mask;
        }
        issued = it + min(kStages, p.last - p.first);
        __syncwarp();
    };
    PagedPiece p = paged_piece(s, w, sh.begin, sh.end);
    begin(w, p);

    while (true) {
        const int rows = p.ntok * a.o.G;
        const bool idle = p.first == p.last && !p.whole;
        WarpState<NT> st;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                st.m[nt][j] = kNegInf;
                st.l[nt][j] = 0.0f;
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) st.o[i][nt][k] = 0.0f;
        st.se = 0;
        st.low = 100;
        if (p.first < p.last) {
            // q rows 8 nt + gid, dims [32 t, 32 t + 32), as bf16 pairs
            uint32_t qf[NT][16];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = 8 * nt + gid;
                const bool use = r < rows;
                const int tok = use ? r / a.o.G : 0, g = use ? r % a.o.G : 0;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (static_cast<int64_t>(w.r.t0) + p.tok0 + tok) * a.qt +
                    (static_cast<int64_t>(w.h) * a.o.G + g) * a.qh + 32 * t);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint4 y = use ? src[x] : make_uint4(0, 0, 0, 0);
                    qf[nt][4 * x + 0] = y.x;
                    qf[nt][4 * x + 1] = y.y;
                    qf[nt][4 * x + 2] = y.z;
                    qf[nt][4 * x + 3] = y.w;
                }
            }
            // INT8: q in fp16, scaled by the power of two that puts the item's
            // largest |q| in [2^14, 2^15); the scores are scaled back exactly
            float qinv = 1.0f;
            if constexpr (kInt8) {
                uint32_t mq = 0;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 16; ++x) mq = __vmaxu2(mq, finite_bits2(qf[nt][x]));
                mq = max(mq & 0xFFFFu, mq >> 16);
                mq = __reduce_max_sync(0xFFFFFFFFu, mq);
                const int bexp = static_cast<int>((mq >> 7) & 0xFFu);
                const int se = bexp == 0 ? 0 : max(-100, min(100, 14 - (bexp - 127)));
                const float qs = __uint_as_float(static_cast<uint32_t>(se + 127) << 23);
                qinv = __uint_as_float(static_cast<uint32_t>(127 - se) << 23);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        qf[nt][x] = pack_f16x2(__uint_as_float(qf[nt][x] << 16) * qs,
                                               __uint_as_float(qf[nt][x] & 0xFFFF0000u) * qs);
            }
            // the positions that this lane's score columns see: [from, upto)
            int from[NT][2], upto[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 8 * nt + 2 * t + j;
                    const int pos = w.r.base + p.tok0 + r / a.o.G;
                    upto[nt][j] = r < rows ? pos + 1 : 0;
                    from[nt][j] = s.window > 0 ? max(pos, 0) - s.window + 1 : 0;
                }
            // tiles that every row sees whole need no mask
            const int pos_first = w.r.base + p.tok0, pos_last = pos_first + p.ntok - 1;
            // (not unrolled over the stages: the two forms of the body fill the
            // instruction cache as it is, and three copies ran at half the speed)
#pragma unroll 1
            for (int x = p.first; x < p.last; ++x) {
                const int sg = it % kStages;
                auto landed = [&](uint64_t &bar, unsigned site) {
                    ok = __all_sync(0xFFFFFFFFu,
                                    ok && mbar_wait(smem_u32(&bar), (it / kStages) & 1, &sm.abort_flag,
                                                    a.err, ROLE_EPILOGUE, site, kWaitLimitNs, KID_ATTN));
                };
                landed(sm.kfull[warp][sg], 3);
                const uint32_t mw = sm.mask[warp][sg];
                ChunkRegs<kInt8> r;
                key_frags<kInt8>(r, sm.k[warp][sg], sm.ks[warp][sg], gid, t);
                const bool more = ok && x + kStages < p.last;
                const int next = p.tile0 + x + kStages;
                int row = -1;
                uint32_t mask = 0;
                if (more) {
                    row = place(next);
                    mask = keys(w, next, row);
                }
                auto values = [&](ChunkRegs<kInt8> &r) {
                    fence_proxy_async_smem();   // (the scores are done: K's fragments are read)
                    __syncwarp();
                    if (more) copy(false, row, it + kStages);
                    landed(sm.vfull[warp][sg], 4);
                    value_frags<kInt8>(r, sm.v[warp][sg], sm.vs[warp][sg], mw, gid, t);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (more) {
                        copy(true, row, it + kStages);
                        if (lane == 0) sm.mask[warp][sg] = mask;
                        issued = it + kStages + 1;
                        if (next + 1 - found_at == 1 << box_shift) {
                            found_at = next + 1;
                            found = find(w, found_at, p.tile0 + p.last);
                        }
                    }
                };
                const int c0 = (p.tile0 + x) * kTilePositions + 32 * warp;
                const bool plain = mw == 0xFFFFFFFFu && c0 + 31 <= pos_first &&
                                   (s.window == 0 || c0 > pos_last - s.window);
                if (plain) {
                    attend_chunk<NT, kInt8, true>(
                        st, r, qf, [](int, int, int) { return true; }, values, a.scale, qinv, 0, gid, t);
                } else {
                    attend_chunk<NT, kInt8, true>(
                        st, r, qf,
                        [&](int row, int nt, int e) {
                            return ((mw >> row) & 1u) && c0 + row < upto[nt][e] &&
                                   c0 + row >= from[nt][e];
                        },
                        values, a.scale, qinv, 0, gid, t);
                }
                ++it;
                if (!ok && issued > it) {   // what is in flight lands before the CTA ends
                    int never = 0;
                    for (uint32_t n = it; n < issued; ++n) {
                        mbar_wait(smem_u32(&sm.kfull[warp][n % kStages]), (n / kStages) & 1, &never,
                                  a.err, ROLE_PRODUCER, 2, kWaitLimitNs, KID_ATTN);
                        mbar_wait(smem_u32(&sm.vfull[warp][n % kStages]), (n / kStages) & 1, &never,
                                  a.err, ROLE_PRODUCER, 2, kWaitLimitNs, KID_ATTN);
                    }
                    issued = it;
                }
            }
        }
        // the next item's first tiles are on their way while this one ends
        const PagedWalk cw = w;
        const PagedPiece cp = p;
        w.next(s);
        const bool last = w.done(s, sh.end);
        if (!last) {
            p = paged_piece(s, w, sh.begin, sh.end);
            if (ok) begin(w, p);
        }
        if (idle) {
            if (last) break;
            continue;
        }

        // ---- join the four warps: every warp's state weighted by
        // e^(its max - the item's max)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = st.l[nt][j];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                if (gid == 0) {
                    sm.red_m[warp][8 * nt + 2 * t + j] = st.m[nt][j];
                    sm.red_l[warp][8 * nt + 2 * t + j] = l;
                }
            }
        named_barrier_sync(1, kRowThreads);
        const float unit = __uint_as_float(static_cast<uint32_t>(127 - st.se) << 23);   // 2^-se
        float mx[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 8 * nt + 2 * t + j;
                float m = sm.red_m[0][r];
#pragma unroll
                for (int x = 1; x < kRowWarps; ++x) m = fmaxf(m, sm.red_m[x][r]);
                mx[nt][j] = m;
                const float mu = m == kNegInf ? 0.0f : m;   // a row that sees nothing
                l[nt][j] = 0.0f;
#pragma unroll
                for (int x = 0; x < kRowWarps; ++x)
                    l[nt][j] += sm.red_l[x][r] * ex2_approx(sm.red_m[x][r] - mu);
                const float f = unit * ex2_approx(st.m[nt][j] - mu);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    st.o[i][nt][j] *= f;
                    st.o[i][nt][j + 2] *= f;
                }
            }
#pragma unroll 1
        for (int giver = 1; giver < kRowWarps; ++giver) {
            if (warp == giver) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sm.merge[(i * NT + nt) * 4 + k][lane] = st.o[i][nt][k];
            }
            named_barrier_sync(1, kRowThreads);
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st.o[i][nt][k] += sm.merge[(i * NT + nt) * 4 + k][lane];
            }
            named_barrier_sync(1, kRowThreads);
        }
        if (warp == 0 && ok) {
            // lane (gid, t) has dims [16 gid, 16 gid + 16) of rows 8 nt + 2 t + j:
            // fragment i, elements j and j + 2 are dims 2 i and 2 i + 1 of them
            float *part = slot_of(a.ws, kRowsMax, blockIdx.x, cp.slot);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int r = 8 * nt + 2 * t + j;
                    if (r >= rows) continue;
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[2 * i] = st.o[i][nt][j];
                        v[2 * i + 1] = st.o[i][nt][j + 2];
                    }
                    if (!cp.whole) {
                        float4 *dst = reinterpret_cast<float4 *>(part + r * kHeadDim + 16 * gid);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        if (gid == 0) {
                            part[kRowsMax * kHeadDim + r] = mx[nt][j];
                            part[kRowsMax * (kHeadDim + 1) + r] = l[nt][j];
                        }
                        continue;
                    }
                    const int64_t orow = out_row(a.o, cw.r, cw.h, cp.tok0, r);
#pragma unroll
                    for (int i = 0; i < 16; ++i)   // (a row that sees nothing: zeros)
                        v[i] = l[nt][j] == 0.0f ? 0.0f : v[i] / l[nt][j];
                    if (a.o.fp32) {
                        float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.o.out) +
                                                                 orow * kHeadDim + 16 * gid);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o.out) +
                                                               orow * kHeadDim + 16 * gid);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            dst[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]),
                                                pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                                pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                                                pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
                    }
                }
        }
        if (last) break;
    }
}

// ------------------------------------------------------------------- combine
// A kernel of its own: it starts on every SM at once, where the last CTA of an item
// would join its shares alone.
constexpr int kCombineThreads = 128;

struct CombineArgs {
    const int32_t *cu;
    int B, T;
    PagedOut o;
    float *ws;
    int rows;               // rows of a slot
    int ctas;               // the attention kernel's grid
    int overhead;           // as in its schedule
};

// Block (c, y): when the border before CTA c is the first one inside an item
// (its cut says so), joins the item's shares for rows 4 y + warp, + 4 gridDim.y,
// ... Lane j works out share j and holds its maximum and sum, so a row costs one
// round of loads for those and one for the shares' outputs. Blocks also write
// zeros to rows of tokens that belong to no request.
__global__ void __launch_bounds__(kCombineThreads)
paged_combine_kernel(const CombineArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;
    const PagedCut cut = cuts_of(a.ws, a.rows, a.ctas)[c];
    {
        const int64_t first = min(max(a.cu[0], 0), a.T), last = min(max(a.cu[a.B], 0), a.T);
        const int64_t per = static_cast<int64_t>(a.o.Hq) * kHeadDim * (a.o.fp32 ? 4 : 2) / 16;
        const int64_t n = (first + a.T - last) * per;
        uint4 *out = static_cast<uint4 *>(a.o.out);
        const int64_t stride = static_cast<int64_t>(gridDim.x) * gridDim.y * kCombineThreads;
        for (int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kCombineThreads +
                         threadIdx.x;
             i < n; i += stride)
            out[i < first * per ? i : i - first * per + last * per] = make_uint4(0, 0, 0, 0);
    }
    if (cut.ntiles <= 0) return;
    PagedRequest r;
    r.t0 = cut.t0;
    const int rows = cut.ntok * a.o.G;
    for (int row = blockIdx.y * (kCombineThreads / 32) + warp; row < rows;
         row += gridDim.y * (kCombineThreads / 32)) {
        float m = kNegInf, l = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // 32 CTAs at a time, from the one that the border ends
        for (int k0 = c - 1; k0 < cut.ctas; k0 += 32) {
            const int k = k0 + lane;
            const long long from = paged_border(cut.total, cut.ctas, min(k, cut.ctas));
            const long long upto = paged_border(cut.total, cut.ctas, min(k + 1, cut.ctas));
            const bool in = k < cut.ctas && from < cut.at + cut.cost;
            PagedPiece p;
            p.ntiles = cut.ntiles;
            p.first = p.last = 0;
            p.whole = false;
            if (in) paged_part(p, cut.at, cut.cost, a.overhead, from, upto);
            if (__any_sync(0xFFFFFFFFu, p.whole)) return;   // one CTA has all its tiles: it wrote it
            const bool has = p.last > p.first;
            const float *part = a.ws + (static_cast<int64_t>(k) * 2 + p.slot) * a.rows * (kHeadDim + 2);
            float pm = kNegInf, pl = 0.0f;
            if (has) {
                pm = part[a.rows * kHeadDim + row];
                pl = part[a.rows * (kHeadDim + 1) + row];
            }
            float mn = pm;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
            mn = fmaxf(mn, m);
            const float mu = mn == kNegInf ? 0.0f : mn;
            const float fo = ex2_approx(m - mu), fn = has ? ex2_approx(pm - mu) : 0.0f;
            m = mn;
            float ls = pl * fn;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xFFFFFFFFu, ls, o);
            l = l * fo + ls;
            acc.x *= fo;
            acc.y *= fo;
            acc.z *= fo;
            acc.w *= fo;
            unsigned todo = __ballot_sync(0xFFFFFFFFu, has);
            while (todo != 0) {      // four shares' outputs at a time
                float4 v[4];
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = todo != 0 ? __ffs(todo) - 1 : 0;
                    const int slot = __shfl_sync(0xFFFFFFFFu, p.slot, j);
                    f[e] = __shfl_sync(0xFFFFFFFFu, fn, j);
                    if (todo == 0) f[e] = 0.0f;
                    v[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (todo != 0)
                        v[e] = reinterpret_cast<const float4 *>(
                            a.ws + (static_cast<int64_t>(k0 + j) * 2 + slot) * a.rows * (kHeadDim + 2) +
                            row * kHeadDim)[lane];
                    todo &= todo - 1;
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc.x = fmaf(v[e].x, f[e], acc.x);
                    acc.y = fmaf(v[e].y, f[e], acc.y);
                    acc.z = fmaf(v[e].z, f[e], acc.z);
                    acc.w = fmaf(v[e].w, f[e], acc.w);
                }
            }
            if (__any_sync(0xFFFFFFFFu, !in)) break;
        }
        const int64_t orow = out_row(a.o, r, cut.h, cut.tok0, row);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (l != 0.0f) v = make_float4(acc.x / l, acc.y / l, acc.z / l, acc.w / l);
        if (a.o.fp32)
            reinterpret_cast<float4 *>(static_cast<float *>(a.o.out) + orow * kHeadDim)[lane] = v;
        else
            reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.o.out) + orow * kHeadDim)[lane] =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
}

// ---------------------------------------------------------------------- host
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                       cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

// A warp of the rows kernel copies its 32 positions in boxes of this many.
int rows_box(const PagedAttnProblem &p) { return gcd(static_cast<int>(p.page), 32); }

// slot: rows of a slot of the workspace, item: rows of an item.
cudaError_t launch_combine(const PagedSetup &u, float *ws, int slot, int item, int ctas,
                           cudaStream_t stream) {
    CombineArgs a;
    a.cu = u.s.cu;
    a.B = u.s.B;
    a.T = u.s.T;
    a.o = u.o;
    a.ws = ws;
    a.rows = slot;
    a.ctas = ctas;
    a.overhead = u.s.overhead;
    // a row per warp, or 4 of the tiles kernel's 256 (with 8 rows per warp a long chunk took
    // 2.05 ms for 2.01, with 1 the blocks cost more than they save: 2.02)
    const int y = std::min(item / (kCombineThreads / 32), 16);
    return launch_pdl(paged_combine_kernel, dim3(ctas, y), kCombineThreads, 0, stream, a);
}

template <int NT, bool kInt8>
cudaError_t launch_rows(const PagedAttnProblem &p, const CUtensorMap &km, const CUtensorMap &vm,
                        int num_sms, unsigned long long *err, cudaStream_t stream) {
    auto kernel = paged_rows_kernel<NT, kInt8>;
    const size_t smem = sizeof(RowsSmem<NT, kInt8>) + 1024;
    static int per_sm[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (per_sm[dev] == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kRowThreads, smem);
        if (e != cudaSuccess) return e;
        per_sm[dev] = n > 0 ? n : 1;
    }
    int ctas = per_sm[dev] * num_sms;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    RowsArgs a;
    PagedSetup u = paged_setup(p, 8 * NT);
    u.c.box = rows_box(p);
    a.s = u.s;
    a.c = u.c;
    a.o = u.o;
    a.q = p.q;
    a.qt = p.qt;
    a.qh = p.qh;
    a.scale = p.scale * kLog2e;
    a.ws = static_cast<float *>(p.workspace);
    a.err = err;
    e = launch_pdl(kernel, dim3(ctas), kRowThreads, smem, stream, km, vm, a);
    if (e != cudaSuccess) return e;
    return launch_combine(u, a.ws, kRowsMax, 8 * NT, ctas, stream);
}

}  // namespace

PagedSetup paged_setup(const PagedAttnProblem &p, int rows) {
    PagedSetup u;
    u.o.out = p.out;
    u.o.fp32 = p.out_fp32 ? 1 : 0;
    u.o.Hq = static_cast<int>(p.Hq);
    u.o.G = static_cast<int>(p.Hq / p.Hkv);
    u.s.cu = p.cu_new;
    u.s.kv = p.kv_lens;
    u.s.B = static_cast<int>(p.B);
    u.s.T = static_cast<int>(p.T);
    u.s.Hkv = static_cast<int>(p.Hkv);
    // (an item of the tiles kernel is two halves of whole tokens)
    u.s.tile_tokens = rows == kPagedTileRows ? 2 * (rows / 2 / u.o.G) : rows / u.o.G;
    u.s.capacity = p.W * p.page;
    // a window that reaches past the first position of any row masks nothing
    u.s.window = p.window >= u.s.capacity ? 0 : static_cast<int>(p.window);
    // (what an item takes beside its tiles: measured, in tiles of each kernel)
    u.s.overhead = rows == kPagedTileRows ? 11 * kTilePositions / 4 : 3 * kTilePositions / 2;
    u.s.min_share = 2 * kTilePositions;
    u.c.table = p.block_table;
    u.c.ks = p.ks;
    u.c.vs = p.vs;
    u.c.W = static_cast<int>(p.W);
    u.c.P = static_cast<int>(p.P);
    u.c.Hkv = static_cast<int>(p.Hkv);
    u.c.page = static_cast<int>(p.page);
    u.c.box = gcd(u.c.page, kTilePositions);
    u.c.page_shift = (u.c.page & (u.c.page - 1)) == 0 ? __builtin_ctz(u.c.page) : -1;
    return u;
}

bool paged_encode_cache(CUtensorMap *map, const void *ptr, bool int8, const PagedAttnProblem &p,
                        int box) {
    auto fn = tensor_map_encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(p.P * p.Hkv * p.page)};
    cuuint64_t strides[1] = {int8 ? 128u : 256u};
    cuuint32_t bx[2] = {int8 ? 128u : 64u, static_cast<cuuint32_t>(box)};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void *>(ptr), dims, strides, bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t paged_attn_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv) {
    if (T <= 0 || B <= 0) return 0;
    const size_t row = (kHeadDim + 2) * sizeof(float);
    const size_t few = kMaxCtas * (2 * kRowsMax * row + sizeof(PagedCut));
    // (calls for the tiles kernel may take the rows kernel, by q's strides)
    const size_t many = kPagedTileCtas * (2 * kPagedTileRows * row + sizeof(PagedCut));
    return uses_tiles(T, B, Hq / Hkv) && many > few ? many : few;
}

cudaError_t launch_paged_attention(const PagedAttnProblem &p, cudaStream_t stream) {
    DeviceInfo info;
    cudaError_t e = current_device_info(&info);
    if (e != cudaSuccess) return e;
    unsigned long long *err = nullptr;
    e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    const int64_t G = p.Hq / p.Hkv;
    // (the tiles kernel copies q by tensor map, which takes rows apart from one
    // another; the rows kernel takes any strides)
    if (uses_tiles(p.T, p.B, G) && p.qt >= kHeadDim && p.qh >= kHeadDim) {
        const PagedSetup u = paged_setup(p, kPagedTileRows);
        const int ctas = info.num_sms < kPagedTileCtas ? info.num_sms : kPagedTileCtas;
        e = launch_paged_tiles(p, u, ctas, err, stream);
        if (e != cudaSuccess) return e;
        return launch_combine(u, static_cast<float *>(p.workspace), kPagedTileRows, kPagedTileRows,
                              ctas, stream);
    }
    const bool int8 = p.ks != nullptr;
    CUtensorMap km, vm;
    if (!paged_encode_cache(&km, p.kc, int8, p, rows_box(p)) ||
        !paged_encode_cache(&vm, p.vc, int8, p, rows_box(p)))
        return cudaErrorInvalidValue;
    // An item takes whole tokens: 8 rows when requests have that many on average, else
    // 16 (two tokens of 4 query heads, 32 requests at 4096 positions: 64 us, and 82 in
    // items of 16).
    const bool one = G <= 8 && p.T * G <= 8 * p.B;
    if (int8)
        return one ? launch_rows<1, true>(p, km, vm, info.num_sms, err, stream)
                   : launch_rows<2, true>(p, km, vm, info.num_sms, err, stream);
    return one ? launch_rows<1, false>(p, km, vm, info.num_sms, err, stream)
               : launch_rows<2, false>(p, km, vm, info.num_sms, err, stream);
}

}  // namespace w8a8
