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
constexpr int kRowThreads = (kRowWarps + 1) * 32;   // and a warp that loads
constexpr int kRowStages = 2;
constexpr float kNegInf = -INFINITY;

// The kernel of a call, by the query rows that a request and kv head have on
// average: up to 16 fit one item of the rows kernel, which reads the cache
// once; more take the tiles kernel.
bool uses_tiles(int64_t T, int64_t B, int64_t G) { return T * G > kRowsMax * B; }


// ------------------------------------------------------------ the rows kernel
struct RowsArgs {
    PagedSchedule s;
    PagedCache c;
    PagedOut o;
    const uint16_t *q;      // [T, Hq, 128], token stride qt, head stride qh
    int64_t qt, qh;
    float scale;
    float *ws;
    unsigned long long *err;
};

template <int NT, bool kInt8>
struct RowsSmem {
    struct Stage {
        uint4 k[Tile<kInt8>::kBytes / 16];
        uint4 v[Tile<kInt8>::kBytes / 16];
    };
    Stage stage[kRowStages];                        // 1024-byte aligned
    float ks[kRowStages][kTilePositions], vs[kRowStages][kTilePositions];
    TileMask mask[kRowStages];
    float merge[2][8 * NT * 4][32];                 // two warps' outputs, as fragments
    float red_m[kRowWarps][8 * NT], red_l[kRowWarps][8 * NT];
    uint64_t full[kRowStages], empty[kRowStages];
    volatile int abort_flag;
};

// A lane's fragments of a landed tile (attention_math.cuh: ChunkRegs).
template <bool kInt8>
__device__ __forceinline__ void tile_frags(ChunkRegs<kInt8> &r, const uint4 *k, const uint4 *v,
                                           const float *ks, const float *vs, const TileMask &mask,
                                           bool full, int pw, int gid, int t) {
    using R = ChunkRegs<kInt8>;
    auto at = [](int row, int piece) {
        const int half = piece >> 3;
        return (half * kTilePositions + row) * 8 + ((piece & 7) ^ (row & 7));
    };
    auto ok = [&](int row) { return full || ((mask.w[row >> 5] >> (row & 31)) & 1u); };
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int row = pw + 16 * mt + gid + 8 * hf;
#pragma unroll
            for (int x = 0; x < R::KV; ++x) r.k[mt][hf][x] = k[at(row, t * R::KV + x)];
            if constexpr (kInt8) {
                r.ks[mt][hf] = ks[row];
                r.vs[mt][hf] = ok(row) ? vs[row] : 0.0f;
            } else {
                r.ks[mt][hf] = 1.0f;
                r.vs[mt][hf] = ok(row) ? 1.0f : 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = pw + 16 * mt + 2 * t + (j < 2 ? j : j + 6);
#pragma unroll
            for (int x = 0; x < R::VV; ++x) {
                r.v[mt][j][x] = v[at(row, gid * R::VV + x)];
                // what lies in a masked BF16 position may be no number at all
                if (!kInt8 && !ok(row)) r.v[mt][j][x] = make_uint4(0, 0, 0, 0);
            }
        }
    }
}

// A persistent CTA: four warps of 32 positions of a tile each, and one that
// keeps tiles in flight. Query row r of an item is query head r % G of its new
// token r / G. Arithmetic as in the contiguous-cache kernel (attention.cu):
// scores and outputs by mma.sync with FP32 sums, the probabilities split into
// two fp16 (three bf16) parts, running maximum and sum per warp, joined when
// the item ends.
template <int NT, bool kInt8>
__global__ void __launch_bounds__(kRowThreads)
paged_rows_kernel(const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                  const RowsArgs a) {
    extern __shared__ uint8_t smem_raw[];
    using Smem = RowsSmem<NT, kInt8>;
    Smem &sm = *reinterpret_cast<Smem *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, t = lane & 3;
    const PagedSchedule &s = a.s;
    if (tid == 0) {
        for (int i = 0; i < kRowStages; ++i) {
            mbar_init(smem_u32(&sm.full[i]), 1);
            mbar_init(smem_u32(&sm.empty[i]), kRowWarps * 32);
        }
        sm.abort_flag = 0;
        fence_mbarrier_init();
    }
    griddep_launch_dependents();
    griddep_wait();   // lengths, tables and the cache may come from the kernel before
    const PagedShare sh = paged_share<kRowThreads>(s, blockIdx.x, gridDim.x);   // (synchronises)
    if (static_cast<int>(blockIdx.x) >= sh.ctas) return;
    PagedWalk w;
    w.start(s, sh);
    uint32_t it = 0;   // tiles so far: stage it % kRowStages, phase it / kRowStages
    bool ok = true;

    if (warp == kRowWarps) {
        for (; !w.done(s, sh.end); w.next(s)) {
            const PagedPiece p = paged_piece(s, w, sh.begin, sh.end);
            int lo, hi;
            request_span(s, w.r, lo, hi);
            for (int x = p.first; x < p.last; ++x, ++it) {
                const int st = it % kRowStages;
                if (ok && it >= kRowStages)
                    ok = mbar_wait(smem_u32(&sm.empty[st]), (it / kRowStages - 1) & 1, &sm.abort_flag,
                                   a.err, ROLE_PRODUCER, 1, kWaitLimitNs, KID_ATTN);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const TileBoxes tb = find_boxes(a.c, w.b, w.h, p.tile0 + x, lo, hi, a.err);
                const uint32_t bar = smem_u32(&sm.full[st]);
                if (lane == 0) {
                    sm.mask[st] = tb.mask;
                    mbar_arrive_expect_tx(bar, 2 * tile_bytes<kInt8>(a.c, tb) +
                                                   (kInt8 ? 2 * scale_bytes(a.c, tb) : 0));
                }
                __syncwarp();
                copy_boxes<kInt8>(a.c, tb, &km, smem_u32(sm.stage[st].k), bar);
                copy_boxes<kInt8>(a.c, tb, &vm, smem_u32(sm.stage[st].v), bar);
                if constexpr (kInt8) {
                    copy_scales(a.c, tb, a.c.ks, smem_u32(sm.ks[st]), bar);
                    copy_scales(a.c, tb, a.c.vs, smem_u32(sm.vs[st]), bar);
                }
            }
            if (!ok) break;
        }
        // nothing may be in flight when the CTA ends
        if (!ok)
            for (uint32_t x = it > kRowStages ? it - kRowStages : 0; x < it; ++x)
                mbar_wait(smem_u32(&sm.full[x % kRowStages]), (x / kRowStages) & 1, &sm.abort_flag,
                          a.err, ROLE_PRODUCER, 2, kWaitLimitNs, KID_ATTN);
        return;
    }

    const int pw = warp * 32;
    for (; !w.done(s, sh.end); w.next(s)) {
        const PagedPiece p = paged_piece(s, w, sh.begin, sh.end);
        if (p.first == p.last && !p.whole) continue;
        const int rows = p.ntok * a.o.G;
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
                const uint4 y = use ? __ldg(src + x) : make_uint4(0, 0, 0, 0);
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
                for (int x = 0; x < 16; ++x) mq = __vmaxu2(mq, qf[nt][x] & 0x7FFF7FFFu);
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

        for (int x = p.first; x < p.last; ++x, ++it) {
            const int sg = it % kRowStages;
            if (ok)
                ok = mbar_wait(smem_u32(&sm.full[sg]), (it / kRowStages) & 1, &sm.abort_flag, a.err,
                               ROLE_EPILOGUE, 3, kWaitLimitNs, KID_ATTN);
            __syncwarp();
            const TileMask m = sm.mask[sg];
            const bool full = (m.w[0] & m.w[1] & m.w[2] & m.w[3]) == 0xFFFFFFFFu;
            ChunkRegs<kInt8> r;
            tile_frags<kInt8>(r, sm.stage[sg].k, sm.stage[sg].v, sm.ks[sg], sm.vs[sg], m, full, pw,
                              gid, t);
            mbar_arrive(smem_u32(&sm.empty[sg]));
            const int c0 = (p.tile0 + x) * kTilePositions;
            const bool plain = full && c0 + kTilePositions - 1 <= pos_first &&
                               (s.window == 0 || c0 > pos_last - s.window);
            if (plain) {
                attend_chunk<NT, kInt8>(
                    st, r, qf, [](int, int, int) { return true; }, a.scale, qinv, pw, gid, t);
            } else {
                const uint32_t mw = m.w[warp];   // this warp's 32 positions
                attend_chunk<NT, kInt8>(
                    st, r, qf,
                    [&](int row, int nt, int j) {
                        return ((mw >> (row - pw)) & 1u) && c0 + row < upto[nt][j] &&
                               c0 + row >= from[nt][j];
                    },
                    a.scale, qinv, pw, gid, t);
            }
        }

        // ---- join the four warps: every warp's state weighted by
        // e^(its max - the item's max); warps 2, 3 into 0, 1, then 1 into 0
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
        named_barrier_sync(1, kRowWarps * 32);
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
                    l[nt][j] += sm.red_l[x][r] * expf(sm.red_m[x][r] - mu);
                const float f = unit * expf(st.m[nt][j] - mu);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    st.o[i][nt][j] *= f;
                    st.o[i][nt][j + 2] *= f;
                }
            }
#pragma unroll
        for (int step = 2; step > 0; step >>= 1) {
            if (warp >= step && warp < 2 * step) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sm.merge[warp - step][(i * NT + nt) * 4 + k][lane] = st.o[i][nt][k];
            }
            named_barrier_sync(1, kRowWarps * 32);
            if (warp < step) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st.o[i][nt][k] += sm.merge[warp][(i * NT + nt) * 4 + k][lane];
            }
            named_barrier_sync(1, kRowWarps * 32);
        }
        if (warp != 0 || !ok) continue;
        // lane (gid, t) has dims [16 gid, 16 gid + 16) of rows 8 nt + 2 t + j:
        // fragment i, elements j and j + 2 are dims 2 i and 2 i + 1 of them
        float *part = slot_of(a.ws, kRowsMax, blockIdx.x, p.slot);
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
                if (!p.whole) {
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
                const int64_t orow = out_row(a.o, w.r, w.h, p.tok0, r);
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
}

// ------------------------------------------------------------------- combine
constexpr int kCombineThreads = 128;

struct CombineArgs {
    PagedSchedule s;
    PagedOut o;
    const float *ws;
    int rows;               // rows of a slot
    int max_ctas;           // the attention kernel's grid
};

// Block (c, y): when the border before CTA c is the first one inside an item,
// joins the item's shares for rows 4 y + warp, + 4 gridDim.y, ... The other
// blocks find that out and end. Blocks also write zeros to rows of tokens that
// belong to no request.
__global__ void __launch_bounds__(kCombineThreads)
paged_combine_kernel(const CombineArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const PagedSchedule &s = a.s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    {
        const int64_t first = min(max(s.cu[0], 0), s.T), last = min(max(s.cu[s.B], 0), s.T);
        const int64_t per = static_cast<int64_t>(a.o.Hq) * kHeadDim * (a.o.fp32 ? 4 : 2) / 16;
        const int64_t n = (first + s.T - last) * per;
        uint4 *out = static_cast<uint4 *>(a.o.out);
        const int64_t stride = static_cast<int64_t>(gridDim.x) * gridDim.y * kCombineThreads;
        for (int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kCombineThreads +
                         threadIdx.x;
             i < n; i += stride)
            out[i < first * per ? i : i - first * per + last * per] = make_uint4(0, 0, 0, 0);
    }
    const int c = blockIdx.x + 1;   // (the first CTA's border cuts nothing)
    const PagedShare sh = paged_share<kCombineThreads>(s, c, a.max_ctas);
    if (c >= sh.ctas || sh.b >= s.B) return;
    PagedWalk w;
    w.start(s, sh);
    if (w.at >= sh.begin) return;                                  // between two items
    if (paged_border(sh.total, sh.ctas, c - 1) > w.at) return;     // an earlier border cut it first
    // the last CTA that has a share of the item
    int end = c;
    while (end + 1 < sh.ctas && paged_border(sh.total, sh.ctas, end + 1) < w.at + w.cost) ++end;
    const PagedPiece first = paged_piece(s, w, paged_border(sh.total, sh.ctas, c - 1), sh.begin);
    if (first.ntiles == 0) return;                                 // its zeros are written
    const int rows = first.ntok * a.o.G;
    for (int r = blockIdx.y * (kCombineThreads / 32) + warp; r < rows;
         r += gridDim.y * (kCombineThreads / 32)) {
        float m = kNegInf, l = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bool whole = false;
        for (int k = c - 1; k <= end && !whole; ++k) {
            const PagedPiece p = paged_piece(s, w, paged_border(sh.total, sh.ctas, k),
                                             paged_border(sh.total, sh.ctas, k + 1));
            whole = p.whole;
            if (p.first == p.last) continue;
            const float *part =
                a.ws + (static_cast<int64_t>(k) * 2 + p.slot) * a.rows * (kHeadDim + 2);
            const float pm = part[a.rows * kHeadDim + r], pl = part[a.rows * (kHeadDim + 1) + r];
            const float4 v = reinterpret_cast<const float4 *>(part + r * kHeadDim)[lane];
            const float mn = fmaxf(m, pm);
            const float mu = mn == kNegInf ? 0.0f : mn;
            const float fo = expf(m - mu), fn = expf(pm - mu);
            m = mn;
            l = l * fo + pl * fn;
            acc.x = acc.x * fo + v.x * fn;
            acc.y = acc.y * fo + v.y * fn;
            acc.z = acc.z * fo + v.z * fn;
            acc.w = acc.w * fo + v.w * fn;
        }
        if (whole) return;                                         // one CTA wrote the item
        const int64_t orow = out_row(a.o, w.r, w.h, first.tok0, r);
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

cudaError_t launch_combine(const PagedSchedule &s, const PagedOut &o, const float *ws, int rows,
                           int max_ctas, cudaStream_t stream) {
    CombineArgs a;
    a.s = s;
    a.o = o;
    a.ws = ws;
    a.rows = rows;
    a.max_ctas = max_ctas;
    const unsigned y = rows <= 16 ? 2 : 8;
    return launch_pdl(paged_combine_kernel, dim3(max_ctas, y), kCombineThreads, 0, stream, a);
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
    const PagedSetup u = paged_setup(p, 8 * NT);
    a.s = u.s;
    a.c = u.c;
    a.o = u.o;
    a.q = p.q;
    a.qt = p.qt;
    a.qh = p.qh;
    a.scale = p.scale;
    a.ws = static_cast<float *>(p.workspace);
    a.err = err;
    e = launch_pdl(kernel, dim3(ctas), kRowThreads, smem, stream, km, vm, a);
    if (e != cudaSuccess) return e;
    return launch_combine(a.s, a.o, a.ws, kRowsMax, ctas, stream);
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
    // (the tiles kernel's start and end of an item take about as long as 3.75 tiles)
    u.s.overhead = rows == kPagedTileRows ? 15 * kTilePositions / 4 : kTilePositions;
    u.s.min_share = 2 * kTilePositions;
    u.c.table = p.block_table;
    u.c.ks = p.ks;
    u.c.vs = p.vs;
    u.c.W = static_cast<int>(p.W);
    u.c.P = static_cast<int>(p.P);
    u.c.Hkv = static_cast<int>(p.Hkv);
    u.c.page = static_cast<int>(p.page);
    u.c.box = gcd(u.c.page, kTilePositions);
    return u;
}

bool paged_encode_cache(CUtensorMap *map, const void *ptr, bool int8, const PagedAttnProblem &p) {
    auto fn = tensor_map_encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(p.P * p.Hkv * p.page)};
    cuuint64_t strides[1] = {int8 ? 128u : 256u};
    cuuint32_t bx[2] = {int8 ? 128u : 64u,
                        static_cast<cuuint32_t>(gcd(static_cast<int>(p.page), kTilePositions))};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void *>(ptr), dims, strides, bx, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t paged_attn_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv) {
    if (T <= 0 || B <= 0) return 0;
    const size_t slots = uses_tiles(T, B, Hq / Hkv)
                             ? static_cast<size_t>(kPagedTileCtas) * 2 * kPagedTileRows
                             : static_cast<size_t>(kMaxCtas) * 2 * kRowsMax;
    return slots * (kHeadDim + 2) * sizeof(float);
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
        return launch_combine(u.s, u.o, static_cast<float *>(p.workspace), kPagedTileRows, ctas,
                              stream);
    }
    const bool int8 = p.ks != nullptr;
    CUtensorMap km, vm;
    if (!paged_encode_cache(&km, p.kc, int8, p) || !paged_encode_cache(&vm, p.vc, int8, p))
        return cudaErrorInvalidValue;
    // An item takes whole tokens: 8 rows when the group fits and the call has
    // about one token per request, else 16.
    const bool one = G <= 8 && p.T <= p.B;
    if (int8)
        return one ? launch_rows<1, true>(p, km, vm, info.num_sms, err, stream)
                   : launch_rows<2, true>(p, km, vm, info.num_sms, err, stream);
    return one ? launch_rows<1, false>(p, km, vm, info.num_sms, err, stream)
               : launch_rows<2, false>(p, km, vm, info.num_sms, err, stream);
}

}  // namespace w8a8
