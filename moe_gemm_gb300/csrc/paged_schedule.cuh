// How the work of one paged-attention call is shared out over a persistent
// grid, worked out on the device from the request lengths (the host never
// reads them).
//
// An item is (request, kv head, tile of whole new tokens): its query rows, and
// the 128-position tiles of the cache that they see. Items are laid on a line
// in order, each as long as its cost (about the positions it reads, plus a
// constant for its start and end); CTA c of C takes the c-th C-th of the
// line. An item that a border cuts is shared by the CTAs on both sides: its
// cache tiles are divided in proportion, every share's running softmax state
// goes to the workspace, and the combine kernel joins them. A CTA is cut at
// most twice, so the workspace depends on the grid, not on the lengths.
//
// The cost needs to be the same function everywhere, not exact, so it has a
// closed form: the start of any CTA's share takes one scan over the requests
// and one binary search.
#pragma once

#include <cstdint>

namespace w8a8 {

constexpr int kTilePositions = 128;

struct PagedSchedule {
    const int32_t *cu;      // [B + 1] first new token of each request
    const int32_t *kv;      // [B] positions, the new tokens' included
    int B, T, Hkv;
    int tile_tokens;        // new tokens per item
    int window;             // 0: none
    int64_t capacity;       // positions a block table row can hold
    int overhead;           // cost of an item beside its positions
    int min_share;          // least cost worth a CTA of its own
};

struct PagedRequest {
    int n, t0, kv;          // new tokens, the first one's row, positions
    int base;               // position of the first new token (< 0: rows that see nothing)
    int tiles;              // items per kv head
    long long b0;
};

__device__ __forceinline__ PagedRequest paged_request(const PagedSchedule &s, int b) {
    PagedRequest r;
    const int a = min(max(s.cu[b], 0), s.T), z = min(max(s.cu[b + 1], a), s.T);
    r.t0 = a;
    r.n = z - a;
    r.kv = static_cast<int>(min(static_cast<int64_t>(max(s.kv[b], 0)), s.capacity));
    r.base = r.kv - r.n;
    r.b0 = max(r.base, 0);
    r.tiles = (r.n + s.tile_tokens - 1) / s.tile_tokens;
    return r;
}

// Cost of a request's first m items of one kv head: item i reads about
// min(b0 + (i + 1) tile, window + tile) positions.
__device__ __forceinline__ long long paged_cum(const PagedSchedule &s, const PagedRequest &r,
                                               int m) {
    const long long tt = s.tile_tokens;
    long long grow = m;     // items not yet limited by the window
    if (s.window > 0) {
        grow = r.b0 > s.window ? 0 : (s.window - r.b0) / tt + 1;
        grow = min(grow, static_cast<long long>(m));
    }
    return grow * (s.overhead + r.b0) + tt * (grow * (grow + 1) / 2) +
           (m - grow) * (s.overhead + s.window + tt);
}

struct PagedShare {
    long long total, begin, end;   // on the line
    int ctas;                      // CTAs that take part
    int b;                         // the request that begin falls in
    long long off;                 // and how far into it
};

__device__ __forceinline__ long long paged_border(long long total, int ctas, int c) {
    return c >= ctas ? total : total * c / ctas;   // (total < 2^50, c < 2^10)
}

// The share of CTA `cta` (for the combine: the border where it begins). Every
// thread of the block calls it; THREADS is the block size.
template <int THREADS>
__device__ PagedShare paged_share(const PagedSchedule &s, int cta, int max_ctas) {
    __shared__ long long s_part[THREADS / 32];
    __shared__ PagedShare s_share;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (s.B + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, s.B), b1 = min(b0 + per, s.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const PagedRequest r = paged_request(s, b);
        mine += paged_cum(s, r, r.tiles) * s.Hkv;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) s_part[warp] = incl;
    if (tid == 0) s_share.b = s.B;
    __syncthreads();
    long long base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += s_part[w];
        total += s_part[w];
    }
    const long long first = base + incl - mine;
    const long long want = max(total / s.min_share, 1ll);
    const int ctas = static_cast<int>(min(want, static_cast<long long>(max_ctas)));
    const long long begin = paged_border(total, ctas, cta);
    if (cta < ctas && begin >= first && begin < first + mine) {
        long long at = first;
        for (int b = b0; b < b1; ++b) {
            const PagedRequest r = paged_request(s, b);
            const long long c = paged_cum(s, r, r.tiles) * s.Hkv;
            if (begin < at + c) {
                s_share.b = b;
                s_share.off = begin - at;
                break;
            }
            at += c;
        }
    }
    __syncthreads();
    PagedShare out;
    out.total = total;
    out.ctas = ctas;
    out.begin = begin;
    out.end = cta < ctas ? paged_border(total, ctas, cta + 1) : begin;
    out.b = s_share.b;
    out.off = s_share.off;
    return out;
}

// Walks the items from the one that holds a position of the line.
struct PagedWalk {
    PagedRequest r;
    int b, h, i;
    long long at, cost;     // the item's place on the line

    __device__ __forceinline__ void start(const PagedSchedule &s, const PagedShare &sh) {
        b = sh.b;
        at = sh.begin;
        if (b >= s.B) return;
        r = paged_request(s, b);
        const long long head = paged_cum(s, r, r.tiles);
        h = static_cast<int>(sh.off / head);
        const long long rem = sh.off - h * head;
        int lo = 0, hi = r.tiles;   // the last item that begins at or before rem
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (paged_cum(s, r, mid) <= rem) lo = mid;
            else hi = mid;
        }
        i = lo;
        at = sh.begin - (rem - paged_cum(s, r, lo));
        cost = paged_cum(s, r, lo + 1) - paged_cum(s, r, lo);
    }
    __device__ __forceinline__ void next(const PagedSchedule &s) {
        at += cost;
        if (++i == r.tiles) {
            i = 0;
            if (++h == s.Hkv) {
                h = 0;
                do {
                    if (++b >= s.B) return;
                    r = paged_request(s, b);
                } while (r.n == 0);
            }
        }
        cost = paged_cum(s, r, i + 1) - paged_cum(s, r, i);
    }
    __device__ __forceinline__ bool done(const PagedSchedule &s, long long end) const {
        return b >= s.B || at >= end;
    }
};

// What the combine kernel needs of an item that a border cuts: written, for the
// first border inside the item, by the CTA that begins there.
struct PagedCut {
    long long total, at, cost;   // of the line, and the item's place on it
    int ctas, ntiles;            // ntiles 0: this border is not the first inside an item
    int t0, tok0, ntok, h;       // the item
};

// One CTA's part of an item.
struct PagedPiece {
    int tok0, ntok;         // the item's new tokens within the request
    int tile0, ntiles;      // the cache tiles that the item sees
    int first, last;        // this piece: tiles [tile0 + first, tile0 + last)
    bool whole;             // no other CTA has a part of the item
    int slot;               // the CTA's workspace slot for it
};

// The part of an item of `ntiles` cache tiles that lies in [begin, end). The item's
// constant cost lies at its front and a border goes to the nearest tile: every CTA has
// one piece more than item fronts, so CTAs differ by a tile at most.
__device__ __forceinline__ void paged_part(PagedPiece &p, long long at, long long cost, int overhead,
                                           long long begin, long long end) {
    const long long x0 = max(begin - at, 0ll), x1 = min(end - at, cost);
    const long long tiles = cost - overhead;
    auto before = [&](long long x) {
        return x <= overhead ? 0 : static_cast<int>(((x - overhead) * p.ntiles + tiles / 2) / tiles);
    };
    p.first = before(x0);
    p.last = x1 == cost ? p.ntiles : before(x1);
    p.whole = p.first == 0 && p.last == p.ntiles && (p.ntiles > 0 || x0 == 0);
    p.slot = x0 > 0 ? 0 : 1;
}

__device__ __forceinline__ PagedPiece paged_piece(const PagedSchedule &s, const PagedWalk &w,
                                                  long long begin, long long end) {
    PagedPiece p;
    p.tok0 = w.i * s.tile_tokens;
    p.ntok = min(w.r.n - p.tok0, s.tile_tokens);
    const int hi = max(w.r.base + p.tok0 + p.ntok, 0);
    const int lo = s.window > 0 ? max(max(w.r.base + p.tok0, 0) - s.window + 1, 0) : 0;
    p.tile0 = lo / kTilePositions;
    p.ntiles = hi > lo ? (hi + kTilePositions - 1) / kTilePositions - p.tile0 : 0;
    paged_part(p, w.at, w.cost, s.overhead, begin, end);
    return p;
}

// Called by one thread of every CTA of the attention kernel.
__device__ __forceinline__ void paged_write_cut(const PagedSchedule &s, const PagedShare &sh,
                                                const PagedWalk &w, int cta, PagedCut *cuts) {
    PagedCut c;
    c.ntiles = 0;
    if (cta > 0 && cta < sh.ctas && w.b < s.B && w.at < sh.begin &&
        paged_border(sh.total, sh.ctas, cta - 1) <= w.at) {
        const PagedPiece p = paged_piece(s, w, sh.begin, sh.end);
        c.total = sh.total;
        c.at = w.at;
        c.cost = w.cost;
        c.ctas = sh.ctas;
        c.ntiles = p.ntiles;
        c.t0 = w.r.t0;
        c.tok0 = p.tok0;
        c.ntok = p.ntok;
        c.h = w.h;
    }
    cuts[cta] = c;
}

}  // namespace w8a8
