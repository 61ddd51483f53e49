// The router's gate, on sm_103a: from the router's logits x [T, E] to the
// top-k expert ids and weights that the expert FFN takes ("Deploying Hunyuan
// 770B in INT8 on domestic accelerators", §1.3: each token goes to the experts
// its router picked).
//
//   score  s = softmax(x) or 1 / (1 + e^-x); key = s + bias (s without a bias);
//   groups the E experts form n_group equal runs; a group's score is its largest
//          key (with a bias, the sum of its two largest); the topk_group best
//          groups stay;
//   pick   the k largest keys of the groups that stay, largest first, ties to
//          the lower expert;
//   weight s of the picked (renormalize: over their sum), times a factor.
//
// One warp per token. Lane l holds experts [V l, V l + V), so a token's logits
// are one coalesced read, lane order is expert order (a tie goes to the first
// lane that holds the maximum) and, in the usual layouts, a group is a run of
// lanes. A pick is one warp-wide unsigned maximum (redux) over keys mapped to
// ordered integers.
//
// Whole numbers depend on comparisons, so they are made exact:
//  * without a bias the logits themselves are compared: softmax and sigmoid
//    keep their order;
//  * with a bias, keys in 32 bits decide unless two compared keys are closer
//    than their error bound; such a token (43 of 16384 with 256 experts and random
//    logits) is decided again with scores in 64 bits.
//
// What bounds it: instructions. 16384 x 256 FP32 logits, sigmoid with a bias, 4 of 8
// groups, top 8, take 21.6 us (0.8 TB/s; the copy of its bytes takes 2.6), 15 without
// the tokens decided again, of which one that starts late ends the call. Softmax with a
// bias takes 35 (30 without groups): its close tokens take all experts' scores in 64 bits. Rows
// that a persistent warp reads ahead took 8 us more (the registers halve the warps of an
// SM), the 64-bit part out of line 3.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"

namespace w8a8 {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kGateWarps = 4;

// Ordered integers: a < b as numbers <=> ord(a) < ord(b); 0 is kept for "not
// available" (the mapping of -infinity is above 0). -0 counts as +0.
__device__ __forceinline__ uint32_t ord(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t ord(double v) {
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ float unord(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ double unord(uint64_t k) {
    return __longlong_as_double(static_cast<long long>((k >> 63) ? k & 0x7FFFFFFFFFFFFFFFull : ~k));
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(kFull, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = static_cast<uint32_t>(v >> 32);
    const uint32_t mh = __reduce_max_sync(kFull, hi);
    const uint32_t ml = __reduce_max_sync(kFull, hi == mh ? static_cast<uint32_t>(v) : 0u);
    return (static_cast<uint64_t>(mh) << 32) | ml;
}

template <typename R>
struct KeyOf;
template <>
struct KeyOf<float> { using type = uint32_t; };
template <>
struct KeyOf<double> { using type = uint64_t; };

// (Ordinary loads, here and below: the kernel before may have written the logits while
// this one had started already, and read-only loads are for what nobody writes as long as
// a kernel lives.)
__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t *p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

struct GateArgs {
    const float *bias;
    int vec;                // rows and bias may be read 16 bytes at a time
    int64_t ldx;
    int T, E, k, n_group, topk_group;
    int size;               // experts of a group
    int run_shift;          // log2 of the lanes of a group, -1: groups are not such runs
    int sigmoid, renormalize;
    float scale;
    int32_t *ids;
    float *w;
};

__device__ __forceinline__ float ex2_approx(float v) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float rcp_approx(float v) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}

// Out of line: it runs for few tokens, and once per expert of a lane.
__device__ __noinline__ double exp_f64(double v) { return exp(v); }

// A lane's V logits (-inf past the last expert).
template <int V>
__device__ __forceinline__ void load_row(const float *row, const GateArgs &a, int lane, float (&x)[V]) {
    if constexpr (V >= 4) {
        if (a.vec) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (lane * V + i < a.E) v = *reinterpret_cast<const float4 *>(row + lane * V + i);
                x[i] = v.x;
                x[i + 1] = v.y;
                x[i + 2] = v.z;
                x[i + 3] = v.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = lane * V + i < a.E ? row[lane * V + i] : -INFINITY;
}
template <int V>
__device__ __forceinline__ void load_row(const uint16_t *row, const GateArgs &a, int lane,
                                         float (&x)[V]) {
    if constexpr (V >= 8) {
        if (a.vec) {
#pragma unroll
            for (int i = 0; i < V; i += 8) {
                uint4 v = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
                if (lane * V + i < a.E) v = *reinterpret_cast<const uint4 *>(row + lane * V + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i + 2 * j] = __uint_as_float(w[j] << 16);
                    x[i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = lane * V + i < a.E ? load_logit(row + lane * V + i) : -INFINITY;
}

// The picks of one token: pick j is held by lane j & 31, in element j >> 5 (-1:
// none).
struct Picks {
    int id[2];
};

// The two largest of the union of {a1 >= a2} and {b1 >= b2}.
template <typename R>
__device__ __forceinline__ void top2_merge(R &a1, R &a2, R b1, R b2) {
    const R lo = fmin(a1, b1);
    a1 = fmax(a1, b1);
    a2 = fmax(lo, fmax(a2, b2));
}

// Which groups stay (bit g of kept), from their scores (lane l: groups l and l +
// 32).
template <typename R>
__device__ __forceinline__ void rank_groups(const R (&gs)[2], const GateArgs &a, int lane,
                                            unsigned (&kept)[2]) {
    // rank of each group: those with a larger score, or an equal one and a lower index
    int rank[2] = {0, 0};
    if (a.n_group <= 32) {
        for (int g = 0; g < a.n_group; ++g) {
            const R s = __shfl_sync(kFull, gs[0], g);
            rank[0] += (s > gs[0] || (s == gs[0] && g < lane)) ? 1 : 0;
        }
    } else {
        for (int g = 0; g < a.n_group; ++g) {
            const R s = __shfl_sync(kFull, g < 32 ? gs[0] : gs[1], g & 31);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                rank[h] += (s > gs[h] || (s == gs[h] && g < lane + 32 * h)) ? 1 : 0;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        kept[h] = __ballot_sync(kFull, lane + 32 * h < a.n_group && rank[h] < a.topk_group);
}

// The last group kept and the first one left out, over the groups of all lanes, each
// score at its worst: off by tol / 2, relative to 1 and to the sum of the
// magnitudes of the keys in it (they may cancel: the error goes by them, not by the score).
struct GroupBorder {
    float in = INFINITY, out = -INFINITY;
    __device__ __forceinline__ void add(bool stays, float score, float size, float tol) {
        const float err = 0.5f * tol * fmaxf(1.0f, size);
        const bool known = size < INFINITY;     // (else a sum may have overflowed)
        if (stays) in = fminf(in, known ? score - err : -INFINITY);
        else out = fmaxf(out, known ? score + err : INFINITY);
    }
    // (which of the unavailable groups stay, all -inf, does not matter)
    __device__ __forceinline__ bool clear() const {
        const uint32_t worst_in = __reduce_min_sync(kFull, ord(in));
        const uint32_t best_out = __reduce_max_sync(kFull, ord(out));
        return worst_in > best_out || best_out == ord(-INFINITY);
    }
};

// Marks the experts outside the topk_group best groups as not available
// (kr = -inf there). Returns false when errors within tol (GroupBorder; 0: none) may
// change which those are.
template <typename R, int V>
__device__ __forceinline__ bool keep_groups(R (&kr)[V], const GateArgs &a, int lane, bool sum2,
                                            R tol) {
    const int size = a.size;
    const R none = -INFINITY;
    R gs[2] = {none, none};   // lane l: the scores of groups l and l + 32
    [[maybe_unused]] float size_of[2] = {0.0f, 0.0f};   // and the magnitudes in them
    auto magnitude = [&](R m1, R m2) {
        return m1 > none ? static_cast<float>(fabs(m1) + (sum2 && m2 > none ? fabs(m2) : R(0))) : 0.0f;
    };
    const int run = 1 << max(a.run_shift, 0);
    GroupBorder border;
    unsigned kept[2];
    if (a.run_shift >= 0) {
        // a group is a run of a power of two lanes: every group at once
        R m1 = none, m2 = none;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            m2 = fmax(m2, fmin(m1, kr[i]));
            m1 = fmax(m1, kr[i]);
        }
        for (int o = 1; o < run; o <<= 1)
            top2_merge<R>(m1, m2, __shfl_xor_sync(kFull, m1, o), __shfl_xor_sync(kFull, m2, o));
        const R s = sum2 && m2 > none ? m1 + m2 : m1;
        gs[0] = __shfl_sync(kFull, s, (lane * run) & 31);
        if (lane >= a.n_group) gs[0] = none;
        rank_groups<R>(gs, a, lane, kept);
        const bool stays = (kept[0] >> (lane >> a.run_shift)) & 1u;
#pragma unroll
        for (int i = 0; i < V; ++i) kr[i] = stays ? kr[i] : none;
        if constexpr (sizeof(R) == 4) {
            if (tol > R(0)) {
                if ((lane >> a.run_shift) < a.n_group) border.add(stays, s, magnitude(m1, m2), tol);
                return border.clear();
            }
        }
        return true;
    }
    for (int g = 0; g < a.n_group; ++g) {
        R m1 = none, m2 = none;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            top2_merge<R>(m1, m2, e >= g * size && e < (g + 1) * size ? kr[i] : none, none);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            top2_merge<R>(m1, m2, __shfl_xor_sync(kFull, m1, o), __shfl_xor_sync(kFull, m2, o));
        const R s = sum2 && m2 > none ? m1 + m2 : m1;
        if (lane == (g & 31)) {
            if (g < 32) gs[0] = s;
            else gs[1] = s;
            if (g < 32) size_of[0] = magnitude(m1, m2);
            else size_of[1] = magnitude(m1, m2);
        }
    }
    rank_groups<R>(gs, a, lane, kept);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int g = min((lane * V + i) / size, 63);
        if (!((kept[g >> 5] >> (g & 31)) & 1u)) kr[i] = none;
    }
    if constexpr (sizeof(R) == 4) {
        if (tol > R(0)) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (lane + 32 * h < a.n_group)
                    border.add((kept[h] >> lane) & 1u, gs[h], size_of[h], tol);
            return border.clear();
        }
    }
    return true;
}

// Picks the k largest of the available keys (kr > -inf). Returns false when
// two keys whose order decides are within tol of one another.
template <typename R, int V>
__device__ __forceinline__ bool pick(R (&kr)[V], const GateArgs &a, int lane, R tol, Picks &out,
                                     float &least) {
    using K = typename KeyOf<R>::type;
    K key[V];
    K best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = kr[i] > R(-INFINITY) ? ord(kr[i]) : K(0);
        best = best > key[i] ? best : key[i];
    }
    out.id[0] = out.id[1] = -1;
    float last = INFINITY;
    bool clear = true;
    const int rounds = tol > R(0) ? a.k + 1 : a.k;   // the first key left out decides too
    for (int j = 0; j < rounds; ++j) {
        const K mx = warp_max(best);
        if (mx == 0) break;
        if constexpr (sizeof(K) == 4) {
            if (tol > R(0)) {
                const float v = unord(mx);
                if (last - v <= tol * fmaxf(1.0f, fabsf(v))) clear = false;
                last = v;
                if (j < a.k) least = v;
            }
        }
        if (j == a.k) break;
        const int owner = __ffs(__ballot_sync(kFull, best == mx)) - 1;
        // the owner's first element that holds it, taken out (every lane does the
        // same steps: a branch for one lane costs as many)
        uint32_t held = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) held |= key[i] == mx ? 1u << i : 0u;
        const int at = __ffs(held) - 1;
        const int gone = lane == owner ? at : -1;
        best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            key[i] = i == gone ? K(0) : key[i];
            best = best > key[i] ? best : key[i];
        }
        const int id = __shfl_sync(kFull, lane * V + at, owner);
        if (lane == (j & 31)) {
            if (j < 32) out.id[0] = id;
            else out.id[1] = id;
        }
    }
    return clear;
}

// The same picks by fewer steps: keys as integers whose low log2(V) bits give way to
// the element's place, each lane's sorted once, so that a pick is one redux and one
// step of the owner's list. Returns false when keys that these bits (or, with a
// bias, the tolerance) cannot tell apart may matter; exact: their loss is none
// (BF16 logits).
template <int V>
__device__ __forceinline__ bool pick_sorted(const float (&kr)[V], const GateArgs &a, int lane,
                                            float tol, bool exact, Picks &out, float &least) {
    constexpr uint32_t kPlace = V - 1;
    uint32_t c[V];
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = (ord(kr[i]) & ~kPlace) | (kPlace - i);
    // Batcher's odd-even merge sort, largest first
#pragma unroll
    for (int p = 1; p < V; p <<= 1)
#pragma unroll
        for (int q = p; q >= 1; q >>= 1)
#pragma unroll
            for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i) {
                    const int x = i + j, y = i + j + q;
                    if (y < V && x / (2 * p) == y / (2 * p)) {
                        const uint32_t hi = max(c[x], c[y]), lo = min(c[x], c[y]);
                        c[x] = hi;
                        c[y] = lo;
                    }
                }
    out.id[0] = out.id[1] = -1;
    const uint32_t none = ord(-INFINITY) | kPlace;
    uint32_t last = 0xFFFFFFFFu;
    float last_v = INFINITY;
    bool clear = true;
    for (int j = 0; j <= a.k; ++j) {    // (the first key left out decides too)
        const uint32_t mx = warp_max(c[0]) & ~kPlace;
        if (mx <= none) break;
        if (tol > 0.0f) {
            const float v = unord(mx);
            if (last_v - v <= tol * fmaxf(1.0f, fabsf(v))) clear = false;
            last_v = v;
            if (j < a.k) least = v;
        } else if (!exact && mx == last) {
            clear = false;
        }
        last = mx;
        if (j == a.k) break;
        const int owner = __ffs(__ballot_sync(kFull, (c[0] & ~kPlace) == mx)) - 1;
        const int id = owner * V + static_cast<int>(kPlace - (__shfl_sync(kFull, c[0], owner) & kPlace));
        if (lane == owner) {
#pragma unroll
            for (int i = 0; i + 1 < V; ++i) c[i] = c[i + 1];
            c[V - 1] = 0;
        }
        if (lane == (j & 31)) {
            if (j < 32) out.id[0] = id;
            else out.id[1] = id;
        }
    }
    return clear;
}

// Decides a token with sigmoid scores again in 64 bits, on the experts that can
// matter alone, one per lane (a whole token in 64 bits takes nine microseconds,
// and one such token held up the call): those that are their group's two largest
// within the tolerance, and those that reach `least`, the smallest key that the
// 32-bit choice needed. kr: 32-bit keys, all groups. Returns false when there are
// more than 32 of them, or too few for the groups that stay.
template <int V, typename Tin>
__device__ __forceinline__ bool decide_again(const Tin *row, const float (&kr)[V], const GateArgs &a,
                                          int lane, float tol, float least, int *list, Picks &out) {
    if (a.n_group > 32) return false;
    const int size = a.size;
    const bool groups = a.topk_group < a.n_group;
    unsigned mine = 0;
    if (groups && a.run_shift >= 0) {   // every group at once, as above
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) top2_merge<float>(m1, m2, kr[i], -INFINITY);
        for (int o = 1; o < 1 << a.run_shift; o <<= 1)
            top2_merge<float>(m1, m2, __shfl_xor_sync(kFull, m1, o), __shfl_xor_sync(kFull, m2, o));
        const float bar = m2 > -INFINITY ? m2 - 2.0f * tol * fmaxf(1.0f, fabsf(m2)) : m1;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (kr[i] > -INFINITY && kr[i] >= bar) mine |= 1u << i;
    } else if (groups) {
        for (int g = 0; g < a.n_group; ++g) {
            float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                top2_merge<float>(m1, m2, e >= g * size && e < (g + 1) * size ? kr[i] : -INFINITY,
                                  -INFINITY);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1)
                top2_merge<float>(m1, m2, __shfl_xor_sync(kFull, m1, o), __shfl_xor_sync(kFull, m2, o));
            const float bar = m2 > -INFINITY ? m2 - 2.0f * tol * fmaxf(1.0f, fabsf(m2)) : m1;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                if (e >= g * size && e < (g + 1) * size && kr[i] > -INFINITY && kr[i] >= bar)
                    mine |= 1u << i;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (kr[i] > -INFINITY && kr[i] >= least) mine |= 1u << i;
    int at = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += u;
    }
    const int n = __shfl_sync(kFull, at, 31);
    if (n > 32) return false;
    at -= __popc(mine);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if ((mine >> i) & 1u) list[at++] = lane * V + i;
    __syncwarp();
    const int e = lane < n ? list[lane] : -1;
    const int group = e >= 0 ? e / size : -1;
    double key = -INFINITY;
    if (e >= 0) {
        const float x = fminf(load_logit(row + e), 3.402823466e38f);
        key = 1.0 / (1.0 + exp_f64(-static_cast<double>(x))) + static_cast<double>(a.bias[e]);
    }
    // (The barrier keeps the compiler from putting the exponential off to its uses: with
    // groups such a token took 9 us then, and takes 4.5.)
    __syncwarp();
    if (groups) {
        // The candidates of a group are neighbours: its two largest by doubling, which
        // leaves them with its first lane. Ordered integers: numbers of 64 bits compare
        // at a fraction of their rate.
        uint64_t m1 = e >= 0 ? ord(key) : 0, m2 = 0;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t n1 = __shfl_down_sync(kFull, m1, o), n2 = __shfl_down_sync(kFull, m2, o);
            const int there = __shfl_down_sync(kFull, group, o);
            if (lane + o < 32 && there == group) {
                const uint64_t lo = m1 < n1 ? m1 : n1, second = m2 < n2 ? n2 : m2;
                m1 = m1 < n1 ? n1 : m1;
                m2 = lo < second ? second : lo;
            }
        }
        const int before = __shfl_up_sync(kFull, group, 1);
        uint64_t gs = 0;
        if (e >= 0 && (lane == 0 || before != group)) gs = m2 != 0 ? ord(unord(m1) + unord(m2)) : m1;
        unsigned kept = 0;
#pragma unroll 1
        for (int j = 0; j < a.topk_group; ++j) {
            const uint64_t mx = warp_max(gs);
            if (mx == 0) break;     // the others are empty
            const int owner = __ffs(__ballot_sync(kFull, gs == mx)) - 1;
            kept |= 1u << __shfl_sync(kFull, group, owner);
            if (lane == owner) gs = 0;
        }
        if (e >= 0 && !((kept >> group) & 1u)) key = -INFINITY;
    }
    // enough of those at or above `least` (all of them are here) must be left
    const bool good = key > -INFINITY && key >= static_cast<double>(least) + tol * fmax(1.0, fabs(key));
    if (__popc(__ballot_sync(kFull, good)) < a.k) return false;
    uint64_t left = good ? ord(key) : 0;
    out.id[0] = out.id[1] = -1;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        const uint64_t mx = warp_max(left);
        const int owner = __ffs(__ballot_sync(kFull, left == mx)) - 1;   // (lists rise by expert)
        const int id = __shfl_sync(kFull, e, owner);
        if (lane == owner) left = 0;
        if (lane == j) out.id[0] = id;
    }
    return true;
}

template <int V, typename Tin>
__global__ void __launch_bounds__(kGateWarps * 32)
moe_gate_kernel(const Tin *logits, const GateArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ int s_list[kGateWarps][32];
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const Tin *row = logits + t * a.ldx;
    // logits: NaN and -inf mark experts that are never picked; +inf counts as
    // the largest finite number
    float x[V];
    load_row<V>(row, a, lane, x);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = x[i] == x[i] ? fminf(x[i], 3.402823466e38f) : -INFINITY;
        m = fmaxf(m, x[i]);
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    }
    if (m == -INFINITY) m = 0.0f;   // no expert is available
    // sum of e^(x - m): softmax's denominator
    float sum = 1.0f;
    if (!a.sigmoid && (a.bias != nullptr || !a.renormalize)) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += expf(x[i] - m);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
    }
    Picks p;
    float least = -INFINITY;    // the smallest 32-bit key picked
    if (a.bias == nullptr) {
        float kr[V];
#pragma unroll
        for (int i = 0; i < V; ++i) kr[i] = x[i];
        if (a.topk_group < a.n_group) keep_groups<float, V>(kr, a, lane, false, 0.0f);
        if (!pick_sorted<V>(kr, a, lane, 0.0f, sizeof(Tin) == 2, p, least))
            pick<float, V>(kr, a, lane, 0.0f, p, least);
    } else {
        // A 32-bit key is off by at most: sigmoid, by the hardware's power of two
        // and reciprocal (2^-22 each, of a number <= 1), the argument's rounding
        // (|x| 2^-24 s (1 - s) < 2^-25) and the sum's; softmax, by those of its sum of E
        // terms as well, relative to the score. 2^-19 and 2^-18 cover twice that
        // (two keys compared).
        // The places in the keys' low bits take 2^-23 V more of each.
        const float tol = (a.sigmoid ? 0x1p-19f : 0x1p-19f + 0x1p-18f / fmaxf(sum, 1.0f)) + V * 0x1p-22f;
        const float inv = __fdiv_rn(1.0f, sum);
        float kr[V], bias[V];
        load_row<V>(a.bias, a, lane, bias);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float s = a.sigmoid ? rcp_approx(1.0f + ex2_approx(-1.44269504f * x[i]))
                                      : expf(x[i] - m) * inv;
            const float key = s + bias[i];
            kr[i] = x[i] > -INFINITY && key == key ? key : -INFINITY;   // (a NaN bias: never picked)
        }
        float all[V];
#pragma unroll
        for (int i = 0; i < V; ++i) all[i] = kr[i];
        bool clear = true;
        if (a.topk_group < a.n_group)
            clear = keep_groups<float, V>(kr, a, lane, true, 2.0f * tol);
        clear = pick_sorted<V>(kr, a, lane, tol, false, p, least) && clear;
        if (!clear && a.sigmoid)   // (the same in every lane)
            clear = decide_again<V>(row, all, a, lane, tol,
                                    least - 2.0f * tol * fmaxf(1.0f, fabsf(least)), s_list[threadIdx.x >> 5],
                                    p);
        if (!clear) {
            double kd[V];
            double dsum = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                kd[i] = exp_f64(a.sigmoid ? -static_cast<double>(x[i])
                                          : static_cast<double>(x[i]) - static_cast<double>(m));
                dsum += kd[i];
            }
            if (!a.sigmoid) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) dsum += __shfl_xor_sync(kFull, dsum, o);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                const double s = a.sigmoid ? 1.0 / (1.0 + kd[i]) : kd[i] / dsum;
                const double key = s + static_cast<double>(e < a.E ? a.bias[e] : 0.0f);
                // (a NaN must not reach the groups' maxima, which would take it for a number)
                kd[i] = x[i] > -INFINITY && key == key ? key : -INFINITY;
            }
            if (a.topk_group < a.n_group) keep_groups<double, V>(kd, a, lane, true, 0.0);
            pick<double, V>(kd, a, lane, 0.0, p, least);
        }
    }
    // weights. Renormalised softmax: e^(x - x_max) over the picked; sigmoid as
    // e^min(x, 0) / (1 + e^-|x|), with the common factor e^r taken out before
    // it can underflow (r = 0 when any picked logit is positive).
    float xm = -INFINITY;
    float px[2];
    const int parts = a.k > 32 ? 2 : 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        px[h] = 0.0f;
        if (h >= parts || p.id[h] < 0) continue;
        px[h] = fminf(load_logit(row + p.id[h]), 3.402823466e38f);
        xm = fmaxf(xm, px[h]);
    }
    if (a.renormalize) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) xm = fmaxf(xm, __shfl_xor_sync(kFull, xm, o));
    }
    const float r = a.sigmoid ? (a.renormalize ? fminf(xm, 0.0f) : 0.0f)
                              : (a.renormalize ? xm : m);
    float num[2], den = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        num[h] = 0.0f;
        if (h >= parts || p.id[h] < 0) continue;
        if (a.sigmoid)
            num[h] = __fdividef(expf(fminf(px[h], 0.0f) - r), 1.0f + expf(-fabsf(px[h])));
        else
            num[h] = expf(px[h] - r);
        den += num[h];
    }
    if (a.renormalize) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) den += __shfl_xor_sync(kFull, den, o);
    } else {
        den = a.sigmoid ? 1.0f : sum;
    }
    const float f = __fdiv_rn(a.scale, den);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int j = lane + 32 * h;
        if (h < parts && j < a.k) {
            a.ids[t * a.k + j] = p.id[h];
            a.w[t * a.k + j] = p.id[h] >= 0 ? num[h] * f : 0.0f;
        }
    }
}

template <int V, typename Tin>
cudaError_t launch_v(const Tin *x, const GateArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.T + kGateWarps - 1) / kGateWarps));
    cfg.blockDim = dim3(kGateWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, moe_gate_kernel<V, Tin>, x, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <typename Tin>
cudaError_t launch_any(const void *logits, const GateArgs &a, cudaStream_t stream) {
    const Tin *x = static_cast<const Tin *>(logits);
    if (a.E <= 32) return launch_v<1>(x, a, stream);
    if (a.E <= 64) return launch_v<2>(x, a, stream);
    if (a.E <= 128) return launch_v<4>(x, a, stream);
    if (a.E <= 256) return launch_v<8>(x, a, stream);
    if (a.E <= 512) return launch_v<16>(x, a, stream);
    return launch_v<32>(x, a, stream);
}

}  // namespace

cudaError_t launch_moe_gate(const GateProblem &p, cudaStream_t stream) {
    GateArgs a;
    a.bias = p.bias;
    auto aligned16 = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    const int per16 = p.fp32 ? 4 : 8;
    a.vec = p.E % 8 == 0 && p.ldx % per16 == 0 && aligned16(p.logits) && aligned16(p.bias);
    a.ldx = p.ldx;
    a.T = static_cast<int>(p.T);
    a.E = static_cast<int>(p.E);
    a.k = static_cast<int>(p.k);
    a.n_group = static_cast<int>(p.n_group);
    a.topk_group = static_cast<int>(p.topk_group);
    a.size = a.E / a.n_group;
    const int per_lane = a.E <= 32 ? 1 : a.E <= 64 ? 2 : a.E <= 128 ? 4 : a.E <= 256 ? 8
                                                                     : a.E <= 512 ? 16 : 32;
    const int run = a.size / per_lane;   // (as launch_any picks V)
    a.run_shift = a.size % per_lane == 0 && (run & (run - 1)) == 0 ? __builtin_ctz(run) : -1;
    a.sigmoid = p.sigmoid ? 1 : 0;
    a.renormalize = p.renormalize ? 1 : 0;
    a.scale = p.scale;
    a.ids = p.ids;
    a.w = p.w;
    return p.fp32 ? launch_any<float>(p.logits, a, stream)
                  : launch_any<uint16_t>(p.logits, a, stream);
}

}  // namespace w8a8
