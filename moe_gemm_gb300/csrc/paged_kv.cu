// The paged KV cache, on sm_103a ("Deploying Hunyuan 770B in INT8 on domestic
// accelerators", §3.4: every key and value vector gets its own scale when it
// is written). The cache of one layer is a pool of pages [P, Hkv, page, 128];
// a request's block table names the pages that hold its positions in order.
//  * paged_kv_plan_kernel brings the block tables from the lengths they hold
//    to the lengths asked for: pages of requests that shrink go back to the
//    stack of free pages, requests that grow take theirs off it, and every new
//    token gets its position and its slot (page * page_size + offset).
//  * paged_kv_write_kernel puts the new tokens' K and V vectors into their
//    slots: INT8 codes with one scale per vector, or the BF16 values.
// The plan is bound by latency: a chain of loads, three scans and the stores, 4.8 us
// for 32 requests and 6.2 for 1021 requests with 8.6 thousand new tokens, which eight
// CTAs of a cluster share. So is the write at decode sizes (2.3 us for 32 tokens); the
// INT8 write of 8192 tokens' 8 heads takes 14.5 us (51 MB: 3.5 TB/s) and waits for its
// loads: 26 warps per SM use 44 % of the issue slots, and the first stall is for memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "quant_math.cuh"

namespace w8a8 {
namespace {

// ---------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// What the call does with one request, in shared memory.
struct PlanEntry {
    int lens;     // positions held before the call
    int target;   // positions held after it; < 0: refused (its rows get no slot)
    int first;    // shrinking: its first place on the free stack; growing: pages taken before its own
    int cu;       // new tokens of the requests before it
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

// Exclusive prefix sum over the block's threads; total receives the sum.
__device__ __forceinline__ long long block_scan(long long v, long long *part, long long &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += u;
    }
    __syncthreads();   // the previous scan's sums have been read
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    const long long p = part[lane];
    long long psum = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, psum, o);
        if (lane >= o) psum += u;
    }
    total = __shfl_sync(0xFFFFFFFFu, psum, 31);
    const long long base = __shfl_sync(0xFFFFFFFFu, psum - p, warp);
    return base + incl - v;
}

struct PlanArgs {
    int32_t *table;      // [B, W]
    int32_t *lens;       // [B] in: held, out: held after the call
    const int32_t *target;
    int32_t *free_pages; // [P]
    int32_t *n_free;     // [1]
    int B, W, P, page, n_tokens;
    int32_t *cu_new, *kv_lens, *slots, *positions;
};

// One cluster. Every CTA reads all the lengths and works out the same plan (B
// is at most a few thousand; one scan costs less than handing it around); the
// CTAs then share out the pages and the tokens. The stack's released entries
// are written between the two cluster barriers and read after the second.
__global__ void __launch_bounds__(kPlanThreads)
paged_kv_plan_kernel(const PlanArgs a) {
    extern __shared__ PlanEntry s_plan[];   // [B]
    __shared__ long long s_part[kPlanWarps];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x;
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    const int n_free0 = min(max(a.n_free[0], 0), a.P);
    auto pages = [&](int n) { return static_cast<int>((static_cast<long long>(n) + a.page - 1) / a.page); };
    // lengths, and what a request with impossible ones becomes: refused, no rows
    long long asked = 0, back = 0;
    for (int b = b0; b < b1; ++b) {
        const int l = a.lens[b], t = a.target[b];
        const bool bad = l < 0 || t < 0 || pages(l) > a.W;
        s_plan[b].lens = max(l, 0);
        s_plan[b].target = bad ? -1 : t;
        if (l >= 0 && t > l) asked += static_cast<long long>(t) - l;
        if (!bad && t < l) back += pages(l) - pages(t);
    }
    long long n_asked, n_back;
    long long cu = block_scan(asked, s_part, n_asked);
    long long first = block_scan(back, s_part, n_back) + n_free0;
    const long long top = min(static_cast<long long>(a.P), n_free0 + n_back);
    long long need = 0;
    for (int b = b0; b < b1; ++b) {
        const int l = s_plan[b].lens, t = s_plan[b].target;
        s_plan[b].cu = static_cast<int>(min(cu, 0x7FFFFFFFll));
        const int raw = a.target[b];
        if (a.lens[b] >= 0 && raw > l) cu += static_cast<long long>(raw) - l;
        if (t >= 0 && t < l) {
            s_plan[b].first = static_cast<int>(min(first, 0x7FFFFFFFll));
            first += pages(l) - pages(t);
        } else if (t > l) {
            if (pages(t) > a.W || cu > a.n_tokens) s_plan[b].target = -1;
            else need += pages(t) - pages(l);
        }
    }
    long long n_need;
    long long before = block_scan(need, s_part, n_need);
    long long taken = 0;
    for (int b = b0; b < b1; ++b) {
        const int l = s_plan[b].lens, t = s_plan[b].target;
        if (t <= l) continue;
        const int n = pages(t) - pages(l);
        s_plan[b].first = static_cast<int>(min(before, 0x7FFFFFFFll));
        before += n;
        if (n > 0 && before > top) s_plan[b].target = -1;
        else taken += n;
    }
    long long n_taken;
    block_scan(taken, s_part, n_taken);
    __syncthreads();
    const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
    cluster_sync();   // every CTA has read lens, target and n_free
    if (rank == 0) {
        for (int b = tid; b < a.B; b += kPlanThreads) {
            const PlanEntry e = s_plan[b];
            a.cu_new[b] = e.cu;
            a.kv_lens[b] = e.target < 0 ? 0 : e.target;
            if (e.target >= 0) a.lens[b] = e.target;
        }
        if (tid == 0) {
            a.cu_new[a.B] = static_cast<int>(min(n_asked, 0x7FFFFFFFll));
            a.n_free[0] = static_cast<int>(top - n_taken);
        }
    }
    // pages given back: one warp per request
    const int warp = rank * kPlanWarps + (tid >> 5), lane = tid & 31, warps = ranks * kPlanWarps;
    if (n_back > 0) {
        for (int b = warp; b < a.B; b += warps) {
            const PlanEntry e = s_plan[b];
            if (e.target < 0 || e.target >= e.lens) continue;
            const int want = pages(e.target), n = pages(e.lens) - want;
            int32_t *row = a.table + static_cast<int64_t>(b) * a.W + want;
            for (int j = lane; j < n; j += 32) {
                const int at = e.first + j;
                if (at < a.P) a.free_pages[at] = row[j];
                row[j] = -1;
            }
        }
    }
    cluster_sync();
    const int itop = static_cast<int>(top);
    for (int b = warp; b < a.B; b += warps) {
        const PlanEntry e = s_plan[b];
        if (e.target <= e.lens) continue;
        const int have = pages(e.lens), n = pages(e.target) - have;
        int32_t *row = a.table + static_cast<int64_t>(b) * a.W + have;
        for (int j = lane; j < n; j += 32) row[j] = a.free_pages[itop - 1 - (e.first + j)];
    }
    // a slot and a position for every new token
    // (counted without a sign: the last step passes 2^31 when n_tokens is near it)
    for (unsigned n = rank * kPlanThreads + tid; n < static_cast<unsigned>(a.n_tokens);
         n += ranks * kPlanThreads) {
        const int t = static_cast<int>(n);
        int slot = -1, pos = -1;
        if (t < n_asked) {
            int lo = 0, hi = a.B;   // the last request with cu <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_plan[mid].cu <= t) lo = mid;
                else hi = mid;
            }
            const PlanEntry e = s_plan[lo];
            const int at = e.lens + (t - e.cu);
            if (e.target > at) {
                const int i = at / a.page, have = pages(e.lens);
                const int id = i < have ? a.table[static_cast<int64_t>(lo) * a.W + i]
                                        : a.free_pages[itop - 1 - (e.first + i - have)];
                slot = id * a.page + (at - i * a.page);
                pos = at;
            }
        }
        a.slots[t] = slot;
        a.positions[t] = pos;
    }
}

// --------------------------------------------------------------------- write
constexpr int kWriteThreads = 256;

struct WriteArgs {
    const uint16_t *k, *v;            // BF16, token strides kt, vt, head strides kh, vh
    int64_t kt, kh, vt, vh;
    const int32_t *slots;             // [T]
    int T, Hkv, page;
    int n_slots;                      // P * page
    void *kc, *vc;
    float *ks, *vs;
};

// One warp per token and H kv heads: lanes 0-15 take the K vectors, lanes
// 16-31 the V vectors, 8 values (16 bytes) of each, all of them loaded before the
// first is worked on (and beside the slot). The INT8 form takes a vector's amax by
// four shuffles, the scale by one division, and rounds x / scale as the activation
// quantizer does. A long call takes several heads per warp, for more loads in flight
// and one look at the slot: 8192 tokens of 8 heads take 19.2 us
// with H = 1, 14.5 with 4 and 16.4 with 8 (whose registers cost warps). A decode step
// has warps to fill: 32 tokens take 2.3 us with H = 1, 3.7 with 4.
template <bool kInt8, int H>
__global__ void __launch_bounds__(kWriteThreads)
paged_kv_write_kernel(const WriteArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    // (counts and slots are below 2^31: divisions in 32 bits)
    const uint32_t i = blockIdx.x * (kWriteThreads / 32) + (threadIdx.x >> 5);
    const uint32_t groups = static_cast<uint32_t>(a.Hkv + H - 1) / H;
    const uint32_t t = i / groups;
    if (t >= static_cast<uint32_t>(a.T)) return;
    const int h0 = static_cast<int>(i - t * groups) * H;
    const int n = min(a.Hkv - h0, H);
    const bool is_v = (threadIdx.x & 16) != 0;
    const int c = threadIdx.x & 15;
    const int64_t hs = is_v ? a.vh : a.kh;
    const uint16_t *src = (is_v ? a.v + t * a.vt : a.k + t * a.kt) + h0 * hs + c * 8;
    uint4 x[H];
#pragma unroll
    for (int j = 0; j < H; ++j)
        if (j < n) x[j] = __ldcs(reinterpret_cast<const uint4 *>(src + j * hs));
    const int slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) return;   // the token has no slot
    const int p = slot / a.page;
    const int64_t row0 = (static_cast<int64_t>(p) * a.Hkv + h0) * a.page + (slot - p * a.page);
#pragma unroll
    for (int j = 0; j < H; ++j) {
        if (j >= n) break;
        const int64_t row = row0 + static_cast<int64_t>(j) * a.page;
        if constexpr (!kInt8) {
            reinterpret_cast<uint4 *>(is_v ? a.vc : a.kc)[row * 16 + c] = x[j];
        } else {
            uint32_t m = amax_bits8(x[j]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float s = __fdiv_rn(bf16_bits_to_f32(m), 127.0f);
            const bool fast = s >= 1.17549435e-38f;   // a normal scale: 1 / s is finite
            const uint2 q = quantize8(x[j], s, fast ? __frcp_rn(s) : 0.0f, fast);
            reinterpret_cast<uint2 *>(is_v ? a.vc : a.kc)[row * 16 + c] = q;
            if (c == 0) (is_v ? a.vs : a.ks)[row] = s;
        }
    }
}

}  // namespace

cudaError_t launch_paged_kv_plan(const PagedPlanProblem &p, cudaStream_t stream) {
    PlanArgs a;
    a.table = p.block_table;
    a.lens = p.lens;
    a.target = p.target;
    a.free_pages = p.free_pages;
    a.n_free = p.n_free;
    a.B = static_cast<int>(p.B);
    a.W = static_cast<int>(p.W);
    a.P = static_cast<int>(p.P);
    a.page = static_cast<int>(p.page);
    a.n_tokens = static_cast<int>(p.n_tokens);
    a.cu_new = p.cu_new;
    a.kv_lens = p.kv_lens;
    a.slots = p.slots;
    a.positions = p.positions;
    static int attr_done[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && !attr_done[dev]) {
        e = cudaFuncSetAttribute(paged_kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kPagedMaxRequests * sizeof(PlanEntry)));
        if (e != cudaSuccess) return e;
        attr_done[dev] = 1;
    }
    // one CTA for a decode step; a cluster of eight when there is work to share
    const int ctas = p.B > 256 || p.n_tokens > 2048 ? 8 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.B) * sizeof(PlanEntry);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, paged_kv_plan_kernel, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t launch_paged_kv_write(const PagedWriteProblem &p, cudaStream_t stream) {
    WriteArgs a;
    a.k = p.k;
    a.v = p.v;
    a.kt = p.kt;
    a.kh = p.kh;
    a.vt = p.vt;
    a.vh = p.vh;
    a.slots = p.slots;
    a.T = static_cast<int>(p.T);
    a.Hkv = static_cast<int>(p.Hkv);
    a.page = static_cast<int>(p.page);
    a.n_slots = static_cast<int>(p.P * p.page);
    a.kc = p.kc;
    a.vc = p.vc;
    a.ks = p.ks;
    a.vs = p.vs;
    constexpr int kPerCta = kWriteThreads / 32;
    cudaLaunchConfig_t cfg = {};
    // (four heads per warp once the warps of one head each are several times those
    // that the SMs hold)
    const int heads = p.T * p.Hkv >= 32768 ? 4 : 1;
    const int64_t warps = p.T * ((p.Hkv + heads - 1) / heads);
    cfg.gridDim = dim3(static_cast<unsigned>((warps + kPerCta - 1) / kPerCta));
    cfg.blockDim = dim3(kWriteThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*kernel)(WriteArgs) =
        p.int8 ? (heads == 4 ? paged_kv_write_kernel<true, 4> : paged_kv_write_kernel<true, 1>)
               : (heads == 4 ? paged_kv_write_kernel<false, 4> : paged_kv_write_kernel<false, 1>);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace w8a8
