// Internal declarations shared by the translation units of libw8a8 (host side).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace w8a8 {

cudaError_t launch_quant_act(const uint16_t *a, int64_t M, int64_t K, int64_t lda, int8_t *qa,
                             int64_t ldq, float *sa, cudaStream_t stream);

// The same codes as launch_quant_act, written as fp16 (row stride K) into
// x16 for the tensor-core GEMM, which then needs no staging kernel; also
// zeroes n_cnt split counters at cnt (if not null) for that GEMM.
cudaError_t launch_quant_act_f16(const uint16_t *a, int64_t M, int64_t K, int64_t lda, void *x16,
                                 float *sa, int *cnt, int n_cnt, cudaStream_t stream);

cudaError_t launch_quant_weight(const float *w, int64_t N, int64_t K, int8_t *qw, float *sw,
                                cudaStream_t stream);

// Scale-format variants: activations with power-of-two (UE8M0) scales
// (int8 codes, or fp16 codes into a GEMM workspace), and weights over
// [block_rows x 128] blocks (block_rows 1 or 128) with amax/127 or
// power-of-two scales, sw [ceil(N / block_rows), K / 128].
cudaError_t launch_quant_act_ex(const uint16_t *a, int64_t M, int64_t K, int64_t lda, int8_t *qa,
                                int64_t ldq, float *sa, bool pow2, cudaStream_t stream);
cudaError_t launch_quant_act_f16_ex(const uint16_t *a, int64_t M, int64_t K, int64_t lda,
                                    void *x16, float *sa, int *cnt, int n_cnt, bool pow2,
                                    cudaStream_t stream);
cudaError_t launch_quant_weight_blocks(const float *w, int64_t N, int64_t K, int block_rows,
                                       bool pow2, int8_t *qw, float *sw, cudaStream_t stream);

// Per-token quantization with a row gather: output row r (row stride K)
// quantizes input row src_rows[r] of a (row stride lda); rows whose entry is
// negative are skipped. Codes as fp16 (f16) or int8.
cudaError_t launch_quant_act_rows(const uint16_t *a, int64_t rows, int64_t K, int64_t lda,
                                  const int32_t *src_rows, void *out, bool f16, float *sa,
                                  cudaStream_t stream);

// MoE expert FFN steps (moe.cu).
constexpr int kMoeMaxTopK = 64;
constexpr int64_t kSwigluMaxI = 8192;
cudaError_t launch_moe_route(const int32_t *ids, int64_t T, int64_t k, int64_t E, int32_t *offsets,
                             int32_t *row_of, int32_t *token_of_row, int32_t *pair_of_row,
                             cudaStream_t stream);
// out_kind: 0 int8 codes, 1 fp16 codes (+ scales sh), 2 h itself (FP32)
cudaError_t launch_swiglu_quant(const float *U, int64_t rows, int64_t I, const int32_t *offsets,
                                int64_t E, void *out, int out_kind, float *sh,
                                cudaStream_t stream);
cudaError_t launch_moe_unpermute(const float *D, const int32_t *row_of, const float *w, int64_t T,
                                 int64_t k, int64_t H, void *y, bool out_fp32,
                                 cudaStream_t stream);

// int8 codes [rows, K] (row stride ldq) -> fp16 codes [rows, K] in `out`;
// also zeroes n_cnt split-tile counters at cnt (if not null) for the GEMM
// launched after it.
cudaError_t launch_widen_codes(const int8_t *q, int64_t rows, int64_t K, int64_t ldq, void *out,
                               int num_sms, cudaStream_t stream, int *cnt = nullptr,
                               int n_cnt = 0);

struct GemmProblem {
    const int8_t *qa;         // [R, K] int8 activation codes
    const float *sa;          // [R]
    const float *sw;          // [E*N, G]
    const int8_t *qw;         // [E*N, K]
    const void *x16;          // [R, K] fp16 copy of the int8 activation codes (staging)
    const int32_t *offsets;   // [E+1] device, or nullptr for one dense segment [0, R)
    void *y;                  // [R, N]
    int32_t *debug_partials;  // nullable [R, N, G]
    int64_t R, E, N, K;
    bool out_fp32;
    // Dense calls of <= kGemvMaxTokens rows only: BF16 activations [R, lda]
    // that the GEMV quantizes itself (then qa and sa are not read).
    const uint16_t *act = nullptr;
    int64_t lda = 0;
    // Stream-K split of dense calls; null sk_cnt: whole tiles only.
    // Weight scales per [sw_block_rows x 128] block: 1 (per row) or 128.
    int sw_block_rows = 1;
    // Weight-only path: x16 holds the caller's BF16 activations (row stride
    // ldx elements), sa is null (no token scale).
    bool a16 = false;
    int64_t ldx = 0;
    int *sk_cnt = nullptr;        // [2 * kSkMaxCtas] counters, zeroed before the GEMM
    float *sk_part = nullptr;     // [kSkMaxCtas][2][sk_ld][128] FP32 partials
    int sk_ld = 0;
    // The launch before is a kernel of the same call that lets this one start
    // behind its own wait (the quantizers, widen_codes, swiglu_quant): weights,
    // their scales and offsets may be read before the wait for it. After any
    // other kernel the GEMM waits first, as what comes before that one may
    // still write them.
    bool early = false;
};

// Dense calls with at most kGemvMaxTokens token rows run on the CUDA cores
// (batched GEMV over the int8 codes; no fp16 staging copy is made).
constexpr int kGemvMaxTokens = 4;
inline bool uses_gemv(int64_t R, bool grouped) { return !grouped && R <= kGemvMaxTokens; }

// The GEMV can quantize its token rows itself when their codes for all of K
// (K * MR bytes, MR = R rounded up to 1, 2 or 4) fit beside its weight
// stages, and the activation rows allow 16-byte vector loads.
inline bool gemv_can_fuse_quant(int64_t R, int64_t K, int64_t lda, const void *a) {
    const int64_t mr = R <= 1 ? 1 : (R <= 2 ? 2 : 4);
    return R >= 1 && R <= kGemvMaxTokens && K * mr <= 96 * 1024 && lda % 8 == 0 &&
           (reinterpret_cast<uintptr_t>(a) % 16) == 0;
}

// Dense calls of 5..64 token rows (narrow tensor-core tiles) split tiles
// across CTAs (stream-K) when the workspace holds the split area: arrival
// counters and two FP32 partial slots per CTA (token rows x 128 weight rows),
// for at most kSkMaxCtas CTAs. A narrow tile is bound by its MMA issue, not
// by the weight stream, so the steps of a partial last wave are worth
// spreading over all SMs.
constexpr int kSkMaxCtas = 160;
constexpr int kNarrowSplitMaxRows = 64;
inline bool uses_split(int64_t R, bool grouped) {
    return !grouped && R > kGemvMaxTokens && R <= kNarrowSplitMaxRows;
}
inline size_t sk_counter_bytes() { return 2 * kSkMaxCtas * sizeof(int); }
inline size_t sk_area_bytes(int64_t R, bool grouped) {
    if (R <= 0 || !uses_split(R, grouped)) return 0;
    return sk_counter_bytes() +
           static_cast<size_t>(kSkMaxCtas) * 2 * static_cast<size_t>(R) * 128 * sizeof(float);
}

// Dense calls of at least this many token rows run tiles of 128 weight rows x
// 192 token rows (one 192-column MMA per 16 K, two partial buffers in TMEM).
constexpr int kWide256MinRows = 256;
// RMSNorm + per-token quantization (quant.cu): out_kind 0 int8 codes, 1 fp16
// codes (dense rows of K; zeroes n_cnt split counters), 2 the BF16 rows.
// K a multiple of 8, at most kRmsNormMaxK; x, gamma 16-byte aligned, out 16
// (8 for int8 codes); row strides multiples of 8 elements.
constexpr int64_t kRmsNormMaxK = 32768;
cudaError_t launch_rmsnorm_quant(const uint16_t *x, int64_t M, int64_t K, int64_t ldx,
                                 const uint16_t *gamma, float eps, int out_kind, void *out,
                                 int64_t ldo, float *sa, int *cnt, int n_cnt, bool pow2,
                                 cudaStream_t stream);

inline bool uses_wide256(int64_t R, bool grouped) { return !grouped && R >= kWide256MinRows; }

// Decode attention over a KV cache [B, Hkv, S_max, 128] (attention.cu): INT8
// codes with one scale per vector (ks, vs [B, Hkv, S_max]), or BF16 values.
struct AttnProblem {
    const uint16_t *q;      // [B, Hq, 128] BF16
    const void *kc, *vc;    // caches
    const float *ks, *vs;   // INT8 caches: per-vector scales
    const int32_t *lens;    // [B] device
    int64_t B, Hq, Hkv, S_max;
    float scale;
    bool int8;
    void *out;              // [B, Hq, 128]
    bool out_fp32;
    float *part_o, *part_ml;   // workspace: per-chunk partial outputs and statistics
};
constexpr int kAttnHeadDim = 128;
size_t attn_workspace_bytes(int64_t B, int64_t Hq, int64_t S_max);
cudaError_t launch_attention_decode(const AttnProblem &p, cudaStream_t stream);
// Quantizes n vectors of 128 BF16 values into rows dst_rows[i] (or i) of an
// INT8 cache [rows, 128] with one scale per row.
cudaError_t launch_kv_quant(const uint16_t *x, int64_t n, const int32_t *dst_rows, int8_t *cache,
                            float *scales, cudaStream_t stream);

// The router's gate (gate.cu): top-k ids and weights from logits [T, E].
struct GateProblem {
    const void *logits;     // [T, ldx] FP32 or BF16
    bool fp32;
    int64_t ldx, T, E, k, n_group, topk_group;
    const float *bias;      // [E] or null
    bool sigmoid, renormalize;
    float scale;
    int32_t *ids;           // [T, k]
    float *w;               // [T, k]
    const struct MoeFewTokens *tokens = nullptr;   // what the kernel launched next wants made too
};
constexpr int kGateMaxGroups = 64;
cudaError_t launch_moe_gate(const GateProblem &p, cudaStream_t stream);

// The paged KV cache (paged_kv.cu): pages [P, Hkv, page, 128].
constexpr int64_t kPagedMaxRequests = 4096;
struct PagedPlanProblem {
    int32_t *block_table, *lens;
    const int32_t *target;
    int32_t *free_pages, *n_free;
    int64_t B, W, P, page, n_tokens;
    int32_t *cu_new, *kv_lens, *slots, *positions;
};
cudaError_t launch_paged_kv_plan(const PagedPlanProblem &p, cudaStream_t stream);

struct PagedWriteProblem {
    const uint16_t *k, *v;           // BF16 [T, Hkv, 128]
    int64_t kt, kh, vt, vh;          // token and head strides (elements)
    const int32_t *slots;            // [T]
    int64_t T, Hkv, P, page;
    bool int8;
    void *kc, *vc;
    float *ks, *vs;                  // INT8: [P, Hkv, page]
};
cudaError_t launch_paged_kv_write(const PagedWriteProblem &p, cudaStream_t stream);

// The same write behind the position rotation of q and k (paged_append.cu).
struct PagedAppendProblem {
    PagedWriteProblem w;
    const uint16_t *q;               // BF16 [T, Hq, 128]; Hq may be 0
    int64_t qt, qh, Hq;
    const int32_t *positions;        // [T]
    const float *inv_freq;           // [rot / 2]
    int64_t rot;
    bool interleaved;
    float amplitude;
    uint16_t *q_out;                 // BF16 [T, Hq, 128]
    int64_t ot, oh;
};
cudaError_t launch_paged_kv_append(const PagedAppendProblem &p, int num_sms, cudaStream_t stream);

// Attention of each request's new tokens over its pages (paged_attention.cu).
struct PagedAttnProblem {
    const uint16_t *q;               // BF16 [T, Hq, 128]
    int64_t qt, qh;                  // token and head strides (elements)
    const void *kc, *vc;
    const float *ks, *vs;            // INT8 pages: [P, Hkv, page]; null: BF16 pages
    const int32_t *block_table;      // [B, W]
    const int32_t *kv_lens;          // [B]
    const int32_t *cu_new;           // [B + 1]
    int64_t T, B, W, Hq, Hkv, P, page;
    float scale;
    int64_t window;                  // 0: none
    void *out;                       // [T, Hq, 128]
    bool out_fp32;
    void *workspace;
};
constexpr int kPagedMaxGroup = 16;   // Hq / Hkv
size_t paged_attn_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv);
cudaError_t launch_paged_attention(const PagedAttnProblem &p, cudaStream_t stream);

// Maximum number of experts a grouped call may have.
constexpr int kMaxExperts = 1024;

// The experts of a few tokens in one kernel (moe_layer.cu), after the gate, whose
// launch makes moe_few_tokens() as well: the tokens' codes and scales, and zeros.
// (8 of 64 experts, H 4096, I 1536, this kernel / the six of moe_ffn, with the gate: 1 token 45 / 77
// us, 16 tokens 221 / 299, 32 tokens 302 / 311; 8 of 256, H 2048, I 640: 19 / 37, 92 / 127, 134 /
// 179. Experts with more than 32 tokens would need tiles that its registers do not hold.)
constexpr int64_t kMoeFewMaxTokens = 32;
constexpr int64_t kMoeFewMaxPairs = 512;
struct MoeFewProblem {
    const uint16_t *x;               // BF16 [T, ldx]
    int64_t ldx;
    const int32_t *ids;              // [T, k], each token's different
    const float *w;                  // [T, k]
    int64_t T, k, E, H, I;
    const int8_t *qw_up, *qw_down;
    const float *sw_up, *sw_down;
    void *y;                         // [T, H]
    bool out_fp32;
    void *workspace;
};
struct MoeFewTokens {
    const uint16_t *x;               // BF16 [T, ldx]
    int64_t ldx;
    int T, H, vec;                   // vec: rows may be read 16 bytes at a time
    float *sx;                       // [T]
    int8_t *xq;                      // [T, H] codes
    uint32_t *zeros;
    int n_zeros;
};
bool uses_moe_few(int64_t T, int64_t k, int64_t H, int num_sms);
size_t moe_few_workspace_bytes(int64_t T, int64_t k, int64_t H, int64_t I);
MoeFewTokens moe_few_tokens(const MoeFewProblem &p);
cudaError_t launch_moe_few(const MoeFewProblem &p, int num_sms, cudaStream_t stream);

cudaError_t launch_gemm(const GemmProblem &p, int num_sms, cudaStream_t stream);

// FP8 (e4m3) with a scale per block of 128: quantizers (quant_fp8.cu) and the product
// (gemm_fp8.cu).
// chained: the next launch is the product of these codes, and may start once this kernel's own wait is
// over: whatever ran before is done then.
cudaError_t launch_quant_act_fp8(const uint16_t *a, int64_t M, int64_t K, int64_t lda, void *qa,
                                 float *sa, bool pow2, bool chained, cudaStream_t stream);
cudaError_t launch_quant_weight_fp8(const float *w, int64_t N, int64_t K, bool pow2, void *qw,
                                    float *sw, cudaStream_t stream);
struct Fp8Problem {
    const void *qa, *qw;             // e4m3 [M, K], [N, K]
    const float *sa, *sw;            // [M, K / 128], [ceil(N / 128), K / 128]
    void *y;                         // [M, N]
    bool out_fp32;
    int64_t M, N, K;
    // The launch before is the call's chained quantizer: weights may be read before the wait for it. After
    // any other kernel the product waits first, as what comes before that one may still write them.
    bool chained;
};
cudaError_t launch_gemm_fp8(const Fp8Problem &p, int num_sms, cudaStream_t stream);

// Launches the bounded-wait diagnostic (see gemm.cu): its wait gives up after
// limit_ns and records a code in the device error word.
cudaError_t launch_selftest_wait(unsigned long long limit_ns, cudaStream_t stream);

// Device error word of the GEMM kernel (read/clear; synchronising).
cudaError_t read_device_error(unsigned long long *value, bool clear);

// Device address of the error word (for kernels of other translation units).
cudaError_t device_error_word(unsigned long long **out);

// Rate probes of the MMA paths (probe.cu): tcgen05.mma kind::f16, M = 128,
// N = n, K = 16, A in tensor memory, `chains` accumulators taking turns (on
// the same operands, or each on its own when distinct),
// 8 * chains * steps instructions per CTA on num_sms CTAs; and dp4a,
// 16 * iters per thread on 4 * num_sms CTAs of 512 threads.
cudaError_t launch_probe_tc(int n, int chains, int distinct, long long steps, int num_sms,
                            cudaStream_t stream);
cudaError_t launch_probe_dp4a(long long iters, int num_sms, cudaStream_t stream);

// Per-device properties cached on first use.
struct DeviceInfo {
    int device = -1;
    int cc_major = 0, cc_minor = 0;
    int num_sms = 0;
};
cudaError_t current_device_info(DeviceInfo *out);

}  // namespace w8a8
