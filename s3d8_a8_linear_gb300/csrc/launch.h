// Internal launcher interface between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace s3d8 {

struct LinearArgs {
    const uint8_t *packed;      // [G, K]
    const int8_t *C;            // [32 * 3]
    const __nv_bfloat16 *cs;    // [N]            (unused when acc != nullptr)
    const int8_t *xq;           // [M, K]
    const float *xscale;        // [M]            (unused when acc != nullptr)
    int M, N, K;
    __nv_bfloat16 *out;         // [M, N] bf16 output, or
    int32_t *acc;               // [M, N] int32 accumulators (test entry)
    void *ws;                   // device workspace
    size_t ws_bytes;
    int *status;                // device status word
};

// One linear of a grouped launch (see s3d8_linear_job in include/s3d8.h).
struct GroupJob {
    const uint8_t *packed;
    const int8_t *C;
    const __nv_bfloat16 *cs;
    const __nv_bfloat16 *x;     // bf16 activations to quantise in-kernel, or nullptr
    const int8_t *xq;           // pre-quantised codes (when x == nullptr)
    const float *xscale;
    int8_t *xq_out;             // optional copies of the in-kernel codes / scales
    float *xscale_out;
    __nv_bfloat16 *out;
    int32_t *acc;
    int N, K;
};

constexpr int kMaxJobs = 8;

struct GroupArgs {
    GroupJob jobs[kMaxJobs];
    int njobs;
    int M;
    int cta_begin[kMaxJobs + 1];   // filled by the launcher
    int *status;
};

int device_sm_count();
void *tensor_map_encoder_fn();   // cuTensorMapEncodeTiled, or nullptr
int *device_status_ptr();   // this device's sticky status word, or nullptr

cudaError_t launch_quantize_act(const __nv_bfloat16 *x, int M, int K, int8_t *xq, float *xscale,
                                cudaStream_t stream);
cudaError_t launch_encode(const __nv_bfloat16 *w, const int8_t *C, int N, int K, uint8_t *packed,
                          __nv_bfloat16 *chan_scale, void *workspace, cudaStream_t stream);
cudaError_t launch_fake_quant(const __nv_bfloat16 *w, const int8_t *C, int N, int K,
                              __nv_bfloat16 *w_hat, __nv_bfloat16 *chan_scale, void *workspace,
                              cudaStream_t stream);
size_t fit_workspace_bytes(int64_t N, int64_t K);
cudaError_t launch_fit(const __nv_bfloat16 *w, int N, int K, const uint32_t *r, int iters,
                       float *cf, int8_t *C, void *workspace, cudaStream_t stream);
cudaError_t launch_selftest_scaled_abs(const __nv_bfloat16 *x, const __nv_bfloat16 *alpha,
                                       int64_t n, float *out, cudaStream_t stream);
cudaError_t launch_decode(const uint8_t *packed, const int8_t *C, int N, int K, int8_t *w,
                          cudaStream_t stream);
cudaError_t launch_gemv(const LinearArgs &a, cudaStream_t stream);
bool gemv_tma_supported(int M, int K);
cudaError_t launch_wait_timeout(int polls, int *status, cudaStream_t stream);
bool gemv_group_job_ok(int M, int K, bool fused);
cudaError_t launch_gemv_group(GroupArgs &g, cudaStream_t stream);
cudaError_t launch_gemv_tma(const LinearArgs &a, cudaStream_t stream);
// Tensor-core path, three kernels: one SM per tile (decoding packed tiles
// itself), SM pairs decoding packed tiles themselves, or SM pairs on weights
// expanded to bf16 in the workspace first.  prefill_kind(M, K) picks by token
// count and row length.
constexpr int kTcOneSm = 0, kTcPairFused = 1, kTcPairExpanded = 2;
int prefill_kind(int M, int K);
size_t prefill_workspace_bytes(int M, int N, int K, int kind);
cudaError_t launch_prefill_tc(const LinearArgs &a, int kind, cudaStream_t stream);
cudaError_t launch_prefill_pair(const LinearArgs &a, const __nv_bfloat16 *act, const __nv_bfloat16 *wdec,
                                int32_t *part, int nsplit, int kbps, cudaStream_t stream);
cudaError_t launch_prefill_fused(const LinearArgs &a, const uint16_t *act_f16, int32_t *part, int nsplit, int kbps,
                                 int g2, cudaStream_t stream);
// Split-K finish shared by the tensor-core paths: sums int32 partials
// [nsplit][M][N] into a.out (epilogue) or a.acc.
cudaError_t launch_splitk_finalize(const int32_t *part, int nsplit, const LinearArgs &a, cudaStream_t stream);
// tcgen05 GEMM with the weights decoded into tensor memory (decode_tmem.cu):
// 1..64 tokens.
bool tmem_supported(int M);
// AUTO takes it for 5..32 tokens, and up to 64 when its tiles fit in one wave
// (not with more 128-row tiles than SMs).
bool tmem_preferred(int M, int N, int K);
size_t tmem_workspace_bytes(int M, int N, int K);
cudaError_t launch_tmem(const LinearArgs &a, cudaStream_t stream);

// ---- between two linears (residual_norm.cu, rope_append.cu, paged_attention.cu, pages.cu)
struct NormArgs {
    const __nv_bfloat16 *h, *y, *w_post, *gate, *w_pre;   // all but h may be null
    int gate_n, tanh_gate;
    float alpha, eps;
    int M, D;
    __nv_bfloat16 *h_out, *x;
    int8_t *xq;
    float *xscale;
    int *status;
};
struct NormGradArgs {
    NormArgs f;                         // h = h', and the forward call's parameters
    const __nv_bfloat16 *dh, *dx;       // either may be null
    __nv_bfloat16 *dh_in, *dy;
    float *dw_pre, *dw_post, *dgate;
    float *part;                        // [CTAs][2 D + 4]
};
cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t stream);
size_t residual_norm_backward_workspace(int64_t M, int64_t D);
cudaError_t launch_residual_norm_backward(const NormGradArgs &g, cudaStream_t stream);

// One layer's paged cache as the kernels see it (strides in elements).
struct KvCache {
    void *k, *v;
    float *k_scale, *v_scale;           // int8 only
    int64_t ks[3], vs[3], ss[3];        // page, token, head
    int pages, page_size, heads, dim;
    int int8;
};
struct RopeArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t qs[2], ks[2], vs[2];        // token, head
    const float *cos, *sin;
    int64_t max_pos;
    int rotary, interleaved;
    const int32_t *positions, *rows;
    int64_t T;
    int Hq;
    const int32_t *table;
    int64_t table_rows, width;
    KvCache kv;
    __nv_bfloat16 *q_out;
    int *status;
    const __nv_bfloat16 *q_norm, *k_norm;   // [dim], or null: as they are
    float eps;
};
cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t stream);

struct AttnArgs {
    const __nv_bfloat16 *q;
    KvCache kv;
    const int32_t *table, *lens;
    int64_t width;
    int B, Hq;
    float scale;
    int64_t window;
    __nv_bfloat16 *out;
    float *lse;
    void *ws;
    int *status;
};
size_t paged_attention_workspace(const KvCache &kv, int64_t B, int64_t Hq);
cudaError_t launch_paged_attention(const AttnArgs &a, cudaStream_t stream);

constexpr int kPoolLayers = 64;         // layers of one copy launch
struct PoolArgs {
    KvCache geo;                        // geometry and strides (its pointers are unused)
    void *k[kPoolLayers], *v[kPoolLayers];
    float *k_scale[kPoolLayers], *v_scale[kPoolLayers];
    int layers;
};
struct PagesArgs {
    int32_t *table, *lens, *refs;
    int64_t rows, width;
    int pages, page_size;
    const int32_t *who, *other;         // seqs and add, or parents and children
    int n;
    int32_t *got;                       // got [n], or live [1]
    int32_t *ws;
    int *status;
};
size_t pages_workspace(int64_t pages, int64_t rows);
// Copies page src[i] to dst[i]: whole pages, or the first tokens[i] tokens of each
// (tokens != nullptr); the pair count is n, or *count on the device when given.
cudaError_t launch_copy_pages(const PoolArgs &p, const int32_t *src, const int32_t *dst, const int32_t *tokens,
                              int n, const int32_t *count, int *status, cudaStream_t stream);
cudaError_t launch_extend_pages(const PagesArgs &a, cudaStream_t stream);
// On return `pairs` holds the workspace's lists of copies to make: src, dst, tokens.
struct PagePairs {
    const int32_t *src, *dst, *tokens, *count;
};
cudaError_t launch_fork_pages(const PagesArgs &a, PagePairs *pairs, cudaStream_t stream);
cudaError_t launch_free_pages(const PagesArgs &a, cudaStream_t stream);
cudaError_t launch_compact_pages(const PagesArgs &a, PagePairs *pairs, cudaStream_t stream);

// ---- a vision decoder's calls (norm_rope.cu, cross_attention.cu, sample.cu)
struct NormRopeArgs {
    const __nv_bfloat16 *x[2];          // queries and keys; the keys may have no heads
    int64_t xs[2][2];                   // token, head
    const __nv_bfloat16 *w[2];          // [dim], or null: not normed
    int heads[2];
    const float *cos, *sin;
    int64_t max_pos;
    int rotary, interleaved;
    const int32_t *positions;           // or null: token t at t
    int64_t T;
    int dim;
    float eps;
    __nv_bfloat16 *out[2];              // z, or dx
    const __nv_bfloat16 *dz[2];         // backward only
    int64_t dzs[2][2];
    float *dw[2], *part;                // part: [CTAs][dim]
    int *status;
};
cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream);
size_t norm_rope_backward_workspace(int64_t T, int heads, int dim);
cudaError_t launch_norm_rope_backward(const NormRopeArgs &a, cudaStream_t stream);

struct CrossArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t qs[2], ks[2], vs[2];        // token, head
    const int32_t *spans;               // [T, 2], or null: every state
    int T, S, Hq, heads, dim;
    float scale;
    __nv_bfloat16 *out;
    float *lse;
    void *ws;
    int *status;
    // backward: out and lse are inputs
    const __nv_bfloat16 *dout;
    int64_t ds[2];
    __nv_bfloat16 *dq, *dk, *dv;
};
size_t cross_attention_workspace(int64_t T, int64_t S, int64_t Hq, int64_t heads, int64_t dim);
cudaError_t launch_cross_attention(const CrossArgs &a, cudaStream_t stream);
// Without states: zeros into out, -inf into lse (if any), and the spans looked at.
cudaError_t launch_cross_nothing(const CrossArgs &a, cudaStream_t stream);
size_t cross_attention_backward_workspace(int64_t T, int64_t S, int64_t Hq, int64_t heads, int64_t dim);
cudaError_t launch_cross_attention_backward(const CrossArgs &a, cudaStream_t stream);

struct SampleArgs {
    const __nv_bfloat16 *logits;        // [B, V], rows `stride` elements apart
    int64_t stride;
    int B, V;
    const float *u, *temperature, *top_p, *min_p;   // [B]; all but u may be null
    const int32_t *top_k;
    int32_t *tokens;
    float *logprob;                     // or null
};
cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream);

}  // namespace s3d8
