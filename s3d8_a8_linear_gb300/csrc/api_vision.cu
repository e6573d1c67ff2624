// C ABI of a vision decoder's calls: normed rotary heads, cross attention and the next
// token.  As in api.cu, every check runs before the first CUDA call.
#include "../../include/s3d8.h"
#include "launch.h"

#include <cuda_runtime.h>
#include <math.h>

using namespace s3d8;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? S3D8_OK : S3D8_ERR_CUDA; }

constexpr int64_t kMaxInt = 0x7FFFFFFF;

const __nv_bfloat16 *bf(const void *p) { return static_cast<const __nv_bfloat16 *>(p); }
__nv_bfloat16 *bf(void *p) { return static_cast<__nv_bfloat16 *>(p); }

int check_workspace(const void *ws, size_t bytes, size_t need)
{
    if (need && (!ws || bytes < need))
        return S3D8_ERR_WORKSPACE;
    return aligned(ws, 16) ? S3D8_OK : S3D8_ERR_ALIGNMENT;
}

// A tensor of rows [tokens, heads, dim] with strides (token, head): 16-byte rows.
int check_rows(const void *p, const int64_t stride[2])
{
    if (!p || !stride || stride[0] < 0 || stride[1] < 0)
        return S3D8_ERR_INVALID_ARG;
    return aligned(p, 16) && stride[0] % 8 == 0 && stride[1] % 8 == 0 ? S3D8_OK : S3D8_ERR_ALIGNMENT;
}

// What both directions of norm_rope share; sets everything but the outputs.
int norm_rope_args(NormRopeArgs *a, const void *q, const int64_t q_stride[2], int64_t Hq, const void *k, const int64_t k_stride[2],
                   int64_t Hk, const void *q_norm, const void *k_norm, const float *cos, const float *sin, int64_t max_pos,
                   int64_t rotary, int interleaved, const int32_t *positions, int64_t T, int64_t dim, float eps)
{
    if (T < 0 || T > S3D8_MAX_M || Hq < 1 || Hq > 65535 || Hk < 0 || Hk > 65535 || dim < 16 || dim > 256 || dim % 16 != 0 ||
        rotary < 0 || rotary % 2 != 0 || rotary > dim || max_pos < 0 || (k_norm && !Hk))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(q_norm, 16) || !aligned(k_norm, 16))
        return S3D8_ERR_ALIGNMENT;
    if (T > 0) {
        int st = check_rows(q, q_stride);
        if (st == S3D8_OK && Hk)
            st = check_rows(k, k_stride);
        if (st != S3D8_OK)
            return st;
        if (rotary && (!cos || !sin))
            return S3D8_ERR_INVALID_ARG;
        if (!aligned(cos, 4) || !aligned(sin, 4) || !aligned(positions, 4))
            return S3D8_ERR_ALIGNMENT;
        for (int j = 0; j < 2; ++j) {
            a->xs[0][j] = q_stride[j];
            a->xs[1][j] = Hk ? k_stride[j] : 0;
        }
    }
    a->x[0] = bf(q);
    a->x[1] = bf(k);
    a->w[0] = bf(q_norm);
    a->w[1] = bf(k_norm);
    a->heads[0] = (int)Hq;
    a->heads[1] = (int)Hk;
    a->cos = cos;
    a->sin = sin;
    a->max_pos = max_pos;
    a->rotary = (int)rotary;
    a->interleaved = interleaved;
    a->positions = positions;
    a->T = T;
    a->dim = (int)dim;
    a->eps = eps;
    a->dz[0] = a->dz[1] = nullptr;
    a->dw[0] = a->dw[1] = a->part = nullptr;
    return S3D8_OK;
}

// What both directions of cross attention share; sets everything but out, lse and the gradients.
int cross_args(CrossArgs *a, const void *q, const int64_t q_stride[2], const void *k, const int64_t k_stride[2], const void *v,
               const int64_t v_stride[2], const int32_t *spans, int64_t T, int64_t S, int64_t Hq, int64_t heads, int64_t dim,
               float scale)
{
    if (T < 0 || S < 0 || T > S3D8_MAX_M || S > S3D8_MAX_M || heads < 1 || Hq < 1 || Hq > 65535 || Hq % heads != 0 || dim < 8 ||
        dim % 8 != 0 || !isfinite(scale))
        return S3D8_ERR_INVALID_ARG;
    if (dim > S3D8_MAX_CROSS_DIM || Hq / heads > S3D8_MAX_CROSS_GROUP || T * Hq > kMaxInt || S * heads > kMaxInt)
        return S3D8_ERR_UNSUPPORTED;
    if (T > 0) {
        const int st = check_rows(q, q_stride);
        if (st != S3D8_OK)
            return st;
    }
    if (S > 0) {
        int st = check_rows(k, k_stride);
        if (st == S3D8_OK)
            st = check_rows(v, v_stride);
        if (st != S3D8_OK)
            return st;
    }
    if (!aligned(spans, 8))
        return S3D8_ERR_ALIGNMENT;
    for (int j = 0; j < 2; ++j) {
        a->qs[j] = T > 0 ? q_stride[j] : 0;
        a->ks[j] = S > 0 ? k_stride[j] : 0;
        a->vs[j] = S > 0 ? v_stride[j] : 0;
        a->ds[j] = 0;
    }
    a->q = bf(q);
    a->k = bf(k);
    a->v = bf(v);
    a->spans = spans;
    a->T = (int)T;
    a->S = (int)S;
    a->Hq = (int)Hq;
    a->heads = (int)heads;
    a->dim = (int)dim;
    a->scale = scale;
    a->dout = nullptr;
    a->dq = a->dk = a->dv = nullptr;
    return S3D8_OK;
}

bool cross_sizes_ok(int64_t T, int64_t S, int64_t Hq, int64_t heads, int64_t dim)
{
    CrossArgs a;
    const int64_t stride[2] = {0, 0};
    alignas(16) static const char some[16] = {};
    return T > 0 && cross_args(&a, some, stride, some, stride, some, stride, nullptr, T, S, Hq, heads, dim, 1.0f) == S3D8_OK;
}

}  // namespace

extern "C" {

int s3d8_norm_rope(const void *q_bf16, const int64_t q_stride[2], int64_t Hq, const void *k_bf16, const int64_t k_stride[2],
                   int64_t Hk, const void *q_norm_bf16, const void *k_norm_bf16, const float *cos, const float *sin,
                   int64_t max_pos, int64_t rotary, int interleaved, const int32_t *positions, int64_t T, int64_t dim, float eps,
                   void *q_out_bf16, void *k_out_bf16, void *stream)
{
    NormRopeArgs a;
    const int st = norm_rope_args(&a, q_bf16, q_stride, Hq, k_bf16, k_stride, Hk, q_norm_bf16, k_norm_bf16, cos, sin, max_pos,
                                  rotary, interleaved, positions, T, dim, eps);
    if (st != S3D8_OK || T == 0)
        return st;
    if (!q_out_bf16 || (Hk && !k_out_bf16))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(q_out_bf16, 16) || !aligned(k_out_bf16, 16))
        return S3D8_ERR_ALIGNMENT;
    a.out[0] = bf(q_out_bf16);
    a.out[1] = bf(k_out_bf16);
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

size_t s3d8_norm_rope_backward_workspace_size(int64_t T, int64_t Hq, int64_t Hk, int64_t dim)
{
    if (T <= 0 || T > S3D8_MAX_M || Hq < 1 || Hq > 65535 || Hk < 0 || Hk > 65535 || dim < 16 || dim > 256 || dim % 16 != 0)
        return 0;
    return norm_rope_backward_workspace(T, (int)(Hq + Hk), (int)dim);
}

int s3d8_norm_rope_backward(const void *dq_bf16, const int64_t dq_stride[2], const void *dk_bf16, const int64_t dk_stride[2],
                            const void *q_bf16, const int64_t q_stride[2], int64_t Hq, const void *k_bf16,
                            const int64_t k_stride[2], int64_t Hk, const void *q_norm_bf16, const void *k_norm_bf16,
                            const float *cos, const float *sin, int64_t max_pos, int64_t rotary, int interleaved,
                            const int32_t *positions, int64_t T, int64_t dim, float eps, void *dq_in_bf16, void *dk_in_bf16,
                            float *dq_norm, float *dk_norm, void *workspace, size_t workspace_bytes, void *stream)
{
    NormRopeArgs a;
    int st = norm_rope_args(&a, q_bf16, q_stride, Hq, k_bf16, k_stride, Hk, q_norm_bf16, k_norm_bf16, cos, sin, max_pos, rotary,
                            interleaved, positions, T, dim, eps);
    if (st != S3D8_OK)
        return st;
    if ((dq_norm != nullptr) != (q_norm_bf16 != nullptr) || (dk_norm != nullptr) != (k_norm_bf16 != nullptr))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(dq_norm, 4) || !aligned(dk_norm, 4))
        return S3D8_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // no rows: the weights' gradients are zero
        cudaError_t e = dq_norm ? cudaMemsetAsync(dq_norm, 0, dim * sizeof(float), s) : cudaSuccess;
        if (e == cudaSuccess && dk_norm)
            e = cudaMemsetAsync(dk_norm, 0, dim * sizeof(float), s);
        return cuda_status(e);
    }
    st = check_rows(dq_bf16, dq_stride);
    if (st == S3D8_OK && Hk)
        st = check_rows(dk_bf16, dk_stride);
    if (st != S3D8_OK)
        return st;
    if (!dq_in_bf16 || (Hk && !dk_in_bf16))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(dq_in_bf16, 16) || !aligned(dk_in_bf16, 16))
        return S3D8_ERR_ALIGNMENT;
    st = check_workspace(workspace, workspace_bytes, norm_rope_backward_workspace(T, (int)(Hq + Hk), (int)dim));
    if (st != S3D8_OK)
        return st;
    for (int j = 0; j < 2; ++j) {
        a.dzs[0][j] = dq_stride[j];
        a.dzs[1][j] = Hk ? dk_stride[j] : 0;
    }
    a.dz[0] = bf(dq_bf16);
    a.dz[1] = bf(dk_bf16);
    a.out[0] = bf(dq_in_bf16);
    a.out[1] = bf(dk_in_bf16);
    a.dw[0] = dq_norm;
    a.dw[1] = dk_norm;
    a.part = static_cast<float *>(workspace);
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_norm_rope_backward(a, s));
}

size_t s3d8_cross_attention_workspace_size(int64_t T, int64_t S, int64_t Hq, int64_t heads, int64_t dim)
{
    return cross_sizes_ok(T, S, Hq, heads, dim) ? cross_attention_workspace(T, S, Hq, heads, dim) : 0;
}

int s3d8_cross_attention(const void *q_bf16, const int64_t q_stride[2], const void *k_bf16, const int64_t k_stride[2],
                         const void *v_bf16, const int64_t v_stride[2], const int32_t *spans, int64_t T, int64_t S, int64_t Hq,
                         int64_t heads, int64_t dim, float scale, void *out_bf16, float *lse, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    CrossArgs a;
    int st = cross_args(&a, q_bf16, q_stride, k_bf16, k_stride, v_bf16, v_stride, spans, T, S, Hq, heads, dim, scale);
    if (st != S3D8_OK || T == 0)
        return st;
    if (!out_bf16)
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(out_bf16, 16) || !aligned(lse, 4))
        return S3D8_ERR_ALIGNMENT;
    st = check_workspace(workspace, workspace_bytes, cross_attention_workspace(T, S, Hq, heads, dim));
    if (st != S3D8_OK)
        return st;
    a.out = bf(out_bf16);
    a.lse = lse;
    a.ws = workspace;
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_cross_attention(a, static_cast<cudaStream_t>(stream)));
}

size_t s3d8_cross_attention_backward_workspace_size(int64_t T, int64_t S, int64_t Hq, int64_t heads, int64_t dim)
{
    return cross_sizes_ok(T, S, Hq, heads, dim) ? cross_attention_backward_workspace(T, S, Hq, heads, dim) : 0;
}

int s3d8_cross_attention_backward(const void *dout_bf16, const int64_t dout_stride[2], const void *q_bf16,
                                  const int64_t q_stride[2], const void *k_bf16, const int64_t k_stride[2], const void *v_bf16,
                                  const int64_t v_stride[2], const void *out_bf16, const float *lse, const int32_t *spans,
                                  int64_t T, int64_t S, int64_t Hq, int64_t heads, int64_t dim, float scale, void *dq_bf16,
                                  void *dk_bf16, void *dv_bf16, void *workspace, size_t workspace_bytes, void *stream)
{
    CrossArgs a;
    int st = cross_args(&a, q_bf16, q_stride, k_bf16, k_stride, v_bf16, v_stride, spans, T, S, Hq, heads, dim, scale);
    if (st != S3D8_OK || (T == 0 && S == 0))
        return st;
    if ((T > 0 && (!out_bf16 || !lse || !dq_bf16)) || (S > 0 && (!dk_bf16 || !dv_bf16)))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(out_bf16, 16) || !aligned(lse, 4) || !aligned(dq_bf16, 16) || !aligned(dk_bf16, 16) || !aligned(dv_bf16, 16))
        return S3D8_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {       // no tokens: the states' gradients are zero
        const size_t bytes = (size_t)S * heads * dim * sizeof(__nv_bfloat16);
        const cudaError_t e = cudaMemsetAsync(dk_bf16, 0, bytes, s);
        return cuda_status(e == cudaSuccess ? cudaMemsetAsync(dv_bf16, 0, bytes, s) : e);
    }
    st = check_rows(dout_bf16, dout_stride);
    if (st == S3D8_OK)
        st = check_workspace(workspace, workspace_bytes, cross_attention_backward_workspace(T, S, Hq, heads, dim));
    if (st != S3D8_OK)
        return st;
    a.dout = bf(dout_bf16);
    a.ds[0] = dout_stride[0];
    a.ds[1] = dout_stride[1];
    a.out = const_cast<__nv_bfloat16 *>(bf(out_bf16));
    a.lse = const_cast<float *>(lse);
    a.dq = bf(dq_bf16);
    a.dk = bf(dk_bf16);
    a.dv = bf(dv_bf16);
    a.ws = workspace;
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_cross_attention_backward(a, s));
}

int s3d8_sample(const void *logits_bf16, int64_t logits_stride, int64_t B, int64_t V, const float *u, const float *temperature,
                const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens, float *logprob, void *stream)
{
    if (B < 0 || B > S3D8_MAX_M || V < 1 || logits_stride < 0)
        return S3D8_ERR_INVALID_ARG;
    if (V > S3D8_MAX_SAMPLE_V)
        return S3D8_ERR_UNSUPPORTED;
    if (B == 0)
        return S3D8_OK;
    if (!logits_bf16 || !u || !tokens)
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(logits_bf16, 2) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
        !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprob, 4))
        return S3D8_ERR_ALIGNMENT;
    SampleArgs a;
    a.logits = bf(logits_bf16);
    a.stride = logits_stride;
    a.B = (int)B;
    a.V = (int)V;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.logprob = logprob;
    return cuda_status(launch_sample(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
