// C ABI of the calls between two linears: argument checks and launches.  As in
// api.cu, every check runs before the first CUDA call.
#include "../../include/s3d8.h"
#include "launch.h"

#include <cuda_runtime.h>

using namespace s3d8;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? S3D8_OK : S3D8_ERR_CUDA; }

constexpr int64_t kMaxInt = 0x7FFFFFFF;

const __nv_bfloat16 *bf(const void *p) { return static_cast<const __nv_bfloat16 *>(p); }

// The parts of a norm call that both directions share.
int check_norm(const void *h, const void *y, const void *w_post, const void *gate, int64_t gate_n, const void *w_pre,
               int64_t M, int64_t D)
{
    if (M < 0 || M > S3D8_MAX_M || D < 8 || D % 8 != 0 || D > S3D8_MAX_NORM_D)
        return S3D8_ERR_INVALID_ARG;
    if ((gate != nullptr) != (gate_n != 0) || (gate_n != 0 && gate_n != 1 && gate_n != D))
        return S3D8_ERR_INVALID_ARG;
    if (M > 0 && (!h || (!y && (w_post || gate || !w_pre))))   // of no rows, y may be null
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(h, 16) || !aligned(y, 16) || !aligned(w_post, 16) || !aligned(w_pre, 16) ||
        !aligned(gate, gate_n == 1 ? 2 : 16))
        return S3D8_ERR_ALIGNMENT;
    return S3D8_OK;
}

int check_cache(const s3d8_kv_cache *c, KvCache *out)
{
    if (!c || !c->k || !c->v || c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->heads > 65535 || c->dim < 16 ||
        c->dim > 256 || c->dim % 16 != 0 || (c->dtype != S3D8_KV_BF16 && c->dtype != S3D8_KV_INT8))
        return S3D8_ERR_INVALID_ARG;
    if (c->pages > kMaxInt / c->page_size || (int64_t)c->heads * c->dim > kMaxInt / c->page_size)
        return S3D8_ERR_INVALID_ARG;
    const bool int8 = c->dtype == S3D8_KV_INT8;
    if (int8 && (!c->k_scale || !c->v_scale))
        return S3D8_ERR_INVALID_ARG;
    const int unit = int8 ? 16 : 8;
    for (int i = 0; i < 3; ++i) {
        if (c->k_stride[i] < 0 || c->v_stride[i] < 0 || (int8 && c->scale_stride[i] < 0))
            return S3D8_ERR_INVALID_ARG;
        if (c->k_stride[i] / unit > 0xFFFFFFFFLL || c->v_stride[i] / unit > 0xFFFFFFFFLL ||
            (int8 && c->scale_stride[i] > 0xFFFFFFFFLL))
            return S3D8_ERR_UNSUPPORTED;   // 64 GB from one page to the next
        if (c->k_stride[i] % unit != 0 || c->v_stride[i] % unit != 0)
            return S3D8_ERR_ALIGNMENT;
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || (int8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))))
        return S3D8_ERR_ALIGNMENT;
    out->k = c->k;
    out->v = c->v;
    out->k_scale = int8 ? c->k_scale : nullptr;
    out->v_scale = int8 ? c->v_scale : nullptr;
    for (int i = 0; i < 3; ++i) {
        out->ks[i] = c->k_stride[i];
        out->vs[i] = c->v_stride[i];
        out->ss[i] = int8 ? c->scale_stride[i] : 0;
    }
    out->pages = (int)c->pages;
    out->page_size = c->page_size;
    out->heads = c->heads;
    out->dim = c->dim;
    out->int8 = int8;
    return S3D8_OK;
}

bool same_geometry(const KvCache &a, const KvCache &b)
{
    for (int i = 0; i < 3; ++i)
        if (a.ks[i] != b.ks[i] || a.vs[i] != b.vs[i] || a.ss[i] != b.ss[i])
            return false;
    return a.pages == b.pages && a.page_size == b.page_size && a.heads == b.heads && a.dim == b.dim && a.int8 == b.int8;
}

int check_layers(const s3d8_kv_cache *layers, int64_t count, KvCache *geo)
{
    if (!layers || count < 1 || count > 65536)
        return S3D8_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        KvCache c;
        const int st = check_cache(layers + i, &c);
        if (st != S3D8_OK)
            return st;
        if (i == 0)
            *geo = c;
        else if (!same_geometry(*geo, c))
            return S3D8_ERR_INVALID_ARG;
    }
    return S3D8_OK;
}

// The page copies of a pool, kPoolLayers layers a launch.
cudaError_t copy_layers(const s3d8_kv_cache *layers, int64_t count, const KvCache &geo, const int32_t *src,
                        const int32_t *dst, const int32_t *tokens, int n, const int32_t *on_device, int *status,
                        cudaStream_t stream)
{
    PoolArgs p;
    p.geo = geo;
    for (int64_t at = 0; at < count; at += kPoolLayers) {
        p.layers = (int)(count - at < kPoolLayers ? count - at : kPoolLayers);
        for (int i = 0; i < p.layers; ++i) {
            p.k[i] = layers[at + i].k;
            p.v[i] = layers[at + i].v;
            p.k_scale[i] = geo.int8 ? layers[at + i].k_scale : nullptr;
            p.v_scale[i] = geo.int8 ? layers[at + i].v_scale : nullptr;
        }
        const cudaError_t e = launch_copy_pages(p, src, dst, tokens, n, on_device, status, stream);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

int check_tables(const int32_t *table, int64_t rows, int64_t width, const int32_t *refs, int64_t pages)
{
    if (rows < 0 || width < 0 || rows > S3D8_MAX_M || width > kMaxInt || pages < 1 || pages > kMaxInt - 4096)
        return S3D8_ERR_INVALID_ARG;
    if (!refs || (!table && rows * width > 0))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(table, 4) || !aligned(refs, 4))
        return S3D8_ERR_ALIGNMENT;
    return S3D8_OK;
}

int check_workspace(const void *ws, size_t bytes, size_t need)
{
    if (!ws || bytes < need)
        return S3D8_ERR_WORKSPACE;
    return aligned(ws, 16) ? S3D8_OK : S3D8_ERR_ALIGNMENT;
}

}  // namespace

extern "C" {

int s3d8_residual_norm(const void *h_bf16, const void *y_bf16, const void *w_post_bf16, const void *gate_bf16,
                       int64_t gate_n, int tanh_gate, const void *w_pre_bf16, float alpha, float eps, int64_t M, int64_t D,
                       void *h_out_bf16, void *x_bf16, int8_t *xq, float *xscale, void *stream)
{
    int st = check_norm(h_bf16, y_bf16, w_post_bf16, gate_bf16, gate_n, w_pre_bf16, M, D);
    if (st != S3D8_OK)
        return st;
    if ((xq != nullptr) != (xscale != nullptr) || (xq && D % 16 != 0))
        return S3D8_ERR_INVALID_ARG;
    if (M == 0)
        return S3D8_OK;
    if ((h_out_bf16 != nullptr) != (y_bf16 != nullptr) || (w_pre_bf16 != nullptr) != (x_bf16 || xq) || (x_bf16 && xq))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(h_out_bf16, 16) || !aligned(x_bf16, 16) || !aligned(xq, 16) || !aligned(xscale, 4))
        return S3D8_ERR_ALIGNMENT;
    NormArgs a;
    a.h = bf(h_bf16);
    a.y = bf(y_bf16);
    a.w_post = bf(w_post_bf16);
    a.gate = bf(gate_bf16);
    a.w_pre = bf(w_pre_bf16);
    a.gate_n = (int)gate_n;
    a.tanh_gate = tanh_gate;
    a.alpha = alpha;
    a.eps = eps;
    a.M = (int)M;
    a.D = (int)D;
    a.h_out = static_cast<__nv_bfloat16 *>(h_out_bf16);
    a.x = static_cast<__nv_bfloat16 *>(x_bf16);
    a.xq = xq;
    a.xscale = xscale;
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_residual_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t s3d8_residual_norm_backward_workspace_size(int64_t M, int64_t D)
{
    if (M <= 0 || M > S3D8_MAX_M || D < 8 || D % 8 != 0 || D > S3D8_MAX_NORM_D)
        return 0;
    return residual_norm_backward_workspace(M, D);
}

int s3d8_residual_norm_backward(const void *dh_bf16, const void *dx_bf16, const void *h_bf16, const void *y_bf16,
                                const void *w_post_bf16, const void *gate_bf16, int64_t gate_n, int tanh_gate,
                                const void *w_pre_bf16, float alpha, float eps, int64_t M, int64_t D, void *dh_in_bf16,
                                void *dy_bf16, float *dw_pre, float *dw_post, float *dgate, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    int st = check_norm(h_bf16, y_bf16, w_post_bf16, gate_bf16, gate_n, w_pre_bf16, M, D);
    if (st != S3D8_OK)
        return st;
    if ((dx_bf16 && !w_pre_bf16) || (dw_pre != nullptr) != (w_pre_bf16 != nullptr) ||
        (dw_post != nullptr) != (w_post_bf16 != nullptr) || (dgate != nullptr) != (gate_bf16 != nullptr))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(dw_pre, 16) || !aligned(dw_post, 16) || !aligned(dgate, 4))
        return S3D8_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {   // no rows: the weights' gradients are zero
        cudaError_t e = dw_pre ? cudaMemsetAsync(dw_pre, 0, D * sizeof(float), s) : cudaSuccess;
        if (e == cudaSuccess && dw_post)
            e = cudaMemsetAsync(dw_post, 0, D * sizeof(float), s);
        if (e == cudaSuccess && dgate)
            e = cudaMemsetAsync(dgate, 0, gate_n * sizeof(float), s);
        return cuda_status(e);
    }
    if (!dh_in_bf16 || (dy_bf16 != nullptr) != (y_bf16 != nullptr))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(dh_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(dh_in_bf16, 16) || !aligned(dy_bf16, 16))
        return S3D8_ERR_ALIGNMENT;
    st = check_workspace(workspace, workspace_bytes, residual_norm_backward_workspace(M, D));
    if (st != S3D8_OK)
        return st;
    NormGradArgs g;
    g.f.h = bf(h_bf16);
    g.f.y = bf(y_bf16);
    g.f.w_post = bf(w_post_bf16);
    g.f.gate = bf(gate_bf16);
    g.f.w_pre = bf(w_pre_bf16);
    g.f.gate_n = (int)gate_n;
    g.f.tanh_gate = tanh_gate;
    g.f.alpha = alpha;
    g.f.eps = eps;
    g.f.M = (int)M;
    g.f.D = (int)D;
    g.f.h_out = g.f.x = nullptr;
    g.f.xq = nullptr;
    g.f.xscale = nullptr;
    g.dh = bf(dh_bf16);
    g.dx = bf(dx_bf16);
    g.dh_in = static_cast<__nv_bfloat16 *>(dh_in_bf16);
    g.dy = static_cast<__nv_bfloat16 *>(dy_bf16);
    g.dw_pre = dw_pre;
    g.dw_post = dw_post;
    g.dgate = dgate;
    g.part = static_cast<float *>(workspace);
    if (!(g.f.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_residual_norm_backward(g, s));
}

int s3d8_norm_rope_append(const void *q_bf16, const int64_t q_stride[2], const void *k_bf16, const int64_t k_stride[2],
                     const void *v_bf16, const int64_t v_stride[2], const float *cos, const float *sin, int64_t max_pos,
                     int64_t rotary, int interleaved, const int32_t *positions, const int32_t *rows, int64_t T, int64_t Hq,
                     const int32_t *table, int64_t table_rows, int64_t width, const void *q_norm_bf16, const void *k_norm_bf16, float eps,
                          const s3d8_kv_cache *cache, void *q_out_bf16, void *stream)
{
    RopeArgs a;
    int st = check_cache(cache, &a.kv);
    if (st != S3D8_OK)
        return st;
    if (T < 0 || T > S3D8_MAX_M || Hq < 1 || Hq > 65535 || rotary < 0 || rotary % 2 != 0 || rotary > cache->dim ||
        max_pos < 0 || table_rows < 0 || width < 0 || table_rows > kMaxInt || width > kMaxInt || !q_stride || !k_stride ||
        !v_stride)
        return S3D8_ERR_INVALID_ARG;
    if (T == 0)
        return S3D8_OK;
    if (!q_bf16 || !k_bf16 || !v_bf16 || !positions || !q_out_bf16 || (rotary && (!cos || !sin)) ||
        (!table && table_rows * width > 0))
        return S3D8_ERR_INVALID_ARG;
    const int64_t *strides[3] = {q_stride, k_stride, v_stride};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 2; ++j) {
            if (strides[i][j] < 0)
                return S3D8_ERR_INVALID_ARG;
            if (strides[i][j] % 8 != 0)
                return S3D8_ERR_ALIGNMENT;
        }
    if (!aligned(q_bf16, 16) || !aligned(k_bf16, 16) || !aligned(v_bf16, 16) || !aligned(q_out_bf16, 16) ||
        !aligned(cos, 4) || !aligned(sin, 4) || !aligned(positions, 4) || !aligned(rows, 4) || !aligned(table, 4) ||
        !aligned(q_norm_bf16, 16) || !aligned(k_norm_bf16, 16))
        return S3D8_ERR_ALIGNMENT;
    a.q = bf(q_bf16);
    a.k = bf(k_bf16);
    a.v = bf(v_bf16);
    for (int j = 0; j < 2; ++j) {
        a.qs[j] = q_stride[j];
        a.ks[j] = k_stride[j];
        a.vs[j] = v_stride[j];
    }
    a.cos = cos;
    a.sin = sin;
    a.max_pos = max_pos;
    a.rotary = (int)rotary;
    a.interleaved = interleaved;
    a.positions = positions;
    a.rows = rows;
    a.T = T;
    a.Hq = (int)Hq;
    a.table = table;
    a.table_rows = table_rows;
    a.width = width;
    a.q_out = static_cast<__nv_bfloat16 *>(q_out_bf16);
    a.q_norm = bf(q_norm_bf16);
    a.k_norm = bf(k_norm_bf16);
    a.eps = eps;
    a.status = device_status_ptr();
    if (!a.status)
        return S3D8_ERR_CUDA;
    return cuda_status(launch_rope_append(a, static_cast<cudaStream_t>(stream)));
}

int s3d8_rope_append(const void *q_bf16, const int64_t q_stride[2], const void *k_bf16, const int64_t k_stride[2],
                     const void *v_bf16, const int64_t v_stride[2], const float *cos, const float *sin, int64_t max_pos,
                     int64_t rotary, int interleaved, const int32_t *positions, const int32_t *rows, int64_t T, int64_t Hq,
                     const int32_t *table, int64_t table_rows, int64_t width, const s3d8_kv_cache *cache, void *q_out_bf16,
                     void *stream)
{
    return s3d8_norm_rope_append(q_bf16, q_stride, k_bf16, k_stride, v_bf16, v_stride, cos, sin, max_pos, rotary, interleaved,
                                 positions, rows, T, Hq, table, table_rows, width, nullptr, nullptr, 0.0f, cache, q_out_bf16,
                                 stream);
}

size_t s3d8_paged_attention_workspace_size(const s3d8_kv_cache *cache, int64_t B, int64_t Hq)
{
    KvCache kv;
    if (check_cache(cache, &kv) != S3D8_OK || B <= 0 || B > S3D8_MAX_M || Hq < 1 || Hq > 65535 || Hq % kv.heads != 0)
        return 0;
    return paged_attention_workspace(kv, B, Hq);
}

int s3d8_paged_attention(const void *q_bf16, const s3d8_kv_cache *cache, const int32_t *table, int64_t width,
                         const int32_t *lens, int64_t B, int64_t Hq, float scale, int64_t window, void *out_bf16,
                         float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    AttnArgs a;
    int st = check_cache(cache, &a.kv);
    if (st != S3D8_OK)
        return st;
    if (B < 0 || B > S3D8_MAX_M || Hq < 1 || Hq > 65535 || Hq % a.kv.heads != 0 || B * Hq > kMaxInt || width < 0 ||
        width > (kMaxInt - 64) / a.kv.page_size || window < 0)
        return S3D8_ERR_INVALID_ARG;
    if (B == 0)
        return S3D8_OK;
    if (!q_bf16 || !lens || !out_bf16 || (!table && width > 0))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16) || !aligned(lens, 4) || !aligned(table, 4) || !aligned(lse, 4))
        return S3D8_ERR_ALIGNMENT;
    st = check_workspace(workspace, workspace_bytes, paged_attention_workspace(a.kv, B, Hq));
    if (st != S3D8_OK)
        return st;
    a.q = bf(q_bf16);
    a.table = table;
    a.lens = lens;
    a.width = width;
    a.B = (int)B;
    a.Hq = (int)Hq;
    a.scale = scale;
    a.window = window;
    a.out = static_cast<__nv_bfloat16 *>(out_bf16);
    a.lse = lse;
    a.ws = workspace;
    a.status = device_status_ptr();
    if (!a.status)
        return S3D8_ERR_CUDA;
    return cuda_status(launch_paged_attention(a, static_cast<cudaStream_t>(stream)));
}

size_t s3d8_pages_workspace_size(int64_t pages, int64_t rows)
{
    if (pages < 1 || pages > kMaxInt - 4096 || rows < 0 || rows > S3D8_MAX_M)
        return 0;
    return pages_workspace(pages, rows);
}

int s3d8_copy_pages(const s3d8_kv_cache *layers, int64_t count, const int32_t *src, const int32_t *dst, int64_t n,
                    void *stream)
{
    KvCache geo;
    int st = check_layers(layers, count, &geo);
    if (st != S3D8_OK)
        return st;
    if (n < 0 || n > kMaxInt)
        return S3D8_ERR_INVALID_ARG;
    if (n == 0)
        return S3D8_OK;
    if (!src || !dst)
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4))
        return S3D8_ERR_ALIGNMENT;
    int *status = device_status_ptr();
    if (!status)
        return S3D8_ERR_CUDA;
    return cuda_status(copy_layers(layers, count, geo, src, dst, nullptr, (int)n, nullptr, status,
                                   static_cast<cudaStream_t>(stream)));
}

// The arguments that the calls on the tables share; `n` distinct rows at most.
static int page_args(PagesArgs *a, int32_t *table, int64_t rows, int64_t width, int32_t *lens, int32_t *refs, int64_t pages,
                     int64_t page_size, const int32_t *who, const int32_t *other, bool two, int64_t n, int32_t *got,
                     bool needs_got, void *ws)
{
    if (n < 0 || n > rows || page_size < 1 || page_size > kMaxInt)
        return S3D8_ERR_INVALID_ARG;
    if (n > 0 && (!lens || !who || (two && !other) || (needs_got && !got)))
        return S3D8_ERR_INVALID_ARG;
    if (!aligned(lens, 4) || !aligned(who, 4) || !aligned(other, 4) || !aligned(got, 4))
        return S3D8_ERR_ALIGNMENT;
    a->table = table;
    a->lens = lens;
    a->refs = refs;
    a->rows = rows;
    a->width = width;
    a->pages = (int)pages;
    a->page_size = (int)page_size;
    a->who = who;
    a->other = other;
    a->n = (int)n;
    a->got = got;
    a->ws = static_cast<int32_t *>(ws);
    return S3D8_OK;
}

int s3d8_extend_pages(int32_t *table, int64_t rows, int64_t width, int32_t *lens, int32_t *refs, int64_t pages,
                      int64_t page_size, const int32_t *seqs, const int32_t *add, int64_t n, int32_t *got, void *workspace,
                      size_t workspace_bytes, void *stream)
{
    int st = check_tables(table, rows, width, refs, pages);
    PagesArgs a;
    if (st == S3D8_OK)
        st = page_args(&a, table, rows, width, lens, refs, pages, page_size, seqs, add, true, n, got, true, workspace);
    if (st != S3D8_OK || n == 0)
        return st;
    st = check_workspace(workspace, workspace_bytes, pages_workspace(pages, rows));
    if (st != S3D8_OK)
        return st;
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_extend_pages(a, static_cast<cudaStream_t>(stream)));
}

int s3d8_fork_pages(const s3d8_kv_cache *layers, int64_t count, int32_t *table, int64_t rows, int64_t width, int32_t *lens,
                    int32_t *refs, const int32_t *parents, const int32_t *children, int64_t n, int32_t *got, void *workspace,
                    size_t workspace_bytes, void *stream)
{
    KvCache geo;
    int st = check_layers(layers, count, &geo);
    if (st == S3D8_OK)
        st = check_tables(table, rows, width, refs, geo.pages);
    PagesArgs a;
    if (st == S3D8_OK)
        st = page_args(&a, table, rows, width, lens, refs, geo.pages, geo.page_size, parents, children, true, n, got, true,
                       workspace);
    if (st != S3D8_OK || n == 0)
        return st;
    st = check_workspace(workspace, workspace_bytes, pages_workspace(geo.pages, rows));
    if (st != S3D8_OK)
        return st;
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    PagePairs pairs;
    cudaError_t e = launch_fork_pages(a, &pairs, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess)
        e = copy_layers(layers, count, geo, pairs.src, pairs.dst, pairs.tokens, (int)n, pairs.count, a.status,
                        static_cast<cudaStream_t>(stream));
    return cuda_status(e);
}

int s3d8_free_pages(int32_t *table, int64_t rows, int64_t width, int32_t *lens, int32_t *refs, int64_t pages,
                    const int32_t *seqs, int64_t n, void *stream)
{
    int st = check_tables(table, rows, width, refs, pages);
    PagesArgs a;
    if (st == S3D8_OK)
        st = page_args(&a, table, rows, width, lens, refs, pages, 1, seqs, nullptr, false, n, nullptr, false, nullptr);
    if (st != S3D8_OK || n == 0)
        return st;
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    return cuda_status(launch_free_pages(a, static_cast<cudaStream_t>(stream)));
}

int s3d8_compact_pages(const s3d8_kv_cache *layers, int64_t count, int32_t *table, int64_t rows, int64_t width,
                       int32_t *refs, int32_t *live, void *workspace, size_t workspace_bytes, void *stream)
{
    KvCache geo;
    int st = check_layers(layers, count, &geo);
    if (st == S3D8_OK)
        st = check_tables(table, rows, width, refs, geo.pages);
    PagesArgs a;
    if (st == S3D8_OK)
        st = page_args(&a, table, rows, width, nullptr, refs, geo.pages, geo.page_size, nullptr, nullptr, false, 0, live,
                       true, workspace);
    if (st != S3D8_OK)
        return st;
    if (!live)
        return S3D8_ERR_INVALID_ARG;
    st = check_workspace(workspace, workspace_bytes, pages_workspace(geo.pages, rows));
    if (st != S3D8_OK)
        return st;
    if (!(a.status = device_status_ptr()))
        return S3D8_ERR_CUDA;
    PagePairs pairs;
    cudaError_t e = launch_compact_pages(a, &pairs, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess)
        e = copy_layers(layers, count, geo, pairs.src, pairs.dst, pairs.tokens, geo.pages / 2, pairs.count, a.status,
                        static_cast<cudaStream_t>(stream));
    return cuda_status(e);
}

}  // extern "C"
