// gdn_recurrence.cu -- gated linear recurrence (include/gdn.h): forward, backward
// and the single-token step, with their C entry points.
#include <string.h>

#include "gdn_layer_ops.cuh"
#include "gdn_recurrence.cuh"

namespace gdn {
namespace {

struct RecProblem {
    gdn_recurrence_desc d;
    const void *x, *a, *b, *grad_out;
    const float *A_log, *dt_bias;
    const int32_t *cu;
    const float *h0;
    void *out;
    float *hT, *cs;              // final states; states carried into every 64th token
    int32_t *status;
    const float *grad_final;
    void *dx, *da, *db;
    float *dA_log, *ddt_bias, *dh0, *part;
};

__device__ __forceinline__ Gate2 gate1(float a, float b, float bias, float rate2) {
    return gate2(splat2(a), splat2(b), splat2(bias), splat2(rate2));
}

// One thread per (sequence, channel) walks the sequence.
template <typename T>
__global__ void __launch_bounds__(128) rec_forward_kernel(const RecProblem p) {
    const gdn_recurrence_desc &d = p.d;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    const int c = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y;
    if (!ok || c >= d.D) return;
    const int row = p.cu ? 0 : n;
    const int t0 = p.cu ? p.cu[n] : 0, t1 = p.cu ? p.cu[n + 1] : d.T;
    const float rate2 = -expf(p.A_log[c]) * kLog2e, bias = p.dt_bias[c];
    const T *x = (const T *)p.x + row * d.x_stride_b + c;
    const T *a = (const T *)p.a + row * d.a_stride_b + c;
    const T *b = (const T *)p.b + row * d.b_stride_b + c;
    float h = p.h0 ? p.h0[(int64_t)n * d.D + c] : 0.f;
    const int64_t chunks = (d.T + GDN_RECURRENCE_CHUNK - 1) / GDN_RECURRENCE_CHUNK;
    for (int t = t0; t < t1; ++t) {
        if (p.cs && t % GDN_RECURRENCE_CHUNK == 0)
            p.cs[((int64_t)row * chunks + t / GDN_RECURRENCE_CHUNK) * d.D + c] = h;
        const Gate2 g = gate1(to_f<T>(a[t * d.a_stride_t]), to_f<T>(b[t * d.b_stride_t]), bias, rate2);
        h = fmaf(g.alpha.x, h, g.s.x * g.beta.x * to_f<T>(x[t * d.x_stride_t]));
        if (p.out) ((T *)p.out)[((int64_t)row * d.T + t) * d.D + c] = from_f<T>(h);
    }
    if (p.hT) p.hT[(int64_t)n * d.D + c] = h;
}

// One thread per (sequence, channel): chunks last to first, each recomputed forward
// from its carried state, then walked backward.
template <typename T>
__global__ void __launch_bounds__(128) rec_backward_kernel(const RecProblem p) {
    const gdn_recurrence_desc &d = p.d;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    const int c = blockIdx.x * 128 + threadIdx.x, n = blockIdx.y;
    if (!ok || c >= d.D) return;
    const int row = p.cu ? 0 : n;
    const int t0 = p.cu ? p.cu[n] : 0, t1 = p.cu ? p.cu[n + 1] : d.T;
    const float rate2 = -expf(p.A_log[c]) * kLog2e, bias = p.dt_bias[c];
    const T *x = (const T *)p.x + row * d.x_stride_b + c;
    const T *a = (const T *)p.a + row * d.a_stride_b + c;
    const T *b = (const T *)p.b + row * d.b_stride_b + c;
    const int64_t chunks = (d.T + GDN_RECURRENCE_CHUNK - 1) / GDN_RECURRENCE_CHUNK;
    float carry = p.grad_final ? p.grad_final[(int64_t)n * d.D + c] : 0.f;
    float sA = 0.f, sb = 0.f;
    float hp[GDN_RECURRENCE_CHUNK];
    for (int q1 = t1; q1 > t0;) {
        const int k = (q1 - 1) / GDN_RECURRENCE_CHUNK;
        const int q0 = max(t0, k * GDN_RECURRENCE_CHUNK);
        float h = q0 == t0 ? (p.h0 ? p.h0[(int64_t)n * d.D + c] : 0.f) : p.cs[((int64_t)row * chunks + k) * d.D + c];
        for (int t = q0; t < q1; ++t) {
            hp[t - q0] = h;
            const Gate2 g = gate1(to_f<T>(a[t * d.a_stride_t]), to_f<T>(b[t * d.b_stride_t]), bias, rate2);
            h = fmaf(g.alpha.x, h, g.s.x * g.beta.x * to_f<T>(x[t * d.x_stride_t]));
        }
        for (int t = q1 - 1; t >= q0; --t) {
            const int64_t o = ((int64_t)row * d.T + t) * d.D + c;
            const Gate2 g = gate1(to_f<T>(a[t * d.a_stride_t]), to_f<T>(b[t * d.b_stride_t]), bias, rate2);
            const float xv = to_f<T>(x[t * d.x_stride_t]);
            const float del = to_f<T>(((const T *)p.grad_out)[o]) + carry;
            carry = g.alpha.x * del;
            const float sg = sigmoid_from_t(g.z, g.t).x;
            ((T *)p.dx)[o] = from_f<T>(del * g.s.x * g.beta.x);
            ((T *)p.db)[o] = from_f<T>(del * g.s.x * g.beta.x * (1.f - g.beta.x) * xv);
            const float dg = del * (g.alpha.x * hp[t - q0] - g.beta.x * xv * g.alpha.x * g.alpha.x * g.rs.x);
            const float dz = dg * rate2 * (1.f / kLog2e) * sg;
            ((T *)p.da)[o] = from_f<T>(dz);
            sb += dz;
            sA += dg * g.G.x * (1.f / kLog2e);
        }
        q1 = q0;
    }
    if (p.dh0) p.dh0[(int64_t)n * d.D + c] = carry;
    p.part[((int64_t)n * 2) * d.D + c] = sA;
    p.part[((int64_t)n * 2 + 1) * d.D + c] = sb;
}

__global__ void __launch_bounds__(128) rec_params_kernel(const RecProblem p, int parts) {
    const int c = blockIdx.x * 128 + threadIdx.x;
    if (c >= p.d.D || *p.status != GDN_OK) return;
    float sA = 0.f, sb = 0.f;
    for (int i = 0; i < parts; ++i) {
        sA += p.part[((int64_t)i * 2) * p.d.D + c];
        sb += p.part[((int64_t)i * 2 + 1) * p.d.D + c];
    }
    p.dA_log[c] = sA;
    p.ddt_bias[c] = sb;
}

template <typename T>
__global__ void __launch_bounds__(128) rec_step_kernel(const RecProblem p, float *state) {
    const gdn_recurrence_desc &d = p.d;
    const int c = blockIdx.x * 128 + threadIdx.x;
    const int64_t n = blockIdx.y;
    if (c >= d.D) return;
    const Gate2 g = gate1(to_f<T>(((const T *)p.a)[n * d.a_stride_b + c]), to_f<T>(((const T *)p.b)[n * d.b_stride_b + c]),
                          p.dt_bias[c], -expf(p.A_log[c]) * kLog2e);
    const float h = fmaf(g.alpha.x, state[n * d.D + c],
                         g.s.x * g.beta.x * to_f<T>(((const T *)p.x)[n * d.x_stride_b + c]));
    state[n * d.D + c] = h;
    ((T *)p.out)[n * d.D + c] = from_f<T>(h);
}

template <typename F>
int by_dtype(int dtype, F &&f) {
    switch (dtype) {
    case GDN_F32: return f((float)0);
    case GDN_BF16: return f(__nv_bfloat16());
    default: return f(__half());
    }
}

int check_desc(const gdn_recurrence_desc *d, bool packed) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->N < 1 || d->D < 1) return GDN_ERR_INVALID_ARG;
    if (packed ? d->B != 1 : d->N != d->B) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return GDN_ERR_UNSUPPORTED;
    const int64_t strides[] = {d->x_stride_b, d->x_stride_t, d->a_stride_b, d->a_stride_t, d->b_stride_b, d->b_stride_t};
    for (int64_t s : strides)
        if (s < 0) return GDN_ERR_INVALID_ARG;
    if (d->T > 1 && (d->x_stride_t < d->D || d->a_stride_t < d->D || d->b_stride_t < d->D)) return GDN_ERR_INVALID_ARG;
    if ((double)d->B * d->T * d->D > 4.0e12 || (double)d->N * d->D > 1.0e12) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

struct RecLayout {
    size_t status, part, cs, total;
};
RecLayout bwd_layout(const gdn_recurrence_desc &d) {
    RecLayout L;
    size_t off = 0;
    const size_t chunks = ((size_t)d.T + GDN_RECURRENCE_CHUNK - 1) / GDN_RECURRENCE_CHUNK;
    L.status = off; off += kStatusBytes;
    L.part = off;   off = align_up(off + (size_t)d.N * 2 * d.D * 4, 256);
    L.cs = off;     off = align_up(off + (size_t)d.B * chunks * d.D * 4, 256);
    L.total = off;
    return L;
}

bool act_aligned(int dtype, const void *p) { return ptr_aligned(p, act_size(dtype)); }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_recurrence_desc_init(gdn_recurrence_desc *d, int B, int T, int packed, int D, int dtype) {
    if (!d) return GDN_ERR_INVALID_ARG;
    memset(d, 0, sizeof(*d));
    d->B = B;
    d->T = T;
    d->N = packed ? packed : B;
    d->D = D;
    d->dtype = dtype;
    d->x_stride_t = d->a_stride_t = d->b_stride_t = D;
    d->x_stride_b = d->a_stride_b = d->b_stride_b = (int64_t)D * T;
    return check_desc(d, packed != 0);
}

int gdn_recurrence_workspace_bytes(const gdn_recurrence_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

int gdn_recurrence_backward_workspace_bytes(const gdn_recurrence_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = bwd_layout(*d).total;
    return GDN_OK;
}

int gdn_recurrence_forward(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b,
                           const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                           const float *initial_state, void *out, float *final_state, float *chunk_states,
                           void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d, cu_seqlens != nullptr);
    if (rc != GDN_OK) return rc;
    const bool tok = (int64_t)d->B * d->T > 0;   // token tensors may be empty (null)
    if ((tok && (!x || !a || !b || !out)) || !A_log || !dt_bias) return GDN_ERR_INVALID_ARG;
    if (!act_aligned(d->dtype, x) || !act_aligned(d->dtype, a) || !act_aligned(d->dtype, b) ||
        !act_aligned(d->dtype, out) || !ptr_aligned(A_log, 4) || !ptr_aligned(dt_bias, 4) ||
        !ptr_aligned(cu_seqlens, 4) || !ptr_aligned(initial_state, 4) || !ptr_aligned(final_state, 4) ||
        !ptr_aligned(chunk_states, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    RecProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.a = a;
    p.b = b;
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.cu = cu_seqlens;
    p.h0 = initial_state;
    p.out = out;
    p.hT = final_state;
    p.cs = chunk_states;
    p.status = (int32_t *)workspace;
    return by_dtype(d->dtype, [&](auto t) {
        rec_forward_kernel<decltype(t)><<<dim3((d->D + 127) / 128, d->N), 128, 0, (cudaStream_t)stream>>>(p);
        return layer_status(cudaGetLastError());
    });
}

int gdn_recurrence_backward(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b,
                            const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                            const float *initial_state, const float *chunk_states, const void *grad_out,
                            const float *grad_final, void *dx, void *da, void *db, float *dA_log, float *ddt_bias,
                            float *dinitial_state, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d, cu_seqlens != nullptr);
    if (rc != GDN_OK) return rc;
    const bool tok = (int64_t)d->B * d->T > 0;   // token tensors may be empty (null)
    if ((tok && (!x || !a || !b || !grad_out || !dx || !da || !db)) || !A_log || !dt_bias || !dA_log || !ddt_bias)
        return GDN_ERR_INVALID_ARG;
    const void *acts[] = {x, a, b, grad_out, dx, da, db};
    for (const void *q : acts)
        if (!act_aligned(d->dtype, q)) return GDN_ERR_INVALID_ARG;
    const void *words[] = {A_log, dt_bias, cu_seqlens, initial_state, chunk_states, grad_final, dA_log, ddt_bias, dinitial_state};
    for (const void *q : words)
        if (!ptr_aligned(q, 4)) return GDN_ERR_INVALID_ARG;
    const RecLayout L = bwd_layout(*d);
    if ((rc = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return rc;
    char *w = (char *)workspace;
    RecProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.a = a;
    p.b = b;
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.cu = cu_seqlens;
    p.h0 = initial_state;
    p.cs = chunk_states ? const_cast<float *>(chunk_states) : (float *)(w + L.cs);
    p.status = (int32_t *)workspace;
    p.part = (float *)(w + L.part);
    p.grad_out = grad_out;
    p.grad_final = grad_final;
    p.dx = dx;
    p.da = da;
    p.db = db;
    p.dA_log = dA_log;
    p.ddt_bias = ddt_bias;
    p.dh0 = dinitial_state;
    const cudaStream_t s = (cudaStream_t)stream;
    return by_dtype(d->dtype, [&](auto t) {
        using T = decltype(t);
        const dim3 grid((d->D + 127) / 128, d->N);
        if (!chunk_states) rec_forward_kernel<T><<<grid, 128, 0, s>>>(p);   // chunk states only
        rec_backward_kernel<T><<<grid, 128, 0, s>>>(p);
        rec_params_kernel<<<(d->D + 127) / 128, 128, 0, s>>>(p, d->N);
        return layer_status(cudaGetLastError());
    });
}

int gdn_recurrence_step(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b, const float *A_log,
                        const float *dt_bias, float *state, void *out, gdn_stream_t stream) {
    int rc = check_desc(d, false);
    if (rc != GDN_OK) return rc;
    if (d->T != 1) return GDN_ERR_INVALID_ARG;
    if (!x || !a || !b || !A_log || !dt_bias || !state || !out) return GDN_ERR_INVALID_ARG;
    if (!act_aligned(d->dtype, x) || !act_aligned(d->dtype, a) || !act_aligned(d->dtype, b) ||
        !act_aligned(d->dtype, out) || !ptr_aligned(A_log, 4) || !ptr_aligned(dt_bias, 4) || !ptr_aligned(state, 4))
        return GDN_ERR_INVALID_ARG;
    RecProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.a = a;
    p.b = b;
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.out = out;
    return by_dtype(d->dtype, [&](auto t) {
        rec_step_kernel<decltype(t)><<<dim3((d->D + 127) / 128, d->B), 128, 0, (cudaStream_t)stream>>>(p, state);
        return layer_status(cudaGetLastError());
    });
}

}  // extern "C"
