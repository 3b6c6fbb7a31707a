// gdn_group_norm.cu -- group norm with an activation, channels last (include/gdn.h):
// forward and backward.
#include <string.h>

#include "gdn_layer_ops.cuh"

namespace gdn {
namespace {

struct NormProblem {
    gdn_group_norm_desc d;
    const void *x, *w, *b, *dy;
    void *out, *dx;
    float *mean, *rstd, *dw, *db;
};

__device__ __forceinline__ float block_sum(float v) {
    __shared__ float red[8];
    __syncthreads();
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < 8; ++i) s += red[i];
    return s;
}

__device__ __forceinline__ float param(const void *p, int dtype, int c, float none) {
    if (!p) return none;
    return dtype == GDN_F32 ? ((const float *)p)[c]
           : dtype == GDN_BF16 ? __bfloat162float(((const __nv_bfloat16 *)p)[c]) : __half2float(((const __half *)p)[c]);
}

__device__ __forceinline__ float act_grad(float z, int act) {   // d act(z) / dz
    if (act == GDN_ACT_NONE) return 1.f;
    const float s = 1.f / (1.f + __expf(-z));
    return s * (1.f + z * (1.f - s));
}

// One block of 256 threads per (instance, group).
template <typename T>
__global__ void __launch_bounds__(256) norm_forward_kernel(const NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const int64_t n = blockIdx.x / d.G;
    const int g = blockIdx.x % d.G, cg = d.C / d.G;
    const int64_t count = (int64_t)d.L * cg;
    const T *x = (const T *)p.x + n * d.x_stride_n + (int64_t)g * cg;
    float s = 0.f;
    for (int64_t i = threadIdx.x; i < count; i += 256) s += to_f<T>(x[i / cg * d.x_stride_l + i % cg]);
    const float mean = block_sum(s) / (float)count;
    s = 0.f;
    for (int64_t i = threadIdx.x; i < count; i += 256) {
        const float v = to_f<T>(x[i / cg * d.x_stride_l + i % cg]) - mean;
        s += v * v;
    }
    const float rstd = rsqrtf(block_sum(s) / (float)count + d.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[blockIdx.x] = mean;
        if (p.rstd) p.rstd[blockIdx.x] = rstd;
    }
    for (int64_t i = threadIdx.x; i < count; i += 256) {
        const int c = g * cg + (int)(i % cg);
        const float z = (to_f<T>(x[i / cg * d.x_stride_l + i % cg]) - mean) * rstd * param(p.w, d.weight_dtype, c, 1.f) +
                        param(p.b, d.weight_dtype, c, 0.f);
        ((T *)p.out)[(n * d.L + i / cg) * d.C + c] = from_f<T>(d.act == GDN_ACT_SILU ? silu_f(z) : z);
    }
}

template <typename T>
__global__ void __launch_bounds__(256) norm_dx_kernel(const NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const int64_t n = blockIdx.x / d.G;
    const int g = blockIdx.x % d.G, cg = d.C / d.G;
    const int64_t count = (int64_t)d.L * cg;
    const T *x = (const T *)p.x + n * d.x_stride_n + (int64_t)g * cg;
    const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x];
    float s1 = 0.f, s2 = 0.f, m1 = 0.f, m2 = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t i = threadIdx.x; i < count; i += 256) {
            const int c = g * cg + (int)(i % cg);
            const int64_t o = (n * d.L + i / cg) * d.C + c;
            const float xh = (to_f<T>(x[i / cg * d.x_stride_l + i % cg]) - mean) * rstd;
            const float w = param(p.w, d.weight_dtype, c, 1.f);
            const float z = xh * w + param(p.b, d.weight_dtype, c, 0.f);
            const float t = to_f<T>(((const T *)p.dy)[o]) * act_grad(z, d.act) * w;
            if (pass == 0) {
                s1 += t;
                s2 += t * xh;
            } else {
                ((T *)p.dx)[o] = from_f<T>(rstd * (t - m1 - xh * m2));
            }
        }
        if (pass == 0) {
            m1 = block_sum(s1) / (float)count;
            m2 = block_sum(s2) / (float)count;
        }
    }
}

// One thread per channel.
template <typename T>
__global__ void __launch_bounds__(256) norm_params_kernel(const NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d.C) return;
    const int g = c / (d.C / d.G);
    const float w = param(p.w, d.weight_dtype, c, 1.f), b = param(p.b, d.weight_dtype, c, 0.f);
    float sw = 0.f, sb = 0.f;
    for (int64_t n = 0; n < d.N; ++n)
        for (int64_t l = 0; l < d.L; ++l) {
            const float xh = (to_f<T>(((const T *)p.x)[n * d.x_stride_n + l * d.x_stride_l + c]) - p.mean[n * d.G + g]) *
                             p.rstd[n * d.G + g];
            const float dz = to_f<T>(((const T *)p.dy)[(n * d.L + l) * d.C + c]) * act_grad(xh * w + b, d.act);
            sw += dz * xh;
            sb += dz;
        }
    if (p.dw) p.dw[c] = sw;
    if (p.db) p.db[c] = sb;
}

int check_desc(const gdn_group_norm_desc *d) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->N < 0 || d->L < 0 || d->C < 1 || d->G < 1 || d->C % d->G != 0) return GDN_ERR_INVALID_ARG;
    if (d->act != GDN_ACT_NONE && d->act != GDN_ACT_SILU) return GDN_ERR_UNSUPPORTED;
    if (!dtype_ok(d->dtype) || (d->weight_dtype != d->dtype && d->weight_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f) || d->x_stride_n < 0 || d->x_stride_l < 0) return GDN_ERR_INVALID_ARG;
    if (d->L > 1 && d->x_stride_l < d->C) return GDN_ERR_INVALID_ARG;
    if ((double)d->N * d->L * d->C > 4.0e12 || (int64_t)d->N * d->G > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int check_tensors(const gdn_group_norm_desc &d, const void *w, const void *b) {
    return ptr_aligned(w, act_size(d.weight_dtype)) && ptr_aligned(b, act_size(d.weight_dtype)) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_group_norm_desc_init(gdn_group_norm_desc *d, int N, int L, int C, int G, int dtype) {
    if (!d) return GDN_ERR_INVALID_ARG;
    memset(d, 0, sizeof(*d));
    d->N = N;
    d->L = L;
    d->C = C;
    d->G = G;
    d->dtype = d->weight_dtype = dtype;
    d->act = GDN_ACT_SILU;
    d->eps = 1e-5f;
    d->x_stride_l = C;
    d->x_stride_n = (int64_t)C * L;
    return check_desc(d);
}

int gdn_group_norm_workspace_bytes(const gdn_group_norm_desc *d, size_t *bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

int gdn_group_norm_backward_workspace_bytes(const gdn_group_norm_desc *d, size_t *bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

int gdn_group_norm_forward(const gdn_group_norm_desc *d, const void *x, const void *weight, const void *bias, void *out,
                           float *mean, float *rstd, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    const bool any = (int64_t)d->N * d->L > 0;
    if (any && (!x || !out)) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(x, es) || !ptr_aligned(out, es) || !ptr_aligned(mean, 4) || !ptr_aligned(rstd, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_tensors(*d, weight, bias)) != GDN_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    if (!any) return GDN_OK;
    NormProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.w = weight;
    p.b = bias;
    p.out = out;
    p.mean = mean;
    p.rstd = rstd;
    const unsigned grid = (unsigned)d->N * d->G;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d->dtype) {
    case GDN_F32: norm_forward_kernel<float><<<grid, 256, 0, s>>>(p); break;
    case GDN_BF16: norm_forward_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p); break;
    default: norm_forward_kernel<__half><<<grid, 256, 0, s>>>(p); break;
    }
    return layer_status(cudaGetLastError());
}

int gdn_group_norm_backward(const gdn_group_norm_desc *d, const void *x, const void *weight, const void *bias,
                            const float *mean, const float *rstd, const void *grad_out, void *dx, float *dweight,
                            float *dbias, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    const bool any = (int64_t)d->N * d->L > 0;
    if (any && (!x || !mean || !rstd || !grad_out || !dx)) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(x, es) || !ptr_aligned(grad_out, es) || !ptr_aligned(dx, es) || !ptr_aligned(mean, 4) ||
        !ptr_aligned(rstd, 4) || !ptr_aligned(dweight, 4) || !ptr_aligned(dbias, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_tensors(*d, weight, bias)) != GDN_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    NormProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.w = weight;
    p.b = bias;
    p.mean = const_cast<float *>(mean);
    p.rstd = const_cast<float *>(rstd);
    p.dy = grad_out;
    p.dx = dx;
    p.dw = dweight;
    p.db = dbias;
    const unsigned grid = (unsigned)d->N * d->G, gc = (d->C + 255) / 256;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d->dtype) {
    case GDN_F32:
        if (any) norm_dx_kernel<float><<<grid, 256, 0, s>>>(p);
        norm_params_kernel<float><<<gc, 256, 0, s>>>(p);
        break;
    case GDN_BF16:
        if (any) norm_dx_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
        norm_params_kernel<__nv_bfloat16><<<gc, 256, 0, s>>>(p);
        break;
    default:
        if (any) norm_dx_kernel<__half><<<grid, 256, 0, s>>>(p);
        norm_params_kernel<__half><<<gc, 256, 0, s>>>(p);
        break;
    }
    return layer_status(cudaGetLastError());
}

}  // extern "C"
