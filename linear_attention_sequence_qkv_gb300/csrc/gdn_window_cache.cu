// gdn_window_cache.cu -- the window attention's cache of fixed size (include/gdn.h): its
// filling, and one token per sequence over it.
#include <string.h>

#include <algorithm>

#include "gdn_window.cuh"

namespace gdn {

int window_check_desc(const gdn_window_attention_desc *d, bool packed);   // gdn_window_attention.cu

namespace {

struct CacheProblem {
    gdn_window_attention_desc d;
    const void *q, *k, *v;
    const int32_t *cu, *lengths;
    void *kc, *vc, *out;
    int32_t *status;
};

// The slot that holds a position
__device__ __forceinline__ int64_t slot_of(int64_t position, int sinks, int slots) {
    return position < sinks ? position : sinks + (position - sinks) % (slots - sinks);
}

// A thread copies single elements of the tokens that stay
template <typename T>
__global__ void __launch_bounds__(256) cache_write_kernel(const __grid_constant__ CacheProblem p) {
    const gdn_window_attention_desc &d = p.d;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.Tk);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int64_t per = (int64_t)d.Hk * d.d, total = (int64_t)d.B * d.Tk * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t tok = i / per, c = i - tok * per;
        const int n = p.cu ? upper_index(p.cu, d.N, tok) : (int)(tok / d.Tk);
        const int64_t at = tok - (p.cu ? p.cu[n] : (int64_t)n * d.Tk), count = p.cu ? p.cu[n + 1] - p.cu[n] : d.Tk;
        if (p.lengths[n] < 0) continue;
        const int64_t pos = p.lengths[n] + at;
        if (pos >= d.sinks && at < count - (d.slots - d.sinks)) continue;   // a later token of this call takes its slot
        const int64_t h = c / d.d, to = ((n * (int64_t)d.Hk + h) * d.slots + slot_of(pos, d.sinks, d.slots)) * d.d + (c - h * d.d);
        const int64_t row = p.cu ? 0 : n;
        ((T *)p.kc)[to] = ((const T *)p.k)[row * d.k_stride_b + (p.cu ? tok : at) * d.k_stride_t + c];
        ((T *)p.vc)[to] = ((const T *)p.v)[row * d.v_stride_b + (p.cu ? tok : at) * d.v_stride_t + c];
    }
}

constexpr int kStepWarps = 4;

// A CTA takes one sequence and head of keys, a warp one head of queries at a time
template <typename T, int NC>
__global__ void __launch_bounds__(32 * kStepWarps) step_rows(const __grid_constant__ CacheProblem p) {
    const gdn_window_attention_desc &d = p.d;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = GDN_OK;
    const int n = blockIdx.x, hk = blockIdx.y, lane = threadIdx.x & 31, group = d.Hq / d.Hk;
    T *out = (T *)p.out + ((int64_t)n * d.Hq + (int64_t)hk * group) * d.d;
    const int64_t pos = p.lengths[n];
    if (pos < 0) {
        for (int i = threadIdx.x; i < group * d.d; i += blockDim.x) out[i] = from_f<T>(0.0f);
        return;
    }
    T *kc = (T *)p.kc + ((int64_t)n * d.Hk + hk) * d.slots * d.d, *vc = (T *)p.vc + ((int64_t)n * d.Hk + hk) * d.slots * d.d;
    const T *kn = (const T *)p.k + n * d.k_stride_b + (int64_t)hk * d.d, *vn = (const T *)p.v + n * d.v_stride_b + (int64_t)hk * d.d;
    const int64_t here = slot_of(pos, d.sinks, d.slots);
    for (int c = threadIdx.x; c < d.d; c += blockDim.x) {
        kc[here * d.d + c] = kn[c];
        vc[here * d.d + c] = vn[c];
    }
    __syncthreads();
    // the keys seen: sinks before the window, then the window's
    const int64_t lo = pos >= d.window ? pos - d.window + 1 : 0, first = min((int64_t)d.sinks, lo), total = first + pos - lo + 1;
    for (int g = threadIdx.x >> 5; g < group; g += kStepWarps) {
        float qr[NC], o[NC], m = -INFINITY, l = 0.0f;
        row_load<T, NC>((const T *)p.q + n * d.q_stride_b + ((int64_t)hk * group + g) * d.d, d.d, lane, qr);
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c] = 0.0f;
        for (int64_t t0 = 0; t0 < total; t0 += 32) {
            const int cnt = (int)min((int64_t)32, total - t0);
            const int64_t t = t0 + lane, j = t < first ? t : min(lo + t - first, pos), sl = slot_of(j, d.sinks, d.slots);
            const float s = row_dot<T, NC>(qr, kc + sl * d.d, d.d) * d.scale, x = lane < cnt ? s : -INFINITY;
            const float mn = fmaxf(m, warp_max(x)), mm = mn == -INFINITY ? 0.0f : mn;
            const float corr = expf(m - mm), w = lane < cnt ? expf(x - mm) : 0.0f;
            l = l * corr + warp_sum(w);
#pragma unroll
            for (int c = 0; c < NC; ++c) o[c] *= corr;
            rows_add<T, NC>(o, w, vc + sl * d.d, cnt, d.d, lane);
            m = mn;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c] /= l;
        row_store<T, NC>(out + (int64_t)g * d.d, d.d, lane, o);
    }
}

template <typename T>
cudaError_t launch_step(const CacheProblem &p, cudaStream_t s) {
    const dim3 grid((unsigned)p.d.B, (unsigned)p.d.Hk);
    if (p.d.d <= 64) step_rows<T, 2><<<grid, 32 * kStepWarps, 0, s>>>(p);
    else if (p.d.d <= 128) step_rows<T, 4><<<grid, 32 * kStepWarps, 0, s>>>(p);
    else step_rows<T, 8><<<grid, 32 * kStepWarps, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_write(const CacheProblem &p, cudaStream_t s) {
    const int64_t total = (int64_t)p.d.B * p.d.Tk * p.d.Hk * p.d.d;
    const int64_t blocks = std::min<int64_t>(std::max<int64_t>(cdiv64(total, 256), 1), 64 * kSms);
    cache_write_kernel<T><<<(unsigned)blocks, 256, 0, s>>>(p);
    return cudaGetLastError();
}

int check_cache(const gdn_window_attention_desc *d, bool packed) {
    const int rc = window_check_desc(d, packed);
    if (rc != GDN_OK) return rc;
    if (d->slots < (int64_t)d->sinks + d->window) return GDN_ERR_INVALID_ARG;
    if (d->Hk > 65535) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int bytes_of(const gdn_window_attention_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_cache(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_window_attention_step_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes) { return bytes_of(d, bytes); }
int gdn_window_cache_write_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes) { return bytes_of(d, bytes); }

int gdn_window_cache_write(const gdn_window_attention_desc *d, const void *k, const void *v, const int32_t *cu_seqlens,
                           const int32_t *lengths, void *k_cache, void *v_cache, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream) {
    int rc = check_cache(d, cu_seqlens != nullptr);
    if (rc != GDN_OK) return rc;
    if ((int64_t)d->B * d->Tk > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;   // no tokens: these may be null
    if (!lengths || !k_cache || !v_cache) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(k, es) || !ptr_aligned(v, es) || !ptr_aligned(k_cache, es) || !ptr_aligned(v_cache, es) ||
        !ptr_aligned(lengths, 4) || !ptr_aligned(cu_seqlens, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    CacheProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.k = k, p.v = v, p.cu = cu_seqlens, p.lengths = lengths;
    p.kc = k_cache, p.vc = v_cache;
    p.status = (int32_t *)workspace;
    const cudaStream_t s = (cudaStream_t)stream;
    return layer_status(act_size(d->dtype) == 4 ? launch_write<uint32_t>(p, s) : launch_write<uint16_t>(p, s));
}

int gdn_window_attention_step(const gdn_window_attention_desc *d, const void *q, const void *k, const void *v, const int32_t *lengths,
                              void *k_cache, void *v_cache, void *out, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_cache(d, false);
    if (rc != GDN_OK) return rc;
    if (d->Tq != 1 || d->Tk != 1) return GDN_ERR_INVALID_ARG;
    if (!q || !k || !v || !lengths || !k_cache || !v_cache || !out) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(q, es) || !ptr_aligned(k, es) || !ptr_aligned(v, es) || !ptr_aligned(k_cache, es) || !ptr_aligned(v_cache, es) ||
        !ptr_aligned(out, es) || !ptr_aligned(lengths, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    CacheProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.q = q, p.k = k, p.v = v, p.lengths = lengths;
    p.kc = k_cache, p.vc = v_cache, p.out = out;
    p.status = (int32_t *)workspace;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d->dtype) {
    case GDN_F32: return layer_status(launch_step<float>(p, s));
    case GDN_BF16: return layer_status(launch_step<__nv_bfloat16>(p, s));
    default: return layer_status(launch_step<__half>(p, s));
    }
}

}  // extern "C"
