// gdn_norm_rotary.cu -- the norm of every head of q and k with the rotary positions in the
// same pass (include/gdn.h), forward and backward.
//
// A warp takes one head of one token at a time: its channels go through shared memory as
// fp32, the sum of squares over the lanes, and every pair is normalised, weighted and turned
// from there.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "gdn_layer_ops.cuh"
#include "gdn_rotary.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kMostChannels = 1024;   // of a head: a warp keeps four rows of them in shared memory
constexpr int kBwdCtas = 4 * kSms;    // CTAs of the backward, each with a row of partial weight gradients

struct NormRotaryProblem {
    gdn_norm_rotary_desc n;
    const void *q, *k, *qw, *kw;
    const uint64_t *turns;
    const int32_t *pos, *cu, *off;
    void *qo, *ko;                    // forward: written; backward: the incoming gradients
    void *dq, *dk;
    float *dqw, *dkw, *part;          // part: [CTAs][2][d]
    int32_t *status;
    int ctas;
};

__device__ __forceinline__ float weight_at(const void *w, int dtype, int c) {
    if (!w) return 1.0f;
    if (dtype == GDN_F32) return ((const float *)w)[c];
    return dtype == GDN_BF16 ? __bfloat162float(((const __nv_bfloat16 *)w)[c]) : __half2float(((const __half *)w)[c]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A head of a token: offsets of its channels in the input, the output (or its gradient) and a dense gradient
struct HeadAt {
    bool isk;
    int row, t;
    int64_t in, out, dense;
};
__device__ __forceinline__ HeadAt head_at(const gdn_rotary_desc &d, int64_t i) {
    const int heads = d.Hq + d.Hk;
    const int64_t tok = i / heads;
    int h = (int)(i - tok * heads);
    HeadAt a;
    a.isk = h >= d.Hq;
    if (a.isk) h -= d.Hq;
    a.row = (int)(tok / d.T);
    a.t = (int)(tok - (int64_t)a.row * d.T);
    a.in = a.row * (a.isk ? d.k_stride_b : d.q_stride_b) + a.t * (a.isk ? d.k_stride_t : d.q_stride_t) + (int64_t)h * d.d;
    a.out = a.row * (a.isk ? d.k_out_stride_b : d.q_out_stride_b) + a.t * (a.isk ? d.k_out_stride_t : d.q_out_stride_t) +
            (int64_t)h * d.d;
    a.dense = (tok * (a.isk ? d.Hk : d.Hq) + h) * d.d;
    return a;
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) norm_rotary_rows(const __grid_constant__ NormRotaryProblem p) {
    extern __shared__ float sm[];
    const gdn_rotary_desc &d = p.n.rotary;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = d.rot / 2;
    float *x = sm + warp * d.d;
    const int64_t total = (int64_t)d.B * d.T * (d.Hq + d.Hk);
    for (int64_t i = (int64_t)blockIdx.x * kWarps + warp; i < total; i += (int64_t)gridDim.x * kWarps) {
        const HeadAt a = head_at(d, i);
        const T *src = (const T *)(a.isk ? p.k : p.q) + a.in;
        T *dst = (T *)(a.isk ? p.ko : p.qo) + a.out;
        const void *w = a.isk ? p.kw : p.qw;
        float ss = 0.0f;
        for (int c = lane; c < d.d; c += 32) {
            x[c] = to_f<T>(src[c]);
            ss += x[c] * x[c];
        }
        const float rstd = rsqrtf(warp_sum(ss) / d.d + p.n.eps);
        __syncwarp();
        const int64_t at = rotary_position(d, p.pos, p.cu, p.off, a.row, a.t);
        for (int j = lane; j < half; j += 32) {
            const float2 cs = cos_sin<sizeof(T) == 2>(at, p.turns[j]);
            const int c1 = d.layout == GDN_ROTARY_HALF ? j : 2 * j, c2 = d.layout == GDN_ROTARY_HALF ? j + half : 2 * j + 1;
            const float z1 = x[c1] * rstd * weight_at(w, p.n.weight_dtype, c1), z2 = x[c2] * rstd * weight_at(w, p.n.weight_dtype, c2);
            dst[c1] = from_f<T>(d.scale * (z1 * cs.x - z2 * cs.y));
            dst[c2] = from_f<T>(d.scale * (z2 * cs.x + z1 * cs.y));
        }
        for (int c = d.rot + lane; c < d.d; c += 32) dst[c] = from_f<T>(x[c] * rstd * weight_at(w, p.n.weight_dtype, c));
        __syncwarp();
    }
}

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) norm_rotary_rows_backward(const __grid_constant__ NormRotaryProblem p) {
    extern __shared__ float sm[];
    const gdn_rotary_desc &d = p.n.rotary;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = d.rot / 2;
    float *x = sm + warp * 2 * d.d, *dz = x + d.d, *acc = sm + kWarps * 2 * d.d;   // acc: [warp][2][d]
    for (int c = threadIdx.x; c < kWarps * 2 * d.d; c += 32 * kWarps) acc[c] = 0.0f;
    __syncthreads();
    const int64_t total = (int64_t)d.B * d.T * (d.Hq + d.Hk);
    for (int64_t i = (int64_t)blockIdx.x * kWarps + warp; i < total; i += (int64_t)gridDim.x * kWarps) {
        const HeadAt a = head_at(d, i);
        const T *src = (const T *)(a.isk ? p.k : p.q) + a.in;
        const T *g = (const T *)(a.isk ? p.ko : p.qo) + a.out;
        T *dst = (T *)(a.isk ? p.dk : p.dq) + a.dense;
        const void *w = a.isk ? p.kw : p.qw;
        float ss = 0.0f, st = 0.0f;
        for (int c = lane; c < d.d; c += 32) {
            x[c] = to_f<T>(src[c]);
            ss += x[c] * x[c];
        }
        const float rstd = rsqrtf(warp_sum(ss) / d.d + p.n.eps);
        const int64_t at = rotary_position(d, p.pos, p.cu, p.off, a.row, a.t);
        for (int j = lane; j < half; j += 32) {
            const float2 cs = cos_sin<sizeof(T) == 2>(at, p.turns[j]);
            const int c1 = d.layout == GDN_ROTARY_HALF ? j : 2 * j, c2 = d.layout == GDN_ROTARY_HALF ? j + half : 2 * j + 1;
            const float g1 = to_f<T>(g[c1]), g2 = to_f<T>(g[c2]);
            dz[c1] = d.scale * (g1 * cs.x + g2 * cs.y);
            dz[c2] = d.scale * (g2 * cs.x - g1 * cs.y);
        }
        for (int c = d.rot + lane; c < d.d; c += 32) dz[c] = to_f<T>(g[c]);
        __syncwarp();
        for (int c = lane; c < d.d; c += 32) st += dz[c] * weight_at(w, p.n.weight_dtype, c) * x[c];
        const float mean = rstd * warp_sum(st) / d.d;   // of t xh
        for (int c = lane; c < d.d; c += 32) {
            const float xh = x[c] * rstd;
            acc[(warp * 2 + a.isk) * d.d + c] += dz[c] * xh;
            dst[c] = from_f<T>(rstd * (dz[c] * weight_at(w, p.n.weight_dtype, c) - xh * mean));
        }
        __syncwarp();
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * d.d; c += 32 * kWarps) {
        float s = 0.0f;
        for (int w = 0; w < kWarps; ++w) s += acc[w * 2 * d.d + c];
        p.part[(int64_t)blockIdx.x * 2 * d.d + c] = s;
    }
}

// The sum of the CTAs' partial weight gradients: a warp per channel.
__global__ void __launch_bounds__(256) norm_rotary_weights(const __grid_constant__ NormRotaryProblem p) {
    if (*p.status != GDN_OK) return;
    const int d = p.n.rotary.d, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (c >= 2 * d) return;
    float s = 0.0f;
    for (int i = lane; i < p.ctas; i += 32) s += p.part[(int64_t)i * 2 * d + c];
    s = warp_sum(s);
    float *to = c < d ? p.dqw : p.dkw;
    if (lane == 0 && to) to[c < d ? c : c - d] = s;
}

int check_desc(const gdn_norm_rotary_desc *n, bool packed) {
    if (!n) return GDN_ERR_INVALID_ARG;
    const int rc = rotary_check_desc(&n->rotary, packed);
    if (rc != GDN_OK) return rc;
    if (n->rotary.inverse != 0 || !(n->eps >= 0.0f) || !isfinite(n->eps) || !isfinite(n->rotary.scale)) return GDN_ERR_INVALID_ARG;
    if (n->weight_dtype != n->rotary.dtype && n->weight_dtype != GDN_F32) return GDN_ERR_UNSUPPORTED;
    if (n->rotary.d > kMostChannels) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int64_t heads_of(const gdn_rotary_desc &d) { return (int64_t)d.B * d.T * (d.Hq + d.Hk); }
int bwd_ctas(const gdn_rotary_desc &d) { return (int)std::min<int64_t>(std::max<int64_t>(cdiv64(heads_of(d), kWarps), 1), kBwdCtas); }
size_t bwd_bytes(const gdn_rotary_desc &d) { return kStatusBytes + (size_t)bwd_ctas(d) * 2 * d.d * 4; }

template <typename T>
cudaError_t launch_forward(const NormRotaryProblem &p, cudaStream_t s) {
    const gdn_rotary_desc &d = p.n.rotary;
    const int64_t blocks = std::min<int64_t>(std::max<int64_t>(cdiv64(heads_of(d), kWarps), 1), 16 * kSms);
    norm_rotary_rows<T><<<(unsigned)blocks, 32 * kWarps, (size_t)kWarps * d.d * 4, s>>>(p);
    return cudaGetLastError();
}
template <typename T>
cudaError_t launch_backward_rows(const NormRotaryProblem &p, cudaStream_t s) {
    const gdn_rotary_desc &d = p.n.rotary;
    const size_t smem = (size_t)kWarps * 4 * d.d * 4;
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_shared(norm_rotary_rows_backward<T>, (size_t)kWarps * 4 * kMostChannels * 4);
        if (e != cudaSuccess) return e;
    }
    norm_rotary_rows_backward<T><<<(unsigned)p.ctas, 32 * kWarps, smem, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!p.dqw && !p.dkw)) return e;
    norm_rotary_weights<<<(unsigned)cdiv64(2 * d.d, 8), 256, 0, s>>>(p);
    return cudaGetLastError();
}

// The checks that forward and backward share; on success p holds the inputs
int fill(NormRotaryProblem &p, const gdn_norm_rotary_desc *n, const void *q, const void *k, const void *qw, const void *kw,
         const uint64_t *turns, const int32_t *positions, const int32_t *cu, const int32_t *offsets, const void *qo,
         const void *ko, void *workspace, size_t workspace_bytes, bool backward) {
    int rc = check_desc(n, cu != nullptr);
    if (rc != GDN_OK) return rc;
    const gdn_rotary_desc &d = n->rotary;
    const bool tok = (int64_t)d.B * d.T > 0;   // token tensors may be empty (null)
    if (tok && (!q || !qo || (d.Hk && (!k || !ko)))) return GDN_ERR_INVALID_ARG;
    if (!turns || (positions && offsets)) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d.dtype), ws = act_size(n->weight_dtype);
    if (!ptr_aligned(q, es) || !ptr_aligned(k, es) || !ptr_aligned(qo, es) || !ptr_aligned(ko, es) || !ptr_aligned(qw, ws) ||
        !ptr_aligned(kw, ws) || !ptr_aligned(turns, 8) || !ptr_aligned(positions, 4) || !ptr_aligned(cu, 4) || !ptr_aligned(offsets, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, backward ? bwd_bytes(d) : kStatusBytes)) != GDN_OK) return rc;
    memset(&p, 0, sizeof(p));
    p.n = *n;
    p.q = q, p.k = k, p.qw = qw, p.kw = kw;
    p.turns = turns;
    p.pos = positions, p.cu = cu, p.off = offsets;
    p.qo = const_cast<void *>(qo), p.ko = const_cast<void *>(ko);
    p.status = (int32_t *)workspace;
    p.part = (float *)((char *)workspace + kStatusBytes);
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_norm_rotary_desc_init(gdn_norm_rotary_desc *n, int B, int T, int packed, int Hq, int Hk, int head_dim, int dtype) {
    if (!n) return GDN_ERR_INVALID_ARG;
    memset(n, 0, sizeof(*n));
    const int rc = gdn_rotary_desc_init(&n->rotary, B, T, packed, Hq, Hk, head_dim, dtype);
    n->weight_dtype = dtype;
    n->eps = 1e-6f;
    return rc != GDN_OK ? rc : check_desc(n, packed != 0);
}

int gdn_norm_rotary_workspace_bytes(const gdn_norm_rotary_desc *n, size_t *bytes) {
    if (!n || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(n, n->rotary.N != n->rotary.B);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

int gdn_norm_rotary_backward_workspace_bytes(const gdn_norm_rotary_desc *n, size_t *bytes) {
    if (!n || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(n, n->rotary.N != n->rotary.B);
    if (rc != GDN_OK) return rc;
    *bytes = bwd_bytes(n->rotary);
    return GDN_OK;
}

int gdn_norm_rotary_forward(const gdn_norm_rotary_desc *n, const void *q, const void *k, const void *q_weight,
                            const void *k_weight, const uint64_t *turns, const int32_t *positions, const int32_t *cu_seqlens,
                            const int32_t *offsets, void *q_out, void *k_out, void *workspace, size_t workspace_bytes,
                            gdn_stream_t stream) {
    NormRotaryProblem p;
    const int rc = fill(p, n, q, k, q_weight, k_weight, turns, positions, cu_seqlens, offsets, q_out, k_out, workspace,
                        workspace_bytes, false);
    if (rc != GDN_OK) return rc;
    const gdn_rotary_desc &d = n->rotary;
    // in place means the same elements
    if ((q && q == q_out && (d.q_stride_b != d.q_out_stride_b || d.q_stride_t != d.q_out_stride_t)) ||
        (k && k == k_out && (d.k_stride_b != d.k_out_stride_b || d.k_stride_t != d.k_out_stride_t)))
        return GDN_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d.dtype) {
    case GDN_F32: return layer_status(launch_forward<float>(p, s));
    case GDN_BF16: return layer_status(launch_forward<__nv_bfloat16>(p, s));
    default: return layer_status(launch_forward<__half>(p, s));
    }
}

int gdn_norm_rotary_backward(const gdn_norm_rotary_desc *n, const void *q, const void *k, const void *q_weight,
                             const void *k_weight, const uint64_t *turns, const int32_t *positions, const int32_t *cu_seqlens,
                             const int32_t *offsets, const void *grad_q, const void *grad_k, void *dq, void *dk,
                             float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    NormRotaryProblem p;
    const int rc = fill(p, n, q, k, q_weight, k_weight, turns, positions, cu_seqlens, offsets, grad_q, grad_k, workspace,
                        workspace_bytes, true);
    if (rc != GDN_OK) return rc;
    const gdn_rotary_desc &d = n->rotary;
    const size_t es = act_size(d.dtype);
    if ((int64_t)d.B * d.T > 0 && (!dq || (d.Hk && !dk))) return GDN_ERR_INVALID_ARG;
    if (!ptr_aligned(dq, es) || !ptr_aligned(dk, es) || !ptr_aligned(dq_weight, 4) || !ptr_aligned(dk_weight, 4))
        return GDN_ERR_INVALID_ARG;
    p.dq = dq, p.dk = dk, p.dqw = dq_weight, p.dkw = dk_weight;
    p.ctas = bwd_ctas(d);
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d.dtype) {
    case GDN_F32: return layer_status(launch_backward_rows<float>(p, s));
    case GDN_BF16: return layer_status(launch_backward_rows<__nv_bfloat16>(p, s));
    default: return layer_status(launch_backward_rows<__half>(p, s));
    }
}

}  // extern "C"
