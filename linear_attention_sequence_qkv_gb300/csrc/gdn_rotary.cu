// gdn_rotary.cu -- rotary positions (include/gdn.h): the table of turns on the host
// and the rotation of q and k.
#include <math.h>
#include <string.h>

#include "gdn_layer_ops.cuh"

namespace gdn {
namespace {

struct RotaryProblem {
    gdn_rotary_desc d;
    const void *q, *k;
    const uint64_t *turns;
    const int32_t *pos, *cu, *off;
    void *qo, *ko;
    int32_t *status;
};

// Position of token t of row `row` (see gdn_rotary in include/gdn.h)
__device__ __forceinline__ int64_t token_position(const RotaryProblem &p, int row, int t) {
    const gdn_rotary_desc &d = p.d;
    if (p.pos) return p.pos[(int64_t)row * d.T + t];
    int n = row;
    int64_t at = t;
    if (p.cu) {
        n = upper_index(p.cu, d.N, t);
        at -= p.cu[n];
    }
    return at + (p.off ? p.off[n] : 0);
}

// cos and sin of 2 pi frac(position * turn / 2^64): the 64-bit product wraps at whole
// turns, and its upper half as a signed fraction has 32 bits of the remaining angle.
__device__ __forceinline__ float2 cos_sin(int64_t position, uint64_t turn) {
    const uint64_t phase = (uint64_t)position * turn;
    float c, s;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: in half turns
    return make_float2(c, s);
}

// One thread per pair or copied channel of a token.
template <typename T>
__global__ void __launch_bounds__(128) rotary_kernel(const RotaryProblem p) {
    const gdn_rotary_desc &d = p.d;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int half = d.rot / 2, units = half + d.d - d.rot, H = d.Hq + d.Hk;
    for (int64_t tok = blockIdx.x; tok < (int64_t)d.B * d.T; tok += gridDim.x) {
        const int row = (int)(tok / d.T), t = (int)(tok - (int64_t)row * d.T);
        const int64_t position = token_position(p, row, t);
        for (int i = threadIdx.x; i < H * units; i += 128) {
            const int h = i / units, u = i - h * units;
            const bool isk = h >= d.Hq;
            const T *src = (const T *)(isk ? p.k : p.q) + row * (isk ? d.k_stride_b : d.q_stride_b) +
                           t * (isk ? d.k_stride_t : d.q_stride_t) + (int64_t)(isk ? h - d.Hq : h) * d.d;
            T *dst = (T *)(isk ? p.ko : p.qo) + row * (isk ? d.k_out_stride_b : d.q_out_stride_b) +
                     t * (isk ? d.k_out_stride_t : d.q_out_stride_t) + (int64_t)(isk ? h - d.Hq : h) * d.d;
            if (u >= half) {
                dst[d.rot + u - half] = src[d.rot + u - half];
                continue;
            }
            float2 cs = cos_sin(position, p.turns[u]);
            cs.x *= d.scale;
            cs.y *= d.inverse ? -d.scale : d.scale;
            const int i1 = d.layout == GDN_ROTARY_HALF ? u : 2 * u, i2 = d.layout == GDN_ROTARY_HALF ? u + half : 2 * u + 1;
            const float x1 = to_f<T>(src[i1]), x2 = to_f<T>(src[i2]);
            dst[i1] = from_f<T>(x1 * cs.x - x2 * cs.y);
            dst[i2] = from_f<T>(x2 * cs.x + x1 * cs.y);
        }
    }
}

int check_desc(const gdn_rotary_desc *d, bool packed) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->N < 1 || d->Hq < 1 || d->Hk < 0 || d->d < 2) return GDN_ERR_INVALID_ARG;
    if (packed ? d->B != 1 : d->N != d->B) return GDN_ERR_INVALID_ARG;
    if (d->rot < 2 || d->rot > d->d || d->rot % 2) return GDN_ERR_INVALID_ARG;
    if (d->layout != GDN_ROTARY_HALF && d->layout != GDN_ROTARY_INTERLEAVED) return GDN_ERR_INVALID_ARG;
    if (d->inverse != 0 && d->inverse != 1) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)d->d * ((int64_t)d->Hq + d->Hk) > (1 << 30)) return GDN_ERR_UNSUPPORTED;
    const int64_t strides[] = {d->q_stride_b, d->q_stride_t, d->q_out_stride_b, d->q_out_stride_t,
                               d->k_stride_b, d->k_stride_t, d->k_out_stride_b, d->k_out_stride_t};
    for (int i = 0; i < (d->Hk ? 8 : 4); ++i)
        if (strides[i] < 0) return GDN_ERR_INVALID_ARG;
    const int64_t rq = (int64_t)d->Hq * d->d, rk = (int64_t)d->Hk * d->d;
    if (d->T > 1 && (d->q_stride_t < rq || d->q_out_stride_t < rq)) return GDN_ERR_INVALID_ARG;
    if (d->T > 1 && d->Hk && (d->k_stride_t < rk || d->k_out_stride_t < rk)) return GDN_ERR_INVALID_ARG;
    // outputs of different rows must be different places
    if (d->B > 1 && d->T > 0 && (d->q_out_stride_b < rq || (d->Hk && d->k_out_stride_b < rk))) return GDN_ERR_INVALID_ARG;
    if ((double)d->B * d->T * (rq + rk) > 4.0e12) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_rotary_desc_init(gdn_rotary_desc *d, int B, int T, int packed, int Hq, int Hk, int head_dim, int dtype) {
    if (!d) return GDN_ERR_INVALID_ARG;
    memset(d, 0, sizeof(*d));
    d->B = B;
    d->T = T;
    d->N = packed ? packed : B;
    d->Hq = Hq;
    d->Hk = Hk;
    d->d = head_dim;
    d->rot = head_dim & ~1;
    d->dtype = dtype;
    d->scale = 1.0f;
    d->q_stride_t = d->q_out_stride_t = (int64_t)Hq * head_dim;
    d->k_stride_t = d->k_out_stride_t = (int64_t)Hk * head_dim;
    d->q_stride_b = d->q_out_stride_b = d->q_stride_t * T;
    d->k_stride_b = d->k_out_stride_b = d->k_stride_t * T;
    return check_desc(d, packed != 0);
}

int gdn_rotary_table(int rot, double theta, int scaling, double factor, double low, double high, double original,
                     uint64_t *turns) {
    if (rot < 2 || rot % 2 || !(theta > 0.0) || !isfinite(theta) || !turns) return GDN_ERR_INVALID_ARG;
    if (scaling != GDN_ROTARY_PLAIN && scaling != GDN_ROTARY_LINEAR && scaling != GDN_ROTARY_BY_PARTS)
        return GDN_ERR_INVALID_ARG;
    if (scaling != GDN_ROTARY_PLAIN && (!(factor > 0.0) || !isfinite(factor))) return GDN_ERR_INVALID_ARG;
    if (scaling == GDN_ROTARY_BY_PARTS && (!(high > low) || !isfinite(high - low) || !(original > 0.0) || !isfinite(original)))
        return GDN_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925286766559;
    for (int i = 0; i < rot / 2; ++i) {
        double f = pow(theta, -2.0 * i / rot);
        if (scaling == GDN_ROTARY_LINEAR) f /= factor;
        if (scaling == GDN_ROTARY_BY_PARTS) {
            double keep = (original * f / two_pi - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = keep * f + (1.0 - keep) * f / factor;
        }
        const double t = f / two_pi;
        // whole turns drop out; 1 - 2^-53 is the largest fraction, so the product stays below 2^64
        turns[i] = (uint64_t)ldexp(t - floor(t), 64);
    }
    return GDN_OK;
}

int gdn_rotary_workspace_bytes(const gdn_rotary_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

int gdn_rotary(const gdn_rotary_desc *d, const void *q, const void *k, const uint64_t *turns, const int32_t *positions,
               const int32_t *cu_seqlens, const int32_t *offsets, void *q_out, void *k_out, void *workspace,
               size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d, cu_seqlens != nullptr);
    if (rc != GDN_OK) return rc;
    const bool tok = (int64_t)d->B * d->T > 0;   // token tensors may be empty (null)
    if (tok && (!q || !q_out || (d->Hk && (!k || !k_out)))) return GDN_ERR_INVALID_ARG;
    if (!turns || (positions && offsets)) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(q, es) || !ptr_aligned(k, es) || !ptr_aligned(q_out, es) || !ptr_aligned(k_out, es) ||
        !ptr_aligned(turns, 8) || !ptr_aligned(positions, 4) || !ptr_aligned(cu_seqlens, 4) || !ptr_aligned(offsets, 4))
        return GDN_ERR_INVALID_ARG;
    // in place means the same elements
    if ((q == q_out && (d->q_stride_b != d->q_out_stride_b || d->q_stride_t != d->q_out_stride_t)) ||
        (d->Hk && k == k_out && (d->k_stride_b != d->k_out_stride_b || d->k_stride_t != d->k_out_stride_t)))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    RotaryProblem p = {*d, q, k, turns, positions, cu_seqlens, offsets, q_out, k_out, (int32_t *)workspace};
    const int64_t ntok = (int64_t)d->B * d->T;
    const unsigned grid = (unsigned)(ntok < 1 ? 1 : ntok < 65536 ? ntok : 65536);
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d->dtype) {
    case GDN_F32: rotary_kernel<float><<<grid, 128, 0, s>>>(p); break;
    case GDN_BF16: rotary_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(p); break;
    default: rotary_kernel<__half><<<grid, 128, 0, s>>>(p); break;
    }
    return layer_status(cudaGetLastError());
}

}  // extern "C"
