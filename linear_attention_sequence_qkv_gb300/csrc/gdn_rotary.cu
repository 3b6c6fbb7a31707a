// gdn_rotary.cu -- rotary positions (include/gdn.h): the table of turns on the host
// and the rotation of q and k.
//
// A streaming kernel, bound by HBM: every channel is read and written once (in place,
// the channels behind the rotated ones are not touched at all). The angle depends on
// the token and the pair alone, so a CTA computes the cosines and sines of its few
// tokens once, into shared memory, for all heads. A unit of work is one vector per
// half of a rotated head (half layout), one vector of whole pairs (interleaved), or one
// copied vector; a thread has several in flight. 131072 tokens of 32 heads of 128 in bf16
// take 309 us (2.1 GB, 102 % of the copy rate; 330 us in 64 packed sequences, whose positions
// are looked up for every entry of the table). With few heads per token the table counts: one
// head of 64 for 64 x 60000 tokens takes 389 us, 37 % of it.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "gdn_layer_ops.cuh"
#include "gdn_rotary.cuh"

namespace gdn {
namespace {

struct RotaryProblem {
    gdn_rotary_desc d;
    const void *q, *k;
    const uint64_t *turns;
    const int32_t *pos, *cu, *off;
    void *qo, *ko;
    int32_t *status;
    int tokens;             // per CTA
    int u_rot;              // units of a head's rotated channels
    int u_q, u_k;           // units of q's and of k's rotated channels per token
    int c_q, c_k;           // units of their copied channels (0 in place)
    int u_copy, copy_bytes; // units of a head's copied channels, and their size
};

__device__ __forceinline__ int64_t token_position(const RotaryProblem &p, int row, int t) {
    return rotary_position(p.d, p.pos, p.cu, p.off, row, t);
}

template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };
template <typename T, int V> union Vec {
    typename Raw<V * sizeof(T)>::type raw;
    T e[V];
};

constexpr int kThreads = 256;
constexpr int kBatch = 2;              // units in flight per thread
constexpr int kBatches = 4;
constexpr int kTableBytes = 32768;     // cosines and sines of a CTA's tokens
constexpr int kMostRotated = 32768;    // channels of a head: one token's cosines and sines have to fit

// A head of a token, and the unit u of it, from the index r of a unit among a token's: units_q of them q's, per
// head `per`.
template <typename T> struct Head {
    const T *src;
    T *dst;
    int u;
};
template <typename T>
__device__ __forceinline__ Head<T> head_of(const RotaryProblem &p, uint32_t tok, int r, int units_q, int per) {
    const gdn_rotary_desc &d = p.d;
    const uint32_t row = tok / (uint32_t)d.T, t = tok - row * d.T;   // tok is below 2^31
    const bool isk = r >= units_q;
    if (isk) r -= units_q;
    const int h = r / per;
    Head<T> x;
    x.u = r - h * per;
    x.src = (const T *)(isk ? p.k : p.q) + row * (isk ? d.k_stride_b : d.q_stride_b) + t * (isk ? d.k_stride_t : d.q_stride_t) +
            (int64_t)h * d.d;
    x.dst = (T *)(isk ? p.ko : p.qo) + row * (isk ? d.k_out_stride_b : d.q_out_stride_b) +
            t * (isk ? d.k_out_stride_t : d.q_out_stride_t) + (int64_t)h * d.d;
    return x;
}

// The channels behind the rotated ones, in vectors of R
template <typename T, typename R>
__device__ __forceinline__ void copy_rest(const RotaryProblem &p, int64_t tok0, int nt) {
    constexpr int kB = 4;
    const int per = p.c_q + p.c_k, total = nt * per, step = kThreads * gridDim.y;
    for (int i0 = blockIdx.y * kThreads + threadIdx.x; i0 < total; i0 += kB * step) {
        R v[kB], *to[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int i = i0 + j * step;
            if (i >= total) continue;
            const int t = i / per;
            // without q's copies (q in place) the first of them are k's
            const Head<T> hd = head_of<T>(p, (uint32_t)(tok0 + t), i - t * per, p.c_q, p.u_copy);
            v[j] = ((const R *)(hd.src + p.d.rot))[hd.u];
            to[j] = (R *)(hd.dst + p.d.rot) + hd.u;
        }
#pragma unroll
        for (int j = 0; j < kB; ++j)
            if (i0 + j * step < total) *to[j] = v[j];
    }
}

// V: elements per vector. HALF: a unit is the vectors at u V and rot/2 + u V; else the V elements from u V (two
// single elements for V = 1).
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryProblem p) {
    constexpr int NP = HALF ? V : (V > 1 ? V / 2 : 1);   // pairs per unit
    constexpr int W = NP < 4 ? NP : 4;                   // floats per table entry
    constexpr int Q = NP / W;                            // entries of cosines (and of sines) per unit
    extern __shared__ __align__(16) float tab[];         // [token][2 Q][unit][W]
    const gdn_rotary_desc &d = p.d;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int64_t tok0 = (int64_t)blockIdx.x * p.tokens;
    const int nt = (int)min((int64_t)p.tokens, (int64_t)d.B * d.T - tok0);
    const int half = d.rot / 2;
    const int per = p.u_q + p.u_k;                        // units per token
    const int total = nt * per, step = kThreads * gridDim.y;
    const T *src[kBatch];
    T *dst[kBatch];
    const float *tb[kBatch];                              // the unit's table entries
    Vec<T, V> a[kBatch], b[kBatch];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * step;
            if (i >= total) continue;
            const int t = i / per;
            int r = i - t * per;
            const Head<T> hd = head_of<T>(p, (uint32_t)(tok0 + t), r, p.u_q, p.u_rot);
            const int off = HALF ? hd.u * V : hd.u * 2 * NP;
            src[j] = hd.src + off;
            dst[j] = hd.dst + off;
            tb[j] = tab + (t * 2 * Q * p.u_rot + hd.u) * W;
            a[j].raw = *(const decltype(a[j].raw) *)src[j];
            if (HALF || V == 1) b[j].raw = *(const decltype(b[j].raw) *)(src[j] + (HALF ? half : 1));
        }
    };
    int i0 = blockIdx.y * kThreads + threadIdx.x;
    fetch(i0);   // on their way while the table is computed
    auto position_of = [&](int t) {
        const uint32_t row = (uint32_t)(tok0 + t) / (uint32_t)d.T;
        return token_position(p, row, (int)((uint32_t)(tok0 + t) - row * d.T));
    };
    auto entry = [&](int t, int64_t position, int pr, uint64_t turn) {
        const float2 cs = cos_sin<sizeof(T) == 2>(position, turn);
        const int u = pr / NP, e = pr % NP;
        float *at = tab + ((t * 2 * Q + e / W) * p.u_rot + u) * W + e % W;
        at[0] = cs.x * d.scale;
        at[Q * p.u_rot * W] = cs.y * (d.inverse ? -d.scale : d.scale);
    };
    if (half <= kThreads && nt * half > 8 * kThreads) {
        // Long tables (few heads): a thread keeps its pair and steps over the tokens. 64 x 60000 tokens of one head
        // of 64: 389 us, 544 with the loop below, which is the faster one for short tables (131072 tokens of 32 heads
        // of 128: 308 against 314 us; 4096 of 12 heads of 256 with 64 rotated: 11.2 against 11.7 on the device).
        const int tstep = kThreads / half, t0 = threadIdx.x / half, pr = threadIdx.x - t0 * half;
        const uint64_t turn = p.turns[pr];
        for (int t = t0 < tstep ? t0 : nt; t < nt; t += tstep) entry(t, position_of(t), pr, turn);
    } else {
        for (int i = threadIdx.x; i < nt * half; i += kThreads) {
            const int t = i / half, pr = i - t * half;
            entry(t, position_of(t), pr, p.turns[pr]);
        }
    }
    __syncthreads();
    for (; i0 < total; i0 += kBatch * step, fetch(i0)) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (i0 + j * step >= total) continue;
            float c[NP], s[NP];
#pragma unroll
            for (int e = 0; e < NP; e += W) {
                const float *tc = tb[j] + e / W * p.u_rot * W, *ts = tc + Q * p.u_rot * W;
                if (W == 4) {
                    const float4 c4 = *(const float4 *)tc, s4 = *(const float4 *)ts;
                    c[e] = c4.x, c[e + 1 < NP ? e + 1 : e] = c4.y, c[e + 2 < NP ? e + 2 : e] = c4.z, c[e + 3 < NP ? e + 3 : e] = c4.w;
                    s[e] = s4.x, s[e + 1 < NP ? e + 1 : e] = s4.y, s[e + 2 < NP ? e + 2 : e] = s4.z, s[e + 3 < NP ? e + 3 : e] = s4.w;
                } else {
#pragma unroll
                    for (int w = 0; w < W; ++w) c[e + w] = tc[w], s[e + w] = ts[w];
                }
            }
            if (HALF || V == 1) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float x1 = to_f<T>(a[j].e[e]), x2 = to_f<T>(b[j].e[e]);
                    a[j].e[e] = from_f<T>(x1 * c[e] - x2 * s[e]);
                    b[j].e[e] = from_f<T>(x2 * c[e] + x1 * s[e]);
                }
                *(decltype(a[j].raw) *)dst[j] = a[j].raw;
                *(decltype(b[j].raw) *)(dst[j] + (HALF ? half : 1)) = b[j].raw;
            } else {
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const float x1 = to_f<T>(a[j].e[2 * e]), x2 = to_f<T>(a[j].e[V > 1 ? 2 * e + 1 : 0]);
                    a[j].e[2 * e] = from_f<T>(x1 * c[e] - x2 * s[e]);
                    a[j].e[V > 1 ? 2 * e + 1 : 0] = from_f<T>(x2 * c[e] + x1 * s[e]);
                }
                *(decltype(a[j].raw) *)dst[j] = a[j].raw;
            }
        }
    }
    if (p.c_q + p.c_k == 0) return;
    switch (p.copy_bytes) {
    case 16: copy_rest<T, uint4>(p, tok0, nt); break;
    case 8: copy_rest<T, uint2>(p, tok0, nt); break;
    case 4: copy_rest<T, uint32_t>(p, tok0, nt); break;
    default: copy_rest<T, uint16_t>(p, tok0, nt); break;
    }
}

// Whether vectors of v elements divide `width` channels (and a head) and fit every base and stride
bool fits(const RotaryProblem &p, int v, int width) {
    const gdn_rotary_desc &d = p.d;
    const size_t bytes = v * act_size(d.dtype);
    if (bytes > 16 || width % v || d.d % v) return false;
    const void *ptrs[] = {p.q, p.qo, d.Hk ? p.k : nullptr, d.Hk ? p.ko : nullptr};
    const int64_t st[] = {d.q_stride_t, d.q_out_stride_t, d.Hk ? d.k_stride_t : 0, d.Hk ? d.k_out_stride_t : 0};
    const int64_t sb[] = {d.q_stride_b, d.q_out_stride_b, d.Hk ? d.k_stride_b : 0, d.Hk ? d.k_out_stride_b : 0};
    for (int i = 0; i < 4; ++i)
        if (!ptr_aligned(ptrs[i], bytes) || (d.T > 1 && st[i] % v) || (d.B > 1 && sb[i] % v)) return false;
    return true;
}

template <typename T, int V, bool HALF>
cudaError_t launch_rotary(RotaryProblem p, cudaStream_t s) {
    constexpr int NP = HALF ? V : (V > 1 ? V / 2 : 1);
    const gdn_rotary_desc &d = p.d;
    const int64_t ntok = (int64_t)d.B * d.T;
    p.u_rot = d.rot / 2 / NP;
    int vc = 16 / (int)sizeof(T);   // a head's start, the rotated part and the rest: multiples of the copy's vector
    while (vc > 1 && !fits(p, vc, d.rot)) vc /= 2;
    p.copy_bytes = vc * (int)sizeof(T);
    p.u_copy = (d.d - d.rot) / vc;
    p.u_q = d.Hq * p.u_rot;
    p.u_k = d.Hk * p.u_rot;
    p.c_q = p.q == p.qo ? 0 : d.Hq * p.u_copy;
    p.c_k = p.k == p.ko ? 0 : d.Hk * p.u_copy;
    // tokens per CTA: about four batches of units for every thread (131072 x 32 heads of 128: one 324 us, two 313, four
    // 309, eight 314; 316 at the copy rate), as long as that leaves four CTAs per SM and the
    // table fits; few tokens are split over the heads instead
    const int64_t per = (int64_t)p.u_q + p.u_k + p.c_q + p.c_k;
    int64_t tokens = std::max<int64_t>(1, std::min<int64_t>(kBatches * kBatch * kThreads / per, ntok / (4 * kSms)));
    tokens = std::max<int64_t>(1, std::min<int64_t>(tokens, kTableBytes / (4 * (int64_t)d.rot)));
    p.tokens = (int)tokens;
    const int64_t blocks = cdiv64(ntok, tokens);
    const int64_t split = std::max<int64_t>(1, std::min<int64_t>(cdiv64(tokens * per, kThreads), 4 * kSms / std::max<int64_t>(blocks, 1)));
    const size_t smem = (size_t)tokens * d.rot * 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_shared(rotary_kernel<T, V, HALF>, 4 * kMostRotated);
        if (e != cudaSuccess) return e;
    }
    rotary_kernel<T, V, HALF><<<dim3((unsigned)std::max<int64_t>(blocks, 1), (unsigned)split), kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, bool HALF>
cudaError_t launch_by_vector(const RotaryProblem &p, cudaStream_t s) {
    const int width = HALF ? p.d.rot / 2 : p.d.rot;
    const auto can = [&](int v) { return fits(p, v, width); };
    if constexpr (sizeof(T) == 2)
        if (can(8)) return launch_rotary<T, 8, HALF>(p, s);
    if (can(4)) return launch_rotary<T, 4, HALF>(p, s);
    if (can(2)) return launch_rotary<T, 2, HALF>(p, s);
    return launch_rotary<T, 1, HALF>(p, s);
}

}  // namespace

int rotary_check_desc(const gdn_rotary_desc *d, bool packed) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->N < 1 || d->Hq < 1 || d->Hk < 0 || d->d < 2) return GDN_ERR_INVALID_ARG;
    if (packed ? d->B != 1 : d->N != d->B) return GDN_ERR_INVALID_ARG;
    if (d->rot < 2 || d->rot > d->d || d->rot % 2) return GDN_ERR_INVALID_ARG;
    if (d->layout != GDN_ROTARY_HALF && d->layout != GDN_ROTARY_INTERLEAVED) return GDN_ERR_INVALID_ARG;
    if (d->inverse != 0 && d->inverse != 1) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)d->d * ((int64_t)d->Hq + d->Hk) > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    if (d->rot > kMostRotated) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)d->B * d->T > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
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
    return rotary_check_desc(d, packed != 0);
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
        if (!isfinite(t)) return GDN_ERR_INVALID_ARG;
        // whole turns drop out; 1 - 2^-53 is the largest fraction, so the product stays below 2^64
        turns[i] = (uint64_t)ldexp(t - floor(t), 64);
    }
    return GDN_OK;
}

int gdn_rotary_workspace_bytes(const gdn_rotary_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = rotary_check_desc(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

int gdn_rotary(const gdn_rotary_desc *d, const void *q, const void *k, const uint64_t *turns, const int32_t *positions,
               const int32_t *cu_seqlens, const int32_t *offsets, void *q_out, void *k_out, void *workspace,
               size_t workspace_bytes, gdn_stream_t stream) {
    int rc = rotary_check_desc(d, cu_seqlens != nullptr);
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
    RotaryProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.q = q;
    p.k = k;
    p.turns = turns;
    p.pos = positions;
    p.cu = cu_seqlens;
    p.off = offsets;
    p.qo = q_out;
    p.ko = k_out;
    p.status = (int32_t *)workspace;
    const bool half = d->layout == GDN_ROTARY_HALF;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d->dtype) {
    case GDN_F32: return layer_status(half ? launch_by_vector<float, true>(p, s) : launch_by_vector<float, false>(p, s));
    case GDN_BF16:
        return layer_status(half ? launch_by_vector<__nv_bfloat16, true>(p, s) : launch_by_vector<__nv_bfloat16, false>(p, s));
    default: return layer_status(half ? launch_by_vector<__half, true>(p, s) : launch_by_vector<__half, false>(p, s));
    }
}

}  // extern "C"
