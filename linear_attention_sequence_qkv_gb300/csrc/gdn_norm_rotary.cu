// gdn_norm_rotary.cu -- the norm of every head of q and k with the rotary positions in the
// same pass (include/gdn.h), forward and backward.
//
// Streaming kernels, bound by HBM: a team of lanes (the power of two that a head's vectors
// fill) takes a token, or a part of its heads, computes the token's cosines and sines once into
// registers, and goes through the heads with four of them on their way; the other half of a pair
// comes from its lane by shuffle, as raw bits. Where vectors do not fit (odd widths, unaligned
// rows), a warp takes one head at a time through shared memory. 131072 tokens of 48 heads of 128,
// 16 bits: 520 us, 91 % of the copy rate; the backward 77 % (32768 tokens: 230 us). fp32 at 32768
// tokens: 252 us, 94 %, and 421, 85 %. Few heads per token leave the cosines to be the work
// (65536 tokens of 5 heads of 64: 30 us, 42 %).
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
constexpr int kVectorCtas = 2 * kSms; // of its vector kernel, whose registers leave room for two per SM: twice as many take 2 us more

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

// The sum of the CTAs' partial weight gradients, in order: a warp reads 32 channels of every 32nd CTA's row.
__global__ void __launch_bounds__(1024) norm_rotary_weights(const __grid_constant__ NormRotaryProblem p) {
    __shared__ float part[32][33];
    if (*p.status != GDN_OK) return;
    const int d = p.n.rotary.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < 2 * d)
#pragma unroll 8
        for (int i = warp; i < p.ctas; i += 32) s += p.part[(int64_t)i * 2 * d + c];
    part[warp][lane] = s;
    __syncthreads();
    // a warp adds up one channel
    s = warp_sum(part[lane][warp]);
    const int w = blockIdx.x * 32 + warp;
    float *to = w < d ? p.dqw : p.dkw;
    if (lane == 0 && w < 2 * d && to) to[w < d ? w : w - d] = s;
}

// ------------------------------------------------------------- vectors in registers
template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <typename T, int V> union Vec {
    typename Raw<V * sizeof(T)>::type raw;
    uint32_t w[V * sizeof(T) / 4];
    T e[V];
};

constexpr int kThreads = 256;
constexpr int kFlight = 4;   // heads whose loads are on their way at once

// How channels turn: pairs of neighbours, halves, or halves of an odd number of segments
enum Turn { kNeighbours, kHalves, kOddHalves };

// A lane's place in its team: K vectors of V channels, lane + k team of them; for each the channel it starts at, and for its
// segments of SEG channels what they do in the turn and, for the half layouts, the vector that holds the other half of their
// pairs. Eight 16-bit channels are two segments, so that half the turned channels need only be a multiple of four: with an odd
// number of segments the other half of one lies in the other of its vector (131072 tokens of 8 heads of 96, 24 turned: 160 us,
// with vectors of four channels 213; where halves are whole vectors segments would cost up to 8 %).
template <typename T, int V, int K, Turn M> struct Place {
    static constexpr int S = sizeof(T) == 2 && V == 8 && M != kHalves ? 2 : 1, SEG = V / S;
    int c[K], other[K][S];   // first channel (-1: none); the partner's vector
    bool turned[K][S], upper[K][S];
    __device__ __forceinline__ Place(const gdn_rotary_desc &d, int lane, int team) {
        const int off = d.rot / 2 / SEG;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = k * team + lane;
            c[k] = v * V < d.d ? v * V : -1;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int g = v * S + s;
                turned[k][s] = g * SEG < d.rot;
                upper[k][s] = M != kNeighbours && g >= off;
                other[k][s] = M == kNeighbours || !turned[k][s] ? v : (upper[k][s] ? g - off : g + off) / S;
            }
        }
    }
};
// Pairs of neighbouring channels, in one instruction where the SM has one for two. A turn is y = x A + o B with o the other
// half's channels (half layout) or the pair swapped, and A, B of the lane's pairs at a position, the attention factor among
// them: (cos, cos) and (-+sin, -+sin), or (cos, cos) and (-sin, sin); ones and zeros where nothing turns.
template <typename T, int V, int K, Turn M>
__device__ __forceinline__ void turns_of(const NormRotaryProblem &p, const Place<T, V, K, M> &at, int64_t pos, float2 (&A)[K][V / 2], float2 (&B)[K][V / 2]) {
    const gdn_rotary_desc &d = p.n.rotary;
    auto turn = [&](int pair) {
        const float2 cs = cos_sin<sizeof(T) == 2>(pos, p.turns[pair]);
        return make_float2(cs.x * d.scale, cs.y * d.scale);
    };
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            A[k][e] = splat2(1.0f), B[k][e] = splat2(0.0f);
            const int s = 2 * e / at.SEG;
            if (!at.turned[k][s]) continue;
            if (M != kNeighbours) {
                const int pair = at.c[k] + 2 * e - (at.upper[k][s] ? d.rot / 2 : 0);
                const float2 a = turn(pair), b = turn(pair + 1);
                A[k][e] = make_float2(a.x, b.x);
                B[k][e] = at.upper[k][s] ? make_float2(a.y, b.y) : make_float2(-a.y, -b.y);
            } else {
                const float2 a = turn(at.c[k] / 2 + e);
                A[k][e] = splat2(a.x);
                B[k][e] = make_float2(-a.y, a.y);
            }
        }
}
template <typename T, int V> __device__ __forceinline__ float2 pair_of(const Vec<T, V> &v, int e) {
    if constexpr (sizeof(T) == 4) return make_float2(v.e[2 * e], v.e[2 * e + 1]);
    else return Pairs<T>::word(v.w[e]);
}
template <typename T, int V> __device__ __forceinline__ void set_pair(Vec<T, V> &v, int e, float2 x) {
    if constexpr (sizeof(T) == 4) v.e[2 * e] = x.x, v.e[2 * e + 1] = x.y;
    else v.w[e] = Pairs<T>::pack1(x);
}
__device__ __forceinline__ float2 swapped(float2 x) { return make_float2(x.y, x.x); }
// two channels' weights
__device__ __forceinline__ float2 weights_at(const void *w, int dtype, int c) { return make_float2(weight_at(w, dtype, c), weight_at(w, dtype, c + 1)); }

// the other half's vectors
template <typename T, int V, int K, Turn M>
__device__ __forceinline__ void partners(const Place<T, V, K, M> &at, const Vec<T, V> (&x)[K], Vec<T, V> (&o)[K], int team) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int w = 0; w < (int)(V * sizeof(T) / 4); ++w) {
            constexpr int S = Place<T, V, K, M>::S;
            const int other = at.other[k][S == 2 ? w / 2 : 0];
            uint32_t got = 0;
#pragma unroll
            for (int q = 0; q < K; ++q) {
                const uint32_t v = __shfl_sync(0xffffffffu, x[q].w[S == 2 ? w ^ 2 : w], other & (team - 1), team);
                if (K == 1 || other / team == q) got = v;
            }
            o[k].w[w] = got;
        }
}
template <int TEAM> __device__ __forceinline__ float team_sum(float v) {
#pragma unroll
    for (int o = TEAM / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A team's item: a token and a run of its heads
struct Item {
    int row, t;
    int64_t tok;
    bool ok;
};
__device__ __forceinline__ Item item_at(const gdn_rotary_desc &d, int64_t i, int parts, int &part) {
    Item x = {0, 0, 0, i < (int64_t)d.B * d.T * parts};
    part = 0;
    if (!x.ok) return x;
    x.tok = i / parts;
    part = (int)(i - x.tok * parts);
    x.row = (int)(x.tok / d.T);
    x.t = (int)(x.tok - (int64_t)x.row * d.T);
    return x;
}

template <typename T, int V, int K, int TEAM, Turn M>
__global__ void __launch_bounds__(kThreads, K == 1 ? 3 : 1) norm_rotary_vectors(const __grid_constant__ NormRotaryProblem p, int parts, int per) {
    const gdn_rotary_desc &d = p.n.rotary;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int lane = threadIdx.x % TEAM;
    int part;
    const Item it = item_at(d, (int64_t)blockIdx.x * (kThreads / TEAM) + threadIdx.x / TEAM, parts, part);
    const Place<T, V, K, M> at(d, lane, TEAM);
    const int h0 = part * per, h1 = it.ok ? min(h0 + per, d.Hq + d.Hk) : h0;   // the lanes of a warp stay together: empty runs loop too
    constexpr int NP = V / 2;
    const int64_t pos = it.ok ? rotary_position(d, p.pos, p.cu, p.off, it.row, it.t) : 0;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const void *w = which ? p.kw : p.qw;
        const int a = max(h0, which ? d.Hq : 0), b = min(h1, which ? d.Hq + d.Hk : d.Hq), first = which ? d.Hq : 0;
        const T *src = (const T *)(which ? p.k : p.q) + it.row * (which ? d.k_stride_b : d.q_stride_b) + it.t * (which ? d.k_stride_t : d.q_stride_t);
        T *dst = (T *)(which ? p.ko : p.qo) + it.row * (which ? d.k_out_stride_b : d.q_out_stride_b) + it.t * (which ? d.k_out_stride_t : d.q_out_stride_t);
        const int runs = max(0, b - a), most = __reduce_max_sync(0xffffffffu, runs);
        if (most == 0) continue;
        // the weights go into the turn: y = rstd (x A w + o B w'). It is computed again for k: kept beside the weighted one it
        // takes registers of the loads on their way (32768 tokens of 48 heads of 128: 155 us, 141 so).
        float2 A[K][NP], B[K][NP], Aw[K][NP], Bw[K][NP];
        turns_of<T, V, K, M>(p, at, pos, A, B);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const float2 own = at.c[k] >= 0 ? weights_at(w, p.n.weight_dtype, at.c[k] + 2 * e) : splat2(0.0f);
                Aw[k][e] = mul2(A[k][e], own);
                const int s = 2 * e / at.SEG, half = at.upper[k][s] ? -d.rot / 2 : d.rot / 2;
                if (M != kNeighbours) Bw[k][e] = at.turned[k][s] ? mul2(B[k][e], weights_at(w, p.n.weight_dtype, at.c[k] + 2 * e + half)) : splat2(0.0f);
                else Bw[k][e] = mul2(B[k][e], swapped(own));
            }
        for (int r0 = 0; r0 < most; r0 += kFlight) {
            Vec<T, V> x[kFlight][K];
#pragma unroll
            for (int j = 0; j < kFlight; ++j)
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int q = 0; q < (int)(V * sizeof(T) / 4); ++q) x[j][k].w[q] = 0;
                    if (r0 + j < runs && at.c[k] >= 0) x[j][k].raw = *(const decltype(x[j][k].raw) *)(src + (int64_t)(a + r0 + j - first) * d.d + at.c[k]);
                }
#pragma unroll
            for (int j = 0; j < kFlight; ++j) {
                if (r0 + j >= most) break;
                float2 xs[K][NP], s2 = splat2(0.0f);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        xs[k][e] = pair_of<T, V>(x[j][k], e);
                        s2 = fma2(xs[k][e], xs[k][e], s2);
                    }
                const float2 rstd = splat2(rsqrtf(team_sum<TEAM>(s2.x + s2.y) / d.d + p.n.eps));
                Vec<T, V> o[K], y[K];
                if (M != kNeighbours) partners<T, V, K, M>(at, x[j], o, TEAM);
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        float2 z = mul2(xs[k][e], Aw[k][e]);
                        // (a partner that is not finite must not reach what does not turn)
                        if (M == kNeighbours || at.turned[k][2 * e / at.SEG]) z = fma2(M != kNeighbours ? pair_of<T, V>(o[k], e) : swapped(xs[k][e]), Bw[k][e], z);
                        set_pair<T, V>(y[k], e, mul2(z, rstd));
                    }
                    if (r0 + j < runs && at.c[k] >= 0) *(decltype(y[k].raw) *)(dst + (int64_t)(a + r0 + j - first) * d.d + at.c[k]) = y[k].raw;
                }
            }
        }
    }
}

// Both tensors of kFlight heads are on their way at once: with two heads' 4474 GB/s instead of 5480 (32768 tokens of 48 heads of
// 128, 16 bits), with six, or a third CTA per SM, the registers spill (5092 and 3455 GB/s).
template <typename T, int V, int K, int TEAM, Turn M>
__global__ void __launch_bounds__(kThreads, K == 1 ? 2 : 1) norm_rotary_vectors_backward(const __grid_constant__ NormRotaryProblem p, int parts, int per) {
    extern __shared__ float sm[];   // [teams][2][d]
    const gdn_rotary_desc &d = p.n.rotary;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    constexpr int kTeams = kThreads / TEAM;
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const Place<T, V, K, M> at(d, lane, TEAM);
    constexpr int NP = V / 2;
    float2 acc[2][K][NP];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < NP; ++e) acc[w][k][e] = splat2(0.0f);
    const int64_t items = (int64_t)d.B * d.T * parts;
    for (int64_t i0 = (int64_t)blockIdx.x * kTeams; i0 < items; i0 += (int64_t)gridDim.x * kTeams) {
        int part;
        const Item it = item_at(d, i0 + team, parts, part);
        const int h0 = part * per, h1 = it.ok ? min(h0 + per, d.Hq + d.Hk) : h0;
        float2 A[K][NP], B[K][NP];
        turns_of<T, V, K, M>(p, at, it.ok ? rotary_position(d, p.pos, p.cu, p.off, it.row, it.t) : 0, A, B);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const void *w = which ? p.kw : p.qw;
            const int a = max(h0, which ? d.Hq : 0), b = min(h1, which ? d.Hq + d.Hk : d.Hq), first = which ? d.Hq : 0;
            const T *src = (const T *)(which ? p.k : p.q) + it.row * (which ? d.k_stride_b : d.q_stride_b) + it.t * (which ? d.k_stride_t : d.q_stride_t);
            const T *grd = (const T *)(which ? p.ko : p.qo) + it.row * (which ? d.k_out_stride_b : d.q_out_stride_b) +
                           it.t * (which ? d.k_out_stride_t : d.q_out_stride_t);
            T *dst = (T *)(which ? p.dk : p.dq) + it.tok * (which ? d.Hk : d.Hq) * d.d;
            const int runs = max(0, b - a), most = __reduce_max_sync(0xffffffffu, runs);
            if (most == 0) continue;
            float2 wo[K][NP];
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int e = 0; e < NP; ++e) wo[k][e] = at.c[k] >= 0 ? weights_at(w, p.n.weight_dtype, at.c[k] + 2 * e) : splat2(0.0f);
            for (int r0 = 0; r0 < most; r0 += kFlight) {
                Vec<T, V> x[kFlight][K], g[kFlight][K];
#pragma unroll
                for (int j = 0; j < kFlight; ++j)
#pragma unroll
                    for (int k = 0; k < K; ++k) {
#pragma unroll
                        for (int q = 0; q < (int)(V * sizeof(T) / 4); ++q) x[j][k].w[q] = g[j][k].w[q] = 0;
                        if (r0 + j < runs && at.c[k] >= 0) {
                            x[j][k].raw = *(const decltype(x[j][k].raw) *)(src + (int64_t)(a + r0 + j - first) * d.d + at.c[k]);
                            g[j][k].raw = *(const decltype(g[j][k].raw) *)(grd + (int64_t)(a + r0 + j - first) * d.d + at.c[k]);
                        }
                    }
#pragma unroll
                for (int j = 0; j < kFlight; ++j) {
                    if (r0 + j >= most) break;
                    Vec<T, V> o[K];
                    if (M != kNeighbours) partners<T, V, K, M>(at, g[j], o, TEAM);
                    float2 ss = splat2(0.0f), st = splat2(0.0f), dz[K][NP], xs[K][NP];
#pragma unroll
                    for (int k = 0; k < K; ++k)
#pragma unroll
                        for (int e = 0; e < NP; ++e) {
                            const float2 gv = pair_of<T, V>(g[j][k], e);
                            xs[k][e] = pair_of<T, V>(x[j][k], e);
                            dz[k][e] = mul2(gv, A[k][e]);
                            // the turn back: B the other way round
                            if (M == kNeighbours || at.turned[k][2 * e / at.SEG])
                                dz[k][e] = fma2(M != kNeighbours ? pair_of<T, V>(o[k], e) : swapped(gv), make_float2(-B[k][e].x, -B[k][e].y), dz[k][e]);
                            ss = fma2(xs[k][e], xs[k][e], ss);
                            st = fma2(mul2(dz[k][e], wo[k][e]), xs[k][e], st);
                        }
                    const float rstd = rsqrtf(team_sum<TEAM>(ss.x + ss.y) / d.d + p.n.eps);
                    const float2 r2 = splat2(rstd), mean = splat2(-rstd * team_sum<TEAM>(st.x + st.y) / d.d);   // of t xh
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        Vec<T, V> y;
#pragma unroll
                        for (int e = 0; e < NP; ++e) {
                            const float2 xh = mul2(xs[k][e], r2);
                            // (a team whose run is shorter than its warp's has no head here, and eps may be 0: no 0 x inf into the sums)
                            if (r0 + j < runs) acc[which][k][e] = fma2(dz[k][e], xh, acc[which][k][e]);
                            set_pair<T, V>(y, e, mul2(r2, fma2(xh, mean, mul2(dz[k][e], wo[k][e]))));
                        }
                        if (r0 + j < runs && at.c[k] >= 0) *(decltype(y.raw) *)(dst + (int64_t)(a + r0 + j - first) * d.d + at.c[k]) = y.raw;
                    }
                }
            }
        }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < NP; ++e)
                if (at.c[k] >= 0) *(float2 *)&sm[(team * 2 + w) * d.d + at.c[k] + 2 * e] = acc[w][k][e];
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * d.d; c += kThreads) {
        float s = 0.0f;
        for (int x = 0; x < kTeams; ++x) s += sm[x * 2 * d.d + c];
        p.part[(int64_t)blockIdx.x * 2 * d.d + c] = s;
    }
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

// Whether vectors of v elements divide a head and its rotated part and fit every base and stride
bool fits(const NormRotaryProblem &p, int v) {
    const gdn_rotary_desc &d = p.n.rotary;
    const size_t bytes = v * act_size(d.dtype);
    const int width = d.layout == GDN_ROTARY_HALF ? d.rot / 2 : d.rot;   // made of whole segments (Place)
    if (bytes < 4 || bytes > 16 || v < 2 || width % (v == 8 ? 4 : v) || d.d % v || d.d / v > 64) return false;
    const void *ptrs[] = {p.q, p.qo, p.k, p.ko, p.dq, p.dk};
    for (const void *x : ptrs)
        if (!ptr_aligned(x, bytes)) return false;
    const int64_t st[] = {d.q_stride_t, d.q_out_stride_t, d.Hk ? d.k_stride_t : 0, d.Hk ? d.k_out_stride_t : 0};
    const int64_t sb[] = {d.q_stride_b, d.q_out_stride_b, d.Hk ? d.k_stride_b : 0, d.Hk ? d.k_out_stride_b : 0};
    for (int i = 0; i < 4; ++i)
        if ((d.T > 1 && st[i] % v) || (d.B > 1 && sb[i] % v)) return false;
    return true;
}

// Parts of a token's heads: until there are 32 warps per SM
int parts_of(const gdn_rotary_desc &d, int team) {
    const int64_t ntok = std::max<int64_t>((int64_t)d.B * d.T, 1), teams = (int64_t)kSms * 32 * (32 / team);
    return (int)std::min<int64_t>(d.Hq + d.Hk, cdiv64(teams, ntok));
}

template <typename T, int V, int K, int TEAM, Turn M>
cudaError_t launch_vectors(NormRotaryProblem &p, bool backward, cudaStream_t s) {
    const gdn_rotary_desc &d = p.n.rotary;
    constexpr int kTeams = kThreads / TEAM;
    const int heads = d.Hq + d.Hk, per = (int)cdiv64(heads, parts_of(d, TEAM)), parts = (int)cdiv64(heads, per);
    const int64_t blocks = std::max<int64_t>(cdiv64((int64_t)d.B * d.T * parts, kTeams), 1);
    if (!backward) {
        if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
        norm_rotary_vectors<T, V, K, TEAM, M><<<(unsigned)blocks, kThreads, 0, s>>>(p, parts, per);
        return cudaGetLastError();
    }
    const size_t smem = (size_t)kTeams * 2 * d.d * 4;   // at most 32 KB: a team's channels are at most 16 of its lanes' bytes
    p.ctas = (int)std::min<int64_t>({blocks, p.ctas, kVectorCtas});
    norm_rotary_vectors_backward<T, V, K, TEAM, M><<<(unsigned)p.ctas, kThreads, smem, s>>>(p, parts, per);
    return cudaGetLastError();
}
template <typename T, int V, Turn M>
cudaError_t launch_team(NormRotaryProblem &p, bool backward, cudaStream_t s) {
    const int nv = p.n.rotary.d / V;
    if (nv > 32) return launch_vectors<T, V, 2, 32, M>(p, backward, s);
    if (nv > 16) return launch_vectors<T, V, 1, 32, M>(p, backward, s);
    if (nv > 8) return launch_vectors<T, V, 1, 16, M>(p, backward, s);
    return launch_vectors<T, V, 1, 8, M>(p, backward, s);
}
template <typename T>
cudaError_t launch(NormRotaryProblem &p, bool backward, cudaStream_t s) {
    const gdn_rotary_desc &d = p.n.rotary;
    const bool half = d.layout == GDN_ROTARY_HALF;
    cudaError_t e = cudaSuccess;
    bool done = false;
    if constexpr (sizeof(T) == 2)
        if (fits(p, 8))
            e = !half ? launch_team<T, 8, kNeighbours>(p, backward, s)
                : d.rot % 16 ? launch_team<T, 8, kOddHalves>(p, backward, s) : launch_team<T, 8, kHalves>(p, backward, s), done = true;
    if (!done && fits(p, 4)) e = half ? launch_team<T, 4, kHalves>(p, backward, s) : launch_team<T, 4, kNeighbours>(p, backward, s), done = true;
    if (!done && fits(p, 2)) e = half ? launch_team<T, 2, kHalves>(p, backward, s) : launch_team<T, 2, kNeighbours>(p, backward, s), done = true;
    if (!done && !backward) {
        const int64_t blocks = std::min<int64_t>(std::max<int64_t>(cdiv64(heads_of(d), kWarps), 1), 16 * kSms);
        norm_rotary_rows<T><<<(unsigned)blocks, 32 * kWarps, (size_t)kWarps * d.d * 4, s>>>(p);
        e = cudaGetLastError();
    } else if (!done) {
        const size_t smem = (size_t)kWarps * 4 * d.d * 4;
        if (smem > 48 * 1024) e = allow_shared(norm_rotary_rows_backward<T>, (size_t)kWarps * 4 * kMostChannels * 4);
        if (e != cudaSuccess) return e;
        norm_rotary_rows_backward<T><<<(unsigned)p.ctas, 32 * kWarps, smem, s>>>(p);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || !backward || (!p.dqw && !p.dkw)) return e;
    norm_rotary_weights<<<(unsigned)cdiv64(2 * d.d, 32), 1024, 0, s>>>(p);
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
    case GDN_F32: return layer_status(launch<float>(p, false, s));
    case GDN_BF16: return layer_status(launch<__nv_bfloat16>(p, false, s));
    default: return layer_status(launch<__half>(p, false, s));
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
    case GDN_F32: return layer_status(launch<float>(p, true, s));
    case GDN_BF16: return layer_status(launch<__nv_bfloat16>(p, true, s));
    default: return layer_status(launch<__half>(p, true, s));
    }
}

}  // extern "C"
