// gdn_group_norm.cu -- group norm with an activation, channels last (include/gdn.h):
// forward and backward. Bound by HBM.
//
// A warp works on a fixed set of adjacent channels: 32 / LG groups of LG lanes each
// (LG, a power of two, covers a group's vectors), or a 32-lane slab of a larger group.
// Weights stay in registers, sums cross lanes by shuffles, and rows stream past.
//
//   rows     L = 1 and a group fits LG lanes x NV vectors: a row is read once, its mean
//            and its centred squares are summed from registers, and it is written. Four
//            rows are in flight per warp.
//   general  several positions, or larger groups: partial means and centred sums of
//            squares per (instance, chunk of positions), merged pairwise; a second pass
//            normalises (one kernel where a warp holds a whole group, else two). The
//            second read comes from L2 where the tensor fits.
//
// The backward has the same two forms, with the sums of t and t xh in the statistics'
// place. Parameter gradients are summed per warp over its rows, written as partial rows
// and added up by a last small kernel. Every order is fixed by the sizes.
#include <string.h>

#include <algorithm>

#include "gdn_layer_ops.cuh"

namespace gdn {
namespace {

struct NormProblem {
    gdn_group_norm_desc d;
    const void *x, *w, *b, *dy;
    void *out, *dx;
    float *mean, *rstd, *dw, *db;
    float2 *stat;      // general: [item][part] partial (mean, centred sum of squares), or (sum t, sum t xh)
    float *part;       // [slices][2][C] partial sums of dweight, dbias
    int lg;            // lanes per group or slab
    int sets;          // sets of channels, one per warp
    int slabs;         // slabs per group (1 where a warp holds whole groups)
    int slices;        // warps that share a set
    int chunks, chunk_rows;   // general: chunks of positions per instance
    int64_t items;     // rows, or (instance, chunk) pairs
};

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocksForward = 3, kBlocksBackward = 2, kBlocksGeneral = 4;   // per SM, resident at once

template <typename T> struct VecN { static constexpr int value = 16 / sizeof(T); };

// V elements of T as fp32 (V = 1, or 16 bytes)
template <typename T, int V>
__device__ __forceinline__ void load_v(const T *p, float *v) {
    if constexpr (V == 1) v[0] = to_f<T>(*p);
    else unpack16<T>(*reinterpret_cast<const uint4 *>(p), v);
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T *p, const float *v) {
    if constexpr (V == 1) *p = from_f<T>(v[0]);
    else *reinterpret_cast<uint4 *>(p) = pack16<T>(v);
}

__device__ __forceinline__ float param(const void *p, int dtype, int c, float none) {
    if (!p) return none;
    return dtype == GDN_F32 ? ((const float *)p)[c]
           : dtype == GDN_BF16 ? __bfloat162float(((const __nv_bfloat16 *)p)[c]) : __half2float(((const __half *)p)[c]);
}

__device__ __forceinline__ float lane_sum(float v, int lg) {   // over lg adjacent lanes, the same in all of them
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        if (off < lg) v += o;
    }
    return v;
}

__device__ __forceinline__ float sigmoid_fast(float z) { return rcp_approx(1.f + ex2_approx(-1.4426950408889634f * z)); }
__device__ __forceinline__ float act_f(float z, int act) { return act == GDN_ACT_SILU ? z * sigmoid_fast(z) : z; }
__device__ __forceinline__ float act_grad(float z, int act) {   // d act(z) / dz
    if (act == GDN_ACT_NONE) return 1.f;
    const float s = sigmoid_fast(z), zc = fminf(fmaxf(z, -3e38f), 3e38f);   // no 0 times inf
    return s * fmaf(zc, 1.f - s, 1.f);
}

// The warp's place: its set, its lane's first channel, and whether the lane has channels.
struct Place {
    int set, slice, sub;   // sub: lane within the group's lanes
    int g;                 // group
    int c;                 // the lane's first channel
    bool any;
};
template <int V>
__device__ __forceinline__ Place place(const NormProblem &p) {
    const int w = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    const int cg = p.d.C / p.d.G;
    Place q;
    q.set = w % p.sets;
    q.slice = w / p.sets;
    q.sub = lane % p.lg;
    int in;                // the lane's first element within the group
    if (p.slabs == 1) {
        q.g = q.set * (32 / p.lg) + lane / p.lg;
        in = q.sub * V;
    } else {
        q.g = q.set / p.slabs;
        in = (q.set % p.slabs * 32 + lane) * V;
    }
    q.any = q.slice < p.slices && q.g < p.d.G && in < cg;
    if (q.g >= p.d.G) q.g = p.d.G - 1;
    q.c = q.g * cg + in;
    return q;
}

// ------------------------------------------------------------------ rows
constexpr int kRows = 4;   // vectors in flight per lane

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads, NV == 1 ? kBlocksForward : 1) norm_rows_forward(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (q.slice >= p.slices) return;
    const int cg = d.C / d.G;
    const float inv = 1.f / (float)cg;
    constexpr int kR = kRows / NV;
    bool has[NV];
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        has[i] = q.any && (q.sub + i * p.lg) * V < cg;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[i][e] = has[i] ? param(p.w, d.weight_dtype, q.c + i * p.lg * V + e, 1.f) : 0.f;
            b[i][e] = has[i] ? param(p.b, d.weight_dtype, q.c + i * p.lg * V + e, 0.f) : 0.f;
        }
    }
    for (int64_t n0 = q.slice; n0 < p.items; n0 += (int64_t)kR * p.slices) {
        float x[kR][NV][V], mean[kR], rstd[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int64_t n = n0 + (int64_t)r * p.slices;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (n < p.items && has[i]) load_v<T, V>((const T *)p.x + n * d.x_stride_n + q.c + i * p.lg * V, x[r][i]);
                else
#pragma unroll
                    for (int e = 0; e < V; ++e) x[r][i][e] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) s += x[r][i][e];
            mean[r] = lane_sum(s, p.lg) * inv;
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[r][i][e] -= mean[r];
                    if (has[i]) s = fmaf(x[r][i][e], x[r][i][e], s);
                }
            rstd[r] = rsqrtf(fmaf(lane_sum(s, p.lg), inv, d.eps));
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int64_t n = n0 + (int64_t)r * p.slices;
            if (n >= p.items || !q.any) continue;
            if (q.sub == 0) {
                if (p.mean) p.mean[n * d.G + q.g] = mean[r];
                if (p.rstd) p.rstd[n * d.G + q.g] = rstd[r];
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has[i]) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) x[r][i][e] = act_f(fmaf(x[r][i][e] * rstd[r], w[i][e], b[i][e]), d.act);
                store_v<T, V>((T *)p.out + n * d.C + q.c + i * p.lg * V, x[r][i]);
            }
        }
    }
}

// The element's part of the backward: xh, dz = dout act'(z), t = dz w.
struct Grad {
    float xh, dz, t;
};
__device__ __forceinline__ Grad grad_of(float x, float dy, float mean, float rstd, float w, float b, int act) {
    Grad g;
    g.xh = (x - mean) * rstd;
    g.dz = dy * act_grad(fmaf(g.xh, w, b), act);
    g.t = g.dz * w;
    return g;
}

// Sums of dweight and dbias of a warp's channels: over 16 rows, over all (the second level keeps the
// rounding of long sums down), then into its partial row.
template <int N> struct ParamSums {
    float w[2][N], b[2][N];
    int rows;
    __device__ __forceinline__ ParamSums() {
#pragma unroll
        for (int i = 0; i < N; ++i) w[0][i] = w[1][i] = b[0][i] = b[1][i] = 0.f;
        rows = 0;
    }
    __device__ __forceinline__ void row_done() {
        if (++rows & 15) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[1][i] += w[0][i];
            b[1][i] += b[0][i];
            w[0][i] = b[0][i] = 0.f;
        }
    }
};

template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads, NV == 1 ? kBlocksBackward : 1) norm_rows_backward(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (q.slice >= p.slices) return;
    const int cg = d.C / d.G;
    const float inv = 1.f / (float)cg;
    constexpr int kR = 2 / NV;
    bool has[NV];
    float w[NV][V], b[NV][V];
    ParamSums<NV * V> sums;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        has[i] = q.any && (q.sub + i * p.lg) * V < cg;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[i][e] = has[i] ? param(p.w, d.weight_dtype, q.c + i * p.lg * V + e, 1.f) : 0.f;
            b[i][e] = has[i] ? param(p.b, d.weight_dtype, q.c + i * p.lg * V + e, 0.f) : 0.f;
        }
    }
    for (int64_t n0 = q.slice; n0 < p.items; n0 += (int64_t)kR * p.slices) {
        float x[kR][NV][V], y[kR][NV][V], mean[kR], rstd[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int64_t n = n0 + (int64_t)r * p.slices;
            mean[r] = n < p.items ? p.mean[n * d.G + q.g] : 0.f;
            rstd[r] = n < p.items ? p.rstd[n * d.G + q.g] : 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (n < p.items && has[i]) {
                    load_v<T, V>((const T *)p.x + n * d.x_stride_n + q.c + i * p.lg * V, x[r][i]);
                    load_v<T, V>((const T *)p.dy + n * d.C + q.c + i * p.lg * V, y[r][i]);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) x[r][i][e] = mean[r], y[r][i][e] = 0.f;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int64_t n = n0 + (int64_t)r * p.slices;
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const Grad g = grad_of(x[r][i][e], y[r][i][e], mean[r], rstd[r], w[i][e], b[i][e], d.act);
                    x[r][i][e] = g.xh;
                    y[r][i][e] = g.t;
                    if (n < p.items) {
                        sums.w[0][i * V + e] = fmaf(g.dz, g.xh, sums.w[0][i * V + e]);
                        sums.b[0][i * V + e] += g.dz;
                    }
                    s1 += g.t;
                    s2 = fmaf(g.t, g.xh, s2);
                }
            if (n < p.items) sums.row_done();
            const float m1 = lane_sum(s1, p.lg) * inv, m2 = lane_sum(s2, p.lg) * inv;
            if (n >= p.items) continue;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has[i]) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) y[r][i][e] = rstd[r] * fmaf(-x[r][i][e], m2, y[r][i][e] - m1);
                store_v<T, V>((T *)p.dx + n * d.C + q.c + i * p.lg * V, y[r][i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (has[i]) {
                const int c = q.c + i * p.lg * V + e;
                p.part[((int64_t)q.slice * 2) * d.C + c] = sums.w[1][i * V + e] + sums.w[0][i * V + e];
                p.part[((int64_t)q.slice * 2 + 1) * d.C + c] = sums.b[1][i * V + e] + sums.b[0][i * V + e];
            }
}

// --------------------------------------------------------------- general
// Mean and centred sum of squares of n elements, and their union (n may be 0).
struct Stat {
    float n, mean, m2;
};
__device__ __forceinline__ Stat merge(const Stat &a, const Stat &b) {
    Stat r;
    r.n = a.n + b.n;
    if (r.n == 0.f) return {0.f, 0.f, 0.f};
    const float dl = b.mean - a.mean, f = b.n / r.n;
    r.mean = fmaf(dl, f, a.mean);
    r.m2 = a.m2 + b.m2 + dl * dl * a.n * f;
    return r;
}
__device__ __forceinline__ Stat lane_merge(Stat s, int lg) {   // over lg adjacent lanes, in the same order in all
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Stat o = {__shfl_xor_sync(0xffffffffu, s.n, off), __shfl_xor_sync(0xffffffffu, s.mean, off),
                        __shfl_xor_sync(0xffffffffu, s.m2, off)};
        if (off < lg) s = (lane & off) ? merge(o, s) : merge(s, o);
    }
    return s;
}

// (instance, positions) of an item
__device__ __forceinline__ void item_rows(const NormProblem &p, int64_t item, int64_t &n, int &l0, int &l1) {
    n = item / p.chunks;
    l0 = (int)(item - n * p.chunks) * p.chunk_rows;
    l1 = min(p.d.L, l0 + p.chunk_rows);
}
// where the partial of a set's group (or slab) of an item stands
__device__ __forceinline__ int64_t stat_at(const NormProblem &p, int64_t item, const Place &q) {
    const int64_t parts = (int64_t)p.d.G * p.slabs;
    return item * parts + (p.slabs == 1 ? q.g : q.set);
}

constexpr int kStatRows = 4;

template <typename T, int V>
__device__ __forceinline__ Stat chunk_stat(const NormProblem &p, const Place &q, int64_t n, int l0, int l1) {
    const gdn_group_norm_desc &d = p.d;
    Stat s = {0.f, 0.f, 0.f};
    const T *at = (const T *)p.x + n * d.x_stride_n + q.c;
    for (int l = l0; l < l1; l += kStatRows) {
        float v[kStatRows][V];
        const int rows = min(kStatRows, l1 - l);
#pragma unroll
        for (int r = 0; r < kStatRows; ++r) {
            if (q.any && r < rows) load_v<T, V>(at + (int64_t)(l + r) * d.x_stride_l, v[r]);
            else
#pragma unroll
                for (int e = 0; e < V; ++e) v[r][e] = 0.f;
        }
        float sum = 0.f, m2 = 0.f;
#pragma unroll
        for (int r = 0; r < kStatRows; ++r)
#pragma unroll
            for (int e = 0; e < V; ++e) sum += v[r][e];
        const float cnt = (float)(rows * V), mean = sum / cnt;
#pragma unroll
        for (int r = 0; r < kStatRows; ++r)
            if (r < rows)
#pragma unroll
                for (int e = 0; e < V; ++e) m2 = fmaf(v[r][e] - mean, v[r][e] - mean, m2);
        s = merge(s, {cnt, mean, m2});
    }
    if (!q.any) s = {0.f, 0.f, 0.f};
    return lane_merge(s, p.lg);
}

template <typename T, int V>
__device__ __forceinline__ void normalise(const NormProblem &p, const Place &q, int64_t n, int l0, int l1, float mean, float rstd,
                                          const float *w, const float *b) {
    const gdn_group_norm_desc &d = p.d;
    if (!q.any) return;
    const T *at = (const T *)p.x + n * d.x_stride_n + q.c;
    T *to = (T *)p.out + n * d.L * d.C + q.c;
#pragma unroll 4
    for (int l = l0; l < l1; ++l) {
        float v[V];
        load_v<T, V>(at + (int64_t)l * d.x_stride_l, v);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = act_f(fmaf((v[e] - mean) * rstd, w[e], b[e]), d.act);
        store_v<T, V>(to + (int64_t)l * d.C, v);
    }
}

// The whole group's statistics from the partials of its chunks and slabs
template <int V>
__device__ __forceinline__ Stat group_stat(const NormProblem &p, const Place &q, int64_t n) {
    const gdn_group_norm_desc &d = p.d;
    const int cg = d.C / d.G, parts = p.chunks * p.slabs;
    Stat s = {0.f, 0.f, 0.f};
    for (int i = q.sub; i < parts; i += p.lg) {
        const int k = i / p.slabs, sl = i - k * p.slabs;
        const float2 m = p.stat[((n * p.chunks + k) * d.G + q.g) * p.slabs + sl];
        const int rows = min(d.L, (k + 1) * p.chunk_rows) - k * p.chunk_rows;
        const int width = p.slabs == 1 ? cg : min(cg, (sl + 1) * 32 * V) - sl * 32 * V;
        s = merge(s, {(float)rows * (float)width, m.x, m.y});
    }
    return lane_merge(s, p.lg);
}

template <int V>
__device__ __forceinline__ void load_params(const NormProblem &p, const Place &q, float *w, float *b) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
        w[e] = q.any ? param(p.w, p.d.weight_dtype, q.c + e, 1.f) : 0.f;
        b[e] = q.any ? param(p.b, p.d.weight_dtype, q.c + e, 0.f) : 0.f;
    }
}

// FUSED: one chunk and one slab, so the warp has the whole group and writes it too
template <typename T, int V, bool FUSED>
__global__ void __launch_bounds__(kThreads) norm_stat_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (q.slice >= p.slices) return;
    float w[V], b[V];
    if (FUSED) load_params<V>(p, q, w, b);
    for (int64_t it = q.slice; it < p.items; it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        const Stat s = chunk_stat<T, V>(p, q, n, l0, l1);
        if (FUSED) {
            const float rstd = rsqrtf(s.m2 / s.n + d.eps);
            if (q.any && q.sub == 0) {
                if (p.mean) p.mean[n * d.G + q.g] = s.mean;
                if (p.rstd) p.rstd[n * d.G + q.g] = rstd;
            }
            normalise<T, V>(p, q, n, l0, l1, s.mean, rstd, w, b);
        } else if (q.any && q.sub == 0) {
            p.stat[stat_at(p, it, q)] = make_float2(s.mean, s.m2);
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_apply_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (q.slice >= p.slices) return;
    float w[V], b[V];
    load_params<V>(p, q, w, b);
    for (int64_t it = q.slice; it < p.items; it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        const Stat s = group_stat<V>(p, q, n);
        const float rstd = rsqrtf(s.m2 / s.n + d.eps);
        if (q.any && q.sub == 0 && l0 == 0 && q.c == q.g * (d.C / d.G)) {
            if (p.mean) p.mean[n * d.G + q.g] = s.mean;
            if (p.rstd) p.rstd[n * d.G + q.g] = rstd;
        }
        normalise<T, V>(p, q, n, l0, l1, s.mean, rstd, w, b);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_sums_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (q.slice >= p.slices) return;
    float w[V], b[V];
    load_params<V>(p, q, w, b);
    ParamSums<V> sums;
    for (int64_t it = q.slice; it < p.items; it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        const float mean = p.mean[n * d.G + q.g], rstd = p.rstd[n * d.G + q.g];
        float s1 = 0.f, s2 = 0.f;
        if (q.any) {
            const T *at = (const T *)p.x + n * d.x_stride_n + q.c, *dy = (const T *)p.dy + n * d.L * d.C + q.c;
#pragma unroll 2
            for (int l = l0; l < l1; ++l) {
                float x[V], y[V], r1 = 0.f, r2 = 0.f;
                load_v<T, V>(at + (int64_t)l * d.x_stride_l, x);
                load_v<T, V>(dy + (int64_t)l * d.C, y);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const Grad g = grad_of(x[e], y[e], mean, rstd, w[e], b[e], d.act);
                    sums.w[0][e] = fmaf(g.dz, g.xh, sums.w[0][e]);
                    sums.b[0][e] += g.dz;
                    r1 += g.t;
                    r2 = fmaf(g.t, g.xh, r2);
                }
                s1 += r1;
                s2 += r2;
                sums.row_done();
            }
        }
        s1 = lane_sum(s1, p.lg);
        s2 = lane_sum(s2, p.lg);
        if (q.any && q.sub == 0) p.stat[stat_at(p, it, q)] = make_float2(s1, s2);
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (q.any) {
            p.part[((int64_t)q.slice * 2) * d.C + q.c + e] = sums.w[1][e] + sums.w[0][e];
            p.part[((int64_t)q.slice * 2 + 1) * d.C + q.c + e] = sums.b[1][e] + sums.b[0][e];
        }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (q.slice >= p.slices) return;
    const float count = (float)d.L * (float)(d.C / d.G);
    float w[V], b[V];
    load_params<V>(p, q, w, b);
    for (int64_t it = q.slice; it < p.items; it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        float s1 = 0.f, s2 = 0.f;
        const int parts = p.chunks * p.slabs;
        for (int i = q.sub; i < parts; i += p.lg) {
            const int k = i / p.slabs, sl = i - k * p.slabs;
            const float2 m = p.stat[((n * p.chunks + k) * d.G + q.g) * p.slabs + sl];
            s1 += m.x;
            s2 += m.y;
        }
        const float m1 = lane_sum(s1, p.lg) / count, m2 = lane_sum(s2, p.lg) / count;
        if (!q.any) continue;
        const float mean = p.mean[n * d.G + q.g], rstd = p.rstd[n * d.G + q.g];
        const T *at = (const T *)p.x + n * d.x_stride_n + q.c, *dy = (const T *)p.dy + n * d.L * d.C + q.c;
        T *dx = (T *)p.dx + n * d.L * d.C + q.c;
#pragma unroll 2
        for (int l = l0; l < l1; ++l) {
            float x[V], y[V];
            load_v<T, V>(at + (int64_t)l * d.x_stride_l, x);
            load_v<T, V>(dy + (int64_t)l * d.C, y);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const Grad g = grad_of(x[e], y[e], mean, rstd, w[e], b[e], d.act);
                y[e] = rstd * fmaf(-g.xh, m2, g.t - m1);
            }
            store_v<T, V>(dx + (int64_t)l * d.C, y);
        }
    }
}

// dweight and dbias from part[slices][2][C]: 32 channels a block, 8 strided partial sums each
__global__ void __launch_bounds__(256) norm_params_kernel(const __grid_constant__ NormProblem p) {
    __shared__ float red[2][8][32];
    const int ch = threadIdx.x % 32, c = blockIdx.x * 32 + ch, s = threadIdx.x / 32;
    float v[2] = {0.f, 0.f};
    if (c < p.d.C)
        for (int i = s; i < p.slices; i += 8) {
            v[0] += p.part[((int64_t)i * 2) * p.d.C + c];
            v[1] += p.part[((int64_t)i * 2 + 1) * p.d.C + c];
        }
    red[0][s][ch] = v[0];
    red[1][s][ch] = v[1];
    __syncthreads();
    if (s < 2 && c < p.d.C) {
        float t = 0.f;
        for (int i = 0; i < 8; ++i) t += red[s][i][ch];
        float *to = s ? p.db : p.dw;
        if (to) to[c] = t;
    }
}

// ===================================================================== host
// Which form serves a problem, and its launch: a function of sizes and alignment alone. `general` also
// bounds the workspace, whatever the alignment of a later call.
struct Plan {
    bool rows;
    int v, nv, lg, sets, slabs, slices, chunks, chunk_rows;
    int64_t items;
};
int pow2_at_least(int x) {
    int r = 1;
    while (r < x) r *= 2;
    return r;
}
constexpr int kNvForward = 4, kNvBackward = 2;
// v: elements per vector; nv_most: vectors a lane of the rows form may hold
Plan make_plan(const gdn_group_norm_desc &d, int v, int nv_most) {
    Plan r;
    const int cg = d.C / d.G, cgv = cg / v;
    r.v = v;
    r.lg = std::min(32, pow2_at_least(cgv));
    r.nv = pow2_at_least((int)cdiv64(cgv, r.lg));
    r.rows = d.L == 1 && r.nv <= nv_most;
    r.slabs = r.rows ? 1 : (int)cdiv64(cgv, r.lg);
    r.sets = r.slabs == 1 ? (int)cdiv64(d.G, 32 / r.lg) : d.G * r.slabs;
    r.chunks = 1;
    if (!r.rows) {   // enough chunks of positions to fill the chip, of at least 8 positions
        const int64_t want = cdiv64((int64_t)kSms * kBlocksGeneral * kWarps, std::max<int64_t>(1, (int64_t)d.N * r.sets));
        r.chunks = (int)std::max<int64_t>(1, std::min<int64_t>(want, d.L / 8));
    }
    r.chunk_rows = (int)cdiv64(d.L, r.chunks);
    r.chunks = (int)cdiv64(d.L, std::max(1, r.chunk_rows));
    r.items = (int64_t)d.N * r.chunks;
    const int64_t warps = (int64_t)kSms * kWarps * (!r.rows ? kBlocksGeneral : nv_most == kNvForward ? kBlocksForward : kBlocksBackward);
    r.slices = (int)std::max<int64_t>(1, std::min<int64_t>(warps / r.sets, r.items));
    return r;
}
int vector_of(const gdn_group_norm_desc &d) { return 16 / (int)act_size(d.dtype); }
bool vectors_fit(const gdn_group_norm_desc &d, const void *x, const void *dy, const void *out) {
    const int v = vector_of(d);
    return d.C / d.G % v == 0 && ptr_aligned(x, 16) && ptr_aligned(dy, 16) && ptr_aligned(out, 16) &&
           (d.N <= 1 || d.x_stride_n % v == 0) && (d.L <= 1 || d.x_stride_l % v == 0);
}
size_t stat_bytes(const gdn_group_norm_desc &d, const Plan &pl) {
    return pl.rows ? 0 : align_up((size_t)pl.items * d.G * pl.slabs * sizeof(float2), 256);
}
size_t part_bytes(const gdn_group_norm_desc &d, const Plan &pl) { return align_up((size_t)pl.slices * 2 * d.C * 4, 256); }
// both vector widths, since a call's alignment decides
size_t workspace_need(const gdn_group_norm_desc &d, bool backward) {
    size_t most = 0;
    if ((int64_t)d.N * d.L == 0) return kStatusBytes;
    for (int v : {1, vector_of(d)}) {
        if (d.C / d.G % v) continue;
        const Plan pl = make_plan(d, v, backward ? kNvBackward : kNvForward);
        most = std::max(most, stat_bytes(d, pl) + (backward ? part_bytes(d, pl) : 0));
    }
    return kStatusBytes + most;
}

void apply_plan(NormProblem &p, const Plan &pl, void *ws, bool backward) {
    p.lg = pl.lg;
    p.sets = pl.sets;
    p.slabs = pl.slabs;
    p.slices = pl.slices;
    p.chunks = pl.chunks;
    p.chunk_rows = pl.chunk_rows;
    p.items = pl.items;
    char *w = (char *)ws + kStatusBytes;
    p.stat = (float2 *)w;
    if (backward) p.part = (float *)(w + stat_bytes(p.d, pl));
}
unsigned grid_of(const Plan &pl) { return (unsigned)cdiv64((int64_t)pl.sets * pl.slices, kWarps); }

template <typename T, int V>
cudaError_t run_forward(NormProblem p, void *ws, cudaStream_t s) {
    const Plan pl = make_plan(p.d, V, kNvForward);
    apply_plan(p, pl, ws, false);
    const unsigned grid = grid_of(pl);
    if (pl.rows) {
        if (pl.nv == 1) norm_rows_forward<T, V, 1><<<grid, kThreads, 0, s>>>(p);
        else if (pl.nv == 2) norm_rows_forward<T, V, 2><<<grid, kThreads, 0, s>>>(p);
        else norm_rows_forward<T, V, 4><<<grid, kThreads, 0, s>>>(p);
    } else if (pl.chunks * pl.slabs == 1) {
        norm_stat_kernel<T, V, true><<<grid, kThreads, 0, s>>>(p);
    } else {
        norm_stat_kernel<T, V, false><<<grid, kThreads, 0, s>>>(p);
        norm_apply_kernel<T, V><<<grid, kThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run_backward(NormProblem p, void *ws, cudaStream_t s) {
    const Plan pl = make_plan(p.d, V, kNvBackward);
    apply_plan(p, pl, ws, true);
    const unsigned grid = grid_of(pl);
    if (pl.rows) {
        if (pl.nv == 1) norm_rows_backward<T, V, 1><<<grid, kThreads, 0, s>>>(p);
        else norm_rows_backward<T, V, 2><<<grid, kThreads, 0, s>>>(p);
    } else {
        norm_sums_kernel<T, V><<<grid, kThreads, 0, s>>>(p);
        norm_dx_kernel<T, V><<<grid, kThreads, 0, s>>>(p);
    }
    if (p.dw || p.db) norm_params_kernel<<<(unsigned)cdiv64(p.d.C, 32), 256, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run(const NormProblem &p, bool backward, void *ws, cudaStream_t s) {
    constexpr int V = VecN<T>::value;
    const bool vec = vectors_fit(p.d, p.x, p.dy, backward ? p.dx : p.out);
    if (backward) return vec ? run_backward<T, V>(p, ws, s) : run_backward<T, 1>(p, ws, s);
    return vec ? run_forward<T, V>(p, ws, s) : run_forward<T, 1>(p, ws, s);
}

int run_any(const NormProblem &p, bool backward, void *ws, cudaStream_t s) {
    switch (p.d.dtype) {
    case GDN_F32: return layer_status(run<float>(p, backward, ws, s));
    case GDN_BF16: return layer_status(run<__nv_bfloat16>(p, backward, ws, s));
    default: return layer_status(run<__half>(p, backward, ws, s));
    }
}

int check_desc(const gdn_group_norm_desc *d) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->N < 0 || d->L < 0 || d->C < 1 || d->G < 1 || d->C % d->G != 0) return GDN_ERR_INVALID_ARG;
    if (d->act != GDN_ACT_NONE && d->act != GDN_ACT_SILU) return GDN_ERR_UNSUPPORTED;
    if (!dtype_ok(d->dtype) || (d->weight_dtype != d->dtype && d->weight_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f) || d->x_stride_n < 0 || d->x_stride_l < 0) return GDN_ERR_INVALID_ARG;
    if (d->L > 1 && d->x_stride_l < d->C) return GDN_ERR_INVALID_ARG;
    if (d->C > (1 << 24)) return GDN_ERR_UNSUPPORTED;
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
    *bytes = workspace_need(*d, false);
    return GDN_OK;
}

int gdn_group_norm_backward_workspace_bytes(const gdn_group_norm_desc *d, size_t *bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    *bytes = workspace_need(*d, true);
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
    if ((rc = check_workspace(workspace, workspace_bytes, workspace_need(*d, false))) != GDN_OK) return rc;
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
    return run_any(p, false, workspace, (cudaStream_t)stream);
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
    if ((rc = check_workspace(workspace, workspace_bytes, workspace_need(*d, true))) != GDN_OK) return rc;
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
    if (!any) {   // nothing to sum
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)d->C * 4, (cudaStream_t)stream);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)d->C * 4, (cudaStream_t)stream);
        return layer_status(e);
    }
    return run_any(p, true, workspace, (cudaStream_t)stream);
}

}  // extern "C"
