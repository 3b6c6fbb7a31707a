// gdn_window_simt.cu -- the window attention on CUDA cores (include/gdn.h): fp32, wide heads
// (up to 256 channels), odd widths and unaligned rows. fp32 sums of fp32 products throughout.
//
// A CTA of 256 threads keeps 64 rows in shared memory as fp32 and walks over tiles of the
// other side: forward 64 queries over 64 keys, dq 64 queries over 32 keys, dk and dv 64 keys
// over 32 queries of each head of the group. Thread (ty, tx) of 16 x 16 computes the scores
// of rows 4 ty .. 4 ty + 3 with columns tx, tx + 16, .. (a row's pitch of four words more than
// a multiple of 32 spreads these over the banks), hands P (dS) over through shared memory and
// owns channels 4 tx + 64 c of its rows' sums. Bound by shared memory and FMA issue; small calls
// by latency: 2 x 100 tokens of 6 heads of 64 in fp32, forward 23 us, gradients 30 us
// under a profiler.
#include <algorithm>

#include "gdn_window_rest.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;    // rows that stay
constexpr int kWalk = 32;    // rows of a step of the backward
constexpr int kMostCut = 8;  // tiles of 64 keys that a mask cuts: 2 where windows begin, 2 at their end, 1 with the last sink

template <typename T> __device__ __forceinline__ bool is_wide(const void *base, int64_t stride, int d) {
    return ((uintptr_t)base % 16) == 0 && stride * sizeof(T) % 16 == 0 && d * sizeof(T) % 16 == 0;
}

// `rows` rows of d channels at `src` into [n][D + 4] fp32, zeros behind them. CHECK: values that are not finite are zeroed
// too and noted, a bit for each row.
template <typename T, int D, bool CHECK>
__device__ __forceinline__ void load_rows(float *dst, const T *src, int64_t stride, int n, int rows, int d, bool wide, uint32_t *bad) {
    constexpr int V = 16 / sizeof(T), kPitch = D + 4;
    auto put = [&](int r, float x) {
        if (CHECK && !(fabsf(x) <= 3.402823466e38f)) {
            atomicOr(&bad[r >> 5], 1u << (r & 31));
            return 0.0f;
        }
        return x;
    };
    if (wide) {
        for (int x = threadIdx.x; x < n * (D / V); x += kThreads) {
            const int r = x / (D / V), c = x % (D / V) * V;
            Vec16<T> v;
            v.u = make_uint4(0, 0, 0, 0);
            if (r < rows && c < d) v.u = *(const uint4 *)(src + r * stride + c);
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *(float4 *)(dst + r * kPitch + c + e) =
                    make_float4(put(r, to_f<T>(v.e[e])), put(r, to_f<T>(v.e[e + 1])), put(r, to_f<T>(v.e[e + 2])), put(r, to_f<T>(v.e[e + 3])));
        }
    } else {
        for (int x = threadIdx.x; x < n * D; x += kThreads) {
            const int r = x / D, c = x % D;
            dst[r * kPitch + c] = r < rows && c < d ? put(r, to_f<T>(src[r * stride + c])) : 0.0f;
        }
    }
}

// s[i][j] = a row 4 ty + i . b row tx + 16 j
template <int D, int NJ>
__device__ __forceinline__ void tile_dots(const float *a, const float *b, int ty, int tx, float (&s)[4][NJ]) {
    constexpr int kPitch = D + 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) s[i][j] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[4], y[NJ];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *(const float4 *)(a + (4 * ty + i) * kPitch + c);
#pragma unroll
        for (int j = 0; j < NJ; ++j) y[j] = *(const float4 *)(b + (tx + 16 * j) * kPitch + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]), s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]), s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
    }
}
// o[i] += w row 4 ty + i (n wide, pitch wp) times b, channels 4 tx + 64 c
template <int D>
__device__ __forceinline__ void tile_add(const float *w, int wp, const float *b, int n, int ty, int tx, float4 (&o)[4][D / 64]) {
    constexpr int kPitch = D + 4;
#pragma unroll 2
    for (int k = 0; k < n; k += 4) {
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *(const float4 *)(w + (4 * ty + i) * wp + k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const float4 y = *(const float4 *)(b + (k + e) * kPitch + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
                    o[i][c].x = fmaf(f, y.x, o[i][c].x), o[i][c].y = fmaf(f, y.y, o[i][c].y);
                    o[i][c].z = fmaf(f, y.z, o[i][c].z), o[i][c].w = fmaf(f, y.w, o[i][c].w);
                }
            }
    }
}
template <typename T, int D>
__device__ __forceinline__ void store_rows(T *dst, int64_t stride, int d, int ty, int tx, int from, int to, const float4 (&o)[4][D / 64], const float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r < from || r >= to) continue;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            const float v[4] = {o[i][c].x * f[i], o[i][c].y * f[i], o[i][c].z * f[i], o[i][c].w * f[i]};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * tx + 64 * c + e < d) dst[r * stride + 4 * tx + 64 * c + e] = from_f<T>(v[e]);
        }
    }
}

// A CTA's sequence and tile of kRows queries (or keys): false where there is none
__device__ __forceinline__ bool tile_of(const WindowProblem &p, const int32_t *table, int64_t slot, int T, int &n, int &tile, int &tiles) {
    if (p.cu) {
        if (slot >= table[p.d.N]) return false;
        n = warp_upper_index(table, p.d.N, slot);
        tile = (int)(slot - table[n]);
        tiles = table[n + 1] - table[n];
    } else {
        tiles = (T + kRows - 1) / kRows;
        n = (int)(slot / tiles);
        tile = (int)(slot - (int64_t)n * tiles);
    }
    return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_forward_simt(const __grid_constant__ WindowProblem p) {
    constexpr int kPitch = D + 4;
    extern __shared__ float sm[];
    float *Q = sm, *K = Q + kRows * kPitch, *V = K + 64 * kPitch, *P = K;   // P over K once the scores are there
    __shared__ uint32_t bad[kMostCut][2];
    __shared__ int any_bad;
    if (*p.status != GDN_OK) return;
    const gdn_window_attention_desc &d = p.d;
    const int h = (int)(blockIdx.x % d.Hq), hk = h / (d.Hq / d.Hk);
    int n, tile, tiles;
    if (!tile_of(p, p.q_tiles, blockIdx.x / d.Hq, d.Tq, n, tile, tiles)) return;
    const int i0 = (tiles - 1 - tile) * kRows;   // later queries, which see the most, first
    const WindowSpan sp = window_span(p, n);
    const int past = sp.Lk - sp.Lq, rows = min(kRows, sp.Lq - i0);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const T *k = (const T *)p.k + sp.koff + (int64_t)hk * d.d, *v = (const T *)p.v + sp.voff + (int64_t)hk * d.d;
    const T *q = (const T *)p.q + sp.qoff + i0 * d.q_stride_t + (int64_t)h * d.d;
    const bool kw = is_wide<T>(k, d.k_stride_t, d.d), vw = is_wide<T>(v, d.v_stride_t, d.d);
    load_rows<T, D, false>(Q, q, d.q_stride_t, kRows, rows, d.d, is_wide<T>(q, d.q_stride_t, d.d), nullptr);
    if (tid == 0) any_bad = 0;
    if (tid < 2 * kMostCut) (&bad[0][0])[tid] = 0;
    const int p0 = max(past + i0, 0), p1 = past + i0 + rows - 1;
    const int lo = window_first(p0, d.window);
    const int w0 = lo >> 6, ns = p1 < 0 ? 0 : min((int)(((int64_t)min(d.sinks, lo) + 63) >> 6), w0), count = p1 < 0 ? 0 : ns + (p1 >> 6) - w0 + 1;
    auto tile_at = [&](int u) { return u < ns ? u : w0 + u - ns; };
    auto is_cut = [&](int t) {
        const int64_t a = (int64_t)t * 64, b = a + 63;
        return b > p0 || (a <= (int64_t)p1 - d.window && b >= d.sinks);
    };
    const float c = d.scale * 1.4426950408889634f;
    float m[4], l[4];
    float4 o[4][D / 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY, l[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) o[i][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    int cuts = 0;
    for (int u = 0; u < count; ++u) {
        const int t = tile_at(u), left = min(64, sp.Lk - t * 64);
        const bool cut = is_cut(t);
        __syncthreads();
        load_rows<T, D, false>(K, k + (int64_t)t * 64 * d.k_stride_t, d.k_stride_t, 64, left, d.d, kw, nullptr);
        if (cut) load_rows<T, D, true>(V, v + (int64_t)t * 64 * d.v_stride_t, d.v_stride_t, 64, left, d.d, vw, bad[min(cuts, kMostCut - 1)]);
        else load_rows<T, D, false>(V, v + (int64_t)t * 64 * d.v_stride_t, d.v_stride_t, 64, left, d.d, vw, nullptr);
        cuts += cut;
        __syncthreads();
        float s[4][4];
        tile_dots<D, 4>(Q, K, ty, tx, s);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t pos = (int64_t)past + i0 + 4 * ty + i;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t key = (int64_t)t * 64 + tx + 16 * j;
                if (!(key <= pos && (pos - key < d.window || key < d.sinks))) s[i][j] = -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float mn = fmaxf(m[i], top), mm = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2f((m[i] - mm) * c);
            m[i] = mn;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w = exp2f((s[i][j] - mm) * c);
                sum += w;
                P[(4 * ty + i) * 68 + tx + 16 * j] = w;
            }
#pragma unroll
            for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) o[i][e].x *= f, o[i][e].y *= f, o[i][e].z *= f, o[i][e].w *= f;
        }
        __syncthreads();
        tile_add<D>(P, 68, V, 64, ty, tx, o);
    }
    float f[4];
    const int64_t tok0 = sp.q0 + i0, ntok = (int64_t)d.B * d.Tq;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        const bool none = past + i0 + r < 0;
        f[i] = none ? 0.0f : 1.0f / l[i];
        if (none)
#pragma unroll
            for (int e = 0; e < D / 64; ++e) o[i][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p.lse && tx == 0 && r < rows) p.lse[h * ntok + tok0 + r] = none ? -INFINITY : (m[i] * c + log2f(l[i])) * 0.6931471805599453f;
    }
    T *out = (T *)p.out + (tok0 * d.Hq + h) * d.d;
    store_rows<T, D>(out, (int64_t)d.Hq * d.d, d.d, ty, tx, 0, rows, o, f);
    // queries that see a value which is not finite, on their own
    if (tid < 2 * kMostCut && (&bad[0][0])[tid]) any_bad = 1;
    __syncthreads();
    if (!any_bad) return;
    for (int r = tid >> 5; r < rows; r += kThreads / 32) {
        const int pos = past + i0 + r;
        if (pos < 0) continue;
        bool dirty = false;
        int x = 0;
        for (int u = 0; u < count; ++u) {
            if (!is_cut(tile_at(u))) continue;
            for (int w = 0; w < 2; ++w)
                for (uint32_t bits = bad[x][w]; bits; bits &= bits - 1) {
                    const int j = tile_at(u) * 64 + 32 * w + __ffs(bits) - 1;
                    dirty |= j <= pos && (pos - j < d.window || j < d.sinks);
                }
            x = min(x + 1, kMostCut - 1);
        }
        if (!dirty) continue;
        float row[D / 32], ls;
        row_forward<T, D / 32>(q + r * d.q_stride_t, k, v, d.k_stride_t, d.v_stride_t, d.d, d.scale, pos, d.window, d.sinks, tid & 31, row, ls);
        row_store<T, D / 32>(out + (int64_t)r * d.Hq * d.d, d.d, tid & 31, row);
        if (p.lse && (tid & 31) == 0) p.lse[h * ntok + tok0 + r] = ls;
    }
}

// The part of a backward CTA that has a tile of queries
template <typename T, int D>
__device__ __forceinline__ void dq_tile(const WindowProblem &p, float *sm, int64_t block) {
    constexpr int kPitch = D + 4, kW = kWalk + 4;
    float *Q = sm, *G = Q + kRows * kPitch, *K = G + kRows * kPitch, *V = K + kWalk * kPitch, *S = V + kWalk * kPitch;
    const gdn_window_attention_desc &d = p.d;
    const int h = (int)(block % d.Hq), hk = h / (d.Hq / d.Hk);
    int n, tile, tiles;
    if (!tile_of(p, p.q_tiles, block / d.Hq, d.Tq, n, tile, tiles)) return;
    const int i0 = (tiles - 1 - tile) * kRows;
    const WindowSpan sp = window_span(p, n);
    const int past = sp.Lk - sp.Lq, rows = min(kRows, sp.Lq - i0);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int64_t tok0 = sp.q0 + i0, ntok = (int64_t)d.B * d.Tq, gst = (int64_t)d.Hq * d.d;
    const T *k = (const T *)p.k + sp.koff + (int64_t)hk * d.d, *v = (const T *)p.v + sp.voff + (int64_t)hk * d.d;
    const T *q = (const T *)p.q + sp.qoff + i0 * d.q_stride_t + (int64_t)h * d.d, *g = (const T *)p.dout + (tok0 * d.Hq + h) * d.d;
    const bool kw = is_wide<T>(k, d.k_stride_t, d.d), vw = is_wide<T>(v, d.v_stride_t, d.d);
    load_rows<T, D, false>(Q, q, d.q_stride_t, kRows, rows, d.d, is_wide<T>(q, d.q_stride_t, d.d), nullptr);
    load_rows<T, D, false>(G, g, gst, kRows, rows, d.d, is_wide<T>(g, gst, d.d), nullptr);
    const float c = d.scale * 1.4426950408889634f;
    float lse[4], delta[4];
    float4 o[4][D / 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool in = 4 * ty + i < rows;
        lse[i] = in ? p.lse[h * ntok + tok0 + 4 * ty + i] * 1.4426950408889634f : 0.0f;
        delta[i] = in ? p.delta[h * ntok + tok0 + 4 * ty + i] : 0.0f;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) o[i][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    const int p1 = past + i0 + rows - 1, lo = window_first(max(past + i0, 0), d.window);
    const int w0 = lo / kWalk, ns = p1 < 0 ? 0 : min((int)(((int64_t)min(d.sinks, lo) + kWalk - 1) / kWalk), w0),
              count = p1 < 0 ? 0 : ns + p1 / kWalk - w0 + 1;
    for (int u = 0; u < count; ++u) {
        const int t = u < ns ? u : w0 + u - ns, left = min(kWalk, sp.Lk - t * kWalk);
        __syncthreads();
        load_rows<T, D, false>(K, k + (int64_t)t * kWalk * d.k_stride_t, d.k_stride_t, kWalk, left, d.d, kw, nullptr);
        load_rows<T, D, false>(V, v + (int64_t)t * kWalk * d.v_stride_t, d.v_stride_t, kWalk, left, d.d, vw, nullptr);
        __syncthreads();
        float s[4][2], dp[4][2];
        tile_dots<D, 2>(Q, K, ty, tx, s);
        tile_dots<D, 2>(G, V, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t pos = (int64_t)past + i0 + 4 * ty + i, key = (int64_t)t * kWalk + tx + 16 * j;
                const bool see = key <= pos && (pos - key < d.window || key < d.sinks);
                S[(4 * ty + i) * kW + tx + 16 * j] = see ? exp2f(fmaf(s[i][j], c, -lse[i])) * (dp[i][j] - delta[i]) * d.scale : 0.0f;
            }
        __syncthreads();
        tile_add<D>(S, kW, K, kWalk, ty, tx, o);
    }
    float one[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) one[i] = sees_one((int64_t)past + i0 + 4 * ty + i, d.window, d.sinks) ? 0.0f : 1.0f;
    store_rows<T, D>((T *)p.dq + (tok0 * d.Hq + h) * d.d, gst, d.d, ty, tx, 0, rows, o, one);
}

__device__ __forceinline__ float4 of_rank(const float *own, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(own)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

// The part that has a tile of keys, or a chunk of the sinks' rest: the `splits` CTAs of a cluster take every splits-th step,
// and their sums are added up in the ranks' order. All of a cluster have the same block.
template <typename T, int D>
__device__ __forceinline__ void dkv_tile(const WindowProblem &p, float *sm, int64_t block_of_all, int64_t rest_blocks, int rank, int splits) {
    constexpr int kPitch = D + 4, kW = kWalk + 4;
    float *K = sm, *V = K + kRows * kPitch, *Q = V + kRows * kPitch, *G = Q + kWalk * kPitch, *P = G + kWalk * kPitch, *S = P + kRows * kW;
    __shared__ float lse[kWalk], delta[kWalk];
    const gdn_window_attention_desc &d = p.d;
    const bool rest = block_of_all < rest_blocks;
    const int64_t block = rest ? block_of_all : block_of_all - rest_blocks;
    const int hk = (int)(block % d.Hk), group = d.Hq / d.Hk;
    int n, row0, tile = 0, chunk = 0;
    int64_t slot = block / d.Hk;
    if (rest) {   // a chunk of a sink tile of 128 keys, and which half of it
        const int half = (int)(slot & 1);
        slot >>= 1;
        RestAt at;
        if (!rest_at(p, slot, at)) return;
        n = at.n, tile = at.tile, chunk = at.chunk;
        row0 = tile * 128 + 64 * half;
        if (row0 >= min(d.sinks, window_span(p, n).Lk)) return;
    } else {
        int tiles;
        if (!tile_of(p, p.k_tiles, slot, d.Tk, n, row0, tiles)) return;
        row0 *= kRows;
        tile = row0 >> 7;
    }
    const WindowSpan sp = window_span(p, n);
    const int past = sp.Lk - sp.Lq, rows = min(kRows, sp.Lk - row0);
    // the queries it walks over, in tiles of 64: the window's (with sinks among the keys those of the whole sink tile's, where
    // its chunks begin), or a chunk of the rest
    int64_t first = 0, per_head = 0, it0 = 0, it1;
    if (rest) {
        const SinkRest r = sink_rest(sp.Lq, sp.Lk, tile, d.window, p.rest_shift);
        first = r.e0, per_head = r.tiles;
        it0 = (int64_t)chunk * p.rest_its, it1 = min(it0 + p.rest_its, per_head * group);
    } else {
        const int64_t last = row0 < d.sinks ? min((int64_t)tile * 128 + 127, (int64_t)sp.Lk - 1) : (int64_t)row0 + rows - 1;
        const int64_t lo = max((int64_t)0, (int64_t)row0 - past), hi = min((int64_t)sp.Lq - 1, last + d.window - 1 - past);
        if (hi >= lo) first = lo >> 6, per_head = (hi >> 6) - first + 1;
        it1 = per_head * group;
    }
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int64_t ntok = (int64_t)d.B * d.Tq, gst = (int64_t)d.Hq * d.d;
    const T *k = (const T *)p.k + sp.koff + row0 * d.k_stride_t + (int64_t)hk * d.d, *v = (const T *)p.v + sp.voff + row0 * d.v_stride_t + (int64_t)hk * d.d;
    load_rows<T, D, false>(K, k, d.k_stride_t, kRows, rows, d.d, is_wide<T>(k, d.k_stride_t, d.d), nullptr);
    load_rows<T, D, false>(V, v, d.v_stride_t, kRows, rows, d.d, is_wide<T>(v, d.v_stride_t, d.d), nullptr);
    const float c = d.scale * 1.4426950408889634f;
    float4 dk[4][D / 64], dv[4][D / 64];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < D / 64; ++e) dk[i][e] = dv[i][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t it = 2 * it0 + rank; it < 2 * it1; it += splits) {   // halves of 32 queries
        const int h = hk * group + (int)((it >> 1) / per_head);
        const int i0 = (int)(first + (it >> 1) % per_head) * 64 + (it & 1) * kWalk, left = min(kWalk, sp.Lq - i0);
        if (left <= 0) continue;
        const T *q = (const T *)p.q + sp.qoff + i0 * d.q_stride_t + (int64_t)h * d.d, *g = (const T *)p.dout + ((sp.q0 + i0) * d.Hq + h) * d.d;
        __syncthreads();
        load_rows<T, D, false>(Q, q, d.q_stride_t, kWalk, left, d.d, is_wide<T>(q, d.q_stride_t, d.d), nullptr);
        load_rows<T, D, false>(G, g, gst, kWalk, left, d.d, is_wide<T>(g, gst, d.d), nullptr);
        if (tid < kWalk) {
            const int64_t at = h * ntok + sp.q0 + i0 + tid;
            lse[tid] = tid < left ? p.lse[at] * 1.4426950408889634f : 0.0f;
            delta[tid] = tid < left ? p.delta[at] : 0.0f;
        }
        __syncthreads();
        float s[4][2], dp[4][2];
        tile_dots<D, 2>(K, Q, ty, tx, s);
        tile_dots<D, 2>(V, G, ty, tx, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int x = tx + 16 * j;
                const int64_t pos = (int64_t)past + i0 + x, key = (int64_t)row0 + 4 * ty + i;
                const bool see = x < left && key <= pos && (pos - key < d.window || key < d.sinks);
                const float w = see ? exp2f(fmaf(s[i][j], c, -lse[x])) : 0.0f;
                P[(4 * ty + i) * kW + x] = w;
                S[(4 * ty + i) * kW + x] = see ? w * (dp[i][j] - delta[x]) * d.scale : 0.0f;
            }
        __syncthreads();
        tile_add<D>(P, kW, G, kWalk, ty, tx, dv);
        tile_add<D>(S, kW, Q, kWalk, ty, tx, dk);
    }
    if (splits > 1) {   // K and V make room for the sums; a rank has the rows r with r / 4 % splits == rank in the end
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                *(float4 *)(K + (4 * ty + i) * kPitch + 4 * tx + 64 * e) = dk[i][e];
                *(float4 *)(V + (4 * ty + i) * kPitch + 4 * tx + 64 * e) = dv[i][e];
            }
        cluster_sync();
        if (ty % splits == rank) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
                    for (int x = 0; x < splits; ++x) {
                        const float4 u = of_rank(K + (4 * ty + i) * kPitch + 4 * tx + 64 * e, x), w = of_rank(V + (4 * ty + i) * kPitch + 4 * tx + 64 * e, x);
                        a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
                        b.x += w.x, b.y += w.y, b.z += w.z, b.w += w.w;
                    }
                    dk[i][e] = a, dv[i][e] = b;
                }
        }
        cluster_sync();   // no CTA leaves while another reads its sums
        if (ty % splits != rank) return;
    }
    // rows of sinks whose sum has other parts stay in fp32
    const int apart = rest ? kRows : row0 < d.sinks && rest_chunks(p, sp, tile) > 0 ? min(kRows, d.sinks - row0) : 0;
    const int64_t part = !apart ? 0 : rest ? slot : own_slot(p, n, tile);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i, in_tile = row0 + r - tile * 128;
        if (r >= min(apart, min(rows, d.sinks - row0))) continue;
        float *to = partial_at<D>(p, part, hk) + (int64_t)in_tile * 2 * D;
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
            *(float4 *)(to + 4 * tx + 64 * e) = dk[i][e];
            *(float4 *)(to + D + 4 * tx + 64 * e) = dv[i][e];
        }
    }
    const float one[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    const int64_t at = ((sp.k0 + row0) * d.Hk + hk) * d.d, st = (int64_t)d.Hk * d.d;
    const float k1 = seen_by_such(sp.Lk, d.window, d.sinks) ? 0.0f : 1.0f, of_k[4] = {k1, k1, k1, k1};
    store_rows<T, D>((T *)p.dk + at, st, d.d, ty, tx, apart, rows, dk, of_k);
    store_rows<T, D>((T *)p.dv + at, st, d.d, ty, tx, apart, rows, dv, one);
}

// Clusters of tiles of keys first (the longer ones), then tiles of queries
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) window_backward_simt(const __grid_constant__ WindowProblem p, int64_t key_blocks, int64_t rest_blocks, int64_t query_blocks,
                                                                  int splits) {
    extern __shared__ float sm[];
    if (*p.status != GDN_OK) return;
    const int64_t cluster = blockIdx.x / splits;
    const int rank = blockIdx.x % splits;
    if (cluster < key_blocks) dkv_tile<T, D>(p, sm, cluster, rest_blocks, rank, splits);
    else if (blockIdx.x - key_blocks * splits < query_blocks) dq_tile<T, D>(p, sm, blockIdx.x - key_blocks * splits);
}

template <typename K, typename... A>
cudaError_t go(K kernel, int64_t blocks, int cluster, size_t smem, cudaStream_t s, A... args) {
    if (blocks <= 0) return cudaSuccess;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const cudaError_t e = allow_shared(kernel, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
int64_t tiles_of(const WindowProblem &p, int T) { return p.cu ? cdiv64(T, kRows) + p.d.N : (int64_t)p.d.B * cdiv64(T, kRows); }

template <typename T, int D>
cudaError_t forward(const WindowProblem &p, cudaStream_t s) {
    return go(window_forward_simt<T, D>, p.d.Tq ? tiles_of(p, p.d.Tq) * p.d.Hq : 0, 1, (size_t)3 * 64 * (D + 4) * 4, s, p);
}
template <typename T, int D>
cudaError_t backward(const WindowProblem &p, cudaStream_t s) {
    const size_t smem = ((size_t)(2 * kRows + 2 * kWalk) * (D + 4) + 2 * kRows * (kWalk + 4)) * 4;
    const int64_t rest = 2 * p.rest_slots * p.d.Hk, keys = p.d.Tk ? tiles_of(p, p.d.Tk) * p.d.Hk + rest : 0;
    const int64_t queries = p.d.Tq ? tiles_of(p, p.d.Tq) * p.d.Hq : 0;
    // few tiles of keys: CTAs share one, as long as each has a few steps and all fit the SMs at once
    const int64_t steps = std::min<int64_t>(cdiv64(p.d.Tq, kWalk), cdiv64((int64_t)p.d.window + kRows, kWalk) + 1) * (p.d.Hq / p.d.Hk);
    int splits = 1;
    while (splits < 8 && keys * splits * 2 + queries <= 2 * kSms && steps >= 4 * splits) splits *= 2;
    const cudaError_t e = go(window_backward_simt<T, D>, keys * splits + align_up((size_t)queries, splits), splits, smem, s, p, keys, rest, queries, splits);
    if (e != cudaSuccess) return e;
    return launch_window_sink_sums<T, D>(p, s);
}
template <typename T>
cudaError_t forward_of(const WindowProblem &p, cudaStream_t s) {
    return p.d.d <= 64 ? forward<T, 64>(p, s) : p.d.d <= 128 ? forward<T, 128>(p, s) : forward<T, 256>(p, s);
}
template <typename T>
cudaError_t backward_of(const WindowProblem &p, cudaStream_t s) {
    return p.d.d <= 64 ? backward<T, 64>(p, s) : p.d.d <= 128 ? backward<T, 128>(p, s) : backward<T, 256>(p, s);
}

}  // namespace

cudaError_t launch_window_forward_simt(const WindowProblem &p, cudaStream_t s) {
    const cudaError_t e = launch_window_tables(p, kRows, kRows, s);
    if (e != cudaSuccess) return e;
    switch (p.d.dtype) {
    case GDN_F32: return forward_of<float>(p, s);
    case GDN_BF16: return forward_of<__nv_bfloat16>(p, s);
    default: return forward_of<__half>(p, s);
    }
}
cudaError_t launch_window_backward_simt(const WindowProblem &p, cudaStream_t s) {
    switch (p.d.dtype) {
    case GDN_F32: return backward_of<float>(p, s);
    case GDN_BF16: return backward_of<__nv_bfloat16>(p, s);
    default: return backward_of<__half>(p, s);
    }
}

}  // namespace gdn
