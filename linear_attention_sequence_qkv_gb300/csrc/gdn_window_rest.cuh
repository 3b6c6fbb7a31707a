// gdn_window_rest.cuh -- the window attention's backward: the queries beyond the window of
// keys that stay visible. A CTA of keys takes the queries within the window; what the sinks'
// keys take beyond is cut into chunks of about the same work, whose sums (fp32, of the sinks'
// rows) a last kernel adds up in order.
#pragma once

#include "gdn_window.cuh"

namespace gdn {

// The queries that the sinks of key tile t still have to take beyond the tile's own CTA: tiles of 2^shift queries from e0 on,
// `tiles` of them for each head
struct SinkRest {
    int e0, tiles;
};
__device__ __forceinline__ SinkRest sink_rest(int Lq, int Lk, int t, int window, int shift) {
    const int64_t past = (int64_t)Lk - Lq, j0 = (int64_t)t * 128, j1 = min(j0 + 127, (int64_t)Lk - 1);
    const int64_t hi = min((int64_t)Lq - 1, j1 + window - 1 - past);
    const int64_t lo = max((int64_t)0, j0 - past) >> shift;
    SinkRest r;
    r.e0 = (int)max(hi < 0 ? (int64_t)0 : (hi >> shift) + 1, lo);
    r.tiles = j0 < Lk ? max(0, (int)(((int64_t)Lq + (1 << shift) - 1) >> shift) - r.e0) : 0;
    return r;
}
__device__ __forceinline__ int rest_chunks(const WindowProblem &p, const WindowSpan &s, int t) {
    const int64_t its = (int64_t)sink_rest(s.Lq, s.Lk, t, p.d.window, p.rest_shift).tiles * (p.d.Hq / p.d.Hk);
    return (int)((its + p.rest_its - 1) / p.rest_its);
}

// How many of the sequence's tiles of sinks have one: the first ones
__device__ __forceinline__ int rest_count(const WindowProblem &p, const WindowSpan &s) {
    int lo = 0, hi = min(p.sink_tiles, max(0, s.Lk - p.d.window) / 128);
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (rest_chunks(p, s, mid) > 0) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// The chunk at `slot`: its sequence, sink tile and number there; false behind the last one. Whole warps call it; bad packed offsets are
// to be looked for before its answer is used.
struct RestAt {
    int n, tile, chunk;
};
__device__ __forceinline__ bool rest_at(const WindowProblem &p, int64_t slot, RestAt &at) {
    if (p.rest_packed) {
        if (slot >= p.rest_tiles[p.rest_all]) return false;
        const int x = warp_upper_index(p.rest_tiles, p.rest_all, slot);
        at.n = warp_upper_index(p.rest_of, p.d.N, x);
        at.tile = x - p.rest_of[at.n];
        at.chunk = (int)(slot - p.rest_tiles[x]);
    } else {
        at.n = (int)(slot / p.rest_per);
        at.chunk = (int)(slot - (int64_t)at.n * p.rest_per), at.tile = 0;
        if (p.sink_tiles > 1) {
            at.tile = warp_upper_index(p.rest_tiles, p.sink_tiles, at.chunk);
            at.chunk -= p.rest_tiles[at.tile];
        }
    }
    return true;
}

// The partial sums' place: [slot][Hk][rows][2][D] fp32, slots of the chunks first, then one for each tile with a rest
template <int D>
__device__ __forceinline__ float *partial_at(const WindowProblem &p, int64_t slot, int hk) {
    return p.partial + (slot * p.d.Hk + hk) * ((int64_t)p.sink_rows * 2 * D);
}
__device__ __forceinline__ int64_t own_slot(const WindowProblem &p, int n, int tile) {
    return p.rest_slots + (p.rest_packed ? p.rest_of[n] : n * p.sink_tiles) + tile;
}

// The sinks' gradients: the CTA's own part and the chunks', in order. Bound by the loads' latency: a thread has one sum and eight
// chunks on their way (one CTA per head and one chunk at a time: 13 us for 14 chunks of 4 sinks of 128 channels, 5 so).
template <typename T, int D>
static __global__ void __launch_bounds__(256) window_sink_sums(const __grid_constant__ WindowProblem p) {
    if (*p.status != GDN_OK) return;
    const gdn_window_attention_desc &d = p.d;
    const int hk = blockIdx.x % d.Hk, x = blockIdx.x / d.Hk;   // of all tiles
    if (p.rest_packed && x >= p.rest_of[d.N]) return;
    const int n = p.rest_packed ? upper_index(p.rest_of, d.N, x) : x / p.sink_tiles, t = x - (p.rest_packed ? p.rest_of[n] : n * p.sink_tiles);
    const bool one = !p.rest_packed && p.sink_tiles == 1;
    const int32_t *table = p.rest_tiles + (p.rest_packed ? x : t);
    const int chunks = one ? p.rest_per : table[1] - table[0];
    if (chunks == 0) return;
    const int64_t slot = (p.rest_packed ? 0 : (int64_t)n * p.rest_per) + (one ? 0 : table[0]);
    const WindowSpan sp = window_span(p, n);
    const int rows = min(min(128, d.sinks - t * 128), sp.Lk - t * 128);
    const float *own = partial_at<D>(p, own_slot(p, n, t), hk);
    for (int x = blockIdx.y * 256 + threadIdx.x; x < rows * 2 * D; x += gridDim.y * 256) {
        const int r = x / (2 * D), b = x / D & 1, c = x % D;
        if (c >= d.d) continue;
        float s = own[x];
        const float *part = partial_at<D>(p, slot, hk) + x;
        const int64_t apart = (int64_t)d.Hk * p.sink_rows * 2 * D;
#pragma unroll 8
        for (int i = 0; i < chunks; ++i) s += part[i * apart];
        ((T *)(b ? p.dv : p.dk))[((sp.k0 + t * 128 + r) * d.Hk + hk) * d.d + c] = from_f<T>(s);
    }
}

template <typename T, int D>
cudaError_t launch_window_sink_sums(const WindowProblem &p, cudaStream_t s) {
    if (p.rest_slots == 0) return cudaSuccess;
    const int64_t blocks = (int64_t)p.rest_all * p.d.Hk;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const unsigned parts = (unsigned)std::min<int64_t>(cdiv64((int64_t)p.sink_rows * 2 * D, 256), 64);
    window_sink_sums<T, D><<<dim3((unsigned)blocks, parts), 256, 0, s>>>(p);
    return cudaGetLastError();
}

// fills the chunks' part of p from the sizes, for tiles of 2^shift queries; the bytes of the partial sums
// (gdn_window_attention.cu)
void window_rest_plan(WindowProblem &p, int shift);
size_t window_partial_bytes(const WindowProblem &p);

}  // namespace gdn
