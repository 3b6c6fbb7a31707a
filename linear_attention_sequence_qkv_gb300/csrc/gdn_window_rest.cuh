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

// The partial sums' place: [slot][Hk][rows][2][D] fp32, slots of the chunks first, then one per sequence and sink tile
template <int D>
__device__ __forceinline__ float *partial_at(const WindowProblem &p, int64_t slot, int hk) {
    return p.partial + (slot * p.d.Hk + hk) * ((int64_t)p.sink_rows * 2 * D);
}

// The sinks' gradients: the CTA's own part and the chunks', in order. Bound by the loads' latency: a thread has one sum and eight
// chunks on their way (one CTA per head and one chunk at a time: 13 us for 14 chunks of 4 sinks of 128 channels, 5 so).
template <typename T, int D>
static __global__ void __launch_bounds__(256) window_sink_sums(const __grid_constant__ WindowProblem p) {
    if (*p.status != GDN_OK) return;
    const gdn_window_attention_desc &d = p.d;
    const int hk = blockIdx.x % d.Hk, n = blockIdx.x / d.Hk / p.sink_tiles, t = blockIdx.x / d.Hk % p.sink_tiles;
    const WindowSpan sp = window_span(p, n);
    const int chunks = rest_chunks(p, sp, t);
    if (chunks == 0) return;
    int64_t slot = p.cu ? p.rest_off[n] : (int64_t)n * p.rest_per;
    for (int x = 0; x < t; ++x) slot += rest_chunks(p, sp, x);
    const int rows = min(min(128, d.sinks - t * 128), sp.Lk - t * 128);
    const float *own = partial_at<D>(p, p.rest_slots + (int64_t)n * p.sink_tiles + t, hk);
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
    const int64_t blocks = (int64_t)p.d.N * p.sink_tiles * p.d.Hk;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const unsigned parts = (unsigned)std::min<int64_t>(cdiv64((int64_t)p.sink_rows * 2 * D, 256), 64);
    window_sink_sums<T, D><<<dim3((unsigned)blocks, parts), 256, 0, s>>>(p);
    return cudaGetLastError();
}

// fills the chunks' part of p from the sizes, for tiles of 2^shift queries; the bytes of the partial sums; the packed sequences' table of chunks
// (gdn_window_attention.cu)
void window_rest_plan(WindowProblem &p, int shift);
size_t window_partial_bytes(const WindowProblem &p);
cudaError_t launch_window_rest_table(const WindowProblem &p, cudaStream_t s);

}  // namespace gdn
