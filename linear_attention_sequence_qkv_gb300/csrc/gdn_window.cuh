// gdn_window.cuh -- what the window attention's kernels share: the problem, the place of a
// sequence, which keys a query sees, and a single query computed by one warp (for the queries
// that see a value which is not finite).
#pragma once

#include <math.h>

#include <type_traits>

#include "gdn_layer_ops.cuh"

namespace gdn {

constexpr int kMostHead = 256;   // channels per head

// fp16 weights that are operands of a product are held times 2^6. Against a row's maximum they are at most 2^8 (it is raised only
// where it grew by more), which leaves room for what rounding adds where scores are huge; and the smallest that count are
// 2^-31 of it (without: 2^-25, and 40000 keys of weight 2.5e-8 beside one of weight 1 added up to nothing).
template <typename T> constexpr float kRaised = std::is_same<T, __half>::value ? 6.0f : 0.0f;

struct WindowProblem {
    gdn_window_attention_desc d;
    const void *q, *k, *v, *out_in, *dout;
    const int32_t *cu, *cuk;    // cuk: the keys' offsets (cu's without their own)
    void *out, *dq, *dk, *dv;
    float *lse;                 // forward: written or null; backward: read
    float *delta;               // [Hq][B*Tq] sums of grad_out * out
    uint32_t *norms;            // backward on tensor cores, fp16 (else null): [2][N][Hk] the largest squared 2-norms of rows of
                                // grad_out (of a group's heads) and of v that are finite, as bits (gdn_window_tc.cuh)
    int32_t *status;
    int32_t *q_tiles, *k_tiles; // packed: [N+1] tiles of the sequences before n, by queries and by keys
    int wait_immediate;
    // the backward: what the sinks' keys take beyond their tile's own CTA (gdn_window_rest.cuh)
    float *partial;             // partial sums of their gradients
    int64_t rest_slots;         // chunks at most
    int rest_shift;             // tiles of 2^rest_shift queries
    int rest_its, rest_per;     // tiles per chunk; chunks per row without packing
    int rest_packed;            // the sequences differ
    int sink_tiles, sink_rows;  // tiles of a sequence's sinks that can have a rest (0: none), rows of their partial sums
    int rest_all;               // such tiles of all sequences, at most
    int32_t *rest_of;           // packed: [N+1] tiles with a rest of the sequences before n
    int32_t *rest_tiles;        // [rest_all (packed, else sink_tiles) + 1] chunks before each of them
};

// A sequence: its first query and key among the flattened tokens, their numbers, and the
// element offsets of its first rows
struct WindowSpan {
    int64_t q0, k0, qoff, koff, voff;
    int Lq, Lk;
};
__device__ __forceinline__ WindowSpan window_span(const WindowProblem &p, int n) {
    const gdn_window_attention_desc &d = p.d;
    WindowSpan s;
    if (p.cu) {
        s.q0 = p.cu[n], s.Lq = p.cu[n + 1] - (int)s.q0;
        s.k0 = p.cuk[n], s.Lk = p.cuk[n + 1] - (int)s.k0;
        s.qoff = s.q0 * d.q_stride_t, s.koff = s.k0 * d.k_stride_t, s.voff = s.k0 * d.v_stride_t;
    } else {
        s.q0 = (int64_t)n * d.Tq, s.Lq = d.Tq;
        s.k0 = (int64_t)n * d.Tk, s.Lk = d.Tk;
        s.qoff = n * d.q_stride_b, s.koff = n * d.k_stride_b, s.voff = n * d.v_stride_b;
    }
    return s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// upper_index for x below arr[N], by a whole warp: 32 entries at a time, so that a CTA begins after two round trips to memory where
// 64 sequences take the search by halves six (32768 tokens in 16 sequences, training step: 2336 -> 2311 us)
__device__ __forceinline__ int warp_upper_index(const int32_t *arr, int N, int64_t x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = N;   // the index is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int64_t at = lo + (int64_t)lane * step;
        const int below = __popc(__ballot_sync(0xffffffffu, at < hi && arr[at < hi ? at : lo] <= x));
        lo += (max(below, 1) - 1) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// A query that sees one key has P = 1 and no scores' gradient; dP - delta of rounded sums is not exactly 0, so its dq is stored
// as 0, and dk of keys that only such queries see (in the sums of other keys it is within their rounding)
__device__ __forceinline__ bool sees_one(int64_t pos, int window, int sinks) { return pos == 0 || (window == 1 && sinks == 0); }
__device__ __forceinline__ bool seen_by_such(int Lk, int window, int sinks) { return Lk == 1 || (window == 1 && sinks == 0); }

// The first key of the window of a query at `pos`, and the number of sinks before it
__device__ __forceinline__ int window_first(int pos, int window) { return pos >= window ? pos - window + 1 : 0; }

// ---------------------------------------------------------------- single rows
// A row's channels over the lanes of a warp: channel 32 c + lane in r[c]
template <typename T, int NC>
__device__ __forceinline__ void row_load(const T *src, int d, int lane, float (&r)[NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c) r[c] = 32 * c + lane < d ? to_f<T>(src[32 * c + lane]) : 0.0f;
}
template <typename T, int NC>
__device__ __forceinline__ void row_store(T *dst, int d, int lane, const float (&r)[NC]) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (32 * c + lane < d) dst[32 * c + lane] = from_f<T>(r[c]);
}
// r . src, src a row of this lane's own
template <typename T, int NC>
__device__ __forceinline__ float row_dot(const float (&r)[NC], const T *src, int d) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
        for (int l = 0; l < 32 && 32 * c + l < d; ++l) s = fmaf(__shfl_sync(0xffffffffu, r[c], l), to_f<T>(src[32 * c + l]), s);
    return s;
}
// acc += w_j src_j over the lanes' rows j, taken in the lanes' order
template <typename T, int NC>
__device__ __forceinline__ void rows_add(float (&acc)[NC], float w, const T *src, int n, int d, int lane) {
    for (int j = 0; j < n; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        const T *sj = (const T *)__shfl_sync(0xffffffffu, (unsigned long long)src, j);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (32 * c + lane < d) acc[c] = fmaf(wj, to_f<T>(sj[32 * c + lane]), acc[c]);
    }
}

// One query at position pos >= 0 of a sequence whose keys start at k, v: out (unrounded) and lse
template <typename T, int NC>
__device__ __noinline__ void row_forward(const T *q, const T *k, const T *v, int64_t kst, int64_t vst, int d, float scale,
                                         int pos, int window, int sinks, int lane, float (&o)[NC], float &lse) {
    float qr[NC];
    row_load<T, NC>(q, d, lane, qr);
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) o[c] = 0.0f;
    const int lo = window_first(pos, window), first = min(sinks, lo), total = first + pos - lo + 1;
    for (int t0 = 0; t0 < total; t0 += 32) {
        const int t = t0 + lane, n = min(32, total - t0);
        const int j = t < first ? t : min(lo + t - first, pos);
        const float s = row_dot<T, NC>(qr, k + j * kst, d) * scale;
        const float x = lane < n ? s : -INFINITY;
        const float mn = fmaxf(m, warp_max(x)), mm = mn == -INFINITY ? 0.0f : mn;
        const float corr = expf(m - mm), w = lane < n ? expf(x - mm) : 0.0f;
        l = l * corr + warp_sum(w);
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c] *= corr;
        rows_add<T, NC>(o, w, v + j * vst, n, d, lane);
        m = mn;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) o[c] /= l;
    lse = m + logf(l);
}

// Status and, for packed sequences, the tiles' tables (tile: rows of a tile of queries, of keys)
cudaError_t launch_window_tables(const WindowProblem &p, int q_tile, int k_tile, cudaStream_t s);
// the CUDA-core kernels, of any type, size and alignment (gdn_window_simt.cu); the backward after tables, delta and chunks
cudaError_t launch_window_forward_simt(const WindowProblem &p, cudaStream_t s);
cudaError_t launch_window_backward_simt(const WindowProblem &p, cudaStream_t s);

}  // namespace gdn
