// gdn_window_tc.cuh -- what the window attention's tensor-core kernels share: tensor maps,
// the tiles of keys that a tile of queries needs, masks, and packed conversions.
#pragma once

#include <type_traits>

#include "gdn_tc.cuh"
#include "gdn_window.cuh"

namespace gdn {

// q, k and v (and grad_out) per head; a batch stride of 0 becomes a map of one row
struct WindowMaps {
    CUtensorMap q, k, v, g;
    int q_rows, k_rows, v_rows;   // 1: batch row n is coordinate n, 0: all rows are one
};

// The tiles of 128 keys that queries at positions [p0, p1] (p0 clamped to 0) need: [0, sinks) and [w0, w1]
struct WindowTiles {
    int ns, w0, w1;
    __device__ __forceinline__ bool empty() const { return w1 < w0; }
    __device__ __forceinline__ bool has(int t) const { return t < ns || (t >= w0 && t <= w1); }
};
__device__ __forceinline__ WindowTiles window_tiles(int p0, int p1, int window, int sinks) {
    WindowTiles r;
    if (p1 < 0) {
        r.ns = 0, r.w0 = 0, r.w1 = -1;
        return r;
    }
    const int lo = window_first(max(p0, 0), window);
    r.w0 = lo >> 7;
    r.w1 = p1 >> 7;
    r.ns = min((int)(((int64_t)min(sinks, lo) + 127) >> 7), r.w0);
    return r;
}
// Whether some query at positions [p0, p1] does not see all keys of tile t
__device__ __forceinline__ bool window_partial(int t, int p0, int p1, int window, int sinks) {
    const int64_t a = (int64_t)t * 128, b = a + 127;
    return b > p0 || (a <= (int64_t)p1 - window && b >= sinks);
}

// the n lowest bits, none for n <= 0, all for n >= 32
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; }

// fp16 ends at 6e-5 (6e-8 with lost bits) and at 65504, which P of many keys and the scores' gradients of a small or a large
// grad_out pass. As operands they are held times powers of two, which the fp32 sums are divided by: P times 2^12 (at most 1, and
// room for what rounding adds where scores are huge), P (dP - delta) times 2^12 f. |dP - delta| is at most
// b = 2 max |dO| max |v|, of rows of the sequence and of the heads that share keys; f is the power of two with f b in [2, 4].
// (dq of 1000 queries and keys of 128 channels, grad_out of size 2^-10 | 2^-16: off by 3.1e-4 | 3.1e-4, without 3.7e-3 | 0.18.)
template <typename T> constexpr int kWeightBits = std::is_same<T, __half>::value ? 12 : 0;
template <typename T> constexpr float kWeightUnit = std::is_same<T, __half>::value ? 1.0f / 4096 : 1.0f;
template <typename T> __device__ __forceinline__ float grad_factor(const WindowProblem &p, int n, int hk) {
    if (!std::is_same<T, __half>::value) return 1.0f;
    const int64_t at = (int64_t)n * p.d.Hk + hk;
    const float b2 = 4.0f * __uint_as_float(p.norms[at]) * __uint_as_float(p.norms[at + (int64_t)p.d.N * p.d.Hk]);
    if (b2 == 0.0f) return 1.0f;
    // b < 2^(x / 2), x the exponent after b2's own: f = 2^-ceil(x / 2) * 4 (b2 is in [2^-94, 2^82]: inputs are fp16 values)
    const int x = (int)(__float_as_uint(b2) >> 23) - 127 + 1;
    return __uint_as_float((uint32_t)(127 - ((x + 1) >> 1) + 2) << 23);
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi) { return Pairs<T>::pack1(make_float2(lo, hi)); }

// The kernels' waits: about a second each, then the CTA gives up (GDN_ERR_DEVICE_TIMEOUT); the first that does tells the others
struct WindowWait {
    volatile int *gave_up;   // shared memory
    bool immediate;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (immediate ? tc::mbar_test_now(bar, parity) : tc::mbar_test(bar, parity)) return true;
        if (*gave_up) return false;
        if (!tc::mbar_wait(bar, parity, immediate)) {
            *gave_up = 1;
            return false;
        }
        return true;
    }
};

// A wait of a whole warp, every lane polling, whose answer is the same for all; for two or three barriers the tests' round trips
// overlap (about 100 cycles each, which the warp that issues the products has to wait out)
__device__ __forceinline__ bool warp_wait(const WindowWait &wait, uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
}
__device__ __forceinline__ bool warp_wait2(const WindowWait &wait, uint64_t *b1, uint32_t p1, uint64_t *b2, uint32_t p2) {
    bool ok = wait.immediate ? tc::mbar_test2<true>(b1, p1, b2, p2) : tc::mbar_test2<false>(b1, p1, b2, p2);
    if (!ok) ok = wait(b1, p1) && wait(b2, p2);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait3(const WindowWait &wait, uint64_t *b1, uint32_t p1, uint64_t *b2, uint32_t p2, uint64_t *b3, uint32_t p3) {
    bool ok = wait.immediate ? tc::mbar_test3<true>(b1, p1, b2, p2, b3, p3) : tc::mbar_test3<false>(b1, p1, b2, p2, b3, p3);
    if (!ok) ok = wait(b1, p1) && wait(b2, p2) && wait(b3, p3);
    return __all_sync(0xffffffffu, ok);
}
// a warp's arrival, after what its lanes wrote to tensor or shared memory
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    tc::fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}
// the first lane's value, known to be the warp's
__device__ __forceinline__ int of_warp(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// whether sizes and strides, and with them the pointers, suit the tensor-core kernels
bool window_tc_fits(const gdn_window_attention_desc &d);
bool window_tc_supports(const WindowProblem &p);
cudaError_t launch_window_forward_tc(const WindowProblem &p, cudaStream_t s);
bool window_head_map(CUtensorMap *m, const gdn_window_attention_desc &d, const void *base, int heads, int tokens, int64_t sb, int64_t st,
                     int *rows, uint32_t box);
// after delta, with the chunks planned
cudaError_t launch_window_backward_tc(const WindowProblem &p, cudaStream_t s);
// its dq, where two heads at once are faster; `wide`: maps of 128 rows
bool window_dq_pairs(const gdn_window_attention_desc &d);
cudaError_t launch_window_dq_pair(const WindowMaps &wide, const WindowProblem &p, cudaStream_t s);

}  // namespace gdn
