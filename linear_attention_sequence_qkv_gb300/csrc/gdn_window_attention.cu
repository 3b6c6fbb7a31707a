// gdn_window_attention.cu -- causal attention over a window of recent tokens and a few
// first ones (include/gdn.h): the C entry points of its forward and backward, the check
// of packed offsets, and the sums of grad_out * out that the backward starts from.
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "gdn_window_rest.cuh"
#include "gdn_window_tc.cuh"

namespace gdn {
namespace {

// The sum of c over the threads before this one, and over all (the next call may follow at once; sums begins as zeros)
__device__ __forceinline__ int before_thread(int c, int32_t (&sums)[32], int &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    all = __shfl_sync(0xffffffffu, s, 31);
    const int ahead = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
    __syncthreads();
    return (warp ? ahead : 0) + x - c;
}

// Packed offsets checked, and the tiles of the sequences before each one counted
__global__ void __launch_bounds__(1024) window_tables_kernel(const __grid_constant__ WindowProblem p, int q_tile, int k_tile) {
    const gdn_window_attention_desc &d = p.d;
    if (p.norms)
        for (int64_t i = threadIdx.x; i < 2 * (int64_t)d.N * d.Hk; i += blockDim.x) p.norms[i] = 0;
    if (p.cu == nullptr) {
        if (threadIdx.x == 0) *p.status = GDN_OK;
        return;
    }
    bool ok = seqlens_ok(p.cu, d.N, d.Tq);
    if (p.cuk != p.cu) ok = seqlens_ok(p.cuk, d.N, d.Tk) && ok;
    if (threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    __shared__ int32_t sums[32];
    if (threadIdx.x < 32) sums[threadIdx.x] = 0;
    __syncthreads();
    for (int which = 0; which < 2; ++which) {
        const int32_t *cu = which ? p.cuk : p.cu;
        int32_t *to = which ? p.k_tiles : p.q_tiles;
        const int tile = which ? k_tile : q_tile;
        if (!to) continue;
        int before = 0, all;
        for (int base = 0; base < d.N; base += blockDim.x) {
            const int n = base + threadIdx.x;
            const int c = ok && n < d.N ? (int)(((int64_t)cu[n + 1] - cu[n] + tile - 1) / tile) : 0;
            const int at = before + before_thread(c, sums, all);
            if (n < d.N) to[n] = at;
            before += all;
        }
        if (threadIdx.x == 0) to[d.N] = before;
    }
}

// fp16's norms (gdn_window_tc.cuh): the largest squared norms of a CTA's rows, per sequence and head of keys, go through shared
// memory where its range of tokens has few of them, then into the call's words. A word is read before it is raised, so that few
// CTAs end in atomics; the largest does not depend on their order. Rows that are not finite are passed over.
constexpr int kTable = 1024;
constexpr float kFinite = 3.402823466e38f;
struct RowNorms {
    uint32_t *words, *table;    // the call's [N][Hk], the CTA's
    const int32_t *cu;
    int N, T, Hk, n0, n1;       // the sequences of the CTA's tokens
    // all threads call it, as they do flush
    __device__ __forceinline__ RowNorms(const WindowProblem &p, bool is_v, uint32_t *sm, int64_t first, int64_t last)
        : words(p.norms + (is_v ? (int64_t)p.d.N * p.d.Hk : 0)), table(sm), cu(p.cu ? (is_v ? p.cuk : p.cu) : nullptr), N(p.d.N),
          T(is_v ? p.d.Tk : p.d.Tq), Hk(p.d.Hk) {
        n0 = of(first, 0, N), n1 = of(last, n0, N);
        if ((int64_t)(n1 - n0 + 1) * Hk > kTable) table = nullptr;
        else
            for (int x = threadIdx.x; x < (n1 - n0 + 1) * Hk; x += blockDim.x) table[x] = 0;
        __syncthreads();
    }
    __device__ __forceinline__ int of(int64_t tok, int lo, int hi) const { return cu ? lo + upper_index(cu + lo, hi - lo, tok) : (int)(tok / T); }
    __device__ __forceinline__ void raise(uint32_t *to, uint32_t bits) const {
        if (bits > __ldcg(to)) atomicMax(to, bits);
    }
    __device__ __forceinline__ void add(int64_t tok, int hk, float squared) const {
        if (!(squared <= kFinite)) return;
        const int n = n0 == n1 ? n0 : of(tok, n0, n1 + 1);
        if (table) atomicMax(&table[(n - n0) * Hk + hk], __float_as_uint(squared));
        else raise(words + (int64_t)n * Hk + hk, __float_as_uint(squared));
    }
    __device__ __forceinline__ void flush() const {
        __syncthreads();
        if (table)
            for (int x = threadIdx.x; x < (n1 - n0 + 1) * Hk; x += blockDim.x)
                if (table[x]) raise(words + (int64_t)n0 * Hk + x, table[x]);
        __syncthreads();
    }
};

// A row's token and head, a fixed number of rows on at a time (64-bit divisions would be most of a row's instructions)
struct RowAt {
    int64_t tok, by_tok;
    int head, by_head, heads;
    __device__ __forceinline__ RowAt(int64_t i, int step, int heads_) : tok(i / heads_), by_tok(step / heads_), by_head(step % heads_), heads(heads_) {
        head = (int)(i - tok * heads);
    }
    __device__ __forceinline__ void next() {
        tok += by_tok, head += by_head;
        if (head >= heads) head -= heads, ++tok;
    }
};

// delta = sum of grad_out * out per query and head, 32 rows (of a token's heads, tokens after one another) per warp step, each
// CTA a range of `len` rows. VEC: rows of whole 16 bytes, shared by the power of two of lanes that they fill, ROW of them per lane; a
// lane keeps four rows' loads on their way. Bound by HBM (32768 x 32 rows of 128, 537 MB: 96 us). For fp16 on the tensor cores
// norms are taken besides, and a CTA looks through `v_len` rows of v: 134 MB more, 150 us.
template <typename T, bool VEC, int ROW>
__global__ void __launch_bounds__(256, 3) window_delta(const __grid_constant__ WindowProblem p, int team, int64_t len, int64_t v_len) {
    if (p.cu && *p.status != GDN_OK) return;
    if (!p.cu && blockIdx.x == 0 && threadIdx.x == 0) *p.status = GDN_OK;
    const gdn_window_attention_desc &d = p.d;
    constexpr bool kNorms = VEC && ROW == 1 && std::is_same<T, __half>::value;
    __shared__ uint32_t table[kNorms ? kTable : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t ntok = (int64_t)d.B * d.Tq, total = ntok * d.Hq;
    const T *o = (const T *)p.out_in, *g = (const T *)p.dout;
    if (!VEC) {
        for (int64_t i = (int64_t)blockIdx.x * 8 + warp; i < total; i += (int64_t)gridDim.x * 8) {
            float s = 0.0f;
            for (int c = lane; c < d.d; c += 32) s = fmaf(to_f<T>(o[i * d.d + c]), to_f<T>(g[i * d.d + c]), s);
            s = warp_sum(s);
            const int64_t tok = i / d.Hq;
            if (lane == 0) p.delta[(i - tok * d.Hq) * ntok + tok] = s;
        }
        return;
    }
    constexpr int N = Vec16<T>::N, kR = 4;
    const int sub = lane % team, per = 32 / team, c = sub * N, step = 8 * per;
    const int64_t first = blockIdx.x * len, end = min(first + len, total);
    // note: where a row's norm goes, `one`: a lane's j-th row is of the same sequence and head of keys in every step, whose largest
    // it keeps
    auto rows = [&](bool one, auto note) {
        float best[kR] = {0.0f, 0.0f, 0.0f, 0.0f};
        const RowAt start(first + warp * per + lane / team, step, d.Hq);
        RowAt at = start;
        for (int64_t i0 = first + warp * per + lane / team; i0 - lane / team < end; i0 += kR * step) {
            uint4 a[kR][ROW], b[kR][ROW];
#pragma unroll
            for (int j = 0; j < kR; ++j)
#pragma unroll
                for (int h = 0; h < ROW; ++h) {
                    const int64_t i = i0 + j * step;
                    const int x = c + h * 32 * N;
                    const bool in = i < end && x < d.d;
                    a[j][h] = in ? *(const uint4 *)(o + i * d.d + x) : make_uint4(0, 0, 0, 0);
                    b[j][h] = in ? *(const uint4 *)(g + i * d.d + x) : make_uint4(0, 0, 0, 0);
                }
            float s[kR], norm[kR];
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                float2 s2 = splat2(0.0f), n2 = s2;
#pragma unroll
                for (int h = 0; h < ROW; ++h) {
                    float2 x[N / 2], y[N / 2];
                    Pairs<T>::unpack(a[j][h], x);
                    Pairs<T>::unpack(b[j][h], y);
#pragma unroll
                    for (int e = 0; e < N / 2; ++e) {
                        s2 = fma2(x[e], y[e], s2);
                        if (kNorms) n2 = fma2(y[e], y[e], n2);
                    }
                }
                s[j] = s2.x + s2.y, norm[j] = n2.x + n2.y;
            }
            for (int x = team / 2; x; x >>= 1)   // the rows' shuffles side by side
#pragma unroll
                for (int j = 0; j < kR; ++j) {
                    s[j] += __shfl_xor_sync(0xffffffffu, s[j], x);
                    if (kNorms) norm[j] += __shfl_xor_sync(0xffffffffu, norm[j], x);
                }
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                if (sub == 0 && i0 + j * step < end) {
                    p.delta[at.head * ntok + at.tok] = s[j];
                    if (kNorms && !one) note(at, norm[j]);
                }
                if (kNorms) best[j] = norm[j] <= kFinite ? fmaxf(best[j], norm[j]) : best[j];
                at.next();
            }
        }
        at = start;
        if (kNorms && one)
#pragma unroll
            for (int j = 0; j < kR; ++j, at.next())
                if (sub == 0 && best[j] > 0.0f) note(at, best[j]);
    };
    if (first >= end) {
    } else if (kNorms && p.norms) {
        const RowNorms norms(p, false, table, first / d.Hq, (end - 1) / d.Hq);
        const unsigned group = d.Hq / d.Hk;
        rows(norms.n0 == norms.n1 && kR * step % d.Hq == 0, [&](const RowAt &at, float s) { norms.add(at.tok, (unsigned)at.head / group, s); });
        norms.flush();
    } else {
        rows(false, [](const RowAt &, float) {});
    }
    const int64_t v_rows = p.norms ? (int64_t)d.B * d.Tk * d.Hk : 0;
    if (kNorms && blockIdx.x * v_len < v_rows) {   // v (a row fits 32 lanes' 16 bytes: heads of up to 128 channels)
        const int64_t first = blockIdx.x * v_len, end = min(first + v_len, v_rows);
        const RowNorms norms(p, true, table, first / d.Hk, (end - 1) / d.Hk);
        const bool flat = p.cu || d.B == 1 || d.v_stride_b == d.Tk * d.v_stride_t;   // rows of the batch follow one another
        const bool one = norms.n0 == norms.n1 && kR * step % d.Hk == 0;
        float best[kR] = {0.0f, 0.0f, 0.0f, 0.0f};
        const RowAt start(first + warp * per + lane / team, step, d.Hk);
        RowAt at = start;
        for (int64_t i0 = first + warp * per + lane / team; i0 - lane / team < end; i0 += kR * step) {
            uint4 a[kR];
            RowAt ahead = at;
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                const int64_t row = flat ? 0 : ahead.tok / d.Tk;
                a[j] = make_uint4(0, 0, 0, 0);
                if (i0 + j * step < end && c < d.d)
                    a[j] = *(const uint4 *)((const T *)p.v + row * d.v_stride_b + (ahead.tok - row * d.Tk) * d.v_stride_t + (int64_t)ahead.head * d.d + c);
                ahead.next();
            }
            float s[kR];
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                float2 x[N / 2], s2 = splat2(0.0f);
                Pairs<T>::unpack(a[j], x);
#pragma unroll
                for (int e = 0; e < N / 2; ++e) s2 = fma2(x[e], x[e], s2);
                s[j] = s2.x + s2.y;
            }
            for (int x = team / 2; x; x >>= 1)
#pragma unroll
                for (int j = 0; j < kR; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], x);
#pragma unroll
            for (int j = 0; j < kR; ++j) {
                if (!one && sub == 0 && i0 + j * step < end) norms.add(at.tok, at.head, s[j]);
                best[j] = s[j] <= kFinite ? fmaxf(best[j], s[j]) : best[j];
                at.next();
            }
        }
        at = start;
        if (one)
#pragma unroll
            for (int j = 0; j < kR; ++j, at.next())
                if (sub == 0 && best[j] > 0.0f) norms.add(at.tok, at.head, best[j]);
        norms.flush();
    }
}

// delta of a short sequence's first positions as sum_j P_j (grad_out . v_j), a warp for each and head. With 16-bit types the output is
// rounded, and where a few keys share the weight dP - delta cancels: dq of 2 tokens (one head of 64, scores of deviation 2, bf16, the
// worst of 30) was off by 0.83, of 4 by 0.020, of 8 by 0.0075, of 16 by 0.0056, where rounding dS and dq costs 0.0035. From
// 64 keys on the other positions hold it to 0.0040, and such sequences are left as they are: the launch costs 6 us of a call.
constexpr int kFew = 8, kShort = 64;
template <typename T>
__device__ __forceinline__ void few_rows(const WindowProblem &p, int64_t first, int64_t apart) {
    const gdn_window_attention_desc &d = p.d;
    const int lane = threadIdx.x & 31;
    const int64_t total = (int64_t)d.N * (kFew - 1) * d.Hq;
    for (int64_t x = first; x < total; x += apart) {
        const int head = (int)(x % d.Hq), hk = head / (d.Hq / d.Hk);
        const int64_t at = x / d.Hq;
        const int n = (int)(at / (kFew - 1)), pos = (int)(at - (int64_t)n * (kFew - 1)) + 1;
        const WindowSpan s = window_span(p, n);
        const int64_t i = (int64_t)pos - s.Lk + s.Lq;
        if (i < 0 || i >= s.Lq || s.Lk > kShort) continue;
        const T *q = (const T *)p.q + s.qoff + i * d.q_stride_t + (int64_t)head * d.d, *g = (const T *)p.dout + ((s.q0 + i) * d.Hq + head) * d.d;
        const T *k = (const T *)p.k + s.koff + (int64_t)hk * d.d, *v = (const T *)p.v + s.voff + (int64_t)hk * d.d;
        float sc[kFew], dp[kFew];
        bool see[kFew];
#pragma unroll
        for (int j = 0; j < kFew; ++j) sc[j] = dp[j] = 0.0f, see[j] = j <= pos && (pos - j < d.window || j < d.sinks);
#pragma unroll 2
        for (int c = lane; c < d.d; c += 32) {
            const float qc = to_f<T>(q[c]), gc = to_f<T>(g[c]);
#pragma unroll
            for (int j = 0; j < kFew; ++j)
                if (see[j]) sc[j] = fmaf(qc, to_f<T>(k[j * d.k_stride_t + c]), sc[j]), dp[j] = fmaf(gc, to_f<T>(v[j * d.v_stride_t + c]), dp[j]);
        }
        float top = -INFINITY, l = 0.0f, sum = 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int j = 0; j < kFew; ++j) sc[j] += __shfl_xor_sync(0xffffffffu, sc[j], o), dp[j] += __shfl_xor_sync(0xffffffffu, dp[j], o);
#pragma unroll
        for (int j = 0; j < kFew; ++j) {
            sc[j] = see[j] ? sc[j] * d.scale : -INFINITY;
            top = fmaxf(top, sc[j]);
        }
#pragma unroll
        for (int j = 0; j < kFew; ++j)
            if (see[j]) {
                const float w = expf(sc[j] - top);
                l += w, sum = fmaf(w, dp[j], sum);
            }
        if (lane == 0) p.delta[head * ((int64_t)d.B * d.Tq) + s.q0 + i] = sum / l;
    }
}

// For packed sequences the sink tiles with a rest of those before each one, and for all the chunks before each such tile
__device__ __forceinline__ void rest_table(const WindowProblem &p) {
    __shared__ int32_t sums[32];
    if (threadIdx.x < 32) sums[threadIdx.x] = 0;
    __syncthreads();
    int tiles = p.sink_tiles, all;
    if (p.rest_packed) {
        tiles = 0;
        for (int base = 0; base < p.d.N; base += blockDim.x) {
            const int n = base + threadIdx.x;
            const int at = tiles + before_thread(n < p.d.N ? rest_count(p, window_span(p, n)) : 0, sums, all);
            if (n < p.d.N) p.rest_of[n] = at;
            tiles += all;
        }
        if (threadIdx.x == 0) p.rest_of[p.d.N] = tiles;
        __syncthreads();   // they are read below
    }
    const int total = p.rest_packed ? p.rest_all : p.sink_tiles;
    int before = 0;
    for (int base = 0; base < total; base += blockDim.x) {
        const int x = base + threadIdx.x;
        int c = 0;
        if (x < tiles) {
            const int n = p.rest_packed ? upper_index(p.rest_of, p.d.N, x) : 0;
            c = rest_chunks(p, window_span(p, n), x - (p.rest_packed ? p.rest_of[n] : 0));
        }
        const int at = before + before_thread(c, sums, all);
        if (x < total) p.rest_tiles[x] = at;
        before += all;
    }
    if (threadIdx.x == 0) p.rest_tiles[total] = before;
}

// Between delta and the gradients: CTA 0 makes the tables of the sinks' rest, the others the first positions' delta
template <typename T>
__global__ void __launch_bounds__(256, 3) window_between(const __grid_constant__ WindowProblem p, int table) {
    if (*p.status != GDN_OK) return;
    if (table && blockIdx.x == 0) rest_table(p);
    else if (sizeof(T) == 2) few_rows<T>(p, (int64_t)(blockIdx.x - table) * 8 + (threadIdx.x >> 5), (int64_t)(gridDim.x - table) * 8);
}

template <typename T>
cudaError_t backward_any(WindowProblem &p, cudaStream_t s) {
    const bool tc = (int64_t)p.d.B * p.d.Tq > 0 && p.d.Tk > 0 && window_tc_supports(p);
    if (!tc) p.norms = nullptr;
    const int64_t rows = (int64_t)p.d.B * p.d.Tq * p.d.Hq;
    constexpr int N = 16 / (int)sizeof(T);
    cudaError_t e = cudaSuccess;   // without packing and norms to begin from 0, delta sets the status word
    if ((p.cu || p.norms || !rows) && (e = launch_window_tables(p, tc ? 128 : 64, tc ? 128 : 64, s)) != cudaSuccess) return e;
    if (rows && p.d.d % N == 0 && ptr_aligned(p.out_in, 16) && ptr_aligned(p.dout, 16)) {
        int team = 1;
        while (team < 32 && team * N < p.d.d) team *= 2;
        const int64_t step = 32 * (32 / team), v_rows = p.norms ? (int64_t)p.d.B * p.d.Tk * p.d.Hk : 0;   // a CTA's rows on their way
        const auto len_of = [&](int64_t n) { return std::max<int64_t>(cdiv64(cdiv64(n, step), (p.norms ? 12 : 16) * kSms), 1) * step; };
        const int64_t len = len_of(rows), v_len = len_of(v_rows);
        const unsigned blocks = (unsigned)std::max(cdiv64(rows, len), cdiv64(v_rows, v_len));
        if (p.d.d <= 32 * N) window_delta<T, true, 1><<<blocks, 256, 0, s>>>(p, team, len, v_len);
        else window_delta<T, true, 2><<<blocks, 256, 0, s>>>(p, team, len, v_len);
    } else if (rows) {
        window_delta<T, false, 1><<<(unsigned)std::min<int64_t>(cdiv64(rows, 8), 64 * kSms), 256, 0, s>>>(p, 32, 0, 0);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    window_rest_plan(p, tc ? 7 : 6);
    const int table = p.sink_tiles > 0 && (p.rest_packed || p.sink_tiles > 1);   // one tile a row: no table is read
    const int few = sizeof(T) == 4 || !rows || (!p.rest_packed && p.d.Tk > kShort) ? 0 : (int)std::min<int64_t>(cdiv64((int64_t)p.d.N * (kFew - 1) * p.d.Hq, 8), 16 * kSms);
    if (table + few) window_between<T><<<table + few, 256, 0, s>>>(p, table);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return tc ? launch_window_backward_tc(p, s) : launch_window_backward_simt(p, s);
}

struct WindowLayout {
    size_t status, q_tiles, k_tiles, rest_of, rest_tiles, delta, norms, partial, total;
};
WindowLayout layout_of(const gdn_window_attention_desc &d, bool backward) {
    WindowLayout L;
    size_t off = 0;
    L.status = off;  off += kStatusBytes;
    L.q_tiles = off; off = align_up(off + 4 * ((size_t)d.N + 1), 256);
    L.k_tiles = off; off = align_up(off + 4 * ((size_t)d.N + 1), 256);
    L.rest_of = L.rest_tiles = L.delta = L.norms = L.partial = off;
    if (backward) {
        WindowProblem p;
        p.d = d;
        size_t partial = 0, tiles = 0;   // of either kernels: which it is the pointers say
        for (int shift = 6; shift <= 7; ++shift) {
            window_rest_plan(p, shift);
            partial = std::max(partial, window_partial_bytes(p));
            tiles = std::max(tiles, (size_t)(p.rest_packed ? p.rest_all : p.sink_tiles) + 1);
        }
        L.rest_of = off;    off = align_up(off + (p.rest_packed ? 4 * ((size_t)d.N + 1) : 0), 256);
        L.rest_tiles = off; off = align_up(off + 4 * tiles, 256);
        L.delta = off;   off = align_up(off + (size_t)d.B * d.Tq * d.Hq * 4, 256);
        L.norms = off;   off = align_up(off + (d.dtype == GDN_F16 ? 8 * (size_t)d.N * d.Hk : 0), 256);
        L.partial = off; off = align_up(off + partial, 256);
    }
    L.total = off;
    return L;
}

}  // namespace

cudaError_t launch_window_tables(const WindowProblem &p, int q_tile, int k_tile, cudaStream_t s) {
    window_tables_kernel<<<1, p.cu || p.norms ? 1024 : 32, 0, s>>>(p, q_tile, k_tile);
    return cudaGetLastError();
}

// The sinks' rest. A sink tile has one only where its last key lies more than `window` before the sequence's last, so that of packed
// sequences at most Tk / (window + 128) have any. A chunk is as long as a CTA of keys walks within the window (2048 to 32768
// queries), or longer, so that there are about eight CTAs of them for an SM: each holds 128 KB of partial sums (128 rows of 128
// channels), and more of them than that would grow with the sinks times the queries.
void window_rest_plan(WindowProblem &p, int shift) {
    const gdn_window_attention_desc &d = p.d;
    const int64_t group = d.Hq / d.Hk, unit = (int64_t)1 << shift, q_tiles = cdiv64(d.Tq, unit);
    p.rest_shift = shift;
    p.rest_packed = d.N != d.B;   // (one packed sequence is a row like another)
    p.sink_tiles = d.window >= d.Tk ? 0 : (int)std::min<int64_t>(cdiv64(std::min(d.sinks, d.Tk), 128), ((int64_t)d.Tk - d.window) / 128);
    p.sink_rows = std::min(128, std::min(d.sinks, d.Tk));
    const int64_t rows = p.rest_packed ? std::min<int64_t>(d.N, d.Tk / ((int64_t)d.window + 128)) : d.B;   // that can have one
    p.rest_all = (int)std::min<int64_t>(rows * p.sink_tiles, (int64_t)d.B * d.Tk / 128);
    p.rest_per = 0;
    p.rest_slots = 0;
    // tiles of queries behind the window of sink tile t, for rows that are alike
    const auto rest_tiles = [&](int64_t t) {
        const int64_t past = (int64_t)d.Tk - d.Tq, j0 = t * 128, j1 = std::min<int64_t>(j0 + 127, d.Tk - 1);
        const int64_t hi = std::min<int64_t>(d.Tq - 1, j1 + d.window - 1 - past), lo = std::max<int64_t>(0, j0 - past) >> shift;
        return std::max<int64_t>(0, q_tiles - std::max<int64_t>(hi < 0 ? 0 : (hi >> shift) + 1, lo));
    };
    int64_t visits = 0;   // of all rows, at most
    if (p.rest_packed) visits = p.sink_tiles * (q_tiles + rows);
    else
        for (int t = 0; t < p.sink_tiles; ++t) visits += d.B * rest_tiles(t);
    const int64_t window_its = std::min<int64_t>(32768 / unit, std::max<int64_t>(2048 / unit, group * (((int64_t)d.window + 127) / unit + 1)));
    const int64_t even_its = visits > ((int64_t)1 << 60) / d.Hq ? 1 << 30 : cdiv64(visits * d.Hq, 8 * kSms);
    p.rest_its = (int)std::min<int64_t>(std::max(window_its, even_its), 1 << 30);
    if (p.rest_packed) {   // at most: every tile's last chunk begun
        p.rest_slots = p.rest_all ? (int64_t)((double)visits * group / p.rest_its) + 1 + p.rest_all : 0;
    } else {
        for (int t = 0; t < p.sink_tiles; ++t) p.rest_per += (int)cdiv64(rest_tiles(t) * group, p.rest_its);
        p.rest_slots = (int64_t)d.B * p.rest_per;
    }
    if (p.rest_slots == 0) p.sink_tiles = p.rest_all = 0;
}

size_t window_partial_bytes(const WindowProblem &p) {
    if (p.rest_slots == 0) return 0;
    return (size_t)(p.rest_slots + p.rest_all) * p.d.Hk * p.sink_rows * 2 * (p.d.d <= 64 ? 64 : p.d.d <= 128 ? 128 : 256) * 4;
}

int window_check_desc(const gdn_window_attention_desc *d, bool packed) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->Tq < 0 || d->Tk < 0 || d->N < 1 || d->Hq < 1 || d->Hk < 1 || d->d < 1) return GDN_ERR_INVALID_ARG;
    if (packed ? d->B != 1 : d->N != d->B) return GDN_ERR_INVALID_ARG;
    if (d->window < 1 || d->sinks < 0 || !(d->scale > 0.0f) || !isfinite(d->scale)) return GDN_ERR_INVALID_ARG;
    const int64_t strides[] = {d->q_stride_b, d->q_stride_t, d->k_stride_b, d->k_stride_t, d->v_stride_b, d->v_stride_t};
    for (const int64_t s : strides)
        if (s < 0) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype) || d->Hq % d->Hk || d->d > kMostHead) return GDN_ERR_UNSUPPORTED;
    const int64_t cq = (int64_t)d->Hq * d->d, ck = (int64_t)d->Hk * d->d;
    if (cq > (1 << 24) || d->Tq > 0x7fffffff - 65536 || d->Tk > 0x7fffffff - 65536) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)d->B * d->Tq > 0x7fffffff || (int64_t)d->B * d->Tk > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
    if (d->Tq > 1 && d->q_stride_t < cq) return GDN_ERR_INVALID_ARG;
    if (d->Tk > 1 && (d->k_stride_t < ck || d->v_stride_t < ck)) return GDN_ERR_INVALID_ARG;
    if ((double)d->B * d->Tq * cq > 4.0e12 || (double)d->B * d->Tk * ck > 4.0e12) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

namespace {

// The checks that forward and backward share; on success p holds the inputs and the workspace
int fill(WindowProblem &p, const gdn_window_attention_desc *d, const void *q, const void *k, const void *v, const int32_t *cu,
         const int32_t *cuk, const void *out, const float *lse, void *workspace, size_t workspace_bytes, bool backward) {
    int rc = window_check_desc(d, cu != nullptr);
    if (rc != GDN_OK) return rc;
    if (cuk && !cu) return GDN_ERR_INVALID_ARG;
    if (cu && !cuk && d->Tq != d->Tk) return GDN_ERR_INVALID_ARG;
    const bool nq = (int64_t)d->B * d->Tq > 0, nk = (int64_t)d->B * d->Tk > 0;   // token tensors may be empty (null)
    if ((nq && (!q || !out)) || (nk && (!k || !v))) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(q, es) || !ptr_aligned(k, es) || !ptr_aligned(v, es) || !ptr_aligned(out, es) || !ptr_aligned(lse, 4) ||
        !ptr_aligned(cu, 4) || !ptr_aligned(cuk, 4))
        return GDN_ERR_INVALID_ARG;
    const WindowLayout L = layout_of(*d, backward);
    if ((rc = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return rc;
    char *ws = (char *)workspace;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.q = q, p.k = k, p.v = v;
    p.cu = cu, p.cuk = cuk ? cuk : cu;
    p.lse = const_cast<float *>(lse);
    p.status = (int32_t *)ws;
    p.q_tiles = (int32_t *)(ws + L.q_tiles);
    p.k_tiles = (int32_t *)(ws + L.k_tiles);
    p.rest_of = (int32_t *)(ws + L.rest_of), p.rest_tiles = (int32_t *)(ws + L.rest_tiles);
    p.delta = (float *)(ws + L.delta);
    p.norms = backward && d->dtype == GDN_F16 ? (uint32_t *)(ws + L.norms) : nullptr;   // the tensor cores' alone
    p.partial = (float *)(ws + L.partial);
    p.wait_immediate = wait_test_mode();
    return GDN_OK;
}

int bytes_of(const gdn_window_attention_desc *d, size_t *bytes, bool backward) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = window_check_desc(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = layout_of(*d, backward).total;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_window_attention_desc_init(gdn_window_attention_desc *d, int B, int Tq, int Tk, int packed, int Hq, int Hk, int head_dim,
                                   int window, int sinks, int dtype) {
    if (!d) return GDN_ERR_INVALID_ARG;
    memset(d, 0, sizeof(*d));
    d->B = B, d->Tq = Tq, d->Tk = Tk;
    d->N = packed ? packed : B;
    d->Hq = Hq, d->Hk = Hk, d->d = head_dim;
    d->window = window, d->sinks = sinks;
    d->slots = (int32_t)std::min<int64_t>((int64_t)window + sinks, 0x7fffffff);
    d->dtype = dtype;
    d->scale = head_dim > 0 ? (float)(1.0 / sqrt((double)head_dim)) : 0.0f;
    d->q_stride_t = (int64_t)Hq * head_dim;
    d->k_stride_t = d->v_stride_t = (int64_t)Hk * head_dim;
    d->q_stride_b = d->q_stride_t * Tq;
    d->k_stride_b = d->v_stride_b = d->k_stride_t * Tk;
    return window_check_desc(d, packed != 0);
}

int gdn_window_attention_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes) { return bytes_of(d, bytes, false); }
int gdn_window_attention_backward_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes) { return bytes_of(d, bytes, true); }

int gdn_window_attention_kernel_kind(const gdn_window_attention_desc *d) { return d && window_tc_fits(*d) ? 1 : 0; }

int gdn_window_attention_forward(const gdn_window_attention_desc *d, const void *q, const void *k, const void *v, const int32_t *cu_seqlens,
                                 const int32_t *cu_seqlens_k, void *out, float *lse, void *workspace, size_t workspace_bytes,
                                 gdn_stream_t stream) {
    WindowProblem p;
    const int rc = fill(p, d, q, k, v, cu_seqlens, cu_seqlens_k, out, lse, workspace, workspace_bytes, false);
    if (rc != GDN_OK) return rc;
    p.out = out;
    const cudaStream_t s = (cudaStream_t)stream;
    if ((int64_t)d->B * d->Tq > 0 && d->Tk > 0 && window_tc_supports(p)) return layer_status(launch_window_forward_tc(p, s));
    return layer_status(launch_window_forward_simt(p, s));
}

int gdn_window_attention_backward(const gdn_window_attention_desc *d, const void *q, const void *k, const void *v, const void *out,
                                  const float *lse, const void *grad_out, const int32_t *cu_seqlens, const int32_t *cu_seqlens_k,
                                  void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    WindowProblem p;
    const int rc = fill(p, d, q, k, v, cu_seqlens, cu_seqlens_k, out, lse, workspace, workspace_bytes, true);
    if (rc != GDN_OK) return rc;
    const size_t es = act_size(d->dtype);
    if ((int64_t)d->B * d->Tq > 0 && (!lse || !grad_out || !dq)) return GDN_ERR_INVALID_ARG;
    if ((int64_t)d->B * d->Tk > 0 && (!dk || !dv)) return GDN_ERR_INVALID_ARG;
    if (!ptr_aligned(grad_out, es) || !ptr_aligned(dq, es) || !ptr_aligned(dk, es) || !ptr_aligned(dv, es)) return GDN_ERR_INVALID_ARG;
    p.out_in = out, p.dout = grad_out;
    p.dq = dq, p.dk = dk, p.dv = dv;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d->dtype) {
    case GDN_F32: return layer_status(backward_any<float>(p, s));
    case GDN_BF16: return layer_status(backward_any<__nv_bfloat16>(p, s));
    default: return layer_status(backward_any<__half>(p, s));
    }
}

}  // extern "C"
