// gdn_recurrence.cu -- gated linear recurrence (include/gdn.h): forward, backward
// and the single-token step, with their C entry points.
//
// Forward and backward are scans over the tokens of a row, channel by channel. A
// scan composes affine maps h -> A h + B; a tile of tokens is one such map, so the
// tiles of a row can be worked on at the same time and only their maps have to meet:
//
//   - a chain is one row's tokens by one slab of 128 bytes of channels (64, or 32 of
//     fp32). A cluster of 1 to 16 CTAs walks it, CTA r of the cluster taking the tiles
//     k cs + r of step k = 0, 1, ...; every input is read once.
//   - a tile has 8 tokens for each of the CTA's token groups (4 warps x 2, or x 4 with
//     fp32). A thread owns 4 channels of one group: it composes its 8 tokens in
//     registers, the groups of a warp compose by shuffles, the warps through shared
//     memory, the CTAs through each other's shared memory and one cluster barrier per
//     step. The carried state then goes back down and each thread finishes its tokens.
//   - a sequence's first token has decay 0 and its initial state written into u, which
//     makes packed sequences nothing special to the scan, whatever their lengths.
//
// The order of every composition and sum is fixed by the sizes alone, so results are
// run-to-run identical. Tiles come in by TMA (two stages, from rows that are 16-byte
// aligned; other tensors are read element by element).
#include <algorithm>
#include <string.h>

#include "gdn_layer_ops.cuh"
#include "gdn_recurrence.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

struct RecProblem {
    gdn_recurrence_desc d;
    const void *x, *a, *b, *grad_out;
    const float *A_log, *dt_bias;
    const int32_t *cu;
    const float *h0;
    void *out;
    float *hT, *cs;              // final states; states carried into every 8th token
    int32_t *status;
    const float *grad_final;
    void *dx, *da, *db;
    float *dA_log, *ddt_bias, *dh0, *part;
    int slabs, ntiles, wait_immediate;
};

struct RecMaps {
    CUtensorMap x, a, b, dy;
};

constexpr int kR = GDN_RECURRENCE_CHUNK;   // tokens per thread and tile
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 16;
static_assert(kR == 8, "the start and end masks hold one bit per token");

template <typename T> struct Tile {
    static constexpr int LR = 128 / (4 * (int)sizeof(T));   // lanes per token row, 4 channels each
    static constexpr int G = 32 / LR;                       // token groups per warp
    static constexpr int NG = kWarps * G;                   // per CTA
    static constexpr int TT = NG * kR;                      // tokens
    static constexpr int CH = LR * 4;                       // channels
    static constexpr int kTensor = TT * 128;                // bytes of one tensor's tile
};

struct F4 {          // four channels as two pairs
    float2 lo, hi;
};
__device__ __forceinline__ F4 f4(float v) { return {splat2(v), splat2(v)}; }
__device__ __forceinline__ F4 f4(float4 v) { return {make_float2(v.x, v.y), make_float2(v.z, v.w)}; }
__device__ __forceinline__ float4 to4(const F4 &v) { return make_float4(v.lo.x, v.lo.y, v.hi.x, v.hi.y); }
__device__ __forceinline__ F4 fma4(const F4 &a, const F4 &b, const F4 &c) { return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }
__device__ __forceinline__ F4 mul4(const F4 &a, const F4 &b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ F4 add4(const F4 &a, const F4 &b) { return {add2(a.lo, b.lo), add2(a.hi, b.hi)}; }
// A sequence's first token cuts the chain: its A is -0 (a decay that underflows is +0), and a map whose A
// is -0 takes nothing from before it, not even a NaN. Only packed rows have such maps behind others.
__device__ __forceinline__ float2 cut2(float2 a, float2 yes, float2 no) {
    return make_float2(__float_as_int(a.x) < 0 ? yes.x : no.x, __float_as_int(a.y) < 0 ? yes.y : no.y);
}
// A h + B
__device__ __forceinline__ F4 apply(const F4 &A, const F4 &B, const F4 &h, bool packed) {
    F4 r = fma4(A, h, B);
    if (packed) r = {cut2(A.lo, B.lo, r.lo), cut2(A.hi, B.hi, r.hi)};
    return r;
}
// the A of a map after one with pA
__device__ __forceinline__ F4 compose(const F4 &A, const F4 &pA, bool packed) {
    F4 r = mul4(A, pA);
    if (packed) r = {cut2(A.lo, A.lo, r.lo), cut2(A.hi, A.hi, r.hi)};
    return r;
}
template <bool UP>
__device__ __forceinline__ F4 shfl4(const F4 &v, int by) {
    F4 r;
    if (UP) {
        r.lo.x = __shfl_up_sync(0xffffffffu, v.lo.x, by);
        r.lo.y = __shfl_up_sync(0xffffffffu, v.lo.y, by);
        r.hi.x = __shfl_up_sync(0xffffffffu, v.hi.x, by);
        r.hi.y = __shfl_up_sync(0xffffffffu, v.hi.y, by);
    } else {
        r.lo.x = __shfl_down_sync(0xffffffffu, v.lo.x, by);
        r.lo.y = __shfl_down_sync(0xffffffffu, v.lo.y, by);
        r.hi.x = __shfl_down_sync(0xffffffffu, v.hi.x, by);
        r.hi.y = __shfl_down_sync(0xffffffffu, v.hi.y, by);
    }
    return r;
}

// 4 elements of T from 4 * sizeof(T) bytes
template <typename T> __device__ __forceinline__ F4 unpack4(const void *p);
template <> __device__ __forceinline__ F4 unpack4<float>(const void *p) { return f4(*(const float4 *)p); }
template <> __device__ __forceinline__ F4 unpack4<__nv_bfloat16>(const void *p) {
    const uint2 u = *(const uint2 *)p;
    return {Pairs<__nv_bfloat16>::word(u.x), Pairs<__nv_bfloat16>::word(u.y)};
}
template <> __device__ __forceinline__ F4 unpack4<__half>(const void *p) {
    const uint2 u = *(const uint2 *)p;
    return {Pairs<__half>::word(u.x), Pairs<__half>::word(u.y)};
}
template <typename T> __device__ __forceinline__ void pack4(void *p, const F4 &v) {
    *(uint2 *)p = make_uint2(Pairs<T>::pack1(v.lo), Pairs<T>::pack1(v.hi));
}
template <> __device__ __forceinline__ void pack4<float>(void *p, const F4 &v) { *(float4 *)p = to4(v); }

// Up to four channels of a row in global memory; nc of them exist. VEC: rows are aligned and nc is 4 or 0.
template <typename T, bool VEC>
__device__ __forceinline__ F4 load_row(const T *p, int nc) {
    if (VEC) return nc > 0 ? unpack4<T>(p) : f4(0.f);
    return {make_float2(nc > 0 ? to_f<T>(p[0]) : 0.f, nc > 1 ? to_f<T>(p[1]) : 0.f),
            make_float2(nc > 2 ? to_f<T>(p[2]) : 0.f, nc > 3 ? to_f<T>(p[3]) : 0.f)};
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_row(T *p, const F4 &v, int nc) {
    if (VEC) {
        if (nc > 0) pack4<T>(p, v);
        return;
    }
    if (nc > 0) p[0] = from_f<T>(v.lo.x);
    if (nc > 1) p[1] = from_f<T>(v.lo.y);
    if (nc > 2) p[2] = from_f<T>(v.hi.x);
    if (nc > 3) p[3] = from_f<T>(v.hi.y);
}
// four fp32 values of a row whose alignment is not known
__device__ __forceinline__ F4 load_words(const float *p, int nc) { return load_row<float, false>(p, nc); }
__device__ __forceinline__ void store_words(float *p, const F4 &v, int nc) { store_row<float, false>(p, v, nc); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 8 bytes into the shared memory of CTA `rank` of the cluster, at this CTA's address `p`
__device__ __forceinline__ void remote_store(const void *p, uint32_t rank, float a, float b) {
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
                 "st.shared::cluster.v2.f32 [ra], {%2, %3};\n\t}"
                 :: "r"(tc::smem_u32(p)), "r"(rank), "f"(a), "f"(b) : "memory");
}

// The cross-thread part of a step, for one CTA: composes the maps (A, B) of the token groups in
// walking order (FWD: rising groups, else falling) and carries the state through them.
template <typename T, bool FWD> struct Chain {
    using L = Tile<T>;
    float4 wA[kWarps][L::LR], wB[kWarps][L::LR];            // maps of the warps
    float2 agg[2][kMaxCluster][L::CH];                      // maps of the cluster's CTAs, by step parity

    // In: this group's map. Out: the state carried into this group; `carry`, the state carried into the
    // step (the same in all groups of all CTAs), moves on to the next step.
    __device__ __forceinline__ F4 run(F4 A, F4 B, F4 &carry, int warp, int lane, uint32_t rank, uint32_t cs, int parity,
                                      bool packed) {
        const int g = lane / L::LR, q = lane % L::LR;
        const int og = FWD ? g : L::G - 1 - g, ow = FWD ? warp : kWarps - 1 - warp;   // walking order
#pragma unroll
        for (int off = 1; off < L::G; off *= 2) {
            const F4 pA = shfl4<FWD>(A, off * L::LR), pB = shfl4<FWD>(B, off * L::LR);
            if (og >= off) {
                B = apply(A, B, pB, packed);
                A = compose(A, pA, packed);
            }
        }
        if (og == L::G - 1) {
            wA[ow][q] = to4(A);
            wB[ow][q] = to4(B);
        }
        F4 eA = shfl4<FWD>(A, L::LR), eB = shfl4<FWD>(B, L::LR);   // of the groups before, in the warp
        if (og == 0) eA = f4(1.f), eB = f4(0.f);
        __syncthreads();
        if (cs > 1) {
            // the CTA's map to every CTA of the cluster: one channel and a share of the ranks per thread
            const int c = threadIdx.x % L::CH;
            float tA = 1.f, tB = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float a = ((const float *)wA[w])[c], b = ((const float *)wB[w])[c];
                const bool cut = packed && __float_as_int(a) < 0;
                tB = cut ? b : fmaf(a, tB, b);
                tA = cut ? a : tA * a;
            }
            for (uint32_t r = threadIdx.x / L::CH; r < cs; r += kThreads / L::CH) remote_store(&agg[parity][rank][c], r, tA, tB);
        }
        F4 c = f4(0.f);   // carried into this CTA's tile
        if (cs > 1) {
            cluster_sync();
            c = carry;
            for (uint32_t r = 0; r < cs; ++r) {
                if (r == rank) c = carry;
                const float4 *m = (const float4 *)&agg[parity][r][q * 4];
                const float4 m0 = m[0], m1 = m[1];
                carry = apply({make_float2(m0.x, m0.z), make_float2(m1.x, m1.z)},
                              {make_float2(m0.y, m0.w), make_float2(m1.y, m1.w)}, carry, packed);
            }
        } else {
            c = carry;
        }
        // through the warps before this one, and on to the end for a chain of one CTA
        F4 s = c;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == ow) c = s;
            if (w < ow || cs == 1) s = apply(f4(wA[w][q]), f4(wB[w][q]), s, packed);
        }
        if (cs == 1) carry = s;
        return apply(eA, eB, c, packed);
    }
};

// The sequence that holds the walk's current token. Rows are one sequence each.
struct Seq {
    int n, b0, b1;      // sequence, its first token, one past its last
    __device__ __forceinline__ void init(const RecProblem &p, int row) {
        n = p.cu ? 0 : row;
        b0 = 0;
        b1 = p.cu ? p.cu[1] : p.d.T;
    }
    __device__ __forceinline__ void up_to(const RecProblem &p, int t) {   // forward to the sequence of token t
        if (p.cu == nullptr) return;
        while (b1 <= t && n + 1 < p.d.N) {
            ++n;
            b0 = b1;
            b1 = p.cu[n + 1];
        }
    }
    __device__ __forceinline__ void down_to(const RecProblem &p, int t) {   // backward to it
        if (p.cu == nullptr) return;
        while (b0 > t && n > 0) {
            --n;
            b1 = b0;
            b0 = p.cu[n];
        }
    }
};

// Sequences without tokens: their final state is their initial state (dst, src), zeros without one.
__device__ void copy_empty(const RecProblem &p, int row, int ch, int nc, float *dst, const float *src, int group, int groups) {
    if (dst == nullptr) return;
    for (int n = (p.cu ? 0 : row) + group; n < (p.cu ? p.d.N : row + 1); n += groups) {
        if (p.cu ? p.cu[n] != p.cu[n + 1] : p.d.T != 0) continue;
        store_words(dst + (int64_t)n * p.d.D + ch, src ? load_words(src + (int64_t)n * p.d.D + ch, nc) : f4(0.f), nc);
    }
}

// Waits for a stage (bounded, about a second; see gdn_set_wait_test_mode). `failed` makes every later
// wait a test, so that a CTA whose copies do not arrive ends soon.
__device__ __forceinline__ void stage_wait(uint64_t *bar, uint32_t phase, const RecProblem &p, bool &failed) {
    if (!tc::mbar_wait(bar, phase, failed || p.wait_immediate)) failed = true;
}

// Bound by HBM (8 bytes per 16-bit element) and, near it, by the special-function and issue rates: about
// 30 instructions and 5 special functions per element.
template <typename T, bool TMA>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
rec_forward_kernel(const RecProblem p, const __grid_constant__ RecMaps maps) {
    using L = Tile<T>;
    extern __shared__ __align__(128) unsigned char smem[];   // TMA: 2 stages of x, a, b
    __shared__ Chain<T, true> chain;
    __shared__ uint64_t full[2];
    const gdn_recurrence_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / L::LR, q = lane % L::LR;
    uint32_t cs;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
    const uint32_t rank = cluster_rank();
    const int slab = (int)(blockIdx.x / cs) % p.slabs, row = (int)(blockIdx.x / cs) / p.slabs;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && tid == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;   // the same in every CTA
    const int ch = slab * L::CH + q * 4, nc = min(4, max(0, d.D - ch));
    const int steps = (p.ntiles + (int)cs - 1) / (int)cs;

    auto issue = [&](int k) {   // thread 0: the tile of step k into stage k % 2
        const int tile = k * (int)cs + (int)rank;
        if (tile >= p.ntiles) return;
        unsigned char *st = smem + (k & 1) * 3 * L::kTensor;
        tc::mbar_expect_tx(&full[k & 1], 3 * L::kTensor);
        tc::tma_load_3d(st, &maps.x, slab * L::CH, tile * L::TT, row, &full[k & 1]);
        tc::tma_load_3d(st + L::kTensor, &maps.a, slab * L::CH, tile * L::TT, row, &full[k & 1]);
        tc::tma_load_3d(st + 2 * L::kTensor, &maps.b, slab * L::CH, tile * L::TT, row, &full[k & 1]);
    };
    if (TMA) {
        if (tid == 0) {
            tc::mbar_init(&full[0], 1);
            tc::mbar_init(&full[1], 1);
            tc::mbar_init_fence();
            if (!p.wait_immediate) {
                issue(0);
                issue(1);
            }
        }
        __syncthreads();
    }
    F4 rate = load_words(p.A_log + ch, nc);
    rate = {make_float2(expf(rate.lo.x), expf(rate.lo.y)), make_float2(expf(rate.hi.x), expf(rate.hi.y))};
    const F4 bias = load_words(p.dt_bias + ch, nc);
    if (rank == 0) copy_empty(p, row, ch, nc, p.hT, p.h0, warp * L::G + g, L::NG);
    Seq seq;
    seq.init(p, row);
    F4 carry = f4(0.f);
    bool failed = false;
    if (TMA && tid == 0 && p.wait_immediate) {   // so late that the first wait cannot be over
        issue(0);
        issue(1);
    }
    for (int k = 0; k < steps; ++k) {
        const int tile = k * (int)cs + (int)rank;
        const bool real = tile < p.ntiles;
        const int t0 = tile * L::TT + (warp * L::G + g) * kR;   // this group's first token
        F4 P[kR], h[kR];
        if (real) {
            if (TMA) stage_wait(&full[k & 1], (k >> 1) & 1, p, failed);
            const unsigned char *st = smem + (k & 1) * 3 * L::kTensor + (t0 - tile * L::TT) * 128 + q * 4 * sizeof(T);
            seq.up_to(p, t0);
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                F4 x, a, b;
                if (TMA) {
                    x = unpack4<T>(st + r * 128);
                    a = unpack4<T>(st + L::kTensor + r * 128);
                    b = unpack4<T>(st + 2 * L::kTensor + r * 128);
                } else {
                    const int n = t0 + r < d.T ? nc : 0;
                    const int64_t t = t0 + r;
                    x = load_row<T, false>((const T *)p.x + row * d.x_stride_b + t * d.x_stride_t + ch, n);
                    a = load_row<T, false>((const T *)p.a + row * d.a_stride_b + t * d.a_stride_t + ch, n);
                    b = load_row<T, false>((const T *)p.b + row * d.b_stride_b + t * d.b_stride_t + ch, n);
                }
                const Decay2 e0 = decay2(a.lo, bias.lo, rate.lo), e1 = decay2(a.hi, bias.hi, rate.hi);
                const F4 s = {mul2(e0.w, inv_sqrt2(e0.w)), mul2(e1.w, inv_sqrt2(e1.w))};
                P[r] = {e0.alpha, e1.alpha};
                h[r] = mul4(mul4(s, {sigmoid2(b.lo), sigmoid2(b.hi)}), x);
            }
            if (seq.b0 == t0 || (seq.b1 < t0 + kR && seq.b1 < d.T)) {   // a sequence starts here
                Seq m = seq;
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    m.up_to(p, t0 + r);
                    if (m.b0 == t0 + r && t0 + r < d.T) {
                        if (p.h0) h[r] = fma4(P[r], load_words(p.h0 + (int64_t)m.n * d.D + ch, nc), h[r]);
                        P[r] = f4(-0.f);
                    }
                    if (r > 0) {
                        h[r] = apply(P[r], h[r], h[r - 1], true);
                        P[r] = compose(P[r], P[r - 1], true);
                    }
                }
            } else {
#pragma unroll
                for (int r = 1; r < kR; ++r) {
                    h[r] = fma4(P[r], h[r - 1], h[r]);
                    P[r] = mul4(P[r], P[r - 1]);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < kR; ++r) P[r] = f4(1.f), h[r] = f4(0.f);
        }
        const F4 c = chain.run(P[kR - 1], h[kR - 1], carry, warp, lane, rank, cs, k & 1, p.cu != nullptr);
        // chain.run's barrier: every thread has read this stage
        if (TMA && tid == 0 && !failed) issue(k + 2);
        if (real && t0 < d.T) {
            if (p.cs)
                store_words(p.cs + ((int64_t)row * ((d.T + kR - 1) / kR) + t0 / kR) * d.D + ch, c, nc);
#pragma unroll
            for (int r = 0; r < kR; ++r) h[r] = apply(P[r], h[r], c, p.cu != nullptr);
            if (p.out) {
                T *o = (T *)p.out + ((int64_t)row * d.T + t0) * d.D + ch;
#pragma unroll
                for (int r = 0; r < kR; ++r)
                    if (t0 + r < d.T) store_row<T, TMA>(o + (int64_t)r * d.D, h[r], nc);
            }
            if (p.hT && seq.b1 <= t0 + kR) {   // a sequence ends here
                Seq m = seq;
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    m.up_to(p, t0 + r);
                    if (m.b1 == t0 + r + 1) store_words(p.hT + (int64_t)m.n * d.D + ch, h[r], nc);
                }
            }
        }
        // the warps' maps are read in run() up to here and written again in the next step
        __syncthreads();
    }
    if (failed) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    if (TMA && tid == 0 && failed)   // copies in flight end before the CTA does
        for (int k = max(0, steps - 2); k < steps; ++k)
            if (k * (int)cs + (int)rank < p.ntiles) tc::mbar_wait(&full[k & 1], (k >> 1) & 1);
}

// The reverse scan: c_t = alpha_t (v_t + c_{t+1}), delta_t = v_t + c_{t+1}, tiles last to first. The
// states before every 8th token come from the forward, so h_{t-1} is recomputed within a thread.
template <typename T, bool TMA>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 1)
rec_backward_kernel(const RecProblem p, const __grid_constant__ RecMaps maps) {
    using L = Tile<T>;
    extern __shared__ __align__(128) unsigned char smem[];   // TMA: 2 stages of x, a, b, grad_out
    __shared__ Chain<T, false> chain;
    __shared__ uint64_t full[2];
    const gdn_recurrence_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / L::LR, q = lane % L::LR;
    uint32_t cs;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
    const uint32_t rank = cluster_rank();
    const int chains = (int)(blockIdx.x / cs);
    const int slab = chains % p.slabs, row = chains / p.slabs;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && tid == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int ch = slab * L::CH + q * 4, nc = min(4, max(0, d.D - ch));
    const int steps = (p.ntiles + (int)cs - 1) / (int)cs;

    auto issue = [&](int k) {
        const int back = k * (int)cs + (int)rank, tile = p.ntiles - 1 - back;
        if (tile < 0) return;
        unsigned char *st = smem + (k & 1) * 4 * L::kTensor;
        tc::mbar_expect_tx(&full[k & 1], 4 * L::kTensor);
        tc::tma_load_3d(st, &maps.x, slab * L::CH, tile * L::TT, row, &full[k & 1]);
        tc::tma_load_3d(st + L::kTensor, &maps.a, slab * L::CH, tile * L::TT, row, &full[k & 1]);
        tc::tma_load_3d(st + 2 * L::kTensor, &maps.b, slab * L::CH, tile * L::TT, row, &full[k & 1]);
        tc::tma_load_3d(st + 3 * L::kTensor, &maps.dy, slab * L::CH, tile * L::TT, row, &full[k & 1]);
    };
    if (TMA) {
        if (tid == 0) {
            tc::mbar_init(&full[0], 1);
            tc::mbar_init(&full[1], 1);
            tc::mbar_init_fence();
            if (!p.wait_immediate) issue(0);
        }
        __syncthreads();
    }
    F4 rate = load_words(p.A_log + ch, nc);
    rate = {make_float2(expf(rate.lo.x), expf(rate.lo.y)), make_float2(expf(rate.hi.x), expf(rate.hi.y))};
    const F4 bias = load_words(p.dt_bias + ch, nc);
    if (rank == 0) copy_empty(p, row, ch, nc, p.dh0, p.grad_final, warp * L::G + g, L::NG);
    Seq seq;
    seq.init(p, row);
    seq.up_to(p, d.T - 1);
    F4 carry = f4(0.f);
    // sums of da and of dg g over this thread's tokens: per tile, over 16 tiles, over all
    F4 sA[2] = {f4(0.f), f4(0.f)}, sb[2] = {f4(0.f), f4(0.f)};
    bool failed = false;
    if (TMA && tid == 0 && p.wait_immediate) issue(0);   // so late that the first wait cannot be over
    for (int k = 0; k < steps; ++k) {
        const int tile = p.ntiles - 1 - (k * (int)cs + (int)rank);
        const bool real = tile >= 0;
        const int t0 = tile * L::TT + (warp * L::G + g) * kR;
        const bool any = real && t0 < d.T;
        const unsigned char *st = smem + (k & 1) * 4 * L::kTensor + (warp * L::G + g) * kR * 128 + q * 4 * sizeof(T);
        auto in = [&](int which, const void *base, int64_t sb_, int64_t st_, int r) -> F4 {
            if (TMA) return unpack4<T>(st + which * L::kTensor + r * 128);
            return load_row<T, false>((const T *)base + row * sb_ + (int64_t)(t0 + r) * st_ + ch, t0 + r < d.T ? nc : 0);
        };
        auto dy = [&](int r) -> F4 { return in(3, p.grad_out, (int64_t)d.T * d.D, d.D, r); };
        F4 al[kR], Q = f4(1.f), c = f4(0.f), hs = f4(0.f);
        uint32_t starts = 0, ends = 0;   // tokens of this group that start or end a sequence
        if (real) {
            if (TMA) stage_wait(&full[k & 1], (k >> 1) & 1, p, failed);
            if (any) {
                hs = load_words(p.cs + ((int64_t)row * ((d.T + kR - 1) / kR) + t0 / kR) * d.D + ch, nc);
                seq.down_to(p, t0);
                if (seq.b0 == t0 || seq.b1 <= t0 + kR) {
                    Seq m = seq;
                    for (int r = 0; r < kR && t0 + r < d.T; ++r) {
                        m.up_to(p, t0 + r);
                        starts |= (m.b0 == t0 + r ? 1u : 0u) << r;
                        ends |= (m.b1 == t0 + r + 1 ? 1u : 0u) << r;
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const F4 a = in(1, p.a, d.a_stride_b, d.a_stride_t, r);
                al[r] = {decay2(a.lo, bias.lo, rate.lo).alpha, decay2(a.hi, bias.hi, rate.hi).alpha};
                if (starts >> r & 1) al[r] = f4(-0.f);
            }
#pragma unroll
            for (int r = kR - 1; r >= 0; --r) {
                F4 v = dy(r);
                if (ends >> r & 1 && p.grad_final) {
                    Seq m = seq;
                    m.up_to(p, t0 + r);
                    v = add4(v, load_words(p.grad_final + (int64_t)m.n * d.D + ch, nc));
                }
                c = mul4(al[r], add4(v, c));
                Q = compose(al[r], Q, p.cu != nullptr);
                if (starts >> r & 1) c = f4(0.f);
            }
        }
        c = chain.run(Q, c, carry, warp, lane, rank, cs, k & 1, p.cu != nullptr);
        // chain.run's barrier: every thread is done with the stage of step k - 1
        if (TMA && tid == 0 && !failed) issue(k + 1);
        if (any) {
            F4 dl[kR];
#pragma unroll
            for (int r = kR - 1; r >= 0; --r) {
                F4 v = dy(r);
                if (ends >> r & 1 && p.grad_final) {
                    Seq m = seq;
                    m.up_to(p, t0 + r);
                    v = add4(v, load_words(p.grad_final + (int64_t)m.n * d.D + ch, nc));
                }
                dl[r] = add4(v, c);
                c = mul4(al[r], dl[r]);
                if (starts >> r & 1) c = f4(0.f);
            }
            F4 tA = f4(0.f), tb = f4(0.f);
            const int64_t o = ((int64_t)row * d.T + t0) * d.D + ch;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const F4 x = in(0, p.x, d.x_stride_b, d.x_stride_t, r), a = in(1, p.a, d.a_stride_b, d.a_stride_t, r),
                         b = in(2, p.b, d.b_stride_b, d.b_stride_t, r);
                int n0 = 0;
                if (starts >> r & 1) {
                    Seq m = seq;
                    m.up_to(p, t0 + r);
                    n0 = m.n;
                    hs = p.h0 ? load_words(p.h0 + (int64_t)n0 * d.D + ch, nc) : f4(0.f);
                }
                F4 gx, ga, gb, al1;
                auto pair = [&](float2 xv, float2 av, float2 bv, float2 bi, float2 ra, float2 de, float2 &hh, float2 &qA,
                                float2 &qb, float2 &ox, float2 &oa, float2 &ob, float2 &oal) {
                    const Decay2 e = decay2(av, bi, ra);
                    const float2 rs = inv_sqrt2(e.w), be = sigmoid2(bv), s = mul2(e.w, rs);
                    const float2 sg = sigmoid_from_t(e.z, e.t);
                    const float2 sbx = mul2(mul2(s, be), xv);
                    ox = mul2(mul2(de, s), be);
                    ob = mul2(mul2(mul2(de, sbx), fma2(be, splat2(-1.f), splat2(1.f))), splat2(1.f));
                    // dg = delta (alpha h_{t-1} - beta x alpha^2 / s); 1/s is taken as 0 where s is
                    const float2 rz = make_float2(e.w.x < 1.17549435e-38f ? 0.f : rs.x, e.w.y < 1.17549435e-38f ? 0.f : rs.y);
                    const float2 m1 = mul2(e.alpha, hh);
                    const float2 m2 = mul2(mul2(mul2(be, xv), mul2(e.alpha, e.alpha)), rz);
                    const float2 ndg = mul2(de, fma2(m1, splat2(-1.f), m2));   // -dg
                    oa = mul2(mul2(ndg, ra), sg);
                    qA = fma2(mul2(ndg, ra), e.sp, qA);                        // dg g = -dg rate softplus(z)
                    qb = add2(qb, oa);
                    hh = add2(m1, sbx);
                    oal = e.alpha;
                };
                const bool live = t0 + r < d.T;
                const F4 de = live ? dl[r] : f4(0.f);
                pair(x.lo, a.lo, b.lo, bias.lo, rate.lo, de.lo, hs.lo, tA.lo, tb.lo, gx.lo, ga.lo, gb.lo, al1.lo);
                pair(x.hi, a.hi, b.hi, bias.hi, rate.hi, de.hi, hs.hi, tA.hi, tb.hi, gx.hi, ga.hi, gb.hi, al1.hi);
                if (live) {
                    store_row<T, TMA>((T *)p.dx + o + (int64_t)r * d.D, gx, nc);
                    store_row<T, TMA>((T *)p.da + o + (int64_t)r * d.D, ga, nc);
                    store_row<T, TMA>((T *)p.db + o + (int64_t)r * d.D, gb, nc);
                    if (starts >> r & 1 && p.dh0) store_words(p.dh0 + (int64_t)n0 * d.D + ch, mul4(al1, dl[r]), nc);
                }
            }
            sA[0] = add4(sA[0], tA);
            sb[0] = add4(sb[0], tb);
        }
        if ((k & 15) == 15) {
            sA[1] = add4(sA[1], sA[0]);
            sb[1] = add4(sb[1], sb[0]);
            sA[0] = sb[0] = f4(0.f);
        }
        __syncthreads();
    }
    // this CTA's sums: over the token groups, in order
    chain.agg[0][0][0].x = 0.f;   // (the scan's memory is free now)
    __syncthreads();
    float *red = (float *)&chain.agg[0][0][0];   // [NG][2][CH]
    static_assert(sizeof(chain.agg) >= sizeof(float) * Tile<T>::NG * 2 * Tile<T>::CH, "sums fit the scan's memory");
    {
        const int gi = warp * L::G + g;
        *(float4 *)&red[(gi * 2) * L::CH + q * 4] = to4(add4(sA[1], sA[0]));
        *(float4 *)&red[(gi * 2 + 1) * L::CH + q * 4] = to4(add4(sb[1], sb[0]));
    }
    __syncthreads();
    for (int i = tid; i < 2 * L::CH; i += kThreads) {
        const int which = i / L::CH, c = i % L::CH;
        if (slab * L::CH + c >= d.D) continue;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < L::NG; ++j) s += red[(j * 2 + which) * L::CH + c];
        p.part[(((int64_t)row * cs + rank) * 2 + which) * d.D + slab * L::CH + c] = s;
    }
    if (failed) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    if (TMA && tid == 0 && failed)
        for (int k = max(0, steps - 2); k < steps; ++k)
            if (k * (int)cs + (int)rank < p.ntiles) tc::mbar_wait(&full[k & 1], (k >> 1) & 1);
}

// The parameter gradients: part[parts][2][D] over its rows, 8 strided partial sums per channel.
__global__ void __launch_bounds__(256) rec_params_kernel(const RecProblem p, int parts) {
    __shared__ float red[2][8][32];
    const int c = blockIdx.x * 32 + threadIdx.x % 32, s = threadIdx.x / 32;
    if (*p.status == GDN_ERR_DEVICE_SEQLENS) return;
    float v[2] = {0.f, 0.f};
    if (c < p.d.D)
        for (int i = s; i < parts; i += 8) {
            v[0] += p.part[((int64_t)i * 2) * p.d.D + c];
            v[1] += p.part[((int64_t)i * 2 + 1) * p.d.D + c];
        }
    red[0][s][threadIdx.x % 32] = v[0];
    red[1][s][threadIdx.x % 32] = v[1];
    __syncthreads();
    if (s < 2 && c < p.d.D) {
        float t = 0.f;
        for (int i = 0; i < 8; ++i) t += red[s][i][threadIdx.x % 32];
        (s ? p.ddt_bias : p.dA_log)[c] = t;
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(128) rec_step_kernel(const RecProblem p, float *state) {
    const gdn_recurrence_desc &d = p.d;
    const int quads = (d.D + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (i >= (int64_t)d.B * quads) return;
    const int64_t n = i / quads;
    const int ch = (int)(i - n * quads) * 4, nc = min(4, d.D - ch);
    const F4 a = load_row<T, VEC>((const T *)p.a + n * d.a_stride_b + ch, nc);
    const F4 b = load_row<T, VEC>((const T *)p.b + n * d.b_stride_b + ch, nc);
    const F4 x = load_row<T, VEC>((const T *)p.x + n * d.x_stride_b + ch, nc);
    const F4 h0 = load_row<float, VEC>(state + n * d.D + ch, nc);
    const F4 bias = load_row<float, VEC>(p.dt_bias + ch, nc);
    F4 rate = load_row<float, VEC>(p.A_log + ch, nc);
    rate = {make_float2(expf(rate.lo.x), expf(rate.lo.y)), make_float2(expf(rate.hi.x), expf(rate.hi.y))};
    const Decay2 e0 = decay2(a.lo, bias.lo, rate.lo), e1 = decay2(a.hi, bias.hi, rate.hi);
    const F4 s = {mul2(e0.w, inv_sqrt2(e0.w)), mul2(e1.w, inv_sqrt2(e1.w))};
    const F4 h = fma4({e0.alpha, e1.alpha}, h0, mul4(mul4(s, {sigmoid2(b.lo), sigmoid2(b.hi)}), x));
    store_row<float, VEC>(state + n * d.D + ch, h, nc);
    store_row<T, VEC>((T *)p.out + n * d.D + ch, h, nc);
}

// ===================================================================== host
// CTAs per chain: as many as keep the chip filled (four CTAs per SM) and have a tile each. Clusters
// of 16 need an opt-in and are only used where 8 leave more than half of the SMs idle.
int cluster_size(int64_t chains, int64_t ntiles) {
    int cs = 1;
    while (cs < 8 && chains * cs * 2 <= 4 * kSms && cs < ntiles) cs *= 2;
    if (cs == 8 && chains * 16 <= kSms && ntiles > 8) cs = 16;
    return cs;
}
int tile_tokens(int dtype) { return dtype == GDN_F32 ? Tile<float>::TT : Tile<__half>::TT; }
int tile_channels(int dtype) { return dtype == GDN_F32 ? Tile<float>::CH : Tile<__half>::CH; }

struct RecPlan {
    int slabs, ntiles, cs;
    int64_t chains;
};
RecPlan make_plan(const gdn_recurrence_desc &d) {
    RecPlan r;
    r.slabs = (int)cdiv64(d.D, tile_channels(d.dtype));
    r.ntiles = (int)cdiv64(d.T, tile_tokens(d.dtype));
    r.chains = (int64_t)d.B * r.slabs;
    r.cs = cluster_size(r.chains, r.ntiles);
    return r;
}

template <typename K>
cudaError_t launch_chains(K kernel, const RecPlan &pl, size_t smem, cudaStream_t s, const RecProblem &p, const RecMaps &m) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && pl.cs > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pl.chains * pl.cs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)pl.cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, m);
}

// Whether [B, T, D] at these element strides can be fetched by TMA (16-byte aligned base and pitches).
bool tma_ok(const gdn_recurrence_desc &d, const void *p, int64_t sb, int64_t st) {
    const int64_t es = (int64_t)act_size(d.dtype);
    return ptr_aligned(p, 16) && (st * es) % 16 == 0 && (d.B == 1 || (sb > 0 && (sb * es) % 16 == 0)) &&
           st * es < (1ll << 40) && sb * es < (1ll << 40);
}
bool tma_map(CUtensorMap *m, const gdn_recurrence_desc &d, const void *p, int64_t sb, int64_t st) {
    const uint64_t es = act_size(d.dtype);
    const uint64_t pt = (uint64_t)st * es, pb = d.B == 1 ? (uint64_t)d.T * pt : (uint64_t)sb * es;
    return encode_token_map(m, d.dtype, p, d.B, d.T, d.D, pb, pt, tile_tokens(d.dtype), tile_channels(d.dtype));
}

template <typename T>
cudaError_t launch_forward(const RecProblem &p, const RecPlan &pl, cudaStream_t s) {
    const gdn_recurrence_desc &d = p.d;
    RecMaps m;
    memset(&m, 0, sizeof(m));
    const bool tma = d.T > 0 && (d.D * sizeof(T)) % 16 == 0 && ptr_aligned(p.out, 16) &&
                     tma_ok(d, p.x, d.x_stride_b, d.x_stride_t) && tma_ok(d, p.a, d.a_stride_b, d.a_stride_t) &&
                     tma_ok(d, p.b, d.b_stride_b, d.b_stride_t);
    if (!tma) return launch_chains(rec_forward_kernel<T, false>, pl, 0, s, p, m);
    if (!tma_map(&m.x, d, p.x, d.x_stride_b, d.x_stride_t) || !tma_map(&m.a, d, p.a, d.a_stride_b, d.a_stride_t) ||
        !tma_map(&m.b, d, p.b, d.b_stride_b, d.b_stride_t))
        return cudaErrorInvalidValue;
    return launch_chains(rec_forward_kernel<T, true>, pl, 2 * 3 * Tile<T>::kTensor, s, p, m);
}

template <typename T>
cudaError_t launch_backward_rec(const RecProblem &p, const RecPlan &pl, cudaStream_t s) {
    const gdn_recurrence_desc &d = p.d;
    RecMaps m;
    memset(&m, 0, sizeof(m));
    const bool tma = d.T > 0 && (d.D * sizeof(T)) % 16 == 0 && ptr_aligned(p.dx, 16) && ptr_aligned(p.da, 16) &&
                     ptr_aligned(p.db, 16) && ptr_aligned(p.grad_out, 16) && tma_ok(d, p.x, d.x_stride_b, d.x_stride_t) &&
                     tma_ok(d, p.a, d.a_stride_b, d.a_stride_t) && tma_ok(d, p.b, d.b_stride_b, d.b_stride_t);
    cudaError_t e;
    if (tma) {
        if (!tma_map(&m.x, d, p.x, d.x_stride_b, d.x_stride_t) || !tma_map(&m.a, d, p.a, d.a_stride_b, d.a_stride_t) ||
            !tma_map(&m.b, d, p.b, d.b_stride_b, d.b_stride_t) || !tma_map(&m.dy, d, p.grad_out, (int64_t)d.T * d.D, d.D))
            return cudaErrorInvalidValue;
        e = launch_chains(rec_backward_kernel<T, true>, pl, 2 * 4 * Tile<T>::kTensor, s, p, m);
    } else {
        e = launch_chains(rec_backward_kernel<T, false>, pl, 0, s, p, m);
    }
    if (e != cudaSuccess) return e;
    rec_params_kernel<<<(unsigned)cdiv64(d.D, 32), 256, 0, s>>>(p, d.B * pl.cs);
    return cudaGetLastError();
}

template <typename F>
int by_dtype(int dtype, F &&f) {
    switch (dtype) {
    case GDN_F32: return f((float)0);
    case GDN_BF16: return f(__nv_bfloat16());
    default: return f(__half());
    }
}

int check_desc(const gdn_recurrence_desc *d, bool packed) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->N < 1 || d->D < 1) return GDN_ERR_INVALID_ARG;
    if (packed ? d->B != 1 : d->N != d->B) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(d->dtype)) return GDN_ERR_UNSUPPORTED;
    const int64_t strides[] = {d->x_stride_b, d->x_stride_t, d->a_stride_b, d->a_stride_t, d->b_stride_b, d->b_stride_t};
    for (int64_t s : strides)
        if (s < 0) return GDN_ERR_INVALID_ARG;
    if (d->T > 1 && (d->x_stride_t < d->D || d->a_stride_t < d->D || d->b_stride_t < d->D)) return GDN_ERR_INVALID_ARG;
    if (cdiv64(d->D, 32) * d->B > (1ll << 30)) return GDN_ERR_UNSUPPORTED;   // the launch's grid
    if ((double)d->B * d->T * d->D > 4.0e12 || (double)d->N * d->D > 1.0e12) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

struct RecLayout {
    size_t status, part, cs, total;
};
RecLayout bwd_layout(const gdn_recurrence_desc &d) {
    RecLayout L;
    size_t off = 0;
    const size_t chunks = ((size_t)d.T + GDN_RECURRENCE_CHUNK - 1) / GDN_RECURRENCE_CHUNK;
    L.status = off; off += kStatusBytes;
    L.part = off;   off = align_up(off + (size_t)d.B * make_plan(d).cs * 2 * d.D * 4, 256);
    L.cs = off;     off = align_up(off + (size_t)d.B * chunks * d.D * 4, 256);
    L.total = off;
    return L;
}

bool act_aligned(int dtype, const void *p) { return ptr_aligned(p, act_size(dtype)); }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_recurrence_desc_init(gdn_recurrence_desc *d, int B, int T, int packed, int D, int dtype) {
    if (!d) return GDN_ERR_INVALID_ARG;
    memset(d, 0, sizeof(*d));
    d->B = B;
    d->T = T;
    d->N = packed ? packed : B;
    d->D = D;
    d->dtype = dtype;
    d->x_stride_t = d->a_stride_t = d->b_stride_t = D;
    d->x_stride_b = d->a_stride_b = d->b_stride_b = (int64_t)D * T;
    return check_desc(d, packed != 0);
}

int gdn_recurrence_workspace_bytes(const gdn_recurrence_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

int gdn_recurrence_backward_workspace_bytes(const gdn_recurrence_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = bwd_layout(*d).total;
    return GDN_OK;
}

int gdn_recurrence_forward(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b,
                           const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                           const float *initial_state, void *out, float *final_state, float *chunk_states,
                           void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d, cu_seqlens != nullptr);
    if (rc != GDN_OK) return rc;
    const bool tok = (int64_t)d->B * d->T > 0;   // token tensors may be empty (null)
    if ((tok && (!x || !a || !b || !out)) || !A_log || !dt_bias) return GDN_ERR_INVALID_ARG;
    if (!act_aligned(d->dtype, x) || !act_aligned(d->dtype, a) || !act_aligned(d->dtype, b) ||
        !act_aligned(d->dtype, out) || !ptr_aligned(A_log, 4) || !ptr_aligned(dt_bias, 4) ||
        !ptr_aligned(cu_seqlens, 4) || !ptr_aligned(initial_state, 4) || !ptr_aligned(final_state, 4) ||
        !ptr_aligned(chunk_states, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    RecProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.a = a;
    p.b = b;
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.cu = cu_seqlens;
    p.h0 = initial_state;
    p.out = out;
    p.hT = final_state;
    p.cs = chunk_states;
    p.status = (int32_t *)workspace;
    p.wait_immediate = wait_test_mode();
    const RecPlan pl = make_plan(*d);
    p.slabs = pl.slabs;
    p.ntiles = pl.ntiles;
    return by_dtype(d->dtype, [&](auto t) {
        return layer_status(launch_forward<decltype(t)>(p, pl, (cudaStream_t)stream));
    });
}

int gdn_recurrence_backward(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b,
                            const float *A_log, const float *dt_bias, const int32_t *cu_seqlens,
                            const float *initial_state, const float *chunk_states, const void *grad_out,
                            const float *grad_final, void *dx, void *da, void *db, float *dA_log, float *ddt_bias,
                            float *dinitial_state, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d, cu_seqlens != nullptr);
    if (rc != GDN_OK) return rc;
    const bool tok = (int64_t)d->B * d->T > 0;   // token tensors may be empty (null)
    if ((tok && (!x || !a || !b || !grad_out || !dx || !da || !db)) || !A_log || !dt_bias || !dA_log || !ddt_bias)
        return GDN_ERR_INVALID_ARG;
    const void *acts[] = {x, a, b, grad_out, dx, da, db};
    for (const void *q : acts)
        if (!act_aligned(d->dtype, q)) return GDN_ERR_INVALID_ARG;
    const void *words[] = {A_log, dt_bias, cu_seqlens, initial_state, chunk_states, grad_final, dA_log, ddt_bias, dinitial_state};
    for (const void *q : words)
        if (!ptr_aligned(q, 4)) return GDN_ERR_INVALID_ARG;
    const RecLayout L = bwd_layout(*d);
    if ((rc = check_workspace(workspace, workspace_bytes, L.total)) != GDN_OK) return rc;
    char *w = (char *)workspace;
    RecProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.a = a;
    p.b = b;
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.cu = cu_seqlens;
    p.h0 = initial_state;
    p.cs = chunk_states ? const_cast<float *>(chunk_states) : (float *)(w + L.cs);
    p.status = (int32_t *)workspace;
    p.part = (float *)(w + L.part);
    p.grad_out = grad_out;
    p.grad_final = grad_final;
    p.dx = dx;
    p.da = da;
    p.db = db;
    p.dA_log = dA_log;
    p.ddt_bias = ddt_bias;
    p.dh0 = dinitial_state;
    const cudaStream_t s = (cudaStream_t)stream;
    p.wait_immediate = wait_test_mode();
    const RecPlan pl = make_plan(*d);
    p.slabs = pl.slabs;
    p.ntiles = pl.ntiles;
    return by_dtype(d->dtype, [&](auto t) {
        using T = decltype(t);
        cudaError_t e = cudaSuccess;
        if (!chunk_states && d->T > 0) e = launch_forward<T>(p, pl, s);   // chunk states only
        return layer_status(e != cudaSuccess ? e : launch_backward_rec<T>(p, pl, s));
    });
}

int gdn_recurrence_step(const gdn_recurrence_desc *d, const void *x, const void *a, const void *b, const float *A_log,
                        const float *dt_bias, float *state, void *out, gdn_stream_t stream) {
    int rc = check_desc(d, false);
    if (rc != GDN_OK) return rc;
    if (d->T != 1) return GDN_ERR_INVALID_ARG;
    if (!x || !a || !b || !A_log || !dt_bias || !state || !out) return GDN_ERR_INVALID_ARG;
    if (!act_aligned(d->dtype, x) || !act_aligned(d->dtype, a) || !act_aligned(d->dtype, b) ||
        !act_aligned(d->dtype, out) || !ptr_aligned(A_log, 4) || !ptr_aligned(dt_bias, 4) || !ptr_aligned(state, 4))
        return GDN_ERR_INVALID_ARG;
    RecProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.a = a;
    p.b = b;
    p.A_log = A_log;
    p.dt_bias = dt_bias;
    p.out = out;
    return by_dtype(d->dtype, [&](auto t) {
        using T = decltype(t);
        const size_t row = 4 * sizeof(T);
        const bool vec = d->D % 4 == 0 && ptr_aligned(x, row) && ptr_aligned(a, row) && ptr_aligned(b, row) &&
                         ptr_aligned(out, row) && ptr_aligned(A_log, 16) && ptr_aligned(dt_bias, 16) &&
                         ptr_aligned(state, 16) &&
                         (d->B == 1 || (d->x_stride_b % 4 == 0 && d->a_stride_b % 4 == 0 && d->b_stride_b % 4 == 0));
        const unsigned grid = (unsigned)cdiv64((int64_t)d->B * cdiv64(d->D, 4), 128);
        if (vec) rec_step_kernel<T, true><<<grid, 128, 0, (cudaStream_t)stream>>>(p, state);
        else rec_step_kernel<T, false><<<grid, 128, 0, (cudaStream_t)stream>>>(p, state);
        return layer_status(cudaGetLastError());
    });
}

}  // extern "C"
