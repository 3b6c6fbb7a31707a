// gdn_window_dq_tc.cu -- dq of two heads that share keys and values (include/gdn.h: the
// window attention's backward), on the tensor cores.
//
// One CTA keeps 128 queries of both heads (Q_i, dO_i) and walks over tiles of 64 keys:
//   S = Q K^T, dP = dO V^T, P = exp2(c S - lse), dS = P (dP - delta), dQ += dS K (scale
//   taken out of the sums, fp16 in units: gdn_window_tc.cuh)
// dS takes the place of dP in tensor memory, from where it is an operand of the second product.
// Each head has a warpgroup of its own, a thread per query: while one's dS is computed the
// tensor cores work on the other's products. Four tiles that stay and three stages of K and V
// are all the shared memory, so tiles have 64 keys, at which the scores run at about half the
// tensor cores' rate; against the one-head kernel (gdn_window_bwd_tc.cu) a CTA's start and end,
// about 8000 cycles, are shared by two heads and K and V are read once.
//
// Which of the two, for heads that come in pairs: the whole backward of 16384 tokens of 16
// heads on 8, us with pairs | without, by window:
//   128 channels:  128: 255 | 280   512: 370 | 388   1024: 525 | 534   2048: 804 | 792   8192: 2064 | 2009
//    64 channels:  128: 197 | 228   512: 294 | 326   1024: 419 | 461   2048: 645 | 699   8192: 1679 | 1787
#include <string.h>

#include <algorithm>

#include "gdn_window_tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kThreads = 384;   // warps 0 TMA, 1 MMA, 2-3 rows behind a sequence, 4-7 and 8-11 dS of a head each
constexpr int kStages = 3;      // of the tiles of keys and values

template <int D> struct PairShape {
    static constexpr int kRowA = 128 * 128, kRowB = 64 * 128;   // bytes of 128 (64) rows x 64 channels
    static constexpr int kA = D / 64 * kRowA, kB = D / 64 * kRowB;
    static constexpr int kBs = 4 * kA;                          // behind Q and dO of the first head, then of the second
    static constexpr int kBytes = kBs + kStages * 2 * kB + 1024;
    static constexpr uint32_t kAcc = 256;   // TMEM columns: head b's S at 128 b, dP at 128 b + 64; dQ from here, D each
};

struct PairShared {
    uint64_t a_full, full[kStages], empty[kStages], fit[kStages], s_full[2], ready[2], acc_full, drain;
    uint32_t tmem;
    int gave_up;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) window_dq_pair(const __grid_constant__ WindowMaps a_maps, const __grid_constant__ WindowMaps b_maps,
                                                              const __grid_constant__ WindowProblem p) {
    using L = PairShape<D>;
    extern __shared__ unsigned char smraw[];
    __shared__ PairShared sh;
    unsigned char *sm = (unsigned char *)(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    const gdn_window_attention_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) tma_prefetch_map(&a_maps.q), tma_prefetch_map(&a_maps.g), tma_prefetch_map(&b_maps.k), tma_prefetch_map(&b_maps.v);

    // ---- the CTA's place; later queries, which see the most, first
    const int units = d.Hq / 2, slot = (int)blockIdx.x / units, head0 = 2 * ((int)blockIdx.x - slot * units), hk = head0 / (d.Hq / d.Hk);
    int n, tile;
    if (p.cu) {
        const int32_t status = *p.status, tiles = p.q_tiles[d.N];   // on their way with the search's
        n = warp_upper_index(p.q_tiles, d.N, slot);
        if (status == GDN_ERR_DEVICE_SEQLENS || slot >= tiles) return;
        tile = p.q_tiles[n + 1] - 1 - slot;
    } else {
        const int per = (d.Tq + 127) / 128;
        n = slot / per;
        tile = per - 1 - (slot - n * per);
    }
    const WindowSpan sp = window_span(p, n);
    const int past = sp.Lk - sp.Lq, row0 = tile * 128, rows = min(128, sp.Lq - row0);

    // ---- the tiles of 64 keys: those of the sinks, then the window's
    int first = 0, sinks64 = 0, count = 0;
    const int p1 = past + row0 + rows - 1;
    if (p1 >= 0) {
        const int lo = window_first(max(past + row0, 0), d.window);
        first = lo >> 6;
        sinks64 = min((int)(((int64_t)min(d.sinks, lo) + 63) >> 6), first);
        count = sinks64 + (p1 >> 6) - first + 1;
    }
    auto row_at = [&](int it) { return (it < sinks64 ? it : first + it - sinks64) * 64; };

    const int qrow = p.cu ? (int)sp.q0 : 0, krow = p.cu ? (int)sp.k0 : 0;
    const int qb = p.cu ? 0 : n * a_maps.q_rows, kb = p.cu ? 0 : n * a_maps.k_rows, vb = p.cu ? 0 : n * a_maps.v_rows, gb = p.cu || d.B == 1 ? 0 : n;
    auto load = [&](int it) {   // the it-th tile's keys and values
        const int i = it % kStages, r = row_at(it);
        unsigned char *b1 = sm + L::kBs + i * 2 * L::kB, *b2 = b1 + L::kB;
        mbar_expect_tx(&sh.full[i], 2 * L::kB);
        for (int b = 0; b < D / 64; ++b) {
            tma_load_4d(b1 + b * L::kRowB, &b_maps.k, 64 * b, hk, krow + r, kb, &sh.full[i]);
            tma_load_4d(b2 + b * L::kRowB, &b_maps.v, 64 * b, hk, krow + r, vb, &sh.full[i]);
        }
    };
    if (tid == 0) {
        mbar_init(&sh.a_full, 1);
        for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1), mbar_init(&sh.fit[i], 2);
        for (int b = 0; b < 2; ++b) mbar_init(&sh.s_full[b], 1), mbar_init(&sh.ready[b], 4);
        mbar_init(&sh.acc_full, 1), mbar_init(&sh.drain, 1);
        sh.gave_up = 0;
        mbar_init_fence();
        if (count > 0) {   // the first copies are on their way while the CTA gets its tensor memory
            fence_async_smem();
            mbar_expect_tx(&sh.a_full, 4 * L::kA);
            for (int s = 0; s < 2; ++s)
                for (int b = 0; b < D / 64; ++b) {
                    tma_load_4d(sm + 2 * s * L::kA + b * L::kRowA, &a_maps.q, 64 * b, head0 + s, qrow + row0, qb, &sh.a_full);
                    tma_load_4d(sm + (2 * s + 1) * L::kA + b * L::kRowA, &a_maps.g, 64 * b, head0 + s, qrow + row0, gb, &sh.a_full);
                }
            load(0);
        }
    }
    if (warp == 1) tmem_alloc(&sh.tmem, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tbase = sh.tmem;
    const WindowWait wait{&sh.gave_up, p.wait_immediate != 0};
    constexpr bool kHalf = std::is_same<T, __half>::value;
    const uint32_t idesc_s = kHalf ? idesc_f16(128, 64, false, false) : idesc_bf16(128, 64, false, false);
    const uint32_t idesc_a = kHalf ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0 && count > 0) {
            int it = 1;
            for (; it < count; ++it) {
                if (it >= kStages && !wait(&sh.empty[it % kStages], (uint32_t)(it / kStages - 1) & 1)) break;
                load(it);
            }
            // what is in flight lands before the CTA leaves
            mbar_wait(&sh.a_full, 0);
            for (int u = max(0, it - kStages); u < it; ++u) mbar_wait(&sh.full[u % kStages], (uint32_t)(u / kStages) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const int total = of_warp(count);
        if (total > 0) {
            const uint32_t leader = elect_one(), tb = (uint32_t)of_warp((int)tbase), base = (uint32_t)of_warp((int)smem_u32(sm));
            const uint64_t a1 = sw128_desc(base, 0, 1024), bk = sw128_desc(base + L::kBs, 0, 1024), bn = sw128_desc(base + L::kBs, L::kRowB, 1024);
            int si = 0, pi = 0;        // stages of the next scores and of the next sums
            uint32_t sph = 0;
            auto scores = [&](int b) {   // S and dP of head b
                const uint64_t q = a1 + (uint32_t)(2 * b * (L::kA >> 4)), k = bk + (uint32_t)(si * (2 * L::kB >> 4));
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t aa = ((i >> 2) * L::kRowA + (i & 3) * 32 + x * L::kA) >> 4, ab = ((i >> 2) * L::kRowB + (i & 3) * 32 + x * L::kB) >> 4;
                        warp_mma_f16(leader, tb + 128 * b + 64 * x, q + aa, k + ab, idesc_s, i > 0);
                    }
                warp_mma_commit(leader, &sh.s_full[b]);
            };
            auto sums = [&](int b, uint32_t more) {   // dQ += dS K
                const uint64_t k = bn + (uint32_t)(pi * (2 * L::kB >> 4));
                const uint32_t from = tb + 128 * b + 64, acc = tb + L::kAcc + D * b;
                warp_mma_f16_ta(leader, acc, from, k, idesc_a, more);
#pragma unroll
                for (int i = 1; i < 4; ++i) warp_mma_f16_ta(leader, acc, from + 8 * i, k + (uint32_t)(2048 * i >> 4), idesc_a, 1);
            };
            auto here = [&]() -> bool {   // the next tile of keys
                const bool come = warp_wait2(wait, &sh.full[si], sph, &sh.fit[si], sph);
                fence_after_sync();
                return come;
            };
            auto scored = [&] {
                if (++si == kStages) si = 0, sph ^= 1;
            };
            bool ok = warp_wait(wait, &sh.a_full, 0) && here();
            if (ok) scores(0), scores(1), scored();
            for (int it = 0; ok && it < total; ++it) {
                const bool more = it + 1 < total;
                ok = !more || here();
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    ok = ok && warp_wait(wait, &sh.ready[b], (uint32_t)it & 1);
                    fence_after_sync();
                    if (ok) sums(b, it > 0);
                    if (ok && more) scores(b);
                }
                if (!ok) break;
                warp_mma_commit(leader, &sh.empty[pi]);
                if (++pi == kStages) pi = 0;
                if (more) scored();
            }
            if (ok) warp_mma_commit(leader, &sh.acc_full);
            warp_mma_commit(leader, &sh.drain);
            mbar_wait(&sh.drain, 0);
        }
    } else if (warp < 4) {
        // -------------------------- zeros in rows behind the sequence (0 x NaN is NaN), a warp each for K and V
        const int w = warp - 2;
        for (int it = 0; it < count; ++it) {
            const int i = it % kStages, left = sp.Lk - row_at(it);
            if (left < 64) {
                if (!warp_wait(wait, &sh.full[i], (uint32_t)(it / kStages) & 1)) break;
                unsigned char *t = sm + L::kBs + i * 2 * L::kB + w * L::kB;
                for (int b = 0; b < D / 64; ++b)
                    for (int x = left * 8 + lane; x < 64 * 8; x += 32) *(uint4 *)(t + b * L::kRowB + 16 * x) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.fit[i]);
            // one arrival for each use of the stage: never ahead of the products by a whole round
            if (it >= kStages - 1 && it + 1 < count && !warp_wait(wait, &sh.empty[(it + 1) % kStages], (uint32_t)((it + 1) / kStages - 1) & 1)) break;
        }
    } else {
        // ------------------------------------------------------------ dS
        const int b = (warp - 4) >> 2, r = tid & 127, head = head0 + b;
        const uint32_t ts = tbase + 128 * b + ((uint32_t)(warp & 3) << 21);
        const float c = d.scale * 1.4426950408889634f;
        const int64_t ntok = (int64_t)d.B * d.Tq;
        const float up = grad_factor<T>(p, n, hk);
        float lse = 0.0f, delta = 0.0f;
        if (r < rows) {
            lse = fmaf(p.lse[head * ntok + sp.q0 + row0 + r], 1.4426950408889634f, -(float)kWeightBits<T>);
            delta = p.delta[head * ntok + sp.q0 + row0 + r] * up;
        }
        bool ok = true;
        for (int it = 0; it < count; ++it) {
            const int r0 = row_at(it);
            // the keys that this query sees
            uint32_t see[2];
            {
                const int64_t pos = past + row0 + r, lo = pos - d.window + 1 - r0, hi = pos + 1 - r0, sk = d.sinks - r0;
                const int l = (int)max((int64_t)0, min((int64_t)64, lo)), h = (int)max((int64_t)0, min((int64_t)64, hi)),
                          k = (int)max((int64_t)0, min((int64_t)64, sk));
#pragma unroll
                for (int w = 0; w < 2; ++w) see[w] = low_bits(h - 32 * w) & (~low_bits(l - 32 * w) | low_bits(k - 32 * w));
            }
            if (!(ok = warp_wait(wait, &sh.s_full[b], (uint32_t)it & 1))) break;
            fence_after_sync();
            const bool all = __all_sync(0xffffffffu, (see[0] & see[1]) == 0xffffffffu);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float s[32], g[32], f[16];
                tmem_ld32x2(ts + 32 * w, ts + 64 + 32 * w, s, g);
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    float2 t = fma2(make_float2(s[x], s[x + 1]), splat2(c), splat2(-lse));
                    t = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                    float2 u = mul2(t, fma2(make_float2(g[x], g[x + 1]), splat2(up), splat2(-delta)));
                    if (!all) u.x = see[w] & (1u << x) ? u.x : 0.0f, u.y = see[w] & (2u << x) ? u.y : 0.0f;
                    f[x / 2] = __uint_as_float(pack2<T>(u.x, u.y));
                }
                tmem_st16_nw(ts + 64 + 16 * w, f);   // over columns that have been read
            }
            tmem_wait_st();
            warp_arrive(&sh.ready[b]);
        }
        if (count > 0) {
            if (ok) ok = warp_wait(wait, &sh.acc_full, 0);
            fence_after_sync();
        }
        // ---- dQ, through the head's own Q in shared memory (no product reads it any more)
        const uint32_t from = tbase + L::kAcc + b * D + ((uint32_t)(warp & 3) << 21);
        unsigned char *stage = sm + b * 2 * L::kA;
        const float2 back = splat2(sees_one((int64_t)past + row0 + r, d.window, d.sinks) ? 0.0f : d.scale * kWeightUnit<T> / up);   // out of the operands' units
#pragma unroll
        for (int q = 0; q < D; q += 32) {
            float o[32];
            if (count > 0) {
                tmem_ld32(from + q, o);
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    const float2 s = mul2(make_float2(o[x], o[x + 1]), back);
                    o[x] = s.x, o[x + 1] = s.y;
                }
            } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = 0.0f;
            }
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
                const int ch = (q + x) >> 3;
                *(uint4 *)(stage + (ch >> 3) * L::kRowA + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                    make_uint4(pack2<T>(o[x], o[x + 1]), pack2<T>(o[x + 2], o[x + 3]), pack2<T>(o[x + 4], o[x + 5]), pack2<T>(o[x + 6], o[x + 7]));
            }
        }
        __syncwarp();
        const int w0 = r & ~31, n_rows = ok ? max(0, min(32, rows - w0)) : 0;
        T *out = (T *)p.dq + ((sp.q0 + row0 + w0) * d.Hq + head) * (int64_t)d.d;
#pragma unroll
        for (int x = lane; x < 32 * (D / 8); x += 32) {
            const int q = x / (D / 8), ch = x % (D / 8);
            if (q < n_rows && 8 * ch < d.d)
                *(uint4 *)(out + (int64_t)q * d.Hq * d.d + 8 * ch) =
                    *(const uint4 *)(stage + (ch >> 3) * L::kRowA + (w0 + q) * 128 + (((ch & 7) ^ ((w0 + q) & 7)) << 4));
        }
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && sh.gave_up) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    if (warp == 1) tmem_dealloc(tbase, 512);
}

template <typename T, int D>
cudaError_t launch_pair(const WindowMaps &wide, const WindowProblem &p, cudaStream_t s) {
    const gdn_window_attention_desc &d = p.d;
    WindowMaps slim;
    memset(&slim, 0, sizeof(slim));
    if (!window_head_map(&slim.k, d, p.k, d.Hk, d.Tk, d.k_stride_b, d.k_stride_t, &slim.k_rows, 64) ||
        !window_head_map(&slim.v, d, p.v, d.Hk, d.Tk, d.v_stride_b, d.v_stride_t, &slim.v_rows, 64))
        return cudaErrorInvalidValue;
    const int64_t blocks = (p.cu ? cdiv64(d.Tq, 128) + d.N : (int64_t)d.B * cdiv64(d.Tq, 128)) * (d.Hq / 2);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    constexpr size_t smem = PairShape<D>::kBytes > 117 * 1024 ? PairShape<D>::kBytes : 117 * 1024;   // one CTA per SM: each holds all of the tensor memory
    const cudaError_t a = allow_shared(window_dq_pair<T, D>, smem);
    if (a != cudaSuccess) return a;
    window_dq_pair<T, D><<<(unsigned)blocks, kThreads, smem, s>>>(wide, slim, p);
    return cudaGetLastError();
}

}  // namespace

// by the times at the top of this file; 1536 lies between the two windows where the order changes
bool window_dq_pairs(const gdn_window_attention_desc &d) { return d.Hq / d.Hk % 2 == 0 && (d.d <= 64 || std::min(d.window, d.Tk) <= 1536); }

cudaError_t launch_window_dq_pair(const WindowMaps &wide, const WindowProblem &p, cudaStream_t s) {
    if (p.d.d <= 64) return p.d.dtype == GDN_BF16 ? launch_pair<__nv_bfloat16, 64>(wide, p, s) : launch_pair<__half, 64>(wide, p, s);
    return p.d.dtype == GDN_BF16 ? launch_pair<__nv_bfloat16, 128>(wide, p, s) : launch_pair<__half, 128>(wide, p, s);
}

}  // namespace gdn
