// gdn_window_bwd_tc.cu -- the window attention's backward on the tensor cores
// (include/gdn.h), for 16-bit types and heads of up to 128 channels.
//
// Two kernels of one shape, so that every sum has a fixed order (no atomics): one CTA keeps
// 128 rows and walks over tiles of 64 rows of the other side.
//   keys:    K_j, V_j stay; per head of the group and tile of queries
//            S' = K Q^T, dP' = V dO^T, P' = exp2(c S' - lse), dS' = P' (dP' - delta) scale,
//            dV += P' dO, dK += dS' Q
//   queries: Q_i, dO_i stay; per tile of keys  S, dP as above (not transposed), dQ += dS K;
//            of two heads that share keys and values where the group's size is even
// P and dS take the place of S and dP in tensor memory, from where they are operands of the
// second pair of products. Two such buffers, each with a warpgroup of its own (a thread per
// row), for tiles by turns or for the two heads: while one's P and dS are computed the tensor
// cores work on the other's products.
// Seven products instead of five recompute S and dP, which is the price of no atomics.
//
// Keys below `sinks` are seen by all later queries. A CTA of keys takes the queries within the
// window; what lies beyond is cut into chunks of about the same work, whose sums (of the sinks'
// rows, fp32) a last kernel adds up in order.
#include <string.h>

#include <algorithm>

#include "gdn_window_rest.cuh"
#include "gdn_window_tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kThreads = 384;   // warps 0 TMA, 1 MMA, 2-3 statistics and rows behind a sequence, 4-7 and 8-11 P and dS
template <int D, bool PAIR> struct BwdShape {
    static constexpr int kStages = PAIR ? 3 : 4, kHold = PAIR ? 2 : 1;   // stages of the walked side; pairs of tiles that stay
    static constexpr int kRowA = 128 * 128, kRowB = 64 * 128;   // bytes of 128 (64) rows x 64 channels
    static constexpr int kA = D / 64 * kRowA, kB = D / 64 * kRowB;
    static constexpr int kA1 = 0, kA2 = kA, kBs = kHold * 2 * kA, kEnd = kBs + kStages * 2 * kB;
    static constexpr int kBytes = kEnd + 1024;
    static constexpr uint32_t kAcc = 256;   // TMEM columns: buffer b's S at 128 b, dP at 128 b + 64; sums from here, D each
};

template <bool KEYS> struct BwdShared {
    uint64_t a_full, full[4], empty[4], fit[4], s_full[2], p_ready[2], acc_full, drain;
    uint32_t tmem;
    int gave_up;
    float lse[KEYS ? 4 : 1][64], delta[KEYS ? 4 : 1][64];   // of the tile's queries: lse log2 e, delta scale
};

template <typename T, int D, bool KEYS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) window_backward_tc(const __grid_constant__ WindowMaps a_maps, const __grid_constant__ WindowMaps b_maps,
                                                                  const __grid_constant__ WindowProblem p, int units, int64_t rest_blocks) {
    using L = BwdShape<D, PAIR>;
    constexpr int kStages = L::kStages;
    extern __shared__ unsigned char smraw[];
    __shared__ BwdShared<KEYS> sh;
    unsigned char *sm = (unsigned char *)(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    const gdn_window_attention_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (*p.status == GDN_ERR_DEVICE_SEQLENS) return;

    // ---- the CTA's place
    const int group = d.Hq / d.Hk;
    const bool rest = KEYS && blockIdx.x < rest_blocks;
    const int64_t block = rest ? blockIdx.x : blockIdx.x - rest_blocks;
    const int unit = (int)(block % units);                 // keys: head of k and v; queries: head of q, or two of a group
    const int64_t slot = block / units;
    int n, tile, chunk = 0;
    const int32_t *table = rest ? p.rest_off : KEYS ? p.k_tiles : p.q_tiles;
    if (p.cu) {
        if (slot >= table[d.N]) return;
        n = upper_index(table, d.N, slot);
        tile = (int)(slot - table[n]);
    } else {
        const int per = rest ? p.rest_per : ((KEYS ? d.Tk : d.Tq) + 127) / 128;
        n = (int)(slot / per);
        tile = (int)(slot - (int64_t)n * per);
    }
    const WindowSpan sp = window_span(p, n);
    const int past = sp.Lk - sp.Lq;
    if (rest) {   // `tile` counts the sequence's chunks so far
        chunk = tile;
        for (tile = 0; tile < p.sink_tiles; ++tile) {
            const int c = rest_chunks(p, sp, tile);
            if (chunk < c) break;
            chunk -= c;
        }
        if (tile >= p.sink_tiles) return;
    } else if (!KEYS && p.cu == nullptr) {
        tile = (d.Tq + 127) / 128 - 1 - tile;              // later queries, which see the most, first
    } else if (!KEYS) {
        tile = p.q_tiles[n + 1] - p.q_tiles[n] - 1 - tile;
    }
    const int head0 = PAIR ? 2 * unit : unit, hk = KEYS ? unit : head0 / group;
    const int row0 = tile * 128, rows = min(128, (KEYS ? sp.Lk : sp.Lq) - row0);   // the rows that stay

    // ---- what it walks over: `count` tiles of 64 rows
    int first = 0, per_head = 0, sinks64 = 0, count;
    if (KEYS) {
        if (rest) {
            const SinkRest r = sink_rest(sp.Lq, sp.Lk, tile, d.window);
            first = r.e0, per_head = r.tiles;
            count = (int)min((int64_t)p.rest_its, (int64_t)per_head * group - (int64_t)chunk * p.rest_its);
        } else {
            const int64_t lo = max((int64_t)0, (int64_t)row0 - past);
            const int64_t hi = min((int64_t)sp.Lq - 1, (int64_t)row0 + rows - 1 + d.window - 1 - past);
            if (hi >= lo) first = (int)(lo >> 6), per_head = (int)((hi >> 6) - (lo >> 6) + 1);
            count = per_head * group;
        }
    } else {
        const int p1 = past + row0 + rows - 1;
        if (p1 < 0) {
            count = 0;
        } else {
            const int lo = window_first(max(past + row0, 0), d.window);
            first = lo >> 6;
            sinks64 = min((int)(((int64_t)min(d.sinks, lo) + 63) >> 6), first);
            count = sinks64 + (p1 >> 6) - first + 1;
        }
    }
    // tile `it`: its head of queries and its first row
    auto head_at = [&](int it) { return KEYS ? hk * group + (int)(((int64_t)chunk * p.rest_its + it) / per_head) : head0; };
    auto row_at = [&](int it) {
        if (KEYS) return (first + (int)(((int64_t)chunk * p.rest_its + it) % per_head)) * 64;
        return (it < sinks64 ? it : first + it - sinks64) * 64;
    };
    const int other = KEYS ? sp.Lq : sp.Lk;                // rows of the side walked over

    if (tid == 0) {
        mbar_init(&sh.a_full, 1);
        for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 1), mbar_init(&sh.fit[i], 2);
        for (int b = 0; b < 2; ++b) mbar_init(&sh.s_full[b], 1), mbar_init(&sh.p_ready[b], 4);
        mbar_init(&sh.acc_full, 1), mbar_init(&sh.drain, 1);
        sh.gave_up = 0;
        mbar_init_fence();
    }
    if (warp == 0) tmem_alloc(&sh.tmem, 512);
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
            // maps: q (of keys: of the walked side) and g (grad_out), k and v
            const int64_t qrow = p.cu ? sp.q0 : 0, krow = p.cu ? sp.k0 : 0;
            const int qb = p.cu ? 0 : n * a_maps.q_rows, kb = p.cu ? 0 : n * a_maps.k_rows, vb = p.cu ? 0 : n * a_maps.v_rows;
            const int gb = p.cu || d.B == 1 ? 0 : n;
            mbar_expect_tx(&sh.a_full, L::kHold * 2 * L::kA);
            for (int b = 0; b < D / 64; ++b) {
                if (KEYS) {
                    tma_load_4d(sm + L::kA1 + b * L::kRowA, &a_maps.k, 64 * b, hk, (int)(krow + row0), kb, &sh.a_full);
                    tma_load_4d(sm + L::kA2 + b * L::kRowA, &a_maps.v, 64 * b, hk, (int)(krow + row0), vb, &sh.a_full);
                } else {
                    for (int s = 0; s < L::kHold; ++s) {
                        tma_load_4d(sm + s * 2 * L::kA + L::kA1 + b * L::kRowA, &a_maps.q, 64 * b, head0 + s, (int)(qrow + row0), qb, &sh.a_full);
                        tma_load_4d(sm + s * 2 * L::kA + L::kA2 + b * L::kRowA, &a_maps.g, 64 * b, head0 + s, (int)(qrow + row0), gb, &sh.a_full);
                    }
                }
            }
            int it = 0;
            for (; it < count; ++it) {
                const int i = it % kStages;
                if (it >= kStages && !wait(&sh.empty[i], (uint32_t)(it / kStages - 1) & 1)) break;
                unsigned char *b1 = sm + L::kBs + i * 2 * L::kB, *b2 = b1 + L::kB;
                const int h = head_at(it), r = row_at(it);
                mbar_expect_tx(&sh.full[i], 2 * L::kB);
                for (int b = 0; b < D / 64; ++b) {
                    if (KEYS) {
                        tma_load_4d(b1 + b * L::kRowB, &b_maps.q, 64 * b, h, (int)(qrow + r), qb, &sh.full[i]);
                        tma_load_4d(b2 + b * L::kRowB, &b_maps.g, 64 * b, h, (int)(qrow + r), gb, &sh.full[i]);
                    } else {
                        tma_load_4d(b1 + b * L::kRowB, &b_maps.k, 64 * b, hk, (int)(krow + r), kb, &sh.full[i]);
                        tma_load_4d(b2 + b * L::kRowB, &b_maps.v, 64 * b, hk, (int)(krow + r), vb, &sh.full[i]);
                    }
                }
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
            const uint64_t a1 = sw128_desc(base + L::kA1, 0, 1024), a2 = sw128_desc(base + L::kA2, 0, 1024),
                           bk = sw128_desc(base + L::kBs, 0, 1024), bn = sw128_desc(base + L::kBs, L::kRowB, 1024);
            int si = 0, pi = 0;        // stages of the next scores and of the next sums
            uint32_t sph = 0;
            auto scores = [&](int b) {   // into buffer b; with pairs of the b-th head
                const uint32_t hold = PAIR ? (uint32_t)(b * (2 * L::kA >> 4)) : 0u;
                const uint64_t s1 = bk + (uint32_t)(si * (2 * L::kB >> 4)), s2 = s1 + (uint32_t)(L::kB >> 4);
                const uint32_t to = tb + 128 * b;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t aa = ((i >> 2) * L::kRowA + (i & 3) * 32) >> 4, ab = ((i >> 2) * L::kRowB + (i & 3) * 32) >> 4;
                    warp_mma_f16(leader, to, a1 + hold + aa, s1 + ab, idesc_s, i > 0);
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t aa = ((i >> 2) * L::kRowA + (i & 3) * 32) >> 4, ab = ((i >> 2) * L::kRowB + (i & 3) * 32) >> 4;
                    warp_mma_f16(leader, to + 64, a2 + hold + aa, s2 + ab, idesc_s, i > 0);
                }
                warp_mma_commit(leader, &sh.s_full[b]);
            };
            auto sums = [&](int b, uint32_t more) {
                const uint64_t s1 = bn + (uint32_t)(pi * (2 * L::kB >> 4)), s2 = s1 + (uint32_t)(L::kB >> 4);
                const uint32_t from = tb + 128 * b, acc = tb + L::kAcc + (PAIR ? D * b : 0);
                if (KEYS) {   // dV += P dO
                    warp_mma_f16_ta(leader, acc + D, from, s2, idesc_a, more);
#pragma unroll
                    for (int i = 1; i < 4; ++i) warp_mma_f16_ta(leader, acc + D, from + 8 * i, s2 + (uint32_t)(2048 * i >> 4), idesc_a, 1);
                }
                warp_mma_f16_ta(leader, acc, from + 64, s1, idesc_a, more);   // dK += dS Q, dQ += dS K
#pragma unroll
                for (int i = 1; i < 4; ++i) warp_mma_f16_ta(leader, acc, from + 64 + 8 * i, s1 + (uint32_t)(2048 * i >> 4), idesc_a, 1);
            };
            auto here = [&]() -> bool {   // the next tile of the walked side
                const bool come = warp_wait2(wait, &sh.full[si], sph, &sh.fit[si], sph);
                fence_after_sync();
                return come;
            };
            auto scored = [&] {
                if (++si == kStages) si = 0, sph ^= 1;
            };
            auto summed = [&] {
                warp_mma_commit(leader, &sh.empty[pi]);
                if (++pi == kStages) pi = 0;
            };
            bool ok = warp_wait(wait, &sh.a_full, 0);
            if (PAIR) {   // every tile for both heads
                ok = ok && here();
                if (ok) scores(0), scores(1), scored();
                for (int it = 0; ok && it < total; ++it) {
                    const bool more = it + 1 < total;
                    ok = !more || here();
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        ok = ok && warp_wait(wait, &sh.p_ready[b], (uint32_t)it & 1);
                        fence_after_sync();
                        if (ok) sums(b, it > 0);
                        if (ok && more) scores(b);
                    }
                    if (!ok) break;
                    summed();
                    if (more) scored();
                }
            } else {      // tiles by turns
                for (int b = 0; ok && b < 2 && b < total; ++b) {
                    ok = here();
                    if (ok) scores(b), scored();
                }
                for (int it = 0; ok && it < total; ++it) {
                    const int b = it & 1;
                    ok = warp_wait(wait, &sh.p_ready[b], (uint32_t)(it >> 1) & 1);
                    if (!ok) break;
                    fence_after_sync();
                    sums(b, it > 0);
                    summed();
                    if (it + 2 < total) {
                        ok = here();
                        if (ok) scores(b), scored();
                    }
                }
            }
            if (ok) warp_mma_commit(leader, &sh.acc_full);
            warp_mma_commit(leader, &sh.drain);
            mbar_wait(&sh.drain, 0);
        }
    } else if (warp < 4) {
        // -------------------------- the queries' statistics, and zeros in rows behind the sequence (0 x NaN is NaN)
        const int w = warp - 2;
        const int64_t ntok = (int64_t)d.B * d.Tq;
        for (int it = 0; it < count; ++it) {
            const int i = it % kStages, r0 = row_at(it), left = other - r0;
            if (KEYS) {
                float l = 0.0f, dl = 0.0f;
                const int x = 32 * w + lane;
                if (x < left) {
                    const int64_t at = head_at(it) * ntok + sp.q0 + r0 + x;
                    l = p.lse[at] * 1.4426950408889634f, dl = p.delta[at] * d.scale;
                }
                if (it >= kStages && !warp_wait(wait, &sh.empty[i], (uint32_t)(it / kStages - 1) & 1)) break;
                sh.lse[i][x] = l, sh.delta[i][x] = dl;
            }
            if (left < 64) {
                if (!warp_wait(wait, &sh.full[i], (uint32_t)(it / kStages) & 1)) break;
                unsigned char *t = sm + L::kBs + i * 2 * L::kB + w * L::kB;   // a warp for each of the two
                for (int b = 0; b < D / 64; ++b)
                    for (int x = left * 8 + lane; x < 64 * 8; x += 32) *(uint4 *)(t + b * L::kRowB + 16 * x) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.fit[i]);
            // one arrival for each use of the stage: never ahead of the products by a whole round
            if (!KEYS && it >= kStages - 1 && it + 1 < count && !warp_wait(wait, &sh.empty[(it + 1) % kStages], (uint32_t)((it + 1) / kStages - 1) & 1)) break;
        }
    } else {
        // ------------------------------------------------------------ P and dS
        const int b = (warp - 4) >> 2, r = tid & 127;
        const uint32_t ts = tbase + 128 * b + ((uint32_t)(warp & 3) << 21);
        const float c = d.scale * 1.4426950408889634f;
        const int64_t ntok = (int64_t)d.B * d.Tq;
        float lse = 0.0f, delta = 0.0f;
        const int head = KEYS ? unit : PAIR ? head0 + b : unit;
        if (!KEYS && r < rows) {
            lse = p.lse[head * ntok + sp.q0 + row0 + r] * 1.4426950408889634f;
            delta = p.delta[head * ntok + sp.q0 + row0 + r] * d.scale;
        }
        bool ok = true;
        for (int it = PAIR ? 0 : b; it < count; it += PAIR ? 1 : 2) {
            const uint32_t ph = (uint32_t)(PAIR ? it : it >> 1) & 1;
            const int i = it % kStages, r0 = row_at(it);
            // this row's columns [lo, hi), and those below sk
            uint32_t see[2];
            {
                int64_t lo, hi, sk = 0;
                if (KEYS) {
                    const int64_t j = row0 + r;
                    lo = j - past - r0;
                    hi = min((int64_t)other - r0, j < d.sinks ? (int64_t)64 : j + d.window - past - r0);
                } else {
                    const int64_t pos = past + row0 + r;
                    lo = pos - d.window + 1 - r0, hi = pos + 1 - r0, sk = d.sinks - r0;
                }
                const int l = (int)max((int64_t)0, min((int64_t)64, lo)), h = (int)max((int64_t)0, min((int64_t)64, hi)),
                          k = (int)max((int64_t)0, min((int64_t)64, sk));
#pragma unroll
                for (int w = 0; w < 2; ++w) see[w] = low_bits(h - 32 * w) & (~low_bits(l - 32 * w) | low_bits(k - 32 * w));
            }
            if (!(ok = KEYS ? warp_wait2(wait, &sh.s_full[b], ph, &sh.fit[i], (uint32_t)(it / kStages) & 1) : warp_wait(wait, &sh.s_full[b], ph)))
                break;
            fence_after_sync();
            const bool all = __all_sync(0xffffffffu, (see[0] & see[1]) == 0xffffffffu);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float s[32], g[32], e[16], f[16];
                tmem_ld32x2(ts + 32 * w, ts + 64 + 32 * w, s, g);
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    float2 m = make_float2(-lse, -lse), dl = make_float2(-delta, -delta);
                    if (KEYS) {
                        const float2 a = *(const float2 *)&sh.lse[i][32 * w + x], q = *(const float2 *)&sh.delta[i][32 * w + x];
                        m = make_float2(-a.x, -a.y), dl = make_float2(-q.x, -q.y);
                    }
                    float2 t = fma2(make_float2(s[x], s[x + 1]), splat2(c), m);
                    t = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                    float2 u = mul2(t, fma2(make_float2(g[x], g[x + 1]), splat2(d.scale), dl));
                    if (!all) {
                        const uint32_t v = see[w];
                        t.x = v & (1u << x) ? t.x : 0.0f, t.y = v & (2u << x) ? t.y : 0.0f;
                        u.x = v & (1u << x) ? u.x : 0.0f, u.y = v & (2u << x) ? u.y : 0.0f;
                    }
                    e[x / 2] = __uint_as_float(pack2<T>(t.x, t.y));
                    f[x / 2] = __uint_as_float(pack2<T>(u.x, u.y));
                }
                // over columns that have been read: P's half w in S's half w / 2
                if (KEYS) tmem_st16_nw(ts + 16 * w, e);
                tmem_st16_nw(ts + 64 + 16 * w, f);
            }
            tmem_wait_st();
            warp_arrive(&sh.p_ready[b]);
        }
        if (count > 0) {
            if (ok) ok = warp_wait(wait, &sh.acc_full, 0);
            fence_after_sync();
        }
        // ---- the sums, through the rows that stay in shared memory (no product reads them any more): the second
        // warpgroup takes dV, the other head's dQ, or the other half of dQ's channels
        constexpr int kCols = KEYS || PAIR ? D : D / 2;
        const uint32_t from = tbase + L::kAcc + b * kCols + ((uint32_t)(warp & 3) << 21);
        unsigned char *stage = sm + (KEYS ? b * L::kA : PAIR ? b * 2 * L::kA : 0);
        const int c0 = KEYS || PAIR ? 0 : b * kCols;
        // rows of sinks whose sum has other parts stay in fp32
        const int apart = !KEYS || !ok ? 0 : rest ? 128 : row0 < d.sinks && rest_chunks(p, sp, tile) > 0 ? min(128, d.sinks - row0) : 0;
        const int64_t part_slot = !KEYS ? 0 : rest ? slot : p.rest_slots + (int64_t)n * p.sink_tiles + tile;
#pragma unroll
        for (int q = 0; q < kCols; q += 32) {
            float o[32];
            if (count > 0) {
                tmem_ld32(from + q, o);
            } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = 0.0f;
            }
            if (KEYS && r < min(min(apart, rows), d.sinks - row0)) {
                float *to = partial_at<D>(p, part_slot, hk) + ((int64_t)r * 2 + b) * D + q;
#pragma unroll
                for (int x = 0; x < 32; x += 4) *(float4 *)(to + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
            }
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
                const int ch = (c0 + q + x) >> 3;
                *(uint4 *)(stage + (ch >> 3) * L::kRowA + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                    make_uint4(pack2<T>(o[x], o[x + 1]), pack2<T>(o[x + 2], o[x + 3]), pack2<T>(o[x + 4], o[x + 5]), pack2<T>(o[x + 6], o[x + 7]));
            }
        }
        __syncwarp();
        const int w0 = r & ~31;
        const int heads = KEYS ? d.Hk : d.Hq;
        T *out = (T *)(KEYS ? (b ? p.dv : p.dk) : p.dq) + (((KEYS ? sp.k0 : sp.q0) + row0 + w0) * heads + head) * (int64_t)d.d;
        const int n_rows = ok ? max(0, min(32, rows - w0)) : 0;
        for (int x = lane; x < n_rows * (kCols / 8); x += 32) {
            const int q = x / (kCols / 8), ch = c0 / 8 + x % (kCols / 8);
            if (8 * ch < d.d && w0 + q >= apart)
                *(uint4 *)(out + (int64_t)q * heads * d.d + 8 * ch) =
                    *(const uint4 *)(stage + (ch >> 3) * L::kRowA + (w0 + q) * 128 + (((ch & 7) ^ ((w0 + q) & 7)) << 4));
        }
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && sh.gave_up) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    if (warp == 0) tmem_dealloc(tbase, 512);
}

template <typename T, int D>
cudaError_t launch_backward(const WindowProblem &p, cudaStream_t s) {
    const gdn_window_attention_desc &d = p.d;
    WindowMaps wide, slim;
    memset(&wide, 0, sizeof(wide));
    memset(&slim, 0, sizeof(slim));
    for (WindowMaps *m : {&wide, &slim}) {
        const uint32_t box = m == &wide ? 128 : 64;
        int rows;
        if (!window_head_map(&m->q, d, p.q, d.Hq, d.Tq, d.q_stride_b, d.q_stride_t, &m->q_rows, box) ||
            !window_head_map(&m->k, d, p.k, d.Hk, d.Tk, d.k_stride_b, d.k_stride_t, &m->k_rows, box) ||
            !window_head_map(&m->v, d, p.v, d.Hk, d.Tk, d.v_stride_b, d.v_stride_t, &m->v_rows, box) ||
            !window_head_map(&m->g, d, p.dout, d.Hq, d.Tq, (int64_t)d.Tq * d.Hq * d.d, (int64_t)d.Hq * d.d, &rows, box))
            return cudaErrorInvalidValue;
    }
    cudaError_t e;
    auto go = [&](auto kernel, size_t bytes, int64_t tiles, int units, int64_t rest) {
        const size_t smem = std::max<size_t>(bytes, 117 * 1024);   // one CTA per SM: each holds all of the tensor memory
        if ((tiles + rest) * units > 0x7fffffff) return cudaErrorInvalidValue;
        const cudaError_t a = allow_shared(kernel, smem);
        if (a != cudaSuccess) return a;
        kernel<<<(unsigned)((tiles + rest) * units), kThreads, smem, s>>>(wide, slim, p, units, rest * units);
        return cudaGetLastError();
    };
    const int64_t qt = p.cu ? cdiv64(d.Tq, 128) + d.N : (int64_t)d.B * cdiv64(d.Tq, 128);
    const int64_t kt = p.cu ? cdiv64(d.Tk, 128) + d.N : (int64_t)d.B * cdiv64(d.Tk, 128);
    if ((e = go(window_backward_tc<T, D, true, false>, BwdShape<D, false>::kBytes, kt, d.Hk, p.rest_slots)) != cudaSuccess) return e;
    if (d.Hq / d.Hk % 2 == 0) e = go(window_backward_tc<T, D, false, true>, BwdShape<D, true>::kBytes, qt, d.Hq / 2, 0);
    else e = go(window_backward_tc<T, D, false, false>, BwdShape<D, false>::kBytes, qt, d.Hq, 0);
    if (e != cudaSuccess) return e;
    return launch_window_sink_sums<T, D>(p, s);
}

}  // namespace

cudaError_t launch_window_backward_tc(const WindowProblem &p, cudaStream_t s) {
    if (p.d.d <= 64) return p.d.dtype == GDN_BF16 ? launch_backward<__nv_bfloat16, 64>(p, s) : launch_backward<__half, 64>(p, s);
    return p.d.dtype == GDN_BF16 ? launch_backward<__nv_bfloat16, 128>(p, s) : launch_backward<__half, 128>(p, s);
}

}  // namespace gdn
