// gdn_window_bwd_tc.cu -- the window attention's backward on the tensor cores
// (include/gdn.h), for 16-bit types and heads of up to 128 channels.
//
// Two kernels of one shape, so that every sum has a fixed order (no atomics): one CTA keeps
// 128 rows and walks over tiles of 128 rows of the other side.
//   keys:    K_j, V_j stay; per head of the group and tile of queries
//            S' = K Q^T, dP' = V dO^T, P' = exp2(c S' - lse), dS' = P' (dP' - delta),
//            dV += P' dO, dK += dS' Q (scale taken out of the sums, fp16 in units: gdn_window_tc.cuh)
//   queries: Q_i, dO_i stay; per tile of keys  S, dP as above (not transposed), dQ += dS K;
//            gdn_window_dq_tc.cu has it for two heads at once
// P and dS take the place of S and dP in tensor memory, from where they are operands of the
// second products. Two warpgroups work on a tile, a thread per row and half of the columns. The
// products of tile t and the scores of t + 1 alternate so that the tensor cores have work while
// P, and then dS, are computed:
//     dV(t) [P(t)], S(t+1), dK(t) [dS(t)], dP(t+1), dV(t+1), ..
// Scores are taken for 128 columns at a time: with 64, reading the operand that stays holds the
// tensor cores to half their rate (1280 of 1400 cycles a tile of 64 by a clock trace). Seven
// products instead of five recompute S and dP, which is the price of no atomics. P and dS are
// rounded to the tensors' type, which the second products take; statistics and sums are fp32.
//
// Bound by the tensor cores' rate on operands in shared memory (about 98 cycles a product of 128
// columns, 64 at the nominal rate) and a CTA's start and end: 8192 tokens of 16 heads of 128 on 8, causal
// 698 us (984 TFLOP/s of the five products), 16384 with a window of 1024 516 us (647).
#include <string.h>

#include <algorithm>

#include "gdn_window_rest.cuh"
#include "gdn_window_tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kThreads = 384;   // warps 0 TMA, 1 MMA, 2-3 statistics and rows behind a sequence, 4-11 P and dS
constexpr int kFirst = 3, kSecond = 2;   // stages of the walked side's operand of S (and dK, dQ) and of dP (and dV)

template <int D> struct BwdShape {
    static constexpr int kRow = 128 * 128;                 // bytes of 128 rows x 64 channels
    static constexpr int kTile = D / 64 * kRow;
    static constexpr int kA1 = 0, kA2 = kTile, kB1 = 2 * kTile, kB2 = kB1 + kFirst * kTile, kEnd = kB2 + kSecond * kTile;
    static constexpr uint32_t kS = 0, kP = 128, kAcc = 256;   // TMEM columns: S (P), dP (dS), and the sums, D each
};

struct BwdShared {
    uint64_t a_full, full1[kFirst], empty1[kFirst], fit[kFirst], full2[kSecond], empty2[kSecond], s_full, d_full, p_ready, ds_ready, acc_full, drain;
    uint32_t tmem;
    int gave_up;
    float lse[2][128], delta[2][128];   // of the tile's queries (keys kernel): lse log2 e, delta, in P's and dP's units
};

template <typename T, int D, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) window_backward_tc(const __grid_constant__ WindowMaps maps, const __grid_constant__ WindowProblem p, int units,
                                                                  int64_t rest_blocks) {
    using L = BwdShape<D>;
    extern __shared__ __align__(1024) unsigned char smraw[];
    // 3 KB that start on a multiple of 1024 bytes, so that the tiles behind them do too: together all that a CTA can have
    __shared__ __align__(1024) union {
        BwdShared sh;
        unsigned char all[3 * 1024];
    } head_sh;
    static_assert(sizeof(head_sh) == 3 * 1024, "the tiles follow");
    BwdShared &sh = head_sh.sh;
    unsigned char *sm = smraw;
    const gdn_window_attention_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) tma_prefetch_map(&maps.q), tma_prefetch_map(&maps.k), tma_prefetch_map(&maps.v), tma_prefetch_map(&maps.g);
    if (smem_u32(smraw) & 1023) {   // (never: see above) the swizzled tiles would be read wrongly
        if (tid == 0) *p.status = GDN_ERR_DEVICE_TIMEOUT;
        return;
    }

    // ---- the CTA's place
    const int group = d.Hq / d.Hk;
    const bool rest = KEYS && blockIdx.x < rest_blocks;
    const int64_t block = rest ? blockIdx.x : blockIdx.x - rest_blocks;
    const int slot = (int)((uint32_t)block / (uint32_t)units), unit = (int)block - slot * units;   // unit: head of k and v (queries: of q)
    int n, tile, chunk = 0;
    const int32_t *table = KEYS ? p.k_tiles : p.q_tiles;
    if (rest) {
        RestAt at;
        const bool found = rest_at(p, slot, at);
        if (*p.status == GDN_ERR_DEVICE_SEQLENS || !found) return;
        n = at.n, tile = at.tile, chunk = at.chunk;
    } else if (p.cu) {
        const int32_t status = *p.status, tiles = table[d.N];   // on their way with the search's
        n = warp_upper_index(table, d.N, slot);
        if (status == GDN_ERR_DEVICE_SEQLENS || slot >= tiles) return;
        tile = slot - table[n];
    } else {
        const int per = ((KEYS ? d.Tk : d.Tq) + 127) / 128;
        n = slot / per;
        tile = slot - n * per;
    }
    const WindowSpan sp = window_span(p, n);
    const int past = sp.Lk - sp.Lq;
    if (!KEYS) {                                           // later queries, which see the most, first
        tile = (p.cu ? p.q_tiles[n + 1] - p.q_tiles[n] : (d.Tq + 127) / 128) - 1 - tile;
    }
    const int hk = KEYS ? unit : unit / group;
    const int row0 = tile * 128, rows = min(128, (KEYS ? sp.Lk : sp.Lq) - row0);   // the rows that stay

    // ---- what it walks over: `count` tiles of 128 rows
    int first = 0, per_head = 0, ns = 0, count;
    if (KEYS) {
        if (rest) {
            const SinkRest r = sink_rest(sp.Lq, sp.Lk, tile, d.window, 7);
            first = r.e0, per_head = r.tiles;
            count = (int)min((int64_t)p.rest_its, (int64_t)per_head * group - (int64_t)chunk * p.rest_its);
        } else {
            const int64_t lo = max((int64_t)0, (int64_t)row0 - past);
            const int64_t hi = min((int64_t)sp.Lq - 1, (int64_t)row0 + rows - 1 + d.window - 1 - past);
            if (hi >= lo) first = (int)(lo >> 7), per_head = (int)((hi >> 7) - (lo >> 7) + 1);
            count = per_head * group;
        }
    } else {
        const WindowTiles w = window_tiles(past + row0, past + row0 + rows - 1, d.window, d.sinks);
        ns = w.ns, first = w.w0;
        count = w.empty() ? 0 : w.ns + w.w1 - w.w0 + 1;
    }
    // tile `it`: its head of queries and its first row
    auto head_at = [&](int it) { return KEYS ? hk * group + (int)(((int64_t)chunk * p.rest_its + it) / per_head) : unit; };
    auto row_at = [&](int it) {
        if (KEYS) return (first + (int)(((int64_t)chunk * p.rest_its + it) % per_head)) * 128;
        return (it < ns ? it : first + it - ns) * 128;
    };
    const int other = KEYS ? sp.Lq : sp.Lk;                // rows of the side walked over

    const int qrow = p.cu ? (int)sp.q0 : 0, krow = p.cu ? (int)sp.k0 : 0;
    const int qb = p.cu ? 0 : n * maps.q_rows, kb = p.cu ? 0 : n * maps.k_rows, vb = p.cu ? 0 : n * maps.v_rows, gb = p.cu || d.B == 1 ? 0 : n;
    auto copy = [&](int to, const CUtensorMap *map, int head, int row, int batch, uint64_t *bar) {
        for (int b = 0; b < D / 64; ++b) tma_load_4d(sm + to + b * L::kRow, map, 64 * b, head, row, batch, bar);
    };
    // the walked side's operands of the it-th tile
    auto load1 = [&](int it) {
        const int i = it % kFirst;
        mbar_expect_tx(&sh.full1[i], L::kTile);
        copy(L::kB1 + i * L::kTile, KEYS ? &maps.q : &maps.k, KEYS ? head_at(it) : hk, (KEYS ? qrow : krow) + row_at(it), KEYS ? qb : kb, &sh.full1[i]);
    };
    auto load2 = [&](int it) {
        const int j = it % kSecond;
        mbar_expect_tx(&sh.full2[j], L::kTile);
        copy(L::kB2 + j * L::kTile, KEYS ? &maps.g : &maps.v, KEYS ? head_at(it) : hk, (KEYS ? qrow : krow) + row_at(it), KEYS ? gb : vb, &sh.full2[j]);
    };
    if (tid == 0) {
        mbar_init(&sh.a_full, 1);
        for (int i = 0; i < kFirst; ++i) mbar_init(&sh.full1[i], 1), mbar_init(&sh.empty1[i], 1), mbar_init(&sh.fit[i], 2);
        for (int i = 0; i < kSecond; ++i) mbar_init(&sh.full2[i], 1), mbar_init(&sh.empty2[i], 1);
        mbar_init(&sh.s_full, 1), mbar_init(&sh.d_full, 1), mbar_init(&sh.p_ready, 8), mbar_init(&sh.ds_ready, 8);
        mbar_init(&sh.acc_full, 1), mbar_init(&sh.drain, 1);
        sh.gave_up = 0;
        mbar_init_fence();
        if (count > 0) {   // the first copies are on their way while the CTA gets its tensor memory
            fence_async_smem();
            mbar_expect_tx(&sh.a_full, 2 * L::kTile);
            copy(L::kA1, KEYS ? &maps.k : &maps.q, unit, (KEYS ? krow : qrow) + row0, KEYS ? kb : qb, &sh.a_full);
            load1(0);
            copy(L::kA2, KEYS ? &maps.v : &maps.g, unit, (KEYS ? krow : qrow) + row0, KEYS ? vb : gb, &sh.a_full);
            load2(0);
        }
    }
    if (warp == 1) tmem_alloc(&sh.tmem, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tbase = sh.tmem;
    const WindowWait wait{&sh.gave_up, p.wait_immediate != 0};
    constexpr bool kHalf = std::is_same<T, __half>::value;
    const uint32_t idesc_s = kHalf ? idesc_f16(128, 128, false, false) : idesc_bf16(128, 128, false, false);
    const uint32_t idesc_a = kHalf ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0 && count > 0) {
            int n1 = 1, n2 = 1;   // loaded so far
            for (int it = 1; it < count; ++it) {
                if (it >= kFirst && !wait(&sh.empty1[it % kFirst], (uint32_t)(it / kFirst - 1) & 1)) break;
                load1(it);
                ++n1;
                if (it >= kSecond && !wait(&sh.empty2[it % kSecond], (uint32_t)(it / kSecond - 1) & 1)) break;
                load2(it);
                ++n2;
            }
            // what is in flight lands before the CTA leaves
            mbar_wait(&sh.a_full, 0);
            for (int u = max(0, n1 - kFirst); u < n1; ++u) mbar_wait(&sh.full1[u % kFirst], (uint32_t)(u / kFirst) & 1);
            for (int u = max(0, n2 - kSecond); u < n2; ++u) mbar_wait(&sh.full2[u % kSecond], (uint32_t)(u / kSecond) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        const int total = of_warp(count);
        if (total > 0) {
            const uint32_t leader = elect_one(), tb = (uint32_t)of_warp((int)tbase), base = (uint32_t)of_warp((int)smem_u32(sm));
            const uint64_t a1 = sw128_desc(base + L::kA1, 0, 1024), a2 = sw128_desc(base + L::kA2, 0, 1024),
                           b1 = sw128_desc(base + L::kB1, 0, 1024), b2 = sw128_desc(base + L::kB2, 0, 1024),
                           n1 = sw128_desc(base + L::kB1, L::kRow, 1024), n2 = sw128_desc(base + L::kB2, L::kRow, 1024);
            // stages and phases: of the next scores' operands, and of the next sums'
            int s1 = 0, s2 = 0, t1 = 0, t2 = 0;
            uint32_t ph1 = 0, ph2 = 0;
            auto scores = [&](uint32_t to, uint64_t a, uint64_t b) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t at = ((i >> 2) * L::kRow + (i & 3) * 32) >> 4;
                    warp_mma_f16(leader, tb + to, a + at, b + at, idesc_s, i > 0);
                }
            };
            auto S = [&]() -> bool {
                if (!warp_wait2(wait, &sh.full1[s1], ph1, &sh.fit[s1], ph1)) return false;
                fence_after_sync();
                scores(L::kS, a1, b1 + (uint32_t)(s1 * (L::kTile >> 4)));
                warp_mma_commit(leader, &sh.s_full);
                if (++s1 == kFirst) s1 = 0, ph1 ^= 1;
                return true;
            };
            auto dP = [&]() -> bool {
                if (!warp_wait(wait, &sh.full2[s2], ph2)) return false;
                fence_after_sync();
                scores(L::kP, a2, b2 + (uint32_t)(s2 * (L::kTile >> 4)));
                warp_mma_commit(leader, &sh.d_full);
                if (!KEYS) warp_mma_commit(leader, &sh.empty2[s2]);
                if (++s2 == kSecond) s2 = 0, ph2 ^= 1;
                return true;
            };
            // the rows' 128 values of the walked side lie in two halves of 32 columns, 64 columns apart
            auto sum = [&](uint32_t acc, uint32_t from, uint64_t b, uint32_t more) {
                warp_mma_f16_ta(leader, tb + acc, tb + from, b, idesc_a, more);
#pragma unroll
                for (int i = 1; i < 8; ++i)
                    warp_mma_f16_ta(leader, tb + acc, tb + from + 8 * (i & 3) + 64 * (i >> 2), b + (uint32_t)(2048 * i >> 4), idesc_a, 1);
            };
            bool ok = warp_wait(wait, &sh.a_full, 0) && S() && dP();
            for (int it = 0; ok && it < total; ++it) {
                const bool more = it + 1 < total;
                ok = warp_wait(wait, &sh.p_ready, (uint32_t)it & 1);   // P is there; S has been read
                fence_after_sync();
                if (!ok) break;
                if (KEYS) {   // dV += P dO
                    sum(L::kAcc + D, L::kS, n2 + (uint32_t)(t2 * (L::kTile >> 4)), it > 0);
                    warp_mma_commit(leader, &sh.empty2[t2]);
                    if (++t2 == kSecond) t2 = 0;
                }
                if (more && !(ok = S())) break;
                ok = warp_wait(wait, &sh.ds_ready, (uint32_t)it & 1);
                fence_after_sync();
                if (!ok) break;
                sum(L::kAcc, L::kP, n1 + (uint32_t)(t1 * (L::kTile >> 4)), it > 0);   // dK += dS Q, dQ += dS K
                warp_mma_commit(leader, &sh.empty1[t1]);
                if (++t1 == kFirst) t1 = 0;
                if (more) ok = dP();
            }
            if (ok) warp_mma_commit(leader, &sh.acc_full);
            warp_mma_commit(leader, &sh.drain);
            mbar_wait(&sh.drain, 0);
        }
    } else if (warp < 4) {
        // -------------------------- the queries' statistics, and zeros in rows behind the sequence (0 x NaN is NaN)
        const int w = warp - 2;
        const int64_t ntok = (int64_t)d.B * d.Tq;
        const float up = KEYS ? grad_factor<T>(p, n, hk) : 1.0f;
        for (int it = 0; it < count; ++it) {
            const int i = it % kFirst, j = it % kSecond, r0 = row_at(it), left = other - r0;
            float l[2] = {0.0f, 0.0f}, dl[2] = {0.0f, 0.0f};
            if (KEYS)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = 64 * w + 32 * h + lane;
                    if (x < left) {
                        const int64_t at = head_at(it) * ntok + sp.q0 + r0 + x;
                        l[h] = fmaf(p.lse[at], 1.4426950408889634f, -(float)kWeightBits<T>), dl[h] = p.delta[at] * up;
                    }
                }
            // tile it - 2 is through with its statistics once its dK is; also keeps this warp near the products
            if (it >= 2 && !warp_wait(wait, &sh.empty1[(it - 2) % kFirst], (uint32_t)((it - 2) / kFirst) & 1)) break;
            if (KEYS)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int x = 64 * w + 32 * h + lane;
                    sh.lse[it & 1][x] = l[h], sh.delta[it & 1][x] = dl[h];
                }
            if (left < 128) {   // a warp for each of the two
                const bool come = w ? warp_wait(wait, &sh.full2[j], (uint32_t)(it / kSecond) & 1) : warp_wait(wait, &sh.full1[i], (uint32_t)(it / kFirst) & 1);
                if (!come) break;
                unsigned char *t = sm + (w ? L::kB2 + j * L::kTile : L::kB1 + i * L::kTile);
                for (int b = 0; b < D / 64; ++b)
                    for (int x = left * 8 + lane; x < 128 * 8; x += 32) *(uint4 *)(t + b * L::kRow + 16 * x) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.fit[i]);
        }
    } else {
        // ------------------------------------------------------------ P and dS
        const int half = (warp - 4) >> 2, r = tid & 127;
        const uint32_t ts = tbase + 64 * half + ((uint32_t)(warp & 3) << 21);   // this thread's half of S; dP's is kP further
        const float c = d.scale * 1.4426950408889634f;
        const int64_t ntok = (int64_t)d.B * d.Tq;
        const float up = grad_factor<T>(p, n, hk);
        float lse = 0.0f, delta = 0.0f;
        if (!KEYS && r < rows) {
            lse = fmaf(p.lse[unit * ntok + sp.q0 + row0 + r], 1.4426950408889634f, -(float)kWeightBits<T>);
            delta = p.delta[unit * ntok + sp.q0 + row0 + r] * up;
        }
        bool ok = true;
        for (int it = 0; it < count; ++it) {
            const int r0 = row_at(it) + 64 * half, i = it % kFirst;
            const uint32_t ph = (uint32_t)it & 1;
            // this row's columns [lo, hi) of its half, and those below sk
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
            const bool all = __all_sync(0xffffffffu, (see[0] & see[1]) == 0xffffffffu);
            if (!(ok = KEYS ? warp_wait2(wait, &sh.s_full, ph, &sh.fit[i], (uint32_t)(it / kFirst) & 1) : warp_wait(wait, &sh.s_full, ph))) break;
            fence_after_sync();
            float x[64];   // S, then P
            tmem_ld64(ts, x);
            if (!KEYS) warp_arrive(&sh.p_ready);   // S may be written again
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float e[16];
#pragma unroll
                for (int q = 0; q < 32; q += 2) {
                    float2 m = make_float2(-lse, -lse);
                    if (KEYS) {
                        const float2 a = *(const float2 *)&sh.lse[it & 1][64 * half + 32 * w + q];
                        m = make_float2(-a.x, -a.y);
                    }
                    float2 t = fma2(make_float2(x[32 * w + q], x[32 * w + q + 1]), splat2(c), m);
                    t = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                    if (!all) {
                        t.x = see[w] & (1u << q) ? t.x : 0.0f, t.y = see[w] & (2u << q) ? t.y : 0.0f;
                    }
                    x[32 * w + q] = t.x, x[32 * w + q + 1] = t.y;
                    if (KEYS) e[q / 2] = __uint_as_float(pack2<T>(t.x, t.y));
                }
                if (KEYS) tmem_st16_nw(ts + 16 * w, e);
            }
            if (KEYS) {
                tmem_wait_st();
                warp_arrive(&sh.p_ready);
            }
            if (!(ok = warp_wait(wait, &sh.d_full, ph))) break;
            fence_after_sync();
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float g[32], f[16];
                tmem_ld32(ts + L::kP + 32 * w, g);
#pragma unroll
                for (int q = 0; q < 32; q += 2) {
                    float2 dl = make_float2(-delta, -delta);
                    if (KEYS) {
                        const float2 a = *(const float2 *)&sh.delta[it & 1][64 * half + 32 * w + q];
                        dl = make_float2(-a.x, -a.y);
                    }
                    float2 u = mul2(make_float2(x[32 * w + q], x[32 * w + q + 1]), fma2(make_float2(g[q], g[q + 1]), splat2(up), dl));
                    if (!all) {   // P is 0, but dP may be anything
                        u.x = see[w] & (1u << q) ? u.x : 0.0f, u.y = see[w] & (2u << q) ? u.y : 0.0f;
                    }
                    f[q / 2] = __uint_as_float(pack2<T>(u.x, u.y));
                }
                tmem_st16_nw(ts + L::kP + 16 * w, f);   // over columns that have been read
            }
            tmem_wait_st();
            warp_arrive(&sh.ds_ready);
        }
        if (count > 0) {
            if (ok) ok = warp_wait(wait, &sh.acc_full, 0);
            fence_after_sync();
        }
        // ---- the sums, through the rows that stay in shared memory (no product reads them any more): the second
        // warpgroup takes dV, or the other half of dQ's channels
        constexpr int kCols = KEYS ? D : D / 2;
        const uint32_t from = tbase + L::kAcc + half * kCols + ((uint32_t)(warp & 3) << 21);
        unsigned char *stage = sm + (KEYS ? half * L::kTile : 0);
        const int c0 = KEYS ? 0 : half * kCols;
        // rows of sinks whose sum has other parts stay in fp32
        const int apart = !KEYS || !ok ? 0 : rest ? 128 : row0 < d.sinks && rest_chunks(p, sp, tile) > 0 ? min(128, d.sinks - row0) : 0;
        const bool none = KEYS ? !half && seen_by_such(sp.Lk, d.window, d.sinks) : sees_one((int64_t)past + row0 + r, d.window, d.sinks);
        const float2 back = splat2(none ? 0.0f : KEYS && half ? kWeightUnit<T> : d.scale * kWeightUnit<T> / up);   // out of the operands' units
        const int64_t part_slot = !apart ? 0 : rest ? slot : own_slot(p, n, tile);
#pragma unroll
        for (int q = 0; q < kCols; q += 32) {
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
            if (KEYS && r < min(min(apart, rows), d.sinks - row0)) {
                float *to = partial_at<D>(p, part_slot, hk) + ((int64_t)r * 2 + half) * D + q;
#pragma unroll
                for (int x = 0; x < 32; x += 4) *(float4 *)(to + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
            }
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
                const int ch = (c0 + q + x) >> 3;
                *(uint4 *)(stage + (ch >> 3) * L::kRow + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) =
                    make_uint4(pack2<T>(o[x], o[x + 1]), pack2<T>(o[x + 2], o[x + 3]), pack2<T>(o[x + 4], o[x + 5]), pack2<T>(o[x + 6], o[x + 7]));
            }
        }
        __syncwarp();
        const int w0 = r & ~31, heads = KEYS ? d.Hk : d.Hq;
        T *out = (T *)(KEYS ? (half ? p.dv : p.dk) : p.dq) + (((KEYS ? sp.k0 : sp.q0) + row0 + w0) * heads + unit) * (int64_t)d.d;
        const int n_rows = ok ? max(0, min(32, rows - w0)) : 0;
#pragma unroll
        for (int x = lane; x < 32 * (kCols / 8); x += 32) {
            const int q = x / (kCols / 8), ch = c0 / 8 + x % (kCols / 8);
            if (q < n_rows && 8 * ch < d.d && w0 + q >= apart)
                *(uint4 *)(out + (int64_t)q * heads * d.d + 8 * ch) =
                    *(const uint4 *)(stage + (ch >> 3) * L::kRow + (w0 + q) * 128 + (((ch & 7) ^ ((w0 + q) & 7)) << 4));
        }
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && sh.gave_up) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    if (warp == 1) tmem_dealloc(tbase, 512);
}

template <typename T, int D>
cudaError_t launch_backward(const WindowProblem &p, cudaStream_t s) {
    const gdn_window_attention_desc &d = p.d;
    WindowMaps maps;
    memset(&maps, 0, sizeof(maps));
    int rows;
    if (!window_head_map(&maps.q, d, p.q, d.Hq, d.Tq, d.q_stride_b, d.q_stride_t, &maps.q_rows, 128) ||
        !window_head_map(&maps.k, d, p.k, d.Hk, d.Tk, d.k_stride_b, d.k_stride_t, &maps.k_rows, 128) ||
        !window_head_map(&maps.v, d, p.v, d.Hk, d.Tk, d.v_stride_b, d.v_stride_t, &maps.v_rows, 128) ||
        !window_head_map(&maps.g, d, p.dout, d.Hq, d.Tq, (int64_t)d.Tq * d.Hq * d.d, (int64_t)d.Hq * d.d, &rows, 128))
        return cudaErrorInvalidValue;
    constexpr size_t smem = std::max(BwdShape<D>::kEnd, 114 * 1024);   // one CTA per SM: each holds all of the tensor memory
    auto go = [&](auto kernel, int64_t tiles, int units, int64_t rest) {
        if ((tiles + rest) * units > 0x7fffffff) return cudaErrorInvalidValue;
        const cudaError_t a = allow_shared(kernel, smem);
        if (a != cudaSuccess) return a;
        kernel<<<(unsigned)((tiles + rest) * units), kThreads, smem, s>>>(maps, p, units, rest * units);
        return cudaGetLastError();
    };
    const int64_t qt = p.cu ? cdiv64(d.Tq, 128) + d.N : (int64_t)d.B * cdiv64(d.Tq, 128);
    const int64_t kt = p.cu ? cdiv64(d.Tk, 128) + d.N : (int64_t)d.B * cdiv64(d.Tk, 128);
    cudaError_t e = go(window_backward_tc<T, D, true>, kt, d.Hk, p.rest_slots);
    if (e == cudaSuccess) e = window_dq_pairs(d) ? launch_window_dq_pair(maps, p, s) : go(window_backward_tc<T, D, false>, qt, d.Hq, 0);
    return e == cudaSuccess ? launch_window_sink_sums<T, D>(p, s) : e;
}

}  // namespace

cudaError_t launch_window_backward_tc(const WindowProblem &p, cudaStream_t s) {
    if (p.d.d <= 64) return p.d.dtype == GDN_BF16 ? launch_backward<__nv_bfloat16, 64>(p, s) : launch_backward<__half, 64>(p, s);
    return p.d.dtype == GDN_BF16 ? launch_backward<__nv_bfloat16, 128>(p, s) : launch_backward<__half, 128>(p, s);
}

}  // namespace gdn
