// gdn_window_tc.cu -- the window attention's forward on the tensor cores (include/gdn.h),
// for 16-bit types and heads of up to 128 channels.
//
// One CTA holds two tiles of 128 queries and walks once over the tiles of 128 keys that any
// of them sees, sinks first. Per tile of keys and of queries:
//     S = Q K^T (tensor memory, fp32), P = exp2(c S - m) by one warpgroup, a thread per query
//     (its row of S lies in its lane of tensor memory), P as 16 bits over S, O += P V.
// The two tiles of queries take turns: while one's P is computed the tensor cores work for the
// other. They are two heads that share keys and values where the group's size is even (the
// same mask, half the traffic of K and V), else two neighbouring tiles of one head.
// Softmax in one pass: a row's maximum m is raised, and O scaled, only where it grew by more
// than 2^8 (P stays below 2^8; fp16 takes it times 2^6), so O is rarely read back. P is rounded
// to the tensors' type, which the second product takes; sums, maxima and O are fp32. The methods
// are published ones: one pass by Milakov and Gimelshein (2018), tiles in turns for the tensor
// cores before these (2024), a maximum that moves only where it has to for these (2025).
//
// Bound by the tensor cores where rows see many keys (causal, 16384 tokens of 16 heads of 128 on
// 8: 702 us, 1566 TFLOP/s), else by a CTA's start and end (about 8000 cycles, in which nothing
// else runs: the CTA holds all of tensor memory) and the cut tiles (window 2048: 32768 tokens
// 524 us, 1018 TFLOP/s; 16384 of 64 channels, where the softmax takes more than the products,
// 212 us, 609).
// Slower were: one persistent CTA per SM, four warpgroups of softmax, two CTAs per SM of one
// subtile each (575 us), four subtiles and tiles of 64 keys for 64 channels (small calls twice
// as slow).
//
// Values that a query does not see must not reach it, also where they are infinite or NaN:
// 0 x NaN in the product would. Two warps look through every tile of V that a mask cuts, put
// zeros for what is not finite and note the key; the queries that do see it are computed again
// on their own at the end (row_forward).
#include <string.h>

#include <algorithm>

#include "gdn_window_tc.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kThreads = 384;      // warps 0 TMA, 1 MMA, 2-3 check V, 4-7 and 8-11 softmax
constexpr int kCutTiles = 8;       // tiles of keys that a mask cuts: 3 at the diagonal, 3 where windows begin, the last sinks'

template <int D> struct FwdShape {
    static constexpr int kRow = 128 * 128;                 // bytes of 128 rows x 64 channels
    static constexpr int kTile = D / 64 * kRow;            // a tile of Q, K or V
    static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 3 : 4;   // stages
    static constexpr int kQ = 0, kKs = 2 * kTile, kVs = kKs + kK * kTile, kEnd = kVs + kV * kTile;
    static constexpr int kBytes = kEnd + 1024;             // and what alignment to 1024 may take
    static constexpr uint32_t kO = 256;                    // TMEM column of O; S and P of subtile s at 128 s
};

struct FwdShared {
    uint64_t q_full, k_full[4], k_empty[4], v_full[4], v_empty[4], v_ok[4], s_full[2], p_half[2], p_ready[2], o_full[2], drain;
    uint32_t tmem;
    int gave_up, any_bad;
    int cut_tile[kCutTiles];
    uint32_t bad[kCutTiles][4];   // a bit for every key of a cut tile whose values are not all finite
};

// Subtile s of a CTA: its head, its first query and the positions it covers
struct Subtile {
    int head, i0, rows, p0, p1;
    WindowTiles tiles;
};

template <typename T> __device__ __forceinline__ uint32_t finite_probe(uint32_t w, uint32_t acc);
template <> __device__ __forceinline__ uint32_t finite_probe<__half>(uint32_t w, uint32_t acc) {
    asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));   // 0 x inf and 0 x NaN stay
    return acc;
}
template <> __device__ __forceinline__ uint32_t finite_probe<__nv_bfloat16>(uint32_t w, uint32_t acc) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
    return acc;
}
template <typename T> constexpr uint32_t exponent_bits() { return std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u; }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) window_forward_tc(const __grid_constant__ WindowMaps maps, const __grid_constant__ WindowProblem p,
                                                                 int pair_heads, int units) {
    using L = FwdShape<D>;
    extern __shared__ unsigned char smraw[];
    __shared__ FwdShared sh;
    unsigned char *sm = (unsigned char *)(((uintptr_t)smraw + 1023) & ~(uintptr_t)1023);
    const gdn_window_attention_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) tma_prefetch_map(&maps.q), tma_prefetch_map(&maps.k), tma_prefetch_map(&maps.v);
    if (!p.cu && blockIdx.x == 0 && tid == 0) *p.status = GDN_OK;

    // ---- the CTA's place: later tiles of queries, which see the most keys, first
    const int slot = (int)(blockIdx.x / units), unit = (int)blockIdx.x - slot * units;
    const int rows_per = pair_heads ? 128 : 256;
    int n, qt;
    if (p.cu) {
        const int32_t status = *p.status, tiles = p.q_tiles[d.N];   // on their way with the search's
        n = warp_upper_index(p.q_tiles, d.N, slot);
        if (status != GDN_OK || slot >= tiles) return;
        qt = p.q_tiles[n + 1] - 1 - slot;
    } else {
        const int per = (d.Tq + rows_per - 1) / rows_per;
        n = slot / per;
        qt = per - 1 - (slot - n * per);
    }
    const WindowSpan sp = window_span(p, n);
    const int past = sp.Lk - sp.Lq;
    Subtile st[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        st[s].head = pair_heads ? 2 * unit + s : unit;
        st[s].i0 = qt * rows_per + (pair_heads ? 0 : 128 * s);
        st[s].rows = max(0, min(128, sp.Lq - st[s].i0));
        st[s].p0 = past + st[s].i0;
        st[s].p1 = st[s].rows ? st[s].p0 + st[s].rows - 1 : -1;
        st[s].tiles = window_tiles(st[s].p0, st[s].p1, d.window, d.sinks);
        st[s].p0 = max(st[s].p0, 0);
    }
    // the tiles of either, in order: [0, ns) and [w0, w1] (subtile 1 never reaches back behind subtile 0's first)
    WindowTiles all = st[0].tiles.empty() ? st[1].tiles : st[0].tiles;
    if (!st[0].tiles.empty() && !st[1].tiles.empty()) {
        all.w1 = max(all.w1, st[1].tiles.w1);
        all.ns = min(max(all.ns, st[1].tiles.ns), all.w0);
    }
    const int count = all.empty() ? 0 : all.ns + all.w1 - all.w0 + 1;
    auto tile_at = [&](int u) { return u < all.ns ? u : all.w0 + u - all.ns; };
    const int hk = st[0].head / (d.Hq / d.Hk);

    // K or V of the u-th tile into its stage
    auto load = [&](int u, bool is_v) {
        const int i = u % (is_v ? L::kV : L::kK), krow = p.cu ? (int)sp.k0 : 0, batch = p.cu ? 0 : n * (is_v ? maps.v_rows : maps.k_rows);
        uint64_t *full = is_v ? &sh.v_full[i] : &sh.k_full[i];
        unsigned char *to = sm + (is_v ? L::kVs : L::kKs) + i * L::kTile;
        mbar_expect_tx(full, L::kTile);
        for (int b = 0; b < D / 64; ++b) tma_load_4d(to + b * L::kRow, is_v ? &maps.v : &maps.k, 64 * b, hk, krow + tile_at(u) * 128, batch, full);
    };
    if (tid == 0) {
        mbar_init(&sh.q_full, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sh.k_full[i], 1), mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 1), mbar_init(&sh.v_empty[i], 1), mbar_init(&sh.v_ok[i], 2);
        }
        for (int s = 0; s < 2; ++s) mbar_init(&sh.s_full[s], 1), mbar_init(&sh.p_half[s], 4), mbar_init(&sh.p_ready[s], 4), mbar_init(&sh.o_full[s], 1);
        mbar_init(&sh.drain, 1);
        sh.gave_up = sh.any_bad = 0;
        mbar_init_fence();
        if (count > 0) {   // the first copies are on their way while the CTA gets its tensor memory
            fence_async_smem();
            const int qrow = p.cu ? (int)sp.q0 : 0, qb = p.cu ? 0 : n * maps.q_rows;
            int q_bytes = 0;
            for (int s = 0; s < 2; ++s) q_bytes += st[s].tiles.empty() ? 0 : L::kTile;
            mbar_expect_tx(&sh.q_full, q_bytes);
            for (int s = 0; s < 2; ++s)
                if (!st[s].tiles.empty())
                    for (int b = 0; b < D / 64; ++b)
                        tma_load_4d(sm + L::kQ + s * L::kTile + b * L::kRow, &maps.q, 64 * b, st[s].head, qrow + st[s].i0, qb, &sh.q_full);
            load(0, false);
            load(0, true);
        }
    }
    if (warp == 1) tmem_alloc(&sh.tmem, 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tbase = sh.tmem;
    const WindowWait wait{&sh.gave_up, p.wait_immediate != 0};
    const uint32_t idesc_s = std::is_same<T, __half>::value ? idesc_f16(128, 128, false, false) : idesc_bf16(128, 128, false, false);
    const uint32_t idesc_o = std::is_same<T, __half>::value ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        if (lane == 0 && count > 0) {
            int ku = 1, vu = 1;   // loaded so far
            for (int u = 1; u < count; ++u) {
                if (u >= L::kK && !wait(&sh.k_empty[u % L::kK], (uint32_t)(u / L::kK - 1) & 1)) break;
                load(u, false);
                ++ku;
                if (u >= L::kV && !wait(&sh.v_empty[u % L::kV], (uint32_t)(u / L::kV - 1) & 1)) break;
                load(u, true);
                ++vu;
            }
            // what is in flight lands before the CTA leaves (a wait of a second each at most)
            mbar_wait(&sh.q_full, 0);
            for (int u = max(0, ku - L::kK); u < ku; ++u) mbar_wait(&sh.k_full[u % L::kK], (uint32_t)(u / L::kK) & 1);
            for (int u = max(0, vu - L::kV); u < vu; ++u) mbar_wait(&sh.v_full[u % L::kV], (uint32_t)(u / L::kV) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        // the whole warp goes through this, one lane issues
        const int n_tiles = of_warp(count), first = of_warp(all.ns), w0 = of_warp(all.w0);
        if (n_tiles > 0) {
            const uint32_t leader = elect_one(), tb = (uint32_t)of_warp((int)tbase);
            WindowTiles mine[2];
            int done[2] = {0, 0}, total[2];   // tiles multiplied into O, and how many there are
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                mine[s].ns = of_warp(st[s].tiles.ns), mine[s].w0 = of_warp(st[s].tiles.w0), mine[s].w1 = of_warp(st[s].tiles.w1);
                total[s] = mine[s].empty() ? 0 : mine[s].ns + mine[s].w1 - mine[s].w0 + 1;
            }
            const uint32_t base = (uint32_t)of_warp((int)smem_u32(sm));
            const uint64_t dq = sw128_desc(base + L::kQ, 0, 1024), dk = sw128_desc(base + L::kKs, 0, 1024),
                           dv = sw128_desc(base + L::kVs, L::kRow, 1024);
            int ki = 0, vi = 0;               // stages of the next keys and of the current values, and their phases
            uint32_t kph = 0, vph = 0;
            auto scores = [&](int s) {
                const uint64_t q = dq + (uint32_t)(s * (L::kTile >> 4)), k = dk + (uint32_t)(ki * (L::kTile >> 4));
                const uint32_t to = tb + 128 * s;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t at = ((i >> 2) * L::kRow + (i & 3) * 32) >> 4;
                    warp_mma_f16(leader, to, q + at, k + at, idesc_s, i > 0);
                }
                warp_mma_commit(leader, &sh.s_full[s]);
            };
            auto product = [&](int s, int half) {   // with 64 keys' values
                const uint64_t v = dv + (uint32_t)(vi * (L::kTile >> 4) + half * (64 * 128 >> 4));
                const uint32_t to = tb + L::kO + D * s, from = tb + 128 * s + 32 * half;
                warp_mma_f16_ta(leader, to, from, v, idesc_o, done[s] > 0 || half);
#pragma unroll
                for (int i = 1; i < 4; ++i) warp_mma_f16_ta(leader, to, from + 8 * i, v + (uint32_t)(2048 * i >> 4), idesc_o, 1);
            };
            auto tile_of = [&](int u) { return u < first ? u : w0 + u - first; };
            bool ok = warp_wait(wait, &sh.q_full, 0) && warp_wait(wait, &sh.k_full[0], 0);
            fence_after_sync();
            if (ok) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (mine[s].has(tile_of(0))) scores(s);
                warp_mma_commit(leader, &sh.k_empty[0]);
                if (++ki == L::kK) ki = 0, kph ^= 1;
            }
            for (int u = 0; ok && u < n_tiles; ++u) {
                const int t = tile_of(u), tn = tile_of(u + 1);
                const bool more = u + 1 < n_tiles;
                ok = more ? warp_wait3(wait, &sh.v_full[vi], vph, &sh.v_ok[vi], vph, &sh.k_full[ki], kph)
                          : warp_wait2(wait, &sh.v_full[vi], vph, &sh.v_ok[vi], vph);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (ok && mine[s].has(t)) {
                        ok = warp_wait(wait, &sh.p_half[s], (uint32_t)done[s] & 1);
                        fence_after_sync();
                        if (ok) product(s, 0);
                        ok = ok && warp_wait(wait, &sh.p_ready[s], (uint32_t)done[s] & 1);
                        fence_after_sync();
                        if (ok) {
                            product(s, 1);
                            ++done[s];
                            if (done[s] == total[s]) warp_mma_commit(leader, &sh.o_full[s]);
                        }
                    }
                    if (ok && more && mine[s].has(tn)) scores(s);
                }
                if (!ok) break;
                warp_mma_commit(leader, &sh.v_empty[vi]);
                if (++vi == L::kV) vi = 0, vph ^= 1;
                if (more) {
                    warp_mma_commit(leader, &sh.k_empty[ki]);
                    if (++ki == L::kK) ki = 0, kph ^= 1;
                }
            }
            warp_mma_commit(leader, &sh.drain);
            mbar_wait(&sh.drain, 0);
        }
    } else if (warp < 4) {
        // ------------------------------------------------- values that are not finite
        const int w = warp - 2, row0 = 64 * w;
        int cuts = 0;
        for (int u = 0; u < count; ++u) {
            const int t = tile_at(u), i = u % L::kV;
            if (!warp_wait(wait, &sh.v_full[i], (uint32_t)(u / L::kV) & 1)) break;
            bool cut = false;
            for (int s = 0; s < 2; ++s) cut |= st[s].tiles.has(t) && window_partial(t, st[s].p0, st[s].p1, d.window, d.sinks);
            if (cut) {
                uint4 *v = (uint4 *)(sm + L::kVs + i * L::kTile);
                uint32_t acc = 0;
                for (int b = 0; b < D / 64; ++b)
                    for (int x = lane; x < 64 * 8; x += 32) {   // 64 rows of 128 bytes, whatever their swizzle
                        const uint4 q = v[b * (L::kRow / 16) + row0 * 8 + x];
                        acc = finite_probe<T>(q.x, acc), acc = finite_probe<T>(q.y, acc);
                        acc = finite_probe<T>(q.z, acc), acc = finite_probe<T>(q.w, acc);
                    }
                const uint32_t e = exponent_bits<T>();
                const bool dirty = __any_sync(0xffffffffu, (acc & e) == e || ((acc >> 16) & e) == e);
                for (int h = 0; h < 2; ++h) {
                    const int r = row0 + 32 * h + lane;
                    bool bad = false;
                    for (int x = 0; dirty && x < D; ++x) {
                        uint16_t *at = (uint16_t *)(sm + L::kVs + i * L::kTile + (x >> 6) * L::kRow + sw128_off(r, x & 63));
                        if ((*at & e) == e) *at = 0, bad = true;
                    }
                    const uint32_t bits = __ballot_sync(0xffffffffu, bad && (int64_t)t * 128 + r < sp.Lk);
                    if (lane == 0 && cuts < kCutTiles) {
                        sh.bad[cuts][2 * w + h] = bits;
                        sh.cut_tile[cuts] = t;
                        if (bits) sh.any_bad = 1;
                    }
                }
                if (dirty) fence_async_smem();
                ++cuts;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.v_ok[i]);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int s = (warp - 4) >> 2, r = tid & 127;
        const Subtile &me = st[s];
        const uint32_t ts = tbase + 128 * s + ((uint32_t)(warp & 3) << 21), to = tbase + L::kO + D * s + ((uint32_t)(warp & 3) << 21);
        const int pos = past + me.i0 + r;
        const float c = d.scale * 1.4426950408889634f;
        float m = -INFINITY, l = 0.0f;
        int seen = 0;
        bool ok = true;
        for (int u = 0; u < count; ++u) {
            const int t = tile_at(u);
            if (!me.tiles.has(t)) continue;
            if (!(ok = warp_wait(wait, &sh.s_full[s], (uint32_t)seen & 1))) break;
            fence_after_sync();
            float x[2][64];
            tmem_ld64(ts, x[0]);
            uint32_t see[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
            const bool cut = window_partial(t, me.p0, me.p1, d.window, d.sinks);
            if (cut) {
                // of this tile's keys: up to hi, and from lo on or below sk. As bits: element by element compared, the compiler
                // makes a branch of each (7 us a tile, measured)
                const int64_t a = (int64_t)t * 128;
                const int hi = (int)max((int64_t)-1, min((int64_t)127, pos - a)), lo = (int)max((int64_t)0, min((int64_t)128, (int64_t)pos - d.window + 1 - a));
                const int sk = (int)max((int64_t)0, min((int64_t)128, d.sinks - a));
#pragma unroll
                for (int b = 0; b < 4; ++b) see[b] = low_bits(hi + 1 - 32 * b) & (~low_bits(lo - 32 * b) | low_bits(sk - 32 * b));
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h) tmem_ld64(ts + 64, x[1]);
                if (cut)
#pragma unroll
                    for (int i = 0; i < 64; ++i) x[h][i] = see[2 * h + (i >> 5)] & (1u << (i & 31)) ? x[h][i] : -INFINITY;
#pragma unroll
                for (int i = 0; i < 64; i += 8)
#pragma unroll
                    for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], x[h][i + 2 * q], x[h][i + 2 * q + 1]);
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            // a first maximum, or one that grew by more than 2^8: the sums so far move to it
            const bool grow = top > m && (m == -INFINITY || (top - m) * c > 8.0f);
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? exp2f((m - top) * c) : 1.0f;   // 0 for a first one
                if (grow) m = top;
                l *= f;
                if (seen > 0) {   // the products so far are complete: S of this tile came after them
#pragma unroll
                    for (int b = 0; b < D; b += 32) {
                        float o[32];
                        tmem_ld32(to + b, o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= f;
                        tmem_st32_nw(to + b, o);
                    }
                }
            }
            const float2 cc = splat2(c), mc = splat2(m == -INFINITY ? 0.0f : fmaf(-m, c, kRaised<T>));
            float2 sum[2] = {splat2(0.0f), splat2(0.0f)};
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 e = fma2(make_float2(x[b >> 1][32 * (b & 1) + 2 * i], x[b >> 1][32 * (b & 1) + 2 * i + 1]), cc, mc);
                    e = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                    sum[i & 1] = add2(sum[i & 1], e);
                    w[i] = __uint_as_float(pack2<T>(e.x, e.y));
                }
                tmem_st16_nw(ts + 16 * b, w);
                if (b == 1) {   // the product with the first 64 keys' values may start
                    tmem_wait_st();
                    warp_arrive(&sh.p_half[s]);
                }
            }
            l += sum[0].x + sum[0].y + sum[1].x + sum[1].y;
            tmem_wait_st();
            warp_arrive(&sh.p_ready[s]);
            ++seen;
        }
        if (ok && seen > 0 && (ok = warp_wait(wait, &sh.o_full[s], 0))) fence_after_sync();
        // the checking warps are through with all tiles
        asm volatile("bar.sync 1, 320;" ::: "memory");
        const bool valid = r < me.rows && ok;
        const int64_t tok = sp.q0 + me.i0 + r, ntok = (int64_t)d.B * d.Tq;
        const float inv = pos < 0 ? 0.0f : 1.0f / l;
        // through the subtile's own Q, which no product reads any more, so that a warp stores whole rows (16 bytes of 32
        // rows at a time took 3 us)
        unsigned char *stage = sm + L::kQ + s * L::kTile;
#pragma unroll
        for (int b = 0; b < D; b += 32) {
            float o[32];
            if (seen > 0) tmem_ld32(to + b, o);
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (pos >= 0) {
                    w.x = pack2<T>(o[i] * inv, o[i + 1] * inv), w.y = pack2<T>(o[i + 2] * inv, o[i + 3] * inv);
                    w.z = pack2<T>(o[i + 4] * inv, o[i + 5] * inv), w.w = pack2<T>(o[i + 6] * inv, o[i + 7] * inv);
                }
                *(uint4 *)(stage + ((b + i) >> 6) * L::kRow + r * 128 + (((((b + i) & 63) >> 3) ^ (r & 7)) << 4)) = w;
            }
        }
        __syncwarp();
        const int row0 = r & ~31, rows = ok ? min(32, me.rows - row0) : 0;
        T *out = (T *)p.out + ((sp.q0 + me.i0 + row0) * d.Hq + me.head) * d.d;
#pragma unroll
        for (int x = lane; x < 32 * (D / 8); x += 32) {
            const int q = x / (D / 8), ch = x % (D / 8);
            if (q < rows && 8 * ch < d.d)
                *(uint4 *)(out + (int64_t)q * d.Hq * d.d + 8 * ch) =
                    *(const uint4 *)(stage + (ch >> 3) * L::kRow + (row0 + q) * 128 + (((ch & 7) ^ ((row0 + q) & 7)) << 4));
        }
        __syncwarp();
        float lse = pos < 0 ? -INFINITY : (m * c + (log2f(l) - kRaised<T>)) * 0.6931471805599453f;
        // rows that see a value that is not finite
        if (*(volatile int *)&sh.any_bad) {
            bool dirty = false;
            int cuts = 0;
            for (int u = 0; u < count && cuts < kCutTiles; ++u) {
                bool cut = false;
                for (int q = 0; q < 2; ++q) cut |= st[q].tiles.has(tile_at(u)) && window_partial(tile_at(u), st[q].p0, st[q].p1, d.window, d.sinks);
                if (!cut) continue;
                for (int w = 0; w < 4; ++w)
                    for (uint32_t bits = sh.bad[cuts][w]; bits; bits &= bits - 1) {
                        const int j = sh.cut_tile[cuts] * 128 + 32 * w + __ffs(bits) - 1;
                        dirty |= j <= pos && (pos - j < d.window || j < d.sinks);
                    }
                ++cuts;
            }
            unsigned todo = __ballot_sync(0xffffffffu, dirty && valid && pos >= 0);
            while (todo) {
                const int src = __ffs(todo) - 1;
                todo &= todo - 1;
                const int i = me.i0 + (r & ~31) + src;
                float o[D / 32], ls;
                row_forward<T, D / 32>((const T *)p.q + sp.qoff + i * d.q_stride_t + (int64_t)me.head * d.d, (const T *)p.k + sp.koff + (int64_t)hk * d.d,
                                       (const T *)p.v + sp.voff + (int64_t)hk * d.d, d.k_stride_t, d.v_stride_t, d.d, d.scale, past + i, d.window,
                                       d.sinks, lane, o, ls);
                __syncwarp();
                row_store<T, D / 32>((T *)p.out + ((sp.q0 + i) * d.Hq + me.head) * d.d, d.d, lane, o);
                if (lane == src) lse = ls;
            }
        }
        if (p.lse && valid) p.lse[me.head * ntok + tok] = lse;
    }
    if (warp == 2 || warp == 3) asm volatile("bar.arrive 1, 320;" ::: "memory");
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && sh.gave_up) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    if (warp == 1) tmem_dealloc(tbase, 512);
}

bool strides_fit(const gdn_window_attention_desc &d) {
    const int64_t t[] = {d.Tq > 1 ? d.q_stride_t : 0, d.Tk > 1 ? d.k_stride_t : 0, d.Tk > 1 ? d.v_stride_t : 0,
                         d.B > 1 ? d.q_stride_b : 0, d.B > 1 ? d.k_stride_b : 0, d.B > 1 ? d.v_stride_b : 0};
    for (const int64_t s : t)
        if (s % 8 || s >= ((int64_t)1 << 38)) return false;   // a map's pitches: multiples of 16 bytes below 2^40
    return true;
}

}  // namespace

bool window_tc_fits(const gdn_window_attention_desc &d) { return d.dtype != GDN_F32 && d.d <= 128 && d.d % 8 == 0 && strides_fit(d); }

bool window_tc_supports(const WindowProblem &p) {
    return window_tc_fits(p.d) && ptr_aligned(p.q, 16) && ptr_aligned(p.k, 16) && ptr_aligned(p.v, 16) &&
           ptr_aligned(p.out, 16) && ptr_aligned(p.out_in, 16) && ptr_aligned(p.dout, 16) && ptr_aligned(p.dq, 16) && ptr_aligned(p.dk, 16) &&
           ptr_aligned(p.dv, 16);
}

bool window_head_map(CUtensorMap *m, const gdn_window_attention_desc &d, const void *base, int heads, int tokens, int64_t sb, int64_t st,
                     int *rows, uint32_t box) {
    const bool one = d.B == 1 || sb == 0;
    *rows = one ? 0 : 1;
    const uint64_t pitch_t = (uint64_t)(tokens > 1 ? st : (int64_t)heads * d.d) * 2;
    return encode_head_map(m, d.dtype, base, one ? 1 : d.B, tokens, heads, d.d, one ? pitch_t * 8 : (uint64_t)sb * 2, pitch_t, box);
}

cudaError_t launch_window_forward_tc(const WindowProblem &p, cudaStream_t s) {
    const gdn_window_attention_desc &d = p.d;
    WindowMaps maps;
    memset(&maps, 0, sizeof(maps));
    if (!window_head_map(&maps.q, d, p.q, d.Hq, d.Tq, d.q_stride_b, d.q_stride_t, &maps.q_rows, 128) ||
        !window_head_map(&maps.k, d, p.k, d.Hk, d.Tk, d.k_stride_b, d.k_stride_t, &maps.k_rows, 128) ||
        !window_head_map(&maps.v, d, p.v, d.Hk, d.Tk, d.v_stride_b, d.v_stride_t, &maps.v_rows, 128))
        return cudaErrorInvalidValue;
    const int pair_heads = d.Hq / d.Hk % 2 == 0, units = pair_heads ? d.Hq / 2 : d.Hq, rows = pair_heads ? 128 : 256;
    const int64_t tiles = p.cu ? cdiv64(d.Tq, rows) + d.N : (int64_t)d.B * cdiv64(d.Tq, rows);
    if (tiles * units > 0x7fffffff) return cudaErrorInvalidValue;
    if (p.cu) {
        const cudaError_t e = launch_window_tables(p, rows, 128, s);
        if (e != cudaSuccess) return e;
    }
    auto go = [&](auto kernel, size_t smem) {
        const cudaError_t e = allow_shared(kernel, smem);
        if (e != cudaSuccess) return e;
        kernel<<<(unsigned)(tiles * units), kThreads, smem, s>>>(maps, p, pair_heads, units);
        return cudaGetLastError();
    };
    // one CTA per SM: each holds all of the tensor memory
    constexpr size_t s128 = FwdShape<128>::kBytes, s64 = FwdShape<64>::kBytes < 117 * 1024 ? 117 * 1024 : FwdShape<64>::kBytes;
    if (d.d <= 64) return d.dtype == GDN_BF16 ? go(window_forward_tc<__nv_bfloat16, 64>, s64) : go(window_forward_tc<__half, 64>, s64);
    return d.dtype == GDN_BF16 ? go(window_forward_tc<__nv_bfloat16, 128>, s128) : go(window_forward_tc<__half, 128>, s128);
}

}  // namespace gdn
