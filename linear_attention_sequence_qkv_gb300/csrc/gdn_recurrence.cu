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
//   - a tile has 4 tokens for each of the CTA's token groups (4 warps x 2, or x 4 with
//     fp32). A thread owns 4 channels of one group: it composes its tokens in registers
//     and the groups of a warp compose by shuffles. A fifth warp composes the warps'
//     maps, exchanges them with the other CTAs of the cluster and hands the carried
//     state back; each thread then finishes its tokens. The forward computes the maps of
//     the next tile meanwhile.
//   - a sequence's first token has its initial state written into u and a decay of -0,
//     which cuts the chain: packed sequences are nothing special to the scan, whatever
//     their lengths.
//
// The order of every composition and sum is fixed by the sizes and by whether TMA can take
// the rows, so results are run-to-run identical. Tiles come in by TMA (from rows that are
// 16-byte aligned; other tensors are read element by element, a tile ahead).
//
// What bounds them, measured: fp32 forward the bandwidth (65536 x 4096 634 us, the copy
// rate); 16-bit types, and the backward, the issue rate and the latency of a step together, 42
// instructions per element forward and 67 backward (131072 x 4096 bf16 forward 1036 us, 61 %
// of the copy rate; 65536 x 4096 in 16 sequences 615 us forward, which also writes the states,
// and 1149 us backward, 52 %; fp32 1626 us backward without sequences, 70 %). With few chains a
// step's latency alone.
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
    float *hT, *cs;              // final states; states carried into every 4th token
    int32_t *status;
    const float *grad_final;
    void *dx, *da, *db;
    float *dA_log, *ddt_bias, *dh0, *part;
    int slabs, ntiles, wait_immediate;
    int recomputed;              // backward: the states come from a forward of the same call
};

struct RecMaps {
    CUtensorMap x, a, b, dy;
};

// A tile: R tokens for each of the WARPS x G token groups of a CTA by 128 bytes of channels. One more warp
// carries the state and fetches the tiles.
template <typename T, int R_, int WARPS_, int STAGES_> struct Tile {
    using E = T;
    static constexpr int R = R_, WARPS = WARPS_, STAGES = STAGES_, THREADS = 32 * (WARPS + 1);
    static constexpr int LR = 128 / (4 * (int)sizeof(T));   // lanes per token row, 4 channels each
    static constexpr int G = 32 / LR;                       // token groups per warp
    static constexpr int NG = WARPS * G;                    // per CTA
    static constexpr int TT = NG * R;                       // tokens
    static constexpr int CH = LR * 4;                       // channels
    static constexpr int kTensor = TT * 128;                // bytes of one tensor's tile
};
constexpr int kMaxCluster = 16;   // more than 8 needs an opt-in
template <typename T> using FwdTile = Tile<T, 4, 4, 4>;
template <typename T> using BwdTile = Tile<T, GDN_RECURRENCE_CHUNK, 4, 2>;
template <typename T> constexpr int kBwdStash = 3 * BwdTile<T>::R * 32 * BwdTile<T>::WARPS * 16;   // bytes

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
template <bool PACKED> __device__ __forceinline__ float2 apply2(float2 A, float2 B, float2 h) {
    const float2 r = fma2(A, h, B);
    return PACKED ? cut2(A, B, r) : r;
}
template <bool PACKED> __device__ __forceinline__ float2 compose2(float2 A, float2 pA) {
    const float2 r = mul2(A, pA);
    return PACKED ? cut2(A, A, r) : r;
}
template <bool PACKED> __device__ __forceinline__ F4 apply(const F4 &A, const F4 &B, const F4 &h) {
    F4 r = fma4(A, h, B);
    if (PACKED) r = {cut2(A.lo, B.lo, r.lo), cut2(A.hi, B.hi, r.hi)};
    return r;
}
// the A of a map after one with pA
template <bool PACKED> __device__ __forceinline__ F4 compose(const F4 &A, const F4 &pA) {
    F4 r = mul4(A, pA);
    if (PACKED) r = {cut2(A.lo, A.lo, r.lo), cut2(A.hi, A.hi, r.hi)};
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

// Up to four channels of a row in global memory, STEP apart; nc of them exist. VEC: adjacent ones of an aligned row,
// and nc is 4 or 0.
template <typename T, bool VEC, int STEP = 1>
__device__ __forceinline__ F4 load_row(const T *p, int nc) {
    if (VEC) return nc > 0 ? unpack4<T>(p) : f4(0.f);
    return {make_float2(nc > 0 ? to_f<T>(p[0]) : 0.f, nc > 1 ? to_f<T>(p[STEP]) : 0.f),
            make_float2(nc > 2 ? to_f<T>(p[2 * STEP]) : 0.f, nc > 3 ? to_f<T>(p[3 * STEP]) : 0.f)};
}
template <typename T, bool VEC, int STEP = 1>
__device__ __forceinline__ void store_row(T *p, const F4 &v, int nc) {
    if (VEC) {
        if (nc > 0) pack4<T>(p, v);
        return;
    }
    if (nc > 0) p[0] = from_f<T>(v.lo.x);
    if (nc > 1) p[STEP] = from_f<T>(v.lo.y);
    if (nc > 2) p[2 * STEP] = from_f<T>(v.hi.x);
    if (nc > 3) p[3 * STEP] = from_f<T>(v.hi.y);
}
// four fp32 values of a row whose alignment is not known
template <int STEP> __device__ __forceinline__ F4 load_words(const float *p, int nc) { return load_row<float, false, STEP>(p, nc); }
template <int STEP> __device__ __forceinline__ void store_words(float *p, const F4 &v, int nc) { store_row<float, false, STEP>(p, v, nc); }

// The channels of lane q of a token's LR lanes, from a slab's first channel on: four adjacent ones, or without TMA
// every LR-th, so that the lanes of an element-wise access are neighbours in memory (3 x 19422 x 1147 fp32 with its
// gradient 940 us, with adjacent ones 1175).
template <typename L, bool TMA> struct Columns {
    static constexpr int STEP = TMA ? 1 : L::LR;
    int ch, nc;   // the first, and how many exist
    __device__ __forceinline__ Columns(int slab, int q, int D) {
        ch = slab * L::CH + (TMA ? q * 4 : q);
        nc = min(4, max(0, (D - ch + STEP - 1) / STEP));
    }
    static __device__ __forceinline__ int of(int i) { return TMA ? i : i / 4 + i % 4 * L::LR; }   // value i of a slab's 4 LR
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes into the shared memory of CTA `rank` of the cluster at this CTA's address `p`, counted by the
// barrier at this CTA's address `bar` there. Data and signal travel together: a cluster barrier instead
// would wait for every store to global memory before it.
__device__ __forceinline__ void remote_store(uint32_t p, uint32_t bar, uint32_t rank, float2 a, float2 b) {
    asm volatile("{\n\t.reg .b32 ra, rb;\n\tmapa.shared::cluster.u32 ra, %0, %2;\n\tmapa.shared::cluster.u32 rb, %1, %2;\n\t"
                 "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [ra], {%3, %4, %5, %6}, [rb];\n\t}"
                 :: "r"(p), "r"(bar), "r"(rank), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y) : "memory");
}
// A word into the shared memory of CTA `rank`, seen there after the next cluster barrier
__device__ __forceinline__ void remote_word(uint32_t p, uint32_t rank, uint32_t v) {
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\tst.shared::cluster.u32 [ra], %2;\n\t}"
                 :: "r"(p), "r"(rank), "r"(v) : "memory");
}
// Counts bytes that an mbarrier expects and nobody sends as arrived
__device__ __forceinline__ void never_sent(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" :: "r"(tc::smem_u32(bar)), "r"(bytes) : "memory");
}

// A warp's wait for an mbarrier's phase, a second at most (the library's mbar_wait); all lanes call it and leave it with
// the same answer, since what follows are instructions of the whole warp. `failed` makes every later wait a single test,
// so that a CTA whose copies do not arrive ends soon.
__device__ __forceinline__ void bounded_wait(uint64_t *bar, uint32_t phase, bool immediate, bool &failed) {
    if (__all_sync(0xffffffffu, tc::mbar_test_now(bar, phase))) return;
    if (failed || immediate || !__all_sync(0xffffffffu, tc::mbar_wait(bar, phase))) failed = true;
}

// Named barriers of the CTA: all its threads arrive, one side without waiting.
constexpr int kMapsBar = 1, kStatesBar = 3;   // and the next: by step parity
__device__ __forceinline__ void named_arrive(int id, int threads) {
    asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// The cross-thread part of the walk, for one CTA. The compute warps compose the maps (A, B) of their token
// groups in walking order (FWD: rising groups, else falling), hand one map per warp to the carry warp, and go on
// to the next tile; the carry warp composes them to the CTA's map, exchanges it with the cluster, takes the
// state through it all, and hands back the state carried into each warp. Everything is double-buffered by step
// parity: a compute warp hands in its map of step k after it has the state of step k - 2, so what it overwrites
// has been read. The CTA's own signals are named barriers, at which a warp waits without issuing anything
// (polling mbarriers took up to a third of the issue slots).
template <typename L, bool FWD, bool PACKED> struct Chain {
    float4 wA[2][L::WARPS][L::LR], wB[2][L::WARPS][L::LR];   // maps of the warps
    float4 wc[2][L::WARPS][L::LR];                           // the state carried into each warp
    uint64_t agg_bar[2];                                     // the cluster's maps have arrived
    uint64_t full[L::STAGES];                                // a tile has arrived
    uint32_t sent[kMaxCluster];                              // steps whose maps each CTA of the cluster has sent
    uint32_t gave_up;                                        // the carry warp lost something
    static constexpr uint32_t kMapBytes = L::CH / 2 * 16;    // of one CTA

    __device__ __forceinline__ void init(uint32_t cs, int steps) {      // all threads
        if (threadIdx.x < kMaxCluster) sent[threadIdx.x] = steps;
        if (threadIdx.x == 0) {
            gave_up = 0;
            for (int i = 0; i < 2; ++i) tc::mbar_init(&agg_bar[i], 1);
            for (int i = 0; i < L::STAGES; ++i) tc::mbar_init(&full[i], 1);
            tc::mbar_init_fence();
        }
        if (cs > 1) cluster_sync();   // no CTA sends before every barrier is set up
        else __syncthreads();
    }

    // Compute warp: composes the groups' maps of step k; (eA, eB) is the map from the state carried into the
    // warp to the one carried into this group.
    __device__ __forceinline__ void hand_in(F4 A, F4 B, F4 &eA, F4 &eB, int k, int warp, int lane) {
        const int g = lane / L::LR, q = lane % L::LR;
        const int og = FWD ? g : L::G - 1 - g, ow = FWD ? warp : L::WARPS - 1 - warp;   // walking order
#pragma unroll
        for (int off = 1; off < L::G; off *= 2) {
            eA = shfl4<FWD>(A, off * L::LR), eB = shfl4<FWD>(B, off * L::LR);
            const F4 nB = apply<PACKED>(A, B, eB), nA = compose<PACKED>(A, eA);
            if (og >= off) B = nB, A = nA;
        }
        if (og == L::G - 1) {
            wA[k & 1][ow][q] = to4(A);
            wB[k & 1][ow][q] = to4(B);
        }
        if (L::G > 2) eA = shfl4<FWD>(A, L::LR), eB = shfl4<FWD>(B, L::LR);
        if (og == 0) eA = f4(1.f), eB = f4(0.f);
        named_arrive(kMapsBar + (k & 1), L::THREADS);
    }
    // Compute warp: the state carried into the group in step k.
    __device__ __forceinline__ F4 take(const F4 &eA, const F4 &eB, int k, int warp, int lane) {
        named_sync(kStatesBar + (k & 1), L::THREADS);
        return apply<PACKED>(eA, eB, f4(wc[k & 1][FWD ? warp : L::WARPS - 1 - warp][lane % L::LR]));
    }

    // Carry warp, step k, two channels a lane. `carry`: the state carried into the step, the same in all CTAs of
    // the cluster. agg: [2][cs][CH / 2] of (A, A, B, B), the maps of the cluster's CTAs by step parity. A CTA writes
    // agg[k % 2] of another only after it has that CTA's map of step k - 1, which that CTA's carry warp sends
    // after it is done with step k - 2. `lost`: something did not arrive; nothing more is sent or waited for.
    // immediate: the test mode of the waits. This is the latency of a step: everything else is done beside it.
    __device__ __forceinline__ void carry_step(float2 &carry, int lane, uint32_t rank, uint32_t cs, int k, float4 *agg, bool immediate, bool &lost) {
        constexpr int kHalf = L::CH / 2;
        const int c2 = lane % kHalf;
        named_sync(kMapsBar + (k & 1), L::THREADS);
        float2 a[L::WARPS], b[L::WARPS];
#pragma unroll
        for (int w = 0; w < L::WARPS; ++w) {
            a[w] = ((const float2 *)wA[k & 1][w])[c2];
            b[w] = ((const float2 *)wB[k & 1][w])[c2];
        }
        float2 c = carry;   // carried into this CTA's tile
        if (cs > 1) {
            float2 tA = a[0], tB = b[0];
#pragma unroll
            for (int w = 1; w < L::WARPS; ++w) {
                tB = apply2<PACKED>(a[w], b[w], tB);
                tA = compose2<PACKED>(a[w], tA);
            }
            float4 *at = agg + (k & 1) * cs * kHalf;
            if (!lost) {
                const uint32_t mine = tc::smem_u32(at + rank * kHalf + c2), bar = tc::smem_u32(&agg_bar[k & 1]);
                if (lane == 0) tc::mbar_expect_tx(&agg_bar[k & 1], cs * kMapBytes);
                if (lane < kHalf)
#pragma unroll 4
                    for (uint32_t r = 0; r < cs; ++r) remote_store(mine, bar, r, tA, tB);
                __syncwarp();
                bounded_wait(&agg_bar[k & 1], (k >> 1) & 1, immediate, lost);
            }
#pragma unroll 4
            for (uint32_t r = 0; r < cs; ++r) {
                const float4 m = at[r * kHalf + c2];
                if (r == rank) c = carry;
                carry = apply2<PACKED>(make_float2(m.x, m.y), make_float2(m.z, m.w), carry);
            }
        }
#pragma unroll
        for (int w = 0; w < L::WARPS; ++w) {
            if (lane < kHalf) ((float2 *)wc[k & 1][w])[c2] = c;
            c = apply2<PACKED>(a[w], b[w], c);
        }
        if (cs == 1) carry = c;
        named_arrive(kStatesBar + (k & 1), L::THREADS);
    }

    // The carry warp after its last step: it has issued the copies of `issued` tiles (first lane), of which the last ones
    // may not have been waited for, and sent its maps of `steps_sent` steps.
    __device__ __forceinline__ void end_carry(bool copies, int issued, int steps_sent, bool lost, int lane, uint32_t rank, uint32_t cs, int32_t *status) {
        if (copies && lane == 0)
            for (int k = max(0, issued - L::STAGES); k < issued; ++k) tc::mbar_wait(&full[k % L::STAGES], (k / L::STAGES) & 1);
        if (lost) {
            if (lane == 0) gave_up = 1, *status = GDN_ERR_DEVICE_TIMEOUT;
            if (lane < (int)cs) remote_word(tc::smem_u32(&sent[rank]), lane, steps_sent);
        }
        __syncwarp();
    }

    // The end of a CTA; all threads. No map may be on its way to it when it leaves. A CTA that lost nothing has had them
    // all. One that did, and so sent its own of s steps, may not have all of step s - 1 (those of the CTAs that sent
    // theirs are still waited for), nor any of step s, which it does not expect and a CTA that had all of step s - 1
    // sends. Nothing later: step s + 1 is sent only with this CTA's map of step s.
    __device__ __forceinline__ void leave(uint32_t rank, uint32_t cs) {
        __syncwarp();
        if (cs == 1) {
            __syncthreads();
            return;
        }
        cluster_sync();   // nobody sends any more, and everyone's `sent` is known
        if (!gave_up || threadIdx.x != 0) return;
        const int s = (int)sent[rank];
        for (int k = s - 1; k <= s; ++k) {
            uint32_t n = 0;
            for (uint32_t r = 0; r < cs; ++r) n += (int)sent[r] > k;
            if (k == s && n == 0) break;
            if (k == s) tc::mbar_expect_tx(&agg_bar[k & 1], n * kMapBytes);
            else if (n < cs) never_sent(&agg_bar[k & 1], (cs - n) * kMapBytes);
            tc::mbar_wait(&agg_bar[k & 1], (k >> 1) & 1);
        }
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
template <int STEP> __device__ void copy_empty(const RecProblem &p, int row, int ch, int nc, float *dst, const float *src, int group, int groups) {
    if (dst == nullptr) return;
    for (int n = (p.cu ? 0 : row) + group; n < (p.cu ? p.d.N : row + 1); n += groups) {
        if (p.cu ? p.cu[n] != p.cu[n + 1] : p.d.T != 0) continue;
        store_words<STEP>(dst + (int64_t)n * p.d.D + ch, src ? load_words<STEP>(src + (int64_t)n * p.d.D + ch, nc) : f4(0.f), nc);
    }
}

// Without TMA: R tokens by a lane's four channels of a tensor, element by element, zeros where there is nothing. The loads
// of the next tile are issued while this one is worked on.
template <int STEP, typename T, int R>
__device__ __forceinline__ void fetch_elements(T (&v)[R][4], const T *p, int64_t stride, int tokens, int nc) {
#pragma unroll
    for (int r = 0; r < R; ++r, p += stride)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[r][c] = r < tokens && c < nc ? p[c * STEP] : from_f<T>(0.f);
}
template <typename T> __device__ __forceinline__ F4 of_elements(const T (&v)[4]) {
    return {make_float2(to_f<T>(v[0]), to_f<T>(v[1])), make_float2(to_f<T>(v[2]), to_f<T>(v[3]))};
}

// exp(A_log) and dt_bias log2(e) of four channels
template <int STEP> __device__ __forceinline__ void channel_params(const RecProblem &p, int ch, int nc, float2 (&rate)[2], float2 (&bias2)[2]) {
    const F4 l = load_words<STEP>(p.A_log + ch, nc), b = load_words<STEP>(p.dt_bias + ch, nc);
    rate[0] = make_float2(expf(l.lo.x), expf(l.lo.y));
    rate[1] = make_float2(expf(l.hi.x), expf(l.hi.y));
    bias2[0] = mul2(b.lo, splat2(kLog2e));
    bias2[1] = mul2(b.hi, splat2(kLog2e));
}

// While the carry of tile k - 1 travels, the compute warps work on tile k: its decays and writes need only the
// inputs (one tile after the other, 131072 x 4096 bf16 takes 1218 us against 1036). Three CTAs an SM: fp32 and element-by-element
// reads hold more in registers and run two.
template <typename T, bool TMA, bool PACKED>
__global__ void __launch_bounds__(FwdTile<T>::THREADS, sizeof(T) == 2 && TMA ? 3 : 2)
rec_forward_kernel(const __grid_constant__ RecProblem p, const __grid_constant__ RecMaps maps) {
    using L = FwdTile<T>;
    constexpr int kR = L::R;
    extern __shared__ __align__(128) unsigned char smem[];   // TMA: STAGES tiles of a, b, x; then the cluster's maps
    __shared__ Chain<L, true, PACKED> chain;
    const gdn_recurrence_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint32_t cs;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
    const uint32_t rank = cluster_rank();
    const int slab = (int)(blockIdx.x / cs) % p.slabs, row = (int)(blockIdx.x / cs) / p.slabs;
    const bool ok = !PACKED || seqlens_ok(p.cu, d.N, d.T);
    if (blockIdx.x == 0 && tid == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;   // the same in every CTA
    const int steps = (p.ntiles + (int)cs - 1) / (int)cs;
    const int mine = (p.ntiles - 1 - (int)rank + (int)cs) / (int)cs;   // steps in which this CTA has a tile
    chain.init(cs, steps);
    bool failed = false;

    if (warp == L::WARPS) {   // the carry warp
        float4 *agg = (float4 *)(smem + (TMA ? L::STAGES * 3 * L::kTensor : 0));
        bool lost = false;
        int issued = 0;
        auto issue = [&](int k) {
            if (!TMA || lane != 0 || k >= mine) return;
            issued = k + 1;
            uint64_t *bar = &chain.full[k % L::STAGES];
            unsigned char *st = smem + k % L::STAGES * 3 * L::kTensor;
            const int t = (k * (int)cs + (int)rank) * L::TT;
            tc::mbar_expect_tx(bar, 3 * L::kTensor);
            tc::tma_load_3d(st, &maps.a, slab * L::CH, t, row, bar);
            tc::tma_load_3d(st + L::kTensor, &maps.b, slab * L::CH, t, row, bar);
            tc::tma_load_3d(st + 2 * L::kTensor, &maps.x, slab * L::CH, t, row, bar);
        };
        if (p.wait_immediate) __nanosleep(20000);   // the compute warps' first wait cannot be over
        for (int k = 0; k < L::STAGES; ++k) issue(k);
        float2 carry = splat2(0.f);
        int sent = 0;
        for (int k = 0; k < steps; ++k) {
            if (!lost) sent = k + 1;
            chain.carry_step(carry, lane, rank, cs, k, agg, p.wait_immediate, lost);
            // the maps are in, so every warp has read tile k
            if (TMA && k < mine) bounded_wait(&chain.full[k % L::STAGES], (k / L::STAGES) & 1, false, lost);   // long since
            if (!lost) issue(k + L::STAGES);
            __syncwarp();
        }
        chain.end_carry(TMA, issued, sent, lost, lane, rank, cs, p.status);
    } else {
        const int g = lane / L::LR, q = lane % L::LR;
        const Columns<L, TMA> col(slab, q, d.D);
        const int ch = col.ch, nc = col.nc;
        constexpr int kStep = Columns<L, TMA>::STEP;
        const int tg = (warp * L::G + g) * kR;   // this group's first token in a tile
        const GateConst C(!TMA && sizeof(T) == 2);
        float2 rate[2], bias2[2];
        channel_params<kStep>(p, ch, nc, rate, bias2);
        if (rank == 0) copy_empty<kStep>(p, row, ch, nc, p.hT, p.h0, warp * L::G + g, L::NG);
        Seq seq, seq_out;   // at the tile whose decays are computed, and at the one that is finished
        seq.init(p, row);
        seq_out.init(p, row);

        T ea[kR][4], eb[kR][4], ex[kR][4];   // without TMA: the next tile's elements
        auto fetch = [&](int k) {
            const int tile = k * (int)cs + (int)rank, t0 = tile * L::TT + tg;
            if (TMA || tile >= p.ntiles) return;
            fetch_elements<kStep, T, kR>(ea, (const T *)p.a + row * d.a_stride_b + t0 * d.a_stride_t + ch, d.a_stride_t, d.T - t0, nc);
            fetch_elements<kStep, T, kR>(eb, (const T *)p.b + row * d.b_stride_b + t0 * d.b_stride_t + ch, d.b_stride_t, d.T - t0, nc);
            fetch_elements<kStep, T, kR>(ex, (const T *)p.x + row * d.x_stride_b + t0 * d.x_stride_t + ch, d.x_stride_t, d.T - t0, nc);
        };
        fetch(0);
        // decay products P and local values h of tile k's tokens, and the map to the carry warp
        auto begin = [&](int k, F4 (&P)[kR], F4 (&h)[kR], F4 &eA, F4 &eB) {
            const int tile = k * (int)cs + (int)rank, t0 = tile * L::TT + tg;
            if (tile < p.ntiles) {
                auto in = [&](int which, const T (&e)[kR][4], int r) -> F4 {
                    if (TMA)
                        return unpack4<T>(smem + (k % L::STAGES * 3 + which) * L::kTensor + (tg + r) * 128 + q * 4 * sizeof(T));
                    return of_elements<T>(e[r]);
                };
                if (TMA) bounded_wait(&chain.full[k % L::STAGES], (k / L::STAGES) & 1, p.wait_immediate, failed);
                if (PACKED) seq.up_to(p, t0);
                constexpr int kB = 4;   // tokens at a time
#pragma unroll
                for (int r0 = 0; r0 < kR; r0 += kB) {
                    float2 z[2 * kB], t[2 * kB], Y[2 * kB], al[2 * kB], em[2 * kB];
#pragma unroll
                    for (int r = 0; r < kB; ++r) {
                        const F4 a = in(0, ea, r0 + r);
                        z[2 * r] = a.lo;
                        z[2 * r + 1] = a.hi;
                    }
                    decays<2 * kB, 2>(C, z, bias2, rate, t, Y, al, em);
#pragma unroll
                    for (int r = 0; r < kB; ++r) {
                        const F4 b = in(1, eb, r0 + r), x = in(2, ex, r0 + r);
                        P[r0 + r] = {al[2 * r], al[2 * r + 1]};
                        h[r0 + r] = mul4({write_scale2(C, em[2 * r], al[2 * r], b.lo), write_scale2(C, em[2 * r + 1], al[2 * r + 1], b.hi)}, x);
                    }
                }
                fetch(k + 1);
                if (seq.b0 == t0 || (PACKED && seq.b1 < t0 + kR && seq.b1 < d.T)) {   // a sequence starts here
                    Seq m = seq;
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        m.up_to(p, t0 + r);
                        if (m.b0 == t0 + r && t0 + r < d.T) {
                            if (p.h0) h[r] = fma4(P[r], load_words<kStep>(p.h0 + (int64_t)m.n * d.D + ch, nc), h[r]);
                            P[r] = f4(-0.f);
                        }
                        if (r > 0) {
                            h[r] = apply<true>(P[r], h[r], h[r - 1]);
                            P[r] = compose<true>(P[r], P[r - 1]);
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
            chain.hand_in(P[kR - 1], h[kR - 1], eA, eB, k, warp, lane);
        };
        auto finish = [&](int k, F4 (&P)[kR], F4 (&h)[kR], const F4 &eA, const F4 &eB) {
            const F4 c = chain.take(eA, eB, k, warp, lane);
            const int t0 = (k * (int)cs + (int)rank) * L::TT + tg;
            if (t0 >= d.T) return;
            if (p.cs && t0 % GDN_RECURRENCE_CHUNK == 0)
                store_row<float, TMA, kStep>(p.cs + ((int64_t)row * ((d.T + GDN_RECURRENCE_CHUNK - 1) / GDN_RECURRENCE_CHUNK) +
                                              t0 / GDN_RECURRENCE_CHUNK) * d.D + ch, c, nc);
#pragma unroll
            for (int r = 0; r < kR; ++r) h[r] = apply<PACKED>(P[r], h[r], c);
            if (p.out) {
                T *o = (T *)p.out + ((int64_t)row * d.T + t0) * d.D + ch;
                if (TMA && nc == 4 && t0 + kR <= d.T) {
#pragma unroll
                    for (int r = 0; r < kR; ++r, o += d.D) pack4<T>(o, h[r]);
                } else {
#pragma unroll
                    for (int r = 0; r < kR; ++r, o += d.D)
                        if (t0 + r < d.T) store_row<T, TMA, kStep>(o, h[r], nc);
                }
            }
            if (p.hT) {
                if (PACKED) seq_out.up_to(p, t0);
                if (seq_out.b1 <= t0 + kR) {   // a sequence ends here
                    Seq m = seq_out;
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        m.up_to(p, t0 + r);
                        if (m.b1 == t0 + r + 1) store_words<kStep>(p.hT + (int64_t)m.n * d.D + ch, h[r], nc);
                    }
                }
            }
        };
        F4 P0[kR], h0[kR], P1[kR], h1[kR], eA0, eB0, eA1, eB1;
        if (steps > 0) begin(0, P0, h0, eA0, eB0);
        for (int k = 1; k <= steps; k += 2) {
            if (k < steps) begin(k, P1, h1, eA1, eB1);
            finish(k - 1, P0, h0, eA0, eB0);
            if (k < steps) {
                if (k + 1 < steps) begin(k + 1, P0, h0, eA0, eB0);
                finish(k, P1, h1, eA1, eB1);
            }
        }
    }
    if (failed) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    chain.leave(rank, cs);
}

// The reverse walk: c_t = alpha_t (v_t + c_{t+1}), delta_t = v_t + c_{t+1} with v = grad_out, tiles last to
// first. The states before every 4th token come from the forward, so h_{t-1} is recomputed within a thread: 4 bytes
// per 4 elements more to write and to read, against a second scan. A state every 8 tokens would halve that, but double
// the tile and what a thread keeps of it in shared memory: 130 KB a CTA, and one on an SM in place of three.
template <typename T, bool TMA, bool PACKED>
__global__ void __launch_bounds__(BwdTile<T>::THREADS, sizeof(T) == 2 && TMA ? 3 : 2)
rec_backward_kernel(const __grid_constant__ RecProblem p, const __grid_constant__ RecMaps maps) {
    using L = BwdTile<T>;
    constexpr int kR = L::R;
    static_assert(kR <= 32, "the start mask holds one bit per token");
    extern __shared__ __align__(128) unsigned char smem[];   // TMA: STAGES tiles of x, a, b, grad_out; the cluster's maps
    __shared__ Chain<L, false, PACKED> chain;
    __shared__ float red[L::NG][2][L::CH];
    const gdn_recurrence_desc &d = p.d;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    uint32_t cs;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
    const uint32_t rank = cluster_rank();
    const int slab = (int)(blockIdx.x / cs) % p.slabs, row = (int)(blockIdx.x / cs) / p.slabs;
    const bool ok = !PACKED || seqlens_ok(p.cu, d.N, d.T);
    // after a forward of this call, which may have reported a wait that ran out, only what is worse
    if (blockIdx.x == 0 && tid == 0 && !(ok && p.recomputed)) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int steps = (p.ntiles + (int)cs - 1) / (int)cs;
    const int mine = (p.ntiles - 1 - (int)rank + (int)cs) / (int)cs;
    chain.init(cs, steps);
    bool failed = false;

    if (warp == L::WARPS) {
        float4 *agg = (float4 *)(smem + (TMA ? L::STAGES * 4 * L::kTensor : 0) + kBwdStash<T>);
        bool lost = false;
        int issued = 0;
        auto issue = [&](int k) {
            if (!TMA || lane != 0 || k >= mine) return;
            issued = k + 1;
            uint64_t *bar = &chain.full[k % L::STAGES];
            unsigned char *st = smem + k % L::STAGES * 4 * L::kTensor;
            const int t = (p.ntiles - 1 - (k * (int)cs + (int)rank)) * L::TT;
            tc::mbar_expect_tx(bar, 4 * L::kTensor);
            tc::tma_load_3d(st + L::kTensor, &maps.a, slab * L::CH, t, row, bar);
            tc::tma_load_3d(st + 3 * L::kTensor, &maps.dy, slab * L::CH, t, row, bar);
            tc::tma_load_3d(st, &maps.x, slab * L::CH, t, row, bar);
            tc::tma_load_3d(st + 2 * L::kTensor, &maps.b, slab * L::CH, t, row, bar);
        };
        if (p.wait_immediate) __nanosleep(20000);   // the compute warps' first wait cannot be over
        for (int k = 0; k < L::STAGES; ++k) issue(k);
        float2 carry = splat2(0.f);
        int sent = 0;
        for (int k = 0; k < steps; ++k) {
            if (!lost) sent = k + 1;
            chain.carry_step(carry, lane, rank, cs, k, agg, p.wait_immediate, lost);
            // the maps are in, so every warp is done with the tile before
            const int was = k - 1;
            if (was >= 0) {
                if (TMA && was < mine) bounded_wait(&chain.full[was % L::STAGES], (was / L::STAGES) & 1, false, lost);
                if (!lost) issue(was + L::STAGES);
                __syncwarp();
            }
        }
        chain.end_carry(TMA, issued, sent, lost, lane, rank, cs, p.status);
    } else {
        const int g = lane / L::LR, q = lane % L::LR;
        const Columns<L, TMA> col(slab, q, d.D);
        const int ch = col.ch, nc = col.nc;
        constexpr int kStep = Columns<L, TMA>::STEP;
        const int tg = (warp * L::G + g) * kR;
        const GateConst C(!TMA && sizeof(T) == 2);
        float2 rate[2], bias2[2];
        channel_params<kStep>(p, ch, nc, rate, bias2);
        if (rank == 0) copy_empty<kStep>(p, row, ch, nc, p.dh0, p.grad_final, warp * L::G + g, L::NG);
        Seq seq;
        seq.init(p, row);
        seq.up_to(p, d.T - 1);
        // sums of da and of dg g over this thread's tokens: over 16 tiles, over all
        F4 sA[2] = {f4(0.f), f4(0.f)}, sb[2] = {f4(0.f), f4(0.f)};

        T ea[kR][4], ey[kR][4], ex[kR][4], eb[kR][4];   // without TMA: the next tile's a and grad_out, this one's x and b
        auto tile_of = [&](int k) { return p.ntiles - 1 - (k * (int)cs + (int)rank); };
        auto in = [&](int k, int which, const T (&e)[kR][4], int r) -> F4 {
            if (TMA) return unpack4<T>(smem + (k % L::STAGES * 4 + which) * L::kTensor + (tg + r) * 128 + q * 4 * sizeof(T));
            return of_elements<T>(e[r]);
        };
        auto fetch_ay = [&](int k) {
            const int tile = tile_of(k), t0 = tile * L::TT + tg;
            if (TMA || tile < 0) return;
            fetch_elements<kStep, T, kR>(ea, (const T *)p.a + row * d.a_stride_b + t0 * d.a_stride_t + ch, d.a_stride_t, d.T - t0, nc);
            fetch_elements<kStep, T, kR>(ey, (const T *)p.grad_out + ((int64_t)row * d.T + t0) * d.D + ch, d.D, d.T - t0, nc);
        };
        auto fetch_xb = [&](int k) {
            const int tile = tile_of(k), t0 = tile * L::TT + tg;
            if (TMA || tile < 0) return;
            fetch_elements<kStep, T, kR>(ex, (const T *)p.x + row * d.x_stride_b + t0 * d.x_stride_t + ch, d.x_stride_t, d.T - t0, nc);
            fetch_elements<kStep, T, kR>(eb, (const T *)p.b + row * d.b_stride_b + t0 * d.b_stride_t + ch, d.b_stride_t, d.T - t0, nc);
        };
        fetch_ay(0);
        // Between begin and finish a thread keeps three values per token and channel in its own slots of shared
        // memory: em, Y and rate sigmoid(z) (half of the work of recomputing them).
        float4 *stash = (float4 *)(smem + (TMA ? L::STAGES * 4 * L::kTensor : 0)) + tid;
        constexpr int kSlot = 32 * L::WARPS;
        // decays of tile k's tokens (-0 at a sequence's first), their v_t, and the map to the carry warp
        auto begin = [&](int k, F4 (&al)[kR], F4 (&v)[kR], uint32_t &starts, F4 &eA, F4 &eB) {
            const int tile = tile_of(k), t0 = tile * L::TT + tg;
            F4 Q = f4(1.f), c = f4(0.f);
            starts = 0;
            if (tile >= 0) {
                if (TMA) bounded_wait(&chain.full[k % L::STAGES], (k / L::STAGES) & 1, p.wait_immediate, failed);
                float2 z[2 * kR], t[2 * kR], Y[2 * kR], av[2 * kR], em[2 * kR];
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const F4 a = in(k, 1, ea, r);
                    z[2 * r] = a.lo;
                    z[2 * r + 1] = a.hi;
                }
                decays<2 * kR, 2>(C, z, bias2, rate, t, Y, av, em);
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const float2 s0 = mul2(rate[0], sigmoid_from_t(C, z[2 * r], t[2 * r]));
                    const float2 s1 = mul2(rate[1], sigmoid_from_t(C, z[2 * r + 1], t[2 * r + 1]));
                    stash[(3 * r) * kSlot] = to4({em[2 * r], em[2 * r + 1]});
                    stash[(3 * r + 1) * kSlot] = to4({Y[2 * r], Y[2 * r + 1]});
                    stash[(3 * r + 2) * kSlot] = to4({s0, s1});
                    al[r] = {av[2 * r], av[2 * r + 1]};
                    v[r] = in(k, 3, ey, r);
                }
                fetch_xb(k);
                fetch_ay(k + 1);
                if (t0 < d.T) {
                    if (PACKED) seq.down_to(p, t0);
                    if (seq.b0 == t0 || seq.b1 <= t0 + kR) {   // a sequence starts or ends here
                        Seq m = seq;
#pragma unroll
                        for (int r = 0; r < kR; ++r) {
                            m.up_to(p, t0 + r);
                            if (t0 + r < d.T && m.b0 == t0 + r) {
                                starts |= 1u << r;
                                al[r] = f4(-0.f);
                            }
                            if (m.b1 == t0 + r + 1 && p.grad_final)
                                v[r] = add4(v[r], load_words<kStep>(p.grad_final + (int64_t)m.n * d.D + ch, nc));
                        }
                    }
                }
#pragma unroll
                for (int r = kR - 1; r >= 0; --r) {
                    c = mul4(al[r], add4(v[r], c));
                    Q = compose<PACKED>(al[r], Q);
                    if (PACKED) c = {cut2(al[r].lo, splat2(0.f), c.lo), cut2(al[r].hi, splat2(0.f), c.hi)};
                }
            }
            chain.hand_in(Q, c, eA, eB, k, warp, lane);
        };
        auto finish = [&](int k, F4 (&al)[kR], F4 (&v)[kR], uint32_t starts, const F4 &eA, const F4 &eB) {
            const int tile = tile_of(k), t0 = tile * L::TT + tg;
            const bool any = tile >= 0 && t0 < d.T;
            F4 hs = f4(0.f);
            if (any)
                hs = load_row<float, TMA, kStep>(p.cs + ((int64_t)row * ((d.T + kR - 1) / kR) + t0 / kR) * d.D + ch, nc);
            F4 c = chain.take(eA, eB, k, warp, lane);
            if (any) {
#pragma unroll
                for (int r = kR - 1; r >= 0; --r) {   // v becomes delta; behind the row's end both are 0
                    v[r] = add4(v[r], c);
                    c = mul4(al[r], v[r]);
                    if (PACKED) c = {cut2(al[r].lo, splat2(0.f), c.lo), cut2(al[r].hi, splat2(0.f), c.hi)};
                }
                F4 tA = f4(0.f), tb = f4(0.f);
                const int64_t o = ((int64_t)row * d.T + t0) * d.D + ch;
                T *dx = (T *)p.dx + o, *da = (T *)p.da + o, *db = (T *)p.db + o;
                const bool whole = nc == 4 && t0 + kR <= d.T;
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    const F4 x = in(k, 0, ex, r), b = in(k, 2, eb, r);
                    const F4 em = f4(stash[(3 * r) * kSlot]), Y = f4(stash[(3 * r + 1) * kSlot]), rsg = f4(stash[(3 * r + 2) * kSlot]);
                    if (starts >> r & 1) {   // the decay itself again, the state before, and the state's gradient
                        al[r] = {decay_of(em.lo, Y.lo), decay_of(em.hi, Y.hi)};
                        Seq m = seq;
                        m.up_to(p, t0 + r);
                        hs = p.h0 ? load_words<kStep>(p.h0 + (int64_t)m.n * d.D + ch, nc) : f4(0.f);
                        if (p.dh0) store_words<kStep>(p.dh0 + (int64_t)m.n * d.D + ch, mul4(al[r], v[r]), nc);
                    }
                    F4 gx, ga, gb;
                    auto pair = [&](float2 em, float2 Y, float2 rsg, float2 al, float2 xv, float2 bv, float2 dv, float2 &hh,
                                    float2 &qA, float2 &qb, float2 &ox, float2 &oa, float2 &ob) {
                        const float2 w = fma2(em, al, em), rs = inv_sqrt2(w), be = sigmoid2(C, bv);
                        const float2 bx = mul2(be, xv), s = mul2(w, rs), sbx = mul2(s, bx);
                        ox = mul2(mul2(dv, s), be);
                        ob = mul2(mul2(dv, sbx), one_minus(C, be));
                        // dg = delta (alpha h_{t-1} - beta x alpha^2 / s). Where w counts as 0, so do rate
                        // sigmoid(z) and Y, below 2^-126, and 1/s is kept below 2^63: the product vanishes
                        const float2 m1 = mul2(al, hh), m2 = mul2(mul2(mul2(al, al), rs), bx);
                        const float2 ndg = mul2(dv, fma2(m1, C.neg, m2));   // -dg
                        oa = mul2(ndg, rsg);
                        qA = fma2(ndg, Y, qA);                              // dg g log2(e)
                        qb = add2(qb, oa);
                        hh = add2(m1, sbx);
                    };
                    pair(em.lo, Y.lo, rsg.lo, al[r].lo, x.lo, b.lo, v[r].lo, hs.lo, tA.lo, tb.lo, gx.lo, ga.lo, gb.lo);
                    pair(em.hi, Y.hi, rsg.hi, al[r].hi, x.hi, b.hi, v[r].hi, hs.hi, tA.hi, tb.hi, gx.hi, ga.hi, gb.hi);
                    if (TMA && whole) {
                        pack4<T>(dx, gx);
                        pack4<T>(da, ga);
                        pack4<T>(db, gb);
                    } else if (t0 + r < d.T) {
                        store_row<T, TMA, kStep>(dx, gx, nc);
                        store_row<T, TMA, kStep>(da, ga, nc);
                        store_row<T, TMA, kStep>(db, gb, nc);
                    }
                    dx += d.D;
                    da += d.D;
                    db += d.D;
                }
                sA[0] = add4(sA[0], tA);
                sb[0] = add4(sb[0], tb);
            }
            if ((k & 15) == 15) {
                sA[1] = add4(sA[1], sA[0]);
                sb[1] = add4(sb[1], sb[0]);
                sA[0] = sb[0] = f4(0.f);
            }
        };
        F4 al[kR], v[kR], eA, eB;
        uint32_t starts;
        for (int k = 0; k < steps; ++k) {
            begin(k, al, v, starts, eA, eB);
            finish(k, al, v, starts, eA, eB);
        }
        // this CTA's sums: over the token groups, in order
        const int gi = warp * L::G + g;
        *(float4 *)&red[gi][0][q * 4] = to4(mul4(add4(sA[1], sA[0]), f4(kLn2)));
        *(float4 *)&red[gi][1][q * 4] = to4(add4(sb[1], sb[0]));
    }
    __syncthreads();
    for (int i = tid; i < 2 * L::CH; i += L::THREADS) {
        const int which = i / L::CH, v = i % L::CH, c = slab * L::CH + Columns<L, TMA>::of(v);
        if (c >= d.D) continue;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < L::NG; ++j) s += red[j][which][v];
        p.part[(((int64_t)row * cs + rank) * 2 + which) * d.D + c] = s;
    }
    if (failed) *p.status = GDN_ERR_DEVICE_TIMEOUT;
    chain.leave(rank, cs);
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
    const F4 bias = load_row<float, VEC>(p.dt_bias + ch, nc), l = load_row<float, VEC>(p.A_log + ch, nc);
    const float2 rate[2] = {make_float2(expf(l.lo.x), expf(l.lo.y)), make_float2(expf(l.hi.x), expf(l.hi.y))};
    const float2 bias2[2] = {mul2(bias.lo, splat2(kLog2e)), mul2(bias.hi, splat2(kLog2e))};
    const GateConst C(false);
    float2 z[2] = {a.lo, a.hi}, t[2], Y[2], al[2], em[2];
    decays<2, 2>(C, z, bias2, rate, t, Y, al, em);
    const F4 h = fma4({al[0], al[1]}, h0, mul4({write_scale2(C, em[0], al[0], b.lo), write_scale2(C, em[1], al[1], b.hi)}, x));
    store_row<float, VEC>(state + n * d.D + ch, h, nc);
    store_row<T, VEC>((T *)p.out + n * d.D + ch, h, nc);
}

// ===================================================================== host
// CTAs per chain: as many as leave all clusters resident, since a cluster that waits for another's end costs its whole
// time again (a cluster stays within one of the chip's processing clusters, so larger ones fit worse than their sum of
// CTAs says: the counts here are the occupancy calculator's answers for this chip). At two CTAs per SM up to 16, at
// three, where registers allow that, up to 8: with more than two, larger clusters wait for the slowest SM. Backward over
// 16384 bf16 tokens:
//     24 chains  10 CTAs 157 us, 8 172, 12 225      72 chains  6 CTAs 296 us, 5 323, 7 413
//     36 chains   8 CTAs 201 us, 7 220, 10 277      84 chains  5 CTAs 342 us, 4 383, 6 454
//     50 chains   8 CTAs 218 us, 7 237,  9 319     100 chains  4 CTAs 403 us, 3 495, 5 538
//     56 chains   7 CTAs 248 us, 6 270,  8 344     128 chains  3 CTAs 521 us, 2 631, 4 645
// (the forward's order is the same).
int cluster_size(int64_t chains, int64_t ntiles, int per_sm) {
    constexpr int kResident2[kMaxCluster] = {304, 152, 97, 74, 58, 46, 38, 36, 30, 28, 23, 23, 19, 14, 14, 14};
    constexpr int kResident3[8] = {456, 228, 148, 110, 87, 74, 59, 51};
    int cs = 1;
    for (int i = 1; i <= kMaxCluster; ++i)
        if (kResident2[i - 1] >= chains || (per_sm > 2 && i <= 8 && kResident3[i - 1] >= chains)) cs = i;
    return (int)std::max<int64_t>(1, std::min<int64_t>(cs, ntiles));
}

struct RecPlan {
    int slabs, ntiles, cs;
    int64_t chains;
};
template <typename L> RecPlan make_plan(const gdn_recurrence_desc &d, int per_sm) {
    RecPlan r;
    r.slabs = (int)cdiv64(d.D, L::CH);
    r.ntiles = (int)cdiv64(d.T, L::TT);
    r.chains = (int64_t)d.B * r.slabs;
    r.cs = cluster_size(r.chains, r.ntiles, per_sm);
    return r;
}

// Shared memory that the maps of a chain's CTAs take, by step parity
template <typename L> constexpr size_t exchange_bytes(int cs) { return 2 * (size_t)cs * 2 * L::CH * sizeof(float); }

// fixed: bytes of shared memory beside the exchanged maps
template <typename L, typename K>
cudaError_t launch_chains(K kernel, const RecPlan &pl, size_t fixed, cudaStream_t s, const RecProblem &p, const RecMaps &m) {
    cudaError_t e = allow_shared(kernel, fixed + exchange_bytes<L>(kMaxCluster));
    if (e == cudaSuccess && pl.cs > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pl.chains * pl.cs));
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = fixed + exchange_bytes<L>(pl.cs);
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
template <typename L>
bool tma_map(CUtensorMap *m, const gdn_recurrence_desc &d, const void *p, int64_t sb, int64_t st) {
    const uint64_t es = act_size(d.dtype);
    const uint64_t pt = (uint64_t)st * es, pb = d.B == 1 ? (uint64_t)d.T * pt : (uint64_t)sb * es;
    return encode_token_map(m, d.dtype, p, d.B, d.T, d.D, pb, pt, L::TT, L::CH);
}

template <typename T>
cudaError_t launch_forward(RecProblem p, cudaStream_t s) {
    using L = FwdTile<T>;
    const gdn_recurrence_desc &d = p.d;
    RecMaps m;
    memset(&m, 0, sizeof(m));
    const bool tma = d.T > 0 && (d.D * sizeof(T)) % 16 == 0 && ptr_aligned(p.out, 16) && ptr_aligned(p.cs, 16) &&
                     tma_ok(d, p.x, d.x_stride_b, d.x_stride_t) && tma_ok(d, p.a, d.a_stride_b, d.a_stride_t) &&
                     tma_ok(d, p.b, d.b_stride_b, d.b_stride_t);
    const RecPlan pl = make_plan<L>(d, sizeof(T) == 2 && tma ? 3 : 2);
    p.slabs = pl.slabs;
    p.ntiles = pl.ntiles;
    if (tma && (!tma_map<L>(&m.x, d, p.x, d.x_stride_b, d.x_stride_t) || !tma_map<L>(&m.a, d, p.a, d.a_stride_b, d.a_stride_t) ||
                !tma_map<L>(&m.b, d, p.b, d.b_stride_b, d.b_stride_t)))
        return cudaErrorInvalidValue;
    auto kernel = p.cu ? (tma ? rec_forward_kernel<T, true, true> : rec_forward_kernel<T, false, true>)
                       : (tma ? rec_forward_kernel<T, true, false> : rec_forward_kernel<T, false, false>);
    return launch_chains<L>(kernel, pl, tma ? L::STAGES * 3 * L::kTensor : 0, s, p, m);
}

template <typename T>
cudaError_t launch_backward_rec(RecProblem p, cudaStream_t s) {
    using L = BwdTile<T>;
    const gdn_recurrence_desc &d = p.d;
    RecMaps m;
    memset(&m, 0, sizeof(m));
    const bool tma = d.T > 0 && (d.D * sizeof(T)) % 16 == 0 && ptr_aligned(p.dx, 16) && ptr_aligned(p.da, 16) &&
                     ptr_aligned(p.db, 16) && ptr_aligned(p.grad_out, 16) && ptr_aligned(p.cs, 16) && tma_ok(d, p.x, d.x_stride_b, d.x_stride_t) &&
                     tma_ok(d, p.a, d.a_stride_b, d.a_stride_t) && tma_ok(d, p.b, d.b_stride_b, d.b_stride_t);
    const RecPlan pl = make_plan<L>(d, sizeof(T) == 2 && tma ? 3 : 2);
    p.slabs = pl.slabs;
    p.ntiles = pl.ntiles;
    if (tma && (!tma_map<L>(&m.x, d, p.x, d.x_stride_b, d.x_stride_t) || !tma_map<L>(&m.a, d, p.a, d.a_stride_b, d.a_stride_t) ||
                !tma_map<L>(&m.b, d, p.b, d.b_stride_b, d.b_stride_t) || !tma_map<L>(&m.dy, d, p.grad_out, (int64_t)d.T * d.D, d.D)))
        return cudaErrorInvalidValue;
    auto kernel = p.cu ? (tma ? rec_backward_kernel<T, true, true> : rec_backward_kernel<T, false, true>)
                       : (tma ? rec_backward_kernel<T, true, false> : rec_backward_kernel<T, false, false>);
    const cudaError_t e = launch_chains<L>(kernel, pl, (tma ? L::STAGES * 4 * L::kTensor : 0) + kBwdStash<T>, s, p, m);
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
    if (d->T > 0x7fff0000 || d->D > (1 << 30)) return GDN_ERR_UNSUPPORTED;   // tokens and channels of a tile in 32 bits
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
    // at three CTAs per SM a chain has no fewer of them than at two
    const int cs = d.dtype == GDN_F32 ? make_plan<BwdTile<float>>(d, 3).cs : make_plan<BwdTile<__half>>(d, 3).cs;
    L.part = off;   off = align_up(off + (size_t)d.B * cs * 2 * d.D * 4, 256);
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
    return by_dtype(d->dtype, [&](auto t) {
        return layer_status(launch_forward<decltype(t)>(p, (cudaStream_t)stream));
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
    return by_dtype(d->dtype, [&](auto t) {
        using T = decltype(t);
        cudaError_t e = cudaSuccess;
        p.recomputed = !chunk_states && d->T > 0;
        if (p.recomputed) e = launch_forward<T>(p, s);   // chunk states only
        return layer_status(e != cudaSuccess ? e : launch_backward_rec<T>(p, s));
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
