// gdn_group_norm.cu -- group norm with an activation, channels last (include/gdn.h):
// forward and backward. Bound by HBM.
//
// A warp works on a fixed set of adjacent channels: 32 / LG groups of LG lanes each
// (LG, a power of two, covers a group's vectors), or a 32-lane slab of a larger group
// (in the rows form a block takes a larger group).
// Weights stay in registers, sums cross lanes by shuffles, and rows stream past.
//
//   rows     L = 1 and a group fits LG lanes x NV vectors, or a block's: a row is read once,
//            its mean and its centred squares are summed from registers, and it is written.
//            Two rows are worked on per warp and two are on their way; the backward's come
//            through shared memory, six ahead.
//   general  several positions, or larger groups: partial means and centred sums of
//            squares per (instance, chunk of positions), merged pairwise; a second pass
//            normalises (one kernel where a warp holds a whole group, else two). The
//            second read comes from L2 where the tensor fits.
//
// The backward has the same two forms, with the sums of t and t xh in the statistics'
// place. Parameter gradients are summed per warp over its rows, written as partial rows
// and added up by a last small kernel. Every order is fixed by the sizes and
// by whether vectors fit.
//
// Measured, of the copy rate: rows of 4096 in 32 groups, bf16, 131072 forward 380 us (83 %),
// 65536 fp16 forward 195 us (81 %) and backward 349 us (68 %: 110 registers, two blocks per SM,
// issue slots 58 % used); in one group, 131072 forward, 523 us (60 %: two block-wide sums a
// row). Over positions: 60 x 16384 x 512 in 8 groups, forward, 472 us (63 %; 94 % counting the
// second read); 2 x 2048 x 1536 in 6 groups 10 us and 17 us backward on the device, launches and
// latency. Groups that are no multiple of 16 bytes go element by element: 100000 rows of 4160 in
// 64 groups 1070 us (23 %), issue-bound.
#include <string.h>

#include <algorithm>

#include "gdn_layer_ops.cuh"

namespace gdn {
namespace {

struct NormProblem {
    gdn_group_norm_desc d;
    const void *x, *w, *b, *dy;
    void *out, *dx;
    float *mean, *rstd, *dw, *db;
    float2 *stat;      // general: [item][part] partial (mean, centred sum of squares), or (sum t, sum t xh)
    float *part;       // [part_rows][2][C] partial sums of dweight, dbias
    int lg;            // lanes per group or slab; kThreads: a block per group
    int sets;          // sets of channels, one per warp
    int slabs;         // slabs per group (1 where a warp holds whole groups)
    int slices;        // warps that share a set
    int by_block;      // general backward: the warps of a block share a set, and write one partial row
    int part_rows;
    int chunks, chunk_rows;   // general: chunks of positions per instance
    int64_t items;     // rows, or (instance, chunk) pairs
};

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Blocks per SM, resident at once: rows forward, general forward and backward. Three for the last is
// slower (2 x 2048 x 1536 in 6 groups 21.1 against 17.1 us on the device, 60 x 2000 x 2048 in 16 542 against 464 us):
// registers hold two.
constexpr int kBlocksForward = 3, kBlocksGeneral = 4, kBlocksSums = 2;
// The rows backward: three where their registers fit (vectors of four fp32, or no activation's derivative: 65536 x 4096
// in 32 groups fp32 526 against 625 us with two, in 64 without activation bf16 301 against 323), else two (in 32 with
// SiLU fp16 346 against 454 us with three, spilling).
constexpr int blocks_backward(bool vectors, bool fp32, int act) { return vectors && (fp32 || act == GDN_ACT_NONE) ? 3 : 2; }
constexpr int kRowsForward = 2;   // rows a warp works on at a time (two reductions in flight); as many are on their way
constexpr int kAheadBackward = 6; // rows on their way in the backward
constexpr int kBatch = 8, kBatchBackward = 4;   // rows in flight per warp in the general form

template <typename T> struct VecN { static constexpr int value = 16 / sizeof(T); };

// V elements of T as they stand in memory (V = 1, or 16 bytes), and as pairs of fp32 values: sm_100-class
// SMs run add, multiply and fma on a pair as one instruction. V = 1 fills the first half of one pair.
template <typename T, int V> struct RawV { using type = uint4; };
template <typename T> struct RawV<T, 1> { using type = T; };
template <int V> constexpr int kPairs = V > 1 ? V / 2 : 1;
template <typename T, int V>
__device__ __forceinline__ typename RawV<T, V>::type load_raw(const T *p) {
    return *reinterpret_cast<const typename RawV<T, V>::type *>(p);
}
template <typename T, int V>
__device__ __forceinline__ void unpack_v(const typename RawV<T, V>::type &r, float2 *v) {
    if constexpr (V == 1) v[0] = make_float2(to_f<T>(r), 0.f);
    else Pairs<T>::unpack(r, v);
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T *p, const float2 *v) {
    if constexpr (V == 1) *p = from_f<T>(v[0].x);
    else *reinterpret_cast<uint4 *>(p) = Pairs<T>::pack(v);
}
// the sum over a pair's elements that exist
template <int V> __device__ __forceinline__ float total(float2 v) { return V == 1 ? v.x : v.x + v.y; }

__device__ __forceinline__ float lane_sum(float v, int lg) {   // over lg adjacent lanes, the same in all of them
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        if (off < lg) v += o;
    }
    return v;
}

__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float2 sigmoid2(float2 z) {
    const float2 m = mul2(z, splat2(-1.4426950408889634f));
    const float2 c = add2(make_float2(ex2_approx(m.x), ex2_approx(m.y)), splat2(1.f));
    return make_float2(rcp_approx(c.x), rcp_approx(c.y));
}
template <int ACT> __device__ __forceinline__ float2 act2(float2 z) { return ACT == GDN_ACT_SILU ? silu2_acc(z) : z; }
template <int ACT> __device__ __forceinline__ float2 act_grad2(float2 z) {   // d act(z) / dz
    if (ACT == GDN_ACT_NONE) return splat2(1.f);
    const float2 s = sigmoid2(z);
    return mul2(s, fma2(z, fma2(s, splat2(-1.f), splat2(1.f)), splat2(1.f)));
}

// The same with the number of lanes known (LG), in lg (LG = 0), or over the block (LG = kThreads: all threads call it)
template <int LG> __device__ __forceinline__ float lane_sum_t(float v, int lg) {
    if (LG == 0) return lane_sum(v, lg);
    if constexpr (LG == kThreads) {
        __shared__ float part[kWarps];
        v = lane_sum_t<32>(v, lg);
        float t = 0.f;
        __syncthreads();   // the sum before has been read
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps; ++i) t += part[i];
        return t;
    }
#pragma unroll
    for (int off = LG / 2; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The warp's place: its set, its lane's first channel, and whether the lane has channels.
struct Place {
    int set, slice, sub;   // sub: lane within the group's lanes
    int g;                 // group
    int c;                 // the lane's first channel
    bool any;
};
template <int V>
__device__ __forceinline__ Place place(const NormProblem &p) {
    const int w = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    const int cg = p.d.C / p.d.G;
    Place q;
    if (p.lg == kThreads) {   // a block per group
        q.g = q.set = blockIdx.x % p.sets;
        q.slice = blockIdx.x / p.sets;
        q.sub = threadIdx.x;
        q.any = q.slice < p.slices && q.sub * V < cg;
        q.c = q.g * cg + q.sub * V;
        return q;
    }
    q.set = w % p.sets;
    q.slice = w / p.sets;
    if (p.by_block) {
        q.set = blockIdx.x % p.sets;
        q.slice = blockIdx.x / p.sets * kWarps + threadIdx.x / 32;
    }
    q.sub = lane % p.lg;
    int in;                // the lane's first element within the group
    if (p.slabs == 1) {
        q.g = q.set * (32 / p.lg) + lane / p.lg;
        in = q.sub * V;
    } else {
        q.g = q.set / p.slabs;
        in = (q.set % p.slabs * 32 + lane) * V;
    }
    q.any = (p.by_block || q.slice < p.slices) && q.g < p.d.G && in < cg;
    if (q.g >= p.d.G) q.g = p.d.G - 1;
    q.c = q.g * cg + in;
    return q;
}

// One of weight and bias for the lane's V channels from c on; the loads are independent of one another.
template <typename W, int V>
__device__ __forceinline__ void load_param(const void *p, bool any, int c, float none, float2 *v) {
    const W *at = (const W *)p + c;
#pragma unroll
    for (int e = 0; e < kPairs<V>; ++e) {
        v[e] = splat2(any ? none : 0.f);
        if (any && p) {
            v[e].x = to_f<W>(at[2 * e]);
            if (V > 1) v[e].y = to_f<W>(at[2 * e + 1]);
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ void load_params(const NormProblem &p, bool any, int c, float2 *w, float2 *b) {
    if (sizeof(T) == 4 || p.d.weight_dtype == GDN_F32) {
        load_param<float, V>(p.w, any, c, 1.f, w);
        load_param<float, V>(p.b, any, c, 0.f, b);
    } else {
        load_param<T, V>(p.w, any, c, 1.f, w);
        load_param<T, V>(p.b, any, c, 0.f, b);
    }
    // as fp32 values from here on: the compiler would keep the 16-bit ones and convert them for every row
#pragma unroll
    for (int e = 0; e < kPairs<V>; ++e)
        asm volatile("" : "+f"(w[e].x), "+f"(w[e].y), "+f"(b[e].x), "+f"(b[e].y));
}

// A warp's rows on their way into shared memory: DEPTH rows of NT tensors, 16 bytes per lane and vector. A lane
// reads only what it copied itself, so its own wait is enough.
template <int NT, int NV, int DEPTH> struct RowRing {
    uint4 *base;   // the lane's first slot
    __device__ __forceinline__ RowRing(uint4 *smem) {
        base = smem + (threadIdx.x / 32) * (DEPTH * NT * NV * 32) + threadIdx.x % 32;
    }
    __device__ __forceinline__ uint4 *slot(int j, int t, int i) const { return base + ((j * NT + t) * NV + i) * 32; }
    __device__ __forceinline__ void copy(int j, int t, int i, const void *src) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                     :: "r"((uint32_t)__cvta_generic_to_shared(slot(j, t, i))), "l"(src) : "memory");
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait_oldest() { asm volatile("cp.async.wait_group %0;" :: "n"(DEPTH - 1) : "memory"); }
};
template <int NT, int NV, int DEPTH> constexpr size_t kRingBytes = (size_t)kWarps * DEPTH * NT * NV * 512;

// ------------------------------------------------------------------ rows
template <typename T, int V, int NV, int ACT, int LG>
__global__ void __launch_bounds__(kThreads, NV == 1 ? kBlocksForward : 1) norm_rows_forward(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (q.slice >= p.slices) return;
    constexpr int NP = kPairs<V>;
    constexpr int kR = NV == 1 ? kRowsForward : 1;
    const int cg = d.C / d.G;
    const float inv = 1.f / (float)cg;
    bool has[NV];
    float2 w[NV][NP], b[NV][NP];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        has[i] = q.any && (q.sub + i * p.lg) * V < cg;
        load_params<T, V>(p, has[i], q.c + i * p.lg * V, w[i], b[i]);
    }
    // the next rows are on their way while these are worked on
    typename RawV<T, V>::type raw[kR][NV] = {};
    auto fetch = [&](int64_t n0) {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int64_t n = n0 + (int64_t)r * p.slices;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (n < p.items && has[i]) raw[r][i] = load_raw<T, V>((const T *)p.x + n * d.x_stride_n + q.c + i * p.lg * V);
        }
    };
    fetch(q.slice);
    for (int64_t n0 = q.slice; n0 < p.items; n0 += (int64_t)kR * p.slices) {
        float2 x[kR][NV][NP];
        float mean[kR], rstd[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float2 s = splat2(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                unpack_v<T, V>(raw[r][i], x[r][i]);
#pragma unroll
                for (int e = 0; e < NP; ++e) s = add2(s, x[r][i][e]);   // a lane without channels holds zeros
            }
            mean[r] = total<V>(s);
        }
        fetch(n0 + (int64_t)kR * p.slices);
#pragma unroll
        for (int r = 0; r < kR; ++r) mean[r] = lane_sum_t<LG>(mean[r], p.lg) * inv;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float2 s = splat2(0.f);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    x[r][i][e] = add2(x[r][i][e], splat2(-mean[r]));
                    s = fma2(x[r][i][e], x[r][i][e], s);
                }
                if (has[i]) t += total<V>(s);
            }
            rstd[r] = rsqrtf(fmaf(lane_sum_t<LG>(t, p.lg), inv, d.eps));
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            const int64_t n = n0 + (int64_t)r * p.slices;
            if (n >= p.items || !q.any) continue;
            if (q.sub == 0) {
                if (p.mean) p.mean[n * d.G + q.g] = mean[r];
                if (p.rstd) p.rstd[n * d.G + q.g] = rstd[r];
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has[i]) continue;
#pragma unroll
                for (int e = 0; e < NP; ++e) x[r][i][e] = act2<ACT>(fma2(mul2(x[r][i][e], splat2(rstd[r])), w[i][e], b[i][e]));
                store_v<T, V>((T *)p.out + n * d.C + q.c + i * p.lg * V, x[r][i]);
            }
        }
    }
}

// The backward's part of an element: xh, dz = dout act'(z), t = dz w.
struct Grad2 {
    float2 xh, dz, t;
};
template <int ACT>
__device__ __forceinline__ Grad2 grad_of(float2 x, float2 dy, float mean, float rstd, float2 w, float2 b) {
    Grad2 g;
    g.xh = mul2(add2(x, splat2(-mean)), splat2(rstd));
    g.dz = mul2(dy, act_grad2<ACT>(fma2(g.xh, w, b)));
    g.t = mul2(g.dz, w);
    return g;
}

// Sums of dweight and dbias of a warp's channels: over 16 rows, over all (the second level keeps the
// rounding of long sums down), then into its partial row.
template <int N> struct ParamSums {
    float2 w[2][N], b[2][N];
    int rows;
    __device__ __forceinline__ ParamSums() {
#pragma unroll
        for (int i = 0; i < N; ++i) w[0][i] = w[1][i] = b[0][i] = b[1][i] = splat2(0.f);
        rows = 0;
    }
    __device__ __forceinline__ void row_done() {
        if (++rows & 15) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            w[1][i] = add2(w[1][i], w[0][i]);
            b[1][i] = add2(b[1][i], b[0][i]);
            w[0][i] = b[0][i] = splat2(0.f);
        }
    }
    template <int V> __device__ __forceinline__ void write(const NormProblem &p, int slice, int c, int i) const {
        float *pw = p.part + (int64_t)slice * 2 * p.d.C + c, *pb = pw + p.d.C;
#pragma unroll
        for (int e = 0; e < kPairs<V>; ++e) {
            const float2 sw = add2(w[1][i + e], w[0][i + e]), sb = add2(b[1][i + e], b[0][i + e]);
            pw[2 * e] = sw.x;
            pb[2 * e] = sb.x;
            if (V > 1) {
                pw[2 * e + 1] = sw.y;
                pb[2 * e + 1] = sb.y;
            }
        }
    }
};

template <typename T, int V, int NV, int ACT, int LG>
__global__ void __launch_bounds__(kThreads, NV == 1 || V == 1 ? blocks_backward(V > 1, sizeof(T) == 4, ACT) : 1) norm_rows_backward(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    pdl_trigger();
    if (q.slice >= p.slices) return;
    constexpr int NP = kPairs<V>;
    const int cg = d.C / d.G;
    const float inv = 1.f / (float)cg;
    bool has[NV];
    float2 w[NV][NP], b[NV][NP];
    ParamSums<NV * NP> sums;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        has[i] = q.any && (q.sub + i * p.lg) * V < cg;
        load_params<T, V>(p, has[i], q.c + i * p.lg * V, w[i], b[i]);
    }
    constexpr int kSteps = V > 1 ? kAheadBackward / NV : 1;
    extern __shared__ uint4 ring_smem[];
    const RowRing<2, NV, kSteps> ring(ring_smem);
    T single[2][NV] = {};   // element by element: the next row's
    auto fetch = [&](int j, int64_t n) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (n < p.items && has[i]) {
                const T *x = (const T *)p.x + n * d.x_stride_n + q.c + i * p.lg * V, *y = (const T *)p.dy + n * d.C + q.c + i * p.lg * V;
                if (V > 1) {
                    ring.copy(j, 0, i, x);
                    ring.copy(j, 1, i, y);
                } else {
                    single[0][i] = *x;
                    single[1][i] = *y;
                }
            }
        if (V > 1) ring.commit();
    };
    // (mean, rstd) of this row and the next two
    auto stats = [&](int64_t n) {
        return n < p.items ? make_float2(p.mean[n * d.G + q.g], p.rstd[n * d.G + q.g]) : make_float2(0.f, 0.f);
    };
#pragma unroll
    for (int j = 0; j < kSteps; ++j) fetch(j, q.slice + (int64_t)j * p.slices);
    float2 st0 = stats(q.slice), st1 = stats(q.slice + (int64_t)p.slices);
    int j = 0;
    for (int64_t n = q.slice; n < p.items; n += p.slices) {
        const float2 st2 = stats(n + 2 * (int64_t)p.slices);
        const float mean = st0.x, rstd = st0.y;
        st0 = st1;
        st1 = st2;
        if (V > 1) ring.wait_oldest();
        float2 x[NV][NP], y[NV][NP], s1 = splat2(0.f), s2 = splat2(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!has[i]) continue;   // no part in any sum
            if constexpr (V > 1) {
                unpack_v<T, V>(*ring.slot(j, 0, i), x[i]);
                unpack_v<T, V>(*ring.slot(j, 1, i), y[i]);
            } else {
                unpack_v<T, V>(single[0][i], x[i]);
                unpack_v<T, V>(single[1][i], y[i]);
            }
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                const Grad2 g = grad_of<ACT>(x[i][e], y[i][e], mean, rstd, w[i][e], b[i][e]);
                x[i][e] = g.xh;
                y[i][e] = g.t;
                sums.w[0][i * NP + e] = fma2(g.dz, g.xh, sums.w[0][i * NP + e]);
                sums.b[0][i * NP + e] = add2(sums.b[0][i * NP + e], g.dz);
                s1 = add2(s1, g.t);
                s2 = fma2(g.t, g.xh, s2);
            }
        }
        if (V == 1) fetch(0, n + p.slices);
        sums.row_done();
        const float m1 = lane_sum_t<LG>(total<V>(s1), p.lg) * inv, m2 = lane_sum_t<LG>(total<V>(s2), p.lg) * inv;
        if (V > 1) {   // this row's slots have been read
            fetch(j, n + (int64_t)kSteps * p.slices);
            j = j + 1 < kSteps ? j + 1 : 0;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!has[i]) continue;
#pragma unroll
            for (int e = 0; e < NP; ++e)
                y[i][e] = mul2(fma2(x[i][e], splat2(-m2), add2(y[i][e], splat2(-m1))), splat2(rstd));
            store_v<T, V>((T *)p.dx + n * d.C + q.c + i * p.lg * V, y[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (has[i]) sums.template write<V>(p, q.slice, q.c + i * p.lg * V, i * NP);
}

// --------------------------------------------------------------- general
// Mean and centred sum of squares of n elements, and their union.
struct Stat {
    float n, mean, m2;
};
__device__ __forceinline__ Stat merge(const Stat &a, const Stat &b) {   // b.n > 0
    Stat r;
    r.n = a.n + b.n;
    const float dl = b.mean - a.mean, f = __fdividef(b.n, r.n);
    r.mean = fmaf(dl, f, a.mean);
    r.m2 = a.m2 + b.m2 + dl * dl * a.n * f;
    return r;
}
// The union over lg adjacent lanes: the mean of the means, then the squares about it.
__device__ __forceinline__ Stat lane_union(const Stat &s, int lg) {
    Stat r;
    r.n = lane_sum(s.n, lg);
    r.mean = lane_sum(s.n * s.mean, lg) / r.n;
    const float dl = s.mean - r.mean;
    r.m2 = lane_sum(s.n > 0.f ? fmaf(s.n * dl, dl, s.m2) : 0.f, lg);
    return r;
}

// (instance, positions) of an item
__device__ __forceinline__ void item_rows(const NormProblem &p, int64_t item, int64_t &n, int &l0, int &l1) {
    n = item / p.chunks;
    l0 = (int)(item - n * p.chunks) * p.chunk_rows;
    l1 = min(p.d.L, l0 + p.chunk_rows);
}
// where the partial of a set's group (or slab) of an item stands
__device__ __forceinline__ int64_t stat_at(const NormProblem &p, int64_t item, const Place &q) {
    const int64_t parts = (int64_t)p.d.G * p.slabs;
    return item * parts + (p.slabs == 1 ? q.g : q.set);
}

template <typename T, int V>
__device__ __forceinline__ Stat chunk_stat(const NormProblem &p, const Place &q, int64_t n, int l0, int l1) {
    const gdn_group_norm_desc &d = p.d;
    constexpr int NP = kPairs<V>;
    Stat s = {0.f, 0.f, 0.f};
    const T *at = (const T *)p.x + n * d.x_stride_n + q.c;
    if (q.any)
        for (int l = l0; l < l1; l += kBatch) {
            typename RawV<T, V>::type raw[kBatch] = {};
            const int rows = min(kBatch, l1 - l);
#pragma unroll
            for (int r = 0; r < kBatch; ++r)
                if (r < rows) raw[r] = load_raw<T, V>(at + (int64_t)(l + r) * d.x_stride_l);
            float2 sum = splat2(0.f), sq = splat2(0.f), v[NP];
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                unpack_v<T, V>(raw[r], v);
#pragma unroll
                for (int e = 0; e < NP; ++e) sum = add2(sum, v[e]);
            }
            const float cnt = (float)(rows * V), mean = __fdividef(total<V>(sum), cnt);
#pragma unroll
            for (int r = 0; r < kBatch; ++r) {
                if (r >= rows) break;
                unpack_v<T, V>(raw[r], v);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    v[e] = add2(v[e], splat2(-mean));
                    sq = fma2(v[e], v[e], sq);
                }
            }
            s = merge(s, {cnt, mean, total<V>(sq)});
        }
    return lane_union(s, p.lg);
}

// Rows l .. l + B - 1 (below l1) of a [.., C] tensor at the lane's channels
template <typename T, int V, int B>
__device__ __forceinline__ void fetch_rows(const T *at, int64_t stride, bool any, int l, int l1, typename RawV<T, V>::type (&raw)[B]) {
#pragma unroll
    for (int r = 0; r < B; ++r)
        if (any && l + r < l1) raw[r] = load_raw<T, V>(at + (int64_t)(l + r) * stride);
}

// raw: the first batch, fetched already
template <typename T, int V, int ACT>
__device__ __forceinline__ void normalise(const NormProblem &p, const Place &q, int64_t n, int l0, int l1, float mean, float rstd,
                                          const float2 *w, const float2 *b, typename RawV<T, V>::type (&raw)[kBatch]) {
    const gdn_group_norm_desc &d = p.d;
    if (!q.any) return;
    const T *at = (const T *)p.x + n * d.x_stride_n + q.c;
    T *to = (T *)p.out + n * d.L * d.C + q.c;
    for (int l = l0; l < l1; l += kBatch) {   // loads first: a store could change what is loaded after it
        if (l > l0) fetch_rows<T, V>(at, d.x_stride_l, true, l, l1, raw);
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            if (l + r >= l1) break;
            float2 v[kPairs<V>];
            unpack_v<T, V>(raw[r], v);
#pragma unroll
            for (int e = 0; e < kPairs<V>; ++e)
                v[e] = act2<ACT>(fma2(mul2(add2(v[e], splat2(-mean)), splat2(rstd)), w[e], b[e]));
            store_v<T, V>(to + (int64_t)(l + r) * d.C, v);
        }
    }
}

// Visits the partials of the group's chunks and slabs that fall to this lane, loads in batches: f(part, value)
template <typename F>
__device__ __forceinline__ void each_partial(const NormProblem &p, const Place &q, int64_t n, F &&f) {
    const int parts = p.chunks * p.slabs;
    for (int i0 = q.sub; i0 < parts; i0 += 8 * p.lg) {
        float2 m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * p.lg, k = p.slabs == 1 ? i : i / p.slabs;
            if (i < parts) m[j] = p.stat[((n * p.chunks + k) * p.d.G + q.g) * p.slabs + i - k * p.slabs];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i0 + j * p.lg < parts) f(i0 + j * p.lg, m[j]);
    }
}
// The whole group's statistics
template <int V>
__device__ __forceinline__ Stat group_stat(const NormProblem &p, const Place &q, int64_t n) {
    const gdn_group_norm_desc &d = p.d;
    const int cg = d.C / d.G;
    Stat s = {0.f, 0.f, 0.f};
    each_partial(p, q, n, [&](int i, float2 m) {
        const int k = p.slabs == 1 ? i : i / p.slabs, sl = i - k * p.slabs;
        const int rows = min(d.L, (k + 1) * p.chunk_rows) - k * p.chunk_rows;
        const int width = p.slabs == 1 ? cg : min(cg, (sl + 1) * 32 * V) - sl * 32 * V;
        s = merge(s, {(float)rows * (float)width, m.x, m.y});
    });
    return lane_union(s, p.lg);
}

// FUSED: one chunk and one slab, so the warp has the whole group and writes it too
template <typename T, int V, int ACT, bool FUSED>
__global__ void __launch_bounds__(kThreads) norm_stat_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    if (!FUSED) pdl_trigger();
    if (q.slice >= p.slices) return;
    float2 w[kPairs<V>], b[kPairs<V>];
    if (FUSED) load_params<T, V>(p, q.any, q.c, w, b);
    for (int64_t it = q.slice; it < p.items; it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        const Stat s = chunk_stat<T, V>(p, q, n, l0, l1);
        if (FUSED) {
            const float rstd = rsqrtf(s.m2 / s.n + d.eps);
            if (q.any && q.sub == 0) {
                if (p.mean) p.mean[n * d.G + q.g] = s.mean;
                if (p.rstd) p.rstd[n * d.G + q.g] = rstd;
            }
            typename RawV<T, V>::type raw[kBatch];
            fetch_rows<T, V>((const T *)p.x + n * d.x_stride_n + q.c, d.x_stride_l, q.any, l0, l1, raw);
            normalise<T, V, ACT>(p, q, n, l0, l1, s.mean, rstd, w, b, raw);
        } else if (q.any && q.sub == 0) {
            p.stat[stat_at(p, it, q)] = make_float2(s.mean, s.m2);
        }
    }
}

// A programmatic dependent of norm_stat_kernel
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_apply_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    float2 w[kPairs<V>], b[kPairs<V>];
    load_params<T, V>(p, q.any, q.c, w, b);
    bool waited = false;
    for (int64_t it = q.slice; it < (q.slice < p.slices ? p.items : 0); it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        typename RawV<T, V>::type raw[kBatch];
        fetch_rows<T, V>((const T *)p.x + n * d.x_stride_n + q.c, d.x_stride_l, q.any, l0, l1, raw);
        if (!waited) pdl_wait();
        waited = true;
        const Stat s = group_stat<V>(p, q, n);
        const float rstd = rsqrtf(s.m2 / s.n + d.eps);
        if (q.any && q.sub == 0 && l0 == 0 && q.c == q.g * (d.C / d.G)) {
            if (p.mean) p.mean[n * d.G + q.g] = s.mean;
            if (p.rstd) p.rstd[n * d.G + q.g] = rstd;
        }
        normalise<T, V, ACT>(p, q, n, l0, l1, s.mean, rstd, w, b, raw);
    }
    if (!waited) pdl_wait();
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_sums_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    constexpr int NP = kPairs<V>;
    pdl_trigger();
    float2 w[NP], b[NP];
    load_params<T, V>(p, q.any, q.c, w, b);
    ParamSums<NP> sums;
    for (int64_t it = q.slice; it < (q.slice < p.slices ? p.items : 0); it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        const float mean = p.mean[n * d.G + q.g], rstd = p.rstd[n * d.G + q.g];
        float2 s1 = splat2(0.f), s2 = splat2(0.f);
        if (q.any) {
            const T *at = (const T *)p.x + n * d.x_stride_n + q.c, *dy = (const T *)p.dy + n * d.L * d.C + q.c;
            for (int l = l0; l < l1; l += kBatchBackward) {
                typename RawV<T, V>::type rx[kBatchBackward], ry[kBatchBackward];
                fetch_rows<T, V>(at, d.x_stride_l, true, l, l1, rx);
                fetch_rows<T, V>(dy, d.C, true, l, l1, ry);
#pragma unroll
                for (int r = 0; r < kBatchBackward; ++r) {
                    if (l + r >= l1) break;
                    float2 x[NP], y[NP], r1 = splat2(0.f), r2 = splat2(0.f);
                    unpack_v<T, V>(rx[r], x);
                    unpack_v<T, V>(ry[r], y);
#pragma unroll
                    for (int e = 0; e < NP; ++e) {
                        const Grad2 g = grad_of<ACT>(x[e], y[e], mean, rstd, w[e], b[e]);
                        sums.w[0][e] = fma2(g.dz, g.xh, sums.w[0][e]);
                        sums.b[0][e] = add2(sums.b[0][e], g.dz);
                        r1 = add2(r1, g.t);
                        r2 = fma2(g.t, g.xh, r2);
                    }
                    s1 = add2(s1, r1);
                    s2 = add2(s2, r2);
                    sums.row_done();
                }
            }
        }
        const float t1 = lane_sum(total<V>(s1), p.lg), t2 = lane_sum(total<V>(s2), p.lg);
        if (q.any && q.sub == 0) p.stat[stat_at(p, it, q)] = make_float2(t1, t2);
    }
    if (!p.by_block) {
        if (q.any) sums.template write<V>(p, q.slice, q.c, 0);
        return;
    }
    // the block's warps hold the same channels: warp i sums pair i over them
    __shared__ float2 red[kWarps][2 * NP][32];
    static_assert(2 * NP <= kWarps, "a warp per pair");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int e = 0; e < NP; ++e) {
        red[warp][e][lane] = add2(sums.w[1][e], sums.w[0][e]);
        red[warp][NP + e][lane] = add2(sums.b[1][e], sums.b[0][e]);
    }
    __syncthreads();
    if (warp < 2 * NP && q.any) {
        float2 t = splat2(0.f);
#pragma unroll
        for (int i = 0; i < kWarps; ++i) t = add2(t, red[i][warp][lane]);
        float *to = p.part + ((int64_t)(blockIdx.x / p.sets) * 2 + warp / NP) * d.C + q.c + warp % NP * 2;
        to[0] = t.x;
        if (V > 1) to[1] = t.y;
    }
}

// A programmatic dependent of norm_sums_kernel
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_dx_kernel(const __grid_constant__ NormProblem p) {
    const gdn_group_norm_desc &d = p.d;
    const Place q = place<V>(p);
    constexpr int NP = kPairs<V>;
    const float count = (float)d.L * (float)(d.C / d.G);
    float2 w[NP], b[NP];
    load_params<T, V>(p, q.any, q.c, w, b);
    bool waited = false;
    for (int64_t it = q.slice; it < (q.slice < p.slices ? p.items : 0); it += p.slices) {
        int64_t n;
        int l0, l1;
        item_rows(p, it, n, l0, l1);
        const T *at = (const T *)p.x + n * d.x_stride_n + q.c, *dy = (const T *)p.dy + n * d.L * d.C + q.c;
        typename RawV<T, V>::type rx[kBatchBackward], ry[kBatchBackward];
        fetch_rows<T, V>(at, d.x_stride_l, q.any, l0, l1, rx);
        fetch_rows<T, V>(dy, d.C, q.any, l0, l1, ry);
        const float mean = p.mean[n * d.G + q.g], rstd = p.rstd[n * d.G + q.g];
        if (!waited) pdl_wait();
        waited = true;
        float s1 = 0.f, s2 = 0.f;
        each_partial(p, q, n, [&](int, float2 m) {
            s1 += m.x;
            s2 += m.y;
        });
        const float m1 = lane_sum(s1, p.lg) / count, m2 = lane_sum(s2, p.lg) / count;
        if (!q.any) continue;
        T *dx = (T *)p.dx + n * d.L * d.C + q.c;
        for (int l = l0; l < l1; l += kBatchBackward) {
            if (l > l0) {
                fetch_rows<T, V>(at, d.x_stride_l, true, l, l1, rx);
                fetch_rows<T, V>(dy, d.C, true, l, l1, ry);
            }
#pragma unroll
            for (int r = 0; r < kBatchBackward; ++r) {
                if (l + r >= l1) break;
                float2 x[NP], y[NP];
                unpack_v<T, V>(rx[r], x);
                unpack_v<T, V>(ry[r], y);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    const Grad2 g = grad_of<ACT>(x[e], y[e], mean, rstd, w[e], b[e]);
                    y[e] = mul2(fma2(g.xh, splat2(-m2), add2(g.t, splat2(-m1))), splat2(rstd));
                }
                store_v<T, V>(dx + (int64_t)(l + r) * d.C, y);
            }
        }
    }
    // only after the wait: its dependent relies on norm_sums_kernel, too
    if (!waited) pdl_wait();
    pdl_trigger();
}

// dweight and dbias from part[part_rows][2][C]: 32 channels a block, 32 strided partial sums each. A
// programmatic dependent of the kernel before it.
constexpr int kParamThreads = 1024;
__global__ void __launch_bounds__(kParamThreads) norm_params_kernel(const __grid_constant__ NormProblem p) {
    __shared__ float red[2][32][33];
    const int ch = threadIdx.x % 32, c = blockIdx.x * 32 + ch, s = threadIdx.x / 32;
    float v[2] = {0.f, 0.f};
    pdl_wait();
    if (c < p.d.C)
#pragma unroll 4
        for (int i = s; i < p.part_rows; i += 32) {
            v[0] += p.part[((int64_t)i * 2) * p.d.C + c];
            v[1] += p.part[((int64_t)i * 2 + 1) * p.d.C + c];
        }
    red[0][s][ch] = v[0];
    red[1][s][ch] = v[1];
    __syncthreads();
    // warp s sums channel s of the block over the 32 partial sums
    const float t0 = lane_sum(red[0][ch][s], 32), t1 = lane_sum(red[1][ch][s], 32);
    if (ch == 0 && blockIdx.x * 32 + s < p.d.C) {
        if (p.dw) p.dw[blockIdx.x * 32 + s] = t0;
        if (p.db) p.db[blockIdx.x * 32 + s] = t1;
    }
}

// ===================================================================== host
// Which form serves a problem, and its launch: a function of sizes and alignment alone. `general` also
// bounds the workspace, whatever the alignment of a later call.
struct Plan {
    bool rows, by_block;
    int v, nv, lg, sets, slabs, slices, chunks, chunk_rows;
    int64_t items;
};
int pow2_at_least(int x) {
    int r = 1;
    while (r < x) r *= 2;
    return r;
}
// vectors a lane of the rows form may hold (registers)
int most_vectors(int v, bool backward) { return backward && v > 1 ? 2 : 4; }
// v: elements per vector
Plan make_plan(const gdn_group_norm_desc &d, int v, bool backward) {
    Plan r;
    const int cg = d.C / d.G, cgv = cg / v, most = most_vectors(v, backward);
    r.v = v;
    r.lg = std::min(32, pow2_at_least(cgv));
    r.nv = pow2_at_least((int)cdiv64(cgv, r.lg));
    // rows: a warp where its lanes hold the group, else a block (two vectors or more a lane: 32 lanes)
    if (r.nv > (v > 1 ? 2 : most)) {
        r.lg = kThreads;
        r.nv = pow2_at_least((int)cdiv64(cgv, r.lg));
    }
    r.rows = d.L == 1 && r.nv <= most;
    if (!r.rows) r.lg = std::min(32, pow2_at_least(cgv));
    r.slabs = r.rows ? 1 : (int)cdiv64(cgv, r.lg);
    r.sets = r.lg == kThreads ? d.G : r.slabs == 1 ? (int)cdiv64(d.G, 32 / r.lg) : d.G * r.slabs;
    const int64_t per_sm = !r.rows    ? (backward ? kBlocksSums : kBlocksGeneral)
                           : backward ? blocks_backward(v > 1, d.dtype == GDN_F32, d.act)
                                      : kBlocksForward;
    const int64_t teams = std::max<int64_t>(1, kSms * per_sm * (r.lg == kThreads ? 1 : kWarps) / r.sets);   // that share a set
    r.chunks = 1;
    r.chunk_rows = d.L;
    if (!r.rows && d.L > 1) {
        // Chunks of positions, of at least a batch each: as many as give every team m / 64 of them, for the m that keeps
        // the busiest team's time least, counted in positions: those of its chunks, and for each chunk four more (its
        // last batch, its own partial) and the partials that a lane reads in the second pass (3 x 2176 x 176 in 22
        // groups of one lane each: 272 chunks 43.7 us, so 22.0 us).
        int64_t least = INT64_MAX;
        for (int m = 1; m <= 512; m += m < 64 ? m : 64) {
            const int64_t want = std::max<int64_t>(1, std::min<int64_t>(m * teams / (64ll * std::max(1, d.N)), d.L / kBatch));
            const int64_t rows = cdiv64(d.L, want), chunks = cdiv64(d.L, rows);
            const int64_t cost = cdiv64(d.N * chunks, teams) * (rows + 4 + chunks * r.slabs / r.lg);
            if (cost >= least) continue;
            least = cost;
            r.chunks = (int)chunks;
            r.chunk_rows = (int)rows;
        }
    }
    r.items = (int64_t)d.N * r.chunks;
    r.slices = (int)std::max<int64_t>(1, std::min<int64_t>(teams, r.items));
    // With eight slices or more, a block of one set: an eighth of the partial rows, which weigh as much as the tensors
    // where there are few sets (2 x 2048 x 1536 in 6 groups: 810 rows of 12 KB, against 12.6 MB each of x and grad_out)
    r.by_block = backward && !r.rows && r.slices >= kWarps;
    return r;
}
int part_rows(const Plan &pl) { return pl.by_block ? (int)cdiv64(pl.slices, kWarps) : pl.slices; }
int vector_of(const gdn_group_norm_desc &d) { return 16 / (int)act_size(d.dtype); }
bool vectors_fit(const gdn_group_norm_desc &d, const void *x, const void *dy, const void *out) {
    const int v = vector_of(d);
    return d.C / d.G % v == 0 && ptr_aligned(x, 16) && ptr_aligned(dy, 16) && ptr_aligned(out, 16) &&
           (d.N <= 1 || d.x_stride_n % v == 0) && (d.L <= 1 || d.x_stride_l % v == 0);
}
size_t stat_bytes(const gdn_group_norm_desc &d, const Plan &pl) {
    return pl.rows ? 0 : align_up((size_t)pl.items * d.G * pl.slabs * sizeof(float2), 256);
}
size_t part_bytes(const gdn_group_norm_desc &d, const Plan &pl) { return align_up((size_t)part_rows(pl) * 2 * d.C * 4, 256); }
// both vector widths, since a call's alignment decides
size_t workspace_need(const gdn_group_norm_desc &d, bool backward) {
    size_t most = 0;
    if ((int64_t)d.N * d.L == 0) return kStatusBytes;
    for (int v : {1, vector_of(d)}) {
        if (d.C / d.G % v) continue;
        const Plan pl = make_plan(d, v, backward);
        most = std::max(most, stat_bytes(d, pl) + (backward ? part_bytes(d, pl) : 0));
    }
    return kStatusBytes + most;
}

void apply_plan(NormProblem &p, const Plan &pl, void *ws, bool backward) {
    p.lg = pl.lg;
    p.sets = pl.sets;
    p.slabs = pl.slabs;
    p.slices = pl.slices;
    p.by_block = pl.by_block;
    p.part_rows = part_rows(pl);
    p.chunks = pl.chunks;
    p.chunk_rows = pl.chunk_rows;
    p.items = pl.items;
    char *w = (char *)ws + kStatusBytes;
    p.stat = (float2 *)w;
    if (backward) p.part = (float *)(w + stat_bytes(p.d, pl));
}
unsigned grid_of(const Plan &pl) {
    if (pl.by_block) return (unsigned)(pl.sets * part_rows(pl));
    return (unsigned)cdiv64((int64_t)pl.sets * pl.slices, pl.lg == kThreads ? 1 : kWarps);
}

template <typename T, int V, int ACT>
cudaError_t run_forward(NormProblem p, void *ws, cudaStream_t s) {
    const Plan pl = make_plan(p.d, V, false);
    apply_plan(p, pl, ws, false);
    const dim3 grid = grid_of(pl), block = kThreads;
    if (pl.rows) {
        // several vectors a lane: all 32 lanes, or the block; for one, the usual heads have an instance of their own
        auto kernel = norm_rows_forward<T, V, 1, ACT, 0>;
        if (pl.lg == kThreads)
            kernel = pl.nv == 1   ? norm_rows_forward<T, V, 1, ACT, kThreads>
                     : pl.nv == 2 ? norm_rows_forward<T, V, 2, ACT, kThreads>
                                  : norm_rows_forward<T, V, 4, ACT, kThreads>;
        else if (pl.nv == 2) kernel = norm_rows_forward<T, V, 2, ACT, 32>;
        if constexpr (V == 1)
            if (pl.lg == 32 && pl.nv == 4) kernel = norm_rows_forward<T, V, 4, ACT, 32>;
        if constexpr (V > 1) {
            if (pl.nv == 1 && pl.lg == 8) kernel = norm_rows_forward<T, V, 1, ACT, 8>;
            if (pl.nv == 1 && pl.lg == 16) kernel = norm_rows_forward<T, V, 1, ACT, 16>;
            if (pl.nv == 1 && pl.lg == 32) kernel = norm_rows_forward<T, V, 1, ACT, 32>;
        }
        return launch_kernel(false, kernel, grid, block, 0, s, p);
    }
    if (pl.chunks * pl.slabs == 1) return launch_kernel(false, norm_stat_kernel<T, V, ACT, true>, grid, block, 0, s, p);
    const cudaError_t e = launch_kernel(false, norm_stat_kernel<T, V, ACT, false>, grid, block, 0, s, p);
    return e != cudaSuccess ? e : launch_kernel(true, norm_apply_kernel<T, V, ACT>, grid, block, 0, s, p);
}

template <typename T, int V, int ACT>
cudaError_t run_backward(NormProblem p, void *ws, cudaStream_t s) {
    const Plan pl = make_plan(p.d, V, true);
    apply_plan(p, pl, ws, true);
    const dim3 grid = grid_of(pl), block = kThreads;
    cudaError_t e;
    if (pl.rows) {
        auto kernel = norm_rows_backward<T, V, 1, ACT, 0>;
        if (pl.lg == kThreads)
            kernel = pl.nv == 1 ? norm_rows_backward<T, V, 1, ACT, kThreads> : norm_rows_backward<T, V, 2, ACT, kThreads>;
        else if (pl.nv == 2) kernel = norm_rows_backward<T, V, 2, ACT, 32>;
        if constexpr (V == 1)
            if (pl.nv == 4) kernel = pl.lg == 32 ? norm_rows_backward<T, V, 4, ACT, 32> : norm_rows_backward<T, V, 4, ACT, kThreads>;
        if constexpr (V > 1) {
            if (pl.nv == 1 && pl.lg == 8) kernel = norm_rows_backward<T, V, 1, ACT, 8>;
            if (pl.nv == 1 && pl.lg == 16) kernel = norm_rows_backward<T, V, 1, ACT, 16>;
            if (pl.nv == 1 && pl.lg == 32) kernel = norm_rows_backward<T, V, 1, ACT, 32>;
        }
        const size_t ring = V > 1 ? kRingBytes<2, 1, kAheadBackward> : 0;   // NV vectors of 1 / NV as many rows
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)ring);
        if (e == cudaSuccess) e = launch_kernel(false, kernel, grid, block, ring, s, p);
    } else {
        e = launch_kernel(false, norm_sums_kernel<T, V, ACT>, grid, block, 0, s, p);
        if (e == cudaSuccess) e = launch_kernel(true, norm_dx_kernel<T, V, ACT>, grid, block, 0, s, p);
    }
    if (e != cudaSuccess || (!p.dw && !p.db)) return e;
    return launch_kernel(true, norm_params_kernel, dim3((unsigned)cdiv64(p.d.C, 32)), dim3(kParamThreads), 0, s, p);
}

template <typename T, int V>
cudaError_t run_act(const NormProblem &p, bool backward, void *ws, cudaStream_t s) {
    if (p.d.act == GDN_ACT_SILU)
        return backward ? run_backward<T, V, GDN_ACT_SILU>(p, ws, s) : run_forward<T, V, GDN_ACT_SILU>(p, ws, s);
    return backward ? run_backward<T, V, GDN_ACT_NONE>(p, ws, s) : run_forward<T, V, GDN_ACT_NONE>(p, ws, s);
}

template <typename T>
cudaError_t run(const NormProblem &p, bool backward, void *ws, cudaStream_t s) {
    constexpr int V = VecN<T>::value;
    const bool vec = vectors_fit(p.d, p.x, p.dy, backward ? p.dx : p.out);
    return vec ? run_act<T, V>(p, backward, ws, s) : run_act<T, 1>(p, backward, ws, s);
}

int run_any(const NormProblem &p, bool backward, void *ws, cudaStream_t s) {
    switch (p.d.dtype) {
    case GDN_F32: return layer_status(run<float>(p, backward, ws, s));
    case GDN_BF16: return layer_status(run<__nv_bfloat16>(p, backward, ws, s));
    default: return layer_status(run<__half>(p, backward, ws, s));
    }
}

int check_desc(const gdn_group_norm_desc *d) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->N < 0 || d->L < 0 || d->C < 1 || d->G < 1 || d->C % d->G != 0) return GDN_ERR_INVALID_ARG;
    if (d->act != GDN_ACT_NONE && d->act != GDN_ACT_SILU) return GDN_ERR_UNSUPPORTED;
    if (!dtype_ok(d->dtype) || (d->weight_dtype != d->dtype && d->weight_dtype != GDN_F32)) return GDN_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f) || d->x_stride_n < 0 || d->x_stride_l < 0) return GDN_ERR_INVALID_ARG;
    if (d->L > 1 && d->x_stride_l < d->C) return GDN_ERR_INVALID_ARG;
    if (d->C > (1 << 24) || d->L > 0x7fff0000) return GDN_ERR_UNSUPPORTED;   // 32-bit loops over both
    if ((double)d->N * d->L * d->C > 4.0e12 || (int64_t)d->N * d->G > 0x7fffffff) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

int check_tensors(const gdn_group_norm_desc &d, const void *w, const void *b) {
    return ptr_aligned(w, act_size(d.weight_dtype)) && ptr_aligned(b, act_size(d.weight_dtype)) ? GDN_OK : GDN_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_group_norm_desc_init(gdn_group_norm_desc *d, int N, int L, int C, int G, int dtype) {
    if (!d) return GDN_ERR_INVALID_ARG;
    memset(d, 0, sizeof(*d));
    d->N = N;
    d->L = L;
    d->C = C;
    d->G = G;
    d->dtype = d->weight_dtype = dtype;
    d->act = GDN_ACT_SILU;
    d->eps = 1e-5f;
    d->x_stride_l = C;
    d->x_stride_n = (int64_t)C * L;
    return check_desc(d);
}

int gdn_group_norm_workspace_bytes(const gdn_group_norm_desc *d, size_t *bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    *bytes = workspace_need(*d, false);
    return GDN_OK;
}

int gdn_group_norm_backward_workspace_bytes(const gdn_group_norm_desc *d, size_t *bytes) {
    if (!bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    *bytes = workspace_need(*d, true);
    return GDN_OK;
}

int gdn_group_norm_forward(const gdn_group_norm_desc *d, const void *x, const void *weight, const void *bias, void *out,
                           float *mean, float *rstd, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    const bool any = (int64_t)d->N * d->L > 0;
    if (any && (!x || !out)) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(x, es) || !ptr_aligned(out, es) || !ptr_aligned(mean, 4) || !ptr_aligned(rstd, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_tensors(*d, weight, bias)) != GDN_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, workspace_need(*d, false))) != GDN_OK) return rc;
    if (!any) return GDN_OK;
    NormProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.w = weight;
    p.b = bias;
    p.out = out;
    p.mean = mean;
    p.rstd = rstd;
    return run_any(p, false, workspace, (cudaStream_t)stream);
}

int gdn_group_norm_backward(const gdn_group_norm_desc *d, const void *x, const void *weight, const void *bias,
                            const float *mean, const float *rstd, const void *grad_out, void *dx, float *dweight,
                            float *dbias, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_desc(d);
    if (rc != GDN_OK) return rc;
    const bool any = (int64_t)d->N * d->L > 0;
    if (any && (!x || !mean || !rstd || !grad_out || !dx)) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(x, es) || !ptr_aligned(grad_out, es) || !ptr_aligned(dx, es) || !ptr_aligned(mean, 4) ||
        !ptr_aligned(rstd, 4) || !ptr_aligned(dweight, 4) || !ptr_aligned(dbias, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_tensors(*d, weight, bias)) != GDN_OK) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, workspace_need(*d, true))) != GDN_OK) return rc;
    NormProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.x = x;
    p.w = weight;
    p.b = bias;
    p.mean = const_cast<float *>(mean);
    p.rstd = const_cast<float *>(rstd);
    p.dy = grad_out;
    p.dx = dx;
    p.dw = dweight;
    p.db = dbias;
    if (!any) {   // nothing to sum
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)d->C * 4, (cudaStream_t)stream);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)d->C * 4, (cudaStream_t)stream);
        return layer_status(e);
    }
    return run_any(p, true, workspace, (cudaStream_t)stream);
}

}  // extern "C"
