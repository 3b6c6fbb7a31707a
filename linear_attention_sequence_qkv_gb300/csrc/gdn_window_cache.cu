// gdn_window_cache.cu -- the window attention's cache of fixed size (include/gdn.h): its
// filling, and one token per sequence over it.
#include <string.h>

#include <algorithm>

#include "gdn_window.cuh"

namespace gdn {

int window_check_desc(const gdn_window_attention_desc *d, bool packed);   // gdn_window_attention.cu

namespace {

struct CacheProblem {
    gdn_window_attention_desc d;
    const void *q, *k, *v;
    const int32_t *cu, *lengths;
    void *kc, *vc, *out;
    int32_t *status;
};

// The slot that holds a position
__device__ __forceinline__ int64_t slot_of(int64_t position, int sinks, int slots) {
    return position < sinks ? position : sinks + (position - sinks) % (slots - sinks);
}

// A warp takes a token at a time and copies its rows of K and V in units of V; tokens whose place a later one of the call
// takes are passed over. Bound by HBM: 94 % of the copy rate where all is new (1.4 GB in 222 us); a small call is its launch.
constexpr int kWriteWarps = 8;
template <typename V>
__global__ void __launch_bounds__(32 * kWriteWarps) cache_write_kernel(const __grid_constant__ CacheProblem p, int es) {
    const gdn_window_attention_desc &d = p.d;
    const bool ok = p.cu == nullptr || seqlens_ok(p.cu, d.N, d.Tk);
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = ok ? GDN_OK : GDN_ERR_DEVICE_SEQLENS;
    if (!ok) return;
    const int lane = threadIdx.x & 31;
    const int per = d.d * es / (int)sizeof(V), units = d.Hk * per;   // units of a head's and of a token's row
    const int64_t total = (int64_t)d.B * d.Tk;
    for (int64_t tok = (int64_t)blockIdx.x * kWriteWarps + (threadIdx.x >> 5); tok < total; tok += (int64_t)gridDim.x * kWriteWarps) {
        const int n = p.cu ? upper_index(p.cu, d.N, tok) : (int)(tok / d.Tk);
        const int64_t at = tok - (p.cu ? p.cu[n] : (int64_t)n * d.Tk), count = p.cu ? p.cu[n + 1] - p.cu[n] : d.Tk;
        const int length = p.lengths[n];
        if (length < 0) continue;
        const int64_t pos = length + at;
        if (pos >= d.sinks && at < count - (d.slots - d.sinks)) continue;
        const int64_t row = p.cu ? 0 : n, in = p.cu ? tok : at, slot = slot_of(pos, d.sinks, d.slots);
        const V *k = (const V *)((const char *)p.k + (row * d.k_stride_b + in * d.k_stride_t) * es);
        const V *v = (const V *)((const char *)p.v + (row * d.v_stride_b + in * d.v_stride_t) * es);
        V *kc = (V *)p.kc + ((int64_t)n * d.Hk * d.slots + slot) * per, *vc = (V *)p.vc + ((int64_t)n * d.Hk * d.slots + slot) * per;
        constexpr int kB = 4;   // of each tensor in flight per lane
        for (int u0 = lane; u0 < units; u0 += 32 * kB) {
            V a[kB], b[kB];
#pragma unroll
            for (int j = 0; j < kB; ++j)
                if (u0 + 32 * j < units) a[j] = k[u0 + 32 * j], b[j] = v[u0 + 32 * j];
#pragma unroll
            for (int j = 0; j < kB; ++j)
                if (u0 + 32 * j < units) {
                    const int h = (u0 + 32 * j) / per, c = u0 + 32 * j - h * per;
                    const int64_t to = (int64_t)h * d.slots * per + c;
                    kc[to] = a[j], vc[to] = b[j];
                }
        }
    }
}

constexpr int kStepWarps = 4;
constexpr int kMostSplits = 16;   // CTAs of a cluster that share one sequence and head

// The keys that a new token at `pos` sees, in the cache's slots: [0, a), then b of the ring from r0 on, round its end
struct StepKeys {
    int a, total, r0, ring, sinks;
    __device__ __forceinline__ int slot(int t) const {
        if (t < a) return t;
        const int64_t r = (int64_t)r0 + t - a;
        return sinks + (int)(r >= ring ? r - ring : r);
    }
};
__device__ __forceinline__ StepKeys step_keys(const gdn_window_attention_desc &d, int64_t pos) {
    StepKeys k;
    k.ring = d.slots - d.sinks, k.sinks = d.sinks;
    k.a = (int)min((int64_t)d.sinks, pos + 1);
    const int64_t lo = max((int64_t)d.sinks, pos - d.window + 1);
    k.total = k.a + (int)max((int64_t)0, pos - lo + 1);
    k.r0 = (int)((lo - d.sinks) % k.ring);
    return k;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float of_rank(const float *own, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(own)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// What the warps of a CTA, and then the CTAs of the cluster, found of up to `heads` heads: their sums, maxima (log2) and
// weights are joined in the warps' and the ranks' order and the result stored. part: [kStepWarps][heads][width + 2] in shared
// memory, a row's sums, then m and l. All threads call it.
template <typename T>
__device__ __forceinline__ void step_join(float *part, int heads, int width, int d, T *out, uint32_t rank, int splits) {
    const int row = width + 2;
    __syncthreads();
    // a scale per warp and head first, then every thread its channels, in place into warp 0's rows
    __shared__ float scale[kStepWarps][16];
    for (int x = threadIdx.x; x < heads; x += blockDim.x) {
        float m = -INFINITY, l = 0.0f;
        for (int w = 0; w < kStepWarps; ++w) m = fmaxf(m, part[(w * heads + x) * row + width]);
        const float mm = m == -INFINITY ? 0.0f : m;
        for (int w = 0; w < kStepWarps; ++w) {
            const float f = exp2f(part[(w * heads + x) * row + width] - mm);
            scale[w][x] = f;
            l += f * part[(w * heads + x) * row + width + 1];
        }
        part[x * row + width] = m, part[x * row + width + 1] = l;
    }
    __syncthreads();
    for (int x = threadIdx.x; x < heads * width; x += blockDim.x) {
        const int h = x / width, c = x - h * width;
        float s = 0.0f;
        for (int w = 0; w < kStepWarps; ++w) s += scale[w][h] * part[(w * heads + h) * row + c];
        part[h * row + c] = s;
    }
    if (splits == 1) {
        __syncthreads();
        for (int x = threadIdx.x; x < heads * d; x += blockDim.x) {
            const int h = x / d, c = x - h * d;
            out[x] = from_f<T>(part[h * row + c] / part[h * row + width + 1]);
        }
        return;
    }
    cluster_sync();
    for (int x = rank * blockDim.x + threadIdx.x; x < heads * d; x += splits * blockDim.x) {
        const int h = x / d, c = x - h * d;
        float m[kMostSplits], top = -INFINITY;
#pragma unroll
        for (int r = 0; r < kMostSplits; ++r) {
            m[r] = r < splits ? of_rank(part + h * row + width, r) : -INFINITY;
            top = fmaxf(top, m[r]);
        }
        const float mm = top == -INFINITY ? 0.0f : top;
        float s = 0.0f, l = 0.0f;
#pragma unroll
        for (int r = 0; r < kMostSplits; ++r)
            if (r < splits) {
                const float f = exp2f(m[r] - mm);
                s += f * of_rank(part + h * row + c, r);
                l += f * of_rank(part + h * row + width + 1, r);
            }
        out[x] = from_f<T>(s / l);
    }
    cluster_sync();   // no CTA leaves while another reads its rows
}

template <typename T> __device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma_16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <> __device__ __forceinline__ void mma_16816<__nv_bfloat16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16-bit types, heads of up to 32 NG channels (a multiple of 8), 16-byte aligned rows. Bound by the bytes of the cache:
// these go from memory into registers in the layout that mma.sync takes (no tile of 128 queries to give tcgen05, and no
// shared memory on the way). A warp takes 16 keys at a time, the next 16 on their way:
//   S [heads x keys] = Q K^T: a lane's 16 bytes of a key's row are four of the contraction's indexes in each of two steps,
//     for Q alike, since any order of a contraction does;
//   O [heads x channels] += P V: P as it lies in S's registers; a lane reads 8 channels of keys 2i and 2i + 1 and pairs
//     them up, channel 8 j + t being column j of product t.
// Rows 8 to 15 of the products are heads 8 to 15 (WIDE), else empty. P is rounded to the tensors' type, which the product takes.
// 256 sequences of 4100 keys, 32 heads of 128 on 8: 3.9 GB in 624 us, 91 % of the copy rate; 8 of 1028, 32 heads on 16, whose
// 66 MB are in L2: 13 us in a graph.
template <typename T, int NG, bool WIDE>
__global__ void __launch_bounds__(32 * kStepWarps, 2) step_mma(const __grid_constant__ CacheProblem p, int splits, int head_tiles) {
    constexpr int NV = (NG + 1) / 2, kHeads = WIDE ? 16 : 8;
    extern __shared__ float part[];
    const gdn_window_attention_desc &d = p.d;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = GDN_OK;
    const uint32_t rank = splits > 1 ? cluster_rank() : 0;
    const int unit = blockIdx.x / splits, group = d.Hq / d.Hk;
    const int ht = unit % head_tiles, hk = unit / head_tiles % d.Hk, n = unit / head_tiles / d.Hk;
    const int h0 = ht * kHeads, heads = min(kHeads, group - h0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = lane & 3, oct = lane >> 2;
    T *out = (T *)p.out + ((int64_t)n * d.Hq + hk * group + h0) * d.d;
    const int64_t pos = p.lengths[n];
    if (pos < 0) {   // the whole cluster leaves
        if (rank == 0)
            for (int x = threadIdx.x; x < heads * d.d; x += blockDim.x) out[x] = from_f<T>(0.0f);
        return;
    }
    const StepKeys keys = step_keys(d, pos);
    const int64_t here = slot_of(pos, d.sinks, d.slots);
    T *kc = (T *)p.kc + ((int64_t)n * d.Hk + hk) * d.slots * d.d, *vc = (T *)p.vc + ((int64_t)n * d.Hk + hk) * d.slots * d.d;
    const T *kn = (const T *)p.k + n * d.k_stride_b + (int64_t)hk * d.d, *vn = (const T *)p.v + n * d.v_stride_b + (int64_t)hk * d.d;
    // the new token's place is written here and read nowhere: its key and value come from the call's arguments
    if (rank == 0 && ht == 0 && threadIdx.x < 2 * (d.d / 8)) {
        const int c = threadIdx.x % (d.d / 8);
        const bool isv = threadIdx.x >= d.d / 8;
        *(uint4 *)((isv ? vc : kc) + here * d.d + 8 * c) = *(const uint4 *)((isv ? vn : kn) + 8 * c);
    }
    const int groups = (keys.total + 15) / 16, chunk = (groups + splits - 1) / splits;
    const int g1 = min(groups, (int)(rank + 1) * chunk);
    int g = rank * chunk + warp;

    uint4 q[NG][2];
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int c = 32 * i + 8 * quad, h = oct + 8 * r;
            q[i][r] = make_uint4(0, 0, 0, 0);
            if ((r == 0 || WIDE) && h < heads && c < d.d)
                q[i][r] = *(const uint4 *)((const T *)p.q + n * d.q_stride_b + (int64_t)(hk * group + h0 + h) * d.d + c);
        }
    float o[NV * 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NV * 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    const float c = d.scale * 1.4426950408889634f;

    uint4 kr[2][NG], vr[4][NV];   // keys oct, oct + 8; keys 2 quad + {0, 1, 8, 9}
    auto fetch = [&](int at) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int s = keys.slot(min(16 * at + 8 * r + oct, keys.total - 1));
            const T *row = s == here ? kn : kc + (int64_t)s * d.d;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                kr[r][i] = make_uint4(0, 0, 0, 0);
                if (32 * i + 8 * quad < d.d) kr[r][i] = *(const uint4 *)(row + 32 * i + 8 * quad);
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * at + 2 * quad + (r & 1) + 8 * (r >> 1), s = keys.slot(min(t, keys.total - 1));
            const T *row = s == here ? vn : vc + (int64_t)s * d.d;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                vr[r][i] = make_uint4(0, 0, 0, 0);   // also for keys past the end: 0 x inf would be NaN
                if (64 * i + 8 * oct < d.d && t < keys.total) vr[r][i] = *(const uint4 *)(row + 64 * i + 8 * oct);
            }
        }
    };
    if (g < g1) fetch(g);
    for (; g < g1; g += kStepWarps) {
        float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                mma_16816<T>(s[r], q[i][0].x, q[i][1].x, q[i][0].y, q[i][1].y, kr[r][i].x, kr[r][i].y);
                mma_16816<T>(s[r], q[i][0].z, q[i][1].z, q[i][0].w, q[i][1].w, kr[r][i].z, kr[r][i].w);
            }
        uint32_t v[NV][8][2];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t a[4] = {vr[2 * r][i].x, vr[2 * r][i].y, vr[2 * r][i].z, vr[2 * r][i].w};
                const uint32_t b[4] = {vr[2 * r + 1][i].x, vr[2 * r + 1][i].y, vr[2 * r + 1][i].z, vr[2 * r + 1][i].w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    v[i][2 * w][r] = __byte_perm(a[w], b[w], 0x5410);
                    v[i][2 * w + 1][r] = __byte_perm(a[w], b[w], 0x7632);
                }
            }
        const int left = keys.total - 16 * g;
        if (g + kStepWarps < g1) fetch(g + kStepWarps);
        if (left < 16)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[r][e] = 8 * r + 2 * quad + (e & 1) < left ? s[r][e] : -INFINITY;
        float pr[2][4];
        bool grow = false;
        float top[2];
#pragma unroll
        for (int x = 0; x < (WIDE ? 2 : 1); ++x) {
            float t = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
            top[x] = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
            grow |= top[x] > m[x] && (m[x] == -INFINITY || (top[x] - m[x]) * c > 8.0f);
        }
        if (__any_sync(0xffffffffu, grow)) {   // rare: the maximum grew by more than 2^8 (or is the first)
#pragma unroll
            for (int x = 0; x < (WIDE ? 2 : 1); ++x) {
                const float f = top[x] > m[x] ? exp2f((m[x] - top[x]) * c) : 1.0f;
                m[x] = fmaxf(m[x], top[x]);
                l[x] *= f;
#pragma unroll
                for (int i = 0; i < NV * 8; ++i) o[i][2 * x] *= f, o[i][2 * x + 1] *= f;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float w = 0.0f;
                    if (x == 0 || WIDE) {
                        w = ex2_approx(fmaf(s[r][2 * x + e], c, m[x] == -INFINITY ? 0.0f : fmaf(-m[x], c, kRaised<T>)));
                        l[x] += w;
                    }
                    pr[r][2 * x + e] = w;
                }
        const uint32_t a0 = Pairs<T>::pack1(make_float2(pr[0][0], pr[0][1])), a1 = Pairs<T>::pack1(make_float2(pr[0][2], pr[0][3]));
        const uint32_t a2 = Pairs<T>::pack1(make_float2(pr[1][0], pr[1][1])), a3 = Pairs<T>::pack1(make_float2(pr[1][2], pr[1][3]));
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int t = 0; t < 8; ++t) mma_16816<T>(o[8 * i + t], a0, a1, a2, a3, v[i][t][0], v[i][t][1]);
    }
    // rows of the warp: sums, then m (log2) and l
    constexpr int kWidth = NV * 64;
#pragma unroll
    for (int x = 0; x < (WIDE ? 2 : 1); ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int h = oct + 8 * x;
        if (h < heads) {
            float *to = part + (warp * heads + h) * (kWidth + 2);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    to[64 * i + 16 * quad + t] = o[8 * i + t][2 * x];
                    to[64 * i + 16 * quad + 8 + t] = o[8 * i + t][2 * x + 1];
                }
            if (quad == 0) to[kWidth] = m[x] * c, to[kWidth + 1] = l[x];
        }
    }
    step_join<T>(part, heads, kWidth, d.d, out, rank, splits);
}

// fp32 with 16-byte aligned rows of up to 32 NG channels, a multiple of 4: 8 lanes share a key, a lane has the channels
// 32 i + 4 (lane % 8) .. + 3, a warp four keys at a time for up to 4 heads. Products and sums in fp32. Bound by HBM where a head of
// keys serves one of queries (128 sequences of 2052 keys, 16 heads of 128: 4.3 GB in 703 us, 90 % of the copy rate), else by the
// products of a step, during which no next keys are on their way (256 sequences, 32 heads on 8: 935 us, 68 %).
template <int NG>
__global__ void __launch_bounds__(32 * kStepWarps) step_f32(const __grid_constant__ CacheProblem p, int splits, int head_tiles) {
    constexpr int kHeads = 4, kKeys = 2;   // heads of a CTA; keys of a lane's group in flight
    extern __shared__ float part[];
    const gdn_window_attention_desc &d = p.d;
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = GDN_OK;
    const uint32_t rank = splits > 1 ? cluster_rank() : 0;
    const int unit = blockIdx.x / splits, group = d.Hq / d.Hk;
    const int ht = unit % head_tiles, hk = unit / head_tiles % d.Hk, n = unit / head_tiles / d.Hk;
    const int h0 = ht * kHeads, heads = min(kHeads, group - h0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7, kg = lane >> 3;
    float *out = (float *)p.out + ((int64_t)n * d.Hq + hk * group + h0) * d.d;
    const int64_t pos = p.lengths[n];
    if (pos < 0) {
        if (rank == 0)
            for (int x = threadIdx.x; x < heads * d.d; x += blockDim.x) out[x] = 0.0f;
        return;
    }
    const StepKeys keys = step_keys(d, pos);
    const int64_t here = slot_of(pos, d.sinks, d.slots);
    float *kc = (float *)p.kc + ((int64_t)n * d.Hk + hk) * d.slots * d.d, *vc = (float *)p.vc + ((int64_t)n * d.Hk + hk) * d.slots * d.d;
    const float *kn = (const float *)p.k + n * d.k_stride_b + (int64_t)hk * d.d, *vn = (const float *)p.v + n * d.v_stride_b + (int64_t)hk * d.d;
    if (rank == 0 && ht == 0)
        for (int x = threadIdx.x; x < d.d; x += blockDim.x) kc[here * d.d + x] = kn[x], vc[here * d.d + x] = vn[x];
    constexpr int kStep = 4 * kKeys;   // keys of a warp's step
    const int groups = (keys.total + kStep - 1) / kStep, chunk = (groups + splits - 1) / splits;
    const int g1 = min(groups, (int)(rank + 1) * chunk);
    const float c = d.scale * 1.4426950408889634f;
    float4 q[kHeads][NG], o[kHeads][NG];
    float m[kHeads], l[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        m[h] = -INFINITY, l[h] = 0.0f;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            q[h][i] = o[h][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (h < heads && 32 * i + 4 * sub < d.d)
                q[h][i] = *(const float4 *)((const float *)p.q + n * d.q_stride_b + (int64_t)(hk * group + h0 + h) * d.d + 32 * i + 4 * sub);
        }
    }
    for (int g = rank * chunk + warp; g < g1; g += kStepWarps) {
        float4 kr[kKeys][NG], vr[kKeys][NG];
        bool in[kKeys];
#pragma unroll
        for (int x = 0; x < kKeys; ++x) {
            const int t = g * kStep + 4 * x + kg, s = keys.slot(min(t, keys.total - 1));
            in[x] = t < keys.total;
            const float *krow = s == here ? kn : kc + (int64_t)s * d.d, *vrow = s == here ? vn : vc + (int64_t)s * d.d;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                kr[x][i] = vr[x][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (32 * i + 4 * sub < d.d && in[x]) {
                    kr[x][i] = *(const float4 *)(krow + 32 * i + 4 * sub);
                    vr[x][i] = *(const float4 *)(vrow + 32 * i + 4 * sub);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h >= heads) break;
            float s[kKeys];
            float t = -INFINITY;
#pragma unroll
            for (int x = 0; x < kKeys; ++x) {
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    a = fmaf(q[h][i].x, kr[x][i].x, a), a = fmaf(q[h][i].y, kr[x][i].y, a);
                    a = fmaf(q[h][i].z, kr[x][i].z, a), a = fmaf(q[h][i].w, kr[x][i].w, a);
                }
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                a += __shfl_xor_sync(0xffffffffu, a, 2);
                a += __shfl_xor_sync(0xffffffffu, a, 4);
                s[x] = in[x] ? a : -INFINITY;
                t = fmaxf(t, s[x]);
            }
            const float mn = fmaxf(m[h], t), mm = mn == -INFINITY ? 0.0f : mn;   // each group of 8 lanes its own maximum
            const float f = exp2f((m[h] - mm) * c);
            m[h] = mn;
            float w[kKeys];
            l[h] *= f;
#pragma unroll
            for (int x = 0; x < kKeys; ++x) w[x] = in[x] ? exp2f((s[x] - mm) * c) : 0.0f, l[h] += w[x];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                o[h][i].x *= f, o[h][i].y *= f, o[h][i].z *= f, o[h][i].w *= f;
#pragma unroll
                for (int x = 0; x < kKeys; ++x) {
                    o[h][i].x = fmaf(w[x], vr[x][i].x, o[h][i].x), o[h][i].y = fmaf(w[x], vr[x][i].y, o[h][i].y);
                    o[h][i].z = fmaf(w[x], vr[x][i].z, o[h][i].z), o[h][i].w = fmaf(w[x], vr[x][i].w, o[h][i].w);
                }
            }
        }
    }
    constexpr int kWidth = 32 * NG;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (h >= heads) break;
        float top = fmaxf(m[h], __shfl_xor_sync(0xffffffffu, m[h], 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float f = exp2f((m[h] - (top == -INFINITY ? 0.0f : top)) * c);
        float lw = l[h] * f;
        lw += __shfl_xor_sync(0xffffffffu, lw, 8);
        lw += __shfl_xor_sync(0xffffffffu, lw, 16);
        float *to = part + (warp * heads + h) * (kWidth + 2);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            float4 a = make_float4(o[h][i].x * f, o[h][i].y * f, o[h][i].z * f, o[h][i].w * f);
#pragma unroll
            for (int e = 8; e < 32; e *= 2) {
                a.x += __shfl_xor_sync(0xffffffffu, a.x, e), a.y += __shfl_xor_sync(0xffffffffu, a.y, e);
                a.z += __shfl_xor_sync(0xffffffffu, a.z, e), a.w += __shfl_xor_sync(0xffffffffu, a.w, e);
            }
            if (kg == 0) {
                float *at = to + 32 * i + 4 * sub;
                at[0] = a.x, at[1] = a.y, at[2] = a.z, at[3] = a.w;
            }
        }
        if (lane == 0) to[kWidth] = top * c, to[kWidth + 1] = lw;
    }
    step_join<float>(part, heads, kWidth, d.d, out, rank, splits);
}


// Any type, size and alignment: a CTA takes one sequence and head of keys, a warp one head of queries at a time
template <typename T, int NC>
__global__ void __launch_bounds__(32 * kStepWarps) step_rows(const __grid_constant__ CacheProblem p) {
    const gdn_window_attention_desc &d = p.d;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.status = GDN_OK;
    const int n = blockIdx.x, hk = blockIdx.y, lane = threadIdx.x & 31, group = d.Hq / d.Hk;
    T *out = (T *)p.out + ((int64_t)n * d.Hq + (int64_t)hk * group) * d.d;
    const int64_t pos = p.lengths[n];
    if (pos < 0) {
        for (int i = threadIdx.x; i < group * d.d; i += blockDim.x) out[i] = from_f<T>(0.0f);
        return;
    }
    T *kc = (T *)p.kc + ((int64_t)n * d.Hk + hk) * d.slots * d.d, *vc = (T *)p.vc + ((int64_t)n * d.Hk + hk) * d.slots * d.d;
    const T *kn = (const T *)p.k + n * d.k_stride_b + (int64_t)hk * d.d, *vn = (const T *)p.v + n * d.v_stride_b + (int64_t)hk * d.d;
    const int64_t here = slot_of(pos, d.sinks, d.slots);
    for (int c = threadIdx.x; c < d.d; c += blockDim.x) {
        kc[here * d.d + c] = kn[c];
        vc[here * d.d + c] = vn[c];
    }
    __syncthreads();
    // the keys seen: sinks before the window, then the window's
    const int64_t lo = pos >= d.window ? pos - d.window + 1 : 0, first = min((int64_t)d.sinks, lo), total = first + pos - lo + 1;
    for (int g = threadIdx.x >> 5; g < group; g += kStepWarps) {
        float qr[NC], o[NC], m = -INFINITY, l = 0.0f;
        row_load<T, NC>((const T *)p.q + n * d.q_stride_b + ((int64_t)hk * group + g) * d.d, d.d, lane, qr);
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c] = 0.0f;
        for (int64_t t0 = 0; t0 < total; t0 += 32) {
            const int cnt = (int)min((int64_t)32, total - t0);
            const int64_t t = t0 + lane, j = t < first ? t : min(lo + t - first, pos), sl = slot_of(j, d.sinks, d.slots);
            const float s = row_dot<T, NC>(qr, kc + sl * d.d, d.d) * d.scale, x = lane < cnt ? s : -INFINITY;
            const float mn = fmaxf(m, warp_max(x)), mm = mn == -INFINITY ? 0.0f : mn;
            const float corr = expf(m - mm), w = lane < cnt ? expf(x - mm) : 0.0f;
            l = l * corr + warp_sum(w);
#pragma unroll
            for (int c = 0; c < NC; ++c) o[c] *= corr;
            rows_add<T, NC>(o, w, vc + sl * d.d, cnt, d.d, lane);
            m = mn;
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c] /= l;
        row_store<T, NC>(out + (int64_t)g * d.d, d.d, lane, o);
    }
}

template <typename T>
cudaError_t launch_step_rows(const CacheProblem &p, cudaStream_t s) {
    const dim3 grid((unsigned)p.d.B, (unsigned)p.d.Hk);
    if (p.d.d <= 64) step_rows<T, 2><<<grid, 32 * kStepWarps, 0, s>>>(p);
    else if (p.d.d <= 128) step_rows<T, 4><<<grid, 32 * kStepWarps, 0, s>>>(p);
    else step_rows<T, 8><<<grid, 32 * kStepWarps, 0, s>>>(p);
    return cudaGetLastError();
}

// Rows of 16 bytes everywhere
bool step_aligned(const CacheProblem &p) {
    const gdn_window_attention_desc &d = p.d;
    const int64_t v = 16 / (int64_t)act_size(d.dtype);
    return d.d <= 128 && d.d % v == 0 && (d.B == 1 || (d.q_stride_b % v == 0 && d.k_stride_b % v == 0 && d.v_stride_b % v == 0)) &&
           ptr_aligned(p.q, 16) && ptr_aligned(p.k, 16) && ptr_aligned(p.v, 16) && ptr_aligned(p.kc, 16) && ptr_aligned(p.vc, 16) &&
           ptr_aligned(p.out, 16);
}

// CTAs per sequence and head: as many as make the rounds of two CTAs per SM cheapest, a CTA costing its keys and a start
// that is worth about 100 KB of them. By measurement, us a call with 1 | 2 | 4 | 8 | 16 (cache not in L2; * the rule's):
//   1 sequence of 1028, 32 heads of 128 on 8, bf16:  27 | 21 | 17 | 15* | 15    of 8196:  148 | 83 | 48 | 31 | 23*
//   8 of 1028, 32 on 16:  33 | 27* | 33 | 46 | 85     32 of them:  68* | 83 | 95 | 142 | 296
//   64 of 4100, 8 heads of 64, fp32:  295 | 244 | 224* | 267 | 367
int step_splits(const gdn_window_attention_desc &d, int64_t units) {
    const int64_t bytes = ((int64_t)d.sinks + d.window) * d.d * 2 * (int64_t)act_size(d.dtype);
    int best = 1;
    int64_t least = INT64_MAX;
    for (int s = 1; s <= kMostSplits; s *= 2) {
        const int64_t cost = cdiv64(units * s, 2 * kSms) * (100000 + bytes / s);
        if (cost < least) least = cost, best = s;
    }
    return best;
}

template <typename K>
cudaError_t launch_split(K kernel, const CacheProblem &p, int heads, int width, int head_tiles, cudaStream_t s) {
    const gdn_window_attention_desc &d = p.d;
    const int64_t units = (int64_t)d.B * d.Hk * head_tiles;
    const int splits = step_splits(d, units);
    if (units * splits > 0x7fffffff) return cudaErrorInvalidValue;
    static_assert(kStepWarps * 16 * (128 + 2) * 4 <= 40 * 1024, "what every kernel has without asking, beside its static part");
    const size_t smem = (size_t)kStepWarps * heads * (width + 2) * 4;   // at most 16 heads of 128
    cudaError_t e = cudaSuccess;
    if (splits > 8 && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * splits));
    cfg.blockDim = dim3(32 * kStepWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, splits, head_tiles);
}

template <typename T, int NG>
cudaError_t launch_step_mma(const CacheProblem &p, cudaStream_t s) {
    const int group = p.d.Hq / p.d.Hk, width = (NG + 1) / 2 * 64;
    if (group <= 8) return launch_split(step_mma<T, NG, false>, p, std::min(group, 8), width, 1, s);
    return launch_split(step_mma<T, NG, true>, p, 16, width, (group + 15) / 16, s);
}

template <typename T>
cudaError_t launch_step(const CacheProblem &p, cudaStream_t s) {
    if (!step_aligned(p)) return launch_step_rows<T>(p, s);
    const int ng = (p.d.d + 31) / 32;
    if constexpr (sizeof(T) == 4) {
        const int tiles = (p.d.Hq / p.d.Hk + 3) / 4;
        switch (ng) {
        case 1: return launch_split(step_f32<1>, p, 4, 32, tiles, s);
        case 2: return launch_split(step_f32<2>, p, 4, 64, tiles, s);
        case 3: return launch_split(step_f32<3>, p, 4, 96, tiles, s);
        default: return launch_split(step_f32<4>, p, 4, 128, tiles, s);
        }
    } else {
        switch (ng) {
        case 1: return launch_step_mma<T, 1>(p, s);
        case 2: return launch_step_mma<T, 2>(p, s);
        case 3: return launch_step_mma<T, 3>(p, s);
        default: return launch_step_mma<T, 4>(p, s);
        }
    }
}

template <typename V>
cudaError_t launch_write(const CacheProblem &p, int es, cudaStream_t s) {
    const int64_t total = (int64_t)p.d.B * p.d.Tk;
    const int64_t blocks = std::min<int64_t>(std::max<int64_t>(cdiv64(total, kWriteWarps), 1), 8 * kSms);
    cache_write_kernel<V><<<(unsigned)blocks, 32 * kWriteWarps, 0, s>>>(p, es);
    return cudaGetLastError();
}
// Whether units of `bytes` divide a head's row and fit every base and stride
bool units_fit(const CacheProblem &p, size_t bytes) {
    const gdn_window_attention_desc &d = p.d;
    const size_t es = act_size(d.dtype);
    const int64_t st[] = {d.d, d.Tk > 1 ? d.k_stride_t : 0, d.Tk > 1 ? d.v_stride_t : 0, d.B > 1 ? d.k_stride_b : 0, d.B > 1 ? d.v_stride_b : 0};
    for (const int64_t x : st)
        if (x * es % bytes) return false;
    return ptr_aligned(p.k, bytes) && ptr_aligned(p.v, bytes) && ptr_aligned(p.kc, bytes) && ptr_aligned(p.vc, bytes);
}

int check_cache(const gdn_window_attention_desc *d, bool packed) {
    const int rc = window_check_desc(d, packed);
    if (rc != GDN_OK) return rc;
    if (d->slots < (int64_t)d->sinks + d->window) return GDN_ERR_INVALID_ARG;
    if (d->Hk > 65535 || d->slots > 0x7fffffff - 65535) return GDN_ERR_UNSUPPORTED;   // keys are counted in groups, in 32 bits
    return GDN_OK;
}

int bytes_of(const gdn_window_attention_desc *d, size_t *bytes) {
    if (!d || !bytes) return GDN_ERR_INVALID_ARG;
    const int rc = check_cache(d, d->N != d->B);
    if (rc != GDN_OK) return rc;
    *bytes = kStatusBytes;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_window_attention_step_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes) { return bytes_of(d, bytes); }
int gdn_window_cache_write_workspace_bytes(const gdn_window_attention_desc *d, size_t *bytes) { return bytes_of(d, bytes); }

int gdn_window_cache_write(const gdn_window_attention_desc *d, const void *k, const void *v, const int32_t *cu_seqlens,
                           const int32_t *lengths, void *k_cache, void *v_cache, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream) {
    int rc = check_cache(d, cu_seqlens != nullptr);
    if (rc != GDN_OK) return rc;
    if ((int64_t)d->B * d->Tk > 0 && (!k || !v)) return GDN_ERR_INVALID_ARG;   // no tokens: these may be null
    if (!lengths || !k_cache || !v_cache) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(k, es) || !ptr_aligned(v, es) || !ptr_aligned(k_cache, es) || !ptr_aligned(v_cache, es) ||
        !ptr_aligned(lengths, 4) || !ptr_aligned(cu_seqlens, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    CacheProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.k = k, p.v = v, p.cu = cu_seqlens, p.lengths = lengths;
    p.kc = k_cache, p.vc = v_cache;
    p.status = (int32_t *)workspace;
    const cudaStream_t s = (cudaStream_t)stream;
    if (units_fit(p, 16)) return layer_status(launch_write<uint4>(p, (int)es, s));
    if (units_fit(p, 4)) return layer_status(launch_write<uint32_t>(p, (int)es, s));
    return layer_status(launch_write<uint16_t>(p, (int)es, s));
}

int gdn_window_attention_step(const gdn_window_attention_desc *d, const void *q, const void *k, const void *v, const int32_t *lengths,
                              void *k_cache, void *v_cache, void *out, void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
    int rc = check_cache(d, false);
    if (rc != GDN_OK) return rc;
    if (d->Tq != 1 || d->Tk != 1) return GDN_ERR_INVALID_ARG;
    if (!q || !k || !v || !lengths || !k_cache || !v_cache || !out) return GDN_ERR_INVALID_ARG;
    const size_t es = act_size(d->dtype);
    if (!ptr_aligned(q, es) || !ptr_aligned(k, es) || !ptr_aligned(v, es) || !ptr_aligned(k_cache, es) || !ptr_aligned(v_cache, es) ||
        !ptr_aligned(out, es) || !ptr_aligned(lengths, 4))
        return GDN_ERR_INVALID_ARG;
    if ((rc = check_workspace(workspace, workspace_bytes, kStatusBytes)) != GDN_OK) return rc;
    CacheProblem p;
    memset(&p, 0, sizeof(p));
    p.d = *d;
    p.q = q, p.k = k, p.v = v, p.lengths = lengths;
    p.kc = k_cache, p.vc = v_cache, p.out = out;
    p.status = (int32_t *)workspace;
    const cudaStream_t s = (cudaStream_t)stream;
    switch (d->dtype) {
    case GDN_F32: return layer_status(launch_step<float>(p, s));
    case GDN_BF16: return layer_status(launch_step<__nv_bfloat16>(p, s));
    default: return layer_status(launch_step<__half>(p, s));
    }
}

}  // extern "C"
