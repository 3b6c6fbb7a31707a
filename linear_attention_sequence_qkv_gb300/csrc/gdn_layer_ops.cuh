// gdn_layer_ops.cuh -- what the operators beside the gated delta rule share: host
// checks of sizes and alignment, and the device check of cu_seqlens.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr size_t kStatusBytes = 256;   // the status word's block at the start of a workspace
constexpr int kSms = 152;

inline bool ptr_aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool dtype_ok(int dtype) { return dtype >= GDN_F32 && dtype <= GDN_F16; }
inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int layer_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }
inline int check_workspace(const void *ws, size_t have, size_t need) {
    return ws && ptr_aligned(ws, 256) && have >= need ? GDN_OK : GDN_ERR_WORKSPACE;
}

// gdn_set_wait_test_mode's state (gdn_api.cu)
int wait_test_mode();

// Whole-block check of cu_seqlens: 0-based, non-decreasing, ending at T. Every
// block of a launch reads the same N + 1 words (they stay in L2) and so comes to
// the same answer; this costs no launch of its own. All threads must call it.
__device__ __forceinline__ bool seqlens_ok(const int32_t *cu, int N, int T) {
    bool bad = false;
    for (int i = threadIdx.x; i <= N; i += blockDim.x) {
        const int v = cu[i];
        bad |= (i == 0 && v != 0) || (i == N && v != T) || (i < N && cu[i + 1] < v);
    }
    return !__syncthreads_or(bad);
}

}  // namespace gdn
