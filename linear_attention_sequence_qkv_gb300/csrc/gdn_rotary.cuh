// gdn_rotary.cuh -- what the rotary kernels share: a token's position and the cosine and
// sine of a pair's angle (include/gdn.h).
#pragma once

#include "gdn_common.cuh"

namespace gdn {

// the validation of a rotary descriptor (gdn_rotary.cu)
int rotary_check_desc(const gdn_rotary_desc *d, bool packed);

// Position of token t of row `row` (see gdn_rotary in include/gdn.h)
__device__ __forceinline__ int64_t rotary_position(const gdn_rotary_desc &d, const int32_t *pos, const int32_t *cu,
                                                   const int32_t *off, int row, int t) {
    if (pos) return pos[(int64_t)row * d.T + t];
    int n = row;
    int64_t at = t;
    if (cu) {
        n = upper_index(cu, d.N, t);
        at -= cu[n];
    }
    return at + (off ? off[n] : 0);
}

// cos and sin of 2 pi frac(position * turn / 2^64): the 64-bit product wraps at whole
// turns, and its upper half as a signed fraction has 32 bits of the remaining angle. For
// 16-bit outputs the hardware's functions on [-pi, pi] are exact enough (absolute error about
// 2^-21, against a rounding of 2^-9 or 2^-12), and where a token has few heads they are what
// bounds the kernel (one head of 64 for 64 x 60000 tokens: 389 us, 464 with sincospif).
template <bool FAST>
__device__ __forceinline__ float2 cos_sin(int64_t position, uint64_t turn) {
    const uint64_t phase = (uint64_t)position * turn;
    if (FAST) {
        const float a = (float)(int32_t)(phase >> 32) * 1.4629180792671596e-9f;   // 2 pi 2^-32
        return make_float2(__cosf(a), __sinf(a));
    }
    float c, s;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: in half turns
    return make_float2(c, s);
}

}  // namespace gdn
