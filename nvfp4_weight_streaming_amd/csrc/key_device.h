// 64-bit keys whose order is (value descending, index ascending), and the
// wave-wide maximum over them: shared by the top-k and beam-selection kernels.
#pragma once

#include "common.h"

namespace nvfp4 {

typedef unsigned long long u64;

__device__ __forceinline__ u64 topk_key(float v, int i) {
    unsigned int b = __float_as_uint(v);
    if (b == 0x80000000u) b = 0u;  // -0 -> +0
    const unsigned int o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return ((u64)o << 32) | (unsigned int)(~i);
}

__device__ __forceinline__ u64 max64(u64 a, u64 b) { return a > b ? a : b; }

// v from the lane that DPP control `ctrl` selects (both halves).
template <int CTRL>
__device__ __forceinline__ u64 dpp64(u64 v) {
    const int lo = __builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp((int)(v >> 32), (int)(v >> 32), CTRL, 0xF, 0xF,
                                               false);
    return ((u64)(unsigned int)hi << 32) | (unsigned int)lo;
}

__device__ __forceinline__ u64 lane64(u64 v, int lane) {
    const unsigned int lo = __builtin_amdgcn_readlane((int)v, lane);
    const unsigned int hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
    return ((u64)hi << 32) | lo;
}

// The wave's largest key, uniform.  Within each row of 16 lanes: swap lane
// pairs, then quad halves (quad_perm [1,0,3,2] and [2,3,0,1]), then the
// mirrors of each 8 and of the 16; every lane of a row then holds the row's
// maximum.  The four rows' maxima are read from lanes 0, 16, 32 and 48.
__device__ __forceinline__ u64 wave_max64(u64 v) {
    v = max64(v, dpp64<0xB1>(v));   // quad_perm [1,0,3,2]
    v = max64(v, dpp64<0x4E>(v));   // quad_perm [2,3,0,1]
    v = max64(v, dpp64<0x141>(v));  // row_half_mirror
    v = max64(v, dpp64<0x140>(v));  // row_mirror
    return max64(max64(lane64(v, 0), lane64(v, 16)), max64(lane64(v, 32), lane64(v, 48)));
}

}  // namespace nvfp4
