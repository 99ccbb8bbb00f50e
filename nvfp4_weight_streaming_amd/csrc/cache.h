// The paged key/value cache as its kernels see it, and the checks and small
// device helpers they share.
#pragma once

#include "common.h"

namespace nvfp4 {

// A validated nvfp4_cache.  Byte strides; a page of one layer holds
//   K: [kv head][token][dim]    V: [kv head][token / 16][dim][token % 16]
// so that 16 bytes at consecutive addresses are consecutive dims of one key,
// and consecutive tokens of one value dim: both are MFMA operands as they lie
// in memory (the reduction of q k^T runs over dims, that of p v over tokens).
// Blocks of 16 tokens make both one run of 16 x dim values.
struct CacheView {
    uint8_t* k;
    uint8_t* v;
    long long layer_stride, page_stride;
    int layers, pages, kv_heads, dim;
    int log_page;  // log2 of tokens per page
    float k_scale, v_scale;
    int fp8;
};

// Checks `c` and fills `out`; layer -1: the caller takes all layers.
int cache_view(const nvfp4_cache* c, int layer, CacheView* out);
// Checks a lane count and a page table.
int check_lanes(const CacheView& c, int lanes, const int* table, int table_ld);

constexpr int kMaxLanes = 65535;  // a grid dimension

// The lane that owns row r: the number of lanes whose rows end at or before r.
// Every lane of the wave calls it with the same r (wave-parallel: one load per
// 64 lanes instead of a dependent search).
__device__ __forceinline__ int lane_of_row(const int* __restrict__ row_start, int lanes, int r) {
    int n = 0;
    for (int b0 = 0; b0 < lanes; b0 += 64) {
        const int b = b0 + (int)(threadIdx.x & 63);
        const bool before = b < lanes && row_start[b + 1] <= r;
        n += __popcll(__ballot(before));
    }
    return n;
}

// Element of V for dim index e = head x dims + d and token t of a page.
__device__ __forceinline__ long long v_element(const CacheView& c, int e, int t) {
    const int head = e / c.dim, d = e - head * c.dim;
    return ((((long long)head << (c.log_page - 4)) + (t >> 4)) * c.dim + d) * 16 + (t & 15);
}

// E4M3 of x / scale: nearest, ties to even, saturating at 448; two values.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    a = a != a ? a : fminf(fmaxf(a, -448.f), 448.f);
    b = b != b ? b : fminf(fmaxf(b, -448.f), 448.f);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

}  // namespace nvfp4
