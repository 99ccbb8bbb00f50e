// Reductions over a wave and the selection of the best of many distinct keys:
// shared by beam selection and log probabilities.
#pragma once

#include "key_device.h"

namespace nvfp4 {

// The wave's maximum and sum, uniform: as wave_max64, within rows of 16 lanes by
// DPP, then over the four rows.
template <int CTRL>
__device__ __forceinline__ float dppf(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lanef(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dppf<0xB1>(v));
    v = fmaxf(v, dppf<0x4E>(v));
    v = fmaxf(v, dppf<0x141>(v));
    v = fmaxf(v, dppf<0x140>(v));
    return fmaxf(fmaxf(lanef(v, 0), lanef(v, 16)), fmaxf(lanef(v, 32), lanef(v, 48)));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dppf<0xB1>(v);
    v += dppf<0x4E>(v);
    v += dppf<0x141>(v);
    v += dppf<0x140>(v);
    return (lanef(v, 0) + lanef(v, 16)) + (lanef(v, 32) + lanef(v, 48));
}
template <int CTRL>
__device__ __forceinline__ double dppd(double v) {
    return __longlong_as_double((long long)dpp64<CTRL>((u64)__double_as_longlong(v)));
}
__device__ __forceinline__ double laned(double v, int lane) {
    return __longlong_as_double((long long)lane64((u64)__double_as_longlong(v), lane));
}
__device__ __forceinline__ double wave_sumd(double v) {
    v += dppd<0xB1>(v);
    v += dppd<0x4E>(v);
    v += dppd<0x141>(v);
    v += dppd<0x140>(v);
    return (laned(v, 0) + laned(v, 16)) + (laned(v, 32) + laned(v, 48));
}
// exp(x - m): the difference is rounded before it is scaled, so that terms near
// the maximum, which make up the sum, are off by 2^-22 or less.
__device__ __forceinline__ float exp_diff(float x, float m) {
    return __builtin_amdgcn_exp2f((x - m) * 1.44269504088896340736f);
}

// Merges the lane's N keys into the wave's sorted list (lane r: the r-th
// largest; 0: none) and keeps the k largest.  Keys are distinct.
template <int N>
__device__ __forceinline__ u64 wave_keep(u64 kept, u64 (&x)[N], int k, int lane) {
    u64 out = 0;
    for (int r = 0; r < k; ++r) {
        u64 head = kept;
#pragma unroll
        for (int j = 0; j < N; ++j) head = max64(head, x[j]);
        const u64 top = wave_max64(head);
        if (top == 0) break;
        out = lane == r ? top : out;
        kept = kept == top ? 0 : kept;
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = x[j] == top ? 0 : x[j];
    }
    return out;
}

// Inserts the wave's keys, those with `take`, one by one into its sorted list (lane r: the r-th
// largest) of k.
__device__ __forceinline__ u64 wave_insert(u64 kept, u64 key, bool take, int k, int lane) {
    unsigned long long todo = __ballot(take && key > lane64(kept, k - 1));
    while (todo) {
        const u64 v = lane64(key, __ffsll(todo) - 1);
        todo &= todo - 1;
        u64 prev = ((u64)(unsigned int)__shfl_up((int)(kept >> 32), 1) << 32) | (unsigned int)__shfl_up((int)kept, 1);
        if (lane == 0) prev = ~0ull;
        kept = kept > v ? kept : prev > v ? v : prev;
    }
    return kept;
}

// Appends the wave's keys that have `take` to a list in LDS (in no
// particular order); *count goes on past the end of its LIST places.
template <int LIST>
__device__ __forceinline__ void append_keys(u64 key, bool take, u64* list, int* count, int lane) {
    const unsigned long long mine = __ballot(take);
    if (!mine) return;
    int at = 0;
    if (lane == 0) at = atomicAdd(count, __popcll(mine));
    at = __builtin_amdgcn_readfirstlane(at) + __popcll(mine & ((1ull << lane) - 1ull));
    if (take && at < LIST) list[at] = key;
}

// The k largest of n distinct keys, in order: a key's place is the number of
// larger ones.  best[] past n is 0.
template <int THREADS>
__device__ __forceinline__ void rank_keys(const u64* list, int n, int k, u64* best) {
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const u64 x = list[i];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) place += list[j] > x ? 1 : 0;
        if (place < k) best[place] = x;
    }
    if ((int)threadIdx.x >= n && (int)threadIdx.x < k) best[threadIdx.x] = 0;
}

// Largest key of each row of 16 lanes, and the sum of a count, in all of its lanes.
__device__ __forceinline__ u64 row_max64(u64 v) {
    v = max64(v, dpp64<0xB1>(v));
    v = max64(v, dpp64<0x4E>(v));
    v = max64(v, dpp64<0x141>(v));
    return max64(v, dpp64<0x140>(v));
}
template <int CTRL>
__device__ __forceinline__ int dppi(int v) {
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ int row_sum(int v) {
    v += dppi<0xB1>(v);
    v += dppi<0x4E>(v);
    v += dppi<0x141>(v);
    return v + dppi<0x140>(v);
}

}  // namespace nvfp4
