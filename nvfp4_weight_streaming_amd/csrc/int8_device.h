// What the kernels of the 8-bit product share: the packed layout, arguments and
// the epilogue.
#pragma once

#include "common.h"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Packed weights: [ceil(N / 16)][steps][lane][16 bytes], steps = 2 ceil(K / 128);
// lane l of a step holds channel l % 16, k = 64 step + 16 (l / 16) .. + 15.
constexpr int kI8Step = 64;             // k of an operand
constexpr int kI8Bytes = 16 * kI8Step;  // bytes of an operand

inline int i8_steps(int K) { return 2 * ((K + 127) / 128); }
inline int i8_tiles(int N) { return (N + 15) / 16; }
inline bool i8_shape(int K, int N) { return K >= 16 && K % 16 == 0 && K <= NVFP4_INT8_MAX_K && N >= 1 && N <= (1 << 30); }

struct I8Args {
    const int8_t* a;
    const float* a_scale;
    const int8_t* w;
    const float* w_scale;
    const float* bias;
    void* out;
    long long a_ld, out_ld;
    int M, K, N, steps, tiles;
    int vec, wide;  // outputs may be stored four at a time; 16 bytes at a time
};

// Global memory through buffer resources: a base and a size in scalar registers, a 32-bit offset a lane; what lies
// past the size reads zero.
constexpr int kI8Raw = 0x00020000;  // resource word 3: raw 32-bit data
constexpr int kI8Stream = 2;        // non-temporal
__device__ __forceinline__ __amdgpu_buffer_rsrc_t i8_rsrc(const void* base, long long bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes > 0x7FFFFFFF ? 0x7FFFFFFF : (int)bytes, kI8Raw);
}
template <int AUX>
__device__ __forceinline__ u32x4 i8_load(__amdgpu_buffer_rsrc_t from, int at) {
    return __builtin_amdgcn_raw_buffer_load_b128(from, at, 0, AUX);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
// Two values to bf16, nearest even.
__device__ __forceinline__ uint32_t i8_bf16x2(float a, float b) {
    const bf16x2v v = __builtin_convertvector((f32x2{a, b}), bf16x2v);
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}

// A sum to its output.  No step is contracted into the next, so that every kernel gives the same value.
__device__ __forceinline__ float i8_value(int sum, float as, float ws) {
#pragma clang fp contract(off)
    return (float)sum * as * ws;
}
__device__ __forceinline__ float i8_biased(float y, float bias) {
#pragma clang fp contract(off)
    return y + bias;
}

// Four outputs of row m from n on, with its scale and the channels' scales and bias.
template <bool BF16>
__device__ __forceinline__ void i8_store_scaled(const I8Args& p, int m, int n, i32x4 acc, float as, const float (&ws)[4], const float (&bias)[4]) {
    if (m >= p.M || n >= p.N) return;
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        y[r] = i8_value(acc[r], as, ws[r]);
        if (p.bias) y[r] = i8_biased(y[r], bias[r]);
    }
    const long long at = (long long)m * p.out_ld + n;
    if (p.vec && n + 4 <= p.N) {
        if (BF16)
            *(uint2*)((uint16_t*)p.out + at) = make_uint2(i8_bf16x2(y[0], y[1]), i8_bf16x2(y[2], y[3]));
        else
            *(float4*)((float*)p.out + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < p.N) {
                if (BF16)
                    ((uint16_t*)p.out)[at + r] = (uint16_t)i8_bf16x2(y[r], 0.f);
                else
                    ((float*)p.out)[at + r] = y[r];
            }
    }
}

// Launchers (no validation).
int launch_int8_tile(const I8Args& p, bool bf16, void* ws, hipStream_t s);
size_t int8_tile_ws(int M, int K, int N);

}  // namespace nvfp4
