// The product of 8-bit rows and 8-bit weights.
//
//   out[m][n] = float(sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
//
// v_mfma_i32_16x16x64_i8 takes both operands as 16 bytes a lane (lane l: row or
// column l % 16, 16 values of k from 16 * (l / 16)) and adds in 32 bits, exactly.
// The weights are its first operand, so that a lane ends with four consecutive
// outputs of one row.
//
// Packed weights: [ceil(N / 16)][ceil(K / 64)][lane][16 bytes], one 1 KiB operand
// after the other as a wave reads them, zeros past K and N.  Past K an activation
// is read from the row's last 16 values instead, and meets a zero.
#include "common.h"

namespace nvfp4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
constexpr int kI8Step = 64;                // k of an operand
constexpr int kI8Bytes = 16 * kI8Step;     // bytes of an operand
constexpr int kI8MaxSplit = 16;            // waves over K

inline int i8_steps(int K) { return (K + kI8Step - 1) / kI8Step; }
inline int i8_tiles(int N) { return (N + 15) / 16; }
inline bool i8_shape(int K, int N) { return K >= 16 && K % 16 == 0 && K <= NVFP4_INT8_MAX_K && N >= 1; }

// One 16-byte piece a thread; UNPACK: the other way, and no padding.
template <bool UNPACK>
__global__ __launch_bounds__(256) void int8_pack_kernel(const int8_t* __restrict__ from, int8_t* __restrict__ to, int K, int N,
                                                        int steps, long long pieces) {
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (long long)gridDim.x * 256) {
        const int lane = (int)(i & 63);
        const long long op = i >> 6;
        const int tile = (int)(op / steps), step = (int)(op - (long long)tile * steps);
        const long long n = (long long)tile * 16 + (lane & 15);
        const int k = step * kI8Step + 16 * (lane >> 4);
        const bool real = n < N && k < K;
        if (UNPACK) {
            if (real) *(uint4*)(to + n * K + k) = *(const uint4*)(from + i * 16);
        } else {
            *(uint4*)(to + i * 16) = real ? *(const uint4*)(from + n * K + k) : make_uint4(0, 0, 0, 0);
        }
    }
}

struct I8Args {
    const int8_t* a;
    const float* a_scale;
    const int8_t* w;
    const float* w_scale;
    const float* bias;
    void* out;
    long long a_ld, out_ld;
    int M, K, N, steps, tiles;
    int vec;  // outputs are stored four at a time
};

__device__ __forceinline__ uint32_t i8_bf16(float x) {
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// Four outputs of row m from n on.
template <bool BF16>
__device__ __forceinline__ void i8_store(const I8Args& p, int m, int n, i32x4 acc) {
    if (m >= p.M || n >= p.N) return;
    const float as = p.a_scale[m];
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int c = min(n + r, p.N - 1);
        y[r] = (float)acc[r] * as * p.w_scale[c];
        if (p.bias) y[r] += p.bias[c];
    }
    const long long at = (long long)m * p.out_ld + n;
    if (p.vec && n + 4 <= p.N) {
        if (BF16)
            *(uint2*)((uint16_t*)p.out + at) = make_uint2(i8_bf16(y[0]) | i8_bf16(y[1]) << 16, i8_bf16(y[2]) | i8_bf16(y[3]) << 16);
        else
            *(float4*)((float*)p.out + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (n + r < p.N) {
                if (BF16)
                    ((uint16_t*)p.out)[at + r] = (uint16_t)i8_bf16(y[r]);
                else
                    ((float*)p.out)[at + r] = y[r];
            }
    }
}

// Up to 16 G rows: a workgroup takes C column tiles over all of K, its waves
// splitting K and adding in LDS.
template <int G, int C, bool BF16>
__global__ __launch_bounds__(1024) void int8_stream_kernel(I8Args p) {
    constexpr int U = 4;  // steps a wave has in flight
    extern __shared__ i32x4 sums[];  // [wave][C][G][lane]
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const int tile0 = blockIdx.x * C, row0 = blockIdx.y * 16 * G;
    const int s0 = (int)((long long)p.steps * wave / waves), s1 = (int)((long long)p.steps * (wave + 1) / waves);
    const int8_t* w[C];
    const int8_t* a[G];
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = p.w + (long long)min(tile0 + c, p.tiles - 1) * p.steps * kI8Bytes + 16 * lane;
#pragma unroll
    for (int g = 0; g < G; ++g) a[g] = p.a + (long long)min(row0 + 16 * g + (lane & 15), p.M - 1) * p.a_ld;
    const int k0 = 16 * (lane >> 4), kmax = p.K - 16;
    i32x4 acc[C][G] = {};
    for (int s = s0; s < s1; s += U) {
        u32x4 wv[U][C], av[U][G];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = min(s + u, s1 - 1);
#pragma unroll
            for (int c = 0; c < C; ++c) wv[u][c] = __builtin_nontemporal_load((const u32x4*)(w[c] + (long long)t * kI8Bytes));
#pragma unroll
            for (int g = 0; g < G; ++g) av[u][g] = *(const u32x4*)(a[g] + min(t * kI8Step + k0, kmax));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + u >= s1) break;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int g = 0; g < G; ++g)
                    acc[c][g] = __builtin_amdgcn_mfma_i32_16x16x64_i8((i32x4)wv[u][c], (i32x4)av[u][g], acc[c][g], 0, 0, 0);
        }
    }
    if (waves > 1) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int g = 0; g < G; ++g) sums[((wave * C + c) * G + g) * 64 + lane] = acc[c][g];
        __syncthreads();
        for (int i = wave; i < C * G; i += waves) {
            i32x4 all = sums[i * 64 + lane];
            for (int v = 1; v < waves; ++v) all += sums[(v * C * G + i) * 64 + lane];
            i8_store<BF16>(p, row0 + 16 * (i % G) + (lane & 15), (tile0 + i / G) * 16 + 4 * (lane >> 4), all);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int g = 0; g < G; ++g) i8_store<BF16>(p, row0 + 16 * g + (lane & 15), (tile0 + c) * 16 + 4 * (lane >> 4), acc[c][g]);
    }
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_int8_packed_bytes(int K, int N) {
    if (!i8_shape(K, N)) return 0;
    return (size_t)i8_tiles(N) * i8_steps(K) * kI8Bytes;
}

static int int8_repack(const int8_t* from, const char* from_name, int8_t* to, const char* to_name, int K, int N, bool unpack,
                       void* stream) {
    clear_error();
    if (K < 16 || K % 16 || K > NVFP4_INT8_MAX_K) return set_error(NVFP4_EINVAL, "K: %d is not a multiple of 16 in [16, %d]", K, NVFP4_INT8_MAX_K);
    if (N < 1) return set_error(NVFP4_EINVAL, "N: %d < 1", N);
    if (!from || ((uintptr_t)from & 15)) return set_error(NVFP4_EINVAL, "%s: NULL or not 16-byte aligned", from_name);
    if (!to || ((uintptr_t)to & 15)) return set_error(NVFP4_EINVAL, "%s: NULL or not 16-byte aligned", to_name);
    const int steps = i8_steps(K);
    const long long pieces = (long long)i8_tiles(N) * steps * 64, blocks = (pieces + 255) / 256;
    const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
    if (unpack)
        hipLaunchKernelGGL(int8_pack_kernel<true>, grid, dim3(256), 0, (hipStream_t)stream, from, to, K, N, steps, pieces);
    else
        hipLaunchKernelGGL(int8_pack_kernel<false>, grid, dim3(256), 0, (hipStream_t)stream, from, to, K, N, steps, pieces);
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

int nvfp4_int8_pack(const int8_t* codes_dev, int K, int N, int8_t* packed_dev, void* stream) {
    return int8_repack(codes_dev, "codes", packed_dev, "packed", K, N, false, stream);
}

int nvfp4_int8_unpack(const int8_t* packed_dev, int K, int N, int8_t* codes_dev, void* stream) {
    return int8_repack(packed_dev, "packed", codes_dev, "codes", K, N, true, stream);
}

size_t nvfp4_int8_gemm_workspace_bytes(int M, int K, int N) {
    if (M < 1 || !i8_shape(K, N)) return 0;
    return 0;
}

int nvfp4_int8_gemm(const int8_t* a_dev, int64_t a_ld, const float* a_scale_dev, const int8_t* w_packed_dev,
                    const float* w_scale_dev, const float* bias_dev, int M, int K, int N, void* out_dev, int out_dtype,
                    int64_t out_ld, void* workspace_dev, size_t workspace_bytes, void* stream) {
    clear_error();
    if (M < 0) return set_error(NVFP4_EINVAL, "M: %d < 0", M);
    if (K < 16 || K % 16 || K > NVFP4_INT8_MAX_K) return set_error(NVFP4_EINVAL, "K: %d is not a multiple of 16 in [16, %d]", K, NVFP4_INT8_MAX_K);
    if (N < 1) return set_error(NVFP4_EINVAL, "N: %d < 1", N);
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return set_error(NVFP4_EINVAL, "out_dtype: %d", out_dtype);
    if (a_ld < K || a_ld % 16) return set_error(NVFP4_EINVAL, "a_ld: %lld is not a multiple of 16 of at least K = %d", (long long)a_ld, K);
    if (out_ld < N) return set_error(NVFP4_EINVAL, "out_ld: %lld < N = %d", (long long)out_ld, N);
    if (M == 0) return NVFP4_OK;
    const bool bf16 = out_dtype == NVFP4_OUT_BF16;
    if (!a_dev || ((uintptr_t)a_dev & 15)) return set_error(NVFP4_EINVAL, "a: NULL or not 16-byte aligned");
    if (!a_scale_dev || ((uintptr_t)a_scale_dev & 3)) return set_error(NVFP4_EINVAL, "a_scale: NULL or not 4-byte aligned");
    if (!w_packed_dev || ((uintptr_t)w_packed_dev & 15)) return set_error(NVFP4_EINVAL, "w_packed: NULL or not 16-byte aligned");
    if (!w_scale_dev || ((uintptr_t)w_scale_dev & 3)) return set_error(NVFP4_EINVAL, "w_scale: NULL or not 4-byte aligned");
    if ((uintptr_t)bias_dev & 3) return set_error(NVFP4_EINVAL, "bias: not 4-byte aligned");
    if (!out_dev || ((uintptr_t)out_dev & (bf16 ? 1 : 3))) return set_error(NVFP4_EINVAL, "out: NULL or not aligned to its type");
    const size_t need = nvfp4_int8_gemm_workspace_bytes(M, K, N);
    if (workspace_bytes < need) return set_error(NVFP4_EINVAL, "workspace_bytes: %zu < %zu needed", workspace_bytes, need);
    if (need && (!workspace_dev || ((uintptr_t)workspace_dev & 15))) return set_error(NVFP4_EINVAL, "workspace: NULL or not 16-byte aligned");
    I8Args p;
    p.a = a_dev;
    p.a_scale = a_scale_dev;
    p.w = w_packed_dev;
    p.w_scale = w_scale_dev;
    p.bias = bias_dev;
    p.out = out_dev;
    p.a_ld = a_ld;
    p.out_ld = out_ld;
    p.M = M;
    p.K = K;
    p.N = N;
    p.steps = i8_steps(K);
    p.tiles = i8_tiles(N);
    p.vec = ((uintptr_t)out_dev & (bf16 ? 7 : 15)) == 0 && out_ld % 4 == 0;
    const hipStream_t s = (hipStream_t)stream;
    const int g = M <= 16 ? 1 : M <= 32 ? 2 : 4, c = g;
    const int groups = (p.tiles + c - 1) / c, rows = (M + 16 * g - 1) / (16 * g);
    int waves = 4;
    while (waves < kI8MaxSplit && (long long)groups * waves < 4096 && p.steps >= 8 * waves && waves * c * g < 64) waves *= 2;
    if (waves > p.steps) waves = p.steps;
    const dim3 grid((unsigned)groups, (unsigned)rows), block(64 * waves);
    const size_t lds = (size_t)waves * c * g * 1024;
#define NVFP4_STREAM(G, B)                                                                            \
    if (g == G && bf16 == B) hipLaunchKernelGGL((int8_stream_kernel<G, G, B>), grid, block, lds, s, p);
    NVFP4_STREAM(1, false)
    NVFP4_STREAM(1, true)
    NVFP4_STREAM(2, false)
    NVFP4_STREAM(2, true)
    NVFP4_STREAM(4, false)
    NVFP4_STREAM(4, true)
#undef NVFP4_STREAM
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

}  // extern "C"
