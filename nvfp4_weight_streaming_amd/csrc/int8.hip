// The product of 8-bit rows and 8-bit weights.
//
//   out[m][n] = float(sum_k a[m][k] w[n][k]) * a_scale[m] * w_scale[n] + bias[n]
//
// v_mfma_i32_16x16x64_i8 takes both operands as 16 bytes a lane (lane l: row or
// column l % 16, 16 values of k from 16 * (l / 16)) and adds in 32 bits, exactly.
// The weights are its first operand, so that a lane ends with four consecutive
// outputs of one row.
//
// Packed weights lie one 1 KiB operand after the other as a wave reads them, zeros
// past K and N.  What is read of a row past K (the next row, or zeros past the last) meets a zero.
//
// Up to 16 rows, and up to 32 of some K and N, the weights are streamed (here): 16 rows of 5120 x 152064 take 129 us here and 140 as
// tiles on the matrix cores (int8_tile.hip), 8 of 5120 x 34816 28.8 and 41, 1 of 5120 x 7168 8.8 and 10.4.  Tiles take all else:
// more rows, 5 to 16 rows of a long K with few columns, and any number of rows of a K above 20480, whose part a wave could not hold.
#include "int8_device.h"

namespace nvfp4 {

constexpr int kI8MaxSplit = 16;    // waves over K
constexpr int kI8MaxRows = 1 << 22;

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

// G groups of 16 rows: the weights are streamed once.  The waves of a workgroup split K, and each holds the
// rows' part of its own steps (NP at most) in registers for all of the column tiles that the workgroup takes, one after
// the other; the waves' sums meet in LDS.  A wave has U steps of weights in flight, those of the
// next tile behind those of this one.
//
// (Read anew for each tile, rows cost as much of the vector cache's time as weights: 8 rows of 5120 x 34816 took
// 35.0 us, and 29.2 with one load of them.)
template <int NP, int U, int G, bool BF16>
__global__ __launch_bounds__(1024) void int8_stream_kernel(I8Args p) {
    static_assert(NP % U == 0, "a step of any tile has one place");
    extern __shared__ i32x4 sums[];  // [2][wave][G][lane]
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int waves = blockDim.x >> 6;
    const int s0 = p.steps * wave / waves, n = p.steps * (wave + 1) / waves - s0;
    const int row = lane & 15, quarter = lane >> 4;
    // Steps past the wave's last one are read past the end of what their resource covers: zeros, with no
    // branch and no traffic.
    const __amdgpu_buffer_rsrc_t ra = i8_rsrc(p.a, (long long)(p.M - 1) * p.a_ld + p.K);
    u32x4 av[G][NP], wv[U];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const int at = min(16 * g + row, p.M - 1) * (int)p.a_ld + s0 * kI8Step + 16 * quarter;
#pragma unroll
        for (int i = 0; i < NP; ++i) av[g][i] = i8_load<0>(ra, i < n ? at + i * kI8Step : 0x7FFFFFFF);
    }
    const long long stride = (long long)p.steps * kI8Bytes;
    const int8_t* w = p.w + blockIdx.x * stride + s0 * kI8Bytes;
    const long long jump = gridDim.x * stride;
    __amdgpu_buffer_rsrc_t rw = i8_rsrc(w, n * kI8Bytes);
#pragma unroll
    for (int i = 0; i < U; ++i) wv[i] = i8_load<kI8Stream>(rw, 16 * lane + i * kI8Bytes);
    int turn = 0, half = 0;  // the first wave that stores the tile's outputs (each a group of rows), and their place in LDS
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        w += jump;
        const __amdgpu_buffer_rsrc_t next = i8_rsrc(w, tile + (int)gridDim.x < p.tiles ? n * kI8Bytes : 0);
        const int c = tile * 16 + 4 * quarter;
        const int mine = wave < turn ? wave - turn + waves : wave - turn;
        float ws[4], bias[4], as = 0.f;
        if (mine < G) {
            as = p.a_scale[min(16 * mine + row, p.M - 1)];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                ws[r] = p.w_scale[min(c + r, p.N - 1)];
                bias[r] = p.bias ? p.bias[min(c + r, p.N - 1)] : 0.f;
            }
        }
        i32x4 acc[G] = {};
#pragma unroll
        for (int i = 0; i < NP; ++i) {
#pragma unroll
            for (int g = 0; g < G; ++g) acc[g] = __builtin_amdgcn_mfma_i32_16x16x64_i8((i32x4)wv[i % U], (i32x4)av[g][i], acc[g], 0, 0, 0);
            wv[i % U] = i8_load<kI8Stream>(i + U < NP ? rw : next, 16 * lane + (i + U) % NP * kI8Bytes);
        }
        rw = next;
#pragma unroll
        for (int g = 0; g < G; ++g) sums[((half * waves + wave) * G + g) * 64 + lane] = acc[g];
        // (no fence, which would wait for the weights in flight; the wait stands between two points that no access to
        // memory is moved across, as its counter is of the sums above)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (mine < G) {
            const i32x4* from = sums + (half * waves * G + mine) * 64 + lane;
            i32x4 all = from[0];
            for (int v = 1; v < waves; ++v) all += from[v * G * 64];
            i8_store_scaled<BF16>(p, 16 * mine + row, c, all, as, ws, bias);
        }
        turn += G;
        if (turn >= waves) turn -= waves;
        half ^= 1;
    }
}

template <int NP, int U, int G>
static int launch_stream(const I8Args& p, bool bf16, int waves, hipStream_t s) {
    // As many workgroups as the device holds at once, or one for each tile.
    const int room = device_cus() * (16 / waves);
    const dim3 grid((unsigned)(p.tiles < room ? p.tiles : room)), block(64 * waves);
    const size_t lds = (size_t)2 * waves * G * 64 * sizeof(i32x4);
    if (bf16)
        hipLaunchKernelGGL((int8_stream_kernel<NP, U, G, true>), grid, block, lds, s, p);
    else
        hipLaunchKernelGGL((int8_stream_kernel<NP, U, G, false>), grid, block, lds, s, p);
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

// Steps a wave, at most.
constexpr int kI8MaxSteps = 20;
// Of 5 to 16 rows, those of more than 12 steps a wave are streamed where workgroups have more than 1.25 tiles on average: with
// few, a wave first waits for its rows and then, 4 steps at a time, for its one tile. 16 rows of 17408 x 5120 take 23.5 us
// here and 20.5 as tiles, of 20480 x 2048 18.3 and 11.8, 8 of 17408 x 2048 13.3 and 10.7; 16 of 17408 x 7168 25.3 and 26.5, 1 of 17408 x
// 5120 19.6 and 20.5, 8 of 12288 x 2048 9.3 and 9.8.
// 17 to 32 rows are streamed where a wave has 5 to 8 steps of them and each workgroup two tiles or more: 32 rows of
// 5120 x 34816 take 34.0 us here and 44.9 as tiles, of 8192 x 100000 139 and 161, 20 of 5120 x 12288 14.3 and 18.9; inside the rule
// 32 of 5120 x 65536 lose 2%, 58.5 and 57.3. With fewer tiles or steps they would be slower: 32 of 5120 x 5120 11.9 and 10.2, of
// 2048 x 17408 13.1 and 8.3. (64 rows, four groups of 5 steps: 64 x 5120 x 34816 42 and 51, x 17408 26.5 and 24.3,
// 1024 x 32000 14.8 and 8.7.)
static bool int8_streams(int M, int K, int N) {
    const int steps = i8_steps(K);
    if (M <= 16 && (M <= 4 || steps <= 12 * kI8MaxSplit || 4ll * i8_tiles(N) > 5ll * device_cus())) return steps <= kI8MaxSplit * kI8MaxSteps;
    return M > 16 && M <= 32 && steps > 4 * kI8MaxSplit && steps <= 8 * kI8MaxSplit && i8_tiles(N) >= 2 * device_cus();
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
    if (N < 1 || N > (1 << 30)) return set_error(NVFP4_EINVAL, "N: %d outside [1, 2^30]", N);
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
    if (M < 1 || M > kI8MaxRows || !i8_shape(K, N)) return 0;
    return int8_streams(M, K, N) ? 0 : int8_tile_ws(M, K, N);
}

int nvfp4_int8_gemm(const int8_t* a_dev, int64_t a_ld, const float* a_scale_dev, const int8_t* w_packed_dev,
                    const float* w_scale_dev, const float* bias_dev, int M, int K, int N, void* out_dev, int out_dtype,
                    int64_t out_ld, void* workspace_dev, size_t workspace_bytes, void* stream) {
    clear_error();
    if (M < 0) return set_error(NVFP4_EINVAL, "M: %d < 0", M);
    if (K < 16 || K % 16 || K > NVFP4_INT8_MAX_K) return set_error(NVFP4_EINVAL, "K: %d is not a multiple of 16 in [16, %d]", K, NVFP4_INT8_MAX_K);
    if (N < 1 || N > (1 << 30)) return set_error(NVFP4_EINVAL, "N: %d outside [1, 2^30]", N);
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return set_error(NVFP4_EINVAL, "out_dtype: %d", out_dtype);
    if (M > kI8MaxRows) return set_error(NVFP4_EINVAL, "M: %d > 2^22", M);
    if (a_ld < K || a_ld % 16 || a_ld > (1 << 22)) return set_error(NVFP4_EINVAL, "a_ld: %lld is not a multiple of 16 in [K = %d, 2^22]", (long long)a_ld, K);
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
    p.wide = ((uintptr_t)out_dev & 15) == 0 && out_ld % (bf16 ? 8 : 4) == 0;
    const hipStream_t s = (hipStream_t)stream;
    if (!int8_streams(M, K, N)) return launch_int8_tile(p, bf16, workspace_dev, s);
    // Four to eight steps a wave, where 16 waves are enough for that: 8 x 5120 x 152064 takes 121 us
    // with 16 waves of 5 steps, 127 with 4 of 20; 8 x 1024 x 100000 18.4 with 4 of 4, 32 with 16 of 1. And
    // waves for every compute unit, where there are few tiles.
    int waves = 4;
    while (waves < kI8MaxSplit && (p.steps > 8 * waves || ((long long)p.tiles * waves < 4096 && p.steps >= 8 * waves))) waves *= 2;
    if (waves > p.steps) waves = p.steps;
    const int most = (p.steps + waves - 1) / waves;
    if (M > 16) return launch_stream<8, 8, 2>(p, bf16, waves, s);
    if (most <= 4) return launch_stream<4, 4, 1>(p, bf16, waves, s);
    if (most <= 8) return launch_stream<8, 8, 1>(p, bf16, waves, s);
    if (most <= 12) return launch_stream<12, 4, 1>(p, bf16, waves, s);
    return launch_stream<20, 4, 1>(p, bf16, waves, s);
}

}  // extern "C"
