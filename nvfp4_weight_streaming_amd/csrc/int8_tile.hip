// The 8-bit product in tiles on the matrix cores: of more than 16 rows but for those that are streamed, of 5 to 16 rows of a long
// K with few columns, and of any K above 20480.
//
// A workgroup of four waves takes 32 TI rows x 128 TJ outputs, K in stages of 128; each wave has
// the rows and 32 TJ of the outputs, as TI x TJ products of v_mfma_i32_32x32x32_i8 for each 32 k.
//
// Rows go through LDS, as the four waves share them: a ring of four stages, copied directly, three
// stages ahead.  Each wave reads its own weights straight into registers, one or two stages ahead, in
// the packed order, where a product's operand is two runs of 512 bytes.  Through LDS as well they
// would double what its port carries and halve the workgroups that fit: 128 x 256 outputs (TI = 4, TJ = 2) take 67 KiB
// and half the registers of a compute unit, so that two workgroups share it, and the one's
// products run beside the other's outputs.
//
// LDS rows are 128 bytes, 8 segments of 16; segment s of row r sits in slot s ^ (r / 2) % 8, so that
// the 16 rows of one operand read pass cover all banks once.
#include "int8_device.h"

namespace nvfp4 {

typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kTK = 128;           // k of a stage
constexpr int kTRing = 4;          // stages in LDS
constexpr int kTMaxSplits = 12;    // pieces along K
constexpr int kTMinStages = 4;     // stages of a piece
constexpr int t_stage_bytes(int ti) { return 32 * ti * kTK; }

__device__ __forceinline__ int t_key(int row) { return (row >> 1) & 7; }

// 16 bytes a lane to 1 KiB of LDS.
__device__ __forceinline__ void t_copy(__amdgpu_buffer_rsrc_t from, int8_t* to, int lane_at, int at) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, lane_at, at, 0, 0);
}
// Waits until at most N of the wave's loads and copies are in flight.
template <int N>
__device__ __forceinline__ void t_wait() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// (no fence, which would wait for the copies in flight)
__device__ __forceinline__ void t_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

struct TileNo {
    static constexpr bool value = false;
};
struct TileYes {
    static constexpr bool value = true;
};

// Stages of weights that a wave reads ahead: two where registers are left for them (64 x 5120 x 7168 in 32 x 128
// tiles: 11.9 us, 13.4 one ahead; 64 x 128 tiles gain 1 to 4%).
constexpr int t_ahead(int ti, int tj) { return ti * tj <= 2 ? 2 : 1; }

// Stages u0 .. u1 - 1 of the tile at (m0, n0), added to acc.
template <int TI, int TJ>
__device__ __forceinline__ void tile_sum(i32x16 (&acc)[TI][TJ], int8_t* lds, const I8Args& p, int m0, int n0, int u0, int u1) {
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int r32 = lane & 31, half = lane >> 5;

    // Copies of 1 KiB, TI a wave: 8 rows (those past M read zero), lane i filling slot i % 8 of row i / 8 with
    // the segment that belongs there.
    const int rows = min(32 * TI, p.M - m0);
    const __amdgpu_buffer_rsrc_t ra = i8_rsrc(p.a + (long long)m0 * p.a_ld, (long long)(rows - 1) * p.a_ld + p.K);
    int va[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const int r = (wave * TI + i) * 8 + (lane >> 3);
        va[i] = r * (int)p.a_ld + 16 * ((lane & 7) ^ t_key(r));
    }
    auto copy = [&](int u) {
        int8_t* to = lds + (u & 3) * t_stage_bytes(TI) + wave * TI * 1024;
        const int at = min(u, u1 - 1) * kTK;
#pragma unroll
        for (int i = 0; i < TI; ++i) t_copy(ra, to + i * 1024, va[i], at);
    };

    // Weights: operand (ks, j) of a stage covers channels 32 j .. + 31 of the wave's and k = 32 ks .. + 31.
    const int t0 = n0 / 16;
    const __amdgpu_buffer_rsrc_t rw = i8_rsrc(p.w + (long long)t0 * p.steps * kI8Bytes, (long long)(p.tiles - t0) * p.steps * kI8Bytes);
    int vw[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) vw[j] = ((wave * TJ + j) * 2 + (r32 >> 4)) * p.steps * kI8Bytes + (half * 16 + (lane & 15)) * 16;
    auto load = [&](i32x4 (&w)[4][TJ], int u) {
        const int at = min(u, u1 - 1) * 2 * kI8Bytes;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int j = 0; j < TJ; ++j) w[ks][j] = (i32x4)__builtin_amdgcn_raw_buffer_load_b128(rw, vw[j], at + 512 * ks, 0);
    };

    const int8_t* rows_at = lds + r32 * kTK;
    const int key = t_key(r32);
    auto read = [&](i32x4 (&a)[TI], int u, int ks) {
        const int8_t* from = rows_at + (u & 3) * t_stage_bytes(TI) + 16 * ((2 * ks + half) ^ key);
#pragma unroll
        for (int i = 0; i < TI; ++i) a[i] = *(const i32x4*)(from + 32 * i * kTK);
    };
    auto multiply = [&](const i32x4 (&w)[TJ], const i32x4 (&a)[TI]) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[j], a[i], acc[i][j], 0, 0, 0);
        __builtin_amdgcn_s_setprio(0);
    };
    constexpr int kAhead = t_ahead(TI, TJ);
    i32x4 w[kAhead + 1][4][TJ], a0[TI], a1[TI];
    // (in the order in which stages would have issued them, which the waits below count on)
    copy(u0);
    __builtin_amdgcn_sched_barrier(0);
    load(w[0], u0);
    __builtin_amdgcn_sched_barrier(0);
    copy(u0 + 1);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kAhead == 2) load(w[1], u0 + 1);
    __builtin_amdgcn_sched_barrier(0);
    copy(u0 + 2);
    __builtin_amdgcn_sched_barrier(0);
    t_wait<2 * TI + 4 * TJ * (kAhead - 1)>();
    t_barrier();
    read(a0, u0, 0);

    // The barrier stands in the middle of a stage, so that no wave begins a stage with its operands
    // still to be read.  Behind it, stage u + 1 has landed for every wave, and all have left stage
    // u - 1, whose place the copy of stage u + 3 takes.
    auto stage = [&](int u, const i32x4 (&now)[4][TJ], i32x4 (&later)[4][TJ], auto last) {
        load(later, u + kAhead);
        read(a1, u, 1);
        multiply(now[0], a0);
        read(a0, u, 2);
        multiply(now[1], a1);
        __builtin_amdgcn_sched_barrier(0);
        // What was issued after that copy may be in flight: the next one, the weights above and, two ahead, those
        // before.  In the last stages the weights above are nobody's, and no load: only the next copy is counted on.
        t_wait<TI + (last.value ? 0 : 4 * TJ * kAhead)>();
        t_barrier();
        copy(u + 3);
        __builtin_amdgcn_sched_barrier(0);
        read(a1, u, 3);
        multiply(now[2], a0);
        read(a0, u + 1, 0);
        multiply(now[3], a1);
    };
    int u = u0;
    for (; u + kAhead < u1; u += kAhead + 1) {
#pragma unroll
        for (int i = 0; i <= kAhead; ++i) stage(u + i, w[i], w[(i + kAhead) % (kAhead + 1)], TileNo{});
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (u + i < u1) stage(u + i, w[i], w[(i + kAhead) % (kAhead + 1)], TileYes{});
    // (no copy may land after the workgroup has left its LDS, or in what the outputs are turned in)
    t_wait<0>();
    t_barrier();
}

// The scales and bias of the tile at (m0, n0), after the ring in LDS; thread i's of them, in flight while the
// sums are made.
struct TileScales {
    float row[128], channel[256], bias[256];
};
struct TileScale {
    float row, channel, bias;
};
__device__ __forceinline__ TileScale tile_scale_load(const I8Args& p, int m0, int n0) {
    const int i = threadIdx.x, n = min(n0 + i, p.N - 1);
    return {p.a_scale[min(m0 + i, p.M - 1)], p.w_scale[n], p.bias ? p.bias[n] : 0.f};
}
template <int TI, int TJ>
__device__ __forceinline__ void tile_scale_put(TileScales& s, const TileScale& mine) {
    const int i = threadIdx.x;
    if (i < 32 * TI) s.row[i] = mine.row;
    if (i < 128 * TJ) s.channel[i] = mine.channel, s.bias[i] = mine.bias;
    __syncthreads();
}

// The tile's outputs.  A lane has four consecutive ones of a row in each quarter of a product, lanes
// l and l + 32 eight (bf16 halves of two quarters change places between those lanes); the wave turns 32 rows
// at a time in its share of the ring, so that a store covers whole runs of 32 TJ outputs.  16-byte piece s of
// row r lies in place s ^ r % 8.  (Stored from the products' own layout, 32 bytes of a row at a time,
// the end of a tile of 256 x 256 took 14 us.)
template <int TI, int TJ, bool BF16>
__device__ __forceinline__ void tile_store(const i32x16 (&acc)[TI][TJ], int8_t* lds, int share, const TileScales& sc, const I8Args& p,
                                           int m0, int n0) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5, r32 = lane & 31;
    const int nw = wave * 32 * TJ;
    const bool inside = m0 + 32 * TI <= p.M && n0 + 128 * TJ <= p.N && p.wide;
    int8_t* turn = lds + wave * share;
    constexpr int kRow = (BF16 ? 64 : 128) * TJ;  // bytes of 32 TJ outputs
    constexpr int kAt = kRow / 16;                // pieces of a row
    constexpr int kMask = kAt < 16 ? kAt - 1 : 15;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        const float as = sc.row[32 * i + r32];
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
            float y[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = nw + 32 * j + 8 * q + 4 * half;
                const float4 ws = *(const float4*)&sc.channel[n];
                const float4 b = *(const float4*)&sc.bias[n];
                const float w[4] = {ws.x, ws.y, ws.z, ws.w}, more[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    y[4 * q + r] = i8_value(acc[i][j][4 * q + r], as, w[r]);
                    if (p.bias) y[4 * q + r] = i8_biased(y[4 * q + r], more[r]);
                }
            }
            if (BF16) {
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const uint32_t a0 = i8_bf16x2(y[4 * q], y[4 * q + 1]), a1 = i8_bf16x2(y[4 * q + 2], y[4 * q + 3]);
                    const uint32_t b0 = i8_bf16x2(y[4 * q + 4], y[4 * q + 5]), b1 = i8_bf16x2(y[4 * q + 6], y[4 * q + 7]);
                    const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
                    const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
                    *(uint4*)(turn + r32 * kRow + 16 * ((4 * j + q + half) ^ (r32 & kMask))) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *(float4*)(turn + r32 * kRow + 16 * ((8 * j + 2 * q + half) ^ (r32 & kMask))) =
                        make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
            }
        }
#pragma unroll
        for (int s = 0; s < kAt / 2; ++s) {
            const int r = s * (64 / kAt) + lane / kAt, piece = lane % kAt;
            const uint4 v = *(const uint4*)(turn + r * kRow + 16 * (piece ^ (r & kMask)));
            const int m = m0 + 32 * i + r, n = n0 + nw + piece * (BF16 ? 8 : 4);
            const long long at = (long long)m * p.out_ld + n;
            if (inside || (m < p.M && n + (BF16 ? 8 : 4) <= p.N && p.wide)) {
                *(uint4*)((int8_t*)p.out + at * (BF16 ? 2 : 4)) = v;
            } else if (m < p.M) {
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < (BF16 ? 8 : 4); ++e)
                    if (n + e < p.N) {
                        if (BF16)
                            ((uint16_t*)p.out)[at + e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
                        else
                            ((uint32_t*)p.out)[at + e] = u[e % 4];
                    }
            }
        }
    }
}

// What a launch computes: tiles of 32 TI x 128 TJ, rows first, in `splits` pieces along K each.
struct TilePlan {
    int mblocks, tiles, splits;
    int per_xcd;  // workgroups on one XCD
    i32x4* part;  // pieces: [tile][split][wave][TI][TJ][4][lane]
};

template <int TI, int TJ, bool BF16>
__global__ __launch_bounds__(256, 2) void int8_tile_kernel(I8Args p, TilePlan g) {
    extern __shared__ __attribute__((aligned(16))) int8_t lds[];
    constexpr int kRing = kTRing * t_stage_bytes(TI);
    static_assert(kRing / 4 >= 32 * 128 * TJ, "a wave's share holds 32 rows of fp32 outputs");
    TileScales& scales = *(TileScales*)(lds + kRing);
    // Neighbouring tiles go to one XCD.
    const int w = (blockIdx.x & 7) * g.per_xcd + (blockIdx.x >> 3);
    if (w >= g.tiles * g.splits) return;  // whole workgroup
    const int t = w / g.splits, s = w - t * g.splits;
    const int m0 = t % g.mblocks * 32 * TI, n0 = t / g.mblocks * 128 * TJ;
    const int stages = p.steps / 2, u0 = (int)((long long)stages * s / g.splits), u1 = (int)((long long)stages * (s + 1) / g.splits);
    i32x16 acc[TI][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] = i32x16{};
    const TileScale mine = tile_scale_load(p, m0, n0);
    tile_sum<TI, TJ>(acc, lds, p, m0, n0, u0, u1);
    if (g.splits == 1) {
        tile_scale_put<TI, TJ>(scales, mine);
        tile_store<TI, TJ, BF16>(acc, lds, kRing / 4, scales, p, m0, n0);
        return;
    }
    i32x4* part = g.part + (long long)w * (TI * TJ * 1024) + (threadIdx.x >> 6) * (TI * TJ * 256) + (threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                part[((i * TJ + j) * 4 + q) * 64] = i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
}

// The pieces' sums and the outputs, four a thread, all pieces in flight at once (those past the last read zero).
template <int TI, int TJ, bool BF16>
__global__ __launch_bounds__(256) void int8_join_kernel(I8Args p, TilePlan g) {
    constexpr int kTile = TI * TJ * 1024, kBlocks = kTile / 256;  // groups of four; workgroups of a tile
    const int t = blockIdx.x / kBlocks, at = blockIdx.x % kBlocks * 256 + threadIdx.x;
    const int lane = at & 63, q = at >> 6 & 3, j = at / 256 % TJ, k = at / (256 * TJ) % TI, wave = at / (256 * TI * TJ);
    const int m = t % g.mblocks * 32 * TI + 32 * k + (lane & 31);
    const int n = t / g.mblocks * 128 * TJ + wave * 32 * TJ + 32 * j + 8 * q + 4 * (lane >> 5);
    if (m >= p.M || n >= p.N) return;
    const __amdgpu_buffer_rsrc_t from = i8_rsrc(g.part + (long long)t * g.splits * kTile, (long long)g.splits * kTile * 16);
    u32x4 piece[kTMaxSplits];
#pragma unroll
    for (int s = 0; s < kTMaxSplits; ++s) piece[s] = i8_load<0>(from, (s * kTile + at) * 16);
    float ws[4], bias[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int c = min(n + r, p.N - 1);
        ws[r] = p.w_scale[c];
        bias[r] = p.bias ? p.bias[c] : 0.f;
    }
    i32x4 sum = (i32x4)piece[0];
#pragma unroll
    for (int s = 1; s < kTMaxSplits; ++s) sum += (i32x4)piece[s];
    i8_store_scaled<BF16>(p, m, n, sum, p.a_scale[m], ws, bias);
}

// Which tiles, and in how many pieces along K: the fewest microseconds by what was measured. A stage of one tile
// takes `alone` where a compute unit has one of them, and `beside` in each unit's time where it has
// several; pieces cost a second kernel and their sums' way through memory.
// Over 25 shapes (64 < M <= 2048, 512 <= K <= 17408, 256 <= N <= 34816) this comes within 1.6% of the best of
// 50 choices on average, 8% at most (below 64 rows, where memory bounds all of them, 13%: 64 x 5120 x 34816 takes
// 50.6 us in the 32 x 128 tiles chosen, 45 in 128 x 256):
//   2048 x 5120 x 34816   322 us in 128 x 256 tiles, 389 in 128 x 128
//   2048 x 5120 x 5120    60.0 in 128 x 128, 72.5 in 64 x 128
//   256 x 5120 x 7168     15.3 in 64 x 128, 18.9 in 32 x 128, 20.9 in 128 x 128
//   128 x 17408 x 5120    27.3 in 6 pieces of 128 x 128, 79.6 in one
struct TileChoice {
    int ti, tj, splits;
};
struct TileCost {
    int ti, tj;
    float alone, beside;
};
constexpr TileCost kTileCosts[] = {{4, 2, 0.80f, 0.84f}, {4, 1, 0.47f, 0.47f}, {2, 1, 0.33f, 0.34f}, {1, 1, 0.26f, 0.25f}};

static TileChoice choose_tile(int M, int K, int N) {
    const int cus = device_cus(), stages = i8_steps(K) / 2;
    TileChoice best = {0, 0, 0};
    double least = 0;
    for (const TileCost& c : kTileCosts) {
        const double tiles = (double)((M + 32 * c.ti - 1) / (32 * c.ti)) * ((N + 128 * c.tj - 1) / (128 * c.tj));
        for (int s = 1; s <= kTMaxSplits && (s == 1 || (stages >= kTMinStages * s && tiles * s <= 2 * cus)); ++s) {
            const double work = tiles * s, load = work <= cus ? 1 : work <= 2 * cus ? 2 : work / cus + 0.5;
            double us = (stages + s - 1) / s * (load * c.beside > c.alone ? load * c.beside : c.alone);
            if (s > 1) us += 5 + work * c.ti * c.tj * (32 * 128 * 4 * 2) / 4.5e6;
            if (!best.splits || us < least) {
                least = us;
                best = {c.ti, c.tj, s};
            }
        }
    }
    return best;
}

size_t int8_tile_ws(int M, int K, int N) {
    const TileChoice c = choose_tile(M, K, N);
    if (c.splits == 1) return 0;
    const size_t mb = (M + 32 * c.ti - 1) / (32 * c.ti), nb = (N + 128 * c.tj - 1) / (128 * c.tj);
    return mb * nb * c.splits * (size_t)(c.ti * c.tj) * 1024 * sizeof(i32x4);
}

template <int TI, int TJ, bool BF16>
static int launch_tile_t(const I8Args& p, int splits, void* ws, hipStream_t s) {
    TilePlan g;
    g.mblocks = (p.M + 32 * TI - 1) / (32 * TI);
    const long long tiles = (long long)g.mblocks * ((p.N + 128 * TJ - 1) / (128 * TJ));
    if (tiles * splits > (1 << 22)) return set_error(NVFP4_EUNSUPPORTED, "M, N: %d x %d make %lld tiles, more than 2^22", p.M, p.N, tiles);
    g.tiles = (int)tiles;
    g.splits = splits;
    g.per_xcd = (g.tiles * splits + 7) / 8;
    g.part = (i32x4*)ws;
    hipLaunchKernelGGL((int8_tile_kernel<TI, TJ, BF16>), dim3(8 * g.per_xcd), dim3(256), kTRing * t_stage_bytes(TI) + sizeof(TileScales), s,
                       p, g);
    NVFP4_HIP(hipGetLastError());
    if (splits > 1) {
        hipLaunchKernelGGL((int8_join_kernel<TI, TJ, BF16>), dim3(g.tiles * TI * TJ * 4), dim3(256), 0, s, p, g);
        NVFP4_HIP(hipGetLastError());
    }
    return NVFP4_OK;
}

int launch_int8_tile(const I8Args& p, bool bf16, void* ws, hipStream_t s) {
    const TileChoice c = choose_tile(p.M, p.K, p.N);
#define NVFP4_TILE(I, J) \
    if (c.ti == I && c.tj == J) return bf16 ? launch_tile_t<I, J, true>(p, c.splits, ws, s) : launch_tile_t<I, J, false>(p, c.splits, ws, s);
    NVFP4_TILE(4, 2)
    NVFP4_TILE(4, 1)
    NVFP4_TILE(2, 1)
    NVFP4_TILE(1, 1)
#undef NVFP4_TILE
    return NVFP4_OK;
}

}  // namespace nvfp4
