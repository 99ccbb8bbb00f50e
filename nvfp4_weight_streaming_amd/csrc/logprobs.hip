// Log probabilities of given tokens, the entropy, and the best tokens with theirs.
//
// For a row of logits x, z = scale * x:
//     logprob(t) = z_t - log sum exp z,   entropy = log sum exp z - sum p z.
// With d = scale (x - m) for a maximum m, S = sum exp d and T = sum d exp(d) / ln 2 carry
// both over any part of a row, and two parts' join by the difference of their maxima.
//
// The first kernel reads the logits once, a wave 4096 of them (all loads in flight at
// once, the maximum before the sums, so nothing is rescaled), and leaves m, S and T of
// each such unit and the maximum of each group of 512 consecutive logits in it.  The
// k best lie in the k best groups: a group's best one is its maximum, the one of a
// lower group going before an equal one, and if k groups have a better one, those k are
// better than everything in it.  The second kernel, a workgroup per row, joins the
// units in fp64, takes the k best groups and rereads only those.
//
// A row need not be aligned: its logits stand at positions p = token + shift, with shift
// the row's offset from a 16-byte boundary; vectors that cross an end of the row are read
// one by one.
#include "select_device.h"

namespace nvfp4 {

constexpr int kLpUnit = 4096;           // logits of a wave
constexpr int kLpGroup = 512;
constexpr int kLpGroups = kLpUnit / kLpGroup;
constexpr int kLpThreads = 256;
constexpr int kLpFew = 256;             // rows that the second kernel gives 1024 threads each
constexpr int kLpList = 1024;           // keys the second kernel ranks at once
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;

struct LpArgs {
    const void* logits;
    long long ld;
    int rows, V, units, n_tokens, k;
    int blocks;  // workgroups of a row in the first kernel
    float scale;
    const int* tokens;
    float4* part;    // [rows][units]: m, S, T
    float* groups;   // [rows][units * 8]
    float* logprob;
    float* entropy;
    int* top_token;
    float* top_logprob;
};

template <bool BF16>
__device__ __forceinline__ int lp_shift(const LpArgs& a, int row) {
    constexpr int S = BF16 ? 2 : 4;
    return (int)(((uintptr_t)a.logits + (uintptr_t)((long long)row * a.ld * S)) & 15) / S;
}
template <bool BF16>
__device__ __forceinline__ float lp_at(const LpArgs& a, int row, int token) {
    const long long i = (long long)row * a.ld + token;
    return BF16 ? __uint_as_float((uint32_t)((const uint16_t*)a.logits)[i] << 16) : ((const float*)a.logits)[i];
}

// The 16 bytes at position p (a multiple of their number); -inf outside the row.
template <bool BF16>
__device__ __forceinline__ void lp_vector(const LpArgs& a, int row, int shift, int p, float (&x)[BF16 ? 8 : 4]) {
    constexpr int W = BF16 ? 8 : 4;
    const int t = p - shift;
    if (t >= 0 && t <= a.V - W) {
        const long long i = (long long)row * a.ld + t;
        if (BF16) {
            const uint4 b = *(const uint4*)((const uint16_t*)a.logits + i);
            const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < W; ++e) x[e] = __uint_as_float(e % 2 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16);
        } else {
            const float4 b = *(const float4*)((const float*)a.logits + i);
            x[0] = b.x, x[1] = b.y, x[2] = b.z, x[3] = b.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) x[e] = t + e >= 0 && t + e < a.V ? lp_at<BF16>(a, row, t + e) : -__builtin_inff();
    }
}

template <bool BF16, bool TOP>
__global__ __launch_bounds__(kLpThreads) void logprobs_scan_kernel(LpArgs a) {
    constexpr int W = BF16 ? 8 : 4, J = kLpUnit / 64 / W;  // vectors of a lane
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int row = blockIdx.x / a.blocks, unit = (blockIdx.x - row * a.blocks) * (kLpThreads / 64) + wave;
    if (unit >= a.units) return;  // whole wave
    const int shift = lp_shift<BF16>(a, row), p0 = unit * kLpUnit;
    float x[J][W];
    if (p0 >= shift && p0 + kLpUnit <= a.V + shift) {
        const char* at = (const char*)a.logits + ((long long)row * a.ld + (p0 - shift)) * (BF16 ? 2 : 4) + 16 * lane;
        uint4 b[J];
#pragma unroll
        for (int j = 0; j < J; ++j) b[j] = *(const uint4*)(at + 1024 * j);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t u[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
#pragma unroll
            for (int e = 0; e < W; ++e)
                x[j][e] = __uint_as_float(!BF16 ? u[e % 4] : e % 2 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16);
        }
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j) lp_vector<BF16>(a, row, shift, p0 + (j * 64 + lane) * W, x[j]);
    }

    // Maxima of the lane's share of each group: one (bf16) or two vectors.
    float g[kLpGroups];
#pragma unroll
    for (int i = 0; i < kLpGroups; ++i) {
        g[i] = x[i * J / kLpGroups][0];
#pragma unroll
        for (int j = i * J / kLpGroups; j < (i + 1) * J / kLpGroups; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) g[i] = fmaxf(g[i], x[j][e]);
    }
    float m = g[0];
#pragma unroll
    for (int i = 1; i < kLpGroups; ++i) m = fmaxf(m, g[i]);
    m = wave_max(m);
    if (TOP) {
        // The wave's maximum of each of the 8: every step halves what a lane holds, until
        // lane l has that of group l % 8 over its 8 lanes.
        const bool b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
        float h[4], q[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = fmaxf(b2 ? g[i + 4] : g[i], dppf<0x141>(b2 ? g[i] : g[i + 4]));  // row_half_mirror: lane ^ 7
#pragma unroll
        for (int i = 0; i < 2; ++i) q[i] = fmaxf(b1 ? h[i + 2] : h[i], dppf<0x4E>(b1 ? h[i] : h[i + 2]));  // lane ^ 2
        float v = fmaxf(b0 ? q[1] : q[0], dppf<0xB1>(b0 ? q[0] : q[1]));                                   // lane ^ 1
        v = fmaxf(v, dppf<0x128>(v));  // row_ror 8: lane ^ 8
        v = fmaxf(v, __shfl_xor(v, 16));
        v = fmaxf(v, __shfl_xor(v, 32));
        if (lane < kLpGroups) a.groups[((long long)row * a.units + unit) * kLpGroups + lane] = v;
    }
    const float use = m == -__builtin_inff() ? 0.f : m, c = a.scale * kLog2e, mc = use * c;
    float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
    // exp(scale (x - m)) as 2^(x c - m c), the product m c rounded: what that loses is the same for every term and
    // put right once.  (The vector units bind here, with 40 cycles a logit of bf16: a difference and a product
    // are one more of 4.)  Large maxima, or scales, take the difference first, of halves: that of two fp32 values may
    // pass fp32.  And they scale it before the constant, whose product with the largest scales is infinite.
    float sum, moment;
    if (fabsf(mc) < 0x1p20f && c > 0x1p-60f && c < 0x1p60f) {
        const float lost = __builtin_fmaf(use, c, -mc);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float z = __builtin_fmaf(x[j][e], c, -mc), p = __builtin_amdgcn_exp2f(z);
                s[e % 4] += p;  // (a NaN stays in it)
                t[e % 4] = __builtin_fmaf(p, fmaxf(z, -3e38f), t[e % 4]);
            }
        const float back = __builtin_amdgcn_exp2f(-lost);
        sum = wave_sum((s[0] + s[1]) + (s[2] + s[3])) * back;
        moment = wave_sum((t[0] + t[1]) + (t[2] + t[3])) * back - lost * sum;
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float z = (0.5f * x[j][e] - 0.5f * use) * a.scale * (2.f * kLog2e), p = __builtin_amdgcn_exp2f(z);
                s[e % 4] += p;
                t[e % 4] = __builtin_fmaf(p, fmaxf(z, -3e38f), t[e % 4]);
            }
        sum = wave_sum((s[0] + s[1]) + (s[2] + s[3]));
        moment = wave_sum((t[0] + t[1]) + (t[2] + t[3]));
    }
    if (lane == 0) a.part[(long long)row * a.units + unit] = make_float4(m, sum, moment, 0.f);
}

// The workgroup's sums of two fp64 values, in all threads.
template <int WAVES>
__device__ __forceinline__ void lp_sums(double& s, double& t, double (*lds)[WAVES]) {
    s = wave_sumd(s);
    t = wave_sumd(t);
    if ((threadIdx.x & 63) == 0) {
        lds[0][threadIdx.x >> 6] = s;
        lds[1][threadIdx.x >> 6] = t;
    }
    __syncthreads();
    s = lds[0][0];
    t = lds[1][0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) {
        s += lds[0][i];
        t += lds[1][i];
    }
}

// THREADS: 1024 for few rows, whose groups are then read by 16 waves at once (the 20 best of 8 rows of 152064: 9.0 us,
// 12.4 with 256 threads); 256 for many (the 8 best of 256 rows: 7.7 us both, of 512 8.9 and 10.8, of 1024 11.0 and 20.8).
template <bool BF16, bool TOP, int THREADS>
__global__ __launch_bounds__(THREADS) void logprobs_finish_kernel(LpArgs a) {
    constexpr int kWaves = THREADS / 64;
    constexpr int W = BF16 ? 8 : 4;
    __shared__ float row_m[kWaves];
    __shared__ double sums[2][kWaves];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int row = blockIdx.x;
    const float4* part = a.part + (long long)row * a.units;
    const int shift = lp_shift<BF16>(a, row), n = (int)(((long long)a.V + shift + kLpGroup - 1) / kLpGroup);
    const float* groups = a.groups + (long long)row * a.units * kLpGroups;

    // What waits for nothing is read first, all at once: a token and its logit, the first unit and the first groups
    // of each thread.
    constexpr int kPer = THREADS / 64, kHeld = 2;
    const int sub = threadIdx.x / kPer, mine = threadIdx.x % kPer * 64 + sub;
    const float4 nothing = make_float4(-__builtin_inff(), 0.f, 0.f, 0.f);
    const long long token_at = (long long)row * a.n_tokens + threadIdx.x;
    const int token0 = (int)threadIdx.x < a.n_tokens ? a.tokens[token_at] : -1;
    const float4 part0 = (int)threadIdx.x < a.units ? part[threadIdx.x] : nothing;
    float held[kHeld];
    if (TOP)
#pragma unroll
        for (int c = 0; c < kHeld; ++c) held[c] = mine + c * THREADS < n ? groups[mine + c * THREADS] : 0.f;
    const float logit0 = token0 >= 0 && token0 < a.V ? lp_at<BF16>(a, row, token0) : -__builtin_inff();

    // The row's maximum, then its sums about it.
    float m = part0.x;
    for (int i = threadIdx.x + THREADS; i < a.units; i += THREADS) m = fmaxf(m, part[i].x);
    m = wave_max(m);
    if (lane == 0) row_m[wave] = m;
    __syncthreads();
    m = row_m[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) m = fmaxf(m, row_m[i]);
    double s = 0.0, t = 0.0;
    for (int i = threadIdx.x; i < a.units; i += THREADS) {
        const float4 p = i < THREADS ? part0 : part[i];
        if (p.x == -__builtin_inff()) {
            s += p.y;  // 0, or NaN
        } else {
            const double d = a.scale * ((double)p.x - (double)m), f = exp(d);
            s += f * p.y;
            if (f > 0) t += f * (kLn2 * p.z + d * p.y);
        }
    }
    lp_sums<kWaves>(s, t, sums);
    const double z = log(s);
    const bool none = s == 0.0;  // every logit is -inf
    auto logprob = [&](float x) -> float {
        if (x == -__builtin_inff() && s == s) return x;
        return (float)((double)a.scale * ((double)x - (double)m) - z);
    };
    if (threadIdx.x == 0 && a.entropy) a.entropy[row] = none ? 0.f : (float)(z - t / s);
    for (int i = threadIdx.x; i < a.n_tokens; i += THREADS) {
        const long long at = (long long)row * a.n_tokens + i;
        const int token = i < THREADS ? token0 : a.tokens[at];
        const bool real = token >= 0 && token < a.V;
        a.logprob[at] = real ? logprob(i < THREADS ? logit0 : lp_at<BF16>(a, row, token)) : -__builtin_inff();
    }
    if (!TOP) return;

    __shared__ u64 list[kLpList];
    __shared__ u64 best[64], tops[64], bar;
    __shared__ int counts[2];
    if (threadIdx.x < 2) counts[threadIdx.x] = 0;
    auto key_of = [&](int i, float v) -> u64 { return i < n ? topk_key(v, max(0, i * kLpGroup - shift)) : 0; };
    auto group_key = [&](int i) -> u64 { return i < n ? key_of(i, groups[i]) : 0; };

    // The k best groups: what passes a bar that at least k pass is ranked.  The bar is
    // the k-th largest of 64 maxima, each over the groups of `kPer` threads; threads kPer
    // apart take neighbouring groups, as the best of a row may lie together.
    u64 head = 0;
#pragma unroll
    for (int c = 0; c < kHeld; ++c) head = max64(head, key_of(mine + c * THREADS, held[c]));
    for (int i = mine + kHeld * THREADS; i < n; i += THREADS) head = max64(head, group_key(i));
    head = max64(head, dpp64<0xB1>(head));
    head = max64(head, dpp64<0x4E>(head));
    if (kPer == 16) {
        head = max64(head, dpp64<0x141>(head));
        head = max64(head, dpp64<0x140>(head));
    }
    if (lane % kPer == 0) tops[sub] = head;
    if (threadIdx.x == 0) bar = 1;  // fewer than k: all
    __syncthreads();
    int above = 0;
#pragma unroll
    for (int j = 0; j < 64 / kPer; ++j) above += tops[64 / kPer * (lane % kPer) + j] > head ? 1 : 0;
    above += dppi<0xB1>(above);
    above += dppi<0x4E>(above);
    if (kPer == 16) {
        above += dppi<0x141>(above);
        above += dppi<0x140>(above);
    }
    if (above == a.k - 1 && head) bar = head;  // (distinct keys: one sub)
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
        const u64 key = key_of(mine + c * THREADS, held[c]);
        append_keys<kLpList>(key, key && key >= bar, list, &counts[0], lane);
    }
    for (int i0 = kHeld * THREADS; i0 < n; i0 += THREADS) {
        const u64 key = group_key(i0 + mine);
        append_keys<kLpList>(key, key && key >= bar, list, &counts[0], lane);
    }
    __syncthreads();
    auto join = [&](u64 kept) {  // the waves' sorted lists to best[]
        list[wave * 64 + lane] = lane < a.k ? kept : 0;
        __syncthreads();
        if (wave == 0) {
            u64 x[kWaves];
#pragma unroll
            for (int j = 0; j < kWaves; ++j) x[j] = list[j * 64 + lane];
            best[lane] = wave_keep<kWaves>(0, x, a.k, lane);
        }
        __syncthreads();
    };
    if (counts[0] <= kLpList) {
        rank_keys<THREADS>(list, counts[0], a.k, best);
        __syncthreads();
    } else {  // too many pass (over half a million logits): the waves insert them one by one
        __syncthreads();
        u64 kept = 0;
        for (int i0 = 0; i0 < n; i0 += THREADS) {
            const u64 key = group_key(i0 + threadIdx.x);
            kept = wave_insert(kept, key, key != 0, a.k, lane);
        }
        join(kept);
    }

    // Their logits: none below the last group's best one can be listed.
    const u64 last = best[a.k - 1];
    const u64 floor = last ? ((last >> 32) << 32) | (unsigned int)((unsigned int)last - (kLpGroup - 1)) : 1;
    auto for_candidates = [&](auto&& f) {
        // (two groups of a wave at a time, read before either is looked at)
        for (int q = wave; q < a.k; q += 2 * kWaves) {
            constexpr int kV = kLpGroup / 64 / W;
            float x[2][kV][W];
            int first[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const u64 key = q + g * kWaves < a.k ? best[q + g * kWaves] : 0;
                first[g] = key ? ((int)~(unsigned int)key + shift) / kLpGroup * kLpGroup : -1;
                if (first[g] >= 0)
#pragma unroll
                    for (int j = 0; j < kV; ++j) lp_vector<BF16>(a, row, shift, first[g] + (j * 64 + lane) * W, x[g][j]);
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (first[g] < 0) continue;
#pragma unroll
                for (int j = 0; j < kV; ++j)
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const int token = first[g] + (j * 64 + lane) * W - shift + e;
                        f(token >= 0 && token < a.V ? topk_key(x[g][j][e], token) : 0);
                    }
            }
        }
    };
    for_candidates([&](u64 key) { append_keys<kLpList>(key, key && key >= floor, list, &counts[1], lane); });
    __syncthreads();
    if (counts[1] <= kLpList) {
        __shared__ u64 winners[64];
        rank_keys<THREADS>(list, counts[1], a.k, winners);
        __syncthreads();
        if (threadIdx.x < 64) best[threadIdx.x] = winners[threadIdx.x];
        __syncthreads();
    } else {  // many equal logits, or fewer groups than k
        __syncthreads();
        u64 kept = 0;
        for_candidates([&](u64 key) { kept = wave_insert(kept, key, key && key >= floor, a.k, lane); });
        join(kept);
    }
    if ((int)threadIdx.x < a.k) {
        const u64 key = best[threadIdx.x];
        // (a NaN among the logits can leave a place empty: token 0)
        const int token = key ? (int)~(unsigned int)key : 0;
        const unsigned int o = (unsigned int)(key >> 32);
        const long long at = (long long)row * a.k + threadIdx.x;
        a.top_token[at] = token;
        a.top_logprob[at] = logprob(__uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o));
    }
}

// Units of a row whose first logit is up to 7 past a 16-byte boundary.
long long lp_units(int V) { return ((long long)V + 7 + kLpUnit - 1) / kLpUnit; }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_logprobs_workspace_bytes(int rows, int V, int k) {
    if (rows < 1 || V < 1 || V > (1 << 30) || k < 0 || k > NVFP4_TOPK_MAX_K || k > V) return 0;
    return (size_t)rows * lp_units(V) * (sizeof(float4) + (k ? kLpGroups * sizeof(float) : 0));
}

int nvfp4_logprobs(const void* logits_dev, int logits_dtype, int64_t ld, int rows, int V, float scale, const int* tokens_dev,
                   int n_tokens, int k, float* logprob_dev, float* entropy_dev, int* top_token_dev, float* top_logprob_dev,
                   void* workspace_dev, size_t workspace_bytes, void* stream) {
    clear_error();
    if (logits_dtype != NVFP4_OUT_F32 && logits_dtype != NVFP4_OUT_BF16)
        return set_error(NVFP4_EINVAL, "logits_dtype: %d", logits_dtype);
    if (V < 1 || V > (1 << 30)) return set_error(NVFP4_EINVAL, "V: %d outside [1, 2^30]", V);
    const long long units = lp_units(V), blocks = (units + kLpThreads / 64 - 1) / (kLpThreads / 64);
    const int most = (int)(0xFFFFFFFFll / kLpThreads / blocks);  // a launch has fewer than 2^32 threads
    if (rows < 0 || rows > most) return set_error(NVFP4_EINVAL, "rows: %d outside [0, %d]", rows, most);
    if (ld < V) return set_error(NVFP4_EINVAL, "ld: %lld < V = %d", (long long)ld, V);
    if (!(scale > 0.f) || scale == __builtin_inff()) return set_error(NVFP4_EINVAL, "scale: %g is not finite and above 0", scale);
    if (n_tokens < 0 || n_tokens > 1024) return set_error(NVFP4_EINVAL, "n_tokens: %d outside [0, 1024]", n_tokens);
    if (k < 0 || k > NVFP4_TOPK_MAX_K || k > V)
        return set_error(NVFP4_EINVAL, "k: %d outside [0, min(V, %d)]", k, NVFP4_TOPK_MAX_K);
    if (rows == 0) return NVFP4_OK;
    const bool bf16 = logits_dtype == NVFP4_OUT_BF16;
    if (!logits_dev || ((uintptr_t)logits_dev & (bf16 ? 1 : 3)))
        return set_error(NVFP4_EINVAL, "logits: NULL or not aligned to its type");
    if (n_tokens && (!tokens_dev || ((uintptr_t)tokens_dev & 3))) return set_error(NVFP4_EINVAL, "tokens: NULL or not 4-byte aligned");
    if (n_tokens && (!logprob_dev || ((uintptr_t)logprob_dev & 3))) return set_error(NVFP4_EINVAL, "logprob: NULL or not 4-byte aligned");
    if ((uintptr_t)entropy_dev & 3) return set_error(NVFP4_EINVAL, "entropy: not 4-byte aligned");
    if (k && (!top_token_dev || ((uintptr_t)top_token_dev & 3))) return set_error(NVFP4_EINVAL, "top_token: NULL or not 4-byte aligned");
    if (k && (!top_logprob_dev || ((uintptr_t)top_logprob_dev & 3)))
        return set_error(NVFP4_EINVAL, "top_logprob: NULL or not 4-byte aligned");
    const size_t need = nvfp4_logprobs_workspace_bytes(rows, V, k);
    if (workspace_bytes < need) return set_error(NVFP4_EINVAL, "workspace_bytes: %zu < %zu needed", workspace_bytes, need);
    if (!workspace_dev || ((uintptr_t)workspace_dev & 15)) return set_error(NVFP4_EINVAL, "workspace: NULL or not 16-byte aligned");
    LpArgs a;
    a.logits = logits_dev;
    a.ld = ld;
    a.rows = rows;
    a.V = V;
    a.units = (int)units;
    a.n_tokens = n_tokens;
    a.k = k;
    a.blocks = (int)blocks;
    a.scale = scale;
    a.tokens = tokens_dev;
    a.part = (float4*)workspace_dev;
    a.groups = (float*)((float4*)workspace_dev + (size_t)rows * units);
    a.logprob = logprob_dev;
    a.entropy = entropy_dev;
    a.top_token = top_token_dev;
    a.top_logprob = top_logprob_dev;
    const hipStream_t s = (hipStream_t)stream;
    const bool wide = rows <= kLpFew;
#define NVFP4_LOGPROBS(B, T)                                                                                          \
    if (bf16 == B && (k > 0) == T) {                                                                                  \
        hipLaunchKernelGGL((logprobs_scan_kernel<B, T>), dim3((unsigned)(rows * blocks)), dim3(kLpThreads), 0, s, a); \
        NVFP4_HIP(hipGetLastError());                                                                                 \
        if (wide)                                                                                                     \
            hipLaunchKernelGGL((logprobs_finish_kernel<B, T, 1024>), dim3((unsigned)rows), dim3(1024), 0, s, a);      \
        else                                                                                                          \
            hipLaunchKernelGGL((logprobs_finish_kernel<B, T, 256>), dim3((unsigned)rows), dim3(256), 0, s, a);        \
    }
    NVFP4_LOGPROBS(false, false)
    NVFP4_LOGPROBS(false, true)
    NVFP4_LOGPROBS(true, false)
    NVFP4_LOGPROBS(true, true)
#undef NVFP4_LOGPROBS
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

}  // extern "C"
