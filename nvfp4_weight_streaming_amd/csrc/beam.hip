// Beam selection: the best continuations over beams and vocabulary.
//
// The step after the output head when a request keeps several beams instead of
// one greedy token ("Ignis" README, "Speculative decoding (DFlash2)" has the
// top-k over the vocabulary as its last step; here its rows are beams that
// compete).  For a row with running score c and logits x,
//     score(v) = c + ((x_v - max) - log sum exp(x - max)),
// and of the beams x V candidates of a request the k best are listed, equal
// scores by ascending row, then token.
//
// The logits are read once.  They are cut into groups of 1024 tokens, and the
// first kernel (two groups a wave, a pure stream) keeps each group's maximum and
// sum of exponentials.  The k best candidates lie in the k best groups: a
// group's best candidate is its maximum, and if k other groups have a better
// one, those k are better than everything in it.  The second kernel, one
// workgroup per request, forms each row's log-sum, takes the k best groups by
// score and rereads only those (at most 64 x 1024 logits).
//
// Measured over 152064 tokens: 128 rows in bf16 (39 MB) scan 11.3 us, 3.5 TB/s: ten vector
// instructions a logit keep the vector units busy for 5 us, and a wave, all of whose loads
// go out at once, has none left to hide behind that work (its waves wait for 63% of their
// time); 4 rows in fp32 3.5.  The second kernel is a chain of small reads and barriers:
// 6.0 us for one request of 4 beams, 8.3 for 16 of 8.
#include "key_device.h"

namespace nvfp4 {

constexpr int kBeamGroup = 1024;
constexpr int kBeamThreads = 256;       // scan: 4 waves
constexpr int kBeamRun = 2;             // groups per wave
constexpr int kBeamPickThreads = 1024;  // pick: 16 waves
constexpr int kBeamList = 1024;        // keys the pick kernel ranks at once

struct BeamArgs {
    const void* logits;
    long long ld;
    int beams, V, k, groups;
    const float* score;
    const uint8_t* done;  // null: none
    int eos;
    float2* part;  // [rows][groups] maximum, sum of exp(x - maximum)
    float* score_out;
    int* parent_out;
    int* token_out;
    uint8_t* done_out;
};

// How a row's logits are taken: as they are; a finished row has one candidate
// (its end token at its own score); a row with score -inf has none.
enum { kRowLive = 0, kRowDone = 1, kRowDead = 2 };
__device__ __forceinline__ int row_state(const BeamArgs& a, int row) {
    if (a.score[row] == -__builtin_inff()) return kRowDead;
    return a.done && a.done[row] ? kRowDone : kRowLive;
}

__device__ __forceinline__ float bf16_up(uint32_t h) { return __uint_as_float(h << 16); }

// Token of the lane's element e of a group (vector loads: 4 or 8 in a row).
template <bool BF16, bool VEC>
__device__ __forceinline__ int token_of(int group, int lane, int e) {
    constexpr int W = VEC ? (BF16 ? 8 : 4) : 1;
    return group * kBeamGroup + (e / W) * 64 * W + lane * W + e % W;
}

// The lane's 16 logits of a group; -inf past V.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load_group(const BeamArgs& a, int row, int group, int lane, int state,
                                           float (&x)[16]) {
    const float none = -__builtin_inff();
    if (state != kRowLive) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            x[e] = state == kRowDone && token_of<BF16, VEC>(group, lane, e) == a.eos ? 0.f : none;
        return;
    }
    const uint16_t* h = (const uint16_t*)a.logits + (long long)row * a.ld;
    const float* f = (const float*)a.logits + (long long)row * a.ld;
    if (VEC) {
        // Vectors that cross V are read element by element: the caller's rows
        // may end there.  (Compared with V less a vector: for the largest V the sum
        // t + 8 of the group after the last one would pass 2^31.)
        if (BF16) {
            uint4 v[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = token_of<BF16, VEC>(group, lane, 8 * j);
                v[j] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
                if (t <= a.V - 8) v[j] = *(const uint4*)(h + t);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[8 * j + 2 * i] = bf16_up(w[i] & 0xFFFFu);
                    x[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
                const int t = token_of<BF16, VEC>(group, lane, 8 * j);
                if (t < a.V && t > a.V - 8)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (t + i < a.V) x[8 * j + i] = bf16_up(h[t + i]);
            }
        } else {
            float4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = token_of<BF16, VEC>(group, lane, 4 * j);
                v[j] = make_float4(none, none, none, none);
                if (t <= a.V - 4) v[j] = *(const float4*)(f + t);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[4 * j] = v[j].x;
                x[4 * j + 1] = v[j].y;
                x[4 * j + 2] = v[j].z;
                x[4 * j + 3] = v[j].w;
                const int t = token_of<BF16, VEC>(group, lane, 4 * j);
                if (t < a.V && t > a.V - 4)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t + i < a.V) x[4 * j + i] = f[t + i];
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int t = min(token_of<BF16, VEC>(group, lane, e), a.V - 1);
            x[e] = BF16 ? bf16_up(h[t]) : f[t];
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (token_of<BF16, VEC>(group, lane, e) >= a.V) x[e] = none;
    }
}

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
// exp(x - m): the difference is rounded before it is scaled, so that terms near
// the maximum, which make up the sum, are off by 2^-22 or less.
__device__ __forceinline__ float exp_diff(float x, float m) {
    return __builtin_amdgcn_exp2f((x - m) * 1.44269504088896340736f);
}

// A wave takes kBeamRun groups, all of their loads in flight at once.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(kBeamThreads) void beam_scan_kernel(BeamArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int group0 = (blockIdx.x * (kBeamThreads / 64) + wave) * kBeamRun, row = blockIdx.y;
    if (group0 >= a.groups) return;  // whole wave
    const int state = row_state(a, row);
    float x[kBeamRun][16];
#pragma unroll
    for (int u = 0; u < kBeamRun; ++u) load_group<BF16, VEC>(a, row, group0 + u, lane, state, x[u]);
#pragma unroll
    for (int u = 0; u < kBeamRun; ++u) {
        float m = x[u][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) m = fmaxf(m, x[u][e]);
        m = wave_max(m);
        // exp(x - m) as 2^(x c - m c), the product m c rounded: what that loses is
        // the same for every term and put right once.  From |m| = 2^30 on it would be
        // more than 2^64, but there fp32 numbers are 64 apart and more: equal logits
        // count 1 and others nothing, which 2^(x - m) says as well and exactly.
        const float use = m == -__builtin_inff() ? 0.f : m;
        const float c = fabsf(use) < 1073741824.f ? 1.44269504088896340736f : 1.f;
        const float mc = use * c, lost = __builtin_fmaf(use, c, -mc);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s += __builtin_amdgcn_exp2f(__builtin_fmaf(x[u][e], c, -mc));
        s = wave_sum(s) * __builtin_amdgcn_exp2f(-lost);
        if (lane == 0 && group0 + u < a.groups) a.part[(long long)row * a.groups + group0 + u] = make_float2(m, s);
    }
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

__device__ __forceinline__ float beam_score(float c, float x, float m, float z) {
    return x == -__builtin_inff() ? x : c + ((x - m) - z);
}

// Appends the wave's keys that are at least `bar` to a list in LDS (in no
// particular order); *count goes on past the list's end.
__device__ __forceinline__ void append_keys(u64 key, bool take, u64* list, int* count, int lane) {
    const unsigned long long mine = __ballot(take);
    if (!mine) return;
    int at = 0;
    if (lane == 0) at = atomicAdd(count, __popcll(mine));
    at = __builtin_amdgcn_readfirstlane(at) + __popcll(mine & ((1ull << lane) - 1ull));
    if (take && at < kBeamList) list[at] = key;
}

// The k largest of n distinct keys, in order: a key's place is the number of
// larger ones.  best[] past n is 0.
__device__ __forceinline__ void rank_keys(const u64* list, int n, int k, u64* best) {
    for (int i = threadIdx.x; i < n; i += kBeamPickThreads) {
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

template <bool BF16, bool VEC>
__global__ __launch_bounds__(kBeamPickThreads) void beam_pick_kernel(BeamArgs a) {
    constexpr int kWaves = kBeamPickThreads / 64;
    __shared__ float row_m[NVFP4_BEAM_MAX_BEAMS], row_z[NVFP4_BEAM_MAX_BEAMS], row_c[NVFP4_BEAM_MAX_BEAMS];
    __shared__ int row_s[NVFP4_BEAM_MAX_BEAMS];
    __shared__ u64 list[kBeamList];
    __shared__ u64 best[64], tops[64], bar;
    __shared__ int counts[2];
    static_assert(kBeamList >= kWaves * 64, "the waves' lists fit");
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int row0 = blockIdx.x * a.beams;
    if (threadIdx.x < 2) counts[threadIdx.x] = 0;

    // Each row's maximum and log-sum.
    for (int r = wave; r < a.beams; r += kWaves) {
        const float2* part = a.part + (long long)(row0 + r) * a.groups;
        const float c = a.score[row0 + r];
        const int state = row_state(a, row0 + r);
        float m = -__builtin_inff(), s = 0.f;
        for (int i0 = 0; i0 < a.groups; i0 += 64 * 4) {
            float2 p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + 64 * j + lane;
                p[j] = part[min(i, a.groups - 1)];
                if (i >= a.groups) p[j] = make_float2(-__builtin_inff(), 0.f);
            }
            const float mx = fmaxf(fmaxf(fmaxf(p[0].x, p[1].x), fmaxf(p[2].x, p[3].x)), m);
            const float use = mx == -__builtin_inff() ? 0.f : mx;
            s *= exp_diff(m, use);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = __builtin_fmaf(p[j].y, exp_diff(p[j].x, use), s);
            m = mx;
        }
        const float mx = wave_max(m), use = mx == -__builtin_inff() ? 0.f : mx;
        s = wave_sum(s * exp_diff(m, use));
        if (lane == 0) {
            row_m[r] = use;
            row_z[r] = logf(s);
            row_c[r] = c;
            row_s[r] = state;
        }
    }
    __syncthreads();

    // The k best groups: what passes a bar that at least k pass is ranked.
    const int n = a.beams * a.groups;
    auto group_key = [&](int i) -> u64 {
        if (i >= n) return 0;
        const int r = (int)((unsigned)i / (unsigned)a.groups), g = i - r * a.groups;
        const float m = a.part[(long long)(row0 + r) * a.groups + g].x;
        return topk_key(beam_score(row_c[r], m, row_m[r], row_z[r]), r * a.V + g * kBeamGroup);
    };
    // The bar is the k-th largest of 64 maxima, each over 16 threads' groups: k groups
    // reach it, and few more where the best ones are spread; threads 16 apart take
    // neighbouring groups, so that those of one row are.  (16 requests of 8 beams: 8.5 us
    // for the kernel; 11.5 with a bar found by halving over each wave's keys.)
    const int sub = threadIdx.x >> 4, mine = (threadIdx.x & 15) * 64 + sub;
    static_assert(kBeamPickThreads == 1024, "64 rows of 16 lanes");
    const u64 own = group_key(mine);
    u64 head = own;
    for (int i0 = kBeamPickThreads; i0 < n; i0 += kBeamPickThreads) head = max64(head, group_key(i0 + mine));
    head = row_max64(head);
    if ((lane & 15) == 0) tops[sub] = head;
    if (threadIdx.x == 0) bar = 1;  // fewer than k: all
    __syncthreads();
    int above = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) above += tops[4 * (lane & 15) + j] > head ? 1 : 0;
    if (row_sum(above) == a.k - 1 && head) bar = head;
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kBeamPickThreads) {
        const u64 key = i0 ? group_key(i0 + mine) : own;
        append_keys(key, key >= bar, list, &counts[0], lane);
    }
    __syncthreads();
    if (counts[0] <= kBeamList) {
        rank_keys(list, counts[0], a.k, best);
        __syncthreads();
    } else {
        // Too many pass (a large k over many beams): every wave keeps the k
        // best of what it looks at, and the first joins them.
        __syncthreads();
        u64 kept = 0;
        for (int i0 = wave * 64 * 4; i0 < n; i0 += kBeamPickThreads * 4) {
            u64 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = group_key(i0 + 64 * j + lane);
            kept = wave_keep<4>(kept, x, a.k, lane);
        }
        list[wave * 64 + lane] = lane < a.k ? kept : 0;
        __syncthreads();
        if (wave == 0) {
            u64 x[kWaves];
#pragma unroll
            for (int j = 0; j < kWaves; ++j) x[j] = list[j * 64 + lane];
            best[lane] = wave_keep<kWaves>(0, x, a.k, lane);
        }
        __syncthreads();
    }

    // Their candidates: none below the last group's best one can be listed.
    const u64 last = best[a.k - 1];
    const u64 floor = last ? ((last >> 32) << 32) | (unsigned int)((unsigned int)last - (kBeamGroup - 1)) : 1;
    auto for_candidates = [&](auto&& f) {
        for (int q = wave; q < a.k && best[q]; q += kWaves) {
            const int flat = (int)~(unsigned int)best[q];
            const int r = (int)((unsigned)flat / (unsigned)a.V), g = (flat - r * a.V) / kBeamGroup;
            float x[16];
            load_group<BF16, VEC>(a, row0 + r, g, lane, row_s[r], x);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = token_of<BF16, VEC>(g, lane, e);
                f(t < a.V ? topk_key(beam_score(row_c[r], x[e], row_m[r], row_z[r]), r * a.V + t) : 0);
            }
        }
    };
    for_candidates([&](u64 key) { append_keys(key, key >= floor, list, &counts[1], lane); });
    __syncthreads();
    if (counts[1] <= kBeamList) {
        const int found = counts[1];
        __shared__ u64 winners[64];
        rank_keys(list, found, a.k, winners);
        __syncthreads();
        if (threadIdx.x < 64) best[threadIdx.x] = winners[threadIdx.x];
    } else {
        // Many equal scores, or fewer groups than k, so that every candidate passes (a
        // vocabulary of a few thousand): the waves insert their candidates one by one
        // into sorted lists of their own.
        __syncthreads();
        u64 kept = 0;
        for_candidates([&](u64 key) {
            unsigned long long todo = __ballot(key >= floor && key > lane64(kept, a.k - 1));
            while (todo) {
                const u64 v = lane64(key, __ffsll(todo) - 1);
                todo &= todo - 1;
                u64 prev = ((u64)(unsigned int)__shfl_up((int)(kept >> 32), 1) << 32) | (unsigned int)__shfl_up((int)kept, 1);
                if (lane == 0) prev = ~0ull;
                kept = kept > v ? kept : prev > v ? v : prev;
            }
        });
        list[wave * 64 + lane] = lane < a.k ? kept : 0;
        __syncthreads();
        if (wave == 0) {
            u64 x[kWaves];
#pragma unroll
            for (int j = 0; j < kWaves; ++j) x[j] = list[j * 64 + lane];
            best[lane] = wave_keep<kWaves>(0, x, a.k, lane);
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < a.k) {
        const u64 key = best[threadIdx.x];
        const int flat = (int)~(unsigned int)key;
        // (a NaN among the logits can leave a place empty: token -1, in bounds)
        const int r = key ? (int)((unsigned)flat / (unsigned)a.V) : 0, t = key ? flat - r * a.V : -1;
        const unsigned int o = (unsigned int)(key >> 32);
        const long long at = (long long)blockIdx.x * a.k + threadIdx.x;
        a.score_out[at] = __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
        a.parent_out[at] = row0 + r;
        a.token_out[at] = t;
        if (a.done_out) a.done_out[at] = (a.done && a.done[row0 + r]) || t == a.eos ? 1 : 0;
    }
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_beam_workspace_bytes(int batch, int beams, int V) {
    if (batch < 1 || beams < 1 || beams > NVFP4_BEAM_MAX_BEAMS || V < 1) return 0;
    return (size_t)batch * beams * ((V + kBeamGroup - 1) / kBeamGroup) * sizeof(float2);
}

int nvfp4_beam_select(const void* logits_dev, int logits_dtype, int64_t ld, int batch, int beams, int V,
                      const float* score_dev, const uint8_t* done_dev, int eos, int k,
                      float* score_out_dev, int* parent_dev, int* token_dev, uint8_t* done_out_dev,
                      void* workspace_dev, size_t workspace_bytes, void* stream) {
    clear_error();
    if (logits_dtype != NVFP4_OUT_F32 && logits_dtype != NVFP4_OUT_BF16)
        return set_error(NVFP4_EINVAL, "logits_dtype: %d", logits_dtype);
    if (batch < 1 || batch > 65535) return set_error(NVFP4_EINVAL, "batch: %d outside [1, 65535]", batch);
    if (beams < 1 || beams > NVFP4_BEAM_MAX_BEAMS)
        return set_error(NVFP4_EINVAL, "beams: %d outside [1, %d]", beams, NVFP4_BEAM_MAX_BEAMS);
    if ((long long)batch * beams > 65535) return set_error(NVFP4_EINVAL, "batch: %d x %d beams exceed 65535 rows", batch, beams);
    if (V < 1 || (long long)V * beams > 0x7FFFFFFFll - kBeamGroup)
        return set_error(NVFP4_EINVAL, "V: %d outside [1, (2^31 - 1025) / beams]", V);
    if (ld < V) return set_error(NVFP4_EINVAL, "ld: %lld < V = %d", (long long)ld, V);
    if (k < 1 || k > NVFP4_TOPK_MAX_K || k > V)
        return set_error(NVFP4_EINVAL, "k: %d outside [1, min(V, %d)]", k, NVFP4_TOPK_MAX_K);
    const bool bf16 = logits_dtype == NVFP4_OUT_BF16;
    if (!logits_dev || ((uintptr_t)logits_dev & (bf16 ? 1 : 3)))
        return set_error(NVFP4_EINVAL, "logits: NULL or not aligned to its type");
    if (!score_dev || ((uintptr_t)score_dev & 3)) return set_error(NVFP4_EINVAL, "score: NULL or not 4-byte aligned");
    if (!score_out_dev || ((uintptr_t)score_out_dev & 3)) return set_error(NVFP4_EINVAL, "score_out: NULL or not 4-byte aligned");
    if (!parent_dev || ((uintptr_t)parent_dev & 3)) return set_error(NVFP4_EINVAL, "parent: NULL or not 4-byte aligned");
    if (!token_dev || ((uintptr_t)token_dev & 3)) return set_error(NVFP4_EINVAL, "token: NULL or not 4-byte aligned");
    if (done_dev && (eos < 0 || eos >= V)) return set_error(NVFP4_EINVAL, "eos: %d outside [0, V) with finished rows", eos);
    const size_t need = nvfp4_beam_workspace_bytes(batch, beams, V);
    if (workspace_bytes < need) return set_error(NVFP4_EINVAL, "workspace_bytes: %zu < %zu needed", workspace_bytes, need);
    if (!workspace_dev || ((uintptr_t)workspace_dev & 15)) return set_error(NVFP4_EINVAL, "workspace: NULL or not 16-byte aligned");
    BeamArgs a;
    a.logits = logits_dev;
    a.ld = ld;
    a.beams = beams;
    a.V = V;
    a.k = k;
    a.groups = (V + kBeamGroup - 1) / kBeamGroup;
    a.score = score_dev;
    a.done = done_dev;
    a.eos = eos;
    a.part = (float2*)workspace_dev;
    a.score_out = score_out_dev;
    a.parent_out = parent_dev;
    a.token_out = token_dev;
    a.done_out = done_out_dev;
    const bool vec = ((uintptr_t)logits_dev & 15) == 0 && ld % (bf16 ? 8 : 4) == 0;
    hipStream_t s = (hipStream_t)stream;
    const int per_block = kBeamThreads / 64 * kBeamRun;
    const dim3 scan((unsigned)(a.groups + per_block - 1) / per_block, (unsigned)(batch * beams));
    const dim3 pick((unsigned)batch);
#define NVFP4_BEAM(B, W)                                                                          \
    if (bf16 == B && vec == W) {                                                                  \
        hipLaunchKernelGGL((beam_scan_kernel<B, W>), scan, dim3(kBeamThreads), 0, s, a);          \
        NVFP4_HIP(hipGetLastError());                                                             \
        hipLaunchKernelGGL((beam_pick_kernel<B, W>), pick, dim3(kBeamPickThreads), 0, s, a);      \
    }
    NVFP4_BEAM(false, false)
    NVFP4_BEAM(false, true)
    NVFP4_BEAM(true, false)
    NVFP4_BEAM(true, true)
#undef NVFP4_BEAM
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

}  // extern "C"
