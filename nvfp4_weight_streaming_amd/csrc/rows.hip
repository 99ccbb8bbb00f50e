// Rows between the products: the root-mean-square norm with the residual's
// addition, and rows in 8-bit integers with one scale each (of x itself, or of
// the SwiGLU of a [gate | up] row), which the 8-bit product takes.
//
//   h = x + residual, rounded to the residual's type and written back
//   y = h / sqrt(mean(h^2) + eps) * (weight + offset)
//   s = fl32(max |y| / 127),  code = y / s to the nearest integer, ties to even
//
// Results are the definition's in fp64, rounded once: a code next to a border, and the
// scale, do not depend on how a sum was ordered (but within 2^-48 or so of a border).  The sum of
// squares is in fp64.  A value is first formed in fp32, with a bound of its error; where that leaves
// open how it rounds, or which one is the largest, it is formed again in fp64.  To bf16 those are 17 of 65536 values; to codes, about 1 in
// 10^4 or fewer, but where a vector of SwiGLU has a gate far below 0, whose bound grows with it (at -30, 1 in 2000 codes of 30).
// (All of it in fp64, the SwiGLU of 2048 x 17408 took 124 us, and its exponentials and divisions were what it waited for.)
//
// A row is read once: 64, 256 or 1024 threads hold up to 3 vectors of 8 values each (1536, 6144, 24576 values);
// longer rows are read again for each step.  From 4097 to 8192 values 1024 threads hold a vector each: always above
// 6144 (codes of 1026 rows of 6400: 11.5 us, 12.4 with room for three), and below it for few rows, for less work one after the
// other (codes of 65 rows of 5120: 5.1 us, 7.1 with 256 threads; 513 rows 6.5 and 7.4, 1025 rows 10.8 and 9.0; 8 rows of 2048
// would take 4.3 and 3.7).
#include "select_device.h"
#include "swiglu_device.h"

namespace nvfp4 {

enum { kRowNorm = 0, kRowPlain = 1, kRowSwiglu = 2 };
enum { kRowNone = -1 };  // a type: there is no such operand
constexpr int kRowMaxRows = (1 << 22) - 1;  // a launch has fewer than 2^32 threads
constexpr int kRowFew = 512;
constexpr int kRowVecs = 3;  // vectors of 8 values a thread holds

struct RowArgs {
    const void* x;
    const void* residual;
    void* residual_out;
    const void* weight;
    void* out;
    float* scale;
    long long x_ld, residual_ld, out_ld;
    int x_type, residual_type, weight_type;  // nvfp4_out_dtype; kRowNone
    int rows, K;
    double offset, eps;
};

// Where value e of a thread's vector v stands in the row: eight in a row, or,
// for rows that are not aligned, one from each of eight runs of T.
template <int T, bool VEC>
__device__ __forceinline__ int row_at(int v, int t, int e) {
    return VEC ? (v * T + t) * 8 + e : (v * 8 + e) * T + t;
}

// A vector as it is read: 8 bf16 in `a`, or 8 fp32 in both.  Unaligned rows have
// one value in each word.  (The conversion stands apart, so that all of a row's
// loads are in flight before the first is waited for.)
template <bool B16>
struct RowRaw {
    uint4 a, b;
};
template <>
struct RowRaw<true> {
    uint4 a;
};

// B16: every operand is bf16 (and rows are read in vectors), known as the kernel is compiled.
template <int T, bool VEC, bool B16>
__device__ __forceinline__ RowRaw<B16> row_load(const void* p, int type, long long at, int v, int t, int K) {
    const uint16_t* h = (const uint16_t*)p + at;
    const uint32_t* w = (const uint32_t*)p + at;
    RowRaw<B16> r;
    r.a = make_uint4(0, 0, 0, 0);
    if constexpr (B16) {
        const int i = row_at<T, VEC>(v, t, 0);
        if (i < K) r.a = *(const uint4*)(h + i);
        return r;
    } else {
    r.b = make_uint4(0, 0, 0, 0);
    if (VEC) {
        const int i = row_at<T, VEC>(v, t, 0);
        if (i >= K) return r;
        if (type == NVFP4_OUT_BF16) {
            r.a = *(const uint4*)(h + i);
        } else {
            r.a = *(const uint4*)(w + i);
            r.b = *(const uint4*)(w + i + 4);
        }
    } else {
        uint32_t u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = row_at<T, VEC>(v, t, e);
            u[e] = i >= K ? 0u : type == NVFP4_OUT_BF16 ? h[i] : w[i];
        }
        r.a = make_uint4(u[0], u[1], u[2], u[3]);
        r.b = make_uint4(u[4], u[5], u[6], u[7]);
    }
    return r;
    }
}

// Its values as fp32 (exact); 0 past the row's end.
template <bool VEC, bool B16>
__device__ __forceinline__ void row_values(const RowRaw<B16>& r, int type, float (&f)[8]) {
    uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w};
    if constexpr (!B16) u[4] = r.b.x, u[5] = r.b.y, u[6] = r.b.z, u[7] = r.b.w;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (type != NVFP4_OUT_BF16)
            f[e] = __uint_as_float(u[e]);
        else if (VEC)
            f[e] = __uint_as_float(e % 2 ? u[e / 2] & 0xFFFF0000u : u[e / 2] << 16);
        else
            f[e] = __uint_as_float(u[e] << 16);
    }
}

// Two fp32 values to bf16, nearest even.
typedef float row_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 row_bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t row_pack(float a, float b) {
    const row_bf16x2 v = __builtin_convertvector((row_f32x2{a, b}), row_bf16x2);
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}
// An fp64 value as an fp32 one that rounds to the same bf16: its last bit set if anything
// was lost, so that no tie appears or disappears.
__device__ __forceinline__ float row_odd(double d) {
    const float f = (float)d;
    const double back = (double)f;
    uint32_t u = __float_as_uint(f);
    if (fabs(back) > fabs(d)) u -= 1;
    if (back != d) u |= 1;
    return __uint_as_float(u);
}

// A vector to a row of `type`: fp32 values, exact in that type or (bf16) rounded here.
template <int T, bool VEC>
__device__ __forceinline__ void row_store(void* p, int type, long long at, int v, int t, int K, const float (&y)[8]) {
    uint16_t* h = (uint16_t*)p + at;
    float* w = (float*)p + at;
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = row_pack(y[2 * e], y[2 * e + 1]);
    if (VEC) {
        const int i = row_at<T, VEC>(v, t, 0);
        if (i >= K) return;
        if (type == NVFP4_OUT_BF16) {
            *(uint4*)(h + i) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
            *(float4*)(w + i) = make_float4(y[0], y[1], y[2], y[3]);
            *(float4*)(w + i + 4) = make_float4(y[4], y[5], y[6], y[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = row_at<T, VEC>(v, t, e);
            if (i >= K) continue;
            if (type == NVFP4_OUT_BF16)
                h[i] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
            else
                w[i] = y[e];
        }
    }
}

// Joins the waves' values over the T threads of a row, in all of them.
template <int T, class F>
__device__ __forceinline__ u64 row_join(u64 mine, u64* lds, F f) {
    if (T == 64) return mine;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = mine;
    __syncthreads();
    u64 all = lds[0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) all = f(all, lds[i]);
    return all;
}

// The code of y: y * inv is off by 2^-52 of itself, so the nearest integer is q or, next to a border, its
// neighbour; what is left of y says which.
__device__ __forceinline__ int row_code(double y, double s, double inv) {
    const double q = rint(y * inv), rest = __builtin_fma(-q, s, y), half = 0.5 * s;
    const int i = (int)q;
    const bool move = fabs(rest) > half || (fabs(rest) == half && (i & 1));
    return min(127, max(-127, move ? i + (rest > 0 ? 1 : -1) : i));
}

// One value, read anew, in fp64.
template <int MODE>
__device__ __forceinline__ double row_exact(const RowArgs& a, long long xo, long long ro, int i, double factor) {
    auto one = [](const void* p, int type, long long at) {
        return type == NVFP4_OUT_BF16 ? (double)__uint_as_float((uint32_t)((const uint16_t*)p)[at] << 16) : (double)((const float*)p)[at];
    };
    if (MODE == kRowNorm) {
        const double h = a.residual ? one(a.residual_out, a.residual_type, ro + i) : one(a.x, a.x_type, xo + i);
        return h * factor * (one(a.weight, a.weight_type, i) + a.offset);
    }
    const double x = one(a.x, a.x_type, xo + i);
    return MODE == kRowPlain ? x : x * one(a.x, a.x_type, xo + a.K + i) / (1.0 + exp(-x));
}

// Where fp32 is trusted: away from its smallest and largest numbers.
constexpr float kRowLeast = 0x1p-100f, kRowMost = 0x1p100f;
// Codes do not depend on what is far below the row's largest value: a row of at least this may have values of
// less than 2^-58 whose fp32 form says no more than that.
template <int MODE>
constexpr float row_floor() {
    return MODE == kRowPlain ? kRowLeast : 0x1p-50f;
}

// One row per T threads, R vectors a thread.  HELD: the row lies in registers between the steps.
// (Two rows of 1024 threads a compute unit where rows are held; rows read again need more registers than that leaves: 1024 SwiGLU rows
// of 32768 took 153 us so, and take 85.)
template <int T, int R, int MODE, int OUT, bool VEC, bool HELD, bool B16>
__global__ __launch_bounds__(T < 256 ? 256 : T, T == 1024 && B16 && HELD && MODE != kRowNorm ? 8 : 1) void rows_kernel(RowArgs a) {
    constexpr int kPer = T < 256 ? 256 / T : 1;  // rows per workgroup
    __shared__ u64 lds[2][T / 64];
    __shared__ u64 top;
    const int t = threadIdx.x % T;
    const int row = blockIdx.x * kPer + threadIdx.x / T;
    if (T == 64 && row >= a.rows) return;  // whole wave (T = 64 meets no barrier)
    const int K = a.K;
    const int chunks = HELD ? 1 : (K + T * R * 8 - 1) / (T * R * 8);
    const long long xo = (long long)row * a.x_ld, ro = (long long)row * a.residual_ld;
    const int x_type = B16 ? NVFP4_OUT_BF16 : a.x_type, r_type = B16 ? NVFP4_OUT_BF16 : a.residual_type;

    float h[R][8], w[R][8];  // norm: h and the weight; plain: x; SwiGLU: gate and up
    auto load = [&](int c, bool first) {
        RowRaw<B16> x[R], r[R], o[R];
        const bool kept = MODE == kRowNorm && a.residual && !first;  // h as it was stored
        const int type = kept ? r_type : x_type, other = B16 ? NVFP4_OUT_BF16 : MODE == kRowNorm ? a.weight_type : x_type;
        const bool adds = MODE == kRowNorm && a.residual && first;
#pragma unroll
        for (int j = 0; j < R; ++j) x[j] = row_load<T, VEC, B16>(kept ? a.residual_out : a.x, type, kept ? ro : xo, c * R + j, t, K);
        if (adds)
#pragma unroll
            for (int j = 0; j < R; ++j) r[j] = row_load<T, VEC, B16>(a.residual, r_type, ro, c * R + j, t, K);
        if (MODE == kRowSwiglu || (MODE == kRowNorm && (HELD || !first)))
#pragma unroll
            for (int j = 0; j < R; ++j)
                o[j] = row_load<T, VEC, B16>(MODE == kRowNorm ? a.weight : a.x, other, MODE == kRowNorm ? 0 : xo + K, c * R + j, t, K);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            row_values<VEC, B16>(x[j], type, h[j]);
            if (adds) {
                float s[8];
                row_values<VEC, B16>(r[j], r_type, s);
                // fp32 + fp32 and bf16 + fp32 are rounded once to fp32.  A sum of two bf16 that fp32 has
                // to round is within 2^-15 of one of them, far from a tie between two bf16.  fp32 + bf16
                // to bf16 goes by fp64.
                if (r_type == NVFP4_OUT_BF16 && x_type != NVFP4_OUT_BF16) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[j][e] = row_odd((double)h[j][e] + (double)s[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[j][e] += s[e];
                }
                if (r_type == NVFP4_OUT_BF16) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const uint32_t u = row_pack(h[j][e], h[j][e + 1]);
                        h[j][e] = __uint_as_float(u << 16);
                        h[j][e + 1] = __uint_as_float(u & 0xFFFF0000u);
                    }
                }
                row_store<T, VEC>(a.residual_out, r_type, ro, c * R + j, t, K, h[j]);
            }
            if (MODE == kRowSwiglu || (MODE == kRowNorm && (HELD || !first))) row_values<VEC, B16>(o[j], other, w[j]);
        }
    };

    double factor = 1.0;
    bool zeros = MODE != kRowNorm;  // a row whose fp32 values are all 0 is one of zeros
    if (MODE == kRowNorm) {
        double sum = 0.0;
        for (int c = 0; c < chunks; ++c) {
            load(c, true);
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)h[j][e], (double)h[j][e], sum);
        }
        const u64 all = row_join<T>((u64)__double_as_longlong(wave_sumd(sum)), lds[0], [](u64 p, u64 q) {
            return (u64)__double_as_longlong(__longlong_as_double((long long)p) + __longlong_as_double((long long)q));
        });
        factor = 1.0 / sqrt(__longlong_as_double((long long)all) / K + a.eps);
        zeros = all == 0;
    } else if (HELD) {
        load(0, true);
    }
    const float f32 = (float)factor, off32 = (float)a.offset;
    // Value (j, e) in fp32.
    auto value = [&](int j, int e) -> float {
        const float x = h[j][e];
        if (MODE == kRowPlain) return x;
        if (MODE == kRowNorm) return x * f32 * (w[j][e] + off32);
        return x * w[j][e] * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * -1.44269504088896340736f));
    };

    if constexpr (OUT == NVFP4_OUT_F32) {
        for (int c = 0; c < chunks; ++c) {
            if (!HELD) load(c, false);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = (float)((double)h[j][e] * factor * ((double)w[j][e] + a.offset));
                row_store<T, VEC>(a.out, OUT, (long long)row * a.out_ld, c * R + j, t, K, y);
            }
        }
    } else if constexpr (OUT == NVFP4_OUT_BF16) {
        for (int c = 0; c < chunks; ++c) {
            if (!HELD) load(c, false);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (row_at<T, VEC>(c * R + j, t, 0) >= K) continue;
                float y[8];
                uint32_t open = 0;  // elements that may round either way
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (four roundings, of 2^-24 each: the factor's, the sum's and two products'; at most four of the
                    // last bit, which is more where a product is tiny)
                    y[e] = value(j, e);
                    const bool far = (__float_as_uint(y[e]) & 0xFFFFu) - 0x7FF8u > 16u;
                    const bool sound = fabsf(h[j][e] * f32) >= kRowLeast && fabsf(y[e]) >= kRowLeast && fabsf(y[e]) <= kRowMost;
                    open |= (sound && far) || (h[j][e] == 0.f && y[e] == 0.f) ? 0u : 1u << e;
                }
                while (open) {
                    const int at = __ffs(open) - 1, i = row_at<T, VEC>(c * R + j, t, at);
                    open &= open - 1;
                    if (i >= K) continue;
                    const float better = row_odd(row_exact<MODE>(a, xo, ro, i, factor));
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = e == at ? better : y[e];
                }
                row_store<T, VEC>(a.out, OUT, (long long)row * a.out_ld, c * R + j, t, K, y);
            }
        }
    } else {
        // Values; of each vector the largest magnitude's bits (NaN above all), a bound of the relative errors in
        // units of 2^-24, and whether there is one.
        float y[R][8], eps[R];
        uint32_t peak[R];
        bool fine[R];
        auto form = [&](int c) {
            if (!HELD) load(c, false);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                float side = 0.f;
                peak[j] = 0;
                eps[j] = 0.f;
                fine[j] = true;
                // (a vector past the row's end, as most waves' third of 17408 values: with them 2048 such SwiGLU rows took 49 us, and take 44 to 46)
                if (row_at<T, VEC>(c * R + j, t, 0) >= K) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (past the row's end x is 0, and so is y, or NaN as the row's others)
                    y[j][e] = value(j, e);
                    peak[j] = max(peak[j], __float_as_uint(y[j][e]) & 0x7FFFFFFFu);
                    if (MODE == kRowNorm) side = fmaxf(side, fabsf(w[j][e] + off32));
                    if (MODE == kRowSwiglu) side = fmaxf(side, -h[j][e]);
                }
                fine[j] = peak[j] <= __float_as_uint(kRowMost);
                if (MODE == kRowNorm) {
                    // Four roundings, the factor's, the sum's and two products'; a first product below fp32's range
                    // makes no value that matters.
                    eps[j] = 8.f;
                    fine[j] = fine[j] && side <= 0x1p40f;
                }
                if (MODE == kRowSwiglu) {
                    // The exponential's argument is off by 1.5 |x| 2^-24, itself by 2, and is nothing beside 1 for large x; the sum,
                    // its inverse and the products by 6.  Below -87 the exponential passes fp32, y is 0 here and less than
                    // |x u| 2^-125.
                    eps[j] = 16.f + 4.f * fminf(side, 87.f);
                    if (side > 87.f) {
                        peak[j] = max(peak[j], 1u);  // no row of zeros
#pragma unroll
                        for (int e = 0; e < 8; ++e) fine[j] = fine[j] && (h[j][e] >= -87.f || fabsf(h[j][e] * w[j][e]) <= 0x1p60f);
                    }
                }
            }
        };
        // The largest magnitude: by fp32 first, then exactly among those that may be it.  (Bits of magnitudes are
        // in their order, NaN above all.)
        float most = 0.f;
        if (threadIdx.x == 0) top = 0;
        if (HELD) form(0);
        for (int c = 0; c < chunks; ++c) {
            if (!HELD) form(c);
#pragma unroll
            for (int j = 0; j < R; ++j) most = fmaxf(most, fine[j] ? __uint_as_float(peak[j]) : __builtin_inff());
        }
        const u64 found = row_join<T>((u64)__float_as_uint(wave_max(most)), lds[1], [](u64 p, u64 q) { return max64(p, q); });
        const float near = __uint_as_float((uint32_t)found);  // infinite: some value has no bound
        const bool tame = near >= row_floor<MODE>() && near <= kRowMost;
        // (at most (16 + 4 * 87) 2^-24 off either way)
        const float bar = near == 0.f && zeros ? __builtin_inff() : tame ? near * (1.f - 0x1p-14f) : 0.f;
        u64 mine = 0;
        for (int c = 0; c < chunks; ++c) {
            if (!HELD) form(c);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                if (fine[j] && __uint_as_float(peak[j]) < bar) continue;
                uint32_t open = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) open |= !fine[j] || fabsf(y[j][e]) >= bar ? 1u << e : 0u;
                while (open) {
                    const int i = row_at<T, VEC>(c * R + j, t, __ffs(open) - 1);
                    open &= open - 1;
                    if (i < K) mine = max64(mine, (u64)__double_as_longlong(row_exact<MODE>(a, xo, ro, i, factor)) & 0x7FFFFFFFFFFFFFFFull);
                }
            }
        }
        if (T == 64) {
            mine = wave_max64(mine);
        } else {
            if (mine) atomicMax(&top, mine);
            __syncthreads();
            mine = top;
        }
        const float s32 = (float)(__longlong_as_double((long long)mine) / 127.0);
        if (t == 0) a.scale[row] = s32;
        const bool none = !(s32 > 0.f && s32 < __builtin_inff());
        const double s = none ? 1.0 : (double)s32, inv = 1.0 / s;
        const float i32 = none ? 0.f : (float)inv;
        int8_t* out = (int8_t*)a.out + (long long)row * a.out_ld;
        for (int c = 0; c < chunks; ++c) {
            if (!HELD) form(c);
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int v = c * R + j;
                if (row_at<T, VEC>(v, t, 0) >= K) continue;
                // Adding 1.5 * 2^23 rounds to a whole number, ties to even, and leaves it in the last byte. (Two more
                // roundings, the inverse's and the product's; compared so that a NaN is open.)
                const float off = (eps[j] + 4.f) * 0x1p-24f;
                uint32_t q[8];
                bool some = !tame || !fine[j];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float z = y[j][e] * i32, up = z + 12582912.f, r = up - 12582912.f;
                    some |= !(fabsf(z - r) <= 0.5f - fabsf(z) * off);
                    q[e] = __float_as_uint(up);
                }
                if (some && !none) {
                    uint32_t open = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float z = y[j][e] * i32, r = (z + 12582912.f) - 12582912.f;
                        open |= tame && fine[j] && fabsf(z - r) <= 0.5f - fabsf(z) * off ? 0u : 1u << e;
                    }
                    while (open) {
                        const int at = __ffs(open) - 1, i = row_at<T, VEC>(v, t, at);
                        open &= open - 1;
                        if (i >= K) continue;
                        const uint32_t better = (uint32_t)row_code(row_exact<MODE>(a, xo, ro, i, factor), s, inv);
#pragma unroll
                        for (int e = 0; e < 8; ++e) q[e] = e == at ? better : q[e];
                    }
                }
                const uint32_t lo = none ? 0u : (q[0] & 255u) | (q[1] & 255u) << 8 | (q[2] & 255u) << 16 | q[3] << 24;
                const uint32_t hi = none ? 0u : (q[4] & 255u) | (q[5] & 255u) << 8 | (q[6] & 255u) << 16 | q[7] << 24;
                if (VEC) {
                    *(uint2*)(out + row_at<T, VEC>(v, t, 0)) = make_uint2(lo, hi);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = row_at<T, VEC>(v, t, e);
                        if (i < K) out[i] = (int8_t)((e < 4 ? lo : hi) >> (8 * (e & 3)));
                    }
                }
            }
        }
    }
}

template <int MODE, int OUT>
int launch_rows(const RowArgs& a, bool vec, hipStream_t s) {
    const bool single = vec && a.K > 4096 && a.K <= 8192 && (a.rows <= kRowFew || a.K > 256 * kRowVecs * 8);
    const int t = single ? 1024 : a.K <= 64 * kRowVecs * 8 ? 64 : a.K <= 256 * kRowVecs * 8 ? 256 : 1024;
    // (unaligned rows of 1024 threads would not fit the registers)
    const bool held = a.K <= t * kRowVecs * 8 && (vec || t < 1024);
    const unsigned grid = t == 64 ? (unsigned)((a.rows + 3) / 4) : (unsigned)a.rows;
    const bool b16 = vec && a.x_type == NVFP4_OUT_BF16 && (!a.residual || a.residual_type == NVFP4_OUT_BF16) &&
                     (MODE != kRowNorm || a.weight_type == NVFP4_OUT_BF16);
#define NVFP4_ROWS(T, R, V, H, B)                                                                             \
    if (t == T && single == (R == 1) && vec == V && held == H && b16 == B)                                       \
        hipLaunchKernelGGL((rows_kernel<T, R, MODE, OUT, V, H, B>), dim3(grid), dim3(T < 256 ? 256 : T), 0, s, a);
    NVFP4_ROWS(1024, 1, true, true, true)
    NVFP4_ROWS(1024, 1, true, true, false)
    NVFP4_ROWS(64, kRowVecs, true, true, true)
    NVFP4_ROWS(64, kRowVecs, true, true, false)
    NVFP4_ROWS(64, kRowVecs, false, true, false)
    NVFP4_ROWS(256, kRowVecs, true, true, true)
    NVFP4_ROWS(256, kRowVecs, true, true, false)
    NVFP4_ROWS(256, kRowVecs, false, true, false)
    NVFP4_ROWS(1024, kRowVecs, true, true, true)
    NVFP4_ROWS(1024, kRowVecs, true, true, false)
    NVFP4_ROWS(1024, kRowVecs, true, false, true)
    NVFP4_ROWS(1024, kRowVecs, true, false, false)
    NVFP4_ROWS(1024, kRowVecs, false, false, false)
#undef NVFP4_ROWS
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

// One operand's pointer and row stride; `n` values a row.
int check_rows(const char* name, const void* p, int type, long long ld, int rows, long long n) {
    if (rows > 0 && !p) return set_error(NVFP4_EINVAL, "%s: NULL", name);
    const uintptr_t mask = type == NVFP4_OUT_F32 ? 3 : type == NVFP4_OUT_BF16 ? 1 : 0;
    if ((uintptr_t)p & mask) return set_error(NVFP4_EINVAL, "%s: not aligned to its type", name);
    if (ld < n) return set_error(NVFP4_EINVAL, "%s_ld: %lld < %lld values a row", name, ld, n);
    return NVFP4_OK;
}

bool row_type(int t) { return t == NVFP4_OUT_F32 || t == NVFP4_OUT_BF16; }

// Whether rows of `type` at p, ld apart, are read or written in vectors of 8 values.
bool row_vec(const void* p, int type, long long ld) {
    const int size = type == NVFP4_OUT_F32 ? 4 : type == NVFP4_OUT_BF16 ? 2 : 1;
    const int align = size == 1 ? 8 : 16;
    return ((uintptr_t)p & (align - 1)) == 0 && ld * size % align == 0;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_rms_norm(const nvfp4_norm* n, int rows, int K, void* stream) {
    clear_error();
    if (!n) return set_error(NVFP4_EINVAL, "norm: NULL");
    if (rows < 0 || rows > kRowMaxRows) return set_error(NVFP4_EINVAL, "rows: %d outside [0, %d]", rows, kRowMaxRows);
    if (K < 1 || K > NVFP4_ROW_MAX_K) return set_error(NVFP4_EINVAL, "K: %d outside [1, %d]", K, NVFP4_ROW_MAX_K);
    if (!row_type(n->x_dtype)) return set_error(NVFP4_EINVAL, "x_dtype: %d", n->x_dtype);
    if (!row_type(n->weight_dtype)) return set_error(NVFP4_EINVAL, "weight_dtype: %d", n->weight_dtype);
    if (!row_type(n->out_dtype) && n->out_dtype != NVFP4_OUT_INT8) return set_error(NVFP4_EINVAL, "out_dtype: %d", n->out_dtype);
    if (!(n->eps >= 0.f)) return set_error(NVFP4_EINVAL, "eps: %g is not 0 or more", n->eps);
    if (n->weight_offset != n->weight_offset) return set_error(NVFP4_EINVAL, "weight_offset: NaN");
    if (int st = check_rows("x", n->x_dev, n->x_dtype, n->x_ld, rows, K)) return st;
    if (int st = check_rows("weight", n->weight_dev, n->weight_dtype, K, rows, K)) return st;
    if (int st = check_rows("out", n->out_dev, n->out_dtype, n->out_ld, rows, K)) return st;
    bool vec = K % 8 == 0 && row_vec(n->x_dev, n->x_dtype, n->x_ld) && row_vec(n->weight_dev, n->weight_dtype, 0) &&
               row_vec(n->out_dev, n->out_dtype, n->out_ld);
    RowArgs a = {};
    a.residual_type = kRowNone;
    if (n->residual_dev || n->residual_out_dev) {
        if (!row_type(n->residual_dtype)) return set_error(NVFP4_EINVAL, "residual_dtype: %d", n->residual_dtype);
        if (int st = check_rows("residual", n->residual_dev, n->residual_dtype, n->residual_ld, rows, K)) return st;
        if (int st = check_rows("residual_out", n->residual_out_dev, n->residual_dtype, n->residual_ld, rows, K)) return st;
        vec = vec && row_vec(n->residual_dev, n->residual_dtype, n->residual_ld) &&
              row_vec(n->residual_out_dev, n->residual_dtype, n->residual_ld);
        a.residual = n->residual_dev;
        a.residual_out = n->residual_out_dev;
        a.residual_ld = n->residual_ld;
        a.residual_type = n->residual_dtype;
    }
    if (n->out_dtype == NVFP4_OUT_INT8 && rows > 0 && (!n->scale_dev || ((uintptr_t)n->scale_dev & 3)))
        return set_error(NVFP4_EINVAL, "scale: NULL or not 4-byte aligned");
    if (rows == 0) return NVFP4_OK;
    a.x = n->x_dev;
    a.weight = n->weight_dev;
    a.out = n->out_dev;
    a.scale = n->scale_dev;
    a.x_ld = n->x_ld;
    a.out_ld = n->out_ld;
    a.x_type = n->x_dtype;
    a.weight_type = n->weight_dtype;
    a.rows = rows;
    a.K = K;
    a.offset = n->weight_offset;
    a.eps = n->eps;
    const hipStream_t s = (hipStream_t)stream;
    if (n->out_dtype == NVFP4_OUT_F32) return launch_rows<kRowNorm, NVFP4_OUT_F32>(a, vec, s);
    if (n->out_dtype == NVFP4_OUT_BF16) return launch_rows<kRowNorm, NVFP4_OUT_BF16>(a, vec, s);
    return launch_rows<kRowNorm, NVFP4_OUT_INT8>(a, vec, s);
}

int nvfp4_int8_quantize(const void* x_dev, int x_dtype, int64_t x_ld, int rows, int K, int swiglu, int8_t* codes_dev,
                        int64_t codes_ld, float* scale_dev, void* stream) {
    clear_error();
    if (rows < 0 || rows > kRowMaxRows) return set_error(NVFP4_EINVAL, "rows: %d outside [0, %d]", rows, kRowMaxRows);
    if (K < 1 || K > NVFP4_ROW_MAX_K) return set_error(NVFP4_EINVAL, "K: %d outside [1, %d]", K, NVFP4_ROW_MAX_K);
    if (!row_type(x_dtype)) return set_error(NVFP4_EINVAL, "x_dtype: %d", x_dtype);
    if (swiglu != 0 && swiglu != 1) return set_error(NVFP4_EINVAL, "swiglu: %d is not 0 or 1", swiglu);
    if (int st = check_rows("x", x_dev, x_dtype, x_ld, rows, swiglu ? 2ll * K : K)) return st;
    if (int st = check_rows("codes", codes_dev, NVFP4_OUT_INT8, codes_ld, rows, K)) return st;
    if (rows > 0 && (!scale_dev || ((uintptr_t)scale_dev & 3))) return set_error(NVFP4_EINVAL, "scale: NULL or not 4-byte aligned");
    if (rows == 0) return NVFP4_OK;
    RowArgs a = {};
    a.x = x_dev;
    a.out = codes_dev;
    a.scale = scale_dev;
    a.x_ld = x_ld;
    a.out_ld = codes_ld;
    a.x_type = x_dtype;
    a.residual_type = a.weight_type = kRowNone;
    a.rows = rows;
    a.K = K;
    const bool vec = K % 8 == 0 && row_vec(x_dev, x_dtype, x_ld) && row_vec(codes_dev, NVFP4_OUT_INT8, codes_ld);
    const hipStream_t s = (hipStream_t)stream;
    return swiglu ? launch_rows<kRowSwiglu, NVFP4_OUT_INT8>(a, vec, s) : launch_rows<kRowPlain, NVFP4_OUT_INT8>(a, vec, s);
}

}  // extern "C"
