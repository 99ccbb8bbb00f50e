// Rows between the products: the root-mean-square norm with the residual's
// addition, and rows in 8-bit integers with one scale each (of x itself, or of
// the SwiGLU of a [gate | up] row), which the 8-bit product takes.
//
//   h = x + residual, rounded to the residual's type and written back
//   y = h / sqrt(mean(h^2) + eps) * (weight + offset)
//   s = fl32(max |y| / 127),  code = y / s to the nearest integer, ties to even
//
// Everything between the inputs and the one rounding of a result is in fp64 (the
// vector units run it at the rate of fp32), so a code next to a border, and the
// scale, do not depend on how a sum was ordered: a result is the
// definition's, except within 2^-48 or so of a border.
//
// A row is read once: 64, 256 or 1024 threads hold up to 3 vectors of 8 values
// each (1536, 6144, 24576 values); longer rows are read again for each step.
#include "key_device.h"
#include "swiglu_device.h"

namespace nvfp4 {

enum { kRowNorm = 0, kRowPlain = 1, kRowSwiglu = 2 };
enum { kRowNone = -1 };  // a type: there is no such operand
constexpr int kRowMaxRows = (1 << 22) - 1;  // a launch has fewer than 2^32 threads
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
struct RowRaw {
    uint4 a, b;
};

template <int T, bool VEC>
__device__ __forceinline__ RowRaw row_load(const void* p, int type, long long at, int v, int t, int K) {
    const uint16_t* h = (const uint16_t*)p + at;
    const uint32_t* w = (const uint32_t*)p + at;
    RowRaw r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
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

// Its values as fp32 (exact); 0 past the row's end.
template <bool VEC>
__device__ __forceinline__ void row_values(const RowRaw& r, int type, float (&f)[8]) {
    const uint32_t u[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
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

// bf16 bits of an fp64 value, rounded once: to fp32 with the last bit set if
// anything was lost (so no tie appears or disappears), then to nearest even.
__device__ __forceinline__ uint32_t row_bf16(double d) {
    const float f = (float)d;
    uint32_t u = __float_as_uint(f);
    const double back = (double)f;
    if (d != d) return 0x7FC0u | (uint32_t)(__double2hiint(d) >> 31 << 15 & 0x8000);
    if (fabs(back) > fabs(d)) u -= 1;
    if (back != d) u |= 1;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

template <int T, bool VEC>
__device__ __forceinline__ void row_store(void* p, int type, long long at, int v, int t, int K, const double (&y)[8]) {
    uint16_t* h = (uint16_t*)p + at;
    float* w = (float*)p + at;
    if (VEC) {
        const int i = row_at<T, VEC>(v, t, 0);
        if (i >= K) return;
        if (type == NVFP4_OUT_BF16) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = row_bf16(y[2 * e]) | row_bf16(y[2 * e + 1]) << 16;
            *(uint4*)(h + i) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
            *(float4*)(w + i) = make_float4((float)y[0], (float)y[1], (float)y[2], (float)y[3]);
            *(float4*)(w + i + 4) = make_float4((float)y[4], (float)y[5], (float)y[6], (float)y[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = row_at<T, VEC>(v, t, e);
            if (i >= K) continue;
            if (type == NVFP4_OUT_BF16)
                h[i] = (uint16_t)row_bf16(y[e]);
            else
                w[i] = (float)y[e];
        }
    }
}

// Sum, or largest of values whose bits order them (magnitudes, NaN above all),
// over the T threads of a row, in all of them.
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

// Codes of 8 values: y * inv is off by 2^-52 of itself, so the nearest integer
// is q or, next to a border, its neighbour; what is left of y says which.
__device__ __forceinline__ void row_codes(const double (&y)[8], double s, double inv, uint32_t& lo, uint32_t& hi) {
    int c[8];
    const double half = 0.5 * s;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        double q = rint(y[e] * inv);
        const double rest = __builtin_fma(-q, s, y[e]);
        const int i = (int)q;
        const int up = rest > 0 ? 1 : -1;
        const bool move = fabs(rest) > half || (fabs(rest) == half && (i & 1));
        c[e] = min(127, max(-127, move ? i + up : i));
    }
    lo = (c[0] & 255) | (c[1] & 255) << 8 | (c[2] & 255) << 16 | (uint32_t)c[3] << 24;
    hi = (c[4] & 255) | (c[5] & 255) << 8 | (c[6] & 255) << 16 | (uint32_t)c[7] << 24;
}

// One row per T threads.  HELD: the row lies in registers between the steps.
template <int T, int MODE, int OUT, bool VEC, bool HELD>
__global__ __launch_bounds__(T < 256 ? 256 : T) void rows_kernel(RowArgs a) {
    constexpr int kPer = T < 256 ? 256 / T : 1;  // rows per workgroup
    __shared__ u64 lds[2][T / 64];
    const int t = threadIdx.x % T;
    const int row = blockIdx.x * kPer + threadIdx.x / T;
    if (T == 64 && row >= a.rows) return;  // whole wave (T = 64 meets no barrier)
    const int K = a.K;
    const int chunks = HELD ? 1 : (K + T * kRowVecs * 8 - 1) / (T * kRowVecs * 8);
    const long long xo = (long long)row * a.x_ld, ro = (long long)row * a.residual_ld;

    float h[kRowVecs][8], w[kRowVecs][8];  // norm: h and the weight; plain: x; SwiGLU: gate and up
    auto load = [&](int c, bool first) {
        RowRaw x[kRowVecs], r[kRowVecs], o[kRowVecs];
        const bool kept = MODE == kRowNorm && a.residual && !first;  // h as it was stored
        const int type = kept ? a.residual_type : a.x_type, other = MODE == kRowNorm ? a.weight_type : a.x_type;
        const bool adds = MODE == kRowNorm && a.residual && first;
#pragma unroll
        for (int j = 0; j < kRowVecs; ++j) x[j] = row_load<T, VEC>(kept ? a.residual_out : a.x, type, kept ? ro : xo, c * kRowVecs + j, t, K);
        if (adds)
#pragma unroll
            for (int j = 0; j < kRowVecs; ++j) r[j] = row_load<T, VEC>(a.residual, a.residual_type, ro, c * kRowVecs + j, t, K);
        if (MODE == kRowSwiglu || (MODE == kRowNorm && (HELD || !first)))
#pragma unroll
            for (int j = 0; j < kRowVecs; ++j)
                o[j] = row_load<T, VEC>(MODE == kRowNorm ? a.weight : a.x, other, MODE == kRowNorm ? 0 : xo + K, c * kRowVecs + j, t, K);
#pragma unroll
        for (int j = 0; j < kRowVecs; ++j) {
            row_values<VEC>(x[j], type, h[j]);
            if (adds) {
                float s[8];
                double sum[8];
                row_values<VEC>(r[j], a.residual_type, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum[e] = (double)h[j][e] + (double)s[e];
                    h[j][e] = a.residual_type == NVFP4_OUT_BF16 ? __uint_as_float(row_bf16(sum[e]) << 16) : (float)sum[e];
                }
                row_store<T, VEC>(a.residual_out, a.residual_type, ro, c * kRowVecs + j, t, K, sum);
            }
            if (MODE == kRowSwiglu || (MODE == kRowNorm && (HELD || !first))) row_values<VEC>(o[j], other, w[j]);
        }
    };

    double factor = 1.0;
    if (MODE == kRowNorm) {
        double sum = 0.0;
        for (int c = 0; c < chunks; ++c) {
            load(c, true);
#pragma unroll
            for (int j = 0; j < kRowVecs; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = __builtin_fma((double)h[j][e], (double)h[j][e], sum);
        }
        const u64 all = row_join<T>((u64)__double_as_longlong(wave_sumd(sum)), lds[0], [](u64 p, u64 q) {
            return (u64)__double_as_longlong(__longlong_as_double((long long)p) + __longlong_as_double((long long)q));
        });
        factor = 1.0 / sqrt(__longlong_as_double((long long)all) / K + a.eps);
    } else if (HELD) {
        load(0, true);
    }
    auto value = [&](int j, double (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double x = h[j][e];
            if (MODE == kRowNorm)
                y[e] = x * factor * ((double)w[j][e] + a.offset);
            else if (MODE == kRowSwiglu)
                y[e] = x * (double)w[j][e] / (1.0 + exp(-x));
            else
                y[e] = x;
        }
    };

    if (OUT != NVFP4_OUT_INT8) {
        for (int c = 0; c < chunks; ++c) {
            if (!HELD) load(c, false);
#pragma unroll
            for (int j = 0; j < kRowVecs; ++j) {
                double y[8];
                value(j, y);
                row_store<T, VEC>(a.out, OUT, (long long)row * a.out_ld, c * kRowVecs + j, t, K, y);
            }
        }
        return;
    }

    u64 most = 0;
    double y[kRowVecs][8];
    for (int c = 0; c < chunks; ++c) {
        if (!HELD) load(c, false);
#pragma unroll
        for (int j = 0; j < kRowVecs; ++j) {
            value(j, y[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (past the row's end: h is 0, and so is y unless the factor is NaN or infinite)
                const bool real = row_at<T, VEC>(c * kRowVecs + j, t, e) < K;
                const u64 b = (u64)__double_as_longlong(y[j][e]) & 0x7FFFFFFFFFFFFFFFull;
                most = max64(most, real ? b : 0);
            }
        }
    }
    most = row_join<T>(wave_max64(most), lds[1], [](u64 p, u64 q) { return max64(p, q); });
    const float s32 = (float)(__longlong_as_double((long long)most) / 127.0);
    if (t == 0) a.scale[row] = s32;
    const double s = s32, inv = 1.0 / s;
    const bool none = !(s32 > 0.f && s32 < __builtin_inff());
    int8_t* out = (int8_t*)a.out + (long long)row * a.out_ld;
    for (int c = 0; c < chunks; ++c) {
        if (!HELD) load(c, false);
#pragma unroll
        for (int j = 0; j < kRowVecs; ++j) {
            if (!HELD) value(j, y[j]);
            const int v = c * kRowVecs + j;
            if (row_at<T, VEC>(v, t, 0) >= K) continue;
            uint32_t lo = 0, hi = 0;
            if (!none) row_codes(y[j], s, inv, lo, hi);
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

template <int MODE, int OUT>
int launch_rows(const RowArgs& a, bool vec, hipStream_t s) {
    const int t = a.K <= 64 * kRowVecs * 8 ? 64 : a.K <= 256 * kRowVecs * 8 ? 256 : 1024;
    // (unaligned rows of 1024 threads would not fit the registers)
    const bool held = a.K <= t * kRowVecs * 8 && (vec || t < 1024);
    const unsigned grid = t == 64 ? (unsigned)((a.rows + 3) / 4) : (unsigned)a.rows;
#define NVFP4_ROWS(T, V, H)                                                                             \
    if (t == T && vec == V && held == H)                                                                \
        hipLaunchKernelGGL((rows_kernel<T, MODE, OUT, V, H>), dim3(grid), dim3(T < 256 ? 256 : T), 0, s, a);
    NVFP4_ROWS(64, true, true)
    NVFP4_ROWS(64, false, true)
    NVFP4_ROWS(256, true, true)
    NVFP4_ROWS(256, false, true)
    NVFP4_ROWS(1024, true, true)
    NVFP4_ROWS(1024, true, false)
    NVFP4_ROWS(1024, false, false)
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
