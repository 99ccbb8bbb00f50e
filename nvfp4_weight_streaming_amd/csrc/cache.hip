// The paged key/value cache: rotary append, page-table update, compaction.
//
// "Ignis" README, "What sets it apart" and "Models and artifacts", "What
// differs, side by side": eight lanes share one pool of key/value pages with a
// fixed budget; prefixes are cloned on the device.  Here a lane's tokens live
// in fixed-size pages named by its row of a page table; the pool is the
// caller's memory.
#include "cache.h"
#include "decode_device.h"

namespace nvfp4 {

int cache_view(const nvfp4_cache* c, int layer, CacheView* out) {
    if (!c) return set_error(NVFP4_EINVAL, "cache: NULL");
    if (c->layers < 1) return set_error(NVFP4_EINVAL, "cache.layers: %d < 1", c->layers);
    if (layer < -1 || layer >= c->layers)
        return set_error(NVFP4_EINVAL, "layer: %d outside [0, %d)", layer, c->layers);
    if (c->pages < 1) return set_error(NVFP4_EINVAL, "cache.pages: %d < 1", c->pages);
    if (c->kv_heads < 1 || c->kv_heads > 1024)
        return set_error(NVFP4_EINVAL, "cache.kv_heads: %d outside [1, 1024]", c->kv_heads);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return set_error(NVFP4_EUNSUPPORTED, "cache.head_dim: %d is not 64, 128 or 256", c->head_dim);
    int log_page = 0;
    while ((1 << log_page) < c->page_tokens && log_page < 10) ++log_page;
    if (c->page_tokens != (1 << log_page) || log_page < 4 || log_page > 8)
        return set_error(NVFP4_EUNSUPPORTED, "cache.page_tokens: %d is not 16, 32, 64, 128 or 256",
                         c->page_tokens);
    if (c->dtype != NVFP4_CACHE_BF16 && c->dtype != NVFP4_CACHE_E4M3)
        return set_error(NVFP4_EINVAL, "cache.dtype: %d", c->dtype);
    const bool fp8 = c->dtype == NVFP4_CACHE_E4M3;
    if (fp8 && (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || c->k_scale > 1e30f ||
                c->v_scale > 1e30f))
        return set_error(NVFP4_EINVAL, "cache.k_scale/v_scale: not positive numbers");
    if (!c->k_dev || ((uintptr_t)c->k_dev & 15))
        return set_error(NVFP4_EINVAL, "cache.k: NULL or not 16-byte aligned");
    if (!c->v_dev || ((uintptr_t)c->v_dev & 15))
        return set_error(NVFP4_EINVAL, "cache.v: NULL or not 16-byte aligned");
    const int64_t page = (int64_t)c->kv_heads * c->page_tokens * c->head_dim * (fp8 ? 1 : 2);
    const int64_t ps = c->page_stride ? c->page_stride : page;
    const int64_t ls = c->layer_stride ? c->layer_stride : ps * c->pages;
    if (ps < page || ps % 16 || ps > ((int64_t)1 << 40))
        return set_error(NVFP4_EINVAL, "cache.page_stride: %lld below a page's %lld bytes or not a multiple of 16",
                         (long long)ps, (long long)page);
    if (ls < page || ls % 16 || ls > ((int64_t)1 << 48))
        return set_error(NVFP4_EINVAL, "cache.layer_stride: %lld below a page's %lld bytes or not a multiple of 16",
                         (long long)ls, (long long)page);
    const int64_t at = layer > 0 ? (int64_t)layer * ls : 0;
    out->k = (uint8_t*)c->k_dev + at;
    out->v = (uint8_t*)c->v_dev + at;
    out->layer_stride = ls;
    out->page_stride = ps;
    out->layers = c->layers;
    out->pages = c->pages;
    out->kv_heads = c->kv_heads;
    out->dim = c->head_dim;
    out->log_page = log_page;
    out->k_scale = fp8 ? c->k_scale : 1.f;
    out->v_scale = fp8 ? c->v_scale : 1.f;
    out->fp8 = fp8;
    return NVFP4_OK;
}

int check_lanes(const CacheView& c, int lanes, const int* table, int table_ld) {
    if (lanes < 1 || lanes > kMaxLanes)
        return set_error(NVFP4_EINVAL, "lanes: %d outside [1, %d]", lanes, kMaxLanes);
    if (table_ld < 1 || ((int64_t)table_ld << c.log_page) > (1 << 30))
        return set_error(NVFP4_EINVAL, "table_ld: %d outside [1, 2^30 / page_tokens]", table_ld);
    if (!table || ((uintptr_t)table & 3))
        return set_error(NVFP4_EINVAL, "page_table: NULL or not 4-byte aligned");
    return NVFP4_OK;
}

// ---- rotary append -----------------------------------------------------------
//
// Pair i of a head (dims i and i + pairs, or 2 i and 2 i + 1) of the row at
// position p turns by the angle a = p inv_freq[i]:
//     (x, y) -> factor (x cos a - y sin a, x sin a + y cos a),
// p being the row's position on the pair's axis (time, height or width).  The
// angle is formed and reduced in fp64: exact for positions below 2^29 (29 + 24 bits),
// off by 2^-53 of it above; one rounding at the end.
//
// Bound by the bytes of the rows (read once, q and the cache written once) and,
// for a few rows, by latency: blocks of 256 threads take one row and a share of
// its heads, a thread one unit of dims with its cosines in registers.  K rows are
// written 4 or 8 bytes at a time.  V blocks are dim-major: a block takes an
// aligned group of 8 tokens and stores a dim's 8 tokens at once.
//
// Measured (48 q and 4 kv heads of 128): 2048 rows, three axes, into 8 bits, 57 MB:
// 15.2 us, 3.8 TB/s against 5.1 of a large copy; 64 rows into bf16 4.8 us.

struct AppendArgs {
    CacheView c;
    const uint16_t* qkv;
    long long ld;
    int q_heads, rows, lanes;
    const int* row_start;
    const int* ctx_len;
    const int* table;
    int table_ld;
    const int* pos;
    int axes;
    const float* inv_freq;
    const uint8_t* axis;
    int pairs, interleaved;
    float factor;
    uint16_t* q_out;
    long long q_ld;
    int shares;  // blocks per row for the rotated heads
    int wide;    // rows of qkv and q are 16-byte aligned
};

constexpr int kAppendThreads = 256;
constexpr int kAppendBatch = 4;

__device__ __forceinline__ float bf16_f32(uint16_t h) { return __uint_as_float((uint32_t)h << 16); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return f32_to_bf16_rne(a) | ((uint32_t)f32_to_bf16_rne(b) << 16);
}

// Four values to four consecutive dims of a K row (or q row).
__device__ __forceinline__ void put4(uint8_t* dst, bool fp8, float scale, const float* x) {
    if (fp8)
        *(uint32_t*)dst = e4m3x2(x[0] / scale, x[1] / scale) | (e4m3x2(x[2] / scale, x[3] / scale) << 16);
    else
        *(uint2*)dst = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

__device__ __forceinline__ void unpack4(const uint2& v, float* x) {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

// V of one aligned group of 8 tokens of a lane: group number `g` over all lanes'
// groups.  A thread takes two dims, and stores a dim's tokens of the group in one go.
__device__ __forceinline__ void append_v(const AppendArgs& a, int g) {
    const int lane = threadIdx.x & 63;
    int b = -1, before = 0, row0 = 0, rows = 0, ctx = 0;
    for (int b0 = 0; b0 < a.lanes && b < 0; b0 += 64) {
        int r0 = 0, n = 0, c = 0;
        if (b0 + lane < a.lanes) {
            r0 = a.row_start[b0 + lane];
            n = min(max(a.row_start[b0 + lane + 1] - r0, 0), a.rows - min(r0, a.rows));
            c = a.ctx_len[b0 + lane];
            if (r0 < 0 || c < 0) n = 0;
        }
        const int mine = n > 0 ? (int)((((long long)c + n - 1) >> 3) - (c >> 3)) + 1 : 0;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int u = __shfl_up(upto, d);
            upto += lane >= d ? u : 0;
        }
        const unsigned long long past = __ballot(before + upto > g);
        if (past) {
            const int first = __ffsll(past) - 1;
            b = b0 + first;
            before += __builtin_amdgcn_readlane(upto, first) - __builtin_amdgcn_readlane(mine, first);
            row0 = __builtin_amdgcn_readlane(r0, first);
            rows = __builtin_amdgcn_readlane(n, first);
            ctx = __builtin_amdgcn_readlane(c, first);
        } else {
            before += __builtin_amdgcn_readlane(upto, 63);
        }
    }
    if (b < 0) return;
    // tokens [p, p + count) of the lane, rows from r on
    const long long p = max(((long long)(ctx >> 3) + (g - before)) * 8, (long long)ctx);
    const int r = row0 + (int)(p - ctx), count = (int)min((p & ~7ll) + 8, (long long)ctx + rows) - (int)p;
    if ((p >> a.c.log_page) >= a.table_ld) return;
    const int id = a.table[(long long)b * a.table_ld + (p >> a.c.log_page)];
    if ((unsigned)id >= (unsigned)a.c.pages) return;
    const int dim = a.c.dim, es = a.c.fp8 ? 1 : 2;
    const uint16_t* src = a.qkv + (long long)r * a.ld + (long long)(a.q_heads + a.c.kv_heads) * dim;
    uint8_t* page = a.c.v + (long long)id * a.c.page_stride;
    const int off = (int)p & ((1 << a.c.log_page) - 1);
    for (int e = 2 * threadIdx.x; e < a.c.kv_heads * dim; e += 2 * kAppendThreads) {
        uint32_t in[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) in[i] = *(const uint32_t*)(src + (long long)min(i, count - 1) * a.ld + e);
        uint8_t* dst = page + v_element(a.c, e, off) * es;
#pragma unroll
        for (int half = 0; half < 2; ++half, dst += 16 * es) {  // the next dim is 16 tokens on
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = half ? in[i] >> 16 : in[i] & 0xFFFFu;
            if (a.c.fp8) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = e4m3x2(bf16_f32((uint16_t)h[2 * i]) / a.c.v_scale, bf16_f32((uint16_t)h[2 * i + 1]) / a.c.v_scale);
                if (count == 8)
                    *(uint2*)dst = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < count) dst[i] = (uint8_t)(w[i >> 1] >> (8 * (i & 1)));
            } else if (count == 8) {
                *(uint4*)dst = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < count) ((uint16_t*)dst)[i] = (uint16_t)h[i];
            }
        }
    }
}

__global__ __launch_bounds__(kAppendThreads) void append_kernel(AppendArgs a) {
    if ((int)blockIdx.x >= a.rows * a.shares) {
        append_v(a, blockIdx.x - a.rows * a.shares);
        return;
    }
    const int r = (int)(blockIdx.x / (unsigned)a.shares), share = blockIdx.x - r * a.shares;
    // A head is dim / 8 units of eight values: pairs / 4 of four pairs, then
    // copied vectors.  A thread keeps one unit, its cosines in registers, and
    // goes through the heads.
    const int dim = a.c.dim, log_units = dim == 64 ? 3 : dim == 128 ? 4 : 5;
    const int rot = a.pairs >> 2, unit = threadIdx.x & ((1 << log_units) - 1);
    const bool turns = unit < rot;
    const int dx = !turns ? 2 * a.pairs + 8 * (unit - rot) : a.interleaved ? 8 * unit : 4 * unit;
    const int dy = !turns || a.interleaved ? dx + 4 : dx + a.pairs;
    const int heads = a.q_heads + a.c.kv_heads, pass = kAppendThreads >> log_units;
    const int head0 = share * pass + (threadIdx.x >> log_units), step = a.shares * pass;
    const uint16_t* row = a.qkv + (long long)r * a.ld;
    const bool wide = a.wide && dy == dx + 4;  // eight values in a row, 16-byte aligned
    uint2 in[kAppendBatch][2];
    auto read = [&](int h0) {
#pragma unroll
        for (int j = 0; j < kAppendBatch; ++j) {
            const uint16_t* src = row + (long long)min(h0 + j * step, heads - 1) * dim;
            if (wide) {
                const uint4 v = *(const uint4*)(src + dx);
                in[j][0] = make_uint2(v.x, v.y);
                in[j][1] = make_uint2(v.z, v.w);
            } else {
                in[j][0] = *(const uint2*)(src + dx);
                in[j][1] = *(const uint2*)(src + dy);
            }
        }
    };
    // The row is on its way while its lane, page and cosines are worked out.
    read(head0);
    const int b = __builtin_amdgcn_readfirstlane(lane_of_row(a.row_start, a.lanes, r));
    if (b >= a.lanes) return;  // a row past the last lane's
    const int row0 = a.row_start[b], t = r - row0;
    if (t < 0) return;
    const int ctx = a.ctx_len[b];
    const long long p = (long long)ctx + t;  // this row's place in the lane
    const int page_tokens = 1 << a.c.log_page;
    const int* tab = a.table + (long long)b * a.table_ld;
    const int es = a.c.fp8 ? 1 : 2;
    const bool placed = ctx >= 0 && (p >> a.c.log_page) < a.table_ld;
    const int id = placed ? tab[p >> a.c.log_page] : -1;
    const bool stored = (unsigned)id < (unsigned)a.c.pages;

    __shared__ float cs[128], sn[128];
    for (int i = threadIdx.x; i < a.pairs; i += kAppendThreads) {
        const int ax = a.axis ? min((int)a.axis[i], a.axes - 1) : 0;
        const double turns = (double)a.pos[(long long)r * a.axes + ax] * (double)a.inv_freq[i] * 0.31830988618379067154;
        float s, c;
        sincospif((float)(turns - 2.0 * rint(0.5 * turns)), &s, &c);
        cs[i] = c * a.factor;
        sn[i] = s * a.factor;
    }
    __syncthreads();

    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c[i] = turns ? cs[4 * unit + i] : 1.f;
        s[i] = turns ? sn[4 * unit + i] : 0.f;
    }
    const bool flat = a.interleaved && turns;  // pairs lie next to each other
    uint8_t* page = a.c.k + (long long)(stored ? id : 0) * a.c.page_stride;
    const int off = (int)p & (page_tokens - 1);
    for (int h0 = head0; h0 < heads; h0 += kAppendBatch * step) {
        if (h0 != head0) read(h0);
#pragma unroll
        for (int j = 0; j < kAppendBatch; ++j) {
            const int head = h0 + j * step;
            if (head >= heads) break;
            const bool is_q = head < a.q_heads;
            if (!is_q && !stored) continue;
            const bool fp8 = !is_q && a.c.fp8;
            uint8_t* dst = is_q ? (uint8_t*)(a.q_out + (long long)r * a.q_ld + (long long)head * dim)
                                : page + ((((long long)(head - a.q_heads) << a.c.log_page) + off) * dim) * es;
            const int de = fp8 ? 1 : 2;
            float v[8];
            unpack4(in[j][0], v);
            unpack4(in[j][1], v + 4);
            if (turns) {
                float o1[4], o2[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = flat ? v[2 * i] : v[i], y = flat ? v[2 * i + 1] : v[4 + i];
                    o1[i] = x * c[i] - y * s[i];
                    o2[i] = x * s[i] + y * c[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i] = flat ? (i & 1 ? o2[i >> 1] : o1[i >> 1]) : o1[i];
                    v[4 + i] = flat ? (i & 1 ? o2[2 + (i >> 1)] : o1[2 + (i >> 1)]) : o2[i];
                }
            }
            if (wide && !fp8) {
                *(uint4*)(dst + dx * 2) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
            } else {
                put4(dst + dx * de, fp8, a.c.k_scale, v);
                put4(dst + dy * de, fp8, a.c.k_scale, v + 4);
            }
        }
    }
}

// ---- compaction of accepted drafts ---------------------------------------------
//
// Token ctx + path[j] of a lane moves to ctx + j, j < accepted.  A block takes
// one lane, layer, kv head and side (K or V), reads every source into LDS, and
// writes after a barrier, so a path in any order is right.
//
// Tokens are numbered in slots from the start of the 16-token block that ctx lies
// in; the 64 drafted ones take at most five blocks, each of which lies in one page.
// K moves whole rows.  V blocks are dim-major: the blocks with a source or a
// destination are read whole (runs of 16 x dim values) and the destinations'
// vectors put together in LDS, so memory sees only 16-byte accesses.
//
// Bound by latency for few lanes (lengths, then table, then data: 8 lanes of 8
// drafts, 16 layers, 5.0 us) and by bytes for many (64 lanes of 64, 8 bits, 78 MB:
// 19 us, 4.1 TB/s against 5.1 of a large copy).

struct CompactArgs {
    CacheView c;
    int lanes;
    const int* ctx_len;
    const int* table;
    int table_ld;
    const int* path;
    int path_ld;
    const int* accepted;
};

constexpr int kCompactThreads = 128;
constexpr int kCompactBlocks = NVFP4_TREE_MAX_ROWS / 16 + 1;

template <typename T>
__global__ __launch_bounds__(kCompactThreads) void compact_kernel(CompactArgs a) {
    extern __shared__ __align__(16) uint8_t lds[];
    __shared__ long long block_at[kCompactBlocks];       // byte offset of the slots' 16 tokens; -1: no page
    __shared__ uint8_t source[16 * kCompactBlocks];      // slot that a slot's content comes from
    __shared__ int ends[2];                              // blocks with a source or destination; rows to read
    const int b = (int)(blockIdx.x / (unsigned)a.c.kv_heads), h = blockIdx.x - b * a.c.kv_heads;
    const bool is_v = blockIdx.z != 0;
    const int dim = a.c.dim, page_mask = (1 << a.c.log_page) - 1;
    const int count = min(max(a.accepted[b], 0), min(a.path_ld, NVFP4_TREE_MAX_ROWS));
    if (count == 0) return;
    const int ctx = a.ctx_len[b], first = ctx & 15;
    if (ctx < 0) return;
    const int token_bytes = dim * (int)sizeof(T);  // of K; V's 16 tokens take as much as 16 of K
    if (threadIdx.x < 64) {  // the first wave works the moves out
        const int j = threadIdx.x;
        const int s = j < count ? a.path[(long long)b * a.path_ld + j] : -1;
        long long at = -1;
        if (j < kCompactBlocks) {
            const long long p = (long long)(ctx >> 4) * 16 + 16 * j;
            if ((p >> a.c.log_page) < a.table_ld) {
                const int id = a.table[(long long)b * a.table_ld + (p >> a.c.log_page)];
                if ((unsigned)id < (unsigned)a.c.pages)
                    at = (long long)id * a.c.page_stride + (long long)((int)p & page_mask) * token_bytes;
            }
            block_at[j] = at;
        }
        const int from = first + s, to = first + j;
        // (every lane takes part in the exchange)
        const int has = at >= 0 ? 1 : 0, has_from = __shfl(has, (from & 127) >> 4), has_to = __shfl(has, (to & 127) >> 4);
        const bool moves = j < count && s >= 0 && s < NVFP4_TREE_MAX_ROWS && s != j && has_from && has_to;
        for (int i = j; i < 16 * kCompactBlocks; i += 64) source[i] = (uint8_t)i;
        __builtin_amdgcn_wave_barrier();
        if (moves) source[to] = (uint8_t)from;
        int last = moves ? max(from, to) : -1;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) last = max(last, __shfl_xor(last, d));
        if (j == 0) ends[0] = (last + 16) >> 4;  // 0: nothing moves
    }
    __syncthreads();
    const int blocks = ends[0];
    if (blocks == 0) return;
    const long long head = ((long long)h * token_bytes) << a.c.log_page;
    uint8_t* base = (is_v ? a.c.v : a.c.k) + (long long)blockIdx.y * a.c.layer_stride + head;
    uint4* buf = (uint4*)lds;
    const int log_vecs = 31 - __clz(token_bytes / 16), vecs = 1 << log_vecs;  // 16-byte vectors of a token
    if (!is_v) {
        for (int e = threadIdx.x; e < count << log_vecs; e += kCompactThreads) {
            const int to = first + (e >> log_vecs), k = e & (vecs - 1), from = source[to];
            if (from != to) buf[e] = *(const uint4*)(base + block_at[from >> 4] + (from & 15) * token_bytes + 16 * k);
        }
        __syncthreads();
        for (int e = threadIdx.x; e < count << log_vecs; e += kCompactThreads) {
            const int to = first + (e >> log_vecs), k = e & (vecs - 1);
            if (source[to] != to) *(uint4*)(base + block_at[to >> 4] + (to & 15) * token_bytes + 16 * k) = buf[e];
        }
        return;
    }
    const int log_block = log_vecs + 4;  // vectors of a V block
    for (int e = threadIdx.x; e < blocks << log_block; e += kCompactThreads) {
        const long long at = block_at[e >> log_block];
        if (at >= 0) buf[e] = *(const uint4*)(base + at + 16 * (e & ((1 << log_block) - 1)));
    }
    __syncthreads();
    // A vector is 16 / sizeof(T) tokens of one dim.
    constexpr int kPer = 16 / (int)sizeof(T);
    const T* in = (const T*)lds;
    const int out_blocks = (first + count + 15) >> 4;
    for (int e = threadIdx.x; e < out_blocks << log_block; e += kCompactThreads) {
        const int blk = e >> log_block, v = e & ((1 << log_block) - 1);
        const int d = v / (16 / kPer), slot0 = 16 * blk + v % (16 / kPer) * kPer;
        union {
            uint4 vec;
            T x[kPer];
        } o;
        bool changed = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int from = source[slot0 + i];
            changed |= from != slot0 + i;
            o.x[i] = in[((from >> 4) * dim + d) * 16 + (from & 15)];
        }
        if (changed) *(uint4*)(base + block_at[blk] + 16 * v) = o.vec;
    }
}

// ---- page-table update -------------------------------------------------------------
//
// See nvfp4_cache_update in the header for the rules.  Whole numbers only, and
// the answer is unique: fresh pages are the lowest-numbered unreferenced ones,
// handed out in lane order.  Phases:
//   1. refs_out = refs_in                                        (count kernel, phase 0)
//   2. less the old rows' entries, plus the inherited ones       (integer atomics)
//   3. one workgroup: which lanes copy their last page, how many fresh pages each
//      lane needs, the free pages in order, and their assignment
//   4. page copies, all layers.
// Integer sums do not depend on the order of the atomics.

struct UpdateArgs {
    CacheView c;
    int lanes_in, lanes_out, table_ld;
    const int* table_in;
    const int* len_in;
    const int* refs_in;
    const int* parent;
    const int* keep;     // null: all
    const int* reserve;  // null: none
    int* table_out;
    int* len_out;
    int* refs_out;
    int* short_out;
    // workspace
    int* part_count;  // [pages] new lanes that hold the page as their partly filled last one
    int* part_first;  // [pages] the lowest of them
    int2* copies;     // [lanes_out] source and destination page, -1 for none
};

struct NewLane {
    int parent, len, held, upto;
};

__device__ __forceinline__ NewLane new_lane(const UpdateArgs& a, int i) {
    NewLane n;
    const int p = a.parent[i];
    const bool has = p >= 0 && p < a.lanes_in;
    n.parent = has ? p : -1;
    const int page_mask = (1 << a.c.log_page) - 1;
    const int most = a.table_ld << a.c.log_page;
    int len = has ? min(max(a.len_in[p], 0), most) : 0;
    if (a.keep) len = min(len, max(a.keep[i], 0));
    n.len = len;
    n.held = (len + page_mask) >> a.c.log_page;
    const long long want = (long long)len + (a.reserve ? max(a.reserve[i], 0) : 0);
    n.upto = (int)min((want + page_mask) >> a.c.log_page, (long long)a.table_ld);
    return n;
}

__device__ __forceinline__ bool is_page(const UpdateArgs& a, int id) {
    return (unsigned)id < (unsigned)a.c.pages;
}

__global__ __launch_bounds__(256) void update_init_kernel(UpdateArgs a) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < a.c.pages) {
        a.refs_out[i] = a.refs_in[i];
        a.part_count[i] = 0;
        a.part_first[i] = 0x7FFFFFFF;
    }
}

// Old rows (blocks [0, lanes_in)) give their entries back, new rows take the
// inherited ones.
__global__ __launch_bounds__(256) void update_count_kernel(UpdateArgs a) {
    if ((int)blockIdx.x < a.lanes_in) {
        const int* row = a.table_in + (long long)blockIdx.x * a.table_ld;
        for (int j = threadIdx.x; j < a.table_ld; j += 256)
            if (is_page(a, row[j])) atomicSub(a.refs_out + row[j], 1);
        return;
    }
    const int i = blockIdx.x - a.lanes_in;
    const NewLane n = new_lane(a, i);
    const int* row = a.table_in + (long long)max(n.parent, 0) * a.table_ld;
    int* out = a.table_out + (long long)i * a.table_ld;
    for (int j = threadIdx.x; j < a.table_ld; j += 256) {
        const int id = j < n.held && is_page(a, row[j]) ? row[j] : -1;
        out[j] = id;
        if (id >= 0) {
            atomicAdd(a.refs_out + id, 1);
            if (j == n.held - 1 && (n.len & ((1 << a.c.log_page) - 1))) {
                atomicAdd(a.part_count + id, 1);
                atomicMin(a.part_first + id, i);
            }
        }
    }
    if (threadIdx.x == 0) a.len_out[i] = n.len;
}

constexpr int kAssignThreads = 1024;

// Exclusive sum over the block's threads and the total.
__device__ __forceinline__ int block_scan(int v, int* lds, int* total) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(s, d);
        s += lane >= d ? u : 0;
    }
    if (lane == 63) lds[wave] = s;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kAssignThreads / 64; ++w) {
        const int x = lds[w];
        before += w < wave ? x : 0;
        all += x;
    }
    __syncthreads();
    *total = all;
    return before + s - v;
}

// Fresh page number r (in lane order, the copy of a lane's last page before its
// reserved ones) is the r-th lowest page with no reference.  Lanes are taken
// 1024 at a time; `slots` (workspace, by request number) maps a request to the
// table entry it fills.
__global__ __launch_bounds__(kAssignThreads) void update_assign_kernel(UpdateArgs a, int* slots) {
    __shared__ int lds[kAssignThreads / 64];
    int requests = 0;
    for (int i0 = 0; i0 < a.lanes_out; i0 += kAssignThreads) {
        const int i = i0 + (int)threadIdx.x;
        int need = 0;
        bool copy = false;
        NewLane n = {-1, 0, 0, 0};
        int last = -1;
        if (i < a.lanes_out) {
            n = new_lane(a, i);
            if (n.len & ((1 << a.c.log_page) - 1)) last = a.table_out[(long long)i * a.table_ld + n.held - 1];
            copy = last >= 0 && !(a.part_count[last] == a.refs_out[last] && a.part_first[last] == i);
            need = (copy ? 1 : 0) + max(n.upto - n.held, 0);
        }
        int all;
        const int first = requests + block_scan(need, lds, &all);
        if (i < a.lanes_out) {
            a.copies[i] = make_int2(copy ? last : -1, -1);
            const int entry0 = n.held - (copy ? 1 : 0);
            for (int j = 0; j < need; ++j) {
                // entries of a lane are consecutive: (lane, entry) as an index
                slots[2 * (size_t)(first + j)] = i;
                slots[2 * (size_t)(first + j) + 1] = entry0 + j;
            }
        }
        requests += all;
    }
    __syncthreads();
    // Free pages in order.  References are read before any is changed: copies'
    // sources have at least one reference, so they are never free here.
    int given = 0;
    for (int p0 = 0; p0 < a.c.pages && given < requests; p0 += kAssignThreads) {
        const int p = p0 + (int)threadIdx.x;
        const int free = p < a.c.pages && a.refs_out[p] == 0 ? 1 : 0;
        int all;
        const int r = given + block_scan(free, lds, &all);
        if (free && r < requests) {
            const int i = slots[2 * (size_t)r], e = slots[2 * (size_t)r + 1];
            a.table_out[(long long)i * a.table_ld + e] = p;
            a.refs_out[p] = 1;
        }
        given += all;
    }
    if (threadIdx.x == 0) *a.short_out = max(requests - given, 0);
    __syncthreads();
    for (int r = min(given, requests) + (int)threadIdx.x; r < requests; r += kAssignThreads)
        a.table_out[(long long)slots[2 * (size_t)r] * a.table_ld + slots[2 * (size_t)r + 1]] = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.lanes_out; i += kAssignThreads) {
        const int src = a.copies[i].x;
        if (src < 0) continue;
        atomicSub(a.refs_out + src, 1);
        const NewLane n = new_lane(a, i);
        a.copies[i].y = a.table_out[(long long)i * a.table_ld + n.held - 1];
    }
}

// Phases 1 to 3 in one workgroup, counts in LDS, for small calls: one launch instead of
// three.  Lanes' partly filled last pages are compared with each other directly.
//
// Its time grows with the table entries (old and new), pages and new lanes, about as
// 2 entries + pages + 256 lanes; that of the three kernels hardly does, but their two
// further launches take the host 5.4 us (14.0 and 19.4 for a call).  Times with the page
// copies of one layer in a captured graph, one workgroup and three kernels, in us: 8
// lanes of 70 pages, 700 in the pool 7.3 and 11.6; 8 of 1024, 8400 10.1 and 13.6; 64 of
// 128, 8400 12.1 and 12.3; 128 of 64, 8400 14.3 and 12.5; 64 of 257, 16832 16.0 and 12.9;
// 256 of 32, 8400 18.9 and 12.8; 64 of 512, 32768 22.4 and 14.3; 1024 of 8, 10300 45 and
// 16.  So they meet near a sum of 50000 in a graph and of 140000 call by call; the
// bound is their geometric mean.  (What the counts may take of LDS bounds the pages.)
constexpr int kFusedWork = 81920, kFusedPages = 32768, kFusedLanes = kFusedWork / 256;
__global__ __launch_bounds__(kAssignThreads) void update_fused_kernel(UpdateArgs a, int* slots) {
    extern __shared__ int refs[];  // [pages]
    __shared__ int lasts[kFusedLanes], parents[kFusedLanes], lens[kFusedLanes];
    __shared__ int lds[kAssignThreads / 64];
    // Loads in flight at once.  More wait longer for less where a call has few entries,
    // fewer leave loads to wait for where it has many (with the page copies): 8 lanes of
    // 70 pages 8.5 us with 8, 7.2 with 2, 7.1 with 1; 64 of 128 pages 12.1, 12.1 and 12.8.
    constexpr int kBatch = 2;
    const int tid = threadIdx.x, i = tid;
    const bool lane = i < a.lanes_out;
    NewLane n = {-1, 0, 0, 0};
    if (lane) {
        n = new_lane(a, i);
        parents[i] = n.parent;
        lens[i] = n.len;
        lasts[i] = -1;
        a.len_out[i] = n.len;
    }
    const int page_mask = (1 << a.c.log_page) - 1;
    for (int p0 = 0; p0 < a.c.pages; p0 += kBatch * kAssignThreads) {
        int v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) v[j] = a.refs_in[min(p0 + j * kAssignThreads + tid, a.c.pages - 1)];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (p0 + j * kAssignThreads + tid < a.c.pages) refs[p0 + j * kAssignThreads + tid] = v[j];
    }
    __syncthreads();
    // Old entries give their references back, inherited ones take theirs.
    const int old = a.lanes_in * a.table_ld, fresh = a.lanes_out * a.table_ld;
    // Row and column of this thread's next entry, carried on (a division for each entry:
    // 12.5 us for 64 lanes of 128 pages, 12.1 without).
    int next_row = (int)((unsigned)tid / (unsigned)a.table_ld), next_col = tid - next_row * a.table_ld;
    const int row_step = (int)((unsigned)kAssignThreads / (unsigned)a.table_ld), col_step = kAssignThreads - row_step * a.table_ld;
    for (int e0 = 0; e0 < max(old, fresh); e0 += kBatch * kAssignThreads) {
        int gone[kBatch], kept[kBatch], row[kBatch], col[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int e = e0 + j * kAssignThreads + tid;
            gone[j] = a.table_in[min(e, old - 1)];
            row[j] = min(next_row, a.lanes_out - 1);
            col[j] = next_col;
            next_row += row_step;
            next_col += col_step;
            if (next_col >= a.table_ld) {
                next_col -= a.table_ld;
                ++next_row;
            }
            kept[j] = a.table_in[(long long)max(parents[row[j]], 0) * a.table_ld + col[j]];
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int e = e0 + j * kAssignThreads + tid;
            if (e < old && is_page(a, gone[j])) atomicSub(&refs[gone[j]], 1);
            if (e < fresh) {
                const int len = lens[row[j]], held = (len + page_mask) >> a.c.log_page;
                const int id = col[j] < held && is_page(a, kept[j]) ? kept[j] : -1;
                a.table_out[e] = id;
                if (id >= 0) atomicAdd(&refs[id], 1);
                if (col[j] == held - 1 && (len & page_mask)) lasts[row[j]] = id;
            }
        }
    }
    __syncthreads();
    int last = -1, same = 0, lowest = i;
    if (lane) last = lasts[i];
    for (int j = 0; j < a.lanes_out; ++j) {
        const bool hit = lasts[j] == last;
        same += hit ? 1 : 0;
        lowest = hit ? min(lowest, j) : lowest;
    }
    const bool copy = last >= 0 && !(same == refs[max(last, 0)] && lowest == i);
    const int need = lane ? (copy ? 1 : 0) + max(n.upto - n.held, 0) : 0;
    int requests;
    const int first = block_scan(need, lds, &requests);
    const int entry0 = n.held - (copy ? 1 : 0);
    for (int j = 0; j < need; ++j) {
        slots[2 * (size_t)(first + j)] = i;
        slots[2 * (size_t)(first + j) + 1] = entry0 + j;
    }
    __syncthreads();
    int given = 0;
    for (int p0 = 0; p0 < a.c.pages && given < requests; p0 += kAssignThreads) {
        const int p = p0 + tid;
        const int free = p < a.c.pages && refs[p] == 0 ? 1 : 0;
        int all;
        const int r = given + block_scan(free, lds, &all);
        if (free && r < requests) {
            a.table_out[(long long)slots[2 * (size_t)r] * a.table_ld + slots[2 * (size_t)r + 1]] = p;
            refs[p] = 1;
        }
        given += all;
    }
    if (tid == 0) *a.short_out = max(requests - given, 0);
    for (int r = min(given, requests) + tid; r < requests; r += kAssignThreads)
        a.table_out[(long long)slots[2 * (size_t)r] * a.table_ld + slots[2 * (size_t)r + 1]] = -1;
    __syncthreads();
    if (copy) atomicSub(&refs[last], 1);
    if (lane) a.copies[i] = make_int2(copy ? last : -1, copy ? a.table_out[(long long)i * a.table_ld + n.held - 1] : -1);
    __syncthreads();
    for (int p = tid; p < a.c.pages; p += kAssignThreads) a.refs_out[p] = refs[p];
}

// Copies K and V of the pages that became a lane's own: block (lane, layer, part).
// (8 lanes of 16 layers, 21 MB read and written: 6.7 us, launch and ramp included.)
__global__ __launch_bounds__(256) void update_copy_kernel(UpdateArgs a, long long page_bytes) {
    const int2 c = a.copies[blockIdx.x];
    if (c.x < 0 || c.y < 0) return;
    const long long at = (long long)blockIdx.y * a.c.layer_stride;
    uint8_t* base = ((blockIdx.z & 1) ? a.c.v : a.c.k) + at;
    const uint4* src = (const uint4*)(base + (long long)c.x * a.c.page_stride);
    uint4* dst = (uint4*)(base + (long long)c.y * a.c.page_stride);
    const int parts = gridDim.z >> 1, part = blockIdx.z >> 1;
    const long long vecs = page_bytes / 16;
    for (long long e = (long long)part * 256 + threadIdx.x; e < vecs; e += (long long)parts * 256) dst[e] = src[e];
}

size_t round16(size_t x) { return (x + 15) / 16 * 16; }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int nvfp4_cache_append(const nvfp4_cache* cache, int layer, const uint16_t* qkv_dev, int64_t qkv_ld,
                       int rows, int q_heads, int lanes, const int* row_start_dev,
                       const int* ctx_len_dev, const int* page_table_dev, int table_ld,
                       const nvfp4_rotary* rotary, uint16_t* q_out_dev, int64_t q_ld, void* stream) {
    clear_error();
    AppendArgs a;
    int st = cache_view(cache, layer, &a.c);
    if (st) return st;
    if (layer < 0) return set_error(NVFP4_EINVAL, "layer: %d < 0", layer);
    const int dim = a.c.dim;
    if (rows < 0 || rows > (1 << 24)) return set_error(NVFP4_EINVAL, "rows: %d outside [0, 2^24]", rows);
    if (q_heads < 1 || q_heads > 65536) return set_error(NVFP4_EINVAL, "q_heads: %d outside [1, 65536]", q_heads);
    if ((st = check_lanes(a.c, lanes, page_table_dev, table_ld))) return st;
    const int64_t width = (int64_t)(q_heads + 2 * a.c.kv_heads) * dim;
    if (qkv_ld < width || qkv_ld % 4)
        return set_error(NVFP4_EINVAL, "qkv_ld: %lld below %lld or not a multiple of 4", (long long)qkv_ld, (long long)width);
    if (q_ld < (int64_t)q_heads * dim || q_ld % 4)
        return set_error(NVFP4_EINVAL, "q_ld: %lld below %lld or not a multiple of 4", (long long)q_ld, (long long)q_heads * dim);
    if (!row_start_dev || ((uintptr_t)row_start_dev & 3)) return set_error(NVFP4_EINVAL, "row_start: NULL or not 4-byte aligned");
    if (!ctx_len_dev || ((uintptr_t)ctx_len_dev & 3)) return set_error(NVFP4_EINVAL, "ctx_len: NULL or not 4-byte aligned");
    if (!rotary) return set_error(NVFP4_EINVAL, "rotary: NULL");
    if (rotary->pairs < 0 || rotary->pairs > dim / 2 || rotary->pairs % 4)
        return set_error(NVFP4_EINVAL, "rotary.pairs: %d is not a multiple of 4 up to %d", rotary->pairs, dim / 2);
    if (rotary->axes < 1 || rotary->axes > 8) return set_error(NVFP4_EINVAL, "rotary.axes: %d outside [1, 8]", rotary->axes);
    if (rows == 0) return NVFP4_OK;  // (the rows' pointers may be NULL: empty tensors have no address)
    if (!qkv_dev || ((uintptr_t)qkv_dev & 7)) return set_error(NVFP4_EINVAL, "qkv: NULL or not 8-byte aligned");
    if (!q_out_dev || ((uintptr_t)q_out_dev & 7)) return set_error(NVFP4_EINVAL, "q_out: NULL or not 8-byte aligned");
    if (rotary->pairs) {
        if (!rotary->positions_dev || ((uintptr_t)rotary->positions_dev & 3)) return set_error(NVFP4_EINVAL, "rotary.positions: NULL or not 4-byte aligned");
        if (!rotary->inv_freq_dev || ((uintptr_t)rotary->inv_freq_dev & 3)) return set_error(NVFP4_EINVAL, "rotary.inv_freq: NULL or not 4-byte aligned");
    }
    a.qkv = qkv_dev;
    a.ld = qkv_ld;
    a.q_heads = q_heads;
    a.rows = rows;
    a.lanes = lanes;
    a.row_start = row_start_dev;
    a.ctx_len = ctx_len_dev;
    a.table = page_table_dev;
    a.table_ld = table_ld;
    a.pos = rotary->positions_dev;
    a.axes = rotary->axes;
    a.inv_freq = rotary->inv_freq_dev;
    a.axis = rotary->pair_axis_dev;
    a.pairs = rotary->pairs;
    a.interleaved = rotary->interleaved != 0;
    a.factor = rotary->factor;
    a.q_out = q_out_dev;
    a.q_ld = q_ld;
    // One head per thread while the rows alone do not fill the card.
    const int pass = kAppendThreads / (dim / 8);
    const int most = (q_heads + a.c.kv_heads + pass - 1) / pass;
    int shares = (8 * device_cus() + rows - 1) / rows;
    a.shares = shares < 1 ? 1 : shares > most ? most : shares;
    a.wide = (((uintptr_t)qkv_dev | (uintptr_t)q_out_dev) & 15) == 0 && qkv_ld % 8 == 0 && q_ld % 8 == 0;
    // V: a lane's rows cover at most rows / 8 + 2 groups of 8 tokens.
    const long long blocks = (long long)rows * a.shares + rows / 8 + 2ll * (lanes < rows ? lanes : rows);
    if (blocks * kAppendThreads > 0xFFFFFFFFll)
        return set_error(NVFP4_EUNSUPPORTED, "rows: %d take more than 2^32 - 1 threads", rows);
    hipLaunchKernelGGL(append_kernel, dim3((unsigned)blocks), dim3(kAppendThreads), 0, (hipStream_t)stream, a);
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

int nvfp4_cache_compact(const nvfp4_cache* cache, int lanes, const int* ctx_len_dev,
                        const int* page_table_dev, int table_ld, const int* path_dev, int path_ld,
                        const int* accepted_dev, void* stream) {
    clear_error();
    CompactArgs a;
    int st = cache_view(cache, -1, &a.c);
    if (st) return st;
    if ((st = check_lanes(a.c, lanes, page_table_dev, table_ld))) return st;
    if (path_ld < 1) return set_error(NVFP4_EINVAL, "path_ld: %d < 1", path_ld);
    if (!ctx_len_dev || ((uintptr_t)ctx_len_dev & 3)) return set_error(NVFP4_EINVAL, "ctx_len: NULL or not 4-byte aligned");
    if (!path_dev || ((uintptr_t)path_dev & 3)) return set_error(NVFP4_EINVAL, "path: NULL or not 4-byte aligned");
    if (!accepted_dev || ((uintptr_t)accepted_dev & 3)) return set_error(NVFP4_EINVAL, "accepted: NULL or not 4-byte aligned");
    if (a.c.layers > 65535) return set_error(NVFP4_EUNSUPPORTED, "cache.layers: %d above 65535", a.c.layers);
    if ((int64_t)lanes * a.c.kv_heads * kCompactThreads > 0xFFFFFFFFll)
        return set_error(NVFP4_EUNSUPPORTED, "lanes: %d lanes of %d kv heads take more than 2^32 - 1 threads", lanes, a.c.kv_heads);
    a.lanes = lanes;
    a.ctx_len = ctx_len_dev;
    a.table = page_table_dev;
    a.table_ld = table_ld;
    a.path = path_dev;
    a.path_ld = path_ld;
    a.accepted = accepted_dev;
    const dim3 grid((unsigned)lanes * a.c.kv_heads, (unsigned)a.c.layers, 2);
    const size_t bytes = (size_t)kCompactBlocks * 16 * a.c.dim * (a.c.fp8 ? 1 : 2);
    if (a.c.fp8)
        hipLaunchKernelGGL((compact_kernel<uint8_t>), grid, dim3(kCompactThreads), bytes, (hipStream_t)stream, a);
    else
        hipLaunchKernelGGL((compact_kernel<uint16_t>), grid, dim3(kCompactThreads), bytes, (hipStream_t)stream, a);
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

size_t nvfp4_cache_update_workspace_bytes(int pages, int lanes_out, int table_ld) {
    if (pages < 1 || lanes_out < 1 || table_ld < 1) return 0;
    return round16((size_t)pages * 8) + round16((size_t)lanes_out * sizeof(int2)) +
           round16((size_t)lanes_out * table_ld * 8);
}

int nvfp4_cache_update(const nvfp4_cache* cache, int lanes_in, const int* table_in_dev,
                       const int* len_in_dev, const int* refs_in_dev, int table_ld, int lanes_out,
                       const int* parent_dev, const int* keep_dev, const int* reserve_dev,
                       int* table_out_dev, int* len_out_dev, int* refs_out_dev, int* short_dev,
                       void* workspace_dev, size_t workspace_bytes, void* stream) {
    clear_error();
    UpdateArgs a;
    int st = cache_view(cache, -1, &a.c);
    if (st) return st;
    if ((st = check_lanes(a.c, lanes_in, table_in_dev, table_ld))) return st;
    if (lanes_out < 1 || lanes_out > kMaxLanes)
        return set_error(NVFP4_EINVAL, "lanes_out: %d outside [1, %d]", lanes_out, kMaxLanes);
    if ((int64_t)lanes_out * table_ld > 0x7FFFFFFF)  // (requests for pages are counted in 32 bits)
        return set_error(NVFP4_EUNSUPPORTED, "lanes_out: %d lanes of %d pages exceed 2^31 - 1 table entries", lanes_out, table_ld);
    if (a.c.layers > 65535) return set_error(NVFP4_EUNSUPPORTED, "cache.layers: %d above 65535", a.c.layers);
    const struct { const void* p; const char* name; int may; } ptrs[] = {
        {len_in_dev, "len_in", 0}, {refs_in_dev, "refs_in", 0}, {parent_dev, "parent", 0},
        {keep_dev, "keep", 1}, {reserve_dev, "reserve", 1}, {table_out_dev, "table_out", 0},
        {len_out_dev, "len_out", 0}, {refs_out_dev, "refs_out", 0}, {short_dev, "short", 0}};
    for (const auto& x : ptrs)
        if ((!x.p && !x.may) || ((uintptr_t)x.p & 3))
            return set_error(NVFP4_EINVAL, "%s: NULL or not 4-byte aligned", x.name);
    if (table_out_dev == table_in_dev) return set_error(NVFP4_EINVAL, "table_out: is table_in");
    if (len_out_dev == len_in_dev) return set_error(NVFP4_EINVAL, "len_out: is len_in");
    if (refs_out_dev == refs_in_dev) return set_error(NVFP4_EINVAL, "refs_out: is refs_in");
    const size_t need = nvfp4_cache_update_workspace_bytes(a.c.pages, lanes_out, table_ld);
    if (workspace_bytes < need) return set_error(NVFP4_EINVAL, "workspace_bytes: %zu < %zu needed", workspace_bytes, need);
    if (!workspace_dev || ((uintptr_t)workspace_dev & 15)) return set_error(NVFP4_EINVAL, "workspace: NULL or not 16-byte aligned");
    a.lanes_in = lanes_in;
    a.lanes_out = lanes_out;
    a.table_ld = table_ld;
    a.table_in = table_in_dev;
    a.len_in = len_in_dev;
    a.refs_in = refs_in_dev;
    a.parent = parent_dev;
    a.keep = keep_dev;
    a.reserve = reserve_dev;
    a.table_out = table_out_dev;
    a.len_out = len_out_dev;
    a.refs_out = refs_out_dev;
    a.short_out = short_dev;
    char* ws = (char*)workspace_dev;
    a.part_count = (int*)ws;
    a.part_first = a.part_count + a.c.pages;
    ws += round16((size_t)a.c.pages * 8);
    a.copies = (int2*)ws;
    ws += round16((size_t)lanes_out * sizeof(int2));
    int* slots = (int*)ws;
    hipStream_t s = (hipStream_t)stream;
    if (a.c.pages <= kFusedPages &&
        2 * ((long long)lanes_in + lanes_out) * table_ld + a.c.pages + 256ll * lanes_out <= kFusedWork) {
        hipLaunchKernelGGL(update_fused_kernel, dim3(1), dim3(kAssignThreads), (size_t)a.c.pages * sizeof(int), s, a, slots);
        NVFP4_HIP(hipGetLastError());
    } else {
        hipLaunchKernelGGL(update_init_kernel, dim3((unsigned)(a.c.pages + 255) / 256), dim3(256), 0, s, a);
        NVFP4_HIP(hipGetLastError());
        hipLaunchKernelGGL(update_count_kernel, dim3((unsigned)(lanes_in + lanes_out)), dim3(256), 0, s, a);
        NVFP4_HIP(hipGetLastError());
        hipLaunchKernelGGL(update_assign_kernel, dim3(1), dim3(kAssignThreads), 0, s, a, slots);
        NVFP4_HIP(hipGetLastError());
    }
    const long long page_bytes = ((long long)a.c.kv_heads * a.c.dim << a.c.log_page) * (a.c.fp8 ? 1 : 2);
    hipLaunchKernelGGL(update_copy_kernel, dim3((unsigned)lanes_out, (unsigned)a.c.layers, 8), dim3(256), 0, s, a, page_bytes);
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

}  // extern "C"
