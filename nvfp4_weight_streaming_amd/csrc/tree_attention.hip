// Attention of drafted tokens over a paged cache.
//
// "Ignis" README, "Speculative decoding (DFlash2)": a lane's drafts are checked
// in one pass.  Row t of a lane sees the lane's whole context (positions
// p < ctx) and, of the drafted tokens at positions ctx + j, those whose bit j is
// set in its mask word, so any tree of drafts takes one call; one row with mask
// 1 is a plain decode step.
//
//     o_t = sum_p w_p v_p / sum_p w_p,   w_p = exp(scale q_t . k_p)
//
// One pass with a running maximum.  The q heads that share a kv head are rows
// of the same product: a lane of T tokens and G heads per kv head has R = T G
// rows, and each K and V byte is read once for all of them.
//
// Operands.  The kernel computes S^T = K Q^T and O^T = V^T P^T with
// v_mfma_f32_16x16x32_bf16: tokens (then dims) are the M side, rows the N side.
//  - A lane's K operand is 8 consecutive dims of one token and its V operand 8
//    consecutive tokens of one dim: 16 bytes of a page as it lies.
//  - Result lane (g = lane / 16, n = lane % 16) holds rows 4 g + j of row n.  With
//    the M index 4 c + j of S tile i standing for token 16 c + 4 i + j of a
//    64-token tile, the lane holds tokens 16 g .. 16 g + 15 of row n after four S
//    tiles: the k slots 8 g .. 8 g + 7 of two PV steps, with no exchange between
//    lanes.  Row statistics are one value per lane, and the rescale of O is a
//    multiplication by it.
//
// Staging.  A workgroup's four waves copy a tile's K and V straight into LDS
// (wave w the w-th 16 tokens: one run of 16 x dim values of each), the copies of
// the next step, or of the next three, in flight while a step is computed.  K segments of 16
// bytes sit in slots xor-ed with their token, and V segments with their dim, so
// that the operand reads spread over the banks.
//
// Measured (12 rows of dim 128 a kv head, 4 kv heads, times with the joining
// kernel): 8 lanes of up to 40960 tokens, bf16, 451 MB: 78.5 us, 5.7 TB/s (copies
// alone, nothing computed: 79), in 8 bits 55 us; 8 of up to 4096, 45 MB: 17.5 us, of
// which about 10 are launches and loads that wait for each other.  64 drafted tokens
// a lane (768 rows a head), 4 lanes of up to 16384: 123 to 135 us over boxes, 540 to
// 590 TFLOP/s of the formula's arithmetic, half as much again of what the matrix units
// do (weights enter the second product as two bf16 numbers), against 1250 of a large
// product: bound by the vector work of the softmax beside the matrix instructions, 2.9
// for each (the matrix units are busy for 39% of the time, a third of the LDS cycles,
// 20% of the time in all, are bank conflicts).  In 8 bits every wave of a block of
// 128 rows converts the tiles for itself, 4.3 for each: 112 us for 8 lanes of 8 rows and
// up to 40960 tokens, whose 96 rows a head also leave a quarter of the block empty.
#include <cfloat>
#include <type_traits>

#include "cache.h"
#include "decode_device.h"

namespace nvfp4 {

constexpr int kTile = 64;        // tokens per tile
constexpr int kAttWaves = 4;
constexpr int kAttThreads = 64 * kAttWaves;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
// O and the sums are rescaled only when a row's maximum passes the one in use
// by 2^8: weights stay below 2^8, far from fp32's and bf16's limits.
constexpr float kRescaleAt = 8.f;
// Fewest tiles a worker takes where there are more workers than items: below,
// storing and joining partial results costs more than the shorter walk saves
// (8 lanes of 4096 tokens and 12 rows: 19.1 us with 5 tiles, 19.6 with 8).
constexpr int kMinTiles = 5;
// Where page tables hold no more than so many tiles, items are never shared and no
// joining kernel runs (one lane of 300 tokens of dim 256, 5 tiles: 13.3 us with a table
// of 6 pages of 64; 15.7, shared and joined, with one of 640).
constexpr int kWholeTiles = 8;
constexpr int kNoPieces = 1 << 28;  // a piece that holds any item
// Pieces may be so many tiles longer than an equal share.  A worker whose share goes
// over an item's end reads the new item's lengths, page numbers and rows before its
// first tile (3 to 4 us, the time of 5 tiles of few rows), and one such worker holds
// up the call: 8 lanes of 4096 tokens 18.8 us in pieces, 21.2 in equal shares; one
// lane of 40960 24.4 against 27.0; 4 lanes of 768 rows and 16384 tokens 131 and 132.
constexpr int kMoreTiles = 6;

// How the tiles are shared out.  An item has parts(tiles) parts: its tiles
// (piece 0), or pieces of at most `piece` tiles.  Worker r < active takes parts
// [begin(r), begin(r + 1)) of all: an equal number of tiles, over the items' ends,
// or a piece (several only where items are whole).
struct Shares {
    int active, each, rem, piece;
    __device__ __forceinline__ int parts(int tiles) const {
        return piece ? (int)((unsigned)(tiles + piece - 1) / (unsigned)piece) : tiles;
    }
    __device__ __forceinline__ int begin(int r) const { return r * each + min(r, rem); }
    __device__ __forceinline__ int owner(int part) const {
        const int wide = rem * (each + 1);
        return part < wide ? (int)((unsigned)part / (unsigned)(each + 1))
                           : rem + (int)((unsigned)(part - wide) / (unsigned)each);
    }
};

struct AttArgs {
    CacheView c;  // base pointers of the layer
    const uint16_t* q;
    long long q_ld;
    int q_heads, group;  // group = q_heads / kv_heads
    int lanes, rows, max_rows;  // rows: of q and out; max_rows: of a lane
    const int* row_start;
    const int* ctx_len;
    const int* table;
    int table_ld;
    const unsigned long long* mask;
    float scale2;  // softmax scale x log2(e) x K scale
    uint16_t* out;
    long long out_ld;
    float* lse;  // [rows][q_heads] or null
    Shares* shares;   // for the joining kernel
    float2* part_ml;  // [2 x workers][block rows]: maximum (log2 units), sum
    float* part_o;    // [2 x workers][block rows][dim]
    int workers;
    int whole;   // items are not shared: a worker's range is in items
    int stream;  // K and V are read with the streaming hint
};

// One lane's share of the work: items (kv head x row block) of `tiles`.
struct LaneWork {
    int row0, rows, ctx, tokens, blocks, tiles;
};

__device__ __forceinline__ LaneWork lane_work(const AttArgs& a, int b, int block_rows) {
    LaneWork w;
    w.row0 = a.row_start[b];
    w.rows = min(max(a.row_start[b + 1] - w.row0, 0), a.max_rows);
    if (w.row0 < 0 || w.row0 > a.rows - w.rows) w.rows = 0;  // rows that do not exist
    w.ctx = max(a.ctx_len[b], 0);
    w.tokens = (int)min((long long)w.ctx + w.rows, (long long)a.table_ld << a.c.log_page);
    w.blocks = (w.rows * a.group + block_rows - 1) / block_rows;
    w.tiles = w.rows > 0 ? (w.tokens + kTile - 1) / kTile : 0;
    return w;
}

// Inclusive sum over the wave's lanes: within rows of 16 by shifts, then the rows'
// totals carried on.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = dpp_add<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xF>(v);
    v = dpp_add<0x114, 0xF>(v);
    v = dpp_add<0x118, 0xF>(v);
    v = dpp_add<0x142, 0xA>(v);  // row_bcast 15 into rows 1 and 3
    return dpp_add<0x143, 0xC>(v);  // row_bcast 31 into rows 2 and 3
}

// Items of a lane's work.
__device__ __forceinline__ int lane_items(const AttArgs& a, const LaneWork& w) {
    return w.tiles > 0 ? w.blocks * a.c.kv_heads : 0;
}

// The shares, worked out by a wave: its lane l looks at lanes l, l + 64, ... of
// the call.  first, upto: lane l's own work (none past the last) and the sum of
// parts of lanes 0 .. l, for the first 64.
__device__ __forceinline__ Shares shares_of(const AttArgs& a, int block_rows, LaneWork& first, int& upto) {
    const int l = threadIdx.x & 63;
    first = LaneWork{0, 0, 0, 0, 0, 0};
    if (l < a.lanes) first = lane_work(a, l, block_rows);
    // Sum over all lanes of items x each(tiles).
    auto sum = [&](auto&& each) {
        upto = wave_scan(lane_items(a, first) * each(first.tiles));
        int all = __builtin_amdgcn_readlane(upto, 63);
        for (int b0 = 64; b0 < a.lanes; b0 += 64) {
            LaneWork w = {0, 0, 0, 0, 0, 0};
            if (b0 + l < a.lanes) w = lane_work(a, b0 + l, block_rows);
            all += __builtin_amdgcn_readlane(wave_scan(lane_items(a, w) * each(w.tiles)), 63);
        }
        return all;
    };
    Shares s = {0, 0, 0, kNoPieces};
    const int items = sum([](int) { return 1; });
    int parts = items;
    if (!a.whole) {
        s.piece = 0;
        const int total = sum([](int tiles) { return tiles; });
        // Pieces that start and end with their item, if that many workers can take one
        // each and the longest is not much longer than an equal share.  (An item's
        // last piece is half a piece on average: the first length tried allows for it.)
        if (items <= a.workers) {
            const int most = max(kMinTiles, total / a.workers) + kMoreTiles;
            int piece = max(kMinTiles, (int)((unsigned)total / (unsigned)(a.workers - items / 2)) + 1);
            for (; piece <= most && !s.piece; ++piece) {
                s.piece = piece;
                parts = sum([&](int tiles) { return s.parts(tiles); });
                if (parts > a.workers) s.piece = 0;
            }
        }
        if (!s.piece) parts = sum([](int tiles) { return tiles; });
        s.active = s.piece ? parts : min(a.workers, max(items, total / kMinTiles));
    } else {
        s.active = min(a.workers, items);
    }
    s.active = max(s.active, 1);
    s.each = (int)((unsigned)parts / (unsigned)s.active);
    s.rem = (int)((unsigned)parts % (unsigned)s.active);
    return s;
}

__device__ __forceinline__ bf16x8 bytes8(const uint4& v) {
    bf16x8 r;
    __builtin_memcpy(&r, &v, 16);
    return r;
}

__device__ __forceinline__ bf16x8 e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Keeps the first n of 16 bytes.
__device__ __forceinline__ uint4 keep_first(uint4 v, int n) {
    auto part = [](uint32_t w, int m) {
        return m >= 4 ? w : m <= 0 ? 0u : (w & ((1u << (8 * m)) - 1u));
    };
    return make_uint4(part(v.x, n), part(v.y, n - 4), part(v.z, n - 8), part(v.w, n - 12));
}

// Copies 1024 bytes straight into LDS: lane l's 16 bytes at src + at + off to
// dst + 16 l; reads past src + bytes give zeros.
__device__ __forceinline__ void copy_to_lds(uint8_t* src, int bytes, int at, int off, uint8_t* dst) {
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(src, 0, bytes, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16,
                                             off, at, 0, 0);
}
// The same with the streaming hint.
__device__ __forceinline__ void stream_to_lds(uint8_t* src, int bytes, int at, int off, uint8_t* dst) {
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(src, 0, bytes, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16,
                                             off, at, 0, 2);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint2 bf16x4(float a, float b, float c, float d) {
    return make_uint2(f32_to_bf16_rne(a) | ((uint32_t)f32_to_bf16_rne(b) << 16),
                      f32_to_bf16_rne(c) | ((uint32_t)f32_to_bf16_rne(d) << 16));
}

// Largest block of rows that is taken to be bound by memory.
constexpr int kFewRows = 32;

// How the four waves share a block: RW waves split its rows (NR row tiles of 16
// each), TW the token halves of a tile, DW the dims of O (those repeat S).
// SPLIT: weights enter the second product as two bf16 numbers.
template <int D, bool FP8, int NR, int RW, int TW, int DW, bool SPLIT>
struct AttTraits {
    static_assert(RW * TW * DW == kAttWaves, "four waves");
    static constexpr int ES = FP8 ? 1 : 2;
    static constexpr int kRows = 16 * NR * RW;          // rows of a block
    static constexpr int kRowBytes = D * ES;            // a token's K
    static constexpr int kSegs = kRowBytes / 16;
    static constexpr int kChunk = 16 * kRowBytes;       // 16 tokens of K, or of V
    static constexpr int kCopies = kChunk / 1024;       // 64 lanes x 16 bytes each
    static constexpr int kTileBytes = 8 * kChunk;       // K and V of 64 tokens
    // Tiles per step: 32 KiB in flight per workgroup and step.
    static constexpr int SUB = kTileBytes >= 32768 ? 1 : 32768 / kTileBytes;
    static constexpr int kStepBytes = SUB * kTileBytes;
    // Workgroups per compute unit: two, whose phases overlap, but one for few
    // rows, where memory is the bound and twice the partial results cost more (8
    // lanes of 16384 tokens of dim 256: 47 us against 55), or where LDS has room
    // for no more.
    static constexpr int kPerUnit = kRows <= kFewRows || kStepBytes > 32768 ? 1 : 2;
    // Buffers: all but one in flight.  (8 lanes of 40960 tokens, 12 rows: 80.5 us with
    // four, 87.5 with two; one of 40960: 24.4 and 26.1.)
    static constexpr int NB = kPerUnit == 1 && kStepBytes <= 32768 ? 4 : 2;
    static constexpr int kStepCopies = kStepBytes / kAttWaves / 1024;  // a wave's
};

// The kernel's arguments read anew where they are used: kept in registers from its
// start they fill the scalar file, and what the tile loop needs spills (37 to 90
// scalar registers; 14 to 45, none of them in the loop, with the arguments and the
// copies' addresses formed where they are used).  Of the vector registers one variant
// spills: bf16, dim 128, blocks of 64 rows (33 to 64 rows a head) takes 256 and 28 more
// in scratch, 116 bytes a lane (8 lanes of 4 rows of 12 heads and up to 16384 tokens,
// 181 MB: 47 us and 7 for the join; of 2 rows, in blocks of 32 without a spill, 33 and 5).
using ArgsRef = const __attribute__((address_space(4))) AttArgs&;
__device__ __forceinline__ ArgsRef args_anew() {
    auto at = (uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
    return *(const __attribute__((address_space(4))) AttArgs*)at;
}

template <int D, bool FP8, int NR, int RW, int TW, int DW, bool SPLIT>
__global__ __launch_bounds__(kAttThreads, (AttTraits<D, FP8, NR, RW, TW, DW, SPLIT>::kPerUnit)) void attend_kernel(AttArgs a) {
    using T = AttTraits<D, FP8, NR, RW, TW, DW, SPLIT>;
    constexpr int ES = T::ES, kRows = T::kRows, kSegs = T::kSegs, kChunk = T::kChunk, SUB = T::SUB, NB = T::NB;
    constexpr int KS = D / 32;       // K steps of 32 dims
    constexpr int DB = D / 16 / DW;  // this wave's dim blocks of O
    constexpr int HH = 2 / TW;       // token halves a wave takes
    constexpr int KL = FP8 ? KS / 2 : KS;  // 16-byte reads of a token's K
    using VRaw = typename std::conditional<FP8, uint2, uint4>::type;  // 8 tokens of V
    constexpr int KA = kSegs >= 16 ? 4 : kSegs / 4;  // distinct K operand addresses
    // Arrays of their own, so that the compiler can tell the copies in flight from
    // the reads of another one.
    __shared__ __align__(16) uint8_t lds0[T::kStepBytes];
    __shared__ __align__(16) uint8_t lds1[T::kStepBytes];
    __shared__ __align__(16) uint8_t lds2[NB == 4 ? T::kStepBytes : 16];
    __shared__ __align__(16) uint8_t lds3[NB == 4 ? T::kStepBytes : 16];
    __shared__ int lds_page[NB][SUB][4];  // page of each 16-token chunk of a step, -1: none
    __shared__ float2 lds_ml[TW > 1 ? kRows : 1];
    static_assert(TW == 1 || (RW <= 2 && NR * 16 * D * 4 <= T::kStepBytes), "sums of a row wave fit");

    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int lane = threadIdx.x & 63;
    const int g = lane >> 4, n = lane & 15;
    const int rw = wave % RW, tw = wave / RW % TW, dw = wave / (RW * TW);

    // Every workgroup works its share out of the lanes' lengths by itself.
    LaneWork w;
    int first_upto;
    const Shares share = shares_of(a, kRows, w, first_upto);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.shares = share;
    int worker = blockIdx.x;
    // Consecutive ranges on one XCD (workgroup b runs on XCD b mod 8), so that
    // the row blocks of one lane and head share their K and V in its L2.
    if (a.workers % 8 == 0) {
        const int each = (share.active + 7) >> 3;
        if (worker >> 3 >= each) return;
        worker = (worker & 7) * each + (worker >> 3);
    }
    if (worker >= share.active) return;
    int at = share.begin(worker);
    const int end = share.begin(worker + 1);
    if (at >= end) return;

    // The lane, item and part that `at` falls on.
    int b, parts, item, part;
    {
        int b0 = 0, upto = first_upto, base = 0;
        unsigned long long past = __ballot(upto > at);
        while (!past) {
            base += __builtin_amdgcn_readlane(upto, 63);
            b0 += 64;
            w = LaneWork{0, 0, 0, 0, 0, 0};
            if (b0 + lane < a.lanes) w = lane_work(a, b0 + lane, kRows);
            upto = wave_scan(lane_items(a, w) * share.parts(w.tiles));
            past = __ballot(base + upto > at);
        }
        const int first = __ffsll(past) - 1;
        w.row0 = __builtin_amdgcn_readlane(w.row0, first);
        w.rows = __builtin_amdgcn_readlane(w.rows, first);
        w.ctx = __builtin_amdgcn_readlane(w.ctx, first);
        w.tokens = __builtin_amdgcn_readlane(w.tokens, first);
        w.blocks = __builtin_amdgcn_readlane(w.blocks, first);
        w.tiles = __builtin_amdgcn_readlane(w.tiles, first);
        b = b0 + first;
        parts = share.parts(w.tiles);
        const int left = at - (base + __builtin_amdgcn_readlane(upto, first) - lane_items(a, w) * parts);
        item = (int)((unsigned)left / (unsigned)parts);
        part = left - item * parts;
    }

    const int page_mask = (1 << a.c.log_page) - 1;
    const long long head_bytes = (long long)T::kRowBytes << a.c.log_page;

    // Lane offsets of the copies.  K: slot s of the chunk's row r holds segment
    // s ^ swz(r), swz = r mod 4 plus 4 x (chunk mod 4) where a row has as many
    // segments; a copy covers 1024 bytes, rows in order.  V (bf16): dim d's two
    // segments are swapped where d / 4 is odd.
    int k_off[kSegs == 32 ? 2 : 1];
#pragma unroll
    for (int u = 0; u < (kSegs == 32 ? 2 : 1); ++u) {
        const int q = u * 64 + lane, r = q / kSegs, s = q % kSegs;
        const int swz = ((r & 3) | (wave << 2)) & (kSegs - 1) & 15;
        k_off[u] = (r * kSegs + (s ^ swz)) * 16 - u * 1024;
    }
    const int v_off = FP8 ? lane * 16 : (lane >> 1) * 32 + ((lane & 1) ^ ((lane >> 3) & 1)) * 16;
    // Lane offsets of the operand reads.
    int k_at[KA];
#pragma unroll
    for (int u = 0; u < KA; ++u) {
        const int swz = ((n & 3) | ((n >> 2) << 2)) & (kSegs - 1) & 15;
        k_at[u] = (n >> 2) * kChunk + (n & 3) * T::kRowBytes + (((4 * u + g) ^ swz) * 16);
    }
    const int v_at = g * kChunk + (FP8 ? n * 16 : n * 32);
    const int v_flip = FP8 ? 0 : ((n >> 2) & 1);

    while (at < end) {
        // Tiles [t0, t1): a piece (the item's are equal to one tile), or what is left.
        int t0 = part, t1 = min(w.tiles, t0 + (end - at));
        if (share.piece) {
            const int each = (int)((unsigned)w.tiles / (unsigned)parts), rem = w.tiles - each * parts;
            t0 = part * each + min(part, rem);
            t1 = t0 + each + (part < rem ? 1 : 0);
        }
        const int h = (int)((unsigned)item / (unsigned)w.blocks), rb = item - h * w.blocks;
        const int rows = w.rows * a.group;  // rows of the item's lane and head
        // (constant address space: scalar loads, which wait apart from the copies)
        const auto* tab = (const __attribute__((address_space(4))) int*)(uintptr_t)(a.table + (long long)b * a.table_ld);
        uint8_t* kbase = a.c.k + h * head_bytes;
        uint8_t* vbase = a.c.v + h * head_bytes;

        auto good = [&](int id) { return (unsigned)id < (unsigned)a.c.pages; };
        // Page of this wave's 16 tokens in the tiles of the step at t (past the
        // last token: its page).
        auto load_ids = [&](int t, int (&id)[SUB]) {
#pragma unroll
            for (int u = 0; u < SUB; ++u)
                id[u] = tab[min((t + u) * kTile + 16 * wave, w.tokens - 1) >> a.c.log_page];
        };
        // Copies of the step at tile t.  A missing page is read as page 0 (and
        // masked); past the range the copies read nothing (zero records).
        auto issue = [&](int t, const int (&id)[SUB], uint8_t* buf, int (*pages)[4]) {
            const int records = t < t1 ? kChunk : 0;
            // (formed anew in each step: the addresses of all copies of all steps, kept,
            // are more than the scalar file holds)
            int mine_at = wave * kChunk;
            asm volatile("" : "+s"(mine_at));
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                const int mine = id[u];
                if (lane == 0) pages[u][wave] = good(mine) ? mine : -1;
                const int tok = min((t + u) * kTile + 16 * wave, (w.tokens - 1) & ~15) & page_mask;
                const long long off = (long long)(good(mine) ? mine : 0) * a.c.page_stride + (long long)tok * T::kRowBytes;
                uint8_t* kd = buf + u * T::kTileBytes + mine_at;
                if (a.stream) {
#pragma unroll
                    for (int c = 0; c < T::kCopies; ++c)
                        stream_to_lds(kbase + off, records, c * 1024, k_off[kSegs == 32 ? c & 1 : 0], kd + c * 1024);
#pragma unroll
                    for (int c = 0; c < T::kCopies; ++c)
                        stream_to_lds(vbase + off, records, c * 1024, v_off, kd + 4 * kChunk + c * 1024);
                } else {
#pragma unroll
                    for (int c = 0; c < T::kCopies; ++c)
                        copy_to_lds(kbase + off, records, c * 1024, k_off[kSegs == 32 ? c & 1 : 0], kd + c * 1024);
#pragma unroll
                    for (int c = 0; c < T::kCopies; ++c)
                        copy_to_lds(vbase + off, records, c * 1024, v_off, kd + 4 * kChunk + c * 1024);
                }
            }
        };

        int ids[NB - 1][SUB], next_ids[SUB];
#pragma unroll
        for (int u = 0; u < NB - 1; ++u) load_ids(t0 + u * SUB, ids[u]);
        load_ids(t0 + (NB - 1) * SUB, next_ids);
        // Q operand: row n of each row tile, 8 dims per step (past the last row:
        // row 0's, whose results are not kept).  It is read ahead of the copies: they
        // end in order, and its first use waits for none of them.
        bf16x8 qf[NR][KS];
        unsigned long long mask[NR];
        ArgsRef aq = args_anew();
        const int group = aq.group;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = rb * kRows + (rw * NR + r) * 16 + n;
            const int t = row < rows ? (int)((unsigned)row / (unsigned)group) : 0;
            const int head = h * group + (row < rows ? row - t * group : 0);
            const uint16_t* src = aq.q + (long long)(w.row0 + t) * aq.q_ld + (long long)head * D;
            mask[r] = aq.mask[w.row0 + t];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                // fp8: 16 bytes hold 16 dims of a token, two steps' slots
                const int d = FP8 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
                qf[r][s] = bytes8(*(const uint4*)(src + d));
            }
        }
        issue(t0, ids[0], lds0, lds_page[0]);
        if constexpr (NB == 4) {
            issue(t0 + SUB, ids[1], lds1, lds_page[1]);
            issue(t0 + 2 * SUB, ids[2], lds2, lds_page[2]);
        }
        f32x4 o[NR][DB];
        float m[NR], mu[NR], l[NR];  // maximum, the one in use (0 for -inf), sum
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r] = -__builtin_inff();
            mu[r] = 0.f;
            l[r] = 0.f;
#pragma unroll
            for (int db = 0; db < DB; ++db) o[r][db] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // One tile of a step, at byte `base` of buf.  (Operand addresses are one
        // unsigned sum past the array: through longer chains of pointers the
        // compiler loses which array a read is from, and makes it wait for the
        // copies in flight into the other one.)
        auto tile = [&](int t, int page, const uint8_t* buf, uint32_t base) {
            // Tiles past the context, and those with a missing page, are masked.
            const bool masked = (t + 1) * kTile > w.ctx || __any(page < 0);
            const int chunk0 = t * kTile + 16 * g;  // this lane's first token
            const int present = page >= 0 ? min(max(w.tokens - chunk0, 0), 16) : 0;
            f32x4 s[HH][NR][2];
            // Operand reads go out well before their products, all of K first and
            // V of a half during the products before it (left alone, the compiler
            // waits for each read).
            uint4 kr[HH][KL][2];
            VRaw vr[HH][DB];
            auto read_k = [&](int hu) {
                const uint32_t kb = base + (uint32_t)((TW == 2 ? tw : hu) * 8 * T::kRowBytes);
#pragma unroll
                for (int u = 0; u < KL; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        kr[hu][u][i] = *(const uint4*)(buf + (kb + (uint32_t)k_at[u % KA] + (uint32_t)((u / KA) * KA * 64 + i * 4 * T::kRowBytes)));
            };
            auto read_v = [&](int hu) {
                const int hh = TW == 2 ? tw : hu;
                const uint32_t vo = base + 4u * kChunk + (uint32_t)v_at + (uint32_t)(dw * DB * (FP8 ? 256 : 512)) +
                                    (uint32_t)(FP8 ? 8 * hh : (hh ^ v_flip) * 16);
#pragma unroll
                for (int db = 0; db < DB; ++db) vr[hu][db] = *(const VRaw*)(buf + (vo + db * (FP8 ? 256u : 512u)));
            };
            // S of a half, instruction i of kDots.
            constexpr int kDots = KS * 2 * NR;
            auto dot = [&](int hu, int j) {
                const int ks = j / (2 * NR), i = j / NR % 2, r = j % NR;
                bf16x8 kv;
                if (FP8)
                    kv = (ks & 1) ? e4m3x8_to_bf16(kr[hu][ks / 2][i].z, kr[hu][ks / 2][i].w) : e4m3x8_to_bf16(kr[hu][ks / 2][i].x, kr[hu][ks / 2][i].y);
                else
                    kv = bytes8(kr[hu][FP8 ? 0 : ks][i]);
                const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                s[hu][r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv, qf[r][ks], ks == 0 ? zero : s[hu][r][i], 0, 0, 0);
            };
            // Masks a half and raises the rows' maxima where they grew too far; then
            // `before` runs ahead of the rescale of O.  True if there was one.
            auto settle = [&](int hu, auto&& before) -> bool {
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = 8 * (TW == 2 ? tw : hu) + e, p = chunk0 + c;
                        const int j = p - w.ctx;  // place among the drafted tokens
#pragma unroll
                        for (int r = 0; r < NR; ++r) {
                            const bool seen = c < present && (j < 0 || ((mask[r] >> (j & 63)) & 1));
                            s[hu][r][e >> 2][e & 3] = seen ? s[hu][r][e >> 2][e & 3] : -__builtin_inff();
                        }
                    }
                }
                float top[NR];
                bool grow = false;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float x = s[hu][r][0][0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) x = fmaxf(x, s[hu][r][e >> 2][e & 3]);
                    top[r] = x * a.scale2;
                    grow |= top[r] > m[r] + kRescaleAt;
                }
                if (!__any(grow)) return false;
                before();
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float mx = fmaxf(top[r], __shfl_xor(top[r], 16));
                    mx = fmaxf(mx, __shfl_xor(mx, 32));
                    mx = fmaxf(mx, m[r]);
                    const float use = mx == -__builtin_inff() ? 0.f : mx;
                    const float f = exp2_fast(m[r] - use);  // 0 for the first maximum
                    m[r] = mx;
                    mu[r] = use;
                    l[r] *= f;
#pragma unroll
                    for (int db = 0; db < DB; ++db)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[r][db][j] *= f;
                }
                return true;
            };
            // Weights of a half, as one or two bf16 operands: piece u is the pair
            // u % 4 of row tile u / 4.
            uint32_t pw[HH][NR][SPLIT ? 2 : 1][4];
            constexpr int kPieces = 4 * NR;
            auto weights = [&](int hu, int u) {
                const int r = u / 4, e = u % 4 * 2;
                f32x2v p;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    p[q] = exp2_fast(__builtin_fmaf(s[hu][r][(e + q) >> 2][(e + q) & 3], a.scale2, -mu[r]));
                    l[r] += p[q];
                }
                const bf16x2v hi = __builtin_convertvector(p, bf16x2v);
                uint32_t bits;
                __builtin_memcpy(&bits, &hi, 4);
                opaque(bits);  // formed here, not where it is used
                pw[hu][r][0][e / 2] = bits;
                if (SPLIT) {
                    const f32x2v back = {__uint_as_float(bits << 16), __uint_as_float(bits & 0xFFFF0000u)};
                    const f32x2v rest = {p[0] - back[0], p[1] - back[1]};
                    const bf16x2v lo = __builtin_convertvector(rest, bf16x2v);
                    __builtin_memcpy(&bits, &lo, 4);
                    opaque(bits);
                    pw[hu][r][1][e / 2] = bits;
                }
            };
            // The product of a half, instruction i of kSteps.  The two of an
            // accumulator stand apart: the second waits for the first.
            constexpr int kSteps = NR * DB * (SPLIT ? 2 : 1);
            bf16x8 vv[DB];
            auto convert = [&](int hu) {
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    if constexpr (FP8)
                        vv[db] = e4m3x8_to_bf16(vr[hu][db].x, vr[hu][db].y);
                    else
                        vv[db] = bytes8(vr[hu][db]);
                }
            };
            auto product = [&](int hu, int i) {
                const int db = i % (NR * DB) / NR, r = i % NR;
                const uint32_t(&w)[4] = pw[hu][r][i < NR * DB ? 0 : SPLIT];
                o[r][db] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vv[db], bytes8(make_uint4(w[0], w[1], w[2], w[3])), o[r][db], 0, 0, 0);
            };

#pragma unroll
            for (int hu = 0; hu < HH; ++hu) read_k(hu);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kDots; ++j) dot(0, j);
            if (HH == 1) {
                read_v(0);
                __builtin_amdgcn_sched_barrier(0);
                settle(0, [] {});
#pragma unroll
                for (int u = 0; u < kPieces; ++u) weights(0, u);
                convert(0);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) product(0, i);
                return;
            }
            // Two halves: the vector work of each stands beside matrix instructions
            // that do not need it, piece by piece: the first half's weights beside
            // the second half's S, the second's beside the first's product.
            constexpr int H = HH - 1;
            settle(0, [] {});
            read_v(0);
#pragma unroll
            for (int u = 0; u < kPieces; ++u) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = u * kDots / kPieces; j < (u + 1) * kDots / kPieces; ++j) dot(H, j);
                weights(0, u);
            }
            __builtin_amdgcn_sched_barrier(0);
            convert(0);
            const bool grew = settle(H, [&] {
#pragma unroll
                for (int i = 0; i < kSteps; ++i) product(0, i);
            });
            read_v(H);
            if (grew) {
#pragma unroll
                for (int u = 0; u < kPieces; ++u) weights(H, u);
            } else {
#pragma unroll
                for (int u = 0; u < kPieces; ++u) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = u * kSteps / kPieces; i < (u + 1) * kSteps / kPieces; ++i) product(0, i);
                    weights(H, u);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            convert(H);
#pragma unroll
            for (int i = 0; i < kSteps; ++i) product(H, i);
        };
        // Tokens past the end, and those of a missing page, may hold anything,
        // NaN included: their values are zeroed in LDS, each wave in the chunk that
        // it copied.
        auto clear = [&](int t, int page, uint8_t* buf) {
            const int left = w.tokens - (t * kTile + 16 * wave);
            const int keep = page >= 0 ? min(max(left, 0), 16) : 0;
            if (keep == 16) return;
            uint8_t* v = buf + (4 + wave) * kChunk;
            for (int e = lane; e < kChunk / 16; e += 64) {
                // bf16: first token of the segment in slot e
                const int first = FP8 ? 0 : 8 * ((e & 1) ^ ((e >> 3) & 1));
                uint4* p = (uint4*)(v + e * 16);
                *p = keep_first(*p, (keep - first) * ES);
            }
        };
        // One step: its copies have landed, those into the buffer of the step before
        // are issued, and it is computed.  The barrier also ends every wave's reads of
        // that buffer.
        auto step = [&](int t, uint8_t* buf, int (*pages)[4], uint8_t* other, int (*other_pages)[4]) {
            __builtin_amdgcn_s_waitcnt(vmcnt_imm((NB - 2) * T::kStepCopies));
            __builtin_amdgcn_s_waitcnt(kLgkmcnt0);
            barrier_nofence();
            issue(t + (NB - 1) * SUB, next_ids, other, other_pages);
            load_ids(t + NB * SUB, next_ids);
            int page[SUB];  // of this lane's chunk, g
            bool missing = (t + SUB) * kTile > w.tokens;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                page[u] = pages[u][g];
                missing |= __any(page[u] < 0) != 0;
            }
            if (missing) {
#pragma unroll
                for (int u = 0; u < SUB; ++u) clear(t + u, pages[u][wave], buf + u * T::kTileBytes);
                __builtin_amdgcn_s_waitcnt(kLgkmcnt0);
                barrier_nofence();
            }
#pragma unroll
            for (int u = 0; u < SUB; ++u)
                if (t + u < t1) tile(t + u, page[u], buf, u * T::kTileBytes);
        };
        for (int t = t0; t < t1; t += NB * SUB) {
            if constexpr (NB == 4) {
                step(t, lds0, lds_page[0], lds3, lds_page[3]);
                if (t + SUB < t1) step(t + SUB, lds1, lds_page[1], lds0, lds_page[0]);
                if (t + 2 * SUB < t1) step(t + 2 * SUB, lds2, lds_page[2], lds1, lds_page[1]);
                if (t + 3 * SUB < t1) step(t + 3 * SUB, lds3, lds_page[3], lds2, lds_page[2]);
            } else {
                step(t, lds0, lds_page[0], lds1, lds_page[1]);
                if (t + SUB < t1) step(t + SUB, lds1, lds_page[1], lds0, lds_page[0]);
            }
        }

        // Sums over the four token groups of a row.
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            l[r] += __shfl_xor(l[r], 16);
            l[r] += __shfl_xor(l[r], 32);
        }
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // the last, empty copies
        __syncthreads();
        // The two waves that split the token halves meet in LDS.
        if (TW > 1) {
            float* sums = (float*)(rw == 0 ? lds0 : lds1);
            if (tw > 0) {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int row = r * 16 + n;
                    if (g == 0 && dw == 0) lds_ml[rw * NR * 16 + row] = make_float2(m[r], l[r]);
#pragma unroll
                    for (int db = 0; db < DB; ++db)
                        *(f32x4*)(sums + row * D + ((16 * (dw * DB + db) + 4 * g) ^ (4 * (n & 7)))) = o[r][db];
                }
            }
            __syncthreads();
            if (tw == 0) {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const int row = r * 16 + n;
                    const float2 ml = lds_ml[rw * NR * 16 + row];
                    const float mx = fmaxf(m[r], ml.x);
                    const float use = mx == -__builtin_inff() ? 0.f : mx;
                    const float f0 = exp2_fast(m[r] - use), f1 = exp2_fast(ml.x - use);
                    m[r] = mx;
                    l[r] = l[r] * f0 + ml.y * f1;
#pragma unroll
                    for (int db = 0; db < DB; ++db) {
                        const f32x4 v = *(const f32x4*)(sums + row * D + ((16 * (dw * DB + db) + 4 * g) ^ (4 * (n & 7))));
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[r][db][j] = o[r][db][j] * f0 + v[j] * f1;
                    }
                }
            }
            __syncthreads();
        }
        const bool whole = t0 == 0 && t1 == w.tiles;
        if (tw == 0) {
            ArgsRef ae = args_anew();
            const int group = ae.group;
            const int slot = 2 * worker + (t0 > 0 ? 0 : 1);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int in_block = (rw * NR + r) * 16 + n;
                const int row = rb * kRows + in_block;
                if (row >= rows) continue;
                if (whole) {
                    const int tt = (int)((unsigned)row / (unsigned)group), head = h * group + row - tt * group;
                    const float inv = l[r] == 0.f ? 0.f : ae.c.v_scale / l[r];
                    uint16_t* dst = ae.out + (long long)(w.row0 + tt) * ae.out_ld + (long long)head * D + 16 * dw * DB;
#pragma unroll
                    for (int db = 0; db < DB; ++db)
                        *(uint2*)(dst + 16 * db + 4 * g) = bf16x4(o[r][db][0] * inv, o[r][db][1] * inv, o[r][db][2] * inv, o[r][db][3] * inv);
                    if (ae.lse && g == 0 && dw == 0)
                        ae.lse[(long long)(w.row0 + tt) * ae.q_heads + head] = l[r] == 0.f ? -__builtin_inff() : (m[r] + log2f(l[r])) * kLn2;
                } else {
                    float* dst = ae.part_o + ((long long)slot * kRows + in_block) * D + 16 * dw * DB;
#pragma unroll
                    for (int db = 0; db < DB; ++db) *(f32x4*)(dst + 16 * db + 4 * g) = o[r][db];
                    if (g == 0 && dw == 0) ae.part_ml[(long long)slot * kRows + in_block] = make_float2(m[r], l[r]);
                }
            }
        }
        // Next item.
        const int done = share.piece ? 1 : t1 - t0;
        at += done;
        part += done;
        if (at < end && part == parts) {
            part = 0;
            if (++item == w.blocks * a.c.kv_heads) {
                item = 0;
                do {
                    w = lane_work(a, ++b, kRows);
                } while (w.tiles == 0);
                parts = share.parts(w.tiles);
            }
        }
    }
}

// Joins the partial results of items that several workers shared.  A row is taken
// by one wave, or by the block's four (WIDE); a wave loads kFan of its contributors
// at once.  The order of the sums is that of the workers.  Bound by the chain launch,
// shares and lengths, partial results (4.3 us for 8 lanes of one token), or by the bytes
// of the partial results (8 x 8 rows over 512 workers: 24 MB, 12 us).
constexpr int kFan = 16;
template <int D, bool WIDE>
__global__ __launch_bounds__(256) void attend_join_kernel(AttArgs a, int block_rows, int max_blocks) {
    constexpr int E = D / 64;
    typedef float vec __attribute__((ext_vector_type(E)));
    __shared__ float lds_acc[WIDE ? 4 : 1][D];
    __shared__ float2 lds_ml[4];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int b = blockIdx.z, h = (int)(blockIdx.y / (unsigned)max_blocks), rb = blockIdx.y - h * max_blocks;
    const int in_block = WIDE ? blockIdx.x : blockIdx.x * 4 + wave, row = rb * block_rows + in_block;
    const Shares share = *a.shares;
    LaneWork w = {0, 0, 0, 0, 0, 0};
    int before = 0;  // parts of the lanes before b
    if (b < 64) {
        if (lane <= b) w = lane_work(a, lane, block_rows);
        const int upto = wave_scan(lane_items(a, w) * share.parts(w.tiles));
        before = b > 0 ? __builtin_amdgcn_readlane(upto, b - 1) : 0;
        w.row0 = __builtin_amdgcn_readlane(w.row0, b);
        w.rows = __builtin_amdgcn_readlane(w.rows, b);
        w.blocks = __builtin_amdgcn_readlane(w.blocks, b);
        w.tiles = __builtin_amdgcn_readlane(w.tiles, b);
    } else {
        for (int b0 = 0; b0 < b; b0 += 64) {
            LaneWork o = {0, 0, 0, 0, 0, 0};
            if (b0 + lane < b) o = lane_work(a, b0 + lane, block_rows);
            before += __builtin_amdgcn_readlane(wave_scan(lane_items(a, o) * share.parts(o.tiles)), 63);
        }
        w = lane_work(a, b, block_rows);
    }
    if (rb >= w.blocks || row >= w.rows * a.group || in_block >= block_rows || w.tiles == 0) return;  // whole wave (WIDE: block)
    const int parts = share.parts(w.tiles);
    const int start = before + (h * w.blocks + rb) * parts;  // the item's first part
    const int r0 = share.owner(start), r1 = share.owner(start + parts - 1);
    if (r0 == r1) return;
    auto slot = [&](int r) { return (long long)(2 * r + (r > r0 ? 0 : 1)) * block_rows + in_block; };
    float mx = -__builtin_inff(), sum = 0.f;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const int each = WIDE ? (r1 - r0 + 4) / 4 : 0;
    const int from = WIDE ? r0 + wave * each : r0, to = WIDE ? min(from + each - 1, r1) : r1;
    for (int r = from; r <= to; r += kFan) {
        float2 ml[kFan];
        vec v[kFan];
#pragma unroll
        for (int u = 0; u < kFan; ++u) {
            const long long s = slot(min(r + u, to));
            ml[u] = a.part_ml[s];
            v[u] = *(const vec*)(a.part_o + s * D + E * lane);
        }
        float top = mx;
#pragma unroll
        for (int u = 0; u < kFan; ++u) top = fmaxf(top, ml[u].x);
        const float use = top == -__builtin_inff() ? 0.f : top;
        const float old = exp2_fast(mx - use);
        mx = top;
        sum *= old;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= old;
#pragma unroll
        for (int u = 0; u < kFan; ++u) {
            const float f = r + u <= to ? exp2_fast(ml[u].x - use) : 0.f;
            sum = __builtin_fmaf(ml[u].y, f, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(v[u][e], f, acc[e]);
        }
    }
    if (WIDE) {
        if (lane == 0) lds_ml[wave] = make_float2(mx, sum);
#pragma unroll
        for (int e = 0; e < E; ++e) lds_acc[wave][E * lane + e] = acc[e];
        __syncthreads();
        if (wave != 0) return;
        mx = fmaxf(fmaxf(lds_ml[0].x, lds_ml[1].x), fmaxf(lds_ml[2].x, lds_ml[3].x));
        const float use = mx == -__builtin_inff() ? 0.f : mx;
        sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float f = exp2_fast(lds_ml[u].x - use);
            sum = __builtin_fmaf(lds_ml[u].y, f, sum);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(lds_acc[u][E * lane + e], f, acc[e]);
        }
    }
    const int tt = (int)((unsigned)row / (unsigned)a.group), head = h * a.group + row - tt * a.group;
    const float inv = sum == 0.f ? 0.f : a.c.v_scale / sum;
    uint16_t* dst = a.out + (long long)(w.row0 + tt) * a.out_ld + (long long)head * D + E * lane;
    if constexpr (E == 1) {
        dst[0] = f32_to_bf16_rne(acc[0] * inv);
    } else if constexpr (E == 2) {
        *(uint32_t*)dst = f32_to_bf16_rne(acc[0] * inv) | ((uint32_t)f32_to_bf16_rne(acc[1] * inv) << 16);
    } else {
        *(uint2*)dst = bf16x4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
    }
    if (a.lse && lane == 0)
        a.lse[(long long)(w.row0 + tt) * a.q_heads + head] = sum == 0.f ? -__builtin_inff() : (mx + log2f(sum)) * kLn2;
}

// How a call's rows are cut: the smallest block that holds the largest lane's, up to
// 128 rows; spare row tiles cost their matrix and vector work.  12 rows: 18.5 us in a
// block of 16, 19.0 in one of 32 (8 lanes of 4096); 24 rows: 39 in 32, 50 in 64 (8 of
// 16384); 48 rows: 42 in 64, 57 in 128 (8 of 16384 in 8 bits).  Dim 256 has no room in
// the registers for two row tiles of O beside two of Q.
struct AttShape {
    int nr, rw, tw, dw;
    int block_rows() const { return 16 * nr * rw; }
};

AttShape att_shape(int rows, int dim) {
    // rows: the largest lane's tokens x heads per kv head
    const int tiles = (rows + 15) / 16;
    if (tiles <= 1) return {1, 1, 2, 2};
    if (tiles <= 2) return {1, 2, 2, 1};
    if (dim == 256) return {1, 4, 1, 1};
    if (tiles <= 4) return {2, 2, 2, 1};
    return {2, 4, 1, 1};
}

// Workgroups: as many as the compute units hold at once.
int att_workers(const AttShape& sh, int dim, bool fp8) {
    const int step = dim == 256 && !fp8 ? 65536 : 32768;
    const int per_unit = step > 32768 || sh.block_rows() <= kFewRows ? 1 : 2;
    return per_unit * device_cus() / 8 * 8;
}

template <int D, bool FP8>
void launch_shape(const AttShape& sh, const AttArgs& a, hipStream_t s) {
#define NVFP4_ATT(NR_, RW_, TW_, DW_, SPLIT_)                                                     \
    if (sh.nr == NR_ && sh.rw == RW_) {                                                           \
        hipLaunchKernelGGL((attend_kernel<D, FP8, NR_, RW_, TW_, DW_, SPLIT_>), dim3(a.workers),  \
                           dim3(kAttThreads), 0, s, a);                                           \
        return;                                                                                   \
    }
    NVFP4_ATT(1, 1, 2, 2, true)
    NVFP4_ATT(1, 2, 2, 1, true)
    if constexpr (D == 256) {
        NVFP4_ATT(1, 4, 1, 1, true)
    } else {
        NVFP4_ATT(2, 2, 2, 1, true)
        NVFP4_ATT(2, 4, 1, 1, true)
    }
#undef NVFP4_ATT
}

template <int D>
int launch_attend(const AttShape& sh, const AttArgs& a, bool joins, hipStream_t s) {
    if (a.c.fp8)
        launch_shape<D, true>(sh, a, s);
    else
        launch_shape<D, false>(sh, a, s);
    NVFP4_HIP(hipGetLastError());
    if (!joins) return NVFP4_OK;
    const int rows = a.max_rows * a.group, br = sh.block_rows();
    const int max_blocks = (rows + br - 1) / br;
    // WIDE where rows have many contributors and are too few to fill the chip with a
    // wave each (8 lanes of 16384 tokens of dim 256, 12 rows: 39.9 us with, 42.3
    // without; 8 x 8 rows of 40960 in 8 bits: 112.9 with, 109.5 without).
    const int in_block = rows < br ? rows : br;
    const long long items = (long long)a.lanes * a.c.kv_heads * max_blocks;
    const bool wide = a.workers / items >= kFan && items * in_block <= 4 * device_cus();
    const dim3 grid((unsigned)(wide ? in_block : (in_block + 3) / 4), (unsigned)(a.c.kv_heads * max_blocks), (unsigned)a.lanes);
    if (wide)
        hipLaunchKernelGGL((attend_join_kernel<D, true>), grid, dim3(256), 0, s, a, br, max_blocks);
    else
        hipLaunchKernelGGL((attend_join_kernel<D, false>), grid, dim3(256), 0, s, a, br, max_blocks);
    NVFP4_HIP(hipGetLastError());
    return NVFP4_OK;
}

// Most partial results of a call: two per worker, of a block's rows.
size_t part_rows(const AttShape& sh) { return (size_t)2 * 2 * device_cus() * sh.block_rows(); }

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_tree_attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_rows) {
    if (kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || max_rows < 1 ||
        max_rows > NVFP4_TREE_MAX_ROWS || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
        q_heads > 65536)
        return 0;
    const AttShape sh = att_shape(max_rows * (q_heads / kv_heads), head_dim);
    return sizeof(Shares) + part_rows(sh) * (sizeof(float2) + head_dim * sizeof(float));
}

int nvfp4_tree_mask(const int* parent, int n, uint64_t* mask, int* depth) {
    clear_error();
    if (n < 1 || n > NVFP4_TREE_MAX_ROWS)
        return set_error(NVFP4_EINVAL, "n: %d outside [1, %d]", n, NVFP4_TREE_MAX_ROWS);
    if (!parent) return set_error(NVFP4_EINVAL, "parent: NULL");
    if (!mask) return set_error(NVFP4_EINVAL, "mask: NULL");
    for (int i = 0; i < n; ++i)
        if (parent[i] < -1 || parent[i] >= i)
            return set_error(NVFP4_EINVAL, "parent[%d]: %d outside [-1, %d]", i, parent[i], i - 1);
    for (int i = 0; i < n; ++i) {
        const int p = parent[i];
        mask[i] = (p >= 0 ? mask[p] : 0ull) | (1ull << i);
        if (depth) depth[i] = p >= 0 ? depth[p] + 1 : 0;
    }
    return NVFP4_OK;
}

int nvfp4_tree_attention(const nvfp4_cache* cache, int layer, const uint16_t* q_dev, int64_t q_ld,
                         int q_heads, int rows, int lanes, int max_rows, const int* row_start_dev,
                         const int* ctx_len_dev, const int* page_table_dev, int table_ld,
                         const uint64_t* mask_dev, float scale, uint16_t* out_dev, int64_t out_ld,
                         float* lse_dev, void* workspace_dev, size_t workspace_bytes, void* stream) {
    clear_error();
    AttArgs a;
    int st = cache_view(cache, layer, &a.c);
    if (st) return st;
    if (layer < 0) return set_error(NVFP4_EINVAL, "layer: %d < 0", layer);
    const int dim = a.c.dim, kv = a.c.kv_heads;
    if (q_heads < kv || q_heads % kv || q_heads > 65536)
        return set_error(NVFP4_EINVAL, "q_heads: %d is not a multiple of kv_heads %d up to 65536", q_heads, kv);
    if (rows < 0 || rows > (1 << 24)) return set_error(NVFP4_EINVAL, "rows: %d outside [0, 2^24]", rows);
    if (max_rows < (rows > 0 ? 1 : 0) || max_rows > NVFP4_TREE_MAX_ROWS)
        return set_error(NVFP4_EINVAL, "max_rows: %d outside [1, %d]", max_rows, NVFP4_TREE_MAX_ROWS);
    if ((st = check_lanes(a.c, lanes, page_table_dev, table_ld))) return st;
    const int64_t width = (int64_t)q_heads * dim;
    if (q_ld < width || q_ld % 8) return set_error(NVFP4_EINVAL, "q_ld: %lld below %lld or not a multiple of 8", (long long)q_ld, (long long)width);
    if (out_ld < width || out_ld % 4) return set_error(NVFP4_EINVAL, "out_ld: %lld below %lld or not a multiple of 4", (long long)out_ld, (long long)width);
    if (!row_start_dev || ((uintptr_t)row_start_dev & 3)) return set_error(NVFP4_EINVAL, "row_start: NULL or not 4-byte aligned");
    if (!ctx_len_dev || ((uintptr_t)ctx_len_dev & 3)) return set_error(NVFP4_EINVAL, "ctx_len: NULL or not 4-byte aligned");
    if (!(scale > 0.f) || scale > 1e30f) return set_error(NVFP4_EINVAL, "scale: not a positive number");
    a.scale2 = scale * kLog2e * a.c.k_scale;
    if (a.scale2 == 0.f || a.scale2 > FLT_MAX)  // a masked score times 0, or 0 times inf, would be NaN
        return set_error(NVFP4_EINVAL, "scale: %g times cache.k_scale %g is outside fp32's range", scale, a.c.k_scale);
    if (rows == 0) return NVFP4_OK;  // (the rows' pointers may be NULL: empty tensors have no address)
    if (!q_dev || ((uintptr_t)q_dev & 15)) return set_error(NVFP4_EINVAL, "q: NULL or not 16-byte aligned");
    if (!out_dev || ((uintptr_t)out_dev & 7)) return set_error(NVFP4_EINVAL, "out: NULL or not 8-byte aligned");
    if (!mask_dev || ((uintptr_t)mask_dev & 7)) return set_error(NVFP4_EINVAL, "mask: NULL or not 8-byte aligned");
    if ((uintptr_t)lse_dev & 3) return set_error(NVFP4_EINVAL, "lse: not 4-byte aligned");
    const size_t need = nvfp4_tree_attention_workspace_bytes(q_heads, kv, dim, max_rows);
    if (workspace_bytes < need) return set_error(NVFP4_EINVAL, "workspace_bytes: %zu < %zu needed", workspace_bytes, need);
    if (!workspace_dev || ((uintptr_t)workspace_dev & 15)) return set_error(NVFP4_EINVAL, "workspace: NULL or not 16-byte aligned");
    const AttShape sh = att_shape(max_rows * (q_heads / kv), dim);
    const int blocks = (max_rows * (q_heads / kv) + sh.block_rows() - 1) / sh.block_rows();
    const long long tiles = (long long)lanes * kv * blocks * ((((int64_t)table_ld << a.c.log_page) + kTile - 1) / kTile);
    if (tiles > 0x7FFFFFFFll)
        return set_error(NVFP4_EUNSUPPORTED, "lanes: %d lanes of %d kv heads, %d row blocks and %d pages exceed 2^31 tiles", lanes, kv, blocks, table_ld);
    if ((long long)kv * blocks > 65535)
        return set_error(NVFP4_EUNSUPPORTED, "q_heads: %d kv heads of %d row blocks exceed 65535", kv, blocks);
    a.q = q_dev;
    a.q_ld = q_ld;
    a.q_heads = q_heads;
    a.group = q_heads / kv;
    a.lanes = lanes;
    a.rows = rows;
    a.max_rows = max_rows;
    a.row_start = row_start_dev;
    a.ctx_len = ctx_len_dev;
    a.table = page_table_dev;
    a.table_ld = table_ld;
    a.mask = (const unsigned long long*)mask_dev;
    a.out = out_dev;
    a.out_ld = out_ld;
    a.lse = lse_dev;
    // No more workgroups than the tables could ever feed.
    const long long items = (long long)lanes * kv * blocks, per_item = tiles / items;
    a.whole = per_item <= kWholeTiles;
    const long long shared = (tiles + kMinTiles - 1) / kMinTiles, most = a.whole || shared < items ? items : shared;
    const int workers = att_workers(sh, dim, a.c.fp8 != 0);
    a.workers = most < workers ? (int)most : workers;
    static_assert(sizeof(Shares) % 16 == 0, "what follows is read by 16 bytes");
    a.shares = (Shares*)workspace_dev;
    a.part_ml = (float2*)(a.shares + 1);
    a.part_o = (float*)(a.part_ml + part_rows(sh));
    const bool joins = !a.whole && a.workers > 1;
    // The streaming hint, where K and V are read once (one block holds every row of a
    // lane and head): always for few rows, and for more rows if the pool is larger than
    // the 256 MiB that the chip's last cache can keep from call to call.  8 lanes of one
    // row, 12 heads, without the hint and with it, the pool just read and 640 MB of
    // others read in between: 45 MB 17.6 -> 16.4 and 20.0 -> 18.4 us, 181 MB 37.4 -> 37.4
    // and 44.5 -> 40.1, 451 MB 89 -> 79 and 92 -> 81.  4 rows (48 a head): 181 MB 47 -> 53
    // and 56 -> 54, 451 MB 110 -> 100 and 114 -> 102; 8 rows: 46 MB 30.4 -> 32.6 and
    // 32.3 -> 33.3.  Four blocks of 128 rows: 131 -> 149.
    const double cache_bytes = 2.0 * a.c.layers * a.c.pages * ((double)kv * dim * (a.c.fp8 ? 1 : 2) * (1 << a.c.log_page));
    a.stream = blocks == 1 && (sh.block_rows() <= kFewRows || cache_bytes > 256.0 * (1 << 20));
    hipStream_t s = (hipStream_t)stream;
    if (dim == 64) return launch_attend<64>(sh, a, joins, s);
    if (dim == 128) return launch_attend<128>(sh, a, joins, s);
    return launch_attend<256>(sh, a, joins, s);
}

}  // extern "C"
