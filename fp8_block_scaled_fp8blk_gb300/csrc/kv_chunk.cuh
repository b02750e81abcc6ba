// kv_chunk.cuh -- attention of any number of new rows per request over the
// paged e4m3 cache (prompts, chunks of prompts), on the fifth-generation tensor
// cores.
//
// For one request and cache head, a tile of 128 query rows (row = new token x
// query head of the group) against a tile of T tokens:
//   S[r][t] = sum_d q[r][d] k[t][d]                    (first MMA, kind::f16)
//   a = S s_k(t) c_r,   w = 2^(a + e_t + K - R_r)      (e_t: exponent of s_v(t))
//   O[r][d] += sum_t w[r][t] v[t][d]                   (second MMA, w out of tensor memory)
// K's and V's codes become f16 on their way to shared memory (exact: every e4m3
// value is an f16 value; the scales stay outside), once for 256 query rows.
// q is brought by a power of two of its row's own into [2^14, 2^15): f16 then
// holds a bf16 q exactly, down to 2^-39 of the row's largest; an f32 q, already
// times the softmax scale, is carried as two f16 planes (2^-22 of itself).
// The weights take V's scales with them, so each row's weights fill f16's range
// under its own largest p |s_v|: R_r, a whole power of two, is the running
// maximum of ceil(a) + e_t (kept as its distance from the running maximum of
// ceil(a)), and moves only when a tile passes it by 2^8 (O is
// rescaled in tensor memory then, seldom after a row's first tiles).  A weight
// keeps 2^-11 of itself (bf16 queries: an eighth of the rounding of the bf16
// output) or, as two planes, 2^-22 (f32), and 2^-30 of its row's largest.  A
// value scale that is no power of two leaves its mantissa to the weight.
// Scores, statistics and sums are f32; the softmax denominator is summed from
// the f32 weights, sixteen tokens (one scale) at a time.
//
// What a row does not see has no part in it: its weight is a selected zero, codes
// past the request's end are zeros, and a value whose code is NaN (or under a
// scale that is not finite, or in a block outside the pool) is replaced by zero
// in the tile and makes the rows that see it NaN at the end.
//
// The tensor cores cut sums to f32 instead of rounding them, which shows in f32
// results (a systematic 2e-6 over 1024 tokens).  So with f32 each tile's product
// starts anew, its second planes first, and is added to the sums by a group of
// warps of its own; one such product shrinks by 2e-7.
//
// Work: all (request, row tile, cache head, token tile) quadruples in one list,
// cut into one contiguous range per CTA, so ragged and causal lengths balance.
// Row tiles are 256 rows (two products' rows, whose softmax and MMAs take turns)
// for bf16 with head_dim <= 128, else 128 (scores of the next tile beside the
// softmax of this one).  A unit (request, row tile, head) that lies across CTAs
// leaves partial sums in the workspace, which a second kernel joins, in CTA order
// (deterministic, no counters).
//
// Roles (640 threads, one CTA per SM): warps 0-3 softmax (TMEM lane = row), warps
// 4-7 softmax of the unit's second 128 rows, or f32's sums, warps 8-15 convert q, K
// and V, warp 16 issues the MMAs.  Every wait is bounded; a timeout raises a
// CTA-wide flag, the outputs and lse of the CTA's rows become NaN, MMAs in flight
// are waited for, and the status word records it.
#pragma once

#include "kv_attn.cuh"
#include "rope.cuh"

#include <type_traits>

namespace fp8blk {

constexpr int kChThreads = 640;
constexpr int kChConvertWarp = 8, kChConvertWarps = 8, kChMmaWarp = 16;
constexpr int kChMaxGrid = 160;          // bound on CTAs: partial sums in the workspace
constexpr int kChInfo = 4;               // tiles whose scales (and sums' factors) are held
// Registers a thread of each role (of the 96 of the launch).
constexpr int kChSoftmaxRegs = 136, kChConvertRegs = 80, kChIssueRegs = 40;
static_assert(256 * kChSoftmaxRegs + 256 * kChConvertRegs + 128 * kChIssueRegs <= kChThreads * 96, "registers");
constexpr int kChLift = 6;               // K: a row's largest weight is below 2^6 when R moves, below 2^15 at most
constexpr int kChSlack = 8;              // ... which it does when a tile passes it by more than 2^8
constexpr float kChNone = -3.0e38f;      // maximum of a row that has seen nothing
constexpr float kChMinLog = -60.f;       // weights under value scales smaller than 2^-60 of their row's are zero in f16 anyway
constexpr int kChJoinRows = 8;           // rows a CTA of the join takes
constexpr size_t kChHeaderBytes = kChMaxGrid * 2 * sizeof(int4);
constexpr int kChNoNan = 0x7FFFFFFF;

struct ChunkArgs {
    const void *q;
    void *out;
    float *lse;                       // or null
    const uint8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int32_t *table, *seq_lens, *q_starts;
    int4 *heads;                      // [grid][2]: what each CTA's last unit is, and whether it or the first is cut
    float *partials;                  // [grid][2][U x head_dim sums | U maxima | U denominators]
    unsigned int *status;
    uint64_t wait_limit_ns;
    int64_t q_stride, out_stride, n_blocks;
    int n_seqs, total_rows, kv_heads, group, head_dim, block_log2, width;
    int max_tiles;                    // a table's tiles and one more
    float c, c_low;                   // softmax scale x log2 e, and what c leaves of it
};

// PL: planes of f16 for q and the weights (1: bf16, 2: f32).  WIDE: head_dim > 128.
template <int PL_, bool WIDE_>
struct ChunkShape {
    static constexpr int PL = PL_;
    static constexpr bool WIDE = WIDE_;
    static constexpr bool SUMS = PL == 2;               // products of a tile are added to the sums outside the tensor cores
    static constexpr int NS = WIDE || SUMS ? 1 : 2;     // 128-row products of a unit
    static constexpr int U = NS * 128;                  // rows of a unit
    static constexpr int T = WIDE ? 64 : 128;           // tokens of a tile
    static constexpr int kBlocks = WIDE ? 4 : 2;        // 64-wide column blocks of a head
    static constexpr int kSlot = T * kBlocks * 128;     // K or V of a tile as f16: 32 KiB
    static constexpr int kSlots = PL == 2 && WIDE ? 2 : 4;
    static constexpr int kQPlane = 128 * kBlocks * 128;  // one plane of 128 rows
    static constexpr int kQ = NS * PL * kQPlane;
    static constexpr size_t kSmem = 1024 + kQ + kSlots * kSlot;
    static constexpr int kGranules = T / 16;            // scales of a tile
    // Tensor memory, in columns: scores (and the weights, in their place; two buffers of one product, or one of each of
    // two), f32's product of a tile (half of a wide head at a time), the sums.
    static constexpr int kProductCol = WIDE ? 128 : 256;
    static constexpr int kSumCol = SUMS && !WIDE ? 384 : 256;
    static constexpr int kHalves = SUMS && WIDE ? 2 : 1;
};

struct ChunkShared {
    // Whoever waits on a barrier is never a whole turn of it behind: a wait could not tell the next phase but one from
    // its own.  So what a role may skip or be late for goes by the unit's or the score buffer's parity.
    uint64_t slot_full[4], slot_free[4], s_full[2], p_full[2], o_done[2], info_full[kChInfo];
    uint64_t q_full[2], values_done[2], unit_done[2], q_free, mma_done;
    uint64_t factor_full[kChInfo], last_full[2], product_free;  // f32's sums
    float4 info[kChInfo][8];     // per sixteen tokens: |k scale|, exponent of the v scale, its mantissa
    float qs[2][256];            // per row: what a score is times |s_k| of
    float factor[kChInfo][128];  // f32: what the sums so far are times, per row of a tile
    float last[2][3][128];       // f32: a unit's maxima, references and denominators
    int vnan[2][256];            // first position whose value is NaN, per element
    int any_nan[2];
    int64_t scan[kChThreads / 32];
    int64_t cut[2];              // this CTA's range
    int at[4];                   // its first request, row tile, head and slot
    int abort;
    uint32_t tmem;
};

// ------------------------------------------------------------------ the list
// sum of floor((a + step i) / g) over i < n, step 1 or 2.  The floors of all
// integers from a to a + n add up in closed form.  For every other one of a to
// a + 2 n: of two neighbours x, x + 1 the second's floor is one more only where g
// divides x + 1, and those are counted.
__host__ __device__ inline int64_t ch_floors_below(uint32_t x, uint32_t g) {
    const uint32_t q = x / g, r = x - q * g;
    return static_cast<int64_t>(g) * (static_cast<int64_t>(q) * (static_cast<int64_t>(q) - 1) / 2) + static_cast<int64_t>(q) * r;
}
__host__ __device__ inline int64_t ch_floor_sum(uint32_t a, uint32_t g, uint32_t n, int step) {
    if (n == 0) return 0;
    const uint32_t hi = a + step * n;
    const int64_t all = ch_floors_below(hi, g) - ch_floors_below(a, g);
    if (step == 1) return all;
    int64_t more = 0;
    if (g % 2 == 0) {
        if (a % 2 == 1) more = static_cast<int64_t>((hi - 1) / g) - a / g;
    } else if (a % 2 == 1) {
        more = static_cast<int64_t>((hi - 1) / (2 * g)) - a / (2 * g);
    } else {
        more = static_cast<int64_t>((hi - 1 + g) / (2 * g)) - (a + g) / (2 * g);
    }
    return (all - more) / 2;
}

// One request as the kernel takes it.  Row tile i's last row sees the tiles
// 0 .. floor((a + step i) / g), as far as there are any; a row tile's rows are
// step tiles' tokens.
struct ChunkSeq {
    int first, rows, len;  // rows 0: nothing to do
    int tiles;             // of the whole cache
    int row_tiles;
    int a, g, step, kv_heads;
    int full, last;        // list entries of a tile: of a row tile, of the last one
    bool bad;
    __host__ __device__ int seen(int i) const {  // tiles of row tile i
        const int t = (a + step * i) / g + 1;
        return t < tiles ? t : tiles;
    }
    __host__ __device__ int weight(int i) const { return i + 1 == row_tiles ? last : full; }
    // Entries of the row tiles below i, i < row_tiles: each unit has one slot for its set-up and one per tile.
    __host__ __device__ int64_t before(int i) const {
        const int64_t lack = static_cast<int64_t>(tiles - 1) * g - a;  // from row tile ceil(lack / step) on all tiles are seen
        const int64_t all = lack <= 0 ? 0 : (lack + step - 1) / step, some = all < i ? all : i;
        const int64_t slots = ch_floor_sum(static_cast<uint32_t>(a), static_cast<uint32_t>(g), static_cast<uint32_t>(some), step) + some +
                              (i - some) * tiles + i;
        return slots * full * kv_heads;
    }
    __host__ __device__ int64_t entries() const {
        if (row_tiles == 0) return 0;
        return before(row_tiles - 1) + static_cast<int64_t>(kv_heads) * last * (seen(row_tiles - 1) + 1);
    }
};

__host__ __device__ inline ChunkSeq ch_seq_of(int first, int64_t rows, int len, int total_rows, int group, int kv_heads, int max_tiles,
                                              int unit_rows, int tile) {
    ChunkSeq q;
    q.first = first;
    const bool off = first < 0 || rows < 0 || first + rows > total_rows;
    q.bad = off || len < 0;
    q.rows = off ? 0 : static_cast<int>(rows);
    q.len = len < 0 ? 0 : len;
    const int all = q.len / tile + (q.len % tile != 0);
    q.tiles = all < max_tiles ? all : max_tiles;
    const int64_t flat = static_cast<int64_t>(q.rows) * group;
    q.row_tiles = static_cast<int>((flat + unit_rows - 1) / unit_rows);
    // The first row's position, no further than the table's end (all tiles are seen from there on).
    int64_t p = static_cast<int64_t>(q.len) - q.rows;
    const int64_t end = static_cast<int64_t>(max_tiles) * tile;
    p = p < 0 ? 0 : p < end ? p : end;
    q.a = static_cast<int>((p * group + unit_rows - 1) / tile);
    q.g = group;
    q.step = unit_rows / tile;
    q.kv_heads = kv_heads;
    q.full = unit_rows / 128;
    q.last = flat - static_cast<int64_t>(q.row_tiles - 1) * unit_rows > 128 ? q.full : 1;
    return q;
}
template <typename Sh>
__device__ __forceinline__ ChunkSeq ch_seq(const ChunkArgs &a, int s) {
    const int first = a.q_starts[s];
    return ch_seq_of(first, static_cast<int64_t>(a.q_starts[s + 1]) - first, a.seq_lens[s], a.total_rows, a.group, a.kv_heads, a.max_tiles,
                     Sh::U, Sh::T);
}

// The place of entry x of a request: its row tile, head and slot, by `search`
// (the number of row tiles i > 0 whose entries begin at or below x), and the
// entry moved back to the slot's start.  A cut in a unit's set-up or first two
// tiles goes to the unit's start: joining parts costs more than they do.
constexpr int kChSmallCut = 2;
struct ChunkPlace {
    int row_tile, head, slot;
    int64_t at;
};
template <typename Search>
__host__ __device__ inline ChunkPlace ch_place(const ChunkSeq &q, int64_t x, Search search) {
    ChunkPlace p;
    p.row_tile = search(q, x);
    const int64_t base = q.before(p.row_tile);
    const int w = q.weight(p.row_tile), unit = w * (q.seen(p.row_tile) + 1);
    const int off = static_cast<int>(x - base);  // within a row tile's units: kv_heads x unit < 2^31
    p.head = off / unit;
    p.slot = (off - p.head * unit) / w;
    if (p.slot <= kChSmallCut) p.slot = 0;
    p.at = base + static_cast<int64_t>(p.head) * unit + p.slot * w;
    return p;
}

// A position in a CTA's range of the list: request, row tile and head, the
// unit's slots from e0 on (slot 0 is the set-up, slot j + 1 tile j), tiles
// [j0, j1), and the list entries left after them.
template <typename Sh>
struct ChunkWalk {
    const ChunkArgs &a;
    ChunkSeq q;
    int s, row_tile, head, tiles, weight, e0, j0, j1;
    int64_t left;
    __device__ __forceinline__ ChunkWalk(const ChunkArgs &args, const int (&at)[4], int64_t count) : a(args), left(count) {
        s = at[0];
        row_tile = at[1];
        head = at[2];
        e0 = at[3];
        q = ch_seq<Sh>(a, s);
        unit();
    }
    __device__ __forceinline__ void unit() {
        tiles = q.seen(row_tile);
        weight = q.weight(row_tile);
        const int64_t room = left / weight;
        const int e1 = e0 + room < tiles + 1 ? static_cast<int>(e0 + room) : tiles + 1;
        left -= static_cast<int64_t>(e1 - e0) * weight;
        j0 = max(e0 - 1, 0);
        j1 = e1 - 1;
    }
    __device__ __forceinline__ bool none() const { return j1 <= j0; }
    __device__ __forceinline__ bool starts() const { return e0 == 0; }
    __device__ __forceinline__ bool ends() const { return j1 == tiles; }
    __device__ __forceinline__ int row0() const { return row_tile * Sh::U; }
    __device__ __forceinline__ int products() const { return Sh::NS == 1 ? 1 : weight; }  // 128-row products with rows
    __device__ __forceinline__ bool next() {
        if (left <= 0) return false;
        if (++head == a.kv_heads) {
            head = 0;
            if (++row_tile == q.row_tiles) {
                row_tile = 0;
                do q = ch_seq<Sh>(a, ++s);
                while (q.rows == 0);
            }
        }
        e0 = 0;
        unit();
        return true;
    }
};

// ------------------------------------------------------------------ pieces
// kind::f16 instruction descriptor: f16 A and B, f32 D; B K-major or MN-major.
__host__ __device__ constexpr uint32_t ch_idesc(int n, bool mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24) | (mn_major ? 1u << 16 : 0u);
}
// 128-byte swizzle, 8-row groups 1024 bytes apart; `lead`: bytes between 64-element blocks along N of an MN-major operand.
__device__ __forceinline__ uint64_t ch_desc(uint32_t saddr, uint32_t lead) {
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}
__device__ __forceinline__ void ch_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}
__device__ __forceinline__ void ch_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}
// 32 or 16 consecutive columns of this warp's lanes.
__device__ __forceinline__ void ch_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,"
        "%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void ch_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void ch_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t ch_pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 ch_unpack_f16(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }
// Two f32 at a time.
__device__ __forceinline__ uint64_t ch_pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void ch_unpair(uint64_t p, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }
__device__ __forceinline__ uint64_t ch_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t ch_add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float ch_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
template <typename Sh, typename T>
__device__ __forceinline__ void ch_queries(const ChunkArgs &a, const ChunkWalk<Sh> &w, uint8_t *sq, float *qs, int warp, int lane) {
    // A warp takes two rows at a time (one of a wide head), sixteen (32) lanes a row, eight values a lane.
    constexpr int L = Sh::WIDE ? 32 : 16, RW = 32 / L, PL = Sh::PL;
    const int sub = lane / L, d0 = (lane % L) * 8, rows = w.products() * 128;
    const int flat = w.q.rows * a.group - w.row0();  // rows of the unit that exist
    const bool negative = a.c < 0.f;
    const T *q = static_cast<const T *>(a.q) + w.q.first * a.q_stride + static_cast<int64_t>(w.head) * a.group * a.head_dim;
    constexpr int kBatch = 4;
#pragma unroll 1
    for (int r0 = warp * RW + sub; r0 < rows; r0 += kChConvertWarps * RW * kBatch) {
        float x[kBatch][8];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + b * kChConvertWarps * RW;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[b][i] = 0.f;
            if (r < rows && r < flat && d0 < a.head_dim) {
                const int token = (w.row0() + r) / a.group;
                rope_load8(q + token * a.q_stride + (w.row0() + r - token * a.group) * a.head_dim + d0, x[b]);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int r = r0 + b * kChConvertWarps * RW;
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (PL == 2) x[b][i] = fmaf(x[b][i], a.c, x[b][i] * a.c_low);  // the scale per value, rounded at random
                else if (negative) x[b][i] = -x[b][i];
                top = max(top, __float_as_uint(fabsf(x[b][i])));
            }
#pragma unroll
            for (int d = L / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            const bool good = top < 0x7F800000u;
            int e = 0;  // the row's largest times 2^e is in [2^14, 2^15)
            if (good && top != 0) e = top >= 0x800000u ? 14 + 127 - static_cast<int>(top >> 23) : 14 + 149 - (31 - __clz(top));
            const float f1 = ch_pow2(e >> 1), f2 = ch_pow2(e - (e >> 1));
            if (r >= rows) continue;
            if (lane % L == 0) {
                const float back = ch_pow2(-(e >> 1)) * (PL == 2 ? 1.f : fabsf(a.c)) * ch_pow2(-(e - (e >> 1)));
                qs[r] = good ? back : __int_as_float(0x7FC00000);
            }
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = good ? x[b][2 * i] * f1 * f2 : 0.f, v = good ? x[b][2 * i + 1] * f1 * f2 : 0.f;
                h[i] = ch_pack_f16(u, v);
                if (PL == 2) {
                    const float2 f = ch_unpack_f16(h[i]);
                    l[i] = ch_pack_f16(u - f.x, v - f.y);
                }
            }
            uint8_t *dst = sq + (r >> 7) * (PL * Sh::kQPlane) + (d0 >> 6) * (128 * 128) + (r & 127) * 128 + ((((d0 >> 3) & 7) ^ (r & 7)) << 4);
            if (d0 < Sh::kBlocks * 64) {
                *reinterpret_cast<uint4 *>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
                if (PL == 2) *reinterpret_cast<uint4 *>(dst + Sh::kQPlane) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
    }
}

// ------------------------------------------------------------------ converters
// Warps 8-15: q of each unit, then K and V of its tiles.  A thread has up to
// four groups of sixteen codes of a tile; the next tile's codes are on their way
// while this one's are converted, their block ids a tile earlier.
template <typename Sh, typename T>
__device__ __forceinline__ void ch_convert(const ChunkArgs &a, ChunkWalk<Sh> w, ChunkShared &sh, uint8_t *sq, uint8_t *slots, int tid) {
    constexpr int kEach = 4, kThreads = kChConvertWarps * 32;
    const int warp = tid >> 5, lane = tid & 31, per = a.head_dim / 16, total = Sh::T * per, block = 1 << a.block_log2;
    int token[kEach], col[kEach];  // of the thread's groups in a tile
    uint32_t dst[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int g = tid + i * kThreads;
        token[i] = g < total ? g / per : Sh::T;  // T: none
        col[i] = g < total ? g - token[i] * per : 0;
        dst[i] = (col[i] >> 2) * (Sh::T * 128) + token[i] * 128 + (((2 * (col[i] & 3)) ^ (token[i] & 7)) << 4);
    }
    int n = 0;        // slots filled so far
    int it = 0;       // tiles
    int unit = 0;
    bool more = !w.none();
    while (!more && w.next()) more = !w.none();
    const float nanf = __int_as_float(0x7FC00000);
    while (more) {
        const int ub = unit & 1, len = w.q.len, j1 = w.j1;
        const int32_t *row = a.table + static_cast<int64_t>(w.s) * a.width;
        // A group's block: its id, -1 for one that is not there, -2 for tokens past the end.
        auto ids_of = [&](int j, int (&id)[kEach]) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int64_t t = static_cast<int64_t>(j) * Sh::T + token[i];
                id[i] = -2;
                if (j < j1 && token[i] < Sh::T && t < len) {
                    const int page = static_cast<int>(t >> a.block_log2);
                    id[i] = page < a.width ? row[page] : -1;
                }
            }
        };
        auto fetch = [&](int j, const int (&id)[kEach], const uint8_t *codes, const float *scales, uint4 (&x)[kEach], float (&sc)[kEach]) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                x[i] = make_uint4(0, 0, 0, 0);
                sc[i] = 1.f;
                if (id[i] == -2) continue;
                if (id[i] < 0 || id[i] >= a.n_blocks) {
                    sc[i] = nanf;
                    atomicOr(a.status, 4u);
                    continue;
                }
                const int64_t bh = static_cast<int64_t>(id[i]) * a.kv_heads + w.head;
                // (Plain loads: the kernel before this one may have written the cache after this one had begun.)
                x[i] = *reinterpret_cast<const uint4 *>(codes + ((bh << a.block_log2) + ((j * Sh::T + token[i]) & (block - 1))) * a.head_dim +
                                                        16 * col[i]);
                sc[i] = scales[bh];
            }
        };
        int id[kEach], id_next[kEach];
        uint4 kx[kEach], vx[kEach];
        float ks[kEach], vs[kEach];
        ids_of(w.j0, id);
        ids_of(w.j0 + 1, id_next);
        fetch(w.j0, id, a.k_codes, a.k_scales, kx, ks);
        fetch(w.j0, id, a.v_codes, a.v_scales, vx, vs);
        // The unit's queries, once the MMAs have read the last one's, and the softmax has written out the one before that.
        if (unit >= 1 && !at_warp_wait(smem_addr(&sh.q_free), static_cast<uint32_t>(unit - 1) & 1u, &sh.abort, a.wait_limit_ns)) return;
        if (unit >= 2 && !at_warp_wait(smem_addr(&sh.unit_done[ub]), static_cast<uint32_t>((unit >> 1) - 1) & 1u, &sh.abort, a.wait_limit_ns)) return;
        sh.vnan[ub][tid] = kChNoNan;
        if (tid == 0) sh.any_nan[ub] = 0;
        asm volatile("bar.sync 4, %0;" ::"n"(kThreads) : "memory");
        ch_queries<Sh, T>(a, w, sq, sh.qs[ub], warp, lane);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[ub]));
        for (int j = w.j0; j < j1; ++j, ++it) {
#pragma unroll 1
            for (int is_v = 0; is_v < 2; ++is_v, ++n) {
                const int slot = n % Sh::kSlots;
                const uint32_t ph = static_cast<uint32_t>(n / Sh::kSlots) & 1u;
                if (n >= Sh::kSlots && !at_warp_wait(smem_addr(&sh.slot_free[slot]), ph ^ 1u, &sh.abort, a.wait_limit_ns)) return;
                uint8_t *to = slots + slot * Sh::kSlot;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    if (token[i] >= Sh::T) continue;
                    const float scale = is_v ? vs[i] : ks[i];
                    const uint4 c = is_v ? vx[i] : kx[i];
                    uint32_t x[4] = {c.x, c.y, c.z, c.w};
                    const bool finite = fabsf(scale) < INFINITY;
                    const uint32_t sign = scale < 0.f ? 0x80808080u : 0u;  // the scale's magnitude is what the softmax uses
#pragma unroll
                    for (int y = 0; y < 4; ++y) x[y] ^= sign;
                    if (is_v) {
                        uint32_t bad = 0;
#pragma unroll
                        for (int y = 0; y < 4; ++y) bad |= (x[y] & 0x7F7F7F7Fu) + 0x01010101u;
                        if ((bad & 0x80808080u) != 0 || !finite) {  // seldom: which elements, from which position on
                            const int p = j * Sh::T + token[i];
                            sh.any_nan[ub] = 1;
#pragma unroll 1
                            for (int y = 0; y < 16; ++y) {
                                const uint32_t word = y < 8 ? (y < 4 ? x[0] : x[1]) : (y < 12 ? x[2] : x[3]);
                                const uint32_t code = (word >> (8 * (y & 3))) & 0x7Fu;
                                if (!finite || code == 0x7Fu) {
                                    atomicMin(&sh.vnan[ub][16 * col[i] + y], p);
                                    const uint32_t keep = ~(0xFFu << (8 * (y & 3)));
#pragma unroll
                                    for (int z = 0; z < 4; ++z)
                                        if (z == y >> 2) x[z] &= keep;
                                }
                            }
                        }
                    } else if (!finite) {
#pragma unroll
                        for (int y = 0; y < 4; ++y) x[y] = 0x7F7F7F7Fu;
                    }
                    uint32_t h[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        h[2 * y] = at_e4m3x2_f16x2(x[y]);
                        h[2 * y + 1] = at_e4m3x2_f16x2(x[y] >> 16);
                    }
                    *reinterpret_cast<uint4 *>(to + dst[i]) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(to + (dst[i] ^ 16u)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                if (!is_v && warp == 0) {
                    // Scales of the tile's sixteens (both, for the softmax).
                    if (lane < Sh::kGranules) {
                        const int64_t t = static_cast<int64_t>(j) * Sh::T + 16 * lane;
                        float k1 = 1.f, v1 = 1.f;
                        if (t < len && (t >> a.block_log2) < a.width) {
                            const int b = row[t >> a.block_log2];
                            if (b >= 0 && b < a.n_blocks) {
                                k1 = fabsf(a.k_scales[static_cast<int64_t>(b) * a.kv_heads + w.head]);
                                v1 = fabsf(a.v_scales[static_cast<int64_t>(b) * a.kv_heads + w.head]);
                            }
                        }
                        if (!(k1 < INFINITY)) k1 = 1.f;  // K's codes are NaN there
                        if (!(v1 < INFINITY)) v1 = 1.f;  // V's are zero
                        float e = 0.f, m = 1.f;
                        const bool small = v1 < 0x1p-126f;
                        const uint32_t u = __float_as_uint(small ? v1 * 0x1p64f : v1);
                        if (v1 == 0.f) {
                            e = -1000.f;
                        } else {
                            e = static_cast<float>(static_cast<int>(u >> 23) - 127 - (small ? 64 : 0));
                            m = __uint_as_float((u & 0x7FFFFFu) | 0x3F800000u);
                        }
                        sh.info[it & (kChInfo - 1)][lane] = make_float4(k1, e, m, 0.f);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.info_full[it & (kChInfo - 1)]));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // generic stores -> the MMA
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.slot_full[slot]));
                if (is_v) {
                    fetch(j + 1, id_next, a.v_codes, a.v_scales, vx, vs);
#pragma unroll
                    for (int i = 0; i < kEach; ++i) id[i] = id_next[i];
                    ids_of(j + 2, id_next);
                } else {
                    fetch(j + 1, id_next, a.k_codes, a.k_scales, kx, ks);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.values_done[ub]));
        ++unit;
        do more = w.next();
        while (more && w.none());
    }
}

// ------------------------------------------------------------------ MMAs
template <typename Sh>
__device__ __forceinline__ bool ch_issue(const ChunkArgs &a, ChunkWalk<Sh> w, ChunkShared &sh, uint32_t tmem, uint32_t sq, uint32_t slots) {
    constexpr int PL = Sh::PL, T = Sh::T;
    constexpr uint32_t qk_idesc = ch_idesc(T, false);
    const uint64_t q_desc = ch_desc(sq, 16), k_desc = ch_desc(slots, 16), v_desc = ch_desc(slots, T * 128);
    const int steps = a.head_dim / 16;
    bool any = false;
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        const bool ok = at_wait(smem_addr(&bar), parity, &sh.abort, a.wait_limit_ns);
        t8_fence_after();
        return ok;
    };
    int n = 0, unit = 0;               // slots consumed in order K, V, K, V ..; units
    int done[2] = {0, 0};              // tiles of each product whose weights have been taken
    int begun[2] = {0, 0};             // ... whose scores have been issued
    int products = 0;                  // f32: products of a tile (of half a wide head) issued
    auto scores = [&](int i, int slot) {  // product i's scores against K in the slot, the second plane's first
        const uint32_t d = tmem + static_cast<uint32_t>(Sh::NS == 1 ? (begun[0] & 1) * T : i * 128);
        const uint64_t k = k_desc + static_cast<uint32_t>(slot) * (Sh::kSlot / 16);
#pragma unroll 1
        for (int p = PL - 1; p >= 0; --p) {
            const uint64_t q = q_desc + static_cast<uint32_t>(i * PL + p) * (Sh::kQPlane / 16);
#pragma unroll 4
            for (int s = 0; s < steps; ++s)
                ch_mma_ss(d, q + (s >> 2) * (128 * 128 / 16) + (s & 3) * 2, k + (s >> 2) * (T * 128 / 16) + (s & 3) * 2, qk_idesc,
                          p + 1 < PL || s > 0);
        }
        t8_commit(smem_addr(&sh.s_full[Sh::NS == 1 ? (begun[0] & 1) : i]));
        ++begun[i];
        any = true;
    };
    auto sums = [&](int i, int slot, bool acc) {  // product i's weights times V in the slot
        const uint32_t p0 = tmem + static_cast<uint32_t>(Sh::NS == 1 ? (done[0] & 1) * T : i * 128);
        const uint64_t v = v_desc + static_cast<uint32_t>(slot) * (Sh::kSlot / 16);
#pragma unroll 1
        for (int h = 0; h < Sh::kHalves; ++h) {
            if (Sh::SUMS && products > 0 && !wait(sh.product_free, static_cast<uint32_t>(products - 1) & 1u)) return false;
            const uint32_t d = tmem + static_cast<uint32_t>(Sh::SUMS ? Sh::kProductCol : Sh::kSumCol + i * 128);
            const uint32_t idesc = ch_idesc(Sh::kHalves == 1 ? a.head_dim : h == 0 ? 128 : a.head_dim - 128, true);
#pragma unroll
            for (int p = PL - 1; p >= 0; --p)
#pragma unroll
                for (int s = 0; s < T / 16; ++s)
                    ch_mma_ts(d, p0 + (PL == 1 ? 8 * s : 32 * (s >> 1) + 16 * p + 8 * (s & 1)),
                              v + h * (2 * T * 128 / 16) + s * (16 * 128 / 16), idesc, (!Sh::SUMS && acc) || p + 1 < PL || s > 0);
            t8_commit(smem_addr(&sh.o_done[i]));
            ++products;
        }
        ++done[i];
        return true;
    };
    auto slot_ready = [&](int m) { return wait(sh.slot_full[m % Sh::kSlots], static_cast<uint32_t>(m / Sh::kSlots) & 1u); };
    bool more = !w.none();
    while (!more && w.next()) more = !w.none();
    while (more) {
        const int np = w.products(), tiles = w.j1 - w.j0;
        if (!wait(sh.q_full[unit & 1], static_cast<uint32_t>(unit >> 1) & 1u)) return any;
        if (!slot_ready(n)) return any;
        for (int i = 0; i < np; ++i) scores(i, n % Sh::kSlots);
        t8_commit(smem_addr(&sh.slot_free[n % Sh::kSlots]));
        if (tiles == 1) t8_commit(smem_addr(&sh.q_free));
        for (int j = 0; j < tiles; ++j, n += 2) {
            const bool next = j + 1 < tiles;
            if (Sh::NS == 1 && next) {  // the next scores have a buffer of their own
                if (!slot_ready(n + 2)) return any;
                scores(0, (n + 2) % Sh::kSlots);
                t8_commit(smem_addr(&sh.slot_free[(n + 2) % Sh::kSlots]));
                if (j + 2 == tiles) t8_commit(smem_addr(&sh.q_free));
            }
            if (!slot_ready(n + 1)) return any;
            for (int i = 0; i < np; ++i) {
                if (!wait(sh.p_full[Sh::NS == 1 ? done[0] & 1 : i], static_cast<uint32_t>(Sh::NS == 1 ? done[0] >> 1 : done[i]) & 1u)) return any;
                if (!sums(i, (n + 1) % Sh::kSlots, j > 0)) return any;
                if (i + 1 == np) t8_commit(smem_addr(&sh.slot_free[(n + 1) % Sh::kSlots]));
                // The weights lay where these scores go: MMAs of one thread run in the order of their issue.
                if (Sh::NS == 2 && next) {
                    if (i == 0 && !slot_ready(n + 2)) return any;
                    scores(i, (n + 2) % Sh::kSlots);
                    if (i + 1 == np) {
                        t8_commit(smem_addr(&sh.slot_free[(n + 2) % Sh::kSlots]));
                        if (j + 2 == tiles) t8_commit(smem_addr(&sh.q_free));
                    }
                }
            }
        }
        ++unit;
        do more = w.next();
        while (more && w.none());
    }
    return any;
}

// ------------------------------------------------------------------ softmax
// A row of the unit: where it lies, and what it sees.
struct ChunkRow {
    int64_t out, lse;
    int last;    // last position it sees
    bool valid;
    template <typename Sh>
    __device__ __forceinline__ ChunkRow(const ChunkArgs &a, const ChunkWalk<Sh> &w, int local) {
        const int r = w.row0() + local, token = r / a.group;
        const int64_t row = w.q.first + token, head = static_cast<int64_t>(w.head) * a.group + (r - token * a.group);
        valid = r < w.q.rows * a.group;
        last = valid ? w.q.len - w.q.rows + token : 0x7FFFFFFF;  // (rows that are not there: zeros, stored nowhere)
        out = row * a.out_stride + head * a.head_dim;
        lse = row * (static_cast<int64_t>(a.kv_heads) * a.group) + head;
    }
};

// Writes a unit's row out: its outputs, or its part of them.
template <typename Sh, typename T>
__device__ __forceinline__ void ch_finish(const ChunkArgs &a, const ChunkWalk<Sh> &w, ChunkShared &sh, int unit, const ChunkRow &row, int local,
                                          uint32_t o_col, float M, float R, float l, bool ok) {
    const float nanf = __int_as_float(0x7FC00000);
    const int ub = unit & 1;
    // The converters' word on what is NaN.
    ok = ok && at_warp_wait(smem_addr(&sh.values_done[ub]), static_cast<uint32_t>(unit >> 1) & 1u, &sh.abort, a.wait_limit_ns);
    const bool whole = w.starts() && w.ends();
    const float up = R > kChNone ? R - static_cast<float>(kChLift) : 0.f;  // sums are 2^-up times what they stand for
    float f = 1.f;
    if (!ok) l = nanf;
    if (whole) {
        f = l == 0.f ? 0.f : 1.f / l;
        if (row.valid && a.lse) a.lse[row.lse] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
    }
    float *part = a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + w.starts()) * (static_cast<int64_t>(Sh::U) * (a.head_dim + 2));
    if (!whole) {
        __stcg(part + static_cast<int64_t>(Sh::U) * a.head_dim + local, M);
        __stcg(part + static_cast<int64_t>(Sh::U) * (a.head_dim + 1) + local, l);
    }
    T *out = static_cast<T *>(a.out) + row.out;
    const bool nans = ok && sh.any_nan[ub] != 0;
    // 2^up in two factors, since it may leave the range of one.
    const float u1 = at_exp2(fminf(fmaxf(up, -120.f), 120.f)), u2 = at_exp2(fminf(fmaxf(up - fminf(fmaxf(up, -120.f), 120.f), -120.f), 120.f)) * f;
#pragma unroll 1
    for (int c = 0; c < a.head_dim; c += 16) {
        float v[16];
        if (ok) {
            t8_ld16(o_col + c, v);
            at_wait_ld();
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            v[x] = ok ? v[x] * u1 * u2 : nanf;
            if (nans && sh.vnan[ub][c + x] <= row.last) v[x] = nanf;
        }
        float lo[8], hi[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) lo[x] = v[x], hi[x] = v[8 + x];
        if (whole) {
            if (row.valid) {
                rope_store8(out + c, lo);
                rope_store8(out + c + 8, hi);
            }
        } else {
            float *p = part + static_cast<int64_t>(local) * a.head_dim + c;
            rope_store8(p, lo);
            rope_store8(p + 8, hi);
        }
    }
}
// ... of a unit over an empty cache.
template <typename T>
__device__ __forceinline__ void ch_nothing(const ChunkArgs &a, const ChunkRow &row) {
    if (!row.valid) return;
    const float zero[8] = {};
    for (int d = 0; d < a.head_dim; d += 8) rope_store8(static_cast<T *>(a.out) + row.out + d, zero);
    if (a.lse) a.lse[row.lse] = -INFINITY;
}

// The weights of sixteen columns, from their scores, as f16 words (PL = 2: and
// what those leave), their sum at the row's maximum added to l.
// CAREFUL: columns past `rel` are not seen, and product and difference round one
// by one, as the maxima did, so that no weight is above its reference (past 2^20
// the rounding of a score shows beside that).
template <int PL, bool CAREFUL>
__device__ __forceinline__ void ch_weights(const float *v, int col, int rel, float k, float base, float log, float mantissa, float &l,
                                           uint32_t *hi, uint32_t *lo) {
    const uint64_t k2 = ch_pair(k, k), off2 = ch_pair(log - base, log - base);
    uint64_t sum = 0;
    float w[16];
#pragma unroll
    for (int x = 0; x < 16; x += 2) {
        float t0, t1;
        if (CAREFUL) {
            t0 = __fadd_rn(__fmul_rn(v[x], k), -base) + log;
            t1 = __fadd_rn(__fmul_rn(v[x + 1], k), -base) + log;
            t0 = col + x <= rel ? t0 : -INFINITY;
            t1 = col + x + 1 <= rel ? t1 : -INFINITY;
        } else {
            ch_unpair(ch_fma2(ch_pair(v[x], v[x + 1]), k2, off2), t0, t1);
        }
        w[x] = at_exp2(t0);
        w[x + 1] = at_exp2(t1);
        sum = ch_add2(sum, ch_pair(w[x], w[x + 1]));
    }
    float s0, s1;
    ch_unpair(sum, s0, s1);
    l = fmaf(s0 + s1, at_exp2(-log), l);
    if (mantissa != 1.f) {
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] *= mantissa;
    }
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        hi[x] = ch_pack_f16(w[2 * x], w[2 * x + 1]);
        if (PL == 2) {
            const float2 b = ch_unpack_f16(hi[x]);
            lo[x] = ch_pack_f16(w[2 * x] - b.x, w[2 * x + 1] - b.y);
        }
    }
}

// The scores of a tile in turn, 32 columns at a time, the next ones on their way.
template <int T, typename F>
__device__ __forceinline__ void ch_columns(uint32_t s_col, F f) {
    float v[2][32];
    ch_ld32(s_col, v[0]);
#pragma unroll
    for (int c = 0; c < T; c += 32) {
        at_wait_ld();
        if (c + 32 < T) ch_ld32(s_col + c + 32, v[(c / 32 + 1) & 1]);
        f(c, v[(c / 32) & 1]);
    }
}

template <typename Sh, typename T>
__device__ __forceinline__ void ch_softmax(const ChunkArgs &a, ChunkWalk<Sh> w, ChunkShared &sh, uint32_t tmem, int product, int wq, int lane) {
    constexpr int PL = Sh::PL, kTile = Sh::T;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t o_col = tmem + lanes + static_cast<uint32_t>(Sh::kSumCol + product * 128);
    const int local = product * 128 + wq * 32 + lane;
    int it = 0, unit = 0;   // all tiles of the CTA; units with tiles
    int mine = 0;           // tiles of this product
    bool ok = true;
    do {
        const ChunkRow row(a, w, local);
        if (w.tiles == 0 && !Sh::SUMS) ch_nothing<T>(a, row);
        if (w.none()) continue;
        const int ub = unit & 1, tiles = w.j1 - w.j0;
        // (Also without rows: no product's report runs ahead of the unit.)
        ok = ok && at_warp_wait(smem_addr(&sh.q_full[ub]), static_cast<uint32_t>(unit >> 1) & 1u, &sh.abort, a.wait_limit_ns);
        if (product >= w.products()) {  // no rows
            it += tiles;
            if (lane == 0) mbar_arrive(smem_addr(&sh.unit_done[ub]));
            ++unit;
            continue;
        }
        const float qs = sh.qs[ub][local];
        float M = kChNone, R = kChNone, l = 0.f;  // maximum, the weights' reference less M, denominator
        for (int j = 0; ok && j < tiles; ++j, ++it, ++mine) {
            const int sb = Sh::NS == 1 ? mine & 1 : 0;
            const uint32_t s_col = tmem + lanes + static_cast<uint32_t>(Sh::NS == 1 ? sb * kTile : product * 128);
            ok = at_warp_wait(smem_addr(&sh.s_full[Sh::NS == 1 ? sb : product]), static_cast<uint32_t>(Sh::NS == 1 ? mine >> 1 : mine) & 1u,
                              &sh.abort, a.wait_limit_ns) &&
                 at_warp_wait(smem_addr(&sh.info_full[it & (kChInfo - 1)]), static_cast<uint32_t>(it / kChInfo) & 1u, &sh.abort, a.wait_limit_ns);
            if (!ok) break;
            t8_fence_after();
            const float4 *info = sh.info[it & (kChInfo - 1)];
            const int64_t t0 = static_cast<int64_t>(w.j0 + j) * kTile;
            const int rel = t0 > row.last ? -1 : static_cast<int>(row.last - t0 < kTile ? row.last - t0 : kTile);  // last column this row sees
            const bool masked = __any_sync(0xFFFFFFFFu, rel < kTile - 1);
            // Maxima of sixteens, then the row's.
            float top = M, m16[kTile / 16];
            ch_columns<kTile>(s_col, [&](int c, float (&v)[32]) {
                if (masked) {
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = c + x <= rel ? v[x] : -INFINITY;
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float m = v[16 * g];
#pragma unroll
                    for (int x = 1; x < 16; ++x) m = fmaxf(m, v[16 * g + x]);
                    m = m == -INFINITY ? m : ceilf(m * (info[c / 16 + g].x * qs));
                    top = fmaxf(top, m);
                    m16[c / 16 + g] = m;
                }
            });
            if (top > M) {
                l *= at_exp2(M - top);
                R = R > kChNone ? R - (top - M) : R;
                M = top;
            }
            float ref = kChNone;
#pragma unroll
            for (int g = 0; g < kTile / 16; ++g) ref = fmaxf(ref, (m16[g] - M) + info[g].y);
            const bool move = ref > R + kChSlack;
            const float factor = move && R > kChNone ? at_exp2(R - ref) : 1.f;  // of the sums so far
            if (Sh::SUMS) {
                sh.factor[it & (kChInfo - 1)][local] = factor;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.factor_full[it & (kChInfo - 1)]));
            } else if (j > 0 && __any_sync(0xFFFFFFFFu, move)) {
                ok = at_warp_wait(smem_addr(&sh.o_done[product]), static_cast<uint32_t>(mine - 1) & 1u, &sh.abort, a.wait_limit_ns);
                if (!ok) break;
                t8_fence_after();
#pragma unroll 1
                for (int c = 0; c < a.head_dim; c += 16) {
                    float v[16];
                    t8_ld16(o_col + c, v);
                    at_wait_ld();
                    uint32_t u[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(v[x] * factor);
                    ch_st16(o_col + c, u);
                }
                ch_wait_st();
            }
            if (move) R = ref;
            const float base = M > kChNone ? M : 0.f, lift = R > kChNone ? static_cast<float>(kChLift) - R : 0.f;
            auto weights = [&](auto careful) {
                ch_columns<kTile>(s_col, [&](int c, float (&v)[32]) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 f = info[c / 16 + g];
                        ch_weights<PL, decltype(careful)::value>(v + 16 * g, c + 16 * g, rel, f.x * qs, base, fmaxf(f.y + lift, kChMinLog), f.z, l,
                                                                 hi + 8 * g, lo + 8 * g);
                    }
                    if (PL == 1) {
                        ch_st16(s_col + c / 2, hi);
                    } else {
                        ch_st16(s_col + c, hi);
                        ch_st16(s_col + c + 16, lo);
                    }
                });
            };
            if (masked || __any_sync(0xFFFFFFFFu, fabsf(base) >= 0x1p20f)) weights(std::true_type{});
            else weights(std::false_type{});
            ch_wait_st();
            t8_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[Sh::NS == 1 ? sb : product]));
        }
        if (Sh::SUMS) {
            sh.last[ub][0][local] = M;
            sh.last[ub][1][local] = R;
            sh.last[ub][2][local] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.last_full[ub]));
        } else {
            ok = ok && at_warp_wait(smem_addr(&sh.o_done[product]), static_cast<uint32_t>(mine - 1) & 1u, &sh.abort, a.wait_limit_ns);
            t8_fence_after();
            ch_finish<Sh, T>(a, w, sh, unit, row, local, o_col, M, R, l, ok);
            t8_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.unit_done[ub]));
        }
        ++unit;
    } while (w.next());
}

// f32's sums: each tile's product, out of tensor memory, onto the sums there,
// rounded; at a unit's end its rows are written out.
template <typename Sh, typename T>
__device__ __forceinline__ void ch_sums(const ChunkArgs &a, ChunkWalk<Sh> w, ChunkShared &sh, uint32_t tmem, int wq, int lane) {
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t p_col = tmem + lanes + static_cast<uint32_t>(Sh::kProductCol), o_col = tmem + lanes + static_cast<uint32_t>(Sh::kSumCol);
    const int local = wq * 32 + lane;
    int it = 0, unit = 0, products = 0;
    bool ok = true;
    do {
        const ChunkRow row(a, w, local);
        if (w.tiles == 0) ch_nothing<T>(a, row);
        if (w.none()) continue;
        const int ub = unit & 1, tiles = w.j1 - w.j0;
        for (int j = 0; ok && j < tiles; ++j, ++it) {
            ok = at_warp_wait(smem_addr(&sh.factor_full[it & (kChInfo - 1)]), static_cast<uint32_t>(it / kChInfo) & 1u, &sh.abort, a.wait_limit_ns);
            const float factor = sh.factor[it & (kChInfo - 1)][local];
#pragma unroll 1
            for (int h = 0; ok && h < Sh::kHalves; ++h, ++products) {
                ok = at_warp_wait(smem_addr(&sh.o_done[0]), static_cast<uint32_t>(products) & 1u, &sh.abort, a.wait_limit_ns);
                if (!ok) break;
                t8_fence_after();
                const int c0 = 128 * h, c1 = min(a.head_dim, c0 + 128);
#pragma unroll 1
                for (int c = c0; c < c1; c += 16) {
                    float p[16], o[16];
                    t8_ld16(p_col + c - c0, p);
                    if (j > 0) t8_ld16(o_col + c, o);
                    at_wait_ld();
                    uint32_t u[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) u[x] = __float_as_uint(j > 0 ? fmaf(o[x], factor, p[x]) : p[x]);
                    ch_st16(o_col + c, u);
                }
                t8_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.product_free));
            }
        }
        ch_wait_st();
        ok = ok && at_warp_wait(smem_addr(&sh.last_full[ub]), static_cast<uint32_t>(unit >> 1) & 1u, &sh.abort, a.wait_limit_ns);
        ch_finish<Sh, T>(a, w, sh, unit, row, local, o_col, sh.last[ub][0][local], sh.last[ub][1][local], sh.last[ub][2][local], ok);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.unit_done[ub]));
        ++unit;
    } while (w.next());
}

// ------------------------------------------------------------------ the kernel
template <typename T, int PL, bool WIDE>
__global__ void __launch_bounds__(kChThreads, 1) kv_chunk_kernel(const ChunkArgs a) {
    using Sh = ChunkShape<PL, WIDE>;
    extern __shared__ __align__(1024) uint8_t ch_smem[];
    __shared__ __align__(16) ChunkShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *sq = ch_smem + ((1024u - (smem_addr(ch_smem) & 1023u)) & 1023u);
    uint8_t *slots = sq + Sh::kQ;
    if (tid == 0) {
        for (int i = 0; i < Sh::kSlots; ++i) {
            mbar_init(smem_addr(&sh.slot_full[i]), kChConvertWarps);
            mbar_init(smem_addr(&sh.slot_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_full[i]), 4);
            mbar_init(smem_addr(&sh.o_done[i]), 1);
            mbar_init(smem_addr(&sh.q_full[i]), kChConvertWarps);
            mbar_init(smem_addr(&sh.values_done[i]), kChConvertWarps);
            mbar_init(smem_addr(&sh.unit_done[i]), 4 * Sh::NS);
        }
        for (int i = 0; i < kChInfo; ++i) {
            mbar_init(smem_addr(&sh.info_full[i]), 1);
            mbar_init(smem_addr(&sh.factor_full[i]), 4);
        }
        mbar_init(smem_addr(&sh.last_full[0]), 4);
        mbar_init(smem_addr(&sh.last_full[1]), 4);
        mbar_init(smem_addr(&sh.product_free), 4);
        mbar_init(smem_addr(&sh.q_free), 1);
        mbar_init(smem_addr(&sh.mma_done), 1);
        mbar_init_fence();
        sh.abort = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    t8_fence_before();
    __syncthreads();
    t8_fence_after();
    const uint32_t tmem = sh.tmem;
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the list, scanned by every CTA: thread i sums requests [i each, (i + 1) each).
    int64_t total = 0;
    int grid = 0;
    {
        const int each = (a.n_seqs + kChThreads - 1) / kChThreads;
        const int r0 = min(tid * each, a.n_seqs), r1 = min(r0 + each, a.n_seqs);
        int64_t sum = 0;
        bool bad = false;
        for (int s = r0; s < r1; ++s) {
            const ChunkSeq q = ch_seq<Sh>(a, s);
            sum += q.entries();
            bad |= q.bad;
        }
        if (bad && blockIdx.x == 0) atomicOr(a.status, 4u);
        int64_t pre = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, pre, d);
            if (lane >= d) pre += u;
        }
        if (lane == 31) sh.scan[warp] = pre;
        __syncthreads();
        int64_t base = 0;
        for (int i = 0; i < kChThreads / 32; ++i) {
            const int64_t u = sh.scan[i];
            if (i < warp) base += u;
            total += u;
        }
        // Every CTA's share is a few entries, so no two cuts inside a unit meet.
        grid = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(total / 8, min(total, int64_t(1)))));
        const int64_t from = base + pre - sum;
        if (static_cast<int>(blockIdx.x) < grid) {
            for (int e = 0; e < 2; ++e) {
                const int64_t share = total / grid, rest = total - share * grid, b = blockIdx.x + e;
                const int64_t x = b * share + min(b, rest);
                if (e == 1 && x == total) {
                    if (tid == 0) sh.cut[1] = total;
                } else if (from <= x && x < from + sum) {
                    int64_t here = from;
                    int s = r0;
                    ChunkSeq q = ch_seq<Sh>(a, s);
                    while (x >= here + q.entries()) {
                        here += q.entries();
                        q = ch_seq<Sh>(a, ++s);
                    }
                    const ChunkPlace p = ch_place(q, x - here, [](const ChunkSeq &q, int64_t x) {
                        int lo = 0, hi = q.row_tiles - 1;
                        while (lo < hi) {
                            const int mid = (lo + hi + 1) >> 1;
                            if (q.before(mid) <= x) lo = mid;
                            else hi = mid - 1;
                        }
                        return lo;
                    });
                    sh.cut[e] = here + p.at;
                    if (e == 0) {
                        sh.at[0] = s;
                        sh.at[1] = p.row_tile;
                        sh.at[2] = p.head;
                        sh.at[3] = p.slot;
                    }
                }
            }
        }
        __syncthreads();
    }
    const bool busy = static_cast<int>(blockIdx.x) < grid && sh.cut[0] < sh.cut[1];
    bool issued = false;
    if (busy) {
        ChunkWalk<Sh> w(a, sh.at, sh.cut[1] - sh.cut[0]);
        if (warp < kChConvertWarp) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChSoftmaxRegs));
            if (warp < 4 * Sh::NS) ch_softmax<Sh, T>(a, w, sh, tmem, warp >> 2, warp & 3, lane);
            else if (Sh::SUMS) ch_sums<Sh, T>(a, w, sh, tmem, warp & 3, lane);
        } else if (warp < kChMmaWarp) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChConvertRegs));
            ch_convert<Sh, T>(a, w, sh, sq, slots, tid - kChConvertWarp * 32);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChIssueRegs));
            if (warp != kChMmaWarp) {
            } else if (lane == 0) {
                issued = ch_issue<Sh>(a, w, sh, tmem, smem_addr(sq), smem_addr(slots));
                if (issued) {  // also after a wait that ran out: nothing is in flight at the end
                    t8_commit(smem_addr(&sh.mma_done));
                    (void)mbar_wait_bounded(smem_addr(&sh.mma_done), 0);
                }
            } else if (lane == 1) {
                // What the join needs: the last unit, and which ends of the range are cuts.
                const bool first_cut = !w.starts();
                bool alone = true;
                while (w.next()) alone = false;
                const bool last_cut = !w.ends();
                a.heads[2 * blockIdx.x] = make_int4(w.s, w.row_tile, w.head,
                                                    (last_cut && (w.starts() || !alone) ? 1 : 0) | (alone && first_cut && last_cut ? 2 : 0));
                a.heads[2 * blockIdx.x + 1] = make_int4(w.q.first, w.q.rows, 0, 0);
            }
        }
    } else if (tid == 0) {
        a.heads[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    t8_fence_before();
    __syncthreads();
    if (tid == 0 && *reinterpret_cast<volatile int *>(&sh.abort)) atomicOr(a.status, 1u);
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Joins the parts of units that lie across CTAs.  CTA (x, y): rows [8 y, 8 y + 8)
// of the unit that CTA x of the first kernel began and did not end (if there is
// one); its parts lie with x, x + 1, .. as far as their ranges go on.  Warp r
// weighs the parts of row r, then takes four elements a lane of its sums.
template <typename T, int U>
__global__ void __launch_bounds__(kChJoinRows * 32) kv_chunk_join_kernel(const ChunkArgs a, int grid) {
    __shared__ float weight[kChJoinRows][kChMaxGrid];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    const int4 h = a.heads[2 * b];
    if ((h.w & 1) == 0) return;
    const int4 rows = a.heads[2 * b + 1];
    const int local = blockIdx.y * kChJoinRows + warp, r = h.y * U + local;
    if (r >= rows.y * a.group) return;  // (warps go their own ways from here on)
    int parts = 2;
    while (b + parts < grid && (a.heads[2 * (b + parts - 1)].w & 2) != 0) ++parts;
    const int64_t size = static_cast<int64_t>(U) * (a.head_dim + 2);
    auto part = [&](int p) { return a.partials + (static_cast<int64_t>(b + p) * 2 + (p == 0)) * size; };
    float M = kChNone;
    bool nan = false;
    for (int p = lane; p < parts; p += 32) M = fmaxf(M, __ldcg(part(p) + static_cast<int64_t>(U) * a.head_dim + local));
#pragma unroll
    for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
        const float f = at_exp2(__ldcg(part(p) + static_cast<int64_t>(U) * a.head_dim + local) - M);
        const float pl = __ldcg(part(p) + static_cast<int64_t>(U) * (a.head_dim + 1) + local);
        weight[warp][p] = f;
        l = fmaf(pl, f, l);
        nan |= pl != pl;
    }
    // One order, one result.
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const float o = __shfl_xor_sync(0xFFFFFFFFu, l, d);
        l = lane & d ? o + l : l + o;
    }
    nan = __any_sync(0xFFFFFFFFu, nan);
    if (nan) l = __int_as_float(0x7FC00000);
    __syncwarp();
    const int token = r / a.group;
    const int64_t row = rows.x + token, head = static_cast<int64_t>(h.z) * a.group + (r - token * a.group);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (lane == 0 && a.lse) a.lse[row * (static_cast<int64_t>(a.kv_heads) * a.group) + head] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + head * a.head_dim;
    for (int d = 4 * lane; d < a.head_dim; d += 128) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int p = 0; p < parts; ++p) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(part(p) + static_cast<int64_t>(local) * a.head_dim + d));
            const float f = weight[warp][p];
            o.x = fmaf(x.x, f, o.x);
            o.y = fmaf(x.y, f, o.y);
            o.z = fmaf(x.z, f, o.z);
            o.w = fmaf(x.w, f, o.w);
        }
        at_store4(out + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
}

}  // namespace fp8blk
