// kv_chunk.cuh -- attention of any number of new rows per request over the
// paged e4m3 cache (prompts, chunks of prompts), on the fifth-generation tensor
// cores.
//
// For one request and cache head, a tile of 128 query rows (row = new token x
// query head of the group) against a tile of T = 128 tokens (64 where there is one
// product only):
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
// Row tiles are 256 rows (two products' rows) for bf16 with head_dim <= 128, else
// 128.  A unit (request, row tile, head) that lies across CTAs leaves partial sums
// in the workspace, which a second kernel joins, in CTA order (deterministic, no
// counters).
//
// Two products take turns: while one's softmax runs, the other's MMAs do.  The
// second MMA starts on the first half of a tile's weights.  (Tiles of 64 tokens and
// two score buffers a product cost more instructions than they hid latency: 2.3 ms
// for the first call below.)  One product has two score buffers of 64 tokens: the
// next scores are there when a softmax ends.
//
// A unit with 128 rows or fewer gives every other of its tiles to the second
// product, and the two are added up at its end (the third call below took 89 us with
// one product at work).
//
// Measured, calls in a row, the cache not in L2:
//   4096 rows at the end of 16384 tokens, 64 / 8 heads of 128, bf16    2.04 ms, 944 TFLOP/s, 49% of the matrix rate
//   512 rows of 8192 tokens, the same heads                            178 us, 748 TFLOP/s, 39%
//   16 rows of 65536 tokens, 32 / 8 heads, bf16                        82 us, 1.64 TB/s, 24% of the copy rate
//   8 ragged prompts of up to 1024 tokens, 32 / 8 heads, f32           231 us, 132 TFLOP/s, 14% of the rate at two planes
//   8 prompts of 1024, the same heads, bf16; f32                       183 us, 19%; 447 us, 16%
//   16 prompts of 700, 8 / 2 heads of 256, bf16; f32                   138 us, 12%; 224 us, 15%
//   9 requests of up to 2001 tokens, 15 / 3 heads of 80, bf16          55 us
// Long calls are bound by a tile's chain: scores, softmax, weights' MMA.  256 rows x
// 128 tokens take 5100 cycles, 2048 of them MMAs; a softmax group is at work for
// 3500, its 700 instructions a warp slowed by the other roles' and by instruction
// caches (148 KiB of code).  Short calls are bound by what comes before and
// after their tiles, about 45 us: 7 us up to the first unit, 5 for its first tiles,
// 3 for queries, 4 for writing a unit out, the join (9 in the third call).  That a unit
// costs so much beside its tiles is in the list's weights.
//
// Roles (640 threads, one CTA per SM): warps 0-3 softmax (TMEM lane = row), warps
// 4-7 softmax of the unit's second 128 rows, or f32's sums, warps 8-15 convert q, K
// and V, warps 16 and 17 issue the MMAs (of the first and second 128 rows), warp 18
// walks the list and lays out the units to come.  Every wait is bounded; a timeout
// raises a CTA-wide flag, the outputs and lse of the CTA's rows become NaN (also
// those of units that were not laid out any more), MMAs in flight are waited for,
// and the status word records it.
#pragma once

#include "kv_attn.cuh"
#include "kv_chunk_copy.h"
#include "rope.cuh"

#include <type_traits>

namespace fp8blk {

constexpr int kChThreads = 640;
constexpr int kChConvertWarp = 8, kChConvertWarps = 8, kChMmaWarp = 16, kChPlanWarp = 18;
constexpr int kChMaxGrid = 160;          // bound on CTAs: partial sums in the workspace
// CTAs of the join for one of the first kernel: with 4, 8 and 16 of them 9 requests of up to 2001 tokens took 67, 62 and 62 us.
constexpr int kChJoinCtas = 8;
constexpr int kChInfo = 8;               // tiles whose scales (and sums' factors) are held: more than K is ahead of the softmax
// Tiles that a unit costs beside its own: queries, first tiles, writing out.  With 1, 2, 4 and 8 the 8 ragged prompts of f32 rows
// took 316, 264, 234 and 241 us; 8 of 1024 bf16 rows, 32 / 8 heads, 245, 207 and 191 us with 1, 2 and 4.
constexpr int kChSetUp = 4;
constexpr int kChUnits = 4;              // units that are laid out ahead
// Registers a thread of each role (of the 96 of the launch).
constexpr int kChSoftmaxRegs = 112, kChConvertRegs = 104, kChIssueRegs = 48;
static_assert(256 * kChSoftmaxRegs + 256 * kChConvertRegs + 128 * kChIssueRegs <= kChThreads * 96, "registers");
constexpr int kChLift = 6;               // K: a row's largest weight is below 2^6 when R moves, below 2^15 at most
constexpr int kChSlack = 8;              // ... which it does when a tile passes it by more than 2^8
constexpr float kChNone = -3.0e38f;      // maximum of a row that has seen nothing
constexpr float kChMinLog = -60.f;       // weights under value scales smaller than 2^-60 of their row's are zero in f16 anyway
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
    uint32_t group_inverse;           // floor((2^32 - 1) / group)
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
    static constexpr int T = U / 2;                     // tokens of a tile
    static constexpr int kDeep = NS == 1 ? 2 : 1;       // score buffers of a product
    static constexpr int kBlocks = WIDE ? 4 : 2;        // 64-wide column blocks of a head
    static constexpr int kSlot = T * kBlocks * 128;     // K or V of a tile as f16: 16 or 32 KiB
    static constexpr int kSlots = WIDE ? 1 : NS == 2 ? 2 : 3;  // of K, and as many of V
    static constexpr int kRaw = kSlot / 2;              // ... of the codes as they are: copied ahead
    static constexpr int kRaws = NS == 2 ? 1 : !WIDE ? 6 : PL == 1 ? 4 : 1;  // of K and V in turn
    static constexpr int kEach = kSlot / (32 * 256);    // groups of sixteen codes of a converting thread
    static constexpr int kQPlane = 128 * kBlocks * 128;  // one plane of 128 rows
    static constexpr int kQ = NS * PL * kQPlane;
    static constexpr size_t kSmem = 1024 + kQ + 2 * kSlots * kSlot + kRaws * kRaw;
    static constexpr int kGranules = T / 16;            // scales of a tile
    // Tensor memory, in columns: scores (and the weights, in their place), of two products or in two buffers of one; f32's
    // product of a tile (half of a wide head at a time); the sums.
    static constexpr int kProductCol = 128, kSumCol = 256;
    static constexpr int kHalves = SUMS && WIDE ? 2 : 1;
    static constexpr int kIssuers = NS;                 // warps that issue MMAs, one a product
    static_assert(NS * kDeep * T <= 256, "tensor memory");
};

// One unit's tiles in a CTA's range.
struct ChunkUnit {
    int first, rows, len;   // its request: first row, rows, tokens
    int s, row0, head;      // request, first of the flat rows (row x query head of the group), cache head
    int j0, tiles;          // its tiles here (none: the cache is empty)
    int flags;              // below
};
constexpr int kChStarts = 1, kChEnds = 2, kChTwo = 4, kChStop = 8;  // first and last tile are here; two products have rows; no unit

// One request as the kernel takes it.  Tiles of the list are half as many tokens
// as a row tile has rows, so row tile i's last row sees the tiles
// 0 .. floor((a + 2 i) / g), as far as there are any.
struct ChunkSeq {
    int first, rows, len;  // rows 0: nothing to do
    int tiles;             // of the whole cache
    int row_tiles;
    int a, last;           // last: list entries of a tile of the last row tile
    bool bad;
};

struct ChunkShared {
    // Whoever waits on a barrier is never a whole turn of it behind: a wait could not tell the next phase but one from
    // its own.  So what a role may skip or be late for goes by the unit's or the score buffer's parity.
    uint64_t k_full[4], k_free[4], v_full[4], v_free[4], s_full[2], p_half[2], p_full[2], o_done[2], info_full[kChInfo];
    uint64_t q_full[2], values_done[2], unit_done[2], q_free, mma_done[2];
    uint64_t factor_full[kChInfo], last_full[2], product_free;  // f32's sums
    uint64_t merged;             // the first product has taken the second's share of a unit
    uint64_t unit_full[kChUnits], unit_free[kChUnits];
    float4 info[kChInfo][8];     // per sixteen tokens: k scale (NaN if not finite), exponent of the v scale, its signed mantissa
    int info_kind[kChInfo];      // of a tile's scales: 0 one per 64 tokens, 1 several, 2 a negative k scale, or a v scale that is no (positive) power of two
    ChunkUnit units[kChUnits];
    float qs[2][256];            // per row: what a score is times |s_k| of
    float factor[kChInfo][128];  // f32: what the sums so far are times, per row of a tile
    float last[2][3][128];       // f32, and a second product's share: a unit's maxima, references and denominators
    int vnan[2][256];            // first position whose value is NaN, per element
    int any_nan[2];
    int scan[kChThreads / 32];
    uint32_t scan_rows[kChThreads / 32];
    int cut[2];                  // this CTA's range
    int at[2][4];                // where its cuts lie: request (the first cut also: row tile, head and slot)
    ChunkSeq seq;                // the first one's request
    int abort;
    ChunkUnit lost;              // one that the layout does not hand on any more
    uint32_t tmem;
};

// ------------------------------------------------------------------ the list
// r / group and the remainder, r < 2^31 (the estimate is at most one too small).
__device__ __forceinline__ int ch_token(const ChunkArgs &a, int r, int &head) {
    int t = static_cast<int>(__umulhi(static_cast<uint32_t>(r), a.group_inverse));
    head = r - t * a.group;
    if (head >= a.group) {
        ++t;
        head -= a.group;
    }
    return t;
}
// A row of the unit: where it lies, and what it sees.
struct ChunkRow {
    int64_t out, lse;
    int last;    // last position it sees
    bool valid;
    __device__ __forceinline__ ChunkRow(const ChunkArgs &a, const ChunkUnit &w, int local) {
        int in_group;
        const int r = w.row0 + local, token = ch_token(a, r, in_group);
        const int64_t row = w.first + token, head = static_cast<int64_t>(w.head) * a.group + in_group;
        valid = r < w.rows * a.group;
        last = valid ? w.len - w.rows + token : 0x7FFFFFFF;  // (rows that are not there: zeros, stored nowhere)
        out = row * a.out_stride + head * a.head_dim;
        lse = row * (static_cast<int64_t>(a.kv_heads) * a.group) + head;
    }
};

// (Entries are counted in 32 bits: the host sees to it.)
// sum of floor((a + 2 i) / g) over i < n.  The floors of all integers from a to
// a + 2 n add up in closed form; of two neighbours x, x + 1 the second's is one more
// only where g divides x + 1, and those are counted.
__device__ __forceinline__ int64_t ch_floors_below(uint32_t x, uint32_t g) {
    const uint32_t q = x / g, r = x - q * g;
    return static_cast<int64_t>(g) * (static_cast<int64_t>(q) * (static_cast<int64_t>(q) - 1) / 2) + static_cast<int64_t>(q) * r;
}
__device__ __noinline__ int ch_floor_sum(uint32_t a, uint32_t g, uint32_t n) {
    if (n == 0) return 0;
    const uint32_t hi = a + 2 * n;
    int64_t all = ch_floors_below(hi, g) - ch_floors_below(a, g);
    // Multiples of g among a + 1, a + 3, .., hi - 1: of even g all in between, of odd g every other one.
    const bool odd = g & 1u;
    const uint32_t m = odd ? 2 * g : g, shift = odd && a % 2 == 0 ? g : 0;
    if (odd || a % 2 == 1) all -= (hi - 1 + shift) / m - (a + shift) / m;
    return static_cast<int>(all / 2);
}

template <typename Sh>
struct ChunkList {
    static constexpr int kFull = Sh::U / 128;  // list entries of a tile of a full row tile
    const ChunkArgs &a;
    __device__ __noinline__ ChunkSeq seq(int s) const {
        ChunkSeq q;
        q.first = a.q_starts[s];
        const int64_t rows = static_cast<int64_t>(a.q_starts[s + 1]) - q.first;
        const int len = a.seq_lens[s];
        const bool off = q.first < 0 || rows < 0 || q.first + rows > a.total_rows;
        q.bad = off || len < 0;
        q.rows = off ? 0 : static_cast<int>(rows);
        q.len = max(len, 0);
        q.tiles = min(q.len / Sh::T + (q.len % Sh::T != 0), a.max_tiles);
        const int flat = q.rows * a.group;
        q.row_tiles = flat / Sh::U + (flat % Sh::U != 0);
        // The first row's position, no further than the table's end (all tiles are seen from there on).
        const int p = min(max(q.len - q.rows, 0), a.max_tiles * Sh::T);
        q.a = static_cast<int>((static_cast<int64_t>(p) * a.group + Sh::U - 1) / Sh::T);
        q.last = flat - (q.row_tiles - 1) * Sh::U > 128 ? kFull : 1;
        return q;
    }
    __device__ __forceinline__ int seen(const ChunkSeq &q, int i) const { return min((q.a + 2 * i) / a.group + 1, q.tiles); }
    __device__ __forceinline__ int weight(const ChunkSeq &q, int i) const { return i + 1 == q.row_tiles ? q.last : kFull; }
    // Entries of the row tiles below i, i < row_tiles: each unit has kChSetUp slots for what it costs beside its tiles, and one per tile.
    __device__ __noinline__ int before(const ChunkSeq &q, int i) const {
        const int64_t lack = static_cast<int64_t>(q.tiles - 1) * a.group - q.a;  // from row tile ceil(lack / 2) on all tiles are seen
        const int some = lack <= 0 ? 0 : static_cast<int>(min((lack + 1) / 2, static_cast<int64_t>(i)));
        const int slots = ch_floor_sum(q.a, a.group, some) + some + (i - some) * q.tiles + i * kChSetUp;
        return slots * kFull * a.kv_heads;
    }
    __device__ __forceinline__ int entries(const ChunkSeq &q) const {
        return q.row_tiles == 0 ? 0 : before(q, q.row_tiles - 1) + a.kv_heads * q.last * (seen(q, q.row_tiles - 1) + kChSetUp);
    }
};

// A cut in a unit's set-up or first two tiles goes to the unit's start: joining
// parts costs more than they do.
constexpr int kChSmallCut = 2;

// CTA b's share of the list begins at entry floor(b total / grid), so that equal
// units whose number divides the grid are cut at their ends.
struct ChunkSplit {
    int each, more, grid;
    __device__ __forceinline__ ChunkSplit(int total, int grid) : each(total / grid), more(total - each * grid), grid(grid) {}
    __device__ __forceinline__ int begin(int b) const { return b * each + b * more / grid; }
};

// Waits of the ring of units.  They end because all others do: whoever has given up goes on taking units, so a unit's
// place is free at last, and the layout goes on to the end.  (No limit of a second for them: a unit may be a second's
// work, and the layout's wait begins before that of a role that stalls.)  What bounds them nevertheless is counted by
// their polls, so that a GPU that stood still in between does not end them.  The layout's: 16 s, a poll for a
// millisecond at most.
constexpr uint64_t kChLayoutLimitNs = 16 * kWaitLimitNs;
__device__ __forceinline__ bool ch_layout_wait(uint32_t at, uint32_t parity) {
    uint64_t last = global_timer_ns(), spent = 0;
#pragma unroll 1
    while (!mbar_try_wait(at, parity)) {
        const uint64_t now = global_timer_ns(), step = now - last;
        spent += step < 1000000 ? step : 1000000;
        if (spent >= kChLayoutLimitNs) return false;
        last = now;
    }
    return true;
}
// The roles': a minute or more (a poll takes 40 ns to 1.5 us), longer than any silence of the layout.
constexpr uint32_t kChRolePolls = 1u << 30;
__device__ __forceinline__ bool ch_role_wait(uint32_t at, uint32_t parity) {
#pragma unroll 1
    for (uint32_t n = 0; n < kChRolePolls; ++n)
        if (mbar_try_wait_short(at, parity)) return true;
    return false;
}

// The rows of a unit that no role will see: NaN, as where other waits ran out.  (One thread.)
template <typename Sh, typename T>
__device__ __forceinline__ void ch_lose(const ChunkArgs &a, const ChunkUnit &x) {
    const float nanf = __int_as_float(0x7FC00000);
    if ((x.flags & (kChStarts | kChEnds)) != (kChStarts | kChEnds)) {  // a part: by its denominators
        float *l = a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (x.flags & kChStarts)) * (static_cast<int64_t>(Sh::U) * (a.head_dim + 2)) +
                   static_cast<int64_t>(Sh::U) * (a.head_dim + 1);
#pragma unroll 1
        for (int r = 0; r < Sh::U; ++r) __stcg(l + r, nanf);
        return;
    }
#pragma unroll 1
    for (int r = 0; r < Sh::U; ++r) {
        const ChunkRow row(a, x, r);
        if (!row.valid) return;
#pragma unroll 1
        for (int d = 0; d < a.head_dim; ++d) static_cast<T *>(a.out)[row.out + d] = static_cast<T>(nanf);
        if (a.lse) a.lse[row.lse] = nanf;
    }
}

// Lays out the CTA's units (one thread), each in the place of the one kChUnits
// before it.  What the join needs goes to a.heads: the last unit, whether it is cut
// and begins here (1), and whether the whole range is the middle of one unit (2).
//   After a wait that ran out the rest goes round without the roles, which hear of
// it by the flag, and of the end by a stop in the place that was waited for.  (A
// limit shorter than the usual one holds here too: a test comes by such units so.)
template <typename Sh, typename T>
__device__ __forceinline__ void ch_plan(const ChunkArgs &a, ChunkShared &sh) {
    const ChunkList<Sh> list{a};
    int s = sh.at[0][0], row_tile = sh.at[0][1], head = sh.at[0][2], e0 = sh.at[0][3], left = sh.cut[1] - sh.cut[0];
    ChunkSeq q = sh.seq;
    const bool first_cut = e0 != 0;
    bool lost = false;
    for (int u = 0;;) {
        const int slot = u & (kChUnits - 1);
        if (u >= kChUnits && !lost) {
            const uint32_t at = smem_addr(&sh.unit_free[slot]), parity = static_cast<uint32_t>(u / kChUnits - 1) & 1u;
            lost = !(a.wait_limit_ns < kWaitLimitNs ? mbar_wait_limit(at, parity, a.wait_limit_ns) : ch_layout_wait(at, parity));
            if (lost) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
        }
        if (left <= 0) {
            if (lost && !ch_layout_wait(smem_addr(&sh.unit_free[slot]), static_cast<uint32_t>(u / kChUnits - 1) & 1u)) return;
            sh.units[slot].flags = kChStop;
            mbar_arrive(smem_addr(&sh.unit_full[slot]));
            return;
        }
        ChunkUnit &x = lost ? sh.lost : sh.units[slot];
        const int tiles = list.seen(q, row_tile), weight = list.weight(q, row_tile);
        const int e1 = min(tiles + kChSetUp, e0 + (weight == 2 ? left >> 1 : left));
        left -= (e1 - e0) * weight;
        x.first = q.first;
        x.rows = q.rows;
        x.len = q.len;
        x.s = s;
        x.row0 = row_tile * Sh::U;
        x.head = head;
        x.j0 = max(e0 - kChSetUp, 0);
        x.tiles = e1 - kChSetUp - x.j0;
        x.flags = (e0 == 0 ? kChStarts : 0) | (e1 == tiles + kChSetUp ? kChEnds : 0) | (weight == 2 ? kChTwo : 0);
        if (lost) ch_lose<Sh, T>(a, x);
        else mbar_arrive(smem_addr(&sh.unit_full[slot]));
        if (left <= 0) {
            const bool last_cut = e1 != tiles + kChSetUp;
            a.heads[2 * blockIdx.x] = make_int4(s, row_tile, head, (last_cut && e0 == 0 ? 1 : 0) | (u == 0 && first_cut && last_cut ? 2 : 0));
            a.heads[2 * blockIdx.x + 1] = make_int4(q.first, q.rows, 0, 0);
        } else if (++head == a.kv_heads) {
            head = 0;
            if (++row_tile == q.row_tiles) {
                row_tile = 0;
                do q = list.seq(++s);
                while (q.rows == 0);
            }
        }
        e0 = 0;
        u += !lost;
    }
}

// A role's wait, for a whole warp: for at most the limit, or until another role has
// raised the abort flag.
__device__ __forceinline__ bool ch_wait(const ChunkArgs &a, ChunkShared &sh, uint64_t &bar, uint32_t parity) {
    const uint32_t at = smem_addr(&bar);
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait_short(at, parity))) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (int n = 1; !__all_sync(0xFFFFFFFFu, mbar_try_wait_short(at, parity)); ++n) {
        if ((n & 15) != 0) continue;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 >= a.wait_limit_ns) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
        if (__any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int *>(&sh.abort) != 0)) return false;
    }
    return true;
}

// ... with a limit shorter than the usual one, looked at from the first poll on: the
// polls above sleep in between.  (The MMAs' wait for a unit's queries alone takes it,
// and the other roles hear of it by the flag.  Code in every wait costs all roles
// instruction cache: this one in all of them, 3% of a long call.)
__device__ __noinline__ bool ch_wait_brief(uint32_t at, uint32_t parity, uint64_t limit_ns, volatile int *abort) {
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    while (!__all_sync(0xFFFFFFFFu, mbar_test_wait(at, parity))) {
        if (global_timer_ns() - t0 >= limit_ns) *abort = 1;
        if (__any_sync(0xFFFFFFFFu, *abort != 0)) return false;
    }
    return true;
}

// Whether no role has given up.  One that has goes on arriving at the barriers that are a unit's (unit_done, last_full,
// merged), so after a wait at one of those a whole warp asks here: what it waited for may be an arrival of a later unit.
__device__ __forceinline__ bool ch_alive(const ChunkShared &sh) {
    return __all_sync(0xFFFFFFFFu, *reinterpret_cast<const volatile int *>(&sh.abort) == 0);
}

// The u-th unit, for a warp; false after the last one.
__device__ __forceinline__ bool ch_unit(ChunkShared &sh, int u, int lane, ChunkUnit &x) {
    const int slot = u & (kChUnits - 1);
    if (!__all_sync(0xFFFFFFFFu, ch_role_wait(smem_addr(&sh.unit_full[slot]), static_cast<uint32_t>(u / kChUnits) & 1u))) {
        *reinterpret_cast<volatile int *>(&sh.abort) = 1;
        return false;
    }
    x = sh.units[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&sh.unit_free[slot]));
    return (x.flags & kChStop) == 0;
}

// ------------------------------------------------------------------ pieces
// kind::f16 instruction descriptor: f16 A and B, f32 D; B K-major or MN-major.
__host__ __device__ constexpr uint32_t ch_idesc(int n, bool mn_major) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24) | (mn_major ? 1u << 16 : 0u);
}
// Shared-memory descriptors, as two words: 128-byte swizzle, 8-row groups 1024 bytes apart.  `lead`: bytes between
// 64-element blocks along N of an MN-major operand.  An offset inside shared memory adds to the low word, in 16 bytes.
__device__ __forceinline__ uint32_t ch_desc(uint32_t saddr, uint32_t lead) { return ((saddr >> 4) & 0x3FFFu) | (lead >> 4) << 16; }
constexpr uint32_t kChDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
// The MMAs, and the commit, of a converged warp: one thread issues, by a predicate
// inside, so that operands are made once a warp, by the uniform units.  (Alone on an
// SM an MMA takes 42 cycles to issue so, unrolled, 58 in a branch that one thread
// takes, 86 there in a loop.)
__device__ __forceinline__ void ch_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\tmov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(kChDescHigh)
        : "memory");
}
__device__ __forceinline__ void ch_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xFFFFFFFF;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(kChDescHigh)
        : "memory");
}
__device__ __forceinline__ void ch_commit(uint64_t &bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(&bar))
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
// The largest of three.
__device__ __forceinline__ float ch_max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float ch_max16(const float *v) {
    float m = ch_max3(v[0], v[1], v[2]), n = ch_max3(v[3], v[4], v[5]);
#pragma unroll
    for (int x = 6; x < 14; x += 4) {
        m = ch_max3(m, v[x], v[x + 1]);
        n = ch_max3(n, v[x + 2], v[x + 3]);
    }
    m = ch_max3(m, v[14], v[15]);
    return fmaxf(m, n);
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float ch_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// A unit's queries.  They are copied as they are to where their f16 planes will
// lie (all copies in flight at once; a bf16 row is as long as one plane, an f32 row
// as two), and converted in place: a warp takes two rows at a time (one of a wide
// head), sixteen (32) lanes a row, eight values a lane.  (Short loops: this code
// runs once a unit, and unrolled its instructions took longer to come than the
// queries: 13 us a unit.)
template <typename Sh, typename T>
struct ChunkQueries {
    static constexpr int L = Sh::WIDE ? 32 : 16, RW = 32 / L, PL = Sh::PL, kStride = kChConvertWarps * RW;
    const ChunkArgs &a;
    uint8_t *sq;
    float *qs;
    int warp, lane, d0, rows, flat, row0, here;
    const T *q;
    __device__ __forceinline__ ChunkQueries(const ChunkArgs &a, const ChunkUnit &w, uint8_t *sq, float *qs, int warp, int lane)
        : a(a), sq(sq), qs(qs), warp(warp), lane(lane), d0((lane % L) * 8), rows(w.flags & kChTwo ? 256 : 128),
          flat(w.rows * a.group - w.row0),  // rows of the unit that exist
          row0(w.row0), here(min(rows, flat)),
          q(static_cast<const T *>(a.q) + w.first * a.q_stride + static_cast<int64_t>(w.head) * a.group * a.head_dim + d0) {}
    __device__ __forceinline__ uint8_t *place(int r) const {
        return sq + (r >> 7) * (PL * Sh::kQPlane) + (d0 >> 6) * (128 * 128) + (r & 127) * 128 + ((((d0 >> 3) & 7) ^ (r & 7)) << 4);
    }
    __device__ __forceinline__ void copy() const {
#pragma unroll 1
        for (int r = warp * RW + lane / L; r < rows; r += kStride) {
            int head;
            const int token = ch_token(a, row0 + r, head);
            const T *x = q + token * a.q_stride + head * a.head_dim;
            const uint32_t dst = smem_addr(place(r)), bytes = r < flat && d0 < a.head_dim ? 16 : 0;  // the rest is filled with zeros
            if (bytes == 0) x = static_cast<const T *>(a.q);
            if (r >= flat && lane % L == 0) qs[r] = 1.f;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(x), "r"(bytes) : "memory");
            if (PL == 2) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + Sh::kQPlane), "l"(x + (bytes ? 4 : 0)), "r"(bytes) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void convert() const {
        // (Two of a warp's turns in one, so that one's loads and reductions cover the other's.)
#pragma unroll 1
        for (int rb = warp * RW; rb < here; rb += 2 * kStride) {
            float x[2][8];
            uint32_t top[2] = {0, 0};
            uint8_t *const at[2] = {place(rb + lane / L), place(rb + lane / L + kStride)};
            const bool two = rb + kStride < here;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if constexpr (PL == 2) {
                    const float4 u = *reinterpret_cast<const float4 *>(at[b & two]), v = *reinterpret_cast<const float4 *>(at[b & two] + Sh::kQPlane);
                    x[b][0] = u.x, x[b][1] = u.y, x[b][2] = u.z, x[b][3] = u.w, x[b][4] = v.x, x[b][5] = v.y, x[b][6] = v.z, x[b][7] = v.w;
                } else {
                    rope_load8(reinterpret_cast<const __nv_bfloat16 *>(at[b & two]), x[b]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (PL == 2) x[b][i] = fmaf(x[b][i], a.c, x[b][i] * a.c_low);  // the scale per value, rounded at random
                    top[b] = max(top[b], __float_as_uint(fabsf(x[b][i])));
                }
            }
#pragma unroll
            for (int d = L / 2; d; d >>= 1) {
#pragma unroll
                for (int b = 0; b < 2; ++b) top[b] = max(top[b], __shfl_xor_sync(0xFFFFFFFFu, top[b], d));
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const bool good = top[b] < 0x7F800000u;
                int e = 0;  // the row's largest times 2^e is in [2^14, 2^15)
                if (good && top[b] != 0) e = top[b] >= 0x800000u ? 14 + 127 - static_cast<int>(top[b] >> 23) : 14 + 149 - (31 - __clz(top[b]));
                const int e1 = e >> 1, e2 = e - e1;
                // (bf16: the sign of the softmax scale goes here.)
                const float f1 = good ? ch_pow2(e1) : 0.f, f2 = PL == 1 && a.c < 0.f ? -ch_pow2(e2) : ch_pow2(e2);
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
                if (b == 1 && !two) continue;
                if (lane % L == 0)
                    qs[rb + lane / L + b * kStride] = good ? ch_pow2(-e1) * (PL == 2 ? 1.f : fabsf(a.c)) * ch_pow2(-e2) : __int_as_float(0x7FC00000);
                *reinterpret_cast<uint4 *>(at[b]) = make_uint4(h[0], h[1], h[2], h[3]);
                if (PL == 2) *reinterpret_cast<uint4 *>(at[b] + Sh::kQPlane) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
    }
};

// ------------------------------------------------------------------ converters
// Warps 8-15: q of each unit, then K and V of its tiles.  A thread has two or four
// groups of sixteen codes of a tile: it copies them to shared memory several tiles
// ahead (one slot, where there is no room for more, and into L2 four tiles ahead),
// and converts them there when they have come.  (Asynchronous copies, because the
// barriers' releases wait for loads under way: with the codes ahead in registers a
// tile cost 6000 cycles.)  Block ids and scales come four or eight tiles at a time, a
// lane for each sixteen tokens, one and two such windows ahead.
template <typename Sh, typename T>
__device__ __forceinline__ void ch_convert(const ChunkArgs &a, ChunkShared &sh, uint8_t *sq, uint8_t *k_slots, uint8_t *v_slots, uint8_t *raw,
                                           int tid) {
    constexpr int kEach = Sh::kEach, kThreads = kChConvertWarps * 32, kSlots = Sh::kSlots, G = Sh::kGranules, kWindow = 32 / G;
    const int warp = tid >> 5, lane = tid & 31, per = a.head_dim / 16, block = 1 << a.block_log2;
    int token[kEach];  // of the thread's groups, in a tile (T: none)
    uint32_t dst[kEach];
    auto group = [&](int i, int &t, int &c) {
        const ChunkGroup x = ch_group(tid + i * kThreads, Sh::T, per);
        t = x.token;
        c = x.part;
        return (c >> 2) * (Sh::T * 128) + t * 128 + (((2 * (c & 3)) ^ (t & 7)) << 4);
    };
    int from[kEach];   // ... their places in the block of a request's first tile
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        int c;
        dst[i] = group(i, token[i], c);
        from[i] = ch_group_from({token[i], c}, Sh::T, block, a.head_dim);
    }
    const uint8_t *mine = raw + tid * 16;  // the thread's groups of a raw slot lie 16 x threads apart
    const int64_t id_bytes = static_cast<int64_t>(a.kv_heads) * block * a.head_dim;
    const uint32_t n_blocks = static_cast<uint32_t>(a.n_blocks);
    int nt = 0, unit = 0;  // tiles so far; units with tiles
    bool ok = true;
    ChunkUnit w;
    for (int u = 0; ch_unit(sh, u, lane, w); ++u) {
        if (w.tiles == 0) continue;
        if (!ok) {  // (nobody is left behind at the set-up's barrier)
            asm volatile("bar.sync 4, %0;" ::"n"(kThreads) : "memory");
            continue;
        }
        const int ub = unit & 1, j1 = w.j0 + w.tiles;
        const int32_t *row = a.table + static_cast<int64_t>(w.s) * a.width;
        const int64_t head = static_cast<int64_t>(w.head) * block * a.head_dim;
        // Lane: tile lane / G of the window from tile j on, its sixteen tokens lane % G.  The block's id (maybe one outside the
        // pool), -1 where the table ends before it, -2 past the request's end.
        auto window = [&](int j) {
            const int64_t t = static_cast<int64_t>(j + lane / G) * Sh::T + 16 * (lane % G);
            const int64_t page = t >> a.block_log2;
            return j + lane / G >= j1 || t >= w.len ? -2 : page < a.width ? row[page] : -1;
        };
        // The scales of the block in hand.  One that is not finite, and one of a block outside the pool, counts as NaN.
        auto scales = [&](int b, float &k1, float &v1) {
            k1 = v1 = 1.f;
            if (b == -2) return;
            const bool there = static_cast<uint32_t>(b) < n_blocks;
            const int64_t bh = static_cast<int64_t>(b) * a.kv_heads + w.head;
            k1 = there ? a.k_scales[bh] : INFINITY;
            v1 = there ? a.v_scales[bh] : INFINITY;
            if (!there) atomicOr(a.status, 4u);
        };
        // Ids of the window from tile `ahead` on, which the copies have come to, and of the next; scales of the window from tile
        // `first` on (warp 0), and ids and scales of the next.
        int id = window(w.j0), id_next = window(w.j0 + kWindow), ahead = w.j0, first = w.j0, id_scales = id_next;
        float k0 = 1.f, v0 = 1.f, k1 = 1.f, v1 = 1.f;
        // Copies of slot n of the unit (K and V of its tiles in turn), into the raw slot n % kRaws.
        const uint8_t *k_head = a.k_codes + head, *v_head = a.v_codes + head;
        int n_copy = 0, j_copy = w.j0;
        uint32_t to_copy = smem_addr(mine);
        auto copy = [&]() {
            if (j_copy == ahead + kWindow) {
                ahead = j_copy;
                id = id_next;
                id_next = window(j_copy + kWindow);
            }
            const uint8_t *codes = (n_copy & 1 ? v_head : k_head) + ch_tile_from(j_copy, Sh::T, block, a.head_dim);
            const int left = ch_tile_left(w.len, j_copy, Sh::T);  // (past the unit's last tile the ids say so)
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int b = __shfl_sync(0xFFFFFFFFu, id, (j_copy - ahead) * G + (token[i] >> 4));
                const bool there = ch_group_copied(token[i], left, static_cast<uint32_t>(b), n_blocks);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to_copy + i * kThreads * 16),
                             "l"(codes + (there ? b : 0) * id_bytes + from[i]), "r"(there ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (Sh::kRaws == 1 && warp == 1 && (n_copy & 1) == 0) {
                // Into L2: the blocks of the tile four further on, a lane for each sixteen tokens.
                const int of = (j_copy + 4 - ahead) * G + lane % G;
                const int b0 = __shfl_sync(0xFFFFFFFFu, id, of & 31), b1 = __shfl_sync(0xFFFFFFFFu, id_next, of & 31), b = of < 32 ? b0 : b1;
                if (lane < G && (16 * lane & (block - 1)) == 0 && static_cast<uint32_t>(b) < n_blocks) {
                    bulk_prefetch_l2(k_head + b * id_bytes, static_cast<uint32_t>(block * a.head_dim));
                    bulk_prefetch_l2(v_head + b * id_bytes, static_cast<uint32_t>(block * a.head_dim));
                }
            }
            j_copy += n_copy & 1;
            ++n_copy;
            to_copy = n_copy % Sh::kRaws == 0 ? smem_addr(mine) : to_copy + Sh::kRaw;
        };
#pragma unroll 1
        for (int n = 0; n < Sh::kRaws; ++n) copy();
        if (warp == 0) {
            scales(id, k0, v0);
            scales(id_scales, k1, v1);
            id_scales = window(w.j0 + 2 * kWindow);
        }
        // The unit's queries, once the MMAs have read the last one's, and the softmax has written out the one before that.
        const ChunkQueries<Sh, T> queries(a, w, sq, sh.qs[ub], warp, lane);
        ok = (unit < 1 || ch_wait(a, sh, sh.q_free, static_cast<uint32_t>(unit - 1) & 1u)) &&
             (unit < 2 || (ch_wait(a, sh, sh.unit_done[ub], static_cast<uint32_t>((unit >> 1) - 1) & 1u) && ch_alive(sh)));
        if (ok) {
            queries.copy();
            sh.vnan[ub][tid] = kChNoNan;
            if (tid == 0) sh.any_nan[ub] = 0;
        }
        asm volatile("bar.sync 4, %0;" ::"n"(kThreads) : "memory");
        if (!ok) continue;
        asm volatile("cp.async.wait_all;" ::: "memory");
        queries.convert();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.q_full[ub]));
        // One raw slot, which has come, as f16 (the copies that take its place come behind the barrier's release).  The sum of V's values (at most 32 x 448)
        // is not finite where one is a NaN.
        auto convert = [&](int n, uint8_t *to, auto is_v) {
            asm volatile("cp.async.wait_group %0;" ::"n"(Sh::kRaws - 1) : "memory");
            const uint8_t *x = mine + (n % Sh::kRaws) * Sh::kRaw;
            __half2 sum = __half2(__ushort_as_half(0), __ushort_as_half(0));
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const uint4 c = *reinterpret_cast<const uint4 *>(x + i * kThreads * 16);
                const uint32_t y[4] = {c.x, c.y, c.z, c.w};
                uint32_t h[8];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                        : "=r"(h[2 * z]), "=r"(h[2 * z + 1])
                        : "r"(y[z]));
                if (token[i] < Sh::T) {
                    *reinterpret_cast<uint4 *>(to + dst[i]) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(to + (dst[i] ^ 16u)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                if (decltype(is_v)::value) {
#pragma unroll
                    for (int z = 0; z < 8; ++z) sum = __hadd2(sum, *reinterpret_cast<const __half2 *>(h + z));
                }
            }
            return sum;
        };
#pragma unroll 1
        for (int j = w.j0; j < j1; ++j, ++nt) {
            const int slot = nt % kSlots, n = 2 * (j - w.j0);  // (a slot of each ring, and K's place among the raw ones)
            const uint32_t free = (static_cast<uint32_t>(nt / kSlots) & 1u) ^ 1u;
            if (warp == 0 && j == first + kWindow) {
                first = j;
                k0 = k1;
                v0 = v1;
                scales(id_scales, k1, v1);
                id_scales = window(j + 2 * kWindow);
            }
            ok = nt < kSlots || ch_wait(a, sh, sh.k_free[slot], free);
            if (!ok) break;
            (void)convert(n, k_slots + slot * Sh::kSlot, std::false_type{});
            if (warp == 0) {
                const int at = nt & (kChInfo - 1);
                float4 f = make_float4(1.f, 0.f, 1.f, 0.f);
                const bool here = lane / G == j - first;
                if (here) {
                    f.x = fabsf(k0) < INFINITY ? k0 : __int_as_float(0x7FC00000);
                    float v = v0;
                    if (!(fabsf(v) < INFINITY)) {  // every element, from here on
                        sh.any_nan[ub] = 1;
#pragma unroll 1
                        for (int d = 0; d < a.head_dim; ++d) atomicMin(&sh.vnan[ub][d], j * Sh::T + 16 * (lane % G));
                        v = 1.f;
                    }
                    const bool small = fabsf(v) < 0x1p-126f;
                    const uint32_t bits = __float_as_uint(small ? v * 0x1p64f : v), e = bits >> 23 & 0xFFu;
                    f.y = v == 0.f ? -1000.f : static_cast<float>(static_cast<int>(e) - (small ? 191 : 127));
                    f.z = v == 0.f ? 1.f : __uint_as_float((bits & 0x807FFFFFu) | 0x3F800000u);
                    sh.info[at][lane % G] = f;
                }
                // (Tokens past the request's end take any scale.)
                const bool odd = __any_sync(0xFFFFFFFFu, here && (f.x < 0.f || f.z != 1.f));
                const float kf = __shfl_sync(0xFFFFFFFFu, f.x, lane & ~3), vf = __shfl_sync(0xFFFFFFFFu, f.y, lane & ~3);  // of the 64 tokens
                const bool same = __all_sync(0xFFFFFFFFu, !here || (f.x == kf && f.y == vf));
                __syncwarp();
                if (lane == 0) {
                    sh.info_kind[at] = odd ? 2 : same ? 0 : 1;
                    mbar_arrive(smem_addr(&sh.info_full[at]));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.k_full[slot]));
            copy();
            ok = nt < kSlots || ch_wait(a, sh, sh.v_free[slot], free);
            if (!ok) break;
            uint8_t *to = v_slots + slot * Sh::kSlot;
            const __half2 sum = convert(n + 1, to, std::true_type{});
            if (__hisnan(sum.x) || __hisnan(sum.y)) {  // seldom: zeros in their places, and from which position on each element has one
                sh.any_nan[ub] = 1;
#pragma unroll 1
                for (int i = 0; i < kEach; ++i) {
                    int t, c;
                    const uint32_t at = group(i, t, c);
                    if (t >= Sh::T) break;
#pragma unroll 1
                    for (int y = 0; y < 16; ++y) {
                        uint16_t *h = reinterpret_cast<uint16_t *>(to + (y < 8 ? at : at ^ 16u)) + (y & 7);
                        if ((*h & 0x7C00u) != 0x7C00u) continue;
                        *h = 0;
                        atomicMin(&sh.vnan[ub][16 * c + y], j * Sh::T + t);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.v_full[slot]));
            copy();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.values_done[ub]));
        ++unit;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ MMAs
// The MMAs of a product.  The warp goes through the tiles together.  Returns
// whether anything was issued.
template <typename Sh>
__device__ __forceinline__ bool ch_issue(const ChunkArgs &a, ChunkShared &sh, uint32_t tmem_base, uint32_t sq, uint32_t k_slots,
                                         uint32_t v_slots, int product, int lane) {
    constexpr int PL = Sh::PL, T = Sh::T, kSlots = Sh::kSlots;
    constexpr uint32_t qk_idesc = ch_idesc(T, false);
    // (Broadcasts, here and below: so the compiler knows these, and what is counted by them, to be one value a warp, and
    // descriptors and addresses are made by the uniform units.)
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
    const int i = Sh::NS == 1 ? 0 : __shfl_sync(0xFFFFFFFFu, product, 0);
    uint32_t q_desc = 0;
    const uint32_t k_desc = ch_desc(k_slots, 16), v_desc = ch_desc(v_slots, T * 128);
    const int steps = a.head_dim / 16;
    bool any = false, ok = true;
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        ok = ok && ch_wait(a, sh, bar, parity);
        t8_fence_after();
        return ok;
    };
    // The converters' stores, seen through their barriers, before the MMAs' reads.  (The fence is here and not behind the
    // stores: there it waited for the thread's loads of the tiles to come as well, 2000 cycles a tile.)
    auto stores_seen = [&]() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); };
    int nk = 0, nv = 0, unit = 0;  // tiles of K, of V that have gone by; units with tiles
    int ms = 0, mv = 0;            // tiles whose scores, whose sums have been issued
    int products = 0;              // products of the second kind (f32, wide: two a tile)
    // Scores of the next tile against K, the second plane's first.  end: q is read.
    auto scores = [&](bool end) {
        const int slot = nk % kSlots, buf = Sh::NS == 1 ? ms & 1 : i;
        if (!wait(sh.k_full[slot], static_cast<uint32_t>(nk / kSlots) & 1u)) return;
        stores_seen();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * T);
#pragma unroll 1
        for (int p = PL - 1; p >= 0; --p) {
            uint32_t q = q_desc + static_cast<uint32_t>(p) * (Sh::kQPlane / 16), k = k_desc + static_cast<uint32_t>(slot) * (Sh::kSlot / 16);
            bool acc = p + 1 < PL;
#pragma unroll 1
            for (int s = 0; s + 4 <= steps; s += 4) {  // 64 columns of a head
                ch_mma_ss(d, q, k, qk_idesc, acc);
                ch_mma_ss(d, q + 2, k + 2, qk_idesc, true);
                ch_mma_ss(d, q + 4, k + 4, qk_idesc, true);
                ch_mma_ss(d, q + 6, k + 6, qk_idesc, true);
                acc = true;
                q += 128 * 128 / 16;
                k += T * 128 / 16;
            }
#pragma unroll 1
            for (int s = steps & ~3; s < steps; ++s) {
                ch_mma_ss(d, q, k, qk_idesc, acc);
                acc = true;
                q += 2;
                k += 2;
            }
        }
        ch_commit(sh.s_full[buf]);
        ch_commit(sh.k_free[slot]);
        if (end) ch_commit(sh.q_free);
        ++nk;
        ++ms;
        any = true;
    };
    // The next tile's weights times V.  They lie where its scores were and other scores will be: only MMAs of one shape are
    // sure to run in the order of their issue.  So with two products the sums have 128 columns as the scores do (whatever
    // lies past head_dim), and with one, whose next scores go elsewhere, the end of these is waited for.
    auto sums = [&](bool acc) {
        const int slot = nv % kSlots, buf = Sh::NS == 1 ? mv & 1 : i;
        const uint32_t ph = static_cast<uint32_t>(Sh::NS == 1 ? mv >> 1 : mv) & 1u;
        if (!wait(sh.v_full[slot], static_cast<uint32_t>(nv / kSlots) & 1u)) return;
        if (!(Sh::NS == 2 ? wait(sh.p_half[buf], ph) : wait(sh.p_full[buf], ph))) return;
        stores_seen();
        const uint32_t p0 = tmem + static_cast<uint32_t>(buf * T);
        uint32_t v = v_desc + static_cast<uint32_t>(slot) * (Sh::kSlot / 16), p = p0;
        if constexpr (Sh::NS == 2) {
            const uint32_t d = tmem + static_cast<uint32_t>(Sh::kSumCol + i * 128);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && !wait(sh.p_full[buf], ph)) return;
                ch_mma_ts(d, p, v, ch_idesc(128, true), acc || h > 0);
                ch_mma_ts(d, p + 8, v + 16 * 128 / 16, ch_idesc(128, true), true);
                ch_mma_ts(d, p + 16, v + 32 * 128 / 16, ch_idesc(128, true), true);
                ch_mma_ts(d, p + 24, v + 48 * 128 / 16, ch_idesc(128, true), true);
                p += 32;
                v += 64 * 128 / 16;
            }
            ch_commit(sh.o_done[i]);
            ch_commit(sh.v_free[slot]);
        } else {
#pragma unroll 1
            for (int h = 0; h < Sh::kHalves; ++h) {
                if (Sh::SUMS && products > 0 && !wait(sh.product_free, static_cast<uint32_t>(products - 1) & 1u)) return;
                const uint32_t d = tmem + static_cast<uint32_t>(Sh::SUMS ? Sh::kProductCol : Sh::kSumCol);
                const uint32_t idesc = ch_idesc(Sh::kHalves == 1 ? a.head_dim : h == 0 ? 128 : a.head_dim - 128, true);
#pragma unroll 1
                for (int x = PL - 1; x >= 0; --x) {  // the second plane's first
                    constexpr uint32_t kStep = PL == 1 ? 16 : 32;  // columns of 32 tokens' weights; with two planes the second's follow the first's
                    const uint32_t at = p + 16 * x;
                    ch_mma_ts(d, at, v, idesc, (!Sh::SUMS && acc) || x + 1 < PL);
                    ch_mma_ts(d, at + 8, v + 16 * 128 / 16, idesc, true);
                    ch_mma_ts(d, at + kStep, v + 32 * 128 / 16, idesc, true);
                    ch_mma_ts(d, at + kStep + 8, v + 48 * 128 / 16, idesc, true);
                }
                v += 2 * T * 128 / 16;
                ch_commit(sh.o_done[0]);
                if (h + 1 == Sh::kHalves) ch_commit(sh.v_free[slot]);
                if (!wait(sh.o_done[0], static_cast<uint32_t>(products++) & 1u)) return;
            }
        }
        ++nv;
        ++mv;
    };
    ChunkUnit w;
    for (int u = 0; ch_unit(sh, u, lane, w); ++u) {
        const int two = __shfl_sync(0xFFFFFFFFu, w.flags & kChTwo, 0), tiles = __shfl_sync(0xFFFFFFFFu, w.tiles, 0);
        if (tiles == 0 || !ok) continue;
        if (a.wait_limit_ns < kWaitLimitNs)
            ok = ch_wait_brief(smem_addr(&sh.q_full[unit & 1]), static_cast<uint32_t>(unit >> 1) & 1u, a.wait_limit_ns, &sh.abort);
        if (!wait(sh.q_full[unit & 1], static_cast<uint32_t>(unit >> 1) & 1u)) continue;
        if (Sh::NS == 2 && !two) {
            // Every other tile; the slots of the others are given back once they have been filled.
            q_desc = ch_desc(sq, 16);
            auto skip = [&]() {
                if (!wait(sh.k_full[nk % kSlots], static_cast<uint32_t>(nk / kSlots) & 1u)) return;
                if (lane == 0) mbar_arrive(smem_addr(&sh.k_free[nk % kSlots]));
                ++nk;
                if (!wait(sh.v_full[nv % kSlots], static_cast<uint32_t>(nv / kSlots) & 1u)) return;
                if (lane == 0) mbar_arrive(smem_addr(&sh.v_free[nv % kSlots]));
                ++nv;
            };
            if (i == 1) {
                skip();
                if (tiles == 1 && lane == 0) mbar_arrive(smem_addr(&sh.q_free));
            }
            if (ok && i < tiles) scores(i + 2 >= tiles);
#pragma unroll 1
            for (int j = i; ok && j < tiles; j += 2) {
                sums(j >= 2);
                if (ok && j + 1 < tiles) skip();
                if (ok && j + 2 < tiles) scores(j + 4 >= tiles);
            }
            ++unit;
            continue;
        }
        q_desc = ch_desc(sq + i * PL * Sh::kQPlane, 16);
#pragma unroll 1
        for (int j = -Sh::kDeep; ok && j < tiles; ++j) {
            if (j >= 0) sums(j > 0);
            if (ok && j + Sh::kDeep < tiles) scores(j + Sh::kDeep + 1 == tiles);
        }
        ++unit;
    }
    return any;
}

// ------------------------------------------------------------------ softmax
// What a product has of a row: the sums' columns, their maximum, reference and
// denominator.
struct ChunkSums {
    uint32_t col;
    float M, R, l;
    // The sums are 2^-up times what they stand for, relative to 2^top: that, in two factors, since it may leave the range
    // of one.
    __device__ __forceinline__ void factors(float top, float &u1, float &u2) const {
        const float up = R > kChNone ? R - static_cast<float>(kChLift) + (M - top) : 0.f, up1 = fminf(fmaxf(up, -120.f), 120.f);
        u1 = at_exp2(up1);
        u2 = at_exp2(fminf(fmaxf(up - up1, -120.f), 120.f));
    }
};

// Writes a unit's row out: its outputs, or its part of them; of both products'
// sums if `both`.
template <typename Sh, typename T>
__device__ __forceinline__ void ch_finish(const ChunkArgs &a, const ChunkUnit &w, ChunkShared &sh, int unit, const ChunkRow &row, int local,
                                          const ChunkSums &x, const ChunkSums &y, bool both, bool ok) {
    const float nanf = __int_as_float(0x7FC00000);
    const int ub = unit & 1;
    // The converters' word on what is NaN.
    ok = ok && ch_wait(a, sh, sh.values_done[ub], static_cast<uint32_t>(unit >> 1) & 1u) && ch_alive(sh);
    const bool starts = w.flags & kChStarts, whole = starts && (w.flags & kChEnds);
    const float M = both ? fmaxf(x.M, y.M) : x.M;
    float l = both ? x.l * at_exp2(x.M - M) + y.l * at_exp2(y.M - M) : x.l, f = 1.f;
    if (!ok) l = nanf;
    if (whole) {
        f = l == 0.f ? 0.f : 1.f / l;
        if (row.valid && a.lse) a.lse[row.lse] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
    }
    float *part = a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + starts) * (static_cast<int64_t>(Sh::U) * (a.head_dim + 2));
    if (!whole) {
        __stcg(part + static_cast<int64_t>(Sh::U) * a.head_dim + local, M);
        __stcg(part + static_cast<int64_t>(Sh::U) * (a.head_dim + 1) + local, l);
    }
    T *out = static_cast<T *>(a.out) + row.out;
    const bool nans = ok && sh.any_nan[ub] != 0;
    float u1, u2, t1, t2;
    x.factors(M, u1, u2);
    y.factors(M, t1, t2);
    u2 *= ok ? f : nanf;
    t2 *= f;
    part += local;  // (column by column: the warp's rows lie together)
#pragma unroll 1
    for (int c = 0; c < a.head_dim; c += 16) {
        float v[16];
        t8_ld16(x.col + c, v);
        at_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] * u1 * u2;
        if (both) {
            float z[16];
            t8_ld16(y.col + c, z);
            at_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fmaf(z[i] * t1, t2, v[i]);
        }
        if (nans) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = sh.vnan[ub][c + i] <= row.last ? nanf : v[i];
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i) __stcg(part + static_cast<int64_t>(c + i) * Sh::U, v[i]);
        } else if (row.valid) {
            float lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) lo[i] = v[i], hi[i] = v[8 + i];
            rope_store8(out + c, lo);
            rope_store8(out + c + 8, hi);
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

// The weights of N columns, from their scores, as f16 words (PL = 2: and what those
// leave); their sum is the answer.
// CAREFUL: columns past `rel` are not seen, the value scale has a mantissa (or a
// sign), and product and difference round one
// by one, as the maxima did, so that no weight is above its reference (past 2^20
// the rounding of a score shows beside that).
template <int PL, bool CAREFUL, int N>
__device__ __forceinline__ float ch_weights(const float *v, int col, int rel, float k, float base, float log, float mantissa, uint32_t *hi,
                                            uint32_t *lo) {
    const uint64_t k2 = ch_pair(k, k), off2 = ch_pair(log - base, log - base);
    uint64_t sum[2] = {0, 0};
    float w[N];
#pragma unroll
    for (int x = 0; x < N; x += 2) {
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
        sum[(x >> 1) & 1] = ch_add2(sum[(x >> 1) & 1], ch_pair(w[x], w[x + 1]));
    }
    if (CAREFUL) {
#pragma unroll
        for (int x = 0; x < N; ++x) w[x] *= mantissa;
    }
#pragma unroll
    for (int x = 0; x < N / 2; ++x) {
        hi[x] = ch_pack_f16(w[2 * x], w[2 * x + 1]);
        if (PL == 2) {
            const float2 b = ch_unpack_f16(hi[x]);
            lo[x] = ch_pack_f16(w[2 * x] - b.x, w[2 * x + 1] - b.y);
        }
    }
    float s0, s1;
    ch_unpair(ch_add2(sum[0], sum[1]), s0, s1);
    return s0 + s1;
}

// The scores of a tile in turn, 32 columns at a time.  LOOP: what is seldom needed
// stays a loop, for the sake of the instruction caches (with every pass unrolled
// and every role's walk its own, all roles ran three times slower).
template <int T, bool LOOP, typename F>
__device__ __forceinline__ void ch_columns(uint32_t s_col, F f) {
    if constexpr (LOOP) {
#pragma unroll 1
        for (int c = 0; c < T; c += 32) {
            float v[32];
            ch_ld32(s_col + c, v);
            at_wait_ld();
            f(c, v);
        }
    } else {
#pragma unroll
        for (int c = 0; c < T; c += 32) {
            float v[32];
            ch_ld32(s_col + c, v);
            at_wait_ld();
            f(c, v);
        }
    }
}

template <typename Sh, typename T>
__device__ __forceinline__ void ch_softmax(const ChunkArgs &a, ChunkShared &sh, uint32_t tmem, int product, int wq, int lane) {
    constexpr int PL = Sh::PL, kTile = Sh::T;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t o_col = tmem + lanes + static_cast<uint32_t>(Sh::kSumCol + product * 128);
    int it = 0, unit = 0;   // all tiles of the CTA; units with tiles
    int mine = 0;           // tiles of this product (the buffers of a product go by its own count)
    int shared = 0, shared0 = 0, shared1 = 0;  // units shared with the other product: all, and by parity
    bool ok = true;
    ChunkUnit w;
    for (int u = 0; ch_unit(sh, u, lane, w); ++u) {
        const bool alone = Sh::NS == 1 || (w.flags & kChTwo) != 0;  // else the products share the rows and take every other tile
        const int local = (alone ? product * 128 : 0) + wq * 32 + lane, step = alone ? 1 : 2;
        const ChunkRow row(a, w, local);
        const int ub = unit & 1, tiles = w.tiles;
        if (tiles == 0) {
            if (!Sh::SUMS && (alone || product == 0)) ch_nothing<T>(a, row);
            continue;
        }
        ok = ok && ch_wait(a, sh, sh.q_full[ub], static_cast<uint32_t>(unit >> 1) & 1u);
        const float qs = sh.qs[ub][local];
        float M = kChNone, R = kChNone, l = 0.f;  // maximum, the weights' reference less M, denominator
        const int j_first = alone ? 0 : product;
        for (int j = j_first; ok && j < tiles; j += step, ++mine) {
            const int at = (it + j) & (kChInfo - 1), buf = Sh::NS == 1 ? mine & 1 : product;
            const uint32_t ph = static_cast<uint32_t>(Sh::NS == 1 ? mine >> 1 : mine) & 1u;
            const uint32_t s_col = tmem + lanes + static_cast<uint32_t>(buf * kTile);
            ok = ch_wait(a, sh, sh.info_full[at], static_cast<uint32_t>((it + j) / kChInfo) & 1u);
            const float4 *info = sh.info[at];
            const int64_t t0 = static_cast<int64_t>(w.j0 + j) * kTile;
            const int rel = t0 > row.last ? -1 : static_cast<int>(row.last - t0 < kTile ? row.last - t0 : kTile);  // last column this row sees
            // Careful: tiles that are not seen whole, odd scales, and scores past 2^19, where the rounding of a score shows
            // beside its row's reference.  (A unit's first tile has no maximum yet: it is not careful for that, its maxima are
            // rounded the same either way, and its weights go by `base` below.)
            const int kind = ok ? sh.info_kind[at] : 0;
            const bool careful = __any_sync(0xFFFFFFFFu, rel < kTile - 1 || (M > kChNone && fabsf(M) >= 0x1p19f)) || kind == 2;
            ok = ok && ch_wait(a, sh, sh.s_full[buf], ph);
            if (!ok) break;
            t8_fence_after();
            // The row's maximum, and the largest of the sixteens' maxima times their value scales, relative to the former.
            // Both as whole powers of two.
            float top = M, ref = kChNone;
            if (!careful) {
                float m16[kTile / 16];
                ch_columns<kTile, false>(s_col, [&](int c, float (&v)[32]) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) m16[c / 16 + g] = ch_max16(v + 16 * g);
                });
                if (kind == 0) {
                    float m[kTile / 64];
#pragma unroll
                    for (int h = 0; h < kTile / 64; ++h) {
                        m[h] = ceilf(fmaxf(ch_max3(m16[4 * h], m16[4 * h + 1], m16[4 * h + 2]), m16[4 * h + 3]) * (info[4 * h].x * qs));
                        top = fmaxf(top, m[h]);
                    }
#pragma unroll
                    for (int h = 0; h < kTile / 64; ++h) ref = fmaxf(ref, (m[h] - top) + info[4 * h].y);
                } else {
#pragma unroll
                    for (int g = 0; g < kTile / 16; ++g) {
                        m16[g] = ceilf(m16[g] * (info[g].x * qs));
                        top = fmaxf(top, m16[g]);
                    }
#pragma unroll
                    for (int g = 0; g < kTile / 16; ++g) ref = fmaxf(ref, (m16[g] - top) + info[g].y);
                }
            } else {
                ch_columns<kTile, true>(s_col, [&](int c, float (&v)[32]) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 f = info[c / 16 + g];
                        const float k = f.x * qs;
                        float m = -INFINITY;
#pragma unroll
                        for (int x = 0; x < 16; ++x) m = c + 16 * g + x <= rel ? fmaxf(m, v[16 * g + x] * k) : m;
                        m = m == -INFINITY ? m : ceilf(m);
                        const float now = fmaxf(top, m);
                        ref = fmaxf(now > top && ref > kChNone ? ref - (now - top) : ref, (m - now) + f.y);
                        top = now;
                    }
                });
            }
            if (top > M) {
                l *= at_exp2(M - top);
                R = R > kChNone ? R - (top - M) : R;
                M = top;
            }
            const bool move = ref > R + kChSlack;
            const float factor = move && R > kChNone ? at_exp2(R - ref) : 1.f;  // of the sums so far
            if (Sh::SUMS) {
                sh.factor[at][local] = factor;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.factor_full[at]));
            } else if (j > j_first && __any_sync(0xFFFFFFFFu, move)) {
                ok = ch_wait(a, sh, sh.o_done[product], static_cast<uint32_t>(mine - 1) & 1u);
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
            auto put = [&](int c, const uint32_t (&hi)[16], const uint32_t (&lo)[16]) {
                if (PL == 1) {
                    ch_st16(s_col + c / 2, hi);
                } else {
                    ch_st16(s_col + c, hi);
                    ch_st16(s_col + c + 16, lo);
                }
                if (Sh::NS == 2 && c == 32) {  // the first half is there
                    ch_wait_st();
                    t8_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sh.p_half[buf]));
                }
            };
            auto by_sixteens = [&](auto slow) {
                constexpr bool kSlow = decltype(slow)::value;
                ch_columns<kTile, true>(s_col, [&](int c, float (&v)[32]) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 f = info[c / 16 + g];
                        const float log = fmaxf(f.y + lift, kChMinLog);
                        l = fmaf(ch_weights<PL, kSlow, 16>(v + 16 * g, c + 16 * g, rel, f.x * qs, base, log, f.z, hi + 8 * g, lo + 8 * g),
                                 at_exp2(-log), l);
                    }
                    put(c, hi, lo);
                });
            };
            if (careful || __any_sync(0xFFFFFFFFu, fabsf(base) >= 0x1p20f)) {
                by_sixteens(std::true_type{});
            } else if (kind == 1) {
                by_sixteens(std::false_type{});
            } else {
                ch_columns<kTile, false>(s_col, [&](int c, float (&v)[32]) {
                    uint32_t hi[16], lo[16];
                    const float4 f = info[c / 64 * 4];
                    const float log = fmaxf(f.y + lift, kChMinLog);
                    l = fmaf(ch_weights<PL, false, 32>(v, c, rel, f.x * qs, base, log, 1.f, hi, lo), at_exp2(-log), l);
                    put(c, hi, lo);
                });
            }
            ch_wait_st();
            // The sums of the tile before may still be under way: each phase is waited for, so that the last one cannot be
            // taken for the one before it.
            if (Sh::NS == 1 && !Sh::SUMS && j > 0) {
                ok = ch_wait(a, sh, sh.o_done[product], static_cast<uint32_t>(mine - 1) & 1u);
                if (!ok) break;
            }
            t8_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[buf]));
        }
        it += tiles;
        if (!Sh::SUMS && j_first < tiles) ok = ok && ch_wait(a, sh, sh.o_done[product], static_cast<uint32_t>(mine - 1) & 1u);
        t8_fence_after();
        ChunkSums x = {o_col, M, R, ok ? l : __int_as_float(0x7FC00000)}, y = x;
        if (Sh::SUMS || (!alone && product == 1)) {
            const int r = wq * 32 + lane;
            sh.last[ub][0][r] = x.M;
            sh.last[ub][1][r] = x.R;
            sh.last[ub][2][r] = x.l;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.last_full[ub]));
            // The sums stay as they are until the first product has taken them.
            if (!Sh::SUMS) ok = ok && ch_wait(a, sh, sh.merged, static_cast<uint32_t>(shared) & 1u) && ch_alive(sh);
        } else {
            if (!alone) {
                ok = ok && ch_wait(a, sh, sh.last_full[ub], static_cast<uint32_t>((ub == 0 ? shared0 : shared1)) & 1u);
                y = {o_col + 128, sh.last[ub][0][wq * 32 + lane], sh.last[ub][1][wq * 32 + lane], sh.last[ub][2][wq * 32 + lane]};
            }
            ch_finish<Sh, T>(a, w, sh, unit, row, local, x, y, !alone && tiles > 1, ok);
            t8_fence_before();
            __syncwarp();
            if (!alone && lane == 0) mbar_arrive(smem_addr(&sh.merged));
        }
        if (!alone) {
            ++shared;
            if (ub == 0) ++shared0;
            else ++shared1;
        }
        __syncwarp();
        if (!Sh::SUMS && lane == 0) mbar_arrive(smem_addr(&sh.unit_done[ub]));
        ++unit;
    }
}

// f32's sums: each tile's product, out of tensor memory, onto the sums there,
// rounded; at a unit's end its rows are written out.
template <typename Sh, typename T>
__device__ __forceinline__ void ch_sums(const ChunkArgs &a, ChunkShared &sh, uint32_t tmem, int wq, int lane) {
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t p_col = tmem + lanes + static_cast<uint32_t>(Sh::kProductCol), o_col = tmem + lanes + static_cast<uint32_t>(Sh::kSumCol);
    const int local = wq * 32 + lane;
    int it = 0, unit = 0, products = 0;
    bool ok = true;
    ChunkUnit w;
    for (int u = 0; ch_unit(sh, u, lane, w); ++u) {
        const ChunkRow row(a, w, local);
        const int ub = unit & 1, tiles = w.tiles;
        if (tiles == 0) {
            ch_nothing<T>(a, row);
            continue;
        }
        for (int j = 0; ok && j < tiles; ++j, ++it) {
            ok = ch_wait(a, sh, sh.factor_full[it & (kChInfo - 1)], static_cast<uint32_t>(it / kChInfo) & 1u);
            const float factor = sh.factor[it & (kChInfo - 1)][local];
#pragma unroll 1
            for (int h = 0; ok && h < Sh::kHalves; ++h, ++products) {
                ok = ch_wait(a, sh, sh.o_done[0], static_cast<uint32_t>(products) & 1u);
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
                ch_wait_st();  // (the next tile loads them: nothing else orders a load behind a store)
                t8_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sh.product_free));
            }
        }
        ok = ok && ch_wait(a, sh, sh.last_full[ub], static_cast<uint32_t>(unit >> 1) & 1u);
        const ChunkSums x = {o_col, sh.last[ub][0][local], sh.last[ub][1][local], sh.last[ub][2][local]};
        ch_finish<Sh, T>(a, w, sh, unit, row, local, x, x, false, ok);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.unit_done[ub]));
        ++unit;
    }
}

// ------------------------------------------------------------------ the kernel
template <typename T, int PL, bool WIDE>
__global__ void __launch_bounds__(kChThreads, 1) kv_chunk_kernel(const ChunkArgs a) {
    using Sh = ChunkShape<PL, WIDE>;
    extern __shared__ __align__(1024) uint8_t ch_smem[];
    __shared__ __align__(16) ChunkShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *sq = ch_smem + ((1024u - (smem_addr(ch_smem) & 1023u)) & 1023u);
    uint8_t *k_slots = sq + Sh::kQ, *v_slots = k_slots + Sh::kSlots * Sh::kSlot, *raw = v_slots + Sh::kSlots * Sh::kSlot;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&sh.k_full[i]), kChConvertWarps);
            mbar_init(smem_addr(&sh.k_free[i]), Sh::kIssuers);
            mbar_init(smem_addr(&sh.v_full[i]), kChConvertWarps);
            mbar_init(smem_addr(&sh.v_free[i]), Sh::kIssuers);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&sh.s_full[i]), 1);
            mbar_init(smem_addr(&sh.p_half[i]), 4);
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
        mbar_init(smem_addr(&sh.merged), 4);
        for (int i = 0; i < kChUnits; ++i) {
            mbar_init(smem_addr(&sh.unit_full[i]), 1);
            mbar_init(smem_addr(&sh.unit_free[i]), (Sh::NS == 2 || Sh::SUMS ? 8 : 4) + kChConvertWarps + Sh::kIssuers);  // every warp that takes units
        }
        mbar_init(smem_addr(&sh.q_free), Sh::kIssuers);
        mbar_init(smem_addr(&sh.mma_done[0]), 1);
        mbar_init(smem_addr(&sh.mma_done[1]), 1);
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
    bool busy;
    {
        const ChunkList<Sh> list{a};
        const int each = (a.n_seqs + kChThreads - 1) / kChThreads;
        const int r0 = min(tid * each, a.n_seqs), r1 = min(r0 + each, a.n_seqs);
        int sum = 0;
        int64_t rows = 0;
        bool bad = false;
#pragma unroll 1
        for (int s = r0; s < r1; ++s) {
            const ChunkSeq q = list.seq(s);
            sum += list.entries(q);
            rows += q.rows;
            bad |= q.bad;
        }
        // More rows than there are (starts that go back): nothing is done, and no sum below has passed 32 bits otherwise.
        auto add_up = [](uint32_t x) {
            return static_cast<int64_t>(__reduce_add_sync(0xFFFFFFFFu, x & 0xFFFFu)) + (static_cast<int64_t>(__reduce_add_sync(0xFFFFFFFFu, x >> 16)) << 16);
        };
        rows = add_up(static_cast<uint32_t>(min(rows, static_cast<int64_t>(0x7FFFFFFF))));
        if (bad && blockIdx.x == 0) atomicOr(a.status, 4u);
        int pre = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, pre, d);
            if (lane >= d) pre += u;
        }
        if (lane == 31) {
            sh.scan[warp] = pre;
            sh.scan_rows[warp] = static_cast<uint32_t>(min(rows, static_cast<int64_t>(0x7FFFFFFF)));
        }
        __syncthreads();
        const bool over = add_up(lane < kChThreads / 32 ? sh.scan_rows[lane] : 0) > a.total_rows;
        if (over && tid == 0) atomicOr(a.status, 4u);
        const int part = sh.scan[min(lane, kChThreads / 32 - 1)];  // each warp's sum, in the lanes of its number
        const int total = __reduce_add_sync(0xFFFFFFFFu, lane < kChThreads / 32 ? part : 0);
        const int from = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? part : 0) + pre - sum;
        // Every CTA's share is a few entries, so no two cuts inside a unit meet.
        const int grid = min(static_cast<int>(gridDim.x), max(total / 8, min(total, 1)));
        busy = static_cast<int>(blockIdx.x) < grid && !over;
        const ChunkSplit split(total, max(grid, 1));
        if (busy) {  // the requests that the two cuts lie in
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                const int x = split.begin(blockIdx.x + e);
                if (from > x || x >= from + sum) continue;
                int here = from, s = r0;
#pragma unroll 1
                for (int n = each == 1 ? sum : list.entries(list.seq(s)); x >= here + n; n = list.entries(list.seq(s))) {
                    here += n;
                    ++s;
                }
                sh.at[e][0] = s;
                sh.at[e][1] = here;
            }
        }
        __syncthreads();
        if (busy && warp < 2) {  // warp e: cut e
            const int x = split.begin(blockIdx.x + warp);
            if (x == total) {
                if (lane == 0) sh.cut[warp] = total;
            } else {
                const int s = sh.at[warp][0];
                const ChunkSeq q = list.seq(s);
                int here = sh.at[warp][1], lo = 0;  // the row tile: the last one whose entries begin at or below x
#pragma unroll 1
                for (int n = q.row_tiles; n > 1;) {
                    const int step = (n + 31) / 32, i = lane * step;
                    const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, i < n && list.before(q, lo + min(i, n - 1)) <= x - here));
                    lo += k * step;
                    n = min(step, n - k * step);
                }
                here += list.before(q, lo);
                const int weight = list.weight(q, lo), slots = list.seen(q, lo) + kChSetUp;
                const int head = (x - here) / (weight * slots);
                int slot = ((x - here) - head * weight * slots) / weight;
                if (slot < kChSetUp + kChSmallCut) slot = 0;
                if (lane == 0) {
                    sh.cut[warp] = here + (head * slots + slot) * weight;
                    if (warp == 0) {
                        sh.seq = q;
                        sh.at[0][1] = lo;
                        sh.at[0][2] = head;
                        sh.at[0][3] = slot;
                    }
                }
            }
        }
        __syncthreads();
        busy = busy && sh.cut[0] < sh.cut[1];
    }
    if (busy) {
        if (warp < kChConvertWarp) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChSoftmaxRegs));
            if (warp < 4 * Sh::NS) ch_softmax<Sh, T>(a, sh, tmem, warp >> 2, warp & 3, lane);
            else if (Sh::SUMS) ch_sums<Sh, T>(a, sh, tmem, warp & 3, lane);
        } else if (warp < kChMmaWarp) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kChConvertRegs));
            ch_convert<Sh, T>(a, sh, sq, k_slots, v_slots, raw, tid - kChConvertWarp * 32);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kChIssueRegs));
            if (warp < kChMmaWarp + Sh::kIssuers) {
                // Also after a wait that ran out: nothing is in flight at the end.
                const int i = warp - kChMmaWarp;
                if (ch_issue<Sh>(a, sh, tmem, smem_addr(sq), smem_addr(k_slots), smem_addr(v_slots), i, lane)) {
                    ch_commit(sh.mma_done[i]);
                    (void)mbar_wait_bounded(smem_addr(&sh.mma_done[i]), 0);
                }
            } else if (warp == kChPlanWarp && lane == 0) {
                ch_plan<Sh, T>(a, sh);
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

// Joins the parts of units that lie across CTAs.  CTAs (x, ..): the unit that CTA x of
// the first kernel began and did not end (if there is one), in turns of 32 rows and
// 64 columns; its parts lie with x, x + 1, .. as far as their ranges go on.  The
// warps weigh the rows' parts; then a warp adds up eight columns', a lane two of
// four rows, in the parts' order.  Bound by the way of its loads: few rows in many
// parts are few warps, so four parts are under way at a time, the first four while
// the parts are weighed (16 rows in 19 parts: 86 us a call without that, 84 with eight
// parts, 83 with four or two; with eight, whose registers leave two CTAs an SM, 512
// rows of 8192 tokens 185 for 179).
template <typename T, int U>
__global__ void __launch_bounds__(256) kv_chunk_join_kernel(const ChunkArgs a, int grid) {
    __shared__ __align__(16) float weights[kChMaxGrid][32], sums[kChMaxGrid][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    const int4 h = a.heads[2 * b], rows = a.heads[2 * b + 1];
    int middle_of = a.heads[2 * min(b + 1 + lane, grid - 1)].w;  // (asked for at once)
    if ((h.w & 1) == 0) return;
    int parts = 2;  // x + 1, and on as long as a CTA's whole range is the unit's middle
    for (bool on = true; on;) {
        const int x = b + parts - 1 + lane;
        if (parts > 2) middle_of = a.heads[2 * min(x, grid - 1)].w;
        const unsigned middle = __ballot_sync(0xFFFFFFFFu, x < grid - 1 && (middle_of & 2) != 0);
        on = middle == 0xFFFFFFFFu;
        parts += on ? 32 : __ffs(~middle) - 1;
    }
    const int64_t size = static_cast<int64_t>(U) * (a.head_dim + 2), at_m = static_cast<int64_t>(U) * a.head_dim;
    const int flat = rows.y * a.group - h.y * U, row_turns = (min(flat, U) + 31) / 32, turns = row_turns * ((a.head_dim + 63) / 64);
#pragma unroll 1
    for (int turn = blockIdx.y; turn < turns; turn += kChJoinCtas) {
        const int row0 = turn % row_turns * 32, r = h.y * U + row0;
        auto part = [&](int p) { return a.partials + (static_cast<int64_t>(b + p) * 2 + (p == 0)) * size + row0; };
        const int c = turn / row_turns * 64 + warp * 8 + 2 * (lane >> 3), q = 4 * (lane & 7);
        const bool has = c < a.head_dim;
        float4 x[4][2];
        auto load = [&](int p0) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const float *at = part(min(p0 + p, parts - 1)) + static_cast<int64_t>(has ? c : 0) * U + q;
                x[p][0] = *reinterpret_cast<const float4 *>(at);
                x[p][1] = *reinterpret_cast<const float4 *>(at + U);
            }
        };
        load(0);  // (on their way while the parts are weighed)
        __syncthreads();  // (the turn before is done with the weights)
        for (int p = warp; p < parts; p += 8) {
            weights[p][lane] = part(p)[at_m + lane];
            sums[p][lane] = part(p)[at_m + U + lane];
        }
        __syncthreads();
        float M = kChNone, l = 0.f;
#pragma unroll 8
        for (int p = 0; p < parts; ++p) M = fmaxf(M, weights[p][lane]);
#pragma unroll 8
        for (int p = 0; p < parts; ++p) l = fmaf(sums[p][lane], at_exp2(weights[p][lane] - M), l);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __syncthreads();
        for (int p = warp; p < parts; p += 8) weights[p][lane] = at_exp2(weights[p][lane] - M) * inv;
        if (turn < row_turns && warp == 0 && a.lse && r + lane < rows.y * a.group) {
            int in_group;
            const int token = ch_token(a, r + lane, in_group);
            a.lse[(static_cast<int64_t>(rows.x) + token) * (static_cast<int64_t>(a.kv_heads) * a.group) + static_cast<int64_t>(h.z) * a.group + in_group] =
                l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
        }
        __syncthreads();
        float o[2][4] = {};
        for (int p0 = has ? 0 : parts; p0 < parts; p0 += 4) {
            if (p0 > 0) load(p0);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if (p0 + p >= parts) break;
                const float4 f = *reinterpret_cast<const float4 *>(&weights[p0 + p][q]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    o[i][0] = fmaf(x[p][i].x, f.x, o[i][0]);
                    o[i][1] = fmaf(x[p][i].y, f.y, o[i][1]);
                    o[i][2] = fmaf(x[p][i].z, f.z, o[i][2]);
                    o[i][3] = fmaf(x[p][i].w, f.w, o[i][3]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!has || r + q + i >= rows.y * a.group) break;
            int in_group;
            const int token = ch_token(a, r + q + i, in_group);
            T *out = static_cast<T *>(a.out) + (static_cast<int64_t>(rows.x) + token) * a.out_stride +
                     (static_cast<int64_t>(h.z) * a.group + in_group) * a.head_dim + c;
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float2 *>(out) = make_float2(o[0][i], o[1][i]);
            else *reinterpret_cast<__nv_bfloat162 *>(out) = __floats2bfloat162_rn(o[0][i], o[1][i]);
        }
    }
}

}  // namespace fp8blk
