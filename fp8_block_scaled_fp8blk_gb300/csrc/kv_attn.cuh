// kv_attn.cuh -- attention of 1..8 new rows per request over the paged e4m3
// cache, on the fifth-generation tensor cores, with the cached codes fed to
// the MMAs exactly as stored.
//
// For one request and cache head, with R query rows (row r = query head x new
// position) against a tile of 128 tokens:
//   S[t][r] = sum_d k[t][d] q[r][d]            (first MMA,  M = 128 tokens)
//   p[t][r] = 2^(S[t][r] s_k(t) c_r - m_r)     (c_r: softmax scale in base 2, m_r: the tile's maximum)
//   O[d][r] = sum_t v[t][d] p[t][r] s_v(t)     (second MMA, M = 128 of head_dim)
// K's tile is the first MMA's A operand as TMA lands it (K-major, 128-byte
// swizzle), V's tile the second's (the same landing, read M-major), so the
// CUDA cores never touch a code.  q and p s_v are the B operands: each value
// is carried as PL e4m3 planes, each the rounding of what the one before leaves
// (all subtractions exact).  Planes of one weight add up in the same columns of
// tensor memory (an MMA each), planes of another weight lie beside them.
//   f32 queries and outputs: four planes of weight 1, 1, 2^-8, 2^-8; a value keeps
//     2^-16 of itself (rms 5e-7) and 2^-24 of its row's largest, which leaves the
//     result at the error of an f32 computation.
//   bf16: two planes of weight 1, 2^-4; a value keeps 2^-8 of itself and 2^-20 of
//     its row's largest.  bf16's 8 bits fit two planes, so q loses only the
//     2^-21 of its row's largest; p's 2^-8 (rms 5e-4) is a third of the rounding
//     of the bf16 output.  (Two planes of weight 1 would keep 2^-16 of the largest
//     only, which shows in elements where the largest weight meets a small value.
//     Four planes here: 64 requests of 8 rows 128 us instead of 103.)
// Scores, statistics and output sums are f32; the softmax denominator is
// summed from the f32 weights.
//
// p is relative to the maximum over its own tile and row, not to the running
// one, and p s_v is brought by a power of two of the row's own, 2^-k, under
// the row's largest p |s_v| of the tile: every row's weights fill e4m3's range,
// whatever the scales of blocks that the row does not attend to, and a long
// tail of small weights keeps its share.  (k comes
// from the maxima of sixteen tokens, which share a scale, and their scales'
// exponents, so it costs no second maximum.)  Each tile's product is read back
// and added to f32 sums in registers with its factor 2^(m_r - running maximum)
// 2^k, so nothing in tensor memory is ever rescaled.
//
// Work: all (request, cache head, row group, tile) quadruples in one list, cut
// into one contiguous range per CTA, so ragged lengths balance.  A unit
// (request, head, row group) that lies across CTAs is joined by the CTA that
// finishes last, over the partial sums in CTA order (deterministic); one in more
// than 24 parts in two steps, eights first (one request of 53580 tokens, one
// cache head of 256, in 140 parts: 36 us, in one step 103).
//
// Roles (640 threads, one CTA per SM): warps 0-3 and 4-7 softmax of even and odd
// tiles (TMEM lane = token), warps 8-11 output sums (TMEM lane = element of
// head_dim), warps 12-15 query planes of the units to come, warps 16 and 19 TMA
// producers of K and V (a lane per block), warps 17 and 18 the MMAs of even and
// odd tiles.
// Rows go through the softmax eight at a time in a loop, and scores are read
// from tensor memory twice rather than kept: unrolled over 32 rows, the roles'
// code did not fit the instruction caches, and that was the largest stall.
//   Bound: HBM for few query rows, the softmax groups for many (a tile of 32
// rows of f32 took a group about 7000 cycles when references were the tile's:
// 1500 for the maxima, 3500 for weights, planes and sums, the rest waits and
// barriers; of eight rows of bf16, 2400).  Measured in a graph, 8 cache heads of
// 128: 64 requests of 4.2 k tokens on average, eight bf16 rows a head, 105 us
// (79% of the copy rate); one of 131072 tokens 54 us (74%: start-up and join take
// the rest); 16 of 8.4 k with 4..32 f32 rows a head 111 us (37%).  With one
// reference per tile, less exact, these were 101, 54 and 108 us.
//   Measured slower (the last case, then at 119 us): 16 rows at a time (141), a
// third softmax group (140), the planes as a loop over their weights (123);
// redux.sync for the maxima, both products of a tile from one issuer in order,
// the join as a function of its own (most cases by 1 to 7 us).
//   Every wait is bounded; a timeout raises a CTA-wide flag, the rows' outputs and
// lse become NaN, the join still counts, copies and MMAs in flight are waited for,
// and the status word records it.
#pragma once

#include "tc8_gemv.cuh"

namespace fp8blk {

constexpr int kAtThreads = 640;
constexpr int kAtOutWarp = 8, kAtQueryWarp = 12, kAtKWarp = 16, kAtMmaWarp = 17, kAtVWarp = 19;
constexpr int kAtTile = 128;            // tokens per tile
constexpr int kAtDeep = 4;              // tiles between the first product and the sums: scores, weights and products
constexpr int kAtScaleDeep = 16;        // tiles whose scales are held: more than K's ring and the scores can be ahead of the softmax
constexpr int kAtMaxGrid = 256;         // bound on CTAs: arrival counters and partial sums in the workspace
constexpr int kAtJoin = 24;             // parts of a unit that one CTA joins by itself; more are joined in two steps,
constexpr int kAtFanLog2 = 3;           // eights of them first
constexpr size_t kAtHeaderBytes = 2 * kAtMaxGrid * sizeof(uint32_t);
constexpr float kAtNoRef = -3.0e38f;    // maximum of a row that has seen nothing
constexpr int kAtPeakLog2 = 7;          // a row's largest weight of a tile in the planes is in [2^6, 2^8) (e4m3 ends at 448)
constexpr int kAtSpread = 120;          // a row's weights are lifted by up to 2^120: value scales further apart in a tile
                                        // than that lose bits of what lies under the smaller one
constexpr int kAtMinScale = -119;       // value scales below 2^-119 count as 2^-119 (with a smaller factor)

struct AttnArgs {
    const void *q;
    void *out;
    float *lse;                       // or null
    const float *k_scales, *v_scales;
    const int32_t *table, *seq_lens, *q_starts;
    uint32_t *counters;               // [2][kAtMaxGrid] of the joins' first and second steps, zero between calls
    float *partials;                  // [grid][2][R x (ND * 128) sums | R references | R denominators]
    unsigned int *status;
    uint64_t wait_limit_ns;           // of the roles' waits (drains keep kWaitLimitNs)
    int64_t q_stride, out_stride, n_blocks;
    int n_seqs, max_m, total_rows, kv_heads, group, head_dim, block_log2, width;
    int max_tiles;                    // a table's tiles and one more
    float scale_log2;                 // softmax scale x log2 e
};

__device__ float g_attn_nan = __builtin_nanf("");  // what a block outside the pool has for a scale

template <int PL, int R, int ND>
struct AttnShape {
    static constexpr int kGroups = 2;                         // weights, each a group of R columns
    static constexpr int kSteps = PL / kGroups;               // planes of one weight, an MMA each
    static constexpr int N = kGroups * R;                     // columns of a product
    static constexpr int kTileBytes = ND * kAtTile * 128;     // K or V codes of a tile
    static constexpr int kQStep = N * 128;                    // query planes of one step and half of head_dim
    static constexpr int kQBytes = ND * kSteps * kQStep;      // query planes of a unit
    static constexpr int kPStep = kAtTile * N;                // weight planes of one step
    static constexpr int kPBytes = kSteps * kPStep;           // weight planes of a tile
    static constexpr int kPDeep = (PL == 4 && N == 64) || ND == 2 ? 2 : kAtDeep;  // tiles whose weights are held
    static constexpr int kFixed = 1024 + 2 * kQBytes + kPDeep * kPBytes;
    static constexpr int kRoom = (227 - 10) * 1024;           // dynamic shared memory beside the static arrays
    static constexpr int kTiles = (kRoom - kFixed) / kTileBytes;
    // V's tiles are held longer than K's (until the weights are there).
    static constexpr int kStagesV = (kTiles + 1) / 2 > 6 ? 6 : (kTiles + 1) / 2;
    static constexpr int kStagesK = kTiles / 2 > 6 ? 6 : kTiles / 2;
    static constexpr size_t kSmem = kFixed + static_cast<size_t>(kStagesK + kStagesV) * kTileBytes;
    static constexpr int kTmemUsed = N * kAtDeep * (1 + ND);  // scores and products
    static constexpr int kTmem = kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
    static constexpr int kPartial = R * (ND * 128) + 2 * R;   // floats of one partial
    static_assert(kStagesK >= 2 && kStagesK + kAtDeep < kAtScaleDeep && kTmemUsed <= 512 && N % 16 == 0 && N <= 64, "shape");
};

// Shared-memory descriptor of an operand tile whose rows are `row_bytes` (128,
// 64, 32 or 16) long under the swizzle of that width, in groups of 8 rows.
// K-major operands have rows along M or N; MN-major ones along K.
template <int ROW_BYTES>
__device__ __forceinline__ uint64_t at_desc(uint32_t saddr) {
    constexpr uint64_t layout = ROW_BYTES == 128 ? 2 : ROW_BYTES == 64 ? 4 : ROW_BYTES == 32 ? 6 : 0;
    constexpr uint64_t group = 8 * ROW_BYTES;
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= (ROW_BYTES == 16 ? group >> 4 : 1ull) << 16;  // without a swizzle the 8-row groups step by the leading offset
    d |= (group >> 4) << 32;
    d |= 1ull << 46;
    d |= layout << 61;
    return d;
}
__host__ __device__ constexpr uint32_t at_idesc(int n, bool mn_major) {
    return t8_idesc(128, n) | (mn_major ? (1u << 15) | (1u << 16) : 0u);
}
// Byte offset `a` inside a tile under the swizzle of ROW_BYTES-long rows.
template <int ROW_BYTES>
__device__ __forceinline__ uint32_t at_swizzle(uint32_t a) {
    constexpr uint32_t mask = ROW_BYTES / 16 - 1;
    return a ^ (((a >> 7) & mask) << 4);
}

__device__ __forceinline__ void at_ld8(uint32_t taddr, float *v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[j]);
}
__device__ __forceinline__ void at_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// e4m3x2 -> two f16, exactly.
__device__ __forceinline__ uint32_t at_e4m3x2_f16x2(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}
// a -= the low f16 of h, b -= the high one (exact here: a residual of rounding).
__device__ __forceinline__ void at_minus(uint32_t h, float &a, float &b) {
    asm("{\n\t.reg .b16 l, u, m;\n\tmov.b32 {l, u}, %2;\n\tmov.b16 m, 0xBC00;\n\t"
        "fma.rn.f32.f16 %0, l, m, %0;\n\tfma.rn.f32.f16 %1, u, m, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(h));
}
// What is left after a plane is scaled up where the next one has another weight,
// so that it does not end in e4m3's subnormals.  Plane p lies in step p % steps,
// column group p / steps.
template <int PL>
__device__ __forceinline__ float at_join(const float (&d)[2]) { return fmaf(d[1], PL == 2 ? 1.f / 16.f : 1.f / 256.f, d[0]); }
// The four values' plane p as a word of codes; the values become what it leaves.
template <int PL>
__device__ __forceinline__ uint32_t at_plane(int p, float &a, float &b, float &c, float &d) {
    const uint32_t lo = t8_to_e4m3x2(a, b), hi = t8_to_e4m3x2(c, d);
    if (p + 1 < PL) {
        at_minus(at_e4m3x2_f16x2(lo), a, b);
        at_minus(at_e4m3x2_f16x2(hi), c, d);
        if (p + 1 == PL / 2) {
            const float gain = PL == 2 ? 16.f : 256.f;
            a *= gain;
            b *= gain;
            c *= gain;
            d *= gain;
        }
    }
    return lo | (hi << 16);
}
// Eight consecutive words of shared memory (16-byte aligned).
__device__ __forceinline__ void at_lds8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ float at_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Waits of the roles in the tile loop: no suspend hint, every lane polls.  For at
// most limit_ns, or until another role has raised the abort flag.
__device__ __forceinline__ bool at_wait(uint32_t bar, uint32_t parity, int *abort_flag, uint64_t limit_ns) {
    if (mbar_try_wait_short(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait_short(bar, parity)) return true;
        if (*reinterpret_cast<volatile int *>(abort_flag)) return false;
        if (global_timer_ns() - t0 >= limit_ns) {
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
            return false;
        }
    }
}
// The same for a whole warp: one outcome for all lanes.
__device__ __forceinline__ bool at_warp_wait(uint32_t bar, uint32_t parity, int *abort_flag, uint64_t limit_ns) {
    const bool ok = at_wait(bar, parity, abort_flag, limit_ns);
    return __all_sync(0xFFFFFFFFu, ok);
}

// Named barrier over the 128 threads of one role, and the same with an OR.
__device__ __forceinline__ void at_bar(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool at_bar_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(v)), "r"(id)
        : "memory");
    return r != 0;
}

// One of eight values, folded by `op` over the sixteen lanes of each half of the
// warp, as a butterfly that halves the values a lane holds at each step: eight
// shuffles (one redux.sync per value measured about 50 cycles each, one after
// another).  Lane l ends with value at_owned(l) of its half.
__device__ __forceinline__ int at_owned(int lane) { return (lane & 8 ? 4 : 0) + (lane & 4 ? 2 : 0) + (lane & 2 ? 1 : 0); }
template <typename F>
__device__ __forceinline__ float at_butterfly(const float (&x)[8], int lane, F op) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool up = lane & 8;
        v[i] = op(up ? x[i + 4] : x[i], __shfl_xor_sync(0xFFFFFFFFu, up ? x[i] : x[i + 4], 8));
    }
#pragma unroll
    for (int h = 4, n = 2; n; h >>= 1, n >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i < n) {
                const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                v[i] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, give, h));
            }
    }
    return op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], 1));
}

// One request as the kernel takes it.
struct AttnSeq {
    int first, rows, len;  // rows 0: nothing to do
    int tiles;             // per unit; 0 for an empty cache
    int groups;            // row groups
    int weight;            // list entries of a tile
    bool bad;
    // List entries of all its units: each has one tile's worth for its set-up, then its tiles.
    __device__ __forceinline__ int entries(int kv_heads) const { return kv_heads * groups * (tiles + 1) * weight; }
};
template <int R>
__device__ __forceinline__ AttnSeq at_seq(const AttnArgs &a, int s) {
    AttnSeq q;
    q.first = a.q_starts[s];
    const int64_t rows = static_cast<int64_t>(a.q_starts[s + 1]) - q.first;
    const int len = a.seq_lens[s];
    const bool off = q.first < 0 || rows < 0 || rows > a.max_m || q.first + rows > a.total_rows;
    q.bad = off || len < 0;
    q.rows = off ? 0 : static_cast<int>(rows);
    q.len = max(len, 0);
    // A length past the table ends in a tile past it, whose scales are NaN: every row sees some of it.
    q.tiles = min((q.len >> 7) + ((q.len & 127) != 0), a.max_tiles);
    q.groups = (q.rows * a.group + R - 1) / R;
    // Measured on f32 tiles of 8, 16 and 32 rows: 1.1, 1.5 and 1.9 us, about (3 + eighths) x 0.28.  (Lists of bf16 are
    // cut by the same figures, which were not measured for them.)
    q.weight = R == 8 ? 1 : 3 + min(R, q.rows * a.group + 7) / 8;
    return q;
}

// CTA b's range of a list of `total` entries over `grid` <= total CTAs: the first
// total % grid CTAs take one entry more.
struct AttnSplit {
    int each, more;
    __device__ __forceinline__ AttnSplit(int total, int grid) : each(total / grid), more(total - each * grid) {}
    __device__ __forceinline__ int begin(int b) const { return b * each + min(b, more); }
    __device__ __forceinline__ int owner(int x) const {
        const int head = more * (each + 1);
        return x < head ? x / (each + 1) : more + (x - head) / each;
    }
};

// The largest weight of a tile.
__host__ __device__ constexpr int at_max_weight(int rows) { return rows == 8 ? 1 : 3 + rows / 8; }

// A unit of at most kAtSmall tiles is never cut: a cut inside it moves to its
// start (joining two parts costs more than the tiles).  Other cuts move to the
// start of a tile.
constexpr int kAtSmall = 4;

// A position in the CTA's range of the list: request, unit of the request, its
// tiles from slot e0 on (slot 0 is the set-up, slot j + 1 tile j), tiles
// [j0, j1), and the list entries left after them.
template <int R>
struct AttnWalk {
    const AttnArgs &a;
    AttnSeq q;
    int s, unit, e0, j0, j1, left;
    __device__ __forceinline__ AttnWalk(const AttnArgs &args, const AttnSeq &seq, int s0, int slot, int count)
        : a(args), q(seq), s(s0), left(count) {
        unit = slot / (q.tiles + 1);
        e0 = slot - unit * (q.tiles + 1);
        clip();
    }
    __device__ __forceinline__ void clip() {
        const int e1 = min(q.tiles + 1, e0 + (R == 8 ? left : left / q.weight));
        left -= (e1 - e0) * q.weight;
        j0 = max(e0 - 1, 0);
        j1 = e1 - 1;
    }
    __device__ __forceinline__ bool none() const { return j1 <= j0; }  // no tile here
    // The next unit; false at the end of the range.
    __device__ __forceinline__ bool next() {
        if (left <= 0) return false;
        if (++unit == a.kv_heads * q.groups) {
            unit = 0;
            do q = at_seq<R>(a, ++s);
            while (q.rows == 0);
        }
        e0 = 0;
        clip();
        return true;
    }
    __device__ __forceinline__ int head() const { return unit / q.groups; }
    __device__ __forceinline__ int row0() const { return (unit % q.groups) * R; }
    // The unit's rows, up to a multiple of eight.
    __device__ __forceinline__ int rows() const { return R == 8 ? 8 : min(R, (q.rows * a.group - row0() + 7) & ~7); }
};

template <typename T>
__device__ __forceinline__ float4 at_load4(const T *p);
template <>
__device__ __forceinline__ float4 at_load4<float>(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 at_load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    const float2 lo = bf16x2_to_f32(w.x), hi = bf16x2_to_f32(w.y);
    return make_float4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void at_store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void at_store4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Query planes of one unit: a warp takes four rows at a time, eight lanes a row.
// A lane holds four quarters of 4 elements, 32 elements apart, per 128-wide half.
// The row's exponent, scale and last visible position ride along.
template <typename T, int PL, int R, int ND>
__device__ __forceinline__ void at_build_queries(const AttnArgs &a, const AttnWalk<R> &w, uint8_t *dst, float *qs, int *lim, int part,
                                                 int parts, int lane) {
    using Sh = AttnShape<PL, R, ND>;
    const int row0 = w.row0(), valid = min(R, w.q.rows * a.group - row0);
    const T *q = static_cast<const T *>(a.q) + w.q.first * a.q_stride + static_cast<int64_t>(w.head()) * a.group * a.head_dim;
    const int sub = lane >> 3, l8 = lane & 7;
    float4 next[ND][4];
    int i = 0;
    auto fetch = [&](int r) {
        i = (row0 + r) / a.group;
        const T *x = q + i * a.q_stride + (row0 + r - i * a.group) * a.head_dim;
#pragma unroll
        for (int h = 0; h < ND; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int d = h * 128 + k * 32 + 4 * l8;
                next[h][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < valid && d < a.head_dim) next[h][k] = at_load4<T>(x + d);
            }
    };
    if (4 * part < R) fetch(4 * part + sub);
    for (int r = 4 * part + sub; r < R; r += 4 * parts) {
        float4 v[ND][4];
#pragma unroll
        for (int h = 0; h < ND; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[h][k] = next[h][k];
        const int token = i;
        if (r + 4 * parts < R) fetch(r + 4 * parts);  // on their way while these rows are encoded
        uint32_t g = 0;  // largest |x| as bits; a NaN sorts above infinity
#pragma unroll
        for (int h = 0; h < ND; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 f = v[h][k];
                g = max(g, max(max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))),
                               max(__float_as_uint(fabsf(f.z)), __float_as_uint(fabsf(f.w)))));
            }
#pragma unroll
        for (int d = 4; d; d >>= 1) g = max(g, __shfl_xor_sync(0xFFFFFFFFu, g, d));
        const int ex = t8_plane_exponent(__uint_as_float(g));
        float f1, f2;
        t8_pow2_split(ex == kT8Poison ? 0 : ex, f1, f2);
        if (l8 == 0) {
            float g1, g2;
            t8_pow2_split(ex == kT8Poison ? 0 : -ex, g1, g2);
            qs[r] = ex == kT8Poison ? __int_as_float(0x7FC00000) : a.scale_log2 * g1 * g2;
            lim[r] = r < valid ? w.q.len - w.q.rows + token : w.q.len - 1;
        }
#pragma unroll
        for (int h = 0; h < ND; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float t0 = v[h][k].x * f1 * f2, t1 = v[h][k].y * f1 * f2, t2 = v[h][k].z * f1 * f2, t3 = v[h][k].w * f1 * f2;
#pragma unroll
                for (int p = 0; p < PL; ++p) {
                    const int n = p / Sh::kSteps * R + r;
                    *reinterpret_cast<uint32_t *>(dst + (h * Sh::kSteps + p % Sh::kSteps) * Sh::kQStep + at_swizzle<128>(n * 128 + k * 32 + 4 * l8)) =
                        at_plane<PL>(p, t0, t1, t2, t3);
                }
            }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // generic stores -> the MMA
}

template <typename T, int PL, int R, int ND>
__global__ void __launch_bounds__(kAtThreads, 1)
    kv_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const AttnArgs a) {
    using Sh = AttnShape<PL, R, ND>;
    constexpr int N = Sh::N, SK = Sh::kStagesK, SV = Sh::kStagesV, PD = Sh::kPDeep, G = Sh::kGroups;
    extern __shared__ __align__(1024) uint8_t at_smem[];
    __shared__ __align__(8) uint64_t k_full[SK], k_free[SK], v_full[SV], v_free[SV], sc_full[kAtScaleDeep];
    __shared__ __align__(8) uint64_t s_full[kAtDeep], s_free[kAtDeep], p_full[kAtDeep], o_full[kAtDeep], o_free[kAtDeep];
    __shared__ __align__(8) uint64_t q_full[2], ml_full[2], ml_free[2], mma_done[2];
    __shared__ __align__(16) float sc[kAtScaleDeep][2][8];                       // k and v scales of a tile's blocks
    __shared__ __align__(16) float s_qs[2][R];          // per query row: 2^-e x scale x log2 e (NaN: the row is not finite)
    __shared__ __align__(16) int s_lim[2][R];           // last position each row sees
    __shared__ __align__(16) float s_wmax[2][8][R];     // per softmax group: maxima over sixteen tokens of the tile
    __shared__ __align__(16) float s_ve[2][8];          // ... and the exponents of their value scales
    __shared__ __align__(16) float s_tref[kAtDeep][R], s_lf[2][R], s_lc[2][R];  // tile maximum; factors into and of the group's denominator
    __shared__ __align__(16) float s_lift[kAtDeep][R];  // per row: 2^(peak + the tile's top value scale's exponent - k)
    __shared__ uint32_t s_top[kAtDeep];                 // less a lift's bits: the bits of that row's 2^(k - peak)
    __shared__ __align__(16) float s_corr[R], s_of[R];  // output sums: factor of the sums so far, and of the tile's product
    __shared__ float s_l[2][8][R], s_mref[2][2][R], s_inv[R];
    __shared__ int s_vnan[2][ND * 128];                 // first position whose value code is NaN, per element
    __shared__ int s_scan[kAtThreads / 32];
    __shared__ AttnSeq s_seq;
    __shared__ int s_first, s_slot, s_begin, s_end, s_abort, s_last;
    __shared__ uint32_t tmem_slot;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *sQ = at_smem + ((1024u - (smem_addr(at_smem) & 1023u)) & 1023u);
    uint8_t *sP = sQ + 2 * Sh::kQBytes;
    uint8_t *sK = sP + PD * Sh::kPBytes;                // K's ring, then V's
    uint8_t *sV = sK + static_cast<size_t>(SK) * Sh::kTileBytes;

    // A thread per barrier.
    {
        auto init = [&](uint64_t *bars, int n, int first, int count) {
            if (tid >= first && tid < first + n) mbar_init(smem_addr(bars + tid - first), static_cast<uint32_t>(count));
            return first + n;
        };
        int at = init(sc_full, kAtScaleDeep, 0, 32);
        at = init(k_full, SK, at, 1);
        at = init(k_free, SK, at, 1);
        at = init(v_full, SV, at, 1);
        at = init(v_free, SV, at, 1);
        at = init(s_full, kAtDeep, at, 1);
        at = init(s_free, kAtDeep, at, 4);
        at = init(p_full, kAtDeep, at, 4);
        at = init(o_full, kAtDeep, at, 1);
        at = init(o_free, kAtDeep, at, 4);
        at = init(q_full, 2, at, 4);
        at = init(ml_full, 2, at, 8);
        at = init(ml_free, 2, at, 4);
        at = init(mma_done, 2, at, 1);
        if (tid < at) mbar_init_fence();
        if (tid == 0) s_abort = 0;
    }
    for (int i = tid; i < 2 * ND * 128; i += kAtThreads) (&s_vnan[0][0])[i] = 0x7FFFFFFF;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_slot)),
                     "r"(Sh::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    t8_fence_before();
    __syncthreads();
    t8_fence_after();
    const uint32_t tmem = tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the list: tiles of every request, scanned by every CTA -- by every warp for itself (lane = request) up to 32
    // requests, else by all threads together (thread i sums requests [i per, (i + 1) per)).  The host keeps the total
    // below 2^31.
    int total, grid, begin = 0, end = 0, first = 0, slot = 0;  // this CTA's range, its first request and slot
    AttnSeq seq = {};
    {
        const bool alone = a.n_seqs <= 32;
        const int per = alone ? 1 : (a.n_seqs + kAtThreads - 1) / kAtThreads;
        const int r0 = min((alone ? lane : tid) * per, a.n_seqs), r1 = min(r0 + per, a.n_seqs);
        int mine = 0;
        bool bad = false;
        AttnSeq q = {};
        q.weight = 1;
        for (int s = r0; s < r1; ++s) {
            q = at_seq<R>(a, s);
            mine += q.entries(a.kv_heads);
            bad |= q.bad;
        }
        if (bad && blockIdx.x == 0) atomicOr(a.status, 4u);
        int pre = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, pre, d);
            if (lane >= d) pre += u;
        }
        int base = 0;
        total = __shfl_sync(0xFFFFFFFFu, pre, 31);
        if (!alone) {
            if (lane == 31) s_scan[warp] = pre;
            __syncthreads();
            const int sum = s_scan[min(lane, kAtThreads / 32 - 1)];  // each warp's sum, in the lanes of its number
            total = __reduce_add_sync(0xFFFFFFFFu, lane < kAtThreads / 32 ? sum : 0);
            base = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sum : 0);
        }
        // Every CTA's share is at least a tile, so no two cuts move to the same place inside a unit.
        grid = min(static_cast<int>(gridDim.x), max(total / at_max_weight(R), min(total, 1)));
        const int at = base + pre - mine;  // this thread's first entry
        // A cut at entry x of a request that begins at `at`: its slot, and its list position once moved to the slot's
        // start, or to the unit's where the unit is small.
        auto cut = [](int x, int at, int tiles, int weight, int &sl) {
            sl = R == 8 ? x - at : (x - at) / weight;
            if (tiles <= kAtSmall) sl -= sl % (tiles + 1);
            return at + sl * weight;
        };
        if (static_cast<int>(blockIdx.x) < grid) {
            const AttnSplit split(total, grid);
            const int x0 = split.begin(blockIdx.x), x1 = split.begin(blockIdx.x + 1);
            if (alone) {
                int sl;
                const unsigned has1 = __ballot_sync(0xFFFFFFFFu, at <= x1 && x1 < at + mine);
                if (has1 == 0) {
                    end = total;
                } else {
                    const int from = __ffs(has1) - 1;
                    end = cut(x1, __shfl_sync(0xFFFFFFFFu, at, from), __shfl_sync(0xFFFFFFFFu, q.tiles, from),
                              __shfl_sync(0xFFFFFFFFu, q.weight, from), sl);
                }
                first = __ffs(__ballot_sync(0xFFFFFFFFu, at <= x0 && x0 < at + mine)) - 1;
                seq.first = __shfl_sync(0xFFFFFFFFu, q.first, first);
                seq.rows = __shfl_sync(0xFFFFFFFFu, q.rows, first);
                seq.len = __shfl_sync(0xFFFFFFFFu, q.len, first);
                seq.tiles = __shfl_sync(0xFFFFFFFFu, q.tiles, first);
                seq.groups = __shfl_sync(0xFFFFFFFFu, q.groups, first);
                seq.weight = __shfl_sync(0xFFFFFFFFu, q.weight, first);
                begin = cut(x0, __shfl_sync(0xFFFFFFFFu, at, first), seq.tiles, seq.weight, slot);
            } else {
                auto locate = [&](int x, int &r, int &sl) {  // among this thread's requests
                    int here = at;
                    r = r0;
                    if (per > 1) q = at_seq<R>(a, r);
                    while (x >= here + q.entries(a.kv_heads)) {
                        here += q.entries(a.kv_heads);
                        q = at_seq<R>(a, ++r);
                    }
                    return cut(x, here, q.tiles, q.weight, sl);
                };
                int r, sl;
                if (at <= x1 && x1 < at + mine) s_end = locate(x1, r, sl);
                else if (tid == 0 && x1 == total) s_end = total;
                if (at <= x0 && x0 < at + mine) {
                    s_begin = locate(x0, r, sl);
                    s_seq = q;
                    s_first = r;
                    s_slot = sl;
                }
            }
        }
        if (!alone) {
            __syncthreads();
            if (static_cast<int>(blockIdx.x) < grid) {
                begin = s_begin;
                end = s_end;
                first = s_first;
                slot = s_slot;
                seq = s_seq;
            }
        }
    }

    if (begin < end) {
        const AttnSplit split(total, grid);
        AttnWalk<R> w(a, seq, first, slot, end - begin);
        const bool built = !w.none();
        if (warp < kAtKWarp && (built || warp >= kAtQueryWarp)) {
            // ---------------- query planes: all these warps build the first unit's; the last four go on with the others.
            // (One loop: the code is long, and a second copy of it would cost the other roles instruction cache.)
            AttnWalk<R> n(w);
            int ub = 0, iu = 0;
            bool all = built;
            do {
                if (n.none()) continue;
                // The unit before last is written out: nothing reads this buffer, its scales or its limits any more.
                if (iu >= 2 && !at_warp_wait(smem_addr(&ml_free[ub]), static_cast<uint32_t>((iu >> 1) - 1) & 1u, &s_abort, a.wait_limit_ns)) break;
                at_build_queries<T, PL, R, ND>(a, n, sQ + ub * Sh::kQBytes, s_qs[ub], s_lim[ub], all ? warp : warp - kAtQueryWarp,
                                               all ? kAtKWarp : 4, lane);
                if (all) asm volatile("bar.sync 4, %0;" ::"n"(kAtKWarp * 32) : "memory");
                if (warp < kAtQueryWarp) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&q_full[ub]));
                all = false;
                ++iu;
                ub ^= 1;
            } while (n.next());
        }
        if (warp == kAtKWarp || warp == kAtVWarp) {
            // ---------------- TMA producers: lane p copies the tile's p-th block of K (or V); K's brings both scales
            const bool is_v = warp == kAtVWarp;
            const int np = kAtTile >> a.block_log2, block = 1 << a.block_log2;
            const uint64_t pol = l2_policy_evict_first();
            const CUtensorMap *map = is_v ? &vmap : &kmap;
            const uint32_t ring = smem_addr(is_v ? sV : sK);
            uint64_t *full = is_v ? v_full : k_full, *free = is_v ? v_free : k_free;
            const int S = is_v ? SV : SK;
            int st = 0;
            uint32_t ph = 0;
            int64_t it = 0;
            // Block ids, 32 table entries at a time in the lanes' registers: the window in use, the one after it, and
            // the first one of the next unit, each asked for long before its use.
            AttnWalk<R> n(w);
            bool more = !n.none();
            auto skip = [&] {
                do more = n.next();
                while (more && n.none());
            };
            if (!more) skip();
            auto load_ids = [&](int page0) {
                const int page = page0 + lane;
                return more && page < a.width ? a.table[static_cast<int64_t>(n.s) * a.width + page] : -1;
            };
            int ids_unit = load_ids(n.j0 * np);
            bool ok = true;
            while (ok && more) {
                const int j1 = n.j1, len = n.q.len, head = n.head(), page_end = j1 * np;
                const int32_t *row = a.table + static_cast<int64_t>(n.s) * a.width;
                int j = n.j0, win = j * np, ids = ids_unit;
                auto window = [&](int page0) {
                    const int page = page0 + lane;
                    return page0 < page_end && page < a.width ? row[page] : -1;
                };
                int ids_next = window(win + 32);
                skip();
                ids_unit = load_ids(n.j0 * np);
                for (; j < j1; ++j) {
                    const int page0 = j * np;
                    if (page0 >= win + 32) {
                        win += 32;
                        ids = ids_next;
                        ids_next = window(win + 32);
                    }
                    const int pages = min(np, (len >> a.block_log2) + ((len & (block - 1)) != 0) - page0);
                    const int id = __shfl_sync(0xFFFFFFFFu, ids, (page0 - win + lane) & 31);
                    const bool mine = lane < pages, good = id >= 0 && id < a.n_blocks;
                    if (mine && !good) atomicOr(a.status, 4u);
                    const int64_t bh = static_cast<int64_t>(good ? id : 0) * a.kv_heads + head;
                    if (it >= S && !at_warp_wait(smem_addr(&free[st]), ph ^ 1u, &s_abort, a.wait_limit_ns)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_addr(&full[st]);
                    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(pages) * block * 128 * ND);
                    __syncwarp();
                    const int slot = static_cast<int>(it & (kAtScaleDeep - 1));
                    if (mine) {
                        const uint32_t at = ring + static_cast<uint32_t>(st) * Sh::kTileBytes + lane * block * 128;
#pragma unroll
                        for (int h = 0; h < ND; ++h)
                            t8_tma_2d(at + h * kAtTile * 128, map, h * 128, static_cast<int>(bh << a.block_log2), bar, pol);
                        if (!is_v) {
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(&sc[slot][0][lane])),
                                         "l"(good ? a.k_scales + bh : &g_attn_nan)
                                         : "memory");
                            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(&sc[slot][1][lane])),
                                         "l"(good ? a.v_scales + bh : &g_attn_nan)
                                         : "memory");
                        }
                    }
                    if (!is_v)
                        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sc_full[slot])) : "memory");
                    ++it;
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // What is still in flight lands before the CTA's shared memory is released.
            for (int64_t v = it > S ? it - S : 0; v < it; ++v) (void)mbar_wait_bounded(smem_addr(&full[v % S]), static_cast<uint32_t>((v / S) & 1));
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == kAtMmaWarp || warp == kAtMmaWarp + 1) {
            // ---------------- MMA issuers: warp g issues both products of the tiles g, g + 2, ...  Whichever of the two
            // can go next goes, the second product first (it frees a stage).
            if (lane == 0) {
                const int g = warp - kAtMmaWarp;
                constexpr uint32_t qk_idesc = at_idesc(N, false), pv_idesc = at_idesc(N, true);
                // Descriptors of the rings' starts; an offset adds to the address field (16-byte units, 14 bits).
                const uint64_t k_desc = at_desc<128>(smem_addr(sK)), q_desc = at_desc<128>(smem_addr(sQ));
                const uint64_t v_desc = at_desc<128>(smem_addr(sV)), p_desc = at_desc<N>(smem_addr(sP));
                int qt = g, pt = g;         // next tile of each product
                int q_st = g, p_st = g;     // ... and its slot in K's, V's ring
                uint32_t q_ph = 0, p_ph = 0;
                int iu = -1, unit_end = 0;  // the first product's unit, and the tile after its last
                bool more = true;           // false: unit_end is the end of the range
                uint64_t t0 = 0;
                int spins = 0;
                // The clock is read every 32 polls, or every poll under a shorter limit: these polls do not suspend, so
                // that a limit of 0 ends at the first one that finds nothing.
                const int every = a.wait_limit_ns < kWaitLimitNs ? 1 : 32;
                while (more || pt < unit_end) {
                    bool went = false;
                    {
                        const int b = pt & (kAtDeep - 1);
                        const uint32_t bp = static_cast<uint32_t>(pt / kAtDeep) & 1u;
                        if (pt < qt && mbar_test_wait(smem_addr(&p_full[b]), bp) && mbar_test_wait(smem_addr(&v_full[p_st]), p_ph) &&
                            (pt < kAtDeep || mbar_test_wait(smem_addr(&o_free[b]), bp ^ 1u))) {
                            t8_fence_after();
                            const uint64_t va = v_desc + static_cast<uint32_t>(p_st) * (Sh::kTileBytes / 16);
                            const uint64_t pa = p_desc + static_cast<uint32_t>(b & (PD - 1)) * (Sh::kPBytes / 16);
                            const uint32_t d = tmem + static_cast<uint32_t>((kAtDeep + b * ND) * N);
#pragma unroll
                            for (int h = 0; h < ND; ++h)
#pragma unroll
                                for (int x = 0; x < Sh::kSteps; ++x)
#pragma unroll
                                    for (int c = 0; c < 4; ++c)
                                        t8_mma(d + h * N, va + (h * kAtTile * 128 + c * 32 * 128) / 16,
                                               pa + (x * Sh::kPStep + c * 32 * N) / 16, pv_idesc, x + c > 0);
                            t8_commit(smem_addr(&o_full[b]));
                            t8_commit(smem_addr(&v_free[p_st]));
                            pt += 2;
                            p_st += 2;
                            if (p_st >= SV) {
                                p_st -= SV;
                                p_ph ^= 1u;
                            }
                            went = true;
                        }
                    }
                    while (more && qt >= unit_end) {  // on to the unit that tile qt belongs to
                        if (iu >= 0 || w.none()) more = w.next();
                        while (more && w.none()) more = w.next();
                        if (more) {
                            ++iu;
                            unit_end += w.j1 - w.j0;
                        }
                    }
                    if (qt < unit_end) {
                        const int b = qt & (kAtDeep - 1);
                        const uint32_t bp = static_cast<uint32_t>(qt / kAtDeep) & 1u;
                        if (mbar_test_wait(smem_addr(&k_full[q_st]), q_ph) && (qt < kAtDeep || mbar_test_wait(smem_addr(&s_free[b]), bp ^ 1u)) &&
                            mbar_test_wait(smem_addr(&q_full[iu & 1]), static_cast<uint32_t>(iu >> 1) & 1u)) {
                            t8_fence_after();
                            const uint64_t ka = k_desc + static_cast<uint32_t>(q_st) * (Sh::kTileBytes / 16);
                            const uint64_t qa = q_desc + static_cast<uint32_t>(iu & 1) * (Sh::kQBytes / 16);
                            const uint32_t d = tmem + static_cast<uint32_t>(b * N);
#pragma unroll
                            for (int h = 0; h < ND; ++h)
#pragma unroll
                                for (int x = 0; x < Sh::kSteps; ++x)
#pragma unroll
                                    for (int c = 0; c < 4; ++c)
                                        if (h * 128 + c * 32 < a.head_dim)  // columns past head_dim are zeros on both sides
                                            t8_mma(d, ka + (h * kAtTile * 128 + c * 32) / 16,
                                                   qa + ((h * Sh::kSteps + x) * Sh::kQStep + c * 32) / 16, qk_idesc, h + x + c > 0);
                            t8_commit(smem_addr(&s_full[b]));
                            t8_commit(smem_addr(&k_free[q_st]));
                            qt += 2;
                            q_st += 2;
                            if (q_st >= SK) {
                                q_st -= SK;
                                q_ph ^= 1u;
                            }
                            went = true;
                        }
                    }
                    if (went) {
                        spins = 0;
                    } else if ((++spins & (every - 1)) == 0) {  // bounded, as at_wait
                        if (*reinterpret_cast<volatile int *>(&s_abort)) break;
                        const uint64_t now = global_timer_ns();
                        if (spins == every && a.wait_limit_ns != 0) t0 = now;
                        else if (now - t0 >= a.wait_limit_ns) {
                            *reinterpret_cast<volatile int *>(&s_abort) = 1;
                            break;
                        }
                    }
                }
                t8_commit(smem_addr(&mma_done[g]));
                (void)mbar_wait_bounded(smem_addr(&mma_done[g]), 0u);
            }
        } else if (warp < kAtOutWarp) {
            // ---------------- softmax: group g takes the tiles g, g + 2, ...; thread = token of the tile
            const int g = warp >> 2, wg = warp & 3, tg = tid & 127, bar = 1 + g;
            const float nanf = __int_as_float(0x7FC00000);
            const uint32_t lanes = static_cast<uint32_t>(wg * 32) << 16;
            int st = 0, ub = 0;
            uint32_t ph = 0;
            int64_t it = 0, iu = 0;
            bool ok = true;
            do {
                if (w.none()) continue;
                const uint32_t uph = static_cast<uint32_t>((iu >> 1) & 1);
                ok = ok && at_warp_wait(smem_addr(&q_full[ub]), uph, &s_abort, a.wait_limit_ns) &&
                     (iu < 2 || at_warp_wait(smem_addr(&ml_free[ub]), uph ^ 1u, &s_abort, a.wait_limit_ns));
                float ref = kAtNoRef;  // running maximum of row `tg` (threads below R)
                float *den = s_l[ub][warp];  // this warp's denominators; lane l looks after its own of every eight rows
                const int own = at_owned(lane);
                const bool owner = (lane & 17) == 0;
                if (owner) {
#pragma unroll
                    for (int c = 0; c < R; c += 8) den[c + own] = 0.f;
                }
                const int seen_by_all = w.q.len - w.q.rows;  // positions up to here are seen by every row
                const int rows = w.rows();                   // columns past the unit's rows hold what they may
                for (int j = w.j0; j < w.j1; ++j, ++it) {
                    const int vs_st = st;  // V's slot
                    const uint32_t v_ph = ph;
                    if (++st == SV) {
                        st = 0;
                        ph ^= 1u;
                    }
                    if ((it & 1) != g) continue;
                    const uint32_t bp = static_cast<uint32_t>(it / kAtDeep) & 1u;
                    const int b = static_cast<int>(it & (kAtDeep - 1));
                    const int cs = static_cast<int>(it & (kAtScaleDeep - 1));  // the scales' slot
                    const int pos = j * kAtTile + tg;
                    ok = ok && at_warp_wait(smem_addr(&sc_full[cs]), static_cast<uint32_t>(it / kAtScaleDeep) & 1u, &s_abort, a.wait_limit_ns);
                    // This token's value scale, relative to the power of two under the tile's largest.
                    const int blocks = (min(w.q.len - j * kAtTile, kAtTile) - 1) >> a.block_log2;  // the last one's number
                    float vs[8], vtop = 0.f;
                    at_lds8(sc[cs][1], vs);
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const float x = fabsf(vs[p]);
                        if (p <= blocks && x < INFINITY) vtop = fmaxf(vtop, x);
                    }
                    const int ve = max(__float_as_int(vtop) >> 23, 127 + kAtMinScale);  // biased exponent
                    // (A scale that is not finite counts as NaN: as a factor of codes it would saturate in the planes.)
                    const float sv = sc[cs][1][tg >> a.block_log2], sk = sc[cs][0][tg >> a.block_log2];
                    const float vscale = fabsf(sv) < INFINITY ? sv * __int_as_float(ve == 254 ? 0x00400000 : (254 - ve) << 23) : nanf;
                    const float ks = fabsf(sk) < INFINITY ? sk : nanf;
                    if (tg < 8) {
                        const float x = fabsf(sc[cs][1][tg * 16 >> a.block_log2]);
                        s_ve[g][tg] = static_cast<float>(max((__float_as_int(x) >> 23) - 127, kAtMinScale));
                    }
                    ok = ok && at_warp_wait(smem_addr(&s_full[b]), bp, &s_abort, a.wait_limit_ns);
                    const bool edge = (j + 1) * kAtTile - 1 > seen_by_all;  // some row does not see the whole tile
                    // Scores of rows c .. c + 7, in base 2; what a row does not see is -inf.
                    auto scores = [&](int c, float (&s)[8]) {
                        float d[G][8], qs[8];
#pragma unroll
                        for (int x = 0; x < G; ++x) at_ld8(tmem + lanes + static_cast<uint32_t>(b * N + x * R + c), d[x]);
                        at_lds8(s_qs[ub] + c, qs);
                        at_wait_ld();
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            float u[G];
#pragma unroll
                            for (int x = 0; x < G; ++x) u[x] = d[x][r];
                            s[r] = at_join<PL>(u) * (qs[r] * ks);
                        }
                        if (edge) {
#pragma unroll
                            for (int r = 0; r < 8; ++r) s[r] = pos > s_lim[ub][c + r] ? -INFINITY : s[r];
                        }
                    };
                    auto release = [&] {  // the scores' columns may be overwritten
                        t8_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&s_free[b]));
                    };
                    t8_fence_after();
                    float s[8];
                    // Each row's maxima over sixteen tokens.
#pragma unroll 1
                    for (int c = 0; c < rows; c += 8) {
                        scores(c, s);
                        const float top = at_butterfly(s, lane, [](float x, float y) { return fmaxf(x, y); });
                        if ((lane & 1) == 0) s_wmax[g][2 * wg + (lane >> 4)][c + own] = top;
                    }
                    if constexpr (R == 8) release();
                    // One warp waits until the output sums have read what the tile kAtDeep ago left in this slot, another until
                    // the second MMA has read its weights.
                    if (wg == 1 && it >= kAtDeep) ok = at_wait(smem_addr(&o_free[b]), bp ^ 1u, &s_abort, a.wait_limit_ns) && ok;
                    at_bar(bar);
                    if (PD < kAtDeep && wg == 2 && it >= PD)
                        ok = at_wait(smem_addr(&o_full[(it - PD) & (kAtDeep - 1)]), static_cast<uint32_t>((it - PD) / kAtDeep) & 1u, &s_abort, a.wait_limit_ns) && ok;
                    if (tg < rows) {
                        float part[8], exps[8], tref = kAtNoRef, most = -INFINITY;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            part[x] = s_wmax[g][x][tg];
                            tref = fmaxf(tref, part[x]);
                        }
                        const float now = fmaxf(ref, tref);
                        // k: the largest p |s_v| is below 2^(k + 1).  (The difference first: it is exact for scores of any size.)
                        at_lds8(s_ve[g], exps);
#pragma unroll
                        for (int x = 0; x < 8; ++x) most = fmaxf(most, (part[x] - tref) + exps[x]);
                        const int k = min(max(__float2int_ru(most), max(ve - 127 - kAtSpread, kAtMinScale)), ve - 127);
                        s_lift[b][tg] = __int_as_float((kAtPeakLog2 + ve - k) << 23);
                        s_lf[g][tg] = at_exp2(tref - now);
                        s_lc[g][tg] = at_exp2(ref - now);
                        ref = now;
                        s_tref[b][tg] = tref;
                        if (tg == 0) s_top[b] = static_cast<uint32_t>(ve + 127) << 23;
                    }
                    at_bar(bar);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    // This token's row of the weight planes; the swizzle turns on bits that are the row's alone.
                    uint8_t *pb = sP + (b & (PD - 1)) * Sh::kPBytes + tg * N;
                    constexpr uint32_t turns = N / 16 - 1;
                    const uint32_t turn = ((static_cast<uint32_t>(tg * N) >> 7) & turns) << 4;
#pragma unroll 1
                    for (int c = 0; c < rows; c += 8) {
                        if constexpr (R > 8) scores(c, s);
                        float t[8], tref[8];
                        at_lds8(s_tref[b] + c, tref);
#pragma unroll
                        for (int r = 0; r < 8; ++r) s[r] = at_exp2(s[r] - tref[r]);
                        at_lds8(s_lift[b] + c, t);
#pragma unroll
                        for (int r = 0; r < 8; ++r) t[r] = s[r] * t[r] * vscale;
                        if (edge) {
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                if (pos > s_lim[ub][c + r]) t[r] = 0.f;  // whatever the scale
                        }
#pragma unroll
                        for (int p = 0; p < PL; ++p) {
                            uint2 word;
                            word.x = at_plane<PL>(p, t[0], t[1], t[2], t[3]);
                            word.y = at_plane<PL>(p, t[4], t[5], t[6], t[7]);
                            *reinterpret_cast<uint2 *>(pb + p % Sh::kSteps * Sh::kPStep + ((p / Sh::kSteps * R + c) ^ turn)) = word;
                        }
                        float sum = at_butterfly(s, lane, [](float x, float y) { return x + y; });
                        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
                        if (owner) den[c + own] = fmaf(den[c + own], s_lc[g][c + own], sum * s_lf[g][c + own]);
                    }
                    if constexpr (R > 8) release();
                    if (edge) {
                        // This token's row of V: zeros where the request ends (what is there is no token's), and NaN
                        // codes that only later rows see leave the tile and mark the element for those rows.
                        ok = ok && at_warp_wait(smem_addr(&v_full[vs_st]), v_ph, &s_abort, a.wait_limit_ns);
                        if (ok && pos > seen_by_all) {
#pragma unroll
                            for (int h = 0; h < ND; ++h) {
                                uint8_t *row = sV + static_cast<size_t>(vs_st) * Sh::kTileBytes + h * kAtTile * 128;
                                if (pos >= w.q.len) {
#pragma unroll
                                    for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(row + tg * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
                                    continue;
                                }
                                uint32_t nan = 0;
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    const uint4 x = *reinterpret_cast<const uint4 *>(row + tg * 128 + c * 16);
                                    nan |= ((x.x & 0x7F7F7F7Fu) + 0x01010101u) | ((x.y & 0x7F7F7F7Fu) + 0x01010101u) |
                                           ((x.z & 0x7F7F7F7Fu) + 0x01010101u) | ((x.w & 0x7F7F7F7Fu) + 0x01010101u);
                                }
                                if ((nan & 0x80808080u) == 0u) continue;  // no NaN code in the row
#pragma unroll 1
                                for (int c = 0; c < 128; ++c) {
                                    uint8_t *at = row + at_swizzle<128>(tg * 128 + c);
                                    if ((*at & 0x7Fu) != 0x7Fu) continue;
                                    *at = 0;
                                    atomicMin(&s_vnan[ub][h * 128 + c], pos);
                                }
                            }
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // generic stores -> the MMA
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&p_full[b]));
                }
                if (tg < rows) s_mref[ub][g][tg] = ref;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ml_full[ub]));
                ++iu;
                ub ^= 1;
            } while (w.next());
        } else if (warp < kAtQueryWarp) {
            // ---------------- output sums: thread = element d (and d + 128) of head_dim
            const int dt = tid - kAtOutWarp * 32, ow = warp - kAtOutWarp;
            const uint32_t lanes = static_cast<uint32_t>(ow * 32) << 16;
            int ub = 0;
            int64_t it = 0, iu = 0;
            int done = begin;
            bool ok = true;
            const float nanf = __int_as_float(0x7FC00000);
            T *out = static_cast<T *>(a.out);
            do {
                const int row0 = w.row0(), valid = min(R, w.q.rows * a.group - row0), kvh = w.head();
                const int rows = w.rows();
                const bool whole = w.j0 == 0 && w.j1 == w.q.tiles;
                const int unit_begin = done - w.e0 * w.q.weight;  // list position of the unit
                done += (w.j1 + 1 - w.e0) * w.q.weight;
                auto out_row = [&](int r) {  // (row, query head) of the unit's row r
                    const int i = (row0 + r) / a.group;
                    return static_cast<int64_t>(w.q.first + i) * a.out_stride +
                           static_cast<int64_t>(kvh * a.group + (row0 + r - i * a.group)) * a.head_dim;
                };
                auto lse_at = [&](int r) {
                    const int i = (row0 + r) / a.group;
                    return static_cast<int64_t>(w.q.first + i) * (a.kv_heads * a.group) + kvh * a.group + (row0 + r - i * a.group);
                };
                if (w.q.len == 0) {  // nothing cached: zeros, and no part in the pipeline
                    for (int r = 0; r < valid; ++r) {
#pragma unroll
                        for (int h = 0; h < ND; ++h)
                            if (dt + h * 128 < a.head_dim) out[out_row(r) + dt + h * 128] = static_cast<T>(0.f);
                        if (a.lse && dt == 0) a.lse[lse_at(r)] = -INFINITY;
                    }
                    continue;
                }
                if (w.none()) continue;
                float ref = kAtNoRef;  // running maximum of row `dt` (threads below R)
                float acc[ND][R];
#pragma unroll
                for (int h = 0; h < ND; ++h)
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[h][r] = 0.f;
                for (int j = w.j0; j < w.j1; ++j) {
                    const int b = static_cast<int>(it & (kAtDeep - 1));
                    const uint32_t bp = static_cast<uint32_t>(it / kAtDeep) & 1u;
                    ok = ok && at_warp_wait(smem_addr(&o_full[b]), bp, &s_abort, a.wait_limit_ns) &&
                         at_warp_wait(smem_addr(&p_full[b]), bp, &s_abort, a.wait_limit_ns);  // long complete: orders the softmax's words
                    t8_fence_after();
                    bool raised = false;
                    at_bar(3);  // every warp has read the last tile's factors
                    if (dt < rows) {
                        const float tref = s_tref[b][dt], now = fmaxf(ref, tref);
                        raised = now > ref;
                        s_corr[dt] = at_exp2(ref - now);
                        s_of[dt] = at_exp2(tref - now) * __uint_as_float(s_top[b] - __float_as_uint(s_lift[b][dt]));
                        ref = now;
                    }
                    const bool moved = at_bar_or(3, raised);
#pragma unroll
                    for (int c = 0; c < R; c += 8) {
                        if (c < rows) {
                            float f[8];
                            if (moved) {
                                at_lds8(s_corr + c, f);
#pragma unroll
                                for (int h = 0; h < ND; ++h)
#pragma unroll
                                    for (int r = 0; r < 8; ++r) acc[h][c + r] *= f[r];
                            }
                            at_lds8(s_of + c, f);
#pragma unroll
                            for (int h = 0; h < ND; ++h) {
                                float d[G][8];
#pragma unroll
                                for (int x = 0; x < G; ++x)
                                    at_ld8(tmem + lanes + static_cast<uint32_t>((kAtDeep + b * ND + h) * N + x * R + c), d[x]);
                                at_wait_ld();
#pragma unroll
                                for (int r = 0; r < 8; ++r) {
                                    float x[G];
#pragma unroll
                                    for (int y = 0; y < G; ++y) x[y] = d[y][r];
                                    acc[h][c + r] = fmaf(at_join<PL>(x), f[r], acc[h][c + r]);
                                }
                            }
                        }
                    }
                    t8_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&o_free[b]));
                    ++it;
                }
                ok = ok && at_warp_wait(smem_addr(&ml_full[ub]), static_cast<uint32_t>((iu >> 1) & 1), &s_abort, a.wait_limit_ns);
                // One outcome for the group, and no result out of weights that a softmax group gave up on (it raised the flag
                // before it reported the unit).
                ok = !at_bar_or(3, !ok || *reinterpret_cast<volatile int *>(&s_abort) != 0);
                if (!ok) {
#pragma unroll
                    for (int h = 0; h < ND; ++h)
#pragma unroll
                        for (int r = 0; r < R; ++r) acc[h][r] = nanf;
                }
#pragma unroll
                for (int h = 0; h < ND; ++h) {
                    const int p = s_vnan[ub][h * 128 + dt];
                    if (p != 0x7FFFFFFF) {  // a NaN value code: the rows that see it
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            if (s_lim[ub][r] >= p) acc[h][r] = nanf;
                        s_vnan[ub][h * 128 + dt] = 0x7FFFFFFF;
                    }
                }
                float l = 0.f;  // denominator of row `dt` at the maximum `ref`
                if (dt < rows) {
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        l += at_exp2(s_mref[ub][g][dt] - ref) * ((s_l[ub][4 * g][dt] + s_l[ub][4 * g + 1][dt]) +
                                                                 (s_l[ub][4 * g + 2][dt] + s_l[ub][4 * g + 3][dt]));
                    if (!ok) l = nanf;
                }
                if (whole) {
                    if (dt < rows) {
                        s_inv[dt] = l == 0.f ? 0.f : 1.f / l;
                        if (a.lse && dt < valid) a.lse[lse_at(dt)] = l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
                    }
                    at_bar(3);
                    int64_t at = out_row(0);
                    int c = row0 % a.group;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        if (r < valid) {
#pragma unroll
                            for (int h = 0; h < ND; ++h)
                                if (dt + h * 128 < a.head_dim) out[at + dt + h * 128] = static_cast<T>(acc[h][r] * s_inv[r]);
                        }
                        at += a.head_dim;
                        if (++c == a.group) {
                            c = 0;
                            at += a.out_stride - static_cast<int64_t>(a.group) * a.head_dim;
                        }
                    }
                    at_bar(3);  // s_inv is free again
                } else {
                    // A part of a unit: its sums go to the workspace, and the part that arrives last joins them all.
                    float *mine = a.partials + (static_cast<int64_t>(blockIdx.x) * 2 + (w.j0 == 0)) * Sh::kPartial;
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int h = 0; h < ND; ++h) __stcg(mine + r * (ND * 128) + h * 128 + dt, acc[h][r]);
                    if (dt < R) {
                        __stcg(mine + R * ND * 128 + dt, ref);
                        __stcg(mine + R * ND * 128 + R + dt, l);
                    }
                    // The CTAs of the unit's first and last tile: a tile belongs to the last CTA whose range begins in it or
                    // before it.
                    const int b0 = split.owner(unit_begin + 2 * w.q.weight - 1);
                    const int parts = split.owner(unit_begin + (w.q.tiles + 1) * w.q.weight - 1) - b0 + 1;
                    // The CTA that arrives last joins the parts; of many parts, eights first, an eight's sums in place of its
                    // first part's.  An eight of one part is joined already.  (That one lies in the unit's last CTA, which may
                    // begin another unit and then counts that one's parts in its counter; the CTAs of the other eights' first
                    // parts hold nothing else, or begin this unit.)
                    auto part = [&](int p) {  // part p lies in CTA b0 + p, which holds one that begins a unit and one that does not
                        return a.partials + (static_cast<int64_t>(b0 + p) * 2 + (p == 0)) * Sh::kPartial;
                    };
                    int lo = 0, shift = 0, count = parts;  // the parts lo + (p << shift), p < count
                    uint32_t *counter = a.counters + b0;
                    bool eights = false;
                    if (parts > kAtJoin) {
                        lo = (static_cast<int>(blockIdx.x) - b0) >> kAtFanLog2 << kAtFanLog2;
                        count = min(parts - lo, 1 << kAtFanLog2);
                        counter += lo;
                        eights = true;
                    }
#pragma unroll 1
                    while (true) {
                        if (eights && count == 1) {
                            lo = 0;
                            shift = kAtFanLog2;
                            count = (parts + (1 << kAtFanLog2) - 1) >> kAtFanLog2;
                            counter = a.counters + kAtMaxGrid + b0;
                            eights = false;
                        }
                        at_bar(3);
                        if (dt == 0) {  // the barrier and this release order every thread's sums before the count
                            uint32_t old;
                            asm volatile("fence.acq_rel.gpu;\n\tatom.inc.relaxed.gpu.global.u32 %0, [%1], %2;\n\tfence.acq_rel.gpu;"
                                         : "=r"(old)
                                         : "l"(counter), "r"(static_cast<uint32_t>(count - 1))
                                         : "memory");
                            s_last = old == static_cast<uint32_t>(count - 1);
                        }
                        at_bar(3);
                        if (!s_last) break;
                        // Maxima and denominators: 128 / R threads a row.  (Loops, not unrolled code: this runs once or
                        // twice a launch, and fetching its instructions would take longer than the loads.)
                        constexpr int L = 128 / R;
                        const int row = dt / L;
                        float m = kAtNoRef, d = 0.f;
#pragma unroll 4
                        for (int p = dt % L; p < count; p += L) {
                            const float *src = part(lo + (p << shift)) + R * ND * 128 + row;
                            const float pm = __ldcg(src), pl = __ldcg(src + R), top = fmaxf(m, pm);
                            d = d * at_exp2(m - top) + pl * at_exp2(pm - top);
                            m = top;
                        }
#pragma unroll
                        for (int x = L / 2; x; x >>= 1) {
                            const float om = __shfl_xor_sync(0xFFFFFFFFu, m, x), od = __shfl_xor_sync(0xFFFFFFFFu, d, x), top = fmaxf(m, om);
                            // The lower lane's share first on both sides: one order, one result.
                            const float mine = d * at_exp2(m - top), other = od * at_exp2(om - top);
                            d = dt & x ? other + mine : mine + other;
                            m = top;
                        }
                        if (dt % L == 0) {
                            s_corr[row] = m;
                            s_inv[row] = d == 0.f ? 0.f : 1.f / d;
                            if (!eights && a.lse && row < valid) a.lse[lse_at(row)] = d == 0.f ? -INFINITY : (m + log2f(d)) * 0.6931471805599453f;
                        }
                        at_bar(3);
                        // Sums: a thread takes four elements of every 128th quadruple, kItems at a time over all parts.
                        constexpr int kAll = R * ND / 4, kItems = kAll < 4 ? kAll : 4, kAhead = 16 / kItems;
#pragma unroll 1
                        for (int k0 = 0; k0 < kAll; k0 += kItems) {
                            float4 o[kItems];
#pragma unroll
                            for (int k = 0; k < kItems; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll kAhead
                            for (int p = 0; p < count; ++p) {
                                const float *src = part(lo + (p << shift));
#pragma unroll
                                for (int k = 0; k < kItems; ++k) {
                                    const int i = (k0 + k) * 128 + dt, r = i / (ND * 32);
                                    const float f = at_exp2(__ldcg(src + R * ND * 128 + r) - s_corr[r]);
                                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(src) + i);
                                    o[k].x = fmaf(x.x, f, o[k].x);
                                    o[k].y = fmaf(x.y, f, o[k].y);
                                    o[k].z = fmaf(x.z, f, o[k].z);
                                    o[k].w = fmaf(x.w, f, o[k].w);
                                }
                            }
#pragma unroll
                            for (int k = 0; k < kItems; ++k) {
                                const int i = (k0 + k) * 128 + dt, r = i / (ND * 32), e = (i & (ND * 32 - 1)) * 4;
                                if (eights) {
                                    __stcg(reinterpret_cast<float4 *>(part(lo)) + i, o[k]);  // this thread alone reads it above
                                } else if (r < valid && e < a.head_dim) {
                                    const float f = s_inv[r];
                                    at_store4(out + out_row(r) + e, make_float4(o[k].x * f, o[k].y * f, o[k].z * f, o[k].w * f));
                                }
                            }
                        }
                        if (!eights) break;
                        at_bar(3);  // every thread has read the parts' maxima
                        if (dt % L == 0) {
                            __stcg(part(lo) + R * ND * 128 + row, m);
                            __stcg(part(lo) + R * ND * 128 + R + row, d);
                        }
                        count = 1;  // its eight is joined
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ml_free[ub]));
                ++iu;
                ub ^= 1;
            } while (w.next());
        }
    }

    t8_fence_before();
    __syncthreads();
    if (tid == 0 && *reinterpret_cast<volatile int *>(&s_abort)) atomicOr(a.status, 1u);
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(Sh::kTmem) : "memory");
}

}  // namespace fp8blk
