// rope.cu -- rotary positions: frequencies on the host (fp8blk_rope_frequencies,
// fp8blk_rope_turns), a step's cosines and sines (fp8blk_rope_table), and the
// rotation of queries and keys by them (fp8blk_rope).
#include "overlap.h"
#include "rope.cuh"
#include "step.h"

#include <algorithm>
#include <cmath>

namespace fp8blk {

// --------------------------------------------------------------- the table
struct RopeTableArgs {
    const int32_t *positions;  // [n]
    const uint64_t *turns;     // [half], turns a token as a fraction of 2^64
    float *cos_sin;            // [n, 2, half]
    float scale;
    uint32_t items;            // n x groups
    int half, groups;          // threads of a row: four pairs each
};

constexpr int kRopeThreads = 256;
constexpr int kRopeTablePairs = 4;

// Cosine and sine of `phase` / 2^64 turns.  The nearest quarter turn comes off in
// integers, exactly; what is left, at most pi / 4, goes through the Taylor series
// (next terms: 2e-9 of the sine, 2e-10 of the cosine).  With the roundings of
// the angle and of the sums both are within 2^-23 of the exact value.
__device__ __forceinline__ void rope_cos_sin(uint64_t phase, float &c, float &s) {
    const uint32_t quarter = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);
    const int64_t left = static_cast<int64_t>(phase - (static_cast<uint64_t>(quarter) << 62));
    const float x = __ll2float_rn(left);
    const float a = fmaf(x, 0x1.921fb6p-62f, x * -0x1.777a5cp-87f);  // x 2 pi / 2^64, in two parts
    const float u = a * a;
    float p = fmaf(u, 1.f / 362880.f, -1.f / 5040.f);
    p = fmaf(u, p, 1.f / 120.f);
    p = fmaf(u, p, -1.f / 6.f);
    const float sn = fmaf(a * u, p, a);
    float q = fmaf(u, -1.f / 3628800.f, 1.f / 40320.f);
    q = fmaf(u, q, -1.f / 720.f);
    q = fmaf(u, q, 1.f / 24.f);
    q = fmaf(u, q, -0.5f);
    const float cs = fmaf(u, q, 1.f);
    const bool odd = quarter & 1u;
    c = odd ? sn : cs;
    s = odd ? cs : sn;
    if (quarter == 1u || quarter == 2u) c = -c;
    if (quarter >= 2u) s = -s;
}

// A step's table once for all layers: bound by its launch (64 rows of 128: 4.6 us a
// call from the host; 16384 rows, 8.5 MB, 5.1 us, 24% of the copy rate).
// Angles are fractions of a turn in 64 bits: position x frequency wraps where
// the circle does, so a far position costs no precision (2^31 x the 2^-65 of a turn
// that the frequency is rounded by are 2^-34 of one).
__global__ void __launch_bounds__(kRopeThreads) rope_table_kernel(const RopeTableArgs a) {
    const uint32_t item = blockIdx.x * kRopeThreads + threadIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    if (item >= a.items) return;
    const uint32_t row = item / static_cast<uint32_t>(a.groups);
    const int p0 = static_cast<int>(item - row * a.groups) * kRopeTablePairs;
    const int32_t pos = a.positions[row];
    float c[kRopeTablePairs], s[kRopeTablePairs];
#pragma unroll
    for (int i = 0; i < kRopeTablePairs; ++i) {
        const uint64_t t = p0 + i < a.half ? a.turns[p0 + i] : 0;
        rope_cos_sin(static_cast<uint64_t>(static_cast<int64_t>(pos)) * t, c[i], s[i]);
        c[i] = pos < 0 ? 1.f : c[i] * a.scale;
        s[i] = pos < 0 ? 0.f : s[i] * a.scale;
    }
    float *out = a.cos_sin + static_cast<int64_t>(row) * 2 * a.half + p0;
    if (a.half % kRopeTablePairs == 0) {  // the table is 16-byte aligned
        *reinterpret_cast<float4 *>(out) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4 *>(out + a.half) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
#pragma unroll
        for (int i = 0; i < kRopeTablePairs; ++i)
            if (p0 + i < a.half) {
                out[i] = c[i];
                out[a.half + i] = s[i];
            }
    }
}

// ------------------------------------------------------------ the rotation
// Bound by memory: 16384 rows of 64 heads of 128, bf16, 545 MB, 87 us, 93% of the
// copy rate; 1001 f32 rows of 24 heads of 192, 64 of each rotated, 7.4 us, 74%; 64
// rows of 40 heads 6.4 us a call from the host.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs r, uint32_t items) {
    const uint32_t item = blockIdx.x * kRopeThreads + threadIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    if (item < items) rope_item<T, kRopeHeads<T>>(r, item);
}

}  // namespace fp8blk

using namespace fp8blk;

static constexpr double kTwoPi = 6.283185307179586476925286766559;

extern "C" int fp8blk_rope_frequencies(int scaling, int rot_dim, double base, double factor, double original_len, double low,
                                       double high, double *freqs, float *attn_scale) {
    if (!freqs || rot_dim < 2 || rot_dim > FP8BLK_MAX_ROT || rot_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
        return FP8BLK_EINVAL;
    if (scaling < FP8BLK_ROPE_PLAIN || scaling > FP8BLK_ROPE_BANDS) return FP8BLK_EINVAL;
    if (scaling != FP8BLK_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return FP8BLK_EINVAL;
    if (scaling == FP8BLK_ROPE_RAMP || scaling == FP8BLK_ROPE_BANDS) {
        if (!(original_len >= 1.0) || !std::isfinite(original_len) || !(low > 0.0) || !(high > low) || !std::isfinite(high))
            return FP8BLK_EINVAL;
    }
    if (scaling == FP8BLK_ROPE_BASE) {
        if (rot_dim < 4) return FP8BLK_EINVAL;  // the exponent rot / (rot - 2)
        base *= std::pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
    }
    // Ramp: the pair index at which a frequency makes `turns` turns over the original length.
    auto pair_at = [&](double turns) { return rot_dim * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(base)); };
    const bool ramp = scaling == FP8BLK_ROPE_RAMP;
    const double first = ramp ? std::max(std::floor(pair_at(high)), 0.0) : 0.0;
    const double last = ramp ? std::min(std::ceil(pair_at(low)), static_cast<double>(rot_dim - 1)) : 0.0;
    for (int i = 0; i < rot_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rot_dim);
        double stretched = 0.0;  // share of the pair that is divided by the factor
        if (scaling == FP8BLK_ROPE_LINEAR) stretched = 1.0;
        if (ramp) stretched = std::min(std::max((i - first) / std::max(last - first, 0.001), 0.0), 1.0);
        if (scaling == FP8BLK_ROPE_BANDS)
            stretched = 1.0 - std::min(std::max((original_len * f / kTwoPi - low) / (high - low), 0.0), 1.0);
        freqs[i] = f / factor * stretched + f * (1.0 - stretched);
        if (scaling == FP8BLK_ROPE_PLAIN || scaling == FP8BLK_ROPE_BASE) freqs[i] = f;
    }
    if (attn_scale) *attn_scale = ramp ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return FP8BLK_OK;
}

// 1 / 2 pi as the sum of two doubles (what they leave is 2^-110).
static constexpr double kInvTwoPi = 0x1.45f306dc9c883p-3, kInvTwoPiLow = -0x1.6b01ec5417056p-57;

// |f| / 2 pi as hi + rest, hi the f64 product and rest what it leaves of the exact one (2^-106 of it); then the fraction
// of a turn in units of 2^-64, whole ones and the rest's apart.  Off by half a unit and 2^-25 of one (f <= 10^6).
extern "C" int fp8blk_rope_turns(const double *freqs, int n, uint64_t *turns) {
    if (!freqs || !turns || n < 1 || n > FP8BLK_MAX_ROT / 2) return FP8BLK_EINVAL;
    for (int i = 0; i < n; ++i) {
        if (!(std::fabs(freqs[i]) <= 1e6)) return FP8BLK_EINVAL;
        const double f = std::fabs(freqs[i]);
        const volatile double product = f * kInvTwoPi;  // (rounded, whatever the host's compiler would fuse it with)
        const double hi = product, rest = std::fma(f, kInvTwoPi, -hi) + f * kInvTwoPiLow;
        const double units = (hi - std::floor(hi)) * 0x1p64, whole = std::floor(units);  // exact
        const uint64_t t = static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(std::floor((units - whole) + rest * 0x1p64 + 0.5)));
        turns[i] = freqs[i] < 0 ? 0 - t : t;
    }
    return FP8BLK_OK;
}

extern "C" int fp8blk_rope_table(const int32_t *positions, const uint64_t *turns, float scale, float *cos_sin, int64_t n, int rot_dim,
                                 void *stream) {
    if (!positions || !turns || !cos_sin || n < 1 || rot_dim < 2 || rot_dim % 2 != 0) return FP8BLK_EINVAL;
    if (rot_dim > FP8BLK_MAX_ROT || n > kStepMaxIndex / (rot_dim / 2)) return FP8BLK_ERANGE;
    if (!step_aligned(positions, 4) || !step_aligned(turns, 8) || !step_aligned(cos_sin, 16)) return FP8BLK_EALIGN;
    RopeTableArgs a = {positions, turns, cos_sin, scale, 0, rot_dim / 2, 0};
    a.groups = (a.half + kRopeTablePairs - 1) / kRopeTablePairs;
    a.items = static_cast<uint32_t>(n * a.groups);
    return step_from_cuda(step_launch(rope_table_kernel, dim3((a.items + kRopeThreads - 1) / kRopeThreads), kRopeThreads, 0,
                                      static_cast<cudaStream_t>(stream), a));
}

namespace fp8blk {

// Checks and geometry of a rotation, a head a thread.
int rope_plan(const void *x, void *out, const float *cos_sin, int dtype, int64_t n, int heads, int dim, int rot, int start, int interleaved,
              int64_t x_stride, int64_t out_stride, RopeArgs *r, uint32_t *items) {
    if (!x || !out || !cos_sin || (dtype != FP8BLK_F32 && dtype != FP8BLK_BF16) || n < 1 || heads < 1 || dim < 2) return FP8BLK_EINVAL;
    if (rot < 2 || rot % 2 != 0 || start < 0 || rot > dim || start > dim - rot || (interleaved != 0 && interleaved != 1)) return FP8BLK_EINVAL;
    if (dim > FP8BLK_MAX_ROT || heads > 65535 || n > kStepMaxIndex) return FP8BLK_ERANGE;
    const int64_t row = static_cast<int64_t>(heads) * dim;
    if (x_stride < row || out_stride < row) return FP8BLK_EINVAL;
    if (x_stride > kStepMaxIndex || out_stride > kStepMaxIndex) return FP8BLK_ERANGE;
    const int es = dtype == FP8BLK_F32 ? 4 : 2;
    if (!step_aligned(x, es) || !step_aligned(out, es) || !step_aligned(cos_sin, 16)) return FP8BLK_EALIGN;
    if (x == out && x_stride != out_stride) return FP8BLK_EINVAL;
    *r = RopeArgs{x, out, cos_sin, n, x_stride, out_stride, heads, dim, rot, start, interleaved, 0, 0, 0};
    r->fast = dim % 8 == 0 && start % 8 == 0 && rot % 16 == 0 && step_aligned(x, 16) && step_aligned(out, 16) &&
              x_stride * es % 16 == 0 && out_stride * es % 16 == 0;
    const int per = r->fast ? 8 : 1;
    // In place there is nothing to do outside the rotated part.
    r->units = rot / 2 / per + (x == out ? 0 : (dim - rot) / per);
    r->chunks = heads;
    const int64_t a_row = static_cast<int64_t>(r->units) * r->chunks;
    if (n > (int64_t(1) << 31) / a_row) return FP8BLK_ERANGE;
    if (x != out && rows_overlap(x, x_stride * es, row * es, out, out_stride * es, row * es, n)) return FP8BLK_EINVAL;
    *items = static_cast<uint32_t>(n * a_row);
    return FP8BLK_OK;
}

// A planned rotation by a kernel of its own.
static cudaError_t rope_launch(RopeArgs r, int dtype, cudaStream_t stream) {
    const int each = dtype == FP8BLK_F32 ? kRopeHeads<float> : kRopeHeads<__nv_bfloat16>;
    r.chunks = (r.heads + each - 1) / each;
    const uint32_t items = static_cast<uint32_t>(r.n * r.units * r.chunks);
    const dim3 grid((items + kRopeThreads - 1) / kRopeThreads);
    return dtype == FP8BLK_F32 ? step_launch(rope_kernel<float>, grid, kRopeThreads, 0, stream, r, items)
                               : step_launch(rope_kernel<__nv_bfloat16>, grid, kRopeThreads, 0, stream, r, items);
}

}  // namespace fp8blk

extern "C" int fp8blk_rope(const void *x, int dtype, const float *cos_sin, void *out, int64_t n_rows, int heads, int head_dim, int rot_dim,
                           int rot_start, int interleaved, int64_t x_stride, int64_t out_stride, void *stream) {
    RopeArgs r;
    uint32_t items = 0;
    const int rc = rope_plan(x, out, cos_sin, dtype, n_rows, heads, head_dim, rot_dim, rot_start, interleaved, x_stride, out_stride,
                             &r, &items);
    return rc != FP8BLK_OK ? rc : step_from_cuda(rope_launch(r, dtype, static_cast<cudaStream_t>(stream)));
}
