// fp8mm_loss.cuh -- softmax cross entropy over the columns of an FP8 product,
// and its gradients, without the product ever being in memory.
//
//   z[m, n] = acc[m, n] (s_a[m] s_b[n]) + bias[n]
//   lse[m]  = log sum_n exp z[m, n]
//   loss[m] = lse[m] - z[m, t[m]]
//   dz[m, n] = (exp(z[m, n] - lse[m]) - [n = t[m]]) g[m]
//   dA = dz (s_b B)^T,   dB^T = dz^T (s_a A),   dbias = sum_m dz
//
// One kernel in three kinds, all with 2-SM MMAs on tiles of 256 rows (a cluster of
// two CTAs; roles, ring and barriers as in fp8mm_kernel_pair.cuh):
//
//   kStats  the product z of fp8 operands. Each epilogue warp reduces its quarter
//           of a row of the tile, over the tiles of a unit, to (max, sum of
//           exp(z - max)) and writes those 8 bytes; the warp that meets a row's
//           target writes its z. combine_kernel joins a row's parts in a fixed
//           order.
//   kSlope  the same product again for a piece of the vocabulary; the epilogue
//           writes dz as fp16 (and sums of it over 32 rows for dbias), and eight
//           more warps write the other operands of kGrad, W16 and H16.
//   kGrad   dA = dz W16, whose contraction runs over the vocabulary: dz K-major,
//           W16 [n, K] (the piece of B in fp16) MN-major; and dB^T = dz^T H16 over
//           the rows, both MN-major. One launch for both: the tiles of one fill what
//           the other's last turn leaves, and few rows pay for one kernel's start.
//
// Recomputing z costs 2 M N K flops at the fp8 rate; keeping it would cost
// 2 to 4 bytes of memory per logit, written and read (M = 8192, N = 131072:
// 2 GB and more), which the pieces bound instead. The gradients' products run on 16-bit
// operands: fp8 codes of dz would leave 2 to 3 significant bits.
//
// dz in fp16: 11 significant bits against bf16's 8, one rounding of at most
// 2^-11 relative per element of a long sum, and the only one before the
// output's. Its narrow range is met by powers of two: |dz| <= |g| is known
// before anything is computed, so a row is scaled by 2^12 / 2^e(g) of its own g;
// probabilities down to 2^-26 keep all 11 bits, smaller ones are held to 2^-37 of
// the row's |g|, whatever the other rows' (scaled by the largest |g| of all, a row with
// a millionth of it had 5 % of error in dA with 131072 columns). A scale is split
// into its mantissa (in [1, 2)) and its power of two. The powers, over the largest
// one, go with the codes, which is exact: W16 = code 2^e(s_b), H16 = code
// 2^(e(s_a) + e(g)). The mantissas of the scales go with dz before it is rounded,
//
//   dz'[m, n] = dz[m, n] 2^-e(g[m]) m(s_a[m]) m(s_b[n]),
//
// and since a product sums over one of its two indexes, what belongs to the
// other one comes off its row of the result in fp32: 1 / m(s_a) and 2^e(g) of dA's,
// 1 / m(s_b) of dB's. One dz' serves both.
#pragma once

#include <climits>
#include <type_traits>

#include "fp8mm_kernel.cuh"
#include "fp8mm_rows.cuh"

namespace fp8loss {

namespace ptx = fp8mm::ptx;
using fp8mm::Waiter;

enum Kind { kStats, kSlope, kGrad };
constexpr int kOfA = 0, kOfB = 1;      // kGrad's two products

constexpr int kTile = 256;             // rows and columns of a CTA pair's tile
constexpr int kEpiWarps = 16;           // four per 32 rows of a tile, two blocks of 32 columns each (256 wide)
constexpr int kConvertWarps = 8;       // kSlope
constexpr int kNormParts = 32;         // partial maxima per norm

constexpr float kLog2e = 1.4426950408889634f;

template <int KIND>
struct Cfg {
    static constexpr bool kFp8 = KIND != kGrad;
    static constexpr int kThreads = 64 + 32 * (kEpiWarps + (KIND == kSlope ? kConvertWarps : 0));
    static constexpr int kABytes = 128 * 128;
    static constexpr int kStageBytes = 2 * kABytes;                            // 128 rows of A, up to 128 of B
    static constexpr int kStages = KIND == kStats ? 6 : 5;
    // per warp: a block of output (dz 32 x 32 fp16, gradients 32 rows x 128 bytes)
    static constexpr int kBlockBytes = KIND == kStats ? 0 : KIND == kSlope ? 2048 : 4096;
    static constexpr int kStagingBytes = kEpiWarps * kBlockBytes;
    // per warp and column: scale and bias, kSlope: the scale's mantissa
    static constexpr int kColFloats = KIND == kStats ? 2 : KIND == kSlope ? 3 : 0;
    static constexpr int kCols = kTile / 4;
    static constexpr int kColBytes = kEpiWarps * kCols * kColFloats * 4;
    static constexpr int kPowerBytes = KIND == kSlope ? kConvertWarps * 32 * 4 : 0;   // see load_powers
    static constexpr int kNormBytes = KIND == kSlope ? 3 * 64 : 0;                    // see shared_norm
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kStagingBytes + kColBytes + kPowerBytes + kNormBytes + 256;
    static_assert(kSmemBytes <= 232448, "exceeds 227 KB of shared memory");
};

// The tensor maps of a product's operands and output.
struct Maps {
    CUtensorMap a, b, out;
};
template <int KIND>
struct AllMaps {
    Maps of[KIND == kGrad ? 2 : 1];
};

// Tiles of 2 x `half` rows (128, or less of few rows: a multiple of 32) and
// `width` columns (a multiple of 32; 256 for the gradients). The MMA's other rows hold
// what was in shared memory and are not looked at.
struct TileSpace {
    int rows, cols, half, width;
    int kblocks;                       // of 128 bytes of contraction
    int tiles_p, tiles_q, group, splits, run, num_units;
    int units_in_group;                // group x units of a tile row
    uint32_t idesc;
};

// One of kGrad's products.
struct Result {
    int scaled;                        // apply the norms (else a sum of partials does)
    float factor;                      // beside the norms
    int norm_of;                       // dA: kNormB, dB: kNormH
    const float *row_scale;            // of the result's rows: scale_a, or scale_b from the piece on
    int out_type;
    int add;                           // add to the output (fp32)
};

struct LossParams {
    TileSpace t[2];                    // kGrad: of dA and dB; else the first
    int *status;
    unsigned long long timeout_cycles;
    int rowwise;
    const uint32_t *norms;             // see norm_scale
    // fp8 kinds (column vectors start at the piece)
    int M, N;
    const float *scale_a, *scale_b;
    const void *bias;
    int bias_type;
    const int64_t *target;
    long long ignore, col0;            // col0: the piece's first column in the vocabulary
    long long vocabulary;
    // kStats
    float2 *stats;                     // [parts][M]
    float *target_z;                   // [M]
    // kSlope
    const float *lse, *dloss;
    int dloss_step;                    // 0: one value for all rows
    float *colsum;                     // [ceil(M / 32)][n], or nullptr
    long long colsum_ld;
    uint32_t *norms_out;               // not nullptr: few values, of which this kernel finds the norms itself
    __half *w16, *h16;                 // [n, K] and [M, K], or nullptr: not wanted
    int K, a_type, b_type;
    // kGrad (dA also: target, ignore, dloss, dloss_step)
    Result r[2];
};

// ------------------------------------------------------------------ norms ---
// The largest magnitudes of g and s_b as bit patterns (which order like the magnitudes, NaN
// above everything) and the largest row_exponent(), without rows to be ignored, in
// kNormParts partial maxima each.

constexpr int kNormG = 0, kNormB = 1, kNormH = 2;

// The power of two of a magnitude's bits (at least 2^-100, so that its reciprocal is finite;
// infinite for an infinity or NaN, whose results are then NaN).
__device__ __forceinline__ float norm_power(uint32_t most) { return fmaxf(__uint_as_float(most & 0x7F800000u), 0x1p-100f); }

// e(g) of a row, as a power of two.
__device__ __forceinline__ float row_power(float g) { return norm_power(__float_as_uint(g)); }

// e(s_a) + e(g) of a row, 254 above their value; 0 where s_a counts as zero (see power), and
// more than any for an infinity or NaN.
constexpr uint32_t kInfinite = 1024;

__device__ __forceinline__ uint32_t row_exponent(float scale, float g)
{
    const uint32_t es = __float_as_uint(scale) >> 23 & 255, eg = __float_as_uint(row_power(g)) >> 23;
    return es == 255 || eg == 255 ? kInfinite : es == 0 ? 0u : es + eg;
}

struct NormsParams {
    const float *dloss, *scale_b, *scale_a;
    const int64_t *target;
    long long ignore;
    long long count[3];
    int dloss_step, rowwise;
    uint32_t *out;                     // [3][kNormParts]
};

constexpr int kNormThreads = 256;

static __global__ void __launch_bounds__(kNormThreads) norms_kernel(const NormsParams p)
{
    __shared__ uint32_t part[kNormThreads / 32];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int which = blockIdx.y;
    uint32_t most = 0;
    for (long long i = blockIdx.x * kNormThreads + threadIdx.x; i < p.count[which]; i += kNormThreads * kNormParts) {
        if (which == kNormB) {
            most = max(most, __float_as_uint(__ldg(p.scale_b + i)) & 0x7FFFFFFFu);
            continue;
        }
        if (__ldg(p.target + i) == p.ignore)
            continue;
        const float g = __ldg(p.dloss + i * p.dloss_step);
        most = max(most, which == kNormG ? __float_as_uint(g) & 0x7FFFFFFFu : row_exponent(__ldg(p.scale_a + (p.rowwise ? i : 0)), g));
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kNormThreads / 32; ++w)
            most = max(most, part[w]);
        p.out[which * kNormParts + blockIdx.x] = most;
    }
}

// The largest of a norm's parts. Every lane of a warp calls it.
__device__ __forceinline__ uint32_t norm_most(const uint32_t *norms, int which)
{
    return __reduce_max_sync(0xFFFFFFFFu, __ldcg(norms + which * kNormParts + (threadIdx.x & 31)));
}
__device__ __forceinline__ float norm_scale(const uint32_t *norms, int which) { return norm_power(norm_most(norms, which)); }

// What a result's sums have to be multiplied by beside its row's own factor: `factor`, a power
// of two, times the norms that its operands were divided by.
__device__ __forceinline__ float result_scale(const uint32_t *norms, int norm_of, float factor)
{
    if (norm_of == kNormB)
        return factor * norm_scale(norms, kNormG) * norm_scale(norms, kNormB);
    const uint32_t h = norm_most(norms, kNormH);
    return h == kInfinite ? INFINITY : ldexpf(factor, static_cast<int>(h) - 254);
}

// The largest of value(i), i < count, over `threads` threads of a CTA that call it, on a
// hardware barrier of theirs. `shared`: a word for each of their warps.
template <int THREADS, typename F>
__device__ __forceinline__ uint32_t shared_norm(int count, int thread, uint32_t *shared, int barrier, F value)
{
    uint32_t most = 0;
#pragma unroll 4
    for (int i = thread; i < count; i += THREADS)
        most = max(most, value(i));
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if ((thread & 31) == 0)
        shared[thread >> 5] = most;
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "n"(THREADS) : "memory");
    return __reduce_max_sync(0xFFFFFFFFu, (thread & 31) < THREADS / 32 ? shared[thread & 31] : 0u);
}

// dz' is in (-8, 8) without it: below fp16's 65504.
constexpr float kSlopeScale = 0x1p12f;

// Of the codes: 448 x 2^7 and 57344 are below it too.
__host__ __device__ constexpr float code_scale(int fp8_type) { return fp8_type == 0 ? 0x1p7f : 1.0f; }

// A scale's mantissa, with its sign, and its power of two. What is under 2^-126
// counts as zero; an infinity's and a NaN's power is infinite.
__device__ __forceinline__ float mantissa(float s)
{
    const uint32_t b = __float_as_uint(s);
    return (b & 0x7F800000u) ? __uint_as_float((b & 0x807FFFFFu) | 0x3F800000u) : 1.0f;
}
__device__ __forceinline__ float power(float s) { return __uint_as_float(__float_as_uint(s) & 0x7F800000u); }

// ----------------------------------------------------------- tile kernel ---

struct Work {
    int of;                            // kGrad: kOfA or kOfB
    int tp, tq, split, kb0, kb1;
    int unit_q;                        // the unit's place among its tile row's
    bool first, last;                  // of its unit
};

// The tiles of one CTA pair, in order. A unit is `run` tiles of a tile row (the
// last of a row may have fewer) or one K slice of a tile; units go round-robin, one
// slice of all tiles after another, in groups of `group` tile rows that sweep all
// columns, so that what is in use at a time stays in L2.
template <int KIND>
struct Schedule {
    const LossParams &p;
    unsigned u, step;
    int t;
    __device__ __forceinline__ Schedule(const LossParams &params, int pair, int pairs)
        : p(params), u(static_cast<unsigned>(pair)), step(static_cast<unsigned>(pairs)), t(0)
    {
    }

    // (Divisions only where a unit begins: in every tile, in each role, they were a
    // third of the 1.5 us that a tile of K = 128 took without its epilogue's work.)
    __device__ __forceinline__ bool next(Work &w)
    {
        const TileSpace *s = p.t;
        if (t == 0) {
            unsigned v = u;
            w.of = kOfA;
            if (KIND == kGrad && v >= static_cast<unsigned>(s->num_units)) {
                v -= static_cast<unsigned>(s->num_units);
                w.of = kOfB;
                ++s;
            }
            if (v >= static_cast<unsigned>(s->num_units))
                return false;
            w.split = 0;
            if (KIND == kGrad && s->splits > 1) {
                const unsigned tiles = static_cast<unsigned>(s->num_units) / static_cast<unsigned>(s->splits);
                w.split = static_cast<int>(v / tiles);
                v -= static_cast<unsigned>(w.split) * tiles;
            }
            const unsigned in_group = static_cast<unsigned>(s->units_in_group);
            const unsigned group = v / in_group, start = group * static_cast<unsigned>(s->group);
            const unsigned size = min(static_cast<unsigned>(s->tiles_p) - start, static_cast<unsigned>(s->group));
            const unsigned r = v - group * in_group, q = r / size;
            w.tp = static_cast<int>(start + r - q * size);
            w.unit_q = static_cast<int>(q);
            w.tq = w.unit_q * s->run;
            w.kb0 = 0;
            w.kb1 = s->kblocks;
            if (KIND == kGrad && s->splits > 1) {
                w.kb0 = static_cast<int>(static_cast<long long>(w.split) * s->kblocks / s->splits);
                w.kb1 = static_cast<int>(static_cast<long long>(w.split + 1) * s->kblocks / s->splits);
            }
        } else {
            if (KIND == kGrad && w.of == kOfB)
                ++s;
            ++w.tq;
        }
        w.first = t == 0;
        w.last = t + 1 == s->run || w.tq + 1 == s->tiles_q;
        if (w.last) {
            t = 0;
            u += step;
        } else {
            ++t;
        }
        return true;
    }
};

// The K blocks of a tile that kSlope's converting warps take: of its rows of B and of
// A. The tiles that share rows share their blocks in turn.
struct Converted {
    int a, b, step_a, step_b;
    bool of_a, of_b;                   // of the block that has() was last asked for
    __device__ __forceinline__ Converted(const LossParams &p, const Work &w)
        : a(p.h16 ? w.tq : INT_MAX), b(p.w16 ? w.tp : INT_MAX), step_a(p.t[0].tiles_q), step_b(p.t[0].tiles_p), of_a(false), of_b(false)
    {
    }
    // (for each block in order)
    __device__ __forceinline__ bool has(int kb)
    {
        of_a = kb == a;
        of_b = kb == b;
        if (of_a)
            a += step_a;
        if (of_b)
            b += step_b;
        return of_a || of_b;
    }
};

// A converting warp's rows of a stage are 16 i + 2 warp + (0 or 1), i < 8: 16 lanes a
// row, 8 codes each, so that it writes 2 x 256 bytes at once. It takes its codes
// into registers, which gives the stage back early, then converts and writes them.
//
// `powers` holds the powers of two of the warp's rows over the largest one, row 16 i + 2 warp
// + j at 2 i + j, as two fp16: of W16 twice the same (below 2^-24: 0), of H16 two factors,
// since a small one has to reach further, where its row's gradient is all that a column of dB
// has (down to 2^-32); kNoRow for a row to be ignored, whose codes may be NaN.
constexpr uint32_t kNoRow = 0x80008000u;

// (the first one at least 2^-8: times a code it is exact)
__device__ __forceinline__ uint32_t two_factors(float s)
{
    const float first = fmaxf(s, 0x1p-8f);
    const __half2 h = __floats2half2_rn(first, s / first);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Of W16: 2^e(s_b) f.
__device__ __forceinline__ void load_powers_b(uint32_t *powers, int row0, const LossParams &p, float f, int warp, int lane)
{
    const int row = row0 + (lane >> 1) * 16 + 2 * warp + (lane & 1);
    if (lane >= 16)
        return;
    const __half2 s = __float2half2_rn(row < p.N ? power(__ldg(p.scale_b + (p.rowwise ? row : 0))) * f : 0.0f);
    powers[lane] = *reinterpret_cast<const uint32_t *>(&s);
}

// Of H16: 2^(row_exponent - most) code_scale. (By exponents: s_a g may leave fp32's range.)
__device__ __forceinline__ void load_powers_a(uint32_t *powers, int row0, const LossParams &p, uint32_t most, int warp, int lane)
{
    const int row = row0 + (lane >> 1) * 16 + 2 * warp + (lane & 1);
    if (lane >= 16)
        return;
    uint32_t s = 0;
    if (row < p.M) {
        const uint32_t e = row_exponent(__ldg(p.scale_a + (p.rowwise ? row : 0)), __ldg(p.dloss + static_cast<long long>(row) * p.dloss_step));
        if (__ldg(p.target + row) == p.ignore)
            s = kNoRow;
        else if (e == kInfinite)
            s = 0x7E007E00u;           // NaN, as all of dB then
        else if (e != 0)
            s = two_factors(ldexpf(code_scale(p.a_type), static_cast<int>(e) - static_cast<int>(most)));
    }
    powers[lane] = s;
}

__device__ __forceinline__ void take_rows(uint2 (&codes)[8], const uint8_t *stage, int warp, int lane)
{
    const int c = lane & 15, r = 2 * warp + (lane >> 4);
    const uint8_t *from = stage + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        codes[i] = *reinterpret_cast<const uint2 *>(from + i * 2048);
}

template <bool E4M3, bool ROWS>
__device__ __forceinline__ void write_rows(const uint2 (&codes)[8], int count, __half *out, int row0, int rows, int k0, int K,
                                           const uint32_t *powers, int warp, int lane)
{
    const int j = lane >> 4, r = 2 * warp + j, k = k0 + (lane & 15) * 8;
    __half *to = out + static_cast<long long>(row0 + r) * K + k;
    // this lane's rows: 16 i < left (K is a multiple of 16)
    const int left = k < K ? min(count, rows - row0) - r : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (16 * i >= left)
            break;
        const uint32_t s = powers[2 * i + j];
        const __half2 both = *reinterpret_cast<const __half2 *>(&s);
        const __half2 s0 = ROWS ? __low2half2(both) : both, s1 = __high2half2(both);
        uint32_t o[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint16_t two = static_cast<uint16_t>((h < 2 ? codes[i].x : codes[i].y) >> (16 * (h & 1)));
            if constexpr (E4M3)
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[h]) : "h"(two));
            else
                asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(o[h]) : "h"(two));
            __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&o[h]), s0);
            if constexpr (ROWS)
                v = __hmul2(v, s1);
            o[h] = ROWS && s == kNoRow ? 0u : *reinterpret_cast<const uint32_t *>(&v);
        }
        __stcg(reinterpret_cast<uint4 *>(to + static_cast<long long>(16 * i) * K), make_uint4(o[0], o[1], o[2], o[3]));
    }
}

__device__ __forceinline__ float bias_at(const LossParams &p, int n)
{
    float v[1];
    fp8rows::load_param<1>(p.bias, p.bias_type, n, 0.0f, v);
    return v[0];
}

// Sums of 16 columns over a warp's 32 rows: v[i] is this lane's row at column i,
// the result column `lane & 15`'s sum. The lanes' halves are added, then each step
// adds the half of the columns that the other lane keeps.
__device__ __forceinline__ float sum_rows(float (&v)[16], int lane)
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
    }
    return v[0];
}

// z of N columns of a row from the accumulator: times the scales, plus the biases.
template <bool BIASED, int N>
__device__ __forceinline__ void logits(float (&v)[N], const float *scales, const float *biases, float row_scale)
{
    const uint64_t rs2 = ptx::f32x2(row_scale, row_scale);
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        const float4 s = *reinterpret_cast<const float4 *>(scales + k);
        const uint64_t s0 = ptx::mul_f32x2(rs2, ptx::f32x2(s.x, s.y)), s1 = ptx::mul_f32x2(rs2, ptx::f32x2(s.z, s.w));
        uint64_t z0 = ptx::f32x2(v[k], v[k + 1]), z1 = ptx::f32x2(v[k + 2], v[k + 3]);
        if constexpr (BIASED) {
            const float4 b = *reinterpret_cast<const float4 *>(biases + k);
            z0 = ptx::fma_f32x2(z0, s0, ptx::f32x2(b.x, b.y));
            z1 = ptx::fma_f32x2(z1, s1, ptx::f32x2(b.z, b.w));
        } else {
            z0 = ptx::mul_f32x2(z0, s0);
            z1 = ptx::mul_f32x2(z1, s1);
        }
        ptx::unpack_f32x2(z0, v[k], v[k + 1]);
        ptx::unpack_f32x2(z1, v[k + 2], v[k + 3]);
    }
}

// exp(z - off) of many z as 2^(z log2(e) - o) in one operation a value, with o = off
// log2(e) rounded; the rounding is taken off by a factor `rest` of the results, so that
// it does not show where their sum is close to 1. It is up to half a unit in the last place
// of o: 2^-4 at 2^20, where rest is within 5 % of 1, but hundreds from 2^31 on, which
// neither factor would hold. An off beyond 2^20 (columns ruled out by a finite value, as far
// as they are all that a sum has met) is `wild`: (z - off) log2(e), whose difference is
// exact where it counts.
struct Offset {
    uint64_t log2e2, add;              // wild: minus off, twice
    float rest;
    bool wild;
    static constexpr float kWild = 0x1p20f;
    __device__ __forceinline__ explicit Offset(float off)
    {
        const float o = off * kLog2e;
        wild = __any_sync(0xFFFFFFFFu, fabsf(off) > kWild);
        rest = wild ? 1.0f : fp8mm::ex2_approx(-fmaf(off, kLog2e, -o));
        add = wild ? ptx::f32x2(-off, -off) : ptx::f32x2(-o, -o);
        log2e2 = ptx::f32x2(kLog2e, kLog2e);
    }
    template <bool WILD>
    __device__ __forceinline__ void exponentials(float v0, float v1, float &e0, float &e1) const
    {
        const uint64_t v = ptx::f32x2(v0, v1);
        float lo, hi;
        if constexpr (WILD)
            ptx::unpack_f32x2(ptx::mul_f32x2(ptx::add_f32x2(v, add), log2e2), lo, hi);
        else
            ptx::unpack_f32x2(ptx::fma_f32x2(v, log2e2, add), lo, hi);
        e0 = fp8mm::ex2_approx(lo);
        e1 = fp8mm::ex2_approx(hi);
    }
    // v = exp(v - off) / rest
    template <int N>
    __device__ __forceinline__ void exponentials(float (&v)[N]) const
    {
        if (wild) {
#pragma unroll
            for (int k = 0; k < N; k += 2)
                exponentials<true>(v[k], v[k + 1], v[k], v[k + 1]);
        } else {
#pragma unroll
            for (int k = 0; k < N; k += 2)
                exponentials<false>(v[k], v[k + 1], v[k], v[k + 1]);
        }
    }
};

// How far a value may be above the maximum that a sum's terms are relative to: a new one
// for each block of 32 columns costs a tenth of its instructions.
constexpr float kAbove = 4.0f;

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// One warp's block of 32 rows into its swizzled stage: lane `row` writes the
// 16-byte chunk c of rows of 128 bytes, or of 64.
__device__ __forceinline__ void stage_chunk(uint8_t *stage, int lane, int c, uint4 w)
{
    *reinterpret_cast<uint4 *>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = w;
}
__device__ __forceinline__ void stage_chunk64(uint8_t *stage, int lane, int c, uint4 w)
{
    *reinterpret_cast<uint4 *>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) = w;
}

__device__ __forceinline__ uint4 pack8(const float *v, int type)
{
    return make_uint4(fp8rows::pack2(v[0], v[1], type), fp8rows::pack2(v[2], v[3], type),
                      fp8rows::pack2(v[4], v[5], type), fp8rows::pack2(v[6], v[7], type));
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<KIND>::kThreads, 1)
    loss_kernel(const __grid_constant__ AllMaps<KIND> maps, const __grid_constant__ LossParams p)
{
    using C = Cfg<KIND>;
    constexpr int S = C::kStages;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    const uint32_t sbase = raw + pad;
    constexpr int kStagingAt = S * C::kStageBytes, kColsAt = kStagingAt + C::kStagingBytes;
    constexpr int kPowersAt = kColsAt + C::kColBytes, kNormsAt = kPowersAt + C::kPowerBytes;
    constexpr int kBarsAt = kNormsAt + C::kNormBytes;
    uint32_t *shared_norms = reinterpret_cast<uint32_t *>(smem + kNormsAt);
    const uint32_t bar0 = sbase + kBarsAt;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
    const uint32_t done_bar = bar0 + 8u * (2 * S + 4);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kBarsAt + 8 * (2 * S + 5));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // kSlope: the MMA is done with a stage that is to be converted; warps that have it
    auto used_bar = [&](int s) { return bar0 + 8u * (2 * S + 6 + s); };
    int *taken = reinterpret_cast<int *>(smem + kBarsAt + 8 * (3 * S + 6));
    static_assert(8 * (3 * S + 6) + 4 * S <= 256, "barrier area");

    // (known to be the same in a warp's lanes: what follows from it is computed once a warp;
    // kGrad 88 to 57 registers, 300 x 50257 x 4112 gradients 436 to 433 us, 2048 x 2048 x 512 23.1 to 22.4)
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            // (one arrival: the MMA's, or of a converted stage the last warp's that took it)
            ptx::mbar_init(empty_bar(s), 1);
            ptx::mbar_init(used_bar(s), 1);
            taken[s] = 0;
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(tfull_bar(a), 1);
            ptx::mbar_init(tempty_bar(a), 2 * kEpiWarps);
        }
        ptx::mbar_init(done_bar, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        for (const Maps &m : maps.of) {
            ptx::prefetch_tmap(&m.a);
            ptx::prefetch_tmap(&m.b);
            if constexpr (KIND != kStats)
                ptx::prefetch_tmap(&m.out);
        }
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), 2 * kTile);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    // no global memory before this
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();

    const Waiter W{abort_flag, p.status, p.timeout_cycles};

    if (warp == 0) {
        // ------------------------------------------------ TMA producer ---
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int issued = 0;
            bool ok = true;
            Schedule<KIND> tiles(p, pair, pairs);
            Work w;
            while (ok && tiles.next(w)) {
                const TileSpace &t = p.t[KIND == kGrad ? w.of : 0];
                const Maps &m = maps.of[KIND == kGrad ? w.of : 0];
                const int row = (2 * w.tp + static_cast<int>(rank)) * t.half;
                const int col = w.tq * t.width + static_cast<int>(rank) * (t.width / 2);
                const uint32_t bytes = 128u * static_cast<uint32_t>(2 * t.half + t.width);
                // (kGrad's two products in loops of their own: chosen within one, an
                // iteration took 10 % longer than the MMAs)
                auto load = [&](auto mn_major) {
                    for (int kb = w.kb0; kb < w.kb1; ++kb) {
                        if (!W.wait(empty_bar(stage), phase ^ 1u, 0)) {
                            ok = false;
                            break;
                        }
                        const uint32_t sa = sbase + stage * C::kStageBytes, sb = sa + C::kABytes;
                        const uint32_t full = ptx::mapa_shared(full_bar(stage), 0);
                        if (rank == 0)
                            ptx::mbar_arrive_expect_tx(full_bar(stage), bytes);
                        const int k = kb * (C::kFp8 ? 128 : 64);
                        if constexpr (decltype(mn_major)::value) {
                            ptx::tma_load_3d_pair(sa, &m.a, full, row, k, 0);
                            ptx::tma_load_3d_pair(sa + 8192, &m.a, full, row + 64, k, 0);
                        } else {
                            ptx::tma_load_3d_pair(sa, &m.a, full, k, row, 0);
                        }
                        if constexpr (KIND == kGrad) {
                            ptx::tma_load_3d_pair(sb, &m.b, full, col, k, 0);
                            ptx::tma_load_3d_pair(sb + 8192, &m.b, full, col + 64, k, 0);
                        } else {
                            ptx::tma_load_3d_pair(sb, &m.b, full, k, col, 0);
                        }
                        ++issued;
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                };
                if (KIND == kGrad && w.of == kOfB)
                    load(std::integral_constant<bool, KIND == kGrad>{});
                else
                    load(std::false_type{});
            }
            // this CTA's copies land before it may exit (the even CTA sees both
            // CTAs' bytes; the odd one waits until its stages were consumed)
            const int n = issued < S ? issued : S;
            int s = stage;
            uint32_t ph = phase;
            for (int i = 0; i < n; ++i) {
                if (--s < 0) {
                    s = S - 1;
                    ph ^= 1u;
                }
                if (rank == 0)
                    W.drain(full_bar(s), ph, 3);
                else
                    W.drain(empty_bar(s), ph, 6);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------- pair MMA (even CTA only) ---
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool ok = true;
            Schedule<KIND> tiles(p, pair, pairs);
            Work w;
            while (ok && tiles.next(w)) {
                const uint32_t idesc = p.t[KIND == kGrad ? w.of : 0].idesc;
                if (!W.wait_cluster(tempty_bar(acc), acc_phase ^ 1u, 1))
                    break;
                ptx::tc_fence_after();
                const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kTile);
                Converted next(p, w);
                auto multiply = [&](auto mn_major) {
                    for (int kb = w.kb0; kb < w.kb1; ++kb) {
                        if (!W.wait(full_bar(stage), phase, 2)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        const uint32_t sa = sbase + stage * C::kStageBytes, sb = sa + C::kABytes;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t more = (kb > w.kb0 || k > 0) ? 1u : 0u;
                            if constexpr (KIND == kGrad) {
                                const uint64_t da = decltype(mn_major)::value ? ptx::sw128_mnmajor_desc(sa + k * 2048) : ptx::sw128_kmajor_desc(sa + k * 32);
                                ptx::mma_f16_pair(d, da, ptx::sw128_mnmajor_desc(sb + k * 2048), idesc, more);
                            } else {
                                ptx::mma_e4m3_pair(d, ptx::sw128_kmajor_desc(sa + k * 32), ptx::sw128_kmajor_desc(sb + k * 32), idesc, more);
                            }
                        }
                        const bool keep = KIND == kSlope && next.has(kb);
                        ptx::mma_commit_pair_multicast(keep ? used_bar(stage) : empty_bar(stage), 0x3);
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                };
                if (KIND == kGrad && w.of == kOfB)
                    multiply(std::integral_constant<bool, KIND == kGrad>{});
                else
                    multiply(std::false_type{});
                if (!ok)
                    break;
                ptx::mma_commit_pair_multicast(tfull_bar(acc), 0x3);
                if (++acc == 2) {
                    acc = 0;
                    acc_phase ^= 1u;
                }
            }
            ptx::mma_commit_pair_multicast(done_bar, 0x1);
            W.drain(done_bar, 0, 4);
        }
        __syncwarp();
    } else if (KIND == kSlope && warp >= 2 + kEpiWarps) {
        // ------------------------------------------- codes to fp16 ---
        // From the stages, once the MMA is done with them. (By a kernel of its own, early
        // and beside this one: 620 MB more of memory traffic at 300 x 50257 x 4112, 220 us
        // for the two against 150.) The last warp that has its codes gives the stage back;
        // taken[s] is 0 again before the stage can come round.
        const int cw = warp - 2 - kEpiWarps;
        uint32_t most_h, most_b;
        if (p.norms_out) {
            const int thread = cw * 32 + lane;
            most_h = shared_norm<32 * kConvertWarps>(p.M, thread, shared_norms, 1, [&](int i) {
                const uint32_t e = row_exponent(__ldg(p.scale_a + (p.rowwise ? i : 0)), __ldg(p.dloss + i * p.dloss_step));
                return __ldg(p.target + i) == p.ignore ? 0u : e;
            });
            most_b = shared_norm<32 * kConvertWarps>(p.rowwise ? p.N : 1, thread, shared_norms + 16, 1,
                                                     [&](int i) { return __float_as_uint(__ldg(p.scale_b + i)) & 0x7FFFFFFFu; });
            if (blockIdx.x == 0 && cw == 0) {
                p.norms_out[kNormH * kNormParts + lane] = most_h;
                p.norms_out[kNormB * kNormParts + lane] = most_b;
            }
        } else {
            most_h = norm_most(p.norms, kNormH);
            most_b = norm_most(p.norms, kNormB);
        }
        const float fb = code_scale(p.b_type) / norm_power(most_b);
        const TileSpace &t = p.t[0];
        uint32_t *powers = reinterpret_cast<uint32_t *>(smem + kPowersAt) + cw * 32;
        int stage = 0;
        uint32_t used = 0;             // bit s: parity of the next use of stage s that converts
        bool ok = true;
        Schedule<KIND> tiles(p, pair, pairs);
        Work w;
        while (ok && tiles.next(w)) {
            const int row = (2 * w.tp + static_cast<int>(rank)) * t.half;
            const int col = w.tq * t.width + static_cast<int>(rank) * (t.width / 2);
            __syncwarp();
            if (p.h16)
                load_powers_a(powers, row, p, most_h, cw, lane);
            if (p.w16)
                load_powers_b(powers + 16, col, p, fb, cw, lane);
            __syncwarp();
            Converted next(p, w);
            for (int kb = w.kb0; kb < w.kb1; ++kb) {
                const int s = stage;
                if (++stage == S)
                    stage = 0;
                if (!next.has(kb))
                    continue;
                if (!W.wait(used_bar(s), (used >> s) & 1u, 7)) {
                    ok = false;
                    break;
                }
                used ^= 1u << s;
                const uint8_t *at = smem + s * C::kStageBytes;
                uint2 a[8], b[8];
                if (next.of_a)
                    take_rows(a, at, cw, lane);
                if (next.of_b)
                    take_rows(b, at + C::kABytes, cw, lane);
                __syncwarp();
                // (the others' reads before the last one's arrival)
                if (lane == 0 && ptx::shared_inc_acq_rel(ptx::smem_addr(taken + s)) == kConvertWarps - 1) {
                    taken[s] = 0;
                    ptx::mbar_arrive(empty_bar(s));
                }
                if (next.of_a) {
                    if (p.a_type == 0)
                        write_rows<true, true>(a, t.half, p.h16, row, p.M, kb * 128, p.K, powers, cw, lane);
                    else
                        write_rows<false, true>(a, t.half, p.h16, row, p.M, kb * 128, p.K, powers, cw, lane);
                }
                if (next.of_b) {
                    if (p.b_type == 0)
                        write_rows<true, false>(b, t.width / 2, p.w16, col, p.N, kb * 128, p.K, powers + 16, cw, lane);
                    else
                        write_rows<false, false>(b, t.width / 2, p.w16, col, p.N, kb * 128, p.K, powers + 16, cw, lane);
                }
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- epilogue ---
        // Warp (q, part) takes the rows 32 q.. and the columns 64 part.. of the
        // tile, in blocks of 32. (With two warps per 32 rows, of 128 columns each,
        // a tile took 3.6 us whatever it did, K = 512: too few to cover their own
        // latencies.)
        const int q = warp & 3, ew = warp - 2, part = ew / 4;
        uint8_t *stage = smem + kStagingAt + ew * C::kBlockBytes;
        const uint32_t stage_smem = sbase + kStagingAt + ew * C::kBlockBytes;
        float *col_scale = reinterpret_cast<float *>(smem + kColsAt) + ew * C::kCols * C::kColFloats;
        float *col_bias = col_scale + C::kCols, *col_mantissa = col_bias + C::kCols;
        int acc = 0;
        uint32_t acc_phase = 0;
        float norm_g = 1.0f, out_scale[2] = {1.0f, 1.0f};
        if constexpr (KIND == kSlope) {
            if (p.norms_out) {
                const uint32_t g = shared_norm<32 * kEpiWarps>(p.M, ew * 32 + lane, shared_norms + 32, 2, [&](int i) {
                    const uint32_t v = __float_as_uint(__ldg(p.dloss + i * p.dloss_step)) & 0x7FFFFFFFu;
                    return __ldg(p.target + i) == p.ignore ? 0u : v;
                });
                if (blockIdx.x == 0 && ew == 0)
                    p.norms_out[kNormG * kNormParts + lane] = g;
                norm_g = norm_power(g);
            } else {
                norm_g = norm_scale(p.norms, kNormG);
            }
        }
        if constexpr (KIND == kGrad) {
            norm_g = norm_scale(p.norms, kNormG);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (p.r[i].scaled)
                    out_scale[i] = result_scale(p.norms, p.r[i].norm_of, p.r[i].factor);
        }
        const float s_tensor = C::kFp8 && !p.rowwise ? __ldg(p.scale_a) * __ldg(p.scale_b) : 1.0f;
        const float ma_tensor = C::kFp8 && !p.rowwise ? mantissa(__ldg(p.scale_a)) : 1.0f;
        const float mb_tensor = C::kFp8 && !p.rowwise ? mantissa(__ldg(p.scale_b)) : 1.0f;

        // the block's place is free, and a block goes out
        auto stage_free = [&]() {
            if (lane == 0)
                ptx::bulk_wait_group_read<0>();
            __syncwarp();
        };
        auto stage_out = [&](const CUtensorMap *out, bool add, int x, int y, int z, int x_end, int y_end) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && x < x_end && y < y_end) {
                if (KIND == kGrad && add)
                    ptx::tma_add_3d(out, stage_smem, x, y, z);
                else
                    ptx::tma_store_3d(out, stage_smem, x, y, z);
                ptx::bulk_commit_group();
            }
        };

        // what this lane knows of its row of A: scale, lse, g, where its target is
        // (`back`: dz' without its columns' mantissas to dz / G)
        float rs = 1.0f, lse = 0.0f, gs = 0.0f, back = 1.0f, row_factor = 1.0f;
        long long at = -1;                       // (in the piece; -1: none in it)
        bool live = false;
        // of the row in this unit so far: sum of exp(z - top); top is a maximum, which later
        // values exceed by kAbove at most
        float top = -INFINITY, sum = 0.0f;
        Offset from(0.0f);
        Schedule<KIND> tiles(p, pair, pairs);
        Work w{}, ahead{};
        // the columns' scales and biases of a tile, loaded while the one before it is
        // worked on
        float next_scale[2] = {}, next_bias[2] = {};
        auto load_columns = [&]() {
            const int first = ahead.tq * p.t[0].width + part * 64;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // columns past the end: z = -inf, which adds nothing
                const int n = first + i * 32 + lane;
                const bool there = n < p.N;
                next_scale[i] = there ? (p.rowwise ? __ldg(p.scale_b + n) : s_tensor) : 0.0f;
                next_bias[i] = there ? bias_at(p, n) : -INFINITY;
            }
        };
        bool more = tiles.next(ahead);
        if (C::kFp8 && more)
            load_columns();
        while (more) {
            w = ahead;                 // (next() goes on from the tile it gave)
            const TileSpace &t = p.t[KIND == kGrad ? w.of : 0];
            const Maps &m = maps.of[KIND == kGrad ? w.of : 0];
            const int row0 = (2 * w.tp + static_cast<int>(rank)) * t.half + q * 32, row = row0 + lane;
            const int col0 = w.tq * t.width + part * 64;
            // (a narrow tile's last warps have one block or none)
            const int blocks = q * 32 >= t.half ? 0 : min(2, (min(t.width, t.cols - w.tq * t.width) - part * 64 + 31) / 32);
            // what the tile needs beside the accumulator, while the MMAs run
            const bool biased = p.bias || col0 + 64 > t.cols;
            if constexpr (C::kFp8) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    col_scale[i * 32 + lane] = next_scale[i];
                    col_bias[i * 32 + lane] = next_bias[i];
                    if constexpr (KIND == kSlope)
                        col_mantissa[i * 32 + lane] = p.rowwise ? mantissa(next_scale[i]) : mb_tensor;
                }
                __syncwarp();
            }
            more = tiles.next(ahead);
            if (C::kFp8 && more)
                load_columns();
            if constexpr (C::kFp8) {
                if (w.first) {
                    // this row of A
                    rs = 1.0f;
                    gs = 0.0f;
                    back = 1.0f;           // (of rows without a dz)
                    at = -1;
                    live = false;
                    top = -INFINITY;       // (and `from` anew with the first finite value)
                    sum = 0.0f;
                    if (row < p.M) {
                        if (p.rowwise)
                            rs = __ldg(p.scale_a + row);
                        const long long to = __ldg(p.target + row);
                        live = to != p.ignore;
                        if (live && to >= 0 && to < p.vocabulary)
                            at = to - p.col0;
                        if constexpr (KIND == kSlope) {
                            // (an ignored row's may be anything, and the warp's rows go one way)
                            lse = live ? __ldg(p.lse + row) : 0.0f;
                            const float g = __ldg(p.dloss + static_cast<long long>(row) * p.dloss_step);
                            const float ma = p.rowwise ? mantissa(rs) : ma_tensor, pg = row_power(g);
                            gs = g * (kSlopeScale / pg) * ma;
                            if (live)
                                back = pg / norm_g / ma;
                            if (live && (to < 0 || to >= p.vocabulary))
                                gs = NAN;
                        }
                    }
                }
            } else {
                row_factor = w.of == kOfB ? out_scale[1] : out_scale[0];
                if (row < t.rows) {
                    row_factor /= mantissa(__ldg(p.r[w.of].row_scale + (p.rowwise ? row : 0)));
                    // (dz' of a row to be ignored is zero)
                    if (w.of == kOfA && __ldg(p.target + row) != p.ignore)
                        row_factor *= row_power(__ldg(p.dloss + static_cast<long long>(row) * p.dloss_step)) / norm_g;
                }
            }
            if (!W.wait(tfull_bar(acc), acc_phase, 5))
                break;
            ptx::tc_fence_after();
            const uint32_t trow = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kTile + part * 64);
            // the accumulator is the MMA's again as soon as this warp's last block of it is
            // in registers
            bool given_back = false;
            auto give_back = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive_cluster_relaxed(ptx::mapa_shared(tempty_bar(acc), 0));
                given_back = true;
            };

            if constexpr (C::kFp8) {
                const Offset off(lse);           // (kSlope)
                const float gs_rest = gs * off.rest;
#pragma unroll 1
                for (int i = 0; i < blocks; ++i) {
                    const int n0 = col0 + i * 32;
                    const float *scales = col_scale + i * 32, *biases = col_bias + i * 32, *mantissas = col_mantissa + i * 32;
                    const bool mine = at >= n0 && at < n0 + 32;
                    if constexpr (KIND == kStats) {
                        float v[32];
                        ptx::tmem_ld_32cols(trow + i * 32, v);
                        if (i + 1 == blocks)
                            give_back();
                        if (biased)
                            logits<true>(v, scales, biases, rs);
                        else
                            logits<false>(v, scales, biases, rs);
                        // (where the row has an infinite code or scale, a column past the end is
                        // infinity times zero until here)
                        if (n0 + 32 > t.cols) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = n0 + k < t.cols ? v[k] : -INFINITY;
                        }
                        if (mine) {
                            float zt = 0.0f;
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                zt = at == n0 + k ? v[k] : zt;
                            p.target_z[row] = zt;
                        }
                        float most = -INFINITY, most2 = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            most = max3(most, v[k], v[k + 1]);
                            most2 = max3(most2, v[k + 2], v[k + 3]);
                        }
                        most = fmaxf(most, most2);
                        if (__any_sync(0xFFFFFFFFu, most > top + kAbove)) {
                            // (a row without a finite value so far: exp(-inf - 0) = 0)
                            const float old = top;
                            top = fmaxf(top, most);
                            const float ref = top == -INFINITY ? 0.0f : top;
                            sum *= fp8mm::ex2_approx((old - ref) * kLog2e);
                            from = Offset(ref);
                        }
                        from.exponentials(v);
                        uint64_t s2[2] = {0, 0};
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            s2[k & 1] = ptx::add_f32x2(s2[k & 1], ptx::f32x2(v[2 * k], v[2 * k + 1]));
                        float s0, s1;
                        ptx::unpack_f32x2(ptx::add_f32x2(s2[0], s2[1]), s0, s1);
                        sum = fmaf(s0 + s1, from.rest, sum);
                    } else {
                        // 16 columns at a time: 26 warps have 72 registers each
#pragma unroll 1
                        for (int j = 0; j < 2; ++j) {
                            float v[16];
                            ptx::tmem_ld_16cols(trow + i * 32 + j * 16, v);
                            if (j == 1 && i + 1 == blocks)
                                give_back();
                            if (biased)
                                logits<true>(v, scales + j * 16, biases + j * 16, rs);
                            else
                                logits<false>(v, scales + j * 16, biases + j * 16, rs);
                            off.exponentials(v);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                v[k] = live ? v[k] * gs_rest : 0.0f;
                            if (mine) {
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    v[k] = at == n0 + j * 16 + k ? v[k] - gs : v[k];
                            }
                            if (j == 0)
                                stage_free();
#pragma unroll
                            for (int k = 0; k < 16; k += 8) {
                                const float4 x = *reinterpret_cast<const float4 *>(mantissas + j * 16 + k);
                                const float4 y = *reinterpret_cast<const float4 *>(mantissas + j * 16 + k + 4);
                                const float o[8] = {v[k] * x.x, v[k + 1] * x.y, v[k + 2] * x.z, v[k + 3] * x.w,
                                                    v[k + 4] * y.x, v[k + 5] * y.y, v[k + 6] * y.z, v[k + 7] * y.w};
                                stage_chunk64(stage, lane, j * 2 + k / 8, pack8(o, fp8rows::kF16));
                            }
                            if (p.colsum) {
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    v[k] *= back;
                                const float s = sum_rows(v, lane);
                                const int n = n0 + j * 16 + lane;
                                if (row0 < p.M && lane < 16 && n < p.N)
                                    __stcg(p.colsum + (row0 / 32) * p.colsum_ld + n, s);
                            }
                        }
                        stage_out(&m.out, false, n0, row0, 0, p.N, p.M);
                    }
                }
                if constexpr (KIND == kStats) {
                    if (w.last && row < p.M && q * 32 < t.half)
                        __stcg(p.stats + static_cast<long long>(w.unit_q * 4 + part) * p.M + row, make_float2(top, sum));
                }
            } else {
                const Result &r = p.r[w.of];
                const bool f32 = r.out_type == fp8mm::kOutF32;
                // 32 columns of fp32 make a block, 64 of 16 bits
#pragma unroll 1
                for (int i = 0; i < 2 && q * 32 < t.half; ++i) {
                    float v[32];
                    ptx::tmem_ld_32cols(trow + i * 32, v);
                    if (i == 1)
                        give_back();
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        v[k] *= row_factor;
                    if (f32 || i == 0)
                        stage_free();
                    if (f32) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            stage_chunk(stage, lane, k / 4,
                                        make_uint4(__float_as_uint(v[k]), __float_as_uint(v[k + 1]),
                                                   __float_as_uint(v[k + 2]), __float_as_uint(v[k + 3])));
                        stage_out(&m.out, r.add, col0 + i * 32, row0, w.split, t.cols, t.rows);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
                            stage_chunk(stage, lane, i * 4 + k / 8, pack8(v + k, r.out_type));
                        if (i == 1)
                            stage_out(&m.out, r.add, col0, row0, w.split, t.cols, t.rows);
                    }
                }
            }
            if (!given_back)
                give_back();
            if (++acc == 2) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        if (KIND != kStats && lane == 0)
            ptx::bulk_wait_group_all();
        __syncwarp();
    }

    ptx::tc_fence_before();
    ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, 2 * kTile);
    }
}

// ---------------------------------------------------------------- combine ---
// lse and loss from a row's parts (top, sum): most = max top, the sum of sum exp(top -
// most). Always in the same order for the same sizes.

struct CombineParams {
    const float2 *stats;
    const float *target_z;
    const int64_t *target;
    long long ignore, vocabulary;
    float *loss, *lse;
    int rows, parts;
};

// (without a finite value the reference is 0)
__device__ __forceinline__ float reference(float most) { return most == -INFINITY ? 0.0f : most; }

__device__ __forceinline__ void join(float &top, float &sum, float2 b)
{
    const float most = fmaxf(top, b.x), ref = reference(most);
    sum = sum * fp8mm::ex2_approx((top - ref) * kLog2e) + b.y * fp8mm::ex2_approx((b.x - ref) * kLog2e);
    top = most;
}

__device__ __forceinline__ void finish_row(const CombineParams &p, int row, float top, float sum)
{
    const float rest = logf(sum);
    p.lse[row] = top + rest;
    const long long t = p.target[row];
    float loss = 0.0f;
    if (t != p.ignore)
        loss = t >= 0 && t < p.vocabulary ? (top - p.target_z[row]) + rest : NAN;
    p.loss[row] = loss;
}

// 32 rows a CTA, a lane each: warp w joins the parts w, w + 32, ..., the first warp the
// 32 results of a row.
constexpr int kCombineThreads = 1024;

static __global__ void __launch_bounds__(kCombineThreads) combine_kernel(const CombineParams p)
{
    __shared__ float2 part[32][33];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x * 32 + lane;
    float top = -INFINITY, sum = 0.0f;
    if (row < p.rows) {
#pragma unroll 4
        for (int i = warp; i < p.parts; i += 32)
            join(top, sum, __ldcg(p.stats + static_cast<long long>(i) * p.rows + row));
    }
    part[warp][lane] = make_float2(top, sum);
    __syncthreads();
    if (warp != 0 || row >= p.rows)
        return;
    for (int i = 1; i < 32; ++i)
        join(top, sum, part[i][lane]);
    finish_row(p, row, top, sum);
}

// A CTA to a row, for few of them: a thread joins the parts t, t + 256, ..., a warp's and
// the CTA's are added as terms of their common maximum. (One row of 572 parts: 1.5 us
// for 4.5.)
constexpr int kRowThreads = 256;

static __global__ void __launch_bounds__(kRowThreads) combine_row_kernel(const CombineParams p)
{
    __shared__ float tops[kRowThreads / 32], sums[kRowThreads / 32];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x;
    float top = -INFINITY, sum = 0.0f;
#pragma unroll 2
    for (int i = threadIdx.x; i < p.parts; i += kRowThreads)
        join(top, sum, __ldcg(p.stats + static_cast<long long>(i) * p.rows + row));
    float most = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    sum *= fp8mm::ex2_approx((top - reference(most)) * kLog2e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) {
        tops[warp] = most;
        sums[warp] = sum;
    }
    __syncthreads();
    if (threadIdx.x != 0)
        return;
    for (int i = 1; i < kRowThreads / 32; ++i)
        join(most, sum, make_float2(tops[i], sums[i]));
    finish_row(p, row, most, sum);
}

// ------------------------------------------------------- sums of partials ---
// A result from its fp32 partials: out = cast( result_scale sum over s of part[s] ).

struct FinishParams {
    const float *parts;
    long long n;                       // elements of one partial, a multiple of 4
    int count, out_type, norm_of;
    const uint32_t *norms;
    float factor;
    void *out;
};

constexpr int kFinishThreads = 256;

__device__ __forceinline__ void add4(float4 &s, float4 v)
{
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
}

// SPLIT 1: a thread adds all partials of 4 elements. SPLIT 8: a warp adds every
// eighth one, the first warp the eight sums; for few elements of many partials, whose loads
// one thread would wait for in turn (the gradients of 128 x 4096 x 480, 17.2 to 16.7 us).
template <int SPLIT>
static __global__ void __launch_bounds__(kFinishThreads) finish_kernel(const FinishParams p)
{
    __shared__ float4 part[SPLIT][32];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const float f = result_scale(p.norms, p.norm_of, p.factor);
    constexpr int kWide = kFinishThreads / SPLIT;
    const int at = SPLIT == 1 ? threadIdx.x : threadIdx.x & 31, first = SPLIT == 1 ? 0 : threadIdx.x >> 5;
    const long long step = static_cast<long long>(gridDim.x) * kWide, end = p.n / 4;
    for (long long base = static_cast<long long>(blockIdx.x) * kWide; base < end; base += step) {
        const long long i = base + at;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < end) {
#pragma unroll 4
            for (int k = first; k < p.count; k += SPLIT)
                add4(s, __ldcg(reinterpret_cast<const float4 *>(p.parts + k * p.n) + i));
        }
        if constexpr (SPLIT > 1) {
            part[first][at] = s;
            __syncthreads();
            if (first == 0) {
#pragma unroll
                for (int w = 1; w < SPLIT; ++w)
                    add4(s, part[w][at]);
            }
            __syncthreads();
        }
        if (first != 0 || i >= end)
            continue;
        if (p.out_type == fp8mm::kOutF32)
            reinterpret_cast<float4 *>(p.out)[i] = make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
        else
            reinterpret_cast<uint2 *>(p.out)[i] = make_uint2(fp8rows::pack2(s.x * f, s.y * f, p.out_type),
                                                             fp8rows::pack2(s.z * f, s.w * f, p.out_type));
    }
}

// dbias of a piece: out[c] = f sum over p < count of part[p][c], warp w adding
// parts w, w + 8, ... of 32 columns.
struct ColumnsParams {
    const float *parts;
    long long ld;
    int cols, count;
    const uint32_t *norms;
    float *out;
};

constexpr int kColumnsThreads = 256;

static __global__ void __launch_bounds__(kColumnsThreads) columns_kernel(const ColumnsParams p)
{
    __shared__ float part[8][33];
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const float f = norm_scale(p.norms, kNormG) / kSlopeScale;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
        for (int i = warp; i < p.count; i += 8)
            s += __ldcg(p.parts + i * p.ld + c);
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < p.cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            s += part[i][lane];
        p.out[c] = s * f;
    }
}

}  // namespace fp8loss
