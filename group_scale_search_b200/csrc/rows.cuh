// Products with the packed records over any number of token rows: what the
// host entry points (rows.cu) and the kernels compiled per format
// (rows_*.cu, rows_core.cuh) share.  Not part of the C ABI.
#pragma once

#include <cuda.h>

#include "tq_internal.cuh"

namespace tq {

// What the forward kernel does with a finished tile of products.
enum RowsMode {
    ROWS_STORE = 0,      // y = z
    ROWS_GATED = 1,      // h = act(g) u
    ROWS_GATED_BWD = 2,  // D = (dh u act'(g), dh act(g)), f16, scaled by a power of two per token
    ROWS_LOSS = 3,       // per token and tile: max z, sum exp(z - max); the label's z
    ROWS_PROB = 4        // D = exp(z - lse) - [o = label], f16, times 2^13
};

// Of ROWS_PROB's D: probabilities keep 11 bits down to 2^-27 and vanish below
// 2^-38; they may be up to 8, since a logit computed by another kernel than the
// lse's may be above it where logits are so large that fp32 holds them to one or
// two only.
constexpr float ROWS_PROB_SCALE = 8192.f;
// Partial maxima of a matrix's values: enough blocks for one matrix, few of each
// where there are many.
__host__ __device__ __forceinline__ int rows_wmax_parts(int E) { return E <= 2 ? 64 : E >= 32 ? 4 : 128 / E; }
constexpr int ROWS_MAX_MATS = 1024;

struct RowsArgs {
    // the records: [0] the weight, or the gate projection and [1] the up projection
    const uint8_t* packed[2];
    const void* scales[2];
    const uint8_t* zeros[2];
    const float* gs[2];
    int64_t O, I, G, rowbytes;      // rows and columns of a matrix, groups and record bytes of a row
    int64_t o_begin, o_end;         // the weight rows of this launch
    int64_t R;                      // token rows
    const int32_t* offsets;         // [E + 1], or null: one matrix, rows 0 .. R - 1
    int E;
    int m_tiles;                    // tiles (or pairs of them) along the output: weight rows or, backward, columns
    int nk;                         // 64-wide steps (forward: columns; backward: weight rows of one projection)
    int projections;                // 1, or 2 for gate and up
    int splits;                     // backward: parts of the sum over weight rows
    int mode, act;
    unsigned wait_limit;
    // outputs and the rest of the inputs
    void* y;                        // forward: y or h; backward: dx (bf16)
    int64_t ldy;
    int y_bf16;
    const uint16_t* dh;             // bf16 [R][ld_dh]
    int64_t ld_dh;
    uint16_t* D;                    // f16 [projections][R][ldd]
    int64_t ldd;
    const float* row_f;             // [R]: gated backward |dh|max |x|2; matmul backward 2^c; loss backward dloss
    const float* row_x;             // [R]: forward: the power of two beside a token's f16 values
    const float* wmax;              // [projections][E][rows_wmax_parts(E)]: parts of a matrix's largest value (rows_wmax)
    const int64_t* labels;
    const float* lse;
    const uint16_t* x_few;          // few tokens: f16 in the kernel's order, [R][slices of 128 columns][256 bytes]
    const float* x_sums;            // integer formats: 2^-10 times the values' sum per group, [R][slices][groups of one]
    int few;                        // (host) blocks of 8 tokens that its kernel takes at a time, 0: not its call
    int few_wide, few_ks;
    float2* part;                   // ROWS_LOSS: [part_tiles][R]
    int part_tiles;
    float* label_z;                 // [R]
    float* sums;                    // backward: fp32 [splits][R][I], or null (dx written directly)
    int sums_add;                   // backward: add to sums (a later piece of the vocabulary)
};

// How the kernel holds its operands (rows_core.cuh).
enum RowsKind { ROWS_EXACT = 0, ROWS_GRAD = 1, ROWS_SCALED = 2 };

// The column (from a multiple of 16) at place p of an operand row.
__host__ __device__ __forceinline__ int rows_column(int fmt, int p) {
    if (is_int4(fmt)) return (p & ~7) + ((p & 7) >> 1) + 4 * (p & 1);
    if (fmt == TQ_INT3_G64_SYM) return (p & ~15) + ((p & 15) >> 1) + 8 * (p & 1);
    return p;
}

// Whether tiles of nt tokens are shared by two CTAs: with 256 tokens the gated
// 2048-row case took 651 us so, 688 with a CTA to a tile, the loss 720 and 742
// (at 64 tokens and below the weights' half of a stage, which is not shared, is
// most of it, and one CTA alone leaves more tiles to spread over the SMs).
__host__ __device__ constexpr bool rows_pair(int nt) { return nt >= 128; }

// Tokens per tile that the launch should use: 32, 64, 128 or 256.
struct RowsLaunch {
    const CUtensorMap* map;
    int nt;
    int kind;
    int grid;
};

tq_status launch_rows_int3(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st);
tq_status launch_rows_int4g128(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st);
tq_status launch_rows_int4g64(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st);
tq_status launch_rows_int4g32(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st);
tq_status launch_rows_nvfp4(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st);

// The kernel for few tokens per matrix (rows_few.cuh): nb = 1, 2 or 4 blocks
// of 8 tokens at a time; a.m_tiles counts 32 (gated: 16) weight rows.
// nb, mb: see few_blocks_per_sm.
tq_status launch_few_int3(const RowsArgs& a, int nb, int mb, int grid, cudaStream_t st);
tq_status launch_few_int4g128(const RowsArgs& a, int nb, int mb, int grid, cudaStream_t st);
tq_status launch_few_int4g64(const RowsArgs& a, int nb, int mb, int grid, cudaStream_t st);
tq_status launch_few_int4g32(const RowsArgs& a, int nb, int mb, int grid, cudaStream_t st);
tq_status launch_few_nvfp4(const RowsArgs& a, int nb, int mb, int grid, cudaStream_t st);

// Blocks per SM of that kernel, two of which leave a thread 128 registers, one
// 255.  8 tokens: two (int4 g32 spills 216 bytes a thread for it, the others
// none).  16: two where a slice is one group (int4 g128, 104 bytes) or needs no
// group sums (NVFP4, 16 bytes), unless the grid fills no more than one (17408 x
// 5120 int4 g128, 14 rows: 45 us against 53; 4096 x 4096, 16 rows: 13 us with
// one, 17 with two); the other formats take one (11008 x 4096 int4 g64, 12 rows:
// 29 us against 42).  32: one (24 bytes of g32, 36 of g64).
__host__ __device__ constexpr bool few_two_fit(int fmt) { return fmt == TQ_INT4_G128_ASYM || fmt == TQ_NVFP4_G16; }
inline int few_blocks_per_sm(int fmt, int nb, int64_t items, int64_t sms) {
    return nb == 1 ? 2 : nb == 2 && few_two_fit(fmt) && items > sms ? 2 : 1;
}

// The order in which that kernel takes a 128-column slice: lane tig of the
// fragment layouts owns 16 pairs of columns, pair p of them
//   int4 g128   32 tig + 8 (p / 4) + p % 4             and 4 on
//   int4 g64    64 (p / 8) + 16 tig + 8 (p / 4 % 2) + p % 4   and 4 on
//   int4 g32    32 (p / 4) + 8 tig + p % 4              and 4 on
//   int3        64 (p / 8) + 16 tig + p % 8             and 8 on
//   NVFP4       32 tig + 2 p                            and 1 on
// (codes m and m + 4 of a word of int4 codes, i and i + 8 of 16 int3 codes,
// the two of a byte of NVFP4 codes).  A row of x_few is [slice][quarter p / 4]
// [tig][p % 4] pairs, the values scaled by 2^-few_field(p).
//
// few_field: the lowest bit of pair p's code field as it is masked out of a
// record word (int3: after a shift by 10 for the last three of 8).
__host__ __device__ constexpr int few_field(int fmt, int p) {
    return is_int4(fmt) ? 4 * (p & 1) : fmt == TQ_INT3_G64_SYM ? 2 * ((p & 7) < 5 ? (p & 7) : (p & 7) - 5) : 0;
}

// True (and the count cleared) if a launch since the last call gave up on a
// pipeline wait.
bool rows_int3_take_timeouts();
bool rows_int4g128_take_timeouts();
bool rows_int4g64_take_timeouts();
bool rows_int4g32_take_timeouts();
bool rows_nvfp4_take_timeouts();

// ------------------------------------------------------------------ powers of two

// The power of two of x's binade (x >= 0), clamped to 2^-111 .. 2^126, and its
// inverse: p * inv = 1 exactly, and either times 2^14 or 2^-14 is a normal
// number (so that a row of zeros stays one).
struct Pow2 {
    float p, inv;
};
__host__ __device__ __forceinline__ Pow2 pow2_of(float x) {
    uint32_t b;
    memcpy(&b, &x, 4);
    int e = static_cast<int>((b >> 23) & 255u);
    e = e < 16 ? 16 : (e > 253 ? 253 : e);
    const uint32_t pb = static_cast<uint32_t>(e) << 23, ib = static_cast<uint32_t>(254 - e) << 23;
    Pow2 r;
    memcpy(&r.p, &pb, 4);
    memcpy(&r.inv, &ib, 4);
    return r;
}

// The gated backward pass stores D as f16 (dg or du) * inv * 2^14 with inv the
// inverse power of two of a bound on |dg| and |du|: |dh| <= dmax, |u|, |g| <=
// |x|2 |What row|2 <= |x|2 sqrt(I) wm, |act'| <= 1.13, |act(g)| <= |g|.
// wm in two factors, each multiplied to a number between the gradient's size
// and row_f's: NVFP4's two global scales together may leave fp32 where neither
// the tokens' nor the values' size does.
struct RowsBound {
    float wm, g;
};
__device__ __forceinline__ Pow2 gated_bound(float row_f, RowsBound b, float root_i) {
    return pow2_of(row_f * b.wm * (1.13f * root_i) * b.g);
}

// ------------------------------------------------------------------ device helpers

// Row bounds (made monotone and kept within [0, R]) and the number of tiles of
// NT token rows before each matrix, [E + 1] each: a warp's work.
template <int NT>
__device__ __forceinline__ void rows_table(const int32_t* offsets, int E, int R, int* off, int* tiles) {
    const int lane = threadIdx.x & 31;
    if (offsets == nullptr) {   // one matrix, all rows
        if (lane == 0) {
            off[0] = 0;
            off[1] = R;
            tiles[0] = 0;
            tiles[1] = (R + NT - 1) / NT;
        }
        return;
    }
    int carry = 0, before = 0;   // largest offset and tiles so far
    for (int b = 0; b <= E; b += 32) {
        const int i = b + lane;
        int v = i <= E ? min(max(__ldg(offsets + i), 0), R) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(FULL, v, d);
            if (lane >= d) v = max(v, u);
        }
        v = max(v, carry);
        int prev = __shfl_up_sync(FULL, v, 1);
        if (lane == 0) prev = b == 0 ? v : carry;   // (nothing comes before matrix 0)
        int n = i <= E ? (v - prev + NT - 1) / NT : 0;   // tiles of matrix i - 1
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(FULL, n, d);
            if (lane >= d) n += u;
        }
        n += before;
        if (i <= E) {
            off[i] = v;
            tiles[i] = n;
        }
        carry = __shfl_sync(FULL, v, 31);
        before = __shfl_sync(FULL, n, 31);
    }
}

struct ActGrad {
    float a, d;   // act(g), act'(g)
};

// Both activations are g sigmoid(s) with s = g (alpha + beta g^2): SiLU has
// alpha = 1, beta = 0; the tanh form of GELU, g (1 + tanh y) / 2 with
// y = k (g + c g^3), is g sigmoid(2 y): alpha = 2 k, beta = 2 k c, k =
// sqrt(2 / pi), c = 0.044715.  act' = sigmoid + g sigmoid (1 - sigmoid) s'.
// One path for both, without a branch in the unrolled loops.
struct ActCoef {
    float alpha, beta;
};
__device__ __forceinline__ ActCoef rw_act_coef(int act) {
    return act == TQ_ACT_SILU ? ActCoef{1.f, 0.f} : ActCoef{1.5957691216057308f, 0.07135481282553f};
}
__device__ __forceinline__ ActGrad rw_act(ActCoef k, float g) {
    const float g2 = fminf(g * g, 3.0e38f);   // (SiLU multiplies it by 0, which an infinity would make a NaN)
    const float e = __expf(-g * fmaf(k.beta, g2, k.alpha));
    const float p = __fdividef(1.f, 1.f + e);
    const float q = p * __fdividef(e, 1.f + e);   // p (1 - p), without the difference's rounding
    ActGrad r;
    r.a = g * p;
    // (where the sigmoid has reached 0 or 1, e or the last factor may have overflowed)
    r.d = p + (p == 0.f || e == 0.f ? 0.f : g * q * fmaf(3.f * k.beta, g2, k.alpha));
    return r;
}

// e^x for x <= 0 up to rounding: 2^(x log2 e) by the hardware's approximate
// power of two (2 ulp); results below 2^-126 are 0.
__device__ __forceinline__ float rw_exp(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

__device__ __forceinline__ void rows_put(void* y, int64_t at, int bf16, float v) {
    if (bf16) static_cast<uint16_t*>(y)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else static_cast<float*>(y)[at] = v;
}

// What bounds the values of matrix e (of both projections): the largest |s|
// max(z, 15 - z) of int4 groups, whose zero-points are any byte, 4 |s| of int3
// ones; NVFP4: the largest block scale.  A warp's work.
__device__ __forceinline__ float rows_wmax(const RowsArgs& a, int e, int lane) {
    if (a.wmax == nullptr) return 1.f;
    float v = 0.f;
    const int parts = rows_wmax_parts(a.E);
    for (int i = lane; i < a.projections * parts; i += 32) {
        const int proj = i >= parts ? 1 : 0;
        v = fmaxf(v, __ldg(a.wmax + (static_cast<int64_t>(proj) * a.E + e) * parts + i - proj * parts));
    }
    return warp_max_abs(v, 0.f);
}

// The bound's weight part for the gated backward pass: the largest |What| of
// the matrix's projections (NVFP4: D carries each projection's global scale,
// so both scales' product stands in it).
template <int FMT>
__device__ __forceinline__ RowsBound rows_bound_wm(const RowsArgs& a, int e, float wm) {
    if (FMT != TQ_NVFP4_G16) return {wm, 1.f};
    if (a.projections != 2) return {wm * 6.f, 1.f};   // (6: E2M1's largest)
    return {wm * 6.f * fabsf(__ldg(a.gs[0] + e)), fabsf(__ldg(a.gs[1] + e))};
}

}  // namespace tq
