// Products of token rows with packed records on the tensor cores, one format
// per including file.
//
//   forward   z[t][o] = sum_j What[o][j] x[t][j]
//   backward  dx[t][j] = sum_o D[t][o] What[o][j]
//
// Tiles are 128 weight rows (forward) or 128 columns (backward) by NT tokens,
// walked in steps of 64 along the sum.  From NT = 128 on two CTAs of a cluster
// share 256 weight rows (columns) by NT tokens: each decodes its own 128 and
// brings half of the tokens, and one thread of the first issues the MMAs of
// both (cta_group::2).  Shared memory is what bounds a single CTA: at NT = 256
// a step's 16 KB of weights and 32 KB of tokens are written and read once each,
// 96 KB or 768 clocks against the MMAs' 512; a pair's CTA moves 64 KB.  The weights are the A operand: they
// exist only as records in memory and as tensor-core operands in shared
// memory.  One persistent CTA per SM, four to six warpgroups:
//   warp 0       one thread brings the tokens' 64-column slices by TMA
//   warp 1       one thread issues the tcgen05 MMAs (M = 128, N = NT, K = 16)
//   1 to 4 wg    decode: a thread turns the 64 codes of one weight row and
//                step into one 128-byte operand row (16-byte stores at the
//                128-byte swizzle's places, conflict-free), its record bytes
//                loaded PF steps ahead into registers
//   1 or 2 wg    epilogue: tcgen05.ld of the accumulators, scales, outputs
// (Where groups are added in registers, NT = 256 columns of accumulators need
// 256 threads: two epilogue warpgroups, and one that decodes; below that two
// decode.  The other kinds have four, with 80 registers each: 2, 3 or 4 of them
// took 284 / 301 / 246 us for the g32 gradient below, 698 / 684 / 624 for the
// loss's, 603 / 586 / 581 for the 2048 gated rows.  At 32 tokens a tile only
// int3, whose codes take twice the instructions: NVFP4's 3001 rows 226 / 234 /
// 233.  NVFP4 in wider tiles is within 3 % either way: 4096 rows x 8192 x 4096
// with two 258, their gradient 270; with four 255 and 260.  Short runs, at full
// clocks.)
//
// Measured in sustained passes, the dense ones at the power cap (1.6 to 1.8 GHz;
// in brackets short runs): gated 2048 rows x 17408 x 5120 int4 g128 680 us, 1.07
// PFLOP/s (581), where shared memory is the busiest (78 %, the tensor pipe 65
// %); a gradient of 8192 rows x 4096 x 4096 int4 g32 296 us, 0.93 PFLOP/s (246;
// decoding two scales and zero-points a row and step); the loss of 1024 tokens x
// 65536 x 4096 700 us, 0.79 PFLOP/s (680; exact kind: adding groups); 3001 rows
// over 128 NVFP4 experts of 2688 x 1856 222 us, 1.7 TB/s of records: what is
// bound there is the decoding, with few rows to a weight.
//
// Operands are f16: 11 significant bits at the rate of bf16's 8, and powers of
// two beside them give back the range.  The tokens are a copy in f16 with a
// power of two per row (exact but for values 2^-31 below their row's largest).
// Three kinds (RowsKind):
//  exact   (forward) The weights are the exact small integers v or q - z, so
//          every product is exact; a group's sum is taken in a TMEM
//          accumulator of its own and the epilogue adds it, times the group's
//          fp32 scale, to fp32 registers.  No scale is rounded, and no sum is
//          longer than 128 in the tensor core, whose accumulation truncates
//          (a 6000-wide sum in one accumulator cost the loss a factor of 2.5
//          in accuracy).  TMEM holds 2 (NT = 256) or 4 such accumulators, so
//          the MMAs run on while a group is added.  NVFP4: dec(e) dec(c) has
//          at most 6 significant bits, exact, and 128 columns are a group of
//          scale 1.  For fp32 outputs and the loss.
//  scaled  (forward) One accumulator for the whole sum.  Integer formats:
//          What 2^(14 - E), its scale and then its value rounded to 11 bits (E
//          the binade of M, the matrix's largest |s| max(z, 15 - z), int3 4 |s|:
//          operands stay below 2^15 whatever byte a zero-point is): two roundings of at most 2^-11 per product, well inside
//          the 2^-8 of the 16-bit outputs it serves, and it spares the adding
//          of groups, which bounds the exact kind (128 FMAs of 8 warps per
//          64-wide step).  NVFP4 values are exact.
//  grad    (backward) The sum runs over weight rows, so a group's scale cannot
//          leave it: operands as in the scaled kind, D beside a power of two
//          per token.  A is read MN-major: a weight row's 64 columns are
//          contiguous in the records and in the operand.
// A scale loses bits below 2^-28 M, by at most 2^-39 M (times a code less its
// zero-point, and the product 2^-39 M again: 2^-31 M in all), a token's or
// gradient's value below 2^-28 of its bound, by at most 2^-39 of that.
//
// The order of the columns in an operand row is the one that costs least to
// decode (rows_column): a field of a record word is masked in place in both
// halves at once, which pairs int4 codes m and m + 4 of a word and int3 codes
// i and i + 8 of 16.  The copy of the tokens has the same order (grad: the
// epilogue's lanes are columns in that order).  Or-ed with 0x6400 a field at bit
// b is 1024 + 2^b n in f16, and one exact fma takes 1024 and the zero-point
// away and 2^b out: 13 instructions per 8 int4 codes with their scale.
//
// Every wait has an iteration limit; a role that gives up sets a flag that
// the others see, the copies in flight are awaited, TMEM is freed, and tq_sync
// reports it.
#pragma once

#include <atomic>

#include "codes.cuh"
#include "rows.cuh"
#include "walk.cuh"

namespace tq {

// Waits that gave up, of this format: each including file has a counter of its
// own, and so rw_take_timeouts() below is static.  Reading it costs tq_sync a
// copy, so it is read once a kernel of the format has been launched (or
// captured: a graph may run it any time later).
static __device__ unsigned g_rw_timeouts = 0;
static std::atomic<bool> g_rw_launched{false};

constexpr int RW_A_BYTES = 128 * 128;

template <int FMT> struct RwFmt;   // unit: K = 16 MMAs per accumulator (0: the whole sum)
template <> struct RwFmt<TQ_INT3_G64_SYM> { static constexpr int g = 64, unit = 4, step_bytes = 24; };
template <> struct RwFmt<TQ_INT4_G128_ASYM> { static constexpr int g = 128, unit = 8, step_bytes = 32; };
template <> struct RwFmt<TQ_INT4_G64_ASYM> { static constexpr int g = 64, unit = 4, step_bytes = 32; };
template <> struct RwFmt<TQ_INT4_G32_ASYM> { static constexpr int g = 32, unit = 2, step_bytes = 32; };
template <> struct RwFmt<TQ_NVFP4_G16> { static constexpr int g = 16, unit = 8, step_bytes = 32; };   // (128 columns)

template <int FMT, int NT, int KIND>
struct RwCfg {
    static constexpr bool BWD = KIND == ROWS_GRAD;
    static constexpr int CG = rows_pair(NT) ? 2 : 1;   // CTAs that share a tile
    static constexpr int B_BYTES = NT / CG * 128;      // this CTA's tokens of a stage
    static constexpr int STAGE_BYTES = RW_A_BYTES + B_BYTES;
    static constexpr int STAGES = NT == 256 ? 6 : 8;
    static constexpr int UNIT = KIND == ROWS_EXACT ? RwFmt<FMT>::unit : 0;
    static constexpr int NBUF = NT == 256 ? 2 : 4;
    static constexpr int TMEM_COLS = NBUF * NT;
    static constexpr int EPI_WG = NT == 256 && UNIT ? 2 : 1;
    static constexpr int DEC_WG = !UNIT && (NT > 32 || FMT == TQ_INT3_G64_SYM) ? 4 : 3 - EPI_WG;
    static constexpr int THREADS = 128 * (1 + DEC_WG + EPI_WG);
    static constexpr int CW = NT / EPI_WG;   // accumulator columns of an epilogue thread
    static constexpr int PF = DEC_WG == 4 ? 2 : 4;  // steps of records in a decoding thread's registers
    // registers of a thread at launch, and of the control, decode and epilogue
    // warpgroups, whose sum stays within the launch's
    static constexpr int REG_ALL = DEC_WG == 4 ? 80 : 128;
    static constexpr int REG_CTL = DEC_WG == 4 ? 40 : 56, REG_DEC = DEC_WG == 2 ? 120 : DEC_WG == 4 ? 80 : 104,
                         REG_EPI = DEC_WG == 4 ? 112 : 176;
    static_assert(REG_CTL + DEC_WG * REG_DEC + EPI_WG * REG_EPI <= THREADS / 128 * REG_ALL, "registers");
    static_assert(THREADS * REG_ALL <= 65536, "registers");
    static constexpr int BARS = 2 * STAGES + 2 * NBUF + 1;
    static constexpr int SMEM_TAIL = 512 + (ROWS_MAX_MATS + 1) * 8 + (4 + 3) * NT * 4;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + SMEM_TAIL;
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    static_assert(TMEM_COLS <= 512, "tensor memory");
    // kind::f16 (both f16), fp32 accumulator, M = 128 CG, N = NT; backward: A MN-major
    static constexpr uint32_t IDESC = (1u << 4) | (BWD ? (1u << 15) : 0u) |
                                      (static_cast<uint32_t>(NT >> 3) << 17) | (static_cast<uint32_t>(8 * CG) << 24);
};

// ------------------------------------------------------------------ PTX wrappers

__device__ __forceinline__ uint32_t rw_smem(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// How a wait gives up: the CTA's flag, the other CTA's of its pair (0: none)
// and the number of rounds.
struct RwGiveUp {
    volatile int* abort;
    uint32_t peer;
    unsigned limit;
};

// Waits for the phase of parity `parity`; false when another role gave up or
// after `limit` rounds (then it is this one that gives up).
__device__ __forceinline__ bool rw_wait(uint32_t bar, unsigned parity, const RwGiveUp& g) {
    for (unsigned it = 0; it < g.limit; ++it) {
        unsigned ok;
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
        if (*g.abort) return false;
    }
    if (!*g.abort) atomicAdd(&g_rw_timeouts, 1u);
    *g.abort = 1;
    if (g.peer) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(g.peer), "r"(1) : "memory");
    return false;
}

// The same by a whole warp, all lanes agreeing.
__device__ __forceinline__ bool rw_wait_warp(uint32_t bar, unsigned parity, const RwGiveUp& g) {
    return __all_sync(FULL, rw_wait(bar, parity, g));
}

// The address of the same place in CTA `rank` of the pair.
__device__ __forceinline__ uint32_t rw_mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void rw_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Whether that phase has completed, without waiting.
__device__ __forceinline__ bool rw_test(uint32_t bar, unsigned parity) {
    unsigned ok;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool rw_elect() {
    unsigned ok;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(ok));
    return ok != 0;
}

// An arrival at a barrier of this CTA, or (CG = 2: a mapped address) of its pair.
template <int CG>
__device__ __forceinline__ void rw_arrive(uint32_t bar) {
    if (CG == 2)
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
    else
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A box into this CTA's shared memory; its bytes count at `bar` (CG = 2: a
// mapped address, the leader's).
template <int CG>
__device__ __forceinline__ void rw_tma_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
    if (CG == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%3, %4, %5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
            "%5}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// K-major operand, 128-byte swizzle: 128-byte rows, groups of 8 rows 1024 B apart.
__device__ __forceinline__ uint64_t rw_desc_k(uint32_t addr) {
    return (static_cast<uint64_t>((addr >> 4) & 0x3fffu)) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// MN-major operand: boxes of 64 columns x 64 rows of 128 B (8192 B apart),
// groups of 8 rows 1024 B apart.
__device__ __forceinline__ uint64_t rw_desc_mn(uint32_t addr) {
    return (static_cast<uint64_t>((addr >> 4) & 0x3fffu)) | (512ull << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}

template <int CG>
__device__ __forceinline__ void rw_mma(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if (CG == 2)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(tmem_d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(tmem_d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// The MMAs so far arrive at `bar` when they are complete: in this CTA, or in
// both of the pair (ALL).
template <int CG, bool ALL>
__device__ __forceinline__ void rw_commit(uint32_t bar) {
    if (CG == 2 && ALL)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    else if (CG == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}

__device__ __forceinline__ void rw_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"   // (one statement: nothing may read the registers in between)
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void rw_st32(uint32_t taddr, const float* z) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"f"(z[0]),
        "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]), "f"(z[8]), "f"(z[9]), "f"(z[10]),
        "f"(z[11]), "f"(z[12]), "f"(z[13]), "f"(z[14]), "f"(z[15]), "f"(z[16]), "f"(z[17]), "f"(z[18]), "f"(z[19]),
        "f"(z[20]), "f"(z[21]), "f"(z[22]), "f"(z[23]), "f"(z[24]), "f"(z[25]), "f"(z[26]), "f"(z[27]), "f"(z[28]),
        "f"(z[29]), "f"(z[30]), "f"(z[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void rw_bar(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// The same, and whether v holds for all n threads.
__device__ __forceinline__ bool rw_bar_all(int id, int n, bool v) {
    unsigned all;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 q, %3, 0; bar.red.and.pred p, %1, %2, q; selp.u32 %0, 1, 0, p; }"
                 : "=r"(all)
                 : "r"(id), "r"(n), "r"(static_cast<unsigned>(v))
                 : "memory");
    return all != 0;
}

template <int N> __device__ __forceinline__ void rw_regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void rw_regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------ records

// The record bytes of one weight row for one 64-column step, as loaded: nothing
// here may look at a loaded value, or the step's load would wait for memory
// (1000 to 1700 clocks of a gradient's 3600 per step when halves were swapped,
// and missing records replaced, on arrival; rw_decode does both now).
struct RwRaw {
    uint32_t w[8];     // (int3: high planes in 4 and 5)
    uint32_t z;        // int4: zero-points (g32: two bytes); NVFP4: four E4M3 codes
    float s[2];        // scaled and grad kinds, integer formats: the scales of the step's one or two groups
    bool live;         // there is such a step
    bool ok;           // the row has records there (else: zeros)
};

// Where a row's step is read from, and in its place, where there is none, the
// start of the records: each load has an address that is there.
struct RwBase {
    const uint8_t *p, *g;
    const float* s;
};

// p: the record bytes; left: the bytes of the row from p on (<= 0: none);
// gp: zero-points (int4) or E4M3 codes (NVFP4) of the step's first group; sp:
// its scale (scaled and grad kinds, integer formats); words: a step's zeros
// or codes, and its scales, may be read as one word (whole steps of groups,
// aligned).  flip: the codes' halves of 32 columns are kept in the other order.
// whole: steps of 32 bytes start on 32-byte boundaries; then one load brings a
// step (forward: 32 lanes read 32 rows, and each load takes a cycle a row in
// the cache's tags: the 2048-row case 628 -> 594 us; the gradients, where two
// lanes share a row, lose by it: 438 -> 464 us, and the exact kind is not
// bound by it).
template <int FMT, bool SCALE, bool BWD>
__device__ __forceinline__ void rw_load(RwRaw& r, const uint8_t* p, int left, const uint8_t* gp, const float* sp,
                                        const RwBase& base, bool words, bool whole, int flip) {
    using F = RwFmt<FMT>;
    r.s[0] = r.s[1] = 0.f;
    r.z = 0u;
    // (SCALE only: the exact kind's one decoding warpgroup has no registers to
    // spare; the loss took 752 us with selected addresses, 694 with predicated loads)
    const bool there = SCALE || left > 0;
    if (SCALE) {
        r.ok = left > 0;
        p = r.ok ? p : base.p;
        gp = r.ok ? gp : base.g;
        sp = r.ok ? sp : base.s;
    } else {
        r.ok = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = 0u;
    }
    if constexpr (FMT == TQ_INT3_G64_SYM) {
        const uint2* q = reinterpret_cast<const uint2*>(p);
        if (there) {
            const uint2 x0 = __ldg(q + flip), x1 = __ldg(q + 1 - flip), x2 = __ldg(q + 2);
            r.w[0] = x0.x; r.w[1] = x0.y; r.w[2] = x1.x; r.w[3] = x1.y;
            r.w[4] = x2.x; r.w[5] = x2.y;
            if (SCALE) r.s[0] = __ldg(sp);
        }
    } else {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        if ((FMT != TQ_NVFP4_G16 && F::g != 32) || words) {
            if (SCALE && !BWD && whole) {
                asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                    : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                      "=r"(r.w[7])
                    : "l"(p));
            } else {
                if (there) {
                    const uint4 x = __ldg(q + flip);
                    r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
                }
                if (there) {
                    const uint4 x = __ldg(q + 1 - flip);
                    r.w[4] = x.x; r.w[5] = x.y; r.w[6] = x.z; r.w[7] = x.w;
                }
            }
            if (there) {
                if constexpr (FMT == TQ_NVFP4_G16) {
                    r.z = __ldg(reinterpret_cast<const uint32_t*>(gp));
                } else if constexpr (F::g == 32) {
                    r.z = __ldg(reinterpret_cast<const uint16_t*>(gp));
                    if (SCALE) {
                        const float2 v = __ldg(reinterpret_cast<const float2*>(sp));
                        r.s[0] = v.x;
                        r.s[1] = v.y;
                    }
                } else {
                    r.z = __ldg(gp);
                    if (SCALE) r.s[0] = __ldg(sp);
                }
            }
        } else {   // (a row's last step may lack groups, and rows start anywhere)
#pragma unroll
            for (int i = 0; i < 8; ++i) r.w[i] = 0u;
            if constexpr (FMT == TQ_NVFP4_G16) {   // rows start on 8-byte boundaries; up to four blocks
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int k = b ^ (2 * flip);
                    if (8 * k < left) {
                        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p) + k);
                        r.w[2 * b] = x.x;
                        r.w[2 * b + 1] = x.y;
                    }
                    if (8 * b < left) r.z |= static_cast<uint32_t>(__ldg(gp + b)) << (8 * b);
                }
            } else {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (left > 16 * (b ^ flip)) {
                        const uint4 x = __ldg(q + (b ^ flip));
                        r.w[4 * b] = x.x; r.w[4 * b + 1] = x.y; r.w[4 * b + 2] = x.z; r.w[4 * b + 3] = x.w;
                    }
                    if (left > 16 * b) {
                        r.z |= static_cast<uint32_t>(__ldg(gp + b)) << (8 * b);
                        if (SCALE) r.s[b] = __ldg(sp + b);
                    }
                }
            }
        }
    }
}

// First group of a 64-column step.
template <int FMT>
__device__ __forceinline__ int rw_group(int chunk) {
    constexpr int g = RwFmt<FMT>::g;
    return g == 128 ? chunk >> 1 : chunk * (64 / (g < 64 ? g : 64));
}

__device__ __forceinline__ uint32_t f16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

__host__ __device__ constexpr uint32_t rw_half2(float v) {   // v: a power of two or a small integer, exact in f16
    uint32_t e = 0;
    float a = v < 0 ? -v : v;
    if (a == 0.f) return 0u;
    int x = 15;
    while (a >= 2.f) { a *= 0.5f; ++x; }
    while (a < 1.f) { a *= 2.f; --x; }
    e = (v < 0 ? 0x8000u : 0u) | (static_cast<uint32_t>(x) << 10) | static_cast<uint32_t>((a - 1.f) * 1024.f);
    return e | (e << 16);
}

// Decodes a step into the thread's operand row: 128 bytes at `row`, 16-byte
// units swizzled by x7, columns in rows_column's order.  SCALE: times the
// group's scale as f16 (integer formats: s winv, winv = 2^(14 - E)); the exact
// kind's codes of records that are not there meet tokens of 0, or belong to
// rows without an output.
template <int FMT, bool SCALE>
__device__ __forceinline__ void rw_decode(const RwRaw& r, uint8_t* row, int x7, float winv, int flip) {
    constexpr int g = RwFmt<FMT>::g;
    constexpr uint32_t MAGIC = 0x64006400u;
    auto put = [&](int c, uint32_t (&v)[4], uint32_t ss) {
        if (SCALE || FMT == TQ_NVFP4_G16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = f16x2_mul(v[i], ss);
        }
        *reinterpret_cast<uint4*>(row + ((c ^ x7) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    };
    if constexpr (FMT == TQ_INT3_G64_SYM) {
        const uint32_t ss = SCALE && r.ok ? f16x2_dup(r.s[0] * winv) : 0u;
        const uint32_t hi4 = flip ? r.w[5] : r.w[4], hi5 = flip ? r.w[4] : r.w[5];
#pragma unroll
        for (int m = 0; m < 4; ++m) {   // 16 codes: pairs (i, i + 8)
            const uint32_t L = r.w[m], L10 = L >> 10, H2 = __byte_perm(m < 2 ? hi4 : hi5, 0u, m & 1 ? 0x3322 : 0x1100);
              // code i's high bit at i, code i + 8's at 16 + i
            uint32_t v[2][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int b = i < 5 ? 2 * i : 2 * (i - 5);   // the low field's place
                const uint32_t lo = ((i < 5 ? L : L10) & (0x00030003u << b)) | MAGIC;
                const uint32_t hi = b + 2 >= i ? H2 << (b + 2 - i) : H2 >> (i - b - 2);
                const uint32_t f = lo | (hi & (0x00040004u << b));   // 1024 + 2^b (v + 4)
                if (b <= 7) {
                    const float p = 1.f / static_cast<float>(1 << b);
                    v[i >> 2][i & 3] = b == 0 ? f16x2_sub(f, rw_half2(1028.f)) : f16x2_fma(f, rw_half2(p), rw_half2(-(1024.f * p + 4.f)));
                } else {   // i = 4, b = 8: the field would reach bit 10, so its high bit comes apart: 1024 + 16 h
                    const uint32_t hb = (H2 & 0x00100010u) | MAGIC;
                    v[i >> 2][i & 3] = f16x2_fma(hb, rw_half2(0.25f), f16x2_fma(lo, rw_half2(1.f / 256.f), rw_half2(-264.f)));
                }
            }
            put(2 * m, v[0], ss);
            put(2 * m + 1, v[1], ss);
        }
    } else if constexpr (FMT == TQ_NVFP4_G16) {
        // (a block scale's sign bit is no part of it)
        const uint32_t z = r.ok ? __byte_perm(r.z, 0u, flip ? 0x1032 : 0x3210) : 0u;
        const uint32_t e01 = e4m3x2_f16(z & 0x7f7fu), e23 = e4m3x2_f16((z >> 16) & 0x7f7fu);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint32_t v[4];
            e2m1x8_f16(r.w[c], v);
            put(c, v, __byte_perm(c < 4 ? e01 : e23, 0u, (c >> 1) & 1 ? 0x3232 : 0x1010));
        }
    } else {
#pragma unroll
        for (int k = 0; k < (g == 32 ? 2 : 1); ++k) {   // groups of the step
            const int kk = g == 32 ? k ^ flip : 0;   // (the group's place in memory)
            const uint32_t z = (r.z >> (8 * kk)) & 0xffu, z1 = MAGIC | z | (z << 16);   // 1024 + z
            const uint32_t c16 = f16x2_sub(rw_half2(960.f), z1);                      // -(64 + z)
            const uint32_t ss = SCALE && r.ok ? f16x2_dup((g == 32 && kk ? r.s[1] : r.s[0]) * winv) : 0u;
#pragma unroll
            for (int c = 4 * k; c < (g == 32 ? 4 * k + 4 : 8); ++c) {
                const uint32_t w = r.w[c], w8 = w >> 8;
                uint32_t v[4];
                v[0] = f16x2_sub((w & 0x000f000fu) | MAGIC, z1);
                v[1] = f16x2_fma((w & 0x00f000f0u) | MAGIC, rw_half2(0.0625f), c16);   // (1024 + 16 n) / 16 - 64 - z
                v[2] = f16x2_sub((w8 & 0x000f000fu) | MAGIC, z1);
                v[3] = f16x2_fma((w8 & 0x00f000f0u) | MAGIC, rw_half2(0.0625f), c16);
                put(c, v, ss);
            }
        }
    }
}

// ------------------------------------------------------------------ tiles

struct RwTile {
    int e, m, split;     // matrix; this CTA's 128 weight rows or columns; part of the sum
    int row0, row_end;   // token rows
    int k0, k1;          // steps
};

// Row bounds and token-tile counts per matrix (rows_table), in shared memory.
struct RwTable {
    int* off;     // [E + 1] row bounds, made monotone and within [0, R]
    int* tiles;   // [E + 1] token tiles before matrix e
};

// Item i: matrices in order; within one the token tiles vary fastest, so that
// CTAs running side by side decode the same records.
template <int NT, bool BWD>
__device__ __forceinline__ RwTile rw_tile(const RowsArgs& a, RwTable t, int64_t i, int rank) {
    RwTile r;
    const int64_t q = i / a.splits;
    r.split = static_cast<int>(i - q * a.splits);
    int lo = 0, hi = a.E - 1;   // the last matrix whose first item is <= q
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<int64_t>(t.tiles[mid]) * a.m_tiles <= q) lo = mid;
        else hi = mid - 1;
    }
    const int n = t.tiles[lo + 1] - t.tiles[lo];
    const int local = static_cast<int>(q - static_cast<int64_t>(t.tiles[lo]) * a.m_tiles);
    r.e = lo;
    const int m = local / n;
    r.m = rows_pair(NT) ? 2 * m + rank : m;
    r.row0 = t.off[lo] + (local - m * n) * NT;
    r.row_end = t.off[lo + 1];
    const int steps = BWD ? a.nk * a.projections : a.nk;
    r.k0 = static_cast<int>(static_cast<int64_t>(steps) * r.split / a.splits);
    r.k1 = static_cast<int>(static_cast<int64_t>(steps) * (r.split + 1) / a.splits);
    return r;
}

// A role's walk over the steps of its CTA's items, STRIDE steps at a time.
template <int NT, bool BWD>
struct RwWalk {
    const RowsArgs& a;
    RwTable tab;
    int64_t item, items;
    int rank, stride;
    RwTile t;
    int k;
    __device__ __forceinline__ RwWalk(const RowsArgs& args, RwTable table, int64_t n, int cta, int first)
        : a(args), tab(table), item(blockIdx.x / (rows_pair(NT) ? 2 : 1)), items(n), rank(cta),
          stride(gridDim.x / (rows_pair(NT) ? 2 : 1)), k(0) {
        if (item < items) {
            t = rw_tile<NT, BWD>(a, tab, item, rank);
            k = t.k0;
            advance(first);
        }
    }
    __device__ __forceinline__ bool live() const { return item < items; }
    __device__ __forceinline__ void advance(int n) {
        k += n;
        while (k >= t.k1) {
            const int over = k - t.k1;
            item += stride;
            if (item >= items) return;
            t = rw_tile<NT, BWD>(a, tab, item, rank);
            k = t.k0 + over;
        }
    }
};

// ------------------------------------------------------------------ column reductions

// Over the 32 lanes of a warp, for 32 columns held in v (one per register):
// lane l ends with column l's result.  Each round a lane gives away the half
// of its columns that its partner keeps: 31 shuffles for 32 reductions.
template <bool MAX>
__device__ __forceinline__ float rw_columns(float (&v)[32], int lane) {
#pragma unroll
    for (int st = 0; st < 5; ++st) {
        const int off = 16 >> st;
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < (16 >> st); ++i) {
            const float give = up ? v[i] : v[i + off], keep = up ? v[i + off] : v[i];
            const float got = __shfl_xor_sync(FULL, give, off);
            v[i] = MAX ? fmaxf(keep, got) : __fadd_rn(keep, got);
        }
    }
    return v[0];
}

// ------------------------------------------------------------------ epilogue

// What an epilogue thread knows of its place in the tile.
struct RwPlace {
    int lane, warp4;     // lane, warp of its warpgroup
    int col0;            // its first token column
    int bar;             // its warpgroup's named barrier
    float* red;          // [4][CW] of its warpgroup
    float* colf;         // [CW] a factor or statistic per token
    int* lab;            // [CW] labels
    float* xf;           // [CW] forward: what z's column is multiplied by
};

// The epilogues below take their tile 32 columns at a time from get(c0, v)
// (a warp's call: v[i] = z of the thread's weight row and token c0 + i), in a
// loop that is not unrolled: 128 unrolled columns of stores and exponentials
// overran the instruction cache and took longer than the tile's products.

// y = z.
template <int CW, class Get>
__device__ __forceinline__ void rw_store(const RowsArgs& a, const RwTile& t, const RwPlace& p, Get get) {
    const int64_t o = a.o_begin + static_cast<int64_t>(t.m) * 128 + p.warp4 * 32 + p.lane;
    const int r0 = t.row0 + p.col0, n = o < a.o_end ? min(t.row_end - r0, CW) : 0;
#pragma unroll 1
    for (int c0 = 0; c0 < CW; c0 += 32) {
        float v[32];
        get(c0, v);
        const int64_t at = static_cast<int64_t>(r0 + c0) * a.ldy + o;
        if (a.y_bf16) {
            uint16_t* y = static_cast<uint16_t*>(a.y) + at;
#pragma unroll
            for (int i = 0; i < 32; ++i, y += a.ldy)
                if (c0 + i < n) *y = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
        } else {
            float* y = static_cast<float*>(a.y) + at;
#pragma unroll
            for (int i = 0; i < 32; ++i, y += a.ldy)
                if (c0 + i < n) *y = v[i];
        }
    }
}

// Gated: lanes 0-15 of a warp hold gate rows f .. f + 15, lanes 16-31 the up
// rows of the same f.  One shuffle per two columns gives the lower lanes g
// and u of the even column and the upper lanes those of the odd one.  GRAD: the
// gated backward pass may ask for D instead of h (in the scaled kind alone).
template <int CW, bool GRAD, class Get>
__device__ __forceinline__ void rw_gated(const RowsArgs& a, const RwTile& t, const RwPlace& p, RowsBound bound_wm,
                                         Get get) {
    const int up = p.lane >> 4, tid = p.warp4 * 32 + p.lane;
    const int64_t f = static_cast<int64_t>(t.m) * 64 + p.warp4 * 16 + (p.lane & 15);
    const int r0 = t.row0 + p.col0, rows = min(t.row_end - r0, CW), n = f < a.O ? rows : 0;
    const ActCoef k = rw_act_coef(a.act);
    const bool grad = GRAD && a.mode == ROWS_GATED_BWD;
    const float s0 = grad && a.gs[0] ? __ldg(a.gs[0] + t.e) : 1.f, s1 = grad && a.gs[1] ? __ldg(a.gs[1] + t.e) : 1.f;
    if (grad) {
        for (int c = tid; c < CW; c += 128)
            p.colf[c] = c < rows ? gated_bound(__ldg(a.row_f + r0 + c), bound_wm,
                                               sqrtf(static_cast<float>(a.I))).inv * 16384.f : 0.f;
        rw_bar(p.bar, 128);
    }
#pragma unroll 1
    for (int c0 = 0; c0 < CW; c0 += 32) {
        float v[32];
        get(c0, v);
        // (values first, stores after: a branch per column would keep the
        // columns' exponentials from overlapping)
        float g[16], u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float other = __shfl_xor_sync(FULL, up ? v[2 * i] : v[2 * i + 1], 16);
            g[i] = up ? other : v[2 * i];
            u[i] = up ? v[2 * i + 1] : other;
        }
        const int c1 = c0 + up;   // columns c1, c1 + 2, ...
        const int64_t r = r0 + c1;
        if (!grad) {
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] *= rw_act(k, g[i]).a;
            if (a.y_bf16) {
                uint16_t* y = static_cast<uint16_t*>(a.y) + r * a.ldy + f;
#pragma unroll
                for (int i = 0; i < 16; ++i, y += 2 * a.ldy)
                    if (c1 + 2 * i < n) *y = __bfloat16_as_ushort(__float2bfloat16_rn(u[i]));
            } else {
                float* y = static_cast<float*>(a.y) + r * a.ldy + f;
#pragma unroll
                for (int i = 0; i < 16; ++i, y += 2 * a.ldy)
                    if (c1 + 2 * i < n) *y = u[i];
            }
        } else {
            // (loads past the tile's end read its last row and column again:
            // a condition would make each wait for the one before)
            float dh[16];
            const uint16_t* dp = a.dh + static_cast<int64_t>(r0) * a.ld_dh + min(f, a.O - 1);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                dh[i] = bf16_bits_to_f32(__ldg(dp + min(c1 + 2 * i, rows - 1) * a.ld_dh)) * p.colf[c1 + 2 * i];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const ActGrad w = rw_act(k, g[i]);
                g[i] = (dh[i] * u[i]) * (w.d * s0);
                u[i] = (dh[i] * w.a) * s1;
            }
            uint16_t* d = a.D + r * a.ldd + f;
            uint16_t* d2 = d + a.R * a.ldd;
#pragma unroll
            for (int i = 0; i < 16; ++i, d += 2 * a.ldd, d2 += 2 * a.ldd)
                if (c1 + 2 * i < n) {
                    *d = __half_as_ushort(__float2half_rn(g[i]));
                    *d2 = __half_as_ushort(__float2half_rn(u[i]));
                }
        }
    }
}

// The tile's labels (-1: none) into shared memory.
__device__ __forceinline__ void rw_label(const RowsArgs& a, const RwPlace& p, int c, int r0, int n) {
    const int64_t l = c < n ? __ldg(a.labels + r0 + c) : -1;
    p.lab[c] = l >= 0 && l < a.O ? static_cast<int>(l) : -1;
}

// Per token of the tile: the largest z over its 128 weight rows and the sum of
// e^(z - that), and the label's z where its row is in this tile.
template <int CW, class Get>
__device__ __forceinline__ void rw_loss(const RowsArgs& a, const RwTile& t, const RwPlace& p, Get get) {
    const int64_t o = a.o_begin + static_cast<int64_t>(t.m) * 128 + p.warp4 * 32 + p.lane;
    const bool real = o < a.o_end;
    const int mine = real ? static_cast<int>(o) : -2;   // (no label is -2)
    const int r0 = t.row0 + p.col0, n = min(t.row_end - r0, CW), tid = p.warp4 * 32 + p.lane;
    constexpr float NONE = -INFINITY;
    for (int c = tid; c < CW; c += 128) rw_label(a, p, c, r0, n);
#pragma unroll 1
    for (int c0 = 0; c0 < CW; c0 += 32) {
        float v[32];
        get(c0, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = real ? v[i] : NONE;
        p.red[p.warp4 * CW + c0 + p.lane] = rw_columns<true>(v, p.lane);
    }
    rw_bar(p.bar, 128);
    for (int c = tid; c < CW; c += 128) {
        float m = p.red[c];
#pragma unroll
        for (int w = 1; w < 4; ++w) m = fmaxf(m, p.red[w * CW + c]);
        p.colf[c] = m == NONE ? 0.f : m;
    }
    rw_bar(p.bar, 128);
#pragma unroll 1
    for (int c0 = 0; c0 < CW; c0 += 32) {
        float v[32];
        get(c0, v);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (p.lab[c0 + i] == mine) a.label_z[r0 + c0 + i] = v[i];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = real ? rw_exp(v[i] - p.colf[c0 + i]) : 0.f;
        p.red[p.warp4 * CW + c0 + p.lane] = rw_columns<false>(v, p.lane);
    }
    rw_bar(p.bar, 128);
    for (int c = tid; c < n; c += 128) {
        float s = p.red[c];
#pragma unroll
        for (int w = 1; w < 4; ++w) s += p.red[w * CW + c];
        // (no sum: the pair's second tile may be past the end, and all of a
        // tile's logits -inf; its 0 above is no largest that others join)
        a.part[static_cast<int64_t>(t.m) * a.R + r0 + c] = make_float2(s == 0.f ? -3.0e38f : p.colf[c], s);
    }
}

// D = (e^(z - lse) - [o is the label]) 2^13 in f16; 0 for a token without one.
template <int CW, class Get>
__device__ __forceinline__ void rw_prob(const RowsArgs& a, const RwTile& t, const RwPlace& p, Get get) {
    const int64_t o = a.o_begin + static_cast<int64_t>(t.m) * 128 + p.warp4 * 32 + p.lane;
    const int r0 = t.row0 + p.col0, rows = min(t.row_end - r0, CW), n = o < a.o_end ? rows : 0;
    const int tid = p.warp4 * 32 + p.lane;
    for (int c = tid; c < CW; c += 128) {
        rw_label(a, p, c, r0, rows);
        p.colf[c] = c < rows ? __ldg(a.lse + r0 + c) : 0.f;
    }
    rw_bar(p.bar, 128);
#pragma unroll 1
    for (int c0 = 0; c0 < CW; c0 += 32) {
        float v[32];
        get(c0, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int l = p.lab[c0 + i];
            const float w = rw_exp(v[i] - p.colf[c0 + i]);
            v[i] = (l < 0 ? 0.f : l == static_cast<int>(o) ? w - 1.f : w) * ROWS_PROB_SCALE;
        }
        uint16_t* d = a.D + static_cast<int64_t>(r0 + c0) * a.ldd + (o - a.o_begin);
#pragma unroll
        for (int i = 0; i < 32; ++i, d += a.ldd)
            if (c0 + i < n) *d = __half_as_ushort(__float2half_rn(v[i]));
    }
}

// dx (or its partial sums) of 128 columns: a lane is a column, in the
// operand's order.
template <int FMT, int CW, class Get>
__device__ __forceinline__ void rw_grad(const RowsArgs& a, const RwTile& t, const RwPlace& p, RowsBound bound_wm,
                                        float wscale, Get get) {
    const int64_t j = static_cast<int64_t>(t.m) * 128 + rows_column(FMT, p.warp4 * 32 + p.lane);
    const int r0 = t.row0 + p.col0, rows = min(t.row_end - r0, CW), n = j < a.I ? rows : 0;
    const int tid = p.warp4 * 32 + p.lane;
    for (int c = tid; c < CW; c += 128) {
        float f = c < rows ? __ldg(a.row_f + r0 + c) : 0.f;
        if (a.mode == ROWS_GATED_BWD)
            f = gated_bound(f, bound_wm, sqrtf(static_cast<float>(a.I))).p * 6.103515625e-05f;   // 2^-14
        if (a.mode == ROWS_PROB && c < rows) {   // (a token without a label: 0, whatever its loss's gradient says)
            const int64_t l = __ldg(a.labels + r0 + c);
            f = l >= 0 && l < a.O ? f : 0.f;
        }
        p.colf[c] = f;
    }
    rw_bar(p.bar, 128);
#pragma unroll 1
    for (int c0 = 0; c0 < CW; c0 += 32) {
        float v[32];
        get(c0, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = (v[i] * wscale) * p.colf[c0 + i];
        if (a.sums) {
            float* q = a.sums + (static_cast<int64_t>(t.split) * a.R + r0 + c0) * a.I + j;
#pragma unroll
            for (int i = 0; i < 32; ++i, q += a.I)
                if (c0 + i < n) *q = a.sums_add ? *q + v[i] : v[i];
        } else {
            uint16_t* y = static_cast<uint16_t*>(a.y) + static_cast<int64_t>(r0 + c0) * a.ldy + j;
#pragma unroll
            for (int i = 0; i < 32; ++i, y += a.ldy)
                if (c0 + i < n) *y = __bfloat16_as_ushort(__float2bfloat16_rn(v[i]));
        }
    }
}

// ------------------------------------------------------------------ kernel

template <int FMT, int NT, int KIND>
__global__ void __launch_bounds__(RwCfg<FMT, NT, KIND>::THREADS, 1)
k_rows(const __grid_constant__ CUtensorMap map, const __grid_constant__ RowsArgs a) {
    using C = RwCfg<FMT, NT, KIND>;
    using F = RwFmt<FMT>;
    constexpr bool BWD = C::BWD, SCALE = KIND != ROWS_EXACT;
    constexpr int ST = C::STAGES, NBUF = C::NBUF, CW = C::CW, UNIT = C::UNIT, CG = C::CG;
    extern __shared__ uint8_t rw_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(rw_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + ST * C::STAGE_BYTES);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::BARS);
    // [0] steps armed, [1] consumed, [2] abort, [4 ..] steps each decoding warp has passed
    volatile int* st = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* table = reinterpret_cast<int*>(smem + ST * C::STAGE_BYTES + 512);
    const RwTable tab{table, table + ROWS_MAX_MATS + 1};
    float* red = reinterpret_cast<float*>(table + 2 * (ROWS_MAX_MATS + 1));
    float* colf = red + 4 * NT;
    int* lab = reinterpret_cast<int*>(colf + NT);
    float* xf = reinterpret_cast<float*>(lab + NT);
    const uint32_t s_base = rw_smem(smem);
    const uint32_t full = rw_smem(bars), empty = full + 8 * ST;
    const uint32_t acc_full = empty + 8 * ST, acc_empty = acc_full + 8 * NBUF, done = acc_empty + 8 * NBUF;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;
    const int rank = CG == 2 ? static_cast<int>(blockIdx.x & 1u) : 0;   // (clusters are pairs along x)
    const int64_t first_item = blockIdx.x / CG;
    const int stride = static_cast<int>(gridDim.x / CG);

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            // a full stage: the copies (one arrival and the bytes) and each CTA's four decoding warps
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(full + 8 * i), "r"(1 + 4 * CG) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(empty + 8 * i) : "memory");
        }
        for (int i = 0; i < NBUF; ++i) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(acc_full + 8 * i) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(acc_empty + 8 * i), "r"(4 * C::EPI_WG * CG)
                         : "memory");
        }
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(done) : "memory");
        st[0] = 0;
        st[1] = 0;
        st[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) rows_table<NT>(a.offsets, a.E, static_cast<int>(a.R), tab.off, tab.tiles);
    if (warp == 1) {
        if (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(rw_smem(tmem_slot)),
                         "r"(C::TMEM_COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(rw_smem(tmem_slot)),
                         "r"(C::TMEM_COLS));
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (CG == 2) rw_cluster_sync();   // both CTAs' barriers are there
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    const int64_t items = static_cast<int64_t>(tab.tiles[a.E]) * a.m_tiles * a.splits;
    const uint32_t my_abort = rw_smem(const_cast<int*>(st + 2));
    const RwGiveUp gu{st + 2, CG == 2 ? rw_mapa(my_abort, static_cast<uint32_t>(rank ^ 1)) : 0u, a.wait_limit};
    // the pair's barriers of full stages and empty accumulators are the leader's
    const uint32_t full_l = CG == 2 ? rw_mapa(full, 0) : full, acc_empty_l = CG == 2 ? rw_mapa(acc_empty, 0) : acc_empty;

    if (wg == 0) {
        rw_regs_dec<C::REG_CTL>();
        // Whole warps walk and wait; one elected lane issues, so descriptors
        // and coordinates stay in uniform registers.
        if (warp == 0) {   // the tokens' slices
            int q = 0;
            for (RwWalk<NT, BWD> w(a, tab, items, rank, 0); w.live(); w.advance(1), ++q) {
                const int s = q % ST;
                if (!rw_wait_warp(empty + 8 * s, ((q / ST) & 1) ^ 1, gu)) break;
                if (rw_elect()) {
                    st[0] = q + 1;
                    if (rank == 0)   // the leader's arrival stands for both CTAs' copies
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full + 8 * s),
                                     "r"(C::B_BYTES * CG)
                                     : "memory");
                    const int proj = BWD && w.k >= a.nk ? 1 : 0;
                    rw_tma_3d<CG>(s_base + s * C::STAGE_BYTES + RW_A_BYTES, &map, full_l + 8 * s,
                                  (w.k - proj * a.nk) * 64, w.t.row0 + rank * (NT / CG), proj);
                }
                __syncwarp();
            }
        } else if (warp == 1 && rank == 0) {   // MMAs (of both CTAs)
            // One elected thread.  The tensor core's queue is short, so what
            // this loop does between MMAs is time the tensor core may idle: it
            // holds next to nothing but the MMAs (an elected thread's loop
            // issues 4 in 170 clocks where one of `lane == 0` takes 260).
            if (rw_elect()) {
                constexpr uint32_t A_K = (BWD ? 2048 : 32) >> 4, B_K = 32 >> 4, STG = C::STAGE_BYTES >> 4;
                const uint64_t da0 = BWD ? rw_desc_mn(s_base) : rw_desc_k(s_base), db0 = rw_desc_k(s_base + RW_A_BYTES);
                int s = 0, b = 0;               // stage, accumulator
                unsigned ph = 0, ab = 1;        // their phases' parities
                int q = 0;                      // steps whose stages have been waited for
                bool ok = true;
                auto filled = [&]() {
                    ok = rw_test(full + 8 * s, ph) || rw_wait(full + 8 * s, ph, gu);
                    q += ok;
                    return ok;
                };
                auto cleared = [&]() {
                    ok = rw_test(acc_empty + 8 * b, ab) || rw_wait(acc_empty + 8 * b, ab, gu);
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    return ok;
                };
                auto whole = [&]() {
                    rw_commit<CG, true>(acc_full + 8 * b);
                    if (++b == NBUF) {
                        b = 0;
                        ab ^= 1;
                    }
                };
                auto freed = [&]() {
                    rw_commit<CG, true>(empty + 8 * s);
                    if (++s == ST) {
                        s = 0;
                        ph ^= 1;
                    }
                };
                for (int64_t item = first_item; ok && item < items; item += stride) {
                    const RwTile t = rw_tile<NT, BWD>(a, tab, item, rank);
                    const int steps = t.k1 - t.k0;
                    if constexpr (UNIT == 2) {   // two groups in a step
                        for (int k = 0; k < steps && filled(); ++k) {
                            const uint64_t da = da0 + static_cast<uint32_t>(s) * STG, db = db0 + static_cast<uint32_t>(s) * STG;
#pragma unroll
                            for (int h = 0; h < 4; h += 2) {
                                if (!cleared()) break;
                                const uint32_t d = tmem + static_cast<uint32_t>(NT * b);
                                rw_mma<CG>(d, da + h * A_K, db + h * B_K, C::IDESC, 0);
                                rw_mma<CG>(d, da + (h + 1) * A_K, db + (h + 1) * B_K, C::IDESC, 1);
                                whole();
                            }
                            if (!ok) break;
                            freed();
                        }
                    } else {
                        for (int k = 0; k < steps && cleared();) {
                            const uint32_t d = tmem + static_cast<uint32_t>(NT * b);
                            const int end = UNIT ? min(k + UNIT / 4, steps) : steps;
                            for (uint32_t more = 0; k < end && filled(); ++k, more = 1) {
                                const uint64_t da = da0 + static_cast<uint32_t>(s) * STG,
                                               db = db0 + static_cast<uint32_t>(s) * STG;
                                rw_mma<CG>(d, da, db, C::IDESC, more);
#pragma unroll
                                for (int j = 1; j < 4; ++j) rw_mma<CG>(d, da + j * A_K, db + j * B_K, C::IDESC, 1);
                                freed();
                            }
                            if (!ok) break;
                            whole();
                        }
                    }
                }
                st[1] = q;
                rw_commit<CG, false>(done);
            }
            __syncwarp();
        }
    } else if (wg <= C::DEC_WG) {
        if constexpr (C::REG_DEC < C::REG_ALL) rw_regs_dec<C::REG_DEC>();
        else if constexpr (C::REG_DEC > C::REG_ALL) rw_regs_inc<C::REG_DEC>();
        constexpr int STEP = C::DEC_WG, PF = C::PF;
        // backward: lanes 2 i and 2 i + 1 take the two 64-column halves of one
        // weight row, so that a load touches half as many lines; the odd ones
        // keep their units in the other order, which keeps the stores of a
        // quarter of a warp on different banks
        const int tid = threadIdx.x & 127, flip = BWD ? tid & 1 : 0, orow = BWD ? 64 * flip + (tid >> 1) : tid;
        const int x7 = (orow & 7) ^ (4 * flip);
        // forward: the thread's row of the tile; gated: lanes 0-15 of a warp
        // take gate rows, lanes 16-31 the up rows beside them
        const int gproj = (tid >> 4) & 1, grow = (tid >> 5) * 16 + (tid & 15);
        RwRaw raw[PF];
        float winv[PF];
        RwWalk<NT, BWD> w(a, tab, items, rank, wg - 1);
        int we = -1;
        float inv = 1.f;
        // the thread's pointers, recomputed when the walk enters another item
        // (backward: or the other projection)
        int64_t seen = -1;
        const uint8_t *rp = nullptr, *gp = nullptr;
        const float* sp = nullptr;
        int left = 0, o_first = 0;
        const int64_t step_bytes = 64 * a.rowbytes, step_groups = 64 * a.G;   // backward: 64 weight rows on
        const uintptr_t sal = reinterpret_cast<uintptr_t>(a.scales[0]) | reinterpret_cast<uintptr_t>(a.scales[1]),
                        zal = reinterpret_cast<uintptr_t>(a.zeros[0]) | reinterpret_cast<uintptr_t>(a.zeros[1]);
        const bool words = FMT == TQ_NVFP4_G16 ? (a.G & 3) == 0 && (sal & 3) == 0
                                               : F::g == 32 && (a.G & 1) == 0 && (sal & 7) == 0 && (zal & 1) == 0;
        const RwBase base{a.packed[0], FMT == TQ_NVFP4_G16 ? static_cast<const uint8_t*>(a.scales[0]) : a.zeros[0],
                    static_cast<const float*>(a.scales[0])};
        const bool whole = ((reinterpret_cast<uintptr_t>(a.packed[0]) | reinterpret_cast<uintptr_t>(a.packed[1])) & 31) == 0;
        auto load = [&](RwRaw& r, float& wi) {
            r.live = __any_sync(FULL, w.live());
            wi = inv;
            if (!SCALE && !r.live) return;
            const int proj = BWD ? (w.k >= a.nk ? 1 : 0) : (a.projections == 2 ? gproj : 0);
            const int64_t now = BWD ? 2 * w.item + proj : w.item;
            if (r.live && now != seen) {
                seen = now;
                int64_t o;
                if (SCALE && FMT != TQ_NVFP4_G16 && w.t.e != we) {
                    we = w.t.e;
                    inv = pow2_of(rows_wmax(a, we, lane)).inv * 16384.f;
                }
                if constexpr (BWD) {
                    o = a.o_begin + (tid >> 1);
                    o_first = static_cast<int>(o);
                } else {
                    o = a.projections == 2 ? static_cast<int64_t>(w.t.m) * 64 + grow
                                           : a.o_begin + static_cast<int64_t>(w.t.m) * 128 + tid;
                }
                const int chunk = BWD ? 2 * w.t.m + flip : 0;
                const int64_t row = w.t.e * a.O + o, g0 = row * a.G + rw_group<FMT>(chunk);
                rp = a.packed[proj] + row * a.rowbytes + chunk * F::step_bytes;
                left = BWD || o < a.o_end ? static_cast<int>(a.rowbytes) - chunk * F::step_bytes : 0;
                if (FMT == TQ_NVFP4_G16) gp = static_cast<const uint8_t*>(a.scales[proj]) + g0;
                else gp = a.zeros[proj] + g0;
                sp = static_cast<const float*>(a.scales[proj]) + g0;
            }
            wi = inv;
            // (past the CTA's last step: the base's bytes, which nobody looks at)
            if constexpr (BWD) {
                const int k = w.k - proj * a.nk;
                rw_load<FMT, SCALE, BWD>(r, rp + k * step_bytes, r.live && o_first + 64 * k < a.o_end ? left : 0,
                                    gp + k * step_groups, sp + k * step_groups, base, words, whole, flip);
            } else {
                rw_load<FMT, SCALE, BWD>(r, rp + w.k * F::step_bytes, r.live ? left - w.k * F::step_bytes : 0,
                                    gp + rw_group<FMT>(w.k), sp + rw_group<FMT>(w.k), base, words, whole, flip);
            }
            w.advance(STEP);
        };
#pragma unroll
        for (int i = 0; i < PF; ++i) load(raw[i], winv[i]);
        bool go = true;
        int q = wg - 1;
        while (go) {
#pragma unroll
            for (int i = 0; i < PF; ++i, q += STEP) {
                const int s = q % ST;
                if (!raw[i].live || !rw_wait_warp(empty + 8 * s, ((q / ST) & 1) ^ 1, gu)) {
                    go = false;
                    break;
                }
                rw_decode<FMT, SCALE>(raw[i], smem + s * C::STAGE_BYTES + orow * 128, x7, winv[i], flip);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) rw_arrive<CG>(full_l + 8 * s);
                load(raw[i], winv[i]);
            }
        }
        if (lane == 0) st[warp] = q;   // (a warp that ended early has passed its steps before q)
    } else {
        rw_regs_inc<C::REG_EPI>();
        RwPlace p;
        const int ew = wg - 1 - C::DEC_WG;
        p.lane = lane;
        p.warp4 = warp & 3;
        p.col0 = ew * CW;
        p.bar = 1 + ew;
        p.red = red + 4 * CW * ew;
        p.colf = colf + CW * ew;
        p.lab = lab + CW * ew;
        p.xf = xf + CW * ew;
        const uint32_t tlane = tmem + (static_cast<uint32_t>(p.warp4 * 32) << 16) + static_cast<uint32_t>(p.col0);
        int u = 0;
        for (int64_t item = first_item; item < items; item += stride) {
            const RwTile t = rw_tile<NT, BWD>(a, tab, item, rank);
            // (a last, short piece of a vocabulary may leave a split without a
            // step: its sums so far stand)
            if (t.k0 == t.k1) continue;
            // Whether all four warps have the whole tile: where one gave up none
            // goes on to the barriers below.  (It also parts the tiles: the
            // previous one's xf, colf, lab and red are read.)
            auto whole = [&](bool ok) { return rw_bar_all(p.bar, 128, ok); };
            auto finish = [&](auto get) {
                if constexpr (BWD) {
                    const float wm = rows_wmax(a, t.e, lane);
                    // integer formats: the operands were What 2^(14 - E); NVFP4: What / g (gated: g is in D)
                    float ws = FMT != TQ_NVFP4_G16 ? pow2_of(wm).p * 6.103515625e-05f
                               : a.mode == ROWS_GATED_BWD ? 1.f : __ldg(a.gs[0] + t.e);
                    if (a.mode == ROWS_PROB) ws *= 1.f / ROWS_PROB_SCALE;
                    rw_grad<FMT, CW>(a, t, p, rows_bound_wm<FMT>(a, t.e, wm), ws, get);
                } else if (a.mode == ROWS_STORE) {
                    rw_store<CW>(a, t, p, get);
                } else if (KIND == ROWS_SCALED) {   // (the losses are for the exact kind)
                    rw_gated<CW, true>(a, t, p,
                                       a.mode == ROWS_GATED_BWD ? rows_bound_wm<FMT>(a, t.e, rows_wmax(a, t.e, lane))
                                                                : RowsBound{},
                                       get);
                } else if (a.mode == ROWS_LOSS) {
                    rw_loss<CW>(a, t, p, get);
                } else if (a.mode == ROWS_PROB) {
                    rw_prob<CW>(a, t, p, get);
                } else {
                    rw_gated<CW, false>(a, t, p, RowsBound{}, get);
                }
            };
            // A column's factor: the power of two beside its token, and what the
            // weights still lack: 2^(E - 14) or, NVFP4, the global scale (by
            // row: see gs).
            auto factors = [&](float ws) {
                const int r0 = t.row0 + p.col0, tid = p.warp4 * 32 + lane;
                for (int c = tid; c < CW; c += 128) p.xf[c] = r0 + c < t.row_end ? __ldg(a.row_x + r0 + c) * ws : 0.f;
                rw_bar(p.bar, 128);
            };
            if constexpr (UNIT != 0) {   // groups added with their scales
                float z[CW];
                bool go = true;
                const bool gated = a.projections == 2;
                const int proj = gated ? lane >> 4 : 0;
                const int64_t o = gated ? static_cast<int64_t>(t.m) * 64 + p.warp4 * 16 + (lane & 15)
                                        : a.o_begin + static_cast<int64_t>(t.m) * 128 + p.warp4 * 32 + lane;
                const float* sc = static_cast<const float*>(a.scales[proj]) + (t.e * a.O + o) * a.G;
                const int G = o < a.o_end ? static_cast<int>(a.G) : 0;
                const int units = (4 * (t.k1 - t.k0) + UNIT - 1) / UNIT;
#pragma unroll
                for (int c = 0; c < CW; ++c) z[c] = 0.f;
                constexpr bool ONE = FMT == TQ_NVFP4_G16;   // every group's scale
                float s = ONE ? 1.f : 0 < G ? __ldg(sc) : 0.f;
                for (int k = 0; k < units; ++k, ++u) {
                    const int b = u % NBUF;
                    const float next = ONE ? 1.f : k + 1 < G ? __ldg(sc + k + 1) : 0.f;
                    if (!rw_wait_warp(acc_full + 8 * b, (u / NBUF) & 1, gu)) {
                        go = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                    for (int c0 = 0; c0 < CW; c0 += 32) {
                        uint32_t v[32];
                        rw_ld32(tlane + static_cast<uint32_t>(NT * b + c0), v);
                        if (c0 + 32 == CW && k + 1 < units) {   // (the last group's is kept for the finish)
                            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                            if (lane == 0) rw_arrive<CG>(acc_empty_l + 8 * b);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) z[c0 + i] = __fmaf_rn(s, __uint_as_float(v[i]), z[c0 + i]);
                    }
                    s = next;
                }
                if (!whole(go)) break;
                // The finished columns go back to the last group's accumulator:
                // the epilogues below read them 32 at a time in a rolled loop,
                // which 128 registers would not let them index.
                const int b = (u - 1) % NBUF;
#pragma unroll
                for (int c0 = 0; c0 < CW; c0 += 32) rw_st32(tlane + static_cast<uint32_t>(NT * b + c0), &z[c0]);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                float gs = 1.f;   // NVFP4: the global scale of the lane's projection
                if (ONE) gs = __ldg(a.gs[proj] + t.e);
                factors(1.f);
                finish([&](int c0, float (&v)[32]) {
                    uint32_t w[32];
                    rw_ld32(tlane + static_cast<uint32_t>(NT * b + c0), w);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(w[i]) * gs * p.xf[c0 + i];   // (gs first: see below)
                });
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                if (lane == 0) rw_arrive<CG>(acc_empty_l + 8 * b);
            } else {
                const int b = u % NBUF;
                if (!whole(rw_wait_warp(acc_full + 8 * b, (u / NBUF) & 1, gu))) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                float gs = 1.f;   // NVFP4, forward: the global scale of the lane's projection
                if constexpr (!BWD) {
                    if (FMT == TQ_NVFP4_G16) gs = __ldg((a.projections == 2 && lane >= 16 ? a.gs[1] : a.gs[0]) + t.e);
                    factors(FMT == TQ_NVFP4_G16 ? 1.f : pow2_of(rows_wmax(a, t.e, lane)).p * 6.103515625e-05f);   // 2^(E - 14)
                }
                finish([&](int c0, float (&v)[32]) {
                    uint32_t w[32];
                    rw_ld32(tlane + static_cast<uint32_t>(NT * b + c0), w);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[i] = __uint_as_float(w[i]);
                        // (the global scale first: with the tokens' power of
                        // two alone the sum may overflow)
                        if (!BWD && FMT == TQ_NVFP4_G16) v[i] *= gs;
                        if (!BWD) v[i] *= p.xf[c0 + i];
                    }
                });
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                if (lane == 0) rw_arrive<CG>(acc_empty_l + 8 * b);
                ++u;
            }
        }
    }

    // teardown: the copies issued but not consumed and the MMAs committed,
    // with the default limit; then free TMEM
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (CG == 2) rw_cluster_sync();
    if (threadIdx.x == 0 && rank == 0) {
        int quiet = 0;
        const RwGiveUp end{&quiet, 0u, DEFAULT_WAIT_LIMIT};
        const uint32_t st_peer = CG == 2 ? rw_mapa(rw_smem(const_cast<int*>(st)), 1) : 0u;
        auto peer = [&](int i) {
            int v = 0;
            if (CG == 2) asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(st_peer + 4 * i) : "memory");
            return v;
        };
        const int armed = st[0], armed_peer = CG == 2 ? peer(0) : armed;
        for (int k = st[1]; k < max(armed, armed_peer); ++k) {
            // (only after an abort) what the stage is still owed: a CTA's
            // arming and bytes, and the arrivals of decoding warps
            const uint32_t bar = full + 8 * (k % ST);
            auto bytes = [&]() {
                asm volatile("mbarrier.complete_tx.shared::cluster.relaxed.cluster.b64 [%0], %1;" ::"r"(rw_mapa(bar, 0)),
                             "r"(C::B_BYTES)
                             : "memory");
            };
            if (k >= armed) {
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(C::B_BYTES * CG)
                             : "memory");
                bytes();
            }
            if (k >= armed_peer) bytes();
            const int owner = k % C::DEC_WG;
            for (int v = 0; v < 4; ++v) {
                if (k >= st[4 + 4 * owner + v]) rw_arrive<1>(bar);
                if (CG == 2 && k >= peer(4 + 4 * owner + v)) rw_arrive<1>(bar);
            }
            if (!rw_wait(bar, (k / ST) & 1, end)) break;
        }
        rw_wait(done, 0, end);
    }
    __syncthreads();
    if (CG == 2) rw_cluster_sync();   // neither CTA leaves while the other may still reach its memory
    if (warp == 1) {
        if (CG == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
    }
}

// ------------------------------------------------------------------ launch

// Shared memory above 48 KB is asked for once per kernel and device.
template <int FMT, int NT, int KIND>
tq_status rw_launch(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st) {
    using C = RwCfg<FMT, NT, KIND>;
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(k_rows<FMT, NT, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   C::SMEM_BYTES);
        if (e != cudaSuccess) return set_error(TQ_ERR_CUDA, "row products: %s", cudaGetErrorString(e));
        ready.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(l.grid));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C::CG;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = C::CG == 2 ? 1 : 0;
    g_rw_launched.store(true, std::memory_order_relaxed);
    cudaLaunchKernelEx(&cfg, k_rows<FMT, NT, KIND>, *l.map, a);
    return check_launch("row products");
}

template <int FMT, int KIND>
tq_status rw_launch_nt(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st) {
    switch (l.nt) {
        case 32: return rw_launch<FMT, 32, KIND>(a, l, st);
        case 64: return rw_launch<FMT, 64, KIND>(a, l, st);
        case 128: return rw_launch<FMT, 128, KIND>(a, l, st);
        default: return rw_launch<FMT, 256, KIND>(a, l, st);
    }
}

template <int FMT>
tq_status rw_launch_fmt(const RowsArgs& a, const RowsLaunch& l, cudaStream_t st) {
    if (l.kind == ROWS_GRAD) return rw_launch_nt<FMT, ROWS_GRAD>(a, l, st);
    if (l.kind == ROWS_EXACT) return rw_launch_nt<FMT, ROWS_EXACT>(a, l, st);
    return rw_launch_nt<FMT, ROWS_SCALED>(a, l, st);
}

static bool rw_take_timeouts() {
    if (!g_rw_launched.load(std::memory_order_relaxed)) return false;
    unsigned n = 0;
    if (cudaMemcpyFromSymbol(&n, g_rw_timeouts, sizeof(n)) != cudaSuccess || n == 0) return false;
    const unsigned zero = 0;
    cudaMemcpyToSymbol(g_rw_timeouts, &zero, sizeof(zero));
    return true;
}

}  // namespace tq
