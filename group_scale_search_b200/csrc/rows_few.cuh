// Row products for few tokens per matrix, one format per including file:
// decoding, a short prompt, experts that a router gives a handful of rows.
//
//   z[t][o] = sum_j What[o][j] x[t][j],   up to 8 NB tokens of one matrix at a time
//
// The records are read once from HBM and the tokens are next to nothing, so
// the kernel is a stream of records through the registers: mma.sync m16n8k16
// takes its A operand from registers, which saves the trip of a decoded weight
// through shared or tensor memory that tcgen05 would need, and with 8 to 32
// tokens the tensor cores have little to do either way.  Measured: one
// token, two 17408 x 5120 int4 g128 matrices, 33 us, 2.9 TB/s of records (the
// tcgen05 kernel of rows_core.cuh took 93); 48 rows over 128 NVFP4 experts 84
// us, 2.8 TB/s.  Two blocks an SM are all that the registers hold, and their
// 16 warps' instruction latency is the bound (issue 40 %).
//
// A tile is 32 weight rows (gated: 16 gate rows and the 16 up rows beside
// them); ks = 1, 2, 4 or 8 of a block's warps share it, each taking every
// ks-th 128-column slice, and their sums are joined through shared memory in
// warp order.  Blocks are persistent over contiguous runs of tiles; the loads
// of the next PD slices are in flight while a slice is multiplied, across tile
// boundaries.  (ks: the fewest warps that still give every warp of the GPU
// work, since a tile's end costs about as much as two slices.)
//
// The k index of the MMAs is a permutation of a slice's columns: lane (gid,
// tig) of the fragment layouts owns 32 columns of weight rows gid and gid + 8
// and takes them two codes at a time in the order that costs least to decode;
// rows.cuh says which.  The tokens were put into that order, as f16
// beside a power of two per row, by k_few_prep.
//
// Decoding: an f16 below 2^-14 is an integer of up to 10 bits times 2^-24, so a
// field of a record word, masked in place, is the code times 2^(b - 24) with b
// its lowest bit; one exact product by 2^14 per two codes makes it a normal
// number, and the tokens beside it were scaled by 2^-b: int4 costs 9
// instructions per 8 codes (4 lop3, 1 shift, 4 products), int3 4 per 2 codes
// (the high plane's bit is shifted beside the low plane's).  Without the product
// one token is 3 % faster, but the tensor cores line products up by their
// operands' nominal exponents, and a subnormal's is 2^-14 whatever it holds: the
// other 15 columns of an MMA lost up to 10 bits beside a token 2^12 times as
// large (2.4e-5 of sum s (q + z) |x|, 1.7 times the bound).  The zero-point (int3: 4) is
// taken from the group's sum, sum n x - z sum x, with the tokens' sums of
// each group from k_few_prep.  NVFP4: the hardware's E2M1 conversion, then
// dec(e) dec(c) by one f16x2 product (exact: 6 significant bits).
//
// Rounding: every product is exact; a group's sum (NVFP4: a slice's) is taken
// by the tensor cores in fp32, z times the tokens' sum is subtracted and the
// fp32 scale applied by one fma each, and the groups are added in slice order
// per warp and in warp order at the end.
#pragma once

#include <atomic>

#include "codes.cuh"
#include "rows.cuh"
#include "walk.cuh"

namespace tq {

constexpr int FEW_WARPS = 8;

template <int FMT> struct FewFmt;   // g: group; n: groups of a 128-column slice
template <> struct FewFmt<TQ_INT3_G64_SYM> { static constexpr int g = 64, n = 2, rec = 24; };
template <> struct FewFmt<TQ_INT4_G128_ASYM> { static constexpr int g = 128, n = 1, rec = 64; };
template <> struct FewFmt<TQ_INT4_G64_ASYM> { static constexpr int g = 64, n = 2, rec = 32; };
template <> struct FewFmt<TQ_INT4_G32_ASYM> { static constexpr int g = 32, n = 4, rec = 16; };
template <> struct FewFmt<TQ_NVFP4_G16> { static constexpr int g = 16, n = 8, rec = 8; };

__device__ __forceinline__ void few_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// What k_few_prep writes (x_few, x_sums, row_x).  It may still be running when
// this kernel starts, so its results are read after grid_wait() and by
// ordinary loads: the read-only path (__ldg) is for data that nothing writes
// while a kernel runs, and the compiler may move such loads over the wait.
template <typename T>
__device__ __forceinline__ T few_prepared(const T* p) { return *p; }

// What a lane loads of one weight row for one slice.
template <int FMT>
struct FewRaw {
    uint32_t w[4];                                       // codes (int3: low planes in 0, 2, high planes in 1, 3)
    float s[FMT == TQ_NVFP4_G16 ? 1 : FewFmt<FMT>::n];   // scales of the slice's groups
    uint32_t z;                                          // zero-points, or the lane's two E4M3 codes
};

// gi: the weight row's first group of the slice, counted from the start of
// all records; have: groups of the row from there on.  wide: rows start on
// 16-byte boundaries and a slice's per-group values may be read as one word
// (an even number of groups, for g32 a multiple of 4), so a slice needs no
// check of its groups.
template <int FMT>
__device__ __forceinline__ void few_load(FewRaw<FMT>& r, const RowsArgs& a, int proj, uint32_t gi, int have, bool wide,
                                         int tig) {
    using F = FewFmt<FMT>;
    const uint8_t* rec = a.packed[proj] + static_cast<uint64_t>(gi) * F::rec;
    if constexpr (FMT == TQ_NVFP4_G16) {   // this lane's two blocks
        const uint8_t* sc = static_cast<const uint8_t*>(a.scales[proj]) + gi + 2 * tig;
        const bool b0 = 2 * tig < have, b1 = 2 * tig + 1 < have;
        r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0u;
        r.z = 0u;
        if (wide) {
            if (b0) {
                const uint4 v = __ldcs(reinterpret_cast<const uint4*>(rec) + tig);
                r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
                r.z = __ldg(reinterpret_cast<const uint16_t*>(sc));
            }
        } else {
            if (b0) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2*>(rec) + 2 * tig);
                r.w[0] = v.x; r.w[1] = v.y;
                r.z = __ldg(sc);
            }
            if (b1) {
                const uint2 v = __ldcs(reinterpret_cast<const uint2*>(rec) + 2 * tig + 1);
                r.w[2] = v.x; r.w[3] = v.y;
                r.z |= static_cast<uint32_t>(__ldg(sc + 1)) << 8;
            }
        }
    } else {
        const float* sc = static_cast<const float*>(a.scales[proj]) + gi;
        const uint8_t* ze = a.zeros[proj] + gi;
        if constexpr (FMT == TQ_INT4_G128_ASYM) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(rec) + tig);
            r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
            r.s[0] = __ldg(sc);
            r.z = __ldg(ze);
        } else {
            if (wide) {
                if constexpr (F::n == 2) {
                    const float2 v = __ldg(reinterpret_cast<const float2*>(sc));
                    r.s[0] = v.x; r.s[1] = v.y;
                    r.z = is_int4(FMT) ? __ldg(reinterpret_cast<const uint16_t*>(ze)) : 0u;
                } else {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(sc));
                    r.s[0] = v.x; r.s[1] = v.y; r.s[2] = v.z; r.s[3] = v.w;
                    r.z = __ldg(reinterpret_cast<const uint32_t*>(ze));
                }
            } else {
                r.z = 0u;
#pragma unroll
                for (int k = 0; k < F::n; ++k) {   // (a group past the row's end: scale 0, the row's last record)
                    r.s[k] = k < have ? __ldg(sc + k) : 0.f;
                    if (is_int4(FMT)) r.z |= (k < have ? static_cast<uint32_t>(__ldg(ze + k)) : 0u) << (8 * k);
                }
            }
#pragma unroll
            for (int k = 0; k < F::n; ++k) {
                const uint8_t* q = rec + (wide || k < have ? k : 0) * F::rec;
                if constexpr (FMT == TQ_INT4_G64_ASYM) {
                    const uint2 v = __ldcs(reinterpret_cast<const uint2*>(q) + tig);
                    r.w[2 * k] = v.x; r.w[2 * k + 1] = v.y;
                } else if constexpr (FMT == TQ_INT4_G32_ASYM) {
                    r.w[k] = __ldcs(reinterpret_cast<const uint32_t*>(q) + tig);
                } else {
                    r.w[2 * k] = __ldcs(reinterpret_cast<const uint32_t*>(q) + tig);
                    r.w[2 * k + 1] = __ldcs(reinterpret_cast<const uint16_t*>(q + 16) + tig);
                }
            }
        }
    }
}

// Pairs 4 h .. 4 h + 3 of the lane's 16 (rows.cuh) as f16x2; integer formats:
// the codes n times 2^(b - 10), b as few_field() has it.
template <int FMT>
__device__ __forceinline__ void few_decode(const FewRaw<FMT>& r, int h, uint32_t (&p)[4]) {
    constexpr uint32_t UP = 0x74007400u;   // 2^14, twice: normal numbers (see the head of this file)
    if constexpr (FMT == TQ_NVFP4_G16) {   // word h: half a block
        // (a block scale's sign bit is no part of it)
        const uint32_t s = __byte_perm(e4m3x2_f16(r.z & 0x7f7fu), 0u, h < 2 ? 0x1010 : 0x3232);
        e2m1x8_f16(r.w[h], p);
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = f16x2_mul(p[i], s);
    } else if constexpr (FMT == TQ_INT3_G64_SYM) {   // group h / 2, pairs i = 4 (h & 1) ..: codes i and i + 8
        const uint32_t L = r.w[2 * (h >> 1)], H = r.w[2 * (h >> 1) + 1];
        const uint32_t H2 = (H & 0xffu) | (H << 8);   // code i's high bit at i, code i + 8's at 16 + i
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * (h & 1) + i, b = few_field(FMT, n);
            const uint32_t lo = (n < 5 ? L : L >> 10) & (0x00030003u << b);
            const uint32_t hi = b + 2 >= n ? H2 << (b + 2 - n) : H2 >> (n - b - 2);
            p[i] = f16x2_mul(lo | (hi & (0x00040004u << b)), UP);
        }
    } else {   // word h: codes m and m + 4 of its 8, m = 0 .. 3
        const uint32_t w = r.w[h], w8 = w >> 8;
        p[0] = f16x2_mul(w & 0x000f000fu, UP);
        p[1] = f16x2_mul(w & 0x00f000f0u, UP);
        p[2] = f16x2_mul(w8 & 0x000f000fu, UP);
        p[3] = f16x2_mul(w8 & 0x00f000f0u, UP);
    }
}

// A block's items are tiles of weight rows within chunks of 8 NB tokens of one
// matrix, in order; rows_table's counts with NT = 8 NB.
struct FewItem {
    int e, m, row0, n;   // matrix, tile, first token row, token rows
};

// MB: blocks per SM that the registers are kept to (few_blocks_per_sm).
template <int FMT, int NB, int MB>
__global__ void __launch_bounds__(FEW_WARPS * 32, MB)
k_rows_few(const __grid_constant__ RowsArgs a) {
    using F = FewFmt<FMT>;
    constexpr int PD = 2;
    constexpr bool INT = FMT != TQ_NVFP4_G16;
    // the fields' 2^-10, half of it to the sums and half to the tokens' power of
    // two, which goes up to 2^112
    constexpr float HALF_UNIT = INT ? 32.f : 1.f;
    constexpr int VALS = 2 * NB * 4 * 32;   // sums of a warp: 2 tiles of 16 rows x 8 NB tokens
    extern __shared__ float few_smem[];
    float* red = few_smem;                                             // [2][FEW_WARPS][VALS]
    int* table = reinterpret_cast<int*>(few_smem + 2 * FEW_WARPS * VALS);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gid = lane >> 2, tig = lane & 3;
    const bool gated = a.projections == 2;
    // [E + 1] row bounds and [E + 1] chunks before each matrix
    int *off = table, *chunks = table + a.E + 1;
    if (warp == 0) rows_table<8 * NB>(a.offsets, a.E, static_cast<int>(a.R), off, chunks);
    __syncthreads();
    const int64_t items = static_cast<int64_t>(chunks[a.E]) * a.m_tiles;
    const int64_t first = items * blockIdx.x / gridDim.x, last = items * (blockIdx.x + 1) / gridDim.x;
    const int NI = static_cast<int>((a.I + 127) / 128);
    const int G = static_cast<int>(a.G);
    const bool wide = a.few_wide != 0;

    auto item_of = [&](int64_t i) {
        FewItem r;
        const int64_t q = i / a.m_tiles;
        r.m = static_cast<int>(i - q * a.m_tiles);
        int lo = 0, hi = a.E - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (chunks[mid] <= q) lo = mid;
            else hi = mid - 1;
        }
        r.e = lo;
        r.row0 = off[lo] + static_cast<int>(q - chunks[lo]) * 8 * NB;
        r.n = min(off[lo + 1] - r.row0, 8 * NB);
        return r;
    };

    // ks warps share a tile, warp w of them the slices w, w + ks, ...; the
    // block's 8 / ks groups of warps take its tiles in turn
    const int ks = a.few_ks, kw = warp % ks, grp = warp / ks, groups = FEW_WARPS / ks;
    const int gtid = kw * 32 + lane;

    // the load cursor: PD slices ahead of the products
    FewRaw<FMT> raw[PD][2][2];
    uint32_t base[2][2];   // first group of the lane's rows
    int64_t lc_item = first + grp;
    int lc_it = kw;
    auto rows_of = [&](const FewItem& t) {   // rows past the end: the last one again, its sums are not used
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int o = static_cast<int>(a.o_begin) + (gated ? t.m * 16 : t.m * 32 + 16 * tl) + gid + 8 * h;
                base[tl][h] = static_cast<uint32_t>((t.e * a.O + min(o, static_cast<int>(a.o_end) - 1)) * a.G);
            }
    };
    // a tile's two rows of a slot; the second tile's move the cursor on
    auto load = [&](FewRaw<FMT> (&r)[2][2], int tl) {
        if (tl == 0 && lc_it >= NI) {
            lc_it = kw;
            if (lc_item + groups < last) {   // (past the block's last tile: that one again)
                lc_item += groups;
                rows_of(item_of(lc_item));
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            few_load<FMT>(r[tl][h], a, gated ? tl : 0, base[tl][h] + lc_it * F::n, G - lc_it * F::n, wide, tig);
        if (tl == 1) lc_it += ks;
    };
    if (lc_item < last) {
        rows_of(item_of(lc_item));
#pragma unroll
        for (int i = 0; i < PD; ++i) {   // (ks <= NI: every warp has a slice of every tile)
            load(raw[i], 0);
            load(raw[i], 1);
        }
    }
    grid_wait();   // the tokens in fragment order; whatever ran before may still read what this kernel writes

    int slot = 0, turn = 0;
    for (int64_t i = first + grp; i < last; i += groups, turn ^= 1) {
        const FewItem t = item_of(i);
        float y[2][NB][4];
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 4; ++c) y[tl][b][c] = 0.f;
        // this lane's token of each block of 8: its parts of a slice, loaded a
        // slice ahead (a token past the chunk's last reads the last one's; its
        // sums are not used)
        const uint4* xp[NB];
        uint4 x[4][NB];
        // the sums of x over a slice's groups for the tokens of this lane's results
        constexpr int NS = INT ? F::n : 1;
        const float* sp[NB][2];
        float xs[NB][2][NS];
        auto load_sums = [&](int b, int it) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float* sums = sp[b][c] + it * NS;
                if constexpr (NS == 1) {
                    xs[b][c][0] = few_prepared(sums);
                } else if constexpr (NS == 2) {
                    const float2 v = few_prepared(reinterpret_cast<const float2*>(sums));
                    xs[b][c][0] = v.x;
                    xs[b][c][1] = v.y;
                } else {
                    const float4 v = few_prepared(reinterpret_cast<const float4*>(sums));
                    xs[b][c][0] = v.x;
                    xs[b][c][1] = v.y;
                    xs[b][c][2] = v.z;
                    xs[b][c][3] = v.w;
                }
            }
        };
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            xp[b] = reinterpret_cast<const uint4*>(a.x_few) +
                    static_cast<int64_t>(t.row0 + min(8 * b + gid, t.n - 1)) * NI * 16 + tig;
#pragma unroll
            for (int h = 0; h < 4; ++h) x[h][b] = few_prepared(xp[b] + kw * 16 + 4 * h);
            if (INT) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    sp[b][c] = a.x_sums + static_cast<int64_t>(t.row0 + min(8 * b + 2 * tig + c, t.n - 1)) * NI * NS;
                load_sums(b, kw);
            }
        }
        // (No branch in a slice: loads past the end are of the last slice
        // again, so that the compiler may mix all of its instructions.)
        auto slice = [&](FewRaw<FMT> (&r)[2][2], int it) {
            const int ahead = min(it + ks, NI - 1);
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
                constexpr int PER = INT ? 4 / F::n : 4;   // quarters of a slice in a group (NVFP4: the slice)
                float d[NB][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {   // a quarter: 2 MMAs, pairs 4 h .. 4 h + 3
                    if (h % PER == 0) {
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int c = 0; c < 4; ++c) d[b][c] = 0.f;
                    }
                    uint32_t p0[4], p1[4];
                    few_decode<FMT>(r[tl][0], h, p0);
                    few_decode<FMT>(r[tl][1], h, p1);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        few_mma(d[b], p0[0], p1[0], p0[1], p1[1], x[h][b].x, x[h][b].y);
                        few_mma(d[b], p0[2], p1[2], p0[3], p1[3], x[h][b].z, x[h][b].w);
                        if (tl == 1) x[h][b] = few_prepared(xp[b] + ahead * 16 + 4 * h);
                    }
                    if (!INT && h == 3) {
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int c = 0; c < 4; ++c) y[tl][b][c] = __fadd_rn(y[tl][b][c], d[b][c]);
                    }
                    if (INT && h % PER == PER - 1) {
                        const int k = INT ? h / PER : 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {   // weight rows gid and gid + 8
                            const float sc = r[tl][e].s[INT ? k : 0];
                            // -z: 2^23 - (2^23 + z), exactly
                            const float z = FMT == TQ_INT3_G64_SYM
                                                ? -4.f
                                                : 8388608.f - __uint_as_float(0x4b000000u | ((r[tl][e].z >> (8 * k)) & 0xffu));
#pragma unroll
                            for (int b = 0; b < NB; ++b)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    y[tl][b][2 * e + c] =
                                        __fmaf_rn(sc, __fmaf_rn(z, xs[b][c][INT ? k : 0], d[b][2 * e + c]), y[tl][b][2 * e + c]);
                        }
                    }
                }
                load(r, tl);
            }
            if (INT) {
#pragma unroll
                for (int b = 0; b < NB; ++b) load_sums(b, ahead);
            }
        };
        for (int it = kw; it < NI; it += ks) {
            if (slot == 0) slice(raw[0], it);
            else slice(raw[1], it);
            slot ^= 1;
        }
        // the warps' sums: lane (gid, tig) holds token 8 b + 2 tig + (c & 1), row gid + 8 (c >> 1) of tile tl
        float* rd = red + (turn * FEW_WARPS + grp * ks) * VALS;
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 4; ++c) rd[kw * VALS + ((tl * NB + b) * 4 + c) * 32 + lane] = y[tl][b][c];
        asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(ks * 32) : "memory");
        auto sum = [&](int tl, int tok, int r) {   // the joined sum of token tok, row r of tile tl
            const int at = ((tl * NB + (tok >> 3)) * 4 + (tok & 1) + 2 * (r >> 3)) * 32 + (r & 7) * 4 + ((tok & 7) >> 1);
            float v = rd[at];
            for (int w = 1; w < ks; ++w) v = __fadd_rn(v, rd[w * VALS + at]);
            return v;
        };
        if (gated) {
            const bool grad = a.mode == ROWS_GATED_BWD;
            const RowsBound wm = grad ? rows_bound_wm<FMT>(a, t.e, rows_wmax(a, t.e, lane)) : RowsBound{};
            for (int v = gtid; v < 16 * 8 * NB; v += ks * 32) {
                const int tok = v >> 4, r = v & 15;
                const int64_t f = static_cast<int64_t>(t.m) * 16 + r;
                if (tok < t.n && f < a.O) {
                    const float sx = few_prepared(a.row_x + t.row0 + tok) * HALF_UNIT;
                    // (NVFP4: the global scale before the tokens' power of two, with which alone the sum may overflow)
                    const float g = sum(0, tok, r) * (INT ? HALF_UNIT : __ldg(a.gs[0] + t.e)) * sx;
                    const float u = sum(1, tok, r) * (INT ? HALF_UNIT : __ldg(a.gs[1] + t.e)) * sx;
                    const int64_t tr = t.row0 + tok;
                    const ActGrad w = rw_act(rw_act_coef(a.act), g);
                    if (!grad) {
                        rows_put(a.y, tr * a.ldy + f, a.y_bf16, w.a * u);
                    } else {   // as the other kernel's: D beside the token's power of two
                        const float s0 = INT ? 1.f : __ldg(a.gs[0] + t.e), s1 = INT ? 1.f : __ldg(a.gs[1] + t.e);
                        const float dh = bf16_bits_to_f32(__ldg(a.dh + tr * a.ld_dh + f)) *
                                         (gated_bound(__ldg(a.row_f + tr), wm, sqrtf(static_cast<float>(a.I))).inv * 16384.f);
                        uint16_t* d = a.D + tr * a.ldd + f;
                        d[0] = __half_as_ushort(__float2half_rn((dh * u) * (w.d * s0)));
                        d[a.R * a.ldd] = __half_as_ushort(__float2half_rn((dh * w.a) * s1));
                    }
                }
            }
        } else {
            for (int v = gtid; v < 32 * 8 * NB; v += ks * 32) {   // a warp: one token
                const int tok = v >> 5, r = v & 31;
                const int64_t o = a.o_begin + static_cast<int64_t>(t.m) * 32 + r;
                const bool live = tok < t.n && o < a.o_end;
                const float z = live ? sum(r >> 4, tok, r & 15) * (INT ? HALF_UNIT : __ldg(a.gs[0] + t.e)) *
                                           (few_prepared(a.row_x + t.row0 + tok) * HALF_UNIT)
                                     : 0.f;
                if (a.mode == ROWS_STORE) {
                    if (live) rows_put(a.y, (t.row0 + tok) * a.ldy + o, a.y_bf16, z);
                } else if (a.mode == ROWS_PROB) {
                    if (live) {
                        const int64_t tr = t.row0 + tok, l = __ldg(a.labels + tr);
                        float w = rw_exp(z - __ldg(a.lse + tr));
                        w = l < 0 || l >= a.O ? 0.f : l == o ? w - 1.f : w;
                        a.D[tr * a.ldd + (o - a.o_begin)] = __half_as_ushort(__float2half_rn(w * ROWS_PROB_SCALE));
                    }
                } else if (tok < t.n) {   // the loss
                    const int64_t tr = t.row0 + tok;
                    if (live && __ldg(a.labels + tr) == o) a.label_z[tr] = z;
                    float m = live ? z : -INFINITY;
#pragma unroll
                    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, k));
                    if (m == -INFINITY) m = 0.f;
                    float s = live ? rw_exp(z - m) : 0.f;
#pragma unroll
                    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(FULL, s, k);
                    // (no sum: all of the tile's logits are -inf, and the 0 above is no largest that others join)
                    if (r == 0) a.part[static_cast<int64_t>(t.m) * a.R + tr] = make_float2(s == 0.f ? -3.0e38f : m, s);
                }
            }
        }
    }
}

template <int FMT, int NB, int MB>
tq_status few_launch(const RowsArgs& a, int grid_most, cudaStream_t st) {
    constexpr int SUMS = 2 * FEW_WARPS * 2 * NB * 4 * 32 * 4;
    const int smem = SUMS + 2 * (a.E + 1) * 4;
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(k_rows_few<FMT, NB, MB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   SUMS + 2 * (ROWS_MAX_MATS + 1) * 4);
        if (e != cudaSuccess) return set_error(TQ_ERR_CUDA, "row products: %s", cudaGetErrorString(e));
        ready.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(grid_most));
    cfg.blockDim = dim3(FEW_WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // starts while the tokens are still being put in order; its first records
    // are in flight when they are
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, k_rows_few<FMT, NB, MB>, a);
    return check_launch("row products");
}

template <int FMT>
tq_status few_launch_nb(const RowsArgs& a, int nb, int mb, int grid, cudaStream_t st) {
    switch (nb) {
        case 1: return few_launch<FMT, 1, 2>(a, grid, st);
        case 2:
            if constexpr (few_two_fit(FMT))
                if (mb == 2) return few_launch<FMT, 2, 2>(a, grid, st);
            return few_launch<FMT, 2, 1>(a, grid, st);
        default: return few_launch<FMT, 4, 1>(a, grid, st);
    }
}

}  // namespace tq
