// Host entry points of the products with the packed records (tq_dequant_matmul,
// tq_gated_ffn, tq_head_loss and their gradients) and the small kernels
// around the tensor-core ones of rows_core.cuh.
#include <atomic>
#include <mutex>

#include "rows.cuh"

namespace tq {

// ------------------------------------------------------------------ before: row factors and the matrices' largest values

constexpr int PREP_THREADS = 256;

__device__ __forceinline__ float block_max(float v) {   // v >= 0 or NaN; NaN counts as the largest
    __shared__ unsigned m[PREP_THREADS / 32];
    unsigned u = __reduce_max_sync(FULL, __float_as_uint(fabsf(v)));
    if ((threadIdx.x & 31) == 0) m[threadIdx.x >> 5] = u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PREP_THREADS / 32; ++i) u = max(u, m[i]);
    __syncthreads();
    return __uint_as_float(u);
}

__device__ __forceinline__ float block_sum(float v) {   // in a fixed order
    __shared__ float m[PREP_THREADS / 32];
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(FULL, v, off);
    if ((threadIdx.x & 31) == 0) m[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < PREP_THREADS / 32; ++i) v += m[i];
    __syncthreads();
    return v;
}

struct PrepArgs {
    int64_t rows;                  // blocks 0 .. rows - 1: one token row each
    const uint16_t* src;           // bf16 rows [rows][src_ld] of src_cols to copy as f16, scaled per row
    int64_t src_cols, src_ld;
    int order;                     // the copy's column order within 16: a format's (rows_column), or 0: as it is
    uint16_t* f16;                 // the copy, [rows][up16(src_cols)], or null
    float* f16_f;                  // its power of two per row
    const uint16_t* dh;            // gated backward: bf16 gradient rows, else null
    int64_t dh_cols, dh_ld;
    float* row_f;                  // gated backward: |dh|max |src|2
    // the blocks after them: parts of the matrices' scales
    const void* scales[2];
    const uint8_t* zeros[2];       // int4, else null
    int64_t per_mat;               // scales of a matrix
    int E, e4m3;
    float* wmax;                   // [projections][E][rows_wmax_parts(E)]
};

// Words of 8 values of a bf16 row, whatever its alignment; past its end, 0.
struct RowReader {
    const uint16_t* p;
    int64_t n;
    bool wide;   // 16-byte aligned
    __device__ RowReader(const uint16_t* row, int64_t cols)
        : p(row), n(cols), wide((reinterpret_cast<uintptr_t>(row) & 15) == 0) {}
    __device__ __forceinline__ int64_t words() const { return (n + 7) / 8; }
    __device__ __forceinline__ uint4 word(int64_t i) const {
        if (wide && 8 * i + 8 <= n) return __ldg(reinterpret_cast<const uint4*>(p) + i);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t j = 8 * i + 2 * k;
            w[k] = (j < n ? __ldg(p + j) : 0u) | (j + 1 < n ? static_cast<uint32_t>(__ldg(p + j + 1)) << 16 : 0u);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The largest of a row's bf16 magnitudes (as fp32).
__device__ __forceinline__ float row_amax(const RowReader& row) {
    unsigned m = 0;   // bf16 magnitudes order as integers; two per word
    for (int64_t i = threadIdx.x; i < row.words(); i += PREP_THREADS) {
        const uint4 v = row.word(i);
        m = __vmaxu2(__vmaxu2(m, __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu)),
                     __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    }
    return block_max(bf16_bits_to_f32(static_cast<uint16_t>(max(m & 0xffffu, m >> 16))));
}

__global__ void __launch_bounds__(PREP_THREADS) k_rows_prep(const __grid_constant__ PrepArgs a) {
    if (blockIdx.x >= a.rows) {   // a part of a matrix's scales
        const int64_t b = blockIdx.x - a.rows;
        const int parts = rows_wmax_parts(a.E), part = static_cast<int>(b % parts);
        const int64_t pe = b / parts;
        const int proj = static_cast<int>(pe / a.E);
        const int64_t e = pe - static_cast<int64_t>(proj) * a.E;
        const int64_t lo = a.per_mat * part / parts, hi = a.per_mat * (part + 1) / parts;
        float m = 0.f;
        if (a.e4m3) {
            const uint8_t* s = static_cast<const uint8_t*>(a.scales[proj]) + e * a.per_mat;
            const uint8_t *p0 = s + lo, *p1 = s + hi;
            // whole words between the ends, four codes at a time
            const uint8_t* q0 = reinterpret_cast<const uint8_t*>((reinterpret_cast<uintptr_t>(p0) + 3) & ~uintptr_t(3));
            const uint8_t* q1 = reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(p1) & ~uintptr_t(3));
            unsigned c = 0;
            if (q0 < q1) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(q0);
                const int64_t n = (q1 - q0) / 4;
                for (int64_t i = threadIdx.x; i < n; i += 4 * PREP_THREADS) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        c = __vmaxu4(c, __ldg(w + min(i + k * PREP_THREADS, n - 1)) & 0x7f7f7f7fu);
                }
                c = max(max(c & 0xffu, (c >> 8) & 0xffu), max((c >> 16) & 0xffu, c >> 24));
            } else {
                q0 = q1 = p1;
            }
            if (p0 + threadIdx.x < q0) c = max(c, __ldg(p0 + threadIdx.x) & 0x7fu);   // (at most 3, or 7 in all)
            if (q1 + threadIdx.x < p1) c = max(c, __ldg(q1 + threadIdx.x) & 0x7fu);
            m = e4m3_value(c);
        } else {
            // |s| times the furthest a code may be from the zero-point (int4:
            // 0 .. 15, and a zero-point is any byte; int3: -4 .. 3).  Four at a
            // time between the ends: with one a load 1999 rows over 16 int3
            // experts took 329 us, so 314.
            const float* s = static_cast<const float*>(a.scales[proj]) + e * a.per_mat;
            const uint8_t* z = a.zeros[proj] ? a.zeros[proj] + e * a.per_mat : nullptr;
            const float *p0 = s + lo, *p1 = s + hi;
            const float* q0 = reinterpret_cast<const float*>((reinterpret_cast<uintptr_t>(p0) + 15) & ~uintptr_t(15));
            const float* q1 = reinterpret_cast<const float*>(reinterpret_cast<uintptr_t>(p1) & ~uintptr_t(15));
            auto far4 = [&](uint32_t zz) { return z ? __vmaxu4(zz, __vsubus4(0x0f0f0f0fu, zz)) : 0x04040404u; };
            auto take = [&](float v, uint32_t far) {   // (an infinite or NaN scale is its own groups' matter)
                constexpr float MOST = 3.4028234e38f;
                v = fabsf(v);
                m = v <= MOST ? fmaxf(m, fminf(v * static_cast<float>(far & 0xffu), MOST)) : m;
            };
            if (q0 < q1) {
                const float4* w = reinterpret_cast<const float4*>(q0);
                const uint8_t* zw = z ? z + (q0 - s) : nullptr;
                const bool words = (reinterpret_cast<uintptr_t>(zw) & 3) == 0;
                const int64_t n = (q1 - q0) / 4;
                for (int64_t i = threadIdx.x; i < n; i += 4 * PREP_THREADS) {
                    float4 v[4];
                    uint32_t zz[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t j = min(i + k * PREP_THREADS, n - 1);
                        v[k] = __ldg(w + j);
                        if (!z) zz[k] = 0u;
                        else if (words) zz[k] = __ldg(reinterpret_cast<const uint32_t*>(zw) + j);
                        else
                            zz[k] = __ldg(zw + 4 * j) | (__ldg(zw + 4 * j + 1) << 8) | (__ldg(zw + 4 * j + 2) << 16) |
                                    (static_cast<uint32_t>(__ldg(zw + 4 * j + 3)) << 24);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t far = far4(zz[k]);
                        take(v[k].x, far);
                        take(v[k].y, far >> 8);
                        take(v[k].z, far >> 16);
                        take(v[k].w, far >> 24);
                    }
                }
            } else {
                q0 = q1 = p1;
            }
            auto one = [&](const float* p) { take(__ldg(p), far4(z ? __ldg(z + (p - s)) : 0u)); };
            if (p0 + threadIdx.x < q0) one(p0 + threadIdx.x);   // (at most 3, or 7 in all)
            if (q1 + threadIdx.x < p1) one(q1 + threadIdx.x);
        }
        m = block_max(m);
        if (threadIdx.x == 0) a.wmax[b] = m;
        return;
    }
    const int64_t r = blockIdx.x;
    const RowReader d(a.src + r * a.src_ld, a.src_cols);
    const Pow2 c = pow2_of(row_amax(d));
    if (a.dh) {
        const float amax = row_amax(RowReader(a.dh + r * a.dh_ld, a.dh_cols));
        float s = 0.f;   // of the squares beside the row's power of two: the squares alone may leave fp32
        for (int64_t i = threadIdx.x; i < d.words(); i += PREP_THREADS) {
            const uint4 v = d.word(i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float lo = __uint_as_float(w[k] << 16) * c.inv, hi = __uint_as_float(w[k] & 0xffff0000u) * c.inv;
                s = fmaf(lo, lo, fmaf(hi, hi, s));
            }
        }
        s = block_sum(s);
        // (a hair above the norm, whatever the sum's rounding; and a normal
        // number, so that what it is multiplied by later does not uncover a
        // product rounded to 0 here)
        if (threadIdx.x == 0) a.row_f[r] = fmaxf(amax * (sqrtf(s) * 1.0001f * c.p), 1.1754944e-38f);
    }
    if (a.f16 == nullptr) return;
    if (threadIdx.x == 0) a.f16_f[r] = c.p * 6.103515625e-05f;   // 2^-14
    const float f = c.inv * 16384.f;
    const int64_t units = (a.src_cols + 15) / 16;
    uint4* D = reinterpret_cast<uint4*>(a.f16) + r * units * 2;
    for (int64_t i = threadIdx.x; i < units; i += PREP_THREADS) {
        const uint4 v0 = d.word(2 * i), v1 = d.word(2 * i + 1);
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        float v[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16) * f;
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * f;
        }
        uint32_t q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float lo = v[2 * k], hi = v[2 * k + 1];
            if (is_int4(a.order)) {
                lo = v[8 * (k >> 2) + (k & 3)];
                hi = v[8 * (k >> 2) + (k & 3) + 4];
            } else if (a.order == TQ_INT3_G64_SYM) {
                lo = v[k];
                hi = v[k + 8];
            }
            const __half2 h = __floats2half2_rn(lo, hi);
            memcpy(&q[k], &h, 4);
        }
        D[2 * i] = make_uint4(q[0], q[1], q[2], q[3]);
        D[2 * i + 1] = make_uint4(q[4], q[5], q[6], q[7]);
    }
}

// ------------------------------------------------------------------ before: few tokens

// A token row as f16 beside a power of two (its largest in [2^14, 2^15)), in
// that kernel's order: slice, quarter, lane, four pairs.  A thread takes
// 16 columns, which are whole pairs in every format's order and fill two units
// of 16 bytes, and keeps its first 16 in registers between the row's maximum
// and the copy.
constexpr int FEW_PREP_THREADS = 512;
__global__ void __launch_bounds__(FEW_PREP_THREADS) k_few_prep(const uint16_t* x, int64_t ld, int64_t I, int fmt,
                                                               uint16_t* out, float* row_x, float* sums) {
    __shared__ unsigned part[FEW_PREP_THREADS / 32];
    // the products may be launched now: they wait for this grid before they read it
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t r = blockIdx.x;
    const RowReader row(x + r * ld, I);
    const int tid = static_cast<int>(threadIdx.x), chunks = static_cast<int>((I + 127) / 128) * 8;
    auto amax = [](uint4 v) {
        return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    };
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    unsigned m = 0;   // bf16 magnitudes order as integers; two per word
    for (int c = tid; c < chunks; c += FEW_PREP_THREADS) {
        const uint4 v = row.word(2 * c), w = row.word(2 * c + 1);   // (words past the row are 0)
        m = __vmaxu2(m, __vmaxu2(amax(v), amax(w)));
        if (c == tid) {
            a = v;
            b = w;
        }
    }
    m = max(m & 0xffffu, m >> 16);
    m = __reduce_max_sync(FULL, m);
    if ((tid & 31) == 0) part[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < FEW_PREP_THREADS / 32; ++i) m = max(m, part[i]);
    const Pow2 p = pow2_of(bf16_bits_to_f32(static_cast<uint16_t>(m)));
    if (tid == 0) row_x[r] = p.p * 6.103515625e-05f;   // 2^-14
    const float f = p.inv * 16384.f;
    uint4* o = reinterpret_cast<uint4*>(out) + r * chunks * 2;
    const int per = fmt == TQ_INT4_G128_ASYM ? 8 : fmt == TQ_INT4_G32_ASYM ? 2 : 4;   // 16 columns x per: a group
    for (int c = tid; c - (tid & 31) < chunks; c += FEW_PREP_THREADS) {   // whole warps
        if (c != tid) {
            a = row.word(2 * c);
            b = row.word(2 * c + 1);
        }
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16) * f;
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * f;
        }
        if (fmt != TQ_NVFP4_G16) {   // the group's sum of the values as f16 holds them
            float g = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) g += __half2float(__float2half_rn(v[i]));
            for (int k = 1; k < per; k *= 2) g += __shfl_xor_sync(FULL, g, k);
            if (c < chunks && (c & (per - 1)) == 0) sums[(r * chunks + c) / per] = g * 9.765625e-04f;   // 2^-10
        }
        if (c >= chunks) continue;
        // the two units' pairs: int4 (k, k + 4) of each 8, int3 (k, k + 8) of the 16, NVFP4 (2 k, 2 k + 1)
        uint32_t q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float lo, hi;
            if (fmt == TQ_INT3_G64_SYM) {
                lo = v[i];
                hi = v[i + 8];
            } else if (fmt == TQ_NVFP4_G16) {
                lo = v[2 * i];
                hi = v[2 * i + 1];
            } else {
                lo = v[8 * (i >> 2) + (i & 3)];
                hi = v[8 * (i >> 2) + (i & 3) + 4];
            }
            const float k = fmt == TQ_NVFP4_G16 ? 1.f
                            : fmt == TQ_INT3_G64_SYM ? 1.f / static_cast<float>(1 << few_field(TQ_INT3_G64_SYM, i))
                                                     : 1.f / static_cast<float>(1 << few_field(TQ_INT4_G128_ASYM, i));
            const __half2 h = __floats2half2_rn(lo * k, hi * k);
            memcpy(&q[i], &h, 4);
        }
        // where they go: slice, quarter, lane
        const int j = c & 7;
        int u0, u1;
        if (fmt == TQ_INT4_G128_ASYM || fmt == TQ_NVFP4_G16) {   // lane j / 2, quarters 2 (j & 1) and the next
            u0 = 8 * (j & 1) + (j >> 1);
            u1 = u0 + 4;
        } else if (fmt == TQ_INT4_G32_ASYM) {                    // quarter j / 2, lanes 2 (j & 1) and the next
            u0 = 4 * (j >> 1) + 2 * (j & 1);
            u1 = u0 + 1;
        } else {                                                 // quarters 2 (j / 4) and the next, lane j % 4
            u0 = 8 * (j >> 2) + (j & 3);
            u1 = u0 + 4;
        }
        uint4* s = o + (c >> 3) * 16;
        s[u0] = make_uint4(q[0], q[1], q[2], q[3]);
        s[u1] = make_uint4(q[4], q[5], q[6], q[7]);
    }
}

// ------------------------------------------------------------------ after: joined sums

// dx = the splits' sums added in order, rounded once; rows outside the
// offsets stay as they were.
__global__ void __launch_bounds__(256) k_rows_join(const float* sums, int splits, int64_t R, int64_t I,
                                                   const int32_t* offsets, int E, uint16_t* dx, int64_t ldx) {
    const int64_t r = blockIdx.x;
    if (offsets) {
        __shared__ int last;
        if (threadIdx.x == 0) last = 0;
        __syncthreads();
        int m = 0;
        for (int i = threadIdx.x; i <= E; i += blockDim.x) m = max(m, __ldg(offsets + i));
        m = __reduce_max_sync(FULL, m);
        if ((threadIdx.x & 31) == 0) atomicMax(&last, m);
        __syncthreads();
        if (r < __ldg(offsets) || r >= last) return;
    }
    for (int64_t j = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x; j < I; j += 256 * gridDim.y) {
        float v = __ldg(sums + r * I + j);
        for (int s = 1; s < splits; ++s) v += __ldg(sums + (static_cast<int64_t>(s) * R + r) * I + j);
        dx[r * ldx + j] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

// lse and loss, a block per token: thread i joins the tiles i, i + 256, ...,
// then the threads' pairs are joined along a fixed tree.
__global__ void __launch_bounds__(256) k_loss_join(const float2* part, int m_tiles, int64_t R, const int64_t* labels,
                                                   int64_t V, const float* label_z, float* loss, float* lse) {
    __shared__ float2 w8[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    auto join = [](float2 a, float2 b) {   // (max, sum of e^(z - max)) of two sets
        const float m = fmaxf(a.x, b.x);
        return make_float2(m, a.y * expf(a.x - m) + b.y * expf(b.x - m));
    };
    // a thread's pairs four at a time: their largest, then one exponential each
    float2 s = make_float2(-3.0e38f, 0.f);
    for (int i = threadIdx.x; i < m_tiles; i += 1024) {
        float2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = i + 256 * k < m_tiles ? __ldg(part + static_cast<int64_t>(i + 256 * k) * R + t)
                                         : make_float2(-3.0e38f, 0.f);
        const float m = fmaxf(fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x)), s.x);
        float sum = s.y * expf(s.x - m);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += v[k].y * expf(v[k].x - m);
        s = make_float2(m, sum);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1)
        s = join(s, make_float2(__shfl_xor_sync(FULL, s.x, k), __shfl_xor_sync(FULL, s.y, k)));
    if (lane == 0) w8[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 8; ++i) s = join(s, w8[i]);
        const float l = s.x + logf(s.y);
        lse[t] = l;
        const int64_t lab = __ldg(labels + t);
        loss[t] = lab >= 0 && lab < V ? l - __ldg(label_z + t) : 0.f;
    }
}

// ------------------------------------------------------------------ host

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn rows_encode() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Token rows [planes][rows][ld] of `cols` f16 values, in boxes of 64
// columns x nt rows.
static tq_status rows_map(CUtensorMap* map, const void* p, int64_t cols, int64_t rows, int64_t ld,
                          int64_t planes, int nt) {
    EncodeTiledFn enc = rows_encode();
    if (!enc) return set_error(TQ_ERR_CUDA, "row products: cuTensorMapEncodeTiled unavailable");
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>(rows * ld * 2)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows_pair(nt) ? nt / 2 : nt), 1}, estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                           const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return set_error(TQ_ERR_CUDA, "row products: tensor map encoding failed (%d)", static_cast<int>(r));
    return TQ_OK;
}

static tq_status launch_rows(int32_t fmt, const RowsArgs& a, const RowsLaunch& l, cudaStream_t st) {
    switch (fmt) {
        case TQ_INT3_G64_SYM: return launch_rows_int3(a, l, st);
        case TQ_INT4_G128_ASYM: return launch_rows_int4g128(a, l, st);
        case TQ_INT4_G64_ASYM: return launch_rows_int4g64(a, l, st);
        case TQ_INT4_G32_ASYM: return launch_rows_int4g32(a, l, st);
        default: return launch_rows_nvfp4(a, l, st);
    }
}

bool rows_take_timeouts() {
    // (every format's count is read and cleared)
    return rows_int3_take_timeouts() | rows_int4g128_take_timeouts() | rows_int4g64_take_timeouts() |
           rows_int4g32_take_timeouts() | rows_nvfp4_take_timeouts();
}

// Tokens per tile and splits of the sum by a model of the SMs' time in clocks:
// waves of items x (steps x clocks of a step + clocks of an item's start and
// end), plus the traffic of joined splits.  A step's clocks are relative ones,
// one table for every format and kind.  Against runs with each width forced
// (matmul in bf16 and fp32, loss, gated block and both gradients, 4096 columns,
// all formats) the choice was within 2 % of the fastest for one matrix of 6000
// outputs and 40 to 2500 rows (150 runs), and within 5 % for 71 of 100 runs of
// routed rows; the others, 25 to 48 rows a matrix, took up to 1.28 times as long
// as a width less would have, fp32 outputs of int4 g32 1.55.  Microseconds of 32
// / 64 / 128 / 256 tokens a tile: 1999 rows over 16 int3 experts (gated, 2048
// outputs) 481 / 298 / 189 / 173; a gated gradient of 777 rows over them 486 /
// 290 / 309 / 338 (128 is taken); one int4 g64 matrix of 6000 outputs, 100 rows
// 65 / 41 / 43 / 47, 300 rows 112 / 66 / 45 / 48, 1300 rows 342 / 189 / 122 /
// 80; its loss, 300 rows 130 / 108 / 71 / 80.
struct RowsPlan {
    int nt, splits, grid;
};

static int64_t tiles_of(int64_t n, int64_t t) { return (n + t - 1) / t; }

// m128: tiles of 128 weight rows (columns).
static RowsPlan rows_plan(int64_t m128, int64_t R, int64_t E, int64_t steps, bool may_split, int64_t I) {
    static const int NT[4] = {32, 64, 128, 256}, STEP[4] = {520, 640, 730, 880}, ITEM[4] = {1500, 1800, 2500, 3500};
    static const int SPLITS[8] = {1, 2, 3, 4, 6, 8, 12, 16};
    const int64_t sms = num_sms();
    RowsPlan best{32, 1, 1};
    double least = 0;
    for (int i = 0; i < 4; ++i) {
        // (routed rows: half a tile more per matrix than its share of rows
        // fills, at least one, but no more tiles than rows)
        int64_t n = tiles_of(R, NT[i]);
        if (E > 1) {
            const double per = static_cast<double>(R) / static_cast<double>(E) / NT[i] + 0.5;
            n = static_cast<int64_t>(static_cast<double>(E) * (per > 1 ? per : 1));
            if (n > R) n = R;
        }
        const int cg = rows_pair(NT[i]) ? 2 : 1;
        const int64_t m = tiles_of(m128, cg), slots = sms / cg;
        for (int s : SPLITS) {
            if (s > 1 && (!may_split || steps / s < 8)) break;
            const double waves = static_cast<double>(tiles_of(m * n * s, slots));
            const double join = s > 1 ? 3000 + static_cast<double>(R) * I * 8 * s / 3000 : 0;
            const double t = waves * (static_cast<double>((steps + s - 1) / s) * STEP[i] + ITEM[i]) + join;
            if (least == 0 || t < least) {
                least = t;
                best.nt = NT[i];
                best.splits = s;
            }
        }
    }
    const int cg = rows_pair(best.nt) ? 2 : 1;
    const int64_t items = tiles_of(m128, cg) * (tiles_of(R, best.nt) + (E > 1 ? (R < E ? R : E) : 0)) * best.splits;
    const int64_t slots = sms / cg;
    best.grid = cg * static_cast<int>(items < slots ? (items < 1 ? 1 : items) : slots);
    return best;
}


// Workspace regions, each on a 256-byte boundary.
struct Carve {
    uint8_t* base;
    size_t used = 0;
    explicit Carve(void* p) : base(static_cast<uint8_t*>(p)) {}
    template <typename T> T* take(int64_t n) {
        T* p = reinterpret_cast<T*>(base + used);
        used += (static_cast<size_t>(n) * sizeof(T) + 255) & ~size_t(255);
        return p;
    }
};

static int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }

static tq_status check_records(const tq_records* W, const char* name) {
    TQ_REQUIRE(W != nullptr, "%s: null descriptor", name);
    if (group_of(W->fmt) == 0) return set_error(TQ_ERR_UNSUPPORTED, "%s: unknown format %d", name, W->fmt);
    TQ_REQUIRE(W->packed && W->scales, "%s: null packed or scales pointer", name);
    TQ_REQUIRE(aligned16(W->packed), "%s: packed not 16-byte aligned", name);
    TQ_REQUIRE(!is_int4(W->fmt) || W->zeros, "%s: int4 needs zeros", name);
    TQ_REQUIRE(is_int4(W->fmt) || !W->zeros, "%s: zeros are for int4 only", name);
    TQ_REQUIRE(W->fmt != TQ_NVFP4_G16 || W->global_scale, "%s: NVFP4 needs global_scale", name);
    TQ_REQUIRE(W->fmt == TQ_NVFP4_G16 || !W->global_scale, "%s: global_scale is for NVFP4 only", name);
    TQ_REQUIRE(W->fmt == TQ_NVFP4_G16 || (reinterpret_cast<uintptr_t>(W->scales) & 3u) == 0,
               "%s: scales not 4-byte aligned", name);
    TQ_REQUIRE((reinterpret_cast<uintptr_t>(W->global_scale) & 3u) == 0, "%s: global_scale not 4-byte aligned", name);
    TQ_REQUIRE(W->n_mat >= 1 && W->O >= 1 && W->I >= 1, "%s: empty or negative shape", name);
    TQ_REQUIRE(W->n_mat <= ROWS_MAX_MATS, "%s: more than %d matrices", name, ROWS_MAX_MATS);
    TQ_REQUIRE(W->O < (int64_t(1) << 30) && W->I < (int64_t(1) << 30) &&
                   W->n_mat * W->O < (int64_t(1) << 32) / ((W->I + group_of(W->fmt) - 1) / group_of(W->fmt)),
               "%s: more than 2^32 groups", name);
    return TQ_OK;
}

// bf16 token rows: [rows][ld] of `cols`, one matrix; rows may be 0.  No
// alignment beyond an element's: the kernels that prepare them read any.
static tq_status check_tokens(const tq_mat* X, int64_t rows, int64_t cols, const char* name) {
    TQ_REQUIRE(X != nullptr, "%s: null descriptor", name);
    if (X->dtype != TQ_BF16) return set_error(TQ_ERR_UNSUPPORTED, "%s: only bf16 is supported", name);
    TQ_REQUIRE(X->n_mat == 1, "%s: one matrix of token rows expected", name);
    TQ_REQUIRE(X->rows >= 0 && X->rows < (int64_t(1) << 30), "%s: rows out of range", name);
    TQ_REQUIRE(rows < 0 || X->rows == rows, "%s: %lld rows, expected %lld", name, (long long)X->rows, (long long)rows);
    TQ_REQUIRE(X->cols == cols, "%s: %lld columns, expected %lld", name, (long long)X->cols, (long long)cols);
    if (X->rows == 0) return TQ_OK;
    TQ_REQUIRE(X->ptr != nullptr && (reinterpret_cast<uintptr_t>(X->ptr) & 1u) == 0, "%s: null or misaligned data pointer",
               name);
    TQ_REQUIRE(X->ld >= X->cols, "%s: ld (%lld) < cols (%lld)", name, (long long)X->ld, (long long)X->cols);
    return TQ_OK;
}

#define ROWS_TRY(call)                      \
    do {                                    \
        const tq_status s_ = (call);        \
        if (s_ != TQ_OK) return s_;         \
    } while (0)

// Tokens (in blocks of 8) that the kernel for few tokens should take at a
// time, or 0 where the tensor-memory kernel is the faster one: by the rows of
// a matrix (routed: on average).  Microseconds, few / tensor-memory (the same
// records again and again, in L2 where they fit):
//  fewer tiles than SMs: up to 32 rows.  32 rows x 8192 x 4096, int3 32 / 43,
//    int4 g32 36 / 44, NVFP4 24 / 33; 53 rows over 2 int3 experts 24 / 43.
//  one matrix, more tiles: up to 16, int4 g128 up to 32.  Gated 17408 x 5120,
//    16 rows, int3 73 / 84, g128 46 / 80, g64 60 / 87, g32 82 / 99, NVFP4 46 /
//    69; 24 rows 92 / 86, 70 / 79, 84 / 87, 120 / 100, 66 / 69.
//  experts: their ragged ends fill fewer blocks of 8, which the tensor-memory
//    kernel pads for nothing.  64 x 2688 x 1856, 8 rows each, int3 102 / 130,
//    g128 73 / 143, g64 115 / 149, NVFP4 77 / 116; 12 rows int3 139 / 130, g64
//    171 / 150; 16 rows g128 101 / 146, NVFP4 99 / 118; 24 rows g128 162 / 146,
//    NVFP4 153 / 118.  g32 spills at 8 tokens (few_blocks_per_sm), hence its
//    limits: 64 x 2688 x 2048, 4 rows 153 / 175, 8 rows 158 / 176 (not taken);
//    where rows do not end with a slice, 2688 x 1856, 2 rows 171 / 162, 8 rows
//    199 / 163.
static int few_blocks(int32_t fmt, const RowsArgs& a) {
    const int64_t per = (a.R + a.E - 1) / a.E, tiles = a.E * tiles_of(a.O, a.projections == 2 ? 64 : 128);
    int64_t most = 32;
    if (tiles >= num_sms()) {
        if (a.E == 1) most = fmt == TQ_INT4_G128_ASYM ? 32 : 16;
        else most = fmt == TQ_INT4_G32_ASYM ? (a.I % 128 == 0 ? 4 : 1) : fmt == TQ_INT3_G64_SYM || fmt == TQ_INT4_G64_ASYM ? 8 : 16;
    }
    if (per > most) return 0;
    return per <= 8 ? 1 : per <= 16 ? 2 : 4;
}

static RowsArgs rows_args(const tq_records* W, const tq_records* W2, int64_t R, const int32_t* offsets) {
    RowsArgs a;
    memset(&a, 0, sizeof a);
    const tq_records* w[2] = {W, W2 ? W2 : W};
    for (int i = 0; i < 2; ++i) {
        a.packed[i] = w[i]->packed;
        a.scales[i] = w[i]->scales;
        a.zeros[i] = w[i]->zeros;
        a.gs[i] = w[i]->global_scale;
    }
    a.O = W->O;
    a.I = W->I;
    a.G = (W->I + group_of(W->fmt) - 1) / group_of(W->fmt);
    a.rowbytes = a.G * record_bytes(W->fmt);
    a.o_begin = 0;
    a.o_end = W->O;
    a.R = R;
    a.offsets = offsets;
    a.E = static_cast<int>(W->n_mat);
    a.projections = W2 ? 2 : 1;
    a.splits = 1;
    a.wait_limit = pipeline_wait_limit();
    a.few = few_blocks(W->fmt, a);
    return a;
}

struct FewSpace {
    uint16_t* x;
    float* row_x;
    float* sums;
};
static FewSpace few_space(Carve& c, const RowsArgs& a) {
    FewSpace f;
    f.x = c.take<uint16_t>(a.R * tiles_of(a.I, 128) * 128);
    f.row_x = c.take<float>(a.R);
    f.sums = c.take<float>(a.R * tiles_of(a.I, 128) * 4);
    return f;
}

static tq_status few(int32_t fmt, RowsArgs& a, const tq_mat* X, const FewSpace& f, cudaStream_t st) {
    const int nb = a.few;
    a.x_few = f.x;
    a.row_x = f.row_x;
    a.x_sums = f.sums;
    a.m_tiles = static_cast<int>(a.projections == 2 ? tiles_of(a.O, 16) : tiles_of(a.o_end - a.o_begin, 32));
    a.part_tiles = a.m_tiles;
    const int n = fmt == TQ_NVFP4_G16 || fmt == TQ_INT4_G64_ASYM || fmt == TQ_INT3_G64_SYM ? 2 : fmt == TQ_INT4_G32_ASYM ? 4 : 1;
    uintptr_t al = 0;
    for (int i = 0; i < 2; ++i) {
        al |= reinterpret_cast<uintptr_t>(a.zeros[i]) % n;
        al |= reinterpret_cast<uintptr_t>(a.scales[i]) % (fmt == TQ_NVFP4_G16 ? 2 : 4 * n);
    }
    a.few_wide = a.G % n == 0 && al == 0;
    k_few_prep<<<static_cast<unsigned>(a.R), FEW_PREP_THREADS, 0, st>>>(static_cast<const uint16_t*>(X->ptr), X->ld, a.I,
                                                                    fmt, f.x, f.row_x, f.sums);
    ROWS_TRY(check_launch("row products: tokens"));
    // Warps per tile: rounds of tiles x (slices of a warp + a tile's end,
    // about two slices), least over ks.  (Routed rows: the matrices that have
    // any are not known here; as many as there are rows, at most.)
    const int64_t n_slices = tiles_of(a.I, 128);
    const int64_t items = a.m_tiles * (tiles_of(a.R, 8 * nb) + (a.E > 1 ? (a.R < a.E ? a.R : a.E) * 3 / 4 : 0));
    const int mb = few_blocks_per_sm(fmt, nb, items, num_sms());
    const int64_t slots = mb * static_cast<int64_t>(num_sms());
    int64_t least = 0;
    for (int ks = 1; ks <= 8 && ks <= n_slices; ks *= 2) {
        const int64_t t = tiles_of(items, slots * (8 / ks)) * (tiles_of(n_slices, ks) + 2);
        if (least == 0 || t < least) {
            least = t;
            a.few_ks = ks;
        }
    }
    const int64_t blocks = tiles_of(items * 4 / 3 + 1, 8 / a.few_ks);
    const int grid = static_cast<int>(blocks < slots ? blocks : slots);
    switch (fmt) {
        case TQ_INT3_G64_SYM: return launch_few_int3(a, nb, mb, grid, st);
        case TQ_INT4_G128_ASYM: return launch_few_int4g128(a, nb, mb, grid, st);
        case TQ_INT4_G64_ASYM: return launch_few_int4g64(a, nb, mb, grid, st);
        case TQ_INT4_G32_ASYM: return launch_few_int4g32(a, nb, mb, grid, st);
        default: return launch_few_nvfp4(a, nb, mb, grid, st);
    }
}

// What a forward launch needs beside the records: the tokens in f16 with their
// powers of two, and the matrices' largest values (integer formats, scaled
// kind; the gated backward pass).
struct ForwardSpace {
    uint16_t* x16;
    float* row_x;
    float* wmax;
};
static ForwardSpace forward_space(Carve& c, const RowsArgs& a) {
    ForwardSpace f;
    f.x16 = c.take<uint16_t>(a.R * up16(a.I));
    f.row_x = c.take<float>(a.R);
    f.wmax = c.take<float>(static_cast<int64_t>(a.projections) * a.E * rows_wmax_parts(a.E));
    return f;
}

// The kind of a forward launch: exact where the result is not rounded to 16
// bits.
static int forward_kind(bool to16) { return to16 ? ROWS_SCALED : ROWS_EXACT; }

// The forward launch: the tokens' f16 copy against rows o_begin .. o_end - 1.
static tq_status forward(int32_t fmt, int kind, RowsArgs& a, const uint16_t* x16, cudaStream_t st) {
    const int64_t m128 = a.projections == 2 ? tiles_of(a.O, 64) : tiles_of(a.o_end - a.o_begin, 128);
    a.nk = static_cast<int>(tiles_of(a.I, 64));
    const RowsPlan p = rows_plan(m128, a.R, a.E, a.nk, false, a.I);
    a.m_tiles = static_cast<int>(tiles_of(m128, rows_pair(p.nt) ? 2 : 1));
    a.part_tiles = a.m_tiles * (rows_pair(p.nt) ? 2 : 1);
    CUtensorMap map;
    ROWS_TRY(rows_map(&map, x16, up16(a.I), a.R, up16(a.I), 1, p.nt));
    const RowsLaunch l{&map, p.nt, kind, p.grid};
    return launch_rows(fmt, a, l, st);
}

// The tokens' f16 copy in the records' column order.
static PrepArgs tokens_prep(const tq_mat* X, int32_t fmt, const ForwardSpace& f) {
    PrepArgs p;
    memset(&p, 0, sizeof p);
    p.rows = X->rows;
    p.src = static_cast<const uint16_t*>(X->ptr);
    p.src_cols = X->cols;
    p.src_ld = X->ld;
    p.order = fmt;
    p.f16 = f.x16;
    p.f16_f = f.row_x;
    return p;
}

static RowsPlan backward_plan(const RowsArgs& a, int64_t rows_of_w) {
    return rows_plan(tiles_of(a.I, 128), a.R, a.E, tiles_of(rows_of_w, 64) * a.projections, true, a.I);
}

// The backward launch: a.D against rows o_begin .. o_end - 1 (of each projection).
static tq_status backward(int32_t fmt, RowsArgs& a, const RowsPlan& p, cudaStream_t st) {
    a.m_tiles = static_cast<int>(tiles_of(a.I, rows_pair(p.nt) ? 256 : 128));
    a.nk = static_cast<int>(tiles_of(a.o_end - a.o_begin, 64));
    a.splits = p.splits;
    CUtensorMap map;
    ROWS_TRY(rows_map(&map, a.D, a.o_end - a.o_begin, a.R, a.ldd, a.projections, p.nt));
    const RowsLaunch l{&map, p.nt, ROWS_GRAD, p.grid};
    return launch_rows(fmt, a, l, st);
}

static tq_status join(const RowsArgs& a, void* dx, int64_t ldx, cudaStream_t st) {
    const int64_t y = tiles_of(a.I, 2048) < 65535 ? tiles_of(a.I, 2048) : 65535;   // (the grid's limit along y)
    k_rows_join<<<dim3(static_cast<unsigned>(a.R), static_cast<unsigned>(y)), 256, 0, st>>>(
        a.sums, a.splits, a.R, a.I, a.offsets, a.E, static_cast<uint16_t*>(dx), ldx);
    return check_launch("row products: join");
}

static tq_status prep(PrepArgs& p, const RowsArgs& a, int32_t fmt, cudaStream_t st) {
    p.scales[0] = a.scales[0];
    p.scales[1] = a.scales[1];
    p.zeros[0] = a.zeros[0];
    p.zeros[1] = a.zeros[1];
    p.per_mat = a.O * a.G;
    p.E = a.E;
    p.e4m3 = fmt == TQ_NVFP4_G16;
    p.wmax = const_cast<float*>(a.wmax);
    const int64_t blocks = p.rows + (p.wmax ? static_cast<int64_t>(a.projections) * a.E * rows_wmax_parts(a.E) : 0);
    if (blocks == 0) return TQ_OK;
    k_rows_prep<<<static_cast<unsigned>(blocks), PREP_THREADS, 0, st>>>(p);
    return check_launch("row products: prep");
}

// Weight rows per piece of the loss's backward pass: D of a piece at most 256
// MB.  (The last piece may be much shorter, down to one row.)
static int64_t loss_piece(int64_t R, int64_t V) {
    const int64_t most = (int64_t(128) << 20) / (R < 1 ? 1 : R);
    const int64_t rows = most < 1024 ? 1024 : most / 128 * 128;
    if (rows >= V) return V;
    const int64_t pieces = tiles_of(V, rows);
    return tiles_of(tiles_of(V, pieces), 128) * 128;
}

struct BackwardSpace {
    int few;               // the forward part's blocks of 8 tokens (few tokens), or 0
    FewSpace few_x;
    ForwardSpace fwd;
    uint16_t* D;
    float* row_f;
    float* wmax;
    float* sums;
    size_t bytes;
    RowsPlan plan;
};

// fwd: with what the forward part needs (its wmax serves both).
static BackwardSpace backward_space(const RowsArgs& a, bool fwd, int64_t rows_of_w, bool own_row_f, bool sums,
                                    void* ws) {
    BackwardSpace b;
    b.plan = backward_plan(a, rows_of_w);
    Carve c(ws);
    memset(&b.fwd, 0, sizeof b.fwd);
    memset(&b.few_x, 0, sizeof b.few_x);
    b.few = fwd ? a.few : 0;
    if (b.few) b.few_x = few_space(c, a);
    else if (fwd) b.fwd = forward_space(c, a);
    b.D = c.take<uint16_t>(a.projections * a.R * up16(rows_of_w));
    b.row_f = own_row_f ? c.take<float>(a.R) : nullptr;
    b.wmax = fwd && !b.few ? b.fwd.wmax : c.take<float>(static_cast<int64_t>(a.projections) * a.E * rows_wmax_parts(a.E));
    b.sums = sums || b.plan.splits > 1 ? c.take<float>(b.plan.splits * a.R * a.I) : nullptr;
    b.bytes = c.used;
    return b;
}

static tq_status check_workspace(const void* ws, size_t have, size_t need, const char* what) {
    TQ_REQUIRE(need == 0 || ws, "%s: null workspace", what);
    TQ_REQUIRE(have >= need, "%s: workspace of %zu bytes, needs %zu", what, have, need);
    TQ_REQUIRE(aligned16(ws), "%s: workspace not 16-byte aligned", what);
    return TQ_OK;
}

static tq_status check_offsets(const tq_records* W, const int32_t* offsets, const char* what) {
    TQ_REQUIRE(W->n_mat == 1 || offsets, "%s: %lld matrices need offsets", what, (long long)W->n_mat);
    TQ_REQUIRE((reinterpret_cast<uintptr_t>(offsets) & 3u) == 0, "%s: offsets not 4-byte aligned", what);
    return TQ_OK;
}

static tq_status check_out(const void* y, int32_t dtype, int64_t ld, int64_t cols, int64_t rows, const char* what) {
    if (dtype != TQ_BF16 && dtype != TQ_F32) return set_error(TQ_ERR_UNSUPPORTED, "%s: output dtype %d", what, dtype);
    TQ_REQUIRE(rows == 0 || y, "%s: null output", what);
    TQ_REQUIRE((reinterpret_cast<uintptr_t>(y) & (dtype == TQ_BF16 ? 1u : 3u)) == 0, "%s: output misaligned", what);
    TQ_REQUIRE(ld >= cols, "%s: output row stride %lld < %lld columns", what, (long long)ld, (long long)cols);
    return TQ_OK;
}

static tq_status check_pair(const tq_records* gate, const tq_records* up, const char* what) {
    TQ_REQUIRE(gate->fmt == up->fmt && gate->n_mat == up->n_mat && gate->O == up->O && gate->I == up->I,
               "%s: gate and up must have one format and shape", what);
    return TQ_OK;
}

}  // namespace tq

using namespace tq;

// ------------------------------------------------------------------ y = x What^T

// The forward product: few tokens per matrix, or tiles of them.
static tq_status product(int32_t fmt, RowsArgs& a, const tq_mat* X, void* workspace, size_t bytes, const char* what,
                         cudaStream_t st) {
    Carve c(workspace);
    if (a.few) {
        const FewSpace f = few_space(c, a);
        ROWS_TRY(check_workspace(workspace, bytes, c.used, what));
        return few(fmt, a, X, f, st);
    }
    const ForwardSpace f = forward_space(c, a);
    ROWS_TRY(check_workspace(workspace, bytes, c.used, what));
    const int kind = forward_kind(a.y_bf16);
    a.row_x = f.row_x;
    a.wmax = kind == ROWS_SCALED && fmt != TQ_NVFP4_G16 ? f.wmax : nullptr;
    PrepArgs p = tokens_prep(X, fmt, f);
    ROWS_TRY(prep(p, a, fmt, st));
    return forward(fmt, kind, a, f.x16, st);
}

static size_t product_bytes(const tq_records* W, const tq_records* W2, int64_t rows) {
    if (rows < 1) return 0;
    const RowsArgs a = rows_args(W, W2, rows, nullptr);
    Carve c(nullptr);
    if (a.few) few_space(c, a);
    else forward_space(c, a);
    return c.used;
}

TQ_API size_t tq_dequant_matmul_workspace_bytes(const tq_records* W, int64_t rows) {
    return check_records(W, "W") == TQ_OK ? product_bytes(W, nullptr, rows) : 0;
}

TQ_API tq_status tq_dequant_matmul(const tq_records* W, const tq_mat* X, const int32_t* offsets, void* y,
                                   int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes,
                                   tq_stream_t stream) {
    clear_error();
    ROWS_TRY(check_records(W, "tq_dequant_matmul W"));
    ROWS_TRY(check_tokens(X, -1, W->I, "tq_dequant_matmul X"));
    ROWS_TRY(check_offsets(W, offsets, "tq_dequant_matmul"));
    ROWS_TRY(check_out(y, y_dtype, ldy, W->O, X->rows, "tq_dequant_matmul"));
    if (X->rows == 0) return TQ_OK;
    RowsArgs a = rows_args(W, nullptr, X->rows, offsets);
    a.mode = ROWS_STORE;
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = y_dtype == TQ_BF16;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return product(W->fmt, a, X, workspace, workspace_bytes, "tq_dequant_matmul", st);
}

TQ_API size_t tq_dequant_matmul_backward_workspace_bytes(const tq_records* W, int64_t rows) {
    if (check_records(W, "W") != TQ_OK || rows < 1) return 0;
    return backward_space(rows_args(W, nullptr, rows, nullptr), false, W->O, true, false, nullptr).bytes;
}

TQ_API tq_status tq_dequant_matmul_backward(const tq_records* W, const tq_mat* dY, const int32_t* offsets, void* dx,
                                            int64_t ldx, void* workspace, size_t workspace_bytes,
                                            tq_stream_t stream) {
    clear_error();
    ROWS_TRY(check_records(W, "tq_dequant_matmul_backward W"));
    ROWS_TRY(check_tokens(dY, -1, W->O, "tq_dequant_matmul_backward dY"));
    ROWS_TRY(check_offsets(W, offsets, "tq_dequant_matmul_backward"));
    ROWS_TRY(check_out(dx, TQ_BF16, ldx, W->I, dY->rows, "tq_dequant_matmul_backward"));
    if (dY->rows == 0) return TQ_OK;
    RowsArgs a = rows_args(W, nullptr, dY->rows, offsets);
    const BackwardSpace b = backward_space(a, false, W->O, true, false, workspace);
    ROWS_TRY(check_workspace(workspace, workspace_bytes, b.bytes, "tq_dequant_matmul_backward"));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    a.mode = ROWS_STORE;
    a.y = dx;
    a.ldy = ldx;
    a.D = b.D;
    a.ldd = up16(W->O);
    a.row_f = b.row_f;
    a.wmax = W->fmt != TQ_NVFP4_G16 ? b.wmax : nullptr;
    a.sums = b.sums;
    PrepArgs p;
    memset(&p, 0, sizeof p);
    p.rows = a.R;
    p.src = static_cast<const uint16_t*>(dY->ptr);
    p.src_cols = W->O;
    p.src_ld = dY->ld;
    p.f16 = b.D;
    p.f16_f = b.row_f;
    ROWS_TRY(prep(p, a, W->fmt, st));
    ROWS_TRY(backward(W->fmt, a, b.plan, st));
    return a.sums ? join(a, dx, ldx, st) : TQ_OK;
}

// ------------------------------------------------------------------ gated feed-forward

TQ_API size_t tq_gated_ffn_workspace_bytes(const tq_records* gate, int64_t rows) {
    return check_records(gate, "gate") == TQ_OK ? product_bytes(gate, gate, rows) : 0;
}

TQ_API tq_status tq_gated_ffn(const tq_records* gate, const tq_records* up, int32_t act, const tq_mat* X,
                              const int32_t* offsets, void* h, int32_t h_dtype, int64_t ldh, void* workspace,
                              size_t workspace_bytes, tq_stream_t stream) {
    clear_error();
    ROWS_TRY(check_records(gate, "tq_gated_ffn gate"));
    ROWS_TRY(check_records(up, "tq_gated_ffn up"));
    ROWS_TRY(check_pair(gate, up, "tq_gated_ffn"));
    if (act != TQ_ACT_SILU && act != TQ_ACT_GELU_TANH)
        return set_error(TQ_ERR_UNSUPPORTED, "tq_gated_ffn: activation %d", act);
    ROWS_TRY(check_tokens(X, -1, gate->I, "tq_gated_ffn X"));
    ROWS_TRY(check_offsets(gate, offsets, "tq_gated_ffn"));
    ROWS_TRY(check_out(h, h_dtype, ldh, gate->O, X->rows, "tq_gated_ffn"));
    if (X->rows == 0) return TQ_OK;
    RowsArgs a = rows_args(gate, up, X->rows, offsets);
    a.mode = ROWS_GATED;
    a.act = act;
    a.y = h;
    a.ldy = ldh;
    a.y_bf16 = h_dtype == TQ_BF16;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return product(gate->fmt, a, X, workspace, workspace_bytes, "tq_gated_ffn", st);
}

TQ_API size_t tq_gated_ffn_backward_workspace_bytes(const tq_records* gate, int64_t rows) {
    if (check_records(gate, "gate") != TQ_OK || rows < 1) return 0;
    return backward_space(rows_args(gate, gate, rows, nullptr), true, gate->O, true, false, nullptr).bytes;
}

TQ_API tq_status tq_gated_ffn_backward(const tq_records* gate, const tq_records* up, int32_t act, const tq_mat* X,
                                       const tq_mat* dH, const int32_t* offsets, void* dx, int64_t ldx,
                                       void* workspace, size_t workspace_bytes, tq_stream_t stream) {
    clear_error();
    ROWS_TRY(check_records(gate, "tq_gated_ffn_backward gate"));
    ROWS_TRY(check_records(up, "tq_gated_ffn_backward up"));
    ROWS_TRY(check_pair(gate, up, "tq_gated_ffn_backward"));
    if (act != TQ_ACT_SILU && act != TQ_ACT_GELU_TANH)
        return set_error(TQ_ERR_UNSUPPORTED, "tq_gated_ffn_backward: activation %d", act);
    ROWS_TRY(check_tokens(X, -1, gate->I, "tq_gated_ffn_backward X"));
    ROWS_TRY(check_tokens(dH, X->rows, gate->O, "tq_gated_ffn_backward dH"));
    ROWS_TRY(check_offsets(gate, offsets, "tq_gated_ffn_backward"));
    ROWS_TRY(check_out(dx, TQ_BF16, ldx, gate->I, X->rows, "tq_gated_ffn_backward"));
    if (X->rows == 0) return TQ_OK;
    RowsArgs a = rows_args(gate, up, X->rows, offsets);
    const BackwardSpace b = backward_space(a, true, gate->O, true, false, workspace);
    ROWS_TRY(check_workspace(workspace, workspace_bytes, b.bytes, "tq_gated_ffn_backward"));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    a.mode = ROWS_GATED_BWD;
    a.act = act;
    a.dh = static_cast<const uint16_t*>(dH->ptr);
    a.ld_dh = dH->ld;
    a.y = dx;
    a.ldy = ldx;
    a.D = b.D;
    a.ldd = up16(gate->O);
    a.row_f = b.row_f;
    a.row_x = b.fwd.row_x;
    a.wmax = b.wmax;
    PrepArgs p = tokens_prep(X, gate->fmt, b.fwd);
    p.dh = a.dh;
    p.dh_cols = gate->O;
    p.dh_ld = dH->ld;
    p.row_f = b.row_f;
    ROWS_TRY(prep(p, a, gate->fmt, st));
    if (b.few) ROWS_TRY(few(gate->fmt, a, X, b.few_x, st));
    else ROWS_TRY(forward(gate->fmt, ROWS_SCALED, a, b.fwd.x16, st));
    a.sums = b.sums;
    ROWS_TRY(backward(gate->fmt, a, b.plan, st));
    return a.sums ? join(a, dx, ldx, st) : TQ_OK;
}

// ------------------------------------------------------------------ cross entropy of the packed head

struct LossSpace {
    float2* part;
    float* label_z;
    FewSpace few;
    ForwardSpace fwd;
    size_t bytes;
};
static LossSpace loss_space(void* ws, const RowsArgs& a) {
    LossSpace l;
    Carve c(ws);
    const bool is_few = a.few != 0;
    l.part = c.take<float2>((is_few ? tiles_of(a.O, 32) : tiles_of(a.O, 256) * 2) * a.R);
    l.label_z = c.take<float>(a.R);
    memset(&l.few, 0, sizeof l.few);
    memset(&l.fwd, 0, sizeof l.fwd);
    if (is_few) l.few = few_space(c, a);
    else l.fwd = forward_space(c, a);
    l.bytes = c.used;
    return l;
}

TQ_API size_t tq_head_loss_workspace_bytes(const tq_records* W, int64_t rows) {
    if (check_records(W, "W") != TQ_OK || rows < 1) return 0;
    return loss_space(nullptr, rows_args(W, nullptr, rows, nullptr)).bytes;
}

TQ_API tq_status tq_head_loss(const tq_records* W, const tq_mat* X, const int64_t* labels, float* loss, float* lse,
                              void* workspace, size_t workspace_bytes, tq_stream_t stream) {
    clear_error();
    ROWS_TRY(check_records(W, "tq_head_loss W"));
    TQ_REQUIRE(W->n_mat == 1, "tq_head_loss: one matrix expected");
    ROWS_TRY(check_tokens(X, -1, W->I, "tq_head_loss X"));
    if (X->rows == 0) return TQ_OK;
    TQ_REQUIRE(labels && loss && lse, "tq_head_loss: null pointer");
    TQ_REQUIRE((reinterpret_cast<uintptr_t>(labels) & 7u) == 0, "tq_head_loss: labels not 8-byte aligned");
    TQ_REQUIRE(((reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(lse)) & 3u) == 0,
               "tq_head_loss: loss or lse not 4-byte aligned");
    RowsArgs a = rows_args(W, nullptr, X->rows, nullptr);
    const LossSpace l = loss_space(workspace, a);
    ROWS_TRY(check_workspace(workspace, workspace_bytes, l.bytes, "tq_head_loss"));
    a.mode = ROWS_LOSS;
    a.part = l.part;
    a.label_z = l.label_z;
    a.labels = labels;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (a.few) {
        ROWS_TRY(few(W->fmt, a, X, l.few, st));
    } else {
        a.row_x = l.fwd.row_x;
        PrepArgs p = tokens_prep(X, W->fmt, l.fwd);
        ROWS_TRY(prep(p, a, W->fmt, st));
        ROWS_TRY(forward(W->fmt, forward_kind(false), a, l.fwd.x16, st));
    }
    k_loss_join<<<static_cast<unsigned>(a.R), 256, 0, st>>>(a.part, a.part_tiles, a.R, labels, W->O,
                                                                          a.label_z, loss, lse);
    return check_launch("tq_head_loss");
}

TQ_API size_t tq_head_loss_backward_workspace_bytes(const tq_records* W, int64_t rows) {
    if (check_records(W, "W") != TQ_OK || rows < 1) return 0;
    const int64_t piece = loss_piece(rows, W->O);
    return backward_space(rows_args(W, nullptr, rows, nullptr), true, piece, false, piece < W->O, nullptr).bytes;
}

TQ_API tq_status tq_head_loss_backward(const tq_records* W, const tq_mat* X, const int64_t* labels, const float* lse,
                                       const float* dloss, void* dx, int64_t ldx, void* workspace,
                                       size_t workspace_bytes, tq_stream_t stream) {
    clear_error();
    ROWS_TRY(check_records(W, "tq_head_loss_backward W"));
    TQ_REQUIRE(W->n_mat == 1, "tq_head_loss_backward: one matrix expected");
    ROWS_TRY(check_tokens(X, -1, W->I, "tq_head_loss_backward X"));
    ROWS_TRY(check_out(dx, TQ_BF16, ldx, W->I, X->rows, "tq_head_loss_backward"));
    if (X->rows == 0) return TQ_OK;
    TQ_REQUIRE(labels && lse && dloss, "tq_head_loss_backward: null pointer");
    TQ_REQUIRE((reinterpret_cast<uintptr_t>(labels) & 7u) == 0, "tq_head_loss_backward: labels not 8-byte aligned");
    TQ_REQUIRE(((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(dloss)) & 3u) == 0,
               "tq_head_loss_backward: lse or dloss not 4-byte aligned");
    RowsArgs a = rows_args(W, nullptr, X->rows, nullptr);
    const int64_t piece = loss_piece(a.R, W->O);
    const BackwardSpace b = backward_space(a, true, piece, false, piece < W->O, workspace);
    ROWS_TRY(check_workspace(workspace, workspace_bytes, b.bytes, "tq_head_loss_backward"));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    a.mode = ROWS_PROB;
    a.labels = labels;
    a.lse = lse;
    a.row_f = dloss;
    a.y = dx;
    a.ldy = ldx;
    a.D = b.D;
    a.ldd = up16(piece);
    a.row_x = b.fwd.row_x;
    a.wmax = W->fmt != TQ_NVFP4_G16 ? b.wmax : nullptr;
    PrepArgs p = tokens_prep(X, W->fmt, b.fwd);
    if (b.few) p.rows = 0;   // (few() prepares the tokens itself)
    ROWS_TRY(prep(p, a, W->fmt, st));
    for (int64_t v = 0; v < W->O; v += piece) {
        a.o_begin = v;
        a.o_end = v + piece < W->O ? v + piece : W->O;
        a.splits = 1;
        a.sums = nullptr;
        if (b.few) ROWS_TRY(few(W->fmt, a, X, b.few_x, st));
        else ROWS_TRY(forward(W->fmt, forward_kind(false), a, b.fwd.x16, st));
        a.sums = b.sums;
        a.sums_add = v > 0;
        ROWS_TRY(backward(W->fmt, a, b.plan, st));
    }
    return a.sums ? join(a, dx, ldx, st) : TQ_OK;
}
