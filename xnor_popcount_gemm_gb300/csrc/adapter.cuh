// Declarations and device helpers shared by the adapters' kernels (see adapter.cu).
#pragma once

#include <type_traits>

#include "adapter_plan.h"
#include "bt_device.cuh"
#include "tc_ptx.cuh"

namespace bt {
namespace adapter {

constexpr int kThreads = 256;
constexpr int kStep = 64;                  // long-axis elements of a stage

// ---------------------------------------------------------------------------
// Matrix instructions: D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

// ---------------------------------------------------------------------------
// 16-bit values
// ---------------------------------------------------------------------------
template <typename T> __device__ __forceinline__ T to16(float v);
template <> __device__ __forceinline__ __nv_bfloat16 to16<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half to16<__half>(float v) { return __float2half_rn(v); }
template <typename T> __device__ __forceinline__ uint32_t bits16(T v) { return *reinterpret_cast<const uint16_t *>(&v); }
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    return bits16(to16<T>(lo)) | (bits16(to16<T>(hi)) << 16);
}
template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// v as the sum of two 16-bit values, pairwise: hi and lo words of (v0, v1).
// Infinities keep a zero low part.
template <typename T> __device__ __forceinline__ void split2(float v0, float v1, uint32_t &hi, uint32_t &lo) {
    hi = pack2<T>(v0, v1);
    const float2 h = unpack2<T>(hi);
    lo = pack2<T>(isinf(h.x) ? 0.0f : v0 - h.x, isinf(h.y) ? 0.0f : v1 - h.y);
}
// What the two leave of v, given them.
template <typename T> __device__ __forceinline__ uint32_t split_rest(float v0, float v1, uint32_t hi, uint32_t lo) {
    const float2 h = unpack2<T>(hi), l = unpack2<T>(lo);
    return pack2<T>(isinf(h.x) ? 0.0f : (v0 - h.x) - l.x, isinf(h.y) ? 0.0f : (v1 - h.y) - l.y);
}
// How many 16-bit values an fp32 sum enters a product as: three bf16 ones hold all of its 24 bits, two half-precision
// ones 22. (Two bf16 values hold 16: no less than a bf16 result shows, but its rounding then falls the other way now
// and then, and ranks that cancel show it in full.)
template <typename T> constexpr int kValues = std::is_same<T, __nv_bfloat16>::value ? 3 : 2;
// Half precision reaches 65504 and ends at 2^-24: rows of u are brought to a
// largest value of about 2^14 by a power of two first (taken out again in fp32).
// An infinity is one at any scale: the others count.
__device__ __forceinline__ float finite_size(float v) { return isinf(v) ? 0.0f : fabsf(v); }
template <typename T> __device__ __forceinline__ float row_power(float amax) {
    if constexpr (std::is_same<T, __half>::value) {
        if (!(amax > 0.0f)) return 1.0f;
        int e = 14 - ilogbf(amax);
        e = e > 100 ? 100 : e < -100 ? -100 : e;
        return exp2f(static_cast<float>(e));
    }
    return 1.0f;
}

// ---------------------------------------------------------------------------
// Eight consecutive elements of a global row to shared memory (16 bytes, 16-byte
// aligned), `valid` of them there (<= 0: none), the rest zeros.
// ---------------------------------------------------------------------------
template <int B> __device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(B), "r"(bytes) : "memory");
}
__device__ __forceinline__ int clamp_to(int v, int hi) { return v < 0 ? 0 : v > hi ? hi : v; }
// The words of eight elements at any element address, from the aligned words that hold a valid one.
__device__ __forceinline__ uint4 load8(const uint16_t *src, int valid) {
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 2) >> 1;
    const uint32_t *p = reinterpret_cast<const uint32_t *>(src - odd);
    uint32_t w[5], r[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = 2 * i - odd < valid && (i < 4 || odd) ? __ldg(p + i) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[i] = odd ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
        const int left = valid - 2 * i;
        r[i] = left >= 2 ? r[i] : left == 1 ? r[i] & 0xFFFFu : 0u;
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
// How an operand's rows are fetched, by what they start at multiples of.
constexpr int kRows16 = 0;                 // 16 bytes: asynchronous copies
constexpr int kRows4 = 1;                  // 4 bytes: asynchronous copies of 4, 8 or 16
constexpr int kRows2 = 2;                  // less: through registers
inline int rows_mode(int al) { return al == 16 ? kRows16 : al >= 4 ? kRows4 : kRows2; }
template <int MODE> __device__ __forceinline__ void copy8(void *dst, const uint16_t *src, int valid, int al) {
    if (MODE == kRows16 || (MODE == kRows4 && al == 16)) {
        cp_async_16(dst, src, clamp_to(valid, 8) * 2);
    } else if (MODE == kRows4) {
        const uint32_t d = smem_u32(dst);
        if (al == 8) {
            cp_async_small<8>(d, src, clamp_to(valid, 4) * 2);
            cp_async_small<8>(d + 8, valid > 4 ? src + 4 : src, clamp_to(valid - 4, 4) * 2);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cp_async_small<4>(d + 4 * i, valid > 2 * i ? src + 2 * i : src, clamp_to(valid - 2 * i, 2) * 2);
        }
    } else {
        *reinterpret_cast<uint4 *>(dst) = valid > 0 ? load8(src, valid) : make_uint4(0u, 0u, 0u, 0u);
    }
}

// The 128-byte swizzle: chunk j (16 bytes) of row r of a tile of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int row, int chunk) { return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4)); }
constexpr int kAtom = 8192;                // 64 rows of 128 bytes

// A wait for copies or products in flight: if it gives up (which it records),
// it still lets them land before memory is given back.
__device__ __forceinline__ void wait_landed(uint64_t &bar, uint32_t parity, uint32_t *abort_flag, unsigned int *err,
                                            unsigned long long limit_ns) {
    if (!tc::wait_fast(smem_u32(&bar), parity, abort_flag, err, limit_ns)) {
        uint32_t drain = 0;
        tc::wait_bounded(smem_u32(&bar), parity, &drain, err);
    }
}

// The rows in the plan's order, and the tiles (or parts) a launch walks.
struct Plan {
    const int32_t *rows;
    const AdapterTile *tiles;
};

// Tokens without an adapter: out = cast(base), u = 0.
struct PassArgs {
    const int32_t *rows;
    int n, N, R;
    const void *base;
    int base_f32;
    int64_t ldb;
    void *out;                 // NULL: the rows are in place already
    int64_t ldo;
    float *u;
};
// Pieces first, first + step, ... of them (8 columns a thread of 256): CTAs of the kernels below that are left
// over take them along.
constexpr int kPassCols = 2048;
inline int64_t pass_pieces(const PassArgs &a) { return static_cast<int64_t>(a.n) * ((a.N + kPassCols - 1) / kPassCols); }
template <typename T> __device__ void pass_rows(const PassArgs &a, bool out_f32, int first, int step) {
    const int per = (a.N + kPassCols - 1) / kPassCols;
    if (threadIdx.x >= 256) return;
    for (int64_t i = first; i < static_cast<int64_t>(a.n) * per; i += step) {
        const int64_t row = a.rows[i / per];
        const int c0 = static_cast<int>(i % per) * kPassCols;
        if (a.u != nullptr && c0 == 0)
            for (int r = threadIdx.x; r < a.R; r += 256) a.u[row * a.R + r] = 0.0f;
        if (a.out == nullptr) continue;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {                       // neighbours take neighbours: any alignment travels together
            const int c = c0 + static_cast<int>(threadIdx.x) + 256 * k;
            v[k] = 0.0f;
            if (a.base != nullptr && c < a.N)
                v[k] = a.base_f32 ? static_cast<const float *>(a.base)[row * a.ldb + c]
                                  : Elem<T>::to_f32(static_cast<const T *>(a.base)[row * a.ldb + c]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int c = c0 + static_cast<int>(threadIdx.x) + 256 * k;
            if (c >= a.N) continue;
            if (out_f32) static_cast<float *>(a.out)[row * a.ldo + c] = v[k];
            else static_cast<T *>(a.out)[row * a.ldo + c] = to16<T>(v[k]);
        }
    }
}
cudaError_t launch_pass(bt_dtype t, bool out_f32, const PassArgs &a, cudaStream_t s);

// u and dU between the products: rows in the plan's order, padded to RP = 16,
// 32, 64 or 128 ranks, as the sum of three bf16 values or of two in half precision, these
// times a power of two of the row's own, whose inverse is in unpower.
struct SplitRows {
    uint16_t *hi, *lo;         // [T, RP]
    uint16_t *rest;            // what the two leave, the third value (bf16)
    float *unpower;            // [T], NULL: 1
};
inline int padded_rank(int R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }

// Rows of an odd width, copied to rows that start at 16-byte multiples: `rows` of them, or, with parts, the R rows
// of every adapter that has tokens.
struct AlignArgs {
    const uint16_t *src;
    int64_t lds;
    uint16_t *dst;
    int64_t ldd;
    int C;
    int64_t rows;
    const AdapterTile *parts;
    int R, nparts;
};
cudaError_t launch_align(const AlignArgs &a, cudaStream_t s);

// U[t, :] = s sum_c X[t, c] W[c, :] over tiles of 128 rows. WT = false: W is
// [R, C] (A, for u), true: [C, R] (B, for dU).
struct ShrinkArgs {
    Plan plan;
    const uint16_t *x;
    int64_t ldx;
    int ax, aw;                // alignment of the rows of X and W, bytes
    const uint16_t *w;         // [L, R, ldw] or [L, C, R]
    int64_t ldw;               // (WT = false)
    int C, R;
    const float *scale;        // NULL: 1
    float *u;                  // [T, R] by token; NULL: not wanted
    SplitRows out;
    const float *given;        // (WT) [T, R] by token, to be split as well; into given_out
    SplitRows given_out;
    unsigned int *zero;        // words to be zeroed for the kernels that follow
    int zeros;
    int cluster;
    unsigned int *err;
    unsigned long long limit_ns;
};
cudaError_t launch_shrink(bt_dtype t, bool wt, const ShrinkArgs &a, int tiles, cudaStream_t s);

// OUT[t, c] = cast(BASE[t, c] + s sum_r U[t, r] W[r, c]) over tiles of 128 rows.
// WT = false: W is [C, R] (B, for out), true: [R, C] (A, for dX; bf16 only).
struct ExpandArgs {
    Plan plan;
    SplitRows u;
    const uint16_t *w;         // [L, C, R] or [L, R, ldw]
    int64_t ldw;               // (WT = true)
    int aw;                    // alignment of its rows, bytes
    int C, R;
    const float *scale;        // NULL: 1
    const void *base;          // NULL: 0
    int base_f32;
    int64_t ldb;
    void *out;
    int64_t ldo;
    int wide;                  // rows of base and out start at 16-byte multiples, C a multiple of 8
    int tiles, splits;         // column ranges per tile
    PassArgs pass;             // rows that the CTAs after the tiles' take along (n = 0: none)
    unsigned int *err;
    unsigned long long limit_ns;
};
cudaError_t launch_expand(bt_dtype t, bool wt, bool out_f32, const ExpandArgs &a, int tiles, cudaStream_t s);



// G[r, c] = s sum_t U[t, r] X[t, c] over every part of the adapters' tokens, for
// two products in one launch: dA = dU^T x as [R, K], dB = s u^T g as [N, R].
struct GradProduct {
    SplitRows u;
    const uint16_t *x;         // [T, C]
    int64_t ldx;
    int ax;                    // alignment of the rows of X, bytes
    int C;
    int rc;                    // 1: G is [R, C], 0: [C, R]
    const float *scale;        // NULL: 1
    float *grad;               // [L, R * C]
    float *slots;              // the parts' sums: slot i at i * slot_stride
    int slices;                // column ranges
};
struct GradArgs {
    Plan plan;                 // tiles: the parts
    GradProduct p[2];
    int R;
    int64_t slot_stride;
    unsigned int *arrived;     // zeros: parts of a split adapter's column range that are done
    int parts;
    bool alone;                // no kernel of this call comes before
    unsigned int *err;
    unsigned long long limit_ns;
};
cudaError_t launch_grad(const GradArgs &a, int parts, cudaStream_t s);

// Tiles of up to 16 tokens: the whole adapter in one kernel.

struct SmallArgs {
    Plan plan;
    const uint16_t *x, *A, *B;
    int64_t ldx;
    int K, N, R;
    int ax, aa, ab;            // alignment of the rows of x, A and B, bytes
    int wide;                  // rows of base and out start at 16-byte multiples, N a multiple of 8
    const float *scale;
    const void *base;
    int base_f32;
    int64_t ldb;
    void *out;
    int64_t ldo;
    float *u;                  // NULL: not wanted
    int tiles, cluster;
    PassArgs pass;             // rows that the CTAs after the tiles' take along (n = 0: none)
};
// CTAs a tile (1, 2, 4, 8) and what the launch takes then, in microseconds; most: tokens of the fullest tile
int small_cluster(int64_t tiles, int most, int64_t K, int64_t N, int64_t R, double *us);
cudaError_t launch_small(bt_dtype t, bool out_f32, const SmallArgs &a, int tiles, int most, cudaStream_t s);

// `grid` CTAs in clusters of c, programmatic dependent launch allowed.
template <typename K, typename Args>
cudaError_t launch_cluster(K kern, int grid, int c, int threads, int smem, cudaStream_t s, const Args &a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(c);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace adapter
}  // namespace bt
