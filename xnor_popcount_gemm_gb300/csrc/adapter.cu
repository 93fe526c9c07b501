// Low-rank adapters of many requests beside one shared projection:
//   out_t = cast(base_t + s_a B_a (A_a x_t)),     a = the adapter of token t
// and the gradients
//   dU_t = s_a B_a^T g_t,   dX_t = cast(gbase_t + A_a^T dU_t),
//   dA_a = sum_t dU_t x_t^T,   dB_a = s_a sum_t g_t u_t^T     (u_t = A_a x_t).
//
// Four products around a rank R of at most 128, all bound by the long rows
// that they read or write once (x, g, base, out: 2 R operations for 2 or 4
// bytes), not by arithmetic:
//   shrink   u = x A^T, dU = g B           reduces the long axis
//   expand   out = base + s u B^T, dX      writes the long axis
//   grad     dA = dU^T x, dB = g^T u       reduces the tokens
// The 16-bit operands go to the matrix instructions as they are; u and dU, fp32
// sums, go as the sum of two 16-bit values (16 bits or more of mantissa), so
// that the only rounding to 16 bits is the result's own.
//
// Tokens of an adapter are gathered through the plan's row list: a tile's rows
// lie anywhere in the batch.
#include <cmath>
#include <mutex>
#include <type_traits>

#include "adapter_plan.h"
#include "bt_device.cuh"
#include "tc_ptx.cuh"

namespace bt {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 64;                  // reduction elements of a stage

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
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
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
// Half precision reaches 65504 and ends at 2^-24: rows of u are brought to a
// largest value of about 2^14 by a power of two first (taken out again in fp32).
template <typename T> __device__ __forceinline__ float row_power(float amax) {
    if constexpr (std::is_same<T, __half>::value) {
        if (!(amax > 0.0f) || isinf(amax)) return 1.0f;
        int e = 14 - ilogbf(amax);
        e = e > 100 ? 100 : e < -100 ? -100 : e;
        return exp2f(static_cast<float>(e));
    }
    return 1.0f;
}

// ---------------------------------------------------------------------------
// Eight consecutive elements of a global row to shared memory (16 bytes, 16-byte
// aligned), `valid` of them there (<= 0: none), the rest zeros. AL: bytes that
// every row of the operand starts at a multiple of.
// ---------------------------------------------------------------------------
template <int B> __device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(B), "r"(bytes) : "memory");
}
__device__ __forceinline__ int clamp_to(int v, int hi) { return v < 0 ? 0 : v > hi ? hi : v; }
__device__ __forceinline__ void copy8(uint16_t *dst, const uint16_t *src, int valid, int al) {
    if (al == 16) {
        cp_async_16(dst, src, clamp_to(valid, 8) * 2);
    } else if (al >= 4) {
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
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < valid ? __ldg(src + 2 * i) : 0u, hi = 2 * i + 1 < valid ? __ldg(src + 2 * i + 1) : 0u;
            w[i] = lo | (hi << 16);
        }
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

struct Plan {
    const int32_t *rows;
    const AdapterTile *tiles;
};

// ---------------------------------------------------------------------------
// shrink: U[t, :] = s sum_c X[t, c] W[c, :] over a tile of 128 rows.
//   WT = false: W is [R, C] (A for u), WT = true: [C, R] (B for dU).
// A cluster of 1 to 8 CTAs shares a tile, each reducing a piece of the long
// axis; the pieces are added in a fixed order through distributed shared
// memory, so that u leaves once and no partial sum touches memory. Eight warps
// of a CTA: 32 rows each, two groups that take every other 16 of a stage's 64
// elements (each B fragment from shared memory then serves two row blocks).
// ---------------------------------------------------------------------------
struct ShrinkArgs {
    Plan plan;
    const uint16_t *x;
    int64_t ldx;
    int ax, aw;                // alignment of the rows of X and W
    const uint16_t *w;         // [L, R, C] or [L, C, R]
    int C, R;
    const float *scale;        // NULL: 1
    float *u;                  // [T, R]
    int cluster;
};

constexpr int kXPitch = kStep + 8;

template <int RP, bool WT> constexpr int kShrinkWElems = WT ? kStep * (RP + 8) : RP * kXPitch;
template <int RP, bool WT> constexpr int kShrinkStageBytes = 2 * (kAdapterTile * kXPitch + kShrinkWElems<RP, WT>);
template <int RP> constexpr int kShrinkStages = RP <= 64 ? 4 : 3;
template <int RP> constexpr int kShrinkSumBytes = 2 * kAdapterTile * RP * 4;
template <int RP, bool WT> constexpr int kShrinkRing = kShrinkStages<RP> * kShrinkStageBytes<RP, WT>;
template <int RP, bool WT> constexpr int kShrinkSmem = kShrinkRing<RP, WT> > kShrinkSumBytes<RP> ? kShrinkRing<RP, WT> : kShrinkSumBytes<RP>;

template <typename T, int RP, bool WT>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) shrink_kernel(const ShrinkArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int rows[kAdapterTile];
    constexpr int S = kShrinkStages<RP>, NB = RP / 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = a.cluster;
    const uint32_t rank = c > 1 ? tc::cluster_ctarank() : 0u;
    pdl_launch_dependents();
    pdl_wait();
    const AdapterTile tile = a.plan.tiles[blockIdx.x / c];
    if (tid < kAdapterTile) rows[tid] = a.plan.rows[tile.first + (tid < tile.n ? tid : 0)];
    const uint16_t *w = a.w + static_cast<int64_t>(tile.adapter) * a.R * a.C;
    const int total = (a.C + kStep - 1) / kStep;
    const int s0 = static_cast<int>(static_cast<int64_t>(total) * rank / c);
    const int n = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / c) - s0;
    __syncthreads();
    // this thread's chunks of a stage: column chunk tid % 8 of rows tid / 8 + 32 i
    const int cc = (tid & 7) * 8;
    const uint16_t *xr[4];
    bool live[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 3) + 32 * i;
        live[i] = r < tile.n;
        xr[i] = a.x + static_cast<int64_t>(rows[r]) * a.ldx;
    }
    auto load = [&](int s) {
        uint16_t *xs = reinterpret_cast<uint16_t *>(smem + (s % S) * kShrinkStageBytes<RP, WT>);
        uint16_t *ws = xs + kAdapterTile * kXPitch;
        const int k0 = (s0 + s) * kStep;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int valid = live[i] ? a.C - k0 - cc : 0;
            copy8(xs + ((tid >> 3) + 32 * i) * kXPitch + cc, valid > 0 ? xr[i] + k0 + cc : a.x, valid, a.ax);
        }
        if constexpr (!WT) {
            for (int i = tid; i < RP * 8; i += kThreads) {
                const int r = i >> 3, k = (i & 7) * 8, valid = r < a.R ? a.C - k0 - k : 0;
                copy8(ws + r * kXPitch + k, valid > 0 ? w + static_cast<int64_t>(r) * a.C + k0 + k : a.w, valid, a.aw);
            }
        } else {
            for (int i = tid; i < kStep * (RP / 8); i += kThreads) {
                const int k = i / (RP / 8), r = (i % (RP / 8)) * 8, valid = k0 + k < a.C ? a.R - r : 0;
                copy8(ws + k * (RP + 8) + r, valid > 0 ? w + static_cast<int64_t>(k0 + k) * a.R + r : a.w, valid, a.aw);
            }
        }
    };
    const int group = warp >> 2, m0 = (warp & 3) * 32;
    float acc[2][NB][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
#pragma unroll
    for (int s = 0; s < S - 1; ++s) {
        if (s < n) load(s);
        cp_async_commit();
    }
    for (int s = 0; s < n; ++s) {
        cp_async_wait<S - 2>();
        __syncthreads();
        if (s + S - 1 < n) load(s + S - 1);
        cp_async_commit();
        const uint16_t *xs = reinterpret_cast<const uint16_t *>(smem + (s % S) * kShrinkStageBytes<RP, WT>);
        const uint16_t *ws = xs + kAdapterTile * kXPitch;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int k = (2 * q + group) * 16;
            uint32_t af[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
                ldsm4(af[m], smem_u32(xs + (m0 + 16 * m + (lane & 15)) * kXPitch + k + (lane >> 4) * 8));
#pragma unroll
            for (int j = 0; j < NB; j += 2) {
                uint32_t bf[4];                              // (k 0-7, k 8-15) of columns 8j.., then of 8(j+1)..
                if constexpr (!WT)
                    ldsm4(bf, smem_u32(ws + (8 * j + (lane >> 4) * 8 + (lane & 7)) * kXPitch + k + ((lane >> 3) & 1) * 8));
                else
                    ldsm4t(bf, smem_u32(ws + (k + (lane & 15)) * (RP + 8) + 8 * j + (lane >> 4) * 8));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma<T>(acc[m][j], af[m], bf[0], bf[1]);
                    mma<T>(acc[m][j + 1], af[m], bf[2], bf[3]);
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    // the two groups' sums, [group][row][r]
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float *p = sums + (group * kAdapterTile + m0 + 16 * m + 8 * h + (lane >> 2)) * RP + 8 * j + 2 * (lane & 3);
                *reinterpret_cast<float2 *>(p) = make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
            }
    if (c > 1) tc::cluster_sync();
    else __syncthreads();
    const float mul = a.scale != nullptr ? a.scale[tile.adapter] : 1.0f;
    const int r0 = kAdapterTile * static_cast<int>(rank) / c, r1 = kAdapterTile * (static_cast<int>(rank) + 1) / c;
    for (int i = tid; i < (r1 - r0) * (RP / 4); i += kThreads) {
        const int row = r0 + i / (RP / 4), r = (i % (RP / 4)) * 4;
        if (row >= tile.n) break;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int q = 0; q < c; ++q)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const uint32_t at = smem_u32(sums + (g * kAdapterTile + row) * RP + r);
                float4 p;
                if (c > 1) {
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w) : "r"(tc::mapa(at, q)) : "memory");
                } else {
                    p = *reinterpret_cast<const float4 *>(sums + (g * kAdapterTile + row) * RP + r);
                }
                v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
            }
        float *u = a.u + static_cast<int64_t>(rows[row]) * a.R + r;
        const float f[4] = {v.x * mul, v.y * mul, v.z * mul, v.w * mul};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (r + e < a.R) u[e] = f[e];
    }
    if (c > 1) tc::cluster_sync();                          // nobody leaves while its sums are read
}

// ---------------------------------------------------------------------------
// expand: OUT[t, c] = cast(BASE[t, c] + s sum_r U[t, r] W[r, c]) over a tile of
// 128 rows and a range of columns, 64 at a time.
//   WT = false: W is [C, R] (B for out), WT = true: [R, C] (A for dX).
// A warp keeps its 16 rows of U in registers, as two 16-bit values each, for
// all columns; W's next 64 columns arrive while these are multiplied.
// ---------------------------------------------------------------------------
struct ExpandArgs {
    Plan plan;
    const float *u;            // [T, R]
    const uint16_t *w;         // [L, C, R] or [L, R, C]
    int aw;
    int C, R;
    const float *scale;        // NULL: 1
    const void *base;          // NULL: 0
    int base_f32;
    int64_t ldb;
    void *out;
    int64_t ldo;
    int wide;                  // rows of base and out start at 16-byte multiples
    int splits;                // column ranges per tile
};

template <int RP, bool WT> constexpr int kExpandWElems = WT ? RP * kXPitch : kStep * (RP + 8);

// 4 x 4 transpose of words across a quad: lane t gives word j to lane j's word t.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t) {
    uint32_t p = (t & 1) ? w[0] : w[1], q = (t & 1) ? w[2] : w[3];
    p = __shfl_xor_sync(0xFFFFFFFFu, p, 1);
    q = __shfl_xor_sync(0xFFFFFFFFu, q, 1);
    if (t & 1) { w[0] = p; w[2] = q; } else { w[1] = p; w[3] = q; }
    p = (t & 2) ? w[0] : w[2];
    q = (t & 2) ? w[1] : w[3];
    p = __shfl_xor_sync(0xFFFFFFFFu, p, 2);
    q = __shfl_xor_sync(0xFFFFFFFFu, q, 2);
    if (t & 2) { w[0] = p; w[1] = q; } else { w[2] = p; w[3] = q; }
}

template <typename T, int RP, bool WT, bool OF32>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) expand_kernel(const ExpandArgs a) {
    __shared__ __align__(128) uint16_t wbuf[2][kExpandWElems<RP, WT>];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    const AdapterTile tile = a.plan.tiles[blockIdx.x / a.splits];
    const int part = blockIdx.x % a.splits;
    const int total = (a.C + kStep - 1) / kStep;
    const int s0 = static_cast<int>(static_cast<int64_t>(total) * part / a.splits);
    const int s1 = static_cast<int>(static_cast<int64_t>(total) * (part + 1) / a.splits);
    const uint16_t *w = a.w + static_cast<int64_t>(tile.adapter) * a.R * a.C;
    auto load = [&](int s) {
        uint16_t *ws = wbuf[s & 1];
        const int c0 = s * kStep;
        if constexpr (!WT) {
            for (int i = tid; i < kStep * (RP / 8); i += kThreads) {
                const int k = i / (RP / 8), r = (i % (RP / 8)) * 8, valid = c0 + k < a.C ? a.R - r : 0;
                copy8(ws + k * (RP + 8) + r, valid > 0 ? w + static_cast<int64_t>(c0 + k) * a.R + r : a.w, valid, a.aw);
            }
        } else {
            for (int i = tid; i < RP * 8; i += kThreads) {
                const int r = i >> 3, k = (i & 7) * 8, valid = r < a.R ? a.C - c0 - k : 0;
                copy8(ws + r * kXPitch + k, valid > 0 ? w + static_cast<int64_t>(r) * a.C + c0 + k : a.w, valid, a.aw);
            }
        }
    };
    load(s0);
    cp_async_commit();
    // U's fragments: rows g and g + 8 of the warp's 16
    const int m0 = warp * 16;
    int row[2];
    bool live[2];
    float mul[2];
    uint32_t uh[RP / 16][4], ul[RP / 16][4];
    const float s = a.scale != nullptr ? a.scale[tile.adapter] : 1.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = m0 + 8 * h + g;
        live[h] = m < tile.n;
        row[h] = a.plan.rows[tile.first + (live[h] ? m : 0)];
        const float *u = a.u + static_cast<int64_t>(row[h]) * a.R;
        float v[RP / 16][4], amax = 0.0f;
#pragma unroll
        for (int k = 0; k < RP / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * k + 2 * t + (e & 1) + (e >> 1) * 8;
                v[k][e] = live[h] && r < a.R ? u[r] : 0.0f;
                amax = fmaxf(amax, fabsf(v[k][e]));
            }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const float p = row_power<T>(amax);
        mul[h] = s / p;
#pragma unroll
        for (int k = 0; k < RP / 16; ++k) {
            split2<T>(v[k][0] * p, v[k][1] * p, uh[k][h], ul[k][h]);
            split2<T>(v[k][2] * p, v[k][3] * p, uh[k][2 + h], ul[k][2 + h]);
        }
    }
    for (int st = s0; st < s1; ++st) {
        cp_async_wait<0>();
        __syncthreads();
        if (st + 1 < s1) load(st + 1);
        cp_async_commit();
        const uint16_t *ws = wbuf[st & 1];
        float acc[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < RP / 16; ++k)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                uint32_t bf[4];
                if constexpr (!WT)
                    ldsm4(bf, smem_u32(ws + (8 * j + (lane >> 4) * 8 + (lane & 7)) * (RP + 8) + 16 * k + ((lane >> 3) & 1) * 8));
                else
                    ldsm4t(bf, smem_u32(ws + (16 * k + (lane & 15)) * kXPitch + 8 * j + (lane >> 4) * 8));
                mma<T>(acc[j], uh[k], bf[0], bf[1]);
                mma<T>(acc[j + 1], uh[k], bf[2], bf[3]);
                mma<T>(acc[j], ul[k], bf[0], bf[1]);
                mma<T>(acc[j + 1], ul[k], bf[2], bf[3]);
            }
        const int c0 = st * kStep;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t bo = static_cast<int64_t>(row[h]) * a.ldb, oo = static_cast<int64_t>(row[h]) * a.ldo;
            if (a.wide) {
                // C a multiple of 8 (16-bit) or 4 (fp32): whole vectors
#pragma unroll
                for (int q = 0; q < 2; ++q) {               // 32 columns: blocks 4q .. 4q + 3
                    float2 v[4];                            // base, then base + s * sum in one rounding each
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = make_float2(0.0f, 0.0f);
                    const int cq = c0 + 32 * q;
                    if (a.base != nullptr) {
                        if (a.base_f32) {
                            const float *b = static_cast<const float *>(a.base) + bo;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int cj = cq + 8 * j + 2 * t;
                                if (live[h] && cj < a.C) v[j] = *reinterpret_cast<const float2 *>(b + cj);
                            }
                        } else {
                            const int cj = cq + 8 * t;
                            uint4 x = make_uint4(0u, 0u, 0u, 0u);
                            if (live[h] && cj < a.C)
                                x = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.base) + bo + cj);
                            uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                            quad_transpose(xw, t);
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] = unpack2<T>(xw[j]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = make_float2(__fmaf_rn(acc[4 * q + j][2 * h], mul[h], v[j].x),
                                           __fmaf_rn(acc[4 * q + j][2 * h + 1], mul[h], v[j].y));
                    if constexpr (OF32) {
                        float *o = static_cast<float *>(a.out) + oo;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int cj = cq + 8 * j + 2 * t;
                            if (live[h] && cj < a.C) *reinterpret_cast<float2 *>(o + cj) = v[j];
                        }
                    } else {
                        uint32_t ow[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) ow[j] = pack2<T>(v[j].x, v[j].y);
                        quad_transpose(ow, t);
                        const int cj = cq + 8 * t;
                        if (live[h] && cj < a.C)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + oo + cj) =
                                make_uint4(ow[0], ow[1], ow[2], ow[3]);
                    }
                }
            } else if (live[h]) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int cj = c0 + 8 * j + 2 * t + e;
                        if (cj >= a.C) continue;
                        float v = 0.0f;
                        if (a.base != nullptr)
                            v = a.base_f32 ? static_cast<const float *>(a.base)[bo + cj]
                                           : Elem<T>::to_f32(static_cast<const T *>(a.base)[bo + cj]);
                        v = __fmaf_rn(acc[j][2 * h + e], mul[h], v);
                        if constexpr (OF32) static_cast<float *>(a.out)[oo + cj] = v;
                        else static_cast<T *>(a.out)[oo + cj] = to16<T>(v);
                    }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Tokens without an adapter: out = cast(base), u = 0.
// ---------------------------------------------------------------------------
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
template <typename T, bool OF32> __global__ void __launch_bounds__(kThreads) pass_kernel(const PassArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = a.rows[blockIdx.x];
    if (a.u != nullptr && blockIdx.y == 0)
        for (int r = threadIdx.x; r < a.R; r += kThreads) a.u[row * a.R + r] = 0.0f;
    if (a.out == nullptr) return;
    for (int c = blockIdx.y * kThreads + threadIdx.x; c < a.N; c += gridDim.y * kThreads) {
        float v = 0.0f;
        if (a.base != nullptr)
            v = a.base_f32 ? static_cast<const float *>(a.base)[row * a.ldb + c]
                           : Elem<T>::to_f32(static_cast<const T *>(a.base)[row * a.ldb + c]);
        if constexpr (OF32) static_cast<float *>(a.out)[row * a.ldo + c] = v;
        else static_cast<T *>(a.out)[row * a.ldo + c] = to16<T>(v);
    }
}

// ---------------------------------------------------------------------------
// grad: G[r, c] = s sum_t U[t, r] X[t, c] over a part of an adapter's tokens and
// 128 columns; a warp has 16 of them and all ranks. Both operands arrive as
// token rows and are transposed on the way to the matrix instruction. A part
// that is its adapter's only one writes the gradient; the others write their
// sums to the workspace, which sum_kernel adds up in order.
// ---------------------------------------------------------------------------
struct GradArgs {
    Plan plan;                 // tiles: the parts
    const float *u;            // [T, R]
    const uint16_t *x;         // [T, C]
    int64_t ldx;
    int ax;
    int C, R;
    int rc;                    // 1: G is [R, C] (dA), 0: [C, R] (dB)
    const float *scale;        // NULL: 1
    float *grad;               // [L, R * C]
    float *slots;              // the parts' sums: slot i at i * slot_stride
    int64_t slot_stride;
    int slices;
};
constexpr int kGradCols = 128, kGradTok = 64, kGradXPitch = kGradCols + 8;
constexpr int kGradStageBytes = 2 * kGradTok * kGradXPitch, kGradStages = 3;
template <int RP> constexpr int kGradUBytes = 2 * 2 * kGradTok * (RP + 8);        // hi and lo
template <int RP> constexpr int kGradSmem = kGradStages * kGradStageBytes + 2 * kGradUBytes<RP>;

template <int RP>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) grad_kernel(const GradArgs a) {
    using T = __nv_bfloat16;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int MB = RP / 16, UP = RP + 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    pdl_wait();
    const AdapterTile part = a.plan.tiles[blockIdx.x / a.slices];
    const int c0 = static_cast<int>(blockIdx.x % a.slices) * kGradCols;
    const int32_t *rows = a.plan.rows + part.first;
    const int n = (part.n + kGradTok - 1) / kGradTok;
    uint8_t *ubase = smem + kGradStages * kGradStageBytes;
    auto load_x = [&](int s) {
        uint16_t *xs = reinterpret_cast<uint16_t *>(smem + (s % kGradStages) * kGradStageBytes);
#pragma unroll
        for (int i = 0; i < kGradTok * (kGradCols / 8) / kThreads; ++i) {
            const int k = i * kThreads + tid, tok = k / (kGradCols / 8), c = (k % (kGradCols / 8)) * 8;
            const int at = s * kGradTok + tok;
            const int valid = at < part.n ? a.C - c0 - c : 0;
            copy8(xs + tok * kGradXPitch + c, valid > 0 ? a.x + static_cast<int64_t>(rows[at]) * a.ldx + c0 + c : a.x, valid, a.ax);
        }
    };
    // U's chunk: thread (token tid / 4, a quarter of the ranks), pairs of ranks
    constexpr int UV = RP / 8;                              // pairs per thread
    const int utok = tid >> 2, ur = (tid & 3) * 2;
    float2 uv[UV];
    auto load_u = [&](int s) {
        const int at = s * kGradTok + utok;
        const bool ok = at < part.n;
        const float *u = a.u + static_cast<int64_t>(ok ? rows[at] : 0) * a.R;
#pragma unroll
        for (int i = 0; i < UV; ++i) {
            const int r = ur + 8 * i;
            uv[i].x = ok && r < a.R ? u[r] : 0.0f;
            uv[i].y = ok && r + 1 < a.R ? u[r + 1] : 0.0f;
        }
    };
    auto store_u = [&](int s) {
        uint16_t *hi = reinterpret_cast<uint16_t *>(ubase + (s & 1) * kGradUBytes<RP>), *lo = hi + kGradTok * UP;
#pragma unroll
        for (int i = 0; i < UV; ++i) {
            uint32_t h, l;
            split2<T>(uv[i].x, uv[i].y, h, l);
            *reinterpret_cast<uint32_t *>(hi + utok * UP + ur + 8 * i) = h;
            *reinterpret_cast<uint32_t *>(lo + utok * UP + ur + 8 * i) = l;
        }
    };
    float acc[MB][2][4];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
#pragma unroll
    for (int s = 0; s < kGradStages - 1; ++s) {
        if (s < n) load_x(s);
        cp_async_commit();
    }
    if (n > 0) {
        load_u(0);
        store_u(0);
        if (n > 1) load_u(1);
    }
    for (int s = 0; s < n; ++s) {
        cp_async_wait<kGradStages - 2>();
        __syncthreads();
        if (s + kGradStages - 1 < n) load_x(s + kGradStages - 1);
        cp_async_commit();
        if (s + 1 < n) {
            store_u(s + 1);
            if (s + 2 < n) load_u(s + 2);
        }
        const uint16_t *xs = reinterpret_cast<const uint16_t *>(smem + (s % kGradStages) * kGradStageBytes);
        const uint16_t *hi = reinterpret_cast<const uint16_t *>(ubase + (s & 1) * kGradUBytes<RP>), *lo = hi + kGradTok * UP;
#pragma unroll
        for (int k = 0; k < kGradTok; k += 16) {
            uint32_t bf[4];
            ldsm4t(bf, smem_u32(xs + (k + (lane & 15)) * kGradXPitch + 16 * warp + (lane >> 4) * 8));
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                uint32_t af[4];
                const int off = (k + (lane >> 4) * 8 + (lane & 7)) * UP + 16 * m + ((lane >> 3) & 1) * 8;
                ldsm4t(af, smem_u32(hi + off));
                mma<T>(acc[m][0], af, bf[0], bf[1]);
                mma<T>(acc[m][1], af, bf[2], bf[3]);
                ldsm4t(af, smem_u32(lo + off));
                mma<T>(acc[m][0], af, bf[0], bf[1]);
                mma<T>(acc[m][1], af, bf[2], bf[3]);
            }
        }
    }
    cp_async_wait<0>();
    const float s = a.scale != nullptr ? a.scale[part.adapter] : 1.0f;
    float *out = part.slot >= 0 ? a.slots + part.slot * a.slot_stride
                                : a.grad + static_cast<int64_t>(part.adapter) * a.R * a.C;
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * m + (lane >> 2) + (e >> 1) * 8, c = c0 + 16 * warp + 8 * j + 2 * (lane & 3) + (e & 1);
                if (r < a.R && c < a.C)
                    out[a.rc ? static_cast<int64_t>(r) * a.C + c : static_cast<int64_t>(c) * a.R + r] = acc[m][j][e] * s;
            }
}

// Adds the parts of every adapter that has several; those come first in the
// plan, and block y takes part y if an adapter begins there.
struct SumArgs {
    const AdapterTile *parts;
    int n;                     // parts with a slot
    const float *slots;
    int64_t slot_stride;
    int64_t len_a, len_b;      // R * K, R * N: the two gradients lie one after the other in a slot
    int64_t off_b;             // where the second begins in a slot
    float *grad_a, *grad_b;
};
__global__ void __launch_bounds__(kThreads) sum_kernel(const SumArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int p = blockIdx.y;
    const AdapterTile first = a.parts[p];
    if (p > 0 && a.parts[p - 1].adapter == first.adapter) return;
    int k = 1;
    while (p + k < a.n && a.parts[p + k].adapter == first.adapter) ++k;
    const float *s = a.slots + first.slot * a.slot_stride;
    const int64_t total = a.len_a + a.len_b;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t at = i < a.len_a ? i : a.off_b + (i - a.len_a);
        float v = s[at];
        for (int q = 1; q < k; ++q) v += s[q * a.slot_stride + at];
        if (i < a.len_a) a.grad_a[first.adapter * a.len_a + i] = v;
        else a.grad_b[first.adapter * a.len_b + i - a.len_a] = v;
    }
}

// ---------------------------------------------------------------------------
// Few tokens of many adapters (decoding): the whole adapter in one kernel. A
// cluster of 1 to 8 CTAs takes up to 16 tokens of one adapter. Each CTA reduces
// a piece of the long axis, the pieces are exchanged through distributed shared
// memory, and each CTA writes a range of the columns. Weights go from memory
// straight to the registers of the matrix instructions, 16 bytes a lane: the
// reduction index may be permuted as long as both operands agree, so lane t of
// a quad takes elements 8t .. 8t + 7 of 32 as its share of two instructions.
// The first of B's rows are fetched before anything waits for the sums: a
// token costs about one trip to memory and one exchange.
//
// The rank (A's rows) and the columns (B's rows) are the 16 rows of the
// instruction, tokens its 8 columns.
// ---------------------------------------------------------------------------
struct SmallArgs {
    Plan plan;
    const uint16_t *x, *A, *B;
    int64_t ldx;
    int K, N, R;
    int vec_k, vec_r;          // rows of x and A, rows of B start at 16-byte multiples (B: R a multiple of 8)
    const float *scale;
    const void *base;
    int base_f32;
    int64_t ldb;
    void *out;
    int64_t ldo;
    float *u;                  // NULL: not wanted
    int cluster;
};

// Elements k .. k + 7 of a row of n, zeros beyond; VEC: k + 8 <= n or k >= n, and 16-byte aligned.
__device__ __forceinline__ uint4 row8(const uint16_t *p, int k, int n, bool vec) {
    if (vec) return k < n ? __ldg(reinterpret_cast<const uint4 *>(p + k)) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = k + 2 * i < n ? __ldg(p + k + 2 * i) : 0u, hi = k + 2 * i + 1 < n ? __ldg(p + k + 2 * i + 1) : 0u;
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// RB: blocks of 16 ranks; NB: blocks of 8 tokens.
template <typename T, int RB, int NB, bool OF32>
__global__ void __launch_bounds__(kThreads, RB <= 4 ? 2 : 1) small_kernel(const SmallArgs a) {
    constexpr int RP = 16 * RB, TOK = 8 * NB, UP = RP + 4;
    constexpr int RK = (RB + 1) / 2;                        // 32-rank pieces of B's rows
    constexpr int PRE = RK == 1 ? 4 : RK == 2 ? 2 : 1;      // B's row blocks fetched ahead
    extern __shared__ __align__(128) uint8_t smem[];
    float(*part)[TOK][UP] = reinterpret_cast<float(*)[TOK][UP]>(smem);                                 // [warp]
    float(*slot)[TOK][RP] = reinterpret_cast<float(*)[TOK][RP]>(smem + 8 * TOK * UP * sizeof(float));  // [rank]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int c = a.cluster;
    const int rank = c > 1 ? static_cast<int>(tc::cluster_ctarank()) : 0;
    pdl_launch_dependents();
    pdl_wait();
    const AdapterTile tile = a.plan.tiles[blockIdx.x / c];
    const uint16_t *A = a.A + static_cast<int64_t>(tile.adapter) * a.R * a.K;
    const uint16_t *B = a.B + static_cast<int64_t>(tile.adapter) * a.R * a.N;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

    // columns of this CTA, in blocks of 16; this warp's are b0 + warp, b0 + warp + 8, ...
    const int blocks = (a.N + 15) / 16;
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / c);
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / c);
    auto load_b = [&](int b, uint4 (&w)[RK][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int n = 16 * b + 8 * h + g;
            const uint16_t *p = B + static_cast<int64_t>(n) * a.R;
#pragma unroll
            for (int q = 0; q < RK; ++q) w[q][h] = b < b1 && n < a.N ? row8(p, 32 * q + 8 * t, a.R, a.vec_r) : zero;
        }
    };

    float acc[RB][NB][4];
#pragma unroll
    for (int m = 0; m < RB; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
    const uint16_t *xr[NB];
    bool live[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        live[j] = 8 * j + g < tile.n;
        xr[j] = a.x + static_cast<int64_t>(a.plan.rows[tile.first + (live[j] ? 8 * j + g : 0)]) * a.ldx;
    }
    uint4 wb[PRE][RK][2];
#pragma unroll
    for (int i = 0; i < PRE; ++i) load_b(b0 + warp + 8 * i, wb[i]);
    // this warp's steps of 32 elements
    const int steps = (a.K + 31) / 32, who = rank * 8 + warp, all = c * 8;
#pragma unroll 2
    for (int s = who; s < steps; s += all) {
        const int k = 32 * s + 8 * t;
        uint4 xv[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) xv[j] = live[j] ? row8(xr[j], k, a.K, a.vec_k) : zero;
#pragma unroll
        for (int m = 0; m < RB; ++m) {
            const int r0 = 16 * m + g, r1 = r0 + 8;
            const uint4 w0 = r0 < a.R ? row8(A + static_cast<int64_t>(r0) * a.K, k, a.K, a.vec_k) : zero;
            const uint4 w1 = r1 < a.R ? row8(A + static_cast<int64_t>(r1) * a.K, k, a.K, a.vec_k) : zero;
            const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                mma<T>(acc[m][j], f0, xv[j].x, xv[j].y);
                mma<T>(acc[m][j], f1, xv[j].z, xv[j].w);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < RB; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[warp][8 * j + 2 * t + (e & 1)][16 * m + g + (e >> 1) * 8] = acc[m][j][e];
    __syncthreads();
    if (c > 1) tc::cluster_sync();                          // every CTA of the cluster has started
    for (int i = tid; i < TOK * RP; i += kThreads) {
        const int tok = i / RP, r = i % RP;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += part[w][tok][r];
        const uint32_t at = smem_u32(&slot[rank][tok][r]);
        if (c == 1) {
            slot[0][tok][r] = v;
        } else {
            for (int q = 0; q < c; ++q)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa(at, q)), "f"(v) : "memory");
        }
    }
    if (c > 1) tc::cluster_sync();
    else __syncthreads();
    // u of this tile's tokens, whole, in part[0]
    float(*u)[UP] = part[0];
    for (int i = tid; i < TOK * RP; i += kThreads) {
        const int tok = i / RP, r = i % RP;
        float v = 0.0f;
        for (int q = 0; q < c; ++q) v += slot[q][tok][r];
        u[tok][r] = v;
        if (a.u != nullptr && rank == 0 && tok < tile.n && r < a.R)
            a.u[static_cast<int64_t>(a.plan.rows[tile.first + tok]) * a.R + r] = v;
    }
    __syncthreads();
    // its fragments: lane t of a quad holds ranks 32q + 8t .. + 7 of token g
    const float s = a.scale[tile.adapter];
    uint32_t uh[RK][NB][4], ul[RK][NB][4];
    float mul[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        float v[RK][8], amax = 0.0f;
#pragma unroll
        for (int q = 0; q < RK; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int r = 32 * q + 8 * t + e;
                v[q][e] = r < RP ? u[8 * j + g][r] : 0.0f;
                amax = fmaxf(amax, fabsf(v[q][e]));
            }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const float p = row_power<T>(amax);
        mul[j] = s / p;
#pragma unroll
        for (int q = 0; q < RK; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) split2<T>(v[q][2 * e] * p, v[q][2 * e + 1] * p, uh[q][j][e], ul[q][j][e]);
    }
    // a result's tokens are 2t and 2t + 1: their rows and multipliers
    int64_t row[NB][2];
    bool there[NB][2];
    float m2[NB][2];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int tok = 8 * j + 2 * t + e;
            there[j][e] = tok < tile.n;
            row[j][e] = a.plan.rows[tile.first + (there[j][e] ? tok : 0)];
            m2[j][e] = __shfl_sync(0xFFFFFFFFu, mul[j], (2 * t + e) * 4);
        }
    for (int first = b0 + warp; first < b1; first += 8 * PRE) {
#pragma unroll
        for (int i = 0; i < PRE; ++i) {
            const int b = first + 8 * i;
            if (b >= b1) break;
            float d[NB][4];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.0f;
#pragma unroll
                for (int q = 0; q < RK; ++q) {
                    const uint4 w0 = wb[i][q][0], w1 = wb[i][q][1];
                    const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
                    mma<T>(d[j], f0, uh[q][j][0], uh[q][j][1]);
                    mma<T>(d[j], f1, uh[q][j][2], uh[q][j][3]);
                    mma<T>(d[j], f0, ul[q][j][0], ul[q][j][1]);
                    mma<T>(d[j], f1, ul[q][j][2], ul[q][j][3]);
                }
            }
            load_b(b + 8 * PRE, wb[i]);
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int n = 16 * b + g + (e >> 1) * 8;
                    if (!there[j][e & 1] || n >= a.N) continue;
                    float v = 0.0f;
                    if (a.base != nullptr)
                        v = a.base_f32 ? static_cast<const float *>(a.base)[row[j][e & 1] * a.ldb + n]
                                       : Elem<T>::to_f32(static_cast<const T *>(a.base)[row[j][e & 1] * a.ldb + n]);
                    v = __fmaf_rn(d[j][e], m2[j][e & 1], v);
                    if constexpr (OF32) static_cast<float *>(a.out)[row[j][e & 1] * a.ldo + n] = v;
                    else static_cast<T *>(a.out)[row[j][e & 1] * a.ldo + n] = to16<T>(v);
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// The largest of 16, 8, 4, 2 bytes that p and every multiple of `bytes` share.
int align_of(const void *p, int64_t bytes) {
    const uintptr_t v = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(bytes);
    return v % 16 == 0 ? 16 : v % 8 == 0 ? 8 : v % 4 == 0 ? 4 : 2;
}
template <typename K> cudaError_t allow_smem(K kern, int bytes, std::once_flag &once, cudaError_t &err) {
    std::call_once(once, [&] { err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
    return err;
}

// `grid` CTAs in clusters of c, programmatic dependent launch allowed.
template <typename K, typename Args>
cudaError_t launch_cluster(K kern, int grid, int c, int smem, cudaStream_t s, const Args &a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(c);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, int RP, bool WT> cudaError_t launch_shrink_rp(ShrinkArgs a, int tiles, cudaStream_t s) {
    auto kern = shrink_kernel<T, RP, WT>;
    constexpr int smem = kShrinkSmem<RP, WT>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(kern, smem, once, err) != cudaSuccess) return err;
    const int steps = (a.C + kStep - 1) / kStep;
    int c = 1;
    // pieces of at least four stages until the CTAs fill the machine twice
    while (c < 8 && tiles * c < 2 * device_sm_count() && steps >= 8 * c) c *= 2;
    a.cluster = c;
    return launch_cluster(kern, tiles * c, c, smem, s, static_cast<const ShrinkArgs>(a));
}
template <typename T, bool WT> cudaError_t launch_shrink(const ShrinkArgs &a, int tiles, cudaStream_t s) {
    if (tiles == 0) return cudaSuccess;
    if (a.R <= 16) return launch_shrink_rp<T, 16, WT>(a, tiles, s);
    if (a.R <= 32) return launch_shrink_rp<T, 32, WT>(a, tiles, s);
    if (a.R <= 64) return launch_shrink_rp<T, 64, WT>(a, tiles, s);
    return launch_shrink_rp<T, 128, WT>(a, tiles, s);
}

template <typename T, bool WT, bool OF32> cudaError_t launch_expand(ExpandArgs a, int tiles, cudaStream_t s) {
    if (tiles == 0) return cudaSuccess;
    const int steps = (a.C + kStep - 1) / kStep;
    int splits = (4 * device_sm_count() + tiles - 1) / tiles;
    if (splits > steps) splits = steps;
    a.splits = splits < 1 ? 1 : splits;
    const dim3 grid(static_cast<unsigned>(tiles * a.splits)), block(kThreads);
    if (a.R <= 16) return launch_pdl(expand_kernel<T, 16, WT, OF32>, grid, block, s, a);
    if (a.R <= 32) return launch_pdl(expand_kernel<T, 32, WT, OF32>, grid, block, s, a);
    if (a.R <= 64) return launch_pdl(expand_kernel<T, 64, WT, OF32>, grid, block, s, a);
    return launch_pdl(expand_kernel<T, 128, WT, OF32>, grid, block, s, a);
}

template <int RP> cudaError_t launch_grad_rp(const GradArgs &a, int parts, cudaStream_t s) {
    auto kern = grad_kernel<RP>;
    constexpr int smem = kGradSmem<RP>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(kern, smem, once, err) != cudaSuccess) return err;
    return launch_pdl_smem(kern, dim3(static_cast<unsigned>(parts * a.slices)), dim3(kThreads), smem, s, a);
}
cudaError_t launch_grad(GradArgs a, int parts, cudaStream_t s) {
    a.slices = (a.C + kGradCols - 1) / kGradCols;
    if (a.R <= 16) return launch_grad_rp<16>(a, parts, s);
    if (a.R <= 32) return launch_grad_rp<32>(a, parts, s);
    if (a.R <= 64) return launch_grad_rp<64>(a, parts, s);
    return launch_grad_rp<128>(a, parts, s);
}

template <typename T, int RB, int NB, bool OF32> cudaError_t launch_small_rn(SmallArgs a, int tiles, cudaStream_t s) {
    int c = 1;
    // the widest cluster with two CTAs an SM, or up to 8 where the tiles do not fill the machine once
    while (c < 8 && tiles * c * 2 <= 2 * device_sm_count()) c *= 2;
    a.cluster = c;
    auto kern = small_kernel<T, RB, NB, OF32>;
    constexpr int smem = 8 * 8 * NB * (32 * RB + 4) * static_cast<int>(sizeof(float));
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(kern, smem, once, err) != cudaSuccess) return err;
    return launch_cluster(kern, tiles * c, c, smem, s, static_cast<const SmallArgs>(a));
}
template <typename T, int NB, bool OF32> cudaError_t launch_small_n(const SmallArgs &a, int tiles, cudaStream_t s) {
    if (a.R <= 16) return launch_small_rn<T, 1, NB, OF32>(a, tiles, s);
    if (a.R <= 32) return launch_small_rn<T, 2, NB, OF32>(a, tiles, s);
    if (a.R <= 64) return launch_small_rn<T, 4, NB, OF32>(a, tiles, s);
    return launch_small_rn<T, 8, NB, OF32>(a, tiles, s);
}
// most: tokens of the largest tile
template <typename T, bool OF32> cudaError_t launch_small(const SmallArgs &a, int tiles, int most, cudaStream_t s) {
    if (tiles == 0) return cudaSuccess;
    return most <= 8 ? launch_small_n<T, 1, OF32>(a, tiles, s) : launch_small_n<T, 2, OF32>(a, tiles, s);
}

template <typename T, bool OF32> cudaError_t launch_pass(const PassArgs &a, cudaStream_t s) {
    if (a.n == 0 || (a.out == nullptr && a.u == nullptr)) return cudaSuccess;
    const unsigned y = static_cast<unsigned>(a.N < 4 * kThreads ? 1 : a.N < 16 * kThreads ? 2 : 4);
    return launch_pdl(pass_kernel<T, OF32>, dim3(static_cast<unsigned>(a.n), y), dim3(kThreads), s, a);
}

constexpr int64_t kMaxSide = int64_t(1) << 24;

bool plan_fits(const bt_adapter_plan_info &p, int64_t T) {
    return p.tokens == T && p.adapters >= 1 && p.adapters <= kAdapterMaxAdapters && p.without >= 0 && p.without <= T &&
           p.tiles >= 0 && p.tiles <= T && p.large_tiles >= 0 && p.large_tiles <= p.tiles && p.small_tiles >= 0 &&
           p.small_tiles <= T && p.small_most >= 0 && p.small_most <= kAdapterSmall && p.parts >= 1 && p.parts <= 2 * kAdapterParts + p.adapters + 1 && p.slots >= 0 &&
           p.slots <= 2 * kAdapterParts;
}
bt_status sizes_fit(int64_t T, int64_t K, int64_t N, int64_t R) {
    if (T < 0 || K < 1 || N < 0 || R < 1) return BT_ERR_INVALID_ARG;
    if (T > kAdapterMaxTokens || K >= kMaxSide || N >= kMaxSide || R > kAdapterMaxRank) return BT_ERR_UNSUPPORTED;
    return BT_OK;
}

struct Forward {
    const uint16_t *x, *A, *B;
    int64_t ldx, ldb, ldo;
    const float *scale;
    const int32_t *plan;
    const bt_adapter_plan_info *info;
    int64_t T;
    int K, N, R;
    const void *base;
    int base_f32;
    void *out;
    float *u;
    bool want_u;
};

template <typename T, bool OF32> cudaError_t forward(const Forward &f, cudaStream_t s) {
    const AdapterPlanLayout lay = adapter_plan_layout(f.T, f.info->adapters);
    const Plan plan{f.plan + lay.rows, reinterpret_cast<const AdapterTile *>(f.plan + lay.tiles)};
    cudaError_t e;
    if (f.info->small_tiles > 0) {
        SmallArgs sm = {};
        sm.plan = Plan{plan.rows, reinterpret_cast<const AdapterTile *>(f.plan + lay.small)};
        sm.x = f.x; sm.A = f.A; sm.B = f.B; sm.ldx = f.ldx;
        sm.K = f.K; sm.N = f.N; sm.R = f.R;
        sm.vec_k = f.K % 8 == 0 && align_of(f.x, f.ldx * 2) == 16 && align_of(f.A, 16) == 16;
        sm.vec_r = f.R % 8 == 0 && align_of(f.B, 16) == 16;
        sm.scale = f.scale;
        sm.base = f.base; sm.base_f32 = f.base_f32; sm.ldb = f.ldb;
        sm.out = f.out; sm.ldo = f.ldo;
        sm.u = f.want_u ? f.u : nullptr;
        e = launch_small<T, OF32>(sm, f.info->small_tiles, f.info->small_most, s);
        if (e != cudaSuccess) return e;
    }
    ShrinkArgs sh = {};
    sh.plan = plan;
    sh.x = f.x; sh.ldx = f.ldx; sh.ax = align_of(f.x, f.ldx * 2);
    sh.w = f.A; sh.aw = align_of(f.A, int64_t(f.K) * 2);
    sh.C = f.K; sh.R = f.R; sh.u = f.u;
    e = launch_shrink<T, false>(sh, f.info->large_tiles, s);
    if (e != cudaSuccess) return e;
    ExpandArgs ex = {};
    ex.plan = plan;
    ex.u = f.u; ex.w = f.B; ex.aw = align_of(f.B, int64_t(f.R) * 2);
    ex.C = f.N; ex.R = f.R; ex.scale = f.scale;
    ex.base = f.base; ex.base_f32 = f.base_f32; ex.ldb = f.ldb;
    ex.out = f.out; ex.ldo = f.ldo;
    ex.wide = align_of(f.out, f.ldo * (OF32 ? 4 : 2)) == 16 &&
              (f.base == nullptr || align_of(f.base, f.ldb * (f.base_f32 ? 4 : 2)) == 16) && f.N % 8 == 0;
    e = launch_expand<T, false, OF32>(ex, f.info->large_tiles, s);
    if (e != cudaSuccess) return e;
    PassArgs pa = {};
    pa.n = f.info->without;
    pa.rows = plan.rows + (f.T - pa.n);
    pa.N = f.N; pa.R = f.R;
    pa.base = f.base; pa.base_f32 = f.base_f32; pa.ldb = f.ldb;
    pa.out = f.out == f.base ? nullptr : f.out; pa.ldo = f.ldo;
    pa.u = f.want_u ? f.u : nullptr;
    return launch_pass<T, OF32>(pa, s);
}

}  // namespace
}  // namespace bt

using namespace bt;

extern "C" {

size_t bt_adapter_linear_workspace(int64_t T, int64_t R, const bt_adapter_plan_info *info, int have_u) {
    if (have_u || sizes_fit(T, 1, 0, R) != BT_OK || info == nullptr || info->large_tiles == 0) return 0;
    return round_up256(static_cast<size_t>(T * R) * 4);
}

bt_status bt_adapter_linear(const void *x, bt_dtype x_dtype, int64_t ldx, const void *A, const void *B,
                            const float *scale, const void *plan, const bt_adapter_plan_info *info, int64_t T,
                            int64_t K, int64_t N, int64_t R, const void *base, bt_dtype base_dtype, int64_t ldb,
                            void *out, bt_dtype out_dtype, int64_t ldo, float *u, void *workspace,
                            size_t workspace_bytes, bt_stream stream) {
    if (x_dtype != BT_BF16 && x_dtype != BT_F16) return BT_ERR_INVALID_ARG;
    if (out_dtype != BT_F32 && out_dtype != x_dtype) return BT_ERR_INVALID_ARG;
    if (base != nullptr && base_dtype != BT_F32 && base_dtype != x_dtype) return BT_ERR_INVALID_ARG;
    const bt_status fit = sizes_fit(T, K, N, R);
    if (fit != BT_OK) return fit;
    if (ldx < K || ldo < N || (base != nullptr && ldb < N)) return BT_ERR_INVALID_ARG;
    if (ldx > (int64_t(1) << 36) || ldo > (int64_t(1) << 36) || ldb > (int64_t(1) << 36)) return BT_ERR_UNSUPPORTED;
    if (info == nullptr || !plan_fits(*info, T)) return BT_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return BT_OK;
    if (x == nullptr || A == nullptr || B == nullptr || scale == nullptr || plan == nullptr || out == nullptr)
        return BT_ERR_INVALID_ARG;
    if (out == base && (out_dtype != base_dtype || ldo != ldb)) return BT_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(scale, 4) || !aligned(plan, 16) || !aligned(u, 4) ||
        !aligned(out, dtype_bytes(out_dtype)) || (base != nullptr && !aligned(base, dtype_bytes(base_dtype))))
        return BT_ERR_ALIGNMENT;
    const size_t need = bt_adapter_linear_workspace(T, R, info, u != nullptr);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BT_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return BT_ERR_ALIGNMENT;
    Forward f = {};
    f.x = static_cast<const uint16_t *>(x);
    f.A = static_cast<const uint16_t *>(A);
    f.B = static_cast<const uint16_t *>(B);
    f.ldx = ldx; f.ldb = ldb; f.ldo = ldo;
    f.scale = scale;
    f.plan = static_cast<const int32_t *>(plan);
    f.info = info;
    f.T = T; f.K = static_cast<int>(K); f.N = static_cast<int>(N); f.R = static_cast<int>(R);
    f.base = base; f.base_f32 = base_dtype == BT_F32;
    f.out = out;
    f.want_u = u != nullptr;
    f.u = u != nullptr ? u : static_cast<float *>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (x_dtype == BT_BF16) e = out_dtype == BT_F32 ? forward<__nv_bfloat16, true>(f, s) : forward<__nv_bfloat16, false>(f, s);
    else e = out_dtype == BT_F32 ? forward<__half, true>(f, s) : forward<__half, false>(f, s);
    return e == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

size_t bt_adapter_linear_backward_workspace(int64_t T, int64_t K, int64_t N, int64_t R,
                                            const bt_adapter_plan_info *info) {
    if (sizes_fit(T, K, N, R) != BT_OK || info == nullptr || !plan_fits(*info, T)) return 0;
    const size_t slot = round_up256(static_cast<size_t>(R * K) * 4) + round_up256(static_cast<size_t>(R * N) * 4);
    return round_up256(static_cast<size_t>(T * R) * 4) + static_cast<size_t>(info->slots) * slot;
}

bt_status bt_adapter_linear_backward(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *u,
                                     const void *A, const void *B, const float *scale, const void *plan,
                                     const bt_adapter_plan_info *info, int64_t T, int64_t K, int64_t N, int64_t R,
                                     const void *grad_base, int64_t ldgb, void *grad_x, int64_t ldgx, float *grad_A,
                                     float *grad_B, void *workspace, size_t workspace_bytes, bt_stream stream) {
    const bt_status fit = sizes_fit(T, K, N, R);
    if (fit != BT_OK) return fit;
    if (N < 1 || ldx < K || ldg < N || ldgx < K || (grad_base != nullptr && ldgb < K)) return BT_ERR_INVALID_ARG;
    if (ldx > (int64_t(1) << 36) || ldg > (int64_t(1) << 36) || ldgx > (int64_t(1) << 36) || ldgb > (int64_t(1) << 36))
        return BT_ERR_UNSUPPORTED;
    if (info == nullptr || !plan_fits(*info, T)) return BT_ERR_INVALID_ARG;
    if (static_cast<int64_t>(info->parts) * ((K > N ? K : N) / kGradCols + 1) > 0x7FFFFFFF) return BT_ERR_UNSUPPORTED;
    if (plan == nullptr || grad_A == nullptr || grad_B == nullptr) return BT_ERR_INVALID_ARG;
    if (T > 0 && (x == nullptr || g == nullptr || u == nullptr || A == nullptr || B == nullptr || scale == nullptr ||
                  grad_x == nullptr))
        return BT_ERR_INVALID_ARG;
    if (grad_x != nullptr && grad_x == grad_base && ldgx != ldgb) return BT_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(g, 2) || !aligned(u, 4) || !aligned(A, 2) || !aligned(B, 2) || !aligned(scale, 4) ||
        !aligned(plan, 16) || !aligned(grad_base, 2) || !aligned(grad_x, 2) || !aligned(grad_A, 4) || !aligned(grad_B, 4))
        return BT_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        const size_t n = static_cast<size_t>(info->adapters) * static_cast<size_t>(R) * 4;
        return cudaMemsetAsync(grad_A, 0, n * static_cast<size_t>(K), s) == cudaSuccess &&
               cudaMemsetAsync(grad_B, 0, n * static_cast<size_t>(N), s) == cudaSuccess ? BT_OK : BT_ERR_CUDA;
    }
    const size_t need = bt_adapter_linear_backward_workspace(T, K, N, R, info);
    if (workspace == nullptr || workspace_bytes < need) return BT_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BT_ERR_ALIGNMENT;

    using E = __nv_bfloat16;
    const uint16_t *xp = static_cast<const uint16_t *>(x), *gp = static_cast<const uint16_t *>(g);
    const uint16_t *Ap = static_cast<const uint16_t *>(A), *Bp = static_cast<const uint16_t *>(B);
    const int32_t *pw = static_cast<const int32_t *>(plan);
    const AdapterPlanLayout lay = adapter_plan_layout(T, info->adapters);
    const Plan tiles{pw + lay.rows, reinterpret_cast<const AdapterTile *>(pw + lay.tiles)};
    const Plan parts{pw + lay.rows, reinterpret_cast<const AdapterTile *>(pw + lay.parts)};
    float *du = static_cast<float *>(workspace);
    float *slots = du + round_up256(static_cast<size_t>(T * R) * 4) / 4;
    const int64_t off_b = static_cast<int64_t>(round_up256(static_cast<size_t>(R * K) * 4) / 4);
    const int64_t stride = off_b + static_cast<int64_t>(round_up256(static_cast<size_t>(R * N) * 4) / 4);
    const int ax = align_of(x, ldx * 2), ag = align_of(g, ldg * 2);

    ShrinkArgs sh = {};
    sh.plan = tiles;
    sh.x = gp; sh.ldx = ldg; sh.ax = ag;
    sh.w = Bp; sh.aw = align_of(B, R * 2);
    sh.C = static_cast<int>(N); sh.R = static_cast<int>(R);
    sh.scale = scale; sh.u = du;
    cudaError_t e = launch_shrink<E, true>(sh, info->tiles, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;

    GradArgs gr = {};
    gr.plan = parts;
    gr.u = u; gr.x = gp; gr.ldx = ldg; gr.ax = ag;
    gr.C = static_cast<int>(N); gr.R = static_cast<int>(R);
    gr.rc = 0; gr.scale = scale; gr.grad = grad_B;
    gr.slots = slots + off_b; gr.slot_stride = stride;
    e = launch_grad(gr, info->parts, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;

    gr.u = du; gr.x = xp; gr.ldx = ldx; gr.ax = ax;
    gr.C = static_cast<int>(K);
    gr.rc = 1; gr.scale = nullptr; gr.grad = grad_A;
    gr.slots = slots;
    e = launch_grad(gr, info->parts, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;

    ExpandArgs ex = {};
    ex.plan = tiles;
    ex.u = du; ex.w = Ap; ex.aw = align_of(A, K * 2);
    ex.C = static_cast<int>(K); ex.R = static_cast<int>(R);
    ex.base = grad_base; ex.ldb = ldgb;
    ex.out = grad_x; ex.ldo = ldgx;
    ex.wide = align_of(grad_x, ldgx * 2) == 16 && (grad_base == nullptr || align_of(grad_base, ldgb * 2) == 16) && K % 8 == 0;
    e = launch_expand<E, true, false>(ex, info->tiles, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;

    PassArgs pa = {};
    pa.n = info->without;
    pa.rows = tiles.rows + (T - pa.n);
    pa.N = static_cast<int>(K); pa.R = static_cast<int>(R);
    pa.base = grad_base; pa.ldb = ldgb;
    pa.out = grad_x == grad_base ? nullptr : grad_x; pa.ldo = ldgx;
    e = launch_pass<E, false>(pa, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;

    if (info->slots > 0) {
        SumArgs su = {};
        su.parts = parts.tiles; su.n = info->slots;
        su.slots = slots; su.slot_stride = stride;
        su.len_a = R * K; su.len_b = R * N; su.off_b = off_b;
        su.grad_a = grad_A; su.grad_b = grad_B;
        const int64_t blocks = (su.len_a + su.len_b + kThreads * 4 - 1) / (kThreads * 4);
        e = launch_pdl(sum_kernel, dim3(static_cast<unsigned>(blocks < 512 ? blocks : 512), static_cast<unsigned>(info->slots)),
                       dim3(kThreads), s, su);
        if (e != cudaSuccess) return BT_ERR_CUDA;
    }
    return BT_OK;
}

}  // extern "C"
