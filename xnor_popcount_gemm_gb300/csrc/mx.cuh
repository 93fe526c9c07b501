// Microscaled operands (OCP MX): 32 consecutive values of a row share a power of
// two 2^(s - 127), s one byte, and are E4M3 (8 bits) or E2M1 (4 bits) values of it.
//   s     = max(exponent of the block's largest magnitude - the format's largest exponent + 127, 0)
//   value = x / 2^(s - 127) rounded to nearest, ties to even, beyond the largest value to that
// x / 2^(s - 127) is exact but for values below 2^-126, far below half a step, so
// the codes do not depend on who computes them. A NaN or infinity among the 32
// makes s = 255, the NaN of these scales, and the block NaN.
//
// Codes: rows of a multiple of 128 bytes (128 E4M3 or 256 E2M1 values), zero past
// K; E2M1: element 2i in the low nibble of byte i. Scales: what the tensor cores take. An atom of
// 512 bytes holds 128 rows x 4 blocks: row r's block b at (r % 32) * 16 +
// (r / 32) * 4 + b, which one tcgen05.cp brings to 32 lanes x 4 columns of TMEM.
// Atoms lie in row order of [rows / 128, blocks / 4], a whole number of them (1 or 2) for 128 bytes of codes.
#pragma once

#include <type_traits>

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "bt_device.cuh"
#include "mx_layout.h"

namespace bt {
namespace mx {

template <int CODE> struct Format;
template <> struct Format<BT_CODE_E4M3> {
    static constexpr int kMaxExp = 8;          // 448 = 1.75 * 2^8
    static constexpr int kBytes8 = 8;          // bytes of eight codes
};
template <> struct Format<BT_CODE_E2M1> {
    static constexpr int kMaxExp = 2;          // 6 = 1.5 * 2^2
    static constexpr int kBytes8 = 4;
};

// Bits of |v|: their order is that of the magnitudes, infinity and then NaN last.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kNanScale = 255u;

// The scale byte of a block whose largest magnitude has the bits `top`.
template <int CODE> __device__ __forceinline__ uint32_t scale_of(uint32_t top) {
    if (top >= kInfBits) return kNanScale;
    const int e = static_cast<int>(top >> 23) - Format<CODE>::kMaxExp;
    return static_cast<uint32_t>(e > 0 ? e : 0);
}
// 2^(127 - s), what values are multiplied by; 0 for the NaN scale (codes 0 then).
__device__ __forceinline__ float inverse_of(uint32_t s) {
    return s == kNanScale ? 0.0f : __uint_as_float((254u - s) << 23);
}
// 2^(s - 127).
__device__ __forceinline__ float power_of(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == kNanScale ? 0x7FFFFFFFu : s << 23);
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 x, y, r;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 r, x, y;\nmov.b64 {%0, %1}, r;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 x, y, r;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmul.rn.f32x2 r, x, y;\nmov.b64 {%0, %1}, r;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 x, y, z, r;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\nfma.rn.f32x2 r, x, y, z;\n"
        "mov.b64 {%0, %1}, r;\n}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

// Two codes: lo in the low byte (nibble).
template <int CODE> __device__ __forceinline__ uint32_t code2(float lo, float hi) {
    if constexpr (CODE == BT_CODE_E4M3)
        return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
    else
        return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}
// Eight codes of v * inv; zeros where inv is 0 (a NaN block).
template <int CODE> __device__ __forceinline__ uint2 code8(const float (&v)[8], float inv) {
    if (inv == 0.0f) return make_uint2(0u, 0u);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = mul2(make_float2(v[2 * i], v[2 * i + 1]), make_float2(inv, inv));
        c[i] = code2<CODE>(q.x, q.y);
    }
    if constexpr (CODE == BT_CODE_E4M3) return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    else return make_uint2(c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24), 0u);
}
template <int CODE> __device__ __forceinline__ void store8(uint8_t *p, const uint2 &c) {
    if constexpr (CODE == BT_CODE_E4M3) *reinterpret_cast<uint2 *>(p) = c;
    else *reinterpret_cast<uint32_t *>(p) = c.x;
}
// The values of eight codes.
template <int CODE> __device__ __forceinline__ void value8(const uint2 &c, float (&v)[8]) {
    if constexpr (CODE == BT_CODE_E4M3) {
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c.x >> (8 * i)), __NV_E2M1);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <int CODE> __device__ __forceinline__ uint2 load8(const uint8_t *p) {
    if constexpr (CODE == BT_CODE_E4M3) return *reinterpret_cast<const uint2 *>(p);
    else return make_uint2(*reinterpret_cast<const uint32_t *>(p), 0u);
}

// fp32 to an element type, rounded to nearest.
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Eight consecutive elements as 16 or 32 bytes.
template <typename T> struct Raw8;
template <> struct Raw8<float> { uint4 a, b; };
template <> struct Raw8<__nv_bfloat16> { uint4 a; };
template <> struct Raw8<__half> { uint4 a; };
// FIXED: nothing writes there from before the kernel's start to its end (a load through the read-only path). Operands that are
// written in place, or by the kernel before, which may still be running when this one starts, may not take it.
template <bool FIXED, typename V> __device__ __forceinline__ V load_as(const V *p) {
    if constexpr (FIXED) return __ldg(p);
    else return *p;
}
template <typename T, bool FIXED = true> __device__ __forceinline__ Raw8<T> raw_load(const T *p) {
    Raw8<T> r;
    r.a = load_as<FIXED>(reinterpret_cast<const uint4 *>(p));
    if constexpr (sizeof(T) == 4) r.b = load_as<FIXED>(reinterpret_cast<const uint4 *>(p) + 1);
    return r;
}
template <typename T> __device__ __forceinline__ void raw_unpack(const Raw8<T> &r, float (&v)[8]) {
    Elem<T>::unpack(r.a, v);
    if constexpr (sizeof(T) == 4) Elem<T>::unpack(r.b, v + 4);
}
template <typename T> __device__ __forceinline__ Raw8<T> raw_pack(const float (&v)[8]) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return r;
}
template <typename T> __device__ __forceinline__ void raw_store(T *p, const Raw8<T> &r) {
    *reinterpret_cast<uint4 *>(p) = r.a;
    if constexpr (sizeof(T) == 4) *(reinterpret_cast<uint4 *>(p) + 1) = r.b;
}
// The same at any element address: `valid` of them are there (<= 0: none), the rest zeros. al: what p is a multiple of
// (16, 8, 4 or 2; smaller than 16 goes by the widest loads that it allows).
template <typename T, bool FIXED = true> __device__ __forceinline__ Raw8<T> raw_load_any(const T *p, int valid, int al) {
    if (valid <= 0) return Raw8<T>{};       // (p may lie anywhere then)
    if (al == 16 && valid >= 8) return raw_load<T, FIXED>(p);
    uint32_t w[sizeof(T) * 2] = {};
    if (valid >= 8 && al == 8) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) {
            const uint2 v = load_as<FIXED>(reinterpret_cast<const uint2 *>(p) + i);
            w[2 * i] = v.x;
            w[2 * i + 1] = v.y;
        }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) w[i] = __float_as_uint(load_as<FIXED>(p + i));
    } else {
        // from the aligned words that hold a valid one
        const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 2) >> 1;
        const uint32_t *q = reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint16_t *>(p) - odd);
        uint32_t r[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) r[i] = 2 * i - odd < valid && (i < 4 || odd) ? load_as<FIXED>(q + i) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = odd ? __funnelshift_r(r[i], r[i + 1], 16) : r[i];
            w[i] = valid - 2 * i >= 2 ? v : valid - 2 * i == 1 ? v & 0xFFFFu : 0u;
        }
    }
    Raw8<T> r;
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (sizeof(T) == 4) r.b = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}
template <typename T> __device__ __forceinline__ void raw_store_any(T *p, const Raw8<T> &r, int valid, int al) {
    if (al == 16 && valid >= 8) return raw_store<T>(p, r);
    uint32_t w[sizeof(T) * 2];
    w[0] = r.a.x; w[1] = r.a.y; w[2] = r.a.z; w[3] = r.a.w;
    if constexpr (sizeof(T) == 4) { w[4] = r.b.x; w[5] = r.b.y; w[6] = r.b.z; w[7] = r.b.w; }
    if (valid >= 8 && al == 8) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) reinterpret_cast<uint2 *>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < valid) p[i] = __uint_as_float(w[i]);
    } else {
        uint16_t *h = reinterpret_cast<uint16_t *>(p);
        if (valid >= 8) {
            if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
            } else {
                h[0] = static_cast<uint16_t>(w[0]);
#pragma unroll
                for (int i = 0; i < 3; ++i) reinterpret_cast<uint32_t *>(h + 1)[i] = __funnelshift_r(w[i], w[i + 1], 16);
                h[7] = static_cast<uint16_t>(w[3] >> 16);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < valid) h[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}
// The largest of 16, 8, 4, 2 bytes that p and every multiple of ld elements share.
template <typename T> inline int rows_align(const T *p, int64_t ld, int elem) {
    const uintptr_t v = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * elem);
    return v % 16 == 0 ? 16 : v % 8 == 0 ? 8 : v % 4 == 0 ? 4 : 2;
}

// Four lanes next to one another hold a block: the bits of its largest magnitude as fp32, in all of them. 16-bit values go
// two by two (the order of their bits is that of their magnitudes too).
template <typename T> __device__ __forceinline__ uint32_t quad_top(const Raw8<T> &r) {
    if constexpr (sizeof(T) == 4) {
        const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, w[e] & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    } else {
        constexpr uint32_t kMag = 0x7FFF7FFFu;
        uint32_t m = __vmaxu2(__vmaxu2(r.a.x & kMag, r.a.y & kMag), __vmaxu2(r.a.z & kMag, r.a.w & kMag));
        m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        m = max(m & 0xFFFFu, m >> 16);
        if constexpr (std::is_same<T, __half>::value) {
            const uint16_t h = static_cast<uint16_t>(m);
            return __float_as_uint(__half2float(*reinterpret_cast<const __half *>(&h)));
        }
        return m << 16;
    }
}
// Sixteen lanes hold an atom's four blocks of a row, quad by quad: their scale bytes as one word, in the first of them.
__device__ __forceinline__ uint32_t atom_word(uint32_t s) {
    s |= __shfl_down_sync(0xFFFFFFFFu, s, 4) << 8;
    return s | (__shfl_down_sync(0xFFFFFFFFu, s, 8) << 16);
}

}  // namespace mx
}  // namespace bt
