// Rows to microscaled operands and back (see mx.cuh for the format).
//
// Streams: 2 or 4 bytes read for 1/2 or 1 written and 1/32 of scales, or the
// other way round. A thread has eight consecutive values, four lanes a block, so
// that a block's largest magnitude takes two exchanges; a thread's four groups are
// loaded before the first is used.
#include "bt_internal.h"
#include "mx.cuh"

namespace bt {
namespace {

using namespace mx;

constexpr int kThreads = 256;
constexpr int kGroups = 4;                  // groups of eight a thread takes, kThreads apart

struct QuantArgs {
    const void *x;
    int64_t ldx;
    int R, K, al;                           // al: what x's rows start at multiples of
    uint32_t groups;                        // eights of a row, up to the end of its last atom
    FastDiv per_row;
    uint32_t total;
    int64_t atoms;
    uint8_t *q, *s;
};

// (Tiles of 128 rows, whose scales are whole atoms put together in shared memory, take the same time where rows are long and
// twice as long where they are few.)
// WIDE: rows at 16-byte multiples, K a multiple of 8 (as below): a tenth fewer instructions, which bound it beside memory.
template <typename T, int CODE, bool WIDE> __global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const QuantArgs a) {
    pdl_wait();
    pdl_launch_dependents();                // after the wait: what follows may rely on everything before this kernel
    const uint32_t first = blockIdx.x * (kThreads * kGroups) + threadIdx.x;
    uint32_t row[kGroups], g[kGroups];
    Raw8<T> raw[kGroups];
    const T *x = static_cast<const T *>(a.x);
    row[0] = fdiv(first < a.total ? first : 0u, a.per_row);
    g[0] = (first < a.total ? first : 0u) - row[0] * a.groups;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        if (i > 0) {
            row[i] = row[i - 1];
            g[i] = g[i - 1] + kThreads;
            while (g[i] >= a.groups) {      // (once, for rows of 2048 values and more)
                g[i] -= a.groups;
                ++row[i];
            }
        }
        const int k = static_cast<int>(g[i]) * 8;
        const T *p = x + static_cast<int64_t>(row[i]) * a.ldx + k;
        const int valid = first + i * kThreads < a.total ? a.K - k : 0;
        if (!WIDE) raw[i] = raw_load_any<T, false>(p, valid, a.al);
        else raw[i] = valid > 0 ? raw_load<T, false>(p) : Raw8<T>{};
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const uint32_t t = first + i * kThreads, s = scale_of<CODE>(quad_top<T>(raw[i])), word = atom_word(s);
        if (t >= a.total) continue;         // (a row is a multiple of 16 groups)
        float v[8];
        raw_unpack<T>(raw[i], v);
        store8<CODE>(a.q + static_cast<int64_t>(t) * Format<CODE>::kBytes8, code8<CODE>(v, inverse_of(s)));
        if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t *>(a.s + scale_at(row[i], g[i] >> 2, a.atoms)) = word;
    }
}

struct DequantArgs {
    const uint8_t *q, *s;
    int R, K;
    uint32_t groups;                        // eights of a row
    FastDiv per_row;
    uint32_t total;
    int64_t row_bytes, atoms;
    void *out;
    int64_t ldo;
    int al;
};

template <typename T, int CODE, bool WIDE> __global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const DequantArgs a) {
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const uint32_t first = blockIdx.x * (kThreads * kGroups) + threadIdx.x;
    uint2 c[kGroups];
    uint32_t s[kGroups], row[kGroups], g[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const uint32_t t = first + i * kThreads;
        row[i] = fdiv(t < a.total ? t : 0u, a.per_row);
        g[i] = (t < a.total ? t : 0u) - row[i] * a.groups;
        c[i] = load8<CODE>(a.q + static_cast<int64_t>(row[i]) * a.row_bytes + static_cast<int64_t>(g[i]) * Format<CODE>::kBytes8);
        s[i] = a.s[scale_at(row[i], g[i] >> 2, a.atoms)];
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        if (first + i * kThreads >= a.total) continue;
        float v[8];
        value8<CODE>(c[i], v);
        const float p = power_of(s[i]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 x = mul2(make_float2(v[e], v[e + 1]), make_float2(p, p));
            v[e] = x.x;
            v[e + 1] = x.y;
        }
        const int k = static_cast<int>(g[i]) * 8;
        T *o = static_cast<T *>(a.out) + static_cast<int64_t>(row[i]) * a.ldo + k;
        if (WIDE) raw_store<T>(o, raw_pack<T>(v));
        else raw_store_any<T>(o, raw_pack<T>(v), a.K - k, a.al);
    }
}

// fp32 rows of odd alignment or width: a warp 256 neighbours, so that its stores are whole lines (eights a thread store four
// bytes 32 apart: 4093 wide 105 us instead of 38 for 134 MB).
template <int CODE> __global__ void __launch_bounds__(kThreads) mx_dequantize_odd_kernel(const DequantArgs a) {
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const uint32_t t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.total) return;
    const uint32_t row = fdiv(t, a.per_row), k0 = (t - row * a.groups) * 256;
    const uint8_t *q = a.q + static_cast<int64_t>(row) * a.row_bytes;
    float *o = static_cast<float *>(a.out) + static_cast<int64_t>(row) * a.ldo;
    uint32_t c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {           // a block each
        const int k = static_cast<int>(k0) + 32 * i + static_cast<int>(lane);
        c[i] = s[i] = 0u;
        if (k >= a.K) continue;
        c[i] = q[CODE == BT_CODE_E4M3 ? k : k >> 1];
        s[i] = a.s[scale_at(row, k >> 5, a.atoms)];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = static_cast<int>(k0) + 32 * i + static_cast<int>(lane);
        float v[8];
        value8<CODE>(make_uint2(CODE == BT_CODE_E4M3 ? c[i] : c[i] >> (4 * (k & 1)) & 15u, 0u), v);
        if (k < a.K) o[k] = v[0] * power_of(s[i]);
    }
}

// out[k, n] = bf16(value of row n, column k), zeros for R <= n < ld: tiles of 64 x 64 through shared memory.
struct TransposeArgs {
    const uint8_t *q, *s;
    int R, K, ld;
    int64_t row_bytes, atoms;
    __nv_bfloat16 *out;
};
template <int CODE> __global__ void __launch_bounds__(kThreads) mx_transpose_kernel(const TransposeArgs a) {
    __shared__ __nv_bfloat16 tile[64][64 + 2];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int n0 = blockIdx.x * 64, k0 = blockIdx.y * 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {           // 64 rows x 8 groups of eight
        const int j = threadIdx.x + kThreads * i, r = j >> 3, k = k0 + (j & 7) * 8;
        float v[8] = {};
        if (n0 + r < a.R && k < a.K) {      // (a row's codes are zero past K)
            value8<CODE>(load8<CODE>(a.q + static_cast<int64_t>(n0 + r) * a.row_bytes + static_cast<int64_t>(k / 8) * Format<CODE>::kBytes8), v);
            const float p = power_of(a.s[scale_at(n0 + r, k / kBlock, a.atoms)]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= p;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) tile[r][(j & 7) * 8 + e] = __float2bfloat16_rn(v[e]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {           // 64 columns x 32 pairs of rows
        const int j = threadIdx.x + kThreads * i, k = j >> 5, n = (j & 31) * 2;
        if (k0 + k >= a.K || n0 + n >= a.ld) continue;
        __nv_bfloat162 w;
        w.x = tile[n][k];
        w.y = tile[n + 1][k];
        *reinterpret_cast<__nv_bfloat162 *>(a.out + static_cast<int64_t>(k0 + k) * a.ld + n0 + n) = w;
    }
}

bool mx_code(bt_code c) { return c == BT_CODE_E4M3 || c == BT_CODE_E2M1; }
bool float_type(bt_dtype t) { return t == BT_F32 || t == BT_BF16 || t == BT_F16; }
unsigned blocks_of(uint32_t total) { return static_cast<unsigned>((static_cast<uint64_t>(total) + kThreads * kGroups - 1) / (kThreads * kGroups)); }

template <typename T, int CODE> cudaError_t quantize(const QuantArgs &a, cudaStream_t s) {
    return launch_pdl(a.al == 16 && a.K % 8 == 0 ? mx_quantize_kernel<T, CODE, true> : mx_quantize_kernel<T, CODE, false>, dim3(blocks_of(a.total)), dim3(kThreads), s, a);
}
template <typename T, int CODE> cudaError_t dequantize(const DequantArgs &a, cudaStream_t s) {
    return launch_pdl(a.al == 16 && a.K % 8 == 0 ? mx_dequantize_kernel<T, CODE, true> : mx_dequantize_kernel<T, CODE, false>, dim3(blocks_of(a.total)), dim3(kThreads), s, a);
}

// What every call on such an operand checks of it.
bt_status sides(int64_t R, int64_t K, bt_code code) {
    if (!mx_code(code) || R < 0 || K < 1) return BT_ERR_INVALID_ARG;
    if (R >= kMaxSide || K >= kMaxSide || ((R + 127) / 128 * 128) * (k_atoms(K, code) * 16) >= (int64_t(1) << 31)) return BT_ERR_UNSUPPORTED;
    return BT_OK;
}

}  // namespace

bt_status mx_sides(int64_t R, int64_t K, bt_code code) { return sides(R, K, code); }

cudaError_t launch_mx_quantize(const void *x, bt_dtype xt, int64_t ldx, int64_t R, int64_t K, bt_code code, void *q, void *scales,
                               cudaStream_t s) {
    QuantArgs a = {};
    a.x = x; a.ldx = ldx;
    a.R = static_cast<int>(R); a.K = static_cast<int>(K);
    a.atoms = k_atoms(K, code);
    a.groups = static_cast<uint32_t>(a.atoms * 16);
    a.per_row = make_fastdiv(a.groups);
    a.total = static_cast<uint32_t>(R) * a.groups;
    a.q = static_cast<uint8_t *>(q); a.s = static_cast<uint8_t *>(scales);
    a.al = rows_align(static_cast<const char *>(x), ldx, dtype_bytes(xt));
    if (code == BT_CODE_E4M3)
        return xt == BT_F32    ? quantize<float, BT_CODE_E4M3>(a, s)
               : xt == BT_BF16 ? quantize<__nv_bfloat16, BT_CODE_E4M3>(a, s)
                               : quantize<__half, BT_CODE_E4M3>(a, s);
    return xt == BT_F32    ? quantize<float, BT_CODE_E2M1>(a, s)
           : xt == BT_BF16 ? quantize<__nv_bfloat16, BT_CODE_E2M1>(a, s)
                           : quantize<__half, BT_CODE_E2M1>(a, s);
}

}  // namespace bt

using namespace bt;
using namespace bt::mx;

extern "C" {

int64_t bt_mx_row_bytes(int64_t K, bt_code code) { return mx_code(code) && K >= 1 && K < kMaxSide ? code_bytes(K, code) : 0; }

size_t bt_mx_scale_bytes(int64_t R, int64_t K, bt_code code) { return sides(R, K, code) == BT_OK ? scale_bytes(R, K, code) : 0; }

bt_status bt_mx_quantize(const void *x, bt_dtype x_dtype, int64_t ldx, int64_t R, int64_t K, bt_code code, void *out, void *scales,
                         bt_stream stream) {
    if (!float_type(x_dtype)) return BT_ERR_INVALID_ARG;
    const bt_status fit = sides(R, K, code);
    if (fit != BT_OK) return fit;
    if (ldx < K) return BT_ERR_INVALID_ARG;
    if (ldx > (int64_t(1) << 36)) return BT_ERR_UNSUPPORTED;
    if (R == 0) return BT_OK;
    if (x == nullptr || out == nullptr || scales == nullptr) return BT_ERR_INVALID_ARG;
    if (!aligned(x, dtype_bytes(x_dtype)) || !aligned(out, 16) || !aligned(scales, 16)) return BT_ERR_ALIGNMENT;
    return launch_mx_quantize(x, x_dtype, ldx, R, K, code, out, scales, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? BT_OK
               : BT_ERR_CUDA;
}

bt_status bt_mx_dequantize(const void *q, const void *scales, int64_t R, int64_t K, bt_code code, void *out, bt_dtype out_dtype,
                           int64_t ldo, bt_stream stream) {
    if (!float_type(out_dtype)) return BT_ERR_INVALID_ARG;
    const bt_status fit = sides(R, K, code);
    if (fit != BT_OK) return fit;
    if (ldo < K) return BT_ERR_INVALID_ARG;
    if (ldo > (int64_t(1) << 36)) return BT_ERR_UNSUPPORTED;
    if (R == 0) return BT_OK;
    if (q == nullptr || out == nullptr || scales == nullptr) return BT_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(scales, 16) || !aligned(out, dtype_bytes(out_dtype))) return BT_ERR_ALIGNMENT;
    DequantArgs a = {};
    a.q = static_cast<const uint8_t *>(q); a.s = static_cast<const uint8_t *>(scales);
    a.R = static_cast<int>(R); a.K = static_cast<int>(K);
    a.atoms = k_atoms(K, code);
    a.groups = static_cast<uint32_t>((K + 7) / 8);
    a.per_row = make_fastdiv(a.groups);
    a.total = static_cast<uint32_t>(R) * a.groups;
    a.row_bytes = code_bytes(K, code);
    a.out = out; a.ldo = ldo;
    a.al = rows_align(static_cast<const char *>(out), ldo, dtype_bytes(out_dtype));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (out_dtype == BT_F32 && !(a.al == 16 && a.K % 8 == 0)) {
        a.groups = static_cast<uint32_t>((K + 255) / 256);
        a.per_row = make_fastdiv(a.groups);
        a.total = static_cast<uint32_t>(R) * a.groups;
        const dim3 grid((a.total + kThreads / 32 - 1) / (kThreads / 32));
        e = code == BT_CODE_E4M3 ? launch_pdl(mx_dequantize_odd_kernel<BT_CODE_E4M3>, grid, dim3(kThreads), s, a)
                                 : launch_pdl(mx_dequantize_odd_kernel<BT_CODE_E2M1>, grid, dim3(kThreads), s, a);
    } else if (code == BT_CODE_E4M3)
        e = out_dtype == BT_F32    ? dequantize<float, BT_CODE_E4M3>(a, s)
            : out_dtype == BT_BF16 ? dequantize<__nv_bfloat16, BT_CODE_E4M3>(a, s)
                                   : dequantize<__half, BT_CODE_E4M3>(a, s);
    else
        e = out_dtype == BT_F32    ? dequantize<float, BT_CODE_E2M1>(a, s)
            : out_dtype == BT_BF16 ? dequantize<__nv_bfloat16, BT_CODE_E2M1>(a, s)
                                   : dequantize<__half, BT_CODE_E2M1>(a, s);
    return e == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

bt_status bt_mx_transpose(const void *q, const void *scales, int64_t R, int64_t K, bt_code code, int64_t ld, void *out,
                          bt_stream stream) {
    const bt_status fit = sides(R, K, code);
    if (fit != BT_OK) return fit;
    if (ld < R || ld % 8 != 0) return BT_ERR_INVALID_ARG;
    if (ld >= kMaxSide || K > int64_t(65535) * 64) return BT_ERR_UNSUPPORTED;
    if (ld == 0) return BT_OK;
    if (out == nullptr || (R > 0 && (q == nullptr || scales == nullptr))) return BT_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(scales, 16) || !aligned(out, 16)) return BT_ERR_ALIGNMENT;
    TransposeArgs a = {};
    a.q = static_cast<const uint8_t *>(q); a.s = static_cast<const uint8_t *>(scales);
    a.R = static_cast<int>(R); a.K = static_cast<int>(K); a.ld = static_cast<int>(ld);
    a.row_bytes = code_bytes(K, code);
    a.atoms = k_atoms(K, code);
    a.out = static_cast<__nv_bfloat16 *>(out);
    const dim3 grid(static_cast<unsigned>((ld + 63) / 64), static_cast<unsigned>((K + 63) / 64));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = code == BT_CODE_E4M3 ? launch_pdl(mx_transpose_kernel<BT_CODE_E4M3>, grid, dim3(kThreads), s, a)
                                               : launch_pdl(mx_transpose_kernel<BT_CODE_E2M1>, grid, dim3(kThreads), s, a);
    return e == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

}  // extern "C"
