// Root-mean-square norm before a projection, with the residual's addition, its
// result in the input's type and / or as a microscaled operand, and its backward.
//
//   h = T(x + r)      y = T(f32(h w / sqrt(mean h^2 + eps)))      codes = mx(y)
//   n = h / sqrt(mean h^2 + eps)      gx = (g w - n mean(g w n)) / sqrt(..) + gs
//   gw = sum over the rows of g n
//
// Streams: every row is read once, kept in registers by its CTA and written once.
//
// What is rounded to 8 or 4 bits falls one way or the other, so y is the correctly
// rounded fp32 value (but for about one in 2^24): the squares are summed with the
// rounding errors of the sums beside them, and 1 / sqrt(mean) is a pair of floats,
// the second from one Newton step on the residual 1 - m q^2, which an fma gives
// exactly. That is 13 operations a value where a plain norm has 4.
#include <cmath>
#include <cstdlib>

#include "bt_internal.h"
#include "mx.cuh"

namespace bt {
namespace {

using namespace mx;

constexpr int kNoCode = -1;

struct NormArgs {
    const void *x, *r, *w;                  // r, w: NULL where there is none
    int64_t ldx, ldr;
    int w_f32;
    int T, N;
    float n_inv, n_inv_lo, eps, eps_lo;     // 1 / N and eps as pairs
    void *sum, *out;                        // NULL: not wanted
    int64_t lds, ldo;
    int code;                               // kNoCode, or a bt_code
    uint8_t *q, *s;
    int64_t row_bytes, atoms;
    int cols;                               // N, or the columns up to the end of the last atom
};

// A sum and the rounding errors made in it.
struct Sum2 {
    float s, c;
    __device__ __forceinline__ void add(float p) {
        const float t = s + p, b = t - s;
        c += (s - (t - b)) + (p - b);
        s = t;
    }
    __device__ __forceinline__ void join(float os, float oc) {
        add(os);
        c += oc;
    }
};

// The block's sum, in every thread, in an order that the thread count alone decides.
__device__ __forceinline__ Sum2 block_sum(Sum2 v, float2 (&red)[32]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float s = __shfl_xor_sync(0xFFFFFFFFu, v.s, o), c = __shfl_xor_sync(0xFFFFFFFFu, v.c, o);
        v.join(s, c);
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(v.s, v.c);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float2 p = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
    v.s = p.x;
    v.c = p.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float s = __shfl_xor_sync(0xFFFFFFFFu, v.s, o), c = __shfl_xor_sync(0xFFFFFFFFu, v.c, o);
        v.join(s, c);
    }
    return v;
}

// Rows whose squares leave fp32 are summed again, their values times this power of two.
__device__ __forceinline__ float power_for(float s, const float eps, int N) {
    if (!(s <= 3.4e38f)) return 0x1p-80f;
    if (fmaf(eps, static_cast<float>(N), s) < 0x1p-80f) return 0x1p100f;
    return 1.0f;
}

// 1 / sqrt(mean + eps) for values times k, as hi + lo.
struct Inverse {
    float hi, lo;
};
__device__ __forceinline__ Inverse inverse_rms(const Sum2 &v, const NormArgs &a, float k) {
    if (!(v.s <= 3.4e38f)) return Inverse{rsqrtf(v.s), 0.0f};       // infinity: 0, NaN: NaN
    const float p = v.s * a.n_inv;
    float lo = fmaf(v.s, a.n_inv, -p) + fmaf(v.s, a.n_inv_lo, v.c * a.n_inv);
    const float eh = (a.eps * k) * k, el = (a.eps_lo * k) * k;
    const float t = p + eh, b = t - p;
    lo += (p - (t - b)) + (eh - b) + el;
    const float m = t + lo, ml = lo - (m - t);
    const float r = rsqrtf(m), q = r * r;
    // 1 - m r^2 in the exact r^2 = q + (r^2 - q)
    const float e = fmaf(-m, q, 1.0f) - fmaf(m, fmaf(r, r, -q), ml * q);
    return Inverse{r, r * (0.5f * e + 0.375f * e * e)};
}
__device__ __forceinline__ float normed(float v, float w, const Inverse &i) {
    const float p = v * w;
    return fmaf(p, i.hi, fmaf(p, i.lo, fmaf(v, w, -p) * i.hi));
}

// A row by its CTA, eight consecutive columns at a time: thread t has the eights
// t, t + threads, ... (V of them). Rows 16-byte aligned, N a multiple of 8.
template <typename T, int V>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormArgs a) {
    __shared__ float2 red[2][32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const T *r = static_cast<const T *>(a.r) + row * a.ldr;
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    Raw8<T> h[V], rr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        h[i] = Raw8<T>{};
        if (c >= a.N) continue;
        h[i] = raw_load<T>(x + c);
        if (a.r != nullptr) rr[i] = raw_load<T>(r + c);
    }
    if (a.r != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
            if (c >= a.N) continue;
            float v[8], o[8];
            raw_unpack<T>(h[i], v);
            raw_unpack<T>(rr[i], o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
            h[i] = raw_pack<T>(v);
            if (a.sum != nullptr) raw_store<T>(static_cast<T *>(a.sum) + row * a.lds + c, h[i]);
        }
    }
    auto squares = [&](float k) {
        Sum2 p{0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v[8];
            raw_unpack<T>(h[i], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = v[e] * k, sq = u * u;
                p.add(sq);
                if (sizeof(T) == 4) p.c += fmaf(u, u, -sq);      // (16-bit values have exact squares)
            }
        }
        return p;
    };
    Sum2 total = block_sum(squares(1.0f), red[0]);
    const float k = power_for(total.s, a.eps, a.N);
    if (k != 1.0f) total = block_sum(squares(k), red[1]);
    const Inverse inv = inverse_rms(total, a, k);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int g = threadIdx.x + i * blockDim.x, c = g * 8;
        if (c - static_cast<int>(threadIdx.x & 31) * 8 >= a.cols) continue;      // (whole warps)
        float y[8] = {};
        if (c < a.N) {
            float v[8], w[8];
            raw_unpack<T>(h[i], v);
            if (a.w == nullptr) {
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 1.0f;
            } else if (a.w_f32) {
                raw_unpack<float>(raw_load<float>(static_cast<const float *>(a.w) + c), w);
            } else {
                raw_unpack<T>(raw_load<T>(static_cast<const T *>(a.w) + c), w);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = normed(v[e] * k, w[e], inv);
            const Raw8<T> o = raw_pack<T>(y);
            if (a.out != nullptr) raw_store<T>(static_cast<T *>(a.out) + row * a.ldo + c, o);
            raw_unpack<T>(o, y);
        }
        if (a.code == kNoCode) continue;
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = mag_bits(y[e]);
            top = m > top ? m : top;
        }
        top = quad_max(top);
        if (c >= a.cols) continue;
        const bool e4m3 = a.code == BT_CODE_E4M3;
        const uint32_t s = e4m3 ? scale_of<BT_CODE_E4M3>(top) : scale_of<BT_CODE_E2M1>(top);
        const int64_t at = static_cast<int64_t>(g) * (e4m3 ? 8 : 4);
        uint8_t *p = a.q + row * a.row_bytes + at;
        if (e4m3) store8<BT_CODE_E4M3>(p, code8<BT_CODE_E4M3>(y, inverse_of(s)));
        else store8<BT_CODE_E2M1>(p, code8<BT_CODE_E2M1>(y, inverse_of(s)));
        if ((threadIdx.x & 3) == 0) a.s[scale_at(row, g >> 2, a.atoms)] = static_cast<uint8_t>(s);
    }
}

// Rows of any alignment and width: thread t has the columns t, t + threads, ..., a
// warp's 32 columns being a block. The first E of a thread's values stay in
// registers; what is beyond (wider rows than 1024 E) is read a second time.
template <typename T, int E>
__global__ void __launch_bounds__(1024) rms_norm_any_kernel(const NormArgs a) {
    __shared__ float2 red[2][32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.ldx;
    const T *r = static_cast<const T *>(a.r) + row * a.ldr;
    T *sum = static_cast<T *>(a.sum) + row * a.lds;
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int step = blockDim.x;
    auto load = [&](int c, bool keep) {
        if (c >= a.N) return 0.0f;
        float v = Elem<T>::to_f32(x[c]);
        if (a.r != nullptr) {
            const T t = from_f32<T>(v + Elem<T>::to_f32(r[c]));
            if (keep && a.sum != nullptr) sum[c] = t;
            v = Elem<T>::to_f32(t);
        }
        return v;
    };
    // a value that was loaded before: where sum is written it may be x or r, and holds h
    auto again = [&](int c) {
        if (c >= a.N) return 0.0f;
        return a.r != nullptr && a.sum != nullptr ? Elem<T>::to_f32(sum[c]) : load(c, false);
    };
    float h[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = threadIdx.x + i * step;
        h[i] = c < a.N ? Elem<T>::to_f32(x[c]) : 0.0f;
    }
    if (a.r != nullptr) {
        T rr[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = threadIdx.x + i * step;
            rr[i] = c < a.N ? r[c] : from_f32<T>(0.0f);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = threadIdx.x + i * step;
            const T t = from_f32<T>(h[i] + Elem<T>::to_f32(rr[i]));
            if (c < a.N && a.sum != nullptr) sum[c] = t;
            h[i] = Elem<T>::to_f32(t);
        }
    }
    auto add = [&](Sum2 &p, float v, float k) {
        const float u = v * k, sq = u * u;
        p.add(sq);
        if (sizeof(T) == 4) p.c += fmaf(u, u, -sq);
    };
    auto squares = [&](float k, bool first) {
        Sum2 p{0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < E; ++i) add(p, h[i], k);
        for (int c = threadIdx.x + E * step; c < a.N; c += step) add(p, first ? load(c, true) : again(c), k);
        return p;
    };
    Sum2 total = block_sum(squares(1.0f, true), red[0]);
    const float k = power_for(total.s, a.eps, a.N);
    if (k != 1.0f) total = block_sum(squares(k, false), red[1]);
    const Inverse inv = inverse_rms(total, a, k);
    auto finish = [&](int c, float v) {
        float y = 0.0f;
        if (c < a.N) {
            const float w = a.w == nullptr ? 1.0f
                            : a.w_f32      ? __ldg(static_cast<const float *>(a.w) + c)
                                           : Elem<T>::to_f32(static_cast<const T *>(a.w)[c]);
            const T o = from_f32<T>(normed(v * k, w, inv));
            if (a.out != nullptr) static_cast<T *>(a.out)[row * a.ldo + c] = o;
            y = Elem<T>::to_f32(o);
        }
        if (a.code == kNoCode) return;
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, mag_bits(y));
        const bool e4m3 = a.code == BT_CODE_E4M3;
        const uint32_t s = e4m3 ? scale_of<BT_CODE_E4M3>(top) : scale_of<BT_CODE_E2M1>(top);
        const float f = inverse_of(s);
        if (e4m3) {
            a.q[row * a.row_bytes + c] = f == 0.0f ? 0 : static_cast<uint8_t>(code2<BT_CODE_E4M3>(y * f, 0.0f));
        } else {
            const float o = __shfl_down_sync(0xFFFFFFFFu, y, 1);
            if ((threadIdx.x & 1) == 0)
                a.q[row * a.row_bytes + c / 2] = f == 0.0f ? 0 : static_cast<uint8_t>(code2<BT_CODE_E2M1>(y * f, o * f));
        }
        if ((threadIdx.x & 31) == 0) a.s[scale_at(row, c >> 5, a.atoms)] = static_cast<uint8_t>(s);
    };
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = threadIdx.x + i * step;
        if (c - static_cast<int>(threadIdx.x & 31) < a.cols) finish(c, h[i]);       // (whole warps)
    }
    for (int c = threadIdx.x + E * step; c - static_cast<int>(threadIdx.x & 31) < a.cols; c += step) finish(c, again(c));
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
struct BackArgs {
    const void *g, *h, *w, *gs;             // w, gs: NULL where there is none
    int64_t ldg, ldh, ldgs, ldgx;
    int w_f32;
    int T, N;
    float n_inv, eps;
    void *gx;
    float *parts;                           // [chunks, N], NULL: gw not wanted
    float4 *rows;                           // (any) 1 / rms of the values times k, mean(g w n), k of every row
    int chunks;
};

__device__ __forceinline__ float2 block_pair(float2 v, float2 (&red)[32]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
    }
    return v;
}
__device__ __forceinline__ float inverse_plain(float s, const BackArgs &a, float k) {
    return 1.0f / sqrtf(fmaf(s, a.n_inv, (a.eps * k) * k));
}

template <typename T> __device__ __forceinline__ void weight8(const void *w, int w_f32, int c, float (&o)[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 1.0f;
    } else if (w_f32) {
        raw_unpack<float>(raw_load<float>(static_cast<const float *>(w) + c), o);
    } else {
        raw_unpack<T>(raw_load<T>(static_cast<const T *>(w) + c), o);
    }
}

// Aligned rows: a CTA takes rows blockIdx.x, + chunks, ... and keeps its threads'
// columns of gw in registers; the next row's g and h are on their way meanwhile.
template <typename T, int V>
__global__ void __launch_bounds__(512) rms_back_kernel(const BackArgs a) {
    __shared__ float2 red[4][32];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
    Raw8<T> g[V], h[V], gn[V], hn[V];
    auto fetch = [&](int row, Raw8<T> (&pg)[V], Raw8<T> (&ph)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
            pg[i] = ph[i] = Raw8<T>{};
            if (c < a.N && row < a.T) {
                pg[i] = raw_load<T>(static_cast<const T *>(a.g) + row * a.ldg + c);
                ph[i] = raw_load<T>(static_cast<const T *>(a.h) + row * a.ldh + c);
            }
        }
    };
    fetch(blockIdx.x, g, h);
    int odd = 0;
    for (int row = blockIdx.x; row < a.T; row += gridDim.x, odd ^= 1) {
        fetch(row + gridDim.x, gn, hn);
        Raw8<T> gs[V];
        if (a.gs != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (threadIdx.x + i * blockDim.x) * 8;
                if (c < a.N) gs[i] = raw_load<T>(static_cast<const T *>(a.gs) + row * a.ldgs + c);
            }
        }
        auto sums = [&](float k) {
            float2 p = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (threadIdx.x + i * blockDim.x) * 8;
                if (c >= a.N) continue;
                float vg[8], vh[8], w[8];
                raw_unpack<T>(g[i], vg);
                raw_unpack<T>(h[i], vh);
                weight8<T>(a.w, a.w_f32, c, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = vh[e] * k;
                    p.x = fmaf(u, u, p.x);
                    p.y = fmaf(vg[e] * w[e], u, p.y);
                }
            }
            return p;
        };
        float2 p = block_pair(sums(1.0f), red[odd]);
        const float k = power_for(p.x, a.eps, a.N);
        if (k != 1.0f) p = block_pair(sums(k), red[2 + odd]);
        const float inv = inverse_plain(p.x, a, k), mean = p.y * inv * a.n_inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (threadIdx.x + i * blockDim.x) * 8;
            if (c >= a.N) continue;
            float vg[8], vh[8], w[8], o[8];
            raw_unpack<T>(g[i], vg);
            raw_unpack<T>(h[i], vh);
            weight8<T>(a.w, a.w_f32, c, w);
            if (a.gs != nullptr) raw_unpack<T>(gs[i], o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = vh[e] * k * inv;
                acc[i][e] = fmaf(vg[e], n, acc[i][e]);
                const float d = (inv * k) * fmaf(-n, mean, vg[e] * w[e]);
                o[e] = a.gs != nullptr ? d + o[e] : d;
            }
            raw_store<T>(static_cast<T *>(a.gx) + row * a.ldgx + c, raw_pack<T>(o));
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            g[i] = gn[i];
            h[i] = hn[i];
        }
    }
    if (a.parts == nullptr) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * 8;
        if (c < a.N) {
            float *p = a.parts + static_cast<int64_t>(blockIdx.x) * a.N + c;
            raw_store<float>(p, raw_pack<float>(acc[i]));
        }
    }
}

// Rows of any alignment and width: the rows' sums, then strips of columns.
template <typename T> __device__ __forceinline__ float weight1(const BackArgs &a, int c) {
    return a.w == nullptr ? 1.0f : a.w_f32 ? __ldg(static_cast<const float *>(a.w) + c) : Elem<T>::to_f32(static_cast<const T *>(a.w)[c]);
}
template <typename T> __global__ void __launch_bounds__(512) rms_back_rows_kernel(const BackArgs a) {
    __shared__ float2 red[2][32];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T *g = static_cast<const T *>(a.g) + row * a.ldg, *h = static_cast<const T *>(a.h) + row * a.ldh;
    auto sums = [&](float k) {
        float2 p = make_float2(0.0f, 0.0f);
#pragma unroll 4
        for (int c = threadIdx.x; c < a.N; c += blockDim.x) {
            const float u = Elem<T>::to_f32(h[c]) * k;
            p.x = fmaf(u, u, p.x);
            p.y = fmaf(Elem<T>::to_f32(g[c]) * weight1<T>(a, c), u, p.y);
        }
        return p;
    };
    float2 p = block_pair(sums(1.0f), red[0]);
    const float k = power_for(p.x, a.eps, a.N);
    if (k != 1.0f) p = block_pair(sums(k), red[1]);
    const float inv = inverse_plain(p.x, a, k);
    if (threadIdx.x == 0) a.rows[row] = make_float4(inv, p.y * inv * a.n_inv, k, 0.0f);
}
constexpr int kStrip = 128;
template <typename T> __global__ void __launch_bounds__(kStrip) rms_back_strips_kernel(const BackArgs a) {
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int c = blockIdx.x * kStrip + threadIdx.x;
    if (c >= a.N) return;
    const float w = weight1<T>(a, c);
    float acc = 0.0f;
#pragma unroll 4
    for (int row = blockIdx.y; row < a.T; row += a.chunks) {
        const float4 s = __ldg(a.rows + row);
        const float vg = Elem<T>::to_f32(static_cast<const T *>(a.g)[row * a.ldg + c]);
        const float n = Elem<T>::to_f32(static_cast<const T *>(a.h)[row * a.ldh + c]) * s.z * s.x;
        acc = fmaf(vg, n, acc);
        float d = (s.x * s.z) * fmaf(-n, s.y, vg * w);
        if (a.gs != nullptr) d += Elem<T>::to_f32(static_cast<const T *>(a.gs)[row * a.ldgs + c]);
        static_cast<T *>(a.gx)[row * a.ldgx + c] = from_f32<T>(d);
    }
    if (a.parts != nullptr) a.parts[static_cast<int64_t>(blockIdx.y) * a.N + c] = acc;
}

// gw = the parts' sum: 32 columns a CTA, 32 rows of parts at a time.
__global__ void __launch_bounds__(1024) rms_back_join_kernel(const float *parts, int chunks, int N, float *gw) {
    __shared__ float red[32][33];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < N)
        for (int i = warp; i < chunks; i += 32) v += parts[static_cast<int64_t>(i) * N + c];
    red[warp][lane] = v;
    __syncthreads();
    v = red[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0 && blockIdx.x * 32 + warp < N) gw[blockIdx.x * 32 + warp] = v;
}

bool float_type(bt_dtype t) { return t == BT_F32 || t == BT_BF16 || t == BT_F16; }
bool wide_rows(const void *p, int64_t ld, bt_dtype t) { return p == nullptr || (aligned(p, 16) && (ld * dtype_bytes(t)) % 16 == 0); }
unsigned whole_warps(int64_t n) { return static_cast<unsigned>((n + 31) / 32 * 32); }

template <typename T> cudaError_t norm(const NormArgs &a, bool vec, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.T));
    if (vec) {
        const int64_t groups = (a.cols + 7) / 8;
        // few rows: as many threads as there are loads; many: two loads a thread in flight
        const int v = groups > 2048 ? 4 : groups > 1024 || a.T > 2 * device_sm_count() ? 2 : 1;
        const dim3 block(whole_warps((groups + v - 1) / v));
        if (v == 1) return launch_pdl(rms_norm_kernel<T, 1>, grid, block, s, a);
        if (v == 2) return launch_pdl(rms_norm_kernel<T, 2>, grid, block, s, a);
        return launch_pdl(rms_norm_kernel<T, 4>, grid, block, s, a);
    }
    if (a.cols <= 8192) return launch_pdl(rms_norm_any_kernel<T, 8>, grid, dim3(whole_warps((a.cols + 7) / 8)), s, a);
    return launch_pdl(rms_norm_any_kernel<T, 16>, grid, dim3(a.cols < 16384 ? whole_warps((a.cols + 15) / 16) : 1024), s, a);
}

constexpr int kBackMost = 512 * 8 * 4;      // the widest row that rms_back_kernel takes

int back_chunks(int64_t T, int64_t N, bool vec) {
    const int64_t sms = device_sm_count();
    int64_t n = vec ? 2 * sms : (8 * sms + (N + kStrip - 1) / kStrip - 1) / ((N + kStrip - 1) / kStrip);
    if (n > T) n = T;
    return static_cast<int>(n < 1 ? 1 : n);
}

template <typename T> cudaError_t backward(BackArgs a, bool vec, cudaStream_t s) {
    a.chunks = back_chunks(a.T, a.N, vec);
    if (vec) {
        const int64_t groups = a.N / 8;
        const int v = groups > 1024 ? 4 : groups > 256 ? 2 : 1;
        const dim3 grid(static_cast<unsigned>(a.chunks)), block(whole_warps((groups + v - 1) / v));
        if (v == 1) return launch_pdl(rms_back_kernel<T, 1>, grid, block, s, a);
        if (v == 2) return launch_pdl(rms_back_kernel<T, 2>, grid, block, s, a);
        return launch_pdl(rms_back_kernel<T, 4>, grid, block, s, a);
    }
    const cudaError_t e = launch_pdl(rms_back_rows_kernel<T>, dim3(static_cast<unsigned>(a.T)), dim3(512), s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(rms_back_strips_kernel<T>,
                      dim3(static_cast<unsigned>((a.N + kStrip - 1) / kStrip), static_cast<unsigned>(a.chunks)), dim3(kStrip), s, a);
}

}  // namespace
}  // namespace bt

using namespace bt;
using namespace bt::mx;

extern "C" {

bt_status bt_rms_norm(const void *x, bt_dtype dtype, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                      bt_dtype weight_dtype, int64_t T, int64_t N, double eps, void *sum, int64_t lds, void *out, int64_t ldo,
                      bt_code code, void *q, void *scales, bt_stream stream) {
    if (!float_type(dtype) || (weight != nullptr && weight_dtype != BT_F32 && weight_dtype != dtype)) return BT_ERR_INVALID_ARG;
    if (T < 0 || N < 1 || !std::isfinite(eps) || eps < 0.0 || eps > 1e30) return BT_ERR_INVALID_ARG;
    if (q != nullptr) {
        const bt_status fit = mx_sides(T, N, code);
        if (fit != BT_OK) return fit;
    }
    if (T >= kMaxSide || N >= kMaxSide) return BT_ERR_UNSUPPORTED;
    const bool res = residual != nullptr;
    if (ldx < N || (res && ldr < N) || (sum != nullptr && lds < N) || (out != nullptr && ldo < N)) return BT_ERR_INVALID_ARG;
    const int64_t far = int64_t(1) << 36;
    if (ldx > far || (res && ldr > far) || (sum != nullptr && lds > far) || (out != nullptr && ldo > far)) return BT_ERR_UNSUPPORTED;
    if (T == 0) return BT_OK;
    if ((sum != nullptr && !res) || (q == nullptr) != (scales == nullptr)) return BT_ERR_INVALID_ARG;
    if (out == nullptr && q == nullptr) return BT_ERR_INVALID_ARG;
    if (x == nullptr) return BT_ERR_INVALID_ARG;
    // in place: row for row
    if ((sum != nullptr && sum == x && lds != ldx) || (sum != nullptr && sum == residual && lds != ldr) || (out != nullptr && out == x && ldo != ldx) ||
        (out != nullptr && out == residual && ldo != ldr) || (out != nullptr && out == sum))
        return BT_ERR_INVALID_ARG;
    const size_t e = static_cast<size_t>(dtype_bytes(dtype));
    if (!aligned(x, e) || !aligned(residual, e) || !aligned(sum, e) || !aligned(out, e) ||
        (weight != nullptr && !aligned(weight, static_cast<size_t>(dtype_bytes(weight_dtype)))) || !aligned(q, 16) || !aligned(scales, 16))
        return BT_ERR_ALIGNMENT;
    NormArgs a = {};
    a.x = x; a.r = residual; a.w = weight;
    a.ldx = ldx; a.ldr = ldr;
    a.w_f32 = weight_dtype == BT_F32;
    a.T = static_cast<int>(T); a.N = static_cast<int>(N);
    const double inv = 1.0 / static_cast<double>(N);
    a.n_inv = static_cast<float>(inv);
    a.n_inv_lo = static_cast<float>(inv - a.n_inv);
    a.eps = static_cast<float>(eps);
    a.eps_lo = static_cast<float>(eps - a.eps);
    a.sum = sum; a.out = out;
    a.lds = lds; a.ldo = ldo;
    a.code = q == nullptr ? kNoCode : static_cast<int>(code);
    a.cols = a.N;
    if (q != nullptr) {
        a.q = static_cast<uint8_t *>(q);
        a.s = static_cast<uint8_t *>(scales);
        a.row_bytes = code_bytes(N, code);
        a.atoms = k_atoms(N, code);
        a.cols = static_cast<int>(a.atoms * 128);
    }
    const bool vec = N % 8 == 0 && a.cols <= 32768 && wide_rows(x, ldx, dtype) && wide_rows(residual, ldr, dtype) &&
                     wide_rows(sum, lds, dtype) && wide_rows(out, ldo, dtype) && aligned(weight, 16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = dtype == BT_F32 ? norm<float>(a, vec, s) : dtype == BT_BF16 ? norm<__nv_bfloat16>(a, vec, s) : norm<__half>(a, vec, s);
    return err == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

// The parts of gw (as many as either path has) and the rows' sums.
size_t bt_rms_norm_backward_workspace(int64_t T, int64_t N) {
    if (T < 1 || N < 1 || T >= kMaxSide || N >= kMaxSide) return 0;
    const int a = back_chunks(T, N, true), b = back_chunks(T, N, false);
    return round_up256(static_cast<size_t>(T) * 16) + round_up256(static_cast<size_t>(a > b ? a : b) * static_cast<size_t>(N) * 4);
}

bt_status bt_rms_norm_backward(const void *g, bt_dtype dtype, int64_t ldg, const void *h, int64_t ldh, const void *weight,
                               bt_dtype weight_dtype, int64_t T, int64_t N, double eps, const void *grad_sum, int64_t ldgs,
                               void *grad_x, int64_t ldgx, float *grad_weight, void *workspace, size_t workspace_bytes,
                               bt_stream stream) {
    if (!float_type(dtype) || (weight != nullptr && weight_dtype != BT_F32 && weight_dtype != dtype)) return BT_ERR_INVALID_ARG;
    if (T < 0 || N < 1 || !std::isfinite(eps) || eps < 0.0 || eps > 1e30) return BT_ERR_INVALID_ARG;
    if (T >= kMaxSide || N >= kMaxSide) return BT_ERR_UNSUPPORTED;
    if (ldg < N || ldh < N || ldgx < N || (grad_sum != nullptr && ldgs < N)) return BT_ERR_INVALID_ARG;
    const int64_t far = int64_t(1) << 36;
    if (ldg > far || ldh > far || ldgx > far || (grad_sum != nullptr && ldgs > far)) return BT_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (!aligned(grad_weight, 4)) return BT_ERR_ALIGNMENT;
    if (T == 0)
        return grad_weight == nullptr || cudaMemsetAsync(grad_weight, 0, static_cast<size_t>(N) * 4, s) == cudaSuccess ? BT_OK : BT_ERR_CUDA;
    if (g == nullptr || h == nullptr || grad_x == nullptr) return BT_ERR_INVALID_ARG;
    if ((grad_x == g && ldgx != ldg) || (grad_x == h && ldgx != ldh) || (grad_x == grad_sum && ldgx != ldgs)) return BT_ERR_INVALID_ARG;
    const size_t e = static_cast<size_t>(dtype_bytes(dtype));
    if (!aligned(g, e) || !aligned(h, e) || !aligned(grad_sum, e) || !aligned(grad_x, e) ||
        (weight != nullptr && !aligned(weight, static_cast<size_t>(dtype_bytes(weight_dtype)))))
        return BT_ERR_ALIGNMENT;
    const size_t need = bt_rms_norm_backward_workspace(T, N);
    if (workspace == nullptr || workspace_bytes < need) return BT_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BT_ERR_ALIGNMENT;
    BackArgs a = {};
    a.g = g; a.h = h; a.w = weight; a.gs = grad_sum;
    a.ldg = ldg; a.ldh = ldh; a.ldgs = ldgs; a.ldgx = ldgx;
    a.w_f32 = weight_dtype == BT_F32;
    a.T = static_cast<int>(T); a.N = static_cast<int>(N);
    a.n_inv = static_cast<float>(1.0 / static_cast<double>(N));
    a.eps = static_cast<float>(eps);
    a.gx = grad_x;
    a.rows = static_cast<float4 *>(workspace);
    float *parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + round_up256(static_cast<size_t>(T) * 16));
    a.parts = grad_weight == nullptr ? nullptr : parts;
    const bool vec = N % 8 == 0 && N <= kBackMost && wide_rows(g, ldg, dtype) && wide_rows(h, ldh, dtype) && wide_rows(grad_sum, ldgs, dtype) &&
                     wide_rows(grad_x, ldgx, dtype) && aligned(weight, 16);
    cudaError_t err = dtype == BT_F32 ? backward<float>(a, vec, s) : dtype == BT_BF16 ? backward<__nv_bfloat16>(a, vec, s) : backward<__half>(a, vec, s);
    if (err == cudaSuccess && grad_weight != nullptr)
        err = launch_pdl(rms_back_join_kernel, dim3(static_cast<unsigned>((N + 31) / 32)), dim3(1024), s, static_cast<const float *>(parts),
                         back_chunks(T, N, vec), static_cast<int>(N), grad_weight);
    return err == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

}  // extern "C"
