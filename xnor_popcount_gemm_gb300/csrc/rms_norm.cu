// Root-mean-square norm before a projection, with the residual's addition, its
// result in the input's type and / or as a microscaled operand, and its backward.
//
//   h = T(x + r)      y = T(f32(h w / sqrt(mean h^2 + eps)))      codes = mx(y)
//   n = h / sqrt(mean h^2 + eps)      gx = (g w - n mean(g w n)) / sqrt(..) + gs
//   gw = sum over the rows of g n
//
// Streams: every row is read once, kept in registers by its CTA (short rows: by some lanes of a warp) and written once. 8192 x 4096
// bf16 with a residual 42 us (268 MB, 95 % of the copy rate), with E4M3 codes as well 48.6 (302 MB, 92 %).
//
// What is rounded to 8 or 4 bits falls one way or the other, so y is the correctly rounded fp32 value (but for about one
// in 2^24): the squares are summed with the rounding errors of the sums beside them, and 1 / sqrt(mean) is a pair of
// floats, the second from one Newton step on the residual 1 - m q^2, which an fma gives exactly. That is about three
// times a plain norm's arithmetic, done two by two.
#include <cmath>

#include "bt_internal.h"
#include "mx.cuh"
#include "tc_ptx.cuh"

namespace bt {
namespace {

using namespace mx;

constexpr int kNoCode = -1;

// Rows whose squares' sum lies beyond kMost (below kLeast) are taken times kDown (kUp): their sum, their mean's inverse and the last
// digits of both, which a pair of floats has, are normal fp32 numbers then. (A sum of 2^124, in fp32's range, has an inverse whose
// second half is not: of 4 million values of rows of 64 around 2^60, 1036 were rounded the other way.) eps as a pair, and as it counts
// beside the squares of values times kUp, where it may be too small for a float by itself.
constexpr float kUp = 0x1p90f, kDown = 0x1p-80f, kMost = 0x1p100f, kLeast = 0x1p-80f;
struct Eps {
    float hi, lo, up_hi, up_lo;
};
Eps eps_of(double eps) {
    // (beyond 1e38 no row is taken times kUp; a positive one stays a normal number, so that its root's inverse is finite)
    const double up = eps > 0.0 ? std::fmin(std::fmax(std::ldexp(eps, 180), 0x1p-126), 1e38) : 0.0;
    Eps e;
    e.hi = static_cast<float>(eps);
    e.lo = static_cast<float>(eps - e.hi);
    e.up_hi = static_cast<float>(up);
    e.up_lo = static_cast<float>(up - e.up_hi);
    return e;
}

struct NormArgs {
    const void *x, *r, *w;                  // r, w: NULL where there is none
    int64_t ldx, ldr;
    int w_f32;
    int T, N;
    float n_inv, n_inv_lo;                  // 1 / N as a pair
    Eps eps;
    void *sum, *out;                        // NULL: not wanted
    int64_t lds, ldo;
    int code;                               // kNoCode, or a bt_code
    uint8_t *q, *s;
    int64_t row_bytes, atoms;
    int cols;                               // N, or the columns up to the end of the last atom
    int al_x, al_r, al_sum, al_out, al_w;   // what their rows start at multiples of
};

// A sum and the rounding errors made in it.
struct Sum2 {
    float s, c;
    __device__ __forceinline__ void join(float os, float oc) {
        const float t = s + os, b = t - s;
        c += (s - (t - b)) + (os - b) + oc;
        s = t;
    }
};
// Two of them, side by side.
struct Sums {
    float2 s, c;
    __device__ __forceinline__ void add(float2 p) {
        const float2 t = add2(s, p), b = sub2(t, s);
        c = add2(c, add2(sub2(s, sub2(t, b)), sub2(p, b)));
        s = t;
    }
    // the square of two values; 16-bit ones have exact squares
    template <bool EXACT> __device__ __forceinline__ void square(float2 v) {
        const float2 p = mul2(v, v);
        add(p);
        if (!EXACT) c = add2(c, fma2(v, v, make_float2(-p.x, -p.y)));
    }
    __device__ __forceinline__ Sum2 joined() const {
        Sum2 r{s.x, c.x};
        r.join(s.y, c.y);
        return r;
    }
};

// The lanes that hold a row, LANES neighbours of a warp.
template <int LANES> __device__ __forceinline__ uint32_t row_lanes() {
    return LANES == 32 ? 0xFFFFFFFFu : ((1u << (LANES & 31)) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
}

// Their sum, and the block's, in every thread, in an order that the thread count alone decides.
template <int LANES = 32> __device__ __forceinline__ Sum2 warp_sum(Sum2 v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        const float s = __shfl_xor_sync(row_lanes<LANES>(), v.s, o), c = __shfl_xor_sync(row_lanes<LANES>(), v.c, o);
        v.join(s, c);
    }
    return v;
}
__device__ __forceinline__ Sum2 block_sum(Sum2 v, float2 (&red)[32]) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(v.s, v.c);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float2 p = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
    return warp_sum(Sum2{p.x, p.y});
}

// Rows that are summed again, their values times a power of two.
__device__ __forceinline__ bool leaves_fp32(float s, const Eps &eps, int N) { return !(s <= kMost && fmaf(eps.hi, static_cast<float>(N), s) >= kLeast); }
__device__ __forceinline__ float power_for(float s) { return s < 1.0f ? kUp : kDown; }

// 1 / sqrt(mean + eps) for values times k, as hi + lo.
struct Inverse {
    float hi, lo;
};
__device__ __forceinline__ Inverse inverse_rms(const Sum2 &v, const NormArgs &a, float k) {
    if (!(v.s <= 3.4e38f)) return Inverse{rsqrtf(v.s), 0.0f};       // infinity: 0, NaN: NaN
    const float p = v.s * a.n_inv;
    float lo = fmaf(v.s, a.n_inv, -p) + fmaf(v.s, a.n_inv_lo, v.c * a.n_inv);
    const float eh = k == kUp ? a.eps.up_hi : (a.eps.hi * k) * k, el = k == kUp ? a.eps.up_lo : (a.eps.lo * k) * k;
    const float t = p + eh, b = t - p;
    lo += (p - (t - b)) + (eh - b) + el;
    const float m = t + lo, ml = lo - (m - t);
    const float r = rsqrtf(m), q = r * r;
    // 1 - m r^2 in the exact r^2 = q + (r^2 - q)
    const float e = fmaf(-m, q, 1.0f) - fmaf(m, fmaf(r, r, -q), ml * q);
    return Inverse{r, r * (0.5f * e + 0.375f * e * e)};
}
// v w / rms; exact: v w has no more than 24 bits.
__device__ __forceinline__ float2 normed(float2 v, float2 w, const Inverse &i, bool exact) {
    const float2 p = mul2(v, w), hi = make_float2(i.hi, i.hi), lo = make_float2(i.lo, i.lo);
    const float2 rest = exact ? mul2(p, lo) : fma2(p, lo, mul2(fma2(v, w, make_float2(-p.x, -p.y)), hi));
    return fma2(p, hi, rest);
}

// Rows eight consecutive columns at a time: thread t has the eights t, t + threads, ... (V of them).
enum Kind {
    kWide,          // rows 16-byte aligned, N a multiple of 8; a row by its CTA; the weight is of type T (or fp32 where T is)
    kWideF32,       // the same with an fp32 weight beside 16-bit rows
    kAligned2,      // 16-bit rows of any alignment and width, a row by its CTA
    kWarp,          // as kWide with any weight; a row by LANES lanes of a warp, for many short ones
};
template <typename T, int V, Kind KIND, int LANES = 32>
__global__ void __launch_bounds__(KIND == kWarp ? 256 : 1024) rms_norm_kernel(const NormArgs a) {
    __shared__ float2 red[2][32];
    constexpr bool kWhole = KIND != kAligned2;
    static_assert(LANES == 32 || KIND == kWarp, "several rows to a warp");
    const int threads = KIND == kWarp ? LANES : blockDim.x, tid = KIND == kWarp ? threadIdx.x & (LANES - 1) : threadIdx.x;
    const int rows = KIND == kWarp ? gridDim.x * (256 / LANES) : gridDim.x;
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    // (a warp's lanes stay together: first is its first row)
    for (int64_t first = KIND == kWarp ? (blockIdx.x * 8 + (threadIdx.x >> 5)) * (32 / LANES) : blockIdx.x; first < a.T; first += rows) {
        const int64_t row = LANES == 32 ? first : first + (threadIdx.x & 31) / LANES;
        const int N = LANES < 32 && row >= a.T ? 0 : a.N, cols = LANES < 32 && row >= a.T ? 0 : a.cols;     // (behind the last: no columns)
        const T *x = static_cast<const T *>(a.x) + row * a.ldx;
        const T *r = static_cast<const T *>(a.r) + row * a.ldr;
        // (x and r may be written in place; another row's elements that a word holds beside this one's are not used)
        auto load = [&](const T *p, int c, int al) { return kWhole ? raw_load<T, false>(p + c) : raw_load_any<T, false>(p + c, a.N - c, al); };
        auto store = [&](void *p, int64_t ld, int c, int al, const Raw8<T> &v) {
            T *q = static_cast<T *>(p) + row * ld + c;
            if (kWhole) raw_store<T>(q, v);
            else raw_store_any<T>(q, v, a.N - c, al);
        };
        Raw8<T> h[V], rr[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (tid + i * threads) * 8;
            h[i] = Raw8<T>{};
            if (c >= N) continue;
            h[i] = load(x, c, a.al_x);
            if (a.r != nullptr) rr[i] = load(r, c, a.al_r);
        }
        if (a.r != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = (tid + i * threads) * 8;
                if (c >= N) continue;
                float v[8], o[8];
                raw_unpack<T>(h[i], v);
                raw_unpack<T>(rr[i], o);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += o[e];
                h[i] = raw_pack<T>(v);
                if (a.sum != nullptr) store(a.sum, a.lds, c, a.al_sum, h[i]);
            }
        }
        auto squares = [&](float k) {
            Sums p{};
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float v[8];
                raw_unpack<T>(h[i], v);
#pragma unroll
                for (int e = 0; e < 8; e += 2) p.square<sizeof(T) == 2>(make_float2(v[e] * k, v[e + 1] * k));
            }
            return p.joined();
        };
        auto together = [&](Sum2 v, float2 (&x2)[32]) { return KIND == kWarp ? warp_sum<LANES>(v) : block_sum(v, x2); };
        Sum2 total = together(squares(1.0f), red[0]);
        float k = 1.0f;
        if (leaves_fp32(total.s, a.eps, a.N)) {
            k = power_for(total.s);
            total = together(squares(k), red[1]);
        }
        const Inverse inv = inverse_rms(total, a, k);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = tid + i * threads, c = g * 8;
            if (c - (tid & 31) * 8 >= a.cols) continue;                 // (whole warps)
            Raw8<T> o = {};
            if (c < N) {
                float v[8], w[8], y[8];
                raw_unpack<T>(h[i], v);
                if (k != 1.0f) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= k;
                }
                const bool f32 = KIND == kWideF32 || (sizeof(T) == 2 && (KIND == kAligned2 || KIND == kWarp) && a.w_f32);
                if (a.w == nullptr) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
                } else if (f32) {
                    const float *p = static_cast<const float *>(a.w) + c;
                    raw_unpack<float>(kWhole ? raw_load<float>(p) : raw_load_any<float>(p, a.N - c, a.al_w), w);
                } else {
                    const T *p = static_cast<const T *>(a.w) + c;
                    raw_unpack<T>(kWhole ? raw_load<T>(p) : raw_load_any<T>(p, a.N - c, a.al_w), w);
                }
                const bool exact = sizeof(T) == 2 && !f32;
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 n = normed(make_float2(v[e], v[e + 1]), make_float2(w[e], w[e + 1]), inv, exact);
                    y[e] = n.x;
                    y[e + 1] = n.y;
                }
                if (!kWhole) {                                          // (what is past N was zero: 0 / 0 stays out of the block)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = c + e < a.N ? y[e] : 0.0f;
                }
                o = raw_pack<T>(y);
                if (a.out != nullptr) store(a.out, a.ldo, c, a.al_out, o);
            }
            if (LANES < 16 || a.code == kNoCode) continue;              // (sixteen lanes make a word of scales)
            const uint32_t top = quad_top<T>(o);
            const bool e4m3 = a.code == BT_CODE_E4M3;
            const uint32_t s = e4m3 ? scale_of<BT_CODE_E4M3>(top) : scale_of<BT_CODE_E2M1>(top), word = atom_word(s);
            if (c >= cols) continue;
            float y[8];
            raw_unpack<T>(o, y);
            uint8_t *p = a.q + row * a.row_bytes + static_cast<int64_t>(g) * (e4m3 ? 8 : 4);
            if (e4m3) store8<BT_CODE_E4M3>(p, code8<BT_CODE_E4M3>(y, inverse_of(s)));
            else store8<BT_CODE_E2M1>(p, code8<BT_CODE_E2M1>(y, inverse_of(s)));
            if ((tid & 15) == 0) *reinterpret_cast<uint32_t *>(a.s + scale_at(row, g >> 2, a.atoms)) = word;
        }
        if (KIND != kWarp) break;                                       // (a row a CTA)
    }
}

// fp32 rows of odd widths or alignments, and rows wider than the registers above hold: thread t has the columns t, t + threads, ..., a
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
    auto squares = [&](float k, bool first) {
        Sums p{};
#pragma unroll
        for (int i = 0; i < E; i += 2) p.square<sizeof(T) == 2>(make_float2(h[i] * k, h[i + 1] * k));
        for (int c = threadIdx.x + E * step; c < a.N; c += step) p.square<sizeof(T) == 2>(make_float2((first ? load(c, true) : again(c)) * k, 0.0f));
        return p.joined();
    };
    Sum2 total = block_sum(squares(1.0f, true), red[0]);
    float k = 1.0f;
    if (leaves_fp32(total.s, a.eps, a.N)) {
        k = power_for(total.s);
        total = block_sum(squares(k, false), red[1]);
    }
    const Inverse inv = inverse_rms(total, a, k);
    auto finish = [&](int c, float v) {
        float y = 0.0f;
        if (c < a.N) {
            const float w = a.w == nullptr ? 1.0f
                            : a.w_f32      ? __ldg(static_cast<const float *>(a.w) + c)
                                           : Elem<T>::to_f32(static_cast<const T *>(a.w)[c]);
            const T o = from_f32<T>(normed(make_float2(v * k, 0.0f), make_float2(w, 0.0f), inv, sizeof(T) == 2 && !a.w_f32).x);
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
    float n_inv;
    Eps eps;
    void *gx;
    float *parts;                           // [chunks, N], NULL: gw not wanted
    float4 *rows;                           // (any) 1 / rms of the values times k, mean(g w n), k of every row
    int chunks;
    int ahead, pitch;                       // rows of the ring, bytes of one of a row's arrays in it
    unsigned int *err;
    unsigned long long wait_ns;
};
constexpr int kMostAhead = 3;
constexpr int kWarpRow = 512, kBackWarpRow = 256;   // the longest row that goes to a warp, forward and backward
constexpr int kBackCtas = 2;                // an SM: three hold fewer rows and leave more parts of gw (31 -> 40 us)
constexpr int kNarrowRow = 1024;            // up to which there are more of them
constexpr int kNarrowCtas = 6;

template <int LANES = 32> __device__ __forceinline__ float2 warp_pair(float2 v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(row_lanes<LANES>(), v.x, o);
        v.y += __shfl_xor_sync(row_lanes<LANES>(), v.y, o);
    }
    return v;
}
__device__ __forceinline__ float2 block_pair(float2 v, float2 (&red)[32]) {
    v = warp_pair(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return warp_pair(lane < warps ? red[lane] : make_float2(0.0f, 0.0f));
}
__device__ __forceinline__ float eps_times(const Eps &eps, float k) { return k == kUp ? eps.up_hi : (eps.hi * k) * k; }
__device__ __forceinline__ float inverse_plain(float s, float n_inv, float eps) { return 1.0f / sqrtf(fmaf(s, n_inv, eps)); }

// Eight of a row's values: eight neighbours (VEC: rows 16-byte aligned, N a multiple of 8), thread t's i-th eight at
// (t + i threads) 8, or, at any alignment, every `threads`-th from t + 8 i threads on, so that neighbours take neighbours.
template <bool VEC> struct Columns {
    int first, step, N;
    __device__ __forceinline__ Columns(int t, int i, int n, int threads) : first(VEC ? (t + i * threads) * 8 : t + i * 8 * threads), step(VEC ? 1 : threads), N(n) {}
    template <typename T> __device__ __forceinline__ Raw8<T> load(const T *row) const {
        Raw8<T> r = {};
        if constexpr (VEC) {
            if (first < N) {
                r.a = *reinterpret_cast<const uint4 *>(row + first);
                if constexpr (sizeof(T) == 4) r.b = *(reinterpret_cast<const uint4 *>(row + first) + 1);
            }
        } else {
            uint32_t w[sizeof(T) * 2] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (first + e * step >= N) continue;
                if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(row[first + e * step]);
                else w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[first + e * step]) << (16 * (e & 1));
            }
            r.a = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (sizeof(T) == 4) r.b = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return r;
    }
    template <typename T> __device__ __forceinline__ void store(T *row, const float (&v)[8]) const {
        if constexpr (VEC) {
            if (first < N) raw_store<T>(row + first, raw_pack<T>(v));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (first + e * step < N) row[first + e * step] = from_f32<T>(v[e]);
        }
    }
};

// Waits for a row, or until the asking warp, which keeps the time, has given up: then the loop goes on with whatever is there, so
// that all threads meet at the exchanges, and the results are incomplete. (A function of few registers: 4096 x 4096 bf16 33.4 us
// with the clock read here, 32.8 with the loop in line, 32.1 so.)
__device__ __noinline__ void await_row(uint32_t bar, uint32_t parity, uint32_t flag) {
    uint32_t given_up = 0;
    while (!tc::mbar_try_wait(bar, parity) && given_up == 0u) asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(given_up) : "r"(flag) : "memory");
}

// A CTA takes rows blockIdx.x, + gridDim.x, ..., keeps its threads' columns of gw in registers, and has the next two rows on
// their way into a ring in shared memory: bulk copies of the 16-byte pieces that hold a row, asked for by a warp of its
// own. Memory: 4096 x 4096 bf16 with gs 27 us (134 MB, 73 % of the copy rate), and 4 for the parts of gw and their sum;
// with rows loaded when they are due 41.
template <typename T, int V, int MOST, bool VEC>
__global__ void __launch_bounds__(MOST + 32, MOST == 128 ? kNarrowCtas : MOST == 256 ? kBackCtas : 1) rms_back_kernel(const BackArgs a) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 red[2][2][16];
    __shared__ uint64_t bars[2 * kMostAhead];
    __shared__ uint32_t abort_word;
    volatile uint32_t *abort_flag = &abort_word;
    const int threads = static_cast<int>(blockDim.x) - 32, warps = threads >> 5;       // but for the last warp, which asks
    const int rows = (a.T - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const int D = a.ahead, arrays = a.gs != nullptr ? 3 : 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full = [&](int i) { return smem_u32(&bars[i]); };
    auto empty = [&](int i) { return smem_u32(&bars[kMostAhead + i]); };
    if (threadIdx.x == 0) {
        for (int i = 0; i < D; ++i) {
            tc::mbar_init(full(i), 1);
            tc::mbar_init(empty(i), static_cast<uint32_t>(warps));
        }
        abort_word = 0u;
        tc::fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const T *const src[3] = {static_cast<const T *>(a.g), static_cast<const T *>(a.h), static_cast<const T *>(a.gs)};
    const int64_t lds[3] = {a.ldg, a.ldh, a.ldgs};
    auto start = [&](int n, int k) { return reinterpret_cast<uintptr_t>(src[k] + (blockIdx.x + static_cast<int64_t>(n) * gridDim.x) * lds[k]); };

    if (warp == warps) {
        if (lane == 0) {
            int n = 0, slot = 0;
            uint32_t phase = 1;
            for (; n < rows; ++n) {
                if (!tc::wait_fast(empty(slot), phase, abort_flag, a.err, a.wait_ns)) break;
                uint32_t to = smem_u32(ring) + static_cast<uint32_t>(slot * arrays * a.pitch), all = 0, bytes[3];
                uintptr_t from[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    if (k >= arrays) continue;
                    const uintptr_t p = start(n, k);
                    from[k] = p & ~uintptr_t(15);
                    bytes[k] = static_cast<uint32_t>(((p + static_cast<uintptr_t>(a.N) * sizeof(T) + 15) & ~uintptr_t(15)) - from[k]);
                    all += bytes[k];
                }
                tc::mbar_arrive_expect_tx(full(slot), all);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (k < arrays) tc::bulk_load(to + static_cast<uint32_t>(k * a.pitch), reinterpret_cast<const void *>(from[k]), bytes[k], full(slot));
                if (++slot == D) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            // What was asked for lands before shared memory is given back, also where a wait ran out. Those who wait for it watch
            // the flag alone.
            for (int m = n > D ? n - D : 0; m < n; ++m) {
                uint32_t never = 0;
                const uint32_t bar = full(m % D), parity = static_cast<uint32_t>(m / D) & 1u;
                if (!tc::wait_bounded(bar, parity, abort_flag, a.err, a.wait_ns)) tc::wait_bounded(bar, parity, &never, a.err);
            }
        }
        return;
    }

    // The weight as floats behind the ring, each thread reading what it wrote. Rows of more than 4096 values (MOST = 512) need the
    // room: their weight comes from L2, and beyond 8192 (V = 4) g and h are read a second time too.
    constexpr bool kKeep = MOST <= 256, kHold = V < 4;
    float *const weight = reinterpret_cast<float *>(ring + D * arrays * a.pitch) + 8 * V * threadIdx.x;
    float2 acc[V][4];
    auto weight_of = [&](int i, float (&v)[8]) {
        const Columns<VEC> c(threadIdx.x, i, a.N, threads);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 1.0f;
        if (a.w != nullptr && a.w_f32) raw_unpack<float>(c.template load<float>(static_cast<const float *>(a.w)), v);
        else if (a.w != nullptr) raw_unpack<T>(c.template load<T>(static_cast<const T *>(a.w)), v);
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (kKeep) {
            float v[8];
            weight_of(i, v);
            raw_store<float>(weight + 8 * i, raw_pack<float>(v));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = make_float2(0.0f, 0.0f);
    }
    auto weights = [&](int i, float2 (&w)[4]) {
        float v[8];
        if (kKeep) {
            const float4 lo = *reinterpret_cast<const float4 *>(weight + 8 * i), hi = *reinterpret_cast<const float4 *>(weight + 8 * i + 4);
            v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
            v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
        } else {
            weight_of(i, v);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = make_float2(v[2 * e], v[2 * e + 1]);
    };
    // the block's sums, in every thread
    auto together = [&](float2 v, float2 (&x)[16]) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
            v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
        }
        if (lane == 0) x[warp] = v;
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
        v = x[0];
#pragma unroll
        for (int i = 1; i < MOST / 32; ++i)
            if (i < warps) v = add2(v, x[i]);
        return v;
    };
    int slot = 0;
    uint32_t phase = 0;
    for (int n = 0; n < rows; ++n) {
        if (!tc::mbar_test_wait(full(slot), phase)) await_row(full(slot), phase, smem_u32(&abort_word));
        auto row_of = [&](int k) {
            const uint8_t *p = ring + (slot * arrays + k) * a.pitch;
            return reinterpret_cast<const T *>(VEC ? p : p + (start(n, k) & 15));
        };
        Raw8<T> g[V], h[V];
        auto take = [&](int i) {
            const Columns<VEC> c(threadIdx.x, i, a.N, threads);
            g[i] = c.template load<T>(row_of(0));
            h[i] = c.template load<T>(row_of(1));
        };
        if (kHold) {
#pragma unroll
            for (int i = 0; i < V; ++i) take(i);
        }
        auto sums = [&](float k) {
            float2 s = make_float2(0.0f, 0.0f), d = s;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (!kHold) take(i);
                float vg[8], vh[8];
                raw_unpack<T>(g[i], vg);
                raw_unpack<T>(h[i], vh);
                float2 w[4];
                weights(i, w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 u = mul2(make_float2(vh[2 * e], vh[2 * e + 1]), make_float2(k, k));
                    s = fma2(u, u, s);
                    d = fma2(mul2(make_float2(vg[2 * e], vg[2 * e + 1]), w[e]), u, d);
                }
            }
            return make_float2(s.x + s.y, d.x + d.y);
        };
        float2 p = together(sums(1.0f), red[0][n & 1]);
        float k = 1.0f, eps = a.eps.hi;
        if (leaves_fp32(p.x, a.eps, a.N)) {
            k = power_for(p.x);
            eps = eps_times(a.eps, k);
            p = together(sums(k), red[1][n & 1]);
        }
        const float inv = inverse_plain(p.x, a.n_inv, eps), mean = p.y * inv * a.n_inv, n1 = k * inv;
        T *gx = static_cast<T *>(a.gx) + (blockIdx.x + static_cast<int64_t>(n) * gridDim.x) * a.ldgx;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Columns<VEC> c(threadIdx.x, i, a.N, threads);
            if (!kHold) take(i);
            float vg[8], vh[8], o[8];
            raw_unpack<T>(g[i], vg);
            raw_unpack<T>(h[i], vh);
            if (a.gs != nullptr) raw_unpack<T>(c.template load<T>(row_of(2)), o);
            float2 w[4];
            weights(i, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // (h k first: k brings it into range)
                const float2 u = mul2(mul2(make_float2(vh[2 * e], vh[2 * e + 1]), make_float2(k, k)), make_float2(inv, inv));
                const float2 gg = make_float2(vg[2 * e], vg[2 * e + 1]);
                acc[i][e] = fma2(gg, u, acc[i][e]);
                float2 d = mul2(fma2(u, make_float2(-mean, -mean), mul2(gg, w[e])), make_float2(n1, n1));
                if (a.gs != nullptr) d = add2(d, make_float2(o[2 * e], o[2 * e + 1]));
                o[2 * e] = d.x;
                o[2 * e + 1] = d.y;
            }
            c.template store<T>(gx, o);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty(slot));
        if (++slot == D) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (a.parts == nullptr) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v[8] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y, acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y};
        Columns<VEC>(threadIdx.x, i, a.N, threads).template store<float>(a.parts + static_cast<int64_t>(blockIdx.x) * a.N, v);
    }
}

// Many short rows: one to LANES lanes, eight columns a lane, no exchange but theirs; the CTA's rows join their parts of gw
// at the end.
template <typename T, bool VEC, int LANES>
__global__ void __launch_bounds__(256, 3) rms_back_warp_kernel(const BackArgs a) {
    constexpr int kRow = LANES * 8, kRows = 256 / LANES;
    __shared__ __align__(16) float join[kRows][kRow];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int part = threadIdx.x / LANES, lane = threadIdx.x & (LANES - 1);
    float2 acc[4], w[4];
    {
        const Columns<VEC> c(lane, 0, a.N, LANES);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 1.0f;
        if (a.w != nullptr && a.w_f32) raw_unpack<float>(c.template load<float>(static_cast<const float *>(a.w)), v);
        else if (a.w != nullptr) raw_unpack<T>(c.template load<T>(static_cast<const T *>(a.w)), v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = make_float2(v[2 * e], v[2 * e + 1]);
            acc[e] = make_float2(0.0f, 0.0f);
        }
    }
    // (a warp's lanes stay together: first is its first row)
    for (int64_t first = blockIdx.x * kRows + (threadIdx.x >> 5) * (32 / LANES); first < a.T; first += gridDim.x * kRows) {
        const int64_t row = LANES == 32 ? first : first + (threadIdx.x & 31) / LANES;
        const bool real = LANES == 32 || row < a.T;
        const Columns<VEC> c(lane, 0, real ? a.N : 0, LANES);           // (behind the last: no columns)
        const Raw8<T> g = c.template load<T>(static_cast<const T *>(a.g) + row * a.ldg);
        const Raw8<T> h = c.template load<T>(static_cast<const T *>(a.h) + row * a.ldh);
        Raw8<T> gs;
        if (a.gs != nullptr) gs = c.template load<T>(static_cast<const T *>(a.gs) + row * a.ldgs);
        auto sums = [&](float k) {
            float2 s = make_float2(0.0f, 0.0f), d = s;
            float vg[8], vh[8];
            raw_unpack<T>(g, vg);
            raw_unpack<T>(h, vh);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = mul2(make_float2(vh[2 * e], vh[2 * e + 1]), make_float2(k, k));
                s = fma2(u, u, s);
                d = fma2(mul2(make_float2(vg[2 * e], vg[2 * e + 1]), w[e]), u, d);
            }
            return warp_pair<LANES>(make_float2(s.x + s.y, d.x + d.y));
        };
        float2 p = sums(1.0f);
        float k = 1.0f, eps = a.eps.hi;
        if (leaves_fp32(p.x, a.eps, a.N)) {
            k = power_for(p.x);
            eps = eps_times(a.eps, k);
            p = sums(k);
        }
        const float inv = real ? inverse_plain(p.x, a.n_inv, eps) : 0.0f, mean = p.y * inv * a.n_inv, n1 = k * inv;
        float vg[8], vh[8], o[8];
        raw_unpack<T>(g, vg);
        raw_unpack<T>(h, vh);
        if (a.gs != nullptr) raw_unpack<T>(gs, o);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (h k first: k brings it into range)
            const float2 u = mul2(mul2(make_float2(vh[2 * e], vh[2 * e + 1]), make_float2(k, k)), make_float2(inv, inv));
            const float2 gg = make_float2(vg[2 * e], vg[2 * e + 1]);
            acc[e] = fma2(gg, u, acc[e]);
            float2 d = mul2(fma2(u, make_float2(-mean, -mean), mul2(gg, w[e])), make_float2(n1, n1));
            if (a.gs != nullptr) d = add2(d, make_float2(o[2 * e], o[2 * e + 1]));
            o[2 * e] = d.x;
            o[2 * e + 1] = d.y;
        }
        c.template store<T>(static_cast<T *>(a.gx) + row * a.ldgx, o);
    }
    if (a.parts == nullptr) return;
    const float v[8] = {acc[0].x, acc[0].y, acc[1].x, acc[1].y, acc[2].x, acc[2].y, acc[3].x, acc[3].y};
    Columns<VEC>(lane, 0, a.N, LANES).template store<float>(join[part], v);
    __syncthreads();
    for (int col = threadIdx.x; col < a.N; col += 256) {
        float sum = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) sum += join[r][col];
        a.parts[static_cast<int64_t>(blockIdx.x) * a.N + col] = sum;
    }
}

// Wider rows than a ring holds: the rows' sums, then strips of columns, eight a thread, so that g and h are read twice. 1024 x 32768
// bf16 with gs 77 us (268 MB, 51 % of the copy rate where 67 can be had; 236 with a column a thread).
template <typename T, bool VEC> __device__ __forceinline__ void weight8(const BackArgs &a, const Columns<VEC> &c, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
    if (a.w != nullptr && a.w_f32) raw_unpack<float>(c.template load<float>(static_cast<const float *>(a.w)), v);
    else if (a.w != nullptr) raw_unpack<T>(c.template load<T>(static_cast<const T *>(a.w)), v);
}
template <typename T, bool VEC> __global__ void __launch_bounds__(512) rms_back_rows_kernel(const BackArgs a) {
    __shared__ float2 red[2][32];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T *g = static_cast<const T *>(a.g) + row * a.ldg, *h = static_cast<const T *>(a.h) + row * a.ldh;
    auto sums = [&](float k) {
        float2 s = make_float2(0.0f, 0.0f), d = s;
        const int eights = (a.N + 8 * 512 - 1) / (8 * 512);
#pragma unroll 2
        for (int i = 0; i < eights; ++i) {
            const Columns<VEC> c(threadIdx.x, i, a.N, 512);
            float vg[8], vh[8], w[8];
            raw_unpack<T>(c.template load<T>(g), vg);
            raw_unpack<T>(c.template load<T>(h), vh);
            weight8<T, VEC>(a, c, w);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 u = mul2(make_float2(vh[e], vh[e + 1]), make_float2(k, k));
                s = fma2(u, u, s);
                d = fma2(mul2(make_float2(vg[e], vg[e + 1]), make_float2(w[e], w[e + 1])), u, d);
            }
        }
        return make_float2(s.x + s.y, d.x + d.y);
    };
    float2 p = block_pair(sums(1.0f), red[0]);
    float k = 1.0f, eps = a.eps.hi;
    if (leaves_fp32(p.x, a.eps, a.N)) {
        k = power_for(p.x);
        eps = eps_times(a.eps, k);
        p = block_pair(sums(k), red[1]);
    }
    const float inv = inverse_plain(p.x, a.n_inv, eps);
    if (threadIdx.x == 0) a.rows[row] = make_float4(inv, p.y * inv * a.n_inv, k, 0.0f);
}
constexpr int kStrip = 128, kStripColumns = kStrip * 8, kStripCtas = 5;     // threads, columns, CTAs an SM
template <typename T, bool VEC> __global__ void __launch_bounds__(kStrip, kStripCtas) rms_back_strips_kernel(const BackArgs a) {
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const Columns<VEC> c(threadIdx.x, blockIdx.x, a.N, kStrip);
    float w[8];
    weight8<T, VEC>(a, c, w);
    float2 acc[4] = {};
    // (two rows' loads before either's stores, which may go where they came from)
    for (int64_t first = blockIdx.y; first < a.T; first += 2 * static_cast<int64_t>(a.chunks)) {
        Raw8<T> g[2] = {}, h[2] = {}, gs[2] = {};
        float4 s[2] = {};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t row = first + r * static_cast<int64_t>(a.chunks);
            if (row >= a.T) continue;
            s[r] = a.rows[row];
            g[r] = c.template load<T>(static_cast<const T *>(a.g) + row * a.ldg);
            h[r] = c.template load<T>(static_cast<const T *>(a.h) + row * a.ldh);
            if (a.gs != nullptr) gs[r] = c.template load<T>(static_cast<const T *>(a.gs) + row * a.ldgs);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t row = first + r * static_cast<int64_t>(a.chunks);
            if (row >= a.T) continue;
            const float n1 = s[r].x * s[r].z;
            float vg[8], vh[8], o[8];
            raw_unpack<T>(g[r], vg);
            raw_unpack<T>(h[r], vh);
            raw_unpack<T>(gs[r], o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // (h k first: k brings it into range)
                const float2 u = mul2(mul2(make_float2(vh[2 * e], vh[2 * e + 1]), make_float2(s[r].z, s[r].z)), make_float2(s[r].x, s[r].x));
                const float2 gg = make_float2(vg[2 * e], vg[2 * e + 1]);
                acc[e] = fma2(gg, u, acc[e]);
                float2 d = mul2(fma2(u, make_float2(-s[r].y, -s[r].y), mul2(gg, make_float2(w[2 * e], w[2 * e + 1]))), make_float2(n1, n1));
                if (a.gs != nullptr) d = add2(d, make_float2(o[2 * e], o[2 * e + 1]));
                o[2 * e] = d.x;
                o[2 * e + 1] = d.y;
            }
            c.template store<T>(static_cast<T *>(a.gx) + row * a.ldgx, o);
        }
    }
    if (a.parts == nullptr) return;
    const float v[8] = {acc[0].x, acc[0].y, acc[1].x, acc[1].y, acc[2].x, acc[2].y, acc[3].x, acc[3].y};
    float *to = a.parts + static_cast<int64_t>(blockIdx.y) * a.N;
    c.template store<float>(to, v);
}

// gw = the parts' sum: 32 columns a CTA, 32 rows of parts at a time, eight of them on their way a thread.
__global__ void __launch_bounds__(1024) rms_back_join_kernel(const float *parts, int chunks, int N, float *gw) {
    __shared__ float red[32][33];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < N) {
        for (int i = warp; i < chunks; i += 32 * 8) {
            float p[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) p[k] = i + 32 * k < chunks ? parts[static_cast<int64_t>(i + 32 * k) * N + c] : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) v += p[k];
        }
    }
    red[warp][lane] = v;
    __syncthreads();
    v = red[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (lane == 0 && blockIdx.x * 32 + warp < N) gw[blockIdx.x * 32 + warp] = v;
}

int rows_align(const void *p, int64_t ld, bt_dtype t) { return mx::rows_align(static_cast<const char *>(p), ld, dtype_bytes(t)); }
bool float_type(bt_dtype t) { return t == BT_F32 || t == BT_BF16 || t == BT_F16; }
bool wide_rows(const void *p, int64_t ld, bt_dtype t) { return p == nullptr || (aligned(p, 16) && (ld * dtype_bytes(t)) % 16 == 0); }
unsigned whole_warps(int64_t n) { return static_cast<unsigned>((n + 31) / 32 * 32); }

// Many short rows go to the lanes of a warp: 131072 rows of 256 bf16 with a residual 43 us (131 with a CTA each), backward 61 (231). Of
// 1024 values a CTA a row is faster forward (with codes 48 us, 53 by a warp), and backward of 512 already (59 and 69).
bool warp_rows(int64_t T, int64_t N) { return N <= kWarpRow && T >= 16 * device_sm_count(); }

// Two eights a lane on no more lanes than that takes: a row's exchange and its root then serve as many rows as a warp holds
// (bf16, 134 MB: 524288 x 128 57 us, 82 with one eight on sixteen lanes and 156 with a warp each; 262144 x 256 66, 81 with a
// warp each). A word of scales takes sixteen lanes.
template <typename T> cudaError_t norm_warps(const NormArgs &a, cudaStream_t s) {
    const int64_t groups = (a.cols + 7) / 8;
    auto go = [&](void (*kern)(const NormArgs), int lanes) {
        const int64_t each = 256 / lanes, ctas = (a.T + each - 1) / each, most = 8 * device_sm_count();
        return launch_pdl(kern, dim3(static_cast<unsigned>(ctas < most ? ctas : most)), dim3(256), s, a);
    };
    if (groups <= 8) return go(rms_norm_kernel<T, 2, kWarp, 4>, 4);
    if (groups <= 16 && a.code == kNoCode) return go(rms_norm_kernel<T, 2, kWarp, 8>, 8);
    if (groups <= 16) return go(rms_norm_kernel<T, 1, kWarp, 16>, 16);
    if (groups <= 32) return go(rms_norm_kernel<T, 2, kWarp, 16>, 16);
    return go(rms_norm_kernel<T, 2, kWarp, 32>, 32);
}
template <typename T, Kind KIND> cudaError_t norm_rows(const NormArgs &a, cudaStream_t s) {
    const int64_t groups = (a.cols + 7) / 8, sms = device_sm_count();
    // few rows: as many threads as there are loads (16 x 4096: 2.8 us, 4.3 with four loads a thread); many: four loads
    // a thread on their way (8192 x 4096 with codes: 53 us, 64 with one, 58.5 with two, 65 with eight)
    const int v = groups > 2048 || a.T > 8 * sms ? 4 : groups > 1024 || a.T > 2 * sms ? 2 : 1;
    const dim3 grid(static_cast<unsigned>(a.T)), block(whole_warps((groups + v - 1) / v));
    return launch_pdl(v == 1   ? rms_norm_kernel<T, 1, KIND>
                      : v == 2 ? rms_norm_kernel<T, 2, KIND>
                               : rms_norm_kernel<T, 4, KIND>, grid, block, s, a);
}
template <typename T> cudaError_t norm(const NormArgs &a, bool vec, cudaStream_t s) {
    if (vec && warp_rows(a.T, a.cols)) return norm_warps<T>(a, s);
    if constexpr (sizeof(T) == 2) {
        if (vec && a.w != nullptr && a.w_f32) return norm_rows<T, kWideF32>(a, s);
        // (fp32 rows of odd alignments go by neighbours)
        if (!vec && a.cols <= 32768) return norm_rows<T, kAligned2>(a, s);
    }
    if (vec) return norm_rows<T, kWide>(a, s);
    const dim3 grid(static_cast<unsigned>(a.T));
    if (a.cols <= 8192) return launch_pdl(rms_norm_any_kernel<T, 8>, grid, dim3(whole_warps((a.cols + 7) / 8)), s, a);
    return launch_pdl(rms_norm_any_kernel<T, 16>, grid, dim3(a.cols < 16384 ? whole_warps((a.cols + 15) / 16) : 1024), s, a);
}

// Rows that rms_back_kernel takes: two of them (g, h and gs) fit in its ring.
constexpr int kRingMost = 208 * 1024;
int row_pitch(int64_t N, int elem) { return static_cast<int>((N * elem + 15) / 16 * 16 + 16); }
int weight_bytes(int64_t N) {
    if (N <= kNarrowRow) return static_cast<int>(whole_warps((N + 7) / 8) * 32);
    return N <= 4096 ? static_cast<int>((N + 2047) / 2048 * 2048 * 4) : 0;
}
bool back_ring(int64_t N, int elem) { return N <= 16384 && 6 * row_pitch(N, elem) + weight_bytes(N) <= kRingMost; }

// CTAs an SM. A short row leaves its CTA waiting for its exchange, so there are as many as an SM holds at 64 registers a thread
// (32768 x 1024 bf16: 51 us with six, 57 with five, 68 with four, 90 with two; 61 with seven, of which one waits for the others).
// Below eight rows each, the parts of gw cost more than that gives (3000 x 1024: 12 us with two, 14 with six).
int back_ctas(int64_t N) { return N > kNarrowRow ? kBackCtas : 32 / static_cast<int>(whole_warps((N + 7) / 8) / 32 + 1); }
// (backward: the longest row that goes to a warp is shorter)
bool back_warp_rows(int64_t T, int64_t N) { return N <= kBackWarpRow && warp_rows(T, N); }

int back_chunks(int64_t T, int64_t N, int elem) {
    const int64_t sms = device_sm_count(), strips = (N + kStripColumns - 1) / kStripColumns;
    int64_t n;
    if (back_warp_rows(T, N)) n = 3 * sms;
    else if (back_ring(N, elem)) n = (T < 8 * back_ctas(N) * sms ? kBackCtas : back_ctas(N)) * sms;
    else n = (kStripCtas * sms + strips - 1) / strips;
    if (n > T) n = T;
    return static_cast<int>(n < 1 ? 1 : n);
}

template <typename T, int V, int MOST, bool VEC> cudaError_t back_launch(const BackArgs &a, cudaStream_t s) {
    auto kern = rms_back_kernel<T, V, MOST, VEC>;
    static ContextOnce once;
    if (const cudaError_t e = allow_all_smem(kern, kRingMost, once); e != cudaSuccess) return e;
    const unsigned threads = whole_warps(((a.N + 7) / 8 + V - 1) / V) + 32;
    const size_t smem = static_cast<size_t>(a.ahead) * (a.gs != nullptr ? 3 : 2) * static_cast<size_t>(a.pitch) + (MOST <= 256 ? (threads - 32) * V * 32 : 0);
    return launch_pdl_smem(kern, dim3(static_cast<unsigned>(a.chunks)), dim3(threads), smem, s, a);
}
template <typename T, bool VEC> cudaError_t back_rows(BackArgs a, cudaStream_t s) {
    const int64_t groups = (a.N + 7) / 8;
    a.pitch = row_pitch(a.N, sizeof(T));
    const int per = (a.gs != nullptr ? 3 : 2) * a.pitch;
    // (a short row's CTAs are many: 2 KB each for what a CTA has besides, of 213)
    const int share = a.N > kNarrowRow ? kRingMost / kBackCtas : 213 * 1024 / back_ctas(a.N) - 2048;
    a.ahead = (share - weight_bytes(a.N)) / per;
    a.ahead = a.ahead < 2 ? 2 : a.ahead > 3 ? 3 : a.ahead;
    if (a.N <= kNarrowRow) return back_launch<T, 1, 128, VEC>(a, s);
    if (groups <= 256) return back_launch<T, 1, 256, VEC>(a, s);
    if (groups <= 512) return back_launch<T, 2, 256, VEC>(a, s);
    if (groups <= 1024) return back_launch<T, 2, 512, VEC>(a, s);
    return back_launch<T, 4, 512, VEC>(a, s);
}
template <typename T, bool VEC> cudaError_t back_warps(const BackArgs &a, cudaStream_t s) {
    const int64_t groups = (a.N + 7) / 8;
    // one eight a lane: with two its registers hide less of memory's delay (524288 x 128 bf16: 142 us, 93 with one)
    return launch_pdl(groups <= 8    ? rms_back_warp_kernel<T, VEC, 8>
                      : groups <= 16 ? rms_back_warp_kernel<T, VEC, 16>
                                     : rms_back_warp_kernel<T, VEC, 32>, dim3(static_cast<unsigned>(a.chunks)), dim3(256), s, a);
}
template <typename T> cudaError_t backward(BackArgs a, bool vec, cudaStream_t s) {
    a.chunks = back_chunks(a.T, a.N, sizeof(T));
    if (back_warp_rows(a.T, a.N)) return vec ? back_warps<T, true>(a, s) : back_warps<T, false>(a, s);
    if (back_ring(a.N, sizeof(T))) return vec ? back_rows<T, true>(a, s) : back_rows<T, false>(a, s);
    const cudaError_t e = launch_pdl(vec ? rms_back_rows_kernel<T, true> : rms_back_rows_kernel<T, false>, dim3(static_cast<unsigned>(a.T)), dim3(512), s, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(vec ? rms_back_strips_kernel<T, true> : rms_back_strips_kernel<T, false>,
                      dim3(static_cast<unsigned>((a.N + kStripColumns - 1) / kStripColumns), static_cast<unsigned>(a.chunks)), dim3(kStrip), s, a);
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
    a.eps = eps_of(eps);
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
    a.al_x = rows_align(x, ldx, dtype);
    a.al_r = rows_align(residual, ldr, dtype);
    a.al_sum = rows_align(sum, lds, dtype);
    a.al_out = rows_align(out, ldo, dtype);
    a.al_w = rows_align(weight, 0, weight_dtype);
    const bool vec = N % 8 == 0 && a.cols <= 32768 && wide_rows(x, ldx, dtype) && wide_rows(residual, ldr, dtype) &&
                     wide_rows(sum, lds, dtype) && wide_rows(out, ldo, dtype) && aligned(weight, 16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t err = dtype == BT_F32 ? norm<float>(a, vec, s) : dtype == BT_BF16 ? norm<__nv_bfloat16>(a, vec, s) : norm<__half>(a, vec, s);
    return err == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

// The parts of gw, and the sums of rows that are wider than a CTA keeps.
size_t bt_rms_norm_backward_workspace(int64_t T, int64_t N) {
    if (T < 1 || N < 1 || T >= kMaxSide || N >= kMaxSide) return 0;
    // (the largest that any type needs)
    size_t most = 0;
    for (int elem = 2; elem <= 4; elem += 2) {
        const size_t n = (back_ring(N, elem) ? 0 : round_up256(static_cast<size_t>(T) * 16)) + static_cast<size_t>(back_chunks(T, N, elem)) * static_cast<size_t>(N) * 4;
        most = n > most ? n : most;
    }
    return round_up256(most);
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
    a.eps = eps_of(eps);
    a.gx = grad_x;
    a.rows = static_cast<float4 *>(workspace);
    const int elem = dtype_bytes(dtype);
    float *parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + (back_ring(N, elem) ? 0 : round_up256(static_cast<size_t>(T) * 16)));
    a.err = device_error_word();
    if (a.err == nullptr) return BT_ERR_CUDA;
    a.wait_ns = wait_limit_ns();
    a.parts = grad_weight == nullptr ? nullptr : parts;
    const bool vec = N % 8 == 0 && wide_rows(g, ldg, dtype) && wide_rows(h, ldh, dtype) && wide_rows(grad_sum, ldgs, dtype) &&
                     wide_rows(grad_x, ldgx, dtype) && aligned(weight, 16);
    cudaError_t err = dtype == BT_F32 ? backward<float>(a, vec, s) : dtype == BT_BF16 ? backward<__nv_bfloat16>(a, vec, s) : backward<__half>(a, vec, s);
    if (err == cudaSuccess && grad_weight != nullptr)
        err = launch_pdl(rms_back_join_kernel, dim3(static_cast<unsigned>((N + 31) / 32)), dim3(1024), s, static_cast<const float *>(parts),
                         back_chunks(T, N, elem), static_cast<int>(N), grad_weight);
    return err == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

}  // extern "C"
