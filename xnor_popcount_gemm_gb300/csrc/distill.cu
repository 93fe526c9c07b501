// Distillation from a teacher's top logits: for every row (token) the loss
//   a = z / tau                     the student's logits at the temperature
//   q_k                             the teacher's probabilities of the row's slots: softmax(t / tau)
//                                   over them, or exp(t / tau - teacher_lse) with what is left,
//                                   q_r = 1 - sum q, as one more outcome
//   lse = log sum_v exp a_v         r = log sum over the v outside the slots
//   loss = sum_k q_k (log q_k - a_k + lse)  [+ q_r (log q_r - r + lse)]
// and its gradient
//   d loss / d z_v = (exp(a_v - lse) - q_v) / tau                      v in a slot
//                  = exp(a_v - lse) / tau                              else, without the rest
//                  = (exp(r - lse) - q_r) exp(a_v - r) / tau           else, with it
// for a teacher whose probabilities sum to one. Where stored logits of fewer bits
// than teacher_lse sum to more, or the rest's term is left out since the student
// has no rest, the gradient stays this one, not the derivative of what is left.
// The slots' own logits are taken out of the running sum as the row is read,
// so that r comes from a sum of its own and not from a difference that cancels
// where the student is as sure as the teacher. Sums and statistics are fp32.
//
// Bound: HBM, with the issue slots close behind: a 16-bit logit of the step
// moves 4 bytes, 0.17 clocks of an SM's share of the memory; its two passes take
// ten instructions, 0.08 clocks, and two exp2, 0.12 clocks at 16 a clock.
//
// Measured, of the bytes that each must move: the step, 4096 x 131072 bf16, 396
// us, 5.2 TB/s (issue slots two thirds busy); 16 x 131072 f32 10.5 us; the loss
// alone, 512 x 50001 f32, 29 us, 3.2 TB/s (304 CTAs take one or two rows each: the
// second ones have the machine half to themselves), 8 x 32000 bf16 4.8 us; the
// backward, 2048 x 32000 bf16, 44 us, 5.4 TB/s, 300 x 50001 f16 10.9 us.
#include <cmath>
#include <type_traits>

#include "bt_device.cuh"
#include "bt_internal.h"
#include "tc_ptx.cuh"

namespace bt {
namespace {

constexpr int kMaxSlots = 1024;
constexpr int kMaxV = 1 << 28;
constexpr float kLog2e = 1.4426950408889634f;

// ex2.approx rounds down: its mean relative error is -5.0e-8 below the first
// octave, where a row's sum has its weight (measured on GB300 against exp2 in
// double: -4.86e-8 over [-16, 0], -2.2e-8 over [-1, 0]). Single errors average
// out in the sum, the mean does not and is taken out of it.
constexpr float kEx2Mean = 5.0e-8f;

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n"
        ".reg .b64 x, y, z, r;\n"
        "mov.b64 x, {%2, %3};\n"
        "mov.b64 y, {%4, %5};\n"
        "mov.b64 z, {%6, %7};\n"
        "fma.rn.f32x2 r, x, y, z;\n"
        "mov.b64 {%0, %1}, r;\n"
        "}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n"
        ".reg .b64 x, y, r;\n"
        "mov.b64 x, {%2, %3};\n"
        "mov.b64 y, {%4, %5};\n"
        "add.rn.f32x2 r, x, y;\n"
        "mov.b64 {%0, %1}, r;\n"
        "}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n"
        ".reg .b64 x, y, r;\n"
        "mov.b64 x, {%2, %3};\n"
        "mov.b64 y, {%4, %5};\n"
        "mul.rn.f32x2 r, x, y;\n"
        "mov.b64 {%0, %1}, r;\n"
        "}\n"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// A running maximum and the sum of 2^((v - m) c) relative to it. m starts far
// below any logit that is one: what lies lower, -inf and the values that masks
// are filled with, adds 0, and s = 0 says that there was nothing else.
constexpr float kMasked = -1.0e30f;
struct MaxSum {
    float m, s;
};
__device__ __forceinline__ MaxSum ms_empty() { return MaxSum{kMasked, 0.0f}; }
__device__ __forceinline__ void ms_add(MaxSum &a, float v, float c) {
    if (v > a.m) {
        a.s *= ex2((a.m - v) * c);
        a.m = v;
    }
    a.s += ex2((v - a.m) * c);
}
// The sum of n of them, which lie `stride` floats apart in shared memory,
// with what each addition rounds off carried along (Knuth's two-sum): these
// few additions would else make most of the sum's error. `mean`: take
// ex2.approx's mean error out.
__device__ __forceinline__ MaxSum ms_sum(const float *p, int n, int stride, float c, bool mean) {
    float m = p[0];
    for (int i = 1; i < n; ++i) m = fmaxf(m, p[i * stride]);
    float s = 0.0f, lost = 0.0f;
    for (int i = 0; i < n; ++i) {
        const float v = p[i * stride + 1] * ex2((p[i * stride] - m) * c);
        const float t = __fadd_rn(s, v), b = __fsub_rn(t, s);
        lost += __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(v, b));
        s = t;
    }
    if (mean) lost += s * kEx2Mean;
    return MaxSum{m, s + lost};
}
__device__ __forceinline__ MaxSum ms_join(const MaxSum &a, const MaxSum &b, float c) {
    const float m = fmaxf(a.m, b.m);
    return MaxSum{m, a.s * ex2((a.m - m) * c) + b.s * ex2((b.m - m) * c)};
}
// A warp's sum, relative to the largest `m`.
__device__ __forceinline__ MaxSum ms_warp(MaxSum a, float m, float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float s = a.s * ex2((a.m - m) * c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return MaxSum{m, s};
}

struct Args {
    const void *z;
    int V;
    int64_t ld;
    const void *ids;
    int ids_bytes;
    const void *top;
    int top_dt;
    int S;
    const float *tlse;         // NULL: the teacher's softmax over the slots
    float inv_tau, c;          // 1 / tau, log2(e) / tau
    float slack;               // a maximum this much below the true one is kept (2^16 at most in the sum)
    float *loss, *stats;
    const float *w;            // upstream gradient per row
    void *grad;
    int64_t ldg;
    int64_t rows;
    int cluster, shift;        // few rows: CTAs a row, 1 << shift
    int blocks;                // gradient alone: CTAs a row
    unsigned int *err;
    unsigned long long limit_ns;
};

__device__ __forceinline__ int slot_id(const Args &a, int64_t i) {
    const int64_t v = a.ids_bytes == 8 ? __ldg(static_cast<const long long *>(a.ids) + i)
                                       : static_cast<int64_t>(__ldg(static_cast<const int *>(a.ids) + i));
    return v >= 0 && v < a.V ? static_cast<int>(v) : -1;
}
__device__ __forceinline__ float slot_logit(const Args &a, int64_t i) {
    if (a.top_dt == BT_F32) return __ldg(static_cast<const float *>(a.top) + i);
    if (a.top_dt == BT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(a.top)[i]);
    return __half2float(static_cast<const __half *>(a.top)[i]);
}

// The teacher's side of a row: log q_k = (t_k - m) inv_tau - l, and q_r.
struct Teacher {
    float m, l, qr;
};
__device__ __forceinline__ float rest_of(float q) { return q < 1.0f ? 1.0f - q : (q >= 1.0f ? 0.0f : q); }   // a NaN stays one
// One warp; t and id in shared memory (id -1: an empty slot).
__device__ __forceinline__ Teacher teacher_of(const Args &a, const int *ids, const float *t, int64_t row, int lane) {
    Teacher r;
    if (a.tlse == nullptr) {
        MaxSum x{-INFINITY, 0.0f};                          // any finite logit counts, however low
        for (int k = lane; k < a.S; k += 32)
            if (ids[k] >= 0) ms_add(x, t[k], a.c);
        x = ms_warp(x, x.m, a.c);
        r = Teacher{x.m, logf(x.s), 0.0f};
    } else {
        r = Teacher{0.0f, __ldg(a.tlse + row), 0.0f};
        float q = 0.0f;
        for (int k = lane; k < a.S; k += 32)
            if (ids[k] >= 0) q += expf(t[k] * a.inv_tau - r.l);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
        r.qr = rest_of(q);
    }
    return r;
}
__device__ __forceinline__ float log_q(const Args &a, const Teacher &t, float v) {
    return (v - t.m) * a.inv_tau - t.l;
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T> __device__ __forceinline__ uint4 pack_vec(const float *f) {
    uint4 q;
    uint32_t *w = reinterpret_cast<uint32_t *>(&q);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
    return q;
}

// 16 bytes to an address of any element alignment.
template <typename T> __device__ __forceinline__ void store_vec(T *p, bool wide, const float *f) {
    constexpr int VEC = 16 / sizeof(T);
    if (wide) {
        st_stream_v4(p, pack_vec<T>(f));
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = from_f32<T>(f[e]);
    }
}

// How a row splits into 16-byte vectors: `head` elements before the first
// aligned address, nb vectors, the rest of the elements.
struct RowSplit {
    int head, nb, tail0;       // tail0: the first element after the vectors
};
template <typename T> __device__ __forceinline__ RowSplit split_row(const T *p, int V) {
    constexpr int VEC = 16 / sizeof(T);
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) / static_cast<int>(sizeof(T));
    const int head = min((VEC - mis) & (VEC - 1), V), nb = (V - head) / VEC;
    return RowSplit{head, nb, head + nb * VEC};
}

// The largest of a vector's elements.
template <typename T> __device__ __forceinline__ float max_of(const uint4 &q, const float *f) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
    } else {                                                // two at a time
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        const T2 *w = reinterpret_cast<const T2 *>(&q);
        const T2 m = __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3]));
        return fmaxf(Elem<T>::to_f32(m.x), Elem<T>::to_f32(m.y));
    }
}

// The running sum of one lane: 2^(f c - mc), mc being m c rounded; what that
// misses, less than 2^-4, comes back into the sum in the end. Where m c is so
// large that its rounding is an exponent of its own (`far`: a lane that has met
// nothing but masked values yet, or a row of huge ones) the sum is relative to m
// itself, 2^((f - m) c). `seen` is the largest logit so far, which m may trail by
// the slack.
constexpr float kNear = 1048576.0f;        // 2^20
struct Running {
    float m, mc, s, seen;
    bool far;
};
__device__ __forceinline__ bool is_far(float mc) { return !(fabsf(mc) <= kNear); }
__device__ __forceinline__ Running running_empty() { return Running{kMasked, 0.0f, 0.0f, kMasked, true}; }
__device__ __forceinline__ Running running_from(const MaxSum &x, float c) {
    const float mc = __fmul_rn(x.m, c);
    const bool far = is_far(mc);
    return Running{x.m, mc, far ? x.s : x.s * ex2(__fmaf_rn(x.m, c, -mc)), x.m, far};
}
// The sum relative to m itself.
__device__ __forceinline__ MaxSum running_sum(const Running &r, float c) {
    return MaxSum{r.m, r.far ? r.s : r.s * ex2(__fmaf_rn(-r.m, c, r.mc))};
}
// A larger reference.
__device__ __forceinline__ void running_move(Running &r, float m, float c) {
    const float mc = __fmul_rn(m, c);
    if (r.far || is_far(mc)) {
        MaxSum x = running_sum(r, c);
        x.s *= ex2((x.m - m) * c);
        x.m = m;
        const float seen = r.seen;
        r = running_from(x, c);
        r.seen = seen;
    } else {
        r.s *= ex2(r.mc - mc);
        r.m = m;
        r.mc = mc;
    }
}
template <typename T> __device__ __forceinline__ void running_add(Running &r, const uint4 &q, const Args &a) {
    constexpr int VEC = 16 / sizeof(T);
    float f[VEC];
    Elem<T>::unpack(q, f);
    const float mx = max_of<T>(q, f);
    r.seen = fmaxf(r.seen, mx);
    if (mx > r.m + a.slack) running_move(r, mx, a.c);
    if (r.far) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) r.s += ex2((f[e] - r.m) * a.c);
        return;
    }
    float2 sum;
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
        const float2 x = fma2(make_float2(f[e], f[e + 1]), make_float2(a.c, a.c), make_float2(-r.mc, -r.mc));
        const float2 p = make_float2(ex2(x.x), ex2(x.y));
        sum = e == 0 ? p : add2(sum, p);
    }
    r.s += sum.x + sum.y;
}
__device__ __forceinline__ MaxSum running_warp(const Running &r, float c) { return ms_warp(running_sum(r, c), r.seen, c); }

// The gradient outside the slots: coef * 2^(z c1 - shift), or, where the
// rounding of shift would be an exponent of its own (`far`, as above), coef *
// 2^((z k1 - base) k2), c1 = k1 k2. base is a largest logit, or the log sum of
// logits that it cannot tell from the largest: no such exponent is above 0 (in a
// slot, which is written over, it may be).
struct Slope {
    float coef, c1, shift;
    bool far;
    float k1, base, k2;
};
__device__ __forceinline__ Slope slope_make(float coef, float c1, float k1, float base, float k2) {
    const float shift = __fmul_rn(base, k2);                // the factor takes what the rounding misses
    const bool far = is_far(shift);
    return Slope{far ? coef : coef * ex2(__fmaf_rn(-base, k2, shift)), c1, shift, far, k1, base, k2};
}
__device__ __forceinline__ float not_above_0(float x) { return x > 0.0f ? 0.0f : x; }   // a NaN stays one
// Nothing: 0 wherever the logits are masked.
__device__ __forceinline__ Slope slope_none(float c1) { return Slope{0.0f, c1, 0.0f, false, 0.0f, 0.0f, 0.0f}; }
// (not far)
template <typename T> __device__ __forceinline__ void slope_vec(const Slope &g, const uint4 &q, float *f) {
    constexpr int VEC = 16 / sizeof(T);
    Elem<T>::unpack(q, f);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
        const float2 x = fma2(make_float2(f[e], f[e + 1]), make_float2(g.c1, g.c1), make_float2(-g.shift, -g.shift));
        const float2 p = mul2(make_float2(ex2(x.x), ex2(x.y)), make_float2(g.coef, g.coef));
        f[e] = p.x;
        f[e + 1] = p.y;
    }
}
__device__ __forceinline__ float slope_of(const Slope &g, float v) {
    return g.coef * ex2(g.far ? not_above_0(__fmul_rn(v, g.k1) - g.base) * g.k2 : __fmaf_rn(v, g.c1, -g.shift));
}
template <typename T> __device__ __forceinline__ void slope_any(const Slope &g, const uint4 &q, float *f) {
    if (g.far) {
        Elem<T>::unpack(q, f);
#pragma unroll
        for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) f[e] = slope_of(g, f[e]);
    } else {
        slope_vec<T>(g, q, f);
    }
}

// Both from a row's sums: over the slots, outside them, over all.
__device__ __forceinline__ Slope slope_from(const Args &a, const Teacher &te, float w, const MaxSum &rest, const MaxSum &all) {
    const bool other = a.tlse != nullptr;
    if (other ? rest.s == 0.0f : all.s == 0.0f) return slope_none(a.c);
    if (!other) return slope_make(w / all.s, a.c, 1.0f, all.m, a.c);
    const float pr = rest.s * ex2((rest.m - all.m) * a.c) / all.s;
    return slope_make(w * (pr - te.qr) / rest.s, a.c, 1.0f, rest.m, a.c);
}

// One warp: the loss of a row, with the student's logits of the slots in zt.
// Where lse and r are below 16 it is taken from them as they are returned and as
// the backward reads them: fp32 log probabilities, rounded by up to 5e-7. Larger
// ones would be rounded by more (logits with a common offset of 4096: 2e-4,
// beside losses of 1e-3), so that they are taken relative to the row's largest
// logit then: the loss of a row does not depend on what all its logits share.
__device__ __forceinline__ void write_loss(const Args &a, int64_t row, const int *ids, const float *tt, const float *zt,
                                           const Teacher &te, const MaxSum &rest, const MaxSum &all, int lane) {
    const bool empty = all.s == 0.0f;                       // the student has nothing left
    // (rounded as the backward rounds z / tau: of a huge row lse is its largest)
    const float lse = empty ? -INFINITY : __fadd_rn(__fmul_rn(all.m, a.inv_tau), logf(all.s));
    const float r = rest.s == 0.0f ? -INFINITY : __fadd_rn(__fmul_rn(rest.m, a.inv_tau), logf(rest.s));
    const bool small = fmaxf(fabsf(lse), fabsf(r)) < 16.0f;
    const float ref = small ? 0.0f : all.m, lse0 = small ? lse : logf(all.s);
    float l = 0.0f;
    for (int k = lane; k < a.S; k += 32) {
        if (ids[k] < 0) continue;
        const float q = expf(log_q(a, te, tt[k]));
        if (!(q == 0.0f)) l += q * (logf(q) - ((zt[k] - ref) * a.inv_tau - lse0));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    if (lane == 0) {
        const float r0 = small ? r : (rest.m - ref) * a.inv_tau + logf(rest.s);
        if (a.tlse != nullptr && rest.s != 0.0f && !(te.qr == 0.0f)) l += te.qr * (logf(te.qr) - (r0 - lse0));
        a.loss[row] = empty ? 0.0f : l;
        if (a.stats != nullptr) {
            a.stats[2 * row] = lse;
            a.stats[2 * row + 1] = r;
        }
    }
}

// A wait for copies in flight: if it gives up (which it records), it still
// lets them land before the CTA's memory is given back.
__device__ __forceinline__ void wait_landed(uint32_t bar, uint32_t parity, uint32_t *abort_flag, const Args &a) {
    if (!tc::wait_fast(bar, parity, abort_flag, a.err, a.limit_ns)) {
        uint32_t drain = 0;
        tc::wait_bounded(bar, parity, &drain, a.err);
    }
}

// ---------------------------------------------------------------------------
// Many rows: a CTA a row. The row streams through a ring of 2 KB chunks in
// shared memory, every warp with a ring and chunks of its own (chunk j belongs
// to warp j mod 12), first for the sums, then, for the gradient, once more out
// of the L2 cache, which holds the rows at work (304 of 256 KB are 78 MB). The
// ring runs on over the join between the two passes and into the next row, so
// that the copies never pause; two CTAs an SM take turns with arithmetic. A
// cluster that holds the row in its CTAs' shared memory, read once, was slower
// (4096 x 131072 bf16: 505 us, 570 with the next row's prefetch, against 396):
// its per-row joins idle more of the machine than the second read costs.
// ---------------------------------------------------------------------------
constexpr int kStreamWarps = 12, kStreamThreads = 32 * kStreamWarps;
constexpr int kChunkVecs = 128, kRing = 4;                  // 2 KB

template <typename T, bool STEP>
__global__ void __launch_bounds__(kStreamThreads, 2) distill_stream_kernel(const Args a) {
    constexpr int VEC = 16 / sizeof(T), NW = kStreamWarps, KT = (kMaxSlots + kStreamThreads - 1) / kStreamThreads;
    constexpr int kChunkElems = kChunkVecs * VEC;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ alignas(8) uint64_t bars[NW][kRing];
    __shared__ float4 red[NW];
    __shared__ T edge[32];
    __shared__ Teacher teacher;
    __shared__ uint32_t abort_flag, live_slots[4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *ring = smem + warp * kRing * kChunkVecs * 16;
    int *ids_all = reinterpret_cast<int *>(smem + NW * kRing * kChunkVecs * 16);     // of four units
    float *tt_all = reinterpret_cast<float *>(ids_all + 4 * a.S), *zt = tt_all + 4 * a.S;
    uint16_t *list = reinterpret_cast<uint16_t *>(zt + a.S) + warp * a.S;            // this warp's slots

    pdl_launch_dependents();
    if (tid < NW * kRing) {
        tc::mbar_init(smem_u32(&bars[tid / kRing][tid % kRing]), 1);
        tc::fence_mbar_init();
    }
    if (tid < 4) live_slots[tid] = 0;
    if (tid == 0) abort_flag = 0;
    pdl_wait();
    __syncthreads();

    int kid[KT];
    float kt[KT];
    auto fetch_ids = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int k = tid + i * kStreamThreads;
            kid[i] = -1;
            if (k < a.S && row < a.rows) {
                kid[i] = slot_id(a, row * a.S + k);
                kt[i] = slot_logit(a, row * a.S + k);
            }
        }
    };
    auto store_ids = [&](int at) {
        uint32_t some = 0;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int k = tid + i * kStreamThreads;
            if (k < a.S) {
                const int id = kt[i] == -INFINITY ? -1 : kid[i];
                ids_all[at * a.S + k] = id;
                tt_all[at * a.S + k] = kt[i];
                some += id >= 0;
            }
        }
        some = __reduce_add_sync(0xFFFFFFFFu, some);
        if (some != 0 && lane == 0) atomicAdd(&live_slots[at], some);
    };
    // A row's chunks: this warp takes the warp-th, the (warp + 12)-th, ...
    struct Row {
        const T *z;
        RowSplit sp;
        int mine;
    };
    auto row_of = [&](int64_t row) {
        Row x;
        x.z = static_cast<const T *>(a.z) + row * a.ld;
        x.sp = split_row(x.z, a.V);
        const int left = (x.sp.nb + kChunkVecs - 1) / kChunkVecs - warp;
        x.mine = left > 0 ? (left + NW - 1) / NW : 0;
        return x;
    };
    uint32_t issued = 0, used = 0;                          // chunks, over all rows
    auto issue = [&](const Row &x, int i, bool last) {      // its i-th chunk of this warp
        if (lane == 0) {
            const int b = (warp + i * NW) * kChunkVecs;
            const uint32_t n = static_cast<uint32_t>(min(kChunkVecs, x.sp.nb - b)) * 16u, at = issued % kRing;
            const uint32_t bar = smem_u32(&bars[warp][at]), dst = smem_u32(ring + at * kChunkVecs * 16);
            const T *src = x.z + x.sp.head + static_cast<int64_t>(b) * VEC;
            tc::mbar_arrive_expect_tx(bar, n);
            if (last) tc::bulk_load_once(dst, src, n, bar);
            else tc::bulk_load(dst, src, n, bar);
        }
        ++issued;
    };

    const int64_t step = gridDim.x;
    int64_t row = blockIdx.x;
    fetch_ids(row);
    store_ids(0);
    fetch_ids(row + step);
    store_ids(1);
    __syncthreads();
    Row cur = row_of(row);
    constexpr int kPasses = STEP ? 2 : 1;
    int sent = 0;                                           // chunks of this row (and the next) asked for
    for (int it = 0; row < a.rows; row += step, ++it) {
        const bool live = live_slots[it & 3] != 0;
        const bool next_live = row + step < a.rows && live_slots[(it + 1) & 3] != 0;
        const Row nxt = row_of(row + step < a.rows ? row + step : row);
        const int total = live ? kPasses * cur.mine : 0, ahead = total + (next_live ? kPasses * nxt.mine : 0);
        // one more chunk into the ring, as far as the next row's
        auto feed = [&]() {
            if (sent >= ahead) return;
            const bool of_next = sent >= total;
            int i = of_next ? sent - total : sent;
            const int mine = of_next ? nxt.mine : cur.mine;
            const bool again = kPasses == 2 && i >= mine;
            if (again) i -= mine;
            issue(of_next ? nxt : cur, i, again);
            ++sent;
        };
        while (sent < ahead && issued - used < kRing) feed();
        const int *ids = ids_all + (it & 3) * a.S;
        const float *tt = tt_all + (it & 3) * a.S;
        const int nhead = cur.sp.head, ntail = a.V - cur.sp.tail0;
        const bool edges = warp == 0;
        T *grad = STEP ? static_cast<T *>(a.grad) + row * a.ldg : nullptr;
        const bool wide = STEP && ((reinterpret_cast<uintptr_t>(grad) ^ reinterpret_cast<uintptr_t>(cur.z)) & 15) == 0;
        T ez = from_f32<T>(-INFINITY);
        if (edges && live) {
            if (lane < nhead) ez = cur.z[lane];
            else if (lane >= 16 && lane - 16 < ntail) ez = cur.z[cur.sp.tail0 + lane - 16];
        }
        fetch_ids(row + 2 * step);

        // this warp's slots: those in its chunks, and warp 0's outside the vectors
        int count = 0;
        if (live) {
            for (int k0 = 0; k0 < a.S; k0 += 32) {
                const int k = k0 + lane, id = k < a.S ? ids[k] : -1, e = id - nhead;
                bool my = false;
                if (id >= 0) {
                    if (e < 0 || id >= cur.sp.tail0) my = edges;
                    else my = (e / kChunkElems) % NW == warp;
                }
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, my);
                if (my) list[count + __popc(who & ((1u << lane) - 1u))] = static_cast<uint16_t>(k);
                count += __popc(who);
            }
            __syncwarp();
        }
        // lane l holds the l-th of them: its place as an element of the vectors (< 0: outside)
        int my_e = -1, my_k = 0;
        if (lane < count) {
            my_k = list[lane];
            const int id = ids[my_k];
            my_e = id >= nhead && id < cur.sp.tail0 ? id - nhead : -1;
        }
        auto place = [&](int l, int &k) {                   // of the l-th, l >= 32
            k = list[l];
            const int id = ids[k];
            return id >= nhead && id < cur.sp.tail0 ? id - nhead : -1;
        };

        MaxSum rest = ms_empty(), top = ms_empty(), all = ms_empty();
        Teacher te = {};
        if (live) {
            if (warp == NW - 1) {
                const Teacher t = teacher_of(a, ids, tt, row, lane);
                if (lane == 0) teacher = t;
            }
            if (edges) edge[lane] = ez;
            {
                auto take = [&](int k, T *p) {              // take slot k's logit out of the row
                    const float v = Elem<T>::to_f32(*p);
                    *p = from_f32<T>(-INFINITY);
                    zt[k] = v;
                    ms_add(top, v, a.c);
                };
                Running run = running_empty();
                if (edges) {
                    __syncwarp();
                    for (int l = lane; l < count; l += 32) {
                        int k = my_k;
                        if ((l < 32 ? my_e : place(l, k)) >= 0) continue;
                        const int id = ids[k];
                        take(k, &edge[id < nhead ? id : 16 + id - cur.sp.tail0]);
                    }
                    __syncwarp();
                    MaxSum one = ms_empty();
                    ms_add(one, Elem<T>::to_f32(edge[lane]), a.c);
                    run = running_from(one, a.c);
                }
                for (int i = 0; i < cur.mine; ++i) {
                    const uint32_t at = used % kRing;
                    wait_landed(smem_u32(&bars[warp][at]), (used / kRing) & 1u, &abort_flag, a);
                    const int j = warp + i * NW, n = min(kChunkVecs, cur.sp.nb - j * kChunkVecs);
                    T *p = reinterpret_cast<T *>(ring + at * kChunkVecs * 16);
                    if (my_e >= 0 && my_e / kChunkElems == j) take(my_k, p + (my_e & (kChunkElems - 1)));
                    for (int l = lane + 32; l < count; l += 32) {
                        int k;
                        const int e = place(l, k);
                        if (e >= 0 && e / kChunkElems == j) take(k, p + (e & (kChunkElems - 1)));
                    }
                    __syncwarp();
                    const uint4 *q = reinterpret_cast<const uint4 *>(p);
                    if (n == kChunkVecs) {
#pragma unroll
                        for (int u = 0; u < kChunkVecs / 32; ++u) running_add<T>(run, q[lane + 32 * u], a);
                    } else {
                        for (int v = lane; v < n; v += 32) running_add<T>(run, q[v], a);
                    }
                    tc::fence_proxy_async_smem();           // the slot's values were overwritten through this proxy
                    __syncwarp();
                    ++used;
                    feed();
                }
                rest = running_warp(run, a.c);
                top = ms_warp(top, top.m, a.c);
                if (lane == 0) red[warp] = make_float4(rest.m, rest.s, top.m, top.s);
            }
        }
        store_ids((it + 2) & 3);
        if (tid == 0) live_slots[(it + 3) & 3] = 0;
        __syncthreads();
        if (live) {
            te = teacher;
            // even lanes the sum outside the slots, odd ones that of the slots
            const MaxSum mine = ms_sum(&red[0].x + 2 * (lane & 1), NW, 4, a.c, true);
            rest = MaxSum{__shfl_sync(0xFFFFFFFFu, mine.m, 0), __shfl_sync(0xFFFFFFFFu, mine.s, 0)};
            top = MaxSum{__shfl_sync(0xFFFFFFFFu, mine.m, 1), __shfl_sync(0xFFFFFFFFu, mine.s, 1)};
            all = ms_join(rest, top, a.c);
            if (warp == (it % NW)) write_loss(a, row, ids, tt, zt, te, rest, all, lane);
            if constexpr (STEP) {
                const float w = __ldg(a.w + row) * a.inv_tau;
                const Slope slope = slope_from(a, te, w, rest, all);
                for (int i = 0; i < cur.mine; ++i) {
                    const uint32_t at = used % kRing;
                    wait_landed(smem_u32(&bars[warp][at]), (used / kRing) & 1u, &abort_flag, a);
                    const int j = warp + i * NW, n = min(kChunkVecs, cur.sp.nb - j * kChunkVecs);
                    const uint4 *q = reinterpret_cast<const uint4 *>(ring + at * kChunkVecs * 16);
                    T *out = grad + nhead + static_cast<int64_t>(j) * kChunkElems;
                    if (n == kChunkVecs && wide && !slope.far) {
#pragma unroll
                        for (int u = 0; u < kChunkVecs / 32; ++u) {
                            float f[VEC];
                            slope_vec<T>(slope, q[lane + 32 * u], f);
                            st_stream_v4(out + (lane + 32 * u) * VEC, pack_vec<T>(f));
                        }
                    } else {
                        for (int v = lane; v < n; v += 32) {
                            float f[VEC];
                            slope_any<T>(slope, q[v], f);
                            store_vec<T>(out + v * VEC, wide, f);
                        }
                    }
                    __syncwarp();
                    ++used;
                    feed();
                }
                if (edges) {
                    const float f = slope_of(slope, Elem<T>::to_f32(edge[lane]));
                    if (lane < nhead) grad[lane] = from_f32<T>(f);
                    else if (lane >= 16 && lane - 16 < ntail) grad[cur.sp.tail0 + lane - 16] = from_f32<T>(f);
                }
                __syncwarp();
                // the slots, over what was just written there
                for (int l = lane; l < count; l += 32) {
                    const int k = l < 32 ? my_k : list[l];
                    const float p = ex2((zt[k] - all.m) * a.c) / all.s;
                    grad[ids[k]] = from_f32<T>(all.s == 0.0f ? 0.0f : w * (p - expf(log_q(a, te, tt[k]))));
                }
            }
        } else {                                            // padding
            if (tid == 0) {
                a.loss[row] = 0.0f;
                if (a.stats != nullptr) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
            }
            if constexpr (STEP) {
                const float zero[VEC] = {};
                for (int v = tid; v < cur.sp.nb; v += kStreamThreads) store_vec<T>(grad + nhead + v * VEC, wide, zero);
                if (edges) {
                    if (lane < nhead) grad[lane] = from_f32<T>(0.0f);
                    else if (lane >= 16 && lane - 16 < ntail) grad[cur.sp.tail0 + lane - 16] = from_f32<T>(0.0f);
                }
            }
        }
        // red, zt, teacher and edge are this row's until every warp is here
        __syncthreads();
        sent -= total;
        cur = nxt;
    }
}

// ---------------------------------------------------------------------------
// Few rows: a cluster of 1 to 8 CTAs a row, which it holds in its shared memory,
// so that the whole machine works on the rows and the logits are read once.
// Every warp fetches its piece with bulk copies of 4 KB and sums them as they
// land; the sums are joined in the CTA, then across the cluster through
// distributed shared memory, and the gradient is computed from shared memory.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256, kRowWarps = 8;
constexpr int kMaxCluster = 8;             // portable cluster size
constexpr int kPieceBytes = 4096;          // one bulk copy
constexpr int kMaxPieces = 6;              // of a warp
constexpr int kSliceMax = kRowWarps * (kMaxPieces - 1) * kPieceBytes;   // bytes of a row that one CTA holds

template <typename T, bool STEP>
__global__ void __launch_bounds__(kRowThreads) distill_rows_kernel(const Args a) {
    constexpr int VEC = 16 / sizeof(T);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ alignas(8) uint64_t bars[kRowWarps][kMaxPieces];
    __shared__ float4 red[kRowWarps], slot[kMaxCluster];
    __shared__ T edge[32];
    __shared__ Teacher teacher;
    __shared__ uint32_t abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = a.cluster;
    const int rank = c > 1 ? static_cast<int>(tc::cluster_ctarank()) : 0;
    const int64_t row = blockIdx.x >> a.shift;

    pdl_launch_dependents();
    if (lane == 0) {
        for (int j = 0; j < kMaxPieces; ++j) tc::mbar_init(smem_u32(&bars[warp][j]), 1);
        tc::fence_mbar_init();
    }
    if (tid == 0) abort_flag = 0;
    pdl_wait();

    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    const RowSplit sp = split_row(z, a.V);
    const int v0 = (sp.nb * rank) >> a.shift, v1 = (sp.nb * (rank + 1)) >> a.shift;             // this CTA's vectors
    const int w0 = v0 + (((v1 - v0) * warp) >> 3), w1 = v0 + (((v1 - v0) * (warp + 1)) >> 3);    // this warp's
    T *data = reinterpret_cast<T *>(smem);                                                       // vector v at (v - v0) * VEC
    const size_t data_bytes = static_cast<size_t>((sp.nb + c - 1) >> a.shift) * 16;
    float *zt = reinterpret_cast<float *>(smem + data_bytes);                                    // the student's logits of the slots
    float *tt = zt + a.S;                                                                        // the teacher's
    int *ids = reinterpret_cast<int *>(tt + a.S);

    int any = 0;
    for (int k = tid; k < a.S; k += kRowThreads) {
        int id = slot_id(a, row * a.S + k);
        const float t = slot_logit(a, row * a.S + k);
        if (t == -INFINITY) id = -1;
        ids[k] = id;
        tt[k] = t;
        any |= id >= 0;
    }
    constexpr int kPieceVecs = kPieceBytes / 16;
    const int pieces = (w1 - w0 + kPieceVecs - 1) / kPieceVecs;
    // few rows: asked for before the slots say whether the row is needed
    if (lane == 0) {
        for (int j = 0; j < pieces; ++j) {
            const int b = w0 + j * kPieceVecs;
            const uint32_t n = static_cast<uint32_t>(min(kPieceVecs, w1 - b)) * 16u, bar = smem_u32(&bars[warp][j]);
            tc::mbar_arrive_expect_tx(bar, n);
            tc::bulk_load(smem_u32(data + (b - v0) * VEC), z + sp.head + b * VEC, n, bar);
        }
    }
    const bool edges = rank == 0 && warp == 0;              // the elements outside the vectors
    const int nhead = sp.head, ntail = a.V - sp.tail0;
    if (edges) {
        T v = from_f32<T>(-INFINITY);
        if (lane < nhead) v = z[lane];
        else if (lane >= 16 && lane - 16 < ntail) v = z[sp.tail0 + lane - 16];
        edge[lane] = v;
    }
    const bool live = __syncthreads_or(any) != 0;
    T *grad = STEP ? static_cast<T *>(a.grad) + row * a.ldg : nullptr;
    const bool wide = STEP && ((reinterpret_cast<uintptr_t>(grad) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    if (!live) {                                            // padding: the same for the whole cluster
        for (int j = 0; j < pieces; ++j) wait_landed(smem_u32(&bars[warp][j]), 0, &abort_flag, a);
        if (rank == 0 && tid == 0) {
            a.loss[row] = 0.0f;
            if (a.stats != nullptr) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
        }
        if constexpr (STEP) {
            const float zero[VEC] = {};
            for (int v = w0 + lane; v < w1; v += 32) store_vec<T>(grad + sp.head + v * VEC, wide, zero);
            if (edges) {
                if (lane < nhead) grad[lane] = from_f32<T>(0.0f);
                else if (lane >= 16 && lane - 16 < ntail) grad[sp.tail0 + lane - 16] = from_f32<T>(0.0f);
            }
        }
        return;
    }
    if (warp == kRowWarps - 1) {
        const Teacher t = teacher_of(a, ids, tt, row, lane);
        if (lane == 0) teacher = t;
    }
    MaxSum top = ms_empty();
    Running run = running_empty();
    const uint32_t zt_rank0 = c > 1 ? tc::mapa(smem_u32(zt), 0) : 0u;
    auto take = [&](int k, T *p) {                          // take slot k's logit out of the row
        const float v = Elem<T>::to_f32(*p);
        *p = from_f32<T>(-INFINITY);
        zt[k] = v;
        if (rank != 0) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(zt_rank0 + 4u * k), "f"(v) : "memory");
        ms_add(top, v, a.c);
    };
    if (c > 1) tc::cluster_sync();                          // the cluster's CTAs have all started
    if (edges) {
        for (int k = lane; k < a.S; k += 32) {
            const int id = ids[k];
            if (id >= 0 && id < nhead) take(k, &edge[id]);
            else if (id >= sp.tail0) take(k, &edge[16 + id - sp.tail0]);
        }
        __syncwarp();
        MaxSum one = ms_empty();
        ms_add(one, Elem<T>::to_f32(edge[lane]), a.c);
        run = running_from(one, a.c);
    }
    for (int j = 0; j < pieces; ++j) {
        wait_landed(smem_u32(&bars[warp][j]), 0, &abort_flag, a);
        const int b = w0 + j * kPieceVecs, n = min(kPieceVecs, w1 - b), first = sp.head + b * VEC;
        T *p = data + (b - v0) * VEC;
        for (int k = lane; k < a.S; k += 32) {
            const unsigned off = static_cast<unsigned>(ids[k]) - static_cast<unsigned>(first);
            if (ids[k] >= 0 && off < static_cast<unsigned>(n * VEC)) take(k, p + off);
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32) running_add<T>(run, reinterpret_cast<const uint4 *>(p)[i], a);
    }
    MaxSum rest = running_warp(run, a.c);
    top = ms_warp(top, top.m, a.c);
    if (lane == 0) red[warp] = make_float4(rest.m, rest.s, top.m, top.s);
    __syncthreads();
    if (warp == 0) {
        rest = ms_sum(&red[0].x, kRowWarps, 4, a.c, false);
        top = ms_sum(&red[0].z, kRowWarps, 4, a.c, false);
        if (c == 1) {
            if (lane == 0) slot[0] = make_float4(rest.m, rest.s, top.m, top.s);
        } else if (lane < c) {
            const uint32_t dst = tc::mapa(smem_u32(&slot[rank]), lane);
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(rest.m), "f"(rest.s),
                         "f"(top.m), "f"(top.s)
                         : "memory");
        }
    }
    if (c > 1) tc::cluster_sync();
    else __syncthreads();
    rest = ms_sum(&slot[0].x, c, 4, a.c, true);
    top = ms_sum(&slot[0].z, c, 4, a.c, true);
    const MaxSum all = ms_join(rest, top, a.c);
    const Teacher te = teacher;
    if (rank == 0 && warp == kRowWarps - 1) write_loss(a, row, ids, tt, zt, te, rest, all, lane);
    if constexpr (STEP) {
        const float w = __ldg(a.w + row) * a.inv_tau;
        const Slope slope = slope_from(a, te, w, rest, all);
        auto write = [&](auto values) {
            for (int v = w0 + lane; v < w1; v += 32) {
                float f[VEC];
                values(reinterpret_cast<const uint4 *>(data)[v - v0], f);
                store_vec<T>(grad + sp.head + v * VEC, wide, f);
            }
        };
        if (!slope.far) write([&](const uint4 &q, float *f) { slope_vec<T>(slope, q, f); });
        else write([&](const uint4 &q, float *f) { slope_any<T>(slope, q, f); });
        if (edges) {
            const float f = slope_of(slope, Elem<T>::to_f32(edge[lane]));
            if (lane < nhead) grad[lane] = from_f32<T>(f);
            else if (lane >= 16 && lane - 16 < ntail) grad[sp.tail0 + lane - 16] = from_f32<T>(f);
        }
        __syncwarp();
        // the slots of this warp's piece, over what was just written there
        const int lo = sp.head + w0 * VEC, hi = sp.head + w1 * VEC;
        for (int k = lane; k < a.S; k += 32) {
            const int id = ids[k];
            if (id < 0) continue;
            if ((id >= lo && id < hi) || (edges && (id < nhead || id >= sp.tail0))) {
                const float p = ex2((zt[k] - all.m) * a.c) / all.s;
                grad[id] = from_f32<T>(all.s == 0.0f ? 0.0f : w * (p - expf(log_q(a, te, tt[k]))));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The gradient from a forward's statistics. A CTA takes 2048 vectors of a row
// (32 KB in, 32 KB out), all asked for at once; meanwhile it works out the
// teacher's side and reads the slots' logits, before anything is written, so
// that the gradient may take the logits' place. (A warp of its own for every
// 4 KB, which waits for no other, took 46 us for 2048 x 32000 bf16 against 44:
// every warp then goes through the slots. One warp alone at the slots: 49 us.)
// ---------------------------------------------------------------------------
constexpr int kBackThreads = 256, kBackLoads = 8;
constexpr int kBackBlockVecs = kBackThreads * kBackLoads;

template <typename T>
__global__ void __launch_bounds__(kBackThreads, 4) distill_backward_kernel(const Args a) {
    constexpr int VEC = 16 / sizeof(T);
    extern __shared__ float slots_s[];
    float *zt = slots_s, *tt = zt + a.S;                    // of the slots in this piece
    int *ids = reinterpret_cast<int *>(tt + a.S);
    __shared__ Teacher teacher;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t row32 = blockIdx.x / static_cast<uint32_t>(a.blocks);
    const int piece = static_cast<int>(blockIdx.x - row32 * a.blocks);
    const int64_t row = row32;
    pdl_launch_dependents();
    pdl_wait();
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    T *grad = static_cast<T *>(a.grad) + row * a.ldg;
    const bool wide = ((reinterpret_cast<uintptr_t>(grad) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    const RowSplit sp = split_row(z, a.V);
    const int v0 = piece * kBackBlockVecs, n = max(0, min(kBackBlockVecs, sp.nb - v0));
    // its vectors' elements, and with the first piece the ones outside all vectors
    const int lo = sp.head + v0 * VEC, hi = lo + n * VEC, nhead = sp.head, ntail = a.V - sp.tail0;
    const bool edges = piece == 0;
    auto mine = [&](int id) { return id >= 0 && ((id >= lo && id < hi) || (edges && (id < nhead || id >= sp.tail0))); };
    uint4 q[kBackLoads];
#pragma unroll
    for (int i = 0; i < kBackLoads; ++i)
        if (tid + kBackThreads * i < n) q[i] = ld_stream_v4(z + lo + (tid + kBackThreads * i) * VEC);
    float ez = -INFINITY;
    const float lse = __ldg(a.stats + 2 * row), r = __ldg(a.stats + 2 * row + 1);
    const float w = __ldg(a.w + row) * a.inv_tau;
    int any = 0;
    for (int k = tid; k < a.S; k += kBackThreads) {
        int id = slot_id(a, row * a.S + k);
        const float t = slot_logit(a, row * a.S + k);
        if (t == -INFINITY) id = -1;
        any |= id >= 0;
        ids[k] = id;
        tt[k] = t;
        if (mine(id)) zt[k] = Elem<T>::to_f32(z[id]);
    }
    if (edges && warp == 0) {
        if (lane < nhead) ez = Elem<T>::to_f32(z[lane]);
        else if (lane >= 16 && lane - 16 < ntail) ez = Elem<T>::to_f32(z[sp.tail0 + lane - 16]);
    }
    const bool alive = __syncthreads_or(any) != 0;
    if (warp == 0) {
        const Teacher t = teacher_of(a, ids, tt, row, lane);
        if (lane == 0) teacher = t;
    }
    __syncthreads();
    const Teacher te = teacher;
    const bool dead = !alive || lse == -INFINITY;
    // exp(z / tau - base) as 2^(z c - base log2 e)
    const bool other = a.tlse != nullptr, none = dead || (other && r == -INFINITY);
    const Slope slope = none ? slope_none(a.c)
                             : slope_make(other ? w * (expf(r - lse) - te.qr) : w, a.c, a.inv_tau, other ? r : lse, kLog2e);
#pragma unroll
    for (int i = 0; i < kBackLoads; ++i) {
        const int v = tid + kBackThreads * i;
        if (v >= n) continue;
        float f[VEC];
        slope_any<T>(slope, q[i], f);
        if (dead) {                                         // whatever the row holds
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = 0.0f;
        }
        store_vec<T>(grad + lo + v * VEC, wide, f);
    }
    if (edges && warp == 0) {
        const T f = from_f32<T>(dead ? 0.0f : slope_of(slope, ez));
        if (lane < nhead) grad[lane] = f;
        else if (lane >= 16 && lane - 16 < ntail) grad[sp.tail0 + lane - 16] = f;
    }
    __syncthreads();
    if (dead) return;
    // the slots, over what was just written there
    for (int k = tid; k < a.S; k += kBackThreads) {
        const int id = ids[k];
        if (!mine(id)) continue;
        const float p = expf(slope.far ? not_above_0(__fmul_rn(zt[k], a.inv_tau) - lse) : __fmaf_rn(zt[k], a.inv_tau, -lse));
        grad[id] = from_f32<T>(w * (p - expf(log_q(a, te, tt[k]))));
    }
}

int elem_bytes(bt_dtype t) { return t == BT_F32 ? 4 : 2; }
bool float_type(int t) { return t == BT_F32 || t == BT_BF16 || t == BT_F16; }

template <typename T, bool STEP> cudaError_t launch_stream(const Args &a, cudaStream_t s) {
    auto kern = distill_stream_kernel<T, STEP>;
    const auto smem = [](int S) { return kStreamWarps * kRing * kChunkVecs * 16 + S * (9 * 4 + 2 * kStreamWarps); };
    static ContextOnce once;
    if (const cudaError_t err = allow_smem(kern, smem(kMaxSlots), once); err != cudaSuccess) return err;
    const int64_t slots = 2 * device_sm_count();
    return launch_pdl_smem(kern, dim3(static_cast<unsigned>(a.rows < slots ? a.rows : slots)), dim3(kStreamThreads),
                           static_cast<size_t>(smem(a.S)), s, a);
}
template <typename T> cudaError_t launch_backward(Args a, cudaStream_t s) {
    constexpr int VEC = 16 / sizeof(T);
    a.blocks = (a.V / VEC + kBackBlockVecs - 1) / kBackBlockVecs;
    if (a.blocks < 1) a.blocks = 1;
    return launch_pdl_smem(distill_backward_kernel<T>, dim3(static_cast<unsigned>(a.rows * a.blocks)), dim3(kBackThreads),
                           3 * sizeof(float) * static_cast<size_t>(a.S), s, static_cast<const Args>(a));
}

// CTAs a row: doubled while the rows' CTAs fill less than half the machine and a
// CTA keeps at least 4 KB; 0 where one would have to hold more than fits.
int rows_cluster(int64_t rows, int64_t row_bytes, int sms) {
    int c = 1;
    while (c < kMaxCluster && rows * c * 2 <= sms && row_bytes >= static_cast<int64_t>(c) * 8192) c *= 2;
    return row_bytes <= static_cast<int64_t>(c) * kSliceMax ? c : 0;
}

template <typename T, bool STEP> cudaError_t launch_rows(Args a, cudaStream_t s) {
    auto kern = distill_rows_kernel<T, STEP>;
    static ContextOnce once;
    if (const cudaError_t err = allow_smem(kern, kSliceMax + 16 + 12 * kMaxSlots, once); err != cudaSuccess) return err;
    a.shift = 0;
    while ((1 << a.shift) < a.cluster) ++a.shift;
    const int64_t bytes = a.V * static_cast<int64_t>(sizeof(T));
    const int64_t slice = (bytes / 16 + a.cluster - 1) / a.cluster * 16;      // the most any alignment needs
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * a.cluster));
    cfg.blockDim = dim3(kRowThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(slice) + 12u * static_cast<size_t>(a.S);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const Args>(a));
}

enum class Pass { kLoss, kStep, kBackward };

template <typename T> cudaError_t launch(Pass pass, Args a, cudaStream_t s) {
    if (pass == Pass::kBackward) return launch_backward<T>(a, s);
    const int sms = device_sm_count();
    // Up to half a machine of rows a cluster each; more go one to a CTA.
    a.cluster = 2 * a.rows <= sms ? rows_cluster(a.rows, a.V * static_cast<int64_t>(sizeof(T)), sms) : 0;
    if (a.cluster > 0) return pass == Pass::kStep ? launch_rows<T, true>(a, s) : launch_rows<T, false>(a, s);
    return pass == Pass::kStep ? launch_stream<T, true>(a, s) : launch_stream<T, false>(a, s);
}

bt_status distill(Pass pass, const float *grad_loss, const void *logits, bt_dtype dtype, int64_t T, int64_t V, int64_t ld,
                  const void *ids, int ids_bytes, const void *top, bt_dtype top_dtype, int64_t S, const float *tlse,
                  float tau, float *loss, float *stats, void *grad, int64_t ldg, bt_stream stream) {
    if (!float_type(dtype) || !float_type(top_dtype) || (ids_bytes != 4 && ids_bytes != 8)) return BT_ERR_INVALID_ARG;
    if (T < 0 || V < 1 || S < 1 || ld < V || !(std::isfinite(tau) && tau > 0.0f)) return BT_ERR_INVALID_ARG;
    Args a = {};
    a.inv_tau = 1.0f / tau;
    a.c = kLog2e / tau;
    a.slack = 16.0f / a.c;
    if (!std::isfinite(a.inv_tau) || !std::isfinite(a.c) || !std::isfinite(a.slack)) return BT_ERR_INVALID_ARG;
    const bool wants_grad = pass != Pass::kLoss;
    if (wants_grad && ldg < V) return BT_ERR_INVALID_ARG;
    const int e = elem_bytes(dtype);
    if (S > kMaxSlots || V > kMaxV || T > (int64_t(1) << 24) || ld > (int64_t(1) << 36) || ldg > (int64_t(1) << 36))
        return BT_ERR_UNSUPPORTED;
    // the backward's CTAs a launch
    if (wants_grad && T * (V * e / (kBackBlockVecs * 16) + 1) > 0x7FFFFFFF) return BT_ERR_UNSUPPORTED;
    if (T == 0) return BT_OK;
    if (logits == nullptr || ids == nullptr || top == nullptr) return BT_ERR_INVALID_ARG;
    if (pass != Pass::kBackward && loss == nullptr) return BT_ERR_INVALID_ARG;
    if (pass == Pass::kBackward && stats == nullptr) return BT_ERR_INVALID_ARG;
    if (wants_grad && (grad == nullptr || grad_loss == nullptr)) return BT_ERR_INVALID_ARG;
    // the gradient may take the logits' place, row for row
    if (wants_grad && grad == logits && ldg != ld) return BT_ERR_INVALID_ARG;
    if (!aligned(logits, e) || !aligned(grad, e) || !aligned(ids, ids_bytes) || !aligned(top, elem_bytes(top_dtype)) ||
        !aligned(tlse, 4) || !aligned(loss, 4) || !aligned(stats, 4) || !aligned(grad_loss, 4))
        return BT_ERR_ALIGNMENT;
    unsigned int *err = device_error_word();
    if (err == nullptr) return BT_ERR_CUDA;
    a.z = logits; a.V = static_cast<int>(V); a.ld = ld;
    a.ids = ids; a.ids_bytes = ids_bytes; a.top = top; a.top_dt = top_dtype; a.S = static_cast<int>(S);
    a.tlse = tlse;
    a.loss = loss; a.stats = stats; a.w = grad_loss; a.grad = grad; a.ldg = ldg;
    a.err = err;
    a.limit_ns = wait_limit_ns();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    a.rows = T;
    const cudaError_t r = dtype == BT_F32 ? launch<float>(pass, a, s) : dtype == BT_BF16 ? launch<__nv_bfloat16>(pass, a, s)
                                                                                         : launch<__half>(pass, a, s);
    return r == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

}  // namespace
}  // namespace bt

using namespace bt;

extern "C" {

bt_status bt_distill_topk(const void *logits, bt_dtype dtype, int64_t T, int64_t V, int64_t ld, const void *ids,
                          int ids_bytes, const void *top, bt_dtype top_dtype, int64_t S, const float *teacher_lse,
                          float temperature, float *loss, float *stats, bt_stream stream) {
    return distill(Pass::kLoss, nullptr, logits, dtype, T, V, ld, ids, ids_bytes, top, top_dtype, S, teacher_lse,
                   temperature, loss, stats, nullptr, 0, stream);
}

bt_status bt_distill_topk_backward(const float *grad_loss, const void *logits, bt_dtype dtype, int64_t T, int64_t V,
                                   int64_t ld, const void *ids, int ids_bytes, const void *top, bt_dtype top_dtype,
                                   int64_t S, const float *stats, const float *teacher_lse, float temperature,
                                   void *grad, int64_t ldg, bt_stream stream) {
    return distill(Pass::kBackward, grad_loss, logits, dtype, T, V, ld, ids, ids_bytes, top, top_dtype, S, teacher_lse,
                   temperature, nullptr, const_cast<float *>(stats), grad, ldg, stream);
}

bt_status bt_distill_topk_step(const float *grad_loss, const void *logits, bt_dtype dtype, int64_t T, int64_t V,
                               int64_t ld, const void *ids, int ids_bytes, const void *top, bt_dtype top_dtype,
                               int64_t S, const float *teacher_lse, float temperature, float *loss, float *stats,
                               void *grad, int64_t ldg, bt_stream stream) {
    return distill(Pass::kStep, grad_loss, logits, dtype, T, V, ld, ids, ids_bytes, top, top_dtype, S, teacher_lse,
                   temperature, loss, stats, grad, ldg, stream);
}

}  // extern "C"
