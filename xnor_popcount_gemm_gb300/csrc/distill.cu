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
// The slots' own logits are taken out of the running sum as the row is read,
// so that r comes from a sum of its own and not from a difference that cancels
// where the student is as sure as the teacher. Sums and statistics are fp32.
//
// Bound: HBM. A logit costs 2 or 4 bytes each way and about seven instructions
// and one exp2 a pass; at 16 exp2 a clock and SM, the two passes of the step
// over a 16-bit row take 0.12 clocks a logit, its 4 bytes 0.17.
#include <cfloat>
#include <cmath>
#include <mutex>

#include "bt_device.cuh"
#include "bt_internal.h"
#include "tc_ptx.cuh"

namespace bt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunkBytes = 4096;          // one bulk copy
constexpr int kMaxChunks = 7;              // bulk copies of a warp: up to 28 KB
constexpr int kMaxCluster = 8;             // portable cluster size
constexpr int kMaxSlots = 1024;
constexpr int kSliceMax = kWarps * (kMaxChunks - 1) * kChunkBytes;   // bytes of a row one CTA holds (192 KB)
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

// A running maximum and the sum of 2^((v - m) c) relative to it. m starts at
// the lowest finite float, so that -inf adds 0 and a row of lowest values is a
// row like any other; s = 0 says that nothing but -inf was seen.
struct MaxSum {
    float m, s;
};
__device__ __forceinline__ MaxSum ms_empty() { return MaxSum{-FLT_MAX, 0.0f}; }
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

// Logits that are all a mask's fill value (the lowest float, or one as far
// down) are no logits at all: log-sum-exp would lose the sum beside the value.
constexpr float kMaskedBelow = -1.7e38f;
__device__ __forceinline__ bool masked(const MaxSum &a) { return a.m <= kMaskedBelow && a.s >= 0.0f; }

struct Args {
    const void *z;
    int64_t V, ld;
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
    int cluster;
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
// One warp; t and id in shared memory (id -1: an empty slot).
__device__ __forceinline__ Teacher teacher_of(const Args &a, const int *ids, const float *t, int64_t row, int lane) {
    Teacher r;
    if (a.tlse == nullptr) {
        MaxSum x = ms_empty();
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
        r.qr = q < 1.0f ? 1.0f - q : (q >= 1.0f ? 0.0f : q);       // a NaN stays one
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
            const T lo = from_f32<T>(f[2 * i]), hi = from_f32<T>(f[2 * i + 1]);
            w[i] = static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(&lo)) |
                   (static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(&hi)) << 16);
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
    int64_t head, nb, tail0;   // tail0: the first element after the vectors
};
template <typename T> __device__ __forceinline__ RowSplit split_row(const T *p, int64_t V) {
    constexpr int VEC = 16 / sizeof(T);
    const int64_t mis = static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T);
    int64_t head = mis == 0 ? 0 : VEC - mis;
    if (head > V) head = V;
    const int64_t nb = (V - head) / VEC;
    return RowSplit{head, nb, head + nb * VEC};
}

// Loss, and the gradient in the same read of the row (STEP). One cluster of
// 1 to 8 CTAs holds a row in shared memory: every warp owns a piece of it,
// fetched by bulk copies of 4 KB and summed as they land, so that no barrier
// stands between the copies and the arithmetic; the pieces' sums are joined in
// the CTA, then across the cluster through distributed shared memory, and the
// gradient is computed from shared memory. Several CTAs on an SM keep copies,
// arithmetic and stores of different rows in flight together.
template <typename T, bool STEP>
__global__ void __launch_bounds__(kThreads, 3) distill_rows_kernel(const Args a) {
    constexpr int VEC = 16 / sizeof(T);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ alignas(8) uint64_t bars[kWarps][kMaxChunks];
    __shared__ float4 red[kWarps], slot[kMaxCluster];
    __shared__ T edge[32];
    __shared__ Teacher teacher;
    __shared__ uint32_t abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = a.cluster;
    const uint32_t rank = c > 1 ? tc::cluster_ctarank() : 0u;
    const int64_t row = blockIdx.x / c;

    pdl_launch_dependents();
    if (lane == 0) {
        for (int j = 0; j < kMaxChunks; ++j) tc::mbar_init(smem_u32(&bars[warp][j]), 1);
        tc::fence_mbar_init();
    }
    if (tid == 0) abort_flag = 0;
    pdl_wait();

    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    const RowSplit sp = split_row(z, a.V);
    const int64_t v0 = sp.nb * rank / c, v1 = sp.nb * (rank + 1) / c;          // this CTA's vectors
    const int64_t w0 = v0 + (v1 - v0) * warp / kWarps, w1 = v0 + (v1 - v0) * (warp + 1) / kWarps;
    T *data = reinterpret_cast<T *>(smem);                                     // vector v at (v - v0) * VEC
    const size_t data_bytes = static_cast<size_t>((sp.nb + c - 1) / c) * 16;
    float *zt = reinterpret_cast<float *>(smem + data_bytes);                  // the student's logits of the slots
    float *tt = zt + a.S;                                                      // the teacher's
    int *ids = reinterpret_cast<int *>(tt + a.S);

    int any = 0;
    for (int k = tid; k < a.S; k += kThreads) {
        int id = slot_id(a, row * a.S + k);
        const float t = slot_logit(a, row * a.S + k);
        if (t == -INFINITY) id = -1;
        ids[k] = id;
        tt[k] = t;
        zt[k] = 0.0f;
        any |= id >= 0;
    }
    const bool live = __syncthreads_or(any) != 0;
    T *grad = STEP ? static_cast<T *>(a.grad) + row * a.ldg : nullptr;
    const bool wide = STEP && ((reinterpret_cast<uintptr_t>(grad) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    if (!live) {                                            // padding: the same for the whole cluster
        if (rank == 0 && tid == 0) {
            a.loss[row] = 0.0f;
            if (a.stats != nullptr) a.stats[2 * row] = a.stats[2 * row + 1] = 0.0f;
        }
        if constexpr (STEP) {
            const float zero[VEC] = {};
            for (int64_t v = v0 + tid; v < v1; v += kThreads) store_vec<T>(grad + sp.head + v * VEC, wide, zero);
            if (rank == 0) {
                if (tid < sp.head) grad[tid] = from_f32<T>(0.0f);
                if (tid < a.V - sp.tail0) grad[sp.tail0 + tid] = from_f32<T>(0.0f);
            }
        }
        return;
    }

    const int nchunk = static_cast<int>(((w1 - w0) * 16 + kChunkBytes - 1) / kChunkBytes);
    constexpr int kChunkVecs = kChunkBytes / 16;
    if (lane == 0) {
        for (int j = 0; j < nchunk; ++j) {
            const int64_t b = w0 + static_cast<int64_t>(j) * kChunkVecs;
            const uint32_t n = static_cast<uint32_t>(min(static_cast<int64_t>(kChunkVecs), w1 - b)) * 16u;
            const uint32_t bar = smem_u32(&bars[warp][j]);
            tc::mbar_arrive_expect_tx(bar, n);
            tc::bulk_load_once(smem_u32(data + (b - v0) * VEC), z + sp.head + b * VEC, n, bar);
        }
    }
    // The elements outside the vectors (at most 7 on either side): rank 0, warp 0.
    const bool edges = rank == 0 && warp == 0;
    const int nhead = static_cast<int>(sp.head), ntail = static_cast<int>(a.V - sp.tail0);
    if (edges) {
        T v = from_f32<T>(-INFINITY);
        if (lane < nhead) v = z[lane];
        else if (lane >= 16 && lane - 16 < ntail) v = z[sp.tail0 + lane - 16];
        edge[lane] = v;
        __syncwarp();
    }
    if (warp == kWarps - 1) {
        const Teacher t = teacher_of(a, ids, tt, row, lane);
        if (lane == 0) teacher = t;
    }

    const uint32_t zt_rank0 = c > 1 ? tc::mapa(smem_u32(zt), 0) : 0u;
    MaxSum rest = ms_empty(), top = ms_empty();
    float seen = -FLT_MAX;                                  // the largest logit so far; rest.m may trail it by the slack
    // take slot k's logit out of the row
    auto take = [&](int k, T *p) {
        const float v = Elem<T>::to_f32(*p);
        *p = from_f32<T>(-INFINITY);
        zt[k] = v;
        if (c > 1 && rank != 0)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(zt_rank0 + 4u * k), "f"(v) : "memory");
        ms_add(top, v, a.c);
    };
    // a cluster's CTAs must all have started before the first remote store
    if (c > 1) tc::cluster_sync();
    if (edges) {
        for (int k = lane; k < a.S; k += 32) {
            const int id = ids[k];
            if (id < 0) continue;
            if (id < nhead) take(k, &edge[id]);
            else if (id >= sp.tail0) take(k, &edge[16 + id - static_cast<int>(sp.tail0)]);
        }
        __syncwarp();
        ms_add(rest, Elem<T>::to_f32(edge[lane]), a.c);
        seen = rest.m;
    }
    for (int j = 0; j < nchunk; ++j) {
        const uint32_t bar = smem_u32(&bars[warp][j]);
        if (!tc::wait_fast(bar, 0, &abort_flag, a.err, a.limit_ns)) {
            // gave up (recorded): the copy must still land before the CTA's memory is given back
            uint32_t drain = 0;
            tc::wait_bounded(bar, 0, &drain, a.err);
        }
        const int64_t b = w0 + static_cast<int64_t>(j) * kChunkVecs;
        const int n = static_cast<int>(min(static_cast<int64_t>(kChunkVecs), w1 - b));
        T *p = data + (b - v0) * VEC;
        const int first = static_cast<int>(sp.head + b * VEC);
        for (int k = lane; k < a.S; k += 32) {
            const unsigned off = static_cast<unsigned>(ids[k]) - static_cast<unsigned>(first);
            if (ids[k] >= 0 && off < static_cast<unsigned>(n * VEC)) take(k, p + off);
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
            float f[VEC];
            Elem<T>::unpack(reinterpret_cast<const uint4 *>(p)[i], f);
            float mx = f[0];
#pragma unroll
            for (int e = 1; e < VEC; ++e) mx = fmaxf(mx, f[e]);
            seen = fmaxf(seen, mx);
            if (mx > rest.m + a.slack) {
                rest.s *= ex2((rest.m - mx) * a.c);
                rest.m = mx;
            }
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += ex2((f[e] - rest.m) * a.c);
            rest.s += s;
        }
    }
    rest = ms_warp(rest, seen, a.c);
    top = ms_warp(top, top.m, a.c);
    if (lane == 0) red[warp] = make_float4(rest.m, rest.s, top.m, top.s);
    __syncthreads();
    if (warp == 0) {
        rest = ms_sum(&red[0].x, kWarps, 4, a.c, false);
        top = ms_sum(&red[0].z, kWarps, 4, a.c, false);
        if (lane < c) {
            if (c == 1) {
                slot[0] = make_float4(rest.m, rest.s, top.m, top.s);
            } else {
                const uint32_t dst = tc::mapa(smem_u32(&slot[rank]), lane);
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(rest.m), "f"(rest.s),
                             "f"(top.m), "f"(top.s)
                             : "memory");
            }
        }
    }
    if (c > 1) tc::cluster_sync();
    else __syncthreads();
    rest = ms_sum(&slot[0].x, c, 4, a.c, true);
    top = ms_sum(&slot[0].z, c, 4, a.c, true);
    if (masked(rest)) rest.s = 0.0f;
    if (masked(top)) top.s = 0.0f;
    const MaxSum all = ms_join(rest, top, a.c);
    const bool empty = all.s == 0.0f;                       // the student has nothing left
    const Teacher te = teacher;

    if (rank == 0 && warp == 0) {
        // from the statistics as they are returned: the loss and its backward belong to the same lse and r
        const float lse = empty ? -INFINITY : all.m * a.inv_tau + logf(all.s);
        const float r = rest.s == 0.0f ? -INFINITY : rest.m * a.inv_tau + logf(rest.s);
        float l = 0.0f;
        for (int k = lane; k < a.S; k += 32) {
            if (ids[k] < 0) continue;
            const float q = expf(log_q(a, te, tt[k]));
            if (!(q == 0.0f)) l += q * (logf(q) - (zt[k] * a.inv_tau - lse));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (lane == 0) {
            if (a.tlse != nullptr && rest.s != 0.0f && !(te.qr == 0.0f)) l += te.qr * (logf(te.qr) - (r - lse));
            a.loss[row] = empty ? 0.0f : l;
            if (a.stats != nullptr) {
                a.stats[2 * row] = lse;
                a.stats[2 * row + 1] = r;
            }
        }
    }
    if constexpr (STEP) {
        const float w = __ldg(a.w + row) * a.inv_tau;
        // outside the slots: coef * 2^((z - base) c)
        float coef, base;
        if (a.tlse != nullptr) {
            const float pr = rest.s * ex2((rest.m - all.m) * a.c) / all.s;
            coef = rest.s == 0.0f ? 0.0f : w * (pr - te.qr) / rest.s;
            base = rest.m;
        } else {
            coef = empty ? 0.0f : w / all.s;
            base = all.m;
        }
        for (int64_t v = w0 + lane; v < w1; v += 32) {
            float f[VEC];
            Elem<T>::unpack(reinterpret_cast<const uint4 *>(data)[v - v0], f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = coef * ex2((f[e] - base) * a.c);
            store_vec<T>(grad + sp.head + v * VEC, wide, f);
        }
        if (edges) {
            const float f = coef * ex2((Elem<T>::to_f32(edge[lane]) - base) * a.c);
            if (lane < nhead) grad[lane] = from_f32<T>(f);
            else if (lane >= 16 && lane - 16 < ntail) grad[sp.tail0 + lane - 16] = from_f32<T>(f);
        }
        __syncwarp();
        // the slots of this warp's piece, over what was just written there
        const int64_t lo = sp.head + w0 * VEC, hi = sp.head + w1 * VEC;
        for (int k = lane; k < a.S; k += 32) {
            const int64_t id = ids[k];
            if (id < 0) continue;
            if ((id >= lo && id < hi) || (edges && (id < sp.head || id >= sp.tail0))) {
                const float p = ex2((zt[k] - all.m) * a.c) / all.s;
                grad[id] = from_f32<T>(empty ? 0.0f : w * (p - expf(log_q(a, te, tt[k]))));
            }
        }
    }
}

// The gradient from a forward's statistics: pieces of kPiece vectors of a row,
// one CTA each, read and written once. The slots' logits are read before
// anything is written, so the gradient may take the logits' place.
constexpr int kPiece = kThreads * 8;

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_backward_kernel(const Args a, int pieces) {
    constexpr int VEC = 16 / sizeof(T);
    __shared__ float zt[kMaxSlots], tt[kMaxSlots];
    __shared__ int ids[kMaxSlots];
    __shared__ Teacher teacher;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / pieces;
    const int piece = static_cast<int>(blockIdx.x % pieces);
    pdl_launch_dependents();
    pdl_wait();
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    T *grad = static_cast<T *>(a.grad) + row * a.ldg;
    const bool wide = ((reinterpret_cast<uintptr_t>(grad) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    const RowSplit sp = split_row(z, a.V);
    const int64_t v0 = static_cast<int64_t>(piece) * kPiece, v1 = min(v0 + kPiece, sp.nb);
    // this CTA's elements: its vectors, and with the first piece the ones outside all vectors
    const int64_t lo = sp.head + v0 * VEC, hi = sp.head + v1 * VEC;

    uint4 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t v = v0 + tid + i * kThreads;
        if (v < v1) q[i] = ld_stream_v4(z + sp.head + v * VEC);
    }
    int any = 0;
    for (int k = tid; k < a.S; k += kThreads) {
        int id = slot_id(a, row * a.S + k);
        const float t = slot_logit(a, row * a.S + k);
        if (t == -INFINITY) id = -1;
        any |= id >= 0;
        ids[k] = id;
        tt[k] = t;
        const bool mine = id >= 0 && ((id >= lo && id < hi) || (piece == 0 && (id < sp.head || id >= sp.tail0)));
        zt[k] = mine ? Elem<T>::to_f32(z[id]) : 0.0f;
    }
    const bool outside = piece == 0 && tid < 32;
    const int nhead = static_cast<int>(sp.head), ntail = static_cast<int>(a.V - sp.tail0);
    float ez = -INFINITY;
    if (outside) {
        if (tid < nhead) ez = Elem<T>::to_f32(z[tid]);
        else if (tid >= 16 && tid - 16 < ntail) ez = Elem<T>::to_f32(z[sp.tail0 + tid - 16]);
    }
    const bool live = __syncthreads_or(any) != 0;
    if (warp == 0) {
        const Teacher t = teacher_of(a, ids, tt, row, lane);
        if (lane == 0) teacher = t;
    }
    __syncthreads();
    const Teacher te = teacher;
    const float lse = __ldg(a.stats + 2 * row), r = __ldg(a.stats + 2 * row + 1);
    const bool dead = !live || lse == -INFINITY;
    const float w = __ldg(a.w + row) * a.inv_tau;
    float coef = dead ? 0.0f : w, base = dead ? 0.0f : lse;
    if (a.tlse != nullptr && !dead) {
        const bool none = r == -INFINITY;
        coef = none ? 0.0f : w * (expf(r - lse) - te.qr);
        base = none ? 0.0f : r;
    }
    // exp(z / tau - base); a row that gives nothing must give 0 whatever it holds
    auto value = [&](float v) { return dead ? 0.0f : coef * ex2((v * a.inv_tau - base) * kLog2e); };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t v = v0 + tid + i * kThreads;
        if (v < v1) {
            float f[VEC];
            Elem<T>::unpack(q[i], f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = value(f[e]);
            store_vec<T>(grad + sp.head + v * VEC, wide, f);
        }
    }
    if (outside) {
        if (tid < nhead) grad[tid] = from_f32<T>(value(ez));
        else if (tid >= 16 && tid - 16 < ntail) grad[sp.tail0 + tid - 16] = from_f32<T>(value(ez));
    }
    __syncthreads();
    if (dead) return;
    for (int k = tid; k < a.S; k += kThreads) {
        const int64_t id = ids[k];
        if (id >= 0 && ((id >= lo && id < hi) || (piece == 0 && (id < sp.head || id >= sp.tail0)))) {
            const float p = ex2((zt[k] * a.inv_tau - lse) * kLog2e);
            grad[id] = from_f32<T>(w * (p - expf(log_q(a, te, tt[k]))));
        }
    }
}

int elem_bytes(bt_dtype t) { return t == BT_F32 ? 4 : 2; }
bool float_type(int t) { return t == BT_F32 || t == BT_BF16 || t == BT_F16; }

// CTAs per row: enough that a CTA holds at most 68 KB of it, so that three
// fit an SM; with few rows more, down to 4 KB each, until every SM has a CTA.
int rows_cluster(int64_t T, int64_t row_bytes, int sms) {
    int c = 1;
    while (c < kMaxCluster && row_bytes > static_cast<int64_t>(c) * 68 * 1024) c *= 2;
    while (c < kMaxCluster && T * c * 2 <= sms && row_bytes >= static_cast<int64_t>(c) * 8192) c *= 2;
    return c;
}

template <typename T, bool STEP>
cudaError_t launch_rows(Args a, int64_t rows, cudaStream_t s) {
    auto kern = distill_rows_kernel<T, STEP>;
    constexpr int kDynMax = kSliceMax + 16 + 12 * kMaxSlots;
    static std::once_flag once;
    static cudaError_t attr_err = cudaSuccess;
    std::call_once(once, [&] { attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynMax); });
    if (attr_err != cudaSuccess) return attr_err;
    const int64_t bytes = a.V * static_cast<int64_t>(sizeof(T));
    a.cluster = rows_cluster(rows, bytes, device_sm_count());
    const int64_t slice = (bytes / 16 + a.cluster - 1) / a.cluster * 16;      // the most any alignment needs
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(rows * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(slice) + 12u * static_cast<size_t>(a.S);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const Args>(a));
}

template <typename T>
cudaError_t launch_backward(const Args &a, int64_t rows, cudaStream_t s) {
    constexpr int VEC = 16 / sizeof(T);
    const int64_t pieces = a.V / VEC == 0 ? 1 : (a.V / VEC + kPiece - 1) / kPiece;
    return launch_pdl(distill_backward_kernel<T>, dim3(static_cast<unsigned>(rows * pieces)), dim3(kThreads), s, a,
                      static_cast<int>(pieces));
}

enum class Pass { kLoss, kStep, kBackward };

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
    // kSliceMax of a row for each CTA of the largest cluster
    if (S > kMaxSlots || V > static_cast<int64_t>(kMaxCluster) * kSliceMax / e || T > (int64_t(1) << 24) ||
        ld > (int64_t(1) << 36) || ldg > (int64_t(1) << 36))
        return BT_ERR_UNSUPPORTED;                          // a grid of T * 96 pieces and T * ld * 4 bytes fit their types
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
    a.z = logits; a.V = V; a.ld = ld;
    a.ids = ids; a.ids_bytes = ids_bytes; a.top = top; a.top_dt = top_dtype; a.S = static_cast<int>(S);
    a.tlse = tlse;
    a.loss = loss; a.stats = stats; a.w = grad_loss; a.grad = grad; a.ldg = ldg;
    a.err = err;
    a.limit_ns = wait_limit_ns();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto tag) {
        using E = decltype(tag);
        if (pass == Pass::kBackward) return launch_backward<E>(a, T, s);
        return pass == Pass::kStep ? launch_rows<E, true>(a, T, s) : launch_rows<E, false>(a, T, s);
    };
    const cudaError_t r = dtype == BT_F32 ? go(float{}) : dtype == BT_BF16 ? go(__nv_bfloat16{}) : go(__half{});
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
