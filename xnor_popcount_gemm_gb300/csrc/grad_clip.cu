// The global norm of many gradients and clipping by it:
//   norm = sqrt(sum over all tensors of g^2)      g *= min(1, max_norm / (norm + eps))
//
// Two streams over the same bytes, the second of them (read and write) only where
// the factor is below one, from the end backwards: what the first read last is
// still in L2. The tensors' addresses go along as a kernel's parameter, so that
// nothing is copied to the device and a captured graph holds them; up to 1536 go
// with one launch.
//
// A piece of 16 KB is one CTA's work at a time; pieces do not cross tensors. Squares are summed in fp32 over a thread's
// part of a piece (at most 33 values), then in double. A part whose sum leaves the range where fp32 squares are exact
// enough (tiny or huge values) is summed again in double. Partial sums are joined in an order that the sizes decide:
// equal calls give equal results. 448 tensors of 40.7 million floats: 41 us on the GPU, the norm alone 33 (163 MB, 73 % of
// the copy rate); a call takes about 175, which is Python looking at 448 tensors.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "bt_internal.h"
#include "mx.cuh"

namespace bt {
namespace {

constexpr int kThreads = 256;
constexpr int kPieceBytes = 16384;
constexpr int kCtasPerSm = 6;             // as many as fit
constexpr int kFew = 64, kMany = 1536;      // tensors of a launch

// The tensors of a launch: elements and element type (bt_dtype) in one word, the pieces before each.
template <int MOST> struct Table {
    void *p[MOST];
    uint64_t n[MOST];                       // elements * 4 + type
    uint32_t before[MOST + 1];
    int count;
};
static_assert(sizeof(Table<kMany>) < 32000, "kernel parameters end at 32764 bytes");

struct ClipArgs {
    double *partial;                        // one of every CTA of every norm launch
    int first, all;                         // this launch's CTAs in it; all of them
    float max_norm, eps;
    float *norm;
};

// Where a piece lies: its tensor's type, its address and its elements.
struct Piece {
    void *p;
    int n, type;
};
template <int MOST> __device__ __forceinline__ Piece piece_of(const Table<MOST> &t, uint32_t i) {
    int lo = 0, hi = t.count;               // before[lo] <= i < before[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (t.before[m] <= i) lo = m; else hi = m;
    }
    const int type = static_cast<int>(t.n[lo] & 3);
    const int64_t n = static_cast<int64_t>(t.n[lo] >> 2), size = type == BT_F32 ? 4 : 2, per = kPieceBytes / size;
    const int64_t at = static_cast<int64_t>(i - t.before[lo]) * per;
    return Piece{static_cast<uint8_t *>(t.p[lo]) + at * size, static_cast<int>(n - at < per ? n - at : per), type};
}

// Squares of a piece's elements, this thread's part. F(v): what is summed.
template <typename T, typename F> __device__ __forceinline__ void walk(const Piece &p, F f) {
    constexpr int VEC = 16 / sizeof(T);
    const T *g = static_cast<const T *>(p.p);
    // up to the first 16-byte boundary, whole 16 bytes, the rest
    int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / static_cast<int>(sizeof(T));
    head = head < p.n ? head : p.n;
    const int vecs = (p.n - head) / VEC, tail = head + vecs * VEC;
    const uint4 *v = reinterpret_cast<const uint4 *>(g + head);
    constexpr int kLoads = kPieceBytes / 16 / kThreads;
    uint4 raw[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int j = threadIdx.x + i * kThreads;
        raw[i] = j < vecs ? v[j] : make_uint4(0u, 0u, 0u, 0u);
    }
    float edge = 0.0f;
    if (threadIdx.x < head) edge = Elem<T>::to_f32(g[threadIdx.x]);
    else if (threadIdx.x >= 32 && static_cast<int>(threadIdx.x) - 32 < p.n - tail) edge = Elem<T>::to_f32(g[tail + threadIdx.x - 32]);
    f(raw, edge);
}

template <typename T> __device__ __forceinline__ double squares(const Piece &p) {
    constexpr int VEC = 16 / sizeof(T);
    double out = 0.0;
    walk<T>(p, [&](const uint4 (&raw)[kPieceBytes / 16 / kThreads], float edge) {
        float s0 = edge * edge, s1 = 0.0f;
        uint32_t any = __float_as_uint(edge);
#pragma unroll
        for (int i = 0; i < kPieceBytes / 16 / kThreads; ++i) {
            float v[VEC];
            Elem<T>::unpack(raw[i], v);
            any |= raw[i].x | raw[i].y | raw[i].z | raw[i].w;
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                s0 = fmaf(v[e], v[e], s0);
                s1 = fmaf(v[e + 1], v[e + 1], s1);
            }
        }
        const float s = s0 + s1;
        // between these no square that counts was rounded away or overflowed
        if (s > 1e-24f && s < 1e36f) {
            out = static_cast<double>(s);
        } else if ((any & 0x7FFFFFFFu) != 0u || s != 0.0f) {
            double d = static_cast<double>(edge) * edge;
            for (int i = 0; i < kPieceBytes / 16 / kThreads; ++i) {
                float v[VEC];
                Elem<T>::unpack(raw[i], v);
                for (int e = 0; e < VEC; ++e) d = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), d);
            }
            out = d;
        }
    });
    return out;
}

__device__ __forceinline__ double block_total(double v, double *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) t += red[i];
    return t;
}

template <int MOST> __global__ void __launch_bounds__(kThreads, kCtasPerSm) clip_norm_kernel(const __grid_constant__ Table<MOST> t, const ClipArgs a) {
    __shared__ double red[kThreads / 32];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    double sum = 0.0;
    for (uint32_t i = blockIdx.x; i < t.before[t.count]; i += gridDim.x) {
        const Piece p = piece_of(t, i);
        sum += p.type == BT_F32 ? squares<float>(p) : p.type == BT_BF16 ? squares<__nv_bfloat16>(p) : squares<__half>(p);
    }
    sum = block_total(sum, red);
    if (threadIdx.x == 0) a.partial[a.first + blockIdx.x] = sum;
}

template <typename T> __device__ __forceinline__ void scale(const Piece &p, float f) {
    constexpr int VEC = 16 / sizeof(T);
    T *g = static_cast<T *>(p.p);
    int head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(g) & 15)) & 15) / static_cast<int>(sizeof(T));
    head = head < p.n ? head : p.n;
    const int vecs = (p.n - head) / VEC, tail = head + vecs * VEC;
    walk<T>(p, [&](const uint4 (&raw)[kPieceBytes / 16 / kThreads], float edge) {
        uint4 *v = reinterpret_cast<uint4 *>(g + head);
#pragma unroll
        for (int i = 0; i < kPieceBytes / 16 / kThreads; ++i) {
            const int j = threadIdx.x + i * kThreads;
            if (j >= vecs) continue;
            float x[8];
            Elem<T>::unpack(raw[i], x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] *= f;
            if constexpr (sizeof(T) == 4)
                v[j] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            else
                v[j] = mx::raw_pack<T>(x).a;
        }
        if (threadIdx.x < head) g[threadIdx.x] = mx::from_f32<T>(edge * f);
        else if (threadIdx.x >= 32 && static_cast<int>(threadIdx.x) - 32 < p.n - tail) g[tail + threadIdx.x - 32] = mx::from_f32<T>(edge * f);
    });
}

template <int MOST> __global__ void __launch_bounds__(kThreads, kCtasPerSm) clip_scale_kernel(const __grid_constant__ Table<MOST> t, const ClipArgs a) {
    __shared__ double red[kThreads / 32];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait();
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.all; i += kThreads) sum += a.partial[i];
    const double total = block_total(sum, red);
    const float norm = static_cast<float>(sqrt(total));
    if (a.first == 0 && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
    // not below one, or nothing but zeros (whose factor would be 0 / 0 without max_norm and eps): nothing to do; a NaN norm
    // makes every gradient NaN, unless none was to be clipped
    const float f = a.max_norm / (norm + a.eps);
    if (f >= 1.0f || total == 0.0 || isinf(a.max_norm)) return;
    const uint32_t n = t.before[t.count];
    for (uint32_t i = blockIdx.x; i < n; i += gridDim.x) {
        const Piece p = piece_of(t, n - 1 - i);
        if (p.type == BT_F32) scale<float>(p, f);
        else if (p.type == BT_BF16) scale<__nv_bfloat16>(p, f);
        else scale<__half>(p, f);
    }
}

__global__ void clip_no_norm_kernel(float *norm) {
    pdl_wait();
    *norm = 0.0f;
}

// Tensors from `first` on, as many as go with one launch; returns how many it took (empty ones among them).
template <int MOST> int64_t fill(Table<MOST> &t, void *const *p, const int64_t *n, const int32_t *type, int64_t first, int64_t count) {
    t.count = 0;
    uint64_t pieces = 0;
    int64_t i = first;
    for (; i < count && t.count < MOST; ++i) {
        if (n[i] == 0) continue;
        const int64_t per = kPieceBytes / (type[i] == BT_F32 ? 4 : 2), more = (n[i] + per - 1) / per;
        if (pieces + static_cast<uint64_t>(more) > 0x7FFFFFFFu) break;
        t.p[t.count] = p[i];
        t.n[t.count] = static_cast<uint64_t>(n[i]) * 4 + static_cast<uint64_t>(type[i]);
        t.before[t.count] = static_cast<uint32_t>(pieces);
        pieces += static_cast<uint64_t>(more);
        ++t.count;
    }
    t.before[t.count] = static_cast<uint32_t>(pieces);
    return i - first;
}

int grid_of(uint32_t pieces) {
    const int64_t most = static_cast<int64_t>(kCtasPerSm) * device_sm_count();
    return static_cast<int>(static_cast<int64_t>(pieces) < most ? pieces : most);
}

template <int MOST> bt_status clip(void *const *p, const int64_t *n, const int32_t *type, int64_t count, ClipArgs a, cudaStream_t s) {
    Table<MOST> *t = new (std::nothrow) Table<MOST>;        // 31 KB: not on the caller's stack
    if (t == nullptr) return BT_ERR_CUDA;
    cudaError_t e = cudaSuccess;
    for (int pass = 0; pass < 2 && e == cudaSuccess; ++pass) {
        int at = 0;
        for (int64_t i = 0; i < count && e == cudaSuccess;) {
            i += fill(*t, p, n, type, i, count);
            if (t->count == 0) continue;
            const int grid = pass == 1 && std::isinf(a.max_norm) ? 1 : grid_of(t->before[t->count]);
            a.first = at;
            e = launch_pdl(pass == 0 ? clip_norm_kernel<MOST> : clip_scale_kernel<MOST>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), s,
                           static_cast<const Table<MOST> &>(*t), static_cast<const ClipArgs &>(a));
            at += grid;
        }
        if (pass == 0) a.all = at;
    }
    if (e == cudaSuccess && a.all == 0) e = launch_pdl(clip_no_norm_kernel, dim3(1), dim3(1), s, a.norm);
    delete t;
    return e == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

int64_t element(int32_t type) { return type == BT_F32 ? 4 : 2; }

}  // namespace
}  // namespace bt

using namespace bt;

extern "C" {

// The partial sums: a launch for every kMany tensors that hold anything, at least one for 2^31 pieces.
size_t bt_clip_grads_workspace(int64_t count) {
    if (count < 1 || count > (int64_t(1) << 20)) return 0;
    const size_t launches = static_cast<size_t>((count + kMany - 1) / kMany) + 64;
    return round_up256(launches * static_cast<size_t>(kCtasPerSm) * static_cast<size_t>(device_sm_count()) * 8);
}

bt_status bt_clip_grads(void *const *grads, const int64_t *numels, const int32_t *dtypes, int64_t count, float max_norm, float eps,
                        float *norm, void *workspace, size_t workspace_bytes, bt_stream stream) {
    if (count < 0 || std::isnan(max_norm) || max_norm < 0.0f || !std::isfinite(eps) || eps < 0.0f) return BT_ERR_INVALID_ARG;
    if (count > (int64_t(1) << 20)) return BT_ERR_UNSUPPORTED;
    if (norm == nullptr || (count > 0 && (grads == nullptr || numels == nullptr || dtypes == nullptr))) return BT_ERR_INVALID_ARG;
    if (!aligned(norm, 4)) return BT_ERR_ALIGNMENT;
    struct Range {
        uintptr_t from, to;
    };
    const size_t room = static_cast<size_t>(count > 0 ? count : 1);
    Range *ranges = new (std::nothrow) Range[room];
    if (ranges == nullptr) return BT_ERR_CUDA;
    bt_status bad = BT_OK;
    size_t used = 0;
    int64_t pieces = 0;
    bool sorted = true;
    for (int64_t i = 0; i < count && bad == BT_OK; ++i) {
        if (dtypes[i] != BT_F32 && dtypes[i] != BT_BF16 && dtypes[i] != BT_F16) bad = BT_ERR_INVALID_ARG;
        else if (numels[i] < 0 || (numels[i] > 0 && grads[i] == nullptr)) bad = BT_ERR_INVALID_ARG;
        else if (numels[i] > (int64_t(1) << 40)) bad = BT_ERR_UNSUPPORTED;
        else if (numels[i] > 0 && !aligned(grads[i], static_cast<size_t>(element(dtypes[i])))) bad = BT_ERR_ALIGNMENT;
        if (bad != BT_OK || numels[i] == 0) continue;
        const uintptr_t from = reinterpret_cast<uintptr_t>(grads[i]);
        ranges[used] = Range{from, from + static_cast<uintptr_t>(numels[i] * element(dtypes[i]))};
        pieces += numels[i] * element(dtypes[i]) / kPieceBytes + 1;
        if (used > 0 && ranges[used].from < ranges[used - 1].to) sorted = false;
        ++used;
    }
    if (bad == BT_OK && pieces > (int64_t(1) << 35)) bad = BT_ERR_UNSUPPORTED;
    if (bad == BT_OK && !sorted) {          // an element that two tensors share would be scaled twice
        std::sort(ranges, ranges + used, [](const Range &x, const Range &y) { return x.from < y.from; });
        for (size_t i = 1; i < used; ++i)
            if (ranges[i].from < ranges[i - 1].to) bad = BT_ERR_INVALID_ARG;
    }
    delete[] ranges;
    if (bad != BT_OK) return bad;
    const size_t need = bt_clip_grads_workspace(count);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BT_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return BT_ERR_ALIGNMENT;
    ClipArgs a = {};
    a.partial = static_cast<double *>(workspace);
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = norm;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return count <= kFew ? clip<kFew>(grads, numels, dtypes, count, a, s) : clip<kMany>(grads, numels, dtypes, count, a, s);
}

}  // extern "C"
