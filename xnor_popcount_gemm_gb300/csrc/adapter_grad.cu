// The adapters' gradients (dA = dU^T x, dB = s u^T g) and the sum of their parts: see adapter.cu.
#include "adapter.cuh"

namespace bt {
namespace adapter {
namespace {

// A CTA takes 128 columns of x (or g) and a part of one adapter's tokens, 64 at
// a time: D (128 columns x rank, fp32, tensor memory) += X^T (U_hi + U_lo). Both
// operands lie as they arrive, a token a row, and go to the tensor cores
// MN-major: nothing is transposed. U is fp32 in memory and is split into its
// two 16-bit values on the way to shared memory, a stage ahead. A part that is
// its adapter's only one writes the gradient; the others write their sums to
// the workspace, which sum_kernel adds up in order. Both products run in one
// launch, so that neither leaves the machine half empty at its end.
using T = __nv_bfloat16;
constexpr int kCols = 128, kTok = 64;
constexpr int kAtom = 8192;                                 // 64 tokens' rows of 128 bytes
constexpr int kXBytes = 2 * kAtom;                          // 128 columns
constexpr int kStages = 4;
template <int RP> constexpr int kUPart = (RP <= 64 ? 1 : 2) * kAtom;       // one of hi, lo
template <int RP> constexpr int kSmem = kStages * kXBytes + 2 * 2 * kUPart<RP> + 1024;

__device__ __forceinline__ uint32_t sw128(int row, int chunk) { return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4)); }

template <int RP>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) grad_kernel(const GradArgs a) {
    extern __shared__ uint8_t dyn[];
    __shared__ alignas(8) uint64_t bars[kStages];
    __shared__ uint32_t tmem_slot, abort_flag;
    constexpr int kTmem = RP < 32 ? 32 : RP;
    uint8_t *smem = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    uint8_t *ubase = smem + kStages * kXBytes;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();                                             // before tensor memory is taken, see shrink_kernel
    if (warp == 0) {
        tc::tmem_alloc(smem_u32(&tmem_slot), kTmem);
        tc::tmem_relinquish();
        if (lane == 0) {
            abort_flag = 0;
            for (int i = 0; i < kStages; ++i) tc::mbar_init(smem_u32(&bars[i]), 1);
            tc::fence_mbar_init();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_slot;

    const int both = a.p[0].slices + a.p[1].slices;
    const AdapterTile part = a.plan.tiles[blockIdx.x / both];
    const int sl = static_cast<int>(blockIdx.x % both);
    const GradProduct &p = a.p[sl < a.p[0].slices ? 0 : 1];
    const int c0 = (sl < a.p[0].slices ? sl : sl - a.p[0].slices) * kCols;
    const int32_t *rows = a.plan.rows + part.first;
    const int n = (part.n + kTok - 1) / kTok;
    // this thread's chunks of X: column chunk tid % 16 of tokens tid / 16 + 16 i
    const int cj = tid & 15, ct = tid >> 4;
    int xrow[4];
    auto fetch_rows = [&](int s) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = s * kTok + ct + 16 * i;
            xrow[i] = at < part.n ? rows[at] : -1;
        }
    };
    auto load_x = [&](int s) {
        uint8_t *xs = smem + (s % kStages) * kXBytes + (cj >> 3) * kAtom;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int valid = xrow[i] >= 0 ? p.C - c0 - 8 * cj : 0;
            copy8(reinterpret_cast<uint16_t *>(xs + sw128(ct + 16 * i, cj & 7)),
                  valid > 0 ? p.x + static_cast<int64_t>(xrow[i]) * p.ldx + c0 + 8 * cj : p.x, valid, p.ax);
        }
    };
    // U: thread (token tid / 4, a quarter of the ranks), pairs of ranks
    constexpr int UV = RP / 8;
    const int utok = tid >> 2, ur = (tid & 3) * 2;
    float2 uv[UV];
    int urow;
    auto fetch_urow = [&](int s) {
        const int at = s * kTok + utok;
        urow = at < part.n ? rows[at] : -1;
    };
    auto load_u = [&]() {
        const float *u = p.u + static_cast<int64_t>(urow < 0 ? 0 : urow) * a.R;
        if ((a.R & 1) == 0) {
#pragma unroll
            for (int i = 0; i < UV; ++i) {
                const int r = ur + 8 * i;
                uv[i] = urow >= 0 && r < a.R ? *reinterpret_cast<const float2 *>(u + r) : make_float2(0.0f, 0.0f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < UV; ++i) {
                const int r = ur + 8 * i;
                uv[i].x = urow >= 0 && r < a.R ? u[r] : 0.0f;
                uv[i].y = urow >= 0 && r + 1 < a.R ? u[r + 1] : 0.0f;
            }
        }
    };
    auto store_u = [&](int s) {
        uint8_t *hi = ubase + (s & 1) * 2 * kUPart<RP>, *lo = hi + kUPart<RP>;
#pragma unroll
        for (int i = 0; i < UV; ++i) {
            uint32_t h, l;
            split2<T>(uv[i].x, uv[i].y, h, l);
            const uint32_t off = (i >> 3) * kAtom + sw128(utok, i & 7) + 2 * ur;
            *reinterpret_cast<uint32_t *>(hi + off) = h;
            *reinterpret_cast<uint32_t *>(lo + off) = l;
        }
    };
    auto wait_mma = [&](int s) {
        const uint32_t bar = smem_u32(&bars[s % kStages]), parity = static_cast<uint32_t>(s / kStages) & 1u;
        if (!tc::wait_fast(bar, parity, &abort_flag, a.err, a.limit_ns)) {
            uint32_t drain = 0;                             // recorded; the products in flight must still land
            tc::wait_bounded(bar, parity, &drain, a.err);
        }
    };
    // fp32 sums, bf16 operands, both MN-major, N = RP, M = 128
    constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                                ((static_cast<uint32_t>(RP) >> 3) << 17) | ((128u >> 4) << 24);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (s < n) {
            fetch_rows(s);
            load_x(s);
        }
        cp_async_commit();
    }
    if (n > 0) {
        fetch_urow(0);
        load_u();
        store_u(0);
        fetch_urow(1);
        load_u();
        fetch_urow(2);
    }
    fetch_rows(kStages - 1);
    for (int s = 0; s < n; ++s) {
        cp_async_wait<kStages - 2>();
        tc::fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc::fence_after_sync();
            const uint32_t xs = smem_u32(smem + (s % kStages) * kXBytes);
            const uint32_t hi = smem_u32(ubase + (s & 1) * 2 * kUPart<RP>), lo = hi + kUPart<RP>;
#pragma unroll
            for (int k = 0; k < 4; ++k) {                   // 16 tokens: 16 rows of either operand
                const uint64_t da = tc::sw128_mnmajor_desc(xs + 2048 * k, kAtom);
                tc::mma_f16(tmem, da, tc::sw128_mnmajor_desc(hi + 2048 * k, kAtom), kIdesc, (s | k) != 0);
                tc::mma_f16(tmem, da, tc::sw128_mnmajor_desc(lo + 2048 * k, kAtom), kIdesc, 1);
            }
            tc::mma_commit(smem_u32(&bars[s % kStages]));
        }
        if (s > 0) wait_mma(s - 1);                         // X's slot and U's buffer are free again
        if (s + kStages - 1 < n) {
            load_x(s + kStages - 1);
            fetch_rows(s + kStages);
        }
        cp_async_commit();
        if (s + 1 < n) {
            store_u(s + 1);
            load_u();
            fetch_urow(s + 3);
        }
    }
    cp_async_wait<0>();
    if (n > 0) wait_mma(n - 1);
    tc::fence_after_sync();
    const float scale = p.scale != nullptr ? p.scale[part.adapter] : 1.0f;
    float *out = part.slot >= 0 ? p.slots + part.slot * a.slot_stride : p.grad + static_cast<int64_t>(part.adapter) * a.R * p.C;
    const int col = c0 + (warp & 3) * 32 + lane;            // the accumulator's lane
    for (int r0 = (warp >> 2) * 32; r0 < RP; r0 += 64) {
        uint32_t v[32];
        if (n > 0) {
            tc::tmem_ld32(tmem + (static_cast<uint32_t>(warp & 3) << 21) + r0, v);
            tc::tmem_ld_wait();
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (col < p.C) {
            if (p.rc) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (r0 + i < a.R) out[static_cast<int64_t>(r0 + i) * p.C + col] = __uint_as_float(v[i]) * scale;
            } else if ((a.R & 3) == 0) {
                float *o = out + static_cast<int64_t>(col) * a.R + r0;
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (r0 + i < a.R)
                        *reinterpret_cast<float4 *>(o + i) =
                            make_float4(__uint_as_float(v[i]) * scale, __uint_as_float(v[i + 1]) * scale,
                                        __uint_as_float(v[i + 2]) * scale, __uint_as_float(v[i + 3]) * scale);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (r0 + i < a.R) out[static_cast<int64_t>(col) * a.R + r0 + i] = __uint_as_float(v[i]) * scale;
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmem);
    }
}

// Split adapters' parts come first in the plan; block y takes part y if an
// adapter begins there.
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
#pragma unroll 4
        for (int q = 1; q < k; ++q) v += s[q * a.slot_stride + at];
        if (i < a.len_a) a.grad_a[first.adapter * a.len_a + i] = v;
        else a.grad_b[first.adapter * a.len_b + i - a.len_a] = v;
    }
}

template <int RP> cudaError_t launch_rp(const GradArgs &a, int parts, cudaStream_t s) {
    auto kern = grad_kernel<RP>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(kern, kSmem<RP>, once, err) != cudaSuccess) return err;
    return launch_pdl_smem(kern, dim3(static_cast<unsigned>(parts * (a.p[0].slices + a.p[1].slices))), dim3(kThreads),
                           kSmem<RP>, s, a);
}

}  // namespace

cudaError_t launch_grad(const GradArgs &args, int parts, cudaStream_t s) {
    GradArgs a = args;
    for (GradProduct &p : a.p) p.slices = (p.C + kCols - 1) / kCols;
    if (a.R <= 16) return launch_rp<16>(a, parts, s);
    if (a.R <= 32) return launch_rp<32>(a, parts, s);
    if (a.R <= 64) return launch_rp<64>(a, parts, s);
    return launch_rp<128>(a, parts, s);
}

cudaError_t launch_sum(const SumArgs &a, cudaStream_t s) {
    const int64_t blocks = (a.len_a + a.len_b + kThreads - 1) / kThreads;
    return launch_pdl(sum_kernel, dim3(static_cast<unsigned>(blocks < 2048 ? blocks : 2048), static_cast<unsigned>(a.n)),
                      dim3(kThreads), s, a);
}

}  // namespace adapter
}  // namespace bt
