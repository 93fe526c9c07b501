// The adapters' gradients (dA = dU^T x, dB = s u^T g) and the sum of their parts: see adapter.cu.
#include "adapter.cuh"

namespace bt {
namespace adapter {
namespace {

// A CTA takes 128 columns of x (or g) and a part of one adapter's tokens, 64 at
// a time: D (128 columns x twice the rank, fp32, tensor memory) += X^T (U_hi |
// U_lo), the two halves of D being added when it is read. Both operands lie as
// they arrive, a token a row, and go to the tensor cores MN-major: nothing is
// transposed. Eight warps gather, a ninth issues the
// products. A part that is its adapter's only one writes the gradient; the
// others write their sums to the workspace, which sum_kernel adds up in order.
// Both products run in one launch, so that neither leaves the machine half
// empty at its end.
using T = __nv_bfloat16;
constexpr int kCols = 128, kTok = 64;
constexpr int kWarps = 9;
constexpr int kXBytes = 2 * kAtom;                          // 64 tokens x 128 columns
template <int RP> constexpr int kUBytes = (RP <= 32 ? 1 : RP / 32) * kAtom;   // hi and lo side by side, 64 ranks an atom
template <int RP> constexpr int kStageBytes = kXBytes + kUBytes<RP>;
template <int RP> constexpr int kStages = RP <= 32 ? 4 : RP == 64 ? 3 : 4;
template <int RP> constexpr int kLag = kStages<RP> - 2;     // see adapter_shrink.cu
template <int RP> constexpr int kSmem = kStages<RP> * kStageBytes<RP> + 1024;

template <int RP, int MODE>
__global__ void __launch_bounds__(32 * kWarps, RP <= 64 ? 2 : 1) grad_kernel(const GradArgs a) {
    extern __shared__ uint8_t dyn[];
    constexpr int S = kStages<RP>, D = kLag<RP>, kTmem = 2 * RP;
    __shared__ alignas(8) uint64_t full[S], empty[S], done;
    __shared__ uint32_t tmem_slot, abort_flag;
    uint8_t *smem = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int both = a.p[0].slices + a.p[1].slices;
    const int sl = static_cast<int>(blockIdx.x % both);
    const GradProduct &p = a.p[sl < a.p[0].slices ? 0 : 1];
    const int c0 = (sl < a.p[0].slices ? sl : sl - a.p[0].slices) * kCols;
    pdl_wait();                                             // before tensor memory is taken, see shrink_kernel
    const AdapterTile part = a.plan.tiles[blockIdx.x / both];
    if (warp == kWarps - 1) {
        tc::tmem_alloc(smem_u32(&tmem_slot), kTmem);
        tc::tmem_relinquish();
        if (lane == 0) {
            abort_flag = 0;
            for (int i = 0; i < S; ++i) {
                tc::mbar_init(smem_u32(&full[i]), kWarps - 1);
                tc::mbar_init(smem_u32(&empty[i]), 1);
            }
            tc::mbar_init(smem_u32(&done), 1);
            tc::fence_mbar_init();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_slot;
    const int n = (part.n + kTok - 1) / kTok;
    if (warp < kWarps - 1) {
        const int32_t *rows = a.plan.rows + part.first;
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
        const int left = p.C - c0 - 8 * cj;
        const uint16_t *x = p.x + c0 + 8 * cj;
        uint4 held[MODE == kRows2 ? 4 : 1];                 // (kRows2) the next stage, on its way
        auto hold = [&]() {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                held[MODE == kRows2 ? i : 0] = xrow[i] >= 0 && left > 0 ? load8(x + static_cast<int64_t>(xrow[i]) * p.ldx, left)
                                                                        : make_uint4(0u, 0u, 0u, 0u);
        };
        fetch_rows(0);
        if (MODE == kRows2) {
            hold();
            fetch_rows(1);
        }
        for (int s = 0; s < n + D; ++s) {
            if (s < n) {
                if (s >= S) wait_landed(empty[s % S], static_cast<uint32_t>(s / S - 1) & 1u, &abort_flag, a.err, a.limit_ns);
                uint8_t *xs = smem + (s % S) * kStageBytes<RP>, *us = xs + kXBytes;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint8_t *dst = xs + (cj >> 3) * kAtom + sw128(ct + 16 * i, cj & 7);
                    if (MODE == kRows2) {
                        *reinterpret_cast<uint4 *>(dst) = held[MODE == kRows2 ? i : 0];
                    } else {
                        const int valid = xrow[i] >= 0 ? left : 0;
                        copy8<MODE>(dst, valid > 0 ? x + static_cast<int64_t>(xrow[i]) * p.ldx : p.x, valid, p.ax);
                    }
                }
                if (MODE == kRows2) {
                    hold();
                    fetch_rows(s + 2);
                } else {
                    fetch_rows(s + 1);
                }
                // U: its two parts, RP / 8 chunks of 64 tokens
#pragma unroll
                for (int i = 0; i < 2 * kTok * (RP / 8) / 256; ++i) {
                    const int at = tid + 256 * i, part2 = at / (kTok * (RP / 8)), k = at % (kTok * (RP / 8));
                    const int tok = k / (RP / 8), j = k % (RP / 8), row = s * kTok + tok;
                    const uint16_t *u = part2 ? p.u.lo : p.u.hi;
                    const int at8 = part2 * (RP / 8) + j;   // its chunk of the token's row
                    cp_async_16(us + (at8 >> 3) * kAtom + sw128(tok, at8 & 7),
                                row < part.n ? u + static_cast<int64_t>(part.first + row) * RP + 8 * j : u, row < part.n ? 16 : 0);
                }
            }
            cp_async_commit();
            if (s >= D) {                                   // the stage asked for D turns ago has landed
                cp_async_wait<D>();
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(smem_u32(&full[(s - D) % S]));
            }
        }
    } else if (lane == 0) {
        // fp32 sums, bf16 operands, both MN-major, N = 2 RP, M = 128
        constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                                    ((static_cast<uint32_t>(2 * RP) >> 3) << 17) | ((128u >> 4) << 24);
        for (int s = 0; s < n; ++s) {
            wait_landed(full[s % S], static_cast<uint32_t>(s / S) & 1u, &abort_flag, a.err, a.limit_ns);
            tc::fence_after_sync();
            const uint32_t xs = smem_u32(smem + (s % S) * kStageBytes<RP>), us = xs + kXBytes;
#pragma unroll
            for (int k = 0; k < 4; ++k)                     // 16 tokens: 16 rows of either operand
                tc::mma_f16(tmem, tc::sw128_mnmajor_desc(xs + 2048 * k, kAtom), tc::sw128_mnmajor_desc(us + 2048 * k, kAtom), kIdesc,
                            (s | k) != 0);
            tc::mma_commit(smem_u32(&empty[s % S]));
        }
        if (n > 0) tc::mma_commit(smem_u32(&done));
        else tc::mbar_arrive(smem_u32(&done));
    }
    __syncwarp();
    wait_landed(done, 0, &abort_flag, a.err, a.limit_ns);
    tc::fence_after_sync();
    if (warp < kWarps - 1) {
        const float scale = p.scale != nullptr ? p.scale[part.adapter] : 1.0f;
        float *out = part.slot >= 0 ? p.slots + part.slot * a.slot_stride : p.grad + static_cast<int64_t>(part.adapter) * a.R * p.C;
        const int col = c0 + (warp & 3) * 32 + lane;        // the accumulator's lane
        for (int r0 = (warp >> 2) * 32; r0 < RP; r0 += 64) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            if (n > 0) {
                uint32_t h[32];
                tc::tmem_ld32(tmem + (static_cast<uint32_t>(warp & 3) << 21) + r0, h);
                tc::tmem_ld_wait();
                if constexpr (RP == 16) {                   // both halves at once
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = (__uint_as_float(h[i]) + __uint_as_float(h[16 + i])) * scale;
                } else {
                    uint32_t l[32];
                    tc::tmem_ld32(tmem + (static_cast<uint32_t>(warp & 3) << 21) + RP + r0, l);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = (__uint_as_float(h[i]) + __uint_as_float(l[i])) * scale;
                }
            }
            if (col < p.C) {
                if (p.rc) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (r0 + i < a.R) out[static_cast<int64_t>(r0 + i) * p.C + col] = v[i];
                } else if ((a.R & 3) == 0) {
                    float *o = out + static_cast<int64_t>(col) * a.R + r0;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (r0 + i < a.R)
                            *reinterpret_cast<float4 *>(o + i) =
                                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (r0 + i < a.R) out[static_cast<int64_t>(col) * a.R + r0 + i] = v[i];
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kWarps - 1) {
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
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 4;
    // both gradients are laid out in whole 16-byte vectors, but for their last values
    const bool of_a = i < a.off_b;
    const int64_t j = of_a ? i : i - a.off_b, len = of_a ? a.len_a : a.len_b;
    if (j >= len) return;
    float4 v = *reinterpret_cast<const float4 *>(s + i);
#pragma unroll 4
    for (int q = 1; q < k; ++q) {
        const float4 w = *reinterpret_cast<const float4 *>(s + q * a.slot_stride + i);
        v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
    }
    float *o = (of_a ? a.grad_a + first.adapter * a.len_a : a.grad_b + first.adapter * a.len_b) + j;
    if ((len & 3) == 0) {
        *reinterpret_cast<float4 *>(o) = v;
    } else {
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < len) o[e] = f[e];
    }
}

template <int RP, int MODE> cudaError_t launch_m(const GradArgs &a, int parts, cudaStream_t s) {
    auto kern = grad_kernel<RP, MODE>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(kern, kSmem<RP>, once, err) != cudaSuccess) return err;
    return launch_pdl_smem(kern, dim3(static_cast<unsigned>(parts * (a.p[0].slices + a.p[1].slices))), dim3(32 * kWarps),
                           kSmem<RP>, s, a);
}
template <int RP> cudaError_t launch_rp(const GradArgs &a, int parts, cudaStream_t s) {
    switch (rows_mode(a.p[0].ax < a.p[1].ax ? a.p[0].ax : a.p[1].ax)) {
        case kRows16: return launch_m<RP, kRows16>(a, parts, s);
        case kRows4: return launch_m<RP, kRows4>(a, parts, s);
        default: return launch_m<RP, kRows2>(a, parts, s);
    }
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
    const int64_t blocks = (a.off_b + a.len_b + 4 * kThreads - 1) / (4 * kThreads);
    return launch_pdl(sum_kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(a.n)),
                      dim3(kThreads), s, a);
}

}  // namespace adapter
}  // namespace bt
