// The adapters' gradients (dA = dU^T x, dB = s u^T g): see adapter.cu.
#include "adapter.cuh"

namespace bt {
namespace adapter {
namespace {

// A CTA takes 128 columns of x (or g) and a part of one adapter's tokens, 64 or
// 32 at a time: D (128 columns x twice the rank, fp32, tensor memory) += X^T (U_hi
// | U_lo), and U_rest onto the second half; the halves are added when D is
// read. (fp32 gradients: two 16-bit values of U alone left them 2.5e-6 off, three
// do not show.) Both operands lie as they arrive, a token a row, and go to the
// tensor cores MN-major: nothing is transposed. Eight warps gather, a ninth
// issues the products. A part that is its adapter's only one writes the gradient;
// the others write their sums to the workspace, and whichever ends last adds
// them up in the parts' order: the result does not depend on which that is. Both
// products run in one launch, so that neither leaves the machine half empty at
// its end. x and g are asked for before the previous kernel, which works out
// dU, has ended.
// Bound: x and g, read once. 4096 tokens of 8 adapters, 4096 x 4096, rank 16:
// 26 us alone, 2.6 TB/s, with DRAM, L2 and issue all under half: 704 short CTAs
// (16 stages at most), which wait for their first copies and, where parts are
// summed, for one another's sums. 64 tokens a stage at rank 16, 32 from rank 32
// on, where U takes more of it.
using T = __nv_bfloat16;
constexpr int kCols = 128;
constexpr int kWarps = 9;
template <int RP> constexpr int kTok = RP <= 16 ? 64 : 32;
template <int RP> constexpr int kTokAtom = kTok<RP> * 128;                  // the tokens' rows of 128 bytes
template <int RP> constexpr int kXBytes = 2 * kTokAtom<RP>;                 // 128 columns
template <int RP> constexpr int kUBytes = (3 * RP + 63) / 64 * kTokAtom<RP>;  // hi, lo, rest side by side, 64 ranks an atom
template <int RP> constexpr int kStageBytes = kXBytes<RP> + kUBytes<RP>;
template <int RP> constexpr int kStages = RP <= 16 ? 3 : 4;
template <int RP> constexpr int kLag = kStages<RP> - 2;     // see adapter_shrink.cu
// Sums of their own for the 16-token steps of a stage, see adapter_shrink.cu.
template <int RP> constexpr int kSums = kTok<RP> / 16;
template <int RP> constexpr int kSmem = kStages<RP> * kStageBytes<RP> + 1024;

template <int RP, int MODE>
__global__ void __launch_bounds__(32 * kWarps, RP <= 32 ? 3 : RP <= 64 ? 2 : 1) grad_kernel(const GradArgs a) {
    extern __shared__ uint8_t dyn[];
    constexpr int S = kStages<RP>, D = kLag<RP>, kTmem = kSums<RP> * 2 * RP;
    __shared__ alignas(8) uint64_t full[S], empty[S], done;
    __shared__ uint32_t tmem_slot, abort_flag;
    uint8_t *smem = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int both = a.p[0].slices + a.p[1].slices;
    const int sl = static_cast<int>(blockIdx.x % both);
    const GradProduct &p = a.p[sl < a.p[0].slices ? 0 : 1];
    const int c0 = (sl < a.p[0].slices ? sl : sl - a.p[0].slices) * kCols;
    // The plan, x and g were there before this call's first kernel began, which waited for all before it: only
    // what that kernel writes has to be waited for.
    if (a.alone) pdl_wait();
    const AdapterTile part = a.plan.tiles[blockIdx.x / both];
    const int n = (part.n + kTok<RP> - 1) / kTok<RP>;
    if (warp == kWarps - 1) {
        pdl_wait();                                         // before tensor memory is taken, see shrink_kernel
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
    if (warp < kWarps - 1) {
        const int32_t *rows = a.plan.rows + part.first;
        // this thread's chunks of X: column chunk tid % 16 of tokens tid / 16 + 16 i
        const int cj = tid & 15, ct = tid >> 4;
        constexpr int kMine = kTok<RP> / 16;
        int xrow[kMine];
        auto fetch_rows = [&](int s) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int at = s * kTok<RP> + ct + 16 * i;
                xrow[i] = at < part.n ? rows[at] : -1;
            }
        };
        const int left = p.C - c0 - 8 * cj;
        const uint16_t *x = p.x + c0 + 8 * cj;
        uint4 held[MODE == kRows2 ? kMine : 1];                 // (kRows2) the next stage, on its way
        auto hold = [&]() {
#pragma unroll
            for (int i = 0; i < kMine; ++i)
                held[MODE == kRows2 ? i : 0] = xrow[i] >= 0 && left > 0 ? load8(x + static_cast<int64_t>(xrow[i]) * p.ldx, left)
                                                                        : make_uint4(0u, 0u, 0u, 0u);
        };
        auto load_x = [&](int s) {
            uint8_t *xs = smem + (s % S) * kStageBytes<RP>;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                uint8_t *dst = xs + (cj >> 3) * kTokAtom<RP> + sw128(ct + 16 * i, cj & 7);
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
        };
        fetch_rows(0);
        if (MODE == kRows2) {
            hold();
            fetch_rows(1);
        }
        const int early = n < S ? n : S;                    // every stage once
        for (int s = 0; s < early; ++s) load_x(s);
        pdl_wait();
        __syncthreads();                                    // the barriers and the tensor memory are there
        pdl_launch_dependents();
        for (int s = 0; s < n + D; ++s) {
            if (s < n) {
                if (s >= S) {
                    wait_landed(empty[s % S], static_cast<uint32_t>(s / S - 1) & 1u, &abort_flag, a.err, a.limit_ns);
                    load_x(s);
                }
                uint8_t *us = smem + (s % S) * kStageBytes<RP> + kXBytes<RP>;
                // U: its three values, RP / 8 chunks of a token each
                constexpr int kChunks = kTok<RP> * (RP / 8);
#pragma unroll
                for (int i = 0; i < (3 * kChunks + 255) / 256; ++i) {
                    const int at = tid + 256 * i, part3 = at / kChunks, k = at % kChunks;
                    if (part3 >= 3) break;
                    const int tok = k / (RP / 8), j = k % (RP / 8), row = s * kTok<RP> + tok;
                    const uint16_t *u = part3 == 0 ? p.u.hi : part3 == 1 ? p.u.lo : p.u.rest;
                    const int at8 = part3 * (RP / 8) + j;   // its chunk of the token's row
                    cp_async_16(us + (at8 >> 3) * kTokAtom<RP> + sw128(tok, at8 & 7),
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
    } else {
        tc::fence_before_sync();
        __syncthreads();
    }
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    if (warp == kWarps - 1 && lane == 0) {
        // fp32 sums, bf16 operands, both MN-major, N = 2 RP (hi, lo) or RP (rest), M = 128
        constexpr uint32_t kCommon = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) | ((128u >> 4) << 24);
        constexpr uint32_t kTwo = kCommon | ((static_cast<uint32_t>(2 * RP) >> 3) << 17);
        constexpr uint32_t kOne = kCommon | ((static_cast<uint32_t>(RP) >> 3) << 17);
        // where rest begins: after 2 RP ranks, 64 to an atom, 2 bytes each
        constexpr uint32_t kRest = (2 * RP / 64) * kTokAtom<RP> + (2 * RP % 64) * 2;
        for (int s = 0; s < n; ++s) {
            wait_landed(full[s % S], static_cast<uint32_t>(s / S) & 1u, &abort_flag, a.err, a.limit_ns);
            tc::fence_after_sync();
            const uint32_t xs = smem_u32(smem + (s % S) * kStageBytes<RP>), us = xs + kXBytes<RP>;
#pragma unroll
            for (int k = 0; k < kTok<RP> / 16; ++k) {       // 16 tokens: 16 rows of either operand
                const uint64_t da = tc::sw128_mnmajor_desc(xs + 2048 * k, kTokAtom<RP>);
                const uint32_t d = tmem + k * 2 * RP;
                tc::mma_f16(d, da, tc::sw128_mnmajor_desc(us + 2048 * k, kTokAtom<RP>), kTwo, s != 0);
                tc::mma_f16(d + RP, da, tc::sw128_mnmajor_desc(us + kRest + 2048 * k, kTokAtom<RP>), kOne, 1);
            }
            tc::mma_commit(smem_u32(&empty[s % S]));
        }
        if (n > 0) tc::mma_commit(smem_u32(&done));
        else tc::mbar_arrive(smem_u32(&done));
    }
    __syncwarp();
    wait_landed(done, 0, &abort_flag, a.err, a.limit_ns);
    tc::fence_after_sync();
    float *const grad = p.grad + static_cast<int64_t>(part.adapter) * a.R * p.C;
    if (warp < kWarps - 1) {
        const float scale = p.scale != nullptr ? p.scale[part.adapter] : 1.0f;
        float *out = part.slot >= 0 ? p.slots + part.slot * a.slot_stride : grad;
        const int col = c0 + (warp & 3) * 32 + lane;        // the accumulator's lane
        for (int r0 = (warp >> 2) * 32; r0 < RP; r0 += 64) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            if (n > 0) {
                float small[RP == 16 ? 16 : 32];
#pragma unroll
                for (int q = 0; q < kSums<RP>; ++q) {
                    uint32_t h[32];
                    const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21) + q * 2 * RP + r0;
                    tc::tmem_ld32(at, h);
                    tc::tmem_ld_wait();
                    if constexpr (RP == 16) {               // both halves at once
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            v[i] += __uint_as_float(h[i]);
                            small[i] = q == 0 ? __uint_as_float(h[16 + i]) : small[i] + __uint_as_float(h[16 + i]);
                        }
                    } else {
                        uint32_t l[32];
                        tc::tmem_ld32(at + RP, l);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            v[i] += __uint_as_float(h[i]);
                            small[i] = q == 0 ? __uint_as_float(l[i]) : small[i] + __uint_as_float(l[i]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < (RP == 16 ? 16 : 32); ++i) v[i] = (v[i] + small[i]) * scale;
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
    if (part.slot >= 0) __threadfence();                    // this part's sums, before it is counted
    __syncthreads();
    if (warp == kWarps - 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmem);
    }
    if (part.slot < 0) return;
    // Of a split adapter: its parts lie next to each other in the plan.
    const int here = static_cast<int>(blockIdx.x) / both;
    int first = here, end = here + 1;
    while (first > 0 && a.plan.tiles[first - 1].adapter == part.adapter) --first;
    while (end < a.parts && a.plan.tiles[end].adapter == part.adapter) ++end;
    __shared__ unsigned int before;
    if (tid == 0) before = atomicAdd(a.arrived + static_cast<int64_t>(first) * both + sl, 1u);
    __syncthreads();
    if (before != static_cast<unsigned int>(end - first - 1)) return;
    __threadfence();
    const int cols = min(kCols, p.C - c0), parts = end - first;
    const float *from = p.slots + (part.slot - (here - first)) * a.slot_stride;
    // four values at a time, four parts' on their way at once: of [R, C] 128 columns of every rank, of [C, R] one stretch
    const int64_t base = p.rc ? c0 : static_cast<int64_t>(c0) * a.R, pitch = p.rc ? p.C : 0;
    const int len = p.rc ? cols : cols * a.R, per = (len + 3) / 4, rows_n = p.rc ? a.R : 1;
    const bool whole = ((base | pitch | len | (static_cast<int64_t>(a.R) * p.C)) & 3) == 0;
    for (int i = tid; i < rows_n * per; i += 32 * kWarps) {
        const int r = i / per, k = (i - r * per) * 4;
        const int64_t at = base + r * pitch + k;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int q0 = 0; q0 < parts; q0 += 4) {
            float w[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float *f = from + (q0 + q) * a.slot_stride + at;
                if (whole) {
                    const float4 t = q0 + q < parts ? __ldcg(reinterpret_cast<const float4 *>(f)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    w[q][0] = t.x; w[q][1] = t.y; w[q][2] = t.z; w[q][3] = t.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[q][e] = q0 + q < parts && k + e < len ? __ldcg(f + e) : 0.0f;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] += w[q][e];
        }
        if (whole) {
            *reinterpret_cast<float4 *>(grad + at) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + e < len) grad[at + e] = v[e];
        }
    }
}

template <int RP, int MODE> cudaError_t launch_m(const GradArgs &a, int parts, cudaStream_t s) {
    auto kern = grad_kernel<RP, MODE>;
    static ContextOnce once;
    if (const cudaError_t err = allow_smem(kern, kSmem<RP>, once); err != cudaSuccess) return err;
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
    a.parts = parts;
    if (a.R <= 16) return launch_rp<16>(a, parts, s);
    if (a.R <= 32) return launch_rp<32>(a, parts, s);
    if (a.R <= 64) return launch_rp<64>(a, parts, s);
    return launch_rp<128>(a, parts, s);
}

}  // namespace adapter
}  // namespace bt
