// The adapters' products that end in the rank (u = A x, dU = s B^T g): see adapter.cu.
#include "adapter.cuh"

namespace bt {
namespace adapter {
namespace {

// A cluster of 1 to 8 CTAs shares a tile of 128 rows, each reducing a piece of
// the long axis on the 5th-generation tensor cores: M = 128 rows, N = the
// rank, fp32 sums in tensor memory. Eight warps gather the rows by 16-byte
// asynchronous copies into the 128-byte swizzle, a ninth issues the products;
// stages are handed over by mbarriers, so that no warp waits for another's
// copies. W needs no transposing for either of its two layouts, the descriptors
// take it K-major or MN-major. The pieces are added in a fixed order through
// distributed shared memory: u leaves once, no partial sum touches memory.
//
// Bound: the long rows, read once. 8192 x 11008 bf16, rank 64: 42 us, 4.3 TB/s,
// with the issue slots half busy (a 16-byte copy and its address for every 8
// elements: rows are gathered, they have no box) and 264 of 304 CTAs' places
// taken. 4096 x 4096, rank 16: 16 us alone, with the join and the beginning as
// long as about six of its stages. (Warp-level matrix instructions kept the tensor
// pipe as long as the rows' reading at rank 64.)
constexpr int kWarps = 9;
constexpr int kXBytes = 2 * kAtom;
template <int RP, bool WT> constexpr int kWBytes = WT ? (RP <= 64 ? 1 : 2) * kAtom : RP * 128;
template <int RP, bool WT> constexpr int kStageBytes = kXBytes + kWBytes<RP, WT>;
template <int RP, bool WT> constexpr int kStages = 100 * 1024 / kStageBytes<RP, WT>;
// A stage is handed over once the one kLag turns later has been asked for, two fewer than there are, so that asking
// never waits for the products of the stage just handed over.
template <int RP, bool WT> constexpr int kLag = kStages<RP, WT> - 2;
// The tensor cores' fp32 sums drop what does not fit instead of rounding it. The 16-element steps of a stage go to
// sums of their own, which are added in fp32 at the end: shorter sums drop less, and not all to one side.
template <int RP> constexpr int kSums = RP <= 64 ? 4 : 2;
template <int RP> constexpr int kSumPitch = RP + 4;
template <int RP, bool WT> constexpr int kSmem = kStages<RP, WT> * kStageBytes<RP, WT> + 1024;
static_assert(kAdapterTile * kSumPitch<128> * 4 <= kStages<128, false> * kStageBytes<128, false>, "sums take the ring's place");
static_assert(kAdapterTile * kSumPitch<128> * 4 <= kStages<128, true> * kStageBytes<128, true>, "sums take the ring's place");

// A row's four values at ranks r .. r + 3 (the row's others lie in the RP / 4 lanes around), split.
template <typename T, int RP>
__device__ __forceinline__ void put_split(const SplitRows &o, int64_t at, int r, const float (&f)[4], bool ok) {
    float p = 1.0f;
    if constexpr (std::is_same<T, __half>::value) {
        float amax = fmaxf(fmaxf(finite_size(f[0]), finite_size(f[1])), fmaxf(finite_size(f[2]), finite_size(f[3])));
#pragma unroll
        for (int d = 1; d < RP / 4; d *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
        p = row_power<T>(amax);
        if (ok && r == 0) o.unpower[at] = 1.0f / p;
    }
    uint2 h, l;
    split2<T>(f[0] * p, f[1] * p, h.x, l.x);
    split2<T>(f[2] * p, f[3] * p, h.y, l.y);
    if (ok) {
        *reinterpret_cast<uint2 *>(o.hi + at * RP + r) = h;
        *reinterpret_cast<uint2 *>(o.lo + at * RP + r) = l;
        if (o.rest != nullptr)
            *reinterpret_cast<uint2 *>(o.rest + at * RP + r) =
                make_uint2(split_rest<T>(f[0] * p, f[1] * p, h.x, l.x), split_rest<T>(f[2] * p, f[3] * p, h.y, l.y));
    }
}

// MODE: how the rows of X and W are fetched.
template <typename T, int RP, bool WT, int MODE>
__global__ void __launch_bounds__(32 * kWarps, 2) shrink_kernel(const ShrinkArgs a) {
    extern __shared__ uint8_t dyn[];
    constexpr int S = kStages<RP, WT>, D = kLag<RP, WT>, kCols = kSums<RP> * RP;
    static_assert(S >= 3 && S <= 8, "stages");
    __shared__ alignas(8) uint64_t full[S], empty[S], done;
    __shared__ uint32_t tmem_slot, abort_flag;
    __shared__ int rows[kAdapterTile];
    uint8_t *smem = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c = a.cluster;
    const int rank = c > 1 ? static_cast<int>(tc::cluster_ctarank()) : 0;
    // Tensor memory is taken after the previous grid has ended and before the
    // next one may start, so that no grid waits for columns of one that waits for it.
    pdl_wait();
    const AdapterTile tile = a.plan.tiles[blockIdx.x / c];
    if (tid < kAdapterTile) rows[tid] = a.plan.rows[tile.first + (tid < tile.n ? tid : 0)];
    if (warp == kWarps - 1) {
        tc::tmem_alloc(smem_u32(&tmem_slot), kCols);
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

    if (blockIdx.x == 0)
        for (int i = tid; i < a.zeros; i += 32 * kWarps) a.zero[i] = 0;
    const int total = (a.C + kStep - 1) / kStep;
    const int s0 = static_cast<int>(static_cast<int64_t>(total) * rank / c);
    const int n = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / c) - s0;
    if (warp < kWarps - 1) {
        const uint16_t *w = a.w + static_cast<int64_t>(tile.adapter) * a.R * (WT ? a.C : a.ldw);
        // this thread's chunks of a stage: column chunk tid % 8 of rows tid / 8 + 32 i
        const int cj = tid & 7, cr = tid >> 3;
        const uint16_t *xr[4];
        bool live[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            live[i] = cr + 32 * i < tile.n;
            xr[i] = a.x + static_cast<int64_t>(rows[cr + 32 * i]) * a.ldx + 8 * cj;
        }
        // its chunk i of stage s: where it goes, where it comes from, how much of it there is
        constexpr int kXChunks = 4, kWChunks = WT ? (kStep * (RP / 8) + 255) / 256 : (RP + 31) / 32;
        auto chunk = [&](int s, int i, uint8_t *&dst, const uint16_t *&src, int &valid) {
            uint8_t *xs = smem + (s % S) * kStageBytes<RP, WT>, *ws = xs + kXBytes;
            const int k0 = (s0 + s) * kStep, left = a.C - k0;
            if (i < kXChunks) {
                valid = live[i] ? left - 8 * cj : 0;
                dst = xs + sw128(cr + 32 * i, cj);
                src = valid > 0 ? xr[i] + k0 : a.x;
            } else if constexpr (!WT) {
                const int r = cr + 32 * (i - kXChunks);
                valid = r < a.R ? left - 8 * cj : 0;
                dst = RP >= 32 || r < RP ? ws + sw128(r, cj) : nullptr;
                src = valid > 0 ? w + static_cast<int64_t>(r) * a.ldw + k0 + 8 * cj : a.w;
            } else {
                // rows of 64 ranks, 64 elements of the long axis to an atom
                const int at = tid + 256 * (i - kXChunks), k = at / (RP / 8), j = at % (RP / 8);
                valid = k < left ? a.R - 8 * j : 0;
                dst = RP >= 32 || k < kStep ? ws + (j >> 3) * kAtom + sw128(k, j & 7) : nullptr;
                src = valid > 0 ? w + static_cast<int64_t>(k0 + k) * a.R + 8 * j : a.w;
            }
        };
        uint4 held[MODE == kRows2 ? kXChunks + kWChunks : 1];    // (kRows2) the next stage, on its way
        auto hold = [&](int s) {
#pragma unroll
            for (int i = 0; i < kXChunks + kWChunks; ++i) {
                uint8_t *dst;
                const uint16_t *src;
                int valid;
                chunk(s, i, dst, src, valid);
                held[MODE == kRows2 ? i : 0] = valid > 0 ? load8(src, valid) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        if (MODE == kRows2) hold(0);
        for (int s = 0; s < n + D; ++s) {
            if (s < n) {
                if (s >= S) wait_landed(empty[s % S], static_cast<uint32_t>(s / S - 1) & 1u, &abort_flag, a.err, a.limit_ns);
#pragma unroll
                for (int i = 0; i < kXChunks + kWChunks; ++i) {
                    uint8_t *dst;
                    const uint16_t *src;
                    int valid;
                    chunk(s, i, dst, src, valid);
                    if (i >= kXChunks && dst == nullptr) continue;
                    if (MODE == kRows2) *reinterpret_cast<uint4 *>(dst) = held[MODE == kRows2 ? i : 0];
                    else copy8<MODE>(dst, src, valid, i < kXChunks ? a.ax : a.aw);
                }
                if (MODE == kRows2 && s + 1 < n) hold(s + 1);
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
        // fp32 sums, bf16 or f16 operands, B MN-major where W is [C, R], N = RP, M = 128
        constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
        constexpr uint32_t kIdesc = (1u << 4) | (kFmt << 7) | (kFmt << 10) | ((WT ? 1u : 0u) << 16) |
                                    ((static_cast<uint32_t>(RP) >> 3) << 17) | ((128u >> 4) << 24);
        for (int s = 0; s < n; ++s) {
            wait_landed(full[s % S], static_cast<uint32_t>(s / S) & 1u, &abort_flag, a.err, a.limit_ns);
            tc::fence_after_sync();
            const uint32_t xs = smem_u32(smem + (s % S) * kStageBytes<RP, WT>), ws = xs + kXBytes;
#pragma unroll
            for (int k = 0; k < 4; ++k) {                   // 16 elements: 32 bytes along a row, or 16 rows
                const uint64_t da = tc::sw128_kmajor_desc(xs + 32 * k);
                const uint64_t db = WT ? tc::sw128_mnmajor_desc(ws + 2048 * k, kAtom) : tc::sw128_kmajor_desc(ws + 32 * k);
                tc::mma_f16(tmem + (k % kSums<RP>) * RP, da, db, kIdesc, s != 0 || k >= kSums<RP>);
            }
            tc::mma_commit(smem_u32(&empty[s % S]));
        }
        tc::mma_commit(smem_u32(&done));
    }
    __syncwarp();
    wait_landed(done, 0, &abort_flag, a.err, a.limit_ns);
    tc::fence_after_sync();
    // the sums, [row][r], where the ring was
    float *sums = reinterpret_cast<float *>(smem);
    if (warp < kWarps - 1) {
        constexpr int kWide = RP < 32 ? RP : 32;            // columns at a time
        for (int col = (warp >> 2) * kWide; col < RP; col += 2 * kWide) {
            float v[kWide];
#pragma unroll
            for (int q = 0; q < kSums<RP>; ++q) {
                // (rank 16: the 32 columns read are this sum and the next)
                uint32_t w[32];
                if (RP >= 32 || (q & 1) == 0) {
                    tc::tmem_ld32(tmem + (static_cast<uint32_t>(warp & 3) << 21) + q * RP + col, w);
                    tc::tmem_ld_wait();
                }
                if constexpr (RP >= 32) {
#pragma unroll
                    for (int i = 0; i < kWide; ++i) v[i] = q == 0 ? __uint_as_float(w[i]) : v[i] + __uint_as_float(w[i]);
                } else if ((q & 1) == 0) {
#pragma unroll
                    for (int i = 0; i < kWide; ++i) {
                        const float two = __uint_as_float(w[i]) + __uint_as_float(w[16 + i]);
                        v[i] = q == 0 ? two : v[i] + two;
                    }
                }
            }
            float *p = sums + ((warp & 3) * 32 + lane) * kSumPitch<RP> + col;
#pragma unroll
            for (int i = 0; i < kWide; i += 4) *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    }
    tc::fence_before_sync();
    if (c > 1) tc::cluster_sync();
    else __syncthreads();
    if (warp == kWarps - 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kCols);
    } else {
        const float mul = a.scale != nullptr ? a.scale[tile.adapter] : 1.0f;
        const int r0 = kAdapterTile * rank / c, r1 = kAdapterTile * (rank + 1) / c;
        // whole warps: 128 / 8 rows of RP / 4 lanes
        for (int i = tid; i < (r1 - r0) * (RP / 4); i += 32 * (kWarps - 1)) {
            const int row = r0 + i / (RP / 4), r = (i % (RP / 4)) * 4;
            const bool ok = row < tile.n;
            const float *at = sums + row * kSumPitch<RP> + r;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c == 1) {
                v = *reinterpret_cast<const float4 *>(at);
            } else {
#pragma unroll 4
                for (int q = 0; q < c; ++q) {
                    float4 p;
                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w) : "r"(tc::mapa(smem_u32(at), q)) : "memory");
                    v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
                }
            }
            float f[4] = {v.x * mul, v.y * mul, v.z * mul, v.w * mul};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (r + e >= a.R) f[e] = 0.0f;              // an infinity among X makes NaN of it and the padding's zeros
            if (a.u != nullptr && ok) {
                float *u = a.u + static_cast<int64_t>(rows[row]) * a.R + r;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (r + e < a.R) u[e] = f[e];
            }
            put_split<T, RP>(a.out, tile.first + row, r, f, ok);
            if constexpr (WT) {
                const float *u = a.given + static_cast<int64_t>(rows[row]) * a.R + r;
                float g[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = ok && r + e < a.R ? u[e] : 0.0f;
                put_split<T, RP>(a.given_out, tile.first + row, r, g, ok);
            }
        }
    }
    if (c > 1) tc::cluster_sync();                          // nobody leaves while its sums are read
}

__global__ void __launch_bounds__(kThreads) align_kernel(const AlignArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int chunks = (a.C + 7) / 8;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    auto copy = [&](int64_t first, int64_t rows) {
#pragma unroll 4
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < rows * chunks; i += step) {
            const int64_t row = first + i / chunks;
            const int j = static_cast<int>(i % chunks) * 8;
            *reinterpret_cast<uint4 *>(a.dst + row * a.ldd + j) = load8(a.src + row * a.lds + j, a.C - j);
        }
    };
    if (a.parts == nullptr) return copy(0, a.rows);
    for (int i = blockIdx.y; i < a.nparts; i += gridDim.y) {
        const AdapterTile part = a.parts[i];
        if (part.n == 0) return;                            // adapters without tokens come last
        if (i == 0 || a.parts[i - 1].adapter != part.adapter) copy(static_cast<int64_t>(part.adapter) * a.R, a.R);
    }
}

template <typename T, int RP, bool WT, int MODE> cudaError_t launch_m(ShrinkArgs a, int tiles, cudaStream_t s) {
    auto kern = shrink_kernel<T, RP, WT, MODE>;
    static ContextOnce once;
    if (const cudaError_t err = allow_smem(kern, kSmem<RP, WT>, once); err != cudaSuccess) return err;
    // CTAs a tile, as many as end soonest: in waves of two CTAs an SM, each of its steps and of what it
    // costs to begin, join and end, about six steps' time. (Half precision joins rows by whole warps:
    // powers of two.)
    const int steps = (a.C + kStep - 1) / kStep, slots = 2 * device_sm_count();
    int64_t best = 0;
    for (int c = 1; c <= 8; ++c) {
        if (std::is_same<T, __half>::value && (c & (c - 1)) != 0) continue;
        const int64_t waves = (static_cast<int64_t>(tiles) * c + slots - 1) / slots, cost = waves * ((steps + c - 1) / c + 6);
        if (c == 1 || (cost < best && steps >= 2 * c)) {
            best = cost;
            a.cluster = c;
        }
    }
    return launch_cluster(kern, tiles * a.cluster, a.cluster, 32 * kWarps, kSmem<RP, WT>, s, static_cast<const ShrinkArgs>(a));
}
template <typename T, int RP, bool WT> cudaError_t launch_rp(const ShrinkArgs &a, int tiles, cudaStream_t s) {
    switch (rows_mode(a.ax < a.aw ? a.ax : a.aw)) {
        case kRows16: return launch_m<T, RP, WT, kRows16>(a, tiles, s);
        case kRows4: return launch_m<T, RP, WT, kRows4>(a, tiles, s);
        default: return launch_m<T, RP, WT, kRows2>(a, tiles, s);
    }
}
template <typename T, bool WT> cudaError_t launch_t(const ShrinkArgs &a, int tiles, cudaStream_t s) {
    if (a.R <= 16) return launch_rp<T, 16, WT>(a, tiles, s);
    if (a.R <= 32) return launch_rp<T, 32, WT>(a, tiles, s);
    if (a.R <= 64) return launch_rp<T, 64, WT>(a, tiles, s);
    return launch_rp<T, 128, WT>(a, tiles, s);
}

}  // namespace

cudaError_t launch_align(const AlignArgs &a, cudaStream_t s) {
    const int64_t total = (a.parts != nullptr ? a.R : a.rows) * ((a.C + 7) / 8);
    if (total == 0) return cudaSuccess;
    const int64_t blocks = (total + 4 * kThreads - 1) / (4 * kThreads), most = 8 * device_sm_count();
    const int parts = a.parts == nullptr ? 1 : a.nparts < 1024 ? a.nparts : 1024;
    return launch_pdl(align_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most), static_cast<unsigned>(parts)), dim3(kThreads), s, a);
}

cudaError_t launch_shrink(bt_dtype t, bool wt, const ShrinkArgs &a, int tiles, cudaStream_t s) {
    if (tiles == 0) return cudaSuccess;
    if (wt) return launch_t<__nv_bfloat16, true>(a, tiles, s);
    return t == BT_F16 ? launch_t<__half, false>(a, tiles, s) : launch_t<__nv_bfloat16, false>(a, tiles, s);
}

}  // namespace adapter
}  // namespace bt
