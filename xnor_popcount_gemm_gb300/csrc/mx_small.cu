// The product of microscaled operands for few rows of x (a token of every request): bound by the weights' bytes and by
// latency. The weights take the MMA's 128 rows and x its columns (16 or 32), so that nothing is spent on rows that are not there:
//   D [128 rows of W, 32 of x] = sum over this CTA's slices of K
// and a cluster of up to 8 CTAs shares a tile's K, joining its parts through distributed shared memory in the CTAs'
// order. Up to 16 rows of x are quantised where they are used: two warps take a slice of all rows (8 KB of bf16 at 16 rows
// and 256 values), which costs less than a launch for it, and the codes never leave shared memory. One row by 4096 x 4096,
// E2M1, weights out of DRAM: 4.3 us (5.7 with x quantised first), 16 rows 6.5 (6.9); by 11008 x 4096 7.6 (8.6) and 11.9 (11.0).
// More rows, up to 32, come as an operand: 8.1 us and 13.0 with x quantised first (9.2 and 18.7 where each CTA did it, not kept;
// by 11008 x 4096 tiles of 128 rows, which take those, 11.3).
//   warp 0 lane 0   TMA: weights and their scales, a slice a stage
//   warp 1          scales to TMEM, the slice's four MMAs
//   warps 2..9      x to codes and scales, two warps a stage, half of the rows each; then (four of them) the epilogue
// Two CTAs an SM with 80 KB each on their way. One row by 11008 x 4096, weights out of DRAM: 172 CTAs, 3.2 TB/s; what is left is the launch, a trip to memory
// and the join. The weights' boxes asked into L2 before the grid before has ended: 8.0 us instead of 7.6.
#include "mx_linear.cuh"

namespace bt {
namespace {

using namespace mx;

constexpr int kRows = 128;                      // of W
constexpr int kXWarps = 8;                      // two a stage
constexpr int kThreads = 64 + 32 * kXWarps;
constexpr int kStages = kXWarps / 2;
constexpr uint32_t kTmemCols = 64;              // 32 of sums, two sets of 16 of scales
constexpr uint32_t kSfCol = 32;

__host__ __device__ constexpr int w_bytes(int code) { return kRows * kSliceBytes + atoms_a_slice(code) * kAtomBytes; }
__host__ __device__ constexpr int x_bytes(int code, int nb) { return nb * kSliceBytes + atoms_a_slice(code) * kAtomBytes; }

struct SmallArgs {
    const void *x;
    const uint8_t *xs;
    int64_t ldx, atoms, row_bytes;              // atoms, row_bytes: of an operand x
    int f16;                                    // 2-byte x: half precision
    int wide;                                   // x's rows start at 16-byte multiples
    int M, N, K, slices;
    int split;                                  // CTAs of a cluster
    uint32_t idesc;
    void *out;
    int out_t;
    int64_t ldo;
    unsigned int *err;
    unsigned long long wait_ns;
};

__device__ __forceinline__ void st_shared(uint32_t a, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void st_shared16(uint32_t a, const uint4 &v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// XB: bytes of an element of x; 0: x is an operand.
template <int XB> struct X8 { uint4 a, b; };
template <> struct X8<2> { uint4 a; };

template <int XB> __device__ __forceinline__ X8<XB> load_x(const SmallArgs &a, int row, int k) {
    X8<XB> r = {};
    if (row >= a.M || k >= a.K) return r;
    const uint8_t *p = static_cast<const uint8_t *>(a.x) + (row * a.ldx + k) * XB;
    if (a.wide && k + 8 <= a.K) {
        r.a = *reinterpret_cast<const uint4 *>(p);
        if constexpr (XB == 4) r.b = *reinterpret_cast<const uint4 *>(p + 16);
        return r;
    }
    uint32_t w[8] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (k + e >= a.K) continue;
        if constexpr (XB == 4) w[e] = reinterpret_cast<const uint32_t *>(p)[e];
        else w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[e]) << (16 * (e & 1));
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (XB == 4) r.b = make_uint4(w[4], w[5], w[6], w[7]);
    return r;
}
template <int XB> __device__ __forceinline__ void values_of(const SmallArgs &a, const X8<XB> &r, float (&v)[8]) {
    if constexpr (XB == 4) {
        Elem<float>::unpack(r.a, v);
        Elem<float>::unpack(r.b, v + 4);
    } else {
        if (a.f16) Elem<__half>::unpack(r.a, v);
        else Elem<__nv_bfloat16>::unpack(r.a, v);
    }
}

template <int XB> __device__ __forceinline__ uint32_t top_of(const SmallArgs &a, const X8<XB> &r) {
    if constexpr (XB == 4) return quad_top<float>(Raw8<float>{r.a, r.b});
    else return a.f16 ? quad_top<__half>(Raw8<__half>{r.a}) : quad_top<__nv_bfloat16>(Raw8<__nv_bfloat16>{r.a});
}

// Slice `slice` of the rows of x from `from` on, NB / 2 of them, as the MMA takes it: codes in rows of 128 bytes in the 128-byte swizzle, atoms of scales.
// ready(): waits for the stage; false: it ran out.
template <int CODE, int NB, int XB, typename F>
__device__ __forceinline__ void x_slice(const SmallArgs &a, int slice, int from, uint32_t codes, uint32_t atoms, int lane, F ready) {
    constexpr int kAtoms = atoms_a_slice(CODE);
    auto at = [&](int row, int byte) { return codes + static_cast<uint32_t>(row * 128 + ((((byte >> 4) ^ row) & 7) << 4) + (byte & 15)); };
    if constexpr (XB == 0) {
        const int row0 = from + (lane >> 3), c = (lane & 7) * 16, own = from + lane;
        const bool has = lane < NB / 2 && own < a.M;
        uint4 q[NB / 8];
        uint32_t s[kAtoms];
#pragma unroll
        for (int i = 0; i < NB / 8; ++i) {
            const int row = row0 + 4 * i;
            q[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < a.M) q[i] = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.x) + row * a.row_bytes + static_cast<int64_t>(slice) * 128 + c);
        }
#pragma unroll
        for (int j = 0; j < kAtoms; ++j)
            s[j] = has ? *reinterpret_cast<const uint32_t *>(a.xs + scale_at(own, (static_cast<int64_t>(slice) * kAtoms + j) * 4, a.atoms)) : 0u;
        if (!ready()) return;
#pragma unroll
        for (int i = 0; i < NB / 8; ++i)
            if (row0 + 4 * i < a.M) st_shared16(at(row0 + 4 * i, c), q[i]);
#pragma unroll
        for (int j = 0; j < kAtoms; ++j)
            if (has) st_shared(atoms + j * kAtomBytes + own * 16, s[j]);
    } else {
        constexpr int kG = 128 / Format<CODE>::kBytes8, kPer = 32 / kG;       // eights of a row; rows at a time
        constexpr int kIn = XB == 4 ? 4 : 8;                                  // loads in flight
        const int g = lane % kG, row0 = lane / kG;
        const int k = slice * kG * 8 + g * 8;
        const int end = a.M < from + NB / 2 ? a.M : from + NB / 2;
        bool first = true;
#pragma unroll 1
        for (int r0 = from; r0 < end || first; r0 += kPer * kIn) {
            X8<XB> raw[kIn];
#pragma unroll
            for (int i = 0; i < kIn; ++i) raw[i] = load_x<XB>(a, r0 + i * kPer + row0 < end ? r0 + i * kPer + row0 : a.M, k);
            if (first && !ready()) return;
            first = false;
#pragma unroll
            for (int i = 0; i < kIn; ++i) {
                const int row = r0 + i * kPer + row0;
                if (r0 + i * kPer >= end) break;                              // (the same for all lanes)
                float v[8];
                const uint32_t top = top_of<XB>(a, raw[i]);
                values_of<XB>(a, raw[i], v);
                if (row >= end) continue;
                const uint32_t s = scale_of<CODE>(top);
                const uint2 c = code8<CODE>(v, inverse_of(s));
                const uint32_t to = at(row, g * Format<CODE>::kBytes8);
                st_shared(to, c.x);
                if constexpr (CODE == BT_CODE_E4M3) st_shared(to + 4, c.y);
                if ((lane & 3) == 0) {
                    const int b = g >> 2;
                    asm volatile("st.shared.u8 [%0], %1;" ::"r"(atoms + static_cast<uint32_t>((b >> 2) * kAtomBytes + row * 16 + (b & 3))), "r"(s) : "memory");
                }
            }
        }
    }
}

template <int CODE, int NB, int XB>
__global__ void __launch_bounds__(kThreads, 2)
mx_small_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS, const SmallArgs a) {
    constexpr int kAtoms = atoms_a_slice(CODE);
    constexpr bool kE2M1 = CODE == BT_CODE_E2M1;
    constexpr uint32_t kWTile = kRows * kSliceBytes, kXTile = NB * kSliceBytes, kSf = kAtoms * kAtomBytes;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[3 * kStages + 1];
    __shared__ uint32_t slot_word, abort_word;
    const uint32_t raw = smem_u32(smem_raw);
    // tiles of W, tiles of x, scales of W, scales of x
    const uint32_t sW = (raw + 1023u) & ~1023u, sX = sW + kStages * kWTile, sSw = sX + kStages * kXTile, sSx = sSw + kStages * kSf;
    auto w_full = [&](int s) { return smem_u32(&bars[s]); };            // the weights' bytes
    auto x_full = [&](int s) { return smem_u32(&bars[kStages + s]); };  // x's codes and scales
    auto empty = [&](int s) { return smem_u32(&bars[2 * kStages + s]); };
    const uint32_t done = smem_u32(&bars[3 * kStages]);
    volatile uint32_t *abort_flag = &abort_word;
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x % a.split), n0 = static_cast<int>(blockIdx.x / a.split) * kRows;
    // this CTA's slices: as many as the others', or one more
    const int per = a.slices / a.split, more = a.slices % a.split;
    const int k0 = rank * per + (rank < more ? rank : more), cnt = per + (rank < more ? 1 : 0);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(w_full(s), 1);
            tc::mbar_init(x_full(s), 2);
            tc::mbar_init(empty(s), 1);
        }
        tc::mbar_init(done, 1);
        abort_word = 0u;
        tc::fence_mbar_init();
        tc::prefetch_map(&tmW);
        tc::prefetch_map(&tmS);
    }
    // Tensor memory is taken after the grids before this one have ended and before the next may begin: none waits for
    // columns that are held by one that waits for it.
    pdl_wait();
    if (warp == 1) {
        tc::tmem_alloc(smem_u32(&slot_word), kTmemCols);
        tc::tmem_relinquish();
    }
    // rows of x that are not there are zeros in every stage
    for (uint32_t i = threadIdx.x * 16; i < kStages * kXTile; i += kThreads * 16) st_shared16(sX + i, make_uint4(0u, 0u, 0u, 0u));
    for (uint32_t i = threadIdx.x * 16; i < kStages * kSf; i += kThreads * 16) st_shared16(sSx + i, make_uint4(0u, 0u, 0u, 0u));
    tc::fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *static_cast<volatile uint32_t *>(&slot_word), 0);

    if (warp == 0) {
        if (lane == 0) {
            int i = 0;
            for (; i < cnt; ++i) {
                const int s = i % kStages;
                if (!tc::wait_fast(empty(s), static_cast<uint32_t>(i / kStages & 1) ^ 1u, abort_flag, a.err, a.wait_ns)) break;
                tc::mbar_arrive_expect_tx(w_full(s), kWTile + kSf);
                tc::tma_load_3d(sW + s * kWTile, &tmW, 0, n0, k0 + i, w_full(s));
                tc::tma_load_3d(sSw + s * kSf, &tmS, 0, (k0 + i) * kAtoms, n0 / kRows, w_full(s));
            }
            // whatever happens elsewhere, what was asked for lands before shared memory is given back
            for (int j = i > kStages ? i - kStages : 0; j < i; ++j) {
                uint32_t never = 0;
                if (!tc::wait_bounded(w_full(j % kStages), static_cast<uint32_t>(j / kStages & 1), &never, a.err)) break;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t me = tc::elect_one();
        const uint64_t op0 = tc::sw128_kmajor_desc(0), sf0 = tc::scale_atom_desc(0);
        uint32_t id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) id[k] = with_id(a.idesc, kE2M1 ? 2 * (k & 1) : k);
        int s = 0;
        uint32_t ph = 0, turn = 0;
        for (int i = 0; i < cnt; ++i) {
            if (!tc::wait_warp(w_full(s), ph, abort_flag, a.err, a.wait_ns) || !tc::wait_warp(x_full(s), ph, abort_flag, a.err, a.wait_ns)) break;
            tc::fence_after_sync();
            const uint32_t sfa = tmem + kSfCol + (turn ^= 16u), sfb = sfa + 4 * kAtoms;
#pragma unroll
            for (int j = 0; j < kAtoms; ++j) {
                tc::cp_scales<false>(me, sfa + 4 * j, sf0 + ((sSw + s * kSf + j * kAtomBytes) >> 4));
                tc::cp_scales<false>(me, sfb + 4 * j, sf0 + ((sSx + s * kSf + j * kAtomBytes) >> 4));
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t fa = kE2M1 ? sfa + 4 * (kk >> 1) : sfa, fb = kE2M1 ? sfb + 4 * (kk >> 1) : sfb;
                tc::mma_scaled<kE2M1, false>(me, tmem, op0 + ((sW + s * kWTile + kk * 32) >> 4), op0 + ((sX + s * kXTile + kk * 32) >> 4),
                                             id[kE2M1 ? kk & 1 : kk], fa, fb, (i | kk) != 0 ? 1u : 0u);
            }
            tc::commit_warp<false>(me, empty(s), 0);
            if (++s == kStages) { s = 0; ph ^= 1u; }
        }
        // also after a wait that ran out: what was issued has ended before anything is given back
        tc::commit_warp<false>(me, done, 0);
    } else {
        // (a warp sees every use of its stage: a barrier's phase is known by its parity alone)
        const int s = (warp - 2) % kStages, from = (warp - 2) / kStages * (NB / 2);
        for (int i = s; i < cnt; i += kStages) {
            bool ok = true;
            x_slice<CODE, NB, XB>(a, k0 + i, from, sX + s * kXTile, sSx + s * kSf, lane, [&] {
                ok = tc::wait_warp(empty(s), static_cast<uint32_t>(i / kStages & 1) ^ 1u, abort_flag, a.err, a.wait_ns);
                return ok;
            });
            if (!ok) break;
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(x_full(s));
        }
    }

    // The sums: through shared memory (the stages are free then), [row of x][row of W].
    float *part = reinterpret_cast<float *>(smem_raw + (sW - raw));
    uint32_t never = 0;                                         // (also where a wait ran out: what was issued ends first)
    bool ok = tc::wait_warp(done, 0u, &never, a.err, kWaitNs);
    __syncthreads();
    ok = ok && *abort_flag == 0u;
    const int quarter = warp & 3;
    if (warp >= 2 && warp < 6 && ok) {
        tc::fence_after_sync();
        uint32_t r[32];
        tc::tmem_ld32(tmem + (static_cast<uint32_t>(quarter * 32) << 16), r);
        tc::tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < NB; ++t)
            if (t < a.M) part[t * kRows + quarter * 32 + lane] = __uint_as_float(r[t]);
        tc::fence_before_sync();
    }
    if (a.split > 1) tc::cluster_sync();
    else __syncthreads();
    if (warp >= 2 && warp < 6) {
        const int n = n0 + quarter * 32 + lane;
        const uint32_t mine = smem_u32(part) + static_cast<uint32_t>((quarter * 32 + lane) * 4);
        // rows of x by the cluster's CTAs in turn
        for (int t = rank; t < a.M && ok; t += a.split) {
            float v = 0.0f;
            if (a.split == 1) {
                v = part[t * kRows + quarter * 32 + lane];
            } else {
                float p[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    p[c] = 0.0f;
                    if (c < a.split)
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p[c]) : "r"(tc::mapa(mine + static_cast<uint32_t>(t * kRows * 4), static_cast<uint32_t>(c))) : "memory");
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) v += p[c];
            }
            if (n >= a.N) continue;
            const int64_t o = t * a.ldo + n;
            if (a.out_t == BT_F32) static_cast<float *>(a.out)[o] = v;
            else if (a.out_t == BT_BF16) static_cast<__nv_bfloat16 *>(a.out)[o] = __float2bfloat16_rn(v);
            else static_cast<__half *>(a.out)[o] = __float2half_rn(v);
        }
    }
    __syncthreads();
    if (a.split > 1) tc::cluster_sync();                        // nobody leaves while others read its parts
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

template <int CODE, int NB, int XB> cudaError_t launch(const Product &p, int split, cudaStream_t s) {
    SmallArgs a = {};
    a.x = p.x; a.xs = p.xs;
    a.ldx = p.ldx;
    a.atoms = k_atoms(p.K, CODE);
    a.row_bytes = code_bytes(p.K, CODE);
    a.f16 = p.x_t == BT_F16;
    a.wide = XB != 0 && aligned(p.x, 16) && (p.ldx * XB) % 16 == 0;
    a.M = static_cast<int>(p.M); a.N = static_cast<int>(p.N); a.K = static_cast<int>(p.K);
    a.slices = static_cast<int>(slices(p.K, CODE));
    const int64_t tiles = (p.N + kRows - 1) / kRows;
    if (split == 0) {
        split = 1;
        while (split < 8 && tiles * split * 2 <= 2 * device_sm_count()) split *= 2;
    }
    while (split > a.slices) split /= 2;
    a.split = split;
    a.idesc = make_idesc(CODE, kRows, NB);
    a.out = p.out; a.out_t = p.out_t; a.ldo = p.ldo;
    a.err = p.err;
    a.wait_ns = wait_limit_ns();
    CUtensorMap mw, ms;
    if (!map_codes(&mw, p.w, p.N, a.slices, kRows, 1) || !map_scales(&ms, p.ws, p.N, a.atoms, 1, atoms_a_slice(CODE))) return cudaErrorInvalidValue;
    auto kern = mx_small_kernel<CODE, NB, XB>;
    const int smem = kStages * (w_bytes(CODE) + x_bytes(CODE, NB)) + 1024;
    static ContextOnce once;
    if (const cudaError_t e = allow_smem(kern, smem, once); e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, mw, ms, static_cast<const SmallArgs>(a));
}
template <int CODE> cudaError_t launch_rows(const Product &p, int split, cudaStream_t s) {
    if (p.M > kOwnRows) return p.x_t == BT_PACKED ? launch<CODE, kSmallRows, 0>(p, split, s) : cudaErrorInvalidValue;   // (quantised before)
    return p.x_t == BT_PACKED ? launch<CODE, kOwnRows, 0>(p, split, s)
           : p.x_t == BT_F32  ? launch<CODE, kOwnRows, 4>(p, split, s)
                              : launch<CODE, kOwnRows, 2>(p, split, s);
}

}  // namespace

cudaError_t mx::launch_small(const Product &p, int split, cudaStream_t s) {
    return p.code == BT_CODE_E2M1 ? launch_rows<BT_CODE_E2M1>(p, split, s) : launch_rows<BT_CODE_E4M3>(p, split, s);
}

}  // namespace bt
