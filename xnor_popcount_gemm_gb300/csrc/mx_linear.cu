// Y = X W^T on microscaled operands (see mx.cuh): E2M1 x E2M1 or E4M3 x E4M3, the blocks' scales applied by the tensor
// cores, fp32 sums in TMEM.
//
// Persistent and warp-specialised, one CTA per SM; tiles of 128 rows by BN columns (256 or 128), or, on CTA pairs (tcgen05
// cta_group::2), 256 by BN: each CTA brings its 128 rows of X and half of the tile's rows of W, and the scales of its rows
// of X and of all the tile's rows of W.
//   warp 0 lane 0   TMA: stages of D 128-byte slices of K, operands (128-byte swizzle) and atoms of scales
//   warp 1          scales of a slice to TMEM (tcgen05.cp), its four MMAs
//   warps 2..9      epilogue: two (or one) a TMEM lane quarter, 32 columns at a time, through shared memory so that whole
//                   row pieces are stored
// TMEM: two accumulators and two times 32 columns of scales. At BN = 256 the accumulators share 64 columns: a tile's
// epilogue takes those first, and the next tile's MMAs begin when they are free.
//
// What bounds it: 8192 x 4096 x 11008 in E2M1 takes 100 us on pairs (7400 TFLOP/s), 640 clocks a slice where its MMAs need 512 and
// its shared-memory traffic (copies in, operands out) about 650; the tensor pipe is 71 % busy. E4M3 204 to 230 us, by the
// clock under load. Getting there: the issue of MMAs and copies from a whole warp with its operands in uniform registers
// (tc_ptx.cuh) 160 -> 104 us. Copies of scales run in order with the MMAs and need no barrier. Not kept, same size: the
// scales by tcgen05.st from four warps (a store waits about 1000 clocks under an MMA; 250 us on pairs), copies from a
// warp of their own (157), a slice ahead of their MMAs (244), two slices' at once (175).
// Every wait is bounded, as in the other tensor-core kernels.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "adapter.cuh"
#include "mx_linear.cuh"

namespace bt {
namespace {

using namespace mx;

constexpr int kBM = 128;
constexpr int kRowB = 128;
constexpr int kEpiWarps = 8;                    // at most
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol = 448;                // two times 32 columns: at most 2 atoms x (4 of X + 8 of W)
constexpr int kReserve = 1024 + 256;            // alignment, barriers
constexpr int kMaxStages = 8;
__host__ __device__ constexpr int staging_bytes(int elem, int epi) { return epi * 32 * 32 * elem; }
// Rows of W that a CTA brings.
__host__ __device__ constexpr int b_rows(int bn, bool pair) { return pair ? bn / 2 : bn; }
__host__ __device__ __forceinline__ int slice_bytes(int code, int bn, bool pair) {
    return (kBM + b_rows(bn, pair)) * kRowB + atoms_a_slice(code) * (1 + bn / 128) * kAtomBytes;
}

struct MxArgs {
    int64_t M, N, ldo;
    int slices, d, nk, stages;                  // slices of K, of a stage; stages of a tile, of the ring
    int bn, num_n, num_tiles, epi;              // epi: epilogue warps, 4 or 8
    uint32_t idesc;
    void *out;
    int vec;                                    // out's rows start at 16-byte multiples and N is a whole number of 16 bytes
    unsigned int *err;
    unsigned long long wait_ns;
};

template <typename T> __device__ __forceinline__ uint4 chunk16(const uint32_t (&r)[32], int j0) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(r[j0], r[j0 + 1], r[j0 + 2], r[j0 + 3]);
    } else {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[j0 + e]);
        return raw_pack<T>(v).a;
    }
}
// 16-byte chunk q of a staged row: swizzled, so that 32 lanes writing their rows' chunk q meet different banks.
template <int ELEM> __device__ __forceinline__ uint32_t box_chunk(int q, int row) {
    return ELEM == 4 ? static_cast<uint32_t>(q ^ (row & 7)) : static_cast<uint32_t>(q ^ ((row >> 1) & 3));
}

template <int CODE, typename T, bool PAIR, int BN>
__global__ void __launch_bounds__(kThreads, 1)
mx_linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb, const MxArgs a) {
    constexpr int kElem = sizeof(T);
    constexpr int kBoxInner = 32 * kElem;
    constexpr int kAtoms = atoms_a_slice(CODE);
    constexpr bool kE2M1 = CODE == BT_CODE_E2M1;
    constexpr uint32_t kASlice = kBM * kRowB;
    constexpr int bn = BN;
    const int S = a.stages, D = a.d;
    constexpr uint32_t kBSlice = static_cast<uint32_t>(b_rows(bn, PAIR) * kRowB);
    const uint32_t kSaStage = static_cast<uint32_t>(kAtoms * D * kAtomBytes), kSbStage = kSaStage * static_cast<uint32_t>(bn / 128);

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sA = (raw + 1023u) & ~1023u, sB = sA + S * kASlice * D;
    const uint32_t sSa = sB + S * kBSlice * D, sSb = sSa + S * kSaStage;
    const uint32_t sStage = sSb + S * kSbStage;
    const uint32_t bars = sStage + staging_bytes(kElem, a.epi);
    uint8_t *gbars = smem_raw + (bars - raw);
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(gbars + 8 * (2 * kMaxStages + 6));
    volatile uint32_t *abort_flag = tmem_slot + 1;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kMaxStages + s); };
    auto tfull = [&](int b) { return bars + 8u * (2 * kMaxStages + b); };       // accumulator b written
    auto tempty = [&](int b) { return bars + 8u * (2 * kMaxStages + 2 + b); };  // accumulator b read
    const uint32_t shared_read = bars + 8u * (2 * kMaxStages + 4);              // a tile's shared columns read
    const uint32_t drain = bars + 8u * (2 * kMaxStages + 5);

    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t crank = PAIR ? __shfl_sync(0xFFFFFFFFu, tc::cluster_ctarank(), 0) : 0u;
    const bool leader = !PAIR || crank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(full(s), 1);
            tc::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(tfull(b), 1);
            tc::mbar_init(tempty(b), (PAIR ? 2 : 1) * a.epi);
        }
        tc::mbar_init(shared_read, (PAIR ? 2 : 1) * a.epi);
        tc::mbar_init(drain, 1);
        *abort_flag = 0u;
        tc::fence_mbar_init();
        tc::prefetch_map(&tmA);
        tc::prefetch_map(&tmB);
        tc::prefetch_map(&tmSa);
        tc::prefetch_map(&tmSb);
    }
    // Tensor memory is taken after the grids before this one have ended and before the next may begin: none waits for
    // columns that are held by one that waits for it.
    pdl_wait();
    if (warp == 1) {
        if (PAIR) {
            tc::tmem_alloc_pair(smem_u32(const_cast<uint32_t *>(tmem_slot)), kTmemCols);
            tc::tmem_relinquish_pair();
        } else {
            tc::tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), kTmemCols);
            tc::tmem_relinquish();
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (PAIR) tc::cluster_sync();
    tc::fence_after_sync();
    if (threadIdx.x == 0) pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
    constexpr bool shared = bn == 256;                      // the accumulators overlap
    auto acc_col = [&](int buf) { return static_cast<uint32_t>(buf) * (shared ? 192u : 256u); };

    const int unit = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int nunits = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);
    const int tile_rows = PAIR ? 2 * kBM : kBM;
    auto slice_count = [&](int kb) { return a.slices - kb * D < D ? a.slices - kb * D : D; };

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>((PAIR ? 2 : 1) * D) * ((kASlice + kBSlice) + static_cast<uint32_t>(kAtoms * (1 + bn / 128) * kAtomBytes));
            int s = 0;
            uint32_t ph = 0, last_phase[kMaxStages];
#pragma unroll
            for (int i = 0; i < kMaxStages; ++i) last_phase[i] = 2u;
            bool ok = true;
            for (int tl = unit; tl < a.num_tiles && ok; tl += nunits) {
                const int mt = tl / a.num_n, nt = tl % a.num_n;
                const int am = mt * tile_rows + static_cast<int>(crank) * kBM, bm = nt * bn + static_cast<int>(crank) * b_rows(bn, PAIR);
                for (int kb = 0; kb < a.nk; ++kb) {
                    if (!tc::wait_fast(empty(s), ph ^ 1u, abort_flag, a.err, a.wait_ns)) { ok = false; break; }
                    if (leader) tc::mbar_arrive_expect_tx(full(s), bytes);
                    // whole boxes always: slices and rows past the end are filled with zeros
                    const int k0 = kb * D;
                    const uint32_t ad = sA + s * kASlice * D, bd = sB + s * kBSlice * D, sa = sSa + s * kSaStage, sb = sSb + s * kSbStage;
                    if (PAIR) {
                        const uint32_t bar = tc::mapa(full(s), 0u);
                        tc::tma_load_3d_pair(ad, &tmA, 0, am, k0, bar);
                        tc::tma_load_3d_pair(bd, &tmB, 0, bm, k0, bar);
                        tc::tma_load_3d_pair(sa, &tmSa, 0, k0 * kAtoms, am / kBM, bar);
                        tc::tma_load_3d_pair(sb, &tmSb, 0, k0 * kAtoms, nt * (bn / 128), bar);
                    } else {
                        tc::tma_load_3d(ad, &tmA, 0, am, k0, full(s));
                        tc::tma_load_3d(bd, &tmB, 0, bm, k0, full(s));
                        tc::tma_load_3d(sa, &tmSa, 0, k0 * kAtoms, am / kBM, full(s));
                        tc::tma_load_3d(sb, &tmSb, 0, k0 * kAtoms, nt * (bn / 128), full(s));
                    }
                    last_phase[s] = ph;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            // whatever happens elsewhere, what was asked for (a pair's: on the even CTA's barriers) lands before shared
            // memory is given back
            if (leader) {
                for (int i = 0; i < S; ++i) {
                    uint32_t never = 0;
                    if (last_phase[i] < 2u && !tc::wait_bounded(full(i), last_phase[i], &never, a.err)) break;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            const uint32_t me = tc::elect_one();
            // the low words of the descriptors: one addition an instruction
            const uint64_t op0 = tc::sw128_kmajor_desc(0), sf0 = tc::scale_atom_desc(0);
            auto desc = [](uint64_t d, uint32_t at) { return d + at; };
            auto copy_sf = [&](uint32_t col, uint32_t at) { tc::cp_scales<PAIR>(me, col, desc(sf0, at)); };
            uint32_t id[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) id[k] = with_id(a.idesc, CODE == BT_CODE_E2M1 ? 2 * (k & 1) : k);
            int s = 0, local = 0;
            uint32_t ph = 0, turn = 0;
            bool ok = true;
            for (int tl = unit; tl < a.num_tiles && ok; tl += nunits, ++local) {
                const int buf = local & 1;
                if (local >= 2 && !tc::wait_warp(tempty(buf), static_cast<uint32_t>((local - 2) >> 1) & 1u, abort_flag, a.err, a.wait_ns)) break;
                if (shared && local >= 1 && !tc::wait_warp(shared_read, static_cast<uint32_t>(local - 1) & 1u, abort_flag, a.err, a.wait_ns)) break;
                tc::fence_after_sync();
                const uint32_t acc = tmem + acc_col(buf);
                for (int kb = 0; kb < a.nk; ++kb) {
                    if (!tc::wait_warp(full(s), ph, abort_flag, a.err, a.wait_ns)) { ok = false; break; }
                    tc::fence_after_sync();
                    const int cnt = slice_count(kb);
                    uint32_t la = (sA + s * kASlice * D) >> 4, lb = (sB + s * kBSlice * D) >> 4;
                    uint32_t lsa = (sSa + s * kSaStage) >> 4, lsb = (sSb + s * kSbStage) >> 4;
                    const uint32_t next = static_cast<uint32_t>(kAtoms * D * kAtomBytes / 16);      // the other 128 rows of W
                    for (int i = 0; i < cnt; ++i) {
                        // the slice's scales: X's 128 rows 4 columns an atom, then W's bn rows 8 (4)
                        const uint32_t sfa = tmem + kSfCol + (turn ^= 32u), sfb = sfa + 4 * kAtoms;
#pragma unroll
                        for (int j = 0; j < kAtoms; ++j) {
                            copy_sf(sfa + 4 * j, lsa + 32 * j);
                            copy_sf(sfb + 8 * j, lsb + 32 * j);
                            if (bn == 256) copy_sf(sfb + 8 * j + 4, lsb + next + 32 * j);
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t more = kk != 0 || (kb | i) != 0 ? 1u : 0u;
                            // E2M1: 64 values, two bytes from 0 or 2 of one of two columns; E4M3: 32 values, byte kk
                            const uint32_t fa = kE2M1 ? sfa + 4 * (kk >> 1) : sfa, fb = kE2M1 ? sfb + 8 * (kk >> 1) : sfb;
                            tc::mma_scaled<kE2M1, PAIR>(me, acc, desc(op0, la + 2 * kk), desc(op0, lb + 2 * kk), id[kE2M1 ? kk & 1 : kk], fa, fb, more);
                        }
                        la += kASlice / 16;
                        lb += kBSlice / 16;
                        lsa += 32 * kAtoms;
                        lsb += 32 * kAtoms;
                    }
                    tc::commit_warp<PAIR>(me, empty(s), 0x3);
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (ok) {
                    tc::commit_warp<PAIR>(me, tfull(buf), 0x3);
                }
            }
            tc::commit_warp<PAIR>(me, drain, 0x1);
            const unsigned long long t0 = globaltimer_ns();
            while (!tc::mbar_try_wait(drain, 0u) && globaltimer_ns() - t0 < kWaitNs) {}
        }
        __syncwarp();
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t sbox = sStage + static_cast<uint32_t>((warp - 2) * 32 * kBoxInner);
        const int boxes = bn / 32;                          // of 32 columns; this warp has every second
        int local = 0;
        for (int tl = unit; tl < a.num_tiles; tl += nunits, ++local) {
            const int mt = tl / a.num_n, nt = tl % a.num_n, buf = local & 1;
            const int64_t row0 = static_cast<int64_t>(mt) * tile_rows + static_cast<int64_t>(crank) * kBM + quarter * 32;
            const int64_t n0 = static_cast<int64_t>(nt) * bn;
            const int64_t ncols = a.N - n0 < bn ? a.N - n0 : bn;
            const int live = row0 < a.M ? static_cast<int>((ncols + 31) / 32) : 0;      // boxes that hold anything
            if (!tc::wait_fast(tfull(buf), static_cast<uint32_t>(local >> 1) & 1u, abort_flag, a.err, a.wait_ns)) break;
            tc::fence_after_sync();
            const uint32_t tbase = tmem + lane_base + acc_col(buf);
            // accumulator 0 backwards, 1 forwards: the columns that they share come first
            const int per = a.epi / 4, steps = boxes / per;
            auto box_of = [&](int j) { return buf == 0 ? boxes - 1 - half - per * j : half + per * j; };
            auto give = [&](uint32_t bar) {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && crank != 0) tc::mbar_arrive_cluster(tc::mapa(bar, 0u));
                    else tc::mbar_arrive(bar);
                }
            };
            auto emit = [&](const uint32_t (&r)[32], int box) {
                constexpr int kChunks = kBoxInner / 16;
                const int64_t c0 = n0 + 32 * box, cend = n0 + ncols;
                __syncwarp();                               // the box before is read back
#pragma unroll
                for (int q = 0; q < kChunks; ++q) {
                    const uint4 w = chunk16<T>(r, q * (16 / kElem));
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 ::"r"(sbox + static_cast<uint32_t>(lane * kBoxInner) + (box_chunk<kElem>(q, lane) << 4)), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                                 : "memory");
                }
                __syncwarp();
                uint8_t *out = static_cast<uint8_t *>(a.out);
                if (a.vec) {
                    constexpr int kRowsPer = 32 / kChunks, kIters = 32 / kRowsPer;
                    const int q = lane % kChunks;
                    const int64_t col = c0 + q * (16 / kElem), row = row0 + lane / kChunks;
                    uint4 v[kIters];
#pragma unroll
                    for (int i = 0; i < kIters; ++i) {
                        const int rr = i * kRowsPer + lane / kChunks;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                                     : "r"(sbox + static_cast<uint32_t>(rr * kBoxInner) + (box_chunk<kElem>(q, rr) << 4)));
                    }
                    if (col < cend) {
                        uint8_t *p = out + (row * a.ldo + col) * kElem;
#pragma unroll
                        for (int i = 0; i < kIters; ++i)
                            if (row + i * kRowsPer < a.M) st_stream_v4(p + static_cast<int64_t>(i * kRowsPer) * a.ldo * kElem, v[i]);
                    }
                } else {
                    // rows of any alignment: 32 columns of one row at a time
                    constexpr int kPer = 16 / kElem;
                    const uint32_t off = static_cast<uint32_t>((lane % kPer) * kElem);
                    const int64_t col = c0 + lane;
#pragma unroll 4
                    for (int rr = 0; rr < 32; ++rr) {
                        const uint32_t addr = sbox + static_cast<uint32_t>(rr * kBoxInner) + (box_chunk<kElem>(lane / kPer, rr) << 4) + off;
                        uint32_t v;
                        if (kElem == 4) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
                        else asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr));
                        const int64_t row = row0 + rr;
                        if (row < a.M && col < cend) {
                            if (kElem == 4) reinterpret_cast<uint32_t *>(out)[row * a.ldo + col] = v;
                            else reinterpret_cast<uint16_t *>(out)[row * a.ldo + col] = static_cast<uint16_t>(v);
                        }
                    }
                }
            };
            uint32_t r0[32], r1[32];
            if (box_of(0) < live) tc::tmem_ld32(tbase + 32 * box_of(0), r0);
            if (box_of(1) < live) tc::tmem_ld32(tbase + 32 * box_of(1), r1);
            tc::tmem_ld_wait();
            give(shared_read);                              // two boxes a warp hold all that is shared
            if (steps == 2) give(tempty(buf));
#pragma unroll 1
            for (int j = 0; j < steps; j += 2) {
                if (j > 0) tc::tmem_ld_wait();              // box j + 1
                if (j > 0 && j + 2 == steps) give(tempty(buf));
                if (box_of(j) < live) emit(r0, box_of(j));
                if (j + 2 < steps && box_of(j + 2) < live) tc::tmem_ld32(tbase + 32 * box_of(j + 2), r0);
                if (box_of(j + 1) < live) emit(r1, box_of(j + 1));
                if (j + 2 < steps) {
                    tc::tmem_ld_wait();
                    if (box_of(j + 3) < live) tc::tmem_ld32(tbase + 32 * box_of(j + 3), r1);
                }
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (PAIR) tc::cluster_sync();
    if (warp == 1) {
        tc::fence_after_sync();
        if (PAIR) tc::tmem_dealloc_pair(tmem, kTmemCols);
        else tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// How a product is cut: rows of a tile (256 on a pair of CTAs, else 128), its columns, slices a stage, epilogue warps.
struct Shape {
    bool pair;
    int bn, d, epi;
};
int num_stages(int code, const Shape &sh, int elem) {
    const int n = (kSmemMax - kReserve - staging_bytes(elem, sh.epi)) / (slice_bytes(code, sh.bn, sh.pair) * sh.d);
    return n > kMaxStages ? kMaxStages : n;
}

// Whether few rows go through mx_small.cu (its figures there): always up to 16, and up to 32 where its tiles of W are not
// more than half of the SMs, so that a cluster shares each.
bool takes_small(int64_t M, int64_t N) {
    if (const char *e = std::getenv("BT_MX_CONFIG")) return std::strncmp(e, "small", 5) == 0 && M <= kSmallRows;
    return M <= kOwnRows || (M <= kSmallRows && (N + 127) / 128 * 2 <= device_sm_count());
}
// Whether x is quantised by a kernel before the product's.
bool quantises_first(int64_t M, int64_t N) { return !takes_small(M, N) || M > kOwnRows; }

// The fastest of four shapes by a model of their times in ns, fitted on GB300 (E2M1 and E4M3, 128 to 8192 rows): a slice of
// K, what a tile costs beside its slices, the epilogue (which the next tile's MMAs overlap), the launch. Model and measured,
// us: 8192 x 4096 x 11008 E2M1 pairs of 256 columns 107 and 102 (single CTAs 120 and 113, pairs of 128 133 and 131); 4096^3
// pairs of 128 29.7 and 29.8 (30.0 and 32.3; 30.2 and 31.0); 1024 x 4096 x 4096 single CTAs of 256 9.7 and 8.8 (11.7 and
// 11.7 with 128); 256 x 4096 x 4096 single CTAs of 128 7.3 and 7.2; 8192 x 11008 x 512 single CTAs of 256 42 and 39.5
// (pairs 61). Two slices a stage at 128 columns halve what a stage costs its issuer (162 and 182 us), at 256 they leave too
// few stages. BT_MX_CONFIG="[pair,]columns,slices[,epilogue warps]" or "small[,split]" in the environment decides instead.
struct Timing {
    bool pair;
    int bn, d;
    double slice, tile, epilogue, launch;
};
constexpr Timing kTimings[] = {{true, 256, 1, 310, 1300, 3200, 5000}, {false, 256, 1, 347, 1300, 2080, 2800},
                               {true, 128, 2, 213, 200, 2190, 4500},  {false, 128, 2, 265, 200, 1090, 2900}};
Shape choose(const Product &p) {
    const int elem = dtype_bytes(p.out_t);
    if (const char *e = std::getenv("BT_MX_CONFIG")) {
        int bn = 0, d = 0, epi = 8;
        const bool pair = std::strncmp(e, "pair,", 5) == 0;
        if (std::sscanf(pair ? e + 5 : e, "%d,%d,%d", &bn, &d, &epi) >= 2 && (bn == 128 || bn == 256) && d >= 1 && d <= 4 && (epi == 4 || epi == 8) &&
            num_stages(p.code, Shape{pair, bn, d, epi}, elem) >= 2)
            return Shape{pair, bn, d, epi};
    }
    const bool wide = aligned(p.out, 16) && (p.ldo * elem) % 16 == 0 && (p.N * elem) % 16 == 0;
    const int64_t k = slices(p.K, p.code), sms = device_sm_count();
    Shape best = {};
    double least = -1.0;
    for (const Timing &t : kTimings) {
        const int rows = t.pair ? 2 * kBM : kBM;
        const int64_t tiles = ((p.M + rows - 1) / rows) * ((p.N + t.bn - 1) / t.bn), units = t.pair ? sms / 2 : sms;
        const double main = static_cast<double>(k) * t.slice + t.tile, epi = t.epilogue * (elem == 4 ? 1.7 : 1.0) * (wide ? 1.0 : 1.5);
        const double us = static_cast<double>((tiles + units - 1) / units) * (main > epi ? main : epi) + t.launch;
        if (least < 0.0 || us < least) {
            least = us;
            best = Shape{t.pair, t.bn, t.d, 8};
        }
    }
    // four epilogue warps make room for a sixth stage where a tile is long enough to hide them (E2M1, eight and four: 8192 x 4096 x 11008
    // 103.4 and 100.0 us, 8192 x 8192 x 6144 122.7 and 119.5, 2048 x 11008 x 11008 80.7 and 75.0, 8192 x 2048 x 8192 48.2 and 47.3,
    // 16384 x 4096 x 6400 130.5 and 124.2)
    if (best.pair && best.bn == 256 && p.code == BT_CODE_E2M1 && k >= 24 && wide && elem == 2) best.epi = 4;
    return best;
}

template <int CODE, typename T, bool PAIR, int BN> cudaError_t launch(const Product &p, const Shape &sh, cudaStream_t s) {
    MxArgs a = {};
    a.M = p.M; a.N = p.N; a.ldo = p.ldo;
    a.slices = static_cast<int>(slices(p.K, CODE));
    a.d = sh.d;
    a.nk = (a.slices + a.d - 1) / a.d;
    a.bn = sh.bn;
    a.epi = sh.epi;
    const int rows = PAIR ? 2 * kBM : kBM, elem = sizeof(T);
    const int64_t num_m = (p.M + rows - 1) / rows, num_n = (p.N + a.bn - 1) / a.bn;
    if (num_m * num_n > (int64_t(1) << 30)) return cudaErrorInvalidValue;
    a.num_n = static_cast<int>(num_n);
    a.num_tiles = static_cast<int>(num_m * num_n);
    a.idesc = make_idesc(CODE, rows, a.bn);
    a.out = p.out;
    a.vec = aligned(p.out, 16) && (p.ldo * elem) % 16 == 0 && (p.N * elem) % 16 == 0;
    a.err = p.err;
    a.wait_ns = wait_limit_ns();
    const int stage = slice_bytes(CODE, a.bn, PAIR) * a.d;
    a.stages = num_stages(CODE, sh, elem);
    if (a.stages < 2) return cudaErrorInvalidValue;
    const int smem = a.stages * stage + staging_bytes(elem, a.epi) + kReserve;
    CUtensorMap ma, mb, sa, sb;
    const int64_t atoms = k_atoms(p.K, CODE);
    const int step = a.d * atoms_a_slice(CODE);
    if (!map_codes(&ma, p.x, p.M, a.slices, kBM, a.d) || !map_codes(&mb, p.w, p.N, a.slices, b_rows(a.bn, PAIR), a.d) ||
        !map_scales(&sa, p.xs, p.M, atoms, 1, step) || !map_scales(&sb, p.ws, p.N, atoms, a.bn / 128, step))
        return cudaErrorInvalidValue;
    auto kern = mx_linear_kernel<CODE, T, PAIR, BN>;
    static ContextOnce once;
    if (const cudaError_t e = allow_smem(kern, kSmemMax, once); e != cudaSuccess) return e;
    int units = device_sm_count() / (PAIR ? 2 : 1);
    if (units > a.num_tiles) units = a.num_tiles;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = PAIR ? 2 : 1;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(units * (PAIR ? 2 : 1)));
    cfg.blockDim = dim3(static_cast<unsigned>(64 + 32 * a.epi));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, ma, mb, sa, sb, static_cast<const MxArgs>(a));
}
template <int CODE, typename T> cudaError_t launch_shape(const Product &p, const Shape &sh, cudaStream_t s) {
    if (sh.bn == 256) return sh.pair ? launch<CODE, T, true, 256>(p, sh, s) : launch<CODE, T, false, 256>(p, sh, s);
    return sh.pair ? launch<CODE, T, true, 128>(p, sh, s) : launch<CODE, T, false, 128>(p, sh, s);
}
template <int CODE> cudaError_t launch_out(const Product &p, const Shape &sh, cudaStream_t s) {
    if (p.out_t == BT_F32) return launch_shape<CODE, float>(p, sh, s);
    if (p.out_t == BT_BF16) return launch_shape<CODE, __nv_bfloat16>(p, sh, s);
    return launch_shape<CODE, __half>(p, sh, s);
}
cudaError_t product(const Product &p, cudaStream_t s) {
    if (takes_small(p.M, p.N)) {
        int split = 0;
        if (const char *e = std::getenv("BT_MX_CONFIG")) {
            if (std::sscanf(e, "small,%d", &split) != 1 || (split != 1 && split != 2 && split != 4 && split != 8)) split = 0;
        }
        return launch_small(p, split, s);
    }
    const Shape sh = choose(p);
    return p.code == BT_CODE_E2M1 ? launch_out<BT_CODE_E2M1>(p, sh, s) : launch_out<BT_CODE_E4M3>(p, sh, s);
}

bool float_type(bt_dtype t) { return t == BT_F32 || t == BT_BF16 || t == BT_F16; }
size_t codes_room(int64_t M, int64_t K, bt_code code) { return round_up256(static_cast<size_t>(M) * static_cast<size_t>(code_bytes(K, code))); }

int64_t pitch8(int64_t n) { return (n + 7) / 8 * 8; }
bool plain_rows(const void *g, int64_t ldg, int64_t N) { return N % 8 == 0 && ldg % 8 == 0 && aligned(g, 16); }

}  // namespace
}  // namespace bt

using namespace bt;
using namespace bt::mx;

extern "C" {

size_t bt_mx_linear_workspace(int64_t M, int64_t N, int64_t K, bt_dtype x_dtype, bt_code code) {
    if (!float_type(x_dtype) || mx_sides(M, K, code) != BT_OK || M < 1 || N < 1 || !quantises_first(M, N)) return 0;
    return codes_room(M, K, code) + round_up256(scale_bytes(M, K, code));
}

bt_status bt_mx_linear(const void *x, bt_dtype x_dtype, int64_t ldx, const void *x_scales, const void *w, const void *w_scales,
                       bt_code code, int64_t M, int64_t N, int64_t K, void *out, bt_dtype out_dtype, int64_t ldo, void *workspace,
                       size_t workspace_bytes, bt_stream stream) {
    const bool packed = x_dtype == BT_PACKED;
    if ((!packed && !float_type(x_dtype)) || !float_type(out_dtype)) return BT_ERR_INVALID_ARG;
    bt_status fit = mx_sides(M, K, code);
    if (fit == BT_OK) fit = mx_sides(N, K, code);
    if (fit != BT_OK) return fit;
    if (ldo < N || (!packed && ldx < K)) return BT_ERR_INVALID_ARG;
    if (ldo > (int64_t(1) << 36) || (!packed && ldx > (int64_t(1) << 36))) return BT_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return BT_OK;
    if (x == nullptr || w == nullptr || w_scales == nullptr || out == nullptr || (packed && x_scales == nullptr)) return BT_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(w_scales, 16) || !aligned(out, static_cast<size_t>(dtype_bytes(out_dtype))) ||
        !aligned(x, packed ? 16 : static_cast<size_t>(dtype_bytes(x_dtype))) || (packed && !aligned(x_scales, 16)))
        return BT_ERR_ALIGNMENT;
    const size_t need = packed ? 0 : bt_mx_linear_workspace(M, N, K, x_dtype, code);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BT_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return BT_ERR_ALIGNMENT;
    if (!tc_available()) return BT_ERR_UNSUPPORTED;
    Product p = {};
    p.err = device_error_word();
    if (p.err == nullptr) return BT_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    p.x = x;
    p.x_t = x_dtype;
    p.ldx = ldx;
    p.xs = static_cast<const uint8_t *>(x_scales);
    if (need > 0) {
        uint8_t *q = static_cast<uint8_t *>(workspace), *sc = q + codes_room(M, K, code);
        if (launch_mx_quantize(x, x_dtype, ldx, M, K, code, q, sc, s) != cudaSuccess) return BT_ERR_CUDA;
        p.x = q;
        p.xs = sc;
        p.x_t = BT_PACKED;
    }
    p.w = static_cast<const uint8_t *>(w);
    p.ws = static_cast<const uint8_t *>(w_scales);
    p.code = code;
    p.M = M; p.N = N; p.K = K;
    p.out = out; p.ldo = ldo; p.out_t = out_dtype;
    return product(p, s) == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

size_t bt_mx_linear_backward_workspace(int64_t M, int64_t N) {
    return M < 1 || N < 1 || M >= kMaxSide || N >= kMaxSide ? 0 : round_up256(static_cast<size_t>(M) * static_cast<size_t>(pitch8(N)) * 2);
}

bt_status bt_mx_linear_backward(const void *g, int64_t ldg, const void *wt, int64_t ldw, int64_t M, int64_t N, int64_t K, void *grad_x,
                                bt_dtype grad_x_dtype, void *workspace, size_t workspace_bytes, bt_stream stream) {
    if ((grad_x_dtype != BT_BF16 && grad_x_dtype != BT_F32) || M < 0 || N < 0 || K < 1) return BT_ERR_INVALID_ARG;
    if (M >= kMaxSide || N >= kMaxSide || K >= kMaxSide) return BT_ERR_UNSUPPORTED;
    if (ldg < N || ldw < pitch8(N) || ldw % 8 != 0) return BT_ERR_INVALID_ARG;
    if (ldg > (int64_t(1) << 36) || ldw >= kMaxSide) return BT_ERR_UNSUPPORTED;
    if (M == 0) return BT_OK;
    const size_t e = static_cast<size_t>(dtype_bytes(grad_x_dtype));
    if (grad_x == nullptr || (N > 0 && (g == nullptr || wt == nullptr))) return BT_ERR_INVALID_ARG;
    if (!aligned(g, 2) || !aligned(wt, 16) || !aligned(grad_x, e)) return BT_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) return cudaMemsetAsync(grad_x, 0, static_cast<size_t>(M) * static_cast<size_t>(K) * e, s) == cudaSuccess ? BT_OK : BT_ERR_CUDA;
    const bool plain = plain_rows(g, ldg, N);
    if (!plain && (workspace == nullptr || workspace_bytes < bt_mx_linear_backward_workspace(M, N))) return BT_ERR_WORKSPACE;
    if (!plain && !aligned(workspace, 256)) return BT_ERR_ALIGNMENT;
    if (!tc_available()) return BT_ERR_UNSUPPORTED;
    const uint16_t *rows = static_cast<const uint16_t *>(g);
    int64_t pitch = ldg;
    if (!plain) {
        pitch = pitch8(N);
        adapter::AlignArgs al = {};         // (with zeros up to the pitch)
        al.src = rows;
        al.lds = ldg;
        al.dst = static_cast<uint16_t *>(workspace);
        al.ldd = pitch;
        al.C = static_cast<int>(N);
        al.rows = M;
        if (adapter::launch_align(al, s) != cudaSuccess) return BT_ERR_CUDA;
        rows = static_cast<const uint16_t *>(workspace);
    }
    unsigned int *err = device_error_word();
    if (err == nullptr) return BT_ERR_CUDA;
    return launch_tc_bf16(rows, pitch, static_cast<const uint16_t *>(wt), ldw, M, K, pitch8(N), 1.0f, grad_x, grad_x_dtype, nullptr, err,
                          s) == cudaSuccess
               ? BT_OK
               : BT_ERR_CUDA;
}

}  // extern "C"
