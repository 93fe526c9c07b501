// The adapters' products that begin with the rank (out = base + s B u, dX = base + A^T dU): see adapter.cu.
#include "adapter.cuh"

namespace bt {
namespace adapter {
namespace {

// A CTA keeps its tile's 128 rows of U in shared memory, as three bf16 values
// each (two in half precision), side by side, and walks a range of
// columns, 128 at a time: D (128 rows x 128 columns, fp32, tensor memory, two of
// them) = U_hi W + U_lo W (+ U_rest W). While one D is added to base and written,
// the next is worked out, and the columns of W after that and base's next values
// arrive.
// Bound: base and out. D is read in the layout in which a quad's four lanes hold
// 8 columns of a row. WIDE (rows of base and out start at 16-byte multiples):
// a quad's words are turned so that a lane loads and stores 16 bytes. Otherwise a
// warp's results pass through shared memory and every lane walks a column, so
// that a row's elements still travel together.
// 8192 x 4096 bf16, rank 64: 36 us, 3.7 TB/s of base and out (with warp-level
// matrix instructions and U in registers 53 us). Neither memory (29 % busy) nor
// the issue slots (41 %) nor L1 (45 %) is full: 8 warps an SM, of which every one
// takes D, base and the result through its registers, do not hide each other's
// waits, and two D of 128 columns leave room for no third CTA. 4096 x 4096 with
// base, rank 16: 21 us.
constexpr int kTile = 128;                 // columns
template <int RP> constexpr int kParts = RP <= 64 ? 1 : 2;                  // of 64 ranks
template <int RP, int VALS> constexpr int kUBytes = (VALS * RP + 63) / 64 * 2 * kAtom;    // 128 rows of 128 bytes for every 64 ranks
template <int RP, bool WT> constexpr int kWBytes = WT ? 2 * RP * 128 : kParts<RP> * 2 * kAtom;
constexpr int kTurnPitch = 64 + 4;         // floats of a row of a warp's results
// Rows of them at a time: 16, or 8 where two CTAs would not fit on an SM else (4096 x 4093 bf16 to fp32, rank 64: 65 us
// against 105; 16 take 26 us where 8 take 27, 777 x 4093 f16, rank 24).
template <int VALS> constexpr int kTurnRows = VALS == 3 ? 8 : 16;
template <int RP, bool WT, bool WIDE, int VALS> constexpr int kSmem =
    kUBytes<RP, VALS> + 2 * kWBytes<RP, WT> + (WIDE ? 0 : kThreads / 32 * kTurnRows<VALS> * kTurnPitch * 4) + 1024;

// 4 x 4 transpose of words across a quad: lane t gives word j to lane j's word t.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4], int t) {
    uint32_t p = (t & 1) ? w[0] : w[1], q = (t & 1) ? w[2] : w[3];
    p = __shfl_xor_sync(0xFFFFFFFFu, p, 1);
    q = __shfl_xor_sync(0xFFFFFFFFu, q, 1);
    if (t & 1) { w[0] = p; w[2] = q; } else { w[1] = p; w[3] = q; }
    p = (t & 2) ? w[0] : w[2];
    q = (t & 2) ? w[1] : w[3];
    p = __shfl_xor_sync(0xFFFFFFFFu, p, 2);
    q = __shfl_xor_sync(0xFFFFFFFFu, q, 2);
    if (t & 2) { w[0] = p; w[1] = q; } else { w[2] = p; w[3] = q; }
}

// 64 consecutive fp32 columns of 16 lanes (rows): lane 4g + t gets, of every 8
// columns, 2t and 2t + 1 of row g (words 0, 1) and of row g + 8 (words 2, 3).
__device__ __forceinline__ void tmem_ld_16x64(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

// FAST: WIDE, and W's rows start at 16-byte multiples. BF32: base is fp32.
template <typename T, int RP, bool WT, bool OF32, bool FAST, bool BF32>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) expand_kernel(const ExpandArgs a) {
    extern __shared__ uint8_t dyn[];
    __shared__ alignas(8) uint64_t ready[2];
    __shared__ uint32_t tmem_slot, abort_flag;
    __shared__ int64_t rows_s[FAST ? 1 : 128];
    __shared__ float mul_s[FAST ? 1 : 128];
    constexpr int VALS = kValues<T>;                        // of U
    uint8_t *us = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u), *wbuf = us + kUBytes<RP, VALS>;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    float *turn = reinterpret_cast<float *>(wbuf + 2 * kWBytes<RP, WT>) + warp * kTurnRows<VALS> * kTurnPitch;
    // The plan, W and base were there before this call's first kernel began, which waited for all before it: only
    // U, which that kernel writes, has to be waited for.
    if (static_cast<int>(blockIdx.x) >= a.tiles * a.splits) {
        pdl_wait();
        pdl_launch_dependents();
        pass_rows<T>(a.pass, OF32, blockIdx.x - a.tiles * a.splits, gridDim.x - a.tiles * a.splits);
        return;
    }
    const AdapterTile tile = a.plan.tiles[blockIdx.x / a.splits];
    const int part = blockIdx.x % a.splits;
    const int total = (a.C + kTile - 1) / kTile;
    const int s0 = static_cast<int>(static_cast<int64_t>(total) * part / a.splits);
    const int s1 = static_cast<int>(static_cast<int64_t>(total) * (part + 1) / a.splits);
    const uint16_t *w = a.w + static_cast<int64_t>(tile.adapter) * a.R * (WT ? a.ldw : a.C);
    auto put = [&](uint8_t *dst, const uint16_t *src, int valid) {
        if constexpr (FAST) copy8<kRows16>(dst, src, valid, 16);
        else if (a.aw >= 4) copy8<kRows4>(dst, src, valid, a.aw);
        else copy8<kRows2>(dst, src, valid, 2);
    };
    auto load_w = [&](int s) {
        const int c0 = s * kTile;
        uint8_t *ws = wbuf + (s & 1) * kWBytes<RP, WT>;
        if constexpr (!WT) {
            // 128 columns' rows of RP ranks, 64 to an atom
#pragma unroll
            for (int i = 0; i < kTile * (RP / 8) / kThreads; ++i) {
                const int at = tid + kThreads * i, k = at / (RP / 8), j = at % (RP / 8), valid = c0 + k < a.C ? a.R - 8 * j : 0;
                put(ws + (j >> 3) * 2 * kAtom + sw128(k, j & 7), valid > 0 ? w + static_cast<int64_t>(c0 + k) * a.R + 8 * j : a.w, valid);
            }
        } else {
            // RP rows of 128 columns, 64 to an atom
#pragma unroll
            for (int i = 0; i < RP * 16 / kThreads; ++i) {
                const int at = tid + kThreads * i, r = at >> 4, j = at & 15, valid = r < a.R ? a.C - c0 - 8 * j : 0;
                put(ws + (j >> 3) * RP * 128 + sw128(r, j & 7), valid > 0 ? w + static_cast<int64_t>(r) * a.ldw + c0 + 8 * j : a.w, valid);
            }
        }
    };
    load_w(s0);
    // this warp's rows, 32 (warp % 4) .. + 31, in two halves of 16; its 64 columns of a tile
    const int m0 = (warp & 3) * 32, cw = (warp >> 2) * 64;
    const float s = a.scale != nullptr ? a.scale[tile.adapter] : 1.0f;
    int row[2][2];
    bool live[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = m0 + 16 * b + 8 * h + g, at = tile.first + (m < tile.n ? m : 0);
            live[b][h] = m < tile.n;
            row[b][h] = a.plan.rows[at];
        }
    if constexpr (!FAST) {
        if (tid < 128) {
            const int at = tile.first + (tid < tile.n ? tid : 0);
            rows_s[tid] = a.plan.rows[at];
        }
    }
    // (FAST) 16-bit base's values of a step, lane t's columns 8t.. of each 32
    const bool b16 = a.base != nullptr && !BF32;
    uint4 bw[2][2][2];
    auto load_base = [&](int st, int b) {
        const int c0 = st * kTile + cw;
        if constexpr (FAST) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int cj = c0 + 32 * q + 8 * t;
                    bw[b][h][q] = make_uint4(0u, 0u, 0u, 0u);
                    if (b16 && live[b][h] && st < s1 && cj < a.C)
                        bw[b][h][q] = ld_stream_v4(static_cast<const uint16_t *>(a.base) + static_cast<int64_t>(row[b][h]) * a.ldb + cj);
                }
        }
    };
    load_base(s0, 0);
    load_base(s0, 1);
    pdl_wait();                                             // before tensor memory is taken, see shrink_kernel
    // U: 128 rows of RP ranks, hi, lo (and rest)
#pragma unroll
    for (int i = 0; i < VALS * 128 * (RP / 8) / kThreads; ++i) {
        const int at = tid + kThreads * i, val = at / (128 * (RP / 8)), k = at % (128 * (RP / 8));
        const int m = k / (RP / 8), j = k % (RP / 8), to = val * (RP / 8) + j;
        const uint16_t *u = val == 0 ? a.u.hi : val == 1 ? a.u.lo : a.u.rest;
        cp_async_16(us + (to >> 3) * 2 * kAtom + sw128(m, to & 7),
                    m < tile.n ? u + static_cast<int64_t>(tile.first + m) * RP + 8 * j : u, m < tile.n ? 16 : 0);
    }
    cp_async_commit();
    if (s0 + 1 < s1) load_w(s0 + 1);
    cp_async_commit();
    float mul[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = m0 + 16 * b + 8 * h + g;
            mul[b][h] = a.u.unpower != nullptr ? s * a.u.unpower[tile.first + (m < tile.n ? m : 0)] : s;
        }
    if constexpr (!FAST) {
        if (tid < 128) mul_s[tid] = a.u.unpower != nullptr ? s * a.u.unpower[tile.first + (tid < tile.n ? tid : 0)] : s;
    }
    if (warp == 0) {
        tc::tmem_alloc(smem_u32(&tmem_slot), 2 * kTile);
        tc::tmem_relinquish();
        if (lane == 0) {
            abort_flag = 0;
            tc::mbar_init(smem_u32(&ready[0]), 1);
            tc::mbar_init(smem_u32(&ready[1]), 1);
            tc::fence_mbar_init();
        }
    }
    // fp32 sums, W MN-major where it is [R, C], N = M = 128
    constexpr uint32_t kFmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    constexpr uint32_t kIdesc = (1u << 4) | (kFmt << 7) | (kFmt << 10) | ((WT ? 1u : 0u) << 16) |
                                ((static_cast<uint32_t>(kTile) >> 3) << 17) | ((128u >> 4) << 24);
    auto multiply = [&](int st, uint32_t tmem) {            // one thread
        tc::fence_after_sync();
        const uint32_t u0 = smem_u32(us), w0 = smem_u32(wbuf + (st & 1) * kWBytes<RP, WT>);
#pragma unroll
        for (int val = 0; val < VALS; ++val)
#pragma unroll
            for (int k = 0; k < RP / 16; ++k) {             // 16 ranks
                const int from = val * (RP / 16) + k;
                const uint64_t da = tc::sw128_kmajor_desc(u0 + (from >> 2) * 2 * kAtom + 32 * (from & 3));
                const uint64_t db = WT ? tc::sw128_mnmajor_desc(w0 + 2048 * k, RP * 128)
                                       : tc::sw128_kmajor_desc(w0 + (k >> 2) * 2 * kAtom + 32 * (k & 3));
                tc::mma_f16(tmem + (st & 1) * kTile, da, db, kIdesc, (val | k) != 0);
            }
        tc::mma_commit(smem_u32(&ready[st & 1]));
    };
    cp_async_wait<1>();
    tc::fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_launch_dependents();
    const uint32_t tmem = tmem_slot;
    if (tid == 0) multiply(s0, tmem);
    for (int st = s0; st < s1; ++st) {
        // the next columns' product, into the other D, which every warp has read
        cp_async_wait<0>();
        tc::fence_proxy_async_smem();
        tc::fence_before_sync();
        __syncthreads();
        if (tid == 0 && st + 1 < s1) multiply(st + 1, tmem);
        wait_landed(ready[st & 1], static_cast<uint32_t>((st - s0) >> 1) & 1u, &abort_flag, a.err, a.limit_ns);
        tc::fence_after_sync();
        if (st + 2 < s1) load_w(st + 2);                    // over the columns just multiplied
        cp_async_commit();
        const int c0 = st * kTile + cw;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t acc[32];
            tmem_ld_16x64(tmem + (static_cast<uint32_t>(m0 + 16 * b) << 16) + (st & 1) * kTile + cw, acc);
            tc::tmem_ld_wait();
            if constexpr (FAST) {
                // C a multiple of 8: whole vectors
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t bo = static_cast<int64_t>(row[b][h]) * a.ldb, oo = static_cast<int64_t>(row[b][h]) * a.ldo;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {           // 32 columns: blocks 4q .. 4q + 3
                        float2 v[4];                        // base, then base + s * sum in one rounding each
                        const int cq = c0 + 32 * q;
                        if constexpr (BF32) {
                            const float *p = static_cast<const float *>(a.base) + bo;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int cj = cq + 8 * j + 2 * t;
                                v[j] = a.base != nullptr && live[b][h] && cj < a.C ? *reinterpret_cast<const float2 *>(p + cj)
                                                                                   : make_float2(0.0f, 0.0f);
                            }
                        } else {
                            uint32_t xw[4] = {bw[b][h][q].x, bw[b][h][q].y, bw[b][h][q].z, bw[b][h][q].w};
                            quad_transpose(xw, t);
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] = unpack2<T>(xw[j]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[j] = make_float2(__fmaf_rn(__uint_as_float(acc[4 * (4 * q + j) + 2 * h]), mul[b][h], v[j].x),
                                               __fmaf_rn(__uint_as_float(acc[4 * (4 * q + j) + 2 * h + 1]), mul[b][h], v[j].y));
                        if constexpr (OF32) {
                            float *o = static_cast<float *>(a.out) + oo;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int cj = cq + 8 * j + 2 * t;
                                if (live[b][h] && cj < a.C) *reinterpret_cast<float2 *>(o + cj) = v[j];
                            }
                        } else {
                            uint32_t ow[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) ow[j] = pack2<T>(v[j].x, v[j].y);
                            quad_transpose(ow, t);
                            const int cj = cq + 8 * t;
                            if (live[b][h] && cj < a.C)
                                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + oo + cj) =
                                    make_uint4(ow[0], ow[1], ow[2], ow[3]);
                        }
                    }
                }
            } else {
                constexpr int TURN = kTurnRows<VALS>;
                if constexpr (TURN == 16) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint2 *>(turn + (8 * h + g) * kTurnPitch + 8 * j + 2 * t) =
                                make_uint2(acc[4 * j + 2 * h], acc[4 * j + 2 * h + 1]);
                    __syncwarp();
                }
                // eight rows at a time: their base first, all on its way at once
#pragma unroll 1
                for (int m8 = 0; m8 < 16; m8 += 8) {
                    float v[8][2];
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const int at = m0 + 16 * b + m8 + m;
                        const int64_t r = rows_s[at] * a.ldb + c0 + lane;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool ok = a.base != nullptr && at < tile.n && c0 + lane + 32 * e < a.C;
                            if constexpr (BF32) v[m][e] = ok ? static_cast<const float *>(a.base)[r + 32 * e] : 0.0f;
                            else v[m][e] = ok ? Elem<T>::to_f32(static_cast<const T *>(a.base)[r + 32 * e]) : 0.0f;
                        }
                    }
                    if constexpr (TURN == 8) {
                        __syncwarp();                       // the eight before have been read
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint2 *>(turn + g * kTurnPitch + 8 * j + 2 * t) =
                                m8 == 0 ? make_uint2(acc[4 * j], acc[4 * j + 1]) : make_uint2(acc[4 * j + 2], acc[4 * j + 3]);
                        __syncwarp();
                    }
#pragma unroll
                    for (int m = 0; m < 8; ++m) {
                        const int at = m0 + 16 * b + m8 + m;
                        const float ms = mul_s[at];
                        const int64_t r = rows_s[at] * a.ldo + c0 + lane;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            if (at >= tile.n || c0 + lane + 32 * e >= a.C) continue;
                            const float f = __fmaf_rn(turn[(TURN == 16 ? m8 + m : m) * kTurnPitch + lane + 32 * e], ms, v[m][e]);
                            if constexpr (OF32) static_cast<float *>(a.out)[r + 32 * e] = f;
                            else static_cast<T *>(a.out)[r + 32 * e] = to16<T>(f);
                        }
                    }
                }
                __syncwarp();
            }
            load_base(st + 1, b);
        }
    }
    cp_async_wait<0>();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 2 * kTile);
    }
}

template <typename T, int RP, bool WT, bool OF32, bool FAST, bool BF32>
cudaError_t launch_rp(const ExpandArgs &a, cudaStream_t s) {
    auto kern = expand_kernel<T, RP, WT, OF32, FAST, BF32>;
    constexpr int smem = kSmem<RP, WT, FAST, kValues<T>>;
    static ContextOnce once;
    if (const cudaError_t err = allow_smem(kern, smem, once); err != cudaSuccess) return err;
    const int64_t pieces = pass_pieces(a.pass);
    const int pass = static_cast<int>(pieces < 2 * device_sm_count() ? pieces : 2 * device_sm_count());
    return launch_pdl_smem(kern, dim3(static_cast<unsigned>(a.tiles * a.splits + pass)), dim3(kThreads), smem, s, a);
}
template <typename T, bool WT, bool OF32, bool FAST, bool BF32> cudaError_t launch_r(const ExpandArgs &a, cudaStream_t s) {
    if (a.R <= 16) return launch_rp<T, 16, WT, OF32, FAST, BF32>(a, s);
    if (a.R <= 32) return launch_rp<T, 32, WT, OF32, FAST, BF32>(a, s);
    if (a.R <= 64) return launch_rp<T, 64, WT, OF32, FAST, BF32>(a, s);
    return launch_rp<T, 128, WT, OF32, FAST, BF32>(a, s);
}
template <typename T, bool WT, bool OF32> cudaError_t launch_t(const ExpandArgs &a, cudaStream_t s) {
    const bool fast = a.wide && a.aw == 16;
    if constexpr (!WT) {                                    // (dX's base has its type)
        if (a.base != nullptr && a.base_f32)
            return fast ? launch_r<T, WT, OF32, true, true>(a, s) : launch_r<T, WT, OF32, false, true>(a, s);
    }
    return fast ? launch_r<T, WT, OF32, true, false>(a, s) : launch_r<T, WT, OF32, false, false>(a, s);
}

template <typename T> __global__ void __launch_bounds__(kThreads) pass_kernel(const PassArgs a, int out_f32) {
    pdl_launch_dependents();
    pdl_wait();
    pass_rows<T>(a, out_f32 != 0, blockIdx.x, gridDim.x);
}

}  // namespace

cudaError_t launch_expand(bt_dtype t, bool wt, bool out_f32, const ExpandArgs &args, int tiles, cudaStream_t s) {
    if (tiles == 0) return cudaSuccess;
    ExpandArgs a = args;
    a.tiles = tiles;
    // Column ranges a tile, as many as end soonest: in waves of two CTAs an SM, each of its 128-column steps and
    // of what it costs to begin, about two steps' time.
    const int steps = (a.C + kTile - 1) / kTile, slots = 2 * device_sm_count();
    int64_t best = 0;
    for (int waves = 1; waves <= 4; ++waves) {
        int splits = static_cast<int>(static_cast<int64_t>(slots) * waves / tiles);
        if (splits < 1) splits = 1;
        if (splits > steps) splits = steps;
        const int64_t real = (static_cast<int64_t>(tiles) * splits + slots - 1) / slots, cost = real * ((steps + splits - 1) / splits + 2);
        if (waves == 1 || cost < best) {
            best = cost;
            a.splits = splits;
        }
    }
    if (wt) return launch_t<__nv_bfloat16, true, false>(a, s);
    if (t == BT_F16) return out_f32 ? launch_t<__half, false, true>(a, s) : launch_t<__half, false, false>(a, s);
    return out_f32 ? launch_t<__nv_bfloat16, false, true>(a, s) : launch_t<__nv_bfloat16, false, false>(a, s);
}

cudaError_t launch_pass(bt_dtype t, bool out_f32, const PassArgs &a, cudaStream_t s) {
    if (a.n == 0 || (a.out == nullptr && a.u == nullptr)) return cudaSuccess;
    const int64_t pieces = pass_pieces(a), slots = 8 * device_sm_count();
    const dim3 grid(static_cast<unsigned>(pieces < slots ? pieces : slots));
    return t == BT_F16 ? launch_pdl(pass_kernel<__half>, grid, dim3(kThreads), s, a, static_cast<int>(out_f32))
                       : launch_pdl(pass_kernel<__nv_bfloat16>, grid, dim3(kThreads), s, a, static_cast<int>(out_f32));
}

}  // namespace adapter
}  // namespace bt
