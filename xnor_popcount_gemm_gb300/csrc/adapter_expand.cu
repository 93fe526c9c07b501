// The adapters' products that begin with the rank (out = base + s B u, dX = base + A^T dU): see adapter.cu.
#include "adapter.cuh"

namespace bt {
namespace adapter {
namespace {

// A warp keeps its 16 rows of U in registers, as two 16-bit values each, and
// walks a range of columns, 64 at a time: W's next 64 columns and base's next
// values arrive while these are multiplied.
// Bound: base and out. WIDE: their rows start at 16-byte multiples; the results
// of a quad's four lanes are turned so that a lane loads and stores 16
// bytes. Otherwise a warp's 16 x 64 results pass through shared memory and
// every lane walks a column, so that a row's elements still travel together.
template <int RP, bool WT> constexpr int kWElems = WT ? RP * kXPitch : kStep * (RP + 8);
constexpr int kTurnPitch = kStep + 4;      // floats of a row of a warp's results
template <int RP, bool WT, bool WIDE> constexpr int kSmem = 4 * kWElems<RP, WT> + (WIDE ? 0 : kThreads / 32 * 16 * kTurnPitch * 4);

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

template <typename T, int RP, bool WT, bool OF32, bool WIDE>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) expand_kernel(const ExpandArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint16_t *wbuf = reinterpret_cast<uint16_t *>(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    float *turn = reinterpret_cast<float *>(smem + 4 * kWElems<RP, WT>) + warp * 16 * kTurnPitch;
    pdl_launch_dependents();
    pdl_wait();
    const AdapterTile tile = a.plan.tiles[blockIdx.x / a.splits];
    const int part = blockIdx.x % a.splits;
    const int total = (a.C + kStep - 1) / kStep;
    const int s0 = static_cast<int>(static_cast<int64_t>(total) * part / a.splits);
    const int s1 = static_cast<int>(static_cast<int64_t>(total) * (part + 1) / a.splits);
    const uint16_t *w = a.w + static_cast<int64_t>(tile.adapter) * a.R * a.C;
    auto load = [&](int s) {
        uint16_t *ws = wbuf + (s & 1) * kWElems<RP, WT>;
        const int c0 = s * kStep;
        if constexpr (!WT) {
            for (int i = tid; i < kStep * (RP / 8); i += kThreads) {
                const int k = i / (RP / 8), r = (i % (RP / 8)) * 8, valid = c0 + k < a.C ? a.R - r : 0;
                copy8(ws + k * (RP + 8) + r, valid > 0 ? w + static_cast<int64_t>(c0 + k) * a.R + r : a.w, valid, a.aw);
            }
        } else {
            for (int i = tid; i < RP * 8; i += kThreads) {
                const int r = i >> 3, k = (i & 7) * 8, valid = r < a.R ? a.C - c0 - k : 0;
                copy8(ws + r * kXPitch + k, valid > 0 ? w + static_cast<int64_t>(r) * a.C + c0 + k : a.w, valid, a.aw);
            }
        }
    };
    load(s0);
    cp_async_commit();
    const int m0 = warp * 16;
    int row[2];
    bool live[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = m0 + 8 * h + g;
        live[h] = m < tile.n;
        row[h] = a.plan.rows[tile.first + (live[h] ? m : 0)];
    }
    // Base's values of a step. WIDE: 16-bit base as lane t's columns 8t.. of each 32 (one vector per half and row
    // half); else column `lane` and `lane + 32` of the warp's 16 rows, two 16-bit values a word.
    const bool b16 = a.base != nullptr && !a.base_f32;
    uint4 bw[2][2];
    uint32_t bn[16];
    const int mrow = __shfl_sync(0xFFFFFFFFu, row[0], (lane & 7) * 4), mrow8 = __shfl_sync(0xFFFFFFFFu, row[1], (lane & 7) * 4);
    const int lane_row = (lane & 8) ? mrow8 : mrow;         // lane m: row m of the 16
    const int rows_here = tile.n - m0;
    auto load_base = [&](int s) {
        if constexpr (WIDE) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int cj = s * kStep + 32 * q + 8 * t;
                    bw[h][q] = make_uint4(0u, 0u, 0u, 0u);
                    if (b16 && live[h] && s < s1 && cj < a.C)
                        bw[h][q] = ld_stream_v4(static_cast<const uint16_t *>(a.base) + static_cast<int64_t>(row[h]) * a.ldb + cj);
                }
        } else if (b16) {
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                const uint16_t *b = static_cast<const uint16_t *>(a.base) +
                                    static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, lane_row, m)) * a.ldb + s * kStep + lane;
                const bool ok = m < rows_here && s < s1;
                const uint32_t lo = ok && s * kStep + lane < a.C ? b[0] : 0u;
                const uint32_t hi = ok && s * kStep + lane + 32 < a.C ? b[32] : 0u;
                bn[m] = lo | (hi << 16);
            }
        }
    };
    load_base(s0);
    // U's fragments: rows g and g + 8 of the warp's 16
    float mul[2];
    uint32_t uh[RP / 16][4], ul[RP / 16][4];
    const float s = a.scale != nullptr ? a.scale[tile.adapter] : 1.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float *u = a.u + static_cast<int64_t>(row[h]) * a.R;
        float v[RP / 16][4], amax = 0.0f;
        if ((a.R & 1) == 0) {
#pragma unroll
            for (int k = 0; k < RP / 16; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 16 * k + 2 * t + 8 * e;
                    const float2 f = live[h] && r < a.R ? *reinterpret_cast<const float2 *>(u + r) : make_float2(0.0f, 0.0f);
                    v[k][2 * e] = f.x;
                    v[k][2 * e + 1] = f.y;
                }
        } else {
#pragma unroll
            for (int k = 0; k < RP / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = 16 * k + 2 * t + (e & 1) + (e >> 1) * 8;
                    v[k][e] = live[h] && r < a.R ? u[r] : 0.0f;
                }
        }
#pragma unroll
        for (int k = 0; k < RP / 16; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(v[k][e]));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const float p = row_power<T>(amax);
        mul[h] = s / p;
#pragma unroll
        for (int k = 0; k < RP / 16; ++k) {
            split2<T>(v[k][0] * p, v[k][1] * p, uh[k][h], ul[k][h]);
            split2<T>(v[k][2] * p, v[k][3] * p, uh[k][2 + h], ul[k][2 + h]);
        }
    }
    const float mq = __shfl_sync(0xFFFFFFFFu, mul[0], (lane & 7) * 4), mq8 = __shfl_sync(0xFFFFFFFFu, mul[1], (lane & 7) * 4);
    const float lane_mul = (lane & 8) ? mq8 : mq;
    for (int st = s0; st < s1; ++st) {
        cp_async_wait<0>();
        __syncthreads();
        if (st + 1 < s1) load(st + 1);
        cp_async_commit();
        const uint16_t *ws = wbuf + (st & 1) * kWElems<RP, WT>;
        float acc[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < RP / 16; ++k)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                uint32_t bf[4];
                if constexpr (!WT)
                    ldsm4(bf, smem_u32(ws + (8 * j + (lane >> 4) * 8 + (lane & 7)) * (RP + 8) + 16 * k + ((lane >> 3) & 1) * 8));
                else
                    ldsm4t(bf, smem_u32(ws + (16 * k + (lane & 15)) * kXPitch + 8 * j + (lane >> 4) * 8));
                mma<T>(acc[j], uh[k], bf[0], bf[1]);
                mma<T>(acc[j + 1], uh[k], bf[2], bf[3]);
                mma<T>(acc[j], ul[k], bf[0], bf[1]);
                mma<T>(acc[j + 1], ul[k], bf[2], bf[3]);
            }
        const int c0 = st * kStep;
        if constexpr (WIDE) {
            // C a multiple of 8: whole vectors
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t bo = static_cast<int64_t>(row[h]) * a.ldb, oo = static_cast<int64_t>(row[h]) * a.ldo;
#pragma unroll
                for (int q = 0; q < 2; ++q) {               // 32 columns: blocks 4q .. 4q + 3
                    float2 v[4];                            // base, then base + s * sum in one rounding each
                    const int cq = c0 + 32 * q;
                    if (a.base_f32) {
                        const float *b = static_cast<const float *>(a.base) + bo;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int cj = cq + 8 * j + 2 * t;
                            v[j] = a.base != nullptr && live[h] && cj < a.C ? *reinterpret_cast<const float2 *>(b + cj)
                                                                            : make_float2(0.0f, 0.0f);
                        }
                    } else {
                        uint32_t xw[4] = {bw[h][q].x, bw[h][q].y, bw[h][q].z, bw[h][q].w};
                        quad_transpose(xw, t);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] = unpack2<T>(xw[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = make_float2(__fmaf_rn(acc[4 * q + j][2 * h], mul[h], v[j].x),
                                           __fmaf_rn(acc[4 * q + j][2 * h + 1], mul[h], v[j].y));
                    if constexpr (OF32) {
                        float *o = static_cast<float *>(a.out) + oo;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int cj = cq + 8 * j + 2 * t;
                            if (live[h] && cj < a.C) *reinterpret_cast<float2 *>(o + cj) = v[j];
                        }
                    } else {
                        uint32_t ow[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) ow[j] = pack2<T>(v[j].x, v[j].y);
                        quad_transpose(ow, t);
                        const int cj = cq + 8 * t;
                        if (live[h] && cj < a.C)
                            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + oo + cj) =
                                make_uint4(ow[0], ow[1], ow[2], ow[3]);
                    }
                }
            }
            load_base(st + 1);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float2 *>(turn + (8 * h + g) * kTurnPitch + 8 * j + 2 * t) =
                        make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
            __syncwarp();
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                const int64_t r = __shfl_sync(0xFFFFFFFFu, lane_row, m);
                const float ms = __shfl_sync(0xFFFFFFFFu, lane_mul, m);
                if (m >= rows_here) continue;
                const float2 f = unpack2<T>(b16 ? bn[m] : 0u);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int cj = c0 + lane + 32 * e;
                    if (cj >= a.C) continue;
                    float v = e ? f.y : f.x;
                    if (a.base_f32 && a.base != nullptr) v = static_cast<const float *>(a.base)[r * a.ldb + cj];
                    v = __fmaf_rn(turn[m * kTurnPitch + lane + 32 * e], ms, v);
                    if constexpr (OF32) static_cast<float *>(a.out)[r * a.ldo + cj] = v;
                    else static_cast<T *>(a.out)[r * a.ldo + cj] = to16<T>(v);
                }
            }
            __syncwarp();
            load_base(st + 1);
        }
    }
}

template <typename T, int RP, bool WT, bool OF32, bool WIDE> cudaError_t launch_rp(const ExpandArgs &a, int tiles, cudaStream_t s) {
    auto kern = expand_kernel<T, RP, WT, OF32, WIDE>;
    constexpr int smem = kSmem<RP, WT, WIDE>;
    static std::once_flag once;
    static cudaError_t err = cudaSuccess;
    if (allow_smem(kern, smem, once, err) != cudaSuccess) return err;
    return launch_pdl_smem(kern, dim3(static_cast<unsigned>(tiles * a.splits)), dim3(kThreads), smem, s, a);
}
template <typename T, bool WT, bool OF32, bool WIDE> cudaError_t launch_r(const ExpandArgs &a, int tiles, cudaStream_t s) {
    if (a.R <= 16) return launch_rp<T, 16, WT, OF32, WIDE>(a, tiles, s);
    if (a.R <= 32) return launch_rp<T, 32, WT, OF32, WIDE>(a, tiles, s);
    if (a.R <= 64) return launch_rp<T, 64, WT, OF32, WIDE>(a, tiles, s);
    return launch_rp<T, 128, WT, OF32, WIDE>(a, tiles, s);
}
template <typename T, bool WT, bool OF32> cudaError_t launch_t(const ExpandArgs &a, int tiles, cudaStream_t s) {
    return a.wide ? launch_r<T, WT, OF32, true>(a, tiles, s) : launch_r<T, WT, OF32, false>(a, tiles, s);
}

template <typename T, bool OF32> __global__ void __launch_bounds__(kThreads) pass_kernel(const PassArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = a.rows[blockIdx.x];
    if (a.u != nullptr && blockIdx.y == 0)
        for (int r = threadIdx.x; r < a.R; r += kThreads) a.u[row * a.R + r] = 0.0f;
    if (a.out == nullptr) return;
#pragma unroll 4
    for (int c = blockIdx.y * kThreads + threadIdx.x; c < a.N; c += gridDim.y * kThreads) {
        float v = 0.0f;
        if (a.base != nullptr)
            v = a.base_f32 ? static_cast<const float *>(a.base)[row * a.ldb + c]
                           : Elem<T>::to_f32(static_cast<const T *>(a.base)[row * a.ldb + c]);
        if constexpr (OF32) static_cast<float *>(a.out)[row * a.ldo + c] = v;
        else static_cast<T *>(a.out)[row * a.ldo + c] = to16<T>(v);
    }
}
template <typename T> cudaError_t launch_pass_t(bool out_f32, const PassArgs &a, dim3 grid, cudaStream_t s) {
    return out_f32 ? launch_pdl(pass_kernel<T, true>, grid, dim3(kThreads), s, a)
                   : launch_pdl(pass_kernel<T, false>, grid, dim3(kThreads), s, a);
}

}  // namespace

cudaError_t launch_expand(bt_dtype t, bool wt, bool out_f32, const ExpandArgs &args, int tiles, cudaStream_t s) {
    if (tiles == 0) return cudaSuccess;
    ExpandArgs a = args;
    const int steps = (a.C + kStep - 1) / kStep;
    // two CTAs an SM, and twice that many so that the last ones end close together
    int splits = (4 * device_sm_count() + tiles - 1) / tiles;
    if (splits > steps) splits = steps;
    a.splits = splits < 1 ? 1 : splits;
    if (wt) return launch_t<__nv_bfloat16, true, false>(a, tiles, s);
    if (t == BT_F16) return out_f32 ? launch_t<__half, false, true>(a, tiles, s) : launch_t<__half, false, false>(a, tiles, s);
    return out_f32 ? launch_t<__nv_bfloat16, false, true>(a, tiles, s) : launch_t<__nv_bfloat16, false, false>(a, tiles, s);
}

cudaError_t launch_pass(bt_dtype t, bool out_f32, const PassArgs &a, cudaStream_t s) {
    if (a.n == 0 || (a.out == nullptr && a.u == nullptr)) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>(a.n), static_cast<unsigned>(a.N < 4 * kThreads ? 1 : a.N < 16 * kThreads ? 2 : 4));
    return t == BT_F16 ? launch_pass_t<__half>(out_f32, a, grid, s) : launch_pass_t<__nv_bfloat16>(out_f32, a, grid, s);
}

}  // namespace adapter
}  // namespace bt
