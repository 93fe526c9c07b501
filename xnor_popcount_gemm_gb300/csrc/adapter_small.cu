// The adapters of a few tokens each (decoding): see adapter.cu.
#include "adapter.cuh"

namespace bt {
namespace adapter {
namespace {

// The whole adapter in one kernel. A cluster of 1 to 8 CTAs takes up to 16
// tokens of one adapter. Each CTA reduces a piece of the long axis, the pieces
// are exchanged through distributed shared memory, and each CTA writes a range
// of the columns. Weights go from memory straight to the registers of the
// matrix instructions, 16 bytes a lane: the reduction index may be permuted as
// long as both operands agree, so lane t of a quad takes elements 8t .. 8t + 7 of
// 32 as its share of two instructions. The first of B's rows and of base's
// values are fetched before anything waits for the sums: a token costs about
// one trip to memory and one exchange.
//
// First product: the rank is the instruction's 16 rows, tokens its 8 columns.
// Second: 16 tokens are its rows, and the columns 8t + 2j + {0, 1} of a unit of
// 32 are its columns 2t, 2t + 1 in the unit's instruction j, so that a lane ends
// up with 8 consecutive results of a token.
//
// Bound: the adapters' weights, read once, and latency. One token, 4096 x 4096,
// rank 16: 4.0 us. 64 tokens of 48 adapters, 4096 x 11008, rank 32: 12.5 us for
// 50 MB, 4.0 TB/s; warps wait for memory half of their time, in a few trips one
// after another (plan, tokens and A, exchange, B).

// Elements k .. k + 7 of a row of n, zeros beyond. al: bytes the rows start at multiples of (FAST: 16).
template <bool FAST> __device__ __forceinline__ uint4 row8(const uint16_t *p, int k, int n, int al) {
    if (k >= n) return make_uint4(0u, 0u, 0u, 0u);
    if constexpr (FAST) return __ldg(reinterpret_cast<const uint4 *>(p + k));
    if (al == 16 && k + 8 <= n) return __ldg(reinterpret_cast<const uint4 *>(p + k));
    if (al >= 8 && k + 8 <= n) {
        const uint2 lo = __ldg(reinterpret_cast<const uint2 *>(p + k)), hi = __ldg(reinterpret_cast<const uint2 *>(p + k + 4));
        return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    return load8(p + k, n - k);
}

// Eight consecutive values of base, as they lie there (fp32: two vectors).
struct Base8 {
    uint4 v[2];
};

// RB: blocks of 16 ranks; NB: blocks of 8 tokens. FAST: every row starts at a 16-byte multiple and holds whole vectors.
template <typename T, int RB, int NB, bool FAST>
__global__ void __launch_bounds__(kThreads, RB * NB <= 4 ? 2 : 1) small_kernel(const SmallArgs a, int out_f32) {
    constexpr int RP = 16 * RB, TOK = 8 * NB, UP = RP + 4;
    constexpr int RK = (RB + 1) / 2;                        // 32-rank pieces of B's rows
    constexpr int PRE = RK == 1 ? (NB == 1 ? 3 : 2) : 1;      // units fetched ahead: what 128 registers hold
    extern __shared__ __align__(128) uint8_t smem[];
    float(*part)[TOK][UP] = reinterpret_cast<float(*)[TOK][UP]>(smem);                                 // [warp]
    float(*slot)[TOK][RP] = reinterpret_cast<float(*)[TOK][RP]>(smem + 8 * TOK * UP * sizeof(float));  // [rank]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int c = a.cluster;
    const int rank = c > 1 ? static_cast<int>(tc::cluster_ctarank()) : 0;
    pdl_launch_dependents();
    pdl_wait();
    if (static_cast<int>(blockIdx.x) >= a.tiles * c) {      // whole clusters
        pass_rows<T>(a.pass, out_f32 != 0, blockIdx.x - a.tiles * c, gridDim.x - a.tiles * c);
        return;
    }
    if (c > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this CTA has started
    const AdapterTile tile = a.plan.tiles[blockIdx.x / c];
    const uint16_t *A = a.A + static_cast<int64_t>(tile.adapter) * a.R * a.K;
    const uint16_t *B = a.B + static_cast<int64_t>(tile.adapter) * a.R * a.N;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    int row[NB];                                            // tokens g and g + 8
    bool live[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        live[j] = 8 * j + g < tile.n;
        row[j] = a.plan.rows[tile.first + (live[j] ? 8 * j + g : 0)];
    }

    // this CTA's columns, in units of 32; this warp's are n0 + warp, n0 + warp + 8, ...
    const int units = (a.N + 31) / 32;
    const int n0 = static_cast<int>(static_cast<int64_t>(units) * rank / c);
    const int n1 = static_cast<int>(static_cast<int64_t>(units) * (rank + 1) / c);
    auto load_b = [&](int unit, uint4 (&w)[4][RK]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = 32 * unit + 8 * (g >> 1) + 2 * j + (g & 1);
            const uint16_t *p = B + static_cast<int64_t>(n) * a.R;
#pragma unroll
            for (int q = 0; q < RK; ++q) w[j][q] = unit < n1 && n < a.N ? row8<FAST>(p, 32 * q + 8 * t, a.R, a.ab) : zero;
        }
    };
    auto load_base = [&](int unit, Base8 (&b)[NB]) {
        const int n = 32 * unit + 8 * t;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            b[j].v[0] = b[j].v[1] = zero;
            if (a.base == nullptr || !live[j] || unit >= n1 || n >= a.N) continue;
            const int64_t at = row[j] * a.ldb + n;
            if (a.base_f32) {
                const float *p = static_cast<const float *>(a.base) + at;
                if (FAST || a.wide) {
                    b[j].v[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
                    b[j].v[1] = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
                } else {
                    uint32_t f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = n + e < a.N ? __float_as_uint(p[e]) : 0u;
                    b[j].v[0] = make_uint4(f[0], f[1], f[2], f[3]);
                    b[j].v[1] = make_uint4(f[4], f[5], f[6], f[7]);
                }
            } else {
                const uint16_t *p = static_cast<const uint16_t *>(a.base) + at;
                if (FAST || a.wide) {
                    b[j].v[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
                } else {
                    uint32_t f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = (n + 2 * e < a.N ? p[2 * e] : 0u) | (n + 2 * e + 1 < a.N ? static_cast<uint32_t>(p[2 * e + 1]) << 16 : 0u);
                    b[j].v[0] = make_uint4(f[0], f[1], f[2], f[3]);
                }
            }
        }
    };

    uint4 wb[PRE][4][RK];
    Base8 bb[PRE][NB];
#pragma unroll
    for (int i = 0; i < PRE; ++i) {
        load_b(n0 + warp + 8 * i, wb[i]);
        load_base(n0 + warp + 8 * i, bb[i]);
    }
    float acc[RB][NB][4];
#pragma unroll
    for (int m = 0; m < RB; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[m][j][e] = 0.0f;
    // this warp's steps of 32 elements
    const int steps = (a.K + 31) / 32, who = rank * 8 + warp, all = c * 8;
#pragma unroll 2
    for (int s = who; s < steps; s += all) {
        const int k = 32 * s + 8 * t;
        uint4 xv[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) xv[j] = live[j] ? row8<FAST>(a.x + row[j] * a.ldx, k, a.K, a.ax) : zero;
#pragma unroll
        for (int m = 0; m < RB; ++m) {
            const int r0 = 16 * m + g, r1 = r0 + 8;
            const uint4 w0 = r0 < a.R ? row8<FAST>(A + static_cast<int64_t>(r0) * a.K, k, a.K, a.aa) : zero;
            const uint4 w1 = r1 < a.R ? row8<FAST>(A + static_cast<int64_t>(r1) * a.K, k, a.K, a.aa) : zero;
            const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                mma<T>(acc[m][j], f0, xv[j].x, xv[j].y);
                mma<T>(acc[m][j], f1, xv[j].z, xv[j].w);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < RB; ++m)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[warp][8 * j + 2 * t + (e & 1)][16 * m + g + (e >> 1) * 8] = acc[m][j][e];
    __syncthreads();
    if (c > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");             // every CTA of the cluster has
    for (int i = tid; i < TOK * RP; i += kThreads) {
        const int tok = i / RP, r = i % RP;
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += part[w][tok][r];
        const uint32_t at = smem_u32(&slot[rank][tok][r]);
        if (c == 1) {
            slot[0][tok][r] = v;
        } else {
            for (int q = 0; q < c; ++q)
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa(at, q)), "f"(v) : "memory");
        }
    }
    if (c > 1) tc::cluster_sync();
    else __syncthreads();
    // u of this tile's tokens, whole, in part[0]
    float(*u)[UP] = part[0];
    for (int i = tid; i < TOK * RP; i += kThreads) {
        const int tok = i / RP, r = i % RP;
        float v = 0.0f;
        for (int q = 0; q < c; ++q) v += slot[q][tok][r];
        u[tok][r] = r < a.R ? v : 0.0f;                     // an infinity among x makes NaN of it and the padding's zeros
        if (a.u != nullptr && rank == 0 && tok < tile.n && r < a.R)
            a.u[static_cast<int64_t>(a.plan.rows[tile.first + tok]) * a.R + r] = v;
    }
    __syncthreads();
    // its fragments: lane t of a quad holds ranks 32q + 8t .. + 7 of token g (and g + 8)
    const float s = a.scale[tile.adapter];
    constexpr bool REST = kValues<T> == 3;
    uint32_t uh[RK][NB][4], ul[RK][NB][4], ur[RK][NB][4];
    float mul[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        float v[RK][8], amax = 0.0f;
#pragma unroll
        for (int q = 0; q < RK; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int r = 32 * q + 8 * t + e;
                v[q][e] = r < RP ? u[8 * j + g][r] : 0.0f;
                amax = fmaxf(amax, finite_size(v[q][e]));
            }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const float p = row_power<T>(amax);
        mul[j] = s / p;
#pragma unroll
        for (int q = 0; q < RK; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v0 = v[q][2 * e] * p, v1 = v[q][2 * e + 1] * p;
                split2<T>(v0, v1, uh[q][j][e], ul[q][j][e]);
                if constexpr (REST) ur[q][j][e] = split_rest<T>(v0, v1, uh[q][j][e], ul[q][j][e]);
            }
    }
    for (int first = n0 + warp; first < n1; first += 8 * PRE) {
#pragma unroll
        for (int i = 0; i < PRE; ++i) {
            const int unit = first + 8 * i;
            if (unit >= n1) break;
            float d[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.0f;
#pragma unroll
                for (int q = 0; q < RK; ++q) {
                    const uint4 w = wb[i][j][q];
                    auto add = [&](const uint32_t (&lo)[4], const uint32_t (&hi)[4]) {     // rows 0..7 and 8..15
                        const uint32_t f0[4] = {lo[0], hi[0], lo[1], hi[1]}, f1[4] = {lo[2], hi[2], lo[3], hi[3]};
                        mma<T>(d[j], f0, w.x, w.y);
                        mma<T>(d[j], f1, w.z, w.w);
                    };
                    if constexpr (NB == 1) {                // no tokens 8..15: the second value takes their rows
                        const uint32_t none[4] = {0u, 0u, 0u, 0u};
                        add(uh[q][0], ul[q][0]);
                        if constexpr (REST) add(ur[q][0], none);
                    } else {
                        add(uh[q][0], uh[q][NB - 1]);
                        add(ul[q][0], ul[q][NB - 1]);
                        if constexpr (REST) add(ur[q][0], ur[q][NB - 1]);
                    }
                }
                if constexpr (NB == 1) {
                    d[j][0] += d[j][2];
                    d[j][1] += d[j][3];
                }
            }
            load_b(unit + 8 * PRE, wb[i]);
            const int n = 32 * unit + 8 * t;
            float f[NB][8];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const uint4 v0 = bb[i][j].v[0], v1 = bb[i][j].v[1];
                if (a.base_f32) {
                    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[j][e] = __uint_as_float(w[e]);
                } else {
                    const uint32_t w[4] = {v0.x, v0.y, v0.z, v0.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 p = unpack2<T>(w[e]);
                        f[j][2 * e] = p.x;
                        f[j][2 * e + 1] = p.y;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) f[j][e] = __fmaf_rn(d[e >> 1][2 * j + (e & 1)], mul[j], f[j][e]);
            }
            load_base(unit + 8 * PRE, bb[i]);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                if (!live[j] || n >= a.N) continue;
                const int64_t at = row[j] * a.ldo + n;
                if (out_f32) {
                    float *o = static_cast<float *>(a.out) + at;
                    if (FAST || a.wide) {
                        *reinterpret_cast<float4 *>(o) = make_float4(f[j][0], f[j][1], f[j][2], f[j][3]);
                        *(reinterpret_cast<float4 *>(o) + 1) = make_float4(f[j][4], f[j][5], f[j][6], f[j][7]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < a.N) o[e] = f[j][e];
                    }
                } else {
                    uint16_t *o = static_cast<uint16_t *>(a.out) + at;
                    if (FAST || a.wide) {
                        *reinterpret_cast<uint4 *>(o) = make_uint4(pack2<T>(f[j][0], f[j][1]), pack2<T>(f[j][2], f[j][3]),
                                                                   pack2<T>(f[j][4], f[j][5]), pack2<T>(f[j][6], f[j][7]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < a.N) o[e] = static_cast<uint16_t>(bits16(to16<T>(f[j][e])));
                    }
                }
            }
        }
    }
}

template <typename T, int RB, int NB, bool FAST>
cudaError_t launch_f(SmallArgs a, bool out_f32, int tiles, cudaStream_t s) {
    auto kern = small_kernel<T, RB, NB, FAST>;
    constexpr int smem = 8 * 8 * NB * (32 * RB + 4) * static_cast<int>(sizeof(float));
    static ContextOnce once;
    if (const cudaError_t err = allow_smem(kern, smem, once); err != cudaSuccess) return err;
    double us;
    const int c = small_cluster(tiles, 8 * NB, a.K, a.N, a.R, &us);
    a.cluster = c;
    a.tiles = tiles;
    const int64_t pieces = pass_pieces(a.pass);
    const int pass = static_cast<int>(pieces < 2 * device_sm_count() ? pieces : 2 * device_sm_count());
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attribute();
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(c);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>((tiles + (pass + c - 1) / c) * c));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<const SmallArgs>(a), static_cast<int>(out_f32));
}
template <typename T, int RB, int NB> cudaError_t launch_rn(const SmallArgs &a, bool out_f32, int tiles, cudaStream_t s) {
    const bool fast = a.ax == 16 && a.aa == 16 && a.ab == 16 && a.wide;
    return fast ? launch_f<T, RB, NB, true>(a, out_f32, tiles, s) : launch_f<T, RB, NB, false>(a, out_f32, tiles, s);
}
template <typename T, int NB> cudaError_t launch_n(const SmallArgs &a, bool out_f32, int tiles, cudaStream_t s) {
    if (a.R <= 16) return launch_rn<T, 1, NB>(a, out_f32, tiles, s);
    if (a.R <= 32) return launch_rn<T, 2, NB>(a, out_f32, tiles, s);
    if (a.R <= 64) return launch_rn<T, 4, NB>(a, out_f32, tiles, s);
    return launch_rn<T, 8, NB>(a, out_f32, tiles, s);
}
template <typename T> cudaError_t launch_t(const SmallArgs &a, bool out_f32, int tiles, int most, cudaStream_t s) {
    return most <= 8 ? launch_n<T, 1>(a, out_f32, tiles, s) : launch_n<T, 2>(a, out_f32, tiles, s);
}

}  // namespace

int small_cluster(int64_t tiles, int most, int64_t K, int64_t N, int64_t R, double *us) {
    // the model of takes_small (adapter.cu); two CTAs an SM, but one where their registers do not allow it; clusters
    // do not fill every group of SMs
    const int per_sm = padded_rank(static_cast<int>(R)) / 16 * (most <= 8 ? 1 : 2) <= 4 ? 2 : 1;
    const double fill[4] = {1.0, 0.97, 0.9, per_sm == 2 ? 0.88 : 0.75};
    int best = 1;
    for (int i = 0; i < 4; ++i) {
        const int c = 1 << i;
        const double slots = device_sm_count() * per_sm * fill[i];
        const double waves = static_cast<double>(static_cast<int64_t>((static_cast<double>(tiles) * c + slots - 1.0) / slots));
        const double t = 2.3 + (waves < 1.0 ? 1.0 : waves) * (0.7 + static_cast<double>(R) * static_cast<double>(K + N) * 2.0 / c / 42e3);
        if (i == 0 || t < *us) {
            *us = t;
            best = c;
        }
    }
    return best;
}

cudaError_t launch_small(bt_dtype t, bool out_f32, const SmallArgs &a, int tiles, int most, cudaStream_t s) {
    if (tiles == 0) return cudaSuccess;
    return t == BT_F16 ? launch_t<__half>(a, out_f32, tiles, most, s) : launch_t<__nv_bfloat16>(a, out_f32, tiles, most, s);
}

}  // namespace adapter
}  // namespace bt
