// Low-rank adapters of many requests beside one shared projection:
//   out_t = cast(base_t + s_a B_a (A_a x_t)),     a = the adapter of token t
// and the gradients
//   dU_t = s_a B_a^T g_t,   dX_t = cast(gbase_t + A_a^T dU_t),
//   dA_a = sum_t dU_t x_t^T,   dB_a = s_a sum_t g_t u_t^T     (u_t = A_a x_t).
//
// Products around a rank R of at most 128, bound by the long rows that they
// read or write once (x, g, base, out: 2 R operations for 2 or 4 bytes), not
// by arithmetic:
//   adapter_shrink.cu   u = A x, dU = s B^T g: reduce the long axis
//   adapter_expand.cu   out = base + s B u, dX: write the long axis
//   adapter_grad.cu     dA, dB: reduce the tokens
//   adapter_small.cu    the whole forward for a few tokens of each adapter
// The 16-bit operands go to the matrix instructions as they are; u and dU, fp32
// sums, go as the sum of three bf16 values (all 24 bits of mantissa) or of two in
// half precision (22 bits), so that the only rounding to 16 bits is the result's own.
//
// Tokens of an adapter are gathered through the plan's row list: a tile's rows
// lie anywhere in the batch.
#include <cstdlib>
#include <cstring>

#include "adapter.cuh"

namespace bt {
namespace {

using namespace adapter;

// The largest of 16, 8, 4, 2 bytes that p and every multiple of `bytes` share.
int align_of(const void *p, int64_t bytes) {
    const uintptr_t v = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(bytes);
    return v % 16 == 0 ? 16 : v % 8 == 0 ? 8 : v % 4 == 0 ? 4 : 2;
}

constexpr int64_t kMaxSide = int64_t(1) << 24;

bool plan_fits(const bt_adapter_plan_info &p, int64_t T) {
    return p.tokens == T && p.adapters >= 1 && p.adapters <= kAdapterMaxAdapters && p.without >= 0 && p.without <= T &&
           p.tiles >= 0 && p.tiles <= T && p.small_tiles >= 0 &&
           p.small_tiles <= T && p.small_most >= 0 && p.small_most <= kAdapterSmall && p.parts >= 1 && p.parts <= 2 * kAdapterParts + p.adapters + 1 && p.slots >= 0 &&
           p.slots <= 2 * kAdapterParts;
}
bt_status sizes_fit(int64_t T, int64_t K, int64_t N, int64_t R) {
    if (T < 0 || K < 1 || N < 0 || R < 1) return BT_ERR_INVALID_ARG;
    if (T > kAdapterMaxTokens || K >= kMaxSide || N >= kMaxSide || R > kAdapterMaxRank) return BT_ERR_UNSUPPORTED;
    return BT_OK;
}

// u as two or three 16-bit values a rank, in a workspace: the bytes of one, and where they lie (unpower has the
// third one's place).
size_t split_bytes(int64_t T, int64_t R) { return round_up256(static_cast<size_t>(T) * padded_rank(static_cast<int>(R)) * 2); }
SplitRows split_rows(void *p, int64_t T, int R, bool rest, bool unpower) {
    const size_t one = split_bytes(T, R);
    uint8_t *b = static_cast<uint8_t *>(p);
    return SplitRows{reinterpret_cast<uint16_t *>(b), reinterpret_cast<uint16_t *>(b + one),
                     rest ? reinterpret_cast<uint16_t *>(b + 2 * one) : nullptr, unpower ? reinterpret_cast<float *>(b + 2 * one) : nullptr};
}

// Rows whose width is odd in this sense are copied to rows that start at 16-byte multiples first: what fetches them
// 2 bytes at a time costs more than the copy (1500 x 4093 backward, rank 24: 51 us without).
bool odd_width(int64_t C) { return C % 4 != 0; }
int64_t aligned_pitch(int64_t C) { return (C + 7) / 8 * 8; }
size_t aligned_bytes(int64_t rows, int64_t C) { return round_up256(static_cast<size_t>(rows) * static_cast<size_t>(aligned_pitch(C)) * 2); }
cudaError_t align_rows(const uint16_t *src, int64_t lds, int64_t rows, int64_t C, uint16_t *dst, cudaStream_t s) {
    AlignArgs a = {};
    a.src = src; a.lds = lds; a.dst = dst; a.ldd = aligned_pitch(C);
    a.C = static_cast<int>(C); a.rows = rows;
    return launch_align(a, s);
}
cudaError_t align_weights(const uint16_t *src, int R, int64_t C, const AdapterTile *parts, int nparts, uint16_t *dst, cudaStream_t s) {
    AlignArgs a = {};
    a.src = src; a.lds = C; a.dst = dst; a.ldd = aligned_pitch(C);
    a.C = static_cast<int>(C); a.R = R; a.parts = parts; a.nparts = nparts;
    return launch_align(a, s);
}

// Which forward a batch takes: everything in one kernel of small tiles, or in two of large ones. Small tiles read an
// adapter's weights once for 16 tokens, large ones once for 128, but two kernels cost more to begin and to join.
// Microseconds, fitted on GB300 in graphs (1 to 6000 tokens, 1 to 48 adapters, ranks 8 to 128): one kernel 2.3, for
// each wave of CTAs 0.7 and its piece of the weights at 42 bytes a nanosecond, and x, base and out at 4.2 TB/s; two
// kernels 8, 0.3 for every 512 of K, and the longer of x, base and out at 4.5 TB/s and 0.7 a tile. One kernel against
// two, 4096 x 4096, rank 16: one token 4.0 and 10.0, 768 tokens of one adapter 9.4 and 13.4, 6000 54.0 and 43.4; rank
// 64: 256 tokens 11.1 and 12.8, 2048 30.5 and 24.0; 64 tokens of 48 adapters 11.7 and 38.0. BT_ADAPTER_PATH=small|large
// in the environment decides instead.
bool takes_small(const bt_adapter_plan_info &p, int64_t T, int64_t K, int64_t N, int64_t R) {
    if (const char *e = std::getenv("BT_ADAPTER_PATH")) {
        if (std::strcmp(e, "small") == 0) return true;
        if (std::strcmp(e, "large") == 0) return false;
    }
    double small;
    small_cluster(p.small_tiles, p.small_most, K, N, R, &small);
    const double bytes = static_cast<double>(T) * static_cast<double>(K + 2 * N) * 2.0;
    const double rows = bytes / 4.5e6, tiles = 0.7 * static_cast<double>(p.tiles);
    // Widths that are no multiples of 8: one kernel fetches and stores by elements. Over 99 such sizes (515 to 11005
    // wide, ranks 8 to 64, 1 to 2048 tokens of 1 to 48 adapters) the choice by this factor takes 1.3 % longer than the
    // better of the two on average, 43 % at worst; by 2 and by 3 it is 1.6 and 9 %. One kernel against two, 4100 x
    // 4093, rank 24: one token 8.8 and 14.5 us, 777 tokens of 12 adapters 31.2 and 25.8; 2050 x 2051, rank 16: 256
    // tokens 12.5 and 18.8; 4093 x 11005, rank 32: 64 tokens of 12 adapters 21.7 and 35.3, of one 25.6 and 19.3.
    const double slow = (K | N | R) % 8 == 0 ? 1.0 : 2.3;
    return slow * (small + bytes / 4.2e6) < 8.0 + 0.3 * static_cast<double>((K + 511) / 512) + (rows > tiles ? rows : tiles);
}

struct Forward {
    const uint16_t *x, *A, *B;
    int64_t ldx, ldb, ldo;
    const float *scale;
    const int32_t *plan;
    const bt_adapter_plan_info *info;
    int64_t T;
    int K, N, R;
    const void *base;
    int base_f32;
    void *out;
    float *u;                  // NULL: not wanted
    void *workspace;
    bool out_f32, small;
    bt_dtype type;
    unsigned int *err;
};

cudaError_t forward(const Forward &f, cudaStream_t s) {
    const bt_dtype t = f.type;
    const bool of32 = f.out_f32;
    const AdapterPlanLayout lay = adapter_plan_layout(f.T, f.info->adapters);
    const Plan plan{f.plan + lay.rows, reinterpret_cast<const AdapterTile *>(f.plan + lay.tiles)};
    const bool wide = align_of(f.out, f.ldo * (of32 ? 4 : 2)) == 16 && f.N % 8 == 0 &&
                      (f.base == nullptr || align_of(f.base, f.ldb * (f.base_f32 ? 4 : 2)) == 16);
    // tokens without an adapter go along with the first kernel that writes results
    PassArgs pa = {};
    pa.n = f.info->without;
    pa.rows = plan.rows + (f.T - pa.n);
    pa.N = f.N; pa.R = f.R;
    pa.base = f.base; pa.base_f32 = f.base_f32; pa.ldb = f.ldb;
    pa.out = f.out == f.base ? nullptr : f.out; pa.ldo = f.ldo;
    pa.u = f.u;
    if (pa.out == nullptr && pa.u == nullptr) pa.n = 0;
    cudaError_t e;
    if (f.info->tiles == 0) return launch_pass(t, of32, pa, s);
    if (f.small) {
        SmallArgs sm = {};
        sm.plan = Plan{plan.rows, reinterpret_cast<const AdapterTile *>(f.plan + lay.small)};
        sm.x = f.x; sm.A = f.A; sm.B = f.B; sm.ldx = f.ldx;
        sm.K = f.K; sm.N = f.N; sm.R = f.R;
        sm.ax = align_of(f.x, f.ldx * 2);
        sm.aa = align_of(f.A, int64_t(f.K) * 2);
        sm.ab = align_of(f.B, int64_t(f.R) * 2);
        sm.wide = wide;
        sm.scale = f.scale;
        sm.base = f.base; sm.base_f32 = f.base_f32; sm.ldb = f.ldb;
        sm.out = f.out; sm.ldo = f.ldo;
        sm.u = f.u;
        sm.pass = pa;
        return launch_small(t, of32, sm, f.info->small_tiles, f.info->small_most, s);
    }
    ShrinkArgs sh = {};
    sh.plan = plan;
    sh.x = f.x; sh.ldx = f.ldx;
    sh.w = f.A; sh.ldw = f.K;
    if (odd_width(f.K)) {
        uint8_t *ws = static_cast<uint8_t *>(f.workspace) + 3 * split_bytes(f.T, f.R);
        uint16_t *xa = reinterpret_cast<uint16_t *>(ws), *Aa = reinterpret_cast<uint16_t *>(ws + aligned_bytes(f.T, f.K));
        e = align_rows(f.x, f.ldx, f.T, f.K, xa, s);
        if (e == cudaSuccess)
            e = align_weights(f.A, f.R, f.K, reinterpret_cast<const AdapterTile *>(f.plan + lay.parts), f.info->parts, Aa, s);
        if (e != cudaSuccess) return e;
        sh.x = xa; sh.w = Aa;
        sh.ldx = sh.ldw = aligned_pitch(f.K);
    }
    sh.ax = align_of(sh.x, sh.ldx * 2);
    sh.aw = align_of(sh.w, sh.ldw * 2);
    sh.C = f.K; sh.R = f.R; sh.u = f.u;
    sh.out = split_rows(f.workspace, f.T, f.R, t == BT_BF16, t == BT_F16);
    sh.err = f.err; sh.limit_ns = wait_limit_ns();
    e = launch_shrink(t, false, sh, f.info->tiles, s);
    if (e != cudaSuccess) return e;
    ExpandArgs ex = {};
    ex.plan = plan;
    ex.pass = pa;
    ex.u = sh.out; ex.w = f.B; ex.aw = align_of(f.B, int64_t(f.R) * 2);
    ex.C = f.N; ex.R = f.R; ex.scale = f.scale;
    ex.base = f.base; ex.base_f32 = f.base_f32; ex.ldb = f.ldb;
    ex.out = f.out; ex.ldo = f.ldo;
    ex.wide = wide;
    ex.err = f.err; ex.limit_ns = wait_limit_ns();
    return launch_expand(t, false, of32, ex, f.info->tiles, s);
}

}  // namespace
}  // namespace bt

using namespace bt;
using namespace bt::adapter;

extern "C" {

size_t bt_adapter_linear_workspace(int64_t T, int64_t K, int64_t N, int64_t R, const bt_adapter_plan_info *info) {
    if (sizes_fit(T, K, N, R) != BT_OK || info == nullptr || !plan_fits(*info, T) || info->tiles == 0 || takes_small(*info, T, K, N, R))
        return 0;
    size_t n = 3 * split_bytes(T, R);
    if (odd_width(K)) n += aligned_bytes(T, K) + aligned_bytes(info->adapters * R, K);
    return n;
}

bt_status bt_adapter_linear(const void *x, bt_dtype x_dtype, int64_t ldx, const void *A, const void *B,
                            const float *scale, const void *plan, const bt_adapter_plan_info *info, int64_t T,
                            int64_t K, int64_t N, int64_t R, const void *base, bt_dtype base_dtype, int64_t ldb,
                            void *out, bt_dtype out_dtype, int64_t ldo, float *u, void *workspace,
                            size_t workspace_bytes, bt_stream stream) {
    if (x_dtype != BT_BF16 && x_dtype != BT_F16) return BT_ERR_INVALID_ARG;
    if (out_dtype != BT_F32 && out_dtype != x_dtype) return BT_ERR_INVALID_ARG;
    if (base != nullptr && base_dtype != BT_F32 && base_dtype != x_dtype) return BT_ERR_INVALID_ARG;
    const bt_status fit = sizes_fit(T, K, N, R);
    if (fit != BT_OK) return fit;
    if (ldx < K || ldo < N || (base != nullptr && ldb < N)) return BT_ERR_INVALID_ARG;
    if (ldx > (int64_t(1) << 36) || ldo > (int64_t(1) << 36) || ldb > (int64_t(1) << 36)) return BT_ERR_UNSUPPORTED;
    if (info == nullptr || !plan_fits(*info, T)) return BT_ERR_INVALID_ARG;
    if (T == 0 || N == 0) return BT_OK;
    if (x == nullptr || A == nullptr || B == nullptr || scale == nullptr || plan == nullptr || out == nullptr)
        return BT_ERR_INVALID_ARG;
    if (out == base && (out_dtype != base_dtype || ldo != ldb)) return BT_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(scale, 4) || !aligned(plan, 16) || !aligned(u, 16) ||
        !aligned(out, dtype_bytes(out_dtype)) || (base != nullptr && !aligned(base, dtype_bytes(base_dtype))))
        return BT_ERR_ALIGNMENT;
    const size_t need = bt_adapter_linear_workspace(T, K, N, R, info);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return BT_ERR_WORKSPACE;
    if (need > 0 && !aligned(workspace, 256)) return BT_ERR_ALIGNMENT;
    Forward f = {};
    f.x = static_cast<const uint16_t *>(x);
    f.A = static_cast<const uint16_t *>(A);
    f.B = static_cast<const uint16_t *>(B);
    f.ldx = ldx; f.ldb = ldb; f.ldo = ldo;
    f.scale = scale;
    f.plan = static_cast<const int32_t *>(plan);
    f.info = info;
    f.T = T; f.K = static_cast<int>(K); f.N = static_cast<int>(N); f.R = static_cast<int>(R);
    f.base = base; f.base_f32 = base_dtype == BT_F32;
    f.out = out;
    f.u = u;
    f.workspace = workspace;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    f.out_f32 = out_dtype == BT_F32;
    f.type = x_dtype;
    f.small = need == 0;
    if (!f.small && (f.err = device_error_word()) == nullptr) return BT_ERR_CUDA;
    const cudaError_t e = forward(f, s);
    return e == cudaSuccess ? BT_OK : BT_ERR_CUDA;
}

static size_t arrived_bytes(const bt_adapter_plan_info &info, int64_t K, int64_t N) {
    return round_up256(static_cast<size_t>(info.slots) * static_cast<size_t>((K + 127) / 128 + (N + 127) / 128) * 4);
}

size_t bt_adapter_linear_backward_workspace(int64_t T, int64_t K, int64_t N, int64_t R,
                                            const bt_adapter_plan_info *info) {
    if (sizes_fit(T, K, N, R) != BT_OK || info == nullptr || !plan_fits(*info, T)) return 0;
    const size_t slot = round_up256(static_cast<size_t>(R * K) * 4) + round_up256(static_cast<size_t>(R * N) * 4);
    size_t n = 6 * split_bytes(T, R) + static_cast<size_t>(info->slots) * slot + arrived_bytes(*info, K, N);
    if (odd_width(N)) n += aligned_bytes(T, N);
    if (odd_width(K)) n += aligned_bytes(T, K) + aligned_bytes(info->adapters * R, K);
    return n;
}

bt_status bt_adapter_linear_backward(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *u,
                                     const void *A, const void *B, const float *scale, const void *plan,
                                     const bt_adapter_plan_info *info, int64_t T, int64_t K, int64_t N, int64_t R,
                                     const void *grad_base, int64_t ldgb, void *grad_x, int64_t ldgx, float *grad_A,
                                     float *grad_B, void *workspace, size_t workspace_bytes, bt_stream stream) {
    const bt_status fit = sizes_fit(T, K, N, R);
    if (fit != BT_OK) return fit;
    if (N < 1 || ldx < K || ldg < N || ldgx < K || (grad_base != nullptr && ldgb < K)) return BT_ERR_INVALID_ARG;
    if (ldx > (int64_t(1) << 36) || ldg > (int64_t(1) << 36) || ldgx > (int64_t(1) << 36) || ldgb > (int64_t(1) << 36))
        return BT_ERR_UNSUPPORTED;
    if (info == nullptr || !plan_fits(*info, T)) return BT_ERR_INVALID_ARG;
    if (static_cast<int64_t>(info->parts) * ((K + N) / 128 + 2) > 0x7FFFFFFF) return BT_ERR_UNSUPPORTED;
    if (plan == nullptr || grad_A == nullptr || grad_B == nullptr) return BT_ERR_INVALID_ARG;
    if (T > 0 && (x == nullptr || g == nullptr || u == nullptr || A == nullptr || B == nullptr || scale == nullptr ||
                  grad_x == nullptr))
        return BT_ERR_INVALID_ARG;
    if (grad_x != nullptr && grad_x == grad_base && ldgx != ldgb) return BT_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(g, 2) || !aligned(u, 16) || !aligned(A, 2) || !aligned(B, 2) || !aligned(scale, 4) ||
        !aligned(plan, 16) || !aligned(grad_base, 2) || !aligned(grad_x, 2) || !aligned(grad_A, 16) ||
        !aligned(grad_B, 16))
        return BT_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        const size_t n = static_cast<size_t>(info->adapters) * static_cast<size_t>(R) * 4;
        return cudaMemsetAsync(grad_A, 0, n * static_cast<size_t>(K), s) == cudaSuccess &&
               cudaMemsetAsync(grad_B, 0, n * static_cast<size_t>(N), s) == cudaSuccess ? BT_OK : BT_ERR_CUDA;
    }
    const size_t need = bt_adapter_linear_backward_workspace(T, K, N, R, info);
    if (workspace == nullptr || workspace_bytes < need) return BT_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BT_ERR_ALIGNMENT;

    unsigned int *err = device_error_word();
    if (err == nullptr) return BT_ERR_CUDA;
    const uint16_t *xp = static_cast<const uint16_t *>(x), *gp = static_cast<const uint16_t *>(g);
    const uint16_t *Ap = static_cast<const uint16_t *>(A), *Bp = static_cast<const uint16_t *>(B);
    const int32_t *pw = static_cast<const int32_t *>(plan);
    const AdapterPlanLayout lay = adapter_plan_layout(T, info->adapters);
    const Plan tiles{pw + lay.rows, reinterpret_cast<const AdapterTile *>(pw + lay.tiles)};
    const Plan parts{pw + lay.rows, reinterpret_cast<const AdapterTile *>(pw + lay.parts)};
    const size_t split = 3 * split_bytes(T, R);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const SplitRows du = split_rows(ws, T, static_cast<int>(R), true, false);
    const SplitRows us = split_rows(ws + split, T, static_cast<int>(R), true, false);
    float *slots = reinterpret_cast<float *>(ws + 2 * split);
    const int64_t off_b = static_cast<int64_t>(round_up256(static_cast<size_t>(R * K) * 4) / 4);
    const int64_t stride = off_b + static_cast<int64_t>(round_up256(static_cast<size_t>(R * N) * 4) / 4);
    uint8_t *rest = ws + 2 * split + static_cast<size_t>(info->slots) * static_cast<size_t>(stride) * 4;
    unsigned int *arrived = reinterpret_cast<unsigned int *>(rest);
    rest += arrived_bytes(*info, K, N);
    int64_t ldA = K;
    if (odd_width(N)) {
        uint16_t *ga = reinterpret_cast<uint16_t *>(rest);
        rest += aligned_bytes(T, N);
        if (align_rows(gp, ldg, T, N, ga, s) != cudaSuccess) return BT_ERR_CUDA;
        gp = ga;
        ldg = aligned_pitch(N);
    }
    if (odd_width(K)) {
        uint16_t *xa = reinterpret_cast<uint16_t *>(rest), *Aa = reinterpret_cast<uint16_t *>(rest + aligned_bytes(T, K));
        if (align_rows(xp, ldx, T, K, xa, s) != cudaSuccess ||
            align_weights(Ap, static_cast<int>(R), K, parts.tiles, info->parts, Aa, s) != cudaSuccess)
            return BT_ERR_CUDA;
        xp = xa;
        Ap = Aa;
        ldx = ldA = aligned_pitch(K);
    }
    const int ax = align_of(xp, ldx * 2), ag = align_of(gp, ldg * 2);

    ShrinkArgs sh = {};
    sh.plan = tiles;
    sh.x = gp; sh.ldx = ldg; sh.ax = ag;
    sh.w = Bp; sh.aw = align_of(B, R * 2);
    sh.C = static_cast<int>(N); sh.R = static_cast<int>(R);
    sh.scale = scale; sh.out = du;
    sh.given = u; sh.given_out = us;
    sh.zero = arrived;
    sh.zeros = info->slots * static_cast<int>((K + 127) / 128 + (N + 127) / 128);
    sh.err = err; sh.limit_ns = wait_limit_ns();
    cudaError_t e = launch_shrink(BT_BF16, true, sh, info->tiles, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;

    GradArgs gr = {};
    gr.plan = parts;
    gr.R = static_cast<int>(R);
    gr.slot_stride = stride;
    gr.arrived = arrived;
    gr.alone = info->tiles == 0;
    gr.err = err; gr.limit_ns = wait_limit_ns();
    gr.p[0].u = us; gr.p[0].x = gp; gr.p[0].ldx = ldg; gr.p[0].ax = ag;
    gr.p[0].C = static_cast<int>(N); gr.p[0].rc = 0;
    gr.p[0].scale = scale; gr.p[0].grad = grad_B; gr.p[0].slots = slots + off_b;
    gr.p[1].u = du; gr.p[1].x = xp; gr.p[1].ldx = ldx; gr.p[1].ax = ax;
    gr.p[1].C = static_cast<int>(K); gr.p[1].rc = 1;
    gr.p[1].grad = grad_A; gr.p[1].slots = slots;
    e = launch_grad(gr, info->parts, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;

    PassArgs pa = {};
    pa.n = info->without;
    pa.rows = tiles.rows + (T - pa.n);
    pa.N = static_cast<int>(K); pa.R = static_cast<int>(R);
    pa.base = grad_base; pa.ldb = ldgb;
    pa.out = grad_x == grad_base ? nullptr : grad_x; pa.ldo = ldgx;
    if (pa.out == nullptr) pa.n = 0;
    if (info->tiles == 0 && launch_pass(BT_BF16, false, pa, s) != cudaSuccess) return BT_ERR_CUDA;
    ExpandArgs ex = {};
    ex.pass = pa;
    ex.plan = tiles;
    ex.u = du; ex.w = Ap;
    ex.err = err; ex.limit_ns = wait_limit_ns(); ex.ldw = ldA; ex.aw = align_of(Ap, ldA * 2);
    ex.C = static_cast<int>(K); ex.R = static_cast<int>(R);
    ex.base = grad_base; ex.ldb = ldgb;
    ex.out = grad_x; ex.ldo = ldgx;
    ex.wide = align_of(grad_x, ldgx * 2) == 16 && (grad_base == nullptr || align_of(grad_base, ldgb * 2) == 16) && K % 8 == 0;
    e = launch_expand(BT_BF16, true, false, ex, info->tiles, s);
    if (e != cudaSuccess) return BT_ERR_CUDA;


    return BT_OK;
}

}  // extern "C"
