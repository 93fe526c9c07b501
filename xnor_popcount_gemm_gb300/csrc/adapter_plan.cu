// The plan of a batch's adapters, built on the host: which token uses which
// adapter is known to the scheduler that put the batch together, so the sorting
// costs no launch and no synchronisation, and every projection of every layer
// shares one plan. Checks that the kernels rely on (every adapter index in
// range, every row once) are made here.
#include <algorithm>
#include <cstdlib>
#include <cstring>
#include <memory>

#include "adapter_plan.h"

namespace bt {

// Words of the plan: rows [T], the tiles, the small tiles, the gradient's parts.
AdapterPlanLayout adapter_plan_layout(int64_t T, int64_t L) {
    AdapterPlanLayout p;
    const int64_t tiles = T < T / kAdapterTile + L + 1 ? T : T / kAdapterTile + L + 1;
    const int64_t small = T < T / kAdapterSmall + L + 1 ? T : T / kAdapterSmall + L + 1;
    p.rows = 0;
    p.tiles = (T + 3) / 4 * 4;
    p.small = p.tiles + 4 * tiles;
    p.parts = p.small + 4 * small;
    p.words = p.parts + 4 * (2 * kAdapterParts + L + 1);
    return p;
}

}  // namespace bt

using namespace bt;

extern "C" {

size_t bt_adapter_plan_bytes(int64_t T, int64_t L) {
    if (T < 0 || T > kAdapterMaxTokens || L < 1 || L > kAdapterMaxAdapters) return 0;
    return static_cast<size_t>(adapter_plan_layout(T, L).words) * 4;
}

bt_status bt_adapter_plan(const int32_t *adapter, int64_t T, int64_t L, void *plan, size_t plan_bytes,
                          bt_adapter_plan_info *info) {
    if (info == nullptr || T < 0 || L < 1) return BT_ERR_INVALID_ARG;
    if (T > kAdapterMaxTokens || L > kAdapterMaxAdapters) return BT_ERR_UNSUPPORTED;
    if (plan == nullptr || (T > 0 && adapter == nullptr)) return BT_ERR_INVALID_ARG;
    if (!aligned(plan, 4)) return BT_ERR_ALIGNMENT;
    const AdapterPlanLayout lay = adapter_plan_layout(T, L);
    if (plan_bytes < static_cast<size_t>(lay.words) * 4) return BT_ERR_WORKSPACE;
    for (int64_t t = 0; t < T; ++t)
        if (adapter[t] < -1 || adapter[t] >= L) return BT_ERR_INVALID_ARG;
    int32_t *w = static_cast<int32_t *>(plan);
    memset(w, 0, static_cast<size_t>(lay.words) * 4);

    // Stable counting sort by adapter, tokens without one last. last[a]: the end of adapter a's rows.
    std::unique_ptr<int32_t, void (*)(void *)> counts(static_cast<int32_t *>(calloc(2 * static_cast<size_t>(L) + 1, 4)), free);
    int32_t *last = counts.get();
    if (last == nullptr) return BT_ERR_WORKSPACE;
    for (int64_t t = 0; t < T; ++t) ++last[adapter[t] < 0 ? L : adapter[t]];
    int32_t off = 0;
    for (int64_t a = 0; a <= L; ++a) {
        const int32_t n = last[a];
        last[a] = off;
        off += n;
    }
    for (int64_t t = 0; t < T; ++t) w[lay.rows + last[adapter[t] < 0 ? L : adapter[t]]++] = static_cast<int32_t>(t);

    bt_adapter_plan_info r = {};
    r.tokens = T;
    r.adapters = L;
    AdapterTile *tiles = reinterpret_cast<AdapterTile *>(w + lay.tiles);
    AdapterTile *small = reinterpret_cast<AdapterTile *>(w + lay.small);
    auto even = [](AdapterTile *out, int32_t a, int32_t first, int32_t n, int32_t most) {
        const int32_t k = (n + most - 1) / most;
        for (int32_t i = 0; i < k; ++i) {
            const int32_t b = static_cast<int32_t>(static_cast<int64_t>(n) * i / k);
            const int32_t e = static_cast<int32_t>(static_cast<int64_t>(n) * (i + 1) / k);
            out[i] = AdapterTile{a, first + b, e - b, 0};
        }
        return k;
    };
    for (int64_t a = 0; a < L; ++a) {
        const int32_t first = a == 0 ? 0 : last[a - 1], n = last[a] - first;
        if (n == 0) continue;
        r.tiles += even(tiles + r.tiles, static_cast<int32_t>(a), first, n, kAdapterTile);
        const int32_t k = even(small + r.small_tiles, static_cast<int32_t>(a), first, n, kAdapterSmall);
        for (int32_t i = 0; i < k; ++i)
            if (small[r.small_tiles + i].n > r.small_most) r.small_most = small[r.small_tiles + i].n;
        r.small_tiles += k;
        if (n > r.most_tokens) r.most_tokens = n;
        ++r.used;
    }
    r.without = static_cast<int32_t>(T) - last[L - 1];

    // The gradients' parts: at most a quarter of the tokens each, or an eighth where
    // one or two adapters have them all (whole 64s, at least 256), every adapter once
    // at least, so that one without tokens gets its zeros. (4096 tokens of 8 adapters,
    // 4096 x 4096, rank 16, backward: quarters 53.4 us, eighths 56.6, halves 55.1.) A
    // split adapter's parts have a slot each for their sums. Adapters with many tokens
    // first: their parts begin first, and what ends last is short.
    const int64_t cut = r.used <= 2 ? kAdapterParts : kAdapterParts / 2;
    int32_t len = static_cast<int32_t>((T + cut - 1) / cut);
    len = len < 256 ? 256 : (len + 63) / 64 * 64;
    int32_t *order = last + L + 1;
    auto count = [&](int32_t a) { return last[a] - (a == 0 ? 0 : last[a - 1]); };
    for (int64_t a = 0; a < L; ++a) order[a] = static_cast<int32_t>(a);
    std::sort(order, order + L, [&](int32_t a, int32_t b) { return count(a) != count(b) ? count(a) > count(b) : a < b; });
    AdapterTile *parts = reinterpret_cast<AdapterTile *>(w + lay.parts);
    for (int64_t i = 0; i < L; ++i) {
        const int32_t a = order[i], n = count(a), first = last[a] - n;
        if (n <= len) {
            parts[r.parts++] = AdapterTile{a, first, n, -1};
        } else {
            const int32_t k = even(parts + r.parts, a, first, n, len);
            for (int32_t q = 0; q < k; ++q) parts[r.parts++].slot = r.slots++;
        }
    }
    *info = r;
    return BT_OK;
}

}  // extern "C"
