// The adapters' plan as the kernels read it.
#pragma once

#include "bt_internal.h"

namespace bt {

constexpr int kAdapterTile = 128;        // rows of a tile of the two-kernel forward and of the backward
constexpr int kAdapterSmall = 16;        // rows of a tile of the one-kernel forward
constexpr int kAdapterParts = 8;         // parts the tokens of a gradient are cut into, at most
constexpr int64_t kAdapterMaxTokens = int64_t(1) << 24;
constexpr int64_t kAdapterMaxAdapters = int64_t(1) << 16;
constexpr int kAdapterMaxRank = 128;

// Rows plan.rows[first .. first + n) of one adapter.
struct AdapterTile {
    int32_t adapter, first, n, slot;
};

struct AdapterPlanLayout {
    int64_t rows, tiles, small, parts, words;    // offsets in 32-bit words
};
AdapterPlanLayout adapter_plan_layout(int64_t T, int64_t L);

}  // namespace bt
