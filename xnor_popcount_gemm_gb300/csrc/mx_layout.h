// Where a microscaled operand's scales lie (see mx.cuh), for host and device.
#pragma once

#include <cstddef>
#include <cstdint>

#include "bt.h"

#ifdef __CUDACC__
#define BT_HD __host__ __device__ __forceinline__
#else
#define BT_HD inline
#endif

namespace bt {
namespace mx {

constexpr int kBlock = 32;                  // values that share a scale
constexpr int kAtomBytes = 512;             // 128 rows x 4 blocks
constexpr int64_t kMaxSide = int64_t(1) << 24;

// Rows of codes: whole slices of 128 bytes, what the tensor cores take at a time.
BT_HD int64_t slices(int64_t K, int code) { return code == BT_CODE_E2M1 ? (K + 255) / 256 : (K + 127) / 128; }
BT_HD int64_t code_bytes(int64_t K, int code) { return slices(K, code) * 128; }
// Atoms along a row: those of its slices.
BT_HD int64_t k_atoms(int64_t K, int code) { return slices(K, code) * (code == BT_CODE_E2M1 ? 2 : 1); }
BT_HD size_t scale_bytes(int64_t R, int64_t K, int code) {
    return static_cast<size_t>((R + 127) / 128) * static_cast<size_t>(k_atoms(K, code)) * kAtomBytes;
}
// Byte of row r, block b.
BT_HD int64_t scale_at(int64_t r, int64_t b, int64_t atoms) {
    return ((r >> 7) * atoms + (b >> 2)) * kAtomBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

}  // namespace mx
}  // namespace bt
