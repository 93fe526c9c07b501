// Shared by the kernels of the product of microscaled operands (mx_linear.cu for many rows, mx_small.cu for few).
#pragma once

#include "bt_internal.h"
#include "mx.cuh"
#include "tc_ptx.cuh"

namespace bt {
namespace mx {

constexpr int kSliceBytes = 128;                // of K that a row has in one slice: 256 E2M1 or 128 E4M3 values
constexpr int kSmemMax = 232448;
__host__ __device__ constexpr int atoms_a_slice(int code) { return code == BT_CODE_E2M1 ? 2 : 1; }

// Instruction descriptor: D = F32, K-major, UE8M0 scales; `id`: the byte of its 32-bit columns that an MMA's scales lie in
// (from), for both operands.
inline uint32_t make_idesc(int code, int m, int n) {
    const uint32_t mn = ((static_cast<uint32_t>(n) >> 3) << 17) | ((static_cast<uint32_t>(m) >> 7) << 27) | (1u << 23);
    return code == BT_CODE_E2M1 ? mn | (1u << 7) | (1u << 10) : mn;
}
__device__ __forceinline__ uint32_t with_id(uint32_t idesc, uint32_t id) { return idesc | (id << 4) | (id << 29); }

// Codes [rows, slices * 128 bytes] as {128, rows, slices}: one copy brings d slices of `box_rows` rows.
inline bool map_codes(CUtensorMap *m, const void *p, int64_t rows, int64_t slices, int box_rows, int d) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {kSliceBytes, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(slices)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(slices) * kSliceBytes, kSliceBytes};
    cuuint32_t box[3] = {kSliceBytes, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(d)};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Scales as words {128 (an atom), atoms of a row, rows / 128}: `box_atoms` of `box_rows` 128-row groups.
inline bool map_scales(CUtensorMap *m, const void *p, int64_t rows, int64_t atoms, int box_rows, int box_atoms) {
    auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    cuuint64_t dims[3] = {kAtomBytes / 4, static_cast<cuuint64_t>(atoms), static_cast<cuuint64_t>((rows + 127) / 128)};
    cuuint64_t strides[2] = {kAtomBytes, static_cast<cuuint64_t>(atoms) * kAtomBytes};
    cuuint32_t box[3] = {kAtomBytes / 4, static_cast<cuuint32_t>(box_atoms), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t one[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A call: x of float type (xs NULL) or an operand.
struct Product {
    const void *x;
    bt_dtype x_t;                               // BT_PACKED: an operand
    int64_t ldx;
    const uint8_t *xs, *w, *ws;
    bt_code code;
    int64_t M, N, K;
    void *out;
    int64_t ldo;
    bt_dtype out_t;
    unsigned int *err;
};

// Up to kSmallRows rows of x; of float type up to kOwnRows, which the kernel quantises itself. split: CTAs along K (1, 2, 4, 8;
// 0: chosen).
constexpr int kSmallRows = 32, kOwnRows = 16;
cudaError_t launch_small(const Product &p, int split, cudaStream_t s);

}  // namespace mx
}  // namespace bt
