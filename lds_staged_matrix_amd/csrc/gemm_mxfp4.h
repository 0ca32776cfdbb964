// gemm_mxfp4.h -- MXFP4 numbers on gfx950: E2M1 elements, two a byte, even k in
// the low half, and one E8M0 scale for every 32 consecutive k of a row.
//
// The scales of a matrix of M rows stand as rows of M bytes, one for each block
// of 32 k: S[(k / 32) * lds + m].  A tile of a product then finds the scales of
// its rows side by side, in whole 16-byte pieces, where the other order (K / 32
// bytes a row of the matrix) would give it 8 bytes here and there for every
// 256 k.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"

namespace lsm {

constexpr int kMxBlock = 32;             // k that share a scale
constexpr int kMxNaN = 255;              // E8M0's NaN

// Element types of the conversions and of a product's output, values of enum
// gemm_mxfp4_dtype (the OUT_ enumerators in another order).
constexpr int mxfp4_out(int dtype) { return dtype == 0 ? OUT_BF16 : dtype == 1 ? OUT_F16 : OUT_F32; }

// 16 x 16 x 128 of FP4 operands, whose 16 bytes a lane are 32 consecutive k of
// row (column) l & 15: one block, with byte OA (OB) of `sa` (`sb`) for its
// scale.  Each group of lanes l >> 4 holds a block of its own, so that the order
// of k across the groups only has to be the same for both operands.
// The instruction's sums keep fp32's bits: over 6e7 sums of random and sparse
// operands, scales that spread over up to 2^60 and running sums from 2^-30 to 2^30
// times as large it was off by 5.4 * 2^-24 of the sum of sizes at most, unlike
// the fp8 forms (see e4m3_part_as_bf16): products of one block span eight bits.
template <int OA, int OB>
__device__ __forceinline__ v4f32 mfma_mxfp4(v8i16 a, v8i16 b, v4f32 c, int sa, int sb) {
  const auto x = __builtin_bit_cast(u32x4, a), y = __builtin_bit_cast(u32x4, b);
  const v8i32 wa = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
  const v8i32 wb = {(int)y[0], (int)y[1], (int)y[2], (int)y[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, 4, 4, OA, sa, OB, sb);
}

}  // namespace lsm
