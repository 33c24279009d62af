// MXFP4 building blocks for gfx950: the scale of a block of 32 values, E2M1 rounding,
// and the matrix cores' own 4-bit product.
//
// A block's scale byte b stands for 2^(b - 127).  From the block's absolute maximum with
// exponent field f (2^(f - 127) <= maximum < 2^(f - 126)) it is f - 2: 2 is the exponent of
// the largest code, 6 = 1.5 * 2^2, so the maximum over the scale lies in [4, 8) and what
// passes 6 saturates.  Bytes stay in 2 ... 252, where every value is a normal bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mma_common.h"
#include "row_common.h"

namespace moe {
namespace mx {

constexpr int kBlock = 32;        // values that share one scale byte
constexpr int kNanByte = 255;     // E8M0's NaN
constexpr int kZeroByte = 127;    // of a block of zeros: a scale of 1

// Scale byte of a block from the bits of its absolute maximum.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int field = (int)(amax_bits >> 23);
  if (field == 255) return kNanByte;
  if (amax_bits == 0) return kZeroByte;
  return (uint32_t)max(field - 2, 2);
}
// The conversions below read a scale's exponent field alone, as an E8M0 byte: 0 is 2^-127
// and 255 a NaN there (measured for every case).
__device__ __forceinline__ float scale_bits(uint32_t byte) { return __uint_as_float(byte << 23); }

// 4 values over their block's scale as E2M1 codes, to nearest even, saturating; the first
// in the lowest nibble.  Dividing by a power of two is exact, so this is the only rounding.
// A block whose scale is NaN gets zero codes.
__device__ __forceinline__ uint32_t codes4(float v0, float v1, float v2, float v3, uint32_t byte) {
  if (byte == (uint32_t)kNanByte) return 0;
  const float s = scale_bits(byte);
  const uint32_t lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v0, v1, s, 0);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v2, v3, s, 1);
}
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint32_t byte) {
  if (byte == (uint32_t)kNanByte) return 0;
  const float s = scale_bits(byte);
  uint32_t d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0], v[1], s, 0);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[2], v[3], s, 1);
  d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, v[6], v[7], s, 3);
}

// One v_mfma_scale_f32_16x16x128_f8f6f4 on E2M1 codes: lane l feeds row l % 16 of either
// operand with the 32 codes of one block (16 bytes) and that block's scale byte (byte OPA or
// OPB of a dword), and receives D[4 (l / 16) + i][l % 16].  On random codes the result is within
// 6e-8 of the sum of absolute products, with scales 2^20 apart: float32 sums, unlike the
// e4m3 form's.
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int OPA, int OPB>
__device__ __forceinline__ mma::f32x4 mfma(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, mma::f32x4 c) {
  const i32x8 av{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0}, bv{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, OPA, (int)sa, OPB, (int)sb);
}

}  // namespace mx
}  // namespace moe
