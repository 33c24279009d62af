// Row building blocks shared by the gfx950 kernels that stream token rows
// (norm, permutation, epilogues): 8-element pieces of bf16 or float32 rows at any
// element alignment, wave sums on the DPP crossbar, e4m3 rounding.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mma_common.h"

namespace moe {
namespace row {

constexpr int kScaleBlock = 128;             // columns that share one scale of an 8-bit row
constexpr float kE4m3Max = 448.0f;           // largest e4m3fn value
constexpr float kMinScale = 0x1p-126f;       // smallest normal float: a scale never underflows

// A dispatch holds fewer than 2^32 threads in a dimension: past 2^21 workgroups (of up
// to 1024 threads) they go on in a second one.  The last of those may lie past the end.
constexpr int kGridShift = 21;
inline dim3 grid_of(int64_t blocks) {
  const int64_t most = (int64_t)1 << kGridShift;
  return blocks <= most ? dim3((unsigned)blocks) : dim3((unsigned)most, (unsigned)((blocks + most - 1) >> kGridShift));
}
__device__ __forceinline__ int64_t block_index() { return ((int64_t)blockIdx.y << kGridShift) + blockIdx.x; }

// Vectors the compiler may only assume element-aligned: gfx950 serves them with
// full-width loads and stores at any element alignment, so rows of odd length
// need no other path; a 16-byte aligned address costs nothing extra.
typedef uint32_t u32x4_e2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_e4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_e1 __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// float32 pair -> packed bf16, round to nearest even (the hardware conversion; NaN stays NaN)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 v{(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// 8 consecutive elements from column c of a row of H, zero past its end.
__device__ __forceinline__ void load8(const uint16_t* __restrict__ p, int c, int H, float (&v)[8]) {
  if (c + 8 <= H) {
    const u32x4_e2 d = *reinterpret_cast<const u32x4_e2*>(p + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(d[i]);
      v[2 * i + 1] = bf16_hi(d[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < H ? mma::bf16_bits_to_f32(p[c + i]) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* __restrict__ p, int c, int H, float (&v)[8]) {
  if (c + 8 <= H) {
    const u32x4_e4 a = *reinterpret_cast<const u32x4_e4*>(p + c);
    const u32x4_e4 b = *reinterpret_cast<const u32x4_e4*>(p + c + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < H ? p[c + i] : 0.f;
  }
}

__device__ __forceinline__ void store8(uint16_t* __restrict__ p, int c, int H, const float (&v)[8]) {
  uint32_t d[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  if (c + 8 <= H) {
    *reinterpret_cast<u32x4_e2*>(p + c) = u32x4_e2{d[0], d[1], d[2], d[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) p[c + i] = (uint16_t)(d[i / 2] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* __restrict__ p, int c, int H, const float (&v)[8]) {
  if (c + 8 <= H) {
    u32x4_e4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __float_as_uint(v[i]);
      b[i] = __float_as_uint(v[4 + i]);
    }
    *reinterpret_cast<u32x4_e4*>(p + c) = a;
    *reinterpret_cast<u32x4_e4*>(p + c + 4) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < H) p[c + i] = v[i];
  }
}

// 8 consecutive elements as they lie in memory: half the registers of their float32
// values for bf16, so that a wave can hold several rows.
template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
  uint32_t d[4];
  __device__ __forceinline__ void load(const uint16_t* __restrict__ p, int c, int H) {
    if (c + 8 <= H) {
      const u32x4_e2 v = *reinterpret_cast<const u32x4_e2*>(p + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        d[i] = (c + 2 * i < H ? p[c + 2 * i] : 0u) | (c + 2 * i + 1 < H ? (uint32_t)p[c + 2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(d[i / 2]) : bf16_lo(d[i / 2]); }
};
template <>
struct Piece<float> {
  float d[8];
  __device__ __forceinline__ void load(const float* __restrict__ p, int c, int H) { load8(p, c, H, d); }
  __device__ __forceinline__ float get(int i) const { return d[i]; }
};

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp0(float v) {  // lanes without a source read 0
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROW_MASK, 0xF, false));
}

// Sum over each 16-lane row, in every lane of it (butterflies on the DPP crossbar).
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp0<0xB1, 0xF>(v);   // quad_perm [1,0,3,2]
  v += dpp0<0x4E, 0xF>(v);   // quad_perm [2,3,0,1]
  v += dpp0<0x141, 0xF>(v);  // row_half_mirror
  v += dpp0<0x140, 0xF>(v);  // row_mirror
  return v;
}
// The wave's sum, the same bits in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  v += dpp0<0x142, 0xA>(v);  // row_bcast15 into rows 1 and 3
  v += dpp0<0x143, 0xC>(v);  // row_bcast31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Maximum of |v|'s bits over each 16-lane row: as integers NaN > inf > finite, so
// a NaN or an infinity wins.
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  return v;
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale of a block from the bits of its absolute maximum.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (amax_bits == 0) return 1.f;
  return fmaxf(__uint_as_float(amax_bits) / kE4m3Max, kMinScale);
}

// Values over their block's scale s as e4m3fn codes, as if each quotient x = v / s were
// rounded to float32 and that to its code, to nearest even both times.  Rows of few bits
// put many quotients on the border between two codes (products of two bf16 values: 1 in
// 2000), where v times the rounded 1 / s picks the other code now and then, and a division
// for each value costs a quarter of the norm's time (16384 x 2048: 29 against 23 us).  So
// the product q0 is corrected once by its remainder: q = q0 - (q0 s - v) / s, the remainder
// exact in a fused multiply-add.  q can differ from x rounded only where x lies between
// two floats so near to their middle that the relative error of the rounded 1 / s, at most
// 2^-25 m (m the significand of s, in [1, 2)), times |q0 - x| crosses it.  Beside the border
// of two codes q0 is off by less than 1/2 + m 31/32 / 2 < 1.5 steps of float32, so it is one
// of the two floats, |q0 - x| is half a step and the error 2^-26 m of a step; but integers
// v and s of 24 bits leave x at least 2^-24 / m of a step from the middle, which is more.
// (2^-10, the one border that is a power of two, has the same code as all below it.)
struct Codes {
  static constexpr float kTiny = 0x1p-60f;  // below it remainders would be subnormal
  float s, inv, unit;
  __device__ __forceinline__ explicit Codes(float scale) {
    unit = scale < kTiny ? 0x1p64f : 1.f;
    s = scale * unit;
    inv = 1.0f / s;
  }
  // a NaN scale makes every code NaN; |x| is at most 448 (1 + 2^-23), which rounds to 448
  __device__ __forceinline__ float over(float v) const {
    const float q0 = v * inv;
    return fmaf(-fmaf(q0, s, -v), inv, q0);  // a zero keeps its sign
  }
  __device__ __forceinline__ uint32_t x4(float v0, float v1, float v2, float v3) const {
    if (unit != 1.f) {
      v0 *= unit;
      v1 *= unit;
      v2 *= unit;
      v3 *= unit;
    }
    const uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(over(v0), over(v1), 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(over(v2), over(v3), lo, true);
  }
};

}  // namespace row
}  // namespace moe
