// Pieces that the tiled expert products for gfx950 share besides their tiles: the
// activations, a lane's four output columns (bias, activation, residual), and how a
// tile's rows are dealt to its waves.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_mi355x_ops.h"
#include "ops_internal.h"
#include "row_common.h"

namespace moe {
namespace epilogue {

using row::pack_bf16;

// 1 / (1 + exp(-x)) on the hardware's exponential and reciprocal: -x log2(e) as a
// rounded product and its remainder, so that far arguments keep their relative
// precision (a few 2^-24 in all; expf and a division take four times as long, 45 of
// 325 us in the gate+up product's epilogue).
__device__ __forceinline__ float sigmoid(float x) {
  const float t = x * -1.44269504f, rest = fmaf(x, -1.44269504f, -t) + x * -1.92596303e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  return __builtin_amdgcn_rcpf(1.0f + fmaf(e, rest * 0.69314718f, e));
}
// The same for any x: past 87 on either side (and at the infinities) the correction
// would meet an infinity, and float32's normal range has only 0 and 1 there.
__device__ __forceinline__ float sigmoid_all(float x) { return x > 87.0f ? 1.0f : x < -87.0f ? 0.0f : sigmoid(x); }
// the tanh form of gelu: z/2 (1 + tanh(a)) = z sigmoid(2 a), a = sqrt(2/pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu_2a(float z) { return 1.5957691216057308f * fmaf(0.044715f * z * z, z, z); }

__device__ __forceinline__ void unpack4(uint2 v, float (&f)[4]) {
  f[0] = row::bf16_lo(v.x);
  f[1] = row::bf16_hi(v.x);
  f[2] = row::bf16_lo(v.y);
  f[3] = row::bf16_hi(v.y);
}
__device__ __forceinline__ uint2 pack4(const float (&f)[4]) { return make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])); }

// 1 / (1 + exp(-x)) without the remainder of x log2(e), whose rounding costs |x| 2^-24 of the
// result where the exponential dominates (|x| is at most 89 there: 2^-17): for epilogues that
// round to 8 significant bits (bf16) or fewer and are bound by their arithmetic.  The infinities need no care: the exponential is 0 or an
// infinity there, as it is past 89.
__device__ __forceinline__ float sigmoid_short(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// act(z[, u]) of 4 elements.
template <bool GATED, bool SHORT = false>
__device__ __forceinline__ void act4(int act, const float (&z)[4], const float (&u)[4], float (&y)[4]) {
  auto gate = [](float x) { return SHORT ? sigmoid_short(x) : sigmoid_all(x); };
  if constexpr (GATED) {
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = z[c] * gate(z[c]) * u[c];
  } else {
    if (act == MOE_ACT_SILU) {
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] = z[c] * gate(z[c]);
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] = z[c] * gate(gelu_2a(z[c]));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) y[c] = z[c];
    }
  }
}

// v += 4 packed bf16 values.
__device__ __forceinline__ void add4(float (&v)[4], uint2 packed) {
  float f[4];
  unpack4(packed, f);
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] += f[c];
}

// 4 consecutive columns n ... n + 3 of row r of expert e: bias, activation and
// residual on float32 sums; z and u come back as the pre-activations.  `in`: the
// columns and the row exist.
template <bool GATED>
__device__ __forceinline__ void epilogue4(const LinearArgs& a, int e, int64_t r, int n, bool in, float (&z)[4], float (&u)[4],
                                          float (&y)[4]) {
  if (a.bias[0] != nullptr && in) add4(z, *reinterpret_cast<const uint2*>(a.bias[0] + (int64_t)e * a.N + n));
  if constexpr (GATED)
    if (a.bias[1] != nullptr && in) add4(u, *reinterpret_cast<const uint2*>(a.bias[1] + (int64_t)e * a.N + n));
  act4<GATED>(a.act, z, u, y);
  if (a.residual != nullptr && in) add4(y, *reinterpret_cast<const uint2*>(a.residual + r * a.N + n));
}

// Calls f with the smallest of kQ / 4, kQ / 2, 3 kQ / 4 and kQ subtiles that covers `live`.
template <int N>
struct Count {
  static constexpr int value = N;
};
template <int kQ, typename F>
__device__ __forceinline__ void by_live_subtiles(int live, F f) {
  if constexpr (kQ >= 4) {
    if (live <= kQ / 4) return f(Count<kQ / 4>{});
    if (live <= kQ / 2) return f(Count<kQ / 2>{});
    if (live <= kQ * 3 / 4) return f(Count<kQ * 3 / 4>{});
  }
  f(Count<kQ>{});
}

// Rows of a tile are dealt to the WQ rows of waves in subtiles of 16 in turn, so a
// partly filled tile leaves every wave the same share (at most one subtile apart);
// a wave multiplies only its LIVE first subtiles.
template <int WQ>
__device__ __forceinline__ int q_row(int wq, int i) { return (i * WQ + wq) * 16; }

}  // namespace epilogue
}  // namespace moe
