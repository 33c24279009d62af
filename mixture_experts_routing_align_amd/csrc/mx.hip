// Rows of numbers to MXFP4 and back for gfx950.
//
//   quantize:    per block of 32 columns a scale byte and 32 codes (mx_common.h); with
//                positions, token t's codes go to the rows p(t, k) of its slots
//   dequantize:  value = E2M1(code) * 2^(byte - 127)
//
// Both are bound by HBM: a value is read once (2 or 4 bytes) and leaves as half a byte and
// its share of a scale, once per row it goes to.  A lane takes 8 columns, a block is 4
// lanes, whose maximum meets on the DPP crossbar; a row is shared by as many threads as it
// has pieces, up to a workgroup, and a thread's pieces are loaded ahead of their rounding.
//
// Measured (kernels alone): 4096 bf16 rows of 2048 to 32768 sorted rows 14.0 us, 3.7 TB/s;
// 98304 float32 rows of 2048 191 us, 4.8 TB/s (201 million weights), back to bf16 75 us, 6.8
// TB/s; 8 rows to 64 4.0 us, the launch and one trip to memory.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "mx_common.h"
#include "ops_internal.h"
#include "row_common.h"

namespace moe {
namespace {

using namespace row;

constexpr int kThreads = 256;
constexpr int kAhead = 4;   // pieces of a row a thread loads at once
constexpr int kSlots = 8;   // slots of a token handled side by side

// Maximum over each quad of lanes.
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}

// TPT threads a row; H is a multiple of 32, so a quad of lanes is in a row or past it as one.
template <typename T, int TPT, bool PERM>
__global__ __launch_bounds__(kThreads) void quantize_kernel(MxQuantizeArgs a) {
  const int64_t t = block_index() * (kThreads / TPT) + threadIdx.x / TPT;
  if (t >= a.M) return;
  const int j = threadIdx.x % TPT;
  const T* x = static_cast<const T*>(a.x) + t * a.ldx;
  const int64_t row_codes = a.H / 2, row_scales = a.H / mx::kBlock;
  for (int k0 = 0; k0 < (PERM ? a.top_k : 1); k0 += kSlots) {
    int64_t p[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      p[k] = -1;
      if (PERM && k0 + k < a.top_k) {
        const int at = a.perm[t * a.top_k + k0 + k];
        if (at >= 0 && at < a.rows) p[k] = at;
      }
    }
    if (!PERM) p[0] = t;
    for (int c0 = j * 8; c0 < a.H; c0 += kAhead * TPT * 8) {
      Piece<T> piece[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (c0 + i * TPT * 8 < a.H) piece[i].load(x, c0 + i * TPT * 8, a.H);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int c = c0 + i * TPT * 8;
        if (c >= a.H) break;
        float v[8];
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] = piece[i].get(e);
          m = max(m, abs_bits(v[e]));
        }
        const uint32_t byte = mx::scale_byte(quad_umax(m));
        const uint32_t codes = mx::codes8(v, byte);
#pragma unroll
        for (int k = 0; k < (PERM ? kSlots : 1); ++k) {
          if (p[k] < 0) continue;
          *reinterpret_cast<uint32_t*>(a.codes + p[k] * row_codes + c / 2) = codes;
          if (c % mx::kBlock == 0) a.scales[p[k] * row_scales + c / mx::kBlock] = (uint8_t)byte;
        }
      }
    }
  }
}

// 8 codes a thread, kAhead times.
template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(MxDequantizeArgs a) {
  const int64_t at = block_index() * (kThreads * kAhead) + threadIdx.x;
  uint32_t codes[kAhead], byte[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int64_t p = at + i * kThreads;
    if (p < a.pieces) {
      codes[i] = reinterpret_cast<const uint32_t*>(a.codes)[p];
      byte[i] = a.scales[p / 4];
    }
  }
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    const int64_t p = at + i * kThreads;
    if (p >= a.pieces) continue;
    // exact in bf16: the smallest value, 2^-128, is among its subnormals
    const mma::bf16x8 v = mma::fp4x8_to_bf16(codes[i], mx::scale_bits(byte[i]));
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<mma::bf16x8*>(static_cast<uint16_t*>(a.out) + p * 8) = v;
    } else {
      mma::f32x4 lo, hi;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = (float)v[e];
        hi[e] = (float)v[e + 4];
      }
      mma::f32x4* to = reinterpret_cast<mma::f32x4*>(static_cast<float*>(a.out) + p * 8);
      to[0] = lo;
      to[1] = hi;
    }
  }
}

template <typename T, int TPT>
hipError_t quantize_with(const MxQuantizeArgs& a, hipStream_t s) {
  const int64_t blocks = (a.M + kThreads / TPT - 1) / (kThreads / TPT);
  if (a.perm != nullptr)
    hipLaunchKernelGGL((quantize_kernel<T, TPT, true>), grid_of(blocks), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((quantize_kernel<T, TPT, false>), grid_of(blocks), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t quantize(const MxQuantizeArgs& a, hipStream_t s) {
  const int pieces = a.H / 8;
  if (pieces <= 4) return quantize_with<T, 4>(a, s);
  if (pieces <= 16) return quantize_with<T, 16>(a, s);
  if (pieces <= 64 || a.M >= 2048) return quantize_with<T, 64>(a, s);
  return quantize_with<T, 256>(a, s);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantizeArgs& a, bool f32, hipStream_t s) {
  return f32 ? quantize<float>(a, s) : quantize<uint16_t>(a, s);
}

hipError_t launch_mx_dequantize(const MxDequantizeArgs& a, bool f32, hipStream_t s) {
  const dim3 grid = grid_of((a.pieces + kThreads * kAhead - 1) / (kThreads * kAhead));
  if (f32)
    hipLaunchKernelGGL((dequantize_kernel<float>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((dequantize_kernel<uint16_t>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
