// Token rows laid out by expert, brought back with weights applied, and the
// gradient of that, for gfx950.
//
//   permute:   out[p(t, k)] = x[t]
//   unpermute: out[t] = sum_k w[t, k] y[p(t, k)]            (k ascending)
//   backward:  dy[p(t, k)] = w[t, k] dout[t],  dw[t, k] = <dout[t], y[p(t, k)]>
//
// All three are bound by HBM and walk tokens, not sorted rows: a token's own row
// is then read or written once whatever top_k is, each sorted row is touched by
// one wave, and nothing needs an atomic.  Many tokens with short rows: a wave per
// token; else a workgroup of 4 waves, whose loads of a long row run side by side.
// Measured at 2048 columns and top-8: 8-bit rows of 16384 tokens laid out in 50 us
// (5.7 TB/s of what has to move), rows of 8192 tokens back in 53 us (5.7 TB/s), the
// gradient in 120 us (4.7 TB/s).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ops_internal.h"
#include "row_common.h"

namespace moe {
namespace {

using namespace row;

constexpr int kThreads = 256;
constexpr int kBatch = 8;          // slots of a token handled side by side
constexpr int64_t kWaveTokens = 2048;  // from here on a wave per token
constexpr int64_t kCacheBytes = 192 << 20;  // rows past this do not stay in the 256 MB memory-side cache

// A row of `bytes` moves 16 bytes per lane at any 2-byte alignment; the last
// piece may be shorter (an even number of bytes).
__device__ __forceinline__ uint4 load_piece(const uint8_t* p, int c, int bytes) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (c + 16 <= bytes) {
    const u32x4_e2 d = *reinterpret_cast<const u32x4_e2*>(p + c);
    v = make_uint4(d[0], d[1], d[2], d[3]);
  } else {
    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 2 * i < bytes) d[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + c + 2 * i) << (16 * (i & 1));
    v = make_uint4(d[0], d[1], d[2], d[3]);
  }
  return v;
}
// PAST_CACHE: not kept in the caches.
template <bool PAST_CACHE>
__device__ __forceinline__ void store_piece(uint8_t* p, int c, int bytes, uint4 v) {
  if (c + 16 <= bytes) {
    const u32x4_e2 q{v.x, v.y, v.z, v.w};
    if constexpr (PAST_CACHE)
      __builtin_nontemporal_store(q, reinterpret_cast<u32x4_e2*>(p + c));
    else
      *reinterpret_cast<u32x4_e2*>(p + c) = q;
  } else {
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 2 * i < bytes) *reinterpret_cast<uint16_t*>(p + c + 2 * i) = (uint16_t)(d[i / 2] >> (16 * (i & 1)));
  }
}

// The position of slot i, or -1 where it has none (a value outside [0, rows) is
// never followed).
__device__ __forceinline__ int position(const int32_t* perm, int64_t i, int64_t rows) {
  const int p = perm[i];
  return p >= 0 && p < rows ? p : -1;
}

// TPT threads a token (64 or 256).
template <int TPT, bool PAST_CACHE>
__global__ __launch_bounds__(kThreads) void permute_kernel(PermuteArgs a) {
  const int64_t t = row::block_index() * (kThreads / TPT) + threadIdx.x / TPT;
  if (t >= a.M) return;
  const int j = threadIdx.x % TPT;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.row_bytes;
  uint8_t* out = static_cast<uint8_t*>(a.out);
  for (int k0 = 0; k0 < a.top_k; k0 += kBatch) {
    const int kn = min(kBatch, a.top_k - k0);
    int p[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) p[k] = k < kn ? position(a.perm, t * a.top_k + k0 + k, a.rows) : -1;
    for (int c = j * 16; c < a.row_bytes; c += TPT * 16) {
      const uint4 v = load_piece(x, c, a.row_bytes);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (p[k] >= 0) store_piece<PAST_CACHE>(out + (int64_t)p[k] * a.row_bytes, c, a.row_bytes, v);
    }
    if (a.scales) {
      for (int c = j; c < a.scales; c += TPT) {
        const float v = a.x_scale[t * a.scales + c];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (p[k] >= 0) a.out_scale[(int64_t)p[k] * a.scales + c] = v;
      }
    }
  }
}

template <int TPT, bool WEIGHTED>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(UnpermuteArgs a) {
  const int64_t t = row::block_index() * (kThreads / TPT) + threadIdx.x / TPT;
  if (t >= a.M) return;
  const int j = threadIdx.x % TPT;
  const int H = a.H;
  for (int c = j * 8; c < H; c += TPT * 8) {
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < a.top_k; k0 += kBatch) {
      const int kn = min(kBatch, a.top_k - k0);
      int p[kBatch];
      float w[kBatch];
      Piece<uint16_t> v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        p[k] = k < kn ? position(a.perm, t * a.top_k + k0 + k, a.rows) : -1;
        w[k] = WEIGHTED && k < kn ? a.w[t * a.top_k + k0 + k] : 1.f;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (p[k] >= 0) v[k].load(a.y + (int64_t)p[k] * H, c, H);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (p[k] >= 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = WEIGHTED ? fmaf(w[k], v[k].get(i), o[i]) : o[i] + v[k].get(i);
        }
    }
    store8(a.out + t * H, c, H, o);
  }
}

template <int TPT>
__global__ __launch_bounds__(kThreads) void unpermute_backward_kernel(UnpermuteBackwardArgs a) {
  __shared__ float red[kBatch][kThreads / 64];
  const int64_t t = row::block_index() * (kThreads / TPT) + threadIdx.x / TPT;
  if (t >= a.M) return;  // whole waves, and with TPT == 256 no workgroup has one
  const int j = threadIdx.x % TPT, lane = threadIdx.x & 63;
  const int H = a.H;
  for (int k0 = 0; k0 < a.top_k; k0 += kBatch) {
    const int kn = min(kBatch, a.top_k - k0);
    int p[kBatch];
    float w[kBatch], dot[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      p[k] = k < kn ? position(a.perm, t * a.top_k + k0 + k, a.rows) : -1;
      w[k] = k < kn ? a.w[t * a.top_k + k0 + k] : 0.f;
      dot[k] = 0.f;
    }
    for (int c = j * 8; c < H; c += TPT * 8) {
      float d[8];
      Piece<uint16_t> v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (p[k] >= 0) v[k].load(a.y + (int64_t)p[k] * H, c, H);
      load8(a.dout + t * H, c, H, d);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (p[k] >= 0) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[k] = fmaf(d[i], v[k].get(i), dot[k]);
            o[i] = w[k] * d[i];
          }
          store8(a.dy + (int64_t)p[k] * H, c, H, o);
        }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) dot[k] = wave_sum(dot[k]);
    if constexpr (TPT == 64) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (lane == 0 && k < kn) a.dw[t * a.top_k + k0 + k] = dot[k];
    } else {
      __syncthreads();  // the last batch's sums are read
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (lane == 0) red[k][threadIdx.x >> 6] = dot[k];
      __syncthreads();
      if ((int)threadIdx.x < kn) {
        float s = red[threadIdx.x][0];
        for (int i = 1; i < kThreads / 64; ++i) s += red[threadIdx.x][i];
        a.dw[t * a.top_k + k0 + threadIdx.x] = s;
      }
    }
  }
}

// Back to token order: a wave per token where there are many and its row keeps no more
// than half a workgroup busy (8192 tokens x 2048, top-8: 53 us with a workgroup, 66
// with a wave, the gradient 124 and 140; 16384 x 1024, top-4: 30 and 27, 85 and 55).
bool wave_per_token(int64_t M, int H) { return M >= kWaveTokens && H <= 1024; }

dim3 grid_for(int64_t M, int per) { return row::grid_of((M + per - 1) / per); }

}  // namespace

hipError_t launch_permute(const PermuteArgs& a, hipStream_t s) {
  // Rows that the caches cannot keep for their reader go past them (277 MB of 8-bit
  // rows: 50 against 64 us).
  const bool past = a.rows * a.row_bytes > kCacheBytes;
  if (a.M < kWaveTokens)
    hipLaunchKernelGGL((permute_kernel<256, false>), grid_for(a.M, 1), dim3(kThreads), 0, s, a);
  else if (past)
    hipLaunchKernelGGL((permute_kernel<64, true>), grid_for(a.M, 4), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((permute_kernel<64, false>), grid_for(a.M, 4), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_unpermute(const UnpermuteArgs& a, hipStream_t s) {
  const bool wave = wave_per_token(a.M, a.H);
  const dim3 grid = grid_for(a.M, wave ? 4 : 1), block(kThreads);
  if (a.w != nullptr) {
    if (wave)
      hipLaunchKernelGGL((unpermute_kernel<64, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((unpermute_kernel<256, true>), grid, block, 0, s, a);
  } else {
    if (wave)
      hipLaunchKernelGGL((unpermute_kernel<64, false>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((unpermute_kernel<256, false>), grid, block, 0, s, a);
  }
  return hipGetLastError();
}

hipError_t launch_unpermute_backward(const UnpermuteBackwardArgs& a, hipStream_t s) {
  if (wave_per_token(a.M, a.H))
    hipLaunchKernelGGL((unpermute_backward_kernel<64>), grid_for(a.M, 4), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((unpermute_backward_kernel<256>), grid_for(a.M, 1), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
