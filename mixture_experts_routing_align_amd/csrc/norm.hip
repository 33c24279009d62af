// RMS norm with the residual's addition, bf16 or 8-bit rows out, and its
// gradient, for gfx950.
//
//   z = x + r (rounded to r's type), rstd = (mean z^2 + eps)^(-1/2), y = z rstd w
//   t = dy w, n = z rstd, dx = dz + rstd (t - n mean(t n)), dw = sum_rows dy n
//
// Both are bound by HBM: a row is read once and stays in registers between the
// sum and its use, so each element moves once.  A row belongs to one wave or to a
// workgroup of 4, 8 or 16 waves, in pieces of 8 columns per lane; with one wave per
// row the sum needs no LDS and no barrier.  Measured (16384 x 2048): 44 us forward,
// 50 us backward plus 5 us for the columns' sums, 6.1 and 4.9 TB/s of the bytes
// that have to move; 8192 x 7168 to 8 bits 80 to 84 us, 4.9 to 5.2 TB/s.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "moe_internal.h"
#include "ops_internal.h"
#include "row_common.h"

namespace moe {
namespace {

using namespace row;

// The sum of the squares of a row that TPR threads hold; `red` holds one float per wave
// of the workgroup, and a barrier separates two uses of it.  A wave per row adds up each
// piece over the wave before it adds the pieces: these are the sums of a wave per piece,
// so a row's bits do not depend on which of the two its batch takes.
template <int TPR, int NV>
__device__ __forceinline__ float square_sum(const float (&z)[NV][8], float* red) {
  if constexpr (TPR == 64) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float p = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) p = fmaf(z[v][i], z[v][i], p);
      s += wave_sum(p);
    }
    return s;
  } else {
    constexpr int W = TPR / 64;
    float p = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) p = fmaf(z[v][i], z[v][i], p);
    p = wave_sum(p);
    const int wave = threadIdx.x >> 6, base = wave / W * W;
    if ((threadIdx.x & 63) == 0) red[wave] = p;
    __syncthreads();
    float s = red[base];
#pragma unroll
    for (int i = 1; i < W; ++i) s += red[base + i];
    return s;
  }
}

constexpr float kLargeMean = 0x1p100f, kSmallMean = 0x1p-100f, kSmallEps = 0x1p-80f;

template <typename RT, bool HAS_R>
__device__ __forceinline__ void load_z(const uint16_t* x, const RT* r, int c, int H, float (&z)[8]) {
  load8(x, c, H, z);
  if constexpr (HAS_R) {
    float a[8];
    load8(r, c, H, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] += a[i];
      // the stored row is the one that is normalised: round to its type here
      if constexpr (sizeof(RT) == 2) z[i] = (float)(__bf16)z[i];
    }
  }
}

// TPR threads per row, NV pieces of 8 columns per thread, THREADS / TPR rows per workgroup.
template <int TPR, int NV, int THREADS, typename RT, bool HAS_R, bool FP8>
__global__ __launch_bounds__(THREADS) void norm_kernel(NormArgs a) {
  __shared__ float red[THREADS / 64];
  const int sub = threadIdx.x / TPR, j = threadIdx.x % TPR;
  const int64_t m = row::block_index() * (THREADS / TPR) + sub;
  if (m - sub >= a.M) return;  // a whole workgroup past the last row
  const bool live = m < a.M;
  const int64_t mm = live ? m : a.M - 1;  // a row past the last repeats it and stores nothing
  const int H = a.H;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + mm * a.ldx;
  const RT* r = static_cast<const RT*>(a.res) + mm * H;
  float z[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) load_z<RT, HAS_R>(x, r, (v * TPR + j) * 8, H, z[v]);
  float w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) load8(static_cast<const uint16_t*>(a.w), (v * TPR + j) * 8, H, w[v]);
  if constexpr (HAS_R) {
    if (live && a.zout != nullptr) {
      RT* zo = static_cast<RT*>(a.zout) + m * H;
#pragma unroll
      for (int v = 0; v < NV; ++v) store8(zo, (v * TPR + j) * 8, H, z[v]);
    }
  }
  float mean = square_sum<TPR>(z, red) / (float)H, eps = a.eps, unit = 1.f, pre = 1.f;
  // Squares that leave float32's range (means past 2^100, or below 2^-100 with next to no
  // eps) are summed once more in a unit that keeps them inside it: 2^-80 (32768 of the
  // largest value make 2^111) or 2^96 (the smallest subnormal's square is 2^-106, and the
  // sum stays below 2^107).  The whole row takes the same way.  y comes from z in a unit
  // `pre` in which neither z nor rstd leaves the range: large rows in 2^-16, which makes a
  // subnormal rstd (below 2^-126) a normal float and costs bits only of values whose y is
  // 0; small rows in 2^96.
  const bool large = mean > kLargeMean, small = mean < kSmallMean && eps < kSmallEps;
  if (large || small) {
    unit = large ? 0x1p-80f : 0x1p96f;
    pre = large ? 0x1p-16f : unit;
    float t[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[v][i] = z[v][i] * unit;
        z[v][i] *= pre;
      }
    if constexpr (TPR > 64) __syncthreads();  // red is read
    mean = square_sum<TPR>(t, red) / (float)H;
    eps = eps * unit * unit;
  }
  const float rs = unit / pre / sqrtf(mean + eps);  // rstd for z in that unit
  if (!live) return;
  if (a.rstd != nullptr && j == 0) a.rstd[m] = rs * pre;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + j) * 8;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = z[v][i] * rs * w[v][i];
    if constexpr (FP8) {
      // 16 neighbouring lanes hold one scale block (H is a multiple of 128, so a
      // block is wholly inside the row or wholly past it)
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = max(mx, abs_bits(y[i]));
      const float scale = block_scale(row16_umax(mx));
      if (c < H) {
        const Codes codes(scale);
        const uint32_t lo = codes.x4(y[0], y[1], y[2], y[3]), hi = codes.x4(y[4], y[5], y[6], y[7]);
        *reinterpret_cast<u32x2_e1*>(static_cast<uint8_t*>(a.out) + m * H + c) = u32x2_e1{lo, hi};
        if ((j & 15) == 0) a.scale[m * (H / kScaleBlock) + c / kScaleBlock] = scale;
      }
    } else {
      store8(static_cast<uint16_t*>(a.out) + m * H, c, H, y);
    }
  }
}

// Each row group of the workgroup walks rows g, g + groups, ..., the next row's
// loads in flight while this one is reduced; the columns' sums of dy n stay in
// registers, the workgroup's groups add theirs in order through LDS, and each
// workgroup leaves one partial row (or, when it is the only one, the result).
// 8 columns a thread (2048 columns: 4 waves a row) measured faster than a wave per
// row with 32, whose column sums leave room for half the waves: 50 against 93 us
// at 16384 x 2048.  Above 16384 columns 1024 threads hold 32 columns each, which their 128
// registers do not: 162 (bf16) and 212 (float32) of them spill, and 2048 x 32768 takes 387
// and 599 us, 1.4 and 1.6 TB/s.  (float32 above 8192 columns spills 9: 4096 x 8448 in 111
// us, 4.4 TB/s.)
template <int TPR, int NV, int THREADS, typename ZT, bool DW>
__global__ __launch_bounds__(THREADS) void norm_backward_kernel(NormBackwardArgs a) {
  constexpr int R = THREADS / TPR, W = TPR / 64;
  // rows that need the workgroup's barrier have it to themselves
  static_assert(TPR == 64 || R == 1, "one row at a time where waves share it");
  __shared__ float red[2][THREADS / 64];
  __shared__ float cols[DW && R > 1 ? TPR * NV * 8 : 1];
  const int sub = threadIdx.x / TPR, j = threadIdx.x % TPR;
  const int H = a.H;
  struct Row {
    Piece<ZT> z[NV], dz[NV];
    Piece<uint16_t> dy[NV];
    float rstd;
  };
  auto load = [&](int64_t m, Row& r) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + j) * 8;
      r.z[v].load(static_cast<const ZT*>(a.z) + m * H, c, H);
      r.dy[v].load(static_cast<const uint16_t*>(a.dy) + m * H, c, H);
      if (a.dz != nullptr) r.dz[v].load(static_cast<const ZT*>(a.dz) + m * H, c, H);
    }
    r.rstd = a.rstd[m];
  };
  Piece<uint16_t> w[NV];
  float acc[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    w[v].load(static_cast<const uint16_t*>(a.w), (v * TPR + j) * 8, H);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[v][i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t m = (int64_t)blockIdx.x * R + sub;
  constexpr bool kAhead = TPR < 1024;  // 1024 threads leave no registers for a second row
  Row r, next;
  if (kAhead && m < a.M) load(m, r);
  for (int parity = 0; m < a.M; m += step, parity ^= 1) {
    if (!kAhead) load(m, r);
    if (kAhead && m + step < a.M) load(m + step, next);
    const float rstd = r.rstd;
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = r.z[v].get(i) * rstd, g = r.dy[v].get(i);
        if (DW) acc[v][i] = fmaf(g, n, acc[v][i]);
        dot = fmaf(g * w[v].get(i), n, dot);
      }
    dot = wave_sum(dot);
    if constexpr (TPR > 64) {
      // two sets of wave sums in turn: one barrier a row
      if ((threadIdx.x & 63) == 0) red[parity][threadIdx.x >> 6] = dot;
      __syncthreads();
      dot = red[parity][0];
#pragma unroll
      for (int i = 1; i < W; ++i) dot += red[parity][i];
    }
    dot /= (float)H;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = rstd * fmaf(-(r.z[v].get(i) * rstd), dot, r.dy[v].get(i) * w[v].get(i));
        if (a.dz != nullptr) o[i] += r.dz[v].get(i);
      }
      store8(static_cast<ZT*>(a.dx) + m * H, (v * TPR + j) * 8, H, o);
    }
    if (kAhead) r = next;
  }
  if constexpr (DW) {
    if constexpr (R > 1) {
      // groups 0, 1, ... add their columns in turn
#pragma unroll 1
      for (int g = 0; g < R; ++g) {
        if (sub == g) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* p = &cols[(v * 8 + i) * TPR + j];
              *p = g == 0 ? acc[v][i] : *p + acc[v][i];
            }
        }
        __syncthreads();
      }
    }
    if (sub == 0) {
      float* out = a.part + (int64_t)blockIdx.x * H;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (R > 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[v][i] = cols[(v * 8 + i) * TPR + j];
        }
        store8(out, (v * TPR + j) * 8, H, acc[v]);
      }
    }
  }
}

// dw[c] = the partial rows' sum: 16 columns a workgroup, 16 threads a column, each
// every 16th partial row in order, the 16 sums joined in a fixed tree.
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* __restrict__ part, int G, int H, float* __restrict__ dw) {
  __shared__ float red[16][17];
  const int cc = threadIdx.x & 15, s = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + cc;
  float v = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int g = s; g < G; g += 16) v += part[(int64_t)g * H + c];
  }
  red[s][cc] = v;
  __syncthreads();
  for (int d = 8; d > 0; d >>= 1) {
    if (s < d) red[s][cc] += red[s + d][cc];
    __syncthreads();
  }
  if (s == 0 && c < H) dw[c] = red[0][cc];
}

__global__ __launch_bounds__(256) void zero_kernel(float* p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

template <int TPR, int NV, int THREADS, typename RT, bool HAS_R>
hipError_t run_norm(const NormArgs& a, hipStream_t s) {
  const dim3 grid = row::grid_of((a.M + THREADS / TPR - 1) / (THREADS / TPR));
  if (a.scale != nullptr)
    hipLaunchKernelGGL((norm_kernel<TPR, NV, THREADS, RT, HAS_R, true>), grid, dim3(THREADS), 0, s, a);
  else
    hipLaunchKernelGGL((norm_kernel<TPR, NV, THREADS, RT, HAS_R, false>), grid, dim3(THREADS), 0, s, a);
  return hipGetLastError();
}

// A row's threads: one wave up to 512 columns, and up to 1024 where there are rows
// enough to fill the GPU with such waves (16384 x 1024: 23 against 26 us); else
// 256 threads (up to 4096 columns), 512 (8192) or 1024.  More threads with fewer
// columns each measured faster for long rows (16384 x 2048: 44 us with 8 columns a
// thread against 52 with a wave per row; 8192 x 7168 to 8 bits: 80 us with 512
// threads against 102 with 256).
constexpr int64_t kWaveRows = 2048;

template <typename RT, bool HAS_R>
hipError_t norm_by_width(const NormArgs& a, hipStream_t s) {
  const int p = (a.H + 7) / 8;
  if (p <= 64) return run_norm<64, 1, 256, RT, HAS_R>(a, s);
  if (p <= 128 && a.M >= kWaveRows) return run_norm<64, 2, 256, RT, HAS_R>(a, s);
  if (p <= 256) return run_norm<256, 1, 256, RT, HAS_R>(a, s);
  if (p <= 512) return run_norm<256, 2, 256, RT, HAS_R>(a, s);
  if (p <= 1024) return run_norm<512, 2, 512, RT, HAS_R>(a, s);
  if (p <= 2048) return run_norm<1024, 2, 1024, RT, HAS_R>(a, s);
  return run_norm<1024, 4, 1024, RT, HAS_R>(a, s);
}

struct BackwardShape {
  int tpr, nv, threads, groups;
};

BackwardShape backward_shape(int64_t M, int H) {
  const int p = (H + 7) / 8;
  BackwardShape b;
  b.tpr = p <= 64 ? 64 : p <= 512 ? 256 : p <= 1024 ? 512 : 1024;
  b.nv = p <= 256 ? 1 : p <= 2048 ? 2 : 4;
  b.threads = std::max(b.tpr, 256);
  const int64_t per = b.threads / b.tpr;
  // about as many workgroups as the GPU holds at once: each leaves one partial row
  b.groups = (int)std::min<int64_t>((M + per - 1) / per, 1024 * 256 / b.threads);
  return b;
}

template <int TPR, int NV, int THREADS, typename ZT>
void run_backward(const NormBackwardArgs& a, int groups, bool dw, hipStream_t s) {
  if (dw)
    hipLaunchKernelGGL((norm_backward_kernel<TPR, NV, THREADS, ZT, true>), dim3(groups), dim3(THREADS), 0, s, a);
  else
    hipLaunchKernelGGL((norm_backward_kernel<TPR, NV, THREADS, ZT, false>), dim3(groups), dim3(THREADS), 0, s, a);
}

template <typename ZT>
void backward_by_width(const NormBackwardArgs& a, const BackwardShape& b, bool dw, hipStream_t s) {
  if (b.tpr == 64) return run_backward<64, 1, 256, ZT>(a, b.groups, dw, s);
  if (b.tpr == 256 && b.nv == 1) return run_backward<256, 1, 256, ZT>(a, b.groups, dw, s);
  if (b.tpr == 256) return run_backward<256, 2, 256, ZT>(a, b.groups, dw, s);
  if (b.tpr == 512) return run_backward<512, 2, 512, ZT>(a, b.groups, dw, s);
  if (b.nv == 2) return run_backward<1024, 2, 1024, ZT>(a, b.groups, dw, s);
  return run_backward<1024, 4, 1024, ZT>(a, b.groups, dw, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool res_f32, hipStream_t s) {
  if (a.res == nullptr) return norm_by_width<uint16_t, false>(a, s);
  return res_f32 ? norm_by_width<float, true>(a, s) : norm_by_width<uint16_t, true>(a, s);
}

size_t norm_backward_workspace(int64_t M, int H) {
  const int g = backward_shape(M, H).groups;
  return g > 1 ? (size_t)g * H * 4 : 0;
}

hipError_t launch_norm_backward(const NormBackwardArgs& args, bool z_f32, float* dw, float* ws, hipStream_t s) {
  NormBackwardArgs a = args;
  if (a.M == 0) {
    if (dw != nullptr) hipLaunchKernelGGL(zero_kernel, dim3((a.H + 255) / 256), dim3(256), 0, s, dw, a.H);
    return hipGetLastError();
  }
  const BackwardShape b = backward_shape(a.M, a.H);
  a.part = b.groups > 1 ? ws : dw;
  if (z_f32)
    backward_by_width<float>(a, b, dw != nullptr, s);
  else
    backward_by_width<uint16_t>(a, b, dw != nullptr, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || dw == nullptr || b.groups == 1) return e;
  hipLaunchKernelGGL(norm_dw_kernel, dim3((a.H + 15) / 16), dim3(256), 0, s, ws, b.groups, a.H, dw);
  return hipGetLastError();
}

}  // namespace moe
