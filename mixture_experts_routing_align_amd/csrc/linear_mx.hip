// The experts' matrix products on MXFP4 weights over sorted rows for gfx950: forward with
// bias, activation, residual and MXFP4 rows in the epilogue, and the rows' gradient.
//
//   forward      z[p] = W[e] x[p] + b[e], y[p] = act(z[p]) + residual[p]
//   backward x   dx[p] = sum_n dz[p, n] W[e][n, :]
//
// A weight is its E2M1 code times its block's scale.  With MXFP4 rows the products are the
// matrix cores' own 4-bit ones (mx_common.h); with bf16 rows the codes are widened to bf16
// with their scale, which is exact, so sums are float32 either way.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "linear_epilogue.h"
#include "linear_tile.h"
#include "moe_internal.h"
#include "moe_mi355x_ops.h"
#include "mx_common.h"
#include "row_common.h"

namespace moe {
namespace {

using namespace tile;
using namespace epilogue;

extern __shared__ __attribute__((aligned(1024))) char smem[];

// --------------------------------------------------- forward, few rows --

// Few rows per expert: the weights are read once and nothing is reused enough to stage it,
// so a workgroup takes 16 rows by 16 WC columns, and WK waves split the depth of each 16
// columns in interleaved 256-deep chunks, both operands loaded straight into the matrix
// cores' registers (16 lanes x 128 contiguous bytes of weights a chunk).  Lane l takes
// blocks 2 (l / 16) and 2 (l / 16) + 1 of a chunk; blocks past the depth are zeros.  The WK
// sums meet in LDS in wave order.  MXFP4 rows out need both halves of a block of 32
// columns: WC even.
template <bool ROWS4, bool GATED, int WC, int WK>
__global__ __launch_bounds__(WC* WK * 64) void linear_mx_few_kernel(MxLinearArgs a) {
  constexpr int kParts = GATED ? 2 : 1, kCols = 16 * WC, kBlocks = 8;  // scale blocks of a chunk
  __shared__ f32x4 part[WC][WK][kParts][64];
  __shared__ uint32_t red[WC][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wc = wave % WC, wk = wave / WC, quad = lane >> 4;
  const Item it = find_item(a, row::block_index(), 16, (a.N + kCols - 1) / kCols);
  if (it.e < 0) return;
  const int live = min(16, it.count - it.tq * 16);
  const int64_t first = (int64_t)it.row0 + it.tq * 16;
  const int col0 = it.tp * kCols + wc * 16;
  const int S = a.K / mx::kBlock;
  // rows and columns past the end repeat the last one and are not stored
  const int64_t xr = first + min(lane & 15, live - 1);
  const int64_t wr = (int64_t)it.e * a.N + min(col0 + (lane & 15), a.N - 1);
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + xr * (ROWS4 ? a.K / 2 : a.K * 2);
  const uint8_t* sx = ROWS4 ? a.xs + xr * S : nullptr;
  const uint8_t *w[kParts], *sw[kParts];
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    w[h] = static_cast<const uint8_t*>(a.w[h]) + wr * (a.K / 2);
    sw[h] = a.wsb[h] + wr * S;
  }
  f32x4 acc[kParts];
#pragma unroll
  for (int h = 0; h < kParts; ++h) acc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c = wk; c * kBlocks < S; c += WK) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = c * kBlocks + quad * 2 + i;
      const bool in = b < S;
      const int at = in ? b : 0;
      uint4 wv[kParts];
      uint32_t wb[kParts];
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        wv[h] = *reinterpret_cast<const uint4*>(w[h] + at * 16);
        wb[h] = sw[h][at];
        if (!in) {
          wv[h] = make_uint4(0, 0, 0, 0);
          wb[h] = mx::kZeroByte;
        }
      }
      if constexpr (ROWS4) {
        uint4 xv = *reinterpret_cast<const uint4*>(x + at * 16);
        uint32_t xb = sx[at];
        if (!in) {
          xv = make_uint4(0, 0, 0, 0);
          xb = mx::kZeroByte;
        }
#pragma unroll
        for (int h = 0; h < kParts; ++h) acc[h] = mx::mfma<0>(wv[h], wb[h], xv, xb, acc[h]);
      } else {
        uint4 xv[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          xv[d] = *reinterpret_cast<const uint4*>(x + at * 64 + d * 16);
          if (!in) xv[d] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          const float f = mx::scale_bits(wb[h]);
          const uint32_t d[4] = {wv[h].x, wv[h].y, wv[h].z, wv[h].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[h] = mma::mfma(mma::fp4x8_to_bf16(d[k], f), mma::as_bf16x8(xv[k]), acc[h]);
        }
      }
    }
  }
#pragma unroll
  for (int h = 0; h < kParts; ++h) part[wc][wk][h][lane] = acc[h];
  __syncthreads();
  const int m = lane & 15, n = col0 + quad * 4;
  const bool in = m < live && n < a.N;
  float y[4] = {0.f, 0.f, 0.f, 0.f};
  if (wk == 0) {
    float z[4], u[4];
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      f32x4 s = part[wc][0][h][lane];
#pragma unroll
      for (int k = 1; k < WK; ++k) s += part[wc][k][h][lane];
#pragma unroll
      for (int c = 0; c < 4; ++c) (h == 0 ? z[c] : u[c]) = s[c];
    }
    epilogue4<GATED>(a, it.e, first + m, n, in, z, u, y);
    if (a.preact != nullptr && in) {
      uint16_t* pre = a.preact + (first + m) * kParts * a.N + n;
      *reinterpret_cast<uint2*>(pre) = pack4(z);
      if (GATED) *reinterpret_cast<uint2*>(pre + a.N) = pack4(u);
    }
    if (a.ysb == nullptr && in) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + (first + m) * a.N + n) = pack4(y);
  }
  if constexpr (WC % 2 == 0) {
    if (a.ysb == nullptr) return;
    if (wk == 0) {
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) mx = max(mx, row::abs_bits(y[c]));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
      if (lane < 16) red[wc][lane] = mx;
    }
    __syncthreads();
    if (wk == 0 && in) {
      const uint32_t byte = mx::scale_byte(max(red[wc & ~1][m], red[wc | 1][m]));
      *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(a.y) + ((first + m) * a.N + n) / 2) =
          (uint16_t)mx::codes4(y[0], y[1], y[2], y[3], byte);
      if (n % mx::kBlock == 0) a.ysb[(first + m) * (a.N / mx::kBlock) + n / mx::kBlock] = (uint8_t)byte;
    }
  }
}

// ------------------------------------------------------------- backward x --

// One workgroup: BQ rows by BP columns of dx; the depth is the weight rows, gate's then
// up's.  A thread takes the 16 bytes of one block of 32 columns of one weight row, a step
// ahead in registers, and leaves it in LDS as bf16 lines, from where it is transposed on
// its way to the matrix cores as bf16 weights are.
template <int BQ, int BP, int WQ, int WP>
__global__ __launch_bounds__(WQ* WP * 64, 2) void linear_mx_backward_x_kernel(MxLinearArgs a) {
  constexpr int kWaves = WQ * WP, kQ = BQ / WQ / 16, kP = BP / WP / 16, kD = 64;
  constexpr int kPer = kD * BP / mx::kBlock / (kWaves * 64);  // blocks of a stage a thread widens
  static_assert(kPer >= 1 && kD * BP / mx::kBlock % (kWaves * 64) == 0, "whole blocks per thread");
  using QTile = RowTile<BQ, kWaves>;
  using PTile = DepthTile<BP, kD, kWaves>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wq = wave / WP, wp = wave % WP;
  const Item it = find_item(a, row::block_index(), BQ, (a.K + BP - 1) / BP);
  if (it.e < 0) return;
  const int q0 = it.tq * BQ, p0 = it.tp * BP;
  const int live = min(BQ, it.count - q0);
  const int64_t first = (int64_t)it.row0 + q0;
  const int ldq = a.parts * a.N * 2, S = a.K / mx::kBlock;
  QTile qt;
  qt.init(wave, lane, [&](int r) { return r < live ? (uint32_t)(r * ldq) : kNoFetch; });
  // the depth runs over the N columns of dz's first part, then of its second
  const int per = (a.N + kD - 1) / kD, steps = per * a.parts;
  const __amdgpu_buffer_rsrc_t rq = resource(static_cast<const char*>(a.dz) + first * ldq);
  // past the last step nothing is left: the loads are issued and fetch nothing
  auto issue_q = [&](int s) {
    const int h = s >= per ? 1 : 0, k = s - h * per;
    qt.load(rq, smem + (s % 3) * QTile::kBytes, wave, (h * a.N + k * kD) * 2, s < steps ? (a.N - k * kD) * 2 : 0);
  };
  char* const weights = smem + 3 * QTile::kBytes;
  // this thread's blocks: line d of the stage, block g of its BP / 32
  constexpr int kLineBlocks = BP / mx::kBlock;
  uint4 codes[kPer];
  uint32_t byte[kPer];
  auto fetch = [&](int s) {
    const int h = s >= per ? 1 : 0, k = s - h * per;
    const uint8_t* w = static_cast<const uint8_t*>(a.w[h]);
    const uint8_t* ws = a.wsb[h];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = i * kWaves * 64 + (int)threadIdx.x, d = at / kLineBlocks, g = at % kLineBlocks;
      const int n = k * kD + d, b = p0 / mx::kBlock + g;
      codes[i] = make_uint4(0, 0, 0, 0);
      byte[i] = mx::kZeroByte;
      if (s < steps && n < a.N && b < S) {
        const int64_t r = (int64_t)it.e * a.N + n;
        codes[i] = *reinterpret_cast<const uint4*>(w + r * (a.K / 2) + b * 16);
        byte[i] = ws[r * S + b];
      }
    }
  };
  auto widen = [&](int stage) {
    char* base = weights + stage * PTile::kBytes;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = i * kWaves * 64 + (int)threadIdx.x, d = at / kLineBlocks, g = at % kLineBlocks;
      const float f = mx::scale_bits(byte[i]);
      const uint32_t c[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<bf16x8*>(base + d * PTile::kLine + (((2 * g + k / 2) ^ PTile::swz(d)) * 32) + (k & 1) * 16) =
            mma::fp4x8_to_bf16(c[k], f);
    }
  };
  f32x4 acc[kQ][kP];
#pragma unroll
  for (int i = 0; i < kQ; ++i)
#pragma unroll
    for (int j = 0; j < kP; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  fetch(0);
  issue_q(0);
  widen(0);
  fetch(1);
  issue_q(1);
  auto multiply = [&](auto live_subtiles) {
    constexpr int L = decltype(live_subtiles)::value;
    for (int s = 0; s < steps; ++s) {
      wait_and_meet<0>();
      widen((s + 1) & 1);  // the other stage, whose readers have passed the barrier
      fetch(s + 2);
      issue_q(s + 2);
      const char* b = smem + (s % 3) * QTile::kBytes;
      const char* w = weights + (s & 1) * PTile::kBytes;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        bf16x8 q[L], p[kP];
#pragma unroll
        for (int i = 0; i < L; ++i) q[i] = QTile::frag(b, q_row<WQ>(wq, i), kk, lane);
#pragma unroll
        for (int j = 0; j < kP; ++j) p[j] = PTile::frag(w, wp * (BP / WP) + j * 16, kk, lane);
#pragma unroll
        for (int j = 0; j < kP; ++j)
#pragma unroll
          for (int i = 0; i < L; ++i) acc[i][j] = mma::mfma(p[j], q[i], acc[i][j]);
      }
    }
  };
  by_live_subtiles<kQ>((live - wq * 16 + 16 * WQ - 1) / (16 * WQ), multiply);
  wait_and_meet<0>();
  using Rows = OutTile<BQ, BP * 2, kWaves * 64>;
  static_assert(BQ * BP * 2 <= 3 * QTile::kBytes + 2 * PTile::kBytes, "the output tile fits where the stages were");
#pragma unroll
  for (int i = 0; i < kQ; ++i)
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      Rows::put(smem, q_row<WQ>(wq, i) + (lane & 15), (wp * (BP / WP) + j * 16 + (lane >> 4) * 4) * 2, pack4(v));
    }
  __syncthreads();
  Rows::flush(smem, reinterpret_cast<char*>(static_cast<uint16_t*>(a.y) + first * a.K + p0), (int64_t)a.K * 2, live,
              min(BP, a.K - p0) * 2);
}

// ---------------------------------------------------------------- launch --

// Instantiated by name: the host pass of this compiler otherwise leaves out the
// launch stubs of some kernel templates that are only reached through pointers.
#define MOE_MX_TILES(R, G)                                          \
  template __global__ void linear_mx_few_kernel<R, G, 2, 8>(MxLinearArgs);
MOE_MX_TILES(false, false)
MOE_MX_TILES(false, true)
MOE_MX_TILES(true, false)
MOE_MX_TILES(true, true)
#undef MOE_MX_TILES
template __global__ void linear_mx_backward_x_kernel<128, 128, 2, 2>(MxLinearArgs);

template <typename K>
hipError_t launch(K kern, int64_t items, int threads, int lds, const MxLinearArgs& a, hipStream_t s,
                  std::atomic<size_t> (&allowed)[kMaxCachedDevices]) {
  const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(kern), lds, allowed);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, row::grid_of((items + 7) / 8 * 8), dim3(threads), lds, s, a);
  return hipGetLastError();
}

template <bool ROWS4, bool GATED, int WC, int WK>
hipError_t run_few(const MxLinearArgs& a, hipStream_t s) {
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, 16) * ((a.N + 16 * WC - 1) / (16 * WC));
  hipLaunchKernelGGL((linear_mx_few_kernel<ROWS4, GATED, WC, WK>), row::grid_of((items + 7) / 8 * 8), dim3(WC * WK * 64), 0, s, a);
  return hipGetLastError();
}

template <int BQ, int BP, int WQ, int WP>
hipError_t run_backward_x(const MxLinearArgs& a, hipStream_t s) {
  static std::atomic<size_t> allowed[kMaxCachedDevices];
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, BQ) * ((a.K + BP - 1) / BP);
  return launch(&linear_mx_backward_x_kernel<BQ, BP, WQ, WP>, items, WQ * WP * 64, (3 * BQ + 2 * BP) * 128, a, s, allowed);
}

}  // namespace

hipError_t launch_linear_mx(const MxLinearArgs& a, hipStream_t s) {
  if (a.xs != nullptr) return a.parts == 2 ? run_few<true, true, 2, 8>(a, s) : run_few<true, false, 2, 8>(a, s);
  return a.parts == 2 ? run_few<false, true, 2, 8>(a, s) : run_few<false, false, 2, 8>(a, s);
}

hipError_t launch_linear_mx_backward_x(const MxLinearArgs& a, hipStream_t s) { return run_backward_x<128, 128, 2, 2>(a, s); }

}  // namespace moe
