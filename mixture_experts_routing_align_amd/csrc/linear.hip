// The experts' matrix products over sorted rows for gfx950: forward with bias,
// activation, residual and 8-bit rows in the epilogue, and both gradients.
//
//   forward      z[p] = W[e] x[p] + b[e], y[p] = act(z[p]) + residual[p]
//   backward x   dx[p] = sum_n dz[p, n] W[e][n, :]
//   backward w   dW[e][n, :] = sum_p dz[p, n] x[p, :], db[e][n] = sum_p dz[p, n]
//
// All three are one tiled product on the matrix cores that differs in how its
// operands lie in memory (linear_tile.h).
//
// Measured on 128 experts with 32768 rows unevenly routed (17 to 1238 an expert),
// 2 x 768 weight rows of 2048 columns, on random data:
//   gate+up, SwiGLU, pre-activations kept    320 us  640 TFLOP/s, 3.4 TB/s of its bytes
//   the same with 8-bit operands and result  302 us  680 TFLOP/s
//   rows' gradient                           377 us  550 TFLOP/s
//   weights' gradient                        351 us  590 TFLOP/s (805 MB written)
// and 1.17 PFLOP/s for 32768 dense rows of the first; a square library product of 8192
// reaches 1.3.  The matrix cores are busy 20 to 32% of the cycles.  The 805 MB of
// weights take 167 us at a large copy's rate, a fraction of the time, and loads alone
// (no reads, no products) took 280 to 300 of 325 us in the gate+up product, so it is
// the loads that bound it.  Equal runs of 256 rows measure 270 us against 330 there,
// 275 against 308 in 8 bits and 649 against 779 for both gradients, in one loop each.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "linear_epilogue.h"
#include "linear_tile.h"
#include "moe_internal.h"
#include "moe_mi355x_ops.h"
#include "row_common.h"

namespace moe {
namespace {

using namespace tile;
using namespace epilogue;

extern __shared__ __attribute__((aligned(1024))) char smem[];

// ---------------------------------------------------------------- forward --

// A workgroup's tile: BQ rows by BP weight rows (SwiGLU: BP / 2 of the gate and
// the same BP / 2 of the up weight, so that a lane holds z and u of its elements),
// WQ x WP waves, QS stages of rows and PS of weights in LDS.
template <bool FP8, bool GATED, int BQ, int BP, int WQ, int WP, int QS, int PS>
struct Forward {
  static constexpr int kWaves = WQ * WP, kThreads = kWaves * 64;
  static constexpr int kParts = GATED ? 2 : 1;
  static constexpr int kCols = BP / kParts;      // output columns of a tile
  static constexpr int kQ = BQ / WQ / 16;        // 16-row subtiles per wave
  static constexpr int kP = BP / WP / 16;        // 16-column subtiles per wave, all parts
  static constexpr int kC = kP / kParts;         // of them per part
  using QTile = RowTile<BQ, kWaves>;
  using PTile = RowTile<kCols, kWaves>;
  static constexpr int kPBytes = kParts * PTile::kBytes;
  static constexpr int kPLoads = kParts * PTile::kLoads;
  static constexpr int kLds = QS * QTile::kBytes + PS * kPBytes;
};

// The loop's order.  All stages are filled ahead of it; half-way through step s, when
// its last operands are in registers, the waves meet, the buffers of step s are
// filled with rows of step s + QS and weights of step s + PS, and the first operands
// of step s + 1 are read, so that a wave's LDS reads and the next stages' loads run
// beside its matrix instructions.  (With the reads in front of the instructions that
// use them the matrix cores idled through them: 57% busy without any loads.)
//
// Loads of a wave that may be outstanding at that meeting: with two stages of rows
// the weights of step s + 2 where there is a third weight stage (weights come from
// HBM, rows mostly from L2, where several column tiles read them); with more, as
// many of each, all stages but the next.
constexpr int in_flight(int QS, int PS, int q_loads, int p_loads) {
  return QS == 2 ? (PS - 2) * p_loads : (PS - 2) * (q_loads + p_loads);
}
// ... and before step 0: those of the stages behind the first.  With two stages of
// rows their number depends on the rows, so only the weights' are counted on.
constexpr int in_flight_first(int QS, int PS, int q_loads, int p_loads) {
  return QS == 2 ? (PS - 1) * p_loads : (PS - 1) * (q_loads + p_loads);
}

template <bool FP8, bool GATED, int BQ, int BP, int WQ, int WP, int QS, int PS>
__global__ __launch_bounds__(WQ* WP * 64, 2) void linear_kernel(LinearArgs a) {
  using T = Forward<FP8, GATED, BQ, BP, WQ, WP, QS, PS>;
  static_assert((QS == 2 && (PS == 2 || PS == 3)) || (QS > 2 && QS == PS), "the waits are counted for these");
  constexpr int kQ = T::kQ, kP = T::kP, kC = T::kC, kParts = T::kParts, kCols = T::kCols;
  static_assert(kDB == row::kScaleBlock, "a stage of 8-bit depth is one scale block");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wq = wave / WP, wp = wave % WP;
  const Item it = find_item(a, row::block_index(), BQ, (a.N + kCols - 1) / kCols);
  if (it.e < 0) return;
  const int ld = FP8 ? a.K : a.K * 2;
  const int q0 = it.tq * BQ, p0 = it.tp * kCols;
  const int live = min(BQ, it.count - q0);  // rows of this tile
  const int64_t first = (int64_t)it.row0 + q0;
  const __amdgpu_buffer_rsrc_t rx = resource(static_cast<const char*>(a.x) + first * ld);
  const int64_t expert = (int64_t)it.e * a.N * ld;
  __amdgpu_buffer_rsrc_t rw[kParts];
#pragma unroll
  for (int h = 0; h < kParts; ++h) rw[h] = resource(static_cast<const char*>(a.w[h]) + expert);

  typename T::QTile qt;
  typename T::PTile pt;
  qt.init(wave, lane, [&](int r) { return r < live ? (uint32_t)(r * ld) : kNoFetch; });
  pt.init(wave, lane, [&](int r) { return p0 + r < a.N ? (uint32_t)((p0 + r) * ld) : kNoFetch; });
  const int steps = (ld + kDB - 1) / kDB;
  // past the last step nothing is left: the loads are issued and fetch nothing
  auto issue_q = [&](int s, int stage) {
    char* b = smem + stage * T::QTile::kBytes;
    if constexpr (QS == 2)
      qt.load_live(rx, b, wave, s * kDB, ld - s * kDB, live);
    else  // the waits count on every load
      qt.load(rx, b, wave, s * kDB, ld - s * kDB);
  };
  char* const weights = smem + QS * T::QTile::kBytes;
  auto issue_p = [&](int s, int stage) {
#pragma unroll
    for (int h = 0; h < kParts; ++h)
      pt.load(rw[h], weights + stage * T::kPBytes + h * T::PTile::kBytes, wave, s * kDB, ld - s * kDB);
  };

  f32x4 acc[kQ][kP];
#pragma unroll
  for (int i = 0; i < kQ; ++i)
#pragma unroll
    for (int j = 0; j < kP; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // 8-bit: where this lane's row scales and its columns' scales are
  const int blocks = a.K / row::kScaleBlock;
  const float* sx[kQ];
  const float* sw[kParts];
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < kQ; ++i)
      sx[i] = a.x_scale + (first + min(q_row<WQ>(wq, i) + (lane & 15), live - 1)) * blocks;
    static_assert(kCols / WP <= row::kScaleBlock && row::kScaleBlock % (kCols / WP) == 0, "a wave's columns share a scale");
    const int nb = a.N / row::kScaleBlock;
    const int cb = min((p0 + wp * (kCols / WP)) / row::kScaleBlock, nb - 1);
#pragma unroll
    for (int h = 0; h < kParts; ++h) sw[h] = a.ws[h] + ((int64_t)it.e * nb + cb) * blocks;
  }

#pragma unroll
  for (int s = 0; s < PS; ++s) {
    if (QS == 2 && s == 0) issue_p(0, 0);
    if (s < QS) issue_q(s, s);
    if (QS != 2 || s > 0) issue_p(s, s);
  }

  auto p_row = [&](int j) { return wp * (kCols / WP) + (j % kC) * 16; };
  auto multiply = [&](auto live_subtiles) {
    constexpr int L = decltype(live_subtiles)::value;
    float sc[L], sn[L];  // row scales of this step and of the next
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < L; ++i) sn[i] = sx[i][0];
    }
    constexpr int kFirst = in_flight_first(QS, PS, T::QTile::kLoads, T::kPLoads);
    constexpr int kNext = in_flight(QS, PS, T::QTile::kLoads, T::kPLoads);
    int stage = 0, qstage = 0;
    // fills the buffers of step s and moves on to those of step s + 1
    auto advance = [&](int s) {
      wait_and_meet<kNext>();
      issue_q(s + QS, qstage);
      issue_p(s + PS, stage);
      qstage = qstage == QS - 1 ? 0 : qstage + 1;
      stage = stage == PS - 1 ? 0 : stage + 1;
    };
    auto q_lds = [&] { return smem + qstage * T::QTile::kBytes; };
    auto p_lds = [&](int j) { return weights + stage * T::kPBytes + j / kC * T::PTile::kBytes; };
    wait_and_meet<kFirst>();
    if constexpr (FP8) {
      // The matrix cores' own 8-bit products lose the low bits of their sums
      // (measured 1.5e-5 of the result on 128 terms), so the codes are widened to
      // bf16, which is exact, and each scale block is scaled as it is added.
      for (int s = 0; s < steps; ++s) {
        float swc[kParts];
        const int nx = min(s + 1, steps - 1);
#pragma unroll
        for (int i = 0; i < L; ++i) {
          sc[i] = sn[i];
          sn[i] = sx[i][nx];
        }
#pragma unroll
        for (int h = 0; h < kParts; ++h) swc[h] = sw[h][s];
        bf16x8 q[L][4];
        {
          typename T::QTile::Raw8 raw[L];
#pragma unroll
          for (int i = 0; i < L; ++i) raw[i] = T::QTile::raw8(q_lds(), q_row<WQ>(wq, i), lane);
#pragma unroll
          for (int i = 0; i < L; ++i) T::QTile::widen(raw[i], q[i]);
        }
        typename T::PTile::Raw8 next = T::PTile::raw8(p_lds(0), p_row(0), lane);
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          const typename T::PTile::Raw8 raw = next;
          if (j + 1 < kP)
            next = T::PTile::raw8(p_lds(j + 1), p_row(j + 1), lane);
          else
            advance(s);  // the stage's last operands are in registers
          bf16x8 p[4];
          T::PTile::widen(raw, p);
          f32x4 t[L];
#pragma unroll
          for (int i = 0; i < L; ++i) t[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int i = 0; i < L; ++i) t[i] = mma::mfma(p[kk], q[i][kk], t[i]);
#pragma unroll
          for (int i = 0; i < L; ++i) {
            const float f = sc[i] * swc[j / kC];
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(t[i][c], f, acc[i][j][c]);
          }
        }
      }
    } else {
      static_assert(kDB == 128, "two 32-deep halves a stage");
      bf16x8 q[2][L], p[2][kP];
      auto read = [&](int kk) {
#pragma unroll
        for (int i = 0; i < L; ++i) q[kk][i] = T::QTile::frag(q_lds(), q_row<WQ>(wq, i), kk, lane);
#pragma unroll
        for (int j = 0; j < kP; ++j) p[kk][j] = T::PTile::frag(p_lds(j), p_row(j), kk, lane);
      };
      auto products = [&](int kk) {
#pragma unroll
        for (int j = 0; j < kP; ++j)
#pragma unroll
          for (int i = 0; i < L; ++i) acc[i][j] = mma::mfma(p[kk][j], q[kk][i], acc[i][j]);
      };
      read(0);
      for (int s = 0; s < steps; ++s) {
        read(1);
        __builtin_amdgcn_sched_barrier(0);  // the reads are on their way before the products
        products(0);
        __builtin_amdgcn_sched_barrier(0);
        advance(s);
        read(0);  // of step s + 1; past the last one whatever lies there, unused
        __builtin_amdgcn_sched_barrier(0);
        products(1);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  by_live_subtiles<kQ>((live - wq * 16 + 16 * WQ - 1) / (16 * WQ), multiply);
  wait_and_meet<0>();  // the loads past the last step have landed: LDS is free

  // Epilogue: lane l holds row l % 16 and 4 consecutive columns of each subtile.
  const int quad = lane >> 4, row16 = lane & 15;
  const int colw = wp * (kCols / WP) + quad * 4;  // this lane's first column of the tile
  const int cols = min(kCols, a.N - p0);
  using Rows = OutTile<BQ, kCols * 2, T::kThreads>;
  static_assert(BQ * kCols * 2 <= T::kLds, "the output tile fits where the stages were");
  auto columns = [&](auto f) {  // f(subtile row i, subtile column j, tile row, tile column)
#pragma unroll
    for (int i = 0; i < kQ; ++i)
#pragma unroll
      for (int j = 0; j < kC; ++j) f(i, j, q_row<WQ>(wq, i) + row16, colw + j * 16);
  };
  // act(z, u) + residual in place of z; the pre-activations, where they are kept,
  // need the bias on both
  columns([&](int i, int j, int m, int n) {
    float z[4], u[4], y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      z[c] = acc[i][j][c];
      u[c] = acc[i][(GATED ? kC : 0) + j][c];
    }
    epilogue4<GATED>(a, it.e, first + m, p0 + n, m < live && n < cols, z, u, y);
    if (a.preact != nullptr) {
      Rows::put(smem, m, n * 2, pack4(z));
      if (GATED) {
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][kC + j][c] = u[c];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][j][c] = y[c];
  });
  if (a.preact != nullptr) {
    char* pre = reinterpret_cast<char*>(a.preact + first * kParts * a.N + p0);
    __syncthreads();
    Rows::flush(smem, pre, (int64_t)kParts * a.N * 2, live, cols * 2);
    __syncthreads();
    if constexpr (GATED) {
      columns([&](int i, int j, int m, int n) {
        const float u[4] = {acc[i][kC + j][0], acc[i][kC + j][1], acc[i][kC + j][2], acc[i][kC + j][3]};
        Rows::put(smem, m, n * 2, pack4(u));
      });
      __syncthreads();
      Rows::flush(smem, pre + (int64_t)a.N * 2, (int64_t)2 * a.N * 2, live, cols * 2);
      __syncthreads();
    }
  }
  // a tile can write 8-bit rows if it holds whole scale blocks of columns
  constexpr bool kCodes = kCols % row::kScaleBlock == 0;
  if (!kCodes || a.y_scale == nullptr) {
    columns([&](int i, int j, int m, int n) {
      const float y[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      Rows::put(smem, m, n * 2, pack4(y));
    });
    __syncthreads();
    Rows::flush(smem, reinterpret_cast<char*>(static_cast<uint16_t*>(a.y) + first * a.N + p0), (int64_t)a.N * 2, live, cols * 2);
    return;
  }
  if constexpr (kCodes) {
    // each scale block is spread over the waves that hold its columns
    constexpr int kShare = row::kScaleBlock * WP / kCols;  // waves per block
    uint32_t* red = reinterpret_cast<uint32_t*>(smem);     // [WP][BQ] absolute maxima
    char* codes = smem + WP * BQ * 4;
    using Codes = OutTile<BQ, kCols, T::kThreads>;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      uint32_t mx = 0;
#pragma unroll
      for (int j = 0; j < kC; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) mx = max(mx, row::abs_bits(acc[i][j][c]));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
      if (lane < 16) red[wp * BQ + q_row<WQ>(wq, i) + lane] = mx;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      const int m = q_row<WQ>(wq, i) + row16;
      uint32_t mx = 0;
#pragma unroll
      for (int w = 0; w < kShare; ++w) mx = max(mx, red[(wp / kShare * kShare + w) * BQ + m]);
      const float scale = row::block_scale(mx);
      if (m < live && colw < cols && colw % row::kScaleBlock == 0)
        a.y_scale[(first + m) * (a.N / row::kScaleBlock) + (p0 + colw) / row::kScaleBlock] = scale;
      const row::Codes to(scale);
#pragma unroll
      for (int j = 0; j < kC; ++j)
        Codes::put(codes, m, colw + j * 16, to.x4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]));
    }
    __syncthreads();
    Codes::flush(codes, static_cast<char*>(a.y) + first * a.N + p0, a.N, live, cols);
  }
}

// --------------------------------------------------- forward, few rows --

// Few rows per expert: the weights are read once and nothing is reused enough to
// stage it, so a workgroup takes 16 rows by 16 WC columns, and WK waves split the
// depth of each 16 columns in interleaved 128-deep chunks, both operands loaded
// straight into the matrix cores' registers (16 lanes x 256 contiguous bytes a
// chunk).  All loads of a chunk are in flight at once; the WK sums meet in LDS in
// wave order.  8-bit rows out need all 128 columns of a scale block: WC = 8.
// 8 dense rows by 2048 x 2048 take 6.2 us, 8.4 MB of weights at 1.3 TB/s: 128 workgroups
// leave half of the compute units without one, and each walks one dependent memory trip
// (16 waves of one chunk) and the join.  Over experts, 64 rows on 51 of 128, SwiGLU of
// 2 x 768 x 2048: 117 us in bf16, 47 us in 8 bits with 8-bit rows out (2.7 and 3.4 TB/s of
// the active weights).
template <bool FP8, bool GATED, int WC, int WK>
__global__ __launch_bounds__(WC* WK * 64) void linear_few_kernel(LinearArgs a) {
  constexpr int kParts = GATED ? 2 : 1, kCols = 16 * WC, kChunk = 128;
  __shared__ f32x4 part[WC][WK][kParts][64];
  __shared__ uint32_t red[WC][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wc = wave % WC, wk = wave / WC, quad = lane >> 4;
  const Item it = find_item(a, row::block_index(), 16, (a.N + kCols - 1) / kCols);
  if (it.e < 0) return;
  const int live = min(16, it.count - it.tq * 16);
  const int64_t first = (int64_t)it.row0 + it.tq * 16;
  const int col0 = it.tp * kCols + wc * 16;
  // rows and columns past the end repeat the last one and are not stored
  const int64_t xr = first + min(lane & 15, live - 1);
  const int64_t wr = (int64_t)it.e * a.N + min(col0 + (lane & 15), a.N - 1);
  constexpr int kItem = FP8 ? 1 : 2;
  const uint8_t* x = static_cast<const uint8_t*>(a.x) + xr * a.K * kItem;
  const uint8_t* w[kParts];
#pragma unroll
  for (int h = 0; h < kParts; ++h) w[h] = static_cast<const uint8_t*>(a.w[h]) + wr * a.K * kItem;
  f32x4 acc[kParts];
#pragma unroll
  for (int h = 0; h < kParts; ++h) acc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int chunks = (a.K + kChunk - 1) / kChunk;
  constexpr int kLoads = FP8 ? 2 : 4;  // 16-byte pieces of a lane's 32 depth elements
  if constexpr (FP8) {
    const int nb = a.N / row::kScaleBlock;
    const float* sx = a.x_scale + xr * chunks;
    const float* sw[kParts];
#pragma unroll
    for (int h = 0; h < kParts; ++h) sw[h] = a.ws[h] + ((int64_t)it.e * nb + min(col0, a.N - 1) / row::kScaleBlock) * chunks;
    for (int c = wk; c < chunks; c += WK) {
      uint4 xv[kLoads], wv[kParts][kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = c * kChunk + quad * 32 + i * 16;
        xv[i] = *reinterpret_cast<const uint4*>(x + at);
#pragma unroll
        for (int h = 0; h < kParts; ++h) wv[h][i] = *reinterpret_cast<const uint4*>(w[h] + at);
      }
      const float f = sx[c];
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        f32x4 t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          t = mma::mfma(mma::fp8x8_to_bf16(wv[h][i].x, wv[h][i].y), mma::fp8x8_to_bf16(xv[i].x, xv[i].y), t);
          t = mma::mfma(mma::fp8x8_to_bf16(wv[h][i].z, wv[h][i].w), mma::fp8x8_to_bf16(xv[i].z, xv[i].w), t);
        }
        const float g = f * sw[h][c];
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[h][k] = fmaf(t[k], g, acc[h][k]);
      }
    }
  } else {
    for (int c = wk; c < chunks; c += WK) {
      uint4 xv[kLoads], wv[kParts][kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int d = c * kChunk + quad * 32 + i * 8;
        const bool in = d < a.K;  // K is a multiple of 8
        const int at = in ? d * 2 : 0;
        xv[i] = *reinterpret_cast<const uint4*>(x + at);
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          wv[h][i] = *reinterpret_cast<const uint4*>(w[h] + at);
          if (!in) wv[h][i] = make_uint4(0, 0, 0, 0);
        }
        if (!in) xv[i] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int h = 0; h < kParts; ++h) acc[h] = mma::mfma(mma::as_bf16x8(wv[h][i]), mma::as_bf16x8(xv[i]), acc[h]);
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
    if (a.y_scale == nullptr && in) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + (first + m) * a.N + n) = pack4(y);
  }
  if constexpr (WC == 8) {
    if (a.y_scale == nullptr) return;
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
      uint32_t mx = 0;
#pragma unroll
      for (int i = 0; i < WC; ++i) mx = max(mx, red[i][m]);
      const float scale = row::block_scale(mx);
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.y) + (first + m) * a.N + n) = row::Codes(scale).x4(y[0], y[1], y[2], y[3]);
      if (n % row::kScaleBlock == 0) a.y_scale[(first + m) * (a.N / row::kScaleBlock) + n / row::kScaleBlock] = scale;
    }
  }
}

// ------------------------------------------------------------- backward x --

// One workgroup: BQ rows by BP columns of dx; the depth is the weight rows, gate's then
// up's.  The weights lie across the depth, so they are transposed on their way from LDS
// to the registers.  Measured 377 us (see the top), 292 to 297 with equal runs.
template <int BQ, int BP, int WQ, int WP, int PS>
__global__ __launch_bounds__(WQ* WP * 64, 2) void linear_backward_x_kernel(LinearArgs a) {
  constexpr int kWaves = WQ * WP, kQ = BQ / WQ / 16, kP = BP / WP / 16, kD = 64;
  static_assert(PS == 2 || PS == 3, "waits are counted for two or three weight stages");
  using QTile = RowTile<BQ, kWaves>;
  using PTile = DepthTile<BP, kD, kWaves>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wq = wave / WP, wp = wave % WP;
  const Item it = find_item(a, row::block_index(), BQ, (a.K + BP - 1) / BP);
  if (it.e < 0) return;
  const int q0 = it.tq * BQ, p0 = it.tp * BP;
  const int live = min(BQ, it.count - q0);
  const int64_t first = (int64_t)it.row0 + q0;
  const int ldq = a.parts * a.N * 2, ldp = a.K * 2;
  const char* dz = static_cast<const char*>(a.dz) + first * ldq;
  const int64_t expert = (int64_t)it.e * a.N * ldp + p0 * 2;
  QTile qt;
  PTile pt;
  qt.init(wave, lane, [&](int r) { return r < live ? (uint32_t)(r * ldq) : kNoFetch; });
  pt.init(wave, lane, ldp, [&](int g) { return p0 + g * 8 < a.K ? (uint32_t)(g * 16) : kNoFetch; });
  // the depth runs over the N columns of dz's first part, then of its second
  const int per = (a.N + kD - 1) / kD, steps = per * a.parts;
  const __amdgpu_buffer_rsrc_t rq = resource(dz);
  // past the last step nothing is left: the loads are issued and fetch nothing
  auto issue_q = [&](int s) {
    const int h = s >= per ? 1 : 0, k = s - h * per;
    qt.load_live(rq, smem + (s & 1) * QTile::kBytes, wave, (h * a.N + k * kD) * 2, s < steps ? (a.N - k * kD) * 2 : 0, live);
  };
  char* const weights = smem + 2 * QTile::kBytes;
  const char* const w0 = static_cast<const char*>(a.w[0]) + expert;
  const char* const w1 = a.parts == 2 ? static_cast<const char*>(a.w[1]) + expert : w0;
  auto issue_p = [&](int s, int stage) {
    const int h = s >= per ? 1 : 0, k = s - h * per;
    pt.load(resource((h ? w1 : w0) + (int64_t)k * kD * ldp), weights + stage * PTile::kBytes, wave, 0,
            s < steps ? a.N - k * kD : 0);
  };
  f32x4 acc[kQ][kP];
#pragma unroll
  for (int i = 0; i < kQ; ++i)
#pragma unroll
    for (int j = 0; j < kP; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < PS; ++s) {
    issue_p(s, s);
    if (s < 2) issue_q(s);
  }
  auto multiply = [&](auto live_subtiles) {
    constexpr int L = decltype(live_subtiles)::value;
    int stage = 0;
    bf16x8 q[2][L], p[2][kP];
    auto read = [&](int s, int kk) {
      const char* b = smem + (s & 1) * QTile::kBytes;
#pragma unroll
      for (int i = 0; i < L; ++i) q[kk][i] = QTile::frag(b, q_row<WQ>(wq, i), kk, lane);
#pragma unroll
      for (int j = 0; j < kP; ++j) p[kk][j] = PTile::frag(weights + stage * PTile::kBytes, wp * (BP / WP) + j * 16, kk, lane);
    };
    auto products = [&](int kk) {
#pragma unroll
      for (int j = 0; j < kP; ++j)
#pragma unroll
        for (int i = 0; i < L; ++i) acc[i][j] = mma::mfma(p[kk][j], q[kk][i], acc[i][j]);
    };
    wait_and_meet<in_flight_first(2, PS, QTile::kLoads, PTile::kLoads)>();
    read(0, 0);
    for (int s = 0; s < steps; ++s) {  // in the forward kernel's order
      read(s, 1);
      __builtin_amdgcn_sched_barrier(0);
      products(0);
      __builtin_amdgcn_sched_barrier(0);
      wait_and_meet<in_flight(2, PS, QTile::kLoads, PTile::kLoads)>();
      issue_q(s + 2);
      issue_p(s + PS, stage);
      stage = stage == PS - 1 ? 0 : stage + 1;
      read(s + 1, 0);
      __builtin_amdgcn_sched_barrier(0);
      products(1);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  by_live_subtiles<kQ>((live - wq * 16 + 16 * WQ - 1) / (16 * WQ), multiply);
  wait_and_meet<0>();
  using Rows = OutTile<BQ, BP * 2, kWaves * 64>;
  static_assert(BQ * BP * 2 <= 2 * QTile::kBytes + PS * PTile::kBytes, "the output tile fits where the stages were");
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

// ------------------------------------------------------------- backward w --

// One workgroup: BQ weight rows by BP columns of one expert's gradient, over one of
// `splits` equal parts of its rows.  Its 805 MB of results bound it (see the top): 351 us
// alone, 284 with equal runs, 407 to 435 right behind the rows' gradient under a tracer.
template <bool BIAS, int BQ, int BP, int WQ, int WP, int kD, int STAGES, int OCC>
__global__ __launch_bounds__(WQ* WP * 64, OCC) void linear_backward_w_kernel(LinearArgs a) {
  constexpr int kWaves = WQ * WP, kQ = BQ / WQ / 16, kP = BP / WP / 16;
  using QTile = DepthTile<BQ, kD, kWaves>;
  using PTile = DepthTile<BP, kD, kWaves>;
  constexpr int kStage = QTile::kBytes + PTile::kBytes, kLoads = QTile::kLoads + PTile::kLoads;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wq = wave / WP, wp = wave % WP;
  // experts dealt to XCDs in 8 equal runs of workgroups, as find_item does
  const int tn = (a.N + BQ - 1) / BQ, tk = (a.K + BP - 1) / BP;
  const int total = a.E * a.parts * tn * tk * a.splits, chunk = (total + 7) / 8;
  const int b = (int)row::block_index();
  int i = (b & 7) * chunk + (b >> 3);
  if ((b >> 3) >= chunk || i >= total) return;
  const int split = i % a.splits;
  i /= a.splits;
  const int tp = i % tk;
  i /= tk;
  const int tq = i % tn;
  i /= tn;
  const int h = i % a.parts, e = i / a.parts;
  const int row0 = a.offsets != nullptr ? a.offsets[e] : 0;
  const int count = a.offsets != nullptr ? run_length(row0, a.counts[e], a.rows) : a.rows;
  const RowRange range = split_rows(count, split, a.splits, kD);
  const int begin = range.begin, rows = range.rows;
  const int q0 = tq * BQ, p0 = tp * BP;
  const int ldq = a.parts * a.N * 2, ldp = a.K * 2;
  const int64_t first = count > 0 ? (int64_t)row0 + begin : 0;
  const char* dz = static_cast<const char*>(a.dz) + first * ldq + ((int64_t)h * a.N + q0) * 2;
  const char* x = static_cast<const char*>(a.x) + first * ldp + p0 * 2;
  QTile qt;
  PTile pt;
  qt.init(wave, lane, ldq, [&](int g) { return q0 + g * 8 < a.N ? (uint32_t)(g * 16) : kNoFetch; });
  pt.init(wave, lane, ldp, [&](int g) { return p0 + g * 8 < a.K ? (uint32_t)(g * 16) : kNoFetch; });
  const int steps = ceil_div(rows, kD);
  auto issue = [&](int s, int stage) {
    char* b = smem + stage * kStage;
    const int left = rows_left(rows, s, kD);
    qt.load(resource(dz + (int64_t)s * kD * ldq), b, wave, 0, left);
    pt.load(resource(x + (int64_t)s * kD * ldp), b + QTile::kBytes, wave, 0, left);
  };
  f32x4 acc[kQ][kP], ones_acc[BIAS ? kQ : 1];
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    if (BIAS) ones_acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < kP; ++p) acc[q][p] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // the bias gradient is the product with a column of ones: by the workgroups of
  // the first column tile, in their first column of waves
  const bool sums = BIAS && tp == 0 && wp == 0;
  const __bf16 one = (__bf16)1.0f;
  const bf16x8 ones{one, one, one, one, one, one, one, one};
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s, s);
  int stage = 0;
  for (int s = 0; s < steps; ++s) {
    wait_and_meet<(STAGES - 2) * kLoads>();
    issue(s + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
    const char* b = smem + stage * kStage;
    stage = stage == STAGES - 1 ? 0 : stage + 1;
#pragma unroll
    for (int kk = 0; kk < kD / 32; ++kk) {
      bf16x8 q[kQ], p[kP];
#pragma unroll
      for (int r = 0; r < kQ; ++r) q[r] = QTile::frag(b, wq * (BQ / WQ) + r * 16, kk, lane);
#pragma unroll
      for (int c = 0; c < kP; ++c) p[c] = PTile::frag(b + QTile::kBytes, wp * (BP / WP) + c * 16, kk, lane);
      if (sums) {
#pragma unroll
        for (int r = 0; r < (BIAS ? kQ : 0); ++r) ones_acc[r] = mma::mfma(ones, q[r], ones_acc[r]);
      }
#pragma unroll
      for (int c = 0; c < kP; ++c)
#pragma unroll
        for (int r = 0; r < kQ; ++r) acc[r][c] = mma::mfma(p[c], q[r], acc[r][c]);
    }
  }
  wait_and_meet<0>();
  // with splits the sums go to the workspace: per split dw (all parts), then db
  const int64_t weight = (int64_t)a.E * a.N * a.K;
  const bool whole = a.splits == 1;
  float* part = whole ? nullptr : a.part + split * (a.parts * (weight + (BIAS ? (int64_t)a.E * a.N : 0)));
  const int64_t line0 = (int64_t)e * a.N + q0;
  if constexpr (BIAS) {
    if (sums && lane < 16) {
      float* db = (whole ? a.db[h] : part + a.parts * weight + (int64_t)h * a.E * a.N) + line0;
#pragma unroll
      for (int r = 0; r < kQ; ++r) {
        const int n = wq * (BQ / WQ) + r * 16 + lane;
        if (q0 + n < a.N) db[n] = ones_acc[r][0];
      }
    }
  }
  if (whole && !a.dw_f32) {
    using Rows = OutTile<BQ, BP * 2, kWaves * 64>;
    static_assert(BQ * BP * 2 <= STAGES * kStage, "the output tile fits where the stages were");
#pragma unroll
    for (int r = 0; r < kQ; ++r)
#pragma unroll
      for (int c = 0; c < kP; ++c) {
        const float v[4] = {acc[r][c][0], acc[r][c][1], acc[r][c][2], acc[r][c][3]};
        Rows::put(smem, wq * (BQ / WQ) + r * 16 + (lane & 15), (wp * (BP / WP) + c * 16 + (lane >> 4) * 4) * 2, pack4(v));
      }
    __syncthreads();
    Rows::template flush<true>(smem, reinterpret_cast<char*>(static_cast<uint16_t*>(a.dw[h]) + line0 * a.K + p0), (int64_t)a.K * 2,
                min(BQ, a.N - q0), min(BP, a.K - p0) * 2);
    return;
  }
  // float32: a lane's 16 bytes go out as they are, 64 bytes of each of 16 rows at a time
  // (both gradients of 128 experts, 2 x 768 x 2048, 32768 rows: 1150 us, 810 with bf16
  // results, which are half the bytes and leave as whole lines)
  float* out = (whole ? static_cast<float*>(a.dw[h]) : part + h * weight) + line0 * a.K;
#pragma unroll
  for (int r = 0; r < kQ; ++r) {
    const int n = wq * (BQ / WQ) + r * 16 + (lane & 15);
    if (q0 + n >= a.N) continue;
#pragma unroll
    for (int c = 0; c < kP; ++c) {
      const int k = p0 + wp * (BP / WP) + c * 16 + (lane >> 4) * 4;
      if (k < a.K) __builtin_nontemporal_store(acc[r][c], reinterpret_cast<f32x4*>(out + (int64_t)n * a.K + k));
    }
  }
}

// Joins the splits' sums in order, 4 elements a thread (every part is a multiple
// of 8 elements long).
__global__ __launch_bounds__(256) void join_splits_kernel(LinearArgs a) {
  const int64_t weight = (int64_t)a.E * a.N * a.K, bias = a.db[0] != nullptr ? (int64_t)a.E * a.N : 0;
  const int64_t total = a.parts * (weight + bias);
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= total) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(a.part + i);
  for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const f32x4*>(a.part + s * total + i);
  if (i < a.parts * weight) {
    const int h = i >= weight ? 1 : 0;
    const int64_t at = i - h * weight;
    const float f[4] = {v[0], v[1], v[2], v[3]};
    if (a.dw_f32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.dw[h]) + at) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dw[h]) + at) = pack4(f);
  } else {
    const int64_t b = i - a.parts * weight;
    const int h = b >= bias ? 1 : 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) a.db[h][b - h * bias + c] = v[c];
  }
}

// ---------------------------------------------------- activation gradient --

// Element by element: dy, the pre-activations and dz pass once.  32768 rows of 768 over 128
// experts: 65 us for SwiGLU, 42 us for the others, 3.9 and 3.6 TB/s of those bytes, short of
// what HBM gives the norm (6 TB/s): a workgroup searches its run before its first load.
constexpr int kActRows = 16;  // rows a workgroup takes

__global__ __launch_bounds__(256) void act_backward_kernel(LinearArgs a, const uint16_t* __restrict__ dy,
                                                           const uint16_t* pre, uint16_t* dz) {
  const Item it = find_item(a, row::block_index(), kActRows, 1);
  if (it.e < 0) return;
  const int per = a.N / 8, rows = min(kActRows, it.count - it.tq * kActRows);
  const int64_t first = (int64_t)it.row0 + it.tq * kActRows;
  for (int i = threadIdx.x; i < rows * per; i += 256) {
    const int rr = i / per, c = (i - rr * per) * 8;
    const int64_t r = first + rr;
    float g[8], z[8], o[8];
    row::load8(dy + r * a.N, c, a.N, g);
    row::load8(pre + r * a.parts * a.N, c, a.N, z);
    if (a.act == MOE_ACT_GELU) {
      // s + 2 z s (1 - s) a', s = sigmoid(2 a)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = sigmoid_all(gelu_2a(z[j]));
        const float d = 1.5957691216057308f * fmaf(3.0f * 0.044715f * z[j], z[j], 1.0f);
        // where the sigmoid has reached 0 or 1 its slope is 0, also where a' overflows
        const float bend = s * (1.0f - s);
        o[j] = g[j] * (s + (bend > 0.f ? z[j] * bend * d : 0.f));
      }
    } else {
      float u[8], o2[8];
      if (a.act == MOE_ACT_SWIGLU) row::load8(pre + r * 2 * a.N + a.N, c, a.N, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = sigmoid_all(z[j]);
        const float d = s * fmaf(z[j], 1.0f - s, 1.0f);
        if (a.act == MOE_ACT_SWIGLU) {
          o[j] = g[j] * u[j] * d;
          o2[j] = g[j] * (z[j] * s);
        } else {
          o[j] = g[j] * d;
        }
      }
      if (a.act == MOE_ACT_SWIGLU) row::store8(dz + r * 2 * a.N + a.N, c, a.N, o2);
    }
    row::store8(dz + r * a.parts * a.N, c, a.N, o);
  }
}

// ---------------------------------------------------------------- launch --

// Instantiated by name: the host pass of this compiler otherwise leaves out the
// launch stubs of some kernel templates that are only reached through pointers.
#define MOE_TILES(F, G)                                                              \
  template __global__ void linear_kernel<F, G, F ? 32 : 64, 64, 2, 2, 3, 3>(LinearArgs);  \
  template __global__ void linear_kernel<F, G, 128, 128, F ? 4 : 2, 2, 2, 3>(LinearArgs); \
  template __global__ void linear_few_kernel<F, G, 1, 16>(LinearArgs);               \
  template __global__ void linear_few_kernel<F, G, 8, 2>(LinearArgs);
MOE_TILES(false, false)
MOE_TILES(false, true)
MOE_TILES(true, false)
MOE_TILES(true, true)
#undef MOE_TILES
template __global__ void linear_kernel<false, false, 32, 64, 2, 2, 4, 4>(LinearArgs);
template __global__ void linear_kernel<false, false, 256, 256, 2, 4, 2, 3>(LinearArgs);
template __global__ void linear_kernel<false, true, 256, 256, 2, 4, 2, 3>(LinearArgs);
template __global__ void linear_kernel<true, true, 64, 256, 2, 4, 2, 2>(LinearArgs);
template __global__ void linear_backward_x_kernel<32, 128, 2, 2, 3>(LinearArgs);
template __global__ void linear_backward_x_kernel<64, 128, 2, 2, 3>(LinearArgs);
template __global__ void linear_backward_x_kernel<128, 128, 2, 2, 3>(LinearArgs);
template __global__ void linear_backward_x_kernel<256, 256, 2, 4, 3>(LinearArgs);
template __global__ void linear_backward_w_kernel<false, 128, 128, 2, 2, 32, 2, 4>(LinearArgs);
template __global__ void linear_backward_w_kernel<true, 128, 128, 2, 2, 32, 2, 3>(LinearArgs);

template <typename K>
hipError_t launch(K kern, int64_t items, int threads, int lds, const LinearArgs& a, hipStream_t s,
                  std::atomic<size_t> (&allowed)[kMaxCachedDevices]) {
  const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(kern), lds, allowed);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, row::grid_of((items + 7) / 8 * 8), dim3(threads), lds, s, a);
  return hipGetLastError();
}

template <bool FP8, bool GATED, int BQ, int BP, int WQ, int WP, int QS, int PS>
hipError_t run_forward(const LinearArgs& a, hipStream_t s) {
  using T = Forward<FP8, GATED, BQ, BP, WQ, WP, QS, PS>;
  static std::atomic<size_t> allowed[kMaxCachedDevices];
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, BQ) * ((a.N + T::kCols - 1) / T::kCols);
  void (*const kern)(LinearArgs) = &linear_kernel<FP8, GATED, BQ, BP, WQ, WP, QS, PS>;
  return launch(kern, items, T::kThreads, T::kLds, a, s, allowed);
}

template <bool FP8, bool GATED, int WC, int WK>
hipError_t run_few(const LinearArgs& a, hipStream_t s) {
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, 16) * ((a.N + 16 * WC - 1) / (16 * WC));
  hipLaunchKernelGGL((linear_few_kernel<FP8, GATED, WC, WK>), row::grid_of((items + 7) / 8 * 8), dim3(WC * WK * 64), 0, s, a);
  return hipGetLastError();
}

constexpr int kBQ = 128, kBP = 128;

// Rows per expert on average, of the matrix's height: the runs themselves are known on the
// device only, so the alignment's padding counts, here and in tiles().  With a block
// size far above the runs it weighs more than the rows do (64 rows over 128 experts, SwiGLU
// of 2 x 768 x 2048, bf16: 117 us aligned to 16, 154 to 64, in the same form with more
// empty workgroups; 512 rows: 253 and 164 us, in the depth-split form and in 128-wide tiles).
int64_t mean_rows(const LinearArgs& a) { return ceil_div(a.rows, a.E); }

// Square tiles of `edge` that the rows and `cols` columns make.
int64_t tiles(const LinearArgs& a, int64_t cols, int64_t edge) {
  return (a.rows + edge - 1) / edge * ((cols + edge - 1) / edge);
}

// 256-wide tiles read each operand byte half as often as 128-wide ones and are four
// times the work: taken where they fill the GPU and the runs fill most of them
// (32768 dense rows, gate+up of 1536 x 2048: 177 against 196 us; 128 experts of 256
// rows on average: 303 against 309).
bool wide_tiles(const LinearArgs& a, int64_t cols) { return tiles(a, cols, 256) >= 256 && mean_rows(a) >= 160; }

// Rows per expert up to which the depth-split kernel is taken.
constexpr int64_t kFewRows = 32;

template <bool FP8, bool GATED>
hipError_t forward_by_shape(const LinearArgs& a, hipStream_t s) {
  if (mean_rows(a) <= kFewRows) return a.y_scale != nullptr ? run_few<FP8, GATED, 8, 2>(a, s) : run_few<FP8, GATED, 1, 16>(a, s);
  const bool codes = a.y_scale != nullptr;  // 8-bit rows need whole scale blocks of columns in a tile
  if (GATED && codes) {
    // a tile with 128 columns of SwiGLU takes 256 weight rows; 8-bit operands: 32 x 64
    // per wave, which leaves room for 4 waves per SIMD (291 us at 32768 rows; 64 x 64
    // with 2: 322).  There is no smaller tile for few rows (512 rows of 8 experts, 768 x
    // 2048, 8-bit operands: 30 us, against 14.5 with bf16 rows out, which have one).
    if constexpr (FP8 && GATED) return run_forward<FP8, GATED, 64, 256, 2, 4, 2, 2>(a, s);
    if constexpr (!FP8 && GATED) return run_forward<FP8, GATED, 256, 256, 2, 4, 2, 3>(a, s);
  }
  // Few tiles: smaller ones, of which more than one shares a compute unit (six stages of
  // 64 x 64, which leave one: 19.5 against 12.5 us at 1554 rows of 12 experts, 520 x 1000).
  // 32 x 64 for 8-bit operands, whose widening it spreads (the same, 512 x 1024: 9.0
  // against 13.0 us with 64 x 64; 256 x 2048 x 2048: 9.6 and 14.6; equal, 18.5, at 1024
  // rows), and for bf16 while 64 x 64 tiles would not fill the GPU (256 x 2048 x 2048:
  // 9.1 against 11.7; 1024 rows: 21.4 and 15.9), except under SwiGLU, where it loses
  // (512 rows of 8 experts, 768 x 2048: 12.7 against 11.8).
  if (!codes && tiles(a, a.parts * (int64_t)a.N, 128) < 256) {
    if constexpr (FP8) return run_forward<FP8, GATED, 32, 64, 2, 2, 3, 3>(a, s);
    if constexpr (!FP8 && !GATED)
      if (tiles(a, a.N, 64) < 256) return run_forward<FP8, GATED, 32, 64, 2, 2, 4, 4>(a, s);
    if constexpr (!FP8) return run_forward<FP8, GATED, 64, 64, 2, 2, 3, 3>(a, s);
  }
  if constexpr (!FP8)
    if (wide_tiles(a, a.parts * (int64_t)a.N)) return run_forward<FP8, GATED, 256, 256, 2, 4, 2, 3>(a, s);
  return run_forward<FP8, GATED, 128, 128, FP8 ? 4 : 2, 2, 2, 3>(a, s);
}
}  // namespace

hipError_t launch_linear(const LinearArgs& a, bool fp8, hipStream_t s) {
  if (fp8) return a.parts == 2 ? forward_by_shape<true, true>(a, s) : forward_by_shape<true, false>(a, s);
  return a.parts == 2 ? forward_by_shape<false, true>(a, s) : forward_by_shape<false, false>(a, s);
}

template <int BQ, int BP, int WQ, int WP>
hipError_t run_backward_x(const LinearArgs& a, hipStream_t s) {
  static std::atomic<size_t> allowed[kMaxCachedDevices];
  constexpr int kPS = 3;
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, BQ) * ((a.K + BP - 1) / BP);
  return launch(&linear_backward_x_kernel<BQ, BP, WQ, WP, kPS>, items, WQ * WP * 64, (2 * BQ + kPS * BP) * 128, a, s, allowed);
}

hipError_t launch_linear_backward_x(const LinearArgs& a, hipStream_t s) {
  if (wide_tiles(a, a.K)) return run_backward_x<256, 256, 2, 4>(a, s);
  // Few tiles: fewer rows each, so that more than one shares a compute unit (1024 x 2048 x
  // 2048: 24 us with 64 x 128, 27 with 32 x 128, 36 with 128 x 128; 8 experts of 64 rows,
  // 2 x 768 x 2048: 23, 21 and 23).
  if (tiles(a, a.K, 128) < 256)
    return mean_rows(a) <= 64 ? run_backward_x<32, 128, 2, 2>(a, s) : run_backward_x<64, 128, 2, 2>(a, s);
  return run_backward_x<128, 128, 2, 2>(a, s);
}

int backward_w_splits(int64_t rows, int E, int N, int K, int parts) {
  const int64_t tiles = (int64_t)E * parts * ((N + kBQ - 1) / kBQ) * ((K + kBP - 1) / kBP);
  if (tiles >= 256) return 1;
  // workgroups for two rounds of the GPU, as long as a split keeps 256 rows on average
  return (int)std::max<int64_t>(1, std::min<int64_t>((512 + tiles - 1) / tiles, rows / E / 256));
}

// Stages of 32 rows: an expert's run is short (256 rows: 8 steps), so what counts is
// that 4 workgroups share a compute unit and one's stores overlap another's loads
// (128 experts x 1536 x 2048: 296 us; 128 x 256 tiles 315, 256 x 256 in 64-row stages 338).
template <bool BIAS, int OCC>
hipError_t run_backward_w(const LinearArgs& a, hipStream_t s) {
  static std::atomic<size_t> allowed[kMaxCachedDevices];
  constexpr int kD = 32, kStages = 2;
  const int64_t items = (int64_t)a.E * a.parts * ((a.N + kBQ - 1) / kBQ) * ((a.K + kBP - 1) / kBP) * a.splits;
  return launch(&linear_backward_w_kernel<BIAS, kBQ, kBP, 2, 2, kD, kStages, OCC>, items, 256, kStages * (kBQ + kBP) * kD * 2, a, s,
                allowed);
}

hipError_t launch_linear_backward_w(const LinearArgs& a, hipStream_t s) {
  const hipError_t e = a.db[0] != nullptr ? run_backward_w<true, 3>(a, s) : run_backward_w<false, 4>(a, s);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t total = (int64_t)a.parts * a.E * a.N * (a.K + (a.db[0] != nullptr ? 1 : 0));
  hipLaunchKernelGGL(join_splits_kernel, dim3((unsigned)((total / 4 + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_act_backward(const LinearArgs& a, const uint16_t* dy, const uint16_t* pre, uint16_t* dz, hipStream_t s) {
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, kActRows);
  hipLaunchKernelGGL(act_backward_kernel, row::grid_of((items + 7) / 8 * 8), dim3(256), 0, s, a, dy, pre, dz);
  return hipGetLastError();
}

}  // namespace moe
