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

__device__ __forceinline__ u32x4 as_vec(uint4 v) { return u32x4{v.x, v.y, v.z, v.w}; }

// Calls f with 0, 1, ... N - 1, each a constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f(Count<I>{});
    each<N, I + 1>(f);
  }
}

// ---------------------------------------------------------------- forward --

// Scale bytes of R operand rows, staged by direct 4-byte loads in groups of G steps of 256
// depth elements (8 bytes a step): every line that a load touches is a request to L2, as
// dear as one for 64 bytes of codes, and 8 bytes a row and step were as many requests as
// the codes' (16384 rows by 4096 x 7168 over 16 experts: 395 us, all of it the loads').
// ALIGNED: a row's bytes begin at a multiple of 4, as they do where the depth is a multiple
// of 128 and the array is 4-byte aligned.  Else they are loaded from the dword that holds
// the first one on (none that holds no byte of the row), and the row's shift into it is
// added when they are read.
template <int R, int WAVES, int G, bool ALIGNED>
struct ScaleTile {
  static constexpr int kWords = 2 * G + (ALIGNED ? 0 : 1);  // dwords of LDS a row
  static constexpr int kBytes = (R * kWords * 4 + 15) / 16 * 16;
  static constexpr int kPerWave = R * kWords / WAVES;
  static constexpr int kLoads = (kPerWave + 63) / 64;
  static_assert(R * kWords % WAVES == 0, "equal loads for all waves");
  uint32_t off[kLoads];  // byte offset of each of this lane's dwords in group 0, or kNoFetch
  int end[kLoads];       // bytes from there to the end of its row

  // `lead`: bytes from the resource's (aligned) base to row 0; `row_of(r)`: the row of the
  // array that operand row r is, or -1; `S` bytes a row.
  template <typename F>
  __device__ __forceinline__ void init(int wave, int lane, int lead, int S, F row_of) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int d = wave * kPerWave + i * 64 + lane, r = row_of(d / kWords), w = d % kWords;
      const int begin = lead + r * S, at = (begin & ~3) + w * 4;
      off[i] = r < 0 ? kNoFetch : (uint32_t)at;
      end[i] = begin + S - at;
    }
  }
  // Fills `lds` with the bytes of group g.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, char* lds, int wave, int lane, int g) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i * 64 + 64 <= kPerWave || i * 64 + lane < kPerWave)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (wave * kPerWave + i * 64) * 4), 4,
                                                 g * G * 8 < end[i] ? off[i] : kNoFetch, g * G * 8, 0, 0);
  }
  // Where lane l finds the bytes of blocks 2 q and 2 q + 1 (q = l / 16) of operand row l % 16
  // in step 0 of a group; the same for row r0 + l % 16, r0 a multiple of 16, r0 kRow on.
  static constexpr int kRow = kWords * 4;
  __device__ static __forceinline__ int lane_at(int lane, int lead, int S) {
    const int r = lane & 15;
    return r * kRow + (lane >> 4) * 2 + (ALIGNED ? 0 : (lead + r * S) & 3);
  }
  // The two bytes at p, the first in the lowest; `left`: blocks from there to the row's last,
  // past which the codes are zeros and the byte must not be a NaN's.
  __device__ static __forceinline__ uint32_t pair(const char* p, int left) {
    if constexpr (ALIGNED) {
      return *reinterpret_cast<const uint16_t*>(p);
    } else {
      const uint32_t lo = *reinterpret_cast<const uint8_t*>(p), hi = *reinterpret_cast<const uint8_t*>(p + 1);
      return (0 < left ? lo : 0u) | (1 < left ? hi << 8 : 0u);
    }
  }
};

// The end of a tile: bias, activation and residual on the float32 sums, pre-activations,
// bf16 or MXFP4 rows.  Lane l holds row l % 16 and 4 consecutive columns of each subtile,
// acc[i][j] of a wave's row subtiles i and its columns' subtiles j (SwiGLU: kC of z, then kC
// of u).  LDS is free.
template <bool GATED, int BQ, int kCols, int WQ, int WP, int kQ, int kC>
__device__ __forceinline__ void finish(const MxLinearArgs& a, int e, int64_t first, int live, int p0, int wq, int wp,
                                       f32x4 (&acc)[kQ][GATED ? 2 * kC : kC]) {
  constexpr int kParts = GATED ? 2 : 1, kThreads = WQ * WP * 64;
  static_assert(kC % 2 == 0, "a wave holds whole scale blocks of its rows' columns");
  const int lane = threadIdx.x & 63, quad = lane >> 4, row16 = lane & 15;
  const int colw = wp * (kCols / WP) + quad * 4;  // this lane's first column of the tile
  const int cols = min(kCols, a.N - p0);
  using Rows = OutTile<BQ, kCols * 2, kThreads>;
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
    epilogue4<GATED>(a, e, first + m, p0 + n, m < live && n < cols, z, u, y);
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
  if (a.ysb == nullptr) {
    columns([&](int i, int j, int m, int n) {
      const float y[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      Rows::put(smem, m, n * 2, pack4(y));
    });
    __syncthreads();
    Rows::flush(smem, reinterpret_cast<char*>(static_cast<uint16_t*>(a.y) + first * a.N + p0), (int64_t)a.N * 2, live, cols * 2);
    return;
  }
  // a scale block is two subtiles over the four quads of one wave
  using Codes = OutTile<BQ, kCols / 2, kThreads>;
#pragma unroll
  for (int i = 0; i < kQ; ++i) {
    const int m = q_row<WQ>(wq, i) + row16;
#pragma unroll
    for (int j = 0; j < kC; j += 2) {
      uint32_t mx = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) mx = max(mx, max(row::abs_bits(acc[i][j][c]), row::abs_bits(acc[i][j + 1][c])));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
      mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
      const uint32_t byte = mx::scale_byte(mx);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        Codes::put(smem, m, (colw + (j + h) * 16) / 2,
                   (uint16_t)mx::codes4(acc[i][j + h][0], acc[i][j + h][1], acc[i][j + h][2], acc[i][j + h][3], byte));
      const int n = wp * (kCols / WP) + j * 16;
      if (quad == 0 && m < live && n < cols) a.ysb[(first + m) * (a.N / mx::kBlock) + (p0 + n) / mx::kBlock] = (uint8_t)byte;
    }
  }
  __syncthreads();
  Codes::flush(smem, static_cast<char*>(a.y) + (first * a.N + p0) / 2, a.N / 2, live, cols / 2);
}

// MXFP4 rows: a workgroup's tile is BQ rows by BP weight rows (SwiGLU: BP / 2 of the gate
// and the same BP / 2 of the up weight), WQ x WP waves, STAGES stages of 256 depth elements,
// 128 bytes of codes a row, and two groups of G steps' scale bytes.  Lane l takes blocks
// 2 (l / 16) and 2 (l / 16) + 1 of a stage, one for each of its two halves.
template <bool GATED, bool ALIGNED, int BQ, int BP, int WQ, int WP, int STAGES, int G>
struct Rows4 {
  static constexpr int kWaves = WQ * WP, kThreads = kWaves * 64;
  static constexpr int kParts = GATED ? 2 : 1;
  static constexpr int kCols = BP / kParts;
  static constexpr int kQ = BQ / WQ / 16, kP = BP / WP / 16, kC = kP / kParts;
  using QTile = RowTile<BQ, kWaves>;
  using PTile = RowTile<kCols, kWaves>;
  using QScale = ScaleTile<BQ, kWaves, G, ALIGNED>;
  using PScale = ScaleTile<kCols, kWaves, G, ALIGNED>;
  static constexpr int kStage = QTile::kBytes + kParts * PTile::kBytes;
  static constexpr int kGroup = QScale::kBytes + kParts * PScale::kBytes;
  static constexpr int kLoads = QTile::kLoads + kParts * PTile::kLoads;  // of codes
  static constexpr int kLds = STAGES * kStage + 2 * kGroup;
  static_assert(BQ * kCols * 2 <= kLds, "the output tile fits where the stages were");
  static_assert(G >= 2, "a group's loads are waited for at a meeting before it is read");
};

template <bool GATED, bool ALIGNED, int BQ, int BP, int WQ, int WP, int STAGES, int G>
__global__ __launch_bounds__(WQ* WP * 64, 2) void linear_rows4_kernel(MxLinearArgs a) {
  using T = Rows4<GATED, ALIGNED, BQ, BP, WQ, WP, STAGES, G>;
  constexpr int kQ = T::kQ, kP = T::kP, kC = T::kC, kParts = T::kParts, kCols = T::kCols;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wq = wave / WP, wp = wave % WP;
  const Item it = find_item(a, row::block_index(), BQ, (a.N + kCols - 1) / kCols);
  if (it.e < 0) return;
  const int ld = a.K / 2, S = a.K / mx::kBlock;
  const int q0 = it.tq * BQ, p0 = it.tp * kCols;
  const int live = min(BQ, it.count - q0);  // rows of this tile
  const int64_t first = (int64_t)it.row0 + q0, wfirst = (int64_t)it.e * a.N + p0;
  const int wlive = min(kCols, a.N - p0);
  const __amdgpu_buffer_rsrc_t rx = resource(static_cast<const char*>(a.x) + first * ld);
  // the scales' resources begin at the aligned dword that holds the tile's first byte
  const uint8_t* const xs = a.xs + first * S;
  const int xlead = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(xs) & 3);
  const __amdgpu_buffer_rsrc_t rxs = resource(xs - xlead);
  __amdgpu_buffer_rsrc_t rw[kParts], rws[kParts];
  int wlead[kParts];
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    rw[h] = resource(static_cast<const char*>(a.w[h]) + wfirst * ld);
    const uint8_t* const ws = a.wsb[h] + wfirst * S;
    wlead[h] = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(ws) & 3);
    rws[h] = resource(ws - wlead[h]);
  }
  typename T::QTile qt;
  typename T::PTile pt;
  typename T::QScale qs;
  typename T::PScale ps[kParts];
  qt.init(wave, lane, [&](int r) { return r < live ? (uint32_t)(r * ld) : kNoFetch; });
  pt.init(wave, lane, [&](int r) { return r < wlive ? (uint32_t)(r * ld) : kNoFetch; });
  qs.init(wave, lane, xlead, S, [&](int r) { return r < live ? r : -1; });
#pragma unroll
  for (int h = 0; h < kParts; ++h) ps[h].init(wave, lane, wlead[h], S, [&](int r) { return r < wlive ? r : -1; });
  const int steps = (ld + kDB - 1) / kDB;
  char* const groups = smem + STAGES * T::kStage;
  // past the last step nothing is left: the loads are issued and fetch nothing
  auto issue_scales = [&](int g) {
    char* b = groups + (g & 1) * T::kGroup;
    qs.load(rxs, b, wave, lane, g);
#pragma unroll
    for (int h = 0; h < kParts; ++h) ps[h].load(rws[h], b + T::QScale::kBytes + h * T::PScale::kBytes, wave, lane, g);
  };
  auto issue = [&](int s, int stage) {
    char* b = smem + stage * T::kStage;
    qt.load(rx, b, wave, s * kDB, ld - s * kDB);
#pragma unroll
    for (int h = 0; h < kParts; ++h)
      pt.load(rw[h], b + T::QTile::kBytes + h * T::PTile::kBytes, wave, s * kDB, ld - s * kDB);
  };
  f32x4 acc[kQ][kP];
#pragma unroll
  for (int i = 0; i < kQ; ++i)
#pragma unroll
    for (int j = 0; j < kP; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  issue_scales(0);
#pragma unroll
  for (int s = 0; s < STAGES; ++s) issue(s, s);

  // A step is 2 L units: row subtile u % L times all column subtiles, first of the stage's
  // lower halves, then of the upper ones.  A unit's rows are read kAhead units before it,
  // into a ring of as many and one, the columns' other half beside the first unit; once the
  // last rows are read the waves meet, the stage is filled again, and the rest of the units
  // run beside the first reads of the next stage.
  auto multiply = [&](auto live_subtiles) {
    constexpr int L = decltype(live_subtiles)::value, kUnits = 2 * L;
    constexpr int kRing = L >= 4 ? 4 : L == 3 ? 3 : 2, kAhead = kRing - 1, kMeet = kUnits - kAhead;
    static_assert(kUnits % kRing == 0 && kMeet >= L, "units keep their places; the lower halves are done at the meeting");
    int stage = 0;
    u32x4 q[kRing], p[2][kP];
    // scales of this step and of the next, those of two subtiles in a register
    constexpr int kSq = (L + 1) / 2, kSp = (kP + 1) / 2;
    uint32_t sq[kSq], sp[kSp], nq[kSq], np[kSp];
    // Lane l reads the pieces 2 (l / 16) + k of line l % 16 of a subtile; a line's swizzle
    // repeats every 16 lines, so one offset a half serves all subtiles.  (As a vector, not a
    // uint4: of a struct the compiler loses the type, takes the read to depend on every
    // direct load and waits for the one just issued.)
    int at[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) at[k] = (lane & 15) * kDB + ((2 * (lane >> 4) + k) ^ T::QTile::swz(lane & 15)) * 16;
    const int sx_at = T::QScale::lane_at(lane, xlead, S) + wq * 16 * T::QScale::kRow;
    int sw_at[kParts];
#pragma unroll
    for (int h = 0; h < kParts; ++h)
      sw_at[h] = T::PScale::lane_at(lane, wlead[h], S) + wp * (kCols / WP) * T::PScale::kRow + T::QScale::kBytes + h * T::PScale::kBytes;
    auto read_q = [&](int u) {
      const char* b = smem + stage * T::kStage + wq * 16 * kDB + at[u / L];
      q[u % kRing] = *reinterpret_cast<const u32x4*>(b + u % L * WQ * 16 * kDB);
    };
    auto read_p = [&](int k) {
      const char* b = smem + stage * T::kStage + T::QTile::kBytes + wp * (kCols / WP) * kDB + at[k];
#pragma unroll
      for (int j = 0; j < kP; ++j) p[k][j] = *reinterpret_cast<const u32x4*>(b + j / kC * T::PTile::kBytes + j % kC * 16 * kDB);
    };
    auto read_scales = [&](int s) {
      const char* b = groups + (s / G & 1) * T::kGroup + s % G * 8;
      const int left = S - s * 8 - 2 * (lane >> 4);
      auto of_q = [&](int i) { return T::QScale::pair(b + sx_at + i * WQ * 16 * T::QScale::kRow, left); };
      auto of_p = [&](int j) { return T::PScale::pair(b + sw_at[j / kC] + j % kC * 16 * T::PScale::kRow, left); };
#pragma unroll
      for (int i = 0; i < kSq; ++i) nq[i] = of_q(2 * i) | (2 * i + 1 < L ? of_q(2 * i + 1) << 16 : 0u);
#pragma unroll
      for (int j = 0; j < kSp; ++j) np[j] = of_p(2 * j) | (2 * j + 1 < kP ? of_p(2 * j + 1) << 16 : 0u);
    };
    auto unit = [&](auto index) {
      constexpr int u = decltype(index)::value, i = u % L, H = u / L, O = H + 2 * (i & 1);
#pragma unroll
      for (int j = 0; j < kP; ++j)
        acc[i][j] = j & 1 ? mx::mfma<H + 2, O>(p[H][j], sp[j / 2], q[u % kRing], sq[i / 2], acc[i][j])
                          : mx::mfma<H, O>(p[H][j], sp[j / 2], q[u % kRing], sq[i / 2], acc[i][j]);
    };
    wait_and_meet<(STAGES - 1) * T::kLoads>();
    read_p(0);
    read_scales(0);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) read_q(u);
    for (int s = 0; s < steps; ++s) {
      // the next group: the last bytes of the one before this, whose place it takes, were
      // read before the meeting of step s - 1 (a branch behind the meeting would draw the
      // products in front of it into its far side)
      if (s % G == 0) issue_scales(s / G + 1);
#pragma unroll
      for (int i = 0; i < kSq; ++i) sq[i] = nq[i];
#pragma unroll
      for (int j = 0; j < kSp; ++j) sp[j] = np[j];
      each<kUnits>([&](auto index) {
        constexpr int u = decltype(index)::value;
        if constexpr (u == kMeet) {
          wait_and_meet<(STAGES - 2) * T::kLoads>();  // this step's operands are in registers, the next stage has landed
          issue(s + STAGES, stage);
          stage = stage == STAGES - 1 ? 0 : stage + 1;
          read_p(0);  // of step s + 1; past the last one whatever lies there, unused
          read_scales(s + 1);
        }
        read_q(u < kMeet ? u + kAhead : u - kMeet);
        if constexpr (u == 0) read_p(1);
        __builtin_amdgcn_sched_barrier(0);  // the reads are on their way before the products
        unit(index);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  };
  by_live_subtiles<kQ>((live - wq * 16 + 16 * WQ - 1) / (16 * WQ), multiply);
  wait_and_meet<0>();  // the loads past the last step have landed: LDS is free
  finish<GATED, BQ, kCols, WQ, WP, kQ, kC>(a, it.e, first, live, p0, wq, wp, acc);
}

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
        for (int h = 0; h < kParts; ++h) acc[h] = mx::mfma<0, 0>(as_vec(wv[h]), wb[h], as_vec(xv), xb, acc[h]);
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
#define MOE_MX_ROWS4(G, A)                                                    \
  template __global__ void linear_rows4_kernel<G, A, 256, 256, 2, 4, 2, 2>(MxLinearArgs); \
  template __global__ void linear_rows4_kernel<G, A, 128, 128, 2, 2, 2, 4>(MxLinearArgs); \
  template __global__ void linear_rows4_kernel<G, A, 64, 64, G ? 4 : 2, G ? 1 : 2, 3, 4>(MxLinearArgs);
MOE_MX_ROWS4(false, false)
MOE_MX_ROWS4(false, true)
MOE_MX_ROWS4(true, false)
MOE_MX_ROWS4(true, true)
#undef MOE_MX_ROWS4
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

template <bool GATED, bool ALIGNED, int BQ, int BP, int WQ, int WP, int STAGES, int G>
hipError_t run_rows4(const MxLinearArgs& a, hipStream_t s) {
  using T = Rows4<GATED, ALIGNED, BQ, BP, WQ, WP, STAGES, G>;
  static std::atomic<size_t> allowed[kMaxCachedDevices];
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, BQ) * ((a.N + T::kCols - 1) / T::kCols);
  void (*const kern)(MxLinearArgs) = &linear_rows4_kernel<GATED, ALIGNED, BQ, BP, WQ, WP, STAGES, G>;
  return launch(kern, items, T::kThreads, T::kLds, a, s, allowed);
}

// Rows per expert on average, of the matrix's height, in which the alignment's padding
// counts: the runs themselves are known on the device only.
int64_t mean_rows(const MxLinearArgs& a) { return ceil_div(a.rows, a.E); }

// Square tiles of `edge` that the rows and `cols` columns make.
int64_t tiles(const MxLinearArgs& a, int64_t cols, int64_t edge) {
  return (a.rows + edge - 1) / edge * ((cols + edge - 1) / edge);
}

bool wide_tiles(const MxLinearArgs& a, int64_t cols) { return tiles(a, cols, 256) >= 256 && mean_rows(a) >= 160; }

// Rows per expert up to which the depth-split kernel is taken.
constexpr int64_t kFewRows = 32;

template <bool GATED, bool ALIGNED>
hipError_t rows4_by_shape(const MxLinearArgs& a, hipStream_t s) {
  if (mean_rows(a) <= kFewRows) return run_few<true, GATED, 2, 8>(a, s);
  const int64_t cols = a.parts * (int64_t)a.N;
  if (tiles(a, cols, 128) < 256) return run_rows4<GATED, ALIGNED, 64, 64, GATED ? 4 : 2, GATED ? 1 : 2, 3, 4>(a, s);
  if (wide_tiles(a, cols)) return run_rows4<GATED, ALIGNED, 256, 256, 2, 4, 2, 2>(a, s);
  return run_rows4<GATED, ALIGNED, 128, 128, 2, 2, 2, 4>(a, s);
}

template <int BQ, int BP, int WQ, int WP>
hipError_t run_backward_x(const MxLinearArgs& a, hipStream_t s) {
  static std::atomic<size_t> allowed[kMaxCachedDevices];
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, BQ) * ((a.K + BP - 1) / BP);
  return launch(&linear_mx_backward_x_kernel<BQ, BP, WQ, WP>, items, WQ * WP * 64, (3 * BQ + 2 * BP) * 128, a, s, allowed);
}

}  // namespace

hipError_t launch_linear_mx(const MxLinearArgs& a, hipStream_t s) {
  if (a.xs != nullptr) {
    const uintptr_t lead = reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.wsb[0]) | reinterpret_cast<uintptr_t>(a.wsb[1]);
    if (a.K % 128 == 0 && lead % 4 == 0) return a.parts == 2 ? rows4_by_shape<true, true>(a, s) : rows4_by_shape<false, true>(a, s);
    return a.parts == 2 ? rows4_by_shape<true, false>(a, s) : rows4_by_shape<false, false>(a, s);
  }
  return a.parts == 2 ? run_few<false, true, 2, 8>(a, s) : run_few<false, false, 2, 8>(a, s);
}

hipError_t launch_linear_mx_backward_x(const MxLinearArgs& a, hipStream_t s) { return run_backward_x<128, 128, 2, 2>(a, s); }

}  // namespace moe
