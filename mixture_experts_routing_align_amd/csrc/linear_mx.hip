// The experts' matrix products on MXFP4 weights over sorted rows for gfx950: forward with
// bias, activation, residual and MXFP4 rows in the epilogue, and the rows' gradient.
//
//   forward      z[p] = W[e] x[p] + b[e], y[p] = act(z[p]) + residual[p]
//   backward x   dx[p] = sum_n dz[p, n] W[e][n, :]
//
// A weight is its E2M1 code times its block's scale.  With MXFP4 rows the products are the
// matrix cores' own 4-bit ones (mx_common.h); with bf16 rows the codes are widened to bf16
// with their scale, which is exact, so sums are float32 either way.
//
// Three kinds of products share one driver (linear_mx_kernel), in tiles staged in LDS by
// direct loads: Rows4, Rows16 and Back16.  A few rows take linear_mx_few_kernel.  32768 rows
// over 128 experts, 2 x 768 x 2048, SwiGLU, runs of uneven length, against the bytes at a
// large copy's 4.9 TB/s or the operations at a large bf16 product's 1.43 PFLOP/s:
//   bf16 rows, pre-activations kept     230 us, floor 144 (operations); matrix cores busy 44%
//   MXFP4 rows                          110 us, floor  61 (bytes); 23%
//   the gradient of the bf16 rows       264 us, floor 144 (operations); 36%
// Equal runs with one expert's weights take 181, 71 and 189 us: the rest is partly filled
// tiles and weights that come from HBM.  MXFP4 rows, dense, 8192 x 2048 x 7168, bias and
// residual: 76 us, 3.2 PFLOP/s; 62 without the residual, whose rows are read one subtile
// ahead after the last product while the compute unit has nothing else to do (7 us of bytes
// for 15).  Ablations in copies (80 us then): without the loads of its loop 64, without its
// products 60, also without the reads of scales and weights from LDS 57, the reads of rows
// still in.  So the loads are hidden but for a fifth, and more than half of the rest is reads
// of rows, the products' issue, and a tile's start and end.  A tile has its compute unit
// alone, and its two stages leave one step's time for the next one's loads; three stages need
// smaller tiles, which load more (256 x 128 and 128 x 256: 88 us), and lines touched ahead of
// their loads cost what they hide (82 us).  8 tokens top-8 in 16-row runs, 54 of 128 experts:
// 29 us, floor 19 (bytes), MXFP4 rows 19: what the bf16 rows lack is not the weights' rate but
// longer steps, 32 meetings of 64 deep for 8 of 256, and weights that have to land a step
// after they are asked for.

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "linear_epilogue.h"
#include "linear_tile.h"
#include "moe_internal.h"
#include "moe_mi355x_ops.h"
#include "mx_common.h"
#include "mx_forms.h"
#include "row_common.h"

namespace moe {
namespace {

using namespace tile;
using namespace epilogue;
using mx::Form;

extern __shared__ __attribute__((aligned(1024))) char smem[];

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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
//
// The dwords are dealt to the waves 64 at a time; no lane is left out of a load, since a load
// behind a branch that lanes take differently may be merged with another one's, whose place
// in LDS is then taken for both.
template <int R, int WAVES, int G, bool ALIGNED>
struct ScaleTile {
  static constexpr int kWords = 2 * G + (ALIGNED ? 0 : 1);  // dwords of LDS a row
  static constexpr int kPieces = (R * kWords + 63) / 64;    // loads of a wave in all
  static constexpr int kBytes = kPieces * 256;
  static constexpr int kLoads = (kPieces + WAVES - 1) / WAVES;
  uint32_t off[kLoads];  // byte offset of each of this lane's dwords in group 0, or kNoFetch
  int end[kLoads];       // bytes from there to the end of its row

  // `lead`: bytes from the resource's (aligned) base to row 0; `row_of(r)`: the row of the
  // array that operand row r is, or -1; `S` bytes a row.
  template <typename F>
  __device__ __forceinline__ void init(int wave, int lane, int lead, int S, F row_of) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int d = (i * WAVES + wave) * 64 + lane, r = d < R * kWords ? row_of(d / kWords) : -1, w = d % kWords;
      const int begin = lead + r * S, at = (begin & ~3) + w * 4;
      off[i] = r < 0 ? kNoFetch : (uint32_t)at;
      end[i] = begin + S - at;
    }
  }
  // Fills `lds` with the bytes of group g.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, char* lds, int wave, int g) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if ((i + 1) * WAVES <= kPieces || i * WAVES + wave < kPieces)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (i * WAVES + wave) * 256), 4,
                                                 g * G * 8 < end[i] ? off[i] : kNoFetch, g * G * 8, 0, 0);
  }
  // Where lane l finds the bytes of blocks 2 q and 2 q + 1 (q = l / 16) of operand row l % 16
  // in step 0 of a group; the same for row r0 + l % 16, r0 a multiple of 16, r0 kRow on.
  static constexpr int kRow = kWords * 4;
  __device__ static __forceinline__ int lane_at(int lane, int lead, int S) { return row_at(lane, lead, S) + (lane >> 4) * 2; }
  // And the row's first byte.
  __device__ static __forceinline__ int row_at(int lane, int lead, int S) {
    const int r = lane & 15;
    return r * kRow + (ALIGNED ? 0 : (lead + r * S) & 3);
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

// What a tile of the forward products is made of: BQ rows by BP weight rows (SwiGLU: BP / 2
// of the gate and the same BP / 2 of the up weight, so that a lane holds z and u of its
// elements), WQ x WP waves.
template <bool GATED, int BQ_, int BP, int WQ_, int WP_>
struct Shape {
  static constexpr bool kGated = GATED;
  static constexpr int BQ = BQ_, WQ = WQ_, WP = WP_;
  static constexpr int kWaves = WQ * WP, kThreads = kWaves * 64;
  static constexpr int kParts = GATED ? 2 : 1;
  static constexpr int kCols = BP / kParts;                // output columns of a tile
  static constexpr int kWaveCols = kCols / WP;             // and of a wave
  static constexpr int kQ = BQ / WQ / 16, kP = BP / WP / 16, kC = kP / kParts;
  static_assert(kC % 2 == 0, "a wave holds whole scale blocks of its rows' columns");
  // Columns of the result.
  __device__ static __forceinline__ int width(const MxLinearArgs& a) { return a.N; }
};

// 16 rows of BYTES that a wave gathers in LDS to store them as lines.  Pieces of 16 bytes
// are swizzled by which 256 bytes of LDS (all banks) their row lies in, so that 16 rows'
// same piece spreads over them.
template <int BYTES>
struct WaveRows {
  static constexpr int kPieces = BYTES / 16;
  __device__ static __forceinline__ int swz(int r) { return (r * BYTES / 256) & (kPieces - 1); }
  template <typename V>
  __device__ static __forceinline__ void put(char* lds, int r, int byte, V v) {
    *reinterpret_cast<V*>(lds + r * BYTES + (((byte >> 4) ^ swz(r)) << 4) + (byte & 15)) = v;
  }
  // The rows below `live`, their first `valid` bytes (a multiple of 16), to dst; ld bytes from
  // row to row.
  __device__ static __forceinline__ void flush(const char* lds, char* dst, int64_t ld, int live, int valid) {
    const int lane = threadIdx.x & 63;
    asm volatile("" ::: "memory");  // a wave's LDS operations are done in order
#pragma unroll
    for (int i = 0; i < 16 * kPieces; i += 64) {
      const int r = (i + lane) / kPieces, g = (i + lane) % kPieces;
      if (r < min(live, 16) && g * 16 < valid)
        *reinterpret_cast<u32x4*>(dst + r * ld + g * 16) = *reinterpret_cast<const u32x4*>(lds + r * BYTES + ((g ^ swz(r)) << 4));
    }
    asm volatile("" ::: "memory");
  }
};

// The end of a tile: bias, activation and residual on the float32 sums, pre-activations,
// bf16 or MXFP4 rows.  Lane l holds row l % 16 and 4 consecutive columns of each subtile,
// acc[i][j] of a wave's row subtiles i and its columns' subtiles j (SwiGLU: kC of z, then kC
// of u).  Every wave turns its own 16 rows at a time into lines in LDS of its own, so that
// no wave waits for another here and the next tile's operands may be on their way.  The
// bias and the first rows' residual are loaded in front of those (loads come back in
// order), the other rows' ahead of the rows before them.
template <class T>
struct Finish {
  int e, live, p0;
  int64_t first;
  uint2 bias[T::kParts][T::kC], residual[2][T::kC];

  // Column subtile j's first column of this lane.
  __device__ __forceinline__ int column(int wave, int j) const {
    return p0 + wave % T::WP * T::kWaveCols + j * 16 + (int)(threadIdx.x & 63) / 16 * 4;
  }
  __device__ __forceinline__ void load_residual(const MxLinearArgs& a, int wave, int i) {
    const int m = q_row<T::WQ>(wave / T::WP, i) + (int)(threadIdx.x & 15);
#pragma unroll
    for (int j = 0; j < T::kC; ++j) {
      const int n = column(wave, j);
      residual[i & 1][j] = make_uint2(0, 0);
      if (m < live && n < T::width(a)) residual[i & 1][j] = *reinterpret_cast<const uint2*>(a.residual + (first + m) * T::width(a) + n);
    }
  }
  __device__ __forceinline__ void load(const MxLinearArgs& a, int wave) {
#pragma unroll
    for (int h = 0; h < T::kParts; ++h)
#pragma unroll
      for (int j = 0; j < T::kC; ++j) {
        const int n = column(wave, j);
        bias[h][j] = make_uint2(0, 0);
        if (a.bias[h] != nullptr && n < a.N) bias[h][j] = *reinterpret_cast<const uint2*>(a.bias[h] + (int64_t)e * a.N + n);
      }
    if (a.residual != nullptr) load_residual(a, wave, 0);
  }
  __device__ __forceinline__ void store(const MxLinearArgs& a, int wave, char* lds, f32x4 (&acc)[T::kQ][T::kP]);
};

template <class T>
__device__ __forceinline__ void Finish<T>::store(const MxLinearArgs& a, int wave, char* lds, f32x4 (&acc)[T::kQ][T::kP]) {
  constexpr int kC = T::kC;
  const int N = T::width(a);
  const int wq = wave / T::WP, wp = wave % T::WP;
  const int lane = threadIdx.x & 63, quad = lane >> 4, row16 = lane & 15;
  constexpr int kO = T::kOutCols / 16;  // column subtiles gathered at a time
  using Rows = WaveRows<T::kOutCols * 2>;
  using Codes = WaveRows<T::kOutCols / 2>;
#pragma unroll
  for (int i = 0; i < T::kQ; ++i) {
    const int left = live - q_row<T::WQ>(wq, i);
    if (left <= 0) break;
    if (a.residual != nullptr && i + 1 < T::kQ) load_residual(a, wave, i + 1);
    const int64_t r0 = first + q_row<T::WQ>(wq, i);
#pragma unroll
    for (int j0 = 0; j0 < kC; j0 += kO) {
      const int n0 = p0 + wp * T::kWaveCols + j0 * 16, cols = min(T::kOutCols, N - n0);
      if (cols <= 0) break;
      float y[kO][4], u[kO][4];
#pragma unroll
      for (int j = 0; j < kO; ++j) {
        const int n = j * 16 + quad * 4;
        float z[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          z[c] = acc[i][j0 + j][c];
          u[j][c] = acc[i][(T::kGated ? kC : 0) + j0 + j][c];
        }
        add4(z, bias[0][j0 + j]);
        if constexpr (T::kGated) add4(u[j], bias[1][j0 + j]);
        act4<T::kGated, true>(a.act, z, u[j], y[j]);
        if (a.residual != nullptr) add4(y[j], residual[i & 1][j0 + j]);
        if (a.preact != nullptr) Rows::put(lds, row16, n * 2, pack4(z));
      }
      if (a.preact != nullptr) {
        char* pre = reinterpret_cast<char*>(a.preact + r0 * T::kParts * N + n0);
        Rows::flush(lds, pre, (int64_t)T::kParts * N * 2, left, cols * 2);
        if constexpr (T::kGated) {
#pragma unroll
          for (int j = 0; j < kO; ++j) Rows::put(lds, row16, (j * 16 + quad * 4) * 2, pack4(u[j]));
          Rows::flush(lds, pre + (int64_t)N * 2, (int64_t)2 * N * 2, left, cols * 2);
        }
      }
      if (a.ysb == nullptr) {
#pragma unroll
        for (int j = 0; j < kO; ++j) Rows::put(lds, row16, (j * 16 + quad * 4) * 2, pack4(y[j]));
        Rows::flush(lds, reinterpret_cast<char*>(static_cast<uint16_t*>(a.y) + r0 * N + n0), (int64_t)N * 2, left,
                                 cols * 2);
        continue;
      }
      // a scale block is two subtiles over the four quads
#pragma unroll
      for (int j = 0; j < kO; j += 2) {
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) mx = max(mx, max(row::abs_bits(y[j][c]), row::abs_bits(y[j + 1][c])));
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16));
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32));
        const uint32_t byte = mx::scale_byte(mx);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          Codes::put(lds, row16, ((j + h) * 16 + quad * 4) / 2, (uint16_t)mx::codes4(y[j + h][0], y[j + h][1], y[j + h][2], y[j + h][3], byte));
        if (quad == 0 && row16 < left && j * 16 < cols)
          a.ysb[(r0 + row16) * (N / mx::kBlock) + (n0 + j * 16) / mx::kBlock] = (uint8_t)byte;
      }
      Codes::flush(lds, static_cast<char*>(a.y) + (r0 * N + n0) / 2, N / 2, left, cols / 2);
    }
  }
}

// Lane l's 16-byte piece 2 (l / 16) + k of line l % 16 of a subtile of RowTile lines, k = 0
// and 1: a line's swizzle repeats every 16 lines, so the offset serves all subtiles.
__device__ __forceinline__ int piece_at(int lane, int k) {
  return (lane & 15) * kDB + ((2 * (lane >> 4) + k) ^ RowTile<16, 1, true>::swz(lane & 15)) * 16;
}

// How a wave's products of one step run: 2 L units, row subtile u % L times all its column
// subtiles, with the lower half of the operands' depth first and then the upper one.  A
// unit's rows are read kAhead units before it into a ring of one more; once the last rows
// are read the waves meet, the step's stage is filled again, and the rest of the units run
// beside the first reads of the next step.
template <int L>
struct Units {
  static constexpr int kCount = 2 * L;
  static constexpr int kRing = L >= 4 ? 4 : L == 3 ? 3 : 2, kAhead = kRing - 1, kMeet = kCount - kAhead;
  static_assert(kCount % kRing == 0 && kMeet >= L, "units keep their places; the lower halves are done at the meeting");
};

// MXFP4 rows: STAGES stages of 256 depth elements, 128 bytes of codes a row, and two groups
// of G steps' scale bytes.  Lane l takes blocks 2 (l / 16) and 2 (l / 16) + 1 of a stage, one
// for each half of its products.  LDS cycles of 32768 rows (see the top): 10.7M, 17.7M before
// the lines' swizzle was made for pairs of pieces.
template <class T, bool ALIGNED, int STAGES, int G>
struct Rows4 : T {
  // columns of its 16 rows a wave gathers in LDS at a time: all of them where there is room
  static constexpr int kOutCols = ALIGNED ? T::kWaveCols : 32;
  using T::kP;
  using T::kParts;
  using QTile = RowTile<T::BQ, T::kWaves, true>;
  using PTile = RowTile<T::kCols, T::kWaves, true>;
  using QScale = ScaleTile<T::BQ, T::kWaves, G, ALIGNED>;
  using PScale = ScaleTile<T::kCols, T::kWaves, G, ALIGNED>;
  static constexpr int kStage = QTile::kBytes + kParts * PTile::kBytes;
  static constexpr int kGroup = QScale::kBytes + kParts * PScale::kBytes;
  static constexpr int kLoads = QTile::kLoads + kParts * PTile::kLoads;  // of a stage's codes
  static constexpr int kLds = STAGES * kStage + 2 * kGroup;
  static_assert(G >= 2, "a group's loads are waited for at a meeting before it is read");

  __amdgpu_buffer_rsrc_t rx, rxs, rw[kParts], rws[kParts];
  int xlead, wlead[kParts], ld, S, steps;
  QTile qt;
  PTile pt;
  QScale qs;
  PScale ps[kParts];

  // The tile of expert e with rows `first` ... + live - 1 and the columns from p0 on.
  __device__ __forceinline__ void setup(const MxLinearArgs& a, int e, int64_t first, int live, int p0, int wave, int lane) {
    const int64_t wfirst = (int64_t)e * a.N + p0;
    const int wlive = min(T::kCols, a.N - p0);
    ld = a.K / 2;
    S = a.K / mx::kBlock;
    steps = (ld + kDB - 1) / kDB;
    rx = resource(static_cast<const char*>(a.x) + first * ld);
    // the scales' resources begin at the aligned dword that holds the tile's first byte
    const uint8_t* const xs = a.xs + first * S;
    xlead = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(xs) & 3);
    rxs = resource(xs - xlead);
    auto row = [](int l) { return [l](int r) { return r < l ? r : -1; }; };
    auto off = [this](int l) { return [l, this](int r) { return r < l ? (uint32_t)(r * ld) : kNoFetch; }; };
    qt.init(wave, lane, off(live));
    qs.init(wave, lane, xlead, S, row(live));
    pt.init(wave, lane, off(wlive));
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      rw[h] = resource(static_cast<const char*>(a.w[h]) + wfirst * ld);
      const uint8_t* const ws = a.wsb[h] + wfirst * S;
      wlead[h] = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(ws) & 3);
      rws[h] = resource(ws - wlead[h]);
      ps[h].init(wave, lane, wlead[h], S, row(wlive));
    }
  }
  __device__ __forceinline__ char* group(int g) const { return smem + STAGES * kStage + (g & 1) * kGroup; }
  __device__ __forceinline__ void issue_scales(int g, int wave) const {
    qs.load(rxs, group(g), wave, g);
#pragma unroll
    for (int h = 0; h < kParts; ++h) ps[h].load(rws[h], group(g) + QScale::kBytes + h * PScale::kBytes, wave, g);
  }
  // past the last step nothing is left: the loads are issued and fetch nothing
  __device__ __forceinline__ void issue(int s, int stage, int wave) const {
    char* b = smem + stage * kStage;
    qt.load(rx, b, wave, s * kDB, ld - s * kDB);
#pragma unroll
    for (int h = 0; h < kParts; ++h) pt.load(rw[h], b + QTile::kBytes + h * PTile::kBytes, wave, s * kDB, ld - s * kDB);
  }
  __device__ __forceinline__ void start(int wave) const {
    issue_scales(0, wave);
#pragma unroll
    for (int s = 0; s < STAGES; ++s) issue(s, s, wave);
  }
  // The tile's products, the first L row subtiles of a wave's.
  template <int L>
  __device__ __forceinline__ void multiply(int wave, int lane, f32x4 (&acc)[T::kQ][kP]) const {
    using U = Units<L>;
    constexpr int kC = T::kC, kSq = (L + 1) / 2, kSp = (kP + 1) / 2;
    const int wq = wave / T::WP, wp = wave % T::WP;
    int stage = 0;
    u32x4 q[U::kRing], p[2][kP];
    uint32_t sq[kSq], sp[kSp], nq[kSq], np[kSp];  // scales of this step and of the next, two subtiles' in a register
    // (Reads are of a vector, not of a uint4: of a struct the compiler loses the type, takes
    // the read to depend on every direct load and waits for the one just issued.)
    const int at[2] = {piece_at(lane, 0), piece_at(lane, 1)};
    const int sx_at = QScale::lane_at(lane, xlead, S) + wq * 16 * QScale::kRow;
    int sw_at[kParts];
#pragma unroll
    for (int h = 0; h < kParts; ++h)
      sw_at[h] = PScale::lane_at(lane, wlead[h], S) + wp * T::kWaveCols * PScale::kRow + QScale::kBytes + h * PScale::kBytes;
    auto read_q = [&](int u) {
      const char* b = smem + stage * kStage + wq * 16 * kDB + at[u / L];
      q[u % U::kRing] = *reinterpret_cast<const u32x4*>(b + u % L * T::WQ * 16 * kDB);
    };
    auto read_p = [&](int k) {
      const char* b = smem + stage * kStage + QTile::kBytes + wp * T::kWaveCols * kDB + at[k];
#pragma unroll
      for (int j = 0; j < kP; ++j) p[k][j] = *reinterpret_cast<const u32x4*>(b + j / kC * PTile::kBytes + j % kC * 16 * kDB);
    };
    auto read_scales = [&](int s) {
      const char* b = group(s / G) + s % G * 8;
      const int left = S - s * 8 - 2 * (lane >> 4);
      auto of_q = [&](int i) { return QScale::pair(b + sx_at + i * T::WQ * 16 * QScale::kRow, left); };
      auto of_p = [&](int j) { return PScale::pair(b + sw_at[j / kC] + j % kC * 16 * PScale::kRow, left); };
#pragma unroll
      for (int i = 0; i < kSq; ++i) nq[i] = of_q(2 * i) | (2 * i + 1 < L ? of_q(2 * i + 1) << 16 : 0u);
#pragma unroll
      for (int j = 0; j < kSp; ++j) np[j] = of_p(2 * j) | (2 * j + 1 < kP ? of_p(2 * j + 1) << 16 : 0u);
    };
    auto unit = [&](auto index) {
      constexpr int u = decltype(index)::value, i = u % L, H = u / L, O = H + 2 * (i & 1);
#pragma unroll
      for (int j = 0; j < kP; ++j)
        acc[i][j] = j & 1 ? mx::mfma<H + 2, O>(p[H][j], sp[j / 2], q[u % U::kRing], sq[i / 2], acc[i][j])
                          : mx::mfma<H, O>(p[H][j], sp[j / 2], q[u % U::kRing], sq[i / 2], acc[i][j]);
    };
    wait_and_meet<(STAGES - 1) * kLoads>();
    read_p(0);
    read_scales(0);
#pragma unroll
    for (int u = 0; u < U::kAhead; ++u) read_q(u);
    for (int s = 0; s < steps; ++s) {
      // the next group: the last bytes of the one before this, whose place it takes, were
      // read before the meeting of step s - 1 (a branch behind the meeting would draw the
      // products in front of it into its far side)
      if (s % G == 0) issue_scales(s / G + 1, wave);
#pragma unroll
      for (int i = 0; i < kSq; ++i) sq[i] = nq[i];
#pragma unroll
      for (int j = 0; j < kSp; ++j) sp[j] = np[j];
      each<U::kCount>([&](auto index) {
        constexpr int u = decltype(index)::value;
        if constexpr (u == U::kMeet) {
          wait_and_meet<(STAGES - 2) * kLoads>();  // this step's operands are in registers, the next stage has landed
          issue(s + STAGES, stage, wave);
          stage = stage == STAGES - 1 ? 0 : stage + 1;
          read_p(0);  // of step s + 1; past the last one whatever lies there, unused
          read_scales(s + 1);
        }
        read_q(u < U::kMeet ? u + U::kAhead : u - U::kMeet);
        if constexpr (u == 0) read_p(1);
        __builtin_amdgcn_sched_barrier(0);  // the reads are on their way before the products
        unit(index);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  }
};

// bf16 rows: two or four stages of 64 depth elements, 128 bytes a row, beside two stages of 256 of
// the weights, 128 bytes of codes and 8 of scales a row, each for four steps.  Lane l takes
// the elements 16 (l / 16) ... + 15 of a step, which lie in one scale block, the first 8 in
// the lower half of its products; it reads their codes as 8 bytes and widens them with the
// scale as it goes, a half beside the products of the other.  LDS cycles of 32768 rows (see
// the top): 29.7M, 46.2M with a swizzle for single pieces (254 and 257 us).
template <class T, bool ALIGNED>
struct Rows16 : T {
  using T::kP;
  using T::kParts;
  using QTile = RowTile<T::BQ, T::kWaves, true>;
  using PTile = RowTile<T::kCols, T::kWaves, true>;
  using PScale = ScaleTile<T::kCols, T::kWaves, 1, ALIGNED>;
  static constexpr int kOutCols = T::kWaveCols;
  static constexpr int kPStage = kParts * (PTile::kBytes + PScale::kBytes);
  static constexpr int kPLoads = kParts * PTile::kLoads;  // of a stage's codes
  // Loads come back in order, so weights asked for have to land before rows asked for later
  // are used.  With four stages of rows that is as late as the weights are used themselves;
  // with two it is a step after they were asked for, which tiles of many rows spend
  // multiplying.  256 dense rows by 2048 x 2048 in 32 x 64 tiles: 13.8 us, 15.7 with two.
  // In 32 x 128 tiles four leave two workgroups a compute unit for three: 8 tokens top-8 over
  // 128 experts 34.8 us, 29.3 with two.
  static constexpr int kQStages = T::BQ <= 32 && kParts * T::kCols <= 64 ? 4 : 2;
  static constexpr int kLds = kQStages * QTile::kBytes + 2 * kPStage;

  __amdgpu_buffer_rsrc_t rx, rw[kParts], rws[kParts];
  int wlead[kParts], K, S, steps;
  QTile qt;
  PTile pt;
  PScale ps[kParts];

  __device__ __forceinline__ void setup(const MxLinearArgs& a, int e, int64_t first, int live, int p0, int wave, int lane) {
    const int64_t wfirst = (int64_t)e * a.N + p0;
    const int wlive = min(T::kCols, a.N - p0);
    K = a.K;
    S = K / mx::kBlock;
    steps = (K * 2 + kDB - 1) / kDB;
    rx = resource(static_cast<const char*>(a.x) + first * K * 2);
    qt.init(wave, lane, [&](int r) { return r < live ? (uint32_t)(r * K * 2) : kNoFetch; });
    pt.init(wave, lane, [&](int r) { return r < wlive ? (uint32_t)(r * (K / 2)) : kNoFetch; });
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      rw[h] = resource(static_cast<const char*>(a.w[h]) + wfirst * (K / 2));
      const uint8_t* const ws = a.wsb[h] + wfirst * S;
      wlead[h] = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(ws) & 3);
      rws[h] = resource(ws - wlead[h]);
      ps[h].init(wave, lane, wlead[h], S, [&](int r) { return r < wlive ? r : -1; });
    }
  }
  __device__ __forceinline__ char* weights(int m) const { return smem + kQStages * QTile::kBytes + (m & 1) * kPStage; }
  // past the last step nothing is left: the loads are issued and fetch nothing
  __device__ __forceinline__ void issue_q(int s, int wave) const {
    qt.load(rx, smem + (s & (kQStages - 1)) * QTile::kBytes, wave, s * kDB, K * 2 - s * kDB);
  }
  __device__ __forceinline__ void issue_p(int m, int wave) const {
    char* b = weights(m);
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      ps[h].load(rws[h], b + kParts * PTile::kBytes + h * PScale::kBytes, wave, m);
      pt.load(rw[h], b + h * PTile::kBytes, wave, m * kDB, K / 2 - m * kDB);
    }
  }
  __device__ __forceinline__ void start(int wave) const {
    issue_p(0, wave);
#pragma unroll
    for (int s = 0; s < kQStages; ++s) issue_q(s, wave);
  }
  // The tile's products, the first L row subtiles of a wave's.
  template <int L>
  __device__ __forceinline__ void multiply(int wave, int lane, f32x4 (&acc)[T::kQ][kP]) const {
    using U = Units<L>;
    constexpr int kC = T::kC;
    const int wq = wave / T::WP, wp = wave % T::WP, quad = lane >> 4;
    bf16x8 q[U::kRing], p[2][kP];
    u32x2 codes[kP];
    float scale[kP];
    const int at[2] = {piece_at(lane, 0), piece_at(lane, 1)};
    // 8 bytes of piece l / 32 of a line, in step 0 of a stage; a step later two pieces on
    const int code_at = (lane & 15) * kDB + ((quad >> 1) ^ PTile::swz(lane & 15)) * 16 + (quad & 1) * 8 + wp * T::kWaveCols * kDB;
    int scale_at[kParts];
#pragma unroll
    for (int h = 0; h < kParts; ++h)
      scale_at[h] = PScale::row_at(lane, wlead[h], S) + (quad >> 1) + wp * T::kWaveCols * PScale::kRow + kParts * PTile::kBytes + h * PScale::kBytes;
    auto read_q = [&](int s, int u) {
      const char* b = smem + (s & (kQStages - 1)) * QTile::kBytes + wq * 16 * kDB + at[u / L];
      q[u % U::kRing] = *reinterpret_cast<const bf16x8*>(b + u % L * T::WQ * 16 * kDB);
    };
    auto read_p = [&](int s) {
      const char* b = weights(s >> 2);
      const int c = code_at ^ (s & 3) << 5;
      const bool in = ALIGNED || (s * 2 + (quad >> 1)) < S;  // past the depth the codes are zeros, and the byte must not be a NaN's
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        codes[j] = *reinterpret_cast<const u32x2*>(b + c + j / kC * PTile::kBytes + j % kC * 16 * kDB);
        const uint32_t byte = *reinterpret_cast<const uint8_t*>(b + scale_at[j / kC] + (s & 3) * 2 + j % kC * 16 * PScale::kRow);
        scale[j] = mx::scale_bits(in ? byte : 0u);
      }
    };
    auto widen = [&](int k) {
#pragma unroll
      for (int j = 0; j < kP; ++j) p[k][j] = mma::fp4x8_to_bf16(codes[j][k], scale[j]);
    };
    wait_and_meet<(kQStages - 1) * QTile::kLoads>();
    read_p(0);
#pragma unroll
    for (int u = 0; u < U::kAhead; ++u) read_q(0, u);
    widen(0);
    for (int s = 0; s < steps; ++s) {
      // the next weights: those before this step's, whose place they take, were in registers
      // at the last meeting
      if ((s & 3) == 0) issue_p((s >> 2) + 1, wave);
      each<U::kCount>([&](auto index) {
        constexpr int u = decltype(index)::value;
        if constexpr (u == U::kMeet) {
          // this step's operands are in registers and the next one's have landed, behind which
          // there may be later rows and those weights on their way
          constexpr int kLater = (kQStages - 2) * QTile::kLoads;
          if ((s & 3) <= kQStages - 2)
            wait_and_meet<kLater + kPLoads>();
          else
            wait_and_meet<kLater>();
          issue_q(s + kQStages, wave);
          read_p(s + 1);
        }
        read_q(u < U::kMeet ? s : s + 1, u < U::kMeet ? u + U::kAhead : u - U::kMeet);
        __builtin_amdgcn_sched_barrier(0);  // the reads are on their way before the products
#pragma unroll
        for (int j = 0; j < kP; ++j) acc[u % L][j] = mma::mfma(p[u / L][j], q[u % U::kRing], acc[u % L][j]);
        if constexpr (u == 0) widen(1);
        if constexpr (u == U::kCount - 1) widen(0);  // of the next step
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  }
};

// Rows' gradient: BQ rows by BP columns of dx; the depth is the weight rows, gate's then
// up's, 64 a step, in two stages of either operand.  The weights lie across the depth, so
// they are transposed on their way from LDS to the registers as bf16 weights are: a thread
// takes the 16 bytes of one block of 32 columns of one weight row, a step ahead in
// registers, widens them with their scale and leaves them in LDS as bf16.
template <class T>
struct Back16 : T {
  using T::kP;
  static constexpr int kD = 64, BP = T::kCols;
  static constexpr int kOutCols = T::kWaveCols;
  static constexpr int kLineBlocks = BP / mx::kBlock;
  static constexpr int kPer = kD * kLineBlocks / T::kThreads;  // blocks of a stage a thread widens
  static_assert(kD * kLineBlocks % T::kThreads == 0, "whole blocks per thread");
  using QTile = RowTile<T::BQ, T::kWaves>;
  using PTile = DepthTile<BP, kD, T::kWaves>;
  static constexpr int kLds = 2 * QTile::kBytes + 2 * PTile::kBytes;
  __device__ static __forceinline__ int width(const MxLinearArgs& a) { return a.K; }

  __amdgpu_buffer_rsrc_t rq, rw[2], rws[2];
  int N, S, per, steps, b;  // b: this thread's block of columns
  QTile qt;
  u32x4 codes[kPer];
  uint32_t byte[kPer];

  __device__ __forceinline__ static int line(int i) { return (i * T::kThreads + (int)threadIdx.x) / kLineBlocks; }
  __device__ __forceinline__ static int block() { return (int)threadIdx.x % kLineBlocks; }

  __device__ __forceinline__ void setup(const MxLinearArgs& a, int e, int64_t first, int live, int p0, int wave, int lane) {
    const int ldq = a.parts * a.N * 2;
    N = a.N;
    S = a.K / mx::kBlock;
    per = (N + kD - 1) / kD;
    steps = per * a.parts;
    rq = resource(static_cast<const char*>(a.dz) + first * ldq);
    qt.init(wave, lane, [&](int r) { return r < live ? (uint32_t)(r * ldq) : kNoFetch; });
    b = p0 / mx::kBlock + block();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      rw[h] = resource(static_cast<const char*>(a.w[h < a.parts ? h : 0]) + (int64_t)e * N * S * 16);
      rws[h] = resource(a.wsb[h < a.parts ? h : 0] + (int64_t)e * N * S);
    }
  }
  // past the last step nothing is left: the loads are issued and fetch nothing
  __device__ __forceinline__ void issue_q(int s, int wave) const {
    const int h = s >= per ? 1 : 0, k = s - h * per;
    qt.load(rq, smem + (s & 1) * QTile::kBytes, wave, (h * N + k * kD) * 2, s < steps ? (N - k * kD) * 2 : 0);
  }
  static constexpr int kFetches = 2 * kPer;
  __device__ __forceinline__ void fetch(int s) {
    const int h = s >= per ? 1 : 0, k = s - h * per;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int n = k * kD + line(i);
      const uint32_t at = s < steps && n < N && b < S ? (uint32_t)(n * S + b) : kNoFetch;
      codes[i] = __builtin_amdgcn_raw_buffer_load_b128(h ? rw[1] : rw[0], at == kNoFetch ? kNoFetch : at * 16, 0, 0);
      byte[i] = __builtin_amdgcn_raw_buffer_load_b8(h ? rws[1] : rws[0], at, 0, 0);
    }
  }
  __device__ __forceinline__ char* weights(int s) const { return smem + 2 * QTile::kBytes + (s & 1) * PTile::kBytes; }
  // A block is two 32-byte segments of its line; of 16 lanes that write side by side, half
  // begin with the other 16 bytes of theirs, so that they reach all banks.
  __device__ __forceinline__ void widen(int s) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int d = line(i), g = block();
      const bool turn = kLineBlocks >= 8 ? g & 4 : d & 2;
      const float f = mx::scale_bits(byte[i]);
      char* const to = weights(s) + d * PTile::kLine;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<bf16x8*>(to + ((2 * g + k / 2) ^ PTile::swz(d)) * 32 + ((k ^ (turn ? 1 : 0)) & 1) * 16) =
            mma::fp4x8_to_bf16(turn ? codes[i][k ^ 1] : codes[i][k], f);
    }
  }
  __device__ __forceinline__ void start(int wave) {
    fetch(0);
    issue_q(0, wave);
    widen(0);
    fetch(1);
  }
  template <int L>
  __device__ __forceinline__ void multiply(int wave, int lane, f32x4 (&acc)[T::kQ][kP]) {
    using U = Units<L>;
    const int wq = wave / T::WP, wp = wave % T::WP;
    bf16x8 q[U::kRing], p[2][kP], upper[kP];
    const int at[2] = {(lane & 15) * kDB + ((lane >> 4) ^ QTile::swz(lane & 15)) * 16,
                       (lane & 15) * kDB + ((4 + (lane >> 4)) ^ QTile::swz(lane & 15)) * 16};
    auto read_q = [&](int s, int u) {
      const char* b = smem + (s & 1) * QTile::kBytes + wq * 16 * kDB + at[u / L];
      q[u % U::kRing] = *reinterpret_cast<const bf16x8*>(b + u % L * T::WQ * 16 * kDB);
    };
    // A transposing read waits for every direct load before it, needed or not (the compiler
    // takes it to depend on them), so both halves of a step's weights are read ahead of the
    // next rows' loads, the upper one into registers of its own.
    auto read_p = [&](int s) {
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        p[0][j] = PTile::frag(weights(s), wp * T::kWaveCols + j * 16, 0, lane);
        upper[j] = PTile::frag(weights(s), wp * T::kWaveCols + j * 16, 1, lane);
      }
    };
    wait_and_meet<0>();
    read_p(0);
    issue_q(1, wave);
#pragma unroll
    for (int u = 0; u < U::kAhead; ++u) read_q(0, u);
    for (int s = 0; s < steps; ++s) {
      // the next step's weights, in the place of the last one's, which were in registers at
      // the last meeting; then those of the step after it
      widen(s + 1);
      fetch(s + 2);
#pragma unroll
      for (int j = 0; j < kP; ++j) p[1][j] = upper[j];
      each<U::kCount>([&](auto index) {
        constexpr int u = decltype(index)::value;
        if constexpr (u == U::kMeet) {
          // this step's operands are in registers and the next one's in LDS; behind its rows
          // there are the weights just asked for
          wait_and_meet<kFetches>();
          read_p(s + 1);
          issue_q(s + 2, wave);
        }
        read_q(u < U::kMeet ? s : s + 1, u < U::kMeet ? u + U::kAhead : u - U::kMeet);
        __builtin_amdgcn_sched_barrier(0);  // the reads are on their way before the products
#pragma unroll
        for (int j = 0; j < kP; ++j) acc[u % L][j] = mma::mfma(p[u / L][j], q[u % U::kRing], acc[u % L][j]);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
  }
};

// Orders of all experts' tiles, dealt to the XCDs (workgroup b runs on XCD b mod 8).
// Expert by expert in 8 equal runs, as in find_item:
struct ByExpert : Runs {
  // Tile `at` of XCD x.
  __device__ __forceinline__ Item item(const LinearArgs& a, int x, int64_t at) const {
    const int chunk = (total + 7) / 8;
    return at < chunk && x * chunk + at < total ? Runs::item(a, x * chunk + (int)at) : Item{-1, 0, 0, 0, 0};
  }
};

// By what a tile costs: the full row tiles first, then the last ones of the runs that fill
// three quarters of theirs, half and a quarter (rounded up, as the products are:
// by_live_subtiles), each kind dealt to the XCDs in 8 equal parts.  Every XCD has the same
// work then, and what its compute units begin last is short.  256 rows an expert on average,
// 256 x 256 tiles, a third of them partly filled (128 experts, 2 x 768 x 2048, expert by expert and by cost):
// bf16 rows 259 and 241 us, their gradient 287 and 271, MXFP4 rows 117 and 115.  It takes 1 us
// longer to find a tile so: the tables of experts are read for every kind.
// Within a kind tiles are in the order of Runs, whose scan this is; the three partial kinds
// have at most a row tile per expert and are scanned as fields of one number.
struct ByCost {
  static constexpr int kKinds = 4, kField = 20;
  static_assert(MOE_MAX_EXPERTS < 1 << kField, "a field holds every expert");
  int bq, cp, J;
  int full, full_incl;       // full row tiles of this lane's experts, and with those of the lanes before it
  uint64_t part, part_incl;  // the same of the partial kinds, kind k in field k - 1
  int total[kKinds];         // tiles

  // Kind of the last `rest` rows of a run, 0 < rest < bq, or of a whole tile's.
  __device__ __forceinline__ int kind(int rest) const { return kKinds - (int)((unsigned)rest * kKinds + bq - 1) / bq; }
  // Row tiles of kind 0 of a run of n rows.
  __device__ __forceinline__ int whole(int n) const { return n / bq + (n % bq > 0 && kind(n % bq) == 0 ? 1 : 0); }

  __device__ __forceinline__ void scan(const LinearArgs& a, int rows_per_tile, int column_tiles) {
    bq = rows_per_tile;
    cp = column_tiles;
    full = full_incl = J = 0;
    part = part_incl = 0;
#pragma unroll
    for (int k = 0; k < kKinds; ++k) total[k] = 0;
    if (a.offsets == nullptr) {
      total[0] = ceil_div(a.rows, bq) * cp;
      return;
    }
    const int lane = threadIdx.x & 63;
    J = (a.E + 63) >> 6;
    const int most = a.rows / bq + min(a.E, a.rows);  // as in Runs
    for (int j = 0; j < J; ++j) {
      const int e = lane * J + j;
      if (e >= a.E) break;
      const int n = run_length(a.offsets[e], a.counts[e], a.rows), rest = n % bq, k = rest > 0 ? kind(rest) : 0;
      full = min(most, full + whole(n));
      if (k > 0) part += (uint64_t)1 << (k - 1) * kField;
    }
    full_incl = full;
    part_incl = part;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(full_incl, d);
      const uint64_t w = __shfl_up((unsigned long long)part_incl, d);
      if (lane >= d) {
        full_incl = min(most, full_incl + v);
        part_incl += w;
      }
    }
    total[0] = __builtin_amdgcn_readlane(full_incl, 63) * cp;
#pragma unroll
    for (int k = 1; k < kKinds; ++k) total[k] = __builtin_amdgcn_readlane(field(part_incl, k), 63) * cp;
  }
  __device__ __forceinline__ static int field(uint64_t v, int k) { return (int)(v >> (k - 1) * kField) & ((1 << kField) - 1); }

  // Tile `at` of XCD x, of any kind.
  __device__ __forceinline__ Item item(const LinearArgs& a, int x, int64_t at) const {
    int turn = 0;  // the XCD that gets the first tile left over of a kind
#pragma unroll
    for (int k = 0; k < kKinds; ++k) {
      const int each = total[k] >> 3, over = total[k] & 7, r = (x - turn) & 7;
      const int mine = each + (r < over ? 1 : 0);
      if (at < mine) return of_kind(a, k, r * each + min(r, over) + (int)at);
      at -= mine;
      turn += over;
    }
    return Item{-1, 0, 0, 0, 0};
  }
  __device__ __forceinline__ Item of_kind(const LinearArgs& a, int k, int i) const {
    Item it{0, 0, a.rows, 0, 0};
    if (a.offsets == nullptr) {
      tile_of(i, ceil_div(a.rows, bq), cp, it);
      return it;
    }
    const int lane = threadIdx.x & 63;
    const int mine = k == 0 ? full : field(part, k), incl = k == 0 ? full_incl : field(part_incl, k);
    const int owner = __builtin_ctzll(__ballot(i < incl * cp));
    int rest = i - (incl - mine) * cp, e = lane * J, off = 0, cnt = 0, rt = 1;
    for (int j = 0; j < J; ++j) {
      const int c = lane * J + j;
      if (c >= a.E) break;
      const int o = a.offsets[c], n = run_length(o, a.counts[c], a.rows);
      const int r = k == 0 ? whole(n) : n % bq > 0 && kind(n % bq) == k ? 1 : 0;
      e = c;
      off = o;
      cnt = n;
      rt = r;
      if (rest < r * cp) break;
      rest -= r * cp;
    }
    it.e = __builtin_amdgcn_readlane(e, owner);
    it.row0 = __builtin_amdgcn_readlane(off, owner);
    it.count = __builtin_amdgcn_readlane(cnt, owner);
    rt = __builtin_amdgcn_readlane(rt, owner);
    rest = __builtin_amdgcn_readlane(rest, owner);
    tile_of(rest, rt, cp, it);
    if (k > 0) it.tq = it.count / bq;
    return it;
  }
};

// Tiles one after another (SERIES): workgroup b takes tile b / 8 and every (grid / 8)-th one
// after it of those that XCD b % 8 is dealt.  A tile's first stages are loaded
// while the results of the one before it leave; with a tile per workgroup the search for it,
// the first loads' latency and the results' way out were half of the time where the depth
// is short.  Else a workgroup takes tile b / 8 alone: stores and loads come back in one
// order, so a tile's first stage waits for the results before it, which a workgroup that
// has a compute unit to itself pays for (128 experts, 32768 rows by 2048 x 768, 256 x 256
// tiles: 143 us in series, 118 alone; 128 x 128, two to a compute unit: 106 and 115).
template <class C, bool SERIES>
__global__ __launch_bounds__(C::kThreads, 2) void linear_mx_kernel(MxLinearArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // large tiles alone in a compute unit by their cost; the search is dear for small ones
  std::conditional_t<!SERIES && C::kQ % 4 == 0, ByCost, ByExpert> tiles;
  tiles.scan(a, C::BQ, (C::width(a) + C::kCols - 1) / C::kCols);
  const int64_t b = row::block_index();
  const int stride = (int)gridDim.x >> 3;
  int64_t at = b >> 3;
  auto next = [&] { return tiles.item(a, (int)(b & 7), at); };
  Item it = next();
  if (it.e < 0) return;
  char* const out = smem + C::kLds + wave * (16 * C::kOutCols * 2);
  C core;
  int64_t first;
  int live, p0;
  auto begin = [&] {
    first = (int64_t)it.row0 + it.tq * C::BQ;
    live = min(C::BQ, it.count - it.tq * C::BQ);
    p0 = it.tp * C::kCols;
    core.setup(a, it.e, first, live, p0, wave, lane);
    core.start(wave);
  };
  begin();
  while (true) {
    f32x4 acc[C::kQ][C::kP];
#pragma unroll
    for (int i = 0; i < C::kQ; ++i)
#pragma unroll
      for (int j = 0; j < C::kP; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    by_live_subtiles<C::kQ>((live - wave / C::WP * 16 + 16 * C::WQ - 1) / (16 * C::WQ),
                            [&](auto l) { core.template multiply<decltype(l)::value>(wave, lane, acc); });
    wait_and_meet<0>();  // every wave is done with the stages, and the loads past the last step have landed
    Finish<C> finish{it.e, live, p0, first};
    finish.load(a, wave);
    if constexpr (SERIES) {
      at += stride;
      it = next();
      if (it.e >= 0) begin();
    }
    finish.store(a, wave, out, acc);
    if (!SERIES || it.e < 0) break;
  }
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
  // a chunk of weights on its way while the one before it is multiplied (rows come from L2)
  struct Chunk {
    u32x4 w[kParts][2];
    uint32_t s[kParts][2];
  };
  auto fetch = [&](int c) {
    Chunk t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = c * kBlocks + quad * 2 + i, at = b < S ? b : 0;
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        t.w[h][i] = *reinterpret_cast<const u32x4*>(w[h] + at * 16);
        t.s[h][i] = sw[h][at];
      }
    }
    return t;
  };
  Chunk next = fetch(wk);
  for (int c = wk; c * kBlocks < S; c += WK) {
    const Chunk now = next;
    u32x4 xv[2][ROWS4 ? 1 : 4];
    uint32_t xb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int b = c * kBlocks + quad * 2 + i, at = b < S ? b : 0;
#pragma unroll
      for (int d = 0; d < (ROWS4 ? 1 : 4); ++d) xv[i][d] = *reinterpret_cast<const u32x4*>(x + at * (ROWS4 ? 16 : 64) + d * 16);
      xb[i] = ROWS4 ? sx[at] : 0u;
    }
    next = fetch(c + WK);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = c * kBlocks + quad * 2 + i < S;
      const u32x4 zero{0u, 0u, 0u, 0u};
#pragma unroll
      for (int d = 0; d < (ROWS4 ? 1 : 4); ++d)
        if (!in) xv[i][d] = zero;
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        const u32x4 wv = in ? now.w[h][i] : zero;
        const uint32_t wb = in ? now.s[h][i] : (uint32_t)mx::kZeroByte;
        if constexpr (ROWS4) {
          acc[h] = mx::mfma<0, 0>(wv, wb, xv[i][0], in ? xb[i] : (uint32_t)mx::kZeroByte, acc[h]);
        } else {
          const float f = mx::scale_bits(wb);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[h] = mma::mfma(mma::fp4x8_to_bf16(wv[k], f), __builtin_bit_cast(bf16x8, xv[i][k]), acc[h]);
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

// ---------------------------------------------------------------- launch --

// Instantiated by name: the host pass of this compiler otherwise leaves out the
// launch stubs of some kernel templates that are only reached through pointers.
#define MOE_MX_TILES(R, G)                                                     \
  template __global__ void linear_mx_few_kernel<R, G, 1, 8>(MxLinearArgs);     \
  template __global__ void linear_mx_few_kernel<R, G, 2, 8>(MxLinearArgs);     \
  template __global__ void linear_mx_few_kernel<R, G, 2, 2>(MxLinearArgs);
MOE_MX_TILES(false, false)
MOE_MX_TILES(false, true)
MOE_MX_TILES(true, false)
MOE_MX_TILES(true, true)
#undef MOE_MX_TILES
template <bool GATED, bool ALIGNED, int BQ, int BP, int WQ, int WP, int STAGES, int G>
using R4 = Rows4<Shape<GATED, BQ, BP, WQ, WP>, ALIGNED, STAGES, G>;
#define MOE_MX_ROWS4(G, A)                                                     \
  template __global__ void linear_mx_kernel<R4<G, A, 256, 256, 2, 4, 2, 2>, false>(MxLinearArgs); \
  template __global__ void linear_mx_kernel<R4<G, A, 128, 128, 2, 2, 2, 2>, true>(MxLinearArgs); \
  template __global__ void linear_mx_kernel<R4<G, A, 64, 128, 2, 2, 2, 2>, false>(MxLinearArgs);   \
  template __global__ void linear_mx_kernel<R4<G, A, 32, 128, 2, 2, 2, 2>, true>(MxLinearArgs);
MOE_MX_ROWS4(false, false)
MOE_MX_ROWS4(false, true)
MOE_MX_ROWS4(true, false)
MOE_MX_ROWS4(true, true)
#undef MOE_MX_ROWS4
template <bool GATED, bool ALIGNED, int BQ, int BP, int WQ, int WP>
using R16 = Rows16<Shape<GATED, BQ, BP, WQ, WP>, ALIGNED>;
#define MOE_MX_ROWS16(G, A)                                                    \
  template __global__ void linear_mx_kernel<R16<G, A, 256, 256, 2, 4>, false>(MxLinearArgs); \
  template __global__ void linear_mx_kernel<R16<G, A, 128, 128, 2, 2>, true>(MxLinearArgs); \
  template __global__ void linear_mx_kernel<R16<G, A, 64, 64, G ? 4 : 2, G ? 1 : 2>, false>(MxLinearArgs); \
  template __global__ void linear_mx_kernel<R16<G, A, 32, 64, 2, G ? 1 : 2>, false>(MxLinearArgs); \
  template __global__ void linear_mx_kernel<R16<G, A, 32, 128, 2, 2>, true>(MxLinearArgs);
MOE_MX_ROWS16(false, false)
MOE_MX_ROWS16(false, true)
MOE_MX_ROWS16(true, false)
MOE_MX_ROWS16(true, true)
#undef MOE_MX_ROWS16
template <int BQ, int BP, int WQ, int WP>
using B16 = Back16<Shape<false, BQ, BP, WQ, WP>>;
template __global__ void linear_mx_kernel<B16<256, 256, 2, 4>, false>(MxLinearArgs);
template __global__ void linear_mx_kernel<B16<128, 128, 2, 2>, true>(MxLinearArgs);
template __global__ void linear_mx_kernel<B16<64, 128, 2, 2>, true>(MxLinearArgs);
template __global__ void linear_mx_kernel<B16<32, 128, 2, 2>, true>(MxLinearArgs);

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

// A workgroup per tile, or in series as many as run at once: kCUs compute units, as many
// workgroups on each as have room in LDS.
constexpr int64_t kCUs = 256;
template <class C, bool SERIES>
hipError_t run_tiles(const MxLinearArgs& a, int cols, hipStream_t s) {
  static std::atomic<size_t> allowed[kMaxCachedDevices];
  constexpr int lds = C::kLds + C::kWaves * 16 * C::kOutCols * 2;
  static_assert(lds <= 160 * 1024, "a compute unit's LDS");
  const int64_t items = row_tiles_bound(a.rows, a.E, a.offsets == nullptr, C::BQ) * ((cols + C::kCols - 1) / C::kCols);
  void (*const kern)(MxLinearArgs) = &linear_mx_kernel<C, SERIES>;
  return launch(kern, SERIES ? std::min(items, kCUs * (160 * 1024 / lds)) : items, C::kThreads, lds, a, s, allowed);
}

mx::Sizes sizes_of(const MxLinearArgs& a) {
  return mx::Sizes{a.rows, a.E, a.offsets == nullptr, a.N, a.K, a.parts, a.ysb != nullptr};
}

// The forms, as the rules of mx_forms.h choose them.
template <bool GATED, bool ALIGNED>
hipError_t rows4_by_form(const MxLinearArgs& a, hipStream_t s) {
  switch (mx::rows4_form(sizes_of(a))) {
    case Form::kSplit16: return run_few<true, GATED, 1, 8>(a, s);
    case Form::kSplit32: return run_few<true, GATED, 2, 8>(a, s);
    case Form::kSplit32By2: return run_few<true, GATED, 2, 2>(a, s);
    case Form::k32x128: return run_tiles<R4<GATED, ALIGNED, 32, 128, 2, 2, 2, 2>, true>(a, a.N, s);
    case Form::k64x128: return run_tiles<R4<GATED, ALIGNED, 64, 128, 2, 2, 2, 2>, false>(a, a.N, s);
    case Form::k256x256: return run_tiles<R4<GATED, ALIGNED, 256, 256, 2, 4, 2, 2>, false>(a, a.N, s);
    default: return run_tiles<R4<GATED, ALIGNED, 128, 128, 2, 2, 2, 2>, true>(a, a.N, s);
  }
}

template <bool GATED, bool ALIGNED>
hipError_t rows16_by_form(const MxLinearArgs& a, hipStream_t s) {
  switch (mx::rows16_form(sizes_of(a))) {
    case Form::kSplit16: return run_few<false, GATED, 1, 8>(a, s);
    case Form::kSplit32: return run_few<false, GATED, 2, 8>(a, s);
    case Form::kSplit32By2: return run_few<false, GATED, 2, 2>(a, s);
    case Form::k32x64: return run_tiles<R16<GATED, ALIGNED, 32, 64, 2, GATED ? 1 : 2>, false>(a, a.N, s);
    case Form::k32x128: return run_tiles<R16<GATED, ALIGNED, 32, 128, 2, 2>, true>(a, a.N, s);
    case Form::k64x64: return run_tiles<R16<GATED, ALIGNED, 64, 64, GATED ? 4 : 2, GATED ? 1 : 2>, false>(a, a.N, s);
    case Form::k256x256: return run_tiles<R16<GATED, ALIGNED, 256, 256, 2, 4>, false>(a, a.N, s);
    default: return run_tiles<R16<GATED, ALIGNED, 128, 128, 2, 2>, true>(a, a.N, s);
  }
}

}  // namespace

hipError_t launch_linear_mx(const MxLinearArgs& a, hipStream_t s) {
  const uintptr_t lead = reinterpret_cast<uintptr_t>(a.xs) | reinterpret_cast<uintptr_t>(a.wsb[0]) | reinterpret_cast<uintptr_t>(a.wsb[1]);
  const bool aligned = a.K % 128 == 0 && lead % 4 == 0, gated = a.parts == 2;
  if (a.xs != nullptr) {
    if (aligned) return gated ? rows4_by_form<true, true>(a, s) : rows4_by_form<false, true>(a, s);
    return gated ? rows4_by_form<true, false>(a, s) : rows4_by_form<false, false>(a, s);
  }
  if (aligned) return gated ? rows16_by_form<true, true>(a, s) : rows16_by_form<false, true>(a, s);
  return gated ? rows16_by_form<true, false>(a, s) : rows16_by_form<false, false>(a, s);
}

hipError_t launch_linear_mx_backward_x(const MxLinearArgs& a, hipStream_t s) {
  switch (mx::back_form(sizes_of(a))) {
    case Form::k32x128: return run_tiles<B16<32, 128, 2, 2>, true>(a, a.K, s);
    case Form::k64x128: return run_tiles<B16<64, 128, 2, 2>, true>(a, a.K, s);
    case Form::k256x256: return run_tiles<B16<256, 256, 2, 4>, false>(a, a.K, s);
    default: return run_tiles<B16<128, 128, 2, 2>, true>(a, a.K, s);
  }
}

}  // namespace moe
