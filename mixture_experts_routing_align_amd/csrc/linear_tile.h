// Building blocks of the tiled expert products for gfx950 (linear.hip): finding a
// workgroup's expert and tile, staging operand tiles in LDS with direct
// global-to-LDS loads, and reading them back as matrix-core fragments.
//
// Every product is D[q, p] = sum_d Q(q, d) P(p, d): Q gives the rows of the output,
// P its contiguous columns, d is the depth.  One v_mfma_f32_16x16x32_bf16 takes 16
// P columns as its A operand and 16 Q rows as its B operand, so lane l ends up
// with row l % 16 and the 4 consecutive columns 4 (l / 16) ... + 3 of the tile.
// An operand tile sits in LDS in one of two orders:
//  - by rows ("R"): one line per operand row, 128 bytes of depth each; a lane's 8
//    consecutive depth elements are one 16-byte piece.
//  - by depth ("D"): one line per depth step, the operand's rows along it (the
//    memory order of a matrix whose rows are the depth); ds_read_b64_tr_b16
//    transposes 4 depth steps x 16 rows on the way to the registers.
// Pieces are swizzled within their line so that a wave's reads spread over all
// banks; a direct load writes 16 bytes per lane in lane order, so the swizzle is
// applied to the address each lane loads from.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mma_common.h"
#include "ops_internal.h"
#include "row_runs.h"

namespace moe {
namespace tile {

typedef __attribute__((address_space(3))) void lds_void;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
using mma::bf16x8;
using mma::f32x4;

// A byte offset past every buffer resource built here (each ends at 2^31 - 1): a
// direct load from it fetches nothing and leaves zeros in LDS.
constexpr uint32_t kNoFetch = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7fffffff, 0x00020000);
}

// Wait until at most N of this wave's memory loads are outstanding and its LDS
// reads are done, then meet the workgroup.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ------------------------------------------------------------ work items --

struct Item {
  int e;       // expert, or -1: nothing to do
  int row0;    // its first row in the sorted matrices
  int count;   // its rows
  int tq, tp;  // tile indexes along the rows and along the columns
};

// Item i of an expert with rt row tiles and cp column tiles: the 32 workgroups an XCD
// runs at once then hold 8 row tiles by 4 column tiles, 12 operand tiles for 64 reads,
// which its L2 serves (33 TB/s against 15 where the reads miss it).
__device__ __forceinline__ void tile_of(int i, int rt, int cp, Item& it) {
  const int g = i / (8 * cp), rows = min(8, rt - 8 * g), r = i - g * 8 * cp;
  it.tp = r / rows;
  it.tq = 8 * g + r - it.tp * rows;
}

// All experts' tiles, `bq` rows a tile and `cp` column tiles.  Every wave scans the tables
// by itself: lane l sums the tiles of experts l J ... l J + J - 1, a scan over the wave gives
// each lane's first tile, and the lane that holds an item names its expert.  Tiles are
// numbered expert by expert, within an expert 8 row tiles by 8 row tiles, there column tile
// by column tile.
struct Runs {
  int bq, cp, J;
  int mine, incl;  // row tiles of this lane's experts, and with those of the lanes before it
  int total;       // tiles

  __device__ __forceinline__ void scan(const LinearArgs& a, int rows_per_tile, int column_tiles) {
    bq = rows_per_tile;
    cp = column_tiles;
    mine = incl = J = 0;
    if (a.offsets == nullptr) {
      total = ceil_div(a.rows, bq) * cp;
      return;
    }
    const int lane = threadIdx.x & 63;
    J = (a.E + 63) >> 6;
    // No sum passes what runs that do not overlap can make (row_tiles_bound), so tables
    // that claim more cannot wrap the products below; their items past it are left out.
    const int most = a.rows / bq + min(a.E, a.rows);
    for (int j = 0; j < J; ++j) {
      const int e = lane * J + j;
      if (e < a.E) mine = min(most, mine + ceil_div(run_length(a.offsets[e], a.counts[e], a.rows), bq));
    }
    incl = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl = min(most, incl + v);
    }
    total = __builtin_amdgcn_readlane(incl, 63) * cp;
  }

  // Tile i < total.
  __device__ __forceinline__ Item item(const LinearArgs& a, int i) const {
    Item it{0, 0, a.rows, 0, 0};
    if (a.offsets == nullptr) {
      tile_of(i, ceil_div(a.rows, bq), cp, it);
      return it;
    }
    // the lane whose experts hold item i, and the expert within it
    const int lane = threadIdx.x & 63;
    const uint64_t after = __ballot(i < incl * cp);
    const int owner = __builtin_ctzll(after);
    int rest = i - (incl - mine) * cp, e = lane * J, off = 0, cnt = 0, rt = 1;
    for (int j = 0; j < J; ++j) {
      const int c = lane * J + j;
      if (c >= a.E) break;
      const int o = a.offsets[c], n = run_length(o, a.counts[c], a.rows), r = ceil_div(n, bq);
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
    return it;
  }
};

// The tile of workgroup `b`: tiles are dealt to the 8 XCDs in 8 equal runs (workgroup b runs
// on XCD b mod 8), so an expert's weights and rows stay in one XCD's L2.
__device__ __forceinline__ Item find_item(const LinearArgs& a, int b, int bq, int cp) {
  Runs runs;
  runs.scan(a, bq, cp);
  const int chunk = (runs.total + 7) / 8, i = (b & 7) * chunk + (b >> 3);
  if ((b >> 3) >= chunk || i >= runs.total) return Item{-1, 0, 0, 0, 0};
  return runs.item(a, i);
}

// ---------------------------------------------------------- staging, "R" --

// Bytes of depth a stage holds of each operand row: 64 bf16 or 128 8-bit elements (one
// scale block), and one whole cache line.  (64-byte lines ask L2 twice as often and
// measured slower, 256-byte lines leave too few stages.)
constexpr int kDB = 128;

// A tile of R operand rows by kDB bytes of depth, staged by WAVES waves: each direct
// load of a wave fills 1 KB = 8 lines.  PAIRS: made for reads in which neighbouring quads
// of lanes take pieces two apart (a quad has a pair of them), not neighbouring ones.
template <int R, int WAVES, bool PAIRS = false>
struct RowTile {
  static constexpr int kBytes = R * kDB;
  static constexpr int kLines = 1024 / kDB;  // lines one load of a wave fills
  static constexpr int kLoads = kBytes / 1024 / WAVES;
  static constexpr int kPieces = kDB / 16;
  static_assert(kBytes % (1024 * WAVES) == 0, "whole loads per wave");
  // Piece g of line r sits at g ^ swz(r): two lines make 256 bytes of LDS (all banks),
  // and the 16 lines that the lanes of a quad read at one piece land on 16 different
  // pieces of them (measured: no bank conflicts).  The LDS serves 16 lanes at a time, some
  // of one quad and the others of the next one, so what the rows of either add to the
  // piece has to stay apart under the distance of their pieces: the lowest bit of r / 2
  // does for a distance of 1, the second one, which PAIRS puts in its place, for 2.
  __device__ static __forceinline__ int swz(int r) {
    const int i = (r / 2) & (kPieces - 1);
    return PAIRS ? (i & ~3) | (i & 1) << 1 | (i >> 1 & 1) : i;
  }

  uint32_t off[kLoads];  // this lane's byte offset of each of its loads at depth 0, or kNoFetch
  int piece;             // and the depth byte its piece starts at

  // `row_off(r)` gives the byte offset of operand row r in the resource, or kNoFetch.
  template <typename F>
  __device__ __forceinline__ void init(int wave, int lane, F row_off) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = (i * WAVES + wave) * kLines + lane / kPieces;
      const int g = (lane % kPieces) ^ swz(r);
      const uint32_t o = row_off(r);
      off[i] = o == kNoFetch ? kNoFetch : o + g * 16;
      if (i == 0) piece = g * 16;
    }
    // a line's swizzle repeats every 16 lines, so all of a lane's loads take the same
    // piece where the loads are that far apart
    static_assert(kLoads == 1 || (WAVES * kLines) % (2 * kPieces) == 0, "one piece index per lane");
  }
  // Fill `lds` from depth byte `d` on; pieces at or past `left` bytes from there are zero.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, char* lds, int wave, uint32_t d, int left) const {
    const bool cut = piece >= left;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) one(r, lds, wave, d, cut, i);
  }
  // The same, without the loads of lines at or past `live` (the same for the
  // workgroup): what LDS holds there feeds only output rows that are not stored.
  __device__ __forceinline__ void load_live(__amdgpu_buffer_rsrc_t r, char* lds, int wave, uint32_t d, int left, int live) const {
    const bool cut = piece >= left;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if ((i * WAVES + wave) * kLines < live) one(r, lds, wave, d, cut, i);
  }
  __device__ __forceinline__ void one(__amdgpu_buffer_rsrc_t r, char* lds, int wave, uint32_t d, bool cut, int i) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (i * WAVES + wave) * 1024), 16, cut ? kNoFetch : off[i], d, 0, 0);
  }
  // Piece g of line r.
  __device__ static __forceinline__ const char* at(const char* lds, int r, int g) {
    return lds + r * kDB + ((g ^ swz(r)) * 16);
  }
  // 8 consecutive depth elements of step kk (32 deep) for operand row r0 + l % 16.
  __device__ static __forceinline__ bf16x8 frag(const char* lds, int r0, int kk, int lane) {
    return *reinterpret_cast<const bf16x8*>(at(lds, r0 + (lane & 15), kk * 4 + (lane >> 4)));
  }
  // A stage of 128 8-bit depth elements for operand row r0 + l % 16: pieces q and
  // q + 4, 16 elements each, which widen() makes the bf16 operands of four 32-deep
  // steps (e4m3 is exact in bf16; which element meets which step does not matter as
  // long as both operands agree).
  struct Raw8 {
    uint4 v[2];
  };
  __device__ static __forceinline__ Raw8 raw8(const char* lds, int r0, int lane) {
    Raw8 r;
#pragma unroll
    for (int h = 0; h < 2; ++h) r.v[h] = *reinterpret_cast<const uint4*>(at(lds, r0 + (lane & 15), (lane >> 4) + 4 * h));
    return r;
  }
  __device__ static __forceinline__ void widen(const Raw8& r, bf16x8 (&f)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[2 * h] = mma::fp8x8_to_bf16(r.v[h].x, r.v[h].y);
      f[2 * h + 1] = mma::fp8x8_to_bf16(r.v[h].z, r.v[h].w);
    }
  }
};

// ---------------------------------------------------------- staging, "D" --

// A tile of D depth steps by C bf16 operand rows (contiguous in memory).
template <int C, int D, int WAVES>
struct DepthTile {
  static constexpr int kLine = C * 2;
  static constexpr int kBytes = D * kLine;
  static constexpr int kLines = 1024 / kLine;
  static constexpr int kLoads = kBytes / 1024 / WAVES;
  static constexpr int kPieces = kLine / 16;
  static_assert(kBytes % (1024 * WAVES) == 0 && kLine >= 256, "whole loads per wave");
  // 32-byte segments (16 operand rows of one depth step) are swizzled by the depth
  // step: one transposing read takes depth steps 8 q + 0..3 of the same segment
  // for q = 0..3, which land on 8 different segments of a 256-byte line.
  __device__ static __forceinline__ int swz(int d) { return (d & 3) | ((d >> 1) & 4); }

  uint32_t off[kLoads];
  int line[kLoads];  // depth step of each load within the tile

  // `row_off(g)` gives the byte offset, within a depth line, of the piece of 8
  // operand rows 8 g ... 8 g + 7, or kNoFetch; `ld` the bytes from line to line.
  template <typename F>
  __device__ __forceinline__ void init(int wave, int lane, uint32_t ld, F row_off) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int d = (i * WAVES + wave) * kLines + lane / kPieces;
      const int s = lane % kPieces;
      const int g = (((s >> 1) ^ swz(d)) << 1) | (s & 1);
      const uint32_t o = row_off(g);
      line[i] = d;
      off[i] = o == kNoFetch ? kNoFetch : o + d * ld;
    }
  }
  // Fill `lds` with `left` depth lines (the rest zero) from byte `d` on.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, char* lds, int wave, uint32_t d, int left) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(lds + (i * WAVES + wave) * 1024), 16,
                                               line[i] >= left ? kNoFetch : off[i], d, 0, 0);
  }
  // 8 consecutive depth elements of step kk (32 deep) for operand row r0 + l % 16
  // (r0 a multiple of 16): two transposing reads of 4 depth steps x 16 rows.
  __device__ static __forceinline__ bf16x8 frag(const char* lds, int r0, int kk, int lane) {
    const int q = lane >> 4, i = lane & 15;
    const int d = kk * 32 + q * 8 + (i >> 2);
    const int seg = (r0 >> 4) ^ swz(d);  // the same for d and d + 4
    const char* p = lds + d * kLine + seg * 32 + (i & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p + 4 * kLine));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
  }
};

// ------------------------------------------------------------ tile stores --

// An output tile of ROWS rows of ROW_BYTES, gathered in LDS so that it leaves as
// whole lines, 16 bytes a lane: the fragments' own 8-byte pieces of 16 rows at a
// time cost as much as the whole product (256 rows an expert, weight gradient:
// 270 of 490 us).  Pieces of 16 bytes are swizzled by the row, so a wave's writes
// spread over the banks without padding.
template <int ROWS, int ROW_BYTES, int THREADS>
struct OutTile {
  static constexpr int kPieces = ROW_BYTES / 16, kMask = kPieces < 16 ? kPieces - 1 : 15;
  template <typename T>
  __device__ static __forceinline__ void put(char* lds, int r, int byte, T v) {
    *reinterpret_cast<T*>(lds + r * ROW_BYTES + (((byte >> 4) ^ (r & kMask)) << 4) + (byte & 15)) = v;
  }
  // Rows below `live`, their first `valid` bytes (a multiple of 16), to dst; ld bytes
  // from row to row.  PAST_CACHE: not kept in the caches, for outputs too large to be
  // read from there (weight gradient of 805 MB: 417 -> 296 us; no difference for
  // outputs of 150 MB).
  template <bool PAST_CACHE = false>
  __device__ static __forceinline__ void flush(const char* lds, char* dst, int64_t ld, int live, int valid) {
    for (int i = threadIdx.x; i < ROWS * kPieces; i += THREADS) {
      const int r = i / kPieces, g = i % kPieces;
      if (r < live && g * 16 < valid) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds + r * ROW_BYTES + ((g ^ (r & kMask)) << 4));
        u32x4* to = reinterpret_cast<u32x4*>(dst + r * ld + g * 16);
        if constexpr (PAST_CACHE)
          __builtin_nontemporal_store(v, to);
        else
          *to = v;
      }
    }
  }
};

}  // namespace tile
}  // namespace moe
