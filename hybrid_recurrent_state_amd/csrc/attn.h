// Device side of attn_verify_span, shared by the translation units that build
// it for one span and cache type each (attn.hip: host side and join;
// attn_f32.hip, attn_bf16.hip, attn_f8.hip: the kernels).
#pragma once

#include <hip/hip_runtime.h>

#include "device.h"
#include "internal.h"

namespace hrs {

constexpr int kAttnCus = 256;          // compute units that a launch is cut for
constexpr int kAttnReqs = 256;         // requests of a launch at most
constexpr int kF32 = 0, kB16 = 1, kF8 = 2;   // span/cache types: f32/f32, bf16/bf16, bf16/e4m3

struct AttnBase {
  const void* q;
  const void* k;
  const void* v;
  const char* k_cache;
  const char* v_cache;
  const int32_t* page_table;
  const int32_t* seq_len;
  const float* k_scale;
  const float* v_scale;
  void* out;
  int32_t* status;
  int32_t* plan;      // workspace: units before every request [n + 1], for the join
  float* part;        // workspace: partial sums [2 * blocks][rows / 16][d / 16][64 lanes][4]
  float2* part_ml;    // workspace: their maximum and sum [2 * blocks][rows]
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  float scale;
  int32_t window;
  int32_t n_req;      // of the whole call
  int32_t req0;       // of this launch
  int32_t n_pos;
  int32_t kvheads;
  int32_t group;      // query heads per key/value head
  int32_t rows;       // n_pos * group
  int32_t row_blocks;
  int32_t n_pages;
  int32_t page_shift;
  int32_t table_len;
  int32_t tree;
};
// Chains and the join do without the trees: every launch copies its arguments.
struct AttnTree : AttnBase {
  int8_t parent[kGeomBytes];
};

// What the cut needs to know. These are kernel arguments of their own, at the
// front, which the hardware has in registers when a wave starts: the lengths'
// loads, the first of a chain of dependent ones, need not wait for the
// argument block's.
struct AttnLens {
  const int32_t* len;   // of the launch's first request
  int32_t n;            // requests
  int32_t heads;        // key/value heads times row blocks
  int32_t most;         // slots of a table
  int32_t window;
  int32_t n_pos;
  int32_t log_blocks;   // of the launch's blocks
};

// How a block is built for a type, a head size and a class of row counts
// (0: at most 16 rows a key/value head, 1: 32, 2: 64, 3: blocks of 128, 4:
// e4m3 caches with 65 to 96 rows of at most 128 elements). WR waves share the
// slots of a tile with different rows, WK such groups take different slots; a
// wave holds RT tiles of 16 rows and SS slots of a tile. Measured, one request
// (time of the whole call):
//  - 16 rows a wave below 64 rows, more waves instead: 32 rows a wave took 65
//    instead of 37 us (30 rows, 9000 slots of 4 heads of 256, f32), 39 / 34
//    (26,758 slots, bf16), 37.6 / 34.3 (48 rows, 30,000 slots of 8 heads of
//    128, bf16), 34.3 / 30.5 (the same, e4m3).
//  - class 4: an e4m3 tile is widened by every wave that reads it, so two
//    waves of 48 rows instead of four of 32 (8 heads of 128, the same at 65,
//    68, 80 and 96 rows: 154 / 197 us at 262,144 slots, 37.5 / 38 at 30,000, 22
//    / 20 at 3000; lengths are not known where the class is chosen); bf16 is
//    bound by the read either way.
//  - 32 slots a wave in class 1 where a row is at most 128 bytes (24.7 / 26.5
//    us, 28 rows, e4m3); 16 for longer ones (34.0 / 35.4 us, bf16).
//  - four waves with slots of their own in class 0: eight, or 32 slots each,
//    took 14.5 and 14.8 instead of 13.6 us at 1000 slots of 128 and gained
//    nothing at 30,000.
template <int KIND, int D, int CLS> struct AttnCfg {
  static constexpr int ESZ = KIND == kF32 ? 4 : 2;          // bytes of an element in LDS
  static constexpr int ESZC = KIND == kF32 ? 4 : KIND == kB16 ? 2 : 1;   // of a cached one
  static constexpr bool WIDE = D == 256;
  static constexpr int RT = CLS == 4 ? 3 : CLS < 3 || WIDE ? 1 : 2;
  static constexpr int WR = CLS == 0 ? 1 : CLS == 1 || CLS == 4 ? 2 : CLS == 2 || !WIDE ? 4 : 8;
  static constexpr int WK = CLS < 2 ? (WIDE ? 2 : 4) : CLS == 2 || CLS == 4 ? 2 : 1;
  static constexpr int SS = CLS == 0   ? 16
                            : CLS == 1 ? (D * ESZC <= 128 ? 32 : 16)
                            : CLS == 2 ? (WIDE ? 16 : 32)
                                       : (KIND == kF32 && D == 128 ? 16 : 32);
  // Blocks of a CU: two where they fit (their waits and sums overlap).
  static constexpr int PER_CU = CLS >= 3 && !WIDE ? 2 : 1;
  static constexpr int NW = WR * WK;
  static constexpr int NT = 64 * NW;
  static constexpr int ROWS = 16 * RT * WR;
  static constexpr int TS = SS * WK;                        // slots of a tile
  static constexpr int STAGE = 2 * TS * D * ESZ;            // keys and values of a tile, in the span's type
  static constexpr int RAW = 2 * TS * D * ESZC;             // in the cache's
  static constexpr int ROOM = 131072 / PER_CU;
  // Tiles of the ring; a fourth gained nothing (26,758 slots of 256: 47 / 46 us).
  static constexpr int NST = ROOM / RAW < 3 ? ROOM / RAW : 3;
  static constexpr int JOIN = WK / 2 * WR * RT * 64 * (D + 8);   // sums of half the wave groups
  static constexpr int TILES = NST * RAW > STAGE ? NST * RAW : STAGE;   // an e4m3 cache's span tiles take the ring's place
  static constexpr int LDS = TILES > JOIN ? TILES : JOIN;
  static_assert(NST >= 2 && LDS <= 155 * 1024 / PER_CU, "tiles fit");
};

// Units without a tile at the end of every head: its last run of tiles also
// takes the span's masks, the end of a sum and, for most blocks, the start of
// another one, about the time of that many tiles (measured at 26,758 slots of
// 256: the blocks with a span tile ended 5 us behind the others).
constexpr int kExtraUnits = 4;

// Work is counted in units: a unit is one tile of one (request, key/value
// head, row block); the context's tiles come first, the span's last.
struct AttnUnits {
  int first;   // first context tile that a window leaves in reach
  int ctx;     // context tiles
  int all;     // and the span's, and kExtraUnits
  __device__ __forceinline__ int tiles() const { return all - kExtraUnits; }
};

__device__ __forceinline__ AttnUnits attn_units(const AttnLens& a, int len, unsigned ts) {
  const bool ok = len >= 0 && len <= a.most;
  const unsigned n = ok ? len : 0;
  const unsigned first = a.window > 0 ? static_cast<unsigned>(max(static_cast<int>(n) + 1 - a.window, 0)) / ts : 0;
  const int ctx = static_cast<int>((n + ts - 1) / ts - min(first, (n + ts - 1) / ts));
  return {static_cast<int>(first), ctx, ok ? ctx + static_cast<int>((a.n_pos + ts - 1) / ts) + kExtraUnits : 0};
}

// Where block b's run of units starts: an even cut where there are at least
// as many units as blocks (a power of two), one unit a block otherwise.
__device__ __forceinline__ int attn_cut(int b, int total, int log_blocks) {
  if (total <= (1 << log_blocks)) return min(b, total);
  return static_cast<int>((static_cast<int64_t>(b) * total) >> log_blocks);
}

// Launches of one type (rows class cls, head size d); the number of rows a
// block holds and the slots of its tile for it.
struct AttnShape {
  int rows, ts, blocks;
};
template <int KIND> AttnShape attn_shape(int d, int cls);
template <int KIND> void attn_launch(const AttnTree& args, const AttnLens& lens, int d, int cls, hipStream_t s);

}  // namespace hrs
