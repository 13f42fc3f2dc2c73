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

// attn_verify_shared: a prefix that all requests of a launch share.
struct AttnShared : AttnBase {
  const int32_t* prefix_table;
  const int32_t* prefix_len;
  int32_t prefix_pages;
  int32_t pad;
};
struct AttnSharedTree : AttnShared {
  int8_t parent[kGeomBytes];
};
// What a launch computes: attn_verify_span; the same without the slots that
// attn_verify_shared takes for all requests at once; those slots, for the rows
// of all requests.
constexpr int kSpan = 0, kOwn = 1, kPrefix = 2;

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

// The slots that all requests of a launch count at every position, in the
// prefix's pages: whole tiles of every block shape. What is left of the prefix
// at either end (a window's start, a length that is no multiple) is read by
// each request for itself.
constexpr int kHoleStep = 128;
struct AttnHole {
  int first, end;    // slots; equal: none
  int prefix;        // slots of the prefix, -1: not a length
};

__device__ __forceinline__ AttnHole attn_hole(const AttnLens& a, const AttnShared& args, const int (&len)[kAttnReqs / 64]) {
  const int32_t given = *args.prefix_len;
  const bool ok = given >= 0 && given <= args.prefix_pages << args.page_shift;
  int lo = 0, hi = ok ? given : 0;
#pragma unroll
  for (int k = 0; k < kAttnReqs / 64; ++k) {
    if (len[k] < 0 || len[k] > a.most) continue;
    hi = min(hi, len[k]);
    if (a.window > 0) lo = max(lo, len[k] + a.n_pos - a.window);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    lo = max(lo, __shfl_xor(lo, d));
    hi = min(hi, __shfl_xor(hi, d));
  }
  lo = __builtin_amdgcn_readfirstlane((lo + kHoleStep - 1) & ~(kHoleStep - 1));
  hi = __builtin_amdgcn_readfirstlane(hi & ~(kHoleStep - 1));
  return AttnHole{lo < hi ? lo : 0, lo < hi ? hi : 0, ok ? given : -1};
}

// Units of a request that leaves out the hole: its own tiles of the prefix
// (`before` of them), then those of its own pages. The tile that the prefix
// ends in is of both kinds.
struct AttnSharedUnits : AttnUnits {
  int before;
  int hole, skip;    // first tile of the hole, and its tiles
  int own;           // first tile of its own pages
};
__device__ __forceinline__ AttnSharedUnits attn_shared_units(const AttnLens& a, const AttnHole& hole, int len, int ts) {
  AttnSharedUnits un{};
  const bool ok = len >= 0 && len <= a.most && hole.prefix >= 0;
  if (!ok) return un;
  const int reach = a.window > 0 ? max(len + 1 - a.window, 0) : 0;     // first slot that counts for anyone
  const int shared = min(len, hole.prefix);
  un.first = reach / ts;
  un.hole = hole.first / ts;
  un.skip = (hole.end - hole.first) / ts;
  un.before = reach < shared ? (shared + ts - 1) / ts - un.first - un.skip : 0;
  un.own = max(hole.prefix, reach) / ts;
  const int mine = len > hole.prefix && len > reach ? (len + ts - 1) / ts - un.own : 0;
  un.ctx = un.before + mine;
  un.all = un.ctx + (a.n_pos + ts - 1) / ts + kExtraUnits;
  return un;
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
// Launches of attn_verify_shared: the requests' own part, the prefix.
template <int KIND> void attn_own_launch(const AttnSharedTree& args, const AttnLens& lens, int d, int cls, hipStream_t s);
// How the prefix launch for large batches is built (attn_prefix.h).
template <int KIND, int D> struct PrefixCfg {
  static constexpr int RT = D >= 128 ? 3 : 4;   // tiles of 16 rows a wave
  static constexpr int NW = 4;
  static constexpr bool NEXT = D == 256;                       // the next tile's scores under this one's weights
  static constexpr int PER_CU = NEXT ? 1 : 2;                  // blocks
  static constexpr int ROWS = 16 * RT * NW;
  static constexpr int TS = 32;                                // slots of a tile
  static constexpr int STAGE = 2 * TS * D * 2;                 // bytes of its keys and values
  static constexpr int NST = KIND == kF8 ? 3 : 4;              // tiles of the ring
  static constexpr int LDS = NST * STAGE;
};
template <int KIND> void attn_prefix_wide(const AttnShared& args, const AttnLens& lens, int runs, int d, hipStream_t s);
template <int KIND> void attn_prefix_launch(const AttnShared& args, const AttnLens& lens, int d, int cls, hipStream_t s);

inline bool sizes_ok(const hrs_attn_desc* d) {
  return d && d->n_req >= 1 && d->n_req <= 4096 && d->n_pos >= 1 && d->n_pos <= HRS_MAX_POS && d->n_heads >= 1 &&
         d->n_kvheads >= 1 && d->n_kvheads <= 1024 && d->n_heads % d->n_kvheads == 0 &&
         d->n_heads / d->n_kvheads <= 64;
}

// The class of AttnCfg; its comment has both sides of each border.
inline int rows_class(int kind, int d, int64_t rows) {
  if (kind == kF8 && d <= 128 && rows > 64 && rows <= 96) return 4;
  return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3;
}

inline AttnShape shape_of(int kind, int d, int64_t rows) {
  const int cls = rows_class(kind, d, rows);
  return kind == kF32 ? attn_shape<kF32>(d, cls) : kind == kB16 ? attn_shape<kB16>(d, cls) : attn_shape<kF8>(d, cls);
}
inline AttnShape shape_of(const hrs_attn_desc* d, int kind) {
  return shape_of(kind, d->d, static_cast<int64_t>(d->n_pos) * (d->n_heads / d->n_kvheads));
}

}  // namespace hrs
