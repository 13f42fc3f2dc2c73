// The kernel of attn_verify_span.
//
//   S^T = K Q^T,  P = exp2(c S - m),  O^T += V^T P^T,  l += P,  out = O / l
//
// over tiles of slots with a running reference m per query row.
//
// MI355X design. The rows of a key/value head are all query heads of its
// group at all span positions (17 positions x 6 heads = 102), so its keys and
// values are read once for up to 128 of them (every further block of rows
// reads them again). That read is the bound of
// every long context; short ones are bound by latency (lengths, page numbers,
// tiles, the parts' join: four dependent reads and two launches). The tiles of
// all requests and heads form one list that is cut into equal runs, one per
// block, so ragged lengths leave no CU idle and the host needs no lengths; a
// run that ends inside a head leaves a partial sum (f32) for the join.
//  - Tiles travel from memory to LDS without registers (16 bytes per lane), a
//    ring of three; a wave waits for the loads it issued itself and one
//    barrier per tile makes them everybody's (none where a wave has its slots
//    to itself). A compiler-made wait for all loads inside the loop, as for a
//    spilled register or a transposing LDS read, costs a memory latency per
//    tile (e4m3, 262,144 slots: 160 vs 195 us for one spilled register).
//    Page numbers are read a tile ahead by scalar loads; a page never ends
//    inside 16 slots, so a load's base address is wave-uniform.
//  - 16-byte pieces are permuted within a row (on the memory side, since the
//    LDS side of such a load is linear) so that the 16 rows of an operand lie
//    in different banks.
//  - The transposed products need no data movement between them: a lane of
//    S^T holds one query row's scores of four consecutive slots, which is the
//    layout of P^T as the second operand when the slots of a 32-slot step are
//    taken in the order 4 g + i, 16 + 4 g + i; V^T in that order comes from
//    plain reads of rows and byte permutations (Values). Row maxima and the
//    rescaling of O are per-lane numbers.
//  - The reference m moves only when a row's maximum exceeds it by more than
//    8 (in log2), so most tiles neither reduce across lanes nor rescale; P is
//    at most 2^8 and l and O are f32, which loses nothing.
//  - P for the product with bf16 values is the sum of two bf16 parts, the upper
//    bits and what they leave: 2^-15 of a weight at most is lost. One part
//    alone (2^-9) made the result's error 0.0023 instead of 0.0017, which is
//    what rounding the result costs, and took 6% less time (26,758 slots: 41.5
//    / 44.1 us; 16 trees: 109.9 / 113.7; 1000 slots: no difference, since 16
//    slots fill half of a matrix instruction and the second part the other).
//    Beside e4m3 values P is float16 (2^-11 of a weight, or 2^-32 of the row's
//    largest where that is more), which the values are widened to as well: the
//    same matrix rate, no second part (two parts took 190 instead of 160 us at
//    262,144 slots in bf16, 206 instead of 167 in float16).
//  - e4m3 tiles stay e4m3 in LDS and are widened (exactly) to 16 bits between
//    LDS and the products; the scales are factors of c and of O. (Widened once
//    per block into a second LDS tile: 215 us instead of 160 at 262,144 slots:
//    the extra pass and its barrier were not hidden.) The span's own tile is of
//    the span's type and takes the ring's place after the cache's tiles.
//  - Tiles with a mask (the span, the context's end, a window's border,
//    absent pages) drop scores that do not count; values that are not finite
//    leave the product (0 * NaN) and are added after the segment for the rows
//    that count them (add_odd).
//
// Measured (bf16 unless noted, whole call with the join; other cards gave up
// to 10% more): 1 position, 1000 slots of 4 heads of 256: 13.4 us (main kernel
// 8.8, join 5.2); chain of 17 over 26,758 slots of 4 heads of 256 (110 MB): 44
// us; 16 trees of 23 over 4368 to 8191 slots of 8 heads of 128 (427 MB): 114
// us, 3.8 TB/s; chain of 17 over 262,144 e4m3 slots of 8 heads of 128 (537 MB):
// 146 us, 3.7 TB/s, where the vector units' work per tile (widening,
// exponentials, permutations) is as long as its read and hides behind it only
// in part.
#pragma once

#include <type_traits>

#include "attn.h"

namespace hrs {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char lds_char;

// The same number, but what is computed from it is computed after this point:
// keeps addresses that are needed once per segment out of the registers of the
// tile loop (where a spilled register's reload waits for all tiles on their
// way).
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ void mem_fence() { asm volatile("" ::: "memory"); }

// Waits until at most n of this wave's vector memory operations are on their
// way (they end in order).
template <int N> __device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The wave's own LDS reads and writes have ended: what was read may be loaded
// over.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// All waves' LDS reads and writes before, all after; loads to LDS only where
// each wave has waited for its own.
__device__ __forceinline__ void block_barrier() {
  wait_lds();
  __builtin_amdgcn_s_barrier();
  mem_fence();
}

__device__ __forceinline__ uint32_t lds_address(const char* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_char*)p));
}
// LDS by its byte address.
template <typename T> __device__ __forceinline__ const __attribute__((address_space(3))) T* lds_at(uint32_t a) {
  return reinterpret_cast<const __attribute__((address_space(3))) T*>(a);
}

// Larger (or sum) over the four lanes that hold one query row.
__device__ __forceinline__ float row_max(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_sum(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Where piece c of a tile row lies: pieces are exchanged within groups of 16
// (8 in a 128-byte row) so that equal pieces of 16 rows, and pairs of pieces
// of 4 consecutive rows, are in different banks.
template <int CPR> __device__ __forceinline__ uint32_t swizzle(uint32_t row) {
  return CPR == 4 ? (row >> 2) & 3 : CPR >= 16 ? ((row & 7) << 1) | ((row >> 3) & 1) : (((row >> 1) & 3) << 1) | ((row >> 3) & 1);
}

__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u; }

// What a mask needs to know of a block's query rows.
template <int ROWS> struct AttnRows {
  uint64_t anc[ROWS];     // span positions that count, one bit each
  int32_t first[ROWS];    // first context slot that counts; no row: past all
};

template <int KIND, int D, int CLS> struct AttnBlock {
  using C = AttnCfg<KIND, D, CLS>;
  static constexpr int ESZ = C::ESZ, CPR = D * ESZ / 16, SB = C::SS / 16;
  static constexpr int CSZ = KIND == kF32 ? 4 : KIND == kB16 ? 2 : 1;      // bytes of a cached element
  static constexpr int RCPR = D * CSZ / 16;                               // pieces of a cached row
  static constexpr int LPS = 2 * C::SS * RCPR / (64 * C::WR);             // loads of a wave per tile
  static constexpr int SPS = 2 * C::SS * CPR / (64 * C::WR);              // pieces of a wave per tile in LDS
  static constexpr int DT = D / 16;
  static constexpr int QC = D * ESZ / 64;                                 // pieces of a query row per lane
  static_assert(SB <= 2, "one or two blocks of 16 slots");
  // P's exponent is lifted beside an e4m3 cache: at most 8 + 7, so that the
  // small weights of many slots are not lost below float16's range (2^-24:
  // 2^-31 of the reference's weight).
  static constexpr float kLift = KIND == kF8 ? 7.0f : 0.0f;
  static_assert(LPS >= 1 && LPS * 64 * C::WR == 2 * C::SS * RCPR && (C::NST - 1) * LPS < 64, "whole loads");

  const AttnBase& a;
  char* lds;
  AttnRows<C::ROWS>* rows;
  int wave, lane, wr, kg, n16, g;
  // the segment
  int r, h, len, n_units, rb;
  AttnUnits un;
  bool idle;                   // no row of the wave exists
  bool odd_seen;               // a masked tile held values that are not finite
  u32x4 q[C::RT][QC];
  f32x4 o[C::RT][DT];
  float m[C::RT], l[C::RT];
  float c_ctx, c_span, vs;
  uint32_t head_groups;        // groups of 16 rows of a page of all heads
  uint32_t h_groups;           // and those ahead of this head's
  uint32_t ring;               // SB bits a started tile: 16-slot groups whose page is there
  int next;                    // next tile to start
  int pg[SB];                  // pages of the next tile to load

  __device__ __forceinline__ AttnBlock(const AttnBase& args, char* l_, AttnRows<C::ROWS>* rows_) : a(args), lds(l_), rows(rows_) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    wr = wave % C::WR;
    kg = wave / C::WR;
    n16 = lane & 15;
    g = lane >> 4;
  }

  // Slot of tile u where this wave group starts.
  __device__ __forceinline__ int slot0(int u) const { return (un.first + u) * C::TS + kg * C::SS; }

  // In a scalar register: the compiler keeps some uniform numbers in vector
  // ones, with the arithmetic on them.
  static __device__ __forceinline__ uint32_t uniform_int(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

  // Page numbers of context tile u: scalar loads, nothing waits for them here.
  __device__ __forceinline__ void fetch_pages(int u) {
    typedef const __attribute__((address_space(4))) int32_t* cptr;
    const cptr table = (cptr)(a.page_table + static_cast<int64_t>(r) * a.table_len);
#pragma unroll
    for (int i = 0; i < SB; ++i) {
      const int j = slot0(u) + 16 * i;
      pg[i] = table[min(j >> a.page_shift, a.table_len - 1)];
    }
  }

  // Where the rows of context tile u (whose pages were fetched) are in the
  // caches, in bytes, by groups of 16; which groups' pages are there (others
  // stand for the first page). A group's number counts 16-row groups: page
  // times heads times groups of a page, and so on.
  __device__ __forceinline__ uint32_t page_rows(int u, int64_t (&at)[SB]) const {
    uint32_t there = 0;
#pragma unroll
    for (int i = 0; i < SB; ++i) {
      const bool ok = static_cast<uint32_t>(pg[i]) < static_cast<uint32_t>(a.n_pages) && slot0(u) + 16 * i < len;
      there |= ok ? 1u << i : 0u;
      const uint32_t in_page = ((slot0(u) >> 4) + i) & ((1u << (a.page_shift - 4)) - 1);
      const uint32_t group = uniform_int((ok ? pg[i] : 0) * uniform_int(head_groups) + uniform_int(h_groups) + in_page);
      at[i] = static_cast<int64_t>(group) * (16 * D * CSZ);
    }
    return there;
  }

  // Starts the loads of tile u into its place of the ring.
  __device__ __forceinline__ void issue(int u, int i_ring) {
    char* const dst = lds + i_ring * C::RAW + kg * (C::RAW / C::WK);
    const bool span = u >= un.ctx;
    if (!span) {
      int64_t at[SB];
      ring = uniform_int(ring << SB | page_rows(u, at));
      constexpr int kRows = 64 * C::WR / RCPR;              // rows that one load of all the group's waves covers
      const uint32_t row_l = wr * (64 / RCPR) + static_cast<uint32_t>(lane) / RCPR;   // the lane's among them
#pragma unroll
      for (int i = 0; i < LPS; ++i) {
        const int p0 = (i * C::WR + wr) * 64;               // first piece of this load
        // Its group of 16 rows: known here where the waves' rows fit in one.
        const int row0 = kRows <= 16 ? i * kRows : p0 / RCPR;
        const bool is_v = row0 >= C::SS;
        const int grp = (row0 % C::SS) / 16;
        int64_t off64 = at[0];
#pragma unroll
        for (int x = 1; x < SB; ++x) off64 = grp == x ? at[x] : off64;
        const char* const base = (is_v ? a.v_cache : a.k_cache) + off64;
        const uint32_t row = i * kRows + row_l;
        const uint32_t c = (static_cast<uint32_t>(lane) % RCPR) ^ swizzle<RCPR>(row);
        const uint32_t off = (row & 15) * (D * CSZ) + c * 16;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + off),
                                         (__attribute__((address_space(3))) void*)(dst + p0 * 16), 16, 0, 0);
      }
    } else if constexpr (KIND != kF8) {
      ring <<= SB;
#pragma unroll
      for (int i = 0; i < LPS; ++i) {
        const int p0 = (i * C::WR + wr) * 64;
        const char* src = span_piece(u, p0 + lane);
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                         (__attribute__((address_space(3))) void*)(dst + p0 * 16), 16, 0, 0);
      }
    }
  }

  // Address of piece p of the wave group's part of span tile u, permuted;
  // rows behind the span repeat its last one.
  __device__ __forceinline__ const char* span_piece(int u, int p) const {
    p = fresh(p);
    const int row = p / CPR;
    const int c = (p % CPR) ^ swizzle<CPR>(row);
    const int s = min((u - un.ctx) * C::TS + kg * C::SS + row % C::SS, a.n_pos - 1);
    const bool is_v = row >= C::SS;
    const int64_t at = (static_cast<int64_t>(r) * a.n_pos + s) * (is_v ? a.v_stride : a.k_stride) +
                       static_cast<int64_t>(h) * D;
    return static_cast<const char*>(is_v ? a.v : a.k) + at * ESZ + c * 16;
  }

  // e4m3 caches: the wave's part of a span tile, which is of the span's type,
  // to the start of the ring.
  __device__ __forceinline__ void issue_span(int u) {
    char* const dst = lds + kg * (C::STAGE / C::WK);
#pragma unroll
    for (int i = 0; i < SPS; ++i) {
      const int p0 = (i * C::WR + wr) * 64;
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)span_piece(u, p0 + lane),
                                       (__attribute__((address_space(3))) void*)(dst + p0 * 16), 16, 0, 0);
    }
  }

  // Query rows of the segment: pieces, and what masks need to know.
  __device__ __forceinline__ void load_rows() {
    const int n16 = fresh(this->n16), g = fresh(this->g);
    idle = rb * C::ROWS + wr * (16 * C::RT) >= a.rows;
    odd_seen = false;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      const int row = rb * C::ROWS + (wr * C::RT + rt) * 16 + n16;
      const bool on = row < a.rows;
      const int t = on ? row / a.group : 0;
      const int hq = h * a.group + (on ? row - t * a.group : 0);
      const char* src = static_cast<const char*>(a.q) +
                        ((static_cast<int64_t>(r) * a.n_pos + t) * a.q_stride + static_cast<int64_t>(hq) * D) * ESZ;
#pragma unroll
      for (int c = 0; c < QC; ++c) {
        q[rt][c] = u32x4{};
        if (on) q[rt][c] = *reinterpret_cast<const u32x4*>(src + (step_piece(c) + (KIND == kF8 ? 2 * g : g)) * 16);
      }
      m[rt] = -__builtin_inff();
      l[rt] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[rt][dt] = f32x4{};
    }
  }
  // Waits for the rows (and scales) here: in the tile loop, a wait for a load
  // of the past would be a wait for the tiles on their way.
  static __device__ __forceinline__ float uniform(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
  }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
      for (int c = 0; c < QC; ++c) asm volatile("" : "+v"(q[rt][c]));
    vs = uniform(vs);
    c_ctx = uniform(c_ctx);
  }
  template <bool TREE> __device__ __forceinline__ void mask_rows(const int8_t* par) {
    if (kg != 0) return;
    const int n16 = fresh(this->n16), g = fresh(this->g);
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      const int lrow = (wr * C::RT + rt) * 16 + n16;
      const int row = rb * C::ROWS + lrow;
      const bool on = row < a.rows;
      const int t = on ? row / a.group : 0;
      uint64_t path = 0;
      int dep = 0;
      if constexpr (TREE) {
        int up = t;
        for (int i = 0; up >= 0; ++i, up = par[up]) {
          if (a.window == 0 || i < a.window) path |= uint64_t{1} << up;
          dep = i;
        }
      } else {
        path = ~uint64_t{0} >> (63 - t);
        if (a.window > 0 && a.window <= t) path &= ~uint64_t{0} << (t + 1 - a.window);
        dep = t;
      }
      if (g == 0) {
        rows->anc[lrow] = on ? path : 0;
        rows->first[lrow] = !on ? INT32_MAX : a.window > 0 ? max(0, len + dep - a.window + 1) : 0;
      }
    }
  }

  // Groups of 16 slots of a started context tile whose page is there.
  __device__ __forceinline__ uint32_t here(int u) const { return (ring >> (((next - 1 - u) * SB) & 31)) & ((1u << SB) - 1); }

  // Which of a tile's slots that this lane holds count for its row (bit 4 sb
  // + i: slot 16 sb + 4 g + i of the wave group's part).
  __device__ __forceinline__ uint32_t visible(int u, int rt, bool span, uint32_t there) const {
    const int lrow = (wr * C::RT + rt) * 16 + n16;
    uint32_t bits = 0;
    if (span) {
      const uint64_t anc = rows->anc[lrow];
      const int s0 = (u - un.ctx) * C::TS + kg * C::SS + 4 * g;
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
        if (s0 + 16 * sb < 64) bits |= static_cast<uint32_t>((anc >> (s0 + 16 * sb)) & 15) << (4 * sb);
      return bits;
    }
    const int j0 = slot0(u) + 4 * g;
    const int first = rows->first[lrow];
#pragma unroll
    for (int sb = 0; sb < SB; ++sb) {
      if (!((there >> sb) & 1)) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + 16 * sb + i;
        bits |= j >= first && j < len ? 1u << (4 * sb + i) : 0u;
      }
    }
    return bits;
  }

  // Piece of a row (of the span's type) that lane group 0 takes in step c of
  // the products; group g's is g on, or 2 g with an e4m3 cache, where one
  // 16-byte read holds the keys' elements of two steps.
  static __device__ __forceinline__ constexpr int step_piece(int c) {
    return KIND == kF8 ? 8 * (c >> 1) + (c & 1) : 4 * c;
  }

  // One tile: its scores, weights and the product with the values. F8: the
  // tile is e4m3, widened (exactly) on the way to the products, keys to bf16,
  // values to float16.
  template <bool F8> __device__ __forceinline__ void tile(int u, const char* base, bool span, bool mask, uint32_t there) {
    constexpr int EB = F8 ? 1 : ESZ, ROW = D * EB, PIECES = ROW / 16;
    constexpr bool kRare = KIND == kF8 && !F8;       // a span tile after the loop over the cache's
    constexpr bool kFew = kRare || (F8 && C::RT > 2);
    const int lane = kFew ? fresh(this->lane) : this->lane, n16 = lane & 15, g = lane >> 4;
    const char* const kt = base + kg * (2 * C::SS * ROW);
    const char* const vt = kt + C::SS * ROW;
    f32x4 s[C::RT][SB];
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) s[rt][sb] = f32x4{};
    // The lane's piece of row n16 in step 0, permuted: the permutation is an
    // exclusive or of address bits, so the steps' pieces are one address apart
    // from constants.
    const uint32_t ka = lds_address(kt) + n16 * ROW + (((kRare ? 2 * g : g) ^ swizzle<PIECES>(n16)) << 4);
    u32x4 kk[F8 ? QC / 2 : QC][SB];
#pragma unroll
    for (int c = 0; c < (F8 ? QC / 2 : QC); ++c)
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) kk[c][sb] = *lds_at<u32x4>((ka ^ ((F8 ? 4 * c : step_piece(c)) << 4)) + sb * 16 * ROW);
#pragma unroll
    for (int c = 0; c < QC; ++c)
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
        u32x4 k;
        if constexpr (F8) k = widen8(kk[c / 2][sb][2 * (c & 1)], kk[c / 2][sb][2 * (c & 1) + 1]);
        else k = kk[c][sb];
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt) {
          if constexpr (KIND == kF32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[rt][sb] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[e]), __uint_as_float(q[rt][c][e]),
                                                               s[rt][sb], 0, 0, 0);
          } else {
            s[rt][sb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k),
                                                                __builtin_bit_cast(bf16x8, q[rt][c]), s[rt][sb], 0, 0, 0);
          }
        }
      }
    // The values' reads go out before the weights are formed.
    Values<F8> v;
    if constexpr (KIND != kF32) v.load(vt, n16, g, 0);
    // c S - m is one operation on the raw products; c is positive (a negative
    // one turns the products' sign, one that is not a number goes to them: the
    // scores that do not count must not have it).
    float c = span ? c_span : c_ctx;
    if (!(c >= 0.0f)) {
      const float turn = c < 0.0f ? -1.0f : c;
      c = -c;
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) s[rt][sb] *= turn;
    }
    c = fmaxf(c, 1e-37f);          // masked scores stay below everything at a scale of zero (or NaN)
    if (mask) {
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt) {
        const uint32_t seen = visible(u, rt, span, there);
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen >> (4 * sb + i)) & 1)) s[rt][sb][i] = -__builtin_inff();
      }
    }
    float top[C::RT];
    bool more = false;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      top[rt] = -__builtin_inff();
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top[rt] = fmaxf(top[rt], s[rt][sb][i]);
      top[rt] *= c;
      more = more || top[rt] - m[rt] > 8.0f;
    }
    if (__any(more)) {
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt) {
        // Only the rows that ask for it: moved along with its neighbours, a
        // row's rounding would depend on scores that it does not count.
        const float mt = row_max(top[rt]);
        const bool moves = mt - m[rt] > 8.0f;
        const float keep = moves ? __builtin_amdgcn_exp2f(m[rt] - mt) : 1.0f;
        m[rt] = moves ? mt : m[rt];
        l[rt] *= keep;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[rt][dt] *= keep;
      }
    }
    // Far out the rounding of c S in m is whole powers of two beside the
    // unrounded one: rounded alike, and lifted afterwards, P stays within its
    // range. The other rows' arguments are what they would be.
    float mb[C::RT];
    bool far = false;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      mb[rt] = m[rt] == -__builtin_inff() ? 0.0f : m[rt];
      far = far || fabsf(mb[rt]) >= 0x1p22f;
      mb[rt] -= kLift;
    }
    if (__any(far)) {
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt) {
        const bool own = fabsf(m[rt]) >= 0x1p22f && m[rt] != -__builtin_inff();
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = s[rt][sb][i];
            s[rt][sb][i] = own ? (x * c - m[rt]) + kLift : fmaf(x, c, -mb[rt]);
          }
        mb[rt] = 0.0f;
      }
      c = 1.0f;
    }
    // P^T as the products' second operand. float16 beside e4m3 values, which
    // it holds exactly as well; beside bf16 values two bf16 parts, the upper
    // bits and what they leave (and 2^-40 of P, so that it is positive where P
    // is: infinite values must not meet a zero).
    u32x2 pb[C::RT][F8 ? 1 : 2][SB];
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      float sum = 0.0f;
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(fmaf(s[rt][sb][i], c, -mb[rt]));
          sum += p;
          s[rt][sb][i] = p;
        }
        const f32x4 p = s[rt][sb];
        if constexpr (F8) {
          pb[rt][0][sb] = u32x2{pack_f16(p[0], p[1]), pack_f16(p[2], p[3])};
        } else if constexpr (KIND != kF32) {
          auto rest = [&](int i) {
            return fmaf(p[i], 0x1p-40f, p[i] - __uint_as_float(__float_as_uint(p[i]) & 0xFFFF0000u));
          };
          auto upper = [&](int i) { return __builtin_amdgcn_perm(__float_as_uint(p[i + 1]), __float_as_uint(p[i]), 0x07060302u); };
          pb[rt][0][sb] = u32x2{upper(0), upper(2)};
          pb[rt][1][sb] = u32x2{pack_bf16(rest(0), rest(1)), pack_bf16(rest(2), rest(3))};
        }
      }
      l[rt] += sum;
    }
    if constexpr (KIND == kF32) {
      values_f32(vt, s, mask);
    } else {
#pragma unroll
      for (int half = 0; half < kHalves; ++half) {
        if (half > 0) v.load(vt, n16, g, half);
        if (mask) odd_seen = __any(v.drop_odd()) || odd_seen;
        values_16<F8>(v, half, pb);
      }
    }
  }

  // Eight e4m3 numbers as bf16.
  static __device__ __forceinline__ uint32_t widen2(uint32_t w, bool high) {
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
  }
  // Two of them as float16.
  static __device__ __forceinline__ uint32_t widen2_f16(uint32_t w, bool high) {
    return __builtin_bit_cast(uint32_t, high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
                                             : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
  }
  // Two float32 rounded to float16 (nearest), the first in the low half.
  static __device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(lo), static_cast<_Float16>(hi)});
  }
  static __device__ __forceinline__ u32x4 widen8(uint32_t a, uint32_t b) {
    return u32x4{widen2(a, false), widen2(a, true), widen2(b, false), widen2(b, true)};
  }

  // The values of a tile (or of 128 of its 256 columns) as a lane reads them:
  // kCols consecutive elements, from kCols n16 on, of the slots 4 g + j and 16
  // + 4 g + j. Element x of all of them is the lane's part of V^T for the
  // columns kCols r + x, r = 0 .. 15: the lane's rows turned into columns by
  // byte permutations (one a word of bf16; of e4m3 one for two columns of two
  // rows, which the widening takes apart). (The transposing LDS read gives the
  // same without the permutations, but the compiler waits for every load to
  // LDS on its way ahead of it, and in assembly it has to be waited for on the
  // spot.)
  static constexpr int kCols = D >= 128 ? 8 : 4;
  static constexpr int kHalves = D / (16 * kCols);
  template <bool F8> struct Values {
    static constexpr int EB = F8 ? 1 : 2, ROW = D * EB;
    static constexpr int RUN = kCols * EB;                  // bytes of a read
    static constexpr int WORDS = RUN / 4;
    uint32_t w[SB][4][WORDS];
    __device__ __forceinline__ void load(const char* vt, int n16, int g, int half) {
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 4 * g + j;       // 16 rows on: the same permutation
          const int byte = half * (16 * RUN) + n16 * RUN;
          const uint32_t at = lds_address(vt) + row * ROW + (((byte >> 4) ^ swizzle<ROW / 16>(row)) << 4) + (byte & 15) +
                              sb * 16 * ROW;
          if constexpr (WORDS == 4) {
            const u32x4 x = *lds_at<u32x4>(at);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[sb][j][e] = x[e];
          } else if constexpr (WORDS == 2) {
            const u32x2 x = *lds_at<u32x2>(at);
#pragma unroll
            for (int e = 0; e < 2; ++e) w[sb][j][e] = x[e];
          } else {
            w[sb][j][0] = *lds_at<uint32_t>(at);
          }
        }
    }
    // Values that are not finite leave the product (0 * inf); whether there
    // were any.
    __device__ __forceinline__ bool drop_odd() {
      uint32_t dropped = 0;
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < WORDS; ++e) {
            const uint32_t y = w[sb][j][e];
            if constexpr (F8) {
              const uint32_t odd = ((y & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // 0x7F with either sign
              w[sb][j][e] = y & ~(odd | (odd - (odd >> 7)));
            } else {
              w[sb][j][e] = ((y & 0x7F80u) == 0x7F80u ? 0u : y & 0xFFFFu) |
                            ((y & 0x7F800000u) == 0x7F800000u ? 0u : y & 0xFFFF0000u);
            }
            dropped |= w[sb][j][e] ^ y;
          }
      return dropped != 0;
    }
    // Words 2 sb and 2 sb + 1 of the operand for element x.
    __device__ __forceinline__ u32x2 operand(int sb, int x) const {
      if constexpr (F8) {
        const uint32_t sel = x & 2 ? 0x07030602u : 0x05010400u;
        return u32x2{widen2_f16(__builtin_amdgcn_perm(w[sb][1][x >> 2], w[sb][0][x >> 2], sel), x & 1),
                     widen2_f16(__builtin_amdgcn_perm(w[sb][3][x >> 2], w[sb][2][x >> 2], sel), x & 1)};
      } else {
        const uint32_t sel = x & 1 ? 0x07060302u : 0x05040100u;
        return u32x2{__builtin_amdgcn_perm(w[sb][1][x >> 1], w[sb][0][x >> 1], sel),
                     __builtin_amdgcn_perm(w[sb][3][x >> 1], w[sb][2][x >> 1], sel)};
      }
    }
  };

  // O^T += V^T P^T. P in two parts: both in one product where a tile has 16
  // slots of a wave, otherwise the second ones behind all columns' first.
  template <bool F8>
  __device__ __forceinline__ void values_16(const Values<F8>& v, int half, const u32x2 (&pb)[C::RT][F8 ? 1 : 2][SB]) {
    constexpr int STEPS = F8 ? 1 : SB, AT = STEPS == 1 ? 1 : kCols;
#pragma unroll
    for (int x0 = 0; x0 < kCols; x0 += AT) {
      u32x2 w[AT][SB];
#pragma unroll
      for (int x = 0; x < AT; ++x)
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) w[x][sb] = v.operand(sb, x0 + x);
#pragma unroll
      for (int part = 0; part < STEPS; ++part)
#pragma unroll
        for (int x = 0; x < AT; ++x)
#pragma unroll
          for (int rt = 0; rt < C::RT; ++rt) {
            f32x4& acc = o[rt][half * kCols + x0 + x];
            if constexpr (F8) acc = product_f16(w[x], pb[rt][0], acc);
            else if constexpr (SB == 1) acc = product_bf16(w[x][0], w[x][0], pb[rt][0][0], pb[rt][1][0], acc);
            else acc = product_bf16(w[x][0], w[x][1], pb[rt][part][0], pb[rt][part][1], acc);
          }
    }
  }
  static __device__ __forceinline__ f32x4 product_bf16(u32x2 w0, u32x2 w1, u32x2 p0, u32x2 p1, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, u32x4{w0.x, w0.y, w1.x, w1.y}),
                                                   __builtin_bit_cast(bf16x8, u32x4{p0.x, p0.y, p1.x, p1.y}), acc, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 product_f16(const u32x2 (&w)[SB], const u32x2 (&p)[SB], f32x4 acc) {
    if constexpr (SB == 1)
      return __builtin_amdgcn_mfma_f32_16x16x16f16(__builtin_bit_cast(f16x4, w[0]), __builtin_bit_cast(f16x4, p[0]), acc, 0,
                                                   0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(
          __builtin_bit_cast(f16x8, u32x4{w[0].x, w[0].y, w[SB - 1].x, w[SB - 1].y}),
          __builtin_bit_cast(f16x8, u32x4{p[0].x, p[0].y, p[SB - 1].x, p[SB - 1].y}), acc, 0, 0, 0);
  }

  // The same for float32: row 16 sb + 4 g + i, column 16 dt + n16.
  __device__ __forceinline__ void values_f32(const char* vt, const f32x4 (&s)[C::RT][SB], bool mask) {
    uint32_t va[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      va[i] = lds_address(vt) + (4 * g + i) * (D * 4) + (((n16 >> 2) ^ swizzle<CPR>(4 * g + i)) << 4) + (n16 & 3) * 4;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      float v[SB][4];
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[sb][i] = *lds_at<float>((va[i] ^ (dt << 6)) + sb * 16 * D * 4);
      if (mask) {
        bool dropped = false;
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dropped = dropped || not_finite(v[sb][i]);
            v[sb][i] = not_finite(v[sb][i]) ? 0.0f : v[sb][i];
          }
        odd_seen = __any(dropped) || odd_seen;
      }
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int rt = 0; rt < C::RT; ++rt)
            o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x4f32(v[sb][i], s[rt][sb][i], o[rt][dt], 0, 0, 0);
    }
  }

  // After the segment, where a masked tile held values that are not finite and
  // left them out (rare): they are added for the rows that count
  // their slots, one slot after the other.
  __device__ __forceinline__ void add_odd(int i0, int i1) {
    const int n16 = fresh(this->n16), g = fresh(this->g);
#pragma unroll 1
    for (int u = i0; u < i1; ++u) {
      const bool span = u >= un.ctx;
      uint32_t there = 0;
      int64_t at[SB];
      if (!span) {
        fetch_pages(u);
        there = page_rows(u, at);
        if (!masked(u, there)) continue;
      }
      uint32_t seen[C::RT];
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt) seen[rt] = visible(u, rt, span, there);
#pragma unroll 1
      for (int x = 0; x < C::SS; ++x) {
        const int bit = 4 * (x / 16) + x % 4, from = (x % 16) / 4 * 16 + n16;
        bool vis[C::RT], any = false;
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt) {
          vis[rt] = (__shfl(seen[rt], from) >> bit) & 1;
          any = any || vis[rt];
        }
        if (!__any(any)) continue;
        const char* row;
        if (span) {
          const int s = min((u - un.ctx) * C::TS + kg * C::SS + x, a.n_pos - 1);
          row = static_cast<const char*>(a.v) +
                ((static_cast<int64_t>(r) * a.n_pos + s) * a.v_stride + static_cast<int64_t>(h) * D) * ESZ;
        } else {
          row = a.v_cache + at[SB > 1 && x >= 16 ? SB - 1 : 0] + (x % 16) * (D * CSZ);
        }
#pragma unroll
        for (int j = 0; j < D / 16 / kRun * 4; ++j)
#pragma unroll
          for (int e = 0; e < kRun; ++e) {
            const int col = run_column(j, g) + e;
            float y;
            if (KIND == kF32) y = reinterpret_cast<const float*>(row)[col];
            else if (KIND == kB16 || span) y = bf16_one(reinterpret_cast<const uint16_t*>(row)[col]);
            else y = (reinterpret_cast<const uint8_t*>(row)[col] & 0x7F) == 0x7F ? __builtin_nanf("") : 0.0f;
#pragma unroll
            for (int rt = 0; rt < C::RT; ++rt) o[rt][KIND == kF32 ? j : j / 4 * kRun + e][KIND == kF32 ? e : j % 4] += vis[rt] && not_finite(y) ? y : 0.0f;
          }
      }
    }
  }

  // Whether some row of the block does not count some slot of context tile u.
  __device__ __forceinline__ bool masked(int u, uint32_t there) const {
    const int j0 = slot0(u);
    return j0 + C::SS > len || (a.window > 0 && j0 <= len + a.n_pos - 1 - a.window) || there != (1u << SB) - 1;
  }

  // Tile u of the ring (an e4m3 cache's span tiles do not pass through it).
  __device__ __forceinline__ void compute(int u, const char* base) {
    if (idle) return;
    const bool span = KIND != kF8 && u >= un.ctx;
    const uint32_t there = here(u);
    tile<KIND == kF8>(u, base, span, span || masked(u, there), there);
  }

  // Waits for a tile of this wave's loads with `after` later tiles on their way.
  static __device__ __forceinline__ void wait_tile(int after) {
    if (C::NST > 3 && after >= 3) wait_vm<(C::NST > 3 ? 3 : 0) * LPS>();
    else if (C::NST > 2 && after == 2) wait_vm<(C::NST > 2 ? 2 : 0) * LPS>();
    else if (after == 1) wait_vm<LPS>();
    else wait_vm<0>();
  }

  // The next tile of units [i0, i1) on its way, if there is one.
  __device__ __forceinline__ void start(int i0, int i1) {
    const int loaded = KIND == kF8 ? min(i1, un.ctx) : i1;   // tiles that pass through the ring
    if (next < loaded) {
      issue(next, static_cast<uint32_t>(next - i0) % C::NST);
      ++next;
      if (next < un.ctx && next < loaded) fetch_pages(next);
    }
  }
  // The first tiles of the segment; pages of the very first were fetched.
  __device__ __forceinline__ void start_ring(int i0, int i1) {
    ring = 0;
    next = i0;
    for (int x = 0; x < C::NST - 1; ++x) start(i0, i1);
  }

  // Units [i0, i1) of the segment; the ring was started.
  __device__ __forceinline__ void run(int i0, int i1) {
    const int loaded = KIND == kF8 ? min(i1, un.ctx) : i1;
    for (int u = i0; u < loaded; ++u) {
      wait_tile(next - 1 - u);
      if (C::WR > 1) block_barrier();
      else wait_lds();
      start(i0, i1);
      mem_fence();
      compute(u, lds + (static_cast<uint32_t>(u - i0) % C::NST) * C::RAW);
      mem_fence();
    }
    if constexpr (KIND == kF8) {
      // The values' scale, once for all tiles of the cache, of the rows that
      // count a slot of them (the others' sums are zero, the scale may be
      // anything).
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt) {
        const float f = m[rt] == -__builtin_inff() ? 1.0f : vs;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[rt][dt] *= f;
      }
      for (int u = max(i0, un.ctx); u < i1; ++u) {
        block_barrier();
        issue_span(u);
        wait_vm<0>();
        block_barrier();
        if (!idle) tile<false>(u, lds, true, true, 0);
      }
    }
  }

  // The segment's result (whole) or its part for the join kernel. The wave
  // groups' sums are added in halves: a lane of one group takes over what the
  // same lane of another group holds, so LDS is used in order of the lanes.
  __device__ __forceinline__ void finish(bool whole, int slot) {
    constexpr int kLanes = C::WR * C::RT * 64;       // lanes and row tiles of a group
    const int n16 = fresh(this->n16), g = fresh(this->g), lane = fresh(this->lane);
#pragma unroll
    for (int half = C::WK / 2; half >= 1; half >>= 1) {
      block_barrier();
      const int from = (kg >= half ? kg - half : kg) * kLanes;
      f32x4* const sums = reinterpret_cast<f32x4*>(lds);
      float2* const ml = reinterpret_cast<float2*>(lds + C::WK / 2 * kLanes * D);
      if (!idle && kg >= half && kg < 2 * half) {
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt) {
          const int at = from + (wr * C::RT + rt) * 64 + lane;
          ml[at] = float2{m[rt], l[rt]};
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) sums[(from + (wr * C::RT + rt) * 64) * DT + dt * 64 + lane] = o[rt][dt];
        }
      }
      block_barrier();
      if (!idle && kg < half) {
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt) {
          const float2 w = ml[from + (wr * C::RT + rt) * 64 + lane];
          const float M = fmaxf(m[rt], w.x);
          const float mb = M == -__builtin_inff() ? 0.0f : M;
          const float f0 = __builtin_amdgcn_exp2f(m[rt] - mb), f1 = __builtin_amdgcn_exp2f(w.x - mb);
          m[rt] = M;
          l[rt] = l[rt] * f0 + w.y * f1;
#pragma unroll
          for (int dt = 0; dt < DT; ++dt)
            o[rt][dt] = o[rt][dt] * f0 + sums[(from + (wr * C::RT + rt) * 64) * DT + dt * 64 + lane] * f1;
        }
      }
    }
    if (idle || kg != 0) return;
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      const float ls = row_sum(l[rt]);
      const int row = (wr * C::RT + rt) * 16 + n16;
      if (whole) {
        if (rb * C::ROWS + row >= a.rows) continue;
        const int at_row = rb * C::ROWS + row;
        const int t = at_row / a.group, hq = h * a.group + at_row - t * a.group;
        const float inv = 1.0f / ls;      // scores of -inf alone: 0 * inf, as the formula's 0 / 0
        const int64_t at = ((static_cast<int64_t>(r) * a.n_pos + t) * (a.kvheads * a.group) + hq) * D;
#pragma unroll
        for (int j = 0; j < D / 16 / kRun * 4; ++j) {
          float y[kRun];
#pragma unroll
          for (int e = 0; e < kRun; ++e) y[e] = run_at(o[rt], j, e) * inv;
          if constexpr (KIND == kF32) {
            *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at + run_column(j, g)) = f32x4{y[0], y[1], y[2], y[3]};
          } else {
            uint32_t* const to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at + run_column(j, g));
            if constexpr (kRun == 8)
              *reinterpret_cast<u32x4*>(to) = u32x4{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                                                    pack_bf16(y[6], y[7])};
            else
              *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
          }
        }
      } else {
        // In the order of the lanes: whole lines per store; the join undoes it.
        f32x4* const at = reinterpret_cast<f32x4*>(a.part) +
                          (static_cast<int64_t>(slot) * (C::ROWS / 16) + wr * C::RT + rt) * (DT * 64) + lane;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) at[dt * 64] = o[rt][dt];
        if (g == 0) a.part_ml[slot * C::ROWS + row] = float2{m[rt], ls};
      }
    }
  }

  // A lane's sums by runs of consecutive columns: float32 holds columns 16 j +
  // 4 g + e in one register group, bf16 columns 16 kRun half + kRun (4 g + i) +
  // e in element i of kRun of them (j = 4 half + i).
  static constexpr int kRun = KIND == kF32 ? 4 : kCols;
  static __device__ __forceinline__ float run_at(const f32x4 (&sum)[DT], int j, int e) {
    return KIND == kF32 ? sum[j][e] : sum[j / 4 * kRun + e][j % 4];
  }
  static __device__ __forceinline__ int run_column(int j, int g) {
    return KIND == kF32 ? 16 * j + 4 * g : 16 * kRun * (j / 4) + kRun * (4 * g + j % 4);
  }
};

// The units of up to 256 requests, four consecutive ones a lane, the same in
// every wave: no barrier and one round of loads.
struct AttnPlan {
  int len[kAttnReqs / 64], all[kAttnReqs / 64];
  int before;     // units before the lane's requests
  int total;

  __device__ __forceinline__ AttnPlan(const AttnLens& a, int ts) {
    const int lane = fresh(threadIdx.x) & 63;
#pragma unroll
    for (int k = 0; k < kAttnReqs / 64; ++k) len[k] = a.len[min(lane * (kAttnReqs / 64) + k, a.n - 1)];
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kAttnReqs / 64; ++k) {
      const int n = attn_units(a, len[k], ts).all * a.heads;
      all[k] = lane * (kAttnReqs / 64) + k < a.n ? n : 0;
      sum += all[k];
    }
    // Inclusive sum over the lanes: within rows of 16, then across them.
    int c = sum;
    c += __builtin_amdgcn_update_dpp(0, c, 0x111, 0xF, 0xF, false);
    c += __builtin_amdgcn_update_dpp(0, c, 0x112, 0xF, 0xF, false);
    c += __builtin_amdgcn_update_dpp(0, c, 0x114, 0xF, 0xF, false);
    c += __builtin_amdgcn_update_dpp(0, c, 0x118, 0xF, 0xF, false);
    c += __builtin_amdgcn_update_dpp(0, c, 0x142, 0xA, 0xF, false);
    c += __builtin_amdgcn_update_dpp(0, c, 0x143, 0xC, 0xF, false);
    before = c - sum;
    total = __builtin_amdgcn_readlane(c, 63);
  }

  // For the join kernel: units before every request, and the total.
  __device__ __forceinline__ void write(int32_t* plan, int n) const {
    if (threadIdx.x >= 64) return;
    int at = before;
#pragma unroll
    for (int k = 0; k < kAttnReqs / 64; ++k) {
      const int i = threadIdx.x * (kAttnReqs / 64) + k;
      if (i <= n) plan[i] = at;
      at += all[k];
    }
    if (threadIdx.x == 63 && n == kAttnReqs) plan[kAttnReqs] = at;
  }

  // Request of unit u (uniform, below the total), the unit's number in it and
  // the request's length.
  __device__ __forceinline__ int find(int u, int* in_req, int* n) const {
    int lane_units = 0;
#pragma unroll
    for (int k = 0; k < kAttnReqs / 64; ++k) lane_units += all[k];
    const int L = __builtin_ctzll(__ballot(before + lane_units > u));
    int x = u - __builtin_amdgcn_readlane(before, L);
    int i = L * (kAttnReqs / 64);
    int at = __builtin_amdgcn_readlane(len[0], L);
    int got = 0;
#pragma unroll
    for (int k = 0; k < kAttnReqs / 64; ++k) {
      const int here = __builtin_amdgcn_readlane(all[k], L), ln = __builtin_amdgcn_readlane(len[k], L);
      if (!got) {
        at = ln;
        if (x < here) {
          got = 1;
        } else {
          x -= here;
          ++i;
        }
      }
    }
    *in_req = x;
    *n = at;
    return i;
  }
};

// Refused requests of the whole call: a count per thread, added in order.
template <int NT> __device__ __forceinline__ void count_refused(const AttnBase& a, int32_t* sums) {
  int bad = 0;
  for (int i = threadIdx.x; i < a.n_req; i += NT) {
    const int n = a.seq_len[i];
    bad += n < 0 || n > (a.table_len << a.page_shift);
  }
  sums[threadIdx.x] = bad;
  block_barrier();
  if (threadIdx.x == 0) {
    bad = 0;
    for (int i = 0; i < NT; ++i) bad += sums[i];
    *a.status = bad;
  }
  block_barrier();
}

template <int KIND, int D, int CLS, typename Args>
__global__ __launch_bounds__((AttnCfg<KIND, D, CLS>::NT), (AttnCfg<KIND, D, CLS>::NT * AttnCfg<KIND, D, CLS>::PER_CU + 255) / 256)
void attn_kernel(const int32_t* len, int n, int heads, int most, int window, int n_pos, int log_blocks, const Args args) {
  using C = AttnCfg<KIND, D, CLS>;
  constexpr bool kTree = std::is_same<Args, AttnTree>::value;
  const AttnLens lens{len, n, heads, most, window, n_pos, log_blocks};
  extern __shared__ __align__(1024) char lds[];   // rows of a tile start at multiples of their size
  __shared__ int8_t par[kTree ? HRS_MAX_POS : 1];
  __shared__ AttnRows<C::ROWS> rows;
  const int tid = threadIdx.x;
  AttnBlock<KIND, D, CLS> blk(args, lds, &rows);
  int u, u1, in_req = 0, i = 0;
  {
    const AttnPlan plan(lens, C::TS);
    u = attn_cut(blockIdx.x, plan.total, log_blocks);
    u1 = attn_cut(blockIdx.x + 1, plan.total, log_blocks);
    if (u < u1) i = plan.find(u, &in_req, &blk.len);
    if (blockIdx.x == 0) {
      plan.write(args.plan, n);
      if (args.status && args.req0 == 0) count_refused<C::NT>(args, reinterpret_cast<int32_t*>(lds));
    }
  }

  bool again = false;
  while (u < u1) {
    if (again) {
      // Counted again for every further segment rather than kept in registers
      // over the tiles; everybody is done with the last segment's tiles and
      // masks after the barrier.
      i = AttnPlan(lens, C::TS).find(u, &in_req, &blk.len);
      block_barrier();
    }
    again = true;
    blk.r = args.req0 + i;
    blk.un = attn_units(lens, blk.len, C::TS);
    const int seg = __builtin_amdgcn_readfirstlane(in_req / blk.un.all);
    const int u0 = in_req - seg * blk.un.all;
    const int ue = min(blk.un.all, u0 + (u1 - u));
    blk.h = __builtin_amdgcn_readfirstlane(seg / args.row_blocks);
    blk.rb = seg - blk.h * args.row_blocks;
    blk.head_groups = static_cast<uint32_t>(args.kvheads) << (args.page_shift - 4);
    blk.h_groups = static_cast<uint32_t>(blk.h) << (args.page_shift - 4);
    if (u0 < blk.un.ctx) blk.fetch_pages(u0);
    const float ks = KIND == kF8 && args.k_scale ? args.k_scale[blk.h] : 1.0f;
    blk.vs = KIND == kF8 && args.v_scale ? args.v_scale[blk.h] : 1.0f;
    blk.c_span = args.scale * 1.4426950408889634f;
    blk.c_ctx = blk.c_span * ks;
    blk.load_rows();
    mem_fence();
    // The tiles' part of the segment (what is left are units that stand for
    // the time that the span's masks and a segment's end take).
    const int last = min(ue, blk.un.tiles());
    blk.start_ring(u0, last);
    if constexpr (kTree) {
      if (tid < args.n_pos) par[tid] = args.parent[i * args.n_pos + tid];
      block_barrier();
    }
    blk.template mask_rows<kTree>(par);
    blk.settle();
    block_barrier();
    blk.run(u0, last);
    if (blk.odd_seen) blk.add_odd(u0, last);
    blk.finish(u0 == 0 && ue == blk.un.all, 2 * static_cast<int>(blockIdx.x) + (u0 == 0 ? 1 : 0));
    u += ue - u0;
  }
}

}  // namespace

namespace {

template <int KIND, int D, int CLS, typename Args>
void launch_as(const Args& args, const AttnLens& l, hipStream_t s) {
  using C = AttnCfg<KIND, D, CLS>;
  hipLaunchKernelGGL((attn_kernel<KIND, D, CLS, Args>), dim3(1 << l.log_blocks), dim3(C::NT), C::LDS, s, l.len, l.n, l.heads,
                     l.most, l.window, l.n_pos, l.log_blocks, args);
}
template <int KIND, int D, int CLS> void launch_one(const AttnTree& args, const AttnLens& l, hipStream_t s) {
  if (args.tree) launch_as<KIND, D, CLS>(args, l, s);
  else launch_as<KIND, D, CLS>(static_cast<const AttnBase&>(args), l, s);
}
template <int KIND, int D, int CLS> AttnShape shape_one() {
  using C = AttnCfg<KIND, D, CLS>;
  return {C::ROWS, C::TS, kAttnCus * C::PER_CU};
}

}  // namespace

template <int KIND> AttnShape attn_shape(int d, int cls) {
  switch (d * 8 + cls) {
    case 64 * 8 + 0: return shape_one<KIND, 64, 0>();
    case 64 * 8 + 1: return shape_one<KIND, 64, 1>();
    case 64 * 8 + 2: return shape_one<KIND, 64, 2>();
    case 64 * 8 + 3: return shape_one<KIND, 64, 3>();
    case 128 * 8 + 0: return shape_one<KIND, 128, 0>();
    case 128 * 8 + 1: return shape_one<KIND, 128, 1>();
    case 128 * 8 + 2: return shape_one<KIND, 128, 2>();
    case 128 * 8 + 3: return shape_one<KIND, 128, 3>();
    case 256 * 8 + 0: return shape_one<KIND, 256, 0>();
    case 256 * 8 + 1: return shape_one<KIND, 256, 1>();
    case 256 * 8 + 2: return shape_one<KIND, 256, 2>();
    case 256 * 8 + 3: return shape_one<KIND, 256, 3>();
  }
  if constexpr (KIND == kF8) {
    if (cls == 4) return d == 64 ? shape_one<KIND, 64, 4>() : shape_one<KIND, 128, 4>();
  }
  return {0, 0, 0};
}

template <int KIND> void attn_launch(const AttnTree& args, const AttnLens& lens, int d, int cls, hipStream_t s) {
  switch (d * 8 + cls) {
    case 64 * 8 + 0: return launch_one<KIND, 64, 0>(args, lens, s);
    case 64 * 8 + 1: return launch_one<KIND, 64, 1>(args, lens, s);
    case 64 * 8 + 2: return launch_one<KIND, 64, 2>(args, lens, s);
    case 64 * 8 + 3: return launch_one<KIND, 64, 3>(args, lens, s);
    case 128 * 8 + 0: return launch_one<KIND, 128, 0>(args, lens, s);
    case 128 * 8 + 1: return launch_one<KIND, 128, 1>(args, lens, s);
    case 128 * 8 + 2: return launch_one<KIND, 128, 2>(args, lens, s);
    case 128 * 8 + 3: return launch_one<KIND, 128, 3>(args, lens, s);
    case 256 * 8 + 0: return launch_one<KIND, 256, 0>(args, lens, s);
    case 256 * 8 + 1: return launch_one<KIND, 256, 1>(args, lens, s);
    case 256 * 8 + 2: return launch_one<KIND, 256, 2>(args, lens, s);
    case 256 * 8 + 3: return launch_one<KIND, 256, 3>(args, lens, s);
  }
  if constexpr (KIND == kF8) {
    if (cls == 4) return d == 64 ? launch_one<KIND, 64, 4>(args, lens, s) : launch_one<KIND, 128, 4>(args, lens, s);
  }
}

}  // namespace hrs
