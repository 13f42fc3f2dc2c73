// The kernel of attn_verify_span.
//
//   S^T = K Q^T,  P = exp2(c S - m),  O^T += V^T P^T,  l += P,  out = O / l
//
// over tiles of slots with a running reference m per query row.
//
// MI355X design. The rows of a key/value head are all query heads of its
// group at all span positions (17 positions x 6 heads = 102), so its keys and
// values are read from memory once for all of them; with few rows the job is
// bound by that read. Blocks are one per CU. The tiles of all requests and
// heads form one list that is cut into equal runs, so ragged lengths leave no
// CU idle and the host needs no lengths; a run that ends inside a head leaves
// a partial sum (f32) for the join.
//  - Tiles travel from memory to LDS without registers (16 bytes per lane), a
//    ring of tiles ahead; a wave waits for the loads it issued itself and one
//    barrier per tile makes them everybody's (none where a wave has its slots
//    to itself). Page numbers are read a tile ahead by scalar loads; a page
//    never ends inside 16 slots, so a load's base address is wave-uniform.
//  - 16-byte pieces are permuted within a row (on the memory side, since the
//    LDS side of such a load is linear) so that the 16 rows of an operand lie
//    in different banks.
//  - The transposed products need no data movement between them: a lane of
//    S^T holds one query row's scores of four consecutive slots, which is the
//    layout of P^T as the second operand when the slots of a 32-slot step are
//    taken in the order 4 g + i, 16 + 4 g + i; V^T in that order is what the
//    transposing LDS read returns. Row maxima and the rescaling of O are
//    per-lane numbers.
//  - The reference m moves only when a row's maximum exceeds it by more than
//    8 (in log2), so most tiles neither reduce across lanes nor rescale; P is
//    at most 2^8 and l and O are f32, which loses nothing.
//  - e4m3 tiles are widened to bf16 once per block, from a ring of raw tiles
//    to the tile that the products read (the scales are factors of c and P).
//  - Tiles with a mask (the span, the context's end, a window's border,
//    absent pages) take a second form of the tile: scores that do not count
//    are dropped, and values that are not finite leave the product (0 * NaN)
//    and are added back for the rows that count them.
#pragma once

#include "attn.h"

namespace hrs {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ void mem_fence() { asm volatile("" ::: "memory"); }

// Waits until at most n of this wave's vector memory operations are on their
// way (they end in order).
template <int N> __device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// All waves' LDS writes before, all reads after.
__device__ __forceinline__ void block_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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

// Within each group of 16 lanes, lane i receives as its j-th value element
// i % 4 of the four 16-bit values that lane 4 j + i / 4 addresses.
__device__ __forceinline__ u32x2 read_tr16(uint32_t a) {
  const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)a);
  return __builtin_bit_cast(u32x2, v);
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
template <int CPR> __device__ __forceinline__ int swizzle(int row) {
  return CPR >= 16 ? ((row & 7) << 1) | ((row >> 3) & 1) : (((row >> 1) & 3) << 1) | ((row >> 3) & 1);
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
  static_assert(LPS >= 1 && LPS * 64 * C::WR == 2 * C::SS * RCPR && (C::NST - 1) * LPS < 64, "whole loads");

  const AttnArgs& a;
  char* lds;
  AttnRows<C::ROWS>* rows;
  int wave, lane, wr, kg, n16, g;
  // the segment
  int r, h, len, n_units, rb;
  AttnUnits un;
  bool idle;                   // no row of the wave exists
  u32x4 q[C::RT][QC];
  f32x4 o[C::RT][DT];
  float m[C::RT], l[C::RT];
  float c_ctx, c_span, vs;
  uint32_t head_bytes;         // a page of all heads
  uint64_t h_bytes;            // this head's part of it
  uint64_t present;            // 4 bits a tile: 16-slot groups whose page is there
  int pg[SB];                  // pages of the next tile to load

  __device__ __forceinline__ AttnBlock(const AttnArgs& args, char* l_, AttnRows<C::ROWS>* rows_) : a(args), lds(l_), rows(rows_) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    wr = wave % C::WR;
    kg = wave / C::WR;
    n16 = lane & 15;
    g = lane >> 4;
  }

  // Slot of tile u where this wave group starts.
  __device__ __forceinline__ int slot0(int u) const { return (un.first + u) * C::TS + kg * C::SS; }

  // Page numbers of context tile u (scalar loads; a number of -1 for slots
  // past the length).
  __device__ __forceinline__ void fetch_pages(int u) {
    typedef const __attribute__((address_space(4))) int32_t* cptr;
    const cptr table = (cptr)(a.page_table + static_cast<int64_t>(r) * a.table_len);
#pragma unroll
    for (int i = 0; i < SB; ++i) {
      const int j = slot0(u) + 16 * i;
      const int p = table[min(j >> a.page_shift, a.table_len - 1)];
      pg[i] = j < len ? p : -1;
    }
  }

  // Starts the loads of tile u into its place of the ring.
  __device__ __forceinline__ void issue(int u, int i_ring) {
    char* const dst = lds + C::RING + i_ring * C::RAW + kg * (C::RAW / C::WK);
    const bool span = u >= un.ctx;
    if (!span) {
      uint32_t here = 0;
      int64_t at[SB];
#pragma unroll
      for (int i = 0; i < SB; ++i) {
        const bool ok = pg[i] >= 0 && pg[i] < a.n_pages;
        here |= ok ? 1u << i : 0u;
        const int in_page = (slot0(u) + 16 * i) & ((1 << a.page_shift) - 1);
        // Bytes: (page * heads + head) rows of a page, then the row.
        at[i] = static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(ok ? pg[i] : 0)) * head_bytes) +
                static_cast<int64_t>(h_bytes + static_cast<uint32_t>(in_page) * (D * CSZ));
      }
      present = (present & ~(uint64_t{15} << (4 * (u & 15)))) | (static_cast<uint64_t>(here) << (4 * (u & 15)));
      constexpr int kRows = 64 * C::WR / RCPR;              // rows that one load of all the group's waves covers
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
        const int p = p0 + lane;
        const int row = p / RCPR;
        int c = p % RCPR;
        if constexpr (KIND != kF8) c ^= swizzle<CPR>(row);
        const uint32_t off = (row & 15) * (D * CSZ) + c * 16;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + off),
                                         (__attribute__((address_space(3))) void*)(dst + p0 * 16), 16, 0, 0);
      }
    } else if constexpr (KIND != kF8) {
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
    asm volatile("" : "+v"(p));     // formed here, not kept in registers over the context's tiles
    const int row = p / CPR;
    const int c = (p % CPR) ^ swizzle<CPR>(row);
    const int s = min((u - un.ctx) * C::TS + kg * C::SS + row % C::SS, a.n_pos - 1);
    const bool is_v = row >= C::SS;
    const int64_t at = (static_cast<int64_t>(r) * a.n_pos + s) * (is_v ? a.v_stride : a.k_stride) +
                       static_cast<int64_t>(h) * D;
    return static_cast<const char*>(is_v ? a.v : a.k) + at * ESZ + c * 16;
  }

  // e4m3: the wave's own pieces of a loaded tile (or of the span) to the tile
  // that the products read.
  __device__ __forceinline__ void widen_tile(int u, int i_ring, int i_buf) {
    char* const dst = lds + i_buf * C::STAGE + kg * (C::STAGE / C::WK);
    if (u >= un.ctx) {
#pragma unroll
      for (int i = 0; i < SPS; ++i) {
        const int p = (i * C::WR + wr) * 64 + lane;
        *reinterpret_cast<u32x4*>(dst + p * 16) = *reinterpret_cast<const u32x4*>(span_piece(u, p));
      }
      return;
    }
    const char* const src = lds + C::RING + i_ring * C::RAW + kg * (C::RAW / C::WK);
#pragma unroll
    for (int i = 0; i < LPS; ++i) {
      const int p = (i * C::WR + wr) * 64 + lane;
      const u32x4 w = *reinterpret_cast<const u32x4*>(src + p * 16);
      const int row = p / RCPR, c8 = p % RCPR;
      const int f = swizzle<CPR>(row);
      u32x4 lo, hi;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        lo[2 * x] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[x], 1.0f, false));
        lo[2 * x + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[x], 1.0f, true));
        hi[2 * x] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 + x], 1.0f, false));
        hi[2 * x + 1] =
            __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 + x], 1.0f, true));
      }
      *reinterpret_cast<u32x4*>(dst + (row * CPR + ((2 * c8) ^ f)) * 16) = lo;
      *reinterpret_cast<u32x4*>(dst + (row * CPR + ((2 * c8 + 1) ^ f)) * 16) = hi;
    }
  }

  // Query rows of the segment: pieces, root paths.
  __device__ __forceinline__ void load_rows(const int8_t* par) {
    idle = rb * C::ROWS + wr * (16 * C::RT) >= a.rows;
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
        if (on) q[rt][c] = *reinterpret_cast<const u32x4*>(src + (4 * c + g) * 16);
      }
      uint64_t path = 0;
      int dep = 0;
      if (a.tree) {
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
      if (kg == 0 && g == 0) {
        rows->anc[(wr * C::RT + rt) * 16 + n16] = on ? path : 0;
        rows->first[(wr * C::RT + rt) * 16 + n16] = !on ? INT32_MAX : a.window > 0 ? max(0, len + dep - a.window + 1) : 0;
      }
      m[rt] = -__builtin_inff();
      l[rt] = 0.0f;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[rt][dt] = f32x4{};
    }
  }

  // Which of a tile's slots that this lane holds count for its row (bit 4 sb
  // + i: slot 16 sb + 4 g + i of the wave group's part).
  __device__ __forceinline__ uint32_t visible(int u, int rt, bool span) const {
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
      if (!((present >> (4 * (u & 15) + sb)) & 1)) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + 16 * sb + i;
        bits |= j >= first && j < len ? 1u << (4 * sb + i) : 0u;
      }
    }
    return bits;
  }

  // Whether the wave group's values of a tile hold an infinity or a NaN.
  __device__ __forceinline__ bool any_odd(const char* vt) const {
    bool odd = false;
#pragma unroll
    for (int x = 0; x < C::SS * CPR / 64; ++x) {
      const u32x4 w = *reinterpret_cast<const u32x4*>(vt + (x * 64 + lane) * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        odd = odd || (w[e] & 0x7F800000u) == 0x7F800000u;
        if (ESZ == 2) odd = odd || (w[e] & 0x7F80u) == 0x7F80u;
      }
    }
    return __any(odd);
  }

  // One tile: its scores, weights and the product with the values.
  __device__ __forceinline__ void tile(int u, const char* base, bool span, bool mask) {
    const char* const kt = base + kg * (C::STAGE / C::WK);
    const char* const vt = kt + C::SS * D * ESZ;
    f32x4 s[C::RT][SB];
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) s[rt][sb] = f32x4{};
    // Piece 4 c + g of row n16, permuted: the permutation is an exclusive or
    // of address bits, so the pieces are one address apart from constants.
    const uint32_t ka = lds_address(kt) + n16 * (D * ESZ) +
                        ((g ^ swizzle<CPR>(n16)) << 4);
#pragma unroll
    for (int c = 0; c < QC; ++c) {
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
        const u32x4 kk = *lds_at<u32x4>((ka ^ (c << 6)) + sb * 16 * D * ESZ);
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt) {
          if constexpr (KIND == kF32) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              s[rt][sb] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kk[e]), __uint_as_float(q[rt][c][e]),
                                                               s[rt][sb], 0, 0, 0);
          } else {
            s[rt][sb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kk),
                                                                __builtin_bit_cast(bf16x8, q[rt][c]), s[rt][sb], 0, 0, 0);
          }
        }
      }
    }
    // c S - m is one operation on the raw products; c is positive (a negative
    // one turns the products' sign).
    float c = span ? c_span : c_ctx;
    if (c < 0.0f) {
      c = -c;
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) s[rt][sb] = -s[rt][sb];
    }
    c = fmaxf(c, 1e-37f);          // masked scores stay below everything at a scale of zero
    bool odd = false;
    if (mask) {
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt) {
        const uint32_t seen = visible(u, rt, span);
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen >> (4 * sb + i)) & 1)) s[rt][sb][i] = -__builtin_inff();
      }
      odd = any_odd(vt);
    }
    u32x2 pb[C::RT][SB];       // P^T as the products' second operand (bf16)
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      float top = -__builtin_inff();
#pragma unroll
      for (int sb = 0; sb < SB; ++sb)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[rt][sb][i]);
      top *= c;
      if (__any(top > m[rt] + 8.0f)) {
        const float mn = fmaxf(m[rt], row_max(top));
        const float keep = m[rt] == mn ? 1.0f : __builtin_amdgcn_exp2f(m[rt] - mn);
        m[rt] = mn;
        l[rt] *= keep;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) o[rt][dt] *= keep;
      }
      const float mb = m[rt] == -__builtin_inff() ? 0.0f : m[rt];
      float sum = 0.0f;
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float p = __builtin_amdgcn_exp2f(fmaf(s[rt][sb][i], c, -mb));
          sum += p;
          if (KIND == kF8) p *= span ? 1.0f : vs;
          s[rt][sb][i] = p;
        }
        if constexpr (KIND != kF32)
          pb[rt][sb] = u32x2{pack_bf16(s[rt][sb][0], s[rt][sb][1]), pack_bf16(s[rt][sb][2], s[rt][sb][3])};
      }
      l[rt] += sum;
    }
    if (odd) {
      values<true>(vt, s, pb, u, span);
    } else {
      values<false>(vt, s, pb, u, span);
    }
  }

  // O^T += V^T P^T. ODD: values that are not finite leave the product; the
  // products of "counts" with "+inf or NaN" and with "-inf or NaN" say which
  // rows' sums get +inf, -inf or both (NaN).
  template <bool ODD>
  __device__ __forceinline__ void values(const char* vt, const f32x4 (&s)[C::RT][SB], const u32x2 (&pb)[C::RT][SB], int u,
                                         bool span) {
    const float inf = __builtin_inff();
    uint32_t seen[C::RT];
    if (ODD) {
#pragma unroll
      for (int rt = 0; rt < C::RT; ++rt) seen[rt] = visible(u, rt, span);
    }
    const uint32_t vb = lds_address(vt);
    if constexpr (KIND == kF32) {
      // Row 16 sb + 4 g + i, element 16 dt + n16: one address per i.
      uint32_t va[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        va[i] = vb + (4 * g + i) * (D * 4) + (((n16 >> 2) ^ swizzle<CPR>(4 * g + i)) << 4) + (n16 & 3) * 4;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        f32x4 up[C::RT], down[C::RT];
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt) up[rt] = down[rt] = f32x4{};
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = *lds_at<float>((va[i] ^ (dt << 6)) + sb * 16 * D * 4);
            if (ODD) {
              const float hi = v == inf || v != v ? 1.0f : 0.0f, lo = v == -inf || v != v ? 1.0f : 0.0f;
              v = not_finite(v) ? 0.0f : v;
#pragma unroll
              for (int rt = 0; rt < C::RT; ++rt) {
                const float p = (seen[rt] >> (4 * sb + i)) & 1 ? 1.0f : 0.0f;
                up[rt] = __builtin_amdgcn_mfma_f32_16x16x4f32(hi, p, up[rt], 0, 0, 0);
                down[rt] = __builtin_amdgcn_mfma_f32_16x16x4f32(lo, p, down[rt], 0, 0, 0);
              }
            }
#pragma unroll
            for (int rt = 0; rt < C::RT; ++rt)
              o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, s[rt][sb][i], o[rt][dt], 0, 0, 0);
          }
        if (ODD) {
#pragma unroll
          for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[rt][dt][e] += (up[rt][e] > 0.0f ? inf : 0.0f) - (down[rt][e] > 0.0f ? inf : 0.0f);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
      const int vrow = 4 * g + (n16 >> 2);
      const uint32_t va = vb + vrow * (D * ESZ) + ((((n16 & 3) >> 1) ^ swizzle<CPR>(vrow)) << 4) + (n16 & 1) * 8;
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) {
        u32x2 w[SB];
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) w[sb] = read_tr16((va ^ (dt << 5)) + sb * 16 * D * ESZ);
        if (ODD) {
          f32x4 up[C::RT], down[C::RT];
#pragma unroll
          for (int rt = 0; rt < C::RT; ++rt) up[rt] = down[rt] = f32x4{};
#pragma unroll
          for (int sb = 0; sb < SB; ++sb) {
            s16x4 hi, lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t half = (w[sb][i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
              const bool nan = (half & 0x7FFFu) > 0x7F80u;
              hi[i] = half == 0x7F80u || nan ? 0x3F80 : 0;
              lo[i] = half == 0xFF80u || nan ? 0x3F80 : 0;
              if ((half & 0x7F80u) == 0x7F80u) w[sb][i >> 1] &= 0xFFFFu << (16 * (1 - (i & 1)));
            }
#pragma unroll
            for (int rt = 0; rt < C::RT; ++rt) {
              s16x4 p;
#pragma unroll
              for (int i = 0; i < 4; ++i) p[i] = (seen[rt] >> (4 * sb + i)) & 1 ? 0x3F80 : 0;
              up[rt] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(hi, p, up[rt], 0, 0, 0);
              down[rt] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(lo, p, down[rt], 0, 0, 0);
            }
          }
#pragma unroll
          for (int rt = 0; rt < C::RT; ++rt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[rt][dt][e] += (up[rt][e] > 0.0f ? inf : 0.0f) - (down[rt][e] > 0.0f ? inf : 0.0f);
        }
#pragma unroll
        for (int rt = 0; rt < C::RT; ++rt) {
          if constexpr (SB == 1) {
            o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, w[0]),
                                                                 __builtin_bit_cast(s16x4, pb[rt][0]), o[rt][dt], 0, 0, 0);
          } else {
#pragma unroll
            for (int sb = 0; sb < SB; sb += 2)
              o[rt][dt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8, u32x4{w[sb].x, w[sb].y, w[sb + 1].x, w[sb + 1].y}),
                  __builtin_bit_cast(bf16x8, u32x4{pb[rt][sb].x, pb[rt][sb].y, pb[rt][sb + 1].x, pb[rt][sb + 1].y}),
                  o[rt][dt], 0, 0, 0);
          }
        }
        if (ODD) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  __device__ __forceinline__ bool masked(int u) const {
    if (u >= un.ctx) return true;
    const int j0 = slot0(u);
    if (j0 + C::SS > len) return true;
    if (a.window > 0 && j0 <= len + a.n_pos - 1 - a.window) return true;
    return ((present >> (4 * (u & 15))) & ((1u << SB) - 1)) != (1u << SB) - 1;
  }

  __device__ __forceinline__ void compute(int u, const char* base) {
    if (idle) return;
    tile(u, base, u >= un.ctx, masked(u));
  }

  // Waits for a tile of this wave's loads with `after` later tiles on their way.
  static __device__ __forceinline__ void wait_tile(int after) {
    if (C::NST > 3 && after >= 3) wait_vm<(C::NST > 3 ? 3 : 0) * LPS>();
    else if (C::NST > 2 && after == 2) wait_vm<(C::NST > 2 ? 2 : 0) * LPS>();
    else if (after == 1) wait_vm<LPS>();
    else wait_vm<0>();
  }

  // Units [i0, i1) of the segment.
  __device__ __forceinline__ void run(int i0, int i1) {
    present = 0;
    const int loaded = KIND == kF8 ? min(i1, un.ctx) : i1;   // tiles that pass through the ring
    int next = i0;
    auto start = [&]() {
      if (next < loaded) {
        issue(next, (next - i0) % C::NST);
        ++next;
        if (next < un.ctx && next < loaded) fetch_pages(next);
      }
    };
    if (i0 < un.ctx) fetch_pages(i0);
    if constexpr (KIND != kF8) {
      for (int x = 0; x < C::NST - 1; ++x) start();
      for (int u = i0; u < i1; ++u) {
        wait_tile(next - 1 - u);
        if (C::WR > 1) block_barrier();
        start();
        mem_fence();
        compute(u, lds + C::RING + ((u - i0) % C::NST) * C::RAW);
        mem_fence();
      }
    } else {
      for (int x = 0; x < C::NST; ++x) start();
      auto convert = [&](int u) {
        if (u < loaded) wait_tile(next - 1 - u);
        widen_tile(u, (u - i0) % C::NST, C::NB == 2 ? (u - i0) & 1 : 0);
        // The raw pieces are in registers (they were converted) before their
        // place is loaded again.
        mem_fence();
        start();
        mem_fence();
      };
      if (C::NB == 2) {
        convert(i0);
        for (int u = i0; u < i1; ++u) {
          block_barrier();
          if (u + 1 < i1) convert(u + 1);
          compute(u, lds + ((u - i0) & 1) * C::STAGE);
        }
      } else {
        for (int u = i0; u < i1; ++u) {
          convert(u);
          compute(u, lds);
          mem_fence();
        }
      }
    }
  }

  // Joins the wave groups' sums in LDS and writes the segment's result (whole)
  // or its part for the join kernel.
  __device__ __forceinline__ void finish(bool whole, int slot) {
    __syncthreads();
    float2* const ml = reinterpret_cast<float2*>(lds + C::WK * C::ROWS * C::OROW);
#pragma unroll
    for (int rt = 0; rt < C::RT; ++rt) {
      const int row = (wr * C::RT + rt) * 16 + n16;
      const float ls = row_sum(l[rt]);
      if (g == 0) ml[kg * C::ROWS + row] = float2{m[rt], ls};
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
        *reinterpret_cast<f32x4*>(lds + (kg * C::ROWS + row) * C::OROW + (dt * 16 + 4 * g) * 4) = o[rt][dt];
    }
    __syncthreads();
    const int n_rows = min(C::ROWS, a.rows - rb * C::ROWS);
    for (int x = threadIdx.x; x < n_rows * (D / 4); x += C::NT) {
      const int row = x / (D / 4), d4 = x % (D / 4);
      float M = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < C::WK; ++i) M = fmaxf(M, ml[i * C::ROWS + row].x);
      f32x4 sum = {};
      float ls = 0.0f;
#pragma unroll
      for (int i = 0; i < C::WK; ++i) {
        const float2 w = ml[i * C::ROWS + row];
        if (w.x == -__builtin_inff() && w.y == 0.0f) continue;
        const float f = w.x == M ? 1.0f : __builtin_amdgcn_exp2f(w.x - M);
        ls += w.y * f;
        sum += *reinterpret_cast<const f32x4*>(lds + (i * C::ROWS + row) * C::OROW + d4 * 16) * f;
      }
      if (whole) {
        write_out(a, r, h, rb * C::ROWS + row, d4, sum, ls);
      } else {
        *reinterpret_cast<f32x4*>(a.part + (static_cast<int64_t>(slot) * C::ROWS + row) * D + d4 * 4) = sum;
        if (d4 == 0) a.part_ml[slot * C::ROWS + row] = float2{M, ls};
      }
    }
    __syncthreads();
  }

  static __device__ __forceinline__ void write_out(const AttnArgs& a, int r, int h, int row, int d4, f32x4 sum, float ls) {
    const int t = row / a.group, hq = h * a.group + row - t * a.group;
    const float inv = ls == 0.0f ? 0.0f : 1.0f / ls;
    const f32x4 y = ls == 0.0f ? f32x4{} : sum * inv;
    const int64_t at = ((static_cast<int64_t>(r) * a.n_pos + t) * (a.kvheads * a.group) + hq) * D + d4 * 4;
    if constexpr (KIND == kF32)
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = y;
    else
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) =
          u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
  }
};

template <int KIND, int D, int CLS>
__global__ __launch_bounds__((AttnCfg<KIND, D, CLS>::NT)) void attn_kernel(const AttnArgs args) {
  using C = AttnCfg<KIND, D, CLS>;
  extern __shared__ __align__(1024) char lds[];   // rows of a tile start at multiples of their size
  __shared__ int64_t before[kAttnReqs + 1];
  __shared__ int64_t wave_sum[kAttnReqs / 64];
  __shared__ int8_t par[HRS_MAX_POS];
  __shared__ AttnRows<C::ROWS> rows;
  const int tid = threadIdx.x, lane = tid & 63;
  const int heads = args.kvheads * args.row_blocks;
  // Units before every request: a scan over the lengths, 256 at most.
  for (int i0 = 0; i0 < kAttnReqs; i0 += C::NT) {
    const int i = i0 + tid;
    if (i < kAttnReqs) {
      int len;
      int64_t x = i < args.n_here ? static_cast<int64_t>(attn_units(args, args.req0 + i, C::TS, &len).all) * heads : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up(x, d);
        x += lane >= d ? y : 0;
      }
      before[i + 1] = x;
      if (lane == 63) wave_sum[i >> 6] = x;
    }
  }
  if (tid == 0) before[0] = 0;
  __syncthreads();
  for (int i = tid; i < kAttnReqs; i += C::NT) {
    int64_t add = 0;
    for (int w = 0; w < (i >> 6); ++w) add += wave_sum[w];
    before[i + 1] += add;
  }
  __syncthreads();
  const int64_t total = before[args.n_here];
  if (blockIdx.x == 0) {
    for (int i = tid; i <= args.n_here; i += C::NT) args.plan[i] = before[i];
    if (args.status && args.req0 == 0 && tid == 0) {
      int bad = 0;
      for (int i = 0; i < args.n_req; ++i) {
        const int n = args.seq_len[i];
        bad += n < 0 || n > (args.table_len << args.page_shift);
      }
      *args.status = bad;
    }
  }
  const int64_t blocks = min(static_cast<int64_t>(gridDim.x), total);
  if (blockIdx.x >= blocks) return;
  int64_t u = blockIdx.x * total / blocks;
  const int64_t u1 = (blockIdx.x + 1) * total / blocks;
  int i = 0;                           // the request of unit u: the last with before <= u and units of its own
  for (int step = kAttnReqs / 2; step; step >>= 1)
    if (i + step < args.n_here && before[i + step] <= u) i += step;

  AttnBlock<KIND, D, CLS> blk(args, lds, &rows);
  while (u < u1) {
    while (before[i + 1] <= u) ++i;
    i = __builtin_amdgcn_readfirstlane(i);
    blk.r = args.req0 + i;
    blk.un = attn_units(args, blk.r, C::TS, &blk.len);
    const int64_t in_req = u - before[i];
    const int seg = __builtin_amdgcn_readfirstlane(static_cast<int>(in_req / blk.un.all));
    const int u0 = __builtin_amdgcn_readfirstlane(static_cast<int>(in_req - static_cast<int64_t>(seg) * blk.un.all));
    const int ue = static_cast<int>(min(static_cast<int64_t>(blk.un.all), u0 + (u1 - u)));
    blk.h = seg / args.row_blocks;
    blk.rb = seg - blk.h * args.row_blocks;
    const float ks = KIND == kF8 && args.k_scale ? args.k_scale[blk.h] : 1.0f;
    blk.vs = KIND == kF8 && args.v_scale ? args.v_scale[blk.h] : 1.0f;
    blk.c_span = args.scale * 1.4426950408889634f;
    blk.c_ctx = blk.c_span * ks;
    blk.head_bytes = static_cast<uint32_t>(args.kvheads) * (D * C::ESZC << args.page_shift);
    blk.h_bytes = static_cast<uint64_t>(blk.h) * (D * C::ESZC << args.page_shift);
    if (args.tree) {
      if (tid < args.n_pos) par[tid] = args.parent[i * args.n_pos + tid];
      __syncthreads();
    }
    blk.load_rows(par);
    __syncthreads();
    blk.run(u0, __builtin_amdgcn_readfirstlane(ue));
    blk.finish(u0 == 0 && ue == blk.un.all, 2 * static_cast<int>(blockIdx.x) + (u0 == 0 ? 1 : 0));
    u += ue - u0;
  }
}

}  // namespace

namespace {

template <int KIND, int D, int CLS>
void launch_one(const AttnArgs& args, int blocks, hipStream_t s) {
  using C = AttnCfg<KIND, D, CLS>;
  hipLaunchKernelGGL((attn_kernel<KIND, D, CLS>), dim3(blocks), dim3(C::NT), C::LDS, s, args);
}
template <int KIND, int D, int CLS> AttnShape shape_one() {
  using C = AttnCfg<KIND, D, CLS>;
  return {C::ROWS, C::TS, C::NT};
}

}  // namespace

template <int KIND> AttnShape attn_shape(int d, int cls) {
  switch (d * 4 + cls) {
    case 256: return shape_one<KIND, 64, 0>();
    case 257: return shape_one<KIND, 64, 1>();
    case 258: return shape_one<KIND, 64, 2>();
    case 259: return shape_one<KIND, 64, 3>();
    case 512: return shape_one<KIND, 128, 0>();
    case 513: return shape_one<KIND, 128, 1>();
    case 514: return shape_one<KIND, 128, 2>();
    case 515: return shape_one<KIND, 128, 3>();
    case 1024: return shape_one<KIND, 256, 0>();
    case 1025: return shape_one<KIND, 256, 1>();
    case 1026: return shape_one<KIND, 256, 2>();
    case 1027: return shape_one<KIND, 256, 3>();
    default: return {0, 0, 0};
  }
}

template <int KIND> void attn_launch(const AttnArgs& args, int d, int cls, int blocks, hipStream_t s) {
  switch (d * 4 + cls) {
    case 256: return launch_one<KIND, 64, 0>(args, blocks, s);
    case 257: return launch_one<KIND, 64, 1>(args, blocks, s);
    case 258: return launch_one<KIND, 64, 2>(args, blocks, s);
    case 259: return launch_one<KIND, 64, 3>(args, blocks, s);
    case 512: return launch_one<KIND, 128, 0>(args, blocks, s);
    case 513: return launch_one<KIND, 128, 1>(args, blocks, s);
    case 514: return launch_one<KIND, 128, 2>(args, blocks, s);
    case 515: return launch_one<KIND, 128, 3>(args, blocks, s);
    case 1024: return launch_one<KIND, 256, 0>(args, blocks, s);
    case 1025: return launch_one<KIND, 256, 1>(args, blocks, s);
    case 1026: return launch_one<KIND, 256, 2>(args, blocks, s);
    case 1027: return launch_one<KIND, 256, 3>(args, blocks, s);
  }
}

}  // namespace hrs
