// The prefix launch of attn_verify_shared for large batches.
//
//   S^T = K Q^T,  P = exp2(c S - m),  O^T += V^T P^T,  l += P
//
// for the rows (request, position, query head of a group) of all requests over
// the slots that all of them count: no masks but for absent pages.
//
// MI355X design. With hundreds of rows the matrix units' work is as long as
// everything else together, so what counts is how much of it runs at the same
// time. A wave holds RT tiles of 16 rows, their results and their queries in
// registers, and every key and value that it reads from LDS serves all of them.
// 48 rows of 128 elements, or 64 of 64, are what half a SIMD's registers hold: two
// blocks share a CU, and one's exponentials run under the other's products
// (e4m3, 23,552 rows of 128 over 8,191 slots: 131 us; 80 rows a wave and one
// block 167, 96 rows 229). 48 rows of 256 elements take all registers, and the
// wave does that for itself: the scores of the next tile are formed under this
// tile's exponentials (6,528 rows of 256 over 26,752 slots: 216 us; without that
// 298). A product lets two vector operations of its wave pass (17 cycles without
// any, 18 with two, five more for each further one), so the order of a tile's
// instructions is written down and kept, one or two behind each product (274 and
// 145 us where the compiler orders within steps of RT products, 285 and 165
// where it orders everything), the next loads are among them, and scores leave
// the matrix units' registers once (245 us without these two).
// The path for smaller batches (attn_kernel.h) takes 376 and 156 us here.
//
// Weights are rounded to 16 bits once, at most 2^-8 of a bf16 weight (2^-11 of a
// float16 one) and as likely up as down; a second part for what they lose, as
// smaller batches have it, is half as much matrix work again. Their sum is that
// of the rounded ones, by a product with ones, so that equal weights lose
// nothing. Values are turned into columns by byte permutations as in
// attn_kernel.h; e4m3 tiles are widened once a block on their way into LDS.
// The slots are cut into as many equal runs for each (head, block of rows) as
// fill the card, and blocks that read the same run sit on one XCD and read it at
// the same time, so that it comes from its L2. What bounds it: matrix
// instructions are busy 45% of the cycles, 830 TFLOP/s at the 1.8 GHz that the
// card keeps under them (e4m3: 38%, 750), the rest being what does not fit
// under them (permutations, maxima, barriers; e4m3: widening).
#pragma once

#include "attn_kernel.h"

namespace hrs {
namespace {

template <int KIND, int D> struct PrefixBlock {
  using C = PrefixCfg<KIND, D>;
  static constexpr int RT = C::RT, NW = C::NW, TS = C::TS, ROW = D * 2, PIECES = ROW / 16;
  static constexpr int DT = D / 16, QC = D / 32;
  static constexpr int LPS = 2 * TS * PIECES / (64 * NW);        // loads of a thread per tile (bf16)
  static constexpr int LP8 = 2 * TS * D / 16 / (64 * NW);        // and for e4m3
  static constexpr float kLift = KIND == kF8 ? 7.0f : 0.0f;      // as AttnBlock's
  static_assert(KIND != kF32 && TS == 32, "16-bit products, 32 slots each");

  const AttnShared& a;
  char* const lds;
  int wave, lane, n16, g;
  int h, rb;
  bool idle;
  u32x4 q[RT][QC];
  f32x4 o[RT][DT];
  f32x4 l[RT];
  float m[RT];
  float off[RT];               // taken_off, where there are registers to keep it
  float c, vs;
  int held, pg[TS / 16];             // pages of the next tile to load
  uint32_t v_at[4];            // a lane's places in a tile's values
  uint32_t ring;               // two bits a place of the ring: groups of 16 slots whose page is there

  __device__ __forceinline__ PrefixBlock(const AttnShared& args, char* l_) : a(args), lds(l_) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = threadIdx.x & 63;
    n16 = lane & 15;
    g = lane >> 4;
    constexpr int kBytes = D >= 128 ? 16 : 8;    // of a lane's columns
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = 4 * g + j, byte = n16 * kBytes;
      v_at[j] = row * ROW + (((byte >> 4) ^ swizzle<PIECES>(row)) << 4) + (byte & 15);
    }
  }

  // The pages of the next tile to load, the run's i-th. A lane holds one group's
  // page; scalar loads would be counted with the reads of LDS, out of order, and
  // have each of those waited for to the last.
  __device__ __forceinline__ void fetch_pages(int tile, int i) {
    constexpr int kGroups = TS / 16;
    if (i % (64 / kGroups) == 0) {
      const int64_t page = static_cast<int64_t>(tile * TS + 16 * lane) >> a.page_shift;
      held = a.prefix_table[min(static_cast<int>(page), a.prefix_pages - 1)];
      asm volatile("" : "+v"(held));
    }
#pragma unroll
    for (int j = 0; j < kGroups; ++j) pg[j] = __builtin_amdgcn_readlane(held, (i * kGroups + j) & 63);
  }
  // Where the tile's groups of 16 rows are in the caches, in bytes (those of
  // absent pages: the first page).
  __device__ __forceinline__ void places(int tile, int stage, int64_t (&at)[TS / 16]) {
    constexpr int CSZ = KIND == kF8 ? 1 : 2;
    const uint32_t per_page = 1u << (a.page_shift - 4);
    uint32_t there = 0;
#pragma unroll
    for (int i = 0; i < TS / 16; ++i) {
      const bool ok = static_cast<uint32_t>(pg[i]) < static_cast<uint32_t>(a.n_pages);
      there |= ok ? 1u << i : 0u;
      const uint32_t group = __builtin_amdgcn_readfirstlane((static_cast<uint32_t>(ok ? pg[i] : 0) * a.kvheads + h) * per_page +
                                                            ((tile * (TS / 16) + i) & (per_page - 1)));
      at[i] = static_cast<int64_t>(group) * (16 * D * CSZ);
    }
    ring = __builtin_amdgcn_readfirstlane((ring & ~(3u << (2 * stage))) | there << (2 * stage));
  }

  // bf16: a wave's i-th load of a tile, or all of them, straight into the
  // tile's place of the ring, pieces of a row permuted as in attn_kernel.h.
  __device__ __forceinline__ void issue(const int64_t (&at)[TS / 16], int stage, int i) {
    const int p0 = (i * NW + wave) * 64;
    const uint32_t row = static_cast<uint32_t>(p0 + lane) / PIECES % 16;
    const uint32_t off = row * ROW + ((static_cast<uint32_t>(lane) % PIECES) ^ swizzle<PIECES>(row)) * 16;
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(source<PIECES>(i, at) + off),
                                     (__attribute__((address_space(3))) void*)(lds + stage * C::STAGE + p0 * 16), 16, 0, 0);
  }
  __device__ __forceinline__ void issue(int tile, int stage) {
    int64_t at[TS / 16];
    places(tile, stage, at);
#pragma unroll
    for (int i = 0; i < LPS; ++i) issue(at, stage, i);
  }
  // Which 16 rows a wave's i-th load belongs to, a row being kPieces pieces.
  template <int kPieces> __device__ __forceinline__ const char* source(int i, const int64_t (&at)[TS / 16]) const {
    const int row = first_row<kPieces>(i);
    return (row >= TS ? a.v_cache : a.k_cache) + at[row % TS / 16];
  }
  template <int kPieces> __device__ __forceinline__ int first_row(int i) const {
    constexpr int kRows = NW * 64 / kPieces;     // that the block's i-th loads cover
    return i * kRows + (kRows > 16 ? wave * (64 / kPieces) : 0);
  }
  // e4m3: into registers, and from there widened into LDS, keys to bf16, values
  // to float16.
  __device__ __forceinline__ void load8(int tile, int stage, u32x4 (&x)[LP8]) {
    int64_t at[TS / 16];
    places(tile, stage, at);
#pragma unroll
    for (int i = 0; i < LP8; ++i) {
      const uint32_t row = ((i * NW + wave) * 64 + lane) / (D / 16);
      x[i] = *reinterpret_cast<const u32x4*>(source<D / 16>(i, at) + (row & 15) * D + (static_cast<uint32_t>(lane) % (D / 16)) * 16);
    }
  }
  __device__ __forceinline__ void store8(const u32x4 (&x)[LP8], int stage) {
    using B = AttnBlock<KIND, D, 3, kPrefix>;
    char* const dst = lds + stage * C::STAGE;
#pragma unroll
    for (int i = 0; i < LP8; ++i) {
      const int p0 = (i * NW + wave) * 64;
      const uint32_t row = (p0 + lane) / (D / 16);
      const uint32_t piece = (static_cast<uint32_t>(lane) % (D / 16)) * 2;
      const bool is_v = first_row<D / 16>(i) >= TS;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        u32x4 y;
        if (is_v)
          y = u32x4{B::widen2_f16(x[i][2 * j], false), B::widen2_f16(x[i][2 * j], true), B::widen2_f16(x[i][2 * j + 1], false),
                    B::widen2_f16(x[i][2 * j + 1], true)};
        else
          y = B::widen8(x[i][2 * j], x[i][2 * j + 1]);
        *reinterpret_cast<u32x4*>(dst + row * ROW + (((piece + j) ^ swizzle<PIECES>(row)) << 4)) = y;
      }
    }
  }

  __device__ __forceinline__ void load_rows() {
    idle = rb * C::ROWS + wave * (16 * RT) >= a.rows;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = rb * C::ROWS + (wave * RT + rt) * 16 + n16;
      const bool on = row < a.rows;
      const int t = on ? row / a.group : 0;
      const int hq = h * a.group + (on ? row - t * a.group : 0);
      const char* src = static_cast<const char*>(a.q) + (static_cast<int64_t>(t) * a.q_stride + static_cast<int64_t>(hq) * D) * 2;
#pragma unroll
      for (int x = 0; x < QC; ++x) {
        q[rt][x] = u32x4{};
        if (on) q[rt][x] = *reinterpret_cast<const u32x4*>(src + (4 * x + g) * 16);
      }
      m[rt] = -__builtin_inff();
      if constexpr (C::NEXT) off[rt] = -kLift;
      l[rt] = f32x4{};
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) o[rt][dt] = f32x4{};
    }
  }
  __device__ __forceinline__ void settle() {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int x = 0; x < QC; ++x) asm volatile("" : "+v"(q[rt][x]));
    vs = AttnBlock<KIND, D, 3, kPrefix>::uniform(vs);
    c = AttnBlock<KIND, D, 3, kPrefix>::uniform(c);
  }

  static __device__ __forceinline__ f32x4 product(u32x4 x, u32x4 y, f32x4 acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), acc, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 product_v(u32x4 x, u32x4 y, f32x4 acc) {
    if constexpr (KIND == kF8)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), acc, 0, 0, 0);
    else
      return product(x, y, acc);
  }

  // In the matrix units' own registers. Where vector operations see the running
  // results as they go from tile to tile, the compiler keeps them in the vector
  // units' registers, of which there are too few, and moves all of them twice a
  // tile.
  static __device__ __forceinline__ void pin(f32x4& x) {
    if constexpr (C::NEXT) asm volatile("" : "+a"(x));
  }

  static constexpr int SB = 2;                 // groups of 16 slots
  typedef f32x4 Scores[RT][SB];

  static constexpr int kAhead = QC * SB < 4 ? QC * SB : 4;       // reads of LDS before their products

  __device__ __forceinline__ uint32_t k_place(const char* kt) const {
    return lds_address(kt) + n16 * ROW + ((g ^ swizzle<PIECES>(n16)) << 4);
  }
  // Step i's keys, and the first steps'.
  static __device__ __forceinline__ u32x4 read_k(uint32_t ka, int i) {
    return *lds_at<u32x4>((ka ^ ((i / SB) << 6)) + (i % SB) * 16 * ROW);
  }
  __device__ __forceinline__ void first_k(const char* kt, u32x4 (&k)[kAhead]) const {
    const uint32_t ka = k_place(kt);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) k[i] = read_k(ka, i);
  }

  __device__ __forceinline__ void scores(const char* kt, Scores& s) const {
    const uint32_t ka = k_place(kt);
    u32x4 k[kAhead];
    first_k(kt, k);
#pragma unroll
    for (int i = 0; i < QC * SB; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      const u32x4 now = k[i % kAhead];
      if (i + kAhead < QC * SB) k[i % kAhead] = read_k(ka, i + kAhead);
      const int x = i / SB, sb = i % SB;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][sb] = product(now, q[rt][x], x == 0 ? f32x4{} : s[rt][sb]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }

  // Scores out of the matrix units' registers, once for all that follows.
  static __device__ __forceinline__ void fetch(f32x4 (&s)[SB]) {
    if constexpr (C::NEXT) {
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) asm volatile("" : "+v"(s[sb]));
    }
  }
  static __device__ __forceinline__ float highest(const f32x4 (&s)[SB]) {
    float x = -__builtin_inff();
#pragma unroll
    for (int sb = 0; sb < SB; ++sb)
#pragma unroll
      for (int i = 0; i < 4; ++i) x = fmaxf(x, s[sb][i]);
    return x;
  }

  // What is taken off a row's scores: m, but for rows without any yet.
  __device__ __forceinline__ float taken_off(int rt) const { return (m[rt] == -__builtin_inff() ? 0.0f : m[rt]) - kLift; }

  // Everything about a tile's scores that is rare (top: their highest, a lane's): a scale that is negative or
  // no number, absent pages, a reference that moves, scores far out. f: what the
  // scores are still to be multiplied with; mb: and what is to be taken off.
  __device__ __forceinline__ void settle_scores(Scores& s, float (&top)[RT], uint32_t there, float& f, float (&mb)[RT]) {
    f = c;
    if (!(f >= 0.0f)) {
      const float turn = f < 0.0f ? -1.0f : f;
      f = -f;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) s[rt][sb] *= turn;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) top[rt] = highest(s[rt]);
    }
    f = fmaxf(f, 1e-37f);
    if (there != 3) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
          if (!((there >> sb) & 1)) s[rt][sb] = f32x4{-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) top[rt] = highest(s[rt]);
    }
    bool more = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      top[rt] *= f;
      more = more || top[rt] - m[rt] > 8.0f;
    }
    if (__any(more)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float mt = row_max(top[rt]);
        const bool moves = mt - m[rt] > 8.0f;
        const float keep = moves ? __builtin_amdgcn_exp2f(m[rt] - mt) : 1.0f;
        m[rt] = moves ? mt : m[rt];
        auto scale = [&](f32x4& x) {
          pin(x);
          x *= keep;
          pin(x);
        };
        scale(l[rt]);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) scale(o[rt][dt]);
        if constexpr (C::NEXT) off[rt] = taken_off(rt);
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) mb[rt] = C::NEXT ? off[rt] : taken_off(rt);
    // References so large that differences to them round.
    float most = 0.0f;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) most = fmaxf(most, fabsf(mb[rt]));
    if (__any(most >= 0x1p22f - 8.0f)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const bool own = fabsf(m[rt]) >= 0x1p22f && m[rt] != -__builtin_inff();
#pragma unroll
        for (int sb = 0; sb < SB; ++sb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = s[rt][sb][i];
            s[rt][sb][i] = own ? (x * f - m[rt]) + kLift : fmaf(x, f, -mb[rt]);
          }
        mb[rt] = 0.0f;
      }
      f = 1.0f;
    }
  }

  // A tile's weights from its scores, O^T += V^T P^T and the weights' sums; under
  // the weights, the scores of the next tile. Written product by product, in an
  // order that the compiler keeps: operands are read from LDS well before their
  // products, and the vector operations stand one or two behind each product,
  // whose 16 cycles they take. Values: a lane's rows turned into columns by byte
  // permutations, as attn_kernel.h's Values.
  // load(i): the i-th of kLoads loads.
  template <int kLoads, typename Load>
  __device__ __forceinline__ void tile(const Scores& s, float f, const float (&mb)[RT], const char* vt, const char* kt,
                                       u32x4 (&k)[kAhead], Scores& then, float (&top)[RT], Load load) {
    constexpr int kSteps = QC * SB, kValues = RT * SB * 4, kSlots = kSteps * RT;
    constexpr int kCols = D >= 128 ? 8 : 4, kHalves = D / (16 * kCols), kWords = kCols / 2, kReads = SB * 4;
    const uint32_t ka = k_place(kt);
    uint32_t va[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) va[j] = lds_address(vt) + v_at[j];
    uint32_t w[kHalves][kReads][kWords];
    u32x4 p[RT];
    auto read_v = [&](int half, int i) {
      const uint32_t at = va[i % 4] + half * (32 * kCols) + (i / 4) * 16 * ROW;
      if constexpr (kWords == 4) {
        const u32x4 x = *lds_at<u32x4>(at);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[half][i][e] = x[e];
      } else {
        const u32x2 x = *lds_at<u32x2>(at);
#pragma unroll
        for (int e = 0; e < 2; ++e) w[half][i][e] = x[e];
      }
    };
    // The i-th score as a weight, in two parts.
    float e[4];
    auto weigh = [&](int i) {
      const int sb = i / (4 * RT), rt = i / 4 % RT;
      e[i % 4] = fmaf(s[rt][sb][i % 4], f, -mb[rt]);
    };
    auto weigh2 = [&](int i) {
      const int sb = i / (4 * RT), rt = i / 4 % RT;
      e[i % 4] = __builtin_amdgcn_exp2f(e[i % 4]);
      if (i % 2) {
        if constexpr (KIND == kF8) p[rt][2 * sb + i % 4 / 2] = AttnBlock<KIND, D, 3, kPrefix>::pack_f16(e[i % 4 - 1], e[i % 4]);
        else p[rt][2 * sb + i % 4 / 2] = pack_bf16(e[i % 4 - 1], e[i % 4]);
      }
    };
    if constexpr (C::NEXT) {
      static_assert(kSlots % kValues == 0 && kSteps >= kReads + 2, "each value in its slots");
      constexpr int kEach = kSlots / kValues;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const u32x4 now = k[i % kAhead];
        if (i + kAhead < kSteps) k[i % kAhead] = read_k(ka, i + kAhead);
        const int first = i - (kSteps - 2 - kReads);
        if (first >= 0 && first < kReads) read_v(0, first);
        const int x = i / SB, sb = i % SB;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          then[rt][sb] = product(now, q[rt][x], x == 0 ? f32x4{} : then[rt][sb]);
          const int slot = i * RT + rt;
          if (slot % kEach == 0) weigh(slot / kEach);
          if (slot % kEach == kEach - 1) weigh2(slot / kEach);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kReads; ++i) read_v(0, i);
#pragma unroll
      for (int i = 0; i < kValues; ++i) {
        weigh(i);
        weigh2(i);
      }
    }
    u32x4 v, after;
    auto turn = [&](int col, int i) {            // a quarter of a column's operand
      const int half = col / kCols, x = col % kCols, at = i / 2 * 4 + i % 2 * 2;
      after[i] = __builtin_amdgcn_perm(w[half][at + 1][x >> 1], w[half][at][x >> 1], x & 1 ? 0x07060302u : 0x05040100u);
    };
    const uint32_t one = KIND == kF8 ? 0x3C003C00u : 0x3F803F80u;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      l[rt] = product_v(u32x4{one, one, one, one}, p[rt], l[rt]);
#pragma unroll
      for (int i = rt * 4 / RT; i < (rt + 1) * 4 / RT; ++i) turn(0, i);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int col = 0; col < DT; ++col) {
      v = after;
      if (col / kCols + 1 < kHalves && col % kCols < kReads / 2) {
        read_v(col / kCols + 1, 2 * (col % kCols));
        read_v(col / kCols + 1, 2 * (col % kCols) + 1);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        o[rt][col] = product_v(v, p[rt], o[rt][col]);
        if (col + 1 < DT) {
#pragma unroll
          for (int i = rt * 4 / (RT - 1); i < (rt + 1) * 4 / (RT - 1) && i < 4; ++i) turn(col + 1, i);
        }
        if (C::NEXT && rt == 0 && col < RT) {
          fetch(then[col]);
          top[col] = highest(then[col]);
        }
        if (rt == RT - 1 && col >= DT - kLoads) load(col - (DT - kLoads));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  __device__ __forceinline__ char* stage_of(int i) const { return lds + (static_cast<uint32_t>(i) % C::NST) * C::STAGE; }

  // Values of absent pages, which weights of 0 multiply: no numbers may be there.
  __device__ __forceinline__ void clear(char* vt, uint32_t there) {
    for (int i = threadIdx.x; i < TS * PIECES; i += 64 * NW)
      if (!((there >> (i / (16 * PIECES))) & 1)) *reinterpret_cast<u32x4*>(vt + i * 16) = u32x4{};
  }

  // Tiles [t0, t1). The next tile's scores are formed while this one's become
  // weights: the matrix units work under the vector units' longest stretch.
  __device__ __forceinline__ void run(int t0, int t1) {
    // bf16 tiles that the wave's own work hides are loaded among its products,
    // the last tile again where there are no more.
    constexpr bool kAmong = C::NEXT && KIND != kF8;
    ring = 0;
    fetch_pages(t0, 0);
    int next = t0;               // next tile to load
    u32x4 x[KIND == kF8 ? LP8 : 1];
    auto step = [&]() {
      ++next;
      if (next < t1) fetch_pages(next, next - t0);
    };
    auto start = [&]() {
      const int stage = static_cast<uint32_t>(next - t0) % C::NST;
      if (!kAmong && next >= t1) return;
      if constexpr (KIND == kF8) load8(next, stage, x);
      else issue(min(next, t1 - 1), stage);
      step();
    };
    // e4m3: what was loaded last, into its place.
    auto store = [&](int before) {
      if constexpr (KIND == kF8)
        if (next > before) store8(x, static_cast<uint32_t>(next - 1 - t0) % C::NST);
    };
    if constexpr (KIND == kF8) {
      start();
      store(t0);
      const int before = next;
      start();
      store(before);
    } else {
      for (int i = 0; i < C::NST - 1; ++i) start();
    }
    load_rows();
    settle();
    Scores s;
    float top[RT];
    for (int u = t0; u < t1; ++u) {
      // Tile u (with NEXT also the next) is there for everybody, and everybody is
      // done with tile u - 1.
      if constexpr (kAmong) {
        wait_vm<(C::NST - 3) * LPS>();
      } else if constexpr (KIND != kF8) {
        const int later = next - 1 - u;          // tiles that may be on their way
        if (later > 1) wait_vm<2 * LPS>();
        else if (later == 1) wait_vm<LPS>();
        else wait_vm<0>();
      }
      block_barrier();
      // (The first keys of tile u + 1 come under the next loads' addresses.)
      u32x4 k[kAhead];
      if constexpr (C::NEXT) first_k(stage_of(u + 1 - t0), k);
      const int before = next;
      const int stage = static_cast<uint32_t>(next - t0) % C::NST;
      int64_t at[TS / 16];
      if constexpr (kAmong) {
        places(min(next, t1 - 1), stage, at);
        step();
      } else {
        start();
      }
      mem_fence();
      const uint32_t there = (ring >> (2 * (static_cast<uint32_t>(u - t0) % C::NST))) & 3;
      if (there != 3) {          // (the whole block's)
        clear(stage_of(u - t0) + TS * ROW, there);
        block_barrier();
      }
      if (!idle) {
        if (!C::NEXT || u == t0) {
          scores(stage_of(u - t0), s);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            fetch(s[rt]);
            top[rt] = highest(s[rt]);
          }
        }
        float f, mb[RT];
        settle_scores(s, top, there, f, mb);
        // (Behind the last tile: scores of what the ring holds, for nobody. A
        // branch would part the products.)
        Scores then;
        tile<kAmong ? LPS : 0>(s, f, mb, stage_of(u - t0) + TS * ROW, stage_of(u + 1 - t0), k, then, top,
                               [&](int i) { issue(at, stage, i); });
        if constexpr (C::NEXT) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) s[rt][sb] = then[rt][sb];
        }
      } else if constexpr (kAmong) {
#pragma unroll
        for (int i = 0; i < LPS; ++i) issue(at, stage, i);
      }
      mem_fence();
      store(before);
    }
    if constexpr (kAmong) wait_vm<0>();          // nothing is on its way into LDS when the block ends
  }

  __device__ __forceinline__ void finish(int64_t slot) {
    if (idle) return;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int tile = wave * RT + rt;
      f32x4* const at = reinterpret_cast<f32x4*>(a.part) + (slot * (C::ROWS / 16) + tile) * (DT * 64) + lane;
      const float f = KIND == kF8 && m[rt] != -__builtin_inff() ? vs : 1.0f;
      pin(l[rt]);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) pin(o[rt][dt]);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) at[dt * 64] = KIND == kF8 ? o[rt][dt] * f : o[rt][dt];
      if (g == 0) a.part_ml[slot * C::ROWS + tile * 16 + n16] = float2{m[rt], l[rt][0]};
    }
  }
};

// Grid: see prefix_grid. runs: runs of slots a head is cut into at most.
template <int KIND, int D>
__global__ __launch_bounds__((64 * PrefixCfg<KIND, D>::NW), (PrefixCfg<KIND, D>::PER_CU)) void attn_prefix_kernel(const AttnLens lens, int runs, const AttnShared args) {
  using C = PrefixCfg<KIND, D>;
  extern __shared__ __align__(1024) char lds[];
  // Blocks of one XCD (every eighth) take consecutive places of the list (head,
  // run, block of rows).
  const int total = args.kvheads * runs * args.row_blocks, per = (total + 7) / 8;
  const int place = static_cast<int>(blockIdx.x & 7) * per + static_cast<int>(blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= per || place >= total) return;
  PrefixBlock<KIND, D> blk(args, lds);
  const int pair = place / args.row_blocks;
  blk.rb = place - pair * args.row_blocks;
  blk.h = pair / runs;
  const int run = pair - blk.h * runs;
  AttnHole hole;
  {
    int len[kAttnReqs / 64];
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int k = 0; k < kAttnReqs / 64; ++k) len[k] = lens.len[min(lane * (kAttnReqs / 64) + k, lens.n - 1)];
    hole = attn_hole(lens, args, len);
  }
  const int tiles = (hole.end - hole.first) / C::TS, first = hole.first / C::TS;
  // A run has six tiles where there are as many: more parts cost the join what
  // shorter runs gain (768 rows of 128 over 512 slots: 47 us, runs of one 53; over
  // 2,048 56 and 56).
  constexpr int kLeast = 6;
  const int used = min(runs, (tiles + kLeast - 1) / kLeast);
  if (blockIdx.x == 0 && threadIdx.x == 0) args.plan[0] = used;
  if (run >= used) return;
  const int t0 = first + static_cast<int>(static_cast<int64_t>(run) * tiles / used);
  const int t1 = first + static_cast<int>(static_cast<int64_t>(run + 1) * tiles / used);
  const float ks = KIND == kF8 && args.k_scale ? args.k_scale[blk.h] : 1.0f;
  blk.vs = KIND == kF8 && args.v_scale ? args.v_scale[blk.h] : 1.0f;
  blk.c = args.scale * 1.4426950408889634f * ks;
  blk.run(t0, t1);
  blk.finish((static_cast<int64_t>(blk.h) * runs + run) * args.row_blocks + blk.rb);
}

template <int KIND, int D> void launch_prefix(const AttnShared& args, const AttnLens& l, int runs, hipStream_t s) {
  using C = PrefixCfg<KIND, D>;
  const int total = args.kvheads * runs * args.row_blocks;
  hipLaunchKernelGGL((attn_prefix_kernel<KIND, D>), dim3((total + 7) / 8 * 8), dim3(64 * C::NW), C::LDS, s, l, runs, args);
}

}  // namespace

template <int KIND> void attn_prefix_wide(const AttnShared& args, const AttnLens& lens, int runs, int d, hipStream_t s) {
  if (d == 64) launch_prefix<KIND, 64>(args, lens, runs, s);
  else if (d == 128) launch_prefix<KIND, 128>(args, lens, runs, s);
  else launch_prefix<KIND, 256>(args, lens, runs, s);
}

}  // namespace hrs
