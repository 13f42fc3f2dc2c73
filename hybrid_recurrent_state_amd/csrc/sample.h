// Shared by the entry points that accept drafts by sampling (sample.hip,
// filter.hip): weights of logits, reductions, the walk over a chain or tree of
// drafts and the search for the drawn token.
#pragma once

#include <hip/hip_runtime.h>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

constexpr int kThreads = 256;
constexpr int kPiece = kThreads * 8;                // logits per node block

enum : int32_t { kPlain = 0, kWithout = 1, kRest = 2 };   // weights: p; p without tokens; max(p - q, 0)

struct NodeInfo {
  int32_t node;
  int32_t mode;
  int32_t n_gone;
  int32_t bad;       // temperature refused: nothing is written
  int32_t gone[HRS_MAX_POS];
};

struct SampleArgs {
  const void* logits;
  const int32_t* tokens;
  const float* uniforms;
  const void* draft;
  const float* temperature;
  float* token_prob;
  int32_t* accept_node;
  int32_t* accept_len;
  int32_t* path;
  int32_t* bonus;
  int32_t* status;
  double2* stats;     // workspace [rows][n_chunks]: maximum, sum
  double2* part;      // workspace [R][n_pieces]: maximum, sum of the node's row
  double* rest;       // workspace [R][n_pieces]: sum of max(p - q, 0)
  NodeInfo* info;     // workspace [R]
  int32_t n_req;
  int32_t n_pos;
  int32_t vocab;
  int32_t n_chunks;
  int32_t n_pieces;
  int32_t req0;
  int32_t draft_bf16;
};
// Trees carry their parents; chains and the kernels behind the walk do not,
// since every launch copies its arguments.
template <typename Base> struct WithTree : Base {
  int8_t parent[kGeomBytes];
};
using SampleTree = WithTree<SampleArgs>;
template <typename Args> constexpr bool is_tree = false;
template <typename Base> constexpr bool is_tree<WithTree<Base>> = true;
__device__ __forceinline__ int parent_of(const SampleArgs&, int, int t) { return t - 1; }
template <typename Base> __device__ __forceinline__ int parent_of(const WithTree<Base>& a, int i, int) { return a.parent[i]; }

__device__ __forceinline__ float temperature_of(const SampleArgs& a, int r) {
  return a.temperature ? a.temperature[r] : 1.0f;
}
__device__ __forceinline__ bool bad_temperature(float tau) { return !(tau >= 0.0f); }

// e^x for x <= 0: x = n ln 2 + r with |r| <= ln 2 / 2, the power series of
// e^r to r^12 (what is left out is below 2e-16 of it), n into the exponent.
// About half the operations of the general function.
__device__ __forceinline__ double exp_down(double x) {
  x = fmax(x, -746.0);                    // below: zero
  const double n = rint(x * 1.4426950408889634074);
  double r = fma(n, -0.69314718055994530942, x);      // ln 2 in two parts: the nearest double
  r = fma(n, -2.3190468138462995584e-17, r);          // and what it leaves
  double y = 1.0 / 479001600.0;
  y = fma(y, r, 1.0 / 39916800.0);
  y = fma(y, r, 1.0 / 3628800.0);
  y = fma(y, r, 1.0 / 362880.0);
  y = fma(y, r, 1.0 / 40320.0);
  y = fma(y, r, 1.0 / 5040.0);
  y = fma(y, r, 1.0 / 720.0);
  y = fma(y, r, 1.0 / 120.0);
  y = fma(y, r, 1.0 / 24.0);
  y = fma(y, r, 1.0 / 6.0);
  y = fma(y, r, 0.5);
  y = fma(y, r, 1.0);
  y = fma(y, r, 1.0);
  return ldexp(y, static_cast<int>(n));
}

// Weight of a logit beside the maximum m: e^((z - m) / tau). Hard rows
// (temperature 0, or +inf logits) give the largest logits one, the rest zero;
// NaN has none, and neither has anything where there is no maximum.
struct Weigher {
  double m, inv;
  bool hard, none;
  __device__ Weigher(double m_, float tau) : m(m_) {
    none = m == -__builtin_inf();
    hard = tau == 0.0f || m == __builtin_inf();
    inv = tau > 0.0f ? fmax(1.0 / static_cast<double>(tau), 1e-300) : 1.0;
  }
  __device__ __forceinline__ double operator()(double z) const {
    if (none || z != z) return 0.0;
    if (hard) return z == m ? 1.0 : 0.0;
    return exp_down((z - m) * inv);
  }
};

// A double's two halves through the same lane move.
template <int CTRL> __device__ __forceinline__ double dpp_move(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// Sum or maximum over the wave, in a fixed order, the same in every lane:
// four moves inside 16 lanes, two exchanges of rows.
template <typename Op> __device__ __forceinline__ double wave_reduce(double x, Op op) {
  x = op(x, dpp_move<0xB1>(x));
  x = op(x, dpp_move<0x4E>(x));
  x = op(x, dpp_move<0x141>(x));
  x = op(x, dpp_move<0x140>(x));
  auto join = [&](auto swap) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const auto lo = swap(static_cast<uint32_t>(b));
    const auto hi = swap(static_cast<uint32_t>(b >> 32));
    x = op(__builtin_bit_cast(double, (static_cast<uint64_t>(hi[0]) << 32) | lo[0]),
           __builtin_bit_cast(double, (static_cast<uint64_t>(hi[1]) << 32) | lo[1]));
  };
  join([](uint32_t v) { return __builtin_amdgcn_permlane16_swap(v, v, false, false); });
  join([](uint32_t v) { return __builtin_amdgcn_permlane32_swap(v, v, false, false); });
  return x;
}

// The same over the block.
template <typename Op> __device__ __forceinline__ double block_reduce(double x, Op op, double* lds) {
  x = wave_reduce(x, op);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) x = op(x, lds[i]);
  return x;
}
__device__ __forceinline__ double add(double a, double b) { return a + b; }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

// Eight logits with nontemporal loads (read once by the statistics).
template <typename T> __device__ __forceinline__ void load8_nt(const T* p, float* o);
template <> __device__ __forceinline__ void load8_nt<uint16_t>(const uint16_t* p, float* o) {
  const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  o[0] = bf16_lo(w.x); o[1] = bf16_hi(w.x);
  o[2] = bf16_lo(w.y); o[3] = bf16_hi(w.y);
  o[4] = bf16_lo(w.z); o[5] = bf16_hi(w.z);
  o[6] = bf16_lo(w.w); o[7] = bf16_hi(w.w);
}
template <> __device__ __forceinline__ void load8_nt<float>(const float* p, float* o) {
  const f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
  const f32x4 y = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
  o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
  o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
}

__device__ __forceinline__ double draft_value(const SampleArgs& a, int64_t i) {
  return a.draft_bf16 ? bf16_one(static_cast<const uint16_t*>(a.draft)[i]) : static_cast<const float*>(a.draft)[i];
}

struct WalkLds {
  double prob[HRS_MAX_POS];
  double need[HRS_MAX_POS];      // u q (q = 1 for a picked draft)
  int32_t tok[HRS_MAX_POS];
  NodeInfo info;
};

// The walk by the drafts' probabilities (w.prob, w.need, w.tok), by the whole
// block; `write`: the request's outputs as well.
template <typename Args>
__device__ __forceinline__ void decide(const Args& args, int rl, bool write, WalkLds& w) {
  const int r = args.req0 + rl, T_ = args.n_pos;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = static_cast<int64_t>(r) * T_;
  if (wave == 0) {
    const int tl = min(lane, T_ - 1);
    const int par = lane >= T_ ? -2 : parent_of(args, rl * T_ + tl, lane);
    const int tok = w.tok[tl];
    const double need = w.need[tl];
    const double prob = w.prob[tl];
    int node = 0, len = 0, mode = kPlain, n_gone = 0;
    uint64_t on_path = 1;
    if constexpr (!is_tree<Args>) {
      // One comparison per position; the accepted length is the run of
      // successes from position 1.
      const bool ok = lane >= 1 && lane < T_ && need < prob;
      const uint64_t hits = __ballot(ok);
      len = __builtin_ctzll(~(hits >> 1));
      node = len;
      on_path = ~uint64_t{0} >> (63 - len);
      if (node < T_ - 1) {
        mode = args.draft ? kRest : kWithout;
        n_gone = args.draft ? 0 : 1;
        if (lane == node + 1) w.info.gone[0] = tok;
      }
    } else {
      for (;;) {
        uint64_t kids = __ballot(par == node && lane > 0);
        uint64_t out = 0;              // rejected children, one per token
        double left = 1.0;
        int next = -1;
        while (kids) {
          const int c = __builtin_ctzll(kids);
          kids &= kids - 1;
          const int tc = __builtin_amdgcn_readlane(tok, c);
          if (__ballot(tok == tc) & out) continue;
          const double pc = __shfl(prob, c), uc = __shfl(need, c);
          if (uc * left < pc) {
            next = c;
            break;
          }
          left -= pc;
          out |= uint64_t{1} << c;
        }
        if (next < 0) {
          n_gone = __popcll(out);
          mode = n_gone ? kWithout : kPlain;
          if ((out >> lane) & 1) w.info.gone[__popcll(out & ((uint64_t{1} << lane) - 1))] = tok;
          break;
        }
        node = __builtin_amdgcn_readfirstlane(next);
        on_path |= uint64_t{1} << node;
        ++len;
      }
    }
    if (lane == 0) {
      w.info.node = node;
      w.info.mode = mode;
      w.info.n_gone = n_gone;
      w.info.bad = 0;
      if (write) {
        args.accept_node[r] = node;
        args.accept_len[r] = len;
      }
    }
    if (write && lane < T_) {
      // A path's positions increase, so the i-th one is the i-th bit.
      if ((on_path >> lane) & 1) args.path[row0 + __popcll(on_path & ((uint64_t{1} << lane) - 1))] = lane;
      if (lane > len) args.path[row0 + lane] = -1;
    }
  }
  __syncthreads();
}

// The thread's eight logits of a piece (those past the row's end: count 0).
template <typename T> __device__ __forceinline__ int load_piece(const T* row, int V, int piece, float* z) {
  const int e = piece * kPiece + threadIdx.x * 8;
  load8<T>(row + min(e, V - 8), z);
  return e < V ? 8 : 0;
}

// Which of the eight tokens from v0 were taken out, one bit each.
__device__ __forceinline__ uint32_t gone_mask(const NodeInfo& info, int v0) {
  uint32_t mask = 0;
  for (int i = 0; i < info.n_gone; ++i) {
    const uint32_t d = static_cast<uint32_t>(info.gone[i]) - static_cast<uint32_t>(v0);
    mask |= d < 8 ? 1u << d : 0u;
  }
  return mask;
}

// The pieces of a request, by every wave for itself (no barrier): each lane
// takes consecutive ones, the first kHeld of them in registers, so that all
// loads go out at once (up to 524,288 logits a row).
constexpr int kHeld = 4;
template <typename V> struct Pieces {
  const V* p;
  int i0, i1;
  V held[kHeld];
  __device__ __forceinline__ Pieces(const V* p_, int n) : p(p_) {
    const int lane = threadIdx.x & 63;
    const int per = (n + 63) / 64;
    i0 = min(n, lane * per);
    i1 = min(n, i0 + per);
#pragma unroll
    for (int k = 0; k < kHeld; ++k) held[k] = p[min(i0 + k, n - 1)];
  }
  template <typename F> __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (i0 + k < i1) f(i0 + k, held[k]);
    for (int i = i0 + kHeld; i < i1; ++i) f(i, p[i]);
  }
};

// Inclusive sum over the block's threads, in order.
__device__ __forceinline__ double block_scan(double x, double* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(x, d);
    x += lane >= d ? y : 0.0;
  }
  __syncthreads();
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  double before = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) before += i < wave ? lds[i] : 0.0;
  return before + x;
}

// First thread for which hit holds, or kThreads; the same in every thread.
__device__ __forceinline__ int first_hit(bool hit, int32_t* lds) {
  const uint64_t b = __ballot(hit);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = b ? __builtin_ctzll(b) : 64;
  __syncthreads();
  int first = kThreads;
  for (int i = kThreads / 64 - 1; i >= 0; --i) first = lds[i] < 64 ? i * 64 + lds[i] : first;
  return first;
}
// Last thread for which hit holds, or -1.
__device__ __forceinline__ int last_hit(bool hit, int32_t* lds) {
  const uint64_t b = __ballot(hit);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = b ? 63 - __builtin_clzll(b) : -1;
  __syncthreads();
  int last = -1;
  for (int i = 0; i < kThreads / 64; ++i) last = lds[i] >= 0 ? i * 64 + lds[i] : last;
  return last;
}

// The piece where the cumulative sum of weight(piece) passes u times the
// total, the sum before it and the total; by every wave for itself. None
// passes: the last piece with any weight and a sum before it that nothing
// passes; no weight at all: -1. Each lane takes consecutive pieces.
struct Found {
  int piece;
  double before, total;
};
template <typename V, typename W> __device__ __forceinline__ Found find_piece(const Pieces<V>& pieces, W weight, double u) {
  const int lane = threadIdx.x & 63;
  double sum = 0.0;
  pieces.each([&](int, V x) { sum += weight(x); });
  double c = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double y = __shfl_up(c, d);
    c += lane >= d ? y : 0.0;
  }
  Found f{-1, 0.0, __shfl(c, 63)};
  const uint64_t some = __ballot(sum > 0.0);
  if (!some) return f;
  const double target = u * f.total;
  const uint64_t hits = __ballot(sum > 0.0 && c > target);
  const int owner = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
  // The owner lane's pieces one by one.
  double run = c - sum;
  int piece = -1;
  double before = 0.0;
  bool done = false;
  pieces.each([&](int i, V v) {
    const double x = weight(v);
    if (x > 0.0 && !done) {
      piece = i;
      before = run;
      done = hits && run + x > target;
    }
    run += x;
  });
  f.piece = __shfl(piece, owner);
  f.before = hits ? __shfl(before, owner) : -__builtin_inf();
  return f;
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace hrs
