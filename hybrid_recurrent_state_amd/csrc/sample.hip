// accept_sample: verification of drafted tokens against the target's
// probabilities from given random numbers, for a chain (with or without the
// draft's probabilities) or a draft tree, and the draw of the next token.
//
// It stands beside accept_greedy (accept.hip) for requests that sample
// (openinfer PR #626, "feat(qwen35): add opt-in DFlash speculative decoding",
// Summary: greedy requests only; sampling falls back to plain decoding).
//
// MI355X design: three or four dependent launches, no host round trip.
//  1. Row statistics: every 32 KB chunk of every row that has a child
//     (a leaf's probabilities are needed only if the walk ends there) is read
//     once with nontemporal loads into registers, reduced to its maximum m and
//     then to sum e^((z - m) / tau), float32 per thread, 64 bits across the
//     block: bound by the read of the logits, at about ten vector operations a
//     logit.
//  2. Walk and node sums: blocks of 2048 logits of the row where the walk
//     ends. Every block first repeats its request's walk (the statistics are
//     small and cached; handing the node over would be one more launch): lane
//     t holds position t, a chain is one ballot, a tree visits a node's
//     children by lane reads. Then it sums its logits' weights in 64 bits.
//  3. With draft probabilities: the sums of max(p - q, 0), which need the
//     row's total from 2.
//  4. One block per request finds the drawn token's 2048-logit piece by a
//     cumulative sum of the pieces and the token by one inside it.
// Why 64 bits in 2 to 4: a cumulative float32 sum over 151,936 weights is off
// by about 1e-6 of the total, and a token of an even distribution spans 7e-6.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

constexpr int kThreads = 256;
// Logits per statistics block, 32 KB of either type (16 rows of 151,936 bf16
// logits: 8192 logits a block level, 32,768 8% slower; float32: 16,384 7%
// slower).
template <typename T> constexpr int kChunk = 32768 / sizeof(T);
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
struct SampleTree : SampleArgs {
  int8_t parent[kGeomBytes];
};
template <typename Args> constexpr bool is_tree = std::is_same<Args, SampleTree>::value;
__device__ __forceinline__ int parent_of(const SampleArgs&, int, int t) { return t - 1; }
__device__ __forceinline__ int parent_of(const SampleTree& a, int i, int) { return a.parent[i]; }

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

// 1. Grid: (request, position with a child, chunk).
template <typename T, typename Args>
__global__ __launch_bounds__(kThreads) void row_stats_kernel(const Args args) {
  const int rows = is_tree<Args> ? args.n_pos : args.n_pos - 1;
  const int chunk = blockIdx.x % args.n_chunks;
  const int rt = blockIdx.x / args.n_chunks;
  const int rl = rt / rows, t = rt - rl * rows;
  const int64_t row = static_cast<int64_t>(args.req0 + rl) * args.n_pos + t;
  if constexpr (is_tree<Args>) {
    const int lane = threadIdx.x & 63;
    const int p = args.parent[rl * args.n_pos + min(lane, args.n_pos - 1)];
    if (!__any(p == t && lane > 0)) return;
  }
  const float tau = temperature_of(args, args.req0 + rl);
  const T* base = static_cast<const T*>(args.logits) + row * args.vocab;
  constexpr int kIter = kChunk<T> / (kThreads * 8);   // 8-logit slices per thread
  const int begin = chunk * kChunk<T>;
  const int end = min(args.vocab, begin + kChunk<T>);
  float v[kIter][8];
  float m = -__builtin_inff();
  // Slices past the row's end re-read its last eight logits: they change no
  // maximum, and their weights are left out.
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int e = begin + (it * kThreads + threadIdx.x) * 8;
    load8_nt<T>(base + min(e, end - 8), v[it]);
  }
#pragma unroll
  for (int it = 0; it < kIter; ++it)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[it][i] = __builtin_canonicalizef(v[it][i]);   // a quiet NaN loses against every number
      m = fmaxf(m, v[it][i]);
    }
#pragma unroll
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  __shared__ float wave_m[kThreads / 64];
  __shared__ double lds[kThreads / 64];
  if ((threadIdx.x & 63) == 0) wave_m[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) m = fmaxf(m, wave_m[i]);
  float sum = 0.0f;
  if (tau == 0.0f || m == __builtin_inff()) {
#pragma unroll
    for (int it = 0; it < kIter; ++it)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (begin + (it * kThreads + threadIdx.x) * 8 < end) sum += v[it][i] == m ? 1.0f : 0.0f;
  } else if (m > -__builtin_inff()) {
    const float c = fminf(fmaxf(1.4426950408889634f / tau, 1.2e-38f), 3.4e38f);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      float s8 = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)       // a NaN becomes -inf, of weight zero
        s8 += __builtin_amdgcn_exp2f(fmaxf((v[it][i] - m) * c, -__builtin_inff()));
      if (begin + (it * kThreads + threadIdx.x) * 8 < end) sum += s8;
    }
  }
  const double total = block_reduce(sum, add, lds);
  if (threadIdx.x == 0) args.stats[row * args.n_chunks + chunk] = double2{m, total};
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

// The walk of request r, by the whole block; the first block of the request
// writes its outputs.
template <typename T, typename Args>
__device__ __forceinline__ void walk(const Args& args, int rl, bool write, WalkLds& w) {
  const int r = args.req0 + rl, T_ = args.n_pos, V = args.vocab;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float tau = temperature_of(args, r);
  const int64_t row0 = static_cast<int64_t>(r) * T_;
  if (bad_temperature(tau)) {
    if (threadIdx.x == 0) w.info.bad = 1;
    __syncthreads();
    return;
  }
  // Probability of every draft: four lanes per position, each with every
  // fourth chunk of the parent's row; all positions' loads go out together.
  {
    const int t = min(static_cast<int>(threadIdx.x) >> 2, T_ - 1);
    const int sub = threadIdx.x & 3;
    const int p = max(0, parent_of(args, rl * T_ + t, t));
    const int x = args.tokens[row0 + t];
    const double u = args.uniforms[row0 + t];
    const bool valid = t > 0 && x >= 0 && x < V;
    double pr = t == 0 ? 1.0 : 0.0;
    double q = 1.0;
    constexpr int kHeld = 5;           // chunks a lane keeps in registers
    if (T_ > 1) {
      const double2* st = args.stats + (row0 + p) * args.n_chunks;
      double2 held[kHeld];
      double M = -__builtin_inf(), s = 0.0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) held[i] = st[min(sub + 4 * i, args.n_chunks - 1)];
      const double z =
          load_elem<T>(static_cast<const T*>(args.logits), (row0 + p) * V + (valid ? x : 0));
      if (args.draft) q = draft_value(args, (row0 + p) * V + (valid ? x : 0));
#pragma unroll
      for (int i = 0; i < kHeld; ++i) M = fmax(M, held[i].x);
      for (int i = sub + 4 * kHeld; i < args.n_chunks; i += 4) M = fmax(M, st[i].x);
      M = fmax(M, __shfl_xor(M, 1));
      M = fmax(M, __shfl_xor(M, 2));
      const Weigher weigh(M, tau);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) s += sub + 4 * i < args.n_chunks ? held[i].y * weigh(held[i].x) : 0.0;
      for (int i = sub + 4 * kHeld; i < args.n_chunks; i += 4) s += st[i].y * weigh(st[i].x);
      s += __shfl_xor(s, 1);
      s += __shfl_xor(s, 2);
      if (valid && s > 0.0) pr = weigh(z) / s;
    }
    if (sub == 0 && static_cast<int>(threadIdx.x) >> 2 < T_) {
      w.prob[t] = pr;
      w.need[t] = valid || !args.draft ? u * q : __builtin_inf();
      w.tok[t] = x;
      if (write) args.token_prob[row0 + t] = static_cast<float>(pr);
    }
  }
  __syncthreads();
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

// 2. Grid: (piece, request).
template <typename T, typename Args>
__global__ __launch_bounds__(kThreads) void node_kernel(const Args args) {
  __shared__ WalkLds w;
  __shared__ double lds[kThreads / 64];
  const int piece = blockIdx.x, rl = blockIdx.y, r = args.req0 + rl;
  if (piece == 0 && r == 0 && args.status) {
    int bad = 0;
    for (int i = threadIdx.x; i < args.n_req; i += kThreads) bad += bad_temperature(temperature_of(args, i));
    const double all = block_reduce(bad, add, lds);
    if (threadIdx.x == 0) *args.status = static_cast<int32_t>(all);
  }
  walk<T>(args, rl, piece == 0, w);
  if (piece == 0) {
    const int32_t* src = reinterpret_cast<const int32_t*>(&w.info);
    int32_t* dst = reinterpret_cast<int32_t*>(args.info + r);
    for (int i = threadIdx.x; i < static_cast<int>(sizeof(NodeInfo) / 4); i += kThreads) dst[i] = src[i];
  }
  if (w.info.bad) return;
  const T* row = static_cast<const T*>(args.logits) +
                 (static_cast<int64_t>(r) * args.n_pos + w.info.node) * args.vocab;
  float z[8];
  const int n = load_piece(row, args.vocab, piece, z);
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, __builtin_canonicalizef(z[i]));
  const double M = block_reduce(m, larger, lds);
  const Weigher weigh(M, temperature_of(args, r));
  double sum = 0.0;
  if (n) {
    const uint32_t gone = w.info.mode == kWithout ? gone_mask(w.info, piece * kPiece + threadIdx.x * 8) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (gone >> i) & 1 ? 0.0 : weigh(z[i]);
  }
  sum = block_reduce(sum, add, lds);
  if (threadIdx.x == 0) args.part[static_cast<int64_t>(r) * args.n_pieces + piece] = double2{M, sum};
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

// Maximum and total of the node's row.
__device__ __forceinline__ double2 row_total(const Pieces<double2>& part, float tau) {
  double M = -__builtin_inf(), s = 0.0;
  part.each([&](int, double2 x) { M = fmax(M, x.x); });
  M = wave_reduce(M, larger);
  const Weigher weigh(M, tau);
  part.each([&](int, double2 x) { s += x.y * weigh(x.x); });
  return double2{M, wave_reduce(s, add)};
}

// Weights of the thread's eight logits: mode kRest with the row's maximum and
// total (max(p - q, 0); a NaN in q leaves none), otherwise unnormalised.
template <typename T>
__device__ __forceinline__ double piece_weights(const SampleArgs& a, const NodeInfo& info, int mode, int r, int piece,
                                                double2 mz, float tau, double* x) {
  const int64_t row = (static_cast<int64_t>(r) * a.n_pos + info.node) * a.vocab;
  float z[8];
  const int n = load_piece(static_cast<const T*>(a.logits) + row, a.vocab, piece, z);
  const int v0 = piece * kPiece + threadIdx.x * 8;
  const Weigher weigh(mz.x, tau);
  float q[8] = {};
  if (mode == kRest && n) {
    if (a.draft_bf16) load8<uint16_t>(static_cast<const uint16_t*>(a.draft) + row + v0, q);
    else load8<float>(static_cast<const float*>(a.draft) + row + v0, q);
  }
  const uint32_t gone = mode == kWithout ? gone_mask(info, v0) : 0;
  const double inv = 1.0 / mz.y;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    double y = n ? weigh(z[i]) : 0.0;
    if (mode == kRest) {
      y = y * inv - static_cast<double>(q[i]);
      y = n && y > 0.0 ? y : 0.0;
    } else if ((gone >> i) & 1) {
      y = 0.0;
    }
    x[i] = y;
    sum += y;
  }
  return sum;
}

// 3. Grid: (piece, request).
template <typename T>
__global__ __launch_bounds__(kThreads) void rest_kernel(const SampleArgs args) {
  __shared__ double lds[kThreads / 64];
  const int piece = blockIdx.x, r = args.req0 + blockIdx.y;
  const NodeInfo& info = args.info[r];
  const float tau = temperature_of(args, r);
  const Pieces<double2> part(args.part + static_cast<int64_t>(r) * args.n_pieces, args.n_pieces);
  if (info.bad || info.mode != kRest) return;
  const double2 mz = row_total(part, tau);
  double x[8];
  double sum = mz.y > 0.0 ? piece_weights<T>(args, info, kRest, r, piece, mz, tau, x) : 0.0;
  sum = block_reduce(sum, add, lds);
  if (threadIdx.x == 0) args.rest[static_cast<int64_t>(r) * args.n_pieces + piece] = sum;
}

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

// 4. Grid: request.
template <typename T>
__global__ __launch_bounds__(kThreads) void draw_kernel(const SampleArgs args) {
  __shared__ double lds[kThreads / 64];
  __shared__ int32_t ilds[kThreads / 64];
  const int r = args.req0 + blockIdx.x;
  const NodeInfo& info = args.info[r];
  const float tau = temperature_of(args, r);
  const double u = args.uniforms[static_cast<int64_t>(r) * args.n_pos];
  const Pieces<double2> part(args.part + static_cast<int64_t>(r) * args.n_pieces, args.n_pieces);
  const Pieces<double> rest((args.draft ? args.rest : &args.part[0].x) + static_cast<int64_t>(r) * args.n_pieces,
                            args.n_pieces);
  if (info.bad) return;
  const double2 mz = row_total(part, tau);
  const Weigher weigh(mz.x, tau);
  auto whole = [&](double2 x) { return x.y * weigh(x.x); };
  int mode = info.mode;
  Found f = mode == kRest ? find_piece(rest, [](double x) { return x; }, u) : find_piece(part, whole, u);
  if (f.piece < 0 && mode != kPlain) {
    // Nothing is left over: the row itself. Its pieces' sums are at hand after
    // a rest; with tokens taken out they are formed here, piece by piece.
    mode = kPlain;
    if (info.mode == kRest) {
      f = find_piece(part, whole, u);
    } else {
      double x[8];
      for (int i = 0; i < args.n_pieces; ++i)
        f.total += block_reduce(piece_weights<T>(args, info, kPlain, r, i, mz, tau, x), add, lds);
      double c = 0.0;
      for (int i = 0; f.total > 0.0 && i < args.n_pieces; ++i) {
        const double s = block_reduce(piece_weights<T>(args, info, kPlain, r, i, mz, tau, x), add, lds);
        if (s > 0.0) {
          f.piece = i;
          f.before = c;
          if (c + s > u * f.total) break;
        }
        c += s;
      }
    }
  }
  const int piece = f.piece;
  const double before = f.before, total = f.total;
  int pick = 0;
  if (piece >= 0) {
    double x[8];
    const double sum = piece_weights<T>(args, info, mode, r, piece, mz, tau, x);
    const double c = before + block_scan(sum, lds);
    const double target = u * total;
    int owner = first_hit(sum > 0.0 && c > target, ilds);
    const bool passes = owner < kThreads;
    if (!passes) owner = last_hit(sum > 0.0, ilds);
    __shared__ int32_t pick_s;
    if (threadIdx.x == 0) pick_s = 0;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) == owner) {
      double run = c - sum;
      int p = 0;
      bool done = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        run += x[i];
        if (x[i] > 0.0 && !done) {
          p = i;
          done = passes && run > target;
        }
      }
      pick_s = piece * kPiece + threadIdx.x * 8 + p;
    }
    __syncthreads();
    pick = pick_s;
  }
  if (threadIdx.x == 0) args.bonus[r] = pick;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace hrs

using namespace hrs;

static bool sample_desc_ok(const hrs_sample_desc* d) {
  return d && d->n_req >= 1 && d->n_req <= 65535 && d->vocab >= 8 && d->vocab <= (1 << 30) && d->vocab % 8 == 0 && dtype_ok(d->logit_dtype) &&
         (d->topo == HRS_CHAIN || d->topo == HRS_TREE) && d->n_pos >= 1 && d->n_pos <= HRS_MAX_POS &&
         static_cast<int64_t>(d->n_req) * d->n_pos * ((static_cast<int64_t>(d->vocab) + 16383) / 16384) <= (1 << 24);
}

static int sample_chunks(const hrs_sample_desc* d) {
  const int chunk = d->logit_dtype == HRS_F32 ? kChunk<float> : kChunk<uint16_t>;
  return (d->vocab + chunk - 1) / chunk;
}
static int sample_pieces(const hrs_sample_desc* d) { return (d->vocab + kPiece - 1) / kPiece; }

extern "C" size_t accept_sample_workspace_bytes(const hrs_sample_desc* d) {
  if (!sample_desc_ok(d)) return 0;
  const size_t r = d->n_req;
  const size_t chunks = (d->vocab + kChunk<float> - 1) / kChunk<float>;   // enough for either type
  return round256(r * d->n_pos * chunks * sizeof(double2)) + round256(r * sample_pieces(d) * sizeof(double2)) +
         round256(r * sample_pieces(d) * sizeof(double)) + r * sizeof(NodeInfo);
}

// Statistics, walk and node sums of the n requests from req0.
template <typename T, typename Args> static bool launch_walk(const Args& args, int n, hipStream_t s) {
  const int rows = is_tree<Args> ? args.n_pos : args.n_pos - 1;
  if (rows > 0) {
    hipLaunchKernelGGL((row_stats_kernel<T, Args>), dim3(n * rows * args.n_chunks), dim3(kThreads), 0, s, args);
    if (launch_error() != hipSuccess) return false;
  }
  hipLaunchKernelGGL((node_kernel<T, Args>), dim3(args.n_pieces, n), dim3(kThreads), 0, s, args);
  return launch_error() == hipSuccess;
}

template <typename T> static int sample_launch(const hrs_sample_desc* d, SampleTree& tree_args, hipStream_t s) {
  SampleArgs& args = tree_args;
  const bool tree = d->topo == HRS_TREE;
  const int per_launch = tree ? std::max(1, kGeomBytes / d->n_pos) : d->n_req;
  (void)hipGetLastError();
  for (int r0 = 0; r0 < d->n_req; r0 += per_launch) {
    const int n = std::min(per_launch, d->n_req - r0);
    args.req0 = r0;
    if (tree)
      for (int i = 0; i < n * d->n_pos; ++i)
        tree_args.parent[i] = static_cast<int8_t>(d->parent[static_cast<size_t>(r0) * d->n_pos + i]);
    if (!(tree ? launch_walk<T>(tree_args, n, s) : launch_walk<T>(args, n, s))) return HRS_EDEVICE;
    if (args.draft) {
      hipLaunchKernelGGL(rest_kernel<T>, dim3(args.n_pieces, n), dim3(kThreads), 0, s, args);
      if (launch_error() != hipSuccess) return HRS_EDEVICE;
    }
    hipLaunchKernelGGL(draw_kernel<T>, dim3(n), dim3(kThreads), 0, s, args);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}

extern "C" int accept_sample(const hrs_sample_desc* d, const void* logits, const int32_t* tokens,
                             const float* uniforms, const void* draft_probs, const float* temperature,
                             float* token_prob, int32_t* accept_node, int32_t* accept_len, int32_t* path,
                             int32_t* bonus, int32_t* status, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (d == nullptr) return HRS_EINVAL;
  if (d->topo == HRS_TREE || d->topo == HRS_CHAIN) {
    const int geo = check_topology(d->topo, d->parent, d->n_req < 1 ? 0 : d->n_req, d->n_pos);
    if (geo != HRS_OK) return geo;
  }
  if (!sample_desc_ok(d) || (draft_probs && !dtype_ok(d->draft_dtype))) return HRS_EINVAL;
  if (draft_probs && d->topo == HRS_TREE) return HRS_EUNSUPPORTED;
  if (!logits || !tokens || !uniforms || !token_prob || !accept_node || !accept_len || !path || !bonus)
    return HRS_EINVAL;
  if (!workspace || workspace_bytes < accept_sample_workspace_bytes(d)) return HRS_EINVAL;
  if (!aligned16(logits) || !aligned16(tokens) || !aligned16(uniforms) || !aligned16(draft_probs) ||
      !aligned16(temperature) || !aligned16(token_prob) || !aligned16(accept_node) || !aligned16(accept_len) ||
      !aligned16(path) || !aligned16(bonus) || !aligned16(status) || !aligned16(workspace))
    return HRS_EALIGN;

  SampleTree args;
  args.logits = logits; args.tokens = tokens; args.uniforms = uniforms; args.draft = draft_probs;
  args.temperature = temperature; args.token_prob = token_prob; args.accept_node = accept_node;
  args.accept_len = accept_len; args.path = path; args.bonus = bonus; args.status = status;
  args.n_req = d->n_req; args.n_pos = d->n_pos; args.vocab = d->vocab;
  args.n_chunks = sample_chunks(d); args.n_pieces = sample_pieces(d);
  args.draft_bf16 = d->draft_dtype == HRS_BF16;
  char* at = static_cast<char*>(workspace);
  const size_t r = d->n_req;
  args.stats = reinterpret_cast<double2*>(at);
  at += round256(r * d->n_pos * args.n_chunks * sizeof(double2));
  args.part = reinterpret_cast<double2*>(at);
  at += round256(r * args.n_pieces * sizeof(double2));
  args.rest = reinterpret_cast<double*>(at);
  at += round256(r * args.n_pieces * sizeof(double));
  args.info = reinterpret_cast<NodeInfo*>(at);
  return d->logit_dtype == HRS_BF16 ? sample_launch<uint16_t>(d, args, static_cast<hipStream_t>(stream))
                                    : sample_launch<float>(d, args, static_cast<hipStream_t>(stream));
}
