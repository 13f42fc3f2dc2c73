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

#include "sample.h"

namespace hrs {
namespace {

// Logits per statistics block, 32 KB of either type (16 rows of 151,936 bf16
// logits: 8192 logits a block level, 32,768 8% slower; float32: 16,384 7%
// slower).
template <typename T> constexpr int kChunk = 32768 / sizeof(T);

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
    // Differences times 1 / (tau ln 2), either scaled by a power of two where
    // one of them would leave float32's range and their product not: logits far
    // apart at a large temperature, logits near zero at a very small one (others
    // that differ are too far apart there).
    const float by = tau >= 0x1p60f ? 0x1p-64f : tau < 0x1p-100f && fabsf(m) < 0x1p-40f ? 0x1p64f : 1.0f;
    const float c = fminf(1.4426950408889634f / (tau * by), 3.4e38f);
    const float mb = m * by;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      float s8 = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i)       // a NaN becomes -inf, of weight zero
        s8 += __builtin_amdgcn_exp2f(fmaxf(fmaf(v[it][i], by, -mb) * c, -__builtin_inff()));
      if (begin + (it * kThreads + threadIdx.x) * 8 < end) sum += s8;
    }
  }
  const double total = block_reduce(sum, add, lds);
  if (threadIdx.x == 0) args.stats[row * args.n_chunks + chunk] = double2{m, total};
}

// The walk of request r, by the whole block; the first block of the request
// writes its outputs.
template <typename T, typename Args>
__device__ __forceinline__ void walk(const Args& args, int rl, bool write, WalkLds& w) {
  const int r = args.req0 + rl, T_ = args.n_pos, V = args.vocab;
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
  decide(args, rl, write, w);
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
