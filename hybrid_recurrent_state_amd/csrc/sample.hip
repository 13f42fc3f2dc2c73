// accept_sample: verification of drafted tokens against the target's
// probabilities from given random numbers, for a chain (with or without the
// draft's probabilities) or a draft tree, and the draw of the next token.
//
// It stands beside accept_greedy (accept.hip) for requests that sample
// (openinfer PR #626, "feat(qwen35): add opt-in DFlash speculative decoding",
// Summary: greedy requests only; sampling falls back to plain decoding).
//
// Simple form: one block per row for its maximum and sum, then one block per
// request for the walk and the draw.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

constexpr int kThreads = 256;

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
  double2* stats;     // workspace [rows]: maximum, sum
  int32_t n_req;
  int32_t n_pos;
  int32_t vocab;
  int32_t req0;
  int32_t tree;
  int32_t draft_bf16;
  int8_t parent[kGeomBytes];
};

__device__ __forceinline__ bool bad_temperature(const SampleArgs& a, int r) {
  return a.temperature && !(a.temperature[r] >= 0.0f);
}

// Weight of a logit below the row's maximum m: e^((z - m) / tau). Hard rows
// (temperature 0, or +inf logits) give the largest logits one, the rest zero.
struct Weigher {
  double m, inv;
  bool hard, none;
  __device__ Weigher(double m_, float tau) : m(m_) {
    none = m == -__builtin_inf();
    hard = tau == 0.0f || m == __builtin_inf();
    inv = tau > 0.0f ? fmax(1.0 / static_cast<double>(tau), 1e-300) : 1.0;
  }
  __device__ double operator()(float z) const {
    if (none || z != z) return 0.0;
    if (hard) return z == m ? 1.0 : 0.0;
    return exp((static_cast<double>(z) - m) * inv);
  }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void row_stats_kernel(const SampleArgs args) {
  const int row = blockIdx.x;
  const T* z = static_cast<const T*>(args.logits) + static_cast<int64_t>(row) * args.vocab;
  __shared__ double red[kThreads];
  float m = -__builtin_inff();
  for (int i = threadIdx.x; i < args.vocab; i += kThreads) m = fmaxf(m, load_elem<T>(z, i));
  red[threadIdx.x] = m;
  __syncthreads();
  for (int s = kThreads / 2; s; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] = fmax(red[threadIdx.x], red[threadIdx.x + s]);
    __syncthreads();
  }
  const Weigher w(red[0], args.temperature ? args.temperature[row / args.n_pos] : 1.0f);
  __syncthreads();
  double sum = 0.0;
  for (int i = threadIdx.x; i < args.vocab; i += kThreads) sum += w(load_elem<T>(z, i));
  red[threadIdx.x] = sum;
  __syncthreads();
  for (int s = kThreads / 2; s; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  if (threadIdx.x == 0) args.stats[row] = double2{w.m, red[0]};
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs args) {
  const int rl = blockIdx.x, r = args.req0 + rl, T_ = args.n_pos, V = args.vocab;
  const int tid = threadIdx.x;
  if (r == 0 && tid == 0 && args.status) {
    int bad = 0;
    for (int i = 0; i < args.n_req; ++i) bad += bad_temperature(args, i);
    *args.status = bad;
  }
  if (bad_temperature(args, r)) return;
  const float tau = args.temperature ? args.temperature[r] : 1.0f;
  const int64_t row0 = static_cast<int64_t>(r) * T_;
  const T* logits = static_cast<const T*>(args.logits) + row0 * V;
  __shared__ double prob[HRS_MAX_POS];
  __shared__ int32_t par[HRS_MAX_POS], tok[HRS_MAX_POS], gone[HRS_MAX_POS];
  __shared__ int32_t node_s, gone_n, drafted_s;
  auto draft_at = [&](int t, int v) -> double {
    const int64_t i = (row0 + t) * V + v;
    return args.draft_bf16 ? bf16_one(static_cast<const uint16_t*>(args.draft)[i])
                           : static_cast<const float*>(args.draft)[i];
  };
  if (tid < T_) {
    const int p = args.tree ? args.parent[rl * T_ + tid] : tid - 1;
    const int x = args.tokens[row0 + tid];
    par[tid] = p;
    tok[tid] = x;
    double pr = tid == 0 ? 1.0 : 0.0;
    if (tid > 0 && x >= 0 && x < V) {
      const double2 st = args.stats[row0 + p];
      const Weigher w(st.x, tau);
      if (st.y > 0.0) pr = w(load_elem<T>(logits, static_cast<int64_t>(p) * V + x)) / st.y;
    }
    prob[tid] = pr;
    args.token_prob[row0 + tid] = static_cast<float>(pr);
  }
  __syncthreads();
  if (tid == 0) {
    const float* u = args.uniforms + row0;
    int node = 0, len = 0, n_gone = 0, path_n = 1;
    bool drafted = false;
    args.path[row0] = 0;
    for (;;) {
      int next = -1;
      double left = 1.0;
      n_gone = 0;
      for (int t = node + 1; t < T_ && next < 0; ++t) {
        if (par[t] != node) continue;
        if (args.draft) {
          const bool valid = tok[t] >= 0 && tok[t] < V;
          if (valid && static_cast<double>(u[t]) * draft_at(node, tok[t]) < prob[t]) next = t;
          else drafted = true;
          continue;
        }
        bool seen = false;
        for (int i = 0; i < n_gone; ++i) seen = seen || gone[i] == tok[t];
        if (seen) continue;
        if (static_cast<double>(u[t]) * left < prob[t]) {
          next = t;
        } else {
          left -= prob[t];
          gone[n_gone++] = tok[t];
        }
      }
      if (next < 0) break;
      node = next;
      ++len;
      args.path[row0 + path_n++] = node;
    }
    for (int i = path_n; i < T_; ++i) args.path[row0 + i] = -1;
    args.accept_node[r] = node;
    args.accept_len[r] = len;
    node_s = node;
    gone_n = n_gone;
    drafted_s = drafted;
  }
  __syncthreads();
  const int node = node_s;
  const T* z = logits + static_cast<int64_t>(node) * V;
  const double2 st = args.stats[row0 + node];
  const Weigher w(st.x, tau);
  const int per = (V + kThreads - 1) / kThreads;
  const int v0 = min(V, tid * per), v1 = min(V, v0 + per);
  __shared__ double sums[kThreads];
  __shared__ int32_t pick_s;
  for (int mode = drafted_s || gone_n ? 1 : 0; mode >= 0; --mode) {
    auto weight = [&](int v) -> double {
      double x = w(load_elem<T>(z, v));
      if (mode == 0) return x;
      if (drafted_s) {
        x = x / st.y - draft_at(node, v);
        return x > 0.0 ? x : 0.0;
      }
      for (int i = 0; i < gone_n; ++i) x = gone[i] == v ? 0.0 : x;
      return x;
    };
    double sum = 0.0;
    for (int v = v0; v < v1; ++v) sum += weight(v);
    sums[tid] = sum;
    __syncthreads();
    double total = 0.0;
    for (int i = 0; i < kThreads; ++i) total += sums[i];
    if (total > 0.0) {
      const double target = static_cast<double>(args.uniforms[row0]) * total;
      double before = 0.0;
      int owner = -1, last = 0;
      for (int i = 0; i < kThreads; ++i) {
        if (sums[i] > 0.0) last = i;
        if (owner < 0 && sums[i] > 0.0 && before + sums[i] > target) owner = i;
        if (owner < 0) before += sums[i];
      }
      if (owner < 0) {   // no cumulative sum passes: the last positive weight
        owner = last;
        before = -__builtin_inf();
      }
      if (tid == owner) {
        int pick = v0;
        for (int v = v0; v < v1; ++v) {
          const double x = weight(v);
          if (!(x > 0.0)) continue;
          pick = v;
          before += x;
          if (before > target) break;
        }
        pick_s = pick;
      }
      __syncthreads();
      if (tid == 0) args.bonus[r] = pick_s;
      return;
    }
    __syncthreads();
  }
  if (tid == 0) args.bonus[r] = 0;
}

}  // namespace
}  // namespace hrs

using namespace hrs;

static bool sample_desc_ok(const hrs_sample_desc* d) {
  return d && d->n_req >= 1 && d->n_req <= 65535 && d->vocab >= 8 && d->vocab % 8 == 0 && dtype_ok(d->logit_dtype) &&
         (d->topo == HRS_CHAIN || d->topo == HRS_TREE) && d->n_pos >= 1 && d->n_pos <= HRS_MAX_POS &&
         static_cast<int64_t>(d->n_req) * d->n_pos * ((static_cast<int64_t>(d->vocab) + 16383) / 16384) <= (1 << 24);
}

extern "C" size_t accept_sample_workspace_bytes(const hrs_sample_desc* d) {
  if (!sample_desc_ok(d)) return 0;
  return static_cast<size_t>(d->n_req) * d->n_pos * sizeof(double2);
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

  SampleArgs args;
  args.logits = logits; args.tokens = tokens; args.uniforms = uniforms; args.draft = draft_probs;
  args.temperature = temperature; args.token_prob = token_prob; args.accept_node = accept_node;
  args.accept_len = accept_len; args.path = path; args.bonus = bonus; args.status = status;
  args.stats = static_cast<double2*>(workspace);
  args.n_req = d->n_req; args.n_pos = d->n_pos; args.vocab = d->vocab; args.req0 = 0;
  args.tree = d->topo == HRS_TREE;
  args.draft_bf16 = d->draft_dtype == HRS_BF16;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf16 = d->logit_dtype == HRS_BF16;
  (void)hipGetLastError();
  const dim3 rows(d->n_req * d->n_pos);
  if (bf16)
    hipLaunchKernelGGL(row_stats_kernel<uint16_t>, rows, dim3(kThreads), 0, s, args);
  else
    hipLaunchKernelGGL(row_stats_kernel<float>, rows, dim3(kThreads), 0, s, args);
  if (launch_error() != hipSuccess) return HRS_EDEVICE;
  const int per_launch = args.tree ? std::max(1, kGeomBytes / d->n_pos) : d->n_req;
  for (int r0 = 0; r0 < d->n_req; r0 += per_launch) {
    const int n = std::min(per_launch, d->n_req - r0);
    args.req0 = r0;
    if (args.tree)
      for (int i = 0; i < n * d->n_pos; ++i)
        args.parent[i] = static_cast<int8_t>(d->parent[static_cast<size_t>(r0) * d->n_pos + i]);
    if (bf16)
      hipLaunchKernelGGL(sample_kernel<uint16_t>, dim3(n), dim3(kThreads), 0, s, args);
    else
      hipLaunchKernelGGL(sample_kernel<float>, dim3(n), dim3(kThreads), 0, s, args);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}
