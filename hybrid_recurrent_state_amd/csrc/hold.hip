// accept_hold: takes the requests that cannot go on out of an acceptance,
// before anything is committed.
//
// lucebox PR #506 ("perf(dflash): split-chain fast rollback with F32 SSM
// checkpoints"), Safety boundary: what cannot be carried out is rejected
// before it starts; lucebox PR #533, Changes: nothing goes through the host
// between acceptance and commit, so neither does this decision.
//
// MI355X design: bound by the launch (a 1.9 us kernel). A wave holds a
// request, a lane one of its positions: path entries in one round of loads with
// the lengths, the pages of the accepted rows in the next.
#include <hip/hip_runtime.h>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

constexpr int kThreads = 256;

struct HoldArgs {
  const int32_t* page_table;
  const int32_t* seq_len;
  const float* temperature;
  int32_t* accept_node;
  int32_t* accept_len;
  int32_t* path;
  int32_t* bonus;
  int32_t* held;
  int32_t* last_node;
  int32_t* held_node;
  int32_t n_req;
  int32_t n_pos;
  int32_t n_pages;
  int32_t page_shift;
  int32_t table_len;
  int32_t prefix_len;
};

__global__ __launch_bounds__(kThreads) void hold_kernel(const HoldArgs a) {
  const int r = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (r >= a.n_req) return;
  const int64_t row = static_cast<int64_t>(r) * a.n_pos;
  const int entry = a.path[row + min(lane, a.n_pos - 1)];
  const int len = a.seq_len[r], n = a.accept_len[r], node = a.accept_node[r], before = a.held[r];
  const float tau = a.temperature ? a.temperature[r] : 1.0f;
  const int64_t slots = static_cast<int64_t>(a.table_len) << a.page_shift;
  bool ok = before == 0 && n >= 0 && n < a.n_pos && node >= 0 && node < a.n_pos && tau >= 0.0f && len >= a.prefix_len &&
            static_cast<int64_t>(len) + n + 1 <= slots;
  if (ok) {
    bool fits = true;
    if (lane <= n) {
      const int page = a.page_table[static_cast<int64_t>(r) * a.table_len + ((len + lane) >> a.page_shift)];
      fits = entry >= 0 && entry < a.n_pos && page >= 0 && page < a.n_pages;
    }
    ok = __all(fits);
  }
  if (ok) {
    if (lane == 0) a.last_node[r] = node;
    return;
  }
  if (lane < a.n_pos) a.path[row + lane] = -1;
  if (lane == 0) {
    if (before == 0) {
      a.held[r] = 1;
      if (a.held_node) a.held_node[r] = a.last_node[r];
    }
    a.accept_node[r] = -1;
    a.accept_len[r] = -1;
    a.bonus[r] = -1;
  }
}

}  // namespace
}  // namespace hrs

using namespace hrs;

extern "C" int accept_hold_behind(const hrs_hold_desc* d, int32_t prefix_len, const int32_t* page_table, const int32_t* seq_len,
                                  const float* temperature, int32_t* accept_node, int32_t* accept_len, int32_t* path,
                                  int32_t* bonus, int32_t* held, int32_t* last_node, int32_t* held_node, void* stream) {
  if (d == nullptr) return HRS_EINVAL;
  const bool pages_ok = d->page_size >= 16 && d->page_size <= 1024 && (d->page_size & (d->page_size - 1)) == 0 &&
                        d->n_pages >= 1 && d->table_len >= 1 &&
                        static_cast<int64_t>(d->table_len) * d->page_size <= INT32_MAX - HRS_MAX_CHUNKED_POS;
  if (d->n_req < 1 || d->n_req > 65535 || d->n_pos < 1 || d->n_pos > HRS_MAX_POS || prefix_len < 0 || !pages_ok)
    return HRS_EINVAL;
  if (!page_table || !seq_len || !accept_node || !accept_len || !path || !bonus || !held || !last_node)
    return HRS_EINVAL;
  if (!aligned16(page_table) || !aligned16(seq_len) || !aligned16(temperature) || !aligned16(accept_node) ||
      !aligned16(accept_len) || !aligned16(path) || !aligned16(bonus) || !aligned16(held) || !aligned16(last_node) ||
      !aligned16(held_node))
    return HRS_EALIGN;
  const HoldArgs args{page_table, seq_len, temperature, accept_node, accept_len, path, bonus, held, last_node, held_node,
                      d->n_req, d->n_pos, d->n_pages, __builtin_ctz(static_cast<unsigned>(d->page_size)), d->table_len,
                      prefix_len};
  (void)hipGetLastError();
  hipLaunchKernelGGL(hold_kernel, dim3((d->n_req + kThreads / 64 - 1) / (kThreads / 64)), dim3(kThreads), 0,
                     static_cast<hipStream_t>(stream), args);
  return launch_error() == hipSuccess ? HRS_OK : HRS_EDEVICE;
}

extern "C" int accept_hold(const hrs_hold_desc* d, const int32_t* page_table, const int32_t* seq_len,
                           const float* temperature, int32_t* accept_node, int32_t* accept_len, int32_t* path,
                           int32_t* bonus, int32_t* held, int32_t* last_node, int32_t* held_node, void* stream) {
  return accept_hold_behind(d, 0, page_table, seq_len, temperature, accept_node, accept_len, path, bonus, held, last_node,
                            held_node, stream);
}
