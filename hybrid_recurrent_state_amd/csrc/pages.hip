// kv_pages_reserve(_step), kv_pages_release: page tables that grow from a free list
// and shrink back into it on the device, and the slots of new positions.
//
// openinfer PR #626 ("feat(qwen35): add opt-in DFlash speculative decoding"),
// What Changed: the hybrid state includes a paged KV cache; lucebox PR #533
// ("feat: DFlash support for tensor-parallel Qwen3.6 targets"), Changes:
// nothing goes through the host between the parts of a step.
//
// The list is a stack. What all requests of a call take or give back is one
// block of it, in request order, so a request's place is a prefix sum over the
// requests before it and every entry can be written independently of the
// others; giving back what was taken restores the stack.
//
// MI355X design. A verify step's lists are a few entries a request: one block
// of 1024 threads sums in LDS and then takes the entries of all requests as one
// flat list (a binary search names an entry's request), so neither many short
// nor a few long requests leave threads idle; the launch bounds it (reserve 6.0
// us, release 4.7 for 16 requests). Prompts (reserve) and long tables (release)
// take a second launch of many blocks behind the sums, bound by the slot map's
// writes (67 MB for 256 prompts: 15.1 us, 4.5 TB/s). Reserve chooses by the slot
// map: few new positions whose requests get all entries of long tables at once
// are one block's work (calls: 256 requests that start behind 1672 pages of a
// prefix 71 us, that get 1673 pages each 368). Release's second launch sums what
// is before each request again (4096 requests of 2 pages: 17 us).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

constexpr int kReqs = 4096;            // requests of a call at most
constexpr int kThreads = 1024;
constexpr int kPer = kReqs / kThreads;
constexpr int kFill = 256;             // threads of a block of the second launch
constexpr int kFillSlots = 4096;       // positions of a request that one of its blocks takes

struct PagesArgs {
  const int32_t* len;        // seq_len or keep_len
  const int32_t* n_new;
  const int32_t* skip;
  const int32_t* prefix_table;
  int32_t* page_table;
  int32_t* n_held;
  int32_t* free_pages;
  int32_t* n_free;
  int64_t* slot_map;
  int32_t* status;
  struct Plan* plan;         // workspace [R + 1]
  int32_t n_req;
  int32_t n_pos;
  int32_t n_pages;
  int32_t page_shift;
  int32_t table_len;
  int32_t n_prefix;
  int32_t clip;
};

// What the second launch needs to know of a request.
struct Plan {
  int32_t len;       // reserve: seq_len; -1: refused or passed over
  int32_t n_new;
  int32_t held;      // entries before the call
  int32_t have;      // reserve: entries with the prefix's; release: entries that stay
  int32_t count;     // entries taken; release: entries given back that name pages
  int32_t first;     // place of the first in the list (release: of the call's first, in the plan behind the last)
};

__device__ __forceinline__ int32_t clamp_free(int32_t n, int32_t n_pages) { return max(0, min(n, n_pages)); }

// Sum of x over the threads up to and with this one; *total over all. Two
// barriers; lds has a place per wave.
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* lds, int64_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    x += lane >= d ? y : 0;
  }
  __syncthreads();
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    before += i < wave ? lds[i] : 0;
    all += lds[i];
  }
  *total = all;
  return before + x;
}

// Page of table entry e of a request, as it will be after the call.
__device__ __forceinline__ int32_t page_at(const PagesArgs& a, int r, const Plan& p, int e) {
  if (e < p.held) return a.page_table[static_cast<int64_t>(r) * a.table_len + e];
  if (e < p.have) return a.prefix_table[e];
  return e - p.have < p.count ? a.free_pages[p.first + e - p.have] : -1;
}

__device__ __forceinline__ void write_slot(const PagesArgs& a, int r, const Plan& p, int t) {
  int64_t slot = -1;
  if (p.len >= 0 && t < p.n_new) {
    const int64_t j = static_cast<int64_t>(p.len) + t;
    const int e = static_cast<int>(min(j >> a.page_shift, static_cast<int64_t>(a.table_len)));
    const int32_t page = page_at(a, r, p, e);
    if (page >= 0 && page < a.n_pages)
      slot = (static_cast<int64_t>(page) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
  }
  a.slot_map[static_cast<int64_t>(r) * a.n_pos + t] = slot;
}

// One block: the requests' places, lengths and the list's; with ALL also the
// entries and the slot map.
template <bool ALL> __global__ __launch_bounds__(kThreads) void reserve_kernel(const PagesArgs a) {
  __shared__ int64_t lds[kThreads / 64];
  __shared__ int32_t before[ALL ? kReqs : 1];
  __shared__ Plan plans[ALL ? kReqs : 1];
  const int tid = threadIdx.x;
  const int32_t in_list = clamp_free(*a.n_free, a.n_pages);
  Plan p[kPer];
  int64_t need[kPer], sum = 0;
  int32_t skips[kPer] = {};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = tid * kPer + k, rr = min(r, a.n_req - 1);
    p[k].len = a.len[rr];
    p[k].n_new = a.n_new ? a.n_new[rr] : a.n_pos;
    p[k].held = a.n_held[rr];
  }
  if (a.skip) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) skips[k] = a.skip[min(tid * kPer + k, a.n_req - 1)];
  }
  // Slots that new positions may take (kv_pages_reserve refuses longer requests).
  const int32_t room = a.clip ? a.table_len << a.page_shift : INT32_MAX;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const bool in_range = p[k].len >= 0 && p[k].n_new >= 0 && p[k].n_new <= a.n_pos;
    if (in_range) p[k].n_new = min(p[k].n_new, max(0, room - p[k].len));
    const int64_t want = (static_cast<int64_t>(p[k].len) + p[k].n_new + (1 << a.page_shift) - 1) >> a.page_shift;
    const bool ok = in_range && want <= a.table_len && p[k].held >= 0 && p[k].held <= a.table_len && skips[k] == 0;
    if (!ok) p[k].len = -1;
    p[k].have = max(p[k].held, a.n_prefix);
    need[k] = ok && tid * kPer + k < a.n_req ? max(want - p[k].have, int64_t{0}) : 0;
    sum += need[k];
  }
  int64_t total;
  int64_t upto = block_sum(sum, lds, &total) - sum;      // of the requests before the thread's
  int64_t taken = 0;
  int bad = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = tid * kPer + k;
    p[k].first = static_cast<int32_t>(min(upto, static_cast<int64_t>(in_list)));
    upto += need[k];
    p[k].count = upto <= in_list ? static_cast<int32_t>(need[k]) : 0;
    taken += p[k].count;
    bad += r < a.n_req && skips[k] == 0 && (p[k].len < 0 || p[k].count < need[k]);
  }
  int64_t all_taken, all_bad;
  block_sum(taken, lds, &all_taken);
  if (a.status) block_sum(bad, lds, &all_bad);
  const int32_t base = in_list - static_cast<int32_t>(all_taken);
  bool starts = false;                                   // some request gets the prefix's pages
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = tid * kPer + k;
    if constexpr (ALL) before[r] = p[k].first;           // (what is not served stands behind all that is)
    p[k].first += base;
    if (r >= a.n_req) continue;
    if constexpr (ALL) plans[r] = p[k];
    else a.plan[r] = p[k];
    if (p[k].len < 0) continue;
    a.n_held[r] = p[k].have + p[k].count;
    starts = starts || p[k].held < a.n_prefix;
  }
  if (tid == 0) {
    *a.n_free = base;
    if (a.status) *a.status = static_cast<int32_t>(all_bad);
  }
  if constexpr (ALL) {
    __syncthreads();
    for (int32_t e = tid; e < all_taken; e += kThreads) {
      // The last request whose first entry is at or before e: of those with
      // the same first only the last one takes any.
      int lo = 0, hi = a.n_req - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= e) lo = mid;
        else hi = mid - 1;
      }
      const Plan& q = plans[lo];
      a.page_table[static_cast<int64_t>(lo) * a.table_len + q.have + (e - before[lo])] = a.free_pages[base + e];
    }
    if (__syncthreads_or(starts))
      for (int r = tid >> 6; r < a.n_req; r += kThreads / 64)
        if (plans[r].len >= 0)
          for (int e = plans[r].held + (tid & 63); e < a.n_prefix; e += 64)
            a.page_table[static_cast<int64_t>(r) * a.table_len + e] = a.prefix_table[e];
    if (a.slot_map)
      for (int i = tid; i < a.n_req * a.n_pos; i += kThreads) {
        const int r = i / a.n_pos;
        write_slot(a, r, plans[r], i - r * a.n_pos);
      }
  }
}

// Grid: (request, part of its positions).
__global__ __launch_bounds__(kFill) void reserve_fill_kernel(const PagesArgs a) {
  const int r = blockIdx.x, step = gridDim.y * kFill;
  const Plan p = a.plan[r];
  const int first = blockIdx.y * kFill + threadIdx.x;
  if (p.len >= 0) {
    int32_t* const table = a.page_table + static_cast<int64_t>(r) * a.table_len;
    for (int e = p.held + first; e < p.have; e += step) table[e] = a.prefix_table[e];
    for (int e = first; e < p.count; e += step) table[p.have + e] = a.free_pages[p.first + e];
  }
  if (a.slot_map)
    for (int t = first; t < a.n_pos; t += step) write_slot(a, r, p, t);
}

// Entries of request r that go back: [keep, held).
struct Back {
  int keep, held;
  bool ok;
};
__device__ __forceinline__ Back back_of(const PagesArgs& a, int r) {
  const int32_t len = a.len[r], held = a.n_held[r];
  const bool ok = len >= 0 && held >= 0 && held <= a.table_len;
  const int64_t pages = (static_cast<int64_t>(len) + (1 << a.page_shift) - 1) >> a.page_shift;
  const int keep = static_cast<int>(max(min(pages, static_cast<int64_t>(a.table_len)), static_cast<int64_t>(a.n_prefix)));
  return {keep, ok ? max(held, keep) : keep, ok};
}

// One block, the whole call: the entries of all requests as one list, 1024 at
// a time.
__global__ __launch_bounds__(kThreads) void release_kernel(const PagesArgs a) {
  __shared__ int64_t lds[kThreads / 64];
  __shared__ int32_t before[kReqs], keep[kReqs];
  const int tid = threadIdx.x;
  const int32_t in_list = clamp_free(*a.n_free, a.n_pages);
  Back b[kPer];
  int64_t sum = 0;
  int bad = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = tid * kPer + k;
    b[k] = back_of(a, min(r, a.n_req - 1));
    if (r >= a.n_req) b[k].held = b[k].keep;
    sum += b[k].held - b[k].keep;
    bad += r < a.n_req && !b[k].ok;
  }
  int64_t total, all_bad;
  int64_t upto = block_sum(sum, lds, &total) - sum;
  if (a.status) block_sum(bad, lds, &all_bad);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = tid * kPer + k;
    before[r] = static_cast<int32_t>(upto);              // (R x table_len is bounded by the host)
    keep[r] = b[k].keep;
    upto += b[k].held - b[k].keep;
    if (r < a.n_req && b[k].held > b[k].keep) a.n_held[r] = b[k].keep;
  }
  __syncthreads();
  int64_t top = in_list;
  for (int64_t e0 = 0; e0 < total; e0 += kThreads) {
    const int64_t e = e0 + tid;
    int32_t page = -1;
    if (e < total) {
      int lo = 0, hi = a.n_req - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= e) lo = mid;
        else hi = mid - 1;
      }
      int32_t* const at = a.page_table + static_cast<int64_t>(lo) * a.table_len + keep[lo] + (e - before[lo]);
      page = *at;
      *at = -1;
    }
    const bool is_page = page >= 0 && page < a.n_pages;
    int64_t n;
    const int64_t place = top + block_sum(is_page, lds, &n) - 1;
    if (is_page && place < a.n_pages) a.free_pages[place] = page;
    top += n;
  }
  if (tid == 0) {
    *a.n_free = static_cast<int32_t>(min(top, static_cast<int64_t>(a.n_pages)));
    if (a.status) *a.status = static_cast<int32_t>(all_bad);
  }
}

// Sum over the block of kFill threads.
__device__ __forceinline__ int64_t fill_sum(int64_t x, int64_t* lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}

// Long tables, first launch. Grid: request. How many entries go back; the
// list's length and the refused requests, which the second launch changes or
// can no longer tell, go into the plan behind the last request.
__global__ __launch_bounds__(kFill) void release_count_kernel(const PagesArgs a) {
  __shared__ int64_t lds[kFill / 64];
  const int r = blockIdx.x;
  const Back b = back_of(a, r);
  const int32_t* const table = a.page_table + static_cast<int64_t>(r) * a.table_len;
  int n = 0;
  for (int e = b.keep + static_cast<int>(threadIdx.x); e < b.held; e += kFill) {
    const int32_t page = table[e];
    n += page >= 0 && page < a.n_pages;
  }
  const int64_t count = fill_sum(n, lds);
  if (threadIdx.x == 0) a.plan[r] = Plan{b.ok ? 0 : -1, 0, b.held, b.keep, static_cast<int32_t>(count), 0};
  if (r == 0) {
    int bad = 0;
    if (a.status)
      for (int i = threadIdx.x; i < a.n_req; i += kFill) bad += !back_of(a, i).ok;
    const int64_t all_bad = fill_sum(bad, lds);
    if (threadIdx.x == 0) {
      a.plan[a.n_req] = Plan{0, 0, 0, 0, 0, clamp_free(*a.n_free, a.n_pages)};
      if (a.status) *a.status = static_cast<int32_t>(all_bad);
    }
  }
}

// Second launch. Grid: request.
__global__ __launch_bounds__(kFill) void release_fill_kernel(const PagesArgs a) {
  __shared__ int64_t lds[kFill / 64];
  __shared__ int32_t waves[kFill / 64];
  const int r = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Plan p = a.plan[r];
  int64_t n = 0;
  for (int i = threadIdx.x; i < r; i += kFill) n += a.plan[i].count;
  int64_t top = a.plan[a.n_req].first + fill_sum(n, lds);
  int32_t* const table = a.page_table + static_cast<int64_t>(r) * a.table_len;
  for (int e0 = p.have; e0 < p.held; e0 += kFill) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int32_t page = e < p.held ? table[e] : -1;
    const bool is_page = page >= 0 && page < a.n_pages;
    const uint64_t b = __ballot(is_page);
    __syncthreads();
    if (lane == 0) waves[wave] = __popcll(b);
    __syncthreads();
    int64_t place = top + __popcll(b & ((uint64_t{1} << lane) - 1));
    for (int i = 0; i < kFill / 64; ++i) {
      place += i < wave ? waves[i] : 0;
      top += waves[i];
    }
    if (is_page && place < a.n_pages) a.free_pages[place] = page;
    if (e < p.held) table[e] = -1;
  }
  if (threadIdx.x == 0) {
    if (p.held > p.have) a.n_held[r] = p.have;
    if (r == a.n_req - 1) *a.n_free = static_cast<int32_t>(min(top, static_cast<int64_t>(a.n_pages)));
  }
}

bool pages_desc_ok(const hrs_pages_desc* d) {
  return d && d->n_req >= 1 && d->n_req <= kReqs && d->n_pos >= 1 && d->n_pos <= HRS_MAX_CHUNKED_POS &&
         d->page_size >= 16 && d->page_size <= 1024 && (d->page_size & (d->page_size - 1)) == 0 && d->n_pages >= 1 &&
         d->table_len >= 1 && static_cast<int64_t>(d->table_len) * d->page_size <= INT32_MAX - HRS_MAX_CHUNKED_POS &&
         d->n_prefix >= 0 && d->n_prefix <= d->table_len;
}

PagesArgs pages_args(const hrs_pages_desc* d, const int32_t* len, int32_t* page_table, int32_t* n_held,
                     int32_t* free_pages, int32_t* n_free, int32_t* status, void* workspace) {
  PagesArgs a{};
  a.len = len; a.page_table = page_table; a.n_held = n_held; a.free_pages = free_pages; a.n_free = n_free;
  a.status = status; a.plan = static_cast<Plan*>(workspace);
  a.n_req = d->n_req; a.n_pos = d->n_pos; a.n_pages = d->n_pages; a.table_len = d->table_len; a.n_prefix = d->n_prefix;
  a.page_shift = __builtin_ctz(static_cast<unsigned>(d->page_size));
  return a;
}

}  // namespace
}  // namespace hrs

using namespace hrs;

extern "C" size_t kv_pages_workspace_bytes(const hrs_pages_desc* d) {
  if (!pages_desc_ok(d)) return 0;
  return (static_cast<size_t>(d->n_req) + 1) * sizeof(Plan);
}

static int reserve(const hrs_pages_desc* d, bool clip, const int32_t* seq_len, const int32_t* n_new, const int32_t* skip,
                   const int32_t* prefix_table, int32_t* page_table, int32_t* n_held, const int32_t* free_pages,
                   int32_t* n_free, int64_t* slot_map, int32_t* status, void* workspace, size_t workspace_bytes,
                   void* stream) {
  if (!pages_desc_ok(d)) return HRS_EINVAL;
  if (!seq_len || !page_table || !n_held || !free_pages || !n_free || (d->n_prefix > 0) != (prefix_table != nullptr))
    return HRS_EINVAL;
  if (!workspace || workspace_bytes < kv_pages_workspace_bytes(d)) return HRS_EINVAL;
  if (!aligned16(seq_len) || !aligned16(n_new) || !aligned16(prefix_table) || !aligned16(page_table) || !aligned16(n_held) ||
      !aligned16(free_pages) || !aligned16(n_free) || !aligned16(slot_map) || !aligned16(status) || !aligned16(workspace) ||
      !aligned16(skip))
    return HRS_EALIGN;
  PagesArgs a = pages_args(d, seq_len, page_table, n_held, const_cast<int32_t*>(free_pages), n_free, status, workspace);
  a.n_new = n_new; a.skip = skip; a.clip = clip; a.prefix_table = prefix_table; a.slot_map = slot_map;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  // One block where the slot map has few entries: it writes 1024 at a time.
  if (static_cast<int64_t>(d->n_req) * d->n_pos <= 16384) {
    hipLaunchKernelGGL(reserve_kernel<true>, dim3(1), dim3(kThreads), 0, s, a);
    return launch_error() == hipSuccess ? HRS_OK : HRS_EDEVICE;
  }
  hipLaunchKernelGGL(reserve_kernel<false>, dim3(1), dim3(kThreads), 0, s, a);
  if (launch_error() != hipSuccess) return HRS_EDEVICE;
  hipLaunchKernelGGL(reserve_fill_kernel, dim3(d->n_req, (d->n_pos + kFillSlots - 1) / kFillSlots), dim3(kFill), 0, s, a);
  return launch_error() == hipSuccess ? HRS_OK : HRS_EDEVICE;
}

extern "C" int kv_pages_reserve(const hrs_pages_desc* d, const int32_t* seq_len, const int32_t* n_new,
                                const int32_t* prefix_table, int32_t* page_table, int32_t* n_held,
                                const int32_t* free_pages, int32_t* n_free, int64_t* slot_map, int32_t* status,
                                void* workspace, size_t workspace_bytes, void* stream) {
  return reserve(d, false, seq_len, n_new, nullptr, prefix_table, page_table, n_held, free_pages, n_free, slot_map, status,
                 workspace, workspace_bytes, stream);
}

extern "C" int kv_pages_reserve_step(const hrs_pages_desc* d, const int32_t* seq_len, const int32_t* n_new,
                                     const int32_t* skip, const int32_t* prefix_table, int32_t* page_table, int32_t* n_held,
                                     const int32_t* free_pages, int32_t* n_free, int64_t* slot_map, int32_t* status,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  return reserve(d, true, seq_len, n_new, skip, prefix_table, page_table, n_held, free_pages, n_free, slot_map, status,
                 workspace, workspace_bytes, stream);
}

extern "C" int kv_pages_release(const hrs_pages_desc* d, const int32_t* keep_len, int32_t* page_table, int32_t* n_held,
                                int32_t* free_pages, int32_t* n_free, int32_t* status, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (!pages_desc_ok(d)) return HRS_EINVAL;
  if (!keep_len || !page_table || !n_held || !free_pages || !n_free) return HRS_EINVAL;
  if (!workspace || workspace_bytes < kv_pages_workspace_bytes(d)) return HRS_EINVAL;
  if (!aligned16(keep_len) || !aligned16(page_table) || !aligned16(n_held) || !aligned16(free_pages) || !aligned16(n_free) ||
      !aligned16(status) || !aligned16(workspace))
    return HRS_EALIGN;
  const PagesArgs a = pages_args(d, keep_len, page_table, n_held, free_pages, n_free, status, workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  // One block where the tables have few entries: it takes 1024 at a time.
  if (static_cast<int64_t>(d->n_req) * d->table_len <= 65536) {
    hipLaunchKernelGGL(release_kernel, dim3(1), dim3(kThreads), 0, s, a);
    return launch_error() == hipSuccess ? HRS_OK : HRS_EDEVICE;
  }
  hipLaunchKernelGGL(release_count_kernel, dim3(d->n_req), dim3(kFill), 0, s, a);
  if (launch_error() != hipSuccess) return HRS_EDEVICE;
  hipLaunchKernelGGL(release_fill_kernel, dim3(d->n_req), dim3(kFill), 0, s, a);
  return launch_error() == hipSuccess ? HRS_OK : HRS_EDEVICE;
}
