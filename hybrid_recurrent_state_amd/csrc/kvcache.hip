// kv_cache_append: the accepted rows of a span into the cache pages of every
// layer, in one launch, with the accepted path, the lengths and the page
// table read on the device.
//
// openinfer PR #626 ("feat(qwen35): add opt-in DFlash speculative decoding"),
// What Changed: the hybrid state that a commit advances is the recurrent
// state, the conv state and the attention layers' cache; lucebox PR #533,
// Changes: nothing goes through the host between acceptance and commit.
//
// MI355X design: a scattered copy bound by memory and, for the few rows of a
// verify step, by the launch. The span's rows stay outside the pages until
// they are accepted, so drafts never occupy cache slots, a rejected branch
// leaves no trace and no row has to move inside the cache (rows that move
// onto each other's slots would need an order). A block takes four rows of one
// layer: lengths and path come in one round of loads, the pages in the next,
// then 16-byte pieces of all heads' keys and values, four per thread on their
// way at once.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* accept_len;
  const int32_t* path;
  const float* k_scale;
  const float* v_scale;
  int32_t* seq_len_out;
  int32_t* status;
  int64_t k_stride;
  int64_t v_stride;
  int32_t n_req;
  int32_t n_pos;
  int32_t heads;
  int32_t d;
  int32_t n_pages;
  int32_t page_shift;
  int32_t table_len;
  int32_t lens_here;   // this launch writes seq_len_out and status
};

// Whether request r's call is valid; its length and accepted rows.
__device__ __forceinline__ bool request_ok(const AppendArgs& a, int r, int* len, int* n) {
  *len = a.seq_len[r];
  const int al = a.accept_len[r];
  *n = al + 1;
  if (al < 0 || al >= a.n_pos || *len < 0) return false;
  return static_cast<int64_t>(*len) + al + 1 <= (static_cast<int64_t>(a.table_len) << a.page_shift);
}

// The new lengths and the count of refused requests, by one block, a request
// per thread (its path's loads do not depend on each other).
__device__ void write_lengths(const AppendArgs& a) {
  __shared__ int32_t bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int r = threadIdx.x; r < a.n_req; r += kThreads) {
    int len, n;
    bool ok = request_ok(a, r, &len, &n);
    if (ok && a.path) {
      for (int i = 0; i < n; ++i) {
        const int p = a.path[static_cast<int64_t>(r) * a.n_pos + i];
        ok = ok && p >= 0 && p < a.n_pos;
      }
    }
    if (a.seq_len_out) a.seq_len_out[r] = ok ? len + n : len;
    if (!ok) atomicAdd(&bad, 1);
  }
  __syncthreads();
  if (a.status && threadIdx.x == 0) *a.status = bad;
}

// Eight bf16 values to e4m3: divided by the scale (rounded once), limited to
// the largest e4m3 number, NaN kept.
__device__ __forceinline__ float e4m3_range(float x, float scale) {
  const float y = x / scale;
  return y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
}
__device__ __forceinline__ u32x2 to_e4m3(u32x4 w, float scale) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = e4m3_range(bf16_lo(w[i]), scale);
    x[2 * i + 1] = e4m3_range(bf16_hi(w[i]), scale);
  }
  uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  uint32_t hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
  return u32x2{lo, hi};
}

constexpr int kRows = 4;      // span rows of a block
constexpr int kBatch = 4;     // pieces of a thread whose loads go out together

// Grid: (blocks of kRows rows, request, layer). ESZ: bytes of a span element;
// F8: the cache is e4m3. A piece is 16 bytes of the span; the block's pieces
// are (row, K or V, head, piece of the head).
template <int ESZ, bool F8>
__global__ __launch_bounds__(kThreads) void append_kernel(const AppendArgs args) {
  const int r = blockIdx.y;
  const int layer = blockIdx.z;
  if (args.lens_here && blockIdx.x == 0 && r == 0 && layer == 0) write_lengths(args);
  // Lengths and path in one round of loads.
  const int lane = threadIdx.x & 63;
  const int i0 = blockIdx.x * kRows;
  int entry = lane;
  if (args.path) entry = args.path[static_cast<int64_t>(r) * args.n_pos + min(lane, args.n_pos - 1)];
  int len, n;
  if (!request_ok(args, r, &len, &n)) return;
  if (args.path && !__all(lane >= n || (entry >= 0 && entry < args.n_pos))) return;
  const int i1 = min(n, i0 + kRows);
  if (i0 >= i1) return;
  // Page and span position of every row of the block.
  int page[kRows], pos[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = min(i0 + i, n - 1);
    page[i] = args.page_table[static_cast<int64_t>(r) * args.table_len + ((len + row) >> args.page_shift)];
    pos[i] = args.path ? __builtin_amdgcn_readlane(entry, row) : row;
  }
  const int d = args.d, heads = args.heads;
  const int per_head = d * ESZ / 16;
  const int per_row = 2 * heads * per_head;
  const int pieces = (i1 - i0) * per_row;
  const int64_t span_row0 = (static_cast<int64_t>(layer) * args.n_req + r) * args.n_pos;
  const int page_mask = (1 << args.page_shift) - 1;
  constexpr int kOut = F8 ? 8 : 16;               // bytes of a piece in the cache
  for (int p0 = threadIdx.x; p0 < pieces; p0 += kThreads * kBatch) {
    u32x4 x[kBatch];
    float scale[kBatch];
    char* to[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int p = min(p0 + b * kThreads, pieces - 1);
      const int row = p / per_row, in_row = p - row * per_row;
      const int item = in_row / per_head, piece = in_row - item * per_head;
      const bool is_v = item >= heads;
      const int h = is_v ? item - heads : item;
      int pg = page[0], ps = pos[0];
#pragma unroll
      for (int i = 1; i < kRows; ++i) {
        pg = row == i ? page[i] : pg;
        ps = row == i ? pos[i] : ps;
      }
      const char* const src = static_cast<const char*>(is_v ? args.v : args.k) +
                              ((span_row0 + ps) * (is_v ? args.v_stride : args.k_stride) + static_cast<int64_t>(h) * d) * ESZ;
      x[b] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src) + piece);
      if constexpr (F8) {
        const float* sc = is_v ? args.v_scale : args.k_scale;
        scale[b] = sc ? sc[static_cast<int64_t>(layer) * heads + h] : 1.0f;
      }
      const int slot = len + i0 + row;
      const int64_t at = ((static_cast<int64_t>(layer) * args.n_pages + pg) * heads + h) * (page_mask + 1) +
                         (slot & page_mask);
      const bool there = pg >= 0 && pg < args.n_pages && p0 + b * kThreads < pieces;
      to[b] = there ? static_cast<char*>(is_v ? args.v_cache : args.k_cache) + (at * per_head + piece) * kOut : nullptr;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (to[b] == nullptr) continue;
      if constexpr (F8) *reinterpret_cast<u32x2*>(to[b]) = to_e4m3(x[b], scale[b]);
      else *reinterpret_cast<u32x4*>(to[b]) = x[b];
    }
  }
}

// Lengths after the rows, where seq_len_out is seq_len itself and the rows'
// blocks still read it.
__global__ __launch_bounds__(kThreads) void append_lengths_kernel(const AppendArgs args) { write_lengths(args); }

}  // namespace
}  // namespace hrs

using namespace hrs;

extern "C" int kv_cache_append(const hrs_append_desc* d, const void* k, const void* v, void* k_cache, void* v_cache,
                               const int32_t* page_table, const int32_t* seq_len, const int32_t* accept_len,
                               const int32_t* path, const float* k_scale, const float* v_scale,
                               int32_t* seq_len_out, int32_t* status, void* stream) {
  if (d == nullptr) return HRS_EINVAL;
  if (d->n_layers < 1 || d->n_layers > 65535 || d->n_req < 1 || d->n_req > 65535 || d->n_pos < 1 ||
      d->n_pos > (path ? HRS_MAX_POS : HRS_MAX_CHUNKED_POS) || d->n_kvheads < 1 || d->n_kvheads > 65535 ||
      static_cast<int64_t>(d->n_req) * d->n_pos > (1 << 24) || !dtype_ok(d->dtype))
    return HRS_EINVAL;
  const int cc = check_cache(d->cache, d->dtype);
  if (cc != HRS_OK) return cc;
  if (d->d < 16 || d->d > 256 || d->d % 16 != 0) return HRS_EUNSUPPORTED;
  AppendArgs args;
  const int64_t dense = static_cast<int64_t>(d->n_kvheads) * d->d;
  if (!span_stride(d->k_stride, dense, &args.k_stride) || !span_stride(d->v_stride, dense, &args.v_stride))
    return HRS_EINVAL;
  if (!k || !v || !k_cache || !v_cache || !page_table || !seq_len || !accept_len) return HRS_EINVAL;
  if (d->cache.dtype != HRS_F8E4M3 && (k_scale || v_scale)) return HRS_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(page_table) ||
      !aligned16(seq_len) || !aligned16(accept_len) || !aligned16(path) || !aligned4(k_scale) ||
      !aligned4(v_scale) || !aligned16(seq_len_out) || !aligned16(status))
    return HRS_EALIGN;
  // Lengths in place or apart; a partial overlap would be read after it is
  // written.
  if (seq_len_out && seq_len_out != seq_len && seq_len_out < seq_len + d->n_req && seq_len < seq_len_out + d->n_req)
    return HRS_EINVAL;

  args.k = k; args.v = v; args.k_cache = k_cache; args.v_cache = v_cache; args.page_table = page_table;
  args.seq_len = seq_len; args.accept_len = accept_len; args.path = path; args.k_scale = k_scale;
  args.v_scale = v_scale; args.seq_len_out = seq_len_out; args.status = status;
  args.n_req = d->n_req; args.n_pos = d->n_pos; args.heads = d->n_kvheads; args.d = d->d;
  args.n_pages = d->cache.n_pages; args.table_len = d->cache.table_len;
  args.page_shift = __builtin_ctz(static_cast<unsigned>(d->cache.page_size));
  args.lens_here = seq_len_out != seq_len;
  const dim3 grid((d->n_pos + kRows - 1) / kRows, d->n_req, d->n_layers);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (d->dtype == HRS_F32)
    hipLaunchKernelGGL((append_kernel<4, false>), grid, dim3(kThreads), 0, s, args);
  else if (d->cache.dtype == HRS_BF16)
    hipLaunchKernelGGL((append_kernel<2, false>), grid, dim3(kThreads), 0, s, args);
  else
    hipLaunchKernelGGL((append_kernel<2, true>), grid, dim3(kThreads), 0, s, args);
  if (launch_error() != hipSuccess) return HRS_EDEVICE;
  if (!args.lens_here) {
    hipLaunchKernelGGL(append_lengths_kernel, dim3(1), dim3(kThreads), 0, s, args);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}
