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
// onto each other's slots would need an order). One wave copies one row of
// one layer's keys or values at a time, 16 bytes per lane.
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
  int32_t rows_per_block;
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

// Whether every accepted entry of the request's path names a span position
// (n <= 64 where there is a path); the answer is the wave's, each lane looks
// at one entry.
__device__ __forceinline__ bool path_ok(const AppendArgs& a, int r, int n) {
  if (a.path == nullptr) return true;
  const int lane = threadIdx.x & 63;
  const int p = a.path[static_cast<int64_t>(r) * a.n_pos + min(lane, n - 1)];
  return __all(p >= 0 && p < a.n_pos);
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

// One 16-byte piece of a span row to the cache row.
__device__ __forceinline__ void copy_row(const char* src, char* dst, int bytes, int lane, int lanes) {
  for (int i = lane * 16; i < bytes; i += lanes * 16)
    *reinterpret_cast<u32x4*>(dst + i) = *reinterpret_cast<const u32x4*>(src + i);
}

// bf16 row to e4m3: divided by the scale (rounded once), limited to the
// largest e4m3 number, NaN kept.
__device__ __forceinline__ float e4m3_range(float x, float scale) {
  const float y = x / scale;
  return y != y ? y : fminf(fmaxf(y, -448.0f), 448.0f);
}
__device__ __forceinline__ void quant_row(const char* src, char* dst, int d, float scale, int lane, int lanes) {
  for (int i = lane * 8; i < d; i += lanes * 8) {
    float x[8];
    load8<uint16_t>(reinterpret_cast<const uint16_t*>(src) + i, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = e4m3_range(x[j], scale);
    uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
    uint32_t hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
    *reinterpret_cast<u32x2*>(dst + i) = u32x2{lo, hi};
  }
}

// Grid: (blocks of rows, request, layer). ESZ: bytes of a span element; F8:
// the cache is e4m3. A row here is one position's keys or values of all heads
// of one layer; the block's items are (position, K or V, head).
template <int ESZ, bool F8>
__global__ __launch_bounds__(kThreads) void append_kernel(const AppendArgs args) {
  const int r = blockIdx.y;
  const int layer = blockIdx.z;
  if (args.lens_here && blockIdx.x == 0 && r == 0 && layer == 0) write_lengths(args);
  int len, n;
  if (!request_ok(args, r, &len, &n) || !path_ok(args, r, n)) return;
  const int i0 = blockIdx.x * args.rows_per_block;
  const int i1 = min(n, i0 + args.rows_per_block);
  if (i0 >= i1) return;
  const int d = args.d;
  constexpr int kPiece = F8 ? 8 : 16 / ESZ;      // elements per lane step
  const int lanes = min(64, (d + kPiece - 1) / kPiece);
  // Lanes per row: the power of two that holds it, so that a wave takes
  // several short rows at once.
  int lp = 1;
  while (lp < lanes) lp <<= 1;
  const int sub = threadIdx.x / lp, lane = threadIdx.x % lp;
  const int subs = kThreads / lp;
  const int items = (i1 - i0) * 2 * args.heads;
  const int64_t span_row0 = (static_cast<int64_t>(layer) * args.n_req + r) * args.n_pos;
  const int page_mask = (1 << args.page_shift) - 1;
  const int csz = F8 ? 1 : ESZ;
  for (int it = sub; it < items; it += subs) {
    const int h = it % args.heads;
    const int kv = (it / args.heads) & 1;
    const int i = i0 + it / (2 * args.heads);
    const int slot = len + i;
    const int page = args.page_table[static_cast<int64_t>(r) * args.table_len + (slot >> args.page_shift)];
    if (page < 0 || page >= args.n_pages) continue;
    const int pos = args.path ? args.path[static_cast<int64_t>(r) * args.n_pos + i] : i;
    const int64_t stride = kv ? args.v_stride : args.k_stride;
    const char* src = static_cast<const char*>(kv ? args.v : args.k) +
                      ((span_row0 + pos) * stride + static_cast<int64_t>(h) * d) * ESZ;
    const int64_t row = ((static_cast<int64_t>(layer) * args.n_pages + page) * args.heads + h) *
                            (page_mask + 1) + (slot & page_mask);
    char* dst = static_cast<char*>(kv ? args.v_cache : args.k_cache) + row * d * csz;
    if constexpr (F8) {
      const float* sc = kv ? args.v_scale : args.k_scale;
      quant_row(src, dst, d, sc ? sc[layer * args.heads + h] : 1.0f, lane, lp);
    } else {
      copy_row(src, dst, d * ESZ, lane, lp);
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
  args.rows_per_block = 16;
  args.lens_here = seq_len_out != seq_len;
  const dim3 grid((d->n_pos + args.rows_per_block - 1) / args.rows_per_block, d->n_req, d->n_layers);
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
