// attn_verify_span: attention of a verify span (chain or draft tree) over a
// paged cache and the span's own root paths.
//
//   out = sum_j w_j v_j,  w = softmax_j(scale q . k_j)
//
// openinfer PR #626 ("feat(qwen35): add opt-in DFlash speculative decoding"),
// file table: the paged causal-window attention of the verify forward;
// lucebox PR #533 ("feat: DFlash support for tensor-parallel Qwen3.6
// targets"), Verification: DDTree.
//
// One wave per query head and position, slots in groups of 64 with a running
// maximum and sum: the plain form of the softmax in one pass.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* k_cache;
  const void* v_cache;
  const int32_t* page_table;
  const int32_t* seq_len;
  const float* k_scale;
  const float* v_scale;
  void* out;
  int32_t* status;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  float scale;
  int32_t window;
  int32_t n_req;      // of the whole call
  int32_t n_pos;
  int32_t heads;
  int32_t kvheads;
  int32_t n_pages;
  int32_t page_shift;
  int32_t table_len;
  int32_t req0;
  int32_t tree;
  int8_t parent[kGeomBytes];
};

struct F8 { uint8_t b; };   // e4m3

template <typename T> __device__ __forceinline__ float elem(const T* p);
template <> __device__ __forceinline__ float elem<float>(const float* p) { return *p; }
template <> __device__ __forceinline__ float elem<uint16_t>(const uint16_t* p) { return bf16_one(*p); }
template <> __device__ __forceinline__ float elem<F8>(const F8* p) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<int>(p->b), 0);
}

template <typename T, typename C, int D>
__global__ __launch_bounds__(64) void attn_simple_kernel(const AttnArgs args) {
  const int lane = threadIdx.x;
  const int h = blockIdx.x, t = blockIdx.y, rl = blockIdx.z, r = args.req0 + rl;
  const int g = h / (args.heads / args.kvheads);
  if (h == 0 && t == 0 && r == 0 && lane == 0 && args.status) {
    int bad = 0;
    for (int i = 0; i < args.n_req; ++i) {
      const int n = args.seq_len[i];
      bad += n < 0 || n > (args.table_len << args.page_shift);
    }
    *args.status = bad;
  }
  const int len = args.seq_len[r];
  if (len < 0 || len > (args.table_len << args.page_shift)) return;
  // Root path and window inside the span.
  uint64_t path = 0;
  int depth = 0;
  for (int a = t; a >= 0; a = args.tree ? args.parent[rl * args.n_pos + a] : a - 1) ++depth;
  --depth;
  for (int a = t, i = 0; a >= 0 && (args.window == 0 || i < args.window);
       a = args.tree ? args.parent[rl * args.n_pos + a] : a - 1, ++i)
    path |= uint64_t{1} << a;
  const int first = args.window ? max(0, len + depth + 1 - args.window) : 0;

  const int64_t row = static_cast<int64_t>(r) * args.n_pos + t;
  __shared__ float qs[D];
  __shared__ float ps[64];
  const T* q = static_cast<const T*>(args.q) + row * args.q_stride + static_cast<int64_t>(h) * D;
  for (int i = lane; i < D; i += 64) qs[i] = elem<T>(q + i);
  __syncthreads();
  float o[D / 64] = {};
  float m = -__builtin_inff(), l = 0.0f;
  const float ks = args.k_scale ? args.k_scale[g] : 1.0f, vs = args.v_scale ? args.v_scale[g] : 1.0f;
  const int end = len + args.n_pos;
  for (int j0 = first & ~63; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    const bool ctx = j < len;
    bool on = ctx ? j >= first : j < end && ((path >> (j - len)) & 1);
    const C* kc = nullptr;
    const T* kt = nullptr;
    int64_t off = 0;
    if (on) {
      if (ctx) {
        const int page = args.page_table[static_cast<int64_t>(r) * args.table_len + (j >> args.page_shift)];
        on = page >= 0 && page < args.n_pages;
        off = (((static_cast<int64_t>(page) * args.kvheads + g) << args.page_shift) + (j & ((1 << args.page_shift) - 1))) * D;
        kc = static_cast<const C*>(args.k_cache) + off;
      } else {
        kt = static_cast<const T*>(args.k) + (static_cast<int64_t>(r) * args.n_pos + j - len) * args.k_stride +
             static_cast<int64_t>(g) * D;
      }
    }
    float s = -__builtin_inff();
    if (on) {
      float a = 0.0f;
      if (ctx)
        for (int i = 0; i < D; ++i) a = fmaf(qs[i], elem<C>(kc + i), a);
      else
        for (int i = 0; i < D; ++i) a = fmaf(qs[i], elem<T>(kt + i), a);
      s = a * args.scale * (ctx ? ks : 1.0f);
    }
    float mx = s;
    for (int x = 32; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor(mx, x));
    const float mn = fmaxf(m, mx);
    const float base = mn == -__builtin_inff() ? 0.0f : mn;
    const float keep = expf(m - base);
    const float p = on ? expf(s - base) : 0.0f;
    float sum = p;
    for (int x = 32; x >= 1; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * keep + sum;
    m = mn;
    for (int i = 0; i < D / 64; ++i) o[i] *= keep;
    ps[lane] = p;
    const uint64_t live = __ballot(on);
    __syncthreads();
    for (uint64_t b = live; b; b &= b - 1) {
      const int i = __builtin_ctzll(b);
      const int jj = j0 + i;
      const int64_t o2 = __shfl(off, i);
      for (int e = 0; e < D / 64; ++e) {
        float v;
        if (jj < len)
          v = elem<C>(static_cast<const C*>(args.v_cache) + o2 + e * 64 + lane) * vs;
        else
          v = elem<T>(static_cast<const T*>(args.v) +
                      (static_cast<int64_t>(r) * args.n_pos + jj - len) * args.v_stride +
                      static_cast<int64_t>(g) * D + e * 64 + lane);
        o[e] = fmaf(ps[i], v, o[e]);
      }
    }
    __syncthreads();
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  for (int e = 0; e < D / 64; ++e) {
    const float y = l == 0.0f ? 0.0f : o[e] * inv;
    const int64_t at = (row * args.heads + h) * D + e * 64 + lane;
    if constexpr (sizeof(T) == 2)
      static_cast<uint16_t*>(args.out)[at] = static_cast<uint16_t>(pack_bf16(y, 0.0f) & 0xFFFFu);
    else
      static_cast<float*>(args.out)[at] = y;
  }
}

}  // namespace
}  // namespace hrs

using namespace hrs;

static bool attn_sizes_ok(const hrs_attn_desc* d) {
  return d && d->n_req >= 1 && d->n_req <= 4096 && d->n_pos >= 1 && d->n_pos <= HRS_MAX_POS && d->n_heads >= 1 &&
         d->n_kvheads >= 1 && d->n_kvheads <= 1024 && d->n_heads % d->n_kvheads == 0 &&
         d->n_heads / d->n_kvheads <= 64;
}

extern "C" size_t attn_verify_span_workspace_bytes(const hrs_attn_desc* d) {
  if (!attn_sizes_ok(d) || (d->d != 64 && d->d != 128 && d->d != 256)) return 0;
  return 16;
}

extern "C" int attn_verify_span(const hrs_attn_desc* d, const void* q, const void* k, const void* v,
                                const void* k_cache, const void* v_cache, const int32_t* page_table,
                                const int32_t* seq_len, const float* k_scale, const float* v_scale, void* out,
                                int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (d == nullptr) return HRS_EINVAL;
  if (d->topo == HRS_TREE || d->topo == HRS_CHAIN) {
    const int geo = check_topology(d->topo, d->parent, d->n_req < 1 ? 0 : d->n_req, d->n_pos);
    if (geo != HRS_OK) return geo;
  } else {
    return HRS_EINVAL;
  }
  if (!attn_sizes_ok(d) || !dtype_ok(d->dtype) || d->window < 0) return HRS_EINVAL;
  const int cc = check_cache(d->cache, d->dtype);
  if (cc != HRS_OK) return cc;
  if (d->d != 64 && d->d != 128 && d->d != 256) return HRS_EUNSUPPORTED;
  AttnArgs args;
  const int64_t kv_dense = static_cast<int64_t>(d->n_kvheads) * d->d;
  if (!span_stride(d->q_stride, static_cast<int64_t>(d->n_heads) * d->d, &args.q_stride) ||
      !span_stride(d->k_stride, kv_dense, &args.k_stride) || !span_stride(d->v_stride, kv_dense, &args.v_stride))
    return HRS_EINVAL;
  if (!q || !k || !v || !k_cache || !v_cache || !page_table || !seq_len || !out) return HRS_EINVAL;
  if (d->cache.dtype != HRS_F8E4M3 && (k_scale || v_scale)) return HRS_EINVAL;
  if (!workspace || workspace_bytes < attn_verify_span_workspace_bytes(d)) return HRS_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(page_table) || !aligned16(seq_len) || !aligned4(k_scale) || !aligned4(v_scale) ||
      !aligned16(out) || !aligned16(status) || !aligned16(workspace))
    return HRS_EALIGN;

  args.q = q; args.k = k; args.v = v; args.k_cache = k_cache; args.v_cache = v_cache; args.page_table = page_table;
  args.seq_len = seq_len; args.k_scale = k_scale; args.v_scale = v_scale; args.out = out; args.status = status;
  args.scale = d->scale; args.window = d->window; args.n_req = d->n_req; args.n_pos = d->n_pos;
  args.heads = d->n_heads; args.kvheads = d->n_kvheads;
  args.n_pages = d->cache.n_pages; args.table_len = d->cache.table_len;
  args.page_shift = __builtin_ctz(static_cast<unsigned>(d->cache.page_size));
  args.tree = d->topo == HRS_TREE;
  const int per_launch = args.tree ? std::max(1, kGeomBytes / d->n_pos) : d->n_req;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  for (int r0 = 0; r0 < d->n_req; r0 += per_launch) {
    const int n = std::min(per_launch, d->n_req - r0);
    args.req0 = r0;
    if (args.tree)
      for (int i = 0; i < n * d->n_pos; ++i)
        args.parent[i] = static_cast<int8_t>(d->parent[static_cast<size_t>(r0) * d->n_pos + i]);
    const dim3 grid(d->n_heads, d->n_pos, n);
#define HRS_ATTN(T, C)                                                                                  \
  do {                                                                                                  \
    if (d->d == 64) hipLaunchKernelGGL((attn_simple_kernel<T, C, 64>), grid, dim3(64), 0, s, args);     \
    if (d->d == 128) hipLaunchKernelGGL((attn_simple_kernel<T, C, 128>), grid, dim3(64), 0, s, args);   \
    if (d->d == 256) hipLaunchKernelGGL((attn_simple_kernel<T, C, 256>), grid, dim3(64), 0, s, args);   \
  } while (0)
    if (d->dtype == HRS_F32)
      HRS_ATTN(float, float);
    else if (d->cache.dtype == HRS_BF16)
      HRS_ATTN(uint16_t, uint16_t);
    else
      HRS_ATTN(uint16_t, F8);
#undef HRS_ATTN
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}
