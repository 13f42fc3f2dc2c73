// attn_verify_span: attention of a verify span (chain or draft tree) over a
// paged cache and the span's own root paths. Host side, and the join of the
// parts that the kernel (attn_kernel.h) leaves where a block's run of tiles
// ends inside a (request, key/value head).
//
// openinfer PR #626 ("feat(qwen35): add opt-in DFlash speculative decoding"),
// file table: the paged causal-window attention of the verify forward;
// lucebox PR #533 ("feat: DFlash support for tensor-parallel Qwen3.6
// targets"), Verification: DDTree.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn.h"

namespace hrs {
namespace {

// Sum of a segment's parts: out = sum_b 2^(m_b - M) O_b / sum_b 2^(m_b - M)
// l_b. A wave takes two column groups (four columns of a lane each) of 16
// rows of a segment (request, head, row block), in the lanes' order of the
// kernel that wrote them. NS waves take every NS-th part and are added in LDS
// (in order, so results repeat): with few rows and many parts, as for one
// long request, more loads are on their way (4 heads x 102 rows x 64 parts of
// 256: 35.7 us with all parts in one thread group per row).
template <bool F32, int D, int NS>
__global__ __launch_bounds__(NS > 1 ? 64 * NS : 256) void attn_join_kernel(const int32_t* plan, const f32x4* part,
                                                                          const float2* part_ml, int n_here, int heads,
                                                                          int log_blocks, int rows_per_block,
                                                                          const AttnBase args) {
  constexpr int DT = D / 16;
  const int i = blockIdx.x / heads;
  const int seg = blockIdx.x - i * heads;
  const int total = plan[n_here];
  const int first = plan[i], end = plan[i + 1];
  const int h = seg / args.row_blocks, rb = seg - h * args.row_blocks;
  const int r = args.req0 + i;
  if (end == first) return;
  const int units = (end - first) / heads;
  const int s0 = first + seg * units, s1 = s0 + units;
  // Block of a unit: the last whose run starts at or before it.
  auto block_of = [&](int u) {
    if (total <= (1 << log_blocks)) return u;
    return static_cast<int>((((static_cast<int64_t>(u) + 1) << log_blocks) - 1) / total);
  };
  const int b0 = block_of(s0), b1 = block_of(s1 - 1);
  if (b0 == b1) return;                       // one block had all of it and wrote the result
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int task = NS > 1 ? blockIdx.y : blockIdx.y * 4 + wave;
  const int tiles = (min(rows_per_block, args.rows - rb * rows_per_block) + 15) / 16;
  const int tile = task / (DT / 2), dp = task % (DT / 2);
  if (tile >= tiles) return;
  const int n16 = lane & 15, g = lane >> 4;
  const int row = tile * 16 + n16;
  const int ns = NS > 1 ? wave : 0;
  float M = -__builtin_inff(), ls = 0.0f;
  f32x4 sum[2] = {};
  constexpr int kAtOnce = NS > 1 ? 8 : 4;     // parts whose loads go out together
  for (int b = b0 + ns; b <= b1; b += NS * kAtOnce) {
    float2 w[kAtOnce];
    f32x4 x[kAtOnce][2];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int bj = min(b + j * NS, b1);
      // The segment's first block left its part as its last, the others theirs
      // as their first.
      const int64_t slot = 2 * bj + (bj == b0 ? 1 : 0);
      w[j] = part_ml[slot * rows_per_block + row];
      const f32x4* at = part + (slot * (rows_per_block / 16) + tile) * (DT * 64) + lane;
      x[j][0] = at[(2 * dp) * 64];
      x[j][1] = at[(2 * dp + 1) * 64];
    }
    float top = M;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) top = fmaxf(top, w[j].x);
    const float keep = M == top ? 1.0f : __builtin_amdgcn_exp2f(M - top);
    M = top;
    ls *= keep;
    sum[0] *= keep;
    sum[1] *= keep;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      // Parts past the last, and parts that no slot counted in, weigh nothing.
      if (b + j * NS > b1 || (w[j].x == -__builtin_inff() && w[j].y == 0.0f)) continue;
      const float f = w[j].x == M ? 1.0f : __builtin_amdgcn_exp2f(w[j].x - M);
      ls += w[j].y * f;
      sum[0] += x[j][0] * f;
      sum[1] += x[j][1] * f;
    }
  }
  if constexpr (NS > 1) {
    __shared__ f32x4 sums[NS][2][64];
    __shared__ float2 ml[NS][64];
    sums[wave][0][lane] = sum[0];
    sums[wave][1][lane] = sum[1];
    ml[wave][lane] = float2{M, ls};
    __syncthreads();
    if (wave != 0) return;
    float top = M;
#pragma unroll
    for (int j = 1; j < NS; ++j) top = fmaxf(top, ml[j][lane].x);
    const float f0 = M == top ? 1.0f : __builtin_amdgcn_exp2f(M - top);
    ls *= f0;
    sum[0] *= f0;
    sum[1] *= f0;
#pragma unroll
    for (int j = 1; j < NS; ++j) {
      const float2 w = ml[j][lane];
      if (w.x == -__builtin_inff() && w.y == 0.0f) continue;
      const float f = w.x == top ? 1.0f : __builtin_amdgcn_exp2f(w.x - top);
      ls += w.y * f;
      sum[0] += sums[j][0][lane] * f;
      sum[1] += sums[j][1][lane] * f;
    }
  }
  const int at_row = rb * rows_per_block + row;
  if (at_row >= args.rows) return;
  const int t = at_row / args.group, hq = h * args.group + at_row - t * args.group;
  const float inv = 1.0f / ls;      // scores of -inf alone: 0 * inf, as the formula's 0 / 0
  const int64_t at = ((static_cast<int64_t>(r) * args.n_pos + t) * (args.kvheads * args.group) + hq) * D;
#pragma unroll
  for (int e = 0; e < 2; ++e) sum[e] *= inv;
  if constexpr (F32) {
    float* const out = static_cast<float*>(args.out) + at + 32 * dp + 4 * g;
    *reinterpret_cast<f32x4*>(out) = sum[0];
    *reinterpret_cast<f32x4*>(out + 16) = sum[1];
  } else {
    // Group dt = EPL half + x holds columns 16 EPL half + EPL (4 g + i) + x.
    constexpr int EPL = D >= 128 ? 8 : 4;
    const int half = 2 * dp / EPL, x = 2 * dp % EPL;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(args.out) + at + 16 * EPL * half + EPL * (4 * g + c) + x) =
          pack_bf16(sum[0][c], sum[1][c]);
  }
}

template <bool F32, int D> void launch_join_d(const AttnBase& args, const AttnLens& l, const AttnShape& sh, hipStream_t s) {
  const int segs = l.n * l.heads;
  const f32x4* const part = reinterpret_cast<const f32x4*>(args.part);
  const int tasks = (std::min(sh.rows, args.rows) + 15) / 16 * (D / 32);
  if (static_cast<int64_t>(segs) * tasks <= 1024)
    hipLaunchKernelGGL((attn_join_kernel<F32, D, 8>), dim3(segs, tasks), dim3(512), 0, s, args.plan, part, args.part_ml, l.n,
                       l.heads, l.log_blocks, sh.rows, args);
  else
    hipLaunchKernelGGL((attn_join_kernel<F32, D, 1>), dim3(segs, (tasks + 3) / 4), dim3(256), 0, s, args.plan,
                       part, args.part_ml, l.n, l.heads, l.log_blocks, sh.rows, args);
}

template <bool F32> void launch_join(const AttnBase& args, const AttnLens& l, int d, const AttnShape& sh, hipStream_t s) {
  if (d == 64) launch_join_d<F32, 64>(args, l, sh, s);
  if (d == 128) launch_join_d<F32, 128>(args, l, sh, s);
  if (d == 256) launch_join_d<F32, 256>(args, l, sh, s);
}

bool sizes_ok(const hrs_attn_desc* d) {
  return d && d->n_req >= 1 && d->n_req <= 4096 && d->n_pos >= 1 && d->n_pos <= HRS_MAX_POS && d->n_heads >= 1 &&
         d->n_kvheads >= 1 && d->n_kvheads <= 1024 && d->n_heads % d->n_kvheads == 0 &&
         d->n_heads / d->n_kvheads <= 64;
}

// The class of AttnCfg; its comment has both sides of each border.
int rows_class(int kind, int d, int rows) {
  if (kind == kF8 && d <= 128 && rows > 64 && rows <= 96) return 4;
  return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3;
}

AttnShape shape_of(const hrs_attn_desc* d, int kind) {
  const int cls = rows_class(kind, d->d, d->n_pos * (d->n_heads / d->n_kvheads));
  return kind == kF32 ? attn_shape<kF32>(d->d, cls) : kind == kB16 ? attn_shape<kB16>(d->d, cls)
                                                                   : attn_shape<kF8>(d->d, cls);
}

constexpr size_t kPlanBytes = ((kAttnReqs + 1) * sizeof(int32_t) + 255) / 256 * 256;

}  // namespace
}  // namespace hrs

using namespace hrs;

extern "C" size_t attn_verify_span_workspace_bytes(const hrs_attn_desc* d) {
  if (!sizes_ok(d) || (d->d != 64 && d->d != 128 && d->d != 256)) return 0;
  // Enough for every type: the blocks depend on the sizes alone, and a class
  // of one type only has fewer rows.
  const AttnShape sh = shape_of(d, kB16);
  const size_t rows = sh.rows;
  return kPlanBytes + 2 * static_cast<size_t>(sh.blocks) * rows * (static_cast<size_t>(d->d) * sizeof(float) + sizeof(float2));
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
  if (!sizes_ok(d) || !dtype_ok(d->dtype) || d->window < 0) return HRS_EINVAL;
  const int cc = check_cache(d->cache, d->dtype);
  if (cc != HRS_OK) return cc;
  if (d->d != 64 && d->d != 128 && d->d != 256) return HRS_EUNSUPPORTED;
  AttnTree args;
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

  const int kind = d->dtype == HRS_F32 ? kF32 : d->cache.dtype == HRS_BF16 ? kB16 : kF8;
  const AttnShape sh = shape_of(d, kind);
  args.q = q; args.k = k; args.v = v;
  args.k_cache = static_cast<const char*>(k_cache); args.v_cache = static_cast<const char*>(v_cache);
  args.page_table = page_table; args.seq_len = seq_len; args.k_scale = k_scale; args.v_scale = v_scale;
  args.out = out; args.status = status;
  char* const ws = static_cast<char*>(workspace);
  args.plan = reinterpret_cast<int32_t*>(ws);
  args.part = reinterpret_cast<float*>(ws + kPlanBytes);
  args.part_ml = reinterpret_cast<float2*>(ws + kPlanBytes + sizeof(float) * 2 * sh.blocks * sh.rows * d->d);
  args.scale = d->scale; args.window = d->window; args.n_req = d->n_req; args.n_pos = d->n_pos;
  args.kvheads = d->n_kvheads; args.group = d->n_heads / d->n_kvheads;
  args.rows = args.n_pos * args.group;
  args.row_blocks = (args.rows + sh.rows - 1) / sh.rows;
  args.n_pages = d->cache.n_pages; args.table_len = d->cache.table_len;
  args.page_shift = __builtin_ctz(static_cast<unsigned>(d->cache.page_size));
  args.tree = d->topo == HRS_TREE;
  // Units are counted in 32 bits: fewer requests a launch for tables of very
  // many slots.
  const int64_t slots = (static_cast<int64_t>(args.table_len) << args.page_shift) + HRS_MAX_POS;
  const int64_t most = static_cast<int64_t>(args.kvheads) * args.row_blocks * (slots / sh.ts + 4 + kExtraUnits);
  // Rows of the cache are counted by groups of 16, in 32 bits.
  const int64_t groups = static_cast<int64_t>(args.n_pages) * args.kvheads * (d->cache.page_size / 16);
  if (most > INT32_MAX || groups > UINT32_MAX) return HRS_EINVAL;
  const int per_launch =
      static_cast<int>(std::min<int64_t>(args.tree ? std::min(kAttnReqs, std::max(1, kGeomBytes / d->n_pos)) : kAttnReqs,
                                         INT32_MAX / most));
  const int cls = rows_class(kind, d->d, args.rows);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  for (int r0 = 0; r0 < d->n_req; r0 += per_launch) {
    args.req0 = r0;
    AttnLens lens{seq_len + r0, std::min(per_launch, d->n_req - r0), args.kvheads * args.row_blocks,
                  args.table_len << args.page_shift, d->window, d->n_pos, 0};
    if (args.tree)
      for (int i = 0; i < lens.n * d->n_pos; ++i)
        args.parent[i] = static_cast<int8_t>(d->parent[static_cast<size_t>(r0) * d->n_pos + i]);
    // No more blocks than the longest contexts the table could hold have
    // tiles, a power of two.
    while ((1 << lens.log_blocks) < sh.blocks && (1 << lens.log_blocks) < lens.n * most) ++lens.log_blocks;
    if (kind == kF32) attn_launch<kF32>(args, lens, d->d, cls, s);
    else if (kind == kB16) attn_launch<kB16>(args, lens, d->d, cls, s);
    else attn_launch<kF8>(args, lens, d->d, cls, s);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
    if (kind == kF32) launch_join<true>(args, lens, d->d, sh, s);
    else launch_join<false>(args, lens, d->d, sh, s);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}
