// attn_verify_shared: attention of the verify spans of requests that share a
// prefix. Host side, and the join of what the two launches leave.
//
// openinfer PR #626 ("feat(qwen35): add opt-in DFlash speculative decoding"),
// file table: the paged causal-window attention of the verify forward;
// lucebox PR #533 ("feat: DFlash support for tensor-parallel Qwen3.6
// targets"), Verification: DDTree.
//
//   out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p
//
// over the parts p of a row: those of the prefix, which one launch computes for
// the rows of all requests as if they were one request's positions, and those
// of the request's own slots and span, as attn_verify_span computes them with
// the shared slots left out. Parts are never whole results, so each segment
// (head, block of rows, and request) has at least one from each block that
// worked on it.
//
// 16 single positions behind 4,096 slots (24/4 heads of 256): prefix 13.3 us, own
// slots 14.8, join 15.0: latency, and 25 MB of the prefix's parts (256 runs of two
// tiles, each of which reads 64 KB and leaves 98), written and read beside its 17
// MB; 16 chains of 17 behind 26,758: 216, 37 and
// 21 (60 MB of parts, 2.9 TB/s); 32 trees of 23 behind 8,191 e4m3 slots (32/8
// heads of 128): 131, 46 and 21.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attn.h"

namespace hrs {
namespace {

// Parts of a launch: how its list of units was cut. runs > 0: attn_prefix.h's
// launch, plan[0] of them for every (head, block of rows).
struct Cut {
  const f32x4* part;
  const float2* ml;
  const int32_t* plan;   // units before every request, [n + 1]; prefix: [2]
  int32_t runs;
  int32_t n;             // requests (prefix: 1)
  int32_t heads;         // segments of a request
  int32_t row_blocks;
  int32_t log_blocks;
  int32_t rows;          // of a block
};

// The parts of row `row` of a request's segments for head h.
struct Parts {
  int b0, count;         // blocks that worked on it
  int64_t slot0;         // first part
  int step;              // from one part to the next
  int tile, n16;         // row's place in a part
  __device__ __forceinline__ Parts(const Cut& c, int i, int h, int row) {
    tile = row % c.rows / 16;
    n16 = row % 16;
    if (c.runs > 0) {
      b0 = 0;
      count = c.plan[0];
      slot0 = static_cast<int64_t>(h) * c.runs * c.row_blocks + row / c.rows;
      step = c.row_blocks;
      return;
    }
    const int first = c.plan[i], units = (c.plan[i + 1] - first) / c.heads, total = c.plan[c.n];
    const int seg = h * c.row_blocks + row / c.rows;
    const int s0 = first + seg * units, s1 = s0 + units;
    auto block_of = [&](int u) {
      if (total <= (1 << c.log_blocks)) return u;
      return static_cast<int>((((static_cast<int64_t>(u) + 1) << c.log_blocks) - 1) / total);
    };
    b0 = units > 0 ? block_of(s0) : 0;
    count = units > 0 ? block_of(s1 - 1) - b0 + 1 : 0;
    slot0 = static_cast<int64_t>(i) * c.heads + seg + b0;
    step = 1;
  }
};

// Grid: (request, head, 16 rows), pairs of column groups. A wave takes two
// column groups of 16 rows; NS waves take every NS-th part and are added in
// LDS, in order.
template <bool F32, int D, int NS>
__global__ __launch_bounds__(NS > 1 ? 64 * NS : 256) void shared_join_kernel(const Cut own, const Cut pre, int tiles,
                                                                            const AttnBase args) {
  constexpr int DT = D / 16;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int n16 = lane & 15, g = lane >> 4;
  const int i = blockIdx.x / (args.kvheads * tiles);
  const int ht = blockIdx.x - i * (args.kvheads * tiles);
  const int h = ht / tiles, tile = ht - h * tiles;
  const int dp = NS > 1 ? blockIdx.y : blockIdx.y * 4 + wave;
  if (dp >= DT / 2) return;
  const int row = tile * 16 + n16;       // of the request
  const bool on = row < args.rows;
  const int at = on ? row : tile * 16;
  const Parts po(own, i, h, at), pp(pre, 0, h, i * args.rows + at);
  if (po.count == 0) return;             // refused (the same for all rows)
  const int ns = NS > 1 ? wave : 0;
  float M = -__builtin_inff(), ls = 0.0f;
  f32x4 sum[2] = {};
  constexpr int kAtOnce = NS > 1 ? 8 : 4;
  // The prefix's parts and then the request's own, as one list (one after the
  // other the small float32 case took 7.8 instead of 6.2 us, 16 chains 22.2
  // instead of 21.2, 16 single positions of 256 13.8 instead of 15.0). A tile's
  // rows may lie in two of the prefix's segments: lanes differ in their number
  // of parts.
  const int count = pp.count + po.count;
  int most = count;
#pragma unroll
  for (int d = 32; d; d >>= 1) most = max(most, __shfl_xor(most, d));
  for (int b = ns; b < most; b += NS * kAtOnce) {
    float2 w[kAtOnce];
    f32x4 x[kAtOnce][2];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int k = min(b + j * NS, count - 1);
      const bool shared = k < pp.count;
      const int64_t slot = shared ? pp.slot0 + static_cast<int64_t>(k) * pp.step : po.slot0 + (k - pp.count);
      const int rows = shared ? pre.rows : own.rows;
      const int t = shared ? pp.tile : po.tile, n = shared ? pp.n16 : po.n16;
      w[j] = (shared ? pre.ml : own.ml)[slot * rows + t * 16 + n];
      const f32x4* from = (shared ? pre.part : own.part) + (slot * (rows / 16) + t) * (DT * 64) + g * 16 + n;
      x[j][0] = from[(2 * dp) * 64];
      x[j][1] = from[(2 * dp + 1) * 64];
    }
    float top = M;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (b + j * NS < count) top = fmaxf(top, w[j].x);
    const float keep = M == top ? 1.0f : __builtin_amdgcn_exp2f(M - top);
    M = top;
    ls *= keep;
    sum[0] *= keep;
    sum[1] *= keep;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      // Parts that no slot counted in weigh nothing.
      if (b + j * NS >= count || (w[j].x == -__builtin_inff() && w[j].y == 0.0f)) continue;
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
  if (!on) return;
  const int t = row / args.group, hq = h * args.group + row - t * args.group;
  const float inv = 1.0f / ls;      // scores of -inf alone: 0 * inf, as the formula's 0 / 0
  const int64_t to = ((static_cast<int64_t>(args.req0 + i) * args.n_pos + t) * (args.kvheads * args.group) + hq) * D;
#pragma unroll
  for (int e = 0; e < 2; ++e) sum[e] *= inv;
  if constexpr (F32) {
    float* const out = static_cast<float*>(args.out) + to + 32 * dp + 4 * g;
    *reinterpret_cast<f32x4*>(out) = sum[0];
    *reinterpret_cast<f32x4*>(out + 16) = sum[1];
  } else {
    // Group dt = EPL half + x holds columns 16 EPL half + EPL (4 g + i) + x.
    constexpr int EPL = D >= 128 ? 8 : 4;
    const int half = 2 * dp / EPL, x = 2 * dp % EPL;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(args.out) + to + 16 * EPL * half + EPL * (4 * g + c) + x) =
          pack_bf16(sum[0][c], sum[1][c]);
  }
}

template <bool F32, int D> void launch_join(const Cut& own, const Cut& pre, const AttnBase& args, hipStream_t s) {
  const int tiles = (args.rows + 15) / 16;
  const int segs = own.n * args.kvheads * tiles;
  if (static_cast<int64_t>(segs) * (D / 32) <= 2048)
    hipLaunchKernelGGL((shared_join_kernel<F32, D, 8>), dim3(segs, D / 32), dim3(512), 0, s, own, pre, tiles, args);
  else
    hipLaunchKernelGGL((shared_join_kernel<F32, D, 1>), dim3(segs, (D / 32 + 3) / 4), dim3(256), 0, s, own, pre, tiles, args);
}
template <bool F32> void launch_join(const Cut& own, const Cut& pre, const AttnBase& args, int d, hipStream_t s) {
  if (d == 64) launch_join<F32, 64>(own, pre, args, s);
  else if (d == 128) launch_join<F32, 128>(own, pre, args, s);
  else launch_join<F32, 256>(own, pre, args, s);
}

// More rows of a key head than this go to attn_prefix.h's launch. Whole calls
// there and here, 4 key heads of 256 in bf16: 192 rows over 2,048 slots 46 and
// 37 us, over 16,384 slots 58 and 61; 288 rows 48 and 44, 65 and 81; 768 rows 61
// and 60, 99 and 139. (8 heads of 128, e4m3, 288 rows: 43 and 40, 65 and 68; 768
// rows 64 and 62, 106 and 120.) So behind short prefixes the kernels for
// smaller batches take up to 8% less at 288 and 768 rows too, and behind long ones
// up to 40% more. The rule goes by rows alone: the host knows the prefix's table,
// not its length.
constexpr int64_t kWideRows = 256;

// How a launch's parts are laid out in the workspace.
struct PartSizes {
  AttnShape shape;
  int row_blocks;
  int64_t segs, parts;
  size_t ml_bytes, bytes;
};
PartSizes part_sizes(int kind, int d, int64_t n, int64_t kvheads, int64_t rows) {
  PartSizes p;
  p.shape = shape_of(kind, d, rows);
  p.row_blocks = static_cast<int>((rows + p.shape.rows - 1) / p.shape.rows);
  p.segs = n * kvheads * p.row_blocks;
  p.parts = p.segs + p.shape.blocks;
  p.ml_bytes = (p.parts * p.shape.rows * sizeof(float2) + 255) / 256 * 256;
  p.bytes = p.ml_bytes + static_cast<size_t>(p.parts) * p.shape.rows * d * sizeof(float);
  return p;
}

// The prefix launch for large batches: rows of a block, and the runs that a
// head's slots are cut into, as many as let all blocks run at once or, where
// there are more (head, block of rows) than that, leave the last round of
// blocks nearly full.
bool prefix_wide(int kind, int64_t rows) { return kind != kF32 && rows > kWideRows; }
int prefix_rows(int d) { return d == 256 ? PrefixCfg<kB16, 256>::ROWS : d == 128 ? PrefixCfg<kB16, 128>::ROWS : PrefixCfg<kB16, 64>::ROWS; }
int prefix_runs(int64_t segs, int d) {
  const int64_t room = kAttnCus * static_cast<int64_t>(d == 256 ? PrefixCfg<kB16, 256>::PER_CU : PrefixCfg<kB16, 128>::PER_CU);
  const int64_t most = std::max<int64_t>(1, room / segs);
  if (segs * most * 10 >= room * 8 || segs > 8 * room) return static_cast<int>(most);
  int best = static_cast<int>(most);
  double least = 1.0 / best;
  for (int r = best + 1; r <= 4 * most; ++r) {
    const double t = static_cast<double>((segs * r + room - 1) / room) / r * (1.0 + 0.02 * (r - most) / most);
    if (t < least) {
      least = t;
      best = r;
    }
  }
  return best;
}
PartSizes wide_sizes(int d, int64_t kvheads, int64_t rows, int* runs) {
  PartSizes p;
  p.shape = {prefix_rows(d), 0, 0};
  p.row_blocks = static_cast<int>((rows + p.shape.rows - 1) / p.shape.rows);
  *runs = prefix_runs(kvheads * p.row_blocks, d);
  p.segs = kvheads * p.row_blocks;
  p.parts = p.segs * *runs;
  p.ml_bytes = (p.parts * p.shape.rows * sizeof(float2) + 255) / 256 * 256;
  p.bytes = p.ml_bytes + static_cast<size_t>(p.parts) * p.shape.rows * d * sizeof(float);
  return p;
}

constexpr size_t kPlanBytes = ((kAttnReqs + 1) * sizeof(int32_t) + 255) / 256 * 256;

// Requests of a launch: as many trees as its arguments hold.
int reqs_per_launch(const hrs_attn_desc* d) {
  return d->topo == HRS_TREE ? std::min(kAttnReqs, std::max(1, kGeomBytes / d->n_pos)) : kAttnReqs;
}

}  // namespace
}  // namespace hrs

using namespace hrs;

extern "C" size_t attn_verify_shared_workspace_bytes(const hrs_attn_desc* d) {
  if (!sizes_ok(d) || (d->d != 64 && d->d != 128 && d->d != 256)) return 0;
  // Enough for every type and topology.
  const int n = std::min(d->n_req, kAttnReqs);
  const int64_t rows = static_cast<int64_t>(d->n_pos) * (d->n_heads / d->n_kvheads);
  size_t most = 0;
  for (const int kind : {kF32, kB16, kF8}) {
    const size_t own = part_sizes(kind, d->d, n, d->n_kvheads, rows).bytes;
    most = std::max(most, own + part_sizes(kind, d->d, 1, d->n_kvheads, n * rows).bytes);
    int runs;
    // (Smaller batches may be cut into more runs.)
    int64_t last = 0;
    for (int m = n; prefix_wide(kind, m * rows); --m) {
      const int64_t blocks = (m * rows + prefix_rows(d->d) - 1) / prefix_rows(d->d);
      if (blocks != last) most = std::max(most, own + wide_sizes(d->d, d->n_kvheads, m * rows, &runs).bytes);
      last = blocks;
    }
  }
  return 2 * kPlanBytes + most;
}

extern "C" int attn_verify_shared(const hrs_attn_desc* d, int32_t prefix_pages, const void* q, const void* k, const void* v,
                                  const void* k_cache, const void* v_cache, const int32_t* prefix_table,
                                  const int32_t* prefix_len, const int32_t* page_table, const int32_t* seq_len,
                                  const float* k_scale, const float* v_scale, void* out, int32_t* status, void* workspace,
                                  size_t workspace_bytes, void* stream) {
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
  if (prefix_pages < 1 || static_cast<int64_t>(prefix_pages) * d->cache.page_size > INT32_MAX - HRS_MAX_CHUNKED_POS)
    return HRS_EINVAL;
  if (d->d != 64 && d->d != 128 && d->d != 256) return HRS_EUNSUPPORTED;
  AttnSharedTree args;
  const int64_t kv_dense = static_cast<int64_t>(d->n_kvheads) * d->d;
  if (!span_stride(d->q_stride, static_cast<int64_t>(d->n_heads) * d->d, &args.q_stride) ||
      !span_stride(d->k_stride, kv_dense, &args.k_stride) || !span_stride(d->v_stride, kv_dense, &args.v_stride))
    return HRS_EINVAL;
  if (!q || !k || !v || !k_cache || !v_cache || !prefix_table || !prefix_len || !page_table || !seq_len || !out)
    return HRS_EINVAL;
  if (d->cache.dtype != HRS_F8E4M3 && (k_scale || v_scale)) return HRS_EINVAL;
  if (!workspace || workspace_bytes < attn_verify_shared_workspace_bytes(d)) return HRS_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(prefix_table) || !aligned16(prefix_len) || !aligned16(page_table) || !aligned16(seq_len) ||
      !aligned4(k_scale) || !aligned4(v_scale) || !aligned16(out) || !aligned16(status) || !aligned16(workspace))
    return HRS_EALIGN;

  const int kind = d->dtype == HRS_F32 ? kF32 : d->cache.dtype == HRS_BF16 ? kB16 : kF8;
  args.k = k; args.v = v;
  args.k_cache = static_cast<const char*>(k_cache); args.v_cache = static_cast<const char*>(v_cache);
  args.page_table = page_table; args.seq_len = seq_len; args.k_scale = k_scale; args.v_scale = v_scale;
  args.out = out; args.status = status;
  args.prefix_table = prefix_table; args.prefix_len = prefix_len; args.prefix_pages = prefix_pages; args.pad = 0;
  args.scale = d->scale; args.window = d->window; args.n_req = d->n_req;
  args.kvheads = d->n_kvheads; args.group = d->n_heads / d->n_kvheads;
  args.n_pages = d->cache.n_pages; args.table_len = d->cache.table_len;
  args.page_shift = __builtin_ctz(static_cast<unsigned>(d->cache.page_size));
  args.tree = d->topo == HRS_TREE;
  const int64_t rows = static_cast<int64_t>(d->n_pos) * args.group;
  // Units are counted in 32 bits: fewer requests a launch where there could be
  // very many.
  const int64_t own_slots = (static_cast<int64_t>(std::max(args.table_len, prefix_pages)) << args.page_shift) + HRS_MAX_POS;
  const PartSizes one = part_sizes(kind, d->d, 1, args.kvheads, rows);
  const int64_t own_most = args.kvheads * static_cast<int64_t>(one.row_blocks) * (own_slots / one.shape.ts + 6 + kExtraUnits);
  const int64_t groups = static_cast<int64_t>(args.n_pages) * args.kvheads * (d->cache.page_size / 16);
  if (own_most > INT32_MAX || groups > UINT32_MAX) return HRS_EINVAL;
  const int per_launch = static_cast<int>(std::min<int64_t>(reqs_per_launch(d), INT32_MAX / own_most));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  char* const ws = static_cast<char*>(workspace);
  (void)hipGetLastError();
  for (int r0 = 0; r0 < d->n_req; r0 += per_launch) {
    const int n = std::min(per_launch, d->n_req - r0);
    const PartSizes po = part_sizes(kind, d->d, n, args.kvheads, rows);
    int runs = 0;
    const PartSizes pp = prefix_wide(kind, n * rows) ? wide_sizes(d->d, args.kvheads, n * rows, &runs)
                                                     : part_sizes(kind, d->d, 1, args.kvheads, n * rows);
    char* const own_at = ws + 2 * kPlanBytes;
    char* const pre_at = own_at + po.bytes;
    auto blocks_of = [](const AttnShape& sh, int64_t units) {
      int log = 0;
      while ((1 << log) < sh.blocks && (1 << log) < units) ++log;
      return log;
    };
    AttnLens lens{seq_len + r0, n, args.kvheads * pp.row_blocks, args.table_len << args.page_shift, d->window, d->n_pos, 0};
    const int64_t pre_slots = static_cast<int64_t>(prefix_pages) << args.page_shift;
    if (runs == 0) {
      const int64_t pre_units = static_cast<int64_t>(lens.heads) * (pre_slots / pp.shape.ts + kExtraUnits);
      if (pre_units > INT32_MAX) return HRS_EINVAL;
      lens.log_blocks = blocks_of(pp.shape, pre_units);
    }
    // The prefix: the rows of all requests as one's.
    AttnShared pre = args;
    pre.q = static_cast<const char*>(q) + static_cast<int64_t>(r0) * d->n_pos * args.q_stride * (d->dtype == HRS_F32 ? 4 : 2);
    pre.req0 = 0;
    pre.n_pos = n * d->n_pos;
    pre.rows = static_cast<int>(n * rows);
    pre.row_blocks = pp.row_blocks;
    pre.plan = reinterpret_cast<int32_t*>(ws + kPlanBytes);
    pre.part_ml = reinterpret_cast<float2*>(pre_at);
    pre.part = reinterpret_cast<float*>(pre_at + pp.ml_bytes);
    const Cut pre_cut{reinterpret_cast<const f32x4*>(pre.part), pre.part_ml, pre.plan, runs, 1, lens.heads,
                      pp.row_blocks, lens.log_blocks, pp.shape.rows};
    const int pre_cls = rows_class(kind, d->d, n * rows);
    if (runs > 0 && kind == kB16) attn_prefix_wide<kB16>(pre, lens, runs, d->d, s);
    else if (runs > 0) attn_prefix_wide<kF8>(pre, lens, runs, d->d, s);
    else if (kind == kF32) attn_prefix_launch<kF32>(pre, lens, d->d, pre_cls, s);
    else if (kind == kB16) attn_prefix_launch<kB16>(pre, lens, d->d, pre_cls, s);
    else attn_prefix_launch<kF8>(pre, lens, d->d, pre_cls, s);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
    // What is left, for each request.
    args.q = q;
    args.req0 = r0;
    args.n_pos = d->n_pos;
    args.rows = static_cast<int>(rows);
    args.row_blocks = po.row_blocks;
    args.plan = reinterpret_cast<int32_t*>(ws);
    args.part_ml = reinterpret_cast<float2*>(own_at);
    args.part = reinterpret_cast<float*>(own_at + po.ml_bytes);
    lens.heads = args.kvheads * po.row_blocks;
    lens.log_blocks = blocks_of(po.shape, n * own_most);
    const Cut own_cut{reinterpret_cast<const f32x4*>(args.part), args.part_ml, args.plan, 0, n, lens.heads, po.row_blocks,
                      lens.log_blocks, po.shape.rows};
    if (args.tree)
      for (int i = 0; i < n * d->n_pos; ++i)
        args.parent[i] = static_cast<int8_t>(d->parent[static_cast<size_t>(r0) * d->n_pos + i]);
    const int own_cls = rows_class(kind, d->d, rows);
    if (kind == kF32) attn_own_launch<kF32>(args, lens, d->d, own_cls, s);
    else if (kind == kB16) attn_own_launch<kB16>(args, lens, d->d, own_cls, s);
    else attn_own_launch<kF8>(args, lens, d->d, own_cls, s);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
    if (kind == kF32) launch_join<true>(own_cut, pre_cut, args, d->d, s);
    else launch_join<false>(own_cut, pre_cut, args, d->d, s);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}
