// qk_norm_rope: RMS norm over every query and key head and the rotation of
// its first `rot` elements by position, in one pass over q and k.
//
//   n = x / sqrt(mean(x^2) + eps) * (offset + w)
//   (n[a], n[b]) -> (n[a] cos - n[b] sin, n[b] cos + n[a] sin)
//
// openinfer PR #626 ("feat(qwen35): add opt-in DFlash speculative decoding"),
// file table: batched query/key norm and rotation ahead of the attention.
//
// MI355X design: a copy with a little arithmetic, bound by memory for long
// spans (4096 positions of 28 heads of 256: 21.7 us, 5.4 TB/s) and by launch
// latency for one token (a 3.5 us kernel). A head is held by a group of 8, 16
// or 32 lanes, eight elements each (one 16-byte load of bf16), four heads of a
// group on their way at once; the sum of squares is a butterfly inside the
// group and the partner half of a rotated pair comes from another lane of it,
// so a head is read and written once and never leaves registers. The angles
// depend on the position alone: a block forms them once per position (the
// product with the frequency and its reduction to a turn in 64 bits: at
// position 262,144 a float32 product is off by up to 0.016 radians) while its
// first heads are on the way; a lane keeps the sines of its elements in
// registers over all heads of a position (with a division per head to find
// its position and the sines read per head the arithmetic was the bound: 36
// us).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "device.h"
#include "internal.h"

namespace hrs {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRot = 256;
constexpr int kMaxTokens = 4;   // positions a block takes at most
constexpr int kBatch = 4;       // heads of a lane group whose loads go out together

struct RopeArgs {
  const void* q;
  const void* k;
  const void* qw;
  const void* kw;
  const double* freq;
  const int32_t* seq_len;
  void* q_out;
  void* k_out;
  int64_t q_stride;
  int64_t k_stride;
  float eps;
  float offset;
  int32_t n_q;        // query heads
  int32_t n_heads;    // query and key heads
  int32_t d;
  int32_t rot;
  int32_t interleaved;
  int32_t n_pos;
  int32_t req0;
  int32_t n_tok;      // positions of this launch (requests x n_pos)
  int32_t per_block;  // positions per block
};
// Trees carry their positions' depths; chains do not, since every launch
// copies its arguments (one position: 5.9 us a call with 3 KB more of them,
// 4.5 without).
struct RopeTree : RopeArgs {
  int8_t depth[kGeomBytes];
};
__device__ __forceinline__ int depth_of(const RopeArgs&, int, int pos) { return pos; }
__device__ __forceinline__ int depth_of(const RopeTree& a, int i, int) { return a.depth[i]; }

template <int LPH> __device__ __forceinline__ float head_sum(float x) {
  if constexpr (LPH == 32) {
    x = group_sum<16>(x);
    return x + __shfl_xor(x, 16);
  } else {
    return group_sum<LPH>(x);
  }
}

// Eight elements; past the caches (nt) in launches of many positions (4096
// positions of 28 heads of 256: 24.9 vs 30.3 us).
template <bool NT> __device__ __forceinline__ void store16(u32x4* p, u32x4 v) {
  if constexpr (NT) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool NT> __device__ __forceinline__ void store8(float* p, const float* v) {
  store16<NT>(reinterpret_cast<u32x4*>(p), __builtin_bit_cast(u32x4, f32x4{v[0], v[1], v[2], v[3]}));
  store16<NT>(reinterpret_cast<u32x4*>(p) + 1, __builtin_bit_cast(u32x4, f32x4{v[4], v[5], v[6], v[7]}));
}
template <bool NT> __device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  store16<NT>(reinterpret_cast<u32x4*>(p),
              u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
}

template <typename T, int LPH, bool MANY, typename Args>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(const Args args) {
  constexpr int kGroups = kThreads / LPH;
  __shared__ __align__(16) float cs[kMaxTokens][kMaxRot / 2];
  __shared__ __align__(16) float sn[kMaxTokens][kMaxRot / 2];
  const int tok0 = blockIdx.x * args.per_block;
  const int n_tok = min(args.per_block, args.n_tok - tok0);
  const int group = threadIdx.x / LPH;
  const int lane = threadIdx.x % LPH;       // eight elements from 8 * lane
  const int half = args.rot >> 1;
  const bool mine = lane * 8 < args.d;
  // A lane group takes heads h0, h0 + step, ... of every position, kBatch of
  // them at a time.
  const int step = kGroups * gridDim.y;
  const int h0 = blockIdx.y * kGroups + group;
  const int batches = (args.n_heads + step * kBatch - 1) / (step * kBatch);

  // Eight elements as they were loaded; kBatch heads of a group on their way
  // at once.
  struct Raw {
    u32x4 w[sizeof(T) / 2];
    __device__ __forceinline__ void widen(float* o) const {
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[2 * i] = bf16_lo(w[0][i]);
          o[2 * i + 1] = bf16_hi(w[0][i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __uint_as_float(w[i / 4][i % 4]);
      }
    }
  };
  const T* const q = static_cast<const T*>(args.q);
  const T* const k = static_cast<const T*>(args.k);
  auto load_head = [&](int t, int h) {
    const int64_t row = static_cast<int64_t>(args.req0) * args.n_pos + tok0 + min(t, n_tok - 1);
    h = min(h, args.n_heads - 1);
    const T* p = h < args.n_q ? q + row * args.q_stride + h * args.d
                              : k + row * args.k_stride + (h - args.n_q) * args.d;
    Raw x = {};
    if (mine) {
      const u32x4* src = reinterpret_cast<const u32x4*>(p + lane * 8);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) x.w[i] = src[i];
    }
    return x;
  };

  Raw next[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b)
    if (b * step + h0 - group < args.n_heads) next[b] = load_head(0, h0 + b * step);
  float wq[8] = {}, wk[8] = {};
  if (mine && args.qw) load8<T>(static_cast<const T*>(args.qw) + lane * 8, wq);
  if (mine && args.kw) load8<T>(static_cast<const T*>(args.kw) + lane * 8, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    wq[i] += args.offset;
    wk[i] += args.offset;
  }
  for (int i = threadIdx.x; i < n_tok * half; i += kThreads) {
    const int t = i / half;
    const int f = i - t * half;
    const int rt = tok0 + t;
    const int rl = rt / args.n_pos;
    const int pos = rt - rl * args.n_pos;
    const int depth = depth_of(args, rl * args.n_pos + pos, pos);
    // Turns: at most 2^31 positions times 1 / 2 pi, off by a few 2^-53 of
    // that; what is left after whole turns is good to 32 bits.
    double a = static_cast<double>(static_cast<int64_t>(args.seq_len[args.req0 + rl]) + depth) * args.freq[f];
    a *= 0.15915494309189533577;
    a -= rint(a);
    float s, c;
    sincospif(2.0f * static_cast<float>(a), &s, &c);
    cs[t][f] = c;
    sn[t][f] = s;
  }
  __syncthreads();

  const float inv_d = 1.0f / static_cast<float>(args.d);
  // The lane's angles: of its eight elements where a pair's halves are apart
  // (half is a multiple of 8, so the partner's eight are one other lane's), of
  // its four pairs otherwise.
  const int hl = half >> 3;
  const bool low = lane < hl;
  const bool turns = args.interleaved ? lane * 8 < args.rot : lane < 2 * hl;
  const int f0 = !turns ? 0 : args.interleaved ? lane * 4 : (low ? lane : lane - hl) * 8;
  const int src = (threadIdx.x & 63) - lane + (!turns ? lane : low ? lane + hl : lane - hl);
  for (int t = 0; t < n_tok; ++t) {
    f32x4 c4[2], s4[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c4[i] = turns ? *reinterpret_cast<const f32x4*>(&cs[t][f0 + 4 * i]) : f32x4{1.0f, 1.0f, 1.0f, 1.0f};
      s4[i] = turns ? *reinterpret_cast<const f32x4*>(&sn[t][f0 + 4 * i]) : f32x4{};
    }
    for (int hb = 0; hb < batches; ++hb) {
      Raw now[kBatch];
      const bool last = hb + 1 == batches;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        now[b] = next[b];
        const int h = (last ? 0 : (hb + 1) * kBatch * step) + b * step + h0;
        if (h - group < args.n_heads && !(last && t + 1 == n_tok)) next[b] = load_head(t + last, h);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int h = (hb * kBatch + b) * step + h0;
        if (h - group >= args.n_heads) break;         // no group of the block has this head
        const bool is_q = h < args.n_q;
        float v[8];
        now[b].widen(v);
        if (is_q ? args.qw != nullptr : args.kw != nullptr) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
          const float r = __builtin_amdgcn_rsqf(fmaf(head_sum<LPH>(ss), inv_d, args.eps));
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] * r * (is_q ? wq[i] : wk[i]);
        }
        if (args.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float c = c4[0][i / 2], sv = s4[0][i / 2];
            const float x = v[i], y = v[i + 1];
            v[i] = turns ? x * c - y * sv : x;
            v[i + 1] = turns ? y * c + x * sv : y;
          }
        } else if (args.rot) {
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __shfl(v[i], src);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float sv = low ? -s4[i / 4][i % 4] : s4[i / 4][i % 4];
            v[i] = turns ? v[i] * c4[i / 4][i % 4] + o[i] * sv : v[i];
          }
        }
        if (mine && h < args.n_heads) {
          const int64_t row = static_cast<int64_t>(args.req0) * args.n_pos + tok0 + t;
          T* p = is_q ? static_cast<T*>(args.q_out) + (row * args.n_q + h) * args.d
                      : static_cast<T*>(args.k_out) + (row * (args.n_heads - args.n_q) + (h - args.n_q)) * args.d;
          store8<MANY>(p + lane * 8, v);
        }
      }
    }
  }
}

template <typename T, bool MANY, typename Args> void launch_heads(const Args& args, dim3 grid, hipStream_t s) {
  if (args.d > 128)
    hipLaunchKernelGGL((qk_norm_rope_kernel<T, 32, MANY, Args>), grid, dim3(kThreads), 0, s, args);
  else if (args.d > 64)
    hipLaunchKernelGGL((qk_norm_rope_kernel<T, 16, MANY, Args>), grid, dim3(kThreads), 0, s, args);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<T, 8, MANY, Args>), grid, dim3(kThreads), 0, s, args);
}
template <typename Args> void launch_rope(const Args& args, bool bf16, bool few, dim3 grid, hipStream_t s) {
  if (bf16) few ? launch_heads<uint16_t, false>(args, grid, s) : launch_heads<uint16_t, true>(args, grid, s);
  else few ? launch_heads<float, false>(args, grid, s) : launch_heads<float, true>(args, grid, s);
}

}  // namespace
}  // namespace hrs

using namespace hrs;

extern "C" int qk_norm_rope(const hrs_qk_desc* d, const void* q, const void* k, const void* q_weight,
                            const void* k_weight, const double* freq, const int32_t* seq_len, void* q_out,
                            void* k_out, void* stream) {
  if (d == nullptr || d->n_req < 1) return HRS_EINVAL;
  if (d->topo == HRS_TREE) {
    const int geo = check_topology(d->topo, d->parent, d->n_req, d->n_pos);
    if (geo != HRS_OK) return geo;
  } else if (d->topo != HRS_CHAIN || d->n_pos < 1 || d->n_pos > HRS_MAX_CHUNKED_POS) {
    return HRS_EINVAL;
  }
  if (d->n_heads < 1 || d->n_kvheads < 1 || d->n_heads > 65535 || d->n_kvheads > 65535 || !dtype_ok(d->dtype))
    return HRS_EINVAL;
  if (static_cast<int64_t>(d->n_req) * d->n_pos > (1 << 24)) return HRS_EINVAL;
  if (d->d < 16 || d->d > 256 || d->d % 16 != 0 || d->rot < 0 || d->rot > d->d || d->rot % 16 != 0)
    return HRS_EUNSUPPORTED;
  RopeTree args;
  if (!span_stride(d->q_stride, static_cast<int64_t>(d->n_heads) * d->d, &args.q_stride) ||
      !span_stride(d->k_stride, static_cast<int64_t>(d->n_kvheads) * d->d, &args.k_stride))
    return HRS_EINVAL;
  if (!q || !k || !seq_len || !q_out || !k_out || (d->rot > 0 && !freq)) return HRS_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_weight) || !aligned16(k_weight) || !aligned16(freq) ||
      !aligned16(seq_len) || !aligned16(q_out) || !aligned16(k_out))
    return HRS_EALIGN;

  args.q = q; args.k = k; args.qw = q_weight; args.kw = k_weight; args.freq = freq; args.seq_len = seq_len;
  args.q_out = q_out; args.k_out = k_out;
  args.eps = d->eps; args.offset = d->weight_offset;
  args.n_q = d->n_heads; args.n_heads = d->n_heads + d->n_kvheads;
  args.d = d->d; args.rot = d->rot; args.interleaved = d->interleaved != 0; args.n_pos = d->n_pos;
  const bool tree = d->topo == HRS_TREE;
  const int groups = kThreads / (d->d > 128 ? 32 : d->d > 64 ? 16 : 8);
  const int per_launch = tree ? std::max(1, kGeomBytes / d->n_pos) : d->n_req;
  (void)hipGetLastError();
  for (int r0 = 0; r0 < d->n_req; r0 += per_launch) {
    const int n = std::min(per_launch, d->n_req - r0);
    args.req0 = r0;
    args.n_tok = n * d->n_pos;
    if (tree)
      for (int r = 0; r < n; ++r)
        tree_depths(d->parent + static_cast<size_t>(r0 + r) * d->n_pos, d->n_pos, args.depth + r * d->n_pos);
    // Few positions: one per block and its heads over several blocks, one
    // head per lane group. Many: a block takes all heads of its positions,
    // so that the angles are formed once, and stores past the caches. The
    // border is a count of positions alone, not where the two meet: 28 heads of
    // 256 take 8.8 us at 511 positions, 12.0 at 512 (128 blocks), 12.7 at
    // 1024, 15.1 at 2048 and 22 at 4096; 10 heads of 128 4.8 at 511 and 6.5 at
    // 512, whose 1.3 MB the caches would have held.
    const bool few = args.n_tok < 512;
    args.per_block = few ? 1 : kMaxTokens;
    const dim3 grid((args.n_tok + args.per_block - 1) / args.per_block,
                    few ? std::min((args.n_heads + groups - 1) / groups, 65535) : 1);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (tree) launch_rope(args, d->dtype == HRS_BF16, few, grid, st);
    else launch_rope(static_cast<const RopeArgs&>(args), d->dtype == HRS_BF16, few, grid, st);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}
