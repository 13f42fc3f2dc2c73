// accept_sample_filtered: accept_sample (sample.hip) for requests that sample
// from the target's probabilities after top-k, top-p and min-p.
//
// openinfer PR #626 ("feat(qwen35): add opt-in DFlash speculative decoding"),
// Summary: greedy requests only; sampling falls back to plain decoding.
//
// The tokens that stay are the first n of a row in the order of their logits
// (equal ones by index): each limit keeps a beginning of that order. So a row
// is described by its last token that stays (the border: its logit's key above
// its complemented index, one number that compares in the order), its largest
// logit and the sum of the weights that stay.
//
// MI355X design: four dependent launches, no host round trip.
//  1. Candidates: every 32 KB chunk of every row is read once into registers. A
//     wave's j-th largest of its lanes' maxima bounds from below what can be
//     among the chunk's 4 j largest, so one comparison a logit leaves a short
//     list that holds everything above the bound. Bound by the read: rows with
//     a small top-k need no exponential here, others ten operations a logit.
//  2. Borders, a block a row: the chunks' largest bound T; everything above T is
//     in their lists. They are sorted in LDS with 64-bit weights and sums, which
//     settles top-k, and top-p and min-p where their border lies above T
//     (language models' rows). What stays is left behind as a list.
//     Rows that this does not settle (even distributions, hundreds of tokens)
//     read their logits again: a histogram of weights over 2048 bins, in whole
//     numbers of 2^-44 and less so that the order of the additions does not
//     matter, names the border's bin, whose members are sorted as above; bins
//     of too many members are divided by their keys until one number is left,
//     whose ties go by index.
//  3. Walk and draw: as accept_sample's, with the rows' descriptions; where the
//     node's row is a list the token is drawn from it at once.
//  4. Otherwise pieces' sums from 3 name the token's piece.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "sample.h"

namespace hrs {
namespace {

template <typename T> constexpr int kChunk = 32768 / sizeof(T);
constexpr int kList = 256;             // candidates that a chunk leaves at most
constexpr int kRow = 1024;             // threads of a row's block, and tokens of its list
constexpr int kBins = 2048;
constexpr int kSmallK = 64;            // a top-k up to this needs no row sums
constexpr double kCut = 48.0;          // e^-48 of the largest weight: no weight

struct ChunkInfo {
  double sum;        // of the weights beside the chunk's own maximum (not for a small top-k)
  float top;         // largest logit
  float low;         // smallest finite one
  uint32_t bound;    // everything with a key from here on is in the list
  int32_t n;         // how many that are; more than kList: the list is not whole
};

struct RowInfo {
  double top, sum;   // largest logit, sum of the weights that stay
  uint64_t border;   // order number of the last token that stays
  int32_t n;         // tokens of the list, -1: no list
  int32_t pad;
};

struct FilterArgs : SampleArgs {
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  ChunkInfo* chunks;   // workspace [rows][n_chunks]
  uint64_t* lists;     // workspace [rows][n_chunks][kList]: order numbers
  RowInfo* rows;       // workspace [rows]
  uint64_t* kept;      // workspace [rows][kRow]: complemented index above key, by index
};
using FilterTree = WithTree<FilterArgs>;

// Order-preserving key of a logit; zero for what never has a weight (NaN,
// -inf), and one key for both zeros.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return z > -__builtin_inff() ? k : 0;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
// Place in a row's order: larger comes first.
__device__ __forceinline__ uint64_t order_of(uint32_t key, int index) {
  return static_cast<uint64_t>(key) << 32 | ~static_cast<uint32_t>(index);
}

// What a request asks for. top_k outside (0, V): none; top_p: none from 1 on
// (or NaN); min_p: none up to 0 (or NaN), at most 1.
struct Limits {
  int k;             // V: none
  double p, m;       // 1: none; 0: none
  float tau;
  __device__ __forceinline__ Limits(const FilterArgs& a, int r) {
    k = a.top_k ? a.top_k[r] : 0;
    k = k <= 0 || k > a.vocab ? a.vocab : k;
    const float p_ = a.top_p ? a.top_p[r] : 1.0f, m_ = a.min_p ? a.min_p[r] : 0.0f;
    p = p_ < 1.0f ? fmax(static_cast<double>(p_), 0.0) : 1.0;
    m = m_ > 0.0f ? fmin(static_cast<double>(m_), 1.0) : 0.0;
    tau = temperature_of(a, r);
  }
};

// A logit below this beside the largest one has no weight.
__device__ __forceinline__ uint32_t cut_key(float top, float tau) {
  if (top == -__builtin_inff()) return 1;
  const float z = static_cast<float>(static_cast<double>(top) - kCut * fmax(static_cast<double>(tau), 0.0));
  return max(key_of(z), 1u);          // (+inf - inf, a NaN, gives 1; see below)
}

// e^((z - top) / tau) in float32 with the argument good to 2^-40 or so: its
// rounding error, which would be the same sign for all of a row's logits, goes
// back in as a factor.
struct FastWeigher {
  float top, hi, lo;
  bool hard;
  __device__ FastWeigher(float top_, float tau) : top(top_) {
    hard = tau == 0.0f || top == __builtin_inff();
    const double c = hard ? 1.0 : 1.4426950408889634074 / static_cast<double>(tau);
    hi = static_cast<float>(fmin(fmax(c, 1.2e-38), 3.4e38));
    lo = c < 1e30 ? static_cast<float>(c - hi) : 0.0f;
  }
  __device__ __forceinline__ float operator()(float z) const {
    if (hard) return z == top ? 1.0f : 0.0f;
    const float d = z - top;
    const float y = d * hi;
    const float rest = fmaf(d, lo, fmaf(d, hi, -y));
    const float w = __builtin_amdgcn_exp2f(y);
    return z > -__builtin_inff() && y > -200.0f ? fmaf(w, rest * 0.69314718f, w) : 0.0f;   // (NaN has none)
  }
};

// 1. Grid: (row, chunk).
template <typename T> __global__ __launch_bounds__(kThreads) void candidate_kernel(const FilterArgs args) {
  const int chunk = blockIdx.x % args.n_chunks;
  const int64_t row = static_cast<int64_t>(args.req0) * args.n_pos + blockIdx.x / args.n_chunks;
  const int r = static_cast<int>(row / args.n_pos);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* base = static_cast<const T*>(args.logits) + row * args.vocab;
  constexpr int kIter = kChunk<T> / (kThreads * 8);   // 8-logit slices per thread
  const int begin = chunk * kChunk<T>;
  const int end = min(args.vocab, begin + kChunk<T>);
  float v[kIter][8];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const int e = begin + (it * kThreads + static_cast<int>(threadIdx.x)) * 8;
    load8_nt<T>(base + min(e, end - 8), v[it]);
  }
  const Limits lim(args, r);
  // Slices past the row's end count as NaN.
  float m = -__builtin_inff(), low = __builtin_inff();
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const bool on = begin + (it * kThreads + static_cast<int>(threadIdx.x)) * 8 < end;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[it][i] = on ? __builtin_canonicalizef(v[it][i]) : __builtin_nanf("");
      m = fmaxf(m, v[it][i]);
      low = fminf(low, v[it][i] > -__builtin_inff() ? v[it][i] : __builtin_inff());
    }
  }
  // The wave's j-th largest of the lanes' maxima, a bit at a time; the bits that
  // a bf16 key has no say in stay zero.
  const bool small = lim.k <= kSmallK && lim.k < args.vocab;
  const int j = small ? (lim.k + 3) / 4 : kSmallK / 4;
  const uint32_t mine = key_of(m);
  uint32_t bound = 0;
#pragma unroll
  for (int b = 31; b >= (sizeof(T) == 2 ? 16 : 0); --b) {
    const uint32_t up = bound | 1u << b;
    if (__popcll(__ballot(mine >= up)) >= j) bound = up;
  }
  float top = m;
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    top = fmaxf(top, __shfl_xor(top, d));
    low = fminf(low, __shfl_xor(low, d));
  }
  __shared__ float tops[kThreads / 64], lows[kThreads / 64];
  __shared__ uint32_t bounds[kThreads / 64];
  __shared__ int32_t count;
  __shared__ double lds[kThreads / 64];
  if (lane == 0) {
    tops[wave] = top;
    lows[wave] = low;
    bounds[wave] = bound;
  }
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    top = fmaxf(top, tops[i]);
    low = fminf(low, lows[i]);
    bound = min(bound, bounds[i]);
  }
  bound = max(bound, cut_key(top, lim.tau));
  if (top == __builtin_inff()) bound = key_of(top);
  uint64_t* const list = args.lists + (row * args.n_chunks + chunk) * kList;
  if (mine >= bound) {
#pragma unroll
    for (int it = 0; it < kIter; ++it)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t k = key_of(v[it][i]);
        if (k >= bound) {
          const int at = atomicAdd(&count, 1);
          if (at < kList) list[at] = order_of(k, begin + (it * kThreads + static_cast<int>(threadIdx.x)) * 8 + i);
        }
      }
  }
  double sum = 0.0;
  if (!small && top > -__builtin_inff()) {
    const FastWeigher weigh(top, lim.tau);
    float s = 0.0f;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      float s8 = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s8 += weigh(v[it][i]);
      s += s8;
    }
    sum = s;
  }
  if (!small) sum = block_reduce(sum, add, lds);
  else __syncthreads();
  if (threadIdx.x == 0) args.chunks[row * args.n_chunks + chunk] = ChunkInfo{sum, top, low, bound, count};
}

// Sums over the first n threads' values, in order, over a block of kRow threads.
template <typename V> __device__ __forceinline__ V row_scan(V x, V* lds, V* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const V y = __shfl_up(x, d);
    x += lane >= d ? y : V(0);
  }
  __syncthreads();
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kRow / 64; ++i) {
    before += i < wave ? lds[i] : V(0);
    all += lds[i];
  }
  *total = all;
  return before + x;
}
// Smallest value over the block.
__device__ __forceinline__ int row_min(int x, int* lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = min(x, __shfl_xor(x, d));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  x = lds[0];
#pragma unroll
  for (int i = 1; i < kRow / 64; ++i) x = min(x, lds[i]);
  return x;
}

// a[0 .. n) (n a power of two, at most 2 kRow) in descending order. Up to 128
// numbers are one wave's work and need no barrier of the block.
__device__ __forceinline__ void sort_step(uint64_t* a, int i, int size, int apart) {
  const int lo = 2 * apart * (i / apart) + i % apart, hi = lo + apart;
  const uint64_t x = a[lo], y = a[hi];
  if (((lo & size) == 0) == (x < y)) {
    a[lo] = y;
    a[hi] = x;
  }
}
__device__ __forceinline__ void sort_down(uint64_t* a, int n) {
  const int tid = threadIdx.x;
  __syncthreads();
  for (int size = 2; size <= n; size <<= 1)
    for (int apart = size >> 1; apart > 0; apart >>= 1) {
      if (n > 128) {
        if (tid < n / 2) sort_step(a, tid, size, apart);
        __syncthreads();
      } else {
        if (tid < n / 2) sort_step(a, tid, size, apart);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }
  __syncthreads();
}
__device__ __forceinline__ int padded(int n) {
  int p = 2;
  while (p < n) p <<= 1;
  return p;
}

struct RowLds {
  uint64_t list[2 * kRow];
  uint64_t hist[kBins];
  union {
    double d[kRow / 64];
    uint64_t u[kRow / 64];
    int i[kRow / 64];
  } sums;
  uint64_t found;        // hand-over from one thread to all
  uint64_t above;
  uint32_t least, most;
  int32_t n;
};

// A row's logits, eight a thread, four slices on their way at once; f(index of
// the first, eight logits).
template <typename T, typename F> __device__ __forceinline__ void each_slice(const T* row, int V, F f) {
  for (int e0 = threadIdx.x * 8; e0 < V; e0 += 4 * 8 * kRow) {
    float z[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) load8<T>(row + min(e0 + u * 8 * kRow, V - 8), z[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e0 + u * 8 * kRow < V) f(e0 + u * 8 * kRow, z[u]);
  }
}

// A weight as a whole number of 2^-shift.
struct WholeWeigher {
  FastWeigher w;
  double scale;
  __device__ WholeWeigher(float top, float tau, int shift) : w(top, tau), scale(ldexp(1.0, shift)) {}
  __device__ __forceinline__ uint64_t operator()(float z) const {
    // The whole number is what a double's mantissa holds beside 2^52.
    return __builtin_bit_cast(uint64_t, fma(static_cast<double>(w(z)), scale, 0x1p52)) & ((uint64_t{1} << 52) - 1);
  }
};

// Order number of the first token, of those that `in` admits, at which the sum
// of amount(logit) over the order reaches `target`; zero if it is not reached.
// Everything from `ceiling` on is before the row's first token. Several reads of
// the row.
template <typename T, typename In, typename Amount>
__device__ uint64_t select_border(const T* row, int V, float top, float low, uint64_t target, In in, Amount amount, RowLds& s) {
  const int tid = threadIdx.x;
  // First by equal steps of the logits: neighbours in memory then seldom meet
  // in a bin (keys crowd around powers of two).
  const float step = top > low && top < __builtin_inff() ? fminf((kBins - 1) / (top - low), 3.0e38f) : 0.0f;
  auto bin_of = [&](float z) {
    if (!(step > 0.0f)) return z == top ? 0 : kBins - 1;
    return static_cast<int>(fminf((top - z) * step, static_cast<float>(kBins - 1)));
  };
  uint32_t from = 1, to = 0xFFFFFFFFu;   // keys of the border's bin
  int shift = -1;                        // -1: bins by steps
  uint64_t above = 0;                    // amount in front of the bin
  for (;;) {
    for (int i = tid; i < kBins; i += kRow) s.hist[i] = 0;
    __syncthreads();
    each_slice(row, V, [&](int e, const float* z) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t k = key_of(z[i]);
        if (k < from || k > to || !in(k, e + i)) continue;
        const uint64_t x = amount(z[i]);
        if (x == 0) continue;
        const int b = shift < 0 ? bin_of(z[i]) : static_cast<int>((to - k) >> shift);
        atomicAdd(reinterpret_cast<unsigned long long*>(&s.hist[b]), static_cast<unsigned long long>(x));
      }
    });
    __syncthreads();
    const uint64_t h0 = s.hist[2 * tid], h1 = s.hist[2 * tid + 1];
    uint64_t total;
    const uint64_t upto = row_scan(h0 + h1, s.sums.u, &total);
    if (above + total < target) return 0;
    const uint64_t before = above + upto - h0 - h1;
    if (before < target && above + upto >= target) {
      const bool second = before + h0 < target;
      s.found = 2 * tid + second;
      s.above = before + (second ? h0 : 0);
    }
    __syncthreads();
    const int bin = static_cast<int>(s.found);
    above = s.above;
    // The bin's members.
    __syncthreads();
    if (tid == 0) {
      s.n = 0;
      s.least = 0xFFFFFFFFu;
      s.most = 0;
    }
    __syncthreads();
    each_slice(row, V, [&](int e, const float* z) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t k = key_of(z[i]);
        if (k < from || k > to || !in(k, e + i) || amount(z[i]) == 0) continue;
        if ((shift < 0 ? bin_of(z[i]) : static_cast<int>((to - k) >> shift)) != bin) continue;
        const int at = atomicAdd(&s.n, 1);
        if (at < 2 * kRow) s.list[at] = order_of(k, e + i);
        atomicMin(&s.least, k);
        atomicMax(&s.most, k);
      }
    });
    __syncthreads();
    const int n = s.n;
    from = s.least;
    to = s.most;
    if (n <= 2 * kRow) {
      const int size = padded(n);
      for (int i = tid; i < size; i += kRow)
        if (i >= n) s.list[i] = 0;
      sort_down(s.list, size);
      uint64_t x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) x[i] = 2 * tid + i < n ? amount(logit_of(s.list[2 * tid + i] >> 32)) : 0;
      uint64_t all;
      const uint64_t c = above + row_scan(x[0] + x[1], s.sums.u, &all);
      const uint64_t b = c - x[0] - x[1];
      if (b < target && c >= target) s.found = s.list[2 * tid + (b + x[0] < target)];
      __syncthreads();
      return s.found;
    }
    if (from == to) {
      // Ties: the border is the one with so many of the same in front of it.
      const uint64_t each = amount(logit_of(from));
      uint64_t left = (target - above + each - 1) / each;
      for (int e0 = 0; e0 < V; e0 += 8 * kRow) {
        const int e = e0 + tid * 8;
        float z[8];
        load8<T>(row + min(e, V - 8), z);
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) hits |= e < V && key_of(z[i]) == from && in(from, e + i) ? 1u << i : 0;
        uint64_t all;
        const uint64_t c = row_scan(static_cast<uint64_t>(__popc(hits)), s.sums.u, &all);
        if (c >= left && c - __popc(hits) < left) {
          uint32_t h = hits;
          for (uint64_t i = c - __popc(hits) + 1; i < left; ++i) h &= h - 1;
          s.found = order_of(from, e + __ffs(h) - 1);
        }
        if (all >= left) break;
        left -= all;
      }
      __syncthreads();
      return s.found;
    }
    // Bins of equal numbers of keys.
    shift = 0;
    while (((to - from) >> shift) >= kBins) ++shift;
  }
}

// 2. Grid: row.
template <typename T> __global__ __launch_bounds__(kRow) void border_kernel(const FilterArgs args) {
  __shared__ RowLds s;
  const int64_t row = static_cast<int64_t>(args.req0) * args.n_pos + blockIdx.x;
  const int r = static_cast<int>(row / args.n_pos);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int V = args.vocab;
  const ChunkInfo* const chunks = args.chunks + row * args.n_chunks;
  const Limits lim(args, r);
  // The chunks' maxima and the largest bound, by every wave for itself.
  float top = -__builtin_inff(), low = __builtin_inff();
  uint32_t bound = 1;
  for (int c = lane; c < args.n_chunks; c += 64) {
    const ChunkInfo x = chunks[c];
    top = fmaxf(top, x.top);
    low = fminf(low, x.low);
    bound = max(bound, x.bound);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    top = fmaxf(top, __shfl_xor(top, d));
    low = fminf(low, __shfl_xor(low, d));
    bound = max(bound, static_cast<uint32_t>(__shfl_xor(static_cast<int>(bound), d)));
  }
  RowInfo* const out = args.rows + row;
  if (top == -__builtin_inff() || bad_temperature(lim.tau)) {
    if (tid == 0) *out = RowInfo{top, 0.0, 0, 0, 0};
    return;
  }
  const Weigher weigh(top, lim.tau);
  const bool small = lim.k <= kSmallK && lim.k < V;
  double all = 0.0;                      // sum of the row's weights
  if (!small) {
    for (int c = lane; c < args.n_chunks; c += 64) {
      const ChunkInfo x = chunks[c];
      all += x.top > -__builtin_inff() ? x.sum * weigh(x.top) : 0.0;
    }
    all = wave_reduce(all, add);
  }
  if (lim.k == V && lim.p >= 1.0 && lim.m <= 0.0) {
    if (tid == 0) *out = RowInfo{top, all, 0, -1, 0};
    return;
  }
  // Everything from the bound on, from the chunks' lists.
  if (tid == 0) s.n = 0;
  __syncthreads();
  bool whole = true;
  for (int c = wave; c < args.n_chunks; c += kRow / 64) {
    const ChunkInfo x = chunks[c];
    if (key_of(x.top) < bound) continue;
    whole = whole && x.n <= kList;
    for (int i = lane; i < min(x.n, kList); i += 64) {
      const uint64_t o = args.lists[(row * args.n_chunks + c) * kList + i];
      if (o >> 32 < bound) continue;
      const int at = atomicAdd(&s.n, 1);
      if (at < kRow) s.list[at] = o;
    }
  }
  whole = __syncthreads_and(whole);
  const int n = s.n;
  if (whole && n <= kRow) {
    const int size = padded(n);
    if (tid >= n && tid < size) s.list[tid] = 0;
    sort_down(s.list, size);
    const uint64_t mine = tid < n ? s.list[tid] : 0;
    const double w = tid < n ? weigh(logit_of(mine >> 32)) : 0.0;
    double listed;
    const double c = row_scan(w, s.sums.d, &listed);
    // Below the bound is nothing that counts, or nothing of the first k.
    const bool ends = bound <= cut_key(top, lim.tau) || top == __builtin_inff() || lim.tau == 0.0f || lim.k <= n;
    const int nk = min(lim.k, n);
    if (tid == nk - 1) s.found = __builtin_bit_cast(uint64_t, c);
    __syncthreads();
    const double of_k = ends ? __builtin_bit_cast(double, s.found) : all;
    const bool known = ends || lim.k == V;               // the sum that top-p is a share of
    const int np = lim.p < 1.0 ? row_min(tid < nk && c >= lim.p * of_k ? tid + 1 : kRow + 1, s.sums.i) : kRow + 1;
    const int nm = lim.m > 0.0 ? row_min(tid < n && w < lim.m ? tid : kRow + 1, s.sums.i) : kRow + 1;
    if ((lim.p >= 1.0 || known) && (ends || np <= n || nm < n)) {
      const int stay = min(nk, min(np, nm));
      __syncthreads();
      if (tid == stay - 1) *out = RowInfo{top, c, mine, stay, 0};
      // By index, for the draw: order numbers with their halves exchanged.
      const int pad = padded(stay);
      if (tid < pad)
        s.list[tid] = tid < stay ? static_cast<uint64_t>(static_cast<uint32_t>(mine)) << 32 | static_cast<uint32_t>(mine >> 32) : 0;
      sort_down(s.list, pad);
      if (tid < stay) args.kept[row * kRow + tid] = s.list[tid];
      return;
    }
  }
  // The row itself. Weights as whole numbers: at most 2^62 over all of it.
  const T* const logits = static_cast<const T*>(args.logits) + row * V;
  const int shift = min(50, __builtin_clz(V - 1) + 30);
  const WholeWeigher amount(top, lim.tau, shift);
  const float least = fmaxf(low, static_cast<float>(static_cast<double>(top) - kCut * static_cast<double>(lim.tau)));
  uint64_t border = order_of(1, 0x7FFFFFFF);             // everything that has a weight
  if (lim.k < V) {
    const uint64_t b = select_border(
        logits, V, top, low, static_cast<uint64_t>(lim.k), [](uint32_t k, int) { return k > 0; },
        [](float z) { return z > -__builtin_inff() ? uint64_t{1} : uint64_t{0}; }, s);
    border = max(border, b);
  }
  auto stays = [&](uint32_t k, int i) { return order_of(k, i) >= border; };
  auto sum_of = [&]() {
    uint64_t x = 0, total;
    each_slice(logits, V, [&](int e, const float* z) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x += stays(key_of(z[i]), e + i) ? amount(z[i]) : 0;
    });
    row_scan(x, s.sums.u, &total);
    return total;
  };
  if (lim.p < 1.0) {
    const uint64_t of_k = sum_of();
    const uint64_t target = max(uint64_t{1}, static_cast<uint64_t>(ceil(lim.p * static_cast<double>(of_k))));
    const uint64_t b = select_border(logits, V, top, least, target, stays, amount, s);
    border = max(border, b);
  }
  if (lim.m > 0.0) {
    // The smallest key whose weight is large enough: near the logit where it is
    // equal, and there by trying.
    uint32_t k = max(key_of(static_cast<float>(static_cast<double>(top) + static_cast<double>(lim.tau) * log(lim.m))), 1u);
    k = min(k, key_of(top));
    for (int i = 0; i < 4 && k > 1 && weigh(logit_of(k - 1)) >= lim.m; ++i) --k;
    for (int i = 0; i < 8 && k < key_of(top) && !(weigh(logit_of(k)) >= lim.m); ++i) ++k;
    border = max(border, order_of(k, 0x7FFFFFFF));
  }
  const uint64_t stay = sum_of();
  if (tid == 0) *out = RowInfo{top, ldexp(static_cast<double>(stay), -shift), border, -1, 0};
}

// The drafts' probabilities from the rows' descriptions, then the walk.
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
  const int t = threadIdx.x;
  if (t < T_) {
    const int p = max(0, parent_of(args, rl * T_ + t, t));
    const int x = args.tokens[row0 + t];
    const double u = args.uniforms[row0 + t];
    const RowInfo ri = args.rows[row0 + p];
    const bool valid = t > 0 && x >= 0 && x < V;
    const float z = load_elem<T>(static_cast<const T*>(args.logits), (row0 + p) * V + (valid ? x : 0));
    const double q = args.draft ? draft_value(args, (row0 + p) * V + (valid ? x : 0)) : 1.0;
    double pr = t == 0 ? 1.0 : 0.0;
    if (valid && ri.sum > 0.0 && order_of(key_of(z), x) >= ri.border) pr = Weigher(ri.top, tau)(z) / ri.sum;
    w.prob[t] = pr;
    w.need[t] = valid || !args.draft ? u * q : __builtin_inf();
    w.tok[t] = x;
    if (write) args.token_prob[row0 + t] = static_cast<float>(pr);
  }
  __syncthreads();
  decide(args, rl, write, w);
}

__device__ __forceinline__ bool is_gone(const NodeInfo& info, int token) {
  bool gone = false;
  for (int i = 0; i < info.n_gone; ++i) gone = gone || info.gone[i] == token;
  return gone;
}

// The drawn token of a node whose row is a list, by one block.
__device__ __forceinline__ int draw_listed(const FilterArgs& a, const NodeInfo& info, const RowInfo& ri, int r, double u,
                                           double* lds, int32_t* ilds) {
  const float tau = temperature_of(a, r);
  const int64_t row = static_cast<int64_t>(r) * a.n_pos + info.node;
  const Weigher weigh(ri.top, tau);
  constexpr int kPer = kRow / kThreads;
  double plain[kPer], x[kPer], sum = 0.0, whole = 0.0;
  int token[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = threadIdx.x * kPer + i;
    const uint64_t e = at < ri.n ? a.kept[row * kRow + at] : 0;
    token[i] = static_cast<int>(~static_cast<uint32_t>(e >> 32));
    plain[i] = at < ri.n ? weigh(logit_of(static_cast<uint32_t>(e))) : 0.0;
    x[i] = plain[i];
    if (at < ri.n && info.mode == kRest) {
      const double y = plain[i] / ri.sum - draft_value(a, row * a.vocab + token[i]);
      x[i] = y > 0.0 ? y : 0.0;
    } else if (at < ri.n && info.mode == kWithout && is_gone(info, token[i])) {
      x[i] = 0.0;
    }
    sum += x[i];
    whole += plain[i];
  }
  double total = block_reduce(sum, add, lds);
  if (!(total > 0.0)) {                  // nothing is left over: the row itself
    total = block_reduce(whole, add, lds);
    sum = whole;
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = plain[i];
  }
  const double c = block_scan(sum, lds);
  const double target = u * total;
  int owner = first_hit(sum > 0.0 && c > target, ilds);
  const bool passes = owner < kThreads;
  if (!passes) owner = last_hit(sum > 0.0, ilds);
  __shared__ int32_t pick;
  if (threadIdx.x == 0) pick = 0;
  __syncthreads();
  if (static_cast<int>(threadIdx.x) == owner) {
    double run = c - sum;
    bool done = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      run += x[i];
      if (x[i] > 0.0 && !done) {
        pick = token[i];
        done = passes && run > target;
      }
    }
  }
  __syncthreads();
  return pick;
}

// Weights of the thread's eight logits of a piece; *plain: without what the
// walk left out.
template <typename T>
__device__ __forceinline__ double filtered_weights(const FilterArgs& a, const NodeInfo& info, const RowInfo& ri, int mode, int r,
                                                   int piece, double* x, double* plain) {
  const int64_t row = (static_cast<int64_t>(r) * a.n_pos + info.node) * a.vocab;
  float z[8];
  const int n = load_piece(static_cast<const T*>(a.logits) + row, a.vocab, piece, z);
  const int v0 = piece * kPiece + threadIdx.x * 8;
  const Weigher weigh(ri.top, temperature_of(a, r));
  float q[8] = {};
  if (mode == kRest && n) {
    if (a.draft_bf16) load8<uint16_t>(static_cast<const uint16_t*>(a.draft) + row + v0, q);
    else load8<float>(static_cast<const float*>(a.draft) + row + v0, q);
  }
  const uint32_t gone = mode == kWithout ? gone_mask(info, v0) : 0;
  double sum = 0.0, all = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    double y = n && order_of(key_of(z[i]), v0 + i) >= ri.border ? weigh(z[i]) : 0.0;
    all += y;
    if (mode == kRest) {
      y = y / ri.sum - static_cast<double>(q[i]);
      y = n && y > 0.0 ? y : 0.0;
    } else if ((gone >> i) & 1) {
      y = 0.0;
    }
    x[i] = y;
    sum += y;
  }
  *plain = all;
  return sum;
}

// 3. Grid: (piece, request).
template <typename T, typename Args>
__global__ __launch_bounds__(kThreads) void filter_node_kernel(const Args args) {
  __shared__ WalkLds w;
  __shared__ double lds[kThreads / 64];
  __shared__ int32_t ilds[kThreads / 64];
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
  const RowInfo ri = args.rows[static_cast<int64_t>(r) * args.n_pos + w.info.node];
  if (ri.n >= 0) {
    if (piece != 0) return;
    const double u = args.uniforms[static_cast<int64_t>(r) * args.n_pos];
    const int pick = draw_listed(args, w.info, ri, r, u, lds, ilds);
    if (threadIdx.x == 0) args.bonus[r] = pick;
    return;
  }
  double x[8], plain;
  double sum = filtered_weights<T>(args, w.info, ri, w.info.mode, r, piece, x, &plain);
  sum = block_reduce(sum, add, lds);
  plain = block_reduce(plain, add, lds);
  if (threadIdx.x == 0) args.part[static_cast<int64_t>(r) * args.n_pieces + piece] = double2{sum, plain};
}

// 4. Grid: request.
template <typename T> __global__ __launch_bounds__(kThreads) void filter_draw_kernel(const FilterArgs args) {
  __shared__ double lds[kThreads / 64];
  __shared__ int32_t ilds[kThreads / 64];
  __shared__ int32_t pick;
  const int r = args.req0 + blockIdx.x;
  const NodeInfo& info = args.info[r];
  if (info.bad) return;
  const RowInfo ri = args.rows[static_cast<int64_t>(r) * args.n_pos + info.node];
  if (ri.n >= 0) return;
  const double u = args.uniforms[static_cast<int64_t>(r) * args.n_pos];
  const Pieces<double2> part(args.part + static_cast<int64_t>(r) * args.n_pieces, args.n_pieces);
  int mode = info.mode;
  Found f = find_piece(part, [](double2 x) { return x.x; }, u);
  if (f.piece < 0 && mode != kPlain) {   // nothing is left over: the row itself
    mode = kPlain;
    f = find_piece(part, [](double2 x) { return x.y; }, u);
  }
  if (threadIdx.x == 0) pick = 0;
  if (f.piece >= 0) {
    double x[8], plain;
    const double sum = filtered_weights<T>(args, info, ri, mode, r, f.piece, x, &plain);
    const double c = f.before + block_scan(sum, lds);
    const double target = u * f.total;
    int owner = first_hit(sum > 0.0 && c > target, ilds);
    const bool passes = owner < kThreads;
    if (!passes) owner = last_hit(sum > 0.0, ilds);
    if (static_cast<int>(threadIdx.x) == owner) {
      double run = c - sum;
      bool done = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        run += x[i];
        if (x[i] > 0.0 && !done) {
          pick = f.piece * kPiece + threadIdx.x * 8 + i;
          done = passes && run > target;
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) args.bonus[r] = pick;
}

bool filter_desc_ok(const hrs_sample_desc* d) {
  return d && d->n_req >= 1 && d->n_req <= 65535 && d->vocab >= 8 && d->vocab <= (1 << 30) && d->vocab % 8 == 0 &&
         dtype_ok(d->logit_dtype) && (d->topo == HRS_CHAIN || d->topo == HRS_TREE) && d->n_pos >= 1 &&
         d->n_pos <= HRS_MAX_POS &&
         static_cast<int64_t>(d->n_req) * d->n_pos * ((static_cast<int64_t>(d->vocab) + 16383) / 16384) <= (1 << 24);
}

size_t filter_layout(const hrs_sample_desc* d, FilterArgs* args, char* ws) {
  const size_t rows = static_cast<size_t>(d->n_req) * d->n_pos;
  // Enough for either type.
  const size_t chunks = (static_cast<size_t>(d->vocab) + kChunk<float> - 1) / kChunk<float>;
  const size_t pieces = (static_cast<size_t>(d->vocab) + kPiece - 1) / kPiece;
  size_t at = 0;
  auto place = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return ws + here;
  };
  char* const p0 = place(rows * chunks * sizeof(ChunkInfo));
  char* const p1 = place(rows * chunks * kList * sizeof(uint64_t));
  char* const p2 = place(rows * sizeof(RowInfo));
  char* const p3 = place(rows * kRow * sizeof(uint64_t));
  char* const p4 = place(d->n_req * pieces * sizeof(double2));
  char* const p5 = place(d->n_req * sizeof(NodeInfo));
  if (args) {
    args->chunks = reinterpret_cast<ChunkInfo*>(p0);
    args->lists = reinterpret_cast<uint64_t*>(p1);
    args->rows = reinterpret_cast<RowInfo*>(p2);
    args->kept = reinterpret_cast<uint64_t*>(p3);
    args->part = reinterpret_cast<double2*>(p4);
    args->info = reinterpret_cast<NodeInfo*>(p5);
  }
  return at;
}

template <typename T> int filter_launch(const hrs_sample_desc* d, FilterTree& tree_args, hipStream_t s) {
  FilterArgs& args = tree_args;
  const bool tree = d->topo == HRS_TREE;
  // A launch's rows times chunks fit a grid (2^24 at most altogether).
  const int per_launch = tree ? std::max(1, kGeomBytes / d->n_pos) : d->n_req;
  (void)hipGetLastError();
  for (int r0 = 0; r0 < d->n_req; r0 += per_launch) {
    const int n = std::min(per_launch, d->n_req - r0);
    args.req0 = r0;
    if (tree)
      for (int i = 0; i < n * d->n_pos; ++i)
        tree_args.parent[i] = static_cast<int8_t>(d->parent[static_cast<size_t>(r0) * d->n_pos + i]);
    hipLaunchKernelGGL(candidate_kernel<T>, dim3(n * args.n_pos * args.n_chunks), dim3(kThreads), 0, s, args);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
    hipLaunchKernelGGL(border_kernel<T>, dim3(n * args.n_pos), dim3(kRow), 0, s, args);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
    if (tree)
      hipLaunchKernelGGL((filter_node_kernel<T, FilterTree>), dim3(args.n_pieces, n), dim3(kThreads), 0, s, tree_args);
    else
      hipLaunchKernelGGL((filter_node_kernel<T, FilterArgs>), dim3(args.n_pieces, n), dim3(kThreads), 0, s, args);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
    hipLaunchKernelGGL(filter_draw_kernel<T>, dim3(n), dim3(kThreads), 0, s, args);
    if (launch_error() != hipSuccess) return HRS_EDEVICE;
  }
  return HRS_OK;
}

}  // namespace
}  // namespace hrs

using namespace hrs;

extern "C" size_t accept_sample_filtered_workspace_bytes(const hrs_sample_desc* d) {
  return filter_desc_ok(d) ? filter_layout(d, nullptr, nullptr) : 0;
}

extern "C" int accept_sample_filtered(const hrs_sample_desc* d, const void* logits, const int32_t* tokens,
                                      const float* uniforms, const void* draft_probs, const float* temperature,
                                      const int32_t* top_k, const float* top_p, const float* min_p, float* token_prob,
                                      int32_t* accept_node, int32_t* accept_len, int32_t* path, int32_t* bonus,
                                      int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (d == nullptr) return HRS_EINVAL;
  if (d->topo == HRS_TREE || d->topo == HRS_CHAIN) {
    const int geo = check_topology(d->topo, d->parent, d->n_req < 1 ? 0 : d->n_req, d->n_pos);
    if (geo != HRS_OK) return geo;
  }
  if (!filter_desc_ok(d) || (draft_probs && !dtype_ok(d->draft_dtype))) return HRS_EINVAL;
  if (draft_probs && d->topo == HRS_TREE) return HRS_EUNSUPPORTED;
  if (!logits || !tokens || !uniforms || !token_prob || !accept_node || !accept_len || !path || !bonus)
    return HRS_EINVAL;
  if (!workspace || workspace_bytes < accept_sample_filtered_workspace_bytes(d)) return HRS_EINVAL;
  if (!aligned16(logits) || !aligned16(tokens) || !aligned16(uniforms) || !aligned16(draft_probs) ||
      !aligned16(temperature) || !aligned16(top_k) || !aligned16(top_p) || !aligned16(min_p) || !aligned16(token_prob) ||
      !aligned16(accept_node) || !aligned16(accept_len) || !aligned16(path) || !aligned16(bonus) || !aligned16(status) ||
      !aligned16(workspace))
    return HRS_EALIGN;

  FilterTree args;
  args.logits = logits; args.tokens = tokens; args.uniforms = uniforms; args.draft = draft_probs;
  args.temperature = temperature; args.token_prob = token_prob; args.accept_node = accept_node;
  args.accept_len = accept_len; args.path = path; args.bonus = bonus; args.status = status;
  args.stats = nullptr; args.rest = nullptr;
  args.top_k = top_k; args.top_p = top_p; args.min_p = min_p;
  args.n_req = d->n_req; args.n_pos = d->n_pos; args.vocab = d->vocab;
  const int chunk = d->logit_dtype == HRS_F32 ? kChunk<float> : kChunk<uint16_t>;
  args.n_chunks = (d->vocab + chunk - 1) / chunk;
  args.n_pieces = (d->vocab + kPiece - 1) / kPiece;
  args.draft_bf16 = d->draft_dtype == HRS_BF16;
  filter_layout(d, &args, static_cast<char*>(workspace));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return d->logit_dtype == HRS_BF16 ? filter_launch<uint16_t>(d, args, s) : filter_launch<float>(d, args, s);
}
