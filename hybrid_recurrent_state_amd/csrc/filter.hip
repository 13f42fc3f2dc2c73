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
// MI355X design: three dependent launches, no host round trip.
//  1. Candidates: every 32 KB chunk of every row is read once into registers. A
//     wave's j-th largest of its lanes' maxima bounds from below what can be
//     among the chunk's 4 j largest, so one comparison a logit leaves a short
//     list that holds everything above the bound. Bound by the read (272 rows of
//     151,936 bf16 logits, 83 MB: 21.3 us): rows with a small top-k need no
//     exponential here, others ten operations a logit, some of 64 bits.
//  2. Borders, a block a row: the chunks' largest bound T; everything above T is
//     in their lists. Of that the few dozen largest (a histogram of the logits
//     names them) are put in order by counting, and one wave with their weights
//     and sums in 64 bits settles top-k, and top-p and min-p where their border
//     lies among them (language models' rows: 9 us for 272); if not, and all
//     candidates' weights reach top-p's share, the block sorts and sums all of
//     them. What stays is left behind as a list.
//     Rows that this does not settle (even distributions, hundreds of tokens)
//     are read again, by the one block: 18 bytes a nanosecond, 17 us for
//     151,936 bf16 logits. A bf16 row's values are counted one by one, the 15,360
//     from the largest down, and a second read finds the border among equal ones
//     (72 rows: 50 us). From a largest logit of 0.0078 on they end above zero: a
//     row whose border is not above it is counted in vain and goes on as float32
//     rows do (even rows cut by top-p, whole calls: 91 us; the same logits less
//     four 279, less eight 289; float32 247 wherever the border is).
//     A float32 row has a histogram of weights over 2048 bins, in whole numbers
//     of 2^-50 or so that the order of the additions does not matter, that
//     names the border's bin, whose members are sorted; bins of too many members
//     are divided by their keys until one number is left, whose ties go by
//     index.
//  3. Walk and draw: as accept_sample's, with the rows' descriptions; where the
//     node's row is a list the token is drawn from it at once (5 us). Otherwise
//     the row's pieces are summed by many blocks, and the last of them to be
//     done finds the token's piece and the token: 23 us, where a launch of its
//     own for that took 8 and 7 but also 4 for rows that need nothing of it.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sample.h"

namespace hrs {
namespace {

template <typename T> constexpr int kChunk = 32768 / sizeof(T);
constexpr int kList = 256;             // candidates that a chunk leaves at most
constexpr int kRow = 512;              // threads of a row's block
constexpr int kTokens = 1024;          // tokens of a row's list at most
constexpr int kPool = 2048;            // candidates that a block sorts at most
constexpr int kFew = 256;              // candidates that one wave settles
constexpr int kBins = 2048;
constexpr int kValues = 15360;         // values of a bf16 row that are counted one by one, from the largest down
constexpr int kGroup = 4;              // pieces of a row that a block sums
constexpr int kSmallK = 64;            // a top-k up to this needs no row sums
constexpr double kCut = 48.0;          // e^-48 of the largest weight: no weight
constexpr uint32_t kLeastKey = 0x00800000u;   // of the lowest finite logit

struct ChunkInfo {
  double sum;        // of the weights beside the chunk's own maximum (not for a small top-k), good to 18 u
  float top;         // largest logit
  uint32_t bound;    // everything with a key from here on is in the list
  int32_t n;         // how many that are; more than kList: the list is not whole
  int32_t pad;
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
  uint64_t* kept;      // workspace [rows][kTokens]: complemented index above key, by index
  int32_t* done;       // workspace [R]: pieces that are summed
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

// A logit below this key's beside the largest one has no weight.
__device__ __forceinline__ uint32_t cut_key(float top, float tau) {
  if (top == __builtin_inff()) return key_of(top);
  if (top == -__builtin_inff()) return kLeastKey;
  return max(key_of(static_cast<float>(static_cast<double>(top) - kCut * fmax(static_cast<double>(tau), 0.0))), kLeastKey);
}

// e^((z - top) / tau) as a float32 good to 3 u, u = 2^-24: the argument is formed
// in 64 bits, where neither differences nor temperatures at the ends of float32
// leave the range, and what its rounding for the exponential loses (the same
// sign for all of a row's logits, if they are alike) goes back in as a factor.
struct FastWeigher {
  double top, c;
  bool hard;
  __device__ FastWeigher(float top_, float tau) : top(top_) {
    hard = tau == 0.0f || top_ == __builtin_inff();
    c = hard ? 1.0 : 1.4426950408889634074 / static_cast<double>(tau);
  }
  __device__ __forceinline__ float operator()(float z) const {
    if (hard) return z == top ? 1.0f : 0.0f;
    const double x = (static_cast<double>(z) - top) * c;
    const float y = static_cast<float>(x);
    const float rest = static_cast<float>(x - static_cast<double>(y));
    const float w = __builtin_amdgcn_exp2f(y);
    return z > -__builtin_inff() && y > -200.0f ? fmaf(w, rest * 0.69314718f, w) : 0.0f;   // (NaN has none)
  }
};

// Largest number over the wave, the same in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  auto dpp = [&](auto ctrl) {
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, false)));
  };
  dpp(std::integral_constant<int, 0xB1>{});
  dpp(std::integral_constant<int, 0x4E>{});
  dpp(std::integral_constant<int, 0x141>{});
  dpp(std::integral_constant<int, 0x140>{});
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return max(b[0], b[1]);
}

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
  float m = -__builtin_inff();
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    const bool on = begin + (it * kThreads + static_cast<int>(threadIdx.x)) * 8 < end;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[it][i] = on ? __builtin_canonicalizef(v[it][i]) : __builtin_nanf("");
      m = fmaxf(m, v[it][i]);
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
  __shared__ uint32_t tops[kThreads / 64], bounds[kThreads / 64];
  __shared__ int32_t count;
  __shared__ double lds[kThreads / 64];
  uint32_t top_key = wave_max(mine);
  if (lane == 0) {
    tops[wave] = top_key;
    bounds[wave] = bound;
  }
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    top_key = max(top_key, tops[i]);
    bound = min(bound, bounds[i]);
  }
  const float top = top_key ? logit_of(top_key) : -__builtin_inff();
  bound = max(bound, cut_key(top, lim.tau));
  const float least = logit_of(bound);
  uint64_t* const list = args.lists + (row * args.n_chunks + chunk) * kList;
  if (m >= least) {
#pragma unroll
    for (int it = 0; it < kIter; ++it)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (v[it][i] >= least) {
          const int at = atomicAdd(&count, 1);
          if (at < kList)
            list[at] = order_of(key_of(v[it][i]), begin + (it * kThreads + static_cast<int>(threadIdx.x)) * 8 + i);
        }
  }
  double sum = 0.0;
  if (!small && top_key) {
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
  if (threadIdx.x == 0) args.chunks[row * args.n_chunks + chunk] = ChunkInfo{sum, top, bound, count, 0};
}

// Sum over the block's threads up to and with this one, in order.
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

// Sum over the lanes up to and with this one.
__device__ __forceinline__ double lane_scan(double x) {
  auto dpp = [&](auto ctrl, auto rows) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    constexpr int C = decltype(ctrl)::value, M = decltype(rows)::value;
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), C, M, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), C, M, 0xF, false);
    x += __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
  };
  using std::integral_constant;
  dpp(integral_constant<int, 0x111>{}, integral_constant<int, 0xF>{});
  dpp(integral_constant<int, 0x112>{}, integral_constant<int, 0xF>{});
  dpp(integral_constant<int, 0x114>{}, integral_constant<int, 0xF>{});
  dpp(integral_constant<int, 0x118>{}, integral_constant<int, 0xF>{});
  dpp(integral_constant<int, 0x142>{}, integral_constant<int, 0xA>{});
  dpp(integral_constant<int, 0x143>{}, integral_constant<int, 0xC>{});
  return x;
}
__device__ __forceinline__ double lane_of(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// a[0 .. n) (n a power of two) in descending order.
__device__ __forceinline__ void sort_down(uint64_t* a, int n) {
  __syncthreads();
  for (int size = 2; size <= n; size <<= 1)
    for (int apart = size >> 1; apart > 0; apart >>= 1) {
      for (int i = threadIdx.x; i < n / 2; i += kRow) {
        const int lo = 2 * apart * (i / apart) + i % apart, hi = lo + apart;
        const uint64_t x = a[lo], y = a[hi];
        if (((lo & size) == 0) == (x < y)) {
          a[lo] = y;
          a[hi] = x;
        }
      }
      __syncthreads();
    }
}
__device__ __forceinline__ int padded(int n) {
  int p = 2;
  while (p < n) p <<= 1;
  return p;
}

struct RowLds {
  alignas(16) uint64_t list[kPool];
  union {
    uint64_t hist[kBins];                // of whole-number weights
    uint32_t count[kValues + 1];         // of values, and of a negative zero behind the last
    struct {
      alignas(16) uint64_t few[kFew];    // the largest candidates
      alignas(16) uint64_t sorted[kFew];
      uint32_t bins[kFew];
    };
  };
  union {
    double d[kRow / 64];
    uint64_t u[kRow / 64];
    int i[kRow / 64];
  } sums;
  uint64_t found;        // hand-over from one thread to all
  uint64_t above;
  double weight;
  uint32_t least, most;
  int32_t n, m;
};
static_assert(sizeof(RowLds) <= 80 * 1024, "two blocks a CU");

// A row's logits, eight a thread; f(index of the first, eight logits). The next
// 256 bytes of a thread are on their way while it goes through the last: one
// block has a row to itself and nothing else hides the reads.
template <typename T> struct Slice {
  u32x4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) w[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  __device__ __forceinline__ void widen(float* z) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      z[i] = sizeof(T) == 4 ? __uint_as_float(w[i / 4 * (sizeof(T) / 4)][i % 4]) : i % 2 ? bf16_hi(w[0][i / 2]) : bf16_lo(w[0][i / 2]);
  }
};
template <typename T, typename F> __device__ __forceinline__ void each_raw(const T* row, int V, F f) {
  constexpr int kAhead = 16 / sizeof(T);
  constexpr int64_t kStep = static_cast<int64_t>(kAhead) * 8 * kRow;
  Slice<T> x[2][kAhead];
  const int64_t e0 = threadIdx.x * 8;
  auto load = [&](Slice<T>(&y)[kAhead], int64_t e) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) y[u].load(row + min(e + u * 8 * kRow, static_cast<int64_t>(V - 8)));
  };
  auto use = [&](const Slice<T>(&y)[kAhead], int64_t e) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (e + u * 8 * kRow < V) f(static_cast<int>(e + u * 8 * kRow), y[u]);
  };
  load(x[0], e0);
  for (int64_t e = e0; e < V; e += 2 * kStep) {
    load(x[1], e + kStep);
    use(x[0], e);
    load(x[0], e + 2 * kStep);
    use(x[1], e + kStep);
  }
}

template <typename T, typename F> __device__ __forceinline__ void each_slice(const T* row, int V, F f) {
  each_raw(row, V, [&](int e, const Slice<T>& x) {
    float z[8];
    x.widen(z);
    f(e, z);
  });
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

// The index of the nth (from 1) token with this key, by the whole block. Waves
// count their slices of 64 rounds at a time; the slice where the count is
// reached is looked through again.
template <typename T> __device__ int nth_of_key(const T* row, int V, uint32_t key, uint64_t nth, RowLds& s) {
  constexpr int kWaves = kRow / 64, kRounds = 64, kPart = kRounds * 8 * kRow;
  static_assert(kRounds * kWaves == kRow, "a count a thread");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t* const counts = reinterpret_cast<uint32_t*>(s.list);          // [rounds][waves]
  auto hits_of = [&](const float* z) {
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) hits |= key_of(z[i]) == key ? 1u << i : 0;
    return hits;
  };
  const bool zero = key == 0x80000000u;                // two patterns
  const uint32_t pattern = (__float_as_uint(logit_of(key)) >> 16) * 0x00010001u;
  uint64_t left = nth;
  for (int64_t base = 0; base < V; base += kPart) {
    __syncthreads();
    counts[tid] = 0;
    __syncthreads();
    each_raw(row + base, static_cast<int>(min(static_cast<int64_t>(kPart), V - base)), [&](int e, const Slice<T>& x) {
      int n = 8;
      if (sizeof(T) == 2 && !zero) {
        // Halves of words that differ from the value's have their upper bit set.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t y = x.w[0][i] ^ pattern;
          n -= __popc((((y & 0x7FFF7FFFu) + 0x7FFF7FFFu) | y) & 0x80008000u);
        }
      } else {
        float z[8];
        x.widen(z);
        n = __popc(hits_of(z));
      }
      if (n) atomicAdd(&counts[e / (8 * kRow) * kWaves + wave], static_cast<uint32_t>(n));
    });
    __syncthreads();
    uint64_t all;
    const uint32_t mine = counts[tid];
    const uint64_t upto = row_scan(static_cast<uint64_t>(mine), s.sums.u, &all);
    if (all >= left) {
      if (upto >= left && upto - mine < left) {
        s.found = tid;
        s.above = upto - mine;
      }
      __syncthreads();
      const int slice = static_cast<int>(s.found);
      left -= s.above;
      __syncthreads();
      if (wave == 0) {
        const int64_t e = base + (static_cast<int64_t>(slice / kWaves) * kRow + slice % kWaves * 64 + lane) * 8;
        uint32_t hits = 0;
        if (e < V) {
          float z[8];
          load8<T>(row + e, z);
          hits = hits_of(z);
        }
        int c = __popc(hits);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
          const int y = __shfl_up(c, d);
          c += lane >= d ? y : 0;
        }
        const int before = c - __popc(hits);
        if (static_cast<uint64_t>(c) >= left && static_cast<uint64_t>(before) < left) {
          for (int i = before + 1; i < static_cast<int>(left); ++i) hits &= hits - 1;
          s.found = static_cast<uint64_t>(e) + __ffs(hits) - 1;
        }
      }
      __syncthreads();
      const int index = static_cast<int>(s.found);
      __syncthreads();
      return index;
    }
    left -= all;
  }
  return 0;
}

struct Border {
  uint64_t order;    // zero: the target was not reached
  uint64_t sum;      // of the amounts up to and with it
};

// The first token, of those that `in` admits, at which the sum of
// amount(logit) over the order reaches the target: a share of the sum of all of
// them (share >= 0, rounded up, at least 1) or `target`. Bins divide the logits
// from `least` to `top`; what is below is in the last one. Two reads of the row,
// as a rule.
template <typename T, typename In, typename Amount>
__device__ Border select_border(const T* row, int V, float top, float least, double share, uint64_t target, In in, Amount amount,
                                RowLds& s) {
  const int tid = threadIdx.x;
  // First by equal steps of the logits: neighbours in memory then seldom meet
  // in a bin (keys crowd around powers of two).
  const float step = top > least && top < __builtin_inff() ? fminf((kBins - 1) / (top - least), 3.0e38f) : 0.0f;
  const bool steps = step > 0.0f;
  auto bin_of = [&](float z) {
    return steps ? static_cast<int>(fminf((top - z) * step, static_cast<float>(kBins - 1))) : z == top ? 0 : kBins - 1;
  };
  uint32_t from = kLeastKey, to = 0xFFFFFFFFu;   // keys of the border's bin
  int shift = -1;                                // -1: bins by steps
  uint64_t above = 0;                            // amount in front of the bin
  for (;;) {
    __syncthreads();
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
    constexpr int kPer = kBins / kRow;
    uint64_t h[kPer], sum = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += h[i] = s.hist[kPer * tid + i];
    const uint64_t upto = row_scan(sum, s.sums.u, &total);
    if (share >= 0.0) {
      target = max(uint64_t{1}, static_cast<uint64_t>(ceil(share * static_cast<double>(total))));
      share = -1.0;
    }
    if (above + total < target) return Border{0, above + total};
    uint64_t before = above + upto - sum;
    if (before < target && above + upto >= target) {
      int at = 0;
#pragma unroll
      for (int i = 0; i + 1 < kPer; ++i)
        if (at == i && before + h[i] < target) {
          before += h[i];
          ++at;
        }
      s.found = kPer * tid + at;
      s.above = before;
      s.n = 0;
      s.least = 0xFFFFFFFFu;
      s.most = 0;
    }
    __syncthreads();
    const int bin = static_cast<int>(s.found);
    above = s.above;
    // The bin's members.
    each_slice(row, V, [&](int e, const float* z) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (shift < 0 && bin_of(z[i]) != bin) continue;                  // (a NaN is in some bin)
        const uint32_t k = key_of(z[i]);
        if (k < from || k > to || !in(k, e + i) || amount(z[i]) == 0) continue;
        if (shift >= 0 && static_cast<int>((to - k) >> shift) != bin) continue;
        const int at = atomicAdd(&s.n, 1);
        if (at < kPool) s.list[at] = order_of(k, e + i);
        atomicMin(&s.least, k);
        atomicMax(&s.most, k);
      }
    });
    __syncthreads();
    const int n = s.n;
    from = s.least;
    to = s.most;
    if (n <= kPool) {
      const int size = padded(n);
      for (int i = tid; i < size; i += kRow)
        if (i >= n) s.list[i] = 0;
      sort_down(s.list, size);
      constexpr int kMine = kPool / kRow;
      uint64_t x[kMine], part = 0, all;
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        part += x[i] = kMine * tid + i < n ? amount(logit_of(s.list[kMine * tid + i] >> 32)) : 0;
      const uint64_t c = above + row_scan(part, s.sums.u, &all);
      uint64_t b = c - part;
      if (b < target && c >= target) {
        int at = 0;
#pragma unroll
        for (int i = 0; i + 1 < kMine; ++i)
          if (at == i && b + x[i] < target) {
            b += x[i];
            ++at;
          }
        s.found = s.list[kMine * tid + at];
        s.above = b + amount(logit_of(s.found >> 32));
      }
      __syncthreads();
      const Border found{s.found, s.above};
      __syncthreads();
      return found;
    }
    if (from == to) {
      // Ties: the border is the one with so many of the same in front of it
      // (`in` admits whole rows or, by index, a beginning of each key's).
      const uint64_t each = amount(logit_of(from));
      const uint64_t nth = (target - above + each - 1) / each;
      return Border{order_of(from, nth_of_key(row, V, from, nth, s)), above + nth * each};
    }
    // Bins of equal numbers of keys.
    shift = 0;
    while (((to - from) >> shift) >= kBins) ++shift;
  }
}

// 2. Grid: row.
template <typename T> __global__ __launch_bounds__(kRow, 4) void border_kernel(const FilterArgs args) {
  __shared__ RowLds s;
  const int64_t row = static_cast<int64_t>(args.req0) * args.n_pos + blockIdx.x;
  const int r = static_cast<int>(row / args.n_pos);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int V = args.vocab;
  const ChunkInfo* const chunks = args.chunks + row * args.n_chunks;
  const ChunkInfo mine = chunks[min(lane, args.n_chunks - 1)];
  const Limits lim(args, r);
  if (tid < kFew) s.bins[tid] = 0;
  if (tid == 0) {
    s.n = s.m = 0;
    if (row == static_cast<int64_t>(r) * args.n_pos) args.done[r] = 0;
  }
  // The chunks' maxima and the largest bound, by every wave for itself.
  uint32_t top_key = key_of(mine.top), bound = max(mine.bound, kLeastKey);
  for (int c = lane + 64; c < args.n_chunks; c += 64) {
    top_key = max(top_key, key_of(chunks[c].top));
    bound = max(bound, chunks[c].bound);
  }
  top_key = wave_max(top_key);
  bound = wave_max(bound);
  RowInfo* const out = args.rows + row;
  if (top_key == 0 || bad_temperature(lim.tau)) {
    if (tid == 0) *out = RowInfo{-__builtin_inf(), 0.0, 0, 0, 0};
    return;
  }
  const float top = logit_of(top_key);
  const Weigher weigh(top, lim.tau);
  const bool hard = lim.tau == 0.0f || top == __builtin_inff();
  const bool small = lim.k <= kSmallK && lim.k < V;
  double all = 0.0;                      // sum of the row's weights
  if (!small) {
    for (int c = lane; c < args.n_chunks; c += 64) {
      const ChunkInfo x = c < 64 ? mine : chunks[c];
      all += x.top > -__builtin_inff() ? x.sum * weigh(x.top) : 0.0;
    }
    all = wave_reduce(all, add);
  }
  if (lim.k == V && lim.p >= 1.0 && lim.m <= 0.0) {
    if (tid == 0) *out = RowInfo{top, all, 0, -1, 0};
    return;
  }
  const uint32_t cut = cut_key(top, lim.tau);
  __syncthreads();
  // Everything from the bound on, from the chunks' lists, and how it is spread
  // from there to the largest logit.
  const float low = logit_of(bound);
  const float per = top > low && top < __builtin_inff() ? fminf((kFew - 1) / (top - low), 3.0e38f) : 0.0f;
  auto bin_of = [&](float z) { return per > 0.0f ? static_cast<int>(fminf((top - z) * per, static_cast<float>(kFew - 1))) : 0; };
  bool whole = true;
  for (int c = wave; c < args.n_chunks; c += kRow / 64) {
    const ChunkInfo x = chunks[c];
    if (key_of(x.top) < bound) continue;
    whole = whole && x.n <= kList;
    for (int i = lane; i < min(x.n, kList); i += 64) {
      const uint64_t o = args.lists[(row * args.n_chunks + c) * kList + i];
      if (o >> 32 < bound) continue;
      const int at = atomicAdd(&s.n, 1);
      if (at < kPool) s.list[at] = o;
      atomicAdd(&s.bins[bin_of(logit_of(o >> 32))], 1u);
    }
  }
  whole = __syncthreads_and(whole);
  const int n = s.n;
  whole = whole && n <= kPool;
  // Language models' rows: the first few dozen settle it, by one wave. A bin's
  // end that leaves as many as top-k asks for, 64 at least.
  if (whole) {
    const int wanted = lim.k <= kFew / 2 ? max(lim.k, 64) : 64;
    int last = kFew - 1;                 // last bin that is taken
    {
      uint32_t c[kFew / 64], sum = 0;
#pragma unroll
      for (int i = 0; i < kFew / 64; ++i) sum += c[i] = s.bins[lane * (kFew / 64) + i];
      uint32_t upto = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = __shfl_up(static_cast<int>(upto), d);
        upto += lane >= d ? y : 0;
      }
      const uint64_t hit = __ballot(upto >= static_cast<uint32_t>(wanted));
      if (hit) {
        const int L = __builtin_ctzll(hit);
        uint32_t run = upto - sum;
        int at = kFew / 64 - 1;
        for (int i = kFew / 64 - 1; i >= 0; --i) {
          uint32_t x = run;
          for (int k = 0; k <= i; ++k) x += c[k];
          if (x >= static_cast<uint32_t>(wanted)) at = i;
        }
        last = L * (kFew / 64) + __builtin_amdgcn_readlane(at, L);
      }
    }
    for (int i = tid; i < n; i += kRow) {
      const uint64_t o = s.list[i];
      if (bin_of(logit_of(o >> 32)) > last) continue;
      const int at = atomicAdd(&s.m, 1);
      if (at < kFew) s.few[at] = o;
    }
    __syncthreads();
    const int m = s.m;
    if (m <= kFew) {
      // Places by counting what is larger.
      if (tid == 0 && (m & 1)) s.few[m] = 0;            // (kFew is even)
      __syncthreads();
      if (tid < m) {
        const uint64_t o = s.few[tid];
        int place = 0;
        for (int i = 0; i < m; i += 2) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(&s.few[i]);
          place += (static_cast<uint64_t>(x.y) << 32 | x.x) > o;
          place += (static_cast<uint64_t>(x.w) << 32 | x.z) > o;
        }
        s.sorted[place] = o;
      }
      __syncthreads();
      if (wave == 0) {
        constexpr int kPer = kFew / 64;
        double w[kPer], c[kPer], sum = 0.0;
        uint64_t o[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int at = lane * kPer + i;
          o[i] = at < m ? s.sorted[at] : 0;
          w[i] = at < m ? weigh(logit_of(o[i] >> 32)) : 0.0;
          sum += w[i];
          c[i] = sum;
        }
        const double before = lane_scan(sum) - sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) c[i] += before;
        auto at_place = [&](const double* x, int place) {
          const int L = place / kPer, k = place % kPer;
          double y = x[0];
#pragma unroll
          for (int i = 1; i < kPer; ++i) y = k == i ? x[i] : y;
          return lane_of(y, L);
        };
        // The first place where a condition holds, or kTokens.
        auto first = [&](auto holds) {
          int at = kTokens;
#pragma unroll
          for (int i = kPer - 1; i >= 0; --i) at = holds(lane * kPer + i, i) ? lane * kPer + i : at;
          const uint64_t hit = __ballot(at < kTokens);
          return hit ? __builtin_amdgcn_readlane(at, __builtin_ctzll(hit)) : kTokens;
        };
        // What is not here has no weight, or is none of the first k.
        const bool ends = (m == n && bound <= cut) || hard || lim.k <= m;
        const int nk = min(lim.k, m);
        const double of_k = ends ? at_place(c, nk - 1) : all;
        const bool known = lim.p >= 1.0 || ends || lim.k == V;
        const int np = lim.p < 1.0 ? first([&](int at, int i) { return at < nk && c[i] >= lim.p * of_k; }) + 1 : kTokens + 1;
        const int nm = lim.m > 0.0 ? first([&](int at, int i) { return at < m && w[i] < lim.m; }) : kTokens + 1;
        const bool settled = known && (ends || np <= m || nm < m);
        if (settled) {
          const int stay = min(nk, min(np, nm));
          const double kept = at_place(c, stay - 1);
          if (lane == 0) {
            *out = RowInfo{top, kept, s.sorted[stay - 1], stay, 0};
            s.m = -1;
          }
          // By index, for the draw: order numbers with their halves exchanged,
          // which places count what has a smaller index of.
          for (int e = lane; e < stay; e += 64) {
            const uint64_t x = s.sorted[e];
            int place = 0;
            for (int i = 0; i < stay; ++i) place += static_cast<uint32_t>(s.sorted[i]) > static_cast<uint32_t>(x);
            args.kept[row * kTokens + place] = x << 32 | x >> 32;
          }
        }
      }
      __syncthreads();
      if (s.m < 0) return;
    }
  }
  // All candidates, by the block, where they can settle it: not if their
  // weights fall short of top-p's share of the same total (by more than another
  // order of the additions makes).
  bool worth = whole && n <= kTokens;
  if (worth && lim.p < 1.0 && lim.k > n && bound > cut && !hard) {
    if (lim.k < V) {
      worth = false;                     // the sum of the first k is not known
    } else if (!(lim.m > 0.0 && weigh(low) < lim.m * (1.0 + 1e-9))) {
      double x = 0.0, listed;
      for (int i = tid; i < n; i += kRow) x += weigh(logit_of(s.list[i] >> 32));
      row_scan(x, s.sums.d, &listed);
      worth = listed >= lim.p * all * (1.0 - 1e-9);
    }
  }
  if (worth) {
    const int size = padded(n);
    for (int i = n + tid; i < size; i += kRow) s.list[i] = 0;
    sort_down(s.list, size);
    constexpr int kPer = kTokens / kRow;
    uint64_t o[kPer];
    double w[kPer], c[kPer], sum = 0.0, listed;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = kPer * tid + i;
      o[i] = at < n ? s.list[at] : 0;
      w[i] = at < n ? weigh(logit_of(o[i] >> 32)) : 0.0;
      sum += w[i];
      c[i] = sum;
    }
    const double before = row_scan(sum, s.sums.d, &listed) - sum;
    const bool ends = bound <= cut || hard || lim.k <= n;
    const int nk = min(lim.k, n);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] += before;
      if (kPer * tid + i == nk - 1) s.weight = c[i];
    }
    __syncthreads();
    const double of_k = ends ? s.weight : all;
    const bool known = lim.p >= 1.0 || ends || lim.k == V;               // the sum that top-p is a share of
    int np = kTokens + 1, nm = kTokens + 1;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) {
      const int at = kPer * tid + i;
      if (lim.p < 1.0 && at < nk && c[i] >= lim.p * of_k) np = at + 1;
      if (lim.m > 0.0 && at < n && w[i] < lim.m) nm = at;
    }
    np = row_min(np, s.sums.i);
    nm = row_min(nm, s.sums.i);
    if (known && (ends || np <= n || nm < n)) {
      const int stay = min(nk, min(np, nm));
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (kPer * tid + i == stay - 1) *out = RowInfo{top, c[i], o[i], stay, 0};
      // By index, for the draw.
      const int pad = padded(stay);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = kPer * tid + i;
        if (at < pad) s.list[at] = at < stay ? o[i] << 32 | o[i] >> 32 : 0;
      }
      sort_down(s.list, pad);
      for (int i = tid; i < stay; i += kRow) args.kept[row * kTokens + i] = s.list[i];
      return;
    }
  }
  // The row itself.
  const T* const logits = static_cast<const T*>(args.logits) + row * V;
  // Beside the largest weight, min-p is a key: near the logit where the weight
  // is equal, and there by trying.
  uint32_t key_m = kLeastKey;
  if (lim.m > 0.0) {
    key_m = max(key_of(static_cast<float>(static_cast<double>(top) + static_cast<double>(lim.tau) * log(lim.m))), kLeastKey);
    key_m = min(key_m, top_key);
    for (int i = 0; i < 4 && key_m > kLeastKey && weigh(logit_of(key_m - 1)) >= lim.m; ++i) --key_m;
    for (int i = 0; i < 8 && key_m < top_key && !(weigh(logit_of(key_m)) >= lim.m); ++i) ++key_m;
  }
  if constexpr (sizeof(T) == 2) {
    // A bf16 row has few values: they are counted one by one, from the largest
    // down to the cut if there is room, and every limit whose border is among
    // them is a number of tokens that follows from the counts, with sums in 64
    // bits. Ties at the border go by index.
    if (!hard) {
      const uint32_t first = top_key >> 16;
      const int down = static_cast<int>(first - (cut >> 16)) + 1, values = min(kValues, down);
      const bool ends = values == down;          // nothing behind the values has a weight
      auto value_key = [&](int at) {
        const uint32_t v = first - at;
        return v << 16 | (v < 0x8000u ? 0xFFFFu : 0u);
      };
      // A negative zero stands one place behind the other and counts there, also
      // where zero is the last of the values.
      const int zero = static_cast<int>(first - 0x8000u);
      const int places = values + (zero == values - 1);
      __syncthreads();
      for (int i = tid; i < places; i += kRow) s.count[i] = 0;
      __syncthreads();
      each_raw(logits, V, [&](int, const Slice<T>& x) {
        // Two patterns a word: keys as key_of's, but for the negative zero's,
        // which is one below the other's.
        typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w = x.w[0][i];
          const uint32_t sign = __builtin_bit_cast(uint32_t, __builtin_bit_cast(i16x2, w) >> i16x2{15, 15});
          const u16x2 key = __builtin_bit_cast(u16x2, w ^ (sign | 0x80008000u));
          const uint32_t at = __builtin_bit_cast(uint32_t, u16x2{static_cast<uint16_t>(first), static_cast<uint16_t>(first)} - key);
          if ((at & 0xFFFFu) < static_cast<uint32_t>(places)) atomicAdd(&s.count[at & 0xFFFFu], 1u);
          if (at >> 16 < static_cast<uint32_t>(places)) atomicAdd(&s.count[at >> 16], 1u);
        }
      });
      __syncthreads();
      if (tid == 0 && zero >= 0 && zero + 1 < places) {
        s.count[zero] += s.count[zero + 1];
        s.count[zero + 1] = 0;
      }
      __syncthreads();
      // A run of values a thread, in order, up to the last that there is.
      int end = 0;
      for (int i = tid; i < values; i += kRow) end = s.count[i] ? i + 1 : end;
      end = -row_min(-end, s.sums.i);
      const int run_len = (end + kRow - 1) / kRow;
      const int at0 = min(end, tid * run_len), at1 = min(end, at0 + run_len);
      uint64_t tokens = 0, all_tokens;
      double weight = 0.0, all_weight;
      for (int at = at0; at < at1; ++at) {
        const uint32_t c = s.count[at];
        tokens += c;
        if (c) weight += c * weigh(logit_of(value_key(at)));
      }
      const uint64_t upto = row_scan(tokens, s.sums.u, &all_tokens);
      const double mass = row_scan(weight, s.sums.d, &all_weight);
      // Of the thread whose run holds the n-th token: its value, its number
      // among those of this value, and the sum with it.
      struct Place {
        int at;
        uint64_t nth;
        double sum;
        bool last;
      };
      auto place_of = [&](uint64_t n) {
        uint64_t run = upto - tokens;
        double x = mass - weight;
        for (int at = at0; at < at1; ++at) {
          const uint64_t c = s.count[at];
          if (c == 0) continue;
          const uint64_t take = min(c, n - run);
          x += take * weigh(logit_of(value_key(at)));
          run += take;
          if (run == n) return Place{at, take, x, take == c};
        }
        return Place{at1 - 1, 1, x, true};
      };
      auto holds = [&](uint64_t n) { return upto >= n && upto - tokens < n; };
      const bool has_k = lim.k < V && static_cast<uint64_t>(lim.k) <= all_tokens;
      if (has_k && holds(lim.k)) s.weight = place_of(lim.k).sum;
      __syncthreads();
      const bool known = lim.p >= 1.0 || has_k || lim.k == V || ends;
      const double share = lim.p * (has_k ? s.weight : ends ? all_weight : all);
      uint64_t n = has_k ? static_cast<uint64_t>(lim.k) : ~uint64_t{0};
      if (lim.p < 1.0) {
        const int owner = row_min(tokens > 0 && mass >= share ? tid : kRow, s.sums.i);
        if (tid == owner) {
          uint64_t run = upto - tokens, reached = 0;
          double x = mass - weight;
          for (int at = at0; at < at1 && reached == 0; ++at) {
            const uint64_t c = s.count[at];
            if (c == 0) continue;
            const double w = weigh(logit_of(value_key(at)));
            if (x + c * w >= share)
              reached = run + (x < share ? min(c, static_cast<uint64_t>(fmax(ceil((share - x) / w), 1.0))) : 1);
            x += c * w;
            run += c;
          }
          s.found = reached ? reached : run;     // (the run's own sum may round below the share)
        }
        __syncthreads();
        if (owner < kRow) n = min(n, s.found);
        __syncthreads();
      }
      if (lim.m > 0.0) {
        // Values from key_m on, and how many tokens have them.
        const uint32_t v = (key_m >> 16) + (key_m >= 0x80000000u && (key_m & 0xFFFFu) ? 1 : 0);
        const int stay = static_cast<int>(first - v) + 1;
        if (stay < values) {
          if (tid == 0) s.above = all_tokens;
          __syncthreads();
          if (stay >= at0 && stay < at1) {
            uint64_t run = upto - tokens;
            for (int at = at0; at < stay; ++at) run += s.count[at];
            s.above = run;
          }
          __syncthreads();
          n = min(n, s.above);
          __syncthreads();
        }
      }
      if (known && (n <= all_tokens || ends)) {
        if (n > all_tokens) {
          if (tid == 0) *out = RowInfo{top, all_weight, order_of(cut, 0x7FFFFFFF), -1, 0};
          return;
        }
        if (holds(n)) {
          const Place p = place_of(n);
          s.found = p.at;
          s.above = p.last ? 0 : p.nth;
          s.weight = p.sum;
        }
        __syncthreads();
        const uint32_t key = value_key(static_cast<int>(s.found));
        const uint64_t nth = s.above;
        const double sum = s.weight;
        __syncthreads();
        const int index = nth ? nth_of_key(logits, V, key, nth, s) : 0x7FFFFFFF;
        if (tid == 0) *out = RowInfo{top, sum, order_of(key, index), -1, 0};
        return;
      }
    }
  }
  // Weights as whole numbers: at most 2^62 over all that can stay, whose sum is
  // `all` or below kSmallK. They are off by half each, V 2^-51 of the sum at
  // most.
  const int shift = small ? 50 : min(50, 61 - ilogb(fmax(all, 1.0)));
  const WholeWeigher amount(top, lim.tau, shift);
  const float least = hard ? top : logit_of(cut);
  uint64_t border = order_of(kLeastKey, 0x7FFFFFFF);     // everything that can have a weight
  uint64_t stay = 0;
  bool summed = false;
  if (lim.k < V) {
    const Border b = select_border(
        logits, V, top, least, -1.0, static_cast<uint64_t>(lim.k), [](uint32_t k, int) { return k >= kLeastKey; },
        [&](float z) { return z >= least ? uint64_t{1} : uint64_t{0}; }, s);
    border = max(border, b.order);
  }
  auto stays = [&](uint32_t k, int i) { return order_of(k, i) >= border; };
  if (lim.p < 1.0) {
    const Border b = select_border(logits, V, top, least, lim.p, 0, stays, amount, s);
    border = max(border, b.order);
    stay = b.sum;
    summed = true;
  }
  if (lim.m > 0.0 && order_of(key_m, 0x7FFFFFFF) > border) {
    border = order_of(key_m, 0x7FFFFFFF);
    summed = false;
  }
  if (!summed) {
    uint64_t x = 0;
    each_slice(logits, V, [&](int e, const float* z) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x += stays(key_of(z[i]), e + i) ? amount(z[i]) : 0;
    });
    row_scan(x, s.sums.u, &stay);
  }
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
  constexpr int kPer = kTokens / kThreads;
  double plain[kPer], x[kPer], sum = 0.0, whole = 0.0;
  int token[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int at = threadIdx.x * kPer + i;
    const uint64_t e = at < ri.n ? a.kept[row * kTokens + at] : 0;
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

// 3. Grid: (group of pieces, request). The request's last block to have summed its piece
// goes on to the draw (counted in memory; sums are added in the pieces' order
// whoever it is).
template <typename T, typename Args>
__global__ __launch_bounds__(kThreads) void filter_node_kernel(const Args args) {
  __shared__ WalkLds w;
  __shared__ double lds[kThreads / 64];
  __shared__ int32_t ilds[kThreads / 64];
  __shared__ int32_t pick;
  const int group = blockIdx.x, rl = blockIdx.y, r = args.req0 + rl;
  if (group == 0 && r == 0 && args.status) {
    int bad = 0;
    for (int i = threadIdx.x; i < args.n_req; i += kThreads) bad += bad_temperature(temperature_of(args, i));
    const double all = block_reduce(bad, add, lds);
    if (threadIdx.x == 0) *args.status = static_cast<int32_t>(all);
  }
  walk<T>(args, rl, group == 0, w);
  if (w.info.bad) return;
  const RowInfo ri = args.rows[static_cast<int64_t>(r) * args.n_pos + w.info.node];
  const double u = args.uniforms[static_cast<int64_t>(r) * args.n_pos];
  if (ri.n >= 0) {
    if (group != 0) return;
    const int token = draw_listed(args, w.info, ri, r, u, lds, ilds);
    if (threadIdx.x == 0) args.bonus[r] = token;
    return;
  }
  double x[8], plain[kGroup], sum[kGroup];
#pragma unroll
  for (int i = 0; i < kGroup; ++i)
    sum[i] = filtered_weights<T>(args, w.info, ri, w.info.mode, r, min(group * kGroup + i, args.n_pieces - 1), x, &plain[i]);
#pragma unroll
  for (int i = 0; i < kGroup; ++i) {
    sum[i] = block_reduce(sum[i], add, lds);
    plain[i] = block_reduce(plain[i], add, lds);
  }
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (group * kGroup + i < args.n_pieces)
        args.part[static_cast<int64_t>(r) * args.n_pieces + group * kGroup + i] = double2{sum[i], plain[i]};
    pick = __hip_atomic_fetch_add(&args.done[r], 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (pick != static_cast<int>(gridDim.x) - 1) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  const Pieces<double2> part(args.part + static_cast<int64_t>(r) * args.n_pieces, args.n_pieces);
  int mode = w.info.mode;
  Found f = find_piece(part, [](double2 y) { return y.x; }, u);
  if (f.piece < 0 && mode != kPlain) {   // nothing is left over: the row itself
    mode = kPlain;
    f = find_piece(part, [](double2 y) { return y.y; }, u);
  }
  __syncthreads();
  if (threadIdx.x == 0) pick = 0;
  if (f.piece >= 0) {
    const double mine = filtered_weights<T>(args, w.info, ri, mode, r, f.piece, x, plain);
    const double c = f.before + block_scan(mine, lds);
    const double target = u * f.total;
    int owner = first_hit(mine > 0.0 && c > target, ilds);
    const bool passes = owner < kThreads;
    if (!passes) owner = last_hit(mine > 0.0, ilds);
    if (static_cast<int>(threadIdx.x) == owner) {
      double run = c - mine;
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
  char* const p3 = place(rows * kTokens * sizeof(uint64_t));
  char* const p4 = place(d->n_req * pieces * sizeof(double2));
  char* const p5 = place(d->n_req * sizeof(int32_t));
  if (args) {
    args->chunks = reinterpret_cast<ChunkInfo*>(p0);
    args->lists = reinterpret_cast<uint64_t*>(p1);
    args->rows = reinterpret_cast<RowInfo*>(p2);
    args->kept = reinterpret_cast<uint64_t*>(p3);
    args->part = reinterpret_cast<double2*>(p4);
    args->done = reinterpret_cast<int32_t*>(p5);
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
      hipLaunchKernelGGL((filter_node_kernel<T, FilterTree>), dim3((args.n_pieces + kGroup - 1) / kGroup, n), dim3(kThreads), 0, s, tree_args);
    else
      hipLaunchKernelGGL((filter_node_kernel<T, FilterArgs>), dim3((args.n_pieces + kGroup - 1) / kGroup, n), dim3(kThreads), 0, s, args);
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
  args.stats = nullptr; args.rest = nullptr; args.info = nullptr;
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
