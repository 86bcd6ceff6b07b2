// The next token of each row of logits, by temperature, top-k, min-p and top-p.
//
// With x_i = (l_i - max l) / temperature and w_i = e^(x_i), the tokens that remain are a
// prefix of the descending order (ties to the lower id): the top_k first ones, of those
// the ones with w_i >= min_p, and of those the shortest prefix whose weights sum to at
// least top_p of the sum of all of them. The drawn token is the first one in ascending
// order of ids whose running sum exceeds u times the sum of what remains.
//
// Every comparison is one of sums of many weights, and a token whose side of it
// changes with a rounding would change with the order of the sum. So the weights are
// worked out in fp64 and rounded once to whole multiples of 2^-42 of the largest one;
// their sums are sums of 64-bit integers, exact (a row has at most 2^20 tokens) and the
// same in any order.
//
// The first pass over a row finds its maximum. The second puts every weight (or, for top-k
// alone, every token) into a histogram over x, 64 bins to the unit, from which the
// running sums at the bins' edges follow. The third collects the tokens of the few bins in
// which a filter cuts, and sums what surely remains in segments of 512 tokens; the cut is
// found among the collected ones by dividing the range of their places in the order, and what
// remains of them is added to the segments. A cut in a bin of too many tokens (flat rows, many
// equal logits) is found by a radix descent over the row.
//
// Long rows are bound by vector work: 256 rows of 151643 bf16 logits by top-p 118 us (maximum 14,
// histogram 40, collection 45, cut and draw 17; their bytes once, 15). Short ones by the latency
// of one pass behind the other: 4 rows of 32000 by all filters 29 us. Rows that need the descent take
// its passes over the row, by one workgroup each: nearly flat rows by top-p 130 us (4 of 32000), 450 (64
// of 128000) and 620 (256 of 151643), by top-k and top-p 200, 750 and 1040; by temperature alone any row
// takes two passes (19, 25 and 67 us).
//
// Many rows: one workgroup each, all in one launch. Few: several workgroups each, a launch
// a pass, the last one to finish the third pass drawing the token. The sums being exact,
// both give the same bits.
#include <algorithm>

#include "misa_common.hpp"
#include "misa_evict.hpp"

namespace misa {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;             // of 1 / 64 each: weights below e^-32 round to 0
constexpr int kSeg = 512;               // tokens of a segment: 8 a lane
constexpr int kMaxSegs = kMaxVocab / kSeg;
static_assert(kMaxSegs == kBins && kBins == 2 * kThreads, "the running sums take two entries a thread");
constexpr int kList = 4096;             // tokens of the bins with a cut, at most
constexpr int kOne = 42;                // a weight of 1 is 2^kOne

typedef unsigned long long u64;

template <int TYPE>
__device__ __forceinline__ float logit_of(uint32_t bits) {   // 16 bits, or 32
  if (TYPE == 1) return __uint_as_float(bits << 16);
  if (TYPE == 2) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  return __uint_as_float(bits);
}

// What a row is sampled by.
struct Row {
  const void* logits;
  int V;
  float top;            // largest logit (0 where that is infinite, and all others -inf)
  bool inf;             // it is infinite: such logits stand for 0, all others for -inf
  float lift;           // depth_of's first factor, and
  float high, fine;     // top times it; 64 / temperature by it
  double inv;           // log2(e) / temperature
  double min_w;         // least weight, in units of 2^-kOne
  int top_k;            // 0: all
  bool by_sum;          // top-p cuts
  double share;
  __device__ __forceinline__ bool filtered() const { return top_k || by_sum; }
};

typedef u32x4 __attribute__((aligned(2))) u32x4_any;

// Eight neighbouring logits of a row on their way.
template <int TYPE>
struct Raw {
  u32x4 x[TYPE == 3 ? 2 : 1];
  __device__ __forceinline__ void load(const void* row, int i) {
    if (TYPE == 3) {
      x[0] = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(row) + i);
      x[TYPE == 3] = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(row) + i + 4);
    } else {
      x[0] = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(row) + i);
    }
  }
  __device__ __forceinline__ void get(float (&l)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      l[j] = TYPE == 3 ? __uint_as_float(x[j >> 2][j & 3])
                       : logit_of<TYPE>(j & 1 ? x[0][j >> 1] >> 16 : x[0][j >> 1] & 0xffffu);
  }
};
__device__ __forceinline__ float logit(const Row& r, float l) {
  return r.inf ? (l == __builtin_inff() ? 0.f : -__builtin_inff()) : l;
}

// How far below the maximum, in bins: 64 (top - l) / temperature. The order of logits is kept
// (every step rounds monotonically), no finite logit overflows, and NaN and -inf give no number
// below kBins. What lies below kBins deep has an exponent above -47 in units of log2, which
// weights_of relies on.
__device__ __forceinline__ float depth_of(const Row& r, float l) { return __builtin_fmaf(l, -r.lift, r.high) * r.fine; }

// 2^t in units of 2^-kOne, of two numbers t <= 0 at a time. 2^f of the rest |f| <= 1/2 is 1 + f
// times the polynomial through (2^f - 1) / f at the zeros of a Chebyshev polynomial (degree 10
// in all, 6e-16 off). The two run side by side, with the constants in scalar registers: left to
// itself the compiler copies every constant into vector registers before it is used up there,
// and does one number after the other, each step waiting for the one before.
struct Two {
  double a, b;
};
__device__ __forceinline__ Two weights_of(double t0, double t1) {
  const double magic = 6755399441055744.0;     // 1.5 2^52: to the next integer
  const double whole0 = t0 + magic, whole1 = t1 + magic, f0 = t0 - (whole0 - magic), f1 = t1 - (whole1 - magic);
  double p0, p1;
  asm("v_fma_f64 %0, %4, %2, %5\n\tv_fma_f64 %1, %4, %3, %5\n\t"
      "v_fma_f64 %0, %0, %2, %6\n\tv_fma_f64 %1, %1, %3, %6\n\t"
      "v_fma_f64 %0, %0, %2, %7\n\tv_fma_f64 %1, %1, %3, %7\n\t"
      "v_fma_f64 %0, %0, %2, %8\n\tv_fma_f64 %1, %1, %3, %8\n\t"
      "v_fma_f64 %0, %0, %2, %9\n\tv_fma_f64 %1, %1, %3, %9\n\t"
      "v_fma_f64 %0, %0, %2, %10\n\tv_fma_f64 %1, %1, %3, %10\n\t"
      "v_fma_f64 %0, %0, %2, %11\n\tv_fma_f64 %1, %1, %3, %11\n\t"
      "v_fma_f64 %0, %0, %2, %12\n\tv_fma_f64 %1, %1, %3, %12\n\t"
      "v_fma_f64 %0, %0, %2, %13\n\tv_fma_f64 %1, %1, %3, %13\n\t"
      "v_fma_f64 %0, %0, %2, 1.0\n\tv_fma_f64 %1, %1, %3, 1.0"
      : "=&v"(p0), "=&v"(p1)
      : "v"(f0), "v"(f1), "v"(7.070976083807186e-09), "s"(1.0205905476607851e-07), "s"(1.3215451644483806e-06),
        "s"(1.525267292453816e-05), "s"(0.00015403530424751012), "s"(0.0013333558200795041), "s"(0.00961812910761869),
        "s"(0.05550410866465167), "s"(0.24022650695910075), "s"(0.6931471805599462));
  const int n0 = (int)__builtin_bit_cast(u64, whole0), n1 = (int)__builtin_bit_cast(u64, whole1);
  return {p0 * __builtin_bit_cast(double, (u64)(uint32_t)(n0 + kOne + 1023) << 52),
          p1 * __builtin_bit_cast(double, (u64)(uint32_t)(n1 + kOne + 1023) << 52)};
}
__device__ __forceinline__ double exponent(const Row& r, float l) { return ((double)l - (double)r.top) * r.inv; }
// The weights of two logits that are less than kBins deep, to the nearest whole number; 0
// where min_p drops them. As numbers in fp64, and as integers.
__device__ __forceinline__ Two rounded(const Row& r, float l0, float l1) {
  const Two w = weights_of(exponent(r, l0), exponent(r, l1));
  const double magic = 4503599627370496.0;     // 2^52
  const double y0 = (w.a + magic) - magic, y1 = (w.b + magic) - magic;
  return {w.a < r.min_w ? 0.0 : y0, w.b < r.min_w ? 0.0 : y1};
}
__device__ __forceinline__ void weights(const Row& r, float l0, float l1, u64& y0, u64& y1) {
  const Two w = weights_of(exponent(r, l0), exponent(r, l1));
  y0 = w.a < r.min_w ? 0 : __builtin_bit_cast(u64, w.a + 4503599627370496.0) & 0xfffffffffffffull;
  y1 = w.b < r.min_w ? 0 : __builtin_bit_cast(u64, w.b + 4503599627370496.0) & 0xfffffffffffffull;
}
__device__ __forceinline__ u64 weight(const Row& r, float l) {
  u64 y, same;
  weights(r, l, l, y, same);
  return y;
}

// Data-parallel moves within rows of 16 lanes (0x110 + n: from n lanes below) and from row to
// row (0x142: lane 15 to the next row, 0x143: lane 31 to the upper half). Lanes without a source
// get `none`. Sums and scans over a wave by these take a fifth of the time of shuffles
// through LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 dpp(u64 none, u64 v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp((int)(uint32_t)none, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp((int)(none >> 32), (int)(v >> 32), CTRL, ROWS, 0xf, false);
  return (u64)hi << 32 | lo;
}
// op(op(first lane, second), ...) up to and with each lane; of all in lane 63.
template <typename Op>
__device__ __forceinline__ u64 scan_wave(u64 none, u64 v, Op op) {
  v = op(v, dpp<0x111, 0xf>(none, v));
  v = op(v, dpp<0x112, 0xf>(none, v));
  v = op(v, dpp<0x114, 0xf>(none, v));
  v = op(v, dpp<0x118, 0xf>(none, v));
  v = op(v, dpp<0x142, 0xa>(none, v));
  return op(v, dpp<0x143, 0xc>(none, v));
}
// The sum of a whole number below 2^47 per lane, in lane 63.
__device__ __forceinline__ double wave_total(double v) {
  auto add = [](u64 x, u64 y) {
    return __builtin_bit_cast(u64, __builtin_bit_cast(double, x) + __builtin_bit_cast(double, y));
  };
  return __builtin_bit_cast(double, scan_wave(0, __builtin_bit_cast(u64, v), add));
}

// Tokens in descending order: larger logit first, then the lower id. 0: none (NaN).
__device__ __forceinline__ u64 order_of(float l, int i) {
  return l != l ? 0 : (u64)score_key(l) << 20 | (u64)(kMaxVocab - 1 - i);
}
__device__ __forceinline__ int id_of(u64 order) { return kMaxVocab - 1 - (int)(order & (kMaxVocab - 1)); }
__device__ __forceinline__ float logit_of_order(u64 order) { return key_score((uint32_t)(order >> 20)); }

// A workgroup's share of LDS.
struct Shared {
  u64 bins[2][kBins];       // number and sum of weights of the tokens of a bin, then of the bins up to and with it
  u64 list[kList];          // tokens of the bins with a cut
  u64 seg[kMaxSegs];        // sums of the weights that remain, by segment
  u64 near[64];
  u64 slots[kWaves];
  u64 found[3];
  uint32_t n;
  Row row;
};
__device__ __forceinline__ Shared& lds() {
  __shared__ Shared s;
  return s;
}
constexpr int kCount = 0, kMass = 1, kSegments = 2;
__device__ __forceinline__ u64* bins_of(int which) {
  return which == kSegments ? lds().seg : lds().bins[which];
}

// What is done once a row stands in functions of its own: a row passes through it once, so
// its instructions come from memory each time (inlined and unrolled the kernel had 45 KB of code, and
// four rows of 32000 tokens took 41 us instead of 29).
#define MISA_ONCE __attribute__((noinline))

// Inclusive sum of a value per thread, in thread order.
__device__ MISA_ONCE u64 scan_block(u64 v) {
  Shared& s = lds();
  const int wave = threadIdx.x >> 6;
  v = scan_wave(0, v, [](u64 x, u64 y) { return x + y; });
  __syncthreads();
  if ((threadIdx.x & 63) == 63) s.slots[wave] = v;
  __syncthreads();
  u64 before = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) before += i < wave ? s.slots[i] : 0;
  return before + v;
}

// Running sums over the bins, in place: thread i owns bins 2 i and 2 i + 1.
__device__ MISA_ONCE void scan_bins(int which) {
  u64* bins = bins_of(which);
  __syncthreads();
  const u64 a = bins[2 * threadIdx.x], b = bins[2 * threadIdx.x + 1];
  const u64 incl = scan_block(a + b);
  bins[2 * threadIdx.x] = incl - b;
  bins[2 * threadIdx.x + 1] = incl;
  __syncthreads();
}

// First bin whose running sum is at least `target` (kBins: none).
__device__ MISA_ONCE int first_bin(int which, u64 target) {
  Shared& s = lds();
  const u64* bins = bins_of(which);
  const u64 z = threadIdx.x ? bins[2 * threadIdx.x - 1] : 0, a = bins[2 * threadIdx.x], b = bins[2 * threadIdx.x + 1];
  if (bins[kBins - 1] < target) return kBins;
  if (z < target && b >= target) s.n = 2 * threadIdx.x + (a < target);
  __syncthreads();
  const int bin = __builtin_amdgcn_readfirstlane((int)s.n);
  __syncthreads();
  return bin;
}

__device__ __forceinline__ u64 upto(int which, int bin) { return bin > 0 ? bins_of(which)[bin - 1] : 0; }

__device__ __forceinline__ u64 share_of(double share, u64 total) {     // least sum that is `share` of the total
  const double x = __builtin_ceil(share * (double)total);
  return x < 1.0 ? 1 : (x >= (double)total ? total : (u64)x);
}

__device__ MISA_ONCE void clear_bins() {
#pragma unroll 1
  for (int i = threadIdx.x; i < 2 * kBins; i += kThreads) lds().bins[0][i] = 0;
}

__device__ __forceinline__ bool in_bins(const Row& r, float l, int b0, int b1) {
  const float d = depth_of(r, l);
  return d >= (float)b0 && d < (float)(b1 + 1);
}

// Of the n listed tokens of bins [b0, b1] with an order in [lo, hi]: least and largest order in
// found[0] and [1], their number is returned.
__device__ MISA_ONCE uint32_t range_of(int n, int b0, int b1, u64 lo, u64 hi) {
  Shared& s = lds();
  const Row r = s.row;
  __syncthreads();
  if (threadIdx.x == 0) {
    s.found[0] = ~0ull;
    s.found[1] = 0;
    s.n = 0;
  }
  __syncthreads();
  u64 least = ~0ull, most = 0;
  uint32_t here = 0;
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const u64 o = s.list[i];
    if (o >= lo && o <= hi && in_bins(r, logit_of_order(o), b0, b1)) {
      least = min(least, o);
      most = max(most, o);
      ++here;
    }
  }
  if (__ballot(here != 0)) {
    least = ~scan_wave(0, ~least, [](u64 x, u64 y) { return max(x, y); });
    most = scan_wave(0, most, [](u64 x, u64 y) { return max(x, y); });
    here = (uint32_t)scan_wave(0, here, [](u64 x, u64 y) { return x + y; });
    if ((threadIdx.x & 63) == 63) {
      atomicMin(&s.found[0], least);
      atomicMax(&s.found[1], most);
      atomicAdd(&s.n, here);
    }
  }
  __syncthreads();
  const uint32_t all = __builtin_amdgcn_readfirstlane(s.n);
  __syncthreads();
  return all;
}

__device__ __forceinline__ u64 lane_of(u64 v, int lane) {
  return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
}

// The cut among the n listed tokens of bins [b0, b1]: the one, in the order, at which the
// running count (or sum of weights), which starts at `base`, reaches `target`. found[2]
// gets the running sum of weights there, from `sum` before those bins. The range of the tokens
// in question is divided into 2048 equal parts, until at most 64 are left: once where
// logits differ, twice where ids decide.
__device__ MISA_ONCE u64 cut_list(int n, int b0, int b1, int by, u64 base, u64 target, u64 sum) {
  Shared& s = lds();
  const Row r = s.row;
  uint32_t here = range_of(n, b0, b1, 0, ~0ull);
  u64 least = s.found[0], most = s.found[1];
  while (here > 64) {
    clear_bins();
    const int shift = max(0, 53 - __builtin_clzll(most - least));    // 2048 parts at most
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const u64 o = s.list[i];
      if (o >= least && o <= most) {
        const int part = (int)((most - o) >> shift);
        atomicAdd(&s.bins[kCount][part], (u64)1);
        atomicAdd(&s.bins[kMass][part], weight(r, logit_of_order(o)));
      }
    }
    scan_bins(kCount);
    scan_bins(kMass);
    const int part = min(first_bin(by, target - base), kBins - 1);
    base += upto(by, part);
    sum += upto(kMass, part);
    const u64 hi = most - ((u64)part << shift), width = (u64)1 << shift;
    here = range_of(n, b0, b1, hi - least >= width ? hi - width + 1 : least, hi);
    least = s.found[0];
    most = s.found[1];
  }
  __syncthreads();
  if (threadIdx.x == 0) s.n = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const u64 o = s.list[i];
    if (o >= least && o <= most) s.near[atomicAdd(&s.n, 1u)] = o;
  }
  __syncthreads();
  if (threadIdx.x < 64) {       // each lane sums what lies at or before its token
    const u64 mine = threadIdx.x < here ? s.near[threadIdx.x] : 0;
    const u64 w = weight(r, logit_of_order(mine));
    u64 c = 0, m = 0;
#pragma unroll 1
    for (uint32_t i = 0; i < here; ++i) {
      const u64 other = lane_of(mine, (int)i), v = lane_of(w, (int)i);
      if (other >= mine) {
        ++c;
        m += v;
      }
    }
    const u64 at = base + (by == kMass ? m : c);
    if (mine && at >= target && at - (by == kMass ? w : 1) < target) {
      s.found[0] = mine;
      s.found[2] = sum + m;
    }
  }
  __syncthreads();
  return s.found[0];
}

template <int TYPE>
struct Sampler {
  const SampleArgs& a;
  int64_t row;
  int g0, g1;               // segments of this workgroup
  Row r;

  __device__ __forceinline__ Sampler(const SampleArgs& a_, int64_t row_, int part, int parts) : a(a_), row(row_) {
    const int nseg = (a.V + kSeg - 1) / kSeg, per = (nseg + parts - 1) / parts;
    g0 = min(part * per, nseg);
    g1 = min(g0 + per, nseg);
    r.logits = static_cast<const char*>(a.logits) + row * a.row_stride * (TYPE == 3 ? 4 : 2);
    r.V = a.V;
    r.inf = false;
  }

  __device__ __forceinline__ static float load1(const Row& r, int i) {
    return TYPE == 3 ? static_cast<const float*>(r.logits)[i] : logit_of<TYPE>(static_cast<const uint16_t*>(r.logits)[i]);
  }

  // f(segment, token, logits as logit() has them) for 8 neighbouring tokens a lane, a segment a wave; the next
  // segment on its way
  template <typename F>
  __device__ __forceinline__ static void each(const Row& r, int from, int to, F f) {
    const int lane8 = 8 * (threadIdx.x & 63), full = min(to, r.V / kSeg);
    int g = from + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    float l[8];
    Raw<TYPE> now, next;
    if (g < full) now.load(r.logits, g * kSeg + lane8);
    for (; g < to; g += kWaves) {
      if (g < full) {
        next.load(r.logits, min(g + kWaves, full - 1) * kSeg + lane8);
        now.get(l);
        now = next;
      } else {                        // the last segment of the row; -inf behind its end
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = g * kSeg + lane8 + j;
          const float x = load1(r, min(i, r.V - 1));
          l[j] = i < r.V ? x : -__builtin_inff();
        }
      }
      if (r.inf) {
#pragma unroll
        for (int j = 0; j < 8; ++j) l[j] = logit(r, l[j]);
      }
      f(g, g * kSeg + lane8, l);
    }
  }

  // The largest logit of this workgroup's segments (-inf: none; NaN is passed over, and by
  // comparisons: the maximum instruction gives NaN for a signalling one, and loses what came before).
  __device__ __forceinline__ float find_top() {
    float top = -__builtin_inff();
    each(r, g0, g1, [&](int, int, const float* l) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) top = l[j] > top ? l[j] : top;
    });
#pragma unroll
    for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    Shared& s = lds();
    if ((threadIdx.x & 63) == 0) s.slots[threadIdx.x >> 6] = __float_as_uint(top);
    __syncthreads();
    top = __uint_as_float((uint32_t)s.slots[threadIdx.x & (kWaves - 1)]);
#pragma unroll
    for (int off = kWaves / 2; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    __syncthreads();
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top)));
  }

  // What the row asks for. false: there is nothing to choose, and the token is written if
  // this workgroup is to.
  __device__ __forceinline__ bool set_up(float top, bool writes) {
    const float temperature = a.temperature ? a.temperature[row] : 1.f;
    if (top == -__builtin_inff() || !(temperature > 0.f)) {
      if (writes) {             // the first of the largest logits, or -1
        Shared& s = lds();
        if (threadIdx.x == 0) s.n = 0xffffffffu;
        __syncthreads();
        if (top != -__builtin_inff()) {
#pragma unroll 1
          for (int i = threadIdx.x; i < r.V; i += kThreads)
            if (load1(r, i) == top) {
              atomicMin(&s.n, (uint32_t)i);
              break;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
          a.token[row] = (int)s.n;
          if (a.logprob) a.logprob[row] = s.n == 0xffffffffu ? -__builtin_inff() : 0.f;
        }
      }
      return false;
    }
    r.inf = top == __builtin_inff();
    r.top = r.inf ? 0.f : top;
    // Differences are halved, so that they do not overflow, and scaled. Temperatures below
    // 2^-120 want a factor beyond fp32. Of a largest logit of 2^-40 and more all different
    // ones are then far below it (2^-65 at least) by any factor; around smaller ones
    // differences are lifted first: exact for the largest, and infinite only for logits far below.
    const bool tiny = temperature < 0x1p-120f, near = tiny && fabsf(r.top) < 0x1p-40f;
    r.lift = near ? 0x1p60f : 0.5f;
    r.high = r.lift * r.top;
    r.fine = near ? (float)(0x1p-54 / (double)temperature) : tiny ? 0x1p127f : 128.f / temperature;
    r.inv = 1.4426950408889634 / (double)temperature;
    const float min_p = a.min_p ? a.min_p[row] : 0.f;
    r.min_w = min_p > 0.f ? (double)fminf(min_p, 1.f) * (double)(1ull << kOne) : 0.0;
    const int k = a.top_k ? a.top_k[row] : 0;
    r.top_k = k > 0 && k < r.V ? k : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f;
    r.by_sum = p < 1.f;
    r.share = p > 0.f ? (double)p : 0.0;
    if (threadIdx.x == 0) lds().row = r;
    return true;
  }

  // The histogram of this workgroup's segments.
  __device__ __forceinline__ void fill_bins() {
    Shared& s = lds();
    clear_bins();
    __syncthreads();
    each(r, g0, g1, [&](int, int, const float* l) __attribute__((always_inline)) {
      float d[8];
      u64 w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = depth_of(r, l[j]);
      if (r.top_k) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (d[j] < (float)kBins) atomicAdd(&s.bins[kCount][(int)d[j]], (u64)1);
      }
      if (r.by_sum) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) weights(r, l[j], l[j + 1], w[j], w[j + 1]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (d[j] < (float)kBins) atomicAdd(&s.bins[kMass][(int)d[j]], w[j]);
      }
    });
  }

  int bk, p0, p1;           // the bin of the k-th token (kBins: none); the bins that may hold top-p's last one
  // Running sums over the bins, and where the filters cut.
  __device__ __forceinline__ void find_bins() {
    bk = p0 = kBins;
    p1 = -1;
    if (r.top_k) {
      scan_bins(kCount);
      bk = first_bin(kCount, (u64)r.top_k);
    }
    if (r.by_sum) {
      scan_bins(kMass);
      const u64 most = upto(kMass, min(bk + 1, kBins)), least = bk < kBins ? upto(kMass, bk) : most;
      p0 = min(bk, first_bin(kMass, share_of(r.share, max(least, (u64)1))));
      p1 = least == most ? p0 : min(bk, first_bin(kMass, share_of(r.share, most)));
    }
  }

  // The tokens of the bins with a cut into the list (s.n of them; those beyond kList are
  // only counted), and the segments' sums of what lies above those bins.
  __device__ __forceinline__ void collect() {
    Shared& s = lds();
    __syncthreads();
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    const float sure = (float)min(bk, p0);                   // bins below it remain whole
    const float k0 = (float)bk, k1 = bk < kBins ? k0 + 1.f : k0, q0 = (float)p0, q1 = (float)(p1 + 1);
    each(r, g0, g1, [&](int g, int i, const float* l) __attribute__((always_inline)) {
      float d[8], least = __builtin_inff();
      uint32_t cut = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = depth_of(r, l[j]);
        least = fminf(least, d[j]);
        cut = (d[j] >= k0 && d[j] < k1) || (d[j] >= q0 && d[j] < q1) ? cut | 1u << j : cut;
      }
      double sum = 0.0;            // whole numbers below 2^53
      if (__ballot(least < sure)) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const Two w = rounded(r, l[j], l[j + 1]);
          sum += (d[j] < sure ? w.a : 0.0) + (d[j + 1] < sure ? w.b : 0.0);
        }
        sum = wave_total(sum);
      }
      if ((threadIdx.x & 63) == 63) s.seg[g] = (u64)sum;
      // few of a segment's, one a lane at a time (a ballot and an atomic for each of the eight:
      // 256 rows of 151643 tokens 127 us, like this 122; one place for a segment's, 136)
      while (__ballot(cut != 0)) {
        if (cut) {
          const int j = __builtin_ctz(cut);
          float x = l[0];
#pragma unroll
          for (int q = 1; q < 8; ++q) x = q == j ? l[q] : x;
          const uint32_t at = atomicAdd(&s.n, 1u);
          if (at < kList) s.list[at] = order_of(x, i + j);
          cut &= cut - 1;
        }
      }
    });
    __syncthreads();
  }

  // The last kept token's place in the order, among the n listed ones; what remains of them
  // is added to the segments' sums.
  __device__ __forceinline__ u64 cut_lists(int n) {
    Shared& s = lds();
    u64 total = r.by_sum ? s.bins[kMass][kBins - 1] : 0, cut = 0;
    const u64 before_p = r.by_sum ? upto(kMass, p0) : 0;
    if (bk < kBins) {
      cut = cut_list(n, bk, bk, kCount, upto(kCount, bk), (u64)r.top_k, upto(kMass, bk));
      total = s.found[2];
    }
    if (r.by_sum) cut = max(cut, cut_list(n, p0, p1, kMass, before_p, share_of(r.share, total), 0));
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const u64 o = s.list[i];
      if (o >= cut) atomicAdd(&s.seg[id_of(o) / kSeg], weight(r, logit_of_order(o)));
    }
    return cut;
  }

  // The cut among the tokens of bins [b0, b1] of the whole row, found digit by digit: the
  // token at which the running count (or sum of weights), which starts at `base`, reaches
  // `target`.
  __device__ __forceinline__ static u64 descend(const Row& r, int b0, int b1, int by, u64 base, u64 target) {
    Shared& s = lds();
    u64 prefix = 0;
#pragma unroll 1
    for (int shift = 44; shift >= 0; shift -= 11) {       // 5 digits of 11 bits for 32 + 20 bits
      __syncthreads();
      clear_bins();
      __syncthreads();
#pragma unroll 1
      for (int i = threadIdx.x; i < r.V; i += kThreads) {
        const float x = logit(r, load1(r, i));
        const u64 o = order_of(x, i);
        if (in_bins(r, x, b0, b1) && o >> (shift + 11) == prefix)
          atomicAdd(&s.bins[by][kBins - 1 - (int)(o >> shift & (kBins - 1))], by == kMass ? weight(r, x) : (u64)1);
      }
      scan_bins(by);
      const int d = min(first_bin(by, target - base), kBins - 1);
      base += upto(by, d);
      prefix = prefix << 11 | (u64)(kBins - 1 - d);
    }
    return prefix;
  }

  // The segments' sums of the tokens at or before the cut, of bins from b0 on; their sum.
  __device__ __forceinline__ static u64 sum_to(const Row& r, int b0, u64 cut) {
    Shared& s = lds();
    __syncthreads();
#pragma unroll 1
    for (int g = threadIdx.x; g < kMaxSegs; g += kThreads) s.seg[g] = 0;
    __syncthreads();
    u64 sum = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < r.V; i += kThreads) {
      const float x = logit(r, load1(r, i));
      if (in_bins(r, x, b0, kBins - 1) && order_of(x, i) >= cut) {
        const u64 w = weight(r, x);
        atomicAdd(&s.seg[i / kSeg], w);
        sum += w;
      }
    }
    const u64 incl = scan_block(sum);
    __syncthreads();
    if (threadIdx.x == kThreads - 1) s.found[2] = incl;
    __syncthreads();
    return s.found[2];
  }

  // More tokens share the bins with a cut than the list holds.
  __device__ MISA_ONCE static u64 cut_row(int bk) {
    const Row r = lds().row;
    u64 total = r.by_sum ? lds().bins[kMass][kBins - 1] : 0, cut = 0;
    if (bk < kBins) {
      const u64 upto_k = upto(kCount, bk), mass_k = upto(kMass, bk);
      cut = descend(r, bk, bk, kCount, upto_k, (u64)r.top_k);
      if (r.by_sum) total = mass_k + sum_to(r, bk, cut);
    }
    if (r.by_sum) cut = max(cut, descend(r, 0, kBins - 1, kMass, 0, share_of(r.share, total)));
    sum_to(r, 0, cut);
    return cut;
  }

  // The token, from the segments' sums of what remains.
  __device__ __forceinline__ void draw(u64 cut) {
    Shared& s = lds();
    scan_bins(kSegments);
    const u64 total = s.seg[kMaxSegs - 1];
    const float u = a.u[row];          // a product beyond 64 bits has no defined value
    u64 drawn = u > 0.f ? (u64)((double)fminf(u, 1.f) * (double)total) : 0;
    if (drawn >= total) drawn = total - 1;
    const int g = first_bin(kSegments, drawn + 1), i = g * kSeg + (int)threadIdx.x;
    const u64 before = upto(kSegments, g);
    float x = 0.f;
    u64 w = 0;
    if (threadIdx.x < kSeg && i < r.V) {
      x = logit(r, load1(r, i));
      if (depth_of(r, x) < (float)kBins && order_of(x, i) >= cut) w = weight(r, x);
    }
    const u64 run = before + scan_block(w);
    if (drawn < run && run - w <= drawn) {
      a.token[row] = i;
      if (a.logprob)
        a.logprob[row] =
            (float)(exponent(r, x) * 0.6931471805599453 - log((double)total * (1.0 / (double)(1ull << kOne))));
    }
  }
};

// One workgroup a row.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  Shared& s = lds();
  Sampler<TYPE> z(a, blockIdx.x, 0, 1);
  if (!z.set_up(z.find_top(), true)) return;
  for (int g = threadIdx.x; g < kMaxSegs; g += kThreads) s.seg[g] = 0;
  z.bk = z.p0 = kBins;
  z.p1 = -1;
  if (z.r.filtered()) {
    z.fill_bins();
    z.find_bins();
  }
  z.collect();
  u64 cut = 0;
  if (z.r.filtered()) {
    const uint32_t n = s.n;
    cut = n <= kList ? z.cut_lists((int)n) : Sampler<TYPE>::cut_row(z.bk);
  }
  z.draw(cut);
}

// ---------------------------------------------------------------- several workgroups a row
// Each takes a part of the segments. What they leave for the next launch, or for the last
// of them to finish:
struct Parts {
  float* top;               // [T][parts]
  uint32_t* listed;         // [T][parts] tokens of the bins with a cut
  uint32_t* done;           // [T] workgroups that have finished the last launch
  u64* seg;                 // [T][kMaxSegs]
  u64* bins;                // [T][parts][2][kBins]
  u64* list;                // [T][parts][kList]
  int parts;
};

template <int TYPE>
__global__ __launch_bounds__(kThreads) void top_kernel(SampleArgs a, Parts w) {
  const int row = blockIdx.x / w.parts, part = blockIdx.x % w.parts;
  Sampler<TYPE> z(a, row, part, w.parts);
  const float top = z.find_top();
  if (threadIdx.x == 0) {
    w.top[blockIdx.x] = top;
    if (part == 0) w.done[row] = 0;
  }
}

__device__ __forceinline__ float top_of(const Parts& w, int row) {
  float top = -__builtin_inff();
  for (int i = 0; i < w.parts; ++i) top = fmaxf(top, w.top[(int64_t)row * w.parts + i]);
  return top;
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void bins_kernel(SampleArgs a, Parts w) {
  const int row = blockIdx.x / w.parts, part = blockIdx.x % w.parts;
  Sampler<TYPE> z(a, row, part, w.parts);
  if (!z.set_up(top_of(w, row), false) || !z.r.filtered()) return;
  z.fill_bins();
  __syncthreads();
  u64* out = w.bins + (int64_t)blockIdx.x * 2 * kBins;
  for (int i = threadIdx.x; i < 2 * kBins; i += kThreads)
    if (i < kBins ? z.r.top_k != 0 : z.r.by_sum) out[i] = lds().bins[0][i];
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void draw_kernel(SampleArgs a, Parts w) {
  Shared& s = lds();
  const int row = blockIdx.x / w.parts, part = blockIdx.x % w.parts;
  Sampler<TYPE> z(a, row, part, w.parts);
  if (!z.set_up(top_of(w, row), part == 0)) return;
  z.bk = z.p0 = kBins;
  z.p1 = -1;
  if (z.r.filtered()) {
    const u64* in = w.bins + (int64_t)row * w.parts * 2 * kBins;
    for (int i = threadIdx.x; i < 2 * kBins; i += kThreads) {
      u64 v = 0;
      if (i < kBins ? z.r.top_k != 0 : z.r.by_sum) {
#pragma unroll 4
        for (int j = 0; j < w.parts; ++j) v += in[(int64_t)j * 2 * kBins + i];
      }
      s.bins[0][i] = v;
    }
    z.find_bins();
  }
  z.collect();
  // hand over: sums of the segments, listed tokens, their number
  u64* seg = w.seg + (int64_t)row * kMaxSegs;
  u64* list = w.list + (int64_t)row * w.parts * kList;
  const uint32_t mine = s.n;
  for (int g = z.g0 + (int)threadIdx.x; g < z.g1; g += kThreads) store_coherent((uint64_t*)seg + g, (uint64_t)s.seg[g]);
  for (int i = threadIdx.x; i < (int)min(mine, (uint32_t)kList); i += kThreads)
    store_coherent((uint64_t*)list + (int64_t)part * kList + i, (uint64_t)s.list[i]);
  if (threadIdx.x == 0) store_coherent(w.listed + blockIdx.x, mine);
  wait_stores();
  __syncthreads();
  if (threadIdx.x == 0) s.n = atomic_add_coherent(w.done + row, 1u);
  __syncthreads();
  if (s.n + 1 != (uint32_t)w.parts) return;
  // the last one has them all
  const int nseg = (a.V + kSeg - 1) / kSeg;
  for (int g = threadIdx.x; g < kMaxSegs; g += kThreads) s.seg[g] = g < nseg ? (u64)load_coherent((const uint64_t*)seg + g) : 0;
  uint32_t n = 0;
  for (int j = 0; j < w.parts; ++j) {
    const uint32_t m = load_coherent(w.listed + (int64_t)row * w.parts + j);
    if (n + m <= kList)
      for (uint32_t i = threadIdx.x; i < m; i += kThreads)
        s.list[n + i] = (u64)load_coherent((const uint64_t*)list + (int64_t)j * kList + i);
    n += m;
  }
  __syncthreads();
  u64 cut = 0;
  if (z.r.filtered()) cut = n <= kList ? z.cut_lists((int)n) : Sampler<TYPE>::cut_row(z.bk);
  z.draw(cut);
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Workgroups a row: one where the rows fill the chip (64 rows of 128000 tokens with four each
// 66 us, with one 97, with eight, whose workgroups then wait for each other, 92) or are short
// (4 rows of 32000 tokens 29 us with one, 31 with four). A workgroup has 16 waves, and a wave
// takes 512 tokens at a time.
int parts_of(int64_t T, int32_t V) {
  const int64_t room = 256 / T, most = (V + kSeg * kWaves - 1) / (kSeg * kWaves);
  if (room < 2 || most < 8) return 1;
  return (int)std::min<int64_t>({room, most, 32});
}

Parts carve(void* ws, int64_t T, int parts, size_t* bytes) {
  char* p = static_cast<char*>(ws);
  auto take = [&](size_t n) {
    char* q = p;
    p += round_up(n);
    return q;
  };
  Parts w{};
  w.parts = parts;
  w.top = reinterpret_cast<float*>(take((size_t)T * parts * sizeof(float)));
  w.listed = reinterpret_cast<uint32_t*>(take((size_t)T * parts * sizeof(uint32_t)));
  w.done = reinterpret_cast<uint32_t*>(take((size_t)T * sizeof(uint32_t)));
  w.seg = reinterpret_cast<u64*>(take((size_t)T * kMaxSegs * sizeof(u64)));
  w.bins = reinterpret_cast<u64*>(take((size_t)T * parts * 2 * kBins * sizeof(u64)));
  w.list = reinterpret_cast<u64*>(take((size_t)T * parts * kList * sizeof(u64)));
  *bytes = (size_t)(p - static_cast<char*>(ws));
  return w;
}

template <int TYPE>
void launch_type(const SampleArgs& a, void* ws, hipStream_t st) {
  const int parts = parts_of(a.T, a.V);
  if (parts == 1) {
    hipLaunchKernelGGL(sample_kernel<TYPE>, dim3((unsigned)a.T), dim3(kThreads), 0, st, a);
    return;
  }
  size_t bytes;
  const Parts w = carve(ws, a.T, parts, &bytes);
  const dim3 grid((unsigned)(a.T * parts));
  hipLaunchKernelGGL(top_kernel<TYPE>, grid, dim3(kThreads), 0, st, a, w);
  if (a.top_k || a.top_p) hipLaunchKernelGGL(bins_kernel<TYPE>, grid, dim3(kThreads), 0, st, a, w);
  hipLaunchKernelGGL(draw_kernel<TYPE>, grid, dim3(kThreads), 0, st, a, w);
}

}  // namespace

size_t sample_ws_bytes(int64_t T, int32_t V) {
  const int parts = parts_of(T, V);
  if (parts == 1) return 0;
  size_t bytes;
  carve(nullptr, T, parts, &bytes);
  return bytes;
}

hipError_t launch_sample(const SampleArgs& a, int type, void* ws, hipStream_t st) {
  if (type == 1) launch_type<1>(a, ws, st);
  else if (type == 2) launch_type<2>(a, ws, st);
  else launch_type<3>(a, ws, st);
  return hipGetLastError();
}

}  // namespace misa
