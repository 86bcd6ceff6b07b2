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
// One workgroup a row. Its first pass finds the maximum. The second puts every weight
// into a histogram over x, 64 bins to the unit, from which the running sums at the bins'
// edges follow. The last one collects the tokens of the few bins in which a filter
// cuts, sorts those, and sums what surely remains in segments of 512 tokens. A cut in
// a bin of too many tokens (flat rows, many equal logits) is found by a radix descent.
#include "misa_common.hpp"
#include "misa_evict.hpp"

namespace misa {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;             // of 1 / 64 each: all weights above e^-32
constexpr int kSeg = 512;               // tokens of a segment: 8 a lane
constexpr int kMaxSegs = kMaxVocab / kSeg;
static_assert(kMaxSegs == kBins && kBins == 2 * kThreads, "the running sums take two entries a thread");
constexpr int kList = 4096;             // tokens that are sorted
constexpr int kOne = 42;                // a weight of 1 is 2^kOne
constexpr double kLeast = -29.8;        // e^x rounds to 0 below (2^-43)

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
  float top;            // largest logit
  double inv;           // log2(e) / temperature
  double min_w;         // in units of 2^-kOne
};

template <int TYPE>
__device__ __forceinline__ float load_logit(const void* row, int i) {
  if (TYPE == 3) return static_cast<const float*>(row)[i];
  return logit_of<TYPE>(static_cast<const uint16_t*>(row)[i]);
}

typedef u32x4 __attribute__((aligned(2))) u32x4_any;

// Logits i .. i + 7 of a row; -inf behind its end.
template <int TYPE>
__device__ __forceinline__ void load8(const void* row, int i, int V, float (&l)[8]) {
  if (i + 8 <= V) {
    if (TYPE == 3) {
      const u32x4 a = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(row) + i);
      const u32x4 b = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(row) + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        l[j] = __uint_as_float(a[j]);
        l[4 + j] = __uint_as_float(b[j]);
      }
    } else {
      const u32x4 a = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(row) + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        l[2 * j] = logit_of<TYPE>(a[j] & 0xffffu);
        l[2 * j + 1] = logit_of<TYPE>(a[j] >> 16);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) l[j] = i + j < V ? load_logit<TYPE>(row, i + j) : -__builtin_inff();
  }
}

// x log2(e), 0 for the largest logit also where it is infinite. NaN for NaN.
__device__ __forceinline__ double exponent(const Row& r, float l) {
  return l == r.top ? 0.0 : ((double)l - (double)r.top) * r.inv;
}

// 2^t in units of 2^-kOne, to the nearest; t <= 0. 2^f of the rest |f| <= 1/2 by its
// Taylor polynomial of degree 11 (6e-15 off).
__device__ __forceinline__ double weight_of(double t) {
  const double n = __builtin_rint(t), f = t - n;
  double p = 4.4455382718708110e-10;            // ln(2)^k / k!
  p = __builtin_fma(p, f, 7.0549116208011225e-09);
  p = __builtin_fma(p, f, 1.0178086009239699e-07);
  p = __builtin_fma(p, f, 1.3215486790144309e-06);
  p = __builtin_fma(p, f, 1.5252733804059841e-05);
  p = __builtin_fma(p, f, 1.5403530393381608e-04);
  p = __builtin_fma(p, f, 1.3333558146428443e-03);
  p = __builtin_fma(p, f, 9.6181291076284770e-03);
  p = __builtin_fma(p, f, 5.5504108664821580e-02);
  p = __builtin_fma(p, f, 2.4022650695910072e-01);
  p = __builtin_fma(p, f, 6.9314718055994531e-01);
  p = __builtin_fma(p, f, 1.0);
  return p * __builtin_bit_cast(double, (u64)((int)n + kOne + 1023) << 52);
}
// A weight as an integer; 0 where min_p drops it, below the least one, and for NaN.
__device__ __forceinline__ u64 weight(const Row& r, double t) {
  if (!(t > kLeast * 1.4426950408889634)) return 0;
  const double w = weight_of(t);
  const u64 y = __builtin_bit_cast(u64, w + 4503599627370496.0) & 0xfffffffffffffull;   // 2^52
  return w >= r.min_w ? y : 0;
}
__device__ __forceinline__ int bin_of(double t) {      // t > kLeast log2(e)
  return min((int)(t * (-64.0 / 1.4426950408889634)), kBins - 1);
}

// Tokens in descending order: larger logit first, then the lower id. 0: none (NaN).
__device__ __forceinline__ u64 order_of(float l, int i) {
  return l != l ? 0 : (u64)score_key(l) << 20 | (u64)(kMaxVocab - 1 - i);
}
__device__ __forceinline__ int id_of(u64 order) { return kMaxVocab - 1 - (int)(order & (kMaxVocab - 1)); }
__device__ __forceinline__ float logit_of_order(u64 order) { return key_score((uint32_t)(order >> 20)); }

template <typename T>
__device__ __forceinline__ T scan_wave(T v) {     // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T x = __shfl_up(v, off, 64);
    if (lane >= off) v += x;
  }
  return v;
}

struct Shared {
  u64 mass[kBins];          // of a bin, then of the bins up to and with it
  uint32_t count[kBins];
  u64 list[kList];
  u64 seg[kMaxSegs];
  u64 slots[kWaves];
  u64 found[4];
  uint32_t n;
};

// Inclusive sum of a value per thread, in thread order.
template <typename T>
__device__ __forceinline__ T scan_block(T v, u64* slots) {
  const T incl = scan_wave(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) slots[threadIdx.x >> 6] = (u64)incl;
  __syncthreads();
  T before = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) before += i < (int)(threadIdx.x >> 6) ? (T)slots[i] : (T)0;
  return before + incl;
}

// Running sums over the bins, in place: thread i owns bins 2 i and 2 i + 1.
template <typename T>
__device__ __forceinline__ void scan_bins(T* bins, u64* slots) {
  const T a = bins[2 * threadIdx.x], b = bins[2 * threadIdx.x + 1];
  const T incl = scan_block<T>(a + b, slots);
  bins[2 * threadIdx.x] = incl - b;
  bins[2 * threadIdx.x + 1] = incl;
  __syncthreads();
}

// First bin whose running sum is at least `target` (kBins: none).
template <typename T>
__device__ __forceinline__ int first_bin(const T* bins, T target, uint32_t* out) {
  __syncthreads();
  if (threadIdx.x == 0) *out = kBins;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int b = 2 * threadIdx.x + j;
    if (bins[b] >= target && (b == 0 || bins[b - 1] < target)) *out = b;
  }
  __syncthreads();
  return (int)*out;
}

__device__ __forceinline__ u64 share_of(double share, u64 total) {     // least sum that is `share` of the total
  const double x = __builtin_ceil(share * (double)total);
  return x < 1.0 ? 1 : (x >= (double)total ? total : (u64)x);
}

// The list, descending, padded with zeros to a power of two.
__device__ __forceinline__ void sort_list(u64* list, int n) {
  int m = 64;
  while (m < n) m <<= 1;
  for (int i = n + (int)threadIdx.x; i < m; i += kThreads) list[i] = 0;
  __syncthreads();
  for (int k = 2; k <= m; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      for (int i = threadIdx.x; i < m / 2; i += kThreads) {
        const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
        const u64 x = list[lo], y = list[hi];
        if ((x < y) == ((lo & k) == 0)) {
          list[lo] = y;
          list[hi] = x;
        }
      }
      __syncthreads();
    }
}

template <int TYPE>
struct Sampler {
  Row r;
  Shared& s;
  int nseg;

  // f(token, logit) for all tokens of a segment that a wave takes; 8 neighbours a lane
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int g = threadIdx.x >> 6; g < nseg; g += kWaves) {
      const int i = g * kSeg + 8 * (threadIdx.x & 63);
      float l[8];
      load8<TYPE>(r.logits, i, r.V, l);
      f(g, i, l);
    }
  }

  // The cut among the tokens of bins [b0, b1], found digit by digit: the token at which
  // the running count (or sum of weights), which starts at `base`, reaches `target`.
  __device__ u64 descend(int b0, int b1, bool by_mass, u64 base, u64 target) {
    u64 prefix = 0;
    for (int shift = 44; shift >= 0; shift -= 11) {       // 5 digits of 11 bits: 32 + 20 bits and a little
      for (int i = threadIdx.x; i < kBins; i += kThreads) s.list[i] = 0;
      __syncthreads();
      each([&](int, int i, const float* l) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double t = exponent(r, l[j]);
          if (!(t > kLeast * 1.4426950408889634)) continue;
          const int b = bin_of(t);
          const u64 o = order_of(l[j], i + j);
          if (b < b0 || b > b1 || o >> (shift + 11) != prefix) continue;
          const u64 w = by_mass ? weight(r, t) : 1;
          if (w) atomicAdd(&s.list[kBins - 1 - (int)(o >> shift & (kBins - 1))], w);
        }
      });
      __syncthreads();
      scan_bins<u64>(s.list, s.slots);
      const int d = first_bin<u64>(s.list, target - base, &s.n);
      const u64 before = d == 0 || d >= kBins ? 0 : s.list[d - 1];
      __syncthreads();
      base += before;
      prefix = prefix << 11 | (u64)(kBins - 1 - min(d, kBins - 1));
    }
    return prefix;
  }

  // Sum of the weights of the tokens of bins [b0, b1] that lie at or before the cut.
  __device__ u64 sum_to(int b0, int b1, u64 cut) {
    u64 sum = 0;
    each([&](int, int i, const float* l) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double t = exponent(r, l[j]);
        if (!(t > kLeast * 1.4426950408889634)) continue;
        const int b = bin_of(t);
        if (b >= b0 && b <= b1 && order_of(l[j], i + j) >= cut) sum += weight(r, t);
      }
    });
    const u64 incl = scan_block<u64>(sum, s.slots);
    if (threadIdx.x == kThreads - 1) s.found[3] = incl;
    __syncthreads();
    const u64 all = s.found[3];
    __syncthreads();
    return all;
  }
};

template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a) {
  __shared__ Shared s;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x;
  Sampler<TYPE> z{{}, s, (a.V + kSeg - 1) / kSeg};
  Row& r = z.r;
  r.logits = static_cast<const char*>(a.logits) + row * a.row_stride * (TYPE == 3 ? 4 : 2);
  r.V = a.V;

  // 1. the first of the largest logits
  u64 best = 0;
  z.each([&](int, int i, const float* l) {
#pragma unroll
    for (int j = 0; j < 8; ++j) best = i + j < r.V ? max(best, order_of(l[j], i + j)) : best;
  });
#pragma unroll
  for (int off = 32; off; off >>= 1) best = max(best, (u64)__shfl_xor(best, off, 64));
  if (lane == 0) s.slots[wave] = best;
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s.mass[i] = 0;
    s.count[i] = 0;
  }
  if (threadIdx.x == 0) s.n = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWaves; ++i) best = max(best, s.slots[i]);
  __syncthreads();
  r.top = logit_of_order(best);
  const float temperature = a.temperature ? a.temperature[row] : 1.f;
  const bool none = best == 0 || r.top == -__builtin_inff();
  if (none || !(temperature > 0.f)) {        // nothing to choose from, or the first largest
    if (threadIdx.x == 0) {
      a.token[row] = none ? -1 : id_of(best);
      if (a.logprob) a.logprob[row] = none ? -__builtin_inff() : 0.f;
    }
    return;
  }
  r.inv = 1.4426950408889634 / (double)temperature;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  r.min_w = min_p > 0.f ? (double)fminf(min_p, 1.f) * (double)(1ull << kOne) : 0.0;
  const int top_k = a.top_k && a.top_k[row] > 0 && a.top_k[row] < r.V ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.f;
  const bool by_sum = top_p < 1.f;
  const double share = top_p > 0.f ? (double)top_p : 0.0;

  // 2. the histogram, and where the filters cut
  u64 cut = 0;            // tokens at or before it remain
  if (top_k || by_sum) {
    z.each([&](int, int, const float* l) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double t = exponent(r, l[j]);
        if (!(t > kLeast * 1.4426950408889634)) continue;
        const int b = bin_of(t);
        if (top_k) atomicAdd(&s.count[b], 1u);
        if (by_sum) {
          const u64 w = weight(r, t);
          if (w) atomicAdd(&s.mass[b], w);
        }
      }
    });
    __syncthreads();
    int bk = kBins, p0 = kBins, p1 = -1;      // the bin of the k-th token, the bins that may hold top-p's last one
    if (top_k) {
      scan_bins<uint32_t>(s.count, s.slots);
      bk = first_bin<uint32_t>(s.count, (uint32_t)top_k, &s.n);
    }
    if (by_sum) {
      scan_bins<u64>(s.mass, s.slots);
      const u64 most = s.mass[min(bk, kBins - 1)], least = bk < kBins ? (bk ? s.mass[bk - 1] : 0) : most;
      p0 = first_bin<u64>(s.mass, share_of(share, max(least, (u64)1)), &s.n);
      p1 = first_bin<u64>(s.mass, share_of(share, most), &s.n);
      p0 = min(p0, bk);
      p1 = min(p1, bk);
    }
    if (bk < kBins || by_sum) {
      __syncthreads();
      if (threadIdx.x == 0) s.n = 0;
      __syncthreads();
      z.each([&](int, int i, const float* l) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double t = exponent(r, l[j]);
          if (!(t > kLeast * 1.4426950408889634)) continue;
          const int b = bin_of(t);
          if (b == bk || (b >= p0 && b <= p1)) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < kList) s.list[at] = order_of(l[j], i + j);
          }
        }
      });
      __syncthreads();
      const uint32_t n = s.n;
      __syncthreads();
      const u64 upto_k = bk < kBins && bk ? s.count[bk - 1] : 0;
      const u64 mass_k = bk < kBins && bk ? s.mass[bk - 1] : 0;
      u64 total = by_sum ? s.mass[kBins - 1] : 0;
      if (n <= kList) {
        sort_list(s.list, (int)n);
        // four tokens a thread, in order: those of a bin stand next to each other
        u64 o[4], w[4];
        int bin[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * (int)threadIdx.x + j;
          o[j] = i < (int)n ? s.list[i] : 0;
          const double t = exponent(r, logit_of_order(o[j]));
          bin[j] = i < (int)n ? bin_of(t) : -1;
          w[j] = i < (int)n && by_sum ? weight(r, t) : 0;
        }
        if (threadIdx.x < 3) s.found[threadIdx.x] = 0;
        if (bk < kBins) {
          uint32_t c = 0;
          u64 m = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            c += bin[j] == bk;
            m += bin[j] == bk ? w[j] : 0;
          }
          c = scan_block<uint32_t>(c, s.slots) - c + (uint32_t)upto_k;
          m = scan_block<u64>(m, s.slots) - m + mass_k;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (bin[j] == bk) {
              m += w[j];
              if (++c == (uint32_t)top_k) {
                s.found[0] = o[j];
                s.found[1] = m;
              }
            }
          __syncthreads();
          cut = s.found[0];
          total = s.found[1];
        }
        if (by_sum) {
          const u64 target = share_of(share, total);
          u64 m = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) m += bin[j] >= p0 && bin[j] <= p1 ? w[j] : 0;
          m = scan_block<u64>(m, s.slots) - m + (p0 ? s.mass[p0 - 1] : 0);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (bin[j] >= p0 && bin[j] <= p1) {
              if (m < target && m + w[j] >= target) s.found[2] = o[j];
              m += w[j];
            }
          __syncthreads();
          cut = max(cut, s.found[2]);
        }
      } else {
        if (bk < kBins) {
          cut = z.descend(bk, bk, false, upto_k, (u64)top_k);
          if (by_sum) total = mass_k + z.sum_to(bk, bk, cut);
        }
        if (by_sum) cut = max(cut, z.descend(0, kBins - 1, true, 0, share_of(share, total)));
      }
    }
  }

  // 3. sums of what remains in segments, the segment of the drawn token, the token
  for (int g = threadIdx.x; g < kMaxSegs; g += kThreads) s.seg[g] = 0;
  __syncthreads();
  z.each([&](int g, int i, const float* l) {
    u64 sum = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double t = exponent(r, l[j]);
      if (!(t > kLeast * 1.4426950408889634)) continue;
      if (order_of(l[j], i + j) >= cut) sum += weight(r, t);
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if (lane == 0) s.seg[g] = sum;
  });
  __syncthreads();
  scan_bins<u64>(s.seg, s.slots);
  const u64 total = s.seg[kMaxSegs - 1];
  const float u = a.u[row];
  u64 drawn = u > 0.f ? (u64)((double)u * (double)total) : 0;
  if (drawn >= total) drawn = total - 1;
  const int g = first_bin<u64>(s.seg, drawn + 1, &s.n);
  if (wave == 0 && g < z.nseg) {
    const u64 before = g ? s.seg[g - 1] : 0;
    const int i = g * kSeg + 8 * lane;
    float l[8];
    load8<TYPE>(r.logits, i, r.V, l);
    u64 w[8], mine = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = order_of(l[j], i + j) >= cut ? weight(r, exponent(r, l[j])) : 0;
      mine += w[j];
    }
    u64 run = before + scan_wave(mine) - mine;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (run <= drawn && drawn < run + w[j]) {
        a.token[row] = i + j;
        if (a.logprob)
          a.logprob[row] = (float)(exponent(r, l[j]) * 0.6931471805599453 -
                                   log((double)total * (1.0 / (double)(1ull << kOne))));
      }
      run += w[j];
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int type, hipStream_t st) {
  const dim3 grid((unsigned)a.T), block(kThreads);
  if (type == 1) hipLaunchKernelGGL(sample_kernel<1>, grid, block, 0, st, a);
  else if (type == 2) hipLaunchKernelGGL(sample_kernel<2>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(sample_kernel<3>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace misa
