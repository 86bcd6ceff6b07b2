// How much attention weight each cached token got:
//   out[n][g][s] = in[n][g][s] + sum over the queries t of sequence n that see s and
//                  the heads j of kv head g of  e^(x_s - lse[t][j]),
// x_s being attention's score (scaled, capped, biased) and lse its log-sum, so the
// keys are read once and no value at all.
//
// The keys are what stays: a workgroup takes 128 keys of one kv head, holds them in
// registers as the first operand of the matrix instructions, and walks the (query,
// head) rows that see some of them: S^T [keys x rows] = K Q^T. A lane's scores are of
// ONE row, so the row's interval and log-sum are a lane's own, and the sum over rows is
// an addition into one register a key; lanes are summed once, at the end. No two
// workgroups add to the same sum and the order is fixed: results do not depend on
// when workgroups run.
#include "attend_kernel.hpp"
#include "misa_evict.hpp"

namespace misa {
namespace {

using namespace attend;

constexpr int kThreads = 256;
constexpr int kKeys = 128;      // keys of a workgroup

// What a lane knows of its row.
struct Row {
  int lo, hi;       // visible tokens
  int pos;
  float lse2;       // log-sum in units of log2
  float slope2;
};

// Row r of the rows (query, head) of kv head g, queries from t0 on.
template <int MODE>
__device__ __forceinline__ Row row_info(const MassArgs& a, int n, int g, int64_t t0, uint32_t r, uint32_t rows) {
  Row x{0, 0, 0, 0.f, 0.f};
  if (r >= rows) return x;
  const uint32_t qi = fast_quot(a.by_group, r);
  const int64_t t = t0 + qi;
  const int head = g * a.group + (int)(r - qi * a.group);
  const int seq = a.q_seq[t], len = a.q_len[t];
  const int start = a.q_start ? a.q_start[t] : 0;
  const float lse = a.lse[t * a.Hq + head];
  if constexpr (MODE == kBias) {
    x.pos = a.q_pos ? a.q_pos[t] : len - 1;
    x.slope2 = a.slopes ? a.slopes[head] * kLog2e : 0.f;
  }
  x.lse2 = lse * kLog2e;
  x.hi = clamp_len(len, a.kv.Lmax);
  x.lo = start < 0 ? 0 : start;
  if (seq != n || lse == -__builtin_inff()) x.lo = x.hi = 0;
  return x;
}

// The queries that see some of the keys [k0, k0 + kKeys), of [t_lo, t_hi): from the
// first to the last one. All threads of the workgroup call it.
__device__ __forceinline__ void seeing(const MassArgs& a, int n, int k0, int64_t t_lo, int64_t t_hi, int64_t& t0,
                                       int64_t& t1) {
  __shared__ int first[kThreads / 64], last[kThreads / 64];
  int lo = 0x7fffffff, hi = -1;
  for (int64_t t = t_lo + threadIdx.x; t < t_hi; t += kThreads) {
    const int len = clamp_len(a.q_len[t], a.kv.Lmax);
    const int start = a.q_start ? a.q_start[t] : 0;
    if (a.q_seq[t] == n && start < len && len > k0 && start < k0 + kKeys) {
      lo = min(lo, (int)t);
      hi = max(hi, (int)t);
    }
  }
  lo = wave_min_of(lo);
  hi = wave_max_of(hi);
  const int w = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    first[w] = lo;
    last[w] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) {
    lo = min(lo, first[i]);
    hi = max(hi, last[i]);
  }
  t0 = uniform(lo);
  t1 = (int64_t)uniform(hi) + 1;
}

// Address of key s of sequence n, or null.
__device__ __forceinline__ const uint16_t* key_row(const MassArgs& a, int n, int g, int s) {
  if (s >= a.kv.Lmax) return nullptr;
  const uint32_t col = fast_quot(a.kv.by_page, (uint32_t)s);
  const int page = kv_page(a.kv, n, col);
  if (page < 0) return nullptr;
  return a.kv.k + page * a.kv.page_stride + (int64_t)(s - (int)col * a.kv.page) * a.kv.tok_stride + g * a.kv.head_stride;
}

// Weights of MR rows and MR keys (one accumulator tile) added to the keys' sums.
// off: the first key that the lane's registers hold, relative to the row's numbers.
template <int MR, int MODE, bool MASK, typename Acc>
__device__ __forceinline__ void add_weights(const Acc& s, Acc& sum, const Row& r, int key, uint64_t have, float c,
                                            const FarCap& cap) {
  constexpr int AR = MR * MR / 64;
#pragma unroll
  for (int j = 0; j < AR; ++j) {
    const int o = MR == 32 ? 8 * (j >> 2) + (j & 3) : j;
    float x;
    if constexpr (MODE == kPlain) {
      x = s[j] * c - r.lse2;
    } else {
      float off = r.lse2;
      if constexpr (MODE == kBias) off += r.slope2 * (float)abs(r.pos - (key + o));
      x = cap.cap2 != 0.f ? cap.chosen(s[j], off) : s[j] * c - off;
    }
    float p = __builtin_amdgcn_exp2f(x);
    if constexpr (MASK) p = (key + o >= r.lo && key + o < r.hi && (have >> o & 1)) ? p : 0.f;
    sum[j] += p;
  }
}

// Sum over the lanes of a group of MR (16 or 32) neighbouring lanes.
template <int MR>
__device__ __forceinline__ float sum_lanes(float v) {
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xb1, 0xf, 0xf, false));    // 1, 0, 3, 2
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4e, 0xf, 0xf, false));    // 2, 3, 0, 1
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, false));   // 7 - i of 8
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, false));   // 15 - i of 16
  if (MR == 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// Writes the sums of the keys [k0, k0 + kKeys), which lie in LDS.
__device__ __forceinline__ void store_sums(const MassArgs& a, int n, int g, int split, int k0, const float* sums) {
  const int s = k0 + (int)threadIdx.x;
  if (threadIdx.x >= kKeys || s >= a.kv.Lmax) return;
  const float v = sums ? sums[threadIdx.x] : 0.f;
  if (a.part) {
    a.part[(((int64_t)split * a.kv.nseq + n) * a.Hkv + g) * a.kv.Lmax + s] = v;
  } else {
    const int64_t i = ((int64_t)n * a.Hkv + g) * a.kv.Lmax + s;
    a.out[i] = (a.in ? a.in[i] : 0.f) + v;
  }
}

// Few rows a sequence (decode steps): each wave takes 32 keys and all rows, 16 at a time.
template <bool HALF, int D, int MODE>
__global__ __launch_bounds__(kThreads) void mass_few_kernel(MassArgs a) {
  constexpr int KF = D / 32;
  __shared__ float sums[kKeys];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lists = (int)a.kv.nseq * a.Hkv;
  const int tile = blockIdx.x / lists, list = blockIdx.x % lists;
  const int n = list / a.Hkv, g = list % a.Hkv, k0 = tile * kKeys;
  int64_t t0, t1;
  seeing(a, n, k0, 0, a.T, t0, t1);
  if (t0 >= t1) {
    if (a.part || a.in != a.out) store_sums(a, n, g, 0, k0, nullptr);
    return;
  }
  const int key0 = k0 + 32 * wave;
  u32x4 kf[2][KF];
  uint64_t have[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t* p = key_row(a, n, g, key0 + 16 * i + (lane & 15));
    have[i] = __ballot(p != nullptr);
#pragma unroll
    for (int f = 0; f < KF; ++f)
      kf[i][f] = p ? *reinterpret_cast<const u32x4*>(p + 32 * f + 8 * (lane >> 4)) : u32x4{0, 0, 0, 0};
  }
  const uint32_t rows = (uint32_t)(t1 - t0) * a.group;
  const float c = a.scale * kLog2e;
  const FarCap cap = a.cap != 0.f ? far_cap(a.cap, a.scale / a.cap) : FarCap{0.f, 0.f, 0.f, false};
  floatx4 sum[2] = {};
  for (uint32_t r0 = 0; r0 < rows; r0 += 16) {
    const uint32_t r = r0 + (lane & 15);
    const Row x = row_info<MODE>(a, n, g, t0, r, rows);
    const uint32_t rr = r < rows ? r : 0, qi = fast_quot(a.by_group, rr);
    const uint16_t* q = a.q + (t0 + qi) * a.q_ts + (int64_t)(g * a.group + (int)(rr - qi * a.group)) * a.q_hs + 8 * (lane >> 4);
    u32x4 qf[KF];
#pragma unroll
    for (int f = 0; f < KF; ++f) qf[f] = *reinterpret_cast<const u32x4*>(q + 32 * f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int f = 0; f < KF; ++f) s = mfma16<HALF>(kf[i][f], qf[f], s);
      const int key = key0 + 16 * i + 4 * (lane >> 4);
      add_weights<16, MODE, true>(s, sum[i], x, key, have[i] >> (4 * (lane >> 4)), c, cap);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = sum_lanes<16>(sum[i][j]);
      if ((lane & 15) == j) sums[32 * wave + 16 * i + 4 * (lane >> 4) + j] = v;
    }
  __syncthreads();
  store_sums(a, n, g, 0, k0, sums);
}

// Many rows (prompts, windows of queries): 64 rows at a time go through LDS, the next
// ones under way in registers meanwhile. Two groups of waves hold 64 keys each, and the
// two waves of a group take the first and the last 32 of the rows; at d = 256 four
// waves hold 32 keys each and take the same 32 rows (64 keys would spill).
template <int D>
struct ManyShape {
  static constexpr int NT = D == 256 ? 1 : 2;            // tiles of 32 keys a wave
  static constexpr int KG = kKeys / (32 * NT);           // groups of keys
  static constexpr int RG = kThreads / 64 / KG;          // groups of rows
  static constexpr int ROWS = 32 * RG;
};

template <bool HALF, int D, int MODE>
__global__ __launch_bounds__(kThreads, 2) void mass_many_kernel(MassArgs a) {
  using S = ManyShape<D>;
  constexpr int KF = D / 16, PIECES = D / 8, NT = S::NT, ROWS = S::ROWS, NLD = ROWS * PIECES / kThreads;
  __shared__ __align__(16) uint16_t stage[2][ROWS * D];
  __shared__ float sums[S::RG][kKeys];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kg = wave % S::KG, rg = wave / S::KG;
  const int lists = (int)a.kv.nseq * a.Hkv;
  const int split = blockIdx.x % a.splits, rest = blockIdx.x / a.splits;
  const int tile = rest / lists, list = rest % lists;
  const int n = list / a.Hkv, g = list % a.Hkv, k0 = tile * kKeys;
  int64_t t0, t1;
  seeing(a, n, k0, a.T * split / a.splits, a.T * (split + 1) / a.splits, t0, t1);
  if (t0 >= t1) {
    if (a.part || a.in != a.out) store_sums(a, n, g, split, k0, nullptr);
    return;
  }
  const int key0 = k0 + 32 * NT * kg;
  u32x4 kf[NT][KF];
  uint64_t have[NT];
  bool all_there = true;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const uint16_t* p = key_row(a, n, g, key0 + 32 * i + (lane & 31));
    have[i] = __ballot(p != nullptr);
    all_there &= have[i] == ~0ull;
#pragma unroll
    for (int f = 0; f < KF; ++f)
      kf[i][f] = p ? *reinterpret_cast<const u32x4*>(p + 16 * f + 8 * (lane >> 5)) : u32x4{0, 0, 0, 0};
  }
  const uint32_t rows = (uint32_t)(t1 - t0) * a.group;
  const float c = a.scale * kLog2e;
  const FarCap cap = a.cap != 0.f ? far_cap(a.cap, a.scale / a.cap) : FarCap{0.f, 0.f, 0.f, false};

  u32x4 next[NLD];
  Row row_next;
  auto fetch = [&](uint32_t r0) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int at = (int)threadIdx.x + i * kThreads;
      const uint32_t r = r0 + at / PIECES, rr = r < rows ? r : 0, qi = fast_quot(a.by_group, rr);
      next[i] = *reinterpret_cast<const u32x4*>(a.q + (t0 + qi) * a.q_ts +
                                                (int64_t)(g * a.group + (int)(rr - qi * a.group)) * a.q_hs + 8 * (at % PIECES));
    }
    row_next = row_info<MODE>(a, n, g, t0, r0 + 32 * rg + (lane & 31), rows);
  };
  auto put = [&](int b) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int at = (int)threadIdx.x + i * kThreads, r = at / PIECES, p = at % PIECES;
      *reinterpret_cast<u32x4*>(&stage[b][r * D + 8 * (p ^ swizzle<D>(r))]) = next[i];
    }
  };
  floatx16 sum[NT] = {};
  fetch(0);
  put(0);
  Row x = row_next;
  __syncthreads();
  int b = 0;
  for (uint32_t r0 = 0; r0 < rows; r0 += ROWS, b ^= 1) {
    const bool more = r0 + ROWS < rows;
    if (more) fetch(r0 + ROWS);
    const bool sees = x.lo < x.hi && x.hi > key0 && x.lo < key0 + 32 * NT;
    if (__ballot(sees)) {
      const bool whole = all_there && __ballot(x.lo <= key0 && x.hi >= key0 + 32 * NT) == ~0ull;
      floatx16 s[NT] = {};
      const int r = 32 * rg + (lane & 31);
#pragma unroll
      for (int f = 0; f < KF; ++f) {
        const u32x4 qf = *reinterpret_cast<const u32x4*>(&stage[b][r * D + 8 * ((2 * f + (lane >> 5)) ^ swizzle<D>(r))]);
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i] = mfma32<HALF>(kf[i][f], qf, s[i]);
      }
      const int sh = 4 * (lane >> 5), key = key0 + sh;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (whole) add_weights<32, MODE, false>(s[i], sum[i], x, key + 32 * i, 0, c, cap);
        else add_weights<32, MODE, true>(s[i], sum[i], x, key + 32 * i, have[i] >> sh, c, cap);
      }
    }
    if (more) {
      put(b ^ 1);
      x = row_next;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float v = sum_lanes<32>(sum[i][j]);
      if ((lane & 31) == j) sums[rg][32 * NT * kg + 32 * i + 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3)] = v;
    }
  __syncthreads();
  if (S::RG > 1 && threadIdx.x < kKeys) sums[0][threadIdx.x] += sums[S::RG - 1][threadIdx.x];
  store_sums(a, n, g, split, k0, sums[0]);
}

// out = in + the sums of all query ranges (and, for G = 1, of all heads), in a fixed order.
__global__ __launch_bounds__(kThreads) void mass_join_kernel(MassArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.kv.nseq * a.G * a.kv.Lmax) return;
  const int64_t list = i / a.kv.Lmax, s = i - list * a.kv.Lmax;
  const int64_t n = list / a.G;
  const int heads = a.G == 1 ? a.Hkv : 1, g0 = a.G == 1 ? 0 : (int)(list - n * a.G);
  float v = 0.f;
  for (int c = 0; c < a.splits; ++c)
    for (int h = 0; h < heads; ++h) v += a.part[(((int64_t)c * a.kv.nseq + n) * a.Hkv + g0 + h) * a.kv.Lmax + s];
  a.out[i] = (a.in ? a.in[i] : 0.f) + v;
}

bool few_rows(int64_t T, int64_t nseq, int group) { return (T + nseq - 1) / nseq * group <= 16; }

int64_t key_tiles(const KvView& kv) { return (kv.Lmax + kKeys - 1) / kKeys; }

template <bool HALF, int D, int MODE>
void launch_mode(const MassArgs& a, unsigned blocks, hipStream_t st) {
  if (few_rows(a.T, a.kv.nseq, a.group))
    hipLaunchKernelGGL((mass_few_kernel<HALF, D, MODE>), dim3(blocks), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((mass_many_kernel<HALF, D, MODE>), dim3(blocks), dim3(kThreads), 0, st, a);
}
template <bool HALF, int D>
void launch_dim(const MassArgs& a, unsigned blocks, hipStream_t st) {
  if (a.slopes) launch_mode<HALF, D, kBias>(a, blocks, st);
  else if (a.cap != 0.f) launch_mode<HALF, D, kCap>(a, blocks, st);
  else launch_mode<HALF, D, kPlain>(a, blocks, st);
}
template <bool HALF>
void launch_type(const MassArgs& a, unsigned blocks, hipStream_t st) {
  if (a.d == 64) launch_dim<HALF, 64>(a, blocks, st);
  else if (a.d == 128) launch_dim<HALF, 128>(a, blocks, st);
  else launch_dim<HALF, 256>(a, blocks, st);
}

}  // namespace

int mass_splits(int64_t T, int64_t nseq, int heads, int group, int64_t Lmax, int d) {
  if (few_rows(T, nseq, group)) return 1;
  const int64_t tiles = (Lmax + kKeys - 1) / kKeys * nseq * heads;
  int s = 1;
  while (s < 16 && tiles * s < 2048 && T * group / (s * 2) >= 1024) s *= 2;
  return s;
}

int64_t mass_blocks(const MassArgs& a) {
  return key_tiles(a.kv) * a.kv.nseq * a.Hkv * a.splits;
}

hipError_t launch_mass(const MassArgs& a, bool half, hipStream_t st) {
  const unsigned blocks = (unsigned)mass_blocks(a);
  if (half) launch_type<true>(a, blocks, st);
  else launch_type<false>(a, blocks, st);
  if (a.part) {
    const int64_t n = a.kv.nseq * a.G * a.kv.Lmax;
    hipLaunchKernelGGL(mass_join_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace misa
