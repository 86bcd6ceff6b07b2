// How much attention weight each cached token got:
//   out[n][g][s] = in[n][g][s] + sum over the queries t of sequence n that see s and
//                  the heads j of kv head g of  e^(x_s - lse[t][j]),
// x_s being attention's score (scaled, capped, biased) and lse its log-sum, so only keys
// are read, once for each part that their queries are split into, and no value at all.
//
// The keys are what stays: a workgroup takes 256 keys of one kv head (128 of d = 256; a wave
// of its own 64, for few rows), holds them in registers as the first operand of the matrix
// instructions, and walks the (query, head) rows that see some of them: S^T [keys x rows] =
// K Q^T. A lane's scores are of ONE row, so the row's interval and log-sum are a lane's own,
// and the sum over rows is an addition into one register a key; lanes are summed once, at the
// end. No two workgroups add to the same sum and the order is fixed: results do not depend on
// when workgroups run. Sums are fp32, scores as the attention kernels have them.
#include "attend_kernel.hpp"
#include "misa_evict.hpp"

namespace misa {
namespace {

using namespace attend;

constexpr int kThreads = 256;

// What a score goes through, as a kernel's MODE. (A branch on the cap beside the bias, taken for
// each score, cost more than the rest of it: 83 -> 75 us for two prompts of 2000 tokens, d = 256.)
constexpr int kCapped = 1, kBiased = 2;

// What a lane knows of its row.
struct Row {
  int lo, hi;       // visible tokens
  int pos;
  float lse2;       // log-sum in units of log2
  float slope2;
};

// Row of query t and a head; `is`: there is such a row.
template <int MODE>
__device__ __forceinline__ Row row_info(const MassArgs& a, int n, int64_t t, int head, bool is) {
  Row x{0, 0, 0, 0.f, 0.f};
  if (!is) return x;
  const int seq = a.q_seq[t], len = a.q_len[t];
  const int start = a.q_start ? a.q_start[t] : 0;
  const float lse = a.lse[t * a.Hq + head];
  if constexpr (MODE & kBiased) {
    x.pos = a.q_pos ? a.q_pos[t] : len - 1;
    x.slope2 = a.slopes ? a.slopes[head] * kLog2e : 0.f;
  }
  x.lse2 = lse * kLog2e;
  x.hi = clamp_len(len, a.kv.Lmax);
  x.lo = start < 0 ? 0 : start;
  if (seq != n || lse == -__builtin_inff() || x.lo > x.hi) x.lo = x.hi = 0;
  return x;
}

// The same in two parts, loads alone (by 32-bit offsets behind query t and a head: query t + qi,
// head + h; no branch, nothing looked at: what there is no array of is read from another one) and
// the rest. A wait between them at the loads' place held every step up by a trip to memory.
struct RawRow {
  int seq, len, start, pos;
  float lse, slope;
};
template <int MODE>
__device__ __forceinline__ RawRow row_behind(const MassArgs& a, int64_t t, int head, int qi, int h, bool is) {
  const int o = is ? 4 * qi : 0;
  auto load = [](const void* p, int o) __attribute__((always_inline)) {
    return (int)__builtin_amdgcn_raw_buffer_load_b32(buffer_view(p, 0xfffffff0u), o, 0, 0);
  };
  RawRow x;
  x.seq = load(a.q_seq + t, o);
  x.len = load(a.q_len + t, o);
  x.start = load((a.q_start ? a.q_start : a.q_len) + t, o);
  x.lse = __int_as_float(load(a.lse + t * a.Hq + head, is ? 4 * (qi * a.Hq + h) : 0));
  if constexpr (MODE & kBiased) {
    x.pos = load((a.q_pos ? a.q_pos : a.q_len) + t, o);
    x.slope = __int_as_float(load(a.slopes + head, is ? 4 * h : 0));
  }
  return x;
}
template <int MODE>
__device__ __forceinline__ Row row_of(const MassArgs& a, int n, const RawRow& r, bool is) {
  Row x;
  x.pos = 0;
  x.slope2 = 0.f;
  if constexpr (MODE & kBiased) {
    x.pos = r.pos - (a.q_pos ? 0 : 1);
    x.slope2 = r.slope * kLog2e;
  }
  x.lse2 = r.lse * kLog2e;
  x.lo = a.q_start ? max(r.start, 0) : 0;
  x.hi = min(r.len, (int)a.kv.Lmax);
  if (!is || r.seq != n || r.lse == -__builtin_inff() || x.lo >= x.hi) x.lo = x.hi = 0;
  return x;
}

// The first and the last of T queries that see some of the keys [k0, k0 + KEYS), as thread i of
// THREADS finds them: four of them a load, 16 under way.
typedef int32_t int32x4_any __attribute__((ext_vector_type(4), aligned(4)));
template <int KEYS, int THREADS>
__device__ __forceinline__ void look(const MassArgs& a, int n, int k0, int i, int& lo, int& hi) {
  lo = 0x7fffffff;
  hi = -1;
  auto one = [&](int64_t t, int seq, int len, int start) __attribute__((always_inline)) {
    len = clamp_len(len, a.kv.Lmax);
    if (seq == n && start < len && len > k0 && start < k0 + KEYS) {
      lo = min(lo, (int)t);
      hi = max(hi, (int)t);
    }
  };
#pragma unroll 4
  for (int64_t t = 4 * i; t + 4 <= a.T; t += 4 * THREADS) {
    const int32x4_any seq = *reinterpret_cast<const int32x4_any*>(a.q_seq + t);
    const int32x4_any len = *reinterpret_cast<const int32x4_any*>(a.q_len + t);
    const int32x4_any start = a.q_start ? *reinterpret_cast<const int32x4_any*>(a.q_start + t) : int32x4_any{};
#pragma unroll
    for (int j = 0; j < 4; ++j) one(t + j, seq[j], len[j], start[j]);
  }
  const int64_t t = (a.T & ~(int64_t)3) + i;
  if (t < a.T) one(t, a.q_seq[t], a.q_len[t], a.q_start ? a.q_start[t] : 0);
}

// From the first to behind the last query that sees some of the keys [k0, k0 + KEYS). All
// threads of the workgroup call it.
template <int KEYS>
__device__ __forceinline__ void seeing(const MassArgs& a, int n, int k0, int& t0, int& t1) {
  __shared__ int first[kThreads / 64], last[kThreads / 64];
  int lo, hi;
  look<KEYS, kThreads>(a, n, k0, (int)threadIdx.x, lo, hi);
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
  t1 = uniform(hi) + 1;
}

// Address of key s of sequence n, or null.
__device__ __forceinline__ const uint16_t* key_row(const MassArgs& a, int n, int g, int s) {
  if (s >= a.kv.Lmax) return nullptr;
  const uint32_t col = fast_quot(a.kv.by_page, (uint32_t)s);
  const int page = kv_page(a.kv, n, col);
  if (page < 0) return nullptr;
  return a.kv.k + page * a.kv.page_stride + (int64_t)(s - (int)col * a.kv.page) * a.kv.tok_stride + g * a.kv.head_stride;
}

// Scores of MR rows and MR keys (one accumulator tile), less the rows' log-sums, in units
// of log2. key: the first key that the lane's registers hold.
template <int MR, int MODE, typename Acc>
__device__ __forceinline__ void finish_scores(Acc& s, const Row& r, int key, float c, const FarCap& cap) {
#pragma unroll
  for (int j = 0; j < MR * MR / 64; ++j) {
    const int o = MR == 32 ? 8 * (j >> 2) + (j & 3) : j;
    float off = r.lse2;
    if constexpr (MODE & kBiased) off += r.slope2 * (float)abs(r.pos - (key + o));
    s[j] = MODE & kCapped ? cap.chosen(s[j], off) : s[j] * c - off;
  }
}

// What a row does not see adds nothing, whatever its score is.
template <int MR, typename Acc>
__device__ __forceinline__ void hide(Acc& s, const Row& r, int key) {
  const int first = r.lo - key;
  const uint32_t many = (uint32_t)(r.hi - r.lo);
#pragma unroll
  for (int j = 0; j < MR * MR / 64; ++j) {
    const int o = MR == 32 ? 8 * (j >> 2) + (j & 3) : j;
    s[j] = (uint32_t)(o - first) < many ? s[j] : -__builtin_inff();
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

// Writes the sums of the keys [k0, k0 + KEYS), which lie in LDS.
template <int KEYS>
__device__ __forceinline__ void store_sums(const MassArgs& a, int n, int g, int split, int k0, const float* sums) {
  const int s = k0 + (int)threadIdx.x;
  if (threadIdx.x >= KEYS || s >= a.kv.Lmax) return;
  const float v = sums ? sums[threadIdx.x] : 0.f;
  if (a.part) {
    a.part[(((int64_t)split * a.kv.nseq + n) * a.Hkv + g) * a.kv.Lmax + s] = v;
  } else {
    const int64_t i = ((int64_t)n * a.Hkv + g) * a.kv.Lmax + s;
    a.out[i] = (a.in ? a.in[i] : 0.f) + v;
  }
}

// Few rows a sequence (decode steps): memory-bound, so each wave is on its own. It takes
// 64 keys of one kv head, all under way at once, and all rows, 16 at a time. The look-up
// of the keys' pages goes beside the search for the queries. Neighbouring waves take the
// kv heads of the same keys, then the next keys, one sequence after the other: 8 x 32768 tokens
// of 8 heads of 128 in 87 us, 4.5 TB/s (the sequences side by side 101; runs of 2 to 8 such
// pieces a wave, the next one under way, 88 to 108; keys through LDS, whole rows an
// instruction, 107).
constexpr int kFewTiles = 4, kFewKeys = 16 * kFewTiles;

template <bool HALF, int D, int MODE>
__global__ __launch_bounds__(kThreads, 2) void mass_few_kernel(MassArgs a) {
  constexpr int KF = D / 32, NT = kFewTiles;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + uniform((int)threadIdx.x >> 6);
  const int64_t of_seq = (a.kv.Lmax + kFewKeys - 1) / kFewKeys * a.Hkv;
  const int n = (int)(unit / of_seq);
  if (n >= a.kv.nseq) return;
  const int64_t rest = unit - n * of_seq;
  const int g = (int)(rest % a.Hkv), key0 = (int)(rest / a.Hkv) * kFewKeys;
  // lanes 0 .. 15 of each 16 take one key's sum each
  const int mine = key0 + 16 * ((lane & 15) >> 2) + 4 * (lane >> 4) + (lane & 3);
  const bool holds = mine < a.kv.Lmax;
  const int64_t at = ((int64_t)n * a.Hkv + g) * a.kv.Lmax + mine;
  const uint16_t* p[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) p[i] = key_row(a, n, g, key0 + 16 * i + (lane & 15));
  const float before = holds && !a.part && a.in ? a.in[at] : 0.f;
  int lo, hi;
  look<kFewKeys, 64>(a, n, key0, lane, lo, hi);
  const int64_t t0 = wave_min_of(lo), t1 = (int64_t)wave_max_of(hi) + 1;
  float total = 0.f;
  if (t0 < t1) {
    u32x4 kf[NT][KF];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int f = 0; f < KF; ++f)
        kf[i][f] = p[i] ? *reinterpret_cast<const u32x4*>(p[i] + 32 * f + 8 * (lane >> 4)) : u32x4{0, 0, 0, 0};
    const uint32_t rows = (uint32_t)(t1 - t0) * a.group;
    const float c = a.scale * kLog2e;
    const FarCap cap = a.cap != 0.f ? far_cap(a.cap, a.scale / a.cap) : FarCap{0.f, 0.f, 0.f, false};
    float sum[NT][4] = {};
    for (uint32_t r0 = 0; r0 < rows; r0 += 16) {
      const uint32_t r = r0 + (lane & 15), rr = r < rows ? r : 0, qi = fast_quot(a.by_group, rr);
      const int head = g * a.group + (int)(rr - qi * a.group);
      const Row x = row_info<MODE>(a, n, t0 + qi, head, r < rows);
      const uint16_t* q = a.q + (t0 + qi) * a.q_ts + (int64_t)head * a.q_hs + 8 * (lane >> 4);
      u32x4 qf[KF];
#pragma unroll
      for (int f = 0; f < KF; ++f) qf[f] = *reinterpret_cast<const u32x4*>(q + 32 * f);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < KF; ++f) s = mfma16<HALF>(kf[i][f], qf[f], s);
        const int key = key0 + 16 * i + 4 * (lane >> 4);
        finish_scores<16, MODE>(s, x, key, c, cap);
        hide<16>(s, x, key);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] += __builtin_amdgcn_exp2f(s[j]);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint64_t there = __ballot(p[i] != nullptr);     // a key without a page is given nothing
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = sum_lanes<16>(sum[i][j]);
        if ((lane & 15) == 4 * i + j && there >> (4 * (lane >> 4) + j) & 1) total = v;
      }
    }
  }
  if (!holds) return;
  if (a.part) a.part[at] = total;
  else if (t0 < t1 || a.in != a.out) a.out[at] = before + total;
}

// Many rows (prompts, windows of queries): steps of 64 (d = 256: 32) rows go through LDS,
// the next ones under way in registers meanwhile. Each wave holds 64 (32) keys and takes
// all rows. 8192 causal tokens of 64 heads of 128 over 8 kv heads: 620 us, 0.89 PFLOP/s of the
// products that somebody sees, beside one exponential (8 cycles a wave), one multiply-add and
// one addition a score, which bound it with the products; a wave's products go beside the
// weights of its 32 rows before. (128 keys a workgroup, products and weights in turn, a step's
// intervals waited for: 1640.)
template <int D>
struct ManyShape {
  static constexpr int NT = D == 256 ? 1 : 2;            // tiles of 32 keys a wave
  static constexpr int KEYS = 32 * NT * kThreads / 64;   // keys of a workgroup
  static constexpr int RT = D == 256 ? 1 : 2;            // tiles of 32 rows a step
  static constexpr int ROWS = 32 * RT;
};

template <bool HALF, int D, int MODE>
__global__ __launch_bounds__(kThreads, 2) void mass_many_kernel(MassArgs a) {
  using S = ManyShape<D>;
  constexpr int KF = D / 16, PIECES = D / 8, NT = S::NT, RT = S::RT, ROWS = S::ROWS, NLD = ROWS * PIECES / kThreads;
  __shared__ __align__(16) uint16_t stage[2][ROWS * D];
  __shared__ float sums[S::KEYS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lists = (int)a.kv.nseq * a.Hkv;
  // the lists next to each other (on XCDs of their own where there are eight), the first
  // keys before later ones: the most work first
  const int list = blockIdx.x % lists, rest = blockIdx.x / lists;
  const int split = rest % a.splits, tile = rest / a.splits;
  const int n = list / a.Hkv, g = list % a.Hkv, k0 = tile * S::KEYS;
  // a step takes all heads of `per` queries, or up to ROWS heads of one query
  const int per = a.group < ROWS ? ROWS / a.group : 1;
  int t0, t1;                           // T is below 2^31
  seeing<S::KEYS>(a, n, k0, t0, t1);
  if (t0 < t1 && a.splits > 1) {        // the workgroup's part of them, in whole steps
    const uint32_t all = (uint32_t)(t1 - t0), steps = (all + per - 1) / per;
    const uint32_t part = (steps + a.splits - 1) / a.splits * per, from = min(part * split, all);
    t1 = t0 + (int)min(from + part, all);
    t0 += (int)from;
  }
  if (t0 >= t1) {
    if (a.part || a.in != a.out) store_sums<S::KEYS>(a, n, g, split, k0, nullptr);
    return;
  }
  const int key0 = k0 + 32 * NT * wave;
  u32x4 kf[NT][KF];
  uint64_t there[NT];     // a key without a page is given nothing at the end
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const uint16_t* p = key_row(a, n, g, key0 + 32 * i + (lane & 31));
    there[i] = __ballot(p != nullptr);
#pragma unroll
    for (int f = 0; f < KF; ++f)
      kf[i][f] = p ? *reinterpret_cast<const u32x4*>(p + 16 * f + 8 * (lane >> 5)) : u32x4{0, 0, 0, 0};
  }
  const float c = a.scale * kLog2e;
  const FarCap cap = a.cap != 0.f ? far_cap(a.cap, a.scale / a.cap) : FarCap{0.f, 0.f, 0.f, false};

  // A thread's place in a step is the same in all steps: 32-bit offsets behind a uniform base.
  const int piece = 16 * ((int)threadIdx.x % PIECES);
  uint32_t off[NLD];
  int mark[NLD];        // query of the step, or head where a step has one query
#pragma unroll
  for (int i = 0; i < NLD; ++i) {
    const int r = ((int)threadIdx.x + i * kThreads) / PIECES;
    const int qi = per > 1 ? min((int)fast_quot(a.by_group, (uint32_t)r), per - 1) : 0;
    mark[i] = per > 1 ? qi : r;
    off[i] = 2u * (uint32_t)(qi * (int)a.q_ts + (per > 1 ? min(r - qi * a.group, a.group - 1) : r) * (int)a.q_hs) + piece;
  }
  int my_q[RT], my_h[RT];     // the lane's rows
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int my = 32 * i + (lane & 31);
    my_q[i] = per > 1 ? (int)fast_quot(a.by_group, (uint32_t)my) : 0;
    my_h[i] = my - my_q[i] * a.group;
  }
  u32x4 next[NLD];
  RawRow raw[RT];
  bool is[RT];
  Row x[RT];
  int t = t0;           // first query of the next step to fetch
  int h0 = 0;           // and first of its heads
  auto fetch = [&]() __attribute__((always_inline)) {
    const int head = g * a.group + h0;
    const int left = per > 1 ? min(t1 - t, per) : a.group - h0;
    // in the place of what lies behind the last query or head: a row that there is
    const __amdgpu_buffer_rsrc_t q = buffer_view(a.q + (int64_t)t * a.q_ts + (int64_t)head * a.q_hs, 0xfffffff0u);
#pragma unroll
    for (int i = 0; i < NLD; ++i)
      next[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(q, (int)(mark[i] < left ? off[i] : piece), 0, 0));
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      is[i] = (per > 1 ? my_q[i] : my_h[i]) < left && my_q[i] < per;
      raw[i] = row_behind<MODE>(a, t, head, my_q[i], my_h[i], is[i]);
    }
    h0 += ROWS;
    if (h0 >= a.group) {
      h0 = 0;
      t += per;
    }
  };
  auto put = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int at = (int)threadIdx.x + i * kThreads, r = at / PIECES, p = at % PIECES;
      *reinterpret_cast<u32x4*>(&stage[b][r * D + 8 * (p ^ swizzle<D>(r))]) = next[i];
    }
  };
  float sum[NT][16] = {};
  // The scores of 32 rows go into s[u] while the weights of the 32 rows before, whose
  // scores are finished, are added from s[1 - u].
  floatx16 s[2][NT];
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int j = 0; j < 16; ++j) s[1][k][j] = -__builtin_inff();
  auto add = [&](int u) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        sum[k][j] += __builtin_amdgcn_exp2f(s[u][k][j]);
        asm volatile("" : "+v"(sum[k][j]));      // here, beside the products, not behind a later branch
      }
  };
  // rows r .. r + 31 of stage[b]
  auto rows32 = [&](int b, int u, int r, const Row& x) __attribute__((always_inline)) {
    r += lane & 31;
#pragma unroll
    for (int k = 0; k < NT; ++k) s[u][k] = floatx16{};
#pragma unroll
    for (int f = 0; f < KF; ++f) {
      const u32x4 qf = *reinterpret_cast<const u32x4*>(&stage[b][r * D + 8 * ((2 * f + (lane >> 5)) ^ swizzle<D>(r))]);
#pragma unroll
      for (int k = 0; k < NT; ++k) s[u][k] = mfma32<HALF>(kf[k][f], qf, s[u][k]);
    }
    add(u ^ 1);
    const int key = key0 + 4 * (lane >> 5);
#pragma unroll
    for (int k = 0; k < NT; ++k) finish_scores<32, MODE>(s[u][k], x, key + 32 * k, c, cap);
    if (__ballot(x.lo <= key0 && x.hi >= key0 + 32 * NT) != ~0ull) {
#pragma unroll
      for (int k = 0; k < NT; ++k) hide<32>(s[u][k], x, key + 32 * k);
    }
  };
  uint32_t steps = (uint32_t)(t1 - t0);
  steps = per > 1 ? (steps + per - 1) / per : steps * ((a.group + ROWS - 1) / ROWS);
  auto turn = [&](auto which) __attribute__((always_inline)) {        // false: that was the last step
    constexpr int b = decltype(which)::value;
    const bool more = --steps != 0;
    if (more) fetch();
    if constexpr (RT == 1) {
      rows32(b, b, 0, x[0]);
    } else {
      rows32(b, 0, 0, x[0]);
      rows32(b, 1, 32, x[1]);
    }
    if (more) {
      put(b ^ 1);
#pragma unroll
      for (int i = 0; i < RT; ++i) x[i] = row_of<MODE>(a, n, raw[i], is[i]);
      __syncthreads();
    } else {
      add(RT == 1 ? b : 1);
    }
    return more;
  };
  fetch();
  put(0);
#pragma unroll
  for (int i = 0; i < RT; ++i) x[i] = row_of<MODE>(a, n, raw[i], is[i]);
  __syncthreads();
  while (turn(std::integral_constant<int, 0>{}) && turn(std::integral_constant<int, 1>{})) {
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float v = sum_lanes<32>(sum[i][j]);
      const int k = 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
      if ((lane & 31) == j) sums[32 * NT * wave + 32 * i + k] = there[i] >> k & 1 ? v : 0.f;
    }
  __syncthreads();
  store_sums<S::KEYS>(a, n, g, split, k0, sums);
}

// out = in + the sums of all query ranges (and, for G = 1, of all heads), in a fixed order.
__global__ __launch_bounds__(kThreads) void mass_join_kernel(MassArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.kv.nseq * a.G * a.kv.Lmax) return;
  const int64_t list = i / a.kv.Lmax, s = i - list * a.kv.Lmax;
  const int64_t n = list / a.G;
  const int heads = a.G == 1 ? a.Hkv : 1, g0 = a.G == 1 ? 0 : (int)(list - n * a.G);
  const float* p = a.part + ((int64_t)n * a.Hkv + g0) * a.kv.Lmax + s;
  const int64_t step = a.kv.nseq * a.Hkv * a.kv.Lmax;
  float v = 0.f;
  for (int c0 = 0; c0 < a.splits * heads; c0 += 8) {      // 8 of them on their way at a time
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + j, split = c / heads;
      x[j] = c < a.splits * heads ? p[split * step + (int64_t)(c - split * heads) * a.kv.Lmax] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v += x[j];
  }
  a.out[i] = (a.in ? a.in[i] : 0.f) + v;
}

// Keys of a workgroup of the kernel for many rows.
int many_keys(int d) { return d == 256 ? ManyShape<256>::KEYS : ManyShape<128>::KEYS; }

template <bool HALF, int D, int MODE>
void launch_mode(const MassArgs& a, unsigned blocks, hipStream_t st) {
  if (a.few)
    hipLaunchKernelGGL((mass_few_kernel<HALF, D, MODE>), dim3(blocks), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((mass_many_kernel<HALF, D, MODE>), dim3(blocks), dim3(kThreads), 0, st, a);
}
template <bool HALF, int D>
void launch_dim(const MassArgs& a, unsigned blocks, hipStream_t st) {
  if (a.slopes && a.cap != 0.f) launch_mode<HALF, D, kCapped | kBiased>(a, blocks, st);
  else if (a.slopes) launch_mode<HALF, D, kBiased>(a, blocks, st);
  else if (a.cap != 0.f) launch_mode<HALF, D, kCapped>(a, blocks, st);
  else launch_mode<HALF, D, 0>(a, blocks, st);
}
template <bool HALF>
void launch_type(const MassArgs& a, unsigned blocks, hipStream_t st) {
  if (a.d == 64) launch_dim<HALF, 64>(a, blocks, st);
  else if (a.d == 128) launch_dim<HALF, 128>(a, blocks, st);
  else launch_dim<HALF, 256>(a, blocks, st);
}

}  // namespace

// 16 rows a sequence on average and fewer, or queries whose rows lie further apart than the
// other kernel's 32-bit offsets reach over a step of 64 rows. How the queries are spread over the
// sequences is known on the device alone, so a table with many more slots than sequences that ask
// is taken for a decode step (64 queries of 64 heads over 8192 keys of 8 heads of 128: 24 us with one
// slot, 62 with 64 of them).
bool mass_few(int64_t T, int64_t nseq, int group, int64_t q_ts, int64_t q_hs) {
  return (T + nseq - 1) / nseq * group <= 16 || q_ts >= (1 << 23) || q_hs >= (1 << 23);
}

// The chip holds some 512 workgroups. One takes some 4 us before its first product, the time
// of a few hundred rows. So what sees a tile of keys is split until the workgroups fill the chip
// once, with 128 rows of a sequence each and more, or four times, so that uneven ones even out,
// with 2048 (two prompts of 2000 tokens of 7 documents, d = 256: 54 us whole, 34 with 512
// workgroups, 40 with 1024; 8192 causal tokens: 1522 us whole, 669 with 1024, 634 with 2048, 654
// with 4096; windows of 64 queries behind 32K keys, 2048 workgroups: 98 us whole, 124 in two).
int mass_splits(int64_t T, int64_t nseq, int heads, int group, int64_t Lmax, int d) {
  const int64_t tiles = (Lmax + many_keys(d) - 1) / many_keys(d) * nseq * heads, rows = T * group / nseq;
  int s = 1;
  while (s < 64 && ((tiles * s < 512 && rows > 256 * s) || (tiles * s < 2048 && rows > 4096 * s))) s *= 2;
  return s;
}

int64_t mass_blocks(const MassArgs& a) {
  const int64_t keys = a.few ? kFewKeys : many_keys(a.d), units = (a.kv.Lmax + keys - 1) / keys * a.kv.nseq * a.Hkv;
  return a.few ? (units + kThreads / 64 - 1) / (kThreads / 64) : units * a.splits;
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
