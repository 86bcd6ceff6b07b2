// Attention over a paged cache.
//
// A row is one (query, head) pair; its score of the visible key s is
//   x = scale q.k_s,  then cap tanh(x / cap),  then - slope |position - s|,
// and its result sum_s e^(x_s - m) v_s / sum_s e^(x_s - m). The sums are kept
// against the running maximum m and rescaled when it grows, so that the keys
// are read once. Scores, m and both sums are fp32; the weights e^(x - m) are
// rounded to the cache's 16-bit type (to nearest) for the second product, whose
// sums are fp32 again, while the sum of the weights adds the unrounded ones.
// Rounded, they take one product. A second one of what the rounding left would
// halve its share of the output's error (decode of 8 x 32768: 0.0023 of the output in
// bf16, of which the result's own rounding is 0.0016; fp16 0.00027 and 0.00021), but
// takes prompts 13 to 33% longer (8192 tokens 1.17 -> 1.52 ms; steps of 4 and 8
// queries 1 to 2%, single queries nothing), and a remainder below zero makes a NaN of
// an infinite value.
//
// A workgroup takes a tile of R rows that read one kv head (the heads of a
// group, of one or several queries of a sequence) and a run of their keys:
// RW waves split the rows (MR = 16 or 32 a wave), KW groups of waves split the
// keys, NK at a time. Both products are MFMAs with the keys or the values as
// the first operand and the queries or weights as the second one:
//   S^T [keys x rows] = K Q^T,   O^T [d x rows] += V^T P^T.
// A lane then holds scores of ONE row (its column), so the maximum and the sum
// are sums over its registers and one or two lane exchanges, the rescaling is a
// product by a lane's own factor, and the weights already lie where the second
// product wants them: the order of the keys within a product is free, so the
// lane's own score registers are its share of P^T, and V^T is read to match by
// transposing LDS reads (ds_read_b64_tr_b16: 16 lanes read a 4 x 16 block of
// 16-bit values and each gets one column).
//
// Keys and values go through LDS: while one tile is used, the next one's rows
// are on their way into registers and the page ids of the tile after it are
// looked up. The 16-byte pieces of a row are permuted by the row's low bits
// (swizzle) so that neither the row-wise nor the transposing reads meet in a bank
// (counted: none at 8192 tokens).
//
// Batches of up to kPlanMax queries are planned: every workgroup sums the key
// tiles of all segments (runs of queries of one sequence that share a row
// tile), and the flat list of (segment, head tile, key tile) is cut into G
// equal runs, so that a ragged batch loads all CUs evenly. A segment that a cut
// divides leaves unfinished parts, at most two a workgroup, which a second
// launch joins in a fixed order. Larger batches take one workgroup per row tile.
//
// What bounds it (MI355X; a large copy moves 5.07 TB/s, a large bf16 product runs at
// 1.29 PFLOP/s). Decode: memory; 8 sequences of up to 32768 tokens, 64 / 8 heads of
// 128, read at 5.1 TB/s (145 us). Prompts: vector instructions; 8192 causal tokens
// with capped scores take 1.37 ms, 0.80 PFLOP/s. A tile of 32 rows x 64 keys costs a
// wave 1024 cycles of MFMA and some 1600 of vector issue (polynomial cap, exp2, sums,
// rounding), and the two waves of a SIMD overlap little: 34% and 52% of the cycles.
// Three waves a SIMD (spills at 168 registers), halves of the keys a step, the score
// product split over two accumulators, and wave priorities around the products were
// each measured slower or the same.
#pragma once

#include <type_traits>

#include "misa_attend.hpp"
#include "misa_common.hpp"

namespace misa {
namespace attend {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <bool HALF>
__device__ __forceinline__ floatx16 mfma32(const u32x4& a, const u32x4& b, const floatx16& c) {
  if (HALF)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <bool HALF>
__device__ __forceinline__ floatx4 mfma16(const u32x4& a, const u32x4& b, const floatx4& c) {
  if (HALF)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(halfx8, a), __builtin_bit_cast(halfx8, b), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two fp32 values in 16 bits each, to nearest, ties to even.
template <bool HALF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (HALF)
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 r;
  r[0] = (__bf16)lo;
  r[1] = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, r);
}

// What a kernel does to the scores besides the scale.
enum Mode : int {
  kPlain = 0,
  kCap = 1,    // a cap up to kPlainCap
  kBias = 2,   // anything
};

// Tile shapes. NK keys per group of waves and step; KT = KW * NK keys a step.
// With RW = 1 a wave's keys are its own: one LDS buffer and no barrier in the
// loop (8 x 32768 tokens of decode: 148 us, 175 with barriers and one workgroup a
// CU). Otherwise the RW waves of a group share them, in two buffers. Tiles of 64
// rows split the keys over two groups of waves: one group of four waves of 16 rows
// took 264 us for the selected prompt (2048 queries x 2048 tokens, 64 heads), one of
// two waves 301, two of two 238. At d = 256 tiles of 32 rows take two waves of 16:
// a wave of 32 rows holds 128 output registers and spills (139 -> 78 us for 4 x 4
// queries of 16384 tokens).
template <int D, int R>
struct Shape {
  static_assert(D < 256 || R > 16, "head dimension 256 takes tiles of 32 rows and more");
  static constexpr int MR = R == 16 || (D == 256 && R == 32) ? 16 : 32;
  static constexpr int RW = R / MR;
  static constexpr int KW = RW >= 4 ? 1 : 4 / RW;
  static constexpr int NK = D == 256 ? 32 : (D == 128 ? (R == 128 ? 64 : 32) : 64);
  static constexpr int waves = D == 256 ? 1 : 2;   // a SIMD, by their registers
  static constexpr int KT = KW * NK;
  static constexpr int WR = NK / RW;     // rows of a step that each wave loads
  static constexpr int threads = 64 * RW * KW;
  static constexpr int buffers = RW == 1 ? 1 : 2;
  static constexpr int stage_bytes = KT * D * 2 * 2;
  // the keys' waves join their sums through LDS: rows of D + 4 floats
  static constexpr int merge_bytes = KW > 1 ? KW * R * (D + 4) * 4 + KW * R * 8 + R * 8 : 0;
  static constexpr int lds_bytes = buffers * stage_bytes > merge_bytes ? buffers * stage_bytes : merge_bytes;
  // workgroups that fit a CU: 160 KiB of LDS (the plan's share included), and the
  // waves that their registers allow
  static constexpr int by_lds = 160 * 1024 / (lds_bytes + kPlanMax * 20 + 64), by_waves = waves * 256 / threads;
  static constexpr int per_cu = by_lds < 1 ? 1 : (by_lds < by_waves ? by_lds : by_waves);
};

// 16-byte piece c of row r lies at piece c ^ swizzle(r) of its row in LDS. The
// row-wise reads (16 or 32 rows, one piece each) and the transposing ones (four
// consecutive rows, four pieces each) then spread over all 64 banks.
template <int D>
__device__ __forceinline__ int swizzle(int r) {
  if (D == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  return ((r & 3) << 2) | ((r >> 2) & 3);
}

// Zeros that stand in for a row without a key.
static __device__ __align__(16) const uint32_t kZeroRow[128] = {};

// A row unit that stands for no key: beyond every buffer view, its pieces included.
constexpr uint32_t kNoRow = 0xffff8000u;

struct QueryInfo {
  int seq;        // row of the table, -1: none
  int lo, hi;     // visible tokens of that row
  int kbase;      // position of its token 0
  int pos;        // position of the query
};

__device__ __forceinline__ int clamp_len(int64_t v, int64_t most) { return (int)(v < 0 ? 0 : (v > most ? most : v)); }

__device__ __forceinline__ QueryInfo query_info(const AttendArgs& a, int64_t t) {
  // all loads first: they wait for nothing but t
  const bool prefix = a.mode == kAttendPrefix;
  const int own = (prefix ? a.own_seq : a.q_seq)[t];
  const int len = a.q_len[t];
  int start = 0, pos = 0, pre = -1;
  if (a.q_start) start = a.q_start[t];
  if (a.q_pos) pos = a.q_pos[t];
  if (a.mode != kAttendPlain) pre = a.pre[t];
  const bool ok = own >= 0 && own < (prefix ? a.own_nseq : a.kv.nseq);
  int plen = 0;
  if (pre >= 0 && pre < a.npre) plen = clamp_len(a.pre_len[pre], a.pre_max);
  else pre = -1;
  QueryInfo r;
  r.lo = 0;
  if (prefix) {
    r.seq = ok ? pre : -1;
    r.hi = r.seq >= 0 ? plen : 0;
    r.kbase = 0;
  } else {
    r.seq = ok ? own : -1;
    r.hi = ok ? clamp_len(len, a.kv.Lmax) : 0;
    r.lo = start < 0 ? 0 : (start > r.hi ? r.hi : start);
    r.kbase = plen;
  }
  r.pos = a.q_pos ? pos : plen + len - 1;
  return r;
}

// Key tiles of KT keys that a segment of queries visits (at least one, so that
// a segment without keys still writes its rows).
__device__ __forceinline__ int tiles_of(int lo, int hi, int KT) { return hi > lo ? (hi - lo + KT - 1) / KT : 1; }

// Values that are the same in all lanes, as scalars.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  return (int64_t)(uint32_t)uniform((int)(uint32_t)v) | (int64_t)uniform((int)(v >> 32)) << 32;
}

// The launch's arguments, read anew: what was loaded from them before need not
// stay in scalar registers.
typedef const __attribute__((address_space(4))) AttendArgs* ArgPtr;
__device__ __forceinline__ const AttendArgs& fresh(ArgPtr p) {
  asm volatile("" : "+s"(p));
  return *(const AttendArgs*)p;
}

// Work of a part of a segment.
struct Part {
  int64_t t0;      // first query
  int nq;          // queries
  int hh;          // kv head * head_tiles + head tile
  int tile0, tile1;   // key tiles of it
  bool whole;      // all of the segment's
  int slot;        // unfinished parts: where they are kept
};

// Reductions over a wave by data-parallel moves (rows of 16 lanes, then from row
// to row); the result, of lane 63, as a scalar. A shuffle through LDS costs some
// 130 cycles a step, and a part begins with eight of these.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_max(int v) {
  return max(v, __builtin_amdgcn_update_dpp((int)0x80000000, v, CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ int wave_max_of(int v) {
  v = dpp_max<0x111, 0xf>(v);   // from 1, 2, 4, 8 lanes below in the row
  v = dpp_max<0x112, 0xf>(v);
  v = dpp_max<0x114, 0xf>(v);
  v = dpp_max<0x118, 0xf>(v);
  v = dpp_max<0x142, 0xa>(v);   // lane 15 of a row to the next row
  v = dpp_max<0x143, 0xc>(v);   // lane 31 to the upper half
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ int wave_min_of(int v) { return ~wave_max_of(~v); }

// What a workgroup keeps of its queries (of the whole batch where it is planned)
// in LDS: entry t - t0 for query t.
struct Interval {
  int seq, lo, hi;
  int pos;          // position relative to the row's token 0
};
struct Known {
  Interval* at;
  int64_t t0;
  __device__ __forceinline__ const Interval& operator[](int64_t t) const { return at[(int)(t - t0)]; }
};
__device__ __forceinline__ Interval interval_of(const AttendArgs& a, int64_t t) {
  const QueryInfo q = query_info(a, t);
  return Interval{q.seq, q.lo, q.hi, q.pos - q.kbase};
}

// Sequence and span of the visible keys of queries t0 .. t0 + nq - 1 (one sequence).
struct Span {
  int seq, lo, hi;   // keys that any of them sees lie in [lo, hi)
  int some;          // keys that all of them see
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, const Known& known, int64_t t0, int nq) {
  const int lane = threadIdx.x & 63;
  Span s;
  if (nq == 1) {
    const Interval r = known[t0];
    s.seq = uniform(r.seq);
    s.lo = uniform(r.lo);
    s.hi = uniform(r.hi);
    if (a.idx) {
      s.hi = s.hi > s.lo ? a.topk : 0;
      s.lo = 0;
    }
    if (s.hi <= s.lo) s.lo = s.hi = 0;
    s.some = s.hi - s.lo;
    s.lo &= -a.align;
    return s;
  }
  int lo = 0x7fffffff, hi = 0, seq = -1, all_lo = 0, all_hi = 0x7fffffff;
  for (int i = lane; i < nq; i += 64) {
    const Interval r = known[t0 + i];
    seq = max(seq, r.seq);
    if (r.hi > r.lo) {
      lo = min(lo, r.lo);
      hi = max(hi, r.hi);
    }
    all_lo = max(all_lo, r.lo);
    all_hi = min(all_hi, r.hi);
  }
  s.seq = wave_max_of(seq);
  s.lo = wave_min_of(lo);
  s.hi = wave_max_of(hi);
  if (s.hi <= s.lo) s.lo = s.hi = 0;
  s.some = wave_min_of(all_hi) - wave_max_of(all_lo);
  s.lo &= -a.align;
  return s;
}

// tanh(y) for |y| <= kNear as y times a polynomial in y^2, fitted to 6e-8 of the
// value (one half step of fp32).
constexpr float kNear = 0.35f;
constexpr float kTanh[4] = {0.9999999403953552f, -0.33332425355911255f, 0.13295884430408478f, -0.04896282404661179f};
// Smaller values need one term less for the same error. A prompt of 8192 tokens takes
// 1360 us where all scores are that small, 1408 where they pass kNearest, 1515 where
// they pass kNear, and 1165 without a cap.
constexpr float kNearest = 0.18f;
constexpr float kTanh2[3] = {0.9999999403953552f, -0.3333021402359009f, 0.13075149059295654f};

// Caps up to this one take 1 - 2 / (1 + e^2y) for all scores of a run of keys that
// every row sees whole, where one of them is beyond kNear or the cap goes with a
// distance bias: exp2, the sum and the reciprocal lose at most 9 half steps of fp32
// of one, times the cap (1.4e-4 of a score at the limit, 3e-5 at 50), for rows that
// see these 32 keys at least. Larger caps, runs that are seen in part and the
// guarded form choose for each score. Choosing everywhere: an 8192-token prompt with
// scores up to the cap 1525 -> 1846 us.
constexpr float kPlainCap = 256.f;

// The cap in units of log2 for scores of |y| <= kNear: x P(x^2), y = c x.
struct NearCap {
  float k0, k1, k2, k3;
  __device__ __forceinline__ float factor(float x) const {
    const float z = x * x;
    return k0 + z * (k1 + z * (k2 + z * k3));
  }
};
__device__ __forceinline__ NearCap near_cap(float cap, float c) {
  const float g = cap * kLog2e * c, c2 = c * c;
  return NearCap{g * kTanh[0], g * kTanh[1] * c2, g * kTanh[2] * c2 * c2, g * kTanh[3] * c2 * c2 * c2};
}
struct NearestCap {
  float k0, k1, k2;
  __device__ __forceinline__ float factor(float x) const {
    const float z = x * x;
    return k0 + z * (k1 + z * k2);
  }
};
__device__ __forceinline__ NearestCap nearest_cap(float cap, float c) {
  const float g = cap * kLog2e * c, c2 = c * c;
  return NearestCap{g * kTanh2[0], g * kTanh2[1] * c2, g * kTanh2[2] * c2 * c2};
}
// The cap in units of log2, less off, for any score.
struct FarCap {
  float cap2, e, c;
  bool choose;        // a large cap: per score
  __device__ __forceinline__ float plain(float x, float off) const {
    return (cap2 - off) - 2.f * cap2 * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * e));
  }
  __device__ __forceinline__ float chosen(float x, float off) const {
    const float y = x * c, z = y * y;
    const float small = y * (kTanh[0] + z * (kTanh[1] + z * (kTanh[2] + z * kTanh[3])));
    float big = plain(x, off);
    asm("" : "+v"(big));   // both, then a select: a branch for each score costs more
    return fabsf(y) < kNear ? cap2 * small - off : big;
  }
};
__device__ __forceinline__ FarCap far_cap(float cap, float c) {
  return FarCap{cap * kLog2e, c * (2.f * kLog2e), c, cap > kPlainCap};
}
// the coefficients stay normal numbers for c in this range
__device__ __forceinline__ bool near_cap_holds(float c) { return c > 1e-4f && c < 1e4f; }

// A finished row: sums relative to 2^m (m in units of log2) to the result and its log-sum.
template <bool HALF, int D>
__device__ __forceinline__ void write_row(const AttendArgs& a, int64_t row, int d0, float m, float sum, floatx4 o) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;   // a row without a key: zeros
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= inv;
  if (a.out) {
    u32x2 w;
    w[0] = pack2<HALF>(o[0], o[1]);
    w[1] = pack2<HALF>(o[2], o[3]);
    *reinterpret_cast<u32x2*>(a.out + row * D + d0) = w;
  } else {
    *reinterpret_cast<floatx4*>(a.out32 + row * D + d0) = o;
  }
  if (d0 == 0 && a.lse) a.lse[row] = sum == 0.f ? -__builtin_inff() : (m + __log2f(sum)) * kLn2;
}

template <bool HALF, int D, int R, int MODE, bool ALIGNED, bool GUARD>
struct Kernel {
  using S = Shape<D, R>;
  static constexpr int MR = S::MR, RW = S::RW, KW = S::KW, NK = S::NK, KT = S::KT, WR = S::WR, TH = S::threads;
  static constexpr int RPI = 512 / D;              // rows a wave's load instruction covers
  static constexpr int LPR = D / 8;                // lanes (16-byte pieces) per row
  static constexpr int NLD = NK / RW / RPI;        // load instructions per tensor, wave and step
  static constexpr int QF = D * MR / 512;          // query fragments: d / 16 or d / 32 products deep
  static constexpr int OT = D / MR;                // output tiles of MR dims
  static constexpr int KS = 32;                    // keys of a step that are taken at a time
  static constexpr int NS = NK / KS;
  static constexpr int ST = KS / MR;               // score tiles of MR keys
  static constexpr int AR = MR * MR / 64;          // accumulator registers of a tile: 16 or 4
  static_assert(NLD >= 1 && NK % MR == 0, "tile shape");
  // The values of a run of keys are read from LDS before its weights are worked out
  // (selected prompt 237 -> 224 us) where the registers hold them: the other shapes
  // and forms would spill.
  static constexpr bool AHEAD = !GUARD && (D == 64 || (D == 256 ? R == 32 : R == 16 || (R == 64 && MODE == kPlain) ||
                                                                               (R == 128 && (ALIGNED || MODE == kPlain))));
  using Acc = typename std::conditional<MR == 32, floatx16, floatx4>::type;

  __device__ static __forceinline__ Acc mma(const u32x4& x, const u32x4& y, const Acc& c) {
    if constexpr (MR == 32) return mfma32<HALF>(x, y, c);
    else return mfma16<HALF>(x, y, c);
  }
  // key (or output dim) within a tile that accumulator register j of this lane holds
  __device__ static __forceinline__ int acc_row(int j, int lane) {
    if constexpr (MR == 32) return 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
    else return 4 * (lane >> 4) + j;
  }

  struct Rows {     // a lane's row
    int lo, hi;     // visible keys
    float slope;
    int pos;        // position - kbase
  };
  // Query and head of row r of a part's tile; false: no such row.
  __device__ static __forceinline__ bool row_of(const AttendArgs& a, const Part& p, int r, int64_t& t, int& head) {
    const int kvh = p.hh / a.head_tiles, hb = p.hh % a.head_tiles;
    const int qi = (int)fast_quot(a.by_gw, (uint32_t)r);
    head = kvh * a.group + hb * a.gw + (r - qi * a.gw);
    t = p.t0 + qi;
    return qi < p.nq && head < (kvh + 1) * a.group;
  }

  struct Stage {        // a step's rows on their way to LDS
    u32x4 k[NLD], v[NLD];
    uint64_t valid;     // keys that there are
    int token;          // this lane's key
  };

  // The keys of one step for one group of waves: lane l looks up key l, in three
  // steps of the loop: its token (the key's number, or a selected id), the table
  // entry of its page, and its row. A load is issued in one step and used in the
  // next, so none is waited for.
  struct Keys {
    int token;        // -1: none
    int within;       // its row of the page
    int page;
  };
  // token of the lane's key s + lane (before `end`; selected ids still unchecked)
  __device__ static __forceinline__ int token_of(const int32_t* ids, int s, int end) {
    const int lane = threadIdx.x & 63;
    const int at = s + lane;
    const bool in = lane < NK && at < end;
    if (!ids) return in ? at : -1;
    const int id = ids[min(at, end - 1)];
    return in ? id : -1;
  }
  __device__ static __forceinline__ Keys page_of(const KvView& kv, const int32_t* table, int seq, int token, int lo, int hi) {
    Keys k;
    k.token = token >= lo && token < hi ? token : -1;
    const uint32_t t = (uint32_t)max(k.token, 0);
    const uint32_t col = fast_quot(kv.by_page, t);
    k.within = (int)(t - col * (uint32_t)kv.page);
    k.page = table ? table[col] : seq;
    return k;
  }
  // where the row lies, in the view's units; kNoRow: no key
  __device__ static __forceinline__ uint32_t row_unit(const KvView& kv, const Keys& k) {
    const uint32_t at = (uint32_t)k.page * kv.page_units + (uint32_t)k.within * kv.tok_units;
    return k.token >= 0 && (uint32_t)k.page < (uint32_t)kv.npages ? at : kNoRow;
  }

  // Bases of one kv head's rows. Caches of less than 4 GiB (to the last row) are
  // read through buffer views with 32-bit byte offsets, whose range check gives
  // zeros for kNoRow; others by 64-bit addresses, with zeros kept for such rows.
  struct Bases {
    const uint16_t *k, *v;
    __amdgpu_buffer_rsrc_t kb, vb;
    uint32_t shift;   // 64-bit addresses: log2 of a unit's elements; 0: byte offsets
  };
  __device__ static __forceinline__ Bases bases_of(const KvView& kv, int kvh) {
    const int64_t off = (int64_t)kvh * kv.head_stride;
    Bases b;
    b.k = kv.k + off;
    b.v = kv.v + off;
    b.shift = kv.unit_shift;
    const uint32_t bytes = kv.unit_shift ? 0u : (uint32_t)(kv.bytes - off * 2);
    b.kb = buffer_view(b.k, bytes);
    b.vb = buffer_view(b.v, bytes);
    return b;
  }
  __device__ static __forceinline__ u32x4 buffer_row(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
  }

  // Loads of this wave's rows: instruction i covers rows i * RPI + lane / LPR of
  // its WR, whose units are given.
  __device__ static __forceinline__ void load_units(const Bases& b, const uint32_t (&unit)[NLD], int rw, u32x4 (&kr)[NLD],
                                                    u32x4 (&vr)[NLD]) {
    const int lane = threadIdx.x & 63;
    if (b.shift == 0) {
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const uint32_t at = unit[i] + 16 * ((lane % LPR) ^ swizzle<D>(rw * WR + i * RPI + lane / LPR));
        kr[i] = buffer_row(b.kb, at);
        vr[i] = buffer_row(b.vb, at);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const int c = 8 * ((lane % LPR) ^ swizzle<D>(rw * WR + i * RPI + lane / LPR));
        const uint16_t* z = reinterpret_cast<const uint16_t*>(kZeroRow);
        const uint64_t at = (uint64_t)unit[i] << b.shift;
        kr[i] = *reinterpret_cast<const u32x4*>((unit[i] != kNoRow ? b.k + at : z) + c);
        vr[i] = *reinterpret_cast<const u32x4*>((unit[i] != kNoRow ? b.v + at : z) + c);
      }
    }
  }
  __device__ static __forceinline__ void load_rows(const Bases& b, uint32_t unit, int rw, u32x4 (&kr)[NLD], u32x4 (&vr)[NLD]) {
    const int lane = threadIdx.x & 63;
    uint32_t u[NLD];
#pragma unroll
    for (int i = 0; i < NLD; ++i) u[i] = (uint32_t)__shfl((int)unit, rw * WR + i * RPI + lane / LPR, 64);
    load_units(b, u, rw, kr, vr);
  }

  // Aligned pages (of a cache that ends before 4 GiB): a step's keys start at a
  // multiple of WR, which divides the page, so that each wave's WR rows lie in one
  // page. Lane j looks up the page of wave j's rows (every wave has to know which of
  // them are keys); a wave's own page is then a scalar, and its rows follow each
  // other. It spares the shuffles and most of the arithmetic of the general look-up
  // (8192-token capped prompt 1.65 -> 1.53 ms).
  __device__ static __forceinline__ int page_entry(const KvView& kv, const int32_t* table, int seq, int base, int end) {
    const int lane = threadIdx.x & 63;
    const int s = min(base + (lane & (RW - 1)) * WR, end - 1);
    return table ? table[fast_quot(kv.by_page, (uint32_t)s)] : seq;
  }
  // Where this lane's pieces lie behind the first of its wave's rows (byte offsets).
  __device__ static __forceinline__ void piece_offsets(const KvView& kv, int rw, uint32_t (&piece)[NLD]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int r = i * RPI + lane / LPR;
      piece[i] = (uint32_t)r * kv.tok_units + 16 * ((lane % LPR) ^ swizzle<D>(rw * WR + r));
    }
  }
  __device__ static __forceinline__ uint64_t load_aligned(const KvView& kv, const Bases& b, const uint32_t (&piece)[NLD], int entry,
                                                          int base, int end, int rw, u32x4 (&kr)[NLD], u32x4 (&vr)[NLD]) {
    const int lane = threadIdx.x & 63;
    const bool ok = (uint32_t)entry < (uint32_t)kv.npages && base + (lane & (RW - 1)) * WR < end;
    const uint32_t bits = (uint32_t)__ballot(ok) & ((1u << RW) - 1);
    const int s0 = base + rw * WR;
    const uint32_t page = (uint32_t)__builtin_amdgcn_readlane(entry, rw);
    const uint32_t within = (uint32_t)s0 - fast_quot(kv.by_page, (uint32_t)s0) * (uint32_t)kv.page;
    const uint32_t first = page * kv.page_units + within * kv.tok_units;
    const int rows = (bits >> rw & 1) ? end - s0 : 0;
    if (rows >= WR) {
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        kr[i] = buffer_row(b.kb, first + piece[i]);
        vr[i] = buffer_row(b.vb, first + piece[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NLD; ++i) {
        const uint32_t at = i * RPI + lane / LPR < rows ? first + piece[i] : kNoRow;
        kr[i] = buffer_row(b.kb, at);
        vr[i] = buffer_row(b.vb, at);
      }
    }
    uint64_t valid = ~0ull;
    if (bits != (1u << RW) - 1) {
      valid = 0;
#pragma unroll
      for (int j = 0; j < RW; ++j) valid |= (bits >> j & 1) ? ((WR == 64 ? 0ull : 1ull << (WR & 63)) - 1) << (j * WR) : 0;
    }
    return NK == 64 ? valid : valid & ((1ull << (NK & 63)) - 1);
  }
  __device__ static __forceinline__ void store_rows(uint16_t* ks, uint16_t* vs, int rw, const u32x4 (&kr)[NLD],
                                                    const u32x4 (&vr)[NLD]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NLD; ++i) {
      const int at = (rw * NLD + i) * RPI * D + lane * 8;
      *reinterpret_cast<u32x4*>(ks + at) = kr[i];
      *reinterpret_cast<u32x4*>(vs + at) = vr[i];
    }
  }

  // Orders the LDS accesses of the waves that share rows: a barrier, or, within
  // one wave (whose LDS instructions run in order), the compiler's alone.
  __device__ static __forceinline__ void sync_rows() {
    if constexpr (RW > 1) {
      __syncthreads();
    } else {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
  }

  // LDS addresses. A piece's place is its row's start with the piece number XORed
  // by the row's swizzle, so the places of one row differ from a base by an XOR
  // with a constant. The bases are made anew for each run of keys (opaque to the
  // compiler): kept in the loop, the 16 to 24 places of a lane would take as many
  // registers as its output tile.
  typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
  typedef __attribute__((address_space(3))) shortx4 lds_shortx4;
  __device__ static __forceinline__ uint32_t lds_address(const uint16_t* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint16_t*)p;
  }
  __device__ static __forceinline__ u32x4 read_lds(uint32_t at) {
    const u32x4 v = *(lds_u32x4*)(uintptr_t)at;
    return v;
  }
  __device__ static __forceinline__ uint32_t key_base(const uint16_t* ks) {
    const int lane = threadIdx.x & 63;
    const int r = lane % MR;
    uint32_t b = lds_address(ks) + r * (2 * D) + 16 * ((lane / MR) ^ swizzle<D>(r));
    asm volatile("" : "+v"(b));
    return b;
  }
  // the operand K of KS keys
  __device__ static __forceinline__ void key_frags(const uint16_t* ks, u32x4 (&kf)[QF][ST]) {
    const uint32_t b = key_base(ks);
#pragma unroll
    for (int f = 0; f < QF; ++f)
#pragma unroll
      for (int i = 0; i < ST; ++i)   // 16 rows further on the swizzle is the same
        kf[f][i] = read_lds((b ^ (f * (64 / MR) * 16)) + i * MR * 2 * D);
  }
  // scores of KS keys: S^T tiles of this wave's rows
  __device__ static __forceinline__ void score(const u32x4 (&kf)[QF][ST], const u32x4 (&qf)[QF], Acc (&s)[ST]) {
#pragma unroll
    for (int i = 0; i < ST; ++i)
#pragma unroll
      for (int j = 0; j < AR; ++j) s[i][j] = 0.f;
#pragma unroll
    for (int f = 0; f < QF; ++f)
#pragma unroll
      for (int i = 0; i < ST; ++i) s[i] = mma(kf[f][i], qf[f], s[i]);
  }

  // Base of the transposing reads: 16 lanes read 4 rows (keys) of 16 dims, 4 values
  // each, and get one dim of the 4 keys.
  __device__ static __forceinline__ uint32_t value_base(const uint16_t* vs) {
    const int lane = threadIdx.x & 63;
    const int r = (MR == 32 ? 4 * (lane >> 5) : 4 * (lane >> 4)) + ((lane & 15) >> 2);
    const int piece = (MR == 32 ? (lane & 16) >> 3 : 0) + ((lane & 3) >> 1);
    uint32_t b = lds_address(vs) + r * (2 * D) + 16 * (piece ^ swizzle<D>(r)) + 8 * (lane & 1);
    asm volatile("" : "+v"(b));
    return b;
  }
  __device__ static __forceinline__ u32x2 read_tr(uint32_t at) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_shortx4*)(uintptr_t)at));
  }

  // The halves of x without infinities and NaNs.
  __device__ static __forceinline__ uint32_t finite_only(uint32_t x) {
    constexpr uint32_t e = HALF ? 0x7c00u : 0x7f80u;
    return x & (((x & e) == e ? 0u : 0xffffu) | ((x & (e << 16)) == (e << 16) ? 0u : 0xffff0000u));
  }

  // The operand V^T of product p, output tile i: MR == 32: keys 16 p + 4 (lane / 32)
  // + 0..3 and 8 further (another swizzle); MR == 16: 32 p + 4 (lane / 16) + 0..3 and
  // 16 further (the same one).
  __device__ static __forceinline__ u32x4 value_frag(uint32_t base, int p, int i) {
    const uint32_t a = base ^ (i * (MR / 8) * 16);
    const u32x2 x = read_tr(a + p * (MR == 32 ? 16 : 32) * 2 * D);
    const u32x2 y = read_tr(MR == 32 ? (a ^ 32) + (16 * p + 8) * 2 * D : a + (32 * p + 16) * 2 * D);
    return u32x4{x[0], x[1], y[0], y[1]};
  }
  // The operand P^T of product p from this lane's score registers: MR == 32: 16
  // keys (registers 8 (p & 1) .. + 7 of tile p / 2); MR == 16: 32 keys (two tiles).
  __device__ static __forceinline__ u32x4 weight_frag(const Acc (&s)[ST], int p) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (MR == 32) w[i] = pack2<HALF>(s[p / 2][8 * (p & 1) + 2 * i], s[p / 2][8 * (p & 1) + 2 * i + 1]);
      else w[i] = pack2<HALF>(s[2 * p + i / 2][2 * (i & 1)], s[2 * p + i / 2][2 * (i & 1) + 1]);
    }
    return w;
  }
  static constexpr int NP = MR == 32 ? KS / 16 : KS / 32;

  // O^T += V^T P^T over KS keys
  __device__ static __forceinline__ void accumulate(const u32x4 (&vf)[NP][OT], const Acc (&s)[ST], Acc (&o)[OT]) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const u32x4 w = weight_frag(s, p);
#pragma unroll
      for (int i = 0; i < OT; ++i) o[i] = mma(vf[p][i], w, o[i]);
    }
  }

  __device__ static __forceinline__ void accumulate_now(const uint16_t* vs, const Acc (&s)[ST], Acc (&o)[OT]) {
    const uint32_t base = value_base(vs);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const u32x4 w = weight_frag(s, p);
#pragma unroll
      for (int i = 0; i < OT; ++i) o[i] = mma(value_frag(base, p, i), w, o[i]);
    }
  }

  // The same for a step of which some rows do not see every key, and whose values
  // are not all finite: the product would carry 0 * inf = NaN into rows that do
  // not see them. The finite values are multiplied as above; then, for +inf, -inf
  // and NaN in turn, a product of marks counts those that each row sees.
  __device__ static __forceinline__ void accumulate_guarded(const uint16_t* vs, Acc (&s)[ST], Acc (&o)[OT], uint32_t see) {
    const int lane = threadIdx.x & 63;
    const uint32_t base = value_base(vs);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const u32x4 w = weight_frag(s, p);
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        u32x4 v = value_frag(base, p, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = finite_only(v[e]);
        o[i] = mma(v, w, o[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < ST; ++i)
#pragma unroll
      for (int j = 0; j < AR; ++j) {
        s[i][j] = see >> (i * MR + acc_row(j, lane)) & 1 ? 1.f : 0.f;
      }
    constexpr uint32_t one = HALF ? 0x3c00u : 0x3f80u, inf = HALF ? 0x7c00u : 0x7f80u;
#pragma unroll 1
    for (int kind = 0; kind < 3; ++kind) {
      const float value = kind == 0 ? __builtin_inff() : kind == 1 ? -__builtin_inff() : __builtin_nanf("");
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        Acc n;
#pragma unroll
        for (int j = 0; j < AR; ++j) n[j] = 0.f;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          u32x4 v = value_frag(base, p, i);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t mark = 0;
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              const uint32_t x = (v[e] >> h) & 0xffffu;
              const bool is = kind == 0 ? x == inf : kind == 1 ? x == (inf | 0x8000u) : (x & 0x7fffu) > inf;
              mark |= is ? one << h : 0u;
            }
            v[e] = mark;
          }
          n = mma(v, weight_frag(s, p), n);
        }
#pragma unroll
        for (int j = 0; j < AR; ++j) o[i][j] = n[j] > 0.f ? o[i][j] + value : o[i][j];
      }
    }
  }

  // the largest magnitude of this lane's scores
  __device__ static __forceinline__ float largest(const Acc (&s)[ST]) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < ST; ++i)
#pragma unroll
      for (int j = 0; j < AR; ++j) big = fmaxf(big, fabsf(s[i][j]));
    return big;
  }
  __device__ static __forceinline__ float highest(const Acc (&s)[ST]) {
    float mx = s[0][0];
#pragma unroll
    for (int i = 0; i < ST; ++i)
#pragma unroll
      for (int j = 0; j < AR; ++j) mx = fmaxf(mx, s[i][j]);
    return mx;
  }

  // The exponent (of 2) that a row's weights and sums are relative to: its reference m
  // or, for weights in fp16, kLift below it. Those weights are then normal numbers down
  // to 2^-21 of the row's largest and zero below 2^-32 of it, not 2^-14 and 2^-25:
  // thousands of keys that small, beside one whose value is near zero, make the
  // result. The largest stays below 2^15: `follow` lets it pass 2^m by 2^8, and the
  // reference is rounded up by at least what m sc lost to rounding, which would
  // otherwise be a factor of all the row's weights (2^4 at the largest documented
  // scores, exponents of 2^26; rounded up it takes at most 2^12 from them there). The
  // range of bf16 holds that factor.
  static constexpr float kLift = HALF ? 7.f : 0.f;
  __device__ static __forceinline__ float reference(float m, float sc) {
    const float r = m * sc;
    return HALF && m != -__builtin_inff() ? __builtin_fmaf(fabsf(r), 0x1p-23f, r) - kLift : r;
  }
  __device__ static __forceinline__ float finite_reference(float m, float sc) {
    return m == -__builtin_inff() ? 0.f : reference(m, sc);
  }

  // Moves the reference m where a row's maximum mx (of this lane's row, over all of
  // its keys of the step) passes it by more than slack.
  __device__ static __forceinline__ void follow(float mx, float slack, float sc, float& m, float& sum, Acc (&o)[OT]) {
    if (!__any(mx - m > slack)) return;   // exact, however large they are
    const float mn = fmaxf(m, mx);
    const float alpha = __builtin_amdgcn_exp2f((m - (mn == -__builtin_inff() ? 0.f : mn)) * sc);
    sum *= alpha;
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int j = 0; j < AR; ++j) o[i][j] *= alpha;
    m = mn;
  }

  __device__ static __forceinline__ void cap_far(const FarCap& g, bool choose, float off, Acc (&s)[ST]) {
    if (GUARD || choose) {
#pragma unroll
      for (int i = 0; i < ST; ++i)
#pragma unroll
        for (int j = 0; j < AR; ++j) s[i][j] = g.chosen(s[i][j], off);
    } else {
#pragma unroll
      for (int i = 0; i < ST; ++i)
#pragma unroll
        for (int j = 0; j < AR; ++j) s[i][j] = g.plain(s[i][j], off);
    }
  }

  // Cap and bias. Capped scores leave in units of log2, others still without the
  // scale (the bias divided by it).
  __device__ static __forceinline__ void shape(const AttendArgs& a, Acc (&s)[ST], const Rows& row, const int32_t* ids, int base,
                                               int token, int sub, bool full) {
    const int lane = threadIdx.x & 63;
    if (a.cap > 0.f) {
      const float c = a.scale / a.cap;
      const FarCap g = far_cap(a.cap, c);
      cap_far(g, g.choose || !full, 0.f, s);
    }
    if (!a.slopes) return;
    const float slope = a.cap > 0.f ? row.slope * kLog2e : row.slope / a.scale;
    if (ids) {
#pragma unroll
      for (int i = 0; i < ST; ++i)
#pragma unroll
        for (int j = 0; j < AR; ++j)
          s[i][j] -= slope * fabsf((float)(row.pos - __shfl(token, sub * KS + i * MR + acc_row(j, lane), 64)));
    } else {
      const int first = row.pos - base - acc_row(0, lane);
      if (__any(first > (1 << 23) || first < -(1 << 23))) {
#pragma unroll
        for (int i = 0; i < ST; ++i)
#pragma unroll
          for (int j = 0; j < AR; ++j) s[i][j] -= slope * fabsf((float)(first - (i * MR + acc_row(j, 0))));
      } else {   // differences that fp32 holds exactly
        const float f = (float)first;
#pragma unroll
        for (int i = 0; i < ST; ++i)
#pragma unroll
          for (int j = 0; j < AR; ++j) s[i][j] -= slope * fabsf(f - (float)(i * MR + acc_row(j, 0)));
      }
    }
  }

  // Bits from b on of 32.
  __device__ static __forceinline__ uint32_t bits_from(int b) { return b >= 32 ? 0u : ~0u << (b > 0 ? b : 0); }
  // -inf for the scores of keys whose bit in `see` is not set.
  __device__ static __forceinline__ void hide(uint32_t see, Acc (&s)[ST]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      const uint32_t w = see >> (i * MR) >> acc_row(0, lane);
#pragma unroll
      for (int j = 0; j < AR; ++j) {
        // the bit as a mask of all bits: the score or the bits of -inf
        const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)w, acc_row(j, 0), 1);
        s[i][j] = __uint_as_float((__float_as_uint(s[i][j]) & keep) | (0xff800000u & ~keep));
      }
    }
  }

  // Over the lanes that hold a row (MR apart): the permutations swap rows of 16 or
  // 32 lanes between their two operands, so both halves come out for every lane.
  __device__ static __forceinline__ void halves(float v, bool by16, float& x, float& y) {
    const auto r = by16 ? __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false)
                        : __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    x = __uint_as_float(r[0]);
    y = __uint_as_float(r[1]);
  }
  __device__ static __forceinline__ float over_rows_max(float v) {
    float x, y;
    if constexpr (MR == 16) {
      halves(v, true, x, y);
      v = fmaxf(x, y);
    }
    halves(v, false, x, y);
    return fmaxf(x, y);
  }
  __device__ static __forceinline__ float over_rows_sum(float v) {
    float x, y;
    if constexpr (MR == 16) {
      halves(v, true, x, y);
      v = x + y;
    }
    halves(v, false, x, y);
    return x + y;
  }

  // Result or unfinished sums of row r (of the tile), dims d0 .. d0 + 3.
  // m in units of log2; sum and o relative to 2^m.
  __device__ static __forceinline__ void emit(const AttendArgs& a, const Part& p, int64_t t, int head, int r,
                                              int d0, float m, float sum, floatx4 o) {
    if (!p.whole) {
      *reinterpret_cast<floatx4*>(a.part_out + ((int64_t)p.slot * R + r) * D + d0) = o;
      if (d0 == 0) {
        a.part_ml[((int64_t)p.slot * R + r) * 2] = m;
        a.part_ml[((int64_t)p.slot * R + r) * 2 + 1] = sum;
      }
      return;
    }
    const int64_t row = t * a.Hq + head;
    write_row<HALF, D>(a, row, d0, m, sum, o);
  }

  // One part. A product with a value that is not finite leaves a NaN also in rows
  // that do not see it (0 * inf). Where the queries of a part do not see the same
  // keys (odd is not null) and anything comes out infinite or NaN, *odd is set
  // and the guarded form computes the workgroup's parts again.
  __device__ static __forceinline__ void run_part(ArgPtr ap, const Part& p, unsigned char* lds, const Known& known,
                                                  int* odd) {
    const AttendArgs& a = fresh(ap);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % RW, kw = wave / RW;
    const int kvh = p.hh / a.head_tiles;
    const Span sp = span_of(a, known, p.t0, p.nq);
    // p.tile1 * KT may pass the last key (and 2^31): 64 bits
    const int begin = sp.lo + p.tile0 * KT;
    const int end = (int)min((int64_t)sp.hi, sp.lo + (int64_t)p.tile1 * KT);
    const int steps = end > begin ? (end - begin + KT - 1) / KT : 0;

    // this lane's row
    const int r = rw * MR + lane % MR;
    int64_t row_t;
    int row_head;
    const bool active = row_of(a, p, r, row_t, row_head);
    Rows row;
    row.lo = row.hi = 0;
    row.slope = 0.f;
    row.pos = 0;
    if (active) {
      const Interval q = known[row_t];
      row.lo = a.idx ? 0 : q.lo;
      row.hi = a.idx ? a.topk : q.hi;
      row.pos = q.pos;
      if (MODE == kBias && a.slopes) row.slope = a.slopes[row_head];
    }
    // visible token ids of selected tokens (one query a segment; also for waves
    // without a row, which load for the others)
    const int32_t* ids = nullptr;
    int id_lo = 0, id_hi = 0x7fffffff;
    if (a.idx) {
      const Interval q = known[p.t0];
      ids = a.idx + p.t0 * a.topk;
      id_lo = uniform(q.lo);
      id_hi = uniform(q.hi);
    }
    // keys that every row of this wave sees, and keys that any of them sees
    const int all_lo = wave_max_of(active ? row.lo : 0);
    const int all_hi = wave_min_of(active ? row.hi : 0x7fffffff);
    const int any_lo = wave_min_of(active ? row.lo : 0x7fffffff);
    const int any_hi = wave_max_of(active ? row.hi : 0);

    u32x4 qf[QF];
    {
      const uint16_t* src = a.q + row_t * a.q_ts + row_head * a.q_hs + 8 * (lane / MR);
#pragma unroll
      for (int f = 0; f < QF; ++f) {
        if (active) qf[f] = *reinterpret_cast<const u32x4*>(src + f * (512 / MR));
        else qf[f] = u32x4{0u, 0u, 0u, 0u};
      }
    }

    float m = -__builtin_inff(), sum = 0.f;
    Acc o[OT];
#pragma unroll
    for (int i = 0; i < OT; ++i)
#pragma unroll
      for (int j = 0; j < AR; ++j) o[i][j] = 0.f;
    const float sc = MODE == kPlain || (MODE == kBias && a.cap == 0.f) ? a.scale * kLog2e : 1.f;

    uint16_t* buf = reinterpret_cast<uint16_t*>(lds);
    constexpr int GB = NK * D;             // elements of one tensor of one group's step
    constexpr int SB = KW * 2 * GB;        // of one buffer
    const Bases bases = bases_of(a.kv, kvh);
    const int32_t* table = a.kv.table ? a.kv.table + (int64_t)max(sp.seq, 0) * a.kv.table_stride : nullptr;
    const int k0 = begin + kw * NK;
    // steps of this wave: its own where no other shares its keys
    const int mine = RW > 1 ? steps : (end > k0 ? (end - k0 + KT - 1) / KT : 0);
    // rows on their way to LDS; what is looked up for them (tokens, pages) runs one
    // and two steps further ahead
    Stage stage;
    Keys nxt;
    nxt.token = -1;
    nxt.within = nxt.page = 0;
    int far = -1, entry = 0;
    uint32_t piece[NLD];
    auto fetch = [&](int it) __attribute__((always_inline)) {
      if constexpr (ALIGNED) {
        const int now = entry;
        entry = page_entry(a.kv, table, sp.seq, k0 + (it + 1) * KT, end);
        stage.valid = load_aligned(a.kv, bases, piece, now, k0 + it * KT, end, rw, stage.k, stage.v);
        stage.token = -1;
      } else {
        const uint32_t unit = row_unit(a.kv, nxt);
        stage.valid = __ballot(unit != kNoRow);
        stage.token = nxt.token;
        nxt = page_of(a.kv, table, sp.seq, far, id_lo, id_hi);
        far = token_of(ids, k0 + (it + 2) * KT, end);
        load_rows(bases, unit, rw, stage.k, stage.v);
      }
    };
    uint64_t valid = 0;
    int cur_token = -1;
    auto land = [&](int it) __attribute__((always_inline)) {
      uint16_t* to = buf + (S::buffers > 1 ? (it & 1) * SB : 0) + kw * 2 * GB;
      store_rows(to, to + GB, rw, stage.k, stage.v);
      valid = stage.valid;
      cur_token = stage.token;
    };
    if (mine > 0) {
      if constexpr (ALIGNED) {
        piece_offsets(a.kv, rw, piece);
        entry = page_entry(a.kv, table, sp.seq, k0, end);
      } else {
        const int first = token_of(ids, k0, end);
        far = token_of(ids, k0 + KT, end);
        nxt = page_of(a.kv, table, sp.seq, first, id_lo, id_hi);
      }
      fetch(0);
      land(0);
    }
    // the loop's first products wait for these loads here, not for its own
#pragma unroll
    for (int f = 0; f < QF; ++f) asm volatile("" : "+v"(qf[f]));
    // the maximum is followed lazily: the reference m moves when a row's maximum
    // passes it by more than 2^8, so that rescaling is rare after the first step
    const float slack = 8.f / sc;
    const float cap_c = MODE == kCap ? a.scale / a.cap : 0.f;
    const bool near_holds = near_cap_holds(cap_c);
    sync_rows();
    for (int it = 0; it < mine; ++it) {
      if (it + 1 < mine) fetch(it + 1);
      const uint16_t* ks = buf + (S::buffers > 1 ? (it & 1) * SB : 0) + kw * 2 * GB;
#pragma unroll
      for (int sub = 0; sub < NS; ++sub) {
        // one run of KS keys after the other: their registers are the same
        if (sub > 0) __builtin_amdgcn_sched_barrier(0);
        const int base = k0 + it * KT + sub * KS;
        const uint32_t have = (uint32_t)(valid >> (sub * KS));
        if (base >= any_hi || base + KS <= any_lo || have == 0) continue;
        Acc s[ST];
        u32x4 kf[QF][ST];
        key_frags(ks + sub * KS * D, kf);
        if (AHEAD) __builtin_amdgcn_sched_barrier(0);   // all reads first
        score(kf, qf, s);
        const uint16_t* vs = ks + GB + sub * KS * D;
        u32x4 vf[NP][OT];
        if constexpr (AHEAD) {
          const uint32_t vb = value_base(vs);
#pragma unroll
          for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int i = 0; i < OT; ++i) vf[n][i] = value_frag(vb, n, i);
        }
        if (AHEAD) __builtin_amdgcn_sched_barrier(0);
        const bool full = have == ~0u && base >= all_lo && base + KS <= all_hi;
        // the keys that the row sees: worked out only in tiles of which some are hidden
        // (8192-token prompt 1458 -> 1428 us; selected tokens, whose pages are not
        // aligned, 226 -> 229, so theirs are always)
        uint32_t see = ALIGNED ? 0u : have & bits_from(row.lo - base) & ~bits_from(row.hi - base);
        if constexpr (MODE == kBias) shape(a, s, row, ids, base, cur_token, sub, full);
        if (!full) {
          if (ALIGNED) see = have & bits_from(row.lo - base) & ~bits_from(row.hi - base);
          if constexpr (MODE == kCap) {
            // The ends of intervals, which may be all that a row sees: chosen per score,
            // before the maximum. The form's terms are made here: kept in the loop they
            // take its registers (d = 128, 32 rows a tile: 91 spilled, 10 like this; 4 x 4
            // queries of 16384 tokens 72 -> 57 us).
            float cap = a.cap, c = cap_c;
            asm volatile("" : "+s"(cap), "+v"(c));
            const FarCap g = far_cap(cap, c);
#pragma unroll
            for (int i = 0; i < ST; ++i)
#pragma unroll
              for (int j = 0; j < AR; ++j) {
                s[i][j] = g.chosen(s[i][j], 0.f);
                if (j % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // few scores' terms at a time
              }
          }
          hide(see, s);
        }
        float mx = over_rows_max(highest(s));
        if constexpr (MODE == kCap) {
          // the cap grows with the score, so where all keys are seen the maximum is
          // taken before it and the reference is subtracted in its last step
          bool near = near_holds && full, nearest = false;
          if (near) {
            const float big = largest(s) * cap_c;
            near = !__any(!(big <= kNear));
            nearest = !__any(!(big <= kNearest));
          }
          const NearCap f = near_cap(a.cap, cap_c);
          const FarCap g = far_cap(a.cap, cap_c);
          follow(!full ? mx : near ? mx * f.factor(mx) : g.plain(mx, 0.f), slack, sc, m, sum, o);
          const float off = finite_reference(m, sc);
          if (nearest) {
            const NearestCap f2 = nearest_cap(a.cap, cap_c);
#pragma unroll
            for (int i = 0; i < ST; ++i)
#pragma unroll
              for (int j = 0; j < AR; ++j) s[i][j] = __builtin_fmaf(s[i][j], f2.factor(s[i][j]), -off);
          } else if (near) {
#pragma unroll
            for (int i = 0; i < ST; ++i)
#pragma unroll
              for (int j = 0; j < AR; ++j) s[i][j] = __builtin_fmaf(s[i][j], f.factor(s[i][j]), -off);
          } else if (full) {
#pragma unroll
            for (int i = 0; i < ST; ++i)
#pragma unroll
              for (int j = 0; j < AR; ++j) s[i][j] = g.plain(s[i][j], off);
          } else {
#pragma unroll
            for (int i = 0; i < ST; ++i)
#pragma unroll
              for (int j = 0; j < AR; ++j) s[i][j] -= off;
          }
        } else {
          follow(mx, slack, sc, m, sum, o);
          const float off = finite_reference(m, sc);
#pragma unroll
          for (int i = 0; i < ST; ++i)
#pragma unroll
            for (int j = 0; j < AR; ++j) s[i][j] = s[i][j] * sc - off;
        }
        float add[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < ST; ++i)
#pragma unroll
          for (int j = 0; j < AR; ++j) {
            s[i][j] = __builtin_amdgcn_exp2f(s[i][j]);
            add[j & 1] += s[i][j];
          }
        sum += add[0] + add[1];
        if constexpr (GUARD) accumulate_guarded(vs, s, o, see);
        else if constexpr (AHEAD) accumulate(vf, s, o);
        else accumulate_now(vs, s, o);
      }
      if (S::buffers == 1) sync_rows();   // this wave has read what it now overwrites
      if (it + 1 < mine) land(it + 1);
      sync_rows();
    }
    finish(fresh(ap), p, sp, lds, odd, r, kw, reference(m, sc), sum, o);
  }

  // The end of a part: joins the groups of waves and writes the rows.
  __device__ static __forceinline__ void finish(const AttendArgs& a, const Part& p, const Span& sp, unsigned char* lds,
                                                int* odd, int r, int kw, float m, float sum,
                                                Acc (&o)[OT]) {
    const int lane = threadIdx.x & 63;
    if constexpr (!GUARD) {
      if (odd && sp.some < sp.hi - sp.lo) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
          for (int j = 0; j < AR; ++j) z = __builtin_fmaf(o[i][j], 0.f, z);
        if (z != z) *odd = 1;
      }
    }
    sum = over_rows_sum(sum);
    if constexpr (KW == 1) {
      int64_t t;
      int head;
      if (row_of(a, p, r, t, head)) {
#pragma unroll
        for (int i = 0; i < OT; ++i)
#pragma unroll
          for (int j = 0; j < AR; j += 4)
            emit(a, p, t, head, r, i * MR + acc_row(j, lane), m, sum,
                 floatx4{o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]});
      }
    } else {
      // join the groups of waves: maxima and sums first, then the scaled outputs
      float* ob = reinterpret_cast<float*>(lds);             // [KW][R][D + 4]
      float* ml = ob + KW * R * (D + 4);                     // [KW][R][2]
      float* fin = ml + KW * R * 2;                          // [R][2]
      __syncthreads();   // every wave is done with its rows
      if (lane < MR) {
        ml[(kw * R + r) * 2] = m;
        ml[(kw * R + r) * 2 + 1] = sum;
      }
      __syncthreads();
      float M = -__builtin_inff(), total = 0.f;
#pragma unroll
      for (int i = 0; i < KW; ++i) M = fmaxf(M, ml[(i * R + r) * 2]);
      const float ref = M == -__builtin_inff() ? 0.f : M;
#pragma unroll
      for (int i = 0; i < KW; ++i)
        total += ml[(i * R + r) * 2 + 1] * __builtin_amdgcn_exp2f(ml[(i * R + r) * 2] - ref);
      const float w = __builtin_amdgcn_exp2f(m - ref);
      if (kw == 0 && lane < MR) {
        fin[r * 2] = M;
        fin[r * 2 + 1] = total;
      }
#pragma unroll
      for (int i = 0; i < OT; ++i)
#pragma unroll
        for (int j = 0; j < AR; j += 4)
          *reinterpret_cast<floatx4*>(ob + (kw * R + r) * (D + 4) + i * MR + acc_row(j, lane)) =
              floatx4{o[i][j] * w, o[i][j + 1] * w, o[i][j + 2] * w, o[i][j + 3] * w};
      __syncthreads();
      for (int e = threadIdx.x; e < R * (D / 4); e += TH) {
        const int rr = e / (D / 4), d0 = (e % (D / 4)) * 4;
        int64_t t;
        int head;
        if (!row_of(a, p, rr, t, head)) continue;
        floatx4 x = *reinterpret_cast<const floatx4*>(ob + rr * (D + 4) + d0);
#pragma unroll
        for (int i = 1; i < KW; ++i) x += *reinterpret_cast<const floatx4*>(ob + (i * R + rr) * (D + 4) + d0);
        emit(a, p, t, head, rr, d0, fin[rr * 2], fin[rr * 2 + 1], x);
      }
      __syncthreads();   // the next part's first rows go to the same memory
    }
  }

  // Queries from t0 on that belong to t0's sequence and row tile.
  __device__ static __forceinline__ int run_length(const AttendArgs& a, const Known& known, int64_t t0) {
    const int lane = threadIdx.x & 63;
    int64_t end = (t0 / a.qt + 1) * a.qt;
    if (end > a.T) end = a.T;
    const int n = (int)(end - t0);
    if (n <= 1) return n;
    const int seq = known[t0].seq;
    for (int i = 0; i < n; i += 64) {
      const bool other = i + lane < n && known[t0 + i + lane].seq != seq;
      const uint64_t b = __ballot(other);
      if (b) return __builtin_amdgcn_readfirstlane(i + (int)__builtin_ctzll(b));
    }
    return n;
  }

  // Key tiles before each query's segment: cum[t] for t < T, and their sum; the
  // queries' intervals.
  __device__ static __forceinline__ int make_plan(const AttendArgs& a, int* cum, const Known& known) {
    const int T = (int)a.T, tid = threadIdx.x;
    for (int t = tid; t < T; t += TH) known.at[t] = interval_of(a, t);
    __syncthreads();
    constexpr int PER = kPlanMax / TH;       // queries a thread sums
    int w[PER];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int t = tid * PER + i;
      w[i] = 0;
      if (t < T) {
        const int seq = known[t].seq;
        if (t % a.qt == 0 || known[t - 1].seq != seq) {
          int lo = 0x7fffffff, hi = 0;
          const int last = min(T, (t / a.qt + 1) * a.qt);
          for (int u = t; u < last && known[u].seq == seq; ++u) {
            const Interval z = known[u];
            if (z.hi > z.lo) {
              lo = min(lo, z.lo);
              hi = max(hi, z.hi);
            }
          }
          if (a.idx && hi > lo) {
            lo = 0;
            hi = a.topk;
          }
          w[i] = tiles_of(lo & -a.align, hi, KT);
        }
      }
      mine += w[i];
    }
    // prefix sum over the threads
    __shared__ int wsum[TH / 64];
    const int lane = tid & 63;
    int inc = mine;
    inc += __builtin_amdgcn_update_dpp(0, inc, 0x111, 0xf, 0xf, false);
    inc += __builtin_amdgcn_update_dpp(0, inc, 0x112, 0xf, 0xf, false);
    inc += __builtin_amdgcn_update_dpp(0, inc, 0x114, 0xf, 0xf, false);
    inc += __builtin_amdgcn_update_dpp(0, inc, 0x118, 0xf, 0xf, false);
    inc += __builtin_amdgcn_update_dpp(0, inc, 0x142, 0xa, 0xf, false);
    inc += __builtin_amdgcn_update_dpp(0, inc, 0x143, 0xc, 0xf, false);
    if (lane == 63) wsum[tid >> 6] = inc;
    __syncthreads();
    int before = inc - mine, total = 0;
#pragma unroll
    for (int i = 0; i < TH / 64; ++i) {
      if (i < (tid >> 6)) before += wsum[i];
      total += wsum[i];
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int t = tid * PER + i;
      if (t < T) cum[t] = before;
      before += w[i];
    }
    __syncthreads();
    return total;
  }

  __device__ static __forceinline__ void body(ArgPtr ap, unsigned char* lds, int* cum, Interval* intervals, int* odd, unsigned block) {
    const AttendArgs& a = fresh(ap);
    const bool mixed = a.odd != nullptr;
    if (!GUARD && mixed) {
      if (threadIdx.x == 0) *odd = 0;
      __syncthreads();
    }
    // units of work [u, u1): queries of this workgroup's row tile, or key tiles of the plan
    const int NH = a.NH, T = (int)a.T;
    const bool planned = a.planned;
    int total = 0;
    int64_t u, u1;
    int hh = 0;
    Known known{intervals, 0};
    if (planned) {
      total = uniform(make_plan(a, cum, known));
      const int64_t units = (int64_t)total * NH;
      u = block * units / a.G;
      u1 = ((int64_t)block + 1) * units / a.G;
      if (block == 0 && !GUARD) publish_plan(a, cum, known, total);
    } else {
      // one workgroup per row tile, the last queries (the longest of a causal prompt) first
      const unsigned ntiles = (unsigned)((T + a.qt - 1) / a.qt);
      const unsigned tile = ntiles - 1 - block / (unsigned)NH;
      hh = block % (unsigned)NH;
      u = (int64_t)tile * a.qt;
      u1 = min((int64_t)T, u + a.qt);
      known.t0 = u;
      for (int i = threadIdx.x; i < (int)(u1 - u); i += TH) intervals[i] = interval_of(a, u + i);
      __syncthreads();
    }
    while (u < u1) {
      Part p;
      if (planned) {
        // the last query whose segment starts at or before unit u
        int lo = 0, hi = T - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if ((int64_t)cum[mid] * NH <= u) lo = mid;
          else hi = mid - 1;
        }
        lo = uniform(lo);
        const int first = uniform(cum[lo]);
        p.t0 = lo;
        p.nq = run_length(a, known, lo);
        const int next = lo + p.nq;
        const int tiles = (next < T ? uniform(cum[next]) : total) - first;
        const int64_t in = u - (int64_t)first * NH;
        p.hh = (int)(in / tiles);
        p.tile0 = (int)(in - (int64_t)p.hh * tiles);
        const int64_t left = u1 - u;
        p.tile1 = left < tiles - p.tile0 ? p.tile0 + (int)left : tiles;
        p.whole = p.tile0 == 0 && p.tile1 == tiles;
        p.slot = (int)(2 * block + (p.tile0 > 0 ? 0 : 1));
        u += p.tile1 - p.tile0;
      } else {
        p.t0 = u;
        p.nq = run_length(a, known, u);
        p.hh = hh;
        p.tile0 = 0;
        p.tile1 = 0x7fffffff;
        p.whole = true;
        p.slot = 0;
        u += p.nq;
      }
      run_part(ap, p, lds, known, mixed ? odd : nullptr);
    }
    if (!GUARD && mixed) {
      __syncthreads();
      if (threadIdx.x == 0) fresh(ap).odd[block] = *odd;
    }
  }

  // What the join needs: every query takes the entry of its segment.
  __device__ static __forceinline__ void publish_plan(const AttendArgs& a, const int* cum, const Known& known,
                                                     int total) {
    for (int t = threadIdx.x; t < (int)a.T; t += TH) {
      int t0 = t, next = t + 1;
      const int seq = known[t].seq;
      while (t0 % a.qt != 0 && known[t0 - 1].seq == seq) --t0;
      while (next < (int)a.T && next % a.qt != 0 && known[next].seq == seq) ++next;
      PlanEntry e;
      e.first = cum[t0];
      e.tiles = (next < (int)a.T ? cum[next] : total) - cum[t0];
      e.t0 = t0;
      a.plan[t] = e;
    }
    if (threadIdx.x == 0) *a.plan_total = total;
  }
};

template <bool HALF, int D, int R, int MODE, bool ALIGNED, bool GUARD>
__global__ __launch_bounds__((Shape<D, R>::threads), (Shape<D, R>::per_cu * Shape<D, R>::threads / 256 > 0
                                                          ? Shape<D, R>::per_cu * Shape<D, R>::threads / 256
                                                          : 1)) void attend_kernel(AttendArgs) {
  __shared__ __align__(1024) unsigned char lds[Shape<D, R>::lds_bytes];
  __shared__ int cum[kPlanMax];
  __shared__ Interval intervals[kPlanMax];
  __shared__ int odd;
  // the arguments are read where they lie (see fresh)
  const ArgPtr args = (ArgPtr)__builtin_amdgcn_kernarg_segment_ptr();
  if constexpr (GUARD) {
    // each workgroup looks over the words of a run of them at once
    const unsigned blocks = args->blocks, per = (blocks + gridDim.x - 1) / gridDim.x;
    for (unsigned b0 = blockIdx.x * per; b0 < blocks && b0 < (blockIdx.x + 1) * per; b0 += blockDim.x) {
      const unsigned n = min(min(blocks, (blockIdx.x + 1) * per) - b0, blockDim.x);
      if (!__syncthreads_or(threadIdx.x < n && args->odd[b0 + threadIdx.x])) continue;
      for (unsigned b = b0; b < b0 + n; ++b) {
        if (!args->odd[b]) continue;
        __syncthreads();
        Kernel<HALF, D, R, MODE, ALIGNED, GUARD>::body(args, lds, cum, intervals, &odd, b);
      }
    }
  } else {
    Kernel<HALF, D, R, MODE, ALIGNED, GUARD>::body(args, lds, cum, intervals, &odd, blockIdx.x);
  }
}

template <bool HALF, int D, int R>
hipError_t launch_shape(const AttendArgs& a, unsigned blocks, hipStream_t st) {
  const dim3 grid(blocks), block(Shape<D, R>::threads);
  const int mode = a.slopes || a.cap > kPlainCap ? kBias : a.cap > 0.f ? kCap : kPlain;
#define MISA_ATTEND(MODE_, ALIGNED_) \
  hipLaunchKernelGGL((attend_kernel<HALF, D, R, MODE_, ALIGNED_, false>), grid, block, 0, st, a)
  if (a.align > 1) {
    if constexpr (Shape<D, R>::RW > 1) {
      if (mode == kPlain) MISA_ATTEND(kPlain, true);
      if (mode == kCap) MISA_ATTEND(kCap, true);
      if (mode == kBias) MISA_ATTEND(kBias, true);
    }
  } else {
    if (mode == kPlain) MISA_ATTEND(kPlain, false);
    if (mode == kCap) MISA_ATTEND(kCap, false);
    if (mode == kBias) MISA_ATTEND(kBias, false);
  }
#undef MISA_ATTEND
  // workgroups that met values that are not finite where not all rows see them
  if (a.odd)
    hipLaunchKernelGGL((attend_kernel<HALF, D, R, kBias, false, true>), dim3(blocks < 256 ? blocks : 256), block, 0, st, a);
  return hipGetLastError();
}

template <int D>
hipError_t launch_dim(const AttendArgs& a, int R, bool half, unsigned blocks, hipStream_t st) {
  switch (R) {
    case 16:
      if constexpr (D < 256) return half ? launch_shape<true, D, 16>(a, blocks, st) : launch_shape<false, D, 16>(a, blocks, st);
      break;
    case 32: return half ? launch_shape<true, D, 32>(a, blocks, st) : launch_shape<false, D, 32>(a, blocks, st);
    case 64: return half ? launch_shape<true, D, 64>(a, blocks, st) : launch_shape<false, D, 64>(a, blocks, st);
    case 128: return half ? launch_shape<true, D, 128>(a, blocks, st) : launch_shape<false, D, 128>(a, blocks, st);
  }
  return hipErrorInvalidValue;
}

}  // namespace attend
}  // namespace misa
