// Attention over a paged cache: tile choice, workspace layout and the join of
// the parts that a planned launch leaves unfinished.
#include "attend_kernel.hpp"

namespace misa {
namespace {

using attend::Shape;

constexpr int kCUs = 256;

// What the join reads of a pass.
struct Pass {
  const PlanEntry* plan;    // null: every row is whole
  const int32_t* plan_total;
  const float* part_out;
  const float* part_ml;
  const float* whole_out;   // [T][Hq][D] and [T][Hq], for rows that are whole
  const float* whole_lse;
  int32_t G, R, NH, group, head_tiles, gw;
};
Pass pass_of(const AttendArgs& a, int R) {
  Pass p;
  p.plan = a.planned ? a.plan : nullptr;
  p.plan_total = a.plan_total;
  p.part_out = a.part_out;
  p.part_ml = a.part_ml;
  p.whole_out = a.out32;
  p.whole_lse = a.lse;
  p.G = a.G;
  p.R = R;
  p.NH = a.NH;
  p.group = a.group;
  p.head_tiles = a.head_tiles;
  p.gw = a.gw;
  return p;
}

// Workgroup i of a planned pass takes units [i units / G, (i + 1) units / G).
struct Parts {
  int64_t units, u0;   // units of the pass; the row's first
  int i0, i1;          // workgroups that share the row
  int r;               // its row of their tiles
};
__device__ __forceinline__ Parts parts_of(const Pass& p, int64_t t, int head) {
  Parts x;
  const PlanEntry e = p.plan[t];
  const int in = head % p.group;
  const int hh = head / p.group * p.head_tiles + in / p.gw;
  x.units = (int64_t)*p.plan_total * p.NH;
  x.u0 = (int64_t)e.first * p.NH + (int64_t)hh * e.tiles;
  x.r = (int)(t - e.t0) * p.gw + in % p.gw;
  x.i0 = (int)(((x.u0 + 1) * p.G - 1) / x.units);
  x.i1 = (int)(((x.u0 + e.tiles) * p.G - 1) / x.units);
  return x;
}

// One row's parts: out = sum_i 2^(m_i - M) o_i over the same of the sums. WPR waves
// take one row, each every WPR-th chunk of its parts; in a wave D / 4 lanes add up
// every (256 / D)-th part, eight at a time. The sums of lanes and waves are added
// in a fixed order. The outputs of a chunk of parts are
// requested together with their maxima and sums: the launch is bound by its
// dependent loads (plan, parts). TWO passes over different keys give their parts,
// or a whole row each (one part with m = lse and a sum of one). With one pass a
// row that one workgroup of the attention finished is left alone.
template <bool HALF, int D, bool TWO, int WPR>
__global__ __launch_bounds__(256) void attend_join_kernel(Pass pa, Pass pb, int64_t rows, int Hq, uint16_t* out, float* lse) {
  constexpr int LPR = D / 4, GR = 64 / LPR, PER = 8, CH = PER * GR;
  __shared__ float wave_ml[4][2];
  __shared__ floatx4 wave_o[4][LPR];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = (int64_t)blockIdx.x * (4 / WPR) + wave / WPR;
  const int part = wave % WPR;
  if (row >= rows) return;
  const int lane = threadIdx.x & 63;
  const int64_t t = row / Hq;
  const int head = (int)(row - t * Hq);
  float M = -__builtin_inff(), sum = 0.f;
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  const int g = lane / LPR, d0 = (lane % LPR) * 4;
  Parts xs[2];
#pragma unroll
  for (int which = 0; which < (TWO ? 2 : 1); ++which) {
    const Pass& p = which ? pb : pa;
    xs[which].i0 = xs[which].i1 = 0;
    if (p.plan) xs[which] = parts_of(p, t, head);
  }
#pragma unroll
  for (int which = 0; which < (TWO ? 2 : 1); ++which) {
    const Pass& p = which ? pb : pa;
    const Parts& x = xs[which];
    if (x.i0 == x.i1) {
      if (!TWO) return;
      const float l = p.whole_lse[row];
      const floatx4 y = *reinterpret_cast<const floatx4*>(p.whole_out + row * D + d0);
      if (l == -__builtin_inff() || part != 0) continue;
      const float m = l * attend::kLog2e;
      const float top = fmaxf(M, m);
      const float old = __builtin_amdgcn_exp2f(M - top), w = l == l ? __builtin_amdgcn_exp2f(m - top) : l;
      sum = sum * old + w;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = o[j] * old + (g == 0 ? y[j] * w : 0.f);
      M = top;
      continue;
    }
    const int64_t G = p.G;
    // only the row's first part can be its workgroup's second (see Part::slot)
    const int second = x.i0 * x.units / G <= x.u0 ? x.i0 : -1;
    for (int base = x.i0 + part * CH; base <= x.i1; base += WPR * CH) {
      floatx4 y[PER];
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const int i = min(base + k * GR + g, x.i1);
        y[k] = *reinterpret_cast<const floatx4*>(p.part_out + ((2 * (int64_t)i + (i == second ? 1 : 0)) * p.R + x.r) * D + d0);
      }
      // maxima and sums of the chunk's parts, one a lane
      const int i = base + lane;
      float m = -__builtin_inff(), s = 0.f;
      bool part_here = false;
      if (lane < CH && i <= x.i1) {
        const float* ml = p.part_ml + ((2 * (int64_t)i + (i == second ? 1 : 0)) * p.R + x.r) * 2;
        const float m1 = ml[0], s1 = ml[1];
        if (i * x.units / G != ((int64_t)i + 1) * x.units / G) {   // a workgroup with work
          m = m1;
          s = s1;
          part_here = true;
        }
      }
      float top = m;
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
      top = fmaxf(top, M);
      const float ref = top == -__builtin_inff() ? 0.f : top;
      const float w = __builtin_amdgcn_exp2f(m - ref), old = __builtin_amdgcn_exp2f(M - ref);
      M = top;
      sum = sum * old + wave_sum(s * w);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] *= old;
      // Where there is no part y is anything and is left out (-1); a part whose weight
      // vanishes is not: a NaN or an infinity among its values reaches the row.
      const float mark = part_here ? w : -1.f;
#pragma unroll
      for (int k = 0; k < PER; ++k) {
        const float wk = __shfl(mark, k * GR + g, 64);
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += wk == -1.f ? 0.f : y[k][j] * wk;
      }
    }
  }
#pragma unroll
  for (int off = LPR; off < 64; off <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], off, 64);
  if constexpr (WPR > 1) {
    if (g == 0) wave_o[wave][lane] = o;
    if (lane == 0) {
      wave_ml[wave][0] = M;
      wave_ml[wave][1] = sum;
    }
    __syncthreads();
    if (wave > 0 || g > 0) return;
    float top = M;
#pragma unroll
    for (int k = 1; k < WPR; ++k) top = fmaxf(top, wave_ml[k][0]);
    const float ref = top == -__builtin_inff() ? 0.f : top;
    const float w0 = __builtin_amdgcn_exp2f(M - ref);
    sum *= w0;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] *= w0;
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      const float w = __builtin_amdgcn_exp2f(wave_ml[k][0] - ref);
      const floatx4 y = wave_o[k][lane];
      sum += wave_ml[k][1] * w;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] += y[j] * w;
    }
    M = top;
  }
  if (g > 0) return;
  AttendArgs a{};
  a.out = out;
  a.lse = lse;
  attend::write_row<HALF, D>(a, row, d0, M, sum, o);
}

// Rows a wave loads at a time where several waves share them, 0 elsewhere.
template <int D, int R>
constexpr int shared_rows() { return Shape<D, R>::RW > 1 ? Shape<D, R>::WR : 0; }
template <int D>
int shared_rows_of(int R) {
  switch (R) {
    case 32: return shared_rows<D, 32>();
    case 64: return shared_rows<D, 64>();
    case 128: return shared_rows<D, 128>();
  }
  return 0;
}

template <int D>
int per_cu(int R) {
  switch (R) {
    case 16:
      if constexpr (D < 256) return Shape<D, 16>::per_cu;
      break;
    case 32: return Shape<D, 32>::per_cu;
    case 64: return Shape<D, 64>::per_cu;
  }
  return Shape<D, 128>::per_cu;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int attend_rows(int64_t T, int64_t nseq, int group, int d, bool single) {
  const int64_t each = single ? 1 : (T + nseq - 1) / nseq;
  const int64_t rows = each * group;
  return rows <= 16 && d < 256 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

// (32 keys a tile is the least of all shapes: the tiles of all segments fit 31 bits)
bool attend_planned(int64_t T, int64_t most_keys) {
  return T <= kPlanMax && T * (most_keys / 32 + 2) < (int64_t(1) << 31);
}

int attend_groups(int d, int R) { return kCUs * (d == 64 ? per_cu<64>(R) : d == 128 ? per_cu<128>(R) : per_cu<256>(R)); }

// Head tiles and queries of a row tile of R rows.
struct Tile {
  int gw, head_tiles, qt;
};
static Tile tile_of(int group, int R, bool single) {
  Tile t;
  t.gw = group < R ? group : R;
  t.head_tiles = (group + t.gw - 1) / t.gw;
  t.qt = single ? 1 : R / t.gw;
  return t;
}

static int64_t blocks_of(int64_t T, int heads, int d, int R, const Tile& t, bool planned) {
  return planned ? attend_groups(d, R) : (T + t.qt - 1) / t.qt * heads * t.head_tiles;
}

size_t attend_ws_bytes(int64_t T, int Hq, int heads, int d, int R, bool single, bool mixed) {
  const Tile t = tile_of(Hq / heads, R, single);
  size_t b = 0;
  const int64_t direct = blocks_of(T, heads, d, R, t, false);
  if (T > kPlanMax) return mixed ? up((size_t)direct * 4) : 0;
  const int64_t most = direct > attend_groups(d, R) ? direct : attend_groups(d, R);
  if (mixed) b += up((size_t)most * 4);
  const size_t slots = 2 * (size_t)attend_groups(d, R);
  return b + up(slots * R * d * 4) + up(slots * R * 8) + up((size_t)T * sizeof(PlanEntry)) + 256;
}

void attend_setup(AttendArgs& a, int R, bool single, bool mixed, void* ws) {
  const int d = a.d;
  a.group = a.Hq / a.Hkv;
  const Tile t = tile_of(a.group, R, single);
  a.gw = t.gw;
  a.head_tiles = t.head_tiles;
  a.qt = t.qt;
  a.NH = a.Hkv * a.head_tiles;
  a.by_gw = fast_div((uint32_t)a.gw);
  // pages that hold whole groups of a wave's rows take the kernels that look a
  // page up once a group (a row cache is one page a sequence)
  const int wr = d == 64 ? shared_rows_of<64>(R) : d == 128 ? shared_rows_of<128>(R) : shared_rows_of<256>(R);
  a.align = wr && !a.idx && a.kv.unit_shift == 0 && (!a.kv.table || a.kv.page % wr == 0) ? wr : 1;
  a.planned = attend_planned(a.T, a.idx ? a.topk : a.kv.Lmax);
  a.G = a.planned ? attend_groups(d, R) : 0;
  a.odd = nullptr;
  a.blocks = (uint32_t)blocks_of(a.T, a.Hkv, d, R, t, a.planned);
  char* p = static_cast<char*>(ws);
  if (mixed) {
    a.odd = reinterpret_cast<int32_t*>(p);
    p += up((size_t)a.blocks * 4);
  }
  if (!a.planned) return;
  const size_t slots = 2 * (size_t)a.G;
  a.part_out = reinterpret_cast<float*>(p);
  p += up(slots * R * d * 4);
  a.part_ml = reinterpret_cast<float*>(p);
  p += up(slots * R * 8);
  a.plan = reinterpret_cast<PlanEntry*>(p);
  p += up((size_t)a.T * sizeof(PlanEntry));
  a.plan_total = reinterpret_cast<int32_t*>(p);
}

int64_t attend_blocks(const AttendArgs& a) {
  return a.planned ? a.G : (a.T + a.qt - 1) / a.qt * (int64_t)a.NH;
}

hipError_t launch_attend(const AttendArgs& a, int R, bool half, hipStream_t st) {
  const unsigned blocks = (unsigned)attend_blocks(a);
  hipError_t e = hipErrorInvalidValue;
  if (a.d == 64) e = launch_attend_d64(a, R, half, blocks, st);
  if (a.d == 128) e = launch_attend_d128(a, R, half, blocks, st);
  if (a.d == 256) e = launch_attend_d256(a, R, half, blocks, st);
  return e;
}

hipError_t launch_attend_join(const AttendArgs& a, int Ra, const AttendArgs* b, int Rb, uint16_t* out, float* lse,
                              bool half, hipStream_t st) {
  if (!b && !a.planned) return hipSuccess;
  const Pass pa = pass_of(a, Ra), pb = b ? pass_of(*b, Rb) : pa;
  const int64_t rows = a.T * a.Hq;
  // few rows are spread over four waves each (256 rows of 32 parts: 8 us, 13 with a
  // wave each); many fill the chip anyway (4096 rows of 24 parts: 12 us, 21 with four)
  const bool few = rows <= 1024;
  const dim3 grid((unsigned)(few ? rows : (rows + 3) / 4));
#define MISA_JOIN_(HALF_, D_, TWO_, W_) \
  hipLaunchKernelGGL((attend_join_kernel<HALF_, D_, TWO_, W_>), grid, dim3(256), 0, st, pa, pb, rows, a.Hq, out, lse)
#define MISA_JOIN(HALF_, D_)                                                     \
  do {                                                                           \
    if (b && few) MISA_JOIN_(HALF_, D_, true, 4);                                \
    else if (b) MISA_JOIN_(HALF_, D_, true, 1);                                  \
    else if (few) MISA_JOIN_(HALF_, D_, false, 4);                               \
    else MISA_JOIN_(HALF_, D_, false, 1);                                        \
  } while (0)
  if (a.d == 64) { if (half) MISA_JOIN(true, 64); else MISA_JOIN(false, 64); }
  if (a.d == 128) { if (half) MISA_JOIN(true, 128); else MISA_JOIN(false, 128); }
  if (a.d == 256) { if (half) MISA_JOIN(true, 256); else MISA_JOIN(false, 256); }
#undef MISA_JOIN
#undef MISA_JOIN_
  return hipGetLastError();
}

}  // namespace misa
