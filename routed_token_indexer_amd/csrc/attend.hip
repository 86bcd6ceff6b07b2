// Attention over a paged cache: tile choice, workspace layout and the join of
// the parts that a planned launch leaves unfinished.
#include "attend_kernel.hpp"

namespace misa {
namespace {

using attend::Shape;

constexpr int kCUs = 256;

// One row's parts: out = sum_i 2^(m_i - M) o_i over the same of the sums. A
// workgroup takes one row; D / 4 lanes add up every (1024 / D)-th part, and the
// groups' sums are added in a fixed order. A row that one workgroup of the
// attention finished by itself is left alone.
template <bool HALF, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int R) {
  constexpr int LPR = D / 4, GR = 256 / LPR;
  __shared__ float weight[256];
  __shared__ float wsum[4], wmax[4];
  __shared__ floatx4 acc[256];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t t = row / a.Hq;
  const int head = (int)(row - t * a.Hq);
  const PlanEntry e = a.plan[t];
  const int64_t units = *a.plan_total * a.NH, G = a.G;
  const int in = head % a.group;
  const int hh = head / a.group * a.head_tiles + in / a.gw;
  const int r = (int)(t - e.t0) * a.gw + in % a.gw;
  const int64_t u0 = e.first * a.NH + (int64_t)hh * e.tiles, u1 = u0 + e.tiles;
  // workgroup i takes units [i units / G, (i + 1) units / G)
  const int i0 = (int)(((u0 + 1) * G - 1) / units), i1 = (int)((u1 * G - 1) / units);
  if (i0 == i1) return;
  float M = -__builtin_inff(), sum = 0.f;
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  const int g = tid / LPR, d0 = (tid % LPR) * 4;
  for (int base = i0; base <= i1; base += 256) {
    // maxima and sums of up to 256 parts
    const int i = base + tid;
    float m = -__builtin_inff(), s = 0.f;
    if (i <= i1) {
      const int64_t b = i * units / G;
      if (b != ((int64_t)i + 1) * units / G) {
        const float* ml = a.part_ml + ((2 * (int64_t)i + (b > u0 ? 0 : 1)) * R + r) * 2;
        m = ml[0];
        s = ml[1];
      }
    }
    float wm = m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) wm = fmaxf(wm, __shfl_xor(wm, off, 64));
    if ((tid & 63) == 0) wmax[tid >> 6] = wm;
    __syncthreads();
    const float top = fmaxf(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])), M);
    const float ref = top == -__builtin_inff() ? 0.f : top;
    const float w = __builtin_amdgcn_exp2f(m - ref);
    weight[tid] = w;
    s = wave_sum(s * w);
    if ((tid & 63) == 0) wsum[tid >> 6] = s;
    const float old = __builtin_amdgcn_exp2f(M - ref);
    M = top;
    __syncthreads();
    sum = sum * old + wsum[0] + wsum[1] + wsum[2] + wsum[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] *= old;
    const int n = min(256, i1 - base + 1);
#pragma unroll 4
    for (int k = g; k < n; k += GR) {
      const float wk = weight[k];
      // only the row's first part can be its workgroup's second (see Part::slot)
      const int64_t slot = 2 * ((int64_t)base + k) + (base + k == i0 && i0 * units / G <= u0 ? 1 : 0);
      if (wk == 0.f) continue;   // no part, or one without a key
      const floatx4 x = *reinterpret_cast<const floatx4*>(a.part_out + (slot * R + r) * D + d0);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] += x[j] * wk;
    }
    __syncthreads();
  }
  acc[tid] = o;
  __syncthreads();
  if (g > 0) return;
#pragma unroll
  for (int k = 1; k < GR; ++k) o += acc[k * LPR + tid];
  attend::write_row<HALF, D>(a, row, d0, M, sum, o);
}

template <int D>
int per_cu(int R) {
  switch (R) {
    case 16: return Shape<D, 16>::per_cu;
    case 32: return Shape<D, 32>::per_cu;
    case 64: return Shape<D, 64>::per_cu;
  }
  return Shape<D, 128>::per_cu;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int attend_rows(int64_t T, int64_t nseq, int group, bool single) {
  const int64_t each = single ? 1 : (T + nseq - 1) / nseq;
  const int64_t rows = each * group;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

bool attend_planned(int64_t T) { return T <= kPlanMax; }

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

static int64_t blocks_of(int64_t T, int heads, int d, int R, const Tile& t) {
  return attend_planned(T) ? attend_groups(d, R) : (T + t.qt - 1) / t.qt * heads * t.head_tiles;
}

size_t attend_ws_bytes(int64_t T, int Hq, int heads, int d, int R, bool single, bool mixed) {
  const Tile t = tile_of(Hq / heads, R, single);
  size_t b = 0;
  if (mixed && t.qt > 1) b += up((size_t)blocks_of(T, heads, d, R, t) * 4);
  if (!attend_planned(T)) return b;
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
  a.planned = attend_planned(a.T);
  a.G = a.planned ? attend_groups(d, R) : 0;
  a.odd = nullptr;
  char* p = static_cast<char*>(ws);
  if (mixed && t.qt > 1) {
    a.odd = reinterpret_cast<int32_t*>(p);
    p += up((size_t)blocks_of(a.T, a.Hkv, d, R, t) * 4);
  }
  if (!a.planned) return;
  const size_t slots = 2 * (size_t)a.G;
  a.part_out = reinterpret_cast<float*>(p);
  p += up(slots * R * d * 4);
  a.part_ml = reinterpret_cast<float*>(p);
  p += up(slots * R * 8);
  a.plan = reinterpret_cast<PlanEntry*>(p);
  p += up((size_t)a.T * sizeof(PlanEntry));
  a.plan_total = reinterpret_cast<int64_t*>(p);
}

int64_t attend_blocks(const AttendArgs& a) {
  return a.planned ? a.G : (a.T + a.qt - 1) / a.qt * a.NH;
}

hipError_t launch_attend(const AttendArgs& a, int R, bool half, hipStream_t st) {
  const unsigned blocks = (unsigned)attend_blocks(a);
  hipError_t e = hipErrorInvalidValue;
  if (a.d == 64) e = launch_attend_d64(a, R, half, blocks, st);
  if (a.d == 128) e = launch_attend_d128(a, R, half, blocks, st);
  if (a.d == 256) e = launch_attend_d256(a, R, half, blocks, st);
  if (e != hipSuccess || !a.planned) return e;
  const dim3 grid((unsigned)(a.T * a.Hq));
#define MISA_JOIN(HALF_, D_) hipLaunchKernelGGL((attend_join_kernel<HALF_, D_>), grid, dim3(256), 0, st, a, R)
  if (a.d == 64) { if (half) MISA_JOIN(true, 64); else MISA_JOIN(false, 64); }
  if (a.d == 128) { if (half) MISA_JOIN(true, 128); else MISA_JOIN(false, 128); }
  if (a.d == 256) { if (half) MISA_JOIN(true, 256); else MISA_JOIN(false, 256); }
#undef MISA_JOIN
  return hipGetLastError();
}

}  // namespace misa
