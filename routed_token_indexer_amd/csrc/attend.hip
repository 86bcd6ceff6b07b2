// Attention over a paged cache: tile choice, workspace layout and the join of
// the parts that a planned launch leaves unfinished.
#include "attend_kernel.hpp"

namespace misa {
namespace {

using attend::Shape;

constexpr int kCUs = 256;

// One row's parts, in the order of their keys: out = sum_i 2^(m_i - M) o_i over
// the same of the sums. D / 4 lanes take one row; a row that one workgroup
// finished by itself is left alone.
template <bool HALF, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int R) {
  constexpr int LPR = D / 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (row >= a.T * a.Hq) return;
  const int d0 = (threadIdx.x % LPR) * 4;
  const int64_t t = row / a.Hq;
  const int head = (int)(row - t * a.Hq);
  const PlanEntry e = a.plan[t];
  const int64_t units = *a.plan_total * a.NH, G = a.G;
  const int in = head % a.group;
  const int hh = head / a.group * a.head_tiles + in / a.gw;
  const int r = (int)(t - e.t0) * a.gw + in % a.gw;
  const int64_t u0 = e.first * a.NH + (int64_t)hh * e.tiles, u1 = u0 + e.tiles;
  // workgroup i takes units [i units / G, (i + 1) units / G)
  const int64_t i0 = ((u0 + 1) * G - 1) / units, i1 = (u1 * G - 1) / units;
  if (i0 == i1) return;
  float M = -__builtin_inff();
  for (int64_t i = i0; i <= i1; ++i) {
    const int64_t b = i * units / G;
    if (b == (i + 1) * units / G) continue;
    const int64_t slot = 2 * i + (b > u0 ? 0 : 1);
    M = fmaxf(M, a.part_ml[(slot * R + r) * 2]);
  }
  const float ref = M == -__builtin_inff() ? 0.f : M;
  float sum = 0.f;
  floatx4 o = {0.f, 0.f, 0.f, 0.f};
  for (int64_t i = i0; i <= i1; ++i) {
    const int64_t b = i * units / G;
    if (b == (i + 1) * units / G) continue;
    const int64_t slot = 2 * i + (b > u0 ? 0 : 1);
    const float w = __builtin_amdgcn_exp2f(a.part_ml[(slot * R + r) * 2] - ref);
    sum += a.part_ml[(slot * R + r) * 2 + 1] * w;
    const floatx4 x = *reinterpret_cast<const floatx4*>(a.part_out + (slot * R + r) * D + d0);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] += x[j] * w;
  }
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

int attend_rows(int64_t T, int64_t nseq, int group, bool gather) {
  const int64_t each = gather || nseq < 1 ? 1 : (T + nseq - 1) / nseq;
  const int64_t rows = each * group;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
}

bool attend_planned(int64_t T) { return T <= kPlanMax; }

int attend_groups(int d, int R) { return kCUs * (d == 64 ? per_cu<64>(R) : d == 128 ? per_cu<128>(R) : per_cu<256>(R)); }

size_t attend_ws_bytes(int64_t T, int d, int R) {
  if (!attend_planned(T)) return 0;
  const size_t slots = 2 * (size_t)attend_groups(d, R);
  return up(slots * R * d * 4) + up(slots * R * 8) + up((size_t)T * sizeof(PlanEntry)) + 256;
}

void attend_setup(AttendArgs& a, int R, void* ws) {
  const int d = a.d;
  a.group = a.Hq / a.Hkv;
  a.gw = a.group < R ? a.group : R;
  a.head_tiles = (a.group + a.gw - 1) / a.gw;
  a.qt = a.idx ? 1 : R / a.gw;   // the selected tokens are each query's own
  a.NH = a.Hkv * a.head_tiles;
  a.by_gw = fast_div((uint32_t)a.gw);
  a.planned = attend_planned(a.T);
  a.G = 0;
  if (!a.planned) return;
  a.G = attend_groups(d, R);
  const size_t slots = 2 * (size_t)a.G;
  char* p = static_cast<char*>(ws);
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
  const int64_t rows = a.T * a.Hq;
  const int per = 256 / (a.d / 4);
  const dim3 grid((unsigned)((rows + per - 1) / per));
#define MISA_JOIN(HALF_, D_) hipLaunchKernelGGL((attend_join_kernel<HALF_, D_>), grid, dim3(256), 0, st, a, R)
  if (a.d == 64) { if (half) MISA_JOIN(true, 64); else MISA_JOIN(false, 64); }
  if (a.d == 128) { if (half) MISA_JOIN(true, 128); else MISA_JOIN(false, 128); }
  if (a.d == 256) { if (half) MISA_JOIN(true, 256); else MISA_JOIN(false, 256); }
#undef MISA_JOIN
  return hipGetLastError();
}

}  // namespace misa
