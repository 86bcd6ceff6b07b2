// Eviction: which tokens of a cache stay, and the moves that make them its first rows.
//
// A list is the rows of one kv head of a sequence, or of all heads together. Its
// `budget` tokens of highest rank stay: protected ones (first and latest positions),
// then by mass, ties to the lower row. The kept rows among the first `budget` are left
// where they are; the rows of dropped tokens among them (holes, ascending) take the
// kept rows from behind (movers, ascending). Movers all lie behind every hole, so no row
// that is read is written: the moves need no order, and few rows move.
#include "misa_common.hpp"
#include "misa_evict.hpp"

namespace misa {
namespace {

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;
constexpr int kBins = 4096;

constexpr uint32_t kProtected = 0xffffffffu;

// Rank of a token as an unsigned number; 0 stands for no token. NaN ranks above all numbers.
__device__ __forceinline__ uint32_t rank_key(float mass, int pos, int64_t first, int64_t latest) {
  if (pos < first || pos >= latest) return kProtected;
  if (mass != mass) return kProtected - 1;
  return score_key(mass);      // of no number 0 or above the NaN's
}

__device__ __forceinline__ int wave_scan(int v) {   // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int x = __shfl_up(v, off, 64);
    if (lane >= off) v += x;
  }
  return v;
}

// Exclusive sum over the workgroup's waves of a value per wave; total of all in `all`.
__device__ __forceinline__ int waves_before(int v, int* slots, int& all) {
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) slots[w] = v;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int i = 0; i < kSelWaves; ++i) {
    const int x = slots[i];
    before += i < w ? x : 0;
    all += x;
  }
  return before;
}

// One workgroup a list. Wave w owns the rows [w C, (w + 1) C), 64 at a time, so that
// numbers in row order need one sum over the waves. N > 0: at most N runs of 64 rows a
// wave, whose keys stay in registers; 0: any length, keys read again for each sweep.
template <int N>
__global__ __launch_bounds__(kSelThreads) void select_kernel(EvictArgs a) {
  __shared__ uint32_t hist[kBins];
  __shared__ int slots[kSelWaves];
  __shared__ int found[2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t list = blockIdx.x;
  const int64_t n = list / a.G;
  const int Lmax = (int)a.kv.Lmax;
  const int len = min(max(a.lens[n], 0), Lmax);
  const int size = (int)min((int64_t)len, a.budget);
  const float* mass = a.mass + list * Lmax;
  const int32_t* pos = a.pos ? a.pos + list * Lmax : nullptr;
  int32_t* src = a.src + list * a.budget;
  int32_t* movers = a.movers + list * min(a.budget, a.kv.Lmax);
  const int runs = (len + kSelThreads - 1) / kSelThreads;   // of 64 rows, per wave
  const int base = wave * runs * 64 + lane;

  // the latest position
  int newest = len - 1;
  if (pos) {
    newest = (int)0x80000000;
    for (int i = 0; i < runs; ++i) {
      const int e = base + 64 * i;
      if (e < len) newest = max(newest, pos[e]);
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) newest = max(newest, __shfl_xor(newest, off, 64));
    if (lane == 0) slots[wave] = newest;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelWaves; ++i) newest = max(newest, slots[i]);
  }
  const int64_t first = a.sinks, latest = newest - a.recent + 1;

  uint32_t keys[N > 0 ? N : 1];
  auto load = [&](int e) { return e < len ? rank_key(mass[e], pos ? pos[e] : e, first, latest) : 0u; };
  if constexpr (N > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) keys[i] = i < runs ? load(base + 64 * i) : 0u;
  }
  // f(row, key) for the wave's rows in order
  auto sweep = [&](auto f) {
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < runs) f(base + 64 * i, keys[i]);
    } else {
      for (int i = 0; i < runs; ++i) f(base + 64 * i, load(base + 64 * i));
    }
  };

  // the key of the last kept token, and how many of its equals are kept
  uint32_t least = 1;
  int equals = 0x7fffffff;
  if (len > size) {
    int want = size;
    uint32_t prefix = 0;
    bool done = false;
#pragma unroll
    for (int step = 0; step < 3; ++step) {
      const int shift = step == 0 ? 20 : (step == 1 ? 8 : 0), bits = step == 2 ? 8 : 12;
      if (!done) {
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        sweep([&](int, uint32_t k) {
          if (k && (step == 0 || k >> (shift + bits) == prefix)) atomicAdd(&hist[k >> shift & ((1u << bits) - 1)], 1u);
        });
        __syncthreads();
        // from the highest bin down: thread i owns bins 4095 - 4 i .. 4092 - 4 i
        int c[4], mine = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          c[j] = (int)hist[kBins - 1 - 4 * (int)threadIdx.x - j];
          mine += c[j];
        }
        const int incl = wave_scan(mine);
        int all;
        int above = waves_before(__shfl(incl, 63, 64), slots, all) + incl - mine;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (above < want && above + c[j] >= want) {
            found[0] = kBins - 1 - 4 * (int)threadIdx.x - j;
            found[1] = want - above == c[j] ? -c[j] : want - above;
          }
          above += c[j];
        }
        __syncthreads();
        prefix = prefix << bits | (uint32_t)found[0];
        if (found[1] < 0) {        // the whole bin stays
          done = true;
          least = prefix << shift;
        } else {
          want = found[1];
          least = prefix;
          equals = want;
        }
      }
    }
    if (done) equals = 0x7fffffff;
    if (least == 0) least = 1;
  }

  // number of equals before the wave's rows
  int seen = 0;
  if (equals != 0x7fffffff) {
    int ties = 0;
    sweep([&](int, uint32_t k) { ties += __popcll(__ballot(k == least)); });
    int all;
    seen = waves_before(ties, slots, all);
  }
  const int seen0 = seen;
  auto stays = [&](uint32_t k) {
    bool s = k >= least;
    if (equals != 0x7fffffff) {
      const uint64_t m = __ballot(k == least);
      if (k == least) s = seen + (int)lanes_below(m) < equals;
      seen += __popcll(m);
    }
    return s;
  };
  int holes = 0, moves = 0;
  sweep([&](int e, uint32_t k) {
    const bool s = stays(k);
    holes += __popcll(__ballot(!s && e < size));
    moves += __popcll(__ballot(s && e >= size));
  });
  int all_holes, all_moves;
  int hole = waves_before(holes, slots, all_holes);
  int move = waves_before(moves, slots, all_moves);
  seen = seen0;
  sweep([&](int e, uint32_t k) {
    const bool m = stays(k) && e >= size;
    const uint64_t b = __ballot(m);
    if (m) movers[move + lanes_below(b)] = e;
    move += __popcll(b);
  });
  __syncthreads();      // the movers are there, and every key has been read (the rows may be written in place)
  seen = seen0;
  float* mass_out = a.mass_out ? a.mass_out + list * Lmax : nullptr;
  int32_t* pos_out = a.pos_out ? a.pos_out + list * Lmax : nullptr;
  auto place = [&](int e, uint32_t k) {
    const bool h = !stays(k) && e < size;
    const uint64_t b = __ballot(h);
    if (e < size) {
      const int s = h ? movers[hole + lanes_below(b)] : e;
      src[e] = s;
      if (mass_out) mass_out[e] = mass[s];
      if (pos_out) pos_out[e] = pos ? pos[s] : s;
    }
    hole += __popcll(b);
  };
  sweep(place);     // a row whose key is read again here is written by the same thread afterwards
  __syncthreads();
  for (int64_t i = size + (int)threadIdx.x; i < a.budget; i += kSelThreads) src[i] = -1;
  for (int i = size + (int)threadIdx.x; i < Lmax; i += kSelThreads) {
    if (mass_out) mass_out[i] = 0.f;
    if (pos_out) pos_out[i] = -1;
  }
  if (threadIdx.x == 0 && list == n * a.G) a.new_len[n] = size;
}

// ---------------------------------------------------------------- moves
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;       // rows of a list that a workgroup looks at
constexpr int kMoveBatch = 8;       // pieces on their way a thread

// Bound by memory: 16-byte pieces of the rows that move, all heads of a row next to
// each other. The first wave looks up which of the workgroup's rows move, and the pages
// of both ends.
__global__ __launch_bounds__(kMoveThreads) void move_kernel(MoveArgs a, int chunks, int units, FastDiv by_units,
                                                            int heads, FastDiv by_heads) {
  __shared__ int64_t from[kMoveRows], to[kMoveRows];
  __shared__ int count;
  const int64_t list = blockIdx.x / chunks;
  const int chunk = blockIdx.x % chunks;
  const int64_t n = list / a.G;
  const int g = (int)(list - n * a.G);
  if (threadIdx.x < kMoveRows) {
    const int64_t i = (int64_t)chunk * kMoveRows + threadIdx.x;
    const int64_t s = i < a.n && i < a.kv.Lmax ? a.src[list * a.n + i] : -1;
    bool moves = s >= 0 && s < a.kv.Lmax && s != i;
    int64_t p0 = 0, p1 = 0;
    if (moves) {
      const uint32_t c0 = fast_quot(a.kv.by_page, (uint32_t)s), c1 = fast_quot(a.kv.by_page, (uint32_t)i);
      const int page0 = kv_page(a.kv, (int)n, c0), page1 = kv_page(a.kv, (int)n, c1);
      moves = page0 >= 0 && page1 >= 0;
      p0 = page0 * a.kv.page_stride + (s - (int64_t)c0 * a.kv.page) * a.kv.tok_stride;
      p1 = page1 * a.kv.page_stride + (i - (int64_t)c1 * a.kv.page) * a.kv.tok_stride;
    }
    const uint64_t b = __ballot(moves);
    if (moves) {
      const int at = (int)lanes_below(b);
      from[at] = p0;
      to[at] = p1;
    }
    if (threadIdx.x == 0) count = __popcll(b);
  }
  __syncthreads();
  const uint32_t pieces = (uint32_t)count * heads * units;
  const int64_t head0 = a.G == 1 ? 0 : g * a.kv.head_stride;
#pragma unroll 1
  for (int tensor = 0; tensor < (a.kv.v ? 2 : 1); ++tensor) {
    uint16_t* base = (tensor ? a.kv.v : a.kv.k) + head0;
    for (uint32_t i0 = threadIdx.x; i0 < pieces; i0 += kMoveThreads * kMoveBatch) {
      u32x4 x[kMoveBatch];
      uint16_t* dst[kMoveBatch];
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const uint32_t i = i0 + j * kMoveThreads;
        dst[j] = nullptr;
        if (i >= pieces) continue;
        const uint32_t item = fast_quot(by_units, i), u = i - item * units;
        const uint32_t r = fast_quot(by_heads, item), h = item - r * heads;
        const int64_t off = h * a.kv.head_stride + 8 * u;
        x[j] = *reinterpret_cast<const u32x4*>(base + from[r] + off);
        dst[j] = base + to[r] + off;
      }
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j)
        if (dst[j]) *reinterpret_cast<u32x4*>(dst[j]) = x[j];
    }
  }
}

}  // namespace

hipError_t launch_evict_select(const EvictArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.kv.nseq * a.G)), block(kSelThreads);
  const int64_t runs = (a.kv.Lmax + kSelThreads - 1) / kSelThreads;
  if (runs <= 4) hipLaunchKernelGGL(select_kernel<4>, grid, block, 0, st, a);
  else if (runs <= 16) hipLaunchKernelGGL(select_kernel<16>, grid, block, 0, st, a);
  else if (runs <= 48) hipLaunchKernelGGL(select_kernel<48>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(select_kernel<0>, grid, block, 0, st, a);
  return hipGetLastError();
}

static int64_t move_chunks(const MoveArgs& a) {
  const int64_t rows = a.n < a.kv.Lmax ? a.n : a.kv.Lmax;
  return (rows + kMoveRows - 1) / kMoveRows;
}

int64_t move_blocks(const MoveArgs& a) { return move_chunks(a) * a.kv.nseq * a.G; }

hipError_t launch_move(const MoveArgs& a, hipStream_t st) {
  const int heads = a.G == 1 ? a.Hkv : 1, units = a.d / 8;
  hipLaunchKernelGGL(move_kernel, dim3((unsigned)move_blocks(a)), dim3(kMoveThreads), 0, st, a, (int)move_chunks(a), units,
                     fast_div((uint32_t)units), heads, fast_div((uint32_t)heads));
  return hipGetLastError();
}

}  // namespace misa
