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
typedef unsigned long long u64;

constexpr uint32_t kProtected = 0xffffffffu;

// Rank of a token as an unsigned number; 0 stands for no token. Positions from `first` on,
// fewer than `open` of them, are not protected. NaN ranks above all numbers.
__device__ __forceinline__ uint32_t rank_key(float mass, int pos, int first, uint32_t open) {
  const uint32_t u = __float_as_uint(mass + 0.f);                      // -0 becomes 0
  uint32_t k = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);           // of no number 0 or above the NaN's
  k = mass != mass ? kProtected - 1 : k;
  return (uint32_t)pos - (uint32_t)first < open ? k : kProtected;
}

// A wave's maximum or sum, in all lanes (data-parallel moves: rows of 16 lanes, then from row
// to row).
template <int CTRL, int ROWS, typename Op>
__device__ __forceinline__ uint32_t dpp_step(uint32_t none, uint32_t v, Op op) {
  return op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false));
}
template <typename Op>
__device__ __forceinline__ uint32_t scan_wave(uint32_t none, uint32_t v, Op op) {   // up to and with each lane
  v = dpp_step<0x111, 0xf>(none, v, op);
  v = dpp_step<0x112, 0xf>(none, v, op);
  v = dpp_step<0x114, 0xf>(none, v, op);
  v = dpp_step<0x118, 0xf>(none, v, op);
  v = dpp_step<0x142, 0xa>(none, v, op);
  return dpp_step<0x143, 0xc>(none, v, op);
}
struct Add {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};

// Entries e .. e + 3 of an array of n; behind its end the last one. (The array starts at
// any multiple of 4 bytes.)
typedef u32x4 __attribute__((aligned(4))) u32x4_any;
template <typename T>
__device__ __forceinline__ u32x4 four(const T* p, int e, int n) {
  if (e + 4 <= n) return *reinterpret_cast<const u32x4_any*>(p + e);
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(uint32_t, p[min(e + j, n - 1)]);
  return v;
}

// What the workgroups of a list share.
template <int THREADS>
struct Select {
  static constexpr int kWaves = THREADS / 64, kBins = 4 * THREADS, kBits = THREADS == 1024 ? 12 : 11;
  static_assert(1 << kBits == kBins);
  uint32_t bins[kBins];          // then holes and movers
  uint32_t slots[2][kWaves];
  u64 near[64];
  u64 range[2];
  u64 cut;
  uint32_t n, part, above;

  __device__ __forceinline__ static uint32_t last_lane(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  }
  // A value per wave: the sum over the waves before, and over all.
  __device__ __forceinline__ uint32_t before(int which, uint32_t v, uint32_t& all) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) slots[which][w] = v;
    __syncthreads();
    uint32_t b = 0;
    all = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      const uint32_t x = slots[which][i];
      b += i < w ? x : 0;
      all += x;
    }
    return b;
  }
};

// One workgroup a list. Wave w owns the rows [w C, (w + 1) C), 64 at a time, so that
// numbers in row order need one sum over the waves. CAP > 0: at most CAP rows, whose keys
// stay in LDS (in registers the sweeps had to be unrolled, and their code took longer to
// arrive than to run); 0: any length, keys read again for each sweep.
//
// A token's place in the order is its key, then its row from behind: one 64-bit number.
// The last kept one is found by dividing the range of the numbers in question into equal
// parts and counting, until at most 64 are left: once where masses differ, twice where rows
// decide.
//
// Bound by latency: one CU a list, one sweep behind the other. Of 32 lists of up to 32768 rows
// (4 sequences, 8 heads) to 2048, the longest list (29 us): latest position 2, keys 5, the
// division 5, last candidates 3, counts and lists of moves 8.5, writes 5.5. Of 64 lists of 2112
// rows (8.4 us): 0.8, 1.1, 1.9, 0.8, 1.6, 2.2.
template <int THREADS, int CAP>
__global__ __launch_bounds__(THREADS) void select_kernel(EvictArgs a) {
  using S = Select<THREADS>;
  constexpr int kBatch = 8;       // rows on their way a lane
  __shared__ S s;
  __shared__ __align__(16) uint32_t kept[CAP > 0 ? CAP : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t list = blockIdx.x;
  const int64_t n = list / a.G;
  const int Lmax = (int)a.kv.Lmax;
  const int len = min(max(a.lens[n], 0), Lmax);
  const int size = (int)min((int64_t)len, a.budget);
  const float* mass = a.mass + list * Lmax;
  const int32_t* pos = a.pos ? a.pos + list * Lmax : nullptr;
  int32_t* src = a.src + list * a.budget;
  const int runs = (len + THREADS - 1) / THREADS;   // of 64 rows, per wave
  const int base = wave * runs * 64 + lane;
  // the latest position
  int newest = len - 1;
  if (pos && a.recent > 0) {
    uint32_t top = 0;             // positions as unsigned numbers in the same order
#pragma unroll 4
    for (int e = 4 * (int)threadIdx.x; e < len; e += 4 * THREADS) {
      const u32x4 p = four(pos, e, len);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, p[j] ^ 0x80000000u);
    }
    top = S::last_lane(scan_wave(0, top, Max()));
    if (lane == 0) s.slots[0][wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::kWaves; ++i) top = max(top, s.slots[0][i]);
    newest = (int)(top ^ 0x80000000u);
    __syncthreads();
  }
  // open positions: from `sinks` up to the latest ones
  const int first = (int)a.sinks;
  const int64_t latest = a.recent > 0 ? newest - a.recent + 1 : (int64_t)1 << 31;
  const uint32_t open = (uint32_t)max(latest - first, (int64_t)0);

  // keys of the wave's runs i0 .. i0 + 7 (no branch between the loads)
  auto load = [&](int i0, uint32_t (&k)[kBatch]) __attribute__((always_inline)) {
    float m[kBatch];
    int p[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int e = min(base + 64 * (i0 + j), len - 1);
      m[j] = mass[e];
      p[j] = pos ? pos[e] : e;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      k[j] = i0 + j < runs && base + 64 * (i0 + j) < len ? rank_key(m[j], p[j], first, open) : 0u;
  };
  // the protected ones, and the range of the others
  uint32_t safe = 0, low = ~0u, high = 0;
  auto note = [&](uint32_t k) __attribute__((always_inline)) {
    safe += k == kProtected;
    low = min(low, k - 1);        // of no token: the largest number
    high = max(high, k + 1);      // of a protected one: 0
  };
  if constexpr (CAP > 0) {
#pragma unroll 4
    for (int e = 4 * (int)threadIdx.x; e < len; e += 4 * THREADS) {
      const u32x4 m = four(mass, e, len), p = pos ? four(pos, e, len) : u32x4{};
      u32x4 k;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[j] = e + j < len ? rank_key(__uint_as_float(m[j]), pos ? (int)p[j] : e + j, first, open) : 0u;
        note(k[j]);
      }
      *reinterpret_cast<u32x4*>(kept + e) = k;
    }
    for (int e = len + (int)threadIdx.x; e < min(runs * THREADS, CAP); e += THREADS)
      if (e >= (len + 3) / 4 * 4) kept[e] = 0;
    __syncthreads();
  } else {
    for (int i0 = 0; i0 < runs; i0 += kBatch) {
      uint32_t k[kBatch];
      load(i0, k);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) note(k[j]);
    }
  }
  // f(row, key) for the wave's runs in order
  auto sweep = [&](auto f) __attribute__((always_inline)) {
    for (int i0 = 0; i0 < runs; i0 += kBatch) {
      uint32_t k[kBatch];
      if constexpr (CAP > 0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) k[j] = kept[base + 64 * min(i0 + j, runs - 1)];
      } else {
        load(i0, k);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (i0 + j < runs) f(base + 64 * (i0 + j), k[j]);
    }
  };
  auto order = [](int e, uint32_t k) __attribute__((always_inline)) { return (u64)k << 32 | (uint32_t)~e; };

  u64 cut = (u64)1 << 32;      // the last kept token's number: any token's
  if (len > size) {
    safe = S::last_lane(scan_wave(0, safe, Add()));
    low = ~S::last_lane(scan_wave(0, ~low, Max()));
    high = S::last_lane(scan_wave(0, high, Max()));
    if (threadIdx.x == 0) {
      s.range[0] = ~0ull;
      s.range[1] = 0;
    }
    uint32_t all_safe;
    s.before(0, safe, all_safe);
    if (lane == 0) {              // a wave without tokens has low = 2^32 - 1, one of protected ones high = 0
      if (low < kProtected - 1) atomicMin(&s.range[0], (u64)(low + 1));
      if (high > 1) atomicMax(&s.range[1], (u64)(high - 1));
    }
    __syncthreads();
    u64 lo = s.range[0] << 32, hi = s.range[1] << 32 | 0xffffffffu;
    bool whole = true;                        // all rows of the keys from lo to hi
    int want = size - (int)all_safe;          // of those in question
    uint32_t here = (uint32_t)len - all_safe;
    if (want <= 0) {                          // there is no room for all protected ones: the first rows stay
      lo = (u64)kProtected << 32;
      hi = ~0ull;
      want = size;
      here = all_safe;
    }
    while (here > 64) {
      const int shift = max(0, 64 - __builtin_clzll(hi - lo) - S::kBits);   // kBins parts at most
      for (int i = threadIdx.x; i < S::kBins; i += THREADS) s.bins[i] = 0;
      __syncthreads();
      if (whole && shift >= 32) {             // parts of whole keys
        const uint32_t k0 = (uint32_t)(lo >> 32), k1 = (uint32_t)(hi >> 32);
        sweep([&](int, uint32_t k) __attribute__((always_inline)) {
          if (k >= k0 && k <= k1) atomicAdd(&s.bins[(k1 - k) >> (shift - 32)], 1u);
        });
      } else {
        sweep([&](int e, uint32_t k) __attribute__((always_inline)) {
          const u64 o = order(e, k);
          if (o >= lo && o <= hi) atomicAdd(&s.bins[(int)((hi - o) >> shift)], 1u);
        });
      }
      __syncthreads();
      // from the highest part down: thread i owns four
      uint32_t c[4], mine = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[j] = s.bins[4 * threadIdx.x + j];
        mine += c[j];
      }
      const uint32_t incl = scan_wave(0, mine, Add());
      uint32_t all;
      uint32_t above = s.before(1, S::last_lane(incl), all) + incl - mine;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (above < (uint32_t)want && above + c[j] >= (uint32_t)want) {
          s.part = 4 * threadIdx.x + j;
          s.above = above;
          s.n = c[j];
        }
        above += c[j];
      }
      __syncthreads();
      hi -= (u64)s.part << shift;
      const u64 width = (u64)1 << shift;
      lo = hi - lo >= width ? hi - width + 1 : lo;
      whole &= shift >= 32;
      want -= (int)s.above;
      here = s.n;
      __syncthreads();
    }
    if (threadIdx.x == 0) s.n = 0;
    __syncthreads();
    const uint32_t k0 = (uint32_t)(lo >> 32), k1 = (uint32_t)(hi >> 32);
    sweep([&](int e, uint32_t k) __attribute__((always_inline)) {
      if (k >= k0 && k <= k1) {
        const u64 o = order(e, k);
        if (o >= lo && o <= hi) s.near[atomicAdd(&s.n, 1u)] = o;
      }
    });
    __syncthreads();
    if (threadIdx.x < 64) {
      const u64 o = threadIdx.x < here ? s.near[threadIdx.x] : 0;
      int rank = 0;
      for (uint32_t i = 0; i < here; ++i) rank += s.near[i] >= o;
      if (o && rank == want) s.cut = o;
    }
    __syncthreads();
    cut = s.cut;
  }
  auto stays = [&](int e, uint32_t k) __attribute__((always_inline)) { return order(e, k) >= cut; };

  uint32_t holes = 0, moves = 0;
  sweep([&](int e, uint32_t k) __attribute__((always_inline)) {
    const bool stay = stays(e, k);
    const u64 here = __ballot(stay), front = __ballot(e < size);
    holes += __popcll(front & ~here);
    moves += __popcll(here & ~front);
  });
  uint32_t all_holes, all_moves;
  __syncthreads();
  uint32_t hole = s.before(0, holes, all_holes);
  uint32_t move = s.before(1, moves, all_moves);
  // lists of both, in LDS where they fit
  const bool fit = all_holes <= (uint32_t)S::kBins / 2;
  const int64_t room = min(a.budget, a.kv.Lmax);
  int32_t *const far_to = a.lists + 2 * list * room, *const far_from = far_to + room;
  int32_t *const to = reinterpret_cast<int32_t*>(s.bins), *const from = to + S::kBins / 2;
  sweep([&](int e, uint32_t k) __attribute__((always_inline)) {
    const bool stay = stays(e, k), h = e < size && !stay, m = e >= size && stay;
    const u64 bh = __ballot(h), bm = __ballot(m);
    if (bh) {
      const uint32_t i = hole + lanes_below(bh);
      if (h && fit) to[i] = e;
      if (h && !fit) far_to[i] = e;
      hole += __popcll(bh);
    }
    if (bm) {
      const uint32_t i = move + lanes_below(bm);
      if (m && fit) from[i] = e;
      if (m && !fit) far_from[i] = e;
      move += __popcll(bm);
    }
  });
  __syncthreads();
  // rows that stay, then holes; movers lie behind all of them, so that in place nothing is
  // written that is still to be read
  float* mass_out = a.mass_out ? a.mass_out + list * Lmax : nullptr;
  int32_t* pos_out = a.pos_out ? a.pos_out + list * Lmax : nullptr;
#pragma unroll 4
  for (int e = threadIdx.x; e < size; e += THREADS) {
    const float m = mass[e];
    const int p = pos ? pos[e] : e;
    uint32_t k;
    if constexpr (CAP > 0) k = kept[e];
    else k = rank_key(m, p, first, open);
    if (stays(e, k)) {
      src[e] = e;
      if (mass_out) mass_out[e] = m;
      if (pos_out) pos_out[e] = p;
    }
  }
  __syncthreads();
#pragma unroll 2
  for (uint32_t i = threadIdx.x; i < all_holes; i += THREADS) {
    const int e = fit ? to[i] : far_to[i], f = fit ? from[i] : far_from[i];
    src[e] = f;
    if (mass_out) mass_out[e] = mass[f];
    if (pos_out) pos_out[e] = pos ? pos[f] : f;
  }
  __syncthreads();
  for (int64_t i = size + (int)threadIdx.x; i < a.budget; i += THREADS) src[i] = -1;
  for (int i = size + (int)threadIdx.x; i < Lmax; i += THREADS) {
    if (mass_out) mass_out[i] = 0.f;
    if (pos_out) pos_out[i] = -1;
  }
}

// ---------------------------------------------------------------- moves
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;       // rows of a list that a workgroup looks at
constexpr int kMoveBatch = 8;       // pieces on their way a thread

// Bound by memory: 16-byte pieces of the rows that move, all heads of a row next to
// each other. The first wave looks up which of the workgroup's rows move, and the pages
// of both ends. New lengths are written here, one thread a sequence, and not by the selection:
// several of its workgroups read a sequence's length, and the two may be one array.
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
  } else if (threadIdx.x == kMoveRows && a.new_len && chunk == 0 && g == 0) {
    a.new_len[n] = (int)min((int64_t)min(max(a.lens[n], 0), (int)a.kv.Lmax), a.n);
  }
  __syncthreads();
  const uint32_t pieces = (uint32_t)count * heads * units, all = a.kv.v ? 2 * pieces : pieces;
  const int64_t head0 = a.G == 1 ? 0 : g * a.kv.head_stride;
  uint16_t *const k = a.kv.k + head0, *const v = a.kv.v + head0;
  for (uint32_t i0 = threadIdx.x; i0 < all; i0 += kMoveThreads * kMoveBatch) {
    u32x4 x[kMoveBatch];
    uint16_t* dst[kMoveBatch];
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j) {
      const uint32_t at = i0 + j * kMoveThreads, i = at < pieces ? at : at - pieces;
      dst[j] = nullptr;
      if (at >= all) continue;
      const uint32_t item = fast_quot(by_units, i), u = i - item * units;
      const uint32_t r = fast_quot(by_heads, item), h = item - r * heads;
      const int64_t off = h * a.kv.head_stride + 8 * u;
      uint16_t* base = at < pieces ? k : v;
      x[j] = *reinterpret_cast<const u32x4*>(base + from[r] + off);
      dst[j] = base + to[r] + off;
    }
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j)
      if (dst[j]) *reinterpret_cast<u32x4*>(dst[j]) = x[j];
  }
}

}  // namespace

hipError_t launch_evict_select(const EvictArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.kv.nseq * a.G));
  const int64_t L = a.kv.Lmax;
  // By the rows that a sequence can address: how many it holds is known on the device alone.
  // (Times: selection and moves of rows of 8 elements, to a budget of 2048.) Short lists: half the
  // waves and a sixth of the LDS, so that several lists share a CU: 512 lists of 2112 rows 28 us,
  // against 37 with the next shape and 42 with keys read again; 64 lists, which have a CU each, 13.8
  // against 14.8 and 17.8. Keys in LDS as long as they fit: 32 lists of 32768 rows 35 us against 48,
  // 512 of 30000 131 against 163. A shape for 8192 rows gained nothing (512 lists 50 us either way).
  // Few tokens in long rows cost what the rows do: 64 lists of 2112 tokens 14 us in rows of 4096, 19
  // in rows of 32768, 25 in rows of 65536, whose ends are cleared by one workgroup a list.
  if (L <= 4096) hipLaunchKernelGGL((select_kernel<512, 4096>), grid, dim3(512), 0, st, a);
  else if (L <= 32768) hipLaunchKernelGGL((select_kernel<1024, 32768>), grid, dim3(1024), 0, st, a);
  else hipLaunchKernelGGL((select_kernel<1024, 0>), grid, dim3(1024), 0, st, a);
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
