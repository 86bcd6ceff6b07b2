// Appending keys and values to a paged cache, with the rotary positions applied
// on the way (and to the queries of the same tokens, in the same launch).
//
// Pair i of the rotated part turns by the angle of its token's position:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// pairs being (i, i + rot / 2) or (2i, 2i + 1). Both products of a component are
// summed in fp32 and rounded once to the cache's type.
//
// Bound by memory: every element is read and written once. A thread owns the
// same 16 elements (two 16-byte pieces that hold 8 whole pairs) of several
// heads of one token, so that the token's 8 cosines and sines are read once for
// all of them, and requests the pieces of all its heads before it uses the
// first. Measured: 16384 tokens of 64 + 8 + 8 heads of 128 in 119 us, 5.6 TB/s (a
// large copy: 5.07); 64 tokens in 4.8 us, the time of any launch.
#include "misa_common.hpp"
#include "misa_kv.hpp"

namespace misa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsPerThread = 4;

template <bool HALF>
__device__ __forceinline__ float to_float(uint32_t word, int hi) {
  if (HALF) return (float)__builtin_bit_cast(_Float16, (uint16_t)(hi ? word >> 16 : word & 0xffffu));
  return hi ? bf16_hi(word) : bf16_lo(word);
}
template <bool HALF>
__device__ __forceinline__ uint32_t to_word(float lo, float hi) {   // nearest, ties to even
  if (HALF)
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)lo) |
           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)hi) << 16;
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
}

// units: pieces of 16 elements per head (d / 16); lanes: threads that share a
// token's unit, each taking the heads lane, lane + lanes, ...
template <bool HALF, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a, int units, int lanes, int per_block) {
  const int u = threadIdx.x % units;
  const int rest = threadIdx.x / units;
  const int lane = rest % lanes;
  const int slot = rest / lanes;
  const int64_t n = (int64_t)blockIdx.x * per_block + slot;
  if (slot >= per_block || n >= a.N) return;
  const int seq = a.seq[n], tok = a.tok[n];
  if (seq < 0 || seq >= a.kv.nseq || tok < 0 || tok >= a.kv.Lmax) return;
  const int pos = a.pos ? a.pos[n] : tok;
  if (a.rot && (pos < 0 || pos >= a.P)) return;
  const uint32_t col = fast_quot(a.kv.by_page, (uint32_t)tok);
  const int page = kv_page(a.kv, seq, col);
  if (page < 0) return;
  const int64_t row = page * a.kv.page_stride + (int64_t)(tok - (int)col * a.kv.page) * a.kv.tok_stride;

  // the two pieces of this thread: 8 pairs of the rotated part, or 16 elements behind it
  const bool turn = 16 * u < a.rot;
  int c0, c1;
  if (INTERLEAVED || !turn) {
    c0 = 16 * u;
    c1 = c0 + 8;
  } else {
    c0 = 8 * u;
    c1 = c0 + a.rot / 2;
  }
  float cs[8], sn[8];
  if (turn) {
    const float* r = a.cos_sin + (int64_t)pos * a.rot + 8 * u;
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = r[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) sn[i] = r[a.rot / 2 + i];
  }
  const int heads = a.Hq + a.Hkv + (a.v ? a.Hkv : 0);
  for (int h0 = lane; h0 < heads; h0 += lanes * kHeadsPerThread) {
    u32x4 x[kHeadsPerThread][2];
    uint16_t* dst[kHeadsPerThread];
#pragma unroll
    for (int j = 0; j < kHeadsPerThread; ++j) {
      const int h = h0 + j * lanes;
      const uint16_t* src;
      dst[j] = nullptr;
      if (h >= heads) continue;
      if (h < a.Hq) {
        src = a.q + n * a.q_ts + h * a.q_hs;
        dst[j] = a.q_out + n * a.o_ts + h * a.o_hs;
      } else if (h < a.Hq + a.Hkv) {
        src = a.k + n * a.k_ts + (h - a.Hq) * a.k_hs;
        dst[j] = a.kv.k + row + (h - a.Hq) * a.kv.head_stride;
      } else {
        src = a.v + n * a.v_ts + (h - a.Hq - a.Hkv) * a.v_hs;
        dst[j] = a.kv.v + row + (h - a.Hq - a.Hkv) * a.kv.head_stride;
      }
      // values are stored as they are: any split into pieces does
      x[j][0] = *reinterpret_cast<const u32x4*>(src + c0);
      x[j][1] = *reinterpret_cast<const u32x4*>(src + c1);
    }
#pragma unroll
    for (int j = 0; j < kHeadsPerThread; ++j) {
      if (!dst[j]) continue;
      if (turn && h0 + j * lanes < a.Hq + a.Hkv) {
        if (INTERLEAVED) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float xa = to_float<HALF>(x[j][p][e], 0), xb = to_float<HALF>(x[j][p][e], 1);
              const float c = cs[4 * p + e], s = sn[4 * p + e];
              x[j][p][e] = to_word<HALF>(xa * c - xb * s, xb * c + xa * s);
            }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a0 = to_float<HALF>(x[j][0][e], 0), a1 = to_float<HALF>(x[j][0][e], 1);
            const float b0 = to_float<HALF>(x[j][1][e], 0), b1 = to_float<HALF>(x[j][1][e], 1);
            x[j][0][e] = to_word<HALF>(a0 * cs[2 * e] - b0 * sn[2 * e], a1 * cs[2 * e + 1] - b1 * sn[2 * e + 1]);
            x[j][1][e] = to_word<HALF>(b0 * cs[2 * e] + a0 * sn[2 * e], b1 * cs[2 * e + 1] + a1 * sn[2 * e + 1]);
          }
        }
      }
      *reinterpret_cast<u32x4*>(dst[j] + c0) = x[j][0];
      *reinterpret_cast<u32x4*>(dst[j] + c1) = x[j][1];
    }
  }
}

}  // namespace

// Threads of a workgroup: `units` pieces times `lanes` heads times tokens.
static void split_of(const AppendArgs& a, int& units, int& lanes, int& per_block) {
  units = a.d / 16;
  const int heads = a.Hq + a.Hkv + (a.v ? a.Hkv : 0);
  lanes = 1;
  while (2 * lanes * units <= kThreads && lanes < heads) lanes *= 2;
  per_block = kThreads / (units * lanes);
}

int64_t append_blocks(const AppendArgs& a) {
  int units, lanes, per_block;
  split_of(a, units, lanes, per_block);
  return (a.N + per_block - 1) / per_block;
}

hipError_t launch_append(const AppendArgs& a, hipStream_t st) {
  int units, lanes, per_block;
  split_of(a, units, lanes, per_block);
  const dim3 grid((unsigned)append_blocks(a));
#define MISA_APPEND(HALF_, INTER_) \
  hipLaunchKernelGGL((append_kernel<HALF_, INTER_>), grid, dim3(kThreads), 0, st, a, units, lanes, per_block)
  if (a.half) {
    if (a.interleaved) MISA_APPEND(true, true);
    else MISA_APPEND(true, false);
  } else {
    if (a.interleaved) MISA_APPEND(false, true);
    else MISA_APPEND(false, false);
  }
#undef MISA_APPEND
  return hipGetLastError();
}

}  // namespace misa
