// Launcher interface and device helpers of the key/value cache: a paged (or
// one-row-per-sequence) cache addressed by (sequence, token).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace misa {

// Quotient by a divisor that is fixed for a launch, for n < 2^31: with
// l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// floor(n / d) = (mulhi(m, n) + n) >> l (multiplication by the reciprocal,
// Granlund and Montgomery 1994); mulhi(m, n) + n < 2^32 because n < 2^31.
struct FastDiv {
  uint32_t m = 1;
  uint32_t shift = 0;
};

inline FastDiv fast_div(uint32_t d) {
  FastDiv f;
  while (f.shift < 32 && (uint64_t(1) << f.shift) < d) ++f.shift;
  f.m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << f.shift) - d)) / d + 1);
  return f;
}

__device__ __forceinline__ uint32_t fast_quot(FastDiv f, uint32_t n) { return (__umulhi(f.m, n) + n) >> f.shift; }

// One cache: rows of d elements of 16 bits, in pages. Strides in elements.
struct KvView {
  uint16_t* k;
  uint16_t* v;              // may be null (keys alone)
  int64_t page_stride;
  int64_t tok_stride;
  int64_t head_stride;
  int64_t npages;
  int32_t page;             // tokens per page
  FastDiv by_page;
  const int32_t* table;     // [nseq][table_stride] page ids, or null: page = sequence
  int64_t table_stride;
  int64_t nseq;
  int64_t Lmax;             // tokens a sequence can address: cols * page, or page
  // Row (page p, row r) of a head lies p * page_units + r * tok_units units behind
  // the head's first one, in 32 bits: bytes where the cache ends before 4 GiB
  // (unit_shift 0; bytes: its extent), else 2^unit_shift elements.
  uint32_t page_units;
  uint32_t tok_units;
  uint32_t unit_shift;
  uint32_t bytes;
};

// Page of token s of sequence seq (seq, s in range); -1 if the table holds no page of the cache.
__device__ __forceinline__ int kv_page(const KvView& c, int seq, uint32_t col) {
  if (!c.table) return seq;
  const int p = c.table[(int64_t)seq * c.table_stride + col];
  return (p >= 0 && p < c.npages) ? p : -1;
}

struct AppendArgs {
  KvView kv;
  const uint16_t* k;        // [N][Hkv][d], strides below
  const uint16_t* v;        // or null
  const uint16_t* q;        // [N][Hq][d] or null
  uint16_t* q_out;
  int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, o_ts, o_hs;
  const int32_t* seq;       // [N]
  const int32_t* tok;       // [N]
  const int32_t* pos;       // [N] or null: tok
  const float* cos_sin;     // [P][rot] or null
  int64_t P;
  int64_t N;
  int Hq, Hkv, d, rot;
  bool interleaved;
  bool half;                // fp16 (else bf16)
};
int64_t append_blocks(const AppendArgs& a);   // workgroups (of 256 threads) of its launch
hipError_t launch_append(const AppendArgs& a, hipStream_t st);

}  // namespace misa
