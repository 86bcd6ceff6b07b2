// Arguments and launchers of what bounds a cache (accumulated attention weight,
// eviction, moves of rows) and of sampling (mass.hip, evict.hip, sample.hip).
#pragma once

#include "misa_kv.hpp"

namespace misa {

struct MassArgs {
  KvView kv;
  const uint16_t* q;        // [T][Hq][d]
  int64_t q_ts, q_hs;
  const float* lse;         // [T][Hq]
  const int32_t* q_seq;     // [T]
  const int32_t* q_start;   // [T] or null: 0
  const int32_t* q_len;     // [T]
  const int32_t* q_pos;     // [T] or null: q_len - 1
  int64_t T;
  int32_t d;
  int32_t Hq, Hkv, group;
  FastDiv by_group;
  float scale, cap;
  const float* slopes;      // [Hq] or null
  const float* in;          // [nseq][G][Lmax] or null: zeros
  float* out;
  int32_t G;                // Hkv, or 1: summed over the heads
  bool few;                 // few rows a sequence
  // sums over part c of `splits` of what sees a tile of keys in part[c][nseq][Hkv][Lmax]; null: straight to out
  int32_t splits;
  float* part;
};
bool mass_few(int64_t T, int64_t nseq, int group, int64_t q_ts, int64_t q_hs);
// Parts that a tile's queries are split into (1: not split), a power of two.
int mass_splits(int64_t T, int64_t nseq, int heads, int group, int64_t Lmax, int d);
int64_t mass_blocks(const MassArgs& a);   // workgroups (of 256 threads) of its largest launch
hipError_t launch_mass(const MassArgs& a, bool half, hipStream_t st);

struct EvictArgs {
  KvView kv;
  const float* mass;        // [nseq][G][Lmax]
  const int32_t* pos;       // the same shape, or null: row numbers
  const int32_t* lens;      // [nseq]
  int32_t G;                // lists of a sequence: Hkv, or 1 for all heads
  int64_t budget, sinks, recent;
  float* mass_out;          // may be mass, or null
  int32_t* pos_out;         // may be pos, or null
  int32_t* src;             // [nseq][G][budget]
  int32_t* lists;           // [nseq][G][2][min(budget, Lmax)] workspace
};
hipError_t launch_evict_select(const EvictArgs& a, hipStream_t st);

struct MoveArgs {
  KvView kv;
  int32_t Hkv, d;
  const int32_t* src;       // [nseq][G][n]
  int32_t G;
  int64_t n;
  // behind an eviction (null otherwise): new_len[i] = lens[i], clamped to what a sequence can
  // address, n at most; may be the same array
  const int32_t* lens;
  int32_t* new_len;
};
int64_t move_blocks(const MoveArgs& a);   // workgroups (of 256 threads)
hipError_t launch_move(const MoveArgs& a, hipStream_t st);

struct SampleArgs {
  const void* logits;       // [T][V], rows row_stride elements apart
  int64_t row_stride;
  int64_t T;
  int32_t V;
  const float* temperature; // [T] each, or null
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;           // [T]
  int32_t* token;           // [T]
  float* logprob;           // [T] or null
};
constexpr int32_t kMaxVocab = 1 << 20;
size_t sample_ws_bytes(int64_t T, int32_t V);
// type: 1 bf16, 2 fp16, 3 fp32
hipError_t launch_sample(const SampleArgs& a, int type, void* ws, hipStream_t st);

}  // namespace misa
