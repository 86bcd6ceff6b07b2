// Arguments and launchers of the attention kernels (attend_kernel.hpp, attend.hip).
#pragma once

#include "misa_kv.hpp"

namespace misa {

// Which keys a pass visits for query t.
enum AttendMode : int {
  kAttendPlain = 0,   // tokens [start, len) of its sequence, or its selected ids
  kAttendPrefix = 1,  // the tokens of its shared prefix
  kAttendOwn = 2,     // its own tokens behind the shared prefix
};

// Batches of at most this many queries are planned (see attend_kernel.hpp).
constexpr int kPlanMax = 256;

// What the join needs to know of a query's part of the plan.
struct PlanEntry {
  int32_t first;   // key tiles of the segments before its own (per head tile)
  int32_t tiles;   // key tiles of its segment
  int32_t t0;      // first query of its segment
};

struct AttendArgs {
  KvView kv;
  const uint16_t* q;        // [T][Hq][d]
  int64_t q_ts, q_hs;
  const int32_t* q_seq;     // [T]
  const int32_t* q_start;   // [T] or null: 0
  const int32_t* q_len;     // [T]
  const int32_t* q_pos;     // [T] or null: the last visible token's position
  const int32_t* idx;       // [T][topk] selected token ids, or null
  int32_t topk;
  AttendMode mode;
  const int32_t* pre;       // [T] shared prefix of the query (outside [0, npre): none)
  const int32_t* pre_len;   // [npre]
  int64_t npre;
  int64_t pre_max;          // tokens a prefix can address
  const int32_t* own_seq;   // kAttendPrefix: [T] the queries' own sequences, and their count
  int64_t own_nseq;
  int64_t T;
  int32_t d;
  int32_t Hq, Hkv, group;   // group = Hq / Hkv query heads read one kv head
  int32_t gw;               // query heads of a row tile: min(group, R)
  int32_t head_tiles;       // ceil(group / gw)
  int32_t qt;               // queries of a row tile: R / gw
  int32_t NH;               // Hkv * head_tiles
  FastDiv by_gw;
  int32_t align;            // a part's keys start at a multiple of this (1 or Shape::WR)
  float scale;
  float cap;                // 0: none
  const float* slopes;      // [Hq] or null
  uint16_t* out;            // [T][Hq][d]; null: out32
  float* out32;
  float* lse;               // [T][Hq] or null
  // one word a workgroup, set if its parts have to be computed again by the
  // guarded form; null where all rows of a part see the same keys
  int32_t* odd;
  uint32_t blocks;          // workgroups of the launch
  // planned batches
  int32_t planned;
  int32_t G;                // workgroups
  float* part_out;          // [2 G][R][d]
  float* part_ml;           // [2 G][R][2]
  PlanEntry* plan;          // [T]
  int32_t* plan_total;      // [1] key tiles of all segments
};

// Rows (query, head) of a workgroup's tile for a batch: 16, 32, 64 or 128.
// single: a row tile takes one query (selected tokens are each query's own; in a
// decode step no two queries share a sequence).
int attend_rows(int64_t T, int64_t nseq, int group, int d, bool single);
bool attend_planned(int64_t T, int64_t most_keys);
// Workgroups of a planned launch, and the workspace of a pass (the same whether a
// batch of at most kPlanMax queries is planned or has too many key tiles for it).
int attend_groups(int d, int R);
size_t attend_ws_bytes(int64_t T, int Hq, int heads, int d, int R, bool single, bool mixed);
// Fills the fields that depend on the tile and carves the workspace.
// mixed: rows of one part may see different keys, or not all keys of its steps
// (several queries a row tile, intervals that start behind a sequence's first key).
void attend_setup(AttendArgs& a, int R, bool single, bool mixed, void* ws);
int64_t attend_blocks(const AttendArgs& a);
// The rows of one pass; those that it leaves in parts want a join.
hipError_t launch_attend(const AttendArgs& a, int R, bool half, hipStream_t st);
// Joins the parts of planned passes: of one (b null; rows that are whole are
// left alone), or of two over different keys of the same rows, into out and lse
// (both passes' whole rows in their out32 and lse).
hipError_t launch_attend_join(const AttendArgs& a, int Ra, const AttendArgs* b, int Rb, uint16_t* out, float* lse,
                              bool half, hipStream_t st);

// Per head dimension, in translation units of their own.
hipError_t launch_attend_d64(const AttendArgs& a, int R, bool half, unsigned blocks, hipStream_t st);
hipError_t launch_attend_d128(const AttendArgs& a, int R, bool half, unsigned blocks, hipStream_t st);
hipError_t launch_attend_d256(const AttendArgs& a, int R, bool half, unsigned blocks, hipStream_t st);

}  // namespace misa
