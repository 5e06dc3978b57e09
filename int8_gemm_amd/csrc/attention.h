// Arguments and launchers of the attention half of a block (rope.hip, attention.hip).
#pragma once

#include "internal.h"

namespace convrot {

// ---- rotary table ----
constexpr int kMaxRopePairs = 128;
constexpr int kMaxRopeAxes = 8;
enum class PosType { kI32 = 0, kI64 = 1, kF32 = 2 };
struct RopeTableArgs {
  const void* positions;
  int64_t token_stride, axis_stride;  // elements
  int64_t tokens;
  int pairs;
  double log2_theta;
  int axes;
  int first[kMaxRopeAxes + 1];  // first pair of each axis
  int shared;
  float* table;
};
hipError_t launch_rope_table(const RopeTableArgs& a, PosType type, hipStream_t st);

// ---- norms of q and k with the rotation ----
struct HeadsTensor {
  const uint16_t* in;
  uint16_t* out;
  const uint16_t* weight;
  int64_t in_stride, in_head_stride, out_stride, out_head_stride;
  int heads;
};
struct HeadsArgs {
  HeadsTensor t[2];  // q, k (heads 0: absent)
  const float* table;
  int64_t tokens, table_rows;
  int d, pairs;
  NormKind norm;
  bool row;  // norms over all heads of a token
  float eps;
};
// Whether a token's heads fit the lanes of a block (norms over rows).
bool heads_row_fits(int64_t heads, int d);
bool heads_grid_fits(const HeadsArgs& a);  // tokens < 2^31
hipError_t launch_qk_norm_rope(const HeadsArgs& a, bool halves, DType dt, hipStream_t st);

// ---- attention ----
struct AttentionArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;
  int64_t q_stride, q_head_stride, k_stride, k_head_stride, v_stride, v_head_stride, out_stride,
      out_head_stride;
  const int32_t *q_offsets, *k_offsets, *k_lens;
  int64_t q_tokens, k_tokens;
  int batch, q_heads, k_heads, d;
  bool causal;
  float scale;
  int tile;  // rows of a block's tile, 0: by the sizes
  int group, q_each, k_each;  // query heads of a key head; tokens of equal sequences
  // splits > 1: the tiles from `whole` on (few rows: all) go by parts, each split's
  // normalised rows and their log2 sums, joined by a second launch
  int splits;
  uint32_t whole;
  int few_blocks;   // few rows: blocks that the keys in use are shared out to
  float* part;      // few rows: [block][row of its tile][d]; else [tile][split][row][d]
  float* part_lse;  // the same without d
  int part_step;    // rows of a tile
  int64_t parts;    // rows of all blocks' parts
  int64_t* part_map;  // [tile][row]: row of the output, -1 for none; few rows: by row of
                      // the output, its first part and how many there are (int32 each)
};
// How a call is cut.
struct AttentionPlan {
  int rows = 0;        // rows (query, head of the group) of a block's tile; 32: few rows
  int64_t slots = 0;   // tiles per key head, at most
  int64_t whole = 0;   // tiles of a block each
  int splits = 1;      // parts of each of the others
  int64_t part_rows = 0;  // entries of the map
  int part_step = 0;      // rows of a tile's part
  int few_blocks = 0;     // few rows: as above
  int64_t grid = 0;
};
// By sizes and the workspace's bytes alone, so that results do not depend on the device.
AttentionPlan plan_attention(const AttentionArgs& a, size_t workspace);
size_t attention_workspace(const AttentionArgs& a, const AttentionPlan& p);
// Fill in the plan, the workspace's parts and what the kernels need of the sizes.
void attention_use(AttentionArgs* a, const AttentionPlan& p, void* workspace);
hipError_t launch_attention(const AttentionArgs& a, const AttentionPlan& p, DType dt,
                            hipStream_t st);

}  // namespace convrot
