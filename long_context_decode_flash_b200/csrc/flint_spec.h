// flint_spec.h -- kernel parameters and launchers of the speculative-decode
// calls (tree attention, verification, norm and rotary at given positions,
// append of an accepted path).
#pragma once

#include "flint_internal.h"

namespace flint {

constexpr int kMaxTree = FLINT_MAX_TREE;

// ---- flint_qk_norm_rope_at ----------------------------------------------------
struct RopeAtParams {
  const uint16_t* q_raw;     // or nullptr: no q rows
  const uint16_t* k_raw;     // or nullptr: no k rows
  int64_t q_stride, k_stride;  // elements between tokens
  const uint16_t* w_q;       // nullptr: no norm
  const uint16_t* w_k;
  const int32_t* pos;
  uint16_t* q_out;
  uint16_t* k_out;
  int32_t T;
  int32_t rotary_dim;        // 0: no rotation
  int32_t layout;            // flint_rope_layout
  float eps;
  float attn_factor;
  double turns[kDim / 2];    // f_i / (2 pi): a pair's turns per position
};
cudaError_t launch_rope_at(const RopeAtParams& p, int num_sms, cudaStream_t stream);

// ---- flint_kv_append_path -------------------------------------------------------
struct PathLayer {
  const uint16_t* k;
  const uint16_t* v;
  uint8_t* k_rows;           // the cache's buffers
  uint8_t* v_rows;
  const int32_t* table;
  int64_t req_stride;        // elements
  int32_t layout, capacity, max_blocks, num_blocks, fp8;
  float k_scale[4], v_scale[4];
  float k_inv[4], v_inv[4];  // 1 / scale rounded, 0 where that may not be a normal number
};
struct AppendPathParams {
  PathLayer layer[FLINT_MAX_LAYERS];
  int32_t len[FLINT_MAX_BATCH];
  const int32_t* path;
  const int32_t* n_accepted;
  int32_t* dev_err;
  int32_t n_layers, N, B;
};
static_assert(sizeof(AppendPathParams) <= 32000, "kernel parameters exceed 32 KiB");
cudaError_t launch_append_path(const AppendPathParams& p, int num_sms, cudaStream_t stream);

// ---- flint_verify_tree ------------------------------------------------------------
struct VerifyParams {
  const float* target;
  const float* draft;        // or nullptr: fixed candidates
  int64_t target_stride, draft_stride;
  const int32_t* tokens;
  const int32_t* parent;
  const float* u_accept;
  const float* u_sample;
  int32_t* path;
  int32_t* n_accepted;
  int32_t* next_token;
  int32_t* dev_err;
  int32_t B, N, V;
  int8_t n_draft[FLINT_MAX_BATCH];
};
cudaError_t launch_verify(const VerifyParams& p, int num_sms, cudaStream_t stream);

// ---- flint_attn_tree ----------------------------------------------------------------
// A partial: O of 128 rows (16 nodes x 8 heads), m and l, fp32.  A CTA may leave
// two items unfinished (its first and its last) of up to two partials each, and
// CTAs come in groups of four, one per KV head.
constexpr int kTreePartialFloats = 128 * kDim + 2 * 128;
constexpr size_t kTreeGroupBytes = size_t(kKvHeads) * 2 * 2 * kTreePartialFloats * 4;

// A unit: up to 32 nodes of a request (mt row tiles of 16) against its keys, in
// tiles of two 64-key halves: half 0 the drafted tokens, half h >= 1 the cache's
// storage rows (positions; slots of a ring) base + 64 (h - 1) .., of which
// [lo, hi) hold tokens that some node attends.  The part_n rows from part on (of a
// ring: modulo its 513 slots) are those that some node may not attend: a window's
// oldest, and the slot before them.
constexpr int kMaxTreeUnits = FLINT_MAX_BATCH * (kMaxTree / 32);
struct alignas(32) TreeUnit {
  int16_t b;
  int8_t rb, mt;
  int8_t dup;                // copies of the rows in the row tile
  int8_t nodes;              // the request's nodes
  int32_t base, lo, hi;
  int32_t halves, tiles;
  int32_t len;               // the request's committed tokens
  int32_t part, part_n;
  int16_t q0, q1;            // the groups that hold a share of it
};
struct TreeCut {
  int16_t unit, tile;
};
constexpr int kMaxTreeGroups = kMaxCtas / kKvHeads;

struct TreeParams {
  // [128 dims][4 heads][capacity | 64 tokens][B | num_blocks], 128-byte swizzle,
  // boxes of 64 tokens x 128 bytes (64 dims bf16, 128 dims E4M3)
  CUtensorMap k_map, v_map;
  // [128 dims][32 | 4 heads][B * N nodes] bf16, boxes of 64 dims: 8 heads x 8
  // nodes, 1 head x 64 nodes
  CUtensorMap q_map, kd_map, vd_map;
  // the same buffers by address (bf16; k and v: the cache's)
  const uint16_t *q, *k_draft, *v_draft, *k, *v;
  int64_t req_stride;          // elements
  const int32_t* parent;
  const float* sinks;
  uint16_t* out;
  float* partials;
  const int32_t* table;
  int32_t layout, max_blocks, num_blocks, fp8;
  float k_scale[4], v_scale[4];
  double k_inv[4], v_inv[4];   // 1 / scale
  int32_t len[FLINT_MAX_BATCH];
  int8_t n_draft[FLINT_MAX_BATCH];
  int32_t N, B, window;
  int32_t n_units, n_groups;
  int32_t n_cut, cut_nodes;          // units that leave partials, and the most nodes of one
  TreeUnit unit[kMaxTreeUnits];
  TreeCut cut[kMaxTreeGroups + 1];   // group q: from cut[q] to cut[q + 1]
  int16_t cut_unit[kMaxTreeGroups];  // the units that leave partials
  int32_t* dev_err;
};
static_assert(sizeof(TreeParams) <= 32000, "kernel parameters exceed 32 KiB");
// Fills unit, cut, cut_unit and their counts from len, n_draft, B, window,
// layout and fp8, for at most num_groups groups of CTAs.
void plan_tree(TreeParams& p, int num_groups);
cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream);

}  // namespace flint
