// pkv_latent.h -- parameter blocks and launchers of the calls around a latent
// cache, and of the norm and rotation ahead of the append.
#pragma once

#include "pkv_internal.h"

namespace pkv {

constexpr int kLatent = 512;               // dims of a cached latent (the values)
constexpr int kRopeDim = 64;               // dims of the rotated key beside it
constexpr int kLatRow = kLatent + kRopeDim;  // a cached row
constexpr int kNope = 128;                 // an expanded head's unrotated key ...
constexpr int kValDim = 128;               // ... and value
constexpr int kMaxLatentHeads = 128;       // query heads of the absorbed form

// Norm of queries and keys head by head, rotation, append to bf16 pools.
struct NormRopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long q_stride, k_stride, v_stride, out_stride;  // elements between tokens
  const int64_t* positions;
  const float* cos_sin;  // [max_position, rot]: cos | sin
  const int64_t* slot_mapping;
  const __nv_bfloat16* q_weight;  // [128] or null: no norm
  const __nv_bfloat16* k_weight;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_pool;
  __nv_bfloat16* v_pool;
  int* err;
  float eps;
  long long max_position;
  int rot, interleaved;
  int num_tokens, num_q_heads, num_kv_heads, num_blocks;
  int pdl;
};

cudaError_t launch_norm_rope_append(const NormRopeParams& p, int sm_count, cudaStream_t stream);

// Norm of the latent, rotation of its key part, append to a latent pool; and
// the rotation of the queries' part that meets it.
struct AppendLatentParams {
  const __nv_bfloat16* kv;  // [tokens][512 latent | 64 to be rotated]
  long long kv_stride;
  const int64_t* positions;
  const float* cos_sin;  // [max_position, 64]
  const int64_t* slot_mapping;
  const __nv_bfloat16* weight;  // [512] or null
  __nv_bfloat16* pool;          // [num_blocks, 16, 576]
  const __nv_bfloat16* q_rope;  // [tokens][heads][64], or null
  __nv_bfloat16* q_rope_out;
  long long q_stride, q_head_stride, out_stride, out_head_stride;
  int* err;
  float eps;
  long long max_position;
  int interleaved;
  int num_tokens, num_q_heads, num_blocks;
  int pdl;
};

cudaError_t launch_append_latent(const AppendLatentParams& p, int sm_count, cudaStream_t stream);

// Absorbed attention over a paged latent cache.
constexpr int kLatMaxRows = 64;  // MMA columns: (token, head) pairs of one work item

struct LatentDecodeParams {
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* qsl;
  const __nv_bfloat16* pool;
  __nv_bfloat16* out;  // [tokens, Hq, 512]
  // Pieces of rows cut at CTA range boundaries: per CTA its first and its last
  // (LatentPiece), their states and unnormalised outputs.
  int* piece;      // [2 * grid][kPieceWords]
  float* piece_ml; // [2 * grid][piece_rows][2]
  float* piece_o;  // [2 * grid][piece_rows][512]
  int piece_rows;  // group_heads * group_tokens
  int* err;
  int num_reqs, num_q_tokens, num_q_heads, num_blocks, max_blocks;
  int head_groups;  // 1, or 2 for more than 64 heads
  int group_heads;  // heads of a work item (the last group may have fewer)
  int group_tokens; // query tokens of a work item (the last may have fewer)
  int item_cost;    // a work item counts as its keys plus this many
  int min_keys;     // shortest range of a CTA
  int merge;        // rows may be cut: the merge kernel follows
  float scale_log2;
  int early_plan;
  int pdl;
  unsigned long long wait_limit_ns;
};

constexpr int kPieceWords = 8;

struct LatentDecodeLaunch {
  CUtensorMap qmap;  // q as [tokens][Hq][576], box (64, group_heads, group_tokens)
  CUtensorMap kmap;  // pool as [num_blocks * 16][576], box (64, 16), 128-byte swizzle
  LatentDecodeParams p;
  int grid;
};

cudaError_t launch_latent_decode(const LatentDecodeLaunch& L, cudaStream_t stream);

}  // namespace pkv
