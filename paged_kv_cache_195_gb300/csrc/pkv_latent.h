// pkv_latent.h -- parameter blocks and launchers of the calls around a latent
// cache, and of the norm and rotation ahead of the append.
#pragma once

#include "pkv_internal.h"

namespace pkv {

#ifdef __CUDACC__
// mbar_wait with everything past its first probe out of line: the kernels that
// use it run several roles' code at once, and a step of few rows runs most of it
// once, at the price of its instruction fetches.
static __device__ __noinline__ bool wait_spin(uint64_t* bar, uint32_t parity, int* err, WaitCtl* ctl) {
  return mbar_wait(bar, parity, err, ctl);
}

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int* err, WaitCtl* ctl) {
  return mbar_try_wait(bar, parity) || wait_spin(bar, parity, err, ctl);
}

// Ways out of an aborted call.  Copies in flight must land before a CTA ends; those
// whose barrier will not tell (the other CTA of a pair did not issue its part, or it
// counts on the other's barrier) are given a time by which any copy has landed.
constexpr unsigned long long kSettleNs = 10000000ull;

static __device__ __noinline__ void settle() {
  const unsigned long long t0 = global_timer_ns();
  while (global_timer_ns() - t0 < kSettleNs) __nanosleep(1000);
}

static __device__ __noinline__ void drain(uint64_t* bar, uint32_t parity, int* err, WaitCtl* ctl) {
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    const unsigned long long waited = global_timer_ns() - t0;
    if (waited > ctl->limit_ns && waited > kSettleNs) {
      record_error(err, kErrTimeout);
      return;
    }
  }
}

// The same value in all lanes, in a uniform register; and a vote.  Warps that issue
// MMAs or copies keep their control flow uniform with these and guard nothing but
// the instructions with one thread, so that descriptors and coordinates are in
// uniform registers: an MMA takes 24 cycles to issue then, and 50 to 80 else.
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ bool all_of(bool v) { return __all_sync(0xffffffffu, v); }
#endif

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
  int debug_withhold_q;
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

// Cached latents expanded to keys and values of every head.
struct LatentExpandParams {
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* kv_start;     // [num_reqs + 1]: rows of kv of each request
  const __nv_bfloat16* pool;   // [num_blocks, 16, 576]
  __nv_bfloat16* kv;           // [num_rows, num_heads, 256]
  __nv_bfloat16* k_rope;       // [num_rows, 64]
  int* err;
  int num_reqs, num_rows, num_heads, num_blocks, max_blocks;
  int pdl;
  int debug_withhold_q;
  unsigned long long wait_limit_ns;
};

struct LatentExpandLaunch {
  CUtensorMap kmap;  // as LatentDecodeLaunch::kmap
  CUtensorMap wmap;  // weight as [1][num_heads * 256][512], box (64, 128, 1), 128-byte swizzle
  LatentExpandParams p;
  int grid;
};

cudaError_t launch_latent_expand(const LatentExpandLaunch& L, cudaStream_t stream);

// Causal attention of chunks over expanded keys and values.
struct LatentPrefillParams {
  const int32_t* seq_lens;
  const int32_t* qsl;
  const int32_t* kv_start;
  const __nv_bfloat16* kv;     // [num_rows, H, 256]: key | value
  const __nv_bfloat16* k_rope; // [num_rows, 64]
  __nv_bfloat16* out;          // [num_q_tokens, H, 128]
  // Partial states of items split over their keys, by piece number.
  int* piece;                  // [max_pieces][4]: pieces of the item (first pieces only), its rows, head
  int* num_pieces;             // pieces to be joined
  float* piece_ml;             // [max_pieces][128][2]
  float* piece_o;              // [max_pieces][128][128]
  // [0] pieces handed out beyond each CTA's (pair's) first, [1] CTAs done, from bit 32 on
  // those of them that gave up on a wait; zero between launches.
  unsigned long long* sched;
  int* err;
  int wide;                    // out is aligned to 32 bytes
  int num_reqs, num_q_tokens, num_rows, num_heads;
  int max_pieces;              // 0: items are not split
  float scale_log2;
  int pdl;
  int debug_withhold_q;
  unsigned long long wait_limit_ns;
};

struct LatentPrefillLaunch {
  CUtensorMap qmap;   // q as [tokens][H][192], box (64, 1, 128), 128-byte swizzle
  CUtensorMap kvmap;  // values: kv as [rows][H][256], same box
  CUtensorMap kmap;   // keys: the same; a pair's box (64, 1, 64)
  CUtensorMap rmap;   // k_rope as [1][rows][64], box (64, 128, 1); a pair's (64, 64, 1)
  LatentPrefillParams p;
  int pairs;          // two query tiles of a head by two CTAs
  int grid;
};

cudaError_t launch_latent_prefill(const LatentPrefillLaunch& L, cudaStream_t stream);

}  // namespace pkv
