// pkv_api.cu -- the C ABI of libpagedkv.so (declared in include/pagedkv.h):
// argument validation, per-device state, workspace carve-up and launches.
// No call allocates on the hot path (the NULL-workspace convenience path
// allocates once per device), none synchronises, so a whole step can be
// captured in a CUDA graph.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "../../include/pagedkv.h"
#include "pkv_internal.h"
#include "pkv_latent.h"

static_assert(PKV_MAX_REQS == pkv::kMaxReqs, "request limit mismatch");

namespace {

thread_local char g_last_error[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// The device error word lives in this translation unit; kernels get its
// address as an argument.
__device__ int g_device_error;

using pkv::kMaxDevices;

struct DeviceState {
  bool ready = false;
  int sm_count = 0;
  int* err = nullptr;          // device address of g_device_error
  void* own_ws = nullptr;      // the NULL-workspace convenience buffer
  size_t own_ws_bytes = 0;
  size_t own_ws_cnt_bytes = 0; // counter bytes its last user needed zeroed
};

std::mutex g_mutex;
DeviceState g_devices[kMaxDevices];

// Per-device set-up with that device current: SM count and the address of
// the error word.  Returns nullptr (and sets the message) on failure.
DeviceState* device_state() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) {
    cuda_fail(e, "cudaGetDevice");
    return nullptr;
  }
  if (dev < 0 || dev >= kMaxDevices) {
    fail(PKV_ERR_UNSUPPORTED, "device ordinal %d beyond %d", dev, kMaxDevices);
    return nullptr;
  }
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceState& st = g_devices[dev];
  if (!st.ready) {
    e = cudaDeviceGetAttribute(&st.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) {
      cuda_fail(e, "cudaDeviceGetAttribute");
      return nullptr;
    }
    e = cudaGetSymbolAddress(reinterpret_cast<void**>(&st.err), g_device_error);
    if (e != cudaSuccess) {
      cuda_fail(e, "cudaGetSymbolAddress(error word)");
      return nullptr;
    }
    st.ready = true;
  }
  return &st;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int check_dims(const pkv_dims* d, bool for_attention) {
  if (d == nullptr) return fail(PKV_ERR_INVALID, "dims is NULL");
  if (d->head_dim != pkv::kHeadDim)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d unsupported (only 128)", d->head_dim);
  if (d->block_size != pkv::kBlockSize)
    return fail(PKV_ERR_UNSUPPORTED, "block_size %d unsupported (only 16)", d->block_size);
  if (d->num_kv_heads <= 0 || d->num_blocks < 0)
    return fail(PKV_ERR_INVALID, "num_kv_heads %d / num_blocks %d invalid", d->num_kv_heads,
                d->num_blocks);
  if ((long long)d->num_blocks * d->num_kv_heads * pkv::kBlockSize > (1ll << 40))
    return fail(PKV_ERR_INVALID, "pool too large");
  if (!for_attention) return PKV_OK;
  if (d->num_reqs < 0 || d->num_q_tokens < 0 || d->num_q_heads <= 0 ||
      d->max_blocks_per_req < 0)
    return fail(PKV_ERR_INVALID, "negative dims");
  if (d->num_q_heads % d->num_kv_heads != 0)
    return fail(PKV_ERR_INVALID, "num_q_heads %d not a multiple of num_kv_heads %d",
                d->num_q_heads, d->num_kv_heads);
  const int g = d->num_q_heads / d->num_kv_heads;
  if (g < 1 || g > 8) return fail(PKV_ERR_UNSUPPORTED, "group size %d unsupported (1..8)", g);
  if (d->num_reqs > pkv::kMaxReqs)
    return fail(PKV_ERR_UNSUPPORTED, "num_reqs %d beyond %d", d->num_reqs, pkv::kMaxReqs);
  if ((long long)d->max_blocks_per_req * pkv::kBlockSize > (1ll << 30))
    return fail(PKV_ERR_UNSUPPORTED, "max_blocks_per_req too large");
  return PKV_OK;
}

// The sizes that a step's tables and lengths are read with (the calls that
// take them without a group size).
int check_step_dims(const pkv_dims* d) {
  if (d == nullptr) return fail(PKV_ERR_INVALID, "dims is NULL");
  if (d->block_size != pkv::kBlockSize)
    return fail(PKV_ERR_UNSUPPORTED, "block_size %d unsupported (only 16)", d->block_size);
  if (d->num_reqs < 0 || d->num_q_tokens < 0 || d->num_blocks < 0 || d->max_blocks_per_req < 0)
    return fail(PKV_ERR_INVALID, "negative dims");
  if (d->num_reqs > pkv::kMaxReqs)
    return fail(PKV_ERR_UNSUPPORTED, "num_reqs %d beyond %d", d->num_reqs, pkv::kMaxReqs);
  if (d->num_q_tokens > (1 << 30))
    return fail(PKV_ERR_UNSUPPORTED, "num_q_tokens %d beyond 2^30", d->num_q_tokens);
  if ((long long)d->max_blocks_per_req * pkv::kBlockSize > (1ll << 30))
    return fail(PKV_ERR_UNSUPPORTED, "max_blocks_per_req too large");
  return PKV_OK;
}

constexpr int kPartsPerSm = 1;

pkv::WorkspaceLayout layout_for(const pkv_dims* d, int sm_count) {
  return pkv::decode_workspace_layout(d->num_q_tokens, d->num_kv_heads,
                                      d->num_q_heads / d->num_kv_heads, sm_count);
}

// Fewer rows than requests: some sit the step out (pkv_build_step makes such
// steps), and the rows may all be one chunk's.  The block-scaled attention
// launches its prefill for that from 512 rows times KV heads on: without it a
// 512-token chunk on 2000 keys takes 229 us for 34 at eight KV heads and 70 for
// 31 at two, 64 tokens on 4000 keys 75 for 29 at eight; a step that holds no
// chunk pays 5.6 us for the launch (100 decodes of 500 keys, eight KV heads: 27
// for 21; 500 of them 96 for 85).  Below, a chunk loses little or nothing (64
// tokens on 4000 keys at two KV heads 26 for 28, 40 on 1000 11 for 20).
bool idle_chunk(const pkv_dims* d) {
  return d->num_q_tokens < d->num_reqs && (long long)d->num_q_tokens * d->num_kv_heads >= 512;
}

// Partial states of the block-scaled prefill's split items, behind the rest of
// the workspace: for steps that may hold a chunk, one part per SM.
struct PartsLayout {
  size_t ml, o, total;
  int parts;
};

PartsLayout parts_layout(const pkv::WorkspaceLayout& w, const pkv_dims* d, int sm_count) {
  PartsLayout l;
  l.parts = d->num_q_tokens > d->num_reqs || idle_chunk(d) ? kPartsPerSm * sm_count : 0;
  const size_t rows = (size_t)l.parts * pkv::kPrefillRows;
  l.ml = (w.total + 255) & ~(size_t)255;
  l.o = l.ml + rows * sizeof(float2);
  l.total = l.parts ? l.o + rows * pkv::kHeadDim * sizeof(float) : w.total;
  return l;
}

// ----------------------------------------------------------------- options
// Process-wide launch and routing options: built-in defaults, overridden once
// by the environment when first needed, then only by pkv_set_options.  Every
// call works from one copy taken when it starts.
int env_int(const char* name, int dflt) {
  const char* v = getenv(name);
  return (v && *v) ? atoi(v) : dflt;
}

bool options_valid(const pkv_options& o) {
  return o.prefill_min_q >= 0 && o.align_slack >= 0 && o.min_chunk >= 1 && o.decode_grid >= 0 &&
         o.wait_limit_us >= 1 && o.rowgroup_cost >= 0 &&
         o.rowgroup_cost <= 1024;
}

pkv_options options_from_env() {
  pkv_options o{};
  o.pdl = env_int("PKV_PDL", 1);
  o.early_plan = env_int("PKV_EARLY_PLAN", 1);
  o.early_kv = env_int("PKV_EARLY_KV", 1);
  o.early_trigger = env_int("PKV_EARLY_TRIGGER", 0);
  o.plan_cache = env_int("PKV_PLAN_CACHE", 1);
  o.decode_tc = env_int("PKV_DECODE_TC", 1);
  o.decode_tc_fp8 = env_int("PKV_DECODE_TC_FP8", 1);
  o.prefill_min_q = env_int("PKV_PREFILL_MIN_Q", 16);
  o.align = env_int("PKV_ALIGN", 1);
  o.align_slack = env_int("PKV_ALIGN_SLACK", 64);
  o.min_chunk = env_int("PKV_MIN_CHUNK", 4);
  o.decode_grid = env_int("PKV_DECODE_GRID", 0);
  o.wait_limit_us = env_int("PKV_WAIT_LIMIT_US", (int)(pkv::kDefaultWaitLimitNs / 1000));
  o.debug_withhold_q = 0;  // never from the environment
  o.rowgroup_cost = env_int("PKV_ROWGROUP_COST", 16);
  // Out-of-range values from the environment fall back to the defaults.
  if (o.prefill_min_q < 0) o.prefill_min_q = 16;
  if (o.align_slack < 0) o.align_slack = 64;
  if (o.min_chunk < 1) o.min_chunk = 4;
  if (o.decode_grid < 0) o.decode_grid = 0;
  if (o.wait_limit_us < 1) o.wait_limit_us = (int)(pkv::kDefaultWaitLimitNs / 1000);
  if (o.rowgroup_cost < 0 || o.rowgroup_cost > 1024) o.rowgroup_cost = 16;
  return o;
}

std::mutex g_opts_mutex;
bool g_opts_ready = false;
pkv_options g_opts;

pkv_options current_options() {
  std::lock_guard<std::mutex> lock(g_opts_mutex);
  if (!g_opts_ready) {
    g_opts = options_from_env();
    g_opts_ready = true;
  }
  return g_opts;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against libcuda).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// 2-D map of a pool as [num_blocks * Hkv * 16 rows][128] bf16, 64 x 16 boxes.
// e4m3 pools: the same view in bytes, boxes of 16 rows x 128 codes.
int encode_pool_map_e4m3(CUtensorMap* m, const void* pool, const pkv_dims* d) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[2] = {(cuuint64_t)pkv::kHeadDim,
                              (cuuint64_t)d->num_blocks * d->num_kv_heads * pkv::kBlockSize};
  const cuuint64_t strides[1] = {(cuuint64_t)pkv::kHeadDim};
  const cuuint32_t box[2] = {(cuuint32_t)pkv::kHeadDim, (cuuint32_t)pkv::kBlockSize};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "encode e4m3 pool tensor map: CUresult %d", (int)r);
  return PKV_OK;
}

int encode_pool_map(CUtensorMap* m, const void* pool, const pkv_dims* d) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[2] = {(cuuint64_t)pkv::kHeadDim,
                              (cuuint64_t)d->num_blocks * d->num_kv_heads * pkv::kBlockSize};
  const cuuint64_t strides[1] = {(cuuint64_t)pkv::kHeadDim * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)pkv::kBlockSize};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "encode pool tensor map: CUresult %d", (int)r);
  return PKV_OK;
}

// 3-D map of q as [Tq][Hq][128] bf16, boxes of (64 dims, g heads, `tokens` tokens).
int encode_q_map(CUtensorMap* m, const void* q, const pkv_dims* d, int group, int tokens) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[3] = {(cuuint64_t)pkv::kHeadDim, (cuuint64_t)d->num_q_heads,
                              (cuuint64_t)d->num_q_tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)pkv::kHeadDim * 2,
                                 (cuuint64_t)d->num_q_heads * pkv::kHeadDim * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "encode q tensor map: CUresult %d", (int)r);
  return PKV_OK;
}

// ---------------------------------------------------- the latent cache's calls
constexpr int kMaxRopeHeads = 4096;

bool eps_ok(float eps) { return eps >= 0x1p-64f && eps <= 1.f; }

// Whether tokens of `row` elements, `stride` apart, share elements with others: their
// ranges may meet and they still lie side by side, in the rows of one tensor.
bool tokens_meet(const void* a, int64_t a_stride, __int128 a_row, const void* b, int64_t b_stride, __int128 b_row,
                 int tokens) {
  if (a_row == 0 || b_row == 0) return false;
  const __int128 x = (__int128)reinterpret_cast<uintptr_t>(a), y = (__int128)reinterpret_cast<uintptr_t>(b);
  const __int128 x1 = x + 2 * ((__int128)(tokens - 1) * a_stride + a_row);
  const __int128 y1 = y + 2 * ((__int128)(tokens - 1) * b_stride + b_row);
  if (x1 <= y || y1 <= x) return false;
  if (a_stride != b_stride || tokens < 2) return true;
  const __int128 pitch = 2 * (__int128)a_stride;
  __int128 gap = (y - x) % pitch;
  if (gap < 0) gap += pitch;
  return gap < 2 * a_row || gap + 2 * b_row > pitch;
}

// A token stride in elements: rows 16-byte aligned, a token inside one (any for a single token).
bool stride_ok(int64_t stride, int row, int tokens) {
  return stride >= 0 && stride % 8 == 0 && (stride >= row || tokens <= 1);
}

// Rows of 64 bf16 of every (token, head).
struct Rows {
  const void* base;
  int64_t token, head;  // elements between tokens, and heads
  static constexpr int kDims = pkv::kRopeDim;

  __int128 last(int tokens, int heads) const {  // elements from the first row's start to the end
    return (__int128)(tokens - 1) * token + (__int128)(heads - 1) * head + kDims;
  }
  // Heads side by side within tokens that lie apart, or the other way round.
  bool apart(int tokens, int heads) const {
    const bool h = heads == 1 || head >= kDims, t = tokens == 1 || token >= kDims;
    return (h && (tokens == 1 || token >= last(1, heads))) || (t && (heads == 1 || head >= last(tokens, 1)));
  }
  bool same(const Rows& o, int tokens, int heads) const {
    return base == o.base && (tokens == 1 || token == o.token) && (heads == 1 || head == o.head);
  }
  bool meets(const Rows& o, int tokens, int heads) const {
    const __int128 a = (__int128)reinterpret_cast<uintptr_t>(base), b = (__int128)reinterpret_cast<uintptr_t>(o.base);
    return a < b + 2 * o.last(tokens, heads) && b < a + 2 * last(tokens, heads);
  }
  // Whether they share elements with rows of `row` elements, one a token: with heads
  // within tokens the two may lie side by side, else only ranges that do not meet do.
  bool meets_tokens(const void* o, int64_t stride, int row, int tokens, int heads) const {
    const __int128 span = last(1, heads);
    if (tokens == 1 || token >= span) return tokens_meet(base, token, span, o, stride, row, tokens);
    return tokens_meet(base, 0, last(tokens, heads), o, 0, (__int128)(tokens - 1) * stride + row, 1);
  }
};

int check_latent_dims(const pkv_dims* d, bool attention) {
  if (d == nullptr) return fail(PKV_ERR_INVALID, "dims is NULL");
  if (d->head_dim != pkv::kLatRow)
    return fail(PKV_ERR_UNSUPPORTED, "head_dim %d unsupported (a latent row has 576)", d->head_dim);
  if (d->num_kv_heads != 1)
    return fail(PKV_ERR_UNSUPPORTED, "num_kv_heads %d unsupported (a latent cache has 1)", d->num_kv_heads);
  const int rc = check_step_dims(d);
  if (rc != PKV_OK) return rc;
  // (tensor-map rows are addressed with 32-bit coordinates)
  if ((long long)d->num_blocks * pkv::kBlockSize > 0x7fffffffll)
    return fail(PKV_ERR_UNSUPPORTED, "pool beyond 2^31 - 1 rows");
  if (d->num_q_heads < (attention ? 1 : 0)) return fail(PKV_ERR_INVALID, "num_q_heads is %d", d->num_q_heads);
  const int most = attention ? pkv::kMaxLatentHeads : kMaxRopeHeads;
  if (d->num_q_heads > most)
    return fail(PKV_ERR_UNSUPPORTED, "num_q_heads %d unsupported (up to %d)", d->num_q_heads, most);
  return PKV_OK;
}

// (times log2(e) it must still be a number)
bool latent_scale_ok(float scale) { return scale > 0.f && scale <= 0x1p127f; }

// How a step's (token, head) rows are grouped into work items of at most 64.  With no
// more rows than request slots an item is one token's heads: as a rule every request
// has one row then, and items of more would have columns that nobody uses.  Beyond
// that, an item has no more tokens than a request can have if each has one.  (Slots that
// sit the step out are not known here, and count as if they had a row: four drafts of 4
// on 2000 keys, 16 heads 20 us in 64 slots for 19 in 4; a chunk of 60 on 2000 keys,
// which reads its keys token by token then, 66 for 28.)
struct LatentGroups {
  int head_groups, group_heads, group_tokens;
};

LatentGroups latent_groups(const pkv_dims* d) {
  LatentGroups l;
  l.head_groups = d->num_q_heads > pkv::kLatMaxRows ? 2 : 1;
  l.group_heads = (d->num_q_heads + l.head_groups - 1) / l.head_groups;
  const int most = d->num_q_tokens - d->num_reqs + 1;
  l.group_tokens = pkv::kLatMaxRows / l.group_heads;
  if (l.group_tokens > most) l.group_tokens = most < 1 ? 1 : most;
  return l;
}

// The workspace: the prefill's work queue (zero between calls) and, from byte 128
// on, its count of pieces; then records, statistics and outputs of the pieces of
// rows that are cut, written anew by every call.  The prefill's statistics and
// outputs (twice 128 x 130 numbers an SM) take the room of the decode's outputs.
struct LatentLayout {
  size_t piece, ml, o, total;
};

LatentLayout latent_layout(int sm_count) {
  const size_t slots = 2 * (size_t)sm_count;
  LatentLayout l;
  l.piece = 256;
  l.ml = (l.piece + slots * pkv::kPieceWords * sizeof(int) + 255) & ~(size_t)255;
  l.o = l.ml + slots * pkv::kLatMaxRows * 2 * sizeof(float);
  l.total = l.o + slots * pkv::kLatMaxRows * pkv::kLatent * sizeof(float);
  return l;
}

// 3-D map of a bf16 tensor [n2][n1][n0] with strides s2, s1 (elements), 128-byte swizzle.
int encode_bf16_3d(CUtensorMap* m, const void* base, long long n0, long long n1, long long n2,
                   long long s1, long long s2, const cuuint32_t* box, const char* what) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[3] = {(cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
  const cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "encode %s tensor map: CUresult %d", what, (int)r);
  return PKV_OK;
}

// 2-D map of a latent pool as [num_blocks * 16 rows][576] bf16, 64 x 16 boxes.
int encode_latent_map(CUtensorMap* m, const void* pool, const pkv_dims* d) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  const cuuint64_t dims[2] = {(cuuint64_t)pkv::kLatRow, (cuuint64_t)d->num_blocks * pkv::kBlockSize};
  const cuuint64_t strides[1] = {(cuuint64_t)pkv::kLatRow * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)pkv::kBlockSize};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "encode latent pool tensor map: CUresult %d", (int)r);
  return PKV_OK;
}

}  // namespace

namespace pkv {
void set_error_message(const char* msg) { snprintf(g_last_error, sizeof g_last_error, "%s", msg); }

int attention_workspace_bytes(const pkv_dims* dims, size_t* bytes) {
  *bytes = 0;
  const int rc = check_dims(dims, true);
  if (rc != PKV_OK) return rc;
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  *bytes = layout_for(dims, st->sm_count).total;
  return PKV_OK;
}
}  // namespace pkv

namespace {

int append_impl(const void* k_new, const void* v_new, const int64_t* slot_mapping, void* k_pool,
                void* v_pool, int32_t num_new_tokens, const pkv_dims* dims, cudaStream_t stream,
                bool early_trigger) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, false);
  if (rc != PKV_OK) return rc;
  if (num_new_tokens < 0) return fail(PKV_ERR_INVALID, "num_new_tokens < 0");
  if (num_new_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !slot_mapping || !k_pool || !v_pool)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool))
    return fail(PKV_ERR_INVALID, "bf16 buffers must be 16-byte aligned");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::AppendParams p{};
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.slot_mapping = slot_mapping;
  p.k_pool = static_cast<__nv_bfloat16*>(k_pool);
  p.v_pool = static_cast<__nv_bfloat16*>(v_pool);
  p.err = st->err;
  p.num_tokens = num_new_tokens;
  p.num_kv_heads = dims->num_kv_heads;
  p.num_blocks = dims->num_blocks;
  p.pdl = current_options().pdl != 0;
  p.early_trigger = early_trigger && p.pdl;
  cudaError_t e = pkv::launch_append(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "append launch");
  return PKV_OK;
}

int append_fp8_impl(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                    void* k_pool, void* v_pool, const float* k_scale, const float* v_scale,
                    int32_t num_new_tokens, const pkv_dims* dims, cudaStream_t stream,
                    bool early_trigger) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, false);
  if (rc != PKV_OK) return rc;
  if (num_new_tokens < 0) return fail(PKV_ERR_INVALID, "num_new_tokens < 0");
  if (num_new_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !slot_mapping || !k_pool || !v_pool || !k_scale || !v_scale)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool))
    return fail(PKV_ERR_INVALID, "k/v buffers and pools must be 16-byte aligned");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::AppendFp8Params p{};
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.slot_mapping = slot_mapping;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err = st->err;
  p.num_tokens = num_new_tokens;
  p.num_kv_heads = dims->num_kv_heads;
  p.num_blocks = dims->num_blocks;
  p.pdl = current_options().pdl != 0;
  p.early_trigger = early_trigger && p.pdl;
  cudaError_t e = pkv::launch_append_fp8(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "append_fp8 launch");
  return PKV_OK;
}

}  // namespace

extern "C" {

const char* pkv_last_error(void) { return g_last_error; }

int pkv_append(const void* k_new, const void* v_new, const int64_t* slot_mapping, void* k_pool,
               void* v_pool, int32_t num_new_tokens, const pkv_dims* dims, cudaStream_t stream) {
  return append_impl(k_new, v_new, slot_mapping, k_pool, v_pool, num_new_tokens, dims, stream,
                     false);
}

int pkv_append_fp8(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                   void* k_pool, void* v_pool, const float* k_scale, const float* v_scale,
                   int32_t num_new_tokens, const pkv_dims* dims, cudaStream_t stream) {
  return append_fp8_impl(k_new, v_new, slot_mapping, k_pool, v_pool, k_scale, v_scale,
                         num_new_tokens, dims, stream, false);
}

int pkv_copy_blocks(const void* k_src, const void* v_src, void* k_dst, void* v_dst,
                    const int64_t* pairs, int32_t num_pairs, int32_t src_num_blocks,
                    int32_t dst_num_blocks, const pkv_dims* dims, cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, false);
  if (rc != PKV_OK) return rc;
  if (num_pairs < 0 || src_num_blocks < 0 || dst_num_blocks < 0)
    return fail(PKV_ERR_INVALID, "negative count");
  if (num_pairs == 0) return PKV_OK;
  if (!k_src || !v_src || !k_dst || !v_dst || !pairs)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(k_src) || !aligned16(v_src) || !aligned16(k_dst) || !aligned16(v_dst))
    return fail(PKV_ERR_INVALID, "pools must be 16-byte aligned");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::CopyParams p{};
  p.k_src = static_cast<const __nv_bfloat16*>(k_src);
  p.v_src = static_cast<const __nv_bfloat16*>(v_src);
  p.k_dst = static_cast<__nv_bfloat16*>(k_dst);
  p.v_dst = static_cast<__nv_bfloat16*>(v_dst);
  p.pairs = pairs;
  p.err = st->err;
  p.num_pairs = num_pairs;
  p.num_kv_heads = dims->num_kv_heads;
  p.src_blocks = src_num_blocks;
  p.dst_blocks = dst_num_blocks;
  p.pdl = current_options().pdl != 0;
  cudaError_t e = pkv::launch_copy_blocks(p, st->sm_count, stream);
  if (e != cudaSuccess) return cuda_fail(e, "copy_blocks launch");
  return PKV_OK;
}

size_t pkv_attention_workspace_size(const pkv_dims* dims) {
  if (check_dims(dims, true) != PKV_OK) return 0;
  DeviceState* st = device_state();
  if (!st) return 0;
  return parts_layout(layout_for(dims, st->sm_count), dims, st->sm_count).total;
}

int pkv_workspace_init(void* workspace, size_t workspace_bytes, const pkv_dims* dims,
                       cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, true);
  if (rc != PKV_OK) return rc;
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  const pkv::WorkspaceLayout w = layout_for(dims, st->sm_count);
  if (workspace == nullptr || workspace_bytes < w.total)
    return fail(PKV_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, w.total);
  cudaError_t e = cudaMemsetAsync(workspace, 0, w.ml_off, stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(workspace counters)");
  return PKV_OK;
}

}  // extern "C"

namespace {

// Sharing groups of a cascade call (device arrays).
struct CascadeArgs {
  const int32_t* grp_first;
  const int32_t* grp_count;
  const int32_t* grp_blocks;
  int num_groups;
};

// Regions a cascade call adds after the attention workspace.
struct CascadeLayout {
  size_t pre_o, pre_ml, first_block, total;
};

CascadeLayout cascade_layout(const pkv::WorkspaceLayout& w, const pkv_dims* d) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t rows = (size_t)pkv::kPrefixSplits * d->num_q_tokens * d->num_q_heads;
  CascadeLayout c;
  c.pre_o = up(w.total);
  c.pre_ml = c.pre_o + up(rows * pkv::kHeadDim * sizeof(float));
  c.first_block = c.pre_ml + up(rows * 2 * sizeof(float));
  c.total = c.first_block + up((size_t)d->num_reqs * sizeof(int32_t));
  return c;
}

// The attention entry points: bf16 pools (k_scale == nullptr) or e4m3 pools
// (scales per KV head, or with block_scales per block and KV head),
// optionally with shared-prefix groups.
int attention_impl(const void* q, const void* k_pool, const void* v_pool, const float* k_scale,
                   const float* v_scale, const int32_t* block_tables, const int32_t* seq_lens,
                   const int32_t* query_start_loc, float scale, void* out, const pkv_dims* dims,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream,
                   const CascadeArgs* cas = nullptr, bool after_append = false,
                   bool append_triggered_early = false, bool block_scales = false) {
  g_last_error[0] = '\0';
  const bool fp8 = k_scale != nullptr;
  int rc = check_dims(dims, true);
  if (rc != PKV_OK) return rc;
  if (dims->num_reqs == 0 || dims->num_q_tokens == 0) return PKV_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !seq_lens || !query_start_loc || !out)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return fail(PKV_ERR_INVALID, "q, out and the pools must be 16-byte aligned");
  if (!(scale == scale) || scale == 0.f) return fail(PKV_ERR_INVALID, "scale must be finite, non-zero");
  if (cas) {
    if (cas->num_groups < 0) return fail(PKV_ERR_INVALID, "num_groups < 0");
    if (cas->num_groups > 0 && (!cas->grp_first || !cas->grp_count || !cas->grp_blocks))
      return fail(PKV_ERR_INVALID, "NULL group array");
  }
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  const pkv::WorkspaceLayout w = layout_for(dims, st->sm_count);
  const CascadeLayout cl = cascade_layout(w, dims);
  if (cas) {
    if (workspace == nullptr || workspace_bytes < cl.total)
      return fail(PKV_ERR_WORKSPACE, "cascade workspace %zu bytes, need %zu (caller-owned)",
                  workspace_bytes, cl.total);
  }
  const PartsLayout parts = parts_layout(w, dims, st->sm_count);
  const size_t full = block_scales ? parts.total : w.total;
  if (workspace == nullptr) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (st->own_ws_bytes < full) {
      if (st->own_ws) cudaFree(st->own_ws);
      st->own_ws = nullptr;
      st->own_ws_bytes = 0;
      cudaError_t e = cudaMalloc(&st->own_ws, full);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMalloc(workspace)");
      e = cudaMemset(st->own_ws, 0, full);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMemset(workspace)");
      st->own_ws_bytes = full;
      st->own_ws_cnt_bytes = w.ml_off;
    } else if (st->own_ws_cnt_bytes != w.ml_off) {
      // The counter region moved with the dims: zero it again.
      cudaError_t e = cudaMemsetAsync(st->own_ws, 0, w.ml_off, stream);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(workspace)");
      st->own_ws_cnt_bytes = w.ml_off;
    }
    workspace = st->own_ws;
    workspace_bytes = st->own_ws_bytes;
  }
  if (workspace_bytes < w.total)
    return fail(PKV_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, w.total);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PKV_ERR_INVALID, "workspace must be 256-byte aligned");

  const pkv_options opt = current_options();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pkv::DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.kv_fp8 = fp8 ? 1 : 0;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.ws_cnt = reinterpret_cast<int*>(ws + w.cnt_off);
  p.plan_cache = opt.plan_cache != 0 && dims->num_reqs <= pkv::kPlanCacheReqs
                     ? reinterpret_cast<int*>(ws + w.plan_off)
                     : nullptr;
  p.plan_entries = w.plan_entries;
  p.ws_ml = reinterpret_cast<float*>(ws + w.ml_off);
  p.ws_o = reinterpret_cast<float*>(ws + w.o_off);
  p.err = st->err;
  p.num_reqs = dims->num_reqs;
  p.num_q_tokens = dims->num_q_tokens;
  p.num_q_heads = dims->num_q_heads;
  p.num_kv_heads = dims->num_kv_heads;
  p.num_blocks = dims->num_blocks;
  p.max_blocks = dims->max_blocks_per_req;
  p.scale_log2 = scale * 1.4426950408889634f;
  // Requests with at least this many query tokens go to the tensor-core
  // prefill kernel (when the step has that many query tokens at all).
  int prefill_min_q = opt.prefill_min_q;
  if (prefill_min_q < 1) prefill_min_q = 0x7fffffff;
  // Over block scales the decode reads a request's keys once per query token
  // and the prefill splits long items, so it takes over at half as many (64
  // requests of 9 tokens, 500-1000 keys, eight KV heads: 55 us for 132; below,
  // little is left to gain: 8 of 4, 4000 keys, eight KV heads: 40 for 41, four:
  // 28 for 27; 30 of 5, 100-4000 keys, three KV heads: 32 for 34).
  else if (block_scales) prefill_min_q = prefill_min_q / 2 + prefill_min_q % 2;
  // Launch it only when the step can hold such a request next to one query
  // for every other request; otherwise the decode kernel serves every row
  // (it is correct for any q_r, the prefill kernel is only faster).
  // e4m3 pools with scales per head: every row runs in the decode kernel.
  const long long others = block_scales && idle_chunk(dims) ? 0 : dims->num_reqs - 1;
  const bool run_prefill =
      (!fp8 || block_scales) && dims->num_q_tokens - others >= (long long)prefill_min_q;
  p.prefill_min_q = run_prefill ? prefill_min_q : 0x7fffffff;
  p.num_slots = w.num_slots;
  p.pdl = opt.pdl != 0;
  p.min_chunk = opt.min_chunk;
  p.align = opt.align != 0;
  p.align_slack = opt.align_slack;
  p.early_plan = p.pdl && opt.early_plan != 0;
  p.wait_limit_ns = (unsigned long long)opt.wait_limit_us * 1000ull;
  p.debug_withhold_q = opt.debug_withhold_q != 0;
  p.rowgroup_cost = opt.rowgroup_cost;
  const int group = dims->num_q_heads / dims->num_kv_heads;
  int grid = pkv::decode_grid(st->sm_count, group);
  // tuning override, bounded by the workspace's slots
  if (opt.decode_grid > 0 && 2 * opt.decode_grid <= w.num_slots) grid = opt.decode_grid;
  // Groups of 4 or more query heads per KV head make the decode's FP32 FMA
  // work comparable to its HBM time; those run on the tensor cores, e4m3
  // pools included (their tiles widened to f16 in shared memory by two
  // converter warps; decode_tc_fp8 = 0 keeps them on the SIMT decode).
  const bool use_tc = group >= 4 && opt.decode_tc != 0 && (!fp8 || opt.decode_tc_fp8 != 0);
  cudaError_t e;
  // Shared prefixes are read once by the prefix pass when the tensor-core
  // decode serves the step; otherwise every row reads its whole context (the
  // same result, without the sharing).
  const bool cascade = cas && cas->num_groups > 0 && use_tc;
  if (cascade) {
    int32_t* first_block = reinterpret_cast<int32_t*>(ws + cl.first_block);
    e = cudaMemsetAsync(first_block, 0, (size_t)dims->num_reqs * sizeof(int32_t), stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(first blocks)");
    pkv::CascadePrepParams cp{};
    cp.grp_first = cas->grp_first;
    cp.grp_count = cas->grp_count;
    cp.grp_blocks = cas->grp_blocks;
    cp.first_block = first_block;
    cp.err = st->err;
    cp.num_groups = cas->num_groups;
    cp.num_reqs = dims->num_reqs;
    cp.max_blocks = dims->max_blocks_per_req;
    cp.pdl = p.pdl;
    e = pkv::launch_cascade_prep(cp, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cascade set-up launch");
    // Prefix pass: every member's rows against the group's shared blocks.
    pkv::PrefillLaunch L{};
    rc = encode_q_map(&L.qmap, q, dims, group, pkv::prefill_tokens_per_tile(group));
    if (rc == PKV_OK) rc = encode_pool_map(&L.kmap, k_pool, dims);
    if (rc == PKV_OK) rc = encode_pool_map(&L.vmap, v_pool, dims);
    if (rc != PKV_OK) return rc;
    L.p.block_tables = block_tables;
    L.p.seq_lens = seq_lens;
    L.p.qsl = query_start_loc;
    L.p.out = p.out;
    L.p.err = st->err;
    L.p.num_reqs = dims->num_reqs;
    L.p.num_q_tokens = dims->num_q_tokens;
    L.p.num_q_heads = dims->num_q_heads;
    L.p.num_kv_heads = dims->num_kv_heads;
    L.p.num_blocks = dims->num_blocks;
    L.p.max_blocks = dims->max_blocks_per_req;
    L.p.scale_log2 = p.scale_log2;
    L.p.prefill_min_q = 1;
    L.p.pdl = p.pdl;
    L.p.prefix_mode = 1;
    L.p.grp_first = cas->grp_first;
    L.p.grp_count = cas->grp_count;
    L.p.grp_blocks = cas->grp_blocks;
    L.p.num_groups = cas->num_groups;
    L.p.pre_o = reinterpret_cast<float*>(ws + cl.pre_o);
    L.p.pre_ml = reinterpret_cast<float*>(ws + cl.pre_ml);
    L.p.sched = reinterpret_cast<unsigned long long*>(ws + w.sched_off);
    L.p.wait_limit_ns = p.wait_limit_ns;
    L.grid = st->sm_count;
    e = pkv::launch_prefill(L, group, stream);
    if (e != cudaSuccess) return cuda_fail(e, "prefix pass launch");
    // Decode of every row from its first unshared block, merging the prefix.
    p.first_block = first_block;
    p.pre_o = L.p.pre_o;
    p.pre_ml = L.p.pre_ml;
    p.prefill_min_q = 0x7fffffff;
    p.early_plan = 0;  // first_block comes from the set-up kernel, two launches back
  }
  // Right after the append of this step's tokens (pkv_append_attention), the
  // decode kernel streams every tile without a new token before waiting.
  p.early_kv = after_append && !cascade && p.pdl;
  p.early_q = !append_triggered_early;
  const bool do_prefill = run_prefill && !cascade;
  // Long steps run two decode CTAs per SM; steps with at most 8 tiles (64
  // blocks) per SM run on one, so that the next launch's CTAs can prepare
  // beside them.  When the dims alone bound the work that low (every decode
  // row reads at most max_blocks_per_req blocks per KV head) the grid is one
  // CTA per SM; otherwise the plan makes the choice on the device from the
  // lengths.
  constexpr long long kHalfGridBlocks = 64;
  const long long bound = (long long)dims->num_q_tokens * dims->max_blocks_per_req * dims->num_kv_heads;
  const bool small = bound <= kHalfGridBlocks * st->sm_count;
  const int tc_grid = small ? st->sm_count : 2 * st->sm_count;
  // tuning override, bounded by the workspace's slots
  const bool grid_forced = opt.decode_grid > 0 && 2 * opt.decode_grid <= w.num_slots;
  const int half_grid_blocks = small || grid_forced ? 0 : (int)kHalfGridBlocks;
  if (block_scales) {
    pkv::DecodeBlockLaunch B{};
    rc = encode_pool_map_e4m3(&B.kmap, k_pool, dims);
    if (rc == PKV_OK) rc = encode_pool_map_e4m3(&B.vmap, v_pool, dims);
    if (rc != PKV_OK) return rc;
    // The prefill first: the decode's CTAs fill the SMs that have no work item
    // of it, or have finished theirs.
    if (do_prefill) {
      pkv::PrefillBlockLaunch L{};
      rc = encode_q_map(&L.qmap, q, dims, group, pkv::prefill_tokens_per_tile(group));
      if (rc != PKV_OK) return rc;
      L.kmap = B.kmap;
      L.vmap = B.vmap;
      L.p.k_scales = k_scale;
      L.p.v_scales = v_scale;
      L.p.early_plan = p.early_plan;
      // No splitting when the step's rows, if they are all in use, are more
      // items than two thirds of the parts (each request has at most
      // prefill_min_q - 1 tokens that are no chunk's) -- little is left to cut
      // with then, and the kernel without it is 3% faster -- or the workspace
      // has no room for the parts.
      const long long chunk_rows = dims->num_q_tokens - (prefill_min_q - 1ll) * dims->num_reqs;
      const long long items = chunk_rows / pkv::prefill_tokens_per_tile(group) * dims->num_kv_heads;
      L.p.max_parts = 3 * items <= 2 * parts.parts && workspace_bytes >= parts.total ? parts.parts : 0;
      L.p.part_ml = reinterpret_cast<float2*>(ws + parts.ml);
      L.p.part_o = reinterpret_cast<float4*>(ws + parts.o);
      L.p.cnt = p.ws_cnt;
      pkv::PrefillParams& f = L.p.p;
      f.block_tables = block_tables;
      f.seq_lens = seq_lens;
      f.qsl = query_start_loc;
      f.out = p.out;
      f.err = st->err;
      f.num_reqs = dims->num_reqs;
      f.num_q_tokens = dims->num_q_tokens;
      f.num_q_heads = dims->num_q_heads;
      f.num_kv_heads = dims->num_kv_heads;
      f.num_blocks = dims->num_blocks;
      f.max_blocks = dims->max_blocks_per_req;
      f.scale_log2 = p.scale_log2;
      f.prefill_min_q = prefill_min_q;
      f.pdl = p.pdl;
      f.sched = reinterpret_cast<unsigned long long*>(ws + w.sched_off);
      f.wait_limit_ns = p.wait_limit_ns;
      L.grid = st->sm_count;
      e = pkv::launch_prefill_block(L, group, stream);
      if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
    }
    B.p = p;
    // More row-groups than SMs: two CTAs per SM however short they are, one
    // per row-group (plan_cta; 303 row-groups of one tile: 12.0 vs 16.6 us).
    const bool one_each = small && (long long)dims->num_q_tokens * dims->num_kv_heads <= st->sm_count;
    B.grid = grid_forced ? opt.decode_grid : one_each ? st->sm_count : 2 * st->sm_count;
    B.p.half_grid_blocks = one_each || grid_forced ? 0 : (int)kHalfGridBlocks;
    B.after_prefill = do_prefill;
    e = pkv::launch_decode_block(B, group, stream);
  } else if (use_tc) {
    pkv::DecodeTcLaunch T{};
    rc = encode_q_map(&T.qmap, q, dims, group, 1);
    if (rc == PKV_OK) rc = fp8 ? encode_pool_map_e4m3(&T.kmap, k_pool, dims)
                               : encode_pool_map(&T.kmap, k_pool, dims);
    if (rc == PKV_OK) rc = fp8 ? encode_pool_map_e4m3(&T.vmap, v_pool, dims)
                               : encode_pool_map(&T.vmap, v_pool, dims);
    if (rc != PKV_OK) return rc;
    T.p = p;
    T.grid = grid_forced ? opt.decode_grid : tc_grid;
    T.p.half_grid_blocks = half_grid_blocks;
    e = pkv::launch_decode_tc(T, group, stream);
  } else {
    e = pkv::launch_decode(p, group, grid, stream);
  }
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  if (do_prefill && !block_scales) {
    pkv::PrefillLaunch L{};
    rc = encode_q_map(&L.qmap, q, dims, group, pkv::prefill_tokens_per_tile(group));
    if (rc == PKV_OK) rc = encode_pool_map(&L.kmap, k_pool, dims);
    if (rc == PKV_OK) rc = encode_pool_map(&L.vmap, v_pool, dims);
    if (rc != PKV_OK) return rc;
    L.p.block_tables = block_tables;
    L.p.seq_lens = seq_lens;
    L.p.qsl = query_start_loc;
    L.p.out = p.out;
    L.p.err = st->err;
    L.p.num_reqs = dims->num_reqs;
    L.p.num_q_tokens = dims->num_q_tokens;
    L.p.num_q_heads = dims->num_q_heads;
    L.p.num_kv_heads = dims->num_kv_heads;
    L.p.num_blocks = dims->num_blocks;
    L.p.max_blocks = dims->max_blocks_per_req;
    L.p.scale_log2 = p.scale_log2;
    L.p.prefill_min_q = prefill_min_q;
    L.p.pdl = p.pdl;
    L.p.sched = reinterpret_cast<unsigned long long*>(ws + w.sched_off);
    L.p.wait_limit_ns = p.wait_limit_ns;
    L.grid = st->sm_count;
    e = pkv::launch_prefill(L, group, stream);
    if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
  }
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_attention(const void* q, const void* k_pool, const void* v_pool,
                  const int32_t* block_tables, const int32_t* seq_lens,
                  const int32_t* query_start_loc, float scale, void* out, const pkv_dims* dims,
                  void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return attention_impl(q, k_pool, v_pool, nullptr, nullptr, block_tables, seq_lens,
                        query_start_loc, scale, out, dims, workspace, workspace_bytes, stream);
}

int pkv_append_attention(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                         void* k_pool, void* v_pool, const void* q, const int32_t* block_tables,
                         const int32_t* seq_lens, const int32_t* query_start_loc, float scale,
                         void* out, const pkv_dims* dims, void* workspace,
                         size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, true);
  if (rc != PKV_OK) return rc;
  // The attention kernel reads K/V tiles without this step's tokens (and the
  // lengths and tables) before it waits for the append.  PKV_EARLY_TRIGGER=1
  // also lets it launch as soon as the append starts, before the kernel
  // ahead of the append has finished; q, out and the workspace then wait.
  const pkv_options opt = current_options();
  const bool pdl = opt.pdl != 0;
  const bool early = pdl && opt.early_kv != 0;
  const bool trigger = early && opt.early_trigger != 0;
  rc = append_impl(k_new, v_new, slot_mapping, k_pool, v_pool, dims->num_q_tokens, dims, stream,
                   trigger);
  if (rc != PKV_OK) return rc;
  return attention_impl(q, k_pool, v_pool, nullptr, nullptr, block_tables, seq_lens,
                        query_start_loc, scale, out, dims, workspace, workspace_bytes, stream,
                        nullptr, early, trigger);
}

int pkv_append_attention_fp8(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                             void* k_pool, void* v_pool, const float* k_scale,
                             const float* v_scale, const void* q, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* query_start_loc,
                             float scale, void* out, const pkv_dims* dims, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, true);
  if (rc != PKV_OK) return rc;
  if (!k_scale || !v_scale) return fail(PKV_ERR_INVALID, "k_scale / v_scale is NULL");
  // As pkv_append_attention: tiles without this step's tokens are read
  // before the append finishes (early_kv), and with early_trigger the
  // attention launches as soon as the append starts.
  const pkv_options opt = current_options();
  const bool pdl = opt.pdl != 0;
  const bool early = pdl && opt.early_kv != 0;
  const bool trigger = early && opt.early_trigger != 0;
  rc = append_fp8_impl(k_new, v_new, slot_mapping, k_pool, v_pool, k_scale, v_scale,
                       dims->num_q_tokens, dims, stream, trigger);
  if (rc != PKV_OK) return rc;
  return attention_impl(q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                        query_start_loc, scale, out, dims, workspace, workspace_bytes, stream,
                        nullptr, early, trigger);
}

size_t pkv_cascade_workspace_size(const pkv_dims* dims) {
  if (check_dims(dims, true) != PKV_OK) return 0;
  DeviceState* st = device_state();
  if (!st) return 0;
  return cascade_layout(layout_for(dims, st->sm_count), dims).total;
}

int pkv_attention_cascade(const void* q, const void* k_pool, const void* v_pool,
                          const int32_t* block_tables, const int32_t* seq_lens,
                          const int32_t* query_start_loc, const int32_t* group_first_req,
                          const int32_t* group_num_reqs, const int32_t* group_prefix_blocks,
                          int32_t num_groups, float scale, void* out, const pkv_dims* dims,
                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const CascadeArgs cas{group_first_req, group_num_reqs, group_prefix_blocks, num_groups};
  return attention_impl(q, k_pool, v_pool, nullptr, nullptr, block_tables, seq_lens,
                        query_start_loc, scale, out, dims, workspace, workspace_bytes, stream,
                        &cas);
}

int pkv_attention_fp8kv(const void* q, const void* k_pool, const void* v_pool,
                        const float* k_scale, const float* v_scale, const int32_t* block_tables,
                        const int32_t* seq_lens, const int32_t* query_start_loc, float scale,
                        void* out, const pkv_dims* dims, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  if (!k_scale || !v_scale) {
    g_last_error[0] = '\0';
    return fail(PKV_ERR_INVALID, "k_scale / v_scale is NULL");
  }
  return attention_impl(q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                        query_start_loc, scale, out, dims, workspace, workspace_bytes, stream);
}

int pkv_append_fp8_block(const void* k_new, const void* v_new, const int32_t* block_tables,
                         const int32_t* seq_lens, const int32_t* query_start_loc, void* k_pool,
                         void* v_pool, float* k_scales, float* v_scales, const pkv_dims* dims,
                         cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, false);
  if (rc == PKV_OK) rc = check_step_dims(dims);
  if (rc != PKV_OK) return rc;
  if (dims->num_reqs == 0 || dims->num_q_tokens == 0) return PKV_OK;
  if (!k_new || !v_new || !block_tables || !seq_lens || !query_start_loc || !k_pool || !v_pool ||
      !k_scales || !v_scales)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool))
    return fail(PKV_ERR_INVALID, "k/v buffers and pools must be 16-byte aligned");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::AppendBlockParams p{};
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.query_start_loc = query_start_loc;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.err = st->err;
  p.num_reqs = dims->num_reqs;
  p.num_tokens = dims->num_q_tokens;
  p.num_kv_heads = dims->num_kv_heads;
  p.num_blocks = dims->num_blocks;
  p.max_blocks = dims->max_blocks_per_req;
  p.pdl = current_options().pdl != 0;
  const cudaError_t e = pkv::launch_append_fp8_block(p, stream);
  if (e != cudaSuccess) return cuda_fail(e, "append_fp8_block launch");
  return PKV_OK;
}

int pkv_attention_fp8_block(const void* q, const void* k_pool, const void* v_pool,
                            const float* k_scales, const float* v_scales,
                            const int32_t* block_tables, const int32_t* seq_lens,
                            const int32_t* query_start_loc, float scale, void* out,
                            const pkv_dims* dims, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  g_last_error[0] = '\0';
  if (!k_scales || !v_scales) return fail(PKV_ERR_INVALID, "k_scales / v_scales is NULL");
  const int rc = check_dims(dims, true);
  if (rc != PKV_OK) return rc;
  // (tensor-map rows are addressed with 32-bit coordinates)
  if ((long long)dims->num_blocks * dims->num_kv_heads * pkv::kBlockSize > 0x7fffffffll)
    return fail(PKV_ERR_UNSUPPORTED, "pool beyond 2^31 - 1 rows");
  return attention_impl(q, k_pool, v_pool, k_scales, v_scales, block_tables, seq_lens,
                        query_start_loc, scale, out, dims, workspace, workspace_bytes, stream,
                        nullptr, false, false, true);
}

int pkv_build_step(const int32_t* prev_lens, const int32_t* new_tokens, const int32_t* free_list,
                   const int32_t* num_free_in, int32_t* block_tables, int32_t* seq_lens,
                   int32_t* query_start_loc, int64_t* slot_mapping, int32_t* num_free_out,
                   int32_t* num_refused, const pkv_dims* dims, cudaStream_t stream) {
  g_last_error[0] = '\0';
  const int rc = check_step_dims(dims);
  if (rc != PKV_OK) return rc;
  // (arrays without an element may be NULL)
  if (!num_free_in || !query_start_loc || !num_free_out ||
      (!slot_mapping && dims->num_q_tokens > 0) || (!free_list && dims->num_blocks > 0) ||
      (dims->num_reqs > 0 && (!prev_lens || !new_tokens || !seq_lens)) ||
      (dims->num_reqs > 0 && dims->max_blocks_per_req > 0 && !block_tables))
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::StepParams p{};
  p.prev_lens = prev_lens;
  p.new_tokens = new_tokens;
  p.free_list = free_list;
  p.num_free_in = num_free_in;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.query_start_loc = query_start_loc;
  p.slot_mapping = slot_mapping;
  p.num_free_out = num_free_out;
  p.num_refused = num_refused;
  p.err = st->err;
  p.num_reqs = dims->num_reqs;
  p.num_q_tokens = dims->num_q_tokens;
  p.num_blocks = dims->num_blocks;
  p.max_blocks = dims->max_blocks_per_req;
  const cudaError_t e = pkv::launch_build_step(p, current_options().pdl != 0, stream);
  if (e != cudaSuccess) return cuda_fail(e, "build_step launch");
  return PKV_OK;
}

int pkv_release_blocks(const int32_t* block_tables, const int32_t* seq_lens,
                       const int32_t* keep_lens, int32_t* free_list, const int32_t* num_free_in,
                       int32_t* num_free_out, const pkv_dims* dims, cudaStream_t stream) {
  g_last_error[0] = '\0';
  const int rc = check_step_dims(dims);
  if (rc != PKV_OK) return rc;
  // (arrays without an element may be NULL)
  if (!num_free_in || !num_free_out || (!free_list && dims->num_blocks > 0) ||
      (dims->num_reqs > 0 && (!seq_lens || !keep_lens)) ||
      (dims->num_reqs > 0 && dims->max_blocks_per_req > 0 && !block_tables))
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::ReleaseParams p{};
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.keep_lens = keep_lens;
  p.free_list = free_list;
  p.num_free_in = num_free_in;
  p.num_free_out = num_free_out;
  p.err = st->err;
  p.num_reqs = dims->num_reqs;
  p.num_blocks = dims->num_blocks;
  p.max_blocks = dims->max_blocks_per_req;
  const cudaError_t e = pkv::launch_release_blocks(p, current_options().pdl != 0, stream);
  if (e != cudaSuccess) return cuda_fail(e, "release_blocks launch");
  return PKV_OK;
}

int pkv_norm_rope_append(const void* q, const void* k, const void* v, int64_t q_stride,
                         int64_t k_stride, int64_t v_stride, const int64_t* positions,
                         const float* cos_sin, int64_t max_position, int32_t rotary_dim,
                         int32_t interleaved, const void* q_weight, const void* k_weight, float eps,
                         const int64_t* slot_mapping, void* q_out, int64_t q_out_stride, void* k_pool,
                         void* v_pool, const pkv_dims* dims, cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_dims(dims, false);
  if (rc != PKV_OK) return rc;
  if (dims->num_q_tokens < 0 || dims->num_q_heads < 0) return fail(PKV_ERR_INVALID, "negative dims");
  if (dims->num_q_heads > kMaxRopeHeads || dims->num_kv_heads > kMaxRopeHeads)
    return fail(PKV_ERR_UNSUPPORTED, "more than %d heads", kMaxRopeHeads);
  if (rotary_dim < 16 || rotary_dim > pkv::kHeadDim || rotary_dim % 16 != 0)
    return fail(PKV_ERR_UNSUPPORTED, "rotary_dim %d unsupported (16, 32, .. 128)", rotary_dim);
  if ((q_weight || k_weight) && !eps_ok(eps)) return fail(PKV_ERR_INVALID, "eps must be in [2^-64, 1]");
  if (dims->num_q_tokens == 0) return PKV_OK;
  if (!k || !v || !positions || !cos_sin || !slot_mapping || !k_pool || !v_pool ||
      (dims->num_q_heads > 0 && (!q || !q_out)))
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_pool) ||
      !aligned16(v_pool) || !aligned16(cos_sin) || !aligned16(q_weight) || !aligned16(k_weight))
    return fail(PKV_ERR_INVALID, "buffers must be 16-byte aligned");
  if (!stride_ok(q_stride, dims->num_q_heads * pkv::kHeadDim, dims->num_q_tokens) ||
      !stride_ok(q_out_stride, dims->num_q_heads * pkv::kHeadDim, dims->num_q_tokens) ||
      !stride_ok(k_stride, dims->num_kv_heads * pkv::kHeadDim, dims->num_q_tokens) ||
      !stride_ok(v_stride, dims->num_kv_heads * pkv::kHeadDim, dims->num_q_tokens))
    return fail(PKV_ERR_INVALID, "token strides must be multiples of 8 elements and hold a token");
  const int tokens = dims->num_q_tokens;
  const int64_t q_row = (int64_t)dims->num_q_heads * pkv::kHeadDim, kv_row = (int64_t)dims->num_kv_heads * pkv::kHeadDim;
  if ((!(q == q_out && (q_stride == q_out_stride || tokens < 2)) &&
       tokens_meet(q_out, q_out_stride, q_row, q, q_stride, q_row, tokens)) ||
      tokens_meet(q_out, q_out_stride, q_row, k, k_stride, kv_row, tokens) ||
      tokens_meet(q_out, q_out_stride, q_row, v, v_stride, kv_row, tokens))
    return fail(PKV_ERR_INVALID, "q_out may be q, but not overlap the inputs otherwise");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::NormRopeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.out_stride = q_out_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.slot_mapping = slot_mapping;
  p.q_weight = static_cast<const __nv_bfloat16*>(q_weight);
  p.k_weight = static_cast<const __nv_bfloat16*>(k_weight);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_pool = static_cast<__nv_bfloat16*>(k_pool);
  p.v_pool = static_cast<__nv_bfloat16*>(v_pool);
  p.err = st->err;
  p.eps = eps;
  p.max_position = max_position;
  p.rot = rotary_dim;
  p.interleaved = interleaved != 0;
  p.num_tokens = dims->num_q_tokens;
  p.num_q_heads = dims->num_q_heads;
  p.num_kv_heads = dims->num_kv_heads;
  p.num_blocks = dims->num_blocks;
  p.pdl = current_options().pdl != 0;
  const cudaError_t e = pkv::launch_norm_rope_append(p, st->sm_count, stream);
  if (e != cudaSuccess) return cuda_fail(e, "norm_rope_append launch");
  return PKV_OK;
}

int pkv_append_latent(const void* kv, int64_t kv_stride, const int64_t* positions,
                      const float* cos_sin, int64_t max_position, int32_t interleaved,
                      const void* weight, float eps, const int64_t* slot_mapping, void* pool,
                      const void* q_rope, int64_t q_stride, int64_t q_head_stride, void* q_rope_out,
                      int64_t q_out_stride, int64_t q_out_head_stride, const pkv_dims* dims,
                      cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_latent_dims(dims, false);
  if (rc != PKV_OK) return rc;
  if (weight && !eps_ok(eps)) return fail(PKV_ERR_INVALID, "eps must be in [2^-64, 1]");
  if (dims->num_q_tokens == 0) return PKV_OK;
  if (!kv || !positions || !cos_sin || !slot_mapping || !pool)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  const bool turn = dims->num_q_heads > 0 && q_rope != nullptr;
  if (turn && !q_rope_out) return fail(PKV_ERR_INVALID, "q_rope_out is NULL");
  if (!aligned16(kv) || !aligned16(cos_sin) || !aligned16(weight) || !aligned16(pool) ||
      !aligned16(q_rope) || !aligned16(q_rope_out))
    return fail(PKV_ERR_INVALID, "buffers must be 16-byte aligned");
  if (!stride_ok(kv_stride, pkv::kLatRow, dims->num_q_tokens))
    return fail(PKV_ERR_INVALID, "kv_stride must be a multiple of 8 elements and hold a token");
  // (heads and tokens of the queries may lie in either order)
  if (turn && (q_stride % 8 || q_head_stride % 8 || q_out_stride % 8 || q_out_head_stride % 8 ||
               q_stride < 0 || q_head_stride < 0 || q_out_stride < 0 || q_out_head_stride < 0))
    return fail(PKV_ERR_INVALID, "query strides must be multiples of 8 elements");
  if (turn) {
    const Rows in{q_rope, q_stride, q_head_stride}, to{q_rope_out, q_out_stride, q_out_head_stride};
    const int T = dims->num_q_tokens, H = dims->num_q_heads;
    if (!to.apart(T, H)) return fail(PKV_ERR_INVALID, "q_rope_out's rows overlap");
    // (one thread's rows may be another's: only ranges apart, or the same rows)
    if (!in.same(to, T, H) && in.meets(to, T, H))
      return fail(PKV_ERR_INVALID, "q_rope_out may be q_rope, but not overlap it otherwise");
    if (to.meets_tokens(kv, kv_stride, pkv::kLatRow, T, H))
      return fail(PKV_ERR_INVALID, "q_rope_out and kv overlap");
  }
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  pkv::AppendLatentParams p{};
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.kv_stride = kv_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.slot_mapping = slot_mapping;
  p.weight = static_cast<const __nv_bfloat16*>(weight);
  p.pool = static_cast<__nv_bfloat16*>(pool);
  p.q_rope = static_cast<const __nv_bfloat16*>(turn ? q_rope : nullptr);
  p.q_rope_out = static_cast<__nv_bfloat16*>(q_rope_out);
  p.q_stride = q_stride;
  p.q_head_stride = q_head_stride;
  p.out_stride = q_out_stride;
  p.out_head_stride = q_out_head_stride;
  p.err = st->err;
  p.eps = eps;
  p.max_position = max_position;
  p.interleaved = interleaved != 0;
  p.num_tokens = dims->num_q_tokens;
  p.num_q_heads = turn ? dims->num_q_heads : 0;
  p.num_blocks = dims->num_blocks;
  p.pdl = current_options().pdl != 0;
  const cudaError_t e = pkv::launch_append_latent(p, st->sm_count, stream);
  if (e != cudaSuccess) return cuda_fail(e, "append_latent launch");
  return PKV_OK;
}

size_t pkv_latent_workspace_size(const pkv_dims* dims) {
  g_last_error[0] = '\0';
  if (check_latent_dims(dims, false) != PKV_OK) return 0;
  DeviceState* st = device_state();
  if (!st) return 0;
  return latent_layout(st->sm_count).total;
}

int pkv_attention_latent(const void* q, const void* pool, const int32_t* block_tables,
                         const int32_t* seq_lens, const int32_t* query_start_loc, float scale,
                         void* out, const pkv_dims* dims, void* workspace, size_t workspace_bytes,
                         cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_latent_dims(dims, true);
  if (rc != PKV_OK) return rc;
  if (dims->num_reqs == 0 || dims->num_q_tokens == 0) return PKV_OK;
  if (dims->num_blocks == 0) return fail(PKV_ERR_INVALID, "the pool has no blocks");
  if (!q || !pool || !block_tables || !seq_lens || !query_start_loc || !out || !workspace)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(pool) || !aligned16(out))
    return fail(PKV_ERR_INVALID, "q, out and the pool must be 16-byte aligned");
  if (!latent_scale_ok(scale)) return fail(PKV_ERR_INVALID, "scale must be in (0, 2^127]");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  const LatentLayout w = latent_layout(st->sm_count);
  if (workspace_bytes < w.total)
    return fail(PKV_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, w.total);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PKV_ERR_INVALID, "workspace must be 256-byte aligned");
  const pkv_options opt = current_options();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const LatentGroups g = latent_groups(dims);
  pkv::LatentDecodeLaunch L{};
  pkv::LatentDecodeParams& p = L.p;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.pool = static_cast<const __nv_bfloat16*>(pool);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.piece = reinterpret_cast<int*>(ws + w.piece);
  p.piece_ml = reinterpret_cast<float*>(ws + w.ml);
  p.piece_o = reinterpret_cast<float*>(ws + w.o);
  p.piece_rows = g.group_heads * g.group_tokens;
  p.err = st->err;
  p.num_reqs = dims->num_reqs;
  p.num_q_tokens = dims->num_q_tokens;
  p.num_q_heads = dims->num_q_heads;
  p.num_blocks = dims->num_blocks;
  p.max_blocks = dims->max_blocks_per_req;
  p.head_groups = g.head_groups;
  p.group_heads = g.group_heads;
  p.group_tokens = g.group_tokens;
  // What an item costs beside its keys, in keys (500 rows of 30 to 1000 keys, 128 heads:
  // 93 us; at 128 96, at 320 97); pieces of few items hold two tiles at least (192 and 64
  // keys: the same within 1 %; 256: 32 rows of 200 to 700 keys, 32 heads 19.5 us for 18.3).
  p.item_cost = 192;
  p.min_keys = 128;
  // Without cuts, a step whose items have a CTA each and few keys needs no second
  // kernel (four rows, 16 heads: of 480 keys 14.2 us whole, 14.7 cut and joined; of 640
  // 15.9 and 14.6, of 2000 40 and 15; 100 rows of 500 20 and 28).  The table's width
  // stands for the longest row.
  const long long units = st->sm_count / g.head_groups;
  p.merge = dims->num_q_tokens > units || (long long)dims->max_blocks_per_req * pkv::kBlockSize > 512;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.pdl = opt.pdl != 0;
  p.early_plan = p.pdl && opt.early_plan != 0;
  p.debug_withhold_q = opt.debug_withhold_q != 0;
  p.wait_limit_ns = (unsigned long long)opt.wait_limit_us * 1000ull;
  const cuuint32_t qbox[3] = {64, (cuuint32_t)g.group_heads, (cuuint32_t)g.group_tokens};
  rc = encode_bf16_3d(&L.qmap, q, pkv::kLatRow, dims->num_q_heads, dims->num_q_tokens, pkv::kLatRow,
                      (long long)dims->num_q_heads * pkv::kLatRow, qbox, "q");
  if (rc == PKV_OK) rc = encode_latent_map(&L.kmap, pool, dims);
  if (rc != PKV_OK) return rc;
  L.grid = st->sm_count / g.head_groups * g.head_groups;
  const cudaError_t e = pkv::launch_latent_decode(L, stream);
  if (e != cudaSuccess) return cuda_fail(e, "latent attention launch");
  return PKV_OK;
}

int pkv_expand_latent(const void* pool, const void* weight, const int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* kv_start_loc, void* kv, void* k_rope,
                      int32_t num_rows, const pkv_dims* dims, cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_latent_dims(dims, false);
  if (rc != PKV_OK) return rc;
  if (dims->num_q_heads == 0) return fail(PKV_ERR_INVALID, "num_q_heads is 0");
  if (num_rows < 0) return fail(PKV_ERR_INVALID, "num_rows < 0");
  if (dims->num_reqs == 0 || num_rows == 0) return PKV_OK;
  if (dims->num_blocks == 0) return fail(PKV_ERR_INVALID, "the pool has no blocks");
  if (!pool || !weight || !block_tables || !seq_lens || !kv_start_loc || !kv || !k_rope)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(pool) || !aligned16(weight) || !aligned16(kv) || !aligned16(k_rope))
    return fail(PKV_ERR_INVALID, "the pool, weight, kv and k_rope must be 16-byte aligned");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  const pkv_options opt = current_options();
  pkv::LatentExpandLaunch L{};
  pkv::LatentExpandParams& p = L.p;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.kv_start = kv_start_loc;
  p.pool = static_cast<const __nv_bfloat16*>(pool);
  p.kv = static_cast<__nv_bfloat16*>(kv);
  p.k_rope = static_cast<__nv_bfloat16*>(k_rope);
  p.err = st->err;
  p.num_reqs = dims->num_reqs;
  p.num_rows = num_rows;
  p.num_heads = dims->num_q_heads;
  p.num_blocks = dims->num_blocks;
  p.max_blocks = dims->max_blocks_per_req;
  p.pdl = opt.pdl != 0;
  p.debug_withhold_q = opt.debug_withhold_q != 0;
  p.wait_limit_ns = (unsigned long long)opt.wait_limit_us * 1000ull;
  const cuuint32_t wbox[3] = {64, 128, 1};
  rc = encode_latent_map(&L.kmap, pool, dims);
  if (rc == PKV_OK)
    rc = encode_bf16_3d(&L.wmap, weight, pkv::kLatent, dims->num_q_heads * (pkv::kNope + pkv::kValDim), 1,
                        pkv::kLatent, (long long)dims->num_q_heads * (pkv::kNope + pkv::kValDim) * pkv::kLatent,
                        wbox, "weight");
  if (rc != PKV_OK) return rc;
  L.grid = st->sm_count;
  const cudaError_t e = pkv::launch_latent_expand(L, stream);
  if (e != cudaSuccess) return cuda_fail(e, "expand_latent launch");
  return PKV_OK;
}

int pkv_attention_expanded(const void* q, const void* kv, const void* k_rope, const int32_t* seq_lens,
                           const int32_t* query_start_loc, const int32_t* kv_start_loc, float scale,
                           void* out, int32_t num_rows, const pkv_dims* dims, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  g_last_error[0] = '\0';
  int rc = check_latent_dims(dims, false);
  if (rc != PKV_OK) return rc;
  if (dims->num_q_heads == 0) return fail(PKV_ERR_INVALID, "num_q_heads is 0");
  if (num_rows < 0) return fail(PKV_ERR_INVALID, "num_rows < 0");
  if (dims->num_reqs == 0 || dims->num_q_tokens == 0) return PKV_OK;
  if (num_rows == 0) return fail(PKV_ERR_INVALID, "query tokens without keys");
  if (!q || !kv || !k_rope || !seq_lens || !query_start_loc || !kv_start_loc || !out || !workspace)
    return fail(PKV_ERR_INVALID, "NULL pointer argument");
  if (!aligned16(q) || !aligned16(kv) || !aligned16(k_rope) || !aligned16(out))
    return fail(PKV_ERR_INVALID, "q, kv, k_rope and out must be 16-byte aligned");
  if (!latent_scale_ok(scale)) return fail(PKV_ERR_INVALID, "scale must be in (0, 2^127]");
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  const LatentLayout w = latent_layout(st->sm_count);
  if (workspace_bytes < w.total)
    return fail(PKV_ERR_WORKSPACE, "workspace %zu bytes, need %zu", workspace_bytes, w.total);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
    return fail(PKV_ERR_INVALID, "workspace must be 256-byte aligned");
  const pkv_options opt = current_options();
  const int heads = dims->num_q_heads;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  pkv::LatentPrefillLaunch L{};
  pkv::LatentPrefillParams& p = L.p;
  p.seq_lens = seq_lens;
  p.qsl = query_start_loc;
  p.kv_start = kv_start_loc;
  p.kv = static_cast<const __nv_bfloat16*>(kv);
  p.k_rope = static_cast<const __nv_bfloat16*>(k_rope);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.piece = reinterpret_cast<int*>(ws + w.piece);
  p.num_pieces = reinterpret_cast<int*>(ws + 128);
  p.piece_ml = reinterpret_cast<float*>(ws + w.o);
  p.piece_o = p.piece_ml + 4 * (size_t)st->sm_count * 128;
  p.sched = reinterpret_cast<unsigned long long*>(ws);
  p.err = st->err;
  p.wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
  p.num_reqs = dims->num_reqs;
  p.num_q_tokens = dims->num_q_tokens;
  p.num_rows = num_rows;
  p.num_heads = heads;
  // Items are split, and the joining kernel follows, only where the step's rows, were
  // they one request's, are fewer items than CTAs, and the step has keys for an item
  // that is worth it (a chunk of 64, 4 heads: on 700 keys 14.8 us whole, 17.3 split and
  // joined; on 1000 16.5 and 17.3, on 1500 20.5 and 17.4, on 2500 28.8 and 17.4).  The
  // longest request is not known here: many short ones pay 5 us for a join that has
  // nothing to do (30 chunks of 20 on 100 keys 15.2 for 9.5).
  const long long items = ((long long)dims->num_q_tokens + 127) / 128 * heads;
  p.max_pieces = items < st->sm_count && num_rows > 1024 ? 2 * st->sm_count : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.pdl = opt.pdl != 0;
  p.debug_withhold_q = opt.debug_withhold_q != 0;
  p.wait_limit_ns = (unsigned long long)opt.wait_limit_us * 1000ull;
  // In pairs where chunks are long enough for two query tiles on average, and enough (8
  // of 512 on 512-4608 keys, 32 heads 129 us for 138 alone).  Slots that sit the step out
  // count as chunks: four of 1024 on 2000 keys among 60 such run alone, 114 us for 109.
  L.pairs = dims->num_q_tokens >= 192ll * dims->num_reqs &&
            (long long)dims->num_q_tokens * heads >= 256ll * st->sm_count;
  const cuuint32_t keys = L.pairs ? 64 : 128;
  const cuuint32_t box[3] = {64, 1, 128}, kbox[3] = {64, 1, keys}, rbox[3] = {64, keys, 1};
  constexpr int kQ = pkv::kNope + pkv::kRopeDim, kKv = pkv::kNope + pkv::kValDim;
  rc = encode_bf16_3d(&L.qmap, q, kQ, heads, dims->num_q_tokens, kQ, (long long)heads * kQ, box, "q");
  if (rc == PKV_OK)
    rc = encode_bf16_3d(&L.kvmap, kv, kKv, heads, num_rows, kKv, (long long)heads * kKv, box, "kv");
  if (rc == PKV_OK)
    rc = encode_bf16_3d(&L.kmap, kv, kKv, heads, num_rows, kKv, (long long)heads * kKv, kbox, "kv");
  if (rc == PKV_OK)
    rc = encode_bf16_3d(&L.rmap, k_rope, pkv::kRopeDim, num_rows, 1, pkv::kRopeDim,
                        (long long)num_rows * pkv::kRopeDim, rbox, "k_rope");
  if (rc != PKV_OK) return rc;
  L.grid = st->sm_count;
  const cudaError_t e = pkv::launch_latent_prefill(L, stream);
  if (e != cudaSuccess) return cuda_fail(e, "expanded attention launch");
  return PKV_OK;
}

void pkv_get_options(pkv_options* opts) {
  if (opts) *opts = current_options();
}

int pkv_set_options(const pkv_options* opts) {
  g_last_error[0] = '\0';
  if (opts == nullptr) return fail(PKV_ERR_INVALID, "options is NULL");
  if (!options_valid(*opts)) return fail(PKV_ERR_INVALID, "an option is out of range");
  current_options();  // the environment is read once, before the first change
  std::lock_guard<std::mutex> lock(g_opts_mutex);
  g_opts = *opts;
  return PKV_OK;
}

int pkv_get_device_error(cudaStream_t stream) {
  g_last_error[0] = '\0';
  DeviceState* st = device_state();
  if (!st) return PKV_ERR_CUDA;
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int word = 0;
  e = cudaMemcpy(&word, st->err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "read device error word");
  const int zero = 0;
  e = cudaMemcpy(st->err, &zero, sizeof(int), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "clear device error word");
  if (word & pkv::kErrTimeout) return fail(PKV_ERR_TIMEOUT, "a device wait timed out (flags %d)", word);
  if (word & (pkv::kErrBounds | pkv::kErrCapacity))
    return fail(PKV_ERR_DEVICE_BOUNDS, "device bounds violation (flags %d)", word);
  return PKV_OK;
}

#if PKV_PF_TRACE
// Debug builds only: copies the prefill kernel's per-tile timeline.
int pkv_debug_pf_trace(void* host, size_t bytes) {
  return pkv::prefill_trace(host, bytes) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
#endif

#if PKV_TC_TRACE
// Debug builds only: copies the tensor-core decode's per-tile timeline.
int pkv_debug_tc_trace(void* host, size_t bytes) {
  return pkv::decode_tc_trace(host, bytes) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
#endif

#if PKV_TRACE
// Debug builds only: copies the decode kernel's per-CTA phase stamps.
int pkv_debug_trace(void* host, size_t bytes) {
  return pkv::decode_trace(host, bytes) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
#endif

}  // extern "C"
