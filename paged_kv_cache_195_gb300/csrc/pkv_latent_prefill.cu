// pkv_latent_prefill.cu -- causal attention of prefill chunks over expanded keys
// and values of a latent cache, on tcgen05 tensor cores.
//
//   s_j = scale (<q[0:128], k_j,h> + <q[128:192], r_j>),  out = sum_j softmax(s)_j v_j,h
//
// with keys and values of each head side by side in kv [rows, H, 256] and the
// rotated keys r, shared by the heads, in a tensor of their own: a key tile takes
// its three 64-dim chunks from both, and no head's copy of r is ever made.
// Bound: tensor core (640 flops a (row, key, head)).  Measured: 8 chunks of 512 on up
// to 4608 keys, 32 heads 112 us (1199 TFLOP/s; a tile's softmax, 0.85 us a pair's 256
// rows, is longer than its products' 0.67); three odd chunks, 16 heads 12.9 us.
//
// Tiling.  A work item is (request, head, 128 query tokens); a key tile is 128
// keys.  S = Q K^T (12 MMAs of K = 16) and P (bf16) have two TMEM buffers each, so
// that scores run two tiles ahead of the products (over its S, P held that back for
// the product: 1.1 us a tile), and O += P V (8 MMAs, A from TMEM) accumulates in 128
// columns.  Four threads a row run the softmax, 32 keys each; the row maximum moves,
// and O is rescaled, only when a score exceeds it by 2^8, on a vote of the four warps
// that hold the same rows.  Keys and values have rings of their own, of 64-dim chunks,
// each of which goes back as soon as its MMAs are done.
// Steps of long chunks run in pairs of CTAs (cta_group::2): the pair takes two query
// tiles of one head, 256 MMA rows, and each CTA holds half of the keys and half of
// the value dims of a tile: half the copies, half the operand reads, and room for
// four tiles in flight.  A CTA alone holds all 80 KB of a tile, which with the
// MMAs' own reads is more than shared memory and the copies give (1.04-1.09 us a
// tile).
//
// Order.  A CTA's first item is its own by its number, the others come from a queue,
// longest requests first, a head's query tiles one after the other (the CTAs that run
// them at one time read the same keys: L2), later tiles first, as they see more keys.  With too few items for the
// GPU each is cut over its keys into pieces, numbered like items, whose
// unnormalised states a second kernel joins.
//
// A value that only some rows of an item see must not reach the others, whatever
// it holds (0 * NaN): the NaN and infinities among the values of the item's own
// tokens are taken out, by the warp that copies them, and added to the rows that
// see them at the end.
#include <climits>

#include "pkv_latent.h"
#include "pkv_pair.cuh"

namespace pkv {
namespace {

constexpr int kParts = 4;                // softmax threads a row
constexpr int kPartKeys = 128 / kParts;  // keys, and output dims, of each
constexpr int kSoftWarps = 4 * kParts;
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kWarpK = kSoftWarps;       // items, Q, keys
constexpr int kWarpS = kSoftWarps + 1;   // MMAs of the scores
constexpr int kWarpV = kSoftWarps + 2;   // values
constexpr int kWarpO = kSoftWarps + 3;   // MMAs of the outputs
constexpr int kThreads = 32 * (kSoftWarps + 4);  // five warps a quarter SM: up to 96 registers
constexpr int kBarSoft = 1;              // all softmax warps
constexpr int kBarQuad = 2;              // + quad: the four warps with the same rows

constexpr int kRows = 128;
constexpr int kTile = 128;
constexpr int kChunkBytes = 128 * 128;
constexpr int kQDim = kNope + kRopeDim;
constexpr int kKChunks = kQDim / 64;
constexpr int kVChunks = kValDim / 64;
// Chunks in flight.  Alone: of 128 keys, two tiles and a third of keys and two of
// values; a pair's CTA: of 64 keys, four tiles and two thirds, and (64 of the dims of
// all keys) four of values.
constexpr int kBytesK = 7 * kChunkBytes;
constexpr int kRingV = 4;
constexpr int kItems = 4;
constexpr int kBadItems = 8;
constexpr uint32_t kTmemCols = 512;      // S: columns 0 .. 255, O: 256 .. 383, P: 384 .. 511
constexpr int kColO = 2 * kTile;
constexpr int kColP = kColO + kValDim;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kMinPieceTiles = 2;        // (four: a chunk of 128 on 1500 keys, 8 heads 20.7 us for 18.8)

// A piece of an item: key tiles t0 .. t1 - 1 of its keys.
struct Item {
  int row0, nt;  // first query row, query tokens
  int pos0;      // position of the first
  int head;
  int k0;        // first row of the request's keys
  int t0, t1;
  int slot;      // piece number, if the item is split; else -1
  int gpos0;     // of the pair's two query tiles: position of the first token, ...
  int gnt;       // ... query tokens
  int end;
};

struct __align__(1024) Smem {
  uint8_t q[kKChunks][kChunkBytes];
  uint8_t k[kBytesK];
  uint8_t v[kRingV][kChunkBytes];
  uint64_t q_full, q_empty;
  uint64_t k_full[14], k_empty[14], v_full[kRingV], v_empty[kRingV];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2];
  uint64_t o_full, o_empty;
  uint64_t item_full[kItems], next_full[kItems];
  uint64_t drained[2];
  Item items[kItems];
  unsigned long long next[kItems];    // a pair: the piece's number, from its first CTA
  float xrow[kParts][kRows];
  unsigned long long bad[kBadItems][4];  // own tokens whose values were taken out
  uint32_t tmem_base;
  int active;  // CTAs that take pieces
  int split;   // key tiles of a piece (INT_MAX: items are whole)
  int pieces;  // of a step whose items are split, else 0
  WaitCtl wait;
};
// (no room to align it in: a block without static shared memory has it on a KiB)
static_assert(sizeof(Smem) <= 227 * 1024, "latent prefill shared memory");

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct Req {
  int q0, qr, L, k0;
  int nq;  // query tiles of a head (0: nothing to do)
};

// GROUP: query tokens of an item (of a pair's two).
template <int GROUP>
__device__ __forceinline__ Req load_req(const LatentPrefillParams& p, int r, bool* bad) {
  Req a;
  a.q0 = __ldg(p.qsl + r);
  const int q1 = __ldg(p.qsl + r + 1);
  a.L = __ldg(p.seq_lens + r);
  a.k0 = __ldg(p.kv_start + r);
  const int k1 = __ldg(p.kv_start + r + 1);
  a.qr = q1 - a.q0;
  // (ends not before starts: the difference of wild entries may wrap)
  *bad = !(a.q0 >= 0 && q1 >= a.q0 && q1 <= p.num_q_tokens && a.qr <= a.L && a.k0 >= 0 && k1 >= a.k0 &&
           k1 <= p.num_rows && k1 - a.k0 == a.L);
  a.nq = *bad ? 0 : cdiv(a.qr, GROUP);
  return a;
}

// Key tiles of query tile (or pair) i.
template <int GROUP>
__device__ __forceinline__ int item_tiles(const Req& a, int i) {
  return cdiv(a.L - a.qr + min((i + 1) * GROUP, a.qr), kTile);
}

// Pieces of a request's head.
template <int GROUP>
__device__ __forceinline__ int head_pieces(const Req& a, int split) {
  if (split == INT_MAX) return a.nq;
  int n = 0;
  for (int i = 0; i < a.nq; ++i) n += cdiv(item_tiles<GROUP>(a, i), split);
  return n;
}

__device__ __forceinline__ long long warp_sum(long long v) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Key tiles of a piece, from the step's items: whole while they are enough for
// the grid (or there is no room for more), else the key tiles in equal parts.
// One warp; also counts the pieces.
template <int GROUP>
__device__ __forceinline__ int plan_split(const LatentPrefillParams& p, int grid, long long* pieces) {
  const int lane = threadIdx.x & 31;
  long long items = 0, tiles = 0;
  for (int r = lane; r < p.num_reqs; r += 32) {
    bool bad;
    const Req a = load_req<GROUP>(p, r, &bad);
    if (bad && blockIdx.x == 0) record_error(p.err, kErrBounds);  // the request is skipped
    items += (long long)a.nq * p.num_heads;
    if (p.max_pieces > 0)
      for (int i = 0; i < a.nq; ++i) tiles += (long long)item_tiles<GROUP>(a, i) * p.num_heads;
  }
  items = warp_sum(items);
  *pieces = items;
  if (p.max_pieces == 0 || 3 * items >= 2 * grid) return INT_MAX;
  tiles = warp_sum(tiles);
  // ceil(tiles / split) summed over the items is at most grid + items < 2 grid.  More
  // than the grid would take two rounds: longer pieces, up to nearly twice as long, if
  // they come down to it (two chunks of 128 on 3000 keys, 32 heads 35.5 us for 41.7).
  const int least = max(kMinPieceTiles, (int)((tiles + grid - 1) / grid));
  int split = least;
  for (int s = least; s < 2 * least; s += (least + 7) / 8) {
    long long n = 0;
    for (int r = lane; r < p.num_reqs; r += 32) {
      bool bad;
      n += (long long)head_pieces<GROUP>(load_req<GROUP>(p, r, &bad), s) * p.num_heads;
    }
    n = warp_sum(n);
    if (s == least || n <= grid) *pieces = n, split = s;
    if (n <= grid) break;
  }
  return split;
}

// Finds pieces by number, forward.  Pieces are numbered by batches of 32
// requests, within a batch the longest request first, then head by head, then
// from the last query tile to the first, then along the keys.  One warp.
template <int GROUP>
struct Finder {
  int batch;       // first request of the batch
  long long base;  // pieces before it
  Req a;           // this lane's request
  int per_head;
  long long cnt, excl, total;

  __device__ __forceinline__ void load(const LatentPrefillParams& p, int split) {
    const int lane = threadIdx.x & 31, r = batch + lane;
    bool bad;
    a = Req{0, 0, 0, 0, 0};
    if (r < p.num_reqs) a = load_req<GROUP>(p, r, &bad);
    per_head = head_pieces<GROUP>(a, split);
    cnt = (long long)per_head * p.num_heads;
    total = warp_sum(cnt);
    const int key = cnt > 0 ? a.L : -1;
    excl = 0;
    #pragma unroll 4
    for (int s = 0; s < 32; ++s) {
      const int ks = __shfl_sync(0xffffffffu, key, s);
      const long long cs = __shfl_sync(0xffffffffu, cnt, s);
      if (ks > key || (ks == key && s < lane)) excl += cs;
    }
  }
  __device__ __forceinline__ void start(const LatentPrefillParams& p, int split) {
    batch = 0;
    base = 0;
    load(p, split);
  }
  // Numbers must not decrease from call to call.  False: there is no such piece.
  // (rank: which of a pair's query tiles)
  __device__ __forceinline__ bool find(const LatentPrefillParams& p, int split, long long piece, int rank,
                                       Item* it, int* of) {
    while (piece >= base + total) {
      base += total;
      batch += 32;
      if (batch >= p.num_reqs) return false;
      load(p, split);
    }
    const long long rel = piece - base;
    const unsigned own = __ballot_sync(0xffffffffu, cnt > 0 && excl <= rel && rel < excl + cnt);
    const int src = __ffs(own) - 1;
    const long long local = rel - __shfl_sync(0xffffffffu, excl, src);
    Req b;
    b.q0 = __shfl_sync(0xffffffffu, a.q0, src);
    b.qr = __shfl_sync(0xffffffffu, a.qr, src);
    b.L = __shfl_sync(0xffffffffu, a.L, src);
    b.k0 = __shfl_sync(0xffffffffu, a.k0, src);
    b.nq = __shfl_sync(0xffffffffu, a.nq, src);
    const int each = __shfl_sync(0xffffffffu, per_head, src);
    it->head = (int)(local / each);
    int x = (int)(local - (long long)it->head * each), i = b.nq - 1, n = 1;
    if (split == INT_MAX) {
      i -= x;
      x = 0;
    } else {
      for (; (n = cdiv(item_tiles<GROUP>(b, i), split)) <= x; --i) x -= n;
    }
    const int tiles = item_tiles<GROUP>(b, i);
    const int first = i * GROUP + rank * kRows;  // (past the request's tokens: a pair's second may have none)
    it->row0 = b.q0 + first;
    it->nt = min(kRows, b.qr - first);
    it->pos0 = b.L - b.qr + first;
    it->gpos0 = b.L - b.qr + i * GROUP;
    it->gnt = min(GROUP, b.qr - i * GROUP);
    it->k0 = b.k0;
    // n pieces of equal length, but for the rounding
    it->t0 = (int)((long long)tiles * x / n);
    it->t1 = (int)((long long)tiles * (x + 1) / n);
    it->slot = n > 1 ? (int)piece : -1;
    it->end = 0;
    *of = n > 1 && x == 0 ? n : 0;
    return true;
  }
};

// Thirty-two bytes, a whole sector.  (A thread has a row: each store of a warp goes to
// 32 lines, and in sixteens there are twice as many: 8 chunks of 512, 32 heads 113.1 us
// for 117.0, 16 of 256, 40 heads 94.7 for 104.3.)
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// O (32 columns at TMEM address tO) times alpha.
static __device__ __noinline__ void rescale_o32(uint32_t tO, float alpha) {
  float o[32];
  tmem_ld32(tO, o);
  tc_wait_ld();
  #pragma unroll
  for (int i = 0; i < 32; ++i) o[i] *= alpha;
  tmem_st32(tO, o);
  tc_wait_st();
}

__device__ __forceinline__ bool non_finite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Two bf16 numbers, zeros for those that are not finite.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  return (w & 0x7f800000u) == 0x7f800000u ? w & 0xffffu : w;
}

// Values of the tile's keys from pos0 + 1 on, the item's first token's position:
// where any is not finite, such rows that no row of the item sees (from its last
// token's position on) become zeros; in those of its own tokens the numbers that are
// not finite do, and the token is noted in bad (a pair's: in both CTAs').  One warp;
// v: CHUNKS chunks of 64 dims.
template <int CHUNKS, bool PAIR>
static __device__ __noinline__ void clean_values(uint8_t (*v)[kChunkBytes], int key0, int pos0, int nt,
                                                 unsigned long long* bad, int rank, int lane) {
  constexpr int kPieces = 8 * CHUNKS;   // of 16 bytes, a row
  constexpr int kRowsAt = 32 / kPieces; // a warp's rows at a time
  const int piece = lane % kPieces;
  auto at = [&](int row) {
    return reinterpret_cast<uint4*>(v[piece >> 3] + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
  };
  const int first = max(pos0 + 1 - key0, 0);
  uint32_t top = 0;  // the largest exponents, two to a word
  #pragma unroll 1
  for (int r0 = first + lane / kPieces; __any_sync(0xffffffffu, r0 < kTile); r0 += 8 * kRowsAt) {
    uint4 x[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = *at(min(r0 + i * kRowsAt, kTile - 1));
    #pragma unroll
    for (int i = 0; i < 8; ++i)
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7f807f80u, x[i].y & 0x7f807f80u),
                                   __vmaxu2(x[i].z & 0x7f807f80u, x[i].w & 0x7f807f80u)));
  }
  if (!__any_sync(0xffffffffu, non_finite(top))) return;
  #pragma unroll 1
  for (int row = first; row < kTile; ++row) {
    const int b = key0 + row - pos0 - 1;  // the item's token b + 1
    uint4 x = *at(row);
    if (!__any_sync(0xffffffffu, non_finite(x.x) || non_finite(x.y) || non_finite(x.z) || non_finite(x.w))) continue;
    if (b < nt - 1) {
      if (lane == 0) {
        atomicOr(bad + (b >> 6), 1ull << (b & 63));
        if (PAIR) or_other(bad + (b >> 6), rank, 1ull << (b & 63));
      }
      x = make_uint4(finite_only(x.x), finite_only(x.y), finite_only(x.z), finite_only(x.w));
    } else {
      x = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    if (lane < kPieces) *at(row) = x;
  }
}

// Whether the key of row `row` of kv, its part in k_rope with it, is finite.
__device__ __forceinline__ bool finite_key(const LatentPrefillParams& p, long long row, int head) {
  const uint32_t* k = reinterpret_cast<const uint32_t*>(p.kv + (row * p.num_heads + head) * (kNope + kValDim));
  const uint32_t* r = reinterpret_cast<const uint32_t*>(p.k_rope + row * kRopeDim);
  bool out = false;
  for (int i = 0; i < kNope / 2; ++i) out = out || non_finite(k[i]);
  for (int i = 0; i < kRopeDim / 2; ++i) out = out || non_finite(r[i]);
  return !out;
}

// What the values taken out add to a row that sees the first `seen` of them: its
// weight is positive, so a NaN stays one and an infinity keeps its sign.  But where
// the key is not finite either, the row scored it -inf (or is all NaN already), and a
// weight of 0 makes a NaN of an infinity.
static __device__ __noinline__ void add_bad(const LatentPrefillParams& p, const Item& it,
                                            const unsigned long long* bad, int seen, int d0, float (&o)[32]) {
  for (int b = 0; b < seen; ++b) {
    if (!((bad[b >> 6] >> (b & 63)) & 1)) continue;
    const long long row = (long long)it.k0 + it.gpos0 + 1 + b;
    const __nv_bfloat16* v = p.kv + (row * p.num_heads + it.head) * (kNope + kValDim) + kNope + d0;
    const bool weighs = finite_key(p, row, it.head);
    #pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float x = __bfloat162float(v[i]);
      if (!(x - x == 0.f)) o[i] += weighs ? x : NAN;
    }
  }
}

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kvmap, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap rmap, const LatentPrefillParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) record_error(p.err, kErrCapacity);
    return;
  }
  WaitCtl* ctl = &sm.wait;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int GROUP = PAIR ? 2 * kRows : kRows;
  constexpr int kCtas = PAIR ? 2 : 1;
  constexpr int kKeyRows = kTile / kCtas;        // keys of a tile that this CTA holds
  constexpr int kKBytes = kKeyRows * 128;        // ... a chunk of them
  constexpr int kRingK = kBytesK / kKBytes;
  constexpr int kVCount = kVChunks / kCtas;      // chunks of a tile's values that it holds
  const int rank = PAIR ? blockIdx.x & 1 : 0;    // in the pair, whose first CTA issues all MMAs

  if (tid == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int s = 0; s < kRingK; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kRingV; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.p_full[b], kCtas * (kSoftWarps + 1));
      mbar_init(&sm.p_free[b], 1);
      mbar_init(&sm.s_free[b], kCtas * kSoftWarps);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kCtas * kSoftWarps);
    for (int b = 0; b < kItems; ++b) {
      mbar_init(&sm.item_full[b], 1);
      mbar_init(&sm.next_full[b], 1);
    }
    for (int b = 0; b < 4 * kBadItems; ++b) sm.bad[b >> 2][b & 3] = 0;
    mbar_init(&sm.drained[0], 1);
    mbar_init(&sm.drained[1], 1);
    sm.wait.abort = 0;
    sm.wait.limit_ns = p.wait_limit_ns;
    fence_barrier_init();
  }
  if (warp == kWarpV && lane == 0) {
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kvmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&rmap);
  }
  // The plan is made after the wait: the running sum of the lengths is as a rule the work
  // of a kernel just ahead.  (A CTA without work waits too: the next kernel relies on all
  // before this one.)
  grid_dependency_wait();
  allow_dependent_launch();
  // Nothing to join, unless the last CTA to finish says otherwise.
  if (p.max_pieces > 0 && blockIdx.x == 0 && tid == 0) *p.num_pieces = 0;
  Finder<GROUP> f;  // (of warp kWarpK)
  if (warp == kWarpK) {
    long long pieces;
    const int split = plan_split<GROUP>(p, gridDim.x, &pieces);
    f.start(p, split);
    if (lane == 0) {
      sm.split = split;
      sm.pieces = split != INT_MAX ? (int)pieces : 0;
      sm.active = (int)min(pieces, (long long)(PAIR ? gridDim.x >> 1 : gridDim.x));  // CTAs, or pairs
    }
  }
  __syncthreads();
  const int active = sm.active, split = sm.split;
  if ((int)(PAIR ? blockIdx.x >> 1 : blockIdx.x) >= active) return;
  if (warp == kWarpS) {
    if (PAIR) {
      tmem_alloc_pair(&sm.tmem_base, kTmemCols);
    } else {
      tmem_alloc(&sm.tmem_base, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem_base);
  if (PAIR) cluster_barrier();  // both CTAs' barriers are ready

  // Arrive on a barrier -- both CTAs', in a pair -- once the MMAs so far are done.
  auto commit = [](uint64_t* bar) { PAIR ? commit_pair(bar) : tc_commit(bar); };

  if (warp == kWarpK || warp == kWarpV) {
    // =========================== copies ===================================
    const bool vside = warp == kWarpV;
    const bool leader = elect_one();
    int slot = 0, phase = 1, n_chunk = 0;  // the chunk's slot and the parity it waits for; chunks so far
    bool ok = true;
    if (vside) {
      // ---- values: this CTA's chunks, on its own barriers
      int t = 0, f_slot = 0, f_phase = 0;
      // A tile's values have landed: what not every row may see is taken out.  The
      // arrival, beside the softmax warps', lets the tile's product begin.
      auto finish = [&](const Item& it, int n_item, int j, int tt) {
        const int first = f_slot;
        #pragma unroll
        for (int c = 0; c < kVCount; ++c) {
          if (!all_of(wait_for(&sm.v_full[f_slot], f_phase, p.err, ctl))) return false;
          if (++f_slot == kRingV) f_slot = 0, f_phase ^= 1;
        }
        if ((j + 1) * kTile > it.gpos0 + 1)
          clean_values<kVCount, PAIR>(sm.v + first, j * kTile, it.gpos0, it.gnt, sm.bad[n_item % kBadItems], rank, lane);
        fence_proxy_async_smem();
        // (the barrier's phase before, tile tt - 2's, must be over)
        if (tt >= 2 && !all_of(wait_for(&sm.p_free[tt & 1], ((tt >> 1) - 1) & 1, p.err, ctl))) return false;
        __syncwarp();
        if (lane == 0) PAIR ? arrive_at(first_cta(&sm.p_full[tt & 1])) : mbar_arrive(&sm.p_full[tt & 1]);
        return true;
      };
      for (int n_item = 0; ok; ++n_item) {
        ok = all_of(wait_for(&sm.item_full[n_item % kItems], (n_item / kItems) & 1, p.err, ctl));
        if (!ok) break;
        const Item it = sm.items[n_item % kItems];
        if (it.end) break;
        const int head = uniform(it.head), t0 = uniform(it.t0), t1 = uniform(it.t1);
        int y = uniform(it.k0 + it.t0 * kTile);
        #pragma unroll 1
        for (int j = t0; j < t1 && ok; ++j, ++t, y += kTile) {
          #pragma unroll
          for (int c = 0; c < kVCount; ++c) {
            ok = ok && all_of(wait_for(&sm.v_empty[slot], phase, p.err, ctl));
            if (!ok) break;
            if (leader) {
              mbar_arrive_expect_tx(&sm.v_full[slot], kChunkBytes);
              tma_load_3d(sm.v[slot], &kvmap, kNope + (PAIR ? rank : c) * 64, head, y, &sm.v_full[slot]);
            }
            __syncwarp();
            ++n_chunk;
            if (++slot == kRingV) slot = 0, phase ^= 1;
          }
          // (one tile behind, so that the next one's copies are under way)
          if (ok && j > t0) ok = finish(it, n_item, j - 1, t - 1);
        }
        ok = ok && finish(it, n_item, t1 - 1, t - 1);
      }
      if (!ok) {
        // Aborted: the copies in flight must land before the CTA ends.
        for (int i = max(0, n_chunk - kRingV); i < n_chunk; ++i)
          drain(&sm.v_full[i % kRingV], (i / kRingV) & 1, p.err, ctl);
      }
    } else {
      // ---- items, queries and keys; a pair's on the first CTA's barriers
      int n_item = 0;
      for (int n = 0; ok; ++n) {
        // The first piece is the CTA's own, by its number; the others come from the
        // queue.  A pair's first CTA takes the number for both.
        unsigned long long v = PAIR ? blockIdx.x >> 1 : blockIdx.x;
        const int at = (n - 1) % kItems;
        if (n > 0 && (!PAIR || rank == 0)) {
          if (lane == 0) v = active + atomicAdd(p.sched, 1ull);
          v = __shfl_sync(0xffffffffu, v, 0);
          if (PAIR && lane == 0) send_second(&sm.next[at], &sm.next_full[at], v);
        } else if (n > 0) {
          ok = all_of(wait_for(&sm.next_full[at], ((n - 1) / kItems) & 1, p.err, ctl));
          if (!ok) break;
          asm volatile("fence.acq_rel.cluster;" ::: "memory");
          v = *(volatile unsigned long long*)&sm.next[at];
        }
        Item it;
        int of;
        if (!f.find(p, split, (long long)v, rank, &it, &of)) break;
        // For the joining kernel: every piece's record is written anew by whoever
        // takes it.
        if (split != INT_MAX && lane == 0)
          *reinterpret_cast<int4*>(p.piece + 4 * v) = make_int4(of, it.row0, it.nt, it.head);
        const int head = uniform(it.head), row0 = uniform(it.row0), t0 = uniform(it.t0), t1 = uniform(it.t1);
        int y = uniform(it.k0 + it.t0 * kTile) + rank * kKeyRows;
        #pragma unroll 1
        for (int j = t0; j < t1 && ok; ++j, y += kTile) {
          #pragma unroll
          for (int c = 0; c < kKChunks; ++c) {
            ok = ok && all_of(wait_for(&sm.k_empty[slot], phase, p.err, ctl));
            if (!ok) break;
            if (leader) {
              uint8_t* const dst = sm.k + slot * kKBytes;
              uint64_t* const bar = &sm.k_full[slot];
              if (rank == 0) mbar_arrive_expect_tx(bar, kChunkBytes);  // (both CTAs' halves)
              const bool rope = c == kKChunks - 1;
              const CUtensorMap* const map = rope ? &rmap : &kmap;
              const int c0 = rope ? 0 : c * 64, c1 = rope ? y : head, c2 = rope ? 0 : y;
              if (PAIR) tma_load_3d_pair(dst, map, c0, c1, c2, first_cta(bar));
              else tma_load_3d(dst, map, c0, c1, c2, bar);
            }
            __syncwarp();
            ++n_chunk;
            if (++slot == kRingK) slot = 0, phase ^= 1;
          }
          if (ok && j == t0) {
            // The item's queries, once the MMAs of the item before are done with
            // theirs (its first keys are on their way).
            if (n_item > 0) ok = all_of(wait_for(&sm.q_empty, (n_item - 1) & 1, p.err, ctl));
            if (!ok) break;
            if (leader) {
              sm.items[n_item % kItems] = it;
              mbar_arrive(&sm.item_full[n_item % kItems]);
              if (rank == 0) mbar_arrive_expect_tx(&sm.q_full, kCtas * kKChunks * kChunkBytes);
              #pragma unroll
              for (int c = 0; c < kKChunks; ++c) {
                if (p.debug_withhold_q) break;
                if (PAIR) tma_load_3d_pair(sm.q[c], &qmap, c * 64, head, row0, first_cta(&sm.q_full));
                else tma_load_3d(sm.q[c], &qmap, c * 64, head, row0, &sm.q_full);
              }
            }
            ++n_item;
            __syncwarp();
          }
        }
      }
      if (ok && n_item > 0) ok = all_of(wait_for(&sm.q_empty, (n_item - 1) & 1, p.err, ctl));
      if (ok && lane == 0) {
        sm.items[n_item % kItems].end = 1;
        mbar_arrive(&sm.item_full[n_item % kItems]);
        if (rank == 0) mbar_arrive(&sm.q_full);
      }
      __syncwarp();
      if (!ok && rank == 0) {
        // Aborted: the copies in flight must land before the CTA ends (the barrier at
        // the end keeps a pair's other CTA until then).
        if (n_item > 0) drain(&sm.q_full, (n_item - 1) & 1, p.err, ctl);
        for (int i = max(0, n_chunk - kRingK); i < n_chunk; ++i)
          drain(&sm.k_full[i % kRingK], (i / kRingK) & 1, p.err, ctl);
      } else if (!ok) {
        settle();
      }
    }
  } else if (warp == kWarpS && rank == 0) {
    // ========================= MMAs of the scores =========================
    constexpr uint32_t kIdesc = idesc_bf16_f32(kCtas * kRows, kTile, 0, 0);
    constexpr int kStep = kChunkBytes >> 4;
    const uint64_t desc_q = smem_desc_sw128(smem_u32(sm.q[0]), 16, 1024);
    const uint64_t desc_k = smem_desc_sw128(smem_u32(sm.k), 16, 1024);
    const bool leader = elect_one();
    bool ok = true;
    int slot = 0, phase = 0;
    for (int n_item = 0, t = 0;; ++n_item) {
      ok = all_of(wait_for(&sm.q_full, n_item & 1, p.err, ctl));
      if (!ok) break;
      const Item& it = sm.items[n_item % kItems];
      if (uniform(it.end)) break;
      #pragma unroll 1
      for (int left = uniform(it.t1 - it.t0); left > 0; --left, ++t) {
        const int b = t & 1;
        // (the softmax has taken the scores of tile t - 2)
        if (t >= 2) ok = all_of(wait_for(&sm.s_free[b], ((t >> 1) - 1) & 1, p.err, ctl));
        #pragma unroll
        for (int c = 0; c < kKChunks; ++c) {
          ok = ok && all_of(wait_for(&sm.k_full[slot], phase, p.err, ctl));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t db = desc_k + (uint64_t)(slot * (kKBytes >> 4));
            #pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint64_t da = desc_q + (c * kStep + 2 * kk);
              if (PAIR) mma_pair(tmem + b * kTile, da, db + 2 * kk, kIdesc, c > 0 || kk > 0);
              else tc_mma_f16_ss(tmem + b * kTile, da, db + 2 * kk, kIdesc, c > 0 || kk > 0);
            }
            commit(&sm.k_empty[slot]);
          }
          __syncwarp();
          if (++slot == kRingK) slot = 0, phase ^= 1;
        }
        if (!ok) break;
        if (leader) {
          commit(&sm.s_full[b]);
          if (left == 1) commit(&sm.q_empty);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (!ok) {
      // Aborted: the issued MMAs must end before TMEM is freed.
      if (leader) commit(&sm.drained[0]);
      __syncwarp();
      drain(&sm.drained[0], 0, p.err, ctl);
    }
  } else if (warp == kWarpO && rank == 0) {
    // ========================= MMAs of the outputs ========================
    // V is MN-major: atoms of 64 dims x 8 keys.  Alone, a chunk's 64 dims at a time (A
    // comes from TMEM: no slower than all 128).
    constexpr uint32_t kIdesc = idesc_bf16_f32(kCtas * kRows, PAIR ? kValDim : 64, 0, 1);
    constexpr int kStep = kChunkBytes >> 4;
    const uint64_t desc_v = smem_desc_sw128(smem_u32(sm.v[0]), kChunkBytes, 1024);
    const bool leader = elect_one();
    bool ok = true;
    int slot = 0;
    for (int n_item = 0, t = 0;; ++n_item) {
      ok = all_of(wait_for(&sm.item_full[n_item % kItems], (n_item / kItems) & 1, p.err, ctl));
      if (!ok) break;
      const Item& it = sm.items[n_item % kItems];
      if (uniform(it.end)) break;
      const int n = uniform(it.t1 - it.t0);
      #pragma unroll 1
      for (int j = 0; j < n; ++j, ++t) {
        const int b = t & 1;
        // (the values have landed: the warps that copy them arrive on p_full too)
        if (j == 0 && n_item > 0) ok = wait_for(&sm.o_empty, (n_item - 1) & 1, p.err, ctl);
        ok = all_of(ok && wait_for(&sm.p_full[b], (t >> 1) & 1, p.err, ctl));
        if (!ok) break;
        tc_fence_after();
        #pragma unroll
        for (int c = 0; c < kVCount; ++c) {
          if (leader) {
            const uint64_t db = desc_v + (uint64_t)(slot * kStep);
            #pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) {
              // P: two keys a column.
              const uint32_t ta = tmem + kColP + b * (kTile / 2) + kk * 8;
              if (PAIR) mma_pair_ts(tmem + kColO, ta, db + kk * (2048 >> 4), kIdesc, j > 0 || kk > 0);
              else tc_mma_f16_ts(tmem + kColO + c * 64, ta, db + kk * (2048 >> 4), kIdesc, j > 0 || kk > 0);
            }
            commit(&sm.v_empty[slot]);
          }
          __syncwarp();
          if (++slot == kRingV) slot = 0;
        }
        if (leader) {
          commit(&sm.p_free[b]);
          if (j == n - 1) commit(&sm.o_full);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (!ok) {
      // Aborted: the issued MMAs must end before TMEM is freed.
      if (leader) commit(&sm.drained[1]);
      __syncwarp();
      drain(&sm.drained[1], 0, p.err, ctl);
    }
  } else if (warp < kSoftWarps) {
    // ==================== softmax and epilogue (warps 0-15) ==================
    // Warps 4 c .. 4 c + 3 take keys 32 c .. 32 c + 31 of a tile and output dims
    // 32 c ..; warp w reaches TMEM lanes 32 (w % 4) ..
    const int quad = warp & 3, part = warp >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tmem + lane_off + kColO + part * kPartKeys;
    int t = 0;
    bool ok = true;
    for (int n_item = 0;; ++n_item) {
      const bool have = wait_for(&sm.item_full[n_item % kItems], (n_item / kItems) & 1, p.err, ctl);
      const Item it = sm.items[n_item % kItems];
      // Agree before any other barrier: a wait that gave up stops everyone.  (Also:
      // sm.xrow is free again.)
      if (barrier_or(kBarSoft, kSoftThreads, !have || !ok || it.end)) break;
      const unsigned long long* bad = sm.bad[n_item % kBadItems];
      // The item before is done with: its notes are empty again, long before items
      // that have theirs in the same place.
      if (tid < 4 && n_item > 0) sm.bad[(n_item - 1) % kBadItems][tid] = 0;
      const bool valid = row < it.nt;
      const int prow = valid ? it.pos0 + row : -1;  // the last key that the row sees
      float m = -INFINITY, l = 0.f;
      for (int j = it.t0; j < it.t1; ++j, ++t) {
        const int sb = t & 1;
        const uint32_t tS = tmem + lane_off + sb * kTile;
        ok = ok && wait_for(&sm.s_full[sb], (t >> 1) & 1, p.err, ctl);
        tc_fence_after();
        const int kbase = j * kTile + part * kPartKeys;
        float v[kPartKeys];
        tmem_ld32(tS + part * kPartKeys, v);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) PAIR ? arrive_at(first_cta(&sm.s_free[sb])) : mbar_arrive(&sm.s_free[sb]);
        if (kbase + kPartKeys - 1 > prow) {
          #pragma unroll
          for (int i = 0; i < kPartKeys; ++i)
            if (kbase + i > prow) v[i] = -INFINITY;
        }
        float mxp[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) mxp[i] = -INFINITY;
        #pragma unroll
        for (int i = 0; i < kPartKeys / 2; ++i) mxp[i & 3] = fmax3(mxp[i & 3], v[2 * i], v[2 * i + 1]);
        const float mxh = fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])) * p.scale_log2;
        const bool exchange = barrier_or(kBarQuad + quad, 128, j == it.t0 || mxh > m + kRescaleLog2);
        if (exchange) {
          sm.xrow[part][row] = mxh;
          named_barrier(kBarQuad + quad, 128);
          const float mx = fmaxf(fmaxf(sm.xrow[0][row], sm.xrow[1][row]),
                                 fmaxf(sm.xrow[2][row], sm.xrow[3][row]));
          named_barrier(kBarQuad + quad, 128);
          const bool grow = mx > m + kRescaleLog2 || (m == -INFINITY && mx > m);
          const float m_new = grow ? mx : m;
          if (j > it.t0 && __any_sync(0xffffffffu, grow)) {
            // O and l move to the new reference; O must hold the tile before.
            ok = ok && wait_for(&sm.p_free[(t - 1) & 1], ((t - 1) >> 1) & 1, p.err, ctl);
            tc_fence_after();
            const float alpha = grow && m != -INFINITY ? fast_exp2(m - m_new) : 1.f;
            rescale_o32(tO, alpha);
            l *= alpha;
          }
          m = m_new;
        }
        // P = exp2(s scale - m), two keys a column; the sum adds the rounded values
        // that the product uses.  (A row that saw no key yet
        // has m = -inf.)
        const float ref = m == -INFINITY ? 0.f : m;
        const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 nm2 = make_float2(-ref, -ref);
        float sum_lo[2] = {0.f, 0.f}, sum_hi[2] = {0.f, 0.f};
        uint32_t w[kPartKeys / 2];
        #pragma unroll
        for (int e = 0; e < kPartKeys / 2; ++e) {
          const float2 x = ffma2(make_float2(v[2 * e], v[2 * e + 1]), sc2, nm2);
          w[e] = pack_bf16(fast_exp2(x.x), fast_exp2(x.y));
          add_bf16x2(sum_lo[e & 1], sum_hi[e & 1], w[e]);
        }
        // (P's buffer is free once the product of tile t - 2 is done)
        if (t >= 2) ok = ok && wait_for(&sm.p_free[sb], ((t >> 1) - 1) & 1, p.err, ctl);
        tc_fence_after();
        tmem_st16(tmem + lane_off + kColP + sb * (kTile / 2) + part * (kPartKeys / 2), w);
        tc_wait_st();
        l += (sum_lo[0] + sum_hi[0]) + (sum_lo[1] + sum_hi[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) PAIR ? arrive_at(first_cta(&sm.p_full[sb])) : mbar_arrive(&sm.p_full[sb]);
      }
      // ---- epilogue ---------------------------------------------------------
      sm.xrow[part][row] = l;
      named_barrier(kBarQuad + quad, 128);
      const float lrow = (sm.xrow[0][row] + sm.xrow[1][row]) + (sm.xrow[2][row] + sm.xrow[3][row]);
      ok = ok && wait_for(&sm.o_full, n_item & 1, p.err, ctl);
      tc_fence_after();
      const bool gone = (bad[0] | bad[1] | bad[2] | bad[3]) != 0;
      {
        float o[32];
        tmem_ld32(tO, o);
        tc_wait_ld();
        // (ahead of the stores, for which the arrival would wait)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) PAIR ? arrive_at(first_cta(&sm.o_empty)) : mbar_arrive(&sm.o_empty);
        if (gone) {
          float x[32];  // (a copy, so that o itself stays in registers)
          #pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = o[i];
          add_bad(p, it, bad, valid ? rank * kRows + row : 0, part * kPartKeys, x);
          #pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = x[i];
        }
        if (!PAIR && valid && ok && it.slot >= 0) {
          if (part == 0)
            *reinterpret_cast<float2*>(p.piece_ml + ((long long)it.slot * kRows + row) * 2) = make_float2(m, lrow);
          float* dst = p.piece_o + ((long long)it.slot * kRows + row) * kValDim + part * kPartKeys;
          #pragma unroll
          for (int i = 0; i < 32; i += 8) {
            uint32_t r[8];
            #pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(o[i + k]);
            store32(dst + i, r);
          }
        } else if (valid && ok) {
          const float inv = reciprocal(lrow);
          __nv_bfloat16* dst =
              p.out + ((long long)(it.row0 + row) * p.num_heads + it.head) * kValDim + part * kPartKeys;
          #pragma unroll
          for (int i = 0; i < 32; i += 16) {
            uint32_t r[8];
            #pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = pack_bf16(o[i + 2 * k] * inv, o[i + 2 * k + 1] * inv);
            if (p.wide) {
              store32(dst + i, r);
            } else {
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(r[0], r[1], r[2], r[3]);
              *reinterpret_cast<uint4*>(dst + i + 8) = make_uint4(r[4], r[5], r[6], r[7]);
            }
          }
        }
      }
    }
  }
  // (an abort only shortens the loops: every warp gets here)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (PAIR) {
    cluster_barrier();  // nothing of either CTA is under way in the other
    if (warp == kWarpS) tmem_dealloc_pair(tmem, kTmemCols);
    cluster_barrier();
  } else if (warp == kWarpS) {
    tmem_dealloc(tmem, kTmemCols);
  }
  // The last CTA to finish empties the queue for the next launch, and says how many
  // pieces the joining kernel has to look at: all, or none once a CTA gave up on a wait
  // (counted from bit 32 on), for then pieces may be left whose records and states are
  // not of this call.
  if (tid == 0 && rank == 0) {
    __threadfence();
    const unsigned long long mine = 1ull + (sm.wait.abort ? 1ull << 32 : 0);
    const unsigned long long all = atomicAdd(p.sched + 1, mine) + mine;
    if ((unsigned)all == (unsigned)active) {
      if (p.max_pieces > 0 && all >> 32 == 0) *p.num_pieces = sm.pieces;
      p.sched[0] = 0;
      p.sched[1] = 0;
      __threadfence();
    }
  }
}

// Joins the pieces of split items.  Block (b, y): the item whose first piece is
// number b, if any; a warp a row, four dims a lane.
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(32 * kMergeWarps) latent_prefill_merge_kernel(const LatentPrefillParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int4 rec = *reinterpret_cast<const int4*>(p.piece + 4 * blockIdx.x);  // pieces, row0, nt, head
  if ((int)blockIdx.x >= *p.num_pieces || rec.x == 0 || row >= rec.z) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll 4
  for (int i = 0; i < rec.x; ++i) {
    const long long at = (long long)(blockIdx.x + i) * kRows + row;
    const float2 ml = *reinterpret_cast<const float2*>(p.piece_ml + at * 2);
    const float4 v = reinterpret_cast<const float4*>(p.piece_o + at * kValDim)[lane];
    const float top = fmaxf(m, ml.x);
    const float a = m == -INFINITY ? 0.f : fast_exp2(m - top);
    const float b = ml.x == -INFINITY && ml.y == 0.f ? 0.f : fast_exp2(ml.x - top);
    l = l * a + ml.y * b;
    o.x = o.x * a + v.x * b;
    o.y = o.y * a + v.y * b;
    o.z = o.z * a + v.z * b;
    o.w = o.w * a + v.w * b;
    m = top;
  }
  const float inv = 1.f / l;
  uint2 w;
  w.x = pack_bf16(o.x * inv, o.y * inv);
  w.y = pack_bf16(o.z * inv, o.w * inv);
  reinterpret_cast<uint2*>(p.out + ((long long)(rec.y + row) * p.num_heads + rec.w) * kValDim)[lane] = w;
}

template <bool PAIR>
cudaError_t launch_prefill(const LatentPrefillLaunch& L, cudaStream_t stream) {
  const size_t smem = sizeof(Smem);
  static unsigned long long configured = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(latent_prefill_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&configured, bit, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(PAIR ? L.grid / 2 * 2 : L.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = L.p.pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, latent_prefill_kernel<PAIR>, L.qmap, L.kvmap, L.kmap, L.rmap, L.p);
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillLaunch& L, cudaStream_t stream) {
  cudaError_t e = L.pairs ? launch_prefill<true>(L, stream) : launch_prefill<false>(L, stream);
  if (e == cudaSuccess && L.p.max_pieces > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.p.max_pieces, kRows / kMergeWarps);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.p.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, latent_prefill_merge_kernel, L.p);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace pkv
