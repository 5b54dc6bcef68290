// pkv_latent_decode.cu -- attention over a paged cache of latents, absorbed
// form, on tcgen05 tensor cores.
//
// A cached row is one token's 512-dim latent c and 64-dim rotated key k,
// shared by all query heads; the queries took the key expansion into them, so
// a row (token, head) has 576 dims:
//
//   s_j = scale (<q[0:512], c_j> + <q[512:576], k_j>),  out = sum_j softmax(s)_j c_j
//
// The values are the first 512 dims of the keys: a tile that came in for the
// scores is there for the products too, and a key costs 1152 bytes of HBM and
// 2176 flops a head.  Up to 64 heads that is bound by HBM; 128 heads bring the
// tensor core near its own bound.  Measured: 8 rows of 32768 keys, 16 heads, 65 us
// (4.7 TB/s); 64 rows of 4096 keys, 128 heads, 100 us (730 TFLOP/s, 3.2 TB/s); four
// rows of up to 128 keys, 16 heads, 7.7 us.
//
// Tiling.  A work item is a request's `group_tokens` query tokens times
// `group_heads` heads: its (token, head) pairs are the N <= 64 columns of the
// MMAs, so that few heads cost little.  A tile is 64 keys = 4 pool blocks, nine
// 64-dim chunks of [64 keys][128 bytes], fetched block by block with 2-D TMA
// copies (128-byte swizzle).  S^T[64 keys x N] = K Q^T accumulates over the
// chunks; O^T[512 dims x N] += C^T P is four M = 128 tiles whose A operand is
// the same chunks read MN-major.  O^T takes 256 TMEM columns, S^T two buffers
// of 64.  The other way round (rows as M) O would need all 512 columns.
// Shared memory holds Q (72 KB), two tiles (144 KB) and P (8 KB), all there is (three
// tiles of 48 keys, which up to 48 columns leave room for, were no faster anywhere: 8 x
// 32768 keys, 16 heads 66.6 us for 65.1).  A tile is therefore loaded and released in
// five parts (the rotated keys, four pairs of latent chunks), each going back as soon
// as its last MMA is done, so that copies stay in flight while the other tile is
// worked on.
//
// Roles (608 threads).  Sixteen softmax warps: warpgroup g has columns 16 g ..
// 16 g + 15, its four warps 16 keys each (an M = 64 accumulator lies in 16 of
// every 32 TMEM lanes; the 16x256b load spreads it over all lanes, two keys by
// four columns a thread).  The running maximum moves only when a score exceeds
// it by 2^8, on a vote of the warpgroup; then the warps agree on it through
// shared memory and O^T is rescaled.  Warp 16 walks the CTA's work and issues
// the copies, warp 17 the MMAs of S^T, warp 18 those of O^T: neither waits for
// the other, so that a tile goes back to the copies as soon as its own P is
// there (one warp that issued S(t + 1) before PV(t) held every slot until the
// next tile had landed: 106 us where two warps took 83, 8 x 32768 keys, 16 heads).
//
// Work split.  The items' keys (plus a fixed cost an item) form one sequence
// that is cut in equal ranges, one a CTA -- or, with more than 64 heads, one for
// two neighbours that read the same keys for half of the heads each.  Rows cut
// by a range end leave unnormalised partial states, which latent_merge_kernel
// joins; it needs no counters, so the workspace holds no state between calls.
#include <climits>

#include "pkv_latent.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kSoftWarps = 16;
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kWarpLoad = kSoftWarps;
constexpr int kWarpS = kSoftWarps + 1;   // MMAs of the scores
constexpr int kWarpO = kSoftWarps + 2;   // MMAs of the outputs
constexpr int kThreads = 32 * (kSoftWarps + 3);
constexpr int kBarSoft = 1;   // all softmax warps
constexpr int kBarGroup = 2;  // + warpgroup

constexpr int kChunks = kLatRow / 64;     // 64-dim chunks of a row
constexpr int kParts = 5;                 // release units of a tile: four latent pairs, rotated keys
constexpr int kItems = 4;
constexpr int kTile = 64;                 // keys of a tile
constexpr int kTileBlocks = kTile / kBlockSize;
constexpr int kWindow = 32 / kTileBlocks; // tiles of a load of block ids
constexpr int kStages = 2;
constexpr int kChunkBytes = kTile * 128;  // 64 dims of a tile's keys, or of 64 columns' queries
static_assert(kTile == kLatMaxRows, "chunks of keys and of queries are alike");
constexpr uint32_t kTmemCols = 512;
constexpr int kColO = 2 * kLatMaxRows;    // TMEM: S^T buffers, then O^T
constexpr float kRescaleLog2 = 8.0f;

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// A piece of a work item: key tiles t0 .. t1 - 1 of its keys.
struct Item {
  int req;      // block-table row
  int row0;     // first query row
  int nt;       // query tokens
  int pos0;     // position of the first (it sees keys 0 .. pos0)
  int vis;      // keys that the last one sees
  int t0, t1;
  int end;      // no more items
};

// Flags of a piece's record (besides its rows).
constexpr int kPieceFirst = 1;  // holds the item's first tile
constexpr int kPieceLast = 2;   // holds its last

// --------------------------------------------------------------------- plan
struct Req {
  int q0, qr, L;
  int ng;  // token groups (0: nothing to do)
};

// (ng < 0: the fields do not fit together or the step)
__device__ __forceinline__ Req make_req(const LatentDecodeParams& p, int q0, int q1, int L) {
  Req a{q0, q1 - q0, L, 0};
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.num_q_tokens && a.qr <= L &&
                  L <= p.max_blocks * kBlockSize;
  if (!ok) a.ng = -1;
  else if (a.qr > 0) a.ng = p.group_tokens == 1 ? a.qr : cdiv(a.qr, p.group_tokens);
  return a;
}

__device__ __forceinline__ Req load_req(const LatentDecodeParams& p, int r) {
  return make_req(p, __ldg(p.qsl + r), __ldg(p.qsl + r + 1), __ldg(p.seq_lens + r));
}

// The CTA's part of the plan: its range of units, the request that it starts in and
// the units before that.
struct Plan {
  long long part[32];
  int part_count[32];
  long long range_lo, range_hi, start_base;
  Req start;
  int start_req, piece;
};

struct __align__(1024) Smem {
  uint8_t q[kChunks][kChunkBytes];
  uint8_t kv[kStages][kChunks][kChunkBytes];
  uint8_t p[kLatMaxRows * 128];  // P^T: [column][64 keys] bf16, 128-byte swizzle
  uint64_t kv_full[kStages][kParts], kv_empty[kStages][kParts];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full, p_free, o_full, o_empty;
  uint64_t item_full[kItems];
  uint64_t drained[2];
  Item items[kItems];
  union {
    Plan plan;                  // until the softmax begins
    struct {
      float xrow[4][kLatMaxRows];  // a warpgroup's exchange of maxima and sums
      float top[kLatMaxRows];      // the columns' maxima
    };
  };
  unsigned long long bad[2];    // boundary keys taken out of the item's tiles, by item parity
  uint32_t tmem_base;
  WaitCtl wait;
};
static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "latent decode shared memory");

// Part i's chunks: 2 i and 2 i + 1, of the last part the one with the rotated keys.
__host__ __device__ constexpr int part_chunks(int part) { return part == kParts - 1 ? 1 : 2; }

// The unit that the work is cut in.  Many items: keys, and item_cost more an item;
// every CTA takes an equal range, whatever items it holds.  Few (`piece` > 0):
// pieces of at most so many keys, an item's of equal length, one a CTA.
//
// Units of token groups 0 .. i - 1, i <= ng: group m sees L - qr + min((m + 1)
// group_tokens, qr) keys.
__device__ __forceinline__ int group_keys(const LatentDecodeParams& p, const Req& a, int m) {
  return a.L - a.qr + min((m + 1) * p.group_tokens, a.qr);
}

__device__ __forceinline__ long long groups_keys(const LatentDecodeParams& p, const Req& a, int i) {
  if (i <= 0) return 0;
  if (a.ng == 1) return a.L;
  const long long n = i;
  long long w = n * ((long long)a.L - a.qr) + (long long)p.group_tokens * (n * (n + 1) / 2);
  if (i == a.ng) w -= (long long)a.ng * p.group_tokens - a.qr;
  return w;
}

__device__ __forceinline__ long long groups_units(const LatentDecodeParams& p, const Req& a, int i, int piece) {
  if (i <= 0) return 0;
  if (piece == 0) return groups_keys(p, a, i) + (long long)i * p.item_cost;
  if (a.ng == 1) return (a.L - 1) / piece + 1;
  long long w = 0;
  #pragma unroll 1
  for (int m = 0; m < i; ++m) w += (group_keys(p, a, m) - 1) / piece + 1;
  return w;
}

// Over THREADS threads (a warp, or the block): the sum of `mine` over those before
// this one, and the sums of it and of `count` over all.
template <int THREADS>
__device__ __forceinline__ long long scan(Plan& pl, long long mine, int count, long long* total, int* counts) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = mine;
  #pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  count = __reduce_add_sync(0xffffffffu, count);
  if (THREADS == 32) {
    *total = __shfl_sync(0xffffffffu, incl, 31);
    *counts = count;
    return incl - mine;
  }
  if (lane == 31) {
    pl.part[warp] = incl;
    pl.part_count[warp] = count;
  }
  __syncthreads();
  const bool in = lane < THREADS / 32;
  long long all = in ? pl.part[lane] : 0, before = lane < warp ? all : 0;
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  *total = all;
  *counts = __reduce_add_sync(0xffffffffu, in ? pl.part_count[lane] : 0);
  return before + incl - mine;
}

// a / b for a >= 0, b > 0: in 32 bits whenever both fit.
__device__ __forceinline__ long long div_ll(long long a, long long b) {
  if ((unsigned long long)(a | b) <= 0xffffffffull) return (unsigned)a / (unsigned)b;
  return a / b;
}

// Unit `unit` of `units` CTAs' (or, with two head groups, neighbours') share.
// THREADS threads with up to PER requests each in registers: one warp for steps of up
// to kWarpReqs requests, beside which the rest of the CTA is set up, else the block
// (which then needs a __syncthreads before it reads the result), PER = 0: any number,
// read again.
constexpr int kWarpPer = 4;
constexpr int kWarpReqs = 32 * kWarpPer;

template <int THREADS, int PER>
static __device__ __noinline__ void plan_range(const LatentDecodeParams& p, Plan& pl, int unit, int units, int tile) {
  const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int per = cdiv(p.num_reqs, THREADS);
  const int r0 = min(tid * per, p.num_reqs), r1 = min(r0 + per, p.num_reqs);
  Req held[PER > 0 ? PER : 1];
  // f(request, its number) of this thread's requests, until it returns false.
  auto each = [&](auto f) {
    if constexpr (PER > 0) {
      #pragma unroll
      for (int i = 0; i < PER; ++i)
        if (r0 + i < r1 && !f(held[i], r0 + i)) break;
    } else {
      #pragma unroll 1
      for (int r = r0; r < r1; ++r)
        if (!f(load_req(p, r), r)) break;
    }
  };
  if constexpr (PER > 0) {
    int f[PER + 1], n[PER];
    #pragma unroll
    for (int i = 0; i <= PER; ++i) f[i] = r0 + i <= p.num_reqs ? __ldg(p.qsl + r0 + i) : 0;
    #pragma unroll
    for (int i = 0; i < PER; ++i) n[i] = r0 + i < p.num_reqs ? __ldg(p.seq_lens + r0 + i) : 0;
    #pragma unroll
    for (int i = 0; i < PER; ++i) held[i] = make_req(p, f[i], f[i + 1], n[i]);
  }
  long long keys = 0;
  int items = 0;
  each([&](const Req& a, int) {
    if (a.ng < 0 && blockIdx.x == 0) record_error(p.err, kErrBounds);  // the request is skipped
    keys += groups_keys(p, a, a.ng);
    items += max(a.ng, 0);
    return true;
  });
  int piece = INT_MAX, all_items;
  long long total, mine = items, excl, lo, hi;
  if (p.merge) {
    mine = keys + (long long)items * p.item_cost;
    excl = scan<THREADS>(pl, mine, items, &total, &all_items);
    piece = 0;
    if (3ll * all_items <= 2 * units) {
      // ceil(keys / piece) summed over the items is at most their keys / piece + all_items.
      const long long all_keys = total - (long long)all_items * p.item_cost, room = units - all_items;
      auto whole_tiles = [&](long long k) {
        return (int)min(max((k + tile - 1) / tile * tile, (long long)p.min_keys), 1ll << 30);
      };
      auto count = [&]() {
        mine = 0;
        each([&](const Req& a, int) {
          mine += groups_units(p, a, a.ng, piece);
          return true;
        });
      };
      const int most = whole_tiles(div_ll(all_keys + room - 1, room));
      piece = most;
      if (PER > 0) {
        // Often a shorter one does: the shortest of eight steps that leaves no CTA two.
        const int least = whole_tiles(div_ll(all_keys + units - 1, units));
        const int step = max(tile, ((most - least) / 8 + tile - 1) / tile * tile);
        for (piece = least; piece < most; piece += step) {
          count();
          if (__reduce_add_sync(0xffffffffu, (int)mine) <= units) break;
        }
        piece = min(piece, most);
      }
      count();
      if (THREADS > 32) __syncthreads();  // pl.part is free again
    }
  }
  if (piece > 0) {
    excl = scan<THREADS>(pl, mine, 0, &total, &all_items);
    lo = min((long long)unit, total);
    hi = min(lo + 1, total);
  } else {
    const long long chunk = max(div_ll(total + units - 1, units), (long long)p.min_keys);
    lo = min(unit * chunk, total);
    hi = min(lo + chunk, total);
  }
  if (tid == 0) {
    pl.range_lo = lo;
    pl.range_hi = hi;
    pl.piece = piece;
  }
  if (lo < hi && excl <= lo && lo < excl + mine) {
    long long base = excl;
    each([&](const Req& a, int r) {
      const long long w = groups_units(p, a, a.ng, piece);
      if (lo >= base + w) {
        base += w;
        return true;
      }
      pl.start_req = r;
      pl.start = a;
      pl.start_base = base;
      return false;
    });
  }
}

// --------------------------------------------------------------- TMEM, smem
// Two 8-column groups of 16 accumulator rows (TMEM lanes base .. base + 15):
// v[4 c + 2 h + e] is row lane / 4 + 8 h, column 8 c + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, float (&v)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st16f(uint32_t taddr, const float (&v)[16]) {
  tmem_st16(taddr, reinterpret_cast<const uint32_t(&)[16]>(v));
}

// Four 8x8 matrices of 16-bit elements, each stored transposed: lane i gives
// the address of row i % 8 of matrix i / 8 as it is to lie in memory.
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Address of 16-byte piece `piece` (0 .. 63) of key row `row`'s latent in a tile.
__device__ __forceinline__ uint4* latent_piece(uint8_t (*tile)[kChunkBytes], int row, int piece) {
  return reinterpret_cast<uint4*>(tile[piece >> 3] + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ bool non_finite(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Rows of the tile that no row of the item sees (from row vis - key0 on) must
// not reach the product, whatever they hold: 0 * NaN.  Rows that only some of
// the item's tokens see (keys pos0 + 1 .. vis - 1) may hold NaN or infinities
// that the others must not get: those are taken out too and noted, and the
// epilogue gives them to the rows that see them.  Rare or at a range's last
// tiles; one warp a row, out of line.
static __device__ __noinline__ void clean_tile(uint8_t (*tile)[kChunkBytes], int key0, int pos0, int vis,
                                               unsigned long long* bad, int warp, int lane) {
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // (blocks behind the last are zeros already)
  const int end = min(kTile, (vis + kBlockSize - 1) / kBlockSize * kBlockSize - key0);
  for (int row = max(pos0 + 1 - key0, 0) + warp; row < end; row += kSoftWarps) {
    const int key = key0 + row;
    bool out = key >= vis;
    if (!out) {
      const uint4 a = *latent_piece(tile, row, lane), b = *latent_piece(tile, row, lane + 32);
      out = __any_sync(0xffffffffu, non_finite(a.x) || non_finite(a.y) || non_finite(a.z) ||
                                        non_finite(a.w) || non_finite(b.x) || non_finite(b.y) ||
                                        non_finite(b.z) || non_finite(b.w));
      if (out && lane == 0) atomicOr(bad, 1ull << (key - pos0 - 1));
    }
    if (out) {
      *latent_piece(tile, row, lane) = zero;
      *latent_piece(tile, row, lane + 32) = zero;
    }
  }
  fence_proxy_async_smem();
}

// Bit b of the result: boundary key b, taken out of the products, holds a
// non-finite value in dim d.  A row that sees such a key scored it NaN or
// infinite; only where it scored it -inf is the row not all NaN already, and
// then its weight 0 times the value is NaN in this dim.
static __device__ __noinline__ unsigned long long bad_dim(const LatentDecodeParams& p, const Item& it,
                                                          unsigned long long bad, int d) {
  unsigned long long hit = 0;
  for (unsigned long long m = bad; m; m &= m - 1) {
    const int b = __ffsll((long long)m) - 1;
    const int key = it.pos0 + 1 + b;
    const int blk = __ldg(p.block_tables + (long long)it.req * p.max_blocks + key / kBlockSize);
    if ((unsigned)blk >= (unsigned)p.num_blocks) continue;
    const uint16_t v = __ldg(reinterpret_cast<const uint16_t*>(p.pool) +
                             ((long long)blk * kBlockSize + key % kBlockSize) * kLatRow + d);
    if ((v & 0x7f80u) == 0x7f80u) hit |= 1ull << b;
  }
  return hit;
}

// O^T of a warpgroup's 16 columns, 32 dims a warp, from TMEM address ta on: column
// i times the factor that the threads of lanes 0 .. 3 hold for it (alpha[2 c + e]
// of lane q: column 8 c + 2 q + e).  x: room for 16 numbers of this warp's.
static __device__ __noinline__ void rescale_o(float* x, uint32_t ta, const float (&alpha)[4]) {
  const int lane = threadIdx.x & 31;
  if (lane < 4) {
    #pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * lane + 8 * (i >> 1) + (i & 1)] = alpha[i];
  }
  __syncwarp();
  #pragma unroll 1
  for (int mt = 0; mt < 4; ++mt, ta += kLatMaxRows) {
    float o[16];
    tmem_ld16(ta, o);
    tc_wait_ld();
    #pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= x[i];
    tmem_st16f(ta, o);
  }
  tc_wait_st();
}

// What the boundary keys that were taken out mean for the item's outputs, which
// this warp has written (16 columns from col0 on, dims 128 mt + 32 quad + lane):
// NaN where a row sees a key that is not finite in the dim.  dst: the row of
// column 0, out or a piece's.
template <class T>
static __device__ __noinline__ void spread_bad(const LatentDecodeParams& p, const Item& it,
                                               unsigned long long bad, T* dst, int col0, int cols, int quad) {
  __syncwarp();
  for (int mt = 0; mt < 4; ++mt) {
    const int d = mt * 128 + quad * 32 + (threadIdx.x & 31);
    const unsigned long long hit = bad_dim(p, it, bad, d);
    for (int col = col0; col < min(col0 + 16, cols); ++col)
      // Token tk sees boundary keys 0 .. tk - 1.
      if (hit & ((1ull << (col / p.group_heads)) - 1)) dst[(long long)col * kLatent + d] = T(NAN);
  }
}

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// TWO: two groups of heads.
template <bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap, const LatentDecodeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  constexpr int kStep = kChunkBytes >> 4;  // a chunk in the unit of the MMA's descriptors
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + (((raw + 1023u) & ~1023u) - raw));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  WaitCtl* ctl = &sm.wait;
  // CTA b of two: head group b % 2 of range b / 2.
  const int hg = TWO ? blockIdx.x & 1 : 0;
  const int head0 = hg * p.group_heads;
  const int heads = min(p.group_heads, p.num_q_heads - head0);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s)
      for (int i = 0; i < kParts; ++i) {
        mbar_init(&sm.kv_full[s][i], 1);
        mbar_init(&sm.kv_empty[s][i], 1);
      }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.s_full[0], 1);
    mbar_init(&sm.s_full[1], 1);
    mbar_init(&sm.p_full, kSoftWarps);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kSoftWarps);
    for (int i = 0; i < kItems; ++i) mbar_init(&sm.item_full[i], 1);
    mbar_init(&sm.drained[0], 1);
    mbar_init(&sm.drained[1], 1);
    sm.wait.abort = 0;
    sm.wait.limit_ns = p.wait_limit_ns;
    sm.bad[0] = sm.bad[1] = 0;
    fence_barrier_init();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
  }
  if (warp == kWarpS) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  const int unit = TWO ? blockIdx.x >> 1 : blockIdx.x, units = TWO ? gridDim.x >> 1 : gridDim.x;
  if (p.num_reqs <= kWarpReqs) {
    if (warp == kWarpLoad) {
      if (!p.early_plan) grid_dependency_wait();
      plan_range<32, kWarpPer>(p, sm.plan, unit, units, kTile);
    }
  } else {
    if (!p.early_plan) grid_dependency_wait();
    plan_range<kThreads, 0>(p, sm.plan, unit, units, kTile);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem_base);
  const Plan& pl = sm.plan;
  const long long lo = pl.range_lo, hi = pl.range_hi, start_base = pl.start_base;
  const int piece = pl.piece, start_req = pl.start_req;
  const Req start = pl.start;
  // The plan's room is the softmax warps' from here on.
  __syncthreads();
  // (the warp that copies works out its first item before it waits)
  if (warp != kWarpLoad || lo >= hi) {
    grid_dependency_wait();
    allow_dependent_launch();
  }
  // This CTA's piece records, written again by the pieces that it cuts.
  if (p.merge && tid == 0) {
    p.piece[2 * blockIdx.x * kPieceWords] = 0;
    p.piece[(2 * blockIdx.x + 1) * kPieceWords] = 0;
  }

  // Columns of the MMAs.
  const int n_cols = ((p.group_heads * p.group_tokens + 15) / 16) * 16;
  if (lo >= hi) {
    // no work
  } else if (warp == kWarpLoad) {
    // =========================== copies ===================================
    // One thread issues all copies, from uniform registers (a thread a copy, eight
    // at a time, took 1.76 us a tile of 36).
    const bool leader = elect_one();
    int n_item = 0, t = 0;     // items and tiles so far
    int st = 0, phase = 1;     // the tile's stage and the parity that it waits for (the first ones pass)
    int parts = 0;             // parts of tile t that were issued
    bool ok = true;
    int r = start_req;
    long long base = start_base;
    const int oob_row = p.num_blocks * kBlockSize;
    const uint32_t q_bytes = (uint32_t)(kChunks * 128) * p.group_heads * p.group_tokens;
    Req a = start;
    // The next request's raw fields, ahead of its turn.
    int f0 = a.q0 + a.qr, f1 = 0, fl = 0;
    while (ok && base < hi && r < p.num_reqs) {
      if (r + 1 < p.num_reqs) {
        f1 = __ldg(p.qsl + r + 2);
        fl = __ldg(p.seq_lens + r + 1);
      }
      const long long w = groups_units(p, a, a.ng, piece);
      // First token group that the range reaches.
      int g = 0;
      if (base < lo) {
        int top = a.ng;  // groups_units(g) <= lo - base < groups_units(top)
        while (top - g > 1) {
          const int mid = (g + top) >> 1;
          if (groups_units(p, a, mid, piece) <= lo - base) g = mid;
          else top = mid;
        }
      }
      const int32_t* bt = p.block_tables + (long long)r * p.max_blocks;
      for (; g < a.ng && ok; ++g) {
        const long long gbase = g > 0 ? base + groups_units(p, a, g, piece) : base;
        if (gbase >= hi) break;
        Item it;
        it.req = r;
        it.row0 = a.q0 + g * p.group_tokens;
        it.nt = min(p.group_tokens, a.qr - g * p.group_tokens);
        it.pos0 = a.L - a.qr + g * p.group_tokens;
        it.vis = it.pos0 + it.nt;
        const int tiles = cdiv(it.vis, kTile);
        it.t0 = 0;
        it.t1 = tiles;
        if (piece > 0) {
          // Piece lo - gbase of n.
          const int n = (it.vis - 1) / piece + 1, x = (int)(lo - gbase);
          if (n > 1) {
            it.t0 = (int)((long long)tiles * x / n);
            it.t1 = (int)((long long)tiles * (x + 1) / n);
          }
        } else {
          // Tile j belongs to the range that holds unit gbase + kTile j.
          if (gbase < lo) it.t0 = (int)((lo - gbase + kTile - 1) / kTile);
          if (hi - gbase < it.vis) it.t1 = (int)((hi - gbase + kTile - 1) / kTile);
        }
        it.end = 0;
        if (it.t0 >= it.t1) continue;
        const int nbl = cdiv(it.vis, kBlockSize);
        // Block ids, a window of tiles at a time, a lane each; they become rows of the
        // pool when their window begins.  Blocks past the last are read at a row
        // outside the pool, which fills zeros.
        auto ids = [&](int tile) {
          const int x = tile * kTileBlocks + lane;
          return x < nbl && lane < kWindow * kTileBlocks ? __ldg(bt + x) : INT_MIN;
        };
        auto row_of = [&](int id) {
          if ((unsigned)id < (unsigned)p.num_blocks) return id * kBlockSize;
          if (id != INT_MIN) record_error(p.err, kErrBounds);
          return oob_row;
        };
        if (n_item == 0) {
          grid_dependency_wait();
          allow_dependent_launch();
        }
        int nxt = ids(it.t0), cur = 0;
        // The item and its queries, ahead of its first keys.
        if (n_item > 0) ok = all_of(wait_for(&sm.q_empty, (n_item - 1) & 1, p.err, ctl));
        if (!ok) break;
        if (leader) {
          sm.items[n_item % kItems] = it;
          mbar_arrive(&sm.item_full[n_item % kItems]);
          mbar_arrive_expect_tx(&sm.q_full, q_bytes);
          #pragma unroll 1
          for (int c = p.debug_withhold_q ? kChunks : 0; c < kChunks; ++c)
            tma_load_3d(sm.q[c], &qmap, c * 64, head0, it.row0, &sm.q_full);
        }
        __syncwarp();
        ++n_item;
        int k = 0;  // lane of the tile's first block
        int j = uniform(it.t0);
        const int j1 = uniform(it.t1);
        #pragma unroll 1
        for (; j < j1; ++j) {
          if (k == 0) {
            cur = row_of(nxt);
            if (j + kWindow < j1) nxt = ids(j + kWindow);
          }
          // Of two neighbours each brings half of the tile after next into L2, while one
          // tile is in flight and the other worked on (64 rows of 4096 keys, 128 heads: 100
          // us for 108 without; 64 of 2048, 96 heads 57 for 61; one group alone, 8 of 32768,
          // 16 heads, gains nothing: 66.8 for 65.1).
          int ahead[kTileBlocks];
          if (TWO) {
            const int far = row_of(nxt);
            #pragma unroll
            for (int b = 0; b < kTileBlocks; ++b) {
              const int l = k + 2 * kTileBlocks + b;
              const int here = __shfl_sync(0xffffffffu, cur, l);
              const int there = __shfl_sync(0xffffffffu, far, l - kWindow * kTileBlocks);
              ahead[b] = uniform(l < kWindow * kTileBlocks ? here : there);
            }
          }
          int rows[kTileBlocks];
          #pragma unroll
          for (int b = 0; b < kTileBlocks; ++b) rows[b] = uniform(__shfl_sync(0xffffffffu, cur, k + b));
          k += kTileBlocks;
          if (k == kWindow * kTileBlocks) k = 0;
          #pragma unroll
          for (int part = 0; part < kParts; ++part) {
            ok = all_of(wait_for(&sm.kv_empty[st][part], phase, p.err, ctl));
            if (!ok) break;
            if (leader) {
              uint64_t* const bar = &sm.kv_full[st][part];
              mbar_arrive_expect_tx(bar, (uint32_t)part_chunks(part) * kTile * 128);
              #pragma unroll
              for (int i = 0; i < part_chunks(part); ++i) {
                const int c = 2 * part + i;
                #pragma unroll
                for (int b = 0; b < kTileBlocks; ++b)
                  tma_load_2d(sm.kv[st][c] + b * 2048, &kmap, c * 64, rows[b], bar);
              }
            }
            __syncwarp();
            parts = part + 1;
          }
          if (!ok) break;
          if (TWO && leader && j + 2 < j1) {
            #pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              #pragma unroll
              for (int b = 0; b < kTileBlocks; ++b)
                if (((c * kTileBlocks + b) & 1) == hg) tma_prefetch_2d(&kmap, c * 64, ahead[b]);
            }
          }
          __syncwarp();
          parts = 0;
          ++t;
          if (++st == kStages) st = 0, phase ^= 1;
        }
      }
      base += w;
      ++r;
      a = make_req(p, f0, f1, fl);
      f0 = f1;
    }
    // End marker, for the MMA warp (behind its last item) and the softmax warps.
    if (ok && n_item > 0) ok = wait_for(&sm.q_empty, (n_item - 1) & 1, p.err, ctl);
    if (ok && lane == 0) {
      sm.items[n_item % kItems].end = 1;
      mbar_arrive(&sm.item_full[n_item % kItems]);
      mbar_arrive(&sm.q_full);
    }
    __syncwarp();
    if (!ok) {
      // Aborted: the copies in flight must land before the CTA ends.
      #pragma unroll 1
      for (int part = 0; part < kParts; ++part) {
        const int n = t + (part < parts ? 1 : 0);  // tiles whose part was issued
        for (int i = max(0, n - kStages); i < n; ++i)
          drain(&sm.kv_full[i % kStages][part], (i / kStages) & 1, p.err, ctl);
      }
      if (n_item > 0) drain(&sm.q_full, (n_item - 1) & 1, p.err, ctl);
    }
  } else if (warp == kWarpS) {
    // ========================= MMAs of the scores =========================
    // As soon as a tile's chunks land.  Its scores go to the buffer of the tile two
    // before, which had the same place in shared memory: its latents went back behind its
    // P, for which the softmax had read the scores.
    const uint32_t idesc = idesc_bf16_f32(kTile, n_cols, 0, 0);
    const uint64_t desc_k = smem_desc_sw128(smem_u32(sm.kv[0][0]), 16, 1024);
    const uint64_t desc_q = smem_desc_sw128(smem_u32(sm.q[0]), 16, 1024);
    const bool leader = elect_one();
    bool ok = true;
    int st = 0, phase = 0;
    for (int n_item = 0;; ++n_item) {
      ok = all_of(wait_for(&sm.q_full, n_item & 1, p.err, ctl));
      if (!ok) break;
      const Item& it = sm.items[n_item % kItems];
      if (uniform(it.end)) break;
      #pragma unroll 1
      for (int left = uniform(it.t1 - it.t0); left > 0; --left) {
        const uint64_t da = desc_k + (uint64_t)(st * (kChunks * kStep));
        #pragma unroll
        for (int part = 0; part < kParts; ++part) {
          ok = all_of(wait_for(&sm.kv_full[st][part], phase, p.err, ctl));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            #pragma unroll
            for (int kk = 0; kk < (part == kParts - 1 ? 4 : 8); ++kk) {
              const int c = 2 * part + (kk >> 2);
              tc_mma_f16_ss(tmem + st * kLatMaxRows, da + (c * kStep + 2 * (kk & 3)),
                            desc_q + (c * kStep + 2 * (kk & 3)), idesc, part > 0 || kk > 0);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) {
          tc_commit(&sm.s_full[st]);
          tc_commit(&sm.kv_empty[st][kParts - 1]);
          if (left == 1) tc_commit(&sm.q_empty);
        }
        __syncwarp();
        if (++st == kStages) st = 0, phase ^= 1;
      }
      if (!ok) break;
    }
    if (!ok) {
      // Aborted: the issued MMAs must end before TMEM is freed.
      if (leader) tc_commit(&sm.drained[0]);
      __syncwarp();
      drain(&sm.drained[0], 0, p.err, ctl);
    }
  } else if (warp == kWarpO) {
    // ========================= MMAs of the outputs ========================
    const uint32_t idesc = idesc_bf16_f32(128, n_cols, 1, 0);
    // C^T: MN-major atoms of 64 dims x 8 keys, the chunks kTile * 128 bytes apart.
    const uint64_t desc_v = smem_desc_sw128(smem_u32(sm.kv[0][0]), kTile * 128, 1024);
    const uint64_t desc_p = smem_desc_sw128(smem_u32(sm.p), 16, 1024);
    const bool leader = elect_one();
    bool ok = true;
    int st = 0, phase = 0, p_phase = 0;
    for (int n_item = 0;; ++n_item) {
      ok = all_of(wait_for(&sm.item_full[n_item % kItems], (n_item / kItems) & 1, p.err, ctl));
      if (!ok) break;
      const Item& it = sm.items[n_item % kItems];
      if (uniform(it.end)) break;
      const int n = uniform(it.t1 - it.t0);
      #pragma unroll 1
      for (int j = 0; j < n; ++j) {
        // The tile landed long since, the scores came from it.
        #pragma unroll 1
        for (int m = 0; m < 4; ++m) ok = ok && wait_for(&sm.kv_full[st][m], phase, p.err, ctl);
        ok = ok && wait_for(&sm.p_full, p_phase, p.err, ctl);
        if (j == 0 && n_item > 0) ok = ok && wait_for(&sm.o_empty, (n_item - 1) & 1, p.err, ctl);
        ok = all_of(ok);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t da = desc_v + (uint64_t)(st * (kChunks * kStep));
          #pragma unroll
          for (int m = 0; m < 4; ++m) {
            #pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              tc_mma_f16_ss(tmem + kColO + m * kLatMaxRows, da + (2 * m * kStep + kk * (2048 >> 4)),
                            desc_p + 2 * kk, idesc, j > 0 || kk > 0);
            tc_commit(&sm.kv_empty[st][m]);
          }
          tc_commit(&sm.p_free);
          if (j == n - 1) tc_commit(&sm.o_full);
        }
        __syncwarp();
        p_phase ^= 1;
        if (++st == kStages) st = 0, phase ^= 1;
      }
      if (!ok) break;
    }
    if (!ok) {
      // Aborted: the issued MMAs must end before TMEM is freed.
      if (leader) tc_commit(&sm.drained[1]);
      __syncwarp();
      drain(&sm.drained[1], 0, p.err, ctl);
    }
  } else {
    // ==================== softmax and epilogue (warps 0-15) ==================
    const int wg = warp >> 2, quad = warp & 3;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int rows = p.group_heads * p.group_tokens;
    const bool mine = wg * 16 < rows;
    // This thread's columns 16 wg + 8 c + 2 (lane % 4) + e, its keys' places
    // 16 quad + lane / 4 + 8 h.
    const int col0 = wg * 16 + 2 * (lane & 3);
    const int key_lo = quad * 16 + (lane >> 2);
    int tok[4];  // query token of each column; -1: none
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = col0 + 8 * (i >> 1) + (i & 1);
      tok[i] = col < rows && col % p.group_heads < heads ? col / p.group_heads : -1;
    }
    // P^T: this warp's stmatrix rows -- matrix 2 c + h holds columns 8 c .., keys
    // 16 quad + 8 h ..
    const int st_col = wg * 16 + ((lane >> 4) & 1) * 8 + (lane & 7);
    const int st_piece = quad * 2 + ((lane >> 3) & 1);
    const uint32_t st_addr = smem_u32(sm.p) + st_col * 128 + ((st_piece ^ (st_col & 7)) << 4);
    bool ok = true;
    int t = 0;
    for (int n_item = 0;; ++n_item) {
      const bool have = wait_for(&sm.item_full[n_item % kItems], (n_item / kItems) & 1, p.err, ctl);
      const Item it = sm.items[n_item % kItems];
      // Agree before any barrier: a wait that gave up stops everyone.
      if (barrier_or(kBarSoft, kSoftThreads, !have || it.end)) break;
      unsigned long long* bad = &sm.bad[n_item & 1];
      int limit[4];  // the last key that each column sees
      #pragma unroll
      for (int i = 0; i < 4; ++i) limit[i] = tok[i] >= 0 && tok[i] < it.nt ? it.pos0 + tok[i] : -1;
      float m[4], l[4];
      #pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
      for (int j = it.t0; j < it.t1; ++j, ++t) {
        const int key0 = j * kTile;
        ok = ok && wait_for(&sm.s_full[t & 1], (t >> 1) & 1, p.err, ctl);
        tc_fence_after();
        uint32_t w[4];
        if (mine) {
          float v[8];
          tmem_ld_16x16(tmem + lane_off + (t & 1) * kLatMaxRows + wg * 16, v);
          tc_wait_ld();
          float mx[4];
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            // v: column i = 2 c + e at 4 c + e (first key) and 4 c + 2 + e.
            float& a = v[4 * (i >> 1) + (i & 1)];
            float& b = v[4 * (i >> 1) + 2 + (i & 1)];
            a *= p.scale_log2;
            b *= p.scale_log2;
            if (key0 + key_lo > limit[i]) a = -INFINITY;
            if (key0 + key_lo + 8 > limit[i]) b = -INFINITY;
            mx[i] = fmaxf(a, b);
          }
          bool grow = j == it.t0;
          #pragma unroll
          for (int i = 0; i < 4; ++i) grow = grow || mx[i] > m[i] + kRescaleLog2;
          if (barrier_or(kBarGroup + wg, 128, grow)) {
            // The warpgroup's maxima of this tile.
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              #pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
            }
            if (lane < 4) {
              #pragma unroll
              for (int i = 0; i < 4; ++i) sm.xrow[quad][col0 + 8 * (i >> 1) + (i & 1)] = mx[i];
            }
            named_barrier(kBarGroup + wg, 128);
            // New references, for all 16 columns: this thread's, and in lane i
            // < 16 the factor of column i.
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = col0 + 8 * (i >> 1) + (i & 1);
              mx[i] = fmaxf(fmaxf(sm.xrow[0][col], sm.xrow[1][col]), fmaxf(sm.xrow[2][col], sm.xrow[3][col]));
            }
            named_barrier(kBarGroup + wg, 128);
            float alpha[4];
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool up = mx[i] > m[i] + kRescaleLog2 || (m[i] == -INFINITY && mx[i] > m[i]);
              const float m_new = up ? mx[i] : m[i];
              // (nothing summed so far: any factor will do, but not NaN)
              alpha[i] = up && m[i] != -INFINITY ? fast_exp2(m[i] - m_new) : 1.f;
              m[i] = m_new;
              l[i] *= alpha[i];
            }
            if (j > it.t0) {
              // O^T must hold the tile before.
              ok = ok && wait_for(&sm.p_free, (t - 1) & 1, p.err, ctl);
              tc_fence_after();
              rescale_o(sm.xrow[quad] + wg * 16, tmem + lane_off + kColO + wg * 16, alpha);
              named_barrier(kBarGroup + wg, 128);  // sm.xrow is free again
            }
          }
          // P = exp2(s - m) in bf16; the sums add the rounded values that the
          // product uses.  A column that saw no key yet has m = -inf.
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float ref = m[i] == -INFINITY ? 0.f : m[i];
            float& a = v[4 * (i >> 1) + (i & 1)];
            float& b = v[4 * (i >> 1) + 2 + (i & 1)];
            a = fast_exp2(a - ref);
            b = fast_exp2(b - ref);
          }
          #pragma unroll
          for (int c = 0; c < 2; ++c) {
            w[2 * c] = pack_bf16(v[4 * c], v[4 * c + 1]);
            w[2 * c + 1] = pack_bf16(v[4 * c + 2], v[4 * c + 3]);
            add_bf16x2(l[2 * c], l[2 * c + 1], w[2 * c]);
            add_bf16x2(l[2 * c], l[2 * c + 1], w[2 * c + 1]);
          }
        }
        if (key0 + kTile > it.pos0 + 1) {
          // (landed long since: the scores came from them)
          #pragma unroll 1
          for (int part = 0; part < kParts - 1; ++part)
            ok = ok && wait_for(&sm.kv_full[t % kStages][part], (t / kStages) & 1, p.err, ctl);
          clean_tile(sm.kv[t % kStages], key0, it.pos0, it.vis, bad, warp, lane);
        }
        // P's buffer is free once the product before has read it.
        if (t > 0) ok = ok && wait_for(&sm.p_free, (t - 1) & 1, p.err, ctl);
        if (mine) {
          stmatrix4_trans(st_addr, w[0], w[1], w[2], w[3]);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full);
      }
      // ---- epilogue ---------------------------------------------------------
      const int n_tiles = cdiv(it.vis, kTile);
      const bool whole = it.t0 == 0 && it.t1 == n_tiles;
      const int slot = 2 * blockIdx.x + (it.t0 == 0 ? 1 : 0);
      // Columns in use: rows (token, head) of out from the first on, in order
      // (with two head groups an item has one token).
      const int cols = (it.nt - 1) * p.group_heads + heads;
      float inv = 0.f;
      if (mine) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          #pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        }
        if (lane < 4) {
          #pragma unroll
          for (int i = 0; i < 4; ++i) sm.xrow[quad][col0 + 8 * (i >> 1) + (i & 1)] = l[i];
          if (!whole && ok && quad == 0) {
            #pragma unroll
            for (int i = 0; i < 4; ++i) sm.top[col0 + 8 * (i >> 1) + (i & 1)] = m[i];
          }
        }
        named_barrier(kBarGroup + wg, 128);
        // Lane i < 16: column i's sum.
        const int col = wg * 16 + (lane & 15);
        const float sum = (sm.xrow[0][col] + sm.xrow[1][col]) + (sm.xrow[2][col] + sm.xrow[3][col]);
        inv = reciprocal(sum);
        if (!whole && ok && quad == 0 && lane < 16 && col < cols)
          *reinterpret_cast<float2*>(p.piece_ml + ((long long)slot * p.piece_rows + col) * 2) =
              make_float2(sm.top[col], sum);
      }
      // (one answer for the warp: what follows takes all of its lanes)
      ok = all_of(ok && wait_for(&sm.o_full, n_item & 1, p.err, ctl));
      tc_fence_after();
      // Boundary keys that were taken out, by any warp.
      if (it.nt > 1) named_barrier(kBarSoft, kSoftThreads);
      const unsigned long long gone = *bad;
      if (mine && ok) {
        const int n = cols - wg * 16;  // columns of this warpgroup in use (16 at most)
        __nv_bfloat16* dst = p.out + ((long long)it.row0 * p.num_q_heads + head0) * kLatent;
        float* part = p.piece_o + (long long)slot * p.piece_rows * kLatent;
        const uint32_t ta = tmem + lane_off + kColO + wg * 16;
        float scale[16];
        #pragma unroll
        for (int i = 0; i < 16; ++i) scale[i] = __shfl_sync(0xffffffffu, inv, i);
        #pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {
          const int d = mt * 128 + quad * 32 + lane;
          float o[16];
          tmem_ld16(ta + mt * kLatMaxRows, o);
          tc_wait_ld();
          if (whole) {
            // Lanes 2 k and 2 k + 1 hold dims d and d + 1 of both columns of a
            // pair: they swap, so that each stores two dims of one column.
            __nv_bfloat16* at = dst + (long long)(wg * 16 + (lane & 1)) * kLatent + (d & ~1);
            #pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float a = o[i] * scale[i], b = o[i + 1] * scale[i + 1];
              const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
              if (i + (lane & 1) < n)
                *reinterpret_cast<uint32_t*>(at + i * kLatent) = lane & 1 ? pack_bf16(other, b) : pack_bf16(a, other);
            }
          } else {
            float* at = part + (long long)(wg * 16) * kLatent + d;
            #pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i < n) at[i * kLatent] = o[i];
          }
        }
        if (gone) {
          if (whole) spread_bad(p, it, gone, dst, wg * 16, cols, quad);
          else spread_bad(p, it, gone, part, wg * 16, cols, quad);
        }
      }
      // Every warp has read sm.bad, sm.xrow; O^T goes back.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_empty);
      if (barrier_or(kBarSoft, kSoftThreads, !ok)) break;
      if (tid == 0) {
        *bad = 0;
        // The piece is there, every warp's part of it.
        if (!whole) {
          int* rec = p.piece + slot * kPieceWords;
          rec[1] = it.row0;
          rec[2] = cols;
          rec[0] = 4 | (it.t0 == 0 ? kPieceFirst : 0) | (it.t1 == n_tiles ? kPieceLast : 0);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpS) tmem_dealloc(tmem, kTmemCols);
}

// Joins the pieces of rows that were cut.  Block (b, y): eight columns of the item
// whose first piece is in CTA b's last slot, if any; its later pieces are in the
// first slots of the next CTAs of the same head group.  A warp a column; flags and
// statistics of up to 32 pieces are read at once, a lane each, and the loads of the
// outputs depend on nothing but them.
constexpr int kMergeWarps = 8;

__global__ void __launch_bounds__(32 * kMergeWarps) latent_merge_kernel(const LatentDecodeParams p, int grid) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kVecs = 4;  // of four dims, a lane
  const int row = blockIdx.y * kMergeWarps + warp;
  const int4 rec = *reinterpret_cast<const int4*>(p.piece + (2 * cta + 1) * kPieceWords);
  float m = -INFINITY, l = 0.f;
  float4 o[kVecs];
  #pragma unroll
  for (int k = 0; k < kVecs; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  bool last = false;
  for (int first = 0; !last; first += 32) {
    // Lane i: piece first + i.
    const int c = cta + (first + lane) * p.head_groups;
    const int slot = first + lane == 0 ? 2 * cta + 1 : 2 * c;
    int flags = 0;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (c < grid && row < p.piece_rows) {
      flags = p.piece[slot * kPieceWords];
      ml = *reinterpret_cast<const float2*>(p.piece_ml + ((long long)slot * p.piece_rows + row) * 2);
    }
    if (rec.x == 0 || row >= rec.z) return;  // CTA cta cut nothing that begins with it
    const unsigned ends = __ballot_sync(0xffffffffu, (flags & kPieceLast) != 0);
    // (a record that is missing, of an aborted CTA, ends the item as well)
    const unsigned holes = __ballot_sync(0xffffffffu, flags == 0);
    int n = 32;
    if (ends) n = min(n, __ffs(ends));
    if (holes) n = min(n, __ffs(holes) - 1);
    last = n < 32 || ends != 0;
    float top = lane < n ? ml.x : -INFINITY;
    #pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    top = fmaxf(top, m);
    const float keep = m == -INFINITY ? 0.f : fast_exp2(m - top);
    // (a piece of which the row saw no key weighs nothing)
    const float w = lane < n && !(ml.x == -INFINITY && ml.y == 0.f) ? fast_exp2(ml.x - top) : 0.f;
    float sum = lane < n ? ml.y * w : 0.f;
    #pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    l = l * keep + sum;
    #pragma unroll
    for (int k = 0; k < kVecs; ++k) o[k] = make_float4(o[k].x * keep, o[k].y * keep, o[k].z * keep, o[k].w * keep);
    m = top;
    #pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const int si = __shfl_sync(0xffffffffu, slot, i);
      const float4* src = reinterpret_cast<const float4*>(p.piece_o + ((long long)si * p.piece_rows + row) * kLatent);
      #pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        const float4 v = src[k * 32 + lane];
        o[k].x += v.x * wi;
        o[k].y += v.y * wi;
        o[k].z += v.z * wi;
        o[k].w += v.w * wi;
      }
    }
  }
  // (the item's columns are rows of out, in order)
  const long long out_row = (long long)rec.y * p.num_q_heads + (cta % p.head_groups) * p.group_heads + row;
  const float inv = 1.f / l;
  #pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    uint2 v;
    v.x = pack_bf16(o[k].x * inv, o[k].y * inv);
    v.y = pack_bf16(o[k].z * inv, o[k].w * inv);
    reinterpret_cast<uint2*>(p.out + out_row * kLatent)[k * 32 + lane] = v;
  }
}

// The same for few items of many pieces, which the warps of an item's own blocks alone
// took long to read (with the attention, a row of 32768 keys, 128 heads: 57 us, 33
// here; 16 rows of 2000 to 8000 keys, 32 heads 34.0 and 32.5, 8 rows of 32768 keys, 16
// heads 64.8 and 65.8).  A unit is 128 dims of a column;
// every block counts the items from the records and takes its share of the units.
// With units for less than half of the warps, two, four or eight of a block share one:
// its pieces in turn, the sums joined through shared memory.
constexpr int kFewSplit = 4;
constexpr int kFewBlocks = 4;    // an SM
constexpr int kCtaGroups = 8;    // of 32 CTAs' records

__global__ void __launch_bounds__(32 * kMergeWarps, kFewBlocks)
    latent_merge_few_kernel(const LatentDecodeParams p, int grid) {
  __shared__ float4 part[kMergeWarps][32];
  grid_dependency_wait();
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned starts[kCtaGroups];
  int items = 0;
  #pragma unroll
  for (int g = 0; g < kCtaGroups; ++g)
    starts[g] = g * 32 + lane < grid ? p.piece[(2 * (g * 32 + lane) + 1) * kPieceWords] : 0;
  #pragma unroll
  for (int g = 0; g < kCtaGroups; ++g) {
    starts[g] = __ballot_sync(0xffffffffu, starts[g] != 0);
    items += __popc(starts[g]);
  }
  const int per_item = p.piece_rows * kFewSplit, units = items * per_item, warps = gridDim.x * kMergeWarps;
  if (items == 0) return;
  int share = 1;  // warps a unit
  while (share < kMergeWarps && units * share * 2 <= warps) share *= 2;
  for (int u = (blockIdx.x * kMergeWarps + warp) / share; u < units || share > 1; u += warps / share) {
    // (with more than one warp a unit there is one round for all)
    const int nth = u / per_item, row = u % per_item / kFewSplit, at = u % kFewSplit * 32 + lane;
    int cta = -1;
    #pragma unroll
    for (int g = 0, before = 0; g < kCtaGroups; ++g) {
      const bool here = ((starts[g] >> lane) & 1) && before + __popc(starts[g] & ((1u << lane) - 1)) == nth;
      const unsigned who = __ballot_sync(0xffffffffu, here);
      if (who) cta = g * 32 + __ffs(who) - 1;
      before += __popc(starts[g]);
    }
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    int4 rec = make_int4(0, 0, 0, 0);
    if (cta >= 0) rec = *reinterpret_cast<const int4*>(p.piece + (2 * cta + 1) * kPieceWords);
    // Lane i: piece first + i.
    int flags = 0, slot = 0;
    float2 ml = make_float2(-INFINITY, 0.f);
    auto load = [&](int first) {
      const int c = cta + (first + lane) * p.head_groups;
      slot = first + lane == 0 ? 2 * cta + 1 : 2 * c;
      flags = 0;
      if (c < grid) {
        flags = p.piece[slot * kPieceWords];
        ml = *reinterpret_cast<const float2*>(p.piece_ml + ((long long)slot * p.piece_rows + row) * 2);
      }
    };
    if (cta >= 0) load(0);
    const bool have = row < rec.z;
    bool last = !have;
    for (int first = 0; !last; first += 32) {
      const unsigned ends = __ballot_sync(0xffffffffu, (flags & kPieceLast) != 0);
      // (a record that is missing, of an aborted CTA, ends the item as well)
      const unsigned holes = __ballot_sync(0xffffffffu, flags == 0);
      int n = 32;
      if (ends) n = min(n, __ffs(ends));
      if (holes) n = min(n, __ffs(holes) - 1);
      last = n < 32 || ends != 0;
      float top = lane < n ? ml.x : -INFINITY;
      #pragma unroll
      for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      top = fmaxf(top, m);
      const float keep = m == -INFINITY ? 0.f : fast_exp2(m - top);
      // (a piece of which the row saw no key weighs nothing)
      const float w = lane < n && !(ml.x == -INFINITY && ml.y == 0.f) ? fast_exp2(ml.x - top) : 0.f;
      float sum = lane < n ? ml.y * w : 0.f;
      #pragma unroll
      for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
      l = l * keep + sum;
      o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
      m = top;
      const int from = slot;
      if (!last) load(first + 32);
      #pragma unroll 4
      for (int i = warp & (share - 1); i < n; i += share) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const int si = __shfl_sync(0xffffffffu, from, i);
        const float4* src = reinterpret_cast<const float4*>(p.piece_o + ((long long)si * p.piece_rows + row) * kLatent);
        const float4 v = src[at];
        o.x += v.x * wi;
        o.y += v.y * wi;
        o.z += v.z * wi;
        o.w += v.w * wi;
      }
    }
    if (share > 1) {
      part[warp][lane] = o;
      __syncthreads();
      if ((warp & (share - 1)) != 0) return;
      for (int i = 1; i < share; ++i) {
        const float4 v = part[warp + i][lane];
        o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
      }
    }
    if (have) {
      // (the item's columns are rows of out, in order)
      const long long out_row = (long long)rec.y * p.num_q_heads + (cta % p.head_groups) * p.group_heads + row;
      const float inv = 1.f / l;
      uint2 v;
      v.x = pack_bf16(o.x * inv, o.y * inv);
      v.y = pack_bf16(o.z * inv, o.w * inv);
      reinterpret_cast<uint2*>(p.out + out_row * kLatent)[at] = v;
    }
    if (share > 1) return;
  }
}

template <bool TWO>
cudaError_t launch_decode(const LatentDecodeLaunch& L, cudaStream_t stream) {
  constexpr size_t smem = sizeof(Smem) + 1024;
  static unsigned long long configured = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(latent_decode_kernel<TWO>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&configured, bit, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = L.p.pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_decode_kernel<TWO>, L.qmap, L.kmap, L.p);
}

}  // namespace

cudaError_t launch_latent_decode(const LatentDecodeLaunch& L, cudaStream_t stream) {
  const int rows = L.p.group_heads * L.p.group_tokens;
  cudaError_t e = L.p.head_groups == 2 ? launch_decode<true>(L, stream) : launch_decode<false>(L, stream);
  if (e == cudaSuccess && L.p.merge) {
    cudaLaunchConfig_t cfg = {};
    // An item has at least one token: few have eight CTAs and more each.
    const bool few = 8ll * L.p.num_q_tokens * L.p.head_groups <= L.grid && L.grid <= 32 * kCtaGroups;
    cfg.gridDim = few ? dim3(kFewBlocks * L.grid) : dim3(L.grid, (rows + kMergeWarps - 1) / kMergeWarps);
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = L.p.pdl ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = few ? cudaLaunchKernelEx(&cfg, latent_merge_few_kernel, L.p, L.grid)
            : cudaLaunchKernelEx(&cfg, latent_merge_kernel, L.p, L.grid);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace pkv
