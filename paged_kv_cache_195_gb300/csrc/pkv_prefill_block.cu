// pkv_prefill_block.cu -- ragged chunked-prefill attention over e4m3 pools with
// a scale per (16-token block, KV head), on tcgen05 tensor cores.
//
// The tiling is the bf16 prefill kernel's (pkv_prefill.cu): a work item is
// (request, KV head, q-tile), its 128 MMA rows the (query token, head of the
// group) pairs of floor(128 / g) tokens; key tiles of 128 keys = 8 blocks come
// through the block table by TMA; the score matrix stays on the chip.
//
// S = Q K^T takes the K codes as they lie in the pool (kind::f8f6f4): a row of
// Q is scaled by a power of two so that its largest element lies in [128,
// 256) and split into two e4m3 operands, hi = e4m3(q) and lo = e4m3(q - hi),
// whose products accumulate in one TMEM tile.  bf16's eight bits are hi's four
// and lo's four, so the split is exact for every element above 2^-10 of the
// row's largest, and off by at most 2^-18 of the largest below that.  Twice
// the MMAs at twice the bf16 rate: the tensor time of a bf16 K, none of its
// widening.
// A key's block scale multiplies its column of S in the softmax.
//
// O += P V takes bf16: P rows are 128 wide here, and splitting 128 x 128
// probabilities in the softmax, which sets the pace, would cost more than
// widening V once per tile in warps of its own: four converter warps write
// bf16(decode(code) * scale) -- exact for power-of-two scales -- into one of
// two operand buffers, rows past the request's end as zeros.  They also split
// each item's Q, ahead of its first V tile.
//
// Roles (736 threads): warps 0-15 softmax and epilogue, four threads per MMA
// row (see pkv_prefill.cu); 16 takes items from the work queue and copies K
// tiles and their scales; 17 issues the MMAs; 18 copies V tiles and scales;
// 19-22 convert Q and V.  Items travel through a four-entry ring that every
// role reads.
//
// Bound: the softmax's instruction issue, like the bf16 kernel's.
#include <climits>

#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kParts = 4;                // softmax threads per MMA row
constexpr int kPartKeys = 128 / kParts;  // keys (and output dims) per softmax thread
constexpr int kSoftWarps = 4 * kParts;
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kWarpK = kSoftWarps;       // items, K tiles
constexpr int kWarpMma = kSoftWarps + 1;
constexpr int kWarpV = kSoftWarps + 2;
constexpr int kWarpConv = kSoftWarps + 3;
constexpr int kConvWarps = 4;
constexpr int kThreads = 32 * (kWarpConv + kConvWarps);
constexpr int kBarSoftmax = 1;
constexpr int kBarQuad = 2;              // + quad: the four warps holding the same 32 rows
constexpr int kRows = 128;               // MMA M
constexpr int kKeyTile = 128;
constexpr int kBlkPerTile = kKeyTile / kBlockSize;
constexpr int kCodes = kKeyTile * kHeadDim;  // a K or V tile, or a Q operand, in bytes
constexpr int kHalfBytes = kKeyTile * 128;   // one 64-dim half of a widened V tile
constexpr uint32_t kTmemCols = 512;      // S0: cols 0..127, S1: 128..255, O: 256..383
constexpr float kRescaleLog2 = 8.0f;
constexpr float kNegBig = -1.0e30f;
constexpr int kPastEnd = INT_MIN;        // block-table slot past the request (not read)
constexpr int kStages = 3;               // K stages, and raw V stages
constexpr int kItems = 4;                // item ring
constexpr int kScaleRing = 8;            // tiles whose K scales are held

struct Item {
  int r, k;   // request, KV head
  int row0;   // first query row of the tile
  int nt;     // valid tokens in the tile
  int pos0;   // position of its first token
  int L;      // request length
  int nj;     // key tiles
  int end;    // no more items
};

struct __align__(1024) Smem {
  uint8_t q[2][kCodes];              // hi | lo
  uint8_t k[kStages][kCodes];
  uint8_t v[kStages][kCodes];        // V codes
  uint8_t vb[2][2][kHalfBytes];      // widened V: [buffer][d half]
  float xrow[kParts][kRows];         // [key part][row]: partial row maxima, then normalisers
  float qf[kItems][kRows];           // factor of a row's raw scores (log2 units)
  float ks[kScaleRing][kBlkPerTile]; // K scales of a tile's blocks
  float vs[kStages][kBlkPerTile];    // V scales of a stage's blocks
  Item items[kItems];
  uint64_t it_full[kItems], it_free[kItems];
  uint64_t q_full[kItems], q_empty;
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t ks_full[kScaleRing];
  uint64_t vb_full[2], vb_free[2];
  uint64_t s_full[2], p_full[2], p_free[2];
  uint64_t o_full, o_empty;
  uint64_t mma_done;
  uint32_t tmem_base;
  int n_active;
  WaitCtl wait;
};

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

struct Req {
  int q0, qr, L, ntiles;
};

__device__ __forceinline__ Req load_req(const PrefillParams& p, int r, int tq) {
  Req a;
  a.q0 = __ldg(p.qsl + r);
  const int q1 = __ldg(p.qsl + r + 1);
  a.L = __ldg(p.seq_lens + r);
  a.qr = q1 - a.q0;
  const bool ok = a.q0 >= 0 && a.qr >= p.prefill_min_q && q1 <= p.num_q_tokens && a.qr <= a.L &&
                  a.L <= p.max_blocks * kBlockSize;
  if (!ok && a.qr >= p.prefill_min_q && blockIdx.x == 0) record_error(p.err, kErrBounds);
  a.ntiles = ok ? ceil_div(a.qr, tq) : 0;
  return a;
}

__device__ __forceinline__ void copy4_async(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// O (this thread's 32 output columns at TMEM address tO) times alpha.
static __device__ __noinline__ void rescale_o(uint32_t tO, float alpha) {
  float o[32];
  tmem_ld32(tO, o);
  tc_wait_ld();
  #pragma unroll
  for (int i = 0; i < 32; ++i) o[i] *= alpha;
  tmem_st32(tO, o);
  tc_wait_st();
}

// Two fp32 to e4m3 codes (the first in the low byte), and back to fp32 what
// they hold.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_block_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const PrefillBlockParams pb) {
  constexpr int TQ = kRows / G;  // query tokens per item
  const PrefillParams& p = pb.p;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + (((raw + 1023u) & ~1023u) - raw));
  WaitCtl* abort_flag = &sm.wait;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = p.num_kv_heads;

  // Ordering.  The decode kernel launched just before this one in the same
  // call lets it start early; everything read here was complete before the
  // decode kernel signalled, and that kernel writes only decode rows of
  // `out`.  The wait at the end makes this grid finish after the decode grid.
  //
  // CTAs without an item leave before any set-up.
  if (warp == 0) {
    long long total = 0;
    for (int b = 0; b < p.num_reqs; b += 32) {
      const int r = b + lane;
      long long cnt = r < p.num_reqs ? (long long)load_req(p, r, TQ).ntiles * Hkv : 0;
      #pragma unroll
      for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
      total += cnt;
    }
    if (lane == 0) sm.n_active = (int)min(total, (long long)gridDim.x);
  }
  __syncthreads();
  const int n_active = sm.n_active;  // CTAs that take items
  if ((int)blockIdx.x >= n_active) {
    allow_dependent_launch();
    grid_dependency_wait();
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kItems; ++s) {
      mbar_init(&sm.it_full[s], 1);
      mbar_init(&sm.it_free[s], kSoftWarps + kConvWarps + 2);  // softmax, converters, MMA, V
      mbar_init(&sm.q_full[s], kConvWarps);
    }
    mbar_init(&sm.q_empty, 1);  // tcgen05.commit after the item's last S
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1 + kBlkPerTile);  // the tile, and a scale copy per block
      mbar_init(&sm.v_empty[s], kConvWarps);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&sm.ks_full[s], kBlkPerTile);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.vb_full[b], kConvWarps);
      mbar_init(&sm.vb_free[b], 1);
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.p_full[b], kSoftWarps);
      mbar_init(&sm.p_free[b], 1);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kSoftWarps);
    mbar_init(&sm.mma_done, 1);
    sm.wait.abort = 0;
    sm.wait.limit_ns = p.wait_limit_ns;
    fence_barrier_init();
  }
  if (warp == kWarpK && lane == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  allow_dependent_launch();

  // Item n of this CTA from the ring; every warp that reads it releases it.
  auto take_item = [&](int n, Item& it) {
    if (!mbar_wait(&sm.it_full[n % kItems], (n / kItems) & 1, p.err, abort_flag)) return false;
    it = sm.items[n % kItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.it_free[n % kItems]);
    return !it.end;
  };

  if (warp == kWarpK || warp == kWarpV) {
    // ==================== TMA producers (items + K | V) ===================
    const bool vside = warp == kWarpV;
    uint64_t* const full = vside ? sm.v_full : sm.k_full;
    uint64_t* const empty = vside ? sm.v_empty : sm.k_empty;
    const CUtensorMap* const map = vside ? &vmap : &kmap;
    int n_item = 0, t = 0;
    const int oob_row = p.num_blocks * Hkv * kBlockSize;
    auto stream_item = [&](const Item& it) {
      const int nbl = ceil_div(it.L, kBlockSize);
      const int32_t* bt = p.block_tables + (long long)it.r * p.max_blocks;
      auto raw_entries = [&](int x0) {
        const int x = x0 + lane;
        return x < nbl ? __ldg(bt + x) : kPastEnd;
      };
      int ent_cur = raw_entries(0);
      int ent_nxt = it.nj > 4 ? raw_entries(32) : kPastEnd;
      for (int j = 0; j < it.nj; ++j, ++t) {
        if (j > 0 && (j & 3) == 0) {
          ent_cur = ent_nxt;
          if (j + 4 < it.nj) ent_nxt = raw_entries((j + 4) * kBlkPerTile);
        }
        const int st = t % kStages;
        if (t >= kStages && !mbar_wait(&empty[st], ((t / kStages) - 1) & 1, p.err, abort_flag))
          return false;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (uint32_t)kCodes);
        __syncwarp();
        const int phys = __shfl_sync(0xffffffffu, ent_cur, (j & 3) * kBlkPerTile + (lane & 7));
        if (lane < kBlkPerTile) {
          // Blocks past the request (or outside the pool: recorded) are read
          // at an out-of-range row, which TMA fills with zeros, with scale 0.
          const bool good = (unsigned)phys < (unsigned)p.num_blocks;
          if (!good && phys != kPastEnd && !vside) record_error(p.err, kErrBounds);
          tma_load_2d((vside ? sm.v[st] : sm.k[st]) + lane * 2048, map, 0,
                      good ? (phys * Hkv + it.k) * kBlockSize : oob_row, &full[st]);
          const float* src = (vside ? pb.v_scales : pb.k_scales) +
                             (good ? (long long)phys * Hkv + it.k : 0);
          // K scales outlive their stage: a ring entry is reused eight tiles
          // on, when S of the tile three before is done, hence PV of the tile
          // five before, hence the softmax that read the entry.
          static_assert(kScaleRing >= kStages + 3, "K scales outlive their tile's softmax");
          copy4_async(vside ? &sm.vs[st][lane] : &sm.ks[t % kScaleRing][lane], src, good ? 4u : 0u);
          arrive_after_copies(vside ? &sm.v_full[st] : &sm.ks_full[t % kScaleRing]);
        }
        __syncwarp();
      }
      return true;
    };
    if (vside) {
      Item it;
      while (take_item(n_item, it) && stream_item(it)) ++n_item;
    } else {
      // Items are numbered batch of 32 requests by batch, longest request
      // first within a batch, heavier q-tiles first within a request, and
      // taken from the queue in that order (see pkv_prefill.cu).
      auto next_item = [&]() {
        unsigned long long v = 0;
        if (lane == 0) v = atomicAdd(p.sched, 1ull);
        return (long long)__shfl_sync(0xffffffffu, v, 0);
      };
      auto publish = [&](const Item& it) {
        const int s = n_item % kItems;
        if (n_item >= kItems &&
            !mbar_wait(&sm.it_free[s], ((n_item / kItems) - 1) & 1, p.err, abort_flag))
          return false;
        if (lane == 0) {
          sm.items[s] = it;
          mbar_arrive(&sm.it_full[s]);
        }
        __syncwarp();
        return true;
      };
      long long item = next_item();
      long long base = 0;
      bool ok = true;
      for (int b = 0; b < p.num_reqs && ok && !abort_flag->abort; b += 32) {
        Req rq = {0, 0, 0, 0};
        if (b + lane < p.num_reqs) rq = load_req(p, b + lane, TQ);
        const long long cnt = (long long)rq.ntiles * Hkv;
        long long total = cnt;
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (item >= base + total) {
          base += total;
          continue;
        }
        const int key = cnt > 0 ? rq.L : -1;
        long long excl = 0;
        #pragma unroll 4
        for (int s = 0; s < 32; ++s) {
          const int ks = __shfl_sync(0xffffffffu, key, s);
          const long long cs = __shfl_sync(0xffffffffu, cnt, s);
          if (ks > key || (ks == key && s < lane)) excl += cs;
        }
        const long long incl = excl + cnt;
        while (item < base + total && ok && !abort_flag->abort) {
          const long long rel = item - base;
          const unsigned own = __ballot_sync(0xffffffffu, cnt > 0 && excl <= rel && rel < incl);
          const int src = __ffs(own) - 1;
          const long long local = rel - __shfl_sync(0xffffffffu, excl, src);
          const int q0 = __shfl_sync(0xffffffffu, rq.q0, src);
          const int qr = __shfl_sync(0xffffffffu, rq.qr, src);
          const int L = __shfl_sync(0xffffffffu, rq.L, src);
          const int qt = __shfl_sync(0xffffffffu, rq.ntiles, src) - 1 - (int)(local / Hkv);
          Item it;
          it.r = b + src;
          it.k = (int)(local % Hkv);
          it.row0 = q0 + qt * TQ;
          it.nt = min(TQ, qr - qt * TQ);
          it.pos0 = L - qr + qt * TQ;
          it.L = L;
          it.nj = (it.pos0 + it.nt - 1) / kKeyTile + 1;
          it.end = 0;
          ok = publish(it) && stream_item(it);
          ++n_item;
          item = next_item();
        }
        base += total;
      }
      Item fin = {};
      fin.end = 1;
      if (ok) publish(fin);
    }
    if (abort_flag->abort) {
      // Copies in flight land before the CTA's shared memory is released.
      // (V's barriers also count scale copies, so the last stages' data may
      // be complete without their phase; the wait is bounded.)
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int m = max(0, t - kStages); m < t; ++m)
        mbar_wait_drain(&full[m % kStages], (m / kStages) & 1, p.err, abort_flag);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kWarpMma) {
    // ========================= MMA issuer =================================
    // Tile t: S(t) into S buffer t & 1, then O += P(t-1) V(t-1), so S of the
    // next tile runs while the softmax works on the current one.
    constexpr uint32_t kIdescS = idesc_e4m3_f32(kRows, kKeyTile, 0, 0);
    constexpr uint32_t kIdescO = idesc_bf16_f32(kRows, kHeadDim, 0, 1);
    const uint32_t tO = tmem + 2 * kKeyTile;
    int t = 0;
    bool ok = true;
    auto pv = [&](int tt, bool first, int n) {
      const int b = tt & 1;
      ok = ok && mbar_wait(&sm.p_full[b], (tt >> 1) & 1, p.err, abort_flag);
      ok = ok && mbar_wait(&sm.vb_full[b], (tt >> 1) & 1, p.err, abort_flag);
      if (first && n > 0) ok = ok && mbar_wait(&sm.o_empty, (n - 1) & 1, p.err, abort_flag);
      if (!ok) return;
      tc_fence_after();
      #pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        // P: keys 16kk .. +15 in columns 8kk .. +7 of S buffer b; V MN-major,
        // two 64-dim halves.
        const uint64_t db = smem_desc_sw128(smem_u32(sm.vb[b][0]) + kk * 2048, kHalfBytes, 1024);
        tc_mma_f16_ts(tO, tmem + b * kKeyTile + kk * 8, db, kIdescO, !first || kk > 0);
      }
      tc_commit(&sm.vb_free[b]);
      tc_commit(&sm.p_free[b]);
    };
    for (int n = 0; ok; ++n) {
      Item it;
      if (!take_item(n, it)) break;
      if (lane == 0) {
        ok = mbar_wait(&sm.q_full[n % kItems], (n / kItems) & 1, p.err, abort_flag);
        for (int j = 0; j < it.nj && ok; ++j, ++t) {
          const int b = t & 1, st = t % kStages;
          ok = ok && mbar_wait(&sm.k_full[st], (t / kStages) & 1, p.err, abort_flag);
          if (t >= 2) ok = ok && mbar_wait(&sm.p_free[b], ((t >> 1) - 1) & 1, p.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          #pragma unroll
          for (int kk = 0; kk < 8; ++kk) {  // hi rows, then lo rows
            const uint64_t da = smem_desc_sw128(smem_u32(sm.q[kk >> 2]) + (kk & 3) * 32, 16, 1024);
            const uint64_t db = smem_desc_sw128(smem_u32(sm.k[st]) + (kk & 3) * 32, 16, 1024);
            tc_mma_f8_ss(tmem + b * kKeyTile, da, db, kIdescS, kk > 0);
          }
          tc_commit(&sm.k_empty[st]);
          tc_commit(&sm.s_full[b]);
          if (j + 1 == it.nj) tc_commit(&sm.q_empty);
          if (j >= 1) pv(t - 1, j == 1, n);
        }
        if (ok) pv(t - 1, it.nj == 1, n);
        if (ok) tc_commit(&sm.o_full);
      }
      __syncwarp();
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0 && abort_flag->abort) {
      tc_commit(&sm.mma_done);  // MMAs in flight finish before TMEM is freed
      mbar_wait_drain(&sm.mma_done, 0, p.err, abort_flag);
    }
    __syncwarp();
  } else if (warp >= kWarpConv) {
    // ==================== converters: Q of an item, then its V tiles =======
    const int row = tid - kWarpConv * 32, sw = row & 7;
    int t = 0;
    Item it;
    for (int n = 0; take_item(n, it); ++n) {
      {
        // Row `row` of Q: token row / G, head row % G; rows past the tile's
        // tokens become zero.
        const bool valid = row < it.nt * G;
        const uint4* src = reinterpret_cast<const uint4*>(
            pb.q + ((long long)(it.row0 + row / G) * p.num_q_heads + (long long)it.k * G + row % G) *
                       kHeadDim);
        uint4 x[16];
        uint32_t top = 0;
        #pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = valid ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        #pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
          #pragma unroll
          for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
        }
        const int e = max((int)(max(top & 0xffffu, top >> 16) >> 7), 1);
        // sigma = 2^(134 - e) in two factors within fp32's range, NaN for a
        // row that is not finite; the sign of the softmax scale goes to q, so
        // that a tile's largest score is its largest column times its factor.
        const float sgn = p.scale_log2 < 0.f ? -1.f : 1.f;
        const float s1 = e < 255 ? sgn * __uint_as_float((uint32_t)(127 + (134 - e) / 2) << 23)
                                 : __int_as_float(0x7fc00000);
        const float s2 = __uint_as_float((uint32_t)(127 + (134 - e) - (134 - e) / 2) << 23);
        if (n > 0 && !mbar_wait(&sm.q_empty, (n - 1) & 1, p.err, abort_flag)) break;
        #pragma unroll
        for (int c = 0; c < 8; ++c) {  // 16 dims: one 16-byte chunk of each operand
          const uint32_t w[8] = {x[2 * c].x,     x[2 * c].y,     x[2 * c].z,     x[2 * c].w,
                                 x[2 * c + 1].x, x[2 * c + 1].y, x[2 * c + 1].z, x[2 * c + 1].w};
          uint32_t hi[4], lo[4];
          #pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = bf16x2_to_float2(w[i]);
            const float a = f.x * s1 * s2, b = f.y * s1 * s2;
            const uint32_t h = to_e4m3x2(a, b);
            const float2 back = e4m3x2_to_float2(h);
            const uint32_t l = to_e4m3x2(a - back.x, b - back.y);
            if (i & 1) {
              hi[i >> 1] |= h << 16;
              lo[i >> 1] |= l << 16;
            } else {
              hi[i >> 1] = h;
              lo[i >> 1] = l;
            }
          }
          const int at = row * 128 + ((c ^ sw) * 16);
          *reinterpret_cast<uint4*>(sm.q[0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(sm.q[1] + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        sm.qf[n % kItems][row] = p.scale_log2 / s1 / s2;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[n % kItems]);
      }
      bool ok = true;
      for (int j = 0; j < it.nj; ++j, ++t) {
        const int st = t % kStages, b = t & 1;
        ok = mbar_wait(&sm.v_full[st], (t / kStages) & 1, p.err, abort_flag);
        if (!ok) break;
        // Key row `row` of the tile, widened: past the request's end a block
        // may hold anything (NaN codes too), and 0 * V has to stay 0.
        const bool keep = j * kKeyTile + row < it.L;
        const float s = sm.vs[st][row >> 4];
        uint4 c[8];
        #pragma unroll
        for (int i = 0; i < 8; ++i)
          c[i] = keep ? lds128(sm.v[st] + row * 128 + ((i ^ sw) * 16)) : make_uint4(0, 0, 0, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.v_empty[st]);
        if (t >= 2) ok = mbar_wait(&sm.vb_free[b], ((t >> 1) - 1) & 1, p.err, abort_flag);
        if (!ok) break;
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
          uint32_t o[8];
          #pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = e4m3x2_to_float2(w[e] & 0xffffu), v = e4m3x2_to_float2(w[e] >> 16);
            o[2 * e] = pack_bf16x2(u.x * s, u.y * s);
            o[2 * e + 1] = pack_bf16x2(v.x * s, v.y * s);
          }
          uint8_t* dst = sm.vb[b][i >> 2] + row * 128;
          const int at = (i & 3) * 2;
          *reinterpret_cast<uint4*>(dst + ((at ^ sw) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(dst + (((at + 1) ^ sw) * 16)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.vb_full[b]);
      }
      if (!ok) break;
    }
  } else {
    // =================== softmax + epilogue (warps 0-15) ===================
    const int quad = warp & 3;
    const int part = warp >> 2;
    const int row = quad * 32 + lane;  // MMA row == TMEM lane
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tO = tmem + lane_off + 2 * kKeyTile + part * kPartKeys;
    const int t_local = row / G, h = row % G;
    int t = 0;
    for (int n = 0;; ++n) {
      Item it;
      bool have = take_item(n, it);
      have = have && mbar_wait(&sm.q_full[n % kItems], (n / kItems) & 1, p.err, abort_flag);
      // Agree before any barrier: a wait that gave up (abort) stops everyone.
      if (barrier_or(kBarSoftmax, kSoftThreads, !have)) break;
      const bool valid = t_local < it.nt && row < TQ * G;
      const int prow = valid ? it.pos0 + t_local : -1;  // the last key this row sees
      const float qf = sm.qf[n % kItems][row];
      float m = kNegBig, l = 0.f;
      bool ok = true;
      for (int j = 0; j < it.nj; ++j, ++t) {
        const int sb = t & 1;
        const uint32_t tS = tmem + lane_off + sb * kKeyTile;
        ok = ok && mbar_wait(&sm.ks_full[t % kScaleRing], (t / kScaleRing) & 1, p.err, abort_flag);
        // This part's 32 keys are two blocks.  (A factor of 0 would turn a
        // masked -inf into NaN; 1e-30 leaves the scores 0.)
        float sc0 = qf * sm.ks[t % kScaleRing][part * 2], sc1 = qf * sm.ks[t % kScaleRing][part * 2 + 1];
        if (sc0 == 0.f) sc0 = 1e-30f;
        if (sc1 == 0.f) sc1 = 1e-30f;
        ok = ok && mbar_wait(&sm.s_full[sb], (t >> 1) & 1, p.err, abort_flag);
        tc_fence_after();
        const int kbase = j * kKeyTile + part * kPartKeys;
        float v[kPartKeys];
        tmem_ld32(tS + part * kPartKeys, v);
        tc_wait_ld();
        if (kbase + kPartKeys - 1 > prow) {
          #pragma unroll
          for (int i = 0; i < kPartKeys; ++i)
            if (kbase + i > prow) v[i] = -INFINITY;
        }
        float mxp[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) mxp[i] = -INFINITY;
        #pragma unroll
        for (int i = 0; i < kPartKeys / 2; ++i) {
          float& mx = mxp[(i & 1) + (i >= kPartKeys / 4 ? 2 : 0)];
          mx = fmax3(mx, v[2 * i], v[2 * i + 1]);
        }
        const float mxh = fmaxf(fmaxf(mxp[0], mxp[1]) * sc0, fmaxf(mxp[2], mxp[3]) * sc1);
        // Past an item's first tile the maximum is exchanged only when some
        // part exceeds the reference by 2^8; the vote also orders every
        // part's S reads before any P write over them.
        tc_fence_before();
        const bool exchange = barrier_or(kBarQuad + quad, 128, j == 0 || mxh > m + kRescaleLog2);
        tc_fence_after();
        if (exchange) {
          sm.xrow[part][row] = mxh;
          named_barrier(kBarQuad + quad, 128);
          const float mx = fmaxf(fmaxf(sm.xrow[0][row], sm.xrow[1][row]),
                                 fmaxf(sm.xrow[2][row], sm.xrow[3][row]));
          named_barrier(kBarQuad + quad, 128);  // sm.xrow is free again
          const bool grow = j == 0 || mx > m + kRescaleLog2;
          if (j == 0) {
            m = fmaxf(m, mx);
          } else if (__any_sync(0xffffffffu, grow)) {
            // O must first hold the previous tile's PV.
            ok = ok && mbar_wait(&sm.p_free[(t - 1) & 1], ((t - 1) >> 1) & 1, p.err, abort_flag);
            tc_fence_after();
            const float m_new = grow ? fmaxf(m, mx) : m;
            const float alpha = fast_exp2(m - m_new);
            rescale_o(tO, alpha);
            l *= alpha;
            m = m_new;
          }
        }
        // P = exp2(s - m) in bf16, two keys per column, over the row's S; the
        // normaliser sums the rounded values the MMA uses.
        const float2 nm2 = make_float2(-m, -m);
        float sum_lo[2] = {0.f, 0.f}, sum_hi[2] = {0.f, 0.f};
        uint32_t w[kPartKeys / 2];
        #pragma unroll
        for (int e = 0; e < kPartKeys / 2; ++e) {
          const float sc = e < kPartKeys / 4 ? sc0 : sc1;
          const float2 x = ffma2(make_float2(v[2 * e], v[2 * e + 1]), make_float2(sc, sc), nm2);
          w[e] = pack_bf16x2(fast_exp2(x.x), fast_exp2(x.y));
          add_bf16x2(sum_lo[e & 1], sum_hi[e & 1], w[e]);
        }
        tmem_st16(tS + part * (kPartKeys / 2), w);
        tc_wait_st();
        l += (sum_lo[0] + sum_hi[0]) + (sum_lo[1] + sum_hi[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[sb]);
      }
      // ---- epilogue: O / l -> bf16 -> out (this part's 32 dims) ----------
      sm.xrow[part][row] = l;
      named_barrier(kBarQuad + quad, 128);
      const float lrow = (sm.xrow[0][row] + sm.xrow[1][row]) + (sm.xrow[2][row] + sm.xrow[3][row]);
      named_barrier(kBarQuad + quad, 128);  // sm.xrow is free again
      ok = ok && mbar_wait(&sm.o_full, n & 1, p.err, abort_flag);
      tc_fence_after();
      const float inv = lrow == 0.f ? 0.f : 1.f / lrow;
      __nv_bfloat16* dst = p.out + ((long long)(it.row0 + t_local) * p.num_q_heads +
                                    (long long)it.k * G + h) * kHeadDim + part * kPartKeys;
      float o[32];
      tmem_ld32(tO, o);
      tc_wait_ld();
      if (valid && ok) {
        #pragma unroll
        for (int i = 0; i < 32; i += 8) {
          uint4 q4;
          q4.x = pack_bf16x2(o[i] * inv, o[i + 1] * inv);
          q4.y = pack_bf16x2(o[i + 2] * inv, o[i + 3] * inv);
          q4.z = pack_bf16x2(o[i + 4] * inv, o[i + 5] * inv);
          q4.w = pack_bf16x2(o[i + 6] * inv, o[i + 7] * inv);
          *reinterpret_cast<uint4*>(dst + i) = q4;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_empty);
    }
  }
  // Every warp reaches this point (aborts only shorten the loops), so the
  // allocating warp can always free TMEM.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
  grid_dependency_wait();
  // The last CTA to finish empties the work queue for the next launch.
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(p.sched + 1, 1ull) == (unsigned long long)(n_active - 1)) {
      p.sched[0] = 0;
      p.sched[1] = 0;
      __threadfence();
    }
  }
}

static_assert(sizeof(Smem) + 1024 <= 227 * 1024, "prefill shared memory");

template <int G>
cudaError_t launch_g(const PrefillBlockLaunch& L, cudaStream_t stream) {
  const size_t smem = sizeof(Smem) + 1024;  // + alignment slack
  static unsigned long long configured = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(prefill_block_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem);
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
  attr[0].val.programmaticStreamSerializationAllowed = L.p.p.pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_block_kernel<G>, L.kmap, L.vmap, L.p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_block(const PrefillBlockLaunch& L, int group, cudaStream_t stream) {
  switch (group) {
    case 1: return launch_g<1>(L, stream);
    case 2: return launch_g<2>(L, stream);
    case 3: return launch_g<3>(L, stream);
    case 4: return launch_g<4>(L, stream);
    case 5: return launch_g<5>(L, stream);
    case 6: return launch_g<6>(L, stream);
    case 7: return launch_g<7>(L, stream);
    case 8: return launch_g<8>(L, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
