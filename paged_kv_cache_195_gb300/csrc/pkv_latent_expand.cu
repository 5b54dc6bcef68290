// pkv_latent_expand.cu -- cached latents expanded to keys and values of every
// head, on tcgen05 tensor cores: for key j and head h the 256 numbers
//
//   kv[j, h, :] = W_h c_j,   W_h [256 x 512], c_j the latent of position j
//
// a matrix product whose left operand is gathered through the block table.
// Bound: tensor core (512 flops a byte written, the largest stream).  Measured: 8
// contexts of 512 to 4608 keys, 32 heads 83 us (1500 TFLOP/s); 701 keys, 16 heads 8.7.
//
// Tiling.  Two CTAs work as one (cta_group::2): a unit is (256 keys of one request,
// head), D[256 x 256] = C[256 x 512] W_h^T, each CTA holding 128 of the keys, 128
// of the outputs' weight rows, and the 128 x 256 part of D of its own keys in TMEM.
// Alone, a CTA would take each weight row for half as many products: 64 bytes a
// cycle of L2 and, with the MMA's own reads, more than shared memory gives.
// The units form one sequence, heads fastest, cut in equal ranges, one a pair: a
// tile's latents (128 KB a CTA, eight 64-dim chunks gathered by 2-D TMA copies of
// pool blocks) stay in shared memory for all of its heads, and the weights stream
// by from L2, a 64-dim chunk at a time, five in flight (four: 92 us for 83).  D has two
// TMEM buffers of 256 columns, so that a unit's rows are rounded and stored while the next is multiplied.  Keys
// behind the request's end are rows of D that nobody stores.
//
// Roles (224 threads): warps 0-3 take D's rows, one a thread, round them once,
// and turn them through shared memory into stores of whole 128-byte lines (a bulk
// copy a row took longer to issue than the products); warp 4 copies weights, warp 6
// latents, each as its own room comes free; warp 5 of the pair's first CTA issues the
// MMAs of both.  Copies of both CTAs count on the first one's barriers,
// commits arrive on both's.
#include <climits>

#include "pkv_latent.h"
#include "pkv_pair.cuh"

namespace pkv {
namespace {

constexpr int kEpiWarps = 4;
constexpr int kWarpLoad = kEpiWarps;
constexpr int kWarpMma = kEpiWarps + 1;
constexpr int kWarpKeys = kEpiWarps + 2;
constexpr int kThreads = 32 * (kEpiWarps + 3);
constexpr int kKeys = 128;                 // keys of a CTA: half of the MMA's M
constexpr int kPairKeys = 2 * kKeys;
constexpr int kOut = kNope + kValDim;      // outputs of a unit: MMA N
constexpr int kHalf = 128;                 // weight rows of a CTA
constexpr int kChunks = kLatent / 64;
constexpr int kChunkBytes = 128 * 128;     // 128 rows of 64 bf16
constexpr int kStages = 5;                 // weight pieces in flight
constexpr int kRowCols = 64;               // columns that a row stores at a time
constexpr int kRowBytes = kRowCols * 2 + 16;  // (16 bytes apart from a bank-aligned stride)

struct __align__(1024) Smem {
  uint8_t a[kChunks][kChunkBytes];
  uint8_t b[kStages][kChunkBytes];
  uint8_t row[kKeys][kRowBytes];
  uint64_t a_full[kChunks], a_empty[kChunks];
  uint64_t b_full[kStages], b_empty[kStages];
  uint64_t d_full[2], d_empty[2];
  uint64_t drained;
  uint32_t tmem_base;
  WaitCtl wait;
  long long part[kThreads / 32];
  long long range_lo, range_hi, start_base;
  int start_req;
};
// (no room to align it in: a block without static shared memory has it on a KiB)
static_assert(sizeof(Smem) <= 227 * 1024, "latent expand shared memory");

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// A request's keys and the first row of kv that they go to; keys 0: nothing to do.
struct Req {
  int keys, row0;
};

__device__ __forceinline__ Req load_req(const LatentExpandParams& p, int r, bool* bad) {
  const int n = __ldg(p.seq_lens + r), a = __ldg(p.kv_start + r), b = __ldg(p.kv_start + r + 1);
  // (b >= a: the difference of wild entries may wrap)
  *bad = !(n >= 0 && n <= p.max_blocks * kBlockSize && a >= 0 && b >= a && b <= p.num_rows && b - a == n);
  return Req{*bad ? 0 : n, a};
}

__device__ __forceinline__ long long units(const LatentExpandParams& p, const Req& a) {
  return (long long)cdiv(a.keys, kPairKeys) * p.num_heads;
}

// The CTA's range of the units and the request that it starts in.  All threads.
__device__ __forceinline__ void plan_range(const LatentExpandParams& p, Smem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = cdiv(p.num_reqs, kThreads);
  const int r0 = min(tid * per, p.num_reqs), r1 = min(r0 + per, p.num_reqs);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) {
    bool bad;
    mine += units(p, load_req(p, r, &bad));
    if (bad && blockIdx.x == 0) record_error(p.err, kErrBounds);  // the request is skipped
  }
  long long incl = mine;
  #pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.part[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm.part[w];
    total += sm.part[w];
  }
  const long long excl = before + incl - mine;
  const int pairs = gridDim.x >> 1;
  const long long chunk = (total + pairs - 1) / pairs;
  const long long lo = min((blockIdx.x >> 1) * chunk, total), hi = min(lo + chunk, total);
  if (tid == 0) {
    sm.range_lo = lo;
    sm.range_hi = hi;
  }
  if (lo < hi && excl <= lo && lo < excl + mine) {
    long long base = excl;
    for (int r = r0; r < r1; ++r) {
      bool bad;
      const long long w = units(p, load_req(p, r, &bad));
      if (lo < base + w) {
        sm.start_req = r;
        sm.start_base = base;
        break;
      }
      base += w;
    }
  }
  __syncthreads();
}

// The range's runs in order -- heads h0 .. h1 - 1 of the 256-key tile `tile` of request
// `req` -- which every role walks for itself.
struct Walk {
  int req, tile, h0, h1;
  Req a;
  long long base, pos;

  __device__ __forceinline__ void start(const Smem& sm) {
    req = sm.start_req;
    base = sm.start_base;
    pos = sm.range_lo;
    a.keys = -1;  // not read yet
  }
  __device__ __forceinline__ bool next(const LatentExpandParams& p, const Smem& sm) {
    if (pos >= sm.range_hi) return false;
    bool bad;
    if (a.keys < 0) a = load_req(p, req, &bad);
    while (pos >= base + units(p, a)) {
      base += units(p, a);
      // (pos < range_hi: there is a later request, unless someone writes the lengths meanwhile)
      if (++req >= p.num_reqs) return false;
      a = load_req(p, req, &bad);
    }
    const long long local = pos - base;
    tile = (int)(local / p.num_heads);
    h0 = (int)(local - (long long)tile * p.num_heads);
    const long long left = sm.range_hi - pos;
    h1 = (int)min((long long)p.num_heads, h0 + left);
    pos += h1 - h0;
    return true;
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_expand_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap wmap, const LatentExpandParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) record_error(p.err, kErrCapacity);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1;  // in the pair
  WaitCtl* ctl = &sm.wait;
  if (tid == 0) {
    for (int i = 0; i < kChunks; ++i) {
      mbar_init(&sm.a_full[i], 1);
      mbar_init(&sm.a_empty[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.b_full[i], 1);
      mbar_init(&sm.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.d_full[i], 1);
      mbar_init(&sm.d_empty[i], 2 * kEpiWarps);
    }
    mbar_init(&sm.drained, 1);
    sm.wait.abort = 0;
    sm.wait.limit_ns = p.wait_limit_ns;
    fence_barrier_init();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&wmap);
  }
  // The plan is made after the wait: the running sum of the lengths is as a rule the work
  // of the kernel ahead.  (A CTA without work waits too: the next kernel relies on all
  // before this one.)
  grid_dependency_wait();
  allow_dependent_launch();
  plan_range(p, sm);
  if (sm.range_lo >= sm.range_hi) return;  // (so has the pair's other CTA)
  if (warp == kWarpMma) {
    tmem_alloc_pair(&sm.tmem_base, 512);
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem_base);
  Walk w;
  w.start(sm);

  if (warp == kWarpKeys) {
    // =========================== latents ==================================
    const bool leader = elect_one();
    const int oob_row = p.num_blocks * kBlockSize;
    int n_tile = 0, chunks = 0;  // runs so far; chunks of run n_tile
    bool ok = true;
    while (ok && w.next(p, sm)) {
      // Lane b < 8 holds the row of block b; blocks past the end are read at a row
      // outside the pool, which fills zeros.
      const int blk = w.tile * (kPairKeys / kBlockSize) + rank * (kKeys / kBlockSize) + lane;
      int row = oob_row;
      if (lane < 8 && blk * kBlockSize < w.a.keys) {
        const int id = __ldg(p.block_tables + (long long)w.req * p.max_blocks + blk);
        if ((unsigned)id < (unsigned)p.num_blocks) row = id * kBlockSize;
        else record_error(p.err, kErrBounds);
      }
      // (one thread issues all copies, from uniform registers)
      int rows[kKeys / kBlockSize];
      #pragma unroll
      for (int b = 0; b < kKeys / kBlockSize; ++b) rows[b] = uniform(__shfl_sync(0xffffffffu, row, b));
      #pragma unroll 1
      for (chunks = 0; chunks < kChunks; ++chunks) {
        if (n_tile > 0) ok = all_of(wait_for(&sm.a_empty[chunks], (n_tile - 1) & 1, p.err, ctl));
        if (!ok) break;
        if (leader) {
          if (rank == 0) mbar_arrive_expect_tx(&sm.a_full[chunks], 2 * kChunkBytes);
          const uint32_t bar = first_cta(&sm.a_full[chunks]);
          #pragma unroll
          for (int b = 0; b < kKeys / kBlockSize; ++b)
            tma_load_2d_pair(sm.a[chunks] + b * 2048, &kmap, chunks * 64, rows[b], bar);
        }
        __syncwarp();
      }
      if (ok) ++n_tile;
    }
    if (!ok && rank == 0) {
      // Aborted: the copies in flight must land before the pair ends (the barrier
      // at the end keeps the other CTA's memory until then).
      for (int c = 0; c < kChunks; ++c) {
        const int n = n_tile + (c < chunks ? 1 : 0);
        if (n > 0) drain(&sm.a_full[c], (n - 1) & 1, p.err, ctl);
      }
    } else if (!ok) {
      settle();
    }
  } else if (warp == kWarpLoad) {
    // =========================== weights ==================================
    const bool leader = elect_one();
    int n_b = 0, st = 0, phase = 1;  // pieces so far; their stage and the parity it waits for
    bool ok = true;
    while (ok && w.next(p, sm)) {
      #pragma unroll 1
      for (int h = w.h0; h < w.h1 && ok; ++h) {
        #pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          ok = all_of(wait_for(&sm.b_empty[st], phase, p.err, ctl));
          if (!ok) break;
          if (leader) {
            if (rank == 0) mbar_arrive_expect_tx(&sm.b_full[st], 2 * kChunkBytes);
            if (!p.debug_withhold_q)
              tma_load_3d_pair(sm.b[st], &wmap, c * 64, h * kOut + rank * kHalf, 0, first_cta(&sm.b_full[st]));
          }
          __syncwarp();
          ++n_b;
          if (++st == kStages) st = 0, phase ^= 1;
        }
      }
    }
    if (!ok && rank == 0) {
      for (int i = max(0, n_b - kStages); i < n_b; ++i)
        drain(&sm.b_full[i % kStages], (i / kStages) & 1, p.err, ctl);
    } else if (!ok) {
      settle();
    }
  } else if (warp == kWarpMma && rank == 0) {
    // ============================ MMAs ====================================
    constexpr uint32_t kIdesc = idesc_bf16_f32(kPairKeys, kOut, 0, 0);
    const uint64_t desc_a = smem_desc_sw128(smem_u32(sm.a[0]), 16, 1024);
    const uint64_t desc_b = smem_desc_sw128(smem_u32(sm.b[0]), 16, 1024);
    const bool leader = elect_one();
    int n_tile = 0, n_d = 0, st = 0, phase = 0;
    bool ok = true;
    while (ok && w.next(p, sm)) {
      #pragma unroll 1
      for (int h = w.h0; h < w.h1; ++h, ++n_d) {
        const int d = n_d & 1;
        if (n_d >= 2) ok = all_of(wait_for(&sm.d_empty[d], ((n_d >> 1) - 1) & 1, p.err, ctl));
        #pragma unroll 1
        for (int c = 0; c < kChunks && ok; ++c) {
          if (h == w.h0) ok = all_of(wait_for(&sm.a_full[c], n_tile & 1, p.err, ctl));
          ok = ok && all_of(wait_for(&sm.b_full[st], phase, p.err, ctl));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t da = desc_a + (uint64_t)(c * (kChunkBytes >> 4));
            const uint64_t db = desc_b + (uint64_t)(st * (kChunkBytes >> 4));
            #pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_pair(tmem + d * kOut, da + 2 * kk, db + 2 * kk, kIdesc, c > 0 || kk > 0);
            commit_pair(&sm.b_empty[st]);
            if (h == w.h1 - 1) commit_pair(&sm.a_empty[c]);
            if (c == kChunks - 1) commit_pair(&sm.d_full[d]);
          }
          __syncwarp();
          if (++st == kStages) st = 0, phase ^= 1;
        }
        if (!ok) break;
      }
      ++n_tile;
    }
    if (!ok) {
      // Aborted: the issued MMAs must end before TMEM is freed.
      if (leader) commit_pair(&sm.drained);
      __syncwarp();
      drain(&sm.drained, 0, p.err, ctl);
    }
  } else if (warp < kEpiWarps) {
    // ====================== rounding and stores (warps 0-3) ==================
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    uint8_t* mine = sm.row[tid];
    int n_d = 0;
    bool ok = true;
    while (ok && w.next(p, sm)) {
      const int key0 = w.tile * kPairKeys + rank * kKeys;  // of this CTA
      if (w.h0 == 0) {
        // The rotated keys of these 128 keys, eight lanes a row.
        for (int i = tid; i < kKeys * 8; i += 32 * kEpiWarps) {
          const int k = key0 + (i >> 3);
          if (k >= w.a.keys) break;
          const int id = __ldg(p.block_tables + (long long)w.req * p.max_blocks + k / kBlockSize);
          // (zeros for a block outside the pool, as its rows of kv)
          uint4 x = make_uint4(0, 0, 0, 0);
          if ((unsigned)id < (unsigned)p.num_blocks)
            x = reinterpret_cast<const uint4*>(p.pool + ((long long)id * kBlockSize + k % kBlockSize) * kLatRow +
                                               kLatent)[i & 7];
          reinterpret_cast<uint4*>(p.k_rope + ((long long)w.a.row0 + k) * kRopeDim)[i & 7] = x;
        }
      }
      for (int h = w.h0; h < w.h1 && ok; ++h, ++n_d) {
        const int d = n_d & 1;
        ok = wait_for(&sm.d_full[d], (n_d >> 1) & 1, p.err, ctl);
        if (__any_sync(0xffffffffu, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        __nv_bfloat16* dst = p.kv + (((long long)w.a.row0 + key0) * p.num_heads + h) * kOut;
        #pragma unroll 1
        for (int q = 0; q < kOut / kRowCols; ++q) {
          float v[kRowCols / 2], u[kRowCols / 2];
          tmem_ld32(tmem + lane_off + d * kOut + q * kRowCols, v);
          tmem_ld32(tmem + lane_off + d * kOut + q * kRowCols + 32, u);
          tc_wait_ld();
          __syncwarp();  // the warp has read its rows of before
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<uint4*>(mine + 16 * i) =
                make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                           pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
            *reinterpret_cast<uint4*>(mine + 64 + 16 * i) =
                make_uint4(pack_bf16(u[8 * i], u[8 * i + 1]), pack_bf16(u[8 * i + 2], u[8 * i + 3]),
                           pack_bf16(u[8 * i + 4], u[8 * i + 5]), pack_bf16(u[8 * i + 6], u[8 * i + 7]));
          }
          __syncwarp();
          // Eight lanes a row of 128 bytes, four rows at a time.
          #pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = warp * 32 + i * 4 + (lane >> 3);
            if (key0 + r < w.a.keys)
              *reinterpret_cast<uint4*>(dst + (long long)r * p.num_heads * kOut + q * kRowCols + (lane & 7) * 8) =
                  *reinterpret_cast<const uint4*>(sm.row[r] + (lane & 7) * 16);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(first_cta(&sm.d_empty[d]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // nothing of either CTA is under way in the other
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc_pair(tmem, 512);
  cluster_barrier();
}

}  // namespace

cudaError_t launch_latent_expand(const LatentExpandLaunch& L, cudaStream_t stream) {
  const size_t smem = sizeof(Smem);
  static unsigned long long configured = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(latent_expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&configured, bit, __ATOMIC_RELEASE);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(L.grid / 2 * 2);
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
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, latent_expand_kernel, L.kmap, L.wmap, L.p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace pkv
