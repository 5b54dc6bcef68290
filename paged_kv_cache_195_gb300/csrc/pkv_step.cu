// pkv_step.cu -- an engine step's block tables and slot map, built on the GPU
// from request lengths, and the blocks of finished or shortened requests
// given back (pkv_build_step, pkv_release_blocks).
//
// Both are a prefix sum over the requests followed by an expansion: build
// gives request r its new blocks (ceil((p + n) / 16) - ceil(p / 16) entries
// popped from the free list) and its n slots, release gives back the table
// entries past the blocks it keeps.  One cluster does a whole step: each CTA
// takes a contiguous run of requests, scans it in shared memory, exchanges
// totals through distributed shared memory, and then every thread of the
// cluster expands items in order, finding an item's request by a binary
// search of the scan (first over the CTAs, then in the owner's shared
// memory).  No value is read back from global memory that the kernel wrote:
// an item's block is computed from the scan and the free list, so there is no
// second launch and no grid-wide wait.
//
// Bound: latency.  The bytes (16 per request, 8 per token, 8 per block) are
// far below what a launch costs; the time is one load round trip, the scan,
// two cluster barriers, the search and one dependent load.
#include <climits>

#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of the cluster; shared-memory writes before it are visible to
// every CTA after it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t remote_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ int remote_load(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ long long remote_load64(uint32_t addr) {
  long long v;
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int blocks_of(int tokens) {
  return (int)(((unsigned)tokens + kBlockSize - 1) / kBlockSize);
}

struct Pair {
  long long blocks, tokens;
};

// Shared state of one CTA; the per-request arrays follow it.
struct StepSmem {
  Pair warp_sum[32];
  Pair total;           // this CTA's requests
  Pair base[kMaxCluster + 1];  // sums before each CTA (every CTA holds all)
  int granted_tokens;   // of this CTA's requests: the largest granted sums, and
  int granted_blocks;   // the requests refused
  int refused;
  int bad;              // release: entries of this CTA's items outside the pool
};

// Exclusive sums over the cluster's threads of each thread's pair; fills
// sm.base.  Every thread of the cluster.
__device__ __forceinline__ Pair cluster_scan(StepSmem& sm, Pair mine, uint32_t rank,
                                             uint32_t ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  Pair incl = mine;
  #pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long b = __shfl_up_sync(0xffffffffu, incl.blocks, o);
    const long long t = __shfl_up_sync(0xffffffffu, incl.tokens, o);
    if (lane >= o) {
      incl.blocks += b;
      incl.tokens += t;
    }
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    Pair w = lane < warps ? sm.warp_sum[lane] : Pair{0, 0};
    const Pair own = w;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long b = __shfl_up_sync(0xffffffffu, w.blocks, o);
      const long long t = __shfl_up_sync(0xffffffffu, w.tokens, o);
      if (lane >= o) {
        w.blocks += b;
        w.tokens += t;
      }
    }
    if (lane < warps) sm.warp_sum[lane] = Pair{w.blocks - own.blocks, w.tokens - own.tokens};
    if (lane == 31) sm.total = w;
  }
  if (ctas > 1) cluster_barrier(); else __syncthreads();
  if (threadIdx.x == 0) {
    Pair s{0, 0};
    for (uint32_t c = 0; c < ctas; ++c) {
      sm.base[c] = s;
      const uint32_t a = remote_addr(&sm.total, c);
      s.blocks += remote_load64(a);
      s.tokens += remote_load64(a + 8);
    }
    sm.base[ctas] = s;
  }
  __syncthreads();
  const Pair w = sm.warp_sum[warp], c = sm.base[rank];
  return Pair{c.blocks + w.blocks + incl.blocks - mine.blocks,
              c.tokens + w.tokens + incl.tokens - mine.tokens};
}

// The request holding item i of an expansion: the last request whose
// exclusive sum (in `first`, one entry per request of the owning CTA) is at
// most i.  Requests without items share their sum with the next request and
// are never the last.  `lo_of(c)`: the sum before CTA c.
struct Found {
  uint32_t rank;
  int index;  // within the owner's run
  int first;  // its exclusive sum
};
template <typename LoOf>
__device__ __forceinline__ Found find_item(const int* first, int i, uint32_t ctas, int per,
                                           int num_reqs, LoOf lo_of) {
  Found f;
  f.rank = 0;
  for (uint32_t c = 1; c < ctas; ++c)
    if (lo_of(c) <= i) f.rank = c;
  // A CTA after the last request has the total as its sum, which no item reaches.
  int a = 0, b = min(per, num_reqs - (int)f.rank * per) - 1;
  const uint32_t base = remote_addr(first, f.rank);
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (remote_load(base + 4 * mid) <= i) a = mid; else b = mid - 1;
  }
  f.index = a;
  f.first = remote_load(base + 4 * a);
  return f;
}

__device__ __forceinline__ int clamp_int(long long v) { return (int)min(v, (long long)INT_MAX); }

// The number of free blocks, held to what the list can hold.
__device__ __forceinline__ int load_num_free(const int32_t* p, int num_blocks, int* err) {
  const int f = *p;
  if (f < 0 || f > num_blocks) {
    record_error(err, kErrBounds);
    return f < 0 ? 0 : num_blocks;
  }
  return f;
}

__global__ void __launch_bounds__(1024) build_step_kernel(const StepParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  StepSmem& sm = *reinterpret_cast<StepSmem*>(smem_raw);
  int* const tok0 = reinterpret_cast<int*>(smem_raw + sizeof(StepSmem));  // exclusive token sums
  int* const blk0 = tok0 + p.per_cta;                                     // exclusive block sums
  int* const prev = blk0 + p.per_cta;                                     // lengths before the step
  const uint32_t rank = cluster_rank(), ctas = gridDim.x;
  const int tid = threadIdx.x;
  grid_dependency_wait();
  const int F = load_num_free(p.num_free_in, p.num_blocks, tid == 0 && rank == 0 ? p.err : nullptr);
  const long long cap = (long long)p.max_blocks * kBlockSize;
  // This thread's run of requests.
  const int each = (p.per_cta + blockDim.x - 1) / blockDim.x;
  const int i0 = tid * each, i1 = min(min(i0 + each, p.per_cta), p.num_reqs - (int)rank * p.per_cta);
  const long long r0 = (long long)rank * p.per_cta;
  if (tid == 0) {
    sm.granted_tokens = 0;
    sm.granted_blocks = 0;
    sm.refused = 0;
  }
  Pair mine{0, 0};
  for (int i = i0; i < i1; ++i) {
    const int pl = p.prev_lens[r0 + i], n = p.new_tokens[r0 + i];
    const bool ok = pl >= 0 && n >= 0 && (long long)pl + n <= cap;
    prev[i] = ok ? pl : -1;
    tok0[i] = n;  // read back below by this thread
    if (ok) {
      mine.blocks += blocks_of(pl + n) - blocks_of(pl);
      mine.tokens += n;
    } else {
      record_error(p.err, kErrBounds);
    }
  }
  Pair at = cluster_scan(sm, mine, rank, ctas);
  int granted_t = 0, granted_b = 0, refused = 0;
  for (int i = i0; i < i1; ++i) {
    const int pl = prev[i], n = tok0[i];
    const bool ok = pl >= 0;
    const int need = ok ? blocks_of(pl + n) - blocks_of(pl) : 0;
    const int add = ok ? n : 0;
    tok0[i] = clamp_int(at.tokens);
    blk0[i] = clamp_int(at.blocks);
    at.blocks += need;
    at.tokens += add;
    // Both sums never fall, so the requests served are those before the
    // first whose blocks or tokens do not fit.
    const bool go = ok && (add == 0 || (at.blocks <= F && at.tokens <= p.num_q_tokens));
    if (go && add > 0) {
      granted_t = (int)at.tokens;
      granted_b = (int)at.blocks;
    }
    refused += !go;
    p.seq_lens[r0 + i] = !ok ? 0 : go ? pl + add : pl;
  }
  if (granted_t > 0) {
    atomicMax(&sm.granted_tokens, granted_t);
    atomicMax(&sm.granted_blocks, granted_b);
  }
  if (refused > 0) atomicAdd(&sm.refused, refused);
  if (ctas > 1) cluster_barrier(); else __syncthreads();
  int T = 0, N = 0, all_refused = 0;
  for (uint32_t c = 0; c < ctas; ++c) {
    T = max(T, remote_load(remote_addr(&sm.granted_tokens, c)));
    N = max(N, remote_load(remote_addr(&sm.granted_blocks, c)));
    if (rank == 0 && tid == 0) all_refused += remote_load(remote_addr(&sm.refused, c));
  }
  // query_start_loc: a request after the first refused one starts, like every
  // later one, at the served requests' end.
  for (int i = i0; i < i1; ++i) p.query_start_loc[r0 + i] = min(tok0[i], T);
  if (rank == 0 && tid == 0) {
    p.query_start_loc[p.num_reqs] = T;
    *p.num_free_out = F - N;
    if (p.num_refused) *p.num_refused = all_refused;
  }
  const int threads = blockDim.x * ctas, me = rank * blockDim.x + tid;
  // The popped blocks, in request order: pop j is free_list[F - 1 - j].
  for (int j = me; j < N; j += threads) {
    const Found f = find_item(blk0, j, ctas, p.per_cta, p.num_reqs,
                              [&](uint32_t c) { return clamp_int(sm.base[c].blocks); });
    const int pl = remote_load(remote_addr(prev + f.index, f.rank));
    const long long r = (long long)f.rank * p.per_cta + f.index;
    p.block_tables[r * p.max_blocks + blocks_of(pl) + (j - f.first)] = p.free_list[F - 1 - j];
  }
  // The slots, token by token; padding rows get -1.
  for (int t = me; t < p.num_q_tokens; t += threads) {
    long long slot = -1;
    if (t < T) {
      const Found f = find_item(tok0, t, ctas, p.per_cta, p.num_reqs,
                                [&](uint32_t c) { return clamp_int(sm.base[c].tokens); });
      const int pl = remote_load(remote_addr(prev + f.index, f.rank));
      const int first_pop = remote_load(remote_addr(blk0 + f.index, f.rank));
      const long long r = (long long)f.rank * p.per_cta + f.index;
      const int pos = pl + (t - f.first), col = pos / kBlockSize, held = blocks_of(pl);
      const int id = col < held ? p.block_tables[r * p.max_blocks + col]
                                : p.free_list[F - 1 - (first_pop + col - held)];
      if ((unsigned)id < (unsigned)p.num_blocks) slot = (long long)id * kBlockSize + pos % kBlockSize;
      else record_error(p.err, kErrBounds);
    }
    p.slot_mapping[t] = slot;
  }
  // The tables and lengths are in place before the next kernel may start
  // (this one never lets it launch early), and no CTA leaves while another
  // may read its shared memory.
  __threadfence();
  if (ctas > 1) cluster_barrier();
}

__global__ void __launch_bounds__(1024) release_blocks_kernel(const ReleaseParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  StepSmem& sm = *reinterpret_cast<StepSmem*>(smem_raw);
  int* const blk0 = reinterpret_cast<int*>(smem_raw + sizeof(StepSmem));  // exclusive block sums
  int* const col0 = blk0 + p.per_cta;                                     // first column given back
  const uint32_t rank = cluster_rank(), ctas = gridDim.x;
  const int tid = threadIdx.x;
  grid_dependency_wait();
  const int F = load_num_free(p.num_free_in, p.num_blocks, tid == 0 && rank == 0 ? p.err : nullptr);
  const long long cap = (long long)p.max_blocks * kBlockSize;
  const int each = (p.per_cta + blockDim.x - 1) / blockDim.x;
  const int i0 = tid * each, i1 = min(min(i0 + each, p.per_cta), p.num_reqs - (int)rank * p.per_cta);
  const long long r0 = (long long)rank * p.per_cta;
  if (tid == 0) sm.bad = 0;
  Pair mine{0, 0};
  for (int i = i0; i < i1; ++i) {
    const int len = p.seq_lens[r0 + i], keep = p.keep_lens[r0 + i];
    const bool ok = keep >= 0 && keep <= len && len <= cap;
    if (!ok) record_error(p.err, kErrBounds);
    col0[i] = ok ? blocks_of(keep) : 0;
    blk0[i] = ok ? blocks_of(len) - blocks_of(keep) : 0;  // read back below by this thread
    mine.blocks += blk0[i];
  }
  Pair at = cluster_scan(sm, mine, rank, ctas);
  for (int i = i0; i < i1; ++i) {
    const int n = blk0[i];
    blk0[i] = clamp_int(at.blocks);
    at.blocks += n;
  }
  if (ctas > 1) cluster_barrier(); else __syncthreads();
  // What the list has no room for is a block given back twice somewhere.
  const long long all = sm.base[ctas].blocks;
  const int M = (int)min(all, (long long)(p.num_blocks - F));
  if (all > M && rank == 0 && tid == 0) record_error(p.err, kErrBounds);
  const int threads = blockDim.x * ctas, me = rank * blockDim.x + tid;
  for (int j = me; j < M; j += threads) {
    const Found f = find_item(blk0, j, ctas, p.per_cta, p.num_reqs,
                              [&](uint32_t c) { return clamp_int(sm.base[c].blocks); });
    const int col = remote_load(remote_addr(col0 + f.index, f.rank)) + (j - f.first);
    const long long r = (long long)f.rank * p.per_cta + f.index;
    int id = p.block_tables[r * p.max_blocks + col];
    if ((unsigned)id >= (unsigned)p.num_blocks) {
      id = -1;
      atomicAdd(&sm.bad, 1);
      record_error(p.err, kErrBounds);
    }
    p.free_list[F + j] = id;
  }
  __threadfence();
  if (ctas > 1) cluster_barrier(); else __syncthreads();
  if (rank == 0 && tid < 32) {
    int bad = 0;
    for (uint32_t c = 0; c < ctas; ++c) bad += remote_load(remote_addr(&sm.bad, c));
    if (bad > 0) {
      // Entries outside the pool were not given back: close the gaps they
      // left (a caller's error, so one warp and in order).
      int w = F;
      for (int j = 0; j < M; j += 32) {
        const int id = j + tid < M ? __ldcg(p.free_list + F + j + tid) : -1;
        const unsigned good = __ballot_sync(0xffffffffu, id >= 0);
        if (id >= 0) p.free_list[w + __popc(good & ((1u << tid) - 1))] = id;
        w += __popc(good);
        __syncwarp();
      }
    }
    if (tid == 0) *p.num_free_out = F + M - bad;
  }
  __threadfence();
  if (ctas > 1) cluster_barrier();
}

// One CTA while its threads cover the requests and a few items each, else a
// cluster of eight.
template <typename P>
cudaError_t launch_step(void (*kernel)(const P), P p, int arrays, long long items, bool pdl,
                        cudaStream_t stream) {
  const bool small = p.num_reqs <= 1024 && items <= 4096;
  const int ctas = small ? 1 : kMaxCluster;
  p.per_cta = (p.num_reqs + ctas - 1) / ctas;
  const long long widest = items / ctas > p.per_cta ? items / ctas : p.per_cta;
  const int threads = widest <= 256 ? 256 : widest <= 512 ? 512 : 1024;
  const size_t smem = sizeof(StepSmem) + (size_t)arrays * p.per_cta * sizeof(int);
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

static_assert(sizeof(StepSmem) + 3 * (kMaxReqs / kMaxCluster) * sizeof(int) <= 227 * 1024,
              "the largest step's shared memory");

}  // namespace

cudaError_t launch_build_step(const StepParams& p, bool pdl, cudaStream_t stream) {
  return launch_step(build_step_kernel, p, 3, p.num_q_tokens, pdl, stream);
}

cudaError_t launch_release_blocks(const ReleaseParams& p, bool pdl, cudaStream_t stream) {
  return launch_step(release_blocks_kernel, p, 2, 4ll * p.num_reqs, pdl, stream);
}

}  // namespace pkv
