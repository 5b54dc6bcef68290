// pkv_step.cu -- an engine step's block tables and slot map, built on the GPU
// from request lengths, and the blocks of finished or shortened requests
// given back (pkv_build_step, pkv_release_blocks).
//
// Both are a prefix sum over the requests followed by an expansion: build
// gives request r its new blocks (ceil((p + n) / 16) - ceil(p / 16) entries
// popped from the free list) and its n slots, release gives back the table
// entries past the blocks it keeps.
//
// One cluster of eight CTAs (one CTA for small steps) does a whole step in one
// launch, and every CTA scans all requests by itself: a thread sums a
// contiguous run of them, a block-wide scan of the 1024 run sums stays in
// shared memory, and an item (a token, a block) finds its request by a search
// over the run sums and a walk within the run, whose lengths its SM has just
// read.  Reading every length eight times costs less than exchanging sums: with the
// scan split over the CTAs and gathered through distributed shared memory, the
// exchange alone took 8000 cycles of a 4096-request step.  No value is read
// back that the kernel wrote -- an item's block follows from the sums and the
// free list -- so nothing waits on a grid; what may overwrite an input in
// place (seq_lens over prev_lens, the number of free blocks) is written after
// one cluster barrier, when every CTA has read it.
//
// The slots of a large step are a second launch over the whole GPU, from the
// finished tables and lengths: a decode token reads a table sector of its own,
// and eight SMs' path to L2 (64 bytes a clock each) took 8000 cycles for 42
// thousand of them.
//
// Bound: latency.  The bytes (16 per request, 8 per token, 8 per block) are
// far below what a launch costs.  Measured: build 4.1 us for 64 decodes, 11.1
// for 4096 requests with 42 thousand tokens (two launches); release 2.8 us for
// 64 requests, 8.8 for 4096.
#include <climits>

#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kMaxThreads = 1024;
constexpr int kGroup = 4;   // items a thread expands after one search; requests loaded together

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// All threads of the cluster; shared-memory and global writes before it are
// visible to every CTA after it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int remote_load(const void* p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ int blocks_of(int tokens) {
  return (int)(((unsigned)tokens + kBlockSize - 1) / kBlockSize);
}

__device__ __forceinline__ int clamp_int(long long v) { return (int)min(v, (long long)INT_MAX); }

// One request's items: blocks (popped or given back) and tokens, and the
// length that places them.
struct Need {
  int blocks, tokens, base;
  bool ok;
};

struct Pair {
  long long blocks, tokens;
};

struct StepSmem {
  Pair warp_sum[32];
  Pair total;
  int run_blocks[kMaxThreads];  // exclusive sums before each thread's run of
  int run_tokens[kMaxThreads];  // requests, held to INT_MAX (no item is there)
  int served_blocks, served_tokens, refused;
  int bad;
};

// Exclusive sums over the CTA's threads, also in sm.run_*.
__device__ __forceinline__ Pair scan_runs(StepSmem& sm, Pair mine) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto warp_scan = [&](Pair v) {
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long b = __shfl_up_sync(0xffffffffu, v.blocks, o);
      const long long t = __shfl_up_sync(0xffffffffu, v.tokens, o);
      if (lane >= o) {
        v.blocks += b;
        v.tokens += t;
      }
    }
    return v;
  };
  const Pair incl = warp_scan(mine);
  if (lane == 31) sm.warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const Pair own = lane < warps ? sm.warp_sum[lane] : Pair{0, 0};
    const Pair w = warp_scan(own);
    if (lane < warps) sm.warp_sum[lane] = Pair{w.blocks - own.blocks, w.tokens - own.tokens};
    if (lane == 31) sm.total = w;
  }
  __syncthreads();
  const Pair w = sm.warp_sum[warp];
  const Pair at{w.blocks + incl.blocks - mine.blocks, w.tokens + incl.tokens - mine.tokens};
  sm.run_blocks[threadIdx.x] = clamp_int(at.blocks);
  sm.run_tokens[threadIdx.x] = clamp_int(at.tokens);
  return at;
}

// The last of the CTA's runs whose exclusive sum is at most i.
__device__ __forceinline__ int find_run(const int* sums, int i) {
  int a = 0;
  for (int step = blockDim.x >> 1; step > 0; step >>= 1)  // (a power of two)
    if (sums[a + step] <= i) a += step;
  return a;
}

// Consecutive items a thread takes at a time.
__device__ __forceinline__ int group_span(int items, int threads) {
  return items <= threads ? 1 : min(kGroup, (items + threads - 1) / threads);
}

// The number of free blocks, held to what the list can hold.
__device__ __forceinline__ int load_num_free(const int32_t* p, int num_blocks, int* err) {
  const int f = *p;
  if (f < 0 || f > num_blocks) {
    record_error(err, kErrBounds);
    return f < 0 ? 0 : num_blocks;
  }
  return f;
}

// A thread's run of requests [r0, r1) and their two input values; the first
// kGroup of them stay in registers.
struct Run {
  const int32_t *x, *y;
  int r0, r1;
  int a[kGroup], b[kGroup];

  __device__ __forceinline__ void load(int r, int (&u)[kGroup], int (&v)[kGroup]) const {
    if (r + kGroup <= r1 &&
        ((reinterpret_cast<uintptr_t>(x + r) | reinterpret_cast<uintptr_t>(y + r)) & 15) == 0) {
      const int4 p = *reinterpret_cast<const int4*>(x + r), q = *reinterpret_cast<const int4*>(y + r);
      u[0] = p.x, u[1] = p.y, u[2] = p.z, u[3] = p.w;
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
      #pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        u[i] = r + i < r1 ? x[r + i] : 0;
        v[i] = r + i < r1 ? y[r + i] : 0;
      }
    }
  }
  __device__ __forceinline__ Run(const int32_t* x_, const int32_t* y_, int r0_, int r1_)
      : x(x_), y(y_), r0(r0_), r1(r1_) {
    load(r0, a, b);
  }
  template <typename F>
  __device__ __forceinline__ void for_each(F f) const {
    #pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (r0 + i < r1) f(r0 + i, a[i], b[i]);
    #pragma unroll 1
    for (int r = r0 + kGroup; r < r1; r += kGroup) {
      int u[kGroup], v[kGroup];
      load(r, u, v);
      #pragma unroll
      for (int i = 0; i < kGroup; ++i)
        if (r + i < r1) f(r + i, u[i], v[i]);
    }
  }
};
static_assert(kGroup == 4, "vector loads of a group");

// Requests per thread: whole groups where a thread has several.
__device__ __forceinline__ int run_length(int num_reqs) {
  const int each = (num_reqs + blockDim.x - 1) / blockDim.x;
  return each > 1 ? (each + kGroup - 1) / kGroup * kGroup : each;
}

__device__ __forceinline__ Need build_need(const StepParams& p, int base, int n) {
  Need q;
  q.ok = base >= 0 && n >= 0 && (long long)base + n <= (long long)p.max_blocks * kBlockSize;
  q.base = q.ok ? base : 0;
  q.tokens = q.ok ? n : 0;
  q.blocks = blocks_of(q.base + q.tokens) - blocks_of(q.base);
  return q;
}

__global__ void __launch_bounds__(kMaxThreads) build_step_kernel(const StepParams p) {
  __shared__ StepSmem sm;
  const uint32_t rank = cluster_rank(), ctas = gridDim.x;
  const int tid = threadIdx.x, R = p.num_reqs;
  const int each = run_length(R);
  const int r0 = min(tid * each, R), r1 = min(r0 + each, R);
  // The runs whose results this CTA writes.
  const bool mine_to_write = (uint32_t)tid % ctas == rank;
  grid_dependency_wait();
  const int F = load_num_free(p.num_free_in, p.num_blocks, tid == 0 && rank == 0 ? p.err : nullptr);
  if (tid == 0) sm.served_blocks = sm.served_tokens = sm.refused = 0;
  const Run run(p.prev_lens, p.new_tokens, r0, r1);
  Pair sum{0, 0};
  run.for_each([&](int, int len, int n) {
    const Need q = build_need(p, len, n);
    sum.blocks += q.blocks;
    sum.tokens += q.tokens;
  });
  const Pair start = scan_runs(sm, sum);
  // Both sums never fall, so the requests served are those before the first
  // whose blocks or tokens do not fit.
  auto fits = [&](const Need& q, const Pair& end) {
    return q.ok && (q.tokens == 0 || (end.blocks <= F && end.tokens <= p.num_q_tokens));
  };
  int served_b = 0, served_t = 0, refused = 0;
  Pair at = start;
  run.for_each([&](int, int len, int n) {
    const Need q = build_need(p, len, n);
    at.blocks += q.blocks;
    at.tokens += q.tokens;
    const bool go = fits(q, at);
    if (go && q.tokens > 0) {
      served_b = (int)at.blocks;
      served_t = (int)at.tokens;
    }
    refused += !go;
    if (!q.ok && mine_to_write) record_error(p.err, kErrBounds);
  });
  served_b = __reduce_max_sync(0xffffffffu, served_b);
  served_t = __reduce_max_sync(0xffffffffu, served_t);
  refused = __reduce_add_sync(0xffffffffu, refused);
  if ((tid & 31) == 0) {
    if (served_t > 0) {
      atomicMax(&sm.served_blocks, served_b);
      atomicMax(&sm.served_tokens, served_t);
    }
    if (refused > 0) atomicAdd(&sm.refused, refused);
  }
  __syncthreads();
  const int T = sm.served_tokens, N = sm.served_blocks;
  const int threads = blockDim.x * ctas, me = rank * blockDim.x + tid;
  // The slots (a small step's): one search serves up to kGroup consecutive
  // tokens; padding rows get -1.
  const int span = group_span(p.num_q_tokens, threads);
  #pragma unroll 1
  for (int t0 = span * me; ctas == 1 && t0 < p.num_q_tokens; t0 += span * threads) {
    int id[kGroup], off[kGroup];
    int r = 0, first = 0, next = 0, pops = 0;  // of the request: its tokens are [first, next)
    Need q{0, 0, 0, true};
    if (t0 < T) {
      const int at_run = find_run(sm.run_tokens, t0);
      r = at_run * each - 1;
      next = sm.run_tokens[at_run];
      pops = sm.run_blocks[at_run];
    }
    #pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const int t = t0 + u;
      id[u] = off[u] = -1;
      if (u < span && t < T) {
        while (t >= next) {  // (t < T: a request with this token follows)
          pops += q.blocks;
          first = next;
          q = build_need(p, p.prev_lens[r + 1], p.new_tokens[r + 1]), ++r;
          next += q.tokens;
        }
        const int pos = q.base + (t - first), col = pos / kBlockSize, held = blocks_of(q.base);
        id[u] = col < held ? p.block_tables[(long long)r * p.max_blocks + col]
                           : p.free_list[F - 1 - pops - (col - held)];
        off[u] = pos % kBlockSize;
      }
    }
    #pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      if (u >= span || t0 + u >= p.num_q_tokens) break;
      const bool good = (unsigned)id[u] < (unsigned)p.num_blocks;
      if (off[u] >= 0 && !good) record_error(p.err, kErrBounds);
      p.slot_mapping[t0 + u] = off[u] >= 0 && good ? (long long)id[u] * kBlockSize + off[u] : -1;
    }
  }
  // The popped blocks, in request order: pop j is free_list[F - 1 - j].
  for (int j = me; j < N; j += threads) {
    const int id = p.free_list[F - 1 - j];
    const int at_run = find_run(sm.run_blocks, j);
    int r = at_run * each - 1, next = sm.run_blocks[at_run];
    Need q{0, 0, 0, true};
    while (j >= next) {
      q = build_need(p, p.prev_lens[r + 1], p.new_tokens[r + 1]), ++r;
      next += q.blocks;
    }
    p.block_tables[(long long)r * p.max_blocks + blocks_of(q.base) + (j - (next - q.blocks))] = id;
  }
  // query_start_loc: a request after the first refused one starts, like every
  // later one, at the served requests' end.  The lengths follow once every
  // CTA has read the old ones.
  if (mine_to_write) {
    int t = clamp_int(start.tokens);
    run.for_each([&](int r, int len, int n) {
      p.query_start_loc[r] = min(t, T);
      t = clamp_int((long long)t + build_need(p, len, n).tokens);
    });
  }
  if (ctas > 1) cluster_barrier(); else __syncthreads();
  if (mine_to_write) {
    Pair x = start;
    run.for_each([&](int r, int len, int n) {
      const Need q = build_need(p, len, n);
      x.blocks += q.blocks;
      x.tokens += q.tokens;
      p.seq_lens[r] = q.base + (fits(q, x) ? q.tokens : 0);
    });
  }
  if (rank == 0 && tid == 0) {
    p.query_start_loc[R] = T;
    *p.num_free_out = F - N;
    if (p.num_refused) *p.num_refused = sm.refused;
  }
  // The tables and lengths are in place before the next kernel may start:
  // this one never lets it launch early.
  __threadfence();
}

// The slots of a large step, from its finished query_start_loc, lengths and
// tables.  A warp takes 32 consecutive tokens: it finds the first one's
// request together, 32 probes a round, and each lane its own from there.
constexpr int kSlotThreads = 256;
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const StepParams p) {
  grid_dependency_wait();
  const int t = blockIdx.x * kSlotThreads + threadIdx.x, lane = threadIdx.x & 31;
  const int32_t* const qsl = p.query_start_loc;
  const int T = qsl[p.num_reqs];
  int r = 0;  // the last request that starts at or before the warp's first token
  for (int n = p.num_reqs; n > 1;) {
    const int step = (n + 31) / 32, x = lane * step;
    const bool in = x < n && qsl[r + x] <= t - lane;
    const int at = __popc(__ballot_sync(0xffffffffu, in)) - 1;  // starts never fall: a prefix
    r += at * step;
    n = min(step, n - at * step);
  }
  if (t < T) {
    // Mostly within the next 32 requests; then by bisection.
    int b = min(r + 32, p.num_reqs);  // qsl[b] > t
    if (qsl[b] <= t) {
      r = b;
      b = p.num_reqs;
    }
    while (b - r > 1) {
      const int mid = (r + b) >> 1;
      if (qsl[mid] <= t) r = mid; else b = mid;
    }
    const int pos = p.seq_lens[r] - (qsl[r + 1] - t);
    const int id = p.block_tables[(long long)r * p.max_blocks + pos / kBlockSize];
    const bool good = (unsigned)id < (unsigned)p.num_blocks;
    if (!good) record_error(p.err, kErrBounds);
    p.slot_mapping[t] = good ? (long long)id * kBlockSize + pos % kBlockSize : -1;
  } else if (t < p.num_q_tokens) {
    p.slot_mapping[t] = -1;
  }
  __threadfence();
}

__device__ __forceinline__ Need release_need(const ReleaseParams& p, int len, int keep) {
  Need q;
  q.ok = keep >= 0 && keep <= len && (long long)len <= (long long)p.max_blocks * kBlockSize;
  q.base = q.ok ? keep : 0;
  q.tokens = 0;
  q.blocks = q.ok ? blocks_of(len) - blocks_of(keep) : 0;
  return q;
}

__global__ void __launch_bounds__(kMaxThreads) release_blocks_kernel(const ReleaseParams p) {
  __shared__ StepSmem sm;
  const uint32_t rank = cluster_rank(), ctas = gridDim.x;
  const int tid = threadIdx.x, R = p.num_reqs;
  const int each = run_length(R);
  const int r0 = min(tid * each, R), r1 = min(r0 + each, R);
  grid_dependency_wait();
  const int F = load_num_free(p.num_free_in, p.num_blocks, tid == 0 && rank == 0 ? p.err : nullptr);
  if (tid == 0) sm.bad = 0;
  const Run run(p.seq_lens, p.keep_lens, r0, r1);
  Pair sum{0, 0};
  run.for_each([&](int, int len, int keep) {
    const Need q = release_need(p, len, keep);
    sum.blocks += q.blocks;
    if (!q.ok && rank == 0) record_error(p.err, kErrBounds);
  });
  scan_runs(sm, sum);
  __syncthreads();
  // What the list has no room for is a block given back twice somewhere.
  const int M = (int)min(sm.total.blocks, (long long)(p.num_blocks - F));
  if (sm.total.blocks > M && rank == 0 && tid == 0) record_error(p.err, kErrBounds);
  const int threads = blockDim.x * ctas, me = rank * blockDim.x + tid;
  const int span = group_span(M, threads);
  #pragma unroll 1
  for (int j0 = span * me; j0 < M; j0 += span * threads) {
    const int at_run = find_run(sm.run_blocks, j0);
    int r = at_run * each - 1, next = sm.run_blocks[at_run], id[kGroup];
    Need q{0, 0, 0, true};
    #pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      const int j = j0 + u;
      if (u < span && j < M) {
        while (j >= next) {  // (j < M: a request with this block follows)
          q = release_need(p, p.seq_lens[r + 1], p.keep_lens[r + 1]), ++r;
          next += q.blocks;
        }
        id[u] = p.block_tables[(long long)r * p.max_blocks + blocks_of(q.base) + (j - (next - q.blocks))];
      }
    }
    #pragma unroll
    for (int u = 0; u < kGroup; ++u) {
      if (u >= span || j0 + u >= M) break;
      if ((unsigned)id[u] >= (unsigned)p.num_blocks) {
        id[u] = -1;
        atomicAdd(&sm.bad, 1);
        record_error(p.err, kErrBounds);
      }
      p.free_list[F + j0 + u] = id[u];
    }
  }
  if (ctas > 1) cluster_barrier(); else __syncthreads();
  if (rank == 0 && tid < 32) {
    const int b = (uint32_t)tid < ctas ? remote_load(&sm.bad, tid) : 0;
    const int bad = __reduce_add_sync(0xffffffffu, b);
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
  if (ctas > 1) cluster_barrier();  // no CTA leaves while sm.bad may be read
}

template <typename P>
cudaError_t launch(void (*kernel)(const P), const P& p, int ctas, int threads, int cluster,
                   bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// One CTA for small steps: a cluster of eight pays its launch and barrier back
// from a few thousand requests or items on.  Threads are a power of two.
bool one_cta(int num_reqs, long long items) { return num_reqs <= 1024 && items <= 4096; }

template <typename P>
cudaError_t launch_step(void (*kernel)(const P), const P& p, long long items, bool pdl,
                        cudaStream_t stream) {
  if (!one_cta(p.num_reqs, items))
    return launch(kernel, p, kMaxCluster, kMaxThreads, kMaxCluster, pdl, stream);
  const long long widest = items > p.num_reqs ? items : p.num_reqs;
  const int threads = widest <= 256 ? 256 : widest <= 512 ? 512 : kMaxThreads;
  return launch(kernel, p, 1, threads, 1, pdl, stream);
}

}  // namespace

cudaError_t launch_build_step(const StepParams& p, bool pdl, cudaStream_t stream) {
  const cudaError_t e = launch_step(build_step_kernel, p, p.num_q_tokens, pdl, stream);
  if (e != cudaSuccess || one_cta(p.num_reqs, p.num_q_tokens) || p.num_q_tokens == 0) return e;
  const int ctas = (p.num_q_tokens + kSlotThreads - 1) / kSlotThreads;
  return launch(slot_map_kernel, p, ctas, kSlotThreads, 1, pdl, stream);
}

cudaError_t launch_release_blocks(const ReleaseParams& p, bool pdl, cudaStream_t stream) {
  return launch_step(release_blocks_kernel, p, 4ll * p.num_reqs, pdl, stream);
}

}  // namespace pkv
