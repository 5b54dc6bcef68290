// pkv_decode_block.cu -- paged decode attention over e4m3 pools with a scale
// per (16-token block, KV head), the codes fed to the tensor core as they lie
// in the pool.
//
// For a query row and KV head, with ks, vs the scales of key j's block:
//     s_j = scale * <q, decode(K_j)> * ks,   p_j = exp(s_j - max s),
//     out = sum_j p_j * vs * decode(V_j) / sum_j p_j.
//
// No widening.  Both products run on the pool's own bytes (tcgen05
// kind::f8f6f4); what is split instead is the small operand.  A head's q is
// scaled by a power of two so that its largest element lies in [128, 256) and
// written as two e4m3 rows, q = hi + lo / 16 with lo = e4m3(16 (q - hi)): e4m3
// keeps four significant bits and the residual's sign is a fifth, so the pair
// holds bf16's eight exactly for every element whose last bit is no less than
// lo's smallest step, 2^-13 -- from 2^-13 of the largest element's binade up --
// and is off by at most half that step, 2^-14 (2^-21 of that binade), below.
// The eight (at most) heads' hi rows and lo rows are the sixteen columns the
// smallest N of an M = 128 MMA has anyway:
//     S^T[128 keys x (8 hi | 8 lo)] = K[128 x 128 d] . Qhl^T         (A, B K-major)
//
// The probabilities are three e5m2 rows, P = a + b / 8 + c / 64 with b = e5m2(8
// (P - a)), c what is left of 64 (P - a - b / 8): e5m2's three bits, with a sign
// in each remainder, make up the eleven of an f16, and its five exponent bits
// the range.  P lies in [2^11, 2^15) where it is largest, so every weight from
// 2^-23 of the largest on is an f16's rounding, 2^-11 of it, and the smaller ones
// are off by at most 2^-33 of the largest: no row loses its many small weights
// beside a heavy one, however long it is.  (A pair of e4m3 rows ends at 2^-18 of
// the largest: a key of weight 0.9 and value 0 then costs a row of 32768 keys 0.4
// of its output.)
//     O^T[128 d x (G a | G b | G c)] += V^T[128 d x 128 keys] . Pabc^T  (A MN-major)
// fits sixteen columns for groups of up to five heads and takes thirty-two
// beyond; the split costs no tensor time that shows.  A kernel that widens the
// codes to 16 bits in shared memory or TMEM first is bound by that widening's
// latency.
//
// Scales.  ks multiplies the scores after the MMA (a tile's 128 keys are 8
// blocks; TMEM lane = key).  vs joins the probabilities before they are
// rounded: with vs = r 2^lv, r in [1, 2), the value fed to the MMA is
//     P = exp2(s + lv - mo) * r * 2^11,
// where mo is a running maximum of s + lv, next to the running maximum m of s
// that the normaliser uses.  A second maximum because a block that holds most
// of the probability may have a V scale far below its neighbours': P is then
// still of order one where it matters.  The two are raised, and O^T rescaled,
// when a value exceeds its maximum by more than 2^3 (a CTA-wide vote), so P
// stays below 2^15.
//
// Plan, workspace and the log-sum-exp merge are those of the other decode
// kernels (pkv_plan.cuh), but for steps of few rows, which are cut into pieces of
// their own; rows of every request the caller leaves to this kernel, any group
// size 1..8.
//
// Bound: HBM for long steps, the chain of latencies (plan, table, tile, S,
// softmax, PV, merge) for short ones; the tensor pipe is busy 4% of the time.
// Measured, e4m3 codes and scales read over time: 128 rows x 2048 keys, two KV
// heads, 26.1 us = 5.2 TB/s (0.77 of the measured copy rate, launch included;
// the kernel for one scale per head, which widens the codes, 30.4 us); 8 rows x
// 32768 keys, eight KV heads, 86.4 us = 6.2 TB/s (0.92); 1024 rows x 100-500
// keys, two KV heads, 42.6 us = 3.2 TB/s; 64 rows x 512 keys, two KV heads, 8.0
// us; four rows of up to 128 keys, 4.8 us.  (With P in two e4m3 rows 25.9, 86.5,
// 41.7, 8.0 and 4.8: the third row's stores; eight heads 26.4 against 26.2.)
//
// Roles (224 threads, two CTAs per SM): warps 0-3 softmax and epilogue, one
// key (TMEM lane) per thread; warp 4 plans and issues the copies -- K and V
// tiles by TMA into a ring of six 16 KiB slots, the sixteen scales of a tile
// by 4-byte asynchronous copies -- warp 5 issues the MMAs, warp 6 converts
// each piece's q, a piece ahead.
#include <climits>

#include "pkv_internal.h"
#include "pkv_plan.cuh"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

using plan::Piece;
using plan::kEndRow;

constexpr int kWarpProd = 4, kWarpMma = 5, kWarpQ = 6;
constexpr int kThreads = 32 * 7;
constexpr int kTile = 128;                   // keys per tile
constexpr int kBlkPerTile = kTile / kBlockSize;
constexpr int kTileCodes = kTile * kHeadDim; // one K or V tile, bytes
constexpr int kSlots = 6;                    // ring: K of tile t, V of tile t, K of t + 1, ...
constexpr int kScales = 4;                   // tiles whose scales are held (see the producer)
constexpr int kN = 16;                       // MMA N of S: 8 hi columns, 8 lo columns
constexpr int kAtom = 8 * 128;               // 8 operand rows of 128 bytes
constexpr int kPAtoms = 4;                   // operand rows of P, in eights (the most: N = 32)
constexpr uint32_t kColO = 32;               // TMEM columns: S0 0..15, S1 16..31, O0, O1
constexpr float kNegBig = -1.0e30f;
constexpr float kMargin = 3.f;               // log2 of the largest exp2(s - m) allowed
constexpr float kTop = 11.f;                 // P carries 2^kTop: P < 2^(kMargin + 1 + kTop) = 2^15
constexpr float kLo = 16.f;                  // reciprocal of the weight of q's lo rows
constexpr float kPart = 8.f;                 // ... of each row of P relative to the one before
constexpr int kBarSoftmax = 1;
constexpr int kSoftThreads = 128;
constexpr int kPastPiece = INT_MIN;
constexpr int kWindow = 32;                  // block-table entries loaded at a time (4 tiles)

struct __align__(1024) BkSmem {
  uint8_t slot[kSlots][kTileCodes];  // occupant n: K (n even) or V (n odd) of tile n / 2
  uint8_t q[2][2][kAtom];            // [piece buffer][hi | lo][8 heads x 128 d], 128-byte swizzle
  uint8_t pt[2][kPAtoms][kAtom];     // [tile & 1][rows G a, G b, G c x 128 keys]
  float sc[kScales][2][kBlkPerTile]; // [tile % kScales][K | V][block of the tile]
  __align__(16) float qf[2][8];      // [piece buffer]: factor of a head's raw scores (log2 units)
  float4 red[2][4][2];               // per-warp partial maxima (of s, of s + lv), 8 heads
  __align__(16) float st_l[4][8];
  Piece pinfo[2];
  uint64_t pc_full[2];               // piece published by the producer
  uint64_t q_full[2], q_empty[2];    // q converted / read by the piece's last MMA
  uint64_t full[kSlots], empty[kSlots];
  uint64_t sc_full[kScales];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], p_free[2];
  uint64_t o_full[2], o_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  WaitCtl wait;
  int is_last;
  int idle;
};

// Largest value of a warp (NaN skipped), one instruction.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Warp sums of up to eight values in N pairs: value h's sum comes back in the
// lanes with sum_index(lane) == h.  Three halving exchanges spread the values
// over the lanes, two more add up: 9 shuffles for 40.
__device__ __forceinline__ int sum_index(int lane) {
  return (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1);
}

template <int N>
__device__ __forceinline__ float warp_sums(const float2 (&v)[N], int lane) {
  float a[8];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[2 * i] = i < N ? v[i < N ? i : 0].x : 0.f;
    a[2 * i + 1] = i < N ? v[i < N ? i : 0].y : 0.f;
  }
  #pragma unroll
  for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
    const bool up = lane & o;
    #pragma unroll
    for (int h = 0; h < n; ++h) {
      const float keep = up ? a[n + h] : a[h], send = up ? a[h] : a[n + h];
      a[h] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  a[0] += __shfl_xor_sync(0xffffffffu, a[0], 2);
  return a[0] + __shfl_xor_sync(0xffffffffu, a[0], 1);
}

// Two fp32 to two e4m3 codes (the first in the low byte): nearest even,
// saturating, NaN kept.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// hi = e4m3(x) and lo = e4m3(16 (x - hi)) of a pair, low byte first.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = to_e4m3x2(a, b);
  const float2 h = e4m3x2_to_float2(hi);
  lo = to_e4m3x2((a - h.x) * kLo, (b - h.y) * kLo);
}

// a = e5m2(x), b = e5m2(8 (x - a)), c = e5m2(64 (x - a - b / 8)) of a pair
// rounded to f16, low byte first.  The differences are exact in f16.
__device__ __forceinline__ void split_three(float x, float y, uint32_t (&part)[3]) {
  __half2 v = __floats2half2_rn(x, y);
  #pragma unroll
  for (int i = 0; i < 3; ++i) {
    unsigned short code;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;"
        : "=h"(code)
        : "r"(*reinterpret_cast<const uint32_t*>(&v)));
    part[i] = code;
    if (i == 2) break;
    uint32_t back;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(back) : "h"(code));
    v = __hmul2(__hsub2(v, *reinterpret_cast<const __half2*>(&back)), __float2half2_rn(kPart));
  }
}

// 4 bytes global -> shared, asynchronously; `bytes` 0 writes zero instead.
__device__ __forceinline__ void copy4_async(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(bytes)
               : "memory");
}

// Arrive on `bar` once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// mbar_wait with its spin out of line, one copy for all the waits of the kernel.
// The five roles' code is what bounds steps of many short rows: with every spin
// in line, two copies of the MMA warp's PV and of q's conversion one per head,
// the instruction cache missed on a third of its requests (1024 rows of 100-500
// keys, two KV heads: 61.6 us against 45.0 without).
static __device__ __noinline__ bool spin_on(uint64_t* bar, uint32_t parity, int* err, WaitCtl* ctl) {
  return mbar_wait(bar, parity, err, ctl);
}

__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, int* err, WaitCtl* ctl) {
  return mbar_try_wait(bar, parity) || spin_on(bar, parity, err, ctl);
}

// Key row `row` of a staged V tile set to zero.
static __device__ __noinline__ void zero_row(uint8_t* tile, int row) {
  uint4* v = reinterpret_cast<uint4*>(tile + row * 128);
  #pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = make_uint4(0, 0, 0, 0);
}

// The last piece of a split row-group to arrive merges the pieces' partial
// states of output dim d (normalised outputs and (max, normaliser) pairs in
// workspace slots 2 (c0 + s), + 1 for piece 0 when odd0) by log-sum-exp.
template <int G>
static __device__ __noinline__ void merge_row(const float* ws_ml, const float* ws_o,
                                              __nv_bfloat16* out, int c0, int S, int odd0, int d) {
  float M[G], num[G], den[G];
  #pragma unroll
  for (int h = 0; h < G; ++h) {
    M[h] = kNegBig;
    num[h] = den[h] = 0.f;
  }
  // Two pieces' loads in flight at a time (the second repeats the last one
  // when S is odd, and is dropped).
  #pragma unroll 1
  for (int s = 0; s < S; s += 2) {
    float2 ml[2][G];
    float o[2][G];
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = min(s + u, S - 1), slot = 2 * (c0 + x) + ((x == 0 && odd0) ? 1 : 0);
      #pragma unroll
      for (int h = 0; h < G; ++h) {
        const long long at = (long long)slot * G + h;
        ml[u][h] = __ldcg(reinterpret_cast<const float2*>(ws_ml + at * 2));
        o[u][h] = __ldcg(ws_o + at * kHeadDim + d);
      }
    }
    #pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (s + u >= S) break;
      #pragma unroll
      for (int h = 0; h < G; ++h) {
        const float Mn = fmaxf(M[h], ml[u][h].x);
        const float a = fast_exp2(M[h] - Mn), w = fast_exp2(ml[u][h].x - Mn) * ml[u][h].y;
        num[h] = num[h] * a + w * o[u][h];
        den[h] = den[h] * a + w;
        M[h] = Mn;
      }
    }
  }
  #pragma unroll
  for (int h = 0; h < G; ++h)
    out[h * kHeadDim] = __float2bfloat16_rn(den[h] == 0.f ? 0.f : num[h] / den[h]);
}

// The plan of a step with more requests than plan_cta keeps in registers, by
// the whole CTA: every thread sums a contiguous run of requests, the producer
// warp scans the run sums, and only the run that holds the range's first block
// is read again.  (One warp reading all requests twice, 32 at a time, takes
// 0.8 us for every 32 of them.)
struct RunSums {
  long long w[kThreads];
  int nb_min[kThreads / 32], nb_max[kThreads / 32];
  plan::Walker at;  // the result
};

static __device__ plan::Walker find_start(const DecodeParams& p, const RunSums& rs, int per) {
  const int lane = threadIdx.x & 31;
  plan::Walker wk{};
  constexpr int kRuns = kThreads / 32;  // a lane's runs: lane * kRuns ..
  long long part = 0;
  #pragma unroll
  for (int i = 0; i < kRuns; ++i) part += rs.w[lane * kRuns + i];
  const plan::Range rg = plan::finish_range(p, part, rs.nb_min[min(lane, kRuns - 1)],
                                            rs.nb_max[min(lane, kRuns - 1)]);
  wk.rg = rg;
  wk.done = rg.lo >= rg.hi;
  if (wk.done) return wk;
  long long incl = part;
  #pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  long long pos = incl - part;
  const unsigned own = __ballot_sync(0xffffffffu, pos <= rg.lo && rg.lo < incl);
  if (own == 0) {
    record_error(p.err, kErrBounds);  // unreachable when the lengths are stable
    wk.done = true;
    return wk;
  }
  int run = 0;
  const int src = __ffs(own) - 1;
  if (lane == src) {
    run = lane * kRuns;
    #pragma unroll 1
    while (pos + rs.w[run] <= rg.lo) pos += rs.w[run++];
  }
  run = __shfl_sync(0xffffffffu, run, src);
  pos = __shfl_sync(0xffffffffu, pos, src);
  const int end = min(p.num_reqs, (run + 1) * per);
  #pragma unroll 1
  for (int b = run * per; b < end; b += 32) {
    const int r = b + lane;
    long long w = 0;
    if (r < end) {
      const plan::ReqInfo q = plan::load_request(p, r);
      if (q.decode) w = plan::rows_weight(p, q, q.qr) * p.num_kv_heads;
    }
    long long sum = w;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += t;
    }
    const long long before = pos + sum - w;
    const unsigned hit = __ballot_sync(0xffffffffu, w > 0 && before <= rg.lo && rg.lo < before + w);
    if (hit) {
      const int x = __ffs(hit) - 1;
      wk.r = b + x;
      wk.finish_start(p, plan::load_request(p, wk.r), __shfl_sync(0xffffffffu, before, x));
      return wk;
    }
    pos += __shfl_sync(0xffffffffu, sum, 31);
  }
  record_error(p.err, kErrBounds);  // (as above)
  wk.done = true;
  return wk;
}

static __device__ __noinline__ void plan_many(const DecodeParams& p, RunSums& rs) {
  constexpr int kBatch = 4;  // requests whose loads are in flight together
  const int R = p.num_reqs, per = plan::cdiv(R, kThreads), tid = threadIdx.x, lane = tid & 31;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  long long mine = 0;
  int nb_min = INT_MAX, nb_max = 0;
  for (int r = r0; r < r1; r += kBatch) {
    plan::ReqInfo q[kBatch];
    #pragma unroll
    for (int i = 0; i < kBatch; ++i) q[i] = plan::load_request(p, min(r + i, r1 - 1));
    #pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (r + i < r1) plan::tally_request(p, q[i], r + i, mine, nb_min, nb_max);
  }
  rs.w[tid] = mine;
  nb_min = __reduce_min_sync(0xffffffffu, nb_min);
  nb_max = __reduce_max_sync(0xffffffffu, nb_max);
  if (lane == 0) {
    rs.nb_min[tid >> 5] = nb_min;
    rs.nb_max[tid >> 5] = nb_max;
  }
  __syncthreads();
  if ((tid >> 5) != kWarpProd) return;
  const plan::Walker wk = find_start(p, rs, per);
  if (lane == 0) rs.at = wk;
  __syncwarp();
}

template <int G>
__global__ void __launch_bounds__(kThreads, 2)
    decode_block_kernel(const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ DecodeParams p,
                        const int after_prefill) {
  static_assert(G >= 1 && G <= 8, "group size");
  constexpr int kPairs = (G + 1) / 2;
  constexpr int kNO = 3 * G <= 16 ? 16 : 32;                // MMA N of O
  constexpr uint32_t kTmemCols = kColO + 2 * kNO <= 64 ? 64 : 128;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  BkSmem& sm = *reinterpret_cast<BkSmem*>(smem_raw + (((raw + 1023u) & ~1023u) - raw));
  WaitCtl* abort_flag = &sm.wait;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = p.num_kv_heads;
  plan::Range rg;
  plan::Walker wk;
  Piece pc, pn;
  bool have = false, have_n = false;
  // Block-table entries, one window of 32 blocks per load: the current
  // piece's first two and the next piece's, loaded a piece ahead.
  int ent_w0 = kPastPiece, ent_w1 = kPastPiece, ent_n0 = kPastPiece, ent_n1 = kPastPiece;
  auto raw_entries = [&](const Piece& q, int x0) {
    const int x = x0 + lane;
    return x < q.nblk ? __ldg(p.block_tables + (long long)q.r * p.max_blocks + q.b0 + x)
                      : kPastPiece;
  };
  auto advance = [&]() {
    pc = pn;
    have = have_n;
    ent_w0 = ent_n0;
    ent_w1 = ent_n1;
    have_n = have && wk.next<true>(p, pn);
    ent_n0 = have_n ? raw_entries(pn, 0) : kPastPiece;
    ent_n1 = have_n && pn.nblk > kWindow ? raw_entries(pn, kWindow) : kPastPiece;
  };
  // Waits for the kernel ahead, once per warp (see DecodeBlockLaunch).
  auto launch_wait = [&]() {
    if (!after_prefill) grid_dependency_wait();
    allow_dependent_launch();
  };
  const bool many = p.num_reqs > 32 * plan::kPlanRegReqs;
  if (many) {
    if (!p.early_plan && !after_prefill) grid_dependency_wait();
    static_assert(sizeof(RunSums) <= sizeof(sm.slot), "scratch");
    plan_many(p, *reinterpret_cast<RunSums*>(sm.slot));
  }
  if (warp == kWarpProd) {
    if (!p.early_plan) launch_wait();
    if (many)
      wk = reinterpret_cast<const RunSums*>(sm.slot)->at;
    else
      plan::plan_cta<true>(p, lane, rg, wk);
    have_n = true;
    #pragma unroll 1
    for (int i = 0; i < 2; ++i) advance();
    asm volatile("" ::"r"(ent_w0), "r"(ent_w1), "r"(ent_n0), "r"(ent_n1));
    if (lane == 0) sm.idle = !have;
  }
  __syncthreads();
  if (sm.idle) {  // no work: leave, but not before the kernel ahead
    launch_wait();
    if (blockIdx.x == 0) grid_dependency_wait();
    return;
  }

  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.pc_full[b], 1);
      mbar_init(&sm.q_full[b], 1);
      mbar_init(&sm.q_empty[b], 1);
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.s_free[b], 4);
      mbar_init(&sm.p_full[b], 4);
      mbar_init(&sm.p_free[b], 1);
      mbar_init(&sm.o_full[b], 1);
      mbar_init(&sm.o_empty[b], 4);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < kScales; ++s) mbar_init(&sm.sc_full[s], 2 * kBlkPerTile);
    mbar_init(&sm.mma_done, 1);
    sm.wait.abort = 0;
    sm.wait.limit_ns = p.wait_limit_ns;
    fence_barrier_init();
  }
  // Operand rows of padding heads stay zero for the whole kernel.
  for (int i = tid; i < (int)(sizeof(sm.q) + sizeof(sm.pt)) / 16; i += kThreads)
    reinterpret_cast<uint4*>(&sm.q[0][0][0])[i] = make_uint4(0, 0, 0, 0);
  static_assert(offsetof(BkSmem, pt) == offsetof(BkSmem, q) + sizeof(sm.q), "q and pt are adjacent");
  fence_proxy_async_smem();
  if (warp == kWarpProd && lane == 0) {
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
  if (warp == kWarpProd && lane == 0) {  // the first piece, for the q warp
    sm.pinfo[0] = pc;
    mbar_arrive(&sm.pc_full[0]);
  }
  if (warp != kWarpProd || p.early_plan) launch_wait();

  if (warp == kWarpProd) {
    // ========================= plan + copies ===============================
    const int oob_row = p.num_blocks * Hkv * kBlockSize;  // zero-filled by TMA
    const uint64_t pol = l2_policy_evict_first();
    int j = 0, t = 0, n_occ = 0;
    bool ok = true;
    while (ok && have && !abort_flag->abort) {
      const int k = pc.k;
      const int ntile = plan::cdiv(pc.nblk, kBlkPerTile);
      int ent_cur = ent_w0, ent_nxt = ent_w1;
      int ent_nn = ntile > 8 ? raw_entries(pc, 2 * kWindow) : kPastPiece;
      // The piece's buffers are free once the MMAs of piece j - 2 are done.
      const int ub = j & 1;
      if (j >= 2 && !wait_on(&sm.q_empty[ub], ((j >> 1) - 1) & 1, p.err, abort_flag)) break;
      if (lane == 0 && j > 0) {
        sm.pinfo[ub] = pc;
        mbar_arrive(&sm.pc_full[ub]);
      }
      __syncwarp();
      for (int tt = 0; tt < ntile; ++tt, ++t) {
        if (tt > 0 && (tt & 3) == 0) {
          ent_cur = ent_nxt;
          ent_nxt = ent_nn;
          ent_nn = tt + 8 < ntile ? raw_entries(pc, (tt + 8) * kBlkPerTile) : kPastPiece;
        }
        const int phys = __shfl_sync(0xffffffffu, ent_cur, (tt & 3) * kBlkPerTile + (lane & 7));
        const bool good = (unsigned)phys < (unsigned)p.num_blocks;
        if (!good && phys != kPastPiece && lane < 8) record_error(p.err, kErrBounds);
        const int row = good ? (phys * Hkv + k) * kBlockSize : oob_row;
        #pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const int n = 2 * t + kv, s = n % kSlots;
          if (n >= kSlots &&
              !wait_on(&sm.empty[s], ((n / kSlots) - 1) & 1, p.err, abort_flag)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], (uint32_t)kTileCodes);
          __syncwarp();
          if (lane < 8)
            tma_load_2d(sm.slot[s] + lane * 2048, kv ? &vmap : &kmap, 0, row, &sm.full[s], pol);
          if (kv == 0 && lane < 2 * kBlkPerTile) {
            // The tile's scales, K's from lanes 0-7 and V's from lanes 8-15;
            // blocks that are not read get 0.  Their buffer last held tile t
            // - kScales, whose PV is done (its V slot has been refilled), so
            // the softmax has read it.
            static_assert(2 * kScales > kSlots + 1, "scales outlive the tile's ring slots");
            const float* src = (lane < 8 ? p.k_scale : p.v_scale) +
                               (good ? (long long)phys * Hkv + k : 0);
            copy4_async(&sm.sc[t % kScales][lane >> 3][lane & 7], src, good ? 4u : 0u);
            arrive_after_copies(&sm.sc_full[t % kScales]);
          }
          __syncwarp();
          n_occ = n + 1;
        }
        if (!ok) break;
      }
      if (!ok) break;
      ++j;
      advance();
    }
    if (!abort_flag->abort) {
      const int ub = j & 1;  // end marker
      if (j < 2 || wait_on(&sm.q_empty[ub], ((j >> 1) - 1) & 1, p.err, abort_flag)) {
        if (lane == 0) {
          sm.pinfo[ub].row = kEndRow;
          mbar_arrive(&sm.pc_full[ub]);
        }
      }
    }
    if (abort_flag->abort) {
      // Copies in flight land before the CTA's shared memory is released.
      for (int m = max(0, n_occ - kSlots); m < n_occ; ++m)
        mbar_wait_drain(&sm.full[m % kSlots], (m / kSlots) & 1, p.err, abort_flag);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kWarpMma) {
    // ============================ MMA issuer ==============================
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_e4m3_f32(kTile, kN, 0, 0);
      constexpr uint32_t kIdescO = idesc_e4m3_e5m2_f32(kHeadDim, kNO, 1, 0);
      // Descriptors of the first operands: 32 bytes further along a row is 2
      // (16-byte units), 32 rows of V 256.
      const uint64_t dk = smem_desc_sw128(smem_u32(sm.slot[0]), 16, 1024);
      const uint64_t dv = smem_desc_sw128(smem_u32(sm.slot[0]), 1024, 1024);
      const uint64_t dq = smem_desc_sw128(smem_u32(sm.q[0][0]), 16, kAtom);
      const uint64_t dp = smem_desc_sw128(smem_u32(sm.pt[0][0]), 16, kAtom);
      int t = 0;
      bool ok = true;
      auto pv = [&](int tt, bool first, int j) {
        const int n = 2 * tt + 1, s = n % kSlots, ob = j & 1, b = tt & 1;
        const uint32_t tO = tmem + kColO + ob * kNO;
        ok = ok && wait_on(&sm.p_full[b], (tt >> 1) & 1, p.err, abort_flag);
        ok = ok && wait_on(&sm.full[s], (n / kSlots) & 1, p.err, abort_flag);
        if (first && j >= 2)
          ok = ok && wait_on(&sm.o_empty[ob], ((j >> 1) - 1) & 1, p.err, abort_flag);
        if (!ok) return;
        tc_fence_after();
        // V^T is MN-major: one 128-byte atom holds all 128 dims, 8-key
        // groups 1024 bytes apart; 32 keys per MMA.
        const uint64_t da = dv + s * (kTileCodes / 16), db = dp + b * (kPAtoms * kAtom / 16);
        #pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_f8_ss(tO, da + kk * 256, db + kk * 2, kIdescO, !first || kk > 0);
        tc_commit(&sm.empty[s]);
        tc_commit(&sm.p_free[b]);
      };
      for (int j = 0; ok; ++j) {
        const int ub = j & 1;
        if (!wait_on(&sm.q_full[ub], (j >> 1) & 1, p.err, abort_flag)) break;
        const int row = sm.pinfo[ub].row;
        if (row == kEndRow) break;
        const int ntile = plan::cdiv(sm.pinfo[ub].nblk, kBlkPerTile);
        tc_fence_after();
        // S of tile tt, then PV of the tile before it (one copy of each).
        #pragma unroll 1
        for (int tt = 0; tt <= ntile && ok; ++tt) {
          if (tt < ntile) {
            const int b = t & 1, n = 2 * t, s = n % kSlots;
            ok = ok && wait_on(&sm.full[s], (n / kSlots) & 1, p.err, abort_flag);
            if (t >= 2) ok = ok && wait_on(&sm.s_free[b], ((t >> 1) - 1) & 1, p.err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = tmem + b * kN;
            const uint64_t da = dk + s * (kTileCodes / 16), db = dq + ub * (2 * kAtom / 16);
            #pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc_mma_f8_ss(tS, da + kk * 2, db + kk * 2, kIdescS, kk > 0);
            tc_commit(&sm.empty[s]);
            tc_commit(&sm.s_full[b]);
            ++t;
          }
          if (tt > 0) pv(tt < ntile ? t - 2 : t - 1, tt == 1, j);
        }
        tc_commit(&sm.o_full[ub]);
        tc_commit(&sm.q_empty[ub]);
      }
      if (abort_flag->abort) {
        // The MMAs already issued must finish before TMEM is freed.
        tc_commit(&sm.mma_done);
        mbar_wait_drain(&sm.mma_done, 0, p.err, abort_flag);
      }
    }
    __syncwarp();
  } else if (warp == kWarpQ) {
    // ============================ q, a piece ahead ========================
    for (int j = 0;; ++j) {
      const int ub = j & 1;
      if (!wait_on(&sm.pc_full[ub], (j >> 1) & 1, p.err, abort_flag)) break;
      const int row = sm.pinfo[ub].row, k = sm.pinfo[ub].k;
      if (row == kEndRow) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[ub]);
        break;
      }
      // Testing only: the first piece's q never comes, so the waits on it run out.
      if (p.debug_withhold_q && j == 0) continue;
      // Four lanes a head, 32 dims each.
      const int h = lane >> 2, c = lane & 3;
      if (h < G) {
        const uint4* src = reinterpret_cast<const uint4*>(
                               p.q + ((long long)row * p.num_q_heads + (long long)k * G + h) * kHeadDim) +
                           c * 4;
        uint4 x[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __ldg(src + i);
        uint32_t top = 0;
        #pragma unroll
        for (int i = 0; i < 4; ++i)
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                       __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        top = max(top & 0xffffu, top >> 16);
        const unsigned rows = __activemask();
        top = max(top, __shfl_xor_sync(rows, top, 1));
        top = max(top, __shfl_xor_sync(rows, top, 2));
        // sigma = 2^(7 - e) of the largest |q| = 1.f 2^e puts it in [128, 256);
        // a zero or subnormal row is scaled like the smallest normal one.
        // A row with an infinity or a NaN becomes NaN throughout (its scores
        // are undefined).
        const int e = max((int)(top >> 7), 1);  // biased
        const bool finite = e < 255;
        // 2^(134 - e), e biased: 2^-120 .. 2^133, so in two factors; b1 and b2
        // are their inverses.
        const int x1 = (134 - e) / 2, x2 = 134 - e - x1;
        const float s1 = finite ? __uint_as_float((uint32_t)(127 + x1) << 23)
                                : __int_as_float(0x7fc00000);
        const float s2 = __uint_as_float((uint32_t)(127 + x2) << 23);
        const float b1 = finite ? __uint_as_float((uint32_t)(127 - x1) << 23) : s1;
        const float b2 = __uint_as_float((uint32_t)(127 - x2) << 23);
        #pragma unroll 1
        for (int i = 0; i < 4; ++i) {  // 8 dims: half a 16-byte chunk of either row
          const uint4 y4 = __ldg(src + i);
          const uint32_t w[4] = {y4.x, y4.y, y4.z, y4.w};
          uint32_t hi[4], lo[4];
          #pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 f = bf16x2_to_float2(w[y]);
            split_pair(f.x * s1 * s2, f.y * s1 * s2, hi[y], lo[y]);
          }
          const int at = h * 128 + (((c * 2 + (i >> 1)) ^ h) * 16) + (i & 1) * 8;
          *reinterpret_cast<uint2*>(sm.q[ub][0] + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
          *reinterpret_cast<uint2*>(sm.q[ub][1] + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        }
        if (c == 0) sm.qf[ub][h] = p.scale_log2 * b1 * b2;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[ub]);
    }
  } else {
    // ================ softmax + epilogue (warps 0-3) ======================
    const int row = tid, d = tid;  // key `row` of a tile, dim `d` of O^T
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    int t = 0;
    for (int j = 0;; ++j) {
      const int ub = j & 1;
      const bool got = wait_on(&sm.q_full[ub], (j >> 1) & 1, p.err, abort_flag);
      const Piece pc = sm.pinfo[ub];
      // Agree before any barrier: a wait that gave up (abort) stops everyone.
      if (barrier_or(kBarSoftmax, kSoftThreads, !got || pc.row == kEndRow)) break;
      bool ok = true;
      const uint32_t tO = tmem + lane_off + kColO + ub * kNO;
      const int ntile = plan::cdiv(pc.nblk, kBlkPerTile);
      // Heads in pairs; an odd group's last pair has a head whose scores are
      // all -inf.
      float2 m[kPairs], mo[kPairs], l[kPairs], qf[kPairs];
      #pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        m[i] = mo[i] = make_float2(kNegBig, kNegBig);
        l[i] = make_float2(0.f, 0.f);
        qf[i] = *reinterpret_cast<const float2*>(&sm.qf[ub][2 * i]);
        if (2 * i + 1 == G) qf[i].y = 0.f;
      }
      #pragma unroll 1
      for (int tt = 0; tt < ntile; ++tt, ++t) {
        const int b = t & 1;
        ok = ok && wait_on(&sm.sc_full[t % kScales], (t / kScales) & 1, p.err, abort_flag);
        const float ks = sm.sc[t % kScales][0][row >> 4];
        const float vs = sm.sc[t % kScales][1][row >> 4];
        ok = ok && wait_on(&sm.s_full[b], (t >> 1) & 1, p.err, abort_flag);
        tc_fence_after();
        float v[16];
        tmem_ld16(tmem + lane_off + b * kN, v);
        tc_wait_ld();
        const int x = tt * kBlkPerTile + (row >> 4);
        const int pos = (pc.b0 + x) * kBlockSize + (row & 15);
        const bool valid = ok && x < pc.nblk && pos < pc.limit;
        // vs = r 2^lv (a scale that is not finite becomes NaN)
        const int ve = min(max((int)((__float_as_uint(vs) >> 23) & 255u), 1), 253);
        const float lv = (float)(ve - 127);
        const float r = vs - vs == 0.f ? vs * __uint_as_float((uint32_t)(254 - ve) << 23)
                                       : __int_as_float(0x7fc00000);
        // Exponents of the normaliser's and of the MMA's probabilities, and
        // whether one is beyond the margin.
        const float2 lt2 = make_float2(lv + kTop, lv + kTop);
        float2 s[kPairs], y[kPairs], z[kPairs];
        float top_y = -INFINITY, top_z = -INFINITY;
        auto exponents = [&](int i) {
          y[i] = fadd2(s[i], make_float2(-m[i].x, -m[i].y));
          z[i] = fadd2(fadd2(s[i], lt2), make_float2(-mo[i].x, -mo[i].y));
        };
        #pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 c = ffma2(make_float2(v[8 + 2 * i], v[9 + 2 * i]),
                                 make_float2(1.f / kLo, 1.f / kLo), make_float2(v[2 * i], v[2 * i + 1]));
          s[i] = fmul2(c, fmul2(qf[i], make_float2(ks, ks)));
          if (!valid) s[i].x = -INFINITY;
          if (!valid || 2 * i + 1 == G) s[i].y = -INFINITY;
          exponents(i);
          top_y = fmax3(top_y, y[i].x, y[i].y);
          top_z = fmax3(top_z, z[i].x, z[i].y);
        }
        const bool over = top_y > kMargin || top_z > kMargin + kTop;
        // S buffer b has been read: the MMA may overwrite it (tile t + 2).
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_free[b]);
        if (barrier_or(kBarSoftmax, kSoftThreads, over)) {
          // Raise the running maxima to this tile's; O^T and l move along.
          float mx[2][8];
          #pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = i < kPairs ? s[i < kPairs ? i : 0] : make_float2(0.f, 0.f);
            mx[0][2 * i] = i < kPairs ? warp_max(x.x) : 0.f;
            mx[0][2 * i + 1] = 2 * i + 1 < G ? warp_max(x.y) : kNegBig;
            mx[1][2 * i] = i < kPairs ? warp_max(x.x + lv) : 0.f;
            mx[1][2 * i + 1] = 2 * i + 1 < G ? warp_max(x.y + lv) : kNegBig;
          }
          if (lane == 0) {
            #pragma unroll
            for (int x = 0; x < 2; ++x)
              #pragma unroll
              for (int c = 0; c < (G + 3) / 4; ++c)
                sm.red[x][warp][c] = make_float4(mx[x][4 * c], mx[x][4 * c + 1], mx[x][4 * c + 2],
                                                 mx[x][4 * c + 3]);
          }
          // O^T must hold the PV of tile t - 1 before it is rescaled.
          if (tt > 0) ok = ok && wait_on(&sm.p_free[(t - 1) & 1], ((t - 1) >> 1) & 1, p.err, abort_flag);
          named_barrier(kBarSoftmax, kSoftThreads);
          #pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            mx[0][2 * i] = m[i].x;
            mx[0][2 * i + 1] = m[i].y;
            mx[1][2 * i] = mo[i].x;
            mx[1][2 * i + 1] = mo[i].y;
          }
          #pragma unroll
          for (int x = 0; x < 2; ++x)
            #pragma unroll
            for (int c = 0; c < (G + 3) / 4; ++c)
              #pragma unroll
              for (int w = 0; w < 4; w += 2) {
                const float4 y = sm.red[x][w][c], z = sm.red[x][w + 1][c];
                mx[x][4 * c] = fmax3(mx[x][4 * c], y.x, z.x);
                mx[x][4 * c + 1] = fmax3(mx[x][4 * c + 1], y.y, z.y);
                mx[x][4 * c + 2] = fmax3(mx[x][4 * c + 2], y.z, z.z);
                mx[x][4 * c + 3] = fmax3(mx[x][4 * c + 3], y.w, z.w);
              }
          float2 alpha[kPairs];
          bool grow = false;
          #pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const float2 mn = make_float2(mx[0][2 * i], mx[0][2 * i + 1]);
            const float2 mon = make_float2(mx[1][2 * i], mx[1][2 * i + 1]);
            l[i] = fmul2(l[i], make_float2(fast_exp2(m[i].x - mn.x), fast_exp2(m[i].y - mn.y)));
            alpha[i] = make_float2(fast_exp2(mo[i].x - mon.x), fast_exp2(mo[i].y - mon.y));
            grow |= mon.x != mo[i].x || mon.y != mo[i].y;
            m[i] = mn;
            mo[i] = mon;
            exponents(i);
          }
          if (tt > 0 && grow) {
            tc_fence_after();
            auto times = [&](int n, float& x) {
              if (n < 3 * G) x *= n % G & 1 ? alpha[n % G / 2].y : alpha[n % G / 2].x;
            };
            float o[16];
            tmem_ld16(tO, o);
            tc_wait_ld();
            #pragma unroll
            for (int n = 0; n < 16; ++n) times(n, o[n]);
            tmem_st16(tO, reinterpret_cast<const uint32_t(&)[16]>(o));
            if (kNO > 16) {
              float oc[8];
              tmem_ld8(tO + 16, oc);
              tc_wait_ld();
              #pragma unroll
              for (int n = 0; n < 8; ++n) times(16 + n, oc[n]);
              tmem_st8(tO + 16, oc);
            }
            tc_wait_st();
          }
          named_barrier(kBarSoftmax, kSoftThreads);  // sm.red is free again
        }
        // P buffer b was last read by the PV of tile t - 2.
        if (t >= 2) ok = ok && wait_on(&sm.p_free[b], ((t >> 1) - 1) & 1, p.err, abort_flag);
        // Row n of the operand is part n / G of head n % G.
        uint8_t* const rows = sm.pt[b][0] + (row & 15);
        auto put = [&](int n, uint32_t code) {
          rows[(n >> 3) * kAtom + (n & 7) * 128 + (((row >> 4) ^ (n & 7)) * 16)] = (uint8_t)code;
        };
        #pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const int h = 2 * i;
          l[i] = fadd2(l[i], make_float2(fast_exp2(y[i].x), fast_exp2(y[i].y)));
          uint32_t part[3];
          split_three(fast_exp2(z[i].x) * r, fast_exp2(z[i].y) * r, part);
          #pragma unroll
          for (int c = 0; c < 3; ++c) {
            put(c * G + h, part[c]);
            if (h + 1 < G) put(c * G + h + 1, part[c] >> 8);
          }
        }
        // Keys that the row does not see inside its last block -- later tokens of
        // the request, or what lies past its end -- may hold anything (NaN codes
        // too): their V rows become zero, so that 0 * V stays 0.
        if (x < pc.nblk && pos >= pc.limit) {
          const int n = 2 * t + 1, sv = n % kSlots;
          ok = ok && wait_on(&sm.full[sv], (n / kSlots) & 1, p.err, abort_flag);
          zero_row(sm.slot[sv], row);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[b]);
      }
      // ============ epilogue of the piece (same four warps) ================
      const float sw = warp_sums(l, lane);
      if ((lane & 3) == 0) sm.st_l[warp][sum_index(lane)] = sw;
      named_barrier(kBarSoftmax, kSoftThreads);
      const bool okO = ok && wait_on(&sm.o_full[ub], (j >> 1) & 1, p.err, abort_flag);
      tc_fence_after();
      float v[16], vc[8];
      tmem_ld16(tO, v);
      if (kNO > 16) tmem_ld8(tO + 16, vc);
      tc_wait_ld();
      auto column = [&](int n) { return n < 16 ? v[n < 16 ? n : 0] : vc[n >= 16 ? n - 16 : 0]; };
      float o[G], lt[8], mh[G];
      #pragma unroll
      for (int c = 0; c < (G + 3) / 4; ++c) {
        float4 w[4];
        #pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(&sm.st_l[i][4 * c]);
        lt[4 * c] = (w[0].x + w[1].x) + (w[2].x + w[3].x);
        lt[4 * c + 1] = (w[0].y + w[1].y) + (w[2].y + w[3].y);
        lt[4 * c + 2] = (w[0].z + w[1].z) + (w[2].z + w[3].z);
        lt[4 * c + 3] = (w[0].w + w[1].w) + (w[2].w + w[3].w);
      }
      #pragma unroll
      for (int h = 0; h < G; ++h) {
        mh[h] = h & 1 ? m[h / 2].y : m[h / 2].x;
        const float moh = h & 1 ? mo[h / 2].y : mo[h / 2].x;
        // O carries 2^(kTop - mo), the normaliser 2^-m
        const float sum = fmaf(fmaf(column(2 * G + h), 1.f / kPart, column(G + h)), 1.f / kPart, column(h));
        const float num = sum * exp2f(moh - mh[h] - kTop);
        o[h] = lt[h] == 0.f ? 0.f : __fdividef(num, lt[h]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_empty[ub]);
      const bool in_range = pc.row >= 0 && pc.row < p.num_q_tokens && pc.k >= 0 &&
                            pc.k < Hkv && pc.nblk >= 1 && pc.S >= 1 && pc.c0 >= 0 &&
                            2 * (pc.c0 + pc.S) <= p.num_slots && pc.slot >= 0 &&
                            pc.slot < p.num_slots;
      __nv_bfloat16* const out =
          p.out + ((long long)pc.row * p.num_q_heads + (long long)pc.k * G) * kHeadDim + d;
      if (in_range && pc.S == 1) {
        if (okO) {
          #pragma unroll
          for (int h = 0; h < G; ++h) out[h * kHeadDim] = __float2bfloat16_rn(o[h]);
        }
      } else if (in_range) {
        if (okO) {
          #pragma unroll
          for (int h = 0; h < G; ++h) {
            const long long slot = (long long)pc.slot * G + h;
            p.ws_o[slot * kHeadDim + d] = o[h];
            if (d == 0) *reinterpret_cast<float2*>(p.ws_ml + slot * 2) = make_float2(mh[h], lt[h]);
          }
        }
        named_barrier(kBarSoftmax, kSoftThreads);
        if (d == 0) {
          int* cnt = p.ws_cnt + (long long)pc.row * Hkv + pc.k;
          const int old = atom_add_acq_rel_gpu(cnt, 1);
          const int last = (old == pc.S - 1);
          if (last) *cnt = 0;
          sm.is_last = last;
        }
        named_barrier(kBarSoftmax, kSoftThreads);
        if (sm.is_last) merge_row<G>(p.ws_ml, p.ws_o, out, pc.c0, pc.S, pc.odd0, d);
      }
      named_barrier(kBarSoftmax, kSoftThreads);  // sm.st_l and sm.is_last are free again
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
  if (blockIdx.x == 0) grid_dependency_wait();  // (returns at once unless after_prefill)
}

static_assert(sizeof(BkSmem) + 1024 <= (228 * 1024) / 2 - 1024, "two CTAs per SM");

template <int G>
cudaError_t launch_g(const DecodeBlockLaunch& L, cudaStream_t stream) {
  const size_t smem = sizeof(BkSmem) + 1024;  // + alignment slack
  static unsigned long long configured = 0;   // bit per device ordinal
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(decode_block_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(decode_block_kernel<G>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             100);
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
  e = cudaLaunchKernelEx(&cfg, decode_block_kernel<G>, L.kmap, L.vmap, L.p,
                         L.after_prefill);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_block(const DecodeBlockLaunch& L, int group, cudaStream_t stream) {
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
