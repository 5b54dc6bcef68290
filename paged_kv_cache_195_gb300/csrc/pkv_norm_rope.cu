// pkv_norm_rope.cu -- what lies between a layer's projections and its cache:
// root-mean-square norm of each query and key head (or of a latent), rotation
// by the token's position, and the append, in one pass.
//
//   n = w * x / sqrt(mean(x^2) + eps)
//   pair (a, b) at position t with angle i:  a' = a cos - b sin, b' = b cos + a sin
//
// with cos and sin of every (position, pair) in a table that the caller makes
// once, in fp32.  Everything is fp32 from the load to the one rounding to bf16
// at the store.
//
// Bound for chunks: 8 of 512 tokens, 32 + 8 heads of 128 dims take 22 us (4.7 TB/s of
// input and output) with 68 % of the issue slots used and 2.6 TB/s of HBM (what is
// written stays in L2): instructions rather than memory.  A latent and 128 heads' 64
// dims take 27 us (5.4 TB/s, 42 % of the slots): memory.  Decodes (64 tokens: 1.7 and
// 2.0 us) are latency: slot and position, then the table's row, then the store.
// Sixteen lanes hold a 128-dim head, eight lanes the 64 rotated dims of a latent's
// head, each lane two runs of four dims that make four whole pairs -- dims i .. i + 3
// and i + rot/2 .. of a half-split rotation -- so that a rotation needs no shuffles and
// a lane keeps four cos and four sin over all the heads that it turns.  (Eight lanes
// and sixteen dims each: 24 us for 22.)  A thread issues the loads of up to four heads
// before it uses the first.
#include "pkv_latent.h"

namespace pkv {
namespace {

// Small blocks: a token's chain (position, cos and sin, stores) leaves no more of an SM
// idle than its own (256 threads: 8 chunks of 512, 32 + 8 heads 24.1 us for 22.0, 128
// latent heads 29.7 for 26.8; 64 threads: 21.7, but 256 decodes 3.4 us for 2.9).
constexpr int kRopeThreads = 128;
constexpr int kLatentThreads = 128;

// Eight bf16 of a lane, as two runs of four.
struct Raw {
  uint2 a, b;
};

// Where lane l's runs lie in a vector whose leading `rot` dims are rotated.  Lanes
// behind those hold eight dims in a row that stay as they are.
struct Place {
  int a, b;
  bool turned;
};

__device__ __forceinline__ Place place(int l, int rot, bool inter) {
  const bool turned = 8 * l < rot;
  if (inter || !turned) return Place{8 * l, 8 * l + 4, turned};
  return Place{4 * l, rot / 2 + 4 * l, turned};
}

__device__ __forceinline__ Raw load8(const __nv_bfloat16* v, const Place& at) {
  return Raw{*reinterpret_cast<const uint2*>(v + at.a), *reinterpret_cast<const uint2*>(v + at.b)};
}

__device__ __forceinline__ void store8(__nv_bfloat16* v, const Place& at, const Raw& r) {
  *reinterpret_cast<uint2*>(v + at.a) = r.a;
  *reinterpret_cast<uint2*>(v + at.b) = r.b;
}

__device__ __forceinline__ void unpack8(const Raw& r, float2 (&x)[4]) {
  x[0] = bf16x2_to_float2(r.a.x);
  x[1] = bf16x2_to_float2(r.a.y);
  x[2] = bf16x2_to_float2(r.b.x);
  x[3] = bf16x2_to_float2(r.b.y);
}

__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ Raw pack8(const float2 (&x)[4]) {
  return Raw{make_uint2(pack2(x[0]), pack2(x[1])), make_uint2(pack2(x[2]), pack2(x[3]))};
}

// Sum of v over the aligned `WIDTH` lanes.
template <int WIDTH>
__device__ __forceinline__ float lane_sum(float v) {
  #pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// x to x / sqrt(mean of squares + eps) over the N float2 of each of WIDTH lanes;
// where `on` is not set (the same for the WIDTH lanes), x stays.
// rsqrt is off by 2^-22, and the result is rounded to bf16's 2^-8.  Where the
// squares of finite elements leave fp32's range, they are summed again, scaled
// down: x * 2^-70 has squares below 2^116, and eps no weight beside them.
template <int N, int WIDTH>
__device__ __forceinline__ void norm(float2 (&x)[N], float eps, bool on) {
  constexpr float kMean = 1.f / (2 * N * WIDTH);
  float2 s2 = make_float2(0.f, 0.f);
  #pragma unroll
  for (int i = 0; i < N; ++i) s2 = ffma2(x[i], x[i], s2);
  float s = lane_sum<WIDTH>(s2.x + s2.y);
  const bool over = on && s == INFINITY;
  if (__any_sync(0xffffffffu, over)) {
    const float k = over ? 0x1p-70f : 1.f;
    s2 = make_float2(0.f, 0.f);
    #pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = fmul2(x[i], make_float2(k, k));
      s2 = ffma2(x[i], x[i], s2);
    }
    s = lane_sum<WIDTH>(s2.x + s2.y);
    if (over) eps = 0.f;
  }
  const float r = on ? rsqrtf(fmaf(s, kMean, eps)) : 1.f;
  #pragma unroll
  for (int i = 0; i < N; ++i) x[i] = fmul2(x[i], make_float2(r, r));
}

// cos and sin of a lane's four pairs.
struct Turn {
  float4 c, s;
};

__device__ __forceinline__ Turn load_turn(const float* row, int rot, int l) {
  Turn r;
  r.c = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
  r.s = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + 4 * l));
  return r;
}

__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float u = a * c - b * s;
  b = b * c + a * s;
  a = u;
}

// Turns a lane's four pairs: (i, i + 4) of its eight elements, or (2 i, 2 i + 1).
__device__ __forceinline__ void turn(float2 (&x)[4], const Turn& t, bool inter) {
  if (inter) {
    turn_pair(x[0].x, x[0].y, t.c.x, t.s.x);
    turn_pair(x[1].x, x[1].y, t.c.y, t.s.y);
    turn_pair(x[2].x, x[2].y, t.c.z, t.s.z);
    turn_pair(x[3].x, x[3].y, t.c.w, t.s.w);
  } else {
    const float2 c[2] = {make_float2(t.c.x, t.c.y), make_float2(t.c.z, t.c.w)};
    const float2 s[2] = {make_float2(t.s.x, t.s.y), make_float2(t.s.z, t.s.w)};
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = x[i], b = x[i + 2];
      x[i] = ffma2(b, make_float2(-s[i].x, -s[i].y), fmul2(a, c[i]));
      x[i + 2] = ffma2(a, s[i], fmul2(b, c[i]));
    }
  }
}

// A token's slot and position, checked.  Negative slots are padding.
__device__ __forceinline__ bool token_ok(long long slot, long long pos, int num_blocks,
                                         long long max_position, int* err) {
  if (slot < 0) return false;
  if (slot >= (long long)num_blocks * kBlockSize || pos < 0 || pos >= max_position) {
    if (threadIdx.x == 0) record_error(err, kErrBounds);
    return false;
  }
  return true;
}

// Block (t, y): vectors 16 U y .. of token t; its heads in the order q, k, v.
template <int U>
__global__ void __launch_bounds__(kRopeThreads, 9) norm_rope_append_kernel(const NormRopeParams p) {
  grid_dependency_wait();  // inputs and pools may belong to the previous kernel
  allow_dependent_launch();
  constexpr int kVecs = kRopeThreads / 16;
  const int l = threadIdx.x & 15;
  const int hq = p.num_q_heads, hk = hq + p.num_kv_heads, total = hk + p.num_kv_heads;
  const int first = blockIdx.y * (U * kVecs) + (threadIdx.x >> 4);
  const bool inter = p.interleaved != 0;
  const Place at = place(l, p.rot, inter);
  const int t = blockIdx.x;
  const long long slot = __ldg(p.slot_mapping + t), pos = __ldg(p.positions + t);
  Raw raw[U];
  {
    // (each as if its heads were numbered from the token's first vector on)
    const __nv_bfloat16* const q = p.q + t * p.q_stride;
    const __nv_bfloat16* const k = p.k + t * p.k_stride - hq * kHeadDim;
    const __nv_bfloat16* const v = p.v + t * p.v_stride - hk * kHeadDim;
    #pragma unroll
    for (int u = 0; u < U; ++u) {
      const int vec = first + u * kVecs;
      raw[u] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
      if (vec < total) raw[u] = load8((vec < hq ? q : vec < hk ? k : v) + vec * kHeadDim, at);
    }
  }
  Raw wq{make_uint2(0, 0), make_uint2(0, 0)}, wk = wq;
  if (p.q_weight) wq = load8(p.q_weight, at);
  if (p.k_weight) wk = load8(p.k_weight, at);
  if (!token_ok(slot, pos, p.num_blocks, p.max_position, p.err)) return;
  Turn tr{};
  if (at.turned) tr = load_turn(p.cos_sin + pos * p.rot, p.rot, l);
  constexpr int kBlockHead = kBlockSize * kHeadDim;
  const long long row = (slot / kBlockSize * p.num_kv_heads * kBlockSize + slot % kBlockSize) * kHeadDim;
  __nv_bfloat16* const q = p.q_out + t * p.out_stride;
  __nv_bfloat16* const k = p.k_pool + row - hq * kBlockHead;
  __nv_bfloat16* const v = p.v_pool + row - hk * kBlockHead;
  const bool by_q = p.q_weight != nullptr, by_k = p.k_weight != nullptr;
  #pragma unroll
  for (int u = 0; u < U; ++u) {
    const int vec = first + u * kVecs;
    const bool is_q = vec < hq, is_v = vec >= hk;
    // (a warp's two vectors, both values or past the end: nothing to compute)
    if (!__all_sync(0xffffffffu, is_v)) {
      float2 x[4];
      unpack8(raw[u], x);
      if (by_q || by_k) {
        const bool on = is_q ? by_q : by_k && !is_v;
        norm<4, 16>(x, p.eps, on);
        if (on) {
          float2 w[4];
          unpack8(is_q ? wq : wk, w);
          #pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = fmul2(x[i], w[i]);
        }
      }
      if (at.turned) turn(x, tr, inter);
      if (!is_v) raw[u] = pack8(x);
    }
    if (vec < total) store8((is_q ? q : is_v ? v : k) + vec * (is_q ? kHeadDim : kBlockHead), at, raw[u]);
  }
}

// Block (t, y): warp 0 of the blocks y = 0 writes token t's cache row (the
// latent as 16 elements a lane; the rotated key on eight lanes); all warps turn
// the queries' vectors, eight lanes each, the first vectors by the last warps.
template <int U>
__global__ void __launch_bounds__(kLatentThreads, 8) append_latent_kernel(const AppendLatentParams p) {
  grid_dependency_wait();  // inputs and pool may belong to the previous kernel
  allow_dependent_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 7;
  constexpr int kVecs = kLatentThreads / 8;
  const int first = blockIdx.y * (U * kVecs) + (kLatentThreads / 32 - 1 - warp) * 4 + (lane >> 3);
  const bool inter = p.interleaved != 0;
  const Place at = place(l, kRopeDim, inter);
  const int t = blockIdx.x;
  const long long slot = __ldg(p.slot_mapping + t), pos = __ldg(p.positions + t);
  const bool row = warp == 0 && blockIdx.y == 0;
  Raw raw[U], key;
  uint4 lat[2];
  #pragma unroll
  for (int u = 0; u < U; ++u) {
    const int vec = first + u * kVecs;
    raw[u] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
    if (vec < p.num_q_heads) raw[u] = load8(p.q_rope + t * p.q_stride + vec * p.q_head_stride, at);
  }
  if (row) {
    const uint4* src = reinterpret_cast<const uint4*>(p.kv + t * p.kv_stride);
    lat[0] = src[lane];
    lat[1] = src[lane + 32];
    key = load8(p.kv + t * p.kv_stride + kLatent, at);
  }
  if (!token_ok(slot, pos, p.num_blocks, p.max_position, p.err)) return;
  const Turn tr = load_turn(p.cos_sin + pos * kRopeDim, kRopeDim, l);
  if (row) {
    __nv_bfloat16* dst = p.pool + slot * kLatRow;
    if (p.weight != nullptr) {
      const uint4* const wp = reinterpret_cast<const uint4*>(p.weight);
      float2 x[8];
      #pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[4 * h] = bf16x2_to_float2(lat[h].x);
        x[4 * h + 1] = bf16x2_to_float2(lat[h].y);
        x[4 * h + 2] = bf16x2_to_float2(lat[h].z);
        x[4 * h + 3] = bf16x2_to_float2(lat[h].w);
      }
      norm<8, 32>(x, p.eps, true);
      #pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 w = __ldg(wp + lane + 32 * h);
        lat[h] = make_uint4(pack2(fmul2(x[4 * h], bf16x2_to_float2(w.x))),
                            pack2(fmul2(x[4 * h + 1], bf16x2_to_float2(w.y))),
                            pack2(fmul2(x[4 * h + 2], bf16x2_to_float2(w.z))),
                            pack2(fmul2(x[4 * h + 3], bf16x2_to_float2(w.w))));
      }
    }
    reinterpret_cast<uint4*>(dst)[lane] = lat[0];
    reinterpret_cast<uint4*>(dst)[lane + 32] = lat[1];
    float2 x[4];
    unpack8(key, x);
    turn(x, tr, inter);
    if (lane < 8) store8(dst + kLatent, at, pack8(x));
  }
  #pragma unroll
  for (int u = 0; u < U; ++u) {
    const int vec = first + u * kVecs;
    if (vec < p.num_q_heads) {
      float2 x[4];
      unpack8(raw[u], x);
      turn(x, tr, inter);
      store8(p.q_rope_out + t * p.out_stride + vec * p.out_head_stride, at, pack8(x));
    }
  }
}

template <class P>
cudaError_t launch(void (*kernel)(P), const P& p, dim3 grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = p.pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// Vectors a thread holds of the `passes` over a block that a token has: one while
// the blocks are few (latency), up to four, as evenly as it goes, when they would
// fill the GPU several times over (loads in flight, cos and sin used again).
int vectors(long long tokens, int passes, int sm_count) {
  if (tokens * passes <= 16ll * sm_count) return 1;
  const int blocks = (passes + 3) / 4;
  return (passes + blocks - 1) / blocks;
}

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kVecs = kRopeThreads / 16;
  const int passes = (p.num_q_heads + 2 * p.num_kv_heads + kVecs - 1) / kVecs;
  const int u = vectors(p.num_tokens, passes, sm_count);
  const dim3 grid(p.num_tokens, (passes + u - 1) / u);
  switch (u) {
    case 1: return launch(norm_rope_append_kernel<1>, p, grid, kRopeThreads, stream);
    case 2: return launch(norm_rope_append_kernel<2>, p, grid, kRopeThreads, stream);
    case 3: return launch(norm_rope_append_kernel<3>, p, grid, kRopeThreads, stream);
    default: return launch(norm_rope_append_kernel<4>, p, grid, kRopeThreads, stream);
  }
}

cudaError_t launch_append_latent(const AppendLatentParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kVecs = kLatentThreads / 8;
  const int passes = p.num_q_heads > 0 ? (p.num_q_heads + kVecs - 1) / kVecs : 1;
  const int u = vectors(p.num_tokens, passes, sm_count);
  const dim3 grid(p.num_tokens, (passes + u - 1) / u);
  switch (u) {
    case 1: return launch(append_latent_kernel<1>, p, grid, kLatentThreads, stream);
    case 2: return launch(append_latent_kernel<2>, p, grid, kLatentThreads, stream);
    case 3: return launch(append_latent_kernel<3>, p, grid, kLatentThreads, stream);
    default: return launch(append_latent_kernel<4>, p, grid, kLatentThreads, stream);
  }
}

}  // namespace pkv
