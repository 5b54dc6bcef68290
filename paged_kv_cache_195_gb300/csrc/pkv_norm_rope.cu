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
// Bound: HBM for chunks, latency for decodes (slot and position, then the
// table's row, then the store).  Sixteen lanes hold a 128-dim head, eight
// elements (16 bytes) each; a head's sum of squares is four shuffles, and a
// pair of a half-split rotation lies in two lanes one shuffle apart.  A thread
// keeps its cos and sin over all the heads that it turns and issues the loads
// of up to four heads before it uses the first.
#include "pkv_latent.h"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16x2_to_float2(in[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t o[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sum of v over the aligned `width` lanes.
template <int WIDTH>
__device__ __forceinline__ float lane_sum(float v) {
  #pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / sqrt(mean of squares + eps) of the N * WIDTH elements that WIDTH lanes
// hold; `pre` is a factor the elements are to be multiplied with first.  Where
// the squares of finite elements leave fp32's range, they are summed again,
// scaled down: x * 2^-70 has squares below 2^116, and eps no weight beside them.
template <int N, int WIDTH>
__device__ __forceinline__ float inv_rms(const float (&x)[N], float eps, float* pre) {
  constexpr float kMean = 1.f / (N * WIDTH);
  float s = 0.f;
  #pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(x[i], x[i], s);
  s = lane_sum<WIDTH>(s);
  *pre = 1.f;
  const bool over = s == INFINITY;
  if (__any_sync(0xffffffffu, over)) {
    float z = 0.f;
    #pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y = x[i] * 0x1p-70f;
      z = fmaf(y, y, z);
    }
    z = lane_sum<WIDTH>(z);
    if (over) {
      *pre = 0x1p-70f;
      return 1.f / sqrtf(z * kMean);
    }
  }
  return 1.f / sqrtf(fmaf(s, kMean, eps));
}

// The cos and sin that a lane needs for its eight dims 8 l .. 8 l + 7 of a
// rotated vector: of the eight pairs that they belong to (half split: dims i
// and i + rot/2) or of the four pairs that they are (interleaved).
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ void load_turn(Turn& r, const float* row, int rot, int l, bool inter) {
  const int half = rot / 2;
  const int i0 = inter ? 4 * l : (8 * l) % half;
  #pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if (i == 4 && inter) break;
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i0 + i));
    r.c[i] = c.x, r.c[i + 1] = c.y, r.c[i + 2] = c.z, r.c[i + 3] = c.w;
    r.s[i] = s.x, r.s[i + 1] = s.y, r.s[i + 2] = s.z, r.s[i + 3] = s.w;
  }
}

// Turns this lane's eight elements; `l` is the lane's place in the vector (and
// in the shuffle's `width` lanes), all of a warp's lanes take part.
__device__ __forceinline__ void turn(float (&x)[8], const Turn& r, int rot, int l, int width,
                                     bool inter) {
  const bool in = 8 * l < rot;
  if (inter) {
    if (in) {
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * r.c[i] - b * r.s[i];
        x[2 * i + 1] = b * r.c[i] + a * r.s[i];
      }
    }
    return;
  }
  const int step = rot / 16;  // lanes between the halves
  const bool low = l < step;
  const int src = !in ? l : low ? l + step : l - step;
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = __shfl_sync(0xffffffffu, x[i], src, width);
    if (in) x[i] = low ? x[i] * r.c[i] - o * r.s[i] : x[i] * r.c[i] + o * r.s[i];
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
__global__ void __launch_bounds__(kRopeThreads) norm_rope_append_kernel(const NormRopeParams p) {
  grid_dependency_wait();  // inputs and pools may belong to the previous kernel
  allow_dependent_launch();
  const int t = blockIdx.x;
  const int sub = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int hq = p.num_q_heads, hkv = p.num_kv_heads;
  const int total = hq + 2 * hkv;
  const long long slot = __ldg(p.slot_mapping + t), pos = __ldg(p.positions + t);
  uint4 raw[U];
  #pragma unroll
  for (int u = 0; u < U; ++u) {
    const int vec = (blockIdx.y * U + u) * (kRopeThreads / 16) + sub;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (vec < total) {
      const __nv_bfloat16* src = vec < hq         ? p.q + t * p.q_stride + vec * kHeadDim
                                 : vec < hq + hkv ? p.k + t * p.k_stride + (vec - hq) * kHeadDim
                                                  : p.v + t * p.v_stride + (vec - hq - hkv) * kHeadDim;
      raw[u] = *reinterpret_cast<const uint4*>(src + 8 * l);
    }
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4 wq = p.q_weight ? __ldg(reinterpret_cast<const uint4*>(p.q_weight) + l) : zero;
  const uint4 wk = p.k_weight ? __ldg(reinterpret_cast<const uint4*>(p.k_weight) + l) : zero;
  if (!token_ok(slot, pos, p.num_blocks, p.max_position, p.err)) return;
  const bool inter = p.interleaved != 0;
  Turn tr;
  if (8 * l < p.rot) load_turn(tr, p.cos_sin + pos * p.rot, p.rot, l, inter);
  const long long blk = slot / kBlockSize;
  const int off = (int)(slot % kBlockSize);
  #pragma unroll
  for (int u = 0; u < U; ++u) {
    const int vec = (blockIdx.y * U + u) * (kRopeThreads / 16) + sub;
    const bool is_q = vec < hq, is_v = vec >= hq + hkv;
    float x[8];
    unpack8(raw[u], x);
    const bool norm = is_q ? p.q_weight != nullptr : p.k_weight != nullptr;
    float pre;
    const float r = inv_rms<8, 16>(x, p.eps, &pre);
    if (norm) {
      float w[8];
      unpack8(is_q ? wq : wk, w);
      #pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * pre * r * w[i];
    }
    turn(x, tr, p.rot, l, 16, inter);
    if (vec >= total) continue;
    __nv_bfloat16* dst;
    if (is_q) {
      dst = p.q_out + t * p.out_stride + vec * kHeadDim;
    } else {
      const int h = is_v ? vec - hq - hkv : vec - hq;
      dst = (is_v ? p.v_pool : p.k_pool) + ((blk * hkv + h) * kBlockSize + off) * kHeadDim;
    }
    *reinterpret_cast<uint4*>(dst + 8 * l) = is_v ? raw[u] : pack8(x);
  }
}

// Block (t, y): warp 0 of the blocks y = 0 writes token t's cache row (the
// latent as 16 elements a lane, two runs of eight; the rotated key on eight
// lanes); all warps turn the queries' vectors, eight lanes each, the first
// vectors by the last warps.
template <int U>
__global__ void __launch_bounds__(kRopeThreads) append_latent_kernel(const AppendLatentParams p) {
  grid_dependency_wait();  // inputs and pool may belong to the previous kernel
  allow_dependent_launch();
  const int t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane & 7;
  const int sub = (kRopeThreads / 32 - 1 - warp) * 4 + (lane >> 3);
  constexpr int kVecs = kRopeThreads / 8;
  const long long slot = __ldg(p.slot_mapping + t), pos = __ldg(p.positions + t);
  const bool row = warp == 0 && blockIdx.y == 0;
  uint4 raw[U], lat[2], key;
  #pragma unroll
  for (int u = 0; u < U; ++u) {
    const int vec = (blockIdx.y * U + u) * kVecs + sub;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (vec < p.num_q_heads)
      raw[u] = *reinterpret_cast<const uint4*>(p.q_rope + t * p.q_stride + vec * p.q_head_stride + 8 * l);
  }
  if (row) {
    const uint4* src = reinterpret_cast<const uint4*>(p.kv + t * p.kv_stride);
    lat[0] = src[lane];
    lat[1] = src[lane + 32];
    key = src[kLatent / 8 + l];
  }
  if (!token_ok(slot, pos, p.num_blocks, p.max_position, p.err)) return;
  const bool inter = p.interleaved != 0;
  Turn tr;
  load_turn(tr, p.cos_sin + pos * kRopeDim, kRopeDim, l, inter);
  if (row) {
    uint4* dst = reinterpret_cast<uint4*>(p.pool + slot * kLatRow);
    if (p.weight != nullptr) {
      float x[16];
      float a[8], b[8];
      unpack8(lat[0], a);
      unpack8(lat[1], b);
      #pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = a[i], x[8 + i] = b[i];
      float pre;
      const float r = inv_rms<16, 32>(x, p.eps, &pre);
      float w0[8], w1[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight) + lane), w0);
      unpack8(__ldg(reinterpret_cast<const uint4*>(p.weight) + lane + 32), w1);
      #pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = a[i] * pre * r * w0[i];
        b[i] = b[i] * pre * r * w1[i];
      }
      lat[0] = pack8(a);
      lat[1] = pack8(b);
    }
    dst[lane] = lat[0];
    dst[lane + 32] = lat[1];
    float x[8];
    unpack8(key, x);
    turn(x, tr, kRopeDim, l, 8, inter);
    if (lane < 8) dst[kLatent / 8 + l] = pack8(x);
  }
  #pragma unroll
  for (int u = 0; u < U; ++u) {
    const int vec = (blockIdx.y * U + u) * kVecs + sub;
    float x[8];
    unpack8(raw[u], x);
    turn(x, tr, kRopeDim, l, 8, inter);
    if (vec < p.num_q_heads)
      *reinterpret_cast<uint4*>(p.q_rope_out + t * p.out_stride + vec * p.out_head_stride + 8 * l) = pack8(x);
  }
}

template <class P>
cudaError_t launch(void (*kernel)(P), const P& p, dim3 grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads);
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

// One vector a thread while the blocks are few (latency), four when they would
// fill the GPU several times over (loads in flight, cos and sin used again).
bool few(long long blocks, int sm_count) { return blocks <= 8ll * sm_count; }

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kVecs = kRopeThreads / 16;
  const int passes = (p.num_q_heads + 2 * p.num_kv_heads + kVecs - 1) / kVecs;
  if (few((long long)p.num_tokens * passes, sm_count))
    return launch(norm_rope_append_kernel<1>, p, dim3(p.num_tokens, passes), stream);
  return launch(norm_rope_append_kernel<4>, p, dim3(p.num_tokens, (passes + 3) / 4), stream);
}

cudaError_t launch_append_latent(const AppendLatentParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kVecs = kRopeThreads / 8;
  const int heads = p.q_rope ? p.num_q_heads : 0;
  const int passes = heads > 0 ? (heads + kVecs - 1) / kVecs : 1;
  if (few((long long)p.num_tokens * passes, sm_count))
    return launch(append_latent_kernel<1>, p, dim3(p.num_tokens, passes), stream);
  return launch(append_latent_kernel<4>, p, dim3(p.num_tokens, (passes + 3) / 4), stream);
}

}  // namespace pkv
