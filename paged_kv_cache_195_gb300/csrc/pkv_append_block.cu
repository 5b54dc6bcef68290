// pkv_append_block.cu -- KV append into e4m3 pools that hold one scale per
// (16-token block, KV head) (pkv_append_fp8_block).
//
// For each block a request's new tokens fall into, and each KV head and
// tensor, with A the largest finite magnitude among the block's new rows:
//     need = the smallest power of two s >= 2^-126 with A / s <= 448
//     s'   = need                     if the block holds no older row
//            max(old scale, need)     otherwise
//     new code = e4m3(x / s'),  kept code = e4m3(decode(code) * s / s')
// (round to nearest even, saturating).  e4m3 is a floating-point format, so a
// power of two costs nothing against the exact ratio A / 448 -- the relative
// step of a normal code is 2^-4 under any scale -- and when a scale grows, a
// kept code only moves its exponent: it loses bits only where it falls under
// the normal range (below 2^-6 of the new scale), so a block rewritten fifteen times
// is not rounded fifteen times.
//
// One warp per (block, KV head, tensor): half a warp reads a 256-byte row, so
// sixteen rows are eight 16-byte loads a lane, all in flight, and the rows
// stay in registers between the maximum and the conversion: each new byte is
// read once.  Kept rows are touched only when the scale grows.  A request's
// blocks are found without a scan: with F(r) = query_start_loc[r] / 16 + 2 r
// every request has F(r + 1) - F(r) >= floor(q_r / 16) + 2 units, at least
// the blocks q_r tokens can touch, and F rises strictly, so a warp finds its
// request by a 32-way search (one round of loads for 32 requests, two for
// 1024); units past the request's last block leave.
//
// Bound: HBM for prefill chunks (512 bytes read and 256 written per token and
// head, K and V); four dependent loads for a decode step.  Measured: eight
// chunks of 512 tokens, eight KV heads, 7.5 us = 3.4 TB/s (0.50 of the measured
// copy rate: a launch and its four loads are 3 us of it); 64 decode tokens, two
// KV heads, 3.1 us.  (With sixty-four inlined divisions for scales that are no
// powers of two and 64-bit indices, 8.2 and 4.0 us: the instruction cache.)
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__global__ void __launch_bounds__(32 * kWarps) append_fp8_block_kernel(const AppendBlockParams p) {
  grid_dependency_wait();  // inputs and pools may belong to the previous kernel
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * kWarps + (threadIdx.x >> 5), uh = w >> 1;
  const int tensor = (int)(w & 1);
  const int unit = (int)(uh / (unsigned)p.num_kv_heads), h = (int)(uh % (unsigned)p.num_kv_heads);
  const int units = p.num_tokens / kBlockSize + 2 * p.num_reqs;
  if (unit >= units) return;
  // The last request with F(r) <= unit; the last round's lanes bring the
  // requests' records along.
  int r = 0, n = p.num_reqs;
  auto before = [&](int x, int start) { return start / kBlockSize + 2 * x <= unit; };
  while (n > 32) {
    const int step = (n + 31) / 32, x = lane * step;
    const bool in = x < n && (x == 0 || before(r + x, __ldg(p.query_start_loc + r + x)));
    const int at = __popc(__ballot_sync(0xffffffffu, in)) - 1;  // F rises: a prefix of the lanes
    r += at * step;
    n = min(step, n - at * step);
  }
  const int own = r + min(lane, n - 1);
  const int s0 = __ldg(p.query_start_loc + own), s1 = __ldg(p.query_start_loc + own + 1);
  const int len = __ldg(p.seq_lens + own);
  const int at = __popc(__ballot_sync(0xffffffffu, lane < n && (lane == 0 || before(own, s0)))) - 1;
  r += at;
  const int q0 = __shfl_sync(0xffffffffu, s0, at), q1 = __shfl_sync(0xffffffffu, s1, at);
  const int L = __shfl_sync(0xffffffffu, len, at), q = q1 - q0;
  if (q == 0) return;
  const int j = unit - (q0 / kBlockSize + 2 * r);
  if (q0 < 0 || q < 0 || q1 > p.num_tokens || q > L ||
      (long long)L > (long long)p.max_blocks * kBlockSize) {
    if (lane == 0) record_error(p.err, kErrBounds);
    return;
  }
  const int P0 = L - q;  // position of the request's first new token
  const int b = P0 / kBlockSize + j;
  if (j < 0 || b >= (L + kBlockSize - 1) / kBlockSize) return;
  const int id = __ldg(p.block_tables + (long long)r * p.max_blocks + b);
  if ((unsigned)id >= (unsigned)p.num_blocks) {
    if (lane == 0) record_error(p.err, kErrBounds);
    return;
  }
  const int f0 = max(P0 - b * kBlockSize, 0);           // rows f0 .. f1 - 1 are new,
  const int f1 = min(L - b * kBlockSize, kBlockSize);   // rows before f0 are kept
  const long long head = (long long)id * p.num_kv_heads + h;
  float* const sp = (tensor ? p.v_scales : p.k_scales) + head;
  const float s_old = f0 > 0 ? *sp : 0.f;
  const int half = lane >> 4, c = lane & 15;  // row parity; 8 elements of the row
  const uint4* src = reinterpret_cast<const uint4*>(tensor ? p.v_new : p.k_new);
  const int t0 = q0 + b * kBlockSize - P0;  // token of row 0 (new rows only)
  uint4 x[8];
  uint32_t top = 0;  // largest finite |x|, as bf16 bits
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 2 * i + half;
    x[i] = make_uint4(0, 0, 0, 0);
    if (row >= f0 && row < f1)
      x[i] = __ldg(src + ((long long)(t0 + row) * p.num_kv_heads + h) * (kHeadDim / 8) + c);
  }
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = in[e] & 0x7fffu, hi = (in[e] >> 16) & 0x7fffu;
      top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  // A = 1.f 2^(E - 127): A / 448 <= 2^(E - 135) while 1.f <= 1.75, else the
  // next power; bf16 bits hold E above seven fraction bits (1.75: 0x60).
  const int ebits = max((int)(top >> 7) - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0), 1);
  const float need = __uint_as_float((uint32_t)ebits << 23);
  const float s_new = f0 > 0 ? fmaxf(s_old, need) : need;
  uint8_t* const rows = (tensor ? p.v_pool : p.k_pool) + head * (kBlockSize * kHeadDim) + c * 8;
  auto store = [&](int row, const uint4& y, auto quotient) {
    const uint32_t in[4] = {y.x, y.y, y.z, y.w};
    uint32_t code[2] = {0u, 0u};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = bf16x2_to_float2(in[e]);
      code[e >> 1] |= e4m3x2(quotient(v.x), quotient(v.y)) << (16 * (e & 1));
    }
    *reinterpret_cast<uint2*>(rows + row * kHeadDim) = make_uint2(code[0], code[1]);
  };
  if ((__float_as_uint(s_new) & 0x7fffffu) == 0) {  // a power of two: x / s is x times 1 / s
    const float inv = 1.f / s_new;
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 2 * i + half;
      if (row >= f0 && row < f1) store(row, x[i], [&](float v) { return v * inv; });
    }
  } else {  // a scale that the block came with (rows read again: less code)
    #pragma unroll 1
    for (int row = half; row < f1; row += 2)
      if (row >= f0)
        store(row, __ldg(src + ((long long)(t0 + row) * p.num_kv_heads + h) * (kHeadDim / 8) + c),
              [&](float v) { return __fdiv_rn(v, s_new); });
  }
  if (f0 > 0 && s_new != s_old) {
    const float ratio = __fdiv_rn(s_old, s_new);
    #pragma unroll 1
    for (int row = half; row < f0; row += 2) {
      uint2* const at = reinterpret_cast<uint2*>(rows + row * kHeadDim);
      const uint2 old = *at;
      const uint32_t in[2] = {old.x, old.y};
      uint32_t code[2];
      #pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 a = e4m3x2_to_float2(in[e] & 0xffffu), bb = e4m3x2_to_float2(in[e] >> 16);
        code[e] = e4m3x2(a.x * ratio, a.y * ratio) | e4m3x2(bb.x * ratio, bb.y * ratio) << 16;
      }
      *at = make_uint2(code[0], code[1]);
    }
  }
  if (lane == 0 && s_new != s_old) *sp = s_new;
}

}  // namespace

cudaError_t launch_append_fp8_block(const AppendBlockParams& p, cudaStream_t stream) {
  const long long units = (long long)p.num_tokens / kBlockSize + 2ll * p.num_reqs;
  const long long blocks = (units * p.num_kv_heads * 2 + kWarps - 1) / kWarps;
  if (blocks > 0x0fffffff) return cudaErrorInvalidValue;  // (8 TB of new rows; warps are 32-bit)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = p.pdl ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, append_fp8_block_kernel, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace pkv
