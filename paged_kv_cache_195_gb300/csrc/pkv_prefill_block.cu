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
// 256) and split into two operands, hi = e4m3(q) and lo = e5m2(q - hi), whose
// products accumulate in one TMEM tile.  bf16's eight bits are hi's four, lo's
// sign and lo's three, and lo needs e5m2's range where hi is subnormal: the split
// is exact from 2^-13 of the largest element's binade up, and off by at most
// 2^-20 of that binade below (lo in e4m3: from 2^-9, and 2^-17).  Twice the MMAs
// at twice the bf16 rate: the tensor time of a bf16 K, none of its widening.  A
// key's block scale multiplies its column of S in the softmax.
//
// O += P V takes f16: P rows are 128 wide here, and splitting 128 x 128
// probabilities in the softmax, which sets the pace, would cost more than
// widening V once per tile in warps of its own (one hardware conversion per
// pair of codes; every e4m3 value is an f16 value).  The value scales join the
// probabilities: with 2^lv <= vs < 2^(lv + 1) of key j's block,
//     P = exp2(s - m) * F,   F = exp2(m - mo + 6) * vs
// is at most 2^15, mo being a running maximum of s + lv next to the running
// maximum m of s that the normaliser uses; both are raised when exceeded by
// more than 2^8.  So P is precise where it weighs, however far apart the
// blocks' scales are, and F is one factor per row and block.  (bf16 for V, its
// scale multiplied in while widening, needs no F but six instructions a pair of
// codes where one does, and would leave the probabilities eight bits for f16's
// eleven.)
//
// Roles (640 threads): warps 0-15 softmax and epilogue, four threads per MMA
// row (warps with the same index mod 4 hold the same 32 rows); warp 16 takes
// items from the work queue and copies Q, K and V tiles and the scales; 17
// issues the MMAs; 18 and 19 widen V.  Items travel through a four-entry ring
// that every role reads, published a few tiles before the previous item ends,
// with its Q on the way; when an item's last probabilities are out the softmax
// warps split the next one's Q (in place: a row's 256 bytes of bf16 become its
// 128 of hi and 128 of lo) and write the item's output while its first S runs.
// The MMA warp issues an item's last PVs before it waits for the next item's Q:
// the softmax may be waiting for one of them to rescale O, and splits that Q
// only afterwards.
//
// NaN.  A masked probability is 0, and 0 times a NaN code would spoil rows that
// must not see its key.  So the converters set the NaN codes of keys that only
// some of an item's rows see to zero, and note in which dims and from which
// token on; the epilogue writes the NaNs of those rows.  (Keys that every row
// sees are left alone, keys that none does become zero.)
//
// A step with fewer items than CTAs cuts the longer ones over their keys, into
// equal parts of four key tiles or more, each an item of the queue; a part leaves its
// normalised output and (maximum, normaliser) per row in the workspace, and the
// last to arrive merges them by log-sum-exp in part order.  (One chunk of 64
// tokens on 30000 keys, 12 query and two KV heads: 51 us against 333 whole; 16
// chunks of 16 on 500-2000 keys: 21 against 29.  At two parts per CTA the merges
// cost more than the balance gains: 30 us on those, 44 against 40 on a mixed step.)
//
// Bound: the softmax, about 3000 cycles for a tile of 128 x 128 scores of which
// the tensor pipe is busy a third (16 MMAs of 64 cycles) and the exponentials
// take 1000; the rest is issue slots (56% used) and the latencies between a
// tile's scores, maxima and probabilities.  Hence the pipeline inside each
// softmax warp: the scores of tile t + 1 are fetched from TMEM, half a tile at a
// time into the registers that the exponentials of tile t have freed, and P has
// TMEM columns of its own, so that a score buffer is free as soon as it is read.
//
// Measured: eight 512-token chunks after prefixes of up to 4096 tokens, 32 query
// and 8 KV heads: 145 us = 742 TFLOP/s of the 2 x 2 x 128 flops per visible key
// and query head, 0.39 of cuBLAS's bf16 rate (the bf16 prefill kernel: 129 us).
// Of that, 1 us is the largest factors' way into the exponents; 64 chunks of 9
// tokens on 500-1000 keys, eight KV heads, take 55.6 us, 52.5 without the notes
// of NaNs.
#include <climits>

#include "pkv_internal.h"
#include "pkv_tc.cuh"

namespace pkv {
namespace {

constexpr int kParts = 4;                // softmax threads per MMA row
constexpr int kPartKeys = 128 / kParts;  // keys (and output dims) per softmax thread
constexpr int kSoftWarps = 4 * kParts;
constexpr int kWarpLoad = kSoftWarps;    // items, K and V tiles
constexpr int kWarpMma = kSoftWarps + 1;
constexpr int kWarpConv = kSoftWarps + 2;
constexpr int kConvWarps = 2;
constexpr int kThreads = 32 * (kWarpConv + kConvWarps);
constexpr int kBarQuad = 1;              // + quad: the four warps holding the same 32 rows
constexpr int kRows = kPrefillRows;      // MMA M
constexpr int kKeyTile = 128;
constexpr int kBlkPerTile = kKeyTile / kBlockSize;
constexpr int kCodes = kKeyTile * kHeadDim;  // a K or V tile, or a Q operand, in bytes
constexpr int kHalfBytes = kKeyTile * 128;   // one 64-dim half of a widened V tile
// TMEM columns: S0 0..127, S1 128..255, O 256..383, P0 384..447, P1 448..511.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256, kColP = 384;
constexpr float kMargin = 8.0f;          // log2 of the largest exp2(s - m) allowed
constexpr float kTop = 6.0f;             // P carries 2^kTop: below 2^(kMargin + 1 + kTop) = 2^15
constexpr float kNegBig = -1.0e30f;
constexpr float kTopF = 100.f;           // log2 of the largest F, about
constexpr float kMostF = 0x1p100f;
constexpr int kPastEnd = INT_MIN;        // block-table slot past the request (not read)
constexpr int kStages = 3;               // K stages
constexpr int kStagesV = 2;              // V stages (codes)
constexpr int kItems = 4;                // item ring
constexpr int kAhead = 4;                // an item is published this many tiles before the
                                         // previous one's last copies
constexpr int kNanRing = 3;              // items whose NaN notes are held (see note_nans)
constexpr int kNoNan = 255;
constexpr int kScaleRing = 8;            // tiles whose scales are held
constexpr int kMaxSplit = 16;            // parts of an item's keys
constexpr int kMinPart = 4;              // key tiles a part is worth

struct Item {
  int r, k;   // request, KV head
  int row0;   // first query row of the tile
  int nt;     // valid tokens in the tile
  int pos0;   // position of its first token
  int L;      // request length
  int j0;     // first key tile
  int nj;     // key tiles
  int parts;  // parts of the item's keys (1: this is all of them)
  int part;   // this one
  int slot;   // its partial state; the others' are beside it, in order
  int end;    // no more items
};

struct __align__(1024) Smem {
  uint8_t q[2][2][kCodes];           // [item & 1][hi | lo] (first: dims 0..63 | 64..127 in bf16)
  uint8_t k[kStages][kCodes];
  uint8_t v[kStagesV][kCodes];       // V codes
  uint8_t vb[2][2][kHalfBytes];      // widened V: [buffer][d half]
  float2 xrow[kParts][kRows];        // [key part][row]: partial row maxima, then normalisers
  float qf[kItems][kRows];           // factor of a row's raw scores (log2 units)
  float sc[kScaleRing][2][kBlkPerTile];  // [K | V] scales of a tile's blocks
  Item items[kItems];
  uint64_t it_full[kItems], it_free[kItems];
  uint64_t qr_full[2], q_full[kItems], q_empty[2];  // raw Q landed / split / read by its last S
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStagesV], v_empty[kStagesV];
  uint64_t sc_full[kScaleRing];
  uint64_t vb_full[2], vb_free[2];
  uint64_t s_full[2], s_free[2], p_full[2], p_free[2];
  uint64_t o_full, o_empty;
  uint64_t mma_done;
  uint32_t tmem_base;
  long long counts[kThreads / 32];   // items, by the warp that counted them
  int batch_items[kMaxReqs / 32];    // items (parts) of 32 requests
  int n_active;
  int longest_part;                  // key tiles of a split item's longest part (0: none is)
  uint2 extents[kThreads / 32];      // key tiles, the longest request's, by warp
  int last[4];                       // [quad]: the last part to arrive
  // NaN values among the keys that only some rows see, by converter warp: the
  // item that the notes are of; a dim's first such key, counted from the first
  // token's own.
  int nan_item[kNanRing][kConvWarps];
  __align__(16) uint8_t nan_from[kNanRing][kConvWarps][kHeadDim];
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

// Two fp32 to e4m3 or e5m2 codes (the first in the low byte).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint32_t to_e5m2x2(float a, float b) {
  unsigned short r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Four codes (low byte first) to two f16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Waits for the TMEM loads into a and b (as operands, so that nothing reads
// them earlier).
__device__ __forceinline__ void wait_ld32(float (&a)[16], float (&b)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(a[0]), "+f"(a[1]), "+f"(a[2]), "+f"(a[3]), "+f"(a[4]), "+f"(a[5]),
                 "+f"(a[6]), "+f"(a[7]), "+f"(a[8]), "+f"(a[9]), "+f"(a[10]), "+f"(a[11]),
                 "+f"(a[12]), "+f"(a[13]), "+f"(a[14]), "+f"(a[15]), "+f"(b[0]), "+f"(b[1]),
                 "+f"(b[2]), "+f"(b[3]), "+f"(b[4]), "+f"(b[5]), "+f"(b[6]), "+f"(b[7]),
                 "+f"(b[8]), "+f"(b[9]), "+f"(b[10]), "+f"(b[11]), "+f"(b[12]), "+f"(b[13]),
                 "+f"(b[14]), "+f"(b[15])
               :
               : "memory");
}

// Bit 7 of every byte whose code is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// A converter warp's 32 rows `row` on of a staged V tile (first key `key0`),
// whose rows beyond the first token's own position pos0 and below `end` hold a
// NaN code somewhere: those codes become zero, and are noted for item n.  Notes
// of item n - kNanRing are no longer read: a converter is two tiles ahead of PV
// at most, hence past item n - 1 only when item n - 2's probabilities are out,
// which follow item n - 3's epilogue.
static __device__ __noinline__ void note_nans(Smem& sm, uint8_t* tile, int row, int key0, int pos0, int end,
                                              int n) {
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kWarpConv;
  uint32_t* const from = reinterpret_cast<uint32_t*>(sm.nan_from[n % kNanRing][w]) + lane;  // 4 dims a lane
  const bool first = sm.nan_item[n % kNanRing][w] != n;
  __syncwarp();
  if (first) {
    *from = kNoNan * 0x01010101u;
    if (lane == 0) sm.nan_item[n % kNanRing][w] = n;
  }
  for (int i = row; i < row + 32; ++i) {
    const int key = key0 + i;
    if (key <= pos0 || key >= end) continue;
    uint32_t* const at = reinterpret_cast<uint32_t*>(tile + i * 128 + (((lane >> 2) ^ (i & 7)) * 16)) + (lane & 3);
    const uint32_t bad = nan_bytes(*at) >> 7;
    if (bad == 0) continue;
    *at &= ~(bad * 0xffu);
    *from = __vminu4(*from, (uint32_t)(key - pos0) * bad | ~(bad * 0xffu));
  }
  __syncwarp();
}

// The noted NaNs of item n into a row's 32 output dims.
__device__ __forceinline__ void put_nans(const Smem& sm, int n, int part, int token, float (&x0)[16],
                                         float (&x1)[16]) {
  #pragma unroll 1
  for (int w = 0; w < kConvWarps; ++w) {
    if (sm.nan_item[n % kNanRing][w] != n) continue;
    const uint8_t* from = sm.nan_from[n % kNanRing][w] + part * kPartKeys;
    #pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (from[i] <= token) x0[i] = __int_as_float(0x7fc00000);
      if (from[16 + i] <= token) x1[i] = __int_as_float(0x7fc00000);
    }
  }
}

// The exponent of a block's value scale: 2^lv <= vs < 2^(lv + 1) (0 and
// subnormals: -127).
__device__ __forceinline__ float scale_exponent(float vs) {
  return __uint_as_float((__float_as_uint(vs) >> 23) | 0x4b000000u) - (8388608.f + 127.f);
}

// The softmax warps split an item's Q in place: q holds its two 64-dim halves
// in bf16 and gets the hi and the lo operand; qf gets the rows' factors of the
// raw scores, bar every warp's arrival.  Warp w takes rows 8w .. 8w + 7, four
// threads a row, 32 dims each.  (Out of line it costs more than the registers
// that it would spare the tile loop: 151 against 146.5 us on eight 512-token
// chunks.)
static __device__ __forceinline__ void split_q(uint8_t* q, float scale_log2, float* qf, uint64_t* bar) {
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3, sw = r & 7;
  q += r * 128;
  uint4 x[4];
  uint32_t top = 0;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = lds128(q + (c >> 1) * kCodes + ((((c & 1) * 4 + i) ^ sw) * 16));
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                 __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
  }
  top = max(top & 0xffffu, top >> 16);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  __syncwarp();  // the row's four threads (one warp) have read it
  // sigma = 2^(134 - e), e the largest element's biased exponent (from 7 on:
  // below 2^-120 a row is as good as zero); NaN for a row that is not finite.
  // The sign of the softmax scale goes to q, so that a tile's largest score is
  // its largest column times its factor.
  const int e = max((int)(top >> 7), 7);
  const float sigma = e < 255 ? __uint_as_float((uint32_t)(261 - e) << 23)
                              : __int_as_float(0x7fc00000);
  const float s = scale_log2 < 0.f ? -sigma : sigma;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t hi[4], lo[4];
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = bf16x2_to_float2(w[k]);
      const float a = f.x * s, b = f.y * s;
      hi[k] = to_e4m3x2(a, b);
      const float2 back = e4m3x2_to_float2(hi[k]);
      lo[k] = to_e5m2x2(a - back.x, b - back.y);
    }
    uint8_t* const at = q + ((c * 2 + (i >> 1)) ^ sw) * 16 + (i & 1) * 8;
    *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    *reinterpret_cast<uint2*>(at + kCodes) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  }
  if (c == 0) qf[r] = scale_log2 / s;
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Partial states lie with a row's neighbours next to it: float4 c of the 32 of
// row r of slot s at (32 s + c) * 128 + r, so that a warp's accesses are whole
// lines.  The merge of an item's parts (slots `first` on) for one row and 32 of
// its dims, by log-sum-exp: a part's weight is 2^m l.
static __device__ __forceinline__ void merge_parts(const PrefillBlockParams& pb, long long first, int parts,
                                                int row, int part, __nv_bfloat16* dst) {
  float M = kNegBig, den = 0.f;
  #pragma unroll 1
  for (int s = 0; s < parts; ++s) {
    const float2 ml = __ldcg(pb.part_ml + (first + s) * kRows + row);
    const float Mn = fmaxf(M, ml.x);
    den = den * fast_exp2(M - Mn) + fast_exp2(ml.x - Mn) * ml.y;
    M = Mn;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  float4 x[8];
  #pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll 1
  for (int s = 0; s < parts; ++s) {
    const float4* o = pb.part_o + ((first + s) * 32 + part * 8) * kRows + row;
    float4 a[8];
    #pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = __ldcg(o + i * kRows);
    const float2 ml = __ldcg(pb.part_ml + (first + s) * kRows + row);
    const float w = fast_exp2(ml.x - M) * ml.y * inv;
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i].x += w * a[i].x;
      x[i].y += w * a[i].y;
      x[i].z += w * a[i].z;
      x[i].w += w * a[i].w;
    }
  }
  #pragma unroll
  for (int i = 0; i < 8; i += 2)
    reinterpret_cast<uint4*>(dst)[i / 2] =
        make_uint4(pack_bf16x2(x[i].x, x[i].y), pack_bf16x2(x[i].z, x[i].w),
                   pack_bf16x2(x[i + 1].x, x[i + 1].y), pack_bf16x2(x[i + 1].z, x[i + 1].w));
}

// The epilogue of one part of item n: its state to memory, and the merge by the
// part that arrives last -- each quad of warps by itself, whose rows are complete
// in all parts.  Out of line, which keeps its registers out of the tile loop.
template <int G>
static __device__ __noinline__ void finish_part(Smem& sm, const PrefillBlockParams& pb, int n,
                                                uint32_t tO, float m, float l, float inv, bool write,
                                                __nv_bfloat16* dst) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, part = warp >> 2;
  const int row = quad * 32 + lane;
  float x0[16], x1[16];
  tmem_ld16(tO, x0);
  tmem_ld16(tO + 16, x1);
  wait_ld32(x0, x1);
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.o_empty);
  put_nans(sm, n, part, row / G, x0, x1);
  const Item& it = sm.items[n % kItems];
  if (quad * 32 >= it.nt * G) return;  // no query in these rows
  const int slot = it.slot, parts = it.parts;
  if (write) {
    float4* o = pb.part_o + ((long long)slot * 32 + part * 8) * kRows + row;
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i * kRows] = make_float4(x0[4 * i] * inv, x0[4 * i + 1] * inv, x0[4 * i + 2] * inv, x0[4 * i + 3] * inv);
      o[(4 + i) * kRows] =
          make_float4(x1[4 * i] * inv, x1[4 * i + 1] * inv, x1[4 * i + 2] * inv, x1[4 * i + 3] * inv);
    }
    if (part == 0) pb.part_ml[slot * kRows + row] = make_float2(m, l);
  }
  named_barrier(kBarQuad + quad, 128);
  if (part == 0 && lane == 0) {
    // (a row of the item for each quad that has one: 32 quad < G nt)
    int* const cnt = pb.cnt + (long long)(it.row0 + quad) * pb.p.num_kv_heads + it.k;
    const int old = atom_add_acq_rel_gpu(cnt, 1);
    sm.last[quad] = old == parts - 1;
    if (old == parts - 1) *cnt = 0;
  }
  named_barrier(kBarQuad + quad, 128);
  if (sm.last[quad] && write) merge_parts(pb, slot - it.part, parts, row, part, dst);
}

// kSplit: whether items may be cut over their keys.  (A variant of its own for
// steps that hold too many items for that: the calls of the other one cost the
// tile loop registers, 150 against 145 us on eight 512-token chunks.)
template <int G, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_block_kernel(const __grid_constant__ CUtensorMap qmap,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ PrefillBlockParams pb) {
  constexpr int TQ = kRows / G;  // query tokens per item
  const PrefillParams& p = pb.p;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + (((raw + 1023u) & ~1023u) - raw));
  WaitCtl* abort_flag = &sm.wait;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hkv = p.num_kv_heads;

  // Ordering.  This is the call's first kernel: it waits for the kernel ahead
  // (before reading the lengths, unless early_plan says that they are not that
  // kernel's to write) and only then lets the decode kernel launch, which
  // reads nothing that this one writes and takes the SMs that have no item
  // here, or no longer.
  if (!pb.early_plan) grid_dependency_wait();
  // CTAs without an item leave before any set-up.
  auto count_batches = [&](auto items_of) {  // into sm.batch_items; this warp's sum
    long long count = 0;
    for (int b = warp; b * 32 < p.num_reqs; b += kThreads / 32) {
      const int r = b * 32 + lane;
      const int c = __reduce_add_sync(0xffffffffu,
                                      r < p.num_reqs ? items_of(load_req(p, r, TQ)) : 0);
      if (lane == 0) sm.batch_items[b] = c;
      count += c;
    }
    if (lane == 0) sm.counts[warp] = count;
  };
  auto total_count = [&]() {  // (warp 0, after a barrier)
    long long total = lane < kThreads / 32 ? sm.counts[lane] : 0;
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    return total;
  };
  // Key tiles over all items (where they matter the items are few), and of the
  // longest request.
  unsigned tiles = 0, longest = 0;
  count_batches([&](const Req& a) {
    const int c = a.ntiles * Hkv;
    if (kSplit && c > 0) {
      tiles += (unsigned)c * (unsigned)ceil_div(a.L, kKeyTile);
      longest = max(longest, (unsigned)ceil_div(a.L, kKeyTile));
    }
    return c;
  });
  if (kSplit) {
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) sm.extents[warp] = make_uint2(tiles, longest);
  }
  __syncthreads();
  if (warp == 0) {
    const long long total = total_count();
    if (lane == 0) sm.n_active = (int)min(total, (long long)gridDim.x);
    if (kSplit) {
      // The longest part, in key tiles: a request of n tiles is cut into ceil(n
      // / T) parts.  T = tiles / (parts - items) leaves room for every item's
      // rounded-up part, T = longest / (parts / items) gives all as many.
      const uint2 x = lane < kThreads / 32 ? sm.extents[lane] : make_uint2(0u, 0u);
      const unsigned sum = __reduce_add_sync(0xffffffffu, x.x), n = __reduce_max_sync(0xffffffffu, x.y);
      unsigned T = 0;
      if (total > 0 && total <= pb.max_parts) {
        const unsigned items = (unsigned)total, room = (unsigned)pb.max_parts;
        auto up = [](unsigned a, unsigned b) { return (a + b - 1) / b; };
        T = up(n, room / items);
        if (room > items) T = min(T, up(sum, room - items));
        T = max(T, max(up(n, kMaxSplit), (unsigned)kMinPart));
        if (T >= n) T = 0;
      }
      if (lane == 0) sm.longest_part = (int)T;
    }
  }
  __syncthreads();
  const int longest_part = kSplit ? sm.longest_part : 0;
  // Parts of each of a request's items (some may be empty, see take_next).
  auto parts_of = [&](int L) {
    return longest_part > 0 ? ceil_div(ceil_div(L, kKeyTile), longest_part) : 1;
  };
  if (kSplit && longest_part > 0) {
    count_batches([&](const Req& a) { return a.ntiles * Hkv * parts_of(a.L); });
    __syncthreads();
    if (warp == 0) {
      const long long total = total_count();
      if (lane == 0) sm.n_active = (int)min(total, (long long)gridDim.x);
    }
    __syncthreads();
  }
  const int n_active = sm.n_active;  // CTAs that take items
  if ((int)blockIdx.x >= n_active) {
    grid_dependency_wait();
    allow_dependent_launch();
    return;
  }

  if (tid == 0) {
    for (int s = 0; s < kItems; ++s) {
      mbar_init(&sm.it_full[s], 1);
      mbar_init(&sm.it_free[s], kSoftWarps + kConvWarps + 1);  // softmax, converters, MMA
      mbar_init(&sm.q_full[s], kSoftWarps);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kStagesV; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], kConvWarps);
    }
    for (int s = 0; s < kScaleRing; ++s) mbar_init(&sm.sc_full[s], 2 * kBlkPerTile);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.qr_full[b], 1);
      mbar_init(&sm.q_empty[b], 1);  // tcgen05.commit after the item's last S
      mbar_init(&sm.vb_full[b], kConvWarps);
      mbar_init(&sm.vb_free[b], 1);
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.s_free[b], kSoftWarps);
      mbar_init(&sm.p_full[b], kSoftWarps);
      mbar_init(&sm.p_free[b], 1);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kSoftWarps);
    mbar_init(&sm.mma_done, 1);
    for (int i = 0; i < kNanRing * kConvWarps; ++i) sm.nan_item[i / kConvWarps][i % kConvWarps] = -1;
    sm.wait.abort = 0;
    sm.wait.limit_ns = p.wait_limit_ns;
    fence_barrier_init();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  // Q rows that no copy writes stay zero.
  if constexpr (TQ * G < kRows) {
    constexpr int kPad = (kRows - TQ * G) * 8;  // 16-byte chunks of an operand
    for (int i = tid; i < 4 * kPad; i += kThreads)
      *reinterpret_cast<uint4*>(&sm.q[0][0][0] + (i / kPad) * kCodes + TQ * G * 128 + (i % kPad) * 16) =
          make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  grid_dependency_wait();
  allow_dependent_launch();

  // Item n of this CTA from the ring; every warp that reads it releases it (when
  // split, the softmax warps after their epilogue, which reads it again).
  auto release_item = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.it_free[n % kItems]);
  };
  auto take_item = [&](int n, Item& it, bool keep = false) {
    if (!mbar_wait(&sm.it_full[n % kItems], (n / kItems) & 1, p.err, abort_flag)) return false;
    it = sm.items[n % kItems];
    if (!keep) release_item(n);
    return !it.end;
  };

  if (warp == kWarpLoad) {
    // ==================== items, K and V tiles, scales =====================
    int n_item = 0, t = 0, nq = 0, nk = 0, nv = 0;  // items, tiles; Q, K and V copies issued
    const int oob_row = p.num_blocks * Hkv * kBlockSize;
    // Items are numbered batch of 32 requests by batch, longest request first
    // within a batch, heavier q-tiles first within a request, and taken from
    // the queue in that order (see pkv_prefill.cu).
    Req rq = {0, 0, 0, 0};     // this lane's request of the batch
    long long cnt = 0, excl = 0, total = 0, base = 0;
    int batch = -32;
    auto take_next = [&](Item& it) {
      unsigned long long taken = 0;
      if (lane == 0) taken = atomicAdd(p.sched, 1ull);
      const long long item = (long long)__shfl_sync(0xffffffffu, taken, 0);
      while (item >= base + total) {
        base += total;
        do batch += 32; while (batch < p.num_reqs && sm.batch_items[batch / 32] == 0);
        if (batch >= p.num_reqs) {
          it = Item{};
          it.end = 1;
          total = 0;
          batch = p.num_reqs;
          return;
        }
        total = sm.batch_items[batch / 32];
        if (item >= base + total) continue;
        rq = Req{0, 0, 0, 0};
        if (batch + lane < p.num_reqs) rq = load_req(p, batch + lane, TQ);
        cnt = (long long)rq.ntiles * Hkv * parts_of(rq.L);
        const int key = cnt > 0 ? rq.L : -1;
        excl = 0;
        #pragma unroll 4
        for (int s = 0; s < 32; ++s) {
          const int ks = __shfl_sync(0xffffffffu, key, s);
          const long long cs = __shfl_sync(0xffffffffu, cnt, s);
          if (ks > key || (ks == key && s < lane)) excl += cs;
        }
      }
      const long long rel = item - base;
      const unsigned own = __ballot_sync(0xffffffffu, cnt > 0 && excl <= rel && rel < excl + cnt);
      const int src = __ffs(own) - 1;
      long long local = rel - __shfl_sync(0xffffffffu, excl, src);
      const int q0 = __shfl_sync(0xffffffffu, rq.q0, src);
      const int qr = __shfl_sync(0xffffffffu, rq.qr, src);
      const int L = __shfl_sync(0xffffffffu, rq.L, src);
      const int cut = parts_of(L);
      it.part = 0;
      if (kSplit && cut > 1) {
        it.part = (int)(local % cut);
        local /= cut;
      }
      const int qt = __shfl_sync(0xffffffffu, rq.ntiles, src) - 1 - (int)(local / Hkv);
      it.r = batch + src;
      it.k = (int)(local % Hkv);
      it.row0 = q0 + qt * TQ;
      it.nt = min(TQ, qr - qt * TQ);
      it.pos0 = L - qr + qt * TQ;
      it.L = L;
      const int tiles = (it.pos0 + it.nt - 1) / kKeyTile + 1;
      it.parts = kSplit ? min(cut, ceil_div(tiles, kMinPart)) : 1;
      it.j0 = kSplit ? tiles * min(it.part, it.parts) / it.parts : 0;
      it.nj = kSplit ? tiles * min(it.part + 1, it.parts) / it.parts - it.j0 : tiles;  // 0: no such part
      it.slot = (int)item;  // (below max_parts when split)
      it.end = 0;
    };
    auto next_item = [&](Item& it) {
      do take_next(it); while (kSplit && !it.end && it.nj == 0);
    };
    // The next item into nx and the ring.
    Item nx;
    auto publish_next = [&]() {
      next_item(nx);
      const int s = n_item % kItems;
      if (n_item >= kItems &&
          !mbar_wait(&sm.it_free[s], ((n_item / kItems) - 1) & 1, p.err, abort_flag))
        return false;
      if (lane == 0) {
        sm.items[s] = nx;
        mbar_arrive(&sm.it_full[s]);
      }
      __syncwarp();
      if (!nx.end) {  // its Q, into the buffer of the item before the current one
        const int b = n_item & 1;
        if (n_item >= 2 && !mbar_wait(&sm.q_empty[b], ((n_item >> 1) - 1) & 1, p.err, abort_flag))
          return false;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.qr_full[b], 2u * 64u * TQ * G * 2u);
          tma_load_3d(sm.q[b][0], &qmap, 0, nx.k * G, nx.row0, &sm.qr_full[b]);
          tma_load_3d(sm.q[b][1], &qmap, 64, nx.k * G, nx.row0, &sm.qr_full[b]);
        }
        __syncwarp();
        nq = n_item + 1;
      }
      ++n_item;
      return true;
    };
    auto stream_item = [&](const Item& it) {
      const int nbl = ceil_div(it.L, kBlockSize);
      const int32_t* bt = p.block_tables + (long long)it.r * p.max_blocks;
      auto raw_entries = [&](int x0) {
        const int x = (kSplit ? it.j0 * kBlkPerTile : 0) + x0 + lane;
        return x < nbl ? __ldg(bt + x) : kPastEnd;
      };
      int ent_cur = raw_entries(0);
      int ent_nxt = it.nj > 4 ? raw_entries(32) : kPastEnd;
      for (int j = 0; j < it.nj; ++j, ++t) {
        if (j == max(0, it.nj - kAhead) && !publish_next()) return false;
        if (j > 0 && (j & 3) == 0) {
          ent_cur = ent_nxt;
          if (j + 4 < it.nj) ent_nxt = raw_entries((j + 4) * kBlkPerTile);
        }
        // Blocks past the request (or outside the pool: recorded) are read at
        // an out-of-range row, which TMA fills with zeros, with scale 0.
        const int phys = __shfl_sync(0xffffffffu, ent_cur, (j & 3) * kBlkPerTile + (lane & 7));
        const bool good = (unsigned)phys < (unsigned)p.num_blocks;
        const int pool_row = good ? (phys * Hkv + it.k) * kBlockSize : oob_row;
        if (lane < kBlkPerTile && !good && phys != kPastEnd) record_error(p.err, kErrBounds);
        const int sk = t % kStages;
        if (t >= kStages &&
            !mbar_wait(&sm.k_empty[sk], ((t / kStages) - 1) & 1, p.err, abort_flag))
          return false;
        if (lane == 0) mbar_arrive_expect_tx(&sm.k_full[sk], (uint32_t)kCodes);
        __syncwarp();
        if (lane < kBlkPerTile) tma_load_2d(sm.k[sk] + lane * 2048, &kmap, 0, pool_row, &sm.k_full[sk]);
        nk = t + 1;
        if (lane < 2 * kBlkPerTile) {
          // Scales outlive their K stage: a ring entry is reused eight tiles
          // on, when S of the tile three before is done, hence the softmax has
          // taken S and the scales of the tile five before.
          static_assert(kScaleRing >= kStages + 2, "scales outlive their tile");
          const float* src = (lane < kBlkPerTile ? pb.k_scales : pb.v_scales) +
                             (good ? (long long)phys * Hkv + it.k : 0);
          copy4_async(&sm.sc[t % kScaleRing][lane >> 3][lane & 7], src, good ? 4u : 0u);
          arrive_after_copies(&sm.sc_full[t % kScaleRing]);
        }
        const int sv = t % kStagesV;
        if (t >= kStagesV &&
            !mbar_wait(&sm.v_empty[sv], ((t / kStagesV) - 1) & 1, p.err, abort_flag))
          return false;
        if (lane == 0) mbar_arrive_expect_tx(&sm.v_full[sv], (uint32_t)kCodes);
        __syncwarp();
        if (lane < kBlkPerTile) tma_load_2d(sm.v[sv] + lane * 2048, &vmap, 0, pool_row, &sm.v_full[sv]);
        nv = t + 1;
        __syncwarp();
      }
      return true;
    };
    if (publish_next()) {
      while (!nx.end) {
        const Item it = nx;
        if (!stream_item(it)) break;
      }
    }
    if (abort_flag->abort) {
      // Copies in flight land before the CTA's shared memory is released.
      for (int m = max(0, nq - 2); m < nq; ++m)
        mbar_wait_drain(&sm.qr_full[m & 1], (m >> 1) & 1, p.err, abort_flag);
      for (int m = max(0, nk - kStages); m < nk; ++m)
        mbar_wait_drain(&sm.k_full[m % kStages], (m / kStages) & 1, p.err, abort_flag);
      for (int m = max(0, nv - kStagesV); m < nv; ++m)
        mbar_wait_drain(&sm.v_full[m % kStagesV], (m / kStagesV) & 1, p.err, abort_flag);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kWarpMma) {
    // ========================= MMA issuer =================================
    // Tile t: S(t) into S buffer t & 1, then O += P(t-2) V(t-2).  An S buffer
    // is free as soon as the softmax has taken its scores, well before it sends
    // their P, so S runs ahead of PV by two tiles: with S(t) behind PV(t-1) the
    // softmax waited for it (3500 cycles a tile against 3000).
    constexpr uint32_t kIdescHi = idesc_e4m3_f32(kRows, kKeyTile, 0, 0);
    constexpr uint32_t kIdescLo = idesc_e5m2_e4m3_f32(kRows, kKeyTile, 0, 0);
    constexpr uint32_t kIdescO = idesc_f16_f32(kRows, kHeadDim, 0, 1);
    // Descriptors of the operands' first chunks: a chunk of 32 bytes of a row
    // is 2 further (16-byte units), a V chunk of 16 keys 128.
    const uint64_t dq = smem_desc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
    const uint64_t dk = smem_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
    const uint64_t dv = smem_desc_sw128(smem_u32(sm.vb[0][0]), kHalfBytes, 1024);
    const bool leader = elect_one();
    int t = 0;
    bool ok = true;
    // O += P V of tile tt: item n's first, last?
    auto pv = [&](int tt, bool first, bool last, int n) {
      const int b = tt & 1;
      ok = ok && mbar_wait(&sm.p_full[b], (tt >> 1) & 1, p.err, abort_flag);
      ok = ok && mbar_wait(&sm.vb_full[b], (tt >> 1) & 1, p.err, abort_flag);
      if (first && n > 0) ok = ok && mbar_wait(&sm.o_empty, (n - 1) & 1, p.err, abort_flag);
      if (!ok) return;
      tc_fence_after();
      if (leader) {
        // P: keys 16kk .. +15 in columns 8kk .. +7 of P buffer b; V MN-major,
        // two 64-dim halves.
        const uint64_t db = dv + b * (2 * kHalfBytes / 16);
        const uint32_t ta = tmem + kColP + b * 64;
        #pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_f16_ts(tmem + kColO, ta + kk * 8, db + kk * 128, kIdescO, !first || kk > 0);
        tc_commit(&sm.vb_free[b]);
        tc_commit(&sm.p_free[b]);
        if (last) tc_commit(&sm.o_full);
      }
      __syncwarp();
    };
    int st = 0, phase = 0;
    for (int n = 0; ok; ++n) {
      Item it;
      if (!take_item(n, it)) break;
      const int nj = it.nj;
      ok = mbar_wait(&sm.q_full[n % kItems], (n / kItems) & 1, p.err, abort_flag);
      const uint64_t da = dq + (n & 1) * (2 * kCodes / 16);
      for (int j = 0; j < nj && ok; ++j, ++t) {
        const int b = t & 1;
        ok = ok && mbar_wait(&sm.k_full[st], phase, p.err, abort_flag);
        if (t >= 2) ok = ok && mbar_wait(&sm.s_free[b], ((t >> 1) - 1) & 1, p.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t db = dk + st * (kCodes / 16);
          const uint32_t tS = tmem + b * kKeyTile;
          #pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // hi rows, then lo rows
            tc_mma_f8_ss(tS, da + (kk >> 2) * (kCodes / 16) + (kk & 3) * 2, db + (kk & 3) * 2,
                         kk < 4 ? kIdescHi : kIdescLo, kk > 0);
          tc_commit(&sm.k_empty[st]);
          tc_commit(&sm.s_full[b]);
          if (j + 1 == nj) tc_commit(&sm.q_empty[n & 1]);
        }
        __syncwarp();
        if (++st == kStages) {
          st = 0;
          phase ^= 1;
        }
        if (j >= 2) pv(t - 2, j == 2, false, n);
      }
      // The item's last two PVs, before waiting for the next item: its Q is
      // split after this one's last P.
      for (int i = min(nj, 2); i > 0 && ok; --i) pv(t - i, nj == i, i == 1, n);
    }
    if (abort_flag->abort) {
      if (leader) tc_commit(&sm.mma_done);  // MMAs in flight finish before TMEM is freed
      __syncwarp();
      mbar_wait_drain(&sm.mma_done, 0, p.err, abort_flag);
    }
    __syncwarp();
  } else if (warp >= kWarpConv) {
    // ============================ V converters =============================
    constexpr int kConvThreads = 32 * kConvWarps;
    const int row0 = tid - kWarpConv * 32;  // its key rows: row0, row0 + kConvThreads
    int t = 0;
    bool ok = true;
    Item it;
    for (int n = 0; ok && take_item(n, it); ++n) {
      for (int j = 0; j < it.nj && ok; ++j, ++t) {
        const int st = t % kStagesV, b = t & 1;
        ok = mbar_wait(&sm.v_full[st], (t / kStagesV) & 1, p.err, abort_flag);
        if (ok && t >= 2) ok = mbar_wait(&sm.vb_free[b], ((t >> 1) - 1) & 1, p.err, abort_flag);
        if (!ok) break;
        #pragma unroll 1
        for (int row = row0; row < kKeyTile; row += kConvThreads) {
          // A key row widened: past the item's last key a block may hold
          // anything (NaN codes too), and 0 * V has to stay 0.
          const int key0 = ((kSplit ? it.j0 : 0) + j) * kKeyTile, end = it.pos0 + it.nt;
          const bool keep = key0 + row < end;
          const int sw = row & 7;
          uint4 c[8];
          auto fetch = [&]() {
            #pragma unroll
            for (int i = 0; i < 8; ++i)
              c[i] = keep ? lds128(sm.v[st] + row * 128 + ((i ^ sw) * 16)) : make_uint4(0, 0, 0, 0);
          };
          fetch();
          uint32_t bad = 0;
          if (key0 + row > it.pos0) {  // seen by some of the item's rows only
            #pragma unroll
            for (int i = 0; i < 8; ++i)
              bad |= nan_bytes(c[i].x) | nan_bytes(c[i].y) | nan_bytes(c[i].z) | nan_bytes(c[i].w);
          }
          if (__any_sync(0xffffffffu, bad != 0)) {
            note_nans(sm, sm.v[st], row - lane, key0, it.pos0, end, n);
            fetch();
          }
          #pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            uint32_t o[8];
            #pragma unroll
            for (int e = 0; e < 4; ++e) e4m3x4_to_f16x4(w[e], o[2 * e], o[2 * e + 1]);
            uint8_t* dst = sm.vb[b][i >> 2] + row * 128;
            const int at = (i & 3) * 2;
            *reinterpret_cast<uint4*>(dst + ((at ^ sw) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(dst + (((at + 1) ^ sw) * 16)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.v_empty[st]);
          mbar_arrive(&sm.vb_full[b]);
        }
      }
    }
  } else {
    // =================== softmax + epilogue (warps 0-15) ===================
    const int quad = warp & 3;
    const int part = warp >> 2;
    const int row = quad * 32 + lane;  // MMA row == TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t tO = lanes + kColO + part * kPartKeys;
    const int t_local = row / G, h = row % G;
    int t = 0;

    Item it;
    bool ok = true, more = false;
    // Item n into `it`, its Q split; false if there is none.
    auto begin_item = [&](int n) {
      bool have = take_item(n, it, kSplit);
      have = have && mbar_wait(&sm.qr_full[n & 1], (n >> 1) & 1, p.err, abort_flag);
      // Agree before the next barrier of these rows' four warps (the only
      // barriers there are): a wait that gave up (abort) stops them all.
      if (barrier_or(kBarQuad + quad, 128, !have)) return false;
      split_q(sm.q[n & 1][0], p.scale_log2, sm.qf[n % kItems], &sm.q_full[n % kItems]);
      return true;
    };
    more = begin_item(0);
    for (int n = 0; more; ++n) {
      ok = ok && mbar_wait(&sm.q_full[n % kItems], (n / kItems) & 1, p.err, abort_flag);
      const bool valid = t_local < it.nt && row < TQ * G;
      // the last key this row sees, from the item's first key on
      const int prow = valid ? it.pos0 + t_local - (kSplit ? it.j0 * kKeyTile : 0) : -1;
      const int nj = it.nj;
      __nv_bfloat16* const dst = p.out + ((long long)(it.row0 + t_local) * p.num_q_heads +
                                          (long long)it.k * G + h) * kHeadDim + part * kPartKeys;
      const float qf = sm.qf[n % kItems][row];
      float m = kNegBig, mo = kNegBig, l = 0.f, root = 0.f;
      // The tile at hand: this part's 32 scores (two blocks of 16 keys), and
      // the blocks' factors of a score and of a probability, and what is added
      // to a score.
      float x0[16], x1[16], sc0, sc1, f0, f1, up0, up1;
      // Tile tt's scores taken from the registers they were fetched to:
      // masked, the references raised where the maxima exceed them by
      // 2^kMargin.  (A factor of 0 would turn a masked -inf into NaN; 1e-30
      // leaves the scores below 2^-70.)
      auto take = [&](int tt, int g) {
        ok = ok && mbar_wait(&sm.sc_full[g % kScaleRing], (g / kScaleRing) & 1, p.err, abort_flag);
        const float2 ks = *reinterpret_cast<const float2*>(&sm.sc[g % kScaleRing][0][part * 2]);
        const float2 vs = *reinterpret_cast<const float2*>(&sm.sc[g % kScaleRing][1][part * 2]);
        wait_ld32(x0, x1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_free[g & 1]);
        sc0 = qf * ks.x;
        sc1 = qf * ks.y;
        if (sc0 < 1e-30f) sc0 = 1e-30f;
        if (sc1 < 1e-30f) sc1 = 1e-30f;
        const float lv0 = scale_exponent(vs.x), lv1 = scale_exponent(vs.y);
        const int kbase = tt * kKeyTile + part * kPartKeys;
        if (kbase + kPartKeys - 1 > prow) {
          #pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (kbase + i > prow) x0[i] = -INFINITY;
            if (kbase + 16 + i > prow) x1[i] = -INFINITY;
          }
        }
        float a0 = -INFINITY, a1 = -INFINITY, b0 = -INFINITY, b1 = -INFINITY;
        #pragma unroll
        for (int i = 0; i < 16; i += 4) {
          a0 = fmax3(a0, x0[i], x0[i + 1]);
          a1 = fmax3(a1, x0[i + 2], x0[i + 3]);
          b0 = fmax3(b0, x1[i], x1[i + 1]);
          b1 = fmax3(b1, x1[i + 2], x1[i + 3]);
        }
        const float mx0 = fmaxf(a0, a1) * sc0, mx1 = fmaxf(b0, b1) * sc1;
        const float mxh = fmaxf(mx0, mx1), moh = fmaxf(mx0 + lv0, mx1 + lv1);
        if (barrier_or(kBarQuad + quad, 128, tt == 0 || mxh > m + kMargin || moh > mo + kMargin)) {
          sm.xrow[part][row] = make_float2(mxh, moh);
          named_barrier(kBarQuad + quad, 128);
          float m_new = m, mo_new = mo;
          #pragma unroll
          for (int i = 0; i < kParts; ++i) {
            const float2 y = sm.xrow[i][row];
            m_new = fmaxf(m_new, y.x);
            mo_new = fmaxf(mo_new, y.y);
          }
          named_barrier(kBarQuad + quad, 128);  // sm.xrow is free again
          l *= fast_exp2(m - m_new);
          if (tt > 0 && __any_sync(0xffffffffu, mo_new != mo)) {
            // O must first hold the previous tile's PV.
            ok = ok && mbar_wait(&sm.p_free[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err, abort_flag);
            tc_fence_after();
            rescale_o(tO, fast_exp2(mo - mo_new));
            tc_fence_before();
          }
          m = m_new;
          mo = mo_new;
          // 2^up in two factors: either alone is in range
          root = fast_exp2(0.5f * (m - mo + kTop));
        }
        // What F has beyond 2^100 joins the exponent: P is below 2^15, so these
        // probabilities are below 2^-84 of the normaliser with it or without.
        f0 = root * vs.x * root;
        f1 = root * vs.y * root;
        up0 = up1 = -m;
        auto reach = [&](float& up, float& f, float v) {
          if (f > kMostF) {
            up += m - mo + kTop + scale_exponent(v) - kTopF;
            f = kMostF * __uint_as_float((__float_as_uint(v) & 0x7fffffu) | 0x3f800000u);
          }
        };
        if (f0 > kMostF || f1 > kMostF) {
          reach(up0, f0, vs.x);
          reach(up1, f1, vs.y);
        }
      };
      const uint32_t tS = lanes + part * kPartKeys;
      ok = ok && mbar_wait(&sm.s_full[t & 1], (t >> 1) & 1, p.err, abort_flag);
      tc_fence_after();
      tmem_ld16(tS + (t & 1) * kKeyTile, x0);
      tmem_ld16(tS + (t & 1) * kKeyTile + 16, x1);
      take(0, t);
      #pragma unroll 1
      for (int j = 0; j < nj; ++j, ++t) {
        const int b = t & 1;
        const bool more_keys = j + 1 < nj;
        const uint32_t next = tS + (b ^ 1) * kKeyTile;
        // p = exp2(s + up) into the normaliser, P = p F in f16, two keys per
        // column, one block after the other; each block's registers take the
        // next tile's scores.
        float2 sum = make_float2(0.f, 0.f);
        uint32_t w[kPartKeys / 2];
        auto block = [&](const float (&x)[16], float sc, float f, float up, int at) {
          const float2 nm2 = make_float2(up, up);
          #pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 y = ffma2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(sc, sc), nm2);
            const float2 q = make_float2(fast_exp2(y.x), fast_exp2(y.y));
            sum = fadd2(sum, q);
            w[at + e] = pack_f16x2(fmul2(q, make_float2(f, f)));
          }
        };
        block(x0, sc0, f0, up0, 0);
        if (more_keys) {
          ok = ok && mbar_wait(&sm.s_full[b ^ 1], ((t + 1) >> 1) & 1, p.err, abort_flag);
          tc_fence_after();
          tmem_ld16(next, x0);
        }
        block(x1, sc1, f1, up1, 8);
        if (more_keys) tmem_ld16(next + 16, x1);
        l += sum.x + sum.y;
        // P buffer b was last read by the PV of two tiles before.
        if (t >= 2) ok = ok && mbar_wait(&sm.p_free[b], ((t >> 1) - 1) & 1, p.err, abort_flag);
        tc_fence_after();
        tmem_st16(lanes + kColP + b * 64 + part * (kPartKeys / 2), w);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[b]);
        if (more_keys) take(j + 1, t + 1);
      }
      sm.xrow[part][row].x = l;
      more = begin_item(n + 1);  // (also the barrier between this row's parts)
      // ---- epilogue: O / l -> bf16 -> out (this part's 32 dims) ----------
      const float lrow = (sm.xrow[0][row].x + sm.xrow[1][row].x) +
                         (sm.xrow[2][row].x + sm.xrow[3][row].x);
      named_barrier(kBarQuad + quad, 128);  // sm.xrow is free again
      // O carries 2^(kTop - mo), the normaliser 2^-m.
      const float inv = lrow == 0.f ? 0.f : exp2f(mo - m - kTop) / lrow;
      ok = ok && mbar_wait(&sm.o_full, n & 1, p.err, abort_flag);
      tc_fence_after();
      if (kSplit && sm.items[n % kItems].parts > 1) {  // (`it` is the next item)
        finish_part<G>(sm, pb, n, tO, m, lrow, inv, valid && ok, dst);
      } else {
        tmem_ld16(tO, x0);
        tmem_ld16(tO + 16, x1);
        wait_ld32(x0, x1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_empty);
        put_nans(sm, n, part, t_local, x0, x1);
        if (valid && ok) {
          #pragma unroll
          for (int i = 0; i < 16; i += 8) {
            uint4 q4;
            q4.x = pack_bf16x2(x0[i] * inv, x0[i + 1] * inv);
            q4.y = pack_bf16x2(x0[i + 2] * inv, x0[i + 3] * inv);
            q4.z = pack_bf16x2(x0[i + 4] * inv, x0[i + 5] * inv);
            q4.w = pack_bf16x2(x0[i + 6] * inv, x0[i + 7] * inv);
            *reinterpret_cast<uint4*>(dst + i) = q4;
            q4.x = pack_bf16x2(x1[i] * inv, x1[i + 1] * inv);
            q4.y = pack_bf16x2(x1[i + 2] * inv, x1[i + 3] * inv);
            q4.z = pack_bf16x2(x1[i + 4] * inv, x1[i + 5] * inv);
            q4.w = pack_bf16x2(x1[i + 6] * inv, x1[i + 7] * inv);
            *reinterpret_cast<uint4*>(dst + 16 + i) = q4;
          }
        }
      }
      if (kSplit) release_item(n);
    }
  }
  // Every warp reaches this point (aborts only shorten the loops), so the
  // allocating warp can always free TMEM.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
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

template <int G, bool kSplit>
cudaError_t launch_variant(const PrefillBlockLaunch& L, cudaStream_t stream) {
  const size_t smem = sizeof(Smem) + 1024;  // + alignment slack
  static unsigned long long configured = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(__atomic_load_n(&configured, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(prefill_block_kernel<G, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  e = cudaLaunchKernelEx(&cfg, prefill_block_kernel<G, kSplit>, L.qmap, L.kmap, L.vmap, L.p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int G>
cudaError_t launch_g(const PrefillBlockLaunch& L, cudaStream_t stream) {
  return L.p.max_parts > 0 ? launch_variant<G, true>(L, stream) : launch_variant<G, false>(L, stream);
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
