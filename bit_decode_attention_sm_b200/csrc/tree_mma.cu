// headq_tree_attn on the tensor cores: bf16 queries, bf16 or 2-bit values, d 64 or 128,
// r 0, 8 or 16 ("HeadQ: Model-Visible Distortion and Score-Space Correction for KV-Cache
// Quantization", gist.science summary, section 3, step 3).
//
// The n * G query rows of a (sequence, KV head) fill the M side of tcgen05.mma, 128 rows a
// block; 128-token tiles of the cache are the N side of the logits and the K side of the
// readout.  A logit is one dot product of length d + r: q with the decoded base key, and
// U_h^T q with the decoded side code.  Both sides of the latter are fp16 in two parts (22 bits;
// the product of the two smaller parts is left out): in one part each they were the largest
// errors behind the output's own rounding (against 64 bits 0.0025 on the long context, now
// 0.0018, of which the output's is 0.0016), for two more K steps of eleven, 172 -> 177 us there
// and 0 to 3 % elsewhere.
//
// tree_prep_kernel   once per call: query rows as fp16 operands, each scaled by its own
//   power of two (exact for bf16 queries but for elements 2^-28 below the row's largest),
//   U_h^T q behind them, written as the shared-memory image the main kernel copies in; the
//   mask as bits.
// tree_mma_kernel    one CTA of 20 warps per (row blocks, split, sequence x KV head):
//   8 decoder warps  two threads per token, half the channels each: packed codes from HBM
//     (the next tile's loads in flight) to fp16 keys in shared memory, scaled by a power of
//     two per tile.  The four levels min + code * scale of a 32-channel group are rounded to
//     fp16 once, two 2-bit codes then pick their pair by one byte permute; the channels come
//     out as a 4 x 4 transpose within each 16, and the queries are stored in that order too.
//     2-bit values the same way in bf16.
//   1 TMA warp       dense bf16 values, 64 tokens x 64 channels a box
//   2 MMA warps      one per lane (below): logits into TMEM, readout from the weights there
//   2 x 4 softmax warps (two "lanes"), one thread per query row.  PAIR (more than 128 rows):
//     the lanes hold two row blocks over the same tiles, so each decoded tile serves 256
//     rows; else they take alternate tiles of the one block and end as two splits.
// The running maximum is kept with a slack of 2^60 (kSlack): one pass over the logits and no
// search for the maximum in it, and the output accumulator in TMEM is rescaled only when a
// weight reaches 2, which is rare (with a slack of 2^8 it was a third of the steps in peaked
// attention; kSlack has what the offset costs).  Weights are rounded to bf16 and the sum is taken
// over the rounded weights, so that the error of a weight cancels where one token holds most of
// it; the log-sum-exp, when asked for, is summed over the unrounded ones.
//
// Measured: 64 new tokens over 131072 cached ones, 32 heads on 8, 177 us (its products take 89
// at the rate of a large matrix product); 32 over 64 x 4096 in 2-bit values, 28 heads on 4,
// 227 us (78).  The exponential units are 45 % busy, the tensor pipe 52 %, the issue slots
// 54 %; what bounds the kernel is that a tile passes five hand-overs (decoder, logits, weights,
// readout, release), each some 150 cycles even when nothing is left to wait for.  Measured while
// the long case stood at 180: sixteen softmax warps 193, lanes in ping-pong 231, one row block per
// CTA with three logit buffers 201.  A CTA's set-up, first tile and outputs are some 8 us; the
// kernel therefore starts on the cache while the queries are still being prepared.
//
// TMEM (512 columns): logits of lane l at 128 l (its weights overwrite them, two to a
// column), outputs at 256 + 128 l.
#include <cuda_fp16.h>

#include "decode_common.cuh"
#include "tree.cuh"

namespace headq {
namespace {

using dc::mbar_arrive;
using dc::mbar_expect_tx;
using dc::mbar_init;
using dc::smem_addr;

constexpr int kTile = 128;          // tokens per tile
constexpr int kBlock = 128;         // query rows per block
constexpr int kThreads = 20 * 32;  // five whole warpgroups
// registers per thread after the split: 8 x 32 x 128 + 8 x 32 x 80 + 4 x 32 x 48 = 59392, of
// the 640 x 96 = 61440 that the block holds at launch
constexpr int kRegsSoftmax = 128, kRegsDecode = 80, kRegsOther = 48;
constexpr int kDecodeWarp = 8, kMmaWarp = 16, kTmaWarp = 18;  // one MMA warp per lane
constexpr int kKStages = 2;
constexpr int kRing = 8;            // tiles whose key scales are kept (more than can be in flight), a byte each
// A row's weights are 2^(logit - m) with m at least the largest logit so far and, when it is
// set, kSlack above it: the check that a step stays below 2 is then one bit of the weights,
// and m is seldom set again.  Weights and sums have the 8-bit exponent of fp32, so the offset
// costs them no precision (a weight 2^-66 of the largest is still normal).  It does cost the
// readout's range: weight * value with the largest weight near 2^-60 is subnormal for values
// below 2^-66, which lose their last bits, and 0 below 2^-89.  Smaller offsets were slower where
// logits spread: 2^40 233-237 us on the full-KV 2-bit layer, 2^30 248-260, 2^20 279-288 (2^60
// 226-229).
constexpr float kSlack = 60.0f;
constexpr uint32_t kAll = 0xffffffffu;

// bytes of 128 operand rows: d channels in 64-channel blocks (128-byte rows, 128-byte
// swizzle), then 16 side entries (two 8-entry halves, no swizzle), then what their rounding to
// fp16 left, laid out the same
constexpr int kSideBytes = kTile * 32;
__host__ __device__ constexpr int operand_bytes(int d, int r) { return kTile * 2 * d + (r > 0 ? 2 * kSideBytes : 0); }

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The next three are executed by the whole warp and take effect for the thread with `one`
// set: their operands are then the same in every lane, and need no moves out of per-thread
// registers between one product and the next.
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(one)
      : "memory");
}
// descriptors as their two words
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi,
                                          uint32_t idesc, bool acc, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 da, db;\n setp.ne.u32 p, %6, 0;\n setp.ne.u32 q, %7, 0;\n"
      " mov.b64 da, {%1, %2};\n mov.b64 db, {%3, %4};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n}\n" ::"r"(d),
      "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(one)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, bool acc,
                                          uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 db;\n setp.ne.u32 p, %5, 0;\n setp.ne.u32 q, %6, 0;\n"
      " mov.b64 db, {%2, %3};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(one)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tc_ld32(uint32_t a, uint32_t (&v)[N], int o) {
  uint32_t* r = v + o;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void tc_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tc_ld4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void tc_st4(uint32_t a, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0,%1,%2,%3};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(a)
               : "memory");
}
template <int N>
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t (&v)[N], int o) {
  const uint32_t* r = v + o;
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// A try that the hardware itself suspends for a while.  (With a time hint the compiler puts
// a loop of sleeps around it, whose instructions and wake-up times cost this kernel a third
// of its issue slots.)
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait for the phase of the given parity; false after about 2 s.  Short: it is in many
// places, and five roles share the SM's instruction cache.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  if (mbar_try(bar, parity)) return true;
  const long long start = clock64();
  do {
#pragma unroll 1
    for (int k = 0; k < 256; ++k)
      if (mbar_try(bar, parity)) return true;
  } while (clock64() - start < dc::kWaitCycles);
  return false;
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptors: low word, start address and leading byte offset; high
// word, stride byte offset, descriptor version 1 and swizzle (2: 128 bytes, 0: none); all
// offsets in 16-byte units.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr & 0x3ffffu) >> 4) | ((lead >> 4) << 16);
}
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride, uint32_t swizzle) {
  return (stride >> 4) | (1u << 14) | (swizzle << 29);
}
// Instruction descriptor of kind::f16: fp32 accumulator, operand type (0 fp16, 1 bf16),
// B transposed (its N side contiguous), N / 8, M / 16 with M = 128.
__host__ __device__ constexpr uint32_t mma_desc(uint32_t type, uint32_t b_trans, uint32_t n) {
  return (1u << 4) | (type << 7) | (type << 10) | (b_trans << 16) | ((n / 8) << 17) | ((128u / 16) << 24);
}

// 2^(14 - e) and 2^(e - 14), e the binary exponent of m >= 0: m times the first lies in
// [2^14, 2^15), inside fp16 with 28 binades of normal numbers below.  (1, 1) when m is 0 or
// not finite; exponents below -100 are taken as -100.
__device__ __forceinline__ float2 operand_scale(float m) {
  const int b = static_cast<int>(__float_as_uint(m) >> 23);
  if (m == 0.0f || b == 255) return make_float2(1.0f, 1.0f);
  const int e = max(b - 127, -100);
  return make_float2(__uint_as_float(static_cast<uint32_t>(141 - e) << 23),
                     __uint_as_float(static_cast<uint32_t>(max(113 + e, 1)) << 23));
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// channel at position `pos` of an operand row (a 4 x 4 transpose within each 16)
__host__ __device__ constexpr int channel_at(int pos) { return (pos & ~15) + 4 * (pos & 3) + ((pos >> 2) & 3); }

// byte offset of 16-byte chunk c of row x in the swizzled blocks of an operand
__device__ __forceinline__ int swz(int x, int c) { return (c >> 3) * (kTile * 128) + x * 128 + (((c & 7) ^ (x & 7)) << 4); }

// zeroes the bf16 values of a pair that are not finite; whether there were any
__device__ __forceinline__ bool drop_bad(uint32_t& v) {
  const bool lo = (v & 0x7f80u) == 0x7f80u, hi = (v & 0x7f800000u) == 0x7f800000u;
  if (lo) v &= 0xffff0000u;
  if (hi) v &= 0x0000ffffu;
  return lo || hi;
}

// 16 codes of one word as 8 operand pairs, through the group's levels (two per register)
__device__ __forceinline__ void pick16(uint32_t w, uint32_t l01, uint32_t l23, uint4& a, uint4& b) {
  uint32_t o[8];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    // byte j: the code of channel 4 j + s; code c picks bytes 2c, 2c + 1 of the levels
    const uint32_t sel = ((w >> (2 * s)) & 0x03030303u) * 0x22u + 0x10101010u;
    o[2 * s] = __byte_perm(l01, l23, sel);
    o[2 * s + 1] = __byte_perm(l01, l23, sel >> 16);
  }
  a = make_uint4(o[0], o[1], o[2], o[3]);
  b = make_uint4(o[4], o[5], o[6], o[7]);
}

// ---------------------------------------------------------------- prep
// One warp per 4 query rows of a unit's row blocks: D / 4 lanes a row, 4 operand positions
// each; all rows are loaded before the first is worked on, since the main kernel waits for the
// last (one row at a time, 8 rows to a warp, took it 5 us longer).  Blocks past the rows' part
// pack the mask.
constexpr int kPrepRows = 4;

template <int D, int R>
__global__ void __launch_bounds__(256)
tree_prep_kernel(const TreeParams p, const TreeMma t, int row_ctas) {
  let_next_kernel_start();
  const int warp = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (static_cast<int>(blockIdx.x) >= row_ctas) {  // mask bits: one warp per (sequence, row)
    const int bi = (blockIdx.x - row_ctas) * 8 + (threadIdx.x >> 5);
    if (!t.words || bi >= p.c.B * p.span.n) return;
    const int b = bi / p.span.n, i = bi - b * p.span.n;
    const int n = span_seq(p.span, b).n;
    for (int w = 0; w < t.wpr; ++w) {
      const int j = 32 * w + lane;
      const bool see = i < n && j < n && tree_sees(p, b, i, j);
      const uint32_t bits = __ballot_sync(kAll, see);
      if (lane == 0) t.words[static_cast<size_t>(bi) * t.wpr + w] = bits;
    }
    return;
  }
  constexpr int LPR = D / 4, RPW = 32 / LPR;  // lanes per row, rows at a time
  const int per_unit = t.blocks * kBlock / kPrepRows;
  const int unit = warp / per_unit, x0 = (warp - unit * per_unit) * kPrepRows;
  if (unit >= p.c.B * p.c.Hkv) return;
  const int b = unit / p.c.Hkv, kv = unit - b * p.c.Hkv;
  const SpanSeq sq = span_seq(p.span, b);
  const int rows = sq.n * p.G;
  if (x0 / 32 * 32 >= rows) return;  // a 32-row group without rows is never read
  const int ll = lane & (LPR - 1);
  int ch[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) ch[k] = channel_at(4 * ll + k);
  float u[4][R > 0 ? R : 1];
  if constexpr (R > 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(p.U + (static_cast<size_t>(kv) * D + ch[k]) * R + i));
        u[k][i] = v.x; u[k][i + 1] = v.y; u[k][i + 2] = v.z; u[k][i + 3] = v.w;
      }
  }
  const float sign = p.sm_scale < 0.0f ? -1.0f : 1.0f;
  constexpr int IT = kPrepRows / RPW;
  uint16_t qr[IT][4];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int x = x0 + it * RPW + lane / LPR;
#pragma unroll
    for (int k = 0; k < 4; ++k) qr[it][k] = 0;
    if (x < rows) {
      const int i = x / p.G, g = x - i * p.G;
      const uint16_t* src = static_cast<const uint16_t*>(p.q.ptr) + (sq.row0 + i) * p.q.row_stride +
                            (kv * p.G + g) * p.q.head_stride;
#pragma unroll
      for (int k = 0; k < 4; ++k) qr[it][k] = __ldg(src + ch[k]);
    }
  }
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int x = x0 + it * RPW + lane / LPR;
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) q[k] = sign * bf16_bits_to_f32(qr[it][k]);
    float mx = fmaxf(fmaxf(fabsf(q[0]), fabsf(q[1])), fmaxf(fabsf(q[2]), fabsf(q[3])));
    float side = 0.0f;
    if constexpr (R > 0) {
      float a[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        a[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) a[i] = fmaf(q[k], u[k][i], a[i]);
      }
      // halve the entries a lane holds with each exchange, then sum what is left
      int m = LPR / 2;
#pragma unroll
      for (int h = R / 2; h >= 1; h /= 2) {
        const bool up = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
          const float keep = up ? a[i + h] : a[i], give = up ? a[i] : a[i + h];
          a[i] = keep + __shfl_xor_sync(kAll, give, m);
        }
        m /= 2;
      }
      for (; m >= 1; m /= 2) a[0] += __shfl_xor_sync(kAll, a[0], m);
      side = a[0] * p.corr_sign;  // entry ll / (LPR / R)
      mx = fmaxf(mx, fabsf(side));
    }
#pragma unroll
    for (int m = LPR / 2; m >= 1; m /= 2) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, m));
    const float2 s = operand_scale(mx);
    const int xr = x & (kBlock - 1);
    uint8_t* img = t.qimg + (static_cast<size_t>(unit) * t.blocks + x / kBlock) * operand_bytes(D, R);
    *reinterpret_cast<uint2*>(img + swz(xr, ll / 2) + 8 * (ll & 1)) =
        make_uint2(pack_f16(q[0] * s.x, q[1] * s.x), pack_f16(q[2] * s.x, q[3] * s.x));
    if constexpr (R > 0) {
      __half* zb = reinterpret_cast<__half*>(img + D / 64 * (kTile * 128));
      const int e = ll / (LPR / R);
      if (ll % (LPR / R) == 0) {
        const __half hi = __float2half_rn(side * s.x);
        __half* at = zb + (e / 8) * (kTile * 8) + xr * 8 + (e & 7);
        at[0] = hi;
        at[kSideBytes / 2] = __float2half_rn(side * s.x - __half2float(hi));
      }
      if (R == 8 && ll < 8) {
        __half* at = zb + kTile * 8 + xr * 8 + ll;
        at[0] = at[kSideBytes / 2] = __float2half_rn(0.0f);
      }
    }
    if (ll == 0)
      t.qf[static_cast<size_t>(unit) * t.blocks * kBlock + x] = s.y * (fabsf(p.sm_scale) * dc::kLog2e);
  }
}

// ---------------------------------------------------------------- main kernel
template <int D, int R, bool V2, bool PAIR>
struct Layout {
  static constexpr int kVStages = PAIR ? 2 : 3;
  static constexpr int kOperand = operand_bytes(D, R);
  static constexpr int kVTile = kTile * D * 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + (PAIR ? 2 : 1) * kOperand;
  static constexpr int kV = kK + kKStages * kOperand;
  static constexpr int kScale = kV + kVStages * kVTile;  // [kRing][kTile] bytes: exponents of powers of two
  static constexpr int kBars = kScale + kRing * kTile;
  static constexpr int kNumBars = 1 + 2 * kKStages + 2 * kVStages + 12;
  static constexpr int kMisc = (kBars + 8 * kNumBars + 15) & ~15;  // tmem base, bad-value flag, 2 x 8 maxima
  static constexpr int kBytes = kMisc + 128 + 1024;    // and room for the alignment
};

// What a decoder thread holds of its token: the codes of half the channels, all scales and
// minima of the key (both threads of a token take their power of two from them).
template <int D, int R, bool V2>
struct RawToken {
  static constexpr int NG = D / 32, W = D / 32;  // groups, code words of half the channels
  uint32_t kw[W];
  float ks[NG], km[NG];
  uint32_t zc;
  float zs;
  uint32_t vw[V2 ? W : 1];
  float vs[V2 ? NG / 2 : 1], vm[V2 ? NG / 2 : 1];
};

// Loads that stay where they are written: a tile ahead of their use.
template <int N>
__device__ __forceinline__ void load_32(const void* p, uint32_t (&x)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "l"(p));
  else if constexpr (N == 2)
    asm volatile("ld.global.nc.v2.b32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "l"(p));
  else
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(x[0]) : "l"(p));
}
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&x)[N]) {
  uint32_t u[N];
  load_32<N>(p, u);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float(u[i]);
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// half `h` of the token in plane row `row`
template <int D, int R, bool V2>
__device__ __forceinline__ void load_token(const headq_cache& c, long long row, int h, RawToken<D, R, V2>& x) {
  constexpr int NG = D / 32, W = D / 32;
  load_32<W>(c.k_codes + row * (D / 4) + h * (D / 8), x.kw);
  load_f32<NG>(c.k_scale + row * NG, x.ks);
  load_f32<NG>(c.k_min + row * NG, x.km);
  if constexpr (R > 0) {
    uint32_t z[1];
    load_32<1>(c.z_codes + row * (R / 2) + (R == 16 ? 4 * h : 0), z);
    x.zc = z[0];
    float f[1];
    load_f32<1>(c.z_scale + row, f);
    x.zs = f[0];
  } else {
    x.zs = 0.0f;
  }
  if constexpr (V2) {
    load_32<W>(c.v_codes + row * (D / 4) + h * (D / 8), x.vw);
    load_f32<NG / 2>(c.v_scale + row * NG + h * (NG / 2), x.vs);
    load_f32<NG / 2>(c.v_min + row * NG + h * (NG / 2), x.vm);
  }
}

// The plane rows of a decoder thread's tokens, kTile apart; past the end, the last token's.
struct TokenRows {
  const headq_cache& c;
  const int32_t* table;
  long long base;  // contiguous planes: the (sequence, KV head)'s first row
  int kv, t, last;
  unsigned* err;
  __device__ TokenRows(const headq_cache& c_, int b, int kv_, int t_, int t_hi, unsigned* e)
      : c(c_), table(c_.block_table + static_cast<size_t>(b) * c_.max_pages),
        base((static_cast<long long>(b) * c_.Hkv + kv_) * c_.T_cap), kv(kv_), t(t_), last(t_hi - 1), err(e) {}
  __device__ long long next() {
    const int u = min(t, last);
    t += kTile;
    if (c.page_size == 0) return base + u;
    const int i = u / c.page_size;
    int pg = __ldg(table + i);
    if (pg < 0 || pg >= c.num_pages) {
      if (err) atomicOr(err, kDevErrBadPage);
      pg = 0;
    }
    return (static_cast<long long>(pg) * c.Hkv + kv) * c.page_size + (u - i * c.page_size);
  }
};

// 32 mask bits of new token i's row from bit a (new-token index of the first; bits below 0
// are the prefix: seen)
__device__ __forceinline__ uint32_t mask_word(const uint32_t* row, int wpr, int i, int k) {
  if (k < 0) return kAll;
  if (row) return k < wpr ? __ldg(row + k) : 0u;
  const int last = i - 32 * k;  // j <= i
  return last < 0 ? 0u : last >= 31 ? kAll : (2u << last) - 1u;
}
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int wpr, int i, int a) {
  const int k = a >> 5;
  return __funnelshift_r(mask_word(row, wpr, i, k), mask_word(row, wpr, i, k + 1), a & 31);
}

// Running maximum (log2 units), sum of the rounded weights, sum of the exact ones.
struct RowState {
  float m, l, lx;
};

// The rows whose m rises (to `top`; the others pass their m): their sums and their
// accumulator scaled to it.
template <int D>
__device__ __forceinline__ RowState raise_max(RowState st, float top, uint32_t to, bool have_o) {
  const float a = st.m == -INFINITY ? 0.0f : ex2(st.m - top);
  st.l *= a;
  st.lx *= a;
  st.m = top;
  if (have_o) {
#pragma unroll 1
    for (int o = 0; o < D; o += 4) {  // few registers: half a row of logits is held meanwhile
      uint32_t w[4];
      tc_ld4(to + o, w);
      tc_wait_ld();
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * a);
      tc_st4(to + o, w);
    }
    tc_wait_st();
  }
  return st;
}

constexpr int kHalf = kTile / 2;

// a power of two from its exponent field
__device__ __forceinline__ float pow2_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// The logits of half a tile that holds new tokens or ends the sequence, in TMEM: each token
// has its own scale, and is masked.  a: new-token index of the half's first token; f: the row's
// factor to log2 units.
__device__ __forceinline__ void mask_half(uint32_t ts, const uint32_t* row, int wpr, int i, int a,
                                          const uint8_t* col, float f) {
#pragma unroll 1
  for (int c = 0; c < kHalf; c += 16) {
    uint32_t w[16];
    tc_ld16(ts + c, w);
    const uint32_t bits = mask_bits(row, wpr, i, a + c);
    const uint4 e4 = *reinterpret_cast<const uint4*>(col + c);
    const uint32_t e[4] = {e4.x, e4.y, e4.z, e4.w};
    tc_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = __float_as_uint((bits >> j) & 1u ? __uint_as_float(w[j]) * pow2_of((e[j / 4] >> (8 * (j % 4))) & 255u) * f
                                               : -INFINITY);
    tc_st16(ts + c, w, 0);
  }
  tc_wait_st();
}

// Half a tile's 64 logits of this thread's row (times f: log2 units) to weights, two to a
// word; their sum, and all their bits.  The 64 are in registers before the first
// exponential, so that these run back to back.
__device__ __forceinline__ void weights(const uint32_t (&s)[kHalf], float f, float m, uint32_t (&w)[kHalf / 2],
                                        float& sum, uint32_t& bits) {
  const float mm = m == -INFINITY ? 0.0f : m;
  const uint64_t f2 = codec::pk2(f, f), m2 = codec::pk2(-mm, -mm);
  uint64_t a[2] = {0ull, 0ull};
  uint32_t any[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < kHalf / 2; ++j) {
    const uint64_t y = codec::fma2(codec::pk2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), f2, m2);
    w[j] = pack_bf16(ex2(codec::pk_lo(y)), ex2(codec::pk_hi(y)));
    any[j & 1] |= w[j];
    a[j & 1] = codec::add2(a[j & 1], codec::pk2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)));
  }
  const uint64_t t = codec::add2(a[0], a[1]);
  sum = codec::pk_lo(t) + codec::pk_hi(t);
  bits = any[0] | any[1];
}

// Once a row of a warp reaches logits of this size (log2 units), its logits are rounded before
// the maximum is taken off.  weights() takes it off the unrounded product; the maximum itself is
// rounded, which leaves up to half a unit in its last place in every exponent: it cancels in the
// quotient, but passes the range of fp32 when the logits reach 2^32.
constexpr float kBigLogit = 0x1p24f;

// The sum of channel `ch` over the new tokens that row i sees and whose value there is not
// finite once rounded to bf16 (they were left out of the value tiles).
template <bool V2, bool PAIR>
__device__ __forceinline__ float bad_values(const TreeParams& p, const uint32_t* words, int wpr, int i, int b, int kv,
                                         int lo, int t_lo, int t_hi, int P, int wl, int ch) {
  float sum = 0.0f;
  const int d = p.c.d, ng = d / 32;
#pragma unroll 1
  for (int tt = lo; tt < t_hi; ++tt) {
    if (!PAIR && (((tt - t_lo) / kTile) & 1) != wl) continue;
    if (!((mask_word(words, wpr, i, (tt - P) >> 5) >> ((tt - P) & 31)) & 1u)) continue;
    const size_t row = cache_row_read(p.c, b, kv, tt, p.err);
    const float v = V2 ? fmaf(static_cast<float>(code2(p.c.v_codes + row * (d / 4), ch)),
                              p.c.v_scale[row * ng + ch / 32], p.c.v_min[row * ng + ch / 32])
                       : load_elem(p.c.v, row * d + ch, true);
    if (!(fabsf(v) < 0x1.FFp127f)) sum += v;
  }
  return sum;
}

template <int D, int R, bool V2, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
tree_mma_kernel(const TreeParams p, const TreeMma t, const __grid_constant__ CUtensorMap vmap) {
  using Ly = Layout<D, R, V2, PAIR>;
  constexpr int NG = D / 32;
  constexpr int VS = Ly::kVStages;
  extern __shared__ uint8_t raw_smem[];

  const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
  const int unit = blockIdx.z, b = unit / p.c.Hkv, kv = unit - b * p.c.Hkv;
  const SpanSeq sq = span_seq(p.span, b);
  const int rows = sq.n * p.G, xb = blockIdx.x * (PAIR ? 2 : 1) * kBlock;
  if (xb >= rows) {
    wait_for_prior_kernel();
    return;
  }
  const int P = sq.p0, L = sq.p0 < 0 ? 0 : sq.p0 + sq.n;
  const int t_lo = blockIdx.y * p.chunk, t_hi = min(L, t_lo + p.chunk);
  const int tiles = t_hi > t_lo ? (t_hi - t_lo + kTile - 1) / kTile : 0;
  const int lane_parts = p.splits / gridDim.y;  // 2 when the lanes end as two splits
  const size_t part_rows = static_cast<size_t>(p.span.n) * p.G;
  // this softmax thread's query row
  const int wl = (warp >> 2) & 1;  // lane of the softmax warp
  const int x = xb + (PAIR ? wl * kBlock : 0) + (warp & 3) * 32 + lane;

  if (tiles == 0) {  // nothing to read: the rows' share of this split is empty
    wait_for_prior_kernel();
    if (warp < 8 && x < rows && (PAIR || wl < lane_parts)) {
      if (p.splits > 1) {
        p.part_ml[(static_cast<size_t>(unit) * p.splits + blockIdx.y * lane_parts + (PAIR ? 0 : wl)) * part_rows + x] =
            make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
      } else {
        const int i = x / p.G, h = kv * p.G + x - i * p.G;
        const size_t orow = static_cast<size_t>(sq.row0) + i;
        for (int c = 0; c < D; c += 4)
          store_row4(p.out, orow * p.out.row_stride + h * p.out.head_stride + c, make_float4(0, 0, 0, 0));
        if (p.lse) p.lse[orow * p.Hq + h] = -INFINITY;
      }
    }
    return;
  }

  uint8_t* sm = smem_align(raw_smem, 1024);
  const uint32_t base = smem_addr(sm);
  uint8_t* scale_s = sm + Ly::kScale;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + Ly::kMisc);
  const uint32_t bars = base + Ly::kBars;
  const uint32_t q_full = bars;
  auto k_full = [&](int s) { return bars + 8 * (1 + s); };
  auto k_empty = [&](int s) { return bars + 8 * (1 + kKStages + s); };
  auto v_full = [&](int s) { return bars + 8 * (1 + 2 * kKStages + s); };
  auto v_empty = [&](int s) { return bars + 8 * (1 + 2 * kKStages + VS + s); };
  // per lane l and half h (64 tokens) of its tile: logits written, weights written, readout done
  auto s_full = [&](int l, int h) { return bars + 8 * (1 + 2 * kKStages + 2 * VS + 2 * l + h); };
  auto p_full = [&](int l, int h) { return bars + 8 * (5 + 2 * kKStages + 2 * VS + 2 * l + h); };
  auto o_done = [&](int l, int h) { return bars + 8 * (9 + 2 * kKStages + 2 * VS + 2 * l + h); };

  // tiles of lane l: PAIR all of them (when the lane has rows), else those of its parity
  const int lanes_on = PAIR ? (xb + kBlock < rows ? 2 : 1) : (tiles > 1 ? 2 : 1);
  auto lane_tiles = [&](int l) { return l >= lanes_on ? 0 : PAIR ? tiles : (tiles - l + 1) / 2; };
  auto tile_of = [&](int l, int k) { return PAIR ? k : 2 * k + l; };

  if (tid == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(k_full(s), 8);
      mbar_init(k_empty(s), PAIR ? lanes_on : 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(v_full(s), V2 ? 8 : 1);
      mbar_init(v_empty(s), PAIR ? lanes_on : 1);
    }
    for (int l = 0; l < 2; ++l) {
      const int r0 = rows - xb - (PAIR ? l * kBlock : 0);
      for (int h = 0; h < 2; ++h) {
        mbar_init(s_full(l, h), 1);
        mbar_init(p_full(l, h), max(1, min(4, (r0 + 31) / 32)));  // warps that have rows
        mbar_init(o_done(l, h), 1);
      }
    }
    misc[1] = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  // the first tile's planes on their way to L2 while barriers and TMEM are set up
  if (warp >= kDecodeWarp && warp < kDecodeWarp + 4) {
    TokenRows first(p.c, b, kv, t_lo + tid - kDecodeWarp * 32, t_hi, nullptr);
    const long long row = first.next();
    prefetch_l2(p.c.k_codes + row * (D / 4));
    prefetch_l2(p.c.k_scale + row * NG);
    prefetch_l2(p.c.k_min + row * NG);
    if constexpr (R > 0) {
      prefetch_l2(p.c.z_codes + row * (R / 2));
      prefetch_l2(p.c.z_scale + row);
    }
    if constexpr (V2) {
      prefetch_l2(p.c.v_codes + row * (D / 4));
      prefetch_l2(p.c.v_scale + row * NG);
      prefetch_l2(p.c.v_min + row * NG);
    }
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(misc)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc);
  bool ok = true;

  // Registers move from the other warps to the softmax warps, a warpgroup at a time.
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == kTmaWarp) {
    if (lane == 0) {
      wait_for_prior_kernel();  // the query images; the decoders are at work on the cache meanwhile
      fence_async_global();
      const int nq = PAIR ? lanes_on : 1;
      mbar_expect_tx(q_full, nq * Ly::kOperand);
      const uint8_t* img = t.qimg + (static_cast<size_t>(unit) * t.blocks + xb / kBlock) * Ly::kOperand;
      dc::bulk_g2s(base + Ly::kQ, img, nq * Ly::kOperand, q_full);
      if constexpr (!V2) {
        int issued = 0;
        for (int k = 0; k < tiles && ok; ++k) {
          const int s = k % VS;
          if (k >= VS && !mbar_wait(v_empty(s), ((k / VS) - 1) & 1)) { ok = false; break; }
          const int t0 = t_lo + k * kTile;
          const int halves = t0 + 64 < t_hi ? 2 : 1;
          mbar_expect_tx(v_full(s), halves * 64 * D * 2);
          for (int h = 0; h < halves; ++h) {
            const CacheSlab sl = cache_slab_read(p.c, b, kv, t0 + 64 * h, p.err);
            for (int c = 0; c < D / 64; ++c)
              dc::tma_3d(base + Ly::kV + s * Ly::kVTile + c * (kTile * 128) + h * (64 * 128), &vmap, 64 * c, sl.off,
                         static_cast<int>(sl.slab), v_full(s));
          }
          issued = k + 1;
        }
        // no copy is in flight when the CTA ends
        for (int k = max(0, issued - VS); k < issued; ++k) mbar_wait(v_full(k % VS), (k / VS) & 1);
      }
      if (!mbar_wait(q_full, 0)) ok = false;
    }
  } else if (warp < kTmaWarp) {
    // The halves of a lane's tile take turns: while the exponentials of one run, the other's
    // readout and next logits do.
    const int l = warp - kMmaWarp, n = lane_tiles(l);
    constexpr uint32_t kLogit = mma_desc(0, 0, kTile / 2);  // fp16, both operands K-major
    constexpr uint32_t kRead = mma_desc(1, 1, D);           // bf16, values channel-major
    constexpr uint32_t kSwz = desc_hi(1024, 2), kFlat = desc_hi(128, 0);
    constexpr uint32_t kSide = D / 64 * (kTile * 128);  // the side entries within an operand
    const uint32_t one = lane == 0;
    const uint32_t qa = base + Ly::kQ + (PAIR ? l * Ly::kOperand : 0);
    const uint32_t q_lo = desc_lo(qa, 16), qs_lo = desc_lo(qa + kSide, kTile * 16);
    const uint32_t k_lo = desc_lo(base + Ly::kK, 16), ks_lo = desc_lo(base + Ly::kK + kSide, kTile * 16);
    const uint32_t v_lo = desc_lo(base + Ly::kV, kTile * 128);
    auto wait = [&](uint32_t bar, int phase) {
      ok = __all_sync(kAll, ok && mbar_wait(bar, phase & 1));
      return ok;
    };
    // step -1: logits of tile 0; step k: readout of tile k, each half followed by its logits
    // of tile k + 1, which overwrite the weights it read
    if (n > 0) wait(q_full, 0);
#pragma unroll 1
    for (int y = -2; y < 2 * n && ok; ++y) {
      const int k = y >> 1, h = y & 1;
      if (k >= 0) {
        const int tile = tile_of(l, k), s = tile % VS;
        // the stage's last tile was the other lane's: it is read before this one's phase counts
        if (!V2 && !PAIR && h == 0 && tile >= VS && !wait(v_empty(s), tile / VS - 1)) break;
        // (the values first, while the weights are not there: a wait costs some 150 cycles anyway)
        if ((h == 0 && !wait(v_full(s), tile / VS)) || !wait(p_full(l, h), k)) break;
        tc_fence_after();
        const uint32_t va = v_lo + ((s * Ly::kVTile + 8192 * h) >> 4), w = tmem + 128 * l + 64 * h;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tc_mma_ts(tmem + 256 + 128 * l, w + 8 * e, va + (2048 >> 4) * e, kSwz, kRead, y > 0 || e > 0, one);
        tc_commit(o_done(l, h), one);
        if (h == 1) tc_commit(v_empty(s), one);
      }
      if (k + 1 < n) {
        const int tile = tile_of(l, k + 1), s = tile % kKStages;
        if ((h == 0 && !wait(k_full(s), tile / kKStages)) || (k >= 0 && !wait(o_done(l, h), k))) break;
        tc_fence_after();
        const uint32_t ka = (s * Ly::kOperand + 8192 * h) >> 4, d = tmem + 128 * l + 64 * h;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
          const uint32_t off = ((e >> 2) * (kTile * 128) + 32 * (e & 3)) >> 4;
          tc_mma_ss(d, q_lo + off, kSwz, k_lo + ka + off, kSwz, kLogit, e > 0, one);
        }
        if constexpr (R > 0) {  // both sides' leading parts, then each with what the other's rounding left
          const uint32_t ks = ks_lo + ((s * Ly::kOperand + 1024 * h) >> 4);
          tc_mma_ss(d, qs_lo, kFlat, ks, kFlat, kLogit, true, one);
          tc_mma_ss(d, qs_lo + (kSideBytes >> 4), kFlat, ks, kFlat, kLogit, true, one);
          tc_mma_ss(d, qs_lo, kFlat, ks + (kSideBytes >> 4), kFlat, kLogit, true, one);
        }
        tc_commit(s_full(l, h), one);
        if (h == 1) tc_commit(k_empty(s), one);
      }
    }
    // the products are done before TMEM is given back
    if (n > 0 && ok) wait(o_done(l, 1), n - 1);
    __syncwarp();
  }
  } else if (warp >= kDecodeWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsDecode));
    const int tok = (tid - kDecodeWarp * 32) & (kTile - 1), half = (warp - kDecodeWarp) >> 2;
    float* red = reinterpret_cast<float*>(misc + 4);  // [2][8] warp maxima
    constexpr int HG = NG / 2;  // groups of this half
    TokenRows rows_of(p.c, b, kv, t_lo + tok, t_hi, p.err);
    RawToken<D, R, V2> cur, nxt;
    load_token<D, R, V2>(p.c, rows_of.next(), half, cur);
    long long row = rows_of.next();
    // byte offset of chunk j of this half's 16-byte chunks in an operand's row
    auto at = [&](int j) { return D == 128 ? half * (kTile * 128) + swz(tok, j) : swz(tok, 4 * half + j); };
    for (int k = 0; k < tiles; ++k) {
      const int t0 = t_lo + k * kTile, s = k % kKStages, sv = k % VS;
      load_token<D, R, V2>(p.c, row, half, nxt);
      row = rows_of.next();
      const bool tail = t0 + kTile > min(P, t_hi);  // holds new tokens, or ends the sequence
      float mx = 7.0f * fabsf(cur.zs);
#pragma unroll
      for (int g = 0; g < NG; ++g)
        mx = max3(mx, fabsf(cur.km[g]), fabsf(fmaf(3.0f, cur.ks[g], cur.km[g])));
      const uint32_t wm = __reduce_max_sync(kAll, __float_as_uint(mx));
      if (lane == 0) red[(k & 1) * 8 + warp - kDecodeWarp] = __uint_as_float(wm);
      // one warp waits for the stage, the others for the barrier that they meet at anyway
      if (warp == kDecodeWarp && k >= kKStages && ok && !mbar_wait(k_empty(s), ((k / kKStages) - 1) & 1)) ok = false;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (!tail) {  // one power of two per tile; else one per token: an unseen new token's size touches no other
        const float4 m4 = *reinterpret_cast<const float4*>(red + (k & 1) * 8);  // half 0's four have them all
        mx = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w));
      }
      const float2 sc = operand_scale(mx);
      if (half == 0) scale_s[(k % kRing) * kTile + tok] = static_cast<uint8_t>(__float_as_uint(sc.y) >> 23);
      uint8_t* ks = sm + Ly::kK + s * Ly::kOperand;
#pragma unroll
      for (int g = 0; g < HG; ++g) {
        const float m = (half ? cur.km[HG + g] : cur.km[g]) * sc.x, d = (half ? cur.ks[HG + g] : cur.ks[g]) * sc.x;
        // code 0 with its product too: a scale that is not finite makes all four levels NaN or infinite
        const uint32_t l01 = pack_f16(fmaf(0.0f, d, m), m + d), l23 = pack_f16(fmaf(2.0f, d, m), fmaf(3.0f, d, m));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 a, c;
          pick16(cur.kw[2 * g + h], l01, l23, a, c);
          *reinterpret_cast<uint4*>(ks + at(4 * g + 2 * h)) = a;
          *reinterpret_cast<uint4*>(ks + at(4 * g + 2 * h + 1)) = c;
        }
      }
      if constexpr (R > 0) {
        const float zs = cur.zs * sc.x;
        uint32_t o[4] = {0, 0, 0, 0}, left[4] = {0, 0, 0, 0};
        if (8 * half < R) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // nibble ^ 8 is w + 8; 2^23 + that has it in its low mantissa bits
            const uint32_t w = cur.zc >> (8 * e);
            const float a = __uint_as_float((w & 15u) ^ 0x4B000008u) - 8388616.0f;
            const float c = __uint_as_float(((w >> 4) & 15u) ^ 0x4B000008u) - 8388616.0f;
            o[e] = pack_f16(a * zs, c * zs);
            const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&o[e]));
            if (fabsf(zs) < INFINITY) left[e] = pack_f16(fmaf(a, zs, -r.x), fmaf(c, zs, -r.y));
          }
        }
        uint4* side = reinterpret_cast<uint4*>(ks + D / 64 * (kTile * 128)) + half * kTile + tok;
        side[0] = make_uint4(o[0], o[1], o[2], o[3]);
        side[kSideBytes / 16] = make_uint4(left[0], left[1], left[2], left[3]);
      }
      if constexpr (V2) {
        if (k >= VS && ok && !mbar_wait(v_empty(sv), ((k / VS) - 1) & 1)) ok = false;
        uint8_t* vs = sm + Ly::kV + sv * Ly::kVTile;
#pragma unroll
        for (int g = 0; g < HG; ++g) {
          const float m = cur.vm[g], d = cur.vs[g];
          uint32_t l01 = pack_bf16(fmaf(0.0f, d, m), m + d), l23 = pack_bf16(fmaf(2.0f, d, m), fmaf(3.0f, d, m));
          // a new token's value that is not finite must not meet the zero weights of the
          // rows that do not see it: it is left out here and added to the rows that do
          if (t0 + tok >= t_hi) l01 = l23 = 0u;
          if (t0 + tok >= P && (drop_bad(l01) | drop_bad(l23))) misc[1] = 1u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 a, c;
            pick16(cur.vw[2 * g + h], l01, l23, a, c);
            *reinterpret_cast<uint4*>(vs + at(4 * g + 2 * h)) = a;
            *reinterpret_cast<uint4*>(vs + at(4 * g + 2 * h + 1)) = c;
          }
        }
      } else if (tail) {
        // the last rows of the value tile: nothing past the end, and as above for new tokens.
        // A wait for one phase of a barrier passes while the phase before it is open, and this
        // thread has not waited for the stage's earlier tiles: first until the last one is read.
        if (k >= VS && ok && !mbar_wait(v_empty(sv), ((k / VS) - 1) & 1)) ok = false;
        if (ok && !mbar_wait(v_full(sv), (k / VS) & 1)) ok = false;
        uint8_t* vs = sm + Ly::kV + sv * Ly::kVTile;
        if (t0 + tok >= P) {
          const bool past = t0 + tok >= t_hi;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t* w = reinterpret_cast<uint32_t*>(vs + at(c));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t v = past ? 0u : w[e];
              if (drop_bad(v)) misc[1] = 1u;
              w[e] = v;
            }
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(k_full(s));
        if (V2) mbar_arrive(v_full(sv));
      }
      cur = nxt;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
  if (xb + (PAIR ? wl * kBlock : 0) + (warp & 3) * 32 < rows && wl < lanes_on) {
    // ---- softmax and epilogue of this warp's 32 query rows
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + 128 * wl + lane_off, to = tmem + 256 + 128 * wl + lane_off;
    wait_for_prior_kernel();
    const int i = min(x, rows - 1) / p.G;
    const float fq = t.qf[static_cast<size_t>(unit) * t.blocks * kBlock + x];
    const uint32_t* words = t.words ? t.words + (static_cast<size_t>(b) * p.span.n + i) * t.wpr : nullptr;
    const bool want_lse = p.lse != nullptr;
    RowState st{-INFINITY, 0.0f, 0.0f};
    const int nk = lane_tiles(wl);
    // One half-tile at a time; the next one's logits are on their way while this one's
    // weights are written.
    uint32_t s[kHalf];
    float f = 0.0f;
    // tiles from here on hold new tokens or end the sequence, or have logits to be rounded (kBigLogit)
    int round_from = min(P, t_hi) >= t_lo ? (min(P, t_hi) - t_lo) / kTile : 0;
#pragma unroll 1
    for (int y = -1; y < 2 * nk && ok; ++y) {  // step y: half y & 1 of the lane's tile y / 2
      const int h = y & 1;
      if (y >= 0) {
        tc_wait_ld();
        uint32_t w[kHalf / 2], bits;
        float sum;
        weights(s, f, st.m, w, sum, bits);
        // a weight of 2 or more (or not a number), or no m yet: find it, and the weights again
        if (__any_sync(kAll, (bits & 0x40004000u) != 0u || st.m == -INFINITY)) {
          float mx = __uint_as_float(s[0]);
#pragma unroll
          for (int j = 1; j < kHalf - 1; j += 2) mx = max3(mx, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
          const float top = fmaxf(mx, __uint_as_float(s[kHalf - 1])) * f;
          // the accumulator rests once the half before this one is read out
          // (ok stays the same in a whole warp, which works together to the end)
          if (y > 0) ok = __all_sync(kAll, ok && mbar_wait(o_done(wl, 1 - h), ((y - 1) >> 1) & 1));
          tc_fence_after();
          if (__any_sync(kAll, fabsf(top) >= kBigLogit && top != -INFINITY)) {
#pragma unroll
            for (int j = 0; j < kHalf; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) * f);
            f = 1.0f;
            round_from = 0;
          }
          st = raise_max<D>(st, top > st.m ? top + kSlack : st.m, to, y > 0);
          weights(s, f, st.m, w, sum, bits);
        }
        st.l += sum;
        if (want_lse) {  // the unrounded weights once more, rather than their sums beside every other call's
          const float mm = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
          for (int j = 0; j < kHalf; ++j) st.lx += ex2(fmaf(__uint_as_float(s[j]), f, -mm));
        }
        tc_st16(ts + kHalf * h, w, 0);
        tc_st16(ts + kHalf * h + 16, w, 16);
      }
      auto hand_over = [&]() {
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(wl, h));
      };
      bool handed = y < 0;
      if (y + 1 < 2 * nk) {
        const uint32_t bar = s_full(wl, 1 - h), parity = ((y + 1) >> 1) & 1;
        if (!__all_sync(kAll, mbar_test(bar, parity))) {  // not there yet: this one's weights first
          if (!handed) hand_over();
          handed = true;
          ok = __all_sync(kAll, ok && mbar_wait(bar, parity));
        }
        const int tile = tile_of(wl, (y + 1) >> 1);
        const uint8_t* col = scale_s + (tile % kRing) * kTile;
        const uint32_t sa = ts + kHalf * (1 - h);
        tc_fence_after();
        f = fmaxf(fq * pow2_of(col[0]), 1e-37f);
        if (tile >= round_from) {
          mask_half(sa, words, t.wpr, i, t_lo + tile * kTile + kHalf * (1 - h) - P, col + kHalf * (1 - h),
                    fmaxf(fq, 1e-37f));
          f = 1.0f;
        }
        tc_ld32(sa, s, 0);
        tc_ld32(sa + 32, s, 32);
      }
      if (!handed) hand_over();
    }
    const float m = st.m, l = st.l, lx = st.lx;
    let_next_kernel_start();
    if (nk > 0) ok = __all_sync(kAll, ok && mbar_wait(o_done(wl, 1), (nk - 1) & 1));
    tc_fence_after();
    if (ok) {
      const bool bad = *reinterpret_cast<volatile uint32_t*>(misc + 1) != 0u;
      const bool direct = p.splits == 1;
      const int part = blockIdx.y * lane_parts + (PAIR ? 0 : wl);
      const size_t pr = (static_cast<size_t>(unit) * p.splits + part) * part_rows + x;
      const int h = kv * p.G + x - i * p.G;
      const size_t orow = static_cast<size_t>(sq.row0) + i;
      const float inv = !direct ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      if (bad) {  // rare: one column at a time, in TMEM
#pragma unroll 1
        for (int c = 0; c < D; ++c) {
          const float add = bad_values<V2, PAIR>(p, words, t.wpr, i, b, kv, max(P, t_lo), t_lo, t_hi, P, wl,
                                                 V2 ? channel_at(c) : c);
          uint32_t w;
          asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(w) : "r"(to + c));
          tc_wait_ld();
          w = __float_as_uint(__uint_as_float(w) + add);
          asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(to + c), "r"(w) : "memory");
        }
        tc_wait_st();
      }
      // 32 columns at a time.  PAIR: through shared memory (the lane's query image, which its
      // products no longer read), so that 8 lanes store one row's 128 bytes where each lane
      // storing its own row touches 32 lines an instruction (9000 cycles a CTA).
      float4* turn = reinterpret_cast<float4*>(sm + Ly::kQ + (PAIR ? wl : 0) * Ly::kOperand) + (warp & 3) * 256;
      const long long off = static_cast<long long>(orow) * p.out.row_stride + h * p.out.head_stride;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t w[32];
        tc_ld32(to + 32 * c, w, 0);
        tc_wait_ld();
        float o[32];  // in channel order
#pragma unroll
        for (int j = 0; j < 32; ++j) o[V2 ? channel_at(j) : j] = l == 0.0f ? 0.0f : __uint_as_float(w[j]) * inv;
        if constexpr (PAIR) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            turn[lane * 8 + (j ^ (lane & 7))] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int row = 4 * j + (lane >> 3);
            const float4 v = turn[row * 8 + ((lane & 7) ^ (row & 7))];
            const long long ro = __shfl_sync(kAll, off, row);
            if (x - lane + row >= rows) continue;
            if (direct) store_row4(p.out, ro + 32 * c + 4 * (lane & 7), v);
            else *reinterpret_cast<float4*>(p.part_o + (pr - lane + row) * D + 32 * c + 4 * (lane & 7)) = v;
          }
          __syncwarp();
        } else if (x < rows) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (direct) {  // bf16, as the queries of this kernel are
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out.ptr) + off + 32 * c + j) =
                  make_uint4(pack_bf16(o[j], o[j + 1]), pack_bf16(o[j + 2], o[j + 3]), pack_bf16(o[j + 4], o[j + 5]),
                             pack_bf16(o[j + 6], o[j + 7]));
            } else {
              float4* dst = reinterpret_cast<float4*>(p.part_o + pr * D + 32 * c + j);
              dst[0] = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
              dst[1] = make_float4(o[j + 4], o[j + 5], o[j + 6], o[j + 7]);
            }
          }
        }
      }
      if (x < rows) {
        if (!direct) p.part_ml[pr] = make_float4(m * dc::kLn2, l, lx, 0.0f);
        else if (want_lse) p.lse[orow * p.Hq + h] = l == 0.0f ? -INFINITY : m * dc::kLn2 + logf(lx);
      }
    }
  } else if (x < rows && !PAIR && wl < lane_parts) {
    // the lane without a tile: its split is empty
    p.part_ml[(static_cast<size_t>(unit) * p.splits + blockIdx.y * lane_parts + wl) * part_rows + x] =
        make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
  }
  }

  if (!ok) atomicOr(p.err, kDevErrWaitTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D, int R, bool V2, bool PAIR>
cudaError_t launch_main(const TreeParams& p, const TreeMma& t, int grid_splits, cudaStream_t s) {
  CUtensorMap map{};
  if (!V2) {
    const uint64_t slabs = p.c.page_size ? static_cast<uint64_t>(p.c.num_pages) * p.c.Hkv
                                         : static_cast<uint64_t>(p.c.B) * p.c.Hkv;
    const uint64_t rows = p.c.page_size ? p.c.page_size : p.c.T_cap;
    if (!encode_bf16_rows(&map, p.c.v, D, rows, slabs, 64)) return cudaErrorInvalidValue;
  }
  auto k = tree_mma_kernel<D, R, V2, PAIR>;
  constexpr int smem = Layout<D, R, V2, PAIR>::kBytes;
  static_assert(smem <= 232448, "shared memory of one CTA");
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  dim3 grid((t.blocks + (PAIR ? 1 : 0)) / (PAIR ? 2 : 1), grid_splits, p.c.B * p.c.Hkv);
  return launch_after(k, grid, kThreads, smem, s, p, t, map);
}

template <int D, int R>
cudaError_t launch_dr(const TreeParams& p, const TreeMma& t, int grid_splits, bool pair, cudaStream_t s) {
  const long long warps = static_cast<long long>(p.c.B) * p.c.Hkv * t.blocks * (kBlock / kPrepRows);
  const int row_ctas = static_cast<int>((warps + 7) / 8);
  const int mask_ctas = t.words ? (p.c.B * p.span.n + 7) / 8 : 0;
  // Launched in plain stream order, not early like the two kernels behind it: once it starts, all
  // work before this call is complete, so that the main kernel may read the cache and write empty
  // partials without waiting.
  tree_prep_kernel<D, R><<<row_ctas + mask_ctas, 256, 0, s>>>(p, t, row_ctas);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.c.vmode == HEADQ_V_2BIT)
    return pair ? launch_main<D, R, true, true>(p, t, grid_splits, s)
                : launch_main<D, R, true, false>(p, t, grid_splits, s);
  return pair ? launch_main<D, R, false, true>(p, t, grid_splits, s)
              : launch_main<D, R, false, false>(p, t, grid_splits, s);
}

}  // namespace

bool tree_mma_supported(const headq_cache& c) {
  return (c.d == 64 || c.d == 128) && (c.r == 0 || c.r == 8 || c.r == 16) && c.kmode == HEADQ_K_TOKEN &&
         (c.vmode == HEADQ_V_2BIT || c.v_dtype == HEADQ_BF16) && tensor_maps_available();
}

size_t tree_mma_image_bytes(const headq_cache& c) { return operand_bytes(c.d, c.r); }

cudaError_t launch_tree_mma(const TreeParams& p, const TreeMma& t, int grid_splits, bool pair, cudaStream_t s) {
  if (p.c.d == 128) {
    if (p.c.r == 16) return launch_dr<128, 16>(p, t, grid_splits, pair, s);
    if (p.c.r == 8) return launch_dr<128, 8>(p, t, grid_splits, pair, s);
    return launch_dr<128, 0>(p, t, grid_splits, pair, s);
  }
  if (p.c.r == 16) return launch_dr<64, 16>(p, t, grid_splits, pair, s);
  if (p.c.r == 8) return launch_dr<64, 8>(p, t, grid_splits, pair, s);
  return launch_dr<64, 0>(p, t, grid_splits, pair, s);
}

}  // namespace headq
