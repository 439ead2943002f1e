// headq_tree_attn: several new tokens per sequence attend over the HeadQ cache, the new
// ones among themselves under a tree mask ("HeadQ: Model-Visible Distortion and
// Score-Space Correction for KV-Cache Quantization", gist.science summary, section 3,
// step 3: base logit plus the side code's score-space correction; softmax and readout of
// section 2.2).  This file: the split plan, the fp32 kernel for every shape, the merge of
// the splits.  The tensor-core kernel is tree_mma.cu.
//
// tree_any_kernel: one CTA per (32 query rows, split, sequence x KV head).  32-token
// tiles are decoded once into shared memory as rows of d key channels followed by the r
// side-code entries, the query rows as q followed by U_h^T q, so that one dot product of
// length d + r is the corrected logit.  Softmax statistics and outputs stay in registers
// (8 lanes per query row).  Long runs of tiles are bound by its shared-memory reads (one
// 16-byte load per four multiply-adds), small calls by one tile's chain of dependent steps
// and the two launches (8 new tokens, 16 heads, 512 cached: 15.4 us).  It serves fp32 queries
// and the shapes the tensor-core kernel does not take.
#include <math.h>

#include <algorithm>

#include "codec.cuh"
#include "tree.cuh"

namespace headq {
namespace {

constexpr int kRT = 32;   // query rows per CTA
constexpr int kTT = 32;   // tokens per tile
constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// float4 chunks per key / query row in shared memory: odd, so that 8 rows read at the
// same chunk fall in distinct banks
__host__ __device__ inline int row_chunks(int d, int r) { return ((d + r + 3) / 4) | 1; }

// four elements of a tensor that is fp32 or bf16, from a multiple of 4
__device__ __forceinline__ float4 load4(const void* base, long long off, bool bf16) {
  if (!bf16) return *reinterpret_cast<const float4*>(static_cast<const float*>(base) + off);
  const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + off);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

template <int D>
__global__ void __launch_bounds__(kThreads)
tree_any_kernel(const TreeParams p) {
  constexpr int NC = D / 4 > 8 ? D / 32 : 1;  // value chunks per lane
  extern __shared__ float4 smem4[];
  const int r = p.c.r, rc = row_chunks(D, r);
  float4* q_s = smem4;                     // [kRT][rc]
  float4* k_s = q_s + kRT * rc;            // [kTT][rc]
  float4* v_s = k_s + kTT * rc;            // [kTT][D / 4]
  float* s_s = reinterpret_cast<float*>(v_s + kTT * (D / 4));  // [kRT][kTT + 1]
  __shared__ long long row_s[kTT];

  const int tid = threadIdx.x;
  const int unit = blockIdx.z, b = unit / p.c.Hkv, kv = unit - b * p.c.Hkv;
  const int split = blockIdx.y;
  const SpanSeq sq = span_seq(p.span, b);
  const int rows = sq.n * p.G, x0 = blockIdx.x * kRT;
  if (x0 >= rows) return;
  const int L = sq.p0 < 0 ? 0 : sq.p0 + sq.n;  // tokens the call reads; none when it takes no part
  const int t_lo = split * p.chunk, t_hi = min(L, t_lo + p.chunk);

  // query rows, then U_h^T q
  const bool qb = p.q.dtype == HEADQ_BF16;
  float* qf = reinterpret_cast<float*>(q_s);
#pragma unroll 4
  for (int e = tid; e < kRT * (D / 4); e += kThreads) {
    const int x = e / (D / 4), c4 = e - x * (D / 4), xr = x0 + x;
    float4 v = make_float4(0, 0, 0, 0);
    if (xr < rows) {
      const int i = xr / p.G, g = xr - i * p.G;
      v = load4(p.q.ptr, (sq.row0 + i) * p.q.row_stride + (kv * p.G + g) * p.q.head_stride + 4 * c4, qb);
    }
    q_s[x * rc + c4] = v;
  }
  __syncthreads();
  const int r4 = (r + 3) / 4 * 4;
  for (int e = tid; e < kRT * r4; e += kThreads) {
    const int x = e / r4, i = e - x * r4;
    float a = 0.0f;
    if (i < r) {
      const float* up = p.U + static_cast<size_t>(kv) * D * r + i;
#pragma unroll 16
      for (int c = 0; c < D; ++c) a = fmaf(qf[x * rc * 4 + c], up[c * r], a);
    }
    qf[x * rc * 4 + D + i] = a * p.corr_sign;
  }

  // this thread's row and channels in the softmax and readout
  const int orow = tid >> 3, l8 = tid & 7;
  float m = -INFINITY, l = 0.0f;
  float4 acc[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) acc[k] = make_float4(0, 0, 0, 0);
  const int sy = tid >> 4, sx = tid & 15;  // logits of rows sy, sy+16 x tokens sx, sx+16
  const int node[2] = {(x0 + sy) / p.G, (x0 + sy + 16) / p.G};
  const int len4 = (D + r4) / 4;

  for (int t0 = t_lo; t0 < t_hi; t0 += kTT) {
    __syncthreads();  // the previous tile (and the query rows) are done with
    if (tid < kTT) {
      const int t = t0 + tid;
      row_s[tid] = t < t_hi ? static_cast<long long>(cache_row_read(p.c, b, kv, t, p.err)) : -1;
    }
    __syncthreads();
    for (int e = tid; e < kTT * (D / 4); e += kThreads) {
      const int tt = e / (D / 4), c4 = e - tt * (D / 4);
      const long long row = row_s[tt];
      float4 k = make_float4(0, 0, 0, 0), v = k;
      if (row >= 0) {
        const size_t gr = row * num_groups(D) + 4 * c4 / group_size(D);
        k = decode4(p.c.k_codes[row * (D / 4) + c4], p.c.k_scale[gr], p.c.k_min[gr]);
        if (p.c.vmode == HEADQ_V_2BIT) {
          v = decode4(p.c.v_codes[row * (D / 4) + c4], p.c.v_scale[gr], p.c.v_min[gr]);
        } else {
          v = load4(p.c.v, row * D + 4 * c4, p.c.v_dtype == HEADQ_BF16);
        }
      }
      k_s[tt * rc + c4] = k;
      v_s[tt * (D / 4) + c4] = v;
    }
    float* kf = reinterpret_cast<float*>(k_s);
    for (int e = tid; e < kTT * r4; e += kThreads) {
      const int tt = e / r4, i = e - tt * r4;
      const long long row = row_s[tt];
      kf[tt * rc * 4 + D + i] =
          row >= 0 && i < r ? nibble(p.c.z_codes + row * (r / 2), i) * p.c.z_scale[row] : 0.0f;
    }
    __syncthreads();

    float s[2][2] = {{0, 0}, {0, 0}};
    for (int c = 0; c < len4; ++c) {
      float4 a[2], w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) a[k] = q_s[(sy + 16 * k) * rc + c];
#pragma unroll
      for (int k = 0; k < 2; ++k) w[k] = k_s[(sx + 16 * k) * rc + c];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[i][j] = fmaf(a[i].x, w[j].x, s[i][j]);
          s[i][j] = fmaf(a[i].y, w[j].y, s[i][j]);
          s[i][j] = fmaf(a[i].z, w[j].z, s[i][j]);
          s[i][j] = fmaf(a[i].w, w[j].w, s[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int x = x0 + sy + 16 * i, t = t0 + sx + 16 * j;
        const bool see = x < rows && t < t_hi && (t < sq.p0 || tree_sees(p, b, node[i], t - sq.p0));
        s_s[(sy + 16 * i) * (kTT + 1) + sx + 16 * j] = see ? s[i][j] * p.sm_scale : -INFINITY;
      }
    __syncthreads();

    float* sr = s_s + orow * (kTT + 1);
    float sv[4], mx = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      sv[k] = sr[l8 + 8 * k];
      mx = fmaxf(mx, sv[k]);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float base = mx == -INFINITY ? 0.0f : mx;
    const float f = exp2f((m - base) * kLog2e);  // m = -inf: 0
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float e = exp2f((sv[k] - base) * kLog2e);  // differences are taken before the scaling
      sum += e;
      sr[l8 + 8 * k] = e;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f + sum;
    m = mx;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      acc[k].x *= f; acc[k].y *= f; acc[k].z *= f; acc[k].w *= f;
    }
    __syncwarp();
    const int nt = min(kTT, t_hi - t0);
    for (int tt = 0; tt < nt; ++tt) {
      const float e = sr[tt];
      if (e == 0.0f) continue;  // a masked token's values are not looked at
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        if (D / 4 < 8 && l8 >= D / 4) continue;
        const float4 v = v_s[tt * (D / 4) + l8 + 8 * k];
        acc[k].x = fmaf(e, v.x, acc[k].x);
        acc[k].y = fmaf(e, v.y, acc[k].y);
        acc[k].z = fmaf(e, v.z, acc[k].z);
        acc[k].w = fmaf(e, v.w, acc[k].w);
      }
    }
  }

  const int x = x0 + orow;
  if (x >= rows) return;
  if (p.splits > 1) {
    const size_t pr = (static_cast<size_t>(unit) * p.splits + split) * (static_cast<size_t>(p.span.n) * p.G) + x;
#pragma unroll
    for (int k = 0; k < NC; ++k)
      if (l8 + 8 * k < D / 4) reinterpret_cast<float4*>(p.part_o + pr * D)[l8 + 8 * k] = acc[k];
    if (l8 == 0) p.part_ml[pr] = make_float4(m, l, l, 0.0f);
    return;
  }
  const int i = x / p.G, g = x - i * p.G;
  const size_t orow_g = static_cast<size_t>(sq.row0) + i;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c4 = l8 + 8 * k;
    if (c4 >= D / 4) continue;
    const float4 o = make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv);
    store_row4(p.out, orow_g * p.out.row_stride + (kv * p.G + g) * p.out.head_stride + 4 * c4, o);
  }
  if (p.lse && l8 == 0) p.lse[orow_g * p.Hq + kv * p.G + g] = l == 0.0f ? -INFINITY : m + logf(l);
}

// One warp per query row: out = sum_s e^{m_s - M} o_s / sum_s e^{m_s - M} l_s over the
// splits.  A row that sees nothing (every m_s = -inf) gets 0 and -inf.
template <int D>
__global__ void __launch_bounds__(128)
tree_merge_kernel(const TreeParams p) {
  wait_for_prior_kernel();
  const int unit = blockIdx.y, b = unit / p.c.Hkv, kv = unit - b * p.c.Hkv;
  const SpanSeq sq = span_seq(p.span, b);
  const int x = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (x >= sq.n * p.G) return;
  constexpr int NC = (D / 4 + 31) / 32;
  const size_t ru = static_cast<size_t>(p.span.n) * p.G;
  const size_t pr = static_cast<size_t>(unit) * p.splits * ru + x;
  float M = -INFINITY;
  for (int s = lane; s < p.splits; s += 32) M = fmaxf(M, p.part_ml[pr + s * ru].x);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float base = M == -INFINITY ? 0.0f : M;
  float L = 0.0f, Lx = 0.0f;
  float4 acc[NC];
#pragma unroll
  for (int k = 0; k < NC; ++k) acc[k] = make_float4(0, 0, 0, 0);
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) {
    const float4 ml = p.part_ml[pr + s * ru];
    const float w = exp2f((ml.x - base) * kLog2e);
    L = fmaf(w, ml.y, L);
    Lx = fmaf(w, ml.z, Lx);
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      if (lane + 32 * k >= D / 4) continue;
      const float4 o = reinterpret_cast<const float4*>(p.part_o + (pr + s * ru) * D)[lane + 32 * k];
      if (ml.y != 0.0f) {
        acc[k].x = fmaf(w, o.x, acc[k].x);
        acc[k].y = fmaf(w, o.y, acc[k].y);
        acc[k].z = fmaf(w, o.z, acc[k].z);
        acc[k].w = fmaf(w, o.w, acc[k].w);
      }
    }
  }
  const int i = x / p.G, g = x - i * p.G;
  const size_t orow = static_cast<size_t>(sq.row0) + i;
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
  for (int k = 0; k < NC; ++k) {
    const int c4 = lane + 32 * k;
    if (c4 >= D / 4) continue;
    store_row4(p.out, orow * p.out.row_stride + (kv * p.G + g) * p.out.head_stride + 4 * c4,
               make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv));
  }
  if (p.lse && lane == 0) p.lse[orow * p.Hq + kv * p.G + g] = L == 0.0f ? -INFINITY : M + logf(Lx);
}

// Single tokens on the decode kernels: the queries gathered to [B, Hq, d], and the tokens each
// sequence's query sees -- the first p0, and itself unless its mask entry is 0.
__global__ void __launch_bounds__(256)
tree_one_prep_kernel(const TreeParams p, const TreeOne w) {
  const int b = blockIdx.x, tid = threadIdx.x;
  const SpanSeq sq = span_seq(p.span, b);
  const bool part = sq.n > 0 && sq.p0 >= 0;
  if (tid == 0) w.lens[b] = part ? sq.p0 + (tree_sees(p, b, 0, 0) ? 1 : 0) : 0;
  for (int h = tid; h < p.c.Hkv; h += 256) w.counters[b * p.c.Hkv + h] = 0u;
  const int per = p.c.d / 8;  // 16-byte pieces of a bf16 row
  for (int e = tid; e < p.Hq * per; e += 256) {
    const int h = e / per, c = e - h * per;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (part)
      x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.ptr) + sq.row0 * p.q.row_stride +
                                          h * p.q.head_stride + 8 * c);
    static_cast<uint4*>(w.q)[static_cast<size_t>(b) * p.Hq * per + e] = x;
  }
}

// Their results to the packed rows.  The decode kernels give 0 for a sum of weights that is not
// positive; one that is not a number reaches the log-sum-exp (nan_lse) and makes the row NaN.
__global__ void __launch_bounds__(256)
tree_one_finish_kernel(const TreeParams p, const TreeOne w) {
  const int b = blockIdx.x, tid = threadIdx.x;
  const SpanSeq sq = span_seq(p.span, b);
  if (sq.n == 0) return;
  const int per = p.c.d / 4;
  const size_t r0 = static_cast<size_t>(b) * p.Hq;
  for (int e = tid; e < p.Hq * per; e += 256) {
    const int h = e / per, c4 = e - h * per;
    float4 o = reinterpret_cast<const float4*>(w.out)[r0 * per + e];
    const float lse = w.lse[r0 + h];
    if (lse != lse) o.x = o.y = o.z = o.w = NAN;
    store_row4(p.out, sq.row0 * p.out.row_stride + h * p.out.head_stride + 4 * c4, o);
    if (p.lse && c4 == 0) p.lse[static_cast<size_t>(sq.row0) * p.Hq + h] = lse;
  }
}

template <int D>
cudaError_t launch_any(const TreeParams& p, cudaStream_t s) {
  const int rc = row_chunks(D, p.c.r);
  const size_t smem = 16 * (static_cast<size_t>(kRT + kTT) * rc + kTT * (D / 4)) + 4 * kRT * (kTT + 1);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(tree_any_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  dim3 grid((p.span.n * p.G + kRT - 1) / kRT, p.splits, p.c.B * p.c.Hkv);
  tree_any_kernel<D><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_merge(const TreeParams& p, cudaStream_t s) {
  dim3 grid((p.span.n * p.G + 3) / 4, p.c.B * p.c.Hkv);
  return launch_after(tree_merge_kernel<D>, grid, 128, 0, s, p);
}

}  // namespace

// Single tokens: the decode kernels where they use the tensor cores; a 128-row tile of which
// Hq / Hkv <= 8 rows are live waits longer on each step (69 us against 44 at 16 sequences of
// up to 8192 tokens, 28 heads on 4).  Tensor cores: one CTA per SM, so the splits that minimise
// waves x (tiles per CTA + 3), the 3 standing for a CTA's set-up, first loads and epilogue;
// at most kMaxWaves waves, which bounds the workspace.  fp32 kernel: about four CTAs per SM,
// chunks of whole 32-token tiles.
constexpr long long kMaxWaves = 8;

TreePlan tree_plan(const headq_cache& c, int Hq, int n, int T, bool q_bf16) {
  const long long units = static_cast<long long>(c.B) * c.Hkv, rows = static_cast<long long>(n) * (Hq / c.Hkv);
  TreePlan tp{false, q_bf16 && tree_mma_supported(c), false, static_cast<int>((rows + 127) / 128), 1, 1, 128};
  if (n <= 0 || units <= 0) return tp;
  const int sms = sm_count();
  if (tp.mma && n == 1 && units <= kMaxFusedUnits && decode_plan(c, Hq, T).mma) {
    tp.one = true;
    return tp;
  }
  if (tp.mma) {
    tp.pair = tp.blocks > 1;
    const long long ctas = units * (tp.pair ? (tp.blocks + 1) / 2 : tp.blocks);
    const int tiles = T > 128 ? (T + 127) / 128 : 1;
    long long best = -1;
    for (int s = 1; s <= tiles && s <= sms && (s == 1 || ctas * s <= kMaxWaves * sms); ++s) {
      const int per = (tiles + s - 1) / s, used = (tiles + per - 1) / per;
      if (used != s) continue;
      const long long cost = ((ctas * s + sms - 1) / sms) * (per + 3) + (s > 1 ? 1 : 0);
      if (best < 0 || cost < best) {
        best = cost;
        tp.grid_splits = s;
        tp.chunk = per * 128;
      }
    }
    // the two lanes of a CTA that take alternate tiles end as two parts
    tp.parts = tp.grid_splits * (!tp.pair && tp.chunk > 128 ? 2 : 1);
    return tp;
  }
  const int tiles = T > kTT ? (T + kTT - 1) / kTT : 1;
  long long s = 4ll * sms / (units * ((rows + kRT - 1) / kRT));
  s = s < 1 ? 1 : (s > 64 ? 64 : s);
  if (s > tiles) s = tiles;
  const int per = static_cast<int>((tiles + s - 1) / s);
  tp.chunk = per * kTT;
  tp.grid_splits = tp.parts = (tiles + per - 1) / per;
  return tp;
}

// A call's splits are not monotone in its sizes, so the bound comes from what limits them:
// at least `units` CTAs a split, the caps on the grid above, and whole tiles; and a grid of
// C CTAs holds at most C x (rows of a CTA) x (parts of a CTA) partial rows.
size_t tree_max_part_rows(const headq_cache& c, int Hq, int n, int T, bool mma) {
  const long long units = static_cast<long long>(c.B) * c.Hkv, rows = units * n * (Hq / c.Hkv);
  if (rows <= 0) return 0;
  const long long grid = (mma ? kMaxWaves : 4) * sm_count(), tile = mma ? 128 : kTT;
  const long long tiles = T > tile ? (T + tile - 1) / tile : 1;
  const long long splits = std::min<long long>({tiles, std::max(1ll, grid / units), mma ? sm_count() : 64ll});
  return static_cast<size_t>(mma ? std::min(rows * 2 * splits, 256 * std::max(grid, units))
                                 : std::min(rows * splits, kRT * grid));
}

cudaError_t launch_tree_one(const TreeParams& p, const TreeOne& w, cudaStream_t s) {
  tree_one_prep_kernel<<<p.c.B, 256, 0, s>>>(p, w);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const DecodePlan dp = decode_plan(p.c, p.Hq, p.span.T);
  DecodeParams d{};
  d.c = p.c;
  d.q = w.q;
  d.q_bf16 = true;
  d.Hq = p.Hq;
  d.G = p.G;
  d.T = p.span.T;
  d.seq_lens = w.lens;
  d.U = p.U;
  d.sm_scale = p.sm_scale;
  d.corr_sign = p.corr_sign;
  d.splits = dp.splits;
  d.chunk = dp.chunk;
  d.err = p.err;
  d.counters = w.counters;
  d.fused = dp.fused;
  d.part = w.part;
  d.out = w.out;
  d.lse = w.lse;
  d.nan_lse = true;
  if ((e = launch_decode(d, dp.mma, s)) != cudaSuccess) return e;
  tree_one_finish_kernel<<<p.c.B, 256, 0, s>>>(p, w);
  return cudaGetLastError();
}

cudaError_t launch_tree(const TreeParams& p, const TreeMma& t, const TreePlan& plan, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  if (plan.mma) {
    e = launch_tree_mma(p, t, plan.grid_splits, plan.pair, s);
    if (e != cudaSuccess || plan.parts == 1) return e;
    return p.c.d == 128 ? launch_merge<128>(p, s) : launch_merge<64>(p, s);
  }
#define HEADQ_TREE_D(D)                                              \
  case D:                                                            \
    e = launch_any<D>(p, s);                                         \
    if (e == cudaSuccess && p.splits > 1) e = launch_merge<D>(p, s); \
    break;
  switch (p.c.d) {
    HEADQ_TREE_D(8)
    HEADQ_TREE_D(16)
    HEADQ_TREE_D(32)
    HEADQ_TREE_D(64)
    HEADQ_TREE_D(128)
    HEADQ_TREE_D(256)
  }
#undef HEADQ_TREE_D
  return e;
}

}  // namespace headq
