// headq_cache_read: cached tokens decoded to dense rows -- the key the corrected logit
// reads, k^base + sigma U_h z^ ("HeadQ: Model-Visible Distortion and Score-Space
// Correction for KV-Cache Quantization", gist.science summary, section 3, steps 2 and 3),
// and the cached value.  fp32 arithmetic, one rounding to the output's dtype.
//
// Bound by HBM: a token of a KV head is 332 bytes in (d = 128, r = 16, bf16 values) and
// 512 out.  cache_read_kernel (d 64 or 128, r 0, 8 or 16): one warp per 32-token tile of one
// (sequence, KV head).  The side code's part is a product of its small integers (exact in
// bf16) with U_h in three bf16 parts (24 bits), tokens on the M side of mma.sync.m16n8k16,
// summed in fp32: 12 instructions per 16 tokens x 32 channels, where packed multiply-adds
// took 32 per token and the broadcast of the side code kept shared memory 74 % busy (344 us
// on the 131072 x 8 tokens of the long-context layer).  The columns of the products are
// ordered so that a lane ends with 8 neighbouring channels of its tokens: one 16-byte store
// each in bf16.  Four CTAs an SM and a rolled loop over the groups (64 registers) hide the
// loads' latency better than two CTAs with it unrolled: 153 against 185 us there, 5.8 TB/s.
// Every other shape runs cache_read_any_kernel, one thread per 4 channels.
#include "codec.cuh"

namespace headq {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kTok = 32;  // tokens per warp tile

// 2-bit code as an exact float: 2^23 + c has c in its low mantissa bits
__device__ __forceinline__ float code_f(uint32_t bits) {
  return __uint_as_float(0x4B000000u | (bits & 3u)) - 8388608.0f;
}

// min + code * scale of a 2-bit code.  EXACT (fp32 outputs): the product is rounded before the sum,
// which is the base value that the write took the residual from, bit for bit.  Otherwise one fused
// step, whose last bit the rounding to bf16 covers: 78.0 us against 80.4 on the full-KV 2-bit
// prefixes, 160.4 against 162.0 on the long context.
template <bool EXACT>
__device__ __forceinline__ float dequant(uint32_t bits, float scale, float mn) {
  const float c = code_f(bits);
  return EXACT ? __fadd_rn(__fmul_rn(c, scale), mn) : fmaf(c, scale, mn);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// N (4 or 8) consecutive outputs of one row
template <int N>
__device__ __forceinline__ void store_out(const headq_rows& o, size_t off, const float (&x)[N]) {
  if (o.dtype == HEADQ_BF16) {
    uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(o.ptr) + off);
    if constexpr (N == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                                pack_bf16(x[6], x[7]));
    else *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(o.ptr) + off);
#pragma unroll
    for (int k = 0; k < N / 4; ++k) p[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
  }
}

// A warp's tile: packed codes and (minimum, scale) per group; rows a word (a pair) longer
// than their contents, so that 8 rows read at one place fall in distinct banks.
template <int D>
struct WarpTile {
  static constexpr int NG = D / 32;
  uint32_t codes[kTok][D / 16 + 1];
  float2 ms[kTok][NG + 1];
};

// this lane's token's codes, minima and scales into the tile
template <int D>
__device__ __forceinline__ void stage_codes(WarpTile<D>& t, int lane, long long row, const uint8_t* codes,
                                            const float* scale, const float* mn, bool groups) {
  constexpr int NG = D / 32;
  uint4 c[D / 64];
  float s[NG], m[NG];
#pragma unroll
  for (int k = 0; k < D / 64; ++k) c[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int g = 0; g < NG; ++g) s[g] = m[g] = 0.0f;
  if (row >= 0) {
    const uint4* p = reinterpret_cast<const uint4*>(codes + row * (D / 4));
#pragma unroll
    for (int k = 0; k < D / 64; ++k) c[k] = __ldg(p + k);
    if (groups) {
      if constexpr (NG == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(scale) + row);
        const float4 b = __ldg(reinterpret_cast<const float4*>(mn) + row);
        s[0] = a.x; s[1] = a.y; s[2] = a.z; s[3] = a.w;
        m[0] = b.x; m[1] = b.y; m[2] = b.z; m[3] = b.w;
      } else {
        const float2 a = __ldg(reinterpret_cast<const float2*>(scale) + row);
        const float2 b = __ldg(reinterpret_cast<const float2*>(mn) + row);
        s[0] = a.x; s[1] = a.y;
        m[0] = b.x; m[1] = b.y;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < D / 64; ++k) {
    t.codes[lane][4 * k] = c[k].x;
    t.codes[lane][4 * k + 1] = c[k].y;
    t.codes[lane][4 * k + 2] = c[k].z;
    t.codes[lane][4 * k + 3] = c[k].w;
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) t.ms[lane][g] = make_float2(m[g], s[g]);
}

// 8 codes (channels 8 q .. 8 q + 7 of group g) of a token
template <int D>
__device__ __forceinline__ uint32_t codes8(const WarpTile<D>& t, int tok, int g, int q) {
  return reinterpret_cast<const uint16_t*>(t.codes[tok])[4 * g + q];
}
// dequant() of them
template <int D, bool EXACT>
__device__ __forceinline__ void base8(const WarpTile<D>& t, int tok, int g, int q, float (&x)[8]) {
  const uint32_t c = codes8<D>(t, tok, g, q);
  const float2 ms = t.ms[tok][g];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = dequant<EXACT>(c >> (2 * k), ms.y, ms.x);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// entries 2t, 2t + 1 of a side code (one byte) as bf16
__device__ __forceinline__ uint32_t side_pair(uint32_t byte) {
  const float a = __uint_as_float((byte & 15u) ^ 0x4B000008u) - 8388616.0f;  // nibble ^ 8 is w + 8
  const float b = __uint_as_float(((byte >> 4) & 15u) ^ 0x4B000008u) - 8388616.0f;
  return pack_bf16(a, b);
}

// SPLIT: keys (blockIdx.y 0) and values (1) by CTAs of their own.
template <int D, int R, bool KCH, bool SPLIT, bool EXACT>
__global__ void __launch_bounds__(kWarps * 32, 4)
cache_read_kernel(const headq_cache c, const headq_span span, const float* U, float sigma,
                  const headq_rows ko, const headq_rows vo, unsigned* err, int blocks, int sub) {
  constexpr int NG = D / 32;
  using Tile = WarpTile<D>;
  __shared__ Tile tiles[kWarps];
  __shared__ uint2 u_s[R > 0 ? NG * 4 * 3 * 32 : 1];  // [group][n-tile][part][lane]
  Tile& t = tiles[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kv = blockIdx.x % c.Hkv;
  const int bt = blockIdx.x / c.Hkv, b = bt / blocks;
  const int i0 = ((bt - b * blocks) * kWarps + warp) * kTok * sub;
  const SpanSeq sq = span_seq(span, b);
  if (sq.p0 < 0 || (bt - b * blocks) * kWarps * kTok * sub >= sq.n) return;
  const int gq = lane >> 2, tq = lane & 3;  // a lane's tokens gq, gq + 8 and channels 8 tq .. of a group

  if constexpr (R > 0) {
    if (ko.ptr && !(SPLIT && blockIdx.y == 1)) {
      // n-tile j's column 2 t + e is channel 8 t + 2 j + e of its group; parts of U from the
      // leading one down
      for (int e = threadIdx.x; e < NG * 4 * 32; e += kWarps * 32) {
        const int ln = e & 31, j = (e >> 5) & 3, g = e >> 7;
        const int col = ln >> 2, ch = 32 * g + 8 * (col >> 1) + 2 * j + (col & 1), k0 = 2 * (ln & 3);
        const float* up = U + (static_cast<size_t>(kv) * D + ch) * R;
        float x[4] = {__ldg(up + k0), __ldg(up + k0 + 1), 0.0f, 0.0f};
        if (R > 8) {
          x[2] = __ldg(up + k0 + 8);
          x[3] = __ldg(up + k0 + 9);
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint32_t lo = pack_bf16(x[0], x[1]), hi = pack_bf16(x[2], x[3]);
          u_s[((g * 4 + j) * 3 + part) * 32 + ln] = make_uint2(lo, hi);
          x[0] -= __uint_as_float(lo << 16);
          x[1] -= __uint_as_float(lo & 0xffff0000u);
          x[2] -= __uint_as_float(hi << 16);
          x[3] -= __uint_as_float(hi & 0xffff0000u);
        }
      }
    }
    __syncthreads();
  }

  for (int s = 0; s < sub; ++s) {
    const int i1 = i0 + s * kTok;
    if (i1 >= sq.n) return;
    const int nt = min(kTok, sq.n - i1);
    long long row = -1;
    if (lane < nt) {
      row = cache_row(c, b, kv, sq.p0 + i1 + lane);
      if (row < 0 && err) atomicOr(err, kDevErrBadPage);
    }
    const size_t out0 = static_cast<size_t>(sq.row0) + i1;
    if (ko.ptr && !(SPLIT && blockIdx.y == 1)) {
      __syncwarp();
      stage_codes<D>(t, lane, row, c.k_codes, c.k_scale, c.k_min, !KCH);
      uint32_t zc[R > 0 ? R / 8 : 1];
      float zs = 0.0f;
      if constexpr (R > 0) {
#pragma unroll
        for (int k = 0; k < R / 8; ++k) zc[k] = 0x00000000u;
        if (row >= 0) {
          const uint32_t* zp = reinterpret_cast<const uint32_t*>(c.z_codes + row * (R / 2));
#pragma unroll
          for (int k = 0; k < R / 8; ++k) zc[k] = __ldg(zp + k);
          zs = sigma * __ldg(c.z_scale + row);
        }
      }
      __syncwarp();
#pragma unroll 1
      for (int mt = 0; mt < 2 && 16 * mt < nt; ++mt) {
        uint32_t a[4] = {0, 0, 0, 0};
        float zt[2] = {0.0f, 0.0f};
        if constexpr (R > 0) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = 16 * mt + gq + 8 * e;
            const uint32_t lo = __shfl_sync(kFull, zc[0], tok);
            a[e] = side_pair((lo >> (8 * tq)) & 255u);
            if constexpr (R > 8) {
              const uint32_t hi = __shfl_sync(kFull, zc[1], tok);
              a[2 + e] = side_pair((hi >> (8 * tq)) & 255u);
            }
            zt[e] = __shfl_sync(kFull, zs, tok);
          }
        }
        long long rt[2] = {0, 0};
        if constexpr (KCH) {
          rt[0] = __shfl_sync(kFull, row, 16 * mt + gq);
          rt[1] = __shfl_sync(kFull, row, 16 * mt + gq + 8);
        }
#pragma unroll 1
        for (int g = 0; g < NG; ++g) {
          float acc[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
          if constexpr (R > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int part = 2; part >= 0; --part) {  // the small parts first
                const uint2 bu = u_s[((g * 4 + j) * 3 + part) * 32 + lane];
                mma_bf16(acc[j], a, bu.x, bu.y);
              }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = 16 * mt + gq + 8 * e;
            float x[8];
            if constexpr (KCH) {
              const uint32_t cb = codes8<D>(t, tok, g, tq);
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = 0.0f;
              if (rt[e] >= 0) {
                const size_t o = static_cast<size_t>(rt[e] >> 6) * D + 32 * g + 8 * tq;
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = dequant<EXACT>(cb >> (2 * k), __ldg(c.k_scale + o + k), __ldg(c.k_min + o + k));
              }
            } else {
              base8<D, EXACT>(t, tok, g, tq, x);
            }
            if constexpr (R > 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                x[2 * j] = fmaf(acc[j][2 * e], zt[e], x[2 * j]);
                x[2 * j + 1] = fmaf(acc[j][2 * e + 1], zt[e], x[2 * j + 1]);
              }
            }
            if (tok < nt) store_out<8>(ko, (out0 + tok) * ko.row_stride + kv * ko.head_stride + 32 * g + 8 * tq, x);
          }
        }
      }
    }
    if (!vo.ptr || (SPLIT && blockIdx.y == 0)) continue;
    if (c.vmode == HEADQ_V_2BIT) {
      __syncwarp();
      stage_codes<D>(t, lane, row, c.v_codes, c.v_scale, c.v_min, true);
      __syncwarp();
      for (int tok = gq; tok < nt; tok += 8) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float x[8];
          base8<D, EXACT>(t, tok, g, tq, x);
          store_out<8>(vo, (out0 + tok) * vo.row_stride + kv * vo.head_stride + 32 * g + 8 * tq, x);
        }
      }
    } else if (c.v_dtype == HEADQ_BF16 && vo.dtype == HEADQ_BF16) {  // the same bits
      constexpr int CPR = D / 8;        // 16-byte chunks per row
      constexpr int RPI = 32 / CPR;     // rows per warp instruction
      constexpr int NB = 8;             // loads in flight per lane
      const uint16_t* src = static_cast<const uint16_t*>(c.v);
      uint16_t* dst = static_cast<uint16_t*>(vo.ptr);
      for (int r0 = 0; r0 < nt; r0 += RPI * NB) {
        uint4 x[NB];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const int tok = r0 + k * RPI + lane / CPR;
          const long long rt = __shfl_sync(kFull, row, tok & 31);
          x[k] = make_uint4(0, 0, 0, 0);
          if (tok < nt && rt >= 0) x[k] = __ldg(reinterpret_cast<const uint4*>(src + rt * D) + lane % CPR);
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const int tok = r0 + k * RPI + lane / CPR;
          if (tok < nt)
            *reinterpret_cast<uint4*>(dst + (out0 + tok) * vo.row_stride + kv * vo.head_stride + 8 * (lane % CPR)) = x[k];
        }
      }
    } else {
      const bool vb = c.v_dtype == HEADQ_BF16;
      for (int tok = 0; tok < nt; ++tok) {
        const long long rt = __shfl_sync(kFull, row, tok);
        if (lane >= D / 4) continue;
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = rt < 0 ? 0.0f : load_elem(c.v, rt * D + lane * 4 + k, vb);
        store_out<4>(vo, (out0 + tok) * vo.row_stride + kv * vo.head_stride + lane * 4, x);
      }
    }
  }
}

// Any shape: one thread per (row, KV head, 4 channels).
__global__ void __launch_bounds__(256)
cache_read_any_kernel(const headq_cache c, const headq_span span, const float* U, float sigma,
                      const headq_rows ko, const headq_rows vo, unsigned* err) {
  const int b = blockIdx.y;
  const SpanSeq sq = span_seq(span, b);
  if (sq.p0 < 0) return;
  const int d4 = c.d / 4, ng = num_groups(c.d), gs = group_size(c.d);
  const long long total = static_cast<long long>(sq.n) * c.Hkv * d4;
  for (long long x = blockIdx.x * 256ll + threadIdx.x; x < total; x += gridDim.x * 256ll) {
    const int c4 = static_cast<int>(x % d4) * 4;
    const int kv = static_cast<int>(x / d4 % c.Hkv);
    const int i = static_cast<int>(x / d4 / c.Hkv);
    const long long row = cache_row(c, b, kv, sq.p0 + i);
    float k[4] = {0, 0, 0, 0}, v[4] = {0, 0, 0, 0};
    if (row < 0) {
      if (err) atomicOr(err, kDevErrBadPage);
    } else {
      const size_t gr = row * ng + c4 / gs;
      if (ko.ptr) {
        const uint32_t by = c.k_codes[row * d4 + c4 / 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool ch = c.kmode == HEADQ_K_CHANNEL;
          const size_t o = ch ? static_cast<size_t>(row >> 6) * c.d + c4 + e : gr;
          k[e] = dequant<true>(by >> (2 * e), c.k_scale[o], c.k_min[o]);
        }
        if (c.r > 0) {
          const float zs = sigma * c.z_scale[row];
          const float* up = U + (static_cast<size_t>(kv) * c.d + c4) * c.r;
          for (int r = 0; r < c.r; ++r) {
            const float w = zs * nibble(c.z_codes + row * (c.r / 2), r);
#pragma unroll
            for (int e = 0; e < 4; ++e) k[e] = fmaf(up[e * c.r + r], w, k[e]);
          }
        }
      }
      if (vo.ptr) {
        if (c.vmode == HEADQ_V_2BIT) {
          const uint32_t by = c.v_codes[row * d4 + c4 / 4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = dequant<true>(by >> (2 * e), c.v_scale[gr], c.v_min[gr]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = load_elem(c.v, row * c.d + c4 + e, c.v_dtype == HEADQ_BF16);
        }
      }
    }
    const size_t orow = static_cast<size_t>(sq.row0) + i;
    if (ko.ptr) store_out<4>(ko, orow * ko.row_stride + kv * ko.head_stride + c4, k);
    if (vo.ptr) store_out<4>(vo, orow * vo.row_stride + kv * vo.head_stride + c4, v);
  }
}

template <int D, int R, bool EXACT>
auto read_kernel(bool kch, bool split) {
  return split ? (kch ? cache_read_kernel<D, R, true, true, EXACT> : cache_read_kernel<D, R, false, true, EXACT>)
               : (kch ? cache_read_kernel<D, R, true, false, EXACT> : cache_read_kernel<D, R, false, false, EXACT>);
}

template <int D, int R>
cudaError_t launch_fast(const CacheReadParams& p, cudaStream_t s) {
  // Large calls, with several waves of warps: 2 tiles per warp (U_h is then split half as
  // often), keys and values one after the other.  Smaller ones wait on a warp's chain of
  // loads: keys and values by CTAs of their own (8192 tokens x 8 heads 15.6 -> 13.8 us, 296 x 12
  // 4.9 -> 3.9; but 131072 x 8 152 -> 166).
  const long long warps = static_cast<long long>(p.c.B) * p.c.Hkv * ((p.span.n + kTok - 1) / kTok);
  const int sub = warps >= 4ll * 16 * sm_count() ? 2 : 1;
  const int per = kTok * sub * kWarps, blocks = (p.span.n + per - 1) / per;
  const long long grid = static_cast<long long>(p.c.B) * p.c.Hkv * blocks;
  const bool split = sub == 1 && p.k.ptr && p.v.ptr;
  const bool kch = p.c.kmode == HEADQ_K_CHANNEL;
  const bool exact = (p.k.ptr && p.k.dtype == HEADQ_F32) || (p.v.ptr && p.v.dtype == HEADQ_F32);
  auto k = exact ? read_kernel<D, R, true>(kch, split) : read_kernel<D, R, false>(kch, split);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 g(static_cast<unsigned>(grid), split ? 2 : 1);
  k<<<g, kWarps * 32, 0, s>>>(p.c, p.span, p.U, p.sigma, p.k, p.v, p.err, blocks, sub);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_fast_d(const CacheReadParams& p, cudaStream_t s) {
  if (p.c.r == 16) return launch_fast<D, 16>(p, s);
  if (p.c.r == 8) return launch_fast<D, 8>(p, s);
  return launch_fast<D, 0>(p, s);
}

}  // namespace

cudaError_t launch_cache_read(const CacheReadParams& p, cudaStream_t s) {
  if (p.c.r == 0 || p.c.r == 8 || p.c.r == 16) {
    if (p.c.d == 128) return launch_fast_d<128>(p, s);
    if (p.c.d == 64) return launch_fast_d<64>(p, s);
  }
  const long long per = static_cast<long long>(p.span.n) * p.c.Hkv * (p.c.d / 4);
  const long long want = (per + 255) / 256, most = (8ll * sm_count() + p.c.B - 1) / p.c.B;
  dim3 grid(static_cast<unsigned>(want < most ? want : most), p.c.B);
  cache_read_any_kernel<<<grid, 256, 0, s>>>(p.c, p.span, p.U, p.sigma, p.k, p.v, p.err);
  return cudaGetLastError();
}

}  // namespace headq
