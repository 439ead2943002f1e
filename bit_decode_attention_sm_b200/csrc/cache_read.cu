// headq_cache_read: cached tokens decoded to dense rows -- the key the corrected logit
// reads, k^base + sigma U_h z^ ("HeadQ: Model-Visible Distortion and Score-Space
// Correction for KV-Cache Quantization", gist.science summary, section 3, steps 2 and 3),
// and the cached value.  fp32 arithmetic, one rounding to the output's dtype.
//
// Bound by HBM: a token of a KV head is 332 bytes in (d = 128, r = 16, bf16 values) and
// 512 out.  cache_read_kernel (d 64 or 128, r 0, 8 or 16): one warp per 32-token tile of
// one (sequence, KV head), each lane owning d/32 channels whose rows of U_h stay in its
// registers, so a token costs r/2 broadcast loads of its side code and d*r/64 packed
// multiply-adds per lane; codes and scales pass through the warp's shared memory once.
// The 8 warps of a CTA take neighbouring KV heads, so that their output rows are one run
// of memory.  Every other shape runs cache_read_any_kernel, one thread per 4 channels.
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

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// N (2 or 4) consecutive outputs of one row
template <int N>
__device__ __forceinline__ void store_out(const headq_rows& o, size_t off, const float (&x)[N]) {
  if (o.dtype == HEADQ_BF16) {
    uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(o.ptr) + off);
    if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    else *p = pack_bf16(x[0], x[1]);
  } else {
    float* p = static_cast<float*>(o.ptr) + off;
    if constexpr (N == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  }
}

// A warp's tile: packed codes, (minimum, scale) per group, side code entries doubled for
// the packed multiply-add.
template <int D, int R>
struct WarpTile {
  static constexpr int NG = D / 32;
  uint32_t codes[kTok][D / 16];
  float2 ms[kTok][NG];
  float2 w[kTok][R > 0 ? R : 1];
};

// this lane's token's codes, minima and scales into the tile
template <int D, int R>
__device__ __forceinline__ void stage_codes(WarpTile<D, R>& t, int lane, long long row,
                                            const uint8_t* codes, const float* scale,
                                            const float* mn, bool groups) {
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
  uint4* d = reinterpret_cast<uint4*>(t.codes[lane]);
#pragma unroll
  for (int k = 0; k < D / 64; ++k) d[k] = c[k];
#pragma unroll
  for (int g = 0; g < NG; ++g) t.ms[lane][g] = make_float2(m[g], s[g]);
}

// the lane's channels of a token: min + code * scale
template <int D, int R>
__device__ __forceinline__ void base_values(const WarpTile<D, R>& t, int tok, int lane,
                                            float (&x)[D / 32]) {
  constexpr int N = D / 32;
  const uint32_t by = reinterpret_cast<const uint8_t*>(t.codes[tok])[lane * N / 4] >> (N == 4 ? 0 : 4 * (lane & 1));
  const float2 ms = t.ms[tok][lane * N / 32];
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = fmaf(code_f(by >> (2 * k)), ms.y, ms.x);
}

template <int D, int R, bool KCH>
__global__ void __launch_bounds__(kWarps * 32, 2)
cache_read_kernel(const headq_cache c, const headq_span span, const float* U, float sigma,
                  const headq_rows ko, const headq_rows vo, unsigned* err, int tiles, int sub) {
  constexpr int N = D / 32;
  extern __shared__ uint4 smem[];
  using Tile = WarpTile<D, R>;
  Tile& t = reinterpret_cast<Tile*>(smem)[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int kv = static_cast<int>(unit % c.Hkv);
  const long long bt = unit / c.Hkv;
  const int b = static_cast<int>(bt / tiles);
  if (b >= c.B) return;
  const int i0 = static_cast<int>(bt % tiles) * kTok * sub;
  const SpanSeq sq = span_seq(span, b);
  if (sq.p0 < 0 || i0 >= sq.n) return;

  uint64_t u[R > 0 ? R : 1][N / 2];  // (channel pair) of each basis vector
  if constexpr (R > 0) {
    if (ko.ptr) {
      const float* up = U + (static_cast<size_t>(kv) * D + lane * N) * R;
#pragma unroll
      for (int k = 0; k < N / 2; ++k)
#pragma unroll
        for (int i = 0; i < R; ++i)
          u[i][k] = codec::pk2(__ldg(up + 2 * k * R + i), __ldg(up + (2 * k + 1) * R + i));
    }
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
    if (ko.ptr) {
      __syncwarp();
      stage_codes<D, R>(t, lane, row, c.k_codes, c.k_scale, c.k_min, !KCH);
      if constexpr (R > 0) {
        uint32_t zc[R / 8];
        float zs = 0.0f;
#pragma unroll
        for (int k = 0; k < R / 8; ++k) zc[k] = 0u;
        if (row >= 0) {
          const uint32_t* zp = reinterpret_cast<const uint32_t*>(c.z_codes + row * (R / 2));
#pragma unroll
          for (int k = 0; k < R / 8; ++k) zc[k] = __ldg(zp + k);
          zs = sigma * __ldg(c.z_scale + row);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          // nibble ^ 8 is w + 8 for a two's-complement nibble w
          const uint32_t nb = ((zc[i / 8] >> (4 * (i % 8))) & 15u) ^ 8u;
          const float w = (__uint_as_float(0x4B000000u | nb) - 8388616.0f) * zs;
          t.w[lane][i] = make_float2(w, w);
        }
      }
      __syncwarp();
#pragma unroll 2
      for (int tok = 0; tok < nt; ++tok) {
        float x[N];
        if constexpr (KCH) {
          const long long rt = __shfl_sync(kFull, row, tok);
#pragma unroll
          for (int k = 0; k < N; ++k) x[k] = 0.0f;
          if (rt >= 0) {
            const uint32_t by = reinterpret_cast<const uint8_t*>(t.codes[tok])[lane * N / 4] >> (N == 4 ? 0 : 4 * (lane & 1));
            const float* sc = c.k_scale + (rt >> 6) * D + lane * N;
            const float* mn = c.k_min + (rt >> 6) * D + lane * N;
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = fmaf(code_f(by >> (2 * k)), __ldg(sc + k), __ldg(mn + k));
          }
        } else {
          base_values<D, R>(t, tok, lane, x);
        }
        if constexpr (R > 0) {
          uint64_t a[N / 2];
#pragma unroll
          for (int k = 0; k < N / 2; ++k) a[k] = codec::pk2(x[2 * k], x[2 * k + 1]);
          const ulonglong2* wp = reinterpret_cast<const ulonglong2*>(t.w[tok]);
#pragma unroll
          for (int i = 0; i < R; i += 2) {
            const ulonglong2 w2 = wp[i / 2];
#pragma unroll
            for (int k = 0; k < N / 2; ++k) {
              a[k] = codec::fma2(u[i][k], w2.x, a[k]);
              a[k] = codec::fma2(u[i + 1][k], w2.y, a[k]);
            }
          }
#pragma unroll
          for (int k = 0; k < N / 2; ++k) {
            x[2 * k] = codec::pk_lo(a[k]);
            x[2 * k + 1] = codec::pk_hi(a[k]);
          }
        }
        store_out<N>(ko, (out0 + tok) * ko.row_stride + kv * ko.head_stride + lane * N, x);
      }
    }
    if (!vo.ptr) continue;
    if (c.vmode == HEADQ_V_2BIT) {
      __syncwarp();
      stage_codes<D, R>(t, lane, row, c.v_codes, c.v_scale, c.v_min, true);
      __syncwarp();
#pragma unroll 2
      for (int tok = 0; tok < nt; ++tok) {
        float x[N];
        base_values<D, R>(t, tok, lane, x);
        store_out<N>(vo, (out0 + tok) * vo.row_stride + kv * vo.head_stride + lane * N, x);
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
        float x[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
          x[k] = rt < 0 ? 0.0f : load_elem(c.v, rt * D + lane * N + k, vb);
        store_out<N>(vo, (out0 + tok) * vo.row_stride + kv * vo.head_stride + lane * N, x);
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
          k[e] = fmaf(code_f(by >> (2 * e)), c.k_scale[o], c.k_min[o]);
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
          for (int e = 0; e < 4; ++e) v[e] = fmaf(code_f(by >> (2 * e)), c.v_scale[gr], c.v_min[gr]);
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

template <int D, int R>
cudaError_t launch_fast(const CacheReadParams& p, cudaStream_t s) {
  // Tokens per warp: 2 tiles once that leaves several warps for every slot of the GPU (a
  // warp's registers of U_h are then read half as often), else 1.
  const long long warps = static_cast<long long>(p.c.B) * p.c.Hkv * ((p.span.n + kTok - 1) / kTok);
  const int sub = warps >= 8ll * 32 * sm_count() / 2 ? 2 : 1;
  const int tiles = (p.span.n + kTok * sub - 1) / (kTok * sub);
  const long long units = static_cast<long long>(p.c.B) * p.c.Hkv * tiles;
  auto k = p.c.kmode == HEADQ_K_CHANNEL ? cache_read_kernel<D, R, true> : cache_read_kernel<D, R, false>;
  const size_t smem = kWarps * sizeof(WarpTile<D, R>);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const long long grid = (units + kWarps - 1) / kWarps;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  k<<<static_cast<unsigned>(grid), kWarps * 32, smem, s>>>(p.c, p.span, p.U, p.sigma, p.k, p.v, p.err, tiles, sub);
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
