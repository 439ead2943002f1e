// headq_cache_write: the kernel of cache_write.cuh over a dense block of new tokens,
// and the per-channel base code.
#include "cache_write.cuh"

namespace headq {
namespace {

// The alternative base code, per channel over a block of 64 tokens: the CTA's
// tile is one block (writes start on a block boundary).  Phase A1 stages the
// keys (in the residual tile's layout) and stores the values; A2, one thread per
// channel: minimum, maximum and scale over the block's tokens; A3, one thread
// per (token, 4 channels): codes, packed byte, residual in place.  Every step is
// the same IEEE fp32 operation as in the per-token code.
template <int D, int RB, bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 3 : 2)
cache_write_channel_kernel(const CacheWriteParams p) {
  constexpr int GS = group_size(D);
  constexpr int NG = num_groups(D);
  using L = ResTile<D>;
  static_assert(D <= kThreads, "one thread per channel");

  extern __shared__ float4 smem4[];
  const int r = p.c.r;
  float* e_s = reinterpret_cast<float*>(smem4);      // [kTT][RC chunks]: keys, then residuals
  float* u_s = e_s + L::kFloats;
  float* y_s = u_s + BasisTile<D, RB>::floats(r);
  float* mn_s = y_s + kTT * (r + 1);                 // [D]
  float* sc_s = mn_s + D;                            // [D]

  const int b = blockIdx.z, kv = blockIdx.y;
  const int tile0 = blockIdx.x * kTT;
  const int tid = threadIdx.x;
  const size_t bk = static_cast<size_t>(b) * p.c.Hkv + kv;
  const int t0 = p.t0;
  const int nt = min(kTT, p.n - tile0);
  const TileRows tr = tile_rows(p.c, b, kv, t0 + tile0, nt);
  if (r > 0) load_basis<D, RB>(p, kv, u_s);

  // A1: the block's keys, and the values (as for the per-token code)
  for (int task = tid; task < kTT * NG; task += kThreads) {
    const int tt = task / NG, g = task - tt * NG;
    if (tt >= nt) continue;
    const size_t in_off = (bk * p.n + tile0 + tt) * D + g * GS;
    RawGroup<GS, BF16> kraw, vraw;
    load_raw<GS, BF16>(p.k, in_off, kraw);
    if (p.v != nullptr) load_raw<GS, BF16>(p.v, in_off, vraw);
    float x[GS];
    unpack_raw<GS, BF16>(kraw, x);
    float4* er = reinterpret_cast<float4*>(e_s) + tt * L::RC + g * L::GC;
#pragma unroll
    for (int j = 0; j < GS / 4; ++j) er[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    if (p.v != nullptr) {
      const long long row_s = tile_row(p.c, tr, b, kv, t0 + tile0, tt);
      if (row_s >= 0) store_value_group<D, BF16>(p, in_off, vraw, static_cast<size_t>(row_s), g);
    }
  }
  __syncthreads();
  const long long brow_s = cache_row(p.c, b, kv, t0 + tile0);  // the block's first row
  // A2: per channel, over the block's tokens
  if (tid < D) {
    const int o = L::off(tid);
    float lo = e_s[o], hi = e_s[o];
    for (int tt = 1; tt < nt; ++tt) {
      lo = fminf(lo, e_s[tt * 4 * L::RC + o]);
      hi = fmaxf(hi, e_s[tt * 4 * L::RC + o]);
    }
    lo = __fadd_rn(lo, 0.0f);  // a -0 extreme is stored as +0
    hi = __fadd_rn(hi, 0.0f);
    const float scale = __fdiv_rn(__fsub_rn(hi, lo), 3.0f);
    mn_s[tid] = lo;
    sc_s[tid] = scale;
    if (brow_s >= 0) {
      const size_t brow = static_cast<size_t>(brow_s) >> 6;
      p.c.k_min[brow * D + tid] = lo;
      p.c.k_scale[brow * D + tid] = scale;
    }
  }
  __syncthreads();
  // A3: codes of 4 channels of one token -> one byte; residuals in place
  for (int task = tid; task < kTT * (D / 4); task += kThreads) {
    const int tt = task / (D / 4), c4 = (task - tt * (D / 4)) * 4;
    if (tt >= nt) continue;
    float4* ch = reinterpret_cast<float4*>(e_s + tt * 4 * L::RC + L::off(c4));
    const float4 h = *ch;
    const float xs[4] = {h.x, h.y, h.z, h.w};
    float res[4];
    uint32_t byte = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = c4 + k;
      const float x = xs[k], lo = mn_s[c], scale = sc_s[c];
      int code = 0;
      if (scale != 0.0f) {
        const float tq = codec::rint_quot(__fsub_rn(x, lo), scale, __frcp_rn(scale));
        code = tq < 0.0f ? 0 : (tq > 3.0f ? 3 : static_cast<int>(tq));
      }
      byte |= static_cast<uint32_t>(code) << (2 * k);
      res[k] = __fsub_rn(x, __fadd_rn(lo, __fmul_rn(static_cast<float>(code), scale)));
    }
    *ch = make_float4(res[0], res[1], res[2], res[3]);
    const long long row_s = tile_row(p.c, tr, b, kv, t0 + tile0, tt);
    if (row_s >= 0) p.c.k_codes[static_cast<size_t>(row_s) * (D / 4) + c4 / 4] = static_cast<uint8_t>(byte);
  }
  if (r == 0) return;
  __syncthreads();  // residuals complete
  side_code_tile<D, RB>(p, e_s, u_s, y_s, b, kv, tile0, t0, tr, kTT,
                        [&](int tt) { return tile0 + tt < p.n; });
}

template <int D, int RB>
cudaError_t launch_rb(const CacheWriteParams& p, cudaStream_t s) {
  const bool channel = p.c.kmode == HEADQ_K_CHANNEL;
  if (channel && D > kThreads) return cudaErrorInvalidValue;
  const size_t smem = sizeof(float) * cache_write_smem_floats<D, RB>(p.c.r, channel);
  dim3 grid((p.n + kTT - 1) / kTT, p.c.Hkv, p.c.B);
  auto k = channel ? (p.in_bf16 ? cache_write_channel_kernel<D, RB, true>
                               : cache_write_channel_kernel<D, RB, false>)
                   : (p.in_bf16 ? cache_write_kernel<D, RB, true, false>
                               : cache_write_kernel<D, RB, false, false>);
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  k<<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const CacheWriteParams& p, cudaStream_t s) {
  return with_side_rows<D>(p.c.r, [&](auto rb) { return launch_rb<D, decltype(rb)::value>(p, s); });
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p0, cudaStream_t s) {
  CacheWriteParams p = p0;
  p.one = 1.0f;  // see codec::fma2
  switch (p.c.d) {
    case 8: return launch_d<8>(p, s);
    case 16: return launch_d<16>(p, s);
    case 32: return launch_d<32>(p, s);
    case 64: return launch_d<64>(p, s);
    case 128: return launch_d<128>(p, s);
    case 256: return launch_d<256>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace headq
