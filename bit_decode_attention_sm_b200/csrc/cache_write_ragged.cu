// headq_cache_write_ragged: the kernel of cache_write.cuh over a packed batch -- every
// sequence's new tokens at its own positions, from strided (and optionally gathered)
// rows ("HeadQ: Model-Visible Distortion and Score-Space Correction for KV-Cache
// Quantization", gist.science summary, section 3, step 2).
//
// Per token and KV head 512 bytes in and 332 out (d 128, r 16, bf16), but the exact projection
// (d x r rounded products, each followed by a rounded sum) and the codec bound it: 29.7 us for
// 8192 tokens x 8 heads, of which the projection takes 12 (its floor on the fp32 pipe is 7.2)
// and the bytes at the rate of a copy 8.4.  Four projection threads per token instead of two
// (32.6 us), 32-token tiles (30.7) and values by CTAs of their own (31.2) were slower.
#include "cache_write.cuh"

namespace headq {
namespace {

template <int D, int RB>
cudaError_t launch_rb(const CacheWriteParams& p, cudaStream_t s) {
  const size_t smem = sizeof(float) * cache_write_smem_floats<D, RB>(p.c.r, false);
  dim3 grid((p.span.n + kTT - 1) / kTT, p.c.Hkv, p.c.B);
  auto k = p.in_bf16 ? cache_write_kernel<D, RB, true, true> : cache_write_kernel<D, RB, false, true>;
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

cudaError_t launch_cache_write_ragged(const CacheWriteParams& p0, cudaStream_t s) {
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
