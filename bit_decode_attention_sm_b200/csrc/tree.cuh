// Shared by the kernels of headq_tree_attn.
#pragma once

#include "headq_internal.cuh"

namespace headq {

// How a call runs: single tokens on the decode kernels (one), on the tensor cores
// (tree_mma.cu) with one or (pair) two 128-row blocks per CTA, or in fp32 (tree_attn.cu);
// grid_splits T-splits of `chunk` tokens per (sequence, KV head), which leave `parts` partial
// results to merge (1: none).
struct TreePlan {
  bool one, mma, pair;
  int blocks, grid_splits, parts, chunk;
};
TreePlan tree_plan(const headq_cache& c, int Hq, int n, int T, bool q_bf16);
// most partial results (query rows x parts) of any call with up to n new tokens per sequence
// and up to T cached ones, on the tensor cores and in fp32
size_t tree_max_part_rows(const headq_cache& c, int Hq, int n, int T, bool mma);

// Single tokens: the decode kernels' contiguous queries, lengths, outputs and log-sum-exps in
// the workspace.
struct TreeOne {
  void* q;
  int32_t* lens;
  float *out, *lse;
  unsigned* counters;
  float* part;
};
cudaError_t launch_tree_one(const TreeParams& p, const TreeOne& w, cudaStream_t s);

// Operands of the tensor-core kernel in the workspace: shared-memory images of the query
// rows [unit][block], each row's logit factor [unit][block * 128], mask bits [B][n][wpr]
// (null without a mask).
struct TreeMma {
  uint8_t* qimg;
  float* qf;
  uint32_t* words;
  int wpr, blocks;
};
bool tree_mma_supported(const headq_cache& c);
size_t tree_mma_image_bytes(const headq_cache& c);
cudaError_t launch_tree_mma(const TreeParams& p, const TreeMma& t, int grid_splits, bool pair, cudaStream_t s);
cudaError_t launch_tree(const TreeParams& p, const TreeMma& t, const TreePlan& plan, cudaStream_t s);

// Programmatic dependent launch: the kernel may start while the one before it in the stream is
// ending (from that one's launch_dependents on); whatever reads its results, and every CTA
// before it ends, first waits for it to be complete.
__device__ __forceinline__ void wait_for_prior_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;"); }

template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         const Args&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// whether new token i of sequence b sees its new token j (both below span.n)
__device__ __forceinline__ bool tree_sees(const TreeParams& p, int b, int i, int j) {
  return p.mask ? p.mask[b * p.mask_stride + static_cast<long long>(i) * p.span.n + j] != 0 : j <= i;
}

// 4 channels of a 2-bit code: min + code * scale, the product rounded before the sum
__device__ __forceinline__ float4 decode4(uint32_t byte, float scale, float mn) {
  auto at = [&](int k) { return __fadd_rn(__fmul_rn(static_cast<float>((byte >> (2 * k)) & 3u), scale), mn); };
  return make_float4(at(0), at(1), at(2), at(3));
}

// 4 channels of an output row, rounded to its dtype
__device__ __forceinline__ void store_row4(const headq_rows& o, size_t off, float4 x) {
  if (o.dtype == HEADQ_BF16) {
    uint2 u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.x) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u.y) : "f"(x.w), "f"(x.z));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(o.ptr) + off) = u;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(o.ptr) + off) = x;
  }
}

}  // namespace headq
