// What each token of a paged cache was attended to: the sum over the query
// heads of its softmax weights, added to the caller's sums.
//
// The decode kernel has left each head's scores (in exponents of two) and its
// join what they are taken against, m, and 1 / l:
//   weights[b, j] += sum_h 2^(score[b, h, j] - m[b, h]) / l[b, h],
// heads in order, so results do not depend on timing.  A thread takes tokens
// kThreads apart, so that a warp reads 128 bytes of each head's scores; those were
// written by the kernel before and are mostly still in L2.
#include "decode_common.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256, kTokens = 1;  // a thread's

__global__ void __launch_bounds__(kThreads) add_weights_kernel(const __grid_constant__ DecodeArgs a, float* weights) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
  for (int b = blockIdx.y; b < a.B; b += gridDim.y) {
    const int n = len_of(a, b);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kTokens) + threadIdx.x;
    if (j0 >= n) continue;
    const float* score = a.scores + static_cast<int64_t>(b) * a.Hq * a.score_stride + j0;
    const float2* stats = a.stats + static_cast<int64_t>(b) * a.Hq;
    float sum[kTokens] = {};
#pragma unroll 8
    for (int h = 0; h < a.Hq; ++h) {
      const float2 ml = stats[h];
#pragma unroll
      for (int i = 0; i < kTokens; ++i)
        if (j0 + i * kThreads < n) sum[i] = fmaf(ex2(score[h * a.score_stride + i * kThreads] - ml.x), ml.y, sum[i]);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
      if (j0 + i * kThreads < n) weights[b * capacity + j0 + i * kThreads] += sum[i];
  }
}

}  // namespace

cudaError_t launch_add_weights(const DecodeArgs& a, float* weights, cudaStream_t stream) {
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size, each = kThreads * kTokens;
  const dim3 grid(static_cast<unsigned>((capacity + each - 1) / each), static_cast<unsigned>(std::min(a.B, 65535)));
  return launch_dependent(add_weights_kernel, grid, kThreads, 0, stream, a, weights);
}

}  // namespace h3
