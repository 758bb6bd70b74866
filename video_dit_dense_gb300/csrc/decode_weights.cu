// What each token of a paged cache was attended to: the sum over the query
// heads of its softmax weights, added to the caller's sums, for decode calls that do not split (the
// others' join does it, see add_split_weights).
//
// The decode kernel has left each head's scores (in exponents of two), what they
// are taken against, m, and 1 / l:
//   weights[b, j] += sum_h 2^(score[b, h, j] - m[b, h]) / l[b, h],
// heads in order, so results do not depend on timing.  A thread takes a token, so that
// a warp reads 128 bytes of each head's scores, eight heads at a time; those were
// written by the decode kernel and are mostly still in L2.  Bound by its launch and
// three dependent reads (length, scores beside sums, weights).
#include "decode_common.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) add_weights_kernel(const __grid_constant__ DecodeArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
  const int b = blockIdx.y, n = len_of(a, b);
  const float2* stats = a.stats + static_cast<int64_t>(b) * a.Hq;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; j < n; j += static_cast<int64_t>(gridDim.x) * kThreads) {
    const float* score = a.scores + static_cast<int64_t>(b) * a.Hq * a.score_stride + j;
    float* const to = a.weights + b * capacity + j;
    const float before = *to;
    float sum = 0.0f;
#pragma unroll 8
    for (int h = 0; h < a.Hq; ++h) {
      const float2 ml = stats[h];
      sum = fmaf(ex2(score[h * a.score_stride] - ml.x), ml.y, sum);
    }
    *to = before + sum;
  }
}

}  // namespace

cudaError_t launch_add_weights(const DecodeArgs& a, cudaStream_t stream) {
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
  // Not for all the room of the tables: four CTAs a sequence, or as many as fill the GPU (700 sequences of 300 tokens, 8 heads
  // to one of 64, in tables for 32768: one CTA for each 256 of those 143 us, 24 so, as in tables for 320).
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t each = std::max<int64_t>(4, 8LL * sms / a.B);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((capacity + kThreads - 1) / kThreads, each)), static_cast<unsigned>(a.B));  // B <= 65535
  return launch_dependent(add_weights_kernel, grid, kThreads, 0, stream, a);
}

}  // namespace h3
