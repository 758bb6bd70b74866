// Attention of one new token per sequence over a paged cache in 4 bits.
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j,   j < kv_len[b],
// with k = (code - 8) s of 16 channels a scale.  One CTA takes a query head of a sequence, its warps every
// kWarps-th token each, the lanes the channels of a row; running maximum and sum in
// float32, the warps joined through shared memory.
#include "cache4.cuh"
#include "decode_common.cuh"

namespace h3 {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_q4_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int VEC = D / 32;
  __shared__ float part_o[kWarps][D];
  __shared__ float2 part_ml[kWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.Hq, h = blockIdx.x - b * a.Hq, kvh = h / (a.Hq / a.Hkv);
  const int n = len_of(a, b);
  float q[VEC], o[VEC] = {}, m = -FLT_MAX, l = 0.0f;
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    q[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.q)[(static_cast<int64_t>(b) * a.Hq + h) * D + lane * VEC + e]);
  auto row_values = [&](const uint16_t* pages, const uint8_t* scales, int64_t row, float (&x)[VEC]) {
    const uint8_t* c = reinterpret_cast<const uint8_t*>(pages) + row * (D / 2) + lane * (VEC / 2);
    const float s = scale_value(scales[row * (D / 16) + lane * VEC / 16]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = static_cast<float>((c[e / 2] >> (4 * (e & 1)) & 15) - 8) * s;
  };
  for (int j = warp; j < n; j += kWarps) {
    const uint32_t p = fdiv(static_cast<uint32_t>(j), a.div_page);
    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + p];
    float* score = a.scores ? a.scores + (static_cast<int64_t>(b) * a.Hq + h) * a.score_stride + j : nullptr;
    if (page < 0 || page >= a.num_pages) {
      atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));  // not attended
      if (score && lane == 0) *score = -INFINITY;
      continue;
    }
    const int64_t row = (static_cast<int64_t>(page) * a.page_size + (j - static_cast<int>(p) * a.page_size)) * a.Hkv + kvh;
    float k[VEC], v[VEC], s = 0.0f;
    row_values(a.k_pages, a.k_scales, row, k);
    row_values(a.v_pages, a.v_scales, row, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    s *= a.scale_log2;
    if (score && lane == 0) *score = s;
    const float to = fmaxf(m, s), fix = ex2(m - to), w = ex2(s - to);
    l = fmaf(l, fix, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = fmaf(o[e], fix, w * v[e]);
    m = to;
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) part_o[warp][lane * VEC + e] = o[e];
  if (lane == 0) part_ml[warp] = make_float2(m, l);
  __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < kWarps; ++w) m = fmaxf(m, part_ml[w].x);
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = 0.0f;
  for (int w = 0; w < kWarps; ++w) {
    const float weight = ex2(part_ml[w].x - m);
    l = fmaf(part_ml[w].y, weight, l);
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = fmaf(part_o[w][lane * VEC + e], weight, o[e]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no key: zeros
  if (a.stats && lane == 0) a.stats[blockIdx.x] = make_float2(m, inv);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + (static_cast<int64_t>(b) * a.Hq + h) * D + lane * VEC;
#pragma unroll
  for (int e = 0; e < VEC; ++e) out[e] = __float2bfloat16_rn(o[e] * inv);
}

}  // namespace

cudaError_t decode_q4_workspace(const DecodeArgs&, size_t* bytes) {
  *bytes = 0;
  return cudaSuccess;
}

cudaError_t launch_decode_q4(const DecodeArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.Hq);
  switch (a.D) {
    case 64: return launch_dependent(decode_q4_kernel<64>, grid, kWarps * 32, 0, stream, a);
    case 128: return launch_dependent(decode_q4_kernel<128>, grid, kWarps * 32, 0, stream, a);
    case 256: return launch_dependent(decode_q4_kernel<256>, grid, kWarps * 32, 0, stream, a);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
