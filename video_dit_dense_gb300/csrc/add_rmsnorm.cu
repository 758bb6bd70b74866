// Residual add + RMSNorm of transformer hidden rows, with the normed rows in
// bf16 or in e4m3 with scales.
//
//   h = bf16(x + residual)               (h = x without a residual)
//   r = 1 / sqrt(mean_c(h_c^2) + eps)
//   y_c = (h_c * w_c) * r                in float32
//   bf16:  y rounded once
//   row:   s = max_c |y_c| / 448,               y8 = e4m3(y * (1 / s))
//   MX:    s = 2^ceil(log2(max |y| / 448)) of each 32 channels, y8 = e4m3(y / s)
// 448 is the largest e4m3 value, so no element saturates; an all-zero row or
// group has s = 1.  The norm is that of the stored bf16 stream, not of the
// unrounded sum, so that the next layer's reader of h sees the same values.
// y is rounded once, straight from float32 to 8 bits.  max |y| = max |h w| * r
// exactly, since rounding is monotonic: the row's maximum is reduced together
// with its sum of squares, in one pass over the row.
//
// Memory-bound: x and residual are read once, h and y written once; a row
// stays in registers (VPT vectors of 8 channels a thread) between the sum and
// the scaling.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "generate.h"

namespace h3 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Sum and maximum over the TPR threads of a row (TPR <= 32: within a warp).
template <int TPR>
__device__ __forceinline__ void row_reduce(float& sum, float& top) {
#pragma unroll
  for (int off = (TPR < 32 ? TPR : 32) / 2; off >= 1; off >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
  }
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    __shared__ float2 part[(TPR > kThreads ? TPR : kThreads) / 32];
    const int warp = threadIdx.x >> 5, first = warp / kWarps * kWarps;
    if ((threadIdx.x & 31) == 0) part[warp] = make_float2(sum, top);
    __syncthreads();
    sum = 0.0f;
    top = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {  // the same order in every thread of the row
      sum += part[first + i].x;
      top = fmaxf(top, part[first + i].y);
    }
  }
}

// TPR threads hold a row, VPT vectors of 8 channels each (vector k * TPR + thread).
template <int TPR, int VPT, int FORMAT>
__global__ void __launch_bounds__(TPR > kThreads ? TPR : kThreads) add_rmsnorm_kernel(const __grid_constant__ AddNormArgs a) {
  constexpr int kBlock = TPR > kThreads ? TPR : kThreads;
  constexpr int kRows = kBlock / TPR;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = threadIdx.x % TPR, V = a.C >> 3;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const bool live = row < a.T;
  const int64_t base = live ? row * a.C : 0;
  uint4 xv[VPT], rv[VPT];
  float wv[VPT][8];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = k * TPR + t;
    const bool in = live && v < V;
    const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    *reinterpret_cast<float4*>(&wv[k][0]) = in && a.w ? *reinterpret_cast<const float4*>(a.w + 8 * v) : one;
    *reinterpret_cast<float4*>(&wv[k][4]) = in && a.w ? *reinterpret_cast<const float4*>(a.w + 8 * v + 4) : one;
    xv[k] = in ? *reinterpret_cast<const uint4*>(a.x + base + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
    rv[k] = in && a.residual ? *reinterpret_cast<const uint4*>(a.residual + base + 8 * v) : make_uint4(0u, 0u, 0u, 0u);
  }
  float sum = 0.0f, top = 0.0f;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = k * TPR + t;
    if (a.residual) {
      uint32_t* x = &xv[k].x;
      const uint32_t* r = &rv[k].x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = pack2(lo16(x[e]) + lo16(r[e]), hi16(x[e]) + hi16(r[e]));
      if (live && v < V) *reinterpret_cast<uint4*>(a.h + base + 8 * v) = xv[k];
    }
    const uint32_t x[4] = {xv[k].x, xv[k].y, xv[k].z, xv[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sum = fmaf(lo16(x[e]), lo16(x[e]), sum);
      sum = fmaf(hi16(x[e]), hi16(x[e]), sum);
    }
    if constexpr (FORMAT == H3ATTN_Y_E4M3_ROW) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = fmaxf(top, fmaxf(fabsf(lo16(x[e]) * wv[k][2 * e]), fabsf(hi16(x[e]) * wv[k][2 * e + 1])));
    }
  }
  row_reduce<TPR>(sum, top);
  const float r = __frsqrt_rn(__fdiv_rn(sum, static_cast<float>(a.C)) + a.eps);
  float inv = 1.0f;
  if constexpr (FORMAT == H3ATTN_Y_E4M3_ROW) {
    // not below 2^-126, so that 1 / s is finite: such a row is zero or next to it
    const float m = top * r;
    const float s = m > 0.0f ? fmaxf(__fdiv_rn(m, 448.0f), 1.17549435e-38f) : 1.0f;
    inv = __fdiv_rn(1.0f, s);
    if (live && t == 0) static_cast<float*>(a.y_scale)[row] = s;
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = k * TPR + t;
    const bool in = live && v < V;
    const uint32_t x[4] = {xv[k].x, xv[k].y, xv[k].z, xv[k].w};
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (((e & 1) ? hi16(x[e >> 1]) : lo16(x[e >> 1])) * wv[k][e]) * r;
    if constexpr (FORMAT == H3ATTN_Y_BF16) {
      if (in)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + base + 8 * v) =
            make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
    } else {
      if constexpr (FORMAT == H3ATTN_Y_E4M3_MX32) {
        // the four lanes of a 32-channel group hold neighbouring vectors
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(y[e]));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        // least e with 448 * 2^e >= m, 448 = 1.75 * 2^8: the exponent of m less 8, and one more above 1.75
        const uint32_t bits = __float_as_uint(m);
        int e8 = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // biased by 127
        e8 = m > 0.0f ? max(e8, 1) : 127;  // 1 .. 247 (an infinite m): the inverse is a normal float too
        inv = __uint_as_float(static_cast<uint32_t>(254 - e8) << 23);
        if (in && (v & 3) == 0) static_cast<uint8_t*>(a.y_scale)[row * (a.C >> 5) + (v >> 2)] = static_cast<uint8_t>(e8);
      }
      if (in)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + base + 8 * v) =
            make_uint2(pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                       pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
    }
  }
}

template <int TPR, int VPT>
cudaError_t launch_rows(const AddNormArgs& a, cudaStream_t stream) {
  constexpr int kBlock = TPR > kThreads ? TPR : kThreads;
  const int64_t rows = kBlock / TPR;
  const dim3 grid(static_cast<unsigned>((a.T + rows - 1) / rows));
  switch (a.format) {
    case H3ATTN_Y_BF16: return launch_dependent(add_rmsnorm_kernel<TPR, VPT, H3ATTN_Y_BF16>, grid, kBlock, 0, stream, a);
    case H3ATTN_Y_E4M3_ROW:
      return launch_dependent(add_rmsnorm_kernel<TPR, VPT, H3ATTN_Y_E4M3_ROW>, grid, kBlock, 0, stream, a);
    default: return launch_dependent(add_rmsnorm_kernel<TPR, VPT, H3ATTN_Y_E4M3_MX32>, grid, kBlock, 0, stream, a);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, cudaStream_t stream) {
  const int V = a.C >> 3;
  if (V <= 32 * 2) return launch_rows<32, 2>(a, stream);
  if (V <= 64 * 2) return launch_rows<64, 2>(a, stream);
  if (V <= 128 * 2) return launch_rows<128, 2>(a, stream);
  if (V <= 256 * 2) return launch_rows<256, 2>(a, stream);
  if (V <= 256 * 4) return launch_rows<256, 4>(a, stream);
  return launch_rows<512, 4>(a, stream);
}

}  // namespace h3
