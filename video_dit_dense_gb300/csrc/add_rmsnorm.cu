// Residual add + RMSNorm of transformer hidden rows, with the normed rows in
// bf16 or in e4m3 with scales.
//
//   h = bf16(x + residual)               (h = x without a residual)
//   r = 1 / sqrt(mean_c(h_c^2) + eps)
//   y_c = (h_c * w_c) * r                in float32
//   bf16:  y rounded once
//   row:   s = max_c |y_c| / 448,               y8 = e4m3((h w) * (448 / max_c |h_c w_c|)), which is y / s
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
// the scaling.  One row a CTA of as many warps as the row fills, or a warp a
// row; no ring and no second row in flight, the other CTAs of the SM keep the
// memory busy.  At 32760 rows with residual, e4m3 and row scales: 5120 channels
// 168 us, 4096 channels 132 us, 7.0 and 7.1 TB/s (a copy reaches 6.8).
// CTAs that stay on their SM and ask for their next row ahead took 184 us
// (registers) and 186 us and more (shared memory) at 5120.  Threads without a
// vector cost as much as they leave idle: 256 threads for the 640 vectors of
// 5120 channels took 195 us.  So does a register too many: 82 a thread instead of 80
// took 318 us instead of 261 at 8192 channels, two CTAs an SM instead of three.  Row scales
// of up to 16 warps and two vectors a thread do not fit their 48 registers: 4 bytes a thread are
// stored to local memory without a residual, 16 with one, 12 with two rows a block.
// Without a residual a row moves 3 or 4 bytes a channel instead of 6 to 8, and what is left is a
// block's life: load, reduce, store, and 4 bytes of weights a channel from L1.  Two rows a
// block share all of it.  32760 rows of 4096 channels with row scales: 68 us of 59 (a row a block
// 82), of 5120: 94 (109), of 1288: 26 (35); bf16, 4096 channels: 78 of 79 (85), of 1288: 27 (35).
// Products run on two channels at a time (packed float32 operations); the residual's addition
// does not: packed, its operands were waited for together, 20.3 us instead of 18.2
// at 4099 rows of 4096.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "generate.h"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kShortRows = 8;  // short rows that a CTA takes, a warp each
constexpr float kLeastScale = 0x1p-126f;  // of a row that is not zero
constexpr int kManyRows = 2048;  // from here on the memory is what counts, not a row's latencies

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

// Sum and maximum over the threads of a row: a warp (WARPS == 1), or the whole
// block of at most WARPS warps.  A row's time is a chain of latencies, so the
// warps' parts are read side by side and added as a tree.
template <int WARPS, int ROWS>
__device__ __forceinline__ void row_reduce(float (&sum)[ROWS], float (&top)[ROWS]) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], off);
      top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], off));
    }
  }
  if constexpr (WARPS > 1) {
    __shared__ __align__(16) float2 part[ROWS][WARPS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      if ((threadIdx.x & 31) == 0) part[j][threadIdx.x >> 5] = make_float2(sum[j], top[j]);
      if (threadIdx.x < WARPS && threadIdx.x >= (blockDim.x >> 5)) part[j][threadIdx.x] = make_float2(0.0f, 0.0f);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      float s[WARPS / 2], m[WARPS / 2];
#pragma unroll
      for (int i = 0; i < WARPS / 2; ++i) {
        const float4 two = *reinterpret_cast<const float4*>(&part[j][2 * i]);
        s[i] = two.x + two.z;
        m[i] = fmaxf(two.y, two.w);
      }
#pragma unroll
      for (int n = WARPS / 4; n >= 1; n >>= 1) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          s[i] += s[i + n];
          m[i] = fmaxf(m[i], m[i + n]);
        }
      }
      sum[j] = s[0];
      top[j] = m[0];
    }
  }
}

// Vector k * threads + thread of a row is the thread's k-th, of each of the block's ROWS rows.
template <int WARPS, int VPT, int FORMAT, bool RESIDUAL, int ROWS = 1>
__global__ void __launch_bounds__(WARPS == 1 ? kShortRows * 32 : WARPS * 32)
    __maxnreg__(ROWS == 2   ? (FORMAT == H3ATTN_Y_E4M3_ROW ? 48 : 64)
                : VPT == 2   ? 48
                : WARPS == 1 ? 80
                : !RESIDUAL && FORMAT != H3ATTN_Y_E4M3_ROW ? 48
                                                           : 56)
    add_rmsnorm_kernel(const __grid_constant__ AddNormArgs a) {
  constexpr bool SHORT = WARPS == 1;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int TPR = SHORT ? 32 : blockDim.x;
  const int t = SHORT ? threadIdx.x & 31 : threadIdx.x, V = a.C >> 3;
  const int64_t row0 = SHORT ? static_cast<int64_t>(blockIdx.x) * kShortRows + (threadIdx.x >> 5)
                             : static_cast<int64_t>(blockIdx.x) * ROWS;
  // The weights of a vector: kept from the first use to the second, or, where they would take registers that another
  // CTA needs, read again from L1.
  constexpr bool kKeepWeights = SHORT || VPT == 2;
  auto weights = [&](int v, float (&to)[8]) {
    const float4* wp = reinterpret_cast<const float4*>(a.w + 8 * v);
    const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    *reinterpret_cast<float4*>(&to[0]) = v < V && a.w ? wp[0] : one;
    *reinterpret_cast<float4*>(&to[4]) = v < V && a.w ? wp[1] : one;
  };
  auto inside = [&](int j, int v) { return v < V && (!(SHORT || ROWS > 1) || row0 + j < a.T); };
  const int64_t base = row0 * a.C;
  auto at = [&](int j, int v) { return base + j * a.C + 8 * v; };
  uint4 xv[ROWS][VPT], rv[ROWS][VPT];
  float kept[kKeepWeights ? VPT : 1][8];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = k * TPR + t;
    if constexpr (kKeepWeights) weights(v, kept[k]);
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const bool in = inside(j, v);
      xv[j][k] = in ? *reinterpret_cast<const uint4*>(a.x + at(j, v)) : make_uint4(0u, 0u, 0u, 0u);
      rv[j][k] = in && RESIDUAL ? *reinterpret_cast<const uint4*>(a.residual + at(j, v)) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  float sum[ROWS], top[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    float even = 0.0f, odd = 0.0f;
    top[j] = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = k * TPR + t;
      if constexpr (RESIDUAL) {
        uint32_t* x = &xv[j][k].x;
        const uint32_t* r = &rv[j][k].x;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = pack2(lo16(x[e]) + lo16(r[e]), hi16(x[e]) + hi16(r[e]));
        if (inside(j, v)) *reinterpret_cast<uint4*>(a.h + at(j, v)) = xv[j][k];
      }
      const uint32_t x[4] = {xv[j][k].x, xv[j][k].y, xv[j][k].z, xv[j][k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) ffma2(even, odd, lo16(x[e]), hi16(x[e]), lo16(x[e]), hi16(x[e]), even, odd);
      if constexpr (FORMAT == H3ATTN_Y_E4M3_ROW) {
        float w8[8];
        if constexpr (!kKeepWeights) weights(v, w8);
        const float(&wv)[8] = kKeepWeights ? kept[kKeepWeights ? k : 0] : w8;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p0, p1;
          fmul2(p0, p1, lo16(x[e]), hi16(x[e]), wv[2 * e], wv[2 * e + 1]);
          top[j] = fmax3(top[j], fabsf(p0), fabsf(p1));
        }
      }
    }
    sum[j] = even + odd;
  }
  row_reduce<WARPS>(sum, top);
  // What h w is multiplied by: r, and the inverse of the row's scale.
  float factor[ROWS], inverse[ROWS];
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const float r = __frsqrt_rn(fmaf(sum[j], a.inv_C, a.eps));
    factor[j] = r;
    inverse[j] = 1.0f;
    if constexpr (FORMAT == H3ATTN_Y_E4M3_ROW) {
      // y / s = (h w) (448 / max |h w|): r is a factor of both and falls out, with its roundings and those of s.  Not for a
      // row that is zero or next to it (s is held at 2^-126, so that 1 / s is finite), or not finite.
      const float m = top[j] * r;
      const bool plain = m > 448.0f * kLeastScale && m < INFINITY && top[j] > 1e-30f;
      const float s = m > 0.0f ? fmaxf(m * (1.0f / 448.0f), kLeastScale) : 1.0f;
      const float of = __frcp_rn(plain ? top[j] : s);
      factor[j] = plain ? 448.0f * of : r;
      inverse[j] = plain ? 1.0f : of;
      if (inside(j, 0) && t == 0) static_cast<float*>(a.y_scale)[row0 + j] = s;
    }
  }
  auto finish = [&](auto twice) {  // twice: by both of them
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    const float r = factor[j];
    float inv = inverse[j];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = k * TPR + t;
      const bool in = inside(j, v);
      const uint32_t x[4] = {xv[j][k].x, xv[j][k].y, xv[j][k].z, xv[j][k].w};
      float w8[8];
      if constexpr (!kKeepWeights) weights(v, w8);
      const float(&wv)[8] = kKeepWeights ? kept[kKeepWeights ? k : 0] : w8;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        fmul2(y[e], y[e + 1], lo16(x[e >> 1]), hi16(x[e >> 1]), wv[e], wv[e + 1]);
        fmul2(y[e], y[e + 1], y[e], y[e + 1], r, r);
      }
      if constexpr (FORMAT == H3ATTN_Y_BF16) {
        if (in)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + at(j, v)) =
              make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
      } else {
        if constexpr (FORMAT == H3ATTN_Y_E4M3_MX32) {
          // the four lanes of a 32-channel group hold neighbouring vectors
          float m = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; e += 2) m = fmax3(m, fabsf(y[e]), fabsf(y[e + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          // least e with 448 * 2^e >= m, 448 = 1.75 * 2^8: the exponent of m less 8, and one more above 1.75
          const uint32_t bits = __float_as_uint(m);
          int e8 = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // biased by 127
          e8 = m > 0.0f ? max(e8, 1) : 127;  // 1 .. 247 (an infinite m): the inverse is a normal float too
          inv = __uint_as_float(static_cast<uint32_t>(254 - e8) << 23);
          if (in && (v & 3) == 0)
            static_cast<uint8_t*>(a.y_scale)[(row0 + j) * (a.C >> 5) + (v >> 2)] = static_cast<uint8_t>(e8);
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2)
          if constexpr (decltype(twice)::value) fmul2(y[e], y[e + 1], y[e], y[e + 1], inv, inv);
        if (in)
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + at(j, v)) =
              make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
      }
    }
  }
  };
  // Where instructions count, one multiplication less: 32760 rows of 4096 channels 68.2 us (69.2), 1000 of 6144 5.4 (6.4).
  // With a residual the stores of h are what counts, and the other order of things costs more than it saves (32760 rows of
  // 4096 channels 142 us, 132).
  if constexpr (FORMAT == H3ATTN_Y_E4M3_ROW && !RESIDUAL) {
    bool once = true;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) once = once && inverse[j] == 1.0f;
    if (once)
      finish(std::false_type{});
    else
      finish(std::true_type{});
  } else {
    finish(std::true_type{});
  }
}

// WARPS 1: a warp a row; else a block of up to so many warps.
template <int WARPS, int VPT, int FORMAT>
cudaError_t launch_format(const AddNormArgs& a, cudaStream_t stream) {
  const unsigned threads = WARPS == 1 ? kShortRows * 32 : ((a.C >> 3) + VPT * 32 - 1) / (VPT * 32) * 32;
  const dim3 grid(WARPS == 1 ? (static_cast<unsigned>(a.T) + kShortRows - 1) / kShortRows : a.T);
  // Two rows a block (see above)
  if constexpr (VPT == 2 && (WARPS == 8 || (WARPS == 16 && FORMAT == H3ATTN_Y_E4M3_ROW))) {
    if (!a.residual && a.T >= kManyRows)
      return launch_dependent(add_rmsnorm_kernel<WARPS, VPT, FORMAT, false, 2>, dim3((static_cast<unsigned>(a.T) + 1) / 2),
                              threads, 0, stream, a);
  }
  return a.residual ? launch_dependent(add_rmsnorm_kernel<WARPS, VPT, FORMAT, true>, grid, threads, 0, stream, a)
                    : launch_dependent(add_rmsnorm_kernel<WARPS, VPT, FORMAT, false>, grid, threads, 0, stream, a);
}
template <int WARPS, int VPT>
cudaError_t launch_rows(const AddNormArgs& a, cudaStream_t stream) {
  switch (a.format) {
    case H3ATTN_Y_BF16: return launch_format<WARPS, VPT, H3ATTN_Y_BF16>(a, stream);
    case H3ATTN_Y_E4M3_ROW: return launch_format<WARPS, VPT, H3ATTN_Y_E4M3_ROW>(a, stream);
    default: return launch_format<WARPS, VPT, H3ATTN_Y_E4M3_MX32>(a, stream);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, cudaStream_t stream) {
  const int V = a.C >> 3;
  // A warp a row for short rows: at 32760 rows of 520 channels 24 us, two warps a row 33.  From 65 vectors on only when
  // there are many: one row of 1024 channels takes 1.6 us by a warp, 1.3 by a block.
  if (V <= 64) return launch_rows<1, 2>(a, stream);
  if (V <= 128 && a.T >= 512) return launch_rows<1, 4>(a, stream);
  // Two vectors a thread while the rows are short or few (one row of 5120 channels 1.7 us, with four 2.4; 1200 rows 8.5
  // and 11.1), four with weights read twice where the memory is what counts (32760 rows 168 us, with two 174; of 8192
  // channels 265 and 313).
  // Many rows without a residual: scales of 32 channels cost the most instructions, and four vectors a thread share them
  // from 257 on (32760 rows of 4096 channels 69 us; two rows of two 80).  Row scales keep to two rows of two up to 1024
  // vectors (16000 rows of 8192 channels 85 us, one of four 91), bf16 does not (93 and 77).
  const bool many = a.T >= kManyRows, alone = !a.residual && many;
  if (alone && V > 256 && V <= 512 && a.format == H3ATTN_Y_E4M3_MX32) return launch_rows<8, 4>(a, stream);
  if (V <= 512) return launch_rows<8, 2>(a, stream);
  if (V <= 1024 && (!many || (alone && a.format == H3ATTN_Y_E4M3_ROW))) return launch_rows<16, 2>(a, stream);
  if (V <= 1024) return launch_rows<8, 4>(a, stream);
  return launch_rows<16, 4>(a, stream);
}

}  // namespace h3
