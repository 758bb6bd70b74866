// Q/K RMSNorm -> bf16 boundary -> RoPE of a step's new tokens, with K and V
// appended to a paged cache and Q written beside it.
//
// The arithmetic of a normed, half-layout row is that of the fused
// norm/RoPE kernel, operation for operation (see qk_norm_rope.cu): the sum of
// squares is a lane's first 8-channel group, then its second, channels in
// order, then a butterfly over the row's D/16 lanes; r = 1/sqrt(ms + eps)
// correctly rounded; n = bf16((x * r) * w); y_a = fma(a, c, -(b s)),
// y_b = fma(b, c, a s); so a cached K row is bit-identical to what the
// contiguous call writes.  Interleaved pairs (2i, 2i + 1) take the same
// operations on other pairs; without weights n = x.
//
// Memory-bound: every row is read once and written once.  A row is one
// (token, head) vector; rows are numbered token by token with the Hq query
// heads, then the Hkv key heads, then the Hkv value heads, so that a warp's
// rows of a fused QKV projection are one contiguous run.  D/16 lanes own a
// row and hold two 16-byte groups of it.
#include <cuda_bf16.h>

#include "generate.h"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // rows per lane group

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) {
  return f.one ? n : static_cast<uint32_t>(__umul64hi(f.M, static_cast<uint64_t>(n)));
}
enum : int { kQ = 0, kK = 1, kV = 2 };

// How a row's pairs lie in its lanes' groups.
//   kHalf: rotary_dim % 16 == 0, pairs (i, i + h): lane l < h/8 holds groups
//     l and l + h/8, whole pairs.
//   kInterleaved: pairs (2i, 2i + 1): groups l and l + D/16, whole pairs.
//   kStraddling: half layout, other rotary_dim: the partner is in another
//     lane, and the row goes through shared memory.
enum : int { kHalf = 0, kInterleaved = 1, kStraddling = 2 };

template <int D, int LAYOUT>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 16, RPW = 32 / LPR, U = kUnroll;
  constexpr float kInvD = 1.0f / static_cast<float>(D);
  __shared__ __align__(16) uint16_t rowbuf[LAYOUT == kStraddling ? kThreads / LPR : 1][LAYOUT == kStraddling ? D : 1];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31, lr = lane % LPR, slot = lane / LPR;
  if (blockIdx.x == 0 && a.len_out) {
    const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
      const int64_t n = a.new_len ? min(max(a.new_len[b], 0), a.S) : a.S;
      a.len_out[b] = static_cast<int32_t>(min(static_cast<int64_t>(max(a.kv_len[b], 0)) + n, capacity));
    }
  }
  const int half = a.rotary_dim >> 1;
  const uint32_t h8 = static_cast<uint32_t>(half >> 3);
  const bool rotating = lr < h8;
  const uint32_t g0 = LAYOUT == kInterleaved || rotating ? lr : LPR + lr;
  const uint32_t g1 = LAYOUT == kInterleaved ? LPR + lr : lr + h8;
  const int heads = a.Hq + 2 * a.Hkv;

  // The rows of this lane group: where they come from and go to, and their loads.
  uint4 xa[U], xb[U];
  uint16_t* out[U];
  int kind[U], position[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t row = (blockIdx.x * (kThreads / 32) + warp) * (RPW * U) + u * RPW + slot;
    out[u] = nullptr;
    kind[u] = kV;
    position[u] = -1;
    xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
    if (row < a.rows) {
      const uint32_t token = fdiv(row, a.div_heads);
      int head = static_cast<int>(row - token * heads);
      const uint32_t b = fdiv(token, a.div_s);
      const int s = static_cast<int>(token - b * a.S);
      const bool fresh = !a.new_len || s < a.new_len[b];
      const int64_t place = static_cast<int64_t>(max(a.kv_len[b], 0)) + s;
      const uint16_t* src;
      if (head < a.Hq) {
        kind[u] = kQ;
        src = a.q + token * a.q_stride + head * D;
        out[u] = a.q_out + (static_cast<int64_t>(token) * a.Hq + head) * D;
      } else {
        head -= a.Hq;
        kind[u] = head < a.Hkv ? kK : kV;
        if (head >= a.Hkv) head -= a.Hkv;
        src = (kind[u] == kK ? a.k + token * a.k_stride : a.v + token * a.v_stride) + head * D;
        if (fresh) {
          int page = -1, in_page = 0;
          if (place < static_cast<int64_t>(a.max_pages) * a.page_size) {
            const uint32_t p = fdiv(static_cast<uint32_t>(place), a.div_page);
            in_page = static_cast<int>(place) - static_cast<int>(p) * a.page_size;
            page = a.page_table[static_cast<int64_t>(b) * a.max_pages + p];
          }
          if (page >= 0 && page < a.num_pages)
            out[u] = (kind[u] == kK ? a.k_pages : a.v_pages) +
                     ((static_cast<int64_t>(page) * a.page_size + in_page) * a.Hkv + head) * D;
          else if (lr == 0)
            atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));  // no page for this token
        }
      }
      if (!fresh) out[u] = nullptr;
      if (out[u]) {
        xa[u] = *reinterpret_cast<const uint4*>(src + g0 * 8);
        xb[u] = *reinterpret_cast<const uint4*>(src + g1 * 8);
        if (kind[u] != kV && half > 0) {
          const int64_t p = a.pos ? static_cast<int64_t>(a.pos[token]) : place;
          if (p >= 0 && p < a.table_rows)
            position[u] = static_cast<int>(p);
          else if (lr == 0)
            atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));  // no table row: zeros
        }
      }
    }
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t xw[8] = {xa[u].x, xa[u].y, xa[u].z, xa[u].w, xb[u].x, xb[u].y, xb[u].z, xb[u].w};
    uint32_t n[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) n[e] = xw[e];
    float acc = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc = __fmaf_rn(bf16lo(xw[e]), bf16lo(xw[e]), acc);
      acc = __fmaf_rn(bf16hi(xw[e]), bf16hi(xw[e]), acc);
    }
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xFFFFFFFFu, acc, off));
    const float* w = kind[u] == kQ ? a.wq : kind[u] == kK ? a.wk : nullptr;
    if (w) {
      const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(acc, kInvD), a.eps)));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 wv = *reinterpret_cast<const float4*>(w + (e < 2 ? g0 : g1) * 8 + (e & 1) * 4);
        n[2 * e] = pack_bf16(__fmul_rn(__fmul_rn(bf16lo(xw[2 * e]), r), wv.x),
                             __fmul_rn(__fmul_rn(bf16hi(xw[2 * e]), r), wv.y));
        n[2 * e + 1] = pack_bf16(__fmul_rn(__fmul_rn(bf16lo(xw[2 * e + 1]), r), wv.z),
                                 __fmul_rn(__fmul_rn(bf16hi(xw[2 * e + 1]), r), wv.w));
      }
    }
    uint32_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = n[e];
    const bool turn = out[u] && kind[u] != kV && half > 0;
    const int64_t at = static_cast<int64_t>(max(position[u], 0)) * half;
    if constexpr (LAYOUT == kStraddling) {
      uint16_t* buf = rowbuf[warp * RPW + slot];
      *reinterpret_cast<uint4*>(buf + g0 * 8) = make_uint4(n[0], n[1], n[2], n[3]);
      *reinterpret_cast<uint4*>(buf + g1 * 8) = make_uint4(n[4], n[5], n[6], n[7]);
      __syncwarp();
      if (turn) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int d = static_cast<int>((e < 8 ? g0 : g1) * 8) + (e & 7);
          if (d < 2 * half) {
            const int i = d < half ? d : d - half;
            const float na = __uint_as_float(static_cast<uint32_t>(buf[i]) << 16);
            const float nb = __uint_as_float(static_cast<uint32_t>(buf[i + half]) << 16);
            const float c = a.cos[at + i], s = a.sin[at + i];
            const float t = d < half ? __fmaf_rn(na, c, -__fmul_rn(nb, s)) : __fmaf_rn(nb, c, __fmul_rn(na, s));
            const uint32_t tb = pack_bf16(t, 0.0f) & 0xFFFFu;
            y[e >> 1] = (e & 1) ? ((y[e >> 1] & 0xFFFFu) | (tb << 16)) : ((y[e >> 1] & 0xFFFF0000u) | tb);
          }
        }
      }
      __syncwarp();  // the buffer is rewritten by the next row
    } else if constexpr (LAYOUT == kInterleaved) {
      if (turn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // pair of word e: channels 2 i and 2 i + 1
          const int i = static_cast<int>((e < 4 ? g0 : g1) * 4) + (e & 3);
          if (i < half) {
            const float c = a.cos[at + i], s = a.sin[at + i];
            const float na = bf16lo(n[e]), nb = bf16hi(n[e]);
            y[e] = pack_bf16(__fmaf_rn(na, c, -__fmul_rn(nb, s)), __fmaf_rn(nb, c, __fmul_rn(na, s)));
          }
        }
      }
    } else if (turn && rotating) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 c = *reinterpret_cast<const float4*>(a.cos + at + lr * 8 + 4 * q);
        const float4 s = *reinterpret_cast<const float4*>(a.sin + at + lr * 8 + 4 * q);
        const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = 2 * q + j;
          const float a0 = bf16lo(n[e]), a1 = bf16hi(n[e]), b0 = bf16lo(n[4 + e]), b1 = bf16hi(n[4 + e]);
          const float c0 = cv[2 * j], c1 = cv[2 * j + 1], s0 = sv[2 * j], s1 = sv[2 * j + 1];
          y[e] = pack_bf16(__fmaf_rn(a0, c0, -__fmul_rn(b0, s0)), __fmaf_rn(a1, c1, -__fmul_rn(b1, s1)));
          y[4 + e] = pack_bf16(__fmaf_rn(b0, c0, __fmul_rn(a0, s0)), __fmaf_rn(b1, c1, __fmul_rn(a1, s1)));
        }
      }
    }
    if (turn && position[u] < 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = 0u;
    }
    if (out[u]) {
      *reinterpret_cast<uint4*>(out[u] + g0 * 8) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(out[u] + g1 * 8) = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t stream) {
  constexpr uint32_t kRows = kThreads / 32 * (32 / (D / 16)) * kUnroll;
  const dim3 grid((a.rows + kRows - 1) / kRows);
  if (a.interleaved) return launch_dependent(append_kernel<D, kInterleaved>, grid, kThreads, 0, stream, a);
  if (a.rotary_dim % 16 == 0) return launch_dependent(append_kernel<D, kHalf>, grid, kThreads, 0, stream, a);
  return launch_dependent(append_kernel<D, kStraddling>, grid, kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  switch (a.D) {
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    case 256: return launch_d<256>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
