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
// operations on other pairs; without weights n = x.  For a cache in 4 bits the
// K and V rows are rounded to bf16 as for the other, and then to codes and scales
// (see cache4.cuh); the instructions of that bound it: the case below takes 197 us
// for 918 MB, 4.7 TB/s, with 73 % of the issue slots busy.
//
// Memory-bound: every row is read once and written once.  A row is one
// (token, head) vector; D/16 lanes own a row and hold two 16-byte groups of it.
// A lane stays with one token and walks over heads of it, query heads first,
// then key, then value heads, so that what the token alone decides (its place,
// its page, its table row) is looked up once and the coefficients stay in
// registers.  The rows that a warp takes at a time (32 / (D/16)) are heads of one
// token where there are many, so that it reads and writes one stretch, and fewer heads
// of several tokens where there are few, so that no lanes idle.  The heads are
// cut into parts for several warps by what fills the SMs in the end.
// 32760 tokens of 24 + 24 + 24 heads of 128 with norm: 182 us, 6.7 TB/s (a row
// at a time with its own lookups and table reads: 234 us).
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "cache4.cuh"
#include "generate.h"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;        // rows a lane works on at a time
constexpr int kWarpsPerSm = 32;   // resident

__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) {
  return f.one ? n : static_cast<uint32_t>(__umul64hi(f.M, static_cast<uint64_t>(n)));
}
// How a row's pairs lie in its lanes' groups.
//   kHalf: rotary_dim % 16 == 0, pairs (i, i + h): lane l < h/8 holds groups
//     l and l + h/8, whole pairs.
//   kInterleaved: pairs (2i, 2i + 1): groups l and l + D/16, whole pairs.
//   kStraddling: half layout, other rotary_dim: the partner is in another
//     lane, and the row goes through shared memory, 16 bits at a time for the
//     pairs, with three warp barriers a row.  16384 tokens of 24 heads of 128,
//     66 rotated: 46 us (96 rotated: 37; 30 at the copy rate).  The 64 registers
//     that four CTAs an SM leave are not enough here: 20 bytes a thread are
//     stored to local memory and 24 loaded.
enum : int { kHalf = 0, kInterleaved = 1, kStraddling = 2 };

// Q4: a cache in 4 bits.  Its straddling layout runs better in 80 registers, three CTAs an SM (5 prompts of up to 3950 tokens, 20
// and 4 heads of 128, 66 rotated: 49.4 us in 64, 47.3 in 80), the others in 64, although the half layout stores 28 bytes a
// thread to local memory and loads 64 then (clip 279 and 280, 13 prompts of 1167, 16 and 2 heads: 37.5 and 41.1).
template <int D, int LAYOUT, bool Q4>
__global__ void __launch_bounds__(kThreads, Q4 && LAYOUT == kStraddling ? 3 : 4) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 16, RPW = 32 / LPR, U = kUnroll;
  constexpr float kInvD = 1.0f / static_cast<float>(D);
  static_assert(LPR >= U, "a lane for each row that shares the square root and the quotient");
  // kStraddling: a row for each row's lanes, 16 bytes apart so that the warp's rows lie in other banks
  __shared__ __align__(16) uint16_t rowbuf[LAYOUT == kStraddling ? kThreads / LPR : 1][LAYOUT == kStraddling ? D + 8 : 8];
  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31, lr = lane % LPR, slot = lane / LPR;
  // A row's lanes stay with one token, RPW tokens a warp, and walk over its heads [first, last) of Hq + 2 Hkv.
  const uint32_t item = blockIdx.x * (kThreads / 32) + warp;
  const bool used = item < a.items;
  const uint32_t tokens_at = fdiv(used ? item : 0u, a.div_parts), part = (used ? item : 0u) - tokens_at * a.div_parts.d;
  const uint32_t hw = 1u << a.heads_log2, head_slot = slot & (hw - 1), token_slot = slot >> a.heads_log2;
  const uint32_t my_token = (tokens_at * RPW >> a.heads_log2) + token_slot;
  const uint32_t token = min(my_token, a.tokens - 1);
  bool live = my_token < a.tokens;
  const int last = min(static_cast<int>(part + 1) * a.heads_per_part, a.Hq + 2 * a.Hkv);
  int first = static_cast<int>(part) * a.heads_per_part;
  const uint32_t b = fdiv(token, a.div_s);
  const int s = static_cast<int>(token - b * a.S);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && a.len_out) {
    const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
    for (int b = threadIdx.x; b < a.B; b += kThreads) {
      const int64_t n = a.new_len ? min(max(a.new_len[b], 0), a.S) : a.S;
      a.len_out[b] = static_cast<int32_t>(min(static_cast<int64_t>(max(a.kv_len[b], 0)) + n, capacity));
    }
  }
  if (!used) return;
  if (a.new_len) live = live && s < a.new_len[b];  // the others are padding
  if (!__any_sync(0xFFFFFFFFu, live)) return;
  const int half = a.rotary_dim >> 1;
  const uint32_t h8 = static_cast<uint32_t>(half >> 3);
  const bool rotating = lr < h8;
  const uint32_t g0 = LAYOUT == kInterleaved || rotating ? lr : LPR + lr;
  const uint32_t g1 = LAYOUT == kInterleaved ? LPR + lr : lr + h8;

  const uint16_t* const q_src = a.q + token * a.q_stride;
  const uint16_t* const k_src = a.k + token * a.k_stride - a.Hq * D;
  const uint16_t* const v_src = a.v + token * a.v_stride - (a.Hq + a.Hkv) * D;
  uint4 xa[U], xb[U];
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int head = first + u * hw + head_slot;
      xa[u] = xb[u] = make_uint4(0u, 0u, 0u, 0u);
      if (live && head < last) {
        const uint16_t* src = (head < a.Hq ? q_src : head < a.Hq + a.Hkv ? k_src : v_src) + head * D;
        xa[u] = *reinterpret_cast<const uint4*>(src + g0 * 8);
        xb[u] = *reinterpret_cast<const uint4*>(src + g1 * 8);
      }
    }
  };
  load();  // the first rows are on their way while the token is looked up

  const int64_t place = static_cast<int64_t>(max(a.kv_len[b], 0)) + s;
  int64_t cache_row = -1;  // the token's row in the cache
  if (live && last > a.Hq) {
    int page = -1, in_page = 0;
    if (place < static_cast<int64_t>(a.max_pages) * a.page_size) {
      const uint32_t p = fdiv(static_cast<uint32_t>(place), a.div_page);
      in_page = static_cast<int>(place) - static_cast<int>(p) * a.page_size;
      page = a.page_table[static_cast<int64_t>(b) * a.max_pages + p];
    }
    if (page >= 0 && page < a.num_pages)
      cache_row = static_cast<int64_t>(page) * a.page_size + in_page;
    else if (lr == 0)
      atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));  // not stored
  }
  int64_t at = -1;  // the token's row in the tables
  if (live && half > 0 && first < a.Hq + a.Hkv) {
    const int64_t p = a.pos ? static_cast<int64_t>(a.pos[token]) : place;
    if (p >= 0 && p < a.table_rows)
      at = p * half;
    else if (lr == 0)
      atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));  // zeros
  }
  // Coefficients of the lane's eight pairs; those beyond the rotated ones do not turn.
  float cv[8], sv[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cv[e] = 1.0f;
    sv[e] = 0.0f;
  }
  if (at >= 0) {
    if constexpr (LAYOUT == kHalf) {
      if (rotating) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          *reinterpret_cast<float4*>(&cv[4 * q]) = *reinterpret_cast<const float4*>(a.cos + at + lr * 8 + 4 * q);
          *reinterpret_cast<float4*>(&sv[4 * q]) = *reinterpret_cast<const float4*>(a.sin + at + lr * 8 + 4 * q);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = LAYOUT == kInterleaved ? static_cast<int>((e < 4 ? g0 : g1) * 4) + (e & 3)
                                             : static_cast<int>(lr) + LPR * e;
        if (i < half) {
          cv[e] = a.cos[at + i];
          sv[e] = a.sin[at + i];
        }
      }
    }
  }
  uint16_t* const q_dst = a.q_out + static_cast<int64_t>(token) * a.Hq * D;
  uint16_t* const k_dst = a.k_pages + (cache_row * a.Hkv - a.Hq) * D;
  uint16_t* const v_dst = a.v_pages + (cache_row * a.Hkv - a.Hq - a.Hkv) * D;
  // in 4 bits: the lanes of the row that hold the neighbours of this one's groups, the two that share a scale
  auto holder = [&](uint32_t group) {  // lane, and 16 where it is that lane's second group
    if (LAYOUT == kInterleaved) return group < LPR ? group : (group - LPR) | 16u;
    if (group < h8 || group >= LPR + h8) return group < h8 ? group : group - LPR;
    return (group - h8) | 16u;
  };
  const uint32_t other0 = Q4 ? holder(g0 ^ 1u) : 0u, other1 = Q4 ? holder(g1 ^ 1u) : 0u;
  const uint32_t pair_of = (other0 & 16u ? 0x32u : 0x10u) | (other1 & 16u ? 0x7600u : 0x5400u);

  while (true) {
    // acc: sum of squares, channels in order, then the butterfly over the row's lanes
    float acc[U];
    const bool math = first < a.Hq + a.Hkv;  // not value rows alone
    if (math) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t xw[8] = {xa[u].x, xa[u].y, xa[u].z, xa[u].w, xb[u].x, xb[u].y, xb[u].z, xb[u].w};
        acc[u] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[u] = __fmaf_rn(bf16lo(xw[e]), bf16lo(xw[e]), acc[u]);
          acc[u] = __fmaf_rn(bf16hi(xw[e]), bf16hi(xw[e]), acc[u]);
        }
      }
#pragma unroll
      for (int off = LPR / 2; off >= 1; off >>= 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) acc[u] = __fadd_rn(acc[u], __shfl_xor_sync(0xFFFFFFFFu, acc[u], off));
      }
      // lane u of a row takes the root and the quotient of its u-th row, for all its lanes
      float mine = acc[0];
#pragma unroll
      for (int u = 1; u < U; ++u) mine = (lr % U) == static_cast<uint32_t>(u) ? acc[u] : mine;
      mine = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(mine, kInvD), a.eps)));
#pragma unroll
      for (int u = 0; u < U; ++u) acc[u] = __shfl_sync(0xFFFFFFFFu, mine, lane - lr + u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int head = first + u * hw + head_slot;
      const bool is_q = head < a.Hq, is_v = head >= a.Hq + a.Hkv;
      uint32_t n[8] = {xa[u].x, xa[u].y, xa[u].z, xa[u].w, xb[u].x, xb[u].y, xb[u].z, xb[u].w};
      if (math) {
        const float* w = is_v ? nullptr : is_q ? a.wq : a.wk;
        if (w) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 wv = *reinterpret_cast<const float4*>(w + (e < 2 ? g0 : g1) * 8 + (e & 1) * 4);
            float t0, t1;
            fmul2(t0, t1, bf16lo(n[2 * e]), bf16hi(n[2 * e]), acc[u], acc[u]);
            fmul2(t0, t1, t0, t1, wv.x, wv.y);
            n[2 * e] = pack_bf16(t0, t1);
            fmul2(t0, t1, bf16lo(n[2 * e + 1]), bf16hi(n[2 * e + 1]), acc[u], acc[u]);
            fmul2(t0, t1, t0, t1, wv.z, wv.w);
            n[2 * e + 1] = pack_bf16(t0, t1);
          }
        }
        if constexpr (LAYOUT == kStraddling) {
          uint16_t* buf = rowbuf[warp * RPW + slot];
          *reinterpret_cast<uint4*>(buf + g0 * 8) = make_uint4(n[0], n[1], n[2], n[3]);
          *reinterpret_cast<uint4*>(buf + g1 * 8) = make_uint4(n[4], n[5], n[6], n[7]);
          __syncwarp();
          if (!is_v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // pair i = lr + LPR e
              const int i = static_cast<int>(lr) + LPR * e;
              if (i < half) {
                const float na = __uint_as_float(static_cast<uint32_t>(buf[i]) << 16);
                const float nb = __uint_as_float(static_cast<uint32_t>(buf[i + half]) << 16);
                const uint32_t y = pack_bf16(__fmaf_rn(na, cv[e], -__fmul_rn(nb, sv[e])),
                                             __fmaf_rn(nb, cv[e], __fmul_rn(na, sv[e])));
                buf[i] = static_cast<uint16_t>(y);
                buf[i + half] = static_cast<uint16_t>(y >> 16);
              }
            }
          }
          __syncwarp();
          const uint4 ya = *reinterpret_cast<const uint4*>(buf + g0 * 8), yb = *reinterpret_cast<const uint4*>(buf + g1 * 8);
          n[0] = ya.x, n[1] = ya.y, n[2] = ya.z, n[3] = ya.w;
          n[4] = yb.x, n[5] = yb.y, n[6] = yb.z, n[7] = yb.w;
          __syncwarp();  // the buffer is rewritten by the next row
        } else if constexpr (LAYOUT == kInterleaved) {
          if (!is_v) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // the pair of word e: channels 2 i and 2 i + 1
              const float na = bf16lo(n[e]), nb = bf16hi(n[e]);
              float t0, t1, y0, y1;
              fmul2(t0, t1, nb, na, -sv[e], sv[e]);
              ffma2(y0, y1, na, nb, cv[e], cv[e], t0, t1);
              const int i = static_cast<int>((e < 4 ? g0 : g1) * 4) + (e & 3);
              if (i < half) n[e] = pack_bf16(y0, y1);
            }
          }
        } else if (rotating && !is_v) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a0 = bf16lo(n[e]), a1 = bf16hi(n[e]), b0 = bf16lo(n[4 + e]), b1 = bf16hi(n[4 + e]);
            float t0, t1, y0, y1, z0, z1;
            fmul2(t0, t1, b0, b1, -sv[2 * e], -sv[2 * e + 1]);
            ffma2(y0, y1, a0, a1, cv[2 * e], cv[2 * e + 1], t0, t1);
            fmul2(t0, t1, a0, a1, sv[2 * e], sv[2 * e + 1]);
            ffma2(z0, z1, b0, b1, cv[2 * e], cv[2 * e + 1], t0, t1);
            n[e] = pack_bf16(y0, y1);
            n[4 + e] = pack_bf16(z0, z1);
          }
        }
        if (half > 0 && at < 0 && !is_v) {
#pragma unroll
          for (int e = 0; e < 8; ++e) n[e] = 0u;
        }
      }
      if constexpr (Q4) {
        if (first + (u + 1) * static_cast<int>(hw) > a.Hq) {  // not query rows alone; the same in all lanes
          // the largest values of the lane's two groups, and of the neighbours that they share scales with, as pairs
          const uint32_t mine = abs_max8_pair(n, n + 4);
          const uint32_t of0 = __shfl_sync(0xFFFFFFFFu, mine, lane - lr + (other0 & 15u));
          const uint32_t of1 = __shfl_sync(0xFFFFFFFFu, mine, lane - lr + (other1 & 15u));
          const uint32_t top = __vmaxu2(mine, __byte_perm(of0, of1, pair_of));
          uint32_t codes0, codes1, scale0, scale1;
          // One way for the whole warp.  Lanes that store nothing (no head, padding: zeros; query rows) count as well, so where a
          // token's heads are no multiple of a turn's, its last turn goes the long way: 4 prompts of 4096 tokens, 32 and 1 heads
          // of 128, 34 rows a token, 62.5 us; 34 and 1 heads, 36 rows, 63.3.
          if (!__any_sync(0xFFFFFFFFu, !plain_maxima(top))) {
            scale0 = plain_codes(n, top << 16, codes0);
            scale1 = plain_codes(n + 4, top & 0xFFFF0000u, codes1);
          } else {
            scale0 = scale_of(top & 0xFFFFu);
            scale1 = scale_of(top >> 16);
            codes0 = codes_of(n[0], n[1], n[2], n[3], scale0);
            codes1 = codes_of(n[4], n[5], n[6], n[7], scale1);
          }
          if (live && head >= a.Hq && head < last && cache_row >= 0) {
            const int64_t row = cache_row * a.Hkv + head - a.Hq - (is_v ? a.Hkv : 0);
            uint32_t* codes = reinterpret_cast<uint32_t*>(is_v ? a.v_pages : a.k_pages) + row * (D / 8);
            uint8_t* scales = (is_v ? a.v_scales : a.k_scales) + row * (D / 16);
            codes[g0] = codes0;
            codes[g1] = codes1;
            if (!(g0 & 1u)) scales[g0 >> 1] = static_cast<uint8_t>(scale0);
            if (!(g1 & 1u)) scales[g1 >> 1] = static_cast<uint8_t>(scale1);
          }
        }
      }
      if (live && head < last && (is_q || (!Q4 && cache_row >= 0))) {
        uint16_t* dst = (is_q ? q_dst : is_v ? v_dst : k_dst) + head * D;
        *reinterpret_cast<uint4*>(dst + g0 * 8) = make_uint4(n[0], n[1], n[2], n[3]);
        *reinterpret_cast<uint4*>(dst + g1 * 8) = make_uint4(n[4], n[5], n[6], n[7]);
      }
    }
    first += U * hw;
    if (first >= last) break;
    load();
  }
}

template <int D, bool Q4>
cudaError_t launch_d(AppendArgs a, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 16);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int heads = a.Hq + 2 * a.Hkv;
  // Heads of one token that a warp takes at a time: 4 from 48 heads on (72 heads: 182 us; 2: 191, 1: 201), 2 from 16 on
  // (24 heads, 8192 padded tokens: 12.4 us; 4: 14.3, 1: 13.1), 1 below (10 heads: 32.5 us; 2: 35.1, 4: 43.0).
  a.heads_log2 = std::min(heads >= 48 ? 2 : heads >= 16 ? 1 : 0, RPW == 2 ? 1 : 2);
  const int batch = kUnroll << a.heads_log2, most = (heads + batch - 1) / batch;
  const int64_t warps = (static_cast<int64_t>(a.tokens) + (RPW >> a.heads_log2) - 1) / (RPW >> a.heads_log2);
  // Into how many parts, by the turns that a warp then takes.  A warp's lookups cost half a turn, and the last wave of
  // warps fills the SMs half on average: the least of (waves + 1/2) (turns + 1/2), and of one wave where there is less
  // (11680 tokens of 72 heads of 64: 9 turns in one part or 5 in two 42 us, 2 in five 37; 9769 of 34 heads of 128: 5 turns
  // 34 us, 3 31; 22858 of 40: 10 turns 79 us, 5 76; one more part than that takes the lookups' time again: 8192 padded
  // tokens of 24 heads, 2 turns 12.6 us, 1 13.7).
  const double waves = static_cast<double>(warps) / (static_cast<double>(sms) * kWarpsPerSm);
  int best = most;
  double least = HUGE_VAL;
  for (int turns = most; turns >= 1; turns = std::min(turns - 1, 32)) {
    const int parts = (most + turns - 1) / turns;
    const double cost = std::max(waves * parts + 0.5, 1.0) * (turns + 0.5);
    if (cost < least) {
      least = cost;
      best = turns;
    }
  }
  a.heads_per_part = best * batch;
  const int used = (heads + a.heads_per_part - 1) / a.heads_per_part;
  a.div_parts = make_fastdiv(static_cast<uint32_t>(used));
  a.items = static_cast<uint32_t>(warps * used);
  // a block without warps of its own, where there is no token: len_out is written all the same
  const dim3 grid(std::max((a.items + kThreads / 32 - 1) / (kThreads / 32), 1u));
  if (a.interleaved) return launch_dependent(append_kernel<D, kInterleaved, Q4>, grid, kThreads, 0, stream, a);
  if (a.rotary_dim % 16 == 0) return launch_dependent(append_kernel<D, kHalf, Q4>, grid, kThreads, 0, stream, a);
  return launch_dependent(append_kernel<D, kStraddling, Q4>, grid, kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  switch (a.D) {
    case 64: return a.k_scales ? launch_d<64, true>(a, stream) : launch_d<64, false>(a, stream);
    case 128: return a.k_scales ? launch_d<128, true>(a, stream) : launch_d<128, false>(a, stream);
    case 256: return a.k_scales ? launch_d<256, true>(a, stream) : launch_d<256, false>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
