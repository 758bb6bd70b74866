// Tokens of a paged cache as contiguous bf16 rows, from pages in bf16 or in 4
// bits.
//
// Memory-bound: each row is read once and written once.  A warp takes a token (two
// where a token's K and V rows are short, a part of one where there are few tokens), looks up
// its page once, and its lanes walk over the pieces of 8 channels of its K and V rows, kUnroll at a time: a
// piece is 16 bytes of a bf16 row, or 4 bytes of codes and a scale that two
// neighbouring lanes share, and 16 bytes of the output.
#include "cache4.cuh"
#include "decode_common.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

template <bool Q4>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a, int lanes_log2,
                                                        const __grid_constant__ FastDiv parts) {
  const int lane = threadIdx.x & 31, per = 1 << lanes_log2;  // lanes of a token
  const uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), tokens_at = fdiv(item, parts);
  const uint32_t part = item - tokens_at * parts.d;
  const int64_t token = static_cast<int64_t>(tokens_at) * (32 >> lanes_log2) + (lane >> lanes_log2);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (token >= static_cast<int64_t>(a.B) * a.S) return;
  const uint32_t b = fdiv(static_cast<uint32_t>(token), a.div_s);
  const int s = static_cast<int>(token - static_cast<int64_t>(b) * a.S);
  const int64_t at = (a.first ? static_cast<int64_t>(a.first[b]) : 0) + s;
  const int64_t n = min(static_cast<int64_t>(max(a.kv_len[b], 0)), static_cast<int64_t>(a.max_pages) * a.page_size);
  if (at < 0 || at >= n) return;
  const uint32_t p = fdiv(static_cast<uint32_t>(at), a.div_page);
  const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + p];
  if (page < 0 || page >= a.num_pages) {
    if ((lane & (per - 1)) == 0) atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));
    return;
  }
  const int64_t row = static_cast<int64_t>(page) * a.page_size + static_cast<int>(at - static_cast<int64_t>(p) * a.page_size);
  const int pieces = a.Hkv * (a.D / 8);  // of K, and the same of V
  const int begin = a.k ? 0 : pieces, end = a.v ? 2 * pieces : pieces;
  for (int i0 = begin + (lane & (per - 1)) + static_cast<int>(part) * per * kUnroll; i0 < end;
       i0 += per * kUnroll * static_cast<int>(parts.d)) {
    uint4 x[kUnroll];
    uint32_t codes[kUnroll], scale[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * per, of = i < pieces ? i : i - pieces;
      if (i >= end) continue;
      if constexpr (Q4) {
        codes[u] = reinterpret_cast<const uint32_t*>(i < pieces ? a.k_pages : a.v_pages)[row * pieces + of];
        scale[u] = (i < pieces ? a.k_scales : a.v_scales)[(row * pieces + of) >> 1];  // pieces is even
      } else {
        x[u] = reinterpret_cast<const uint4*>(i < pieces ? a.k_pages : a.v_pages)[row * pieces + of];
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * per, of = i < pieces ? i : i - pieces;
      if (i >= end) continue;
      if constexpr (Q4) {
        const float sc = scale_value(scale[u]);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_bf16(static_cast<float>(static_cast<int>(codes[u] >> (8 * e) & 15u) - 8) * sc,
                           static_cast<float>(static_cast<int>(codes[u] >> (8 * e + 4) & 15u) - 8) * sc);
        x[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      reinterpret_cast<uint4*>(i < pieces ? a.k : a.v)[token * pieces + of] = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, cudaStream_t stream) {
  const int pieces = a.Hkv * (a.D / 8) * 2;
  const int lanes_log2 = pieces <= 16 ? 4 : 5;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.S, per_warp = 32 >> lanes_log2, warps = (tokens + per_warp - 1) / per_warp;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // a token in as many parts as it has turns, where the warps are then all resident
  const int64_t turns = (pieces + (kUnroll << lanes_log2) - 1) / (kUnroll << lanes_log2);
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(turns, sms * 32LL / warps));
  const FastDiv div = make_fastdiv(static_cast<uint32_t>(parts));
  const dim3 grid(static_cast<unsigned>((warps * parts + kThreads / 32 - 1) / (kThreads / 32)));
  return a.k_scales ? launch_dependent(read_kernel<true>, grid, kThreads, 0, stream, a, lanes_log2, div)
                    : launch_dependent(read_kernel<false>, grid, kThreads, 0, stream, a, lanes_log2, div);
}

}  // namespace h3
