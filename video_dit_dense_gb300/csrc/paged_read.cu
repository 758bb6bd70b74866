// Tokens of a paged cache as contiguous bf16 rows, from pages in bf16 or in 4
// bits.
//
// Memory-bound: each row is read once and written once.  A warp takes a token (two
// where a token's K and V rows are short, a part of one where there are few tokens), looks up
// its page, and its lanes walk over the pieces of 8 channels of its K and V rows, four at a
// time: a piece is 16 bytes of a bf16 row, or 4 bytes of codes and a scale that two
// neighbouring lanes share, and 16 bytes of the output.  Rows that end before a lane has
// four pieces are taken two or four tokens at a time, so that as much is in flight (31 x 4826 tokens
// of one head of 128 in bf16: one at a time 44 us, four 27; 23 at the copy rate).
#include "cache4.cuh"
#include "decode_common.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256, kPieces = 4;  // of a lane at a time

// TOKENS: tokens that a lane works on at a time.
template <bool Q4, int TOKENS>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadArgs a, int lanes_log2,
                                                        const __grid_constant__ FastDiv parts) {
  constexpr int U = kPieces / TOKENS;
  const int lane = threadIdx.x & 31, per = 1 << lanes_log2, of_token = lane & (per - 1);  // lanes of a token
  const uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), tokens_at = fdiv(item, parts);
  const uint32_t part = item - tokens_at * parts.d;
  const int64_t first = (static_cast<int64_t>(tokens_at) * (32 >> lanes_log2) + (lane >> lanes_log2)) * TOKENS;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int row[TOKENS];  // in the cache, or -1
#pragma unroll
  for (int t = 0; t < TOKENS; ++t) {
    row[t] = -1;
    const int64_t token = first + t;
    if (token >= static_cast<int64_t>(a.B) * a.S) continue;
    const uint32_t b = fdiv(static_cast<uint32_t>(token), a.div_s);
    const int s = static_cast<int>(token - static_cast<int64_t>(b) * a.S);
    const int64_t at = (a.first ? static_cast<int64_t>(a.first[b]) : 0) + s;
    const int64_t n = min(static_cast<int64_t>(max(a.kv_len[b], 0)), static_cast<int64_t>(a.max_pages) * a.page_size);
    if (at < 0 || at >= n) continue;
    const uint32_t p = fdiv(static_cast<uint32_t>(at), a.div_page);
    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + p];
    if (page >= 0 && page < a.num_pages)
      row[t] = page * a.page_size + static_cast<int>(at - static_cast<int64_t>(p) * a.page_size);
    else if (of_token == 0)
      atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));
  }
  const int pieces = a.Hkv * (a.D / 8);  // of K, and the same of V
  const int begin = a.k ? 0 : pieces, end = a.v ? 2 * pieces : pieces;
  for (int i0 = begin + of_token + static_cast<int>(part) * per * U; i0 < end; i0 += per * U * static_cast<int>(parts.d)) {
    uint4 x[TOKENS][U];
    uint32_t codes[TOKENS][U], scale[TOKENS][U];
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * per, of = i < pieces ? i : i - pieces;
        if (i >= end || row[t] < 0) continue;
        const int64_t at = static_cast<int64_t>(row[t]) * pieces + of;
        if constexpr (Q4) {
          codes[t][u] = reinterpret_cast<const uint32_t*>(i < pieces ? a.k_pages : a.v_pages)[at];
          scale[t][u] = (i < pieces ? a.k_scales : a.v_scales)[at >> 1];  // pieces is even
        } else {
          x[t][u] = reinterpret_cast<const uint4*>(i < pieces ? a.k_pages : a.v_pages)[at];
        }
      }
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * per, of = i < pieces ? i : i - pieces;
        if (i >= end || row[t] < 0) continue;
        if constexpr (Q4) {
          const float sc = scale_value(scale[t][u]);
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_bf16(static_cast<float>(static_cast<int>(codes[t][u] >> (8 * e) & 15u) - 8) * sc,
                             static_cast<float>(static_cast<int>(codes[t][u] >> (8 * e + 4) & 15u) - 8) * sc);
          x[t][u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        reinterpret_cast<uint4*>(i < pieces ? a.k : a.v)[(first + t) * pieces + of] = x[t][u];
      }
  }
}

template <bool Q4>
cudaError_t launch(const ReadArgs& a, cudaStream_t stream) {
  const int pieces = a.Hkv * (a.D / 8) * 2;
  const int lanes_log2 = pieces <= 16 ? 4 : 5, turns = (pieces + (1 << lanes_log2) - 1) >> lanes_log2;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.S, resident = sms * 32LL;  // warps
  auto run = [&](auto* kernel, int at_once) {
    const int64_t per_warp = (32 >> lanes_log2) * at_once, warps = (tokens + per_warp - 1) / per_warp;
    // a token in as many parts as it has turns, where the warps are then all resident
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((turns + kPieces - 1) / kPieces, resident / warps));
    const dim3 grid(static_cast<unsigned>((warps * parts + kThreads / 32 - 1) / (kThreads / 32)));
    return launch_dependent(kernel, grid, kThreads, 0, stream, a, lanes_log2, make_fastdiv(static_cast<uint32_t>(parts)));
  };
  // several tokens at a time only where there are warps enough of them
  const bool many = tokens > resident * 4;
  if (many && turns == 1) return run(read_kernel<Q4, 4>, 4);
  if (many && turns <= 2) return run(read_kernel<Q4, 2>, 2);
  return run(read_kernel<Q4, 1>, 1);
}

}  // namespace

cudaError_t launch_read(const ReadArgs& a, cudaStream_t stream) {
  return a.k_scales ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace h3
