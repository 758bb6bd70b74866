// Launcher interface of the generation operators (rotary tables, append to
// a paged cache, reading it, decode attention, eviction, residual add + RMSNorm) between the C-ABI
// layer (api_generate.cu) and the kernels.  Arguments arriving here are
// already validated.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace h3 {

// Launch with programmatic stream serialization: the kernel's CTAs may be
// placed while the kernel before it in the stream drains.  Every thread of a kernel
// launched this way executes griddepcontrol.wait, before it writes anything and
// before it reads what the kernel before it may have written.  One reads global
// memory earlier: the decode attention's join takes the lengths before its wait,
// because the kernel before it only reads them and lets it start
// (griddepcontrol.launch_dependents) after its own wait, when they are final.  A kernel
// that writes lengths or that lets others start before it has waited must not stand
// there.  Some CTAs of that join leave without waiting: those that would add up tokens' weights and have none.  They
// touch nothing, and the kernel is not over before its joining CTAs, of which there is always one, have waited, so that
// a kernel behind it still waits for the decode kernel through it.  A grid of CTAs that may all leave must wait first.
// What the kernels before may have written (lengths, page tables,
// rotary tables) is read with ordinary loads, not through the read-only path,
// which is for data that stays as it is for the whole life of a kernel.
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                                    cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- residual add + RMSNorm, bf16 or scaled e4m3 output ----
struct AddNormArgs {
  const uint16_t* x;         // [T, C] bf16
  const uint16_t* residual;  // [T, C] bf16 or nullptr
  uint16_t* h;               // [T, C] bf16, with residual only
  void* y;                   // [T, C] bf16 or e4m3
  const float* w;            // [C] or nullptr
  void* y_scale;             // [T] float32 (row), [T, C/32] e8m0 (MX), nullptr (bf16)
  int T, C, format;
  float eps, inv_C;
};
constexpr int kAddNormMaxChannels = 16384;
cudaError_t launch_add_rmsnorm(const AddNormArgs& a, cudaStream_t stream);

// ---- rotary tables ----
constexpr int kMaxRotaryPairs = 128;  // head dim 256
struct RopeTableArgs {
  float* cos;            // [N, half]
  float* sin;            // [N, half]
  const int32_t* pos;    // [N] or nullptr: row n is position first + n
  int64_t first;
  int N, half;
  float amplitude;
  uint64_t turn[kMaxRotaryPairs];  // turns per position, as a 64-bit binary fraction
};
cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t stream);

// ---- Q/K RMSNorm + RoPE + append of K and V to a paged cache ----
struct AppendArgs {
  const uint16_t* q;  // token rows at q_stride elements, or nullptr
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;    // [B, S, Hq, D]
  uint16_t* k_pages;  // [num_pages, page_size, Hkv, D]
  uint16_t* v_pages;
  const int32_t* page_table;  // [B, max_pages]
  const int32_t* kv_len;      // [B] tokens in the cache before the call
  const float* wq;            // [D] or nullptr (no norm)
  const float* wk;
  const float* cos;           // [table_rows, rotary_dim / 2]
  const float* sin;
  const int32_t* pos;         // [B, S] or nullptr: the token's place in the cache
  const int32_t* new_len;     // [B] or nullptr: S new tokens each
  int32_t* len_out;           // [B] or nullptr
  int64_t q_stride, k_stride, v_stride;
  FastDiv div_s, div_page;
  uint32_t tokens;  // B * S
  // set by the launcher: warps' worth of work (some tokens, some heads of each), and the heads of one
  uint32_t items;
  FastDiv div_parts;
  int heads_per_part, heads_log2;
  int B, S, Hq, Hkv, D, page_size, max_pages, num_pages, table_rows, rotary_dim, interleaved;
  float eps;
  int* status;
  uint8_t* k_scales;  // a cache in 4 bits: codes in k_pages and v_pages, and their scales; nullptr: bf16
  uint8_t* v_scales;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);

// ---- attention of one new token over a paged cache ----
struct DecodeArgs {
  const uint16_t* q;  // [B, Hq, D]
  uint16_t* o;        // [B, Hq, D]
  const uint16_t* k_pages;
  const uint16_t* v_pages;
  const int32_t* page_table;
  const int32_t* kv_len;
  int B, Hq, Hkv, D, page_size, max_pages, num_pages;
  FastDiv div_page;
  float scale_log2;  // scale * log2(e)
  float* ws;         // partials, or nullptr: each sequence is walked by one CTA
  int* status;
  // a cache in 4 bits: codes in k_pages and v_pages, and their scales
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  // for the tokens' weights, [B, capacity]: scale * log2(e) * score of each query head and token, score_stride tokens a
  // head, and for each query head of a sequence that one range held what exponents were taken against and 1 / their sum;
  // nullptr: not asked for
  float* weights;
  float* scores;
  float2* stats;
  int64_t score_stride;
};
// Workspace bytes of a call on the current device (0: the call does not split).
cudaError_t decode_workspace(const DecodeArgs& a, size_t* bytes);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);
cudaError_t decode_q4_workspace(const DecodeArgs& a, size_t* bytes);
cudaError_t launch_decode_q4(const DecodeArgs& a, cudaStream_t stream);
// Of a call that does not split: weights[b, j] += sum over the heads of 2^(score - stats.x) * stats.y
cudaError_t launch_add_weights(const DecodeArgs& a, cudaStream_t stream);

// ---- cached tokens as contiguous rows ----
struct ReadArgs {
  const void* k_pages;        // bf16, or codes where k_scales is there
  const void* v_pages;
  const uint8_t* k_scales;    // nullptr: a cache in bf16
  const uint8_t* v_scales;
  const int32_t* page_table;
  const int32_t* kv_len;
  const int32_t* first;       // [B] or nullptr: from token 0 on
  uint16_t* k;                // [B, S, Hkv, D] or nullptr
  uint16_t* v;
  FastDiv div_page, div_s;
  int B, S, Hkv, D, page_size, max_pages, num_pages;
  int* status;
};
cudaError_t launch_read(const ReadArgs& a, cudaStream_t stream);

// ---- eviction from a paged cache ----
struct EvictArgs {
  uint8_t* row[4];       // K, V, and their scales (nullptr: a cache in bf16)
  int row_bytes[2];      // of a token in K and V, and in the scales
  const int32_t* page_table;
  const int32_t* kv_len;
  float* weights;        // [B, capacity]
  int32_t* len_out;
  int* ws;               // [B, ints]: counts, rows that move, rows they move to, the latter by where chains begin
  FastDiv div_page;
  int64_t capacity, ints;
  int B, page_size, max_pages, num_pages, keep, recent, most;
  int* status;
};
// Rows of one sequence that move into gaps, at most.
inline int evict_most(int64_t capacity, int keep, int recent) {
  const int64_t n = capacity - keep < keep - recent ? capacity - keep : keep - recent;
  return n > 0 ? static_cast<int>(n) : 0;
}
// Ints of a sequence's part of the workspace.
constexpr int kEvictHeader = 4;  // rows that move into gaps, and those of them from below keep
inline int64_t evict_ints(int64_t capacity, int keep, int recent) {
  const int64_t chains = capacity - keep < recent ? capacity - keep : recent;
  return kEvictHeader + 2 * static_cast<int64_t>(evict_most(capacity, keep, recent)) + (chains > 0 ? chains : 0);
}
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream);

}  // namespace h3
