// Launcher interface of the generation operators (rotary tables, append to
// a paged cache, decode attention, residual add + RMSNorm) between the C-ABI
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
// there.  What the kernels before may have written (lengths, page tables,
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
};
// Workspace bytes of a call on the current device (0: the call does not split).
cudaError_t decode_workspace(const DecodeArgs& a, size_t* bytes);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);

}  // namespace h3
