// Attention of one new token per sequence over a paged cache in 4 bits.
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j,   j < kv_len[b],
// k and v standing for (code - 8) s, 16 channels a scale.  The split of the
// sequences over the SMs, the walk of a range and the join are those of the decode
// attention over a bf16 cache (paged_decode.cu), and so are the two products: the
// cache side is the 16-row operand of mma.sync m16n8k16, query heads the 8 columns.
// What differs is how the cache side gets into registers.
//
// A token and key-value head is D + D / 8 bytes instead of 4 D, so at the memory's
// rate an SM takes 41 channels a cycle: what bounds the kernel is instructions, and
// codes must become operands in few of them.
//   - 1024 + c is the binary16 with bits 0x6400 | c, so (c - 8) s is one fused
//     multiply-add, (1024 + c) s' - 1032 s', of two channels at a time.  It is exact:
//     s' = s / 128 is a binary16 of 4 bits (at least 2^-24, at most 30), 1032 s' = 129 s' 2^3
//     takes 11.  The 128 is undone in the scores' scale and in the output's.
//   - A nibble that lies 4 bits higher is 1024 + 16 c, giving 16 (c - 8) s' with 1152 s';
//     the 16 is undone in the queries (/ 16) and in the output's channels.  So of the four nibbles
//     of a 16-bit half two take a mask, two a shift by 8 and a mask.
//   - Which channel is which row or column of a product is free: the sum over channels
//     is in any order if the queries' are in the same, and the output's rows go where their
//     channels are.  So a lane takes D / 4 neighbouring channels of a K row and D / 8 of a V row, in one
//     load each, with one or few scales.
// Both products are exact in their operands but for P, which is rounded to 11 bits
// (binary16: half a step is 2^-11 of a weight, an eighth of the output's own rounding): P is taken
// 2^7 times larger than the exponents' reference gives it, so that weights down to 2^-21 of that
// keep their bits and only those below 2^-32 are lost.
// Queries are taken in binary16 after a scaling by a power of two for each row.
//
// Measured: 104448 tokens, 24 heads of 128, one sequence: 74.5 us, 4.8 TB/s (bf16:
// 182).  60.7 of them are tiles (by the slope over lengths), at 89 % of the copy rate, 627 instructions and 0.465 us of a
// scheduler for a tile of 32 tokens of a head; around them lie 4.9 us of waits for lengths, pages and rows, 2.1 of
// joining a CTA's warps, 2.7 of unequal CTAs and 3.4 of the join and the launch.  16 sequences of 4096 to 8192
// tokens, 16 and 4 heads of 128: 21 us of 8.5 (bf16: 36).
#include <type_traits>

#include "cache4.cuh"
#include "decode_common.cuh"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr float kLift = 7.0f;  // exponents of two by which P is raised: 2^(kSlack + kLift) is below binary16's largest

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(valid ? BYTES : 0), "n"(BYTES) : "memory");
}
// BYTES of shared memory at addr + off (a constant that becomes the instruction's own).
template <int BYTES>
__device__ __forceinline__ void lds(uint32_t (&w)[BYTES / 4], uint32_t addr, int off) {
  if constexpr (BYTES == 4) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr + off) : "memory");
  if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr + off) : "memory");
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr + off)
                 : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr, int off) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr + off) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr, int off) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr + off) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same with zero for c.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// Two scales, one in each half: s' = s / 128 and what it takes from 1024 + c and from 1024 + 16 c.
struct Scale2 {
  uint32_t m, c0, c1;
};
__device__ __forceinline__ Scale2 scale2(uint32_t shifted) {  // bytes moved up by 7
  return {hmul2(shifted, 0x20002000u), hmul2(shifted, 0xC808C808u), hmul2(shifted, 0xC880C880u)};  // 2^-7, -1032 2^-7, -1152 2^-7
}
// One of the two scales for both halves (an operand modifier, no instruction).
__device__ __forceinline__ uint32_t both(uint32_t x, int which) {
  uint32_t d;
  if (which == 0)
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {l, l};}" : "=r"(d) : "r"(x));
  else
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {h, h};}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ Scale2 both(const Scale2& s, int which) { return {both(s.m, which), both(s.c0, which), both(s.c1, which)}; }
// Nibbles 0 and 4 of x (counted in 4 bits), and nibbles 1 and 5 sixteen times larger.
// k1024 is 0x64006400 in a register that the compiler neither sees through nor takes for the same in all lanes: mask and
// or are one instruction then, where two constants, or a constant and a uniform register, make two (240 instead of 128 of a
// tile's 780 instructions).
__device__ __forceinline__ uint32_t low2(uint32_t x, uint32_t k1024, const Scale2& s) {
  return hfma2((x & 0x000F000Fu) | k1024, s.m, s.c0);
}
__device__ __forceinline__ uint32_t high2(uint32_t x, uint32_t k1024, const Scale2& s) {
  return hfma2((x & 0x00F000F0u) | k1024, s.m, s.c1);
}

// NT: tiles of 8 query heads (1, 2 or 4).
template <int D, int NT, int WARPS>
struct Q4Cfg {
  static constexpr int kTile = 32;  // tokens a warp takes at a time, one a lane where pages are looked up
  static constexpr int kWarps = WARPS;
  static constexpr int kProducts = D * NT <= 256 ? 2 : 1;  // two are more than registers hold with 16 heads of 256
  static constexpr int kStages = WARPS == 8 && D * NT <= 128 ? 4 : 2;
  static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16;  // bytes of K, and the same of V
  static constexpr int kStage = 2 * (kCodes + kScales);
  static constexpr int kRing = kWarps * kStages * kStage;
  // the queries of each warp's sequence, in registers' order; once its tiles are walked, in the same place the joining of
  // the warps of a unit head: accumulators, max and sum of every second warp, 8 heads at a time
  static constexpr int kQueries = NT * D * 16;  // of a warp
  static constexpr int kJoin = kWarps / 2 * 8 * D * 4;
  static constexpr int kStats = kWarps / 2 * 8 * 2 * 4;
  static constexpr int kShared = kWarps * kQueries > kJoin + kStats ? kWarps * kQueries : kJoin + kStats;
  static constexpr int kSmem = kRing + kShared + 2 * kMaxSplitBatch * 4;
  static constexpr int kHeads = NT * 8;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

// Where the 16-byte pieces of token tr's row lie in a stage: moved so that the lanes' loads of K rows (two tokens a
// quarter-warp) and of V rows (tokens 0 2 5 7 or 1 3 4 6 of eight) use all banks.
template <int D>
__device__ __forceinline__ uint32_t swizzle(int tr) {
  if constexpr (D == 64) return 0;
  if constexpr (D == 128) return (tr & 2);
  return (tr & 1) * 5 ^ (tr & 2);
}
// The token of a product's row r among 8: neighbouring rows differ in parity, and rows 0 2 4 6 in their place modulo 4.
__device__ __forceinline__ int token_of(int r) { return r ^ (r >> 2 & 1); }

// W: the scores are kept for the tokens' weights.
template <int D, int NT, int WARPS, bool W>
__global__ void __launch_bounds__(WARPS * 32, 1) decode_q4_kernel(const __grid_constant__ Kernelargs k) {
  using C = Q4Cfg<D, NT, WARPS>;
  constexpr int TILE = C::kTile, STAGES = C::kStages;
  constexpr int MT = C::kProducts;  // products of 16 tokens at a time
  constexpr int CH = D / 32;          // 16-byte pieces of a row's codes
  constexpr int KW = D / 32;          // words of a K row that a lane takes (8 channels each)
  constexpr int VB = D / 16;          // bytes of a V row that a lane takes, and of a row's scales
  constexpr int VW = VB / 4;
  const DecodeArgs& a = k.a;
  const DecodePlan& p = k.p;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + C::kRing);
  float* stats = reinterpret_cast<float*>(smem + C::kRing + C::kJoin);
  int* end = reinterpret_cast<int*>(smem + C::kRing + C::kShared);
  int* lens = end + kMaxSplitBatch;  // without a split: of the one sequence
  // lengths and page table: brought back to L2 while the kernel before this one drains
  if (threadIdx.x * 32 < static_cast<unsigned>(a.B)) prefetch_l2(a.kv_len + threadIdx.x * 32);
  {
    const int64_t line = (static_cast<int64_t>(blockIdx.x) * (C::kWarps * 32) + threadIdx.x) * 32;
    if (line < static_cast<int64_t>(a.B) * a.max_pages) prefetch_l2(a.page_table + line);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wh = warp % p.WH, wt = warp / p.WH;
  const int r = blockIdx.x / p.groups;
  const int unit = (blockIdx.x - r * p.groups) * p.WH + wh;
  const int kvh = unit / p.q_tiles, qt = unit - kvh * p.q_tiles;
  const int G = a.Hq / a.Hkv;
  const int head0 = kvh * G + qt * p.tile_heads;            // first query head of the unit
  const int heads = min(G - qt * p.tile_heads, C::kHeads);  // its query heads

  // This CTA's tiles [t0, t1) of all sequences' tiles.  Without a split the range is sequence r.
  int t0, t1, b0;
  if (p.ranges > 0) {
    const Ranges ranges = scan_tiles<C::kWarps * 32>(a, p, TILE, end, lens);
    if (r >= ranges.count) return;
    t0 = ranges.begin(r);
    t1 = ranges.begin(r + 1);
    if (t0 >= t1) return;
    b0 = sequence_at(end, a.B, t0);
  } else {
    t0 = 0;
    b0 = r;
    if (threadIdx.x == 0) lens[0] = len_of(a, r);
    __syncthreads();
    t1 = (lens[0] + TILE - 1) / TILE;
  }
  auto seq_begin = [&](int b) { return p.ranges > 0 && b > 0 ? end[b - 1] : 0; };
  auto seq_end = [&](int b) { return p.ranges > 0 ? end[b] : t1; };
  // the sequence's tiles that this range holds: [first_tile, stop_tile)
  const int start = p.ranges > 0 ? p.start : 0;
  auto first_tile = [&](int b) { return max(t0 - seq_begin(b) - start, 0); };
  auto stop_tile = [&](int b) { return min(t1, seq_end(b)) - seq_begin(b) - start; };
  auto seq_len = [&](int b) { return lens[p.ranges > 0 ? b : 0]; };

  // The tiles that this warp loads, in the order they are used, over sequence borders.
  struct Walk {
    int b, tile, stop, len;  // sequence, tile of the sequence, the range's end in it, the sequence's tokens
    const int32_t* table;    // its pages
  };
  auto enter = [&](Walk& w) {  // to the first tile at or after the present one that is there
    while (w.tile >= w.stop) {
      if (p.ranges == 0 || seq_end(w.b) >= t1) {
        w.b = -1;
        return;
      }
      ++w.b;
      w.stop = stop_tile(w.b);
      w.tile = wt;
      w.len = seq_len(w.b);
      w.table += a.max_pages;
    }
  };
  Walk ld;
  ld.b = b0;
  ld.tile = first_tile(b0) + wt;
  ld.stop = stop_tile(b0);
  ld.len = seq_len(b0);
  ld.table = a.page_table + static_cast<int64_t>(b0) * a.max_pages;
  enter(ld);

  const uint32_t ring = smem_u32(smem) + warp * (STAGES * C::kStage);

  // The lane's token of the next two tiles to be loaded: its page, asked for two turns ahead and looked at only when
  // the rows are loaded, and its row in the page.  token_row < 0: no such token.  -2: no such tile.
  int page[2], token_row[2];
  auto look_ahead = [&](int i) {
    token_row[i] = -2;
    if (ld.b < 0) return;
    const int token = ld.tile * TILE + lane;
    token_row[i] = -1;
    if (token < ld.len) {
      const uint32_t pg = fdiv(static_cast<uint32_t>(token), a.div_page);
      page[i] = ld.table[pg];
      token_row[i] = token - static_cast<int>(pg) * a.page_size;
    }
    ld.tile += p.WT;
    enter(ld);
  };
  look_ahead(0);
  look_ahead(1);
  uint32_t mask_of[STAGES] = {};  // tokens of the stages' tiles that are attended, the next to be used first
  const uint8_t* const kcodes = reinterpret_cast<const uint8_t*>(a.k_pages) + kvh * (D / 2) + (lane % CH) * 16;
  const uint8_t* const vcodes = reinterpret_cast<const uint8_t*>(a.v_pages) + kvh * (D / 2) + (lane % CH) * 16;
  const uint8_t* const kscales = a.k_scales + kvh * VB;
  const uint8_t* const vscales = a.v_scales + kvh * VB;
  const uint32_t row_codes = a.Hkv * (D / 2), row_scales = a.Hkv * VB;  // bytes from token to token
  // Fills stage `at` with the next tile; rows that are not attended are zeros.
  auto load = [&](int at, uint32_t& mask) {
    if (token_row[0] != -2) {  // the same in all lanes
      uint32_t row = 0;  // of the whole cache
      bool there = token_row[0] >= 0;
      if (there) {
        if (static_cast<uint32_t>(page[0]) < static_cast<uint32_t>(a.num_pages)) {
          row = page[0] * a.page_size + token_row[0];
        } else {
          atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));  // its keys are not attended
          there = false;
        }
      }
      mask = __ballot_sync(0xFFFFFFFFu, there);
      const uint32_t ks = ring + at * C::kStage, vs = ks + C::kCodes, kss = vs + C::kCodes + lane * VB, vss = kss + C::kScales;
      auto rows = [&](auto whole) {  // whole: all tokens are there
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int tr = (i * 32 + lane) / CH, col = lane % CH;
          const uint32_t src = __shfl_sync(0xFFFFFFFFu, row, tr);
          const bool valid = whole || (mask >> tr & 1u);
          const uint32_t dst = tr * (D / 2) + ((col ^ swizzle<D>(tr)) << 4);
          cp_async<16>(ks + dst, kcodes + static_cast<uint64_t>(src) * row_codes, valid);
          cp_async<16>(vs + dst, vcodes + static_cast<uint64_t>(src) * row_codes, valid);
        }
        cp_async<VB>(kss, kscales + static_cast<uint64_t>(row) * row_scales, whole || there);
        cp_async<VB>(vss, vscales + static_cast<uint64_t>(row) * row_scales, whole || there);
      };
      if (mask == 0xFFFFFFFFu)
        rows(std::true_type{});
      else
        rows(std::false_type{});
      page[0] = page[1];
      token_row[0] = token_row[1];
      look_ahead(1);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) load(i, mask_of[i]);

  // The queries of a sequence as the second operand of the score product, in shared memory, each row scaled so that its largest channel
  // lies in [2^9, 2^10), and for the lane's columns what makes exponents of two of their scores.
  const int g = lane >> 2, t = lane & 3;
  const uint32_t queries = smem_u32(smem) + C::kRing + warp * C::kQueries, q_to = queries + lane * 16;
  // lanes of heads that are not there read one and the same of their zeros (batch 21.3 us, 21.1 so)
  const uint32_t q_at = queries + (NT == 1 ? min(lane, heads * 4) : lane) * 16;
  auto load_q = [&](int b, float (&to_log2)[NT][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool there = n * 8 + g < heads;
      const uint4* qp = reinterpret_cast<const uint4*>(a.q + (static_cast<int64_t>(b) * a.Hq + head0 + (there ? n * 8 + g : 0)) * D +
                                                       t * (D / 4));
      uint4 x[KW];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        x[i] = there ? qp[i] : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        top = max(top, abs_max8(w));
      }
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const int up = min(263 - static_cast<int>(top >> 7), 254);  // the factor's exponent, biased by 127
      const float f = __uint_as_float(static_cast<uint32_t>(up) << 23), f16th = f * 0.0625f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {  // channels 0 and 4, 2 and 6; 1 and 5, 3 and 7
        const uint32_t w[4] = {pack_f16(__uint_as_float(x[i].x << 16) * f, __uint_as_float(x[i].z << 16) * f),
                               pack_f16(__uint_as_float(x[i].y << 16) * f, __uint_as_float(x[i].w << 16) * f),
                               pack_f16(__uint_as_float(x[i].x & 0xFFFF0000u) * f16th, __uint_as_float(x[i].z & 0xFFFF0000u) * f16th),
                               pack_f16(__uint_as_float(x[i].y & 0xFFFF0000u) * f16th, __uint_as_float(x[i].w & 0xFFFF0000u) * f16th)};
        sts16(q_to + (n * KW + i) * 512, w);
      }
      // 128 / f; normal, so that -infinity times it is not a NaN, nor 0 times it
      const float back = fminf(fmaxf(a.scale_log2 * __uint_as_float(static_cast<uint32_t>(261 - up) << 23), FLT_MIN), FLT_MAX);
#pragma unroll
      for (int c = 0; c < 2; ++c) to_log2[n][c] = __shfl_sync(0xFFFFFFFFu, back, (2 * t + c) * 4);
    }
  };

  // Where in a stage the lane's K row and its scales begin (row g of the first product; the others are a constant
  // further), and its V rows and their scales (tokens 2 t and 2 t + 1): two 16-bit offsets each, kept from being worked out anew every tile.
  uint32_t of_k, of_v[2];
  {
    const int tr = token_of(g), kt = D == 256 ? 2 * t : D == 128 ? t : t >> 1;
    of_k = tr * (D / 2) + ((kt ^ swizzle<D>(tr)) << 4) + (D == 64 ? (t & 1) * 8 : 0);
    of_k |= static_cast<uint32_t>(2 * C::kCodes + tr * VB + t * (VB / 4)) << 16;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int vr = token_of(2 * t + i), vt = D == 256 ? g : D == 128 ? g >> 1 : g >> 2;
      of_v[i] = C::kCodes + vr * (D / 2) + ((vt ^ swizzle<D>(vr)) << 4) + (D == 128 ? (g & 1) * 8 : D == 64 ? (g & 3) * 4 : 0);
      of_v[i] |= static_cast<uint32_t>(2 * C::kCodes + C::kScales + vr * VB + (D == 256 ? 2 * g : D == 128 ? g : g >> 1)) << 16;
    }
    asm volatile("" : "+r"(of_k), "+r"(of_v[0]), "+r"(of_v[1]));
  }
  uint32_t k1024;
  asm volatile("shfl.sync.idx.b32 %0, %1, %2, 31, 0xFFFFFFFF;" : "=r"(k1024) : "r"(0x64006400u), "r"(lane));
  int turn = 0;  // tiles used by this warp
  int b = b0;
  bool first_segment = true;
  while (true) {
    const int s0 = first_tile(b), s1 = stop_tile(b);
    if (s0 < s1 || p.ranges == 0) {
      // ---- one sequence's tiles [s0, s1) ----
      float to_log2[NT][2];
      load_q(b, to_log2);
      __syncwarp();
      float o[NT][D / 16][4];
      // m: what the exponents are taken against, within 8 of the running maximum; l: the lane's part of the sum
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -FLT_MAX;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) o[n][dt][0] = o[n][dt][1] = o[n][dt][2] = o[n][dt][3] = 0.0f;
      }
      for (int tile = s0 + wt; tile < s1; tile += p.WT) {
        const int st = turn % STAGES;
        cp_async_wait<STAGES - 2>();
        __syncwarp();
        const uint32_t mask = mask_of[0];
        load((turn + STAGES - 1) % STAGES, mask_of[STAGES - 1]);
#pragma unroll
        for (int i = 0; i + 1 < STAGES; ++i) mask_of[i] = mask_of[i + 1];
        ++turn;
        const uint32_t stage = ring + st * C::kStage;
#pragma unroll 1
        for (int sub = 0; sub < TILE / 16; sub += MT) {
        const uint32_t codes_at = stage + sub * (16 * (D / 2)), scales_at = stage + sub * (16 * VB);
        const uint32_t k_at = codes_at + (of_k & 0xFFFFu), ks_at = scales_at + (of_k >> 16);
        const uint32_t v_at[2] = {codes_at + (of_v[0] & 0xFFFFu), codes_at + (of_v[1] & 0xFFFFu)};
        const uint32_t vs_at[2] = {scales_at + (of_v[0] >> 16), scales_at + (of_v[1] >> 16)};
        float s[NT][MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t w[2][KW];
          Scale2 sc[2][(KW + 3) / 4];  // of two blocks each, but for D 64 with one
#pragma unroll
          for (int half = 0; half < 2; ++half) {  // rows g and g + 8 of the product, tokens 8 apart
            const int tr = mt * 16 + half * 8;
            if constexpr (D == 256) {
              uint32_t part[4];
              lds<16>(part, k_at, tr * (D / 2));
#pragma unroll
              for (int i = 0; i < 4; ++i) w[half][i] = part[i];
              lds<16>(part, k_at ^ 16u, tr * (D / 2));  // the other piece of the pair
#pragma unroll
              for (int i = 0; i < 4; ++i) w[half][KW - 4 + i] = part[i];
            } else {
              lds<D / 8>(w[half], k_at, tr * (D / 2));
            }
            if constexpr (D == 64) {
              sc[half][0] = scale2(lds8(ks_at, tr * VB) * 0x00800080u);
            } else {
#pragma unroll
              for (int i = 0; i < KW / 4; ++i)
                sc[half][i] = scale2(__byte_perm(lds16(ks_at, tr * VB + 2 * i), 0u, 0x4140) * 0x80u);
            }
          }
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            const Scale2 a0 = D == 64 ? sc[0][0] : both(sc[0][i / 4], i / 2 % 2), a1 = D == 64 ? sc[1][0] : both(sc[1][i / 4], i / 2 % 2);
            const uint32_t u0 = w[0][i] >> 8, u1 = w[1][i] >> 8;
            const uint32_t even[4] = {low2(w[0][i], k1024, a0), low2(w[1][i], k1024, a1), low2(u0, k1024, a0), low2(u1, k1024, a1)};
            const uint32_t odd[4] = {high2(w[0][i], k1024, a0), high2(w[1][i], k1024, a1), high2(u0, k1024, a0), high2(u1, k1024, a1)};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t q[4];
              lds<16>(q, q_at, (n * KW + i) * 512);
              if (i == 0)
                mma_f16_first(s[n][mt], even, q[0], q[1]);
              else
                mma_f16(s[n][mt], even, q[0], q[1]);
              mma_f16(s[n][mt], odd, q[2], q[3]);
            }
          }
        }
        // lane: tokens token_of(g) and 8 more of each 16, heads 2 t and 2 t + 1 of each 8
        if (mask != 0xFFFFFFFFu) {
          const uint32_t here = mask >> (16 * sub);
          asm volatile("" ::: "memory");  // a branch, not selects
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!((here >> (mt * 16 + token_of(g) + (e < 2 ? 0 : 8))) & 1u)) s[n][mt][e] = -INFINITY;
        }
        if constexpr (W) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int h = n * 8 + 2 * t + c;
              float* row = a.scores + (static_cast<int64_t>(b) * a.Hq + head0 + h) * a.score_stride + tile * TILE + sub * 16 + token_of(g);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                if (h < heads) {
                  row[mt * 16] = s[n][mt][c] * to_log2[n][c];
                  row[mt * 16 + 8] = s[n][mt][c + 2] * to_log2[n][c];
                }
            }
        }
        uint32_t pf[NT][MT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e & 1] = fmaxf(top[e & 1], s[n][mt][e]);
          const bool over = top[0] * to_log2[n][0] > m[n][0] + kSlack || top[1] * to_log2[n][1] > m[n][1] + kSlack;
          if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 4));
              top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 8));
              top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 16));
              const float to = fmaxf(m[n][c], top[c] * to_log2[n][c]);
              const float fix = ex2(m[n][c] - to);
              m[n][c] = to;
              l[n][c] *= fix;
#pragma unroll
              for (int dt = 0; dt < D / 16; ++dt) {
                o[n][dt][c] *= fix;
                o[n][dt][c + 2] *= fix;
              }
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[n][mt][e] = ex2(fmaf(s[n][mt][e], to_log2[n][e & 1], kLift - m[n][e & 1]));
              l[n][e & 1] += s[n][mt][e];
            }
            pf[n][mt][0] = transpose8x8(pack_f16(s[n][mt][0], s[n][mt][1]));
            pf[n][mt][1] = transpose8x8(pack_f16(s[n][mt][2], s[n][mt][3]));
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          // tokens 2 t and 2 t + 1 of the product's 8, and 8 on
          uint32_t w[4][VW];
          Scale2 sc[2][(VW + 1) / 2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int tr = mt * 16 + half * 8;
            lds<VB>(w[2 * half], v_at[0], tr * (D / 2));
            lds<VB>(w[2 * half + 1], v_at[1], tr * (D / 2));
#pragma unroll
            for (int i = 0; i < (VW + 1) / 2; ++i)
              sc[half][i] = scale2((lds8(vs_at[0], tr * VB + i) + lds8(vs_at[1], tr * VB + i) * 0x10000u) * 0x80u);
          }
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const Scale2 &a0 = sc[0][i / 2], &a1 = sc[1][i / 2];
#pragma unroll
            for (int hw = 0; hw < 2; ++hw) {  // channels 0 to 3, 4 to 7 of the word
              const uint32_t x0 = __byte_perm(w[0][i], w[1][i], hw ? 0x7632 : 0x5410);
              const uint32_t x1 = __byte_perm(w[2][i], w[3][i], hw ? 0x7632 : 0x5410);
              const uint32_t u0 = x0 >> 8, u1 = x1 >> 8;
              const uint32_t even[4] = {low2(x0, k1024, a0), low2(u0, k1024, a0), low2(x1, k1024, a1), low2(u1, k1024, a1)};
              const uint32_t odd[4] = {high2(x0, k1024, a0), high2(u0, k1024, a0), high2(x1, k1024, a1), high2(u1, k1024, a1)};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_f16(o[n][4 * i + 2 * hw], even, pf[n][mt][0], pf[n][mt][1]);
                mma_f16(o[n][4 * i + 2 * hw + 1], odd, pf[n][mt][0], pf[n][mt][1]);
              }
            }
          }
        }
        }
        __syncwarp();  // the stage is read; the next turn's load may fill it
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 4);
          l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 8);
          l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], 16);
        }
      // ---- the warps of a unit head are joined, halving their number ----
      for (int step = p.WT >> 1; step >= 1; step >>= 1) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          __syncthreads();  // the buffers are free
          if (wt >= step && wt < 2 * step) {
            const int at = (wt - step) * p.WH + wh;
            float4* dst = reinterpret_cast<float4*>(join + at * (8 * D));
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
              dst[dt * 32 + lane] = make_float4(o[n][dt][0], o[n][dt][1], o[n][dt][2], o[n][dt][3]);
            if (lane < 4) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                stats[(at * 8 + 2 * t + c) * 2] = m[n][c];
                stats[(at * 8 + 2 * t + c) * 2 + 1] = l[n][c];
              }
            }
          }
          __syncthreads();
          if (wt < step) {
            const int at = wt * p.WH + wh;
            const float4* src = reinterpret_cast<const float4*>(join + at * (8 * D));
            float mine[2], theirs[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float mo = stats[(at * 8 + 2 * t + c) * 2], lo = stats[(at * 8 + 2 * t + c) * 2 + 1];
              const float to = fmaxf(m[n][c], mo);
              mine[c] = ex2(m[n][c] - to);
              theirs[c] = ex2(mo - to);
              m[n][c] = to;
              l[n][c] = l[n][c] * mine[c] + lo * theirs[c];
            }
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
              const float4 v = src[dt * 32 + lane];
              o[n][dt][0] = o[n][dt][0] * mine[0] + v.x * theirs[0];
              o[n][dt][1] = o[n][dt][1] * mine[1] + v.y * theirs[1];
              o[n][dt][2] = o[n][dt][2] * mine[0] + v.z * theirs[0];
              o[n][dt][3] = o[n][dt][3] * mine[1] + v.w * theirs[1];
            }
          }
        }
      }
      if (wt == 0) {
        const bool whole = s0 == 0 && s1 == seq_end(b) - seq_begin(b) - start;
        // slot 0: the range's first sequence, slot 1: its last
        float* const part = a.ws + ((static_cast<int64_t>(r) * 2 + (first_segment ? 0 : 1)) * p.unit_heads + unit) *
                                       partial_floats(min(G, C::kHeads), D);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int h = n * 8 + 2 * t + c;
            if (h >= heads) continue;
            // P was raised by 2^kLift, and so are l and o: the weight of a score is 2^(score - (m - kLift)) / l
            const float inv = whole ? (l[n][c] == 0.0f ? 0.0f : 1.0f / l[n][c]) : 1.0f;  // no key: zeros
            float y[D / 8];  // the lane's channels in order
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
              const int at = (dt >> 1) * 4 + (dt & 1);
              const float undo = (dt & 1 ? 8.0f : 128.0f) * inv;
              y[at] = o[n][dt][c] * undo;
              y[at + 2] = o[n][dt][c + 2] * undo;
            }
            if (whole) {
              if (W && g == 0) a.stats[static_cast<int64_t>(b) * a.Hq + head0 + h] = make_float2(m[n][c] - kLift, inv);
              uint4* op = reinterpret_cast<uint4*>(a.o + (static_cast<int64_t>(b) * a.Hq + head0 + h) * D + g * (D / 8));
#pragma unroll
              for (int i = 0; i < D / 64; ++i)
                op[i] = make_uint4(pack_bf16(y[8 * i], y[8 * i + 1]), pack_bf16(y[8 * i + 2], y[8 * i + 3]),
                                   pack_bf16(y[8 * i + 4], y[8 * i + 5]), pack_bf16(y[8 * i + 6], y[8 * i + 7]));
            } else {
              if (g == 0) {
                part[2 * h] = m[n][c] - kLift;
                part[2 * h + 1] = l[n][c];
              }
              float4* op = reinterpret_cast<float4*>(part + partial_o(min(G, C::kHeads)) + h * D + g * (D / 8));
#pragma unroll
              for (int i = 0; i < D / 32; ++i) op[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            }
          }
      }
      first_segment = false;
      if (p.WT > 1) __syncthreads();  // the joins' buffers are read; the next sequence's queries go there
    }
    if (p.ranges == 0 || seq_end(b) >= t1) break;
    ++b;
  }
  cp_async_wait<0>();
}

// Query heads that a warp takes at a time, 8, 16 or 32: codes become operands once for all of them.  With heads of 256
// registers end at 16; 32 of 128 spill (40 bytes a thread stored and 76 loaded, with weights 48 and 68), and are faster all the
// same (16 sequences of 30000 tokens, 32 heads to one: 44.4 us, by 16 at a time 47.8).
int heads_of(const DecodeArgs& a) {
  const int G = a.Hq / a.Hkv;
  return G <= 8 ? 8 : G <= 16 || a.D == 256 ? 16 : 32;
}
// Warps of a CTA.  Heads of 128 and two column tiles, or of 256, leave registers for 8.  Otherwise 16 where each has many
// tiles (one sequence of 104448 tokens, 24 heads of 128: 75 us, with 8 warps 83), although in 128 registers they spill (20 bytes a
// thread stored and 32 loaded, with weights 32 and 56; two column tiles of heads of 64 24 and 40, 36 and 52), and 8 where they
// have few, whose registers leave room for the joining kernel beside them (16 sequences of up to 8192, 16 and 4 heads: 23 and 21).
int warps_of(const DecodeArgs& a, int sms) {
  const int heads = heads_of(a), G = a.Hq / a.Hkv;
  if (a.D * heads > 1024) return 8;
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
  const int64_t units = static_cast<int64_t>(a.Hkv) * ((G + heads - 1) / heads);
  return (capacity + 31) / 32 * a.B * units >= 160LL * sms ? 16 : 8;
}
DecodePlan plan_of(const DecodeArgs& a, int sms, bool split) {
  return make_plan(a, sms, split, warps_of(a, sms), 32, heads_of(a), 1, 2);
}

template <int D, int NT, int WARPS, bool W>
cudaError_t launch_d(const Kernelargs& k, cudaStream_t stream) {
  using C = Q4Cfg<D, NT, WARPS>;
  static std::atomic<bool> attr_set[64];  // calls of several host threads
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(decode_q4_kernel<D, NT, WARPS, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t ranges = k.p.ranges > 0 ? k.p.ranges : k.a.B;
  e = launch_dependent(decode_q4_kernel<D, NT, WARPS, W>, dim3(static_cast<unsigned>(ranges * k.p.groups)), WARPS * 32, C::kSmem,
                       stream, k);
  if (e != cudaSuccess) return e;
  if (k.p.ranges == 0) return W ? launch_add_weights(k.a, stream) : e;
  const int G = k.a.Hq / k.a.Hkv;
  const int joins = k.p.ranges * k.p.groups;
  return launch_dependent(decode_join_kernel<D, W>, dim3(joins + (W ? adding_ctas(k.a, joins) : 0)), kJoinThreads, 0, stream, k,
                          C::kTile, std::min(G, C::kHeads), joins);
}

template <int D, int NT>
cudaError_t launch_warps(const Kernelargs& k, cudaStream_t stream) {
  if constexpr (D * NT <= 128)
    if (k.p.WH * k.p.WT == 16) return k.a.scores ? launch_d<D, NT, 16, true>(k, stream) : launch_d<D, NT, 16, false>(k, stream);
  return k.a.scores ? launch_d<D, NT, 8, true>(k, stream) : launch_d<D, NT, 8, false>(k, stream);
}

template <int D>
cudaError_t launch_heads(const Kernelargs& k, cudaStream_t stream) {
  if constexpr (D < 256)
    if (k.p.tile_heads == 32) return launch_warps<D, 4>(k, stream);
  return k.p.tile_heads == 16 ? launch_warps<D, 2>(k, stream) : launch_warps<D, 1>(k, stream);
}

}  // namespace

cudaError_t decode_q4_workspace(const DecodeArgs& a, size_t* bytes) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const DecodePlan p = plan_of(a, sms, true);
  const int heads = std::min(a.Hq / a.Hkv, p.tile_heads);
  *bytes = static_cast<size_t>(p.ranges) * 2 * p.unit_heads * partial_floats(heads, a.D) * sizeof(float);
  return cudaSuccess;
}

cudaError_t launch_decode_q4(const DecodeArgs& a, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  Kernelargs k{plan_of(a, sms, a.ws != nullptr), a};
  switch (a.D) {
    case 64: return launch_heads<64>(k, stream);
    case 128: return launch_heads<128>(k, stream);
    case 256: return launch_heads<256>(k, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
