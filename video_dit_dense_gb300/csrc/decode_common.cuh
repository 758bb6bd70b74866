// What the decode attentions over paged caches share: how the tiles of all
// sequences are cut into one range an SM, what a range leaves of a sequence that
// others hold parts of, and the kernel that joins those.
#pragma once

#include <cuda_bf16.h>
#include <float.h>

#include <algorithm>
#include <atomic>

#include "generate.h"

namespace h3 {
namespace {

constexpr float kSlack = 8.0f;  // in exponents of two: how far a maximum may grow before the sums are rescaled
constexpr int kMaxSplitBatch = 512;  // sequences whose tile counts fit the CTA's shared memory

__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) {
  return f.one ? n : static_cast<uint32_t>(__umul64hi(f.M, static_cast<uint64_t>(n)));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// The transpose of an 8x8 block of 16-bit values held as an accumulator fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// Unit heads and the shape of the launch, the same on the host and in both kernels.
struct DecodePlan {
  int unit_heads;  // Hkv * tiles of query heads
  int q_tiles;     // tiles of at most tile_heads query heads in a group
  int tile_heads;
  int WH, WT;      // warps of a CTA: unit heads x token splits
  int share;       // neighbouring tiles of query heads whose warps load for one another (1 or 2)
  int groups;      // CTAs across the unit heads
  int ranges;      // ranges of tiles, 0: one range per sequence (no split)
  int min_tiles;   // tiles that a range has at least
  int start;       // what starting on a sequence costs a CTA, in tiles
};

// The plan first, and in both structs what only some calls read last: a kernel's arguments are fetched a line at a time when it
// starts, and what every call reads lies in as few lines as it can (64 sequences of up to 2048 tokens, 16 and 2 heads of 64 in
// bf16: 12.04 us, 12.15 with the plan behind the arguments of the tokens' weights; 43 of 520, 20 and 4 of 128: 15.24 and 15.31).
struct Kernelargs {
  DecodePlan p;
  DecodeArgs a;
};

// Tokens attended of sequence b.  From L2: the joining kernel looks before its own wait.
__device__ __forceinline__ int len_of(const DecodeArgs& a, int b) {
  return min(max(__ldcg(a.kv_len + b), 0), a.max_pages * a.page_size);
}
// T tiles cut into `count` ranges of `each` tiles, the first `longer` of them one longer.
struct Ranges {
  int count, each, longer;
  __device__ __forceinline__ int begin(int r) const { return r * each + min(r, longer); }
  __device__ __forceinline__ int of(int tile) const {
    const int in_longer = longer * (each + 1);
    return tile < in_longer ? tile / (each + 1) : longer + (tile - in_longer) / each;
  }
};
// Ranges of at least min_tiles, but no fewer than there are sequences: a CTA
// that walks several short ones joins its warps once for each.
__device__ __forceinline__ Ranges cut(const DecodePlan& p, int T, int sequences) {
  const int tiles = T - sequences * p.start;
  Ranges c;
  c.count = max(1, min(p.ranges, max((tiles + p.min_tiles - 1) / p.min_tiles, sequences)));
  c.each = T / c.count;
  c.longer = T - c.each * c.count;
  return c;
}

// end[b] = places of sequences 0 .. b on the line that ranges are cut from, and
// len[b] (unless null) their tokens, for all b < B, in shared memory.  A sequence with a key
// has p.start places without a tile, then one for each tile, so that a CTA
// that starts on a sequence inside its range gets fewer tiles.  Every thread of the block takes part; returns
// the ranges that the tiles are cut into.
template <int THREADS>
__device__ __forceinline__ Ranges scan_tiles(const DecodeArgs& a, const DecodePlan& p, int tile, int* end, int* len) {
  __shared__ int2 warp_sum[THREADS / 32];  // tiles, sequences with a tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.B <= 32) {  // every warp for itself, without a barrier: all write the same
    const int tokens = lane < a.B ? len_of(a, lane) : 0;
    int n = tokens > 0 ? (tokens + tile - 1) / tile + p.start : 0;
    const int sequences = __popc(__ballot_sync(0xFFFFFFFFu, n > 0));
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int m = __shfl_up_sync(0xFFFFFFFFu, n, off);
      if (lane >= off) n += m;
    }
    if (lane < a.B) {
      end[lane] = n;
      if (len) len[lane] = tokens;
    }
    __syncwarp();
    return cut(p, __shfl_sync(0xFFFFFFFFu, n, 31), sequences);
  }
  int carry = 0, sequences = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const int tokens = b < a.B ? len_of(a, b) : 0;
    int n = tokens > 0 ? (tokens + tile - 1) / tile + p.start : 0;
    const int there = __popc(__ballot_sync(0xFFFFFFFFu, n > 0));
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int m = __shfl_up_sync(0xFFFFFFFFu, n, off);
      if (lane >= off) n += m;
    }
    if (b0 > 0) __syncthreads();  // the sums of the last turn are read
    if (lane == 31) warp_sum[warp] = make_int2(n, there);
    __syncthreads();
    int before = carry;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const int2 of_warp = warp_sum[w];
      if (w < warp) before += of_warp.x;
      carry += of_warp.x;
      sequences += of_warp.y;
    }
    if (b < a.B) {
      end[b] = before + n;
      if (len) len[b] = tokens;
    }
  }
  __syncthreads();
  return cut(p, carry, sequences);
}
// First sequence whose tiles end after tile t.
__device__ __forceinline__ int sequence_at(const int* end, int B, int t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// A partial: max and sum of each head, padded to 16 bytes, then O of each head.
__host__ __device__ constexpr int partial_o(int heads) { return (2 * heads + 3) / 4 * 4; }
__host__ __device__ constexpr int64_t partial_floats(int heads, int D) {
  return partial_o(heads) + static_cast<int64_t>(heads) * D;
}

constexpr int kJoinThreads = 256;
constexpr int kMaxRanges = kJoinThreads;  // a thread looks at a range, 8 bits number it
constexpr int kFewParts = 4;  // partials that a warp asks for at a time: a head in no more of them takes one warp

// weights[b, j] += sum_h 2^(score[b, h, j] - m[b, h]) / l[b, h], heads in order, of split sequences beside their join: what
// the weights need of it, each head's maximum and sum, every CTA works out for itself, 32 heads at a time, eight lanes to
// a head's ranges.  A thread takes a token; CTA `me` of `all` takes every all-th chunk of kJoinThreads tokens, counted over the
// tokens that are there (over all that the tables have room for: 64 sequences of 2000 tokens, 16 and 4 heads of 128, in tables
// for 131072 118 us, 54 so).  Bound by its chain of reads: lengths; partials' maxima and sums beside the first scores; the
// other scores.  4 sequences of up to 32760 tokens, 24 and 8 heads of 128 in 4 bits, and 16 of up to 8192, 16 and 4 in bf16:
// by a kernel behind the join 43.1 and 47.1 us; beside it 42.1 and 45.0; with scores asked for before the maxima and
// sums, and those in one turn 41.0 and 44.1; these CTAs before the joining ones in the grid 39.1 and
// 43.7; counted over the tokens 38.5 and 42.7.
constexpr int kEarly = 16;       // scores asked for before the maxima and sums
constexpr int kPartsAtOnce = 8;  // partials of a lane
template <int D>
__device__ __forceinline__ void add_split_weights(const Kernelargs& k, const Ranges& ranges, const int* end, const int* len,
                                                  int part_heads, int me, int all) {
  const DecodeArgs& a = k.a;
  const DecodePlan& p = k.p;
  __shared__ float2 ml[32];
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
  // chunks of sequences 0 .. b: every warp for itself, all write the same
  __shared__ int chunks_to[kMaxSplitBatch];
  int chunks = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int lane = threadIdx.x & 31, b = b0 + lane;
    int upto = b < a.B ? (len[b] + kJoinThreads - 1) / kJoinThreads : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int before = __shfl_up_sync(0xFFFFFFFFu, upto, off);
      if (lane >= off) upto += before;
    }
    if (b < a.B) chunks_to[b] = chunks + upto;
    chunks += __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  __syncwarp();
  // Nothing to add: these leave without griddepcontrol.wait (they would hold their place for as long as the decode runs),
  // which is allowed beside the joining CTAs of the same grid only, who wait for it (see launch_dependent).
  if (me >= chunks) return;
  const int G = a.Hq / a.Hkv;
  const int64_t unit_floats = partial_floats(part_heads, D), stride = 2 * p.unit_heads * unit_floats;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int chunk = me; chunk < chunks; chunk += all) {
    const int b = sequence_at(chunks_to, a.B, chunk), n = len[b];
    const int64_t j = static_cast<int64_t>(chunk - (b > 0 ? chunks_to[b - 1] : 0)) * kJoinThreads + threadIdx.x;
    const int begin = b > 0 ? end[b - 1] : 0, r0 = ranges.of(begin + p.start), parts = ranges.of(end[b] - 1) - r0 + 1;
    const int64_t slot1 = ranges.begin(r0) >= begin ? 0 : stride / 2;
    const float* score = a.scores + static_cast<int64_t>(b) * a.Hq * a.score_stride + j;
    float* const to = a.weights + b * capacity + j;
    const float before = j < n ? *to : 0.0f;
    float sum = 0.0f;
    for (int h0 = 0; h0 < a.Hq; h0 += 32) {
      const int heads = min(a.Hq - h0, 32);
      float early[kEarly];  // scores, asked for before what the maxima and sums wait for
#pragma unroll
      for (int i = 0; i < kEarly; ++i) early[i] = j < n && i < heads ? score[(h0 + i) * a.score_stride] : 0.0f;
      const int h = h0 + (threadIdx.x >> 3);
      float m = -FLT_MAX, l = 0.0f;
      if (h < a.Hq && parts > 1) {
        const int kvh = h / G, in_group = h - kvh * G, qt = in_group / p.tile_heads, hh = in_group - qt * p.tile_heads;
        const float* part = a.ws + r0 * stride + (kvh * p.q_tiles + qt) * unit_floats + 2 * hh;
        for (int i0 = threadIdx.x & 7; i0 < parts; i0 += 8 * kPartsAtOnce) {
          float2 of[kPartsAtOnce];
#pragma unroll
          for (int u = 0; u < kPartsAtOnce; ++u) {
            const int i = i0 + 8 * u;
            of[u] = make_float2(-FLT_MAX, 0.0f);
            if (i < parts) of[u] = *reinterpret_cast<const float2*>(part + (i == 0 ? slot1 : i * stride));
          }
#pragma unroll
          for (int u = 0; u < kPartsAtOnce; ++u) {
            const float to_m = fmaxf(m, of[u].x);
            l = l * ex2(m - to_m) + of[u].y * ex2(of[u].x - to_m);
            m = to_m;
          }
        }
      }
#pragma unroll
      for (int off = 4; off >= 1; off >>= 1) {
        const float mo = __shfl_xor_sync(0xFFFFFFFFu, m, off), lo = __shfl_xor_sync(0xFFFFFFFFu, l, off), to_m = fmaxf(m, mo);
        l = l * ex2(m - to_m) + lo * ex2(mo - to_m);
        m = to_m;
      }
      if (h < a.Hq && (threadIdx.x & 7) == 0)
        ml[threadIdx.x >> 3] = parts > 1 ? make_float2(m, l == 0.0f ? 0.0f : 1.0f / l) : a.stats[static_cast<int64_t>(b) * a.Hq + h];
      __syncthreads();
      if (j < n) {
#pragma unroll
        for (int i = 0; i < kEarly; ++i)
          if (i < heads) sum = fmaf(ex2(early[i] - ml[i].x), ml[i].y, sum);
#pragma unroll 8
        for (int i = kEarly; i < heads; ++i) sum = fmaf(ex2(score[(h0 + i) * a.score_stride] - ml[i].x), ml[i].y, sum);
      }
      __syncthreads();
    }
    if (j < n) *to = before + sum;
  }
}

// Joins the partials of the sequences that several ranges hold, each in the
// order of its ranges.  Which sequences those are follows from the lengths, as
// in the decode kernel, and is worked out while that one runs: it lets this
// one start after its own wait, so the lengths are final, and only the partials
// have to be waited for.  Sequences that one range held are written already;
// sequences without a key get their zeros here.  One CTA an SM, small enough to
// sit beside a decode CTA.
// W: the CTAs before the last `joins` ones add up the tokens' weights, in 64 registers, as many CTAs an SM as with 56 but
// without spills.
template <int D, bool W>
__global__ void __launch_bounds__(kJoinThreads) __maxnreg__(D == 256 ? 96 : W ? 64 : 56)
    decode_join_kernel(const __grid_constant__ Kernelargs k, int tile, int part_heads, int joins) {
  constexpr int VEC = D / 32, WARPS = kJoinThreads / 32;
  static_assert((WARPS & (WARPS - 1)) == 0, "warps are shared out to heads in powers of two");
  const DecodeArgs& a = k.a;
  const DecodePlan& p = k.p;
  __shared__ int end[kMaxSplitBatch];
  __shared__ uint32_t split[2][kMaxRanges];  // sequence << 16 | first range << 8 | last: of many ranges, of a few
  __shared__ int in_warp[2][WARPS];
  __shared__ float part_o[WARPS][D];
  __shared__ float2 part_ml[WARPS];
  __shared__ int len[W ? kMaxSplitBatch : 1];
  const Ranges ranges = scan_tiles<kJoinThreads>(a, p, tile, end, W ? len : nullptr);
  if constexpr (W) {
    if (static_cast<int>(blockIdx.x) < static_cast<int>(gridDim.x) - joins) {
      add_split_weights<D>(k, ranges, end, len, part_heads, blockIdx.x, gridDim.x - joins);
      return;
    }
  }
  // A sequence's tiles are in several ranges where one begins among them: the
  // first such range speaks for it.  The lists are in the order of the ranges,
  // so that every CTA has the same ones.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t mine = 0;
  int kind = -1;
  if (const int r = threadIdx.x; r > 0 && r < ranges.count) {
    const int b = sequence_at(end, a.B, ranges.begin(r)), begin = b > 0 ? end[b - 1] : 0;
    const int last = ranges.of(end[b] - 1);
    if (r == ranges.of(begin + p.start) + 1 && r <= last) {
      kind = last - r + 2 > kFewParts ? 0 : 1;
      mine = static_cast<uint32_t>(b) << 16 | static_cast<uint32_t>(r - 1) << 8 | static_cast<uint32_t>(last);
    }
  }
  const uint32_t same[2] = {__ballot_sync(0xFFFFFFFFu, kind == 0), __ballot_sync(0xFFFFFFFFu, kind == 1)};
  if (lane < 2) in_warp[lane][warp] = __popc(same[lane]);
  __syncthreads();
  int n_split[2] = {0, 0}, at = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (i == kind && w < warp) at += in_warp[i][w];
      n_split[i] += in_warp[i][w];
    }
  }
  if (kind >= 0) split[kind][at + __popc(same[kind] & ((1u << lane) - 1u))] = mine;
  __syncthreads();
  const int G = a.Hq / a.Hkv;
  const int64_t unit_floats = partial_floats(part_heads, D), stride = 2 * p.unit_heads * unit_floats;  // from range to range
  // A head of a split sequence: its partial of the first range (slot 1 where that range begins in another sequence), the
  // lane's part of it, and the row it goes to.
  struct Head {
    const float *ml, *o;
    uint16_t* out;
    int64_t slot1;  // from the others' slot to the first one's
    int n;          // ranges
  };
  auto locate = [&](int list, int i) {
    const int in_list = i / a.Hq, h = i - in_list * a.Hq;
    const uint32_t q = split[list][in_list];
    const int b = q >> 16, r0 = (q >> 8) & 255;
    const int kvh = h / G, in_group = h - kvh * G, qt = in_group / p.tile_heads, hh = in_group - qt * p.tile_heads;
    const float* part = a.ws + r0 * stride + (kvh * p.q_tiles + qt) * unit_floats;
    Head x;
    x.ml = part + 2 * hh;
    x.o = part + partial_o(part_heads) + hh * D + lane * VEC;
    x.out = a.o + (static_cast<int64_t>(b) * a.Hq + h) * D + lane * VEC;
    x.slot1 = ranges.begin(r0) >= (b > 0 ? end[b - 1] : 0) ? 0 : stride / 2;
    x.n = static_cast<int>(q & 255) - r0 + 1;
    return x;
  };
  float m, l, o[VEC];
  // Adds up the partials first, first + step, ... of a head: four are asked for at a time.
  auto gather = [&](const Head& x, int first, int step) {
    m = -FLT_MAX;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = 0.0f;
    for (int r = first; r < x.n; r += 4 * step) {
      float mr[4], lr[4], v[4][VEC];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ri = r + i * step;
        mr[i] = -FLT_MAX;
        lr[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = 0.0f;
        if (ri < x.n) {
          const int64_t off = ri == 0 ? x.slot1 : ri * stride;
          const float2 ml = *reinterpret_cast<const float2*>(x.ml + off);
          mr[i] = ml.x;
          lr[i] = ml.y;
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const float2 two = *reinterpret_cast<const float2*>(x.o + off + e);
            v[i][e] = two.x;
            v[i][e + 1] = two.y;
          }
        }
      }
      const float to = fmaxf(fmaxf(fmaxf(mr[0], mr[1]), fmaxf(mr[2], mr[3])), m);
      const float mine = ex2(m - to);
      l *= mine;
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] *= mine;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float theirs = ex2(mr[i] - to);
        l = fmaf(lr[i], theirs, l);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(v[i][e], theirs, o[e]);
      }
      m = to;
    }
  };
  auto write = [&](const Head& x) {
    uint16_t* const out = x.out;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no key was attended: zeros
#pragma unroll
    for (int e = 0; e < VEC; e += 2) reinterpret_cast<uint32_t*>(out)[e >> 1] = pack_bf16(o[e] * inv, o[e + 1] * inv);
  };
  // Heads in few ranges: a warp each.  Heads in many: as many warps on each as there are for all of them.
  const int cta = W ? blockIdx.x - (gridDim.x - joins) : blockIdx.x;
  const int few = n_split[1] * a.Hq, many = n_split[0] * a.Hq;
  int per = WARPS;
  while (per > 2 && many * per > joins * WARPS) per >>= 1;
  const int lead = warp / per * per, at_once = WARPS / per;  // first warp of this one's head, heads a CTA takes at a time
  // the first of each is looked up before the wait
  int i_few = cta * WARPS + warp, i_many = cta * at_once + warp / per;
  Head x_few{}, x_many{};
  if (i_few < few) x_few = locate(1, i_few);
  if (i_many < many) x_many = locate(0, i_many);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  while (i_few < few) {
    gather(x_few, 0, 1);
    write(x_few);
    i_few += joins * WARPS;
    if (i_few < few) x_few = locate(1, i_few);
  }
  for (int i0 = cta * at_once; i0 < many; i0 += joins * at_once) {
    const bool there = i_many < many;
    if (there) {
      gather(x_many, warp - lead, per);
#pragma unroll
      for (int e = 0; e < VEC; ++e) part_o[warp][lane * VEC + e] = o[e];
      if (lane == 0) part_ml[warp] = make_float2(m, l);
    }
    __syncthreads();
    if (there && warp == lead) {
      m = -FLT_MAX;
      for (int w = lead; w < lead + per; ++w) m = fmaxf(m, part_ml[w].x);
      l = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = 0.0f;
      for (int w = lead; w < lead + per; ++w) {
        const float weight = ex2(part_ml[w].x - m);
        l = fmaf(part_ml[w].y, weight, l);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = fmaf(part_o[w][lane * VEC + e], weight, o[e]);
      }
      write(x_many);
    }
    __syncthreads();
    i_many += joins * at_once;
    if (i_many < many) x_many = locate(0, i_many);
  }
  for (int b = cta; b < a.B; b += joins) {
    if (end[b] == (b > 0 ? end[b - 1] : 0)) {  // no key: zeros
      uint2* row = reinterpret_cast<uint2*>(a.o + static_cast<int64_t>(b) * a.Hq * D);
      for (int i = threadIdx.x; i < a.Hq * (D / 4); i += kJoinThreads) row[i] = make_uint2(0u, 0u);
    }
  }
}

// CTAs that add up weights beside the joining ones: one for each kJoinThreads tokens that the tables have room for, up to eight
// beside each of those.
inline int adding_ctas(const DecodeArgs& a, int joins) {
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
  return static_cast<int>(std::min<int64_t>((capacity + kJoinThreads - 1) / kJoinThreads * a.B, 8LL * joins));
}

inline cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// The shape of a launch whose CTAs have `warps` warps that take `tile` tokens and up to `tile_heads` query heads of a
// group at a time; the warps of `share` neighbouring
// tiles of query heads load for one another where there is an even number of those; caches of at most `few` tiles a
// warp are walked whole.
inline DecodePlan make_plan(const DecodeArgs& a, int sms, bool split, int warps, int tile, int tile_heads, int share,
                             int few) {
  DecodePlan p;
  const int G = a.Hq / a.Hkv;
  p.tile_heads = tile_heads;
  p.q_tiles = (G + tile_heads - 1) / tile_heads;
  p.unit_heads = a.Hkv * p.q_tiles;
  p.WH = 1;
  while (p.WH < warps && p.unit_heads % (2 * p.WH) == 0) p.WH *= 2;
  p.WT = warps / p.WH;
  p.groups = p.unit_heads / p.WH;
  p.share = p.q_tiles % 2 == 0 ? share : 1;
  const int loaders = p.WT * p.share;  // warps that load different tiles
  // Split into one range an SM, unless
  // - the cache has no room for sequences of more than `few` tiles a warp: one CTA walks them in less time than the
  //   second kernel takes (bf16, four: 16 query and 4 key-value heads of 128, one sequence: 6.1 us against 6.9 at 128 tokens, 9.0
  //   against 7.2 at 256; 24 heads of each: 5.6 against 6.6 at 64, 8.5 against 6.8 at 128; 8 and 1: 6.8 against 7.7 at
  //   512, 9.7 against 7.8 at 1024; 4 bits, two: 16 and 4 heads of 128 5.6 against 6.7 at 120, 8.4 against 6.5 at 250; 8 and 1
  //   5.9 against 7.0 at 500, 8.5 against 6.8 at 1000);
  // - the batch is too long for the tables in shared memory.  It has sequences enough to fill the GPU then, which is as
  //   good where they are alike and is not where one outlasts the others (16 query and 2 key-value heads of 64; 500 to
  //   1500 tokens: 512 sequences 48 us, 513 48; 0 to 4000 and one of 50000: 512 sequences 91 us, 513 392, 513 in two calls 98);
  // - tiles do not fit 32 bits.
  const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
  // Two tiles a warp, what joining its warps and asking for the next queries take (64 sequences of up to 2048 tokens, 2
  // key-value heads of 64: 13.1 us without them, 11.0 with them; 200 of up to 2000, 8 and 1 head of 128: 27.9 and 24.1).
  p.min_tiles = p.WT;  // one a warp: two or more take longer than their partials (7.6 us against 7.0 at 1024 tokens)
  p.start = 2 * loaders;
  const bool whole =
      capacity <= static_cast<int64_t>(few) * p.WT * tile || a.B > kMaxSplitBatch || (capacity / 16 + 1 + p.start) * a.B > INT32_MAX;
  p.ranges = split && !whole ? std::max(1, std::min(sms / p.groups, kMaxRanges)) : 0;
  // Caches without room for a tile a warp, or two where one or two sequences are all, leave half of the SMs to the
  // call's neighbours and have half the partials to join: one sequence of 8000 tokens, 16 query and 4 key-value heads of
  // 128, 9.3 us (on all SMs 10.0), 32 and 1 head 9.3 (11.2); 4 of 2000 tokens, 8 and 1 head, 6.9 (7.6).  With two tiles
  // a warp and many sequences all SMs are better: 48 of 342 tokens, 4 heads of 64, 7.5 (on half of them 8.5).
  const int64_t tiles = (capacity + tile - 1) / tile * a.B, all = static_cast<int64_t>(p.ranges) * loaders;
  if (tiles < (a.B <= 2 ? 2 * all : all)) p.ranges = (p.ranges + 1) / 2;
  return p;
}

}  // namespace
}  // namespace h3
