// Eviction from a paged cache: of each sequence of n > keep tokens the `recent`
// last ones stay, and of the n - recent older ones the front = keep - recent
// heaviest.  Rows move into places [0, keep):
//   the i-th kept old token beyond `front` (a "mover") goes to the i-th gap below,
//   the recent ones to front, front + 1, ... in their order.
// Few rows move where few tokens are evicted: movers and gaps are at most n - keep.
//
// First kernel, a cluster of 1 to 16 CTAs a sequence by the cache's room: each CTA
// holds its part of the weights in shared memory, as integers in their order.  The
// weight T of the front-th heaviest old token comes from counting passes over
// 8 bits of that order (the CTAs' counts are added up across the cluster), until all
// tokens that begin like T are kept or no bits are left; then
// kept = above T, or equal to it and among the first ones.  (11 bits a pass are one
// pass fewer, but 2048 counts from each of 8 CTAs for each of them took 12 us longer
// on the longest case below.)  Each warp owns a contiguous part of the tokens, so that a
// ballot numbers movers and gaps.  It writes their lists, moves the weights, and
// looks up the rows that the places are.  Bound by latencies: of 16 sequences of up to
// 4352 tokens 11 us, of one of 104448 22 (a load at a time from memory in each pass: 64).  The recent ones' weights
// are moved by the first CTA alone, 4096 at a time with two barriers each: with 50000 recent ones of 52224 kept, of the same 104448,
// the kernel takes 30 us under the profiler, with 1536 of 32760 25.
//
// Second kernel: moves the rows, d = n - keep places down.  Movers from beyond `keep`
// are not in the way of anything: a warp, or as many of its lanes as a short row has
// pieces, takes a row.  The place front + c is read by its mover, if it has one, then
// written by the recent row from old + c = front + c + d, whose place is then written by
// the one from old + c + d, and so on: a chain, in which a warp takes one row after the
// other, so that each of its lanes reads what it later overwrites.  There are
// min(d, recent) chains.  Where they are long and few, a CTA owns a column of pieces of
// all rows instead, and moves the movers first, then the recent rows in tiles from the
// first on.  23286 rows of 3456 bytes: 30 us, 5.4 TB/s read and written.
#include <algorithm>

#include "decode_common.cuh"

namespace h3 {
namespace {

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 256, kPasses = 4;
constexpr uint32_t kMostCtas = 16;  // of a cluster
constexpr int kMostHeld = 200 * 1024 / 4;  // weights in a CTA's shared memory

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of all CTAs of the cluster; what they wrote before is seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_load(const void* mine, uint32_t rank) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
// Weights in the order of unsigned integers: -0 as 0, a NaN above all.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return w != w ? 0xFFFFFFFFu : u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sums of the warps' x, y and z (the same in a warp's lanes): of x and y over the warps before this one in the cluster
// (CTAs in their order), and of all three over all.
struct Scan {
  uint32_t x, y, all_x, all_z;
};
__device__ __forceinline__ Scan cluster_scan(uint32_t x, uint32_t y, uint32_t z, uint32_t ctas, uint32_t rank,
                                             uint32_t (&sums)[3][kSelectWarps + 3]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  static_assert(kSelectWarps == 32, "a lane for each warp");
  if (lane < 3) sums[lane][warp] = lane == 0 ? x : lane == 1 ? y : z;
  __syncthreads();
  // every warp adds up all of them
  uint32_t before[3], all[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t of = sums[i][lane];
    before[i] = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? of : 0u);
    all[i] = __reduce_add_sync(0xFFFFFFFFu, of);
    if (threadIdx.x == 0) sums[i][kSelectWarps] = all[i];
  }
  Scan s{before[0], before[1], all[0], all[2]};
  if (ctas > 1) {
    cluster_sync();
    if (warp < 3) {  // asked for once a CTA (by every warp, the longest case below took 58.0 us instead of 54.5 with its rows)
      const uint32_t theirs = lane < static_cast<int>(ctas) ? peer_load(&sums[warp][kSelectWarps], lane) : 0u;
      const uint32_t earlier = __reduce_add_sync(0xFFFFFFFFu, lane < static_cast<int>(rank) ? theirs : 0u);
      const uint32_t of_all = __reduce_add_sync(0xFFFFFFFFu, theirs);
      if (lane == 0) {
        sums[warp][kSelectWarps + 1] = earlier;
        sums[warp][kSelectWarps + 2] = of_all;
      }
    }
    __syncthreads();
    s.x += sums[0][kSelectWarps + 1];
    s.y += sums[1][kSelectWarps + 1];
    s.all_x = sums[0][kSelectWarps + 2];
    s.all_z = sums[2][kSelectWarps + 2];
  }
  return s;
}

// CTAs that share a sequence of n tokens' select: one up to kAlone, whose barriers are its own; then as many as leave
// 4096 each.
constexpr int kAlone = 8192, kShare = 4096;
__host__ __device__ inline bool more_ctas(int64_t n, uint32_t ctas) { return n > kAlone && n > kShare * static_cast<int64_t>(ctas); }

// Tokens of a warp where a sequence has `old` to choose from: whole turns of 32.
__host__ __device__ inline int64_t tokens_per_warp(int64_t old, uint32_t ctas) {
  const int64_t warps = static_cast<int64_t>(ctas) * kSelectWarps;
  return ((old + warps - 1) / warps + 31) / 32 * 32;
}

// The row of the cache that place j of a sequence is, or -1 (reported).
__device__ __forceinline__ int row_of(const EvictArgs& a, const int32_t* table, int j) {
  const uint32_t p = fdiv(static_cast<uint32_t>(j), a.div_page);
  const int page = table[p];
  if (page < 0 || page >= a.num_pages) {
    atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));
    return -1;
  }
  return page * a.page_size + (j - static_cast<int>(p) * a.page_size);
}

// HELD: the weights' order is kept in shared memory; otherwise (more tokens than fit) it is read anew in each pass.
template <bool HELD>
__global__ void __launch_bounds__(kSelectThreads, 1)
    evict_select_kernel(const __grid_constant__ EvictArgs a, uint32_t most_ctas, int most_held) {
  extern __shared__ uint32_t held[];
  __shared__ uint32_t hist[kPasses][kBins];
  __shared__ uint32_t sums[2][3][kSelectWarps + 3];
  __shared__ uint32_t found[kPasses][3];  // bin, how many of its tokens are still wanted, how many it has
  __shared__ uint32_t above_of[kBins / 32];
  const int b = blockIdx.x / most_ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = most_ctas > 1 ? cluster_rank() : 0;
  for (int i = threadIdx.x; i < kPasses * kBins; i += kSelectThreads) (&hist[0][0])[i] = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), a.capacity));
  int* const list = a.ws + b * a.ints;
  if (rank == 0 && threadIdx.x == 0) a.len_out[b] = min(n, a.keep);
  if (n <= a.keep) return;  // the whole cluster
  float* const weights = a.weights + b * a.capacity;
  const int32_t* const table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
  const int old = n - a.recent, front = a.keep - a.recent;  // front < old
  // The cluster is as large as the cache has room for; a sequence with fewer tokens takes fewer of its CTAs, and the
  // barriers do not wait for those that have left (16 sequences of 2000 tokens in tables for 131072: all CTAs 20.0 us, one
  // 11.9; in tables for 2048 11.2).
  uint32_t ctas = 1;
  while (ctas < most_ctas && (more_ctas(n, ctas) || (HELD && tokens_per_warp(old, ctas) * kSelectWarps > most_held))) ctas *= 2;
  if (rank >= ctas) return;
  auto all_sync = [&] {
    if (ctas > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  // this warp's tokens are neighbours, 32 a turn
  const int64_t per_warp = tokens_per_warp(old, ctas), w0 = (rank * kSelectWarps + warp) * per_warp;
  const int begin = static_cast<int>(min(w0, static_cast<int64_t>(old)));
  const int end = static_cast<int>(min(w0 + per_warp, static_cast<int64_t>(old)));
  uint32_t* const mine = held + warp * per_warp - begin;  // of token j: mine[j]
  if constexpr (HELD) {
    constexpr int U = 8;
    for (int j0 = begin + lane; j0 < end; j0 += 32 * U) {
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = j0 + 32 * u < end ? weights[j0 + 32 * u] : 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + 32 * u < end) mine[j0 + 32 * u] = order_of(w[u]);
    }
    __syncwarp();
  }
  auto order = [&](int j) { return HELD ? mine[j] : order_of(weights[j]); };
  __syncthreads();
  // ---- the weight of the front-th heaviest ----
  uint32_t prefix = 0, seen_bits = 0;               // the bits of T that are known, and which those are
  uint32_t want = static_cast<uint32_t>(front);  // of tokens that begin with them, so many are kept
  bool all_ties = front == 0;
  if (front == 0) prefix = 0xFFFFFFFFu;  // none is kept
#pragma unroll 1
  for (int pass = 0; pass < kPasses && !all_ties; ++pass) {
    const int shift = 24 - 8 * pass;
#pragma unroll 4
    for (int j0 = begin; j0 < end; j0 += 32) {
      const uint32_t o = j0 + lane < end ? order(j0 + lane) : 0u;
      const bool counts = j0 + lane < end && (o & seen_bits) == prefix;
      if (!__any_sync(0xFFFFFFFFu, counts)) continue;
      // lanes with the same bin add to it once
      const uint32_t bin = counts ? o >> shift & 255u : 0xFFFFFFFFu;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, bin);
      if (counts && (same & ((1u << lane) - 1u)) == 0) atomicAdd(&hist[pass][bin], static_cast<uint32_t>(__popc(same)));
    }
    all_sync();
    // a thread adds up a bin over the cluster, from the last bin on
    uint32_t of_bin = 0, above = 0;
    if (threadIdx.x < kBins) {
      const int bin = kBins - 1 - static_cast<int>(threadIdx.x);
      if (ctas > 1) {
#pragma unroll
        for (uint32_t r = 0; r < kMostCtas; ++r)
          if (r < ctas) of_bin += peer_load(&hist[pass][bin], r);
      } else {
        of_bin = hist[pass][bin];
      }
      above = of_bin;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t m = __shfl_up_sync(0xFFFFFFFFu, above, off);
        if (lane >= off) above += m;
      }
      if (lane == 31) above_of[warp] = above;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
      above -= of_bin;
      above += __reduce_add_sync(0xFFFFFFFFu, lane < warp && lane < kBins / 32 ? above_of[lane] : 0u);
      if (above < want && want <= above + of_bin) {
        found[pass][0] = kBins - 1 - threadIdx.x;
        found[pass][1] = want - above;
        found[pass][2] = of_bin;
      }
    }
    __syncthreads();
    prefix |= found[pass][0] << shift;
    seen_bits |= 255u << shift;
    want = found[pass][1];
    all_ties = want == found[pass][2];
  }
  // ---- which are kept: above the prefix, or equal and among the first `want` (all_ties: all of those, or none at all) ----
  uint32_t ties_before = 0;
  if (!all_ties) {
    uint32_t ties = 0;
    for (int j = begin + lane; j < end; j += 32) ties += (order(j) & seen_bits) == prefix;
    ties_before = cluster_scan(__reduce_add_sync(0xFFFFFFFFu, ties), 0, 0, ctas, rank, sums[0]).x;
  }
  auto walk = [&](auto&& each) {
    uint32_t seen = ties_before;
#pragma unroll 2
    for (int j0 = begin; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t o = (j < end ? order(j) : 0u) & seen_bits;
      const bool tie = j < end && o == prefix;
      const uint32_t tied = all_ties ? 0u : __ballot_sync(0xFFFFFFFFu, tie);
      const bool kept =
          j < end && front > 0 && (o > prefix || (tie && (all_ties || seen + __popc(tied & ((1u << lane) - 1u)) < want)));
      seen += __popc(tied);
      const uint32_t movers = __ballot_sync(0xFFFFFFFFu, kept && j >= front);
      const uint32_t gaps = __ballot_sync(0xFFFFFFFFu, j < end && !kept && j < front);
      each(j0, movers, gaps);
    }
  };
  uint32_t n_movers = 0, n_gaps = 0, n_below = 0;  // below: from places below keep
  walk([&](int j0, uint32_t movers, uint32_t gaps) {
    n_movers += __popc(movers);
    n_gaps += __popc(gaps);
    const int64_t left = static_cast<int64_t>(a.keep) - j0;  // this turn's tokens below keep
    n_below += left >= 32 ? __popc(movers) : left > 0 ? __popc(movers & ((1u << left) - 1u)) : 0;
    if constexpr (HELD) {  // in the place of the turn's weights, for the second time over them
      __syncwarp();
      if (lane < 2) mine[j0 + lane] = lane == 0 ? movers : gaps;
    }
  });
  const Scan at = cluster_scan(n_movers, n_gaps, n_below, ctas, rank, sums[1]);
  uint32_t to_mover = at.x, to_gap = at.y;
  int *const from = list + kEvictHeader, *const to = from + a.most, *const chain = to + a.most;
  const int chains = min(a.recent, n - a.keep);
  auto list_turn = [&](int j0, uint32_t movers, uint32_t gaps) {
    const uint32_t before = (1u << lane) - 1u;
    const int c = j0 + lane - front;  // the chain that begins with this place
    if (c >= 0 && c < chains && j0 + lane < end && !(movers >> lane & 1u)) chain[c] = -1;
    if (movers >> lane & 1u) from[to_mover + __popc(movers & before)] = j0 + lane;
    if (gaps >> lane & 1u) to[to_gap + __popc(gaps & before)] = j0 + lane;
    to_mover += __popc(movers);
    to_gap += __popc(gaps);
  };
  if constexpr (HELD) {
#pragma unroll 4
    for (int j0 = begin; j0 < end; j0 += 32) list_turn(j0, mine[j0], mine[j0 + 1]);
  } else {
    walk(list_turn);
  }
  const int moves = static_cast<int>(at.all_x);
  if (rank == 0 && threadIdx.x == 0) {
    list[0] = moves;
    list[1] = static_cast<int>(at.all_z);
  }
  all_sync();
  // ---- the weights move: gaps are below all movers and recent ones; the recent ones, from the first on, to where movers
  // and they themselves have been read ----
  constexpr int U = 2, R = 4;
  const int64_t step = static_cast<int64_t>(ctas) * kSelectThreads, me = static_cast<int64_t>(rank) * kSelectThreads + threadIdx.x;
  float recent_w[R];  // the first CTA's
  auto read_recent = [&](int64_t i0) {
#pragma unroll
    for (int u = 0; u < R; ++u)
      if (i0 + u * kSelectThreads < a.recent) recent_w[u] = weights[old + i0 + u * kSelectThreads];
  };
  auto write_recent = [&](int64_t i0) {
#pragma unroll
    for (int u = 0; u < R; ++u)
      if (i0 + u * kSelectThreads < a.recent) weights[front + i0 + u * kSelectThreads] = recent_w[u];
  };
  if (rank == 0) read_recent(threadIdx.x);
  for (int64_t i0 = me; i0 < moves; i0 += U * step) {
    int f[U], t[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f[u] = i0 + u * step < moves ? from[i0 + u * step] : -1;
      t[u] = f[u] >= 0 ? to[i0 + u * step] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (f[u] < 0) continue;
      weights[t[u]] = weights[f[u]];
      const int to_row = row_of(a, table, t[u]);
      from[i0 + u * step] = row_of(a, table, f[u]);
      to[i0 + u * step] = to_row;
      if (f[u] < a.keep) chain[f[u] - front] = to_row;
    }
  }
  all_sync();
  if (rank == 0) {
    write_recent(threadIdx.x);
    for (int64_t i0 = R * kSelectThreads; i0 < a.recent; i0 += R * kSelectThreads) {
      __syncthreads();
      read_recent(i0 + threadIdx.x);
      __syncthreads();
      write_recent(i0 + threadIdx.x);
    }
  }
  if (a.recent > R * kSelectThreads) all_sync();  // otherwise all recent ones were read before the last one
  for (int64_t j = a.keep + me; j < n; j += step) weights[j] = 0.0f;
}

constexpr int kMoveThreads = 256;
constexpr int kLanes = 8;                       // pieces of a row that a CTA owns where chains are long
constexpr int kAtOnce = kMoveThreads / kLanes;  // rows that it takes at a time
constexpr int kMoveUnroll = 4;

struct MovePlan {
  int columns[4];  // CTAs that own kLanes pieces of each array
  int piece[2];    // bytes of a piece of K and V, and of the scales: 16, 8 or 4
  int lanes_log2;  // lanes that take a row where columns are not owned
};

// The moves that are in order: `below` movers, then the recent rows, of the pieces from piece0 on.
template <class T>
__device__ __forceinline__ void move_column(const EvictArgs& a, uint8_t* base, int bytes, int piece0, int b, int n, const int* list) {
  const int below = list[1], old = n - a.recent, front = a.keep - a.recent;
  const int *from = list + kEvictHeader, *to = from + a.most;
  const int col = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const bool mine = (piece0 + col) * static_cast<int>(sizeof(T)) < bytes;
  uint8_t* const column = base + static_cast<int64_t>(piece0 + col) * sizeof(T);
  const int32_t* const table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
  T x[kMoveUnroll];
  int dst[kMoveUnroll];
  auto move = [&](int count, auto&& src_of, auto&& dst_of) {
    for (int64_t i0 = 0; i0 < count; i0 += kAtOnce * kMoveUnroll) {
      int src[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int64_t i = i0 + u * kAtOnce + slot;
        src[u] = dst[u] = -1;
        if (mine && i < count) {
          src[u] = src_of(static_cast<int>(i));
          dst[u] = dst_of(static_cast<int>(i));
        }
      }
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        if (src[u] < 0 || dst[u] < 0)
          dst[u] = -1;
        else
          x[u] = *reinterpret_cast<const T*>(column + static_cast<int64_t>(src[u]) * bytes);
      }
      __syncthreads();  // what the stores overwrite has been read
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u)
        if (dst[u] >= 0) *reinterpret_cast<T*>(column + static_cast<int64_t>(dst[u]) * bytes) = x[u];
      __syncthreads();
    }
  };
  move(below, [&](int i) { return from[i]; }, [&](int i) { return to[i]; });
  move(a.recent, [&](int i) { return row_of(a, table, old + i); }, [&](int i) { return row_of(a, table, front + i); });
}

// `pieces` pieces of each of two arrays, from row src to row dst, by `lanes` lanes of a warp.
template <class T>
__device__ __forceinline__ void move_row(uint8_t* first, uint8_t* second, int pieces, int64_t src, int64_t dst, int lanes) {
  for (int i0 = threadIdx.x & (lanes - 1); i0 < 2 * pieces; i0 += lanes * kMoveUnroll) {
    T x[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = i0 + lanes * u;
      if (i < 2 * pieces) x[u] = reinterpret_cast<const T*>(i < pieces ? first : second)[src * pieces + (i < pieces ? i : i - pieces)];
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = i0 + lanes * u;
      if (i < 2 * pieces) reinterpret_cast<T*>(i < pieces ? first : second)[dst * pieces + (i < pieces ? i : i - pieces)] = x[u];
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 4) evict_move_kernel(const __grid_constant__ EvictArgs a, const __grid_constant__ MovePlan p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.y;
  const int n = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), a.capacity));
  if (n <= a.keep) return;
  const int* const list = a.ws + b * a.ints;
  const int d = n - a.keep, chains = min(a.recent, d);
  // 16 sequences, 256 recent rows, of 128 on average to be evicted: chains 21.2 us, columns 19.6; 1024 rows in chains of 5
  // 20.1, in columns 23.2
  if (static_cast<int64_t>(d) * max(2, a.recent / (kAtOnce * kMoveUnroll)) >= a.recent) {
    const int *from = list + kEvictHeader, *to = from + a.most, *chain = to + a.most;
    const int32_t* const table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
    const int below = list[1], old = n - a.recent, front = a.keep - a.recent;
    const int64_t items = static_cast<int64_t>(chains) + list[0] - below;
    const int lanes = 1 << p.lanes_log2, at_once = kMoveThreads >> p.lanes_log2;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * at_once + (threadIdx.x >> p.lanes_log2); i < items;
         i += static_cast<int64_t>(gridDim.x) * at_once) {
      // a chain: its first place goes to a gap, if it is a mover's, and each recent row to the place moved or left before
      const bool in_chain = i < chains;
      int src = in_chain ? row_of(a, table, front + static_cast<int>(i)) : from[below + i - chains];
      int dst = in_chain ? chain[i] : to[below + i - chains];
      int64_t r = in_chain ? i : a.recent;
      while (true) {
        if (src >= 0 && dst >= 0) {
          move_row<uint4>(a.row[0], a.row[1], a.row_bytes[0] / 16, src, dst, lanes);
          if (a.row[2]) move_row<uint32_t>(a.row[2], a.row[3], a.row_bytes[1] / 4, src, dst, lanes);
        }
        if (r >= a.recent) break;
        dst = src;
        src = row_of(a, table, old + static_cast<int>(r));
        r += d;
      }
    }
    return;
  }
  int columns = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) columns += p.columns[i];
  if (static_cast<int>(blockIdx.x) >= columns) return;
  int column = blockIdx.x, of = 0;
  while (column >= p.columns[of]) column -= p.columns[of++];
  const int bytes = a.row_bytes[of >> 1], piece = p.piece[of >> 1];
  if (piece == 16)
    move_column<uint4>(a, a.row[of], bytes, column * kLanes, b, n, list);
  else if (piece == 8)
    move_column<uint2>(a, a.row[of], bytes, column * kLanes, b, n, list);
  else
    move_column<uint32_t>(a, a.row[of], bytes, column * kLanes, b, n, list);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // One CTA for up to 8192 tokens, which has no cluster to wait for; then as many as leave 4096 each, up to 16, and up to
  // one an SM over all sequences (35 of 37518 tokens: 16 each, in four waves, 124 us, 4 each 49), but for weights that
  // shared memory does not hold otherwise.
  const int64_t most_old = std::max<int64_t>(a.capacity - a.recent, 0);
  auto held_by = [&](uint32_t ctas) { return tokens_per_warp(most_old, ctas) * kSelectWarps; };
  uint32_t ctas = 1;
  while (ctas < kMostCtas && more_ctas(a.capacity, ctas) &&
         (static_cast<int64_t>(a.B) * ctas * 2 <= sms || held_by(ctas) > kMostHeld))
    ctas *= 2;
  const int64_t each = held_by(ctas);
  const bool fits = each <= kMostHeld;
  auto* const select = fits ? evict_select_kernel<true> : evict_select_kernel<false>;
  static std::atomic<bool> attr_set[64];  // calls of several host threads
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostHeld * 4);
    // clusters of more than 8
    if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(evict_select_kernel<false>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = fits ? static_cast<size_t>(each) * 4 : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, select, a, ctas, static_cast<int>(fits ? each : 0));
  if (e != cudaSuccess) return e;
  MovePlan p = {};
  int columns = 0;
  for (int i = 0; i < 4; ++i) {
    const int bytes = a.row_bytes[i >> 1];
    if (!a.row[i]) continue;
    p.piece[i >> 1] = bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : 4;
    p.columns[i] = (bytes / p.piece[i >> 1] + kLanes - 1) / kLanes;
    columns += p.columns[i];
  }
  while (p.lanes_log2 < 5 && (1 << p.lanes_log2) < a.row_bytes[0] / 16 * 2) ++p.lanes_log2;
  // chains and movers from beyond keep: lanes for each that there may be, up to 8 CTAs an SM over all sequences
  const int64_t longest = std::max<int64_t>(a.capacity - a.keep, 0), at_once = kMoveThreads >> p.lanes_log2;
  const int64_t items = std::min<int64_t>(a.recent, longest) + std::min<int64_t>(a.most, std::max<int64_t>(longest - a.recent, 0));
  const int64_t dealt = std::min<int64_t>((items + at_once - 1) / at_once, std::max(8 * sms / a.B, 1));
  return launch_dependent(evict_move_kernel, dim3(static_cast<unsigned>(std::max<int64_t>(columns, dealt)), static_cast<unsigned>(a.B)),
                          kMoveThreads, 0, stream, a, p);
}

}  // namespace h3
