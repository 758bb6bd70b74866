// Eviction from a paged cache: of each sequence of n > keep tokens the `recent`
// last ones stay, and of the n - recent older ones the front = keep - recent
// heaviest.  Rows move into places [0, keep):
//   the i-th kept old token beyond `front` (a "mover") goes to the i-th gap below,
//   the recent ones to front, front + 1, ... in their order.
// Few rows move where few tokens are evicted: movers and gaps are at most n - keep.
//
// First kernel, a cluster of 1 to 8 CTAs a sequence by the cache's room: the
// weight T of the front-th heaviest old token by three counting passes over 11, 11
// and 10 bits of the weights' order (each CTA counts its part of the tokens, the counts
// are added up across the cluster), then kept = above T, or equal to it and among
// the first ones; each warp owns a contiguous part of the tokens, so that a
// ballot numbers movers and gaps.  It writes their lists, and moves the weights.
//
// Second kernel: moves the rows.  A CTA owns a column of pieces of all rows of one
// sequence, so that the order in which rows are read and written is its own: movers
// from below `keep`, then the recent rows in tiles from the first on (a row moves
// down, so what a tile overwrites has been read).  Movers from beyond `keep` are not in the way
// of anything and are dealt to further CTAs.
#include <algorithm>

#include "decode_common.cuh"

namespace h3 {
namespace {

constexpr int kSelectThreads = 512, kSelectWarps = kSelectThreads / 32;
constexpr int kBins = 2048, kPasses = 3;

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

// Sum of `mine` over the threads before this one in the cluster (CTAs in their order), and over all of them.
struct Scan {
  uint32_t before, all;
};
__device__ __forceinline__ Scan cluster_scan(uint32_t mine, uint32_t ctas, uint32_t rank, uint32_t (&warp_sum)[kSelectWarps + 1]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t n = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t m = __shfl_up_sync(0xFFFFFFFFu, n, off);
    if (lane >= off) n += m;
  }
  if (lane == 31) warp_sum[warp] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t sum = 0;
    for (int w = 0; w < kSelectWarps; ++w) sum += warp_sum[w];
    warp_sum[kSelectWarps] = sum;
  }
  cluster_sync();
  Scan s{n - mine, 0};
  for (int w = 0; w < warp; ++w) s.before += warp_sum[w];
  for (uint32_t r = 0; r < ctas; ++r) {
    const uint32_t of = peer_load(&warp_sum[kSelectWarps], r);
    if (r < rank) s.before += of;
    s.all += of;
  }
  return s;
}

__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(const __grid_constant__ EvictArgs a, uint32_t ctas) {
  __shared__ uint32_t hist[kPasses][kBins];
  __shared__ uint32_t scan[3][kSelectWarps + 1];
  __shared__ uint32_t found[kPasses][2];  // bin, and how many of its tokens are still wanted
  __shared__ uint32_t above_of[kSelectWarps];
  const int b = blockIdx.x / ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ctas > 1 ? cluster_rank() : 0;
  for (int i = threadIdx.x; i < kPasses * kBins; i += kSelectThreads) (&hist[0][0])[i] = 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), a.capacity));
  int* const list = a.ws + static_cast<int64_t>(b) * (kEvictHeader + 2 * static_cast<int64_t>(a.most));
  if (rank == 0 && threadIdx.x == 0) {
    a.len_out[b] = min(n, a.keep);
    list[0] = list[1] = 0;
  }
  if (n <= a.keep) return;  // the whole cluster
  float* const weights = a.weights + b * a.capacity;
  const int old = n - a.recent, front = a.keep - a.recent;  // front < old
  // this thread's tokens: a warp's are neighbours, 32 at a time
  const int64_t warps = static_cast<int64_t>(ctas) * kSelectWarps, per_warp = ((old + warps - 1) / warps + 31) / 32 * 32;
  const int64_t w0 = (rank * kSelectWarps + warp) * per_warp;
  const int begin = static_cast<int>(min(w0, static_cast<int64_t>(old)));
  const int end = static_cast<int>(min(w0 + per_warp, static_cast<int64_t>(old)));
  __syncthreads();
  // ---- the weight of the front-th heaviest ----
  uint32_t prefix = 0, want = static_cast<uint32_t>(front);  // of tokens whose order begins with prefix, so many are kept
  if (front > 0) {
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      for (int j = begin + lane; j < end; j += 32) {
        const uint32_t o = order_of(weights[j]);
        if ((o & mask) == prefix) atomicAdd(&hist[pass][o >> shift & ((1u << bits) - 1u)], 1u);
      }
      cluster_sync();
      // each thread adds up four bins over the cluster, from the last bin on
      uint32_t mine[kBins / kSelectThreads], sum = 0;
#pragma unroll
      for (int i = 0; i < kBins / kSelectThreads; ++i) {
        const int bin = kBins - 1 - (static_cast<int>(threadIdx.x) * (kBins / kSelectThreads) + i);
        mine[i] = 0;
        for (uint32_t r = 0; r < ctas; ++r) mine[i] += peer_load(&hist[pass][bin], r);
        sum += mine[i];
      }
      uint32_t above = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t m = __shfl_up_sync(0xFFFFFFFFu, above, off);
        if (lane >= off) above += m;
      }
      if (lane == 31) above_of[warp] = above;
      __syncthreads();
      above -= sum;
      for (int w = 0; w < warp; ++w) above += above_of[w];
#pragma unroll
      for (int i = 0; i < kBins / kSelectThreads; ++i) {
        if (above < want && want <= above + mine[i]) {
          found[pass][0] = kBins - 1 - (threadIdx.x * (kBins / kSelectThreads) + i);
          found[pass][1] = want - above;
        }
        above += mine[i];
      }
      __syncthreads();
      prefix |= found[pass][0] << shift;
      want = found[pass][1];
    }
  } else {
    prefix = 0xFFFFFFFFu;  // none is kept
    want = 0;
  }
  // ---- which are kept: above the prefix, or equal and among the first `want` ----
  uint32_t ties = 0;
  for (int j = begin + lane; j < end; j += 32) ties += order_of(weights[j]) == prefix;
  ties = __reduce_add_sync(0xFFFFFFFFu, ties);
  const uint32_t ties_before = __shfl_sync(0xFFFFFFFFu, cluster_scan(lane == 0 ? ties : 0u, ctas, rank, scan[0]).before, 0);
  auto walk = [&](auto&& each) {
    uint32_t seen = ties_before;
    for (int j0 = begin; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t o = j < end ? order_of(weights[j]) : 0u;
      const bool tie = j < end && o == prefix;
      const uint32_t tied = __ballot_sync(0xFFFFFFFFu, tie);
      const bool kept = j < end && front > 0 && (o > prefix || (tie && seen + __popc(tied & ((1u << lane) - 1u)) < want));
      seen += __popc(tied);
      const uint32_t movers = __ballot_sync(0xFFFFFFFFu, kept && j >= front);
      const uint32_t gaps = __ballot_sync(0xFFFFFFFFu, j < end && !kept && j < front);
      each(j, movers, gaps);
    }
  };
  uint32_t n_movers = 0, n_gaps = 0, n_below = 0;
  walk([&](int j, uint32_t movers, uint32_t gaps) {
    n_movers += __popc(movers);
    n_gaps += __popc(gaps);
    n_below += __popc(__ballot_sync(0xFFFFFFFFu, (movers >> lane & 1u) && j < a.keep));
  });
  const Scan at_mover = cluster_scan(lane == 0 ? n_movers : 0u, ctas, rank, scan[1]);
  const Scan at_gap = cluster_scan(lane == 0 ? n_gaps : 0u, ctas, rank, scan[2]);
  uint32_t to_mover = __shfl_sync(0xFFFFFFFFu, at_mover.before, 0), to_gap = __shfl_sync(0xFFFFFFFFu, at_gap.before, 0);
  int *const from = list + kEvictHeader, *const to = from + a.most;
  walk([&](int j, uint32_t movers, uint32_t gaps) {
    const uint32_t before = (1u << lane) - 1u;
    if (movers >> lane & 1u) from[to_mover + __popc(movers & before)] = j;
    if (gaps >> lane & 1u) to[to_gap + __popc(gaps & before)] = j;
    to_mover += __popc(movers);
    to_gap += __popc(gaps);
  });
  if (rank == 0 && threadIdx.x == 0) list[0] = static_cast<int>(at_mover.all);
  if (lane == 0 && n_below > 0) atomicAdd(&list[1], static_cast<int>(n_below));
  cluster_sync();
  // ---- the weights move: gaps are below all movers and recent ones, which are read before they are overwritten ----
  const int moves = static_cast<int>(at_mover.all);
  for (int i = static_cast<int>(rank) * kSelectThreads + threadIdx.x; i < moves; i += ctas * kSelectThreads)
    weights[to[i]] = weights[from[i]];
  cluster_sync();
  if (rank == 0) {
    constexpr int U = 4;
    for (int64_t i0 = 0; i0 < a.recent; i0 += U * kSelectThreads) {
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * kSelectThreads + threadIdx.x;
        if (i < a.recent) w[u] = weights[old + i];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * kSelectThreads + threadIdx.x;
        if (i < a.recent) weights[front + i] = w[u];
      }
      __syncthreads();
    }
  }
  cluster_sync();
  for (int64_t j = a.keep + rank * kSelectThreads + static_cast<int>(threadIdx.x); j < n; j += ctas * kSelectThreads) weights[j] = 0.0f;
}

constexpr int kMoveThreads = 256;
constexpr int kLanes = 8;                       // pieces of a row that a CTA owns
constexpr int kAtOnce = kMoveThreads / kLanes;  // rows that it takes a turn
constexpr int kMoveUnroll = 8;

struct MovePlan {
  int columns[4];  // groups of kLanes pieces of each array
  int piece[2];    // bytes of a piece of K and V, and of the scales: 16, 8 or 4
  int parts;       // CTAs a column: one for what is ordered, the others for movers from beyond keep
};

template <class T>
__device__ __forceinline__ void move_rows(const EvictArgs& a, uint8_t* base, int bytes, int piece0, int b, int part, int parts) {
  const int n = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), a.capacity));
  if (n <= a.keep) return;
  const int* list = a.ws + static_cast<int64_t>(b) * (kEvictHeader + 2 * static_cast<int64_t>(a.most));
  const int *from = list + kEvictHeader, *to = from + a.most;
  const int col = threadIdx.x % kLanes, slot = threadIdx.x / kLanes;
  const bool mine = (piece0 + col) * static_cast<int>(sizeof(T)) < bytes;
  const int64_t off = static_cast<int64_t>(piece0 + col) * sizeof(T);
  const int* table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
  auto place = [&](int j) -> uint8_t* {
    const uint32_t p = fdiv(static_cast<uint32_t>(j), a.div_page);
    const int page = table[p];
    if (page < 0 || page >= a.num_pages) {
      atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));
      return nullptr;
    }
    return base + (static_cast<int64_t>(page) * a.page_size + (j - static_cast<int>(p) * a.page_size)) * bytes + off;
  };
  T x[kMoveUnroll];
  uint8_t* dst[kMoveUnroll];
  // `count` rows: the i-th from src_of(i) to dst_of(i), `ordered` turns after one another
  auto move = [&](int first, int count, int step, bool ordered, auto&& src_of, auto&& dst_of) {
    for (int64_t i0 = first; i0 < count; i0 += step) {
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int i = static_cast<int>(min(i0 + u * kAtOnce + slot, static_cast<int64_t>(count)));
        dst[u] = nullptr;
        if (mine && i < count) {
          const uint8_t* src = place(src_of(i));
          dst[u] = place(dst_of(i));
          if (src && dst[u])
            x[u] = *reinterpret_cast<const T*>(src);
          else
            dst[u] = nullptr;
        }
      }
      if (ordered) __syncthreads();
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u)
        if (dst[u]) *reinterpret_cast<T*>(dst[u]) = x[u];
      if (ordered) __syncthreads();
    }
  };
  const int movers = list[0], below = list[1], turn = kAtOnce * kMoveUnroll;
  auto mover = [&](int i) { return from[i]; };
  auto gap = [&](int i) { return to[i]; };
  if (part == 0) {
    move(0, below, turn, false, mover, gap);
    __syncthreads();
    const int old = n - a.recent, front = a.keep - a.recent;
    move(0, a.recent, turn, true, [&](int i) { return old + i; }, [&](int i) { return front + i; });
  }
  if (part > 0 || parts == 1)
    move(below + (parts == 1 ? 0 : part - 1) * turn, movers, (parts == 1 ? 1 : parts - 1) * turn, false, mover, gap);
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a, const __grid_constant__ MovePlan p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int column = blockIdx.x, of = 0;
  while (column >= p.columns[of]) column -= p.columns[of++];
  const int piece = p.piece[of >> 1], bytes = a.row_bytes[of >> 1];
  if (piece == 16)
    move_rows<uint4>(a, a.row[of], bytes, column * kLanes, blockIdx.z, blockIdx.y, p.parts);
  else if (piece == 8)
    move_rows<uint2>(a, a.row[of], bytes, column * kLanes, blockIdx.z, blockIdx.y, p.parts);
  else
    move_rows<uint32_t>(a, a.row[of], bytes, column * kLanes, blockIdx.z, blockIdx.y, p.parts);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t stream) {
  // a CTA's part of the tokens is passed over six times: 4096 of them a CTA, up to the 8 CTAs that any cluster may have
  uint32_t ctas = 1;
  while (ctas < 8 && a.capacity > 4096 * static_cast<int64_t>(ctas)) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, ctas);
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
  // movers from beyond keep: one more CTA for each two turns of them that there may be, up to 32
  const int64_t free_movers = std::max<int64_t>(std::min<int64_t>(a.most, a.capacity - a.keep - a.recent), 0);
  p.parts = 1 + static_cast<int>(std::min<int64_t>((free_movers + 511) / 512, 32));
  return launch_dependent(evict_move_kernel, dim3(static_cast<unsigned>(columns), static_cast<unsigned>(p.parts), static_cast<unsigned>(a.B)),
                          kMoveThreads, 0, stream, a, p);
}

}  // namespace h3
