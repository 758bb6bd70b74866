// Attention of one new token per sequence over a paged key-value cache.
//
//   o_h = sum_j softmax_j(scale q_h . k_j) v_j,   j < kv_len[b]
//
// Memory-bound: every cached K and V row is read once and used for the
// G = Hq / Hkv query heads that share it, 2 G multiply-adds per element read.
// From G = 4 on that is more than the CUDA cores do at the memory's rate, so
// both products are tensor-core products of a warp (mma.sync m16n8k16: a
// tcgen05 tile has 128 rows at least, and a decode step has G).  The cache
// side is the 16-row operand, the query heads the 8 columns:
//   S^T[16 tokens, 8 heads] = K[16, D] q^T[D, 8]
//   O^T[16 channels, 8 heads] += V^T[16, 16 tokens] P^T[16 tokens, 8 heads]
// so that up to 8 heads cost one pass, and P^T is S^T's accumulator with each
// 8x8 block transposed (movmatrix).  Groups of 9 to 16 heads take two column
// tiles; larger groups are cut into tiles of 16.  Where there is an even number
// of those, the two warps of neighbouring ones load every second token tile
// each and use both, a barrier of the pair a turn; an odd number reads the cache
// again for each (from L2, as they run side by side: 28 sequences of 754 thousand tokens,
// 48 heads to one of 128 122 us, 32 to one 74, 16 to one 67).
//
// Work.  Lengths are known on the device only, and are unlike.  A "unit head"
// is a key-value head (and a tile of 16 query heads of its group).  A CTA
// takes WH neighbouring unit heads, so that its warps read one contiguous
// stretch of the pages, and its other factor WT = warps / WH splits the
// tokens.  All sequences' tiles of TILE tokens are numbered through and cut into
// one range an SM, half of the SMs for small caches (for each group of WH unit
// heads), so CTAs differ by one tile however unlike the lengths are; each sequence counts two tiles a warp more than it
// has, which is what starting on one takes.  A range that holds all of a sequence
// writes its output; of a sequence that ranges share, each range writes its
// unnormalised O, its maximum and its sum to the workspace, and a second
// kernel joins them in the order of the ranges (results do not depend on
// timing).  Each warp streams its own tiles through its own ring of
// shared-memory stages with cp.async, ahead over sequence borders, without a
// barrier; a tile's page is asked for two tiles before its rows.
//
// Softmax in float32 with exp2 against a reference that follows the running
// maximum once it is behind by more than 2^8 (rare, so the rescaling of O and
// the exchange of maxima are a branch).  P goes into the second product as the
// sum of two bf16 values, P rounded and what the rounding left: with P rounded
// once the output's error against 64 bits was 1.35 times its own rounding's,
// and the second product is free here (it runs beside the loads).
//
// Measured: 104448 tokens, 24 heads of 128, one sequence: 181 us, 7.1 TB/s (a
// copy reaches 6.8).  16 sequences of 4096 to 8192 tokens, 4 heads of 128: 36 us
// of 30 at that rate: 4 us until the first tile has come through lengths, page
// table and rows, 3 us between the first and the last CTA's end, 2 us for the join.
// 64 sequences of up to 2048 tokens, 2 heads of 64: 11 us of 5.
// One row of 256 bytes a bulk copy instead (any page size, no lane work) took
// 236 us for the first case: about 14 cycles a copy and SM.  Joining in the decode kernel
// by the CTA that arrives last took 41 us for the second: the arrival's fence and atomic,
// and the join by one CTA, are longer than a kernel that waits beside it.
#include "decode_common.cuh"
#include "ptx.cuh"

namespace h3 {
namespace {

// 16 bytes global -> shared; zeros when !valid (the source is not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Of the two warps that use barrier `id`.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NT: tiles of 8 query heads (1 or 2).
template <int D, int NT>
struct DecodeCfg {
  static constexpr int kTile = D == 64 ? 32 : 16;  // tokens a warp takes at a time: 8 KB of K and V at D 64 and 128
  static constexpr int kWarps = D == 256 ? 4 : 8;
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kTile * D * 2;  // of K, and the same of V
  static constexpr int kRing = kWarps * kStages * 2 * kTileBytes;
  // joining the warps of a unit head: accumulators, max and sum of every second warp, 8 heads at a time
  static constexpr int kJoin = kWarps / 2 * 8 * D * 4;
  static constexpr int kStats = kWarps / 2 * 8 * 2 * 4;
  static constexpr int kSmem = kRing + kJoin + kStats + 2 * kMaxSplitBatch * 4;
  static constexpr int kHeads = NT * 8;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

// One column tile at D 128 takes 198 registers a thread, which with the joining kernel's 56 just fill an SM's; two take
// 242, and the join's CTA waits for this one's end.  Held to 200 they spill in the loop: 28 sequences of 0 to 52182
// tokens, 32 heads to one, 73 us and 94.  At D 256 two column tiles take all 255 registers and spill (16 bytes stored and
// 24 loaded a thread; 40 and 72 where warps share their tiles), one takes 244 and does not.
// W: the scores are kept for the tokens' weights.
template <int D, int NT, int SHARE, bool W>
__global__ void __launch_bounds__(DecodeCfg<D, NT>::kWarps * 32, 1) decode_kernel(const __grid_constant__ Kernelargs k) {
  using C = DecodeCfg<D, NT>;
  constexpr int TILE = C::kTile, MT = TILE / 16, STAGES = C::kStages;
  constexpr int CH = D / 8;  // 16-byte pieces of a row
  const DecodeArgs& a = k.a;
  const DecodePlan& p = k.p;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + C::kRing);
  float* stats = reinterpret_cast<float*>(smem + C::kRing + C::kJoin);
  int* end = reinterpret_cast<int*>(smem + C::kRing + C::kJoin + C::kStats);
  int* lens = end + kMaxSplitBatch;  // without a split: of the one sequence
  __shared__ uint32_t shared_mask[SHARE > 1 ? C::kWarps : 1][STAGES];  // tokens of each warp's stages that are attended
  // The lengths and the page table are the first two links of the chain to the first K and V row, and the last
  // step's cache has pushed them out of L2: they are brought back while the kernel before this one drains.  (L2 is
  // where all SMs' writes meet, so what that kernel still writes is not missed.)
  if (threadIdx.x * 32 < static_cast<unsigned>(a.B)) prefetch_l2(a.kv_len + threadIdx.x * 32);
  {
    const int64_t line = (static_cast<int64_t>(blockIdx.x) * (C::kWarps * 32) + threadIdx.x) * 32;
    if (line < static_cast<int64_t>(a.B) * a.max_pages) prefetch_l2(a.page_table + line);
  }
  // The joining kernel may start once every CTA is past its wait: it reads the lengths before its own.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wh = warp % p.WH, wt = warp / p.WH;
  // Warps that share their tiles: of the same tokens, neighbouring unit heads.
  const int peer = warp % SHARE, peer0 = warp - peer;
  const int r = blockIdx.x / p.groups;
  const int unit = (blockIdx.x - r * p.groups) * p.WH + wh;
  const int kvh = unit / p.q_tiles, qt = unit - kvh * p.q_tiles;
  const int G = a.Hq / a.Hkv;
  const int head0 = kvh * G + qt * 16;            // first query head of the unit
  const int heads = min(G - qt * 16, C::kHeads);  // its query heads

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

  // The tiles that this warp and its peers load, in the order they are used, over sequence borders: peer i takes tile + i.
  struct Walk {
    int b, tile, stop, len;  // sequence, tile of the sequence, the range's end in it
  };
  auto enter = [&](Walk& w) {  // to the first tile at or after the present one that is there
    while (w.tile >= w.stop) {
      if (p.ranges == 0 || seq_end(w.b) >= t1) {
        w.b = -1;
        return;
      }
      ++w.b;
      w.stop = stop_tile(w.b);
      w.tile = wt * SHARE;
      w.len = seq_len(w.b);
    }
  };
  Walk ld;
  ld.b = b0;
  ld.tile = first_tile(b0) + wt * SHARE;
  ld.stop = stop_tile(b0);
  ld.len = seq_len(b0);
  enter(ld);

  const uint32_t ring = smem_u32(smem) + warp * (STAGES * 2 * C::kTileBytes);
  const int64_t row_stride = static_cast<int64_t>(a.Hkv) * D;

  // The lane's tokens of the next two tiles to be loaded: their pages, asked for two turns ahead and looked at only when
  // the rows are loaded, and their rows in the pages.  token_row < 0: no such token.  -2: no such tile.
  int page[2], token_row[2];
  auto look_ahead = [&](int i) {
    token_row[i] = -2;
    if (ld.b < 0) return;
    const int token = (ld.tile + peer) * TILE + lane % TILE;
    token_row[i] = -1;
    if (token < ld.len && (SHARE == 1 || ld.tile + peer < ld.stop)) {
      const uint32_t pg = fdiv(static_cast<uint32_t>(token), a.div_page);
      page[i] = a.page_table[static_cast<int64_t>(ld.b) * a.max_pages + pg];
      token_row[i] = token - static_cast<int>(pg) * a.page_size;
    }
    ld.tile += p.WT * SHARE;
    enter(ld);
  };
  look_ahead(0);
  look_ahead(1);
  uint32_t mask_of[STAGES];  // tokens of each stage's tile that are attended
  const uint16_t* kbase = a.k_pages + kvh * D + (lane % CH) * 8;
  const uint16_t* vbase = a.v_pages + kvh * D + (lane % CH) * 8;
  // Fills stage `at` with the next tile; rows that are not attended are zeros.
  auto load = [&](int at, uint32_t& mask) {
    if (token_row[0] != -2) {  // the same in all lanes
      int row = -1;  // of the whole cache
      if (token_row[0] >= 0) {
        if (page[0] >= 0 && page[0] < a.num_pages)
          row = page[0] * a.page_size + token_row[0];
        else
          atomicExch(a.status, static_cast<int>(H3ATTN_ERR_INVALID_ARG));  // its keys are not attended
      }
      mask = __ballot_sync(0xFFFFFFFFu, row >= 0);
      if (SHARE > 1 && lane == 0) shared_mask[warp][at] = mask;
      const uint32_t ks = ring + at * (2 * C::kTileBytes), vs = ks + C::kTileBytes;
#pragma unroll
      for (int i = 0; i < TILE * CH / 32; ++i) {
        const int tr = (i * 32 + lane) / CH, col = lane % CH;
        const int src_row = __shfl_sync(0xFFFFFFFFu, row, tr);
        const int64_t off = max(src_row, 0) * row_stride;
        const uint32_t dst = tr * (D * 2) + ((col ^ (tr & 7)) << 4);
        cp_async16(ks + dst, kbase + off, src_row >= 0);
        cp_async16(vs + dst, vbase + off, src_row >= 0);
      }
      page[0] = page[1];
      token_row[0] = token_row[1];
      look_ahead(1);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) load(i, mask_of[i]);

  // The queries of a sequence as the second operand of the score product; where registers are left, those of the next
  // sequence are loaded while the present one is walked.
  const int g = lane >> 2, t = lane & 3;
  auto load_q = [&](int b, uint32_t (&qf)[NT][D / 16][2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool there = n * 8 + g < heads;
      const uint16_t* qp = a.q + (static_cast<int64_t>(b) * a.Hq + head0 + (there ? n * 8 + g : 0)) * D + 2 * t;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[n][ks][0] = there ? *reinterpret_cast<const uint32_t*>(qp + ks * 16) : 0u;
        qf[n][ks][1] = there ? *reinterpret_cast<const uint32_t*>(qp + ks * 16 + 8) : 0u;
      }
    }
  };
  constexpr bool AHEAD = NT == 1 && D <= 128;
  uint32_t q_next[AHEAD ? NT : 1][AHEAD ? D / 16 : 1][2];
  if constexpr (AHEAD) {
    int b1 = b0;
    while (p.ranges > 0 && seq_end(b1) < t1 && first_tile(b1) >= stop_tile(b1)) ++b1;
    load_q(b1, q_next);
  }

  int turn = 0;  // tiles used by this warp
  int b = b0;
  bool first_segment = true;
  while (true) {
    const int s0 = first_tile(b), s1 = stop_tile(b);
    if (s0 < s1 || p.ranges == 0) {
      // ---- one sequence's tiles [s0, s1) ----
      uint32_t qf[NT][D / 16][2];
      if constexpr (AHEAD) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            qf[n][ks][0] = q_next[n][ks][0];
            qf[n][ks][1] = q_next[n][ks][1];
          }
        int next = b + 1;  // the range's next sequence with a key, if there is one
        while (p.ranges > 0 && seq_end(next - 1) < t1 && first_tile(next) >= stop_tile(next)) ++next;
        if (p.ranges > 0 && seq_end(next - 1) < t1) load_q(next, q_next);
      } else {
        load_q(b, qf);
      }
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
      for (int tile = s0 + wt * SHARE; tile < s1; tile += p.WT * SHARE) {
        const int st = turn % STAGES;
        cp_async_wait<STAGES - 2>();
        if constexpr (SHARE > 1)
          pair_sync(1 + warp / SHARE);  // the peers' tiles are there, and what they read in the last turn is free
        else
          __syncwarp();
        const uint32_t mine = st == 0 ? mask_of[0] : st == 1 ? mask_of[1] : mask_of[2];
        {
          const int at = (turn + STAGES - 1) % STAGES;
          uint32_t fresh = 0;
          load(at, fresh);
#pragma unroll
          for (int i = 0; i < STAGES; ++i) mask_of[i] = i == at ? fresh : mask_of[i];
        }
        ++turn;
#pragma unroll 1
        for (int of = SHARE > 1 ? 0 : peer; of < SHARE; ++of) {
          const uint32_t mask = SHARE > 1 ? shared_mask[peer0 + of][st] : mine;
          // no such tile, or none of its keys is there (whose scores are kept as -infinity)
          if (SHARE > 1 && mask == 0 && !(W && tile + of < s1)) continue;
          const uint32_t ks_base = ring + ((of - peer) * STAGES + st) * (2 * C::kTileBytes);
          const uint32_t vs_base = ks_base + C::kTileBytes;
          // two accumulators a product: a chain of tensor-core products waits for each of its links
          float s[NT][MT][4], s2[NT][MT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[n][mt][e] = s2[n][mt][e] = 0.0f;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t kf[4];
              const int row = mt * 16 + (lane & 15), col = ks * 2 + (lane >> 4);
              ldmatrix4(kf, ks_base + row * (D * 2) + ((col ^ (row & 7)) << 4));
#pragma unroll
              for (int n = 0; n < NT; ++n) mma16816(ks & 1 ? s2[n][mt] : s[n][mt], kf, qf[n][ks][0], qf[n][ks][1]);
            }
          }
          // lane: tokens g and g + 8 of each 16, heads 2 t and 2 t + 1 of each 8
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[n][mt][e] += s2[n][mt][e];
          constexpr uint32_t kAll = TILE == 32 ? 0xFFFFFFFFu : 0xFFFFu;
          if ((mask & kAll) != kAll) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!((mask >> (mt * 16 + g + (e < 2 ? 0 : 8))) & 1u)) s[n][mt][e] = -INFINITY;
          }
          if constexpr (W) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int h = n * 8 + 2 * t + c;
                float* row = a.scores + (static_cast<int64_t>(b) * a.Hq + head0 + h) * a.score_stride + (tile + of) * TILE + g;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                  if (h < heads) {
                    row[mt * 16] = s[n][mt][c] * a.scale_log2;
                    row[mt * 16 + 8] = s[n][mt][c + 2] * a.scale_log2;
                  }
              }
          }
          uint32_t pf[NT][MT][2], pr[NT][MT][2];  // P and what its rounding left
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) top[e & 1] = fmaxf(top[e & 1], s[n][mt][e]);
            const bool over = top[0] * a.scale_log2 > m[n][0] + kSlack || top[1] * a.scale_log2 > m[n][1] + kSlack;
            if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 4));
                top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 8));
                top[c] = fmaxf(top[c], __shfl_xor_sync(0xFFFFFFFFu, top[c], 16));
                const float to = fmaxf(m[n][c], top[c] * a.scale_log2);
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
                s[n][mt][e] = ex2(fmaf(s[n][mt][e], a.scale_log2, -m[n][e & 1]));
                l[n][e & 1] += s[n][mt][e];
              }
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const float p0 = s[n][mt][2 * half], p1 = s[n][mt][2 * half + 1];
                const uint32_t hi = pack_bf16(p0, p1);
                pf[n][mt][half] = transpose8x8(hi);
                pr[n][mt][half] =
                    transpose8x8(pack_bf16(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xFFFF0000u)));
              }
            }
          }
          constexpr int DB = 4;  // channel tiles whose products are interleaved
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int d0 = 0; d0 < D / 16; d0 += DB) {
              uint32_t vf[DB][4];
#pragma unroll
              for (int i = 0; i < DB; ++i) {
                const int row = mt * 16 + (lane >> 4) * 8 + (lane & 7), col = (d0 + i) * 2 + ((lane >> 3) & 1);
                ldmatrix4_trans(vf[i], vs_base + row * (D * 2) + ((col ^ (row & 7)) << 4));
              }
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < DB; ++i) mma16816(o[n][d0 + i], vf[i], pf[n][mt][0], pf[n][mt][1]);
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < DB; ++i) mma16816(o[n][d0 + i], vf[i], pr[n][mt][0], pr[n][mt][1]);
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
        if (whole) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int h = n * 8 + 2 * t + c;
              if (h < heads) {
                const float inv = l[n][c] == 0.0f ? 0.0f : 1.0f / l[n][c];  // no key: zeros
                if (W && g == 0) a.stats[static_cast<int64_t>(b) * a.Hq + head0 + h] = make_float2(m[n][c], inv);
                __nv_bfloat16* op = reinterpret_cast<__nv_bfloat16*>(a.o) +
                                    (static_cast<int64_t>(b) * a.Hq + head0 + h) * D + g;
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                  op[dt * 16] = __float2bfloat16_rn(o[n][dt][c] * inv);
                  op[dt * 16 + 8] = __float2bfloat16_rn(o[n][dt][c + 2] * inv);
                }
              }
            }
        } else {
          // slot 0: the range's first sequence, slot 1: its last
          float* part = a.ws + ((static_cast<int64_t>(r) * 2 + (first_segment ? 0 : 1)) * p.unit_heads + unit) *
                                   partial_floats(min(G, C::kHeads), D);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int h = n * 8 + 2 * t + c;
              if (h < heads) {
                if (g == 0) {
                  part[2 * h] = m[n][c];
                  part[2 * h + 1] = l[n][c];
                }
                float* op = part + partial_o(min(G, C::kHeads)) + h * D + g;
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                  op[dt * 16] = o[n][dt][c];
                  op[dt * 16 + 8] = o[n][dt][c + 2];
                }
              }
            }
        }
      }
      first_segment = false;
    }
    if (p.ranges == 0 || seq_end(b) >= t1) break;
    ++b;
  }
  cp_async_wait<0>();
}

int warps_of(int D) { return D == 256 ? 4 : 8; }
int tile_of(int D) { return D == 64 ? 32 : 16; }
// 28 sequences of 0 to 52182 tokens, 32 heads to one of 128: 83 us without, 73 with; 64 of 0 to 6000, heads of 256: 86 and
// 75.  Neither the memory nor the tensor cores are full then (DRAM 68 %, tensor pipe 46 % busy; heads of 256 36 and 23 %):
// a sub-core has two warps, with heads of 256 one, and each is one chain of loads, products, softmax and products.
// Heads of 64, 9 sequences of 20000 to 40000: 22.9 without, 23.6 with (DRAM 40 %, tensor pipe 29 %).
int share_of(int D) { return D > 64 ? 2 : 1; }
DecodePlan plan_of(const DecodeArgs& a, int sms, bool split) {
  return make_plan(a, sms, split, warps_of(a.D), tile_of(a.D), 16, share_of(a.D), 4);
}

template <int D, int NT, int SHARE, bool W>
cudaError_t launch_d(const Kernelargs& k, cudaStream_t stream) {
  using C = DecodeCfg<D, NT>;
  static std::atomic<bool> attr_set[64];  // calls of several host threads
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(decode_kernel<D, NT, SHARE, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t ranges = k.p.ranges > 0 ? k.p.ranges : k.a.B;
  e = launch_dependent(decode_kernel<D, NT, SHARE, W>, dim3(static_cast<unsigned>(ranges * k.p.groups)), C::kWarps * 32,
                       C::kSmem, stream, k);
  if (e != cudaSuccess) return e;
  if (k.p.ranges == 0) return W ? launch_add_weights(k.a, stream) : e;
  const int G = k.a.Hq / k.a.Hkv;
  const int joins = k.p.ranges * k.p.groups;
  return launch_dependent(decode_join_kernel<D, W>, dim3(joins + (W ? adding_ctas(k.a, joins) : 0)), kJoinThreads, 0, stream, k,
                          C::kTile, std::min(G, C::kHeads), joins);
}

template <int D, bool W>
cudaError_t launch_heads(const Kernelargs& k, cudaStream_t stream) {
  if constexpr (D > 64)
    if (k.p.share == 2) return launch_d<D, 2, 2, W>(k, stream);
  return k.a.Hq / k.a.Hkv > 8 ? launch_d<D, 2, 1, W>(k, stream) : launch_d<D, 1, 1, W>(k, stream);
}
template <int D>
cudaError_t launch_weights(const Kernelargs& k, cudaStream_t stream) {
  return k.a.scores ? launch_heads<D, true>(k, stream) : launch_heads<D, false>(k, stream);
}

}  // namespace

cudaError_t decode_workspace(const DecodeArgs& a, size_t* bytes) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const DecodePlan p = plan_of(a, sms, true);
  const int heads = std::min(a.Hq / a.Hkv, 16);
  *bytes = static_cast<size_t>(p.ranges) * 2 * p.unit_heads * partial_floats(heads, a.D) * sizeof(float);
  return cudaSuccess;
}

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  Kernelargs k{plan_of(a, sms, a.ws != nullptr), a};
  switch (a.D) {
    case 64: return launch_weights<64>(k, stream);
    case 128: return launch_weights<128>(k, stream);
    case 256: return launch_weights<256>(k, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace h3
