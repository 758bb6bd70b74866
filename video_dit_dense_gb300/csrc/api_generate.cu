// C-ABI entry points of the generation operators: residual add + RMSNorm,
// rotary tables, append to a paged cache, decode attention.  Argument
// validation and error mapping; nothing is allocated, and all work is
// enqueued on the caller's stream.
#include <math.h>
#include <stdint.h>

#include "api_common.h"
#include "generate.h"

using h3::aligned16;
using h3::check_device;
using h3::head_dim_ok;
using h3::overlap;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Span {
  const void* p;
  int64_t bytes;
};
bool overlaps_any(const Span& out, const Span* others, int n) {
  for (int i = 0; i < n; ++i)
    if (out.p && others[i].p && out.bytes > 0 && others[i].bytes > 0 &&
        overlap(out.p, out.bytes, others[i].p, others[i].bytes))
      return true;
  return false;
}

// 2^64 / (2 pi) as the sum of two doubles, hi + lo: the turns of one radian
// in units of 2^-64 turn.
constexpr double kTurnHi = 0x1.45f306dc9c883p+61;
constexpr double kTurnLo = -0x1.6b01ec5417056p+7;

// f radians (0 <= f <= 1) as a binary fraction of a turn, rounded to 2^-64:
// f * (hi + lo) with the product's rounding error kept.
uint64_t turn_fraction(double f) {
  const double p = f * kTurnHi;
  const double err = fma(f, kTurnHi, -p) + f * kTurnLo;
  const double whole = floor(p);
  return static_cast<uint64_t>(whole) + static_cast<uint64_t>(static_cast<int64_t>(llrint((p - whole) + err)));
}

// Geometry of a paged cache (its pointers apart).
h3attn_status_t check_cache(const h3attn_paged_kv_t* c) {
  if (!c || c->B < 0 || c->B > 65535 || c->Hkv < 1 || c->Hkv > 65535) return H3ATTN_ERR_INVALID_ARG;
  if (!head_dim_ok(c->D)) return H3ATTN_ERR_UNSUPPORTED_HEAD_DIM;
  if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1) return H3ATTN_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c->num_pages) * c->page_size > INT32_MAX ||
      static_cast<int64_t>(c->max_pages) * c->page_size > INT32_MAX - 63)
    return H3ATTN_ERR_INVALID_ARG;
  return H3ATTN_OK;
}
h3attn_status_t check_cache_pointers(const h3attn_paged_kv_t* c) {
  if (!c->k_pages || !c->v_pages || !c->page_table || !c->kv_len) return H3ATTN_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned4(c->page_table) || !aligned4(c->kv_len))
    return H3ATTN_ERR_MISALIGNED;
  return H3ATTN_OK;
}
int64_t page_bytes(const h3attn_paged_kv_t* c) {
  return static_cast<int64_t>(c->num_pages) * c->page_size * c->Hkv * c->D * 2;
}

void decode_fields(h3::DecodeArgs* a, const h3attn_paged_kv_t* c, int Hq) {
  a->k_pages = static_cast<const uint16_t*>(c->k_pages);
  a->v_pages = static_cast<const uint16_t*>(c->v_pages);
  a->page_table = c->page_table;
  a->kv_len = c->kv_len;
  a->B = c->B;
  a->Hq = Hq;
  a->Hkv = c->Hkv;
  a->D = c->D;
  a->page_size = c->page_size;
  a->max_pages = c->max_pages;
  a->num_pages = c->num_pages;
  a->div_page = h3::make_fastdiv(static_cast<uint32_t>(c->page_size));
}

// Head counts of a decode call: whole groups, and work units in 32 bits.
h3attn_status_t check_decode_heads(const h3attn_paged_kv_t* c, int Hq) {
  if (Hq < 1 || Hq > 65535 || Hq % c->Hkv != 0) return H3ATTN_ERR_INVALID_ARG;
  if (static_cast<int64_t>(c->B) * c->Hkv * ((Hq / c->Hkv + 15) / 16) > INT32_MAX) return H3ATTN_ERR_INVALID_ARG;
  return H3ATTN_OK;
}

}  // namespace

extern "C" {

h3attn_status_t h3attn_add_rmsnorm(const void* x, const void* residual, void* h, void* y, const float* w,
                                   void* y_scale, int T, int C, int y_format, float eps, h3attn_stream_t stream) {
  if (T < 0 || C < 8 || C % 8 != 0 || C > h3::kAddNormMaxChannels) return H3ATTN_ERR_INVALID_ARG;
  if (y_format != H3ATTN_Y_BF16 && y_format != H3ATTN_Y_E4M3_ROW && y_format != H3ATTN_Y_E4M3_MX32)
    return H3ATTN_ERR_INVALID_ARG;
  if (y_format == H3ATTN_Y_E4M3_MX32 && C % 32 != 0) return H3ATTN_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps)) return H3ATTN_ERR_INVALID_ARG;
  if (T == 0) return H3ATTN_OK;
  if (!x || !y || (residual == nullptr) != (h == nullptr)) return H3ATTN_ERR_INVALID_ARG;
  if ((y_scale == nullptr) != (y_format == H3ATTN_Y_BF16)) return H3ATTN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || (residual && (!aligned16(residual) || !aligned16(h))) || (w && !aligned16(w)) ||
      (y_format == H3ATTN_Y_E4M3_ROW && !aligned4(y_scale)))
    return H3ATTN_ERR_MISALIGNED;
  const int64_t n = static_cast<int64_t>(T) * C, rows = 2 * n;
  const int64_t ny = y_format == H3ATTN_Y_BF16 ? rows : n;
  const int64_t ns = y_format == H3ATTN_Y_BF16 ? 0 : y_format == H3ATTN_Y_E4M3_ROW ? 4LL * T : n / 32;
  // an output may be x or residual itself (each thread reads its elements before it writes them): bf16 only
  const bool y_in = y_format == H3ATTN_Y_BF16;
  const Span sx{x, rows}, sr{residual, rows}, sh{h, rows}, sy{y, ny}, sw{w, 4LL * C}, ss{y_scale, ns};
  const Span none{nullptr, 0};
  const Span of_h[] = {h == x ? none : sx, h == residual ? none : sr, sy, sw, ss};
  const Span of_y[] = {y_in && y == x ? none : sx, y_in && y == residual ? none : sr, sw, ss};
  const Span of_s[] = {sx, sr, sw};
  if (overlaps_any(sh, of_h, 5) || overlaps_any(sy, of_y, 4) || overlaps_any(ss, of_s, 3)) return H3ATTN_ERR_INVALID_ARG;
  h3attn_status_t st = check_device();
  if (st != H3ATTN_OK) return st;
  h3::AddNormArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.residual = static_cast<const uint16_t*>(residual);
  a.h = static_cast<uint16_t*>(h);
  a.y = y;
  a.w = w;
  a.y_scale = y_scale;
  a.T = T;
  a.C = C;
  a.format = y_format;
  a.eps = eps;
  a.inv_C = 1.0f / static_cast<float>(C);
  return h3::launch_add_rmsnorm(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? H3ATTN_OK : H3ATTN_ERR_LAUNCH;
}

h3attn_status_t h3attn_rope_table(float* cos, float* sin, const int32_t* pos, int64_t first, int N, int rotary_dim,
                                  double theta, const h3attn_rope_scaling_t* scaling, h3attn_stream_t stream) {
  if (N < 0 || rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > 2 * h3::kMaxRotaryPairs)
    return H3ATTN_ERR_INVALID_ARG;
  if (!(theta >= 1.0) || !isfinite(theta)) return H3ATTN_ERR_INVALID_ARG;
  if (pos ? first != 0 : (first < 0 || first > (1LL << 31) - N)) return H3ATTN_ERR_INVALID_ARG;
  const int kind = scaling ? scaling->kind : static_cast<int>(H3ATTN_ROPE_NONE);
  if (kind < H3ATTN_ROPE_NONE || kind > H3ATTN_ROPE_BY_PARTS) return H3ATTN_ERR_INVALID_ARG;
  const double factor = kind == H3ATTN_ROPE_NONE ? 1.0 : scaling->factor;
  const double amplitude = scaling ? scaling->amplitude : 1.0;
  if (!(factor >= 1.0) || !isfinite(factor)) return H3ATTN_ERR_INVALID_ARG;
  const float amp = static_cast<float>(amplitude);
  if (!(amp > 0.0f) || !isfinite(amp)) return H3ATTN_ERR_INVALID_ARG;
  if (kind == H3ATTN_ROPE_NTK && rotary_dim < 4) return H3ATTN_ERR_INVALID_ARG;
  if (kind == H3ATTN_ROPE_BY_PARTS &&
      (scaling->original_len < 1 || !(scaling->low_turns >= 0.0) || !(scaling->high_turns > scaling->low_turns) ||
       !isfinite(scaling->high_turns)))
    return H3ATTN_ERR_INVALID_ARG;
  if (N == 0) return H3ATTN_OK;
  if (!cos || !sin) return H3ATTN_ERR_INVALID_ARG;
  if (!aligned16(cos) || !aligned16(sin) || (pos && !aligned4(pos))) return H3ATTN_ERR_MISALIGNED;
  const int half = rotary_dim / 2;
  const int64_t bytes = static_cast<int64_t>(N) * half * 4;
  const Span sc{cos, bytes}, ss{sin, bytes}, sp{pos, 4LL * N};
  const Span of_c[] = {ss, sp}, of_s[] = {sp};
  if (overlaps_any(sc, of_c, 2) || overlaps_any(ss, of_s, 1)) return H3ATTN_ERR_INVALID_ARG;
  double base = theta;
  if (kind == H3ATTN_ROPE_NTK) base = theta * pow(factor, rotary_dim / (rotary_dim - 2.0));
  if (!isfinite(base)) return H3ATTN_ERR_INVALID_ARG;
  h3attn_status_t st = check_device();
  if (st != H3ATTN_OK) return st;
  h3::RopeTableArgs a;
  for (int i = 0; i < half; ++i) {
    double f = pow(base, -2.0 * i / rotary_dim);
    if (kind == H3ATTN_ROPE_LINEAR) f /= factor;
    if (kind == H3ATTN_ROPE_BY_PARTS) {
      const double turns = scaling->original_len * f / 6.283185307179586;
      const double keep = fmin(fmax((turns - scaling->low_turns) / (scaling->high_turns - scaling->low_turns), 0.0), 1.0);
      f = (1.0 - keep) * (f / factor) + keep * f;
    }
    a.turn[i] = turn_fraction(f);
  }
  for (int i = half; i < h3::kMaxRotaryPairs; ++i) a.turn[i] = 0;
  a.cos = cos;
  a.sin = sin;
  a.pos = pos;
  a.first = first;
  a.N = N;
  a.half = half;
  a.amplitude = amp;
  return h3::launch_rope_table(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? H3ATTN_OK : H3ATTN_ERR_LAUNCH;
}

h3attn_status_t h3attn_qk_norm_rope_append(const void* q, const void* k, const void* v, void* q_out,
                                           const h3attn_paged_kv_t* cache, const float* wq, const float* wk,
                                           const float* cos, const float* sin, const int32_t* pos,
                                           const int32_t* new_len, int32_t* len_out, int S, int Hq, int64_t q_stride,
                                           int64_t k_stride, int64_t v_stride, int table_rows, int rotary_dim,
                                           int interleaved, float eps, h3attn_stream_t stream) {
  h3attn_status_t st = check_cache(cache);
  if (st != H3ATTN_OK) return st;
  const int B = cache->B, Hkv = cache->Hkv, D = cache->D;
  if (S < 0 || Hq < 0 || Hq > 65535) return H3ATTN_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 2 != 0 || table_rows < 0) return H3ATTN_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !isfinite(eps)) return H3ATTN_ERR_INVALID_ARG;
  const int64_t tokens = static_cast<int64_t>(B) * S;
  if (tokens == 0 && (!len_out || B == 0)) return H3ATTN_OK;  // before the pointers: empty tensors have none
  if (tokens == 0) {
    // no token, but the lengths are asked for: they stay, in len_out
    q = k = v = q_out = nullptr;
    wq = wk = cos = sin = nullptr;
    pos = nullptr;
    Hq = rotary_dim = 0;
    q_stride = k_stride = v_stride = static_cast<int64_t>(Hkv) * D;
  }
  if ((q == nullptr) != (Hq == 0) || (q_out == nullptr) != (q == nullptr)) return H3ATTN_ERR_INVALID_ARG;
  if (tokens > INT32_MAX || tokens * (Hq + 2LL * Hkv) > INT32_MAX) return H3ATTN_ERR_INVALID_ARG;
  if ((tokens > 0 && (!k || !v)) || (wq && !q)) return H3ATTN_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!cos || !sin)) return H3ATTN_ERR_INVALID_ARG;
  if (k_stride < static_cast<int64_t>(Hkv) * D || v_stride < static_cast<int64_t>(Hkv) * D ||
      (q && q_stride < static_cast<int64_t>(Hq) * D))
    return H3ATTN_ERR_INVALID_ARG;
  const int64_t most = INT64_MAX / 4 / (tokens > 0 ? tokens : 1);
  if (k_stride > most || v_stride > most || (q && q_stride > most)) return H3ATTN_ERR_INVALID_ARG;
  st = check_cache_pointers(cache);
  if (st != H3ATTN_OK) return st;
  if (!aligned16(k) || !aligned16(v) || (q && (!aligned16(q) || !aligned16(q_out))) || (wq && !aligned16(wq)) ||
      (wk && !aligned16(wk)) || (cos && !aligned16(cos)) || (sin && !aligned16(sin)) || (pos && !aligned4(pos)) ||
      (new_len && !aligned4(new_len)) || (len_out && !aligned4(len_out)))
    return H3ATTN_ERR_MISALIGNED;
  if (k_stride % 8 != 0 || v_stride % 8 != 0 || (q && q_stride % 8 != 0)) return H3ATTN_ERR_MISALIGNED;
  // spans of the inputs, and of the outputs, none of which may meet another
  const int64_t np = page_bytes(cache);
  const Span sq{q, ((tokens - 1) * q_stride + static_cast<int64_t>(Hq) * D) * 2};
  const Span sk{k, ((tokens - 1) * k_stride + static_cast<int64_t>(Hkv) * D) * 2};
  const Span sv{v, ((tokens - 1) * v_stride + static_cast<int64_t>(Hkv) * D) * 2};
  const Span so{q_out, tokens * Hq * D * 2}, kp{cache->k_pages, np}, vp{cache->v_pages, np};
  const Span sl{len_out, 4LL * B}, kl{cache->kv_len, 4LL * B}, nl{new_len, 4LL * B}, sp{pos, 4 * tokens};
  const Span pt{cache->page_table, 4LL * B * cache->max_pages};
  const int64_t tb = 2LL * rotary_dim * table_rows;
  const Span sc{cos, tb}, ss{sin, tb}, swq{wq, 4LL * D}, swk{wk, 4LL * D}, none{nullptr, 0};
  const bool in_place = q_out == q && q_stride == static_cast<int64_t>(Hq) * D;
  const Span of_o[] = {in_place ? none : sq, sk, sv, kp, vp, sl, kl, nl, sp, pt, sc, ss, swq, swk};
  const Span of_k[] = {vp, sq, sk, sv, sl, kl, nl, sp, pt, sc, ss, swq, swk};
  const Span of_l[] = {kl, nl, sp, pt, sq, sk, sv, sc, ss, swq, swk};
  if (overlaps_any(so, of_o, 14) || overlaps_any(kp, of_k, 13) || overlaps_any(vp, of_k + 1, 12) ||
      overlaps_any(sl, of_l, 11))
    return H3ATTN_ERR_INVALID_ARG;
  st = check_device();
  if (st != H3ATTN_OK) return st;
  h3::AppendArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_pages = static_cast<uint16_t*>(cache->k_pages);
  a.v_pages = static_cast<uint16_t*>(cache->v_pages);
  a.page_table = cache->page_table;
  a.kv_len = cache->kv_len;
  a.wq = wq;
  a.wk = wk;
  a.cos = cos;
  a.sin = sin;
  a.pos = pos;
  a.new_len = new_len;
  a.len_out = len_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.tokens = static_cast<uint32_t>(tokens);
  a.div_s = h3::make_fastdiv(static_cast<uint32_t>(S > 0 ? S : 1));
  a.div_page = h3::make_fastdiv(static_cast<uint32_t>(cache->page_size));
  a.B = B;
  a.S = S;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.page_size = cache->page_size;
  a.max_pages = cache->max_pages;
  a.num_pages = cache->num_pages;
  a.table_rows = table_rows;
  a.rotary_dim = rotary_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.eps = eps;
  a.status = h3::status_word_ptr();
  if (!a.status) return H3ATTN_ERR_LAUNCH;
  return h3::launch_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? H3ATTN_OK : H3ATTN_ERR_LAUNCH;
}

h3attn_status_t h3attn_paged_decode_workspace_size(const h3attn_paged_kv_t* cache, int Hq, size_t* bytes) {
  if (!bytes) return H3ATTN_ERR_INVALID_ARG;
  *bytes = 0;
  h3attn_status_t st = check_cache(cache);
  if (st != H3ATTN_OK) return st;
  st = check_decode_heads(cache, Hq);
  if (st != H3ATTN_OK) return st;
  if (cache->B == 0) return H3ATTN_OK;
  st = check_device();
  if (st != H3ATTN_OK) return st;
  h3::DecodeArgs a;
  decode_fields(&a, cache, Hq);
  return h3::decode_workspace(a, bytes) == cudaSuccess ? H3ATTN_OK : H3ATTN_ERR_LAUNCH;
}

h3attn_status_t h3attn_paged_decode(const void* q, void* o, const h3attn_paged_kv_t* cache, int Hq, float scale,
                                    void* workspace, size_t workspace_bytes, h3attn_stream_t stream) {
  h3attn_status_t st = check_cache(cache);
  if (st != H3ATTN_OK) return st;
  st = check_decode_heads(cache, Hq);
  if (st != H3ATTN_OK) return st;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(scale > 0.0f) || !isfinite(scale_log2)) return H3ATTN_ERR_INVALID_ARG;
  if (cache->B == 0) return H3ATTN_OK;
  if (!q || !o) return H3ATTN_ERR_INVALID_ARG;
  st = check_cache_pointers(cache);
  if (st != H3ATTN_OK) return st;
  if (!aligned16(q) || !aligned16(o) || (workspace && !aligned16(workspace))) return H3ATTN_ERR_MISALIGNED;
  const int64_t nq = static_cast<int64_t>(cache->B) * Hq * cache->D * 2, np = page_bytes(cache);
  const Span so{o, nq};
  const Span inputs[] = {{q, nq},
                         {cache->k_pages, np},
                         {cache->v_pages, np},
                         {cache->kv_len, 4LL * cache->B},
                         {cache->page_table, 4LL * cache->B * cache->max_pages},
                         {o, nq}};
  if (overlaps_any(so, inputs, 5)) return H3ATTN_ERR_INVALID_ARG;
  st = check_device();
  if (st != H3ATTN_OK) return st;
  h3::DecodeArgs a;
  decode_fields(&a, cache, Hq);
  a.ws = nullptr;
  if (workspace) {
    size_t need = 0;
    if (h3::decode_workspace(a, &need) != cudaSuccess) return H3ATTN_ERR_LAUNCH;
    if (workspace_bytes < need || overlaps_any({workspace, static_cast<int64_t>(need)}, inputs, 6))
      return H3ATTN_ERR_INVALID_ARG;
    if (need > 0) a.ws = static_cast<float*>(workspace);
  }
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.scale_log2 = scale_log2;
  a.status = h3::status_word_ptr();
  if (!a.status) return H3ATTN_ERR_LAUNCH;
  return h3::launch_decode(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? H3ATTN_OK : H3ATTN_ERR_LAUNCH;
}

}  // extern "C"
