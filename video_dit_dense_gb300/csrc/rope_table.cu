// Rotary tables cos(p f_i), sin(p f_i) for any positions p and for scaled
// frequencies.
//
// The angle of a far position has more bits than float32 (p f_0 = 2^20 rad
// leaves 2^-4 rad in a float), and double-precision arithmetic is slow on
// this GPU.  So an angle is kept in turns, as a 64-bit binary fraction: with
// u_i = round(2^64 f_i / 2 pi) (host, double-double), the phase of position
// p is p * u_i mod 2^64, exact integer arithmetic that drops whole turns by
// itself, off by at most |p| / 2 units of 2^-64 turn (2^-34 turn at 2^31).
// The two top bits (after adding an eighth) name the quadrant; the rest, a
// signed angle x of at most an eighth of a turn, is rounded to float32 once,
// small ones with all their bits, and its sine and cosine are the Taylor
// polynomials of sin(2 pi x) and cos(2 pi x), whose next terms are below
// 2^-28 and 2^-32 there.
//
// Bound by the stores, 8 bytes for each sine and cosine, as long as the
// arithmetic takes less than 40 instructions a pair: the phase is two 32-bit
// multiplications, and the polynomials run on two pairs at a time (packed
// float32 operations).  524291 rows of 64 pairs: 39 us, 6.9 TB/s (66 us
// with the library's sincospif); the values are 3.6e-8 off, where rounding
// alone leaves 2.7e-8.  A row whose pairs are no multiple of 4 is not 16-byte
// aligned: then a thread keeps one pair, stores 4 bytes at a time and evaluates it twice,
// 524291 rows of 23 pairs 24 us (14 at the copy rate), of 65, where a
// quarter of the threads has no pair, 120 us (40).
#include "generate.h"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;

// sin(2 pi x) = sum kSin[k] x^(2 k + 1) and cos(2 pi x) = 1 + sum kCos[k] x^(2 k + 2): (2 pi)^n / n! with alternating
// signs; the first of the sine's is in two parts.
constexpr double k2Pi = 6.283185307179586;
constexpr double power2pi(int n) { return n == 0 ? 1.0 : power2pi(n - 1) * k2Pi / n; }  // (2 pi)^n / n!
// The angle of position p: its quadrant, and the rest in turns.
__device__ __forceinline__ float reduce(int p, uint64_t turn, uint32_t& quadrant) {
  const uint32_t pu = static_cast<uint32_t>(p), t_lo = static_cast<uint32_t>(turn), t_hi = static_cast<uint32_t>(turn >> 32);
  const uint64_t low = static_cast<uint64_t>(pu) * t_lo;
  uint32_t hi = static_cast<uint32_t>(low >> 32) + pu * t_hi;
  if (p < 0) hi -= t_lo;  // pu is p + 2^32
  quadrant = (hi + (1u << 29)) >> 30;
  const int rest = static_cast<int>(hi - (quadrant << 30));
  return fmaf(static_cast<float>(static_cast<uint32_t>(low)), 0x1p-64f, static_cast<float>(rest) * 0x1p-32f);
}

// Sines and cosines of two angles (in turns, at most an eighth), scaled.
__device__ __forceinline__ void sincos2(const float (&x)[2], const uint32_t (&quadrant)[2], float amplitude, float* sn, float* cs) {
  constexpr float kSinHi = static_cast<float>(power2pi(1));
  constexpr float kSinLo = static_cast<float>(power2pi(1) - static_cast<double>(kSinHi));
  constexpr float kSin[4] = {static_cast<float>(-power2pi(3)), static_cast<float>(power2pi(5)),
                             static_cast<float>(-power2pi(7)), static_cast<float>(power2pi(9))};
  constexpr float kCos[5] = {static_cast<float>(-power2pi(2)), static_cast<float>(power2pi(4)),
                             static_cast<float>(-power2pi(6)), static_cast<float>(power2pi(8)),
                             static_cast<float>(-power2pi(10))};
  float z0, z1, s0, s1, c0, c1, t0, t1;
  fmul2(z0, z1, x[0], x[1], x[0], x[1]);
  s0 = s1 = kSin[3];
  c0 = c1 = kCos[4];
#pragma unroll
  for (int k = 2; k >= 0; --k) ffma2(s0, s1, s0, s1, z0, z1, kSin[k], kSin[k]);
#pragma unroll
  for (int k = 3; k >= 0; --k) ffma2(c0, c1, c0, c1, z0, z1, kCos[k], kCos[k]);
  ffma2(c0, c1, c0, c1, z0, z1, 1.0f, 1.0f);
  ffma2(s0, s1, s0, s1, z0, z1, kSinLo, kSinLo);
  fmul2(t0, t1, s0, s1, x[0], x[1]);
  ffma2(s0, s1, x[0], x[1], kSinHi, kSinHi, t0, t1);
  fmul2(s0, s1, s0, s1, amplitude, amplitude);
  fmul2(c0, c1, c0, c1, amplitude, amplitude);
  const float s[2] = {s0, s1}, c[2] = {c0, c1};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // a quarter turn more: sine from cosine, cosine from minus sine
    const bool odd = quadrant[i] & 1;
    const float a = odd ? c[i] : s[i], b = odd ? s[i] : c[i];
    sn[i] = __uint_as_float(__float_as_uint(a) ^ ((quadrant[i] & 2) << 30));
    cs[i] = __uint_as_float(__float_as_uint(b) ^ (((quadrant[i] + 1) & 2) << 30));
  }
}

// A thread keeps VEC neighbouring pairs of a row and walks down the rows, so
// that their phase steps stay in registers.
template <int VEC>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  // What the launch alone gives is read before the wait on the previous kernel.
  const int per_row = a.half / VEC;  // <= kMaxRotaryPairs < kThreads
  const int rows = kThreads / per_row;
  const int col = threadIdx.x % per_row, lane_row = threadIdx.x / per_row;
  uint64_t turn[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) turn[e] = a.turn[col * VEC + e];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (lane_row >= rows) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  int64_t n = static_cast<int64_t>(blockIdx.x) * rows + lane_row;
  int p_next = a.pos && n < a.N ? a.pos[n] : 0;
  for (; n < a.N; n += step) {
    const int p = a.pos ? p_next : static_cast<int>(a.first + n);
    if (a.pos && n + step < a.N) p_next = a.pos[n + step];
    constexpr int PAIRS = VEC == 1 ? 2 : VEC;  // the polynomials take two at a time
    float x[PAIRS], c[PAIRS], s[PAIRS];
    uint32_t q[PAIRS];
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) x[e] = reduce(p, turn[VEC == 1 ? 0 : e], q[e]);
#pragma unroll
    for (int e = 0; e < PAIRS; e += 2) {
      const float x2[2] = {x[e], x[e + 1]};
      const uint32_t q2[2] = {q[e], q[e + 1]};
      sincos2(x2, q2, a.amplitude, s + e, c + e);
    }
    const int64_t at = n * a.half + col * VEC;
    if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(a.cos + at) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(a.sin + at) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      a.cos[at] = c[0];
      a.sin[at] = s[0];
    }
  }
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int vec = a.half % 4 == 0 ? 4 : 1;
  const int rows = kThreads / (a.half / vec);
  int64_t blocks = (static_cast<int64_t>(a.N) + rows - 1) / rows;
  if (blocks > sms * 6) blocks = sms * 6;  // as many as 40 registers a thread let stay
  const dim3 grid(static_cast<unsigned>(blocks));
  return vec == 4 ? launch_dependent(rope_table_kernel<4>, grid, kThreads, 0, stream, a)
                  : launch_dependent(rope_table_kernel<1>, grid, kThreads, 0, stream, a);
}

}  // namespace h3
