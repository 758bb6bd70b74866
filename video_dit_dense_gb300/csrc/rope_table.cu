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
// signed angle of at most an eighth of a turn, is converted to float32 with
// its leading bits intact.
//
// Bound by the stores: 8 bytes for each sine and cosine pair.
#include "generate.h"

namespace h3 {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void sincos_turn(uint64_t phase, float* s, float* c) {
  const uint32_t quadrant = static_cast<uint32_t>((phase + (1ull << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quadrant) << 62));
  float sn, cs;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &sn, &cs);  // 2 * turns = angle / pi
  const float a = (quadrant & 1) ? cs : sn, b = (quadrant & 1) ? sn : cs;
  *s = (quadrant & 2) ? -a : a;
  *c = ((quadrant + 1) & 2) ? -b : b;
}

// A thread keeps VEC neighbouring pairs of a row and walks down the rows, so
// that their phase steps stay in registers.
template <int VEC>
__global__ void __launch_bounds__(kThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int per_row = a.half / VEC;  // <= kMaxRotaryPairs < kThreads
  const int rows = kThreads / per_row;
  const int col = threadIdx.x % per_row, lane_row = threadIdx.x / per_row;
  if (lane_row >= rows) return;
  uint64_t turn[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) turn[e] = a.turn[col * VEC + e];
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  for (int64_t n = static_cast<int64_t>(blockIdx.x) * rows + lane_row; n < a.N; n += step) {
    const int64_t p = a.pos ? static_cast<int64_t>(a.pos[n]) : a.first + n;
    float c[VEC], s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      sincos_turn(static_cast<uint64_t>(p) * turn[e], &s[e], &c[e]);
      c[e] *= a.amplitude;
      s[e] *= a.amplitude;
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
  if (blocks > sms * 8) blocks = sms * 8;  // 2048 threads an SM
  const dim3 grid(static_cast<unsigned>(blocks));
  return vec == 4 ? launch_dependent(rope_table_kernel<4>, grid, kThreads, 0, stream, a)
                  : launch_dependent(rope_table_kernel<1>, grid, kThreads, 0, stream, a);
}

}  // namespace h3
