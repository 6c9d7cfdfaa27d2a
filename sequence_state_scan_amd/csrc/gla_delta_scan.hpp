// The chain over the segments of a sequence, both directions (gla_delta_fwd.hip, gla_delta_bwd.hip).
#pragma once
#include "gla_delta.hpp"

namespace gla {
namespace delta {

// S <- M S + S_own over the segments; backward from the last segment with M transposed, from the gradient of the last
// state.  A workgroup has 32 columns of a head, a wave of it 16 rows of the state: its rows of the next M and of S_own
// are on their way while the waves exchange the state as the product's operand through LDS, one barrier a step.
template <typename E, int DK, bool BWD>
__global__ __launch_bounds__(4 * DK) void delta_scan_kernel(DeltaArgs a) {
  constexpr int CP = DK / 32, PARTS = Num<E>::PARTS, COLS = 2;
  typedef Tile<E, DK> T;  // [column][row of the state]
  __shared__ __attribute__((aligned(16))) E Ss[2][PARTS][16 * COLS * T::LD];
  const int heads = a.B * a.H, bh = blockIdx.x % heads, b = bh / a.H, lane = lane_id(), n16 = lane & 15, g4 = lane >> 4;
  const int cb = wave_id(), j0 = blockIdx.x / heads * 16 * COLS, r0 = row4_of(cb, g4);
  const int alive = (length_of(a, b) + C - 1) / C, steps = max(1, (alive + a.L - 1) / a.L) - 1;
  const long tiles = a.DVP / 16, plane = (long)heads * a.P * DK * DK;
  const float* from = BWD ? a.dhT : a.h0;
  const E* mp = (const E*)(BWD ? a.trans : a.trans_rows) + (long)bh * a.P * DK * DK + row_of(cb, n16) * DK + 8 * g4;
  const auto place = [&](int seg, int c) { return (((long)bh * a.P + seg) * tiles + j0 / 16 + c) * DK * 16 + cb * 256 + lane * 4; };
  const auto have = [&](int c) { return j0 + 16 * c < a.dv; };
  f32x4 S[COLS], own[COLS];
  Split<E> M[CP];
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = j0 + 16 * c + n16;
      S[c][i] = from && r0 + i < a.dk && col < a.dv ? from[((long)bh * a.dk + r0 + i) * a.dv + col] : 0.f;
    }
  const auto load = [&](int step) {
    const int seg = BWD ? steps - step : step;
#pragma unroll
    for (int p = 0; p < CP; ++p)
#pragma unroll
      for (int part = 0; part < PARTS; ++part) M[p].part[part] = *reinterpret_cast<const Frag<E>*>(mp + part * plane + (long)seg * DK * DK + 32 * p);
#pragma unroll
    for (int c = 0; c < COLS; ++c) own[c] = have(c) ? *reinterpret_cast<const f32x4*>(a.seg + place(seg, c)) : zero4();
  };
  if (steps > 0) load(0);
  for (int step = 0; step < steps; ++step) {
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      if (have(c)) *reinterpret_cast<f32x4*>(a.seg_in + place(BWD ? steps - step : step, c)) = S[c];
      f32x4 x = S[c];
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        T::put4(Ss[step & 1][part], 16 * c + n16, r0, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] -= (float)(E)x[i];
      }
    }
    __syncthreads();  // (the other half is free: every wave has read it before this barrier's last pass)
#pragma unroll
    for (int c = 0; c < COLS; ++c) S[c] = own[c];
#pragma unroll
    for (int p = 0; p < CP; ++p)
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        Split<E> s;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) s.part[part] = T::row(Ss[step & 1][part], 16 * c + n16, 32 * p + 8 * g4);
        S[c] = mma<E>(M[p], s, S[c]);
      }
    if (step + 1 < steps) load(step + 1);
  }
#pragma unroll
  for (int c = 0; c < COLS; ++c)
    if (have(c)) *reinterpret_cast<f32x4*>(a.seg_in + place(BWD ? 0 : steps, c)) = S[c];
}

}  // namespace delta
}  // namespace gla
