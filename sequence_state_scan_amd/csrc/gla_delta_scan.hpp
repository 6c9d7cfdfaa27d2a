// The chain over the segments of a sequence, both directions (gla_delta_fwd.hip, gla_delta_bwd.hip).
#pragma once
#include "gla_delta.hpp"

namespace gla {
namespace delta {

// S <- M S + S_own over the segments; backward from the last segment with M transposed, from the gradient of the last
// state.  A workgroup has 32 columns of a head, a wave of it 16 rows of the state: the waves exchange the state as the
// product's operand through LDS, one barrier a step, while their rows of the next M and S_own are on their way, AHEAD
// steps before their use.  What bounds a step is issuing the loads of M, 64 KB a CU, so M lies in the order of its
// operands and a load takes whole lines (31 steps of 4 heads of 128 x 256: 39 us; by rows, 16 half lines a load, 66, and
// with 16 or 64 columns a workgroup 64 and 118).
template <typename E, int DK, bool BWD>
__global__ __launch_bounds__(4 * DK) void delta_scan_kernel(DeltaArgs a) {
  constexpr int CP = DK / 32, PARTS = Num<E>::PARTS, COLS = 2, AHEAD = 2;
  typedef Tile<E, DK> T;  // [column][row of the state]
  __shared__ __attribute__((aligned(16))) E Ss[2][PARTS][16 * COLS * T::LD];
  const int heads = a.B * a.H, bh = blockIdx.x % heads, b = bh / a.H, lane = lane_id(), n16 = lane & 15, g4 = lane >> 4;
  const int cb = wave_id(), j0 = blockIdx.x / heads * 16 * COLS, r0 = row4_of(cb, g4);
  const int alive = (length_of(a, b) + C - 1) / C, steps = max(1, (alive + a.L - 1) / a.L) - 1;
  const long tiles = a.DVP / 16, plane = (long)heads * a.P * DK * DK;
  const float* from = BWD ? a.dhT : a.h0;
  const E* mp = (const E*)(BWD ? a.trans : a.trans_rows) + (long)bh * a.P * DK * DK + cb * CP * 512 + lane * 8;
  // (a column tile behind the last: the last's place and the last's values)
  const auto place = [&](int seg, int c) { return (((long)bh * a.P + seg) * tiles + min(j0 / 16 + c, (int)tiles - 1)) * DK * 16 + cb * 256 + lane * 4; };
  f32x4 S[COLS], own[AHEAD][COLS];
  Split<E> M[AHEAD][CP];
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int col = min(j0 + 16 * c, a.DVP - 16) + n16;
      S[c][i] = from && r0 + i < a.dk && col < a.dv ? from[((long)bh * a.dk + r0 + i) * a.dv + col] : 0.f;
    }
  if (!BWD && starts_anew(a, b, bh - b * a.H, alive))
#pragma unroll
    for (int c = 0; c < COLS; ++c) S[c] = zero4();
  arrived<COLS>(S);
  const auto load = [&](int step, Split<E> (&m)[CP], f32x4 (&o)[COLS]) {  // every step loads, the last ones again
    const int at = min(step, steps - 1), seg = BWD ? steps - at : at;
#pragma unroll
    for (int p = 0; p < CP; ++p)
#pragma unroll
      for (int part = 0; part < PARTS; ++part) m[p].part[part] = *reinterpret_cast<const Frag<E>*>(mp + part * plane + (long)seg * DK * DK + p * 512);
#pragma unroll
    for (int c = 0; c < COLS; ++c) o[c] = *reinterpret_cast<const f32x4*>(a.seg + place(seg, c));
  };
  if (steps > 0) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      load(k, M[k], own[k]);
      batch<E>();  // in the order of their use
    }
  }
  const auto advance = [&](int step, const Split<E> (&m)[CP], const f32x4 (&o)[COLS]) {
#pragma unroll
    for (int c = 0; c < COLS; ++c) {
      *reinterpret_cast<f32x4*>(a.seg_in + place(BWD ? steps - step : step, c)) = S[c];
      f32x4 x = S[c];
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        T::put4(Ss[step & 1][part], 16 * c + n16, r0, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] -= (float)(E)x[i];
      }
    }
    __syncthreads();  // (the other half is free: every wave has read it before the barrier after)
    Split<E> s[CP][COLS];
#pragma unroll
    for (int p = 0; p < CP; ++p)
#pragma unroll
      for (int c = 0; c < COLS; ++c)
#pragma unroll
        for (int part = 0; part < PARTS; ++part) s[p][c].part[part] = T::row(Ss[step & 1][part], 16 * c + n16, 32 * p + 8 * g4);
    batch<E>();
#pragma unroll
    for (int c = 0; c < COLS; ++c) S[c] = o[c];
#pragma unroll
    for (int p = 0; p < CP; ++p) mma_tiles<E, 0, COLS, PARTS, PARTS, COLS, true>(S, s[p], m[p]);
    batch<E>();
  };
  int step = 0;
  for (; step + AHEAD <= steps; step += AHEAD)  // (whole rounds: a way out of one would make every round wait for all loads)
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      advance(step + k, M[k], own[k]);
      load(step + k + AHEAD, M[k], own[k]);
      batch<E>();
    }
#pragma unroll
  for (int k = 0; k < AHEAD - 1; ++k)
    if (step + k < steps) advance(step + k, M[k], own[k]);
#pragma unroll
  for (int c = 0; c < COLS; ++c)
    *reinterpret_cast<f32x4*>(a.seg_in + place(BWD ? 0 : steps, c)) = S[c];
}

}  // namespace delta
}  // namespace gla
