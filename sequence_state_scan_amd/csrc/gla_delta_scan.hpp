// The chain over the segments of a sequence, both directions (gla_delta_fwd.hip, gla_delta_bwd.hip).
#pragma once
#include "gla_delta.hpp"

namespace gla {
namespace delta {

// S <- M S + S_own over the segments, 16 NW columns of a head a workgroup; backward from the last segment with M
// transposed, from the gradient of the last state.
template <typename E, int DK, int NW, bool BWD>
__global__ __launch_bounds__(64 * NW) void delta_scan_kernel(DeltaArgs a) {
  constexpr int NT = 64 * NW, CB = DK / 16, CP = DK / 32, PARTS = Num<E>::PARTS, LD = ld_of<E>(DK);
  __shared__ __attribute__((aligned(16))) E Ms[PARTS][DK * LD];
  const int heads = a.B * a.H, bh = blockIdx.x % heads, b = bh / a.H, lane = lane_id(), n16 = lane & 15, g4 = lane >> 4;
  const int j = (blockIdx.x / heads * NW + wave_id()) * 16;
  const bool cols = j < a.dv;
  const int alive = (length_of(a, b) + C - 1) / C, live = max(1, (alive + a.L - 1) / a.L);
  const long tiles = a.DVP / 16;
  const auto place = [&](int seg) { return (((long)bh * a.P + seg) * tiles + j / 16) * DK * 16; };
  const float* from = BWD ? a.dhT : a.h0;
  f32x4 S[CB];
  load_state<CB>(S, from ? from + (long)bh * a.dk * a.dv : nullptr, a.dk, a.dv, cols ? j + n16 : a.dv);
  const E* mp = (const E*)a.trans + (long)bh * a.P * DK * DK;
  const long mplane = (long)heads * a.P * DK * DK;
  TileIn<E, DK, DK, NT> min_[PARTS];
  const auto load = [&](int step) {
#pragma unroll
    for (int part = 0; part < PARTS; ++part)
      min_[part].load(mp + part * mplane + (long)(BWD ? live - 1 - step : step) * DK * DK, DK, DK, DK);
  };
  const int steps = live - 1;
  if (steps > 0) load(0);
  for (int step = 0; step < steps; ++step) {
    const int seg = BWD ? live - 1 - step : step;
    if (cols) store_regs<CB>(S, a.seg_in + place(seg));
    f32x4 own[CB];
    if (cols) load_regs<CB>(own, a.seg + place(seg));
    __syncthreads();
#pragma unroll
    for (int part = 0; part < PARTS; ++part) min_[part].store(Ms[part], LD);
    __syncthreads();
    if (step + 1 < steps) load(step + 1);
    Split<E> So[CP];
#pragma unroll
    for (int p = 0; p < CP; ++p) So[p] = split<E>(S[2 * p], S[2 * p + 1]);
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      f32x4 acc = cols ? own[cb] : zero4();
#pragma unroll
      for (int p = 0; p < CP; ++p) {
        Split<E> M;
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
          M.part[part] = BWD ? row_frag(Ms[part] + row_of(cb, n16) * LD + 32 * p + 8 * g4)
                             : col_frag<E, true>(Ms[part], LD, 32 * p, row4_of(cb, 0));
        acc = mma<E>(M, So[p], acc);
      }
      S[cb] = acc;
    }
  }
  if (cols) store_regs<CB>(S, a.seg_in + place(BWD ? 0 : live - 1));
}

}  // namespace delta
}  // namespace gla
