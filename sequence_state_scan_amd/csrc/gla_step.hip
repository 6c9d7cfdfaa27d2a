// A few tokens of gated linear attention for each row of a batch, the rows' states in a pool:
//   S <- diag(exp(g_t)) S + k_t v_t^T,   o_t = S^T q_t,   t = 0 .. n-1
// The state is read and written once (8 dk dv bytes per row and head); everything else is small
// beside it, so the kernel is bound by HBM for many rows and by one memory round trip for few.
// A workgroup holds a tile of 16 VEC columns of one head's state in registers: lane (rg, cl) of
// the 16 x 16 lanes has rows rg + 16 i and VEC adjacent columns, so that a row of the tile is one
// 256-byte access of 16 lanes.  o sums over the rows: within a lane, over the 4 row groups of a
// wave by lane exchange, over the 4 waves through LDS.
#include "gla_block.hpp"

namespace gla {

template <typename E, int RPT, int VEC>
__global__ __launch_bounds__(256) void step_kernel(StepArgs a) {
  constexpr int TC = 16 * VEC;
  const int tiles = (a.dv + TC - 1) / TC;
  const int ct = blockIdx.x % tiles;
  const int bh = blockIdx.x / tiles, b = bh / a.H, h = bh - b * a.H;
  const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int j = ct * TC + cl * VEC;
  const bool col = j < a.dv;
  E* o = (E*)a.o + (long)bh * a.n * a.dv + j;
  const int slot = row_slot(a.slots, b, a.n_slots);
  if (slot < 0) {
    float fill[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) fill[v] = slot == -1 ? 0.f : __builtin_nanf("");
    if (col)
      for (int t = rg; t < a.n; t += 16) store_row<E, VEC>(o + (long)t * a.dv, fill);
    return;
  }
  float* st = a.state + ((long)slot * a.H + h) * a.dk * a.dv + j;
  float S[RPT][VEC];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + 16 * i;
    if (col && r < a.dk) load_row<float, VEC>(st + (long)r * a.dv, S[i]);
    else
#pragma unroll
      for (int v = 0; v < VEC; ++v) S[i][v] = 0.f;
  }
  __shared__ float red[4][TC];
  const E* q = (const E*)a.q + b * a.qs.b + h * a.qs.h;
  const E* k = (const E*)a.k + b * a.ks.b + h * a.ks.h;
  const E* vp = (const E*)a.v + b * a.vs.b + h * a.vs.h + j;
  const float* g = a.g + b * a.gs.b + h * a.gs.h;
  for (int t = 0; t < a.n; ++t) {
    float vv[VEC], acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) vv[v] = acc[v] = 0.f;
    if (col) load_row<E, VEC>(vp + t * a.vs.t, vv);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + 16 * i;
      if (r < a.dk) {
        const float at = decay(g[t * a.gs.t + r]), kt = (float)k[t * a.ks.t + r], qt = (float)q[t * a.qs.t + r];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          S[i][v] = advance(at, S[i][v], kt * vv[v]);
          acc[v] = fmaf(qt, S[i][v], acc[v]);
        }
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      acc[v] += __shfl_xor(acc[v], 16);
      acc[v] += __shfl_xor(acc[v], 32);
    }
    if (t) __syncthreads();  // the last token's sums are read
    if ((threadIdx.x & 63) < 16)
#pragma unroll
      for (int v = 0; v < VEC; ++v) red[wave][cl * VEC + v] = acc[v];
    __syncthreads();
    if (threadIdx.x < 16 && col) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int e = cl * VEC + v;
        acc[v] = (red[0][e] + red[1][e]) + (red[2][e] + red[3][e]);
      }
      store_row<E, VEC>(o + (long)t * a.dv, acc);
    }
  }
  if (col)
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + 16 * i;
      if (r < a.dk) store_row<float, VEC>(st + (long)r * a.dv, S[i]);
    }
}

template <typename E, int VEC>
static void step_rows(const StepArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * a.H * ((a.dv + 16 * VEC - 1) / (16 * VEC)));
  const int rpt = (a.dk + 15) / 16;
  if (rpt <= 1) step_kernel<E, 1, VEC><<<grid, 256, 0, s>>>(a);
  else if (rpt <= 2) step_kernel<E, 2, VEC><<<grid, 256, 0, s>>>(a);
  else if (rpt <= 4) step_kernel<E, 4, VEC><<<grid, 256, 0, s>>>(a);
  else if (rpt <= 8) step_kernel<E, 8, VEC><<<grid, 256, 0, s>>>(a);
  else step_kernel<E, 16, VEC><<<grid, 256, 0, s>>>(a);
}

static bool aligned(const void* p, const Strides& st, int bytes, int n) {
  const auto u = (unsigned long long)p;
  return u % bytes == 0 && st.b % n == 0 && st.h % n == 0 && st.t % n == 0;
}

// Four columns a lane where v's rows, o's and the state's allow it, one otherwise.
hipError_t launch_step(const StepArgs& a, hipStream_t s) {
  const int e = a.dtype == GLA_BF16 ? 2 : 4;
  const bool wide = a.dv % 4 == 0 && (uintptr_t)a.state % 16 == 0 && (uintptr_t)a.o % (4 * e) == 0 &&
                    aligned(a.v, a.vs, 4 * e, 4);
  if (a.dtype == GLA_BF16) {
    if (wide) step_rows<bf16, 4>(a, s);
    else step_rows<bf16, 1>(a, s);
  } else {
    if (wide) step_rows<float, 4>(a, s);
    else step_rows<float, 1>(a, s);
  }
  return hipGetLastError();
}

}  // namespace gla
