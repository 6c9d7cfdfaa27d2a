// A few tokens of gated linear attention for each row of a batch, the rows' states in a pool:
//   S <- diag(exp(g_t)) S + k_t v_t^T,   o_t = S^T q_t,   t = 0 .. n-1
// The state is read and written once (8 dk dv bytes per row and head); everything else is small
// beside it, so the kernel is bound by HBM for many rows and by one memory round trip for few.  Of several
// tokens each adds its row sums and a barrier: 128 rows of 16 heads of 128 x 128 bf16 take 55 us for one
// token, 81 for 4, 127 for 8.
// A workgroup holds a tile of 16 VEC columns of one head's state in registers: lane (rg, cl) of
// the 16 x 16 lanes has rows rg + 16 i and VEC adjacent columns, so that a row of the tile is one
// 256-byte access of 16 lanes.  o sums over the rows: within a lane, over the 4 row groups of a
// wave by lane exchange, over the 4 waves through LDS.
// The state goes past the caches: a layer's states come back only a whole model's states later.
// Measured over enough states of 16 heads of 128 x 128 that none is still cached, us a call: 1 row
// 5.05 (cached accesses 5.46), 8 rows 5.98 (7.63), 32 rows 13.99 (18.45), 256 rows 96.7 (112.8, 5.6
// TB/s); where the same states do come back at once, cached accesses win between 32 rows (11.2
// against 13.1) and 96 (33.5 against 36.8).  Tiles of 128 columns measured the same, of 256 half
// as slow again.
#include "gla_block.hpp"

namespace gla {

// FULL: dk is 16 RPT, there are no rows past it (the selection that keeps those at zero is what several
// tokens a call would notice: 32 rows x 8 heads of 64 x 128, 8 tokens 16.3 us with it, 16.1 without).
template <typename E, int RPT, int VEC, bool FULL>
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
  float* st = a.state + ((long)slot * a.H + h) * a.dk * a.dv + j;
  const E* q = (const E*)a.q + b * a.qs.b + h * a.qs.h;
  const E* k = (const E*)a.k + b * a.ks.b + h * a.ks.h;
  const E* vp = (const E*)a.v + b * a.vs.b + h * a.vs.h + j;
  const float* g = a.g + b * a.gs.b + h * a.gs.h;
  // a token's inputs, loaded a token ahead; the first one's with the state, before the slot is checked
  // against the earlier rows'
  float vv[VEC], gt[RPT], kt[RPT], qt[RPT];
  const auto load_token = [&](int t) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + 16 * i;
      gt[i] = kt[i] = qt[i] = 0.f;
      if (r < a.dk) {
        gt[i] = g[t * a.gs.t + r];
        kt[i] = (float)k[t * a.ks.t + r];
        qt[i] = (float)q[t * a.qs.t + r];
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) vv[v] = 0.f;
    if (col) load_row<E, VEC>(vp + t * a.vs.t, vv);
  };
  load_token(0);
  float S[RPT][VEC];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = rg + 16 * i;
#pragma unroll
    for (int v = 0; v < VEC; ++v) S[i][v] = 0.f;
    if (slot >= 0 && col && r < a.dk) load_stream<float, VEC>(st + (long)r * a.dv, S[i]);
  }
  if (slot < 0 || slot_taken(a.slots, b, slot)) {
    float fill[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) fill[v] = slot == -1 ? 0.f : __builtin_nanf("");
    if (col)
      for (long t = rg; t < a.n; t += 16) store_row<E, VEC>(o + t * a.dv, fill);  // t + 16 may pass 2^31
    return;
  }
  __shared__ float red[2][4][TC];
  for (int t = 0; t < a.n; ++t) {
    float acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float at = decay(gt[i]);
      const bool row = FULL || rg + 16 * i < a.dk;  // rows past dk stay zero, also where v is infinite or NaN
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        S[i][v] = row ? advance(at, S[i][v], kt[i] * vv[v]) : 0.f;
        acc[v] = fmaf(qt[i], S[i][v], acc[v]);
      }
    }
    if (t + 1 < a.n) load_token(t + 1);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      acc[v] += __shfl_xor(acc[v], 16);
      acc[v] += __shfl_xor(acc[v], 32);
    }
    float(&sums)[4][TC] = red[t & 1];  // in turn: the barrier of the token between is behind every read
    if ((threadIdx.x & 63) < 16)
#pragma unroll
      for (int v = 0; v < VEC; ++v) sums[wave][cl * VEC + v] = acc[v];
    __syncthreads();
    if (threadIdx.x < 16 && col) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int e = cl * VEC + v;
        acc[v] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
      }
      store_row<E, VEC>(o + (long)t * a.dv, acc);
    }
  }
  if (col)
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + 16 * i;
      if (r < a.dk) store_stream<float, VEC>(st + (long)r * a.dv, S[i]);
    }
}

template <typename E, int RPT, int VEC>
static void step_tile(const StepArgs& a, unsigned grid, hipStream_t s) {
  if (a.dk == 16 * RPT) step_kernel<E, RPT, VEC, true><<<grid, 256, 0, s>>>(a);
  else step_kernel<E, RPT, VEC, false><<<grid, 256, 0, s>>>(a);
}

template <typename E, int VEC>
static void step_rows(const StepArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * a.H * ((a.dv + 16 * VEC - 1) / (16 * VEC)));
  if (a.dk <= 16) step_tile<E, 1, VEC>(a, grid, s);
  else if (a.dk <= 32) step_tile<E, 2, VEC>(a, grid, s);
  else if (a.dk <= 64) step_tile<E, 4, VEC>(a, grid, s);
  else if (a.dk <= 128) step_tile<E, 8, VEC>(a, grid, s);
  else step_tile<E, 16, VEC>(a, grid, s);
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
