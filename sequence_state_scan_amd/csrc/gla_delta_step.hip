// A few tokens of the gated delta rule for each row of a batch, the rows' states in a pool:
//   A = exp(g_t) S,   e = v_t - A^T k_t,   S <- A + beta_t k_t e^T,   o_t = S^T q_t = A^T q_t + beta_t (k_t . q_t) e
// The state is read and written once (8 dk dv bytes per row and head), in registers between: a workgroup holds 16 VEC
// columns, lane (rg, cl) of its 16 x 16 lanes rows rg + 16 i and VEC adjacent columns.  Both sums over the rows
// (A^T k, A^T q) are taken at once, within a lane, over a wave's 4 row groups by lane exchange and over the 4 waves
// through LDS, so that a token costs one barrier.  Bound by HBM for many rows (bf16, 128 rows of 16 heads of 128 x 128: 53 us,
// 5.1 TB/s), by one memory round trip and the sums for few (one row of 4 such heads: 5.8 us).
#include "gla_delta.hpp"

namespace gla {

template <typename E, int RPT, int VEC>
__global__ __launch_bounds__(256) void delta_step_kernel(DeltaStepArgs a) {
  constexpr int TC = 16 * VEC;
  const int tiles = (a.dv + TC - 1) / TC;
  const int ct = blockIdx.x % tiles;
  const int bh = blockIdx.x / tiles, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
  const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  const int j = ct * TC + cl * VEC;
  const bool col = j < a.dv;
  E* o = (E*)a.o + (long)bh * a.n * a.dv + j;
  const int slot = row_slot(a.slots, b, a.n_slots);
  float* st = a.state + ((long)slot * a.H + h) * a.dk * a.dv + j;
  const E* q = (const E*)a.q + b * a.qs.b + hk * a.qs.h;
  const E* k = (const E*)a.k + b * a.ks.b + hk * a.ks.h;
  const E* vp = (const E*)a.v + b * a.vs.b + h * a.vs.h + j;
  const float* g = a.g + b * a.gs.b + h * a.gs.h;
  const float* beta = a.beta + b * a.bs.b + h * a.bs.h;
  // a token's inputs, loaded a token ahead; the first one's with the state, before the slot is checked against the
  // earlier rows'
  float vv[VEC], kt[RPT], qt[RPT], gt, bt;
  const auto load_token = [&](int t) {
    gt = g[t * a.gs.t];
    bt = beta[t * a.bs.t];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + 16 * i;
      kt[i] = qt[i] = 0.f;
      if (r < a.dk) {
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
  __shared__ float red[2][4][2 * TC + 1];  // a wave's A^T k, A^T q and k . q
  for (int t = 0; t < a.n; ++t) {
    const float at = decay(gt);
    float pk[VEC], pq[VEC], kq = 0.f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) pk[v] = pq[v] = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      kq = fmaf(kt[i], qt[i], kq);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        S[i][v] = pass(at, S[i][v]);
        pk[v] = fmaf(kt[i], S[i][v], pk[v]);
        pq[v] = fmaf(qt[i], S[i][v], pq[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      pk[v] += __shfl_xor(pk[v], 16);
      pq[v] += __shfl_xor(pq[v], 16);
      pk[v] += __shfl_xor(pk[v], 32);
      pq[v] += __shfl_xor(pq[v], 32);
    }
    kq += __shfl_xor(kq, 16);
    kq += __shfl_xor(kq, 32);
    float(&sums)[4][2 * TC + 1] = red[t & 1];  // in turn: the barrier of the token between is behind every read
    if ((threadIdx.x & 63) < 16) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        sums[wave][cl * VEC + v] = pk[v];
        sums[wave][TC + cl * VEC + v] = pq[v];
      }
      if (cl == 0) sums[wave][2 * TC] = kq;
    }
    __syncthreads();
    const auto total = [&](int e) { return (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]); };
    float e[VEC], kr[RPT];
#pragma unroll
    for (int v = 0; v < VEC; ++v) e[v] = bt * (vv[v] - total(cl * VEC + v));
    if (threadIdx.x < 16 && col) {
      const float all = total(2 * TC);
      float out[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) out[v] = fmaf(all, e[v], total(TC + cl * VEC + v));
      store_row<E, VEC>(o + (long)t * a.dv, out);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) kr[i] = kt[i];
    if (t + 1 < a.n) load_token(t + 1);
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) S[i][v] = rg + 16 * i < a.dk ? fmaf(kr[i], e[v], S[i][v]) : 0.f;
  }
  if (col)
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = rg + 16 * i;
      if (r < a.dk) store_stream<float, VEC>(st + (long)r * a.dv, S[i]);
    }
}

template <typename E, int VEC>
static void delta_step_rows(const DeltaStepArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((long long)a.B * a.H * ((a.dv + 16 * VEC - 1) / (16 * VEC)));
  if (a.dk <= 32) delta_step_kernel<E, 2, VEC><<<grid, 256, 0, s>>>(a);
  else if (a.dk <= 64) delta_step_kernel<E, 4, VEC><<<grid, 256, 0, s>>>(a);
  else if (a.dk <= 128) delta_step_kernel<E, 8, VEC><<<grid, 256, 0, s>>>(a);
  else delta_step_kernel<E, 16, VEC><<<grid, 256, 0, s>>>(a);
}

// Four columns a lane where v's rows, o's and the state's allow it, one otherwise.
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s) {
  const int e = a.dtype == GLA_BF16 ? 2 : 4;
  const bool wide = a.dv % 4 == 0 && (uintptr_t)a.state % 16 == 0 && (uintptr_t)a.o % (4 * e) == 0 &&
                    (uintptr_t)a.v % (4 * e) == 0 && a.vs.b % 4 == 0 && a.vs.h % 4 == 0 && a.vs.t % 4 == 0;
  if (a.dtype == GLA_BF16) {
    if (wide) delta_step_rows<bf16, 4>(a, s);
    else delta_step_rows<bf16, 1>(a, s);
  } else {
    if (wide) delta_step_rows<float, 4>(a, s);
    else delta_step_rows<float, 1>(a, s);
  }
  return hipGetLastError();
}

}  // namespace gla
