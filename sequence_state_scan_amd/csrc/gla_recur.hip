// The elementwise gated linear recurrence, per sequence b and channel c:
//   h_t = a_t h_{t-1} + beta(g_t) x_t,  a = exp(g),  beta = 1 | 1 - a | sqrt(1 - a^2)
// and its backward.  One lane owns a channel and walks the tokens.
#include "gla_block.hpp"

namespace gla {

__device__ __forceinline__ int seq_len(const RecurArgs& a, int b) {
  if (!a.lens) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

template <typename E, int MODE>
__global__ __launch_bounds__(64) void recur_fwd_kernel(RecurArgs a) {
  const int c = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
  if (c >= a.D) return;
  const int len = seq_len(a, b);
  const long nch = (a.T + kRecurChunk - 1) / kRecurChunk;
  const E* x = (const E*)a.x + b * a.xs.b + c;
  const float* g = a.g + b * a.gs.b + c;
  E* h = (E*)a.h + (long)b * a.T * a.D + c;
  float s = a.h0 ? a.h0[(long)b * a.D + c] : 0.f;
  for (int t = 0; t < a.T; ++t) {
    if (a.chunk_in && t % kRecurChunk == 0) a.chunk_in[(b * nch + t / kRecurChunk) * a.D + c] = s;
    if (t < len) {
      const float gt = g[t * a.gs.t], at = decay(gt);
      s = advance(at, s, input_factor<MODE>(gt, at) * (float)x[t * a.xs.t]);
    }
    h[(long)t * a.D] = (E)(t < len ? s : 0.f);
  }
  if (a.h_final) a.h_final[(long)b * a.D + c] = s;
}

template <typename E, int MODE>
__global__ __launch_bounds__(64) void recur_bwd_kernel(RecurArgs a) {
  const int c = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
  if (c >= a.D) return;
  const int len = seq_len(a, b);
  const int nch = (a.T + kRecurChunk - 1) / kRecurChunk;
  const E* x = (const E*)a.x + b * a.xs.b + c;
  const float* g = a.g + b * a.gs.b + c;
  const E* dh = (const E*)a.dh + b * a.dhs.b + c;
  E* dx = (E*)a.h + (long)b * a.T * a.D + c;
  float* dg = a.dg + (long)b * a.T * a.D + c;
  float carry = a.dhT ? a.dhT[(long)b * a.D + c] : 0.f;  // a_{t+1} D_{t+1}
  constexpr int R = 16;
  for (int n = nch - 1; n >= 0; --n) {
    float lead[kRecurChunk / R];  // state entering each run of R tokens
    float s = a.chunk_in[((long)b * nch + n) * a.D + c];
    const int t0 = n * kRecurChunk;
    for (int i = 0; i < kRecurChunk; ++i) {
      if (i % R == 0) lead[i / R] = s;
      const int t = t0 + i;
      if (t < len) {
        const float gt = g[t * a.gs.t], at = decay(gt);
        s = advance(at, s, input_factor<MODE>(gt, at) * (float)x[t * a.xs.t]);
      }
    }
    for (int r = kRecurChunk / R - 1; r >= 0; --r) {
      float before[R];
      s = lead[r];
      for (int i = 0; i < R; ++i) {
        const int t = t0 + r * R + i;
        before[i] = s;
        if (t < len) {
          const float gt = g[t * a.gs.t], at = decay(gt);
          s = advance(at, s, input_factor<MODE>(gt, at) * (float)x[t * a.xs.t]);
        }
      }
      for (int i = R - 1; i >= 0; --i) {
        const int t = t0 + r * R + i;
        if (t >= a.T) continue;
        float vx = 0.f, vg = 0.f;
        if (t < len) {
          const float gt = g[t * a.gs.t], at = decay(gt), be = input_factor<MODE>(gt, at), xt = (float)x[t * a.xs.t];
          const float d = carry + (float)dh[t * a.dhs.t];
          vx = be * d;
          vg = at == 0.f ? 0.f : at * before[i] * d;
          vg = fmaf(input_factor_slope<MODE>(at, be) * xt, d, vg);
          carry = at == 0.f ? 0.f : at * d;
        }
        dx[(long)t * a.D] = (E)vx;
        dg[(long)t * a.D] = vg;
      }
    }
  }
  if (a.h_final) a.h_final[(long)b * a.D + c] = carry;
}

#define GLA_RECUR_DISPATCH(KERNEL, A, GRID, BLOCK, S)                                              \
  do {                                                                                             \
    if ((A).dtype == GLA_BF16) {                                                                   \
      if ((A).mode == GLA_RECUR_PLAIN) KERNEL<bf16, GLA_RECUR_PLAIN><<<GRID, BLOCK, 0, S>>>(A);    \
      else if ((A).mode == GLA_RECUR_LERP) KERNEL<bf16, GLA_RECUR_LERP><<<GRID, BLOCK, 0, S>>>(A); \
      else KERNEL<bf16, GLA_RECUR_NORM><<<GRID, BLOCK, 0, S>>>(A);                                 \
    } else {                                                                                       \
      if ((A).mode == GLA_RECUR_PLAIN) KERNEL<float, GLA_RECUR_PLAIN><<<GRID, BLOCK, 0, S>>>(A);   \
      else if ((A).mode == GLA_RECUR_LERP) KERNEL<float, GLA_RECUR_LERP><<<GRID, BLOCK, 0, S>>>(A);\
      else KERNEL<float, GLA_RECUR_NORM><<<GRID, BLOCK, 0, S>>>(A);                                \
    }                                                                                              \
  } while (0)

hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s) {
  GLA_RECUR_DISPATCH(recur_fwd_kernel, a, dim3((a.D + 63) / 64, a.B), dim3(64), s);
  return hipGetLastError();
}

hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s) {
  GLA_RECUR_DISPATCH(recur_bwd_kernel, a, dim3((a.D + 63) / 64, a.B), dim3(64), s);
  return hipGetLastError();
}

// One token for each row of a batch, the rows' states in a pool.  Every workgroup (64 channels of
// one row) looks its slot up and checks it against the earlier rows' by itself.
template <typename E, int MODE>
__global__ __launch_bounds__(64) void recur_step_kernel(RecurStepArgs a) {
  const int c = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
  const int slot = row_slot(a.slots, b, a.n_slots);
  if (c >= a.D) return;
  E* h = (E*)a.h + (long)b * a.D + c;
  if (slot < 0) {
    *h = (E)(slot == -1 ? 0.f : __builtin_nanf(""));
    return;
  }
  const float g = a.g[b * a.gs.b + c], at = decay(g);
  float* st = a.state + (long)slot * a.D + c;
  const float s = advance(at, *st, input_factor<MODE>(g, at) * (float)((const E*)a.x)[b * a.xs.b + c]);
  *st = s;
  *h = (E)s;
}

hipError_t launch_recur_step(const RecurStepArgs& a, hipStream_t s) {
  GLA_RECUR_DISPATCH(recur_step_kernel, a, dim3((a.D + 63) / 64, a.B), dim3(64), s);
  return hipGetLastError();
}

}  // namespace gla
