// Shared by the recurrent-block operators (gla_recur.hip, gla_step.hip, gla_join.hip) and their
// host side (gla_block_api.cpp): argument blocks, launchers, and on the device the row loads.
#pragma once
#include <hip/hip_runtime_api.h>

#include "gla.h"

namespace gla {

constexpr int kRecurChunk = 128;  // tokens between the states gla_recur_fwd keeps (GLA_RECUR_CHUNK)
constexpr int kRecurTile = 256;   // tokens of a scan's tile where there are several
// Token strides and D of the recurrence stay below this, so that 32 tokens span less than 2^31 bytes.
constexpr int kMaxStride = 1 << 24;
constexpr int kStepMaxDk = 256;   // key rows a gla_step workgroup can hold
constexpr int kJoinMaxRow = 8192; // H * d a gla_join row may have
constexpr int kJoinMaxHeads = 2048;  // and heads: a head takes a slot of its own however narrow it is

struct Strides {  // in elements; the last dimension is contiguous
  long long b, h, t;
};

struct RecurArgs {
  const void* x;
  const float* g;
  const void* dh;         // backward: gradient of h
  const float* h0;        // [B][D] or null
  const int* lens;        // [B] or null
  void* h;                // forward [B][T][D]; backward: dx
  float* chunk_in;        // [B][chunks][D]: written by the forward (may be null), read by the backward
  float* h_final;         // [B][D] or null; backward: dh0
  const float* dhT;       // backward: [B][D] or null
  float* dg;              // backward [B][T][D]
  unsigned long long* words;  // the workspace; in the kernels, the tiles' words (null for one tile)
  unsigned* ticket;
  Strides xs, gs, dhs;
  int B, T, D, mode, dtype;
};

struct RecurStepArgs {
  const void* x;
  const float* g;
  float* state;  // [n_slots][D]
  const int* slots;
  void* h;
  Strides xs, gs;
  int B, D, n_slots, mode, dtype;
};

struct StepArgs {
  const void *q, *k, *v;
  const float* g;
  float* state;  // [n_slots][H][dk][dv]
  const int* slots;
  void* o;       // [B][H][n][dv]
  Strides qs, ks, vs, gs;
  int B, H, n, dk, dv, n_slots, dtype;
};

struct JoinArgs {
  const void *y, *z, *residual;
  const float *w_post, *scale, *w_pre;
  void *out, *normed;
  float *rstd_post, *rstd_pre;  // [B][T][H], [B][T]
  // backward
  const void *d_out, *d_normed;
  void *dy, *dz, *d_residual;
  float *dw_post, *dscale, *dw_pre;
  float* partial;
  Strides ys, zs, rs, dos, dns;
  int B, H, T, d, act, dtype, stream_dtype;
  float eps;
};

hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s);
hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s);
size_t recur_workspace_words(int B, int T, int D);  // 8-byte words both need
hipError_t launch_recur_step(const RecurStepArgs& a, hipStream_t s);
hipError_t launch_step(const StepArgs& a, hipStream_t s);
hipError_t launch_join_fwd(const JoinArgs& a, hipStream_t s);
hipError_t launch_join_bwd(const JoinArgs& a, hipStream_t s);
size_t join_partial_floats(int B, int H, int T, int d);  // workspace of launch_join_bwd

}  // namespace gla

#ifdef __HIPCC__
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gla {

typedef __bf16 bf16;

// N elements at p (aligned to min(16, their size) when N > 1) as floats, and back: one 16-byte
// access per 8 bf16 or 4 floats.
template <typename E, int N>
struct Vec {
  typedef E raw __attribute__((ext_vector_type(N), aligned(N * sizeof(E) < 16 ? N * sizeof(E) : 16)));
};
template <typename E, int N>
__device__ __forceinline__ void load_row(const E* p, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = (float)p[0];
  } else {
    typename Vec<E, N>::raw r = *reinterpret_cast<const typename Vec<E, N>::raw*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (float)r[i];
  }
}
template <typename E, int N>
__device__ __forceinline__ void store_row(E* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    p[0] = (E)v[0];
  } else {
    typename Vec<E, N>::raw r;
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = (E)v[i];
    *reinterpret_cast<typename Vec<E, N>::raw*>(p) = r;
  }
}

// The same for data that one pass reads or writes once and no cache should keep.
template <typename E, int N>
__device__ __forceinline__ void load_stream(const E* p, float (&v)[N]) {
  const auto r = __builtin_nontemporal_load(reinterpret_cast<const typename Vec<E, N>::raw*>(p));
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (float)r[i];
}
template <typename E, int N>
__device__ __forceinline__ void store_stream(E* p, const float (&v)[N]) {
  typename Vec<E, N>::raw r;
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = (E)v[i];
  __builtin_nontemporal_store(r, reinterpret_cast<typename Vec<E, N>::raw*>(p));
}

// exp(g) through the hardware's base-2 exponential; exp(-inf) = 0.
__device__ __forceinline__ float decay(float g) { return __builtin_amdgcn_exp2f(g * 1.44269504088896340736f); }

// 1 - exp(g) for g <= 0 without cancellation: the Taylor series of exp(g) - 1 to the 8th power
// near zero (its next term is below 2^-24 of the sum for |g| <= 0.5), the difference elsewhere
// (exp(g) is then below 0.61, so the difference loses at most one bit).  a = exp(g).
__device__ __forceinline__ float one_minus_decay(float g, float a) {
  float p = fmaf(g, 1.f / 40320.f, 1.f / 5040.f);
  p = fmaf(p, g, 1.f / 720.f);
  p = fmaf(p, g, 1.f / 120.f);
  p = fmaf(p, g, 1.f / 24.f);
  p = fmaf(p, g, 1.f / 6.f);
  p = fmaf(p, g, 0.5f);
  p = fmaf(p, g, 1.f);
  return g > -0.5f ? -g * p : 1.f - a;
}

// The factor of the recurrence's input, beta(g), for a = exp(g).
template <int MODE>
__device__ __forceinline__ float input_factor(float g, float a) {
  if constexpr (MODE == GLA_RECUR_PLAIN) return 1.f;
  if constexpr (MODE == GLA_RECUR_LERP) return one_minus_decay(g, a);
  return __builtin_amdgcn_sqrtf(one_minus_decay(2.f * g, a * a));  // the instruction's: one step off at most
}
// Its derivative by g (zero where the norm's factor is zero, at g = 0).  The plain factor has none.
template <int MODE>
__device__ __forceinline__ float input_factor_slope(float a, float beta) {
  if constexpr (MODE == GLA_RECUR_LERP) return -a;
  return beta > 0.f ? -a * a * __builtin_amdgcn_rcpf(beta) : 0.f;
}

// a * h and a * h + b, where a decay of zero (a reset, or an underflow) drops h whatever it holds.
__device__ __forceinline__ float pass(float a, float h) { return a == 0.f ? 0.f : a * h; }
__device__ __forceinline__ float advance(float a, float h, float b) { return a == 0.f ? b : fmaf(a, h, b); }

// Slot of row b: the row itself without slots, -1 for a row that is left out (a negative slot), -2
// for a slot outside the pool.
__device__ __forceinline__ int row_slot(const int* slots, int b, int n_slots) {
  const int s = slots ? slots[b] : b;
  return s < 0 ? -1 : s >= n_slots ? -2 : s;
}
// Whether an earlier row of the call names row b's slot.  Every lane of the wave calls it; apart from
// row_slot, so that the row's loads are on their way meanwhile.  Every wave reads b slots, which needs no
// workspace and no order of the rows: 0.8 us of 5.7 at 256 rows of 4096, but quadratic (16384 rows of 256:
// 50 of 63 us).
__device__ __forceinline__ bool slot_taken(const int* slots, int b, int slot) {
  if (!slots || slot < 0) return false;
  bool dup = false;
  for (int i = threadIdx.x & 63; i < b; i += 64) dup |= slots[i] == slot;
  return __any(dup);
}

}  // namespace gla
#endif
