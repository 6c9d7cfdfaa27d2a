// Rows spread over lanes in slots of 8 elements: what the join (gla_join.hip) and the layer norm
// (gla_layernorm.hip) share.
#pragma once
#include "gla_block.hpp"

namespace gla {

constexpr int VEC = 8;  // elements of a slot

static inline int pow2_up(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// Sum over the lanes of aligned groups of `width` lanes (a power of 2 up to 64), the same in every
// lane of a group: the neighbour's, the other pair's, the other four's (mirrored: by then four
// lanes hold one value), the other eight's, then rows of 16 and halves of 32 swapped.  All in the
// vector unit; lane exchanges through LDS cost a trip there each.
__device__ __forceinline__ float lane_sum(float v, int width) {
  if (width > 1) v += dpp<0xB1>(v);   // quad_perm 1 0 3 2
  if (width > 2) v += dpp<0x4E>(v);   // quad_perm 2 3 0 1
  if (width > 4) v += dpp<0x141>(v);  // row_half_mirror
  if (width > 8) v += dpp<0x140>(v);  // row_mirror
  if (width > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (width > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// The sum of a row's slots in every lane of the row.  red: 2 x 16 floats of LDS, used in turn
// (`turn` 0, 1, 0, ..), so that one barrier a call is enough: who writes a half again has passed
// the barrier of the call between, behind every read of it.  Every lane of the workgroup calls it.
__device__ __forceinline__ float row_sum(float v, int TPR, float* red, int turn) {
  if (TPR <= 64) return lane_sum(v, TPR);
  v = lane_sum(v, 64);
  red += turn * 16;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const int w = TPR / 64, first = (threadIdx.x >> 6) / w * w;
  float s = 0.f;
  for (int i = 0; i < w; ++i) s += red[first + i];
  return s;
}

// VEC elements at any alignment of the element.
template <typename E>
struct Pack {
  typedef E raw __attribute__((ext_vector_type(VEC), aligned(sizeof(E))));
};

// The first `left` of a slot's elements (all of them where left >= VEC), the others zero.
template <bool EVEN, typename E>
__device__ __forceinline__ typename Pack<E>::raw load_slot(const E* p, int left) {
  if (EVEN || left >= VEC) return *reinterpret_cast<const typename Pack<E>::raw*>(p);
  typename Pack<E>::raw r;
#pragma unroll
  for (int v = 0; v < VEC; ++v) r[v] = v < left ? p[v] : (E)0.f;
  return r;
}
template <bool EVEN, typename E>
__device__ __forceinline__ void store_slot(E* p, const float (&v)[VEC], int left) {
  if (EVEN || left >= VEC) {
    typename Pack<E>::raw r;
#pragma unroll
    for (int i = 0; i < VEC; ++i) r[i] = (E)v[i];
    *reinterpret_cast<typename Pack<E>::raw*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < left) p[i] = (E)v[i];
  }
}

// The row a workgroup's lane group is at: (b, t) stepped without a division.  The sums are unsigned: t + dt
// passes 2^31 for the longest T, and b + db behind the last row.
struct RowStep {
  long row;
  int b, t, db, dt;
  __device__ RowStep(long first, int T, long step) {
    row = first;
    b = (int)(first / T);
    t = (int)(first - (long)b * T);
    db = (int)(step / T);
    dt = (int)(step - (long)db * T);
  }
  __device__ void next(int T, long step) {
    row += step;
    b = (int)((unsigned)b + (unsigned)db);
    t = (int)((unsigned)t + (unsigned)dt);
    if ((unsigned)t >= (unsigned)T) {
      t = (int)((unsigned)t - (unsigned)T);
      b = (int)((unsigned)b + 1u);
    }
  }
};

}  // namespace gla
