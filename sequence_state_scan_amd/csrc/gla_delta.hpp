// Shared by the gated delta rule's kernels (gla_delta_fwd.hip, gla_delta_bwd.hip, gla_delta_step.hip) and their
// host side (gla_delta_api.cpp): arguments, the layout of what they keep, and on the device the chunk's products.
#pragma once
#include "gla_block.hpp"

namespace gla {

constexpr int kDeltaChunk = 64;     // tokens of a chunk
constexpr int kDeltaMarks = 4;      // chunks between the float32 states that a training forward keeps
constexpr int kDeltaMaxDk = 128;    // key channels of the chunked calls
constexpr int kDeltaMaxDv = 1024;
constexpr int kDeltaGates = 5 * kDeltaChunk;  // floats of a chunk's gate block: see GateBlock

// Sizes that follow from a call's.  The sequence's chunks are cut into P segments of L chunks.
struct DeltaShape {
  int B, H, Hk, T, dk, dv, dtype;
  int N, P, L, DKP, DVP, marks;  // chunks, segments, their chunks, padded channels and values, marks
};
DeltaShape delta_shape(int B, int H, int Hk, int T, int dk, int dv, int dtype);

struct DeltaArgs : DeltaShape {
  const void *q, *k, *v;
  const float *g, *beta;
  Strides qs, ks, vs, gs, bs;
  const int* lens;      // [B] or null
  const float* h0;      // [B][H][dk][dv] or null
  void* o;              // [B][H][T][dv]
  float* h_final;       // or null
  // backward
  const void* dO;
  Strides dos;
  const float* dhT;
  void *dq, *dk_, *dv_;
  float *dg, *dbeta, *dh0;
  // saved by a training forward for the backward (null in a forward-only call), but for trans and gates, which are
  // scratch there
  float* gates;   // [BH][N][5][64]
  void* solveT;   // [BH][N][64][64]: (I + beta B)^-1, transposed (bf16: the high parts, then the low parts)
  void* trans;    // [BH][P][DKP][DKP]: a segment's transition, transposed (the same)
  float* err;     // [BH][N * 64][DVP]: delta
  short* o_rest;  // [BH][N * 64][DVP]: what o's rounding left (bf16; see rest_of)
  void* state0;   // [BH][N][DVP][DKP]: the state entering a chunk, transposed, in dtype
  float* mark;    // [BH][marks][DVP / 16][DKP / 16][256]: the state leaving every fourth chunk, in registers' order
  // scratch
  void* solve;    // [BH][N][64][64]: (I + B beta)^-1
  float *seg, *seg_in;  // [BH][P][DVP / 16][DKP / 16][256]: a segment's own end state, the state entering it
  float* z;       // [BH][N * 64][DVP]
  void* grad1;    // [BH][N][DVP][DKP]: the gradient of the state leaving a chunk, transposed
  float* carry;   // [BH][marks][DVP / 16]: <state, its gradient> at the marks
  float* at;      // [BH][N * 64]: o . do - v . dv
  float *dq_heads, *dk_heads;  // [B][H][T][dk], where heads share keys
};

// Bytes of the two buffers, and the pointers into them.
size_t delta_saved_bytes(const DeltaShape& s);
size_t delta_scratch_bytes(const DeltaShape& s, bool backward, bool train);
void delta_place(DeltaArgs& a, void* saved, void* scratch, bool backward);

hipError_t launch_delta_fwd(const DeltaArgs& a, hipStream_t s);  // a.err null: forward only
hipError_t launch_delta_bwd(const DeltaArgs& a, hipStream_t s);

struct DeltaStepArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  float* state;  // [n_slots][H][dk][dv]
  const int* slots;
  void* o;  // [B][H][n][dv]
  Strides qs, ks, vs, gs, bs;
  int B, H, Hk, n, dk, dv, n_slots, dtype;
};
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s);

}  // namespace gla

#ifdef __HIPCC__
#include "gla_common.hpp"

namespace gla {
namespace delta {

constexpr int C = kDeltaChunk;
typedef float f32x8 __attribute__((ext_vector_type(8)));

// Operands of 32 contraction steps for a 16 x 16 tile: 8 consecutive values a lane.  What is computed (states,
// errors, the inverse, decayed products) is held in float32; as a bf16 operand it is split into parts, the rounded
// value and the rounded rest, 2^-17 relative together, so that the states and the float32 results are good to a few
// 2^-18 beside bf16 inputs (whose products with either part are exact).  One bf16 would leave 2^-9.  dg is a sum of
// differences, several times less exact than its terms: a training step therefore splits the vectors that enter it
// most (V - e^gamma K S0, W in o, dW) into three parts (dg 3e-5 with two, 64-bit sums of two parts 1.4e-5).
template <typename E>
struct Num;
template <>
struct Num<bf16> {
  typedef bf16x8 frag;
  static constexpr int PARTS = 2;
};
template <>
struct Num<float> {
  typedef f32x8 frag;
  static constexpr int PARTS = 1;
};
template <typename E>
using Frag = typename Num<E>::frag;

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
  for (int s = 0; s < 8; ++s) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
  return c;
}

template <typename E, int N = Num<E>::PARTS>
struct Split {
  Frag<E> part[N];
};
// Of three parts, in bf16: all of float32's bits.
template <typename E>
using Split3 = Split<E, sizeof(E) == 2 ? 3 : 1>;
// A lane's 8 values of 32 rows: those of tiles 2p and 2p + 1 (see row_of).
template <typename E, int N = Num<E>::PARTS>
__device__ __forceinline__ Split<E, N> split(f32x4 x, f32x4 y) {
  Split<E, N> s;
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int part = 0; part < N; ++part)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s.part[part][i] = (bf16)x[i];
        s.part[part][4 + i] = (bf16)y[i];
        x[i] -= (float)s.part[part][i];
        y[i] -= (float)s.part[part][4 + i];
      }
  } else {
    s.part[0] = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return s;
}
// c + a b, the smallest products first; exact in a bf16 factor.  Of two parts by two the product of the low ones
// (2^-18 of the whole) is left out, as the parts' own rounding is that large; of two by three that of the lowest.
template <typename E, int N>
__device__ __forceinline__ f32x4 mma(Frag<E> a, const Split<E, N>& b, f32x4 c) {
#pragma unroll
  for (int i = N - 1; i >= 0; --i) c = mma(a, b.part[i], c);
  return c;
}
template <typename E, int N>
__device__ __forceinline__ f32x4 mma(const Split<E, N>& a, Frag<E> b, f32x4 c) {
#pragma unroll
  for (int i = N - 1; i >= 0; --i) c = mma(a.part[i], b, c);
  return c;
}
template <typename E, int N, int M>
__device__ __forceinline__ f32x4 mma(const Split<E, N>& a, const Split<E, M>& b, f32x4 c) {
  constexpr int MOST = (N > M ? N : M) - 1;
#pragma unroll
  for (int sum = MOST; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (sum - i >= 0 && sum - i < M) c = mma(a.part[i], b.part[sum - i], c);
  return c;
}

// Row m of tile t where tiles 2p and 2p + 1 interleave the rows 32p .. 32p + 31: an accumulator's lane (4 rows of
// group g4 in each) then holds 8 consecutive rows, 32p + 8 g4 + (0 .. 7), and can be the next product's operand as
// it stands.
__device__ __forceinline__ int row_of(int t, int m) { return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3); }
// First of the accumulator's four rows in tile t.
__device__ __forceinline__ int row4_of(int t, int g4) { return 32 * (t >> 1) + 8 * g4 + 4 * (t & 1); }

// Leading dimension of an LDS tile of D columns (rows on 16 bytes).
template <typename E>
__host__ __device__ constexpr int ld_of(int D) { return D + (sizeof(E) == 2 ? 8 : 4); }

// 8 consecutive elements of an LDS row.
template <typename E>
__device__ __forceinline__ Frag<E> row_frag(const E* p) {
  if constexpr (sizeof(E) == 2) {
    return *reinterpret_cast<const bf16x8*>(p);
  } else {
    const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
    return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
  }
}
// 4 rows from row0 of the lane's column (of 16 from col0) of a row-major LDS tile; bf16 through the transposing read
// (lane s of a 16-lane group addresses row s / 4, columns 4 (s % 4), and receives column s).
template <typename E>
__device__ __forceinline__ f32x4 rows4(const E* tile, int ld, int row0, int col0) {
  const int s = lane_id() & 15;
  f32x4 r;
  if constexpr (sizeof(E) == 2) {
    typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v4;
    const v4 x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (__attribute__((address_space(3))) v4*)(tile + (row0 + (s >> 2)) * ld + col0 + 4 * (s & 3)));
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (float)x[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = tile[(row0 + i) * ld + col0 + s];
  }
  return r;
}
// Rows kk + 8 g4 + (0 .. 7) of a column of a row-major LDS tile: column col0 + n16, or with PERM column
// row_of(t, n16) for col0 = row4_of(t, 0).
template <typename E, bool PERM>
__device__ __forceinline__ Frag<E> col_frag(const E* tile, int ld, int kk, int col0) {
  const int l = lane_id(), s = l & 15, g4 = l >> 4;
  Frag<E> r;
  if constexpr (sizeof(E) == 2) {
    typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v4;
    const E* p = tile + (kk + 8 * g4 + (s >> 2)) * ld + col0 + (PERM ? 8 : 4) * (s & 3);
    const v4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) v4*)p);
    const v4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) v4*)(p + 4 * ld));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] = lo[e];
      r[4 + e] = hi[e];
    }
  } else {
    const int col = col0 + (PERM ? 8 * (s >> 2) + (s & 3) : s);
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = tile[(kk + 8 * g4 + e) * ld + col];
  }
  return r;
}

// 8 (4) elements in memory at any alignment of the element.
template <typename E, int N>
struct Raw {
  typedef E type __attribute__((ext_vector_type(N), aligned(sizeof(E))));
};
template <typename E>
__device__ __forceinline__ typename Raw<E, 8>::type load8_part(const E* p, int left) {
  typedef typename Raw<E, 8>::type R;
  if (left >= 8) return *reinterpret_cast<const R*>(p);
  R r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = i < left ? p[i] : (E)0.f;
  return r;
}
template <typename E>
__device__ __forceinline__ void store4_part(E* p, f32x4 x, int left) {
  typedef typename Raw<E, 4>::type R;
  if (left >= 4) {
    R r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (E)x[i];
    *reinterpret_cast<R*>(p) = r;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = (E)x[i];
  }
}

// A tile of ROWS rows of D elements on its way from memory to LDS: rows past `rows` and columns past `cols` zero.
template <typename E, int ROWS, int D, int NT>
struct TileIn {
  static constexpr int UNITS = ROWS * D / 8, PER = (UNITS + NT - 1) / NT;
  typename Raw<E, 8>::type r[PER];
  __device__ __forceinline__ void load(const E* src, long stride, int rows, int cols) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = threadIdx.x + i * NT, row = u / (D / 8), c = u % (D / 8) * 8;
      r[i] = (typename Raw<E, 8>::type){};
      if ((UNITS % NT == 0 || u < UNITS) && row < rows && c < cols) r[i] = load8_part<E>(src + row * stride + c, cols - c);
    }
  }
  __device__ __forceinline__ void store(E* lds, int ld) const {
    typedef E v8 __attribute__((ext_vector_type(8), aligned(16)));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = threadIdx.x + i * NT;
      if (UNITS % NT == 0 || u < UNITS) *reinterpret_cast<v8*>(lds + u / (D / 8) * ld + u % (D / 8) * 8) = r[i];
    }
  }
};

// A chunk's gate block: e^gamma, e^(gamma_C - gamma), gamma as a sum of two floats, beta; gamma the running sum of g
// from the chunk's start (in 64 bits: a decay between two tokens is the exponential of a difference of two of them).
struct GateBlock {
  float lead[C], late[C], high[C], low[C], beta[C];
};
static_assert(sizeof(GateBlock) == kDeltaGates * sizeof(float), "a gate block's floats");
// The decay from token j to token i (gamma_i - gamma_j, not positive).
__device__ __forceinline__ float decay_between(const GateBlock& s, int i, int j) {
  return decay((s.high[i] - s.high[j]) + (s.low[i] - s.low[j]));
}

__device__ __forceinline__ int length_of(const DeltaArgs& a, int b) {
  const int n = a.lens ? a.lens[b] : a.T;
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// Row-major [dk][dv] states in an accumulator: lane's rows row4_of(cb, g4) + i, column j + n16.
template <int CB>
__device__ __forceinline__ void load_state(f32x4 (&S)[CB], const float* p, int dk, int dv, int col) {
  const int g4 = lane_id() >> 4;
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row4_of(cb, g4) + i;
      S[cb][i] = p && r < dk && col < dv ? p[(long)r * dv + col] : 0.f;
    }
}
template <int CB>
__device__ __forceinline__ void store_state(const f32x4 (&S)[CB], float* p, int dk, int dv, int col) {
  const int g4 = lane_id() >> 4;
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row4_of(cb, g4) + i;
      if (r < dk && col < dv) p[(long)r * dv + col] = S[cb][i];
    }
}
// The same in registers' order: [tile][lane][4].
template <int CB>
__device__ __forceinline__ void load_regs(f32x4 (&S)[CB], const float* p) {
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) S[cb] = *reinterpret_cast<const f32x4*>(p + cb * 256 + lane_id() * 4);
}
template <int CB>
__device__ __forceinline__ void store_regs(const f32x4 (&S)[CB], float* p) {
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) *reinterpret_cast<f32x4*>(p + cb * 256 + lane_id() * 4) = S[cb];
}

// An accumulator tile of 4 rows x the lane's column, stored by rows.  p: the first of its rows, the first of 16 columns.
__device__ __forceinline__ void store_rows(f32x4 x, float* p, int pitch) {
  const int s = lane_id() & 15;
  *reinterpret_cast<f32x4*>(p + (s & 3) * pitch + 4 * (s >> 2)) = quad_transpose(x);
}

// A float32's place beside its bf16 rounding: the difference of their bit patterns fits 16 bits (of a tie, up to one
// unit).
__device__ __forceinline__ short rest_of(float x, bf16 rounded) {
  const int d = __float_as_int(x) - ((int)__builtin_bit_cast(unsigned short, rounded) << 16);
  return (short)min(d, 32767);
}
__device__ __forceinline__ float with_rest(bf16 rounded, short rest) {
  return __int_as_float(((int)__builtin_bit_cast(unsigned short, rounded) << 16) + rest);
}

}  // namespace delta
}  // namespace gla
#endif
