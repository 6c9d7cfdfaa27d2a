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
  int N, P, L, NW, DKP, DVP, marks;  // chunks, segments, their chunks, a walk's waves, padded channels and values, marks
  int dkr, dvr;                  // dk and dv rounded up to 8: the rows that the walks read
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
  // saved by a training forward for the backward (null in a forward-only call, but for the gates, which are scratch there)
  float* gates;   // [BH][N][5][64]
  void* solveT;   // [BH][N][64][64]: (I + beta B)^-1, transposed (bf16: the high parts, then the low parts)
  void* trans;    // [BH][P]: a segment's transition M, transposed, in operands' order (frag_at; bf16: high, then low parts)
  // a chunk's tensors in the order of the registers that hold them, so that a wave stores 1024 bytes on end: 16 value
  // columns after the other, [BH][N][DVP / 16]
  float* err;     // [4][64][4]: delta, see rows_at
  short* o_rest;  // [4][64][4]: what o's rounding left (bf16; see rest_of), lane 16 (c / 4) + r % 16 of tile r / 16
  void* state0;   // [DKP / 32][64][8]: the state entering a chunk, in dtype, lane 16 (channel / 8 % 4) + column
  float* mark;    // [BH][1 + marks][DVP / 16][DKP / 16][256]: the first state, the states leaving every fourth chunk
  // scratch
  void* solve;    // [BH][N][64][64]: (I + B beta)^-1
  void* trans_rows;  // a segment's transition, not transposed (as trans)
  float *seg, *seg_in;  // [BH][P][DVP / 16][DKP / 16][256]: a segment's own end state, the state entering it
  float* z;       // as err
  void* grad1;    // the gradient of the state leaving a chunk, as state0
  float* carry;   // [BH][1 + marks][DVP / 16]: <state, its gradient> there
  float* at;      // [BH][N * 64][2]: o . do - v . dv; the sum of its terms' sizes
  float *dq_heads, *dk_heads;  // [B][H][T][dk], where heads share keys
  void *qk_packed, *v_packed;  // q and k, v (and do), with rows of dkr, dvr elements, where dk, dv are no such numbers
};

// Bytes of the two buffers, and the pointers into them.
size_t delta_saved_bytes(const DeltaShape& s);
size_t delta_scratch_bytes(const DeltaShape& s, bool backward, bool train);
void delta_place(DeltaArgs& a, void* saved, void* scratch, bool backward);

// Copies inputs whose rows are no multiple of 8 elements (the walks load 8 at a time, every lane, at any alignment) and
// points the arguments at the copies.
void delta_pack(DeltaArgs& a, bool backward, hipStream_t s);
hipError_t launch_delta_fwd(DeltaArgs a, hipStream_t s);  // a.err null: forward only
hipError_t launch_delta_bwd(DeltaArgs a, hipStream_t s);

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

// Two floats rounded to bf16, in one word.
__device__ __forceinline__ unsigned round2(float x, float y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {x, y};
  return __builtin_bit_cast(unsigned, __builtin_convertvector(v, bf16x2));
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
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int part = 0; part < N; ++part) {
      u32x4 w;  // two rounded values a word; their own values again by shift and mask
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = round2(x[2 * i], x[2 * i + 1]);
        w[2 + i] = round2(y[2 * i], y[2 * i + 1]);
        if (part + 1 < N) {
          x[2 * i] -= __uint_as_float(w[i] << 16);
          x[2 * i + 1] -= __uint_as_float(w[i] & 0xffff0000u);
          y[2 * i] -= __uint_as_float(w[2 + i] << 16);
          y[2 * i + 1] -= __uint_as_float(w[2 + i] & 0xffff0000u);
        }
      }
      s.part[part] = __builtin_bit_cast(bf16x8, w);
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

// acc[t] += a[t] b (or b a[t]) for the tiles t0 .. t1 - 1, part by part, so that consecutive instructions do not wait
// for each other; pairs of parts as in mma above.
template <typename E, int T0, int T1, int N, int M, int TILES, bool SWAP = false>
__device__ __forceinline__ void mma_tiles(f32x4 (&acc)[TILES], const Split<E, N> (&a)[TILES], const Split<E, M>& b) {
  constexpr int MOST = N == 1 || M == 1 ? N + M - 2 : (N > M ? N : M) - 1;
#pragma unroll
  for (int sum = MOST; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int t = T0; t < T1; ++t)
        if (sum - i >= 0 && sum - i < M) acc[t] = SWAP ? mma(b.part[sum - i], a[t].part[i], acc[t]) : mma(a[t].part[i], b.part[sum - i], acc[t]);
}
// Keeps the compiler from moving anything over: LDS reads are issued a batch ahead of the products that take them.
// Left to itself it reads, waits and multiplies one by one.
template <typename E>
__device__ __forceinline__ void batch() {
  if constexpr (sizeof(E) == 2) __builtin_amdgcn_sched_barrier(0);  // (a float32 product takes 16 times as long, and its operands twice the registers)
}

// Row m of tile t where tiles 2p and 2p + 1 interleave the rows 32p .. 32p + 31: an accumulator's lane (4 rows of
// group g4 in each) then holds 8 consecutive rows, 32p + 8 g4 + (0 .. 7), and can be the next product's operand as
// it stands.
__device__ __forceinline__ int row_of(int t, int m) { return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3); }
// First of the accumulator's four rows in tile t.
__device__ __forceinline__ int row4_of(int t, int g4) { return 32 * (t >> 1) + 8 * g4 + 4 * (t & 1); }

// A tile of D columns in LDS.  bf16: rows without padding, a row's 16-byte blocks in an order that depends on the row,
// so that the 16 lanes a 16-byte read serves at once (lanes 0-3, 12-15, 20-23, 24-27 of a half, and the rest) fall on
// distinct banks, both for rows n16 and for rows row_of(t, n16); D is 32, 64 or 128.  float: rows padded to 16 bytes more.
template <typename E, int D>
struct Tile {
  static constexpr int LD = sizeof(E) == 2 ? D : D + 4;
  __device__ __forceinline__ static int at(int row, int col) {
    if constexpr (sizeof(E) == 2) {
      const int own = D == 128 ? 4 * (row & 3) : D == 64 ? 4 * ((row >> 1) & 1) : 0, turn = -(row >> 3) & 3;
      return row * D + (((col >> 3) ^ (own | turn)) << 3) + (col & 7);
    } else {
      return row * LD + col;
    }
  }
  // 8 consecutive elements of a row, from a multiple of 8
  __device__ __forceinline__ static Frag<E> row(const E* tile, int r, int col) {
    const E* p = tile + at(r, col);
    if constexpr (sizeof(E) == 2) {
      return *reinterpret_cast<const bf16x8*>(p);
    } else {
      const f32x4 x = *reinterpret_cast<const f32x4*>(p), y = *reinterpret_cast<const f32x4*>(p + 4);
      return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
  // (s: the lane's n16.)  4 rows from row0 (a multiple of 4) of the lane's column (of 16 from col0); bf16 through the transposing read (lane s
  // of a 16-lane group addresses row s / 4, columns 4 (s % 4), and receives column s)
  __device__ __forceinline__ static f32x4 rows4(const E* tile, int row0, int col0, int s) {
    f32x4 r;
    if constexpr (sizeof(E) == 2) {
      const auto x = transposed(tile + at(row0 + (s >> 2), col0 + 4 * (s & 3)));
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = (float)x[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = tile[at(row0 + i, col0 + s)];
    }
    return r;
  }
  // Rows kk + 8 g4 + (0 .. 7) of a column: col0 + n16, or with PERM row_of(t, n16) for col0 = row4_of(t, 0)
  template <bool PERM>
  __device__ __forceinline__ static Frag<E> col(const E* tile, int kk, int col0, int s, int g4) {
    Frag<E> r;
    if constexpr (sizeof(E) == 2) {
      // (rows r and r + 4 of an aligned eight have their blocks in the same order)
      const E* p = tile + at(kk + 8 * g4 + (s >> 2), col0 + (PERM ? 8 : 4) * (s & 3));
      const auto lo = transposed(p), hi = transposed(p + 4 * LD);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        r[e] = lo[e];
        r[4 + e] = hi[e];
      }
    } else {
      const int c = col0 + (PERM ? 8 * (s >> 2) + (s & 3) : s);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = tile[at(kk + 8 * g4 + e, c)];
    }
    return r;
  }
  // 4 elements of a row, from a multiple of 4
  __device__ __forceinline__ static void put4(E* tile, int r, int col, f32x4 x) { store4(tile + at(r, col), x); }

 private:
  typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 v4;
  __device__ __forceinline__ static v4 transposed(const E* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) v4*)p);
  }
};
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

// A tile of ROWS rows of D elements on its way from memory to LDS: rows past `rows` and columns past `cols` (at least 1
// of the one, 8 of the other and a multiple of 8) are zero there.  Every lane loads, from a place inside the tile where
// its own is outside: with loads under a condition the compiler waits for all those in flight before the next (4 heads
// of 128 x 256 over 64k tokens: the walk 235 us, so 190).
// FRESH: every load and store forms its addresses anew, for a kernel that has no registers to keep them: one that comes
// back from memory waits for the loads before it.
template <typename E, int ROWS, int D, int NT, bool FRESH = false>
struct TileIn {
  static constexpr int UPR = D / 8, UNITS = ROWS * UPR, PER = (UNITS + NT - 1) / NT;
  static_assert(NT % UPR == 0, "whole rows a pass");
  typename Raw<E, 8>::type r[PER];
  __device__ __forceinline__ void load(const E* src, long stride, int rows, int cols) {
    const int t = FRESH ? fresh_tid() : threadIdx.x;
    if (rows >= ROWS && cols >= D && stride < (1 << 20)) {  // the whole tile, from a base and one 32-bit offset
      const int u = UNITS % NT == 0 ? t : t < UNITS ? t : 0;
      const unsigned at = ((unsigned)(u / UPR) * (unsigned)stride + u % UPR * 8) * sizeof(E);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        r[i] = *reinterpret_cast<const typename Raw<E, 8>::type*>(reinterpret_cast<const char*>(src + i * (NT / UPR) * stride) + at);
    } else {  // (rare: no addresses held for it)
      const int t = fresh_tid();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int u = t + i * NT, c = u % UPR * 8;
        r[i] = *reinterpret_cast<const typename Raw<E, 8>::type*>(src + min(u / UPR, min(rows, ROWS) - 1) * stride + (c < cols ? c : 0));
      }
    }
  }
  __device__ __forceinline__ void store(E* lds, int rows, int cols) const {
    typedef E v8 __attribute__((ext_vector_type(8), aligned(16)));
    const int t = FRESH ? fresh_tid() : threadIdx.x;
    if (rows >= ROWS && cols >= D) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int u = t + i * NT;
        if (UNITS % NT == 0 || u < UNITS) *reinterpret_cast<v8*>(lds + Tile<E, D>::at(u / UPR, u % UPR * 8)) = r[i];
      }
    } else {
      const int t = fresh_tid();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int u = t + i * NT, row = u / UPR, c = u % UPR * 8;
        if (UNITS % NT == 0 || u < UNITS) *reinterpret_cast<v8*>(lds + Tile<E, D>::at(row, c)) = row < rows && c < cols ? (v8)r[i] : (v8){};
      }
    }
  }
};

// A chunk's gate block: e^gamma, e^(gamma_C - gamma), gamma as a sum of two floats, beta; gamma the running sum of g
// from the chunk's start (in 64 bits: a decay between two tokens is the exponential of a difference of two of them).
struct GateBlock {
  float lead[C], late[C], high[C], low[C], beta[C];
};
static_assert(sizeof(GateBlock) == kDeltaGates * sizeof(float), "a gate block's floats");

// A gate block on its way, as TileIn.
template <int NT>
struct GateIn {
  static constexpr int PER = (kDeltaGates + NT - 1) / NT;
  float r[PER];
  __device__ __forceinline__ void load(const float* src) {
#pragma unroll
    for (int i = 0; i < PER; ++i) r[i] = src[min((int)threadIdx.x + i * NT, kDeltaGates - 1)];
  }
  __device__ __forceinline__ void store(GateBlock& s) const {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if ((int)threadIdx.x + i * NT < kDeltaGates) reinterpret_cast<float*>(&s)[threadIdx.x + i * NT] = r[i];
  }
};

// The decays from 4 tokens from `from` on to token `to`, zero where that comes before them (with ON, not where it is one
// of them).
template <bool ON>
__device__ __forceinline__ f32x4 decays_from(const GateBlock& s, int to, int from) {
  const f32x4 high = *reinterpret_cast<const f32x4*>(s.high + from), low = *reinterpret_cast<const f32x4*>(s.low + from);
  const float h = s.high[to], l = s.low[to];
  f32x4 e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = decay((h - high[i]) + (l - low[i]));
    e[i] = (ON ? from + i <= to : from + i < to) ? x : 0.f;
  }
  return e;
}
// The decays from token `from` to 4 tokens from `to` on, likewise.
template <bool ON>
__device__ __forceinline__ f32x4 decays_to(const GateBlock& s, int to, int from) {
  const f32x4 high = *reinterpret_cast<const f32x4*>(s.high + to), low = *reinterpret_cast<const f32x4*>(s.low + to);
  const float h = s.high[from], l = s.low[from];
  f32x4 e;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = decay((high[i] - h) + (low[i] - l));
    e[i] = (ON ? from <= to + i : from < to + i) ? x : 0.f;
  }
  return e;
}

// P by 16 x 16 tiles, spread over a workgroup's waves and held until its place in LDS is free: P itself (rows are
// queries) or transposed.  Ten tiles, and the two above the diagonal that a 32-wide product reads as zeros.
template <typename E, int DK, int NW, bool TRANSPOSED>
struct ScoreTiles {
  static constexpr int N = 12 / NW + (12 % NW != 0);
  f32x4 x[N];
  static constexpr int kTiles = 12;
  __device__ __forceinline__ static void place(int u, int& it, int& jt) {  // query and key tile
    it = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : u < 10 ? 3 : u == 10 ? 0 : 2;
    jt = u < 10 ? u - it * (it + 1) / 2 : it + 1;
  }
  __device__ __forceinline__ void form(const E* Qs, const E* Ks, const GateBlock& gates, int wave, int n16, int g4) {
    typedef Tile<E, DK> K;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = zero4();
      const int u = wave + i * NW;
      if (u >= 10) continue;
      int it, jt;
      place(u, it, jt);
      Frag<E> q[DK / 32], k[DK / 32];
#pragma unroll
      for (int p = 0; p < DK / 32; ++p) {
        q[p] = K::row(Qs, 16 * it + n16, 32 * p + 8 * g4);
        k[p] = K::row(Ks, 16 * jt + n16, 32 * p + 8 * g4);
      }
      const f32x4 e = TRANSPOSED ? decays_to<true>(gates, 16 * it + 4 * g4, 16 * jt + n16) : decays_from<true>(gates, 16 * it + n16, 16 * jt + 4 * g4);
      batch<E>();
#pragma unroll
      for (int p = 0; p < DK / 32; ++p) x[i] = TRANSPOSED ? mma(q[p], k[p], x[i]) : mma(k[p], q[p], x[i]);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[i][r] *= e[r];
    }
  }
  template <int PARTS, int LEN>
  __device__ __forceinline__ void put(E (&Ps)[PARTS][LEN], int parts, int wave, int n16, int g4) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = wave + i * NW;
      if (u >= kTiles) continue;
      int it, jt;
      place(u, it, jt);
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        if (part >= parts) continue;
        if (TRANSPOSED) Tile<E, C>::put4(Ps[part], 16 * jt + n16, 16 * it + 4 * g4, x[i]);
        else Tile<E, C>::put4(Ps[part], 16 * it + n16, 16 * jt + 4 * g4, x[i]);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[i][r] -= (float)(E)x[i][r];
      }
    }
  }
};

__device__ __forceinline__ int length_of(const DeltaArgs& a, int b) {
  const int n = a.lens ? a.lens[b] : a.T;
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// Whether a sequence starts from no state although there is an h0: its first token is a reset, which drops a state whatever
// it holds (a product with a decay of zero would keep what is not finite).
__device__ __forceinline__ bool starts_anew(const DeltaArgs& a, int b, int h, int alive) {
  return a.h0 && alive > 0 && decay(a.g[b * a.gs.b + h * a.gs.h]) == 0.f;
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
// Waits here for values on their way from memory, not where a loop first uses them: there the compiler would wait, in
// every pass, for whatever else is in flight.
template <int CB>
__device__ __forceinline__ void arrived(f32x4 (&S)[CB]) {
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) asm volatile("" : "+v"(S[cb]));
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

// Where an operand of 8 values lies: row r, columns 8 k .. 8 k + 7 of a DK x DK matrix, one 1024-byte block for the 64
// lanes of a product's operand (rows row_of(cb, .), columns 32 p + ..).
template <int DK>
__device__ __forceinline__ int frag_at(int r, int k) {
  const int cb = 2 * (r >> 5) + ((r >> 2) & 1), n16 = 4 * ((r >> 3) & 3) + (r & 3);
  return (cb * (DK / 32) + (k >> 2)) * 512 + (16 * (k & 3) + n16) * 8;
}
// Where 4 columns from c (a multiple of 4) of a chunk's row r lie in 16 columns' accumulators, transposed by quads.
__device__ __forceinline__ int rows_at(int r, int c) {
  const int t = 2 * (r >> 5) + ((r >> 2) & 1);
  return t * 256 + (16 * ((r >> 3) & 3) + 4 * (c >> 2) + (r & 3)) * 4;
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
