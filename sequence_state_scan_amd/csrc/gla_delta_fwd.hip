// The gated delta rule by chunks of 64 tokens, forward.  With S0 the state entering a chunk, gamma the running sums
// of g in it, E_ij = e^(gamma_i - gamma_j), B = K K^T . E below the diagonal and P = Q K^T . E on and below it:
//   delta = (I + B beta)^-1 (V - e^gamma K S0),   W = beta delta          what a token writes under its key
//   O = e^gamma Q S0 + P W,   S1 = e^gamma_C S0 + (e^(gamma_C - gamma) K)^T W
// delta_prep_kernel forms the gates and the inverse, every chunk on its own.  delta_fwd_kernel walks the chunks of a
// segment: a wave holds 16 columns of the state in accumulators, K S0, delta and the state's update follow one
// another inside the wave (an accumulator is the next product's operand as it stands), and the waves share the
// chunk's K, Q, V and inverse in LDS, loaded a chunk ahead.
// A sequence of too few heads to fill the chip is cut into P segments: a state pass finds each segment's own end
// state from zero and its transition M (the same walk from the identity with V = 0), delta_scan_kernel chains
// S <- M S + S_own, and the walk then starts from the true states.
// What bounds it: a chunk's steps follow one another, so a CU's 8 waves share their time between the vector ALU (half of
// the cycles: the splits, the scaling of states and errors, the decays), the matrix cores (28 %, in a forward-only call more
// since o's operands are split) and LDS (35 %); a training walk also writes 115 KB a chunk and 128 columns and runs at HBM's
// rate, 4.8 TB/s.  bf16, 4 heads of 64k tokens, 128 x 256, P = 32, kernels traced one by one (500 us in all, where a call takes
// 444 to 474 in a row): gates and inverses 47 us, state pass 192, chain 40, walk 222 (some 20 less with the state, W and P of o as
// one bf16 each, which left o 2.9e-3 off in the 2-norm instead of its own rounding's 1.7e-3), where q, k, v and o are 83 us of HBM.  With
// those operands of one part P formed once in delta_prep_kernel and loaded by the walks saved 6 us here and cost 15 there; 32
// columns a wave or half the waves, two workgroups a CU, took as long.
#include "gla_delta.hpp"
#include "gla_delta_scan.hpp"

namespace gla {
namespace delta {

// Rows of d elements into rows of r, d rounded up to 8, the rest zero; 8 elements a lane.
template <typename E>
__global__ __launch_bounds__(256) void delta_pack_kernel(const E* from, Strides st, E* to, int heads, int T, int d, int r, long units) {
  for (long u = (long)blockIdx.x * 256 + threadIdx.x; u < units; u += (long)gridDim.x * 256) {
    const int c = (int)(u % (r / 8)) * 8;
    const long row = u / (r / 8), bh = row / T, t = row - bh * T, b = bh / heads, h = bh - b * heads;
    typedef E v8 __attribute__((ext_vector_type(8), aligned(16)));
    *reinterpret_cast<v8*>(to + u * 8) = load8_part<E>(from + b * st.b + h * st.h + t * st.t + c, d - c);
  }
}

// ---------------------------------------------------------------------------------------- gates, inverse

// (I + L)^-1 of a unit lower triangular 64 x 64 matrix in float32: its 16 x 16 diagonal blocks by forward
// substitution, a column a lane, then joined two and two, X21 = -X22 L21 X11, on the float32 matrix instructions.
// Two of them at once: L = B beta (columns scaled) and, transposed at the end, L = beta B for the backward.
// Bound by what it writes (4096 chunks, 128 channels, bf16: 46 us, 3.1 TB/s; with the second inverse 58 us, 3.6 TB/s), and
// where there are few chunks by the substitution's 16 steps (7 us).
template <typename E, int DK, bool TRAIN>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a) {
  constexpr int LF = 66;
  typedef Tile<E, DK> K;
  constexpr int KBYTES = C * K::LD * sizeof(E), XBYTES = C * LF * 4;
  __shared__ __attribute__((aligned(16))) unsigned char raw[KBYTES > XBYTES ? KBYTES : XBYTES];
  __shared__ __attribute__((aligned(16))) float Bm[C * LF], X1[C * LF];  // B; the inverse with scaled columns
  __shared__ __attribute__((aligned(16))) GateBlock gates;
  E* Ks = (E*)raw;
  float* X2 = (float*)raw;  // the other inverse, once K is used up
  const int n = blockIdx.x % a.N, bh = blockIdx.x / a.N, b = bh / a.H, h = bh - b * a.H;
  const int len = length_of(a, b);
  if (n * C >= len) return;
  const int lane = lane_id(), wave = wave_id(), n16 = lane & 15, g4 = lane >> 4;
  const long t0 = (long)n * C;
  TileIn<E, C, DK, 256> k;
  k.load((const E*)a.k + b * a.ks.b + (h / (a.H / a.Hk)) * a.ks.h + t0 * a.ks.t, a.ks.t, len - n * C, a.dkr);
  if (wave == 0) {
    const long t = t0 + lane;
    const bool live = t < len;
    // below -200 every decay over the token is an exact zero; NaN (which a maximum would drop) stays
    const float g = live ? a.g[b * a.gs.b + h * a.gs.h + t * a.gs.t] : 0.f;
    double x = g < -200.f ? -200.f : g;
    const float beta = live ? a.beta[b * a.bs.b + h * a.bs.h + t * a.bs.t] : 0.f;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const double y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    const double all = __shfl(x, 63);
    gates.lead[lane] = decay((float)x);
    gates.late[lane] = decay((float)(all - x));
    gates.high[lane] = (float)x;
    gates.low[lane] = (float)(x - (double)(float)x);
    gates.beta[lane] = beta;
  }
  k.store(Ks, len - n * C, a.dkr);
  __syncthreads();
  // B, one row tile a wave
  for (int jt = 0; jt <= wave; ++jt) {
    f32x4 acc = zero4();
#pragma unroll
    for (int p = 0; p < DK / 32; ++p)
      acc = mma(K::row(Ks, 16 * wave + n16, 32 * p + 8 * g4), K::row(Ks, 16 * jt + n16, 32 * p + 8 * g4), acc);
    const int j = 16 * jt + n16, i = 16 * wave + 4 * g4;
    const f32x4 e = decays_to<false>(gates, i, j);
#pragma unroll
    for (int r = 0; r < 4; ++r) Bm[(i + r) * LF + j] = acc[r] * e[r];
  }
  __syncthreads();
  if (threadIdx.x < kDeltaGates / 4)
    reinterpret_cast<f32x4*>(a.gates + ((long)bh * a.N + n) * kDeltaGates)[threadIdx.x] = reinterpret_cast<f32x4*>(&gates)[threadIdx.x];
  const bool second = g4 == 1;  // lanes 16 .. 31: the inverse with scaled rows
  {
    float x[16], y[16];
    const float* L = Bm + 16 * wave * (LF + 1);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float bi = gates.beta[16 * wave + i];
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(L[i * LF + j], y[j], s);
      x[i] = (i == n16 ? 1.f : 0.f) - (second ? bi * s : s);
      if (i < n16) x[i] = 0.f;
      y[i] = second ? x[i] : bi * x[i];
    }
    float* X = second ? X2 : X1;
    if (g4 == 0 || (TRAIN && second))
#pragma unroll
      for (int i = 0; i < 16; ++i) X[(16 * wave + i) * LF + 16 * wave + n16] = x[i];
  }
  __syncthreads();
  // L's element, scaled for the inverse it belongs to
  const auto at = [&](bool rows, int i, int j) { return Bm[i * LF + j] * gates.beta[rows ? i : j]; };
  // acc += L(it, kt) X(kt, jt), 16 x 16 tiles; then out(it, jt) -= X(it, kt) t(kt) for t in an accumulator
  const auto times = [&](bool rows, const float* X, int it, int kt, int jt, f32x4 acc) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(at(rows, 16 * it + n16, 16 * kt + 4 * s + g4), X[(16 * kt + 4 * s + g4) * LF + 16 * jt + n16], acc, 0, 0, 0);
    return acc;
  };
  const auto minus = [&](const float* X, int it, int kt, f32x4 t, f32x4 acc) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(-X[(16 * it + n16) * LF + 16 * kt + 4 * g4 + s], t[s], acc, 0, 0, 0);
    return acc;
  };
  const auto put = [&](float* X, int it, int jt, f32x4 v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) X[(16 * it + 4 * g4 + r) * LF + 16 * jt + n16] = v[r];
  };
  const bool rows = wave & 1;
  float* X = rows ? X2 : X1;
  const int half = wave >> 1;
  if (TRAIN || !rows) {  // blocks (1, 0) and (3, 2)
    const int it = 2 * half + 1, jt = 2 * half;
    put(X, it, jt, minus(X, it, it, times(rows, X, it, jt, jt, zero4()), zero4()));
  }
  __syncthreads();
  if (TRAIN || !rows) {  // column half of the lower left quarter
    f32x4 t2 = times(rows, X, 2, 1, half, zero4()), t3 = times(rows, X, 3, 1, half, zero4());
    if (half == 0) {
      t2 = times(rows, X, 2, 0, 0, t2);
      t3 = times(rows, X, 3, 0, 0, t3);
    }
    put(X, 2, half, minus(X, 2, 2, t2, zero4()));
    put(X, 3, half, minus(X, 3, 3, t3, minus(X, 3, 2, t2, zero4())));
  }
  __syncthreads();
  const long block = ((long)bh * a.N + n) * C * C, plane = (long)a.B * a.H * a.N * C * C;
#pragma unroll
  for (int which = 0; which < (TRAIN ? 2 : 1); ++which) {
    E* out = (E*)(which ? a.solveT : a.solve) + block;
    const float* from = which ? X2 : X1;
    for (int u = threadIdx.x; u < C * C / 8; u += 256) {
      const int i = u / 8, j = u % 8 * 8;
      f32x4 x, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = which ? (i <= j + e ? from[(j + e) * LF + i] : 0.f) : (i >= j + e ? from[i * LF + j + e] : 0.f);
        y[e] = which ? (i <= j + 4 + e ? from[(j + 4 + e) * LF + i] : 0.f) : (i >= j + 4 + e ? from[i * LF + j + 4 + e] : 0.f);
      }
      const Split<E> s = split<E>(x, y);
#pragma unroll
      for (int part = 0; part < Num<E>::PARTS; ++part) *reinterpret_cast<Frag<E>*>(out + part * plane + i * C + j) = s.part[part];
    }
  }
}

// ---------------------------------------------------------------------------------------- the walk

enum { INFER = 0, TRAIN = 1, STATE = 2 };

// Workgroup: one segment and 16 NW columns.  STATE: the segment's own end state where another follows,
// and past the value columns its transition where another follows or, for the backward's chain, precedes.
// (The state pass alone leaves the order of its LDS reads to the compiler: in half the registers two workgroups fit a CU:
// 193 us of 4 heads of 64k, 128 x 256, where one with its reads in order takes 210.)
template <typename E, int DK, int NW, int MODE>
__global__ __launch_bounds__(64 * NW, MODE == STATE && NW == 8 && sizeof(E) == 2 ? 4 : 1) void delta_fwd_kernel(DeltaArgs a) {
  constexpr int NT = 64 * NW, CB = DK / 16, CP = DK / 32, CW = 16 * NW, PARTS = Num<E>::PARTS;
  constexpr int FINE = MODE == TRAIN && PARTS == 2 ? 3 : PARTS;  // parts of W in o, and of Y
  typedef Tile<E, DK> K;
  typedef Tile<E, CW> V;
  typedef Tile<E, C> M;
  __shared__ __attribute__((aligned(16))) E Ks[C * K::LD], Vs[C * V::LD], Qs[MODE == STATE ? 8 : C * K::LD];
  __shared__ __attribute__((aligned(16))) E Ts[PARTS][C * M::LD];  // the inverse, then P in its place
  __shared__ __attribute__((aligned(16))) GateBlock gates;
  const bool chained = MODE == STATE && a.err;  // a backward follows
  const int segments = MODE == STATE && !chained ? a.P - 1 : a.P, units = a.B * a.H * segments;
  const int unit = blockIdx.x % units, tile = blockIdx.x / units;  // a segment's column tiles: the same XCD mostly
  const int bh = unit / segments, seg = unit - bh * segments, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
  const int len = length_of(a, b), alive = (len + C - 1) / C;
  const int first = seg * a.L, last = min(first + a.L, a.N), end = min(last, alive);
  const int lane = lane_id(), wave = wave_id(), n16 = lane & 15, g4 = lane >> 4, k8 = 8 * g4;
  const int value_tiles = (a.dv + CW - 1) / CW;
  const bool transition = MODE == STATE && tile >= value_tiles;
  if (MODE == STATE && last >= alive && !(transition && chained && seg > 0 && first < alive)) return;
  const int col0 = (transition ? tile - value_tiles : tile) * CW, j = col0 + 16 * wave;  // the wave's columns
  const bool cols = j < (transition ? a.DKP : a.dv);
  const long tiles = a.DVP / 16;

  f32x4 S[CB];
  if (MODE == STATE) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[cb][i] = transition && row4_of(cb, g4) + i == j + n16 ? 1.f : 0.f;
  } else if (a.P > 1) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) S[cb] = zero4();
    if (cols && (seg == 0 || first < alive)) load_regs<CB>(S, a.seg_in + (((long)bh * a.P + seg) * tiles + j / 16) * DK * 16);
  } else {
    load_state<CB>(S, a.h0 ? a.h0 + (long)bh * a.dk * a.dv : nullptr, a.dk, a.dv, j + n16);
    if (starts_anew(a, b, h, alive))
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) S[cb] = zero4();
  }
  arrived<CB>(S);
  if (MODE == TRAIN && cols && seg == 0) store_regs<CB>(S, a.mark + ((long)bh * (a.marks + 1) * tiles + j / 16) * DK * 16);

  const E* kp = (const E*)a.k + b * a.ks.b + hk * a.ks.h;
  const E* qp = (const E*)a.q + b * a.qs.b + hk * a.qs.h;
  const E* vp = (const E*)a.v + b * a.vs.b + h * a.vs.h + col0;
  const E* tp = (const E*)a.solve + (long)bh * a.N * C * C;
  const float* gp = a.gates + (long)bh * a.N * kDeltaGates;
  const long plane = (long)a.B * a.H * a.N * C * C;
  constexpr bool TIGHT = MODE == STATE && NW == 8 && PARTS == 2;
  TileIn<E, C, DK, NT, TIGHT> kin, qin;
  TileIn<E, C, CW, NT, TIGHT> vin{};
  TileIn<E, C, C, NT, TIGHT> tin[PARTS];
  GateIn<NT> gin;
  const auto load = [&](int n) {
    const long t0 = (long)n * C;
    const int left = len - n * C;
    kin.load(kp + t0 * a.ks.t, a.ks.t, left, a.dkr);
    if (MODE != STATE) qin.load(qp + t0 * a.qs.t, a.qs.t, left, a.dkr);
    if (!transition) vin.load(vp + t0 * a.vs.t, a.vs.t, left, a.dvr - col0);
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].load(tp + part * plane + (long)n * C * C, C, C, C);
    gin.load(gp + (long)n * kDeltaGates);
  };
  if (first < end) load(first);
  for (int n = first; n < end; ++n) {
    __syncthreads();
    const int left = len - n * C;
    kin.store(Ks, left, a.dkr);
    if (MODE != STATE) qin.store(Qs, left, a.dkr);
    vin.store(Vs, transition ? 0 : left, a.dvr - col0);
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].store(Ts[part], C, C);
    gin.store(gates);
    __syncthreads();
    if (n + 1 < end) load(n + 1);
    // (the lane's number anew in every phase: the LDS addresses formed from it would not fit the registers all at once)
    const int lane = fresh_tid() & 63, n16 = lane & 15, g4 = lane >> 4, k8 = 8 * g4;
    ScoreTiles<E, DK, NW, false> P;
    if constexpr (MODE != STATE) P.form(Qs, Ks, gates, wave, n16, g4);
    // K S0 and Q S0 (transposed: a lane has four columns of one token)
    f32x4 Y[4], W[4], O[4];
    {
      Split<E, 1> kf[2][4], qf[2][4];
      const auto fetch = [&](int p) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          kf[p & 1][t].part[0] = K::row(Ks, row_of(t, n16), 32 * p + k8);
          if constexpr (MODE != STATE) qf[p & 1][t].part[0] = K::row(Qs, 16 * t + n16, 32 * p + k8);
        }
      };
      fetch(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) Y[t] = O[t] = zero4();
#pragma unroll
      for (int p = 0; p < CP; ++p) {
        const Split<E> So = split<E>(S[2 * p], S[2 * p + 1]);
        if (MODE == TRAIN && cols)
          *reinterpret_cast<Frag<E>*>((E*)a.state0 + ((((long)bh * a.N + n) * tiles + j / 16) * CP + p) * 512 + lane * 8) = So.part[0];
        if (p + 1 < CP) fetch(p + 1);
        if constexpr (MODE != STATE) batch<E>();
        mma_tiles<E, 0, 4>(Y, kf[p & 1], So);
        if constexpr (MODE != STATE) mma_tiles<E, 0, 4, 1, PARTS, 4, true>(O, qf[p & 1], So);
        if constexpr (MODE != STATE) batch<E>();
      }
    }
    // delta, W and e^(gamma_C - gamma) W
    {
      Split<E> T[2][4];
      const auto fetch = [&](int p) {
#pragma unroll
        for (int t = 2 * p; t < 4; ++t)
#pragma unroll
          for (int part = 0; part < PARTS; ++part) T[p][t].part[part] = M::row(Ts[part], row_of(t, n16), 32 * p + k8);
      };
      f32x4 lead[4], v[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        lead[t] = *reinterpret_cast<const f32x4*>(gates.lead + row4_of(t, g4));
        v[t] = V::rows4(Vs, row4_of(t, g4), 16 * wave, n16);
      }
      fetch(0);
      if constexpr (MODE != STATE) batch<E>();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) Y[t][i] = fmaf(-lead[t][i], Y[t][i], v[t][i]);
        W[t] = zero4();
      }
      const Split<E, FINE> Yo[2] = {split<E, FINE>(Y[0], Y[1]), split<E, FINE>(Y[2], Y[3])};
      fetch(1);
      if constexpr (MODE != STATE) batch<E>();
      mma_tiles<E, 0, 4>(W, T[0], Yo[0]);
      mma_tiles<E, 2, 4>(W, T[1], Yo[1]);
      if constexpr (MODE != STATE) batch<E>();
    }
    f32x4 beta[4], late[4];
    float leads[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      beta[t] = *reinterpret_cast<const f32x4*>(gates.beta + row4_of(t, g4));
      late[t] = *reinterpret_cast<const f32x4*>(gates.late + row4_of(t, g4));
      leads[t] = gates.lead[16 * t + n16];
    }
    const float whole = gates.lead[C - 1];
    if constexpr (MODE != STATE) batch<E>();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if (MODE == TRAIN && cols) *reinterpret_cast<f32x4*>(a.err + ((((long)bh * a.N + n) * tiles + j / 16) * 4 + t) * 256 + lane * 4) = quad_transpose(W[t]);
#pragma unroll
      for (int i = 0; i < 4; ++i) W[t][i] *= beta[t][i];
    }
    if constexpr (MODE != STATE) {
      const Split<E, FINE> Wo[2] = {split<E, FINE>(W[0], W[1]), split<E, FINE>(W[2], W[3])};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) O[t][i] *= leads[t];
      __syncthreads();
      P.put(Ts, PARTS, wave, n16, g4);
      __syncthreads();
      const int lane = fresh_tid() & 63, n16 = lane & 15, g4 = lane >> 4, k8 = 8 * g4;
      Split<E> Pf[2][4];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 2 * p; t < 4; ++t)
#pragma unroll
          for (int part = 0; part < PARTS; ++part) Pf[p][t].part[part] = M::row(Ts[part], 16 * t + n16, 32 * p + k8);
      if constexpr (MODE != STATE) batch<E>();
      mma_tiles<E, 0, 4, PARTS, FINE, 4, true>(O, Pf[0], Wo[0]);
      mma_tiles<E, 2, 4, PARTS, FINE, 4, true>(O, Pf[1], Wo[1]);
    }
    {
      const int lane = fresh_tid() & 63, n16 = lane & 15, g4 = lane >> 4;
      constexpr int TILES = CB < 4 ? CB : 4;  // a batch
      Split<E, 1> kf[2][TILES];
      const auto fetch = [&](int s) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) kf[s & 1][i].part[0] = K::template col<true>(Ks, 32 * (s * TILES / CB), row4_of(s * TILES % CB + i, 0), n16, g4);
      };
      fetch(0);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) W[t][i] *= late[t][i];
      const Split<E> Wl[2] = {split<E>(W[0], W[1]), split<E>(W[2], W[3])};
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[cb][i] *= whole;
#pragma unroll
      for (int s = 0; s < 2 * CB / TILES; ++s) {
        if (s + 1 < 2 * CB / TILES) fetch(s + 1);
        if constexpr (MODE != STATE) batch<E>();
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
          for (int i = 0; i < TILES; ++i) {
            f32x4& acc = S[s * TILES % CB + i];
            acc = mma(kf[s & 1][i].part[0], Wl[s * TILES / CB].part[part], acc);
          }
        if constexpr (MODE != STATE) batch<E>();
      }
    }
    if constexpr (MODE != STATE) {
      const int lane = fresh_tid() & 63, n16 = lane & 15, g4 = lane >> 4;
      const long row0 = (long)n * C;
      E* to = (E*)a.o + ((long)bh * a.T + row0) * a.dv + j;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = 16 * t + n16;
        if (!cols || row >= left) continue;
        store4_part<E>(to + row * a.dv + 4 * g4, O[t], a.dv - j - 4 * g4);
        if constexpr (MODE == TRAIN && PARTS == 2) {
          typedef short s16x4 __attribute__((ext_vector_type(4)));
          s16x4 rest;
#pragma unroll
          for (int i = 0; i < 4; ++i) rest[i] = rest_of(O[t][i], (bf16)O[t][i]);
          *reinterpret_cast<s16x4*>(a.o_rest + ((((long)bh * a.N + n) * tiles + j / 16) * 4 + t) * 256 + lane * 4) = rest;
        }
      }
    }
    if (MODE == TRAIN && cols && (n % kDeltaMarks == kDeltaMarks - 1 || n == alive - 1))
      store_regs<CB>(S, a.mark + (((long)bh * (a.marks + 1) + n / kDeltaMarks + 1) * tiles + j / 16) * DK * 16);
  }
  if (!cols) return;
  if (MODE == STATE) {
    if (!transition) {
      store_regs<CB>(S, a.seg + (((long)bh * a.P + seg) * tiles + j / 16) * DK * 16);
      return;
    }
    const long block = ((long)bh * a.P + seg) * DK * DK, mplane = (long)a.B * a.H * a.P * DK * DK;
    if (chained) {  // (only the backward's chain reads it)
      E* to = (E*)a.trans + block;
#pragma unroll
      for (int p = 0; p < CP; ++p) {
        const Split<E> s = split<E>(S[2 * p], S[2 * p + 1]);
#pragma unroll
        for (int part = 0; part < PARTS; ++part) *reinterpret_cast<Frag<E>*>(to + part * mplane + frag_at<DK>(j + n16, 4 * p + g4)) = s.part[part];
      }
    }
    const int c = j + 4 * (n16 >> 2);
    E* by_rows = (E*)a.trans_rows + block + (c & 7);
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      f32x4 x = quad_transpose(S[cb]);
      E* p = by_rows + frag_at<DK>(row4_of(cb, g4) + (n16 & 3), c >> 3);
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        store4(p + part * mplane, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] -= (float)(E)x[i];
      }
    }
    return;
  }
  if (a.h_final && (alive ? first < alive && alive <= last : seg == 0))
    store_state<CB>(S, a.h_final + (long)bh * a.dk * a.dv, a.dk, a.dv, j + n16);
  const int stop = min(last * C, a.T);  // rows of this segment behind the sequence's end
  for (int t = max(first * C, len) + (lane >> 2); t < stop; t += 16)
    store4_part<E>((E*)a.o + ((long)bh * a.T + t) * a.dv + j + 4 * (lane & 3), zero4(), a.dv - j - 4 * (lane & 3));
}

}  // namespace delta

using namespace delta;

template <typename E, int DK, int NW>
static void delta_fwd_run(const DeltaArgs& a, hipStream_t s) {
  constexpr int CW = 16 * NW;
  const int heads = a.B * a.H, tiles = (a.dv + CW - 1) / CW;
  const bool train = a.err;
  if (train) delta_prep_kernel<E, DK, true><<<heads * a.N, 256, 0, s>>>(a);
  else delta_prep_kernel<E, DK, false><<<heads * a.N, 256, 0, s>>>(a);
  if (a.P > 1) {
    delta_fwd_kernel<E, DK, NW, STATE><<<heads * (train ? a.P : a.P - 1) * (tiles + (DK + CW - 1) / CW), 64 * NW, 0, s>>>(a);
    delta_scan_kernel<E, DK, false><<<heads * ((a.dv + 31) / 32), 4 * DK, 0, s>>>(a);
  }
  if (train) delta_fwd_kernel<E, DK, NW, TRAIN><<<heads * a.P * tiles, 64 * NW, 0, s>>>(a);
  else delta_fwd_kernel<E, DK, NW, INFER><<<heads * a.P * tiles, 64 * NW, 0, s>>>(a);
}
template <typename E, int DK>
static void delta_fwd_cols(const DeltaArgs& a, hipStream_t s) {
  if (a.NW == 4) delta_fwd_run<E, DK, 4>(a, s);
  else delta_fwd_run<E, DK, 8>(a, s);
}
template <typename E>
static void delta_fwd_rows(const DeltaArgs& a, hipStream_t s) {
  if (a.DKP == 32) delta_fwd_cols<E, 32>(a, s);
  else if (a.DKP == 64) delta_fwd_cols<E, 64>(a, s);
  else delta_fwd_cols<E, 128>(a, s);
}

template <typename E>
static void pack_one(const void*& p, Strides& st, void* to, const DeltaArgs& a, int heads, int d, int r, hipStream_t s) {
  const long units = (long)a.B * heads * a.T * (r / 8);
  const long blocks = (units + 255) / 256;
  delta_pack_kernel<E><<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>((const E*)p, st, (E*)to, heads, a.T, d, r, units);
  p = to;
  st = {(long long)heads * a.T * r, (long long)a.T * r, r};
}
template <typename E>
static void pack_all(DeltaArgs& a, bool backward, hipStream_t s) {
  if (a.qk_packed) {
    pack_one<E>(a.q, a.qs, a.qk_packed, a, a.Hk, a.dk, a.dkr, s);
    pack_one<E>(a.k, a.ks, (E*)a.qk_packed + (long)a.B * a.Hk * a.T * a.dkr, a, a.Hk, a.dk, a.dkr, s);
  }
  if (a.v_packed) {
    pack_one<E>(a.v, a.vs, a.v_packed, a, a.H, a.dv, a.dvr, s);
    if (backward) pack_one<E>(a.dO, a.dos, (E*)a.v_packed + (long)a.B * a.H * a.T * a.dvr, a, a.H, a.dv, a.dvr, s);
  }
}
void delta_pack(DeltaArgs& a, bool backward, hipStream_t s) {
  if (a.dtype == GLA_BF16) pack_all<bf16>(a, backward, s);
  else pack_all<float>(a, backward, s);
}

hipError_t launch_delta_fwd(DeltaArgs a, hipStream_t s) {
  delta_pack(a, false, s);
  if (a.dtype == GLA_BF16) delta_fwd_rows<bf16>(a, s);
  else delta_fwd_rows<float>(a, s);
  return hipGetLastError();
}

}  // namespace gla
