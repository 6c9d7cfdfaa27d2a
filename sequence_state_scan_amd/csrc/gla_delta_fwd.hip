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
#include "gla_delta.hpp"
#include "gla_delta_scan.hpp"

namespace gla {
namespace delta {

// ---------------------------------------------------------------------------------------- gates, inverse

// (I + L)^-1 of a unit lower triangular 64 x 64 matrix in float32: its 16 x 16 diagonal blocks by forward
// substitution, a column a lane, then joined two and two, X21 = -X22 L21 X11, on the float32 matrix instructions.
// Two of them at once: L = B beta (columns scaled) and, transposed at the end, L = beta B for the backward.
template <typename E, int DK, bool TRAIN>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a) {
  constexpr int LD = ld_of<E>(DK), LF = 66;
  constexpr int KBYTES = C * LD * sizeof(E), XBYTES = C * LF * 4;
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
  k.load((const E*)a.k + b * a.ks.b + (h / (a.H / a.Hk)) * a.ks.h + t0 * a.ks.t, a.ks.t, len - n * C, a.dk);
  if (wave == 0) {
    const long t = t0 + lane;
    const bool live = t < len;
    // below -200 every decay over the token is an exact zero
    double x = live ? fmaxf(a.g[b * a.gs.b + h * a.gs.h + t * a.gs.t], -200.f) : 0.f;
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
  k.store(Ks, LD);
  __syncthreads();
  // B, one row tile a wave
  for (int jt = 0; jt <= wave; ++jt) {
    f32x4 acc = zero4();
#pragma unroll
    for (int p = 0; p < DK / 32; ++p)
      acc = mma(row_frag(Ks + (16 * wave + n16) * LD + 32 * p + 8 * g4), row_frag(Ks + (16 * jt + n16) * LD + 32 * p + 8 * g4), acc);
    const int j = 16 * jt + n16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * wave + 4 * g4 + r;
      Bm[i * LF + j] = i > j ? acc[r] * decay_between(gates, i, j) : 0.f;
    }
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

// Workgroup: one segment and 16 NW columns.  STATE: the segment's own end state where another follows, and past the
// value columns its transition where another follows or, for the backward's chain, precedes.
template <typename E, int DK, int NW, int MODE>
__global__ __launch_bounds__(64 * NW) void delta_fwd_kernel(DeltaArgs a) {
  constexpr int NT = 64 * NW, CB = DK / 16, CP = DK / 32, CW = 16 * NW, PARTS = Num<E>::PARTS;
  constexpr int LD = ld_of<E>(DK), LV = ld_of<E>(CW), LT = ld_of<E>(C), FINE = MODE == TRAIN && PARTS == 2 ? 3 : PARTS;
  __shared__ __attribute__((aligned(16))) E Ks[C * LD], Vs[C * LV], Ts[PARTS][C * LT];
  __shared__ __attribute__((aligned(16))) E Qs[MODE == STATE ? 8 : C * LD], Ps[MODE == STATE ? 1 : PARTS][MODE == STATE ? 8 : C * LT];
  __shared__ __attribute__((aligned(16))) GateBlock gates;
  const bool chained = MODE == STATE && a.err;  // a backward follows
  const int segments = MODE == STATE && !chained ? a.P - 1 : a.P, units = a.B * a.H * segments;
  const int unit = blockIdx.x % units, tile = blockIdx.x / units;  // a segment's column tiles: the same XCD mostly
  const int bh = unit / segments, seg = unit - bh * segments, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
  const int len = length_of(a, b), alive = (len + C - 1) / C;
  const int first = seg * a.L, last = min(first + a.L, a.N), end = min(last, alive);
  const int lane = lane_id(), wave = wave_id(), n16 = lane & 15, g4 = lane >> 4;
  const int value_tiles = (a.dv + CW - 1) / CW;
  const bool transition = MODE == STATE && tile >= value_tiles;
  if (MODE == STATE && last >= alive && !(transition && chained && seg > 0 && first < alive)) return;
  const int col0 = (transition ? tile - value_tiles : tile) * CW, j = col0 + 16 * wave;  // the wave's columns
  const bool cols = j < (transition ? a.DKP : a.dv);

  f32x4 S[CB];
  if (MODE == STATE) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int i = 0; i < 4; ++i) S[cb][i] = transition && row4_of(cb, g4) + i == j + n16 ? 1.f : 0.f;
  } else if (a.P > 1) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) S[cb] = zero4();
    if (cols && (seg == 0 || first < alive)) load_regs<CB>(S, a.seg_in + (((long)bh * a.P + seg) * (a.DVP / 16) + j / 16) * DK * 16);
  } else {
    load_state<CB>(S, a.h0 ? a.h0 + (long)bh * a.dk * a.dv : nullptr, a.dk, a.dv, cols ? j + n16 : a.dv);
  }

  const E* kp = (const E*)a.k + b * a.ks.b + hk * a.ks.h;
  const E* qp = (const E*)a.q + b * a.qs.b + hk * a.qs.h;
  const E* vp = (const E*)a.v + b * a.vs.b + h * a.vs.h + col0;
  const E* tp = (const E*)a.solve + (long)bh * a.N * C * C;
  const float* gp = a.gates + (long)bh * a.N * kDeltaGates;
  const long plane = (long)a.B * a.H * a.N * C * C;
  TileIn<E, C, DK, NT> kin, qin;
  TileIn<E, C, CW, NT> vin;
  TileIn<E, C, C, NT> tin[PARTS];
  f32x4 gin = zero4();
  const auto load = [&](int n) {
    const long t0 = (long)n * C;
    const int left = len - n * C;
    kin.load(kp + t0 * a.ks.t, a.ks.t, left, a.dk);
    if (MODE != STATE) qin.load(qp + t0 * a.qs.t, a.qs.t, left, a.dk);
    vin.load(vp + t0 * a.vs.t, a.vs.t, transition ? 0 : left, a.dv - col0);
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].load(tp + part * plane + (long)n * C * C, C, C, C);
    if (threadIdx.x < kDeltaGates / 4) gin = reinterpret_cast<const f32x4*>(gp + (long)n * kDeltaGates)[threadIdx.x];
  };
  if (first < end) load(first);
  if constexpr (MODE != STATE)  // the blocks of P above the diagonal that the products read
    for (int u = threadIdx.x; u < PARTS * C * LT / 8; u += NT) reinterpret_cast<Frag<E>*>(&Ps[0][0])[u] = Frag<E>{};
  for (int n = first; n < end; ++n) {
    __syncthreads();
    kin.store(Ks, LD);
    if (MODE != STATE) qin.store(Qs, LD);
    vin.store(Vs, LV);
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].store(Ts[part], LT);
    if (threadIdx.x < kDeltaGates / 4) reinterpret_cast<f32x4*>(&gates)[threadIdx.x] = gin;
    __syncthreads();
    if (n + 1 < end) load(n + 1);
    if (MODE != STATE) {  // P's ten tiles, transposed products: a lane has four keys of one query
      for (int u = wave; u < 10; u += NW) {
        const int it = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : 3, jt = u - it * (it + 1) / 2;
        f32x4 acc = zero4();
#pragma unroll
        for (int p = 0; p < CP; ++p)
          acc = mma(row_frag(Ks + (16 * jt + n16) * LD + 32 * p + 8 * g4), row_frag(Qs + (16 * it + n16) * LD + 32 * p + 8 * g4), acc);
        const int i = 16 * it + n16, k0 = 16 * jt + 4 * g4;
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = k0 + r <= i ? acc[r] * decay_between(gates, i, k0 + r) : 0.f;
        if constexpr (PARTS == 2) {
          const bf16x4 hi = to_bf16x4(acc);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[r] -= (float)hi[r];
          *reinterpret_cast<bf16x4*>(&Ps[0][i * LT + k0]) = hi;
          *reinterpret_cast<bf16x4*>(&Ps[1][i * LT + k0]) = to_bf16x4(acc);
        } else {
          *reinterpret_cast<f32x4*>(&Ps[0][i * LT + k0]) = acc;
        }
      }
    }
    // V - e^gamma K S0
    Split<E> So[CP];
#pragma unroll
    for (int p = 0; p < CP; ++p) So[p] = split<E>(S[2 * p], S[2 * p + 1]);
    f32x4 Y[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 acc = zero4();
      const E* row = Ks + row_of(t, n16) * LD + 8 * g4;
#pragma unroll
      for (int p = 0; p < CP; ++p) acc = mma<E>(row_frag(row + 32 * p), So[p], acc);
      const int r0 = row4_of(t, g4);
      const f32x4 lead = *reinterpret_cast<const f32x4*>(gates.lead + r0);
      Y[t] = rows4<E>(Vs, LV, r0, 16 * wave);
#pragma unroll
      for (int i = 0; i < 4; ++i) Y[t][i] = fmaf(-lead[i], acc[i], Y[t][i]);
    }
    // delta, W and e^(gamma_C - gamma) W
    const Split<E, FINE> Yo[2] = {split<E, FINE>(Y[0], Y[1]), split<E, FINE>(Y[2], Y[3])};
    f32x4 W[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 acc = zero4();
#pragma unroll
      for (int p = 0; p <= t / 2; ++p) {
        Split<E> T;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) T.part[part] = row_frag(Ts[part] + row_of(t, n16) * LT + 32 * p + 8 * g4);
        acc = mma<E>(T, Yo[p], acc);
      }
      const int r0 = row4_of(t, g4);
      if (MODE == TRAIN && cols) store_rows(acc, a.err + (((long)bh * a.N + n) * C + r0) * a.DVP + j, a.DVP);
      const f32x4 beta = *reinterpret_cast<const f32x4*>(gates.beta + r0);
#pragma unroll
      for (int i = 0; i < 4; ++i) W[t][i] = beta[i] * acc[i];
    }
    if (MODE == TRAIN && cols) {
      E* to = (E*)a.state0 + (((long)bh * a.N + n) * a.DVP + j + n16) * DK + 8 * g4;
#pragma unroll
      for (int p = 0; p < CP; ++p) *reinterpret_cast<Frag<E>*>(to + 32 * p) = So[p].part[0];
    }
    if (MODE != STATE) {
      const Split<E, FINE> Wo[2] = {split<E, FINE>(W[0], W[1]), split<E, FINE>(W[2], W[3])};
      __syncthreads();
      // O, transposed products: a lane has four columns of one token.  A forward-only call rounds the state, W and P
      // to one bf16 here: o is rounded to it after all.
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4 acc = zero4();
        const int row = 16 * t + n16;
#pragma unroll
        for (int p = 0; p < CP; ++p) {
          const Frag<E> q = row_frag(Qs + row * LD + 32 * p + 8 * g4);
          acc = MODE == TRAIN ? mma<E>(So[p], q, acc) : mma(So[p].part[0], q, acc);
        }
        const float lead = gates.lead[row];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] *= lead;
#pragma unroll
        for (int p = 0; p <= t / 2; ++p) {
          Split<E> Pf;
#pragma unroll
          for (int part = 0; part < (MODE == TRAIN ? PARTS : 1); ++part) Pf.part[part] = row_frag(Ps[part] + row * LT + 32 * p + 8 * g4);
          acc = MODE == TRAIN ? mma<E>(Wo[p], Pf, acc) : mma(Wo[p].part[0], Pf.part[0], acc);
        }
        const long token = (long)n * C + row;
        if (cols && token < len) {
          store4_part<E>((E*)a.o + ((long)bh * a.T + token) * a.dv + j + 4 * g4, acc, a.dv - j - 4 * g4);
          if constexpr (MODE == TRAIN && PARTS == 2) {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            s16x4 rest;
#pragma unroll
            for (int i = 0; i < 4; ++i) rest[i] = rest_of(acc[i], (bf16)acc[i]);
            *reinterpret_cast<s16x4*>(a.o_rest + ((long)bh * a.N * C + token) * a.DVP + j + 4 * g4) = rest;
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4 late = *reinterpret_cast<const f32x4*>(gates.late + row4_of(t, g4));
#pragma unroll
      for (int i = 0; i < 4; ++i) W[t][i] *= late[i];
    }
    const Split<E> Wl[2] = {split<E>(W[0], W[1]), split<E>(W[2], W[3])};
    const float whole = gates.lead[C - 1];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) S[cb][i] *= whole;
#pragma unroll
      for (int p = 0; p < 2; ++p) S[cb] = mma<E>(col_frag<E, true>(Ks, LD, 32 * p, row4_of(cb, 0)), Wl[p], S[cb]);
    }
    if (MODE == TRAIN && cols && (n % kDeltaMarks == kDeltaMarks - 1 || n == alive - 1))
      store_regs<CB>(S, a.mark + (((long)bh * a.marks + n / kDeltaMarks) * (a.DVP / 16) + j / 16) * DK * 16);
  }
  if (!cols) return;
  if (MODE == STATE) {
    if (!transition) {
      store_regs<CB>(S, a.seg + (((long)bh * a.P + seg) * (a.DVP / 16) + j / 16) * DK * 16);
    } else {
      E* to = (E*)a.trans + ((long)bh * a.P + seg) * DK * DK + (long)(j + n16) * DK + 8 * g4;
      const long mplane = (long)a.B * a.H * a.P * DK * DK;
#pragma unroll
      for (int p = 0; p < CP; ++p) {
        const Split<E> s = split<E>(S[2 * p], S[2 * p + 1]);
#pragma unroll
        for (int part = 0; part < PARTS; ++part) *reinterpret_cast<Frag<E>*>(to + part * mplane + 32 * p) = s.part[part];
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
    delta_scan_kernel<E, DK, NW, false><<<heads * tiles, 64 * NW, 0, s>>>(a);
  }
  if (train) delta_fwd_kernel<E, DK, NW, TRAIN><<<heads * a.P * tiles, 64 * NW, 0, s>>>(a);
  else delta_fwd_kernel<E, DK, NW, INFER><<<heads * a.P * tiles, 64 * NW, 0, s>>>(a);
}
template <typename E, int DK>
static void delta_fwd_cols(const DeltaArgs& a, hipStream_t s) {
  if (a.dv <= 64) delta_fwd_run<E, DK, 4>(a, s);
  else delta_fwd_run<E, DK, 8>(a, s);
}
template <typename E>
static void delta_fwd_rows(const DeltaArgs& a, hipStream_t s) {
  if (a.DKP == 32) delta_fwd_cols<E, 32>(a, s);
  else if (a.DKP == 64) delta_fwd_cols<E, 64>(a, s);
  else delta_fwd_cols<E, 128>(a, s);
}

hipError_t launch_delta_fwd(const DeltaArgs& a, hipStream_t s) {
  if (a.dtype == GLA_BF16) delta_fwd_rows<bf16>(a, s);
  else delta_fwd_rows<float>(a, s);
  return hipGetLastError();
}

}  // namespace gla
