// The gated delta rule by chunks of 64 tokens, backward (names as in gla_delta_fwd.hip).  With D1 the gradient of the
// state leaving a chunk:
//   dW = P^T dO + (e^(gamma_C - gamma) K) D1,   z = (I + beta B)^-T dW,   dV = beta z,   dbeta = z . delta
//   D0 = e^gamma_C D1 + (e^gamma Q)^T dO - (e^gamma K)^T dV
//   dQ = e^gamma dO S0^T + H K,   H = (dO W^T) . E on and below the diagonal
//   dK = H^T Q + (G + G^T) K - e^gamma dV S0^T + e^(gamma_C - gamma) W D1^T,   G = -(dV W^T) . E below it
//   dg_t = sum over the later tokens of (o . do - v . dv) + <S, D> at a later chunk's end
// (scaling a decay scales what the states before it give to the later outputs, and those are linear in v).
// delta_bwd_kernel walks a segment's chunks from its end, D in accumulators as the forward holds S; what it leaves
// (z, D1) lets delta_grad_kernel form every chunk's gradients on its own.  Segments as in the forward, with the
// forward's transitions.  The float32 results (dg, dbeta, dh0) come from split operands throughout; the products
// that only go into dq and dk round the states, z and W to one bf16 each, as those are rounded themselves.
#include "gla_delta.hpp"
#include "gla_delta_scan.hpp"

namespace gla {
namespace delta {

template <typename E, int DK, int NW, bool STATE>
__global__ __launch_bounds__(64 * NW) void delta_bwd_kernel(DeltaArgs a) {
  constexpr int NT = 64 * NW, CB = DK / 16, CP = DK / 32, CW = 16 * NW, PARTS = Num<E>::PARTS;
  constexpr int LD = ld_of<E>(DK), LV = ld_of<E>(CW), LT = ld_of<E>(C), FINE = !STATE && PARTS == 2 ? 3 : PARTS;
  __shared__ __attribute__((aligned(16))) E Ks[C * LD], Qs[C * LD], Os[C * LV], Ts[PARTS][C * LT], Ps[PARTS][C * LT];
  __shared__ __attribute__((aligned(16))) GateBlock gates;
  const int segments = STATE ? a.P - 1 : a.P, units = a.B * a.H * segments;  // the first one's own gradient: no use
  const int unit = blockIdx.x % units, tile = blockIdx.x / units;
  const int bh = unit / segments, seg = unit - bh * segments + STATE, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
  const int len = length_of(a, b), alive = (len + C - 1) / C;
  const int first = seg * a.L, end = min(first + a.L, alive);
  if (seg > 0 && first >= alive) return;
  const int lane = lane_id(), wave = wave_id(), n16 = lane & 15, g4 = lane >> 4;
  const int col0 = tile * CW, j = col0 + 16 * wave;
  const bool cols = j < a.dv;
  const long tiles = a.DVP / 16;

  f32x4 D[CB];
  if (STATE || a.P > 1) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) D[cb] = zero4();
    if (!STATE && cols) load_regs<CB>(D, a.seg_in + (((long)bh * a.P + seg) * tiles + j / 16) * DK * 16);
  } else {
    load_state<CB>(D, a.dhT ? a.dhT + (long)bh * a.dk * a.dv : nullptr, a.dk, a.dv, cols ? j + n16 : a.dv);
  }

  const E* kp = (const E*)a.k + b * a.ks.b + hk * a.ks.h;
  const E* qp = (const E*)a.q + b * a.qs.b + hk * a.qs.h;
  const E* op = (const E*)a.dO + b * a.dos.b + h * a.dos.h + col0;
  const E* tp = (const E*)a.solveT + (long)bh * a.N * C * C;
  const float* gp = a.gates + (long)bh * a.N * kDeltaGates;
  const long plane = (long)a.B * a.H * a.N * C * C;
  TileIn<E, C, DK, NT> kin, qin;
  TileIn<E, C, CW, NT> oin;
  TileIn<E, C, C, NT> tin[PARTS];
  f32x4 gin = zero4();
  const auto load = [&](int n) {
    const long t0 = (long)n * C;
    const int left = len - n * C;
    kin.load(kp + t0 * a.ks.t, a.ks.t, left, a.dk);
    qin.load(qp + t0 * a.qs.t, a.qs.t, left, a.dk);
    oin.load(op + t0 * a.dos.t, a.dos.t, left, a.dv - col0);
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].load(tp + part * plane + (long)n * C * C, C, C, C);
    if (threadIdx.x < kDeltaGates / 4) gin = reinterpret_cast<const f32x4*>(gp + (long)n * kDeltaGates)[threadIdx.x];
  };
  if (first < end) load(end - 1);
  for (int u = threadIdx.x; u < PARTS * C * LT / 8; u += NT) reinterpret_cast<Frag<E>*>(&Ps[0][0])[u] = Frag<E>{};
  for (int n = end - 1; n >= first; --n) {
    __syncthreads();
    kin.store(Ks, LD);
    qin.store(Qs, LD);
    oin.store(Os, LV);
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].store(Ts[part], LT);
    if (threadIdx.x < kDeltaGates / 4) reinterpret_cast<f32x4*>(&gates)[threadIdx.x] = gin;
    __syncthreads();
    if (n > first) load(n - 1);
    // P^T's ten tiles: a lane has four queries of one key
    for (int u = wave; u < 10; u += NW) {
      const int it = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : 3, jt = u - it * (it + 1) / 2;
      f32x4 acc = zero4();
#pragma unroll
      for (int p = 0; p < CP; ++p)
        acc = mma(row_frag(Qs + (16 * it + n16) * LD + 32 * p + 8 * g4), row_frag(Ks + (16 * jt + n16) * LD + 32 * p + 8 * g4), acc);
      const int key = 16 * jt + n16, i0 = 16 * it + 4 * g4;
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = key <= i0 + r ? acc[r] * decay_between(gates, i0 + r, key) : 0.f;
      if constexpr (PARTS == 2) {
        const bf16x4 hi = to_bf16x4(acc);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] -= (float)hi[r];
        *reinterpret_cast<bf16x4*>(&Ps[0][key * LT + i0]) = hi;
        *reinterpret_cast<bf16x4*>(&Ps[1][key * LT + i0]) = to_bf16x4(acc);
      } else {
        *reinterpret_cast<f32x4*>(&Ps[0][key * LT + i0]) = acc;
      }
    }
    Split<E> Do[CP];
#pragma unroll
    for (int p = 0; p < CP; ++p) Do[p] = split<E>(D[2 * p], D[2 * p + 1]);
    if (!STATE && cols) {
      E* to = (E*)a.grad1 + (((long)bh * a.N + n) * a.DVP + j + n16) * DK + 8 * g4;
#pragma unroll
      for (int p = 0; p < CP; ++p) *reinterpret_cast<Frag<E>*>(to + 32 * p) = Do[p].part[0];
      if (n % kDeltaMarks == kDeltaMarks - 1 || n == alive - 1) {
        const long at = ((long)bh * a.marks + n / kDeltaMarks) * tiles + j / 16;
        f32x4 S[CB];
        load_regs<CB>(S, a.mark + at * DK * 16);
        float dot = 0.f;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
          for (int i = 0; i < 4; ++i) dot = fmaf(S[cb][i], D[cb][i], dot);
        for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
        if (lane == 0) a.carry[at] = dot;
      }
    }
    f32x4 dW[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 acc = zero4();
      const E* row = Ks + row_of(t, n16) * LD + 8 * g4;
#pragma unroll
      for (int p = 0; p < CP; ++p) acc = mma<E>(row_frag(row + 32 * p), Do[p], acc);
      const f32x4 late = *reinterpret_cast<const f32x4*>(gates.late + row4_of(t, g4));
#pragma unroll
      for (int i = 0; i < 4; ++i) dW[t][i] = late[i] * acc[i];
    }
    __syncthreads();  // P^T
    Frag<E> dO[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) dO[p] = col_frag<E, false>(Os, LV, 32 * p, 16 * wave);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int p = t / 2; p < 2; ++p) {
        Split<E> Pf;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) Pf.part[part] = row_frag(Ps[part] + row_of(t, n16) * LT + 32 * p + 8 * g4);
        dW[t] = mma<E>(Pf, dO[p], dW[t]);
      }
    const Split<E, FINE> Wo[2] = {split<E, FINE>(dW[0], dW[1]), split<E, FINE>(dW[2], dW[3])};
    f32x4 Y[4];  // -e^gamma dV
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 acc = zero4();
#pragma unroll
      for (int p = t / 2; p < 2; ++p) {
        Split<E> T;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) T.part[part] = row_frag(Ts[part] + row_of(t, n16) * LT + 32 * p + 8 * g4);
        acc = mma<E>(T, Wo[p], acc);
      }
      const int r0 = row4_of(t, g4);
      if (!STATE && cols) store_rows(acc, a.z + (((long)bh * a.N + n) * C + r0) * a.DVP + j, a.DVP);
      const f32x4 beta = *reinterpret_cast<const f32x4*>(gates.beta + r0), lead = *reinterpret_cast<const f32x4*>(gates.lead + r0);
#pragma unroll
      for (int i = 0; i < 4; ++i) Y[t][i] = -lead[i] * beta[i] * acc[i];
    }
    const Split<E> Yo[2] = {split<E>(Y[0], Y[1]), split<E>(Y[2], Y[3])};
    Split<E> Oo[2];  // e^gamma dO
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const f32x4 l0 = *reinterpret_cast<const f32x4*>(gates.lead + 32 * p + 8 * g4);
      const f32x4 l1 = *reinterpret_cast<const f32x4*>(gates.lead + 32 * p + 8 * g4 + 4);
      f32x4 x, y;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = l0[i] * (float)dO[p][i];
        y[i] = l1[i] * (float)dO[p][4 + i];
      }
      Oo[p] = split<E>(x, y);
    }
    const float whole = gates.lead[C - 1];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) D[cb][i] *= whole;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        D[cb] = mma<E>(col_frag<E, true>(Qs, LD, 32 * p, row4_of(cb, 0)), Oo[p], D[cb]);
        D[cb] = mma<E>(col_frag<E, true>(Ks, LD, 32 * p, row4_of(cb, 0)), Yo[p], D[cb]);
      }
    }
  }
  if (!cols) return;
  if (STATE) store_regs<CB>(D, a.seg + (((long)bh * a.P + seg) * tiles + j / 16) * DK * 16);
  else if (seg == 0 && a.dh0) store_state<CB>(D, a.dh0 + (long)bh * a.dk * a.dv, a.dk, a.dv, j + n16);
}

// One chunk's dq, dk, dv, dbeta and the terms of dg.  A wave has 16 tokens; the value columns come in blocks (dO, W,
// dV by rows, S0 and D1 transposed), then K and Q take their place in LDS.  Products are transposed: a lane has
// eight channels of one token.
template <typename E, int DK>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaArgs a) {
  constexpr int CB = DK / 16, CP = DK / 32, BC = sizeof(E) == 2 ? 64 : 32, UPR = BC / 8, PER = C * UPR / 256;
  constexpr int LD = ld_of<E>(DK), LC = ld_of<E>(BC), LT = ld_of<E>(C);
  constexpr int STAGE = 3 * C * LC + 2 * BC * LD, LATER = 2 * C * LD + 2 * C * LT;
  __shared__ __attribute__((aligned(16))) E lds[STAGE > LATER ? STAGE : LATER];
  __shared__ __attribute__((aligned(16))) GateBlock gates;
  E *Os = lds, *Ws = Os + C * LC, *Ys = Ws + C * LC, *S0 = Ys + C * LC, *D1 = S0 + BC * LD;
  E *Ks = lds, *Qs = Ks + C * LD, *HT = Qs + C * LD, *GT = HT + C * LT;
  const int n = blockIdx.x % a.N, bh = blockIdx.x / a.N, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
  const int len = length_of(a, b), lane = lane_id(), wave = wave_id(), n16 = lane & 15, g4 = lane >> 4;
  const long t0 = (long)n * C, row0 = (long)bh * a.N * C + t0;  // row0: in the padded tensors
  const int left = len - n * C, rows = min(C, a.T - n * C);     // rows of the chunk that exist
  const bool shared = a.H != a.Hk;
  const auto put = [&](void* out, float* heads, int row, int c, f32x4 x, f32x4 y) {
    if (row >= rows || c >= a.dk) return;
    const long at = ((long)bh * a.T + t0 + row) * a.dk + c;
    if (shared) {
      store4_part<float>(heads + at, x, a.dk - c);
      store4_part<float>(heads + at + 4, y, a.dk - c - 4);
    } else {
      store4_part<E>((E*)out + at, x, a.dk - c);
      store4_part<E>((E*)out + at + 4, y, a.dk - c - 4);
    }
  };
  if (left <= 0) {  // behind the sequence's end
    for (int u = threadIdx.x; u < C * CP * 4; u += 256) {
      put(a.dq, a.dq_heads, u / (CP * 4), u % (CP * 4) * 8, zero4(), zero4());
      put(a.dk_, a.dk_heads, u / (CP * 4), u % (CP * 4) * 8, zero4(), zero4());
    }
    for (int u = threadIdx.x; u < rows * ((a.dv + 3) / 4); u += 256) {
      const int r = u / ((a.dv + 3) / 4), c = (u - r * ((a.dv + 3) / 4)) * 4;
      store4_part<E>((E*)a.dv_ + ((long)bh * a.T + t0 + r) * a.dv + c, zero4(), a.dv - c);
    }
    if (threadIdx.x < rows) a.dbeta[(long)bh * a.T + t0 + threadIdx.x] = 0.f;
    return;
  }
  if (threadIdx.x < kDeltaGates / 4)
    reinterpret_cast<f32x4*>(&gates)[threadIdx.x] = reinterpret_cast<const f32x4*>(a.gates + ((long)bh * a.N + n) * kDeltaGates)[threadIdx.x];
  __syncthreads();
  const E* dO = (const E*)a.dO + b * a.dos.b + h * a.dos.h + t0 * a.dos.t;
  const E* v = (const E*)a.v + b * a.vs.b + h * a.vs.h + t0 * a.vs.t;
  const E* o = (const E*)a.o + ((long)bh * a.T + t0) * a.dv;
  typedef typename Raw<E, 8>::type R8;
  f32x4 dQ[CB], dK[CB], dS[CB], dP[4], G[4];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) dQ[cb] = dK[cb] = dS[cb] = zero4();
#pragma unroll
  for (int t = 0; t < 4; ++t) dP[t] = G[t] = zero4();
  float at[PER] = {}, db[PER] = {};
  for (int c0 = 0; c0 < a.DVP; c0 += BC) {
    if (c0) __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = threadIdx.x + i * 256, r = u / UPR, cc = u % UPR * 8, c = c0 + cc;
      typedef short S8 __attribute__((ext_vector_type(8)));
      R8 x = {}, ov = {}, vv = {};
      S8 rest = {};
      f32x8 z = {}, d = {};
      if (r < left && c < a.dv) {
        x = load8_part<E>(dO + r * a.dos.t + c, a.dv - c);
        ov = load8_part<E>(o + (long)r * a.dv + c, a.dv - c);
        vv = load8_part<E>(v + r * a.vs.t + c, a.dv - c);
        if (sizeof(E) == 2) rest = *reinterpret_cast<const S8*>(a.o_rest + (row0 + r) * a.DVP + c);
      }
      if (c < a.DVP) {
        z = row_frag(a.z + (row0 + r) * a.DVP + c);
        d = row_frag(a.err + (row0 + r) * a.DVP + c);
      }
      const float beta = gates.beta[r];
      typedef E v8 __attribute__((ext_vector_type(8), aligned(16)));
      v8 w, y, ox;
      f32x4 y0, y1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yv = beta * z[e];
        float of = (float)ov[e];
        if constexpr (sizeof(E) == 2) of = c + e < a.dv ? with_rest(ov[e], rest[e]) : 0.f;
        at[i] = fmaf((float)x[e], of, at[i]);
        at[i] = fmaf(-yv, (float)vv[e], at[i]);
        db[i] = fmaf(z[e], d[e], db[i]);
        (e < 4 ? y0 : y1)[e & 3] = yv;
        w[e] = (E)(beta * d[e]);
        y[e] = (E)yv;
        ox[e] = x[e];
      }
      *reinterpret_cast<v8*>(Os + r * LC + cc) = ox;
      *reinterpret_cast<v8*>(Ws + r * LC + cc) = w;
      *reinterpret_cast<v8*>(Ys + r * LC + cc) = y;
      if (r < rows && c < a.dv) {
        E* to = (E*)a.dv_ + ((long)bh * a.T + t0 + r) * a.dv + c;
        store4_part<E>(to, y0, a.dv - c);
        store4_part<E>(to + 4, y1, a.dv - c - 4);
      }
    }
    {
      const long st = (((long)bh * a.N + n) * a.DVP + c0) * DK;
      TileIn<E, BC, DK, 256> in;
      in.load((const E*)a.state0 + st, DK, a.DVP - c0, DK);
      in.store(S0, LD);
      in.load((const E*)a.grad1 + st, DK, a.DVP - c0, DK);
      in.store(D1, LD);
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < BC / 32; ++p) {
      const int off = (16 * wave + n16) * LC + 32 * p + 8 * g4;
      const Frag<E> fo = row_frag(Os + off), fw = row_frag(Ws + off), fy = row_frag(Ys + off);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        const Frag<E> s = col_frag<E, true>(S0, LD, 32 * p, row4_of(cb, 0));
        dQ[cb] = mma(s, fo, dQ[cb]);
        dS[cb] = mma(s, fy, dS[cb]);
        dK[cb] = mma(col_frag<E, true>(D1, LD, 32 * p, row4_of(cb, 0)), fw, dK[cb]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t <= wave) {
          const Frag<E> w = row_frag(Ws + (16 * t + n16) * LC + 32 * p + 8 * g4);
          dP[t] = mma(fo, w, dP[t]);
          G[t] = mma(fy, w, G[t]);
        }
    }
  }
  // the rows' sums
#pragma unroll
  for (int i = 0; i < PER; ++i) {
#pragma unroll
    for (int s = 1; s < UPR; s *= 2) {
      at[i] += __shfl_xor(at[i], s);
      db[i] += __shfl_xor(db[i], s);
    }
    const int u = threadIdx.x + i * 256, r = u / UPR;
    if (u % UPR == 0) {
      a.at[row0 + r] = r < left ? at[i] : 0.f;
      if (r < rows) a.dbeta[(long)bh * a.T + t0 + r] = r < left ? db[i] : 0.f;
    }
  }
  __syncthreads();
  {
    TileIn<E, C, DK, 256> in;
    in.load((const E*)a.k + b * a.ks.b + hk * a.ks.h + t0 * a.ks.t, a.ks.t, left, a.dk);
    in.store(Ks, LD);
    in.load((const E*)a.q + b * a.qs.b + hk * a.qs.h + t0 * a.qs.t, a.qs.t, left, a.dk);
    in.store(Qs, LD);
  }
  // H^T and G^T: a lane has four queries of one key
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t > (wave | 1)) continue;
    const int key = 16 * t + n16, i0 = 16 * wave + 4 * g4;
    f32x4 x, y;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float e = key <= i0 + r ? decay_between(gates, i0 + r, key) : 0.f;
      x[r] = dP[t][r] * e;
      y[r] = key < i0 + r ? -G[t][r] * e : 0.f;
    }
    if constexpr (sizeof(E) == 2) {
      *reinterpret_cast<bf16x4*>(HT + key * LT + i0) = to_bf16x4(x);
      *reinterpret_cast<bf16x4*>(GT + key * LT + i0) = to_bf16x4(y);
    } else {
      *reinterpret_cast<f32x4*>(HT + key * LT + i0) = x;
      *reinterpret_cast<f32x4*>(GT + key * LT + i0) = y;
    }
  }
  const int row = 16 * wave + n16;
  const float lead = gates.lead[row], late = gates.late[row];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dQ[cb][i] *= lead;
      dK[cb][i] = fmaf(late, dK[cb][i], -lead * dS[cb][i]);
    }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const bool before = p <= wave / 2, after = p >= wave / 2;  // keys up to the wave's rows, queries from them on
    Frag<E> hi = {}, gi = {}, hj = {}, gj = {};
    if (before) {
      hi = col_frag<E, false>(HT, LT, 32 * p, 16 * wave);
      gi = col_frag<E, false>(GT, LT, 32 * p, 16 * wave);
    }
    if (after) {
      hj = row_frag(HT + row * LT + 32 * p + 8 * g4);
      gj = row_frag(GT + row * LT + 32 * p + 8 * g4);
    }
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const Frag<E> kf = col_frag<E, true>(Ks, LD, 32 * p, row4_of(cb, 0));
      if (before) {
        dQ[cb] = mma(kf, hi, dQ[cb]);
        dK[cb] = mma(kf, gi, dK[cb]);
      }
      if (after) {
        dK[cb] = mma(kf, gj, dK[cb]);
        dK[cb] = mma(col_frag<E, true>(Qs, LD, 32 * p, row4_of(cb, 0)), hj, dK[cb]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < CP; ++p) {
    put(a.dq, a.dq_heads, row, 32 * p + 8 * g4, dQ[2 * p], dQ[2 * p + 1]);
    put(a.dk_, a.dk_heads, row, 32 * p + 8 * g4, dK[2 * p], dK[2 * p + 1]);
  }
}

// dg: the sums of `at` from a token to the next mark (256 tokens a workgroup), and <S, D> there.
__global__ __launch_bounds__(256) void delta_gate_grad_kernel(DeltaArgs a) {
  constexpr int SPAN = C * kDeltaMarks;
  static_assert(SPAN == 256, "a lane a token");
  const int m = blockIdx.x % a.marks, bh = blockIdx.x / a.marks, b = bh / a.H, h = bh - b * a.H;
  const int len = length_of(a, b), lane = lane_id(), wave = wave_id();
  const long t = (long)m * SPAN + threadIdx.x;
  __shared__ float red[4];
  float x = t < len ? a.at[(long)bh * a.N * C + t] : 0.f;
  for (int o = 1; o < 64; o *= 2) {
    const float y = __shfl_down(x, o);
    if (lane + o < 64) x += y;
  }
  if (lane == 0) red[wave] = x;
  __syncthreads();
  if (t >= a.T) return;
  float dg = 0.f;
  if (t < len) {
    const float g = a.g[b * a.gs.b + h * a.gs.h + t * a.gs.t];
    float carry = 0.f;
    const float* c = a.carry + ((long)bh * a.marks + m) * (a.DVP / 16);
    for (int i = 0; i < a.DVP / 16; ++i) carry += c[i];
    for (int w = 3; w > wave; --w) carry += red[w];
    if (decay(g) != 0.f) dg = x + carry;  // a decay of exactly zero has no slope
  }
  a.dg[(long)bh * a.T + t] = dg;
}

// dq and dk of a key head: the sums over its value heads, in their order.
template <typename E>
__global__ __launch_bounds__(256) void delta_heads_kernel(DeltaArgs a) {
  const int G = a.H / a.Hk;
  const long n = (long)a.T * a.dk, all = (long)a.B * a.Hk * n;
  const float* from = blockIdx.y ? a.dk_heads : a.dq_heads;
  E* to = (E*)(blockIdx.y ? a.dk_ : a.dq);
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long)gridDim.x * 256) {
    const long head = i / n, at = head * G * n + (i - head * n);
    float s = from[at];
    for (int g = 1; g < G; ++g) s += from[at + g * n];
    to[i] = (E)s;
  }
}

}  // namespace delta

using namespace delta;

template <typename E, int DK, int NW>
static void delta_bwd_run(const DeltaArgs& a, hipStream_t s) {
  constexpr int CW = 16 * NW;
  const int heads = a.B * a.H, tiles = (a.dv + CW - 1) / CW;
  if (a.P > 1) {
    delta_bwd_kernel<E, DK, NW, true><<<heads * (a.P - 1) * tiles, 64 * NW, 0, s>>>(a);
    delta_scan_kernel<E, DK, NW, true><<<heads * tiles, 64 * NW, 0, s>>>(a);
  }
  delta_bwd_kernel<E, DK, NW, false><<<heads * a.P * tiles, 64 * NW, 0, s>>>(a);
  delta_grad_kernel<E, DK><<<heads * a.N, 256, 0, s>>>(a);
  delta_gate_grad_kernel<<<heads * a.marks, 256, 0, s>>>(a);
  if (a.H != a.Hk) {
    const long long blocks = ((long long)a.B * a.Hk * a.T * a.dk + 255) / 256;
    delta_heads_kernel<E><<<dim3((unsigned)(blocks < 2048 ? blocks : 2048), 2), 256, 0, s>>>(a);
  }
}
template <typename E, int DK>
static void delta_bwd_cols(const DeltaArgs& a, hipStream_t s) {
  if (a.dv <= 64) delta_bwd_run<E, DK, 4>(a, s);
  else delta_bwd_run<E, DK, 8>(a, s);
}
template <typename E>
static void delta_bwd_rows(const DeltaArgs& a, hipStream_t s) {
  if (a.DKP == 32) delta_bwd_cols<E, 32>(a, s);
  else if (a.DKP == 64) delta_bwd_cols<E, 64>(a, s);
  else delta_bwd_cols<E, 128>(a, s);
}

hipError_t launch_delta_bwd(const DeltaArgs& a, hipStream_t s) {
  if (a.dtype == GLA_BF16) delta_bwd_rows<bf16>(a, s);
  else delta_bwd_rows<float>(a, s);
  return hipGetLastError();
}

}  // namespace gla
