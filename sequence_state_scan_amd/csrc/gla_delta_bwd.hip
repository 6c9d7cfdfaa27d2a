// The gated delta rule by chunks of 64 tokens, backward (names as in gla_delta_fwd.hip).  With D1 the gradient of the
// state leaving a chunk:
//   dW = P^T dO + (e^(gamma_C - gamma) K) D1,   z = (I + beta B)^-T dW,   dV = beta z,   dbeta = z . delta
//   D0 = e^gamma_C D1 + (e^gamma Q)^T dO - (e^gamma K)^T dV
//   dQ = e^gamma dO S0^T + H K,   H = (dO W^T) . E on and below the diagonal
//   dK = H^T Q + (G + G^T) K - e^gamma dV S0^T + e^(gamma_C - gamma) W D1^T,   G = -(dV W^T) . E below it
//   dg_t = sum from the token on of (o . do - v . dv) + <S, D> at a later chunk's end, both up to the next reset
// (scaling a decay scales what the states before it give to the later outputs, and those are linear in v).
// delta_bwd_kernel walks a segment's chunks from its end, D in accumulators as the forward holds S; what it leaves
// (z, D1) lets delta_grad_kernel form every chunk's gradients on its own.  Segments as in the forward, with the
// forward's transitions.  Operands are split as in the forward; only the state entering a chunk and the gradient leaving it,
// which pass through memory, are one bf16 each in dq and dk, as those are rounded themselves: dq and dk are 1.78e-3 off in the
// 2-norm where their own rounding is 1.66e-3, up to 2.3e-3 where hardly anything decays (with W, dV, H and G one bf16 too 2.9e-3,
// for 27 us less of the gradients' 314; the states' second parts would be another 0.5 of 3.0 GB).
// What bounds it: HBM.  bf16, 16 heads of 16384 tokens, 128 x 128, P = 16, kernels traced one by one (954 us in all, where a
// call of both directions takes 910 in a row): state pass 112 us, chain 31, walk 140 (628 MB, 4.5 TB/s), delta_grad_kernel 314
// (1148 MB, 3.7 TB/s), dg 6; in the forward gates and inverses 59, state pass 109, chain 23, walk 160 (762 MB, 4.8 TB/s).
#include "gla_delta.hpp"
#include "gla_delta_scan.hpp"

namespace gla {
namespace delta {

template <typename E, int DK, int NW, bool STATE>
__global__ __launch_bounds__(64 * NW) void delta_bwd_kernel(DeltaArgs a) {
  constexpr int NT = 64 * NW, CB = DK / 16, CP = DK / 32, CW = 16 * NW, PARTS = Num<E>::PARTS;
  constexpr int FINE = !STATE && PARTS == 2 ? 3 : PARTS;  // parts of dW
  typedef Tile<E, DK> K;
  typedef Tile<E, CW> V;
  typedef Tile<E, C> M;
  __shared__ __attribute__((aligned(16))) E Ks[C * K::LD], Qs[C * K::LD], Os[C * V::LD];
  __shared__ __attribute__((aligned(16))) E Ts[PARTS][C * M::LD];  // P^T, then the transposed inverse in its place
  __shared__ __attribute__((aligned(16))) GateBlock gates;
  const int segments = STATE ? a.P - 1 : a.P, units = a.B * a.H * segments;  // the first one's own gradient: no use
  const int unit = blockIdx.x % units, tile = blockIdx.x / units;
  const int bh = unit / segments, seg = unit - bh * segments + STATE, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
  const int len = length_of(a, b), alive = (len + C - 1) / C;
  const int first = seg * a.L, end = min(first + a.L, alive);
  if (seg > 0 && first >= alive) return;
  const int lane = lane_id(), wave = wave_id(), n16 = lane & 15, g4 = lane >> 4, k8 = 8 * g4;
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

  arrived<CB>(D);

  const E* kp = (const E*)a.k + b * a.ks.b + hk * a.ks.h;
  const E* qp = (const E*)a.q + b * a.qs.b + hk * a.qs.h;
  const E* op = (const E*)a.dO + b * a.dos.b + h * a.dos.h + col0;
  const E* tp = (const E*)a.solveT + (long)bh * a.N * C * C;
  const float* gp = a.gates + (long)bh * a.N * kDeltaGates;
  const long plane = (long)a.B * a.H * a.N * C * C;
  TileIn<E, C, DK, NT> kin, qin;
  TileIn<E, C, CW, NT> oin;
  TileIn<E, C, C, NT> tin[PARTS];
  GateIn<NT> gin;
  const auto load_rows = [&](int n) {
    const long t0 = (long)n * C;
    const int left = len - n * C;
    kin.load(kp + t0 * a.ks.t, a.ks.t, left, a.dkr);
    qin.load(qp + t0 * a.qs.t, a.qs.t, left, a.dkr);
    oin.load(op + t0 * a.dos.t, a.dos.t, left, a.dvr - col0);
    gin.load(gp + (long)n * kDeltaGates);
  };
  const auto load_inverse = [&](int n) {
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].load(tp + part * plane + (long)n * C * C, C, C, C);
  };
  const auto meet = [&](int m) {  // <state, D> at a mark, for dg
    const long at = ((long)bh * (a.marks + 1) + m) * tiles + j / 16;
    f32x4 S[CB];
    load_regs<CB>(S, a.mark + at * DK * 16);
    arrived<CB>(S);
    float dot = 0.f;
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int i = 0; i < 4; ++i) dot = fmaf(S[cb][i], D[cb][i], dot);
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
    if (lane_id() == 0) a.carry[at] = dot;
  };
  if (first < end) {
    load_rows(end - 1);
    load_inverse(end - 1);
  }
  for (int n = end - 1; n >= first; --n) {
    __syncthreads();
    const int left = len - n * C;
    kin.store(Ks, left, a.dkr);
    qin.store(Qs, left, a.dkr);
    oin.store(Os, left, a.dvr - col0);
    gin.store(gates);
    __syncthreads();
    if (!STATE && cols && (n % kDeltaMarks == kDeltaMarks - 1 || n == alive - 1)) meet(n / kDeltaMarks + 1);
    const int lane = fresh_tid() & 63, n16 = lane & 15, g4 = lane >> 4, k8 = 8 * g4;  // (anew: see the forward)
    ScoreTiles<E, DK, NW, true> P;
    P.form(Qs, Ks, gates, wave, n16, g4);
    P.put(Ts, PARTS, wave, n16, g4);
    f32x4 dW[4], Y[4];
    {
      Split<E, 1> kf[2][4];
      const auto fetch = [&](int p) {
#pragma unroll
        for (int t = 0; t < 4; ++t) kf[p & 1][t].part[0] = K::row(Ks, row_of(t, n16), 32 * p + k8);
      };
      fetch(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) dW[t] = zero4();
#pragma unroll
      for (int p = 0; p < CP; ++p) {
        const Split<E> Do = split<E>(D[2 * p], D[2 * p + 1]);
        if (!STATE && cols)
          *reinterpret_cast<Frag<E>*>((E*)a.grad1 + ((((long)bh * a.N + n) * tiles + j / 16) * CP + p) * 512 + lane * 8) = Do.part[0];
        if (p + 1 < CP) fetch(p + 1);
        batch<E>();
        mma_tiles<E, 0, 4>(dW, kf[p & 1], Do);
        batch<E>();
      }
    }
    f32x4 late[4], beta[4], lead[4];
    Frag<E> dO[2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      late[t] = *reinterpret_cast<const f32x4*>(gates.late + row4_of(t, g4));
      beta[t] = *reinterpret_cast<const f32x4*>(gates.beta + row4_of(t, g4));
      lead[t] = *reinterpret_cast<const f32x4*>(gates.lead + row4_of(t, g4));
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) dO[p] = V::template col<false>(Os, 32 * p, 16 * wave, n16, g4);
    const float whole = gates.lead[C - 1];
    if (n > first) load_rows(n - 1);
    batch<E>();
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) dW[t][i] *= late[t][i];
    __syncthreads();  // P^T
    Split<E> F[2][4];
    const auto fetch = [&](int p) {
#pragma unroll
      for (int t = 0; t < 2 * p + 2; ++t)
#pragma unroll
        for (int part = 0; part < PARTS; ++part) F[p][t].part[part] = M::row(Ts[part], row_of(t, n16), 32 * p + k8);
    };
    fetch(0);
    fetch(1);
    batch<E>();
    mma_tiles<E, 0, 2>(dW, F[0], Split<E, 1>{{dO[0]}});
    mma_tiles<E, 0, 4>(dW, F[1], Split<E, 1>{{dO[1]}});
    __syncthreads();
#pragma unroll
    for (int part = 0; part < PARTS; ++part) tin[part].store(Ts[part], C, C);
    __syncthreads();
    if (n > first) load_inverse(n - 1);
    fetch(0);
    fetch(1);
    const Split<E, FINE> Wo[2] = {split<E, FINE>(dW[0], dW[1]), split<E, FINE>(dW[2], dW[3])};
#pragma unroll
    for (int t = 0; t < 4; ++t) Y[t] = zero4();
    batch<E>();
    mma_tiles<E, 0, 2>(Y, F[0], Wo[0]);
    mma_tiles<E, 0, 4>(Y, F[1], Wo[1]);
    batch<E>();
    {
      const int lane = fresh_tid() & 63, n16 = lane & 15, g4 = lane >> 4;
      constexpr int TILES = 2;  // of Q and of K, a batch
      Frag<E> qf[2][TILES], kf[2][TILES];
      const auto fetch = [&](int s) {
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
          const int kk = 32 * (s * TILES / CB), ch = row4_of(s * TILES % CB + i, 0);
          qf[s & 1][i] = K::template col<true>(Qs, kk, ch, n16, g4);
          kf[s & 1][i] = K::template col<true>(Ks, kk, ch, n16, g4);
        }
      };
      fetch(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) {  // z, then -e^gamma dV
        if (!STATE && cols) *reinterpret_cast<f32x4*>(a.z + ((((long)bh * a.N + n) * tiles + j / 16) * 4 + t) * 256 + lane * 4) = quad_transpose(Y[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) Y[t][i] *= -lead[t][i] * beta[t][i];
      }
      const Split<E> Yo[2] = {split<E>(Y[0], Y[1]), split<E>(Y[2], Y[3])};
      Split<E> Oo[2];  // e^gamma dO: its 8 tokens are those of tiles 2p and 2p + 1
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        f32x4 x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = lead[2 * p][i] * (float)dO[p][i];
          y[i] = lead[2 * p + 1][i] * (float)dO[p][4 + i];
        }
        Oo[p] = split<E>(x, y);
      }
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int i = 0; i < 4; ++i) D[cb][i] *= whole;
#pragma unroll
      for (int s = 0; s < 2 * CB / TILES; ++s) {
        if (s + 1 < 2 * CB / TILES) fetch(s + 1);
        batch<E>();
        const int p = s * TILES / CB;
#pragma unroll
        for (int part = PARTS - 1; part >= 0; --part) {
#pragma unroll
          for (int i = 0; i < TILES; ++i) D[s * TILES % CB + i] = mma(qf[s & 1][i], Oo[p].part[part], D[s * TILES % CB + i]);
#pragma unroll
          for (int i = 0; i < TILES; ++i) D[s * TILES % CB + i] = mma(kf[s & 1][i], Yo[p].part[part], D[s * TILES % CB + i]);
        }
        batch<E>();
      }
    }
  }
  if (!cols) return;
  if (!STATE && seg == 0 && alive > 0) meet(0);
  if (STATE) store_regs<CB>(D, a.seg + (((long)bh * a.P + seg) * tiles + j / 16) * DK * 16);
  else if (seg == 0 && a.dh0) store_state<CB>(D, a.dh0 + (long)bh * a.dk * a.dv, a.dk, a.dv, j + n16);
}

// One chunk's dq, dk, dv, dbeta and the terms of dg.  Waves w and w + 4 have 16 tokens, each half of the channels; one
// of them forms the tokens' rows of H, the other those of G.  The value columns come in blocks (dO, W, dV by rows, S0
// and D1 transposed), then K, Q, H and G take their place in LDS.  Products are transposed: a lane has eight channels of
// one token.  64 columns a block in bf16, 32 in float32 (75 and 104 KB of LDS).
template <typename E, int DK>
__global__ __launch_bounds__(512) void delta_grad_kernel(DeltaArgs a) {
  constexpr int NT = 512, CB = DK / 16, CH = CB / 2, CP = DK / 32, BC = sizeof(E) == 2 ? 64 : 32, UPR = BC / 8, PARTS = Num<E>::PARTS;
  typedef Tile<E, DK> K;
  typedef Tile<E, BC> V;
  typedef Tile<E, C> M;
  constexpr int STAGE = (1 + 2 * PARTS) * C * V::LD + 2 * BC * K::LD, LATER = 2 * C * K::LD + 2 * PARTS * C * M::LD;
  __shared__ __attribute__((aligned(16))) E lds[STAGE > LATER ? STAGE : LATER];
  __shared__ __attribute__((aligned(16))) GateBlock gates;
  // (W, dV, and later H and G: PARTS tiles each)
  E *Os = lds, *Ws = Os + C * V::LD, *Ys = Ws + PARTS * C * V::LD, *S0 = Ys + PARTS * C * V::LD, *D1 = S0 + BC * K::LD;
  E *Ks = lds, *Qs = Ks + C * K::LD, *HT = Qs + C * K::LD, *GT = HT + PARTS * C * M::LD;
  const int n = blockIdx.x % a.N, bh = blockIdx.x / a.N, b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
  const int len = length_of(a, b), lane = lane_id(), n16 = lane & 15, g4 = lane >> 4;
  const int wave = wave_id() & 3, half = wave_id() >> 2;  // half: channels CH * 16 half on, and G
  const long t0 = (long)n * C, chunk = (long)bh * a.N + n, row0 = chunk * C;  // row0: in the padded tensor
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
    for (int u = threadIdx.x; u < C * CP * 4; u += NT) {
      put(a.dq, a.dq_heads, u / (CP * 4), u % (CP * 4) * 8, zero4(), zero4());
      put(a.dk_, a.dk_heads, u / (CP * 4), u % (CP * 4) * 8, zero4(), zero4());
    }
    for (int u = threadIdx.x; u < rows * ((a.dv + 3) / 4); u += NT) {
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
  f32x4 dQ[CH], dK[CH], dS[CH], H[4];  // H: or G
#pragma unroll
  for (int cb = 0; cb < CH; ++cb) dQ[cb] = dK[cb] = dS[cb] = zero4();
#pragma unroll
  for (int t = 0; t < 4; ++t) H[t] = zero4();
  float at = 0.f, size = 0.f, db = 0.f;
  const int r = threadIdx.x / UPR, cc = threadIdx.x % UPR * 8;  // the lane's row and columns of a block
  for (int c0 = 0; c0 < a.DVP; c0 += BC) {
    constexpr int UNITS = BC * DK / 8, PER = UNITS / NT < 1 ? 1 : UNITS / NT;
    typedef E v8 __attribute__((ext_vector_type(8), aligned(16)));
    v8 s0[PER], d1[PER];
    const long st = (chunk * (a.DVP / 16) + c0 / 16) * DK * 16;
#pragma unroll
    for (int i = 0; i < PER; ++i) {  // every lane loads, as in TileIn
      const int u = min((int)threadIdx.x + i * NT, min(UNITS, (a.DVP - c0) * DK / 8) - 1);
      s0[i] = *reinterpret_cast<const v8*>((const E*)a.state0 + st + u * 8);
      d1[i] = *reinterpret_cast<const v8*>((const E*)a.grad1 + st + u * 8);
    }
    if (c0) __syncthreads();
    if (r < C) {
      const int c = c0 + cc;
      typedef short S8 __attribute__((ext_vector_type(8)));
      R8 x = {}, ov = {}, vv = {};
      S8 rest = {};
      f32x8 z = {}, d = {};
      const bool live = r < left && c < a.dv;
      {  // every lane loads, as in TileIn
        const int rr = min(r, min(left, rows) - 1), ci = c < a.dvr ? c : 0;
        x = *reinterpret_cast<const R8*>(dO + rr * a.dos.t + ci);
        vv = *reinterpret_cast<const R8*>(v + rr * a.vs.t + ci);
        if constexpr (sizeof(E) == 2) {
          const short* p = a.o_rest + (chunk * (a.DVP / 16) + ci / 16) * 1024 + (rr >> 4) * 256 + (16 * ((ci & 15) >> 2) + (rr & 15)) * 4;
          typedef short S4 __attribute__((ext_vector_type(4)));
          rest = __builtin_shufflevector(*reinterpret_cast<const S4*>(p), *reinterpret_cast<const S4*>(p + 64), 0, 1, 2, 3, 4, 5, 6, 7);
        }
        if (a.dv % 8 == 0) ov = *reinterpret_cast<const R8*>(o + (long)rr * a.dv + ci);
        else ov = load8_part<E>(o + (long)rr * a.dv + min(ci, a.dv - 1), min(a.dv - ci, 8));
        const int cz = c < a.DVP ? c : 0;
        const long p = (chunk * (a.DVP / 16) + cz / 16) * 1024 + rows_at(r, cz & 15);
        z = __builtin_shufflevector(load4(a.z + p), load4(a.z + p + 16), 0, 1, 2, 3, 4, 5, 6, 7);
        d = __builtin_shufflevector(load4(a.err + p), load4(a.err + p + 16), 0, 1, 2, 3, 4, 5, 6, 7);
      }
      const float beta = gates.beta[r];
      v8 w[PARTS], y[PARTS], ox;
      f32x4 y0, y1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (c >= a.DVP) z[e] = d[e] = 0.f;
        if (!live || c + e >= a.dv) x[e] = vv[e] = (E)0.f;
        const float yv = beta * z[e];
        float of = (float)ov[e];
        if constexpr (sizeof(E) == 2) of = with_rest(ov[e], rest[e]);
        if (!live || c + e >= a.dv) of = 0.f;
        at = fmaf((float)x[e], of, at);
        at = fmaf(-yv, (float)vv[e], at);
        size += fabsf((float)x[e] * of);
        size += fabsf(yv * (float)vv[e]);
        db = fmaf(z[e], d[e], db);
        (e < 4 ? y0 : y1)[e & 3] = yv;
        float wr = beta * d[e], yr = yv;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          w[part][e] = (E)wr;
          y[part][e] = (E)yr;
          wr -= (float)w[part][e];
          yr -= (float)y[part][e];
        }
        ox[e] = x[e];
      }
      *reinterpret_cast<v8*>(Os + V::at(r, cc)) = ox;
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        *reinterpret_cast<v8*>(Ws + part * C * V::LD + V::at(r, cc)) = w[part];
        *reinterpret_cast<v8*>(Ys + part * C * V::LD + V::at(r, cc)) = y[part];
      }
      if (r < rows && c < a.dv) {
        E* to = (E*)a.dv_ + ((long)bh * a.T + t0 + r) * a.dv + c;
        store4_part<E>(to, y0, a.dv - c);
        store4_part<E>(to + 4, y1, a.dv - c - 4);
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int u = threadIdx.x + i * NT, l = u & 63, col = u / (64 * CP) * 16 + (l & 15), at = K::at(col, 32 * (u / 64 % CP) + 8 * (l >> 4));
      if (UNITS % NT == 0 || u < UNITS) {
        *reinterpret_cast<v8*>(S0 + at) = c0 + col < a.DVP ? s0[i] : (v8){};
        *reinterpret_cast<v8*>(D1 + at) = c0 + col < a.DVP ? d1[i] : (v8){};
      }
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < BC / 32; ++p) {
      const int row = 16 * wave + n16, col = 32 * p + 8 * g4;
      const auto parts = [&](const E* tile, int r) {
        Split<E> s;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) s.part[part] = V::row(tile + part * C * V::LD, r, col);
        return s;
      };
      const Frag<E> fo = V::row(Os, row, col);
      const Split<E> fw = parts(Ws, row), fy = parts(Ys, row);
#pragma unroll
      for (int cb = 0; cb < CH; ++cb) {
        const int ch = row4_of(CH * half + cb, 0);
        const Frag<E> s = K::template col<true>(S0, 32 * p, ch, n16, g4);
        dQ[cb] = mma(s, fo, dQ[cb]);
        dS[cb] = mma(s, fy, dS[cb]);
        dK[cb] = mma(K::template col<true>(D1, 32 * p, ch, n16, g4), fw, dK[cb]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t <= wave) {
          const Split<E> w = parts(Ws, 16 * t + n16);
          H[t] = half ? mma(fy, w, H[t]) : mma(fo, w, H[t]);
        }
    }
  }
  TileIn<E, C, DK, NT> kin, qin;
  kin.load((const E*)a.k + b * a.ks.b + hk * a.ks.h + t0 * a.ks.t, a.ks.t, left, a.dkr);
  qin.load((const E*)a.q + b * a.qs.b + hk * a.qs.h + t0 * a.qs.t, a.qs.t, left, a.dkr);
  // the rows' sums
#pragma unroll
  for (int s = 1; s < UPR; s *= 2) {
    at += __shfl_xor(at, s);
    size += __shfl_xor(size, s);
    db += __shfl_xor(db, s);
  }
  if (cc == 0 && r < C) {
    *reinterpret_cast<float2*>(a.at + 2 * (row0 + r)) = r < left ? make_float2(at, size) : make_float2(0.f, 0.f);
    if (r < rows) a.dbeta[(long)bh * a.T + t0 + r] = r < left ? db : 0.f;
  }
  __syncthreads();
  kin.store(Ks, left, a.dkr);
  qin.store(Qs, left, a.dkr);
  // H^T and G^T: a lane has four queries of one key
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t > (wave | 1)) continue;
    const int key = 16 * t + n16, i0 = 16 * wave + 4 * g4;
    f32x4 x = half ? decays_to<false>(gates, i0, key) : decays_to<true>(gates, i0, key);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= half ? -H[t][i] : H[t][i];
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      M::put4((half ? GT : HT) + part * C * M::LD, key, i0, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] -= (float)(E)x[i];
    }
  }
  const int row = 16 * wave + n16;
  const float lead = gates.lead[row], late = gates.late[row];
#pragma unroll
  for (int cb = 0; cb < CH; ++cb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dQ[cb][i] *= lead;
      dK[cb][i] = fmaf(late, dK[cb][i], -lead * dS[cb][i]);
    }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const bool before = p <= wave / 2, after = p >= wave / 2;  // keys up to the wave's rows, queries from them on
    Split<E> hi = {}, gi = {}, hj = {}, gj = {};
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      const E *h = HT + part * C * M::LD, *g = GT + part * C * M::LD;
      if (before) {
        hi.part[part] = M::template col<false>(h, 32 * p, 16 * wave, n16, g4);
        gi.part[part] = M::template col<false>(g, 32 * p, 16 * wave, n16, g4);
      }
      if (after) {
        hj.part[part] = M::row(h, row, 32 * p + 8 * g4);
        gj.part[part] = M::row(g, row, 32 * p + 8 * g4);
      }
    }
#pragma unroll
    for (int cb = 0; cb < CH; ++cb) {
      const int ch = row4_of(CH * half + cb, 0);
      const Frag<E> kf = K::template col<true>(Ks, 32 * p, ch, n16, g4);
      if (before) {
        dQ[cb] = mma(kf, hi, dQ[cb]);
        dK[cb] = mma(kf, gi, dK[cb]);
      }
      if (after) {
        dK[cb] = mma(kf, gj, dK[cb]);
        dK[cb] = mma(K::template col<true>(Qs, 32 * p, ch, n16, g4), hj, dK[cb]);
      }
    }
  }
  // CH tiles: pairs of 8 channels a lane; one tile alone where a half has 16 channels
  if constexpr (CH % 2 == 0) {
#pragma unroll
    for (int p = 0; p < CH / 2; ++p) {
      put(a.dq, a.dq_heads, row, 32 * (CH / 2 * half + p) + 8 * g4, dQ[2 * p], dQ[2 * p + 1]);
      put(a.dk_, a.dk_heads, row, 32 * (CH / 2 * half + p) + 8 * g4, dK[2 * p], dK[2 * p + 1]);
    }
  } else {
    const int c = 8 * g4 + 4 * half;
    if (row < rows && c < a.dk) {
      const long to = ((long)bh * a.T + t0 + row) * a.dk + c;
      if (shared) {
        store4_part<float>(a.dq_heads + to, dQ[0], a.dk - c);
        store4_part<float>(a.dk_heads + to, dK[0], a.dk - c);
      } else {
        store4_part<E>((E*)a.dq + to, dQ[0], a.dk - c);
        store4_part<E>((E*)a.dk_ + to, dK[0], a.dk - c);
      }
    }
  }
}

// dg: the sums of `at` from a token to the next reset, where they end in zero, or to the next mark (256 tokens a workgroup),
// where they end in <S, D>.  A run of tokens between resets and marks has to sum up to what is known of its start, too:
// <S, D> at the mark before, or zero at a reset.  What it is off by is the errors' sum, and goes back to the run's tokens by
// the sizes of their terms.  That leaves the largest error in the middle of a run instead of a larger one at its start (bf16,
// 16 x 16: dg 7e-6 off instead of 1.1e-5; a mark every chunk 6.5e-6), and nothing of one document in another's dg.
__global__ __launch_bounds__(256) void delta_gate_grad_kernel(DeltaArgs a) {
  constexpr int SPAN = C * kDeltaMarks;
  static_assert(SPAN == 256, "a lane a token");
  const int m = blockIdx.x % a.marks, bh = blockIdx.x / a.marks, b = bh / a.H, h = bh - b * a.H;
  const int len = length_of(a, b), lane = lane_id(), wave = wave_id();
  const long t = (long)m * SPAN + threadIdx.x;
  __shared__ float first[2][4], total[2][SPAN];  // the sums (of `at`, of sizes) from a wave's first token; from every token
  __shared__ unsigned long long starts[4];       // a wave's resets
  float2 x = make_float2(0.f, 0.f);
  bool reset = false;
  if (t < len) {
    x = *reinterpret_cast<const float2*>(a.at + 2 * ((long)bh * a.N * C + t));
    reset = decay(a.g[b * a.gs.b + h * a.gs.h + t * a.gs.t]) == 0.f;
  }
  const unsigned long long here = __ballot(reset);
  const unsigned long long after = lane < 63 ? here >> (lane + 1) : 0;
  const int end = after ? lane + __ffsll((long long)after) : 64;  // of the lane's run, in its wave
  for (int o = 1; o < 64; o *= 2) {
    const float y = __shfl_down(x.x, o), size = __shfl_down(x.y, o);
    if (lane + o < end) {
      x.x += y;
      x.y += size;
    }
  }
  if (lane == 0) {
    first[0][wave] = x.x;
    first[1][wave] = x.y;
    starts[wave] = here;
  }
  __syncthreads();
  const float* c = a.carry + ((long)bh * (a.marks + 1) + m) * (a.DVP / 16);
  float before = 0.f, s = 0.f, size = 0.f;
  if (t < len) {
    float off = 0.f, whole = 0.f;  // from behind a wave to its last run's end
    for (int i = 0; i < a.DVP / 16; ++i) {
      before += c[i];
      off += c[a.DVP / 16 + i];
    }
    for (int w = 3; w > wave; --w) {
      const unsigned long long r = starts[w];
      off = r & 1 ? 0.f : r ? first[0][w] : off + first[0][w];
      whole = r & 1 ? 0.f : r ? first[1][w] : whole + first[1][w];
    }
    s = end < 64 ? x.x : off + x.x;
    size = end < 64 ? x.y : whole + x.y;
    total[0][threadIdx.x] = s;
    total[1][threadIdx.x] = size;
  }
  __syncthreads();
  if (t >= a.T) return;
  float dg = 0.f;
  if (t < len) {
    int from = 0;  // the run's first token
    const unsigned long long upto = here & (~0ull >> (63 - lane));
    if (upto) {
      from = 64 * wave + 63 - __clzll((long long)upto);
    } else {
      for (int w = wave - 1; w >= 0 && !from; --w)
        if (starts[w]) from = 64 * w + 63 - __clzll((long long)starts[w]);
    }
    if (starts[from >> 6] >> (from & 63) & 1) before = 0.f;
    const float off = before - total[0][from], whole = total[1][from];
    if (whole > 0.f && whole < __builtin_inff() && fabsf(off) < __builtin_inff()) s = fmaf(off, size / whole, s);
    if (!reset) dg = s;  // a decay of exactly zero has no slope
  }
  a.dg[(long)bh * a.T + t] = dg;
}

// dq and dk of a key head: the sums over its value heads, in their order.  (16 heads on 8, 4096 tokens of 64: 10 us, 4.2
// TB/s.)
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
    delta_scan_kernel<E, DK, true><<<heads * ((a.dv + 31) / 32), 4 * DK, 0, s>>>(a);
  }
  delta_bwd_kernel<E, DK, NW, false><<<heads * a.P * tiles, 64 * NW, 0, s>>>(a);
  delta_grad_kernel<E, DK><<<heads * a.N, 512, 0, s>>>(a);
  delta_gate_grad_kernel<<<heads * a.marks, 256, 0, s>>>(a);
  if (a.H != a.Hk) {
    const long long blocks = ((long long)a.B * a.Hk * a.T * a.dk + 255) / 256;
    delta_heads_kernel<E><<<dim3((unsigned)(blocks < 2048 ? blocks : 2048), 2), 256, 0, s>>>(a);
  }
}
template <typename E, int DK>
static void delta_bwd_cols(const DeltaArgs& a, hipStream_t s) {
  if (a.NW == 4) delta_bwd_run<E, DK, 4>(a, s);
  else delta_bwd_run<E, DK, 8>(a, s);
}
template <typename E>
static void delta_bwd_rows(const DeltaArgs& a, hipStream_t s) {
  if (a.DKP == 32) delta_bwd_cols<E, 32>(a, s);
  else if (a.DKP == 64) delta_bwd_cols<E, 64>(a, s);
  else delta_bwd_cols<E, 128>(a, s);
}

hipError_t launch_delta_bwd(DeltaArgs a, hipStream_t s) {
  delta_pack(a, true, s);
  if (a.dtype == GLA_BF16) delta_bwd_rows<bf16>(a, s);
  else delta_bwd_rows<float>(a, s);
  return hipGetLastError();
}

}  // namespace gla
