// What joins a block's output y [B][H][T][d] to the residual stream [B][T][H d], forward and
// backward, one pass over the rows (b, t) each:
//   yn = y rsqrt(mean_d(y^2) + eps)          (per head; with w_post)
//   m = yn w_post act(z)                     (the gate: silu or sigmoid)
//   out = residual + scale m
//   normed = out rsqrt(mean(out^2) + eps) w_pre
// A row is spread over TPR lanes in slots of 8 elements (16 bytes of bf16; the loads are whole
// whatever the alignment, which the hardware takes, except a head's last slot where d is no
// multiple of 8: EVEN kernels know there is none).  A head takes LPH slots (its last ones are empty
// where d / 8 is not LPH): a power of 2 up to 64, so that a head's sum is a lane exchange inside an
// aligned group, or a multiple of 64, so that no wave's slots belong to two heads and a head's sum
// is a wave sum and a sum of LPH / 64 of them from LDS.  Slot s of a row is lane s % TPR, register
// s / TPR.  All arithmetic is float32, rounded once at the store; the backward recomputes out from
// y, z and the residual instead of reading its rounded value.
//
// Both are bound by HBM: forward 32768 rows of 4 heads of 256 bf16 (norm and gate) in 39.6 us, 5.1
// TB/s; backward 16384 rows of 16 heads of 128 bf16, everything on, in 117 us, 4.6 TB/s.
#include "gla_block.hpp"

namespace gla {

constexpr int VEC = 8;  // elements of a slot

struct JoinShape {
  int LPH, slots, TPR, NV, RPB;  // RPB rows per workgroup of TPR * RPB lanes
  float inv_d, inv_D;
};

static int pow2_up(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// Lanes of a workgroup, where a row takes fewer, and of a row at most.  Rows of more slots take two a
// lane (padded heads four): 8192 rows of 8192 forward bf16 190 us, float32 274; with 1024 lanes of
// one slot 198 and 293.  The backward's registers (one slot a lane 178 in bf16, 204 in float32; two 225
// and 256, where float32 spills 6 to 10) fit 8 waves on a CU.  Four slots a lane, which only padded heads
// reach, are far past them: the backward spills 293 to 812 and takes 1.0 ms for 8192 rows of 20 heads of
// 320 bf16, whose bytes need 0.18; the forward (190 to 242, no spill) 157 us.
constexpr int kJoinThreads = 256, kJoinLanes = 512;
// A lane has at most four slots.  Heads of up to 8 values take one each, kJoinMaxHeads at most.  One of
// n = ceil(d / 8) > 1 slots is padded to at most 2 (n - 1), fewer than 2 d / 8, so a row of such heads has
// fewer than 2 kJoinMaxRow / 8.
static_assert(kJoinMaxHeads <= 4 * kJoinLanes && 2 * kJoinMaxRow / VEC <= 4 * kJoinLanes, "a lane's slots");

static JoinShape join_shape(int H, int d) {
  JoinShape s;
  const int n = (d + VEC - 1) / VEC;
  s.LPH = n <= 64 ? pow2_up(n) : (n + 63) / 64 * 64;
  s.slots = H * s.LPH;
  s.TPR = pow2_up(s.slots);
  if (s.TPR > kJoinLanes) s.TPR = kJoinLanes;
  s.NV = pow2_up((s.slots + s.TPR - 1) / s.TPR);
  s.RPB = s.TPR >= kJoinThreads ? 1 : kJoinThreads / s.TPR;
  s.inv_d = 1.f / d;
  s.inv_D = 1.f / (H * d);
  return s;
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

// Every slot's head sum, in place.  red: 2 x NV * 16 floats of LDS, in turn as above.
template <int NV>
__device__ __forceinline__ void head_sums(float (&v)[NV], const JoinShape& p, int lane, float* red, int turn) {
  if (p.LPH <= 64) {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = lane_sum(v[j], p.LPH);
    return;
  }
  red += turn * 16 * NV;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const float s = lane_sum(v[j], 64);
    if ((threadIdx.x & 63) == 0) red[j * 16 + (threadIdx.x >> 6)] = s;
  }
  __syncthreads();
  const int wpr = p.TPR / 64, w0 = (threadIdx.x >> 6) / wpr * wpr, m = p.LPH / 64;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int chunk = (lane + j * p.TPR) / 64, first = chunk / m * m;  // a head's m wave sums, in slot order
    float s = 0.f;
    for (int i = first; i < first + m; ++i)
      if (i < NV * wpr) s += red[i / wpr * 16 + w0 + i % wpr];
    v[j] = s;
  }
}

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
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

// A lane's slots of a row: the same for every row.
template <int NV>
struct Slots {
  int at[NV], in[NV], head[NV], left[NV];  // column in the row, in the head (-1: an empty slot), head, elements
};
template <int NV>
__device__ __forceinline__ Slots<NV> row_slots(const JoinArgs& a, const JoinShape& p, int lane) {
  Slots<NV> r;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int s = lane + j * p.TPR, h = s / p.LPH, i = (s - h * p.LPH) * VEC;
    r.in[j] = h < a.H && i < a.d ? i : -1;
    r.at[j] = h * a.d + i;
    r.head[j] = h;
    r.left[j] = a.d - i;
  }
  return r;
}

// w's values at a slot, ones where there is no w.
template <bool EVEN>
__device__ __forceinline__ void load_weights(const float* w, int at, int in, int left, float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = 1.f;
  if (w && in >= 0) {
    const auto r = load_slot<EVEN, float>(w + at, left);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r[i];
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

// Hides where a value comes from, so that what is formed from it before is formed again after
// instead of being held in registers.
template <typename T>
__device__ __forceinline__ void forget(T& v) {
  typedef unsigned words __attribute__((ext_vector_type(sizeof(T) / 4)));
  words w = __builtin_bit_cast(words, v);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 4; ++i) {
    unsigned x = w[i];
    asm volatile("" : "+v"(x));
    w[i] = x;
  }
  v = __builtin_bit_cast(T, w);
}

// One row's inputs as they lie in memory (bf16 stays packed).
template <typename E, typename R, int NV, bool BWD, bool EVEN>
struct RowIn {
  typename Pack<E>::raw y[NV], z[NV], dn[BWD ? NV : 1];
  typename Pack<R>::raw r[NV], dout[BWD ? NV : 1];
  float ry[BWD ? NV : 1], rp;
  __device__ __forceinline__ void forget_all() {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      forget(y[j]);
      forget(z[j]);
      forget(r[j]);
      forget(dn[j]);
    }
  }
  __device__ __forceinline__ void load(const JoinArgs& a, const Slots<NV>& s, const RowStep& at) {
    const long b = at.b, t = at.t;
    if constexpr (BWD) rp = a.d_normed ? a.rstd_pre[at.row] : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (s.in[j] < 0) continue;
      const int c = s.at[j], left = s.left[j];
      y[j] = load_slot<EVEN>((const E*)a.y + b * a.ys.b + s.head[j] * a.ys.h + t * a.ys.t + s.in[j], left);
      if (a.z) z[j] = load_slot<EVEN>((const E*)a.z + b * a.zs.b + t * a.zs.t + c, left);
      if (a.residual) r[j] = load_slot<EVEN>((const R*)a.residual + b * a.rs.b + t * a.rs.t + c, left);
      if constexpr (BWD) {
        ry[j] = a.w_post ? a.rstd_post[at.row * a.H + s.head[j]] : 1.f;
        if (a.d_normed) dn[j] = load_slot<EVEN>((const E*)a.d_normed + b * a.dns.b + t * a.dns.t + c, left);
        if (a.d_out) dout[j] = load_slot<EVEN>((const R*)a.d_out + b * a.dos.b + t * a.dos.t + c, left);
      }
    }
  }
};

// The weights at a lane's slots and the next row's inputs are held in registers (a row ahead of
// their use) where a lane has one slot.  With more (LEAN) the weights are loaded when they are used,
// and the next row's inputs once this row's are used up, before its last reduction.  In the forward that
// is a trade: 8192 rows of 8192 bf16 192 us, 196 with the loads at the row's end; of 20 heads of 320 159
// and 166; but one head of float32 loses (8192 wide 275 and 258, 5120 wide 172 and 162).
template <bool LEAN, bool EVEN, int NV>
struct Weights {
  float post[LEAN ? 1 : NV][VEC], scale[LEAN ? 1 : NV][VEC], pre[LEAN ? 1 : NV][VEC];
  __device__ __forceinline__ Weights(const JoinArgs& a, const Slots<NV>& s) {
    if constexpr (!LEAN)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        load_weights<EVEN>(a.w_post, s.in[j], s.in[j], s.left[j], post[j]);
        load_weights<EVEN>(a.scale, s.at[j], s.in[j], s.left[j], scale[j]);
        load_weights<EVEN>(a.w_pre, s.at[j], s.in[j], s.left[j], pre[j]);
      }
  }
  __device__ __forceinline__ void get(const float* w, const float (&held)[LEAN ? 1 : NV][VEC], int at, int in, int left,
                                      int j, float (&v)[VEC]) const {
    if constexpr (LEAN) {
      load_weights<EVEN>(w, at, in, left, v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = held[j][i];
    }
  }
};

template <typename E, typename R, int NV, int NT, bool EVEN>
__global__ __launch_bounds__(NT) void join_fwd_kernel(JoinArgs a, JoinShape p) {
  constexpr bool LEAN = NV > 1;
  __shared__ float red[2 * 16], hred[2 * 16 * NV];
  const int D = a.H * a.d;
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T, step = (long)gridDim.x * p.RPB;
  const Slots<NV> s = row_slots<NV>(a, p, lane);
  const Weights<LEAN, EVEN, NV> w(a, s);
  RowStep at((long)blockIdx.x * p.RPB + sub, a.T, step);
  RowIn<E, R, NV, false, EVEN> in, next;
  if (at.row < rows) in.load(a, s, at);
  int turn = 0;
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += step, turn ^= 1) {
    const RowStep here = at;
    const bool live = here.row < rows;
    at.next(a.T, step);
    if (!LEAN && at.row < rows) next.load(a, s, at);
    float y[NV][VEC], hs[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      hs[j] = 0.f;
      const bool have = live && s.in[j] >= 0;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        y[j][v] = have ? (float)in.y[j][v] : 0.f;
        hs[j] = fmaf(y[j][v], y[j][v], hs[j]);
      }
    }
    if (a.w_post) {
      head_sums<NV>(hs, p, lane, hred, turn);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const float r = rsqrtf(hs[j] * p.inv_d + a.eps);
        if (a.rstd_post && live && s.in[j] == 0) a.rstd_post[here.row * a.H + s.head[j]] = r;
        float wv[VEC];
        w.get(a.w_post, w.post, s.in[j], s.in[j], s.left[j], j, wv);
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] *= r * wv[v];
      }
    }
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || s.in[j] < 0) continue;
      float sc[VEC];
      w.get(a.scale, w.scale, s.at[j], s.in[j], s.left[j], j, sc);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (a.z) {
          const float z = (float)in.z[j][v], g = sigmoid(z);
          y[j][v] *= a.act == GLA_ACT_SILU ? z * g : g;
        }
        y[j][v] = fmaf(sc[v], y[j][v], a.residual ? (float)in.r[j][v] : 0.f);
        sq = fmaf(y[j][v], y[j][v], sq);
      }
      store_slot<EVEN>((R*)a.out + here.row * D + s.at[j], y[j], s.left[j]);
    }
    if (LEAN && at.row < rows) in.load(a, s, at);
    if (a.w_pre) {
      const float r = rsqrtf(row_sum(sq, p.TPR, red, turn) * p.inv_D + a.eps);
      if (a.rstd_pre && live && lane == 0) a.rstd_pre[here.row] = r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!live || s.in[j] < 0) continue;
        float wv[VEC];
        w.get(a.w_pre, w.pre, s.at[j], s.in[j], s.left[j], j, wv);
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] *= r * wv[v];
        store_slot<EVEN>((E*)a.normed + here.row * D + s.at[j], y[j], s.left[j]);
      }
    }
    if constexpr (!LEAN) in = next;
  }
}

// One pass over the rows: recomputes yn, m and out from y, z and the residual, then
//   n = out rp,  e = dn w_pre,  dO = d_out + rp (e - n mean(e n))         d_residual = dO
//   dz = dO scale yn w_post act'(z),  du = dO scale act(z),  e' = du w_post
//   dy = ry (e' - yn mean_d(e' yn))
// and adds up the weights' gradients dn n, dO m, du yn over its rows in registers, then over the
// workgroup's RPB rows and for w_post the heads in LDS; partial: [workgroup][3][D], summed in
// order by join_sum_kernel.  With two slots a lane what the sum over the row stands between is formed
// on both sides of it from the packed inputs, not held: 8192 rows of 8192 float32 533 us, 834 with it
// held (and spilled by the hundred) and no row loaded ahead; with one slot, where it fits, holding it is faster
// (32768 rows of 1024 bf16 121 us, 142 formed twice).
template <typename E, typename R, int NV, int NT, bool EVEN>
__global__ __launch_bounds__(NT) void join_bwd_kernel(JoinArgs a, JoinShape p) {
  constexpr bool LEAN = NV > 1;
  extern __shared__ float lds[];
  float *red = lds, *hred = lds + 32;  // 2 x 16, 2 x 16 NV floats, then RPB rows for the last sums
  const int D = a.H * a.d;
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T, step = (long)gridDim.x * p.RPB;
  const Slots<NV> s = row_slots<NV>(a, p, lane);
  const Weights<LEAN, EVEN, NV> w(a, s);
  float spre[NV][VEC] = {}, sscale[NV][VEC] = {}, spost[NV][VEC] = {};
  RowStep at((long)blockIdx.x * p.RPB + sub, a.T, step);
  RowIn<E, R, NV, true, EVEN> in, next;
  if (at.row < rows) in.load(a, s, at);
  int turn = 0;
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += step, turn ^= 1) {
    const RowStep here = at;
    const bool live = here.row < rows;
    at.next(a.T, step);
    if (!LEAN && at.row < rows) next.load(a, s, at);
    float yn[NV][VEC], f[NV][VEC], n[NV][VEC], e[NV][VEC], hs[NV];  // f: sigmoid(z), e: d_normed w_pre
    const auto form = [&](int j) {
      float wpost[VEC], scale[VEC], wpre[VEC];
      if (a.d_normed) {
        w.get(a.w_post, w.post, s.in[j], s.in[j], s.left[j], j, wpost);
        w.get(a.scale, w.scale, s.at[j], s.in[j], s.left[j], j, scale);
        w.get(a.w_pre, w.pre, s.at[j], s.in[j], s.left[j], j, wpre);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        yn[j][v] = (float)in.y[j][v] * in.ry[j];
        f[j][v] = a.z ? sigmoid((float)in.z[j][v]) : 1.f;
        n[j][v] = e[j][v] = 0.f;
        if (a.d_normed) {
          float m = yn[j][v] * wpost[v] * f[j][v];
          if (a.z && a.act == GLA_ACT_SILU) m *= (float)in.z[j][v];
          n[j][v] = fmaf(scale[v], m, a.residual ? (float)in.r[j][v] : 0.f) * in.rp;
          e[j][v] = (float)in.dn[j][v] * wpre[v];
        }
      }
    };
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || s.in[j] < 0) continue;
      form(j);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (a.d_normed) {
          spre[j][v] = fmaf((float)in.dn[j][v], n[j][v], spre[j][v]);
          dot = fmaf(e[j][v], n[j][v], dot);
        }
    }
    if (a.d_normed) dot = row_sum(dot, p.TPR, red, turn) * p.inv_D;
    if constexpr (LEAN) in.forget_all();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      hs[j] = 0.f;
      if (!live || s.in[j] < 0) continue;
      if constexpr (LEAN) form(j);
      float wpost[VEC], scale[VEC], dO[VEC], dz[VEC];
      w.get(a.w_post, w.post, s.in[j], s.in[j], s.left[j], j, wpost);
      w.get(a.scale, w.scale, s.at[j], s.in[j], s.left[j], j, scale);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        dO[v] = a.d_out ? (float)in.dout[j][v] : 0.f;
        if (a.d_normed) dO[v] = fmaf(in.rp, fmaf(-n[j][v], dot, e[j][v]), dO[v]);
      }
      if (a.d_residual) store_slot<EVEN>((R*)a.d_residual + here.row * D + s.at[j], dO, s.left[j]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float u = yn[j][v] * wpost[v];
        float act = 1.f, slope = 0.f;
        if (a.z) {
          const float z = (float)in.z[j][v], g = f[j][v];
          act = a.act == GLA_ACT_SILU ? z * g : g;
          slope = a.act == GLA_ACT_SILU ? g * fmaf(z, 1.f - g, 1.f) : g * (1.f - g);
        }
        sscale[j][v] = fmaf(dO[v], u * act, sscale[j][v]);
        dO[v] *= scale[v];
        dz[v] = dO[v] * u * slope;
        dO[v] *= act;  // du
        spost[j][v] = fmaf(dO[v], yn[j][v], spost[j][v]);
        e[j][v] = dO[v] * wpost[v];
        hs[j] = fmaf(e[j][v], yn[j][v], hs[j]);
      }
      if (a.z) store_slot<EVEN>((E*)a.dz + here.row * D + s.at[j], dz, s.left[j]);
    }
    typename Pack<E>::raw yk[NV];
    float ryk[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      yk[j] = in.y[j];
      ryk[j] = in.ry[j];
    }
    if (LEAN && at.row < rows) in.load(a, s, at);
    if (a.w_post) head_sums<NV>(hs, p, lane, hred, turn);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || s.in[j] < 0) continue;
      if (a.w_post) {
        const float mean = hs[j] * p.inv_d;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          e[j][v] = ryk[j] * fmaf(LEAN ? -(float)yk[j][v] * ryk[j] : -yn[j][v], mean, e[j][v]);
      }
      store_slot<EVEN>((E*)a.dy + (((long)here.b * a.H + s.head[j]) * a.T + here.t) * a.d + s.in[j], e[j], s.left[j]);
    }
    if constexpr (!LEAN) in = next;
  }
  if (!a.partial) return;
  // the workgroup's sums, through LDS where several rows (and for w_post heads) add up
  float* sums = lds + 32 + 32 * NV;  // [RPB][D]
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (!(which == 0 ? (void*)a.dw_pre : which == 1 ? (void*)a.dscale : (void*)a.dw_post)) continue;
    const int cols = which == 2 ? a.d : D, terms = which == 2 ? p.RPB * a.H : p.RPB;
    float* to = a.partial + ((long)blockIdx.x * 3 + which) * D;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (s.in[j] < 0) continue;
      const float(&acc)[VEC] = which == 0 ? spre[j] : which == 1 ? sscale[j] : spost[j];
      if (terms > 1) {
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (EVEN || v < s.left[j]) sums[sub * D + s.at[j] + v] = acc[v];
      } else {
        store_slot<EVEN>(to + s.at[j], acc, s.left[j]);
      }
    }
    if (terms == 1) continue;
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      float v = 0.f;
      for (int i = 0; i < terms; ++i) v += sums[i * cols + c];
      to[c] = v;
    }
  }
}

// The weights' gradients from the workgroups' partial sums, each added up in one order whatever
// the timing.  A workgroup has 64 columns of one gradient; each of its 16 waves adds every 16th
// of the G partial rows, 8 loads in flight.
__global__ __launch_bounds__(1024) void join_sum_kernel(JoinArgs a, int G) {
  const int D = a.H * a.d, which = blockIdx.y;
  float* out = which == 0 ? a.dw_pre : which == 1 ? a.dscale : a.dw_post;
  const int cols = which == 2 ? a.d : D;
  const int lane = threadIdx.x & 63, c = blockIdx.x * 64 + lane, part = threadIdx.x >> 6;
  if (!out || (int)blockIdx.x * 64 >= cols) return;
  __shared__ float red[16][64];
  float s = 0.f;
  const float* from = a.partial + (long)which * D + c;
  if (c < cols) {
    int g = part;
    for (; g + 7 * 16 < G; g += 8 * 16) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = from[(long)(g + 16 * i) * 3 * D];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; g < G; g += 16) s += from[(long)g * 3 * D];
  }
  red[part][lane] = s;
  __syncthreads();
  if (part == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    out[c] = s;
  }
}

// The most workgroups (of 256 lanes; half as many of 512), each of which leaves a row of partial sums
// backward.  Measured on 16k rows of 2048, forward and backward together: backward 512 x 256 lanes
// 184 us, 256 x 256 238, 384 202, 768 208, 1024 189, 512 x 512 198; on 32k rows of 1024 forward:
// 1024 x 256 38.2 us, 2048 41.8, 4096 42.9.  Elsewhere alike, half and twice as many (us): backward of 131072
// rows of 256 bf16 114, 166 and 121; 8192 of 8192 392, 738 and 403; 500000 of 24 58, 88 and 64; 4096 of 8 heads
// of 64 float32 22.5, 23.3 and 27.8; forward 66, 70 and 67; 197, 264 and 197; 26, 33 and 27; 10.6, 11.8 and
// 10.5; only 16384 of 2048 float32 would take fewer (132, 125 and 131).
constexpr int kBwdGroups = 512, kFwdGroups = 1024;

static int join_groups(long long rows, const JoinShape& p, int most) {
  const long long n = (rows + p.RPB - 1) / p.RPB;
  most = most * kJoinThreads / (p.TPR * p.RPB);
  return (int)(n < most ? n : most);
}

size_t join_partial_floats(int B, int H, int T, int d) {
  return (size_t)join_groups((long long)B * T, join_shape(H, d), kBwdGroups) * 3 * H * d;
}

template <typename E, typename R, bool EVEN>
static void join_fwd_run(const JoinArgs& a, hipStream_t s) {
  const JoinShape p = join_shape(a.H, a.d);
  const int G = join_groups((long long)a.B * a.T, p, kFwdGroups), threads = p.TPR * p.RPB;
  if (threads == 256) join_fwd_kernel<E, R, 1, 256, EVEN><<<G, threads, 0, s>>>(a, p);
  else if (p.NV == 1) join_fwd_kernel<E, R, 1, 512, EVEN><<<G, threads, 0, s>>>(a, p);
  else if (p.NV == 2) join_fwd_kernel<E, R, 2, 512, EVEN><<<G, threads, 0, s>>>(a, p);
  else join_fwd_kernel<E, R, 4, 512, EVEN><<<G, threads, 0, s>>>(a, p);
}

template <typename E, typename R, bool EVEN>
static void join_bwd_run(const JoinArgs& a, hipStream_t s) {
  const JoinShape p = join_shape(a.H, a.d);
  const int G = join_groups((long long)a.B * a.T, p, kBwdGroups), threads = p.TPR * p.RPB;
  const size_t lds = (32 + 32 * p.NV + (a.partial && (p.RPB > 1 || a.dw_post) ? p.RPB * a.H * a.d : 0)) * sizeof(float);
  if (threads == 256) join_bwd_kernel<E, R, 1, 256, EVEN><<<G, threads, lds, s>>>(a, p);
  else if (p.NV == 1) join_bwd_kernel<E, R, 1, 512, EVEN><<<G, threads, lds, s>>>(a, p);
  else if (p.NV == 2) join_bwd_kernel<E, R, 2, 512, EVEN><<<G, threads, lds, s>>>(a, p);
  else join_bwd_kernel<E, R, 4, 512, EVEN><<<G, threads, lds, s>>>(a, p);
  if (a.partial) join_sum_kernel<<<dim3((a.H * a.d + 63) / 64, 3), 1024, 0, s>>>(a, G);
}

template <typename E, typename R, bool EVEN>
static void join_rows(const JoinArgs& a, bool bwd, hipStream_t s) {
  if (bwd) join_bwd_run<E, R, EVEN>(a, s);
  else join_fwd_run<E, R, EVEN>(a, s);
}

template <typename E, typename R>
static void join_vec(const JoinArgs& a, bool bwd, hipStream_t s) {
  if (a.d % VEC == 0) join_rows<E, R, true>(a, bwd, s);
  else join_rows<E, R, false>(a, bwd, s);
}

static hipError_t join_launch(const JoinArgs& a, bool bwd, hipStream_t s) {
  if (a.dtype == GLA_F32) join_vec<float, float>(a, bwd, s);
  else if (a.stream_dtype == GLA_F32) join_vec<bf16, float>(a, bwd, s);
  else join_vec<bf16, bf16>(a, bwd, s);
  return hipGetLastError();
}

hipError_t launch_join_fwd(const JoinArgs& a, hipStream_t s) { return join_launch(a, false, s); }
hipError_t launch_join_bwd(const JoinArgs& a, hipStream_t s) { return join_launch(a, true, s); }

}  // namespace gla
