// What joins a block's output y [B][H][T][d] to the residual stream [B][T][H d], forward and
// backward, one pass over the rows (b, t) each:
//   yn = y rsqrt(mean_d(y^2) + eps)          (per head; with w_post)
//   m = yn w_post act(z)                     (the gate: silu or sigmoid)
//   out = residual + scale m
//   normed = out rsqrt(mean(out^2) + eps) w_pre
// A row is spread over TPR lanes in slots of VEC elements.  A head takes LPH slots (its last ones
// are empty where d / VEC is not LPH): a power of 2 up to 64, so that a head's sum is a lane
// exchange inside an aligned group, or a multiple of 64, so that no wave's slots belong to two
// heads and a head's sum is a wave sum and a sum of LPH / 64 of them from LDS.  Slot s of a row
// is lane s % TPR, register s / TPR.  All arithmetic is float32, rounded once at the store; the
// backward recomputes out from y, z and the residual instead of reading its rounded value.
#include "gla_block.hpp"

namespace gla {

struct JoinShape {
  int LPH, slots, TPR, NV, RPB;  // RPB rows per workgroup of TPR * RPB lanes
  float inv_d, inv_D;
};

static int pow2_up(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

// threads: of a workgroup, where a row takes fewer.
static JoinShape join_shape(int H, int d, int vec, int threads) {
  JoinShape s;
  const int n = (d + vec - 1) / vec;
  s.LPH = n <= 64 ? pow2_up(n) : (n + 63) / 64 * 64;
  s.slots = H * s.LPH;
  s.TPR = pow2_up(s.slots);
  if (s.TPR > 1024) s.TPR = 1024;
  s.NV = pow2_up((s.slots + s.TPR - 1) / s.TPR);
  s.RPB = s.TPR >= threads ? 1 : threads / s.TPR;
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

// A lane's slots of a row: the same for every row.
template <int NV>
struct Slots {
  int at[NV], in[NV], head[NV];  // column in the row, column in the head (-1: an empty slot), head
};
template <int VEC, int NV>
__device__ __forceinline__ Slots<NV> row_slots(const JoinArgs& a, const JoinShape& p, int lane) {
  Slots<NV> r;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int s = lane + j * p.TPR, h = s / p.LPH, i = (s - h * p.LPH) * VEC;
    r.in[j] = h < a.H && i < a.d ? i : -1;
    r.at[j] = h * a.d + i;
    r.head[j] = h;
  }
  return r;
}

// w's values at a lane's slots (`one` where there is no w).
template <int VEC, int NV>
__device__ __forceinline__ void load_weights(const float* w, const int (&at)[NV], const int (&in)[NV], float (&v)[NV][VEC]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[j][i] = 1.f;
    if (w && in[j] >= 0) load_row<float, VEC>(w + at[j], v[j]);
  }
}

// The row a workgroup's lane group is at: (b, t) stepped without a division.
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
    b += db;
    t += dt;
    if (t >= T) {
      t -= T;
      ++b;
    }
  }
};

// One row's inputs as they lie in memory (bf16 stays packed), loaded a row ahead of their use.
template <typename E, typename R, int VEC, int NV, bool BWD>
struct RowIn {
  typename Vec<E, VEC>::raw y[NV], z[NV], dn[BWD ? NV : 1];
  typename Vec<R, VEC>::raw r[NV], dout[BWD ? NV : 1];
  float ry[BWD ? NV : 1], rp;
  __device__ __forceinline__ void load(const JoinArgs& a, const Slots<NV>& s, const RowStep& at) {
    const long b = at.b, t = at.t;
    if constexpr (BWD) rp = a.d_normed ? a.rstd_pre[at.row] : 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (s.in[j] < 0) continue;
      y[j] = *(const typename Vec<E, VEC>::raw*)((const E*)a.y + b * a.ys.b + s.head[j] * a.ys.h + t * a.ys.t + s.in[j]);
      if (a.z) z[j] = *(const typename Vec<E, VEC>::raw*)((const E*)a.z + b * a.zs.b + t * a.zs.t + s.at[j]);
      if (a.residual)
        r[j] = *(const typename Vec<R, VEC>::raw*)((const R*)a.residual + b * a.rs.b + t * a.rs.t + s.at[j]);
      if constexpr (BWD) {
        ry[j] = a.w_post ? a.rstd_post[at.row * a.H + s.head[j]] : 1.f;
        if (a.d_normed)
          dn[j] = *(const typename Vec<E, VEC>::raw*)((const E*)a.d_normed + b * a.dns.b + t * a.dns.t + s.at[j]);
        if (a.d_out)
          dout[j] = *(const typename Vec<R, VEC>::raw*)((const R*)a.d_out + b * a.dos.b + t * a.dos.t + s.at[j]);
      }
    }
  }
};

template <typename E, typename R, int VEC, int NV, int NT>
__global__ __launch_bounds__(NT) void join_fwd_kernel(JoinArgs a, JoinShape p) {
  __shared__ float red[2 * 16], hred[2 * 16 * NV];
  const int D = a.H * a.d;
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T, step = (long)gridDim.x * p.RPB;
  const Slots<NV> s = row_slots<VEC, NV>(a, p, lane);
  float wpost[NV][VEC], scale[NV][VEC], wpre[NV][VEC];
  load_weights<VEC, NV>(a.w_post, s.in, s.in, wpost);
  load_weights<VEC, NV>(a.scale, s.at, s.in, scale);
  load_weights<VEC, NV>(a.w_pre, s.at, s.in, wpre);
  RowStep at((long)blockIdx.x * p.RPB + sub, a.T, step);
  RowIn<E, R, VEC, NV, false> in, next;
  if (at.row < rows) in.load(a, s, at);
  int turn = 0;
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += step, turn ^= 1, in = next) {
    const RowStep here = at;
    const bool live = here.row < rows;
    at.next(a.T, step);
    if (at.row < rows) next.load(a, s, at);
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
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] *= r * wpost[j][v];
      }
    }
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || s.in[j] < 0) continue;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (a.z) {
          const float z = (float)in.z[j][v], g = sigmoid(z);
          y[j][v] *= a.act == GLA_ACT_SILU ? z * g : g;
        }
        y[j][v] = fmaf(scale[j][v], y[j][v], a.residual ? (float)in.r[j][v] : 0.f);
        sq = fmaf(y[j][v], y[j][v], sq);
      }
      store_row<R, VEC>((R*)a.out + here.row * D + s.at[j], y[j]);
    }
    if (a.w_pre) {
      const float r = rsqrtf(row_sum(sq, p.TPR, red, turn) * p.inv_D + a.eps);
      if (a.rstd_pre && live && lane == 0) a.rstd_pre[here.row] = r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!live || s.in[j] < 0) continue;
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] *= r * wpre[j][v];
        store_row<E, VEC>((E*)a.normed + here.row * D + s.at[j], y[j]);
      }
    }
  }
}

// One pass over the rows: recomputes yn, m and out from y, z and the residual, then
//   n = out rp,  e = dn w_pre,  dO = d_out + rp (e - n mean(e n))         d_residual = dO
//   dz = dO scale yn w_post act'(z),  du = dO scale act(z),  e' = du w_post
//   dy = ry (e' - yn mean_d(e' yn))
// and adds up the weights' gradients dn n, dO m, du yn over its rows in registers, then over the
// workgroup's RPB rows and for w_post the heads in LDS; partial: [workgroup][3][D], summed in
// order by join_sum_kernel.
template <typename E, typename R, int VEC, int NV, int NT>
__global__ __launch_bounds__(NT) void join_bwd_kernel(JoinArgs a, JoinShape p) {
  extern __shared__ float lds[];
  float *red = lds, *hred = lds + 32;  // 2 x 16, 2 x 16 NV floats, then RPB rows for the last sums
  const int D = a.H * a.d;
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T, step = (long)gridDim.x * p.RPB;
  const Slots<NV> s = row_slots<VEC, NV>(a, p, lane);
  float wpost[NV][VEC], scale[NV][VEC], wpre[NV][VEC];
  load_weights<VEC, NV>(a.w_post, s.in, s.in, wpost);
  load_weights<VEC, NV>(a.scale, s.at, s.in, scale);
  load_weights<VEC, NV>(a.w_pre, s.at, s.in, wpre);
  float spre[NV][VEC] = {}, sscale[NV][VEC] = {}, spost[NV][VEC] = {};
  RowStep at((long)blockIdx.x * p.RPB + sub, a.T, step);
  RowIn<E, R, VEC, NV, true> in, next;
  if (at.row < rows) in.load(a, s, at);
  int turn = 0;
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += step, turn ^= 1, in = next) {
    const RowStep here = at;
    const bool live = here.row < rows;
    at.next(a.T, step);
    if (at.row < rows) next.load(a, s, at);
    float yn[NV][VEC], f[NV][VEC], n[NV][VEC], e[NV][VEC];  // f: sigmoid(z)
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool have = live && s.in[j] >= 0;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        yn[j][v] = have ? (float)in.y[j][v] * in.ry[j] : 0.f;
        f[j][v] = a.z && have ? sigmoid((float)in.z[j][v]) : 1.f;
        n[j][v] = e[j][v] = 0.f;
        if (a.d_normed && have) {
          float m = yn[j][v] * wpost[j][v] * f[j][v];
          if (a.z && a.act == GLA_ACT_SILU) m *= (float)in.z[j][v];
          n[j][v] = fmaf(scale[j][v], m, a.residual ? (float)in.r[j][v] : 0.f) * in.rp;
          const float dn = (float)in.dn[j][v];
          spre[j][v] = fmaf(dn, n[j][v], spre[j][v]);
          e[j][v] = dn * wpre[j][v];
          dot = fmaf(e[j][v], n[j][v], dot);
        }
      }
    }
    if (a.d_normed) dot = row_sum(dot, p.TPR, red, turn) * p.inv_D;
    float hs[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      hs[j] = 0.f;
      if (!live || s.in[j] < 0) continue;
      float dO[VEC], dz[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        dO[v] = a.d_out ? (float)in.dout[j][v] : 0.f;
        if (a.d_normed) dO[v] = fmaf(in.rp, fmaf(-n[j][v], dot, e[j][v]), dO[v]);
      }
      if (a.d_residual) store_row<R, VEC>((R*)a.d_residual + here.row * D + s.at[j], dO);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float u = yn[j][v] * wpost[j][v];
        float act = 1.f, slope = 0.f;
        if (a.z) {
          const float z = (float)in.z[j][v], g = f[j][v];
          act = a.act == GLA_ACT_SILU ? z * g : g;
          slope = a.act == GLA_ACT_SILU ? g * fmaf(z, 1.f - g, 1.f) : g * (1.f - g);
        }
        sscale[j][v] = fmaf(dO[v], u * act, sscale[j][v]);
        dO[v] *= scale[j][v];
        dz[v] = dO[v] * u * slope;
        dO[v] *= act;  // du
        spost[j][v] = fmaf(dO[v], yn[j][v], spost[j][v]);
        e[j][v] = dO[v] * wpost[j][v];
        hs[j] = fmaf(e[j][v], yn[j][v], hs[j]);
      }
      if (a.z) store_row<E, VEC>((E*)a.dz + here.row * D + s.at[j], dz);
    }
    if (a.w_post) head_sums<NV>(hs, p, lane, hred, turn);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!live || s.in[j] < 0) continue;
      if (a.w_post) {
        const float mean = hs[j] * p.inv_d;
#pragma unroll
        for (int v = 0; v < VEC; ++v) e[j][v] = in.ry[j] * fmaf(-yn[j][v], mean, e[j][v]);
      }
      store_row<E, VEC>((E*)a.dy + (((long)here.b * a.H + s.head[j]) * a.T + here.t) * a.d + s.in[j], e[j]);
    }
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
      store_row<float, VEC>((terms > 1 ? sums + sub * D : to) + s.at[j], acc);
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

static bool rows_aligned(const void* p, const Strides& s, int bytes) {
  return (uintptr_t)p % (bytes < 16 ? bytes : 16) == 0 && s.b % 8 == 0 && s.h % 8 == 0 && s.t % 8 == 0;
}

// Slots of 8 elements where the head width and every pointer and stride allow 16-byte accesses,
// of one element otherwise.
static bool join_wide(const JoinArgs& a) {
  const Strides none{0, 0, 0};
  const void* own[] = {a.w_post, a.scale, a.w_pre, a.out, a.normed, a.dy, a.dz, a.d_residual, a.partial};
  for (const void* q : own)
    if (q && !rows_aligned(q, none, 16)) return false;
  return a.d % 8 == 0 && rows_aligned(a.y, a.ys, 16) && rows_aligned(a.z, a.zs, 16) &&
         rows_aligned(a.residual, a.rs, 16) && rows_aligned(a.d_out, a.dos, 16) && rows_aligned(a.d_normed, a.dns, 16);
}

// Lanes of a workgroup (more where a row needs them) and the most workgroups.  Measured on
// 16k rows of 2048, forward and backward together: backward 512 x 256 lanes 184 us, 256 x 256 238,
// 384 202, 768 208, 1024 189, 512 x 512 198; on 32k rows of 1024 forward: 1024 x 256 38.2 us,
// 2048 41.8, 4096 42.9.
constexpr int kFwdThreads = 256, kBwdThreads = 256, kBwdGroups = 512, kFwdGroups = 1024;

static int join_groups(long long rows, int RPB, int most) {
  const long long n = (rows + RPB - 1) / RPB;
  return (int)(n < most ? n : most);
}

size_t join_partial_floats(int B, int H, int T, int d) {
  int G = 0;
  for (int vec : {1, 8}) {
    const int g = join_groups((long long)B * T, join_shape(H, d, vec, kBwdThreads).RPB, kBwdGroups);
    if (g > G) G = g;
  }
  return (size_t)G * 3 * H * d;
}

template <typename E, typename R, int VEC, int NV, int NT>
static void join_run(const JoinArgs& a, const JoinShape& p, bool bwd, hipStream_t s) {
  const long long rows = (long long)a.B * a.T;
  const int threads = p.TPR * p.RPB;
  if (!bwd) {
    join_fwd_kernel<E, R, VEC, NV, NT><<<join_groups(rows, p.RPB, kFwdGroups), threads, 0, s>>>(a, p);
  } else {
    const int G = join_groups(rows, p.RPB, kBwdGroups);
    const size_t lds = (32 + 32 * NV + (a.partial && (p.RPB > 1 || a.dw_post) ? p.RPB * a.H * a.d : 0)) * sizeof(float);
    join_bwd_kernel<E, R, VEC, NV, NT><<<G, threads, lds, s>>>(a, p);
    if (a.partial) join_sum_kernel<<<dim3((a.H * a.d + 63) / 64, 3), 1024, 0, s>>>(a, G);
  }
}

template <typename E, typename R>
static void join_vec(const JoinArgs& a, bool bwd, hipStream_t s) {
  const int threads = bwd ? kBwdThreads : kFwdThreads;
  if (join_wide(a)) {
    const JoinShape p = join_shape(a.H, a.d, 8, threads);
    if (p.TPR <= 512) join_run<E, R, 8, 1, 512>(a, p, bwd, s);
    else if (p.NV == 1) join_run<E, R, 8, 1, 1024>(a, p, bwd, s);
    else join_run<E, R, 8, 2, 1024>(a, p, bwd, s);
  } else {
    const JoinShape p = join_shape(a.H, a.d, 1, threads);
    if (p.NV == 1) join_run<E, R, 1, 1, 1024>(a, p, bwd, s);
    else if (p.NV == 2) join_run<E, R, 1, 2, 1024>(a, p, bwd, s);
    else if (p.NV == 4) join_run<E, R, 1, 4, 1024>(a, p, bwd, s);
    else if (p.NV == 8) join_run<E, R, 1, 8, 1024>(a, p, bwd, s);
    else join_run<E, R, 1, 16, 1024>(a, p, bwd, s);
  }
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
