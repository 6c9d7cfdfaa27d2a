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
  int VEC, LPH, slots, TPR, NV, RPB;  // RPB rows per workgroup of TPR * RPB lanes
};

static int pow2_up(int n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

static JoinShape join_shape(int H, int d, int vec) {
  JoinShape s;
  s.VEC = vec;
  const int n = (d + vec - 1) / vec;
  s.LPH = n <= 64 ? pow2_up(n) : (n + 63) / 64 * 64;
  s.slots = H * s.LPH;
  s.TPR = pow2_up(s.slots);
  if (s.TPR > 1024) s.TPR = 1024;
  s.NV = pow2_up((s.slots + s.TPR - 1) / s.TPR);
  s.RPB = s.TPR >= 256 ? 1 : 256 / s.TPR;
  return s;
}

// Sum over the lanes of aligned groups of `width` lanes (a power of 2 up to 64).
__device__ __forceinline__ float lane_sum(float v, int width) {
  for (int o = 1; o < width; o *= 2) v += __shfl_xor(v, o);
  return v;
}

// The sum of a row's slots in every lane of the row.  red: 16 floats of LDS; every lane of the
// workgroup calls it.
__device__ __forceinline__ float row_sum(float v, int TPR, float* red) {
  if (TPR <= 64) return lane_sum(v, TPR);
  v = lane_sum(v, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  const int w = TPR / 64, first = (threadIdx.x >> 6) / w * w;
  float s = 0.f;
  for (int i = 0; i < w; ++i) s += red[first + i];
  return s;
}

// Every slot's head sum, in place.  red: NV * 16 floats of LDS, red[j * 16 + wave] a wave's sum.
template <int NV>
__device__ __forceinline__ void head_sums(float (&v)[NV], const JoinShape& p, int lane, float* red) {
  if (p.LPH <= 64) {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = lane_sum(v[j], p.LPH);
    return;
  }
  __syncthreads();
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

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + __expf(-z)); }

// act(z) and its slope.
__device__ __forceinline__ void gate(int act, float z, float& f, float& df) {
  const float s = sigmoid(z);
  if (act == GLA_ACT_SILU) {
    f = z * s;
    df = s * fmaf(z, 1.f - s, 1.f);
  } else {
    f = s;
    df = s * (1.f - s);
  }
}

template <typename E, typename R, int VEC, int NV>
__global__ __launch_bounds__(1024) void join_fwd_kernel(JoinArgs a, JoinShape p) {
  __shared__ float red[16 * NV];
  const int D = a.H * a.d;
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T;
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += (long)gridDim.x * p.RPB) {
    const long row = row0 + sub;
    const bool live = row < rows;
    const long b = live ? row / a.T : 0, t = live ? row - b * a.T : 0;
    float y[NV][VEC], hs[NV];
    int at[NV], in[NV], head[NV];  // column in the row, in the head (-1: an empty slot), head
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int s = lane + j * p.TPR, h = s / p.LPH, i = (s - h * p.LPH) * VEC;
      in[j] = live && h < a.H && i < a.d ? i : -1;
      at[j] = h * a.d + i;
      head[j] = h;
      hs[j] = 0.f;
      if (in[j] >= 0) {
        load_row<E, VEC>((const E*)a.y + b * a.ys.b + h * a.ys.h + t * a.ys.t + i, y[j]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) hs[j] = fmaf(y[j][v], y[j][v], hs[j]);
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] = 0.f;
      }
    }
    if (a.w_post) {
      head_sums<NV>(hs, p, lane, red);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (in[j] < 0) continue;
        const float r = rsqrtf(hs[j] / a.d + a.eps);
        if (a.rstd_post && in[j] == 0) a.rstd_post[row * a.H + head[j]] = r;
        float w[VEC];
        load_row<float, VEC>(a.w_post + in[j], w);
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] *= r * w[v];
      }
    }
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j] < 0) continue;
      if (a.z) {
        float z[VEC];
        load_row<E, VEC>((const E*)a.z + b * a.zs.b + t * a.zs.t + at[j], z);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          float f, df;
          gate(a.act, z[v], f, df);
          y[j][v] *= f;
        }
      }
      if (a.scale) {
        float w[VEC];
        load_row<float, VEC>(a.scale + at[j], w);
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] *= w[v];
      }
      if (a.residual) {
        float r[VEC];
        load_row<R, VEC>((const R*)a.residual + b * a.rs.b + t * a.rs.t + at[j], r);
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[j][v] += r[v];
      }
      store_row<R, VEC>((R*)a.out + row * D + at[j], y[j]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) sq = fmaf(y[j][v], y[j][v], sq);
    }
    if (a.w_pre) {
      const float r = rsqrtf(row_sum(sq, p.TPR, red) / D + a.eps);
      if (a.rstd_pre && live && lane == 0) a.rstd_pre[row] = r;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (in[j] < 0) continue;
        float w[VEC];
        load_row<float, VEC>(a.w_pre + at[j], w);
#pragma unroll
        for (int v = 0; v < VEC; ++v) w[v] *= y[j][v] * r;
        store_row<E, VEC>((E*)a.normed + row * D + at[j], w);
      }
    }
  }
}

// One pass over the rows: recomputes yn, m and out from y, z and the residual, then
//   n = out rp,  e = dn w_pre,  dO = d_out + rp (e - n mean(e n))         d_residual = dO
//   dz = dO scale yn w_post act'(z),  du = dO scale act(z),  e' = du w_post
//   dy = ry (e' - yn mean_d(e' yn))
// and adds up the weights' gradients dn n, dO m, du yn over its rows in registers, then over the
// workgroup's RPB rows in LDS; partial: [workgroup][3][D], summed in order by join_sum_kernel.
template <typename E, typename R, int VEC, int NV>
__global__ __launch_bounds__(1024) void join_bwd_kernel(JoinArgs a, JoinShape p) {
  extern __shared__ float lds[];
  float* red = lds;  // 16 * NV floats, then RPB rows for the sums over rows and heads
  const int D = a.H * a.d;
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T;
  float spre[NV][VEC] = {}, sscale[NV][VEC] = {}, spost[NV][VEC] = {};
  int at[NV], in[NV], head[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int s = lane + j * p.TPR, h = s / p.LPH, i = (s - h * p.LPH) * VEC;
    in[j] = h < a.H && i < a.d ? i : -1;
    at[j] = h * a.d + i;
    head[j] = h;
  }
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += (long)gridDim.x * p.RPB) {
    const long row = row0 + sub;
    const bool live = row < rows;
    const long b = live ? row / a.T : 0, t = live ? row - b * a.T : 0;
    float yn[NV][VEC], f[NV][VEC], m[NV][VEC], out[NV][VEC], dn[NV][VEC], ry[NV], rp = 0.f;
    float dot = 0.f;
    if (a.d_normed && live) rp = a.rstd_pre[row];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      ry[j] = 1.f;
#pragma unroll
      for (int v = 0; v < VEC; ++v) yn[j][v] = f[j][v] = m[j][v] = out[j][v] = dn[j][v] = 0.f;
      if (in[j] < 0 || !live) continue;
      load_row<E, VEC>((const E*)a.y + b * a.ys.b + head[j] * a.ys.h + t * a.ys.t + in[j], yn[j]);
      float w[VEC];
      if (a.w_post) {
        ry[j] = a.rstd_post[row * a.H + head[j]];
        load_row<float, VEC>(a.w_post + in[j], w);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        yn[j][v] *= ry[j];
        m[j][v] = a.w_post ? yn[j][v] * w[v] : yn[j][v];
        f[j][v] = 1.f;
      }
      if (a.z) {
        float z[VEC];
        load_row<E, VEC>((const E*)a.z + b * a.zs.b + t * a.zs.t + at[j], z);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          float df;
          gate(a.act, z[v], f[j][v], df);
          m[j][v] *= f[j][v];
        }
      }
      if (a.d_normed) {
        float sc[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) sc[v] = 1.f;
        if (a.scale) load_row<float, VEC>(a.scale + at[j], sc);
        if (a.residual) load_row<R, VEC>((const R*)a.residual + b * a.rs.b + t * a.rs.t + at[j], out[j]);
        load_row<E, VEC>((const E*)a.d_normed + b * a.dns.b + t * a.dns.t + at[j], dn[j]);
        load_row<float, VEC>(a.w_pre + at[j], w);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          out[j][v] = fmaf(sc[v], m[j][v], out[j][v]) * rp;  // n
          spre[j][v] = fmaf(dn[j][v], out[j][v], spre[j][v]);
          dn[j][v] *= w[v];
          dot = fmaf(dn[j][v], out[j][v], dot);
        }
      }
    }
    if (a.d_normed) dot = row_sum(dot, p.TPR, red) / D;
    float hs[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      hs[j] = 0.f;
      if (in[j] < 0 || !live) continue;
      float dO[VEC];
      if (a.d_out) load_row<R, VEC>((const R*)a.d_out + b * a.dos.b + t * a.dos.t + at[j], dO);
      else
#pragma unroll
        for (int v = 0; v < VEC; ++v) dO[v] = 0.f;
#pragma unroll
      for (int v = 0; v < VEC; ++v) dO[v] = fmaf(rp, dn[j][v] - out[j][v] * dot, dO[v]);
      if (a.d_residual) store_row<R, VEC>((R*)a.d_residual + row * D + at[j], dO);
      if (a.scale) {
        float sc[VEC];
        load_row<float, VEC>(a.scale + at[j], sc);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          sscale[j][v] = fmaf(dO[v], m[j][v], sscale[j][v]);
          dO[v] *= sc[v];
        }
      }
      float w[VEC];
      if (a.w_post) load_row<float, VEC>(a.w_post + in[j], w);
      else
#pragma unroll
        for (int v = 0; v < VEC; ++v) w[v] = 1.f;
      if (a.z) {
        float z[VEC];
        load_row<E, VEC>((const E*)a.z + b * a.zs.b + t * a.zs.t + at[j], z);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          float g, dg;
          gate(a.act, z[v], g, dg);
          z[v] = dO[v] * yn[j][v] * w[v] * dg;
        }
        store_row<E, VEC>((E*)a.dz + row * D + at[j], z);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        dO[v] *= f[j][v];  // du
        if (a.w_post) spost[j][v] = fmaf(dO[v], yn[j][v], spost[j][v]);
        f[j][v] = dO[v] * w[v];
        hs[j] = fmaf(f[j][v], yn[j][v], hs[j]);
      }
    }
    if (a.w_post) head_sums<NV>(hs, p, lane, red);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j] < 0 || !live) continue;
      if (a.w_post) {
        const float mean = hs[j] / a.d;
#pragma unroll
        for (int v = 0; v < VEC; ++v) f[j][v] = ry[j] * (f[j][v] - yn[j][v] * mean);
      }
      store_row<E, VEC>((E*)a.dy + (((long)b * a.H + head[j]) * a.T + t) * a.d + in[j], f[j]);
    }
  }
  if (!a.partial) return;
  // the workgroup's sums, through LDS where several rows (and for w_post heads) add up
  float* sums = lds + 16 * NV;  // [RPB][D]
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (!(which == 0 ? (void*)a.dw_pre : which == 1 ? (void*)a.dscale : (void*)a.dw_post)) continue;
    const int cols = which == 2 ? a.d : D, terms = which == 2 ? p.RPB * a.H : p.RPB;
    float* to = a.partial + ((long)blockIdx.x * 3 + which) * D;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (in[j] < 0) continue;
      const float* acc = which == 0 ? spre[j] : which == 1 ? sscale[j] : spost[j];
      store_row<float, VEC>((terms > 1 ? sums + sub * D : to) + at[j], *(const float(*)[VEC])acc);
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
  const void* own[] = {a.w_post, a.scale, a.w_pre, a.out, a.normed, a.dy, a.dz, a.d_residual};
  for (const void* q : own)
    if (q && !rows_aligned(q, none, 16)) return false;
  return a.d % 8 == 0 && rows_aligned(a.y, a.ys, 16) && rows_aligned(a.z, a.zs, 16) &&
         rows_aligned(a.residual, a.rs, 16) && rows_aligned(a.d_out, a.dos, 16) && rows_aligned(a.d_normed, a.dns, 16);
}

static int join_groups(long long rows, int RPB) {
  const long long n = (rows + RPB - 1) / RPB;
  return (int)(n < 512 ? n : 512);
}

size_t join_partial_floats(int B, int H, int T, int d) {
  const long long rows = (long long)B * T;
  int G = 0;
  for (int vec : {1, 8}) {
    const int g = join_groups(rows, join_shape(H, d, vec).RPB);
    if (g > G) G = g;
  }
  return (size_t)G * 3 * H * d;
}

template <typename E, typename R, int VEC, int NV, bool BWD>
static void join_run(const JoinArgs& a, const JoinShape& p, hipStream_t s) {
  const long long rows = (long long)a.B * a.T;
  const int threads = p.TPR * p.RPB;
  if constexpr (!BWD) {
    const long long n = (rows + p.RPB - 1) / p.RPB;
    join_fwd_kernel<E, R, VEC, NV><<<(unsigned)(n < 4096 ? n : 4096), threads, 0, s>>>(a, p);
  } else {
    const int G = join_groups(rows, p.RPB);
    const size_t lds = (16 * NV + (a.partial && (p.RPB > 1 || a.dw_post) ? p.RPB * a.H * a.d : 0)) * sizeof(float);
    join_bwd_kernel<E, R, VEC, NV><<<G, threads, lds, s>>>(a, p);
    if (a.partial) join_sum_kernel<<<dim3((a.H * a.d + 63) / 64, 3), 1024, 0, s>>>(a, G);
  }
}

template <typename E, typename R, bool BWD>
static void join_vec(const JoinArgs& a, hipStream_t s) {
  if (join_wide(a)) {
    const JoinShape p = join_shape(a.H, a.d, 8);
    if (p.NV == 1) join_run<E, R, 8, 1, BWD>(a, p, s);
    else join_run<E, R, 8, 2, BWD>(a, p, s);
  } else {
    const JoinShape p = join_shape(a.H, a.d, 1);
    if (p.NV == 1) join_run<E, R, 1, 1, BWD>(a, p, s);
    else if (p.NV == 2) join_run<E, R, 1, 2, BWD>(a, p, s);
    else if (p.NV == 4) join_run<E, R, 1, 4, BWD>(a, p, s);
    else if (p.NV == 8) join_run<E, R, 1, 8, BWD>(a, p, s);
    else join_run<E, R, 1, 16, BWD>(a, p, s);
  }
}

template <bool BWD>
static hipError_t join_launch(const JoinArgs& a, hipStream_t s) {
  if (a.dtype == GLA_F32) join_vec<float, float, BWD>(a, s);
  else if (a.stream_dtype == GLA_F32) join_vec<bf16, float, BWD>(a, s);
  else join_vec<bf16, bf16, BWD>(a, s);
  return hipGetLastError();
}

hipError_t launch_join_fwd(const JoinArgs& a, hipStream_t s) { return join_launch<false>(a, s); }
hipError_t launch_join_bwd(const JoinArgs& a, hipStream_t s) { return join_launch<true>(a, s); }

}  // namespace gla
