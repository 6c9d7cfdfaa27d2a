// Layer norm joined to the residual add, forward and backward, one pass over the rows each:
//   out = residual + x,   n = (out - mean) rsqrt(mean((out - mean)^2) + eps),   normed = n w + b
//   e = dn w,   dx = d_residual = d_out + rstd (e - mean(e) - n mean(e n)),   dw = sum dn n,   db = sum dn
// A row is spread over TPR lanes in slots of 8 elements (slot s: lane s % TPR, register s / TPR) and held in
// registers, so that the variance is taken about the mean, not as a difference of two sums.  All arithmetic is
// float32, rounded once at the store; the backward forms out again from x and the residual instead of reading its
// rounded value.  The weights' gradients are sums per workgroup, then a second kernel in a fixed order.
// Bound by HBM: 32768 rows of 2048, bf16, without a residual 56 us, 4.8 TB/s; 16384 rows with one 46 us forward, 73 us and 5
// for the weights' sums backward, 5.9 and 4.6 TB/s (the memory-side cache serves a part).  Rows of 2047 take 39 and 67 us
// for 8000 where whole slots would take 27 and 33.  Rows above 8192 hold four slots a lane; with a float32 stream the backward
// then has more than 256 registers' worth and keeps 13 (bf16) or 45 (float32) of them in memory: 2048 rows of 16384, bf16 with
// float32, 147 us where its bytes take 123.
#include "gla_layernorm.hpp"
#include "gla_rows.hpp"

namespace gla {

struct NormShape {
  int TPR, NV, RPB;  // lanes and slots a lane of a row; rows of a workgroup of TPR * RPB lanes
  float inv_D;
};

// Lanes of a row at most, and of a workgroup where a row takes fewer.
constexpr int kNormLanes = 512, kNormThreads = 256;
static_assert(kNormMaxRow <= 4 * kNormLanes * VEC, "a lane's slots");

static NormShape norm_shape(int D) {
  NormShape s;
  const int slots = (D + VEC - 1) / VEC;
  s.TPR = pow2_up(slots);
  if (s.TPR > kNormLanes) s.TPR = kNormLanes;
  s.NV = pow2_up((slots + s.TPR - 1) / s.TPR);
  s.RPB = s.TPR >= kNormThreads ? 1 : kNormThreads / s.TPR;
  s.inv_D = 1.f / D;
  return s;
}

template <bool EVEN>
__device__ __forceinline__ void norm_weights(const float* w, int c, int left, float fill, float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = fill;
  if (w && left > 0) {
    const auto r = load_slot<EVEN, float>(w + c, left);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r[i];
  }
}

// A row's inputs as they lie in memory.
template <typename E, typename R, int NV, bool BWD, bool EVEN>
struct NormIn {
  typename Pack<E>::raw x[NV], dn[BWD ? NV : 1];
  typename Pack<R>::raw r[NV], dout[BWD ? NV : 1];
  float mean, rstd;
  __device__ __forceinline__ void load(const NormArgs& a, const NormShape& p, int lane, const RowStep& at) {
    const long b = at.b, t = at.t;
    if constexpr (BWD) {
      mean = a.mean[at.row];
      rstd = a.rstd[at.row];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * p.TPR) * VEC, left = a.D - c;
      if (left <= 0) continue;
      x[j] = load_slot<EVEN>((const E*)a.x + b * a.xs.b + t * a.xs.t + c, left);
      if (a.residual) r[j] = load_slot<EVEN>((const R*)a.residual + b * a.rs.b + t * a.rs.t + c, left);
      if constexpr (BWD) {
        dn[j] = load_slot<EVEN>((const E*)a.d_normed + b * a.dns.b + t * a.dns.t + c, left);
        if (a.d_out) dout[j] = load_slot<EVEN>((const R*)a.d_out + b * a.dos.b + t * a.dos.t + c, left);
      }
    }
  }
};

// NV = 1: the next row is loaded before this one is reduced, and the weights stay in registers.
template <typename E, typename R, int NV, int NT, bool EVEN>
__global__ __launch_bounds__(NT) void norm_fwd_kernel(NormArgs a, NormShape p) {
  constexpr bool HELD = NV == 1;
  __shared__ float red[2 * 16];
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T, step = (long)gridDim.x * p.RPB;
  RowStep at((long)blockIdx.x * p.RPB + sub, a.T, step);
  NormIn<E, R, NV, false, EVEN> in, next;
  if (at.row < rows) in.load(a, p, lane, at);
  float w[VEC], bias[VEC];
  if (HELD) {
    norm_weights<EVEN>(a.w, lane * VEC, a.D - lane * VEC, 1.f, w);
    norm_weights<EVEN>(a.b, lane * VEC, a.D - lane * VEC, 0.f, bias);
  }
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += step) {
    const RowStep here = at;
    const bool live = here.row < rows;
    at.next(a.T, step);
    if (HELD && at.row < rows) next.load(a, p, lane, at);
    float h[NV][VEC], sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * p.TPR) * VEC, left = a.D - c;
      const bool have = live && left > 0;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        h[j][v] = have ? (float)in.x[j][v] + (a.residual ? (float)in.r[j][v] : 0.f) : 0.f;
        sum += h[j][v];
      }
      if (have && a.out) store_slot<EVEN>((R*)a.out + here.row * a.D + c, h[j], left);
    }
    if (!HELD && at.row < rows) in.load(a, p, lane, at);
    const float mean = row_sum(sum, p.TPR, red, 0) * p.inv_D;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        h[j][v] = (lane + j * p.TPR) * VEC + v < a.D ? h[j][v] - mean : 0.f;
        sq = fmaf(h[j][v], h[j][v], sq);
      }
    const float rstd = rsqrtf(row_sum(sq, p.TPR, red, 1) * p.inv_D + a.eps);
    if (live && lane == 0 && a.mean) {
      a.mean[here.row] = mean;
      a.rstd[here.row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * p.TPR) * VEC, left = a.D - c;
      if (!live || left <= 0) continue;
      if (!HELD) {
        norm_weights<EVEN>(a.w, c, left, 1.f, w);
        norm_weights<EVEN>(a.b, c, left, 0.f, bias);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) h[j][v] = fmaf(h[j][v] * rstd, w[v], bias[v]);
      store_slot<EVEN>((E*)a.normed + here.row * a.D + c, h[j], left);
    }
    if (HELD) in = next;
  }
}

// partial: [workgroup][2][D], dw and db.
template <typename E, typename R, int NV, int NT, bool EVEN>
__global__ __launch_bounds__(NT) void norm_bwd_kernel(NormArgs a, NormShape p) {
  constexpr bool HELD = NV == 1;
  extern __shared__ float lds[];
  float* red = lds;  // 2 x 2 x 16 floats, then RPB rows for the last sums
  const int lane = threadIdx.x % p.TPR, sub = threadIdx.x / p.TPR;
  const long rows = (long)a.B * a.T, step = (long)gridDim.x * p.RPB;
  RowStep at((long)blockIdx.x * p.RPB + sub, a.T, step);
  NormIn<E, R, NV, true, EVEN> in, next;
  if (at.row < rows) in.load(a, p, lane, at);
  float w[VEC], sw[NV][VEC] = {}, sb[NV][VEC] = {};
  if (HELD) norm_weights<EVEN>(a.w, lane * VEC, a.D - lane * VEC, 1.f, w);
  int turn = 0;
  for (long row0 = (long)blockIdx.x * p.RPB; row0 < rows; row0 += step, turn ^= 1) {
    const RowStep here = at;
    const bool live = here.row < rows;
    at.next(a.T, step);
    if (HELD && at.row < rows) next.load(a, p, lane, at);
    float n[NV][VEC], e[NV][VEC], se = 0.f, sen = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * p.TPR) * VEC, left = a.D - c;
      if (!live || left <= 0) continue;
      if (!HELD) norm_weights<EVEN>(a.w, c, left, 1.f, w);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float h = (float)in.x[j][v] + (a.residual ? (float)in.r[j][v] : 0.f), dn = (float)in.dn[j][v];
        n[j][v] = EVEN || v < left ? (h - in.mean) * in.rstd : 0.f;
        e[j][v] = dn * w[v];
        sw[j][v] = fmaf(dn, n[j][v], sw[j][v]);
        sb[j][v] += dn;
        se += e[j][v];
        sen = fmaf(e[j][v], n[j][v], sen);
      }
    }
    // both sums behind one barrier; halves in turn as in row_sum
    if (p.TPR <= 64) {
      se = lane_sum(se, p.TPR);
      sen = lane_sum(sen, p.TPR);
    } else {
      se = lane_sum(se, 64);
      sen = lane_sum(sen, 64);
      float* r = red + turn * 32;
      if ((threadIdx.x & 63) == 0) {
        r[threadIdx.x >> 6] = se;
        r[16 + (threadIdx.x >> 6)] = sen;
      }
      __syncthreads();
      const int waves = p.TPR / 64, first = (threadIdx.x >> 6) / waves * waves;
      se = sen = 0.f;
      for (int i = 0; i < waves; ++i) {
        se += r[first + i];
        sen += r[16 + first + i];
      }
    }
    se *= p.inv_D;
    sen *= p.inv_D;
    const float rstd = in.rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * p.TPR) * VEC, left = a.D - c;
      if (!live || left <= 0) continue;
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        e[j][v] = fmaf(rstd, e[j][v] - fmaf(n[j][v], sen, se), a.d_out ? (float)in.dout[j][v] : 0.f);
      store_slot<EVEN>((E*)a.dx + here.row * a.D + c, e[j], left);
      if (a.d_residual) store_slot<EVEN>((R*)a.d_residual + here.row * a.D + c, e[j], left);
    }
    if (HELD) in = next;
    else if (at.row < rows) in.load(a, p, lane, at);
  }
  if (!a.partial) return;
  float* sums = lds + 64;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.db : a.dw)) continue;
    float* to = a.partial + ((long)blockIdx.x * 2 + which) * a.D;
    if (p.RPB > 1) __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lane + j * p.TPR) * VEC, left = a.D - c;
      if (left <= 0) continue;
      store_slot<EVEN>(p.RPB > 1 ? sums + sub * a.D + c : to + c, which ? sb[j] : sw[j], left);
    }
    if (p.RPB == 1) continue;
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      float v = 0.f;
      for (int i = 0; i < p.RPB; ++i) v += sums[i * a.D + c];
      to[c] = v;
    }
  }
}

// dw and db from the workgroups' sums, in one order whatever the timing: 64 columns of one a workgroup, each of its
// 16 waves every 16th of the G rows.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormArgs a, int G) {
  float* out = blockIdx.y ? a.db : a.dw;
  if (!out) return;
  const int lane = threadIdx.x & 63, c = blockIdx.x * 64 + lane, part = threadIdx.x >> 6;
  __shared__ float red[16][64];
  const float* from = a.partial + (long)blockIdx.y * a.D + c;
  float s = 0.f;
  if (c < a.D) {
    int g = part;
    for (; g + 7 * 16 < G; g += 8 * 16) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = from[(long)(g + 16 * i) * 2 * a.D];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; g < G; g += 16) s += from[(long)g * 2 * a.D];
  }
  red[part][lane] = s;
  __syncthreads();
  if (part == 0 && c < a.D) {
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    out[c] = s;
  }
}

// Workgroups of 256 lanes at most (half as many of 512): rows in turn, so that the next one's loads are under way and a
// column's sums stay in registers.  16384 rows of 2048, bf16: forward 46 us with 1024, 52 with 2048, 60 with 512; backward
// and sums 80 with 512, 85 with 1024, 113 with 256.
constexpr int kNormBwdGroups = 512, kNormFwdGroups = 1024;

static int norm_groups(long long rows, const NormShape& p, int most) {
  const long long n = (rows + p.RPB - 1) / p.RPB;
  most = most * kNormThreads / (p.TPR * p.RPB);
  return (int)(n < most ? n : most);
}

size_t norm_partial_floats(int B, int T, int D) {
  return (size_t)norm_groups((long long)B * T, norm_shape(D), kNormBwdGroups) * 2 * D;
}

template <typename E, typename R, bool EVEN>
static void norm_run(const NormArgs& a, bool bwd, hipStream_t s) {
  const NormShape p = norm_shape(a.D);
  const int threads = p.TPR * p.RPB, G = norm_groups((long long)a.B * a.T, p, bwd ? kNormBwdGroups : kNormFwdGroups);
  if (!bwd) {
    if (threads == 256) norm_fwd_kernel<E, R, 1, 256, EVEN><<<G, threads, 0, s>>>(a, p);
    else if (p.NV == 1) norm_fwd_kernel<E, R, 1, 512, EVEN><<<G, threads, 0, s>>>(a, p);
    else if (p.NV == 2) norm_fwd_kernel<E, R, 2, 512, EVEN><<<G, threads, 0, s>>>(a, p);
    else norm_fwd_kernel<E, R, 4, 512, EVEN><<<G, threads, 0, s>>>(a, p);
    return;
  }
  const size_t lds = (64 + (a.partial && p.RPB > 1 ? p.RPB * a.D : 0)) * sizeof(float);
  if (threads == 256) norm_bwd_kernel<E, R, 1, 256, EVEN><<<G, threads, lds, s>>>(a, p);
  else if (p.NV == 1) norm_bwd_kernel<E, R, 1, 512, EVEN><<<G, threads, lds, s>>>(a, p);
  else if (p.NV == 2) norm_bwd_kernel<E, R, 2, 512, EVEN><<<G, threads, lds, s>>>(a, p);
  else norm_bwd_kernel<E, R, 4, 512, EVEN><<<G, threads, lds, s>>>(a, p);
  if (a.partial) norm_sum_kernel<<<dim3((a.D + 63) / 64, 2), 1024, 0, s>>>(a, G);
}

template <typename E, typename R>
static void norm_vec(const NormArgs& a, bool bwd, hipStream_t s) {
  if (a.D % VEC == 0) norm_run<E, R, true>(a, bwd, s);
  else norm_run<E, R, false>(a, bwd, s);
}

hipError_t launch_layernorm(const NormArgs& a, bool bwd, hipStream_t s) {
  if (a.dtype == GLA_F32) norm_vec<float, float>(a, bwd, s);
  else if (a.stream_dtype == GLA_F32) norm_vec<bf16, float>(a, bwd, s);
  else norm_vec<bf16, bf16>(a, bwd, s);
  return hipGetLastError();
}

}  // namespace gla
