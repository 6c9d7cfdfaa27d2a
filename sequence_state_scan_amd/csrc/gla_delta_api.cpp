// C ABI of the gated delta rule and of the layer norm (declared in include/gla.h): host-side argument checks, the
// layout of what the delta rule's calls keep, then kernel launches on the caller's stream.  Every check runs before
// the first HIP call.
#include "gla.h"

#include "gla_checks.hpp"
#include "gla_delta.hpp"
#include "gla_layernorm.hpp"

namespace gla {

// A sequence's chunks are cut into segments where the heads and their column tiles would leave CUs idle.
// Segments: as many as give each of the 256 CUs a walk of its own, never more than one (200 heads of 2048 tokens in two
// segments, bf16 128 x 128: forward 369 us, whole 262; training step 1349 and 1046; 128 heads in two 223 and 846, whole 206 and
// 786), and no more than 3 sqrt(N): a segment's two walks of L = N / P chunks take about 6 us a chunk each, the chain between
// them 1.3 us a segment, so the best P is near 3 sqrt(N) (4 heads of 8192 tokens, N = 128: P = 128 201 us, 64 125, 32 (33, in
// whole chunks) 97, 16 107; of 1024, N = 16: P = 16 51, 8 (12) 46, 4 52, 1 87).  Two segments' walks take as long as the one
// whole.
// Columns: 128 a workgroup, 64 where the tiles of 128 and their segments would leave half the CUs or more without a walk (one
// segment of 2048 tokens, 128 x 128, forward and training step with 64 and with 128: 86 heads, bf16 188 / 647 and 207 / 702 us,
// float32 481 / 1365 and 658 / 1787; 128 heads 205 / 786 and 227 / 846, 510 / 1606 and 689 / 2030; 200 heads of 512 tokens, past
// the border, bf16 108 / 386 and 75 / 310, float32 252 / 788 and 197 / 685.  In segments, float32 2 x 3 heads of 333 tokens,
// 48 x 80: 36 / 93 and 41 / 105).
DeltaShape delta_shape(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  DeltaShape s{};
  s.B = B;
  s.H = H;
  s.Hk = Hk;
  s.T = T;
  s.dk = dk;
  s.dv = dv;
  s.dtype = dtype;
  s.N = (T + kDeltaChunk - 1) / kDeltaChunk;
  s.DKP = dk <= 32 ? 32 : dk <= 64 ? 64 : 128;
  s.DVP = (dv + 15) / 16 * 16;
  s.dkr = (dk + 7) / 8 * 8;
  s.dvr = (dv + 7) / 8 * 8;
  s.marks = (s.N + kDeltaMarks - 1) / kDeltaMarks;
  long long most = 1;
  while (most < s.N && (most + 1) * (most + 1) <= 9LL * s.N) ++most;
  const long long heads = (long long)B * H, wide = heads * ((dv + 127) / 128);
  const auto segments = [&](long long units) {
    const long long P = 256 / units < most ? 256 / units : most;
    return P < 3 ? 1 : P;
  };
  s.NW = dv <= 64 || wide * segments(wide) <= 128 ? 4 : 8;
  const long long P = segments(heads * ((dv + 16 * s.NW - 1) / (16 * s.NW)));
  s.L = (int)((s.N + P - 1) / P);
  s.P = (s.N + s.L - 1) / s.L;
  return s;
}

namespace {

// Hands out regions of a buffer, each on 256 bytes; with a null buffer only counts.
struct Regions {
  char* p;
  size_t used = 0;
  template <typename T>
  void take(T*& to, size_t bytes) {
    to = p ? reinterpret_cast<T*>(p + used) : nullptr;
    used += (bytes + 255) / 256 * 256;
  }
};

// Bytes a value takes where it is kept in full: two bf16, or one float.
constexpr size_t kFull = 4;

size_t place_saved(DeltaArgs& a, char* p) {
  Regions r{p};
  const size_t heads = (size_t)a.B * a.H, chunks = heads * a.N, e = a.dtype == GLA_BF16 ? 2 : 4;
  r.take(a.gates, chunks * kDeltaGates * 4);
  r.take(a.solveT, chunks * kDeltaChunk * kDeltaChunk * kFull);
  if (a.P > 1) r.take(a.trans, heads * a.P * a.DKP * a.DKP * kFull);
  r.take(a.err, chunks * kDeltaChunk * a.DVP * 4);
  if (a.dtype == GLA_BF16) r.take(a.o_rest, chunks * kDeltaChunk * a.DVP * 2);
  r.take(a.state0, chunks * a.DVP * a.DKP * e);
  r.take(a.mark, heads * (a.marks + 1) * a.DVP * a.DKP * 4);
  return r.used;
}

size_t place_scratch(DeltaArgs& a, char* p, bool backward, bool train) {
  Regions r{p};
  const size_t heads = (size_t)a.B * a.H, chunks = heads * a.N, e = a.dtype == GLA_BF16 ? 2 : 4;
  const size_t rows = (size_t)a.B * a.T * e * (backward ? 2 : 1);  // of v, and of do
  if (a.dk % 8) r.take(a.qk_packed, (size_t)a.B * a.T * e * 2 * a.Hk * a.dkr);
  if (a.dv % 8) r.take(a.v_packed, rows * a.H * a.dvr);
  if (a.P > 1) {
    r.take(a.seg, heads * a.P * a.DVP * a.DKP * 4);
    r.take(a.seg_in, heads * a.P * a.DVP * a.DKP * 4);
  }
  if (!backward) {
    r.take(a.solve, chunks * kDeltaChunk * kDeltaChunk * kFull);
    if (a.P > 1) r.take(a.trans_rows, heads * a.P * a.DKP * a.DKP * kFull);
    if (!train) r.take(a.gates, chunks * kDeltaGates * 4);
    return r.used;
  }
  r.take(a.z, chunks * kDeltaChunk * a.DVP * 4);
  r.take(a.grad1, chunks * a.DVP * a.DKP * e);
  r.take(a.carry, heads * (a.marks + 1) * (a.DVP / 16) * 4);
  r.take(a.at, chunks * kDeltaChunk * 8);
  if (a.H != a.Hk) {
    r.take(a.dq_heads, heads * a.T * a.dk * 4);
    r.take(a.dk_heads, heads * a.T * a.dk * 4);
  }
  return r.used;
}

}  // namespace

size_t delta_saved_bytes(const DeltaShape& s) {
  DeltaArgs a{};
  static_cast<DeltaShape&>(a) = s;
  return place_saved(a, nullptr);
}
size_t delta_scratch_bytes(const DeltaShape& s, bool backward, bool train) {
  DeltaArgs a{};
  static_cast<DeltaShape&>(a) = s;
  return place_scratch(a, nullptr, backward, train);
}
void delta_place(DeltaArgs& a, void* saved, void* scratch, bool backward) {
  if (saved) place_saved(a, static_cast<char*>(saved));
  place_scratch(a, static_cast<char*>(scratch), backward, saved);
}

}  // namespace gla

namespace {

gla_status check_delta(const char* fn, int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  if (B < 1 || H < 1 || Hk < 1 || T < 1 || dk < 1 || dv < 1)
    return set_error(GLA_ERR_INVALID_ARG, "%s: B, H, Hk, T, dk and dv must be >= 1", fn);
  if (H % Hk != 0) return set_error(GLA_ERR_INVALID_ARG, "%s: H=%d is no multiple of Hk=%d", fn, H, Hk);
  GLA_TRY(check_dtype(fn, dtype));
  if (dk > gla::kDeltaMaxDk || dv > gla::kDeltaMaxDv)
    return set_error(GLA_ERR_UNSUPPORTED, "%s: dk=%d or dv=%d is above %d, %d", fn, dk, dv, gla::kDeltaMaxDk, gla::kDeltaMaxDv);
  // a workgroup a chunk of a head; in the walk at most 256 of segments, or 16 a head (64 columns each)
  const long long heads = (long long)B * H, chunks = ((long long)T + gla::kDeltaChunk - 1) / gla::kDeltaChunk;
  if (heads > kMaxGrid / 16 || heads * chunks > kMaxGrid)
    return set_error(GLA_ERR_UNSUPPORTED, "%s: B*H=%lld heads of T=%d tokens are too many for one call", fn, heads, T);
  return GLA_OK;
}

// The inputs both directions share, as regions and into the arguments.
struct DeltaInputs {
  const void *q, *k, *v;
  const float *g, *beta;
  const gla_strides *q_st, *k_st, *v_st, *g_st, *b_st;
};
gla_status take_inputs(const char* fn, const DeltaInputs& in, gla::DeltaArgs& a) {
  if (!in.q || !in.k || !in.v || !in.g || !in.beta)
    return set_error(GLA_ERR_INVALID_ARG, "%s: q, k, v, g and beta must be non-null", fn);
  const long long T = a.T, kT = a.Hk * T, hT = a.H * T;
  if (!strides(in.q_st, kT * a.dk, T * a.dk, a.dk, &a.qs) || !strides(in.k_st, kT * a.dk, T * a.dk, a.dk, &a.ks) ||
      !strides(in.v_st, hT * a.dv, T * a.dv, a.dv, &a.vs) || !strides(in.g_st, hT, T, 1, &a.gs) ||
      !strides(in.b_st, hT, T, 1, &a.bs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  a.q = in.q;
  a.k = in.k;
  a.v = in.v;
  a.g = in.g;
  a.beta = in.beta;
  return GLA_OK;
}

gla_status check_buffer(const char* fn, const char* name, const void* p, size_t bytes, size_t need) {
  if (!p || bytes < need)
    return set_error(GLA_ERR_INVALID_ARG, "%s: needs %s of %zu bytes, got %zu", fn, name, need, p ? bytes : (size_t)0);
  if ((unsigned long long)p % 16 != 0) return set_error(GLA_ERR_INVALID_ARG, "%s: %s must lie on 16 bytes", fn, name);
  return GLA_OK;
}

}  // namespace

extern "C" {

size_t gla_delta_workspace_size(int which, int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  const char* fn = "gla_delta_workspace_size";
  if (which != GLA_FWD && which != GLA_BWD) {
    set_error(GLA_ERR_INVALID_ARG, "%s: which must be GLA_FWD or GLA_BWD", fn);
    return 0;
  }
  if (check_delta(fn, B, H, Hk, T, dk, dv, dtype) != GLA_OK) return 0;
  set_error(GLA_OK, "");
  return gla::delta_scratch_bytes(gla::delta_shape(B, H, Hk, T, dk, dv, dtype), which == GLA_BWD, false);
}

size_t gla_delta_saved_size(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  if (check_delta("gla_delta_saved_size", B, H, Hk, T, dk, dv, dtype) != GLA_OK) return 0;
  set_error(GLA_OK, "");
  return gla::delta_saved_bytes(gla::delta_shape(B, H, Hk, T, dk, dv, dtype));
}

gla_status gla_delta_fwd(const void* q, const gla_strides* q_st, const void* k, const gla_strides* k_st, const void* v,
                         const gla_strides* v_st, const float* g, const gla_strides* g_st, const float* beta,
                         const gla_strides* b_st, const float* h0, const int* lens, void* o, float* h_final, void* saved,
                         size_t saved_size, int B, int H, int Hk, int T, int dk, int dv, int dtype, void* workspace,
                         size_t workspace_size, void* stream) {
  const char* fn = "gla_delta_fwd";
  GLA_TRY(check_delta(fn, B, H, Hk, T, dk, dv, dtype));
  gla::DeltaArgs a{};
  static_cast<gla::DeltaShape&>(a) = gla::delta_shape(B, H, Hk, T, dk, dv, dtype);
  GLA_TRY(take_inputs(fn, {q, k, v, g, beta, q_st, k_st, v_st, g_st, b_st}, a));
  if (!o) return set_error(GLA_ERR_INVALID_ARG, "%s: o must be non-null", fn);
  const size_t need = gla::delta_scratch_bytes(a, false, saved), keep = saved ? gla::delta_saved_bytes(a) : 0;
  GLA_TRY(check_buffer(fn, "a workspace", workspace, workspace_size, need));
  if (saved) GLA_TRY(check_buffer(fn, "saved", saved, saved_size, keep));
  const int e = size_of(dtype);
  const wide state = (wide)B * H * dk * dv;
  if (overlaps<4, 7>({{o, (wide)B * H * T * dv, e}, {h_final, state}, {saved, (wide)keep, 1}, {workspace, (wide)need, 1}},
                     {{q, e, B, Hk, T, dk, a.qs}, {k, e, B, Hk, T, dk, a.ks}, {v, e, B, H, T, dv, a.vs},
                      {g, 4, B, H, T, 1, a.gs}, {beta, 4, B, H, T, 1, a.bs}, {h0, state}, {lens, B, 4}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs and buffers must not overlap inputs or each other", fn);
  a.h0 = h0;
  a.lens = lens;
  a.o = o;
  a.h_final = h_final;
  gla::delta_place(a, saved, workspace, false);
  return launched(fn, gla::launch_delta_fwd(a, static_cast<hipStream_t>(stream)));
}

gla_status gla_delta_bwd(const void* q, const gla_strides* q_st, const void* k, const gla_strides* k_st, const void* v,
                         const gla_strides* v_st, const float* g, const gla_strides* g_st, const float* beta,
                         const gla_strides* b_st, const void* o, const void* do_, const gla_strides* do_st, void* saved,
                         size_t saved_size, const int* lens, const float* dhT, void* dq, void* dk_, void* dv_, float* dg,
                         float* dbeta, float* dh0, int B, int H, int Hk, int T, int dk, int dv, int dtype,
                         void* workspace, size_t workspace_size, void* stream) {
  const char* fn = "gla_delta_bwd";
  GLA_TRY(check_delta(fn, B, H, Hk, T, dk, dv, dtype));
  gla::DeltaArgs a{};
  static_cast<gla::DeltaShape&>(a) = gla::delta_shape(B, H, Hk, T, dk, dv, dtype);
  GLA_TRY(take_inputs(fn, {q, k, v, g, beta, q_st, k_st, v_st, g_st, b_st}, a));
  if (!o || !do_ || !dq || !dk_ || !dv_ || !dg || !dbeta)
    return set_error(GLA_ERR_INVALID_ARG, "%s: o, do, dq, dk, dv, dg and dbeta must be non-null", fn);
  const long long hT = (long long)H * T;
  if (!strides(do_st, hT * dv, (long long)T * dv, dv, &a.dos))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  const size_t need = gla::delta_scratch_bytes(a, true, true), keep = gla::delta_saved_bytes(a);
  GLA_TRY(check_buffer(fn, "a workspace", workspace, workspace_size, need));
  GLA_TRY(check_buffer(fn, "saved", saved, saved_size, keep));
  const int e = size_of(dtype);
  const wide state = (wide)B * H * dk * dv, keys = (wide)B * Hk * T * dk, values = (wide)B * hT * dv, rows = (wide)B * hT;
  if (overlaps<7, 10>({{dq, keys, e}, {dk_, keys, e}, {dv_, values, e}, {dg, rows}, {dbeta, rows}, {dh0, state},
                       {workspace, (wide)need, 1}},
                      {{q, e, B, Hk, T, dk, a.qs}, {k, e, B, Hk, T, dk, a.ks}, {v, e, B, H, T, dv, a.vs},
                       {g, 4, B, H, T, 1, a.gs}, {beta, 4, B, H, T, 1, a.bs}, {o, values, e}, {do_, e, B, H, T, dv, a.dos},
                       {saved, (wide)keep, 1}, {lens, B, 4}, {dhT, state}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs and the workspace must not overlap inputs or each other", fn);
  a.lens = lens;
  a.o = const_cast<void*>(o);
  a.dO = do_;
  a.dhT = dhT;
  a.dq = dq;
  a.dk_ = dk_;
  a.dv_ = dv_;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dh0 = dh0;
  gla::delta_place(a, saved, workspace, true);
  return launched(fn, gla::launch_delta_bwd(a, static_cast<hipStream_t>(stream)));
}

gla_status gla_delta_step(const void* q, const gla_strides* q_st, const void* k, const gla_strides* k_st, const void* v,
                          const gla_strides* v_st, const float* g, const gla_strides* g_st, const float* beta,
                          const gla_strides* b_st, float* state, const int* slots, void* o, int B, int H, int Hk, int n,
                          int dk, int dv, int n_slots, int dtype, void* stream) {
  const char* fn = "gla_delta_step";
  if (B < 1 || H < 1 || Hk < 1 || n < 1 || dk < 1 || dv < 1)
    return set_error(GLA_ERR_INVALID_ARG, "%s: B, H, Hk, n, dk and dv must be >= 1", fn);
  if (H % Hk != 0) return set_error(GLA_ERR_INVALID_ARG, "%s: H=%d is no multiple of Hk=%d", fn, H, Hk);
  GLA_TRY(check_dtype(fn, dtype));
  if (!q || !k || !v || !g || !beta || !state || !o)
    return set_error(GLA_ERR_INVALID_ARG, "%s: q, k, v, g, beta, state and o must be non-null", fn);
  if (n_slots < 1 || (!slots && n_slots < B))
    return set_error(GLA_ERR_INVALID_ARG, "%s: the pool's %d states do not serve %d rows", fn, n_slots, B);
  gla::DeltaStepArgs a{};
  const long long N = n, KN = (long long)Hk * n, HN = (long long)H * n;
  if (!strides(q_st, KN * dk, N * dk, dk, &a.qs) || !strides(k_st, KN * dk, N * dk, dk, &a.ks) ||
      !strides(v_st, HN * dv, N * dv, dv, &a.vs) || !strides(g_st, HN, N, 1, &a.gs) || !strides(b_st, HN, N, 1, &a.bs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  if (dk > gla::kStepMaxDk) return set_error(GLA_ERR_UNSUPPORTED, "%s: dk=%d is above %d", fn, dk, gla::kStepMaxDk);
  if ((long long)B * H > kMaxGrid / ((dv + 15LL) / 16))
    return set_error(GLA_ERR_UNSUPPORTED, "%s: B*H=%lld heads of dv=%d are too many for one call", fn,
                     (long long)B * H, dv);
  const int e = size_of(dtype);
  if (overlaps<2, 6>({{state, (wide)n_slots * H * dk * dv}, {o, (wide)B * HN * dv, e}},
                     {{q, e, B, Hk, n, dk, a.qs}, {k, e, B, Hk, n, dk, a.ks}, {v, e, B, H, n, dv, a.vs},
                      {g, 4, B, H, n, 1, a.gs}, {beta, 4, B, H, n, 1, a.bs}, {slots, B, 4}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: o and state must not overlap inputs or each other", fn);
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.state = state;
  a.slots = slots;
  a.o = o;
  a.B = B;
  a.H = H;
  a.Hk = Hk;
  a.n = n;
  a.dk = dk;
  a.dv = dv;
  a.n_slots = n_slots;
  a.dtype = dtype;
  return launched(fn, gla::launch_delta_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

gla_status check_norm(const char* fn, int B, int T, int D, int dtype, int stream_dtype) {
  if (B < 1 || T < 1 || D < 1) return set_error(GLA_ERR_INVALID_ARG, "%s: B, T and D must be >= 1", fn);
  GLA_TRY(check_dtype(fn, dtype));
  GLA_TRY(check_dtype(fn, stream_dtype));
  if (dtype == GLA_F32 && stream_dtype != GLA_F32)
    return set_error(GLA_ERR_UNSUPPORTED, "%s: a bf16 stream with float32 blocks", fn);
  if (D > gla::kNormMaxRow) return set_error(GLA_ERR_UNSUPPORTED, "%s: rows of D=%d are above %d", fn, D, gla::kNormMaxRow);
  return GLA_OK;
}

}  // namespace

extern "C" {

size_t gla_layernorm_workspace_size(int B, int T, int D) {
  if (check_norm("gla_layernorm_workspace_size", B, T, D, GLA_F32, GLA_F32) != GLA_OK) return 0;
  set_error(GLA_OK, "");
  return (gla::norm_partial_floats(B, T, D) * sizeof(float) + 255) / 256 * 256;
}

gla_status gla_layernorm_fwd(const void* x, const gla_strides* x_st, const void* residual, const gla_strides* r_st,
                             const float* w, const float* b, void* out, void* normed, float* mean, float* rstd, int B,
                             int T, int D, float eps, int dtype, int stream_dtype, void* stream) {
  const char* fn = "gla_layernorm_fwd";
  GLA_TRY(check_norm(fn, B, T, D, dtype, stream_dtype));
  if (!x || !normed) return set_error(GLA_ERR_INVALID_ARG, "%s: x and normed must be non-null", fn);
  if (out && !residual) return set_error(GLA_ERR_INVALID_ARG, "%s: out needs a residual (without one it is x)", fn);
  if (!mean != !rstd) return set_error(GLA_ERR_INVALID_ARG, "%s: mean and rstd go together", fn);
  if (!(eps > 0.f)) return set_error(GLA_ERR_INVALID_ARG, "%s: eps must be above zero", fn);
  gla::NormArgs a{};
  const long long n = T;
  if (!strides(x_st, n * D, 0, D, &a.xs) || !strides(residual ? r_st : nullptr, n * D, 0, D, &a.rs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  // out may be the residual itself (each lane reads its elements before it writes them), in the same place
  const bool in_place = out && out == residual;
  if (in_place && ((T > 1 && a.rs.t != D) || (B > 1 && a.rs.b != n * D)))
    return set_error(GLA_ERR_INVALID_ARG, "%s: an out in the residual's place needs a contiguous residual", fn);
  const int e = size_of(dtype), se = size_of(stream_dtype);
  const wide rows = (wide)B * T;
  if (overlaps<4, 4>({{out, rows * D, se}, {normed, rows * D, e}, {mean, rows}, {rstd, rows}},
                     {{x, e, B, 1, T, D, a.xs}, {in_place ? nullptr : residual, se, B, 1, T, D, a.rs}, {w, D}, {b, D}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs must not overlap inputs or each other", fn);
  a.x = x;
  a.residual = residual;
  a.w = w;
  a.b = b;
  a.out = out;
  a.normed = normed;
  a.mean = mean;
  a.rstd = rstd;
  a.B = B;
  a.T = T;
  a.D = D;
  a.eps = eps;
  a.dtype = dtype;
  a.stream_dtype = stream_dtype;
  return launched(fn, gla::launch_layernorm(a, false, static_cast<hipStream_t>(stream)));
}

gla_status gla_layernorm_bwd(const void* x, const gla_strides* x_st, const void* residual, const gla_strides* r_st,
                             const float* w, const float* mean, const float* rstd, const void* d_out,
                             const gla_strides* do_st, const void* d_normed, const gla_strides* dn_st, void* dx,
                             void* d_residual, float* dw, float* db, int B, int T, int D, int dtype, int stream_dtype,
                             void* workspace, size_t workspace_size, void* stream) {
  const char* fn = "gla_layernorm_bwd";
  GLA_TRY(check_norm(fn, B, T, D, dtype, stream_dtype));
  if (!x || !mean || !rstd || !d_normed || !dx)
    return set_error(GLA_ERR_INVALID_ARG, "%s: x, mean, rstd, d_normed and dx must be non-null", fn);
  if (d_residual && !residual) return set_error(GLA_ERR_INVALID_ARG, "%s: d_residual needs a residual", fn);
  const bool sums = dw || db;
  const size_t need = sums ? gla_layernorm_workspace_size(B, T, D) : 0;
  if (sums && (!workspace || workspace_size < need))
    return set_error(GLA_ERR_INVALID_ARG, "%s: the weights' gradients need a workspace of %zu bytes, got %zu", fn, need,
                     workspace ? workspace_size : (size_t)0);
  if (sums && (unsigned long long)workspace % 4 != 0)
    return set_error(GLA_ERR_INVALID_ARG, "%s: the workspace must lie on 4 bytes", fn);
  gla::NormArgs a{};
  const long long n = T;
  if (!strides(x_st, n * D, 0, D, &a.xs) || !strides(residual ? r_st : nullptr, n * D, 0, D, &a.rs) ||
      !strides(d_out ? do_st : nullptr, n * D, 0, D, &a.dos) || !strides(dn_st, n * D, 0, D, &a.dns))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  const int e = size_of(dtype), se = size_of(stream_dtype);
  const wide rows = (wide)B * T;
  if (overlaps<5, 7>({{dx, rows * D, e}, {d_residual, rows * D, se}, {dw, D}, {db, D}, {sums ? workspace : nullptr, (wide)need, 1}},
                     {{x, e, B, 1, T, D, a.xs}, {residual, se, B, 1, T, D, a.rs}, {w, D}, {mean, rows}, {rstd, rows},
                      {d_out, se, B, 1, T, D, a.dos}, {d_normed, e, B, 1, T, D, a.dns}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs and the workspace must not overlap inputs or each other", fn);
  a.x = x;
  a.residual = residual;
  a.w = w;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.d_out = d_out;
  a.d_normed = d_normed;
  a.dx = dx;
  a.d_residual = d_residual;
  a.dw = dw;
  a.db = db;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.B = B;
  a.T = T;
  a.D = D;
  a.dtype = dtype;
  a.stream_dtype = stream_dtype;
  return launched(fn, gla::launch_layernorm(a, true, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
