// C ABI of the recurrent-block operators (declared in include/gla.h): host-side argument checks,
// then kernel launches on the caller's stream.  Every check runs before the first HIP call.
#include "gla.h"

#include "gla_block.hpp"
#include "gla_checks.hpp"

namespace {

gla_status check_recur(const char* fn, int B, int T, int D, int mode, int dtype) {
  if (B < 1 || T < 1 || D < 1) return set_error(GLA_ERR_INVALID_ARG, "%s: B, T and D must be >= 1", fn);
  if (mode < GLA_RECUR_PLAIN || mode > GLA_RECUR_NORM)
    return set_error(GLA_ERR_INVALID_ARG, "%s: unknown mode %d", fn, mode);
  GLA_TRY(check_dtype(fn, dtype));
  const long long tiles = B * ((D + 63LL) / 64);
  if (B > 65535 || D >= gla::kMaxStride || tiles > kMaxGrid || tiles * (((long long)T + gla::kRecurTile - 1) / gla::kRecurTile) > kMaxGrid)
    return set_error(GLA_ERR_UNSUPPORTED, "%s: B=%d, T=%d, D=%d are too many for one call", fn, B, T, D);
  return GLA_OK;
}

size_t recur_bytes(int B, int T, int D) {
  return (gla::recur_workspace_words(B, T, D) * sizeof(unsigned long long) + 255) / 256 * 256;
}

// The scan's workspace: recur_bytes, on 8 bytes.
gla_status check_recur_workspace(const char* fn, int B, int T, int D, void* ws, size_t bytes) {
  const size_t need = recur_bytes(B, T, D);
  if (need && (!ws || bytes < need))
    return set_error(GLA_ERR_INVALID_ARG, "%s: needs a workspace of %zu bytes, got %zu", fn, need, ws ? bytes : (size_t)0);
  if (need && (unsigned long long)ws % 8 != 0)
    return set_error(GLA_ERR_INVALID_ARG, "%s: the workspace must lie on 8 bytes", fn);
  return GLA_OK;
}

}  // namespace

extern "C" {

size_t gla_recur_workspace_size(int B, int T, int D) {
  if (check_recur("gla_recur_workspace_size", B, T, D, GLA_RECUR_PLAIN, GLA_F32) != GLA_OK) return 0;
  set_error(GLA_OK, "");
  return recur_bytes(B, T, D);
}

gla_status gla_recur_fwd(const void* x, const gla_strides* x_st, const float* g, const gla_strides* g_st,
                         const float* h0, const int* lens, void* h, float* chunk_in, float* h_final, int B, int T,
                         int D, int mode, int dtype, void* workspace, size_t workspace_size, void* stream) {
  const char* fn = "gla_recur_fwd";
  GLA_TRY(check_recur(fn, B, T, D, mode, dtype));
  if (!x || !g || !h) return set_error(GLA_ERR_INVALID_ARG, "%s: x, g and h must be non-null", fn);
  gla::RecurArgs a{};
  if (!strides(x_st, (long long)T * D, 0, D, &a.xs) || !strides(g_st, (long long)T * D, 0, D, &a.gs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  if (T > 1 && (a.xs.t >= gla::kMaxStride || a.gs.t >= gla::kMaxStride))
    return set_error(GLA_ERR_UNSUPPORTED, "%s: token strides must be below %d elements", fn, gla::kMaxStride);
  GLA_TRY(check_recur_workspace(fn, B, T, D, workspace, workspace_size));
  const int e = size_of(dtype);
  const wide n = (wide)B * T * D, row = (wide)B * D, states = (wide)B * ((T + gla::kRecurChunk - 1LL) / gla::kRecurChunk) * D;
  if (overlaps<4, 4>({{h, n, e}, {chunk_in, states}, {h_final, row}, {workspace, (wide)recur_bytes(B, T, D), 1}},
                     {{x, e, B, 1, T, D, a.xs}, {g, 4, B, 1, T, D, a.gs}, {h0, row}, {lens, B, 4}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs and the workspace must not overlap inputs or each other", fn);
  a.x = x;
  a.g = g;
  a.h0 = h0;
  a.lens = lens;
  a.h = h;
  a.chunk_in = chunk_in;
  a.h_final = h_final;
  a.B = B;
  a.T = T;
  a.D = D;
  a.mode = mode;
  a.dtype = dtype;
  a.words = static_cast<unsigned long long*>(workspace);
  return launched(fn, gla::launch_recur_fwd(a, static_cast<hipStream_t>(stream)));
}

gla_status gla_recur_bwd(const void* x, const gla_strides* x_st, const float* g, const gla_strides* g_st,
                         const void* dh, const gla_strides* dh_st, const float* chunk_in, const int* lens,
                         const float* dhT, void* dx, float* dg, float* dh0, int B, int T, int D, int mode, int dtype,
                         void* workspace, size_t workspace_size, void* stream) {
  const char* fn = "gla_recur_bwd";
  GLA_TRY(check_recur(fn, B, T, D, mode, dtype));
  if (!x || !g || !dh || !chunk_in || !dx || !dg)
    return set_error(GLA_ERR_INVALID_ARG, "%s: x, g, dh, chunk_in, dx and dg must be non-null", fn);
  gla::RecurArgs a{};
  if (!strides(x_st, (long long)T * D, 0, D, &a.xs) || !strides(g_st, (long long)T * D, 0, D, &a.gs) ||
      !strides(dh_st, (long long)T * D, 0, D, &a.dhs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  if (T > 1 && (a.xs.t >= gla::kMaxStride || a.gs.t >= gla::kMaxStride || a.dhs.t >= gla::kMaxStride))
    return set_error(GLA_ERR_UNSUPPORTED, "%s: token strides must be below %d elements", fn, gla::kMaxStride);
  GLA_TRY(check_recur_workspace(fn, B, T, D, workspace, workspace_size));
  const int e = size_of(dtype);
  const wide n = (wide)B * T * D, row = (wide)B * D, states = (wide)B * ((T + gla::kRecurChunk - 1LL) / gla::kRecurChunk) * D;
  if (overlaps<4, 6>({{dx, n, e}, {dg, n}, {dh0, row}, {workspace, (wide)recur_bytes(B, T, D), 1}},
                     {{x, e, B, 1, T, D, a.xs}, {g, 4, B, 1, T, D, a.gs}, {dh, e, B, 1, T, D, a.dhs}, {chunk_in, states},
                      {lens, B, 4}, {dhT, row}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs and the workspace must not overlap inputs or each other", fn);
  a.x = x;
  a.g = g;
  a.dh = dh;
  a.lens = lens;
  a.chunk_in = const_cast<float*>(chunk_in);
  a.dhT = dhT;
  a.h = dx;
  a.dg = dg;
  a.h_final = dh0;
  a.B = B;
  a.T = T;
  a.D = D;
  a.mode = mode;
  a.dtype = dtype;
  a.words = static_cast<unsigned long long*>(workspace);
  return launched(fn, gla::launch_recur_bwd(a, static_cast<hipStream_t>(stream)));
}

gla_status gla_recur_step(const void* x, const gla_strides* x_st, const float* g, const gla_strides* g_st,
                          float* state, const int* slots, void* h, int B, int D, int n_slots, int mode, int dtype,
                          void* stream) {
  const char* fn = "gla_recur_step";
  GLA_TRY(check_recur(fn, B, 1, D, mode, dtype));
  if (!x || !g || !state || !h) return set_error(GLA_ERR_INVALID_ARG, "%s: x, g, state and h must be non-null", fn);
  if (n_slots < 1 || (!slots && n_slots < B))
    return set_error(GLA_ERR_INVALID_ARG, "%s: the pool's %d states do not serve %d rows", fn, n_slots, B);
  gla::RecurStepArgs a{};
  if (!strides(x_st, D, 0, 0, &a.xs) || !strides(g_st, D, 0, 0, &a.gs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  const int e = size_of(dtype);
  if (overlaps<2, 3>({{state, (wide)n_slots * D}, {h, (wide)B * D, e}},
                     {{x, e, B, 1, 1, D, a.xs}, {g, 4, B, 1, 1, D, a.gs}, {slots, B, 4}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: h and state must not overlap inputs or each other", fn);
  a.x = x;
  a.g = g;
  a.state = state;
  a.slots = slots;
  a.h = h;
  a.B = B;
  a.D = D;
  a.n_slots = n_slots;
  a.mode = mode;
  a.dtype = dtype;
  return launched(fn, gla::launch_recur_step(a, static_cast<hipStream_t>(stream)));
}

gla_status gla_step(const void* q, const gla_strides* q_st, const void* k, const gla_strides* k_st, const void* v,
                    const gla_strides* v_st, const float* g, const gla_strides* g_st, float* state, const int* slots,
                    void* o, int B, int H, int n, int dk, int dv, int n_slots, int dtype, void* stream) {
  const char* fn = "gla_step";
  if (B < 1 || H < 1 || n < 1 || dk < 1 || dv < 1)
    return set_error(GLA_ERR_INVALID_ARG, "%s: B, H, n, dk and dv must be >= 1", fn);
  GLA_TRY(check_dtype(fn, dtype));
  if (!q || !k || !v || !g || !state || !o)
    return set_error(GLA_ERR_INVALID_ARG, "%s: q, k, v, g, state and o must be non-null", fn);
  if (n_slots < 1 || (!slots && n_slots < B))
    return set_error(GLA_ERR_INVALID_ARG, "%s: the pool's %d states do not serve %d rows", fn, n_slots, B);
  gla::StepArgs a{};
  const long long N = n, HN = (long long)H * n;
  if (!strides(q_st, HN * dk, N * dk, dk, &a.qs) || !strides(k_st, HN * dk, N * dk, dk, &a.ks) ||
      !strides(v_st, HN * dv, N * dv, dv, &a.vs) || !strides(g_st, HN * dk, N * dk, dk, &a.gs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  if (dk > gla::kStepMaxDk) return set_error(GLA_ERR_UNSUPPORTED, "%s: dk=%d is above %d", fn, dk, gla::kStepMaxDk);
  if ((long long)B * H > kMaxGrid / ((dv + 15LL) / 16))
    return set_error(GLA_ERR_UNSUPPORTED, "%s: B*H=%lld heads of dv=%d are too many for one call", fn,
                     (long long)B * H, dv);
  const int e = size_of(dtype);
  if (overlaps<2, 5>({{state, (wide)n_slots * H * dk * dv}, {o, (wide)B * HN * dv, e}},
                     {{q, e, B, H, n, dk, a.qs}, {k, e, B, H, n, dk, a.ks}, {v, e, B, H, n, dv, a.vs},
                      {g, 4, B, H, n, dk, a.gs}, {slots, B, 4}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: o and state must not overlap inputs or each other", fn);
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.state = state;
  a.slots = slots;
  a.o = o;
  a.B = B;
  a.H = H;
  a.n = n;
  a.dk = dk;
  a.dv = dv;
  a.n_slots = n_slots;
  a.dtype = dtype;
  return launched(fn, gla::launch_step(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

gla_status check_join(const char* fn, int B, int H, int T, int d, int act, int dtype, int stream_dtype) {
  if (B < 1 || H < 1 || T < 1 || d < 1) return set_error(GLA_ERR_INVALID_ARG, "%s: B, H, T and d must be >= 1", fn);
  if (act != GLA_ACT_SILU && act != GLA_ACT_SIGMOID)
    return set_error(GLA_ERR_INVALID_ARG, "%s: unknown act %d", fn, act);
  GLA_TRY(check_dtype(fn, dtype));
  GLA_TRY(check_dtype(fn, stream_dtype));
  if (dtype == GLA_F32 && stream_dtype != GLA_F32)
    return set_error(GLA_ERR_UNSUPPORTED, "%s: a bf16 stream with float32 blocks", fn);
  if ((long long)H * d > gla::kJoinMaxRow)
    return set_error(GLA_ERR_UNSUPPORTED, "%s: rows of H*d=%lld are above %d", fn, (long long)H * d, gla::kJoinMaxRow);
  if (H > gla::kJoinMaxHeads)
    return set_error(GLA_ERR_UNSUPPORTED, "%s: rows of H=%d heads are above %d", fn, H, gla::kJoinMaxHeads);
  return GLA_OK;
}

}  // namespace

extern "C" {

size_t gla_join_workspace_size(int B, int H, int T, int d) {
  if (check_join("gla_join_workspace_size", B, H, T, d, GLA_ACT_SILU, GLA_F32, GLA_F32) != GLA_OK) return 0;
  set_error(GLA_OK, "");
  return (gla::join_partial_floats(B, H, T, d) * sizeof(float) + 255) / 256 * 256;
}

gla_status gla_join_fwd(const void* y, const gla_strides* y_st, const void* z, const gla_strides* z_st,
                        const float* w_post, const void* residual, const gla_strides* r_st, const float* scale,
                        const float* w_pre, void* out, void* normed, float* rstd_post, float* rstd_pre, int B, int H,
                        int T, int d, int act, float eps, int dtype, int stream_dtype, void* stream) {
  const char* fn = "gla_join_fwd";
  GLA_TRY(check_join(fn, B, H, T, d, act, dtype, stream_dtype));
  if (!y || !out) return set_error(GLA_ERR_INVALID_ARG, "%s: y and out must be non-null", fn);
  if ((w_pre != nullptr) != (normed != nullptr))
    return set_error(GLA_ERR_INVALID_ARG, "%s: w_pre and normed go together", fn);
  if ((rstd_post && !w_post) || (rstd_pre && !w_pre))
    return set_error(GLA_ERR_INVALID_ARG, "%s: rstd_post needs w_post and rstd_pre needs w_pre", fn);
  if (!(eps > 0.f)) return set_error(GLA_ERR_INVALID_ARG, "%s: eps must be above zero", fn);
  gla::JoinArgs a{};
  const long long D = (long long)H * d, n = T;
  if (!strides(y_st, n * D, n * d, d, &a.ys) || !strides(z ? z_st : nullptr, n * D, 0, D, &a.zs) ||
      !strides(residual ? r_st : nullptr, n * D, 0, D, &a.rs))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  // out may be the residual itself (each lane reads its elements before it writes them), in the
  // same place: contiguous
  const bool in_place = out == residual;
  if (in_place && ((T > 1 && a.rs.t != D) || (B > 1 && a.rs.b != n * D)))
    return set_error(GLA_ERR_INVALID_ARG, "%s: an out in the residual's place needs a contiguous residual", fn);
  const int e = size_of(dtype), se = size_of(stream_dtype);
  const wide rows = (wide)B * T;
  if (overlaps<4, 6>({{out, rows * D, se}, {normed, rows * D, e}, {rstd_post, rows * H}, {rstd_pre, rows}},
                     {{y, e, B, H, T, d, a.ys}, {z, e, B, 1, T, (int)D, a.zs}, {w_post, d},
                      {in_place ? nullptr : residual, se, B, 1, T, (int)D, a.rs}, {scale, D}, {w_pre, D}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs must not overlap inputs or each other", fn);
  a.y = y;
  a.z = z;
  a.residual = residual;
  a.w_post = w_post;
  a.scale = scale;
  a.w_pre = w_pre;
  a.out = out;
  a.normed = normed;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  a.B = B;
  a.H = H;
  a.T = T;
  a.d = d;
  a.act = act;
  a.eps = eps;
  a.dtype = dtype;
  a.stream_dtype = stream_dtype;
  return launched(fn, gla::launch_join_fwd(a, static_cast<hipStream_t>(stream)));
}

gla_status gla_join_bwd(const void* y, const gla_strides* y_st, const void* z, const gla_strides* z_st,
                        const float* w_post, const void* residual, const gla_strides* r_st, const float* scale,
                        const float* w_pre, const float* rstd_post, const float* rstd_pre, const void* d_out,
                        const gla_strides* do_st, const void* d_normed, const gla_strides* dn_st, void* dy, void* dz,
                        void* d_residual, float* dw_post, float* dscale, float* dw_pre, int B, int H, int T, int d,
                        int act, int dtype, int stream_dtype, void* workspace, size_t workspace_size, void* stream) {
  const char* fn = "gla_join_bwd";
  GLA_TRY(check_join(fn, B, H, T, d, act, dtype, stream_dtype));
  if (!y || !dy) return set_error(GLA_ERR_INVALID_ARG, "%s: y and dy must be non-null", fn);
  if (!d_out && !d_normed) return set_error(GLA_ERR_INVALID_ARG, "%s: d_out or d_normed must be non-null", fn);
  if (d_normed && (!w_pre || !rstd_pre))
    return set_error(GLA_ERR_INVALID_ARG, "%s: d_normed needs w_pre and rstd_pre", fn);
  if ((w_post != nullptr) != (rstd_post != nullptr))
    return set_error(GLA_ERR_INVALID_ARG, "%s: w_post and rstd_post go together", fn);
  if ((z != nullptr) != (dz != nullptr)) return set_error(GLA_ERR_INVALID_ARG, "%s: z and dz go together", fn);
  if ((dw_post && !w_post) || (dscale && !scale) || (dw_pre && !w_pre) || (d_residual && !residual))
    return set_error(GLA_ERR_INVALID_ARG, "%s: a gradient is asked for of an input that is null", fn);
  const bool sums = dw_post || dscale || dw_pre;
  const size_t need = sums ? gla_join_workspace_size(B, H, T, d) : 0;
  if (sums && (!workspace || workspace_size < need))
    return set_error(GLA_ERR_INVALID_ARG, "%s: the weights' gradients need a workspace of %zu bytes, got %zu", fn, need,
                     workspace ? workspace_size : (size_t)0);
  gla::JoinArgs a{};
  const long long D = (long long)H * d, n = T;
  if (!strides(y_st, n * D, n * d, d, &a.ys) || !strides(z ? z_st : nullptr, n * D, 0, D, &a.zs) ||
      !strides(residual ? r_st : nullptr, n * D, 0, D, &a.rs) || !strides(d_out ? do_st : nullptr, n * D, 0, D, &a.dos) ||
      !strides(d_normed ? dn_st : nullptr, n * D, 0, D, &a.dns))
    return set_error(GLA_ERR_INVALID_ARG, "%s: strides must not be negative", fn);
  const int e = size_of(dtype), se = size_of(stream_dtype), W = (int)D;
  const wide rows = (wide)B * T;
  if (overlaps<7, 10>({{dy, rows * D, e}, {dz, rows * D, e}, {d_residual, rows * D, se}, {dw_post, d}, {dscale, D},
                       {dw_pre, D}, {workspace, (wide)need, 1}},
                      {{y, e, B, H, T, d, a.ys}, {z, e, B, 1, T, W, a.zs}, {w_post, d}, {residual, se, B, 1, T, W, a.rs},
                       {scale, D}, {w_pre, D}, {rstd_post, rows * H}, {rstd_pre, rows}, {d_out, se, B, 1, T, W, a.dos},
                       {d_normed, e, B, 1, T, W, a.dns}}))
    return set_error(GLA_ERR_INVALID_ARG, "%s: outputs and the workspace must not overlap inputs or each other", fn);
  a.y = y;
  a.z = z;
  a.residual = residual;
  a.w_post = w_post;
  a.scale = scale;
  a.w_pre = w_pre;
  a.rstd_post = const_cast<float*>(rstd_post);
  a.rstd_pre = const_cast<float*>(rstd_pre);
  a.d_out = d_out;
  a.d_normed = d_normed;
  a.dy = dy;
  a.dz = dz;
  a.d_residual = d_residual;
  a.dw_post = dw_post;
  a.dscale = dscale;
  a.dw_pre = dw_pre;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.B = B;
  a.H = H;
  a.T = T;
  a.d = d;
  a.act = act;
  a.dtype = dtype;
  a.stream_dtype = stream_dtype;
  return launched(fn, gla::launch_join_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
