// The layer norm's arguments and launcher (gla_layernorm.hip, gla_delta_api.cpp).
#pragma once
#include "gla_block.hpp"

namespace gla {

constexpr int kNormMaxRow = 16384;

struct NormArgs {
  const void *x, *residual;
  const float *w, *b;
  void *out, *normed;
  float *mean, *rstd;  // [B][T]
  // backward
  const void *d_out, *d_normed;
  void *dx, *d_residual;
  float *dw, *db, *partial;
  Strides xs, rs, dos, dns;
  int B, T, D, dtype, stream_dtype;
  float eps;
};

hipError_t launch_layernorm(const NormArgs& a, bool bwd, hipStream_t s);
size_t norm_partial_floats(int B, int T, int D);  // workspace of the backward

}  // namespace gla
