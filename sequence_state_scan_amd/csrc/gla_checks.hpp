// Argument checks that the recurrent-block calls' host sides share (gla_block_api.cpp, gla_delta_api.cpp).
#pragma once
#include "gla_block.hpp"
#include "gla_kernels.hpp"

namespace {

using gla::set_error;
using gla::Strides;

constexpr long long kMaxGrid = (1LL << 22) - 1;  // workgroups of a launch: fewer than 2^32 lanes at up to 1024 each

gla_status launched(const char* fn, hipError_t e) {
  if (e != hipSuccess) return set_error(GLA_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return set_error(GLA_OK, "");
}

gla_status check_dtype(const char* fn, int dtype) {
  if (dtype != GLA_F32 && dtype != GLA_BF16) return set_error(GLA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  return GLA_OK;
}

// The strides of a [b][h][t][last] tensor: the caller's, or the contiguous ones b, h and t, which are 0 for
// a dimension that the tensor does not have.  False if negative.
bool strides(const gla_strides* st, long long b, long long h, long long t, Strides* out) {
  *out = st ? Strides{st->b, h ? st->h : 0, t ? st->t : 0} : Strides{b, h, t};
  return out->b >= 0 && out->h >= 0 && out->t >= 0;
}

typedef __int128 wide;  // bytes: a caller's strides may reach past 64 bits

// The memory of a tensor: up to three strided dimensions over runs of `run` bytes.  No memory where it is null.
struct Region {
  wide base = 0, run = 0;
  int dims = 0;
  wide n[3], step[3];

  // count contiguous elements of e bytes
  Region(const void* p, wide count, int e) : base((unsigned long long)p), run(p ? count * e : 0) {}
  Region(const float* p, wide count) : Region(p, count, 4) {}
  // a [b][h][t] view of rows of `last` elements
  Region(const void* p, int e, int b, int h, int t, int last, const Strides& st) : Region(p, last, e) {
    const long long count[3] = {b, h, t}, by[3] = {st.b, st.h, st.t};
    for (int i = 0; i < 3; ++i) {
      if (count[i] == 1 || by[i] == 0) continue;  // one place
      int at = dims++;
      for (; at > 0 && step[at - 1] < (wide)by[i] * e; --at) {  // the largest step first
        n[at] = n[at - 1];
        step[at] = step[at - 1];
      }
      n[at] = count[i];
      step[at] = (wide)by[i] * e;
    }
  }

  wide extent(int from) const {
    wide s = run;
    for (int i = from; i < dims; ++i) s += (n[i] - 1) * step[i];
    return s;
  }
  // Whether the part from dimension `at` on, placed at p, has a byte in [lo, hi).  What lies in a view's
  // gaps does not count, unless its steps are shorter than what they step over.
  bool meets(wide p, int at, wide lo, wide hi) const {
    const wide e = extent(at + 1);
    if (at == dims) return p < hi && p + run > lo;
    wide first = p + e > lo ? 0 : (lo - e - p) / step[at] + 1, last = p >= hi ? -1 : (hi - 1 - p) / step[at];
    if (last > n[at] - 1) last = n[at] - 1;
    if (first > last) return false;
    if (step[at] < e || last - first >= 2) return true;  // of three in a row the second lies inside
    return meets(p + first * step[at], at + 1, lo, hi) || (last > first && meets(p + last * step[at], at + 1, lo, hi));
  }
};

// Whether an output (all contiguous) shares memory with an input or another output.
template <int N, int M>
bool overlaps(const Region (&outs)[N], const Region (&ins)[M]) {
  wide ends[M];
  for (int i = 0; i < M; ++i) ends[i] = ins[i].run ? ins[i].base + ins[i].extent(0) : 0;
  for (int o = 0; o < N; ++o) {
    const wide lo = outs[o].base, hi = lo + outs[o].run;
    if (lo == hi) continue;
    for (int i = 0; i < M; ++i)
      if (ins[i].base < hi && ends[i] > lo && ins[i].meets(ins[i].base, 0, lo, hi)) return true;
    for (int q = 0; q < o; ++q)
      if (outs[q].run && outs[q].base < hi && outs[q].base + outs[q].run > lo) return true;
  }
  return false;
}

int size_of(int dtype) { return dtype == GLA_BF16 ? 2 : 4; }

#define GLA_TRY(e)                     \
  do {                                 \
    const gla_status st_ = (e);        \
    if (st_ != GLA_OK) return st_;     \
  } while (0)

}  // namespace
