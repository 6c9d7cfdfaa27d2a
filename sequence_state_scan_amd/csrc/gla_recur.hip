// The elementwise gated linear recurrence, per sequence b and channel c:
//   h_t = a_t h_{t-1} + beta(g_t) x_t,  a = exp(g),  beta = 1 | 1 - a | sqrt(1 - a^2)
// and its backward, in one pass over the data each (2e + 4 and 3e + 8 bytes per element at e
// bytes of dtype), bound by HBM.
//
// A tile is NW waves of kTw tokens each by 64 V channels; a lane holds its wave's kTw tokens of V
// channels in registers.  The recurrence over a run of tokens is the map h -> A h + B with A the
// product of the a's and B the run's end state from zero.  A lane forms its run's (A, B), the
// waves' pairs meet in LDS, and a tile's pair goes to the workspace, where the later tiles of the
// sequence read it: a tile looks back over its predecessors' words to the nearest whose state is
// already known, and applies the pairs between in order.  It then knows the state entering it,
// writes its own end state over its pair for the tiles behind it, and walks its tokens once more
// in registers.
//
// One 8-byte word per tile and channel: all ones (nothing yet), (A, B) with A >= 0, or (-1, state).
// It is written and read whole, by relaxed atomics at device scope, so no fence orders anything.
// Which of the two a reader finds depends on the timing, the result does not: a state is the map
// applied to the state before, whoever applies it.  Tiles are numbered by a ticket in the order
// they start, and every tile publishes its pair before it waits, so each wait is for a tile that
// runs already and waits for nothing before that.
#include "gla_block.hpp"

namespace gla {

constexpr int kTw = 16;           // tokens of a wave's run
constexpr int kLook = 4;          // predecessors' words a look-back step loads at once
static_assert(kRecurChunk == 8 * kTw, "a full tile of 8 waves is a chunk");

typedef unsigned long long word;
constexpr word kEmpty = ~0ull;

__device__ __forceinline__ word pack(float a, float b) {
  // a NaN is written as the quiet one, never as the all-ones of an empty word
  const unsigned lo = a != a ? 0x7FC00000u : __float_as_uint(a), hi = __float_as_uint(b);
  return (word)hi << 32 | lo;
}
__device__ __forceinline__ float word_a(word w) { return __uint_as_float((unsigned)w); }
__device__ __forceinline__ float word_b(word w) { return __uint_as_float((unsigned)(w >> 32)); }
__device__ __forceinline__ word peek(const word* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(word* p, word w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ int seq_len(const RecurArgs& a, int b) {
  if (!a.lens) return a.T;
  const int n = a.lens[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// The state entering tile `at` (words [tile][stride] at w, for V adjacent channels): `state0`
// enters tile 0, tiles 0 .. at - 1 have published or will.  It needs one known state among the
// kLook tiles before; where there is none yet it waits for the oldest of them, which comes first:
// a state that becomes known so serves kLook tiles at once.
template <int V>
__device__ __forceinline__ void look_back(const word* w, long stride, int at, const float (&state0)[V], float (&state)[V]) {
  word win[kLook][V];
#pragma unroll
  for (int i = 0; i < kLook; ++i) {
    const int p = at - 1 - i;
#pragma unroll
    for (int v = 0; v < V; ++v) win[i][v] = p >= 0 ? peek(w + p * stride + v) : pack(-1.f, state0[v]);
  }
  for (;;) {
    bool all = true;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bool known = false;
#pragma unroll
      for (int i = 0; i < kLook; ++i) known |= word_a(win[i][v]) < 0.f;
      all &= known;
    }
    if (__all(all)) break;
    __builtin_amdgcn_s_sleep(1);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (at >= kLook) win[kLook - 1][v] = peek(w + (at - kLook) * stride + v);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) state[v] = 0.f;  // replaced by the first known state
#pragma unroll
  for (int i = kLook - 1; i >= 0; --i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      word x = win[i][v];
      while (x == kEmpty) {
        __builtin_amdgcn_s_sleep(1);
        x = peek(w + (at - 1 - i) * stride + v);
      }
      const float A = word_a(x), Bv = word_b(x);
      state[v] = A < 0.f ? Bv : advance(A, state[v], Bv);
    }
}

// Number of the tile a workgroup serves: its ticket where tiles wait for each other (the counter
// starts at all ones), else its index.
__device__ __forceinline__ unsigned tile_number(unsigned* ticket, unsigned* shared) {
  if (!ticket) return blockIdx.x;
  if (threadIdx.x == 0)
    *shared = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*shared);
}

template <typename E, int MODE, int V, int NW, int TW>
__global__ __launch_bounds__(64 * NW) void recur_fwd_kernel(RecurArgs a) {
  constexpr int NC = 64 * V, TILE = TW * NW;
  __shared__ float runA[NW][NC], runB[NW][NC], enter[NC];
  __shared__ unsigned num;
  const int ncb = (a.D + NC - 1) / NC;
  const unsigned tile = tile_number(a.ticket, &num);
  const int cb = tile % ncb, b = tile / ncb % a.B, n = tile / ncb / a.B;  // channel block, sequence, tile of it
  const int nch = (a.T + kRecurChunk - 1) / kRecurChunk;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = cb * NC + lane * V, len = seq_len(a, b);
  const int t0 = n * TILE + wave * TW, left = len - t0;
  const bool live = c < a.D;
  E* h = (E*)a.h + ((long)b * a.T + t0) * a.D + c;
  float zero[V] = {};
  if (n * TILE >= len && n > 0) {  // behind the sequence's end: no tile waits for this one
    if (live) {
      for (int i = 0; i < TW && t0 + i < a.T; ++i) store_row<E, V>(h + (long)i * a.D, zero);
      if (a.chunk_in && t0 % kRecurChunk == 0 && t0 < a.T)
        store_row<float, V>(a.chunk_in + ((long)b * nch + t0 / kRecurChunk) * a.D + c, zero);
    }
    return;
  }
  typename Vec<E, V>::raw xr[TW];
  typename Vec<float, V>::raw gr[TW];
  const E* x = (const E*)a.x + b * a.xs.b + t0 * a.xs.t + c;
  const float* g = a.g + b * a.gs.b + t0 * a.gs.t + c;
#pragma unroll
  for (int i = 0; i < TW; ++i)
    if (live && i < left) {
      xr[i] = *(const typename Vec<E, V>::raw*)(x + i * a.xs.t);
      gr[i] = *(const typename Vec<float, V>::raw*)(g + i * a.gs.t);
    }
  float at[TW][V], bt[TW][V], A[V], Bv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.f;
    Bv[v] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < TW; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      at[i][v] = 1.f;
      bt[i][v] = 0.f;
      if (live && i < left) {
        at[i][v] = decay(gr[i][v]);
        bt[i][v] = input_factor<MODE>(gr[i][v], at[i][v]) * (float)xr[i][v];
      }
      A[v] *= at[i][v];
      Bv[v] = advance(at[i][v], Bv[v], bt[i][v]);
    }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    runA[wave][lane * V + v] = A[v];
    runB[wave][lane * V + v] = Bv[v];
  }
  __syncthreads();
  if (wave == 0) {
    float in[V], first[V];
#pragma unroll
    for (int v = 0; v < V; ++v) first[v] = a.h0 && live ? a.h0[(long)b * a.D + c + v] : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        const float wa = runA[w][lane * V + v];
        A[v] *= wa;
        Bv[v] = advance(wa, Bv[v], runB[w][lane * V + v]);
      }
    if (live) {
      const long stride = (long)a.B * a.D, col = (long)b * a.D + c;
      if (a.words && n > 0) {
        if ((n + 1) * TILE < len)
#pragma unroll
          for (int v = 0; v < V; ++v) publish(a.words + n * stride + col + v, pack(A[v], Bv[v]));
        look_back<V>(a.words + col, stride, n, first, in);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) in[v] = first[v];
      }
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        out[v] = advance(A[v], in[v], Bv[v]);
        if (a.words && (n + 1) * TILE < len) publish(a.words + n * stride + col + v, pack(-1.f, out[v]));
        enter[lane * V + v] = in[v];
      }
      if (a.h_final && (n + 1) * TILE >= len) store_row<float, V>(a.h_final + col, out);
    }
  }
  __syncthreads();
  if (!live) return;
  float s[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = enter[lane * V + v];
    for (int w = 0; w < wave; ++w) s[v] = advance(runA[w][lane * V + v], s[v], runB[w][lane * V + v]);
  }
  if (a.chunk_in && t0 % kRecurChunk == 0 && t0 < a.T)
    store_row<float, V>(a.chunk_in + ((long)b * nch + t0 / kRecurChunk) * a.D + c, left > 0 || t0 == 0 ? s : zero);
#pragma unroll
  for (int i = 0; i < TW; ++i) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = advance(at[i][v], s[v], bt[i][v]);
    if (t0 + i < a.T) store_row<E, V>(h + (long)i * a.D, i < left ? s : zero);
  }
}

// The backward: G_t the gradient of the state after token t, u_t = a_t G_t what of it reaches the
// state before (u = A u + B over a run from its end, with the same A as the forward's), and
// h_{t-1} rebuilt from the chunk's incoming state.  Tiles go from the end.
template <typename E, int MODE, int V, int NW, int TW>
__global__ __launch_bounds__(64 * NW) void recur_bwd_kernel(RecurArgs a) {
  constexpr int NC = 64 * V, TILE = TW * NW;
  __shared__ float runA[NW][NC], runH[NW][NC], runU[NW][NC], enter[NC];
  __shared__ unsigned num;
  const int ncb = (a.D + NC - 1) / NC;
  const unsigned tile = tile_number(a.ticket, &num);
  const int nch = (a.T + kRecurChunk - 1) / kRecurChunk, tiles = (a.T + TILE - 1) / TILE;
  const int cb = tile % ncb, b = tile / ncb % a.B, n = tiles - 1 - (int)(tile / ncb / a.B);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = cb * NC + lane * V, len = seq_len(a, b);
  const int t0 = n * TILE + wave * TW, left = len - t0;
  const bool live = c < a.D;
  E* dx = (E*)a.h + ((long)b * a.T + t0) * a.D + c;
  float* dg = a.dg + ((long)b * a.T + t0) * a.D + c;
  float zero[V] = {};
  if (n * TILE >= len && n > 0) {
    if (live)
      for (int i = 0; i < TW && t0 + i < a.T; ++i) {
        store_row<E, V>(dx + (long)i * a.D, zero);
        store_row<float, V>(dg + (long)i * a.D, zero);
      }
    return;
  }
  typename Vec<E, V>::raw xr[TW], dr[TW];
  typename Vec<float, V>::raw gr[TW];
  const E* x = (const E*)a.x + b * a.xs.b + t0 * a.xs.t + c;
  const E* dh = (const E*)a.dh + b * a.dhs.b + t0 * a.dhs.t + c;
  const float* g = a.g + b * a.gs.b + t0 * a.gs.t + c;
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    xr[i] = dr[i] = typename Vec<E, V>::raw{};
    gr[i] = typename Vec<float, V>::raw{};
    if (live && i < left) {
      xr[i] = *(const typename Vec<E, V>::raw*)(x + i * a.xs.t);
      gr[i] = *(const typename Vec<float, V>::raw*)(g + i * a.gs.t);
      dr[i] = *(const typename Vec<E, V>::raw*)(dh + i * a.dhs.t);
    }
  }
  // tokens behind the end hold zeros: a = exp(0) = 1 and no terms, the map that changes nothing
  // (beta = 1 in the plain mode, of x = 0)
  float A[V], Hv[V], U[V], hb[TW][V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = 1.f;
    Hv[v] = U[v] = 0.f;
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const float at = decay(gr[i][v]);
      A[v] *= at;
      Hv[v] = advance(at, Hv[v], input_factor<MODE>(gr[i][v], at) * (float)xr[i][v]);
    }
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
      const float at = decay(gr[i][v]);
      U[v] = at == 0.f ? 0.f : at * ((float)dr[i][v] + U[v]);
    }
    runA[wave][lane * V + v] = A[v];
    runH[wave][lane * V + v] = Hv[v];
    runU[wave][lane * V + v] = U[v];
  }
  __syncthreads();
  if (wave == 0 && live) {
    float in[V], last[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      last[v] = a.dhT ? a.dhT[(long)b * a.D + c + v] : 0.f;
      A[v] = runA[NW - 1][lane * V + v];
      U[v] = runU[NW - 1][lane * V + v];
#pragma unroll
      for (int w = NW - 2; w >= 0; --w) {
        const float wa = runA[w][lane * V + v];
        A[v] *= wa;
        U[v] = advance(wa, U[v], runU[w][lane * V + v]);
      }
    }
    const long stride = (long)a.B * a.D, col = (long)b * a.D + c;
    const int end = len > 0 ? (len - 1) / TILE : 0;  // the sequence's last tile; words count from it
    if (a.words && n < end) {
      if (n > 0)
#pragma unroll
        for (int v = 0; v < V; ++v) publish(a.words + (end - n) * stride + col + v, pack(A[v], U[v]));
      look_back<V>(a.words + col, stride, end - n, last, in);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) in[v] = last[v];
    }
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      out[v] = advance(A[v], in[v], U[v]);
      if (a.words && n > 0) publish(a.words + (end - n) * stride + col + v, pack(-1.f, out[v]));
      enter[lane * V + v] = in[v];
    }
    if (a.h_final && n == 0) store_row<float, V>(a.h_final + col, out);
  }
  float s[V] = {}, u[V];
  const int chunk = t0 / kRecurChunk, lead = (chunk * kRecurChunk - n * TILE) / TW;  // its first wave
  if (live && chunk < nch) load_row<float, V>(a.chunk_in + ((long)b * nch + chunk) * a.D + c, s);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    for (int w = lead; w < wave; ++w) s[v] = advance(runA[w][lane * V + v], s[v], runH[w][lane * V + v]);
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const float at = decay(gr[i][v]);
      hb[i][v] = s[v];
      s[v] = advance(at, s[v], input_factor<MODE>(gr[i][v], at) * (float)xr[i][v]);
    }
  }
  __syncthreads();
  if (!live) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    u[v] = enter[lane * V + v];
    for (int w = NW - 1; w > wave; --w) u[v] = advance(runA[w][lane * V + v], u[v], runU[w][lane * V + v]);
  }
#pragma unroll
  for (int i = TW - 1; i >= 0; --i) {
    float vx[V], vg[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float at = decay(gr[i][v]), be = input_factor<MODE>(gr[i][v], at), G = (float)dr[i][v] + u[v];
      u[v] = at == 0.f ? 0.f : at * G;
      vx[v] = be * G;
      vg[v] = fmaf(input_factor_slope<MODE>(at, be) * (float)xr[i][v], G, at == 0.f ? 0.f : u[v] * hb[i][v]);
      if (i >= left) vx[v] = vg[v] = 0.f;
    }
    if (t0 + i < a.T) {
      store_row<E, V>(dx + (long)i * a.D, vx);
      store_row<float, V>(dg + (long)i * a.D, vg);
    }
  }
}

// All ones: the words empty, the ticket counter one below zero.
__global__ __launch_bounds__(256) void recur_clear_kernel(word* p, long n) {
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) p[i] = kEmpty;
}

constexpr size_t kTicketWords = 32;  // the counter's own 256 bytes

size_t recur_workspace_words(int B, int T, int D) {
  const size_t nch = ((size_t)T + kRecurChunk - 1) / kRecurChunk;
  return nch > 1 ? kTicketWords + nch * B * D : 0;
}

static bool pairs_aligned(const void* p, const Strides& s, int bytes) {
  return (uintptr_t)p % (2 * bytes) == 0 && s.b % 2 == 0 && s.t % 2 == 0;
}

// Two channels a lane where every row allows it, one otherwise.
static bool recur_pairs(const RecurArgs& a) {
  const int e = a.dtype == GLA_BF16 ? 2 : 4;
  const Strides none{0, 0, 0};
  const void* f32s[] = {a.chunk_in, a.h_final, a.dg};
  for (const void* p : f32s)
    if (!pairs_aligned(p, none, 4)) return false;
  return a.D % 2 == 0 && pairs_aligned(a.x, a.xs, e) && pairs_aligned(a.g, a.gs, 4) && pairs_aligned(a.dh, a.dhs, e) &&
         pairs_aligned(a.h, none, e);
}

template <typename E, int MODE, int V, int NW, int TW>
static void recur_run(RecurArgs a, bool bwd, hipStream_t s) {
  const int TILE = NW * TW;
  const unsigned ncb = (a.D + 64 * V - 1) / (64 * V), tiles = (a.T + TILE - 1) / TILE;
  if (tiles > 1) {
    word* ws = (word*)a.words;
    const long n = kTicketWords + (long)tiles * a.B * a.D;
    const long blocks = (n + 1023) / 1024;
    recur_clear_kernel<<<(unsigned)(blocks < 1024 ? blocks : 1024), 256, 0, s>>>(ws, n);
    a.ticket = (unsigned*)ws;
    a.words = ws + kTicketWords;
  } else {
    a.words = nullptr;
  }
  const unsigned grid = ncb * a.B * tiles;
  if (bwd) recur_bwd_kernel<E, MODE, V, NW, TW><<<grid, 64 * NW, 0, s>>>(a);
  else recur_fwd_kernel<E, MODE, V, NW, TW><<<grid, 64 * NW, 0, s>>>(a);
}

template <typename E, int MODE>
static void recur_shape(const RecurArgs& a, bool bwd, hipStream_t s) {
  if (bwd) {
    const bool two = recur_pairs(a) && sizeof(E) == 2;
    if (a.T > 4 * kTw) {
      if (two) recur_run<E, MODE, 2, 8, 16>(a, bwd, s);
      else recur_run<E, MODE, 1, 8, 16>(a, bwd, s);
    } else if (a.T > kTw) {
      if (two) recur_run<E, MODE, 2, 4, 16>(a, bwd, s);
      else recur_run<E, MODE, 1, 4, 16>(a, bwd, s);
    } else {
      if (two) recur_run<E, MODE, 2, 1, 16>(a, bwd, s);
      else recur_run<E, MODE, 1, 1, 16>(a, bwd, s);
    }
  } else {
    if (a.T > 128) recur_run<E, MODE, 1, 8, 32>(a, bwd, s);
    else if (a.T > 64) recur_run<E, MODE, 1, 8, 16>(a, bwd, s);
    else if (a.T > 16) recur_run<E, MODE, 1, 4, 16>(a, bwd, s);
    else recur_run<E, MODE, 1, 1, 16>(a, bwd, s);
  }
}

template <typename E>
static hipError_t recur_mode(const RecurArgs& a, bool bwd, hipStream_t s) {
  if (a.mode == GLA_RECUR_PLAIN) recur_shape<E, GLA_RECUR_PLAIN>(a, bwd, s);
  else if (a.mode == GLA_RECUR_LERP) recur_shape<E, GLA_RECUR_LERP>(a, bwd, s);
  else recur_shape<E, GLA_RECUR_NORM>(a, bwd, s);
  return hipGetLastError();
}

hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s) {
  return a.dtype == GLA_BF16 ? recur_mode<bf16>(a, false, s) : recur_mode<float>(a, false, s);
}
hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s) {
  return a.dtype == GLA_BF16 ? recur_mode<bf16>(a, true, s) : recur_mode<float>(a, true, s);
}

#define GLA_RECUR_DISPATCH(KERNEL, A, GRID, BLOCK, S)                                              \
  do {                                                                                             \
    if ((A).dtype == GLA_BF16) {                                                                   \
      if ((A).mode == GLA_RECUR_PLAIN) KERNEL<bf16, GLA_RECUR_PLAIN><<<GRID, BLOCK, 0, S>>>(A);    \
      else if ((A).mode == GLA_RECUR_LERP) KERNEL<bf16, GLA_RECUR_LERP><<<GRID, BLOCK, 0, S>>>(A); \
      else KERNEL<bf16, GLA_RECUR_NORM><<<GRID, BLOCK, 0, S>>>(A);                                 \
    } else {                                                                                       \
      if ((A).mode == GLA_RECUR_PLAIN) KERNEL<float, GLA_RECUR_PLAIN><<<GRID, BLOCK, 0, S>>>(A);   \
      else if ((A).mode == GLA_RECUR_LERP) KERNEL<float, GLA_RECUR_LERP><<<GRID, BLOCK, 0, S>>>(A);\
      else KERNEL<float, GLA_RECUR_NORM><<<GRID, BLOCK, 0, S>>>(A);                                \
    }                                                                                              \
  } while (0)

// One token for each row of a batch, the rows' states in a pool.  Every workgroup (64 channels of
// one row) looks its slot up and checks it against the earlier rows' by itself.
template <typename E, int MODE>
__global__ __launch_bounds__(64) void recur_step_kernel(RecurStepArgs a) {
  const int c = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
  const int slot = row_slot(a.slots, b, a.n_slots);
  if (c >= a.D) return;
  E* h = (E*)a.h + (long)b * a.D + c;
  if (slot < 0) {
    *h = (E)(slot == -1 ? 0.f : __builtin_nanf(""));
    return;
  }
  const float g = a.g[b * a.gs.b + c], at = decay(g);
  float* st = a.state + (long)slot * a.D + c;
  const float s = advance(at, *st, input_factor<MODE>(g, at) * (float)((const E*)a.x)[b * a.xs.b + c]);
  *st = s;
  *h = (E)s;
}

hipError_t launch_recur_step(const RecurStepArgs& a, hipStream_t s) {
  GLA_RECUR_DISPATCH(recur_step_kernel, a, dim3((a.D + 63) / 64, a.B), dim3(64), s);
  return hipGetLastError();
}

}  // namespace gla
