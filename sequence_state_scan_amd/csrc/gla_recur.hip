// The elementwise gated linear recurrence, per sequence b and channel c:
//   h_t = a_t h_{t-1} + beta(g_t) x_t,  a = exp(g),  beta = 1 | 1 - a | sqrt(1 - a^2)
// and its backward, in one pass over the data each (2e + 4 and 3e + 8 bytes per element at e
// bytes of dtype), bound by HBM: 256k x 1024 bf16 forward in 382 us in calls one after the other (5.6
// TB/s; the memory-side cache still holds part of the inputs), the kernel alone 407 us under a trace;
// 4 x 4096 x 2048 backward alone 105 us, 4.5 TB/s.
//
// A tile is NW waves of TW tokens each by 64 channels; a lane holds its wave's TW tokens of a
// channel in registers.  The recurrence over a run of tokens is the map h -> A h + B with A the
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
// runs already and itself waits only for tiles before it.
#include "gla_block.hpp"

namespace gla {

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

// The state entering tile `at` (its channel's words, `stride` apart, from w): `state0`
// enters tile 0, tiles 0 .. at - 1 have published or will.  It needs one known state among the
// LOOK tiles before; where there is none yet it waits for the oldest of them, which comes first:
// a state that becomes known so serves LOOK tiles at once.
// Every wait ends: after kMaxPolls (seconds, where a wait takes microseconds) it gives up with NaN,
// as happens where two calls that run at once are handed one workspace against the rules.
constexpr int kMaxPolls = 1 << 20;

template <int LOOK>
__device__ __forceinline__ float look_back(const word* w, long stride, int at, float state0) {
  word win[LOOK];
#pragma unroll
  for (int i = 0; i < LOOK; ++i) win[i] = at - 1 - i >= 0 ? peek(w + (at - 1 - i) * stride) : pack(-1.f, state0);
  int polls = 0;
  for (;;) {
    bool known = false;
#pragma unroll
    for (int i = 0; i < LOOK; ++i) known |= word_a(win[i]) < 0.f;
    if (__all(known) || ++polls > kMaxPolls) break;
    __builtin_amdgcn_s_sleep(1);
    if (at >= LOOK) win[LOOK - 1] = peek(w + (at - LOOK) * stride);
  }
  float state = __builtin_nanf("");  // replaced by the first known one
#pragma unroll
  for (int i = LOOK - 1; i >= 0; --i) {
    while (win[i] == kEmpty && ++polls <= kMaxPolls) {
      __builtin_amdgcn_s_sleep(1);
      win[i] = peek(w + (at - 1 - i) * stride);
    }
    if (win[i] == kEmpty) win[i] = pack(-1.f, __builtin_nanf(""));
    const float A = word_a(win[i]), B = word_b(win[i]);
    state = A < 0.f ? B : advance(A, state, B);
  }
  return state;
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

// A channel's element of token i of a run that starts at `row`, the same in every lane: its address
// is two scalar registers and one 32-bit offset a lane (kMaxStride keeps the offset inside), so
// that a run's loads in flight hold few registers.
template <typename E>
__device__ __forceinline__ E& element(E* row, unsigned stride, unsigned i, unsigned c) {
  return *reinterpret_cast<E*>(reinterpret_cast<char*>(row) + (i * stride + c) * (unsigned)sizeof(E));
}

// A channel's TW tokens; those past the `left` live ones repeat the last (their addresses stay inside).
// Read once, past the caches (4 x 4096 x 2048 bf16 forward 60.9 us, 63.5 through them; backward 105.7, 107.5).
template <typename E, int TW>
__device__ __forceinline__ void load_run(const E* row, long stride, int left, unsigned c, E (&r)[TW]) {
  E* p = const_cast<E*>(row);
  if (left >= TW) {
#pragma unroll
    for (int i = 0; i < TW; ++i) r[i] = __builtin_nontemporal_load(&element(p, (unsigned)stride, i, c));
  } else {
#pragma unroll
    for (int i = 0; i < TW; ++i) r[i] = element(p, (unsigned)stride, i < left ? i : left - 1, c);
  }
}

template <typename E, int MODE, int NW, int TW, int LOOK>
__global__ __launch_bounds__(64 * NW) void recur_fwd_kernel(RecurArgs a) {
  constexpr int TILE = TW * NW;
  __shared__ float runA[NW][64], runB[NW][64], enter[64];
  __shared__ unsigned num;
  const int ncb = (a.D + 63) / 64, nch = (a.T + kRecurChunk - 1) / kRecurChunk;
  const unsigned tile = tile_number(a.ticket, &num);
  const int cb = tile % ncb, b = tile / ncb % a.B, n = tile / ncb / a.B;  // channel block, sequence, tile of it
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = cb * 64 + lane, len = seq_len(a, b);
  const int t0 = n * TILE + wave * TW, left = len - t0;
  const bool live = c < a.D;
  const unsigned cl = live ? c : 0;  // lanes past the last channel load the first, and store nothing
  E* h = (E*)a.h + ((long)b * a.T + t0) * a.D;
  float* chunk_in = a.chunk_in && t0 % kRecurChunk == 0 && t0 < a.T
                        ? a.chunk_in + ((long)b * nch + t0 / kRecurChunk) * a.D : nullptr;
  if (n * TILE >= len && n > 0) {  // behind the sequence's end: no tile waits for this one
    if (live) {
      for (int i = 0; i < TW && t0 + i < a.T; ++i) element(h, a.D, i, cl) = (E)0.f;
      if (chunk_in) chunk_in[cl] = 0.f;
    }
    return;
  }
  float at[TW], bt[TW];
  if (left > 0) {
    E xr[TW];
    float gr[TW];
    load_run<float, TW>(a.g + b * a.gs.b + t0 * a.gs.t, a.gs.t, left, cl, gr);
    load_run<E, TW>((const E*)a.x + b * a.xs.b + t0 * a.xs.t, a.xs.t, left, cl, xr);
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      at[i] = decay(gr[i]);
      bt[i] = input_factor<MODE>(gr[i], at[i]) * (float)xr[i];
    }
  }
  if (left < TW) {  // tokens behind the end change nothing
#pragma unroll
    for (int i = 0; i < TW; ++i)
      if (i >= left) {
        at[i] = 1.f;
        bt[i] = 0.f;
      }
  }
  float A = 1.f, B = 0.f;
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    A *= at[i];
    B = advance(at[i], B, bt[i]);
  }
  runA[wave][lane] = A;
  runB[wave][lane] = B;
  __syncthreads();
  if (wave == 0 && live) {
    const long stride = (long)a.B * a.D, col = (long)b * a.D + c;
    float in = a.h0 ? a.h0[col] : 0.f;
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const float wa = runA[w][lane];
      A *= wa;
      B = advance(wa, B, runB[w][lane]);
    }
    // a later tile of the sequence reads this one's word
    const bool wanted = LOOK > 0 && a.words && (n + 1) * TILE < len;
    if constexpr (LOOK > 0) {
      if (a.words && n > 0) {
        if (wanted) publish(a.words + n * stride + col, pack(A, B));
        in = look_back<LOOK>(a.words + col, stride, n, in);
      }
    }
    const float out = advance(A, in, B);
    if (wanted) publish(a.words + n * stride + col, pack(-1.f, out));
    enter[lane] = in;
    if (a.h_final && (n + 1) * TILE >= len) a.h_final[col] = out;
  }
  __syncthreads();
  if (!live) return;
  float s = enter[lane];
  for (int w = 0; w < wave; ++w) s = advance(runA[w][lane], s, runB[w][lane]);
  if (chunk_in) chunk_in[cl] = left > 0 || t0 == 0 ? s : 0.f;
  if (left >= TW) {
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      s = advance(at[i], s, bt[i]);
      element(h, a.D, i, cl) = (E)s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      s = advance(at[i], s, bt[i]);
      if (t0 + i < a.T) element(h, a.D, i, cl) = (E)(i < left ? s : 0.f);
    }
  }
}

// The backward: G_t the gradient of the state after token t, u_t = a_t G_t what of it reaches the
// state before (u = A u + B over a run from its end, with the same A as the forward's), and
// h_{t-1} rebuilt from the chunk's incoming state.  Tiles go from the end.  The inputs stay as they
// were loaded, and a and beta are formed again in each of the three walks: held, they would take
// the registers of a second workgroup on the CU.
template <typename E, int MODE, int NW, int TW, int LOOK>
__global__ __launch_bounds__(64 * NW) void recur_bwd_kernel(RecurArgs a) {
  constexpr int TILE = TW * NW;
  __shared__ float runA[NW][64], runH[NW][64], runU[NW][64], enter[64];
  __shared__ unsigned num;
  const int ncb = (a.D + 63) / 64, nch = (a.T + kRecurChunk - 1) / kRecurChunk, tiles = (a.T + TILE - 1) / TILE;
  const unsigned tile = tile_number(a.ticket, &num);
  const int cb = tile % ncb, b = tile / ncb % a.B, n = tiles - 1 - (int)(tile / ncb / a.B);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = cb * 64 + lane, len = seq_len(a, b);
  const int t0 = n * TILE + wave * TW, left = len - t0;
  const bool live = c < a.D;
  const unsigned cl = live ? c : 0;
  E* dx = (E*)a.h + ((long)b * a.T + t0) * a.D;
  float* dg = a.dg + ((long)b * a.T + t0) * a.D;
  if (n < 0) return;  // a ticket of another call's (a workspace shared against the rules)
  if (n * TILE >= len && n > 0) {
    if (live)
      for (int i = 0; i < TW && t0 + i < a.T; ++i) {
        element(dx, a.D, i, cl) = (E)0.f;
        element(dg, a.D, i, cl) = 0.f;
      }
    return;
  }
  E xr[TW], dr[TW];
  float gr[TW], s = 0.f;
  const int chunk = t0 / kRecurChunk, lead = (chunk * kRecurChunk - n * TILE) / TW;  // its first wave
  if (left > 0) {
    load_run<float, TW>(a.g + b * a.gs.b + t0 * a.gs.t, a.gs.t, left, cl, gr);
    load_run<E, TW>((const E*)a.x + b * a.xs.b + t0 * a.xs.t, a.xs.t, left, cl, xr);
    load_run<E, TW>((const E*)a.dh + b * a.dhs.b + t0 * a.dhs.t, a.dhs.t, left, cl, dr);
    s = a.chunk_in[((long)b * nch + chunk) * a.D + cl];
  }
  if (left < TW) {
    // tokens behind the end hold zeros: a = exp(0) = 1 and no terms, the map that changes nothing
    // (beta = 1 in the plain mode, of x = 0)
#pragma unroll
    for (int i = 0; i < TW; ++i)
      if (i >= left) {
        xr[i] = dr[i] = (E)0.f;
        gr[i] = 0.f;
      }
  }
  float A = 1.f, H = 0.f, U = 0.f, before[TW];
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    const float at = decay(gr[i]);
    A *= at;
    H = advance(at, H, input_factor<MODE>(gr[i], at) * (float)xr[i]);
  }
#pragma unroll
  for (int i = TW - 1; i >= 0; --i) U = pass(decay(gr[i]), (float)dr[i] + U);
  runA[wave][lane] = A;
  runH[wave][lane] = H;
  runU[wave][lane] = U;
  __syncthreads();
  if (wave == 0 && live) {
    const long stride = (long)a.B * a.D, col = (long)b * a.D + c;
    float in = a.dhT ? a.dhT[col] : 0.f;
    A = runA[NW - 1][lane];
    U = runU[NW - 1][lane];
#pragma unroll
    for (int w = NW - 2; w >= 0; --w) {
      const float wa = runA[w][lane];
      A *= wa;
      U = advance(wa, U, runU[w][lane]);
    }
    const int end = len > 0 ? (len - 1) / TILE : 0;  // the sequence's last tile; words count from it
    if constexpr (LOOK > 0) {
      if (a.words && n < end) {
        if (n > 0) publish(a.words + (end - n) * stride + col, pack(A, U));
        in = look_back<LOOK>(a.words + col, stride, end - n, in);
      }
    }
    const float out = advance(A, in, U);
    if (LOOK > 0 && a.words && n > 0) publish(a.words + (end - n) * stride + col, pack(-1.f, out));
    enter[lane] = in;
    if (a.h_final && n == 0) a.h_final[col] = out;
  }
  for (int w = lead; w < wave; ++w) s = advance(runA[w][lane], s, runH[w][lane]);
#pragma unroll
  for (int i = 0; i < TW; ++i) {
    const float at = decay(gr[i]);
    before[i] = s;
    s = advance(at, s, input_factor<MODE>(gr[i], at) * (float)xr[i]);
  }
  __syncthreads();
  if (!live) return;
  float u = enter[lane];
  for (int w = NW - 1; w > wave; --w) u = advance(runA[w][lane], u, runU[w][lane]);
  const bool full = left >= TW;
#pragma unroll
  for (int i = TW - 1; i >= 0; --i) {
    const float at = decay(gr[i]), be = input_factor<MODE>(gr[i], at), G = (float)dr[i] + u;
    u = pass(at, G);
    const float vx = be * G;
    float vg = at == 0.f ? 0.f : u * before[i];
    // a constant factor has no term, not zero times an x or G that may be infinite
    if constexpr (MODE != GLA_RECUR_PLAIN) vg = fmaf(input_factor_slope<MODE>(at, be) * (float)xr[i], G, vg);
    if (full || t0 + i < a.T) {
      element(dx, a.D, i, cl) = (E)(full || i < left ? vx : 0.f);
      element(dg, a.D, i, cl) = full || i < left ? vg : 0.f;
    }
  }
}

// All ones: the words empty, the ticket counter one below zero.
__global__ __launch_bounds__(256) void recur_clear_kernel(word* p, long n) {
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) p[i] = kEmpty;
}

constexpr size_t kTicketWords = 32;  // the counter's own 256 bytes

size_t recur_workspace_words(int B, int T, int D) {
  const size_t tiles = ((size_t)T + kRecurTile - 1) / kRecurTile;
  return tiles > 1 ? kTicketWords + tiles * B * D : 0;
}

template <bool BWD, typename E, int MODE, int NW, int TW, int LOOK>
static void recur_run(RecurArgs a, hipStream_t s) {
  const unsigned ncb = (a.D + 63) / 64, tiles = (a.T + NW * TW - 1) / (NW * TW);
  if (tiles > 1) {
    static_assert(LOOK == 0 || NW * TW == kRecurTile, "the workspace is laid out for tiles of that many tokens");
    word* ws = a.words;
    const long n = (long)recur_workspace_words(a.B, a.T, a.D), blocks = (n + 255) / 256;
    recur_clear_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(ws, n);
    a.ticket = (unsigned*)ws;
    a.words = ws + kTicketWords;
  } else {
    a.words = nullptr;
  }
  const unsigned grid = ncb * a.B * tiles;
  if constexpr (BWD) recur_bwd_kernel<E, MODE, NW, TW, LOOK><<<grid, 64 * NW, 0, s>>>(a);
  else recur_fwd_kernel<E, MODE, NW, TW, LOOK><<<grid, 64 * NW, 0, s>>>(a);
}

// The tile and the look back by size.  Up to 128 tokens one tile does, of as many waves as have
// tokens, with no look back.  Beyond, a tile is 256 tokens: forward 8 waves of 32, whose 64 loads a lane are in flight
// at once (4 x 4096 x 2048 bf16 64 us; 128-token tiles of 64 channels 112, of 128 channels 82).
// With few columns of 64 channels (cols) the tiles of one column wait for each other in a chain of
// T / (256 LOOK) hops of about 1.5 us each, and a longer look pays; with many the words' reads do
// not: 65536 x 256 bf16 44 us with 16 waves of 16 and 16 tiles back, 83 with 8 of 32 and 4; 131072
// x 64 45 with 32 back, 56 with 16; 65536 x 1024 112 with 8 back, 118 with 16 waves and 16, 165 with
// 32.  At the borders, 65536 tokens: 8 columns 73 us with 8 waves and 8 back, 79 with 16 and 16; 7 columns
// 71 and 69; 3 columns 41 with 16 back and 42 with 32; 2 columns 39 and 35.  (Of shorter sequences the
// border would lie higher: 8 x 16384 x 64 takes 37 us with 8 back, 28 with 16.)  Backward 16 waves of 16
// everywhere, which leaves a lane's three inputs in its registers: 4 x 4096 x 2048 105 us, 65536 x 256 58
// (8 waves of 8 pairs of channels: 119 and 171); with 8 back and 16, 65536 tokens: 6 columns 83 and 88, 4
// columns 64 and 64, 3 columns 56 and 53, 2 columns 56 and 46.
template <bool BWD, typename E, int MODE>
static void recur_shape(const RecurArgs& a, hipStream_t s) {
  const long long cols = (long long)a.B * ((a.D + 63) / 64);
  if (a.T <= 16) {
    recur_run<BWD, E, MODE, 1, 16, 0>(a, s);
  } else if (a.T <= 64) {
    recur_run<BWD, E, MODE, 4, 16, 0>(a, s);
  } else if (a.T <= 128) {
    recur_run<BWD, E, MODE, 8, 16, 0>(a, s);
  } else if constexpr (!BWD) {
    if (cols >= 8) recur_run<BWD, E, MODE, 8, 32, 8>(a, s);
    else if (cols >= 3) recur_run<BWD, E, MODE, 16, 16, 16>(a, s);
    else recur_run<BWD, E, MODE, 16, 16, 32>(a, s);
  } else {
    if (cols >= 3) recur_run<BWD, E, MODE, 16, 16, 8>(a, s);
    else recur_run<BWD, E, MODE, 16, 16, 16>(a, s);
  }
}

template <bool BWD, typename E>
static hipError_t recur_mode(const RecurArgs& a, hipStream_t s) {
  if (a.mode == GLA_RECUR_PLAIN) recur_shape<BWD, E, GLA_RECUR_PLAIN>(a, s);
  else if (a.mode == GLA_RECUR_LERP) recur_shape<BWD, E, GLA_RECUR_LERP>(a, s);
  else recur_shape<BWD, E, GLA_RECUR_NORM>(a, s);
  return hipGetLastError();
}

hipError_t launch_recur_fwd(const RecurArgs& a, hipStream_t s) {
  return a.dtype == GLA_BF16 ? recur_mode<false, bf16>(a, s) : recur_mode<false, float>(a, s);
}
hipError_t launch_recur_bwd(const RecurArgs& a, hipStream_t s) {
  return a.dtype == GLA_BF16 ? recur_mode<true, bf16>(a, s) : recur_mode<true, float>(a, s);
}

// One token for each row of a batch, the rows' states in a pool.  A wave has 64 V channels of one
// row; it looks the row's slot up and checks it against the earlier rows' by itself, while its
// loads are on their way.
template <typename E, int MODE, int V>
__global__ __launch_bounds__(64) void recur_step_kernel(RecurStepArgs a) {
  const int c = (blockIdx.x * 64 + threadIdx.x) * V, b = blockIdx.y;
  const bool live = c < a.D;
  float x[V] = {}, g[V] = {}, st[V] = {};
  const int slot = row_slot(a.slots, b, a.n_slots);
  float* state = a.state + (long)slot * a.D + c;
  if (live) {
    load_row<float, V>(a.g + b * a.gs.b + c, g);
    load_row<E, V>((const E*)a.x + b * a.xs.b + c, x);
    if (slot >= 0) load_row<float, V>(state, st);
  }
  const bool good = slot >= 0 && !slot_taken(a.slots, b, slot);
  if (!live) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const float at = decay(g[v]);
    st[v] = advance(at, st[v], input_factor<MODE>(g[v], at) * x[v]);
    if (!good) st[v] = slot == -1 ? 0.f : __builtin_nanf("");
  }
  if (good) store_row<float, V>(state, st);
  store_row<E, V>((E*)a.h + (long)b * a.D + c, st);
}

template <typename E, int MODE>
static void recur_step_run(const RecurStepArgs& a, hipStream_t s) {
  const int e = sizeof(E);
  // four channels a lane where the rows allow it: 256 x 4096 bf16 in 4.8 us, 7.6 with one
  const bool four = a.D % 4 == 0 && a.xs.b % 4 == 0 && a.gs.b % 4 == 0 && (uintptr_t)a.x % (4 * e) == 0 &&
                    (uintptr_t)a.h % (4 * e) == 0 && (uintptr_t)a.g % 16 == 0 && (uintptr_t)a.state % 16 == 0;
  if (four) recur_step_kernel<E, MODE, 4><<<dim3((a.D + 255) / 256, a.B), 64, 0, s>>>(a);
  else recur_step_kernel<E, MODE, 1><<<dim3((a.D + 63) / 64, a.B), 64, 0, s>>>(a);
}

template <typename E>
static void recur_step_mode(const RecurStepArgs& a, hipStream_t s) {
  if (a.mode == GLA_RECUR_PLAIN) recur_step_run<E, GLA_RECUR_PLAIN>(a, s);
  else if (a.mode == GLA_RECUR_LERP) recur_step_run<E, GLA_RECUR_LERP>(a, s);
  else recur_step_run<E, GLA_RECUR_NORM>(a, s);
}

hipError_t launch_recur_step(const RecurStepArgs& a, hipStream_t s) {
  if (a.dtype == GLA_BF16) recur_step_mode<bf16>(a, s);
  else recur_step_mode<float>(a, s);
  return hipGetLastError();
}

}  // namespace gla
