// Gated linear recurrence, the input-gated companion of CEMA:
//   a_t = exp(log_a_t)  (0 where a document starts),
//   h_t = a_t h_{t-1} + x_t,  y_t = h_t                    (per feature)
// and its gradients
//   dh_t = dy_t + a_{t+1} dh_{t+1},  dx_t = dh_t,
//   dlog_a_t = dh_t a_t h_{t-1},     dstate_in = a_0 dh_0.
// A span of tokens maps the state entering it affinely, h_out = A h_in + h,
// with A the product of its decays and h its scan from zero; spans compose.
// Everything is held in fp32 whatever the tensors' type.
//
// The work is bound by HBM (3 values per element forward, 5 backward), so a
// tile of one chunk (128 tokens) by 128 bytes of features is read once, by TMA,
// into shared memory and scanned there: warp w takes tokens 32 w .. 32 w + 31,
// a lane the features of 4 bytes.  First every warp finds the map of its span,
// then the state entering the chunk is fetched, then every warp scans again
// from its own entering state.  Chunks hand the state on in one launch: blocks
// draw tiles in chunk order from a counter, so every tile that a block waits
// for is held by a block that already runs.  A chunk publishes its map as soon
// as it has it; the state entering chunk c is folded, in chunk order, from the
// state entering its group of 16 chunks and the maps of the chunks between, so
// the chain of dependent hand-offs is 16 times shorter than the chain of
// chunks, and the association, and with it every bit of the result, does not
// depend on timing.  What is published is its own flag: the memory starts as
// all ones, a pattern that no result has.
#include "chain.cuh"
#include "common.cuh"
#include "gecko_internal.h"

namespace gecko {
namespace {

constexpr int kWarps = 4, kSpan = kScanChunk / kWarps;   // tokens per warp: 32, one reset bit each in a word
constexpr int kThreads = 32 * kWarps;
constexpr int kGroup = 16;                               // chunks per group of the hand-off
constexpr int kRowBytes = 128;                           // features per tile, in bytes
constexpr int kTileBytes = kScanChunk * kRowBytes;
static_assert(kSpan == 32, "a span's document starts are one 32-bit word");

// Features per lane and per tile.
template <typename T> constexpr int kV = 4 / (int)sizeof(T);
template <typename T> constexpr int kFT = 32 * kV<T>;

// The features of one lane: one fp32 value, or two, bf16 in memory and a packed
// pair in arithmetic.
template <typename T> struct Lane;
template <> struct Lane<float> {
  using Raw = float;
  using Val = float;
  static __device__ __forceinline__ Val open(Raw r) { return r; }
  static __device__ __forceinline__ Raw shut(Val v) { return v; }
  static __device__ __forceinline__ Val all(float v) { return v; }
  static __device__ __forceinline__ Val fma(Val a, Val b, Val c) { return fmaf(a, b, c); }
  static __device__ __forceinline__ Val mul(Val a, Val b) { return a * b; }
  static __device__ __forceinline__ Val add(Val a, Val b) { return a + b; }
  static __device__ __forceinline__ void get(Val v, float (&f)[1]) { f[0] = v; }
  static __device__ __forceinline__ Val put(const float (&f)[1]) { return f[0]; }
  static __device__ __forceinline__ Raw least(Raw a, Raw b) { return fminf(a, b); }
  static __device__ __forceinline__ float lowest(Raw r) { return r; }
  // The full expf: its error stays at 2^-23 however many tokens multiply it.
  static __device__ __forceinline__ Val gate(Val log_a) { return expf(log_a); }
};
template <> struct Lane<__nv_bfloat16> {
  using Raw = uint32_t;
  using Val = uint64_t;
  static __device__ __forceinline__ Val open(Raw r) {
    return pack2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  static __device__ __forceinline__ Raw shut(Val v) {
    float f[2];
    unpack2(v, f[0], f[1]);
    return pack_bf16x2(f[0], f[1]);
  }
  static __device__ __forceinline__ Val all(float v) { return pack2(v, v); }
  static __device__ __forceinline__ Val fma(Val a, Val b, Val c) { return ffma2(a, b, c); }
  static __device__ __forceinline__ Val mul(Val a, Val b) { return fmul2(a, b); }
  static __device__ __forceinline__ Val add(Val a, Val b) { return fadd2(a, b); }
  static __device__ __forceinline__ void get(Val v, float (&f)[2]) { unpack2(v, f[0], f[1]); }
  static __device__ __forceinline__ Val put(const float (&f)[2]) { return pack2(f[0], f[1]); }
  static __device__ __forceinline__ Raw least(Raw a, Raw b) {
    const __nv_bfloat162 m = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const Raw*>(&m);
  }
  static __device__ __forceinline__ float lowest(Raw r) {
    return fminf(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  // The SFU's 2^x: 2^-22 relative, and |log_a| 2^-24 from the scaled argument.
  static __device__ __forceinline__ Val gate(Val log_a) {
    float f[2];
    unpack2(fmul2(log_a, pack2(kLog2e, kLog2e)), f[0], f[1]);
    return pack2(ex2(f[0]), ex2(f[1]));
  }
};

template <typename T>
__device__ __forceinline__ typename Lane<T>::Raw read4(const uint8_t* p) {
  return *reinterpret_cast<const typename Lane<T>::Raw*>(p);
}
template <typename T>
__device__ __forceinline__ void write4(uint8_t* p, typename Lane<T>::Raw v) {
  *reinterpret_cast<typename Lane<T>::Raw*>(p) = v;
}

// A decay of zero drops what came before, even if that is not finite.
__device__ __forceinline__ float decay_fma(float a, float h, float x) { return a == 0.f ? x : fmaf(a, h, x); }

// The decay over several tokens.  It is zero only where one of the gates is: open
// gates keep a NaN or an infinity in the state, however small their product, so that
// is held at the smallest subnormal (what a finite state adds through it is below 2^-149
// of that state).
constexpr float kLeastDecay = 1.4e-45f;
__device__ __forceinline__ float held(float a) { return a == 0.f ? kLeastDecay : a; }   // (of open gates)
__device__ __forceinline__ float join_decays(float a, float b) { return a == 0.f || b == 0.f ? 0.f : held(a * b); }

// log_a above this: the gate is not zero.
constexpr float kOpen = -87.f;

struct ScanArgs {
  const uint8_t* reset;
  const float* enter0;    // state entering the first chunk of the walk (rows enter0_stride apart), or null
  int64_t enter0_stride;
  float* leave;           // [B, D] state leaving the last, or null
  float* chunk_state;     // [B, C, D]
  int64_t L, D;
  int B, C, tiles;        // tiles of features
  // hand-off (ws, all ones at the start): [0] the counter, [1] set if a block
  // gave up; maps (A, h) [B, C, D]; group states [B, G, D]
  int* sync;
  uint64_t* map;
  uint32_t* group;
  int* status;
};

struct Tile {
  int c, b, tile;   // chunk along the walk
};

// Published values: single 64-bit (a map) or 32-bit (a state) words, several of
// them with one access; a word that still is all ones is not there yet.
constexpr uint64_t kNoMap = ~0ull;
constexpr uint32_t kNoState = ~0u;

__device__ __forceinline__ void publish(uint64_t* p, const uint64_t (&v)[2]) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(v[0]), "l"(v[1]) : "memory");
}
__device__ __forceinline__ void publish(uint64_t* p, const uint64_t (&v)[1]) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v[0]) : "memory");
}
__device__ __forceinline__ void publish(uint32_t* p, const uint32_t (&v)[2]) {
  asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(v[0]), "r"(v[1]) : "memory");
}
__device__ __forceinline__ void publish(uint32_t* p, const uint32_t (&v)[1]) {
  asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v[0]) : "memory");
}
__device__ __forceinline__ void peek(const uint64_t* p, uint64_t (&v)[2]) {
  asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "l"(p) : "memory");
}
__device__ __forceinline__ void peek(const uint64_t* p, uint64_t (&v)[1]) {
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v[0]) : "l"(p) : "memory");
}
__device__ __forceinline__ void peek(const uint32_t* p, uint32_t (&v)[2]) {
  asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p) : "memory");
}
__device__ __forceinline__ void peek(const uint32_t* p, uint32_t (&v)[1]) {
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v[0]) : "l"(p) : "memory");
}

// (A, h) as one word.  Arithmetic gives no NaN of all ones; one that an input
// carried through is stored as another NaN.
__device__ __forceinline__ uint32_t not_ones(float v) {
  const uint32_t u = __float_as_uint(v);
  return u == ~0u ? 0x7fffffffu : u;
}
__device__ __forceinline__ uint64_t map_word(float A, float h) {
  return (uint64_t)not_ones(h) << 32 | not_ones(A);
}

// Repeat `look` (true: all there) until it holds for the whole warp.  False if
// that takes longer than the wait limit, or another block gave up.
template <class Look>
__device__ __forceinline__ bool wait_for(const ScanArgs& a, Look&& look) {
  if (__all_sync(0xffffffffu, look())) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, look())) return true;
    if ((it & 63u) == 0) {
      const bool late = globaltimer_ns() - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, late || *reinterpret_cast<volatile int*>(a.sync + 1) == 1)) {
        if ((threadIdx.x & 31) == 0) {
          *reinterpret_cast<volatile int*>(a.sync + 1) = 1;
          atomicOr(a.status, kStatusTimeout);
        }
        return false;
      }
    }
  }
}

template <typename T, bool kBack>
struct ScanSmem {
  float2 map[kWarps][kFT<T>];    // (A, h) of every warp's span
  float2 back[kBack ? kWarps : 1][kBack ? kFT<T> : 1];   // the same of the reverse recurrence
  float2 pre[kWarps][kFT<T>];    // the maps of the group's earlier chunks, a quarter of them each
  float enter[kFT<T>];           // the state entering the group
  uint64_t bar;
  int abort_flag, unit;
};

// One lane's place in the hand-off.
template <int V>
struct Place {
  int first, n;       // the group's first chunk; its chunks before this one
  bool last, on;
  uint64_t* map;      // of this chunk
  uint32_t* group;    // of this group
  int64_t d;
};
template <int V>
__device__ __forceinline__ Place<V> place_of(const ScanArgs& a, const Tile& t, int64_t d) {
  Place<V> p;
  p.first = t.c / kGroup * kGroup;
  p.n = t.c - p.first;
  p.last = t.c + 1 == a.C;
  p.on = d < a.D;
  p.d = d;
  const int64_t G = (a.C + kGroup - 1) / kGroup;
  p.map = a.map + ((int64_t)t.b * a.C + t.c) * a.D + d;
  p.group = a.group + ((int64_t)t.b * G + p.first / kGroup) * a.D + d;
  return p;
}

// The chunk's map for the chunks of the group that come after it.
template <int V>
__device__ __forceinline__ void publish_map(const Place<V>& p, const float (&A)[V], const float (&m)[V]) {
  if (!p.on || p.last || p.n == kGroup - 1) return;
  uint64_t w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) w[i] = map_word(A[i], m[i]);
  publish(p.map, w);
}

// Every warp: wait for a quarter of the group's earlier maps and compose them;
// warp 0 also for the state entering the group.  All of them are asked for at
// once, so the hand-off costs one trip to the L2.  False if the wait ran out.
template <int V, class Smem>
__device__ __forceinline__ bool gather(const ScanArgs& a, const Tile& t, const Place<V>& p, int warp, int f, Smem& sm) {
  constexpr int kEach = kGroup / kWarps;
  const int c0 = warp * kEach;
  uint64_t w[kEach][V];
  uint32_t g[V];
  const bool state = warp == 0 && p.first > 0;
  const bool ok = wait_for(a, [&] {
    if (!p.on) return true;
#pragma unroll
    for (int c = 0; c < kEach; ++c)
      if (c0 + c < p.n) peek(p.map - (int64_t)(p.n - c0 - c) * a.D, w[c]);
    if (state) peek(p.group, g);
    bool there = true;
#pragma unroll
    for (int c = 0; c < kEach; ++c)
      if (c0 + c < p.n)
#pragma unroll
        for (int i = 0; i < V; ++i) there &= w[c][i] != kNoMap;
    if (state)
#pragma unroll
      for (int i = 0; i < V; ++i) there &= g[i] != kNoState;
    return there;
  });
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float A = 1.f, h = 0.f;
    if (p.on)
#pragma unroll
      for (int c = 0; c < kEach; ++c)
        if (c0 + c < p.n) {
          const float ca = __uint_as_float((uint32_t)w[c][i]);
          h = decay_fma(ca, h, __uint_as_float((uint32_t)(w[c][i] >> 32)));
          A = join_decays(A, ca);
        }
    sm.pre[warp][f + i] = make_float2(A, h);
    if (warp == 0) {
      float e = 0.f;
      if (p.on) e = state ? __uint_as_float(g[i]) : a.enter0 ? a.enter0[t.b * a.enter0_stride + p.d + i] : 0.f;
      sm.enter[f + i] = e;
    }
  }
  return ok;
}

// The state leaving the chunk, for the next group and the caller.
template <int V>
__device__ __forceinline__ void pass_on(const ScanArgs& a, const Tile& t, const Place<V>& p, const float (&A)[V],
                                        const float (&m)[V], const float (&h)[V]) {
  if (!p.on) return;
  if (p.n == kGroup - 1 && !p.last) {
    uint32_t w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = not_ones(decay_fma(A[i], h[i], m[i]));
    publish(p.group + a.D, w);
  }
  if (p.last && a.leave) {
#pragma unroll
    for (int i = 0; i < V; ++i) a.leave[(int64_t)t.b * a.D + p.d + i] = decay_fma(A[i], h[i], m[i]);
  }
}

// Which tile this block takes: drawn from the counter, or (one chunk: nothing
// to wait for) the block's own index.
__device__ __forceinline__ Tile draw_tile(const ScanArgs& a, int* slot) {
  if (threadIdx.x == 0) *slot = a.C > 1 ? atomicAdd(a.sync, 1) + 1 : (int)blockIdx.x;   // counts from -1
  __syncthreads();
  const int u = *slot, per_chunk = a.B * a.tiles;
  Tile t;
  t.c = u / per_chunk;
  const int r = u - t.c * per_chunk;
  t.b = r / a.tiles;
  t.tile = r - t.b * a.tiles;
  return t;
}

// Bit s: a document starts at token t0 + s.
__device__ __forceinline__ uint32_t start_bits(const ScanArgs& a, int b, int64_t t0) {
  const int lane = threadIdx.x & 31;
  const bool start = a.reset && t0 + lane < a.L && a.reset[(int64_t)b * a.L + t0 + lane];
  return __ballot_sync(0xffffffffu, start);
}

// One token's gates.  kShut: some gate of the span may be zero (a document
// starts there, or log_a is low enough), and what a zero gate meets is dropped;
// otherwise the products are taken as they are, two features at a time.
template <typename T, bool kShut>
__device__ __forceinline__ typename Lane<T>::Val gate_at(typename Lane<T>::Raw raw, uint32_t starts, int s) {
  using X = Lane<T>;
  const typename X::Val g = X::gate(X::open(raw));
  return kShut && (starts >> s & 1u) ? X::all(0.f) : g;
}

// a h + x, x where a is zero.
template <typename T, bool kShut>
__device__ __forceinline__ typename Lane<T>::Val step(typename Lane<T>::Val a, typename Lane<T>::Val h,
                                                      typename Lane<T>::Val x) {
  using X = Lane<T>;
  if (!kShut) return X::fma(a, h, x);
  float av[kV<T>], hv[kV<T>], xv[kV<T>];
  X::get(a, av);
  X::get(h, hv);
  X::get(x, xv);
#pragma unroll
  for (int i = 0; i < kV<T>; ++i) hv[i] = decay_fma(av[i], hv[i], xv[i]);
  return X::put(hv);
}

// v, 0 where a is zero.
template <typename T, bool kShut>
__device__ __forceinline__ typename Lane<T>::Val passed(typename Lane<T>::Val a, typename Lane<T>::Val v) {
  using X = Lane<T>;
  if (!kShut) return v;
  float av[kV<T>], vv[kV<T>];
  X::get(a, av);
  X::get(v, vv);
#pragma unroll
  for (int i = 0; i < kV<T>; ++i) vv[i] = av[i] == 0.f ? 0.f : vv[i];
  return X::put(vv);
}

// a b, 0 where a is zero.
template <typename T, bool kShut>
__device__ __forceinline__ typename Lane<T>::Val times(typename Lane<T>::Val a, typename Lane<T>::Val b) {
  return passed<T, kShut>(a, Lane<T>::mul(a, b));
}

// The decays' product, one token on.  (kShut = false: zero once it underflows, which
// is looked at behind the span.)
template <typename T, bool kShut>
__device__ __forceinline__ typename Lane<T>::Val next_decay(typename Lane<T>::Val A, typename Lane<T>::Val g) {
  using X = Lane<T>;
  if (!kShut) return X::mul(A, g);
  float Av[kV<T>], gv[kV<T>];
  X::get(A, Av);
  X::get(g, gv);
#pragma unroll
  for (int i = 0; i < kV<T>; ++i) Av[i] = join_decays(Av[i], gv[i]);
  return X::put(Av);
}

// The map of a span: A the product of its gates, h its scan from zero; for the
// backward also e, what the span passes back of its own output gradients.
// Returns the lowest log_a.  Tokens past the end read as zeros: a = 1, x = 0,
// the identity.
template <typename T, bool kShut, bool kBack>
__device__ __forceinline__ float span_map(const uint8_t* pg, const uint8_t* px, const uint8_t* pd, uint32_t starts,
                                          typename Lane<T>::Val& A, typename Lane<T>::Val& h,
                                          typename Lane<T>::Val& e) {
  using X = Lane<T>;
  A = X::all(1.f);
  h = e = X::all(0.f);
  typename X::Raw low = read4<T>(pg);
#pragma unroll 8
  for (int s = 0; s < kSpan; ++s) {
    const typename X::Raw raw = read4<T>(pg + s * kRowBytes);
    low = X::least(low, raw);
    const typename X::Val g = gate_at<T, kShut>(raw, starts, s);
    h = step<T, kShut>(g, h, X::open(read4<T>(px + s * kRowBytes)));
    A = next_decay<T, kShut>(A, g);
    if (kBack) e = X::add(e, times<T, kShut>(A, X::open(read4<T>(pd + s * kRowBytes))));
  }
  return X::lowest(low);
}

// Whether the careful form is needed, decided for the warp; the map that goes
// with it.  (The map alone also needs it where an infinite output gradient met a
// product of open gates that had underflowed, as a NaN shows.)
template <typename T, bool kBack>
__device__ __forceinline__ bool span_map_of(const uint8_t* pg, const uint8_t* px, const uint8_t* pd, uint32_t starts,
                                            typename Lane<T>::Val& A, typename Lane<T>::Val& h,
                                            typename Lane<T>::Val& e) {
  using X = Lane<T>;
  const bool open =
      !starts && __all_sync(0xffffffffu, span_map<T, false, kBack>(pg, px, pd, 0, A, h, e) > kOpen);
  bool whole = open;
  if (open) {
    float v[kV<T>], ev[kV<T>];
    X::get(A, v);
    X::get(e, ev);
    bool lost = false;
#pragma unroll
    for (int i = 0; i < kV<T>; ++i) {
      lost |= v[i] == 0.f && isnan(ev[i]);
      v[i] = held(v[i]);
    }
    A = X::put(v);
    if (kBack) whole = !__any_sync(0xffffffffu, lost);
  }
  if (!whole) span_map<T, true, kBack>(pg, px, pd, starts, A, h, e);
  return !open;
}

// y over the consumed x.
template <typename T, bool kShut>
__device__ __forceinline__ void span_out(const uint8_t* pg, uint8_t* px, uint32_t starts, typename Lane<T>::Val h) {
  using X = Lane<T>;
  // (reads of eight tokens ahead of their writes, which might alias for all the compiler knows)
#pragma unroll
  for (int s0 = 0; s0 < kSpan; s0 += 8) {
    typename X::Raw g[8], x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = read4<T>(pg + (s0 + i) * kRowBytes);
      x[i] = read4<T>(px + (s0 + i) * kRowBytes);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h = step<T, kShut>(gate_at<T, kShut>(g[i], starts, s0 + i), h, X::open(x[i]));
      x[i] = X::shut(h);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) write4<T>(px + (s0 + i) * kRowBytes, x[i]);
  }
}

// The states h_{t-1} of a span.
template <typename T, bool kShut>
__device__ __forceinline__ void span_states(const uint8_t* pg, const uint8_t* px, uint32_t starts,
                                            typename Lane<T>::Val h, typename Lane<T>::Val (&before)[kSpan]) {
  using X = Lane<T>;
#pragma unroll
  for (int s = 0; s < kSpan; ++s) {
    before[s] = h;
    const typename X::Val g = gate_at<T, kShut>(read4<T>(pg + s * kRowBytes), starts, s);
    h = step<T, kShut>(g, h, X::open(read4<T>(px + s * kRowBytes)));
  }
}

// dx over dy, dlog_a over log_a.
template <typename T, bool kShut>
__device__ __forceinline__ void span_back(uint8_t* pg, uint8_t* pd, uint32_t starts, typename Lane<T>::Val e,
                                          const typename Lane<T>::Val (&before)[kSpan]) {
  using X = Lane<T>;
#pragma unroll
  for (int s0 = kSpan - 8; s0 >= 0; s0 -= 8) {
    typename X::Raw g[8], dy[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = read4<T>(pg + (s0 + i) * kRowBytes);
      dy[i] = read4<T>(pd + (s0 + i) * kRowBytes);
    }
#pragma unroll
    for (int i = 7; i >= 0; --i) {
      const typename X::Val a = gate_at<T, kShut>(g[i], starts, s0 + i);
      const typename X::Val dh = X::add(X::open(dy[i]), e);
      e = times<T, kShut>(a, dh);
      dy[i] = X::shut(dh);
      // (where the gate is zero before may not be finite)
      g[i] = X::shut(passed<T, kShut>(a, X::mul(e, before[s0 + i])));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      write4<T>(pd + (s0 + i) * kRowBytes, dy[i]);
      write4<T>(pg + (s0 + i) * kRowBytes, g[i]);
    }
  }
}

// Map of the chunk and, for this thread's span, of what precedes it in the chunk.
template <int V, int F>
__device__ __forceinline__ void fold(const float2 (&map)[kWarps][F], int f, int from, int to, int step, float (&A)[V],
                                     float (&h)[V]) {
  for (int w = from; w != to; w += step)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 m = map[w][f + i];
      h[i] = decay_fma(m.x, h[i], m.y);
      A[i] = join_decays(A[i], m.x);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 6) scan_kernel(const __grid_constant__ CUtensorMap mx,
                                                           const __grid_constant__ CUtensorMap mg,
                                                           const __grid_constant__ CUtensorMap my, const ScanArgs a) {
  constexpr int V = kV<T>, F = kFT<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tx = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint8_t* tg = tx + kTileBytes;
  __shared__ ScanSmem<T, false> sm;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    mbar_init(&sm.bar, 1);
    fence_mbar_init();
  }
  wait_for_previous();   // the hand-off's memory is set
  const Tile t = draw_tile(a, &sm.unit);
  const int64_t t0 = (int64_t)t.c * kScanChunk;
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(&sm.bar, 2 * kTileBytes);
    tma_load_3d(tx, &mx, &sm.bar, t.tile * F, (int)t0, t.b);
    tma_load_3d(tg, &mg, &sm.bar, t.tile * F, (int)t0, t.b);
  }
  const uint32_t starts = start_bits(a, t.b, t0 + warp * kSpan);
  const bool loaded = mbar_wait(&sm.bar, 0, &sm.abort_flag, a.status);
  if (__syncthreads_or(!loaded)) {
    mbar_wait_drain(&sm.bar, 0);
    return;
  }
  uint8_t *px = tx + warp * kSpan * kRowBytes + lane * 4, *pg = tg + warp * kSpan * kRowBytes + lane * 4;
  const int f = lane * V;
  using X = Lane<T>;
  bool shut;
  {
    typename X::Val Av, hv, ev;
    shut = span_map_of<T, false>(pg, px, nullptr, starts, Av, hv, ev);
    float A[V], h[V];
    X::get(Av, A);
    X::get(hv, h);
#pragma unroll
    for (int i = 0; i < V; ++i) sm.map[warp][f + i] = make_float2(A[i], h[i]);
  }
  __syncthreads();
  const Place<V> pl = place_of<V>(a, t, (int64_t)t.tile * F + f);
  float cA[V], cm[V];   // warp 0: the chunk's map
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) cA[i] = 1.f, cm[i] = 0.f;
    fold<V, F>(sm.map, f, 0, kWarps, 1, cA, cm);
    publish_map(pl, cA, cm);
  }
  if (__syncthreads_or(!gather(a, t, pl, warp, f, sm))) return;
  float A[V], h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = sm.enter[f + i], A[i] = 1.f;
  fold<V, F>(sm.pre, f, 0, kWarps, 1, A, h);
  if (warp == 0) {
    pass_on(a, t, pl, cA, cm, h);
    if (a.chunk_state && pl.on) {
#pragma unroll
      for (int i = 0; i < V; ++i) a.chunk_state[((int64_t)t.b * a.C + t.c) * a.D + pl.d + i] = h[i];
    }
  }
  fold<V, F>(sm.map, f, 0, warp, 1, A, h);
  if (shut) span_out<T, true>(pg, px, starts, X::put(h));
  else span_out<T, false>(pg, px, starts, X::put(h));
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x == 0) {
    tma_store_3d(&my, tx, t.tile * F, (int)t0, t.b);
    bulk_commit();
    bulk_wait_read_all();
  }
}

// A few tokens (generation): no tile to fill, a thread walks over the tokens of
// four features.  Measured, this takes 1.5 us + 0.23 us a token, the chunk
// kernel 5 us and, beyond 64 tiles, about 0.008 us a tile more (1 to 128 tokens
// of 512 to 131072 features); past 64 tokens its strided rows lose to TMA's.
bool short_is_faster(int64_t L, int64_t tiles) { return L <= 64 && L <= 16 + tiles / 64; }

template <typename T>
struct alignas(4 * sizeof(T)) Four {
  T v[4];
};

// The same gates as the chunk kernel's.
template <typename T>
__device__ __forceinline__ float gate1(float log_a) {
  return sizeof(T) == 2 ? ex2(log_a * kLog2e) : expf(log_a);
}

template <typename T>
__global__ void __launch_bounds__(128) scan_short_kernel(const T* x, const T* log_a, T* y, const float* state_in,
                                                         float* state_out, const ScanArgs a) {
  const int64_t i = ((int64_t)blockIdx.x * 128 + threadIdx.x) * 4;
  if (i >= a.B * a.D) return;
  const int64_t b = i / a.D, d = i - b * a.D;
  float h[4] = {};
  if (state_in) {
    const float4 s = *reinterpret_cast<const float4*>(state_in + i);
    h[0] = s.x, h[1] = s.y, h[2] = s.z, h[3] = s.w;
  }
  if (a.chunk_state) *reinterpret_cast<float4*>(a.chunk_state + i) = make_float4(h[0], h[1], h[2], h[3]);
  const int64_t at = b * a.L * a.D + d;
  const int L = (int)a.L;
#pragma unroll 4
  for (int t = 0; t < L; ++t) {
    const Four<T> g = *reinterpret_cast<const Four<T>*>(log_a + at + t * a.D);
    const Four<T> u = *reinterpret_cast<const Four<T>*>(x + at + t * a.D);
    const bool start = a.reset && a.reset[b * a.L + t];
    Four<T> o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = decay_fma(start ? 0.f : gate1<T>(to_f32(g.v[j])), h[j], to_f32(u.v[j]));
      o.v[j] = from_f32<T>(h[j]);
    }
    *reinterpret_cast<Four<T>*>(y + at + t * a.D) = o;
  }
  if (state_out) *reinterpret_cast<float4*>(state_out + i) = make_float4(h[0], h[1], h[2], h[3]);
}

// The backward walks the chunks from the last to the first.  A warp finds the
// maps of both recurrences over its span in one ascending pass: with P_t the
// product of the span's gates up to t, what the span passes back is
// e = sum_t P_t dy_t + P e_next.  Then it scans forward again, keeping the 32
// states h_{t-1} in registers, and back over them.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) scan_bwd_kernel(const __grid_constant__ CUtensorMap mx,
                                                               const __grid_constant__ CUtensorMap mg,
                                                               const __grid_constant__ CUtensorMap mdy,
                                                               const __grid_constant__ CUtensorMap mdx,
                                                               const __grid_constant__ CUtensorMap mdg,
                                                               const ScanArgs a) {
  constexpr int V = kV<T>, F = kFT<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* tx = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint8_t *tg = tx + kTileBytes, *td = tg + kTileBytes;
  __shared__ ScanSmem<T, true> sm;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    mbar_init(&sm.bar, 1);
    fence_mbar_init();
  }
  wait_for_previous();   // the hand-off's memory is set
  const Tile t = draw_tile(a, &sm.unit);
  const int c = a.C - 1 - t.c;
  const int64_t t0 = (int64_t)c * kScanChunk;
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(&sm.bar, 3 * kTileBytes);
    tma_load_3d(tx, &mx, &sm.bar, t.tile * F, (int)t0, t.b);
    tma_load_3d(tg, &mg, &sm.bar, t.tile * F, (int)t0, t.b);
    tma_load_3d(td, &mdy, &sm.bar, t.tile * F, (int)t0, t.b);
  }
  const int f = lane * V;
  const int64_t d = (int64_t)t.tile * F + f;
  const uint32_t starts = start_bits(a, t.b, t0 + warp * kSpan);
  float h0[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h0[i] = d < a.D ? a.chunk_state[((int64_t)t.b * a.C + c) * a.D + d + i] : 0.f;
  const bool loaded = mbar_wait(&sm.bar, 0, &sm.abort_flag, a.status);
  if (__syncthreads_or(!loaded)) {
    mbar_wait_drain(&sm.bar, 0);
    return;
  }
  const int off = warp * kSpan * kRowBytes + lane * 4;
  uint8_t *px = tx + off, *pg = tg + off, *pd = td + off;
  using X = Lane<T>;
  bool shut;
  {
    typename X::Val Pv, hv, ev;
    shut = span_map_of<T, true>(pg, px, pd, starts, Pv, hv, ev);
    float P[V], h[V], e[V];
    X::get(Pv, P);
    X::get(hv, h);
    X::get(ev, e);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sm.map[warp][f + i] = make_float2(P[i], h[i]);
      sm.back[warp][f + i] = make_float2(P[i], e[i]);
    }
  }
  __syncthreads();
  const Place<V> pl = place_of<V>(a, t, d);
  float cA[V], cm[V];   // warp 0: the chunk's map
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) cA[i] = 1.f, cm[i] = 0.f;
    fold<V, F>(sm.back, f, kWarps - 1, -1, -1, cA, cm);
    publish_map(pl, cA, cm);
  }
  // the states of this span, while the maps of others arrive
  float A[V], h[V];
#pragma unroll
  for (int i = 0; i < V; ++i) h[i] = h0[i], A[i] = 1.f;
  fold<V, F>(sm.map, f, 0, warp, 1, A, h);
  typename X::Val before[kSpan];
  if (shut) span_states<T, true>(pg, px, starts, X::put(h), before);
  else span_states<T, false>(pg, px, starts, X::put(h), before);
  if (__syncthreads_or(!gather(a, t, pl, warp, f, sm))) return;
  float e[V];
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = sm.enter[f + i];
  fold<V, F>(sm.pre, f, 0, kWarps, 1, A, e);
  if (warp == 0) pass_on(a, t, pl, cA, cm, e);
  fold<V, F>(sm.back, f, kWarps - 1, warp, -1, A, e);
  if (shut) span_back<T, true>(pg, pd, starts, X::put(e), before);
  else span_back<T, false>(pg, pd, starts, X::put(e), before);
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x == 0) {
    tma_store_3d(&mdx, td, t.tile * F, (int)t0, t.b);
    tma_store_3d(&mdg, tg, t.tile * F, (int)t0, t.b);
    bulk_commit();
    bulk_wait_read_all();
  }
}

// ------------------------------------------------------------------- host --

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(p)
               : nullptr;
  }();
  return fn;
}

// [B, L, D] as a 3D map {D, L, B}, box {128 bytes of features, 128, 1}.
template <typename T>
bool make_map(CUtensorMap* m, const void* base, const ScanProblem& p) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  constexpr cuuint64_t e = sizeof(T);
  cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.L, (cuuint64_t)p.B};
  cuuint64_t strides[2] = {(cuuint64_t)p.D * e, (cuuint64_t)p.L * p.D * e};
  cuuint32_t box[3] = {kFT<T>, kScanChunk, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, e == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int64_t tiles_of(int64_t D, int dtype) {
  const int64_t ft = dtype == kBF16 ? kFT<__nv_bfloat16> : kFT<float>;
  return (D + ft - 1) / ft;
}
constexpr size_t kSyncBytes = 256;
int64_t groups_of(int64_t L) { return (scan_chunks(L) + kGroup - 1) / kGroup; }

// All ones over the hand-off's memory.
__global__ void __launch_bounds__(256) scan_clear_kernel(uint4* p, int64_t n) {
  let_next_start();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// Fill the arguments, enter and leave being the states at the walk's ends, and
// set the hand-off's memory to all ones.  The last chunk may be done before others of the
// first group have read the entering state, so if it is to be overwritten
// they read a copy (in the slot of the first group's state).  *chained: the
// scan may be launched as the clearing kernel's next.
cudaError_t set_args(const ScanProblem& p, const float* enter, float* leave, ScanArgs* a, bool* chained,
                     cudaStream_t st) {
  a->reset = p.reset;
  a->chunk_state = p.chunk_state;
  a->L = p.L;
  a->D = p.D;
  a->B = (int)p.B;
  a->C = (int)scan_chunks(p.L);
  a->tiles = (int)tiles_of(p.D, p.dtype);
  a->status = p.status;
  char* ws = static_cast<char*>(p.ws);
  a->sync = reinterpret_cast<int*>(ws);
  const size_t map_bytes = up256(sizeof(uint64_t) * p.B * a->C * p.D);
  a->map = reinterpret_cast<uint64_t*>(ws + kSyncBytes);
  a->group = reinterpret_cast<uint32_t*>(ws + kSyncBytes + map_bytes);
  a->enter0 = enter;
  a->enter0_stride = p.D;
  a->leave = leave;
  *chained = a->C > 1 && !(enter && enter == leave);
  if (a->C == 1) return cudaSuccess;
  const int64_t words = (int64_t)scan_workspace_bytes(p.B, p.L, p.D, p.dtype, false) / 16, blocks = (words + 255) / 256;
  const int64_t wave = 4 * (int64_t)sm_count();
  scan_clear_kernel<<<(unsigned)(blocks < wave ? blocks : wave), 256, 0, st>>>(reinterpret_cast<uint4*>(ws), words);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (enter && enter == leave) {
    a->enter0 = reinterpret_cast<float*>(a->group);
    a->enter0_stride = groups_of(p.L) * p.D;
    const size_t row = sizeof(float) * p.D;
    if (cudaError_t e = cudaMemcpy2DAsync(a->group, row * groups_of(p.L), enter, row, row, p.B,
                                          cudaMemcpyDeviceToDevice, st))
      return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t scan_impl(const ScanProblem& p, cudaStream_t st) {
  if (short_is_faster(p.L, p.B * tiles_of(p.D, p.dtype))) {
    ScanArgs a{};
    a.reset = p.reset;
    a.chunk_state = p.chunk_state;
    a.L = p.L;
    a.D = p.D;
    a.B = (int)p.B;
    scan_short_kernel<T><<<(unsigned)((p.B * p.D / 4 + 127) / 128), 128, 0, st>>>(
        static_cast<const T*>(p.x), static_cast<const T*>(p.log_a), static_cast<T*>(p.y), p.state_in, p.state_out, a);
    return cudaGetLastError();
  }
  CUtensorMap mx, mg, my;
  if (!make_map<T>(&mx, p.x, p) || !make_map<T>(&mg, p.log_a, p) || !make_map<T>(&my, p.y, p))
    return cudaErrorInvalidValue;
  ScanArgs a;
  bool chained;
  cudaError_t e;
  if ((e = set_args(p, p.state_in, p.state_out, &a, &chained, st))) return e;
  constexpr int smem = 2 * kTileBytes + 128;
  if ((e = cudaFuncSetAttribute(scan_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
  return launch_chained(scan_kernel<T>, dim3((unsigned)(a.C * a.B * a.tiles)), kThreads, smem, 0, chained, st, mx, mg,
                        my, a);
}

template <typename T>
cudaError_t scan_bwd_impl(const ScanProblem& p, cudaStream_t st) {
  CUtensorMap mx, mg, mdy, mdx, mdg;
  if (!make_map<T>(&mx, p.x, p) || !make_map<T>(&mg, p.log_a, p) || !make_map<T>(&mdy, p.dy, p) ||
      !make_map<T>(&mdx, p.dx, p) || !make_map<T>(&mdg, p.dlog_a, p))
    return cudaErrorInvalidValue;
  ScanArgs a;
  bool chained;
  cudaError_t e;
  if ((e = set_args(p, p.dstate_out, p.dstate_in, &a, &chained, st))) return e;
  constexpr int smem = 3 * kTileBytes + 128;
  if ((e = cudaFuncSetAttribute(scan_bwd_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
  return launch_chained(scan_bwd_kernel<T>, dim3((unsigned)(a.C * a.B * a.tiles)), kThreads, smem, 0, chained, st, mx,
                        mg, mdy, mdx, mdg, a);
}

}  // namespace

bool scan_grid_fits(int64_t B, int64_t L, int64_t D, int dtype) {
  // one block per tile; a tensor map's strides stay below 2^40 bytes
  return (long double)B * tiles_of(D, dtype) * scan_chunks(L) < 2147483647.0L && (long double)L * D < 2.0e11L;
}

size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t D, int, bool) {
  if (scan_chunks(L) == 1) return 0;
  return kSyncBytes + up256(sizeof(uint64_t) * (size_t)(B * scan_chunks(L) * D)) +
         up256(sizeof(uint32_t) * (size_t)(B * groups_of(L) * D));
}

cudaError_t launch_scan(const ScanProblem& p, cudaStream_t st) {
  return p.dtype == kBF16 ? scan_impl<__nv_bfloat16>(p, st) : scan_impl<float>(p, st);
}

cudaError_t launch_scan_bwd(const ScanProblem& p, cudaStream_t st) {
  return p.dtype == kBF16 ? scan_bwd_impl<__nv_bfloat16>(p, st) : scan_bwd_impl<float>(p, st);
}

}  // namespace gecko
