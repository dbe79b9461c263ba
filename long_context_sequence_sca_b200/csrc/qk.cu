// Queries and keys of one layer from the shared representation z, per head:
//   z' = z / max(|z|_2, eps),   p_i = scale_i (.) z' + shift_i  (i = q, k, q_m, k_m),
// with q and k turned by the token's position: each rotated pair (a, b) with
// angle pos * rate becomes (a cos - b sin, b cos + a sin).  Gradients:
//   dp_q, dp_k turned back;  g = sum_i scale_i (.) dp_i;
//   dz = (g - z' (z'.g)) / |z|   (g / eps where |z| <= eps);
//   dscale_i = sum_{b,t} dp_i (.) z',   dshift_i = sum_{b,t} dp_i.
// Everything is held in fp32; the angles are formed in revolutions in fp64
// (a position of some millions times a rate has no bits left below one
// revolution in fp32) and reduced to [-1/2, 1/2] before the fp32 sincospi.
#include "chain.cuh"
#include "common.cuh"
#include "gecko_internal.h"

namespace gecko {
namespace {

constexpr int kFwdThreads = 256, kFwdBlocks = 2;     // threads per block, blocks per SM (registers)
constexpr int kBwdThreads = 384, kBwdBlocks = 1;
// Rounds of rows on their way to shared memory in the backward (five rows of 16
// or 32 bytes per thread each).
template <typename T> constexpr int kStages = sizeof(T) == 2 ? 4 : 3;
constexpr int kQkTokens = 48;   // tokens per fill of the sine table, at least a round's
enum { kRotNone = 0, kRotHalves = 1, kRotInterleaved = 2 };

struct QkArgs {
  const void* z;
  const float *scale, *shift;
  const int64_t* pos;
  void* out[4];
  const void* dout[4];
  void* dz;
  float* part;         // backward: [rows of partial sums, 8, H * d]
  int64_t n_tokens, T;
  int H, heads_per_block, token_slots, tokens_per_block;
  int tokens_per_fill;   // of the sine table: whole rounds of the token slots
  float eps;
  int64_t pos0;
  int rot_dim;
  double rate[kMaxRotPairs];
};

// 8 features as four packed fp32 pairs.
struct P4 {
  uint64_t v[4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(0.f, 0.f);
  }
};

// 8 elements as loaded, so that a prefetched row takes as few registers as it can.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ P4 get() const {
    return {{pack2(a.x, a.y), pack2(a.z, a.w), pack2(b.x, b.y), pack2(b.z, b.w)}};
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ P4 get() const {
    P4 r;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.v[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    return r;
  }
};
__device__ __forceinline__ P4 load8(const float* p) {
  Raw8<float> r;
  r.load(p);
  return r.get();
}
__device__ __forceinline__ void store8(float* p, const P4& f) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(f.v[i], v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const P4& f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(f.v[i], lo, hi);
    w[i] = pack_bf16x2(lo, hi);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float dot8(const P4& a, const P4& b) {
  const uint64_t s = ffma2(a.v[2], b.v[2], fmul2(a.v[0], b.v[0])), t = ffma2(a.v[3], b.v[3], fmul2(a.v[1], b.v[1]));
  float lo, hi;
  unpack2(fadd2(s, t), lo, hi);
  return lo + hi;
}

// The sine table: (cos, cos, sin, sin) of every two neighbouring rotated pairs
// of the fill's tokens.  A lane reads kPer pairs of a row, two with each
// access; these pieces of a row are ordered so that the lanes of one access
// are consecutive.
template <int kRot>
constexpr int kPer = kRot == kRotInterleaved ? 4 : 8;

template <int kRot, int kThreads>
__device__ __forceinline__ void fill_turns(float4* turns, const double* rate, const QkArgs& a, int64_t n0, int n,
                                           uint32_t t0) {
  constexpr int kPieces = kPer<kRot> / 2;   // pieces per lane
  const int pairs = a.rot_dim / 2, readers = pairs / kPer<kRot>;
  // a thread keeps its pair and steps over tokens
  const int step = kThreads / pairs, pair = threadIdx.x % pairs, piece = pair >> 1;
  float* out = reinterpret_cast<float*>(turns) + 4 * (piece % kPieces * readers + piece / kPieces) + (pair & 1);
  const double r = rate[pair];
  if (threadIdx.x >= step * pairs) return;
  for (int k = threadIdx.x / pairs; k < n; k += step) {
    uint32_t t = t0 + k;
    if (t >= a.T) t %= (uint32_t)a.T;
    const int64_t pos = a.pos ? a.pos[n0 + k] : a.pos0 + t;
    const double rev = (double)pos * r;
    float s, c;
    sincospif((float)(2.0 * (rev - rint(rev))), &s, &c);
    out[2 * k * pairs] = c;
    out[2 * k * pairs + 2] = s;
  }
}

// What turns this lane's 8 features: p -> p c + partner s, as packed pairs; the
// partner is the other half's feature (halves), or the other of the two
// (interleaved).
struct Turn {
  uint64_t c[4], s[4];
};

// Where a lane reads its pieces: `at` + row and pieces `step` apart; a lane beyond
// the rotated features reads an entry behind the table, c = 1 and s = 0.
struct TurnPlace {
  int at, row, step;
  uint64_t sign;   // (halves) of the partner's term
};
template <int kRot>
__device__ __forceinline__ TurnPlace turn_place(float4* turns, int entries, int l, int rot_dim, float sign) {
  const int readers = rot_dim / 2 / kPer<kRot>;
  const bool in = 8 * l < rot_dim, upper = kRot == kRotHalves && l >= readers;
  if (threadIdx.x == 0) turns[entries] = make_float4(1.f, 1.f, 0.f, 0.f);
  const float sg = upper ? sign : -sign;
  return {in ? upper ? l - readers : l : entries, in ? rot_dim / 4 : 0, in ? readers : 0, pack2(sg, sg)};
}

template <int kRot>
__device__ __forceinline__ void load_turn(Turn& r, const float4* turns, const TurnPlace& t, int k) {
  const float4* p = turns + t.at + k * t.row;
  if (kRot == kRotHalves) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = p[i * t.step];
      r.c[i] = pack2(v.x, v.y);
      r.s[i] = fmul2(pack2(v.z, v.w), t.sign);
    }
  } else {
    // partner of the even feature: -sin, of the odd one: +sin (t.sign has the even one's)
    float sg, unused;
    unpack2(t.sign, sg, unused);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = p[i * t.step];
      r.c[2 * i] = pack2(v.x, v.x);
      r.c[2 * i + 1] = pack2(v.y, v.y);
      r.s[2 * i] = pack2(v.z * sg, -v.z * sg);
      r.s[2 * i + 1] = pack2(v.w * sg, -v.w * sg);
    }
  }
}

// src: the lane that holds the partners (halves), which every lane of the
// warp must pass here.
template <int kRot>
__device__ __forceinline__ void turn8(P4& p, const Turn& r, int src) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(p.v[i], lo, hi);
    uint64_t partner;
    if (kRot == kRotHalves)
      partner = pack2(__shfl_sync(0xffffffffu, lo, src), __shfl_sync(0xffffffffu, hi, src));
    else
      partner = pack2(hi, lo);
    p.v[i] = ffma2(partner, r.s[i], fmul2(p.v[i], r.c[i]));
  }
}

// Root and reciprocal, once a row: rounded ones for fp32 tensors, for bf16 the SFU's,
// within a unit or two of the last place.
template <typename T>
__device__ __forceinline__ float root(float x) {
  if (sizeof(T) == 4) return sqrtf(x);
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <typename T>
__device__ __forceinline__ float reciprocal(float x) {
  if (sizeof(T) == 4) return 1.f / x;
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int m = D / 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// One row (token, head) per D / 8 lanes; a row slot keeps its head, so its
// affine parameters stay in registers while it walks over tokens.
struct Slot {
  int lane, l, src, head, tsub;
  bool on;
};
template <int D>
__device__ __forceinline__ Slot my_slot(const QkArgs& a) {
  constexpr int kLanes = D / 8;
  Slot s;
  s.lane = threadIdx.x & 31;
  s.l = s.lane % kLanes;
  const int slot = threadIdx.x / kLanes, hb = blockIdx.y * a.heads_per_block;
  s.head = hb + slot % a.heads_per_block;
  s.tsub = slot / a.heads_per_block;
  s.on = s.tsub < a.token_slots && s.head < a.H;
  const int half = a.rot_dim / 16;
  s.src = s.lane + (s.l < half ? half : s.l < 2 * half ? -half : 0);
  return s;
}

// Where a row slot stands: token n0 + k of the fill, as batch b and token t.
struct Walk {
  int64_t b;
  uint32_t t;
  __device__ __forceinline__ void start(int64_t tok, int64_t T) {
    b = tok / T;
    t = (uint32_t)(tok - b * T);
  }
  __device__ __forceinline__ void step(int by, int64_t T) {
    t += by;
    if (t >= T) {
      const uint32_t q = t / (uint32_t)T;
      b += q;
      t -= q * (uint32_t)T;
    }
  }
  __device__ __forceinline__ int64_t row(int64_t H, int64_t T, int head) const { return (b * H + head) * T + t; }
};

template <typename T, int D, int kRot>
__global__ void __launch_bounds__(kFwdThreads, kFwdBlocks) qk_kernel(const __grid_constant__ QkArgs a) {
  __shared__ float4 turns[kRot == kRotNone ? 1 : kQkTokens * D / 4 + 1];
  __shared__ double rate[kMaxRotPairs];   // the parameter bank would serialise the lanes' reads
  if (kRot != kRotNone && threadIdx.x < a.rot_dim / 2) rate[threadIdx.x] = a.rate[threadIdx.x];
  const int64_t first = (int64_t)blockIdx.x * a.tokens_per_block;
  const int64_t last = min(first + a.tokens_per_block, a.n_tokens);
  const Slot s = my_slot<D>(a);
  P4 sc[4], sh[4];
  if (s.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = ((int64_t)i * a.H + s.head) * D + 8 * s.l;
      sc[i] = load8(a.scale + at);
      sh[i] = load8(a.shift + at);
    }
  }
  TurnPlace place{};
  if (kRot != kRotNone) place = turn_place<kRot>(turns, kQkTokens * D / 4, s.l, a.rot_dim, 1.f);
  const T* zp = static_cast<const T*>(a.z) + (first * a.H + s.head) * D + 8 * s.l;
  const int64_t zrow = (int64_t)a.H * D;
  // z of this round and of the next
  Raw8<T> z0, z1;
  z0.zero();
  z1.zero();
  const int len = (int)(last - first);
  if (s.on && s.tsub < len) z0.load(zp + s.tsub * zrow);
  if (s.on && s.tsub + a.token_slots < len) z1.load(zp + (s.tsub + a.token_slots) * zrow);
  Walk w, w0;
  w0.start(first, a.T);
  w = w0;
  w.step(s.tsub, a.T);
  // every lane of a warp makes the same number of rounds (shuffles)
  for (int k0 = 0, fill = 0, fill0 = 0; k0 < len; k0 += a.token_slots) {
    if (kRot != kRotNone && k0 == fill) {
      const int n = min(a.tokens_per_fill, len - k0);
      __syncthreads();
      fill_turns<kRot, kFwdThreads>(turns, rate, a, first + k0, n, w0.t);
      w0.step(n, a.T);
      fill0 = fill;   // the table's first token; the next fill's
      fill += n;
      __syncthreads();
    }
    const int k = k0 + s.tsub;
    const bool on = s.on && k < len;
    P4 z = z0.get();
    z0 = z1;
    if (s.on && k + 2 * a.token_slots < len) z1.load(zp + (k + 2 * a.token_slots) * zrow);
    const float nrm = root<T>(row_sum<D>(dot8(z, z)));
    const float inv = reciprocal<T>(nrm < a.eps ? a.eps : nrm);   // (a NaN stays)
#pragma unroll
    for (int i = 0; i < 4; ++i) z.v[i] = fmul2(z.v[i], pack2(inv, inv));
    Turn turn;
    if (kRot != kRotNone) load_turn<kRot>(turn, turns, place, on ? k - fill0 : 0);
    const int64_t at = w.row(a.H, a.T, s.head) * D + 8 * s.l;
    w.step(a.token_slots, a.T);
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      P4 p;
#pragma unroll
      for (int i = 0; i < 4; ++i) p.v[i] = ffma2(sc[o].v[i], z.v[i], sh[o].v[i]);
      if (kRot != kRotNone && o < 2) turn8<kRot>(p, turn, s.src);
      if (on) store8(static_cast<T*>(a.out[o]) + at, p);
    }
  }
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}

// Each thread has its rows' pieces (z and the four output gradients) brought
// into its own slots of a ring in shared memory, kStages rounds ahead.  (In
// registers one round ahead was all there was room for beside the 64 running
// sums: 43 us at 2 x 5003 x 16 x 64 against 33, now 31.)
template <typename T, int D, int kRot>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks) qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  constexpr int S = kStages<T>, kParts = sizeof(T) / 2;   // 16-byte parts of a thread's 8 elements
  let_next_start();
  extern __shared__ uint4 smem[];
  uint4* ring = smem;                                          // [S][5][kParts][threads]
  float4* turns = reinterpret_cast<float4*>(smem + S * 5 * kParts * kBwdThreads);
  __shared__ double rate[kMaxRotPairs];
  if (kRot != kRotNone && threadIdx.x < a.rot_dim / 2) rate[threadIdx.x] = a.rate[threadIdx.x];
  const int64_t first = (int64_t)blockIdx.x * a.tokens_per_block;
  const int64_t last = min(first + a.tokens_per_block, a.n_tokens);
  const Slot s = my_slot<D>(a);
  P4 sc[4], ds[4], df[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) ds[i].zero(), df[i].zero(), sc[i].zero();
  if (s.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = load8(a.scale + ((int64_t)i * a.H + s.head) * D + 8 * s.l);
  }
  const int len = (int)(last - first);
  TurnPlace place{};
  if (kRot != kRotNone) place = turn_place<kRot>(turns, kQkTokens * D / 4, s.l, a.rot_dim, -1.f);
  const int64_t zrow = (int64_t)a.H * D;
  const int head = s.on ? s.head : 0;
  T* dz = static_cast<T*>(a.dz) + ((first + s.tsub) * a.H + head) * D + 8 * s.l;   // this round's
  const T* z_next = static_cast<const T*>(a.z) + ((first + s.tsub) * a.H + head) * D + 8 * s.l;
  Walk w, w0;
  w0.start(first, a.T);
  w = w0;
  w.step(s.tsub, a.T);
  int64_t at = w.row(a.H, a.T, head) * D + 8 * s.l;
  auto fetch = [&](int k, int stage) {   // in order of k
    uint4* to = ring + stage * 5 * kParts * kBwdThreads + threadIdx.x;
    const bool on = s.on && k < len;
    constexpr int kStep = 16 / sizeof(T);
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
#pragma unroll
      for (int o = 0; o < 4; ++o)
        copy16(to + (o * kParts + h) * kBwdThreads, static_cast<const T*>(a.dout[o]) + at + h * kStep, on);
      copy16(to + (4 * kParts + h) * kBwdThreads, z_next + h * kStep, on);
    }
    cp_async_commit();
    z_next += a.token_slots * zrow;
    w.t += a.token_slots;
    at += a.token_slots * D;
    if (w.t >= a.T) {
      w.step(0, a.T);
      at = w.row(a.H, a.T, head) * D + 8 * s.l;
    }
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(s.tsub + i * a.token_slots, i);
  int stage = 0;
  for (int k0 = 0, fill = 0, fill0 = 0; k0 < len; k0 += a.token_slots) {
    if (kRot != kRotNone && k0 == fill) {
      const int n = min(a.tokens_per_fill, len - k0);
      __syncthreads();
      fill_turns<kRot, kBwdThreads>(turns, rate, a, first + k0, n, w0.t);
      w0.step(n, a.T);
      fill0 = fill;   // the table's first token; the next fill's
      fill += n;
      __syncthreads();
    }
    const int k = k0 + s.tsub;
    const bool on = s.on && k < len;
    // the stage that the round before was read from is free again (only this thread reads it)
    fetch(k + (S - 1) * a.token_slots, stage == 0 ? S - 1 : stage - 1);
    cp_async_wait<S - 1>();
    P4 z, g, p[4];
    {
      const uint4* from = ring + stage * 5 * kParts * kBwdThreads + threadIdx.x;
      Raw8<T> raw;
#pragma unroll
      for (int o = 0; o < 5; ++o) {
        uint4* to = reinterpret_cast<uint4*>(&raw);
#pragma unroll
        for (int h = 0; h < kParts; ++h) to[h] = from[(o * kParts + h) * kBwdThreads];
        if (o < 4) p[o] = raw.get();
        else z = raw.get();
      }
    }
    if (++stage == S) stage = 0;
    g.zero();
    const float nrm = root<T>(row_sum<D>(dot8(z, z)));
    const float inv = reciprocal<T>(nrm < a.eps ? a.eps : nrm);   // (a NaN stays)
    const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) z.v[i] = fmul2(z.v[i], inv2);
    if (kRot != kRotNone) {
      Turn turn;
      load_turn<kRot>(turn, turns, place, on ? k - fill0 : 0);
      turn8<kRot>(p[0], turn, s.src);
      turn8<kRot>(p[1], turn, s.src);
    }
    // a row that is off is all zeros and adds nothing
#pragma unroll
    for (int o = 0; o < 4; ++o)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g.v[i] = ffma2(sc[o].v[i], p[o].v[i], g.v[i]);
        ds[o].v[i] = ffma2(p[o].v[i], z.v[i], ds[o].v[i]);
        df[o].v[i] = fadd2(df[o].v[i], p[o].v[i]);
      }
    float zg = row_sum<D>(dot8(z, g));
    if (nrm <= a.eps) zg = 0.f;   // z' = z / eps there: no term through the norm
#pragma unroll
    for (int i = 0; i < 4; ++i) g.v[i] = fmul2(ffma2(z.v[i], pack2(-zg, -zg), g.v[i]), inv2);
    if (on) store8(dz, g);
    dz += a.token_slots * zrow;
  }
  cp_async_wait<0>();
  // The token slots' sums into the first slot's, in order, through the ring.
  const int row_threads = a.heads_per_block * (D / 8), me = threadIdx.x % row_threads;
  ulonglong2* box = reinterpret_cast<ulonglong2*>(smem);   // [16][row_threads]
  for (int t = 1; t < a.token_slots; ++t) {
    __syncthreads();
    if (s.tsub == t)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const P4& v = i < 4 ? ds[i] : df[i - 4];
        box[(2 * i) * row_threads + me] = make_ulonglong2(v.v[0], v.v[1]);
        box[(2 * i + 1) * row_threads + me] = make_ulonglong2(v.v[2], v.v[3]);
      }
    __syncthreads();
    if (s.tsub == 0)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        P4& v = i < 4 ? ds[i] : df[i - 4];
        const ulonglong2 lo = box[(2 * i) * row_threads + me], hi = box[(2 * i + 1) * row_threads + me];
        v.v[0] = fadd2(v.v[0], lo.x);
        v.v[1] = fadd2(v.v[1], lo.y);
        v.v[2] = fadd2(v.v[2], hi.x);
        v.v[3] = fadd2(v.v[3], hi.y);
      }
  }
  if (s.on && s.tsub == 0) {
    float* out = a.part + (int64_t)blockIdx.x * 8 * zrow + (int64_t)s.head * D + 8 * s.l;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      store8(out + o * zrow, ds[o]);
      store8(out + (4 + o) * zrow, df[o]);
    }
  }
}

// dscale and dshift: the column sums of the blocks' partial sums, in a fixed
// order.
__global__ void __launch_bounds__(256) qk_bwd_sum_kernel(const float* part, int rows, int64_t cols, float* dscale,
                                                         float* dshift) {
  __shared__ float red[8][32];
  wait_for_previous();
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + cx;
  float acc = 0.f;
  for (int r = ry; r < rows; r += 8) acc += part[(int64_t)r * 2 * cols + col];
  red[ry][cx] = acc;
  __syncthreads();
  if (ry == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += red[i][cx];
    if (col < cols) dscale[col] = acc;
    else dshift[col - cols] = acc;
  }
}

struct Plan {
  int heads_per_block, head_blocks, token_slots;
  int64_t tokens_per_block, token_blocks;
};

// Heads are split over blocks so that a block's row slots hold whole heads, one
// token's or several tokens', and as few slots as possible stay empty; the tokens
// evenly over one wave of blocks.
Plan plan_of(int64_t n_tokens, int64_t H, int64_t d, int threads, int blocks_per_sm) {
  const int64_t slots = threads / (d / 8);
  Plan pl;
  double best = 0.0;
  const int64_t least = (H + slots - 1) / slots;
  for (int64_t n = least; n <= H && n < least + 16; ++n) {
    const int64_t heads = (H + n - 1) / n, tokens = slots / heads;
    const double used = (double)H * tokens / (double)(n * slots);
    if (used > best + 0.05) {   // more blocks fill the sine table more often
      best = used;
      pl.head_blocks = (int)((H + heads - 1) / heads);
      pl.heads_per_block = (int)heads;
      pl.token_slots = (int)tokens;
    }
  }
  int64_t blocks = (int64_t)blocks_per_sm * sm_count() / pl.head_blocks;
  if (blocks < 1) blocks = 1;
  const int64_t most = int64_t(1) << 30;   // tokens of a block are counted in 32 bits
  int64_t tpb = (n_tokens + blocks - 1) / blocks;
  if (tpb > most) tpb = most;
  pl.tokens_per_block = (tpb + pl.token_slots - 1) / pl.token_slots * pl.token_slots;
  pl.token_blocks = (n_tokens + pl.tokens_per_block - 1) / pl.tokens_per_block;
  return pl;
}

QkArgs args_of(const QkProblem& p, const Plan& pl) {
  QkArgs a;
  a.z = p.z;
  a.scale = p.scale;
  a.shift = p.shift;
  a.pos = p.pos;
  for (int i = 0; i < 4; ++i) {
    a.out[i] = p.out[i];
    a.dout[i] = p.dout[i];
  }
  a.dz = p.dz;
  a.part = static_cast<float*>(p.ws);
  a.n_tokens = p.B * p.T;
  a.T = p.T;
  a.H = (int)p.H;
  a.heads_per_block = pl.heads_per_block;
  a.token_slots = pl.token_slots;
  a.tokens_per_block = (int)pl.tokens_per_block;
  a.tokens_per_fill = kQkTokens / pl.token_slots * pl.token_slots;
  a.eps = p.eps;
  a.pos0 = p.pos0;
  a.rot_dim = p.rot_dim;
  for (int i = 0; i < kMaxRotPairs; ++i) a.rate[i] = p.rate[i];
  return a;
}

template <typename T, int D>
cudaError_t run(const QkProblem& p, const Plan& pl, bool backward, cudaStream_t st) {
  const QkArgs a = args_of(p, pl);
  const dim3 grid((unsigned)pl.token_blocks, (unsigned)pl.head_blocks);
  const int rot = p.rot_dim == 0 ? kRotNone : p.interleaved ? kRotInterleaved : kRotHalves;
  if (!backward) {
    if (rot == kRotNone) qk_kernel<T, D, kRotNone><<<grid, kFwdThreads, 0, st>>>(a);
    else if (rot == kRotHalves) qk_kernel<T, D, kRotHalves><<<grid, kFwdThreads, 0, st>>>(a);
    else qk_kernel<T, D, kRotInterleaved><<<grid, kFwdThreads, 0, st>>>(a);
  } else {
    const auto kern = rot == kRotNone     ? qk_bwd_kernel<T, D, kRotNone>
                      : rot == kRotHalves ? qk_bwd_kernel<T, D, kRotHalves>
                                          : qk_bwd_kernel<T, D, kRotInterleaved>;
    const int smem = kStages<T> * 5 * (int)sizeof(T) / 2 * kBwdThreads * 16 + (kQkTokens * D / 4 + 1) * 16;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    kern<<<grid, kBwdThreads, smem, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t run(const QkProblem& p, const Plan& pl, bool backward, cudaStream_t st) {
  if (p.dtype == kBF16)
    return p.d == 128 ? run<__nv_bfloat16, 128>(p, pl, backward, st) : run<__nv_bfloat16, 64>(p, pl, backward, st);
  return p.d == 128 ? run<float, 128>(p, pl, backward, st) : run<float, 64>(p, pl, backward, st);
}

Plan bwd_plan(int64_t B, int64_t T, int64_t H, int64_t d) { return plan_of(B * T, H, d, kBwdThreads, kBwdBlocks); }

}  // namespace

size_t qk_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t d) {
  return sizeof(float) * (size_t)bwd_plan(B, T, H, d).token_blocks * 8 * H * d;
}

cudaError_t launch_qk(const QkProblem& p, cudaStream_t st) {
  return run(p, plan_of(p.B * p.T, p.H, p.d, kFwdThreads, kFwdBlocks), false, st);
}

cudaError_t launch_qk_bwd(const QkProblem& p, cudaStream_t st) {
  const Plan pl = bwd_plan(p.B, p.T, p.H, p.d);
  if (cudaError_t e = run(p, pl, true, st)) return e;
  const int64_t cols = 4 * p.H * p.d;
  return launch_chained(qk_bwd_sum_kernel, dim3((unsigned)(2 * cols / 32)), 256, 0, 0, true, st,
                        static_cast<const float*>(p.ws), (int)pl.token_blocks, cols, p.dscale, p.dshift);
}

}  // namespace gecko
