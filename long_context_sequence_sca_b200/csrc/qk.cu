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
#include "common.cuh"
#include "gecko_internal.h"

namespace gecko {
namespace {

constexpr int kFwdThreads = 256, kBwdThreads = 128;
// Resident blocks per SM, by the registers of their prefetched rows.
constexpr int kFwdBlocks = 2;
constexpr int bwd_blocks(size_t elem) { return elem == 2 ? 3 : 2; }
constexpr int kQkTokens = 32;                          // tokens per fill of the sine table
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

struct F8 {
  float v[8];
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
  __device__ __forceinline__ F8 get() const { return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ F8 get() const {
    F8 r;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = __uint_as_float(w[i] << 16);
      r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return r;
  }
};
__device__ __forceinline__ F8 load8(const float* p) {
  Raw8<float> r;
  r.load(p);
  return r.get();
}
__device__ __forceinline__ void store8(float* p, const F8& f) {
  *reinterpret_cast<float4*>(p) = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
                                            pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7]));
}

// The sine table: (cos, sin) of every rotated pair of the fill's tokens.  A lane
// reads kPer pairs of a row, 16 bytes (two pairs) at a time; the 16-byte pieces
// of a row are ordered so that the lanes of one read are consecutive.
template <int kRot>
constexpr int kPer = kRot == kRotInterleaved ? 4 : 8;

template <int kRot>
__device__ __forceinline__ int turn_slot(int pair, int pairs) {
  constexpr int kPieces = kPer<kRot> / 2;   // pieces per lane
  const int piece = pair >> 1;
  return ((piece % kPieces) * (pairs / kPer<kRot>) + piece / kPieces) * 2 + (pair & 1);
}

template <int kRot, int kThreads>
__device__ __forceinline__ void fill_turns(float2* turns, const double* rate, const QkArgs& a, int64_t n0, int n,
                                           uint32_t t0) {
  const int pairs = a.rot_dim / 2;
  for (int i = threadIdx.x; i < n * pairs; i += kThreads) {
    const int k = i / pairs, pair = i - k * pairs;
    const int64_t pos = a.pos ? a.pos[n0 + k] : a.pos0 + (t0 + k) % (uint32_t)a.T;
    const double rev = (double)pos * rate[pair];
    float s, c;
    sincospif((float)(2.0 * (rev - rint(rev))), &s, &c);
    turns[k * pairs + turn_slot<kRot>(pair, pairs)] = make_float2(c, s);
  }
}

struct Turn8 {
  float2 cs[8];
};

// This lane's (cos, sin) of one row: of its pairs (interleaved), or of the
// pairs that its 8 features belong to (halves; the two halves share them).
template <int kRot>
__device__ __forceinline__ void load_turn(Turn8& r, const float2* row, int l, int rot_dim) {
  const int lanes = rot_dim / 16;   // halves: lanes per half
  const int readers = rot_dim / 2 / kPer<kRot>;
  const int at = kRot == kRotHalves && l >= lanes ? l - lanes : l;
#pragma unroll
  for (int i = 0; i < kPer<kRot> / 2; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(row + (i * readers + (at < readers ? at : 0)) * 2);
    r.cs[2 * i] = make_float2(v.x, v.y);
    r.cs[2 * i + 1] = make_float2(v.z, v.w);
  }
}

// The 8 features 8 l .. 8 l + 7 of a row turned (sign -1: turned back).  src: the
// lane that holds the other half of this lane's pairs (halves), which every
// lane of the warp must pass here.
template <int kRot>
__device__ __forceinline__ void turn8(F8& p, const Turn8& r, int l, int rot_dim, int src, float sign) {
  if (kRot == kRotInterleaved) {
    if (8 * l < rot_dim) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = p.v[2 * i], b = p.v[2 * i + 1], s = sign * r.cs[i].y;
        p.v[2 * i] = a * r.cs[i].x - b * s;
        p.v[2 * i + 1] = b * r.cs[i].x + a * s;
      }
    }
  } else if (kRot == kRotHalves) {
    const int half = rot_dim / 16;   // lanes per half
    const float sg = l >= half ? sign : -sign;
    const bool in = l < 2 * half;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, p.v[i], src);
      const float t = p.v[i] * r.cs[i].x + sg * r.cs[i].y * o;
      if (in) p.v[i] = t;
    }
  }
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
  __shared__ __align__(16) float2 turns[kRot == kRotNone ? 1 : kQkTokens * D / 2];
  __shared__ double rate[kMaxRotPairs];   // the parameter bank would serialise the lanes' reads
  if (kRot != kRotNone && threadIdx.x < a.rot_dim / 2) rate[threadIdx.x] = a.rate[threadIdx.x];
  const int64_t first = (int64_t)blockIdx.x * a.tokens_per_block;
  const int64_t last = min(first + a.tokens_per_block, a.n_tokens);
  const Slot s = my_slot<D>(a);
  F8 sc[4], sh[4];
  if (s.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = ((int64_t)i * a.H + s.head) * D + 8 * s.l;
      sc[i] = load8(a.scale + at);
      sh[i] = load8(a.shift + at);
    }
  }
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
  for (int k0 = 0, fill = 0; k0 < len; k0 += a.token_slots) {
    if (kRot != kRotNone && k0 == fill) {
      const int n = min(a.tokens_per_fill, len - k0);
      __syncthreads();
      fill_turns<kRot, kFwdThreads>(turns, rate, a, first + k0, n, w0.t);
      w0.step(n, a.T);
      fill += n;
      __syncthreads();
    }
    const int k = k0 + s.tsub;
    const bool on = s.on && k < len;
    F8 z = z0.get();
    z0 = z1;
    if (s.on && k + 2 * a.token_slots < len) z1.load(zp + (k + 2 * a.token_slots) * zrow);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(z.v[i], z.v[i], ss);
    const float nrm = sqrtf(row_sum<D>(ss));
    const float inv = 1.f / (nrm < a.eps ? a.eps : nrm);
#pragma unroll
    for (int i = 0; i < 8; ++i) z.v[i] *= inv;
    Turn8 turn;
    if (kRot != kRotNone)
      load_turn<kRot>(turn, turns + (on ? k % a.tokens_per_fill : 0) * (a.rot_dim / 2), s.l, a.rot_dim);
    const int64_t at = w.row(a.H, a.T, s.head) * D + 8 * s.l;
    w.step(a.token_slots, a.T);
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      F8 p;
#pragma unroll
      for (int i = 0; i < 8; ++i) p.v[i] = fmaf(sc[o].v[i], z.v[i], sh[o].v[i]);
      if (kRot != kRotNone && o < 2) turn8<kRot>(p, turn, s.l, a.rot_dim, s.src, 1.f);
      if (on) store8(static_cast<T*>(a.out[o]) + at, p);
    }
  }
}

template <typename T, int D, int kRot>
__global__ void __launch_bounds__(kBwdThreads, bwd_blocks(sizeof(T))) qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  __shared__ __align__(16) float2 turns[kRot == kRotNone ? 1 : kQkTokens * D / 2];
  __shared__ double rate[kMaxRotPairs];
  if (kRot != kRotNone && threadIdx.x < a.rot_dim / 2) rate[threadIdx.x] = a.rate[threadIdx.x];
  const int64_t first = (int64_t)blockIdx.x * a.tokens_per_block;
  const int64_t last = min(first + a.tokens_per_block, a.n_tokens);
  const Slot s = my_slot<D>(a);
  F8 sc[4], ds[4] = {}, df[4] = {};
  if (s.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = load8(a.scale + ((int64_t)i * a.H + s.head) * D + 8 * s.l);
  }
  const int len = (int)(last - first);
  const int64_t zrow = (int64_t)a.H * D, z_at = (first * a.H + s.head) * D + 8 * s.l;
  Walk w, w0;
  w0.start(first, a.T);
  w = w0;
  w.step(s.tsub, a.T);
  // this round's z and output gradients; the next round's are loaded before
  // these are worked on
  Raw8<T> raw[5];
  auto fetch = [&](int k) {
    if (s.on && k < len) {
      const int64_t at = w.row(a.H, a.T, s.head) * D + 8 * s.l;
      raw[4].load(static_cast<const T*>(a.z) + z_at + k * zrow);
#pragma unroll
      for (int o = 0; o < 4; ++o) raw[o].load(static_cast<const T*>(a.dout[o]) + at);
    } else {
#pragma unroll
      for (int o = 0; o < 5; ++o) raw[o].zero();
    }
    w.step(a.token_slots, a.T);
  };
  fetch(s.tsub);
  for (int k0 = 0, fill = 0; k0 < len; k0 += a.token_slots) {
    if (kRot != kRotNone && k0 == fill) {
      const int n = min(a.tokens_per_fill, len - k0);
      __syncthreads();
      fill_turns<kRot, kBwdThreads>(turns, rate, a, first + k0, n, w0.t);
      w0.step(n, a.T);
      fill += n;
      __syncthreads();
    }
    const int k = k0 + s.tsub;
    const bool on = s.on && k < len;
    F8 z = raw[4].get(), g = {}, p[4];
#pragma unroll
    for (int o = 0; o < 4; ++o) p[o] = raw[o].get();
    fetch(k + a.token_slots);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(z.v[i], z.v[i], ss);
    const float nrm = sqrtf(row_sum<D>(ss));
    const float inv = 1.f / (nrm < a.eps ? a.eps : nrm);
#pragma unroll
    for (int i = 0; i < 8; ++i) z.v[i] *= inv;
    if (kRot != kRotNone) {
      Turn8 turn;
      load_turn<kRot>(turn, turns + (on ? k % a.tokens_per_fill : 0) * (a.rot_dim / 2), s.l, a.rot_dim);
      turn8<kRot>(p[0], turn, s.l, a.rot_dim, s.src, -1.f);
      turn8<kRot>(p[1], turn, s.l, a.rot_dim, s.src, -1.f);
    }
    // a row that is off is all zeros and adds nothing
#pragma unroll
    for (int o = 0; o < 4; ++o)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g.v[i] = fmaf(sc[o].v[i], p[o].v[i], g.v[i]);
        ds[o].v[i] = fmaf(p[o].v[i], z.v[i], ds[o].v[i]);
        df[o].v[i] += p[o].v[i];
      }
    float zg = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) zg = fmaf(z.v[i], g.v[i], zg);
    zg = row_sum<D>(zg);
    if (nrm <= a.eps) zg = 0.f;   // z' = z / eps there: no term through the norm
#pragma unroll
    for (int i = 0; i < 8; ++i) g.v[i] = (g.v[i] - z.v[i] * zg) * inv;
    if (on) store8(static_cast<T*>(a.dz) + z_at + k * zrow, g);
  }
  if (s.on) {
    const int64_t hd = (int64_t)a.H * D;
    float* out = a.part + ((int64_t)blockIdx.x * a.token_slots + s.tsub) * 8 * hd + (int64_t)s.head * D + 8 * s.l;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      store8(out + o * hd, ds[o]);
      store8(out + (4 + o) * hd, df[o]);
    }
  }
}

// dscale and dshift: the column sums of the blocks' partial sums, in a fixed
// order.
__global__ void __launch_bounds__(256) qk_bwd_sum_kernel(const float* part, int rows, int64_t cols, float* dscale,
                                                         float* dshift) {
  __shared__ float red[8][32];
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

// Heads are split over blocks so that a block's row slots hold whole heads, the
// tokens evenly over one wave of blocks.
Plan plan_of(int64_t n_tokens, int64_t H, int64_t d, int threads, int blocks_per_sm) {
  const int64_t slots = threads / (d / 8);
  Plan pl;
  pl.head_blocks = (int)((H + slots - 1) / slots);
  pl.heads_per_block = (int)((H + pl.head_blocks - 1) / pl.head_blocks);
  pl.token_slots = (int)(slots / pl.heads_per_block);
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
void run(const QkProblem& p, const Plan& pl, bool backward, cudaStream_t st) {
  const QkArgs a = args_of(p, pl);
  const dim3 grid((unsigned)pl.token_blocks, (unsigned)pl.head_blocks);
  const int rot = p.rot_dim == 0 ? kRotNone : p.interleaved ? kRotInterleaved : kRotHalves;
  if (!backward) {
    if (rot == kRotNone) qk_kernel<T, D, kRotNone><<<grid, kFwdThreads, 0, st>>>(a);
    else if (rot == kRotHalves) qk_kernel<T, D, kRotHalves><<<grid, kFwdThreads, 0, st>>>(a);
    else qk_kernel<T, D, kRotInterleaved><<<grid, kFwdThreads, 0, st>>>(a);
  } else {
    if (rot == kRotNone) qk_bwd_kernel<T, D, kRotNone><<<grid, kBwdThreads, 0, st>>>(a);
    else if (rot == kRotHalves) qk_bwd_kernel<T, D, kRotHalves><<<grid, kBwdThreads, 0, st>>>(a);
    else qk_bwd_kernel<T, D, kRotInterleaved><<<grid, kBwdThreads, 0, st>>>(a);
  }
}

void run(const QkProblem& p, const Plan& pl, bool backward, cudaStream_t st) {
  if (p.dtype == kBF16) {
    if (p.d == 128) run<__nv_bfloat16, 128>(p, pl, backward, st);
    else run<__nv_bfloat16, 64>(p, pl, backward, st);
  } else {
    if (p.d == 128) run<float, 128>(p, pl, backward, st);
    else run<float, 64>(p, pl, backward, st);
  }
}

Plan bwd_plan(int64_t B, int64_t T, int64_t H, int64_t d, int dtype) {
  return plan_of(B * T, H, d, kBwdThreads, bwd_blocks(dtype == kBF16 ? 2 : 4));
}

}  // namespace

size_t qk_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t d, int dtype) {
  const Plan pl = bwd_plan(B, T, H, d, dtype);
  return sizeof(float) * (size_t)(pl.token_blocks * pl.token_slots) * 8 * H * d;
}

cudaError_t launch_qk(const QkProblem& p, cudaStream_t st) {
  run(p, plan_of(p.B * p.T, p.H, p.d, kFwdThreads, kFwdBlocks), false, st);
  return cudaGetLastError();
}

cudaError_t launch_qk_bwd(const QkProblem& p, cudaStream_t st) {
  const Plan pl = bwd_plan(p.B, p.T, p.H, p.d, p.dtype);
  run(p, pl, true, st);
  const int64_t cols = 4 * p.H * p.d;
  qk_bwd_sum_kernel<<<(unsigned)(2 * cols / 32), 256, 0, st>>>(static_cast<const float*>(p.ws),
                                                               (int)(pl.token_blocks * pl.token_slots), cols,
                                                               p.dscale, p.dshift);
  return cudaGetLastError();
}

}  // namespace gecko
