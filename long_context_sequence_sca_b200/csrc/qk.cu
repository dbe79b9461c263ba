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

constexpr int kQkThreads = 256;
constexpr int kQkTokens = 32;       // most tokens per block (rows of the sine table)
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
  float eps;
  int64_t pos0;
  int rot_dim;
  double rate[kMaxRotPairs];
};

struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 load8(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ F8 load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  F8 r;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  return r;
}
__device__ __forceinline__ void store8(float* p, const F8& f) {
  *reinterpret_cast<float4*>(p) = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const F8& f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
                                            pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7]));
}

// (cos, sin) of every rotated pair of the block's tokens.
__device__ __forceinline__ void fill_turns(float2* turns, const QkArgs& a, int64_t n0, int n) {
  __shared__ double rate[kMaxRotPairs];   // the parameter bank would serialise the lanes' reads
  const int pairs = a.rot_dim / 2;
  if (threadIdx.x < pairs) rate[threadIdx.x] = a.rate[threadIdx.x];
  __syncthreads();
  for (int i = threadIdx.x; i < n * pairs; i += kQkThreads) {
    const int64_t tok = n0 + i / pairs;
    const int64_t pos = a.pos ? a.pos[tok] : a.pos0 + tok % a.T;
    const double rev = (double)pos * rate[i % pairs];
    float s, c;
    sincospif((float)(2.0 * (rev - rint(rev))), &s, &c);
    turns[i] = make_float2(c, s);
  }
}

// The 8 elements 8 l .. 8 l + 7 of a row turned by the row's angles
// (sign -1: turned back).  src: the lane that holds the other half of this
// lane's pairs (halves), which every lane of the warp must pass here.
template <int kRot>
__device__ __forceinline__ void turn8(F8& p, const float2* row, int l, int rot_dim, int src, float sign) {
  if (kRot == kRotInterleaved) {
    if (8 * l < rot_dim) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 cs = row[4 * l + i];
        const float a = p.v[2 * i], b = p.v[2 * i + 1], s = sign * cs.y;
        p.v[2 * i] = a * cs.x - b * s;
        p.v[2 * i + 1] = b * cs.x + a * s;
      }
    }
  } else if (kRot == kRotHalves) {
    const int half = rot_dim / 16;   // lanes per half
    const bool upper = l >= half;
    F8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = __shfl_sync(0xffffffffu, p.v[i], src);
    if (l < 2 * half) {
      const float2* r = row + 8 * (upper ? l - half : l);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 cs = r[i];
        p.v[i] = p.v[i] * cs.x + (upper ? sign : -sign) * cs.y * o.v[i];
      }
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

template <typename T, int D, int kRot>
__global__ void __launch_bounds__(kQkThreads) qk_kernel(const __grid_constant__ QkArgs a) {
  __shared__ float2 turns[kRot == kRotNone ? 1 : kQkTokens * D / 2];
  const int64_t n0 = (int64_t)blockIdx.x * a.tokens_per_block;
  const int n = (int)min((int64_t)a.tokens_per_block, a.n_tokens - n0);
  if (kRot != kRotNone) {
    fill_turns(turns, a, n0, n);
    __syncthreads();
  }
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
  // every lane of a warp makes the same number of rounds (shuffles)
  for (int r = 0; r < n; r += a.token_slots) {
    const int k = r + s.tsub;
    const bool on = s.on && k < n;
    const int64_t tok = n0 + k;
    F8 z = {};
    if (on) z = load8(static_cast<const T*>(a.z) + (tok * a.H + s.head) * D + 8 * s.l);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(z.v[i], z.v[i], ss);
    const float nrm = sqrtf(row_sum<D>(ss));
    const float inv = 1.f / (nrm < a.eps ? a.eps : nrm);
#pragma unroll
    for (int i = 0; i < 8; ++i) z.v[i] *= inv;
    const int64_t b = tok / a.T, t = tok % a.T;
    const int64_t at = ((b * a.H + s.head) * a.T + t) * D + 8 * s.l;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      F8 p;
#pragma unroll
      for (int i = 0; i < 8; ++i) p.v[i] = fmaf(sc[o].v[i], z.v[i], sh[o].v[i]);
      if (kRot != kRotNone && o < 2) turn8<kRot>(p, turns + (on ? k : 0) * (a.rot_dim / 2), s.l, a.rot_dim, s.src, 1.f);
      if (on) store8(static_cast<T*>(a.out[o]) + at, p);
    }
  }
}

template <typename T, int D, int kRot>
__global__ void __launch_bounds__(kQkThreads) qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  __shared__ float2 turns[kRot == kRotNone ? 1 : kQkTokens * D / 2];
  const int64_t first = (int64_t)blockIdx.x * a.tokens_per_block;
  const int64_t last = min(first + a.tokens_per_block, a.n_tokens);
  const Slot s = my_slot<D>(a);
  F8 sc[4], ds[4] = {}, df[4] = {};
  if (s.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = load8(a.scale + ((int64_t)i * a.H + s.head) * D + 8 * s.l);
  }
  for (int64_t n0 = first; n0 < last; n0 += kQkTokens) {
    const int n = (int)min((int64_t)kQkTokens, last - n0);
    if (kRot != kRotNone) {
      __syncthreads();
      fill_turns(turns, a, n0, n);
      __syncthreads();
    }
    for (int r = 0; r < n; r += a.token_slots) {
      const int k = r + s.tsub;
      const bool on = s.on && k < n;
      const int64_t tok = n0 + k;
      const int64_t b = tok / a.T, t = tok % a.T;
      const int64_t at = ((b * a.H + s.head) * a.T + t) * D + 8 * s.l;
      const int64_t zat = (tok * a.H + s.head) * D + 8 * s.l;
      F8 z = {}, g = {};
      if (on) z = load8(static_cast<const T*>(a.z) + zat);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(z.v[i], z.v[i], ss);
      const float nrm = sqrtf(row_sum<D>(ss));
      const float inv = 1.f / (nrm < a.eps ? a.eps : nrm);
#pragma unroll
      for (int i = 0; i < 8; ++i) z.v[i] *= inv;
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        F8 p = {};
        if (on) p = load8(static_cast<const T*>(a.dout[o]) + at);
        if (kRot != kRotNone && o < 2)
          turn8<kRot>(p, turns + (on ? k : 0) * (a.rot_dim / 2), s.l, a.rot_dim, s.src, -1.f);
        if (on) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            g.v[i] = fmaf(sc[o].v[i], p.v[i], g.v[i]);
            ds[o].v[i] = fmaf(p.v[i], z.v[i], ds[o].v[i]);
            df[o].v[i] += p.v[i];
          }
        }
      }
      float zg = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) zg = fmaf(z.v[i], g.v[i], zg);
      zg = row_sum<D>(zg);
      if (nrm <= a.eps) zg = 0.f;   // z' = z / eps there: no term through the norm
#pragma unroll
      for (int i = 0; i < 8; ++i) g.v[i] = (g.v[i] - z.v[i] * zg) * inv;
      if (on) store8(static_cast<T*>(a.dz) + zat, g);
    }
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

// Heads are split over blocks so that a block's row slots hold whole heads;
// the tokens over enough blocks to give every SM two.
Plan plan_of(int64_t n_tokens, int64_t H, int64_t d, int64_t max_tokens) {
  const int64_t slots = kQkThreads / (d / 8);
  Plan pl;
  pl.head_blocks = (int)((H + slots - 1) / slots);
  pl.heads_per_block = (int)((H + pl.head_blocks - 1) / pl.head_blocks);
  pl.token_slots = (int)(slots / pl.heads_per_block);
  const int64_t want = 2 * 148;
  int64_t tpb = (n_tokens * pl.head_blocks + want - 1) / want;
  tpb = (tpb + pl.token_slots - 1) / pl.token_slots * pl.token_slots;
  pl.tokens_per_block = tpb > max_tokens ? max_tokens : tpb;
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
    if (rot == kRotNone) qk_kernel<T, D, kRotNone><<<grid, kQkThreads, 0, st>>>(a);
    else if (rot == kRotHalves) qk_kernel<T, D, kRotHalves><<<grid, kQkThreads, 0, st>>>(a);
    else qk_kernel<T, D, kRotInterleaved><<<grid, kQkThreads, 0, st>>>(a);
  } else {
    if (rot == kRotNone) qk_bwd_kernel<T, D, kRotNone><<<grid, kQkThreads, 0, st>>>(a);
    else if (rot == kRotHalves) qk_bwd_kernel<T, D, kRotHalves><<<grid, kQkThreads, 0, st>>>(a);
    else qk_bwd_kernel<T, D, kRotInterleaved><<<grid, kQkThreads, 0, st>>>(a);
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

Plan bwd_plan(int64_t B, int64_t T, int64_t H, int64_t d) { return plan_of(B * T, H, d, int64_t(1) << 30); }

}  // namespace

size_t qk_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t d) {
  const Plan pl = bwd_plan(B, T, H, d);
  return sizeof(float) * (size_t)(pl.token_blocks * pl.token_slots) * 8 * H * d;
}

cudaError_t launch_qk(const QkProblem& p, cudaStream_t st) {
  run(p, plan_of(p.B * p.T, p.H, p.d, kQkTokens), false, st);
  return cudaGetLastError();
}

cudaError_t launch_qk_bwd(const QkProblem& p, cudaStream_t st) {
  const Plan pl = bwd_plan(p.B, p.T, p.H, p.d);
  run(p, pl, true, st);
  const int64_t cols = 4 * p.H * p.d;
  qk_bwd_sum_kernel<<<(unsigned)(2 * cols / 32), 256, 0, st>>>(static_cast<const float*>(p.ws),
                                                               (int)(pl.token_blocks * pl.token_slots), cols,
                                                               p.dscale, p.dshift);
  return cudaGetLastError();
}

}  // namespace gecko
