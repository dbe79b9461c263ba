// Projection y = f(x w^T + bias) + residual and its gradients:
//   u = x w^T + bias,  du = dy (.) f'(u),
//   dx = du w,  dw = du^T x,  db = column sums of du.
// The products run on the tensor cores (linear_tc.cu); here are the pass that
// forms du and db, the pass that splits fp32 operands into bf16 planes, and
// CUDA-core products for GECKO_KERNELS=simt, a second implementation to check
// against.
#include <cstdlib>
#include <cstring>

#include "common.cuh"
#include "gecko_internal.h"
#include "linear.cuh"

namespace gecko {
namespace {

// ------------------------------------------------------ CUDA-core product --

// C[m, n] = sum_k A(m, k) B(n, k) with A(m, k) = A[m am + k ak] and likewise
// B: 64 x 64 tiles, 4 x 4 results per thread, fp32 FMA.
constexpr int kSimtTile = 64, kSimtK = 16;

template <typename T, class Epilogue>
__global__ void __launch_bounds__(256) simt_gemm_kernel(const T* A, int64_t am, int64_t ak, const T* B, int64_t bn,
                                                        int64_t bk, int64_t M, int64_t N, int64_t K, Epilogue ep) {
  __shared__ float As[kSimtK][kSimtTile + 4], Bs[kSimtK][kSimtTile + 4];
  const int64_t m0 = (int64_t)blockIdx.x * kSimtTile, n0 = (int64_t)blockIdx.y * kSimtTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += kSimtK) {
    for (int i = threadIdx.x; i < kSimtTile * kSimtK; i += 256) {
      // consecutive threads along the operand's contiguous dimension
      const int ra = ak == 1 ? i / kSimtK : i % kSimtTile, ka = ak == 1 ? i % kSimtK : i / kSimtTile;
      As[ka][ra] = m0 + ra < M && k0 + ka < K ? to_f32(A[(m0 + ra) * am + (k0 + ka) * ak]) : 0.f;
      const int rb = bk == 1 ? i / kSimtK : i % kSimtTile, kb = bk == 1 ? i % kSimtK : i / kSimtTile;
      Bs[kb][rb] = n0 + rb < N && k0 + kb < K ? to_f32(B[(n0 + rb) * bn + (k0 + kb) * bk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSimtK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = As[k][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = Bs[k][tx * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) ep(m, n, acc[i][j]);
    }
}

// u -> y (and the kept u)
template <typename T>
struct ForwardOut {
  const float* bias;
  const T* residual;
  T* y;
  float* pre;
  OutLayout lay;
  int act;
  __device__ void operator()(int64_t m, int64_t n, float u) const {
    if (bias) u += bias[n];
    const int64_t at = lay.at(m, n);
    if (pre) pre[at] = u;
    float v = activate<T>(u, act);
    if (residual) v += to_f32(residual[at]);
    y[at] = from_f32<T>(v);
  }
};

template <typename T>
struct PlainOut {
  T* c;
  int64_t ld;
  __device__ void operator()(int64_t m, int64_t n, float v) const { c[m * ld + n] = from_f32<T>(v); }
};

template <typename T, class Epilogue>
void simt_gemm(const void* A, int64_t am, int64_t ak, const void* B, int64_t bn, int64_t bk, int64_t M, int64_t N,
               int64_t K, const Epilogue& ep, cudaStream_t st) {
  const dim3 grid((unsigned)((M + kSimtTile - 1) / kSimtTile), (unsigned)((N + kSimtTile - 1) / kSimtTile));
  simt_gemm_kernel<T, Epilogue><<<grid, 256, 0, st>>>(static_cast<const T*>(A), am, ak, static_cast<const T*>(B), bn,
                                                      bk, M, N, K, ep);
}

// ------------------------------------------------- few rows, fp32, forward --

// Up to 16 rows of fp32: the weights' bytes are all there is to it, and splitting
// them into planes would move them three times (8 x 4096 x 4096: 64 us that way,
// 22.7 this way, 10 at HBM's rate).  A warp takes two columns of y (rows of w),
// 16 bytes of each per lane and load; x comes by 512 of the depth through shared
// memory, the next piece under way while one is used.
constexpr int kRowsMost = 16, kRowsDepth = 512, kRowsWarps = 8, kRowsCols = 2 * kRowsWarps;

template <int kM>
__global__ void __launch_bounds__(32 * kRowsWarps) linear_rows_kernel(const float* x, const float* w, int M, int64_t N,
                                                                      int64_t K, ForwardOut<float> ep) {
  extern __shared__ float4 xs[];   // [2][kM][kRowsDepth / 4]
  constexpr int kQ = kRowsDepth / 4;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int64_t n0 = (int64_t)blockIdx.x * kRowsCols + 2 * warp;
  auto bring = [&](int64_t k0, int buf) {
    for (int i = threadIdx.x; i < kM * kQ; i += 32 * kRowsWarps) {
      const int m = i / kQ;
      const int64_t k = k0 + (i - m * kQ) * 4;
      const bool on = m < M && k < K;
      copy16(xs + buf * kM * kQ + i, x + (on ? m * K + k : 0), on);
    }
    cp_async_commit();
  };
  float acc[2][kM] = {};
  bring(0, 0);
  int buf = 0;
  for (int64_t k0 = 0; k0 < K; k0 += kRowsDepth, buf ^= 1) {
    float4 v[2][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t k = k0 + j * 128 + lane * 4;
#pragma unroll
      for (int c = 0; c < 2; ++c)
        v[c][j] = n0 + c < N && k < K ? *reinterpret_cast<const float4*>(w + (n0 + c) * K + k)
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    bring(k0 + kRowsDepth, buf ^ 1);   // (beyond K: zeros)
    cp_async_wait<1>();
    __syncthreads();
    const float4* at = xs + buf * kM * kQ + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const float4 a = at[m * kQ + j * 32];
#pragma unroll
        for (int c = 0; c < 2; ++c)
          acc[c][m] = fmaf(a.x, v[c][j].x, fmaf(a.y, v[c][j].y, fmaf(a.z, v[c][j].z, fmaf(a.w, v[c][j].w, acc[c][m]))));
      }
    __syncthreads();   // the piece after next overwrites this one
  }
  cp_async_wait<0>();
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int m = 0; m < kM; ++m) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[c][m] += __shfl_xor_sync(0xffffffffu, acc[c][m], o);
      if (lane == (c * kM + m) % 32 && m < M && n0 + c < N) ep(m, n0 + c, acc[c][m]);
    }
}

template <int kM>
cudaError_t launch_rows(const LinearProblem& p, const ForwardOut<float>& ep, cudaStream_t st) {
  constexpr int smem = 2 * kM * kRowsDepth * 4;
  if (cudaError_t e = cudaFuncSetAttribute(linear_rows_kernel<kM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))
    return e;
  linear_rows_kernel<kM><<<(unsigned)((p.N + kRowsCols - 1) / kRowsCols), 32 * kRowsWarps, smem, st>>>(
      static_cast<const float*>(p.x), static_cast<const float*>(p.w), (int)p.M(), p.N, p.K, ep);
  return cudaGetLastError();
}

// ----------------------------------------------------- gradient of u, db --

constexpr int kDuCols = 256;     // columns per block: 32 threads x 8
constexpr int kDuRowsPar = 8;    // rows per round of a block
// Blocks per SM.  With four rounds of loads in flight per thread the compiler
// spilled (69 us for 8192 x 4096 SiLU with db; two rounds and three blocks 37,
// one round and four blocks 37).
constexpr int kDuBlocks = 4;
constexpr int kDuOneBlock = 128;    // up to this many rows, one block of rows and no second kernel for db

// du = dy f'(u), [M, N] with rows `pitch` apart in the tensors' type (for bf16 one rounding, to
// the operand type of the two products that follow) or as bf16 planes; the
// column sums of the unrounded values go to part [gridDim.y, N].
template <typename T, int kAct, bool kPlanes>
__global__ void __launch_bounds__(256, kDuBlocks) linear_du_kernel(const T* dy, const float* pre, void* du, float* part,
                                                                   OutLayout lay, int64_t M, int64_t N, int64_t rows,
                                                                   int64_t pitch) {
  __shared__ float red[kDuRowsPar][kDuCols];
  let_next_start();
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t n = (int64_t)blockIdx.x * kDuCols + cx * 8;
  const int64_t m1 = min(M, ((int64_t)blockIdx.y + 1) * rows);
  float acc[8] = {};
  if (n < N) {
    const int64_t col = lay.col((int)n);
    int64_t m = (int64_t)blockIdx.y * rows + ry;
    // where row m begins; the next row of this thread is kDuRowsPar on
    int64_t at = lay.row(m) + col;
    uint32_t t = lay.H ? (uint32_t)m % lay.T : 0;
    const int64_t step = (int64_t)kDuRowsPar * (lay.H ? lay.hd : N);
    auto next = [&](int64_t to) {
      at += step;
      t += kDuRowsPar;
      if (lay.H && t >= lay.T) {
        t = (uint32_t)to % lay.T;
        at = lay.row(to) + col;
      }
    };
    for (; m < m1; m += kDuRowsPar) {
      Vec8<T> g;
      Vec8<float> u;
      g.load(dy + at);
      if (kAct != kActNone) u.load(pre + at);
      next(m + kDuRowsPar);
      float v[8], w[8];
      g.get(v);
      if (kAct != kActNone) {
        u.get(w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], act_slope<T>(w[j], kAct));   // (not fused into the sum below)
      }
      if (du) {
        if (kPlanes) store_planes(static_cast<__nv_bfloat16*>(du) + m * pitch + n, M * pitch, v);
        else store_f8(static_cast<T*>(du) + m * pitch + n, v);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += v[j];
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[ry][cx * 8 + i] = acc[i];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * kDuCols + threadIdx.x;
  if (col < N) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kDuRowsPar; ++i) s += red[i][threadIdx.x];
    part[blockIdx.y * N + col] = s;
  }
}

// db: the partial column sums in a fixed order.
__global__ void __launch_bounds__(256) linear_db_kernel(const float* part, int rows, int64_t N, float* db) {
  __shared__ float red[8][32];
  let_next_start();
  wait_for_previous();
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + cx;
  float acc = 0.f;
  if (col < N)
    for (int r = ry; r < rows; r += 8) acc += part[r * N + col];
  red[ry][cx] = acc;
  __syncthreads();
  if (ry == 0 && col < N) {
#pragma unroll
    for (int i = 1; i < 8; ++i) acc += red[i][cx];
    db[col] = acc;
  }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Blocks of rows of the du pass: one wave, each with four rounds at least.
int64_t du_row_blocks(int64_t M, int64_t N) {
  const int64_t cols = (N + kDuCols - 1) / kDuCols;
  int64_t blocks = (int64_t)kDuBlocks * sm_count() / cols;
  if (blocks < 1) blocks = 1;
  if (blocks > 65535) blocks = 65535;
  if (M <= kDuOneBlock) return 1;
  const int64_t most = (M + 31) / 32;
  return blocks < most ? blocks : most;
}

template <typename T, bool kPlanes>
void launch_du(const LinearProblem& p, void* du, int64_t pitch, float* part, int64_t blocks, cudaStream_t st) {
  const dim3 grid((unsigned)((p.N + kDuCols - 1) / kDuCols), (unsigned)blocks);
  const int64_t rows = (p.M() + blocks - 1) / blocks;
  const T* dy = static_cast<const T*>(p.dy);
  const float* pre = p.pre;
  const OutLayout lay(p);
  if (p.act == kActNone)
    linear_du_kernel<T, kActNone, kPlanes><<<grid, 256, 0, st>>>(dy, pre, du, part, lay, p.M(), p.N, rows, pitch);
  else if (p.act == kActSilu)
    linear_du_kernel<T, kActSilu, kPlanes><<<grid, 256, 0, st>>>(dy, pre, du, part, lay, p.M(), p.N, rows, pitch);
  else
    linear_du_kernel<T, kActGelu, kPlanes><<<grid, 256, 0, st>>>(dy, pre, du, part, lay, p.M(), p.N, rows, pitch);
}

// The bf16 planes of one or two fp32 matrices [rows, inner] (inner a multiple of 8).
struct SplitArgs {
  const float* v[2];
  __nv_bfloat16* planes[2];
  int64_t rows[2];
  uint32_t inner;
  int64_t pitch;
};
__global__ void __launch_bounds__(256) split_kernel(const SplitArgs a) {
  let_next_start();
  wait_for_previous();
  const uint32_t per_row = a.inner / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t r = i / per_row;
  const uint32_t c = (uint32_t)(i - r * per_row) * 8;
  const int which = r >= a.rows[0];
  if (which) r -= a.rows[0];
  if (r >= a.rows[which]) return;
  float w[8];
  load_f8(a.v[which] + r * a.inner + c, w);
  store_planes(a.planes[which] + r * a.pitch + c, a.rows[which] * a.pitch, w);
}

cudaError_t launch_split(const void* v0, void* p0, int64_t rows0, const void* v1, void* p1, int64_t rows1,
                         int64_t inner, bool after, cudaStream_t st) {
  const SplitArgs a{{static_cast<const float*>(v0), static_cast<const float*>(v1)},
                    {static_cast<__nv_bfloat16*>(p0), static_cast<__nv_bfloat16*>(p1)},
                    {rows0, rows1},
                    (uint32_t)inner,
                    plane_pitch(inner)};
  return launch_chained(split_kernel, dim3((unsigned)(((rows0 + rows1) * (inner / 8) + 255) / 256)), 256, 0, 0, after,
                        st, a);
}

// GECKO_KERNELS=simt selects the CUDA-core kernels for every type.
bool use_tc() {
  const char* e = std::getenv("GECKO_KERNELS");
  return !(e && std::strcmp(e, "simt") == 0);
}

// Where the working memory's parts lie.  The CUDA-core path uses du, as the
// tensors' type, and part.
struct Layout {
  bool dy_is_du;       // dy is already laid out as the products need it
  size_t du, part, x, w, gemm, bytes;
};

size_t plane_bytes(int64_t rows, int64_t inner) {
  return up256(3 * sizeof(__nv_bfloat16) * (size_t)rows * plane_pitch(inner));
}

Layout layout_of(const LinearProblem& p, bool backward) {
  const int64_t M = p.M();
  const bool f32 = p.dtype == kF32;
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += up256(n);
    return here;
  };
  l.dy_is_du = !f32 && p.act == kActNone && p.H == 0;
  if (backward) {
    // planes take more than the fp32 values
    l.du = take(l.dy_is_du ? 0 : f32 ? plane_bytes(M, p.N) : 2 * (size_t)M * plane_pitch(p.N));
    l.part = take(sizeof(float) * du_row_blocks(M, p.N) * p.N);
  }
  if (!backward && f32 && M <= kRowsMost) return l;   // no planes
  l.x = take(f32 ? plane_bytes(M, p.K) : 0);
  l.w = take(f32 ? plane_bytes(p.N, p.K) : 0);
  size_t g = backward ? gemm_tc_workspace(M, p.K, p.N, p.dtype) : gemm_tc_workspace(M, p.N, p.K, p.dtype);
  if (backward) {
    const size_t dw = gemm_tc_workspace(p.N, p.K, M, p.dtype);
    if (dw > g) g = dw;
  }
  l.gemm = take(g);
  l.bytes = at;
  return l;
}

template <typename T>
cudaError_t forward_impl(const LinearProblem& p, cudaStream_t st) {
  ForwardOut<T> ep{p.bias, static_cast<const T*>(p.residual), static_cast<T*>(p.y), p.pre, OutLayout(p), p.act};
  if constexpr (sizeof(T) == 4)
    if (p.M() <= kRowsMost)
      return p.M() <= 4   ? launch_rows<4>(p, ep, st)
             : p.M() <= 8 ? launch_rows<8>(p, ep, st)
                          : launch_rows<16>(p, ep, st);
  if (!use_tc()) {
    simt_gemm<T>(p.x, p.K, 1, p.w, p.K, 1, p.M(), p.N, p.K, ep, st);
    return cudaGetLastError();
  }
  const Layout l = layout_of(p, false);
  char* ws = static_cast<char*>(p.ws);
  if (p.dtype == kBF16) return launch_linear_tc(p, p.x, p.w, ws + l.gemm, false, st);
  if (cudaError_t e = launch_split(p.x, ws + l.x, p.M(), p.w, ws + l.w, p.N, p.K, false, st)) return e;
  return launch_linear_tc(p, ws + l.x, ws + l.w, ws + l.gemm, true, st);
}

template <typename T>
cudaError_t backward_impl(const LinearProblem& p, cudaStream_t st) {
  constexpr bool f32 = sizeof(T) == 4;
  const int64_t M = p.M();
  const Layout l = layout_of(p, true);
  char* ws = static_cast<char*>(p.ws);
  float* part = reinterpret_cast<float*>(ws + l.part);
  const bool tc = use_tc(), products = p.dx || p.dw;
  const bool alias = tc ? l.dy_is_du : p.act == kActNone && p.H == 0;
  const int64_t pitch = tc && !alias ? plane_pitch(p.N) : p.N;   // of du
  bool after = false;
  cudaError_t e;
  if (p.db || (!alias && products)) {
    const int64_t blocks = du_row_blocks(M, p.N);
    void* du = products && !alias ? ws + l.du : nullptr;
    float* sums = !p.db ? nullptr : blocks == 1 ? p.db : part;   // one block of rows: its sums are db
    if (tc && f32) launch_du<T, true>(p, du, pitch, sums, blocks, st);
    else launch_du<T, false>(p, du, pitch, sums, blocks, st);
    after = true;
    const dim3 cols((unsigned)((p.N + 31) / 32));
    if (p.db && blocks > 1 &&
        (e = launch_chained(linear_db_kernel, cols, 256, 0, 0, after, st, part, (int)blocks, p.N, p.db)))
      return e;
  }
  const void* g = alias ? p.dy : ws + l.du;
  if (!tc) {
    if (p.dx) simt_gemm<T>(g, p.N, 1, p.w, 1, p.K, M, p.K, p.N, PlainOut<T>{static_cast<T*>(p.dx), p.K}, st);
    if (p.dw) simt_gemm<T>(g, 1, p.N, p.x, 1, p.K, p.N, p.K, M, PlainOut<T>{static_cast<T*>(p.dw), p.K}, st);
    return cudaGetLastError();
  }
  const void *x = p.x, *w = p.w;
  if (f32 && products) {
    if ((e = launch_split(p.x, ws + l.x, p.dw ? M : 0, p.w, ws + l.w, p.dx ? p.N : 0, p.K, after, st))) return e;
    after = true;
    x = ws + l.x;
    w = ws + l.w;
  }
  if (p.dx && (e = launch_linear_dx_tc(p, g, pitch, w, ws + l.gemm, after, st))) return e;
  if (p.dw && (e = launch_linear_dw_tc(p, g, pitch, x, ws + l.gemm, after || p.dx, st))) return e;
  return cudaGetLastError();
}

}  // namespace

size_t linear_workspace_bytes(const LinearProblem& p, bool backward) { return layout_of(p, backward).bytes; }

cudaError_t launch_linear(const LinearProblem& p, cudaStream_t st) {
  return p.dtype == kBF16 ? forward_impl<__nv_bfloat16>(p, st) : forward_impl<float>(p, st);
}

cudaError_t launch_linear_bwd(const LinearProblem& p, cudaStream_t st) {
  return p.dtype == kBF16 ? backward_impl<__nv_bfloat16>(p, st) : backward_impl<float>(p, st);
}

}  // namespace gecko
