// Gated linear recurrence, the input-gated companion of CEMA:
//   a_t = exp(log_a_t)  (0 where a document starts),
//   h_t = a_t h_{t-1} + x_t,  y_t = h_t                    (per feature)
// and its gradients
//   dh_t = dy_t + a_{t+1} dh_{t+1},  dx_t = dh_t,
//   dlog_a_t = dh_t a_t h_{t-1},     dstate_in = a_0 dh_0.
// A span of tokens maps the state entering it affinely, h_out = A h_in + h,
// with A the product of its decays and h its scan from zero; spans compose.
// Everything is held in fp32 whatever the tensors' type.
#include "common.cuh"
#include "gecko_internal.h"

namespace gecko {
namespace {

// A decay of zero drops what came before, even if that is not finite.
__device__ __forceinline__ float decay_fma(float a, float h, float x) { return a == 0.f ? x : fmaf(a, h, x); }

__device__ __forceinline__ float decay_of(float log_a, bool drop) { return drop ? 0.f : expf(log_a); }

// (A, h) of every chunk scanned from zero: agg [B, C, D].
template <typename T>
__global__ void scan_local_kernel(const T* x, const T* log_a, const uint8_t* reset, float2* agg, int64_t L, int64_t D) {
  const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= D) return;
  const int64_t b = blockIdx.z, c = blockIdx.y;
  const int64_t t0 = c * kScanChunk, t1 = min(L, t0 + kScanChunk);
  float A = 1.f, h = 0.f;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t i = (b * L + t) * D + d;
    const float a = decay_of(to_f32(log_a[i]), reset && reset[b * L + t]);
    h = decay_fma(a, h, to_f32(x[i]));
    A *= a;
  }
  agg[(b * gridDim.y + c) * D + d] = make_float2(A, h);
}

// State entering every chunk, and the state after the last one.
__global__ void scan_carry_kernel(const float2* agg, const float* state_in, float* enter, float* state_out, int64_t B,
                                  int64_t C, int64_t D) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= B * D) return;
  const int64_t b = i / D, d = i % D;
  float h = state_in ? state_in[i] : 0.f;
  for (int64_t c = 0; c < C; ++c) {
    const int64_t j = (b * C + c) * D + d;
    enter[j] = h;
    h = decay_fma(agg[j].x, h, agg[j].y);
  }
  if (state_out) state_out[i] = h;
}

template <typename T>
__global__ void scan_out_kernel(const T* x, const T* log_a, const uint8_t* reset, const float* enter, T* y, int64_t L,
                                int64_t D) {
  const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= D) return;
  const int64_t b = blockIdx.z, c = blockIdx.y;
  const int64_t t0 = c * kScanChunk, t1 = min(L, t0 + kScanChunk);
  float h = enter[(b * gridDim.y + c) * D + d];
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t i = (b * L + t) * D + d;
    const float a = decay_of(to_f32(log_a[i]), reset && reset[b * L + t]);
    h = decay_fma(a, h, to_f32(x[i]));
    y[i] = from_f32<T>(h);
  }
}

// Reverse direction: with e_t = a_t dh_t (what token t passes back),
// e = A e_next + r over a chunk: dh_t = dy_t + e_{t+1}.
template <typename T>
__global__ void scan_bwd_local_kernel(const T* dy, const T* log_a, const uint8_t* reset, float2* agg, int64_t L,
                                      int64_t D) {
  const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= D) return;
  const int64_t b = blockIdx.z, c = blockIdx.y;
  const int64_t t0 = c * kScanChunk, t1 = min(L, t0 + kScanChunk);
  float A = 1.f, e = 0.f;
  for (int64_t t = t1 - 1; t >= t0; --t) {
    const int64_t i = (b * L + t) * D + d;
    const float a = decay_of(to_f32(log_a[i]), reset && reset[b * L + t]);
    e = a == 0.f ? 0.f : a * (to_f32(dy[i]) + e);
    A *= a;
  }
  agg[(b * gridDim.y + c) * D + d] = make_float2(A, e);
}

__global__ void scan_bwd_carry_kernel(const float2* agg, const float* dstate_out, float* enter, float* dstate_in,
                                      int64_t B, int64_t C, int64_t D) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= B * D) return;
  const int64_t b = i / D, d = i % D;
  float e = dstate_out ? dstate_out[i] : 0.f;
  for (int64_t c = C - 1; c >= 0; --c) {
    const int64_t j = (b * C + c) * D + d;
    enter[j] = e;
    e = decay_fma(agg[j].x, e, agg[j].y);
  }
  if (dstate_in) dstate_in[i] = e;
}

// One chunk's gradients: the states h_{t-1} again from the chunk's entering
// state (kept in shared memory), then the reverse recurrence.
template <typename T>
__global__ void __launch_bounds__(32) scan_bwd_out_kernel(const T* x, const T* log_a, const T* dy,
                                                          const uint8_t* reset, const float* chunk_state,
                                                          const float* enter, T* dx, T* dlog_a, int64_t L, int64_t D) {
  __shared__ float hs[kScanChunk][32];
  const int64_t d = (int64_t)blockIdx.x * 32 + threadIdx.x;
  if (d >= D) return;
  const int64_t b = blockIdx.z, c = blockIdx.y;
  const int64_t t0 = c * kScanChunk, t1 = min(L, t0 + kScanChunk);
  float h = chunk_state[(b * gridDim.y + c) * D + d];
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t i = (b * L + t) * D + d;
    const float a = decay_of(to_f32(log_a[i]), reset && reset[b * L + t]);
    hs[t - t0][threadIdx.x] = h;
    h = decay_fma(a, h, to_f32(x[i]));
  }
  float e = enter[(b * gridDim.y + c) * D + d];
  for (int64_t t = t1 - 1; t >= t0; --t) {
    const int64_t i = (b * L + t) * D + d;
    const float a = decay_of(to_f32(log_a[i]), reset && reset[b * L + t]);
    const float dh = to_f32(dy[i]) + e;
    e = a == 0.f ? 0.f : a * dh;
    dx[i] = from_f32<T>(dh);
    dlog_a[i] = from_f32<T>(a == 0.f ? 0.f : e * hs[t - t0][threadIdx.x]);
  }
}

template <typename T>
cudaError_t scan_impl(const ScanProblem& p, cudaStream_t st) {
  const int64_t C = scan_chunks(p.L);
  float2* agg = static_cast<float2*>(p.ws);
  float* enter = p.chunk_state ? p.chunk_state : reinterpret_cast<float*>(agg + p.B * C * p.D);
  const dim3 grid((unsigned)((p.D + 127) / 128), (unsigned)C, (unsigned)p.B);
  const T *x = static_cast<const T*>(p.x), *g = static_cast<const T*>(p.log_a);
  scan_local_kernel<T><<<grid, 128, 0, st>>>(x, g, p.reset, agg, p.L, p.D);
  scan_carry_kernel<<<(unsigned)((p.B * p.D + 127) / 128), 128, 0, st>>>(agg, p.state_in, enter, p.state_out, p.B, C,
                                                                         p.D);
  scan_out_kernel<T><<<grid, 128, 0, st>>>(x, g, p.reset, enter, static_cast<T*>(p.y), p.L, p.D);
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_bwd_impl(const ScanProblem& p, cudaStream_t st) {
  const int64_t C = scan_chunks(p.L);
  float2* agg = static_cast<float2*>(p.ws);
  float* enter = reinterpret_cast<float*>(agg + p.B * C * p.D);
  const T *x = static_cast<const T*>(p.x), *g = static_cast<const T*>(p.log_a), *dy = static_cast<const T*>(p.dy);
  const dim3 grid((unsigned)((p.D + 127) / 128), (unsigned)C, (unsigned)p.B);
  scan_bwd_local_kernel<T><<<grid, 128, 0, st>>>(dy, g, p.reset, agg, p.L, p.D);
  scan_bwd_carry_kernel<<<(unsigned)((p.B * p.D + 127) / 128), 128, 0, st>>>(agg, p.dstate_out, enter, p.dstate_in,
                                                                             p.B, C, p.D);
  const dim3 grid32((unsigned)((p.D + 31) / 32), (unsigned)C, (unsigned)p.B);
  scan_bwd_out_kernel<T><<<grid32, 32, 0, st>>>(x, g, dy, p.reset, p.chunk_state, enter, static_cast<T*>(p.dx),
                                                static_cast<T*>(p.dlog_a), p.L, p.D);
  return cudaGetLastError();
}

}  // namespace

size_t scan_workspace_bytes(int64_t B, int64_t L, int64_t D, int, bool) {
  return (size_t)(B * scan_chunks(L) * D) * (sizeof(float2) + sizeof(float));
}

cudaError_t launch_scan(const ScanProblem& p, cudaStream_t st) {
  return p.dtype == kBF16 ? scan_impl<__nv_bfloat16>(p, st) : scan_impl<float>(p, st);
}

cudaError_t launch_scan_bwd(const ScanProblem& p, cudaStream_t st) {
  return p.dtype == kBF16 ? scan_bwd_impl<__nv_bfloat16>(p, st) : scan_bwd_impl<float>(p, st);
}

}  // namespace gecko
