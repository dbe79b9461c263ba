// C-ABI entry points of the layer steps around the SCA + AWM path: the gated
// recurrence, the queries and keys from the shared representation, and the
// projection.  See include/gecko.h for the contract of each.  Working memory
// is the caller's, so the calls share nothing and may overlap.
#include <cmath>
#include <initializer_list>

#include "../../include/gecko.h"
#include "common.cuh"
#include "gecko_internal.h"

namespace gecko {
namespace {

constexpr int64_t kGridYZ = 65535;
static_assert(kScanChunk == GECKO_SCAN_CHUNK, "the contract's chunk length");

int check_pointers(std::initializer_list<const void*> required, std::initializer_list<const void*> optional) {
  int i = 0;
  for (const void* p : required) {
    if (!p) return fail(GECKO_ERR_ARG, "required pointer %d is NULL", i);
    ++i;
  }
  i = 0;
  for (const void* p : required) {
    if (reinterpret_cast<uintptr_t>(p) % 16) return fail(GECKO_ERR_ALIGN, "pointer %d is not 16-byte aligned", i);
    ++i;
  }
  i = 0;
  for (const void* p : optional) {
    if (reinterpret_cast<uintptr_t>(p) % 16)
      return fail(GECKO_ERR_ALIGN, "optional pointer %d is not 16-byte aligned", i);
    ++i;
  }
  return GECKO_OK;
}

int check_dtype(int dtype) {
  return dtype == GECKO_F32 || dtype == GECKO_BF16 ? GECKO_OK : fail(GECKO_ERR_ARG, "unknown dtype %d", dtype);
}

int check_workspace(const void* ws, int64_t have, size_t need) {
  if (have < 0 || (size_t)have < need)
    return fail(GECKO_ERR_ARG, "workspace of %lld bytes, %zu needed", (long long)have, need);
  if (need && !ws) return fail(GECKO_ERR_ARG, "workspace is NULL (%zu bytes needed)", need);
  if (reinterpret_cast<uintptr_t>(ws) % 16) return fail(GECKO_ERR_ALIGN, "workspace is not 16-byte aligned");
  return GECKO_OK;
}

int launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? GECKO_OK : fail(GECKO_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// A C entry point lets no C++ exception out.
template <class F>
int guarded(F&& f) noexcept {
  try {
    return f();
  } catch (...) {
    return GECKO_ERR_ALLOC;
  }
}

// ---------------------------------------------------------- gated scan --

int check_scan_sizes(int64_t B, int64_t L, int64_t D, int dtype) {
  if (int rc = check_dtype(dtype)) return rc;
  if (B < 1 || L < 1 || D < 1)
    return fail(GECKO_ERR_ARG, "sizes must be >= 1 (B=%lld L=%lld D=%lld)", (long long)B, (long long)L, (long long)D);
  if (D % 8) return fail(GECKO_ERR_SHAPE, "D must be a multiple of 8 (got %lld)", (long long)D);
  if (B > kGridYZ || L > kGridYZ * kScanChunk || D > (int64_t(1) << 24) || !scan_grid_fits(B, L, D, dtype))
    return fail(GECKO_ERR_SHAPE, "B, L or D exceeds the kernels' range (B=%lld L=%lld D=%lld)", (long long)B,
                (long long)L, (long long)D);
  return GECKO_OK;
}

int scan_forward(const void* x, const void* log_a, void* y, const uint8_t* reset, const float* state_in,
                 float* state_out, float* chunk_state, int64_t B, int64_t L, int64_t D, int dtype, void* ws,
                 int64_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_scan_sizes(B, L, D, dtype))) return rc;
  if ((rc = check_pointers({x, log_a, y}, {state_in, state_out, chunk_state}))) return rc;
  if ((rc = check_workspace(ws, ws_bytes, scan_workspace_bytes(B, L, D, dtype, false)))) return rc;
  ScanProblem p{};
  if ((rc = device_status_word(&p.status))) return rc;
  p.x = x, p.log_a = log_a, p.y = y, p.reset = reset;
  p.state_in = state_in, p.state_out = state_out, p.chunk_state = chunk_state;
  p.B = B, p.L = L, p.D = D, p.dtype = dtype, p.ws = ws;
  cudaGetLastError();
  return launched(launch_scan(p, static_cast<cudaStream_t>(stream)), "gated scan");
}

int scan_backward(const void* x, const void* log_a, const void* dy, const uint8_t* reset, const float* chunk_state,
                  const float* dstate_out, void* dx, void* dlog_a, float* dstate_in, int64_t B, int64_t L, int64_t D,
                  int dtype, void* ws, int64_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_scan_sizes(B, L, D, dtype))) return rc;
  if ((rc = check_pointers({x, log_a, dy, chunk_state, dx, dlog_a}, {dstate_out, dstate_in}))) return rc;
  if ((rc = check_workspace(ws, ws_bytes, scan_workspace_bytes(B, L, D, dtype, true)))) return rc;
  ScanProblem p{};
  if ((rc = device_status_word(&p.status))) return rc;
  p.x = x, p.log_a = log_a, p.dy = dy, p.reset = reset;
  p.chunk_state = const_cast<float*>(chunk_state);
  p.dstate_out = dstate_out, p.dx = dx, p.dlog_a = dlog_a, p.dstate_in = dstate_in;
  p.B = B, p.L = L, p.D = D, p.dtype = dtype, p.ws = ws;
  cudaGetLastError();
  return launched(launch_scan_bwd(p, static_cast<cudaStream_t>(stream)), "gated scan backward");
}

// ---------------------------------------------------------- queries, keys --

int check_qk_sizes(int64_t B, int64_t T, int64_t H, int64_t d, float eps, int64_t rot_dim, double rot_base,
                   int dtype) {
  if (int rc = check_dtype(dtype)) return rc;
  if (B < 1 || T < 1 || H < 1)
    return fail(GECKO_ERR_ARG, "sizes must be >= 1 (B=%lld T=%lld H=%lld)", (long long)B, (long long)T, (long long)H);
  // (below 2^-60, rows longer than eps could have squares that vanish in fp32)
  if (!(eps >= 0x1p-60f) || !std::isfinite(eps)) return fail(GECKO_ERR_ARG, "eps must be at least 2^-60 and finite");
  if (rot_dim < 0) return fail(GECKO_ERR_ARG, "rot_dim must be >= 0");
  if (rot_dim > 0 && (!(rot_base >= 1.0) || !std::isfinite(rot_base)))
    return fail(GECKO_ERR_ARG, "rot_base must be finite and at least 1");
  if (d != 64 && d != 128) return fail(GECKO_ERR_SHAPE, "d must be 64 or 128 (got %lld)", (long long)d);
  if (rot_dim > d || rot_dim % 16)
    return fail(GECKO_ERR_SHAPE, "rot_dim must be a multiple of 16 and at most d (got %lld)", (long long)rot_dim);
  const int64_t most = int64_t(1) << 31;
  if (B >= most || T >= most || H > kGridYZ || B * T >= int64_t(1) << 35)
    return fail(GECKO_ERR_SHAPE, "B, T or H exceeds the kernels' range (B=%lld T=%lld H=%lld)", (long long)B,
                (long long)T, (long long)H);
  return GECKO_OK;
}

// (read one at a time: a token's slice of a row of positions will do)
int check_positions(const int64_t* pos) {
  return reinterpret_cast<uintptr_t>(pos) % 8 ? fail(GECKO_ERR_ALIGN, "pos is not 8-byte aligned") : GECKO_OK;
}

void set_rotation(QkProblem& p, int64_t rot_dim, double rot_base, int interleaved) {
  p.rot_dim = (int)rot_dim;
  p.interleaved = interleaved != 0;
  for (int i = 0; i < rot_dim / 2; ++i)
    p.rate[i] = std::pow(rot_base, -2.0 * i / (double)rot_dim) / (2.0 * 3.14159265358979323846);
}

int qk_forward(const void* z, const float* scale, const float* shift, const int64_t* pos, void* q, void* k, void* qm,
               void* km, int64_t B, int64_t T, int64_t H, int64_t d, float eps, int64_t pos0, int64_t rot_dim,
               double rot_base, int interleaved, int dtype, void* stream) {
  int rc;
  if ((rc = check_qk_sizes(B, T, H, d, eps, rot_dim, rot_base, dtype))) return rc;
  if ((rc = check_pointers({z, scale, shift, q, k, qm, km}, {})) || (rc = check_positions(pos))) return rc;
  QkProblem p{};
  p.z = z, p.scale = scale, p.shift = shift, p.pos = pos;
  p.out[0] = q, p.out[1] = k, p.out[2] = qm, p.out[3] = km;
  p.B = B, p.T = T, p.H = H, p.d = d, p.eps = eps, p.pos0 = pos0, p.dtype = dtype;
  set_rotation(p, rot_dim, rot_base, interleaved);
  cudaGetLastError();
  return launched(launch_qk(p, static_cast<cudaStream_t>(stream)), "queries and keys");
}

int qk_backward(const void* z, const float* scale, const int64_t* pos, const void* dq, const void* dk,
                const void* dqm, const void* dkm, void* dz, float* dscale, float* dshift, int64_t B, int64_t T,
                int64_t H, int64_t d, float eps, int64_t pos0, int64_t rot_dim, double rot_base, int interleaved,
                int dtype, void* ws, int64_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_qk_sizes(B, T, H, d, eps, rot_dim, rot_base, dtype))) return rc;
  if ((rc = check_pointers({z, scale, dq, dk, dqm, dkm, dz, dscale, dshift}, {})) || (rc = check_positions(pos)))
    return rc;
  if ((rc = check_workspace(ws, ws_bytes, qk_workspace_bytes(B, T, H, d)))) return rc;
  QkProblem p{};
  p.z = z, p.scale = scale, p.pos = pos;
  p.dout[0] = dq, p.dout[1] = dk, p.dout[2] = dqm, p.dout[3] = dkm;
  p.dz = dz, p.dscale = dscale, p.dshift = dshift;
  p.B = B, p.T = T, p.H = H, p.d = d, p.eps = eps, p.pos0 = pos0, p.dtype = dtype, p.ws = ws;
  set_rotation(p, rot_dim, rot_base, interleaved);
  cudaGetLastError();
  return launched(launch_qk_bwd(p, static_cast<cudaStream_t>(stream)), "queries and keys backward");
}

// ------------------------------------------------------------- projection --

int check_linear_sizes(int64_t B, int64_t T, int64_t N, int64_t K, int64_t H, int act, int dtype) {
  if (int rc = check_dtype(dtype)) return rc;
  if (B < 1 || T < 1 || N < 1 || K < 1 || H < 0)
    return fail(GECKO_ERR_ARG, "sizes must be >= 1 and H >= 0 (B=%lld T=%lld N=%lld K=%lld H=%lld)", (long long)B,
                (long long)T, (long long)N, (long long)K, (long long)H);
  if (act < GECKO_ACT_NONE || act > GECKO_ACT_GELU) return fail(GECKO_ERR_ARG, "unknown activation %d", act);
  if (N % 8 || K % 8)
    return fail(GECKO_ERR_SHAPE, "N and K must be multiples of 8 (N=%lld K=%lld)", (long long)N, (long long)K);
  if (H && (N % H || (N / H) % 8))
    return fail(GECKO_ERR_SHAPE, "N / H must be a multiple of 8 (N=%lld H=%lld)", (long long)N, (long long)H);
  const int64_t most = (int64_t(1) << 31) - 256, wide = int64_t(1) << 20;
  if (B > most || T > most || B * T > most || N > wide || K > wide || B * T * (N > K ? N : K) > int64_t(1) << 38)
    return fail(GECKO_ERR_SHAPE, "B * T, N or K exceeds the kernels' range (B=%lld T=%lld N=%lld K=%lld)",
                (long long)B, (long long)T, (long long)N, (long long)K);
  return GECKO_OK;
}

LinearProblem linear_problem(int64_t B, int64_t T, int64_t N, int64_t K, int64_t H, int act, int dtype) {
  LinearProblem p{};
  p.B = B, p.T = T, p.N = N, p.K = K, p.H = H, p.act = act, p.dtype = dtype;
  return p;
}

int linear_forward(const void* x, const void* w, const float* bias, const void* residual, void* y, float* pre,
                   int64_t B, int64_t T, int64_t N, int64_t K, int64_t H, int act, int dtype, void* ws,
                   int64_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_linear_sizes(B, T, N, K, H, act, dtype))) return rc;
  if ((rc = check_pointers({x, w, y}, {bias, residual, pre}))) return rc;
  LinearProblem p = linear_problem(B, T, N, K, H, act, dtype);
  if ((rc = check_workspace(ws, ws_bytes, linear_workspace_bytes(p, false)))) return rc;
  if ((rc = device_status_word(&p.status))) return rc;
  p.x = x, p.w = w, p.bias = bias, p.residual = residual, p.y = y, p.pre = pre, p.ws = ws;
  cudaGetLastError();
  return launched(launch_linear(p, static_cast<cudaStream_t>(stream)), "projection");
}

int linear_backward(const void* x, const void* w, const void* dy, const float* pre, void* dx, void* dw, float* db,
                    int64_t B, int64_t T, int64_t N, int64_t K, int64_t H, int act, int dtype, void* ws,
                    int64_t ws_bytes, void* stream) {
  int rc;
  if ((rc = check_linear_sizes(B, T, N, K, H, act, dtype))) return rc;
  if ((rc = check_pointers({x, w, dy}, {pre, dx, dw, db}))) return rc;
  if (act != GECKO_ACT_NONE && !pre) return fail(GECKO_ERR_ARG, "an activation's gradient needs pre");
  if (!dx && !dw && !db) return fail(GECKO_ERR_ARG, "dx, dw and db are all NULL");
  LinearProblem p = linear_problem(B, T, N, K, H, act, dtype);
  if ((rc = check_workspace(ws, ws_bytes, linear_workspace_bytes(p, true)))) return rc;
  if ((rc = device_status_word(&p.status))) return rc;
  p.x = x, p.w = w, p.dy = dy, p.pre = const_cast<float*>(pre), p.dx = dx, p.dw = dw, p.db = db, p.ws = ws;
  cudaGetLastError();
  return launched(launch_linear_bwd(p, static_cast<cudaStream_t>(stream)), "projection backward");
}

}  // namespace
}  // namespace gecko

using namespace gecko;

extern "C" int gecko_gated_scan_workspace(int64_t B, int64_t L, int64_t D, int dtype, int backward, int64_t* bytes) {
  return guarded([&] {
    if (!bytes) return fail(GECKO_ERR_ARG, "bytes is NULL");
    if (int rc = check_scan_sizes(B, L, D, dtype)) return rc;
    *bytes = (int64_t)scan_workspace_bytes(B, L, D, dtype, backward != 0);
    return GECKO_OK;
  });
}

extern "C" int gecko_gated_scan_forward(const void* x, const void* log_a, void* y, const uint8_t* reset,
                                        const float* state_in, float* state_out, float* chunk_state, int64_t B,
                                        int64_t L, int64_t D, int dtype, void* workspace, int64_t workspace_bytes,
                                        void* stream) {
  return guarded([&] {
    return scan_forward(x, log_a, y, reset, state_in, state_out, chunk_state, B, L, D, dtype, workspace,
                        workspace_bytes, stream);
  });
}

extern "C" int gecko_gated_scan_backward(const void* x, const void* log_a, const void* dy, const uint8_t* reset,
                                         const float* chunk_state, const float* dstate_out, void* dx, void* dlog_a,
                                         float* dstate_in, int64_t B, int64_t L, int64_t D, int dtype,
                                         void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    return scan_backward(x, log_a, dy, reset, chunk_state, dstate_out, dx, dlog_a, dstate_in, B, L, D, dtype,
                         workspace, workspace_bytes, stream);
  });
}

extern "C" int gecko_qk_forward(const void* z, const float* scale, const float* shift, const int64_t* pos, void* q,
                                void* k, void* qm, void* km, int64_t B, int64_t T, int64_t H, int64_t d, float eps,
                                int64_t pos0, int64_t rot_dim, double rot_base, int interleaved, int dtype,
                                void* stream) {
  return guarded([&] {
    return qk_forward(z, scale, shift, pos, q, k, qm, km, B, T, H, d, eps, pos0, rot_dim, rot_base, interleaved,
                      dtype, stream);
  });
}

extern "C" int gecko_qk_workspace(int64_t B, int64_t T, int64_t H, int64_t d, int dtype, int64_t* bytes) {
  return guarded([&] {
    if (!bytes) return fail(GECKO_ERR_ARG, "bytes is NULL");
    if (int rc = check_qk_sizes(B, T, H, d, 1.f, 0, 1.0, dtype)) return rc;
    *bytes = (int64_t)qk_workspace_bytes(B, T, H, d);
    return GECKO_OK;
  });
}

extern "C" int gecko_qk_backward(const void* z, const float* scale, const int64_t* pos, const void* dq,
                                 const void* dk, const void* dqm, const void* dkm, void* dz, float* dscale,
                                 float* dshift, int64_t B, int64_t T, int64_t H, int64_t d, float eps, int64_t pos0,
                                 int64_t rot_dim, double rot_base, int interleaved, int dtype, void* workspace,
                                 int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    return qk_backward(z, scale, pos, dq, dk, dqm, dkm, dz, dscale, dshift, B, T, H, d, eps, pos0, rot_dim, rot_base,
                       interleaved, dtype, workspace, workspace_bytes, stream);
  });
}

extern "C" int gecko_linear_workspace(int64_t B, int64_t T, int64_t N, int64_t K, int64_t H, int act, int dtype,
                                      int backward, int64_t* bytes) {
  return guarded([&] {
    if (!bytes) return fail(GECKO_ERR_ARG, "bytes is NULL");
    if (int rc = check_linear_sizes(B, T, N, K, H, act, dtype)) return rc;
    *bytes = (int64_t)linear_workspace_bytes(linear_problem(B, T, N, K, H, act, dtype), backward != 0);
    return GECKO_OK;
  });
}

extern "C" int gecko_linear_forward(const void* x, const void* w, const float* bias, const void* residual, void* y,
                                    float* pre, int64_t B, int64_t T, int64_t N, int64_t K, int64_t H, int act,
                                    int dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    return linear_forward(x, w, bias, residual, y, pre, B, T, N, K, H, act, dtype, workspace, workspace_bytes,
                          stream);
  });
}

extern "C" int gecko_linear_backward(const void* x, const void* w, const void* dy, const float* pre, void* dx,
                                     void* dw, float* db, int64_t B, int64_t T, int64_t N, int64_t K, int64_t H,
                                     int act, int dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    return linear_backward(x, w, dy, pre, dx, dw, db, B, T, N, K, H, act, dtype, workspace, workspace_bytes, stream);
  });
}
