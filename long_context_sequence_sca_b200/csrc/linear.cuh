// Pieces shared by the projection's kernels: the activations, 8-element
// loads and stores, and the output layouts.
#pragma once

#include "chain.cuh"
#include "common.cuh"
#include "gecko_internal.h"

namespace gecko {

// Phi(u) of the normal distribution and e = exp(-u^2 / 2).  Phi(-x) / e falls off like
// 1 / x: as a function of t = 1 / (1 + c x) it is t times a polynomial, fitted for this
// library to the relative error on 0 <= x <= 14.7 (Lawson's reweighted least squares;
// Phi leaves fp32 at 14.2).  kFine: to 4.4e-8, written in t - 1/2, where it loses least in
// fp32; with the SFU's quotient and exponential Phi is good to 2^-20 and 1.25 u^2 2^-24 of
// itself, however small it is.  Else, for what is rounded to bf16, to 8.5e-6, 1/460 of
// that rounding (8192 x 4096 x 1024 in bf16 82.5 us, with the fine one 85.9).
template <bool kFine>
__device__ __forceinline__ float normal_cdf(float u, float& e) {
  const float t = __fdividef(1.f, fmaf(kFine ? 0.35355338f : 0.4596194f, fabsf(u), 1.f));
  e = __expf(-0.5f * u * u);
  float p;
  if (kFine) {
    const float s = t - 0.5f;
    p = fmaf(-0.02958603f, s, 0.02419536f);
    p = fmaf(p, s, 0.047663148f);
    p = fmaf(p, s, -0.051505312f);
    p = fmaf(p, s, -0.085933305f);
    p = fmaf(p, s, 0.072870664f);
    p = fmaf(p, s, 0.27946958f);
    p = fmaf(p, s, 0.34358048f);
    p = fmaf(p, s, 0.25539568f);
  } else {
    p = fmaf(0.07212547f, t, -0.23665257f);
    p = fmaf(p, t, 0.17863609f);
    p = fmaf(p, t, 0.11572741f);
    p = fmaf(p, t, 0.18697758f);
    p = fmaf(p, t, 0.18319023f);
  }
  const float tail = p * t * e;
  return u < 0.f ? tail : 1.f - tail;
}

// s = 1 / (1 + e^-u) and 1 - s in fp32, both to 2^-22 of themselves.
__device__ __forceinline__ float sigmoid(float u, float& rest) {
  const float e = expf(-fabsf(u)), r = 1.f / (1.f + e), far = e * r;
  rest = u < 0.f ? r : far;
  return u < 0.f ? far : r;
}

// f(u), of which values of type T are made: SiLU u / (1 + e^-u); GELU u Phi(u).  For
// bf16 SiLU's exponential and quotient are the SFU's, good to 2^-21 + |u| 2^-23, far
// below a bf16 step.
template <typename T>
__device__ __forceinline__ float activate(float u, int act) {
  if (act == kActSilu) {
    if (sizeof(T) == 2) return __fdividef(u, 1.f + __expf(-u));
    float rest;
    return u * sigmoid(u, rest);
  }
  if (act == kActGelu) {
    float e;
    return u * normal_cdf<sizeof(T) == 4>(u, e);
  }
  return u;
}

// f'(u): SiLU s (1 + u (1 - s)), s = 1 / (1 + e^-u); GELU Phi(u) + u phi(u).
template <typename T>
__device__ __forceinline__ float act_slope(float u, int act) {
  if (act == kActSilu) {
    if (sizeof(T) == 2) {
      const float s = __fdividef(1.f, 1.f + __expf(-u));
      return s * fmaf(u, 1.f - s, 1.f);
    }
    float rest;
    const float s = sigmoid(u, rest);
    return s * fmaf(u, rest, 1.f);
  }
  if (act == kActGelu) {
    float e;
    const float c = normal_cdf<true>(u, e);
    return fmaf(u * 0.3989422804014327f, e, c);
  }
  return 1.f;
}

__device__ __forceinline__ void load_f8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load_f8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store_f8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_f8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}

// 16 bytes to shared memory without a stop in registers, or zeros.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}

// v = h + m + l in bf16: each plane is the rest of the ones before it rounded to
// nearest, so what is left is below 2^-25 |v|.  h is cut instead where rounding
// would carry a finite v to infinity; an infinite v has no rest.
__device__ __forceinline__ void split3(float v, float& h, float& m, float& l) {
  h = __bfloat162float(__float2bfloat16_rn(v));
  if (isinf(h)) h = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
  const float r = isinf(v) ? 0.f : v - h;
  m = __bfloat162float(__float2bfloat16_rn(r));
  l = r - m;   // rounded when it is stored
}

// The planes of 8 values, `plane` elements apart.
__device__ __forceinline__ void store_planes(__nv_bfloat16* p, int64_t plane, const float (&v)[8]) {
  float h[8], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split3(v[i], h[i], m[i], l[i]);
  store_f8(p, h);
  store_f8(p + plane, m);
  store_f8(p + 2 * plane, l);
}

// 8 elements as loaded.
template <typename T> struct Vec8;
template <> struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <> struct Vec8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// Where element (m, n) of y, pre, residual and dy lies, row(m) + col(n):
// [M, N] row-major, or [B, H, T, N / H] (m = b T + t, n = h N / H + j).
struct OutLayout {
  int64_t N;
  uint32_t T, H, hd;
  explicit OutLayout(const LinearProblem& p)
      : N(p.N), T((uint32_t)p.T), H((uint32_t)p.H), hd(p.H ? (uint32_t)(p.N / p.H) : 1) {}
  __device__ __forceinline__ int64_t row(int64_t m) const {
    if (H == 0) return m * N;
    const uint32_t b = (uint32_t)m / T, t = (uint32_t)m - b * T;
    return ((int64_t)b * H * T + t) * hd;
  }
  __device__ __forceinline__ int64_t col(int n) const {
    if (H == 0) return n;
    const uint32_t h = (uint32_t)n / hd;
    return (int64_t)h * T * hd + ((uint32_t)n - h * hd);
  }
  __device__ __forceinline__ int64_t at(int64_t m, int64_t n) const { return row(m) + col((int)n); }
};

}  // namespace gecko
