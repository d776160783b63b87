// linear_math.cuh — what the products' kernels share: the norm's arithmetic and what is done
// to the sums (linear.cu, linear_few.cu).
#pragma once

#include <math.h>

#include "layer_ops.cuh"
#include "norm.cuh"
#include "pairs.cuh"
#include "sm103.cuh"

namespace dllm {

// x (s_hi + s_lo) g for 8 elements, correctly rounded to bf16.  t = x g is exact, p = fl(t s_hi) is off by a step or so (half
// of one from its rounding, half from s_lo): its own rounding is the right one unless it lies within two steps of a bf16
// midpoint, as one in 13000 does.
__device__ __forceinline__ uint4 normed8_near(const uint4& u, const uint4& gu, float s_hi, float s_lo) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w}, gw[4] = {gu.x, gu.y, gu.z, gu.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float xf = __uint_as_float(h ? (w[i] & 0xFFFF0000u) : (w[i] << 16));
      const float gv = __uint_as_float(h ? (gw[i] & 0xFFFF0000u) : (gw[i] << 16));
      const float t = __fmul_rn(xf, gv);
      const float p0 = __fmul_rn(t, s_hi);
      const float e0 = __fmaf_rn(t, s_lo, __fmaf_rn(t, s_hi, -p0));
      // a second sum leaves |e| at most half a step, so that p alone decides unless it lies on the midpoint, where the
      // sign of e does
      const float p = __fadd_rn(p0, e0), e = __fsub_rn(e0, __fsub_rn(p, p0));
      const uint32_t bits = __float_as_uint(p);
      const uint32_t rn = __bfloat16_as_ushort(__float2bfloat16_rn(p));
      const bool tie = (bits & 0xFFFFu) == 0x8000u && e != 0.f;
      const uint32_t away = ((e > 0.f) == (p > 0.f)) ? 1u : 0u;
      half[h] = tie ? (bits >> 16) + away : rn;
    }
    o[i] = (half[0] & 0xFFFFu) | (half[1] << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint4 normed8(const uint4& u, const uint4& gu, float s_hi, float s_lo) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w}, gw[4] = {gu.x, gu.y, gu.z, gu.w};
  uint32_t o[4];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = mul2(mul2(unpack2(w[i]), unpack2(gw[i])), {s_hi, s_hi});
    near |= (__float_as_uint(p.x) & 0xFFFFu) - 0x7FFEu <= 4u;
    near |= (__float_as_uint(p.y) & 0xFFFFu) - 0x7FFEu <= 4u;
    o[i] = pack_bf16x2(p.x, p.y);
  }
  return near ? normed8_near(u, gu, s_hi, s_lo) : make_uint4(o[0], o[1], o[2], o[3]);
}

// Add the exact squares of 8 bf16 values to the sums (hi, lo) of two at a time, as sumsq_pair_add does one by one.
__device__ __forceinline__ void sumsq2_add(const uint4& u, float2& hi, float2& lo) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  const float2 minus = {-1.f, -1.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2(w[i]), b = mul2(x, x), a = hi;
    hi = add2(a, b);
    const float2 bp = fma2(a, minus, hi);
    const float2 e = add2(fma2(fma2(bp, minus, hi), minus, a), fma2(bp, minus, b));
    lo = add2(lo, e);
  }
}
// The two sums as one.
__device__ __forceinline__ void sums_of(const float2& hi2, const float2& lo2, float& hi, float& lo) {
  hi = hi2.x;
  lo = lo2.x;
  pair_add(hi, lo, hi2.y, lo2.y);
}

// t / (1 + e^-x), by ex2 and a reciprocal that are each off by about 2^-22 (a division and expf cost four times as much).  Both
// terms of the sum, and t, are taken 2^16 times too small: the reciprocal knows no subnormal numbers, and would otherwise be 0
// from x = -87.3 on, where the value is not yet below bf16's.
__device__ __forceinline__ float times_sigmoid(float t, float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(x, -1.4426950408889634f, -16.f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 0x1p-16f));
  return t * 0x1p-16f * r;
}

// t (1 + erf(t / sqrt 2)) / 2 as max(t, 0) - |t| Q(|t|), Q(x) = erfc(x / sqrt 2) / 2 = e^(-x^2 / 2) R(x), which keeps its relative
// accuracy where t is negative (1 + erf cancels: 4% off at -5).  R falls from 1/2 as 1 / x and is a polynomial of degree 7
// in w = 1 / (1 + 0.35 x): the coefficients of the least relative error up to x = 14.7, 2^-21.5, by exchange of its extrema
// (2^-20.1 with the roundings of w and of the sum); behind that the power of two is zero.  It is 2^8 too large and R as much
// too small, so that ex2, which knows no subnormal numbers, ends below bf16's.  (4096 rows of 1024 x 4096:
// 32.5 us, 40.5 with erff, 65 with erfcf.)
__device__ __forceinline__ float gelu(float t) {
  const float x = fminf(fabsf(t), 16.f);
  float w, e;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fmaf(0.35f, x, 1.f)));
  float r = 1.905061508e-04f;
  r = fmaf(r, w, -7.869832334e-04f);
  r = fmaf(r, w, 9.360692347e-04f);
  r = fmaf(r, w, -6.327957090e-05f);
  r = fmaf(r, w, 6.077258731e-04f);
  r = fmaf(r, w, 5.213141558e-04f);
  r = fmaf(r, w, 5.478762905e-04f);
  r = fmaf(r, w, -1.036428117e-07f);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(x * x, -0.72134752044448170f, 8.f)));
  return fmaf(-x * r, e, t < 0.f ? 0.f : t);  // (a NaN is neither)
}

// (1 + tanh u) / 2 is the sigmoid of 2 u.
template <int ACT>
__device__ __forceinline__ float activate(float t) {
  if (ACT == kActSilu) return times_sigmoid(t, t);
  if (ACT == kActGelu) return gelu(t);
  if (ACT == kActGeluTanh) return times_sigmoid(t, 1.5957691216057308f * (t + 0.044715f * t * t * t));
  return t;
}

__device__ __forceinline__ float bf16_at(const void* p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// ------------------------------------------------------------ a few rows (linear_few.cu)
constexpr int few_rows(int k) { return k <= 4096 ? 2 : k <= 16384 ? 1 : 0; }  // how many it takes
cudaError_t launch_linear_few(const LinearArgs& a, int num_sms, cudaStream_t stream);

}  // namespace dllm
