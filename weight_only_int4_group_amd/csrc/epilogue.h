// Fused epilogues: what a product goes through before it is stored once.
//
//   linear  Y = residual + act(Z),       Z = X . W_hat^T + bias
//   gated   H = act(G) * U,              G and U the products with two weights
//
// The fp32 sums stay in fp32 up to the one rounding of each output; Z (or G
// and U), when the caller keeps them for a backward pass, are rounded once from
// the same sums, and Y is formed from the unrounded ones.
//
// Activations (act_value) and their derivatives (act_grad):
//   relu       max(z, 0); derivative 1 for z > 0, else 0
//   silu       z * sg(z), sg(z) = 1 / (1 + exp(-z));  sg + z sg (1 - sg)
//   gelu       z Phi(z), Phi the normal distribution function;  Phi(z) + z phi(z)
//   gelu_tanh  z (1 + tanh u) / 2 = z sg(2u), u = sqrt(2 / pi) (z + 0.044715 z^3);
//              sg(2u) + z sg(2u) (1 - sg(2u)) 2 u'
// sg takes the hardware reciprocal (1 ulp of fp32, 2^-23 relative): far below the
// 2^-11 or 2^-8 of the output's rounding.
#pragma once

#include "w4a16_device.h"

namespace w4a16 {

enum Act { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };
constexpr int kActs = 5;

// One problem's epilogue.  bias [N], residual, pre [M][N] are of the activations'
// type, each null when absent.  gated: the second weight (the "up" matrix, same
// shape as the first), its bias, pre-activation output and outliers.  part, ldx:
// set by the streaming launcher for one K range of a problem: the fp32 sums go to
// part [M][N] (gated: [M][2 N], the two weights' 16-column blocks alternating)
// instead of the epilogue, and X's rows are ldx apart (0: K).
struct Fused {
  const void *bias, *residual;
  void *pre;
  int act;
  int gated;
  const uint8_t *Wq2;
  const _Float16 *scales2, *zeros2;
  const void *bias2;
  void *pre2;
  const int32_t *orp2, *ocol2;
  const _Float16 *oval2;
  float *part;
  int ldx;
};

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// Phi(z), with e = exp(-z^2 / 2) given, which the derivative shares:
// Phi(-|z|) = erfcx(x) e / 2, x = |z| / sqrt 2, and erfcx(x) = exp(x^2) erfc(x) =
// c1 t + ... + c8 t^8, t = 1 / (1 + 0.33 x).  The coefficients are a fit of our own
// for the least relative error over 0 <= x <= 9.5 (a linear program on 2500 points):
// 6.4e-8, 2^-23.9.  The error has to be relative: gelu(z) = z Phi(z) is all tail for
// z below -4, and bf16 holds it down to z = -13.  With the fp32 roundings Phi is
// within 2^-19 + (z^2 / 2) 2^-22 of its value, the second part from the rounding
// of the exponent; below z = -13 it leaves fp32's normal range and goes to 0.
// The device library's erfc takes several times the instructions: the gradient of
// a 2048 x 14336 gelu layer took 54-59 us with it and takes 30 as here, the time
// of its bytes (5.9 TB/s).
__device__ __forceinline__ float normal_cdf(float z, float e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.33f * 0.7071067811865476f, fabsf(z), 1.0f));
  float q = __builtin_fmaf(-0.13582322f, t, 0.4623704f);
  q = __builtin_fmaf(q, t, -0.35508668f);
  q = __builtin_fmaf(q, t, 0.41238376f);
  q = __builtin_fmaf(q, t, 0.045012124f);
  q = __builtin_fmaf(q, t, 0.2019472f);
  q = __builtin_fmaf(q, t, 0.18282963f);
  q = __builtin_fmaf(q, t, 0.18636689f);
  const float half_erfc = 0.5f * q * t * e;
  return z > 0.f ? 1.0f - half_erfc : half_erfc;
}

// 2u of gelu_tanh: 2 sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu_tanh_2u(float z) {
  return 1.5957691216057308f * __builtin_fmaf(0.044715f * z * z, z, z);
}

__device__ __forceinline__ float act_value(float z, int act) {
  switch (act) {
    case kActRelu: return z > 0.f || z != z ? z : 0.f;  // NaN stays NaN
    case kActSilu: return z * sigmoid(z);
    case kActGelu: return z * normal_cdf(z, __expf(-0.5f * z * z));
    case kActGeluTanh: return z * sigmoid(gelu_tanh_2u(z));
    default: return z;
  }
}

__device__ __forceinline__ float act_grad(float z, int act) {
  switch (act) {
    case kActRelu: return z != z ? z : (z > 0.f ? 1.f : 0.f);
    case kActSilu: {
      const float sg = sigmoid(z);
      return sg * __builtin_fmaf(z, 1.f - sg, 1.f);
    }
    case kActGelu: {
      const float e = __expf(-0.5f * z * z);
      return __builtin_fmaf(z * 0.3989422804014327f, e, normal_cdf(z, e));
    }
    case kActGeluTanh: {
      // past |z| = 16 the derivative is 0 or 1 in fp32; z is held there so that
      // the vanishing factor never meets an overflowed one (NaN stays NaN)
      const float zc = z > 16.f ? 16.f : (z < -16.f ? -16.f : z);
      const float sg = sigmoid(gelu_tanh_2u(zc));
      const float du2 = 1.5957691216057308f * __builtin_fmaf(3.f * 0.044715f * zc, zc, 1.f);
      return __builtin_fmaf(zc * sg * (1.f - sg), du2, sg);
    }
    default: return 1.f;
  }
}

// 16-bit activations of either type
template <bool BF>
__device__ __forceinline__ float act_to_f32(uint16_t h) {
  return BF ? bf16_to_f32(h) : (float)__builtin_bit_cast(_Float16, h);
}
template <bool BF>
__device__ __forceinline__ uint16_t f32_to_act(float v) {
  return BF ? f32_to_bf16(v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}

}  // namespace w4a16
