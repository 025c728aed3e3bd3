// Routing of tokens to experts, and its backward.  One wave per token, its logits in
// registers (expert lane + 64 i), no LDS but for groups.
//
//   score    softmax over the experts, or sigmoid
//   choice   the k largest of score + bias, ties to the lower index; with groups, among
//            the experts of the topk_groups groups whose two best sum highest
//   weight   scale * score, or scale * score / (sum of the chosen scores)
//
// An expert whose logit is -inf or NaN is never chosen; where fewer than k are left the
// last slots get id -1 and weight 0.  +inf counts as the largest finite value.
//
// A choice is a comparison, so it must not depend on a rounding: without bias the order
// of the scores is that of the logits, which are compared as they are; with a bias, and
// between groups, scores are formed and compared in 64 bits (two of a thousand experts
// are within 2^-24 of each other in about one token of a thousand, within 2^-53 never).
// The weights are 64-bit too, up to their one rounding: renormalised ones are formed from
// the chosen logits alone, so scores too small for fp32 still have a ratio.
//
// Backward, with q the renormalised score, g = scale * (gradient of the weight):
//   renormalised  softmax  dl = q (g - sum q g)        on the chosen experts, else 0
//                 sigmoid  dl = q (g - sum q g) (1 - score)
//   otherwise     softmax  dl = score (g - sum score g) on all (g = 0 on those not chosen)
//                 sigmoid  dl = g score (1 - score)
//
// Bound by vector instructions: a choice is a maximum over the wave for each of the k, a score an
// fp64 exponential.  One token of 64 experts takes 2.8 us (a launch); 8192 tokens, 8 of 256
// experts each, fp32: 8.4-8.7 us by the logits, 13.5 (sigmoid) and 15.3 (softmax) with a bias (64-bit
// keys), 18.2 and 19.9 with groups too, for a read of 8 MB; their backward 7.9-8.9.  (32-bit keys where
// all of a token's values differ in them, with the rest as before, and sorted lists per lane: sigmoid
// with groups 17.5 to 18.9.)
#include "epilogue.h"
#include "w4a16_device.h"
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

constexpr int kTokens = 4;  // waves, and so tokens, per workgroup

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}

// The largest v of the wave, in every lane (row shifts, then broadcasts of rows' last
// lanes: the maximum gathers in lane 63).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp<0x111, 0xf>(v));
  v = max(v, dpp<0x112, 0xf>(v));
  v = max(v, dpp<0x114, 0xf>(v));
  v = max(v, dpp<0x118, 0xf>(v));
  v = max(v, dpp<0x142, 0xa>(v));
  v = max(v, dpp<0x143, 0xc>(v));
  return __builtin_amdgcn_readlane(v, 63);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Unsigned keys in the order of the values (0: not to be chosen; no finite value's key
// is 0).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);  // -0 as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
  return u >> 63 ? ~u : u | (uint64_t)1 << 63;
}

__device__ __forceinline__ uint32_t wave_max_key(uint32_t k) { return wave_max(k); }
__device__ __forceinline__ uint64_t wave_max_key(uint64_t k) {
  const uint32_t hi = wave_max((uint32_t)(k >> 32));
  const uint32_t lo = wave_max((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ double key_value(uint64_t k) {
  return __builtin_bit_cast(double, k >> 63 ? k & ~((uint64_t)1 << 63) : ~k);
}

template <int TYPE>  // 0 fp16, 1 bf16, 2 fp32
__device__ __forceinline__ float load_logit(const void *p, size_t i) {
  if constexpr (TYPE == 2)
    return static_cast<const float *>(p)[i];
  else
    return act_to_f32<TYPE == 1>(static_cast<const uint16_t *>(p)[i]);
}

// A token's logits: -inf where there is none to choose.
template <int TYPE, int VPL>
__device__ __forceinline__ void load_logits(const RouteDesc &P, size_t token, int lane, float (&l)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    const float v = e < P.E ? load_logit<TYPE>(P.logits, token * P.E + e) : -INFINITY;
    l[i] = v != v ? -INFINITY : fminf(v, 3.402823466e38f);
  }
}

__device__ __forceinline__ float wave_max_logit(float v) {
  const uint32_t k = wave_max(key_of(v));
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// exp(l - m), 0 for l = -inf (whatever m)
__device__ __forceinline__ double exp_from(float l, float m) {
  return l == -INFINITY ? 0.0 : exp((double)l - (double)m);
}
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }
// sigmoid(l) / exp(min(m, 0)): in range for l near m, however small both scores are
__device__ __forceinline__ double sigmoid_from(float l, float m) {
  return l == -INFINITY ? 0.0
                        : exp(fmin((double)l, 0.0) - fmin((double)m, 0.0)) / (1.0 + exp(-fabs((double)l)));
}

// What a chosen expert's score is in proportion to, over the chosen ones (their largest
// logit: m).
__device__ __forceinline__ double share(const RouteDesc &P, float l, float m) {
  return P.sigmoid ? sigmoid_from(l, m) : exp_from(l, m);
}

// The k largest keys in order, slot n's expert in lane n (-1: none); ties to the lowest
// expert.
template <int VPL, typename Key>
__device__ __forceinline__ int choose(Key (&key)[VPL], int k, int lane) {
  int id = -1;
  for (int n = 0; n < k; ++n) {
    Key mine = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (key[i] > mine) {
        mine = key[i];
        at = i;
      }
    const Key best = wave_max_key(mine);
    if (best == 0) break;
    // ties: the lowest expert, that is the lowest i, then the lowest lane
    uint64_t hit = __ballot(mine == best);
    if (VPL > 1 && (hit & (hit - 1))) {
      const uint32_t low = ~wave_max(mine == best ? ~(uint32_t)at : 0u);
      hit = __ballot(mine == best && at == (int)low);
    }
    const int owner = __builtin_ctzll(hit);
    const int e = __builtin_amdgcn_readlane(lane + 64 * at, owner);
    if (lane == n) id = e;
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (at == i) key[i] = 0;
    }
  }
  return id;
}

// WIDE: choice by 64-bit values (bias or groups), else by the logits.
template <int TYPE, int VPL, bool WIDE>
__global__ __launch_bounds__(64 * kTokens) void route_kernel(RouteDesc P) {
  typedef std::conditional_t<WIDE, uint64_t, uint32_t> Key;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = blockIdx.x * kTokens + wave;
  if (token >= P.T) return;
  float l[VPL];
  load_logits<TYPE, VPL>(P, token, lane, l);

  // the softmax's largest logit and sum, where a score itself is wanted
  float top = 0.f;
  double inv = 0.0;
  if (!P.sigmoid && (WIDE || !P.renormalize)) {
    float v = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) v = fmaxf(v, l[i]);
    top = wave_max_logit(v);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) s += exp_from(l[i], top);
    inv = 1.0 / wave_sum(s);
  }
  auto score = [&](float x) { return P.sigmoid ? sigmoid64(x) : exp_from(x, top) * inv; };

  Key key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = 0;
    if (l[i] != -INFINITY) {
      if constexpr (WIDE) {
        const int e = lane + 64 * i;
        key[i] = key_of(score(l[i]) + (P.bias ? (double)P.bias[e] : 0.0));
      } else {
        key[i] = key_of(l[i]);
      }
    }
  }

  if constexpr (WIDE) {
    if (P.groups > 1) {
      __shared__ uint64_t keys[kTokens][64 * VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) keys[wave][lane + 64 * i] = key[i];
      // (a wave's own LDS: written and read in order, also by the compiler)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      // `per` lanes a group (a power of two), each over every per-th of its experts
      int per = 64;
      while (per * P.groups > 64) per /= 2;
      const int size = P.E / P.groups, g = lane / per;
      uint64_t b1 = 0, b2 = 0;
      if (g < P.groups) {
        for (int x = lane % per; x < size; x += per) {
          const uint64_t k = keys[wave][g * size + x];
          b2 = max(b2, min(b1, k));
          b1 = max(b1, k);
        }
      }
      for (int o = 1; o < per; o *= 2) {
        const uint64_t c1 = __shfl_xor(b1, o), c2 = __shfl_xor(b2, o);
        b2 = max(max(b2, c2), min(b1, c1));
        b1 = max(b1, c1);
      }
      // a group's value as a key; 0 for one that has no expert to choose
      uint64_t value = b1 == 0 ? 0 : key_of(key_value(b1) + (b2 ? key_value(b2) : 0.0));
      if (g >= P.groups || lane % per) value = 0;
      uint64_t kept = 0;
      for (int n = 0; n < P.topk_groups; ++n) {
        const uint64_t best = wave_max_key(value);
        if (best == 0) break;
        const int first = __builtin_ctzll(__ballot(value == best));
        kept |= (uint64_t)1 << (first / per);
        if (lane == first) value = 0;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i)  // (past E, where the keys are 0, groups may be numbered 64 and more)
        if (!(kept >> ((lane + 64 * i) / size & 63) & 1)) key[i] = 0;
    }
  }

  // slot n's expert, in lane n: without a bias by the logits, which order the scores
  int id;
  if (WIDE && P.bias) {
    id = choose(key, P.k, lane);
  } else {
    uint32_t by_logit[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) by_logit[i] = key[i] ? key_of(l[i]) : 0u;
    id = choose(by_logit, P.k, lane);
  }
  const float lid = id < 0 ? -INFINITY : fminf(load_logit<TYPE>(P.logits, (size_t)token * P.E + id), 3.402823466e38f);

  double w;
  if (P.renormalize) {
    const float m = wave_max_logit(lid);
    w = share(P, lid, m);
    const double sum = wave_sum(lane < P.k ? w : 0.0);
    w = sum > 0.0 ? w / sum : 0.0;
  } else {
    w = id < 0 ? 0.0 : score(lid);
  }
  if (lane < P.k) {
    P.ids[(size_t)token * P.k + lane] = id;
    P.weights[(size_t)token * P.k + lane] = (float)(w * (double)P.scale);
  }
}

template <int TYPE, int VPL>
__global__ __launch_bounds__(64 * kTokens) void route_grad_kernel(RouteDesc P) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = blockIdx.x * kTokens + wave;
  if (token >= P.T) return;
  float l[VPL];
  load_logits<TYPE, VPL>(P, token, lane, l);
  // slot n in lane n; ids outside 0 .. E - 1 have no gradient
  int id = -1;
  double g = 0.0;
  float lid = -INFINITY;
  if (lane < P.k) {
    id = P.ids[(size_t)token * P.k + lane];
    if (id >= 0 && id < P.E) {
      g = (double)P.scale * (double)P.dweights[(size_t)token * P.k + lane];
      const float v = load_logit<TYPE>(P.logits, (size_t)token * P.E + id);
      lid = v != v ? -INFINITY : fminf(v, 3.402823466e38f);
    } else {
      id = -1;
    }
  }
  if (P.renormalize) {
    const float m = wave_max_logit(lid);
    const double s = share(P, lid, m);
    const double sum = wave_sum(s);
    const double q = sum > 0.0 ? s / sum : 0.0;
    g = q * (g - wave_sum(q > 0.0 ? q * g : 0.0));
    if (P.sigmoid) g *= sigmoid64(-lid);
    if (q == 0.0) g = 0.0;
  } else if (P.sigmoid) {
    g = lid == -INFINITY ? 0.0 : g * sigmoid64(lid) * sigmoid64(-lid);
  }
  double d[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) d[i] = 0.0;
  for (int n = 0; n < P.k; ++n) {  // (an id given twice gets both, in order)
    const int e = __builtin_amdgcn_readlane(id, n);
    const uint64_t bits = __builtin_bit_cast(uint64_t, g);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)bits, n);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(bits >> 32), n);
    const double ge = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e == lane + 64 * i) d[i] += ge;
  }
  if (!P.renormalize && !P.sigmoid) {
    float v = l[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) v = fmaxf(v, l[i]);
    const float top = wave_max_logit(v);
    double p[VPL], s = 0.0, a = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      p[i] = exp_from(l[i], top);
      s += p[i];
      a += p[i] > 0.0 ? p[i] * d[i] : 0.0;
    }
    s = wave_sum(s);
    const double inv = s > 0.0 ? 1.0 / s : 0.0;
    a = wave_sum(a) * inv;
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = p[i] > 0.0 ? p[i] * inv * (d[i] - a) : 0.0;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 64 * i;
    if (e >= P.E) continue;
    const size_t at = (size_t)token * P.E + e;
    if constexpr (TYPE == 2)
      static_cast<float *>(P.dlogits)[at] = (float)d[i];
    else  // one rounding from 64 bits: through fp32 in two, the first far below the second
      static_cast<uint16_t *>(P.dlogits)[at] = f32_to_act<TYPE == 1>((float)d[i]);
  }
}

template <int TYPE, int VPL>
void launch_route_size(const RouteDesc &d, bool grad, hipStream_t stream) {
  const dim3 grid((unsigned)((d.T + kTokens - 1) / kTokens)), th(64 * kTokens);
  if (grad)
    hipLaunchKernelGGL((route_grad_kernel<TYPE, VPL>), grid, th, 0, stream, d);
  else if (d.bias || d.groups > 1)
    hipLaunchKernelGGL((route_kernel<TYPE, VPL, true>), grid, th, 0, stream, d);
  else
    hipLaunchKernelGGL((route_kernel<TYPE, VPL, false>), grid, th, 0, stream, d);
}

template <int TYPE>
void launch_route_typed(const RouteDesc &d, bool grad, hipStream_t stream) {
  if (d.E <= 64)
    launch_route_size<TYPE, 1>(d, grad, stream);
  else if (d.E <= 128)
    launch_route_size<TYPE, 2>(d, grad, stream);
  else if (d.E <= 256)
    launch_route_size<TYPE, 4>(d, grad, stream);
  else if (d.E <= 512)
    launch_route_size<TYPE, 8>(d, grad, stream);
  else
    launch_route_size<TYPE, 16>(d, grad, stream);
}

}  // namespace

hipError_t launch_route(const RouteDesc &d, bool grad, hipStream_t stream) {
  if (d.T == 0) return hipSuccess;
  if (d.type == 2)
    launch_route_typed<2>(d, grad, stream);
  else if (d.type == 1)
    launch_route_typed<1>(d, grad, stream);
  else
    launch_route_typed<0>(d, grad, stream);
  return hipGetLastError();
}

}  // namespace w4a16
