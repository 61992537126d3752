// The router of one token, by one warp: shared by the routing kernels (route.cu)
// and the few-token experts (few_experts.cu), which route in each of their CTAs.
// route.cu describes the selection and the fixed IEEE sequences.
#pragma once

#include "ieee_math.cuh"
#include "moe_common.cuh"

namespace moe {

__device__ __forceinline__ float tanh_ieee(float t) {
  float a = fabsf(t);
  float y;
  if (a >= 10.0f) {
    y = 1.0f;
  } else if (a < 0.5f) {
    float s = __fmul_rn(a, a);
    // tanh Taylor coefficients of t^17 down to t^3
    float q = f32_bits(0x3a1aac12u);
    q = __fmaf_rn(q, s, f32_bits(0xbabed1b2u));
    q = __fmaf_rn(q, s, f32_bits(0x3b6b69e8u));
    q = __fmaf_rn(q, s, f32_bits(0xbc11371bu));
    q = __fmaf_rn(q, s, f32_bits(0x3cb327a4u));
    q = __fmaf_rn(q, s, f32_bits(0xbd5d0dd1u));
    q = __fmaf_rn(q, s, f32_bits(0x3e088889u));
    q = __fmaf_rn(q, s, f32_bits(0xbeaaaaabu));
    y = __fmaf_rn(__fmul_rn(a, s), q, a);
  } else {
    float e = exp_ieee(__fadd_rn(a, a));
    y = __fsub_rn(1.0f, __fdiv_rn(2.0f, __fadd_rn(e, 1.0f)));
  }
  return signbit(t) ? -y : y;
}

// Order-preserving map of a binary32 value to an unsigned key: larger value,
// larger key.  -0.0 is first made +0.0 so that the two zeros tie (and the
// lower expert id wins), as they do under floating-point comparison.
__device__ __forceinline__ uint32_t order_key(float z) {
  uint32_t u = __float_as_uint(z == 0.0f ? 0.0f : z);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// z = softcap * tanh(logit / softcap), or the logit itself (softcap 0).
__device__ __forceinline__ float cap_logit(float l, float softcap) {
  return softcap > 0.0f ? __fmul_rn(softcap, tanh_ieee(__fdiv_rn(l, softcap))) : l;
}

// Selects one token's experts from its capped logits with one warp.  NPL = experts per lane
// (E <= 32 * NPL); lane l owns experts l, l+32, ... (z of those past E is not used).
template <int NPL>
__device__ __forceinline__ int route_select(const float (&z)[NPL], int E, int k, int renorm,
                                            int32_t* __restrict__ ids,
                                            float* __restrict__ weights) {
  const int lane = threadIdx.x & 31;
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    key[i] = lane + 32 * i < E ? order_key(z[i]) : 0u;  // key 0: below every real value

  // this lane's best remaining expert (largest key; the first one wins ties,
  // which is the lowest id because ids grow with i)
  uint32_t hk = 0u;
  int hi = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i)
    if (key[i] > hk) {
      hk = key[i];
      hi = i;
    }

  float my_z = 0.0f;  // lane j keeps the j-th selected value and id
  int my_id = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, hk);
    const uint32_t cand =
        (hk == best && best != 0u) ? static_cast<uint32_t>(lane + 32 * hi) : 0xffffffffu;
    const uint32_t win = __reduce_min_sync(0xffffffffu, cand);
    const int owner = static_cast<int>(win & 31u);
    float zv = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (i == hi) zv = z[i];
    zv = __shfl_sync(0xffffffffu, zv, owner);
    if (lane == j) {
      my_z = zv;
      my_id = static_cast<int>(win);
    }
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == hi) key[i] = 0u;
      hk = 0u;
      hi = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (key[i] > hk) {
          hk = key[i];
          hi = i;
        }
    }
  }
  const float z0 = __shfl_sync(0xffffffffu, my_z, 0);

  float my_e = 0.0f;
  if (lane < k) my_e = exp_ieee(__fsub_rn(my_z, z0));
  float s = 0.0f;
  if (renorm) {
    for (int j = 0; j < k; ++j) s = __fadd_rn(s, __shfl_sync(0xffffffffu, my_e, j));
  } else {
    // sum over all experts in expert-id order
    for (int e = 0; e < E; ++e) {
      float mine = 0.0f;
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (i == (e >> 5)) mine = z[i];
      const float ze = __shfl_sync(0xffffffffu, mine, e & 31);
      s = __fadd_rn(s, exp_ieee(__fsub_rn(ze, z0)));
    }
  }
  if (lane < k) {
    ids[lane] = my_id;
    weights[lane] = __fdiv_rn(my_e, s);
  }
  return my_id;  // lane j < k: the j-th selected expert
}

// Routes one token with one warp.
template <int NPL>
__device__ __forceinline__ int route_token(const float* __restrict__ row, int E, int k,
                                           float softcap, int renorm, int32_t* __restrict__ ids,
                                           float* __restrict__ weights) {
  const int lane = threadIdx.x & 31;
  float z[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    z[i] = e < E ? __ldg(row + e) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NPL; ++i) z[i] = cap_logit(z[i], softcap);
  return route_select<NPL>(z, E, k, renorm, ids, weights);
}

}  // namespace moe
