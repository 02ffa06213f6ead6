// Device helpers shared by the selective-scan kernels.
#pragma once

#include "mixer_common.cuh"
#include "scan_plan.h"

namespace rwkv {

// softplus(v) = log(1 + e^v) = max(v, 0) + log1p(e^-|v|) of two values.  log1p(e) = e P(e) on
// [0, 1], P the polynomial of degree 9 through log1p(e)/e at the Chebyshev points, without a division:
// itself within 0.24 x 2^-24 of log1p(e), in fp32 arithmetic within 3.4 x 2^-24 by a count of its
// roundings and 2.3 x 2^-24 as evaluated over all e (small steps, e^v far below 1, keep their relative
// accuracy); the approximate e comes on top.  e01 receives e^-|v|.  NaN and the infinities pass through.
__device__ __forceinline__ float2 softplus2(float2 v, float2& e01) {
  const float2 a = make_float2(-fabsf(v.x), -fabsf(v.y));
  const float2 e = ex2_2(fma2(a, dup2(kL2eLo), mul2(a, dup2(kL2eHi))));
  e01 = e;
  float2 r = fma2(e, dup2(-0.0031760570127516985f), dup2(0.019542526453733444f));
  r = fma2(r, e, dup2(-0.056373611092567444f));
  r = fma2(r, e, dup2(0.10543623566627502f));
  r = fma2(r, e, dup2(-0.1526966691017151f));
  r = fma2(r, e, dup2(0.1966327428817749f));
  r = fma2(r, e, dup2(-0.24951615929603577f));
  r = fma2(r, e, dup2(0.33329710364341736f));
  r = fma2(r, e, dup2(-0.49999892711639404f));
  r = fma2(r, e, dup2(1.0f));
  return fma2(r, e, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// exp(Δ A) = 2^(Δ a2) of two states.  A state multiplies by this once per token, so a bias of the
// function builds up over as many tokens as the state remembers; for Δ |A| from 0.001 to 0.5 ex2.approx
// measured 0.27 to 0.35 x 2^-24 too small on average (its largest error is 2^-23; rounding to nearest
// would have no bias).  2^-25 more in the exponent, ln 2 / 2 = 0.35 x 2^-24 in the value, takes that away
// at no cost (0.00 to +0.08 x 2^-24 left); Δ = 0 still gives exactly 1.  Slower decays are mostly near 1,
// where the function is off by less: +0.16 to +0.25 x 2^-24 is left for Δ |A| from 10^-7 to 0.001.
__device__ __forceinline__ float2 decay2(float2 delta, float2 a2) { return ex2_2(fma2(delta, a2, dup2(0x1p-25f))); }

// A log2(e) = -exp(a_log) log2(e) of n states, so that exp(Δ A) = 2^(Δ a2).  A rate beyond the
// largest float counts as that one, which keeps 0 · a2 = 0 at the positions past a segment's end.
template <int K>
__device__ __forceinline__ void load_rates(const float* __restrict__ a_log, float (&a2)[K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const float r = -expf(a_log[i]) * kL2eHi;
    a2[i] = r < -3.402823466e+38f ? -3.402823466e+38f : r;  // a NaN stays
  }
}

// 2 P consecutive floats as pairs (P = 1: 8-byte, else 16-byte accesses).
template <int P>
__device__ __forceinline__ void load_pairs(const float* p, float2 (&v)[P]) {
  if constexpr (P == 1) {
    v[0] = *reinterpret_cast<const float2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const float4 x = *reinterpret_cast<const float4*>(p + 2 * i);
      v[i] = make_float2(x.x, x.y), v[i + 1] = make_float2(x.z, x.w);
    }
  }
}
template <int P>
__device__ __forceinline__ void store_pairs(float* p, const float2 (&v)[P]) {
  if constexpr (P == 1) {
    *reinterpret_cast<float2*>(p) = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < P; i += 2)
      *reinterpret_cast<float4*>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
  }
}

// v[k], k < K, each to be summed over L lanes whose numbers differ in the bits of ST·(L - 1); idx
// is the lane's place among them.  Every shuffle halves the sums a lane holds while it holds more
// than one: lane idx ends with the sums of v[idx·(K/L)] .. in v[0 ..] for L <= K, of
// v[idx mod K] in v[0] for L > K.
template <int K, int L, int ST = 1>
__device__ __forceinline__ void fold_lanes(float (&v)[K], int idx) {
  constexpr int M = L < K ? L : K;  // lanes that end up with different sums
  int n = K;
#pragma unroll
  for (int o = M / 2; o > 0; o >>= 1) {
    n >>= 1;
    const bool up = (idx & o) != 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k >= n) continue;
      const float keep = up ? v[k + n] : v[k], give = up ? v[k] : v[k + n];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o * ST);
    }
  }
#pragma unroll
  for (int o = M; o < L; o <<= 1) {
#pragma unroll
    for (int k = 0; k < K / M; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o * ST);
  }
}

}  // namespace rwkv
