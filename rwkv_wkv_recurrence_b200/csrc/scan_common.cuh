// Device helpers shared by the selective-scan kernels.
#pragma once

#include "mixer_common.cuh"

namespace rwkv {

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
