// Selective scan, one token for each of B independent streams (sm_100a): scan_fwd.cu's recurrence
// with T = 1.  A pass over the fp32 state [B,C,N] (read once, written once), which bounds it; a
// thread owns 4 states of one channel (16-byte accesses), N/4 neighbouring lanes a channel, for
// kStreams streams, whose loads are in flight together and share the channel's rates.  A thread
// reads its states before it writes them, so h_out may be h_in.
#include "launch.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 256;
constexpr int kSN = 4;
constexpr int kManyStreams = 4;     // streams per thread where that still fills the GPU
constexpr unsigned kFillCtas = 592;  // 4 CTAs of 256 threads on each of 148 SMs

template <typename T, int N, int kStreams>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const __grid_constant__ ScanParams p) {
  constexpr int L = N / kSN;
  const size_t id = (size_t)blockIdx.x * kThreads + threadIdx.x;
  const int sub = (int)(id % L);
  const size_t q = id / L;  // (group of streams, channel); the last CTA's idle lanes stay for the shuffles
  const size_t b0 = q / p.C * kStreams;
  const bool act = b0 < (size_t)p.B;
  const int c = (int)(q % p.C);
  float2 h[kStreams][2], bv[kStreams][2], cv[kStreams][2];
  float x[kStreams], dt[kStreams], z[kStreams];
#pragma unroll
  for (int k = 0; k < kStreams; ++k) {
    const size_t b = act && b0 + k < (size_t)p.B ? b0 + k : 0;  // past the last stream: stream 0 again, not written
    h[k][0] = h[k][1] = dup2(0.f);
    if (p.h_in != nullptr) load_pairs<2>(p.h_in + (b * p.C + c) * N + sub * kSN, h[k]);
    Raw<T, kSN> rb, rc;
    rb.load(static_cast<const T*>(p.b) + b * p.ldb + sub * kSN, kSN, p.vec_bc);
    rc.load(static_cast<const T*>(p.c) + b * p.ldc + sub * kSN, kSN, p.vec_bc);
    x[k] = IO<T>::to_f(static_cast<const T*>(p.x)[b * p.ldx + c]);
    dt[k] = IO<T>::to_f(static_cast<const T*>(p.dt)[b * p.lddt + c]);
    if (p.z != nullptr) z[k] = IO<T>::to_f(static_cast<const T*>(p.z)[b * p.ldz + c]);
#pragma unroll
    for (int i = 0; i < 2; ++i) bv[k][i] = rb.pair(i), cv[k][i] = rc.pair(i);
  }
  float r[kSN];
  load_rates<kSN>(p.a_log + (size_t)c * N + sub * kSN, r);
  const float2 a2[2] = {make_float2(r[0], r[1]), make_float2(r[2], r[3])};
  const float bias = p.dt_bias != nullptr ? p.dt_bias[c] : 0.f, dsk = p.d != nullptr ? p.d[c] : 0.f;
#pragma unroll
  for (int k = 0; k < kStreams; ++k) {
    float2 e;
    const float delta = softplus2(dup2(dt[k] + bias), e).x;
    const float2 dl = dup2(delta), dx = dup2(delta * x[k]);
    float2 acc = dup2(0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      h[k][i] = fma2(ex2_2(mul2(dl, a2[i])), h[k][i], mul2(dx, bv[k][i]));
      acc = fma2(cv[k][i], h[k][i], acc);
    }
    float y = acc.x + acc.y;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (!act || b0 + k >= (size_t)p.B) continue;
    const size_t b = b0 + k;
    store_pairs<2>(p.h_out + (b * p.C + c) * N + sub * kSN, h[k]);
    if (sub == 0) {
      y = fmaf(dsk, x[k], y);
      if (p.z != nullptr) y *= z[k] * sigmoid_ex2(z[k]);
      static_cast<T*>(p.y)[b * p.C + c] = IO<T>::from_f(y);
    }
  }
}

template <typename T, int N>
cudaError_t step_n(const ScanParams& p, cudaStream_t st) {
  const auto grid = [&](int streams) {
    const size_t n = ((size_t)p.B + streams - 1) / streams * p.C * (N / kSN);
    return (unsigned)((n + kThreads - 1) / kThreads);
  };
  if (grid(kManyStreams) >= kFillCtas)
    scan_step_kernel<T, N, kManyStreams><<<grid(kManyStreams), kThreads, 0, st>>>(p);
  else
    scan_step_kernel<T, N, 1><<<grid(1), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t step_t(const ScanParams& p, cudaStream_t st) {
  switch (p.N) {
    case 8: return step_n<T, 8>(p, st);
    case 16: return step_n<T, 16>(p, st);
    case 32: return step_n<T, 32>(p, st);
    case 64: return step_n<T, 64>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_scan_step(bool bf16, const ScanParams& p, cudaStream_t st) {
  return bf16 ? step_t<__nv_bfloat16>(p, st) : step_t<float>(p, st);
}

}  // namespace rwkv
