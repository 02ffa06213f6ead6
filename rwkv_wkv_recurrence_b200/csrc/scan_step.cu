// Selective scan, one token for each of B independent streams (sm_100a): scan_fwd.cu's recurrence
// with T = 1.  A pass over the fp32 state [B,C,N] (read once, written once); a thread owns 4 states
// of one channel (16-byte accesses), N/4 neighbouring lanes a channel.  Each thread reads its states
// before it writes them, so h_out may be h_in.
#include "launch.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 256;
constexpr int kSN = 4;

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const __grid_constant__ ScanParams p) {
  constexpr int L = N / kSN;
  const size_t id = (size_t)blockIdx.x * kThreads + threadIdx.x;
  const size_t bc = id / L;  // (b, c); the last CTA's idle lanes stay for the shuffles
  const int sub = (int)(id % L);
  const bool act = bc < (size_t)p.B * p.C;
  const size_t b = act ? bc / p.C : 0;
  const int c = act ? (int)(bc % p.C) : 0;
  float a2[kSN], h[kSN] = {0.f, 0.f, 0.f, 0.f}, bv[kSN], cv[kSN];
  const size_t hoff = (b * p.C + c) * N + sub * kSN;
  if (p.h_in != nullptr) load_vec<float, kSN>(p.h_in + hoff, h);
  load_rates<kSN>(p.a_log + (size_t)c * N + sub * kSN, a2);
  load_part<T, kSN>(static_cast<const T*>(p.b) + b * p.ldb + sub * kSN, kSN, p.vec_bc, bv);
  load_part<T, kSN>(static_cast<const T*>(p.c) + b * p.ldc + sub * kSN, kSN, p.vec_bc, cv);
  const float x = IO<T>::to_f(static_cast<const T*>(p.x)[b * p.ldx + c]);
  float v = IO<T>::to_f(static_cast<const T*>(p.dt)[b * p.lddt + c]);
  if (p.dt_bias != nullptr) v += p.dt_bias[c];
  float2 e;
  const float delta = softplus2(dup2(v), e).x, dx = delta * x;
  float y = 0.f;
#pragma unroll
  for (int i = 0; i < kSN; ++i) {
    h[i] = fmaf(ex2(delta * a2[i]), h[i], dx * bv[i]);
    y = fmaf(cv[i], h[i], y);
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  if (!act) return;
  store_vec<float, kSN>(p.h_out + hoff, h);
  if (sub == 0) {
    if (p.d != nullptr) y = fmaf(p.d[c], x, y);
    if (p.z != nullptr) {
      const float z = IO<T>::to_f(static_cast<const T*>(p.z)[b * p.ldz + c]);
      y *= z * sigmoid_ex2(z);
    }
    static_cast<T*>(p.y)[b * p.C + c] = IO<T>::from_f(y);
  }
}

template <typename T>
cudaError_t step_t(const ScanParams& p, cudaStream_t st) {
  const size_t n = (size_t)p.B * p.C * (p.N / kSN);
  const unsigned grid = (unsigned)((n + kThreads - 1) / kThreads);
  switch (p.N) {
    case 8: scan_step_kernel<T, 8><<<grid, kThreads, 0, st>>>(p); break;
    case 16: scan_step_kernel<T, 16><<<grid, kThreads, 0, st>>>(p); break;
    case 32: scan_step_kernel<T, 32><<<grid, kThreads, 0, st>>>(p); break;
    case 64: scan_step_kernel<T, 64><<<grid, kThreads, 0, st>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_step(bool bf16, const ScanParams& p, cudaStream_t st) {
  return bf16 ? step_t<__nv_bfloat16>(p, st) : step_t<float>(p, st);
}

}  // namespace rwkv
