// Selective scan, one token for each of B independent streams (sm_100a): scan_fwd.cu's recurrence
// with T = 1.  A pass over the fp32 state [B,C,N] (read once, written once), which bounds it; a
// thread owns 4 states of one channel (16-byte accesses), N/4 neighbouring lanes a channel, for
// kStreams streams, whose loads are in flight together and share the channel's rates.  A thread
// reads its states before it writes them, so h_out may be h_in.
#include <algorithm>

#include "launch.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 256;
constexpr int kSN = 4;
constexpr int kManyStreams = 4;     // streams per thread where that still fills the GPU
constexpr long long kFillCtas = 592;  // 4 CTAs of 256 threads on each of 148 SMs

template <typename T, int N, int kStreams>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const __grid_constant__ ScanParams p) {
  constexpr int L = N / kSN;
  const unsigned id = blockIdx.x * kThreads + threadIdx.x;  // below 2^31: C N / 4 + 256
  const int sub = (int)(id % L);
  const bool act = id / L < (unsigned)p.C;  // the last CTA's idle lanes stay for the shuffles
  const int c = act ? (int)(id / L) : 0;
  float r[kSN];
  load_rates<kSN>(p.a_log + (size_t)c * N + sub * kSN, r);
  const float2 a2[2] = {make_float2(r[0], r[1]), make_float2(r[2], r[3])};
  const float bias = p.dt_bias != nullptr ? p.dt_bias[c] : 0.f, dsk = p.d != nullptr ? p.d[c] : 0.f;
  const size_t hrow = (size_t)p.C * N, hcol = (size_t)c * N + sub * kSN;

  // streams b0 .. b0 + kStreams - 1, then those of the next row of CTAs' worth
  for (int b0 = blockIdx.y * kStreams; b0 < p.B; b0 += gridDim.y * kStreams) {
    Raw<float, kSN> h0[kStreams];
    Raw<T, kSN> rb[kStreams], rc[kStreams];
    Raw<T, 1> rx[kStreams], rdt[kStreams], rz[kStreams];
    const float* h_at = p.h_in != nullptr ? p.h_in + (size_t)b0 * hrow + hcol : nullptr;
    const T* b_at = static_cast<const T*>(p.b) + (size_t)b0 * p.ldb + sub * kSN;
    const T* c_at = static_cast<const T*>(p.c) + (size_t)b0 * p.ldc + sub * kSN;
    const T* x_at = static_cast<const T*>(p.x) + (size_t)b0 * p.ldx + c;
    const T* dt_at = static_cast<const T*>(p.dt) + (size_t)b0 * p.lddt + c;
    const T* z_at = p.z != nullptr ? static_cast<const T*>(p.z) + (size_t)b0 * p.ldz + c : nullptr;
#pragma unroll
    for (int k = 0; k < kStreams; ++k) {
      if (k > 0 && b0 + k < p.B) {  // past the last stream: it again, and not written
        if (h_at != nullptr) h_at += hrow;
        b_at += p.ldb;
        c_at += p.ldc;
        x_at += p.ldx;
        dt_at += p.lddt;
        if (z_at != nullptr) z_at += p.ldz;
      }
      h0[k].zero();
      if (h_at != nullptr) h0[k].load(h_at);
      rb[k].load(b_at, kSN, p.vec_bc);
      rc[k].load(c_at, kSN, p.vec_bc);
      rx[k].load(x_at);
      rdt[k].load(dt_at);
      if (z_at != nullptr) rz[k].load(z_at);
    }
    float* ho_at = p.h_out + (size_t)b0 * hrow + hcol;
    T* y_at = static_cast<T*>(p.y) + (size_t)b0 * p.C + c;
#pragma unroll
    for (int k = 0; k < kStreams; ++k) {
      const float x = rx[k][0];
      float2 e;
      const float delta = softplus2(dup2(rdt[k][0] + bias), e).x;
      const float2 dl = dup2(delta), dx = dup2(delta * x);
      float2 h[2], acc = dup2(0.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[i] = fma2(ex2_2(mul2(dl, a2[i])), h0[k].pair(i), mul2(dx, rb[k].pair(i)));
        acc = fma2(rc[k].pair(i), h[i], acc);
      }
      float y = acc.x + acc.y;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      if (act && b0 + k < p.B) {
        store_pairs<2>(ho_at, h);
        if (sub == 0) {
          y = fmaf(dsk, x, y);
          if (z_at != nullptr) y *= rz[k][0] * sigmoid_ex2(rz[k][0]);
          *y_at = IO<T>::from_f(y);
        }
      }
      ho_at += hrow;
      y_at += p.C;
    }
  }
}

template <typename T, int N, int kStreams>
void step_launch(const ScanParams& p, cudaStream_t st) {
  const long long lanes = (long long)p.C * (N / kSN);
  const dim3 grid((unsigned)((lanes + kThreads - 1) / kThreads),
                  (unsigned)std::min<long long>(((long long)p.B + kStreams - 1) / kStreams, 65535));
  scan_step_kernel<T, N, kStreams><<<grid, kThreads, 0, st>>>(p);
}

template <typename T, int N>
cudaError_t step_n(const ScanParams& p, cudaStream_t st) {
  const long long ctas = ((long long)p.C * (N / kSN) + kThreads - 1) / kThreads * p.B;  // one stream per thread
  if (ctas >= kManyStreams * kFillCtas)
    step_launch<T, N, kManyStreams>(p, st);
  else
    step_launch<T, N, 1>(p, st);
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
