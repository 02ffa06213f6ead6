// Selective scan, one token for each of B independent streams (sm_100a): scan_fwd.cu's recurrence
// with T = 1.  A pass over the fp32 state [B,C,N] (read once, written once), which bounds it; a
// thread owns 4 states of one channel (16-byte accesses), N/4 neighbouring lanes a channel.  With many
// streams all CTAs fit at once and take the streams in turn, the next two's inputs in flight while two
// are worked on: 512x2560, N = 16, bf16 38.5 us (4.6 TB/s, 72 % of a copy's rate; one stream a thread
// and a CTA 59 us).  A thread reads its states before it writes them, so h_out may be h_in.
#include <algorithm>

#include "mixer.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 256;
constexpr int kSN = 4;
constexpr int kStreams = 2;             // streams per group where there are many
constexpr long long kResident = 148 * 3;  // CTAs the GPU holds at once (72 registers a thread)

template <typename T, int N, int kGroup>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const __grid_constant__ ScanParams p) {
  constexpr int L = N / kSN;
  const unsigned id = blockIdx.x * kThreads + threadIdx.x;  // below 2^31: C N / 4 + 256
  const int sub = (int)(id % L);
  const bool act = id / L < (unsigned)p.C;  // the last CTA's idle lanes stay for the shuffles
  const int c = act ? (int)(id / L) : 0;
  const size_t hrow = (size_t)p.C * N, hcol = (size_t)c * N + sub * kSN;

  // streams b0 .. b0 + kGroup - 1, then those gridDim.y groups on; the next group's inputs are on
  // their way while this one is worked on.  Past the last stream it is read again, and not written.
  struct Group {
    Raw<float, kSN> h[kGroup];
    Raw<T, kSN> b[kGroup], c[kGroup];
    Raw<T, 1> x[kGroup], dt[kGroup], z[kGroup];
  } cur, nx;
  const auto fetch = [&](int b0) {
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const size_t b = (size_t)min(b0 + k, p.B - 1);
      nx.h[k].zero();
      if (p.h_in != nullptr) nx.h[k].load(p.h_in + b * hrow + hcol);
      nx.b[k].load(static_cast<const T*>(p.b) + b * p.ldb + sub * kSN, kSN, p.vec_bc);
      nx.c[k].load(static_cast<const T*>(p.c) + b * p.ldc + sub * kSN, kSN, p.vec_bc);
      nx.x[k].load(static_cast<const T*>(p.x) + b * p.ldx + c);
      nx.dt[k].load(static_cast<const T*>(p.dt) + b * p.lddt + c);
      if (p.z != nullptr) nx.z[k].load(static_cast<const T*>(p.z) + b * p.ldz + c);
    }
  };
  const int step = gridDim.y * kGroup;
  fetch(blockIdx.y * kGroup);
  float r[kSN];
  load_rates<kSN>(p.a_log + (size_t)c * N + sub * kSN, r);
  const float2 a2[2] = {make_float2(r[0], r[1]), make_float2(r[2], r[3])};
  const float bias = p.dt_bias != nullptr ? p.dt_bias[c] : 0.f, dsk = p.d != nullptr ? p.d[c] : 0.f;
  for (int b0 = blockIdx.y * kGroup; b0 < p.B; b0 += step) {
    cur = nx;
    if (b0 + step < p.B) fetch(b0 + step);
    float2 delta[(kGroup + 1) / 2];  // in pairs of streams
#pragma unroll
    for (int k = 0; k < kGroup; k += 2) {
      const int o = k + 1 < kGroup ? k + 1 : k;
      float2 e;
      delta[k / 2] = softplus2(make_float2(cur.dt[k][0] + bias, cur.dt[o][0] + bias), e);
    }
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const float x = cur.x[k][0], dlt = k & 1 ? delta[k / 2].y : delta[k / 2].x;
      const float2 dl = dup2(dlt), dx = dup2(dlt * x);
      float2 h[2], acc = dup2(0.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[i] = fma2(decay2(dl, a2[i]), cur.h[k].pair(i), mul2(dx, cur.b[k].pair(i)));
        acc = fma2(cur.c[k].pair(i), h[i], acc);
      }
      float y = acc.x + acc.y;
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      if (act && b0 + k < p.B) {
        const size_t b = (size_t)(b0 + k);
        store_pairs<2>(p.h_out + b * hrow + hcol, h);
        if (sub == 0) {
          y = fmaf(dsk, x, y);
          if (p.z != nullptr) y *= cur.z[k][0] * sigmoid_ex2(cur.z[k][0]);
          static_cast<T*>(p.y)[b * p.C + c] = IO<T>::from_f(y);
        }
      }
    }
  }
}

template <typename T, int N>
cudaError_t step_n(const ScanParams& p, cudaStream_t st) {
  const long long x = ((long long)p.C * (N / kSN) + kThreads - 1) / kThreads;
  if (x * p.B >= 2 * kStreams * kResident) {  // enough for every resident CTA to take groups of streams in turn
    const long long groups = ((long long)p.B + kStreams - 1) / kStreams;
    const dim3 grid((unsigned)x, (unsigned)std::min({groups, std::max(kResident / x, 1LL), 65535LL}));
    scan_step_kernel<T, N, kStreams><<<grid, kThreads, 0, st>>>(p);
  } else {
    const dim3 grid((unsigned)x, (unsigned)std::min<long long>(p.B, 65535));
    scan_step_kernel<T, N, 1><<<grid, kThreads, 0, st>>>(p);
  }
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
