// Selective scan forward (sm_100a): a diagonal state per channel whose step size, input and output
// weights are data.  Per batch row, channel c and state n,
//   Δ_t = softplus(dt_t + dt_bias),   A = -exp(a_log),
//   h_t[n] = exp(Δ_t A[n]) h_{t-1}[n] + Δ_t x_t B_t[n],
//   p_t = Σ_n C_t[n] h_t[n] + d x_t,   y_t = p_t, or p_t z_t σ(z_t) with a gate z.
// B_t and C_t are shared by all channels of a token.
//
// What bounds it: one exponential per state and token.  With N = 16 an element (b, t, c) moves
// 8 bytes in bf16 but needs 16 ex2, and the special-function unit does 16 a clock and SM, so the
// exponentials take about three times as long as the bytes.
//
// Mapping.  A thread owns 4 states of one channel, N/4 neighbouring lanes a channel; a CTA of 128
// threads owns 512/N channels of one batch row over one time segment, 32 tokens at a time:
//   1. the inputs of a tile are read in runs of 128/N channels per thread (16 bytes in bf16 with
//      N = 16), a tile ahead in registers; Δ and Δx go to shared memory, so softplus is done once
//      per element and not once per lane, and B, C as fp32 rows;
//   2. each thread walks the 32 tokens; Σ_n over a channel's lanes is folded four tokens at a time
//      (three shuffles for four sums instead of eight), the sums go to shared memory;
//   3. the tile's outputs get d x and the gate and leave in the same runs.
//
// Few channels, long axis: time is cut into segments.  A first launch runs every segment but the
// last from a zero state and keeps the state it reaches and ΣΔ; the state entering segment s is
// then folded from these in order (the decay over a segment is exp(A ΣΔ)) by the CTA that needs
// it, in the second launch, which writes the outputs.  Sums run in a fixed order: the same inputs
// give the same bits.
#include <algorithm>

#include "launch.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;  // tokens per tile
constexpr int kSN = 4;     // states per thread

template <int N>
struct Shape {
  static constexpr int kLanes = N / kSN;                // lanes per channel
  static constexpr int kCh = kThreads / kLanes;         // channels per CTA
  static constexpr int kRun = kCh / (kThreads / kTile); // channels per thread in the tile's loads
  static constexpr int kSt = N / (kThreads / kTile);    // states per thread in the tile's loads
};

template <int N>
struct __align__(16) Smem {
  float2 dx[kTile][Shape<N>::kCh];      // (Δ, Δ x)
  float b[kTile][N], c[kTile][N];
  float y[kTile][Shape<N>::kCh + 8];    // Σ_n C h; rows 8 words apart from a multiple of 32 banks
};

// One tile's inputs in registers, as loaded.
template <typename T, int N>
struct Tile {
  float x[Shape<N>::kRun], dt[Shape<N>::kRun], z[Shape<N>::kRun], b[Shape<N>::kSt], c[Shape<N>::kSt];
};

template <typename T, int N, bool OUT>
__device__ __forceinline__ void load_tile(Tile<T, N>& R, const ScanParams& p, int bb, int t, int t1, int c0, int nc,
                                          int s0) {
  constexpr int RUN = Shape<N>::kRun, ST = Shape<N>::kSt;
  const bool ok = t < t1;
  const size_t row = (size_t)bb * p.T + (ok ? t : 0);
  const int n = ok ? nc : 0;
  load_part<T, RUN>(static_cast<const T*>(p.x) + row * p.ldx + c0, n, p.vec, R.x);
  load_part<T, RUN>(static_cast<const T*>(p.dt) + row * p.lddt + c0, n, p.vec, R.dt);
  load_part<T, ST>(static_cast<const T*>(p.b) + row * p.ldb + s0, ok ? ST : 0, p.vec_bc, R.b);
  if constexpr (OUT) {
    if (p.z != nullptr) load_part<T, RUN>(static_cast<const T*>(p.z) + row * p.ldz + c0, n, p.vec, R.z);
    load_part<T, ST>(static_cast<const T*>(p.c) + row * p.ldc + s0, ok ? ST : 0, p.vec_bc, R.c);
  }
}

// OUT: the pass that writes outputs; else the summary pass (states and ΣΔ at the segments' ends).
template <typename T, int N, bool OUT>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(const __grid_constant__ ScanParams p) {
  using S = Shape<N>;
  constexpr int L = S::kLanes, CH = S::kCh, RUN = S::kRun, ST = S::kSt;
  __shared__ Smem<N> sm;
  const int tid = threadIdx.x;
  const int ct = (int)(blockIdx.x % (unsigned)p.ctiles);
  const unsigned rest = blockIdx.x / (unsigned)p.ctiles;
  const int nseg = OUT ? p.nseg : p.nseg - 1;  // the last segment's summary is not needed
  const int seg = (int)(rest % (unsigned)nseg), bb = (int)(rest / (unsigned)nseg);
  const int t0 = seg * p.seg_len, t1 = min(p.T, t0 + p.seg_len);

  // the scan's view: 4 states of one channel
  const int ch = tid / L, sub = tid % L;
  const int c = ct * CH + ch;
  const bool cact = c < p.C;
  const size_t hoff = ((size_t)bb * p.C + c) * N + sub * kSN;  // in a [B,C,N] state
  const size_t plane = (size_t)p.B * p.C * N;
  float a2[kSN], h[kSN];
#pragma unroll
  for (int i = 0; i < kSN; ++i) a2[i] = h[i] = 0.f;
  if (cact) {
    load_rates<kSN>(p.a_log + (size_t)c * N + sub * kSN, a2);
    if (OUT && seg > 0) {
      load_vec<float, kSN>(p.seg_h + hoff, h);  // segment 0's summary starts from h_in
      for (int s = 1; s < seg; ++s) {
        float x[kSN];
        load_vec<float, kSN>(p.seg_h + (size_t)s * plane + hoff, x);
        const float sd = p.seg_dt[((size_t)s * p.B + bb) * p.C + c];
#pragma unroll
        for (int i = 0; i < kSN; ++i) h[i] = fmaf(ex2(sd * a2[i]), h[i], x[i]);
      }
    } else if (seg == 0) {
      // with segments the first launch keeps a copy of h_in, which the second reads: h_out may be
      // the same array, and another CTA of the second launch writes it
      const float* hi = OUT && p.nseg > 1 ? p.seg_h0 : p.h_in;
      if (p.h_in != nullptr) load_vec<float, kSN>(hi + hoff, h);
      if (!OUT && p.h_in != nullptr) store_vec<float, kSN>(p.seg_h0 + hoff, h);
    }
  }

  // the loads' view: one token of the tile, a run of channels, a run of states
  const int lt = tid / (kThreads / kTile), lq = tid % (kThreads / kTile);
  const int c0 = ct * CH + lq * RUN, nc = max(0, min(RUN, p.C - c0));
  float bias[RUN], dsk[RUN];
#pragma unroll
  for (int i = 0; i < RUN; ++i) {
    bias[i] = p.dt_bias != nullptr && i < nc ? p.dt_bias[c0 + i] : 0.f;
    dsk[i] = OUT && p.d != nullptr && i < nc ? p.d[c0 + i] : 0.f;
  }
  Tile<T, N> R;
  load_tile<T, N, OUT>(R, p, bb, t0 + lt, t1, c0, nc, lq * ST);
  float sumdt = 0.f;

  for (int ts = t0; ts < t1; ts += kTile) {
    const bool tact = ts + lt < t1;
    float x[RUN], z[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      float sig, delta = softplus(R.dt[i] + bias[i], sig);
      if (!tact || i >= nc) delta = 0.f;
      x[i] = R.x[i];
      if constexpr (OUT) z[i] = R.z[i];
      sm.dx[lt][lq * RUN + i] = make_float2(delta, tact && i < nc ? delta * x[i] : 0.f);
    }
    store_vec<float, ST>(&sm.b[lt][lq * ST], R.b);
    if constexpr (OUT) store_vec<float, ST>(&sm.c[lt][lq * ST], R.c);
    if (ts + kTile < t1) load_tile<T, N, OUT>(R, p, bb, ts + kTile + lt, t1, c0, nc, lq * ST);
    __syncthreads();

#pragma unroll 2
    for (int g = 0; g < kTile; g += 4) {
      if constexpr (OUT) {
        if (p.ckpt != nullptr && g % kScanCkLen == 0 && cact && ts + g < t1)
          store_vec<float, kSN>(p.ckpt + (size_t)((ts + g) / kScanCkLen) * plane + hoff, h);
      }
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 dx = sm.dx[g + k][ch];
        float bv[kSN], cv[kSN];
        load_vec<float, kSN>(&sm.b[g + k][sub * kSN], bv);
#pragma unroll
        for (int i = 0; i < kSN; ++i) h[i] = fmaf(ex2(dx.x * a2[i]), h[i], dx.y * bv[i]);
        if constexpr (OUT) {
          load_vec<float, kSN>(&sm.c[g + k][sub * kSN], cv);
          y[k] = fmaf(cv[0], h[0], cv[1] * h[1]) + fmaf(cv[2], h[2], cv[3] * h[3]);
        } else {
          sumdt += dx.x;
        }
      }
      if constexpr (OUT) {
        // y[k] of token g + k summed over the channel's L lanes: lane bits 1 and 0 pick tokens
        if constexpr (L >= 4) {
          fold_lanes<4, L>(y, sub);
          if (sub < 4) sm.y[g + sub][ch] = y[0];
        } else {
          fold_lanes<4, L>(y, sub);
#pragma unroll
          for (int k = 0; k < 4 / L; ++k) sm.y[g + sub * (4 / L) + k][ch] = y[k];
        }
      }
    }
    __syncthreads();

    if constexpr (OUT) {
      if (p.y != nullptr && tact && nc > 0) {
        float o[RUN];
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          o[i] = fmaf(dsk[i], x[i], sm.y[lt][lq * RUN + i]);
          if (p.z != nullptr) o[i] *= z[i] * sigmoid(z[i]);
        }
        store_part<T, RUN>(static_cast<T*>(p.y) + ((size_t)bb * p.T + ts + lt) * p.C + c0, nc, p.vec, o);
      }
    }
  }

  if (cact) {
    if constexpr (OUT) {
      if (seg == p.nseg - 1 && p.h_out != nullptr) store_vec<float, kSN>(p.h_out + hoff, h);
    } else {
      store_vec<float, kSN>(p.seg_h + (size_t)seg * plane + hoff, h);
      if (sub == 0) p.seg_dt[((size_t)seg * p.B + bb) * p.C + c] = sumdt;
    }
  }
}

template <typename T, int N>
cudaError_t fwd_n(ScanParams p, cudaStream_t st) {
  p.ctiles = (p.C + Shape<N>::kCh - 1) / Shape<N>::kCh;
  const unsigned rows = (unsigned)p.ctiles * (unsigned)p.B;
  if (p.nseg > 1) {
    scan_fwd_kernel<T, N, false><<<rows * (unsigned)(p.nseg - 1), kThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  scan_fwd_kernel<T, N, true><<<rows * (unsigned)p.nseg, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_t(const ScanParams& p, cudaStream_t st) {
  switch (p.N) {
    case 8: return fwd_n<T, 8>(p, st);
    case 16: return fwd_n<T, 16>(p, st);
    case 32: return fwd_n<T, 32>(p, st);
    case 64: return fwd_n<T, 64>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int scan_fwd_channels(int N) { return kThreads * kSN / N; }
int scan_tile_tokens() { return kTile; }

cudaError_t launch_scan_fwd(bool bf16, const ScanParams& p, cudaStream_t st) {
  return bf16 ? fwd_t<__nv_bfloat16>(p, st) : fwd_t<float>(p, st);
}

}  // namespace rwkv
