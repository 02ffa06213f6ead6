// Layer norm over the N columns of each of G groups of a row, with an optional SiLU gate (sm_100a):
//   x̂ = (x - mean x) / sqrt(var x + eps),   l = x̂ w + b,   y = l, or l · s(z) with s(z) = z σ(z).
// G = 1 is the norm in front of a block's mixers ("RWKV - Transformer 시대에 RNN을 재발명하다",
// architecture: LN before time mixing and channel mixing); G = H, N = 64 the head-wise norm and the
// gate behind the Eagle and Finch operators ("RWKV-5 Eagle과 RWKV-6 Finch", section Eagle).
//
// Backward, with g = gy s(z) (or gy) and u = g w:
//   gx = (u - mean u - x̂ mean(u x̂)) / sqrt(var x + eps),   gw = Σ_rows g x̂,   gb = Σ_rows g,
//   gz = gy l s'(z),   s'(z) = σ(z)(1 + z (1 - σ(z))).
// The mean and variance are formed again from x, which the backward reads anyway: keeping them
// would save no pass over the data.
//
// One pass over the data, so bandwidth bounds it.  A team of 8 to 512 threads holds one group of a
// row in registers (1 or 2 vectors a thread): the variance is the mean of (x - mean)², not a
// difference of large sums.  A team keeps its group and strides over the rows, so w and b, and the
// backward's column sums, stay in registers; teams of neighbouring groups are neighbours, so a
// CTA's accesses are contiguous.  Column sums go to the workspace per team and are added in order
// by a second kernel: no atomics, the same inputs give the same bits.  Groups wider than 1024
// vectors take a kernel that reads the row again for each sum (from L1 / L2).
#include <algorithm>

#include "launch.h"
#include "mixer_common.cuh"

namespace rwkv {
namespace {

constexpr int kMaxTeam = 512;
constexpr int kTargetThreads = 148 * 1536;  // threads a launch aims at (three quarters of what the SMs hold)

// Sums a and b over a team; every thread gets them.  Teams wider than a warp are whole CTAs; `buf`
// alternates between two halves, so one barrier a call is enough.
template <int TS>
struct TeamSum {
  float2* buf;
  int phase = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
    constexpr int W = TS < 32 ? TS : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TS > 32) {
      constexpr int NW = TS / 32;
      float2* s = buf + phase * NW;
      phase ^= 1;
      if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
      __syncthreads();
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        a += s[i].x;
        b += s[i].y;
      }
    }
    return make_float2(a, b);
  }
};

template <int TS>
constexpr int kCtaThreads = TS > 32 ? TS : 256;

// Where a team works: its group, first row, row stride.
template <int TS>
struct Team {
  int lane, g;
  long long m, step, turns;
  __device__ __forceinline__ explicit Team(const NormParams& p) {
    constexpr int PER = kCtaThreads<TS> / TS;
    lane = threadIdx.x % TS;
    const long long id = (long long)blockIdx.x * PER + threadIdx.x / TS;
    g = (int)(id % p.G);
    m = id / p.G;
    step = p.slices;
    // a team past the last slice has no rows; teams of a warp's width or less share a warp with
    // others, whose shuffles they take part in: all take as many turns as the first slice
    turns = TS > 32 ? (p.M - m + step - 1) / step : (p.M + step - 1) / step;
    if (m >= step) m = p.M;
  }
};

// A lane's part of a row as loaded: vectors k = 0 .. K-1 at columns (k TS + lane) V (zeros past N).
template <typename T, int V, int K, int TS>
struct RowPart {
  Raw<T, V> v[K];
  __device__ __forceinline__ void load(const void* base, size_t off, int lane, int N) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int col = (k * TS + lane) * V;
      v[k].load(static_cast<const T*>(base) + off + col, col < N ? V : 0, true);
    }
  }
};

// Parameters of a group in the same places.
template <int V, int K, int TS>
__device__ __forceinline__ void load_params(const float* row, int lane, int N, float (&f)[K][V]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int col = (k * TS + lane) * V;
    if (row != nullptr && col < N) {
      load_vec<float, V>(row + col, f[k]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[k][i] = 0.f;
    }
  }
}

// x - mean (0 past column N); returns 1 / sqrt(var + eps).
template <typename T, int V, int K, int TS>
__device__ __forceinline__ float center(const RowPart<T, V, K, TS>& r, float (&x)[K][V], int lane, int N, float inv_n,
                                        float eps, TeamSum<TS>& sum) {
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) s += x[k][i] = r.v[k][i];
  const float mean = sum(s, 0.f).x * inv_n;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float mk = (k * TS + lane) * V < N ? mean : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[k][i] -= mk;
      q = fmaf(x[k][i], x[k][i], q);
    }
  }
  return 1.f / sqrtf(fmaf(sum(q, 0.f).x, inv_n, eps));
}

// Rows are fetched a turn ahead and left as loaded until they are due.
template <typename T, int V, int K, int TS, bool GATE>
__global__ void __launch_bounds__(kCtaThreads<TS>) norm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 buf[2 * kMaxTeam / 32];
  TeamSum<TS> sum{buf};
  const Team<TS> tm(p);
  const float inv_n = 1.f / (float)p.N;
  float w[K][V], b[K][V];
  const size_t stride = (size_t)tm.step * p.G * p.N;
  size_t off = ((size_t)tm.m * p.G + tm.g) * p.N;
  long long m = tm.m;
  RowPart<T, V, K, TS> rx, rz;
  const auto fetch = [&](size_t o, bool on) {
    rx.load(p.x, on ? o : 0, tm.lane, on ? p.N : 0);
    if constexpr (GATE) rz.load(p.gate, on ? o : 0, tm.lane, on ? p.N : 0);
  };
  fetch(off, m < p.M);
  load_params<V, K, TS>(p.weight + (size_t)tm.g * p.N, tm.lane, p.N, w);
  load_params<V, K, TS>(p.bias != nullptr ? p.bias + (size_t)tm.g * p.N : nullptr, tm.lane, p.N, b);
  for (long long it = 0; it < tm.turns; ++it, m += tm.step, off += stride) {
    const bool on = m < p.M;
    const RowPart<T, V, K, TS> cx = rx, cz = rz;
    fetch(off + stride, m + tm.step < p.M);
    float x[K][V];
    const float rstd = center<T, V, K, TS>(cx, x, tm.lane, p.N, inv_n, p.eps, sum);
    if (!on) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int col = (k * TS + tm.lane) * V;
      if (col >= p.N) continue;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] = fmaf(x[k][i] * rstd, w[k][i], b[k][i]);
        if constexpr (GATE) {
          const float z = cz.v[k][i];
          o[i] *= z * sigmoid_ex2(z);
        }
      }
      store_vec<T, V>(static_cast<T*>(p.y) + off + col, o);
    }
  }
}

template <typename T, int V, int K, int TS, bool GATE>
__global__ void __launch_bounds__(kCtaThreads<TS>) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 buf[2 * kMaxTeam / 32];
  TeamSum<TS> sum{buf};
  const Team<TS> tm(p);
  const float inv_n = 1.f / (float)p.N;
  float w[K][V], b[K][V], gw[K][V], gb[K][V];
  const size_t stride = (size_t)tm.step * p.G * p.N;
  size_t off = ((size_t)tm.m * p.G + tm.g) * p.N;
  long long m = tm.m;
  RowPart<T, V, K, TS> rx, rg, rz;
  const auto fetch = [&](size_t o, bool on) {
    rx.load(p.x, on ? o : 0, tm.lane, on ? p.N : 0);
    rg.load(p.gy, on ? o : 0, tm.lane, on ? p.N : 0);
    if constexpr (GATE) rz.load(p.gate, on ? o : 0, tm.lane, on ? p.N : 0);
  };
  fetch(off, m < p.M);
  load_params<V, K, TS>(p.weight + (size_t)tm.g * p.N, tm.lane, p.N, w);
  if constexpr (GATE)
    load_params<V, K, TS>(p.bias != nullptr ? p.bias + (size_t)tm.g * p.N : nullptr, tm.lane, p.N, b);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) gw[k][i] = gb[k][i] = 0.f;
  for (long long it = 0; it < tm.turns; ++it, m += tm.step, off += stride) {
    const bool on = m < p.M;
    const RowPart<T, V, K, TS> cx = rx, cg = rg, cz = rz;
    fetch(off + stride, m + tm.step < p.M);
    float x[K][V], g[K][V], z[K][V];
    const float rstd = center<T, V, K, TS>(cx, x, tm.lane, p.N, inv_n, p.eps, sum);
    float su = 0.f, sx = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[k][i] *= rstd;
        g[k][i] = cg.v[k][i];  // 0 in a turn without a row
        if constexpr (GATE) {
          const float zi = cz.v[k][i], s = sigmoid_ex2(zi), zs = zi * s, gl = g[k][i];
          z[k][i] = gl * fmaf(x[k][i], w[k][i], b[k][i]) * fmaf(zs, 1.f - s, s);
          g[k][i] = gl * zs;
        }
        if (on) {  // a row that is not there has x = 0 / sqrt(eps), which eps = 0 makes a NaN
          gw[k][i] = fmaf(g[k][i], x[k][i], gw[k][i]);
          gb[k][i] += g[k][i];
        }
        const float u = g[k][i] * w[k][i];
        su += u;
        sx = fmaf(u, x[k][i], sx);
      }
    const float2 r = sum(su, sx);
    if (!on) continue;
    const float c0 = -rstd * r.x * inv_n, c1 = -rstd * r.y * inv_n;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int col = (k * TS + tm.lane) * V;
      if (col >= p.N) continue;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = fmaf(rstd * g[k][i], w[k][i], fmaf(c1, x[k][i], c0));
      store_vec<T, V>(static_cast<T*>(p.gx) + off + col, o);
      if constexpr (GATE) store_vec<T, V>(static_cast<T*>(p.ggate) + off + col, z[k]);
    }
  }
  const long long slice = ((long long)blockIdx.x * (kCtaThreads<TS> / TS) + threadIdx.x / TS) / p.G;
  if (slice >= p.slices) return;
  float* part = p.part + (size_t)slice * 2 * p.G * p.N + (size_t)tm.g * p.N;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int col = (k * TS + tm.lane) * V;
    if (col >= p.N) continue;
    store_vec<float, V>(part + col, gw[k]);
    store_vec<float, V>(part + (size_t)p.G * p.N + col, gb[k]);
  }
}

// Any width: the row is read again for each sum.
template <typename T>
__device__ __forceinline__ float row_stats(const T* row, int N, float inv_n, float eps, float& mean,
                                           TeamSum<kMaxTeam>& sum) {
  float s = 0.f;
  for (int i = threadIdx.x; i < N; i += kMaxTeam) s += IO<T>::to_f(row[i]);
  mean = sum(s, 0.f).x * inv_n;
  float q = 0.f;
  for (int i = threadIdx.x; i < N; i += kMaxTeam) {
    const float d = IO<T>::to_f(row[i]) - mean;
    q = fmaf(d, d, q);
  }
  return 1.f / sqrtf(fmaf(sum(q, 0.f).x, inv_n, eps));
}

template <typename T>
__global__ void __launch_bounds__(kMaxTeam) norm_fwd_wide_kernel(const NormParams p) {
  __shared__ float2 buf[2 * kMaxTeam / 32];
  TeamSum<kMaxTeam> sum{buf};
  Team<kMaxTeam> tm(p);
  for (long long m = tm.m; m < p.M; m += tm.step) {
    const size_t off = ((size_t)m * p.G + tm.g) * p.N;
    const T* x = static_cast<const T*>(p.x) + off;
    float mean;
    const float rstd = row_stats(x, p.N, 1.f / (float)p.N, p.eps, mean, sum);
    for (int i = threadIdx.x; i < p.N; i += kMaxTeam) {
      const size_t col = (size_t)tm.g * p.N + i;
      float o = fmaf((IO<T>::to_f(x[i]) - mean) * rstd, p.weight[col], p.bias != nullptr ? p.bias[col] : 0.f);
      if (p.gate != nullptr) {
        const float z = IO<T>::to_f(static_cast<const T*>(p.gate)[off + i]);
        o *= z * sigmoid_ex2(z);
      }
      static_cast<T*>(p.y)[off + i] = IO<T>::from_f(o);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kMaxTeam) norm_bwd_wide_kernel(const NormParams p) {
  __shared__ float2 buf[2 * kMaxTeam / 32];
  TeamSum<kMaxTeam> sum{buf};
  Team<kMaxTeam> tm(p);
  const float inv_n = 1.f / (float)p.N;
  float* pw = p.part + (size_t)tm.m * 2 * p.G * p.N + (size_t)tm.g * p.N;  // this team's own columns
  float* pb = pw + (size_t)p.G * p.N;
  bool first = true;
  for (long long m = tm.m; m < p.M; m += tm.step) {
    const size_t off = ((size_t)m * p.G + tm.g) * p.N;
    const T* x = static_cast<const T*>(p.x) + off;
    const T* gy = static_cast<const T*>(p.gy) + off;
    const T* gate = p.gate != nullptr ? static_cast<const T*>(p.gate) + off : nullptr;
    float mean;
    const float rstd = row_stats(x, p.N, inv_n, p.eps, mean, sum);
    float su = 0.f, sx = 0.f;
    for (int i = threadIdx.x; i < p.N; i += kMaxTeam) {
      const size_t col = (size_t)tm.g * p.N + i;
      const float xh = (IO<T>::to_f(x[i]) - mean) * rstd, w = p.weight[col];
      float g = IO<T>::to_f(gy[i]);
      if (gate != nullptr) {
        const float z = IO<T>::to_f(gate[i]), s = sigmoid_ex2(z);
        static_cast<T*>(p.ggate)[off + i] = IO<T>::from_f(
            g * fmaf(xh, w, p.bias != nullptr ? p.bias[col] : 0.f) * (s * fmaf(z, 1.f - s, 1.f)));
        g *= z * s;
      }
      pw[i] = first ? g * xh : fmaf(g, xh, pw[i]);
      pb[i] = first ? g : pb[i] + g;
      su = fmaf(g, w, su);
      sx = fmaf(g * w, xh, sx);
    }
    first = false;
    const float2 r = sum(su, sx);
    const float mu = r.x * inv_n, mx = r.y * inv_n;
    for (int i = threadIdx.x; i < p.N; i += kMaxTeam) {
      const float xh = (IO<T>::to_f(x[i]) - mean) * rstd;
      float g = IO<T>::to_f(gy[i]);
      if (gate != nullptr) {
        const float z = IO<T>::to_f(gate[i]);
        g *= z * sigmoid_ex2(z);
      }
      static_cast<T*>(p.gx)[off + i] =
          IO<T>::from_f(rstd * (fmaf(g, p.weight[(size_t)tm.g * p.N + i], -mu) - xh * mx));
    }
  }
}

// gweight, gbias [C]: the slices' sums added in order: 32 columns by 32 rows of threads, a thread's
// loads 8 at a time.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(int slices, int C, const float* __restrict__ part,
                                                           float* gweight, float* gbias) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  const size_t row = 2 * (size_t)C;
  float s = 0.f;
  if (col < 2 * C) {
    const float* q = part + col;
    int k = r;
    for (; k + 7 * 32 < slices; k += 8 * 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = q[(size_t)(k + 32 * i) * row];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; k < slices; k += 32) s += q[(size_t)k * row];
  }
  red[r][lane] = s;
  __syncthreads();
  s = red[lane][r];  // column r of this CTA, row `lane`
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int c = blockIdx.x * 32 + r;
  if (lane == 0 && c < 2 * C) {
    if (c < C)
      gweight[c] = s;
    else if (gbias != nullptr)
      gbias[c - C] = s;
  }
}

// Threads of a team and vectors per thread for nv vectors a group; 0 threads: the wide kernel.
struct TeamShape {
  int ts, k;
};
TeamShape team_shape(int nv) {
  if (nv <= 8) return {8, 1};
  if (nv <= 16) return {16, 1};
  if (nv <= 32) return {32, 1};
  if (nv <= 64) return {32, 2};
  if (nv <= 128) return {128, 1};
  if (nv <= 256) return {128, 2};
  if (nv <= 512) return {512, 1};
  if (nv <= 1024) return {512, 2};
  return {0, 0};
}

template <bool BWD, typename T, int V, int K, int TS>
cudaError_t run_team(const NormParams& p, cudaStream_t st) {
  constexpr int PER = kCtaThreads<TS> / TS;
  const long long teams = (long long)p.slices * p.G;
  const unsigned grid = (unsigned)((teams + PER - 1) / PER);
  const auto kernel =
      BWD ? (p.gate != nullptr ? norm_bwd_kernel<T, V, K, TS, true> : norm_bwd_kernel<T, V, K, TS, false>)
          : (p.gate != nullptr ? norm_fwd_kernel<T, V, K, TS, true> : norm_fwd_kernel<T, V, K, TS, false>);
  kernel<<<grid, kCtaThreads<TS>, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool BWD, typename T, int V>
cudaError_t run_v(const NormParams& p, cudaStream_t st) {
  const TeamShape s = team_shape(p.N / V);
  switch (s.ts * 4 + s.k) {
    case 8 * 4 + 1: return run_team<BWD, T, V, 1, 8>(p, st);
    case 16 * 4 + 1: return run_team<BWD, T, V, 1, 16>(p, st);
    case 32 * 4 + 1: return run_team<BWD, T, V, 1, 32>(p, st);
    case 32 * 4 + 2: return run_team<BWD, T, V, 2, 32>(p, st);
    case 128 * 4 + 1: return run_team<BWD, T, V, 1, 128>(p, st);
    case 128 * 4 + 2: return run_team<BWD, T, V, 2, 128>(p, st);
    case 512 * 4 + 1: return run_team<BWD, T, V, 1, 512>(p, st);
    case 512 * 4 + 2: return run_team<BWD, T, V, 2, 512>(p, st);
  }
  const unsigned grid = (unsigned)((long long)p.slices * p.G);
  if constexpr (BWD)
    norm_bwd_wide_kernel<T><<<grid, kMaxTeam, 0, st>>>(p);
  else
    norm_fwd_wide_kernel<T><<<grid, kMaxTeam, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool BWD>
cudaError_t run(bool bf16, bool vec, const NormParams& p, cudaStream_t st) {
  if (bf16) return vec ? run_v<BWD, __nv_bfloat16, 8>(p, st) : run_v<BWD, __nv_bfloat16, 1>(p, st);
  return vec ? run_v<BWD, float, 4>(p, st) : run_v<BWD, float, 1>(p, st);
}

// Slices that give about kTargetThreads threads, at least `min_rows` rows each.
int slices_for(long long M, int G, int N, bool vec, bool bf16, int min_rows) {
  const int ts0 = team_shape(N / (vec ? (bf16 ? 8 : 4) : 1)).ts, ts = ts0 == 0 ? kMaxTeam : ts0;
  const long long want = std::max<long long>(1, kTargetThreads / ((long long)ts * G));
  return (int)std::max<long long>(1, std::min<long long>(want, (M + min_rows - 1) / min_rows));
}

}  // namespace

// Depends on sizes alone (not on alignment), so that the workspace query needs no pointers.
int norm_bwd_slices(long long M, int G, int N, bool bf16) {
  return slices_for(M, G, N, N % (bf16 ? 8 : 4) == 0, bf16, 4);
}

cudaError_t launch_norm_fwd(bool bf16, bool vec, const NormParams& p0, cudaStream_t st) {
  NormParams p = p0;
  p.slices = slices_for(p.M, p.G, p.N, vec, bf16, 1);
  return run<false>(bf16, vec, p, st);
}

cudaError_t launch_norm_bwd(bool bf16, bool vec, const NormParams& p0, cudaStream_t st) {
  NormParams p = p0;
  p.slices = norm_bwd_slices(p.M, p.G, p.N, bf16);
  const cudaError_t e = run<true>(bf16, vec, p, st);
  if (e != cudaSuccess) return e;
  const int C = p.G * p.N;
  norm_reduce_kernel<<<(unsigned)((2LL * C + 31) / 32), 1024, 0, st>>>(p.slices, C, p.part, p.gweight, p.gbias);
  return cudaGetLastError();
}

}  // namespace rwkv
