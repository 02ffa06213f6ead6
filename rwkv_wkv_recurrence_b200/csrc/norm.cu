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
// row in registers (1 to 3 vectors a thread): the variance is the mean of (x - mean)², not a
// difference of large sums.  A team keeps its group and strides over the rows, so w and b, and the
// backward's column sums, stay in registers; teams of neighbouring groups are neighbours, so a
// CTA's accesses are contiguous.  Column sums go to the workspace per team and are added in order
// by a second kernel: no atomics, the same inputs give the same bits.  Groups wider than 1024
// vectors take a kernel that reads the row again for each sum (from L1 / L2).  Rows are fetched a turn
// ahead.  Measured figures stand with the launch.
#include <algorithm>

#include "launch.h"
#include "mixer_common.cuh"

namespace rwkv {
namespace {

constexpr int kMaxTeam = 512;
// Rows are dealt out to as many teams as fit on the GPU at once: CTAs of a second turn would find
// their SMs half idle (gated heads 16384x40x64 bf16: 45 us forward, 53 with one and a half turns).  The
// backward's kernels hold 80 to 128 registers a thread, so 512 threads an SM; each of its teams' column
// sums cost a pass besides (83 + 8 us with three turns, 78 + 6 with one; fp32 8192x768 16 + 6, 13.6 + 4.8).
constexpr int kSMs = 148, kBwdThreads = kSMs * 512;

template <int TS>
constexpr int kCtaThreads = TS > 256 ? TS : 256;
template <int TS>
constexpr int kTeams = kCtaThreads<TS> / TS;  // teams per CTA

// Sums over a team, for all its threads: one value, or two.  Teams wider than a warp meet at their own
// barrier; `buf` alternates between two halves, so one barrier a call is enough.
template <int TS>
struct TeamSum {
  static constexpr int kWarps = TS > 32 ? TS / 32 : 1;
  static constexpr int kBuf = 2 * kWarps * kTeams<TS>;
  float2* buf;
  int phase = 0;
  template <bool TWO>
  __device__ __forceinline__ float2 run(float a, float b) {
    constexpr int W = TS < 32 ? TS : 32;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      if (TWO) b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TS > 32) {
      const int team = threadIdx.x / TS;
      float2* s = buf + (team * 2 + phase) * kWarps;
      phase ^= 1;
      if ((threadIdx.x & 31) == 0) s[threadIdx.x % TS / 32] = make_float2(a, b);
      if constexpr (kTeams<TS> == 1)
        __syncthreads();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TS) : "memory");
      a = b = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        a += s[i].x;
        if (TWO) b += s[i].y;
      }
    }
    return make_float2(a, b);
  }
  __device__ __forceinline__ float operator()(float a) { return run<false>(a, 0.f).x; }
  __device__ __forceinline__ float2 operator()(float a, float b) { return run<true>(a, b); }
};

// Where a team works: its group, first row, row stride.
template <int TS>
struct Team {
  int lane, g;
  long long m, step, turns;
  __device__ __forceinline__ explicit Team(const NormParams& p) {
    lane = threadIdx.x % TS;
    const long long id = (long long)blockIdx.x * kTeams<TS> + threadIdx.x / TS;
    g = (int)(id % p.G);
    m = id / p.G;
    step = p.slices;
    // a team past the last slice has no rows; teams of a warp's width or less share a warp with
    // others, whose shuffles they take part in: all take as many turns as the first slice
    turns = TS > 32 ? (p.M - m + step - 1) / step : (p.M + step - 1) / step;
    if (m >= step) m = p.M;
  }
};

// A lane's part of a row as loaded: vectors k = 0 .. K-1 at columns (k TS + lane) V; those past
// column N stay zero.
template <typename T, int V, int K, int TS>
struct RowPart {
  Raw<T, V> v[K];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k].zero();
  }
  __device__ __forceinline__ void load(const T* lane0, const bool (&in)[K]) {  // lane0: the lane's first column
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (in[k]) v[k].load(lane0 + k * TS * V);
  }
};

// Parameters of a group in the same places, in pairs (with V = 1 a pair's second half is idle).
template <int V, int K, int TS>
__device__ __forceinline__ void load_params(const float* row, int lane, const bool (&in)[K],
                                            float2 (&f)[K][(V + 1) / 2]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    Raw<float, V> r;
    r.zero();
    if (row != nullptr && in[k]) r.load(row + (k * TS + lane) * V);
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) f[k][i] = r.pair(i);
  }
}

// x - mean (0 past column N); returns 1 / sqrt(var + eps).
template <typename T, int V, int K, int TS>
__device__ __forceinline__ float center(const RowPart<T, V, K, TS>& r, float2 (&x)[K][(V + 1) / 2],
                                        const bool (&in)[K], float inv_n, float eps, TeamSum<TS>& sum) {
  constexpr int P = (V + 1) / 2;
  float2 s = dup2(0.f);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < P; ++i) s = add2(s, x[k][i] = r.v[k].pair(i));
  const float mean = sum(s.x + s.y) * inv_n;
  float2 q = dup2(0.f);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float mk = in[k] ? -mean : 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[k][i] = add2(x[k][i], make_float2(mk, V == 1 ? 0.f : mk));
      q = fma2(x[k][i], x[k][i], q);
    }
  }
  return rsqrtf(fmaf(sum(q.x + q.y), inv_n, eps));
}

// Rows are fetched a turn ahead and left as loaded until they are due; behind the last row the last
// fetch is repeated and not used.
template <typename T, int V, int K, int TS, bool GATE>
__global__ void __launch_bounds__(kCtaThreads<TS>) norm_fwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int P = (V + 1) / 2;
  __shared__ float2 buf[TeamSum<TS>::kBuf];
  TeamSum<TS> sum{buf};
  const Team<TS> tm(p);
  const float inv_n = 1.f / (float)p.N;
  bool in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) in[k] = (k * TS + tm.lane) * V < p.N;
  const ptrdiff_t stride = (ptrdiff_t)tm.step * p.G * p.N;
  const size_t off = ((size_t)(tm.m < p.M ? tm.m : 0) * p.G + tm.g) * p.N + tm.lane * V;
  const T* x_at = static_cast<const T*>(p.x) + off;
  const T* z_at = GATE ? static_cast<const T*>(p.gate) + off : nullptr;
  T* y_at = static_cast<T*>(p.y) + off;
  long long m = tm.m;
  RowPart<T, V, K, TS> rx, rz;
  rx.zero();
  rx.load(x_at, in);
  if constexpr (GATE) {
    rz.zero();
    rz.load(z_at, in);
  }
  float2 w[K][P], b[K][P];
  load_params<V, K, TS>(p.weight + (size_t)tm.g * p.N, tm.lane, in, w);
  load_params<V, K, TS>(p.bias != nullptr ? p.bias + (size_t)tm.g * p.N : nullptr, tm.lane, in, b);
  for (long long it = 0; it < tm.turns; ++it) {
    const bool on = m < p.M;
    const RowPart<T, V, K, TS> cx = rx, cz = rz;
    m += tm.step;
    if (m < p.M) {
      x_at += stride;
      rx.load(x_at, in);
      if constexpr (GATE) {
        z_at += stride;
        rz.load(z_at, in);
      }
    }
    float2 x[K][P];
    const float2 rstd = dup2(center<T, V, K, TS>(cx, x, in, inv_n, p.eps, sum));
    if (on) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!in[k]) continue;
        float2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          o[i] = fma2(mul2(x[k][i], rstd), w[k][i], b[k][i]);
          if constexpr (GATE) {
            const float2 z = cz.v[k].pair(i);
            o[i] = mul2(o[i], mul2(z, sigmoid2(z)));
          }
        }
        store_pairs_as<T, V>(y_at + k * TS * V, o);
      }
    }
    y_at += stride;
  }
}

template <typename T, int V, int K, int TS, bool GATE>
__global__ void __launch_bounds__(kCtaThreads<TS>) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int P = (V + 1) / 2;
  __shared__ float2 buf[TeamSum<TS>::kBuf];
  TeamSum<TS> sum{buf};
  const Team<TS> tm(p);
  const float inv_n = 1.f / (float)p.N;
  bool in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) in[k] = (k * TS + tm.lane) * V < p.N;
  const ptrdiff_t stride = (ptrdiff_t)tm.step * p.G * p.N;
  const size_t off = ((size_t)(tm.m < p.M ? tm.m : 0) * p.G + tm.g) * p.N + tm.lane * V;
  const T* x_at = static_cast<const T*>(p.x) + off;
  const T* g_at = static_cast<const T*>(p.gy) + off;
  const T* z_at = GATE ? static_cast<const T*>(p.gate) + off : nullptr;
  T* gx_at = static_cast<T*>(p.gx) + off;
  T* gz_at = GATE ? static_cast<T*>(p.ggate) + off : nullptr;
  long long m = tm.m;
  RowPart<T, V, K, TS> rx, rg, rz;
  rx.zero();
  rx.load(x_at, in);
  rg.zero();
  rg.load(g_at, in);
  if constexpr (GATE) {
    rz.zero();
    rz.load(z_at, in);
  }
  float2 w[K][P], b[K][P], gw[K][P], gb[K][P];
  load_params<V, K, TS>(p.weight + (size_t)tm.g * p.N, tm.lane, in, w);
  if constexpr (GATE)
    load_params<V, K, TS>(p.bias != nullptr ? p.bias + (size_t)tm.g * p.N : nullptr, tm.lane, in, b);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < P; ++i) gw[k][i] = gb[k][i] = dup2(0.f);
  for (long long it = 0; it < tm.turns; ++it) {
    const bool on = m < p.M;
    const RowPart<T, V, K, TS> cx = rx, cg = rg, cz = rz;
    m += tm.step;
    if (m < p.M) {
      x_at += stride;
      g_at += stride;
      rx.load(x_at, in);
      rg.load(g_at, in);
      if constexpr (GATE) {
        z_at += stride;
        rz.load(z_at, in);
      }
    }
    float2 x[K][P], u[K][P], z[K][P];
    const float rstd = center<T, V, K, TS>(cx, x, in, inv_n, p.eps, sum);
    float2 su = dup2(0.f), sx = dup2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < P; ++i) {
        x[k][i] = mul2(x[k][i], dup2(rstd));
        float2 g = cg.v[k].pair(i);
        if constexpr (GATE) {
          const float2 zi = cz.v[k].pair(i), s = sigmoid2(zi), zs = mul2(zi, s);
          // silu'(z) = s + z s (1 - s)
          z[k][i] = mul2(mul2(g, fma2(x[k][i], w[k][i], b[k][i])), fma2(zs, fma2(s, dup2(-1.f), dup2(1.f)), s));
          g = mul2(g, zs);
        }
        if (on) {
          gw[k][i] = fma2(g, x[k][i], gw[k][i]);
          gb[k][i] = add2(g, gb[k][i]);
        }
        u[k][i] = mul2(g, w[k][i]);
        su = add2(su, u[k][i]);
        sx = fma2(u[k][i], x[k][i], sx);
      }
    const float2 r = sum(su.x + su.y, sx.x + sx.y);
    if (on) {
      const float2 c0 = dup2(-rstd * r.x * inv_n), c1 = dup2(-rstd * r.y * inv_n);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!in[k]) continue;
        float2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = fma2(dup2(rstd), u[k][i], fma2(c1, x[k][i], c0));
        store_pairs_as<T, V>(gx_at + k * TS * V, o);
        if constexpr (GATE) store_pairs_as<T, V>(gz_at + k * TS * V, z[k]);
      }
    }
    gx_at += stride;
    if constexpr (GATE) gz_at += stride;
  }
  // With one group a CTA's teams hold the same columns and add up in shared memory, in order; else
  // each writes its own.
  long long part_id = ((long long)blockIdx.x * kTeams<TS> + threadIdx.x / TS) / p.G;
  bool write = part_id < p.slices;
  if constexpr (kTeams<TS> > 1) {
    __shared__ float2 acc[2][K * TS * P];
    if (p.G == 1) {
      const int team = threadIdx.x / TS;
      for (int t = 0; t < kTeams<TS>; ++t) {
        if (team == t) {
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) {
              float2& a = acc[0][(k * P + i) * TS + tm.lane];
              float2& c = acc[1][(k * P + i) * TS + tm.lane];
              if (t > 0) gw[k][i] = add2(a, gw[k][i]), gb[k][i] = add2(c, gb[k][i]);
              a = gw[k][i], c = gb[k][i];
            }
        }
        __syncthreads();
      }
      part_id = blockIdx.x;
      write = team == kTeams<TS> - 1;  // holds the sum of all
    }
  }
  if (!write) return;
  float* part = p.part + (size_t)part_id * 2 * p.G * p.N + (size_t)tm.g * p.N;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!in[k]) continue;
    const int col = (k * TS + tm.lane) * V;
    store_pairs_as<float, V>(part + col, gw[k]);
    store_pairs_as<float, V>(part + (size_t)p.G * p.N + col, gb[k]);
  }
}

// Any width: the row is read again for each sum.
template <typename T>
__device__ __forceinline__ float row_stats(const T* row, int N, float inv_n, float eps, float& mean,
                                           TeamSum<kMaxTeam>& sum) {
  float s = 0.f;
  for (int i = threadIdx.x; i < N; i += kMaxTeam) s += IO<T>::to_f(row[i]);
  mean = sum(s) * inv_n;
  float q = 0.f;
  for (int i = threadIdx.x; i < N; i += kMaxTeam) {
    const float d = IO<T>::to_f(row[i]) - mean;
    q = fmaf(d, d, q);
  }
  return rsqrtf(fmaf(sum(q), inv_n, eps));
}

template <typename T>
__global__ void __launch_bounds__(kMaxTeam) norm_fwd_wide_kernel(const NormParams p) {
  __shared__ float2 buf[TeamSum<kMaxTeam>::kBuf];
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
  __shared__ float2 buf[TeamSum<kMaxTeam>::kBuf];
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
  if (nv <= 128) return {64, 2};
  if (nv <= 192) return {64, 3};
  if (nv <= 256) return {128, 2};
  if (nv <= 512) return {512, 1};
  if (nv <= 1024) return {512, 2};
  return {0, 0};
}

// Sets of rows (slices), one per team of a group, for `teams` teams; `min_rows` rows or more each.
int slices_for(long long M, int G, long long teams, int min_rows) {
  return (int)std::max<long long>(1, std::min<long long>(teams / G, (M + min_rows - 1) / min_rows));
}

// CTAs of a kernel that the GPU holds at once; asked once per kernel (`known`).
int resident_ctas(const void* kernel, int threads, int* known) {
  int n = __atomic_load_n(known, __ATOMIC_RELAXED);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess || n < 1) n = 1;
    __atomic_store_n(known, n, __ATOMIC_RELAXED);
  }
  return n * kSMs;
}

template <bool BWD, typename T, int V, int K, int TS>
cudaError_t run_team(NormParams p, cudaStream_t st) {
  const bool gate = p.gate != nullptr;
  const auto kernel = BWD ? (gate ? norm_bwd_kernel<T, V, K, TS, true> : norm_bwd_kernel<T, V, K, TS, false>)
                          : (gate ? norm_fwd_kernel<T, V, K, TS, true> : norm_fwd_kernel<T, V, K, TS, false>);
  if (!BWD) {
    static int known[2] = {0, 0};
    const int ctas = resident_ctas(reinterpret_cast<const void*>(kernel), kCtaThreads<TS>, &known[gate]);
    p.slices = slices_for(p.M, p.G, (long long)ctas * kTeams<TS>, 1);
  }
  const long long teams = (long long)p.slices * p.G;
  const unsigned grid = (unsigned)((teams + kTeams<TS> - 1) / kTeams<TS>);
  kernel<<<grid, kCtaThreads<TS>, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool BWD, typename T, int V>
cudaError_t run_v(NormParams p, cudaStream_t st) {
  const TeamShape s = team_shape(p.N / V);
  switch (s.ts * 4 + s.k) {
    case 8 * 4 + 1: return run_team<BWD, T, V, 1, 8>(p, st);
    case 16 * 4 + 1: return run_team<BWD, T, V, 1, 16>(p, st);
    case 32 * 4 + 1: return run_team<BWD, T, V, 1, 32>(p, st);
    case 32 * 4 + 2: return run_team<BWD, T, V, 2, 32>(p, st);
    case 64 * 4 + 2: return run_team<BWD, T, V, 2, 64>(p, st);
    case 64 * 4 + 3: return run_team<BWD, T, V, 3, 64>(p, st);
    case 128 * 4 + 2: return run_team<BWD, T, V, 2, 128>(p, st);
    case 512 * 4 + 1: return run_team<BWD, T, V, 1, 512>(p, st);
    case 512 * 4 + 2: return run_team<BWD, T, V, 2, 512>(p, st);
  }
  if (!BWD) p.slices = slices_for(p.M, p.G, 4 * kSMs, 1);  // wide rows: 4 CTAs of 512 threads an SM
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

int bwd_slices(long long M, int G, int nv) {
  const int ts = team_shape(nv).ts;
  return slices_for(M, G, kBwdThreads / (ts == 0 ? kMaxTeam : ts), 4);
}

}  // namespace

namespace {
// Sets of column sums that the backward's teams write: a CTA's teams share one where there is one group.
int parts_for(int slices, int G, int nv) {
  const int ts = team_shape(nv).ts;
  const int teams = ts == 0 ? 1 : (ts > 256 ? 1 : 256 / ts);
  return G == 1 ? (slices + teams - 1) / teams : slices;
}
}  // namespace

// Bounds the sets of column sums by sizes alone (aligned or not), so that the workspace query needs no
// pointers.
int norm_bwd_parts(long long M, int G, int N, bool bf16) {
  const int v = bf16 ? 8 : 4;
  int n = parts_for(bwd_slices(M, G, N), G, N);
  if (N % v == 0) n = std::max(n, parts_for(bwd_slices(M, G, N / v), G, N / v));
  return n;
}

cudaError_t launch_norm_fwd(bool bf16, bool vec, const NormParams& p, cudaStream_t st) {
  return run<false>(bf16, vec, p, st);
}

cudaError_t launch_norm_bwd(bool bf16, bool vec, const NormParams& p0, cudaStream_t st) {
  NormParams p = p0;
  p.slices = bwd_slices(p.M, p.G, vec ? p.N / (bf16 ? 8 : 4) : p.N);
  const cudaError_t e = run<true>(bf16, vec, p, st);
  if (e != cudaSuccess) return e;
  const int C = p.G * p.N;
  norm_reduce_kernel<<<(unsigned)((2LL * C + 31) / 32), 1024, 0, st>>>(
      parts_for(p.slices, p.G, vec ? p.N / (bf16 ? 8 : 4) : p.N), C, p.part, p.gweight, p.gbias);
  return cudaGetLastError();
}

}  // namespace rwkv
