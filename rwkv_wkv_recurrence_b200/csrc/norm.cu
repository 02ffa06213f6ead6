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
// row in registers (1 to 4 vectors a thread): the variance is the mean of (x - mean)², not a
// difference of large sums.  A team keeps its group and strides over the rows, so w and b, and the
// backward's column sums, stay in registers; teams of neighbouring groups are neighbours, so a
// CTA's accesses are contiguous.  Column sums go to the workspace per team and are added in order
// by a second kernel: no atomics, the same inputs give the same bits.  Groups wider than 2048 vectors
// take a kernel that reads the row again for each sum (from L1 / L2).  Rows are fetched a turn ahead.
// Gated heads 16384x40x64 bf16: 43.6 us forward (5.8 TB/s), 78 and 6 for the column sums
// backward (5.4 TB/s); fp32 8192x768: 9.2, 13.6 and 4.8.
//
// Rows of any length.  Where rows do not start on 16-byte boundaries a team's vectors are laid on those
// boundaries all the same and the row's first and last vector masked (Cols): 8192x767 fp32 11 us and 24
// backward, 34 and 64 with single accesses; 16384x2047 bf16 41 and 116, 126 and 581.
#include <algorithm>

#include "mixer.h"
#include "mixer_common.cuh"

namespace rwkv {
namespace {

constexpr int kMaxTeam = 512;
// Rows are dealt out to as many teams as fit on the GPU at once: CTAs of a second turn would find
// their SMs half idle (gated heads 16384x40x64 bf16: 45 us forward, 53 with one and a half turns).  The
// backward's kernels mostly hold 80 to 128 registers a thread, so 512 threads an SM; each of its teams' column
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

// A lane's columns: vectors k = 0 .. K-1 of V columns from c(k) = (k TS + lane) V on.  SHIFT: rows need not
// start on a vector's boundary in memory; c(k) lies `shift` columns further left, so that every vector is
// aligned, and the first and the last of a row are shared with its neighbours (`part`).  The launch deals
// out rows so that all rows of a team have the same shift: parameters and column sums stay in place.
template <typename T, int V, int K, int TS, bool SHIFT>
struct Cols {
  static constexpr bool kShift = SHIFT;
  int c0, N;
  bool in[K], part[K];
  __device__ __forceinline__ Cols(const Team<TS>& tm, const NormParams& p) {
    N = p.N;
    c0 = tm.lane * V;
    if constexpr (SHIFT) {
      const size_t start = ((size_t)(tm.m < p.M ? tm.m : 0) * p.G + tm.g) * p.N;
      c0 -= (int)((reinterpret_cast<uintptr_t>(p.x) / sizeof(T) + start) % V);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      in[k] = c(k) < N;
      part[k] = SHIFT && in[k] && (c(k) < 0 || c(k) + V > N);
    }
  }
  __device__ __forceinline__ int c(int k) const { return c0 + k * TS * V; }
  __device__ __forceinline__ bool has(int k, int i) const { return (unsigned)(c(k) + i) < (unsigned)N; }
};

// A lane's part of a row as loaded; what lies past column N (in `part` vectors before column 0 too) is
// zero after mask().
template <typename T, int V, int K, int TS, bool SHIFT>
struct RowPart {
  using C = Cols<T, V, K, TS, SHIFT>;
  Raw<T, V> v[K];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k].zero();
  }
  // lane0: the lane's first column.  `inner`: there is a row before and one behind, so shared vectors
  // may be read whole.
  __device__ __forceinline__ void load(const T* lane0, const C& cols, bool inner) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!cols.in[k]) continue;
      if (!cols.part[k] || inner)
        v[k].load(lane0 + k * TS * V);
      else
        v[k].load_range(lane0 + k * TS * V, -cols.c(k), cols.N - cols.c(k));
    }
  }
  __device__ __forceinline__ void mask(const C& cols) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (cols.part[k]) v[k].keep_range(-cols.c(k), cols.N - cols.c(k));
  }
};

// Parameters of a group in a vector's places, in pairs (with V = 1 a pair's second half is idle).
template <int V, typename C>
__device__ __forceinline__ void load_params(const float* row, const C& cols, int k, float2 (&f)[(V + 1) / 2]) {
  Raw<float, V> r;
  r.zero();
  if (row != nullptr && cols.in[k]) {
    if constexpr (C::kShift)
      r.load_range(row + cols.c(k), -cols.c(k), cols.N - cols.c(k));
    else
      r.load(row + cols.c(k));
  }
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) f[i] = r.pair(i);
}

// A vector's results, of a shared vector only the row's own.
template <typename T, int V, typename C>
__device__ __forceinline__ void store_cols(T* at, const C& cols, int k, const float2 (&o)[(V + 1) / 2]) {
  if (!C::kShift || !cols.part[k]) {
    store_pairs_as<T, V>(at, o);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (cols.has(k, i)) at[i] = IO<T>::from_f(i & 1 ? o[i / 2].y : o[i / 2].x);
  }
}

// x - mean (0 outside the row); returns 1 / sqrt(var + eps).
template <typename T, int V, int K, int TS, bool SHIFT>
__device__ __forceinline__ float center(const RowPart<T, V, K, TS, SHIFT>& r, float2 (&x)[K][(V + 1) / 2],
                                        const Cols<T, V, K, TS, SHIFT>& cols, float inv_n, float eps,
                                        TeamSum<TS>& sum) {
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
    const float mk = cols.in[k] ? -mean : 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) x[k][i] = add2(x[k][i], make_float2(mk, V == 1 ? 0.f : mk));
    if (cols.part[k]) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (!cols.has(k, 2 * i)) x[k][i].x = 0.f;
        if (!cols.has(k, 2 * i + 1)) x[k][i].y = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) q = fma2(x[k][i], x[k][i], q);
  }
  return rsqrtf(fmaf(sum(q.x + q.y), inv_n, eps));
}

// Rows are fetched a turn ahead and left as loaded until they are due; behind the last row the last
// fetch is repeated and not used.
template <typename T, int V, int K, int TS, bool GATE, bool SHIFT>
__global__ void __launch_bounds__(kCtaThreads<TS>) norm_fwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int P = (V + 1) / 2;
  __shared__ float2 buf[TeamSum<TS>::kBuf];
  TeamSum<TS> sum{buf};
  const Team<TS> tm(p);
  const float inv_n = 1.f / (float)p.N;
  const Cols<T, V, K, TS, SHIFT> cols(tm, p);
  const ptrdiff_t stride = (ptrdiff_t)tm.step * p.G * p.N;
  const ptrdiff_t off = ((ptrdiff_t)(tm.m < p.M ? tm.m : 0) * p.G + tm.g) * p.N + cols.c0;
  const T* x_at = static_cast<const T*>(p.x) + off;
  const T* z_at = GATE ? static_cast<const T*>(p.gate) + off : nullptr;
  T* y_at = static_cast<T*>(p.y) + off;
  long long m = tm.m;
  const long long last = p.M - 1;
  const bool inner = m > 0 && m < last;
  RowPart<T, V, K, TS, SHIFT> rx, rz;
  rx.zero();
  rx.load(x_at, cols, inner);
  if constexpr (GATE) {
    rz.zero();
    rz.load(z_at, cols, inner);
  }
  float2 w[K][P], b[K][P];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    load_params<V>(p.weight + (size_t)tm.g * p.N, cols, k, w[k]);
    load_params<V>(p.bias != nullptr ? p.bias + (size_t)tm.g * p.N : nullptr, cols, k, b[k]);
  }
  for (long long it = 0; it < tm.turns; ++it) {
    const bool on = m < p.M;
    RowPart<T, V, K, TS, SHIFT> cx = rx, cz = rz;
    m += tm.step;
    if (m < p.M) {
      x_at += stride;
      rx.load(x_at, cols, m < last);
      if constexpr (GATE) {
        z_at += stride;
        rz.load(z_at, cols, m < last);
      }
    }
    cx.mask(cols);  // of the gate only the row's own columns are used
    float2 x[K][P];
    const float2 rstd = dup2(center<T, V, K, TS, SHIFT>(cx, x, cols, inv_n, p.eps, sum));
    if (on) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!cols.in[k]) continue;
        float2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
          o[i] = fma2(mul2(x[k][i], rstd), w[k][i], b[k][i]);
          if constexpr (GATE) {
            const float2 z = cz.v[k].pair(i);
            o[i] = mul2(o[i], mul2(z, sigmoid2(z)));
          }
        }
        store_cols<T, V>(y_at + k * TS * V, cols, k, o);
      }
    }
    y_at += stride;
  }
}

template <typename T, int V, int K, int TS, bool GATE, bool SHIFT>
__global__ void __launch_bounds__(kCtaThreads<TS>, TS == 512 ? 1 : 0) norm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr int P = (V + 1) / 2;
  // Where a row's three inputs, parameters and sums pass what 128 registers a thread hold, parameters are read
  // again for each row (from L1) and no row is fetched ahead: fewer spills (4096 x 6832 fp32 175 us, 219
  // otherwise; x 12288 bf16 225, 577).  Off the 16-byte grid parameters come one by one, and it does not pay.
  constexpr bool kLean = TS == 512 && K >= 3 && GATE && !SHIFT;
  __shared__ float2 buf[TeamSum<TS>::kBuf];
  TeamSum<TS> sum{buf};
  const Team<TS> tm(p);
  const float inv_n = 1.f / (float)p.N;
  const Cols<T, V, K, TS, SHIFT> cols(tm, p);
  const ptrdiff_t stride = (ptrdiff_t)tm.step * p.G * p.N;
  const ptrdiff_t off = ((ptrdiff_t)(tm.m < p.M ? tm.m : 0) * p.G + tm.g) * p.N + cols.c0;
  const T* x_at = static_cast<const T*>(p.x) + off;
  const T* g_at = static_cast<const T*>(p.gy) + off;
  const T* z_at = GATE ? static_cast<const T*>(p.gate) + off : nullptr;
  T* gx_at = static_cast<T*>(p.gx) + off;
  T* gz_at = GATE ? static_cast<T*>(p.ggate) + off : nullptr;
  long long m = tm.m;
  const long long last = p.M - 1;
  const bool inner = m > 0 && m < last;
  RowPart<T, V, K, TS, SHIFT> rx, rg, rz;
  rx.zero();
  rx.load(x_at, cols, inner);
  rg.zero();
  rg.load(g_at, cols, inner);
  if constexpr (GATE) {
    rz.zero();
    rz.load(z_at, cols, inner);
  }
  float2 w[K][P], b[K][P], gw[K][P], gb[K][P];
  const auto params = [&](int k) {
    load_params<V>(p.weight + (size_t)tm.g * p.N, cols, k, w[k]);
    if constexpr (GATE) load_params<V>(p.bias != nullptr ? p.bias + (size_t)tm.g * p.N : nullptr, cols, k, b[k]);
  };
  if constexpr (!kLean) {
#pragma unroll
    for (int k = 0; k < K; ++k) params(k);
  }
  const auto fetch = [&] {  // row m
    if (m < p.M) {
      x_at += stride;
      g_at += stride;
      rx.load(x_at, cols, m < last);
      rg.load(g_at, cols, m < last);
      if constexpr (GATE) {
        z_at += stride;
        rz.load(z_at, cols, m < last);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < P; ++i) gw[k][i] = gb[k][i] = dup2(0.f);
  for (long long it = 0; it < tm.turns; ++it) {
    const bool on = m < p.M;
    RowPart<T, V, K, TS, SHIFT> cx = rx, cg = rg, cz = rz;
    m += tm.step;
    if (!kLean) fetch();
    cx.mask(cols);
    cg.mask(cols);
    if constexpr (GATE) cz.mask(cols);
    float2 x[K][P], u[K][P], z[K][P];
    const float rstd = center<T, V, K, TS, SHIFT>(cx, x, cols, inv_n, p.eps, sum);
    float2 su = dup2(0.f), sx = dup2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (kLean) params(k);
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
    }
    const float2 r = sum(su.x + su.y, sx.x + sx.y);
    if (on) {
      const float2 c0 = dup2(-rstd * r.x * inv_n), c1 = dup2(-rstd * r.y * inv_n);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!cols.in[k]) continue;
        float2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = fma2(dup2(rstd), u[k][i], fma2(c1, x[k][i], c0));
        store_cols<T, V>(gx_at + k * TS * V, cols, k, o);
        if constexpr (GATE) store_cols<T, V>(gz_at + k * TS * V, cols, k, z[k]);
      }
    }
    gx_at += stride;
    if constexpr (GATE) gz_at += stride;
    if (kLean) fetch();
  }
  // With one group a CTA's teams hold the same columns and add up in shared memory, in order; else
  // each writes its own.
  long long part_id = ((long long)blockIdx.x * kTeams<TS> + threadIdx.x / TS) / p.G;
  bool write = part_id < p.slices;
  if constexpr (kTeams<TS> > 1) {
    __shared__ float2 acc[2][K * TS * P];  // SHIFT: by column, as its teams' columns lie differently
    if (p.G == 1) {
      const int team = threadIdx.x / TS;
      for (int t = 0; t < kTeams<TS>; ++t) {
        if (team == t) {
#pragma unroll
          for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < P; ++i) {
              if constexpr (SHIFT) {
                float* a = &acc[0][0].x + cols.c(k) + 2 * i;
                float* c = &acc[1][0].x + cols.c(k) + 2 * i;
                if (cols.has(k, 2 * i)) {
                  if (t > 0) gw[k][i].x += a[0], gb[k][i].x += c[0];
                  a[0] = gw[k][i].x, c[0] = gb[k][i].x;
                }
                if (cols.has(k, 2 * i + 1)) {
                  if (t > 0) gw[k][i].y += a[1], gb[k][i].y += c[1];
                  a[1] = gw[k][i].y, c[1] = gb[k][i].y;
                }
              } else {
                float2& a = acc[0][(k * P + i) * TS + tm.lane];
                float2& c = acc[1][(k * P + i) * TS + tm.lane];
                if (t > 0) gw[k][i] = add2(a, gw[k][i]), gb[k][i] = add2(c, gb[k][i]);
                a = gw[k][i], c = gb[k][i];
              }
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
    if (!cols.in[k]) continue;
    if constexpr (SHIFT) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!cols.has(k, i)) continue;
        part[cols.c(k) + i] = i & 1 ? gw[k][i / 2].y : gw[k][i / 2].x;
        part[(size_t)p.G * p.N + cols.c(k) + i] = i & 1 ? gb[k][i / 2].y : gb[k][i / 2].x;
      }
    } else {
      store_pairs_as<float, V>(part + cols.c(k), gw[k]);
      store_pairs_as<float, V>(part + (size_t)p.G * p.N + cols.c(k), gb[k]);
    }
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

// Threads of a team and vectors per thread for nv vectors a group; 0 threads: the wide kernel.  Few threads with several vectors meet faster than many with one: 512 x 1 for 4096 columns in
// bf16 took 72 us forward and 145 backward (16384 rows), 256 x 2 51 and 84; 128 x 3 for 2560 columns 9.6
// and 22 (4096 rows), 256 x 2 12.7 and 25.  Three and four vectors of 512 threads do not all stay in
// registers, but beat the wide kernel: 4096x6832 gated fp32 54 us and 175, 177 and 553; 4096x16384 bf16
// 62 and 193, 170 and 953.
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
  if (nv <= 384) return {128, 3};
  if (nv <= 512) return {256, 2};
  if (nv <= 768) return {256, 3};
  if (nv <= 1024) return {512, 2};
  if (nv <= 1536) return {512, 3};
  if (nv <= 2048) return {512, 4};
  return {0, 0};
}

// Vectors of a row, at any shift.
int row_vectors(int N, int V, bool shift) { return (shift ? N + 2 * V - 2 : N) / V; }

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

// Rows between two of equal shift (a power of two): rows of a team are a multiple of it apart, unless
// there is a team for every row.
int shift_period(int N, int V) {
  int q = V;
  while (q > 1 && N % 2 == 0) q /= 2, N /= 2;
  return q;
}
int whole_periods(int slices, int q, long long M) {
  return (int)std::min<long long>(M, (long long)std::max(1, slices / q) * q);
}

template <bool BWD, typename T, int V, int K, int TS, bool SHIFT>
cudaError_t run_team(NormParams p, cudaStream_t st) {
  const bool gate = p.gate != nullptr;
  const auto kernel =
      BWD ? (gate ? norm_bwd_kernel<T, V, K, TS, true, SHIFT> : norm_bwd_kernel<T, V, K, TS, false, SHIFT>)
          : (gate ? norm_fwd_kernel<T, V, K, TS, true, SHIFT> : norm_fwd_kernel<T, V, K, TS, false, SHIFT>);
  if (!BWD) {
    static int known[2] = {0, 0};
    const int ctas = resident_ctas(reinterpret_cast<const void*>(kernel), kCtaThreads<TS>, &known[gate]);
    p.slices = slices_for(p.M, p.G, (long long)ctas * kTeams<TS>, 1);
    if (SHIFT) p.slices = whole_periods(p.slices, shift_period(p.N, V), p.M);
  }
  const long long teams = (long long)p.slices * p.G;
  const unsigned grid = (unsigned)((teams + kTeams<TS> - 1) / kTeams<TS>);
  kernel<<<grid, kCtaThreads<TS>, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool BWD, typename T, int V, bool SHIFT>
cudaError_t run_v(NormParams p, cudaStream_t st) {
  const TeamShape s = team_shape(row_vectors(p.N, V, SHIFT));
  switch (s.ts * 8 + s.k) {
    case 8 * 8 + 1: return run_team<BWD, T, V, 1, 8, SHIFT>(p, st);
    case 16 * 8 + 1: return run_team<BWD, T, V, 1, 16, SHIFT>(p, st);
    case 32 * 8 + 1: return run_team<BWD, T, V, 1, 32, SHIFT>(p, st);
    case 32 * 8 + 2: return run_team<BWD, T, V, 2, 32, SHIFT>(p, st);
    case 64 * 8 + 2: return run_team<BWD, T, V, 2, 64, SHIFT>(p, st);
    case 64 * 8 + 3: return run_team<BWD, T, V, 3, 64, SHIFT>(p, st);
    case 128 * 8 + 2: return run_team<BWD, T, V, 2, 128, SHIFT>(p, st);
    case 128 * 8 + 3: return run_team<BWD, T, V, 3, 128, SHIFT>(p, st);
    case 256 * 8 + 2: return run_team<BWD, T, V, 2, 256, SHIFT>(p, st);
    case 256 * 8 + 3: return run_team<BWD, T, V, 3, 256, SHIFT>(p, st);
    case 512 * 8 + 2: return run_team<BWD, T, V, 2, 512, SHIFT>(p, st);
    case 512 * 8 + 3: return run_team<BWD, T, V, 3, 512, SHIFT>(p, st);
    case 512 * 8 + 4: return run_team<BWD, T, V, 4, 512, SHIFT>(p, st);
  }
  if (!BWD) p.slices = slices_for(p.M, p.G, 4 * kSMs, 1);  // wide rows: 4 CTAs of 512 threads an SM
  const unsigned grid = (unsigned)((long long)p.slices * p.G);
  if constexpr (BWD)
    norm_bwd_wide_kernel<T><<<grid, kMaxTeam, 0, st>>>(p);
  else
    norm_fwd_wide_kernel<T><<<grid, kMaxTeam, 0, st>>>(p);
  return cudaGetLastError();
}

template <bool BWD, typename T>
cudaError_t run_t(NormAccess access, const NormParams& p, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  switch (access) {
    case NormAccess::kAligned: return run_v<BWD, T, V, false>(p, st);
    case NormAccess::kShifted: return run_v<BWD, T, V, true>(p, st);
    case NormAccess::kSingle: return run_v<BWD, T, 1, false>(p, st);
  }
  return cudaErrorInvalidValue;
}

template <bool BWD>
cudaError_t run(bool bf16, NormAccess access, const NormParams& p, cudaStream_t st) {
  return bf16 ? run_t<BWD, __nv_bfloat16>(access, p, st) : run_t<BWD, float>(access, p, st);
}

// The backward's slices and sets of column sums: a CTA's teams share a set where there is one group.
struct BwdPlan {
  int slices, parts;
};
BwdPlan bwd_plan(long long M, int G, int N, bool bf16, NormAccess access) {
  const bool shift = access == NormAccess::kShifted;
  const int v = access == NormAccess::kSingle ? 1 : (bf16 ? 8 : 4);
  const int ts = team_shape(row_vectors(N, v, shift)).ts;
  const int teams = ts == 0 || ts > 256 ? 1 : 256 / ts;  // a CTA's
  int slices = slices_for(M, G, kBwdThreads / (ts == 0 ? kMaxTeam : ts), 4);
  if (shift && ts != 0) slices = whole_periods(slices, shift_period(N, v), M);
  return {slices, G == 1 ? (slices + teams - 1) / teams : slices};
}

}  // namespace

// Bounds the sets of column sums by sizes alone (however the arrays lie), so that the workspace query
// needs no pointers.
int norm_bwd_parts(long long M, int G, int N, bool bf16) {
  int n = 0;
  for (const NormAccess a : {NormAccess::kAligned, NormAccess::kShifted, NormAccess::kSingle})
    if (a != NormAccess::kAligned || N % (bf16 ? 8 : 4) == 0) n = std::max(n, bwd_plan(M, G, N, bf16, a).parts);
  return n;
}

cudaError_t launch_norm_fwd(bool bf16, NormAccess access, const NormParams& p, cudaStream_t st) {
  return run<false>(bf16, access, p, st);
}

cudaError_t launch_norm_bwd(bool bf16, NormAccess access, const NormParams& p0, cudaStream_t st) {
  NormParams p = p0;
  const BwdPlan plan = bwd_plan(p.M, p.G, p.N, bf16, access);
  p.slices = plan.slices;
  const cudaError_t e = run<true>(bf16, access, p, st);
  if (e != cudaSuccess) return e;
  const int C = p.G * p.N;
  norm_reduce_kernel<<<(unsigned)((2LL * C + 31) / 32), 1024, 0, st>>>(plan.parts, C, p.part, p.gweight, p.gbias);
  return cudaGetLastError();
}

}  // namespace rwkv
