// Selective scan backward (sm_100a): the chain rule through the recurrence of scan_fwd.cu.  With
// g_t = gy_t z_t σ(z_t) (or gy_t), e_t = exp(Δ_t A), and G_t the gradient of h_t,
//   G_t = C_t g_t + e_{t+1} G_{t+1}         (from gh_out behind the last token),
//   gC_t[n] = Σ_c g_t h_t[n],   gB_t[n] = Σ_c G_t[n] Δ_t x_t,
//   s1_t = Σ_n G_t B_t,   q_t = G_t e_t h_{t-1},   s2_t = Σ_n q_t A,
//   gx_t = Δ_t s1_t + d g_t,   gdt_t = σ(dt_t + dt_bias) (x_t s1_t + s2_t),   gdt_bias = Σ gdt,
//   ga_log = A Σ q_t Δ_t,   gd = Σ g_t x_t,   gz_t = gy_t p_t silu'(z_t),   gh_in = e_0 G_0.
//
// The states come from the forward's checkpoints, one every 16 tokens.  A CTA of 256 threads owns
// 1024/N channels (4 states of one channel per thread) and walks its time segment backwards, a
// 16-token tile at a time: the states are recomputed forward from the checkpoint, 8 tokens at a
// time with e_t and e_t h_{t-1} kept in registers (64 floats), then walked backwards with G.  The
// first 8 tokens of a tile are so computed twice; keeping all 16 would take 128 registers, a
// checkpoint every 8 tokens twice their bytes.
//
// Sums over a channel's states (p, s1, s2) fold four tokens at a time over its lanes.  Sums over
// channels (gB, gC: B and C are shared by all of them) fold over the lanes of a warp, meet in
// shared memory per CTA and go to the workspace per CTA; a last kernel adds the CTAs' parts.  No
// atomics: the same inputs give the same bits.
//
// Few channels: time segments, as in the forward.  The carry G that enters a segment from behind
// is folded from the later segments' own (each from zero, by a first launch) and their ΣΔ.
#include "launch.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = kScanCkLen;  // tokens per tile
constexpr int kSub = 8;            // tokens whose states are in registers at once
constexpr int kSN = 4;             // states per thread
constexpr float kLn2 = 0.693147180559945309f;

template <int N>
struct Shape {
  static constexpr int kLanes = N / kSN;
  static constexpr int kCh = kThreads / kLanes;           // channels per CTA
  static constexpr int kChWarp = 32 / kLanes;             // channels per warp
  static constexpr int kTokThreads = kThreads / kTile;    // threads per token in the tile's loads
  static constexpr int kRun = kCh / kTokThreads;          // channels per thread there
};

template <int N>
struct __align__(16) Smem {
  float4 dxg[kTile][Shape<N>::kCh];  // (Δ, Δ x, g, -)
  float b[kTile][N], c[kTile][N];
  float sum[3][kTile][Shape<N>::kCh + 8];  // Σ_n C h, Σ_n G B, Σ_n q A log2 e
  float red[kWarps][kTile][2 * N];         // per warp: gC, gB of a token
};

template <typename T, int N>
struct Tile {
  float x[Shape<N>::kRun], dt[Shape<N>::kRun], z[Shape<N>::kRun], gy[Shape<N>::kRun];
};

template <typename T, int N>
__device__ __forceinline__ void load_tile(Tile<T, N>& R, const ScanBwdParams& p, int bb, int t, int t1, int c0,
                                          int nc) {
  constexpr int RUN = Shape<N>::kRun;
  const ScanParams& f = p.f;
  const bool ok = t < t1;
  const size_t row = (size_t)bb * f.T + (ok ? t : 0);
  const int n = ok ? nc : 0;
  load_part<T, RUN>(static_cast<const T*>(f.x) + row * f.ldx + c0, n, f.vec, R.x);
  load_part<T, RUN>(static_cast<const T*>(f.dt) + row * f.lddt + c0, n, f.vec, R.dt);
  load_part<T, RUN>(static_cast<const T*>(p.gy) + row * f.C + c0, n, f.vec, R.gy);
  if (f.z != nullptr) load_part<T, RUN>(static_cast<const T*>(f.z) + row * f.ldz + c0, n, f.vec, R.z);
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(const __grid_constant__ ScanBwdParams p) {
  using S = Shape<N>;
  constexpr int L = S::kLanes, CH = S::kCh, CW = S::kChWarp, RUN = S::kRun, TT = S::kTokThreads;
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<N>& sm = *reinterpret_cast<Smem<N>*>(raw);
  const ScanParams& f = p.f;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ct = (int)(blockIdx.x % (unsigned)f.ctiles);
  const unsigned rest = blockIdx.x / (unsigned)f.ctiles;
  const int seg = (int)(rest % (unsigned)f.nseg), bb = (int)(rest / (unsigned)f.nseg);
  const int t0 = seg * f.seg_len, t1 = min(f.T, t0 + f.seg_len);

  const int ch = tid / L, sub = tid % L;
  const int c = ct * CH + ch;
  const bool cact = c < f.C;
  const size_t hoff = ((size_t)bb * f.C + c) * N + sub * kSN;
  const size_t plane = (size_t)f.B * f.C * N;
  float a2[kSN], gh[kSN], ga[kSN];
#pragma unroll
  for (int i = 0; i < kSN; ++i) a2[i] = gh[i] = ga[i] = 0.f;
  if (cact) {
    load_rates<kSN>(f.a_log + (size_t)c * N + sub * kSN, a2);
    if (seg < f.nseg - 1) {  // the last segment's own gradient starts from gh_out
      load_vec<float, kSN>(p.seg_g + (size_t)(f.nseg - 1) * plane + hoff, gh);
      for (int s = f.nseg - 2; s > seg; --s) {
        float x[kSN];
        load_vec<float, kSN>(p.seg_g + (size_t)s * plane + hoff, x);
        const float sd = p.seg_dt[((size_t)s * f.B + bb) * f.C + c];
#pragma unroll
        for (int i = 0; i < kSN; ++i) gh[i] = fmaf(ex2(sd * a2[i]), gh[i], x[i]);
      }
    } else if (p.gh_out != nullptr) {
      // a copy when segmented: gh_in may be the same array, and another CTA writes it
      load_vec<float, kSN>((f.nseg > 1 ? p.seg_g0 : p.gh_out) + hoff, gh);
    }
  }

  const int lt = tid / TT, lq = tid % TT;
  const int c0 = ct * CH + lq * RUN, nc = max(0, min(RUN, f.C - c0));
  float bias[RUN], dsk[RUN], gd[RUN], gbias[RUN];
#pragma unroll
  for (int i = 0; i < RUN; ++i) {
    bias[i] = f.dt_bias != nullptr && i < nc ? f.dt_bias[c0 + i] : 0.f;
    dsk[i] = f.d != nullptr && i < nc ? f.d[c0 + i] : 0.f;
    gd[i] = gbias[i] = 0.f;
  }
  Tile<T, N> R;
  int ts = t0 + (t1 - t0 - 1) / kTile * kTile;
  load_tile<T, N>(R, p, bb, ts + lt, t1, c0, nc);

  for (; ts >= t0; ts -= kTile) {
    const bool tact = ts + lt < t1;
    float sig[RUN], x[RUN], gpre[RUN];  // σ(dt + bias); x; gy silu'(z)
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      const bool on = tact && i < nc;
      float delta = softplus(R.dt[i] + bias[i], sig[i]);
      float g = R.gy[i];
      x[i] = R.x[i];
      gpre[i] = 0.f;
      if (f.z != nullptr) {
        const float s = sigmoid(R.z[i]);
        gpre[i] = g * s * fmaf(R.z[i], 1.f - s, 1.f);
        g *= R.z[i] * s;
      }
      sm.dxg[lt][lq * RUN + i] = on ? make_float4(delta, delta * x[i], g, 0.f) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (on) gd[i] = fmaf(g, x[i], gd[i]);
    }
    for (int i = tid; i < kTile * N; i += kThreads) {
      const int tk = i / N, n = i % N;
      const bool ok = ts + tk < t1;
      const size_t row = (size_t)bb * f.T + (ok ? ts + tk : 0);
      sm.b[tk][n] = ok ? IO<T>::to_f(static_cast<const T*>(f.b)[row * f.ldb + n]) : 0.f;
      sm.c[tk][n] = ok ? IO<T>::to_f(static_cast<const T*>(f.c)[row * f.ldc + n]) : 0.f;
    }
    float h0[kSN] = {0.f, 0.f, 0.f, 0.f};
    if (cact) load_vec<float, kSN>(f.ckpt + (size_t)(ts / kScanCkLen) * plane + hoff, h0);
    if (ts > t0) load_tile<T, N>(R, p, bb, ts - kTile + lt, t1, c0, nc);
    __syncthreads();

    float h[kSN];
#pragma unroll
    for (int i = 0; i < kSN; ++i) h[i] = h0[i];
#pragma unroll
    for (int k = 0; k < kSub; ++k) {
      const float4 d = sm.dxg[k][ch];
      float bv[kSN];
      load_vec<float, kSN>(&sm.b[k][sub * kSN], bv);
#pragma unroll
      for (int i = 0; i < kSN; ++i) h[i] = fmaf(ex2(d.x * a2[i]), h[i], d.y * bv[i]);
    }
#pragma unroll 1
    for (int half = 1; half >= 0; --half) {
      const int s0 = half * kSub;
      float e[kSub][kSN], eh[kSub][kSN];  // e_t, e_t h_{t-1}
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        const float4 d = sm.dxg[s0 + k][ch];
        float bv[kSN];
        load_vec<float, kSN>(&sm.b[s0 + k][sub * kSN], bv);
#pragma unroll
        for (int i = 0; i < kSN; ++i) {
          e[k][i] = ex2(d.x * a2[i]);
          eh[k][i] = e[k][i] * h[i];
          h[i] = fmaf(d.y, bv[i], eh[k][i]);
        }
      }
#pragma unroll
      for (int grp = kSub - 4; grp >= 0; grp -= 4) {
        float sp[4], s1[4], s2[4];
#pragma unroll
        for (int kk = 3; kk >= 0; --kk) {
          const int k = grp + kk;
          const float4 d = sm.dxg[s0 + k][ch];
          float bv[kSN], cv[kSN], v[2 * kSN];
          load_vec<float, kSN>(&sm.b[s0 + k][sub * kSN], bv);
          load_vec<float, kSN>(&sm.c[s0 + k][sub * kSN], cv);
          sp[kk] = s1[kk] = s2[kk] = 0.f;
#pragma unroll
          for (int i = 0; i < kSN; ++i) {
            const float ht = fmaf(d.y, bv[i], eh[k][i]);
            gh[i] = fmaf(cv[i], d.z, gh[i]);
            sp[kk] = fmaf(cv[i], ht, sp[kk]);
            s1[kk] = fmaf(gh[i], bv[i], s1[kk]);
            v[i] = d.z * ht;
            v[kSN + i] = d.y * gh[i];
            const float q = gh[i] * eh[k][i];
            s2[kk] = fmaf(q, a2[i], s2[kk]);
            ga[i] = fmaf(q, d.x, ga[i]);
            gh[i] *= e[k][i];
          }
          constexpr int M = CW < 8 ? CW : 8;  // lanes with different sums
          const int idx = lane / L;
          fold_lanes<2 * kSN, CW, L>(v, idx);
          if (idx < M) {
#pragma unroll
            for (int j = 0; j < 8 / M; ++j) {
              const int vi = idx * (8 / M) + j;
              sm.red[warp][s0 + k][(vi / kSN) * N + sub * kSN + vi % kSN] = v[j];
            }
          }
        }
        fold_lanes<4, L>(sp, sub);
        fold_lanes<4, L>(s1, sub);
        fold_lanes<4, L>(s2, sub);
        constexpr int ML = L < 4 ? L : 4;
        if (sub < ML) {
#pragma unroll
          for (int k = 0; k < 4 / ML; ++k) {
            const int tk = s0 + grp + sub * (4 / ML) + k;
            sm.sum[0][tk][ch] = sp[k];
            sm.sum[1][tk][ch] = s1[k];
            sm.sum[2][tk][ch] = s2[k];
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kSN; ++i) h[i] = h0[i];
    }
    __syncthreads();

    if (tact && nc > 0) {
      float ox[RUN], odt[RUN], oz[RUN];
#pragma unroll
      for (int i = 0; i < RUN; ++i) {
        const int cc = lq * RUN + i;
        const float4 d = sm.dxg[lt][cc];
        const float s1 = sm.sum[1][lt][cc], s2 = sm.sum[2][lt][cc];
        ox[i] = fmaf(d.x, s1, dsk[i] * d.z);
        odt[i] = sig[i] * fmaf(x[i], s1, s2 * kLn2);
        if (i < nc) gbias[i] += odt[i];
        oz[i] = gpre[i] * fmaf(dsk[i], x[i], sm.sum[0][lt][cc]);
      }
      const size_t off = ((size_t)bb * f.T + ts + lt) * f.C + c0;
      store_part<T, RUN>(static_cast<T*>(p.gx) + off, nc, f.vec, ox);
      store_part<T, RUN>(static_cast<T*>(p.gdt) + off, nc, f.vec, odt);
      if (p.gz != nullptr) store_part<T, RUN>(static_cast<T*>(p.gz) + off, nc, f.vec, oz);
    }
    float* part = p.part_bc + (((size_t)ct * f.B + bb) * f.T + ts) * (2 * N);
    for (int i = tid; i < kTile * 2 * N; i += kThreads) {
      const int tk = i / (2 * N), n = i % (2 * N);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sm.red[w][tk][n];
      if (ts + tk < t1) part[i] = s;
    }
    __syncthreads();  // the next tile overwrites Δ and g, which the outputs read
  }

  const size_t prow = (size_t)bb * f.nseg + seg;
  if (cact) {
    store_vec<float, kSN>(p.part_a + (prow * f.C + c) * N + sub * kSN, ga);
    if (seg == 0 && p.gh_in != nullptr) store_vec<float, kSN>(p.gh_in + hoff, gh);
  }
  // gd and gdt_bias: the 16 tokens of a run of channels meet in shared memory
  float* s_gd = &sm.sum[0][0][0];  // [16][CH] each, within sum[0] and sum[1]
  float* s_gb = &sm.sum[1][0][0];
#pragma unroll
  for (int i = 0; i < RUN; ++i) {
    s_gd[lt * CH + lq * RUN + i] = gd[i];
    s_gb[lt * CH + lq * RUN + i] = gbias[i];
  }
  __syncthreads();
  if (tid < CH && ct * CH + tid < f.C) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < kTile; ++k) {
      a += s_gd[k * CH + tid];
      b += s_gb[k * CH + tid];
    }
    p.part_v[(prow * 2 + 0) * f.C + ct * CH + tid] = a;
    p.part_v[(prow * 2 + 1) * f.C + ct * CH + tid] = b;
  }
}

// The gradient that leaves segments 1 .. nseg-1 at their start, from zero at their end (the last
// from gh_out), and their ΣΔ.  Thread = 4 states of one channel; a tile of 16 tokens through
// shared memory.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) scan_bwd_summary_kernel(const __grid_constant__ ScanBwdParams p) {
  using S = Shape<N>;
  constexpr int L = S::kLanes, CH = S::kCh, RUN = S::kRun, TT = S::kTokThreads;
  __shared__ float2 dg[kTile][CH];  // (Δ, g)
  __shared__ __align__(16) float sc[kTile][N];
  const ScanParams& f = p.f;
  const int tid = threadIdx.x;
  const int ct = (int)(blockIdx.x % (unsigned)f.ctiles);
  const unsigned rest = blockIdx.x / (unsigned)f.ctiles;
  const int seg = 1 + (int)(rest % (unsigned)(f.nseg - 1)), bb = (int)(rest / (unsigned)(f.nseg - 1));
  const int t0 = seg * f.seg_len, t1 = min(f.T, t0 + f.seg_len);
  const int ch = tid / L, sub = tid % L;
  const int c = ct * CH + ch;
  const bool cact = c < f.C;
  const size_t hoff = ((size_t)bb * f.C + c) * N + sub * kSN;
  float a2[kSN], gh[kSN];
#pragma unroll
  for (int i = 0; i < kSN; ++i) a2[i] = gh[i] = 0.f;
  if (cact) {
    load_rates<kSN>(f.a_log + (size_t)c * N + sub * kSN, a2);
    if (seg == f.nseg - 1 && p.gh_out != nullptr) {
      load_vec<float, kSN>(p.gh_out + hoff, gh);
      store_vec<float, kSN>(p.seg_g0 + hoff, gh);
    }
  }
  const int lt = tid / TT, lq = tid % TT;
  const int c0 = ct * CH + lq * RUN, nc = max(0, min(RUN, f.C - c0));
  float bias[RUN];
#pragma unroll
  for (int i = 0; i < RUN; ++i) bias[i] = f.dt_bias != nullptr && i < nc ? f.dt_bias[c0 + i] : 0.f;
  float sumdt = 0.f;
  for (int ts = t0 + (t1 - t0 - 1) / kTile * kTile; ts >= t0; ts -= kTile) {
    const bool ok = ts + lt < t1;
    const size_t row = (size_t)bb * f.T + (ok ? ts + lt : 0);
    const int n = ok ? nc : 0;
    float dt[RUN], g[RUN], z[RUN];
    load_part<T, RUN>(static_cast<const T*>(f.dt) + row * f.lddt + c0, n, f.vec, dt);
    load_part<T, RUN>(static_cast<const T*>(p.gy) + row * f.C + c0, n, f.vec, g);
    if (f.z != nullptr) load_part<T, RUN>(static_cast<const T*>(f.z) + row * f.ldz + c0, n, f.vec, z);
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      float sig;
      const float delta = softplus(dt[i] + bias[i], sig);
      if (f.z != nullptr) g[i] *= z[i] * sigmoid(z[i]);
      dg[lt][lq * RUN + i] = i < n ? make_float2(delta, g[i]) : make_float2(0.f, 0.f);
    }
    for (int i = tid; i < kTile * N; i += kThreads) {
      const int tk = i / N;
      sc[tk][i % N] = ts + tk < t1 ? IO<T>::to_f(static_cast<const T*>(f.c)[((size_t)bb * f.T + ts + tk) * f.ldc + i % N])
                                   : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = kTile - 1; k >= 0; --k) {
      const float2 d = dg[k][ch];
      float cv[kSN];
      load_vec<float, kSN>(&sc[k][sub * kSN], cv);
#pragma unroll
      for (int i = 0; i < kSN; ++i) gh[i] = ex2(d.x * a2[i]) * fmaf(cv[i], d.y, gh[i]);
      sumdt += d.x;
    }
    __syncthreads();
  }
  if (cact) {
    store_vec<float, kSN>(p.seg_g + (size_t)seg * f.B * f.C * N + hoff, gh);
    if (sub == 0) p.seg_dt[((size_t)seg * f.B + bb) * f.C + c] = sumdt;
  }
}

// gb, gc: the channel tiles' parts added in order, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_bc_kernel(int ctiles, size_t n, int N, const float* __restrict__ part,
                                                          T* gb, T* gc) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;  // over [B,T][2][N]
  if (i >= n) return;
  float s = 0.f;
  for (int k = 0; k < ctiles; ++k) s += part[(size_t)k * n + i];
  const size_t row = i / (2 * N);
  const int j = (int)(i % (2 * N));
  (j < N ? gc : gb)[row * N + j % N] = IO<T>::from_f(s);
}

// ga_log [C,N], then gd [C] and gdt_bias [C]: the parts of the batch rows and segments in order.
__global__ void __launch_bounds__(256) scan_bwd_param_kernel(int nparts, int C, int N, const float* __restrict__ a_log,
                                                             const float* __restrict__ part_a,
                                                             const float* __restrict__ part_v, float* ga_log, float* gd,
                                                             float* gdt_bias) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, na = (size_t)C * N;
  if (i < na) {
    double s = 0.0;
    for (int k = 0; k < nparts; ++k) s += (double)part_a[(size_t)k * na + i];
    ga_log[i] = (float)(s * -(double)expf(a_log[i]));
  } else if (i < na + 2 * (size_t)C) {
    const size_t j = i - na;
    float* dst = j < (size_t)C ? gd : gdt_bias;
    if (dst == nullptr) return;
    double s = 0.0;
    for (int k = 0; k < nparts; ++k) s += (double)part_v[(size_t)k * 2 * C + j];
    dst[j % C] = (float)s;
  }
}

template <typename T, int N>
cudaError_t bwd_n(ScanBwdParams p, cudaStream_t st) {
  static unsigned mask = 0;
  p.f.ctiles = (p.f.C + Shape<N>::kCh - 1) / Shape<N>::kCh;
  const unsigned rows = (unsigned)p.f.ctiles * (unsigned)p.f.B;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(scan_bwd_kernel<T, N>), (int)sizeof(Smem<N>), &mask);
  if (e != cudaSuccess) return e;
  if (p.f.nseg > 1) {
    scan_bwd_summary_kernel<T, N><<<rows * (unsigned)(p.f.nseg - 1), kThreads, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  scan_bwd_kernel<T, N><<<rows * (unsigned)p.f.nseg, kThreads, sizeof(Smem<N>), st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const size_t n = (size_t)p.f.B * p.f.T * 2 * N;
  scan_bwd_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(p.f.ctiles, n, N, p.part_bc,
                                                                     static_cast<T*>(p.gb), static_cast<T*>(p.gc));
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const size_t m = (size_t)p.f.C * N + 2 * (size_t)p.f.C;
  scan_bwd_param_kernel<<<(unsigned)((m + 255) / 256), 256, 0, st>>>(p.f.B * p.f.nseg, p.f.C, N, p.f.a_log, p.part_a,
                                                                    p.part_v, p.ga_log, p.gd, p.gdt_bias);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const ScanBwdParams& p, cudaStream_t st) {
  switch (p.f.N) {
    case 8: return bwd_n<T, 8>(p, st);
    case 16: return bwd_n<T, 16>(p, st);
    case 32: return bwd_n<T, 32>(p, st);
    case 64: return bwd_n<T, 64>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int scan_bwd_channels(int N) { return kThreads * kSN / N; }

cudaError_t launch_scan_bwd(bool bf16, const ScanBwdParams& p, cudaStream_t st) {
  return bf16 ? bwd_t<__nv_bfloat16>(p, st) : bwd_t<float>(p, st);
}

}  // namespace rwkv
