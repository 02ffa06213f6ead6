// Short causal convolution over time, one filter per channel (sm_100a):
//   pre_t[c] = bias[c] + Σ_{j<W} w[c][j] x_{t-W+1+j}[c],   y = pre or silu(pre) = pre σ(pre),
// with the W-1 tokens before the first taken from a state [B,W-1,C] (oldest first; zero without one).
// W = 2 is the token shift μ x_t + (1-μ) x_{t-1} of "RWKV - Transformer 시대에 RNN을 재발명하다",
// Method / (1); W = 4 stands before a selective scan.
//
// Backward, with g_t = gy_t act'(pre_t) (0 past the end) and silu'(p) = σ(p)(1 + p(1 - σ(p))):
//   gx_t = Σ_j w[j] g_{t+W-1-j} (the same sum at t < 0 is the state's gradient),
//   gw[c][j] = Σ_{b,t} g_t x_{t-W+1+j},   gbias[c] = Σ_{b,t} g_t.
// pre is recomputed from x (W FMAs) rather than kept by the forward.
//
// Everything is one pass over the data, so bandwidth bounds it.  A thread owns V channels of one
// stretch of tokens and slides a W-token window along it in registers; the tokens ahead are fetched
// 8 at a time and left as loaded until they are due.  V is small (8 bytes a load forward, 4 to 8
// backward, whose two windows and W+1 sums are kept besides) so that enough threads fit on an SM to
// keep its loads in flight.  Neighbouring stretches re-read W-1 tokens, which come from L2.
// At 4x4096x2560 bf16, W = 4: forward 32 us (5.2 TB/s, 82 % of a copy's rate), backward 64 + 4 us of
// reduction (3.9 TB/s; about half of its cycles issue, and two CTAs of 128 registers a thread fill an
// SM).  Fetching 4 or 12 tokens together in the backward, or 4 channels a thread, measured 3 to 25 %
// slower.
#include "mixer.h"
#include "mixer_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 128;
// Tokens per thread, forward: as many as keep the re-read of W-1 small, fewer where that would leave
// most of the GPU idle and only the walk's length counts (1 x 37 x 768 in fp32: 4.5 us, 6.0 with 32).
constexpr int kFwdStretch = 32, kShortStretch = 8;
constexpr int kBwdStretch = 64;  // tokens per thread, backward
constexpr int kBwdWarps = 8;     // stretches per CTA (their weight-gradient sums meet in shared memory)
constexpr int kStepStreams = 2;  // streams per thread, step
constexpr int kAhead = 8;        // tokens fetched together, forward
constexpr int kBwdAhead = 8;     // tokens fetched together, backward

// Channels are worked on in pairs (packed arithmetic).  V > 1: a thread owns V neighbouring channels, in
// one access.  V = 1, where rows or bases do not allow that: a pair is a channel of the first half and
// the one as far into the second, each in accesses that lie side by side in a warp (4x4096x2561 bf16: 47
// us and 105 backward; with one channel a thread 51 and 121; in fp32, 2048 tokens, 34 and 68, 34 and 91).
template <int V>
constexpr int kPairs = (V + 1) / 2;
template <int V>
constexpr int kOwn = V == 1 ? 2 : V;  // channels of a thread

// Threads for C channels.
template <int V>
__host__ __device__ __forceinline__ int channel_threads(int C) {
  return V == 1 ? (C + 1) / 2 : C / V;
}
// V = 1: from a thread's first channel c to its second; 0 behind the last of an odd number, where the
// thread then works on c twice.
template <int V>
__device__ __forceinline__ int second(const ConvParams& p, int c) {
  const int half = (p.C + 1) / 2;
  return V == 1 && c + half < p.C ? half : 0;
}

// A thread's channels of one token as loaded.
template <typename T, int V>
struct Elem {
  Raw<T, V> r[V == 1 ? 2 : 1];
  __device__ __forceinline__ void load(const T* p, int off) {
    r[0].load(p);
    if constexpr (V == 1) r[1].load(p + off);
  }
  __device__ __forceinline__ void zero() {
    r[0].zero();
    if constexpr (V == 1) r[1].zero();
  }
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (V == 1)
      return make_float2(r[0][0], r[1][0]);
    else
      return r[0].pair(i);
  }
};
template <typename T, int V>
__device__ __forceinline__ void store_elem(T* p, int off, const float2 (&o)[kPairs<V>]) {
  if constexpr (V == 1) {
    p[0] = IO<T>::from_f(o[0].x);
    p[off] = IO<T>::from_f(off != 0 ? o[0].y : o[0].x);
  } else {
    store_pairs_as<T, V>(p, o);
  }
}

// Element of the concatenation (state, x): position k < W-1 is state row k, the rest token k-(W-1).
template <typename T, int V, int W>
__device__ __forceinline__ void load_pos(const ConvParams& p, int b, int k, int c, int off, float2 (&f)[kPairs<V>]) {
  const int t = k - (W - 1);
  Elem<T, V> r;
  if (t >= 0)
    r.load(static_cast<const T*>(p.x) + ((size_t)b * p.T + t) * p.ldx + c, off);
  else if (p.state_in != nullptr)
    r.load(static_cast<const T*>(p.state_in) + ((size_t)b * (W - 1) + k) * p.C + c, off);
  else
    r.zero();
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) f[i] = r.pair(i);
}

// The filters and biases of a thread's channels (V > 1: W V consecutive floats, aligned for wide loads).
template <int V, int W>
__device__ __forceinline__ void load_filter(const ConvParams& p, int c, int off, float2 (&w)[W][kPairs<V>],
                                            float2 (&bias)[kPairs<V>]) {
  if constexpr (V == 1) {
#pragma unroll
    for (int j = 0; j < W; ++j)
      w[j][0] = make_float2(p.weight[(size_t)c * W + j], p.weight[(size_t)(c + off) * W + j]);
    bias[0] = p.bias != nullptr ? make_float2(p.bias[c], p.bias[c + off]) : dup2(0.f);
  } else {
    constexpr int Q = (V * W) % 4 == 0 ? 4 : 2;
    float f[V * W];
    const float* q = p.weight + (size_t)c * W;
#pragma unroll
    for (int i = 0; i < V * W; i += Q) {
      if constexpr (Q == 4) {
        const float4 x = *reinterpret_cast<const float4*>(q + i);
        f[i] = x.x, f[i + 1] = x.y, f[i + 2] = x.z, f[i + 3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(q + i);
        f[i] = x.x, f[i + 1] = x.y;
      }
    }
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][i] = make_float2(f[2 * i * W + j], f[(2 * i + 1) * W + j]);
      bias[i] = p.bias != nullptr ? make_float2(p.bias[c + 2 * i], p.bias[c + 2 * i + 1]) : dup2(0.f);
    }
  }
}

// Slides a window by one token.
template <int W, int P>
__device__ __forceinline__ void slide(float2 (&win)[W][P]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) win[j][i] = win[j + 1][i];
}

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(const __grid_constant__ ConvParams p) {
  constexpr int P = kPairs<V>;
  const int ncv = channel_threads<V>(p.C);
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int cv = (int)(id % ncv);
  const long long rest = id / ncv;
  const int seg = (int)(rest % p.nseg);
  const long long b64 = rest / p.nseg;
  if (b64 >= p.B) return;
  const int b = (int)b64, c = cv * V, off = second<V>(p, c);
  const int t0 = seg * p.stretch, t1 = min(p.T, t0 + p.stretch);
  const T* xr = static_cast<const T*>(p.x) + ((size_t)b * p.T + t0) * p.ldx + c;
  T* yr = static_cast<T*>(p.y) + ((size_t)b * p.T + t0) * p.C + c;
  Elem<T, V> nx[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a)
    if (t0 + a < t1) nx[a].load(xr + (size_t)a * p.ldx, off);
  float2 w[W][P], bias[P], win[W][P];  // win[j]: the token j - (W-1) steps from the current one
  load_filter<V, W>(p, c, off, w, bias);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, b, t0 + j, c, off, win[j + 1]);
  const auto token = [&](const Elem<T, V>& x, T* y) {
    slide(win);
    float2 o[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      win[W - 1][i] = x.pair(i);
      float2 acc = bias[i];
#pragma unroll
      for (int j = 0; j < W; ++j) acc = fma2(w[j][i], win[j][i], acc);
      o[i] = SILU ? mul2(acc, sigmoid2(acc)) : acc;
    }
    store_elem<T, V>(y, off, o);
  };
  for (int t = t0; t < t1; t += kAhead) {
    Elem<T, V> cur[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) cur[a] = nx[a];
    xr += (size_t)kAhead * p.ldx;
    if (t + 2 * kAhead <= t1) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) nx[a].load(xr + (size_t)a * p.ldx, off);
    } else {
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (t + kAhead + a < t1) nx[a].load(xr + (size_t)a * p.ldx, off);
    }
    if (t + kAhead <= t1) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) token(cur[a], yr + (size_t)a * p.C);
    } else {
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (t + a < t1) token(cur[a], yr + (size_t)a * p.C);
    }
    yr += (size_t)kAhead * p.C;
  }
  // The state after the last token is written by the thread that read the state before the first,
  // so that both may be the same array.
  if (seg == 0 && p.state_out != nullptr) {
    float2 last[W - 1][P];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, b, p.T + j, c, off, last[j]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_elem<T, V>(static_cast<T*>(p.state_out) + ((size_t)b * (W - 1) + j) * p.C + c, off, last[j]);
  }
}

// One warp per stretch: lane = channel group.  part: [B * ceil(nseg / kBwdWarps)][W+1][C] sums of
// the weight gradients (plane W: the bias's).
template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(32 * kBwdWarps) conv_bwd_kernel(const __grid_constant__ ConvParams p) {
  constexpr int P = kPairs<V>;
  constexpr int CW = 32 * kOwn<V>;  // channels of a warp; V = 1: the first half's, then the second's
  __shared__ float red[kBwdWarps][W + 1][CW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ncv = channel_threads<V>(p.C), ncg = (ncv + 31) / 32;  // groups of 32 threads' channels
  const int nsg = (p.nseg + kBwdWarps - 1) / kBwdWarps;            // groups of stretches
  const int cg = (int)(blockIdx.x % (unsigned)ncg);
  const unsigned rest = blockIdx.x / (unsigned)ncg;
  const int b = (int)(rest / (unsigned)nsg), seg = (int)(rest % (unsigned)nsg) * kBwdWarps + warp;
  const int c = (cg * 32 + lane) * V, off = second<V>(p, c);
  const bool act = cg * 32 + lane < ncv && seg < p.nseg;
  float2 gw[W + 1][P];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) gw[j][i] = dup2(0.f);
  if (act) {
    // g_t is needed for the stretch's tokens and the W-1 behind them (0 past the end of the sequence)
    const int t0 = seg * kBwdStretch, t1 = min(p.T, t0 + kBwdStretch), tend = t1 + W - 1;
    float2 w[W][P], bias[P], win[W][P], gp[W][P];  // gp[j]: g of the token j - (W-1) steps from the current one
    const T* xr = static_cast<const T*>(p.x) + ((size_t)b * p.T + t0) * p.ldx + c;
    const T* gr = static_cast<const T*>(p.gy) + ((size_t)b * p.T + t0) * p.C + c;
    T* gxr = static_cast<T*>(p.gx) + ((size_t)b * p.T + t0) * p.C + c;  // of the token being fetched for
    Elem<T, V> nx[kBwdAhead], ng[kBwdAhead];
    const auto fetch = [&](int t) {  // tokens t .. t + kBwdAhead - 1, xr and gr pointing at the first
      if (t + kBwdAhead <= p.T) {
#pragma unroll
        for (int a = 0; a < kBwdAhead; ++a) {
          nx[a].load(xr + (size_t)a * p.ldx, off);
          ng[a].load(gr + (size_t)a * p.C, off);
        }
      } else {
#pragma unroll
        for (int a = 0; a < kBwdAhead; ++a)
          if (t + a < p.T) {
            nx[a].load(xr + (size_t)a * p.ldx, off);
            ng[a].load(gr + (size_t)a * p.C, off);
          }
      }
    };
    fetch(t0);
    load_filter<V, W>(p, c, off, w, bias);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int i = 0; i < P; ++i) gp[j][i] = dup2(0.f);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, b, t0 + j, c, off, win[j + 1]);

    // g of one token; its part of the weight gradients when the stretch owns it
    const auto grad = [&](const Elem<T, V>& x, const Elem<T, V>& gy, bool own) {
      slide(gp);
      slide(win);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        win[W - 1][i] = x.pair(i);
        float2 g = gy.pair(i);
        if constexpr (SILU) {
          float2 pre = bias[i];
#pragma unroll
          for (int j = 0; j < W; ++j) pre = fma2(w[j][i], win[j][i], pre);
          const float2 s = sigmoid2(pre);
          g = mul2(mul2(g, s), fma2(pre, fma2(s, dup2(-1.f), dup2(1.f)), dup2(1.f)));
        }
        gp[W - 1][i] = g;
        if (own) {
#pragma unroll
          for (int j = 0; j < W; ++j) gw[j][i] = fma2(g, win[j][i], gw[j][i]);
          gw[W][i] = add2(g, gw[W][i]);
        }
      }
    };
    // gx of the token W-1 before the current one, on top of e
    const auto back = [&](float2 (&e)[P]) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) e[i] = fma2(w[j][i], gp[W - 1 - j][i], e[i]);
    };
    for (int t = t0; t < tend; t += kBwdAhead) {
      Elem<T, V> cx[kBwdAhead], cg_[kBwdAhead];
#pragma unroll
      for (int a = 0; a < kBwdAhead; ++a) cx[a] = nx[a], cg_[a] = ng[a];
      xr += (size_t)kBwdAhead * p.ldx;
      gr += (size_t)kBwdAhead * p.C;
      if (t + kBwdAhead < tend) fetch(t + kBwdAhead);
      const bool first = t == t0;
      if (t + kBwdAhead <= t1 && !(first && seg == 0 && p.gstate_in != nullptr)) {
        // all tokens owned; the first W-1 gradients of the stretch's first turn belong before it
#pragma unroll
        for (int a = 0; a < kBwdAhead; ++a) {
          grad(cx[a], cg_[a], true);
          if (a < W - 1 && first) continue;
          float2 o[P];
#pragma unroll
          for (int i = 0; i < P; ++i) o[i] = dup2(0.f);
          back(o);
          store_elem<T, V>(gxr + (ptrdiff_t)(a - (W - 1)) * p.C, off, o);
        }
      } else {
#pragma unroll
        for (int a = 0; a < kBwdAhead; ++a) {
          const int ta = t + a;
          if (ta >= tend) break;
          if (ta < p.T) {
            grad(cx[a], cg_[a], ta < t1);
          } else {
            slide(gp);
#pragma unroll
            for (int i = 0; i < P; ++i) gp[W - 1][i] = dup2(0.f);
          }
          // token ta - (W-1), or a row of the state where that is negative; its stretch owns it when it
          // is not before t0 (the first stretch owns the state)
          const int to = ta - (W - 1);
          if (to >= t0 || (seg == 0 && p.gstate_in != nullptr)) {
            float2 o[P];
            const int k = to + W - 1 - p.T;  // its row of the final state, when >= 0
            Elem<T, V> e;
            if (k >= 0 && p.gstate_out != nullptr)
              e.load(static_cast<const T*>(p.gstate_out) + ((size_t)b * (W - 1) + k) * p.C + c, off);
            else
              e.zero();
#pragma unroll
            for (int i = 0; i < P; ++i) o[i] = e.pair(i);
            back(o);
            if (to >= 0)
              store_elem<T, V>(gxr + (ptrdiff_t)(a - (W - 1)) * p.C, off, o);
            else
              store_elem<T, V>(static_cast<T*>(p.gstate_in) + ((size_t)b * (W - 1) + to + W - 1) * p.C + c, off, o);
          }
        }
      }
      gxr += (size_t)kBwdAhead * p.C;
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < kOwn<V>; ++i)
      red[warp][j][V == 1 ? i * 32 + lane : lane * V + i] = i & 1 ? gw[j][i / 2].y : gw[j][i / 2].x;
  __syncthreads();
  float* part = p.part + (size_t)rest * (W + 1) * p.C;
  for (int i = threadIdx.x; i < (W + 1) * CW; i += 32 * kBwdWarps) {
    const int j = i / CW, cc = i % CW, at = cg * 32 + (cc & 31);
    const int col = V == 1 ? at + (cc < 32 ? 0 : ncv) : cg * CW + cc;
    if (col >= p.C || (V == 1 && at >= ncv)) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kBwdWarps; ++k) s += red[k][j][cc];
    part[(size_t)j * p.C + col] = s;
  }
}

// gweight[c][j] and gbias[c]: the parts summed in order, 32 columns by 8 rows of threads, a thread's
// loads 4 at a time.
__global__ void __launch_bounds__(256) conv_reduce_kernel(int nparts, int C, int W, const float* __restrict__ part,
                                                          float* gweight, float* gbias) {
  __shared__ float red[8][32];
  const size_t n = (size_t)(W + 1) * C;
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const size_t i = (size_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (i < n) {
    const float* q = part + i;
    int k = r;
    for (; k + 3 * 8 < nparts; k += 4 * 8) {
      const float a = q[(size_t)k * n], b = q[(size_t)(k + 8) * n], c = q[(size_t)(k + 16) * n],
                  d = q[(size_t)(k + 24) * n];
      s += (a + b) + (c + d);
    }
    for (; k < nparts; k += 8) s += q[(size_t)k * n];
  }
  red[r][lane] = s;
  __syncthreads();
  if (r != 0 || i >= n) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) s += red[k][lane];
  const int j = (int)(i / C), c = (int)(i % C);
  if (j < W)
    gweight[(size_t)c * W + j] = s;
  else if (gbias != nullptr)
    gbias[c] = s;
}

// One token per stream: the window is the state's rows and the token; the rows move up by one.  A
// thread reads every row of its channels before it writes one, so state_out may be state_in.  It
// takes kStepStreams streams, whose loads are in flight together and share the filters.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const __grid_constant__ ConvParams p) {
  constexpr int P = kPairs<V>;
  const int ncv = channel_threads<V>(p.C);
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long b0 = id / ncv * kStepStreams;
  if (b0 >= p.B) return;
  const int c = (int)(id % ncv) * V, off = second<V>(p, c), nb = (int)min((long long)kStepStreams, p.B - b0);
  float2 win[kStepStreams][W][P], w[W][P], bias[P];
#pragma unroll
  for (int k = 0; k < kStepStreams; ++k) {
    const int b = (int)b0 + (k < nb ? k : 0);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, b, j, c, off, win[k][j]);
    Elem<T, V> x;
    x.load(static_cast<const T*>(p.x) + (size_t)b * p.ldx + c, off);
#pragma unroll
    for (int i = 0; i < P; ++i) win[k][W - 1][i] = x.pair(i);
  }
  load_filter<V, W>(p, c, off, w, bias);
#pragma unroll
  for (int k = 0; k < kStepStreams; ++k) {
    if (k >= nb) break;
    const size_t b = (size_t)b0 + k;
    float2 o[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float2 acc = bias[i];
#pragma unroll
      for (int j = 0; j < W; ++j) acc = fma2(w[j][i], win[k][j][i], acc);
      o[i] = p.silu ? mul2(acc, sigmoid2(acc)) : acc;
    }
    store_elem<T, V>(static_cast<T*>(p.y) + b * p.C + c, off, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_elem<T, V>(static_cast<T*>(p.state_out) + (b * (W - 1) + j) * p.C + c, off, win[k][j + 1]);
  }
}

// T = 0: the final state is the first (and its gradient passes through).
__global__ void copy_bytes_kernel(size_t n, const unsigned char* src, unsigned char* dst) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) dst[i] = src != nullptr ? src[i] : 0;
}

template <typename T, int V, int W>
cudaError_t fwd_vw(ConvParams p, cudaStream_t st) {
  const long long threads = (long long)p.B * ((p.T + kFwdStretch - 1) / kFwdStretch) * channel_threads<V>(p.C);
  p.stretch = threads < 148 * kThreads ? kShortStretch : kFwdStretch;
  p.nseg = (p.T + p.stretch - 1) / p.stretch;
  const long long n = (long long)p.B * p.nseg * channel_threads<V>(p.C);
  const auto kernel = p.silu ? conv_fwd_kernel<T, V, W, true> : conv_fwd_kernel<T, V, W, false>;
  kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t bwd_vw(ConvParams p, cudaStream_t st) {
  p.nseg = (p.T + kBwdStretch - 1) / kBwdStretch;
  const int nparts = conv_bwd_parts(p.B, p.T);
  const int ncg = (channel_threads<V>(p.C) + 31) / 32;
  const auto kernel = p.silu ? conv_bwd_kernel<T, V, W, true> : conv_bwd_kernel<T, V, W, false>;
  kernel<<<(unsigned)nparts * (unsigned)ncg, 32 * kBwdWarps, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t n = (size_t)(W + 1) * p.C;
  conv_reduce_kernel<<<(unsigned)((n + 31) / 32), 256, 0, st>>>(nparts, p.C, W, p.part, p.gweight, p.gbias);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t step_vw(const ConvParams& p, cudaStream_t st) {
  const long long n = ((long long)p.B + kStepStreams - 1) / kStepStreams * channel_threads<V>(p.C);
  conv_step_kernel<T, V, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run_v(ConvPass pass, const ConvParams& p, cudaStream_t st) {
  switch (pass) {
    case ConvPass::kForward:
      return p.W == 2 ? fwd_vw<T, V, 2>(p, st) : p.W == 3 ? fwd_vw<T, V, 3>(p, st) : fwd_vw<T, V, 4>(p, st);
    case ConvPass::kBackward: {
      constexpr int VB = V > 2 ? 2 : V;
      return p.W == 2 ? bwd_vw<T, VB, 2>(p, st) : p.W == 3 ? bwd_vw<T, VB, 3>(p, st) : bwd_vw<T, VB, 4>(p, st);
    }
    case ConvPass::kStep:
      return p.W == 2 ? step_vw<T, V, 2>(p, st) : p.W == 3 ? step_vw<T, V, 3>(p, st) : step_vw<T, V, 4>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int conv_bwd_parts(int B, int T) {
  const int nseg = (T + kBwdStretch - 1) / kBwdStretch;
  return B * ((nseg + kBwdWarps - 1) / kBwdWarps);
}

cudaError_t launch_conv(ConvPass pass, bool bf16, int width, const ConvParams& p, cudaStream_t st) {
  if (!bf16) return width >= 2 ? run_v<float, 2>(pass, p, st) : run_v<float, 1>(pass, p, st);
  return width >= 4   ? run_v<__nv_bfloat16, 4>(pass, p, st)
         : width >= 2 ? run_v<__nv_bfloat16, 2>(pass, p, st)
                      : run_v<__nv_bfloat16, 1>(pass, p, st);
}

cudaError_t launch_copy_bytes(size_t n, const void* src, void* dst, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  copy_bytes_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(n, static_cast<const unsigned char*>(src),
                                                                 static_cast<unsigned char*>(dst));
  return cudaGetLastError();
}

}  // namespace rwkv
