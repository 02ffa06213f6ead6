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
#include "launch.h"
#include "mixer_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 128;
constexpr int kFwdStretch = 32;  // tokens per thread, forward
constexpr int kBwdStretch = 64;  // tokens per thread, backward
constexpr int kBwdWarps = 8;     // stretches per CTA (their weight-gradient sums meet in shared memory)
constexpr int kAhead = 8;        // tokens fetched together

// Element of the concatenation (state, x): position k < W-1 is state row k, the rest token k-(W-1).
template <typename T, int V, int W>
__device__ __forceinline__ void load_pos(const ConvParams& p, int b, int k, int c, float (&f)[V]) {
  const int t = k - (W - 1);
  if (t >= 0) {
    load_vec<T, V>(static_cast<const T*>(p.x) + ((size_t)b * p.T + t) * p.ldx + c, f);
  } else if (p.state_in != nullptr) {
    load_vec<T, V>(static_cast<const T*>(p.state_in) + ((size_t)b * (W - 1) + k) * p.C + c, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
  }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(ConvParams p) {
  const int ncv = p.C / V;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int cv = (int)(id % ncv);
  const long long rest = id / ncv;
  const int seg = (int)(rest % p.nseg);
  const long long b64 = rest / p.nseg;
  if (b64 >= p.B) return;
  const int b = (int)b64, c = cv * V;
  const int t0 = seg * kFwdStretch, t1 = min(p.T, t0 + kFwdStretch);
  float w[W][V], bias[V], win[W][V];  // win[j]: the token j - (W-1) steps from the current one
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = p.bias != nullptr ? p.bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = p.weight[(size_t)(c + i) * W + j];
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, b, t0 + j, c, win[j + 1]);
  const T* xr = static_cast<const T*>(p.x) + (size_t)b * p.T * p.ldx + c;
  T* yr = static_cast<T*>(p.y) + (size_t)b * p.T * p.C + c;
  Raw<T, V> nx[kAhead];
  const auto fetch = [&](int t) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (t + a < t1) nx[a].load(xr + (size_t)(t + a) * p.ldx, V, true);
  };
  fetch(t0);
  for (int t = t0; t < t1; t += kAhead) {
    Raw<T, V> cur[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) cur[a] = nx[a];
    fetch(t + kAhead);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (t + a >= t1) break;
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
        win[W - 1][i] = cur[a][i];
        float acc = bias[i];
#pragma unroll
        for (int j = 0; j < W; ++j) acc = fmaf(w[j][i], win[j][i], acc);
        o[i] = p.silu ? acc * sigmoid_ex2(acc) : acc;
      }
      store_vec<T, V>(yr + (size_t)(t + a) * p.C, o);
    }
  }
  // The state after the last token is written by the thread that read the state before the first,
  // so that both may be the same array.
  if (seg == 0 && p.state_out != nullptr) {
    float last[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, b, p.T + j, c, last[j]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      store_vec<T, V>(static_cast<T*>(p.state_out) + ((size_t)b * (W - 1) + j) * p.C + c, last[j]);
  }
}

// One warp per stretch: lane = channel group.  part: [B * ceil(nseg / kBwdWarps)][W+1][C] sums of
// the weight gradients (plane W: the bias's).
template <typename T, int V, int W>
__global__ void __launch_bounds__(32 * kBwdWarps) conv_bwd_kernel(ConvParams p) {
  __shared__ float red[kBwdWarps][W + 1][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ncg = (p.C / V + 31) / 32;                        // channel groups of 32 V
  const int nsg = (p.nseg + kBwdWarps - 1) / kBwdWarps;       // groups of stretches
  const int cg = (int)(blockIdx.x % (unsigned)ncg);
  const unsigned rest = blockIdx.x / (unsigned)ncg;
  const int b = (int)(rest / (unsigned)nsg), seg = (int)(rest % (unsigned)nsg) * kBwdWarps + warp;
  const int c = (cg * 32 + lane) * V;
  const bool act = c < p.C && seg < p.nseg;
  float gw[W + 1][V];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) gw[j][i] = 0.f;
  if (act) {
    const int t0 = seg * kBwdStretch, t1 = min(p.T, t0 + kBwdStretch);
    float w[W][V], bias[V], win[W][V], gp[W][V];  // gp[j]: g of the token j - (W-1) steps from the current one
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = p.bias != nullptr ? p.bias[c + i] : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        w[j][i] = p.weight[(size_t)(c + i) * W + j];
        gp[j][i] = 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, b, t0 + j, c, win[j + 1]);
    const T* xr = static_cast<const T*>(p.x) + (size_t)b * p.T * p.ldx + c;
    const T* gr = static_cast<const T*>(p.gy) + (size_t)b * p.T * p.C + c;
    T* gxr = static_cast<T*>(p.gx) + (size_t)b * p.T * p.C + c;
    const int tend = t1 + W - 1;
    Raw<T, V> nx[kAhead], ng[kAhead];
    const auto fetch = [&](int t) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (t + a < tend && t + a < p.T) {
          nx[a].load(xr + (size_t)(t + a) * p.ldx, V, true);
          ng[a].load(gr + (size_t)(t + a) * p.C, V, true);
        }
    };
    fetch(t0);
    for (int t = t0; t < tend; t += kAhead) {
      Raw<T, V> cx[kAhead], cg[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) cx[a] = nx[a], cg[a] = ng[a];
      fetch(t + kAhead);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int ta = t + a;
        if (ta >= tend) break;
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) gp[j][i] = gp[j + 1][i];
          gp[W - 1][i] = 0.f;
        }
        if (ta < p.T) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j][i] = win[j + 1][i];
            win[W - 1][i] = cx[a][i];
            float g = cg[a][i];
            if (p.silu) {
              float pre = bias[i];
#pragma unroll
              for (int j = 0; j < W; ++j) pre = fmaf(w[j][i], win[j][i], pre);
              const float s = sigmoid_ex2(pre);
              g *= s * fmaf(pre, 1.f - s, 1.f);
            }
            gp[W - 1][i] = g;
            if (ta < t1) {
#pragma unroll
              for (int j = 0; j < W; ++j) gw[j][i] = fmaf(g, win[j][i], gw[j][i]);
              gw[W][i] += g;
            }
          }
        }
        // the gradient of token ta - (W-1), or of a row of the state where that is negative; its
        // stretch owns it when it is not before t0 (the first stretch owns the state)
        const int to = ta - (W - 1);
        if (to >= t0 || (seg == 0 && p.gstate_in != nullptr)) {
          float o[V], e[V];
          const int k = to + W - 1 - p.T;  // its row of the final state, when >= 0
          if (k >= 0 && p.gstate_out != nullptr) {
            load_vec<T, V>(static_cast<const T*>(p.gstate_out) + ((size_t)b * (W - 1) + k) * p.C + c, e);
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float acc = e[i];
#pragma unroll
            for (int j = 0; j < W; ++j) acc = fmaf(w[j][i], gp[W - 1 - j][i], acc);
            o[i] = acc;
          }
          if (to >= 0)
            store_vec<T, V>(gxr + (size_t)to * p.C, o);
          else
            store_vec<T, V>(static_cast<T*>(p.gstate_in) + ((size_t)b * (W - 1) + to + W - 1) * p.C + c, o);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][j][lane * V + i] = gw[j][i];
  __syncthreads();
  float* part = p.part + (size_t)rest * (W + 1) * p.C;
  for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += 32 * kBwdWarps) {
    const int j = i / (32 * V), cc = i % (32 * V), col = cg * 32 * V + cc;
    if (col >= p.C) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kBwdWarps; ++k) s += red[k][j][cc];
    part[(size_t)j * p.C + col] = s;
  }
}

// gweight[c][j] and gbias[c]: the parts summed in order (fp64: their number grows with the batch).
__global__ void __launch_bounds__(kThreads) conv_reduce_kernel(int nparts, int C, int W, const float* __restrict__ part,
                                                               float* gweight, float* gbias) {
  const size_t n = (size_t)(W + 1) * C;
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= n) return;
  double s = 0.0;
  for (int k = 0; k < nparts; ++k) s += (double)part[(size_t)k * n + i];
  const int j = (int)(i / C), c = (int)(i % C);
  if (j < W)
    gweight[(size_t)c * W + j] = (float)s;
  else if (gbias != nullptr)
    gbias[c] = (float)s;
}

// One token per stream: the window is the state's rows and the token; the rows move up by one.  A
// thread reads every row of its channels before it writes one, so state_out may be state_in.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvParams p) {
  const int ncv = p.C / V;
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long b = id / ncv;
  if (b >= p.B) return;
  const int c = (int)(id % ncv) * V;
  float win[W][V], o[V];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_pos<T, V, W>(p, (int)b, j, c, win[j]);
  load_vec<T, V>(static_cast<const T*>(p.x) + (size_t)b * p.ldx + c, win[W - 1]);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float acc = p.bias != nullptr ? p.bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) acc = fmaf(p.weight[(size_t)(c + i) * W + j], win[j][i], acc);
    o[i] = p.silu ? acc * sigmoid_ex2(acc) : acc;
  }
  store_vec<T, V>(static_cast<T*>(p.y) + (size_t)b * p.C + c, o);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    store_vec<T, V>(static_cast<T*>(p.state_out) + ((size_t)b * (W - 1) + j) * p.C + c, win[j + 1]);
}

// T = 0: the final state is the first (and its gradient passes through).
__global__ void copy_bytes_kernel(size_t n, const unsigned char* src, unsigned char* dst) {
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) dst[i] = src != nullptr ? src[i] : 0;
}

template <typename T, int V, int W>
cudaError_t fwd_vw(ConvParams p, cudaStream_t st) {
  p.nseg = (p.T + kFwdStretch - 1) / kFwdStretch;
  const long long n = (long long)p.B * p.nseg * (p.C / V);
  conv_fwd_kernel<T, V, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t bwd_vw(ConvParams p, cudaStream_t st) {
  p.nseg = (p.T + kBwdStretch - 1) / kBwdStretch;
  const int nparts = conv_bwd_parts(p.B, p.T);
  const int ncg = (p.C / V + 31) / 32;
  conv_bwd_kernel<T, V, W><<<(unsigned)nparts * (unsigned)ncg, 32 * kBwdWarps, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const size_t n = (size_t)(W + 1) * p.C;
  conv_reduce_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(nparts, p.C, W, p.part,
                                                                                    p.gweight, p.gbias);
  return cudaGetLastError();
}

template <typename T, int V, int W>
cudaError_t step_vw(const ConvParams& p, cudaStream_t st) {
  const long long n = (long long)p.B * (p.C / V);
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

cudaError_t launch_conv(ConvPass pass, bool bf16, bool vec, const ConvParams& p, cudaStream_t st) {
  if (bf16) return vec ? run_v<__nv_bfloat16, 4>(pass, p, st) : run_v<__nv_bfloat16, 1>(pass, p, st);
  return vec ? run_v<float, 2>(pass, p, st) : run_v<float, 1>(pass, p, st);
}

cudaError_t launch_copy_bytes(size_t n, const void* src, void* dst, cudaStream_t st) {
  if (n == 0) return cudaSuccess;
  copy_bytes_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(n, static_cast<const unsigned char*>(src),
                                                                 static_cast<unsigned char*>(dst));
  return cudaGetLastError();
}

}  // namespace rwkv
