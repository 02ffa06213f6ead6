// Selective scan forward (sm_100a): a diagonal state per channel whose step size, input and output
// weights are data.  Per batch row, channel c and state n,
//   Δ_t = softplus(dt_t + dt_bias),   A = -exp(a_log),
//   h_t[n] = exp(Δ_t A[n]) h_{t-1}[n] + Δ_t x_t B_t[n],
//   p_t = Σ_n C_t[n] h_t[n] + d x_t,   y_t = p_t, or p_t z_t σ(z_t) with a gate z.
// B_t and C_t are shared by all channels of a token.
//
// What bounds it: one exponential per state and token, and the shared-memory pipe.  With N = 16 an
// element (b, t, c) moves 8 bytes in bf16 but needs 16 ex2, and the special-function unit does 16 a
// clock and SM: 0.15 ms at 4x4096x2560, where the bytes take 0.05.  The same work takes that pipe
// about 14 turns per warp and token of 4 states a lane (4 bytes a lane and turn), half again as long:
// with enough channels it is 85 % busy (8x4096x5120: 1.12 ms); at 4x4096x2560 (0.38 ms, 65 %) only eight
// to ten warps an SM share it and latency counts as much.
//
// Mapping.  A thread owns 4 states of one channel, the lanes of a warp are channels; a CTA owns 16
// or 32 channels of one batch row over one time segment, 32 tokens at a time:
//   1. the inputs of a tile are read in runs of channels per thread (16 bytes in bf16 with N = 16; off
//      the 16-byte grid one by one, side by side in a warp: 4x1024x2561 bf16 0.126 ms, 0.151 with runs of
//      single accesses, 0.096 for 2560 channels), a tile ahead, left as loaded in registers until the
//      tile is due; Δ and Δx go to shared memory, so softplus is done once per element and not once per
//      group of states, and B, C as fp32 rows;
//   2. each thread walks the 32 tokens, reading 4 of them ahead; Σ_n over its 4 states goes to
//      shared memory per group of states (folding a channel's states over lanes instead costs
//      three shuffles and nine selects and adds per 4 tokens, and measured 0.473 ms; two channels
//      a thread, to use each B and C twice, 0.49: too few warps; half of the CTA for loads and
//      outputs, half for the scan, 0.44: all at 4x4096x2560);
//   3. the tile's outputs add the groups' sums, d x and the gate and leave in the same runs.
//
// Few channels, long axis: time is cut into segments.  A first launch runs every segment but the
// last from a zero state and keeps the state it reaches and ΣΔ; the state entering segment s is
// then folded from these in order (the decay over a segment is exp(A ΣΔ)) by the CTA that needs
// it, in the second launch, which writes the outputs (1x8192x2048: 0.37 ms whole, 0.21 in 9 segments).
// Sums run in a fixed order: the same inputs give the same bits.
#include <algorithm>

#include "mixer.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kSN = 4;  // states per thread

// kOutputs writes outputs; kSummary the states and ΣΔ at the segments' ends, from zero; kReverse
// the same for the backward's recurrence G <- exp(Δ_t A) (G + C_t g_t) over reversed time, with
// g = gy silu(z): gy in the place of x, C of B, gh_out of h_in.
enum class Pass { kSummary, kOutputs, kReverse };

// Channels per CTA: small CTAs (two warps with N = 16) spread evenly over the SMs; 32 channels
// measured the same there (0.390 against 0.383 ms at 4x4096x2560).
constexpr int scan_channels(int N) { return N == 8 ? 32 : 16; }

// CH channels per CTA; thread tid owns states 4 (tid / CH) .. + 3 of channel tid mod CH.
template <int N, int CH_>
struct Shape {
  static constexpr int kCh = CH_;
  static constexpr int kGroups = N / kSN;                   // threads per channel
  static constexpr int kThreads = kCh * kGroups;
  static constexpr int kTile = 32;                          // tokens per tile
  static constexpr int kTokThreads = kThreads / kTile;      // threads per token in the tile's loads
  static constexpr int kRun = kCh / kTokThreads;            // elements per thread there
  static constexpr int kQuads = kTile * N / 4 / kThreads;   // groups of 4 states of B (and C) per thread there
  static_assert(kTokThreads * kRun == kCh && kQuads * kThreads * 4 == kTile * N, "a tile's loads cover it");
  static_assert(kRun % 2 == 0, "channels are worked on in pairs");
};

// 4 states' B and C of one token.  As fp32: kept in bf16 they would load in half the turns of the
// shared-memory pipe, but unpacking them costs more issue slots than that saves (4x4096x2560 bf16:
// 0.422 against 0.383 ms).
struct __align__(16) BC4 {
  float b[4], c[4];
};

// Rows of dx are padded so that the tile's stores (a run of channels per thread) fall on different
// banks, the groups' sums so that two groups in one warp do.
template <int N, typename S>
struct __align__(16) Smem {
  float2 dx[S::kTile][S::kCh + 2];                          // (Δ, Δ x)
  BC4 bc[S::kTile][S::kGroups];
  float y[S::kGroups][S::kTile * S::kCh + (S::kCh & 31)];   // Σ C h over each group of 4 states
};

// A thread's elements of a tile.  VEC: a run of channels of one token, in wide accesses.  Else rows or
// bases are off the 16-byte grid: one channel of every kGroups-th token, so that a warp's single
// accesses lie side by side.
template <typename S, bool VEC>
struct Place {
  int t, ch;  // the first element's token in the tile and channel in the CTA
  __device__ __forceinline__ Place() {
    const int tid = threadIdx.x;
    t = VEC ? tid / S::kTokThreads : tid / S::kCh;
    ch = VEC ? tid % S::kTokThreads * S::kRun : tid % S::kCh;
  }
  __device__ __forceinline__ int tok(int i) const { return VEC ? t : t + i * S::kGroups; }
  __device__ __forceinline__ int chan(int i) const { return VEC ? ch + i : ch; }
};

// Its elements of one array as loaded; those at or past token t1 or channel C are zero.
template <typename T, typename S, bool VEC>
struct Elems {
  Raw<T, VEC ? S::kRun : 1> r[VEC ? 1 : S::kRun];
  // src: the first element; left: tokens from there to the segment's end, nc: channels to the last
  __device__ __forceinline__ void load(const T* src, int64_t ld, int left, int nc) {
    if constexpr (VEC) {
      r[0].load(src, left > 0 ? nc : 0, true);
    } else {
#pragma unroll
      for (int i = 0; i < S::kRun; ++i) {
        r[i].zero();
        if (i * S::kGroups < left && nc > 0) r[i].load(src + (size_t)(i * S::kGroups) * ld);
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return VEC ? r[0][i] : r[VEC ? 0 : i][0]; }
};

// One tile's inputs in registers, as loaded.
template <typename T, typename S, bool VEC>
struct Tile {
  Elems<T, S, VEC> x, dt, z;
  Raw<T, 4> b[S::kQuads], c[S::kQuads];
};

// The tile at token ts: this thread's first element is token t of channel c0, nc channels to the last.
template <typename T, int N, typename S, Pass PASS, bool VEC>
__device__ __forceinline__ void load_tile(Tile<T, S, VEC>& R, const ScanParams& p, int bb, int ts, int t, int t1,
                                          int c0, int nc) {
  const int left = t1 - t;
  const size_t row = (size_t)bb * p.T + (left > 0 ? t : 0);
  R.x.load(static_cast<const T*>(p.x) + row * p.ldx + c0, p.ldx, left, nc);
  R.dt.load(static_cast<const T*>(p.dt) + row * p.lddt + c0, p.lddt, left, nc);
  if constexpr (PASS != Pass::kSummary)
    if (p.z != nullptr) R.z.load(static_cast<const T*>(p.z) + row * p.ldz + c0, p.ldz, left, nc);
#pragma unroll
  for (int k = 0; k < S::kQuads; ++k) {
    const int id = threadIdx.x + k * S::kThreads, tq = ts + id / (N / 4), s0 = id % (N / 4) * 4;
    const bool on = tq < t1;
    const size_t rq = (size_t)bb * p.T + (on ? tq : 0);
    R.b[k].load(static_cast<const T*>(p.b) + rq * p.ldb + s0, on ? 4 : 0, p.vec_bc);
    if constexpr (PASS == Pass::kOutputs) R.c[k].load(static_cast<const T*>(p.c) + rq * p.ldc + s0, on ? 4 : 0, p.vec_bc);
  }
}

// What the scan reads of 4 tokens from shared memory.
struct Quad {
  float2 dx[4], b[4][2], c[4][2];
  template <typename SM, bool OUT>
  __device__ __forceinline__ void load(const SM& sm, int tk, int ch, int g) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dx[k] = sm.dx[tk + k][ch];
      load_pairs<2>(sm.bc[tk + k][g].b, b[k]);
      if constexpr (OUT) load_pairs<2>(sm.bc[tk + k][g].c, c[k]);
    }
  }
};

template <typename T, int N, int CH_, Pass PASS, bool VEC>
__global__ void __launch_bounds__(Shape<N, CH_>::kThreads) scan_fwd_kernel(const __grid_constant__ ScanParams p) {
  using S = Shape<N, CH_>;
  using SM = Smem<N, S>;
  constexpr int CH = S::kCh, RUN = S::kRun, TL = S::kTile;
  constexpr bool OUT = PASS == Pass::kOutputs, REV = PASS == Pass::kReverse;
  extern __shared__ __align__(16) unsigned char raw[];
  SM& sm = *reinterpret_cast<SM*>(raw);
  const int tid = threadIdx.x;
  const int ct = (int)(blockIdx.x % (unsigned)p.ctiles);
  const unsigned rest = blockIdx.x / (unsigned)p.ctiles;
  const int nseg = OUT ? p.nseg : p.nseg - 1;
  // the last segment in the pass's own time has no segment behind it that would need its summary
  const int seg = (int)(rest % (unsigned)nseg) + (REV ? 1 : 0), bb = (int)(rest / (unsigned)nseg);
  const int t0 = seg * p.seg_len, t1 = segment_end(p.T, t0, p.seg_len);

  // the loads' view
  const Place<S, VEC> at;
  const int c0 = ct * CH + at.ch, nc = max(0, min(RUN, p.C - c0));
  Tile<T, S, VEC> R;
  const int first = REV ? t0 + (t1 - t0 - 1) / TL * TL : t0;  // the first tile worked on
  load_tile<T, N, S, PASS, VEC>(R, p, bb, first, first + at.t, t1, c0, nc);
  constexpr int NC = VEC ? RUN : 1;  // channels of a thread
  float bias[NC], dsk[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    bias[i] = p.dt_bias != nullptr && i < nc ? p.dt_bias[c0 + i] : 0.f;
    dsk[i] = OUT && p.d != nullptr && i < nc ? p.d[c0 + i] : 0.f;
  }

  // the scan's view: 4 states of one channel, in pairs
  const int ch = tid % CH, s0 = tid / CH * kSN;
  const int c = ct * CH + ch;
  const bool cact = c < p.C;
  const size_t hoff = ((size_t)bb * p.C + c) * N + s0;  // in a [B,C,N] state
  const size_t plane = (size_t)p.B * p.C * N;
  float a2f[kSN] = {0.f, 0.f, 0.f, 0.f};
  if (cact) load_rates<kSN>(p.a_log + (size_t)c * N + s0, a2f);
  float2 a2[2] = {make_float2(a2f[0], a2f[1]), make_float2(a2f[2], a2f[3])}, h[2] = {dup2(0.f), dup2(0.f)};
  if (cact) {
    if (OUT && seg > 0) {
      load_pairs<2>(p.seg_h + hoff, h);  // segment 0's summary starts from h_in
#pragma unroll 4
      for (int s = 1; s < seg; ++s) {
        float2 x[2];
        load_pairs<2>(p.seg_h + (size_t)s * plane + hoff, x);
        const float2 sd = dup2(p.seg_dt[((size_t)s * p.B + bb) * p.C + c]);
#pragma unroll
        for (int i = 0; i < 2; ++i) h[i] = fma2(decay2(sd, a2[i]), h[i], x[i]);
      }
    } else if (seg == (REV ? p.nseg - 1 : 0) && p.h_in != nullptr) {
      // with segments the first launch keeps a copy of h_in, which the second reads: h_out may be
      // the same array, and another CTA of the second launch writes it
      load_pairs<2>((OUT && p.nseg > 1 ? p.seg_h0 : p.h_in) + hoff, h);
      if (!OUT) store_pairs<2>(p.seg_h0 + hoff, h);
    }
  }
  float sumdt = 0.f;

  for (int ts = first; ts >= t0 && ts < t1; ts += REV ? -TL : TL) {
    const auto on = [&](int i) { return ts + at.tok(i) < t1 && (VEC ? i : 0) < nc; };
    float x[RUN], z[RUN];
#pragma unroll
    for (int i = 0; i < RUN; i += 2) {
      float2 e;
      const float2 dl = softplus2(make_float2(R.dt[i] + bias[VEC ? i : 0], R.dt[i + 1] + bias[VEC ? i + 1 : 0]), e);
      x[i] = R.x[i], x[i + 1] = R.x[i + 1];
      if constexpr (OUT) z[i] = R.z[i], z[i + 1] = R.z[i + 1];
      float2 in = make_float2(dl.x * x[i], dl.y * x[i + 1]);
      if constexpr (REV) {
        in = make_float2(x[i], x[i + 1]);
        if (p.z != nullptr) {
          const float za = R.z[i], zb = R.z[i + 1];
          in = make_float2(in.x * (za * sigmoid_ex2(za)), in.y * (zb * sigmoid_ex2(zb)));
        }
      }
      const float2 u = on(i) ? make_float2(dl.x, in.x) : dup2(0.f), v = on(i + 1) ? make_float2(dl.y, in.y) : dup2(0.f);
      if constexpr (VEC) {
        *reinterpret_cast<float4*>(&sm.dx[at.t][at.ch + i]) = make_float4(u.x, u.y, v.x, v.y);
      } else {
        sm.dx[at.tok(i)][at.ch] = u;
        sm.dx[at.tok(i + 1)][at.ch] = v;
      }
    }
#pragma unroll
    for (int k = 0; k < S::kQuads; ++k) {
      BC4& q = (&sm.bc[0][0])[tid + k * S::kThreads];
      *reinterpret_cast<float4*>(q.b) = make_float4(R.b[k][0], R.b[k][1], R.b[k][2], R.b[k][3]);
      if constexpr (OUT) *reinterpret_cast<float4*>(q.c) = make_float4(R.c[k][0], R.c[k][1], R.c[k][2], R.c[k][3]);
    }
    const int tn = REV ? ts - TL : ts + TL;
    if (tn >= t0 && tn < t1) load_tile<T, N, S, PASS, VEC>(R, p, bb, tn, tn + at.t, t1, c0, nc);
    __syncthreads();

#pragma unroll 1
    for (int hh = 0; hh < TL; hh += kScanCkLen) {
      const int hf = REV ? TL - kScanCkLen - hh : hh;
      if (ts + hf >= t1) continue;
      if constexpr (OUT) {
        if (p.ckpt != nullptr && cact)
          store_pairs<2>(p.ckpt + (size_t)((ts + hf) / kScanCkLen) * plane + hoff, h);
      }
      Quad q;
      q.template load<SM, OUT>(sm, hf + (REV ? kScanCkLen - 4 : 0), ch, s0 / kSN);
#pragma unroll
      for (int gg = 0; gg < kScanCkLen; gg += 4) {
        const int g = REV ? kScanCkLen - 4 - gg : gg;
        Quad nx = q;  // the next 4 tokens, on their way while these are worked on
        if (gg + 4 < kScanCkLen) nx.template load<SM, OUT>(sm, hf + (REV ? g - 4 : g + 4), ch, s0 / kSN);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int k = REV ? 3 - kk : kk;
          const float2 d2 = dup2(q.dx[k].x), in2 = dup2(q.dx[k].y);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 e = decay2(d2, a2[i]);
            h[i] = REV ? mul2(e, fma2(in2, q.b[k][i], h[i])) : fma2(e, h[i], mul2(in2, q.b[k][i]));
          }
          if constexpr (OUT) {
            const float2 acc = fma2(q.c[k][1], h[1], mul2(q.c[k][0], h[0]));
            sm.y[s0 / kSN][(hf + g + k) * CH + ch] = acc.x + acc.y;
          } else {
            sumdt += q.dx[k].x;
          }
        }
        q = nx;
      }
    }
    __syncthreads();

    if constexpr (OUT) {
      if (p.y != nullptr && nc > 0 && ts + at.t < t1) {
        float o[RUN];
#pragma unroll
        for (int i = 0; i < RUN; ++i) o[i] = dsk[VEC ? i : 0] * x[i];
#pragma unroll
        for (int g = 0; g < S::kGroups; ++g) {
          float v[RUN];
          if constexpr (VEC) {
            load_vec<float, RUN>(&sm.y[g][at.t * CH + at.ch], v);
          } else {
#pragma unroll
            for (int i = 0; i < RUN; ++i) v[i] = sm.y[g][at.tok(i) * CH + at.ch];
          }
#pragma unroll
          for (int i = 0; i < RUN; ++i) o[i] += v[i];
        }
        if (p.z != nullptr) {
#pragma unroll
          for (int i = 0; i < RUN; ++i) o[i] *= z[i] * sigmoid_ex2(z[i]);
        }
        T* y = static_cast<T*>(p.y) + ((size_t)bb * p.T + ts + at.t) * p.C + c0;
        if constexpr (VEC) {
          store_part<T, RUN>(y, nc, true, o);
        } else {
#pragma unroll
          for (int i = 0; i < RUN; ++i)
            if (on(i)) y[(size_t)(i * S::kGroups) * p.C] = IO<T>::from_f(o[i]);
        }
      }
    }
  }

  if (cact) {
    if constexpr (OUT) {
      if (seg == p.nseg - 1 && p.h_out != nullptr) store_pairs<2>(p.h_out + hoff, h);
    } else {
      store_pairs<2>(p.seg_h + (size_t)seg * plane + hoff, h);
      if (s0 == 0) p.seg_dt[((size_t)seg * p.B + bb) * p.C + c] = sumdt;
    }
  }
}

template <typename T, int N, int CH, Pass PASS, bool VEC>
cudaError_t launch_as(const ScanParams& p, cudaStream_t st) {
  constexpr int kThreads = Shape<N, CH>::kThreads, kSmem = (int)sizeof(Smem<N, Shape<N, CH>>);
  static unsigned mask = 0;
  const auto kernel = scan_fwd_kernel<T, N, CH, PASS, VEC>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kSmem, &mask);
  if (e != cudaSuccess) return e;
  const unsigned segs = (unsigned)(PASS == Pass::kOutputs ? p.nseg : p.nseg - 1);
  kernel<<<(unsigned)p.ctiles * (unsigned)p.B * segs, kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int N, int CH, Pass PASS>
cudaError_t launch_pass(const ScanParams& p, cudaStream_t st) {
  return p.vec ? launch_as<T, N, CH, PASS, true>(p, st) : launch_as<T, N, CH, PASS, false>(p, st);
}

template <typename T, int N>
cudaError_t run_n(ScanParams p, bool reverse, cudaStream_t st) {
  constexpr int CH = scan_channels(N);
  p.ctiles = (p.C + CH - 1) / CH;
  if (reverse) return launch_pass<T, N, CH, Pass::kReverse>(p, st);
  if (p.nseg > 1) {
    const cudaError_t e = launch_pass<T, N, CH, Pass::kSummary>(p, st);
    if (e != cudaSuccess) return e;
  }
  return launch_pass<T, N, CH, Pass::kOutputs>(p, st);
}

template <typename T>
cudaError_t run_t(const ScanParams& p, bool reverse, cudaStream_t st) {
  switch (p.N) {
    case 8: return run_n<T, 8>(p, reverse, st);
    case 16: return run_n<T, 16>(p, reverse, st);
    case 32: return run_n<T, 32>(p, reverse, st);
    case 64: return run_n<T, 64>(p, reverse, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

int scan_fwd_channels(int N) { return scan_channels(N); }
int scan_tile_tokens() { return 32; }

cudaError_t launch_scan_fwd(bool bf16, const ScanParams& p, cudaStream_t st) {
  return bf16 ? run_t<__nv_bfloat16>(p, false, st) : run_t<float>(p, false, st);
}

cudaError_t launch_scan_reverse(bool bf16, const ScanParams& p, cudaStream_t st) {
  return bf16 ? run_t<__nv_bfloat16>(p, true, st) : run_t<float>(p, true, st);
}

}  // namespace rwkv
