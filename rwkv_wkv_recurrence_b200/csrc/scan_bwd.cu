// Selective scan backward (sm_100a): the chain rule through the recurrence of scan_fwd.cu.  With
// g_t = gy_t z_t σ(z_t) (or gy_t), e_t = exp(Δ_t A), and G_t the gradient of h_t,
//   G_t = C_t g_t + e_{t+1} G_{t+1}         (from gh_out behind the last token),
//   gC_t[n] = Σ_c g_t h_t[n],   gB_t[n] = Σ_c G_t[n] Δ_t x_t,
//   s1_t = Σ_n G_t B_t,   q_t = G_t e_t h_{t-1},   s2_t = Σ_n q_t A,
//   gx_t = Δ_t s1_t + d g_t,   gdt_t = σ(dt_t + dt_bias) (x_t s1_t + s2_t),   gdt_bias = Σ gdt,
//   ga_log = A Σ q_t Δ_t,   gd = Σ g_t x_t,   gz_t = gy_t p_t silu'(z_t),   gh_in = e_0 G_0.
//
// The states come from the forward's checkpoints, one every 16 tokens; a CTA owns 1024/N channels and
// walks its time segment backwards, a 16-token tile at a time: the states are run forward from the
// checkpoint and kept every 4 tokens; then, from the last 4 tokens to the first, the 4 states and
// decays are formed again in registers and walked backwards with G.
//
// What bounds it: latency and the shared-memory pipe together.  At 4x4096x2560, N = 16, bf16 the main
// kernel takes 0.83 ms; 12 warps an SM (168 registers and 8 to 52 bytes spilled a
// thread, 72 KB a CTA; 94 to 109 KB, and so 8 warps, with N = 8 and 64) issue in 52 % of the cycles, the
// shared-memory pipe is busy 64 %, the special-function unit 37 %.  16 warps an SM (128 registers,
// the decays formed twice) measured 0.85 ms, 8 with 255 registers 0.93, unpacked arithmetic 0.85
// (a third more instructions, 67 % of the cycles).  Every lane needs B_t[n] and C_t[n] of its states,
// and a load costs the shared-memory pipe 4 bytes a lane and turn even where all lanes read the same
// words, so a thread owns 4 states of TWO channels and each loaded word serves both; N/4 neighbouring
// lanes own a channel pair.  (One channel per thread, with selects in its exchanges and the loads
// waited for where they were issued, took 3.9 ms in all.)
//   - Sums over a pair's states (p, s1, s2): half of a pair's lanes hold its two channels in the
//     other order, so the first exchange gives away one channel and keeps the other without selects.
//   - Sums over channels (gB, gC: all channels share B and C): the lanes hold their 4 states in an
//     order XORed with their place in the warp (B and C lie in shared memory in each of the 4
//     orders), so that the exchanges need no selects either; warps meet in shared memory, CTAs in the
//     workspace, added by a last kernel.  No atomics: the same inputs give the same bits.
//   - x, dt, z, gy and the checkpoint arrive by cp.async, a tile ahead, each thread reading back what
//     it fetched; stores to shared memory wait until four tokens are done, so that no load of the next
//     token queues behind one.
//
// Time is cut into segments so that the CTAs fill the SMs evenly; the carry G that enters a segment
// from behind is folded from the later segments' own (each from zero, by a first launch of
// scan_fwd.cu's kernel in reverse) and their ΣΔ.
#include "mixer.h"
#include "scan_common.cuh"

namespace rwkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = kScanCkLen;  // tokens per tile
constexpr int kSub = 4;            // tokens whose states are in registers at once
constexpr int kSN = 4;             // states per thread and channel
constexpr float kLn2 = 0.693147180559945309f;

template <int N>
struct Shape {
  static constexpr int kLanes = N / kSN;                // lanes per channel pair
  static constexpr int kPairs = 32 / kLanes;            // channel pairs per warp
  static constexpr int kCh = 2 * kPairs * kWarps;       // channels per CTA
  static constexpr int kTokThreads = kThreads / kTile;  // threads per token in the tile's loads
  static constexpr int kRun = kCh / kTokThreads;        // channels per thread there
  static constexpr int kQuads = 2 * kTile * N / 4;      // groups of 4 states of B, then of C, in a tile
  // column of channel ch in the (Δ, Δx, g, x) rows: the runs' stores fall on different banks
  __device__ __forceinline__ static int col(int ch) {
    constexpr int M = kRun < 8 ? kRun : 8;
    return ch ^ ((ch / kRun) & (M - 1));
  }
};

// A thread's elements of a tile, as in the forward.  VEC: a run of channels of one token, in wide
// accesses.  Else one channel of every kStep-th token (4x1024x2561, N = 8, bf16: the backward in 0.36 ms,
// 0.58 with runs of single accesses, 0.26 for 2560 channels).
template <typename S, bool VEC>
struct Place {
  static constexpr int kStep = kThreads / S::kCh;
  int t, ch;  // the first element's token in the tile and channel in the CTA
  __device__ __forceinline__ Place() {
    const int tid = threadIdx.x;
    t = VEC ? tid / S::kTokThreads : tid / S::kCh;
    ch = VEC ? tid % S::kTokThreads * S::kRun : tid % S::kCh;
  }
  __device__ __forceinline__ int tok(int i) const { return VEC ? t : t + i * kStep; }
  __device__ __forceinline__ int chan(int i) const { return VEC ? ch + i : ch; }
};

// Elements that a thread fetches into shared memory for itself.  VEC: a run in pieces of up to 16 bytes,
// piece k of thread tid at (k kThreads + tid) pieces.
template <typename T, typename S, bool VEC>
struct Stage {
  static constexpr int RUN = S::kRun;
  using Got = Raw<T, RUN>;
  static constexpr int kBytes = RUN * (int)sizeof(T);
  static constexpr int kPiece = kBytes < 16 ? kBytes : 16;
  static constexpr int kElems = kPiece / (int)sizeof(T);
  static constexpr int kPieces = kBytes / kPiece;
  unsigned char raw[kPieces * kThreads * kPiece];

  // src: the first element; left: tokens from there to the segment's end, nc: channels to the last.
  __device__ __forceinline__ void fetch(const T* src, int64_t, int left, int nc, bool) {
    const int n = left > 0 ? nc : 0;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      T* dst = reinterpret_cast<T*>(raw + (k * kThreads + threadIdx.x) * kPiece);
      if (n >= RUN) {
        const uint32_t d = smem_u32(dst);
        if constexpr (kPiece == 16)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src + k * kElems) : "memory");
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src + k * kElems), "n"(kPiece)
                       : "memory");
      } else {
#pragma unroll
        for (int e = 0; e < kElems; ++e)
          dst[e] = k * kElems + e < n ? src[k * kElems + e] : IO<T>::from_f(0.f);
      }
    }
  }
  // Back into registers, as loaded.
  __device__ __forceinline__ void read(Got& r, const T*, int64_t) const {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      Raw<T, kElems> q;
      q.load(reinterpret_cast<const T*>(raw + (k * kThreads + threadIdx.x) * kPiece));
#pragma unroll
      for (int i = 0; i < kPiece / 4; ++i) r.w[k * (kPiece / 4) + i] = q.w[i];
    }
  }
};

// Single elements, each as the aligned 32-bit word that holds it (an asynchronous copy takes 4 bytes or
// more).  The word's other half is a neighbour in memory: where there may be none (not `inner`: the
// array's first and last token) the element is loaded by itself.
template <typename T, typename S>
struct Stage<T, S, false> {
  static constexpr int RUN = S::kRun, kStep = Place<S, false>::kStep;
  using Got = Raw<float, RUN>;
  uint32_t word[RUN][kThreads];

  __device__ __forceinline__ static bool upper(const T* q) {
    return sizeof(T) == 2 && (reinterpret_cast<uintptr_t>(q) & 2) != 0;
  }
  __device__ __forceinline__ void fetch(const T* src, int64_t ld, int left, int nc, bool inner) {
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      uint32_t* dst = &word[i][threadIdx.x];
      const T* q = src + (size_t)(i * kStep) * ld;
      if (i * kStep >= left || nc <= 0) {
        *dst = 0u;
      } else if (sizeof(T) == 4 || inner) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)),
                     "l"(reinterpret_cast<uintptr_t>(q) & ~(uintptr_t)3)
                     : "memory");
      } else {
        Raw<T, 1> r;
        r.load(q);
        *dst = upper(q) ? r.w[0] << 16 : r.w[0];
      }
    }
  }
  __device__ __forceinline__ void read(Got& r, const T* src, int64_t ld) const {
#pragma unroll
    for (int i = 0; i < RUN; ++i) {
      const uint32_t w = word[i][threadIdx.x];
      if constexpr (sizeof(T) == 4)
        r.w[i] = w;
      else
        r.w[i] = upper(src + (size_t)(i * kStep) * ld) ? w & 0xFFFF0000u : w << 16;
    }
  }
};
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <typename T, int N, bool VEC>
struct __align__(16) Smem {
  using S = Shape<N>;
  float4 dxg[kTile][S::kCh];              // (Δ, Δ x, g, x), then (gx, gdt, gz, -); columns permuted
  float bc[2][kTile][4 * N + 16];         // B and C: copy p (at p N) holds state 4 s + i at 4 s + (i ^ p)
  float red[kWarps][kTile][2 * N];        // per warp: gC, gB of a token
  float bias[S::kCh];                     // dt_bias
  float2 sg[kTile][S::kCh];               // (σ(dt + bias), gy silu'(z)), columns permuted
  // states before tokens 0, 4, 8, 12, each thread's own; then the next tile's checkpoint, except in fp32
  // and in single accesses, where with N = 16 its 4 KB would cost the third CTA an SM: there it waits for
  // the first of these to be free
  static constexpr bool kEarly = sizeof(T) == 2 && VEC;
  float4 snap[kTile / kSub + (kEarly ? 1 : 0)][2][kThreads];
  Stage<T, S, VEC> x, dt, z, gy;
};

// v[i ^ p] of 4 states held as two pairs, p the lane's order.
__device__ __forceinline__ void xor_order(float2 (&v)[2], int p) {
  if (p & 2) {
    const float2 t = v[0];
    v[0] = v[1], v[1] = t;
  }
  if (p & 1) {
    v[0] = make_float2(v[0].y, v[0].x);
    v[1] = make_float2(v[1].y, v[1].x);
  }
}

template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) scan_bwd_kernel(const __grid_constant__ ScanBwdParams p) {
  using S = Shape<N>;
  constexpr int L = S::kLanes, CP = S::kPairs, CH = S::kCh, RUN = S::kRun;
  extern __shared__ __align__(16) unsigned char raw[];
  using SM = Smem<T, N, VEC>;
  SM& sm = *reinterpret_cast<SM*>(raw);
  const ScanParams& f = p.f;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ct = (int)(blockIdx.x % (unsigned)f.ctiles);
  const unsigned rest = blockIdx.x / (unsigned)f.ctiles;
  const int seg = (int)(rest % (unsigned)f.nseg), bb = (int)(rest / (unsigned)f.nseg);
  const int t0 = seg * f.seg_len, t1 = segment_end(f.T, t0, f.seg_len);

  // the scan's view: 4 states, in the order i ^ ord, of channels ch[0] and ch[1]
  const int sub = lane % L, cl = lane / L;
  const int ord = CP >= 4 ? cl & 3 : (cl & 1) * 2;
  const int swap = sub / (L / 2);  // the upper half of a pair's lanes holds its channels swapped
  const int ch[2] = {(warp * CP + cl) * 2 + swap, (warp * CP + cl) * 2 + 1 - swap};
  const int col[2] = {S::col(ch[0]), S::col(ch[1])};
  const size_t plane = (size_t)f.B * f.C * N;
  size_t hoff[2];
  bool cact[2];
  float2 a2[2][2], gh[2][2], ga[2][2];  // [channel][pair of states]
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int c = ct * CH + ch[j];
    cact[j] = c < f.C;
    hoff[j] = ((size_t)bb * f.C + (cact[j] ? c : 0)) * N + sub * kSN;
    float r[kSN] = {0.f, 0.f, 0.f, 0.f};
    if (cact[j]) load_rates<kSN>(f.a_log + (size_t)c * N + sub * kSN, r);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      a2[j][q] = make_float2(r[2 * q], r[2 * q + 1]);
      gh[j][q] = ga[j][q] = dup2(0.f);
    }
    if (cact[j]) {
      if (seg < f.nseg - 1) {  // the last segment's own gradient starts from gh_out
        load_pairs<2>(p.seg_g + (size_t)(f.nseg - 1) * plane + hoff[j], gh[j]);
#pragma unroll 4
        for (int s = f.nseg - 2; s > seg; --s) {
          float2 x[2];
          load_pairs<2>(p.seg_g + (size_t)s * plane + hoff[j], x);
          const float2 sd = dup2(p.seg_dt[((size_t)s * f.B + bb) * f.C + c]);
#pragma unroll
          for (int q = 0; q < 2; ++q) gh[j][q] = fma2(decay2(sd, a2[j][q]), gh[j][q], x[q]);
        }
      } else if (p.gh_out != nullptr) {
        // a copy when segmented: gh_in may be the same array, and another CTA writes it
        load_pairs<2>((f.nseg > 1 ? p.seg_g0 : p.gh_out) + hoff[j], gh[j]);
      }
    }
    xor_order(a2[j], ord);
    xor_order(gh[j], ord);
  }

  const float dsk = f.d != nullptr && cact[0] ? f.d[ct * CH + ch[0]] : 0.f;

  // the loads' view
  const Place<S, VEC> at;
  const int c0 = ct * CH + at.ch, nc = max(0, min(RUN, f.C - c0));
  float gd = 0.f, gbias = 0.f;  // of channel ch[0], over the tokens whose sums this lane ends up with

  for (int i = tid; i < CH; i += kThreads)
    sm.bias[i] = f.dt_bias != nullptr && ct * CH + i < f.C ? f.dt_bias[ct * CH + i] : 0.f;
  __syncthreads();

  constexpr int QT = (S::kQuads + kThreads - 1) / kThreads;
  Raw<T, 4> bc[QT];
  const auto src = [&](const void* a, int64_t ld, int ts) {  // this thread's first element of a tile
    return static_cast<const T*>(a) + ((size_t)bb * f.T + (ts + at.t)) * ld + c0;
  };
  const auto fetch = [&](int ts) {  // a tile's inputs, on their way
    const int left = t1 - ts - at.t;  // none left: zeros, nothing read
    const bool inner = (bb > 0 || ts > 0) && (bb < f.B - 1 || ts + kTile < f.T);
    sm.x.fetch(src(f.x, f.ldx, ts), f.ldx, left, nc, inner);
    sm.dt.fetch(src(f.dt, f.lddt, ts), f.lddt, left, nc, inner);
    sm.gy.fetch(src(p.gy, f.C, ts), f.C, left, nc, inner);
    if (f.z != nullptr) sm.z.fetch(src(f.z, f.ldz, ts), f.ldz, left, nc, inner);
    cp_async_commit();
#pragma unroll
    for (int k = 0; k < QT; ++k) {
      const int id = tid + k * kThreads;
      if (S::kQuads % kThreads != 0 && id >= S::kQuads) continue;
      const bool is_c = id >= S::kQuads / 2;
      const int qi = is_c ? id - S::kQuads / 2 : id, tk = ts + qi / (N / 4), s0 = qi % (N / 4) * 4;
      const bool on = tk < t1;
      const size_t rq = (size_t)bb * f.T + (on ? tk : 0);
      bc[k].load(static_cast<const T*>(is_c ? f.c : f.b) + rq * (is_c ? f.ldc : f.ldb) + s0, on ? 4 : 0, f.vec_bc);
    }
  };
  constexpr bool kEarly = SM::kEarly;
  constexpr int kCk = kEarly ? kTile / kSub : 0;
  const auto fetch_state = [&](int ts) {  // the states before token ts
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float4* dst = &sm.snap[kCk][j][tid];
      if (cact[j])
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)),
                     "l"(f.ckpt + (size_t)(ts / kScanCkLen) * plane + hoff[j])
                     : "memory");
      else
        *dst = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    cp_async_commit();
  };
  int ts = t0 + (t1 - t0 - 1) / kTile * kTile;
  fetch(ts);
  fetch_state(ts);

  for (; ts >= t0; ts -= kTile) {
    const auto on = [&](int i) { return ts + at.tok(i) < t1 && (VEC ? i : 0) < nc; };
    cp_async_wait_all();
    {
      typename decltype(sm.x)::Got rx, rdt, rg, rz;
      sm.x.read(rx, src(f.x, f.ldx, ts), f.ldx);
      sm.dt.read(rdt, src(f.dt, f.lddt, ts), f.lddt);
      sm.gy.read(rg, src(p.gy, f.C, ts), f.C);
      if (f.z != nullptr) sm.z.read(rz, src(f.z, f.ldz, ts), f.ldz);
#pragma unroll
      for (int i = 0; i < RUN; i += 2) {
        const int k0 = at.tok(i), k1 = at.tok(i + 1), w0 = S::col(at.chan(i)), w1 = S::col(at.chan(i + 1));
        float2 g = rg.pair(i / 2), e;
        const float2 x = rx.pair(i / 2);
        const float2 v = add2(rdt.pair(i / 2), make_float2(sm.bias[at.chan(i)], sm.bias[at.chan(i + 1)]));
        float2 dl = softplus2(v, e);
        const float2 d1 = add2(e, dup2(1.f)), r1 = make_float2(rcp_approx(d1.x), rcp_approx(d1.y)), er = mul2(e, r1);
        const float2 sig = make_float2(v.x >= 0.f ? r1.x : er.x, v.y >= 0.f ? r1.y : er.y);
        float2 gpre = dup2(0.f);  // gy silu'(z) = gy (s + z s (1 - s))
        if (f.z != nullptr) {
          const float2 z = rz.pair(i / 2), s = sigmoid2(z), zs = mul2(z, s);
          gpre = mul2(g, fma2(zs, fma2(s, dup2(-1.f), dup2(1.f)), s));
          g = mul2(g, zs);
        }
        // behind the end and past the last channel x = gy = 0 were fetched; Δ = 0 keeps the state
        if (!on(i)) dl.x = 0.f;
        if (!on(i + 1)) dl.y = 0.f;
        const float2 dx = mul2(dl, x);
        sm.dxg[k0][w0] = make_float4(dl.x, dx.x, g.x, x.x);
        sm.dxg[k1][w1] = make_float4(dl.y, dx.y, g.y, x.y);
        sm.sg[k0][w0] = make_float2(sig.x, gpre.x);
        sm.sg[k1][w1] = make_float2(sig.y, gpre.y);
      }
    }
#pragma unroll
    for (int k = 0; k < QT; ++k) {
      const int id = tid + k * kThreads;
      if (S::kQuads % kThreads != 0 && id >= S::kQuads) continue;
      const int which = id >= S::kQuads / 2, qi = which ? id - S::kQuads / 2 : id;
      float* dst = &sm.bc[which][qi / (N / 4)][qi % (N / 4) * 4];
      const float a = bc[k][0], b = bc[k][1], c = bc[k][2], d = bc[k][3];
      *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
      *reinterpret_cast<float4*>(dst + N) = make_float4(b, a, d, c);
      *reinterpret_cast<float4*>(dst + 2 * N) = make_float4(c, d, a, b);
      *reinterpret_cast<float4*>(dst + 3 * N) = make_float4(d, c, b, a);
    }
    float2 h[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 v = sm.snap[kCk][j][tid];
      h[j][0] = make_float2(v.x, v.y), h[j][1] = make_float2(v.z, v.w);
      xor_order(h[j], ord);
    }
    if (ts > t0) {
      fetch(ts - kTile);
      if (kEarly) fetch_state(ts - kTile);
    }
    __syncthreads();

    // the states every 4 tokens
#pragma unroll 4
    for (int k = 0; k < kTile; ++k) {
      if (k % kSub == 0) {  // in the lane's order (the first, as fetched, too)
#pragma unroll
        for (int j = 0; j < 2; ++j) store_pairs<2>(reinterpret_cast<float*>(&sm.snap[k / kSub][j][tid]), h[j]);
        if (k == kTile - kSub) break;
      }
      float2 bv[2];
      load_pairs<2>(&sm.bc[0][k][ord * N + sub * kSN], bv);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 d = *reinterpret_cast<const float2*>(&sm.dxg[k][col[j]]);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          h[j][q] = fma2(decay2(dup2(d.x), a2[j][q]), h[j][q], mul2(dup2(d.y), bv[q]));
      }
    }

#pragma unroll 1
    for (int sb = kTile / kSub - 1; sb >= 0; --sb) {
      const int k0 = sb * kSub;
      float2 hh[kSub + 1][2][2], e[kSub][2][2];  // states before each token and after the last; decays
#pragma unroll
      for (int j = 0; j < 2; ++j) load_pairs<2>(reinterpret_cast<const float*>(&sm.snap[sb][j][tid]), hh[0][j]);
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        float2 bv[2];
        load_pairs<2>(&sm.bc[0][k0 + k][ord * N + sub * kSN], bv);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 d = *reinterpret_cast<const float2*>(&sm.dxg[k0 + k][col[j]]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            e[k][j][q] = decay2(dup2(d.x), a2[j][q]);
            hh[k + 1][j][q] = fma2(e[k][j][q], hh[k][j][q], mul2(dup2(d.y), bv[q]));
          }
        }
      }
      float sp[kSub], s1[kSub], s2[kSub], rv[kSub][CP >= 8 ? 1 : CP == 4 ? 2 : 4];
#pragma unroll
      for (int k = kSub - 1; k >= 0; --k) {
        float2 bv[2], cv[2], vc[2], vb[2];  // vc, vb: this thread's part of gC and gB
        load_pairs<2>(&sm.bc[0][k0 + k][ord * N + sub * kSN], bv);
        load_pairs<2>(&sm.bc[1][k0 + k][ord * N + sub * kSN], cv);
        float tp[2], t1s[2], t2[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 d = sm.dxg[k0 + k][col[j]];
          const float2 dl = dup2(d.x), dx = dup2(d.y), g = dup2(d.z);
          float2 ap, a1, aq;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 ht = hh[k + 1][j][q];
            gh[j][q] = fma2(cv[q], g, gh[j][q]);
            ap = q == 0 ? mul2(cv[q], ht) : fma2(cv[q], ht, ap);
            a1 = q == 0 ? mul2(gh[j][q], bv[q]) : fma2(gh[j][q], bv[q], a1);
            vc[q] = j == 0 ? mul2(g, ht) : fma2(g, ht, vc[q]);
            vb[q] = j == 0 ? mul2(dx, gh[j][q]) : fma2(dx, gh[j][q], vb[q]);
            gh[j][q] = mul2(gh[j][q], e[k][j][q]);
            const float2 qq = mul2(gh[j][q], hh[k][j][q]);
            aq = q == 0 ? mul2(qq, a2[j][q]) : fma2(qq, a2[j][q], aq);
            ga[j][q] = fma2(qq, dl, ga[j][q]);
          }
          tp[j] = ap.x + ap.y, t1s[j] = a1.x + a1.y, t2[j] = aq.x + aq.y;
        }
        // over a pair's states: keep the first channel held, give the other
        sp[k] = tp[0] + __shfl_xor_sync(0xffffffffu, tp[1], L / 2);
        s1[k] = t1s[0] + __shfl_xor_sync(0xffffffffu, t1s[1], L / 2);
        s2[k] = t2[0] + __shfl_xor_sync(0xffffffffu, t2[1], L / 2);
        // over the warp's channels
        constexpr int B1 = CP >= 4 ? 2 * L : L;  // the lane bit behind ord's 2
        vc[0].x += __shfl_xor_sync(0xffffffffu, vc[1].x, B1);
        vc[0].y += __shfl_xor_sync(0xffffffffu, vc[1].y, B1);
        vb[0].x += __shfl_xor_sync(0xffffffffu, vb[1].x, B1);
        vb[0].y += __shfl_xor_sync(0xffffffffu, vb[1].y, B1);
        if constexpr (CP >= 4) {
          vc[0].x += __shfl_xor_sync(0xffffffffu, vc[0].y, L);
          vb[0].x += __shfl_xor_sync(0xffffffffu, vb[0].y, L);
          if constexpr (CP >= 8) {
            const bool up = (cl & 4) != 0;
            float v = up ? vb[0].x : vc[0].x;
            v += __shfl_xor_sync(0xffffffffu, up ? vc[0].x : vb[0].x, 4 * L);
            if constexpr (CP >= 16) v += __shfl_xor_sync(0xffffffffu, v, 8 * L);
            rv[k][0] = v;
          } else {
            rv[k][0] = vc[0].x, rv[k][1] = vb[0].x;
          }
        } else {
          rv[k][0] = vc[0].x, rv[k][1] = vb[0].x;
          rv[k][2] = vc[0].y, rv[k][3] = vb[0].y;
        }
      }
      // stored behind all four tokens: no load above has to wait for a store to shared memory
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        float* red = sm.red[warp][k0 + k] + sub * kSN + ord;
        if constexpr (CP >= 8) {
          if (CP == 8 || cl < 8) red[(cl & 4) != 0 ? N : 0] = rv[k][0];
        } else {
          red[0] = rv[k][0], red[N] = rv[k][1];
          if constexpr (CP == 2) red[1] = rv[k][2], red[N + 1] = rv[k][3];
        }
      }
      constexpr int HL = L / 2, M = HL < kSub ? HL : kSub;  // lanes that hold one channel; with different tokens
      const int hs = sub % HL;
      fold_lanes<kSub, HL>(sp, hs);
      fold_lanes<kSub, HL>(s1, hs);
      fold_lanes<kSub, HL>(s2, hs);
      __syncwarp();  // a warp alone reads its channels' columns, and has read these tokens'
      if (hs < M) {
#pragma unroll
        for (int k = 0; k < kSub / M; ++k) {
          const int tk = k0 + hs * (kSub / M) + k;
          const float4 v = sm.dxg[tk][col[0]];
          const float2 sg = sm.sg[tk][col[0]];
          const float gdt = sg.x * fmaf(v.w, s1[k], s2[k] * kLn2);
          sm.dxg[tk][col[0]] = make_float4(fmaf(v.x, s1[k], dsk * v.z), gdt, sg.y * fmaf(dsk, v.w, sp[k]), 0.f);
          gd = fmaf(v.z, v.w, gd);
          if (ts + tk < t1) gbias += gdt;  // a token that is not there has decays of 1 and a sum s2
        }
      }
    }
    if (!kEarly && ts > t0) fetch_state(ts - kTile);
    __syncthreads();

    if (ts + at.t < t1 && nc > 0) {
      const size_t off = ((size_t)bb * f.T + ts + at.t) * f.C + c0;
      if constexpr (VEC) {
        float ox[RUN], odt[RUN], oz[RUN];
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          const float4 d = sm.dxg[at.t][S::col(at.ch + i)];
          ox[i] = d.x, odt[i] = d.y, oz[i] = d.z;
        }
        store_part<T, RUN>(static_cast<T*>(p.gx) + off, nc, true, ox);
        store_part<T, RUN>(static_cast<T*>(p.gdt) + off, nc, true, odt);
        if (p.gz != nullptr) store_part<T, RUN>(static_cast<T*>(p.gz) + off, nc, true, oz);
      } else {
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
          if (!on(i)) continue;
          const float4 d = sm.dxg[at.tok(i)][S::col(at.ch)];
          const size_t o = off + (size_t)(i * Place<S, VEC>::kStep) * f.C;
          static_cast<T*>(p.gx)[o] = IO<T>::from_f(d.x);
          static_cast<T*>(p.gdt)[o] = IO<T>::from_f(d.y);
          if (p.gz != nullptr) static_cast<T*>(p.gz)[o] = IO<T>::from_f(d.z);
        }
      }
    }
    float* part = p.part_bc + (((size_t)ct * f.B + bb) * f.T + ts) * (2 * N);
#pragma unroll
    for (int i = tid; i < kTile * 2 * N; i += kThreads) {
      const int tk = i / (2 * N), n = i % (2 * N);
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sm.red[w][tk][n];
      if (ts + tk < t1) part[i] = s;
    }
    // no barrier: the next tile's stores before its own barrier go only where this thread alone
    // still reads (its elements of dxg, its stages) or nobody does (bc)
  }

  const size_t prow = (size_t)bb * f.nseg + seg;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (!cact[j]) continue;
    xor_order(ga[j], ord);
    xor_order(gh[j], ord);
    store_pairs<2>(p.part_a + (prow * f.C + ct * CH + ch[j]) * N + sub * kSN, ga[j]);
    if (seg == 0 && p.gh_in != nullptr) store_pairs<2>(p.gh_in + hoff[j], gh[j]);
  }
  // gd and gdt_bias: over the lanes that hold a channel's tokens
#pragma unroll
  for (int o = L / 4; o > 0; o >>= 1) {
    gd += __shfl_xor_sync(0xffffffffu, gd, o);
    gbias += __shfl_xor_sync(0xffffffffu, gbias, o);
  }
  if (sub % (L / 2) == 0 && cact[0]) {
    p.part_v[(prow * 2 + 0) * f.C + ct * CH + ch[0]] = gd;
    p.part_v[(prow * 2 + 1) * f.C + ct * CH + ch[0]] = gbias;
  }
}

// n floats `stride` apart, added in order, 8 loads at a time.
template <typename S>
__device__ __forceinline__ S sum_parts(const float* __restrict__ p, int n, size_t stride) {
  S s = 0;
  int k = 0;
  for (; k + 8 <= n; k += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[(size_t)(k + i) * stride];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (S)v[i];
  }
  for (; k < n; ++k) s += (S)p[(size_t)k * stride];
  return s;
}

// What the parts add up to, in one launch.  The first `vblocks` blocks: ga_log [C,N], then gd [C] and
// gdt_bias [C], the parts of the batch rows and segments in order.  The rest: gb, gc, the channel tiles'
// parts in order, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_sum_kernel(const __grid_constant__ ScanBwdParams p, unsigned vblocks) {
  const int N = p.f.N, C = p.f.C;
  if (blockIdx.x >= vblocks) {
    const size_t i = (size_t)(blockIdx.x - vblocks) * 256 + threadIdx.x, n = (size_t)p.f.B * p.f.T * 2 * N;
    if (i >= n) return;  // over [B,T][2][N]
    const float s = sum_parts<float>(p.part_bc + i, p.f.ctiles, n);
    const size_t row = i / (2 * N);
    const int j = (int)(i % (2 * N));
    static_cast<T*>(j < N ? p.gc : p.gb)[row * N + j % N] = IO<T>::from_f(s);
  } else {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, na = (size_t)C * N;
    const int nparts = p.f.B * p.f.nseg;
    if (i < na) {
      p.ga_log[i] = (float)(sum_parts<double>(p.part_a + i, nparts, na) * -(double)expf(p.f.a_log[i]));
    } else if (i < na + 2 * (size_t)C) {
      const size_t j = i - na;
      float* dst = j < (size_t)C ? p.gd : p.gdt_bias;
      if (dst != nullptr) dst[j % C] = (float)sum_parts<double>(p.part_v + j, nparts, 2 * (size_t)C);
    }
  }
}

template <typename T, int N, bool VEC>
cudaError_t launch_main(const ScanBwdParams& p, cudaStream_t st) {
  static unsigned mask = 0;
  constexpr int kSmem = (int)sizeof(Smem<T, N, VEC>);
  const auto kernel = scan_bwd_kernel<T, N, VEC>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kSmem, &mask);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)p.f.ctiles * (unsigned)p.f.B * (unsigned)p.f.nseg, kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int N>
cudaError_t bwd_n(ScanBwdParams p, cudaStream_t st) {
  p.f.ctiles = (p.f.C + Shape<N>::kCh - 1) / Shape<N>::kCh;
  cudaError_t e;
  if (p.f.nseg > 1) {
    ScanParams r = p.f;
    r.x = p.gy;
    r.ldx = p.f.C;
    r.b = p.f.c;
    r.ldb = p.f.ldc;
    r.h_in = p.gh_out;
    r.seg_h = p.seg_g;
    r.seg_dt = p.seg_dt;
    r.seg_h0 = p.seg_g0;
    if ((e = launch_scan_reverse(sizeof(T) == 2, r, st)) != cudaSuccess) return e;
  }
  if ((e = p.f.vec ? launch_main<T, N, true>(p, st) : launch_main<T, N, false>(p, st)) != cudaSuccess) return e;
  const size_t n = (size_t)p.f.B * p.f.T * 2 * N, m = (size_t)p.f.C * N + 2 * (size_t)p.f.C;
  const unsigned vblocks = (unsigned)((m + 255) / 256);
  scan_bwd_sum_kernel<T><<<vblocks + (unsigned)((n + 255) / 256), 256, 0, st>>>(p, vblocks);
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

int scan_bwd_channels(int N) { return 2 * kThreads * kSN / N; }

cudaError_t launch_scan_bwd(bool bf16, const ScanBwdParams& p, cudaStream_t st) {
  return bf16 ? bwd_t<__nv_bfloat16>(p, st) : bwd_t<float>(p, st);
}

}  // namespace rwkv
