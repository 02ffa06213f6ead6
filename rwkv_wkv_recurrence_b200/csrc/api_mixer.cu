// C-ABI layer of the operators around the WKV recurrence: the causal convolution, the selective
// scan and the layer norm (argument validation, workspace planning, dispatch).
#include <algorithm>
#include <climits>
#include <cstddef>
#include <initializer_list>

#include "../../include/rwkv_wkv.h"
#include "mixer.h"
#include "scan_plan.h"

using namespace rwkv;

namespace {

bool fits_int(int64_t x) { return x >= 0 && x <= INT_MAX; }
bool dtype_ok(rwkv_dtype d) { return d == RWKV_F32 || d == RWKV_BF16; }

// Every non-null pointer a multiple of `bytes`.
bool aligned(size_t bytes, std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (q != nullptr && (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) != 0) return false;
  return true;
}

// Every length a multiple of an access's elements.
bool vec_len(int vec, std::initializer_list<int64_t> lens) {
  for (int64_t l : lens)
    if (l % vec != 0) return false;
  return true;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Kernels count channels in ints, rounded up to a thread's, a warp's or a CTA's (128 at most).
constexpr int64_t kMaxChannels = INT_MAX - 128;

// Blocks of a launch must fit the grid's x dimension.
bool grid_ok(double blocks) { return blocks <= (double)INT_MAX; }

}  // namespace

extern "C" {

// ------------------------------------------------------------------ causal convolution
static int conv_width(int64_t C, int64_t ldx, size_t esz, const float* weight,
                      std::initializer_list<const void*> acts) {
  for (int v = 4; v >= 2; v /= 2)
    if (aligned(v * esz, acts) && aligned(16, {weight}) && vec_len(v, {C, ldx})) return v;
  return 1;
}

static bool conv_bwd_fits(int64_t B, int64_t T, int64_t C, int64_t W) {
  return grid_ok((double)B * ((double)T / 512 + 1) * ((double)C / 32 + 1)) &&
         grid_ok((double)B * ((double)T / 64 + 1)) && grid_ok((double)(W + 1) * (double)C) && T <= INT_MAX - 64;
}

size_t rwkv_causal_conv_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t W) {
  if (B <= 0 || T <= 0 || C <= 0 || W < 2 || W > 4 || !fits_int(B) || !fits_int(T) || !fits_int(C)) return 0;
  if (!conv_bwd_fits(B, T, C, W)) return 0;  // the call refuses it
  return (size_t)conv_bwd_parts((int)B, (int)T) * (W + 1) * C * sizeof(float);
}

rwkv_status rwkv_causal_conv_forward(int64_t B, int64_t T, int64_t C, int64_t W, rwkv_dtype dtype, const float* weight,
                                     const float* bias, int act, const void* x, int64_t ldx, void* y,
                                     const void* state_in, void* state_out, rwkv_stream_t stream) {
  if (!fits_int(B) || !fits_int(T) || !fits_int(C) || !fits_int(W) || !dtype_ok(dtype)) return RWKV_ERR_INVALID_ARG;
  if (act != RWKV_ACT_NONE && act != RWKV_ACT_SILU) return RWKV_ERR_INVALID_ARG;
  if (ldx < C) return RWKV_ERR_INVALID_ARG;
  if (W < 2 || W > 4) return RWKV_ERR_UNSUPPORTED;
  if (B == 0 || C == 0) return RWKV_OK;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned(esz, {state_in, state_out})) return RWKV_ERR_UNSUPPORTED;
  if (T == 0) {
    if (state_out == nullptr || state_out == state_in) return RWKV_OK;
    const size_t n = (size_t)B * (W - 1) * C * esz;
    if (!grid_ok((double)n / 256 + 1)) return RWKV_ERR_UNSUPPORTED;
    return launch_copy_bytes(n, state_in, state_out, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
  }
  if (weight == nullptr || x == nullptr || y == nullptr) return RWKV_ERR_INVALID_ARG;
  if (!aligned(esz, {x, y}) || !aligned(4, {weight, bias})) return RWKV_ERR_UNSUPPORTED;
  if (!grid_ok((double)B * ((double)T / 32 + 1) * (double)C / 128 + 1) || T > INT_MAX - 64 || C > kMaxChannels)
    return RWKV_ERR_UNSUPPORTED;
  ConvParams p{};
  p.B = (int)B;
  p.T = (int)T;
  p.C = (int)C;
  p.W = (int)W;
  p.silu = act == RWKV_ACT_SILU;
  p.ldx = ldx;
  p.weight = weight;
  p.bias = bias;
  p.x = x;
  p.y = y;
  p.state_in = state_in;
  p.state_out = state_out;
  const int width = conv_width(C, ldx, esz, weight, {x, y, state_in, state_out});
  return launch_conv(ConvPass::kForward, bf16, width, p, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
}

rwkv_status rwkv_causal_conv_backward(int64_t B, int64_t T, int64_t C, int64_t W, rwkv_dtype dtype,
                                      const float* weight, const float* bias, int act, const void* x, int64_t ldx,
                                      const void* state_in, const void* gy, const void* gstate_out, void* gx,
                                      float* gweight, float* gbias, void* gstate_in, void* workspace,
                                      size_t workspace_bytes, rwkv_stream_t stream) {
  if (!fits_int(B) || !fits_int(T) || !fits_int(C) || !fits_int(W) || !dtype_ok(dtype)) return RWKV_ERR_INVALID_ARG;
  if (act != RWKV_ACT_NONE && act != RWKV_ACT_SILU) return RWKV_ERR_INVALID_ARG;
  if (ldx < C) return RWKV_ERR_INVALID_ARG;
  if (W < 2 || W > 4) return RWKV_ERR_UNSUPPORTED;
  if (C == 0) return RWKV_OK;
  if (gweight == nullptr) return RWKV_ERR_INVALID_ARG;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned(esz, {gstate_out, gstate_in}) || !aligned(4, {weight, bias, gweight, gbias}))
    return RWKV_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) {  // empty sums; the state's gradient passes through
    if (cudaMemsetAsync(gweight, 0, (size_t)C * W * sizeof(float), st) != cudaSuccess) return RWKV_ERR_CUDA;
    if (gbias != nullptr && cudaMemsetAsync(gbias, 0, (size_t)C * sizeof(float), st) != cudaSuccess)
      return RWKV_ERR_CUDA;
    const size_t n = (size_t)B * (W - 1) * C * esz;
    if (gstate_in == nullptr || gstate_in == gstate_out || n == 0) return RWKV_OK;
    if (!grid_ok((double)n / 256 + 1)) return RWKV_ERR_UNSUPPORTED;
    return launch_copy_bytes(n, gstate_out, gstate_in, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
  }
  if (weight == nullptr || x == nullptr || gy == nullptr || gx == nullptr) return RWKV_ERR_INVALID_ARG;
  if (!aligned(esz, {x, gy, gx, state_in})) return RWKV_ERR_UNSUPPORTED;
  if (!conv_bwd_fits(B, T, C, W)) return RWKV_ERR_UNSUPPORTED;
  const size_t need = rwkv_causal_conv_backward_workspace_bytes(B, T, C, W);
  if (workspace == nullptr || workspace_bytes < need) return RWKV_ERR_WORKSPACE;
  if (!aligned(4, {workspace})) return RWKV_ERR_UNSUPPORTED;
  ConvParams p{};
  p.B = (int)B;
  p.T = (int)T;
  p.C = (int)C;
  p.W = (int)W;
  p.silu = act == RWKV_ACT_SILU;
  p.ldx = ldx;
  p.weight = weight;
  p.bias = bias;
  p.x = x;
  p.state_in = state_in;
  p.gy = gy;
  p.gstate_out = gstate_out;
  p.gx = gx;
  p.gstate_in = gstate_in;
  p.gweight = gweight;
  p.gbias = gbias;
  p.part = static_cast<float*>(workspace);
  const int width = conv_width(C, ldx, esz, weight, {x, gy, gx, state_in, gstate_out, gstate_in});
  return launch_conv(ConvPass::kBackward, bf16, width, p, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
}

rwkv_status rwkv_causal_conv_step(int64_t B, int64_t C, int64_t W, rwkv_dtype dtype, const float* weight,
                                  const float* bias, int act, const void* x, int64_t ldx, void* y,
                                  const void* state_in, void* state_out, rwkv_stream_t stream) {
  if (!fits_int(B) || !fits_int(C) || !fits_int(W) || !dtype_ok(dtype)) return RWKV_ERR_INVALID_ARG;
  if (act != RWKV_ACT_NONE && act != RWKV_ACT_SILU) return RWKV_ERR_INVALID_ARG;
  if (ldx < C) return RWKV_ERR_INVALID_ARG;
  if (W < 2 || W > 4) return RWKV_ERR_UNSUPPORTED;
  if (B == 0 || C == 0) return RWKV_OK;
  if (weight == nullptr || x == nullptr || y == nullptr || state_out == nullptr) return RWKV_ERR_INVALID_ARG;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  if (!aligned(esz, {x, y, state_in, state_out}) || !aligned(4, {weight, bias})) return RWKV_ERR_UNSUPPORTED;
  if (!grid_ok((double)B * (double)C / 128 + 1) || C > kMaxChannels) return RWKV_ERR_UNSUPPORTED;
  ConvParams p{};
  p.B = (int)B;
  p.C = (int)C;
  p.W = (int)W;
  p.T = 1;
  p.silu = act == RWKV_ACT_SILU;
  p.ldx = ldx;
  p.weight = weight;
  p.bias = bias;
  p.x = x;
  p.y = y;
  p.state_in = state_in;
  p.state_out = state_out;
  const int width = conv_width(C, ldx, esz, weight, {x, y, state_in, state_out});
  return launch_conv(ConvPass::kStep, bf16, width, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? RWKV_OK
             : RWKV_ERR_CUDA;
}

}  // extern "C"

// ------------------------------------------------------------------ selective scan
namespace {

bool scan_n_ok(int64_t N) { return N == 8 || N == 16 || N == 32 || N == 64; }

ScanPlan plan_scan_fwd(int64_t B, int64_t T, int64_t C, int64_t N, int algo) {
  const int64_t ch = scan_fwd_channels((int)N);
  return cut_forward(B * ((C + ch - 1) / ch), T, scan_tile_tokens(), algo);
}

ScanPlan plan_scan_bwd(int64_t B, int64_t T, int64_t C, int64_t N) {
  const int64_t ch = scan_bwd_channels((int)N);
  return cut_backward(B * ((C + ch - 1) / ch), T, scan_tile_tokens());
}

struct ScanFwdWs {
  size_t h = 0, dt = 0, h0 = 0, total = 0;
};
ScanFwdWs scan_fwd_ws(int64_t B, int64_t C, int64_t N, int nseg) {
  ScanFwdWs w;
  if (nseg <= 1) return w;
  const size_t state = (size_t)B * C * N * sizeof(float);
  w.dt = up256((size_t)(nseg - 1) * state);
  w.h0 = w.dt + up256((size_t)(nseg - 1) * B * C * sizeof(float));
  w.total = w.h0 + up256(state);
  return w;
}

struct ScanBwdWs {
  size_t bc = 0, a = 0, v = 0, g = 0, dt = 0, g0 = 0, ckpt = 0, fwd = 0, total = 0;
};
ScanBwdWs scan_bwd_ws(int64_t B, int64_t T, int64_t C, int64_t N, bool have_ckpt) {
  ScanBwdWs w;
  const ScanPlan pl = plan_scan_bwd(B, T, C, N);
  const int64_t ch = scan_bwd_channels((int)N), tiles = (C + ch - 1) / ch;
  const size_t state = (size_t)B * C * N * sizeof(float), parts = (size_t)B * pl.nseg;
  w.a = up256((size_t)tiles * B * T * 2 * N * sizeof(float));
  w.v = w.a + up256(parts * C * N * sizeof(float));
  w.g = w.v + up256(parts * 2 * C * sizeof(float));
  w.total = w.g;
  if (pl.nseg > 1) {
    w.dt = w.g + up256((size_t)pl.nseg * state);
    w.g0 = w.dt + up256((size_t)pl.nseg * B * C * sizeof(float));
    w.total = w.g0 + up256(state);
  }
  if (!have_ckpt) {
    w.ckpt = w.total;
    w.fwd = w.ckpt + up256((size_t)((T + kScanCkLen - 1) / kScanCkLen) * state);
    w.total = w.fwd + scan_fwd_ws(B, C, N, plan_scan_fwd(B, T, C, N, RWKV_ALGO_AUTO).nseg).total;
  }
  return w;
}

// CTAs of the forward and the backward, with the most segments a plan makes.
bool scan_grid_ok(int64_t B, int64_t T, int64_t C, int64_t N) {
  const double ch = (double)scan_fwd_channels((int)N);
  return grid_ok((double)B * ((double)C / ch + 1) * ((double)T / 32 + 1)) &&
         grid_ok(((double)B * (double)T * (double)(2 * N) + (double)C * (double)(N + 2)) / 256 + 2) &&
         T <= INT_MAX - 64 && C <= kMaxChannels;
}

struct ScanIn {
  const float *a_log, *d, *dt_bias;
  const void* x;
  int64_t ldx;
  const void* dt;
  int64_t lddt;
  const void* b;
  int64_t ldb;
  const void* c;
  int64_t ldc;
  const void* z;
  int64_t ldz;
};

// Checks of the arguments that all three calls share; RWKV_OK when the call may go on.
rwkv_status scan_check(int64_t B, int64_t T, int64_t C, int64_t N, rwkv_dtype dtype, const ScanIn& in) {
  if (!fits_int(B) || !fits_int(T) || !fits_int(C) || !fits_int(N) || !dtype_ok(dtype)) return RWKV_ERR_INVALID_ARG;
  if (!scan_n_ok(N)) return RWKV_ERR_UNSUPPORTED;
  if (in.ldx < C || in.lddt < C || in.ldb < N || in.ldc < N || (in.z != nullptr && in.ldz < C))
    return RWKV_ERR_INVALID_ARG;
  return RWKV_OK;
}

void scan_fill(ScanParams& p, int64_t B, int64_t T, int64_t C, int64_t N, const ScanIn& in) {
  p.B = (int)B;
  p.T = (int)T;
  p.C = (int)C;
  p.N = (int)N;
  p.ldx = in.ldx;
  p.lddt = in.lddt;
  p.ldb = in.ldb;
  p.ldc = in.ldc;
  p.ldz = in.ldz;
  p.a_log = in.a_log;
  p.d = in.d;
  p.dt_bias = in.dt_bias;
  p.x = in.x;
  p.dt = in.dt;
  p.b = in.b;
  p.c = in.c;
  p.z = in.z;
}

// Runs the forward on checked arguments.
rwkv_status run_scan_fwd(ScanParams p, bool bf16, int algo, void* ws, cudaStream_t st) {
  const ScanPlan pl = plan_scan_fwd(p.B, p.T, p.C, p.N, algo);
  p.seg_len = pl.seg_len;
  p.nseg = pl.nseg;
  if (pl.nseg > 1) {
    const ScanFwdWs w = scan_fwd_ws(p.B, p.C, p.N, pl.nseg);
    char* base = static_cast<char*>(ws);
    p.seg_h = reinterpret_cast<float*>(base + w.h);
    p.seg_dt = reinterpret_cast<float*>(base + w.dt);
    p.seg_h0 = reinterpret_cast<float*>(base + w.h0);
  }
  return launch_scan_fwd(bf16, p, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t rwkv_selective_scan_forward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N, int algo) {
  if (B <= 0 || T <= 0 || C <= 0 || !scan_n_ok(N) || !fits_int(B) || !fits_int(T) || !fits_int(C)) return 0;
  if (!scan_grid_ok(B, T, C, N)) return 0;
  return scan_fwd_ws(B, C, N, plan_scan_fwd(B, T, C, N, algo).nseg).total;
}

rwkv_status rwkv_selective_scan_forward(int64_t B, int64_t T, int64_t C, int64_t N, rwkv_dtype dtype,
                                        const float* a_log, const float* d, const float* dt_bias, const void* x,
                                        int64_t ldx, const void* dt, int64_t lddt, const void* b, int64_t ldb,
                                        const void* c, int64_t ldc, const void* z, int64_t ldz, void* y,
                                        const float* h_in, float* h_out, float* ckpt, int64_t chunk_len, int algo,
                                        void* workspace, size_t workspace_bytes, rwkv_stream_t stream) {
  const ScanIn in{a_log, d, dt_bias, x, ldx, dt, lddt, b, ldb, c, ldc, z, ldz};
  rwkv_status s = scan_check(B, T, C, N, dtype, in);
  if (s != RWKV_OK) return s;
  if (algo < RWKV_ALGO_AUTO || algo > RWKV_ALGO_CHUNKED) return RWKV_ERR_INVALID_ARG;
  if (ckpt != nullptr && (chunk_len <= 0 || chunk_len % 16 != 0)) return RWKV_ERR_INVALID_ARG;
  if (ckpt != nullptr && chunk_len != kScanCkLen) return RWKV_ERR_UNSUPPORTED;
  if (B == 0 || C == 0) return RWKV_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned(16, {h_in, h_out, ckpt})) return RWKV_ERR_UNSUPPORTED;
  if (T == 0) {
    if (h_out == nullptr || h_out == h_in) return RWKV_OK;
    const size_t n = (size_t)B * C * N * sizeof(float);
    if (!grid_ok((double)n / 256 + 1)) return RWKV_ERR_UNSUPPORTED;
    return launch_copy_bytes(n, h_in, h_out, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
  }
  if (a_log == nullptr || x == nullptr || dt == nullptr || b == nullptr || c == nullptr) return RWKV_ERR_INVALID_ARG;
  if (y == nullptr && h_out == nullptr && ckpt == nullptr) return RWKV_ERR_INVALID_ARG;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  if (!aligned(esz, {x, dt, b, c, z, y}) || !aligned(4, {a_log, d, dt_bias})) return RWKV_ERR_UNSUPPORTED;
  if (!scan_grid_ok(B, T, C, N)) return RWKV_ERR_UNSUPPORTED;
  const size_t need = rwkv_selective_scan_forward_workspace_bytes(B, T, C, N, algo);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return RWKV_ERR_WORKSPACE;
  if (need > 0 && !aligned(16, {workspace})) return RWKV_ERR_UNSUPPORTED;
  ScanParams p{};
  scan_fill(p, B, T, C, N, in);
  p.y = y;
  p.h_in = h_in;
  p.h_out = h_out;
  p.ckpt = ckpt;
  const int v = 16 / (int)esz;
  p.vec = aligned(16, {x, dt, z, y}) && vec_len(v, {C, ldx, lddt}) && (z == nullptr || ldz % v == 0);
  p.vec_bc = aligned(16, {b, c}) && vec_len(v, {ldb, ldc});
  return run_scan_fwd(p, bf16, algo, workspace, st);
}

size_t rwkv_selective_scan_backward_workspace_bytes(int64_t B, int64_t T, int64_t C, int64_t N, int64_t chunk_len,
                                                    int have_ckpt) {
  (void)chunk_len;  // one interval is supported
  if (B <= 0 || T <= 0 || C <= 0 || !scan_n_ok(N) || !fits_int(B) || !fits_int(T) || !fits_int(C)) return 0;
  if (!scan_grid_ok(B, T, C, N)) return 0;
  return scan_bwd_ws(B, T, C, N, have_ckpt != 0).total;
}

rwkv_status rwkv_selective_scan_backward(int64_t B, int64_t T, int64_t C, int64_t N, rwkv_dtype dtype,
                                         const float* a_log, const float* d, const float* dt_bias, const void* x,
                                         int64_t ldx, const void* dt, int64_t lddt, const void* b, int64_t ldb,
                                         const void* c, int64_t ldc, const void* z, int64_t ldz, const void* gy,
                                         const float* h_in, const float* gh_out, const float* ckpt, int64_t chunk_len,
                                         void* gx, void* gdt, void* gb, void* gc, void* gz, float* ga_log, float* gd,
                                         float* gdt_bias, float* gh_in, void* workspace, size_t workspace_bytes,
                                         rwkv_stream_t stream) {
  const ScanIn in{a_log, d, dt_bias, x, ldx, dt, lddt, b, ldb, c, ldc, z, ldz};
  rwkv_status s = scan_check(B, T, C, N, dtype, in);
  if (s != RWKV_OK) return s;
  if (chunk_len <= 0 || chunk_len % 16 != 0) return RWKV_ERR_INVALID_ARG;
  if (chunk_len != kScanCkLen) return RWKV_ERR_UNSUPPORTED;
  if (C == 0) return RWKV_OK;
  if (a_log == nullptr || ga_log == nullptr) return RWKV_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned(16, {h_in, gh_out, ckpt, gh_in}) || !aligned(4, {a_log, d, dt_bias, ga_log, gd, gdt_bias}))
    return RWKV_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) {  // empty sums; the state's gradient passes through
    if (cudaMemsetAsync(ga_log, 0, (size_t)C * N * sizeof(float), st) != cudaSuccess) return RWKV_ERR_CUDA;
    if (gd != nullptr && cudaMemsetAsync(gd, 0, (size_t)C * sizeof(float), st) != cudaSuccess) return RWKV_ERR_CUDA;
    if (gdt_bias != nullptr && cudaMemsetAsync(gdt_bias, 0, (size_t)C * sizeof(float), st) != cudaSuccess)
      return RWKV_ERR_CUDA;
    const size_t n = (size_t)B * C * N * sizeof(float);
    if (gh_in == nullptr || gh_in == gh_out || n == 0) return RWKV_OK;
    if (!grid_ok((double)n / 256 + 1)) return RWKV_ERR_UNSUPPORTED;
    return launch_copy_bytes(n, gh_out, gh_in, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
  }
  if (x == nullptr || dt == nullptr || b == nullptr || c == nullptr || gy == nullptr || gx == nullptr ||
      gdt == nullptr || gb == nullptr || gc == nullptr || (z != nullptr && gz == nullptr))
    return RWKV_ERR_INVALID_ARG;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  if (!aligned(esz, {x, dt, b, c, z, gy, gx, gdt, gb, gc, gz})) return RWKV_ERR_UNSUPPORTED;
  if (!scan_grid_ok(B, T, C, N)) return RWKV_ERR_UNSUPPORTED;
  const size_t need = rwkv_selective_scan_backward_workspace_bytes(B, T, C, N, chunk_len, ckpt != nullptr);
  if (workspace == nullptr || workspace_bytes < need) return RWKV_ERR_WORKSPACE;
  if (!aligned(16, {workspace})) return RWKV_ERR_UNSUPPORTED;
  const ScanBwdWs w = scan_bwd_ws(B, T, C, N, ckpt != nullptr);
  char* base = static_cast<char*>(workspace);
  ScanBwdParams p{};
  scan_fill(p.f, B, T, C, N, in);
  const int v = 16 / (int)esz;
  p.f.vec = aligned(16, {x, dt, z, gy, gx, gdt, gz}) && vec_len(v, {C, ldx, lddt}) && (z == nullptr || ldz % v == 0);
  p.f.vec_bc = aligned(16, {b, c}) && vec_len(v, {ldb, ldc});
  p.f.h_in = h_in;
  if (ckpt == nullptr) {  // the states again, by the forward without its outputs
    ScanParams f = p.f;
    f.ckpt = reinterpret_cast<float*>(base + w.ckpt);
    s = run_scan_fwd(f, bf16, RWKV_ALGO_AUTO, base + w.fwd, st);
    if (s != RWKV_OK) return s;
    p.f.ckpt = f.ckpt;
  } else {
    p.f.ckpt = const_cast<float*>(ckpt);  // read only in the backward
  }
  const ScanPlan pl = plan_scan_bwd(B, T, C, N);
  p.f.seg_len = pl.seg_len;
  p.f.nseg = pl.nseg;
  p.gy = gy;
  p.gh_out = gh_out;
  p.gx = gx;
  p.gdt = gdt;
  p.gz = z != nullptr ? gz : nullptr;
  p.gb = gb;
  p.gc = gc;
  p.ga_log = ga_log;
  p.gd = gd;
  p.gdt_bias = gdt_bias;
  p.gh_in = gh_in;
  p.part_bc = reinterpret_cast<float*>(base + w.bc);
  p.part_a = reinterpret_cast<float*>(base + w.a);
  p.part_v = reinterpret_cast<float*>(base + w.v);
  p.seg_g = reinterpret_cast<float*>(base + w.g);
  p.seg_dt = reinterpret_cast<float*>(base + w.dt);
  p.seg_g0 = reinterpret_cast<float*>(base + w.g0);
  return launch_scan_bwd(bf16, p, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
}

rwkv_status rwkv_selective_scan_step(int64_t B, int64_t C, int64_t N, rwkv_dtype dtype, const float* a_log,
                                     const float* d, const float* dt_bias, const void* x, int64_t ldx, const void* dt,
                                     int64_t lddt, const void* b, int64_t ldb, const void* c, int64_t ldc,
                                     const void* z, int64_t ldz, void* y, const float* h_in, float* h_out,
                                     rwkv_stream_t stream) {
  const ScanIn in{a_log, d, dt_bias, x, ldx, dt, lddt, b, ldb, c, ldc, z, ldz};
  const rwkv_status s = scan_check(B, 1, C, N, dtype, in);
  if (s != RWKV_OK) return s;
  if (B == 0 || C == 0) return RWKV_OK;
  if (a_log == nullptr || x == nullptr || dt == nullptr || b == nullptr || c == nullptr || y == nullptr ||
      h_out == nullptr)
    return RWKV_ERR_INVALID_ARG;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  if (!aligned(16, {h_in, h_out}) || !aligned(esz, {x, dt, b, c, z, y}) || !aligned(4, {a_log, d, dt_bias}))
    return RWKV_ERR_UNSUPPORTED;
  if (!grid_ok((double)C * (double)N / 4 + 256) || B > INT_MAX / 2) return RWKV_ERR_UNSUPPORTED;
  ScanParams p{};
  scan_fill(p, B, 1, C, N, in);
  const int v = 16 / (int)esz;
  p.vec = aligned(16, {x, dt, z, y}) && vec_len(v, {C, ldx, lddt}) && (z == nullptr || ldz % v == 0);
  p.vec_bc = aligned(16, {b, c}) && vec_len(v, {ldb, ldc});
  p.y = y;
  p.h_in = h_in;
  p.h_out = h_out;
  return launch_scan_step(bf16, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
}

// ------------------------------------------------------------------ layer norm
static rwkv_status norm_check(int64_t M, int64_t G, int64_t N, rwkv_dtype dtype, float eps) {
  if (M < 0 || !fits_int(G) || !fits_int(N) || !dtype_ok(dtype)) return RWKV_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || eps > 3.402823466e+38f) return RWKV_ERR_INVALID_ARG;
  return RWKV_OK;
}

// `acts`: the activations; absent ones (null) count as lying like x.
static NormAccess norm_access(int64_t N, size_t esz, const void* x, std::initializer_list<const void*> acts,
                              std::initializer_list<const float*> params) {
  const auto at = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16; };
  bool alike = true, on_grid = at(x) == 0 && N % (int64_t)(16 / esz) == 0;
  for (const void* q : acts) alike = alike && (q == nullptr || at(q) == at(x));
  for (const float* q : params) on_grid = on_grid && at(q) == 0;
  if (!alike || N < (int64_t)(16 / esz)) return NormAccess::kSingle;
  return on_grid ? NormAccess::kAligned : NormAccess::kShifted;
}

size_t rwkv_layer_norm_backward_workspace_bytes(int64_t M, int64_t G, int64_t N, rwkv_dtype dtype) {
  if (M <= 0 || G <= 0 || N <= 0 || !fits_int(G) || !fits_int(N) || !dtype_ok(dtype) || G * N > INT_MAX / 2) return 0;
  return (size_t)norm_bwd_parts(M, (int)G, (int)N, dtype == RWKV_BF16) * 2 * G * N * sizeof(float);
}

rwkv_status rwkv_layer_norm_forward(int64_t M, int64_t G, int64_t N, rwkv_dtype dtype, const float* weight,
                                    const float* bias, float eps, const void* x, const void* gate, void* y,
                                    rwkv_stream_t stream) {
  const rwkv_status s = norm_check(M, G, N, dtype, eps);
  if (s != RWKV_OK) return s;
  if (M == 0 || G == 0 || N == 0) return RWKV_OK;
  if (weight == nullptr || x == nullptr || y == nullptr) return RWKV_ERR_INVALID_ARG;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  if (!aligned(esz, {x, gate, y}) || !aligned(4, {weight, bias})) return RWKV_ERR_UNSUPPORTED;
  if (G * N > INT_MAX / 2) return RWKV_ERR_UNSUPPORTED;
  NormParams p{};
  p.M = M;
  p.G = (int)G;
  p.N = (int)N;
  p.eps = eps;
  p.weight = weight;
  p.bias = bias;
  p.x = x;
  p.gate = gate;
  p.y = y;
  const NormAccess access = norm_access(N, esz, x, {gate, y}, {weight, bias});
  return launch_norm_fwd(bf16, access, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? RWKV_OK
                                                                                                : RWKV_ERR_CUDA;
}

rwkv_status rwkv_layer_norm_backward(int64_t M, int64_t G, int64_t N, rwkv_dtype dtype, const float* weight,
                                     const float* bias, float eps, const void* x, const void* gate, const void* gy,
                                     void* gx, void* ggate, float* gweight, float* gbias, void* workspace,
                                     size_t workspace_bytes, rwkv_stream_t stream) {
  const rwkv_status s = norm_check(M, G, N, dtype, eps);
  if (s != RWKV_OK) return s;
  if (G == 0 || N == 0) return RWKV_OK;
  if (gweight == nullptr) return RWKV_ERR_INVALID_ARG;
  if (!aligned(4, {weight, bias, gweight, gbias})) return RWKV_ERR_UNSUPPORTED;
  if (G * N > INT_MAX / 2) return RWKV_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {  // empty sums
    if (cudaMemsetAsync(gweight, 0, (size_t)G * N * sizeof(float), st) != cudaSuccess) return RWKV_ERR_CUDA;
    if (gbias != nullptr && cudaMemsetAsync(gbias, 0, (size_t)G * N * sizeof(float), st) != cudaSuccess)
      return RWKV_ERR_CUDA;
    return RWKV_OK;
  }
  if (weight == nullptr || x == nullptr || gy == nullptr || gx == nullptr || (gate != nullptr && ggate == nullptr))
    return RWKV_ERR_INVALID_ARG;
  const bool bf16 = dtype == RWKV_BF16;
  const size_t esz = bf16 ? 2 : 4;
  if (!aligned(esz, {x, gate, gy, gx, ggate})) return RWKV_ERR_UNSUPPORTED;
  const size_t need = rwkv_layer_norm_backward_workspace_bytes(M, G, N, dtype);
  if (workspace == nullptr || workspace_bytes < need) return RWKV_ERR_WORKSPACE;
  if (!aligned(16, {workspace})) return RWKV_ERR_UNSUPPORTED;
  NormParams p{};
  p.M = M;
  p.G = (int)G;
  p.N = (int)N;
  p.eps = eps;
  p.weight = weight;
  p.bias = bias;
  p.x = x;
  p.gate = gate;
  p.gy = gy;
  p.gx = gx;
  p.ggate = ggate;
  p.gweight = gweight;
  p.gbias = gbias;
  p.part = static_cast<float*>(workspace);
  const NormAccess access = norm_access(N, esz, x, {gate, gy, gx, ggate}, {weight, bias});
  return launch_norm_bwd(bf16, access, p, st) == cudaSuccess ? RWKV_OK : RWKV_ERR_CUDA;
}

}  // extern "C"
