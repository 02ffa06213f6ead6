// Launch interface of the operators around the WKV recurrence: the causal convolution, the selective
// scan and the layer norm.
#pragma once
#include "launch.h"

namespace rwkv {

// Causal convolution (conv.cu).  Rows of x are ldx elements apart, everything else is dense; a null
// optional pointer is absent.
struct ConvParams {
  int B, T, C, W;       // W in 2..4
  int silu;             // 1: y = silu(pre)
  int stretch, nseg;    // tokens per stretch, stretches per batch row (set by the launch)
  long long ldx;
  const float* weight;  // [C,W]
  const float* bias;    // [C] or null
  const void* x;        // [B,T,C]; step: [B,C]
  void* y;
  const void* state_in;  // [B,W-1,C] or null (zero)
  void* state_out;       // [B,W-1,C] or null; may be state_in
  const void* gy;        // backward: [B,T,C]
  const void* gstate_out;  // [B,W-1,C] or null
  void* gx;
  void* gstate_in;      // [B,W-1,C] or null
  float* gweight;       // [C,W]
  float* gbias;         // [C] or null
  float* part;          // [conv_bwd_parts()][W+1][C] workspace
};
enum class ConvPass { kForward, kBackward, kStep };
int conv_bwd_parts(int B, int T);
// width: channels (4, 2 or 1) that C, ldx and every base allow in one access; with 2 or more the filters
// allow 16-byte accesses.
cudaError_t launch_conv(ConvPass pass, bool bf16, int width, const ConvParams& p, cudaStream_t st);
// dst[i] = src[i], or 0 without src.
cudaError_t launch_copy_bytes(size_t n, const void* src, void* dst, cudaStream_t st);

// Selective scan (scan_fwd.cu, scan_bwd.cu, scan_step.cu).  Rows of x, dt, b, c, z are ld* elements
// apart, everything else is dense.
constexpr int kScanCkLen = 16;  // tokens between the states the forward keeps for the backward
struct ScanParams {
  int B, T, C, N;
  int ctiles;           // channel tiles (set by the launch)
  int seg_len, nseg;    // time segments
  int vec;              // x, dt, z, y and the gradients of their shape allow 16-byte accesses
  int vec_bc;           // b and c do
  long long ldx, lddt, ldb, ldc, ldz;
  const float* a_log;   // [C,N]
  const float* d;       // [C] or null
  const float* dt_bias;  // [C] or null
  const void* x;        // [B,T,C]; step: [B,C]
  const void* dt;
  const void* b;        // [B,T,N]; step: [B,N]
  const void* c;
  const void* z;        // [B,T,C] or null
  void* y;              // [B,T,C] or null (states only)
  const float* h_in;    // [B,C,N] or null (zero)
  float* h_out;         // [B,C,N] or null; may be h_in
  float* ckpt;          // [ceil(T/16),B,C,N] states before tokens 0, 16, ... or null
  // workspace of a segmented call
  float* seg_h;         // [nseg-1][B,C,N] states reached by each segment from a zero state
  float* seg_dt;        // [nseg-1][B,C] their sums of Δ
  float* seg_h0;        // [B,C,N] copy of h_in
};
struct ScanBwdParams {
  ScanParams f;         // inputs as the forward's, ckpt read; y, h_out unused
  const void* gy;       // [B,T,C]
  const float* gh_out;  // [B,C,N] or null
  void* gx;             // [B,T,C]
  void* gdt;
  void* gz;             // or null
  void* gb;             // [B,T,N]
  void* gc;
  float* ga_log;        // [C,N]
  float* gd;            // [C] or null
  float* gdt_bias;      // [C] or null
  float* gh_in;         // [B,C,N] or null
  float* part_bc;       // [ctiles][B,T][2][N]: per channel tile, Σ over its channels for gc and gb
  float* part_a;        // [B nseg][C,N]
  float* part_v;        // [B nseg][2][C]
  float* seg_g;         // [nseg][B,C,N] gradient that leaves each segment at its start, from zero at its end
  float* seg_dt;        // [nseg][B,C]
  float* seg_g0;        // [B,C,N] copy of gh_out
};
int scan_fwd_channels(int N);  // channels per CTA
int scan_bwd_channels(int N);
int scan_tile_tokens();
cudaError_t launch_scan_fwd(bool bf16, const ScanParams& p, cudaStream_t st);
// The backward's recurrence over segments 1 .. nseg-1, each from zero at its end (the last from
// gh_out): x = gy, b = c, h_in = gh_out, seg_h, seg_h0, seg_dt its workspace.
cudaError_t launch_scan_reverse(bool bf16, const ScanParams& p, cudaStream_t st);
cudaError_t launch_scan_bwd(bool bf16, const ScanBwdParams& p, cudaStream_t st);
cudaError_t launch_scan_step(bool bf16, const ScanParams& p, cudaStream_t st);

// Layer norm over the N columns of each of G groups of a row (norm.cu); all tensors dense.
struct NormParams {
  long long M;          // rows
  int G, N;
  float eps;
  const float* weight;  // [G,N]
  const float* bias;    // [G,N] or null
  const void* x;        // [M,G,N]
  const void* gate;     // [M,G,N] or null
  void* y;
  const void* gy;       // backward
  void* gx;
  void* ggate;
  float* gweight;       // [G,N]
  float* gbias;         // [G,N] or null
  float* part;          // [norm_bwd_parts()][2][G,N] workspace
  int slices;           // sets of rows whose weight gradients are summed apart
};
// kAligned: N and every base allow 16-byte accesses.  kShifted: the activations' bases lie alike on the
// 16-byte grid and N is a vector or more.  kSingle: any.
enum class NormAccess { kAligned, kShifted, kSingle };
int norm_bwd_parts(long long M, int G, int N, bool bf16);
cudaError_t launch_norm_fwd(bool bf16, NormAccess access, const NormParams& p, cudaStream_t st);
cudaError_t launch_norm_bwd(bool bf16, NormAccess access, const NormParams& p, cudaStream_t st);

}  // namespace rwkv
