// Internal launch interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Not part of the public header.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rwkv {

struct DevCtl;  // the device control block (wkv_common.cuh)

// Parameters of the WKV-4 forward kernel.  A CTA owns 32 channels of one
// batch row over one time segment [seg*seg_len, min(T, (seg+1)*seg_len)).
struct Fwd4Params {
  int B, T, C;
  int ctiles;   // ceil(C / 32)
  int seg_len;  // time steps per segment (multiple of the 64-step tile)
  int nseg;
  int stages;   // TMA pipeline depth
  const float* w;
  const float* u;
  void* y;                        // [B,T,C] or null (state-only pass)
  const float* start;             // start state per segment, or null = zero
  long long start_seg_stride;     // floats between consecutive segments' start states
  float* end;                     // end state per segment, or null
  long long end_seg_stride;
  float* ckpt;                    // [nck,3,B,C] states before tokens 0, L, 2L, ... or null
  int ckpt_len;                   // L (multiple of 16) when ckpt != null
  int tma;                        // 1: k, v (, r) arrive by TMA and y leaves by TMA stores; 0: plain
                                  // element loads and stores (any element-aligned base, any C)
  const void* k;                  // [B,T,C] (read directly when tma == 0)
  const void* v;
  const void* r;                  // [B,T,C] receptance of the gated forward (tma == 0), else null
  DevCtl* ctl;                    // device control block (error word, wait limit)
  // the one-launch chunked schedule (launch_wkv4_fwd_lookback): per segment and lane the summary as
  // (a, b, p) doubles, one flag per (segment, CTA) zeroed before the launch, and the sequence's
  // start state (or null = zero)
  double* lb_agg;                 // [nseg][B*C][3]
  unsigned int* lb_flag;          // [nseg][ctiles*B]
  const float* lb_in;             // [3,B,C] or null
};

struct Bwd4Params {
  int B, T, C;
  int ctiles;
  int stages;
  const float* w;
  const float* u;
  const float* ckpt;  // [ceil(T/16),3,B,C], interval 16
  void* gk;
  void* gv;
  double* part;       // [2,B,C] per-lane gw, gu partial sums
  DevCtl* ctl;        // device control block
  const void* r;      // [B,T,C] receptance (gated backward only)
  void* gr;           // [B,T,C] its gradient (gated backward only)
  int tma;            // 1: k, v, gy (go) by TMA, gk, gv by TMA stores; 0: plain element accesses
  const void* k;      // [B,T,C] (read directly when tma == 0)
  const void* v;
  const void* g;      // gy, or go with the gate (tma == 0)
};

struct Wkv5StepParams {
  int B, H;
  const __nv_bfloat16* r;  // [B,H,64]
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const float* omega;      // [H,64], or [B,H,64] when omega_per_stream
  int omega_per_stream;    // 1: one decay per stream and head (Finch), 0: per head (Eagle)
  const float* u;          // [H,64]
  __nv_bfloat16* y;        // [B,H,64]
  const float* s_in;       // [B,H,64,64] or null (zero state)
  float* s_out;            // [B,H,64,64]; may equal s_in
};

constexpr int kWkv5MaxSlots = 296;  // Eagle forward CTAs: two per SM of a 148-SM part

struct Wkv5Params {
  int B, T, H;
  const __nv_bfloat16* r;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const float* omega;   // [H,64]
  const float* u;       // [H,64]
  __nv_bfloat16* y;
  const float* s_in;    // [B,H,64,64] or null
  float* s_out;         // [B,H,64,64] or null
  DevCtl* ctl;
  // Slot plan (forward only; nslot = 0: one CTA per head).  The heads' 64-token chunks, laid end
  // to end, are dealt out to nslot CTAs in the order they start: slot s takes chunks
  // [slot_first[s], slot_first[s + 1]).
  int nslot;
  int slot_first[kWkv5MaxSlots + 1];
  float* slot_sum;          // [nslot][256 threads][16]: a slot's last segment from a zero state
  unsigned int* slot_flag;  // [nslot] flags, then the ticket counter; zeroed before the launch
};

struct Wkv6Params {
  int B, T, H;
  const __nv_bfloat16* r;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const float* omega;   // [B,T,H,64]: one decay per token and channel
  const float* u;       // [H,64]
  __nv_bfloat16* y;
  const float* s_in;    // [B,H,64,64] or null
  float* s_out;         // [B,H,64,64] or null
  DevCtl* ctl;
};

// One pass of the Eagle backward (wkv5_bwd.cu): for queries q, keys p (both through TMA maps),
// coefficients c and multipliers m (read directly), the state read with the decay on the output
// channel.  Forward pass: gr, the state checkpoints and the gu sums; reversed pass (time reversed
// inside the kernel, the tensors read and written in their own order, chunks those of the forward
// pass, the first `lead` positions empty): gk and the decay-gradient sums.
struct Wkv5BwdParams {
  int B, T, H;
  int lead;                  // positions the first chunk starts before the sequence (reversed pass)
  const __nv_bfloat16* m;    // [B,T,H,64]: r (forward pass) or k (reversed)
  const __nv_bfloat16* c;    // [B,T,H,64]: k (forward pass) or r (reversed)
  const float* omega;        // [H,64]
  const float* u;            // [H,64]
  const float* x0;           // [B,H,64,64] carried state at the start, or null (zero)
  __nv_bfloat16* out;        // [B,T,H,64]: gr (forward pass) or gk (reversed)
  float* ckpt;               // [B,H,nchunk,64,64] forward states at chunk starts (written / read)
  double* part;              // [B,H,64] per-row sums (gu parts / decay-gradient parts)
  DevCtl* ctl;
};

// Finch backward (wkv6_bwd.cu), chunk-parallel: per 64-token chunk the state and gradient increments
// and the decay product (xs, xg, dec); per (batch row, head) the state entering and the gradient
// leaving every chunk (in place over xs, xg) and gs_in; per chunk gr, gk, gv, gomega and the gu
// parts; the gu parts summed over batch rows and chunks.
struct Wkv6BwdParams {
  int B, T, H;
  const __nv_bfloat16* r;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const __nv_bfloat16* gy;
  const float* omega;    // [B,T,H,64]
  const float* u;        // [H,64]
  const float* s_in;     // [B,H,64,64] or null (zero)
  const float* gs_out;   // [B,H,64,64] or null (zero)
  __nv_bfloat16* gr;
  __nv_bfloat16* gk;
  __nv_bfloat16* gv;
  float* gomega;         // [B,T,H,64]
  float* gu;             // [H,64]
  float* gs_in;          // [B,H,64,64] or null (not wanted)
  float* xs;             // wkv6_bwd_block_floats() floats of workspace
  float* xg;             // wkv6_bwd_block_floats() floats
  float* dec;            // wkv6_bwd_row_floats() floats
  float* part;           // wkv6_bwd_row_floats() floats (gu parts)
};
size_t wkv6_bwd_block_floats(int B, int T, int H);
size_t wkv6_bwd_row_floats(int B, int T, int H);
cudaError_t launch_wkv6_bwd(const Wkv6BwdParams& p, cudaStream_t st);

int fwd_tile_steps();
int fwd_store_steps();
// Stage count of the forward's input pipeline (1 on the plain-access path, which has no pipeline).
int fwd_stages(bool bf16, int seg_len, bool gate = false, bool tma = true);
int bwd_tile_steps();
int bwd_store_steps();
int bwd_stages(bool bf16, int T, bool gate = false, bool tma = true);
// mk, mv: [fwd_tile_steps() x 32] boxes over k, v; my: [fwd_store_steps() x 32] boxes over y
// (TMA stores; any valid map when p.y is null).  With p.tma == 0 the maps are not read (any value).
cudaError_t launch_wkv4_fwd(bool bf16, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& my,
                            const Fwd4Params& p, cudaStream_t st);
// The chunked schedule in one launch (TMA only, every tile of a segment resident in the stages,
// p.start null, p.end the final state written by the last segment, p.lb_* set).
cudaError_t launch_wkv4_fwd_lookback(bool bf16, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& my,
                                     const Fwd4Params& p, cudaStream_t st);
// The receptance-gated forward: also reads r ([fwd_tile_steps() x 32] boxes) and writes σ(r) ⊙ WKV.
cudaError_t launch_wkv4_fwd_gated(bool bf16, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& my,
                                  const CUtensorMap& mr, const Fwd4Params& p, cudaStream_t st);
cudaError_t launch_wkv4_carry(int B, int C, int T, int nseg, int seg_len, const float* w, const float* state_in,
                              float* ws, float* state_out, cudaStream_t st);
// mk, mv, mgy: [bwd_tile_steps() x 32] boxes over k, v, gy; mgk, mgv: [bwd_store_steps() x 32]
// boxes over gk, gv (written by TMA stores).
cudaError_t launch_wkv4_bwd(bool bf16, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mgy,
                            const CUtensorMap& mgk, const CUtensorMap& mgv, const Bwd4Params& p, cudaStream_t st);
// The receptance-gated backward: mo are [bwd_tile_steps() x 32] boxes over go; p.r is read and p.gr
// written with plain coalesced accesses.
cudaError_t launch_wkv4_bwd_gated(bool bf16, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                                  const CUtensorMap& mgk, const CUtensorMap& mgv, const Bwd4Params& p,
                                  cudaStream_t st);
cudaError_t launch_wkv4_reduce_wu(int B, int C, const double* part, float* gw, float* gu, cudaStream_t st);
cudaError_t launch_wkv4_step(bool bf16, int B, int C, const float* w, const float* u, const void* k, const void* v,
                             void* y, const float* state_in, float* state_out, bool vec4, cudaStream_t st);
cudaError_t launch_copy_state(int B, int C, const float* state_in, float* state_out, cudaStream_t st);

// Tensor map over a dense [B, T, C] tensor with boxes of [1, box_t, 32].
bool make_btc_map(CUtensorMap* m, const void* base, bool bf16, int B, int T, int C, int box_t);
// Tensor map over a bf16 [B, T, W] tensor with [1, 64, 64] boxes and the 128-byte swizzle.
bool make_bf16_box64_map(CUtensorMap* m, const void* base, int B, int T, int W);
cudaError_t launch_wkv5_step(const Wkv5StepParams& p, cudaStream_t st);
// reversed: the operator over reversed time on tensors kept in their own order (token t of the
// reversed problem is token T-1-t of r, k, v and y).
cudaError_t launch_wkv5_fwd(const CUtensorMap& mr, const CUtensorMap& mk, const CUtensorMap& mv, const Wkv5Params& p,
                            cudaStream_t st, bool reversed = false);
// mw: [1, 64, 32] fp32 boxes (128-byte swizzle) over omega [B, T, H*64].
cudaError_t launch_wkv6_fwd(const CUtensorMap& mr, const CUtensorMap& mk, const CUtensorMap& mv,
                            const CUtensorMap& mw, const Wkv6Params& p, cudaStream_t st);
// Eagle backward passes (maps over q, p, c: [1, 64, 64] bf16 boxes, 128-byte swizzle) and the batch
// reduction of the passes' per-row sums into gomega and gu.
cudaError_t launch_wkv5_bwd_pass(bool rev, const CUtensorMap& mq, const CUtensorMap& mp, const CUtensorMap& mc,
                                 const Wkv5BwdParams& p, cudaStream_t st);
cudaError_t launch_wkv5_bwd_reduce(int B, int H, const double* part_fwd, const double* part_rev, const float* omega,
                                   float* gomega, float* gu, cudaStream_t st);
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

// Tensor map over an fp32 [B, T, W] tensor with [1, 64, 32] boxes and the 128-byte swizzle.
bool make_f32_box32_map(CUtensorMap* m, const void* base, int B, int T, int W);
// Device address of the library's control block on the current device (null on failure).
DevCtl* device_ctl();

// Sets the dynamic shared-memory limit of `func` once per device.
cudaError_t ensure_smem_attr(const void* func, int bytes, unsigned* device_mask);

// Unique id of the context current on this thread; 0 if there is none or the driver cannot say.
unsigned long long current_context_id();

}  // namespace rwkv
