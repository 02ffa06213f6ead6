// How the selective scan cuts time into segments: plain arithmetic, used by the host's planning, by the
// kernels and, without CUDA, by its tests.
#pragma once
#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/rwkv_wkv.h"

#ifdef __CUDACC__
#define RWKV_HD __host__ __device__ __forceinline__
#else
#define RWKV_HD inline
#endif

namespace rwkv {

constexpr int kScanSMs = 148;

struct ScanPlan {
  int seg_len = 0, nseg = 1;  // segment s covers tokens s seg_len .. segment_end - 1
};

// The token behind a segment that starts at t0 < T.  The last segment may reach past T, and with T near
// 2^31 past what an int holds, so the length left is compared, not the sum.
RWKV_HD int segment_end(int T, int t0, int seg_len) { return seg_len < T - t0 ? t0 + seg_len : T; }

// The forward's time segments for `tiles` CTAs of a whole sequence.  Cutting time runs nearly every
// exponential twice (the segments' summaries come first), so it pays only where whole-sequence CTAs
// leave much of the GPU idle.  Measured at one batch row, N = 16, bf16, whole / cut in us:
//   8192 tokens: 64 CTAs 378 / 109, 128 379 / 207, 149 387 / 257, 176 396 / 280, 200 397 / 329,
//                225 394 / 360, 256 398 / 401;
//   2048 tokens: 64 CTAs 96 / 32, 128 96 / 59, 149 98 / 71, 200 99 / 83, 225 99 / 91, 256 99 / 102;
//   128 CTAs: 129 tokens 9.0 / 8.8, 160 9.2 / 9.3, 161 10.5 / 9.8, 256 13.6 / 11.8;
//   48 and 64 CTAs: 96 tokens 6.2 / 7.0, 129 8.9 / 7.4, 160 9.1 / 7.8, 161 10.4 / 8.2, 256 13.6 / 8.9.
// The rule's borders, one CTA an SM and five tiles, are on the side of one pass: the times cross near
// 230 CTAs, and for 64 CTAs or fewer between 96 and 129 tokens.  As many segments as give the SMs 8 CTAs
// each.
inline ScanPlan cut_forward(int64_t tiles, int64_t T, int tile, int algo) {
  ScanPlan pl;
  pl.seg_len = (int)std::min<int64_t>((T + tile - 1) / tile * tile, INT_MAX / tile * tile);
  const bool cut = algo == RWKV_ALGO_CHUNKED || (algo == RWKV_ALGO_AUTO && tiles <= kScanSMs && T > 5 * tile);
  if (!cut || T <= tile) return pl;
  const int64_t want = std::max<int64_t>(2, 8 * (int64_t)kScanSMs / std::max<int64_t>(tiles, 1));
  const int64_t len = ((T + want - 1) / want + tile - 1) / tile * tile;
  pl.seg_len = (int)len;
  pl.nseg = (int)((T + len - 1) / len);
  return pl;
}

// The backward's segments: the cost of a plan is the number of turns in which its CTAs pass through
// the SMs times a segment's length and a tile's worth of starting and ending; segments also take a pass
// of their own before (the reversed recurrence, a quarter of the main pass).  Three CTAs an SM are
// counted, which is what N = 16 and 32 hold (72 to 76 KB of shared memory a CTA); with N = 8 and 64 (94 to
// 109 KB) two fit, and the plan counts three all the same.
inline ScanPlan cut_backward(int64_t tiles, int64_t T, int64_t tile) {
  constexpr int64_t kSlots = 3 * kScanSMs;
  ScanPlan best;
  double cost = 1e30;
  int64_t last = 0;
  for (int64_t k = 1; k <= 64; ++k) {
    const int64_t len = ((T + k - 1) / k + tile - 1) / tile * tile;
    if (len == last) continue;  // more segments than whole tiles allow
    last = len;
    const int64_t n = (T + len - 1) / len, turns = (tiles * n + kSlots - 1) / kSlots;
    const double c = (double)turns * (double)(len + tile) * (n > 1 ? 1.25 : 1.0);
    if (c < cost * 0.999) {
      cost = c;
      best.seg_len = (int)std::min<int64_t>(len, INT_MAX / tile * tile);
      best.nseg = (int)n;
    }
  }
  return best;
}

}  // namespace rwkv
