// The mask of the sliding window with sinks, shared by its forward and
// backward kernels, and their launch parameters.
//
// With i a query row and k a key row of the launch and sh = q_offset - k_offset,
// the pair's distance is t = i + sh - k, and the pair is allowed when
//     t >= 0   and   (t < window   or   k < snk),
// where snk counts the keys of this launch among the sequence's first `sinks`
// positions (sinks - k_offset, clamped to [0, Lk]).
#pragma once
#include "common.cuh"

namespace bss {

struct WindowMask {
  long long sh;        // q_offset - k_offset
  long long window;    // >= 1
  int snk;             // sink keys of this launch
};

struct WindowFwdParams {
  int B, H, Hkv, Lq, Lk;
  float scale_log2;
  WindowMask w;
  __nv_bfloat16* o;    // [B,H,Lq,d]
  float* lse;          // [B,H,Lq]
  int n_items;         // 128-row query tiles of every (b, h)
  int split;           // CTAs of an item (a cluster of them; 1: none)
  int* err;
};

// The key blocks (of 128) a query tile reads: the sink blocks [sb0, sb0 + nsb)
// and the window's blocks [wb0, wb0 + nwb), disjoint and in ascending order.
struct WindowBlocks {
  int nsb, wb0, nwb;
  int sb0;                 // 0, but for a part of a list
  __device__ __forceinline__ int count() const { return nsb + nwb; }
  __device__ __forceinline__ int at(int n) const { return n < nsb ? sb0 + n : wb0 + (n - nsb); }
  // Part `rank` of `split` parts of about as many pairs of blocks each.
  __device__ __forceinline__ WindowBlocks part(int rank, int split) const {
    const int pairs = (count() + 1) / 2;
    const int each = pairs / split, rest = pairs % split;      // (pairs * rank may need more than 32 bits)
    const int b0 = 2 * (each * rank + rest * rank / split);
    const int b1 = min(count(), 2 * (each * (rank + 1) + rest * (rank + 1) / split));
    const int w0 = max(b0 - nsb, 0);
    return WindowBlocks{max(min(b1, nsb) - b0, 0), wb0 + w0, max(b1 - nsb, 0) - w0, b0};
  }
};

// x as an int, where what lies outside [lo, hi] may as well lie on its border.
__device__ __forceinline__ int clamped(long long x, int lo, int hi) {
  return static_cast<int>(max(static_cast<long long>(lo), min(x, static_cast<long long>(hi))));
}

// The keys of a query tile: row r of it sees those from lo + r on up to own + r
// (and sinks).  Limits before the first key or past the last one by more than a
// tile's rows are taken as there: 32 bits do, and the softmax warps' 64-bit
// arithmetic cost 4 %.
struct WindowRows {
  int own, lo;
};
__device__ __forceinline__ WindowRows window_rows(const WindowMask& w, int r0, int Lk) {
  const long long own = static_cast<long long>(r0) + w.sh;
  return WindowRows{clamped(own, -kTileM, Lk), clamped(own - w.window + 1, -kTileM, Lk)};
}

__device__ __forceinline__ WindowBlocks window_blocks(const WindowRows& t, int snk, int rows, int Lk) {
  WindowBlocks b{0, 0, 0, 0};
  const int kmax = min(t.own + rows, Lk) - 1;      // the last row's own key, or the last there is
  if (rows <= 0 || kmax < 0) return b;
  const int lo = max(t.lo, 0);
  const int sink_blocks = (min(snk, kmax + 1) + kTileN - 1) / kTileN;
  if (lo > kmax) {               // the window lies past the last key: sinks alone
    b.nsb = sink_blocks;
    return b;
  }
  b.wb0 = lo / kTileN;
  b.nwb = kmax / kTileN - b.wb0 + 1;
  b.nsb = min(sink_blocks, b.wb0);
  return b;
}

// The lowest n bits (n may lie outside [0, 32]; shl.b32 gives 0 from 32 on).
__device__ __forceinline__ uint32_t bits_below(int n) {
  uint32_t x;
  asm("shl.b32 %0, 1, %1;" : "=r"(x) : "r"(max(n, 0)));
  return x - 1u;
}
// The mask of a launch with Lk keys; false for window < 1 or a negative argument (window_fwd.cu).
bool window_mask(WindowMask* w, int Lk, int64_t window, int64_t sinks, int64_t q_offset,
                 int64_t k_offset);
}  // namespace bss
