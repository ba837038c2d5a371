// attn_fwd_paged: attention of a chunk of new tokens per sequence over a paged
// key/value cache.
//
// Mathematics: row t of sequence s stands at pos = n - (cu[s+1] - t), n the
// sequence's length; over the keys j <= pos (with a window only those with j >
// pos - window or j < sinks)
//     O = sum_j p_j V_j / l,  p_j = exp(scale q . k_j - m),  l = sum_j p_j,
// kept as the running state (m, l, A) of the online softmax, so that any cut of
// the keys can be joined afterwards: with m* = max m_c,
//     l* = sum_c e^{m_c - m*} l_c,   A* = sum_c e^{m_c - m*} A_c.
//
// What bounds it: with few new tokens a K/V head HBM, which every key and value
// comes from once; with many the tensor pipe.  Both ask for full 128-row tiles:
//   * A tile's rows are the (token, query head) pairs of 128 / G tokens, G the
//     query heads of a K/V head: one box of TMA, and a group's heads share every
//     key that is read.
//   * Its keys are blocks of 128, two at a time: S of a pair by M128 N256 MMAs, S
//     (256 columns) | P | O in tensor memory, P V block by block, as in
//     window_fwd.cu; a block is gathered from its pages by boxes of min(page, 128)
//     rows, a lane of the producer warp each.
//   * The work is cut on the GPU, from the lengths (chunk_plan_kernel): pieces
//     are parts of a tile's keys, of about equal length, and CTAs take them by a
//     counter, longest first (32 sequences of up to 8192, every fourth with 512
//     tokens: 140 us with two kinds of pieces in no order otherwise, 120 so).  A
//     sequence's pieces are numbered so that those that run at the same time share
//     their keys (tiles first, then key parts): L2 serves all but one of them.  Where
//     pieces are whole tiles, or few a CTA, those of the last turn are cut once more
//     (4 x 1000 tokens at 16384: 473 us with all tiles in two parts, 424 with whole
//     ones and the last 132 of 512 in four).  The parts of a tile leave (m, l, A) in
//     the workspace, and a last kernel joins them in order (so the counter does not
//     show in a bit).
//   * e4m3 pages are read as they are.  K stays so: Q, scaled row by row by a power
//     of two (largest element in [128, 256)), is held as two 8-bit parts, e4m3 and
//     the rest in e5m2.  A bf16 element's 8 bits less the first part's 4 leave 3
//     and a sign, which e5m2 holds: the parts are exact down to 2^-13 of a row's
//     largest element, below it off by at most 2^-21 of that.  P has to keep more
//     bits than two such parts could over its range, so V is turned into fp16,
//     exactly, on its way through shared memory, and P carries 2^7 and is rounded
//     to fp16, by 2^-11 (and 2^-32 of a row's largest).  With K turned into fp16,
//     too, the turning took 5800 cycles a pair, twice the MMAs.
//   * Over bf16 pages P is rounded to bf16, V's type: by 2^-8 at most (O is off from 64
//     bits by 2.2e-3 of its rms, by its own rounding alone it would be 1.7e-3).  A
//     second part, as attn_decode_paged has, would need 128 columns of tensor memory,
//     which is full at d=128, and half as many MMAs again, 1024 cycles a pair.
// Rows of the caches that hold no token may hold anything: V's are set to zero in
// shared memory, S's are masked.
//
// Measured (GB300, in a graph, d=128, 16 query heads on 4 K/V heads where not said; of the
// bf16 GEMM's 1929 TFLOP/s): 500 tokens at 8191 45 us; 32 sequences of up to 8192,
// every fourth with 512 tokens 120 us, 51 %; 1024 tokens at 131071, 8 heads of their
// own 376 us, 75 %, and every key from HBM once; 4 x 1000 at 16384 over e4m3 428 us,
// 63 %; d=64, window 1000, 16 heads of their own, 6 x <= 700 62 us.  A pair of blocks
// takes 2900 to 3050 cycles (e4m3 3350) for 2048 of MMAs at their peak rate: the
// softmax warps' 570 for the mask and maximum, 320 to exchange it, 1350 for the
// exponentials (1024 at their unit's rate) and the rest in hand-offs.  Of
// short pieces (d=64 with a window: 6 pairs) their beginning and end, 6000 cycles,
// take a third.  Few rows: plan 4 us, then lengths, table, pages, 2 pairs and O, one
// after the other (8 x 5 tokens of 300: 16.5 us).
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "paged.cuh"
#include "window.cuh"

namespace bss {
namespace {

constexpr int kMaxGroup = 128;             // query heads of a K/V head: rows of a tile
constexpr int kMaxParts = 152 * 8;         // parts that wait to be joined
constexpr int kLeastPairs = 4;             // pairs of key blocks of a part at least

// What the plan leaves for the other kernels.  Pieces of the long kind from `tail`
// on are cut once more, into `fine` each; their parts' slots begin at tail_slot.
struct ChunkPlan {
  int pieces1, pieces;       // of the long kind, in all (before they are cut once more)
  int next;                  // pieces taken, past each CTA's first
  int joins;                 // (tile, K/V head)s that are joined: those of cut sequences, then the tail's pieces
  int tail, fine, tail_slot, tail_join;
};
// Of a sequence, in the order of their pieces' lengths, longest first: pieces, slots
// and joins before it; its number and rows (SeqRows); the parts that its tiles' keys
// are cut into; its tiles; whether its pieces are long ones (1) or others (0).
struct __align__(16) ChunkSeq {
  int before, slot0, join0, s;
  int a, b, n, cuts;
  long long shift;
  int nt, kind;
};

struct ChunkParams {
  const int* table;
  const int* lens;
  const int* cu;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* o;
  float* lse;
  ChunkPlan* plan;
  int* first;                // [ctas] the sequence of each CTA's first piece
  ChunkSeq* seq;             // [S]
  float* part;               // [slots]: A as [d / 4][128 rows][4], m (log2 units) [128], l [128]
  int slots;
  int T, S, H, Hkv, G, tpt, M, P;     // tpt: tokens of a tile
  int page_log2;
  int ctas;
  float scale_log2;
  int window;                // no window: more than any position
  int sinks;
  int* err;
};

// A sequence's new tokens: rows [a, b) of the batch, row t at position t + shift.
struct SeqRows {
  int a, b, n;
  long long shift;
  bool bad;                  // its length is out of range
  bool disorder;             // its offsets do not ascend
};
__device__ __forceinline__ SeqRows seq_rows(const ChunkParams& p, int s) {
  SeqRows r;
  const int c0 = __ldg(p.cu + s), c1 = __ldg(p.cu + s + 1);
  const int len = __ldg(p.lens + s);
  r.a = min(max(c0, 0), p.T);
  r.b = max(r.a, min(c1, p.T));
  const long long most = min(static_cast<long long>(p.M) << p.page_log2, static_cast<long long>(kMaxTokens));
  r.n = static_cast<int>(max(0ll, min(static_cast<long long>(len), most)));
  r.bad = len < 0 || len > most;
  r.disorder = c0 > c1;
  r.shift = static_cast<long long>(r.n) - c1;
  return r;
}
// Tile i of a sequence: rows [t0, t0 + ntok) of the batch, the first at position
// p0 (before the first token: at most 128 before it).
struct Tile {
  int t0, ntok, p0;
};
__device__ __forceinline__ Tile seq_tile(const SeqRows& r, int i, int tpt) {
  Tile t;
  t.t0 = r.a + i * tpt;
  t.ntok = min(tpt, r.b - t.t0);
  t.p0 = clamped(t.t0 + r.shift, -kTileM, kMaxTokens);
  return t;
}
__device__ __forceinline__ WindowBlocks tile_blocks(const ChunkParams& p, const Tile& t, int n) {
  return window_blocks(WindowRows{t.p0, t.p0 - p.window + 1}, min(p.sinks, n), t.ntok, n);
}

// ----------------------------------------------------------------------------
// the plan: one CTA, which the main kernel waits for: what counts is the chain of
// its steps (4 to 6 us with one instruction stream for all lengths of parts, 13 with
// every thread weighing all of them)
// ----------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanCuts = 16;              // lengths of parts that are weighed
constexpr int kPlanSorted = 256;           // sequences that are sorted
struct SeqWork {
  int nt, longest;           // tiles; pairs of key blocks of its longest tile
  float mean;                // ... of a tile
};
__device__ __forceinline__ SeqWork seq_work(const ChunkParams& p, const SeqRows& r) {
  SeqWork w{(r.b - r.a + p.tpt - 1) / p.tpt, 0, 0.f};
  if (w.nt == 0) return w;
  const int last = (tile_blocks(p, seq_tile(r, w.nt - 1, p.tpt), r.n).count() + 1) / 2;
  int first = last;
  if (w.nt > 1) first = (tile_blocks(p, seq_tile(r, 0, p.tpt), r.n).count() + 1) / 2;
  w.longest = max(first, last);
  w.mean = 0.5f * static_cast<float>(first + last);
  return w;
}
// Parts of the tiles of a sequence, where a part has about `len` pairs at most.
__device__ __forceinline__ int seq_cuts(int longest, int len) {
  return longest <= len ? 1 : (longest + len - 1) / len;
}
// ... whether those are long pieces: more than half of it.
__device__ __forceinline__ bool long_pieces(int longest, int cuts, int len) {
  return 2ll * longest > static_cast<long long>(len) * cuts;
}

// Exclusive prefix sums of four numbers a thread over the block's first `warps`
// warps; *total gets the sums.
__device__ __forceinline__ int4 plan_scan(int4 v, int4* warp_sums, int warps, int4* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int4 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int4 y = make_int4(__shfl_up_sync(0xFFFFFFFFu, x.x, o), __shfl_up_sync(0xFFFFFFFFu, x.y, o),
                             __shfl_up_sync(0xFFFFFFFFu, x.z, o), __shfl_up_sync(0xFFFFFFFFu, x.w, o));
    if (lane >= o) x = make_int4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int4 before = make_int4(x.x - v.x, x.y - v.y, x.z - v.z, x.w - v.w), sum = make_int4(0, 0, 0, 0);
  for (int w = 0; w < warps; ++w) {
    const int4 y = warp_sums[w];
    if (w < warp) before = make_int4(before.x + y.x, before.y + y.y, before.z + y.z, before.w + y.w);
    sum = make_int4(sum.x + y.x, sum.y + y.y, sum.z + y.z, sum.w + y.w);
  }
  *total = sum;
  return before;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p) {
  __shared__ float4 sums[kPlanThreads / 32][kPlanCuts];
  __shared__ float2 tops[kPlanThreads / 32];
  __shared__ int4 scan[kPlanThreads / 32];
  __shared__ SeqWork works[kPlanThreads];
  __shared__ float keys[kPlanSorted];
  __shared__ int4 sorted[kPlanSorted];
  __shared__ int chosen, chosen_tail, chosen_fine;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int warps = min(kPlanThreads / 32, (p.S + 31) / 32);         // with a sequence of their own
  const bool few = p.S <= kPlanThreads;                              // `works` holds them all

  // ---- the sequences' rows and work; all pairs, and the longest tile's ----
  // (Where the offsets ascend, no row is two sequences', and no sum below passes T
  // H; where they do not, nothing is done.)
  float2 top = make_float2(0.f, 0.f);
  bool disorder = false;
  SeqRows mine{0, 0, 0, 0, false, false};          // (the last one's: the only one's, of few)
  for (int s = tid; s < p.S; s += kPlanThreads) {
    mine = seq_rows(p, s);
    const SeqWork w = seq_work(p, mine);
    if (mine.bad || mine.disorder) record_error(p.err, ATTN_ERR_BAD_PAGES);
    disorder = disorder || mine.disorder;
    if (few) works[s] = w;
    top.x = fmaxf(top.x, static_cast<float>(w.longest));
    top.y += w.mean * static_cast<float>(w.nt);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top.x = fmaxf(top.x, __shfl_xor_sync(0xFFFFFFFFu, top.x, o));
    top.y += __shfl_xor_sync(0xFFFFFFFFu, top.y, o);
  }
  if (lane == 0) tops[warp] = top;
  if (__syncthreads_or(disorder)) {
    if (tid == 0) *p.plan = ChunkPlan{0, 0, 0, 0, 0, 1, 0, 0};
    return;
  }
  top = tops[0];
  for (int w = 1; w < warps; ++w) {
    top.x = fmaxf(top.x, tops[w].x);
    top.y += tops[w].y;
  }
  const int longest = static_cast<int>(top.x);
  const float ctas = static_cast<float>(p.ctas);
  const float share = top.y * static_cast<float>(p.Hkv) / ctas;      // a CTA's fair share of the pairs

  // ---- what lengths of parts cost: a whole tile, and 2 to 1/9 of the share; a thread
  // weighs one of them for every 64th sequence ----
  const int cand = tid & (kPlanCuts - 1);
  const float turns = 0.5f * exp2f(static_cast<float>(cand - 1) * 0.3f);
  const int whole = max(1, longest);
  const int my_len = cand == 0 ? whole : min(whole, max(kLeastPairs, static_cast<int>(ceilf(share / turns))));
  // long pieces; all pairs, with what a piece costs beside them; the shortest long
  // piece; slots
  float4 v = make_float4(0.f, 0.f, 3.4e38f, 0.f);
  for (int s = tid / kPlanCuts; s < p.S; s += kPlanThreads / kPlanCuts) {
    const SeqWork w = few ? works[s] : seq_work(p, seq_rows(p, s));
    const float tiles = static_cast<float>(w.nt) * static_cast<float>(p.Hkv);
    const int cuts = seq_cuts(w.longest, my_len);
    // about a pair's time to begin and end a piece, as much again to leave a part
    const float beside = cuts > 1 ? 2.f : 1.f;
    v.y += tiles * (w.mean + static_cast<float>(cuts) * beside);
    if (long_pieces(w.longest, cuts, my_len)) {
      v.x += tiles * static_cast<float>(cuts);
      v.z = fminf(v.z, w.mean / static_cast<float>(cuts) + beside);
    }
    if (cuts > 1) v.w += tiles * static_cast<float>(cuts);
  }
  auto add = [](const float4& a, const float4& b) {
    return make_float4(a.x + b.x, a.y + b.y, fminf(a.z, b.z), a.w + b.w);
  };
  v = add(v, make_float4(__shfl_xor_sync(0xFFFFFFFFu, v.x, 16), __shfl_xor_sync(0xFFFFFFFFu, v.y, 16),
                         __shfl_xor_sync(0xFFFFFFFFu, v.z, 16), __shfl_xor_sync(0xFFFFFFFFu, v.w, 16)));
  if (lane < kPlanCuts) sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    const int used = min(kPlanThreads / 32, (p.S + 1) / 2);
    v = sums[0][cand];
    for (int w = 1; w < used; ++w) v = add(v, sums[w][cand]);
    const float each = v.x > 0.f ? v.z : 0.f;
    // everybody's share, where the long pieces' turns do not take longer
    float t = fmaxf(v.y / ctas, ceilf(v.x / ctas) * each);
    // ... or, as the second half of the warp weighs it, the last turn's long pieces and
    // some more cut once more: all CTAs end together but for half a piece of those
    float tail = 0.f, fine = 1.f;
    if (lane >= kPlanCuts) {
      tail = v.x - floorf(v.x / ctas) * ctas;
      if (2.f * tail < ctas) tail += floorf(0.5f * ctas);
      fine = each >= 32.f ? 4.f : each >= 12.f ? 3.f : 2.f;
      t = (v.y + tail * (2.f * fine - 1.f)) / ctas + 0.5f * each / fine;
      v.w += tail * fine;
      if (v.x - tail < ctas || each < 6.f || p.slots == 0) t = 3.4e38f;
    }
    // the join: 5.4 us and 6 ns a part, in the 1.55 us that a pair takes
    t += v.w > 0.f ? 3.5f + 0.004f * v.w : 0.f;
    if (lane > 0 && v.w > static_cast<float>(p.slots)) t = 3.4e38f;
    int best = lane;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float t2 = __shfl_xor_sync(0xFFFFFFFFu, t, o);
      const int b2 = __shfl_xor_sync(0xFFFFFFFFu, best, o);
      if (t2 < t || (t2 == t && b2 < best)) {
        t = t2;
        best = b2;
      }
    }
    if (lane == best) {
      chosen = my_len;
      chosen_tail = static_cast<int>(tail);
      chosen_fine = static_cast<int>(fine);
    }
  }
  __syncthreads();
  const int len = chosen;

  // ---- the sequences in the order of their pieces' lengths, and where each one's
  // pieces, slots and joins begin ----
  auto put = [&](int at, int s, const SeqRows& r, int nt, int cuts, bool is_long) {
    ChunkSeq* q = p.seq + at;
    q->s = s;
    *reinterpret_cast<int4*>(&q->a) = make_int4(r.a, r.b, r.n, cuts);
    q->shift = r.shift;
    q->nt = nt;
    q->kind = is_long;
  };
  auto begin = [&](int at, int before, int slot0, int join0, int pieces) {
    ChunkSeq* q = p.seq + at;
    q->before = before;
    q->slot0 = slot0;
    q->join0 = join0;
    for (int i = before; i < min(before + pieces, p.ctas); ++i) p.first[i] = at;
  };
  int4 base = make_int4(0, 0, 0, 0);         // long pieces (or sequences); pieces, slots, joins
  int pieces1 = 0;
  if (p.S <= kPlanSorted) {
    // a rank each, by comparing with all (long pieces before the others whatever the
    // rounding; ties by number)
    int cuts = 1;
    bool is_long = false;
    SeqWork w{0, 0, 0.f};
    if (tid < p.S) {
      w = works[tid];
      cuts = seq_cuts(w.longest, len);
      is_long = long_pieces(w.longest, cuts, len);
      const float pairs = static_cast<float>(w.longest) / static_cast<float>(cuts);
      keys[tid] = is_long ? pairs : -1.f / (pairs + 1.f);
    }
    __syncthreads();
    if (tid < p.S) {
      const float key = keys[tid];
      int rank = 0;
      for (int i = 0; i < p.S; ++i) rank += keys[i] > key || (keys[i] == key && i < tid);
      put(rank, tid, mine, w.nt, cuts, is_long);
      const int tiles = w.nt * p.Hkv, n = tiles * cuts;
      sorted[rank] = make_int4(is_long ? n : 0, n, cuts > 1 ? n : 0, cuts > 1 ? tiles : 0);
    }
    __syncthreads();
    const int4 x = tid < p.S ? sorted[tid] : make_int4(0, 0, 0, 0);
    const int4 y = plan_scan(x, scan, warps, &base);
    if (tid < p.S) begin(tid, y.y, y.z, y.w, x.y);
    pieces1 = base.x;
  } else {
    // (many: the long ones, then the others)
    for (int kind = 1; kind >= 0; --kind) {
      for (int s0 = 0; s0 < p.S; s0 += kPlanThreads) {
        const int s = s0 + tid;
        int4 x = make_int4(0, 0, 0, 0);
        int cuts = 1;
        SeqRows r{0, 0, 0, 0, false, false};
        SeqWork w{0, 0, 0.f};
        if (s < p.S) {
          r = seq_rows(p, s);
          w = few ? works[s] : seq_work(p, r);
          cuts = seq_cuts(w.longest, len);
          if (long_pieces(w.longest, cuts, len) == (kind == 1)) {
            const int tiles = w.nt * p.Hkv, n = tiles * cuts;
            x = make_int4(1, n, cuts > 1 ? n : 0, cuts > 1 ? tiles : 0);
          }
        }
        int4 total;
        const int4 y = plan_scan(x, scan, warps, &total);
        if (x.x) {
          put(base.x + y.x, s, r, w.nt, cuts, kind == 1);
          begin(base.x + y.x, base.y + y.y, base.z + y.z, base.w + y.w, x.y);
        }
        base = make_int4(base.x + total.x, base.y + total.y, base.z + total.z, base.w + total.w);
      }
      if (kind == 1) pieces1 = base.y;
    }
  }
  if (tid == 0) {
    // (the sums above are exact where a tail is chosen: fewer parts than slots)
    const int tail = min(chosen_tail, pieces1);
    *p.plan = ChunkPlan{pieces1, base.y, 0, base.w + tail, pieces1 - tail, chosen_fine, base.z, base.w};
  }
}

// The last sequence with at most x before it, by a whole warp; `before` of it.
template <class Before>
__device__ __forceinline__ int find_seq(int S, int x, int lane, const Before& before) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const uint32_t yes = __ballot_sync(0xFFFFFFFFu, lane == 0 || (i < hi && before(i) <= x));
    lo += (31 - __clz(yes)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// ----------------------------------------------------------------------------
// the main kernel
// ----------------------------------------------------------------------------
// What the roles need of a piece.
struct Piece {
  int s;                     // its sequence's place in the plan
  int t0, p0;                // its tile's first row and that one's position
  int heads;                 // K/V head << 8 | tokens of the tile
  int slot;                  // -1: the whole tile's keys
  WindowBlocks kb;
  __device__ __forceinline__ int ntok() const { return heads & 255; }
  __device__ __forceinline__ int hkv() const { return heads >> 8; }
};
static_assert(sizeof(Piece) == 36, "two pieces fit beside the tiles");

// ... and the producer: the sequence's length, and the first key that some row of
// the sequence has in its window.
struct Work : Piece {
  int n, low, row;           // (and its row of the table)
};
// Rows of a V block that some row of the sequence sees: [low, rows) and below
// `sinks`, in the groups of 16 that have a page.  What the others hold (rows past
// the last token above all) becomes zeros before a product meets it.
struct BlockRows {
  int rows, low, sinks;
  uint32_t groups;
  __device__ __forceinline__ bool all() const {
    return rows == kTileN && groups == 255u && (low == 0 || sinks >= low);
  }
  __device__ __forceinline__ bool has(int r) const {
    return r < rows && (r >= low || r < sinks) && (groups >> (r >> 4) & 1u);
  }
  __device__ __forceinline__ uint32_t packed() const {
    return static_cast<uint32_t>(rows) << 24 | static_cast<uint32_t>(low) << 16 | static_cast<uint32_t>(sinks) << 8 |
           groups;
  }
};
__device__ __forceinline__ BlockRows block_rows(uint32_t x) {
  return BlockRows{static_cast<int>(x >> 24), static_cast<int>(x >> 16 & 255u), static_cast<int>(x >> 8 & 255u),
                   x & 255u};
}

template <int D, bool FP8>
struct ChunkCfg {
  static constexpr int kChunks = D / 64;                   // 128-byte swizzle atoms across d
  static constexpr int kChunkBytes = kTileM * 128;
  static constexpr int kTileBytes = kTileM * D * 2;
  static constexpr int kRawBytes = kTileM * D;             // 128 rows of e4m3
  static constexpr int kStagesQ = D == 64 ? 2 : 1;
  // K: pairs of blocks, side by side for an N = 256 MMA
  static constexpr int kKBytes = 2 * (FP8 ? kRawBytes : kTileBytes);
  static constexpr int kStagesK = FP8 && D == 64 ? 4 : (D == 64 ? 3 : 2);
  static constexpr int kStagesV = D == 64 ? 4 : 2;
  static constexpr int kStagesR = FP8 ? (D == 64 ? 6 : 4) : 0;
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kStagesQ * kTileBytes;
  static constexpr int kVOff = kKOff + kStagesK * kKBytes;
  static constexpr int kROff = kVOff + kStagesV * kTileBytes;
  static constexpr int kBarOff = kROff + kStagesR * kRawBytes;
  static constexpr int kBarQFull = 0;
  static constexpr int kBarQEmpty = kBarQFull + kStagesQ;
  static constexpr int kBarKFull = kBarQEmpty + kStagesQ;
  static constexpr int kBarKEmpty = kBarKFull + kStagesK;
  static constexpr int kBarVFull = kBarKEmpty + kStagesK;
  static constexpr int kBarVEmpty = kBarVFull + kStagesV;
  static constexpr int kBarSFull = kBarVEmpty + kStagesV;  // a pair's S in TMEM
  static constexpr int kBarSFree = kBarSFull + 1;          // ... read into registers by both warpgroups
  // [2] P of key block X written by warpgroup X; block 0's also waits for
  // warpgroup 1's rescale of its half of O
  static constexpr int kBarPFull = kBarSFree + 1;
  static constexpr int kBarPvDone = kBarPFull + 2;         // [2] a pair's P V of block X completed
  static constexpr int kBarXch = kBarPvDone + 2;           // [2] row values exchanged, by parity
  static constexpr int kBarOFull = kBarXch + 2;            // a piece's last P V completed
  static constexpr int kBarOEmpty = kBarOFull + 1;         // ... O and the row factors read
  static constexpr int kBarLFull = kBarOEmpty + 1;         // a piece's row factors written
  static constexpr int kBarWant = kBarLFull + 1;           // the next piece may be chosen
  static constexpr int kBarPieceFull = kBarWant + 1;       // [2] a piece's description written
  static constexpr int kBarPieceEmpty = kBarPieceFull + 2; // [2] ... read by every role
  // [stages] bf16: a V block that wants cleaning has landed (VFull: it is clean); e4m3: Q has
  static constexpr int kBarLand = kBarPieceEmpty + 2;
  static constexpr int kLands = FP8 ? kStagesQ : kStagesV;
  static constexpr int kBarRFull = kBarLand + kLands;      // e4m3's V tiles: landed
  static constexpr int kBarREmpty = kBarRFull + kStagesR;  // ... converted
  static constexpr int kReqs = FP8 ? 0 : 8;                // V blocks to be cleaned: at most the stages', and the end
  static constexpr int kBarReq = kBarREmpty + kStagesR;
  static constexpr int kNumBars = kBarReq + kReqs;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kTmemSlotOff = kMiscOff;
  static constexpr int kAbortOff = kMiscOff + 4;
  // [kRing] which groups of 16 keys of a pair have a page; a pair's entry is
  // written when its K is asked for, and read before its S is given back: at
  // most the K stages, and one, lie between
  static constexpr int kRing = D == 64 ? 8 : 4;
  static_assert(kRing > kStagesK + 1, "a pair's entry is read before it is written again");
  static constexpr int kValidOff = kMiscOff + 8;
  static constexpr int kInfoOff = kValidOff + kRing * 2;           // [stages] BlockRows of a V block that has landed
  static constexpr int kReqOff = kInfoOff + (FP8 ? kStagesR : kStagesV) * 4;   // [requests] stages
  static constexpr int kPieceOff = kReqOff + kReqs * 4;
  static constexpr int kUpOff = kPieceOff + 2 * static_cast<int>(sizeof(Piece));  // exponents of Q's factors
  static constexpr int kXchOff = (kUpOff + (FP8 ? kTileM : 0) + 15) / 16 * 16;
  static constexpr int kInvOff = kXchOff + 2 * 2 * kTileM * 4;
  static constexpr int kSmemBytes = kInvOff + kTileM * 4;
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(kBarOff % 8 == 0 && kInfoOff % 4 == 0, "alignment");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;      // S: 256 fp32 columns (key block X at 128 X)
  static constexpr uint32_t kColP = 256;    // P: 256 keys, 16-bit pairs (block X at 256 + 64 X)
  static constexpr uint32_t kColO = 384;    // O: D fp32 columns
  static constexpr int kThreads = 512;
  static constexpr int kPartFloats = kTileM * (D + 2);
};

// Register split per warpgroup (setmaxnreg): output and conversion (warps 0-3),
// softmax (4-7, 8-11), K and Q, MMA, pieces and V (12 to 15).
// (Output 48 and producers 80, O by 16 columns: bf16 1 to 3 % slower, e4m3 1 % faster.)
constexpr uint32_t kChunkOut = 64;
constexpr uint32_t kChunkSoft = 192;
constexpr uint32_t kChunkLow = 64;
constexpr uint32_t kChunkLaunchRegs = 128;
static_assert(kChunkOut + 2 * kChunkSoft + kChunkLow <= 4 * kChunkLaunchRegs, "register split exceeds the launch");
// Pairs of a piece that are left when the next one is chosen (32 mixed sequences: 3
// 120.2 us, 6 120.0, 10 122, 20 129).
constexpr int kWantPairs = 6;
constexpr float kP2 = 7.f;                  // e4m3: P carries 2^7

// kind::f16 with fp16 operands, kind::f8f6f4 with e4m3 ones: formats 0 (A in e5m2:
// kAIsE5m2, format 1 in bits 7-9).
constexpr uint32_t kAIsE5m2 = 1u << 7;
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[smem desc] * B[smem desc], 32 8-bit elements deep
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Shared-memory matrix descriptor of rows of 64 bytes with the 64-byte swizzle
// (mode 4): 8 rows are 512 bytes.
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr) {
  return (sdesc_sw128(saddr, 16, 512) & ~(static_cast<uint64_t>(7) << 61)) | static_cast<uint64_t>(4) << 61;
}
// One thread of a converged warp, and the compiler knows it: an MMA's operands are
// the warp's, and behind `lane == 0` each MMA's code has to find whose they are (23
// KB of code for the MMA thread instead of 15: 1024 tokens at 131071 412 us, so 378).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0u;
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {     // to L2
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// x and y in e4m3 (the low 16 bits) and what that leaves of them in e5m2 (the high).
__device__ __forceinline__ uint32_t two_parts(float x, float y) {
  uint32_t h, a, b;
  asm("{\n\t.reg .b16 q;\n\tcvt.rn.satfinite.e4m3x2.f32 q, %3, %2;\n\tcvt.u32.u16 %0, q;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
      : "=r"(a), "=r"(h) : "f"(x), "f"(y));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  asm("{\n\t.reg .b16 q;\n\tcvt.rn.satfinite.e5m2x2.f32 q, %2, %1;\n\tcvt.u32.u16 %0, q;\n\t}"
      : "=r"(b) : "f"(x - f.x), "f"(y - f.y));
  return a | b << 16;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <int D, bool FP8>
__global__ void __launch_bounds__(512, 1)
    attn_fwd_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const ChunkParams p) {
  using C = ChunkCfg<D, FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {                      // the swizzle needs it: report, touch nothing
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) record_error(p.err, ATTN_ERR_UNSUPPORTED);
    return;
  }
  auto bar = [&](int i) { return sbase + C::kBarOff + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kTmemSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbortOff);
  volatile uint16_t* valid_ring = reinterpret_cast<volatile uint16_t*>(smem + C::kValidOff);
  volatile uint32_t* block_info = reinterpret_cast<volatile uint32_t*>(smem + C::kInfoOff);
  const float NEG_INF = -__int_as_float(0x7f800000);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int tid = static_cast<int>(threadIdx.x);
  const int status = status_at_entry(p.err);

  if (tid == 0) {
    for (int s = 0; s < C::kStagesQ; ++s) {
      mbar_init(bar(C::kBarQFull + s), FP8 ? kTileM : 1);
      mbar_init(bar(C::kBarQEmpty + s), 1);
    }
    for (int s = 0; s < C::kStagesK; ++s) {
      mbar_init(bar(C::kBarKFull + s), 1);
      mbar_init(bar(C::kBarKEmpty + s), 1);
    }
    for (int s = 0; s < C::kStagesV; ++s) {
      mbar_init(bar(C::kBarVFull + s), FP8 ? kTileM : 4);        // (bf16: a clean block's copy counts for four warps)
      mbar_init(bar(C::kBarVEmpty + s), 1);
    }
    for (int s = 0; s < C::kLands; ++s) mbar_init(bar(C::kBarLand + s), 1);
    for (int s = 0; s < C::kReqs; ++s) mbar_init(bar(C::kBarReq + s), 1);
    for (int s = 0; s < C::kStagesR; ++s) {
      mbar_init(bar(C::kBarRFull + s), 1);
      mbar_init(bar(C::kBarREmpty + s), kTileM);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(C::kBarXch + s), 2 * 4 * 32);
      mbar_init(bar(C::kBarPvDone + s), 1);
      mbar_init(bar(C::kBarPieceFull + s), 1);
      mbar_init(bar(C::kBarPieceEmpty + s), 3 + 2 * 4 + 4);      // the warps that read it: K, V, MMA, softmax, output
    }
    mbar_init(bar(C::kBarSFull), 1);
    mbar_init(bar(C::kBarSFree), 2 * 4 * 32);
    mbar_init(bar(C::kBarPFull + 0), 2 * 4 * 32);
    mbar_init(bar(C::kBarPFull + 1), 4 * 32);
    mbar_init(bar(C::kBarOFull), 1);
    mbar_init(bar(C::kBarOEmpty), 4 * 32);
    mbar_init(bar(C::kBarLFull), 4 * 32);
    mbar_init(bar(C::kBarWant), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(sbase + C::kTmemSlotOff, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool gave_up = __syncthreads_or(status == ATTN_ERR_TIMEOUT);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the plan is there, and all before it (who gives up waits, too: the join reads
  // the plan when this kernel has ended)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (gave_up) {
    if (warp == 0) {
      __syncwarp();
      tmem_dealloc(tmem, C::kTmemCols);
    }
    return;
  }

  // A role's next piece (slot `i & 1` of the ring holds piece i); false at the end
  // or when a wait ran out.  `whole`: all lanes of a warp ask.
  auto piece_slot = [&](int i) { return reinterpret_cast<volatile Piece*>(smem + C::kPieceOff) + (i & 1); };
  auto read_piece = [&](int i, Piece& x) {
    const volatile Piece* src = piece_slot(i);
    x.s = src->s;
    x.t0 = src->t0;
    x.p0 = src->p0;
    x.heads = src->heads;
    x.slot = src->slot;
    x.kb.nsb = src->kb.nsb;
    x.kb.wb0 = src->kb.wb0;
    x.kb.nwb = src->kb.nwb;
    x.kb.sb0 = src->kb.sb0;
  };

  if (warp >= 12) {
    regs_set<kChunkLow, kChunkLaunchRegs>();
    if (warp == 12 || warp == 15) {
      // =================== TMA producers: K and Q (warp 12), V (warp 15) ===================
      // Two warps, for V has no time to lose at d=128: with two stages a block can be
      // asked for when the one two before it has been used, and is wanted 2200 cycles
      // later.  What one warp had to do for K and V between that and the copy cost up
      // to a third of everything (1024 tokens at 131071, at the time: 413 to 540 us).  So
      // all that a copy needs is computed before the wait for its stage.
      const bool is_v = warp == 15;
      const CUtensorMap* map = is_v ? &tmV : &tmK;
      if (lane == 0) {
        tma_prefetch_desc(map);
        if (!is_v) tma_prefetch_desc(&tmQ);
      }
      const int page = 1 << p.page_log2;
      const int br = min(page, kTileN);                    // rows of a box
      const int subs = kTileN / br;                        // boxes of a block, a chunk of d each
      constexpr int kAcross = FP8 ? 1 : C::kChunks;
      const int c_of = lane % kAcross;
      const int sub = lane / kAcross % subs;
      const int t_of = lane / kAcross / subs;              // block of the pair (2 and more: none)
      const uint32_t box_bytes = static_cast<uint32_t>(br) * (FP8 ? D : 128);
      int used = 0;                  // K stages, V tiles or raw tiles filled (over all pieces)
      int qn = 0, np = 0, reqs = 0;
      auto wait = [&](int b, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, wait_bar(bar(b), parity, abort_flag, p.err));
      };
      // bf16: V stage s has to be cleaned when it has landed (-1: no more of this piece)
      auto request = [&](int s) {
        if (lane == 0) {
          reinterpret_cast<volatile int*>(smem + C::kReqOff)[reqs % max(1, C::kReqs)] = s;
          mbar_arrive(bar(C::kBarReq + reqs % max(1, C::kReqs)));
        }
        ++reqs;
      };
      // The next piece, with what the producers alone need of it; false at the end
      // (or where the wait ran out).
      auto next_piece = [&](Work& x) -> bool {
        if (!wait(C::kBarPieceFull + (np & 1), (np >> 1) & 1)) return false;
        read_piece(np, x);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarPieceEmpty + (np & 1)));
        ++np;
        if (x.kb.count() == 0) return false;
        const ChunkSeq* q = p.seq + x.s;
        x.n = q->n;
        x.row = q->s;
        x.low = clamped(q->a + q->shift - p.window + 1, 0, x.n);
        return true;
      };
      // This lane's box of a pair of key blocks: its page (-1: none is copied).
      struct Box {
        int page, key;               // page, first key
        bool seen;                   // a page that some row of the piece sees
      };
      auto fetch = [&](const Work& x, int k) {
        Box b{-1, 0, false};
        if (t_of < 2 && 2 * k + t_of < x.kb.count()) {
          b.key = x.kb.at(2 * k + t_of) * kTileN + sub * br;
          if (b.key < x.n) {
            b.page = __ldg(p.table + static_cast<size_t>(x.row) * p.M + (b.key >> p.page_log2));
            const int last = b.key + br - 1;
            b.seen = b.key <= x.p0 + x.ntok() - 1 && (last > x.p0 - p.window || b.key < p.sinks);
          }
        }
        return b;
      };
      // The copies of a pair; `b` was fetched a pair before.
      auto load = [&](const Work& x, int k, const Box& b) -> bool {
        const bool mine = b.page >= 0 && b.page < p.P;
        if (!mine && b.seen && !is_v) record_error(p.err, ATTN_ERR_BAD_PAGES);
        // of the pair's 16 groups of 16 keys, those with a page
        const uint32_t ok = __reduce_or_sync(
            0xFFFFFFFFu, mine ? ((1u << (br / 16)) - 1u) << (t_of * 8 + sub * (br / 16)) : 0u);
        const uint32_t boxes = __ballot_sync(0xFFFFFFFFu, mine);
        const int row = (x.hkv() << p.page_log2) + (b.key & (page - 1));
        if (!is_v) {
          const int s = used % C::kStagesK;
          const uint32_t at = sbase + C::kKOff + s * C::kKBytes +
                              (FP8 ? t_of * C::kRawBytes + sub * br * D
                                   : (c_of * 2 + t_of) * C::kChunkBytes + sub * br * 128);
          const uint32_t bytes = __popc(boxes) * box_bytes;
          const bool fine = used < C::kStagesK || wait_bar(bar(C::kBarKEmpty + s), ((used / C::kStagesK) & 1) ^ 1,
                                                           abort_flag, p.err);
          // the copies first; the warp agrees on the wait afterwards (bytes may arrive
          // before they are expected: the phase waits for the arrival)
          if (fine && mine) tma_load_3d(at, map, bar(C::kBarKFull + s), c_of * 64, row, b.page);
          if (lane == 0) {
            valid_ring[used % C::kRing] = static_cast<uint16_t>(ok);
            mbar_arrive_expect_tx(bar(C::kBarKFull + s), bytes);
          }
          ++used;
          return __all_sync(0xFFFFFFFFu, fine);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (2 * k + t >= x.kb.count()) break;
          const int k0 = x.kb.at(2 * k + t) * kTileN;
          const BlockRows rows{min(kTileN, x.n - k0), max(0, min(x.low - k0, kTileN)),
                               max(0, min(p.sinks - k0, kTileN)), ok >> (8 * t) & 255u};
          constexpr int kStages = FP8 ? C::kStagesR : C::kStagesV;
          const int s = used % kStages;
          const bool clean = FP8 || rows.all();
          const int full = (FP8 ? C::kBarRFull : clean ? C::kBarVFull : C::kBarLand) + s;
          const int empty = (FP8 ? C::kBarREmpty : C::kBarVEmpty) + s;
          const uint32_t at = sbase + (FP8 ? C::kROff + s * C::kRawBytes + sub * br * D
                                           : C::kVOff + s * C::kTileBytes + c_of * C::kChunkBytes + sub * br * 128);
          const bool go = mine && t_of == t;
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, go)) * box_bytes;
          const bool fine = used < kStages || wait_bar(bar(empty), ((used / kStages) & 1) ^ 1, abort_flag, p.err);
          if (fine && go) tma_load_3d(at, map, bar(full), c_of * 64, row, b.page);
          if (lane == 0) {
            block_info[s] = rows.packed();
            mbar_arrive_expect_tx(bar(full), bytes);
            if (!FP8 && clean) mbar_arrive_n(bar(full), 3);
          }
          ++used;
          if (!__all_sync(0xFFFFFFFFu, fine)) return false;
          if (!clean) request(s);
        }
        return true;
      };
      auto load_q = [&](const Piece& x) -> bool {
        const int s = qn % C::kStagesQ;
        // the last S that read this Q buffer must have completed
        if (qn >= C::kStagesQ && !wait(C::kBarQEmpty + s, ((qn / C::kStagesQ) & 1) ^ 1)) return false;
        if (lane == 0) {
          const int full = (FP8 ? C::kBarLand : C::kBarQFull) + s;
          mbar_arrive_expect_tx(bar(full), static_cast<uint32_t>(C::kChunks * 128 * p.G * p.tpt));
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(sbase + C::kQOff + s * C::kTileBytes + c * C::kChunkBytes, &tmQ, bar(full), c * 64,
                        x.hkv() * p.G, x.t0);
        }
        __syncwarp();
        ++qn;
        return true;
      };

      Work x;
      bool ok = true;
      while (ok && next_piece(x)) {
        const int ns = (x.kb.count() + 1) / 2;
        const bool q_first = !is_v && np == 1;             // (later ones wait for the piece before)
        if (q_first) ok = load_q(x);
        Box now = fetch(x, 0);
        for (int k = 0; k < ns && ok; ++k) {
          if (!is_v && k == max(0, ns - kWantPairs) && lane == 0) mbar_arrive(bar(C::kBarWant));
          const Box then = fetch(x, k + 1);
          ok = load(x, k, now);
          if (k == 0 && !is_v && !q_first && ok) ok = load_q(x);
          now = then;
        }
        if (!FP8 && is_v) request(-1);
      }
      // every copy issued has landed before the CTA may exit
      const int stages = !is_v ? C::kStagesK : FP8 ? C::kStagesR : C::kStagesV;
      const int full = !is_v ? C::kBarKFull : FP8 ? C::kBarRFull : C::kBarVFull;
      for (int j = max(0, used - stages); j < used; ++j) drain_bar(bar(full + j % stages), (j / stages) & 1);
      for (int j = max(0, qn - C::kStagesQ); j < qn; ++j)
        drain_bar(bar((FP8 ? C::kBarLand : C::kBarQFull) + j % C::kStagesQ), (j / C::kStagesQ) & 1);
    } else if (warp == 13) {
      // =================== MMA issuer (one thread) ===================
      // For every pair: S of the next pair (of the next piece at a piece's end),
      // as soon as both softmax warpgroups hold this pair's S in registers, then
      // this pair's P V.
      if (elect_one()) {
        constexpr uint32_t kIdescS = FP8 ? idesc_f32(kTileM, 2 * kTileN, false)
                                         : idesc_bf16_f32(kTileM, 2 * kTileN, false, false);
        constexpr uint32_t kIdescS1 = FP8 ? idesc_f32(kTileM, kTileN, false)
                                          : idesc_bf16_f32(kTileM, kTileN, false, false);   // a block alone
        constexpr uint32_t kIdescPV = FP8 ? idesc_f32(kTileM, D, true) : idesc_bf16_f32(kTileM, D, false, true);
        int ik = 0, iv = 0;     // K stages and V tiles consumed
        int qn = 0;             // Q tiles consumed
        int sn = 0;             // S tiles issued
        int pn = 0;             // P tiles consumed
        int on = 0;             // O results handed to the output warps
        int np = 0;             // pieces read
        // S of pair k of a piece with nb blocks
        auto issue_s = [&](int k, int nb) -> bool {
          if (k == 0) {
            if (!wait_bar(bar(C::kBarQFull + qn % C::kStagesQ), (qn / C::kStagesQ) & 1, abort_flag, p.err))
              return false;
            ++qn;
          }
          if (sn > 0 && !wait_bar(bar(C::kBarSFree), (sn - 1) & 1, abort_flag, p.err)) return false;
          const int qs = (qn - 1) % C::kStagesQ;
          const uint64_t dq = sdesc_sw128(sbase + C::kQOff + qs * C::kTileBytes, 16, 1024);
          const int s = ik % C::kStagesK;
          if (!wait_bar(bar(C::kBarKFull + s), (ik / C::kStagesK) & 1, abort_flag, p.err)) return false;
          tc_fence_after();
          const uint32_t idesc = 2 * k + 1 < nb ? kIdescS : kIdescS1;
          const uint32_t ks = sbase + C::kKOff + s * C::kKBytes;
          if constexpr (FP8) {
            // Q's parts: 32 bytes each, side by side
            const uint64_t dk = D == 128 ? sdesc_sw128(ks, 16, 1024) : sdesc_sw64(ks);
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int kk = 0; kk < D / 32; ++kk)
                mma_ss_f8(tmem + C::kColS, sdesc_add(dq, (kk >> 1) * C::kChunkBytes + (kk & 1) * 64 + part * 32),
                          sdesc_add(dk, kk * 32), part == 0 ? idesc : idesc | kAIsE5m2, part > 0 || kk > 0 ? 1u : 0u);
          } else {
            const uint64_t dk = sdesc_sw128(ks, 16, 1024);
#pragma unroll 2
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t qoff = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
              const uint32_t koff = (kk >> 2) * 2 * C::kChunkBytes + (kk & 3) * 32;
              mma_ss(tmem + C::kColS, sdesc_add(dq, qoff), sdesc_add(dk, koff), idesc, kk > 0 ? 1u : 0u);
            }
          }
          mma_commit(bar(C::kBarKEmpty + s));
          ++ik;
          mma_commit(bar(C::kBarSFull));
          if (2 * k + 2 >= nb) mma_commit(bar(C::kBarQEmpty + qs));   // Q's buffer is free for a later piece
          ++sn;
          return true;
        };
        // P V block by block: block X's MMAs go as soon as warpgroup X has
        // written its P, and their completion frees that block's P columns
        auto issue_pv = [&](int k, int nb) -> bool {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!wait_bar(bar(C::kBarPFull + t), pn & 1, abort_flag, p.err)) return false;
            tc_fence_after();
            if (t == 0 && k == 0 && on > 0) {
              // O still holds the previous piece's result until the output warps read it
              if (!wait_bar(bar(C::kBarOEmpty), (on - 1) & 1, abort_flag, p.err)) return false;
              tc_fence_after();
            }
            if (2 * k + t < nb) {
              const int s = iv % C::kStagesV;
              if (!wait_bar(bar(C::kBarVFull + s), (iv / C::kStagesV) & 1, abort_flag, p.err)) return false;
              tc_fence_after();
              const uint64_t dv = sdesc_sw128(sbase + C::kVOff + s * C::kTileBytes, C::kChunkBytes, 1024);
#pragma unroll 2
              for (int kk = 0; kk < kTileN / 16; ++kk)
                mma_ts(tmem + C::kColO, tmem + C::kColP + (t * 8 + kk) * 8, sdesc_add(dv, kk * 16 * 128),
                       kIdescPV, (k > 0 || t > 0 || kk > 0) ? 1u : 0u);
              mma_commit(bar(C::kBarVEmpty + s));
              ++iv;
            }
            mma_commit(bar(C::kBarPvDone + t));
          }
          ++pn;
          return true;
        };
        // blocks of the next piece (0: none is left)
        auto next_blocks = [&](int& nb) -> bool {
          if (!wait_bar(bar(C::kBarPieceFull + (np & 1)), (np >> 1) & 1, abort_flag, p.err)) return false;
          const volatile Piece* x = piece_slot(np);
          nb = x->kb.nsb + x->kb.nwb;
          mbar_arrive(bar(C::kBarPieceEmpty + (np & 1)));
          ++np;
          return true;
        };
        int nb = 0;
        bool ok = next_blocks(nb) && (nb == 0 || issue_s(0, nb));
        while (ok && nb > 0) {
          int nb2 = 0;
          const int ns = (nb + 1) / 2;
          for (int k = 0; k < ns && ok; ++k) {
            if (k + 1 < ns) ok = issue_s(k + 1, nb);
            else if (!FP8) ok = next_blocks(nb2) && (nb2 == 0 || issue_s(0, nb2));
            if (ok) ok = issue_pv(k, nb);
          }
          if (!ok) break;
          mma_commit(bar(C::kBarOFull));
          ++on;
          // e4m3: the next Q has to be turned, too, which this piece's last V is not to
          // wait for
          if (FP8) ok = next_blocks(nb2) && (nb2 == 0 || issue_s(0, nb2));
          nb = nb2;
        }
        // every MMA issued has completed before tensor memory is released (one phase
        // more of a barrier that nobody waits for by now)
        mma_commit(bar(C::kBarPvDone + 1));
        drain_bar(bar(C::kBarPvDone + 1), pn & 1);
      }
    } else if (warp == 14) {
      // =================== pieces (a whole warp) ===================
      const ChunkPlan plan = *p.plan;
      const int tail = plan.pieces1 - plan.tail;           // pieces that are cut once more
      const int total1 = plan.tail + tail * plan.fine, total = total1 + plan.pieces - plan.pieces1;
      int np = 0;
      // The next piece that has keys; pieces without are seen to here.
      int taken = static_cast<int>(blockIdx.x);
      bool begun = false;
      auto next_piece = [&](Piece& x) -> bool {
        while (true) {
          if (begun && lane == 0) taken = static_cast<int>(gridDim.x) + atomicAdd(&p.plan->next, 1);
          const int index = __shfl_sync(0xFFFFFFFFu, taken, 0);
          if (index < 0 || index >= total) return false;
          // the piece, and which of its cuts (each for all pieces in turn)
          const bool is_long = index < total1;
          const int over = index - plan.tail;
          const int sub = is_long && over >= 0 ? over / tail : 0;
          const int piece = is_long ? index - sub * tail : index - (total1 - plan.pieces1);
          int s;
          if (!begun) s = p.first[index];
          else s = find_seq(p.S, piece, lane, [&](int i) { return p.seq[i].before; });
          begun = true;
          const ChunkSeq q = p.seq[s];
          const int in = piece - q.before;
          // tiles first (the last ones, which see most keys, lead), then parts, then heads
          const int u = in / q.nt, hkv = u / q.cuts;
          int cut = u - hkv * q.cuts, cuts = q.cuts;
          const SeqRows r{q.a, q.b, q.n, q.shift, false, false};
          const Tile t = seq_tile(r, q.nt - 1 - (in - u * q.nt), p.tpt);
          x.s = s;
          x.t0 = t.t0;
          x.p0 = t.p0;
          x.heads = hkv << 8 | t.ntok;
          x.slot = cuts > 1 ? q.slot0 + in : -1;
          if (is_long && over >= 0) {
            cut = cut * plan.fine + sub;
            cuts *= plan.fine;
            x.slot = plan.tail_slot + (piece - plan.tail) * plan.fine + sub;
          }
          x.kb = tile_blocks(p, t, r.n).part(cut, cuts);
          if (t.p0 < 0 && lane == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
          if (x.kb.count() > 0) return true;
          if (x.slot >= 0) {                               // a part without keys
            float* l = p.part + static_cast<size_t>(x.slot) * C::kPartFloats + kTileM * (D + 1);
#pragma unroll 1
            for (int i = lane; i < kTileM; i += 32) l[i] = 0.f;
          } else {                                         // rows that see nothing
#pragma unroll 1
            for (int i = 0; i < x.ntok(); ++i) {
              const size_t row = static_cast<size_t>(x.t0 + i) * p.H + x.hkv() * p.G;
#pragma unroll 1
              for (int e = lane; e < p.G * (D / 8); e += 32)
                reinterpret_cast<uint4*>(p.o + row * D)[e] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
              for (int g = lane; g < p.G; g += 32) p.lse[row + g] = NEG_INF;
            }
          }
        }
      };
      // Hand a piece (or, with no key blocks, the end) to the other roles.
      auto publish = [&](const Piece& x) -> bool {
        if (np >= 2 && !__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarPieceEmpty + (np & 1)), ((np >> 1) & 1) ^ 1,
                                                         abort_flag, p.err)))
          return false;
        if (lane == 0) {
          volatile Piece* dst = piece_slot(np);
          dst->s = x.s;
          dst->t0 = x.t0;
          dst->p0 = x.p0;
          dst->heads = x.heads;
          dst->slot = x.slot;
          dst->kb.nsb = x.kb.nsb;
          dst->kb.wb0 = x.kb.wb0;
          dst->kb.nwb = x.kb.nwb;
          dst->kb.sb0 = x.kb.sb0;
          mbar_arrive(bar(C::kBarPieceFull + (np & 1)));
          // its Q is wanted when the piece before it has had its last S, and not earlier
          if (x.kb.count() > 0) {
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c) prefetch_3d(&tmQ, c * 64, x.hkv() * p.G, x.t0);
          }
        }
        ++np;
        return true;
      };

      // A piece is chosen late, when few pairs of the one before it are left to be
      // asked for: chosen a piece ahead, the last ones waited behind others while
      // CTAs had nothing to do (1024 tokens at 131071, at the time: 557 us, so 425).
      Piece x;
      bool more = true;
      while (more) {
        if (np > 0 && !__all_sync(0xFFFFFFFFu, wait_bar_relaxed(bar(C::kBarWant), (np - 1) & 1, abort_flag, p.err)))
          break;
        more = next_piece(x);
        if (!more) x.kb = WindowBlocks{0, 0, 0, 0};
        if (!publish(x)) break;
      }
    }
  } else if (warp < 4) {
    regs_set<kChunkOut, kChunkLaunchRegs>();
    // =================== output (and e4m3's conversion): thread = row ===================
    const int row = warp * 32 + lane;
    const int tok = row / p.G, head = row - tok * p.G;
    const uint32_t tO = tmem + (static_cast<uint32_t>(warp * 32) << 16) + C::kColO;
    const volatile float* inv_s = reinterpret_cast<const volatile float*>(smem + C::kInvOff);
    int on = 0;             // O results read
    int np = 0;             // pieces read
    auto wait = [&](int b, uint32_t parity) -> bool {
      return __all_sync(0xFFFFFFFFu, wait_bar_relaxed(bar(b), parity, abort_flag, p.err));
    };
    auto next_piece = [&](Piece& x) -> bool {
      if (!wait(C::kBarPieceFull + (np & 1), (np >> 1) & 1)) return false;
      read_piece(np, x);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::kBarPieceEmpty + (np & 1)));
      ++np;
      return x.kb.count() > 0;
    };
    // the piece's O: scaled and rounded, or as it is to its part
    auto output = [&](const Piece& x) -> bool {
      if (!wait(C::kBarLFull, on & 1)) return false;
      const float inv = inv_s[row];
      if (!wait(C::kBarOFull, on & 1)) return false;
      tc_fence_after();
      const bool inb = tok < x.ntok();
      const size_t at = static_cast<size_t>(x.t0 + tok) * p.H + x.hkv() * p.G + head;
      uint4* dst = reinterpret_cast<uint4*>(p.o + at * D);
      float4* part = reinterpret_cast<float4*>(p.part + static_cast<size_t>(max(x.slot, 0)) * C::kPartFloats) + row;
      // 32 columns at a time (the warpgroup has few registers); a row without a
      // key (inv = 0) is 0 whatever the masked keys held
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_ld_wait(o);
        if (c == D / 32 - 1) {
          tc_fence_before();
          mbar_arrive(bar(C::kBarOEmpty));      // the next piece's P V may overwrite O
        }
        if (!inb) continue;
        if (x.slot >= 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            part[(8 * c + e) * kTileM] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                     __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            o[e] = inv == 0.f ? 0u : pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[4 * c + e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      ++on;
      return true;
    };
    if constexpr (!FP8) {
      // V blocks with rows that no row of the sequence sees are handed on when those
      // are zeros.  (A piece's first P V waits for these warps anyway: it overwrites
      // the O that they read.)
      uint32_t phases = 0;           // of the stages' landings
      int reqs = 0;
      auto clean = [&]() -> bool {
        for (;; ++reqs) {
          if (!wait(C::kBarReq + reqs % C::kReqs, (reqs / C::kReqs) & 1)) return false;
          const int s = reinterpret_cast<volatile int*>(smem + C::kReqOff)[reqs % C::kReqs];
          if (s < 0) break;
          if (!wait(C::kBarLand + s, (phases >> s) & 1u)) return false;
          phases ^= 1u << s;
          if (!block_rows(block_info[s]).has(row)) {
            const uint32_t at = sbase + C::kVOff + s * C::kTileBytes + row * 128;
#pragma unroll
            for (int u = 0; u < D / 8; ++u) sts128(at + (u >> 3) * C::kChunkBytes + (u & 7) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kBarVFull + s));
        }
        ++reqs;
        return true;
      };
      Piece x;
      while (next_piece(x) && clean() && output(x)) {
      }
    } else {
      int ir = 0, iv = 0, qn = 0;
      // the next raw tile becomes fp16 tile `dst`, its row `row` by this thread
      // (rows without a token become zeros), once that tile is free
      auto convert = [&](uint32_t dst, int full, int empty, bool used, uint32_t parity) -> bool {
        const int s = ir % C::kStagesR;
        if (!wait(C::kBarRFull + s, (ir / C::kStagesR) & 1)) return false;
        if (used && !wait(empty, parity)) return false;
        const uint32_t src = sbase + C::kROff + s * C::kRawBytes + row * D;
        const uint32_t to = dst + row * 128;
        if (block_rows(block_info[s]).has(row)) {
#pragma unroll
          for (int u0 = 0; u0 < D / 16; u0 += 4) {
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)               // 16 elements each
              w[i] = lds128(src + ((D == 128 ? (u0 + i) ^ (row & 7) : (u0 + i) ^ ((row >> 1) & 3)) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int u = u0 + i, u2 = (2 * u) & 7;
              const uint32_t at = to + (u >> 2) * C::kChunkBytes;
              sts128(at + ((u2 ^ (row & 7)) << 4), e4m3x2_f16x2(w[i].x), e4m3x2_f16x2(w[i].x >> 16),
                     e4m3x2_f16x2(w[i].y), e4m3x2_f16x2(w[i].y >> 16));
              sts128(at + (((u2 + 1) ^ (row & 7)) << 4), e4m3x2_f16x2(w[i].z), e4m3x2_f16x2(w[i].z >> 16),
                     e4m3x2_f16x2(w[i].w), e4m3x2_f16x2(w[i].w >> 16));
            }
          }
        } else {
#pragma unroll 4
          for (int u = 0; u < D / 8; ++u) sts128(to + (u >> 3) * C::kChunkBytes + (u & 7) * 16, 0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(full));
        mbar_arrive(bar(C::kBarREmpty + s));
        ++ir;
        return true;
      };
      auto convert_v = [&](const Piece& x, int k) -> bool {
        for (int t = 0; t < 2 && 2 * k + t < x.kb.count(); ++t) {
          const int s = iv % C::kStagesV;
          if (!convert(sbase + C::kVOff + s * C::kTileBytes, C::kBarVFull + s, C::kBarVEmpty + s,
                       iv >= C::kStagesV, ((iv / C::kStagesV) & 1) ^ 1))
            return false;
          ++iv;
        }
        return true;
      };
      // this thread's row of Q, in place: bf16 to two 8-bit parts, by a power of two
      // that puts its largest element in [128, 256)
      auto convert_q = [&]() -> bool {
        const int s = qn % C::kStagesQ;
        if (!wait(C::kBarLand + s, (qn / C::kStagesQ) & 1)) return false;
        // the softmax has read the previous piece's factors
        if (qn > 0 && !wait(C::kBarPieceEmpty + ((qn - 1) & 1), ((qn - 1) >> 1) & 1)) return false;
        const uint32_t at = sbase + C::kQOff + s * C::kTileBytes + row * 128;
        auto unit = [&](int c, int u) { return at + c * C::kChunkBytes + ((u ^ (row & 7)) << 4); };
        float top = 0.f;
#pragma unroll 4
        for (int u = 0; u < D / 8; ++u) {
          const uint4 w = lds128(unit(u >> 3, u & 7));
          top = fmax3(top, fabsf(bf16lo(w.x)), fabsf(bf16hi(w.x)));
          top = fmax3(top, fabsf(bf16lo(w.y)), fabsf(bf16hi(w.y)));
          top = fmax3(top, fabsf(bf16lo(w.z)), fabsf(bf16hi(w.z)));
          top = fmax3(top, fabsf(bf16lo(w.w)), fabsf(bf16hi(w.w)));
        }
        // 2^(134 - e) for a top of exponent field e, kept a normal number; a row
        // with an infinity becomes NaN, as its scores would be
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        const int field = top == 0.f ? 127 : max(1, min(253, 127 + 134 - e));
        const float up = e == 255 ? __int_as_float(0x7fffffff) : __uint_as_float(static_cast<uint32_t>(field) << 23);
        // 32 elements, which an MMA takes, and their parts have the same 64 bytes (one
        // turn of a loop: this runs once a piece, and what it takes is reading its code)
#pragma unroll 1
        for (int g = 0; g < D / 32; ++g) {
          uint32_t a[8], b[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 w = lds128(unit(g >> 1, (g & 1) * 4 + i));
            const uint32_t x0 = two_parts(bf16lo(w.x) * up, bf16hi(w.x) * up);
            const uint32_t x1 = two_parts(bf16lo(w.y) * up, bf16hi(w.y) * up);
            const uint32_t x2 = two_parts(bf16lo(w.z) * up, bf16hi(w.z) * up);
            const uint32_t x3 = two_parts(bf16lo(w.w) * up, bf16hi(w.w) * up);
            a[2 * i] = __byte_perm(x0, x1, 0x5410);
            b[2 * i] = __byte_perm(x0, x1, 0x7632);
            a[2 * i + 1] = __byte_perm(x2, x3, 0x5410);
            b[2 * i + 1] = __byte_perm(x2, x3, 0x7632);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sts128(unit(g >> 1, (g & 1) * 4 + i), a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
            sts128(unit(g >> 1, (g & 1) * 4 + 2 + i), b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
          }
        }
        *reinterpret_cast<volatile uint8_t*>(smem + C::kUpOff + row) = static_cast<uint8_t>(field);
        fence_proxy_async_smem();
        mbar_arrive(bar(C::kBarQFull + s));
        ++qn;
        return true;
      };
      // (a piece's last V before the next one's Q: the MMAs come in that order)
      Piece x, y;
      bool more = next_piece(x);
      bool ok = !more || convert_q();
      while (ok && more) {
        const int ns = (x.kb.count() + 1) / 2;
        for (int k = 0; k < ns && ok; ++k) ok = convert_v(x, k);
        if (!ok) break;
        more = next_piece(y);
        ok = (!more || convert_q()) && output(x);
        x = y;
      }
    }
  } else {
    regs_set<kChunkSoft, kChunkLaunchRegs>();
    // =================== softmax warpgroups: X = 0 (warps 4-7), 1 (warps 8-11) ===================
    const int X = (warp - 4) >> 2;                // key block X of every pair
    const int wq = warp & 3;                      // TMEM lane quarter of this warp
    const int row_in_tile = wq * 32 + lane;
    const int tok = row_in_tile / p.G;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + C::kColS + X * 128;
    const uint32_t tP = tmem + lane_base + C::kColP + X * 64;
    const uint32_t tO = tmem + lane_base + C::kColO + X * (D / 2);
    float* xch = reinterpret_cast<float*>(smem + C::kXchOff);
    float* inv_s = reinterpret_cast<float*>(smem + C::kInvOff);

    int cnt = 0;        // S tiles consumed (over all pieces)
    int nx = 0;         // row values exchanged
    int on = 0;         // pieces finished
    bool ok = true;
    // hand this row's value to the other warpgroup and take its value back
    auto exchange = [&](float v, float& other) -> bool {
      float* xb = xch + (nx & 1) * 2 * kTileM;
      xb[X * kTileM + row_in_tile] = v;
      mbar_arrive(bar(C::kBarXch + (nx & 1)));
      const bool w = __all_sync(0xFFFFFFFFu,
                                wait_bar(bar(C::kBarXch + (nx & 1)), (nx >> 1) & 1, abort_flag, p.err));
      other = xb[(1 - X) * kTileM + row_in_tile];
      ++nx;
      return w;
    };
    for (int np = 0;; ++np) {
      if (!__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarPieceFull + (np & 1)), (np >> 1) & 1, abort_flag, p.err)))
        break;
      Piece x;
      read_piece(np, x);
      const int nb = x.kb.count();
      // (e4m3: given back with the first S, when Q's factors have been read, too)
      if (!FP8 || nb == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarPieceEmpty + (np & 1)));
      }
      if (nb == 0) break;                         // the end
      const int ns = (nb + 1) / 2;
      const int own = x.p0 + tok;                 // this row's own key, and the first its window holds
      const int low = own - p.window + 1;
      const int low_last = x.p0 + x.ntok() - p.window;
      float sl2 = p.scale_log2;
      if constexpr (FP8) sl2 *= __ldg(p.k_scale + x.hkv());
      float m2 = NEG_INF;     // reference max (log2 units), moved only by > 8
      float l = 0.f;          // this warpgroup's part of the row sum
      for (int k = 0; k < ns; ++k) {
        const bool none = 2 * k + X >= nb;        // the pair's second block is missing
        const int kstart = none ? 0 : x.kb.at(2 * k + X) * kTileN;
        if (!__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarSFull), cnt & 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
        if constexpr (FP8) {
          if (k == 0) {                           // Q's factor, written before this S was
            const uint32_t f = *reinterpret_cast<volatile uint8_t*>(smem + C::kUpOff + row_in_tile);
            sl2 *= __uint_as_float((254u - f) << 23);
            if (sl2 == 0.f) sl2 = __uint_as_float(1u);    // 0 times a masked score would be a NaN
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarPieceEmpty + (np & 1)));
          }
        }
        const uint32_t valid = (valid_ring[cnt % C::kRing] >> (8 * X)) & 255u;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
        // S is in registers: the next pair's S may overwrite its columns
        tc_fence_before();
        mbar_arrive(bar(C::kBarSFree));

        // element mask, 32 columns at a time: a bit for each allowed key of this
        // row (j <= own, which is before the last key; j >= low: window; j < sinks;
        // and the key has a page)
        const bool edge = none || valid != 255u || kTileN - 1 > x.p0 - kstart ||
                          (low_last - kstart > 0 && kstart + kTileN > p.sinks);
        if (edge) {
          const int jhi = none ? -1 : own - kstart;
          const int jlo = low - kstart;
          const int js = p.sinks - kstart;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t bits = bits_below(jhi + 1 - 32 * c) & (~bits_below(jlo - 32 * c) | bits_below(js - 32 * c));
            bits &= (valid >> (2 * c) & 1u ? 0x0000FFFFu : 0u) | (valid >> (2 * c) & 2u ? 0xFFFF0000u : 0u);
            if (!__all_sync(0xFFFFFFFFu, bits == 0xFFFFFFFFu)) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((bits >> j) & 1u)) s[c][j] = __float_as_uint(NEG_INF);
            }
          }
        }
        // row max of this block over 8 chains of three-input max
        float mx[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = __uint_as_float(s[0][u]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = (c == 0 ? 8 : 0); j < 32; j += 16)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              if (j + 8 + u < 32)
                mx[u] = fmax3(mx[u], __uint_as_float(s[c][j + u]), __uint_as_float(s[c][j + 8 + u]));
              else
                mx[u] = fmaxf(mx[u], __uint_as_float(s[c][j + u]));
        const float mmine = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                  fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sl2;
        // the pair's row max: both warpgroups take the same decisions below
        float mothr;
        if (!exchange(mmine, mothr)) {
          ok = false;
          break;
        }
        const float mblk = fmaxf(mmine, mothr);
        float alpha = 1.f;
        bool moved = false;
        if (mblk > m2 + 8.f) {
          alpha = ex2(m2 - mblk);
          m2 = mblk;
          moved = true;
        }
        const float mu = ((m2 == NEG_INF) ? 0.f : m2) - (FP8 ? kP2 : 0.f);
        // Where the reference max moved, this warpgroup's half of O is
        // rescaled: after the previous pair's whole P V (both blocks write
        // all of O).  Warpgroup 1 does it first and then releases block 0's
        // P V; warpgroup 0 after writing its P, before releasing it.
        const bool fix = moved && k > 0;
        const bool any_fix = __any_sync(0xFFFFFFFFu, fix);
        auto rescale_o = [&]() -> bool {
          if (!__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarPvDone + 1), (cnt - 1) & 1, abort_flag, p.err)))
            return false;
          tc_fence_after();
          const float a = fix ? alpha : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
            tmem_st32(tO + c * 32, o);
          }
          return true;
        };
        if (X == 1) {
          if (any_fix && !rescale_o()) {
            ok = false;
            break;
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(C::kBarPFull + 0));
        }
        // P block X is written below: the previous pair's P V of block X
        // (which reads it) must have completed
        if (cnt > 0 &&
            !__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarPvDone + X), (cnt - 1) & 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float rs[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) rs[u] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
            const int c = half * 2 + c2;
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              float x0, x1;
              ffma2(x0, x1, __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]), sl2, sl2, -mu,
                    -mu);
              const float p0 = ex2(x0);
              const float p1 = ex2(x1);
              const int u = (j >> 1) & 3;
              fadd2(rs[2 * u], rs[2 * u + 1], rs[2 * u], rs[2 * u + 1], p0, p1);
              pk[c2 * 16 + j / 2] = FP8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
            }
          }
          tmem_st32(tP + half * 32, pk);
        }
        l = l * alpha + (((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7])));
        if (X == 0 && any_fix && !rescale_o()) {
          ok = false;
          break;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(C::kBarPFull + X));
        ++cnt;
      }
      if (!ok) break;

      // ---- the row sum is the two warpgroups' parts; warpgroup 0 hands its
      // inverse to the output warps, which must have read the previous piece's
      float lo;
      if (!exchange(l, lo)) break;
      if (X == 0) {
        if (on > 0 &&
            !__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarOEmpty), (on - 1) & 1, abort_flag, p.err)))
          break;
        // a row that saw no key has l = 0; a NaN score makes l NaN and goes through
        const float lt = l + lo;
        const float m = FP8 ? m2 - kP2 : m2;      // the max that goes with l
        float vs = 1.f;
        if constexpr (FP8) vs = __ldg(p.v_scale + x.hkv());
        inv_s[row_in_tile] = lt == 0.f ? 0.f : vs / lt;
        mbar_arrive(bar(C::kBarLFull));
        if (tok < x.ntok()) {
          if (x.slot >= 0) {
            float* part = p.part + static_cast<size_t>(x.slot) * C::kPartFloats + kTileM * D + row_in_tile;
            part[0] = m;
            part[kTileM] = lt;
          } else {
            p.lse[static_cast<size_t>(x.t0 + tok) * p.H + x.hkv() * p.G + row_in_tile - tok * p.G] =
                lt == 0.f ? NEG_INF : (m + __log2f(lt)) * kLn2;
          }
        }
      }
      ++on;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ----------------------------------------------------------------------------
// the join: a CTA a (tile, K/V head) and 16 columns, a thread a row and 8 of them
// ----------------------------------------------------------------------------
constexpr int kJoinThreads = 2 * kTileM;
template <int D, bool FP8>
__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const ChunkParams p) {
  constexpr int kPart = kTileM * (D + 2);
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int row = static_cast<int>(threadIdx.x) & (kTileM - 1);
  const int col = static_cast<int>(blockIdx.y) * 16 + static_cast<int>(threadIdx.x >> 7) * 8;
  const int tok = row / p.G;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the parts are complete
  const ChunkPlan plan = *p.plan;
  if (static_cast<int>(blockIdx.x) >= plan.joins) return;
  // (a launch that gave up left parts unwritten)
  if (__syncthreads_or(status_at_entry(p.err) == ATTN_ERR_TIMEOUT)) return;
  for (int j = static_cast<int>(blockIdx.x); j < plan.joins; j += static_cast<int>(gridDim.x)) {
    // a tile of a sequence whose tiles are cut; or a piece of the tail (a tile), if its
    // sequence's are not
    const bool whole = j >= plan.tail_join;
    const int piece = plan.tail + j - plan.tail_join;
    const int s = whole ? find_seq(p.S, piece, lane, [&](int i) { return p.seq[i].before; })
                        : find_seq(p.S, j, lane, [&](int i) { return p.seq[i].join0; });
    const ChunkSeq q = p.seq[s];
    if (whole && q.cuts > 1) continue;
    const SeqRows r{q.a, q.b, q.n, q.shift, false, false};
    const int nt = q.nt;
    const int in = whole ? piece - q.before : j - q.join0;
    const int hkv = in / nt, i = in % nt;                 // the tile's number among its pieces'
    const Tile t = seq_tile(r, nt - 1 - i, p.tpt);
    // its pieces are numbers first, first + nt ..: `plain` of them have one part, those in
    // the tail `fine` each
    const int first = hkv * q.cuts * nt + i;
    const int plain = q.kind == 0 ? q.cuts : max(0, min(q.cuts, (plan.tail - q.before - first + nt - 1) / nt));
    if (tok >= t.ntok) continue;
    float m = NEG_INF, l = 0.f, y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = 0.f;
    // parts `slot`, slot + step .. are added, four's loads in flight together (past the
    // last one the last is read again, and not counted)
    auto add = [&](int slot, int step, int parts) {
      constexpr int kBatch = 4;
      for (int c0 = 0; c0 < parts; c0 += kBatch) {
        float lc[kBatch], mc[kBatch];
        float4 v[kBatch][2];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const float* x = p.part + static_cast<size_t>(slot + min(c0 + u, parts - 1) * step) * kPart;
          mc[u] = x[kTileM * D + row];
          lc[u] = c0 + u < parts ? x[kTileM * (D + 1) + row] : 0.f;
          const float4* a = reinterpret_cast<const float4*>(x) + col / 4 * kTileM + row;
          v[u][0] = a[0];
          v[u][1] = a[kTileM];
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) top = lc[u] != 0.f ? fmaxf(top, mc[u]) : top;
        if (top != m) {                                   // (at first: from -inf, 0 stays 0)
          const float w = ex2(m - top);
          l *= w;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= w;
          m = top;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          if (lc[u] == 0.f) continue;                     // this part saw no key
          const float w = ex2(mc[u] - m);
          l = fmaf(w, lc[u], l);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            y[4 * e] = fmaf(w, v[u][e].x, y[4 * e]);
            y[4 * e + 1] = fmaf(w, v[u][e].y, y[4 * e + 1]);
            y[4 * e + 2] = fmaf(w, v[u][e].z, y[4 * e + 2]);
            y[4 * e + 3] = fmaf(w, v[u][e].w, y[4 * e + 3]);
          }
        }
      }
    };
    add(q.slot0 + first, nt, plain);
    for (int c = plain; c < q.cuts; ++c)
      add(plan.tail_slot + (q.before + first + c * nt - plan.tail) * plan.fine, 1, plan.fine);
    float inv = l == 0.f ? 0.f : 1.f / l;
    if constexpr (FP8) inv *= __ldg(p.v_scale + hkv);
    const size_t at = static_cast<size_t>(t.t0 + tok) * p.H + hkv * p.G + row - tok * p.G;
    uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + col);
    *dst = make_uint4(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv),
                      pack_bf16(y[4] * inv, y[5] * inv), pack_bf16(y[6] * inv, y[7] * inv));
    if (col == 0) p.lse[at] = l == 0.f ? NEG_INF : (m + __log2f(l)) * kLn2;
  }
}

// ----------------------------------------------------------------------------
// host
// ----------------------------------------------------------------------------
bool chunk_sizes(int T, int S, int H, int Hkv, int d, int max_pages, int page) {
  if (T < 1 || S < 1 || S > kMaxSeqs || max_pages < 1) return false;
  if (!valid_page_size(page) || !valid_kv_heads(H, Hkv) || H / Hkv > kMaxGroup) return false;
  return (d == 64 || d == 128) && static_cast<long long>(T) * H <= 0x7FFFFFFFll;
}

// Tiles of all sequences at most, of one K/V head.
long long most_tiles(int T, int S, int G) {
  const int tpt = kTileM / G;
  return std::min<long long>(T, (static_cast<long long>(T) + tpt - 1) / tpt + S);
}
// Parts that the plan may leave to be joined: none where no tile has enough keys
// for two of them.
int most_slots(int T, int S, int Hkv, int G, int M, int page) {
  const long long keys = std::min<long long>(static_cast<long long>(M) * page, kMaxTokens);
  const long long pairs = (keys + 2 * kTileN - 1) / (2 * kTileN) + 1;      // (a window and its sinks: one more)
  if (pairs <= kLeastPairs) return 0;
  const long long cuts = (pairs + kLeastPairs - 1) / kLeastPairs;
  const long long tiles = most_tiles(T, S, G) * Hkv;
  return static_cast<int>(tiles >= kMaxParts ? kMaxParts : std::min<long long>(kMaxParts, tiles * cuts));
}
// plan | first pieces | sequences | parts
constexpr int kMaxSms = 256;
size_t chunk_workspace(int T, int S, int H, int Hkv, int d, int M, int page) {
  return up256(sizeof(ChunkPlan)) + kMaxSms * 4 + up256(static_cast<size_t>(S) * sizeof(ChunkSeq)) +
         static_cast<size_t>(most_slots(T, S, Hkv, H / Hkv, M, page)) * kTileM * (d + 2) * 4;
}

// The kernels' attributes, set once a device; its multiprocessors.
template <int D, bool FP8>
cudaError_t chunk_device(int* sms) {
  constexpr int kMaxDev = 64;
  static int known[kMaxDev] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev] == 0) {
    const void* k = reinterpret_cast<const void*>(attn_fwd_paged_kernel<D, FP8>);
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, k)) != cudaSuccess) return e;
    if (fa.numRegs < static_cast<int>(kChunkLaunchRegs)) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkCfg<D, FP8>::kSmemBytes);
    if (e != cudaSuccess) return e;
    int n = 0;
    if ((e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    known[dev] = std::min(n, kMaxSms);
  }
  *sms = known[dev];
  return cudaSuccess;
}

template <int D, bool FP8>
cudaError_t launch_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, ChunkParams& p,
                         cudaStream_t st) {
  int sms = 0;
  cudaError_t e = chunk_device<D, FP8>(&sms);
  if (e != cudaSuccess) return e;
  const long long pieces = std::max<long long>(most_tiles(p.T, p.S, p.G) * p.Hkv, p.slots);
  p.ctas = static_cast<int>(std::min<long long>(sms, pieces));
  chunk_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the next kernels are set up while the ones before them run; they wait for
  // their ends themselves
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
  cfg.blockDim = dim3(ChunkCfg<D, FP8>::kThreads);
  cfg.dynamicSmemBytes = ChunkCfg<D, FP8>::kSmemBytes;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, attn_fwd_paged_kernel<D, FP8>, tq, tk, tv, p)) != cudaSuccess) return e;
  if (p.slots == 0) return cudaSuccess;
  // (a tile and 16 columns a CTA, as many tiles at a time as there are multiprocessors:
  // what is joined is known on the device alone, and 4576 CTAs that find nothing took
  // 4.4 us)
  const long long joins = std::min<long long>(p.slots / 2, most_tiles(p.T, p.S, p.G) * p.Hkv);
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(joins, sms)), D / 16);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D, FP8>, p);
}

}  // namespace
}  // namespace bss

using namespace bss;

extern "C" size_t attn_fwd_paged_workspace_bytes(int T, int S, int H, int H_kv, int d, int max_pages,
                                                 int page_size) {
  if (!chunk_sizes(T, S, H, H_kv, d, max_pages, page_size)) return 0;
  return chunk_workspace(T, S, H, H_kv, d, max_pages, page_size);
}

extern "C" attn_status_t attn_fwd_paged(
    const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int64_t k_page_stride,
    int64_t v_page_stride, int kv_dtype, const float* k_scale, const float* v_scale,
    const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_q, void* o, float* lse,
    void* workspace, size_t workspace_bytes, int T, int S, int H, int H_kv, int d, int max_pages,
    int n_pages, int page_size, float scale, int64_t window, int64_t sinks, void* stream) {
  // (the sequences' rows are the batch's: one "batch" of T rows)
  attn_status_t s = check_common(1, H, T, 1, d, scale);
  if (s != ATTN_OK) return s;
  if (S < 1) return ATTN_ERR_INVALID_ARG;
  if (!valid_kv_heads(H, H_kv)) return ATTN_ERR_INVALID_ARG;
  if (max_pages < 1 || n_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (!valid_page_size(page_size) || S > kMaxSeqs) return ATTN_ERR_UNSUPPORTED;
  if (kv_dtype != ATTN_KV_BF16 && kv_dtype != ATTN_KV_E4M3) return ATTN_ERR_UNSUPPORTED;
  if (window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return ATTN_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == ATTN_KV_E4M3;
  if (fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr) || !aligned4(k_scale) || !aligned4(v_scale))
    return ATTN_ERR_INVALID_ARG;
  const int64_t least = static_cast<int64_t>(H_kv) * page_size * d;
  const int64_t unit = fp8 ? 16 : 8;
  if (k_page_stride < least || v_page_stride < least || k_page_stride % unit || v_page_stride % unit)
    return ATTN_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(H) * d || q_stride % 8) return ATTN_ERR_INVALID_ARG;
  if (T == 0) return ATTN_OK;
  if (!chunk_sizes(T, S, H, H_kv, d, max_pages, page_size)) return ATTN_ERR_UNSUPPORTED;
  const void* ptrs16[] = {q, k_cache, v_cache, o, workspace};
  for (const void* ptr : ptrs16)
    if (!ptr || !aligned16(ptr)) return ATTN_ERR_INVALID_ARG;
  const void* ptrs4[] = {page_table, seq_lens, cu_q, lse};
  for (const void* ptr : ptrs4)
    if (!ptr || !aligned4(ptr)) return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < chunk_workspace(T, S, H, H_kv, d, max_pages, page_size)) return ATTN_ERR_WORKSPACE;
  ChunkParams p{};
  if ((s = status_word(&p.err)) != ATTN_OK) return s;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.lens = seq_lens;
  p.cu = cu_q;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.T = T;
  p.S = S;
  p.H = H;
  p.Hkv = H_kv;
  p.G = H / H_kv;
  p.M = max_pages;
  p.P = n_pages;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.tpt = kTileM / p.G;
  p.slots = most_slots(T, S, H_kv, p.G, max_pages, page_size);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.plan = reinterpret_cast<ChunkPlan*>(ws);
  ws += up256(sizeof(ChunkPlan));
  p.first = reinterpret_cast<int*>(ws);
  ws += kMaxSms * 4;
  p.seq = reinterpret_cast<ChunkSeq*>(ws);
  ws += up256(static_cast<size_t>(S) * sizeof(ChunkSeq));
  p.part = reinterpret_cast<float*>(ws);
  p.scale_log2 = scale * kLog2e;
  // no position reaches kMaxTokens
  p.window = window == 0 ? kMaxTokens : static_cast<int>(std::min<int64_t>(window, kMaxTokens));
  p.sinks = static_cast<int>(std::min<int64_t>(sinks, kMaxTokens));
  if ((s = get_encoder()) != ATTN_OK) return s;
  const long long rows = static_cast<long long>(H_kv) * page_size;
  if (rows > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;     // a copy's row is an int
  CUtensorMap tq, tk, tv;
  // Q as (d, H, T), a box the query heads of a K/V head of a tile's tokens
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(H), static_cast<uint64_t>(T)};
  const uint64_t strides[2] = {static_cast<uint64_t>(d) * 2, static_cast<uint64_t>(q_stride) * 2};
  const uint32_t boxes[3] = {64, static_cast<uint32_t>(p.G), static_cast<uint32_t>(p.tpt)};
  if ((s = make_map_tiled(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, boxes,
                          CU_TENSOR_MAP_SWIZZLE_128B)) != ATTN_OK)
    return s;
  const size_t item = fp8 ? 1 : 2;
  const int box_rows = std::min(page_size, kTileN);
  if ((s = cache_map(&tk, k_cache, d, fp8, rows, n_pages, static_cast<size_t>(k_page_stride) * item, box_rows)) !=
      ATTN_OK)
    return s;
  if ((s = cache_map(&tv, v_cache, d, fp8, rows, n_pages, static_cast<size_t>(v_page_stride) * item, box_rows)) !=
      ATTN_OK)
    return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (d == 64) e = fp8 ? launch_chunk<64, true>(tq, tk, tv, p, st) : launch_chunk<64, false>(tq, tk, tv, p, st);
  else e = fp8 ? launch_chunk<128, true>(tq, tk, tv, p, st) : launch_chunk<128, false>(tq, tk, tv, p, st);
  return cuda_status("attn_fwd_paged launch", e);
}
