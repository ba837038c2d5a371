// attn_fwd_window: softmax attention in which a query sees the last `window`
// positions up to its own and the sequence's first `sinks` positions.
//
// Mathematics (window.cuh has the mask): O_i = sum_j P_ij V_j with
// P_ij = exp(scale q_i . k_j - LSE_i) over the allowed keys j, LSE_i the log
// of their sum; a row that sees no key gets O = 0, LSE = -inf.
//
// One work item is a 128-row query tile.  Its keys are the sink blocks and the
// window's blocks (128 keys each), disjoint and ascending, taken two at a time
// (an odd last block alone): S of a pair by M128 N256 MMAs (about 170 cycles
// each against 105 for an N=128 one, with every SM issuing), S (256 columns) |
// P | O in tensor memory, P V block by block.
//
// Items are short (a window of 1024 keys is 5 pairs), so what decides is that
// nothing stops between them.  The CTAs are persistent and take items by a
// fixed stride (the items of a window are alike), so every role knows the next
// item; four kinds of warps each run ahead over the items:
//   TMA     K of the next pair, at an item's end the next item's first pair
//           and its Q tile, then V;
//   MMA     S of the next pair, or of the next item's first one, before P V of
//           this one;
//   softmax two warpgroups, one per block of the pair, which exchange their
//           rows' maxima through shared memory; they go on to the next item's
//           S as soon as P is written;
//   output  a warpgroup that waits for the item's last P V, scales and stores
//           O while the softmax works on the next item.
// With the softmax warps writing O themselves an item of one pair took 12000
// cycles and every further pair 3100: 410 us for B2 H16(4) L16384 d128, window
// 1024, sinks 4.  So it takes 287 us in a graph (290 to 293 called from Python):
// 930 TFLOP/s of allowed pairs, 1160 of executed blocks (61 % of a large bf16
// product's).  An item's 20400 cycles are
// 14300 of MMAs (5 pairs); a plain step takes 3300, the two masked ones 1200
// and 600 more (with 64-bit limits in every row 1600 and 900: 310 us), an
// item's end 1300, and the next item's Q comes late, after the last S has freed
// its buffer (shared memory holds one at d=128; prefetching it into L2 made
// everything 3 to 5 % slower).
//
// Where a launch has few items, a cluster of CTAs shares one (window_split).
//
// The element mask is applied in the blocks that the diagonal, the window's
// lower edge or the last sink crosses; all others run without it.
//
// P is rounded to bf16, V's type, which one tcgen05.mma wants of both operands
// (its rest as a second product would add half of an item's MMAs): O is 1.9e-3
// off in norm, of which its own rounding is 1.65e-3.
#include <algorithm>
#include <mutex>

#include "host.cuh"
#include "window.cuh"

namespace bss {
namespace {

constexpr int kMostSplit = 4;      // CTAs that share an item at most

template <int D>
struct WinCfg {
  static constexpr int kChunks = D / 64;                   // 128-byte swizzle atoms across d
  static constexpr int kChunkBytes = kTileM * 128;         // 128 rows x 64 d
  static constexpr int kTileBytes = kTileM * D * 2;        // one 128-row tile
  static constexpr int kPairBytes = 2 * kTileBytes;        // two key blocks
  // 224 KB of tiles at d=128; at d=64 every ring has a stage more
  static constexpr int kStagesQ = D == 64 ? 2 : 1;
  static constexpr int kStagesK = D == 64 ? 3 : 2;         // key-block pairs
  static constexpr int kStagesV = D == 64 ? 4 : 2;         // V tiles
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kStagesQ * kTileBytes;
  static constexpr int kVOff = kKOff + kStagesK * kPairBytes;
  static constexpr int kBarOff = kVOff + kStagesV * kTileBytes;
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
  static constexpr int kBarOFull = kBarXch + 2;            // an item's last P V completed
  static constexpr int kBarOEmpty = kBarOFull + 1;         // ... O and the row factors read
  static constexpr int kBarLFull = kBarOEmpty + 1;         // an item's row factors 1 / l written
  static constexpr int kBarMmaDone = kBarLFull + 1;
  static constexpr int kNumBars = kBarMmaDone + 1;
  // TMEM base | abort flag
  static constexpr int kMiscOff = kBarOff + ((kNumBars + 1) / 2) * 16;
  static constexpr int kTmemSlotOff = kMiscOff;
  static constexpr int kAbortOff = kMiscOff + 4;
  // exchanged row values: [parity][warpgroup][128 rows] fp32
  static constexpr int kXchOff = kMiscOff + 16;
  static constexpr int kInvOff = kXchOff + 2 * 2 * kTileM * 4;   // 1 / l of an item's rows
  static constexpr int kPayload = kInvOff + kTileM * 4;
  // alignment slack: at d=128 less than 1024 bytes are left, and the kernel
  // checks that the dynamic shared memory base leaves room
  static constexpr int kSlack = kPayload + 1024 <= 232448 ? 1024 : 232448 - kPayload;
  static constexpr int kSmemBytes = kPayload + kSlack;
  static_assert(kSlack >= 256, "too little alignment slack");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0;      // S: 256 fp32 columns (key block X at 128 X)
  static constexpr uint32_t kColP = 256;    // P: 256 keys, bf16 pairs (block X at 256 + 64 X)
  static constexpr uint32_t kColO = 384;    // O: D fp32 columns
  static constexpr int kThreads = 512;
  // Split items: when an item's last S is done, its K ring takes the rows'
  // statistics (m, l) and then the other CTAs' parts of this CTA's columns of
  // O, fp32 [CTA][4 columns][128 rows].
  static constexpr int kStatOff = kKOff;
  static constexpr int kRecvOff = kKOff + 2 * kTileM * 4;
  static_assert(kRecvOff + kTileM * D * 4 <= kVOff, "the parts fit the K ring");
  static_assert(D / kMostSplit >= 16, "16 columns of O at least to a CTA");
};

// Register split per warpgroup (setmaxnreg): output (warps 0-3), softmax
// (4-7, 8-11), TMA and MMA (12, 13; two idle warps).  The launch holds 128 a
// thread; each SM sub-partition has one warp of every warpgroup.
constexpr uint32_t kWinOut = 48;
constexpr uint32_t kWinSoft = 192;
constexpr uint32_t kWinLow = 80;
constexpr uint32_t kWinLaunchRegs = 128;
static_assert(kWinOut + 2 * kWinSoft + kWinLow <= 4 * kWinLaunchRegs, "register split exceeds the launch");

// Item -> query tile: tile-major with the heads side by side, so that the CTAs
// running at any moment share the window's K and V tiles in L2; the last tiles
// first (the first tiles of a sequence have shorter windows and fill the tail).
struct WindowItem {
  int b, h, bh, hkv, r0;
  WindowBlocks kb;
};
template <bool SPLIT>
__device__ __forceinline__ WindowItem window_item(int item, const WindowFwdParams& p, int n_tiles) {
  WindowItem it;
  const int BH = p.B * p.H;
  const int rank = item / BH;
  it.bh = item - rank * BH;
  it.b = it.bh / p.H;
  it.h = it.bh - it.b * p.H;
  it.hkv = it.h / (p.H / p.Hkv);
  it.r0 = (n_tiles - 1 - rank) * kTileM;
  it.kb = window_blocks(window_rows(p.w, it.r0, p.Lk), p.w.snk, min(p.Lq - it.r0, kTileM), p.Lk);
  if (SPLIT) it.kb = it.kb.part(static_cast<int>(blockIdx.x) % p.split, p.split);
  return it;
}

// A CTA's first item, and how far the next one is (a split item is its CTAs' only one).
template <bool SPLIT>
__device__ __forceinline__ int window_first(const WindowFwdParams& p) {
  return SPLIT ? static_cast<int>(blockIdx.x) / p.split : static_cast<int>(blockIdx.x);
}
template <bool SPLIT>
__device__ __forceinline__ int window_stride(const WindowFwdParams& p) {
  return SPLIT ? p.n_items : static_cast<int>(gridDim.x);
}
// The first item from `item` on in this CTA's stride that has a key block
// (p.n_items or more: none).
template <bool SPLIT>
__device__ __forceinline__ int window_next(int item, const WindowFwdParams& p, int n_tiles, WindowItem& it) {
  for (; item < p.n_items; item += window_stride<SPLIT>(p)) {
    it = window_item<SPLIT>(item, p, n_tiles);
    if (it.kb.count() > 0) break;
  }
  return item;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address of this CTA's shared memory `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_store4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}

// SPLIT: the CTAs of a cluster share one item's blocks, and join their states.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(512, 1)
    attn_fwd_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const WindowFwdParams p) {
  using C = WinCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  {
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    if (pad > static_cast<uint32_t>(C::kSlack)) {   // layout would not fit: report, touch nothing
      if (threadIdx.x == 0) record_error(p.err, ATTN_ERR_UNSUPPORTED);
      return;
    }
  }
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::kBarOff + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kTmemSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kAbortOff);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int tid = static_cast<int>(threadIdx.x);
  const int status = status_at_entry(p.err);
  const int n_tiles = (p.Lq + kTileM - 1) / kTileM;

  if (tid == 0) {
    for (int s = 0; s < C::kStagesQ; ++s) {
      mbar_init(bar(C::kBarQFull + s), 1);
      mbar_init(bar(C::kBarQEmpty + s), 1);
    }
    for (int s = 0; s < C::kStagesK; ++s) {
      mbar_init(bar(C::kBarKFull + s), 1);
      mbar_init(bar(C::kBarKEmpty + s), 1);
    }
    for (int s = 0; s < C::kStagesV; ++s) {
      mbar_init(bar(C::kBarVFull + s), 1);
      mbar_init(bar(C::kBarVEmpty + s), 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(bar(C::kBarXch + s), 2 * 4 * 32);
    mbar_init(bar(C::kBarSFull), 1);
    mbar_init(bar(C::kBarSFree), 2 * 4 * 32);
    mbar_init(bar(C::kBarPFull + 0), 2 * 4 * 32);
    mbar_init(bar(C::kBarPFull + 1), 4 * 32);
    mbar_init(bar(C::kBarPvDone + 0), 1);
    mbar_init(bar(C::kBarPvDone + 1), 1);
    mbar_init(bar(C::kBarOFull), 1);
    mbar_init(bar(C::kBarOEmpty), 4 * 32);
    mbar_init(bar(C::kBarLFull), 4 * 32);
    mbar_init(bar(C::kBarMmaDone), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(sbase + C::kTmemSlotOff, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool gave_up = __syncthreads_or(!SPLIT && status == ATTN_ERR_TIMEOUT);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (gave_up) {                   // (a cluster's CTAs would have to agree on it)
    if (warp == 0) {
      __syncwarp();
      tmem_dealloc(tmem, C::kTmemCols);
    }
    return;
  }

  if (warp >= 12) {
    regs_set<kWinLow, kWinLaunchRegs>();
    if (warp == 12) {
      // =================== TMA producer ===================
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        int ik = 0, iv = 0;     // pair stages and V tiles loaded (over all items)
        int qn = 0;             // Q tiles loaded
        // the item's pair k: key blocks 2 k and 2 k + 1 of its list (the second
        // may be missing); a block that reaches past the last key reads the
        // zero fill there
        auto load_k = [&](const WindowItem& it, int k) -> bool {
          const int s = ik % C::kStagesK;
          if (ik >= C::kStagesK &&
              !wait_bar(bar(C::kBarKEmpty + s), ((ik / C::kStagesK) & 1) ^ 1, abort_flag, p.err))
            return false;
          const bool two = 2 * k + 1 < it.kb.count();
          const uint32_t ks = sbase + C::kKOff + s * C::kPairBytes;
          mbar_arrive_expect_tx(bar(C::kBarKFull + s), two ? C::kPairBytes : C::kTileBytes);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == 1 && !two) break;
            const int row = it.kb.at(2 * k + t) * kTileN;
#pragma unroll
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_4d(ks + c * 2 * C::kChunkBytes + t * C::kChunkBytes, &tmK, bar(C::kBarKFull + s),
                          c * 64, row, it.hkv, it.b);
          }
          ++ik;
          return true;
        };
        auto load_v = [&](int row, int hkv, int b) -> bool {
          if (row < 0) return true;        // no such block
          const int s = iv % C::kStagesV;
          if (iv >= C::kStagesV &&
              !wait_bar(bar(C::kBarVEmpty + s), ((iv / C::kStagesV) & 1) ^ 1, abort_flag, p.err))
            return false;
          const uint32_t vs = sbase + C::kVOff + s * C::kTileBytes;
          mbar_arrive_expect_tx(bar(C::kBarVFull + s), C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(vs + c * C::kChunkBytes, &tmV, bar(C::kBarVFull + s), c * 64, row, hkv, b);
          ++iv;
          return true;
        };
        auto load_q = [&](const WindowItem& it) -> bool {
          const int s = qn % C::kStagesQ;
          // the last S that read this Q buffer must have completed
          if (qn >= C::kStagesQ &&
              !wait_bar(bar(C::kBarQEmpty + s), ((qn / C::kStagesQ) & 1) ^ 1, abort_flag, p.err))
            return false;
          mbar_arrive_expect_tx(bar(C::kBarQFull + s), C::kTileBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sbase + C::kQOff + s * C::kTileBytes + c * C::kChunkBytes, &tmQ,
                        bar(C::kBarQFull + s), c * 64, it.r0, it.h, it.b);
          ++qn;
          return true;
        };
        WindowItem it;
        int item = window_next<SPLIT>(window_first<SPLIT>(p), p, n_tiles, it);
        bool ok = true;
        if (item < p.n_items) ok = load_k(it, 0) && load_q(it);
        int k = 0;
        while (ok && item < p.n_items) {
          // V of this pair goes after K of the next one
          const int nb = it.kb.count();
          const int hkv = it.hkv, b = it.b;
          const int v0 = it.kb.at(2 * k) * kTileN;
          const int v1 = 2 * k + 1 < nb ? it.kb.at(2 * k + 1) * kTileN : -1;
          if (2 * k + 2 < nb) {
            ok = load_k(it, ++k);
          } else {
            k = 0;
            item = window_next<SPLIT>(item + window_stride<SPLIT>(p), p, n_tiles, it);
            if (item < p.n_items) ok = load_k(it, 0) && load_q(it);
          }
          ok = ok && load_v(v0, hkv, b) && load_v(v1, hkv, b);
        }
        // every copy issued has landed before the CTA may exit
        for (int j = max(0, ik - C::kStagesK); j < ik; ++j)
          drain_bar(bar(C::kBarKFull + j % C::kStagesK), (j / C::kStagesK) & 1);
        for (int j = max(0, iv - C::kStagesV); j < iv; ++j)
          drain_bar(bar(C::kBarVFull + j % C::kStagesV), (j / C::kStagesV) & 1);
        for (int j = max(0, qn - C::kStagesQ); j < qn; ++j)
          drain_bar(bar(C::kBarQFull + j % C::kStagesQ), (j / C::kStagesQ) & 1);
      }
    } else if (warp == 13) {
      // =================== MMA issuer (one thread) ===================
      // For every pair: S of the next pair (of the next item at an item's
      // end), as soon as both softmax warpgroups hold this pair's S in
      // registers, then this pair's P V.
      if (lane == 0) {
        constexpr uint32_t kIdescS = idesc_bf16_f32(kTileM, 2 * kTileN, false, false);
        constexpr uint32_t kIdescS1 = idesc_bf16_f32(kTileM, kTileN, false, false);   // a block alone
        constexpr uint32_t kIdescPV = idesc_bf16_f32(kTileM, D, false, true);
        int ik = 0, iv = 0;     // pair stages and V tiles consumed
        int qn = 0;             // Q tiles consumed
        int sn = 0;             // S tiles issued
        int pn = 0;             // P tiles consumed
        int on = 0;             // O results handed to the output warps
        // S of pair k of an item with nb blocks
        auto issue_s = [&](int k, int nb) -> bool {
          if (k == 0) {
            if (!wait_bar(bar(C::kBarQFull + qn % C::kStagesQ), (qn / C::kStagesQ) & 1, abort_flag, p.err))
              return false;
            ++qn;
          }
          if (sn > 0 && !wait_bar(bar(C::kBarSFree), (sn - 1) & 1, abort_flag, p.err)) return false;
          const int s = ik % C::kStagesK;
          if (!wait_bar(bar(C::kBarKFull + s), (ik / C::kStagesK) & 1, abort_flag, p.err)) return false;
          tc_fence_after();
          const int qs = (qn - 1) % C::kStagesQ;
          const uint64_t dq = sdesc_sw128(sbase + C::kQOff + qs * C::kTileBytes, 16, 1024);
          const uint64_t dk = sdesc_sw128(sbase + C::kKOff + s * C::kPairBytes, 16, 1024);
          const uint32_t idesc = 2 * k + 1 < nb ? kIdescS : kIdescS1;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qoff = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
            const uint32_t koff = (kk >> 2) * 2 * C::kChunkBytes + (kk & 3) * 32;
            mma_ss(tmem + C::kColS, sdesc_add(dq, qoff), sdesc_add(dk, koff), idesc, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar(C::kBarSFull));
          mma_commit(bar(C::kBarKEmpty + s));
          if (2 * k + 2 >= nb) mma_commit(bar(C::kBarQEmpty + qs));   // Q's buffer is free for a later item
          ++ik;
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
              // O still holds the previous item's result until the output warps read it
              if (!wait_bar(bar(C::kBarOEmpty), (on - 1) & 1, abort_flag, p.err)) return false;
              tc_fence_after();
            }
            if (2 * k + t < nb) {
              const int s = iv % C::kStagesV;
              if (!wait_bar(bar(C::kBarVFull + s), (iv / C::kStagesV) & 1, abort_flag, p.err)) return false;
              tc_fence_after();
              const uint64_t dv = sdesc_sw128(sbase + C::kVOff + s * C::kTileBytes, C::kChunkBytes, 1024);
#pragma unroll
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
        WindowItem it;
        int item = window_next<SPLIT>(window_first<SPLIT>(p), p, n_tiles, it);
        int nb = it.kb.count();
        bool ok = item >= p.n_items || issue_s(0, nb);
        while (ok && item < p.n_items) {
          item = window_next<SPLIT>(item + window_stride<SPLIT>(p), p, n_tiles, it);
          const int nb2 = item < p.n_items ? it.kb.count() : 0;
          const int ns = (nb + 1) / 2;
          for (int k = 0; k < ns && ok; ++k) {
            if (k + 1 < ns) ok = issue_s(k + 1, nb);
            else if (nb2 > 0) ok = issue_s(0, nb2);
            if (ok) ok = issue_pv(k, nb);
          }
          if (!ok) break;
          mma_commit(bar(C::kBarOFull));
          ++on;
          nb = nb2;
        }
        // every MMA issued has completed before tensor memory is released
        mma_commit(bar(C::kBarMmaDone));
        drain_bar(bar(C::kBarMmaDone), 0);
      }
    }
  } else if (warp < 4) {
    regs_set<kWinOut, kWinLaunchRegs>();
    // =================== output: thread = query row ===================
    const int row_in_tile = warp * 32 + lane;
    const uint32_t tO = tmem + (static_cast<uint32_t>(warp * 32) << 16) + C::kColO;
    if constexpr (SPLIT) {
      // Every CTA of the cluster is done with its part of the keys; rank r
      // joins columns [r D / split, (r + 1) D / split) of O.  A part is scaled
      // by e^{m_c - m} / l on its way, l = sum_c e^{m_c - m} l_c.
      cluster_arrive();
      cluster_wait();
      tc_fence_after();
      const int rank = static_cast<int>(blockIdx.x) % p.split;
      const int cols = D / p.split;
      const WindowItem it = window_item<SPLIT>(window_first<SPLIT>(p), p, n_tiles);
      const float NEG_INF = -__int_as_float(0x7f800000);
      const uint32_t stat = sbase + C::kStatOff + row_in_tile * 4;
      float m = NEG_INF, l = 0.f, f = 0.f;
      for (int c = 0; c < p.split; ++c)
        if (cluster_load(cluster_addr(stat + kTileM * 4, c)) != 0.f)
          m = fmaxf(m, cluster_load(cluster_addr(stat, c)));
      for (int c = 0; c < p.split; ++c) {
        const float lc = cluster_load(cluster_addr(stat + kTileM * 4, c));
        if (lc == 0.f) continue;                      // this part saw no key
        const float w = ex2(cluster_load(cluster_addr(stat, c)) - m);
        l = fmaf(w, lc, l);
        if (c == rank) f = w;
      }
      if (l != 0.f) f /= l;
      const bool none = it.kb.count() == 0 || f == 0.f;   // O holds nothing, or nothing that counts
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        const int owner = c * 16 / cols;
        if (owner == rank) continue;
        uint32_t o[16];
        tmem_ld16(tO + c * 16, o);
        tmem_ld_wait16(o);
        const uint32_t to = cluster_addr(
            sbase + C::kRecvOff + ((rank * cols + c * 16 - owner * cols) / 4 * kTileM + row_in_tile) * 16, owner);
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          cluster_store4(to + e / 4 * kTileM * 16, none ? 0.f : __uint_as_float(o[e]) * f,
                         none ? 0.f : __uint_as_float(o[e + 1]) * f, none ? 0.f : __uint_as_float(o[e + 2]) * f,
                         none ? 0.f : __uint_as_float(o[e + 3]) * f);
      }
      cluster_arrive();
      cluster_wait();
      const int row = it.r0 + row_in_tile;
      const size_t at = static_cast<size_t>(it.bh) * p.Lq + row;
#pragma unroll 1
      for (int c = rank * cols / 16; c < (rank + 1) * cols / 16; ++c) {
        uint32_t o[16];
        tmem_ld16(tO + c * 16, o);
        tmem_ld_wait16(o);
        float y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = none ? 0.f : __uint_as_float(o[e]) * f;
        for (int s = 0; s < p.split; ++s) {
          if (s == rank) continue;
          const float4* from = reinterpret_cast<const float4*>(smem + C::kRecvOff) +
                               (s * cols + c * 16 - rank * cols) / 4 * kTileM + row_in_tile;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 x = from[e * kTileM];
            y[4 * e] += x.x;
            y[4 * e + 1] += x.y;
            y[4 * e + 2] += x.z;
            y[4 * e + 3] += x.w;
          }
        }
        if (row < p.Lq) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + at * D) + 2 * c;
          dst[0] = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
          dst[1] = make_uint4(pack_bf16(y[8], y[9]), pack_bf16(y[10], y[11]), pack_bf16(y[12], y[13]),
                              pack_bf16(y[14], y[15]));
        }
      }
      if (rank == 0 && row < p.Lq) p.lse[at] = l == 0.f ? NEG_INF : (m + __log2f(l)) * kLn2;
    }
    const volatile float* inv_s = reinterpret_cast<const volatile float*>(smem + C::kInvOff);
    int on = 0;             // O results read
    for (int item = static_cast<int>(blockIdx.x); !SPLIT && item < p.n_items; item += static_cast<int>(gridDim.x)) {
      const WindowItem it = window_item<SPLIT>(item, p, n_tiles);
      const size_t rows0 = static_cast<size_t>(it.bh) * p.Lq;
      const bool inb = it.r0 + row_in_tile < p.Lq;
      uint4* dst = reinterpret_cast<uint4*>(p.o + (rows0 + it.r0 + row_in_tile) * D);
      const bool any = it.kb.count() > 0;
      float inv = 0.f;
      if (any) {
        if (!__all_sync(0xFFFFFFFFu, wait_bar_relaxed(bar(C::kBarLFull), on & 1, abort_flag, p.err))) break;
        inv = inv_s[row_in_tile];
        if (!__all_sync(0xFFFFFFFFu, wait_bar_relaxed(bar(C::kBarOFull), on & 1, abort_flag, p.err))) break;
        tc_fence_after();
      } else if (inb) {
        p.lse[rows0 + it.r0 + row_in_tile] = -__int_as_float(0x7f800000);
      }
      // 16 columns at a time, 32 bytes of the row (the warpgroup has few
      // registers); a row without a key (inv = 0) is 0 whatever the masked
      // keys held
#pragma unroll 1
      for (int c = 0; c < D / 16; ++c) {
        uint32_t o[16];
        if (any) {
          tmem_ld16(tO + c * 16, o);
          tmem_ld_wait16(o);
          if (c == D / 16 - 1) {
            tc_fence_before();
            mbar_arrive(bar(C::kBarOEmpty));      // the next item's P V may overwrite O
          }
        }
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = inv == 0.f ? 0u : pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
        if (inb) {
          dst[2 * c] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[2 * c + 1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (any) ++on;
    }
  } else {
    regs_set<kWinSoft, kWinLaunchRegs>();
    // =================== softmax warpgroups: X = 0 (warps 4-7), 1 (warps 8-11) ===================
    const int X = (warp - 4) >> 2;                // key block X of every pair
    const int wq = warp & 3;                      // TMEM lane quarter of this warp
    const int row_in_tile = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_base + C::kColS + X * 128;
    const uint32_t tP = tmem + lane_base + C::kColP + X * 64;
    const uint32_t tO = tmem + lane_base + C::kColO + X * (D / 2);
    const float sl2 = p.scale_log2;
    const float NEG_INF = -__int_as_float(0x7f800000);
    float* xch = reinterpret_cast<float*>(smem + C::kXchOff);

    float* inv_s = reinterpret_cast<float*>(smem + C::kInvOff);

    int cnt = 0;        // S tiles consumed (over all items)
    int nx = 0;         // row values exchanged
    int on = 0;         // items finished
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
    // the items again, as query tiles (from the last one up) and heads, stepped
    // through without a division
    const int BH = p.B * p.H;
    int rank = window_first<SPLIT>(p) / BH;
    int bh = window_first<SPLIT>(p) - rank * BH;
    const int d_rank = SPLIT ? n_tiles : static_cast<int>(gridDim.x) / BH;
    const int d_bh = SPLIT ? 0 : static_cast<int>(gridDim.x) - d_rank * BH;
    for (; rank < n_tiles; rank += d_rank, bh += d_bh) {
      if (bh >= BH) {
        bh -= BH;
        if (++rank >= n_tiles) break;
      }
      const int r0 = (n_tiles - 1 - rank) * kTileM;
      const WindowRows t = window_rows(p.w, r0, p.Lk);
      WindowBlocks kb = window_blocks(t, p.w.snk, min(p.Lq - r0, kTileM), p.Lk);
      if (SPLIT) kb = kb.part(static_cast<int>(blockIdx.x) % p.split, p.split);
      const int nb = kb.count();
      if (nb == 0) {
        if (SPLIT && X == 0) {                      // a part without a block
          reinterpret_cast<float*>(smem + C::kStatOff)[row_in_tile] = NEG_INF;
          reinterpret_cast<float*>(smem + C::kStatOff)[kTileM + row_in_tile] = 0.f;
        }
        continue;
      }
      const int ns = (nb + 1) / 2;
      float m2 = NEG_INF;     // reference max (log2 units), moved only by > 8
      float l = 0.f;          // this warpgroup's part of the row sum
      for (int k = 0; k < ns; ++k) {
        const bool none = 2 * k + X >= nb;        // the pair's second block is missing
        const int kstart = none ? 0 : kb.at(2 * k + X) * kTileN;
        if (!__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarSFull), cnt & 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
        // S is in registers: the next pair's S may overwrite its columns
        tc_fence_before();
        mbar_arrive(bar(C::kBarSFree));

        // element mask, 32 columns at a time: a bit for each allowed key of this
        // row (j <= jhi: diagonal and last key; j >= jlo: window; j < js:
        // sinks).  Most groups of an edge block are allowed or masked as a
        // whole for the warp's 32 rows; only the others go element by element
        const int diag0 = t.own - kstart;           // first row's own key
        const int low0 = t.lo - kstart;             // the first one its window holds
        const bool edge = none || kstart + kTileN > p.Lk || kTileN - 1 > diag0 ||
                          (low0 + kTileM - 1 > 0 && kstart + kTileN > p.w.snk);
        if (edge) {
          const int jhi = none ? -1 : min(diag0 + row_in_tile, p.Lk - 1 - kstart);
          const int jlo = low0 + row_in_tile;
          const int js = p.w.snk - kstart;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t bits = bits_below(jhi + 1 - 32 * c) & (~bits_below(jlo - 32 * c) | bits_below(js - 32 * c));
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
        const float mu = (m2 == NEG_INF) ? 0.f : m2;
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
              pk[c2 * 16 + j / 2] = pack_bf16(p0, p1);
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
      // inverse to the output warps, which must have read the previous item's
      float lo;
      if (!exchange(l, lo)) break;
      if (SPLIT) {
        if (X == 0) {
          reinterpret_cast<float*>(smem + C::kStatOff)[row_in_tile] = m2;
          reinterpret_cast<float*>(smem + C::kStatOff)[kTileM + row_in_tile] = l + lo;
        }
      } else if (X == 0) {
        if (on > 0 &&
            !__all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarOEmpty), (on - 1) & 1, abort_flag, p.err)))
          break;
        // a row that saw no key has l = 0; a NaN score makes l NaN and goes through
        const float lt = l + lo;
        inv_s[row_in_tile] = lt == 0.f ? 0.f : 1.f / lt;
        mbar_arrive(bar(C::kBarLFull));
        const int row = r0 + row_in_tile;
        if (row < p.Lq)
          p.lse[static_cast<size_t>(bh) * p.Lq + row] =
              lt == 0.f ? NEG_INF : (m2 + __log2f(lt)) * kLn2;
      }
      ++on;
    }
  }

  tc_fence_before();
  if (SPLIT && warp >= 4) {        // the output warps' two meetings with the cluster's other CTAs
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// An item's CTAs.  Where a launch has few items, their steps of a pair of key
// blocks (1.7 us each) follow one another while most SMs idle: a cluster of 2
// or 4 CTAs then shares the item's pairs and joins its states through
// distributed shared memory, which costs 3 to 4 us.  Taken where the clusters
// all run at once (`room` of them) and items have 5 pairs or more, 4 or more
// for 4 CTAs (us with 1, 2, 4 CTAs an item, d=128, 16 heads: 1 query, window
// 512 (2 pairs) 9.0, 10.9, 11.3, window 1024 (4) 12.8, 12.3, 11.5, window 4096
// 33.2, 22.5, 16.4; 500 queries, which leave room for 2, window 1024 (5) 16.0,
// 16.0, window 2048 (9) 22.8, 19.5).  8 CTAs find room for few clusters (16
// of them take two turns).
int window_split(int n_items, int pairs, const int* room) {
  if (pairs >= 4 && n_items <= room[1]) return 4;
  return pairs >= 5 && n_items <= room[0] ? 2 : 1;
}

template <int D, bool SPLIT>
cudaError_t launch_window_kernel(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const WindowFwdParams& p, int sms, cudaStream_t st) {
  using C = WinCfg<D>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(SPLIT ? p.n_items * p.split : std::min(p.n_items, sms));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = SPLIT ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_fwd_window_kernel<D, SPLIT>, tq, tk, tv, p);
}

// What a launch has to know of the device, and the kernels' attributes, set once a device.
struct WindowDevice {
  bool ready;
  int sms;
  int room[2];                  // clusters of 2 and of 4 CTAs that run at once
};
template <int D>
cudaError_t window_device(int dev, const WindowDevice** out) {
  using C = WinCfg<D>;
  constexpr int kMaxDev = 64;
  static WindowDevice devices[kMaxDev] = {};
  static std::mutex mu;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(mu);
  if (!devices[dev].ready) {
    WindowDevice w{};
    const void* kernels[] = {reinterpret_cast<const void*>(attn_fwd_window_kernel<D, false>),
                             reinterpret_cast<const void*>(attn_fwd_window_kernel<D, true>)};
    cudaError_t e;
    for (const void* k : kernels) {
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, k)) != cudaSuccess) return e;
      if (fa.numRegs < static_cast<int>(kWinLaunchRegs)) return cudaErrorInvalidConfiguration;
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
      if (e != cudaSuccess) return e;
    }
    if ((e = cudaDeviceGetAttribute(&w.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    for (int i = 0; i < 2; ++i) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(2 << i);
      cfg.blockDim = dim3(C::kThreads);
      cfg.dynamicSmemBytes = C::kSmemBytes;
      cudaLaunchAttribute attr{};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 2 << i;
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      if ((e = cudaOccupancyMaxActiveClusters(&w.room[i], kernels[1], &cfg)) != cudaSuccess) return e;
    }
    w.ready = true;
    devices[dev] = w;
  }
  *out = &devices[dev];
  return cudaSuccess;
}

// `pairs`: pairs of key blocks that an item has at most.
template <int D>
cudaError_t launch_window_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              WindowFwdParams& p, int pairs, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const WindowDevice* w;
  if ((e = window_device<D>(dev, &w)) != cudaSuccess) return e;
  p.split = window_split(p.n_items, pairs, w->room);
  return p.split > 1 ? launch_window_kernel<D, true>(tq, tk, tv, p, w->sms, st)
                     : launch_window_kernel<D, false>(tq, tk, tv, p, w->sms, st);
}

// Pairs of key blocks of the query tiles that see the most.
int window_pairs(const WindowFwdParams& p) {
  const long long last = std::min<long long>(p.Lq - 1 + p.w.sh, p.Lk - 1);      // the last key anyone sees
  if (last < 0) return 0;
  const long long span = std::min<long long>(p.w.window + std::min(p.Lq, kTileM) - 1, last + 1);
  const long long blocks = (span + kTileN - 1) / kTileN + (p.w.snk + kTileN - 1) / kTileN;
  return static_cast<int>((std::min(blocks, last / kTileN + 1) + 1) / 2);
}

}  // namespace

bool window_mask(WindowMask* w, int Lk, int64_t window, int64_t sinks, int64_t q_offset,
                 int64_t k_offset) {
  if (window < 1 || sinks < 0 || q_offset < 0 || k_offset < 0) return false;
  // positions are compared as differences: bounded so that no sum wraps
  constexpr int64_t kMost = int64_t(1) << 60;
  w->sh = std::min(q_offset, kMost) - std::min(k_offset, kMost);
  w->window = std::min(window, kMost);
  w->snk = static_cast<int>(
      std::max<int64_t>(0, std::min<int64_t>(std::min(sinks, kMost) - std::min(k_offset, kMost), Lk)));
  return true;
}

}  // namespace bss

using namespace bss;

extern "C" attn_status_t attn_fwd_window(const void* q, const void* k, const void* v, void* o,
                                         float* lse, int B, int H, int H_kv, int Lq, int Lk, int d,
                                         float scale, int64_t window, int64_t sinks,
                                         int64_t q_offset, int64_t k_offset, void* stream) {
  attn_status_t s = check_common(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  if (!valid_kv_heads(H, H_kv)) return ATTN_ERR_INVALID_ARG;
  if (Lq > kMaxTokens || Lk > kMaxTokens) return ATTN_ERR_UNSUPPORTED;
  WindowFwdParams p{};
  if (!window_mask(&p.w, Lk, window, sinks, q_offset, k_offset)) return ATTN_ERR_INVALID_ARG;
  if (Lq == 0) return ATTN_OK;
  if (Lk == 0) k = v = q;        // empty tensors may have no address; no key is read
  const void* ptrs16[] = {q, k, v, o};
  for (const void* ptr : ptrs16)
    if (!ptr || !aligned16(ptr)) return ATTN_ERR_INVALID_ARG;
  if (!lse || !aligned4(lse)) return ATTN_ERR_INVALID_ARG;
  if ((s = get_encoder()) != ATTN_OK) return s;
  if ((s = status_word(&p.err)) != ATTN_OK) return s;
  CUtensorMap tq, tk, tv;
  if ((s = make_map(&tq, q, B, H, Lq, d)) != ATTN_OK) return s;
  if ((s = make_map(&tk, k, B, H_kv, Lk, d)) != ATTN_OK) return s;
  if ((s = make_map(&tv, v, B, H_kv, Lk, d)) != ATTN_OK) return s;
  p.B = B;
  p.H = H;
  p.Hkv = H_kv;
  p.Lq = Lq;
  p.Lk = Lk;
  p.scale_log2 = scale * kLog2e;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  const long long items = static_cast<long long>(B) * H * ((static_cast<long long>(Lq) + kTileM - 1) / kTileM);
  if (items > 0x7FFF0000ll) return ATTN_ERR_UNSUPPORTED;   // counted in an int, a grid's stride past the last
  p.n_items = static_cast<int>(items);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int pairs = window_pairs(p);
  const cudaError_t e = d == 64 ? launch_window_fwd<64>(tq, tk, tv, p, pairs, st)
                                : launch_window_fwd<128>(tq, tk, tv, p, pairs, st);
  return cuda_status("attn_fwd_window launch", e);
}
