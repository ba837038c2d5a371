// attn_bwd_window: gradients of attn_fwd_window by recomputation.
//
// Mathematics (window.cuh has the mask; sums run over the allowed pairs):
//   D_i  = dO_i . O_i  (= sum_j P_ij dO_i . V_j)
//   P_ij = exp(scale q_i . k_j - LSE_i)
//   dV_j = sum_i P_ij dO_i
//   dS_ij = scale P_ij (dO_i . V_j - D_i)
//   dK_j = sum_i dS_ij q_i,   dQ_i = sum_j dS_ij k_j
//
// The main kernel is the KV-owned traversal of the dense backward (an item is a
// 128-key tile; scores transposed so that a thread owns a key row, dK and dV
// in tensor memory, dQ added into an fp32 accumulator by bulk reduce-adds)
// over the query tiles that the window lets the key tile meet.
//
// Up to kFewSinks sinks have a kernel of their own, which also takes D.  With
// more, a tile with a sink key meets every later query tile, where window / 128 +
// 1 tiles would be its neighbours' share: its walk is cut into segments of about
// that share, each a CTA of its own that leaves fp32 parts of dK and dV in the
// workspace; a last kernel adds the parts in segment order and rounds once.
// The other tiles' walks are cut the same way when there are too few tiles to
// fill the GPU.  dK and dV come out the same in every run; dQ's fp32 additions
// come in the order the CTAs reach them, so its last bit may differ.
//
// P and dS are rounded to bf16 as the operands of their products, all else is
// fp32 until the results: dQ and dK come out 2.4e-3 off in norm, dV 2.3e-3
// (rounding them alone costs 1.65e-3).  The pairs with up to kFewSinks sinks take
// two bf16 parts: 2.0e-3, 2.0e-3 and 1.7e-3 off in the first case below.
//
// Measured, B1 H16(4) L16384 d128, window 1024, sinks 4: D and the sinks 59 us
// (HBM: 336 MB), main kernel 343 us (970 TFLOP/s of allowed pairs), dQ and parts
// 30 us (HBM: 220 MB, part of it from L2).  What sets the main kernel's pace is
// the chain of hand-offs of a query tile, dQ -> drain -> dP^T -> dS -> dQ, as in
// the dense backward (tensor pipe 49 % busy while an SM has a CTA), and an
// item's set-up and epilogue over walks of 10 tiles a head.
// B4 H16 L2000 d64, window 256: D and clearing 16, main kernel 67, dQ 9.5 us.
#include <algorithm>

#include "host.cuh"
#include "mma.cuh"
#include "window.cuh"

namespace bss {
namespace {

// Which rows get D from its definition (below): those of at most kFewKeys keys
// near the first or past the last key, and all of them where window and sinks
// together are at most kFewWindow keys.
constexpr int kFewKeys = 64;
constexpr int kFewWindow = 32;

// Sinks that have a kernel of their own: up to an N tile of its products.
constexpr int kFewSinks = 8;

// Key tiles j0 .. j0 + n - 1 of every K/V head, their walks cut into `seg`
// segments each; their first item, and the workspace slot of its part (cut
// walks).
struct WindowTiles {
  int j0, n, seg;
  int item0, slot0;
};

struct WindowBwdParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  int B, H, Hkv, Lq, Lk;
  float scale, scale_log2;
  WindowMask w;
  const __nv_bfloat16* o;
  const __nv_bfloat16* dout;
  const float* lse;
  float* delta;
  float* dq_acc;        // fp32 [B,H,Lq,d]
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* part;          // fp32 [slot][dK, dV][128][d]: parts of the cut walks
  float* sink_part;     // fp32 [B H_kv][sink_ctas][dK, dV][kFewSinks][d]
  int sink_ctas;        // CTAs of a K/V head in the sinks' kernel (0: not launched)
  int few_sinks;        // the first keys, which it takes and the main kernel leaves out
  int nk;               // key tiles
  int nst;              // the first of them, which meet every later query tile for a sink key
  WindowTiles tiles[2]; // those, and the others, in the order of their items
  int n_items;          // key tiles, or segments of them, over all heads
  int* err;
};

template <int D>
struct WinBwdCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kChunkBytes = kTileM * 128;
  static constexpr int kTileBytes = kTileM * D * 2;
  static constexpr int kStagesQ = 2;                     // Q_i ring depth (S^T(i+1) and dK(i) overlap)
  static constexpr int kStagesDO = (D == 128) ? 1 : 2;    // dO_i ring depth (room for dQ staging)
  static constexpr int kKOff = 0;
  static constexpr int kVOff = kKOff + kTileBytes;
  static constexpr int kQOff = kVOff + kTileBytes;
  static constexpr int kDOOff = kQOff + kStagesQ * kTileBytes;
  static constexpr int kDSOff = kDOOff + kStagesDO * kTileBytes;  // dS, 128 keys x 128 queries bf16
  static constexpr int kDSBytes = kTileM * kTileN * 2;
  static constexpr int kStageOff = kDSOff + kDSBytes;    // dQ staging: 128 rows x 64 fp32
  static constexpr int kStageBytes = kTileM * 64 * 4;
  static constexpr int kStatOff = kStageOff + kStageBytes;   // 2 x (lse2[128], delta[128])
  static constexpr int kBarOff = kStatOff + 2 * 2 * 128 * 4;
  static constexpr int kBarKV = 0;
  static constexpr int kBarQFull = 1;
  static constexpr int kBarQEmpty = kBarQFull + kStagesQ;
  static constexpr int kBarDOFull = kBarQEmpty + kStagesQ;
  static constexpr int kBarDOEmpty = kBarDOFull + kStagesDO;
  static constexpr int kBarSFull = kBarDOEmpty + kStagesDO;   // S^T of a query tile in TMEM
  static constexpr int kBarDPFull = kBarSFull + 1;            // [2]: dP^T query half h in TMEM
  static constexpr int kBarPReady = kBarDPFull + 2;           // P^T written (S^T read)
  static constexpr int kBarDSReady = kBarPReady + 1;          // dS in shared memory (dP^T read)
  static constexpr int kBarDQFull = kBarDSReady + 1;
  static constexpr int kBarDQFree = kBarDQFull + 1;           // [2]: dQ d-columns [64r, 64r+64) read
  static constexpr int kBarDKVFull = kBarDQFree + 2;
  static constexpr int kBarMmaDone = kBarDKVFull + 1;
  static constexpr int kBarStat = kBarMmaDone + 1;     // [2]: LSE/D of a query tile staged
  static constexpr int kBarStaged = kBarStat + 2;      // dQ round staged (CTA-wide drain)
  static constexpr int kBarStageFree = kBarStaged + 1; // staging read by the reduce (CTA-wide drain)
  static constexpr int kBarKVEmpty = kBarStageFree + 1;  // an item's last MMA that reads K or V completed
  static constexpr int kBarDKVEmpty = kBarKVEmpty + 1;   // its dK and dV read out of TMEM
  static constexpr int kNumBars = kBarDKVEmpty + 1;
  // dQ drain: at d=128 each drain warp reduces its own 32 rows (no barrier
  // among the four warps, which frees dQ's columns for dP^T sooner); at d=64,
  // with one round per tile and a shorter period, one thread reduces all 128
  // rows in two larger boxes after a CTA-wide barrier (measured faster there).
  static constexpr bool kDrainPerWarp = (D == 128);
  static constexpr int kDrainBoxRows = kDrainPerWarp ? 32 : 128;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  // Alignment slack for the 1024-byte aligned layout.  At d=128 the layout
  // leaves less than 1024 bytes: the kernel then relies on the dynamic shared
  // memory base being 1024-aligned and checks that before touching it.
  static constexpr int kPayload = kMiscOff + 16;
  static constexpr int kSlack = (kPayload + 1024 <= 232448) ? 1024 : 232448 - kPayload;
  static constexpr int kSmemBytes = kPayload + kSlack;
  static_assert(kPayload <= 232448, "backward shared memory exceeds the 227 KB a CTA may use");
  static constexpr uint32_t kTmemCols = 512;
  // TMEM columns: S^T (fp32) at [0,128) and dP^T at [128,256).  Half X of the
  // P^T/dS warpgroups (query columns [64X, 64X+64)) writes its P^T (bf16
  // pairs, 32 columns) to S^T columns [64X, 64X+32), inside the range it has
  // itself already read.  dV and dK follow.  dQ of a query tile takes dP^T's
  // columns at d=128 and columns of its own, [384,448), at d=64.
  static constexpr uint32_t kColST = 0;
  static constexpr uint32_t kColDPT = 128;
  static constexpr uint32_t kColDV = 256;
  static constexpr uint32_t kColDK = 256 + D;
  static constexpr uint32_t kColDQ = (D == 128) ? kColDPT : 384;
  static constexpr bool kDQOverDP = (kColDQ == kColDPT);
  // A operand address of query k-step kk (16 queries) inside P^T
  static __device__ __forceinline__ uint32_t pcol(int kk) { return 64 * (kk >> 2) + 8 * (kk & 3); }
  static constexpr int kThreads = 512;
};

// Register split per warpgroup (setmaxnreg): warpgroup 0 (TMA, MMA, two idle
// warps) kLow, the P/dS warpgroups 1-2 kMid (each thread keeps 64 fp32 P
// values between its two phases), the dQ warpgroup 3 kHigh.  This split
// compiles without spills, which matter more than their bytes say: the tiles
// leave L1 next to nothing, so each spilled value comes back from L2 (with 20
// values spilled and the mask compared element by element the main kernel of
// B1 H16(4) L16384 d128, window 1024, sinks 4 took 437 us, now 395).  Each SM
// sub-partition holds one warp of every warpgroup: kLow + 2 kMid + kHigh <= 512
// registers a lane, and the split fits the 512 * 128 registers the launch
// holds (the launcher refuses to launch if ptxas gave the kernel fewer than
// 128 a thread).
template <int D>
struct WinBwdRegs {
  static constexpr uint32_t kLow = 72;
  static constexpr uint32_t kMid = 168;
  static constexpr uint32_t kHigh = 104;
  static constexpr uint32_t kLaunchRegs = 128;
  static_assert(kLow + 2 * kMid + kHigh <= 512, "register split exceeds an SM sub-partition");
  static_assert(128 * (kLow + 2 * kMid + kHigh) <= 512 * kLaunchRegs, "register split exceeds the launch");
};


// Item x: a segment of a key tile's walk; the K/V heads of a tile come side by
// side, so that the running CTAs' Q, dO and dQ accumulator stay in L2.
struct WindowBwdCta {
  int bh, j, seg, nseg, slot;
};
__device__ __forceinline__ WindowBwdCta window_bwd_cta(int x, const WindowBwdParams& p) {
  const WindowTiles& t = x >= p.tiles[1].item0 ? p.tiles[1] : p.tiles[0];
  const int BH = p.B * p.Hkv;
  const int y = x - t.item0;
  WindowBwdCta c;
  c.nseg = t.seg;
  c.slot = t.slot0 + y;
  const int z = y / t.seg;
  c.seg = y - z * t.seg;
  const int jj = z / BH;
  c.bh = z - jj * BH;
  c.j = t.j0 + jj;
  return c;
}

// The (query head of the group, query tile) pairs of a CTA's walk: its segment
// of the tiles first .. first + nt - 1 of every query head, head by head.
struct WindowQWalk {
  int first, nt, n_it;
  int g0, i0;
  __device__ __forceinline__ void start(int& g, int& i) const {
    g = g0;
    i = i0;
  }
  __device__ __forceinline__ void advance(int& g, int& i) const {
    if (++i == first + nt) {
      i = first;
      ++g;
    }
  }
};
__device__ __forceinline__ WindowQWalk window_bwd_walk(const WindowBwdCta& c, const WindowBwdParams& p) {
  WindowQWalk w{0, 0, 0, 0, 0};
  const int k0 = c.j * kTileN;
  const int k1 = min(k0 + kTileN, p.Lk) - 1;
  const long long lo = max(0ll, static_cast<long long>(k0) - p.w.sh);
  long long hi = p.Lq - 1;
  if (c.j >= p.nst) hi = min(hi, static_cast<long long>(k1) - p.w.sh + p.w.window - 1);
  if (lo > hi) return w;
  w.first = static_cast<int>(lo / kTileM);
  w.nt = static_cast<int>(hi / kTileM) - w.first + 1;
  const long long total = static_cast<long long>(w.nt) * (p.H / p.Hkv);
  const long long x0 = total * c.seg / c.nseg;
  const long long x1 = total * (c.seg + 1) / c.nseg;
  w.n_it = static_cast<int>(x1 - x0);
  w.g0 = static_cast<int>(x0 / w.nt);
  w.i0 = w.first + static_cast<int>(x0 - static_cast<long long>(w.g0) * w.nt);
  return w;
}

template <int D>
__global__ void __launch_bounds__(WinBwdCfg<D>::kThreads, 1)
    attn_bwd_window_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                         const __grid_constant__ CUtensorMap tmDQ, const WindowBwdParams p) {
  using C = WinBwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  {
    const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
    if (pad > static_cast<uint32_t>(C::kSlack)) {     // layout would not fit: report, touch nothing
      if (threadIdx.x == 0) record_error(p.err, ATTN_ERR_UNSUPPORTED);
      return;
    }
  }
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::kBarOff + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);
  float* stats = reinterpret_cast<float*>(smem + C::kStatOff);

  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());
  const int tid = static_cast<int>(threadIdx.x);
  const int status = status_at_entry(p.err);

  const int Lk = p.Lk, Lq = p.Lq;
  const int G = p.H / p.Hkv;

  if (tid == 0) {
    mbar_init(bar(C::kBarKV), 1);
    for (int s = 0; s < C::kStagesQ; ++s) {
      mbar_init(bar(C::kBarQFull + s), 1);
      mbar_init(bar(C::kBarQEmpty + s), 1);
    }
    for (int s = 0; s < C::kStagesDO; ++s) {
      mbar_init(bar(C::kBarDOFull + s), 1);
      mbar_init(bar(C::kBarDOEmpty + s), 1);
    }
    mbar_init(bar(C::kBarSFull), 1);
    mbar_init(bar(C::kBarDPFull), 1);
    mbar_init(bar(C::kBarDPFull + 1), 1);
    mbar_init(bar(C::kBarPReady), 256);
    mbar_init(bar(C::kBarDSReady), 256);
    mbar_init(bar(C::kBarDQFull), 1);
    mbar_init(bar(C::kBarDQFree), 128);
    mbar_init(bar(C::kBarDQFree + 1), 128);
    mbar_init(bar(C::kBarStaged), 128);
    mbar_init(bar(C::kBarStageFree), 1);
    mbar_init(bar(C::kBarDKVFull), 1);
    mbar_init(bar(C::kBarDKVEmpty), 256);
    mbar_init(bar(C::kBarKVEmpty), 1);
    mbar_init(bar(C::kBarMmaDone), 1);
    mbar_init(bar(C::kBarStat + 0), 128);
    mbar_init(bar(C::kBarStat + 1), 128);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(sbase + C::kMiscOff, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool gave_up = __syncthreads_or(status == ATTN_ERR_TIMEOUT);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (gave_up) {
    if (warp == 0) {
      __syncwarp();
      tmem_dealloc(tmem, C::kTmemCols);
    }
    return;
  }

  if (warp < 4) {
  regs_set<WinBwdRegs<D>::kLow, WinBwdRegs<D>::kLaunchRegs>();
  if (warp == 0) {
    // =================== TMA producer ===================
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmDO);
      int nq_ld = 0, ndo_ld = 0;   // query tiles' Q and dO loaded (over all items)
      int kv = 0;                  // items' K and V loaded
      bool ok = true;
      for (int x = static_cast<int>(blockIdx.x); x < p.n_items && ok; x += static_cast<int>(gridDim.x)) {
        const WindowBwdCta cta = window_bwd_cta(x, p);
        const WindowQWalk walk = window_bwd_walk(cta, p);
        if (walk.n_it == 0) continue;
        const int b = cta.bh / p.Hkv;
        const int h = cta.bh - b * p.Hkv;
        if (kv > 0 && !wait_bar(bar(C::kBarKVEmpty), (kv - 1) & 1, abort_flag, p.err)) break;
        mbar_arrive_expect_tx(bar(C::kBarKV), 2 * C::kTileBytes);
        for (int c = 0; c < C::kChunks; ++c) {
          tma_load_4d(sbase + C::kKOff + c * C::kChunkBytes, &tmK, bar(C::kBarKV), c * 64, cta.j * kTileN, h, b);
          tma_load_4d(sbase + C::kVOff + c * C::kChunkBytes, &tmV, bar(C::kBarKV), c * 64, cta.j * kTileN, h, b);
        }
        ++kv;
        int g, i;
        walk.start(g, i);
        for (int it = 0; it < walk.n_it; walk.advance(g, i), ++it) {
          const int row = i * kTileM;
          const int hq = h * G + g;
          const int sq = nq_ld % C::kStagesQ;
          if (nq_ld >= C::kStagesQ &&
              !wait_bar(bar(C::kBarQEmpty + sq), ((nq_ld / C::kStagesQ) & 1) ^ 1, abort_flag, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::kBarQFull + sq), C::kTileBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sbase + C::kQOff + sq * C::kTileBytes + c * C::kChunkBytes, &tmQ,
                        bar(C::kBarQFull + sq), c * 64, row, hq, b);
          ++nq_ld;
          const int sd = ndo_ld % C::kStagesDO;
          if (ndo_ld >= C::kStagesDO &&
              !wait_bar(bar(C::kBarDOEmpty + sd), ((ndo_ld / C::kStagesDO) & 1) ^ 1, abort_flag, p.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar(C::kBarDOFull + sd), C::kTileBytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sbase + C::kDOOff + sd * C::kTileBytes + c * C::kChunkBytes, &tmDO,
                        bar(C::kBarDOFull + sd), c * 64, row, hq, b);
          ++ndo_ld;
        }
      }
      // Drain: every load issued has landed before the CTA may exit.
      if (kv > 0) drain_bar(bar(C::kBarKV), (kv - 1) & 1);
      for (int x = max(0, nq_ld - C::kStagesQ); x < nq_ld; ++x)
        drain_bar(bar(C::kBarQFull + x % C::kStagesQ), (x / C::kStagesQ) & 1);
      for (int x = max(0, ndo_ld - C::kStagesDO); x < ndo_ld; ++x)
        drain_bar(bar(C::kBarDOFull + x % C::kStagesDO), (x / C::kStagesDO) & 1);
    }
  } else if (warp == 1) {
    // =================== MMA issuer (one thread) ===================
    // Issue order per query tile i: dV(i), S^T(i+1), dQ(i), dK(i), dP^T(i+1).
    // Every overwrite of TMEM or shared memory is ordered behind the MMAs that
    // read the old contents by issue order (the tensor core executes one
    // thread's MMAs in order) or by the barrier it waits on:
    //   S^T(i+1) over P^T(i): after dV(i);  P^T(i+1) written after S^T(i+1)
    //   completes; dQ(i) over dP^T(i): after ds_ready(i) (dP^T read);
    //   dP^T(i+1) over dQ(i): after dq_free(i); dS(i+1) written after
    //   dP^T(i+1) completes, so after dQ(i) and dK(i) read dS(i).
    // Tiles are counted over all items (n).  An item's S^T and dP^T wait for
    // its K and V, whose buffers are free once the last item's dQ has
    // completed, and its first dV for the last item's dK and dV to be read out.
    if (lane == 0) {
      constexpr uint32_t kIdescT = idesc_bf16_f32(kTileM, kTileN, false, false);  // S^T, dP^T
      constexpr uint32_t kIdescKV = idesc_bf16_f32(kTileM, D, false, true);       // dV, dK
      constexpr uint32_t kIdescQ = idesc_bf16_f32(kTileM, D, true, true);         // dQ
      const uint32_t ka = sbase + C::kKOff, va = sbase + C::kVOff, dsa = sbase + C::kDSOff;
      // K-major and M-/N-major descriptors of a tile, built once per group of
      // MMAs, each of which adds its offset.  They go through an empty asm so
      // that the compiler does not keep every group's in registers across the
      // loop and spill them, to an L1 that the tiles leave almost nothing of.
      auto desc_k = [](uint32_t addr) -> uint64_t {
        uint64_t d = sdesc_sw128(addr, 16, 1024);
        asm volatile("" : "+l"(d));
        return d;
      };
      auto desc_mn = [](uint32_t addr) -> uint64_t {
        uint64_t d = sdesc_sw128(addr, C::kChunkBytes, 1024);
        asm volatile("" : "+l"(d));
        return d;
      };
      auto qaddr = [&](int it) { return sbase + C::kQOff + (it % C::kStagesQ) * C::kTileBytes; };
      auto doaddr = [&](int it) { return sbase + C::kDOOff + (it % C::kStagesDO) * C::kTileBytes; };
      // S^T(it) = K_j Q^T
      auto issue_s = [&](int it) -> bool {
        if (!wait_bar(bar(C::kBarQFull + it % C::kStagesQ), (it / C::kStagesQ) & 1, abort_flag, p.err))
          return false;
        tc_fence_after();
        const uint64_t dq = desc_k(qaddr(it)), dk = desc_k(ka);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
          mma_ss(tmem + C::kColST, sdesc_add(dk, off), sdesc_add(dq, off),
                 kIdescT, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(C::kBarSFull));
        return true;
      };
      // dP^T(it) = V_j dO^T, in two halves of 64 queries (N = 64) when dQ
      // shares dP^T's columns: half h overwrites dQ's d-columns [64h, 64h+64),
      // which round h of the drain frees, and feeds P/dS half X = h alone.
      constexpr uint32_t kIdescTHalf = idesc_bf16_f32(kTileM, kTileN / 2, false, false);
      auto issue_dp_half = [&](int it, int h) -> bool {
        if (h == 0) {
          if (!wait_bar(bar(C::kBarDOFull + it % C::kStagesDO), (it / C::kStagesDO) & 1, abort_flag,
                        p.err))
            return false;
        }
        tc_fence_after();
        const uint64_t ddo = desc_k(doaddr(it) + h * (kTileN / 2) * 128), dv = desc_k(va);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
          mma_ss(tmem + C::kColDPT + h * (kTileN / 2), sdesc_add(dv, off),
                 sdesc_add(ddo, off), kIdescTHalf, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(C::kBarDPFull + h));
        return true;
      };
      constexpr bool kDPHalves = C::kDQOverDP;
      auto issue_dp = [&](int it) -> bool {
        if (kDPHalves) return issue_dp_half(it, 0) && issue_dp_half(it, 1);
        if (!wait_bar(bar(C::kBarDOFull + it % C::kStagesDO), (it / C::kStagesDO) & 1, abort_flag, p.err))
          return false;
        tc_fence_after();
        const uint64_t ddo = desc_k(doaddr(it)), dv = desc_k(va);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
          mma_ss(tmem + C::kColDPT, sdesc_add(dv, off), sdesc_add(ddo, off),
                 kIdescT, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(C::kBarDPFull));
        mma_commit(bar(C::kBarDPFull + 1));
        return true;
      };
      // dP^T(n), over dQ(n - 1) where it shares dQ's columns: each half once
      // its columns have been read out
      auto issue_dp_over = [&](int n) -> bool {
        if (kDPHalves) {
          if (n > 0 && !wait_bar(bar(C::kBarDQFree), (n - 1) & 1, abort_flag, p.err)) return false;
          if (!issue_dp_half(n, 0)) return false;
          if (n > 0 && !wait_bar(bar(C::kBarDQFree + 1), (n - 1) & 1, abort_flag, p.err)) return false;
          return issue_dp_half(n, 1);
        }
        return issue_dp(n);
      };
      bool ok = true;
      int n = 0;               // query tiles done
      int kv = 0;              // items done
      for (int x = static_cast<int>(blockIdx.x); x < p.n_items && ok; x += static_cast<int>(gridDim.x)) {
        const int n_it = window_bwd_walk(window_bwd_cta(x, p), p).n_it;
        if (n_it == 0) continue;
        ok = wait_bar(bar(C::kBarKV), kv & 1, abort_flag, p.err) && issue_s(n) && issue_dp_over(n);
        for (int it = 0; it < n_it && ok; ++it, ++n) {
          const bool more = it + 1 < n_it;               // another query tile follows
          ok = false;
          // dV += P^T dO_i  (K dimension = the 128 queries)
          if (!wait_bar(bar(C::kBarPReady), n & 1, abort_flag, p.err)) break;
          if (it == 0 && kv > 0 && !wait_bar(bar(C::kBarDKVEmpty), (kv - 1) & 1, abort_flag, p.err)) break;
          tc_fence_after();
          const uint64_t ddo = desc_mn(doaddr(n));
#pragma unroll
          for (int kk = 0; kk < kTileM / 16; ++kk) {
            mma_ts(tmem + C::kColDV, tmem + C::kColST + C::pcol(kk),
                   sdesc_add(ddo, kk * 2048), kIdescKV,
                   (it > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(bar(C::kBarDOEmpty + n % C::kStagesDO));   // dP^T(n) and dV(n) read dO_i
          if (more && !issue_s(n + 1)) break;
          // the P/dS warps run for a while: poll gently so that the issue slots
          // they share with this warp stay theirs
          if (!wait_bar_relaxed(bar(C::kBarDSReady), n & 1, abort_flag, p.err)) break;
          tc_fence_after();
          // dQ_i = dS K_j  (M = queries, N = d, K dimension = the 128 keys); with
          // columns of its own, only after the previous dQ has been read
          if (!C::kDQOverDP && n > 0 && !wait_bar(bar(C::kBarDQFree), (n - 1) & 1, abort_flag, p.err))
            break;
          const uint64_t dds = desc_mn(dsa), dk = desc_mn(ka);
#pragma unroll
          for (int kk = 0; kk < kTileN / 16; ++kk) {
            mma_ss(tmem + C::kColDQ, sdesc_add(dds, kk * 2048),
                   sdesc_add(dk, kk * 2048), kIdescQ, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar(C::kBarDQFull));
          if (!more) mma_commit(bar(C::kBarKVEmpty));
          // dK += dS^T Q_i  (dS^T: the same tile read K-major; K dimension = queries)
          const uint64_t dq = desc_mn(qaddr(n)), dds2 = desc_k(dsa);
#pragma unroll
          for (int kk = 0; kk < kTileM / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::kChunkBytes + (kk & 3) * 32;
            mma_ss(tmem + C::kColDK, sdesc_add(dds2, off),
                   sdesc_add(dq, kk * 2048), kIdescKV,
                   (it > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(bar(C::kBarQEmpty + n % C::kStagesQ));
          ok = !more || issue_dp_over(n + 1);
        }
        if (!ok) break;
        mma_commit(bar(C::kBarDKVFull));
        ++kv;
      }
      mma_commit(bar(C::kBarMmaDone));
      drain_bar(bar(C::kBarMmaDone), 0);   // every MMA issued has completed
    }
  }
  } else if (warp < 12) {
    regs_set<WinBwdRegs<D>::kMid, WinBwdRegs<D>::kLaunchRegs>();
    // =================== P^T / dS: two warpgroups, thread = key row ===================
    // Warpgroup X (warps 4-7: X = 0, warps 8-11: X = 1) handles query columns
    // [64X, 64X + 64), 16 at a time.  Phase 1 turns S^T into P (kept in fp32
    // registers) and writes P^T (bf16) to columns [64X + 8c, 64X + 8c + 8) of
    // chunk c, which this half has already read; phase 2 forms dS from P and
    // dP^T and stores it in shared memory.
    const int X = (warp - 4) >> 2;
    const int wq = warp & 3;
    const int kr = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tST = tmem + lane_base + C::kColST;
    const uint32_t tDPT = tmem + lane_base + C::kColDPT;
    const float sl2 = p.scale_log2;
    const float scale = p.scale;
    const float INF = __int_as_float(0x7f800000);
    uint8_t* ds_row = smem + C::kDSOff + X * C::kChunkBytes + kr * 128;   // this key's dS row
    // statistics of query tile i of query head hq0 + g, negated so that
    // P = ex2(S sl2 + nl2) and dP - D = dP scale + ndl are single FMAs
    auto load_stats = [&](int bhq, int i, float& nl2, float& ndl) {
      const int q = i * kTileM + kr;
      if (q < Lq) {
        const size_t stat = static_cast<size_t>(bhq) * Lq + q;
        const float lse = __ldg(p.lse + stat);
        nl2 = (lse == -INF) ? -INF : -(lse * kLog2e);  // an empty row contributes nothing
        ndl = -(__ldg(p.delta + stat) * scale);
      } else {
        nl2 = -INF;
        ndl = 0.f;
      }
    };
    auto store_stats = [&](int n, float nl2, float ndl) {
      float* to = stats + (n & 1) * 256;
      to[kr] = nl2;
      to[128 + kr] = ndl;
      mbar_arrive(bar(C::kBarStat + (n & 1)));
    };
    // Buffer (n & 1) holds the statistics of the n-th query tile met (minus
    // the LSE in log2 units, minus scale * D).  It is rewritten (for tile n + 2)
    // by half 0 after its tile n + 1; by then dP^T(n + 1) has been issued, which
    // waited for dS(n) of both halves, so nobody reads it for tile n any more.
    bool ok = true;
    int n = 0;                 // query tiles done (over all items)
    int kv = 0;                // items with query tiles done
    for (int x = static_cast<int>(blockIdx.x); x < p.n_items && ok; x += static_cast<int>(gridDim.x)) {
    int key0, key, n_it;         // the tile's first key, this thread's
    {
    const WindowBwdCta cta = window_bwd_cta(x, p);
    const WindowQWalk walk = window_bwd_walk(cta, p);
    key0 = cta.j * kTileN;
    key = key0 + kr;
    n_it = walk.n_it;
    const int bhq0 = (cta.bh / p.Hkv) * p.H + (cta.bh % p.Hkv) * G;   // first query head of the group
    int g, i;
    walk.start(g, i);
    if (X == 0 && n_it > 0) {
      float l2, dl;
      load_stats(bhq0 + g, i, l2, dl);
      store_stats(n, l2, dl);
    }
    for (int it = 0; it < n_it; walk.advance(g, i), ++it, ++n) {
      const float* lse2 = stats + (n & 1) * 256 + 64 * X;
      const float* dlt = lse2 + 128;
      float l2n = 0.f, dln = 0.f;
      if (X == 0 && it + 1 < n_it) {
        int gn = g, in = i;
        walk.advance(gn, in);
        load_stats(bhq0 + gn, in, l2n, dln);
      }
      // (a wait that runs out is noted, and at the tile's end the warp leaves as
      // one; up to there it only spoils results that are lost already)
      bool fine = wait_bar(bar(C::kBarSFull), n & 1, abort_flag, p.err) &&
                  wait_bar(bar(C::kBarStat + (n & 1)), (n >> 1) & 1, abort_flag, p.err);
      tc_fence_after();
      // element mask: a bit for each of this half's 64 queries that sees the
      // key (those from its own position on, up to the window's end unless
      // the key is a sink; none for a key past the last one, or one of the sinks
      // that have their own kernel).  The ragged tail
      // (query >= Lq) has -lse2 = -inf, so P is 0 there already
      uint32_t seen[2];
      {
        const long long tile = static_cast<long long>(key0) - p.w.sh - static_cast<long long>(i) * kTileM;
        const int own = clamped(tile, -kTileM, kTileM) + kr - 64 * X;
        const int qlo = key < Lk && key >= p.few_sinks ? own : 64;
        const int end = key < p.w.snk ? 64 : clamped(tile + p.w.window, -kTileM, kTileM) + kr - 64 * X;
        seen[0] = bits_below(end) & ~bits_below(qlo);
        seen[1] = bits_below(end - 32) & ~bits_below(qlo - 32);
      }
      const bool need_mask = __any_sync(0xFFFFFFFFu, (seen[0] & seen[1]) != 0xFFFFFFFFu);
      // ---- phase 1: P (four chunks of 16 queries; chunk c+1's TMEM load is in
      // flight while chunk c is computed) ----
      float pf[4][16];
      {
        uint32_t sv[2][16];
        tmem_ld16(tST + 64 * X, sv[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int cur = c & 1;
          const int col = 64 * X + 16 * c;                 // first query of the chunk
          tmem_ld_wait16(sv[cur]);
          if (c + 1 < 4) tmem_ld16(tST + col + 16, sv[cur ^ 1]);
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 l4 = *reinterpret_cast<const float4*>(lse2 + 16 * c + e);
            float x[4];
            ffma2(x[0], x[1], __uint_as_float(sv[cur][e]), __uint_as_float(sv[cur][e + 1]), sl2,
                  sl2, l4.x, l4.y);
            ffma2(x[2], x[3], __uint_as_float(sv[cur][e + 2]), __uint_as_float(sv[cur][e + 3]),
                  sl2, sl2, l4.z, l4.w);
#pragma unroll
            for (int u = 0; u < 4; ++u) pf[c][e + u] = ex2(x[u]);
          }
          if (need_mask) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!((seen[c >> 1] >> (16 * (c & 1) + e)) & 1u)) pf[c][e] = 0.f;
          }
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) pk[e] = pack_bf16(pf[c][2 * e], pf[c][2 * e + 1]);
          tmem_st8(tST + 64 * X + 8 * c, pk);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(C::kBarPReady));
      // ---- phase 2: dS = P o (dP - D), into shared memory ----
      fine = wait_bar(bar(C::kBarDPFull + X), n & 1, abort_flag, p.err) && fine;
      tc_fence_after();
      {
        uint32_t dv[2][16];
        tmem_ld16(tDPT + 64 * X, dv[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int cur = c & 1;
          const int col = 64 * X + 16 * c;
          tmem_ld_wait16(dv[cur]);
          if (c + 1 < 4) tmem_ld16(tDPT + col + 16, dv[cur ^ 1]);
          uint32_t dk[8];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 d4 = *reinterpret_cast<const float4*>(dlt + 16 * c + e);
            float ds[4];
            ffma2(ds[0], ds[1], __uint_as_float(dv[cur][e]), __uint_as_float(dv[cur][e + 1]), scale,
                  scale, d4.x, d4.y);
            ffma2(ds[2], ds[3], __uint_as_float(dv[cur][e + 2]), __uint_as_float(dv[cur][e + 3]),
                  scale, scale, d4.z, d4.w);
            fmul2(ds[0], ds[1], pf[c][e], pf[c][e + 1], ds[0], ds[1]);
            fmul2(ds[2], ds[3], pf[c][e + 2], pf[c][e + 3], ds[2], ds[3]);
            if (need_mask) {          // a masked pair sends nothing, whatever dP and D hold
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (!((seen[c >> 1] >> (16 * (c & 1) + e + u)) & 1u)) ds[u] = 0.f;
            }
            dk[e / 2] = pack_bf16(ds[0], ds[1]);
            dk[e / 2 + 1] = pack_bf16(ds[2], ds[3]);
          }
          // one 128-byte row per key (queries 64X .. 64X+63), 16-byte units of
          // 8 queries swizzled by the row index: the K-major tile layout
#pragma unroll
          for (int u2 = 0; u2 < 2; ++u2) {
            const int unit = 2 * c + u2;
            *reinterpret_cast<uint4*>(ds_row + ((unit ^ (kr & 7)) * 16)) =
                make_uint4(dk[4 * u2 + 0], dk[4 * u2 + 1], dk[4 * u2 + 2], dk[4 * u2 + 3]);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bar(C::kBarDSReady));
      if (X == 0 && it + 1 < n_it) store_stats(n + 1, l2n, dln);
      if (!__all_sync(0xFFFFFFFFu, fine)) {
        ok = false;
        break;
      }
    }
    }
    // ---- an item's end: half 0 stores dK rows, half 1 stores dV rows ----
    if (ok && n_it > 0)
      ok = __all_sync(0xFFFFFFFFu, wait_bar(bar(C::kBarDKVFull), kv & 1, abort_flag, p.err));
    tc_fence_after();
    if (ok) {
      int xx = x;
      asm volatile("" : "+r"(xx));            // the item again, rather than kept in registers
      const WindowBwdCta cta = window_bwd_cta(xx, p);
      // one 128-byte line (64 columns as bf16 pairs) of this thread's key row
      // at a time; after the octet transpose every store writes whole lines
      const uint32_t tsrc = tmem + lane_base + (X == 0 ? C::kColDK : C::kColDV);
      const int wrow0 = cta.j * kTileN + wq * 32;      // this warp's first key row
      const uint32_t valid = __ballot_sync(0xFFFFFFFFu, key < Lk);
      uint8_t* base = reinterpret_cast<uint8_t*>((X == 0 ? p.dk : p.dv) +
                                                 (static_cast<size_t>(cta.bh) * Lk + wrow0) * D);
      // a cut walk leaves its fp32 part [128][D] of dK and of dV in the workspace
      uint8_t* part = reinterpret_cast<uint8_t*>(
          p.part + ((static_cast<size_t>(cta.slot) * 2 + X) * kTileN + wq * 32) * D);
#pragma unroll 1
      for (int g2 = 0; g2 < D / 64; ++g2) {
        uint32_t a[32], c[32];
        if (n_it > 0) {
          tmem_ld32(tsrc + g2 * 64, a);
          tmem_ld32(tsrc + g2 * 64 + 32, c);
          tmem_ld_wait(a);
          tmem_ld_wait(c);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = c[e] = 0u;
        }
        if (cta.nseg > 1) {
          transpose_octets(a, lane);
          store_octet_lines(a, part + g2 * 256, D * 4, 0xFFFFFFFFu, lane);
          transpose_octets(c, lane);
          store_octet_lines(c, part + g2 * 256 + 128, D * 4, 0xFFFFFFFFu, lane);
        } else {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            w[k] = pack_bf16(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1]));
            w[16 + k] = pack_bf16(__uint_as_float(c[2 * k]), __uint_as_float(c[2 * k + 1]));
          }
          transpose_octets(w, lane);
          store_octet_lines(w, base + g2 * 128, D * 2, valid, lane);
        }
      }
    }
    if (n_it > 0) {
      tc_fence_before();
      mbar_arrive(bar(C::kBarDKVEmpty));
      ++kv;
    }
    }
  } else {
    regs_set<WinBwdRegs<D>::kHigh, WinBwdRegs<D>::kLaunchRegs>();
    // =================== dQ: warps 12-15, thread = query row ===================
    // Each round moves 64 d-columns of the tile's dQ from TMEM to a
    // 128-byte-swizzled fp32 staging buffer, from which bulk tensor
    // reduce-adds (boxes of 32 columns) add it into the fp32 accumulator in
    // global memory; dQ's TMEM columns of a round are handed back right after
    // their reads.  Per-warp drain (d=128): each warp reduces its own 32 rows
    // and reuses its staging rows once its own previous reduces have read them
    // (bulk groups are per thread).  CTA-wide drain (d=64): one thread reduces
    // the 128 rows after all four warps have staged them.  (On the bench
    // shapes, vector red.global from registers, for all of dQ or for one
    // round, measured slower: the reduce stream sets the pace.)
    constexpr bool kPerWarp = C::kDrainPerWarp;
    const int wq = warp & 3;
    const int qr = wq * 32 + lane;
    const uint32_t tDQ = tmem + (static_cast<uint32_t>(wq * 32) << 16) + C::kColDQ;
    constexpr int kRounds = D / 64;
    constexpr int kBoxBytes = kTileM * 32 * 4;    // 128 rows x 32 fp32: one box column
    static_assert(2 * kBoxBytes == C::kStageBytes, "two box columns fill the staging buffer");
    const uint32_t stage = sbase + C::kStageOff + (kPerWarp ? wq * 32 * 128 : 0);
    uint8_t* stage_ptr = smem + C::kStageOff;
    bool ok = true;
    int g = 0;                                    // staged rounds (CTA-wide drain)
    int n = 0;                                    // query tiles done (over all items)
    for (int x = static_cast<int>(blockIdx.x); x < p.n_items && ok; x += static_cast<int>(gridDim.x)) {
    const WindowBwdCta cta = window_bwd_cta(x, p);
    const WindowQWalk walk = window_bwd_walk(cta, p);
    const int b = cta.bh / p.Hkv;
    const int hq0 = (cta.bh - b * p.Hkv) * G;
    int gq, i;                                    // query head of the group, query tile
    walk.start(gq, i);
    for (int it = 0; it < walk.n_it && ok; walk.advance(gq, i), ++it, ++n) {
      bool fine = wait_bar_relaxed(bar(C::kBarDQFull), n & 1, abort_flag, p.err);
      tc_fence_after();
      for (int r = 0; r < kRounds; ++r, ++g) {
        uint32_t v0[32], v1[32];
        tmem_ld32(tDQ + 64 * r, v0);
        tmem_ld32(tDQ + 64 * r + 32, v1);
        tmem_ld_wait(v0);
        tmem_ld_wait(v1);
        // d-columns [64r, 64r + 64) of this tile are read (at d=128 dP^T's
        // half r may overwrite them; at d=64 the next dQ may)
        tc_fence_before();
        mbar_arrive(bar(C::kBarDQFree + r));
        // the staging rows must have been read by the reduces that used them
        if constexpr (kPerWarp) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
        } else if (g > 0) {
          if (qr == 0) {
            bulk_wait_read_all();
            mbar_arrive(bar(C::kBarStageFree));
          }
          fine = wait_bar(bar(C::kBarStageFree), (g - 1) & 1, abort_flag, p.err) && fine;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {               // box column 0: columns 0..31 of the round
          *reinterpret_cast<uint4*>(stage_ptr + qr * 128 + ((u ^ (qr & 7)) * 16)) =
              make_uint4(v0[4 * u], v0[4 * u + 1], v0[4 * u + 2], v0[4 * u + 3]);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {               // box column 1: columns 32..63
          *reinterpret_cast<uint4*>(stage_ptr + kBoxBytes + qr * 128 + ((u ^ (qr & 7)) * 16)) =
              make_uint4(v1[4 * u], v1[4 * u + 1], v1[4 * u + 2], v1[4 * u + 3]);
        }
        fence_proxy_async_smem();
        if constexpr (kPerWarp) {
          __syncwarp();
          if (lane == 0) {
            const int row = i * kTileM + wq * 32;
            tma_reduce_add_4d(&tmDQ, stage, 64 * r, row, hq0 + gq, b);
            tma_reduce_add_4d(&tmDQ, stage + kBoxBytes, 64 * r + 32, row, hq0 + gq, b);
            bulk_commit_group();
          }
        } else {
          mbar_arrive(bar(C::kBarStaged));
          if (qr == 0) fine = wait_bar(bar(C::kBarStaged), g & 1, abort_flag, p.err) && fine;
          if (qr == 0 && fine) {
            const int row = i * kTileM;
            tma_reduce_add_4d(&tmDQ, stage, 64 * r, row, hq0 + gq, b);
            tma_reduce_add_4d(&tmDQ, stage + kBoxBytes, 64 * r + 32, row, hq0 + gq, b);
            bulk_commit_group();
          }
        }
        // reconverge before the next TMEM load, or leave as a warp
        if (!__all_sync(0xFFFFFFFFu, fine)) {
          ok = false;
          break;
        }
      }
    }
    }
    if (kPerWarp ? lane == 0 : qr == 0) bulk_wait_all();   // every reduction has landed
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// The keys query row i sees: the sinks below the window, [0, nsk), and the
// window's [lo, lo + nw).
struct RowKeys {
  int nsk, lo, nw;
};
__device__ __forceinline__ RowKeys window_row_keys(const WindowBwdParams& p, int i) {
  const long long own = static_cast<long long>(i) + p.w.sh;          // the row's own key
  const long long hi = min(own, static_cast<long long>(p.Lk) - 1);
  const long long lo = max(0ll, min(own - p.w.window + 1, static_cast<long long>(p.Lk)));
  RowKeys r;
  r.lo = static_cast<int>(lo);
  r.nw = static_cast<int>(max(0ll, hi - lo + 1));
  r.nsk = own < 0 ? 0 : static_cast<int>(min(static_cast<long long>(p.w.snk), min(lo, own + 1)));
  return r;
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float s) {
  s = fmaf(bf16lo(a.x), bf16lo(b.x), s);
  s = fmaf(bf16hi(a.x), bf16hi(b.x), s);
  s = fmaf(bf16lo(a.y), bf16lo(b.y), s);
  s = fmaf(bf16hi(a.y), bf16hi(b.y), s);
  s = fmaf(bf16lo(a.z), bf16lo(b.z), s);
  s = fmaf(bf16hi(a.z), bf16hi(b.z), s);
  s = fmaf(bf16lo(a.w), bf16lo(b.w), s);
  return fmaf(bf16hi(a.w), bf16hi(b.w), s);
}

// The rows whose D comes from its definition: below first, and from late on, as
// far as they see at most kFewKeys keys.
struct FewRows {
  long long first, late;
  __device__ __forceinline__ bool has(const RowKeys& rk, long long i) const {
    return (i < first || i >= late) && rk.nsk + rk.nw <= kFewKeys;
  }
};
bool every_row_few(const WindowMask& w, int Lk) { return w.window + w.snk <= kFewWindow || Lk <= kFewKeys; }
FewRows window_few_rows(const WindowBwdParams& p) {
  FewRows f;
  const long long Lq = p.Lq;
  if (every_row_few(p.w, p.Lk)) {
    f.first = f.late = Lq;
  } else {
    f.first = std::max(0ll, std::min(Lq, kFewKeys - p.w.sh));
    f.late = std::max(f.first, std::min(Lq, p.Lk - kFewKeys - 1 - p.w.sh + p.w.window));
  }
  return f;
}

// D_i for every row, and the fp32 dQ accumulator cleared.
//
// D_i = dO_i . O_i uses the saved O, rounded to bf16, so it is off by up to
// 2^-8 |dO_i| . |O_i|.  Over many keys O averages out and that is small beside
// the dP_ij = dO_i . V_j it is subtracted from; over a few keys it is as large
// as dQ's own rounding, and more where one key has nearly all of the weight
// (with 3 keys dQ came out 6.9e-3 off, with exact D 2.9e-3; with 63 keys of
// which one is a heavy sink 5.2e-3 and 3.3e-3).  Rows of few keys therefore
// take the definition, D_i = sum_j P_ij dP_ij, in fp32: a warp a row, two lanes
// a key, 16 keys at a time.  Rows of a wide window have few keys only near the
// first key and past the last.  Where every row has (under a window of up to 32
// keys), the sinks' kernel takes them (B1 H16(4) L16384 d128, window 28: a call in
// 255 us, a warp a row 1140).
template <int D>
__global__ void __launch_bounds__(256) attn_bwd_window_pre_kernel(const WindowBwdParams p, const FewRows fr,
                                                                  int few_blocks) {
  constexpr int G = D / 8;                           // threads per row, 16 bytes each
  const long long rows = static_cast<long long>(p.B) * p.H * p.Lq;
  // the first blocks take the rows of few keys, the others stream
  const bool takes_few = static_cast<int>(blockIdx.x) < few_blocks;
  const long long block = takes_few ? blockIdx.x : blockIdx.x - few_blocks;
  const long long tid = block * blockDim.x + threadIdx.x;
  const long long nthreads = static_cast<long long>(takes_few ? few_blocks : gridDim.x - few_blocks) * blockDim.x;
  const int g = static_cast<int>(threadIdx.x % G);
  const int lane = static_cast<int>(threadIdx.x & 31);
  const long long per = fr.first + (p.Lq - fr.late);
  const long long n = takes_few ? per * p.B * p.H : 0;
  for (long long x = tid / 32; x < n; x += nthreads / 32) {
    const long long bhq = x / per;
    long long i = x - bhq * per;
    if (i >= fr.first) i += fr.late - fr.first;
    const RowKeys rk = window_row_keys(p, static_cast<int>(i));
    if (!fr.has(rk, i)) continue;
    const int nk = rk.nsk + rk.nw;
    const long long r = bhq * p.Lq + i;
    const int b = static_cast<int>(bhq / p.H);
    const int h = static_cast<int>(bhq - static_cast<long long>(b) * p.H);
    const size_t kv = (static_cast<size_t>(b) * p.Hkv + h / (p.H / p.Hkv)) * p.Lk;
    const int half = lane & 1;
    const uint4* qr = reinterpret_cast<const uint4*>(p.q + r * D) + half * (D / 16);
    const uint4* dr = reinterpret_cast<const uint4*>(p.dout + r * D) + half * (D / 16);
    const float nl2 = nk > 0 ? -(__ldg(p.lse + r) * kLog2e) : 0.f;
    float s = 0.f;
    for (int t0 = 0; t0 < nk; t0 += 16) {
      const int t = t0 + (lane >> 1);
      float sqk = 0.f, dov = 0.f;
      if (t < nk) {
        const int key = t < rk.nsk ? t : rk.lo + (t - rk.nsk);
        const uint4* kr = reinterpret_cast<const uint4*>(p.k + (kv + key) * D) + half * (D / 16);
        const uint4* vr = reinterpret_cast<const uint4*>(p.v + (kv + key) * D) + half * (D / 16);
#pragma unroll 4
        for (int e = 0; e < D / 16; ++e) {
          sqk = dot8(__ldg(qr + e), __ldg(kr + e), sqk);
          dov = dot8(__ldg(dr + e), __ldg(vr + e), dov);
        }
      }
      sqk += __shfl_xor_sync(0xFFFFFFFFu, sqk, 1);
      dov += __shfl_xor_sync(0xFFFFFFFFu, dov, 1);
      if (t < nk) s += ex2(fmaf(sqk, p.scale_log2, nl2)) * dov;
    }
#pragma unroll
    for (int off = 2; off < 32; off <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    if (lane == 0) p.delta[r] = s;
  }
  if (takes_few) return;
  // kRows rows at a time, so that their loads are in flight together; a thread
  // clears its own 8 columns of the accumulator behind them
  constexpr int kRows = 2;
  const long long step = nthreads / G;
  const int step_row = static_cast<int>(step % p.Lq);
  int row = static_cast<int>(tid / G % p.Lq);        // r % Lq, kept beside r
  for (long long r0 = tid / G;; r0 += kRows * step) {
    if (__all_sync(0xFFFFFFFFu, r0 >= rows)) break;  // every lane of the warp is done
    uint4 o[kRows], d[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const long long r = r0 + u * step;
      o[u] = d[u] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows) {
        o[u] = __ldg(reinterpret_cast<const uint4*>(p.o + r * D) + g);
        d[u] = __ldg(reinterpret_cast<const uint4*>(p.dout + r * D) + g);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const long long r = r0 + u * step;
      const bool active = r < rows;
      if (active) {
        float4* acc = reinterpret_cast<float4*>(p.dq_acc + r * D + g * 8);
        acc[0] = acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      const bool few = active && (row < fr.first || row >= fr.late) && fr.has(window_row_keys(p, row), row);
      float s = dot8(o[u], d[u], 0.f);
#pragma unroll
      for (int off = G / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off, G);
      if (active && g == 0 && !few) p.delta[r] = s;
      row += step_row - (row >= p.Lq - step_row ? p.Lq : 0);
    }
  }
}

// The same where up to kFewSinks keys are sinks, and all that comes of the pairs
// of a query with a sink: their dQ, which the accumulator starts from, and parts
// of the sinks' dK and dV.  (few_sinks = 0: D alone, of rows of few keys.)
//
// A sink's dK and dV are sums over every later query of every head of its
// group: elements of a hundred times the other keys', of which a P and a dS
// rounded to bf16 leave 2e-3 uncertain.  (Taken by the main kernel, single
// elements near 0 came out up to 0.4 of the rms of all dK off: 4 sinks of 16384
// keys, window 1024, 4 heads a group.)  Here P and dS enter their products in
// two bf16 parts each, which hold all but 2^-15 of them.
//
// A warp takes 16 rows at a time, as mma.m16n8k16 has them, with the sinks as its
// 8 columns: S and dP = [Q; dO] [K; V]^T, then dQ = [dS, its rest] [K; K] (the
// rest takes the 8 rows that 8 sinks leave of 16), dK^T += Q^T dS and dV^T +=
// dO^T P with both parts.  A thread's 16 bytes of a row are 8 neighbouring
// d's, of which the first 4 and the last 4 stand in two steps' columns 2c, 2c + 1,
// 2c + 8 and 2c + 9.  sink_ctas CTAs of kSinkWarps warps share the rows of a
// K/V head's group, and a lane's pieces of its warp's next rows are on their way
// into its own places in shared memory (cp.async) while the warp computes.  D of
// rows of few keys comes by the same products, 8 keys at a time (a row at a
// time, as in the kernel above, the warp that meets the first rows ended 100 us
// after the others).
// Bound by HBM (Q, dO, O in, the accumulator out): 59 us for 336 MB, 5.7 TB/s, at
// B1 H16(4) L16384 d128; three CTAs an SM with the pieces in registers took 69.
// With the main kernel's walks of the sink tile gone, that call (window 1024, 4
// sinks) took 474 us instead of 462 (435 with the last wave cut, below), B4 H16
// L2000 d64 105 instead of 114, B2 H8(2) L300 29 instead of 43.
constexpr int kSinkWarps = 4;
constexpr int kSinkCtasPerSm = 2;

// Rows g and g + 8 of a warp's unit, as a lane holds them.
struct SinkRows {
  size_t head;                    // first row of the query head
  int i[2];                       // query rows
  int seen[2];                    // sinks that they see (-1: no row)
  float nl2[2];                   // minus the LSE in log2 units
};
template <int D>
struct SinkSmem {
  static constexpr int NJ = D / 32;                   // 16-byte pieces of a row a lane holds
  union {
    uint4 buf[kSinkWarps][2][3][2][NJ][32];           // [warp][stage][Q, dO, O][row][piece][lane]
    float sum[2][kFewSinks][D];
  };
  uint4 ks[NJ][32], vs[NJ][32];                       // the sinks as B of S and dP
  uint4 kt[NJ][32];                                   // K as B of dQ: tiles 4 j .. 4 j + 3
};

template <int D>
__global__ void __launch_bounds__(kSinkWarps * 32, kSinkCtasPerSm)
    attn_bwd_window_sink_kernel(const WindowBwdParams p, const FewRows fr) {
  constexpr int NJ = D / 32;
  extern __shared__ __align__(16) uint8_t sink_smem[];
  SinkSmem<D>& sm = *reinterpret_cast<SinkSmem<D>*>(sink_smem);
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, c = lane & 3;
  const int snk = p.few_sinks;
  const int bh = static_cast<int>(blockIdx.x) / p.sink_ctas;
  const int cta = static_cast<int>(blockIdx.x) - bh * p.sink_ctas;
  const int b = bh / p.Hkv, hkv = bh - b * p.Hkv;
  const int group = p.H / p.Hkv;
  const int head0 = b * p.H + hkv * group;
  // a unit: 16 rows of one of the group's heads
  const uint32_t tiles = (static_cast<uint32_t>(p.Lq) + 15) / 16, units = group * tiles;
  const uint32_t stride = p.sink_ctas * kSinkWarps;

  auto locate = [&](uint32_t unit) {
    SinkRows w;
    const uint32_t h = unit / tiles;
    w.head = static_cast<size_t>(head0 + h) * p.Lq;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      w.i[u] = static_cast<int>((unit - h * tiles) * 16) + g + 8 * u;
      const bool in = w.i[u] < p.Lq;
      w.seen[u] = in ? clamped(w.i[u] + p.w.sh + 1, 0, snk) : -1;
      w.nl2[u] = in ? -(__ldg(p.lse + w.head + w.i[u]) * kLog2e) : 0.f;
    }
    return w;
  };
  auto fetch = [&](const SinkRows& w, int stage) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const bool in = w.seen[u] >= 0;
      const size_t at = in ? (w.head + w.i[u]) * D + c * 8 : 0;
      const uint32_t to = smem_u32(&sm.buf[warp][stage][0][u][0][lane]);
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) {
        cp_async16(to + jj * 512, p.q + at + jj * 32, in);
        cp_async16(to + (2 * NJ + jj) * 512, p.dout + at + jj * 32, in);
        cp_async16(to + (4 * NJ + jj) * 512, p.o + at + jj * 32, in);
      }
    }
  };
  uint32_t unit = cta * kSinkWarps + warp;
  SinkRows w;
  if (unit < units) {
    w = locate(unit);
    fetch(w, 0);
  }
  cp_commit();

  const __nv_bfloat16* kg = p.k + static_cast<size_t>(bh) * p.Lk * D;
  const __nv_bfloat16* vg = p.v + static_cast<size_t>(bh) * p.Lk * D;
  for (int x = static_cast<int>(threadIdx.x); x < NJ * 32; x += kSinkWarps * 32) {
    const int jj = x >> 5, l = x & 31;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const size_t at = static_cast<size_t>(l >> 2) * D + jj * 32 + (l & 3) * 8;
    sm.ks[jj][l] = (l >> 2) < snk ? *reinterpret_cast<const uint4*>(kg + at) : none;
    sm.vs[jj][l] = (l >> 2) < snk ? *reinterpret_cast<const uint4*>(vg + at) : none;
    // dQ's tile 4 jj + e: columns n stand for d = 16 (2 jj + e / 2) + 4 (n / 2) + 2 (e % 2) + n % 2
    uint32_t word[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = l >> 2, s0 = 2 * (l & 3);
      const int d = 16 * (2 * jj + (e >> 1)) + 4 * (n >> 1) + 2 * (e & 1) + (n & 1);
      const unsigned short* ku = reinterpret_cast<const unsigned short*>(kg) + d;
      const uint32_t lo = s0 < snk ? ku[static_cast<size_t>(s0) * D] : 0u;
      const uint32_t hi = s0 + 1 < snk ? ku[static_cast<size_t>(s0 + 1) * D] : 0u;
      word[e] = lo | hi << 16;
    }
    sm.kt[jj][l] = make_uint4(word[0], word[1], word[2], word[3]);
  }
  __syncthreads();

  float dk[D / 16][4], dv[D / 16][4];
#pragma unroll
  for (int t = 0; t < D / 16; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[t][e] = dv[t][e] = 0.f;
  for (int stage = 0; unit < units; stage ^= 1) {
    SinkRows next = w;
    const bool more = units - unit > stride;
    if (more) {
      next = locate(unit + stride);
      fetch(next, stage ^ 1);
    }
    cp_commit();
    cp_wait<1>();                 // this unit's pieces (each lane reads what it copied)
    const uint4* q = &sm.buf[warp][stage][0][0][0][lane];           // piece jj of row u: [(u NJ + jj) 32]
    const uint4* d_o = q + 2 * NJ * 32;
    const uint4* o = q + 4 * NJ * 32;
    // ---- D: the diagonals of dO O^T, rows 0-7 and 8-15; row g's lies with c = g / 2 ----
    float dd[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const uint4 d0 = d_o[jj * 32], d1 = d_o[(NJ + jj) * 32], o0 = o[jj * 32], o1 = o[(NJ + jj) * 32];
      mma16816<false>(dd[0], d0.x, d1.x, d0.y, d1.y, o0.x, o0.y);
      mma16816<false>(dd[1], d0.x, d1.x, d0.y, d1.y, o1.x, o1.y);
      mma16816<false>(dd[0], d0.z, d1.z, d0.w, d1.w, o0.z, o0.w);
      mma16816<false>(dd[1], d0.z, d1.z, d0.w, d1.w, o1.z, o1.w);
    }
    // ---- S and dP: rows g (0, 1) and g + 8 (2, 3), sinks 2 c and 2 c + 1 ----
    auto products = [&](float (&sc)[4], float (&dp)[4], const uint4& kf, const uint4& vf, int jj) {
      const uint4 q0 = q[jj * 32], q1 = q[(NJ + jj) * 32], d0 = d_o[jj * 32], d1 = d_o[(NJ + jj) * 32];
      mma16816<false>(sc, q0.x, q1.x, q0.y, q1.y, kf.x, kf.y);
      mma16816<false>(dp, d0.x, d1.x, d0.y, d1.y, vf.x, vf.y);
      mma16816<false>(sc, q0.z, q1.z, q0.w, q1.w, kf.z, kf.w);
      mma16816<false>(dp, d0.z, d1.z, d0.w, d1.w, vf.z, vf.w);
    };
    float sc[4] = {0.f, 0.f, 0.f, 0.f}, dp[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) products(sc, dp, sm.ks[jj][lane], sm.vs[jj][lane], jj);
    float pr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      pr[e] = 2 * c + (e & 1) < w.seen[e >> 1] ? ex2(fmaf(sc[e], p.scale_log2, w.nl2[e >> 1])) : 0.f;
    // ---- D of rows of few keys: the sum of P dP over the sinks and, 8 keys at a
    // time, the others: sinks past those, then the window ----
    float dl[2];
    bool few[2];
    int from[2] = {snk, p.Lk}, to[2] = {-1, -1}, lo[2], hi[2], nsk[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      dl[u] = __shfl_sync(0xFFFFFFFFu, (g & 1) ? dd[u][2 * u + 1] : dd[u][2 * u], (lane & 28) | (g >> 1));
      few[u] = false;
      if (w.seen[u] >= 0 && (w.i[u] < fr.first || w.i[u] >= fr.late)) {
        const RowKeys rk = window_row_keys(p, w.i[u]);
        few[u] = fr.has(rk, w.i[u]);
        lo[u] = max(rk.lo, snk);
        hi[u] = rk.lo + rk.nw - 1;
        nsk[u] = rk.nsk;
        if (few[u]) to[0] = max(to[0], nsk[u] - 1);
        if (few[u] && lo[u] <= hi[u]) {
          from[1] = min(from[1], lo[u]);
          to[1] = max(to[1], hi[u]);
        }
      }
    }
    if (__any_sync(0xFFFFFFFFu, few[0] || few[1])) {
      float y[2] = {pr[0] * dp[0] + pr[1] * dp[1], pr[2] * dp[2] + pr[3] * dp[3]};
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        const int end = __reduce_max_sync(0xFFFFFFFFu, part ? to[1] : to[0]);
#pragma unroll 1
        for (int k0 = __reduce_min_sync(0xFFFFFFFFu, part ? from[1] : from[0]); k0 <= end; k0 += 8) {
          const size_t at = static_cast<size_t>(min(k0 + g, p.Lk - 1)) * D + c * 8;
          float sk[4] = {0.f, 0.f, 0.f, 0.f}, dk8[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int jj = 0; jj < NJ; ++jj)
            products(sk, dk8, __ldg(reinterpret_cast<const uint4*>(kg + at + jj * 32)),
                     __ldg(reinterpret_cast<const uint4*>(vg + at + jj * 32)), jj);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int u = e >> 1, key = k0 + 2 * c + (e & 1);
            if (few[u] && (part ? key >= lo[u] && key <= hi[u] : key < nsk[u]))
              y[u] = fmaf(ex2(fmaf(sk[e], p.scale_log2, w.nl2[u])), dk8[e], y[u]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        y[u] += __shfl_xor_sync(0xFFFFFFFFu, y[u], 1);
        y[u] += __shfl_xor_sync(0xFFFFFFFFu, y[u], 2);
        if (few[u]) dl[u] = y[u];
      }
    }
    float4* acc[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (w.seen[u] >= 0 && c == 0) p.delta[w.head + w.i[u]] = dl[u];
      acc[u] = reinterpret_cast<float4*>(p.dq_acc + (w.head + w.i[u]) * D) + c;
    }
    if (snk == 0) {               // D alone was wanted
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          if (w.seen[u] >= 0) acc[u][4 * x] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!more) break;
      w = next;
      unit += stride;
      continue;
    }
    // ---- P and dS = scale P (dP - D), each as two bf16 parts ----
    float ds[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      ds[e] = 2 * c + (e & 1) < w.seen[e >> 1] ? pr[e] * (dp[e] * p.scale - dl[e >> 1] * p.scale) : 0.f;
    uint32_t ph[2], pl[2], sh[2], sl[2];              // rows g, g + 8
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ph[u] = high_bf16(pr[2 * u], pr[2 * u + 1]);
      pl[u] = pack_bf16(low_part(pr[2 * u]), low_part(pr[2 * u + 1]));
      sh[u] = high_bf16(ds[2 * u], ds[2 * u + 1]);
      sl[u] = pack_bf16(low_part(ds[2 * u]), low_part(ds[2 * u + 1]));
    }
    // ---- dQ: columns 4 c .. 4 c + 3 of every 16 ----
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const uint4 kt = sm.kt[jj][lane];
      const uint32_t kw[4] = {kt.x, kt.y, kt.z, kt.w};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float y0[4] = {0.f, 0.f, 0.f, 0.f}, y1[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816<false>(y0, sh[0], sh[1], sl[0], sl[1], kw[2 * x], kw[2 * x]);
        mma16816<false>(y1, sh[0], sh[1], sl[0], sl[1], kw[2 * x + 1], kw[2 * x + 1]);
        if (w.seen[0] >= 0) acc[0][4 * (2 * jj + x)] = make_float4(y0[0], y0[1], y1[0], y1[1]);
        if (w.seen[1] >= 0) acc[1][4 * (2 * jj + x)] = make_float4(y0[2], y0[3], y1[2], y1[3]);
      }
    }
    // ---- dK^T += Q^T dS, dV^T += dO^T P: 16 d's a tile, as S's steps have them ----
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ph[u] = movm(ph[u]);
      pl[u] = movm(pl[u]);
      sh[u] = movm(sh[u]);
      sl[u] = movm(sl[u]);
    }
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const uint4 q0 = q[jj * 32], q1 = q[(NJ + jj) * 32], d0 = d_o[jj * 32], d1 = d_o[(NJ + jj) * 32];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t a0 = movm(x ? q0.z : q0.x), a1 = movm(x ? q0.w : q0.y);
        const uint32_t a2 = movm(x ? q1.z : q1.x), a3 = movm(x ? q1.w : q1.y);
        const uint32_t b0 = movm(x ? d0.z : d0.x), b1 = movm(x ? d0.w : d0.y);
        const uint32_t b2 = movm(x ? d1.z : d1.x), b3 = movm(x ? d1.w : d1.y);
        mma16816<false>(dk[2 * jj + x], a0, a1, a2, a3, sh[0], sh[1]);
        mma16816<false>(dv[2 * jj + x], b0, b1, b2, b3, ph[0], ph[1]);
        mma16816<false>(dk[2 * jj + x], a0, a1, a2, a3, sl[0], sl[1]);
        mma16816<false>(dv[2 * jj + x], b0, b1, b2, b3, pl[0], pl[1]);
      }
    }
    if (!more) break;
    w = next;
    unit += stride;
  }
  if (snk == 0) return;
  __syncthreads();                // the buffers become the warps' sums
  // ---- the warps' sums, added one warp after the other ----
  for (int turn = 0; turn < kSinkWarps; ++turn) {
    if (warp == turn) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // rows g (0, 1) and g + 8 (2, 3) of tile t
          const int d = 32 * (t >> 1) + 8 * (g >> 1) + 4 * (t & 1) + (e & 2) + (g & 1);
          const int s = 2 * c + (e & 1);
          sm.sum[0][s][d] = (turn == 0 ? 0.f : sm.sum[0][s][d]) + dk[t][e];
          sm.sum[1][s][d] = (turn == 0 ? 0.f : sm.sum[1][s][d]) + dv[t][e];
        }
    }
    __syncthreads();
  }
  float* to = p.sink_part + static_cast<size_t>(blockIdx.x) * (2 * kFewSinks * D);
  const float* from = &sm.sum[0][0][0];
  for (int x = static_cast<int>(threadIdx.x); x < 2 * kFewSinks * D; x += kSinkWarps * 32) to[x] = from[x];
}

// dK and dV of the cut walks, their parts added in segment order, and of the
// sinks that have a kernel of their own, its CTAs' parts added by a warp for
// every 4 columns; and dQ (bf16) from the fp32 accumulator (the scale was applied
// to dS already).
template <int D>
__global__ void __launch_bounds__(256) attn_bwd_window_post_kernel(const WindowBwdParams p) {
  const long long tid = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long nthreads = static_cast<long long>(gridDim.x) * blockDim.x;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const long long sink_cols = 2ll * p.B * p.Hkv * p.few_sinks * (D / 4);
  for (long long x = tid / 32; x < sink_cols; x += nthreads / 32) {
    const int c4 = static_cast<int>(x % (D / 4));
    const long long y = x / (D / 4);
    const int key = static_cast<int>(y % p.few_sinks);
    const int which = static_cast<int>(y / p.few_sinks % 2);     // 0: dK, 1: dV
    const long long bh = y / p.few_sinks / 2;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = lane; i < p.sink_ctas; i += 32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p.sink_part) +
                             (((bh * p.sink_ctas + i) * 2 + which) * kFewSinks + key) * (D / 4) + c4);
      s.x += a.x;
      s.y += a.y;
      s.z += a.z;
      s.w += a.w;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, off);
      s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, off);
      s.z += __shfl_xor_sync(0xFFFFFFFFu, s.z, off);
      s.w += __shfl_xor_sync(0xFFFFFFFFu, s.w, off);
    }
    if (lane == 0)
      *(reinterpret_cast<uint2*>((which ? p.dv : p.dk) + (bh * p.Lk + key) * D) + c4) =
          make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  }
  // one thread per 4 columns of a row of dK or dV of a cut tile
  const int BH = p.B * p.Hkv;
  const long long per_tile = 2ll * kTileN * D / 4;
  for (int c = 0; c < 2; ++c) {
    const WindowTiles t = p.tiles[c];
    if (t.seg == 1) continue;
    const long long n = static_cast<long long>(BH) * t.n * per_tile;
    for (long long x = tid; x < n; x += nthreads) {
      const int z = static_cast<int>(x / per_tile);            // tile and K/V head, as in the items
      const int e = static_cast<int>(x - z * per_tile);
      const int jj = z / BH;
      const int bh = z - jj * BH;
      const int j = t.j0 + jj;
      const int nseg = t.seg;
      const long long slot = t.slot0 + static_cast<long long>(z) * nseg;
      const int which = e / (kTileN * D / 4);                  // 0: dK, 1: dV
      const int rest = e - which * (kTileN * D / 4);
      const int r = rest / (D / 4);
      const int c4 = rest - r * (D / 4);
      const int key = j * kTileN + r;
      if (key >= p.Lk || key < p.few_sinks) continue;          // (those sinks are written above)
      const float4* src = reinterpret_cast<const float4*>(p.part) +
                          (static_cast<size_t>(slot) * 2 + which) * (kTileN * D / 4) + rest;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < nseg; ++i) {
        const float4 a = __ldg(src + static_cast<size_t>(i) * 2 * (kTileN * D / 4));
        s.x += a.x;
        s.y += a.y;
        s.z += a.z;
        s.w += a.w;
      }
      uint2 w;
      w.x = pack_bf16(s.x, s.y);
      w.y = pack_bf16(s.z, s.w);
      *(reinterpret_cast<uint2*>((which ? p.dv : p.dk) + (static_cast<size_t>(bh) * p.Lk + key) * D) + c4) = w;
    }
  }
  const long long n8 = static_cast<long long>(p.B) * p.H * p.Lq * D / 8;
  for (long long x = tid; x < n8; x += nthreads) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p.dq_acc) + 2 * x);
    const float4 b = __ldg(reinterpret_cast<const float4*>(p.dq_acc) + 2 * x + 1);
    uint4 w;
    w.x = pack_bf16(a.x, a.y);
    w.y = pack_bf16(a.z, a.w);
    w.z = pack_bf16(b.x, b.y);
    w.w = pack_bf16(b.z, b.w);
    reinterpret_cast<uint4*>(p.dq)[x] = w;
  }
}

// How the walks are cut, and where the parts go.
struct WindowBwdPlan {
  int nk, nst;
  WindowTiles tiles[2];
  long long slots, n_cta;
  bool persistent;
  int sink_ctas, few_sinks;
  size_t part_off, sink_off, bytes;
};
WindowBwdPlan window_bwd_plan(int B, int H, int Hkv, int Lq, int Lk, int d, const WindowMask& w) {
  WindowBwdPlan pl{};
  const long long nq = (static_cast<long long>(Lq) + kTileM - 1) / kTileM;
  const long long G = H / Hkv, BH = static_cast<long long>(B) * Hkv;
  pl.nk = static_cast<int>((static_cast<long long>(Lk) + kTileN - 1) / kTileN);
  const long long sink_tiles = (static_cast<long long>(w.snk) + kTileN - 1) / kTileN;
  // a few sinks have a kernel of their own; the main kernel walks their tile for
  // the windows over its other keys alone
  if (w.snk <= kFewSinks && Lq - 1 + w.sh >= 0) pl.few_sinks = w.snk;
  // ... which also takes D where every row has it from its definition
  if (pl.few_sinks > 0 || every_row_few(w, Lk)) {
    const long long units = G * ((static_cast<long long>(Lq) + 15) / 16);
    pl.sink_ctas = static_cast<int>(std::max(1ll, std::min((units + kSinkWarps - 1) / kSinkWarps,
                                                           152ll * kSinkCtasPerSm / BH)));
  }
  pl.nst = pl.few_sinks > 0 ? 0 : static_cast<int>(sink_tiles);
  // query tiles that a tile without sinks meets at most, over its heads
  const long long share = std::min(nq, std::min<long long>(w.window, 1ll << 40) / kTileM + 2) * G;
  const long long rest = pl.nk - pl.nst;
  long long seg_w = 1;
  // too few key tiles for the 152 SMs: cut every walk so that the CTAs make a wave
  const long long tiles = BH * (rest > 0 ? rest : 1);
  if (tiles < 152) seg_w = std::max(1ll, std::min(share, 152 / tiles));
  // A CTA an SM that takes items by a fixed stride saves an item's set-up
  // (5-8 % over walks of up to 12 tiles); over longer walks, whose lengths
  // differ more, a CTA an item is balanced better by the hardware (equal at 17
  // to 36 tiles, 10 % better at 68: B2 H16(4) L8192, windows of 64 to 8192).
  pl.persistent = share <= 20 * seg_w;
  // a sink tile meets up to nq tiles a head: segments as long as the others'
  // walks, but of at least 8 tiles (a part costs as much memory as 2 tiles)
  const long long each = std::max(8ll, (share + seg_w - 1) / seg_w);
  long long seg_s = std::max(1ll, (nq * G + each - 1) / each);
  // ... and no more of them than 8 an SM: many sink tiles fill the GPU uncut,
  // and their parts would take more memory than everything else (16384 sinks
  // of 16384 keys, 32 heads, d=128: 8.6 GB)
  if (pl.nst > 0) seg_s = std::max(1ll, std::min(seg_s, 152 * 8 / (BH * pl.nst)));
  // The segments of the sink tiles come first: with the last tiles' whole walks
  // they would end late (B1 H16(4) L16384 d128, window 1024, sinks 4: 17 us of
  // 395 more).  Cutting the walks of a last wave that leaves SMs idle into four
  // cost more than it gave there (104 items of 40 tiles on 152 SMs: 6 us more).
  pl.tiles[0] = WindowTiles{0, pl.nst, static_cast<int>(seg_s), 0, 0};
  pl.tiles[1] = WindowTiles{pl.nst, static_cast<int>(rest), static_cast<int>(seg_w), 0, 0};
  // Without the sinks' segments, which filled the SMs beside a last wave of
  // items that leaves some idle, its walks are cut to fill them (where they are
  // not short already, at the sequence's end): 474 -> 436 us at B1 H16(4) L16384
  // d128, window 1024.
  if (pl.few_sinks > 0 && seg_w == 1 && BH * rest > 152) {
    const long long nt = (BH * rest % 152 + BH - 1) / BH;         // key tiles of the last wave
    const long long cut = nt > 0 ? std::min(share, 152 / (nt * BH)) : 1;
    if (cut > 1 && share / G <= nt) {
      pl.tiles[0] = WindowTiles{0, static_cast<int>(rest - nt), 1, 0, 0};
      pl.tiles[1] = WindowTiles{static_cast<int>(rest - nt), static_cast<int>(nt), static_cast<int>(cut), 0, 0};
    }
  }
  for (WindowTiles& t : pl.tiles) {
    if (t.n == 0) t.seg = 1;
    t.item0 = static_cast<int>(std::min(pl.n_cta, 0x7FFFFFFFll));       // (a launch that passes it is refused)
    t.slot0 = static_cast<int>(std::min(pl.slots, 0x7FFFFFFFll));
    pl.n_cta += BH * t.n * t.seg;
    if (t.seg > 1) pl.slots += BH * t.n * t.seg;
  }
  pl.part_off = (static_cast<size_t>(B) * H * Lq * d * 4 + 255) & ~static_cast<size_t>(255);
  pl.sink_off = pl.part_off + static_cast<size_t>(pl.slots) * 2 * kTileN * d * 4;
  pl.bytes = pl.sink_off + (pl.few_sinks > 0 ? static_cast<size_t>(BH) * pl.sink_ctas * 2 * kFewSinks * d * 4 : 0);
  return pl;
}

unsigned window_grid(long long work) {
  return static_cast<unsigned>(std::max(1ll, std::min(152ll * 16, (work + 255) / 256)));
}

template <int D>
cudaError_t launch_window_bwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CUtensorMap& tdq, const WindowBwdParams& p,
                              long long n_cta, bool persistent, cudaStream_t st) {
  using C = WinBwdCfg<D>;
  auto kern = attn_bwd_window_kernel<D>;
  constexpr int kMaxDev = 64;
  static bool configured[kMaxDev] = {};  // the attribute is per device and function
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs < static_cast<int>(WinBwdRegs<D>::kLaunchRegs)) return cudaErrorInvalidConfiguration;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attn_bwd_window_sink_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sizeof(SinkSmem<D>)));
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const long long rows = static_cast<long long>(p.B) * p.H * p.Lq;
  const FewRows few = window_few_rows(p);
  if (p.sink_ctas > 0) {
    attn_bwd_window_sink_kernel<D><<<static_cast<unsigned>(p.B * p.Hkv * p.sink_ctas), kSinkWarps * 32,
                                     sizeof(SinkSmem<D>), st>>>(p, few);
  } else {
    const long long n_few = (few.first + p.Lq - few.late) * p.B * p.H;
    const int few_blocks = n_few > 0 ? static_cast<int>(window_grid(n_few * 32)) : 0;
    // (together no more than the two waves that either takes alone)
    const int stream_blocks =
        std::max(1, std::min(static_cast<int>(window_grid(rows * (D / 8))), std::max(152 * 8, 152 * 16 - few_blocks)));
    attn_bwd_window_pre_kernel<D><<<stream_blocks + few_blocks, 256, 0, st>>>(p, few, few_blocks);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  WindowBwdParams pm = p;
  if (p.few_sinks > 0) pm.w.snk = 0;
  // optional timing of the main kernel alone (attn_bwd_time_main)
  cudaEvent_t begin, end;
  bwd_main_events(&begin, &end);
  if (begin && (e = cudaEventRecord(begin, st)) != cudaSuccess) return e;
  if (n_cta > 0) {
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(persistent ? std::min<long long>(n_cta, sms) : n_cta);
    kern<<<grid, C::kThreads, C::kSmemBytes, st>>>(tq, tk, tv, tdo, tdq, pm);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (end && (e = cudaEventRecord(end, st)) != cudaSuccess) return e;
  attn_bwd_window_post_kernel<D><<<window_grid(rows * D / 8), 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace bss

using namespace bss;

extern "C" size_t attn_bwd_window_workspace_bytes(int B, int H, int H_kv, int Lq, int Lk, int d,
                                                  int64_t window, int64_t sinks, int64_t q_offset,
                                                  int64_t k_offset) {
  WindowMask w;
  if (check_common(B, H, Lq, Lk, d, 1.f) != ATTN_OK || !valid_kv_heads(H, H_kv)) return 0;
  if (Lq > kMaxTokens || Lk > kMaxTokens) return 0;      // as the call refuses them
  if (!window_mask(&w, Lk, window, sinks, q_offset, k_offset)) return 0;
  return window_bwd_plan(B, H, H_kv, Lq, Lk, d, w).bytes;
}

extern "C" attn_status_t attn_bwd_window(const void* q, const void* k, const void* v, const void* o,
                                         const float* lse, const void* dout, void* dq, void* dk,
                                         void* dv, float* delta, void* workspace,
                                         size_t workspace_bytes, int B, int H, int H_kv, int Lq,
                                         int Lk, int d, float scale, int64_t window, int64_t sinks,
                                         int64_t q_offset, int64_t k_offset, void* stream) {
  attn_status_t s = check_common(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  if (!valid_kv_heads(H, H_kv)) return ATTN_ERR_INVALID_ARG;
  if (Lq > kMaxTokens || Lk > kMaxTokens) return ATTN_ERR_UNSUPPORTED;
  WindowBwdParams p{};
  if (!window_mask(&p.w, Lk, window, sinks, q_offset, k_offset)) return ATTN_ERR_INVALID_ARG;
  const WindowBwdPlan pl = window_bwd_plan(B, H, H_kv, Lq, Lk, d, p.w);
  if (workspace_bytes < pl.bytes) return ATTN_ERR_WORKSPACE;
  if (pl.n_cta > 0x7FFF0000ll || pl.slots > 0x7FFF0000ll) return ATTN_ERR_UNSUPPORTED;
  // empty tensors may have no address
  const void* of_keys[] = {k, v, dk, dv};
  for (const void* ptr : of_keys)
    if (Lk > 0 && (!ptr || !aligned16(ptr))) return ATTN_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (Lq == 0) {                 // no query sends anything
    const size_t bytes = static_cast<size_t>(B) * H_kv * Lk * d * 2;
    if (bytes == 0) return ATTN_OK;
    s = cuda_status("attn_bwd_window clear", cudaMemsetAsync(dk, 0, bytes, st));
    return s != ATTN_OK ? s : cuda_status("attn_bwd_window clear", cudaMemsetAsync(dv, 0, bytes, st));
  }
  const void* of_queries[] = {q, o, dout, dq, workspace};
  for (const void* ptr : of_queries)
    if (!ptr || !aligned16(ptr)) return ATTN_ERR_INVALID_ARG;
  if (!lse || !delta || !aligned4(lse) || !aligned4(delta)) return ATTN_ERR_INVALID_ARG;
  if (Lk == 0) k = v = q;        // no key is read
  if ((s = get_encoder()) != ATTN_OK) return s;
  if ((s = status_word(&p.err)) != ATTN_OK) return s;
  CUtensorMap tq, tk, tv, tdo, tdq;
  if ((s = make_map(&tq, q, B, H, Lq, d)) != ATTN_OK) return s;
  if ((s = make_map(&tk, k, B, H_kv, Lk, d)) != ATTN_OK) return s;
  if ((s = make_map(&tv, v, B, H_kv, Lk, d)) != ATTN_OK) return s;
  if ((s = make_map(&tdo, dout, B, H, Lq, d)) != ATTN_OK) return s;
  const int box = d == 128 ? WinBwdCfg<128>::kDrainBoxRows : WinBwdCfg<64>::kDrainBoxRows;
  if ((s = make_map_f32(&tdq, workspace, B, H, Lq, d, box)) != ATTN_OK) return s;
  p.B = B;
  p.H = H;
  p.Hkv = H_kv;
  p.Lq = Lq;
  p.Lk = Lk;
  p.scale = scale;
  p.scale_log2 = scale * kLog2e;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.o = static_cast<const __nv_bfloat16*>(o);
  p.dout = static_cast<const __nv_bfloat16*>(dout);
  p.lse = lse;
  p.delta = delta;
  p.dq_acc = static_cast<float*>(workspace);
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.part_off);
  p.sink_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.sink_off);
  p.sink_ctas = pl.sink_ctas;
  p.few_sinks = pl.few_sinks;
  p.nk = pl.nk;
  p.nst = pl.nst;
  for (int i = 0; i < 2; ++i) p.tiles[i] = pl.tiles[i];
  p.n_items = static_cast<int>(pl.n_cta);
  return cuda_status("attn_bwd_window launch",
                     d == 64 ? launch_window_bwd<64>(tq, tk, tv, tdo, tdq, p, pl.n_cta, pl.persistent, st)
                             : launch_window_bwd<128>(tq, tk, tv, tdo, tdq, p, pl.n_cta, pl.persistent, st));
}
