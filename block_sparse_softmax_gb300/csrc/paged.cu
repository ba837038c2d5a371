// attn_decode_paged: attention of one new token per sequence over a paged
// key/value cache.
//
// Mathematics: for every sequence s and query head h, over the keys j it sees
// (j < n, and with a window j >= n - window or j < sinks),
//     O = sum_j p_j V_j / l,  p_j = exp(scale q . k_j - m),  l = sum_j p_j,
// kept as the running state (m, l, A) of the online softmax, so that any cut
// of the keys can be joined afterwards: with m* = max m_c,
//     l* = sum_c e^{m_c - m*} l_c,   A* = sum_c e^{m_c - m*} A_c.
//
// What bounds it: every key and value is read once and used for the few query
// heads of its group, so HBM bandwidth.  Hence:
//   * The work is cut evenly, whatever the lengths: the steps (16 or 32 keys)
//     of every unit (sequence, K/V head, group of up to 16 query heads) form
//     one line, and every resident warp takes an equal stretch of it.  A unit
//     that lies whole in a stretch is written out; the (at most two) units a
//     warp has only a part of leave their state in the workspace, two slots a
//     warp, and a second kernel, launched programmatically so that it is set
//     up beside the first, joins them in order.  The warps of a CTA share
//     nothing: when they took a unit's tiles in turn and merged at its end,
//     each end cost its CTA 4 us (32 sequences of up to 8192 tokens: the CTAs
//     were done after 28 to 44 us, the warps are after 31 to 40).  Where every
//     unit is short, a CTA a unit in one launch does instead (decode_small).
//   * TMA brings a step's K and V rows (boxes of 16 rows of a page) into the
//     warp's own ring of stages, swizzled for ldmatrix: one lane's four to
//     eight instructions a step.  Only a step with keys that are not seen (a
//     sequence's end, a window's edge) is copied row by row with cp.async,
//     which leaves those rows out and fills in zeros.  The next unit's first
//     steps and its Q are on their way before this unit's state goes out.
//   * The products run transposed on mma.m16n8k16: S^T = K Q^T has 16 keys as
//     rows and 8 query heads as columns, A^T = V^T P^T has 16 columns of d as
//     rows.  A group of up to 8 query heads then costs one tile of N = 8, the
//     16-row side is always full, and a thread's accumulators belong to the
//     same two heads as its softmax state.  (tcgen05 tiles have at least 64
//     rows and would be fed through shared memory twice; these products take a
//     tenth of the time the bytes do.)
//   * Over bf16 pages P enters its product in two bf16 parts, which together
//     hold all but 2^-15 of it: one part alone put 1.4e-3 (in norm) on top of
//     O's own rounding of 1.65e-3.  The bytes leave room for the second
//     product: within 0.3 % on the first and third line below, 1 % on the last.
//   * e4m3 pages are read as they are (half the bytes); a pair of elements
//     becomes fp16 by one conversion, exactly, on the way into an fp16 MMA.
//     (Going on to bf16 takes four instructions: 128 sequences of up to 16384
//     tokens took 174 us that way, 150 so.)  So that Q and P lose nothing
//     there that bf16 holds, a head's Q is scaled by a power of two (largest
//     element in [128, 256)) and P by 2^12: fp16 then rounds by at most 2^-32
//     of Q's largest element, 2^-37 of P's.  The caches' scales multiply the
//     score and the output.
// Measured (GPU time, d=128, 4 K/V heads of 4 query heads where not said):
//   2 sequences of 131071 tokens, 8 heads    161 us, 6.7 TB/s (98 % of a copy's)
//   128 of up to 16384 tokens, e4m3          150 us, 6.1 TB/s (91 %)
//   32 of up to 8192 tokens                   50 us, 4.7 TB/s (69 %)
//   64 of up to 16384 tokens, window 1000,
//     4 sinks, d=64, 16 heads                 46 us, 4.7 TB/s (69 %)
// What the last two lose is about 6 us until the first keys land (lengths,
// table and data, one after the other), 4 us between the first and the last
// warp's end, 5 us for the join and 4 us for the two launches.
#include <algorithm>

#include "mma.cuh"
#include "paged.cuh"

namespace bss {
namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;

struct DecodeParams {
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t* k;
  const uint8_t* v;
  size_t k_stride, v_stride;     // bytes from page to page
  const float* k_scale;
  const float* v_scale;
  const int* table;
  int t_row, t_head;             // its entries from sequence to sequence, from K/V head to K/V head
  bool selected;                 // attn_decode_selected: a row of negative length is nobody's
  const int* lens;
  __nv_bfloat16* o;
  float* lse;
  int2* meta;                    // [workers]: .x the unit whose first part the warp leaves in slot 1
                                 // (-1: none), .y the last warp with a part of it (slots 0)
  float* part;                   // [workers][2][rows][d + 2]: A, m (log2 units), l of the parts
  int rows;                      // query heads of a part (8 or 16)
  int S, H, Hkv, G, M, P;
  int page_log2;
  int q_tiles;                   // groups of 16 query heads of a K/V head
  float scale_log2;
  long long window;
  int sinks;
  int* err;
};

// The tokens a row of the table has room for.
__device__ __forceinline__ int most_tokens(const DecodeParams& p) {
  return static_cast<int>(min(static_cast<long long>(p.M) << p.page_log2, static_cast<long long>(kMaxTokens)));
}

// The steps of KEYS keys a sequence's query reads: the sinks' steps [0,
// nsink), then [first, first + rest).
template <int KEYS>
struct SeqSteps {
  int n, lo, sk;                 // length, first key of the window, sinks below it
  int nsink, first, total;
  __device__ __forceinline__ int key(int t) const {
    return KEYS * (t < nsink ? t : first + (t - nsink));
  }
  __device__ __forceinline__ bool seen(int j) const { return j < n && (j >= lo || j < sk); }
  // every key of the step is seen
  __device__ __forceinline__ bool whole(int key) const {
    return key + KEYS <= n && (key >= lo || key + KEYS <= sk);
  }
};
template <int KEYS>
__device__ __forceinline__ SeqSteps<KEYS> seq_steps(int n, const DecodeParams& p) {
  SeqSteps<KEYS> q;
  q.n = min(max(n, 0), most_tokens(p));
  q.lo = p.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(q.n) - p.window)) : 0;
  q.sk = min(p.sinks, q.lo);
  q.first = q.lo / KEYS;
  q.nsink = min((q.sk + KEYS - 1) / KEYS, q.first);
  q.total = q.nsink + (q.n + KEYS - 1) / KEYS - q.first;
  return q;
}

template <int D, bool FP8, int NT>
struct DecCfg {
  static constexpr int kItem = FP8 ? 1 : 2;
  static constexpr int kRowBytes = D * kItem;
  static constexpr int kKeys = kRowBytes == 256 ? 16 : 32;       // keys of a step
  static constexpr int kRowTiles = kKeys / 16;
  static constexpr int kHalves = kRowBytes > 128 ? 2 : 1;        // boxes across d
  static constexpr int kBoxBytes = 16 * (kRowBytes / kHalves);
  static constexpr int kTileBytes = kHalves * kBoxBytes;         // 16 rows of K or V
  static constexpr int kHalfBytes = kRowTiles * kTileBytes;      // K or V rows of a step
  static constexpr int kStageBytes = 2 * kHalfBytes;
  // Steps of a warp's ring: 16 KB a warp, and three CTAs an SM (two where a
  // group has more than 8 query heads, for the registers).  Two CTAs with
  // three stages measured 3 to 5 % slower, steps of 16 keys 3 % slower on
  // e4m3 pages.
  static constexpr int kStages = kStageBytes == 8192 ? 2 : 4;
  static constexpr int kCtas = NT == 1 ? 3 : 2;
  static constexpr int kRing = kDecWarps * kStages * kStageBytes;
  static constexpr int kBarOff = kRing;                          // mbarriers of every warp's stages
  static constexpr int kSumsOff = kBarOff + kDecWarps * kStages * 8;
  static constexpr int kFoundOff = kSumsOff + kDecWarps * 8;     // each warp's first sequence, steps before it
  static constexpr int kEdgeOff = kFoundOff + kDecWarps * 16;    // where its warps' stretches begin
  static constexpr int kAbortOff = kEdgeOff + (kDecWarps + 1) * 8;
  static constexpr int kSmem = kAbortOff + 16;
  static_assert(kSmem <= 233472 / 3 - 1024, "three CTAs an SM");
};

// Byte offset of 16-byte unit u of row r of 16 rows as TMA lays them out: boxes
// of 128-byte rows with unit ^ (row & 7), or 64-byte rows with unit ^ (row / 2
// & 3); the 8 rows one ldmatrix reads hit 8 different 16-byte banks.
template <int ROW>
__device__ __forceinline__ int dec_off(int r, int u) {
  if constexpr (ROW >= 128) return (u >> 3) * 2048 + r * 128 + (((u & 7) ^ (r & 7)) << 4);
  else return r * ROW + ((u ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// e4m3x2_f16x2 of the high 16 bits.
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(y) : "r"(x));
  return y;
}

// P's rest beside its high half (high_bf16), of which bf16 holds all but 2^-15 of
// P.  It is kept above 0: 0 times an infinity in V would turn it into a NaN.
__device__ __forceinline__ float p_rest(float x) {
  return fmaxf(low_part(x), 1.17549435e-38f);
}

// The running state of a unit in one warp: A^T fragments, and for the thread's
// two heads of each N tile the max (log2 units) and this thread's part of l.
template <int D, int NT>
struct DecState {
  float acc[NT][D / 16][4];
  float m[NT][2], l[NT][2];
};

// The warps' states of one unit become its output, by way of `merge` in shared
// memory (the rings, which every warp is done with).
template <int D, bool FP8, int NT>
__device__ __forceinline__ void decode_merge(const DecodeParams& p, const DecState<D, NT>& a, float* merge, int s,
                                             int h0, int nh, int hkv, int warp, int lane) {
  constexpr int kRow = D + 4;                       // A | m, l; padded against bank conflicts
  static_assert(kDecWarps * 8 * NT * kRow * 4 <= DecCfg<D, FP8, NT>::kRing, "the states fit the rings");
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const float NEG_INF = -__int_as_float(0x7f800000);
  __syncthreads();
#pragma unroll
  for (int n8 = 0; n8 < NT; ++n8) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float l = a.l[n8][u];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
      float* mr = merge + ((warp * NT + n8) * 8 + c2 + u) * kRow;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        mr[16 * i + (FP8 ? 2 * g : g)] = a.acc[n8][i][u];
        mr[16 * i + (FP8 ? 2 * g + 1 : g + 8)] = a.acc[n8][i][2 + u];
      }
      if (g == 0) {
        mr[D] = FP8 ? a.m[n8][u] - 12.f : a.m[n8][u];   // l carries P's 2^12
        mr[D + 1] = l;
      }
    }
  }
  __syncthreads();
  const float vs = FP8 ? __ldg(p.v_scale + hkv) : 1.f;
  for (int e = warp * 32 + lane; e < nh * (D / 2); e += kDecThreads) {
    const int hh = e / (D / 2);
    const int d2 = (e - hh * (D / 2)) * 2;
    const float* mr = merge + hh * kRow;
    constexpr int kWarp = NT * 8 * kRow;
    float m = NEG_INF;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w)
      if (mr[w * kWarp + D + 1] != 0.f) m = fmaxf(m, mr[w * kWarp + D]);
    float l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float* x = mr + w * kWarp;
      if (x[D + 1] == 0.f) continue;                // this warp saw no key
      const float f = ex2(x[D] - m);
      l = fmaf(f, x[D + 1], l);
      y0 = fmaf(f, x[d2], y0);
      y1 = fmaf(f, x[d2 + 1], y1);
    }
    const float inv = l == 0.f ? 0.f : vs / l;
    const size_t oh = static_cast<size_t>(s) * p.H + h0 + hh;
    *reinterpret_cast<uint32_t*>(p.o + oh * D + d2) = pack_bf16(y0 * inv, y1 * inv);
    if (d2 == 0) p.lse[oh] = l == 0.f ? NEG_INF : (m + __log2f(l)) * kLn2;
  }
}

// A warp's part of unit (s, r): steps [ta, tb) of the unit's st.total; x0 steps
// of the line lie before the unit.
template <int KEYS>
struct DecUnit {
  int s, r, ta, tb;
  const int* table;            // its row
  long long x0;
  SeqSteps<KEYS> st;
};

// SMALL: a CTA a unit, whose steps its warps share and whose states they join in
// shared memory; no line, no parts.
template <int D, bool FP8, int NT, bool SMALL>
__global__ void __launch_bounds__(kDecThreads, DecCfg<D, FP8, NT>::kCtas)
    attn_decode_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                             const DecodeParams p) {
  using C = DecCfg<D, FP8, NT>;
  constexpr int KEYS = C::kKeys;
  extern __shared__ __align__(1024) uint8_t dec_smem[];
  volatile long long* sums = reinterpret_cast<volatile long long*>(dec_smem + C::kSumsOff);
  volatile long long* found = reinterpret_cast<volatile long long*>(dec_smem + C::kFoundOff);
  volatile long long* edge = reinterpret_cast<volatile long long*>(dec_smem + C::kEdgeOff);
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c2 = (lane & 3) * 2;     // fragment row, first of two columns
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int units = p.Hkv * p.q_tiles;              // units of a sequence
  const int cta = static_cast<int>(blockIdx.x);
  const int n_cta = static_cast<int>(gridDim.x);
  if (!SMALL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may line up

  const uint32_t bars = smem_u32(dec_smem) + C::kBarOff + warp * C::kStages * 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(dec_smem + C::kAbortOff);
  if (smem_u32(dec_smem) & 1023u) {                 // the swizzle needs it: report, touch nothing
    if (tid == 0) {
      record_error(p.err, ATTN_ERR_UNSUPPORTED);
      for (int w = 0; w < kDecWarps && !SMALL; ++w) p.meta[cta * kDecWarps + w] = make_int2(-1, -1);
    }
    return;
  }
  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(bars + 8 * i, 1);
    if (warp == 0) *abort_flag = 0;
    fence_barrier_init();
  }

  // (the division is for rows that belong to a K/V head, and done once a unit)
  auto table_row = [&](int s, int r) {
    const int* row = p.table + static_cast<size_t>(s) * p.t_row;
    return p.t_head != 0 ? row + static_cast<size_t>(r / p.q_tiles) * p.t_head : row;
  };
  DecUnit<KEYS> un;
  int2 meta = make_int2(-1, -1);
  const int worker = cta * kDecWarps + warp;
  long long steps = 0, x1 = 0;                      // the line's steps, and this warp's last one + 1
  int active = 0;                                   // warps with a stretch of it
  if constexpr (SMALL) {
    un.s = cta / units;
    un.r = cta - un.s * units;
    un.table = table_row(un.s, un.r);
    const int n = __ldg(p.lens + un.s);
    if (p.selected && n < 0) return;                // (the whole block)
    if (tid == 0 && un.r == 0 && (n < 0 || n > most_tokens(p)))
      record_error(p.err, ATTN_ERR_BAD_PAGES);
    un.st = seq_steps<KEYS>(n, p);
    un.x0 = 0;
    un.ta = un.st.total * warp / kDecWarps;
    un.tb = un.st.total * (warp + 1) / kDecWarps;
    __syncthreads();                                // the abort flag
  } else {
    // ---- this warp's stretch [x0, x1) of the line of all steps ----
    long long all = 0;
    for (int s = tid; s < p.S; s += kDecThreads) all += seq_steps<KEYS>(__ldg(p.lens + s), p).total;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    if (lane == 0) sums[warp] = all;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) all += sums[w];
    steps = all * units;
    active = static_cast<int>(min(static_cast<long long>(n_cta) * kDecWarps, steps));
    if (tid <= kDecWarps) {
      const int w = cta * kDecWarps + tid;
      edge[tid] = w < active ? steps * w / active : steps;
    }
    __syncthreads();
    const long long x0 = edge[warp];
    x1 = edge[warp + 1];
    // sequences that see no key, and lengths out of range
    for (int s = cta; s < p.S; s += n_cta) {
      const int n = __ldg(p.lens + s);
      if (p.selected && n < 0) continue;
      if (tid == 0 && (n < 0 || n > most_tokens(p)))
        record_error(p.err, ATTN_ERR_BAD_PAGES);
      if (seq_steps<KEYS>(n, p).total > 0) continue;
      for (int e = tid; e < p.H * D; e += kDecThreads)
        p.o[static_cast<size_t>(s) * p.H * D + e] = __float2bfloat16(0.f);
      for (int h = tid; h < p.H; h += kDecThreads) p.lse[static_cast<size_t>(s) * p.H + h] = NEG_INF;
    }
    // the sequences that hold its warps' first steps, and the steps before
    // them.  (The lengths are read again: should somebody change them in the
    // meantime, the results are lost, but every walk below ends and every
    // index stays in range.)
    if (cta * kDecWarps < active) {
      long long last_x0 = edge[0];
      for (int w = 1; w < kDecWarps; ++w)
        if (cta * kDecWarps + w < active) last_x0 = edge[w];
      long long base = 0;
      if (tid < kDecWarps) found[2 * tid] = -1;
      for (int s0 = 0; s0 < p.S; s0 += kDecThreads) {
        const int s = s0 + tid;
        const long long t = s < p.S ? static_cast<long long>(seq_steps<KEYS>(__ldg(p.lens + s), p).total) * units : 0;
        long long x = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
          if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        long long before = base + x - t;
        for (int w = 0; w < warp; ++w) before += sums[w];
        for (int w = 0; w < kDecWarps; ++w) {
          const long long xw = edge[w];
          if (xw >= before && xw < before + t) {
            found[2 * w] = s;
            found[2 * w + 1] = before;
          }
        }
        for (int w = 0; w < kDecWarps; ++w) base += sums[w];
        if (last_x0 < base) break;
      }
      __syncthreads();
    }
    // from here on the warps go their own ways
    bool any = x0 < x1 && found[2 * warp] >= 0;
    if (any) {
      un.s = static_cast<int>(found[2 * warp]);
      un.st = seq_steps<KEYS>(__ldg(p.lens + un.s), p);
      const long long before = found[2 * warp + 1];
      un.r = un.st.total > 0 ? static_cast<int>((x0 - before) / un.st.total) : units;
      un.x0 = before + static_cast<long long>(un.r) * un.st.total;
      any = un.r < units;
      un.table = table_row(un.s, un.r);
    }
    if (!any) {
      if (lane == 0) p.meta[worker] = meta;
      return;
    }
    un.ta = static_cast<int>(x0 - un.x0);
    un.tb = static_cast<int>(min(static_cast<long long>(un.st.total), x1 - un.x0));
  }

  uint8_t* ring = dec_smem + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);
  int st_in = 0, st_out = 0;                  // next stage to fill, to read
  uint32_t phases = 0;                        // parity of each stage's next TMA phase
  uint32_t by_tma = 0;                        // stages with a TMA copy that was not waited for
  uint32_t ok_bits = 0;                       // (4 a stage) its 16-row tiles whose page is in range

  // The pages of a step's 16-row tiles (-1 past the unit), loaded a step ahead
  // of the copies that need them.
  int pages[C::kRowTiles];
  auto fetch_pages = [&](const DecUnit<KEYS>& u, int t) {
    const bool in = t < u.tb;
#pragma unroll
    for (int m = 0; m < C::kRowTiles; ++m) {
      const int key = in ? u.st.key(t) + 16 * m : 0;
      pages[m] = in && key < u.st.n ? __ldg(u.table + (key >> p.page_log2)) : -1;
    }
  };
  auto valid_page = [&](int pg) { return pg >= 0 && pg < p.P; };
  // The copies of step t into stage st_in, from the pages fetched before.
  auto load = [&](const DecUnit<KEYS>& u, int t) {
    if (t >= u.tb) return;
    const int key = u.st.key(t);
    const int hkv = u.r / p.q_tiles;
    const uint32_t dst = ring_u + st_in * C::kStageBytes;
    uint32_t oks = 0;
#pragma unroll
    for (int m = 0; m < C::kRowTiles; ++m) oks |= valid_page(pages[m]) ? 1u << m : 0u;
    ok_bits = (ok_bits & ~(15u << (4 * st_in))) | oks << (4 * st_in);
    if (u.st.whole(key) && oks == (1u << C::kRowTiles) - 1u) {
      by_tma |= 1u << st_in;
      if (lane == 0) {
        const uint32_t bar = bars + 8 * st_in;
        mbar_arrive_expect_tx(bar, C::kStageBytes);
#pragma unroll
        for (int m = 0; m < C::kRowTiles; ++m) {
          const int row = (hkv << p.page_log2) + ((key + 16 * m) & ((1 << p.page_log2) - 1));
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) {
            const uint32_t at = dst + m * C::kTileBytes + h * C::kBoxBytes;
            tma_load_3d(at, &tmK, bar, h * 64, row, pages[m]);
            tma_load_3d(at + C::kHalfBytes, &tmV, bar, h * 64, row, pages[m]);
          }
        }
      }
    } else {
#pragma unroll 1
      for (int m = 0; m < C::kRowTiles; ++m) {
        const int k16 = key + 16 * m;
        int pg = 0;
#pragma unroll
        for (int i = 0; i < C::kRowTiles; ++i)
          if (i == m) pg = pages[i];
        const bool ok = valid_page(pg);
        if (!ok) {
          bool wanted = false;          // a page that a seen key lies in
          for (int i = 0; i < 16; ++i) wanted = wanted || u.st.seen(k16 + i);
          if (wanted && lane == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
          pg = 0;
        }
        const size_t off = ((static_cast<size_t>(hkv) << p.page_log2) + (k16 & ((1 << p.page_log2) - 1))) * C::kRowBytes;
        const uint8_t* kp = p.k + pg * p.k_stride + off;
        const uint8_t* vp = p.v + pg * p.v_stride + off;
        constexpr int kUnits = C::kRowBytes / 16;
        for (int i = 0; i < C::kTileBytes / 512; ++i) {
          const int x16 = i * 32 + lane;
          const int rr = x16 / kUnits, uu = x16 % kUnits;
          const bool in = ok && u.st.seen(k16 + rr);      // rows that nobody sees are not read
          const uint32_t at = dst + m * C::kTileBytes + dec_off<C::kRowBytes>(rr, uu);
          cp_async16(at, kp + x16 * 16, in);
          cp_async16(at + C::kHalfBytes, vp + x16 * 16, in);
        }
      }
      cp_commit();
    }
    if (++st_in == C::kStages) st_in = 0;
  };
  // The unit after u in this warp's stretch; false at its end.
  auto next_unit = [&](DecUnit<KEYS>& u) -> bool {
    const long long x = u.x0 + u.tb;
    if (SMALL || u.tb != u.st.total || x >= x1) return false;
    u.x0 = x;
    if (++u.r == units) {
      u.r = 0;
      do {
        if (++u.s == p.S) return false;
        u.st = seq_steps<KEYS>(__ldg(p.lens + u.s), p);
      } while (u.st.total == 0);
    }
    u.ta = 0;
    u.tb = static_cast<int>(min(static_cast<long long>(u.st.total), x1 - u.x0));
    u.table = table_row(u.s, u.r);
    return true;
  };
  // The first steps of a unit.
  auto start = [&](const DecUnit<KEYS>& u) {
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      fetch_pages(u, u.ta + i);
      load(u, u.ta + i);
    }
    fetch_pages(u, u.ta + C::kStages - 1);
  };
  // Q^T fragments of a unit: head g of each N tile, 2 columns of d at a time.
  // With e4m3 pages an ldmatrix hands a thread 4 neighbouring d's of a key, so
  // the columns that meet in one MMA step are 4 c, 4 c + 1 and 4 c + 2, 4 c + 3.
  uint32_t qf[NT][D / 16][2];
  auto load_q = [&](const DecUnit<KEYS>& u) {
    const int hkv = u.r / p.q_tiles;
    const int h0 = hkv * p.G + (u.r - hkv * p.q_tiles) * 16;
    const int nh = min(16, (hkv + 1) * p.G - h0);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = t * 8 + g;
      const __nv_bfloat16* qh = p.q + u.s * p.q_stride + static_cast<long long>(h0 + min(h, nh - 1)) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int d0 = FP8 ? 16 * ks + 2 * c2 : 16 * ks + c2;
        const int d1 = FP8 ? d0 + 2 : d0 + 8;
        qf[t][ks][0] = h < nh ? __ldg(reinterpret_cast<const uint32_t*>(qh + d0)) : 0u;
        qf[t][ks][1] = h < nh ? __ldg(reinterpret_cast<const uint32_t*>(qh + d1)) : 0u;
      }
    }
  };
  start(un);
  load_q(un);

  for (bool more = true; more;) {
    const int s = un.s, r = un.r, ta = un.ta, tb = un.tb;
    const long long unit_x = un.x0;
    const SeqSteps<KEYS> st = un.st;
    const int hkv = r / p.q_tiles;
    const int h0 = hkv * p.G + (r - hkv * p.q_tiles) * 16;           // first query head
    const int nh = min(16, (hkv + 1) * p.G - h0);                    // query heads of the unit

    float sl2[NT][2];                   // to log2 units, for the thread's two heads of each N tile
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float up = 1.f;                   // the factor of head g's Q
      if constexpr (FP8) {
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top = fmax3(top, fabsf(bf16lo(qf[t][ks][e])), fabsf(bf16hi(qf[t][ks][e])));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // 2^(134 - e) for a top of exponent field e, kept a normal number (an
        // infinity or NaN stays one, whatever it is multiplied by)
        const int field = static_cast<int>(__float_as_uint(top) >> 23);
        up = __uint_as_float(static_cast<uint32_t>(max(1, min(253, 127 + 134 - field))) << 23);
        if (top == 0.f) up = 1.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[t][ks][e] = pack_f16(bf16lo(qf[t][ks][e]) * up, bf16hi(qf[t][ks][e]) * up);
      }
      const float ks = p.scale_log2 * (FP8 ? __ldg(p.k_scale + hkv) : 1.f);
#pragma unroll
      for (int u = 0; u < 2; ++u)
        sl2[t][u] = FP8 ? ks / __shfl_sync(0xFFFFFFFFu, up, (c2 + u) * 4) : ks;
    }
    DecState<D, NT> a;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) a.acc[t][i][u] = 0.f;
      a.m[t][0] = a.m[t][1] = NEG_INF;
      a.l[t][0] = a.l[t][1] = 0.f;
    }

    bool failed = false;
    for (int t = ta; t < tb; ++t) {
      const int key = st.key(t);
      // the step's stage; a step with a page out of range or keys that are
      // not seen came by cp.async
      const bool whole = (by_tma >> st_out) & 1u;
      const uint32_t ok = ok_bits >> (4 * st_out);
      if (whole) {
        if (!__all_sync(0xFFFFFFFFu, wait_bar(bars + 8 * st_out, (phases >> st_out) & 1, abort_flag, p.err))) {
          failed = true;
          break;
        }
        phases ^= 1u << st_out;
        by_tma ^= 1u << st_out;
      } else {
        cp_wait<0>();
        __syncwarp();
      }
      load(un, t + C::kStages - 1);
      fetch_pages(un, t + C::kStages);
      const uint32_t kb = ring_u + st_out * C::kStageBytes;
      const uint32_t vb = kb + C::kHalfBytes;
      // ---- S^T = K Q^T ----
      float sc[C::kRowTiles][NT][4];
#pragma unroll
      for (int m = 0; m < C::kRowTiles; ++m) {
        const uint32_t km = kb + m * C::kTileBytes;
#pragma unroll
        for (int n8 = 0; n8 < NT; ++n8)
#pragma unroll
          for (int u = 0; u < 4; ++u) sc[m][n8][u] = 0.f;
        if constexpr (!FP8) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t f[4];
            ldsm4(km + dec_off<C::kRowBytes>((lane & 7) + (lane & 8), 2 * ks + (lane >> 4)), f);
#pragma unroll
            for (int n8 = 0; n8 < NT; ++n8)
              mma16816<FP8>(sc[m][n8], f[0], f[1], f[2], f[3], qf[n8][ks][0], qf[n8][ks][1]);
          }
        } else {
#pragma unroll
          for (int k2 = 0; k2 < D / 32; ++k2) {
            uint32_t f[4];        // keys 0-7 and 8-15 of 16 d's, then of the next 16
            ldsm4(km + dec_off<C::kRowBytes>((lane & 7) + (lane & 8), 2 * k2 + (lane >> 4)), f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t a0 = e4m3x2_f16x2(f[2 * i]), a2 = e4m3x2_f16x2_hi(f[2 * i]);
              const uint32_t a1 = e4m3x2_f16x2(f[2 * i + 1]), a3 = e4m3x2_f16x2_hi(f[2 * i + 1]);
#pragma unroll
              for (int n8 = 0; n8 < NT; ++n8)
                mma16816<FP8>(sc[m][n8], a0, a1, a2, a3, qf[n8][2 * k2 + i][0], qf[n8][2 * k2 + i][1]);
            }
          }
        }
      }
      // ---- mask and online softmax; rows g and g + 8 of a tile are its keys ----
      uint32_t pb[C::kRowTiles][NT][2];
      uint32_t pb_lo[FP8 ? 1 : C::kRowTiles][NT][2];      // bf16 pages: P's remainders
#pragma unroll
      for (int n8 = 0; n8 < NT; ++n8) {
        float al[2];
        float pr[C::kRowTiles][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float mx = NEG_INF;
#pragma unroll
          for (int m = 0; m < C::kRowTiles; ++m) {
            float y0 = sc[m][n8][u] * sl2[n8][u], y1 = sc[m][n8][2 + u] * sl2[n8][u];
            if (!whole) {
              if (!((ok >> m & 1u) && st.seen(key + 16 * m + g))) y0 = NEG_INF;
              if (!((ok >> m & 1u) && st.seen(key + 16 * m + g + 8))) y1 = NEG_INF;
            }
            pr[m][u] = y0;
            pr[m][2 + u] = y1;
            mx = fmax3(mx, y0, y1);
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
          const float mn = fmaxf(a.m[n8][u], mx);
          const float mu = mn == NEG_INF ? 0.f : mn;
          al[u] = ex2(a.m[n8][u] - mu);
          a.m[n8][u] = mn;
          const float mp = FP8 ? mu - 12.f : mu;         // P and l carry 2^12
          float sum = 0.f;
#pragma unroll
          for (int m = 0; m < C::kRowTiles; ++m) {
            pr[m][u] = ex2(pr[m][u] - mp);
            pr[m][2 + u] = ex2(pr[m][2 + u] - mp);
            sum += pr[m][u] + pr[m][2 + u];
          }
          a.l[n8][u] = fmaf(a.l[n8][u], al[u], sum);
        }
        if (__any_sync(0xFFFFFFFFu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            a.acc[n8][i][0] *= al[0];
            a.acc[n8][i][1] *= al[1];
            a.acc[n8][i][2] *= al[0];
            a.acc[n8][i][3] *= al[1];
          }
        }
        // P^T as the B operand: rows (keys) become the pairs of a thread
#pragma unroll
        for (int m = 0; m < C::kRowTiles; ++m) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if constexpr (FP8) {
              pb[m][n8][u] = movm(pack_f16(pr[m][2 * u], pr[m][2 * u + 1]));
            } else {
              pb[m][n8][u] = movm(high_bf16(pr[m][2 * u], pr[m][2 * u + 1]));
              pb_lo[m][n8][u] = movm(pack_bf16(p_rest(pr[m][2 * u]), p_rest(pr[m][2 * u + 1])));
            }
          }
        }
      }
      // ---- A^T += V^T P^T ----
#pragma unroll
      for (int m = 0; m < C::kRowTiles; ++m) {
        const uint32_t vm = vb + m * C::kTileBytes;
        if constexpr (!FP8) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t f[4];        // keys 0-7: d 0-7, d 8-15; keys 8-15: the same
            ldsm4t(vm + dec_off<C::kRowBytes>((lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)), f);
#pragma unroll
            for (int n8 = 0; n8 < NT; ++n8) {
              mma16816<FP8>(a.acc[n8][i], f[0], f[1], f[2], f[3], pb[m][n8][0], pb[m][n8][1]);
              mma16816<FP8>(a.acc[n8][i], f[0], f[1], f[2], f[3], pb_lo[m][n8][0], pb_lo[m][n8][1]);
            }
          }
        } else {
#pragma unroll
          for (int i2 = 0; i2 < D / 32; ++i2) {
            uint32_t f[4];        // keys 0-7, keys 8-15 of 16 d's, then of the next 16
            ldsm4t(vm + dec_off<C::kRowBytes>((lane & 7) + (lane & 8), 2 * i2 + (lane >> 4)), f);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // a thread holds d's 2 g, 2 g + 1 of keys c2 and c2 + 1: rows g
              // and g + 8 of the fragment stand for d = 2 g and 2 g + 1
              const uint32_t lo = f[2 * i], hi = f[2 * i + 1];
              const uint32_t a0 = e4m3x2_f16x2(__byte_perm(lo, 0, 0x4420));
              const uint32_t a1 = e4m3x2_f16x2(__byte_perm(lo, 0, 0x4431));
              const uint32_t a2 = e4m3x2_f16x2(__byte_perm(hi, 0, 0x4420));
              const uint32_t a3 = e4m3x2_f16x2(__byte_perm(hi, 0, 0x4431));
#pragma unroll
              for (int n8 = 0; n8 < NT; ++n8)
                mma16816<FP8>(a.acc[n8][2 * i2 + i], a0, a1, a2, a3, pb[m][n8][0], pb[m][n8][1]);
            }
          }
        }
      }
      if (!whole) fence_proxy_async_smem();   // the stage was written by cp.async, TMA may be next
      __syncwarp();                           // the stage may be refilled
      if (++st_out == C::kStages) st_out = 0;
    }
    if (failed) {                       // a copy timed out: let those in flight land, give up
      for (int i = 0; i < C::kStages; ++i)
        if (by_tma >> i & 1u) drain_bar(bars + 8 * i, (phases >> i) & 1);
      cp_wait<0>();
      meta = make_int2(-1, -1);
      if (!SMALL) break;
    }
    // the next unit's first steps and its Q, on their way while this one's
    // state goes out
    more = next_unit(un);
    if (more) {
      start(un);
      load_q(un);
    }

    if constexpr (SMALL) {
      decode_merge<D, FP8, NT>(p, a, reinterpret_cast<float*>(dec_smem), s, h0, nh, hkv, warp, lane);
      return;
    }
    // ---- the state: the output of a unit that is whole, else a part ----
    const bool whole = ta == 0 && tb == st.total;
    const bool head = ta > 0;
    if (!whole && !head) {
      // step y of the line lies in the last warp w with steps w / active <= y
      meta.x = s * units + r;
      meta.y = static_cast<int>(min(((unit_x + st.total) * active + steps - 1) / steps, static_cast<long long>(active))) - 1;
    }
    float* part = p.part + (static_cast<size_t>(worker) * 2 + (head ? 0 : 1)) * p.rows * (D + 2);
    const float vs = FP8 ? __ldg(p.v_scale + hkv) : 1.f;
#pragma unroll
    for (int n8 = 0; n8 < NT; ++n8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float l = a.l[n8][u];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        // l carries P's 2^12: the max that goes with it is 12 lower
        const float m = FP8 ? a.m[n8][u] - 12.f : a.m[n8][u];
        const int hh = n8 * 8 + c2 + u;
        if (hh >= nh) continue;
        if (whole) {
          const float inv = l == 0.f ? 0.f : vs / l;
          const size_t oh = static_cast<size_t>(s) * p.H + h0 + hh;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const float y0 = a.acc[n8][i][u] * inv, y1 = a.acc[n8][i][2 + u] * inv;
            if constexpr (FP8) {
              *reinterpret_cast<uint32_t*>(p.o + oh * D + 16 * i + 2 * g) = pack_bf16(y0, y1);
            } else {
              p.o[oh * D + 16 * i + g] = __float2bfloat16(y0);
              p.o[oh * D + 16 * i + g + 8] = __float2bfloat16(y1);
            }
          }
          if (g == 0) p.lse[oh] = l == 0.f ? NEG_INF : (m + __log2f(l)) * kLn2;
        } else {
          float* pt = part + hh * (D + 2);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            pt[16 * i + (FP8 ? 2 * g : g)] = a.acc[n8][i][u];
            pt[16 * i + (FP8 ? 2 * g + 1 : g + 8)] = a.acc[n8][i][2 + u];
          }
          if (g == 0) {
            pt[D] = m;
            pt[D + 1] = l;
          }
        }
      }
    }
  }
  if (lane == 0) p.meta[worker] = meta;
}

// Joins the units that go on past their first warp: block (c, h) those whose
// first part CTA c's warps have left, for query head h of the unit.  A warp
// takes the parts of one unit, 32 maxima at a time; where there are more than
// 64 (one long sequence over every warp) the block's warps share them.
template <int D>
struct JoinState {
  float m, l, y[D / 32];
};
// Parts first, first + step, ... up to last, of which part c_first lies in slot 1.
template <int D>
__device__ __forceinline__ JoinState<D> join_parts(const DecodeParams& p, int hh, int c_first, int first, int step,
                                                   int last, int lane) {
  constexpr int V = D / 32;
  const float NEG_INF = -__int_as_float(0x7f800000);
  JoinState<D> st;
  st.m = NEG_INF;
  st.l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) st.y[i] = 0.f;
  auto at = [&](int x) {
    return p.part + ((static_cast<size_t>(x) * 2 + (x == c_first ? 1 : 0)) * p.rows + hh) * (D + 2);
  };
  for (int x0 = first; x0 <= last; x0 += 32 * step) {
    const int x = x0 + lane * step;
    const float lx = x <= last ? at(x)[D + 1] : 0.f;
    const float mx = lx != 0.f ? at(x)[D] : NEG_INF;
    float mn = mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
    mn = fmaxf(mn, st.m);
    if (__all_sync(0xFFFFFFFFu, lx == 0.f)) continue;       // no key in these parts
    const float old = st.l == 0.f ? 0.f : ex2(st.m - mn);
    const float w = lx == 0.f ? 0.f : ex2(mx - mn);
    float sum = w * lx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    st.l = fmaf(st.l, old, sum);
    st.m = mn;
#pragma unroll
    for (int i = 0; i < V; ++i) st.y[i] *= old;
    const int n = min(32, (last - x0) / step + 1);
    // eight parts' loads in flight at once (a part without a key has zeros,
    // its weight of 0 needs no branch; past the last part the last one is
    // read again, with a weight of 0)
    for (int i0 = 0; i0 < n; i0 += 8) {
      float v[8][V];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float* pt = at(x0 + min(i0 + i, n - 1) * step);
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = pt[e * 32 + lane];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float wi = i0 + i < n ? __shfl_sync(0xFFFFFFFFu, w, (i0 + i) & 31) : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) st.y[e] = fmaf(v[i][e], wi, st.y[e]);
      }
    }
  }
  return st;
}

constexpr int kJoinWarps = kDecWarps;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_decode_join_kernel(const DecodeParams p) {
  constexpr int V = D / 32;
  __shared__ float sh[kJoinWarps][D + 2];
  const int hh = static_cast<int>(blockIdx.y);
  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int units = p.Hkv * p.q_tiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the parts are complete
  auto store = [&](int unit, const JoinState<D>& st) {
    const int s = unit / units, r = unit - s * units;
    const int hkv = r / p.q_tiles;
    const int h = hkv * p.G + (r - hkv * p.q_tiles) * 16 + hh;
    if (hh >= 16 || h >= (hkv + 1) * p.G) return;
    const float inv = st.l == 0.f ? 0.f : (p.v_scale ? __ldg(p.v_scale + hkv) : 1.f) / st.l;
    const size_t oh = static_cast<size_t>(s) * p.H + h;
#pragma unroll
    for (int e = 0; e < V; ++e) p.o[oh * D + e * 32 + lane] = __float2bfloat16(st.y[e] * inv);
    if (lane == 0) p.lse[oh] = st.l == 0.f ? NEG_INF : (st.m + __log2f(st.l)) * kLn2;
  };
  auto in_unit = [&](int unit) {           // whether the unit has a head hh
    const int r = unit % units;
    const int hkv = r / p.q_tiles;
    return hkv * p.G + (r - hkv * p.q_tiles) * 16 + hh < (hkv + 1) * p.G;
  };
  const int c0 = static_cast<int>(blockIdx.x) * kJoinWarps;
  const int2 mine = p.meta[c0 + warp];
  const bool many = mine.x >= 0 && mine.y - (c0 + warp) >= 64;
  if (mine.x >= 0 && !many && in_unit(mine.x))
    store(mine.x, join_parts<D>(p, hh, c0 + warp, c0 + warp, 1, mine.y, lane));
  if (!__syncthreads_or(many)) return;
  for (int w = 0; w < kJoinWarps; ++w) {
    const int2 meta = p.meta[c0 + w];
    if (meta.x < 0 || meta.y - (c0 + w) < 64 || !in_unit(meta.x)) continue;
    const JoinState<D> st = join_parts<D>(p, hh, c0 + w, c0 + w + warp, kJoinWarps, meta.y, lane);
#pragma unroll
    for (int e = 0; e < V; ++e) sh[warp][e * 32 + lane] = st.y[e];
    if (lane == 0) {
      sh[warp][D] = st.m;
      sh[warp][D + 1] = st.l;
    }
    __syncthreads();
    if (warp == 0) {
      JoinState<D> all;
      all.m = NEG_INF;
#pragma unroll
      for (int x = 0; x < kJoinWarps; ++x)
        if (sh[x][D + 1] != 0.f) all.m = fmaxf(all.m, sh[x][D]);
      all.l = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) all.y[e] = 0.f;
#pragma unroll
      for (int x = 0; x < kJoinWarps; ++x) {
        if (sh[x][D + 1] == 0.f) continue;
        const float f = ex2(sh[x][D] - all.m);
        all.l = fmaf(f, sh[x][D + 1], all.l);
#pragma unroll
        for (int e = 0; e < V; ++e) all.y[e] = fmaf(f, sh[x][e * 32 + lane], all.y[e]);
      }
      store(meta.x, all);
    }
    __syncthreads();
  }
}

constexpr int kDecMaxCtas = 152 * 3;

constexpr int kDecWorkers = kDecMaxCtas * kDecWarps;

// query heads of a part: what a K/V head's group has, at most 16
int decode_rows(int G) { return G <= 8 ? 8 : 16; }
// 16-key steps that the table's rows have room for, over all units: more
// workers than that have nothing to do (rounded up to whole CTAs)
long long decode_workers(int S, int Hkv, int G, int max_pages, int page) {
  const long long steps = static_cast<long long>(max_pages) * (page / 16) * S * Hkv * ((G + 15) / 16);
  return std::min<long long>(kDecWorkers, (steps + kDecWarps - 1) / kDecWarps * kDecWarps);
}
// Whether a CTA a unit does: one launch without a scan of the lengths and
// without parts, instead of sharing all steps evenly.  What that takes grows
// with the longest unit, so it is for tables whose rows hold up to 1024 tokens
// (us, a CTA a unit | shared evenly, rows as long as the table has room for,
// d=128, bf16; S sequences of 16 query heads on 4 K/V heads):
//      tokens    64           256          1024
//      S = 1     6.1 | 10.2   8.2 | 12.2   16.4 | 16.6
//      S = 64    6.2 | 12.3   12.0 | 18.5  27.8 | 33.0
//      S = 512   24 | 29      51 | 58      161 | 173
// A group of more than 8 query heads takes a warp longer over its keys; past
// 512 tokens its few units do better shared by more CTAs (16 query heads on one
// K/V head):
//      tokens    256          512          768          1024
//      S = 1     10.3 | 12.5  14.5 | 14.3  18.5 | 16.4  22.5 | 18.3
//      S = 32    10.3 | 16.3  14.5 | 18.4  18.5 | 18.8  23.2 | 20.5
//      S = 64    11.6 | 16.4  14.4 | 18.8  19.8 | 22.0  24.6 | 23.8
//      S = 128   11.0 | 20.1  16.4 | 24.6  20.5 | 27.6  24.7 | 30.0
// And over many units of few tokens the CTAs' set-up adds up (4 K/V heads; bf16,
// e4m3):
//      tokens    16                        32                        64
//      S = 128   8.2 | 10.2, 10.3 | 11.9   8.9 | 12.7, 9.6 | 11.0    9.6 | 16.4, 10.2 | 13.2
//      S = 512   15.8 | 14.4, 23.2 | 18.4  19.7 | 22.6, 18.5 | 16.4  24.3 | 28.7, 22.4 | 23.6
//      S = 1024  32.5 | 21.9, 38.9 | 25.9  33.1 | 30.6, 35.1 | 24.6  39.1 | 41.0, 38.3 | 32.8
// The host has one launch and one allocation less (20 against 25 us).  Rows that
// are shorter than the table has room for take less by either way, a CTA a
// unit's more so; the lengths are the device's.
constexpr int kSmallKeys = 1024;
constexpr int kSmallKeysLarge = 512;        // groups of more than 8 query heads in few units
constexpr int kSmallUnitsLarge = 64;        // ... fewer than this
constexpr int kSmallUnits = 4096;
constexpr int kSmallUnitsAToken = 32;
bool decode_small(int S, int Hkv, int G, int max_pages, int page) {
  const long long units = static_cast<long long>(S) * Hkv * ((G + 15) / 16);
  const long long tokens = static_cast<long long>(max_pages) * page;
  if (tokens > kSmallKeys || units > std::min<long long>(kSmallUnits, tokens * kSmallUnitsAToken)) return false;
  return G <= 8 || tokens <= kSmallKeysLarge || units >= kSmallUnitsLarge;
}
size_t decode_workspace(int d, int G, long long workers) {
  return static_cast<size_t>(workers) * 8 + static_cast<size_t>(workers) * 2 * decode_rows(G) * (d + 2) * 4;
}

template <int D, bool FP8, int NT, bool SMALL>
cudaError_t launch_decode(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, cudaStream_t st) {
  using C = DecCfg<D, FP8, NT>;
  auto kern = attn_decode_paged_kernel<D, FP8, NT, SMALL>;
  constexpr int kMaxDev = 64;
  static bool configured[kMaxDev] = {};  // the attribute is per device and function
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  if constexpr (SMALL) {
    kern<<<static_cast<unsigned>(p.S * p.Hkv * p.q_tiles), kDecThreads, C::kSmem, st>>>(tk, tv, p);
    return cudaGetLastError();
  }
  // no more CTAs than the table's rows can hold steps for
  const long long most = ((static_cast<long long>(p.M) << p.page_log2) + C::kKeys - 1) / C::kKeys * p.S * p.Hkv * p.q_tiles;
  const int grid = static_cast<int>(std::max(1ll, std::min<long long>(152 * C::kCtas, (most + kDecWarps - 1) / kDecWarps)));
  kern<<<grid, kDecThreads, C::kSmem, st>>>(tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // the join's blocks may be set up while the main kernel runs; they wait for
  // its end themselves
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, std::min(16, p.G));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D>, p);
}

bool decode_sizes(int S, int H, int Hkv, int d, int max_pages, int page) {
  if (max_pages < 1 || !valid_page_size(page)) return false;
  if (S < 1 || H < 1 || !valid_kv_heads(H, Hkv) || (d != 64 && d != 128)) return false;
  return S <= kMaxSeqs && static_cast<long long>(S) * H <= 0x7FFFFFFFll;
}

}  // namespace
}  // namespace bss

using namespace bss;

extern "C" size_t attn_decode_paged_workspace_bytes(int S, int H, int H_kv, int d, int max_pages,
                                                    int page_size) {
  if (!decode_sizes(S, H, H_kv, d, max_pages, page_size)) return 0;
  if (decode_small(S, H_kv, H / H_kv, max_pages, page_size)) return 0;
  return decode_workspace(d, H / H_kv, decode_workers(S, H_kv, H / H_kv, max_pages, page_size));
}

namespace {
// Both entry points: a row of the table per sequence, or per sequence and K/V head (`selected`).
attn_status_t decode(const char* name, const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                     int64_t k_page_stride, int64_t v_page_stride, int kv_dtype, const float* k_scale,
                     const float* v_scale, const int32_t* page_table, const int32_t* seq_lens, void* o,
                     float* lse, void* workspace, size_t workspace_bytes, int S, int H, int H_kv, int d,
                     int max_pages, int n_pages, int page_size, float scale, int64_t window, int64_t sinks,
                     bool selected, void* stream) {
  attn_status_t s = check_common(S, H, 1, 1, d, scale);
  if (s != ATTN_OK) return s;
  if (!valid_kv_heads(H, H_kv)) return ATTN_ERR_INVALID_ARG;
  if (S > kMaxSeqs) return ATTN_ERR_UNSUPPORTED;
  if (max_pages < 1 || n_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (selected && static_cast<long long>(H_kv) * max_pages > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;
  if (!valid_page_size(page_size)) return ATTN_ERR_UNSUPPORTED;
  if (kv_dtype != ATTN_KV_BF16 && kv_dtype != ATTN_KV_E4M3) return ATTN_ERR_UNSUPPORTED;
  if (window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return ATTN_ERR_INVALID_ARG;
  const bool small = decode_small(S, H_kv, H / H_kv, max_pages, page_size);
  const void* ptrs16[] = {q, k_cache, v_cache, o, small ? o : workspace};
  for (const void* ptr : ptrs16)
    if (!ptr || !aligned16(ptr)) return ATTN_ERR_INVALID_ARG;
  const void* ptrs4[] = {page_table, seq_lens, lse};
  for (const void* ptr : ptrs4)
    if (!ptr || !aligned4(ptr)) return ATTN_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == ATTN_KV_E4M3;
  if (fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr) || !aligned4(k_scale) || !aligned4(v_scale))
    return ATTN_ERR_INVALID_ARG;
  const int64_t least = static_cast<int64_t>(H_kv) * page_size * d;
  const int64_t unit = fp8 ? 16 : 8;
  if (k_page_stride < least || v_page_stride < least || k_page_stride % unit || v_page_stride % unit)
    return ATTN_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(H) * d || q_stride % 8) return ATTN_ERR_INVALID_ARG;
  const long long workers = decode_workers(S, H_kv, H / H_kv, max_pages, page_size);
  if (!small && workspace_bytes < decode_workspace(d, H / H_kv, workers)) return ATTN_ERR_WORKSPACE;
  DecodeParams p{};
  if ((s = status_word(&p.err)) != ATTN_OK) return s;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.k = static_cast<const uint8_t*>(k_cache);
  p.v = static_cast<const uint8_t*>(v_cache);
  p.k_stride = static_cast<size_t>(k_page_stride) * (fp8 ? 1 : 2);
  p.v_stride = static_cast<size_t>(v_page_stride) * (fp8 ? 1 : 2);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.lens = seq_lens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.meta = static_cast<int2*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + static_cast<size_t>(workers) * 8);
  p.rows = decode_rows(H / H_kv);
  p.S = S;
  p.H = H;
  p.Hkv = H_kv;
  p.G = H / H_kv;
  p.M = max_pages;
  p.t_head = selected ? max_pages : 0;
  p.t_row = selected ? H_kv * max_pages : max_pages;
  p.selected = selected;
  p.P = n_pages;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.q_tiles = (p.G + 15) / 16;
  p.scale_log2 = scale * kLog2e;
  p.window = std::min<int64_t>(window, int64_t(1) << 60);
  p.sinks = static_cast<int>(std::min<int64_t>(sinks, 0x7FFFFFF0));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool one = p.G <= 8;
  if ((s = get_encoder()) != ATTN_OK) return s;
  CUtensorMap tk, tv;
  const long long rows = static_cast<long long>(H_kv) * page_size;
  if (rows > 0x7FFFFFFFll) return ATTN_ERR_UNSUPPORTED;     // a copy's row is an int
  if ((s = cache_map(&tk, k_cache, d, fp8, rows, n_pages, p.k_stride, 16)) != ATTN_OK) return s;
  if ((s = cache_map(&tv, v_cache, d, fp8, rows, n_pages, p.v_stride, 16)) != ATTN_OK) return s;
  cudaError_t e = cudaErrorInvalidValue;
#define BSS_DECODE_CASE(DD, FP, NN, SM) \
  if (d == DD && fp8 == FP && one == (NN == 1) && small == SM) e = launch_decode<DD, FP, NN, SM>(tk, tv, p, st);
#define BSS_DECODE_CASES(DD, FP)    \
  BSS_DECODE_CASE(DD, FP, 1, false) \
  BSS_DECODE_CASE(DD, FP, 2, false) \
  BSS_DECODE_CASE(DD, FP, 1, true)  \
  BSS_DECODE_CASE(DD, FP, 2, true)
  BSS_DECODE_CASES(64, false)
  BSS_DECODE_CASES(64, true)
  BSS_DECODE_CASES(128, false)
  BSS_DECODE_CASES(128, true)
#undef BSS_DECODE_CASES
#undef BSS_DECODE_CASE
  return cuda_status(name, e);
}
}  // namespace

extern "C" attn_status_t attn_decode_paged(
    const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int64_t k_page_stride,
    int64_t v_page_stride, int kv_dtype, const float* k_scale, const float* v_scale,
    const int32_t* page_table, const int32_t* seq_lens, void* o, float* lse, void* workspace,
    size_t workspace_bytes, int S, int H, int H_kv, int d, int max_pages, int n_pages, int page_size,
    float scale, int64_t window, int64_t sinks, void* stream) {
  return decode("attn_decode_paged launch", q, q_stride, k_cache, v_cache, k_page_stride, v_page_stride, kv_dtype,
                k_scale, v_scale, page_table, seq_lens, o, lse, workspace, workspace_bytes, S, H, H_kv, d,
                max_pages, n_pages, page_size, scale, window, sinks, false, stream);
}

extern "C" attn_status_t attn_decode_selected(
    const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int64_t k_page_stride,
    int64_t v_page_stride, int kv_dtype, const float* k_scale, const float* v_scale, const int32_t* pages,
    const int32_t* lens, void* o, float* lse, void* workspace, size_t workspace_bytes, int T, int H, int H_kv,
    int d, int max_pages, int n_pages, int page_size, float scale, void* stream) {
  return decode("attn_decode_selected launch", q, q_stride, k_cache, v_cache, k_page_stride, v_page_stride,
                kv_dtype, k_scale, v_scale, pages, lens, o, lse, workspace, workspace_bytes, T, H, H_kv, d,
                max_pages, n_pages, page_size, scale, 0, 0, true, stream);
}
