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
//   * The work is cut evenly, whatever the lengths: all tiles of 64 keys of
//     every (sequence, K/V head, group of 16 query heads) form one line, and
//     each of the resident CTAs takes an equal stretch of it.  A stretch that
//     covers a whole unit writes its output; the (at most two) units a CTA
//     has only a part of leave their state in the workspace, two slots a CTA,
//     and a second kernel joins them in order.
//   * A warp works by itself on 16 keys at a time: cp.async copies their K and
//     V rows (one page's, so contiguous) into its own ring of swizzled stages
//     in shared memory, 16 bytes a lane and copy, and only __syncwarp orders
//     them.  Nothing but the unit's end needs the other warps.
//   * The products run transposed on mma.m16n8k16: S^T = K Q^T has the 16 keys
//     as rows and 8 query heads as columns, A^T = V^T P^T has 16 columns of d
//     as rows.  A group of up to 8 query heads then costs one tile of N = 8,
//     the 16-row side is always full, and a thread's accumulators belong to
//     the same two heads as its softmax state.
//   * e4m3 pages are read as they are (half the bytes); a pair of elements
//     becomes bf16 exactly on the way into the MMA.  The scales multiply the
//     score and the output.
#include <cuda_fp8.h>

#include <algorithm>

#include "host.cuh"

namespace bss {
namespace {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecKeys = 16;                        // keys a warp takes at a time
constexpr int kDecTile = kDecWarps * kDecKeys;      // keys of a CTA's turn
constexpr int kMaxSeqs = 65536;

struct DecodeParams {
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t* k;
  const uint8_t* v;
  size_t k_stride, v_stride;     // bytes from page to page
  const float* k_scale;
  const float* v_scale;
  const int* table;
  const int* lens;
  __nv_bfloat16* o;
  float* lse;
  int4* meta;                    // [grid]: .x the unit the CTA leaves in slot 1 (-1: none), .y the
                                 // last CTA with a part of it (the parts between are slots 0)
  float* part;                   // [grid][2][16][d + 2]: A, m (log2 units), l of the parts
  int S, H, Hkv, G, M, P;
  int page_log2;
  int q_tiles;                   // groups of 16 query heads of a K/V head
  float scale_log2;
  long long window;
  int sinks;
  int* err;
};

// The 16-key steps a sequence's query reads: the sinks' steps [0, nsink), then
// [first, first + rest).
struct SeqSteps {
  int n, lo, sk;                 // length, first key of the window, sinks below it
  int nsink, first, total;
  __device__ __forceinline__ int key(int t) const {
    return kDecKeys * (t < nsink ? t : first + (t - nsink));
  }
};
__device__ __forceinline__ SeqSteps seq_steps(int n, const DecodeParams& p) {
  SeqSteps q;
  q.n = min(max(n, 0), static_cast<int>(min(static_cast<long long>(p.M) << p.page_log2, 0x7FFFFFF0ll)));
  q.lo = p.window > 0 ? static_cast<int>(max(0ll, static_cast<long long>(q.n) - p.window)) : 0;
  q.sk = min(p.sinks, q.lo);
  q.first = q.lo / kDecKeys;
  q.nsink = min((q.sk + kDecKeys - 1) / kDecKeys, q.first);
  q.total = q.nsink + (q.n + kDecKeys - 1) / kDecKeys - q.first;
  return q;
}
__device__ __forceinline__ int seq_tiles(int n, const DecodeParams& p) {
  return (seq_steps(n, p).total + kDecWarps - 1) / kDecWarps;
}

template <int D, bool FP8, int NT>
struct DecCfg {
  static constexpr int kItem = FP8 ? 1 : 2;
  static constexpr int kRowBytes = D * kItem;
  static constexpr int kHalfBytes = kDecKeys * kRowBytes;      // K or V rows of a step
  static constexpr int kStageBytes = 2 * kHalfBytes;
  // about 64 KB in flight a CTA, three CTAs on an SM
  static constexpr int kStages = 65536 / (kDecWarps * kStageBytes) > 6 ? 6 : 65536 / (kDecWarps * kStageBytes);
  static constexpr int kRing = kDecWarps * kStages * kStageBytes;
  static constexpr int kMergeRow = D + 4;                      // padded against bank conflicts
  static constexpr int kMergeBytes = kDecWarps * 8 * NT * kMergeRow * 4;
  static constexpr int kSmem = kRing > kMergeBytes ? kRing : kMergeBytes;
};

// Byte offset of 16-byte unit u of row r of a step's K or V rows: units are
// swizzled so that the 8 rows one ldmatrix reads hit 8 different 16-byte banks.
template <int ROW>
__device__ __forceinline__ int dec_off(int r, int u) {
  if constexpr (ROW >= 128) return r * ROW + ((u ^ (r & 7)) << 4);
  else return r * ROW + ((u ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;       // 0: the 16 bytes are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two e4m3 elements (the low 16 bits) as a pair of bf16, exactly: e4m3 fits
// fp16, and its 3 fraction bits fit bf16.
__device__ __forceinline__ uint32_t e4m3x2_bf16x2(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xFFFFu), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return pack_bf16(f.x, f.y);
}

// The running state of a unit in one warp: A^T fragments, and for the thread's
// two heads of each N tile the max (log2 units) and this thread's part of l.
template <int D, int NT>
struct DecState {
  float acc[NT][D / 16][4];
  float m[NT][2], l[NT][2];
};

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(kDecThreads, 3) attn_decode_paged_kernel(const DecodeParams p) {
  using C = DecCfg<D, FP8, NT>;
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ long long sums[kDecWarps + 1];
  __shared__ int found_s;
  __shared__ long long found_before;
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c2 = (lane & 3) * 2;     // fragment row, first of two columns
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int units = p.Hkv * p.q_tiles;              // units of a sequence
  const int cta = static_cast<int>(blockIdx.x);
  const int n_cta = static_cast<int>(gridDim.x);

  // ---- this CTA's stretch [x0, x1) of all tiles ----
  long long mine = 0;
  for (int s = tid; s < p.S; s += kDecThreads) mine += seq_tiles(__ldg(p.lens + s), p);
  long long all = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if (lane == 0) sums[warp] = all;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) all += sums[w];
  const long long tiles = all * units;
  const int active = static_cast<int>(min(static_cast<long long>(n_cta), tiles));
  long long x0 = 0, x1 = 0;
  if (cta < active) {
    x0 = tiles * cta / active;
    x1 = tiles * (cta + 1) / active;
  }
  // sequences that see no key, and lengths out of range
  for (int s = cta; s < p.S; s += n_cta) {
    const int n = __ldg(p.lens + s);
    if (tid == 0 && (n < 0 || n > (static_cast<long long>(p.M) << p.page_log2)))
      record_error(p.err, ATTN_ERR_BAD_PAGES);
    if (seq_tiles(n, p) > 0) continue;
    for (int e = tid; e < p.H * D; e += kDecThreads)
      p.o[static_cast<size_t>(s) * p.H * D + e] = __float2bfloat16(0.f);
    for (int h = tid; h < p.H; h += kDecThreads) p.lse[static_cast<size_t>(s) * p.H + h] = NEG_INF;
  }
  int4 meta = make_int4(-1, -1, 0, 0);
  if (x0 >= x1) {
    if (tid == 0) p.meta[cta] = meta;
    return;
  }
  // the sequence that holds tile x0, and the tiles before it
  {
    long long base = 0;
    for (int s0 = 0;; s0 += kDecThreads) {
      const int s = s0 + tid;
      const long long t = s < p.S ? static_cast<long long>(seq_tiles(__ldg(p.lens + s), p)) * units : 0;
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
      if (x0 >= before && x0 < before + t) {
        found_s = s;
        found_before = before;
      }
      for (int w = 0; w < kDecWarps; ++w) base += sums[w];
      if (x0 < base) break;
    }
    __syncthreads();
  }
  int s = found_s;
  long long unit_x = found_before;                  // the line's tiles before unit (s, r)
  SeqSteps st = seq_steps(__ldg(p.lens + s), p);
  int nt = (st.total + kDecWarps - 1) / kDecWarps;
  int r = static_cast<int>((x0 - unit_x) / nt);
  unit_x += static_cast<long long>(r) * nt;

  uint8_t* ring = dec_smem + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_u = smem_u32(ring);

  for (long long x = x0; x < x1;) {
    // ---- unit (s, r): tiles [ta, tb) of its nt are this CTA's ----
    const int ta = static_cast<int>(x - unit_x);
    const int tb = static_cast<int>(min(static_cast<long long>(nt), x1 - unit_x));
    const int hkv = r / p.q_tiles;
    const int h0 = hkv * p.G + (r - hkv * p.q_tiles) * 16;           // first query head
    const int nh = min(16, (hkv + 1) * p.G - h0);                    // query heads of the unit
    const int* row = p.table + static_cast<size_t>(s) * p.M;
    const size_t head_off = (static_cast<size_t>(hkv) << p.page_log2) * C::kRowBytes;

    // Q^T fragments: head g of each N tile, 2 columns of d at a time.  With
    // e4m3 pages an ldmatrix hands a thread 4 neighbouring d's of a key, so
    // the columns that meet in one MMA step are 4 c, 4 c + 1 and 4 c + 2, 4 c + 3.
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = t * 8 + g;
      const __nv_bfloat16* qh = p.q + s * p.q_stride + static_cast<long long>(h0 + min(h, nh - 1)) * D;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int d0 = FP8 ? 16 * ks + 2 * c2 : 16 * ks + c2;
        const int d1 = FP8 ? d0 + 2 : d0 + 8;
        qf[t][ks][0] = h < nh ? __ldg(reinterpret_cast<const uint32_t*>(qh + d0)) : 0u;
        qf[t][ks][1] = h < nh ? __ldg(reinterpret_cast<const uint32_t*>(qh + d1)) : 0u;
      }
    }
    const float sl2 = p.scale_log2 * (FP8 ? __ldg(p.k_scale + hkv) : 1.f);
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

    // this warp's steps: ta * 4 + warp, + 4, ...
    const int t_first = ta * kDecWarps + warp;
    const int t_end = min(st.total, tb * kDecWarps);
    auto seen = [&](int j) { return j < st.n && (j >= st.lo || j < st.sk); };
    auto load = [&](int t, int stage) {
      if (t < t_end) {
        const int key = st.key(t);
        int page = __ldg(row + (key >> p.page_log2));
        const bool ok = page >= 0 && page < p.P;
        if (!ok) {                      // zeros in, and the mask below leaves the keys out
          if (lane == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
          page = 0;
        }
        const size_t off = head_off + static_cast<size_t>(key & ((1 << p.page_log2) - 1)) * C::kRowBytes;
        const uint8_t* kp = p.k + page * p.k_stride + off;
        const uint8_t* vp = p.v + page * p.v_stride + off;
        const uint32_t dst = ring_u + stage * C::kStageBytes;
        constexpr int kUnits = C::kRowBytes / 16;
#pragma unroll
        for (int i = 0; i < C::kHalfBytes / 512; ++i) {
          const int x16 = i * 32 + lane;
          const int rr = x16 / kUnits, u = x16 % kUnits;
          const bool in = ok && seen(key + rr);      // rows that nobody sees are not read
          cp_async16(dst + dec_off<C::kRowBytes>(rr, u), kp + x16 * 16, in);
          cp_async16(dst + C::kHalfBytes + dec_off<C::kRowBytes>(rr, u), vp + x16 * 16, in);
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) load(t_first + i * kDecWarps, i);
    int stage = 0;
    for (int t = t_first; t < t_end; t += kDecWarps) {
      cp_wait<C::kStages - 2>();
      __syncwarp();
      {
        int ahead = stage + C::kStages - 1;
        if (ahead >= C::kStages) ahead -= C::kStages;
        load(t + (C::kStages - 1) * kDecWarps, ahead);
      }
      const uint32_t kb = ring_u + stage * C::kStageBytes;
      const uint32_t vb = kb + C::kHalfBytes;
      // ---- S^T = K Q^T ----
      float sc[NT][4];
#pragma unroll
      for (int n8 = 0; n8 < NT; ++n8)
#pragma unroll
        for (int u = 0; u < 4; ++u) sc[n8][u] = 0.f;
      if constexpr (!FP8) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t f[4];
          ldsm4(kb + dec_off<C::kRowBytes>((lane & 7) + (lane & 8), 2 * ks + (lane >> 4)), f);
#pragma unroll
          for (int n8 = 0; n8 < NT; ++n8)
            mma16816(sc[n8], f[0], f[1], f[2], f[3], qf[n8][ks][0], qf[n8][ks][1]);
        }
      } else {
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {
          uint32_t f[4];        // keys 0-7 and 8-15 of 16 d's, then of the next 16
          ldsm4(kb + dec_off<C::kRowBytes>((lane & 7) + (lane & 8), 2 * k2 + (lane >> 4)), f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a0 = e4m3x2_bf16x2(f[2 * i]), a2 = e4m3x2_bf16x2(f[2 * i] >> 16);
            const uint32_t a1 = e4m3x2_bf16x2(f[2 * i + 1]), a3 = e4m3x2_bf16x2(f[2 * i + 1] >> 16);
#pragma unroll
            for (int n8 = 0; n8 < NT; ++n8)
              mma16816(sc[n8], a0, a1, a2, a3, qf[n8][2 * k2 + i][0], qf[n8][2 * k2 + i][1]);
          }
        }
      }
      // ---- mask and online softmax; rows g and g + 8 are the keys ----
      const int key = st.key(t);
      const int pg = __ldg(row + (key >> p.page_log2));
      const bool ok = pg >= 0 && pg < p.P;
      const bool in0 = ok && seen(key + g), in1 = ok && seen(key + g + 8);
      uint32_t pb[NT][2];
#pragma unroll
      for (int n8 = 0; n8 < NT; ++n8) {
        float al[2];
        float pr[4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float y0 = in0 ? sc[n8][u] * sl2 : NEG_INF;
          const float y1 = in1 ? sc[n8][2 + u] * sl2 : NEG_INF;
          float mx = fmaxf(y0, y1);
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
          const float mn = fmaxf(a.m[n8][u], mx);
          const float mu = mn == NEG_INF ? 0.f : mn;
          al[u] = ex2(a.m[n8][u] - mu);
          a.m[n8][u] = mn;
          pr[u] = ex2(y0 - mu);
          pr[2 + u] = ex2(y1 - mu);
          a.l[n8][u] = fmaf(a.l[n8][u], al[u], pr[u] + pr[2 + u]);
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
        pb[n8][0] = movm(pack_bf16(pr[0], pr[1]));
        pb[n8][1] = movm(pack_bf16(pr[2], pr[3]));
      }
      // ---- A^T += V^T P^T ----
      if constexpr (!FP8) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t f[4];        // keys 0-7: d 0-7, d 8-15; keys 8-15: the same
          ldsm4t(vb + dec_off<C::kRowBytes>((lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)), f);
#pragma unroll
          for (int n8 = 0; n8 < NT; ++n8)
            mma16816(a.acc[n8][i], f[0], f[1], f[2], f[3], pb[n8][0], pb[n8][1]);
        }
      } else {
#pragma unroll
        for (int i2 = 0; i2 < D / 32; ++i2) {
          uint32_t f[4];        // keys 0-7, keys 8-15 of 16 d's, then of the next 16
          ldsm4t(vb + dec_off<C::kRowBytes>((lane & 7) + (lane & 8), 2 * i2 + (lane >> 4)), f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // a thread holds d's 2 g, 2 g + 1 of keys c2 and c2 + 1: rows g
            // and g + 8 of the fragment stand for d = 2 g and 2 g + 1
            const uint32_t lo = f[2 * i], hi = f[2 * i + 1];
            const uint32_t a0 = e4m3x2_bf16x2(__byte_perm(lo, 0, 0x4420));
            const uint32_t a1 = e4m3x2_bf16x2(__byte_perm(lo, 0, 0x4431));
            const uint32_t a2 = e4m3x2_bf16x2(__byte_perm(hi, 0, 0x4420));
            const uint32_t a3 = e4m3x2_bf16x2(__byte_perm(hi, 0, 0x4431));
#pragma unroll
            for (int n8 = 0; n8 < NT; ++n8)
              mma16816(a.acc[n8][2 * i2 + i], a0, a1, a2, a3, pb[n8][0], pb[n8][1]);
          }
        }
      }
      __syncwarp();                     // the stage may be refilled
      if (++stage == C::kStages) stage = 0;
    }
    cp_wait<0>();

    // ---- the four warps' states become one ----
    __syncthreads();                    // every warp is done with its ring
    float* merge = reinterpret_cast<float*>(dec_smem);     // [warp][head][kMergeRow]: A | m, l
#pragma unroll
    for (int n8 = 0; n8 < NT; ++n8) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float l = a.l[n8][u];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
        float* mr = merge + ((warp * NT + n8) * 8 + c2 + u) * C::kMergeRow;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          mr[16 * i + (FP8 ? 2 * g : g)] = a.acc[n8][i][u];
          mr[16 * i + (FP8 ? 2 * g + 1 : g + 8)] = a.acc[n8][i][2 + u];
        }
        if (g == 0) {
          mr[D] = a.m[n8][u];
          mr[D + 1] = l;
        }
      }
    }
    __syncthreads();
    const bool whole = ta == 0 && tb == nt;
    const bool head = ta > 0;
    float* part = p.part + (static_cast<size_t>(cta) * 2 + (head ? 0 : 1)) * 16 * (D + 2);
    const float vs = FP8 ? __ldg(p.v_scale + hkv) : 1.f;
    for (int e = tid; e < nh * (D / 2); e += kDecThreads) {
      const int hh = e / (D / 2);
      const int d2 = (e - hh * (D / 2)) * 2;
      float m = NEG_INF;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, merge[(w * NT * 8 + hh) * C::kMergeRow + D]);
      float l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float* mr = merge + (w * NT * 8 + hh) * C::kMergeRow;
        if (mr[D + 1] == 0.f) continue;      // this warp saw no key
        const float f = ex2(mr[D] - m);
        l = fmaf(f, mr[D + 1], l);
        y0 = fmaf(f, mr[d2], y0);
        y1 = fmaf(f, mr[d2 + 1], y1);
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : vs / l;
        const size_t oh = static_cast<size_t>(s) * p.H + h0 + hh;
        *reinterpret_cast<uint32_t*>(p.o + oh * D + d2) = pack_bf16(y0 * inv, y1 * inv);
        if (d2 == 0) p.lse[oh] = l == 0.f ? NEG_INF : (m + __log2f(l)) * kLn2;
      } else {
        part[hh * (D + 2) + d2] = y0;
        part[hh * (D + 2) + d2 + 1] = y1;
        if (d2 == 0) {
          part[hh * (D + 2) + D] = m;
          part[hh * (D + 2) + D + 1] = l;
        }
      }
    }
    if (!whole && !head) {
      // the unit's last tile y lies in the last CTA c with tiles c / active <= y
      meta.x = s * units + r;
      meta.y = static_cast<int>(((unit_x + nt) * active + tiles - 1) / tiles) - 1;
    }
    __syncthreads();                    // the merge area is the ring again

    // ---- the next unit ----
    x = unit_x + tb;
    if (tb == nt && x < x1) {
      unit_x += nt;
      if (++r == units) {
        r = 0;
        do {
          ++s;
          st = seq_steps(__ldg(p.lens + s), p);
        } while (st.total == 0);
        nt = (st.total + kDecWarps - 1) / kDecWarps;
      }
    }
  }
  if (tid == 0) p.meta[cta] = meta;
}

// Joins the parts of a unit that begins in CTA blockIdx.x and goes on: one
// block per (CTA, query head); 8 warps take the parts in turn, and their sums
// are added in order.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attn_decode_join_kernel(const DecodeParams p) {
  __shared__ float sh[kJoinWarps][D + 2];
  const int c = static_cast<int>(blockIdx.x), hh = static_cast<int>(blockIdx.y);
  const int unit = p.meta[c].x;
  if (unit < 0) return;
  const int end = p.meta[c].y;
  const int units = p.Hkv * p.q_tiles;
  const int s = unit / units, r = unit - s * units;
  const int hkv = r / p.q_tiles;
  const int h0 = hkv * p.G + (r - hkv * p.q_tiles) * 16;
  if (hh >= min(16, (hkv + 1) * p.G - h0)) return;
  const int warp = static_cast<int>(warp_id()), lane = static_cast<int>(lane_id());
  const float NEG_INF = -__int_as_float(0x7f800000);
  constexpr int V = D / 32;
  float m = NEG_INF, l = 0.f, y[V];
#pragma unroll
  for (int i = 0; i < V; ++i) y[i] = 0.f;
  for (int x = c + warp; x <= end; x += kJoinWarps) {
    const float* pt = p.part + ((static_cast<size_t>(x) * 2 + (x == c ? 1 : 0)) * 16 + hh) * (D + 2);
    const float mx = pt[D], lx = pt[D + 1];
    if (lx == 0.f) continue;
    const float mn = fmaxf(m, mx);
    const float fa = ex2(m - mn), fb = ex2(mx - mn);
    m = mn;
    l = fmaf(l, fa, lx * fb);
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = fmaf(y[i], fa, pt[i * 32 + lane] * fb);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sh[warp][i * 32 + lane] = y[i];
  if (lane == 0) {
    sh[warp][D] = m;
    sh[warp][D + 1] = l;
  }
  __syncthreads();
  const int e = static_cast<int>(threadIdx.x) * 2;
  if (e >= D) return;
  float mm = NEG_INF;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) mm = fmaxf(mm, sh[w][D]);
  float ll = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (sh[w][D + 1] == 0.f) continue;
    const float f = ex2(sh[w][D] - mm);
    ll = fmaf(f, sh[w][D + 1], ll);
    y0 = fmaf(f, sh[w][e], y0);
    y1 = fmaf(f, sh[w][e + 1], y1);
  }
  const float vs = p.v_scale ? __ldg(p.v_scale + hkv) : 1.f;
  const float inv = ll == 0.f ? 0.f : vs / ll;
  const size_t oh = static_cast<size_t>(s) * p.H + h0 + hh;
  *reinterpret_cast<uint32_t*>(p.o + oh * D + e) = pack_bf16(y0 * inv, y1 * inv);
  if (e == 0) p.lse[oh] = ll == 0.f ? NEG_INF : (mm + __log2f(ll)) * kLn2;
}

constexpr int kDecMaxCtas = 152 * 3;

size_t decode_workspace(int d) {
  return static_cast<size_t>(kDecMaxCtas) * 16 + static_cast<size_t>(kDecMaxCtas) * 2 * 16 * (d + 2) * 4;
}

template <int D, bool FP8, int NT>
cudaError_t launch_decode(const DecodeParams& p, cudaStream_t st) {
  using C = DecCfg<D, FP8, NT>;
  auto kern = attn_decode_paged_kernel<D, FP8, NT>;
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
  // no more CTAs than the table's rows can hold tiles
  const long long most = ((static_cast<long long>(p.M) << p.page_log2) + kDecTile - 1) / kDecTile *
                         p.S * p.Hkv * p.q_tiles;
  const int grid = static_cast<int>(std::max(1ll, std::min<long long>(kDecMaxCtas, most)));
  kern<<<grid, kDecThreads, C::kSmem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  attn_decode_join_kernel<D><<<dim3(grid, std::min(16, p.G)), kJoinWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

bool decode_sizes(int S, int H, int Hkv, int d) {
  if (S < 1 || H < 1 || !valid_kv_heads(H, Hkv) || (d != 64 && d != 128)) return false;
  return S <= kMaxSeqs && static_cast<long long>(S) * H <= 0x7FFFFFFFll;
}

}  // namespace
}  // namespace bss

using namespace bss;

extern "C" size_t attn_decode_paged_workspace_bytes(int S, int H, int H_kv, int d) {
  return decode_sizes(S, H, H_kv, d) ? decode_workspace(d) : 0;
}

extern "C" attn_status_t attn_decode_paged(
    const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int64_t k_page_stride,
    int64_t v_page_stride, int kv_dtype, const float* k_scale, const float* v_scale,
    const int32_t* page_table, const int32_t* seq_lens, void* o, float* lse, void* workspace,
    size_t workspace_bytes, int S, int H, int H_kv, int d, int max_pages, int n_pages, int page_size,
    float scale, int64_t window, int64_t sinks, void* stream) {
  attn_status_t s = check_common(S, H, 1, 1, d, scale);
  if (s != ATTN_OK) return s;
  if (!valid_kv_heads(H, H_kv)) return ATTN_ERR_INVALID_ARG;
  if (S > kMaxSeqs) return ATTN_ERR_UNSUPPORTED;
  if (max_pages < 1 || n_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1))) return ATTN_ERR_UNSUPPORTED;
  if (kv_dtype != ATTN_KV_BF16 && kv_dtype != ATTN_KV_E4M3) return ATTN_ERR_UNSUPPORTED;
  if (window < 0 || sinks < 0 || (window == 0 && sinks != 0)) return ATTN_ERR_INVALID_ARG;
  const void* ptrs16[] = {q, k_cache, v_cache, o, workspace};
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
  if (workspace_bytes < decode_workspace(d)) return ATTN_ERR_WORKSPACE;
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
  p.meta = static_cast<int4*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + static_cast<size_t>(kDecMaxCtas) * 16);
  p.S = S;
  p.H = H;
  p.Hkv = H_kv;
  p.G = H / H_kv;
  p.M = max_pages;
  p.P = n_pages;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.q_tiles = (p.G + 15) / 16;
  p.scale_log2 = scale * kLog2e;
  p.window = std::min<int64_t>(window, int64_t(1) << 60);
  p.sinks = static_cast<int>(std::min<int64_t>(sinks, 0x7FFFFFF0));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool one = p.G <= 8;
  cudaError_t e;
  if (d == 64) {
    e = fp8 ? (one ? launch_decode<64, true, 1>(p, st) : launch_decode<64, true, 2>(p, st))
            : (one ? launch_decode<64, false, 1>(p, st) : launch_decode<64, false, 2>(p, st));
  } else {
    e = fp8 ? (one ? launch_decode<128, true, 1>(p, st) : launch_decode<128, true, 2>(p, st))
            : (one ? launch_decode<128, false, 1>(p, st) : launch_decode<128, false, 2>(p, st));
  }
  return cuda_status("attn_decode_paged launch", e);
}
