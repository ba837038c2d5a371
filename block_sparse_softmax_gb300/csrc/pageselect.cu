// Sparse attention over a paged cache, up to the attention itself: the pages'
// mean keys (attn_kv_pool), and for each new token and K/V head the pages whose
// mean keys score highest (attn_select_pages).
//
// Mathematics: mean_p = (1 / page) sum_r K[p][r]; for a row t that sees the first
// n tokens of its sequence, over the slots m of its table row,
//     score(t, m) = (sum of the group's query heads q_h) . mean_{table[m]},
// which is what the mean logits of the group's heads add up to, but for the
// scale.  Taken are the first pages, the last ones (the row's own among them) and
// the top_r others by score, ties to the lower slot, listed in ascending order.
//
// Which page is taken must not hang on a rounding, so a pick is the exact one:
//   * means: the elements are summed as an unevaluated pair of fp32 numbers by
//     Knuth's two-sum.  The pair is the exact sum where the largest element is at
//     most 2^34 / page times the smallest that is not 0 (kPoolSpread); a column of
//     others, or one past fp32's range, is summed again in whole numbers.  The page
//     size is a power of two, so there is one rounding, the mean's own to fp32.
//     (1024 e4m3 elements are a pair in any order; with their scale's product a mean
//     is off by 2^-24 and 2^-46 at most.)
//   * scores: in fp32 first, each off by at most
//         e = (G + r + 2) 2^-24 sum_i A_i max_mi |mean_mi|,   A = sum_h |q_h|
//     (G roundings of the group's sum at most and r of a product's, on terms whose
//     absolute values add up to at most that sum; r = d / 32 + 5 for a lane's chain
//     and the tree over the lanes, d for one chain).  The top_r-th largest of numbers
//     that are off by e is off by e, so what lies more than 2 e above it is taken and
//     more than 2 e below is not.  What lies between (as a rule, that one page) is
//     scored again, in whole numbers of 128 bits, of which the last stands for at
//     most 2^-110 times sum_i A_i max_mi |mean_mi|; each product's bits below that are
//     dropped.  A product of a query's element and a mean's that is not below 2^-60
//     times the largest of both keeps all of its 32 bits, and scores of the same
//     products are the same in any order.  (Pairs of fp64 numbers, which a
//     multiprocessor has two lanes for, took 16 times as long.)
#include <cuda_fp16.h>

#include <algorithm>

#include "paged.cuh"

namespace bss {
namespace {

constexpr int kMaxSelectPages = 32768;        // slots of a table row: their keys fill 128 KB

// ----------------------------------------------------------------------------
// means
// ----------------------------------------------------------------------------
struct PoolParams {
  const uint8_t* k;
  size_t k_stride;          // bytes from page to page
  const float* k_scale;
  float* means;             // [P][Hkv][d]
  const int* table;
  const int* start;
  const int* lens;
  int S, M, P, Hkv, page_log2;
  int warps;                // of a (page, head)
  int* err;
};

// x added to the pair hi + lo, exactly but for lo's rounding.
__device__ __forceinline__ void two_sum(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x);
  const float b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}

// When lo rounds.  With fields f of bf16 exponents between f0 (of an element other
// than 0) and f1, every sum is a multiple of u = 2^(f0 - 134), an element less than A
// = 2^(f1 - 126).  A lane adds up 64 elements at most, two levels of lanes and then
// 8 warps join: over all additions the sums' absolute values come to less than
// 39 page A, and their errors, each at most 2^-24 of its sum, to 2^-18 page A.  That
// is less than 2^24 u, so that lo has bits for all of them, where f1 - f0 <= 34 -
// log2(page).
constexpr int kPoolSpread = 34;

// The means of the eight columns at `src` (rows `stride` apart, bf16) by a warp, a
// lane's in lane / 4, rounded once: a finite element is an 8-bit number times
// 2^(s - 133), s < 254, and counts in the s / 32-th of eight 64-bit sums, shifted by
// s % 32 (8 + 31 bits, a sign and 2^10 rows).  Their carries settled, the sums are
// the 32-bit digits of the whole.
__device__ __noinline__ float exact_mean(const uint16_t* src, int stride, int page_log2) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  long long sum[8];
  float odd = 0.f;                            // infinities and NaN, as they add up
#pragma unroll
  for (int w = 0; w < 8; ++w) sum[w] = 0;
#pragma unroll 8
  for (int r = lane & 3; r < 1 << page_log2; r += 4) {
    const uint32_t x = __ldg(src + static_cast<size_t>(r) * stride + (lane >> 2));
    const int field = static_cast<int>(x >> 7 & 255u);
    if (field == 255) odd += __uint_as_float(x << 16);
    const int s = max(field, 1) - 1;
    long long v = static_cast<long long>((x & 127u) | (field != 0 ? 128u : 0u)) << (s & 31);
    if (x >> 15) v = -v;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum[w] += s >> 5 == w ? v : 0;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    odd += __shfl_xor_sync(0xFFFFFFFFu, odd, o);
#pragma unroll
    for (int w = 0; w < 8; ++w) sum[w] += __shfl_xor_sync(0xFFFFFFFFu, sum[w], o);
  }
  if (odd != 0.f) return odd;
  // the digits of the sum's absolute value; the ninth takes what eight sums carry over
  long long carry = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) carry = (sum[w] + carry) >> 32;
  const bool negative = carry < 0;
  uint32_t digit[9];
  carry = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    carry += negative ? -sum[w] : sum[w];
    digit[w] = static_cast<uint32_t>(carry);
    carry >>= 32;
  }
  digit[8] = static_cast<uint32_t>(carry);
  // the highest digit and the one below it, and a bit for all that lies lower: the
  // rounding to fp32 is the only one (a mean below fp32's normal numbers is a
  // multiple of their last place)
  unsigned long long top = static_cast<unsigned long long>(digit[0]) << 32;
  int at = 0;
#pragma unroll
  for (int w = 1; w < 9; ++w) {
    if (digit[w] != 0u) {
      top = static_cast<unsigned long long>(digit[w]) << 32 | digit[w - 1];
      at = w;
    }
  }
#pragma unroll
  for (int w = 0; w < 7; ++w)
    if (w < at - 1 && digit[w] != 0u) top |= 1ull;
  const float f = ldexpf(__ull2float_rn(top), 32 * (at - 1) - 133 - page_log2);
  return negative ? -f : f;
}

__device__ __forceinline__ float2 e4m3x2_f32x2(uint32_t x) {        // the low 16 bits
  const uint32_t y = e4m3x2_f16x2(x);
  return __half22float2(*reinterpret_cast<const __half2*>(&y));
}

// `W` warps a (page, head), each with all of its part's loads in flight (up to 8 of
// 16 bytes a lane; 32 * 16 / (bytes of a row) rows arrive with each), joined in
// order in shared memory.  A page's part is what a warp waits for once: with a warp
// a page of 64 tokens, four times, a prompt of 16384 took 10.8 us.  (The
// same with more warps, from L2 and among others: 8.8 us, 7.8 without the span of the
// elements' magnitudes; a test of every addition to lo instead took 1 to 2 more.  With
// a column a page that is summed again 13, with all of them 49.)
constexpr int kPoolWarps = 8;
constexpr int kPoolBatch = 8;
template <int D, bool FP8>
__global__ void __launch_bounds__(kPoolWarps * 32) kv_pool_kernel(const PoolParams p) {
  constexpr int kEl = FP8 ? 16 : 8;           // elements of 16 bytes
  constexpr int kLanes = D / kEl;             // lanes of a row
  constexpr int kRows = 32 / kLanes;          // rows of a load
  __shared__ float2 parts[kPoolWarps][D];
  __shared__ uint2 spans[kPoolWarps][FP8 ? 1 : D / 2];
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int loads = (1 << p.page_log2) / kRows;            // of a page (16 rows at least, 8 a load at most)
  const int W = p.warps, each = loads / W;                 // warps of an item, loads of a warp
  const int items_cta = kPoolWarps / W;
  const float share = 1.f / static_cast<float>(1 << p.page_log2);
  for (int sq = static_cast<int>(blockIdx.y); sq < p.S; sq += static_cast<int>(gridDim.y)) {
    const int a = __ldg(p.start + sq), n = __ldg(p.lens + sq);
    if (a < 0) continue;                      // nothing was reserved
    const long long most = static_cast<long long>(p.M) << p.page_log2;
    if (n < 0 || n > most) {
      if (threadIdx.x == 0 && blockIdx.x == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
      continue;
    }
    const int m0 = a >> p.page_log2, pages = max(0, (n >> p.page_log2) - m0);
    // items (a page and head each) in rounds of the whole CTA, whose warps meet in each
    const long long items = static_cast<long long>(pages) * p.Hkv;
    for (long long x = static_cast<long long>(blockIdx.x) * items_cta; x < items;
         x += static_cast<long long>(gridDim.x) * items_cta) {
      const long long item = x + warp / W;
      const int i = item < items ? static_cast<int>(item / p.Hkv) : pages;
      const int h = static_cast<int>(item - static_cast<long long>(i) * p.Hkv);
      int pg = i < pages ? __ldg(p.table + static_cast<size_t>(sq) * p.M + m0 + i) : -1;
      if (pg < -1 || pg >= p.P) {             // (-1: given back already)
        if (lane == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
        pg = -1;
      }
      float hi[kEl], lo[kEl];
      // bf16: two columns' largest magnitudes, bit 15 set, and the smallest less 1, bit
      // 15 set before (as signed numbers: 0 becomes the largest there is)
      uint32_t big[kEl / 2], small[kEl / 2];
#pragma unroll
      for (int e = 0; e < kEl; ++e) hi[e] = lo[e] = 0.f;
#pragma unroll
      for (int e = 0; e < kEl / 2; ++e) {
        big[e] = 0x80008000u;
        small[e] = 0x7FFF7FFFu;
      }
      auto join = [&](int e, float oh, float ol) {
        two_sum(hi[e], lo[e], oh);
        lo[e] = __fadd_rn(lo[e], ol);
      };
      auto widen = [&](int e, uint32_t other_big, uint32_t other_small) {
        big[e] = __vmaxu2(big[e], other_big);
        small[e] = __vmins2(small[e], other_small);
      };
      if (pg >= 0) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.k + pg * p.k_stride + ((static_cast<size_t>(h) << p.page_log2) * D) * (FP8 ? 1 : 2)) + lane +
            warp % W * each * 32;
        for (int i0 = 0; i0 < each; i0 += kPoolBatch) {
          uint4 v[kPoolBatch];
#pragma unroll
          for (int u = 0; u < kPoolBatch; ++u)
            v[u] = i0 + u < each ? __ldg(src + (i0 + u) * 32) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int u = 0; u < kPoolBatch; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if constexpr (FP8) {
                const float2 c0 = e4m3x2_f32x2(w[e]), c1 = e4m3x2_f32x2(w[e] >> 16);
                two_sum(hi[4 * e], lo[4 * e], c0.x);
                two_sum(hi[4 * e + 1], lo[4 * e + 1], c0.y);
                two_sum(hi[4 * e + 2], lo[4 * e + 2], c1.x);
                two_sum(hi[4 * e + 3], lo[4 * e + 3], c1.y);
              } else {
                two_sum(hi[2 * e], lo[2 * e], bf16lo(w[e]));
                two_sum(hi[2 * e + 1], lo[2 * e + 1], bf16hi(w[e]));
                const uint32_t magnitude = w[e] | 0x80008000u;
                widen(e, magnitude, magnitude - 0x00010001u);
              }
            }
          }
        }
        // the lanes that hold the same columns of other rows
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) {
#pragma unroll
          for (int e = 0; e < kEl; ++e) {
            const float oh = __shfl_xor_sync(0xFFFFFFFFu, hi[e], o);
            const float ol = __shfl_xor_sync(0xFFFFFFFFu, lo[e], o);
            join(e, oh, ol);
          }
#pragma unroll
          for (int e = 0; e < (FP8 ? 0 : kEl / 2); ++e) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, big[e], o);
            widen(e, other, __shfl_xor_sync(0xFFFFFFFFu, small[e], o));
          }
        }
      }
      if (W > 1) {
        if (lane < kLanes) {
#pragma unroll
          for (int e = 0; e < kEl; ++e) parts[warp][lane * kEl + e] = make_float2(hi[e], lo[e]);
#pragma unroll
          for (int e = 0; e < (FP8 ? 0 : kEl / 2); ++e)
            spans[warp][lane * (kEl / 2) + e] = make_uint2(big[e], small[e]);
        }
        __syncthreads();
        if (warp % W == 0 && lane < kLanes)
          for (int w = 1; w < W; ++w) {
#pragma unroll
            for (int e = 0; e < kEl; ++e) {
              const float2 y = parts[warp + w][lane * kEl + e];
              join(e, y.x, y.y);
            }
#pragma unroll
            for (int e = 0; e < (FP8 ? 0 : kEl / 2); ++e) {
              const uint2 y = spans[warp + w][lane * (kEl / 2) + e];
              widen(e, y.x, y.y);
            }
          }
      }
      if (pg >= 0 && warp % W == 0) {          // (a whole warp)
        float* dst = p.means + (static_cast<size_t>(pg) * p.Hkv + h) * D;
        bool again = false;                   // bf16: one of this lane's pairs may not be its sum
        if (lane < kLanes) {
          const float f = FP8 ? __ldg(p.k_scale + h) : 1.f;
#pragma unroll
          for (int e = 0; e < kEl; e += 4) {
            float y[4];
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              // the pair (times the scale: with the product's own rest), rounded once; in
              // fp32, for a multiprocessor has two fp64 lanes.  A NaN's lo is a NaN, and
              // left out, as is what a product past fp32's range leaves.
              const float hh = hi[e + i4] * share, ll = lo[e + i4] * share;
              const float pr = hh * f;
              if constexpr (FP8) {
                y[i4] = !isfinite(pr) ? pr : __fadd_rn(pr, fmaf(hh, f, -pr) + ll * f);
              } else {
                y[i4] = __fadd_rn(hi[e + i4], lo[e + i4]) * share;
                const int half = 16 * (i4 & 1), c = (e + i4) / 2;
                const int f1 = static_cast<int>(big[c] >> half >> 7 & 255u);
                const int f0 = static_cast<int>(((small[c] >> half) + 1u) >> 7 & 255u);  // (0, too, where all are 0)
                again = again || f1 - max(f0, 1) > kPoolSpread - p.page_log2 || !isfinite(hi[e + i4]);
              }
            }
            *reinterpret_cast<float4*>(dst + lane * kEl + e) = make_float4(y[0], y[1], y[2], y[3]);
          }
        }
        if constexpr (!FP8) {
          uint32_t todo = __ballot_sync(0xFFFFFFFFu, again);
          if (todo != 0u) __syncwarp();       // (after the stores above)
          for (; todo != 0u; todo &= todo - 1) {
            const int c = (__ffs(todo) - 1) * kEl;
            const float y = exact_mean(reinterpret_cast<const uint16_t*>(p.k + pg * p.k_stride) +
                                           (static_cast<size_t>(h) << p.page_log2) * D + c, D, p.page_log2);
            if ((lane & 3) == 0) dst[c + lane / 4] = y;
          }
        }
      }
      if (W > 1) __syncthreads();             // the parts have been read
    }
  }
}

// ----------------------------------------------------------------------------
// scores
// ----------------------------------------------------------------------------
struct SelectParams {
  const __nv_bfloat16* q;
  long long q_stride;
  const float* means;
  const int* table;
  const int* lens;
  const int* cu;
  int t0, rows;             // the rows of this launch
  int T, S, H, Hkv, G, M, P;
  int page_log2;
  int top, local, first, R;
  int parts;                // score CTAs along a row
  int rounds;               // roundings of a score's sum
  float* score;             // [rows][Hkv][M]; then words of what is scored again
  float* norm;              // [rows][Hkv][parts]: the largest |mean| element met
  int* pages;               // [T][Hkv][R]
  int* out_lens;            // [T]
  int* err;
};

// A row's sequence and what it sees.  Rows of no sequence have s = -1.
struct SelectRow {
  int s;
  int n;                    // tokens, its own among them (0: none)
  int held;                 // pages they lie in
};
__device__ __forceinline__ SelectRow select_row(const SelectParams& p, int t, int lane) {
  int lo = 0, hi = p.S + 1;                   // the last s with cu[s] <= t, by a whole warp
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const uint32_t yes = __ballot_sync(0xFFFFFFFFu, lane == 0 || (i < hi && __ldg(p.cu + i) <= t));
    lo += (31 - __clz(yes)) * step;
    hi = min(hi, lo + step);
  }
  SelectRow r{-1, 0, 0};
  if (lo >= p.S || __ldg(p.cu + lo) > t) return r;
  r.s = lo;
  const long long most = min(static_cast<long long>(p.M) << p.page_log2, static_cast<long long>(kMaxTokens));
  const long long len = min(static_cast<long long>(__ldg(p.lens + lo)), most);
  const long long n = len - (static_cast<long long>(__ldg(p.cu + lo + 1)) - t) + 1;
  r.n = static_cast<int>(max(0ll, min(n, len)));
  r.held = static_cast<int>((static_cast<long long>(r.n) + (1 << p.page_log2) - 1) >> p.page_log2);
  return r;
}
// The slots that are scored: [first, end); those below and from end on are taken anyway.
__device__ __forceinline__ int scored_end(const SelectParams& p, const SelectRow& r) {
  return max(r.held - p.local, min(p.first, r.held));
}

// The larger one; a NaN stays.
__device__ __forceinline__ float larger_or_nan(float a, float b) { return b > a || b != b ? b : a; }

constexpr int kScoreWarps = 4;
constexpr int kScorePages = 8;                // pages of a warp's turn

// Row by row (a token a sequence): bound by reading the means.  CTA x of `parts`
// takes every parts-th group of pages, a warp 8 at a time, a row of means a load.
template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) select_score_kernel(const SelectParams p) {
  constexpr int E = D / 32;                   // elements a lane
  __shared__ float top[kScoreWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int r = static_cast<int>(blockIdx.y), h = static_cast<int>(blockIdx.z);
  const int t = p.t0 + r;
  float q[E];
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = 0.f;
  const __nv_bfloat16* src = p.q + t * p.q_stride + static_cast<long long>(h) * p.G * D + lane * E;
  for (int g = 0; g < p.G; ++g, src += D) {
    if constexpr (E == 4) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
      q[0] += bf16lo(x.x), q[1] += bf16hi(x.x), q[2] += bf16lo(x.y), q[3] += bf16hi(x.y);
    } else {
      const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(src));
      q[0] += bf16lo(x), q[1] += bf16hi(x);
    }
  }
  const SelectRow row = select_row(p, t, lane);
  const int end = row.s < 0 ? 0 : scored_end(p, row);
  const int* tab = p.table + static_cast<size_t>(max(row.s, 0)) * p.M;
  float* score = p.score + (static_cast<size_t>(r) * p.Hkv + h) * p.M;
  float most = 0.f;
  for (long long g = static_cast<long long>(blockIdx.x) * kScoreWarps + warp; p.first + g * kScorePages < end;
       g += static_cast<long long>(p.parts) * kScoreWarps) {
    const int m0 = p.first + static_cast<int>(g) * kScorePages;
    int pg = lane < kScorePages && m0 + lane < end ? __ldg(tab + m0 + lane) : -1;
    if (pg >= p.P || pg < -1) {
      record_error(p.err, ATTN_ERR_BAD_PAGES);
      pg = -1;
    }
    float v[kScorePages][E];
#pragma unroll
    for (int u = 0; u < kScorePages; ++u) {
      const int x = __shfl_sync(0xFFFFFFFFu, pg, u);
      const float* from = p.means + (static_cast<size_t>(max(x, 0)) * p.Hkv + h) * D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) v[u][e] = 0.f;
      if (x >= 0) {
        if constexpr (E == 4) {
          const float4 y = __ldg(reinterpret_cast<const float4*>(from));
          v[u][0] = y.x, v[u][1] = y.y, v[u][2] = y.z, v[u][3] = y.w;
        } else {
          const float2 y = __ldg(reinterpret_cast<const float2*>(from));
          v[u][0] = y.x, v[u][1] = y.y;
        }
      }
    }
    float mine = 0.f;
#pragma unroll
    for (int u = 0; u < kScorePages; ++u) {
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        most = larger_or_nan(most, fabsf(v[u][e]));
        d = fmaf(q[e], v[u][e], d);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
      if (lane == u) mine = d;
    }
    if (lane < kScorePages && m0 + lane < end) score[m0 + lane] = mine;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = larger_or_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  if (lane == 0) top[warp] = most;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kScoreWarps; ++w) most = larger_or_nan(most, top[w]);
    p.norm[(static_cast<size_t>(r) * p.Hkv + h) * p.parts + blockIdx.x] = most;
  }
}

// Chunks: 32 rows share the means of 128 pages of their sequence in shared memory
// (read from L2 once for 32 rows), a thread two pages and 8 rows: a dot product is
// a chain of d fused multiply-adds.  500 rows of 1024 pages, 4 K/V heads: 31 us; half
// the threads, 16 rows each 34; a warp a page and sums over its lanes, 8 rows at a
// time, 142.
constexpr int kTileRows = 32;
constexpr int kTilePages = 128;
constexpr int kTileThreads = 256;
template <int D>
struct ScoreTile {
  static constexpr int kRow = D + 4;          // floats from page to page: 16 bytes of 8 pages hit 8 different banks
  static constexpr int kSmem = (kTilePages * kRow + kTileRows * D) * 4;
};
template <int D>
__global__ void __launch_bounds__(kTileThreads) select_score_tile_kernel(const SelectParams p) {
  using C = ScoreTile<D>;
  extern __shared__ __align__(16) float score_smem[];
  float* means = score_smem;                  // [pages][kRow]
  float* qsum = score_smem + kTilePages * C::kRow;             // [rows][D]
  __shared__ int row_s[kTileRows], row_end[kTileRows];
  __shared__ float top[kTileThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int h = static_cast<int>(blockIdx.z);
  const int r0 = static_cast<int>(blockIdx.y) * kTileRows;
  const int nr = min(kTileRows, p.rows - r0);
  // the group's sums, 8 columns a thread
  for (int i = tid; i < kTileRows * D / 8; i += kTileThreads) {
    const int r = i / (D / 8), e = i % (D / 8) * 8;
    float sum[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) sum[u] = 0.f;
    if (r < nr) {
      const __nv_bfloat16* q = p.q + (p.t0 + r0 + r) * p.q_stride + static_cast<long long>(h) * p.G * D + e;
#pragma unroll 4
      for (int g = 0; g < p.G; ++g) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(q + static_cast<long long>(g) * D));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          sum[2 * u] += bf16lo(w[u]);
          sum[2 * u + 1] += bf16hi(w[u]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) qsum[r * D + e + u] = sum[u];
  }
  // the first row's sequence by search, a later row's mostly the same one
  if (warp == 0) {
    const SelectRow first = select_row(p, p.t0 + r0, lane);
    SelectRow row = first;
    const int t = p.t0 + r0 + lane;
    bool other = false;
    if (lane < nr) {
      other = first.s < 0 || __ldg(p.cu + first.s + 1) <= t;
      row.n = first.n + lane;                 // (in the same sequence)
      row.held = static_cast<int>((static_cast<long long>(row.n) + (1 << p.page_log2) - 1) >> p.page_log2);
    }
    for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, other); todo != 0u; todo &= todo - 1) {
      const int r = __ffs(todo) - 1;
      const SelectRow x = select_row(p, p.t0 + r0 + r, lane);
      if (lane == r) row = x;
    }
    if (lane < kTileRows) {
      row_s[lane] = lane < nr ? row.s : -1;
      row_end[lane] = lane < nr && row.s >= 0 ? scored_end(p, row) : 0;
    }
  }
  __syncthreads();
  constexpr int kWarpPages = kTilePages / (kTileThreads / 32);
  float seen = 0.f;                           // the largest element met, for any of the rows
  for (int a = 0; a < nr;) {                  // runs of rows of one sequence
    const int s = row_s[a];
    int b = a + 1, end = row_end[a];
    while (b < nr && row_s[b] == s) end = max(end, row_end[b++]);
    const int* tab = p.table + static_cast<size_t>(max(s, 0)) * p.M;
    for (long long m1 = p.first + static_cast<long long>(blockIdx.x) * kTilePages; s >= 0 && m1 < end;
         m1 += static_cast<long long>(p.parts) * kTilePages) {
      const int m0 = static_cast<int>(m1);
      const int mine = warp * kWarpPages + lane;           // of its warp's pages
      int pg = lane < kWarpPages && m0 + mine < end ? __ldg(tab + m0 + mine) : -1;
      if (pg >= p.P || pg < -1) {
        record_error(p.err, ATTN_ERR_BAD_PAGES);
        pg = -1;
      }
      __syncthreads();                        // the tile before has been read
      // a warp its pages, 8 rows of means in flight
#pragma unroll 1
      for (int u0 = 0; u0 < kWarpPages; u0 += 8) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int x = __shfl_sync(0xFFFFFFFFu, pg, u0 + u);
          const float* from = p.means + (static_cast<size_t>(max(x, 0)) * p.Hkv + h) * D + lane * 4;
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (x >= 0 && lane * 4 < D) v[u] = __ldg(reinterpret_cast<const float4*>(from));
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          seen = larger_or_nan(larger_or_nan(seen, fabsf(v[u].x)), fabsf(v[u].y));
          seen = larger_or_nan(larger_or_nan(seen, fabsf(v[u].z)), fabsf(v[u].w));
          if (lane * 4 < D)
            *reinterpret_cast<float4*>(means + (warp * kWarpPages + u0 + u) * C::kRow + lane * 4) = v[u];
        }
      }
      __syncthreads();
      constexpr int kHalf = kTileRows / (kTileThreads / 64);
      const int x0 = tid & 63, rh = tid / 64 * kHalf;      // pages x0 and x0 + 64, rows rh ..
      float acc[2][kHalf];
#pragma unroll
      for (int r = 0; r < kHalf; ++r) acc[0][r] = acc[1][r] = 0.f;
#pragma unroll 2
      for (int e = 0; e < D; e += 4) {
        const float4 v0 = *reinterpret_cast<const float4*>(means + x0 * C::kRow + e);
        const float4 v1 = *reinterpret_cast<const float4*>(means + (x0 + 64) * C::kRow + e);
#pragma unroll
        for (int r = 0; r < kHalf; ++r) {
          const float4 q = *reinterpret_cast<const float4*>(qsum + (rh + r) * D + e);
          acc[0][r] = fmaf(q.x, v0.x, fmaf(q.y, v0.y, fmaf(q.z, v0.z, fmaf(q.w, v0.w, acc[0][r]))));
          acc[1][r] = fmaf(q.x, v1.x, fmaf(q.y, v1.y, fmaf(q.z, v1.z, fmaf(q.w, v1.w, acc[1][r]))));
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int m = m0 + x0 + 64 * u;
        if (m >= end) continue;
#pragma unroll
        for (int r = 0; r < kHalf; ++r)
          if (rh + r >= a && rh + r < b)
            p.score[(static_cast<size_t>(r0 + rh + r) * p.Hkv + h) * p.M + m] = acc[u][r];
      }
    }
    a = b;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) seen = larger_or_nan(seen, __shfl_xor_sync(0xFFFFFFFFu, seen, o));
  if (lane == 0) top[warp] = seen;
  __syncthreads();
  if (tid < nr) {
    float x = 0.f;
    for (int w = 0; w < kTileThreads / 32; ++w) x = larger_or_nan(x, top[w]);
    p.norm[(static_cast<size_t>(r0 + tid) * p.Hkv + h) * p.parts + blockIdx.x] = x;
  }
}

// ----------------------------------------------------------------------------
// the pick
// ----------------------------------------------------------------------------
// A column's sum over the group's query heads, in units of 2^(Q - 94); `odd` adds up
// its infinities and NaN (0: there are none).
struct __align__(16) FixedSum {
  unsigned long long lo;
  int hi;
  float odd;
  __device__ __forceinline__ __int128 value() const { return static_cast<__int128>(hi) << 64 | lo; }
};

// The want-th largest (want >= 1) of the keys key(i) of `bits` bits, i in [lo, hi),
// of those that in(i) admits, and how many are larger: eight bits a turn, from the
// top, until at most 32 keys are left, which every warp ranks (three turns for 8192
// keys took 5.8 us, a turn and the ranking 3.4).
template <int NT, class In, class Key>
__device__ uint32_t nth_largest(int bits, int lo, int hi, int want, const In& in, const Key& key, int* larger, int* hist) {
  uint32_t prefix = 0, mask = 0;
  int above = 0;
  for (int shift = bits - 8; shift >= 0; shift -= 8) {
    for (int i = static_cast<int>(threadIdx.x); i < 256; i += NT) hist[i] = 0;
    __syncthreads();
    for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += NT) {
      if (!in(i)) continue;
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(hist + static_cast<int>((k >> shift) & 255), 1);
    }
    __syncthreads();
    // every warp finds the digit by itself: lane l has digits 255 - 8 l ... 248 - 8 l
    const int lane = static_cast<int>(threadIdx.x) & 31;
    int c[8], sum = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) sum += c[u] = hist[255 - 8 * lane - u];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    int before = upto - sum;
    const int left = want - above;
    int digit = -1, more = 0, same = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (digit < 0 && before < left && before + c[u] >= left) {
        digit = 255 - 8 * lane - u;
        more = before;
        same = c[u];
      }
      before += c[u];
    }
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, digit >= 0);
    const int from = who ? __ffs(who) - 1 : 0;           // (who is 0 only where fewer than `want` are in)
    digit = max(0, __shfl_sync(0xFFFFFFFFu, digit, from));
    above += __shfl_sync(0xFFFFFFFFu, more, from);
    prefix |= static_cast<uint32_t>(digit) << shift;
    mask |= 255u << shift;
    same = __shfl_sync(0xFFFFFFFFu, same, from);
    __syncthreads();
    if (shift == 0 || same == 0 || same > 32) continue;
    uint32_t* list = reinterpret_cast<uint32_t*>(hist);
    if (threadIdx.x == 0) hist[255] = 0;
    __syncthreads();
    for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += NT) {
      if (!in(i)) continue;
      const uint32_t k = key(i);
      if ((k & mask) == prefix) list[atomicAdd(hist + 255, 1)] = k;
    }
    __syncthreads();
    const uint32_t mine = lane < same ? list[lane] : 0;
    int larger_ones = 0, equal = 0;
    for (int i = 0; i < same; ++i) {
      const uint32_t k = __shfl_sync(0xFFFFFFFFu, mine, i);
      larger_ones += k > mine;
      equal += k == mine;
    }
    const int place = want - above;
    const uint32_t is = __ballot_sync(0xFFFFFFFFu, lane < same && larger_ones < place && place <= larger_ones + equal);
    const int at = __ffs(is) - 1;
    above += __shfl_sync(0xFFFFFFFFu, larger_ones, at);
    prefix = __shfl_sync(0xFFFFFFFFu, mine, at);
    __syncthreads();
    break;
  }
  *larger = above;
  return prefix;
}

constexpr uint32_t kNoScore = 0xFFFFFFFFu;               // (a NaN that no sum gives)

// A CTA a row and K/V head.
template <int D, int NT>
__global__ void __launch_bounds__(NT) select_pick_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];                     // [M], then a bit for each slot taken
  __shared__ __align__(16) int hist[256];
  __shared__ int sums[NT / 32];
  __shared__ float fsums[2][NT / 32], range[2][NT / 32];
  __shared__ FixedSum qsum[D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int r = static_cast<int>(blockIdx.x), h = static_cast<int>(blockIdx.y);
  const int t = p.t0 + r;
  // what does not need the scores comes before the wait for them: the sum of A =
  // sum_h |q_h|, the table
  const __nv_bfloat16* q_row = p.q + t * p.q_stride + static_cast<long long>(h) * p.G * D;
  float a1 = 0.f, mn = 0.f;
  for (int e = tid; e < D; e += NT) {
#pragma unroll 4
    for (int g = 0; g < p.G; ++g) a1 += fabsf(__bfloat162float(q_row[static_cast<long long>(g) * D + e]));
  }
  // offsets that do not ascend (a share of them a row; no index depends on their order)
  if (h == 0)
    for (long long s = static_cast<long long>(r) * NT + tid; s < p.S; s += static_cast<long long>(p.rows) * NT)
      if (__ldg(p.cu + s) > __ldg(p.cu + s + 1)) record_error(p.err, ATTN_ERR_BAD_PAGES);
  const SelectRow row = select_row(p, t, lane);
  int* out = p.pages + (static_cast<size_t>(t) * p.Hkv + h) * p.R;
  if (row.n == 0) {                                      // nobody's row (-1), or one that sees nothing
    for (int i = tid; i < p.R; i += NT) out[i] = -1;
    if (tid == 0 && h == 0) {
      p.out_lens[t] = row.s < 0 ? -1 : 0;
      if (row.s >= 0) record_error(p.err, ATTN_ERR_BAD_PAGES);        // fewer tokens than new ones
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // no launch ends before the scores' does
    return;
  }
  if (tid == 0 && h == 0) {
    const int len = __ldg(p.lens + row.s);
    if (len < 0 || len > min(static_cast<long long>(p.M) << p.page_log2, static_cast<long long>(kMaxTokens)))
      record_error(p.err, ATTN_ERR_BAD_PAGES);
  }
  const int* tab = p.table + static_cast<size_t>(row.s) * p.M;
  const int begin = min(p.first, row.held), end = scored_end(p, row);
  const size_t at = static_cast<size_t>(r) * p.Hkv + h;
  float* score = p.score + at * p.M;
  uint32_t* taken = keys + p.M;
  const int words = (row.held + 31) / 32;
  // a warp a word: what is taken anyway; the candidates are marked (1: a page, 0: none)
  constexpr int kAhead = 4;                              // loads in flight
  int mine = 0;
  for (int w0 = warp; w0 < words; w0 += kAhead * (NT / 32)) {
    int pg[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int m = 32 * (w0 + u * (NT / 32)) + lane;
      pg[u] = m < row.held ? __ldg(tab + m) : -1;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int w = w0 + u * (NT / 32), m = 32 * w + lane;
      if (w >= words) break;
      const bool is = pg[u] >= 0 && pg[u] < p.P, scored = m >= begin && m < end;
      if (!is && pg[u] != -1 && !scored) record_error(p.err, ATTN_ERR_BAD_PAGES);
      const uint32_t bits = __ballot_sync(0xFFFFFFFFu, is && !scored);
      if (lane == 0) taken[w] = bits;
      if (scored) keys[m] = is ? 1u : 0u;
      mine += is && scored;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");      // the scores are there
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
  if (lane == 0) sums[warp] = mine;
  for (int i = tid; i < p.parts; i += NT) mn = larger_or_nan(mn, p.norm[at * p.parts + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a1 += __shfl_xor_sync(0xFFFFFFFFu, a1, o);
    mn = larger_or_nan(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
  }
  if (lane == 0) {
    fsums[0][warp] = a1;
    fsums[1][warp] = mn;
  }
  __syncthreads();
  int nc = 0;
  a1 = mn = 0.f;
  for (int w = 0; w < NT / 32; ++w) {
    nc += sums[w];
    a1 += fsums[0][w];
    mn = larger_or_nan(mn, fsums[1][w]);
  }
  const bool choose = nc > p.top && p.top > 0;
  // the candidates' scores and their range (a NaN spreads into it)
  float lo = __int_as_float(0x7f800000), hi = -lo;
  bool odd = false;
  if (choose)
    for (int m0 = begin + tid; m0 < end; m0 += kAhead * NT) {
      float x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) x[u] = m0 + u * NT < end ? score[m0 + u * NT] : 0.f;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int m = m0 + u * NT;
        if (m >= end) break;
        if (keys[m] == 0u) {
          keys[m] = kNoScore;
          continue;
        }
        odd = odd || x[u] != x[u];
        lo = fminf(lo, x[u]);
        hi = fmaxf(hi, x[u]);
        keys[m] = __float_as_uint(x[u]);
      }
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
  }
  if (lane == 0) {
    range[0][warp] = lo;
    range[1][warp] = hi;
  }
  odd = __syncthreads_or(odd);
  for (int w = 0; w < NT / 32; ++w) {
    lo = fminf(lo, range[0][w]);
    hi = fmaxf(hi, range[1][w]);
  }
  // Keys of 24 bits, their steps alike over the range: digits that spread, where
  // the scores' own bits would crowd into a few binades.  A score's key is off by
  // less than 3 of its steps (the subtraction's, the product's and the cut's), so
  // with 2 e in steps, and 6, on either side a page's place is certain.  (1 % and
  // the smallest normal number cover the bound's own roundings.)
  const float e2 = 2.02f * static_cast<float>(p.G + p.rounds + 2) * 5.9604645e-8f * a1 * mn + 1.17549435e-38f;
  const float steps = 16777215.f / fmaxf(hi - lo, 1.17549435e-38f);
  const float wide = e2 * steps * 1.01f + 7.f;
  // an infinity or NaN anywhere, or a bound as wide as the range: nothing is certain
  const bool clear = choose && !odd && isfinite(hi) && isfinite(lo) && isfinite(steps) && wide < 16777216.f;
  const int band = clear ? static_cast<int>(wide) : 0;
  if (choose)
    for (int m = begin + tid; m < end; m += NT) {
      const uint32_t x = keys[m];
      keys[m] = x == kNoScore ? 0u
                : clear       ? 1u + min(static_cast<uint32_t>((__uint_as_float(x) - lo) * steps), 16777215u)
                              : 1u;
    }
  __syncthreads();
  auto held_page = [&](int m) { return keys[m] != 0u; };
  // What follows is for pages that are scored again.  A column's sum of queries is less
  // than 2^q_exp = 2^Q, a mean than 2^(mean_field - 126) = 2^M, a score then than 2^125
  // units of 2^(Q + M - 118).
  int q_exp = 0, mean_field = 0;
  auto sum_again = [&]() {
    float qm = a1, mm = mn;
    if (!isfinite(a1) || !isfinite(mn)) {                // the largest ones that are finite
      qm = mm = 0.f;
      for (int i = tid; i < p.G * D; i += NT) {
        const float x = fabsf(__bfloat162float(q_row[i]));
        if (isfinite(x)) qm = fmaxf(qm, x);
      }
      for (int m0 = begin + warp; m0 < end; m0 += NT / 32) {
        if (!held_page(m0)) continue;
        const float* src = p.means + (static_cast<size_t>(__ldg(tab + m0)) * p.Hkv + h) * D;
        for (int e = lane; e < D; e += 32) {
          const float x = fabsf(__ldg(src + e));
          if (isfinite(x)) mm = fmaxf(mm, x);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        qm = fmaxf(qm, __shfl_xor_sync(0xFFFFFFFFu, qm, o));
        mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
      }
      if (lane == 0) {
        fsums[0][warp] = qm;
        fsums[1][warp] = mm;
      }
      __syncthreads();
      for (int w = 0; w < NT / 32; ++w) {
        qm = fmaxf(qm, fsums[0][w]);
        mm = fmaxf(mm, fsums[1][w]);
      }
    }
    // (twice the sum of all magnitudes, for its own rounding; or G times the largest)
    q_exp = static_cast<int>(__float_as_uint(qm) >> 23) - 125 + (qm == a1 ? 0 : 32 - __clz(p.G));
    mean_field = max(1, static_cast<int>(__float_as_uint(mm) >> 23));
    for (int e = tid; e < D; e += NT) {
      __int128 sum = 0;
      float odd = 0.f;
      for (int g = 0; g < p.G; ++g) {
        const float x = __bfloat162float(q_row[static_cast<long long>(g) * D + e]);
        const uint32_t bits = __float_as_uint(x);
        const int field = static_cast<int>(bits >> 23 & 255u);
        if (field == 255) {
          odd += x;
          continue;
        }
        // 8 bits times 2^(field - 134)
        const long long digits = static_cast<long long>((bits >> 16 & 127u) | (field != 0 ? 128u : 0u));
        const int shift = max(field, 1) - 40 - q_exp;
        const __int128 y = shift >= 0 ? static_cast<__int128>(digits) << shift : digits >> min(-shift, 63);
        sum += bits >> 31 ? -y : y;
      }
      qsum[e] = FixedSum{static_cast<unsigned long long>(sum), static_cast<int>(sum >> 64), odd};
    }
  };
  // slot m's score in those units, past 2^126 of them, by a warp; -inf is 1, a NaN 0
  auto score_again = [&](int m) {
    const float* src = p.means + (static_cast<size_t>(__ldg(tab + m)) * p.Hkv + h) * D;
    __int128 sum = 0;
    float odd = 0.f;
    for (int e = lane; e < D; e += 32) {
      const float mean = __ldg(src + e);
      const uint32_t bits = __float_as_uint(mean);
      const int field = static_cast<int>(bits >> 23 & 255u);
      const FixedSum q = qsum[e];
      const __int128 x = q.value();
      if (q.odd != 0.f) {
        odd += q.odd * mean;
      } else if (field == 255) {
        odd += mean * (x > 0 ? 1.f : x < 0 ? -1.f : 0.f);
      } else {
        // 24 bits times 2^(field - 150)
        const int digits = static_cast<int>((bits & 0x7FFFFFu) | (field != 0 ? 0x800000u : 0u));
        sum += x * (bits >> 31 ? -digits : digits) >> min(mean_field - max(field, 1), 127);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long lo = __shfl_xor_sync(0xFFFFFFFFu, static_cast<unsigned long long>(sum), o);
      const long long hi = __shfl_xor_sync(0xFFFFFFFFu, static_cast<long long>(sum >> 64), o);
      sum += static_cast<__int128>(hi) << 64 | lo;
      odd += __shfl_xor_sync(0xFFFFFFFFu, odd, o);
    }
    const unsigned __int128 key = static_cast<unsigned __int128>(sum) + (static_cast<unsigned __int128>(1) << 126);
    return odd == 0.f ? key : odd > 0.f ? ~static_cast<unsigned __int128>(0) : static_cast<unsigned __int128>(odd < 0.f);
  };
  auto take = [&](int m) { atomicOr(taken + (m >> 5), 1u << (m & 31)); };
  if (nc <= p.top) {
    for (int m = begin + tid; m < end; m += NT)
      if (held_page(m)) take(m);
  } else if (p.top > 0) {
    int larger;
    const int kth = clear ? static_cast<int>(nth_largest<NT>(
                                24, begin, end, p.top, held_page, [&](int m) { return keys[m] - 1u; }, &larger, hist)) + 1
                          : 1;
    auto is_sure = [&](int m) { return clear && static_cast<int>(keys[m]) > kth + band; };
    auto is_open = [&](int m) { return held_page(m) && !is_sure(m) && static_cast<int>(keys[m]) >= kth - band; };
    int sure = 0, open = 0;
    for (int m = begin + tid; m < end; m += NT) {
      sure += is_sure(m);
      open += is_open(m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sure += __shfl_xor_sync(0xFFFFFFFFu, sure, o);
      open += __shfl_xor_sync(0xFFFFFFFFu, open, o);
    }
    if (lane == 0) {
      sums[warp] = sure;
      hist[warp] = open;
    }
    __syncthreads();
    sure = open = 0;
    for (int w = 0; w < NT / 32; ++w) {
      sure += sums[w];
      open += hist[w];
    }
    __syncthreads();
    const int want = p.top - sure;                       // of the open ones
    for (int m = begin + tid; m < end; m += NT)
      if (is_sure(m)) take(m);
    if (open <= want) {
      for (int m = begin + tid; m < end; m += NT)
        if (is_open(m)) take(m);
    } else if (want > 0 && open <= 32) {
      // scored again, a warp an open page, and ranked by one warp
      if (tid == 0) sums[0] = 0;
      sum_again();
      __syncthreads();
      for (int m = begin + tid; m < end; m += NT)
        if (is_open(m)) hist[atomicAdd(sums, 1)] = m;
      __syncthreads();
      ulonglong2* again = reinterpret_cast<ulonglong2*>(hist + 32);
      for (int i = warp; i < open; i += NT / 32) {
        const unsigned __int128 k = score_again(hist[i]);
        if (lane == 0)
          again[i] = make_ulonglong2(static_cast<unsigned long long>(k), static_cast<unsigned long long>(k >> 64));
      }
      __syncthreads();
      if (warp == 0) {
        const int m = lane < open ? hist[lane] : 0;
        const ulonglong2 k = lane < open ? again[lane] : make_ulonglong2(0ull, 0ull);
        int better = 0;
        for (int i = 0; i < open; ++i) {
          const unsigned long long lo = __shfl_sync(0xFFFFFFFFu, k.x, i), hi = __shfl_sync(0xFFFFFFFFu, k.y, i);
          const int m2 = __shfl_sync(0xFFFFFFFFu, m, i);
          better += hi > k.y || (hi == k.y && (lo > k.x || (lo == k.x && m2 < m)));
        }
        if (lane < open && better < want) take(m);
      }
    } else if (want > 0) {
      // Scored again, a warp an open page, 32 bits of the number at a time (where the
      // score was): what is larger than the want-th word is taken, what is smaller
      // is no longer open, and so on with those that equal it.
      sum_again();
      int left = want, same = open;
      uint32_t* word = reinterpret_cast<uint32_t*>(score);
      ulonglong2* firsts = reinterpret_cast<ulonglong2*>(hist);
      for (int part = 0; part < 4 && same > left; ++part) {
        __syncthreads();
        unsigned __int128 first = 0;
        int met = 0;                                     // 1: a page, 3: and one of another score
        for (int m0 = begin + warp * 32; m0 < end; m0 += NT) {
          uint32_t todo = __ballot_sync(0xFFFFFFFFu, m0 + lane < end && is_open(m0 + lane));
          for (; todo != 0u; todo &= todo - 1) {
            const int m = m0 + __ffs(todo) - 1;
            const unsigned __int128 k = score_again(m);
            if (lane == 0) word[m] = static_cast<uint32_t>(k >> (96 - 32 * part));
            if (met == 0) first = k;
            met |= k == first ? 1 : 3;
          }
        }
        if (lane == 0) {
          sums[warp] = met;
          firsts[warp] = make_ulonglong2(static_cast<unsigned long long>(first),
                                         static_cast<unsigned long long>(first >> 64));
        }
        __syncthreads();
        bool alike = true;                               // all of them: nothing more to tell apart
        int one = -1;
        for (int w = 0; w < NT / 32; ++w) {
          if (sums[w] == 0) continue;
          if (one < 0) one = w;
          alike = alike && sums[w] == 1 && firsts[w].x == firsts[one].x && firsts[w].y == firsts[one].y;
        }
        __syncthreads();
        if (alike) break;
        int more;
        const uint32_t kw = nth_largest<NT>(32, begin, end, left, is_open, [&](int m) { return word[m]; },
                                                      &more, hist);
        int count = 0;
        for (int m = begin + tid; m < end; m += NT) {
          if (!is_open(m)) continue;
          const uint32_t k = word[m];
          if (k > kw) take(m);
          if (k != kw) keys[m] = 0u;
          count += k == kw;
        }
        left -= more;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) count += __shfl_xor_sync(0xFFFFFFFFu, count, o);
        if (lane == 0) sums[warp] = count;
        __syncthreads();
        same = 0;
        for (int w = 0; w < NT / 32; ++w) same += sums[w];
        __syncthreads();
      }
      // of those that are equal the first ones
      for (int m0 = begin; m0 < end && left > 0; m0 += NT) {
        const int m = m0 + tid;
        const bool is = m < end && is_open(m);
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, is);
        if (lane == 0) sums[warp] = __popc(votes);
        __syncthreads();
        int before = __popc(votes & ((1u << lane) - 1u)), total = 0;
        for (int w = 0; w < NT / 32; ++w) {
          if (w < warp) before += sums[w];
          total += sums[w];
        }
        if (is && before < left) take(m);
        left -= total;
        __syncthreads();
      }
    }
  }
  __syncthreads();
  // the list, in ascending order: where each word's pages begin (in keys' place), then
  // a warp a word, so that the table's entries come together
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += NT) {
    const int w = w0 + tid;
    const int count = w < words ? __popc(taken[w]) : 0;
    int x = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int place = base + x - count;
    for (int v = 0; v < warp; ++v) place += sums[v];
    if (w < words) keys[w] = static_cast<uint32_t>(place);
    for (int v = 0; v < NT / 32; ++v) base += sums[v];
    __syncthreads();
  }
#pragma unroll 4
  for (int w = warp; w < words; w += NT / 32) {
    const uint32_t bits = taken[w];
    const int place = static_cast<int>(keys[w]) + __popc(bits & ((1u << lane) - 1u));
    if ((bits >> lane & 1u) && place < p.R) out[place] = __ldg(tab + 32 * w + lane);
  }
  for (int i = base + tid; i < p.R; i += NT) out[i] = -1;
  if (tid == 0 && h == 0) {
    // every page listed is whole, but for the row's own
    const int last = __ldg(tab + row.held - 1);
    const bool own = last >= 0 && last < p.P;
    if (!own) record_error(p.err, ATTN_ERR_BAD_PAGES);
    p.out_lens[t] = own ? ((base - 1) << p.page_log2) + row.n - ((row.held - 1) << p.page_log2)
                        : base << p.page_log2;
  }
}

// Rows scored together: those of chunks, which share their sequence's means.  (A tile
// takes its rows' sequences one after the other.  Selections in us, row by row | tiles;
// S sequences with `new` rows each, 4 K/V heads, d=128:
//      pages         128              512              1024
//      S = 1,  8     7.7 | 13.5       13.0 | 17.8      16.6 | 18.6
//      S = 1,  32    10.7 | 17.8      17.2 | 19.4      23.6 | 20.9
//      S = 8,  5     12.2 | 60.4      19.9 | 62.1      27.3 | 64.0
//      S = 8,  16    17.1 | 28.8      30.4 | 30.9      47.6 | 33.0
//      S = 8,  32    20.7 | 19.6      46.3 | 22.7      78.9 | 29.1
//      S = 64, 5     25.8 | 76.3      58.4 | 100.3     125.9 | 169.7
//      S = 64, 8     33.4 | 52.4      84.8 | 72.0      167.8 | 138.3
//      S = 64, 16    60.7 | 48.8      159.6 | 95.4     293.4 | 172.8)
constexpr int kTileRowsASeq = 16;
int score_rows(int T, int S) { return T >= static_cast<long long>(kTileRowsASeq) * S ? kTileRows : 1; }
// Rows of a launch: at most 2^26 scores (256 MB), or those of one row of very many
// heads, and a grid's 65535.
long long select_chunk(int T, int Hkv, int M) {
  const long long rows = std::max<long long>(1, (1ll << 26) / (static_cast<long long>(Hkv) * M));
  return std::min<long long>(T, std::min<long long>(rows < 8 ? rows : rows / 8 * 8, 65528));
}
int score_parts(long long rows, int RT, int Hkv, int M) {
  const long long tiles = (rows + RT - 1) / RT * Hkv;
  const int pages = RT == 1 ? kScoreWarps * kScorePages : kTilePages;
  const long long most = (M + pages - 1) / pages;
  return static_cast<int>(std::max<long long>(1, std::min<long long>(most, 152ll * 16 / tiles)));
}

bool select_sizes(int T, int S, int H, int Hkv, int d, int M, int page, int top, int local, int first) {
  if (T < 1 || S < 1 || M < 1 || top < 0 || local < 1 || first < 0) return false;
  if (!valid_kv_heads(H, Hkv) || (d != 64 && d != 128) || S > kMaxSeqs || M > kMaxSelectPages) return false;
  if (!valid_page_size(page)) return false;
  if (H > 65535) return false;
  const long long R = static_cast<long long>(top) + local + first;
  return R <= 0x7FFFFFFFll && static_cast<long long>(T) * Hkv <= 0x7FFFFFFFll / std::max<long long>(R, 1);
}
size_t select_workspace(int T, int S, int Hkv, int M) {
  const long long rows = select_chunk(T, Hkv, M);
  const size_t slots = static_cast<size_t>(rows) * Hkv;
  const int parts = score_parts(rows, score_rows(T, S), Hkv, M);
  return up256(slots * M * 4) + slots * parts * 4;
}

// Threads of a row and K/V head's CTA: 128, or 1024 where the table's rows are long and
// either the CTAs are one a multiprocessor at most or the keys of 128 threads' CTAs
// would fill its shared memory.  (Selections in us, 128 | 1024; `ctas` rows times heads:
//      columns       1024            2048            4096            8192            16384
//      ctas = 4      11.1 | 12.5     16.0 | 14.4     24.0 | 16.0     42.3 | 21.7     72.1 | 28.0
//      ctas = 32     19.7 | 21.4     22.2 | 22.0     28.2 | 23.8     52.5 | 29.4     86.7 | 45.0
//      ctas = 152    -               25.0 | 25.4     35.2 | 30.5     64.5 | 45.1     109 | 69
//      ctas = 200    -               25.1 | 34.3     36.1 | 41.3     68.4 | 59.0     115 | 90
//      ctas = 512    23.3 | 51.7     33.1 | 58.8     50.8 | 78.7     94.5 | 110      217 | 175
//      ctas = 2000   52.2 | 163      83.2 | 196      142 | 261       275 | 377       650 | 598)
constexpr int kLongRow = 2048;
constexpr int kLongRowOfMany = 8192;
constexpr int kFewPicks = 152;
template <int D>
cudaError_t launch_select_pages(SelectParams p, int RT, cudaStream_t st) {
  const int smem = p.M * 4 + (p.M + 31) / 32 * 4;
  constexpr int kMaxDev = 64;
  static bool configured[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(select_pick_kernel<D, 1024>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxSelectPages * 4 + kMaxSelectPages / 8);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(select_score_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ScoreTile<D>::kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int chunk = static_cast<int>(select_chunk(p.T, p.Hkv, p.M));
  for (int t0 = 0; t0 < p.T; t0 += chunk) {
    p.t0 = t0;
    p.rows = std::min(chunk, p.T - t0);
    const dim3 grid(p.parts, (p.rows + RT - 1) / RT, p.Hkv);
    if (RT == 1) select_score_kernel<D><<<grid, kScoreWarps * 32, 0, st>>>(p);
    else select_score_tile_kernel<D><<<grid, kTileThreads, ScoreTile<D>::kSmem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const bool wide = p.M > (static_cast<long long>(p.rows) * p.Hkv <= kFewPicks ? kLongRow : kLongRowOfMany);
    // the pick is set up while the scores are made, and waits for them itself
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.rows, p.Hkv);
    cfg.blockDim = dim3(wide ? 1024 : 128);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, wide ? select_pick_kernel<D, 1024> : select_pick_kernel<D, 128>, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace bss

using namespace bss;

extern "C" attn_status_t attn_kv_pool(const void* k_cache, int64_t k_page_stride, int kv_dtype,
                                      const float* k_scale, float* k_means, const int32_t* page_table,
                                      const int32_t* start, const int32_t* seq_lens, int S, int max_pages,
                                      int n_pages, int H_kv, int d, int page_size, void* stream) {
  if (!k_cache || !aligned16(k_cache) || !k_means || !aligned16(k_means)) return ATTN_ERR_INVALID_ARG;
  if (S < 1 || max_pages < 1 || n_pages < 1 || H_kv < 1 || H_kv > 65536) return ATTN_ERR_INVALID_ARG;
  if (S > kMaxSeqs || (d != 64 && d != 128) || !valid_page_size(page_size)) return ATTN_ERR_UNSUPPORTED;
  if (kv_dtype != ATTN_KV_BF16 && kv_dtype != ATTN_KV_E4M3) return ATTN_ERR_UNSUPPORTED;
  const bool fp8 = kv_dtype == ATTN_KV_E4M3;
  if (fp8 != (k_scale != nullptr) || !aligned4(k_scale)) return ATTN_ERR_INVALID_ARG;
  const void* ptrs4[] = {page_table, start, seq_lens};
  for (const void* ptr : ptrs4)
    if (!ptr || !aligned4(ptr)) return ATTN_ERR_INVALID_ARG;
  if (k_page_stride < static_cast<int64_t>(H_kv) * page_size * d || k_page_stride % (fp8 ? 16 : 8))
    return ATTN_ERR_INVALID_ARG;
  PoolParams p{};
  attn_status_t s = status_word(&p.err);
  if (s != ATTN_OK) return s;
  p.k = static_cast<const uint8_t*>(k_cache);
  p.k_stride = static_cast<size_t>(k_page_stride) * (fp8 ? 1 : 2);
  p.k_scale = k_scale;
  p.means = k_means;
  p.table = page_table;
  p.start = start;
  p.lens = seq_lens;
  p.S = S;
  p.M = max_pages;
  p.P = n_pages;
  p.Hkv = H_kv;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  // loads of 32 lanes a page: a warp for 8 of them
  const int loads = page_size * d * (fp8 ? 1 : 2) / 512;
  p.warps = 1;
  while (p.warps < kPoolWarps && loads > p.warps * kPoolBatch) p.warps *= 2;
  // the pages that became full are known on the device alone: CTAs enough for all
  // of a few sequences, and one a sequence where there are many (each takes its
  // pages in turns; four a sequence, of which three found nothing, took 25 us
  // instead of 10 for 256 sequences with two full pages each)
  const int gy = std::min(S, 65535);
  const long long rounds = (static_cast<long long>(max_pages) * p.warps + kPoolWarps - 1) / kPoolWarps * H_kv;
  const dim3 grid(static_cast<unsigned>(std::max<long long>(1, std::min<long long>(rounds, 152 * 4 / gy))), gy);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 64) {
    if (fp8) kv_pool_kernel<64, true><<<grid, kPoolWarps * 32, 0, st>>>(p);
    else kv_pool_kernel<64, false><<<grid, kPoolWarps * 32, 0, st>>>(p);
  } else {
    if (fp8) kv_pool_kernel<128, true><<<grid, kPoolWarps * 32, 0, st>>>(p);
    else kv_pool_kernel<128, false><<<grid, kPoolWarps * 32, 0, st>>>(p);
  }
  return cuda_status("attn_kv_pool launch", cudaGetLastError());
}

extern "C" size_t attn_select_pages_workspace_bytes(int T, int S, int H, int H_kv, int d, int max_pages,
                                                    int page_size, int top_r, int local_pages,
                                                    int first_pages) {
  if (!select_sizes(T, S, H, H_kv, d, max_pages, page_size, top_r, local_pages, first_pages)) return 0;
  return select_workspace(T, S, H_kv, max_pages);
}

extern "C" attn_status_t attn_select_pages(const void* q, int64_t q_stride, const float* k_means,
                                           const int32_t* page_table, const int32_t* seq_lens,
                                           const int32_t* cu_q, int32_t* pages, int32_t* lens,
                                           void* workspace, size_t workspace_bytes, int T, int S, int H,
                                           int H_kv, int d, int max_pages, int n_pages, int page_size,
                                           int top_r, int local_pages, int first_pages, void* stream) {
  if (T < 0 || S < 1 || H < 1 || !valid_kv_heads(H, H_kv)) return ATTN_ERR_INVALID_ARG;
  if (max_pages < 1 || n_pages < 1 || top_r < 0 || local_pages < 1 || first_pages < 0)
    return ATTN_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !valid_page_size(page_size) || S > kMaxSeqs || max_pages > kMaxSelectPages)
    return ATTN_ERR_UNSUPPORTED;
  if (T == 0) return ATTN_OK;
  if (!select_sizes(T, S, H, H_kv, d, max_pages, page_size, top_r, local_pages, first_pages))
    return ATTN_ERR_UNSUPPORTED;
  const void* ptrs16[] = {q, k_means, workspace};
  for (const void* ptr : ptrs16)
    if (!ptr || !aligned16(ptr)) return ATTN_ERR_INVALID_ARG;
  const void* ptrs4[] = {page_table, seq_lens, cu_q, pages, lens};
  for (const void* ptr : ptrs4)
    if (!ptr || !aligned4(ptr)) return ATTN_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(H) * d || q_stride % 8) return ATTN_ERR_INVALID_ARG;
  if (workspace_bytes < select_workspace(T, S, H_kv, max_pages)) return ATTN_ERR_WORKSPACE;
  SelectParams p{};
  attn_status_t s = status_word(&p.err);
  if (s != ATTN_OK) return s;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.means = k_means;
  p.table = page_table;
  p.lens = seq_lens;
  p.cu = cu_q;
  p.T = T;
  p.S = S;
  p.H = H;
  p.Hkv = H_kv;
  p.G = H / H_kv;
  p.M = max_pages;
  p.P = n_pages;
  while ((1 << p.page_log2) < page_size) ++p.page_log2;
  p.top = top_r;
  p.local = local_pages;
  p.first = first_pages;
  p.R = top_r + local_pages + first_pages;
  p.pages = pages;
  p.out_lens = lens;
  const long long rows = select_chunk(T, H_kv, max_pages);
  const int RT = score_rows(T, S);
  p.parts = score_parts(rows, RT, H_kv, max_pages);
  p.rounds = RT == 1 ? d / 32 + 5 : d;
  const size_t slots = static_cast<size_t>(rows) * H_kv;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.score = reinterpret_cast<float*>(ws);
  p.norm = reinterpret_cast<float*>(ws + up256(slots * max_pages * 4));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = d == 64 ? launch_select_pages<64>(p, RT, st) : launch_select_pages<128>(p, RT, st);
  return cuda_status("attn_select_pages launch", e);
}
