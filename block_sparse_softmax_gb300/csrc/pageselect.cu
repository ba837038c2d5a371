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
//   * means: each element is divided by the page size first (a power of two:
//     exact), then summed as an unevaluated pair of fp32 numbers by Knuth's
//     two-sum, which leaves one rounding, the mean's own to fp32;
//   * scores: in fp32 first, each off by at most
//         e = (G + 16) 2^-24 sum_i A_i max_mi |mean_mi|,   A = sum_h |q_h|
//     (G roundings of the group's sum at most, d / 32 of a lane's chain and 5 of
//     the lanes' tree, of products whose absolute values add up to at most that
//     sum).  The top_r-th largest of numbers that are off by e is off by e, so
//     what lies more than 2 e above it is taken and more than 2 e below is not;
//     only what lies between (as a rule, that one page) is scored again, in 64
//     bits.
#include <cuda_fp16.h>

#include <algorithm>

#include "host.cuh"

namespace bss {
namespace {

constexpr int kMaxSeqs = 65536;
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
  int* err;
};

// x added to the pair hi + lo, exactly but for lo's rounding.
__device__ __forceinline__ void two_sum(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x);
  const float b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}

__device__ __forceinline__ float2 e4m3x2_f32x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(y) : "r"(x));
  return __half22float2(*reinterpret_cast<const __half2*>(&y));
}

// A warp a (page, head): 16 bytes a lane and load, so that 32 * 16 / (bytes of a
// row) rows arrive at once.
constexpr int kPoolWarps = 8;
constexpr int kPoolBatch = 8;                 // loads in flight
template <int D, bool FP8>
__global__ void __launch_bounds__(kPoolWarps * 32) kv_pool_kernel(const PoolParams p) {
  constexpr int kEl = FP8 ? 16 : 8;           // elements of 16 bytes
  constexpr int kLanes = D / kEl;             // lanes of a row
  constexpr int kRows = 32 / kLanes;          // rows of a load
  const int s = static_cast<int>(blockIdx.y);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int page = 1 << p.page_log2;
  for (int sq = s; sq < p.S; sq += static_cast<int>(gridDim.y)) {
    const int a = __ldg(p.start + sq), n = __ldg(p.lens + sq);
    if (a < 0) continue;                      // nothing was reserved
    const long long most = static_cast<long long>(p.M) << p.page_log2;
    if (n < 0 || n > most) {
      if (threadIdx.x == 0 && blockIdx.x == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
      continue;
    }
    const int m0 = a >> p.page_log2, m1 = n >> p.page_log2;
    const long long items = static_cast<long long>(max(0, m1 - m0)) * p.Hkv;
    for (long long x = static_cast<long long>(blockIdx.x) * kPoolWarps + (threadIdx.x >> 5); x < items;
         x += static_cast<long long>(gridDim.x) * kPoolWarps) {
      const int m = m0 + static_cast<int>(x / p.Hkv);
      const int h = static_cast<int>(x % p.Hkv);
      const int pg = __ldg(p.table + static_cast<size_t>(sq) * p.M + m);
      if (pg < 0 || pg >= p.P) {              // -1: given back already
        if (pg != -1 && lane == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
        continue;
      }
      const uint4* src = reinterpret_cast<const uint4*>(
          p.k + pg * p.k_stride + ((static_cast<size_t>(h) << p.page_log2) * D) * (FP8 ? 1 : 2)) + lane;
      const float part = 1.f / static_cast<float>(page);
      float hi[kEl], lo[kEl];
#pragma unroll
      for (int e = 0; e < kEl; ++e) hi[e] = lo[e] = 0.f;
      const int loads = page / kRows;         // page >= 16 >= kRows
      for (int i0 = 0; i0 < loads; i0 += kPoolBatch) {
        uint4 v[kPoolBatch];
#pragma unroll
        for (int u = 0; u < kPoolBatch; ++u)
          v[u] = i0 + u < loads ? src[(i0 + u) * 32] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < kPoolBatch; ++u) {
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (FP8) {
              const float2 c0 = e4m3x2_f32x2(w[e]), c1 = e4m3x2_f32x2(w[e] >> 16);
              two_sum(hi[4 * e], lo[4 * e], c0.x * part);
              two_sum(hi[4 * e + 1], lo[4 * e + 1], c0.y * part);
              two_sum(hi[4 * e + 2], lo[4 * e + 2], c1.x * part);
              two_sum(hi[4 * e + 3], lo[4 * e + 3], c1.y * part);
            } else {
              two_sum(hi[2 * e], lo[2 * e], bf16lo(w[e]) * part);
              two_sum(hi[2 * e + 1], lo[2 * e + 1], bf16hi(w[e]) * part);
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
          two_sum(hi[e], lo[e], oh);
          lo[e] = __fadd_rn(lo[e], ol);
        }
      }
      if (lane < kLanes) {
        const double f = FP8 ? static_cast<double>(__ldg(p.k_scale + h)) : 1.0;
        float* dst = p.means + (static_cast<size_t>(pg) * p.Hkv + h) * D + lane * kEl;
#pragma unroll
        for (int e = 0; e < kEl; e += 4) {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float hh = hi[e + i];       // an infinity's or NaN's lo is a NaN
            const double sum = isfinite(hh) ? static_cast<double>(hh) + static_cast<double>(lo[e + i])
                                            : static_cast<double>(hh);
            y[i] = static_cast<float>(sum * f);
          }
          *reinterpret_cast<float4*>(dst + e) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
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
  float* score;             // [rows][Hkv][M]
  double* exact;            // [rows][Hkv][M], written where needed
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
__device__ __forceinline__ SelectRow select_row(const SelectParams& p, int t) {
  int lo = 0, hi = p.S;
  while (lo < hi) {                           // the last s with cu[s] <= t
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu + mid) <= t) lo = mid;
    else hi = mid - 1;
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

// RT rows (consecutive, scored together where they belong to one sequence) and
// a K/V head: CTA x of `parts` takes every parts-th group of pages.
template <int D, int RT>
__global__ void __launch_bounds__(kScoreWarps * 32) select_score_kernel(const SelectParams p) {
  constexpr int E = D / 32;                   // elements a lane
  __shared__ float qsum[RT][D];
  __shared__ float top[kScoreWarps][RT];
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int h = static_cast<int>(blockIdx.z);
  const int r0 = static_cast<int>(blockIdx.y) * RT;
  const int nr = min(RT, p.rows - r0);
  for (int i = tid; i < RT * D; i += kScoreWarps * 32) {
    const int r = i / D, e = i % D;
    float sum = 0.f;
    if (r < nr) {
      const __nv_bfloat16* q = p.q + (p.t0 + r0 + r) * p.q_stride + static_cast<long long>(h) * p.G * D + e;
      for (int g = 0; g < p.G; ++g) sum += __bfloat162float(q[static_cast<long long>(g) * D]);
    }
    qsum[r][e] = sum;
  }
  __syncthreads();
  float most[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) most[r] = 0.f;
  for (int a = 0; a < nr;) {                  // runs of rows of one sequence
    const SelectRow row = select_row(p, p.t0 + r0 + a);
    int b = a + 1;
    SelectRow last = row;
    while (b < nr) {
      const SelectRow x = select_row(p, p.t0 + r0 + b);
      if (x.s != row.s) break;
      last = x;
      ++b;
    }
    // the run's last row sees the most
    const int end = row.s < 0 ? 0 : scored_end(p, last);
    float q[RT][E];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int e = 0; e < E; ++e) q[r][e] = r >= a && r < b ? qsum[r][lane * E + e] : 0.f;
    const int* tab = p.table + static_cast<size_t>(max(row.s, 0)) * p.M;
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
        if (x >= 0) {
          const float* src = p.means + (static_cast<size_t>(x) * p.Hkv + h) * D + lane * E;
          if constexpr (E == 4) {
            const float4 y = __ldg(reinterpret_cast<const float4*>(src));
            v[u][0] = y.x, v[u][1] = y.y, v[u][2] = y.z, v[u][3] = y.w;
          } else {
            const float2 y = __ldg(reinterpret_cast<const float2*>(src));
            v[u][0] = y.x, v[u][1] = y.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        }
      }
      float norm = 0.f;
#pragma unroll
      for (int u = 0; u < kScorePages; ++u) {
#pragma unroll
        for (int e = 0; e < E; ++e) norm = larger_or_nan(norm, fabsf(v[u][e]));
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        if (r < a || r >= b) continue;
        most[r] = larger_or_nan(most[r], norm);
        float mine = 0.f;
#pragma unroll
        for (int u = 0; u < kScorePages; ++u) {
          float d = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) d = fmaf(q[r][e], v[u][e], d);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
          if (lane == u) mine = d;
        }
        if (lane < kScorePages && m0 + lane < end)
          p.score[(static_cast<size_t>(r0 + r) * p.Hkv + h) * p.M + m0 + lane] = mine;
      }
    }
    a = b;
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most[r] = larger_or_nan(most[r], __shfl_xor_sync(0xFFFFFFFFu, most[r], o));
    if (lane == 0) top[warp][r] = most[r];
  }
  __syncthreads();
  if (tid < nr) {
    float x = 0.f;
    for (int w = 0; w < kScoreWarps; ++w) x = larger_or_nan(x, top[w][tid]);
    p.norm[(static_cast<size_t>(r0 + tid) * p.Hkv + h) * p.parts + blockIdx.x] = x;
  }
}

// ----------------------------------------------------------------------------
// the pick
// ----------------------------------------------------------------------------
// Numbers in an order of whole ones; a NaN comes last, below every other.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);          // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ unsigned long long order_of(double x) {
  if (x != x) return 0ull;
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
  return b >> 63 ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return k == 0u ? __int_as_float(0x7fffffff) : __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

constexpr int kPickThreads = 256;

// The want-th largest (want >= 1) of the keys key(i), i in [lo, hi), of those that
// in(i) admits, and how many are larger: eight bits a turn, from the top.
template <class K, class In, class Key>
__device__ K nth_largest(int lo, int hi, int want, const In& in, const Key& key, int* larger, int* hist) {
  K prefix = 0, mask = 0;
  int above = 0;
  for (int shift = static_cast<int>(sizeof(K)) * 8 - 8; shift >= 0; shift -= 8) {
    for (int i = static_cast<int>(threadIdx.x); i < 256; i += kPickThreads) hist[i] = 0;
    __syncthreads();
    for (int i = lo + static_cast<int>(threadIdx.x); i < hi; i += kPickThreads) {
      if (!in(i)) continue;
      const K k = key(i);
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
    int digit = -1, more = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (digit < 0 && before < left && before + c[u] >= left) {
        digit = 255 - 8 * lane - u;
        more = before;
      }
      before += c[u];
    }
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, digit >= 0);
    const int from = who ? __ffs(who) - 1 : 0;           // (who is 0 only where fewer than `want` are in)
    digit = max(0, __shfl_sync(0xFFFFFFFFu, digit, from));
    above += __shfl_sync(0xFFFFFFFFu, more, from);
    prefix |= static_cast<K>(digit) << shift;
    mask |= static_cast<K>(255) << shift;
    __syncthreads();
  }
  *larger = above;
  return prefix;
}

// A CTA a row and K/V head.
template <int D>
__global__ void __launch_bounds__(kPickThreads) select_pick_kernel(const SelectParams p) {
  extern __shared__ uint32_t keys[];                     // [M], then a bit for each slot taken
  __shared__ int hist[256];
  __shared__ int sums[kPickThreads / 32];
  __shared__ float fsums[2][kPickThreads / 32];
  __shared__ double qd[D];
  const int tid = static_cast<int>(threadIdx.x);
  const int warp = tid >> 5, lane = tid & 31;
  const int r = static_cast<int>(blockIdx.x), h = static_cast<int>(blockIdx.y);
  const int t = p.t0 + r;
  const SelectRow row = select_row(p, t);
  int* out = p.pages + (static_cast<size_t>(t) * p.Hkv + h) * p.R;
  if (row.n == 0) {                                      // nobody's row (-1), or one that sees nothing
    for (int i = tid; i < p.R; i += kPickThreads) out[i] = -1;
    if (tid == 0 && h == 0) {
      p.out_lens[t] = row.s < 0 ? -1 : 0;
      if (row.s >= 0) record_error(p.err, ATTN_ERR_BAD_PAGES);        // fewer tokens than new ones
    }
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
  const float* score = p.score + at * p.M;
  double* exact = p.exact + at * p.M;
  uint32_t* taken = keys + p.M;
  const int words = (row.held + 31) / 32;
  auto held_page = [&](int m) {
    const int pg = __ldg(tab + m);
    return pg >= 0 && pg < p.P;
  };

  // the candidates' keys (0 for those without a page, as for a NaN: told apart by `held_page`)
  int mine = 0;
  for (int m = begin + tid; m < end; m += kPickThreads) {
    const bool is = held_page(m);
    keys[m] = is ? order_of(score[m]) : 0u;
    mine += is;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
  if (lane == 0) sums[warp] = mine;
  // the sum of A = sum_h |q_h| and the largest mean, for the bound
  float a1 = 0.f, mn = 0.f;
  for (int e = tid; e < D; e += kPickThreads) {
    float a = 0.f;
    double x = 0.0;
    const __nv_bfloat16* q = p.q + t * p.q_stride + static_cast<long long>(h) * p.G * D + e;
    for (int g = 0; g < p.G; ++g) {
      const float y = __bfloat162float(q[static_cast<long long>(g) * D]);
      a += fabsf(y);
      x += static_cast<double>(y);
    }
    a1 += a;
    qd[e] = x;
  }
  for (int i = tid; i < p.parts; i += kPickThreads) mn = larger_or_nan(mn, p.norm[at * p.parts + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a1 += __shfl_xor_sync(0xFFFFFFFFu, a1, o);
    mn = larger_or_nan(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
  }
  if (lane == 0) {
    fsums[0][warp] = a1;
    fsums[1][warp] = mn;
  }
  for (int w = tid; w < words; w += kPickThreads) {      // what is taken anyway
    uint32_t bits = 0u;
    for (int i = 0; i < 32; ++i) {
      const int m = 32 * w + i;
      if (m < row.held && (m < begin || m >= end)) {
        const int pg = __ldg(tab + m);
        if (pg >= 0 && pg < p.P) bits |= 1u << i;
        else if (pg != -1) record_error(p.err, ATTN_ERR_BAD_PAGES);
      }
    }
    taken[w] = bits;
  }
  __syncthreads();
  int nc = 0;
  a1 = mn = 0.f;
  for (int w = 0; w < kPickThreads / 32; ++w) {
    nc += sums[w];
    a1 += fsums[0][w];
    mn = larger_or_nan(mn, fsums[1][w]);
  }
  __syncthreads();
  auto take = [&](int m) { atomicOr(taken + (m >> 5), 1u << (m & 31)); };
  if (nc <= p.top) {
    for (int m = begin + tid; m < end; m += kPickThreads)
      if (held_page(m)) take(m);
  } else if (p.top > 0) {
    int larger;
    const uint32_t kth = nth_largest<uint32_t>(begin, end, p.top, held_page, [&](int m) { return keys[m]; },
                                               &larger, hist);
    const float tval = value_of(kth);
    // (1 % and the smallest normal number cover this product's own roundings)
    const float e2 = 2.02f * static_cast<float>(p.G + 16) * 5.9604645e-8f * a1 * mn + 1.17549435e-38f;
    const float hi = tval + e2, lo = tval - e2;          // a NaN or infinity in either: all are undecided
    const bool clear = isfinite(hi) && isfinite(lo);
    int sure = 0, open = 0;
    for (int m = begin + tid; m < end; m += kPickThreads) {
      if (!held_page(m)) continue;
      const float x = value_of(keys[m]);
      if (clear && x > hi) ++sure;
      else if (!(clear && x < lo)) ++open;
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
    for (int w = 0; w < kPickThreads / 32; ++w) {
      sure += sums[w];
      open += hist[w];
    }
    __syncthreads();
    const int want = p.top - sure;                       // of the open ones
    auto is_open = [&](int m) {
      if (!held_page(m)) return false;
      const float x = value_of(keys[m]);
      return !(clear && (x > hi || x < lo));
    };
    for (int m = begin + tid; m < end; m += kPickThreads)
      if (held_page(m) && clear && value_of(keys[m]) > hi) take(m);
    if (open <= want) {
      for (int m = begin + tid; m < end; m += kPickThreads)
        if (is_open(m)) take(m);
    } else if (want > 0) {
      // scored again: a warp an open page
      for (int m0 = begin + warp * 32; m0 < end; m0 += kPickThreads) {
        uint32_t todo = __ballot_sync(0xFFFFFFFFu, m0 + lane < end && is_open(m0 + lane));
        for (; todo != 0u; todo &= todo - 1) {
          const int m = m0 + __ffs(todo) - 1;
          const float* src = p.means + (static_cast<size_t>(__ldg(tab + m)) * p.Hkv + h) * D;
          double d = 0.0;
          for (int e = lane; e < D; e += 32) d = fma(qd[e], static_cast<double>(__ldg(src + e)), d);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
          if (lane == 0) exact[m] = d;
        }
      }
      __syncthreads();
      int more;
      const unsigned long long kd = nth_largest<unsigned long long>(
          begin, end, want, is_open, [&](int m) { return order_of(exact[m]); }, &more, hist);
      // those above it, and of those that equal it the first ones
      int equal = want - more;
      for (int m0 = begin; m0 < end; m0 += kPickThreads) {
        const int m = m0 + tid;
        unsigned long long k = 0;
        const bool is = m < end && is_open(m);
        if (is) k = order_of(exact[m]);
        if (is && k > kd) take(m);
        const bool same = is && k == kd;
        const uint32_t votes = __ballot_sync(0xFFFFFFFFu, same);
        if (lane == 0) sums[warp] = __popc(votes);
        __syncthreads();
        int before = __popc(votes & ((1u << lane) - 1u)), total = 0;
        for (int w = 0; w < kPickThreads / 32; ++w) {
          if (w < warp) before += sums[w];
          total += sums[w];
        }
        if (same && before < equal) take(m);
        equal -= total;
        __syncthreads();
      }
    }
  }
  __syncthreads();
  // the list, in ascending order
  int base = 0;
  for (int w0 = 0; w0 < words; w0 += kPickThreads) {
    const int w = w0 + tid;
    uint32_t bits = w < words ? taken[w] : 0u;
    int x = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int place = base + x - __popc(bits);
    for (int v = 0; v < warp; ++v) place += sums[v];
    for (; bits != 0u; bits &= bits - 1, ++place)
      if (place < p.R) out[place] = __ldg(tab + 32 * w + __ffs(bits) - 1);
    for (int v = 0; v < kPickThreads / 32; ++v) base += sums[v];
    __syncthreads();
  }
  for (int i = base + tid; i < p.R; i += kPickThreads) out[i] = -1;
  if (tid == 0 && h == 0) {
    // every page listed is whole, but for the row's own
    const bool own = held_page(row.held - 1);
    if (!own) record_error(p.err, ATTN_ERR_BAD_PAGES);
    p.out_lens[t] = own ? ((base - 1) << p.page_log2) + row.n - ((row.held - 1) << p.page_log2)
                        : base << p.page_log2;
  }
}

// Rows scored together: a chunk's share their sequence's means.
int score_rows(int T, int S) { return T >= 4ll * S ? 8 : 1; }
// Rows of a launch: at most 2^26 scores (768 MB with the second ones), and a grid's 65535.
long long select_chunk(int T, int Hkv, int M) {
  const long long rows = (1ll << 26) / (static_cast<long long>(Hkv) * M) / 8 * 8;
  return std::min<long long>(T, std::max<long long>(8, std::min<long long>(rows, 65528)));
}
int score_parts(long long rows, int RT, int Hkv, int M) {
  const long long tiles = (rows + RT - 1) / RT * Hkv;
  const long long most = (M + kScoreWarps * kScorePages - 1) / (kScoreWarps * kScorePages);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(most, 152ll * 16 / tiles)));
}
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

bool select_sizes(int T, int S, int H, int Hkv, int d, int M, int page, int top, int local, int first) {
  if (T < 1 || S < 1 || M < 1 || top < 0 || local < 1 || first < 0) return false;
  if (!valid_kv_heads(H, Hkv) || (d != 64 && d != 128) || S > kMaxSeqs || M > kMaxSelectPages) return false;
  if (page < 16 || page > 1024 || (page & (page - 1))) return false;
  if (H > 65535) return false;
  const long long R = static_cast<long long>(top) + local + first;
  return R <= 0x7FFFFFFFll && static_cast<long long>(T) * Hkv <= 0x7FFFFFFFll / std::max<long long>(R, 1);
}
size_t select_workspace(int T, int S, int Hkv, int M) {
  const long long rows = select_chunk(T, Hkv, M);
  const size_t slots = static_cast<size_t>(rows) * Hkv;
  const int parts = score_parts(rows, score_rows(T, S), Hkv, M);
  return up256(slots * M * 4) + up256(slots * M * 8) + slots * parts * 4;
}

bool valid_page_size(int page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }

template <int D>
cudaError_t launch_select_pages(SelectParams p, int RT, cudaStream_t st) {
  auto pick = select_pick_kernel<D>;
  const int smem = p.M * 4 + (p.M + 31) / 32 * 4;
  constexpr int kMaxDev = 64;
  static bool configured[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(pick, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMaxSelectPages * 4 + kMaxSelectPages / 8);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int chunk = static_cast<int>(select_chunk(p.T, p.Hkv, p.M));
  for (int t0 = 0; t0 < p.T; t0 += chunk) {
    p.t0 = t0;
    p.rows = std::min(chunk, p.T - t0);
    const dim3 grid(p.parts, (p.rows + RT - 1) / RT, p.Hkv);
    if (RT == 1) select_score_kernel<D, 1><<<grid, kScoreWarps * 32, 0, st>>>(p);
    else select_score_kernel<D, 8><<<grid, kScoreWarps * 32, 0, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    pick<<<dim3(p.rows, p.Hkv), kPickThreads, smem, st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
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
  // the pages that became full are known on the device alone: CTAs enough for all
  // of a few sequences, and few a sequence where there are many
  const int gy = std::min(S, 65535);
  const long long most = (static_cast<long long>(max_pages) * H_kv + kPoolWarps - 1) / kPoolWarps;
  const dim3 grid(static_cast<unsigned>(std::max<long long>(1, std::min<long long>(most, 152 * 8 / gy))), gy);
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
  const size_t slots = static_cast<size_t>(rows) * H_kv;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.score = reinterpret_cast<float*>(ws);
  p.exact = reinterpret_cast<double*>(ws + up256(slots * max_pages * 4));
  p.norm = reinterpret_cast<float*>(ws + up256(slots * max_pages * 4) + up256(slots * max_pages * 8));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = d == 64 ? launch_select_pages<64>(p, RT, st) : launch_select_pages<128>(p, RT, st);
  return cuda_status("attn_select_pages launch", e);
}
