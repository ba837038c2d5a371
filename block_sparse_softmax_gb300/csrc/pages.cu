// The pages of a key/value cache: reservation and writing of new tokens,
// forking, freeing, eviction behind a sliding window, compaction, and copies.
//
// State, all int32 on the device:
//   page_table [S][M]  the pages of sequence s in order, -1 where it holds none
//   seq_lens   [S]     its tokens; token t lies in slot t / page_size, row t % page_size
//   refs       [P]     how many table entries hold a page; 0: the page is free
// Pages are taken from the lowest free index up, in sequence (or fork) order,
// so the same calls give the same tables in every run.  A page that is not
// full is held by one sequence only (forking copies it), so writing a token
// never touches a shared page.
//
// The bookkeeping kernels are bound by latency: one CTA reads `refs` once or
// twice and decides everything before it changes anything, so a call that
// cannot be met in full changes nothing.  Copying is bound by HBM bandwidth:
// 16 bytes a thread and access, consecutive threads on consecutive addresses.
// Writing moves 16 bytes a thread too; a decoding step's tokens are latency, a
// prompt's are bound by the instructions that find each 16 bytes' place (a
// division, the search for the sequence), which e4m3's divisions add to.
// Measured: a token for each of 256 sequences (14861 pages) reserved in 9 us,
// pages behind a window evicted in 4, the tokens written in 6; 16384 pages,
// half of them in use, compacted in 16 us and their 4096 pages of 64 KB, K and
// V, copied in 163 us (6.6 TB/s read and written, 97 % of a plain copy's).
// Prompts of 4096 tokens, 4 K/V heads of 128: one written in 8 us (2.0 TB/s read
// and written; e4m3 9.6 us, 1.3 TB/s), 64 in 289 us (3.7 TB/s, 55 %; e4m3 386 us,
// 2.1 TB/s, 31 %).
#include <cuda_fp8.h>

#include "host.cuh"

namespace bss {
namespace {

constexpr int kMaxSeqs = 65536;      // rows of a page table (the fork kernel keeps a bit for each)
constexpr int kMaxPages = 1 << 30;   // pages of a cache
constexpr int kBookThreads = 1024;

struct PageState {
  int* table;
  int* lens;
  int* refs;
  int S, M, P, page;
  int* err;
};

__device__ __forceinline__ int ceil_div(long long a, int b) { return static_cast<int>((a + b - 1) / b); }

// Exclusive prefix sum of one number per thread over the 1024 threads; *total
// gets the sum.  Ends with a barrier.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T* total) {
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const T before = (warp > 0 ? warp_sums[warp - 1] : T(0)) + x - v;
  *total = warp_sums[kBookThreads / 32 - 1];
  __syncthreads();
  return before;
}

// A thread's 32 entries of `refs` from 32 * t on as a mask of the pages in use
// (bits past the last page are clear); all eight loads are in flight at once.
constexpr int kSpan = 32 * kBookThreads;          // entries the block looks at in one turn
__device__ __forceinline__ uint32_t used_mask(const int* refs, int P, long long first) {
  uint32_t mask = 0;
  if (first + 32 <= P && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0) {
    int4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const int4*>(refs + first + 4 * u);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      mask |= (v[u].x > 0 ? 1u : 0u) << (4 * u) | (v[u].y > 0 ? 2u : 0u) << (4 * u) |
              (v[u].z > 0 ? 4u : 0u) << (4 * u) | (v[u].w > 0 ? 8u : 0u) << (4 * u);
  } else {
    for (int u = 0; u < 32 && first + u < P; ++u) mask |= (refs[first + u] > 0 ? 1u : 0u) << u;
  }
  return mask;
}
// ... of the pages that exist.
__device__ __forceinline__ uint32_t page_mask(int P, long long first) {
  return first >= P ? 0u : first + 32 <= P ? 0xFFFFFFFFu : (1u << (P - first)) - 1u;
}

// Calls take(rank, page) for the `want` lowest free pages in ascending order,
// or returns false without a call when there are fewer.  Free pages often lie
// side by side, in few threads' masks: up to kPageList of them are listed in
// shared memory and given out by all threads.
constexpr int kPageList = 4096;
template <class Take>
__device__ bool take_free_pages(const int* refs, int P, int want, int* warp_sums, const Take& take) {
  __shared__ int list[kPageList];
  if (want == 0) return true;
  const bool once = P <= kSpan;                   // one turn: counted and given out at a time
  for (int pass = once ? 1 : 0; pass < 2; ++pass) {
    int found = 0;
    for (long long x0 = 0; x0 < P && found < want; x0 += kSpan) {
      const long long x = x0 + 32ll * threadIdx.x;
      uint32_t free = page_mask(P, x) & ~used_mask(refs, P, x);
      int total;
      int rank = found + block_scan(__popc(free), warp_sums, &total);
      if (once && total < want) return false;
      if (pass == 1)
        for (; free != 0 && rank < want; free &= free - 1, ++rank) {
          const int page = static_cast<int>(x) + __ffs(free) - 1;
          if (want <= kPageList) list[rank] = page;
          else take(rank, page);
        }
      found += total;
    }
    if (pass == 0 && found < want) return false;
  }
  __syncthreads();
  if (want <= kPageList)
    for (int r = static_cast<int>(threadIdx.x); r < want; r += kBookThreads) take(r, list[r]);
  __syncthreads();
  return true;
}

// attn_kv_reserve: n_new[s] more tokens for every sequence.  start[s] is the
// place of the first of them, or -1 for every sequence when nothing was done.
__global__ void __launch_bounds__(kBookThreads) kv_reserve_kernel(const PageState st, const int* n_new,
                                                                  int* start) {
  __shared__ int warp_sums[32];
  __shared__ long long wide_sums[32];             // a sum of needs may pass 32 bits
  const int tid = static_cast<int>(threadIdx.x);
  long long want = 0;
  int bad = 0, over = 0;
  for (int s0 = 0; s0 < st.S; s0 += kBookThreads) {
    const int s = s0 + tid;
    long long need = 0;
    if (s < st.S) {
      const int len = st.lens[s], n = n_new[s];
      if (len < 0 || n < 0 ||
          static_cast<long long>(len) + n > min(static_cast<long long>(st.M) * st.page, static_cast<long long>(kMaxTokens)))
        bad = 1;
      else
        need = ceil_div(static_cast<long long>(len) + n, st.page) - ceil_div(len, st.page);
    }
    long long total;
    const long long before = block_scan(need, wide_sums, &total);
    // pages given out before this sequence (at most P where it is used)
    if (s < st.S) start[s] = static_cast<int>(min(want + before, static_cast<long long>(st.P)));
    want += total;
    if (want > st.P) over = 1;
    if (__syncthreads_or(bad | over)) break;
  }
  bad = __syncthreads_or(bad);
  over = __syncthreads_or(over);
  bool ok = !bad && !over;
  if (ok)
    ok = take_free_pages(st.refs, st.P, static_cast<int>(want), warp_sums, [&](int rank, int page) {
      // the last sequence whose first page has at most this rank: sequences
      // that need no page share their successor's rank and are passed over
      int lo = 0, hi = st.S - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= rank) lo = mid;
        else hi = mid - 1;
      }
      const int slot = ceil_div(st.lens[lo], st.page) + rank - start[lo];
      st.table[static_cast<size_t>(lo) * st.M + slot] = page;
      st.refs[page] = 1;
    });
  __syncthreads();
  for (int s = tid; s < st.S; s += kBookThreads) {
    if (ok) {
      const int len = st.lens[s];
      start[s] = len;
      st.lens[s] = len + n_new[s];
    } else {
      start[s] = -1;
    }
  }
  if (!ok && tid == 0) record_error(st.err, bad ? ATTN_ERR_BAD_PAGES : ATTN_ERR_NO_PAGES);
}

// attn_kv_fork: sequence children[f] becomes a copy of parents[f].  Full pages
// are shared; of a last page that is not full the child gets its own, listed
// in copy_src / copy_dst (-1 where there is none).
__global__ void __launch_bounds__(kBookThreads) kv_fork_kernel(const PageState st, const int* parents,
                                                               const int* children, int F, int* copy_src,
                                                               int* copy_dst) {
  __shared__ int warp_sums[32];
  extern __shared__ uint32_t child_bits[];        // one bit per sequence
  const int tid = static_cast<int>(threadIdx.x);
  for (int w = tid; w < (st.S + 31) / 32; w += kBookThreads) child_bits[w] = 0u;
  __syncthreads();
  int bad = 0;
  for (int f = tid; f < F; f += kBookThreads) {
    const int c = children[f];
    if (c < 0 || c >= st.S) {
      bad = 1;
    } else {
      const uint32_t bit = 1u << (c & 31);
      if (atomicOr(child_bits + (c >> 5), bit) & bit) bad = 1;     // the same child twice
      if (st.lens[c] != 0) bad = 1;                                // a child holds nothing before
    }
  }
  __syncthreads();
  int want = 0;
  for (int f0 = 0; f0 < F; f0 += kBookThreads) {
    const int f = f0 + tid;
    int part = 0;
    if (f < F) {
      const int a = parents[f];
      if (a < 0 || a >= st.S || (child_bits[a >> 5] >> (a & 31) & 1u)) {   // a parent that is a child, too
        bad = 1;
      } else {
        const int len = st.lens[a];
        if (len < 0 || len > static_cast<long long>(st.M) * st.page) {
          bad = 1;
        } else if (len % st.page != 0) {
          part = 1;
          const int e = st.table[static_cast<size_t>(a) * st.M + len / st.page];
          if (e < 0 || e >= st.P) bad = 1;
        }
      }
      copy_dst[f] = -1;
    }
    int total;
    const int before = block_scan(part, warp_sums, &total);
    if (f < F) copy_src[f] = want + before;       // for now the new pages of the forks before it
    want += total;
  }
  bad = __syncthreads_or(bad);
  const bool ok = !bad && take_free_pages(st.refs, st.P, want, warp_sums, [&](int rank, int page) {
    // the last fork with at most this many pages before it
    int lo = 0, hi = F - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (copy_src[mid] <= rank) lo = mid;
      else hi = mid - 1;
    }
    copy_dst[lo] = page;
    st.refs[page] = 1;
  });
  __syncthreads();
  if (!ok) {
    for (int f = tid; f < F; f += kBookThreads) copy_src[f] = copy_dst[f] = -1;
    if (tid == 0) record_error(st.err, bad ? ATTN_ERR_BAD_PAGES : ATTN_ERR_NO_PAGES);
    return;
  }
  // the rows, a warp each: shared full pages, then the child's own page
  const int lane = tid & 31;
  for (int f = tid >> 5; f < F; f += kBookThreads / 32) {
    const int a = parents[f], c = children[f];
    const int len = st.lens[a];
    const int full = len / st.page;
    const int* from = st.table + static_cast<size_t>(a) * st.M;
    int* to = st.table + static_cast<size_t>(c) * st.M;
    const int own = copy_dst[f];
    for (int m = lane; m < st.M; m += 32) {
      int e = -1;
      if (m < full) {
        e = from[m];
        if (e >= st.P) {
          record_error(st.err, ATTN_ERR_BAD_PAGES);
          e = -1;
        }
        if (e >= 0) atomicAdd(st.refs + e, 1);
      } else if (m == full) {
        e = own;
      }
      to[m] = e;
    }
    if (lane == 0) {
      copy_src[f] = own >= 0 ? from[full] : -1;
      st.lens[c] = len;
    }
  }
}

// One entry given back: whoever takes it out of the table lowers its count.
__device__ __forceinline__ void release_entry(const PageState& st, int* entry) {
  const int e = atomicExch(entry, -1);
  if (e < 0) return;
  if (e >= st.P) {
    record_error(st.err, ATTN_ERR_BAD_PAGES);
  } else if (atomicSub(st.refs + e, 1) <= 0) {      // held by nobody: the count stays at 0
    atomicAdd(st.refs + e, 1);
    record_error(st.err, ATTN_ERR_BAD_PAGES);
  }
}

// attn_kv_free: the listed sequences give back every page (a sequence listed
// twice is freed once).
__global__ void __launch_bounds__(256) kv_free_kernel(const PageState st, const int* seqs, int n) {
  const long long total = static_cast<long long>(n) * st.M;
  for (long long x = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int i = static_cast<int>(x / st.M);
    const int m = static_cast<int>(x - static_cast<long long>(i) * st.M);
    const int s = seqs[i];
    if (s < 0 || s >= st.S) {
      if (m == 0) record_error(st.err, ATTN_ERR_BAD_PAGES);
      continue;
    }
    release_entry(st, st.table + static_cast<size_t>(s) * st.M + m);
    if (m == 0) st.lens[s] = 0;
  }
}

// attn_kv_evict: every page wholly behind the window and past the sinks is
// given back (the token at position len - 1 sees len - window and later).
__global__ void __launch_bounds__(256) kv_evict_kernel(const PageState st, long long window,
                                                       long long sinks) {
  const long long total = static_cast<long long>(st.S) * st.M;
  for (long long x = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int s = static_cast<int>(x / st.M);
    const long long m = x - static_cast<long long>(s) * st.M;
    if (m * st.page < sinks || (m + 1) * st.page > st.lens[s] - window) continue;
    release_entry(st, st.table + x);
  }
}

// attn_kv_compact: the pages in use at or past the number of pages in use move,
// in ascending order, to the free pages below it.  Where pages and table are
// small enough the block also rewrites the table, by a map in shared memory.
constexpr int kSmallTable = 1 << 16;
__global__ void __launch_bounds__(kBookThreads) kv_compact_kernel(int* refs, int P, int* copy_src,
                                                                  int* copy_dst, int* count, int* table,
                                                                  int entries, int* err) {
  __shared__ int warp_sums[32];
  __shared__ unsigned pair_sums[32];
  extern __shared__ int to[];                     // [P]: a moved page's place, else -1 (entries > 0)
  const int tid = static_cast<int>(threadIdx.x);
  const bool once = P <= kSpan;
  if (entries > 0)
    for (int i = tid; i < P; i += kBookThreads) to[i] = -1;
  int live = 0;
  uint32_t kept = 0;
  for (long long x0 = 0; x0 < P; x0 += kSpan) {
    kept = used_mask(refs, P, x0 + 32ll * tid);
    int total;
    block_scan(__popc(kept), warp_sums, &total);
    live += total;
  }
  int n_src = 0, n_dst = 0;
  for (long long x0 = 0; x0 < P; x0 += kSpan) {
    const long long x = x0 + 32ll * tid;
    const uint32_t used = once ? kept : used_mask(refs, P, x);
    const uint32_t low = page_mask(live, x);      // the places below the number in use
    uint32_t src = used & ~low;
    uint32_t dst = ~used & low;
    unsigned total;
    const unsigned rank = block_scan((static_cast<unsigned>(__popc(src)) << 16) + __popc(dst), pair_sums, &total);
    for (int r = n_src + static_cast<int>(rank >> 16); src != 0; src &= src - 1)
      copy_src[r++] = static_cast<int>(x) + __ffs(src) - 1;
    for (int r = n_dst + static_cast<int>(rank & 0xFFFFu); dst != 0; dst &= dst - 1)
      copy_dst[r++] = static_cast<int>(x) + __ffs(dst) - 1;
    n_src += static_cast<int>(total >> 16);
    n_dst += static_cast<int>(total & 0xFFFFu);
  }
  __syncthreads();
  // a batch's loads are in flight together (one CTA: latency is what counts)
  constexpr int kBatch = 8;
  for (int i0 = tid; i0 < n_src; i0 += kBatch * kBookThreads) {
    int a[kBatch], b[kBatch], held[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kBookThreads;
      a[u] = i < n_src ? copy_src[i] : -1;
      b[u] = i < n_src ? copy_dst[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) held[u] = a[u] >= 0 ? refs[a[u]] : 0;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (a[u] < 0) continue;
      refs[b[u]] = held[u];
      refs[a[u]] = 0;
      if (entries > 0) to[a[u]] = b[u];
    }
  }
  for (int i = n_src + tid; i < P; i += kBookThreads) copy_src[i] = copy_dst[i] = -1;
  if (tid == 0) *count = n_src;
  if (entries == 0) return;
  __syncthreads();
  for (int i0 = tid; i0 < entries; i0 += kBatch * kBookThreads) {
    int e[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kBookThreads;
      e[u] = i < entries ? table[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (e[u] >= P) record_error(err, ATTN_ERR_BAD_PAGES);
      else if (e[u] >= 0 && to[e[u]] >= 0) table[i0 + u * kBookThreads] = to[e[u]];
    }
  }
}

// A larger table's entries follow in a launch of their own (copy_src ascends).
__global__ void __launch_bounds__(256) kv_remap_kernel(int* table, long long entries, int P,
                                                       const int* copy_src, const int* copy_dst,
                                                       const int* count, int* err) {
  const int n = *count;
  const int first = n > 0 ? copy_src[0] : P;      // (nothing moves: entries out of range are still reported)
  for (long long x = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; x < entries;
       x += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int e = table[x];
    if (e < first) continue;
    if (e >= P) {
      record_error(err, ATTN_ERR_BAD_PAGES);
      continue;
    }
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (copy_src[mid] < e) lo = mid + 1;
      else hi = mid;
    }
    if (copy_src[lo] == e) table[x] = copy_dst[lo];
  }
}

struct CopyParams {
  uint8_t* k;
  uint8_t* v;
  size_t k_stride, v_stride;    // bytes from page to page
  long long page_bytes;
  int P;
  const int* src;
  const int* dst;
  int n;
  const int* count;             // null: n pairs
  int* err;
};

// attn_kv_copy_pages: 16 KB of one cache's page per block and turn.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll * 16;
__global__ void __launch_bounds__(kCopyThreads) kv_copy_pages_kernel(const CopyParams p) {
  const int n = p.count ? max(0, min(p.n, __ldg(p.count))) : p.n;
  const long long chunks = (p.page_bytes + kCopyChunk - 1) / kCopyChunk;
  const long long units = 2ll * n * chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long pair2 = u / chunks;
    const long long off = (u - pair2 * chunks) * kCopyChunk;
    const int i = static_cast<int>(pair2 >> 1);
    const int a = __ldg(p.src + i), b = __ldg(p.dst + i);
    if (a < 0 && b < 0) continue;                 // no copy here
    if (a < 0 || a >= p.P || b < 0 || b >= p.P) {
      if (threadIdx.x == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
      continue;
    }
    uint8_t* base = (pair2 & 1) ? p.v : p.k;
    const size_t stride = (pair2 & 1) ? p.v_stride : p.k_stride;
    const uint4* from = reinterpret_cast<const uint4*>(base + a * stride + off);
    uint4* to = reinterpret_cast<uint4*>(base + b * stride + off);
    const int left = static_cast<int>(min(static_cast<long long>(kCopyChunk), p.page_bytes - off) / 16);
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int w = 0; w < kCopyUnroll; ++w) {
      const int t = w * kCopyThreads + static_cast<int>(threadIdx.x);
      if (t < left) x[w] = from[t];
    }
#pragma unroll
    for (int w = 0; w < kCopyUnroll; ++w) {
      const int t = w * kCopyThreads + static_cast<int>(threadIdx.x);
      if (t < left) to[t] = x[w];
    }
  }
}

struct WriteParams {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  long long k_row, v_row;       // elements from token to token
  uint8_t* k;
  uint8_t* v;
  size_t k_stride, v_stride;    // bytes from page to page
  const float* k_scale;         // [Hkv], e4m3 caches
  const float* v_scale;
  const int* table;
  const int* start;
  const int* cu;
  int T, S, M, P, Hkv, d, page;
  int* err;
};

// 8 elements of one token's K or V: a copy, or x / scale rounded to e4m3
// (saturated at 448, as the format holds no infinity).
template <bool FP8>
__global__ void __launch_bounds__(256) kv_write_kernel(const WriteParams p) {
  const int per = p.Hkv * p.d / 8;
  const long long total = 2ll * p.T * per;
  for (long long x = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * blockDim.x) {
    const long long t2 = x / per;
    const int e = static_cast<int>(x - t2 * per) * 8;          // element of [Hkv][d]
    const int t = static_cast<int>(t2 >> 1);
    const bool is_v = t2 & 1;
    // the sequence of token t: the last s with cu[s] <= t
    int lo = 0, hi = p.S;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(p.cu + mid) <= t) lo = mid;
      else hi = mid - 1;
    }
    if (lo >= p.S || __ldg(p.cu + lo) > t) continue;           // a token behind the last sequence
    const int s0 = __ldg(p.start + lo);
    if (s0 < 0) continue;                                      // nothing was reserved
    const long long pos = static_cast<long long>(s0) + t - __ldg(p.cu + lo);
    const long long slot = pos / p.page;
    const int page = slot < p.M ? __ldg(p.table + static_cast<size_t>(lo) * p.M + slot) : -1;
    if (page < 0 || page >= p.P) {
      if (e == 0) record_error(p.err, ATTN_ERR_BAD_PAGES);
      continue;
    }
    const int h = e / p.d;
    const size_t at = (static_cast<size_t>(h) * p.page + (pos - slot * p.page)) * p.d + (e - h * p.d);
    const uint4 raw = *reinterpret_cast<const uint4*>((is_v ? p.v_new + t * p.v_row : p.k_new + t * p.k_row) + e);
    uint8_t* base = is_v ? p.v + page * p.v_stride : p.k + page * p.k_stride;
    if constexpr (!FP8) {
      *reinterpret_cast<uint4*>(base + at * 2) = raw;
    } else {
      const float sc = __ldg((is_v ? p.v_scale : p.k_scale) + h);
      const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t out[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t q = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(bf16lo(in[i]), sc), __fdiv_rn(bf16hi(in[i]), sc)), __NV_SATFINITE, __NV_E4M3);
        out[i >> 1] |= static_cast<uint32_t>(q) << (16 * (i & 1));
      }
      *reinterpret_cast<uint2*>(base + at) = make_uint2(out[0], out[1]);
    }
  }
}

unsigned grid_256(long long work) {
  long long b = (work + 255) / 256;
  return static_cast<unsigned>(b < 1 ? 1 : (b > 152ll * 16 ? 152ll * 16 : b));
}

// The compaction's map in shared memory is past the 48 KB that a kernel has
// without asking: asked for once a device.
attn_status_t allow_compact_smem() {
  constexpr int kMaxDev = 64;
  static bool configured[kMaxDev] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status("cudaGetDevice", e);
  if (dev < 0 || dev >= kMaxDev) return ATTN_ERR_UNSUPPORTED;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(kv_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpan * 4);
    if (e != cudaSuccess) return cuda_status("cudaFuncSetAttribute", e);
    configured[dev] = true;
  }
  return ATTN_OK;
}

bool valid_page_size(int page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }

attn_status_t page_state(PageState* st, int32_t* table, int32_t* lens, int32_t* refs, int S, int M,
                         int P, int page) {
  if (!table || !lens || !refs || !aligned4(table) || !aligned4(lens) || !aligned4(refs))
    return ATTN_ERR_INVALID_ARG;
  if (S < 1 || M < 1 || P < 1) return ATTN_ERR_INVALID_ARG;
  if (S > kMaxSeqs || P > kMaxPages || !valid_page_size(page)) return ATTN_ERR_UNSUPPORTED;
  *st = PageState{table, lens, refs, S, M, P, page, nullptr};
  return ATTN_OK;
}

attn_status_t check_cache(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int P,
                          int Hkv, int d, int page, int kv_dtype) {
  if (!k || !v || !aligned16(k) || !aligned16(v)) return ATTN_ERR_INVALID_ARG;
  if (P < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !valid_page_size(page)) return ATTN_ERR_UNSUPPORTED;
  if (kv_dtype != ATTN_KV_BF16 && kv_dtype != ATTN_KV_E4M3) return ATTN_ERR_UNSUPPORTED;
  const int64_t least = static_cast<int64_t>(Hkv) * page * d;
  const int64_t unit = kv_dtype == ATTN_KV_E4M3 ? 16 : 8;      // elements of 16 bytes
  if (Hkv > 65536 || k_stride < least || v_stride < least || k_stride % unit || v_stride % unit)
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

}  // namespace
}  // namespace bss

using namespace bss;

extern "C" {

attn_status_t attn_kv_reserve(int32_t* page_table, int32_t* seq_lens, int32_t* refs,
                              const int32_t* n_new, int32_t* start, int S, int max_pages,
                              int n_pages, int page_size, void* stream) {
  PageState st;
  attn_status_t s = page_state(&st, page_table, seq_lens, refs, S, max_pages, n_pages, page_size);
  if (s != ATTN_OK) return s;
  if (!n_new || !start || !aligned4(n_new) || !aligned4(start)) return ATTN_ERR_INVALID_ARG;
  if ((s = status_word(&st.err)) != ATTN_OK) return s;
  kv_reserve_kernel<<<1, kBookThreads, 0, static_cast<cudaStream_t>(stream)>>>(st, n_new, start);
  return cuda_status("attn_kv_reserve launch", cudaGetLastError());
}

attn_status_t attn_kv_write(const void* k_new, const void* v_new, int64_t k_new_stride,
                            int64_t v_new_stride, void* k_cache, void* v_cache,
                            int64_t k_page_stride, int64_t v_page_stride, int kv_dtype,
                            const float* k_scale, const float* v_scale, const int32_t* page_table,
                            const int32_t* start, const int32_t* cu_new, int T, int S, int max_pages,
                            int n_pages, int H_kv, int d, int page_size, void* stream) {
  attn_status_t s = check_cache(k_cache, v_cache, k_page_stride, v_page_stride, n_pages, H_kv, d,
                                page_size, kv_dtype);
  if (s != ATTN_OK) return s;
  if (T < 0 || S < 1 || max_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (S > kMaxSeqs) return ATTN_ERR_UNSUPPORTED;
  if (!page_table || !start || !cu_new || !aligned4(page_table) || !aligned4(start) || !aligned4(cu_new))
    return ATTN_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == ATTN_KV_E4M3;
  if (fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr) || !aligned4(k_scale) || !aligned4(v_scale))
    return ATTN_ERR_INVALID_ARG;
  if (T == 0) return ATTN_OK;
  if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return ATTN_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(H_kv) * d;
  if (k_new_stride < row || v_new_stride < row || k_new_stride % 8 || v_new_stride % 8)
    return ATTN_ERR_INVALID_ARG;
  WriteParams p{};
  if ((s = status_word(&p.err)) != ATTN_OK) return s;
  const size_t item = fp8 ? 1 : 2;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.k_row = k_new_stride;
  p.v_row = v_new_stride;
  p.k = static_cast<uint8_t*>(k_cache);
  p.v = static_cast<uint8_t*>(v_cache);
  p.k_stride = static_cast<size_t>(k_page_stride) * item;
  p.v_stride = static_cast<size_t>(v_page_stride) * item;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.table = page_table;
  p.start = start;
  p.cu = cu_new;
  p.T = T;
  p.S = S;
  p.M = max_pages;
  p.P = n_pages;
  p.Hkv = H_kv;
  p.d = d;
  p.page = page_size;
  const unsigned grid = grid_256(2ll * T * (row / 8));
  const cudaStream_t q = static_cast<cudaStream_t>(stream);
  if (fp8) kv_write_kernel<true><<<grid, 256, 0, q>>>(p);
  else kv_write_kernel<false><<<grid, 256, 0, q>>>(p);
  return cuda_status("attn_kv_write launch", cudaGetLastError());
}

attn_status_t attn_kv_fork(int32_t* page_table, int32_t* seq_lens, int32_t* refs,
                           const int32_t* parents, const int32_t* children, int n_forks,
                           int32_t* copy_src, int32_t* copy_dst, int S, int max_pages, int n_pages,
                           int page_size, void* stream) {
  PageState st;
  attn_status_t s = page_state(&st, page_table, seq_lens, refs, S, max_pages, n_pages, page_size);
  if (s != ATTN_OK) return s;
  if (n_forks < 0 || n_forks > kMaxSeqs) return ATTN_ERR_INVALID_ARG;
  if (n_forks == 0) return ATTN_OK;
  const void* ptrs[] = {parents, children, copy_src, copy_dst};
  for (const void* x : ptrs)
    if (!x || !aligned4(x)) return ATTN_ERR_INVALID_ARG;
  if ((s = status_word(&st.err)) != ATTN_OK) return s;
  kv_fork_kernel<<<1, kBookThreads, (S + 31) / 32 * 4, static_cast<cudaStream_t>(stream)>>>(
      st, parents, children, n_forks, copy_src, copy_dst);
  return cuda_status("attn_kv_fork launch", cudaGetLastError());
}

attn_status_t attn_kv_free(int32_t* page_table, int32_t* seq_lens, int32_t* refs,
                           const int32_t* seqs, int n_seqs, int S, int max_pages, int n_pages,
                           int page_size, void* stream) {
  PageState st;
  attn_status_t s = page_state(&st, page_table, seq_lens, refs, S, max_pages, n_pages, page_size);
  if (s != ATTN_OK) return s;
  if (n_seqs < 0) return ATTN_ERR_INVALID_ARG;
  if (n_seqs == 0) return ATTN_OK;
  if (!seqs || !aligned4(seqs)) return ATTN_ERR_INVALID_ARG;
  if ((s = status_word(&st.err)) != ATTN_OK) return s;
  kv_free_kernel<<<grid_256(static_cast<long long>(n_seqs) * max_pages), 256, 0,
                   static_cast<cudaStream_t>(stream)>>>(st, seqs, n_seqs);
  return cuda_status("attn_kv_free launch", cudaGetLastError());
}

attn_status_t attn_kv_evict(int32_t* page_table, const int32_t* seq_lens, int32_t* refs,
                            int64_t window, int64_t sinks, int S, int max_pages, int n_pages,
                            int page_size, void* stream) {
  PageState st;
  attn_status_t s = page_state(&st, page_table, const_cast<int32_t*>(seq_lens), refs, S, max_pages,
                               n_pages, page_size);
  if (s != ATTN_OK) return s;
  if (window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  constexpr int64_t kMost = int64_t(1) << 60;
  if ((s = status_word(&st.err)) != ATTN_OK) return s;
  kv_evict_kernel<<<grid_256(static_cast<long long>(S) * max_pages), 256, 0,
                    static_cast<cudaStream_t>(stream)>>>(st, window < kMost ? window : kMost, sinks);
  return cuda_status("attn_kv_evict launch", cudaGetLastError());
}

attn_status_t attn_kv_compact(int32_t* page_table, int32_t* refs, int32_t* copy_src,
                              int32_t* copy_dst, int32_t* count, int S, int max_pages, int n_pages,
                              void* stream) {
  const void* ptrs[] = {page_table, refs, copy_src, copy_dst, count};
  for (const void* x : ptrs)
    if (!x || !aligned4(x)) return ATTN_ERR_INVALID_ARG;
  if (S < 1 || max_pages < 1 || n_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (S > kMaxSeqs || n_pages > kMaxPages) return ATTN_ERR_UNSUPPORTED;
  int* err = nullptr;
  attn_status_t s = status_word(&err);
  if (s != ATTN_OK) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long entries = static_cast<long long>(S) * max_pages;
  const bool inside = entries <= kSmallTable && n_pages <= kSpan;
  const int smem = inside ? n_pages * 4 : 0;
  if ((s = allow_compact_smem()) != ATTN_OK) return s;
  kv_compact_kernel<<<1, kBookThreads, smem, st>>>(refs, n_pages, copy_src, copy_dst, count, page_table,
                                                   inside ? static_cast<int>(entries) : 0, err);
  if ((s = cuda_status("attn_kv_compact launch", cudaGetLastError())) != ATTN_OK || inside) return s;
  kv_remap_kernel<<<grid_256(entries), 256, 0, st>>>(page_table, entries, n_pages, copy_src, copy_dst,
                                                     count, err);
  return cuda_status("attn_kv_compact launch", cudaGetLastError());
}

attn_status_t attn_kv_copy_pages(void* k_cache, void* v_cache, int64_t k_page_stride,
                                 int64_t v_page_stride, int kv_dtype, const int32_t* copy_src,
                                 const int32_t* copy_dst, int n_copies, const int32_t* count,
                                 int n_pages, int H_kv, int d, int page_size, void* stream) {
  attn_status_t s = check_cache(k_cache, v_cache, k_page_stride, v_page_stride, n_pages, H_kv, d,
                                page_size, kv_dtype);
  if (s != ATTN_OK) return s;
  if (n_copies < 0 || !aligned4(count)) return ATTN_ERR_INVALID_ARG;
  if (n_copies == 0) return ATTN_OK;
  if (!copy_src || !copy_dst || !aligned4(copy_src) || !aligned4(copy_dst)) return ATTN_ERR_INVALID_ARG;
  CopyParams p{};
  if ((s = status_word(&p.err)) != ATTN_OK) return s;
  const size_t item = kv_dtype == ATTN_KV_E4M3 ? 1 : 2;
  p.k = static_cast<uint8_t*>(k_cache);
  p.v = static_cast<uint8_t*>(v_cache);
  p.k_stride = static_cast<size_t>(k_page_stride) * item;
  p.v_stride = static_cast<size_t>(v_page_stride) * item;
  p.page_bytes = static_cast<long long>(H_kv) * page_size * d * item;
  p.P = n_pages;
  p.src = copy_src;
  p.dst = copy_dst;
  p.n = n_copies;
  p.count = count;
  const long long chunks = (p.page_bytes + kCopyChunk - 1) / kCopyChunk;
  const long long units = 2ll * n_copies * chunks;
  const unsigned grid = static_cast<unsigned>(units < 152 * 8 ? units : 152 * 8);
  kv_copy_pages_kernel<<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cuda_status("attn_kv_copy_pages launch", cudaGetLastError());
}

}  // extern "C"
