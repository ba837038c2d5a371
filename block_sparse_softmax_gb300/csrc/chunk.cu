// attn_fwd_paged: attention of a chunk of new tokens per sequence over a paged
// key/value cache.
//
// Mathematics: row t of sequence s stands at pos = n - (cu[s+1] - t), n the
// sequence's length; over the keys j <= pos (with a window only those with j >
// pos - window or j < sinks)
//     O = sum_j p_j V_j / l,  p_j = exp(scale q . k_j - m),  l = sum_j p_j.
//
// The simplest form: a warp a row and query head, a key a lane.
#include <cuda_fp16.h>

#include <algorithm>

#include "host.cuh"

namespace bss {
namespace {

constexpr int kMaxSeqs = 65536;

struct ChunkParams {
  const __nv_bfloat16* q;
  long long q_stride;
  const uint8_t* k;
  const uint8_t* v;
  size_t k_stride, v_stride;     // bytes from page to page
  const float* k_scale;
  const float* v_scale;
  const int* table;
  const int* lens;
  const int* cu;
  __nv_bfloat16* o;
  float* lse;
  int T, S, H, Hkv, G, M, P;
  int page_log2;
  float scale_log2;
  long long window;
  int sinks;
  int* err;
};

template <bool FP8>
__device__ __forceinline__ float element(const uint8_t* x, int i) {
  if constexpr (FP8) {
    uint32_t y;
    asm("{\n\t.reg .b16 v;\n\tcvt.u16.u32 v, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, v;\n\t}" : "=r"(y)
        : "r"(static_cast<uint32_t>(x[i])));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(y & 0xFFFFu)));
  } else {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x)[i]);
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(128) attn_fwd_paged_kernel(const ChunkParams p) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const long long x = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (x >= static_cast<long long>(p.T) * p.H) return;
  const int t = static_cast<int>(x / p.H), h = static_cast<int>(x % p.H), hkv = h / p.G;
  int s = 0, hi = p.S;
  while (s < hi) {
    const int mid = (s + hi + 1) >> 1;
    if (__ldg(p.cu + mid) <= t) s = mid;
    else hi = mid - 1;
  }
  if (s >= p.S || __ldg(p.cu + s) > t) return;               // a row of no sequence
  const long long most = min(static_cast<long long>(p.M) << p.page_log2, static_cast<long long>(kMaxTokens));
  const int len = __ldg(p.lens + s);
  const long long n = max(0ll, min(static_cast<long long>(len), most));
  const long long pos = min(n, n - (static_cast<long long>(__ldg(p.cu + s + 1)) - t) + 1) - 1;
  if (lane == 0 && (len < 0 || len > most || pos < 0)) record_error(p.err, ATTN_ERR_BAD_PAGES);
  float q[D];
  const __nv_bfloat16* qp = p.q + t * p.q_stride + static_cast<long long>(h) * D;
#pragma unroll
  for (int i = 0; i < D; ++i) q[i] = __bfloat162float(qp[i]);
  const float sl2 = p.scale_log2 * (FP8 ? __ldg(p.k_scale + hkv) : 1.f);
  const float NEG_INF = -__int_as_float(0x7f800000);
  float m = NEG_INF, l = 0.f, acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  const long long lo = p.window > 0 ? max(0ll, pos + 1 - p.window) : 0;
  for (long long j0 = 0; j0 <= pos; j0 += 32) {
    if (j0 + 32 <= lo && j0 >= p.sinks) continue;
    const long long j = j0 + lane;
    bool seen = j <= pos && (j >= lo || j < p.sinks);
    int pg = 0;
    if (seen) {
      pg = __ldg(p.table + static_cast<size_t>(s) * p.M + (j >> p.page_log2));
      if (pg < 0 || pg >= p.P) {
        record_error(p.err, ATTN_ERR_BAD_PAGES);
        seen = false;
        pg = 0;
      }
    }
    const size_t off = ((static_cast<size_t>(hkv) << p.page_log2) + (j & ((1 << p.page_log2) - 1))) * D * (FP8 ? 1 : 2);
    float y = NEG_INF;
    if (seen) {
      const uint8_t* kp = p.k + pg * p.k_stride + off;
      float d = 0.f;
      for (int i = 0; i < D; ++i) d = fmaf(q[i], element<FP8>(kp, i), d);
      y = d * sl2;
    }
    float mx = y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    const float mn = fmaxf(m, mx);
    const float mu = mn == NEG_INF ? 0.f : mn;
    const float al = exp2f(m - mu), pr = seen ? exp2f(y - mu) : 0.f;
    m = mn;
    l = l * al + pr;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= al;
    for (int u = 0; u < 32; ++u) {
      if (!__shfl_sync(0xFFFFFFFFu, seen ? 1 : 0, u)) continue;
      const float pu = __shfl_sync(0xFFFFFFFFu, pr, u);
      const uint8_t* vp = p.v + __shfl_sync(0xFFFFFFFFu, pg, u) * p.v_stride + __shfl_sync(0xFFFFFFFFu, off, u);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(pu, element<FP8>(vp, i * 32 + lane), acc[i]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  const float inv = l == 0.f ? 0.f : (FP8 ? __ldg(p.v_scale + hkv) : 1.f) / l;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p.o[x * D + i * 32 + lane] = __float2bfloat16(acc[i] * inv);
  if (lane == 0) p.lse[x] = l == 0.f ? NEG_INF : (m + __log2f(l)) * kLn2;
}

bool chunk_sizes(int T, int S, int H, int Hkv, int d, int max_pages, int page) {
  if (T < 1 || S < 1 || S > kMaxSeqs || max_pages < 1) return false;
  if (page < 16 || page > 1024 || (page & (page - 1))) return false;
  return valid_kv_heads(H, Hkv) && H / Hkv <= 128 && (d == 64 || d == 128) && static_cast<long long>(T) * H <= 0x7FFFFFFFll;
}

size_t chunk_workspace(int, int, int, int, int, int, int) { return 16; }

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
  attn_status_t s = check_common(S, H, T, 1, d, scale);
  if (s != ATTN_OK) return s;
  if (!valid_kv_heads(H, H_kv)) return ATTN_ERR_INVALID_ARG;
  if (max_pages < 1 || n_pages < 1) return ATTN_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) || S > kMaxSeqs)
    return ATTN_ERR_UNSUPPORTED;
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
  p.scale_log2 = scale * kLog2e;
  p.window = std::min<int64_t>(window, int64_t(1) << 60);
  p.sinks = static_cast<int>(std::min<int64_t>(sinks, 0x7FFFFFF0));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(T) * H + 3) / 4);
  if (d == 64) {
    if (fp8) attn_fwd_paged_kernel<64, true><<<grid, 128, 0, st>>>(p);
    else attn_fwd_paged_kernel<64, false><<<grid, 128, 0, st>>>(p);
  } else {
    if (fp8) attn_fwd_paged_kernel<128, true><<<grid, 128, 0, st>>>(p);
    else attn_fwd_paged_kernel<128, false><<<grid, 128, 0, st>>>(p);
  }
  return cuda_status("attn_fwd_paged launch", cudaGetLastError());
}
