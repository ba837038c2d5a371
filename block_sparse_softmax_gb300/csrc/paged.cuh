// What the calls over paged caches share: limits, checks and tensor maps of the
// host, copies and conversions of the device.
#pragma once
#include <algorithm>

#include "host.cuh"

namespace bss {

constexpr int kMaxSeqs = 65536;      // rows of a page table (the fork kernel keeps a bit for each)

inline bool valid_page_size(int page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// K or V pages as a 3-D tensor (d, H_kv * page_size, pages) with boxes of `box_rows`
// rows of a page and up to 128 bytes.
inline attn_status_t cache_map(CUtensorMap* map, const void* ptr, int d, bool fp8, long long rows, int P,
                               size_t page_bytes, int box_rows) {
  const int item = fp8 ? 1 : 2;
  const int box = std::min(d * item, 128);
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(rows), static_cast<uint64_t>(P)};
  const uint64_t strides[2] = {static_cast<uint64_t>(d) * item, page_bytes};
  const uint32_t boxes[3] = {static_cast<uint32_t>(box / item), static_cast<uint32_t>(box_rows), 1};
  return make_map_tiled(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr,
                        dims, strides, boxes, box == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                            int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Two e4m3 elements (the low 16 bits) as a pair of fp16, which holds them all.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t x) {
  uint32_t y;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace bss
