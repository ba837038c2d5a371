// Host-side helpers shared by the files that define C entry points (defined in
// api.cu): argument checks, the per-device status word, tensor-map encoding
// and the thread's error text.
#pragma once
#include "common.cuh"

namespace bss {

// Device address of the kernels' status word on the current device.
attn_status_t status_word(int** out);
// Looks up the driver's tensor-map encoder; make_map needs it.
attn_status_t get_encoder();
// [B, H, L, d] bf16 contiguous as a 4-D tensor map with boxes of 64 x 128.
attn_status_t make_map(CUtensorMap* map, const void* ptr, int B, int H, long long L, int d);
// The fp32 dQ accumulator [B, H, L, d] with boxes of 32 x box_rows.
attn_status_t make_map_f32(CUtensorMap* map, void* ptr, int B, int H, long long L, int d,
                           int box_rows);
// A tiled tensor map of any rank with unit element strides and zero fill.
attn_status_t make_map_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* ptr,
                             const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                             CUtensorMapSwizzle swizzle);
attn_status_t check_common(int B, int H, long long Lq, long long Lk, int d, float scale);
attn_status_t cuda_status(const char* where, cudaError_t e);
// K/V heads: 1 <= Hkv <= H and Hkv divides H.
bool valid_kv_heads(int H, int Hkv);
// Events of attn_bwd_time_main (both nullptr when off).
void bwd_main_events(cudaEvent_t* begin, cudaEvent_t* end);

// Rows of a windowed call, tokens of a sequence in a paged cache: a tile past
// the last one still counts in 32 bits.
constexpr int kMaxTokens = 0x7FFFFF00;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace bss
