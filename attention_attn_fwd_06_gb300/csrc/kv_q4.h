// kv_q4.h -- layout of the 4-bit KV cache pool (host and device).
//
// Pool: [num_pages][Hkv][page_size / 16] tiles.  A tile holds 16 keys of one kv head, G = D / 64 groups of 64 dims:
//   K codes   [G][16 keys][32 bytes]     at 0
//   V codes   [G][16 keys][32 bytes]     at kv_q4_v_off
//   K params  [16 keys][G][2] fp16       at kv_q4_kp_off     (scale, minimum)
//   V params  [16 keys][G][2] fp16       at kv_q4_vp_off
// Byte j of a code row holds dims 2j (low four bits) and 2j + 1 of its group; code u stands for scale * u + minimum.
// K and V of 16 keys sit together so that one bulk copy brings both, a run of a page's tiles is one copy, and every
// tile starts on a 128-byte boundary (2304 bytes at D = 128, 1152 at D = 64).
#pragma once

#include <cstddef>

namespace attn {

constexpr int kTileKeys = 16;

__host__ __device__ constexpr int kv_q4_v_off(int D) { return 8 * D; }
__host__ __device__ constexpr int kv_q4_kp_off(int D) { return 16 * D; }
__host__ __device__ constexpr int kv_q4_vp_off(int D) { return 17 * D; }
__host__ __device__ constexpr int kv_q4_tile_bytes(int D) { return 18 * D; }

// First byte of tile `tile` of page `page`, kv head h (tpp = page_size / 16 tiles a page).
__host__ __device__ inline size_t kv_q4_tile_at(long long page, int h, int tile, int Hkv, int tpp, int D) {
  return (((size_t)page * Hkv + h) * tpp + tile) * (size_t)kv_q4_tile_bytes(D);
}

}  // namespace attn
