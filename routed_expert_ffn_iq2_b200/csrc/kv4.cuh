// kv4.cuh -- the stored form of the 4-bit key/value cache.
//
// A cache is n_pages pages of page_size tokens (a multiple of 16).  A page
// holds, per key/value head, page_size / 16 tiles of 16 tokens; a tile of
// head width D is 20 D bytes.  Values go in groups of 32 along the head:
// value = m + d * code, code 0..15, d and m in fp16.  With NG = D / 32:
//   at 0      key codes, 8 D bytes
//   at 8 D    key steps [16][NG] of {d, m}
//   at 10 D   value codes, 8 D bytes
//   at 18 D   value steps d [16][NG];  at 19 D value minima m [16][NG]
// Code planes are in the order in which a warp's lanes feed them to the
// tensor cores, so that lane l's 16 bytes lie at 16 l of a 512-byte row:
//   keys    token t = 8 h + r, group g, quarter c (values 8 c .. 8 c + 7 of
//           the group, value e at nibble e of one 32-bit word): word
//           (y >> 2) * 128 + (4 r + c) * 4 + (y & 3), y = h NG + g;
//   values  token t = 8 h + 2 c + b, group j, eighth r (values 4 r .. 4 r + 3
//           at the nibbles of one 16-bit unit): unit
//           (x >> 3) * 256 + (4 r + c) * 8 + (x & 7), x = (2 h + b) NG + j.
#pragma once

#include "mixer.cuh"

namespace redlite {

inline bool kv4_shape_ok(int32_t head_dim, int32_t page_size) {
  return (head_dim == 128 || head_dim == 256) && page_size >= 16 && page_size <= 4096 && page_size % 16 == 0;
}

template <int D>
__host__ __device__ __forceinline__ int64_t kv4_tile_offset(int64_t page, int n_heads, int head, int page_size,
                                                            int tile) {
  return ((page * n_heads + head) * (page_size / 16) + tile) * (20 * D);
}
template <int D>
__device__ __forceinline__ int kv4_k_word(int t, int g, int c) {
  const int y = (t >> 3) * (D / 32) + g;
  return 4 * ((y >> 2) * 128 + (4 * (t & 7) + c) * 4 + (y & 3));
}
template <int D>
__device__ __forceinline__ int kv4_k_step(int t, int g) {
  return 8 * D + 4 * (t * (D / 32) + g);
}
template <int D>
__device__ __forceinline__ int kv4_v_unit(int t, int j, int r) {
  const int x = (2 * (t >> 3) + (t & 1)) * (D / 32) + j;
  return 10 * D + 2 * ((x >> 3) * 256 + (4 * r + ((t & 7) >> 1)) * 8 + (x & 7));
}
template <int D>
__device__ __forceinline__ int kv4_v_step(int t, int j) {
  return 18 * D + 2 * (t * (D / 32) + j);
}
template <int D>
__device__ __forceinline__ int kv4_v_min(int t, int j) {
  return 19 * D + 2 * (t * (D / 32) + j);
}

}  // namespace redlite
