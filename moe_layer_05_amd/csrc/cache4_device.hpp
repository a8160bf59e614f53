// The paged cache of keys and values in 4 bits: its layout and its codes.
//
// A group of 32 consecutive features of one token's head shares a power of
// two 2^e (stored as the byte e + 127), and each feature is an E2M1 code
// (sign, 2 exponent and 1 mantissa bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times
// 2^e: 4.25 bits a value.  e is the smallest that brings the group's largest
// magnitude to at most 7: 7 rounds to 6, the largest code, and nothing is off
// by more than half a step of the grid's top interval; over normal values
// the mean squared error is 6% below that of the largest code's own binade
// (amax < 8, which clips 7..8 to 6) and that of never exceeding 6.  A value
// read back is exact in bfloat16.  A group with an infinity or a NaN gets the
// byte 255 and reads back as NaN.
//
// [page][kv head][tile of 16 tokens], a tile of 17 * D bytes:
//   K codes  [16 tokens][D / 2], feature 2i in the low half of byte i
//   K scales [16 tokens][D / 32]
//   V codes  for each 128 features f: [4 quads of tokens][16 n][4 tokens][4]
//            (features f + 8n .. f + 8n + 7), for a last 64 features f:
//            [4 quads][16 n][4 tokens][2] (features f + 4n .. f + 4n + 3)
//   V scales [4 quads][D / 32][4 tokens]
// This is the order in which a wave's matrix operands take them: K codes as
// the rows of K Q^T (lane = token, 32 features in 16 bytes), V codes as the
// rows of V^T P^T (lane = features, 4 tokens in 16 bytes).
#pragma once

#include "device_common.hpp"
#include "internal.hpp"

namespace moe {

constexpr int kTileTokens = 16;

__host__ __device__ constexpr int cache4_tile_bytes(int D) { return 17 * D; }
__host__ __device__ constexpr int cache4_k_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int cache4_v_codes(int D) { return 8 * D + D / 2; }
__host__ __device__ constexpr int cache4_v_scales(int D) { return 16 * D + D / 2; }

// The tile of a place in a page, for a page id that has been checked.
__device__ __forceinline__ uint8_t* cache4_tile(const Cache4& c, int page, int h, int tile) {
  return c.pages +
         (((int64_t)page * c.NKV + h) * c.page_tiles + tile) * cache4_tile_bytes(c.D);
}

// Byte e + 127 of a group with this largest magnitude (of float bits), 255
// if it is not finite.  amax <= 7 * 2^e: 7 = 1.75 * 2^2, so e is the exponent
// of amax less 2, one more when its mantissa is above 1.75 -- a carry of the
// addition below.
__device__ __forceinline__ uint32_t cache4_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const int b = (int)((amax_bits + 0x1FFFFFu) >> 23) - 2;
  return (uint32_t)(b < 2 ? 2 : (b > 252 ? 252 : b));
}

__device__ __forceinline__ float cache4_scale(uint32_t byte) {
  return __uint_as_float(byte << 23);
}

// Eight E2M1 codes of v / scale (a power of two), nearest even, saturating.
__device__ __forceinline__ uint32_t fp4_pack8(const float (&v)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return w;
}

// Two bfloat16 of byte BYTE of a word of codes; a scale whose exponent bits
// are all ones gives NaN.
template <int BYTE>
__device__ __forceinline__ uint32_t fp4_pair(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, BYTE));
}

// The eight values of a word of codes.
__device__ __forceinline__ uint4 fp4_unpack8(uint32_t codes, float scale) {
  return make_uint4(fp4_pair<0>(codes, scale), fp4_pair<1>(codes, scale),
                    fp4_pair<2>(codes, scale), fp4_pair<3>(codes, scale));
}

}  // namespace moe
