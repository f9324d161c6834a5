// The 4-bit paged KV cache: layout of one block and the quantisation rule.
//
// A page holds, for each KV head, page_size / 16 blocks of 2176 bytes; a block is 16
// consecutive tokens of one head:
//   bytes    0 .. 1023  K codes  [4 groups of 32 dims][16 tokens][16 B]
//   bytes 1024 .. 2047  V codes  [128 channels][8 B = 16 tokens]
//   bytes 2048 .. 2111  K scales e4m3 [16 tokens][4 groups]
//   bytes 2112 .. 2175  V scales e4m3 [4 groups][16 tokens]
// In every 32-bit word of codes, nibble p holds element 2p and nibble p + 4 element
// 2p + 1 of eight consecutive ones (dims of a token for K, tokens of a channel for V):
// masking the word, or the word shifted by 8, with 0x000f000f or 0x00f000f0 then gives a
// pair of neighbours in the two halves of a register.
//   value = (code - 8) * scale * g,   one fp32 factor g per tensor (K, V)
// K lies along a token and V along a channel because that is how the attention's tensor-
// core operands take them: a lane of K is a key, a lane of V^T a channel, and either is
// expanded by the thread that reads it.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace dspark {
namespace kv4 {

constexpr int kD = 128;
constexpr int kBlock = 16;          // tokens of a block
constexpr int kBlockBytes = 2176;
constexpr int kOffV = 1024;
constexpr int kOffKs = 2048;
constexpr int kOffVs = 2112;

__device__ __forceinline__ float e4m3_to_float(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return static_cast<float>(v);
}

// The smallest e4m3 number >= t for t >= 0 (448, the largest, above it), as its code:
// rounding the scale up keeps every element of the group within 7 steps.
__device__ __forceinline__ uint8_t e4m3_at_least(float t) {
  uint8_t c = __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
  if (c < 0x7e && e4m3_to_float(c) < t) ++c;
  return c;
}

// Code of x in a group of step sg = scale * g: 8 + x / sg rounded to the nearest
// integer (ties to even) and clamped to +-7.  A NaN and every element of a group whose
// step is 0 become 8 (value 0); infinities saturate.
__device__ __forceinline__ uint32_t code_of(float x, float sg) {
  if (!(sg > 0.f)) return 8u;
  const float q = rintf(__fdiv_rn(x, sg));
  return q != q ? 8u : static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(q, -7.f), 7.f)) + 8);
}

// Nibble of element e (0..7) of a word.
__host__ __device__ constexpr int nibble_of(int e) { return (e >> 1) + ((e & 1) << 2); }

}  // namespace kv4
}  // namespace dspark
