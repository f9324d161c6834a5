// What the two attention kernels over the 4-bit cache share (layout of the cache: kv4.cuh).
//
// Expansion, exact in fp16: a masked pair of nibbles in the mantissa of 1024 (0x6400) is
// 1024 + c (1024 + 16 c for the high nibbles), and one fused multiply-add gives
//   (1024 + c) (s / 16) - 64.5 s = (c - 8) s / 16;   (1024 + 16 c) (s / 256) - 4.5 s = the same
// s has 4 significant bits, so 64.5 s = 129 s / 2 needs 11 and the result 7: every term is
// an fp16 number for every e4m3 s.  That is 9 instructions for 8 elements.  The factor
// 16 g goes into the softmax scale (K) and into the output (V).
//
// Queries become fp16 scaled by a power of two per row (largest element in [2^14, 2^15)),
// undone in the row's softmax scale: exact but for elements below 2^-30 of the largest.
// Probabilities are rounded to fp16 (2^-11, a quarter of the output's own rounding in
// bf16); their reference sits 2^6 below the maximum it was taken from, so that fp16 reaches
// down to 2^-30 of it.  Maxima, sums and accumulators are fp32.
//
// The softmax takes a tile in one pass against the row references of the tiles before; only if
// some key lies 2^8 above its row's maximum then (always in an item's first tile) do the
// references move and O and the sums with them.  Row sums stay in the threads (each sums its
// own keys) until the item ends.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace dspark {
namespace attn {
namespace kv4a {

using namespace dspark::kv4;

constexpr int kKT = 128;               // keys of a tile
constexpr int kSmemItems = 16;         // work items of a CTA kept in shared memory
constexpr int kMaxCtas = 1024;         // the work list's limit
constexpr float kRefDrop = 6.f;        // reference = maximum - 6 (log2)
constexpr float kMove = 14.f;          // a key above reference + 14 moves it
constexpr float kNoRef = -1e30f;       // reference of a row that has seen no key
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

// A cache tile of the ring: its eight blocks, with 32 bytes of padding that put the blocks which a
// quad's four threads read at once in different banks.
constexpr int kBlockStride = kBlockBytes + 32;
constexpr int kBlocks = kKT / kBlock;
constexpr int kStageBytes = kBlocks * kBlockStride;

struct Params {
  const __nv_bfloat16 *q, *k_new, *v_new;
  const uint8_t* cache;
  const int32_t* page_table;
  const AttnItem* items;
  const int* item_begin;
  __nv_bfloat16* out;
  float *lse, *ws_o, *ws_lse;
  unsigned int* err;
  int Hq, Hkv, log2_page, max_pages, n_pages;
  int slot_rows;        // rows of a slot of ws_o and ws_lse
  float sl2;            // scale * log2(e) * 16 * k_scale
  float k_unit, v_unit; // 1 / (16 k_scale), 1 / (16 v_scale)
  float o_unit;         // 16 v_scale
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Wait on a barrier; bounded (the error is raised and the call goes on).
__device__ __forceinline__ void wait_bar(uint32_t bar, uint32_t parity, unsigned int* err) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (ptx::mbar_try_wait_sleep(bar, parity, 20000)) return;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait_sleep(bar, parity, 20000))
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      raise_error(err, DSPARK_DEVERR_WAIT_TIMEOUT);
      return;
    }
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c) {
  return h2_bits(__hfma2(bits_h2(a), bits_h2(b), bits_h2(c)));
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
  return h2_bits(__hmul2(bits_h2(a), bits_h2(b)));
}
// The expansion's constants as fp16 pairs: 1/16, 1/256, -64.5, -4.5.
constexpr uint32_t kSixteenth = 0x2c002c00u, k256th = 0x1c001c00u, kBiasLow = 0xd408d408u,
                   kBiasHigh = 0xc480c480u;
// Two e4m3 numbers in the low (high) half of a register as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3_low(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_high(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
// (w & MASK) | magic in one instruction (magic in a register: two immediates would take two).
template <uint32_t MASK>
__device__ __forceinline__ uint32_t masked(uint32_t w, uint32_t magic) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(magic));
  return r;
}
// Eight codes of a word -> four pairs (code - 8) s / 16: pair p with s[p], b[p] as the
// head of the file has them for even (low nibbles) and odd (high nibbles) p.
__device__ __forceinline__ void expand(uint32_t w, uint32_t magic, uint32_t s0, uint32_t b0,
                                       uint32_t s1, uint32_t b1, uint32_t s2, uint32_t b2,
                                       uint32_t s3, uint32_t b3, uint32_t (&o)[4]) {
  const uint32_t w8 = w >> 8;
  o[0] = hfma2_bits(masked<0x000f000fu>(w, magic), s0, b0);
  o[1] = hfma2_bits(masked<0x00f000f0u>(w, magic), s1, b1);
  o[2] = hfma2_bits(masked<0x000f000fu>(w8, magic), s2, b2);
  o[3] = hfma2_bits(masked<0x00f000f0u>(w8, magic), s3, b3);
}
// Two numbers in cache units as fp16, saturating (a NaN stays one).
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  const __half2 top = __half2half2(__ushort_as_half(0x7bff));  // 65504
  return h2_bits(__hmax2_nan(__hmin2_nan(__floats2half2_rn(a, b), top), __hneg2(top)));
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ AttnItem fetch_item(const AttnItem* s_items, const AttnItem* g_items,
                                               int it, int it_begin) {
  const int k = it - it_begin;
  return k < kSmemItems ? s_items[k] : g_items[it];
}

// The wide kernel (verify_attn_kv4_wide.cu): tiles of up to 32, 48 or 80 rows.
constexpr int kWideCtasPerSm = 2;
int launch_wide(const Params& p, int rows, int ncta, cudaStream_t stream);

}  // namespace kv4a
}  // namespace attn
}  // namespace dspark
