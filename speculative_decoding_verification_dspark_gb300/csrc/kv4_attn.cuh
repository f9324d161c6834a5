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
// Probabilities are rounded to fp16 (2^-11, an eighth of the output's own rounding in
// bf16); their reference sits 2^6 below the maximum it was taken from, so that fp16 reaches
// down to 2^-30 of it.  Maxima, sums and accumulators are fp32.
//
// A NaN in v_new reaches the rows that see it and no others: see pack16_value.
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
// Largest context and segment together.  Each fills tiles of its own, and the lanes of a copying
// warp form positions up to 31 blocks past the start of the last tile, 622 past this end at most.
constexpr long long kMaxEnd = 0x7fffffffll - 6 * kKT;
constexpr int kMaxCtas = 1024;         // (own_items: products of a unit and a CTA in 32 bits)
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
  const int32_t *ctx_len, *cu_seqlens;
  AttnItem* items;      // work items past the first of each CTA (own_items)
  SplitGroup* groups;   // the split group that ends in each CTA
  __nv_bfloat16* out;
  float *lse, *ws_o, *ws_lse;
  unsigned int* err;
  int Hq, Hkv, log2_page, max_pages, n_pages;
  int B, max_rows, rows_per_tile, max_splits;
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
// The same for the values of block rows, every number finite: a NaN stands in the operand as a
// number (the rows that do not see it weigh it 0, which times NaN is NaN) and is kept in `nan`, a
// pair that has_nan tells; write_nans gives it to the rows that see it.
__device__ __forceinline__ uint32_t pack16_value(float a, float b, uint32_t& nan) {
  const __half2 top = __half2half2(__ushort_as_half(0x7bff));
  const __half2 t = __hmin2_nan(__floats2half2_rn(a, b), top);
  nan = h2_bits(__hmax2_nan(bits_h2(nan), t));
  return h2_bits(__hmax2(t, __hneg2(top)));
}
__device__ __forceinline__ bool has_nan(uint32_t pair) {
  return ((pair & 0x7fffu) > 0x7c00u) || ((pair & 0x7fff0000u) > 0x7c000000u);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// ---------------------------------------------------------------- work items
// The key tiles of every (request, row tile, KV head) group are laid end to end (U units) and
// CTA c of n takes units [c U / n, (c + 1) U / n), the same number for each, as the bf16
// cache's kernels do with a list that a kernel of one CTA builds; here each CTA finds its own
// items, which costs it 2 to 3 us in place of that kernel's 5 to 14 (its time grows with the
// groups) and one launch.  A group cut by CTA boundaries becomes pieces, at most max_splits; a
// piece is the first or the last of its CTA and goes to slot 2 c or 2 c + 1; the CTA of a group's
// last piece records the group for the merge.
struct OwnItems {
  int n;                  // items of this CTA
  const AttnItem* more;   // all of them, if n > kSmemItems
};
struct ItemScratch {
  long long off[DSPARK_MAX_B + 1];  // first unit of request r
  int goff[DSPARK_MAX_B + 1];       // first group
  int tt[DSPARK_MAX_B];             // tiles of a group
  long long w_units[32];
  int w_groups[32], w_tmax[32];
};

// Largest r in [a, b) with off[r] <= x (off non-decreasing, off[a] <= x).
template <typename T>
__device__ __forceinline__ int last_le(const T* off, int a, int b, T x) {
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (off[mid] <= x) a = mid; else b = mid;
  }
  return a;
}

// By the whole CTA of THREADS; ends with a barrier behind which the scratch is free.
template <int THREADS>
__device__ __forceinline__ OwnItems own_items(const Params& p, ItemScratch& S, AttnItem* s_items) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, c = blockIdx.x;
  const int B = p.B, rpt = p.rows_per_tile;
  // (with the last row no less than 0, as here, and the others no less than 0, as below, n does not
  // pass 32 bits)
  const bool rows_ok = (unsigned)p.cu_seqlens[B] <= (unsigned)p.max_rows;
  // this thread's requests
  const int per = (B + THREADS - 1) / THREADS, r_begin = tid * per, r_end = min(B, r_begin + per);
  long long units = 0;
  int groups = 0, tmax = 0;
  // a length or a first row below zero, or a segment whose end lies past kMaxEnd: no shares can be
  // made of it
  bool bad = false;
  for (int r = r_begin; r < r_end; ++r) {
    const int c0 = p.cu_seqlens[r], n = p.cu_seqlens[r + 1] - c0, ctx = p.ctx_len[r];
    bad |= c0 < 0 || n < 0 || ctx < 0 || (long long)ctx + n > kMaxEnd;
    const int t = ceil_div(ctx, kKT) + ceil_div(n, kKT), ng = ceil_div(n, rpt) * p.Hkv;
    S.tt[r] = t;
    S.goff[r] = ng;
    units += (long long)t * ng;
    groups += ng;
    if (ng > 0) tmax = max(tmax, t);
  }
  long long u_incl = units;
  int g_incl = groups;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, u_incl, o);
    const int g = __shfl_up_sync(0xffffffffu, g_incl, o);
    if (lane >= o) {
      u_incl += u;
      g_incl += g;
    }
    tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, o));
  }
  if (lane == 31) {
    S.w_units[wid] = u_incl;
    S.w_groups[wid] = g_incl;
    S.w_tmax[wid] = tmax;
  }
  bad = __syncthreads_or(bad);
  long long U = 0, u0 = u_incl - units;
  int g0 = g_incl - groups;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < wid) {
      u0 += S.w_units[i];
      g0 += S.w_groups[i];
    }
    U += S.w_units[i];
    tmax = max(tmax, S.w_tmax[i]);
  }
  for (int r = r_begin; r < r_end; ++r) {
    const int ng = S.goff[r];
    S.off[r] = u0;
    S.goff[r] = g0;
    u0 += (long long)S.tt[r] * ng;
    g0 += ng;
  }
  __syncthreads();
  // No group in more than max_splits pieces: every range holds L = floor(U / n) units, and a group
  // of T meets at most ceil((T - 1) / L) + 1 ranges, so L >= ceil((T - 1) / (max_splits - 1)).
  const bool small = U < (1 << 20);  // (with 1024 CTAs all products fit 32 bits)
  const unsigned l_req = max(1u, (unsigned)(tmax - 1 + p.max_splits - 2) / (unsigned)(p.max_splits - 1));
  long long n_max = small ? (unsigned)U / l_req : U / l_req;
  const int n_cta = (int)max(1ll, min(n_max, (long long)gridDim.x));
  auto first_unit = [&](int cc) -> long long {
    return small ? (unsigned)cc * (unsigned)U / (unsigned)n_cta : (long long)cc * U / n_cta;
  };
  OwnItems own{0, nullptr};
  const bool active = rows_ok && !bad && U > 0 && c < n_cta;
  if (c == 0 && tid == 0 && !rows_ok) raise_error(p.err, DSPARK_DEVERR_ROWS_OVERFLOW);
  if (c == 0 && tid == 0 && bad) raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
  SplitGroup record{};
  if (active) {
    const long long lo = first_unit(c), hi = first_unit(c + 1);
    const int r0 = last_le(S.off, 0, B, lo), r1 = last_le(S.off, r0, B, hi - 1);
    const long long d0 = lo - S.off[r0], d1 = hi - 1 - S.off[r1];
    const int gf = S.goff[r0] + (int)(small ? (unsigned)d0 / (unsigned)S.tt[r0] : d0 / S.tt[r0]);
    const int gl = S.goff[r1] + (int)(small ? (unsigned)d1 / (unsigned)S.tt[r1] : d1 / S.tt[r1]);
    // the CTA of unit x: the largest cc with cc U / n_cta <= x
    auto cta_of = [&](long long x) -> int {
      return small ? (int)(((unsigned)(x + 1) * (unsigned)n_cta - 1) / (unsigned)U)
                   : (int)(((x + 1) * n_cta - 1) / U);
    };
    own.n = gl - gf + 1;
    // (items of earlier CTAs number gf + c at most)
    AttnItem* const list = p.items + gf + c;
    own.more = list;
    for (int i = tid; i < own.n; i += THREADS) {
      const int g = gf + i, r = last_le(S.goff, r0, r1 + 1, g);
      const int lg = g - S.goff[r], t = lg / p.Hkv, t_r = S.tt[r];
      const long long gs = S.off[r] + (long long)lg * t_r, ge = gs + t_r;
      const long long a = max(gs, lo), b = min(ge, hi);
      const int c_first = gs < lo ? cta_of(gs) : c, c_last = ge > hi ? cta_of(ge - 1) : c;
      AttnItem x;
      x.c0 = p.cu_seqlens[r];
      x.n_r = p.cu_seqlens[r + 1] - x.c0;
      x.ctx = p.ctx_len[r];
      x.r = r; x.kvh = lg - t * p.Hkv; x.i0 = t * rpt; x.ni = min(rpt, x.n_r - x.i0);
      x.part = 0; x.split = c - c_first;
      x.tb = (int)(a - gs); x.te = (int)(b - gs);
      x.nsplit = c_last - c_first + 1;
      x.slot = a == lo ? 2 * c : 2 * c + 1;
      x.pad0 = x.pad1 = x.pad2 = 0;
      if (i < kSmemItems) s_items[i] = x;
      if (own.n > kSmemItems) list[i] = x;
      if (i == 0 && gs < lo && ge <= hi) {  // a split group that ends here
        record.r = r; record.kvh = x.kvh; record.part = 0; record.i0 = x.i0;
        record.ni = x.ni; record.c_first = c_first; record.nsplit = x.nsplit;
        record.slot0_last = gs != first_unit(c_first);
      }
    }
  }
  if (tid == 0) p.groups[c] = record;  // (nsplit 0: none)
  ptx::fence_proxy_async_smem();  // (bulk copies land where the scratch is)
  __syncthreads();
  return own;
}

__device__ __forceinline__ AttnItem fetch_item(const AttnItem* s_items, const AttnItem* more, int it) {
  return it < kSmemItems ? s_items[it] : more[it];
}

// After the outputs of rows n0 .. n1 - 1 of an item's tile, in channel ch: NaN for the rows that see
// a NaN of that channel in the block rows of the item's tiles (row n sees block row b from
// n = (b - i0) G on).  For the warp that wrote those outputs, where it met a NaN.
__device__ __forceinline__ void write_nans(const Params& p, const AttnItem& x, int ch, int n0, int n1) {
  const int G = p.Hq / p.Hkv, ct = ceil_div(x.ctx, kKT);
  const long long step = (long long)p.Hkv * kD;
  const __nv_bfloat16* v = p.v_new + ((long long)x.c0 * p.Hkv + x.kvh) * kD + ch;
  int b = max(x.tb - ct, 0) * kKT;
  const int end = min((x.te - ct) * kKT, x.n_r);
#pragma unroll 1
  while (b < end && !__hisnan(v[b * step])) ++b;
  if (b >= end) return;
#pragma unroll 1
  for (int n = max((b - x.i0) * G, n0); n < n1; ++n) {
    if (x.nsplit > 1)
      p.ws_o[((long long)x.slot * p.slot_rows + n) * kD + ch] = __int_as_float(0x7fffffff);
    else
      p.out[(((long long)x.c0 + x.i0 + n / G) * p.Hq + x.kvh * G + n % G) * kD + ch] =
          __ushort_as_bfloat16(0x7fff);
  }
}

// The wide kernel (verify_attn_kv4_wide.cu): tiles of up to 32, 48 or 64 rows.
constexpr int kWideCtasPerSm = 2;
int launch_wide(const Params& p, int rows, int ncta, cudaStream_t stream);

}  // namespace kv4a
}  // namespace attn
}  // namespace dspark
