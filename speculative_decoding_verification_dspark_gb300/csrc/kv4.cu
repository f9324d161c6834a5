// Rows into and out of the 4-bit paged KV cache (layout: kv4.cuh).
//
//   kv4_store_kernel  quantises packed rows into the blocks of their requests' pages
//   kv4_load_kernel   expands committed positions back to packed rows
//
// A byte of V codes holds two tokens of a channel, so a block that is appended to is
// read, changed and written: one CTA owns a (request, 16-token block, head), found from
// the first packed row that falls into it ("leader"), and handles all rows of it.  So no
// two CTAs touch the same bytes, and tokens of the block that are not among the rows
// keep their codes.
//
// A block of a head is six tasks of a warp, which share nothing: K's 4 x 4 tokens (a
// token on eight lanes, 16 dims each: a group of 32 is two lanes) and V's 2 x 64 channels
// (two channels per lane and all 16 tokens, so that a lane holds whole words of codes and
// nothing is transposed; a group is a half-warp).  Every warp finds the leaders of the
// CTA's rows by itself, so the kernels have no barrier.
//
// Prompts (65536 rows of 8 heads, bf16): store 82 us, bound by instruction issue (16 per
// element and lane, 0.60 a cycle; 36 warps per SM by registers, 30 take 88 us), load 58 us,
// 86% of the copy rate.  Reading the next pair's rows ahead cost more warps than it gave (134
// us).  A commit of 32 requests is latency: a search of cu_seqlens, the page, the row or the
// old codes, 4.7 us a kernel (5.1 when what follows is launched early and takes its places).
//
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace dspark {

namespace {

using namespace kv4;

constexpr int kTasks = 6;      // warps of a CTA, and tasks of a block
constexpr int kThreads = 32 * kTasks;
constexpr int kWindow = 16;    // packed rows whose leaders one CTA serves, at most

// The largest r < B with cu[r] <= row, 0 if there is none (cu ascending): a warp narrows
// the range by 32 per round.
__device__ __forceinline__ int find_request(const int32_t* __restrict__ cu, int B, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < n && cu[lo + at] <= row);
    const int k = 31 - __clz(m | 1u);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

struct Kv4Params {
  const int32_t *cu, *pos0, *keep, *page_table;
  const int* ok;  // nullable: nothing is done unless it is set
  unsigned int* err;
  int B, max_rows, Hkv, log2_page, max_pages, n_pages, rows_per_cta, heads_per_cta;
  float gk, gv;
};

// Whether the packed rows cu[0] .. M - 1 lie in the buffers.
__device__ __forceinline__ bool rows_ok(const Kv4Params& p, int M) {
  const int first = p.cu[0];
  if (M <= p.max_rows && first >= 0) return true;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    raise_error(p.err, M > p.max_rows ? DSPARK_DEVERR_ROWS_OVERFLOW : DSPARK_DEVERR_BAD_INPUT);
  return false;
}

// The leaders of a window of packed rows: lane j < 16 holds row row0 + j.
struct Leaders {
  int r, pos, cnt;   // request, cache position and rows in the block (lanes of `mask`)
  long long base;    // index of the block of head 0 (a head further: `per` blocks), -1: no valid page
  unsigned mask;     // lanes whose row is a leader
};

// keep: rows 0 .. keep[r] of a segment take part (nullable: all).  Rows before cu[0] are no
// request's (i < 0: find_request gives them to request 0).
__device__ __forceinline__ Leaders find_leaders(const Kv4Params& p, int row0, int M) {
  const int lane = threadIdx.x & 31, row = row0 + lane;
  Leaders a{0, 0, 0, -1, 0};
  int r = find_request(p.cu, p.B, row0);
  bool leader = false;
  if (lane < p.rows_per_cta && row < M) {
    // the window may run into further requests
    for (int hi = p.B; hi - r > 1 && p.cu[r + 1] <= row;) {  // cu[r] <= row < cu[hi]
      const int mid = (r + hi) >> 1;
      if (p.cu[mid] <= row) r = mid; else hi = mid;
    }
    const int c0 = p.cu[r], i = row - c0;
    int n = min(p.cu[r + 1], M) - c0;
    if (p.keep) n = min(n, max(p.keep[r], 0) + 1);
    a.r = r;
    a.pos = p.pos0[r] + i;
    const int t0 = a.pos & (kBlock - 1);
    leader = i >= 0 && i < n && (i == 0 || t0 == 0);
    if (leader) {
      a.cnt = min(kBlock - t0, n - i);
      const int slot = a.pos >> p.log2_page;
      const int page = a.pos >= 0 && slot < p.max_pages
                           ? p.page_table[(long long)r * p.max_pages + slot] : -1;
      const int per = 1 << (p.log2_page - 4);
      if ((unsigned)page < (unsigned)p.n_pages)
        a.base = (long long)page * p.Hkv * per + ((a.pos >> 4) & (per - 1));
      else
        raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
    }
  }
  a.mask = __ballot_sync(0xffffffffu, leader && a.base >= 0);
  return a;
}

// The maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A group's scale code, step sg and 1 / sg.  `plain`: the step is well inside fp32's range, all
// elements are finite and within 7 steps, and code_pair gives code_of's codes.
struct Step {
  uint8_t code;
  bool plain;
  float neg, inv;  // -sg, 1 / sg
};
__device__ __forceinline__ Step step_of(float amax, float g) {
  Step s;
  s.code = e4m3_at_least(__fdiv_rn(amax, __fmul_rn(7.f, g)));
  const float sg = __fmul_rn(e4m3_to_float(s.code), g);
  s.plain = s.code < 0x7e && sg > 0x1p-60f && sg < 0x1p60f && amax < INFINITY;  // (a NaN fails)
  s.neg = -sg;
  s.inv = __frcp_rn(sg);
  return s;
}
// 8 + rint(x / sg) of two elements, each in the low bits of kCodeBase + code.  The quotient is the
// correctly rounded one, from the correctly rounded reciprocal by two of Markstein's
// corrections q + (x - q sg) / sg (IBM J. Res. Dev. 34, 1990): the first leaves q within an
// ulp, the second rounds it as the division does.  Adding 1.5 2^23 + 8 rounds to an
// integer, ties to even.
constexpr uint32_t kCodeBase = 0x4b400000u;
__device__ __forceinline__ void code_pair(uint64_t x, uint64_t neg, uint64_t inv, uint32_t& c0, uint32_t& c1) {
  uint64_t q = mul2(x, inv);
  q = fma2(fma2(q, neg, x), inv, q);
  q = fma2(fma2(q, neg, x), inv, q);
  q = add2(q, pair(12582920.f, 12582920.f));
  c0 = (uint32_t)q;
  c1 = (uint32_t)(q >> 32);
}
// What eight times kCodeBase, each at its nibble, add up to in a word.
constexpr uint32_t word_base() {
  uint32_t s = 0;
  for (int e = 0; e < 8; ++e) s += kCodeBase << (4 * e);
  return s;
}

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[16]) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = a.z; x[4 * i + 3] = a.w;
  }
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]);
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
template <>
__device__ __forceinline__ void store16<float>(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}

// Two neighbours of a row, as they are read.
template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  uint32_t w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void zero() { w = 0; }
  __device__ __forceinline__ float2 get() const {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  // the two magnitudes, their maximum with others (a NaN stays), and the larger one at the end
  using Mag = uint32_t;
  __device__ __forceinline__ Mag mag() const { return w & 0x7fff7fffu; }
  static __device__ __forceinline__ Mag larger(Mag a, Mag b) {
    const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
  static __device__ __forceinline__ float top(Mag a) {
    return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
};
template <>
struct Two<float> {
  float2 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
  __device__ __forceinline__ float2 get() const { return v; }
  using Mag = float;
  __device__ __forceinline__ Mag mag() const { return max_nan(fabsf(v.x), fabsf(v.y)); }
  static __device__ __forceinline__ Mag larger(Mag a, Mag b) { return max_nan(a, b); }
  static __device__ __forceinline__ float top(Mag a) { return a; }
};
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void store2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

// Four tokens of K: token tok = 4 part + lane / 8, dims 16 (lane % 8) .. + 15.  `src`: the row of
// the block's first token t0.
template <typename T>
__device__ __forceinline__ void store_k(const T* src, long long stride, uint8_t* blk, int part, int t0,
                                        int cnt, float g) {
  const int lane = threadIdx.x & 31, tok = 4 * part + (lane >> 3), seg = lane & 7;
  const bool live = tok >= t0 && tok < t0 + cnt;
  if (!__any_sync(0xffffffffu, live)) return;
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = 0.f;
  if (live) load16(src + (tok - t0) * stride + seg * 16, x);
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) amax = max_nan(amax, fabsf(x[e]));
  amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  if (!live) return;
  Step st = step_of(amax, g);
  uint32_t w[2] = {0, 0};
  if (st.plain) {
    const uint64_t neg = pair(st.neg, st.neg), inv = pair(st.inv, st.inv);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      uint32_t c0, c1;
      code_pair(pair(x[e], x[e + 1]), neg, inv, c0, c1);
      w[e >> 3] += (c0 << (4 * nibble_of(e & 7))) + (c1 << (4 * nibble_of((e + 1) & 7)));
    }
    w[0] -= word_base();
    w[1] -= word_base();
  } else {  // (the other lane of the group is here too)
    amax = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));  // (drops a NaN)
    amax = fmaxf(amax, __shfl_xor_sync(3u << (lane & 30), amax, 1));
    st = step_of(amax, g);
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e >> 3] |= code_of(x[e], -st.neg) << (4 * nibble_of(e & 7));
  }
  *reinterpret_cast<uint2*>(blk + (seg >> 1) * 256 + tok * 16 + (seg & 1) * 8) = make_uint2(w[0], w[1]);
  if (!(seg & 1)) blk[kOffKs + tok * 4 + (seg >> 1)] = st.code;
}

// 64 channels of V: channels c = 64 part + 2 lane, c + 1, all tokens.
template <typename T>
__device__ __forceinline__ void store_v(const T* src, long long stride, uint8_t* blk, int part, int t0,
                                        int cnt, float g, float4 (*s_step)[kBlock]) {
  const int lane = threadIdx.x & 31, c = 64 * part + 2 * lane, tok = lane & 15;
  src += c;
  Two<T> x[kBlock];
  if (cnt == kBlock) {
#pragma unroll
    for (int e = 0; e < kBlock; ++e) x[e].load(src + e * stride);
  } else {
#pragma unroll
    for (int e = 0; e < kBlock; ++e) {
      x[e].zero();
      if (e >= t0 && e < t0 + cnt) x[e].load(src + (e - t0) * stride);
    }
  }
  // the maxima over the half-warp, token `tok` to this lane
  typename Two<T>::Mag a[kBlock];
#pragma unroll
  for (int e = 0; e < kBlock; ++e) a[e] = x[e].mag();
#pragma unroll
  for (int o = kBlock / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int e = 0; e < o; ++e)
      a[e] = Two<T>::larger(up ? a[e + o] : a[e], __shfl_xor_sync(0xffffffffu, up ? a[e] : a[e + o], o));
  }
  const bool live = tok >= t0 && tok < t0 + cnt;
  const Step st = step_of(Two<T>::top(a[0]), g);
  uint8_t* const scales = blk + kOffVs + (c >> 5) * kBlock;
  uint32_t w[2][2] = {{0, 0}, {0, 0}};
  if (__all_sync(0xffffffffu, st.plain || !live)) {
    if (live) scales[tok] = st.code;
    float4* const steps = s_step[lane >> 4];
    // (a step of 1 for tokens without a row, whose codes are then 8)
    steps[tok] = live ? make_float4(st.neg, st.neg, st.inv, st.inv) : make_float4(-1.f, -1.f, 1.f, 1.f);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < kBlock; ++e) {
      const float4 s = steps[e];
      const float2 y = x[e].get();
      uint32_t c0, c1;
      code_pair(pair(y.x, y.y), pair(s.x, s.y), pair(s.z, s.w), c0, c1);
      w[0][e >> 3] += c0 << (4 * nibble_of(e & 7));
      w[1][e >> 3] += c1 << (4 * nibble_of(e & 7));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i][0] -= word_base();
      w[i][1] -= word_base();
    }
  } else {
#pragma unroll 1
    for (int e = t0; e < t0 + cnt; ++e) {
      Two<T> z;
      z.load(src + (e - t0) * stride);
      const float2 y = z.get();
      float amax = fmaxf(fmaxf(0.f, fabsf(y.x)), fabsf(y.y));  // (drops a NaN)
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const Step se = step_of(amax, g);
      if (tok == e) scales[e] = se.code;
      const int at = 4 * nibble_of(e & 7);
      const uint32_t c0 = code_of(y.x, -se.neg) << at, c1 = code_of(y.y, -se.neg) << at;
      w[0][0] |= e < 8 ? c0 : 0;
      w[0][1] |= e < 8 ? 0 : c0;
      w[1][0] |= e < 8 ? c1 : 0;
      w[1][1] |= e < 8 ? 0 : c1;
    }
  }
  uint4* const dst = reinterpret_cast<uint4*>(blk + kOffV + c * 8);
  if (cnt < kBlock) {  // tokens of the block that are not among the rows stay
    uint32_t m[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < kBlock; ++e)
      if (e >= t0 && e < t0 + cnt) m[e >> 3] |= 0xfu << (4 * nibble_of(e & 7));
    const uint4 old = *dst;
    w[0][0] = (w[0][0] & m[0]) | (old.x & ~m[0]);
    w[0][1] = (w[0][1] & m[1]) | (old.y & ~m[1]);
    w[1][0] = (w[1][0] & m[0]) | (old.z & ~m[0]);
    w[1][1] = (w[1][1] & m[1]) | (old.w & ~m[1]);
  }
  *dst = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
}

// (code - 8) * s * g of the pair of codes at nibbles n and n + 4 of a word.
__device__ __forceinline__ float2 value_pair(uint32_t w, int n, uint64_t s, uint64_t g) {
  const uint32_t h = ((w >> (4 * n)) & 0x000f000fu) | 0x64006400u;  // 1024 + code, as fp16
  const float2 c = __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(1032.f)));
  const uint64_t v = mul2(mul2(pair(c.x, c.y), s), g);
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}

template <typename T>
__device__ __forceinline__ void load_k(T* dst, long long stride, const uint8_t* blk, int part, int t0,
                                       int cnt, float g) {
  const int lane = threadIdx.x & 31, tok = 4 * part + (lane >> 3), seg = lane & 7;
  if (tok < t0 || tok >= t0 + cnt) return;
  const uint2 v = *reinterpret_cast<const uint2*>(blk + (seg >> 1) * 256 + tok * 16 + (seg & 1) * 8);
  const float s = e4m3_to_float(blk[kOffKs + tok * 4 + (seg >> 1)]);
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const float2 y = value_pair(e < 8 ? v.x : v.y, (e & 7) >> 1, pair(s, s), pair(g, g));
    x[e] = y.x;
    x[e + 1] = y.y;
  }
  store16(dst + (tok - t0) * stride + seg * 16, x);
}

template <typename T>
__device__ __forceinline__ void load_v(T* dst, long long stride, const uint8_t* blk, int part, int t0,
                                       int cnt, float g) {
  const int lane = threadIdx.x & 31, c = 64 * part + 2 * lane;
  const uint4 v = *reinterpret_cast<const uint4*>(blk + kOffV + c * 8);
  const uint4 sv = *reinterpret_cast<const uint4*>(blk + kOffVs + (c >> 5) * kBlock);
  const uint32_t code[2][2] = {{v.x, v.y}, {v.z, v.w}}, sc[4] = {sv.x, sv.y, sv.z, sv.w};
  dst += c;
#pragma unroll
  for (int e = 0; e < kBlock; e += 2) {
    const uint32_t s2 = sc[e >> 2] >> (8 * (e & 3));
    const uint64_t s = pair(e4m3_to_float(s2 & 0xffu), e4m3_to_float((s2 >> 8) & 0xffu));
    const float2 a = value_pair(code[0][e >> 3], (e & 7) >> 1, s, pair(g, g));
    const float2 b = value_pair(code[1][e >> 3], (e & 7) >> 1, s, pair(g, g));
    if (e >= t0 && e < t0 + cnt) store2(dst + (e - t0) * stride, a.x, b.x);
    if (e + 1 >= t0 && e + 1 < t0 + cnt) store2(dst + (e + 1 - t0) * stride, a.y, b.y);
  }
}

// CTA = (rows_per_cta packed rows, heads_per_cta heads).  The warps take a block's tasks in
// turn, each another one in the next block: V's are twice as long as K's.
template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 6 : 5)
    kv4_store_kernel(const Kv4Params p, const T* __restrict__ k, long long k_stride,
                     const T* __restrict__ v, long long v_stride, uint8_t* __restrict__ cache) {
  pdl_wait();  // inputs come from the kernels before this one
  __shared__ float4 s_step[kTasks][2][kBlock];
  if (p.ok && !*p.ok) return;
  const int M = p.cu[p.B];
  if (!rows_ok(p, M)) return;
  const int groups = ceil_div(p.Hkv, p.heads_per_cta);
  const int h0 = blockIdx.x % groups * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.Hkv);
  const int row0 = blockIdx.x / groups * p.rows_per_cta;
  if (row0 >= M) return;
  const Leaders L = find_leaders(p, row0, M);
  int task = threadIdx.x >> 5;
  for (unsigned m = L.mask; m; m &= m - 1) {
    const int j = __ffs(m) - 1;
    const int t0 = __shfl_sync(0xffffffffu, L.pos, j) & (kBlock - 1);
    const int cnt = __shfl_sync(0xffffffffu, L.cnt, j);
    const long long base = __shfl_sync(0xffffffffu, L.base, j), row = row0 + j;
    for (int h = h0; h < h1; ++h) {
      uint8_t* blk = cache + (base + ((long long)h << (p.log2_page - 4))) * kBlockBytes;
      if (task < 2)
        store_v(v + row * v_stride + h * kD, v_stride, blk, task, t0, cnt, p.gv, s_step[threadIdx.x >> 5]);
      else
        store_k(k + row * k_stride + h * kD, k_stride, blk, task - 2, t0, cnt, p.gk);
      if (++task == kTasks) task = 0;
    }
  }
}

// CTA and tasks as in the store.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv4_load_kernel(const Kv4Params p, const uint8_t* __restrict__ cache, T* __restrict__ k,
                    T* __restrict__ v) {
  pdl_wait();  // inputs come from the kernels before this one
  const int M = p.cu[p.B];
  if (!rows_ok(p, M)) return;
  const int groups = ceil_div(p.Hkv, p.heads_per_cta);
  const int h0 = blockIdx.x % groups * p.heads_per_cta, h1 = min(h0 + p.heads_per_cta, p.Hkv);
  const int row0 = blockIdx.x / groups * p.rows_per_cta;
  if (row0 >= M) return;
  const Leaders L = find_leaders(p, row0, M);
  const long long stride = (long long)p.Hkv * kD;
  int task = threadIdx.x >> 5;
  for (unsigned m = L.mask; m; m &= m - 1) {
    const int j = __ffs(m) - 1;
    const int t0 = __shfl_sync(0xffffffffu, L.pos, j) & (kBlock - 1);
    const int cnt = __shfl_sync(0xffffffffu, L.cnt, j);
    const long long base = __shfl_sync(0xffffffffu, L.base, j), row = row0 + j;
    for (int h = h0; h < h1; ++h) {
      const uint8_t* blk = cache + (base + ((long long)h << (p.log2_page - 4))) * kBlockBytes;
      const long long at = row * stride + h * kD;
      if (task < 2)
        load_v(v + at, stride, blk, task, t0, cnt, p.gv);
      else
        load_k(k + at, stride, blk, task - 2, t0, cnt, p.gk);
      if (++task == kTasks) task = 0;
    }
  }
}

Kv4Params params(const int32_t* cu, const int32_t* pos0, const int32_t* keep, const int* ok, int B,
                 int max_rows, int Hkv, int page_size, const int32_t* page_table, int max_pages,
                 int n_pages, float gk, float gv) {
  Kv4Params p;
  p.cu = cu; p.pos0 = pos0; p.keep = keep; p.ok = ok; p.page_table = page_table;
  p.err = device_error_word();
  p.B = B; p.max_rows = max_rows; p.Hkv = Hkv; p.max_pages = max_pages; p.n_pages = n_pages;
  p.log2_page = 0;
  while ((1 << p.log2_page) < page_size) ++p.log2_page;
  p.gk = gk; p.gv = gv;
  // A prompt's 16 rows hold one or two leaders, a commit's 16 rows up to 16, which one CTA
  // would take one after another: a (row, head) per CTA while that fills the device less than
  // about eight times over, 16 rows and up to eight heads from there on.
  const bool few = (long long)max_rows * Hkv <= 8ll * 8 * num_sms_cached();
  p.rows_per_cta = few ? 1 : kWindow;
  p.heads_per_cta = few ? 1 : min(Hkv, 8);
  return p;
}

long long ctas(const Kv4Params& p) {
  return (long long)ceil_div(p.max_rows, p.rows_per_cta) * ceil_div(p.Hkv, p.heads_per_cta);
}

}  // namespace

int launch_kv4_store(const void* k, long long k_stride, const void* v, long long v_stride, int dtype,
                     const int32_t* cu, const int32_t* pos0, const int32_t* keep, const int* ok,
                     int B, int max_rows, int Hkv, int page_size, const int32_t* page_table,
                     int max_pages, int n_pages, float gk, float gv, void* cache,
                     cudaStream_t stream) {
  const Kv4Params p = params(cu, pos0, keep, ok, B, max_rows, Hkv, page_size, page_table, max_pages,
                             n_pages, gk, gv);
  const dim3 grid((unsigned)ctas(p));
  uint8_t* c = static_cast<uint8_t*>(cache);
  const cudaError_t e =
      dtype == DSPARK_BF16
          ? launch_pdl(kv4_store_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, p,
                       static_cast<const __nv_bfloat16*>(k), k_stride,
                       static_cast<const __nv_bfloat16*>(v), v_stride, c)
          : launch_pdl(kv4_store_kernel<float>, grid, dim3(kThreads), 0, stream, p,
                       static_cast<const float*>(k), k_stride, static_cast<const float*>(v),
                       v_stride, c);
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

int launch_kv4_load(const void* cache, const int32_t* cu, const int32_t* pos0, int B, int max_rows,
                    int Hkv, int page_size, const int32_t* page_table, int max_pages, int n_pages,
                    float gk, float gv, int dtype, void* k, void* v, cudaStream_t stream) {
  const Kv4Params p = params(cu, pos0, nullptr, nullptr, B, max_rows, Hkv, page_size, page_table,
                             max_pages, n_pages, gk, gv);
  const dim3 grid((unsigned)ctas(p));
  const uint8_t* c = static_cast<const uint8_t*>(cache);
  const cudaError_t e =
      dtype == DSPARK_BF16
          ? launch_pdl(kv4_load_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, p, c,
                       static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v))
          : launch_pdl(kv4_load_kernel<float>, grid, dim3(kThreads), 0, stream, p, c,
                       static_cast<float*>(k), static_cast<float*>(v));
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

}  // namespace dspark
