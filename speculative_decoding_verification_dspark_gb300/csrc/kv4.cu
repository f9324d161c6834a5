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
// Bound by HBM for prompts (a row is read once, 136 bytes of it are written); a step's
// commit is latency: a search of cu_seqlens, the row, the old codes.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace dspark {

namespace {

using namespace kv4;

constexpr int kThreads = 256;  // half of them on K, half on V
constexpr int kWindow = 16;    // packed rows whose leaders one CTA serves, at most

// One packed row: its request, index in the segment, rows of the segment that take part
// and cache position.
struct RowInfo {
  int r, i, n, pos, leader;
};

// The largest r < B with cu[r] <= row (cu ascending, cu[0] <= row): a warp narrows the
// range by 32 per round.
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

// Rows row0 .. row0 + nrow - 1 of the packed batch into s_info (whole CTA; ends with a
// barrier).  keep: rows 0 .. keep[r] of a segment take part (nullable: all).
__device__ __forceinline__ void scan_rows(RowInfo* s_info, int row0, int nrow,
                                          const int32_t* __restrict__ cu,
                                          const int32_t* __restrict__ pos0,
                                          const int32_t* __restrict__ keep, int B, int M) {
  const int lane = threadIdx.x & 31;
  for (int j = threadIdx.x >> 5; j < nrow; j += kThreads / 32) {
    RowInfo ri{0, 0, 0, 0, 0};
    if (row0 + j < M) {
      const int r = find_request(cu, B, row0 + j);
      const int c0 = cu[r];
      ri.r = r;
      ri.i = row0 + j - c0;
      ri.n = min(cu[r + 1], M) - c0;
      if (keep) ri.n = min(ri.n, max(keep[r], 0) + 1);
      ri.pos = pos0[r] + ri.i;
      ri.leader = ri.i < ri.n && (ri.i == 0 || (ri.pos & (kBlock - 1)) == 0);
    }
    if (lane == 0) s_info[j] = ri;
  }
  __syncthreads();
}

struct Kv4Params {
  const int32_t *cu, *pos0, *keep, *page_table;
  const int* ok;  // nullable: nothing is done unless it is set
  unsigned int* err;
  int B, max_rows, Hkv, log2_page, max_pages, n_pages, rows_per_cta;
  float gk, gv;
};

// Byte offset of the block that holds position `pos` of request r, head h; -1 (with the
// error raised) when its page is not valid.
__device__ __forceinline__ long long block_offset(const Kv4Params& p, int r, int h, int pos) {
  const int slot = pos >> p.log2_page;
  const int page = pos >= 0 && slot < p.max_pages
                       ? p.page_table[(long long)r * p.max_pages + slot] : -1;
  if (page < 0 || page >= p.n_pages) {
    if (threadIdx.x == 0) raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
    return -1;
  }
  const int per = 1 << (p.log2_page - 4);
  return (((long long)page * p.Hkv + h) * per + ((pos >> 4) & (per - 1))) * kBlockBytes;
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

// CTA = (rows_per_cta packed rows, head).  Threads 0..127 take K and 128..255 V; thread
// t of a half holds 16 elements of token t / 8.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv4_store_kernel(const Kv4Params p, const T* __restrict__ k, long long k_stride,
                     const T* __restrict__ v, long long v_stride, uint8_t* __restrict__ cache) {
  pdl_release();
  pdl_wait();  // inputs come from the kernels before this one
  __shared__ RowInfo s_info[kWindow];
  __shared__ uint8_t s_code[kBlock][kD + 16];  // V codes by token, read back by channel
  if (p.ok && !*p.ok) return;
  const int M = p.cu[p.B];
  if (M > p.max_rows) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(p.err, DSPARK_DEVERR_ROWS_OVERFLOW);
    return;
  }
  const int h = blockIdx.x % p.Hkv;
  const int row0 = blockIdx.x / p.Hkv * p.rows_per_cta;
  if (row0 >= M) return;
  scan_rows(s_info, row0, p.rows_per_cta, p.cu, p.pos0, p.keep, p.B, M);
  const bool is_v = threadIdx.x >= kThreads / 2;
  const int t = threadIdx.x & (kThreads / 2 - 1);
  const int tok = t >> 3, seg = t & 7;  // 16 elements: dims 16 seg ..
  for (int j = 0; j < p.rows_per_cta; ++j) {
    const RowInfo ri = s_info[j];
    if (!ri.leader) continue;  // uniform over the CTA, as is `off`
    const long long off = block_offset(p, ri.r, h, ri.pos);
    if (off < 0) continue;
    uint8_t* blk = cache + off;
    const int t0 = ri.pos & (kBlock - 1);
    const int cnt = min(kBlock - t0, ri.n - ri.i);
    const bool live = tok >= t0 && tok < t0 + cnt;
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
    if (live) {
      const long long row = (long long)row0 + j + tok - t0;
      load16((is_v ? v + row * v_stride : k + row * k_stride) + h * kD + seg * 16, x);
    }
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));  // (fmaxf drops a NaN)
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const float g = is_v ? p.gv : p.gk;
    const uint8_t sc = e4m3_at_least(__fdiv_rn(amax, __fmul_rn(7.f, g)));
    const float sg = __fmul_rn(e4m3_to_float(sc), g);
    uint32_t code[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) code[e] = code_of(x[e], sg);
    if (!is_v) {
      if (live) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e >> 3] |= code[e] << (4 * nibble_of(e & 7));
        *reinterpret_cast<uint2*>(blk + (seg >> 1) * 256 + tok * 16 + (seg & 1) * 8) =
            make_uint2(w[0], w[1]);
        if (!(seg & 1)) blk[kOffKs + tok * 4 + (seg >> 1)] = sc;
      }
    } else {
      uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 16; ++e) b[e >> 2] |= code[e] << (8 * (e & 3));
      *reinterpret_cast<uint4*>(&s_code[tok][seg * 16]) = make_uint4(b[0], b[1], b[2], b[3]);
      if (live && !(seg & 1)) blk[kOffVs + (seg >> 1) * kBlock + tok] = sc;
    }
    __syncthreads();
    if (is_v) {  // t = channel: this block's 16 tokens of it
      uint2* dst = reinterpret_cast<uint2*>(blk + kOffV + t * 8);
      uint32_t w[2] = {0, 0}, m[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < kBlock; ++e)
        if (e >= t0 && e < t0 + cnt) {
          w[e >> 3] |= (uint32_t)s_code[e][t] << (4 * nibble_of(e & 7));
          m[e >> 3] |= 0xfu << (4 * nibble_of(e & 7));
        }
      if (cnt < kBlock) {  // tokens of the block that are not among the rows stay
        const uint2 old = *dst;
        w[0] |= old.x & ~m[0];
        w[1] |= old.y & ~m[1];
      }
      *dst = make_uint2(w[0], w[1]);
    }
    __syncthreads();
  }
}

// CTA = (kWindow packed rows, head); thread roles as in the store.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    kv4_load_kernel(const Kv4Params p, const uint8_t* __restrict__ cache, T* __restrict__ k,
                    T* __restrict__ v) {
  pdl_release();
  pdl_wait();  // inputs come from the kernels before this one
  __shared__ RowInfo s_info[kWindow];
  __shared__ __align__(16) uint8_t s_v[kD * 8];
  const int M = p.cu[p.B];
  if (M > p.max_rows) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(p.err, DSPARK_DEVERR_ROWS_OVERFLOW);
    return;
  }
  const int h = blockIdx.x % p.Hkv;
  const int row0 = blockIdx.x / p.Hkv * p.rows_per_cta;
  if (row0 >= M) return;
  scan_rows(s_info, row0, p.rows_per_cta, p.cu, p.pos0, nullptr, p.B, M);
  const bool is_v = threadIdx.x >= kThreads / 2;
  const int t = threadIdx.x & (kThreads / 2 - 1);
  const int tok = t >> 3, seg = t & 7;
  for (int j = 0; j < p.rows_per_cta; ++j) {
    const RowInfo ri = s_info[j];
    if (!ri.leader) continue;
    const long long off = block_offset(p, ri.r, h, ri.pos);
    if (off < 0) continue;
    const uint8_t* blk = cache + off;
    const int t0 = ri.pos & (kBlock - 1);
    const int cnt = min(kBlock - t0, ri.n - ri.i);
    const bool live = tok >= t0 && tok < t0 + cnt;
    if (is_v) *reinterpret_cast<uint2*>(s_v + t * 8) = *reinterpret_cast<const uint2*>(blk + kOffV + t * 8);
    __syncthreads();
    if (live) {
      const long long row = (long long)row0 + j + tok - t0;
      float x[16];
      if (!is_v) {
        const uint2 w = *reinterpret_cast<const uint2*>(blk + (seg >> 1) * 256 + tok * 16 + (seg & 1) * 8);
        const float s = e4m3_to_float(blk[kOffKs + tok * 4 + (seg >> 1)]);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int c = ((e < 8 ? w.x : w.y) >> (4 * nibble_of(e & 7))) & 15;
          x[e] = (float)(c - 8) * s * p.gk;
        }
        store16(k + (row * p.Hkv + h) * kD + seg * 16, x);
      } else {
        const float s = e4m3_to_float(blk[kOffVs + (seg >> 1) * kBlock + tok]);
        const int nib = nibble_of(tok & 7);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int b = s_v[(seg * 16 + e) * 8 + (tok >> 3) * 4 + (nib >> 1)];
          x[e] = (float)(((b >> (4 * (nib & 1))) & 15) - 8) * s * p.gv;
        }
        store16(v + (row * p.Hkv + h) * kD + seg * 16, x);
      }
    }
    __syncthreads();
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
  // would take one after another: a row per CTA while that fills the device less than
  // about eight times over, 16 rows from there on.
  p.rows_per_cta = (long long)max_rows * Hkv <= 8ll * 8 * num_sms_cached() ? 1 : kWindow;
  return p;
}

long long ctas(const Kv4Params& p) { return (long long)ceil_div(p.max_rows, p.rows_per_cta) * p.Hkv; }

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
