// Verify attention over a paged bf16 cache for trees of drafted tokens, GQA head dim 128.
//
// Packed row cu_seqlens[r] + i, query head h, sees the ctx_len[r] committed keys of its request and
// the block rows j of its segment whose bit j is set in row_mask: o = softmax(scale q.K^T) V,
// lse = log-sum-exp.  A row that sees no key gets o = 0, lse = -inf.
//
// One warp per (row, query head), four dims to a lane, one pass over the keys with the running
// maximum and sum.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "common.cuh"

namespace dspark {
namespace attn {
namespace tree {

namespace {

constexpr int kD = 128;

__global__ void __launch_bounds__(128)
    verify_attn_tree_kernel(const __nv_bfloat16* __restrict__ q,
                            const __nv_bfloat16* __restrict__ k_new,
                            const __nv_bfloat16* __restrict__ v_new,
                            const __nv_bfloat16* __restrict__ k_cache,
                            const __nv_bfloat16* __restrict__ v_cache, int n_pages,
                            const int32_t* __restrict__ page_table, int max_pages,
                            const int32_t* __restrict__ ctx_len, const int32_t* __restrict__ cu, int B,
                            int max_rows, const uint64_t* __restrict__ mask, int words, int Hq,
                            int Hkv, int page_size, float scale, __nv_bfloat16* __restrict__ out,
                            float* __restrict__ lse, unsigned int* __restrict__ err) {
  pdl_release();
  pdl_wait();
  const int row = blockIdx.x, lane = threadIdx.x & 31;
  const int h = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (cu[B] > max_rows || cu[B] < 0) {
    if (row == 0 && h == 0 && lane == 0) raise_error(err, DSPARK_DEVERR_ROWS_OVERFLOW);
    return;
  }
  bool bad = false;
  for (int r = threadIdx.x; r < B; r += blockDim.x) {
    const long long n = (long long)cu[r + 1] - cu[r];
    bad |= cu[r] < 0 || n < 0 || ctx_len[r] < 0 || ctx_len[r] + n > 0x7fffffffll - 768;
  }
  if (__syncthreads_or(bad)) {
    if (row == 0 && threadIdx.x == 0) raise_error(err, DSPARK_DEVERR_BAD_INPUT);
    return;
  }
  if (h >= Hq || row >= cu[B] || row < cu[0]) return;
  const int r = upper_segment(cu, B, row);
  const int c0 = cu[r], n = cu[r + 1] - c0, ctx = ctx_len[r];
  const int kvh = h / (Hq / Hkv);
  auto four = [](const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  };
  const float4 x = four(q + ((long long)row * Hq + h) * kD + 4 * lane);
  float top = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto key = [&](const __nv_bfloat16* kp, const __nv_bfloat16* vp) {
    const float4 k = four(kp + 4 * lane);
    float s = x.x * k.x + x.y * k.y + x.z * k.z + x.w * k.w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= scale;
    const float4 v = four(vp + 4 * lane);
    const float next = fmaxf(top, s);
    const float fall = top == next ? 1.f : expf(top - next);
    const float w = next == -INFINITY ? 0.f : expf(s - next);
    top = next;
    sum = sum * fall + w;
    o.x = o.x * fall + w * v.x;
    o.y = o.y * fall + w * v.y;
    o.z = o.z * fall + w * v.z;
    o.w = o.w * fall + w * v.w;
  };
  for (int t = 0; t < ctx; ++t) {
    const int page = page_table[(long long)r * max_pages + t / page_size];
    if (page < 0 || page >= n_pages) {
      if (lane == 0) raise_error(err, DSPARK_DEVERR_BAD_INPUT);
      continue;
    }
    const long long at = (((long long)page * page_size + t % page_size) * Hkv + kvh) * kD;
    key(k_cache + at, v_cache + at);
  }
  for (int j = 0; j < min(n, 64 * words); ++j) {
    if (!(mask[(long long)row * words + (j >> 6)] >> (j & 63) & 1)) continue;
    const long long at = ((long long)(c0 + j) * Hkv + kvh) * kD;
    key(k_new + at, v_new + at);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = out + ((long long)row * Hq + h) * kD + 4 * lane;
  dst[0] = __float2bfloat16(o.x * inv);
  dst[1] = __float2bfloat16(o.y * inv);
  dst[2] = __float2bfloat16(o.z * inv);
  dst[3] = __float2bfloat16(o.w * inv);
  if (lane == 0) lse[(long long)row * Hq + h] = top + logf(sum);
}

}  // namespace

size_t workspace(int, int, int, int, int) { return 256; }

int launch(const void* q, const void* k_new, const void* v_new, const void* k_cache,
           const void* v_cache, int n_pages, const int32_t* page_table, int max_pages,
           const int32_t* ctx_len, const int32_t* cu, const uint64_t* mask, int words, int B,
           int max_rows, int Hq, int Hkv, int page_size, float scale, int, int, void* out,
           float* lse, void*, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  return launch_pdl(verify_attn_tree_kernel, dim3(max_rows, ceil_div(Hq, 4)), dim3(128), 0, stream,
                    static_cast<const bf*>(q), static_cast<const bf*>(k_new),
                    static_cast<const bf*>(v_new), static_cast<const bf*>(k_cache),
                    static_cast<const bf*>(v_cache), n_pages, page_table, max_pages, ctx_len, cu, B,
                    max_rows, mask, words, Hq, Hkv, page_size, scale, static_cast<bf*>(out), lse,
                    device_error_word()) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ECUDA;
}

}  // namespace tree
}  // namespace attn
}  // namespace dspark
