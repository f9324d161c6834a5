// Varlen verify attention over a 4-bit paged KV cache (layout: kv4.cuh), GQA head dim 128.
//
// For packed row cu_seqlens[r] + i and query head h of KV group kvh:
//   o = softmax(scale q.K^T) V over the ctx_len[r] committed keys, whose K and V are
//   (code - 8) * scale * g, followed by block rows 0..i (bf16); lse = log-sum-exp.
//
// CTA = (packed row, query head), thread = key of a 128-key tile for the scores and
// channel for the values; running maximum and sum in fp32.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"
#include "kv4.cuh"

namespace dspark {
namespace attn {
namespace kv4a {

using namespace dspark::kv4;

struct Params {
  const __nv_bfloat16 *q, *k_new, *v_new;
  const uint8_t* cache;
  const int32_t *page_table, *ctx_len, *cu;
  __nv_bfloat16* out;
  float* lse;
  unsigned int* err;
  int B, max_rows, Hq, Hkv, log2_page, max_pages, n_pages;
  float scale, gk, gv;
};

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  return is_max ? fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]))
                : (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
}

__global__ void __launch_bounds__(128) verify_attn_kv4_kernel(const Params p) {
  pdl_release();
  pdl_wait();
  __shared__ float s_q[kD], s_p[128], s_red[4];
  __shared__ const uint8_t* s_blk[8];
  const int M = p.cu[p.B];
  if (M > p.max_rows) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(p.err, DSPARK_DEVERR_ROWS_OVERFLOW);
    return;
  }
  const int h = blockIdx.x % p.Hq, row = blockIdx.x / p.Hq;
  if (row >= M) return;
  const int kvh = h / (p.Hq / p.Hkv), t = threadIdx.x;
  const int r = upper_segment(p.cu, p.B, row);
  const int c0 = p.cu[r], i = row - c0, ctx = p.ctx_len[r];
  const int keys = ctx + i + 1;
  s_q[t] = __bfloat162float(p.q[((long long)row * p.Hq + h) * kD + t]);
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int k0 = 0; k0 < keys; k0 += 128) {
    __syncthreads();
    if (t < 8) {
      const int pos = k0 + t * 16;
      const uint8_t* b = nullptr;
      if (pos < ctx) {
        const int slot = pos >> p.log2_page;
        const int page = slot < p.max_pages ? p.page_table[(long long)r * p.max_pages + slot] : -1;
        if (page < 0 || page >= p.n_pages) {
          raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
        } else {
          const int per = 1 << (p.log2_page - 4);
          b = p.cache + (((long long)page * p.Hkv + kvh) * per + ((pos >> 4) & (per - 1))) * kBlockBytes;
        }
      }
      s_blk[t] = b;
    }
    __syncthreads();
    const int pos = k0 + t;
    float s = -INFINITY;
    if (pos < ctx) {
      const uint8_t* b = s_blk[t >> 4];
      if (b) {
        float acc = 0.f;
        for (int c = 0; c < 4; ++c) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(b + c * 256 + (t & 15) * 16);
          float part = 0.f;
          for (int e = 0; e < 32; ++e)
            part += s_q[c * 32 + e] * (float)((int)((w[e >> 3] >> (4 * nibble_of(e & 7))) & 15) - 8);
          acc += part * e4m3_to_float(b[kOffKs + (t & 15) * 4 + c]);
        }
        s = acc * p.gk * p.scale;
      }
    } else if (pos < keys) {
      const __nv_bfloat16* kn = p.k_new + ((long long)(c0 + pos - ctx) * p.Hkv + kvh) * kD;
      float acc = 0.f;
      for (int e = 0; e < kD; ++e) acc += s_q[e] * __bfloat162float(kn[e]);
      s = acc * p.scale;
    }
    const float mn = fmaxf(m, block_reduce(s, true, s_red));
    const float e = expf(s - (mn == -INFINITY ? 0.f : mn));  // (a NaN score stays NaN)
    s_p[t] = e;
    const float f = m == -INFINITY ? 0.f : expf(m - mn);
    l = l * f + block_reduce(e, false, s_red);
    o *= f;
    m = mn;
    for (int k = 0; k < 128 && k0 + k < keys; ++k) {
      const int kp = k0 + k;
      float v = 0.f;
      if (kp < ctx) {
        const uint8_t* b = s_blk[k >> 4];
        if (b) {
          const uint32_t w = reinterpret_cast<const uint32_t*>(b + kOffV + t * 8)[(k >> 3) & 1];
          v = (float)((int)((w >> (4 * nibble_of(k & 7))) & 15) - 8) *
              e4m3_to_float(b[kOffVs + (t >> 5) * kBlock + (k & 15)]) * p.gv;
        }
      } else {
        v = __bfloat162float(p.v_new[((long long)(c0 + kp - ctx) * p.Hkv + kvh) * kD + t]);
      }
      o += s_p[k] * v;
    }
  }
  p.out[((long long)row * p.Hq + h) * kD + t] = __float2bfloat16(l == 0.f ? 0.f : o / l);
  if (t == 0) p.lse[(long long)row * p.Hq + h] = m + logf(l);
}

int launch(const void* q, const void* k_new, const void* v_new, const void* cache, int n_pages,
           const int32_t* page_table, int max_pages, const int32_t* ctx_len,
           const int32_t* cu_seqlens, int B, int max_rows, int Hq, int Hkv, int page_size,
           float scale, float gk, float gv, void* out, float* lse, cudaStream_t stream) {
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.cache = static_cast<const uint8_t*>(cache);
  p.page_table = page_table; p.ctx_len = ctx_len; p.cu = cu_seqlens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.err = device_error_word();
  p.B = B; p.max_rows = max_rows; p.Hq = Hq; p.Hkv = Hkv;
  p.log2_page = 0;
  while ((1 << p.log2_page) < page_size) ++p.log2_page;
  p.max_pages = max_pages; p.n_pages = n_pages;
  p.scale = scale; p.gk = gk; p.gv = gv;
  return launch_pdl(verify_attn_kv4_kernel, dim3((unsigned)((long long)max_rows * Hq)), dim3(128), 0,
                    stream, p) == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

}  // namespace kv4a
}  // namespace attn
}  // namespace dspark
