// Per-head RMS norm of the packed rows' queries and keys with the position rotation in
// the same pass, and the values beside them: the projections of the verify rows become
// the q, k_new and v_new that the verify attention reads.
//
// For a head vector x (128 elements) of the row at position p, in fp32:
//   y = w x / sqrt(mean(x^2) + eps)                 (no weights: y = x)
//   c_i = m cos(p f_i),  s_i = m sin(p f_i),        i < R / 2
//   (y_a, y_b) -> (y_a c_i - y_b s_i, y_b c_i + y_a s_i)
// with (a, b) = (i, i + R/2), or (2i, 2i + 1) in the interleaved form; dims >= R keep y.
// One rounding, to bf16, at the end.
//
// The angle: p f_i reaches 10^6 radians, where an fp32 product is off by 0.06, so the
// product, the division by 2 pi and the removal of whole turns are done in fp64 (error
// below 2^-52 of the turns), and the sine and cosine in fp32 on the remaining half turn.
// They are computed once per row (R/2 threads) and shared by its heads, so the slow fp64
// pipe sees R/2 angles per row, not per head.
//
// Layout: one CTA per row; a head is one half-warp, 8 elements per lane (16 bytes of
// bf16), so the norm is an 8-term sum and four shuffles, and the half form's partner
// sits (R/2)/8 lanes away.  Bound by HBM: every element is read and written once.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kBatch = 4;  // heads of a half-warp whose loads are in flight together

struct RopeParams {
  const void *q_in, *k_in, *v_in;  // v_in nullable
  long long q_stride, k_stride, v_stride;  // elements between rows
  const float *q_weight, *k_weight, *inv_freq;
  const int32_t *row_pos, *n_rows;  // n_rows nullable
  __nv_bfloat16 *q, *k, *v;
  int Hq, Hkv, rotary, heads;
  float eps, attn_factor;
};

template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeParams prm) {
  pdl_release();
  pdl_wait();  // inputs come from the kernels before this one
  __shared__ float2 s_cs[kD / 2];
  const long long row = blockIdx.x;
  const int pos = prm.row_pos[row];
  if (pos < 0 || (prm.n_rows && row >= *prm.n_rows)) return;  // padding: outputs left as they are
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int nqk = prm.Hq + prm.Hkv;
  const T* q_in = static_cast<const T*>(prm.q_in) + row * prm.q_stride + l * 8;
  const T* k_in = static_cast<const T*>(prm.k_in) + row * prm.k_stride + l * 8;
  const T* v_in = static_cast<const T*>(prm.v_in) + row * prm.v_stride + l * 8;

  Vec8<T> in[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h0 + b * kHalfWarps;
      if (h >= prm.heads) continue;
      in[b].load(h < prm.Hq ? q_in + h * kD : h < nqk ? k_in + (h - prm.Hq) * kD
                                                      : v_in + (h - nqk) * kD);
    }
  };
  load(hw);
  const int half = prm.rotary >> 1;
  if ((int)threadIdx.x < half) {
    double turns = (double)pos * (double)prm.inv_freq[threadIdx.x] * 0.15915494309189533577;
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    s_cs[threadIdx.x] = make_float2(c * prm.attn_factor, s * prm.attn_factor);
  }
  __syncthreads();
  // this lane's cosines and sines: dims 8l .. 8l + 7 (half form: index of the dim within
  // its half; interleaved: the lane's four pairs)
  const bool rotated = l * 8 < prm.rotary;
  const bool low = l * 8 < half;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = INTERLEAVED ? l * 4 + (i >> 1) : l * 8 - (low ? 0 : half) + i;
    const float2 cs = rotated ? s_cs[at] : make_float2(1.f, 0.f);
    c[i] = cs.x;
    // the partner's sign: y_a c - y_b s, y_b c + y_a s
    s[i] = (INTERLEAVED ? (i & 1) == 0 : low) ? -cs.y : cs.y;
  }
  const int partner = !rotated ? l : low ? l + (half >> 3) : l - (half >> 3);

  for (int h0 = hw; h0 - hw < prm.heads; h0 += kBatch * kHalfWarps) {
    if (h0 != hw) load(h0);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = h0 + b * kHalfWarps;
      if (h - hw >= prm.heads) break;  // uniform over the CTA
      const bool live = h < prm.heads;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (live) in[b].get(x);
      if (h < nqk) {
        const float* w = h < prm.Hq ? prm.q_weight : prm.k_weight;
        if (w) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
          const unsigned m = 0xffffu << (threadIdx.x & 16);  // this half-warp
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(m, ss, o);
          const float r = 1.f / sqrtf(ss * (1.f / kD) + prm.eps);
          const float4 w0 = reinterpret_cast<const float4*>(w)[2 * l];
          const float4 w1 = reinterpret_cast<const float4*>(w)[2 * l + 1];
          x[0] *= r * w0.x; x[1] *= r * w0.y; x[2] *= r * w0.z; x[3] *= r * w0.w;
          x[4] *= r * w1.x; x[5] *= r * w1.y; x[6] *= r * w1.z; x[7] *= r * w1.w;
        }
        float y[8];
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
        } else {
          const unsigned m = 0xffffu << (threadIdx.x & 16);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(m, x[i], partner, 16);
        }
        if (rotated) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], c[i], y[i] * s[i]);
        }
      }
      if (live) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 v2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          o[i] = *reinterpret_cast<const uint32_t*>(&v2);
        }
        __nv_bfloat16* dst = h < prm.Hq ? prm.q + (row * prm.Hq + h) * kD
                             : h < nqk  ? prm.k + (row * prm.Hkv + h - prm.Hq) * kD
                                        : prm.v + (row * prm.Hkv + h - nqk) * kD;
        reinterpret_cast<uint4*>(dst)[l] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

}  // namespace

int launch_qk_norm_rope(const void* q_in, long long q_stride, const void* k_in, long long k_stride,
                        const void* v_in, long long v_stride, int dtype, const float* q_weight,
                        const float* k_weight, float eps, const float* inv_freq, int rotary_dim,
                        int interleaved, float attn_factor, const int32_t* row_pos,
                        const int32_t* n_rows, int rows, int Hq, int Hkv, void* q, void* k_new,
                        void* v_new, cudaStream_t stream) {
  RopeParams p;
  p.q_in = q_in; p.k_in = k_in; p.v_in = v_in;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.q_weight = q_weight; p.k_weight = k_weight; p.inv_freq = inv_freq;
  p.row_pos = row_pos; p.n_rows = n_rows;
  p.q = static_cast<__nv_bfloat16*>(q);
  p.k = static_cast<__nv_bfloat16*>(k_new);
  p.v = static_cast<__nv_bfloat16*>(v_new);
  p.Hq = Hq; p.Hkv = Hkv; p.rotary = rotary_dim;
  p.heads = Hq + Hkv + (v_in ? Hkv : 0);
  p.eps = eps; p.attn_factor = attn_factor;
  void (*fn)(RopeParams) =
      dtype == DSPARK_BF16
          ? (interleaved ? qk_norm_rope_kernel<__nv_bfloat16, true> : qk_norm_rope_kernel<__nv_bfloat16, false>)
          : (interleaved ? qk_norm_rope_kernel<float, true> : qk_norm_rope_kernel<float, false>);
  return launch_pdl(fn, dim3(rows), dim3(kThreads), 0, stream, p) == cudaSuccess ? DSPARK_OK
                                                                                  : DSPARK_ECUDA;
}

}  // namespace dspark
