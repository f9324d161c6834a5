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
// The angle: p f_i reaches 10^6 radians, where an fp32 product is off by 0.06.  So f_i / 2 pi
// is taken once per CTA in fp64 and kept as a 64-bit fixed-point fraction of a turn; its
// product with p modulo 2^64 is the angle less its whole turns, off by p 2^-52 f_i / 2 pi turns
// (1 / 2 pi and the product are rounded, 2^-53 each) and p 2^-65, which goes to the fp32 sine
// and cosine.  A row's R/2 angles are computed once and shared by its heads.
//
// Layout: a persistent CTA takes `group` rows at a time, its 16 half-warps dealt to the rows;
// a half-warp holds a head, 8 elements per lane (16 bytes of bf16), so the norm is an
// 8-term sum and four shuffles, and the half form's partner sits (R/2)/8 lanes away.  The
// first inputs of a group are under way before its positions are known.  Bound by HBM:
// every element is read and written once.
//
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
constexpr int kMaxGroup = 16;

struct RopeParams {
  const void *q_in, *k_in, *v_in;  // v_in nullable
  long long q_stride, k_stride, v_stride;  // elements between rows
  const float *q_weight, *k_weight, *inv_freq;
  const int32_t *row_pos, *n_rows;  // n_rows nullable
  __nv_bfloat16 *q, *k, *v;
  int rows, Hq, Hkv, Hv, rotary, log2_group;  // Hv: 0 without values
  float eps, attn_factor;
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r) : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)),
        "l"(*reinterpret_cast<uint64_t*>(&c)));
  return *reinterpret_cast<float2*>(&r);
}

// Eight elements of a head as they were read; `x` gives them as four pairs, `from` the eight
// of another lane of the half-warp.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
  __device__ __forceinline__ float2 x(int i) const {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ Vec8 from(unsigned mask, int lane) const {
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = __shfl_sync(mask, w[i], lane, 16);
    return o;
  }
  __device__ __forceinline__ uint32_t bf16(int i) const { return w[i]; }
};
template <>
struct Vec8<float> {
  float2 v[4];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = make_float2(a.x, a.y); v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y); v[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ float2 x(int i) const { return v[i]; }
  __device__ __forceinline__ Vec8 from(unsigned mask, int lane) const {
    Vec8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o.v[i] = make_float2(__shfl_sync(mask, v[i].x, lane, 16), __shfl_sync(mask, v[i].y, lane, 16));
    return o;
  }
  __device__ __forceinline__ uint32_t bf16(int i) const {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// The heads first, first + step, .. < n of one part of a row (element pointers of this lane's
// dims in head 0), N of them in flight.
template <typename T, int N>
struct Heads {
  Vec8<T> in[N];
  __device__ __forceinline__ void start(const T* src, int first, int step, int n) {
#pragma unroll
    for (int b = 0; b < N; ++b)
      if (first + b * step < n) in[b].load(src + (first + b * step) * kD);
  }
  template <typename F>
  __device__ __forceinline__ void run(const T* src, __nv_bfloat16* dst, int first, int step, int n, F f) {
    for (int h0 = first; h0 < n; h0 += N * step) {
#pragma unroll
      for (int b = 0; b < N; ++b) {
        const int h = h0 + b * step;
        if (h >= n) break;
        const Vec8<T> x = in[b];
        if (h + N * step < n) in[b].load(src + (h + N * step) * kD);
        *reinterpret_cast<uint4*>(dst + h * kD) = f(x);
      }
    }
  }
};

template <typename T, bool INTERLEAVED, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) qk_norm_rope_kernel(const RopeParams prm) {
  __shared__ float2 s_cs[2][kMaxGroup][kD / 2];
  __shared__ __align__(16) float s_w[2][kD];
  const int hw = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int group = 1 << prm.log2_group, step = kHalfWarps >> prm.log2_group;
  const int half = prm.rotary >> 1;
  const int my_row = hw & (group - 1), first = hw >> prm.log2_group;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);  // this half-warp
  pdl_wait();  // inputs come from the kernels before this one
  // this thread's angles: frequency i of rows threadIdx.x / 64, + 4, .. of the group; and its weight
  const int ai = threadIdx.x & 63;
  const float freq = ai < half ? prm.inv_freq[ai] : 0.f;
  const float* const wp = threadIdx.x < kD ? prm.q_weight : prm.k_weight;
  const float weight = wp ? wp[threadIdx.x % kD] : 1.f;
  unsigned long long turn = 0;  // f / (2 pi) in 2^-64 turns
  float factor = prm.attn_factor;
  const int n_rows = prm.n_rows ? min(*prm.n_rows, prm.rows) : prm.rows;
  const bool rotated = l * 8 < prm.rotary;
  const bool low = l * 8 < half;
  const int partner = !rotated ? l : low ? l + (half >> 3) : l - (half >> 3);

  int buf = 0;
  for (int row0 = blockIdx.x << prm.log2_group; row0 < n_rows; row0 += gridDim.x << prm.log2_group, buf ^= 1) {
    const long long row = row0 + my_row;
    const bool live = row < n_rows;
    const T* q_in = static_cast<const T*>(prm.q_in) + row * prm.q_stride + l * 8;
    const T* k_in = static_cast<const T*>(prm.k_in) + row * prm.k_stride + l * 8;
    const T* v_in = static_cast<const T*>(prm.v_in) + row * prm.v_stride + l * 8;
    Heads<T, CTAS == 4 ? 1 : 2> q;
    Heads<T, 1> k, v;
    int pos = -1;
    if (live) {
      q.start(q_in, first, step, prm.Hq);
      k.start(k_in, first, step, prm.Hkv);
      v.start(v_in, first, step, prm.Hv);
      pos = prm.row_pos[row];
    }
    if (row0 == (int)blockIdx.x << prm.log2_group) {  // the first group, whose inputs are under way
      s_w[threadIdx.x / kD][threadIdx.x % kD] = weight;
      double t = (double)freq * 0.15915494309189533577;
      t -= rint(t);
      turn = (unsigned long long)__double2ll_rn(t * 18446744073709551616.);
      if (t != t) factor = __int_as_float(0x7fc00000);
    }
    for (int ar = threadIdx.x >> 6; ai < half && ar < group && row0 + ar < n_rows; ar += kThreads / 64) {
      const unsigned long long z = turn * (unsigned)prm.row_pos[row0 + ar];
      float s, c;
      sincospif(__ll2float_rn((long long)z) * 0x1p-63f, &s, &c);
      s_cs[buf][ar][ai] = make_float2(c * factor, s * factor);
    }
    __syncthreads();
    if (pos < 0) continue;  // a row of padding: outputs left as they are (uniform over the half-warp)

    v.run(v_in, prm.v + row * prm.Hkv * kD + l * 8, first, step, prm.Hv, [&](const Vec8<T>& x) {
      return make_uint4(x.bf16(0), x.bf16(1), x.bf16(2), x.bf16(3));
    });
    // y = r (x c w + partner's x (+- s w of the partner)): the factors of this lane's dims
    float2 c[4], s[4];
    auto factors = [&](const float* weight) {
      float wc[8], ws[8], w[8];
      load8(weight + l * 8, wc);
      load8(weight + (INTERLEAVED ? l : partner) * 8, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = INTERLEAVED ? l * 4 + (i >> 1) : l * 8 - (low ? 0 : half) + i;
        const float2 cs = rotated ? s_cs[buf][my_row][at] : make_float2(1.f, 0.f);
        wc[i] *= cs.x;
        // y_a c - y_b s, y_b c + y_a s
        ws[i] = w[INTERLEAVED ? i ^ 1 : i] * ((INTERLEAVED ? (i & 1) == 0 : low) ? -cs.y : cs.y);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = make_float2(wc[2 * i], wc[2 * i + 1]);
        s[i] = make_float2(ws[2 * i], ws[2 * i + 1]);
      }
    };
    auto head = [&](const Vec8<T>& v8, bool norm) {
      float2 r = make_float2(1.f, 1.f);
      if (norm) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(v8.x(i), v8.x(i), ss);
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(mask, sum, o);
        r.x = r.y = rsqrtf(sum * (1.f / kD) + prm.eps);
      }
      float2 y[4];
      if (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = make_float2(v8.x(i).y, v8.x(i).x);
      } else {
        const Vec8<T> other = v8.from(mask, partner);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = other.x(i);
      }
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 x = mul2(v8.x(i), c[i]);
        if (rotated) x = fma2(y[i], s[i], x);
        x = mul2(x, r);
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        o[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      return make_uint4(o[0], o[1], o[2], o[3]);
    };
    factors(s_w[0]);
    const bool q_norm = prm.q_weight, k_norm = prm.k_weight;
    q.run(q_in, prm.q + row * prm.Hq * kD + l * 8, first, step, prm.Hq,
          [&](const Vec8<T>& x) { return head(x, q_norm); });
    factors(s_w[1]);
    k.run(k_in, prm.k + row * prm.Hkv * kD + l * 8, first, step, prm.Hkv,
          [&](const Vec8<T>& x) { return head(x, k_norm); });
  }
}

// Many rows: four CTAs per SM for bf16 with one query head of a half-warp under way (16384 rows
// of 56 heads: 94 us; with two under way 97, three CTAs 102, two CTAs 113), two for fp32 with two
// (4099 rows of 12 heads: 7.9 us, three CTAs 9.0).  Groups so that a half-warp has two of a
// row's KV heads, while every CTA has a group: 16384 rows 102 us with groups of 4 against 110
// with 2 and 111 with 8; 4099 rows 7.4 with 8, 9.1 with 4.  Up to two rows per SM each row has
// its CTA and the registers of two CTAs per SM (256 rows: 4.8 us, 6.0 with those of three).
template <typename T, bool INTERLEAVED>
int launch(RopeParams& p, cudaStream_t stream) {
  const int sms = num_sms_cached();
  const bool few = p.rows <= 2 * sms;
  constexpr int kCtas = sizeof(T) == 2 ? 4 : 2;
  p.log2_group = 0;
  if (!few)
    while ((1 << p.log2_group) < kMaxGroup && (p.Hkv << p.log2_group) < 32 &&
           (p.rows >> (p.log2_group + 1)) >= kCtas * sms)
      ++p.log2_group;
  const int groups = ceil_div(p.rows, 1 << p.log2_group);
  void (*fn)(RopeParams) =
      few ? qk_norm_rope_kernel<T, INTERLEAVED, 2> : qk_norm_rope_kernel<T, INTERLEAVED, kCtas>;
  const int grid = few ? groups : min(groups, kCtas * sms);
  return launch_pdl(fn, dim3(grid), dim3(kThreads), 0, stream, p) == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
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
  p.rows = rows; p.Hq = Hq; p.Hkv = Hkv; p.rotary = rotary_dim;
  p.Hv = v_in ? Hkv : 0;
  p.eps = eps; p.attn_factor = attn_factor;
  return dtype == DSPARK_BF16
             ? (interleaved ? launch<__nv_bfloat16, true>(p, stream) : launch<__nv_bfloat16, false>(p, stream))
             : (interleaved ? launch<float, true>(p, stream) : launch<float, false>(p, stream));
}

}  // namespace dspark
