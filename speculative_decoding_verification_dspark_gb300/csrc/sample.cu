// Sampling from logits with temperature, top-k, top-p and min-p, given exponential noise.
//
// A row's tokens in order of their logits l, the lowest index first among equals; m the largest.
// w_v = exp((l_v - m) / T).  Each filter keeps a first part of that order:
//   top-k   the first k
//   min-p   those with w_v >= min_p
//   top-p   the shortest first part that holds p of the mass the two others left
// probs_v = w_v / sum of the kept w (0 for the others); token = argmax_v w_v / e_v over the kept
// ones, lowest index on ties: with e ~ Exp(1) a draw from probs.
//
// A row belongs to a cluster of 1 to 8 CTAs, whose shared memory holds it: logits are read from
// memory once, whatever the filters need.  The end of the kept part is found without sorting the
// row:
//   1  tokens are counted in 2048 buckets of (m - l) / T, 1/32 of an octave of w each;
//   2  a bracket of buckets that must hold the end is taken (for top-p by masses that the counts
//      estimate), and one pass sums the masses above, in and below it and lists its tokens;
//   3  one CTA sorts the list and walks it.
// A bracket of more than kList tokens is cut again by the bits of its logits, one that holds a
// single value is resolved by counting indices.  Where a sum comes so near to the border that
// fp32 cannot tell on which side the end lies (kNear), sums are taken again in pairs of fp32
// numbers (2^-36 or so): the kept set is that of the definition in 64 bits.

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBuckets = 2048;
constexpr float kPerOctave = 32.f;
constexpr int kList = 1024;            // tokens of a bracket that are sorted
constexpr int kMaxCluster = 8;
constexpr int kChunkBytes = 76 * 1024; // of a row in one CTA, while eight CTAs hold the row
// Error of the fp32 sums relative to the mass: ex2.approx and the products before it give 2^-21 per
// token at most for the tokens that matter, far less in the sum of many.
constexpr double kNear = 1e-6;

struct Shared {
  unsigned hist[kBuckets];             // this CTA's counts
  unsigned tot[kBuckets];              // the row's, in order of falling logits
  uint64_t list[kList];                // (order of the logit, index)
  double part[2][kMaxCluster][3];      // exchanged between the CTAs, two sets in turn
  float cmax[kMaxCluster];
  double wsum[kWarps][3];
  float wmax[kWarps];
  unsigned wcnt[kWarps];
  double wmass[kWarps];
  float e2h[17], e2l[17];              // 2^(-j / 16), j = -8 .. 8, in two parts
  float c_hi, c_lo;                    // log2(e) / T in two parts
  double log_min;                      // T ln(min_p)
  int n_list;
  // a decision of one thread or CTA for all
  int b_at;
  unsigned cum_before, cum_in, total;
  float f_lo, f_hi, t_cut;
  int i_cut, n_keep, again;
  double z_kept;
  float best[kWarps];
  double r_best[kWarps];
  int r_idx[kWarps];
  float c_best[kMaxCluster];
  double cr_best[kMaxCluster];
  int cr_idx[kMaxCluster];
};

// Order-preserving code of a float (no NaN, no -0).
__device__ __forceinline__ uint32_t code_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float float_of(uint32_t c) {
  return __uint_as_float(c ^ ((c >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(uint4 u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float one(const void* p, long long i) {
    return static_cast<const float*>(p)[i];
  }
  static constexpr float kTop = FLT_MAX;
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {  // (exact: bf16 numbers)
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float one(const void* p, long long i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  static constexpr float kTop = 3.3895313892515355e38f;
};

// NaN counts as -inf, -0 as 0, and +inf as the type's largest number.
__device__ __forceinline__ float clean(float x, float top) {
  x = x + 0.f;
  return x == x ? fminf(x, top) : -INFINITY;
}

struct Kept {    // tokens with l > t, or l == t and an index of at most i
  float t;
  int i;
};

template <typename T>
struct Row {
  using V = Vec<T>;
  cg::cluster_group cl;
  Shared& S;
  const T* data;      // slots of this CTA's chunk in shared memory
  int C, rank;
  int first, n;       // the chunk: tokens first .. first + n - 1
  int shift, groups;  // token i of the chunk is slot i + shift; 16-byte groups of slots
  int set;            // of S.part
  float m, s;         // largest logit; buckets per unit of logit
  float t_min;        // least logit that min-p leaves
  Kept lim;           // what earlier filters left

  __device__ __forceinline__ float y_of(float l) const { return (m - l) * s; }
  __device__ __forceinline__ float w_of(float l) const { return ex2(y_of(l) * (-1.f / kPerOctave)); }
  __device__ __forceinline__ bool left(float l, int i) const {
    return l > lim.t || (l == lim.t && first + i <= lim.i);
  }

  // fn(l, i) for every token of the chunk.
  template <class Fn>
  __device__ __forceinline__ void each(Fn&& fn) const {
    const uint4* p = reinterpret_cast<const uint4*>(data);
    for (int q = threadIdx.x; q < groups; q += kThreads) {
      float x[V::N];
      V::get(p[q], x);
#pragma unroll
      for (int j = 0; j < V::N; ++j) fn(x[j], q * V::N + j - shift);
    }
  }

  // Sums of three numbers over the row, the same in every thread of the cluster; in fixed order.
  __device__ void sum3(double (&v)[3]) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    __syncthreads();
    if (lane == 0)
      for (int k = 0; k < 3; ++k) S.wsum[wid][k] = v[k];
    __syncthreads();
    if (threadIdx.x < 3) {
      double a = 0;
      for (int w = 0; w < kWarps; ++w) a += S.wsum[w][threadIdx.x];
      for (int r = 0; r < C; ++r) cl.map_shared_rank(&S, r)->part[set][rank][threadIdx.x] = a;
    }
    cl.sync();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      v[k] = 0;
      for (int r = 0; r < C; ++r) v[k] += S.part[set][r][k];
    }
    set ^= 1;
  }

  // Counts of the row's tokens by bucket(l, i) (0 .. kBuckets - 1, or negative: not counted), into
  // S.tot of every CTA.
  template <class Fn>
  __device__ void histogram(Fn&& bucket) {
    __syncthreads();
    for (int b = threadIdx.x; b < kBuckets; b += kThreads) S.hist[b] = 0;
    __syncthreads();
    each([&](float l, int i) {
      const int b = bucket(l, i);
      if (b >= 0) atomicAdd(&S.hist[b], 1u);
    });
    cl.sync();
    const int per = kBuckets / C;
    for (int k = threadIdx.x; k < per; k += kThreads) {
      const int b = rank * per + k;
      unsigned a = 0;
      for (int r = 0; r < C; ++r) a += cl.map_shared_rank(&S, r)->hist[b];
      for (int r = 0; r < C; ++r) cl.map_shared_rank(&S, r)->tot[b] = a;
    }
    cl.sync();
  }

  // Over S.tot: the bucket in which the running count reaches `target`, or (weighted) the running
  // mass reaches the part `share` of the whole, the mass of bucket b being tot[b] * mass(b).
  // Sets S.b_at, S.cum_before (tokens in the buckets before), S.cum_in and S.total.
  template <class Fn>
  __device__ void locate(bool weighted, unsigned target, double share, Fn&& mass) {
    constexpr int kPer = kBuckets / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    unsigned c[kPer], cs = 0;
    float w[kPer], ws = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = S.tot[tid * kPer + j];
      w[j] = weighted ? c[j] * mass(tid * kPer + j) : 0.f;
      cs += c[j];
      ws += w[j];
    }
    unsigned ci = cs;
    double wi = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, ci, o);
      const double d = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) {
        ci += u;
        wi += d;
      }
    }
    __syncthreads();
    if (lane == 31) {
      S.wcnt[wid] = ci;
      S.wmass[wid] = wi;
    }
    if (tid == 0) S.b_at = -1;
    __syncthreads();
    unsigned c0 = ci - cs, last = 0;
    double w0 = wi - ws, total = 0;
    for (int v = 0; v < kWarps; ++v) {
      if (v < wid) {
        c0 += S.wcnt[v];
        w0 += S.wmass[v];
      }
      total += S.wmass[v];
      last += S.wcnt[v];
    }
    const double goal = share * total;
    if (tid == 0) S.total = last;
    for (int j = 0; j < kPer; ++j) {
      const bool here = weighted ? (w0 < goal && w0 + w[j] >= goal) : (c0 < target && c0 + c[j] >= target);
      if (here) {
        // (rounding may let two buckets meet the goal: either will do)
        S.b_at = tid * kPer + j;
        S.cum_before = c0;
        S.cum_in = c[j];
      }
      c0 += c[j];
      w0 += w[j];
    }
    __syncthreads();
    if (S.b_at < 0) {  // the goal lies past the last token (rounding): the last bucket that holds one
      __syncthreads();
      c0 = ci - cs;
      for (int v = 0; v < wid; ++v) c0 += S.wcnt[v];
      for (int j = 0; j < kPer; ++j) {
        if (c[j] && c0 + c[j] == last) {
          S.b_at = tid * kPer + j;
          S.cum_before = c0;
          S.cum_in = c[j];
        }
        c0 += c[j];
      }
      __syncthreads();
    }
  }

  // The least float l with y_of(l) < bound; y falls as l grows, so 32 lanes halve the codes five
  // bits at a time.  By the first warp.
  __device__ float edge(float bound) const {
    const int lane = threadIdx.x & 31;
    uint32_t lo = code_of(-FLT_MAX), hi = code_of(m);  // y(hi) = 0 < bound
    while (hi > lo) {
      const uint32_t step = (hi - lo + 31) / 32, at = lo + min((unsigned)lane * step, hi - lo);
      const unsigned ok = __ballot_sync(0xffffffffu, y_of(float_of(at)) < bound);
      // (at of lane 31 may be below hi: hi stays then)
      const int f = ok ? __ffs(ok) - 1 : 32;
      const uint32_t a = lo + min((unsigned)(f > 0 ? f - 1 : 0) * step, hi - lo);
      const uint32_t z = f < 32 ? lo + min((unsigned)f * step, hi - lo) : hi;
      if (f == 0) return float_of(lo);
      lo = a + 1;
      hi = z;
    }
    return float_of(hi);
  }

  // Masses of the tokens left: above f_hi, in [f_lo, f_hi), and all; those of the bracket are listed
  // in S.list where `gather` is set.
  __device__ void evaluate(float f_lo, float f_hi, bool gather, double (&v)[3]) {
    __syncthreads();
    if (threadIdx.x == 0) S.n_list = 0;
    __syncthreads();
    float above = 0, in = 0, below = 0;
    const bool limited = lim.i != 0x7fffffff;
    each([&](float l, int i) {
      if (l < lim.t) return;
      if (limited && !left(l, i)) return;
      const float w = w_of(l);
      if (l >= f_hi) {
        above += w;
      } else if (l >= f_lo) {
        in += w;
        if (gather) {
          const int at = atomicAdd(&S.n_list, 1);
          if (at < kList)
            S.list[at] = (uint64_t)(~code_of(l)) << 32 | (uint32_t)(first + i);
        }
      } else {
        below += w;
      }
    });
    v[0] = above;
    v[1] = in;
    v[2] = (double)above + (double)in + (double)below;
    sum3(v);
  }

  // w in two parts, 2^-36 of it or better, by table and polynomial (Tang's scheme for the
  // exponential): X = (m - l) log2(e) / T = n + j / 16 + h, w = 2^-n 2^(-j/16) e^(-h ln 2).
  __device__ __forceinline__ void w_pair(float l, float& wh, float& wl) const {
    const float dh = m - l, z = dh - m;
    const float dl = (m - (dh - z)) - (l + z);
    const float ph = dh * S.c_hi;
    const float pl = fmaf(dh, S.c_hi, -ph) + fmaf(dh, S.c_lo, dl * S.c_hi);
    if (!(ph < 120.f)) {
      wh = wl = 0.f;
      return;
    }
    const float n = rintf(ph), f = ph - n, j = rintf(f * 16.f), h = f - j * 0.0625f;
    constexpr float kLn2h = 0.693147182464599609375f, kLn2l = -1.904654290582768e-9f;
    const float uh = -h * kLn2h;
    const float ul = fmaf(-h, kLn2h, -uh) - fmaf(h, kLn2l, pl * kLn2h);
    const float q = uh * uh * fmaf(uh, fmaf(uh, fmaf(uh, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f);
    const float a = q + fmaf(uh, ul, ul);
    const float sh = uh + a, sl = a - (sh - uh);
    const float th = S.e2h[(int)j + 8], tl = S.e2l[(int)j + 8];
    const float p = th * sh, pe = fmaf(th, sh, -p);
    const float r = th + p;
    const float rl = (p - (r - th)) + (pe + fmaf(th, sl, fmaf(tl, sh, tl)));
    const float scale = __int_as_float((127 - (int)n) << 23);
    wh = r * scale;
    wl = rl * scale;
  }

  // evaluate's masses in pairs.
  __device__ void evaluate_pairs(float f_lo, float f_hi, double (&v)[3]) {
    if (threadIdx.x < 17) {
      const double e = exp2(-((int)threadIdx.x - 8) / 16.0);
      S.e2h[threadIdx.x] = (float)e;
      S.e2l[threadIdx.x] = (float)(e - (double)(float)e);
    }
    __syncthreads();
    float ah = 0, al = 0, ih = 0, il = 0, bh = 0, bl = 0;
    auto add = [](float& sh, float& sl, float wh, float wl) {
      const float t = sh + wh, z = t - sh;
      sl += ((sh - (t - z)) + (wh - z)) + wl;
      sh = t;
    };
    each([&](float l, int i) {
      if (l < lim.t || !left(l, i)) return;
      float wh, wl;
      w_pair(l, wh, wl);
      if (l >= f_hi) add(ah, al, wh, wl);
      else if (l >= f_lo) add(ih, il, wh, wl);
      else add(bh, bl, wh, wl);
    });
    v[0] = (double)ah + al;
    v[1] = (double)ih + il;
    v[2] = v[0] + v[1] + ((double)bh + bl);
    sum3(v);
  }

  // The lists of all CTAs into this one's, sorted; n tokens in all (at most kList).
  __device__ int collect() {
    int n = S.n_list;  // (every rank's was written before the last cl.sync)
    __syncthreads();
    for (int r = 1; r < C; ++r) {
      Shared* o = cl.map_shared_rank(&S, r);
      const int k = o->n_list;
      for (int i = threadIdx.x; i < k; i += kThreads)
        if (n + i < kList) S.list[n + i] = o->list[i];
      n += k;
    }
    n = min(n, kList);
    int size = 32;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreads) S.list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k <<= 1)
      for (int d = k >> 1; d > 0; d >>= 1) {
        for (int i = threadIdx.x; i < size / 2; i += kThreads) {
          const int a = 2 * i - (i & (d - 1)), b = a + d;
          const uint64_t x = S.list[a], y = S.list[b];
          if ((x > y) == ((a & k) == 0)) {
            S.list[a] = y;
            S.list[b] = x;
          }
        }
        __syncthreads();
      }
    return n;
  }

  __device__ __forceinline__ float list_l(int i) const {
    return float_of(~(uint32_t)(S.list[i] >> 32));
  }

  // By the first CTA, over its sorted list of n tokens with masses v[0] above and v[2] in all: the
  // end of the first `k` of them (k >= n: all) and, where p < 1, of the p part of what these and
  // the tokens above hold (k_round: v[2] is not that mass yet, the list gives it).  Sets S.t_cut,
  // S.i_cut, S.z_kept (the mass kept with the tokens above), and S.again if the sums in fp32
  // do not decide it.
  __device__ void walk(int n, const double (&v)[3], int k, bool whole_known, bool use_p, double p,
                       bool pairs) {
    constexpr int kPer = kList / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    n = min(n, k);
    double w[kPer], ws = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      w[j] = 0;
      if (i < n) {
        if (pairs) {
          float h, l;
          w_pair(list_l(i), h, l);
          w[j] = (double)h + l;
        } else {
          w[j] = w_of(list_l(i));
        }
      }
      ws += w[j];
    }
    double wi = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double d = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += d;
    }
    if (lane == 31) S.wmass[wid] = wi;
    if (tid == 0) {
      S.n_keep = n;
      S.again = 0;
    }
    __syncthreads();
    double w0 = v[0] + wi - ws, all = v[0];
    for (int q = 0; q < kWarps; ++q) {
      if (q < wid) w0 += S.wmass[q];
      all += S.wmass[q];
    }
    const double whole = whole_known ? v[2] : all, goal = p * whole, near = pairs ? 0 : kNear * whole;
    if (use_p) {
      double run = w0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        if (i < n) {
          // token i is kept if the mass before it is short of the goal
          if (i > 0 && fabs(run - goal) <= near) S.again = 1;
          const bool kept = i == 0 || run < goal;
          run += w[j];
          if (kept && (i + 1 == n || !(run < goal))) S.n_keep = i + 1;
        }
      }
    }
    __syncthreads();
    const int keep = S.n_keep;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      w0 += w[j];
      if (tid * kPer + j == keep - 1) {
        S.z_kept = w0;
        S.t_cut = list_l(keep - 1);
        S.i_cut = (int)(uint32_t)S.list[keep - 1];
      }
    }
    __syncthreads();
  }

  // Of the row's tokens that equal t, the index of the nth (from 1): into S.i_cut of every CTA.
  __device__ void nth_equal(float t, long long nth) {
    // a contiguous run of slots for each thread
    const int slots = groups * V::N, per = (slots + kThreads - 1) / kThreads;
    const int a = min(slots, (int)threadIdx.x * per), z = min(slots, a + per);
    const bool limited = lim.i != 0x7fffffff;
    auto at = [&](int i) { return V::one(data, i) == t && (!limited || left(t, i - shift)); };
    int mine = 0;
    for (int i = a; i < z; ++i) mine += at(i);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    __syncthreads();
    if (lane == 31) S.wcnt[wid] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < wid) before += S.wcnt[w];
      total += S.wcnt[w];
    }
    if (threadIdx.x == 0)
      for (int r = 0; r < C; ++r) cl.map_shared_rank(&S, r)->part[set][rank][0] = (double)total;
    cl.sync();
    for (int r = 0; r < rank; ++r) before += (long long)S.part[set][r][0];
    set ^= 1;
    if (before < nth && nth <= before + mine) {
      for (int i = a; i < z; ++i)
        if (at(i) && ++before == nth) {
          for (int r = 0; r < C; ++r) cl.map_shared_rank(&S, r)->i_cut = first + i - shift;
          break;
        }
    }
    cl.sync();
  }

  // One filter's end (k > 0: top-k, with top-p at once where the list holds all that top-k keeps;
  // else top-p of what is left).  Sets lim; returns the mass kept; done_p: top-p is applied.
  __device__ double cut(int k, bool use_p, double p, bool& done_p) {
    const bool by_count = k > 0;
    // 1: buckets of (m - l) / T
    histogram([&](float l, int i) {
      if (l < lim.t || !left(l, i)) return -1;
      return (int)fminf(y_of(l), (float)(kBuckets - 1));
    });
    locate(!by_count, (unsigned)k, p, [](int b) { return ex2((b + 0.5f) * (-1.f / kPerOctave)); });
    // 2: the bracket [f_lo, f_hi): `before` tokens above it, `in` in it, of `total`
    unsigned before = S.cum_before, in = S.cum_in;
    const unsigned total = S.total;
    const int b1 = S.b_at, b0 = before + in <= (unsigned)kList ? 0 : b1;
    if (b0 == 0) {  // everything down to it fits the list
      in += before;
      before = 0;
    }
    if (threadIdx.x < 32) {
      const float lo = b1 == kBuckets - 1 ? -FLT_MAX : edge(b1 + 1);
      const float hi = b0 == 0 ? INFINITY : edge(b0);
      if (threadIdx.x == 0) {
        S.f_lo = lo;
        S.f_hi = hi;
      }
    }
    __syncthreads();
    float f_lo = S.f_lo, f_hi = S.f_hi;
    // the end lies in [out_lo, out_hi), with out_before tokens above and out_below below
    float out_lo = -FLT_MAX, out_hi = INFINITY;
    unsigned out_before = 0, out_below = 0;
    bool pairs = false;
    double v[3];
    // (each round halves the outer range at least once or cuts it into 2048: far fewer are needed)
    for (int round = 0; round < 100; ++round) {
      const bool gather = in <= (unsigned)kList;
      evaluate(f_lo, f_hi, gather, v);
      if (pairs) evaluate_pairs(f_lo, f_hi, v);
      if (!by_count) {
        // does the bracket hold the end?
        if (!pairs && (fabs(v[0] - p * v[2]) <= kNear * v[2] ||
                       fabs(v[0] + v[1] - p * v[2]) <= kNear * v[2])) {
          pairs = true;
          evaluate_pairs(f_lo, f_hi, v);
        }
        const double goal = p * v[2];
        if (before > out_before && !(v[0] < goal)) {
          out_lo = f_lo = f_hi;
          f_hi = out_hi;
          out_below = total - before;
          in = before - out_before;
          before = out_before;
          continue;
        }
        if (f_lo > out_lo && v[0] + v[1] < goal && before + in + out_below < total) {
          out_hi = f_hi = f_lo;
          f_lo = out_lo;
          out_before = before = before + in;
          in = total - before - out_below;
          continue;
        }
      }
      if (gather) {
        // 3: the list, by the first CTA
        done_p = !by_count || before == 0;
        for (int pass = 0;; ++pass) {
          if (rank == 0) {
            if (pass == 0) {
              const int n = collect();
              if (threadIdx.x == 0) S.n_list = n;
              __syncthreads();
            }
            const int n = S.n_list;
            walk(n, v, by_count ? (int)min((unsigned)n, (unsigned)k - before) : n, !by_count,
                 use_p && done_p, p, pairs);
            if (threadIdx.x == 0)
              for (int r = 1; r < C; ++r) {
                Shared* o = cl.map_shared_rank(&S, r);
                o->t_cut = S.t_cut;
                o->i_cut = S.i_cut;
                o->z_kept = S.z_kept;
                o->again = S.again;
              }
          }
          cl.sync();
          if (!S.again || pairs) break;
          pairs = true;
          evaluate_pairs(f_lo, f_hi, v);
        }
        lim.t = S.t_cut;
        lim.i = S.i_cut;
        const double z = S.z_kept;
        cl.sync();
        return z;
      }
      const uint32_t ka = code_of(f_lo), kz = f_hi == INFINITY ? code_of(m) : code_of(f_hi) - 1;
      if (kz <= ka) {
        // equal logits: a number of them, the lowest indices first
        double w1 = w_of(f_lo);
        long long nth = (long long)k - before;
        if (!by_count) {
          double need = (p * v[2] - v[0]) / w1;
          if (!pairs && fabs(need - rint(need)) * w1 <= kNear * v[2]) {
            pairs = true;
            evaluate_pairs(f_lo, f_hi, v);
          }
          if (pairs) {
            float h, l;
            w_pair(f_lo, h, l);
            w1 = (double)h + l;
            need = (p * v[2] - v[0]) / w1;
          }
          nth = (long long)ceil(need);
        }
        nth = max(1ll, min(nth, (long long)in));
        nth_equal(f_lo, nth);
        lim.t = f_lo;
        lim.i = S.i_cut;
        done_p = !by_count;
        cl.sync();
        return v[0] + nth * w1;
      }
      // 2 again: the bracket is cut by the codes of its logits
      out_lo = f_lo;
      out_hi = f_hi;
      out_before = before;
      out_below = total - before - in;
      int sh = 0;
      while (((kz - ka) >> sh) >= (uint32_t)kBuckets) ++sh;
      histogram([&](float l, int i) {
        if (!(l >= f_lo && l < f_hi) || l < lim.t || !left(l, i)) return -1;
        return (int)((kz - code_of(l)) >> sh);
      });
      locate(!by_count, (unsigned)k - before, by_count ? 0. : (p * v[2] - v[0]) / v[1], [&](int b) {
        const uint32_t off = ((uint32_t)b << sh) + ((1u << sh) >> 1);
        return w_of(float_of(off > kz - ka ? ka : kz - off));
      });
      const uint32_t top = kz - ((uint32_t)S.b_at << sh);
      f_lo = float_of(top - ka < (1u << sh) ? ka : top - (1u << sh) + 1);
      if (top < kz) f_hi = float_of(top + 1);
      before += S.cum_before;
      in = S.cum_in;
    }
    done_p = false;
    return v[2];
  }
};

// (score, index) of the better: higher score, lower index.
__device__ __forceinline__ void better(double& s, int& i, double s2, int i2) {
  if (s2 > s || (s2 == s && i2 < i)) {
    s = s2;
    i = i2;
  }
}

template <typename T, typename P>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(const SampleArgs a, int chunk, int data_bytes) {
  using V = Vec<T>;
  extern __shared__ __align__(16) uint8_t smem[];
  T* data = reinterpret_cast<T*>(smem);
  Shared& S = *reinterpret_cast<Shared*>(smem + data_bytes);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  pdl_release();
  pdl_wait();

  // the row's parameters (every decision below is the same in all threads of the cluster)
  const int req = a.row_req ? a.row_req[row] : row;
  if (req < 0) return;
  bool bad = req >= a.B;
  float temp = 1.f, p = 1.f, mp = 0.f;
  int k = 0;
  if (!bad) {
    if (a.temperature) temp = a.temperature[req];
    if (a.top_k) k = a.top_k[req];
    if (a.top_p) p = a.top_p[req];
    if (a.min_p) mp = a.min_p[req];
    bad = !(temp == 0.f || (temp >= 0x1p-60f && temp <= 0x1p60f)) || !(p == p) || !(mp == mp);
  }
  if (bad) {
    if (rank == 0 && tid == 0) raise_error(a.err, DSPARK_DEVERR_BAD_INPUT);
    return;
  }
  const bool greedy = temp == 0.f;
  if (greedy) temp = p = 1.f, k = 0, mp = 0.f;
  mp = fminf(mp, 1.f);
  if (p <= 0.f) p = 1.f, k = 1;  // the first token alone
  const bool use_k = k > 0 && k < a.V, use_p = p < 1.f;
  cl.barrier_arrive();  // (waited for before the first access to another CTA's memory)

  Row<T> R{cl, S, data};
  R.C = C;
  R.rank = rank;
  R.first = min(a.V, rank * chunk);
  R.n = min(a.V, R.first + chunk) - R.first;
  R.set = 0;
  const T* src = static_cast<const T*>(a.logits) + row * a.stride + R.first;
  R.shift = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  R.groups = (R.n + R.shift + V::N - 1) / V::N;
  if (R.n == 0) R.groups = 0;

  if (tid == kThreads - 1) {  // (while the others load)
    const double c = 1.4426950408889634074 / (double)temp;
    S.c_hi = (float)c;
    S.c_lo = (float)(c - (double)S.c_hi);
    S.log_min = mp > 0.f ? (double)temp * log((double)mp) : 0.0;
  }
  // the chunk into shared memory, and its maximum
  float mx = -INFINITY;
  {
    const uint4* g = reinterpret_cast<const uint4*>(src - R.shift);
    uint4* d = reinterpret_cast<uint4*>(data);
    for (int q = tid; q < R.groups; q += kThreads) {
      const int e0 = q * V::N - R.shift;
      float x[V::N];
      if (e0 >= 0 && e0 + V::N <= R.n) {
        V::get(g[q], x);
      } else {
#pragma unroll
        for (int j = 0; j < V::N; ++j)
          x[j] = (e0 + j >= 0 && e0 + j < R.n) ? V::one(src, e0 + j) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < V::N; ++j) {
        x[j] = clean(x[j], V::kTop);
        mx = fmaxf(mx, x[j]);
      }
      d[q] = V::put(x);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) S.wmax[wid] = mx;
  __syncthreads();
  cl.barrier_wait();
  if (tid < C) {
    float v = S.wmax[0];
    for (int w = 1; w < kWarps; ++w) v = fmaxf(v, S.wmax[w]);
    cl.map_shared_rank(&S, tid)->cmax[rank] = v;
  }
  cl.sync();
  float m = S.cmax[0];
  for (int r = 1; r < C; ++r) m = fmaxf(m, S.cmax[r]);
  R.m = m;
  R.s = S.c_hi * kPerOctave;
  P* const probs = a.probs ? static_cast<P*>(a.probs) + (long long)row * a.V + R.first : nullptr;
  const float* const noise = a.noise ? a.noise + (long long)row * a.V + R.first : nullptr;
  if (m == -INFINITY) {  // no token is left to draw from
    if (probs)
      for (int i = tid; i < R.n; i += kThreads) probs[i] = P(0.f);
    if (a.tokens && rank == 0 && tid == 0) a.tokens[row] = -1;
    cl.sync();
    return;
  }
  R.lim.t = -FLT_MAX;
  R.lim.i = 0x7fffffff;
  if (mp > 0.f) {
    const double t = (double)m + S.log_min;
    float f = (float)t;
    if ((double)f < t) f = float_of(code_of(f + 0.f) + 1);
    R.lim.t = fmaxf(fminf(f, m), -FLT_MAX);
  }

  // the filters
  double z = -1;
  bool done_p = false;
  if (greedy) {
    R.nth_equal(m, 1);
    R.lim.t = m;
    R.lim.i = S.i_cut;
  }
  if (use_k) z = R.cut(k, use_p, p, done_p);
  if (use_p && !done_p) z = R.cut(0, true, p, done_p);
  if (z < 0 && probs) {
    double v[3];
    R.evaluate(INFINITY, INFINITY, false, v);
    z = v[2];
  }
  const float inv = probs ? (float)(1.0 / z) : 0.f;

  // the distribution, and each thread's two best in the race
  float b1 = -1.f, b2 = -1.f;
  int i1 = 0x7fffffff, i2 = 0x7fffffff;
  const bool race = a.tokens != nullptr;
  if (race || probs) {
    for (int i = tid; i < R.n; i += kThreads) {
      const float l = V::one(data, i + R.shift);
      const bool keep = R.left(l, i);
      const float w = keep ? R.w_of(l) : 0.f;
      if (probs) probs[i] = P(w * inv);
      if (race && keep) {
        const float sc = __fdividef(w, noise[i]);
        if (sc > b1) {
          b2 = b1;
          i2 = i1;
          b1 = sc;
          i1 = i;
        } else if (sc > b2) {
          b2 = sc;
          i2 = i;
        }
      }
    }
  }
  if (!race) {
    cl.sync();
    return;
  }
  // the best in fp32, then in 64 bits among those that come near it
  float bb = b1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bb = fmaxf(bb, __shfl_xor_sync(0xffffffffu, bb, o));
  if (lane == 0) S.best[wid] = bb;
  __syncthreads();
  if (tid < C) {
    float v = S.best[0];
    for (int w = 1; w < kWarps; ++w) v = fmaxf(v, S.best[w]);
    cl.map_shared_rank(&S, tid)->c_best[rank] = v;
  }
  cl.sync();
  float top = S.c_best[0];
  for (int r = 1; r < C; ++r) top = fmaxf(top, S.c_best[r]);
  const float near = top * (1.f - 0x1p-16f);  // (fp32's error is 2^-18 at most)
  double rs = -INFINITY;
  int ri = 0x7fffffff;
  auto precise = [&](float b, int i) {
    if (i == 0x7fffffff || !(b >= near)) return;
    const double l = V::one(data, i + R.shift);
    better(rs, ri, (l - (double)m) / (double)temp - log((double)noise[i]), R.first + i);
  };
  precise(b1, i1);
  precise(b2, i2);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    better(rs, ri, __shfl_xor_sync(0xffffffffu, rs, o), __shfl_xor_sync(0xffffffffu, ri, o));
  if (lane == 0) {
    S.r_best[wid] = rs;
    S.r_idx[wid] = ri;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) better(rs, ri, S.r_best[w], S.r_idx[w]);
    Shared* o = cl.map_shared_rank(&S, 0);
    o->cr_best[rank] = rs;
    o->cr_idx[rank] = ri;
  }
  cl.sync();
  if (rank == 0 && tid == 0) {
    rs = S.cr_best[0];
    ri = S.cr_idx[0];
    for (int r = 1; r < C; ++r) better(rs, ri, S.cr_best[r], S.cr_idx[r]);
    a.tokens[row] = ri == 0x7fffffff ? -1 : ri;
  }
}

template <typename T, typename P>
int launch(const SampleArgs& a, cudaStream_t stream) {
  const long long row_bytes = (long long)a.V * sizeof(T);
  int C = 1;
  while (C < kMaxCluster && row_bytes > (long long)C * kChunkBytes) C *= 2;
  const int chunk = ((a.V + C - 1) / C + 7) / 8 * 8;
  // (a chunk that begins anywhere in a 16-byte group touches one group more)
  const int data_bytes = chunk * (int)sizeof(T) + 16;
  const int smem = data_bytes + (int)sizeof(Shared);
  static PerDevice<bool> done;
  if (!once_per_device(done, false, [] {
        return cudaFuncSetAttribute(sample_kernel<T, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    227 * 1024) == cudaSuccess;
      }))
    return DSPARK_ECUDA;
  return launch_pdl_cluster(sample_kernel<T, P>, dim3((unsigned)(a.rows * C)), dim3(kThreads),
                            (size_t)smem, stream, C, a, chunk, data_bytes) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ECUDA;
}

}  // namespace

int launch_sample(const SampleArgs& a, int dtype, int probs_dtype, cudaStream_t stream) {
  if (dtype == DSPARK_F32)
    return probs_dtype == DSPARK_F32 ? launch<float, float>(a, stream)
                                     : launch<float, __nv_bfloat16>(a, stream);
  return probs_dtype == DSPARK_F32 ? launch<__nv_bfloat16, float>(a, stream)
                                   : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace dspark
