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
//   1  tokens are counted in 2048 buckets of (m - l) / T, 1/64 of an octave of w each;
//   2  a bracket of buckets that should hold the end is taken (for top-p by masses that the counts
//      estimate), and one pass sums the masses above and in it and lists its tokens;
//   3  one CTA sorts the list and walks it.
// Before that a bound from below takes out what cannot be kept (for top-k from the threads' largest
// logits, the best of the CTAs' bounds; for top-p from the row's mass): with k up to some hundred what
// passes it fits the list at once.  A bracket that does not hold the end gives way to what lies above or below it, one of more
// than kList tokens is cut again by the bits of its logits, and one that holds a single value is
// resolved by counting indices.  Where a sum comes so near to the border that fp32 cannot tell on
// which side the end lies (near_of), sums are taken again in pairs of fp32 numbers (2^-36 or so): the
// kept set is that of the definition in 64 bits.
//
// What bounds it: instructions, and the meetings of the cluster (some eight a row, 1500 cycles each).
// A pass over a chunk costs 6000 cycles for two CTAs of an SM, loading it 7000.  One row of 151936:
// 16 us; 288 such rows with distributions 234 to 246 us (56 at the copy rate); 1024 rows of 129280 in bf16,
// top-p with wide nuclei, 655 to 670 us (39; 108 instructions a token).  512 threads with 76 KB, two to an
// SM: at a stage when these took 874 us for the last, 256 threads with 38 KB (larger clusters) took 1143
// and 1024 with 152 KB 926.

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
constexpr float kPerOctave = 64.f;
constexpr int kList = 1024;            // tokens of a bracket that are sorted
constexpr int kMaxCluster = 8;
constexpr int kChunkBytes = 76 * 1024; // of a row in one CTA, while eight CTAs hold the row
// Masses from fp32 are summed in fixed point, 44 bits behind the point (w <= 1, V <= 400000: below
// 2^63): without the card's slow 64-bit floating point, which the sums in pairs need.
typedef long long mass_t;
constexpr float kUnit = 0x1p44f;
// Error that a sum of w in fp32 may have against p of the whole, where it lies near that; of n tokens.
// u = 2^-24, a = p and b = 1 - p the parts before the border and behind it, W the whole.
//   w of a token x octaves below the top: its exponent has the roundings of m - l, of the product and of
//   the factor, each u, and u / 4 from log2(e): ln 2 u x of w for each.  Equal logits share them, so
//   nothing averages out.  With X and Y the mean octaves of the two parts the sum is off by at most
//   ln 2 u a b (1.25 (Y - X) + 2 (X + Y)) W, the factor's error being one for all.  A part of mass M
//   and n tokens has a mean of log2(n / M) octaves at most.
//   The exponential is off by 2^-22 of w: 8 a b u W.
//   The sums themselves (Sum): 2 u each, W being 1 at least.
// (At most W / 16, which none of this reaches but a p so small that n / a is infinite.)
__device__ __forceinline__ float near_of(float p, float whole, int n) {
  const float a = p * whole, b = (1 - p) * whole;
  const float x = __log2f(__fdividef(n, a)), y = __log2f(__fdividef(n, b));
  return fminf(0x1p-24f * ((1 - p) * a * (2.3f * y + 1.4f * x + 8.5f) + 4.f), whole / 16);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 d;
  const float2 one = make_float2(-1.f, -1.f);
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<const uint64_t&>(one)),
        "l"(reinterpret_cast<uint64_t&>(a)));
  return d;
}
// Two running sums of w (0 <= w <= 1) that keep what each addition rounds away: they begin at 1, so that
// the sum is the larger addend and that is exact.  What is lost of n tokens is n u (1 + sum) at most and
// its own sum is off by n u of that: over 8192 sums of 49 tokens (the most there are) 1.1 u.
struct Sum {
  float2 s = make_float2(1.f, 1.f), lost = make_float2(0.f, 0.f);
  __device__ __forceinline__ void add(float a, float b) {
    const float2 w = make_float2(a, b), t = add2(s, w);
    lost = add2(lost, sub2(w, sub2(t, s)));
    s = t;
  }
  __device__ __forceinline__ mass_t fixed() const {
    return __float2ll_rn((s.x - 1) * kUnit) + __float2ll_rn((s.y - 1) * kUnit) +
           __float2ll_rn((lost.x + lost.y) * kUnit);
  }
};
// Error of the mass above a bracket beside that (list_by).
__device__ __forceinline__ mass_t slack_of(mass_t above, mass_t in) { return above != 0 ? in >> 17 : 0; }
// What lies before a kept token is short of p of the whole (0 < p < 1).
__device__ __forceinline__ mass_t goal_of(float p, mass_t whole) {
  const unsigned long long f = __float2ull_rn(p * 0x1p64f), w = whole;
  return (mass_t)__umul64hi(f, w) + (f * w != 0);
}
__device__ __forceinline__ double goal_of(float p, double whole) { return (double)p * whole; }
__device__ __forceinline__ mass_t distance(mass_t a, mass_t b) { return a > b ? a - b : b - a; }

struct Shared {
  unsigned hist[kBuckets];             // this CTA's counts
  unsigned tot[kBuckets];              // the row's, in order of falling logits
  uint64_t list[kList];                // (order of the logit, index)
  unsigned long long part[2][kMaxCluster][3];  // exchanged between the CTAs, two sets in turn
  float cmax[kMaxCluster], cleast[kMaxCluster];
  unsigned long long wsum[kWarps][3];
  float wmax[kWarps];
  unsigned wcnt[kWarps];
  unsigned long long wmass[kWarps];
  float wapprox[kWarps];
  float e2h[17], e2l[17];              // 2^(-j / 16), j = -8 .. 8, in two parts
  float c_hi, c_lo;                    // log2(e) / T in two parts
  double log_min;                      // T ln(min_p)
  int n_list, n_sorted;                // tokens that this CTA listed; of all, sorted (the first CTA's)
  // a decision of one thread or CTA for all
  int b_at;
  unsigned cum_before, cum_in, total;
  float f_lo, f_hi, t_cut;
  int i_cut, n_keep, again;
  float z_kept;
  int n_near[kMaxCluster];             // of each CTA: tokens near the race's best
  double r_best[kWarps];
  int r_idx[kWarps];
  float c_best[kMaxCluster];
  double cr_best[kMaxCluster];
  int cr_idx[kMaxCluster];
};

// Order-preserving code of a float (no NaN; -0 as 0).
__device__ __forceinline__ uint32_t code_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
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

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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

struct Kept {    // tokens with l > t, or l == t and an index of at most i
  float t;
  int i;
};

// A thread's two best in the race, the lower index first among equals as they come.  (Where the second
// comes near the row's best the race is run again in 64 bits.)
constexpr int kNone = 0x7fffffff;
struct Racer {
  float s1 = -0x1p-60f, s2 = -0x1p-60f, l1 = 0.f, l2 = 0.f;
  int i1 = kNone, i2 = kNone;
  __device__ __forceinline__ void take(float s, float l, int i) {
    if (s > s1) {
      s2 = s1; l2 = l1; i2 = i1;
      s1 = s; l1 = l; i1 = i;
    } else if (s > s2) {
      s2 = s; l2 = l; i2 = i;
    }
  }
};

template <typename T>
struct Row {
  using V = Vec<T>;
  cg::cluster_group cl;
  Shared& S;
  const T* data;      // slots of this CTA's chunk in shared memory
  int C, rank;
  int first, n;       // the chunk: tokens first .. first + n - 1,
  int n_row;          // of so many
  int shift, groups;  // token i of the chunk is slot i + shift; 16-byte groups of slots
  int set;            // of S.part
  float m, s, nc;     // largest logit; buckets and (negative) octaves per unit of logit
  float t_min;        // least logit that min-p leaves
  Kept lim;           // what earlier filters left, and of that what this one may keep
  Kept lim_all;       // what earlier filters left
  float k_least;      // a logit that k of the row's tokens reach (-inf: none is known)
  mass_t whole;       // its mass (weigh)
  int n_listed;       // tokens of the last list, in all CTAs (more than kList: it is not whole)
  bool sorted;        // the list in the first CTA is
  bool listed;        // it is the first S.n_keep tokens of the first CTA's list
  bool lost;          // the search contradicted itself (counts of one bracket that differ, no end)

  // (rounded by the addition of 2^23: monotone in l, which is all that is asked)
  __device__ __forceinline__ int bucket_of(float l) const {
    return __float_as_int(fminf((m - l) * s, (float)(kBuckets - 1)) + 0x1p23f) & (kBuckets - 1);
  }
  __device__ __forceinline__ float w_of(float l) const { return ex2((m - l) * nc); }
  __device__ __forceinline__ bool left(float l, int i) const {
    return l > lim.t || (l == lim.t && first + i <= lim.i);
  }

  // fn(l, i, j) for every token i of the chunk, j its place in its 16 bytes.
  template <class Fn>
  __device__ __forceinline__ void each(Fn&& fn) const {
    const uint4* p = reinterpret_cast<const uint4*>(data);
    for (int q = threadIdx.x; q < groups; q += kThreads) {
      float x[V::N];
      V::get(p[q], x);
#pragma unroll
      for (int j = 0; j < V::N; ++j) fn(x[j], q * V::N + j - shift, j);
    }
  }

  // fn(l, in, i, j) for the tokens of the groups that have one with l >= least, in: it is such a one and
  // (LIMITED) left.  The others cost a maximum a group.  fn should not branch: in a warp with any
  // such token all of it runs.
  template <bool LIMITED, class Fn>
  __device__ __forceinline__ void each_from(float least, Fn&& fn) const {
    const uint4* p = reinterpret_cast<const uint4*>(data);
    for (int q = threadIdx.x; q < groups; q += kThreads) {
      float x[V::N];
      V::get(p[q], x);
      float top = x[0];
#pragma unroll
      for (int j = 1; j < V::N; ++j) top = fmaxf(top, x[j]);
      if (top >= least)
#pragma unroll
        for (int j = 0; j < V::N; ++j) {
          const int i = q * V::N + j - shift;
          fn(x[j], x[j] >= least && (!LIMITED || left(x[j], i)), i, j);
        }
    }
  }
  template <class Fn>
  __device__ __forceinline__ void each_left_from(float least, Fn&& fn) const {
    if (lim.i == kNone) each_from<false>(least, fn);
    else each_from<true>(least, fn);
  }

  __device__ __forceinline__ mass_t near_fixed(float p, mass_t of) const {
    return __float2ll_ru(near_of(p, (float)of * (1.f / kUnit), n_row) * kUnit);
  }

  // Sums of three numbers (mass_t or double) over the row, the same in every thread of the cluster and
  // in fixed order.
  template <typename M>
  __device__ __forceinline__ void sum3(M (&v)[3]) {
    static_assert(sizeof(M) == 8, "a word of the exchange");
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < 3; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    __syncthreads();
    M* const ws = reinterpret_cast<M*>(&S.wsum[0][0]);
    if (lane < 3) ws[3 * wid + lane] = lane == 0 ? v[0] : lane == 1 ? v[1] : v[2];
    __syncthreads();
    // thread (r, k): this CTA's sum k to CTA r
    if (threadIdx.x < 4 * C && (threadIdx.x & 3) < 3) {
      const int k = threadIdx.x & 3;
      M a = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += ws[3 * w + k];
      *reinterpret_cast<M*>(&cl.map_shared_rank(&S, threadIdx.x >> 2)->part[set][rank][k]) = a;
    }
    cl.sync();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      v[k] = 0;
      for (int r = 0; r < C; ++r) v[k] += *reinterpret_cast<const M*>(&S.part[set][r][k]);
    }
    set ^= 1;
  }

  // Counts of the row's tokens by bucket(l) (0 .. kBuckets - 1, or negative: not counted), into
  // S.tot of every CTA.
  template <class Fn>
  __device__ void histogram(Fn&& bucket) {
    __syncthreads();
    for (int b = threadIdx.x; b < kBuckets; b += kThreads) S.hist[b] = 0;
    __syncthreads();
    each_left_from(lim.t, [&](float l, bool in, int, int) {
      const int b = bucket(l);
      if (in && b >= 0) atomicAdd(&S.hist[b], 1u);
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
  // mass reaches `share`, of_total of the whole, the mass of bucket b being tot[b] * mass(b).
  // Sets S.b_at, S.cum_before (tokens in the buckets before), S.cum_in and S.total.
  template <class Fn>
  __device__ void locate(bool weighted, unsigned target, float share, bool of_total, Fn&& mass) {
    constexpr int kPer = kBuckets / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    unsigned c[kPer];
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
      const uint4 t4 = reinterpret_cast<const uint4*>(S.tot)[(tid * kPer + j) / 4];
      c[j] = t4.x;
      c[j + 1] = t4.y;
      c[j + 2] = t4.z;
      c[j + 3] = t4.w;
    }
    unsigned cs = 0;
    float w[kPer], ws = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      w[j] = weighted && c[j] ? c[j] * mass(tid * kPer + j) : 0.f;
      cs += c[j];
      ws += w[j];
    }
    unsigned ci = cs;
    float wi = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, ci, o);
      const float d = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) {
        ci += u;
        wi += d;
      }
    }
    __syncthreads();
    if (lane == 31) {
      S.wcnt[wid] = ci;
      S.wapprox[wid] = wi;
    }
    if (tid == 0) S.b_at = 0x7fffffff;
    __syncthreads();
    unsigned c0 = ci - cs, last = 0;
    float w0 = wi - ws, total = 0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) {
      if (v < wid) {
        c0 += S.wcnt[v];
        w0 += S.wapprox[v];
      }
      total += S.wapprox[v];
      last += S.wcnt[v];
    }
    const float goal = of_total ? share * total : share;
    const unsigned c_first = c0;
    if (tid == 0) S.total = last;
    // (of masses the first bucket that ends past the goal: fp32 sums of two threads need not join)
    int mine = -1;
    unsigned m_before = 0, m_in = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const bool here = weighted ? (c[j] && w0 + w[j] >= goal)
                                 : (c0 < target && c0 + c[j] >= target);
      if (here && mine < 0) {
        mine = tid * kPer + j;
        m_before = c0;
        m_in = c[j];
        atomicMin(&S.b_at, mine);
      }
      c0 += c[j];
      w0 += w[j];
    }
    __syncthreads();
    if (mine >= 0 && S.b_at == mine) {
      S.cum_before = m_before;
      S.cum_in = m_in;
    }
    __syncthreads();
    if (S.b_at == 0x7fffffff) {  // the goal lies past the last token (rounding): the last bucket that holds one
      __syncthreads();
      c0 = c_first;
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

  // The least float l with a bucket below `bound`; buckets fall as l grows, so 32 lanes halve the codes
  // five bits at a time.  By a warp.
  __device__ float edge(int bound) const {
    const int lane = threadIdx.x & 31;
    uint32_t lo = code_of(-FLT_MAX), hi = code_of(m);  // (bucket 0)
    // a few roundings around the inverse, if it lies between them: two rounds in place of seven
    const float at = m - (bound - 0.5f) / s, off = 4e-7f * (fabsf(m) + fabsf(at));
    if (at - off > -FLT_MAX && at + off < m && bucket_of(at + off) < bound && bucket_of(at - off) >= bound) {
      lo = code_of(at - off + 0.f);
      hi = code_of(at + off + 0.f);
    }
    while (hi > lo) {
      const uint32_t step = (hi - lo + 31) / 32, at = lo + min((unsigned)lane * step, hi - lo);
      const unsigned ok = __ballot_sync(0xffffffffu, bucket_of(float_of(at)) < bound);
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

  // The mass of the tokens left, into `whole`.
  __device__ void weigh() {
    Sum all;
    float even = 0.f;
    auto take = [&](float w, int j) {
      if (j & 1) all.add(even, w);
      else even = w;
    };
    if (lim.t == -FLT_MAX) {
      each([&](float l, int, int j) { take(w_of(l), j); });
    } else {
      each_left_from(lim.t, [&](float l, bool in, int, int j) { take(in ? w_of(l) : 0.f, j); });
    }
    mass_t v[3] = {all.fixed(), 0, 0};
    sum3(v);
    whole = v[0];
  }
  // Of the tokens left with l >= least: lists those of place 1 and adds up the masses of those of
  // place 0, which lie above them (none_above: none do), and 1 (place(l): 0, 1 or 2, no part), over the
  // row.  Their sum is exact as Sum is, the second mass alone to 98 u (a thread's tokens one by one), and
  // so is the first's part in their sum: slack_of.
  template <class Fn>
  __device__ __forceinline__ void list_by(float least, bool gather, bool none_above, mass_t (&v)[3], Fn&& place) {
    __syncthreads();
    if (threadIdx.x == 0) S.n_list = 0;
    __syncthreads();
    Sum down;
    float even = 0.f;
    float in = 0.f;
    int count = 0;
    each_left_from(least, [&](float l, bool is, int i, int j) {
      const int at = is ? place(l) : 2;
      const float w = w_of(l), part = at <= 1 ? w : 0.f;
      if (j & 1) down.add(even, part);
      else even = part;
      if (at == 1) {
        in += w;
        ++count;
        if (gather && *(volatile int*)&S.n_list < kList) {
          const int slot = atomicAdd(&S.n_list, 1);
          if (slot < kList) S.list[slot] = (uint64_t)(~code_of(l)) << 32 | (uint32_t)(first + i);
        }
      }
    });
    v[0] = down.fixed();
    v[1] = __float2ll_rn(in * kUnit);
    v[2] = count;
    sum3(v);
    n_listed = (int)v[2];
    if (none_above) v[1] = v[0];
    v[0] -= v[1];
    v[2] = whole;
  }
  // The bracket [f_lo, f_hi).
  __device__ void evaluate(float f_lo, float f_hi, bool gather, bool none_above, mass_t (&v)[3]) {
    list_by(fmaxf(f_lo, lim.t), gather, none_above, v, [&](float l) { return l >= f_hi ? 0 : 1; });
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

  // w_pair's table, before its first use in a row.
  __device__ void make_table() {
    __syncthreads();
    if (threadIdx.x < 17) {
      const double e = exp2(-((int)threadIdx.x - 8) / 16.0);  // (few: 64 bits are slow here)
      S.e2h[threadIdx.x] = (float)e;
      S.e2l[threadIdx.x] = (float)(e - (double)(float)e);
    }
    __syncthreads();
  }
  // list_by's masses in pairs, v[2] that of all tokens that earlier filters left.
  template <class Fn>
  __device__ __forceinline__ void weigh_pairs(double (&v)[3], Fn&& place) {
    make_table();
    float ah = 0, al = 0, ih = 0, il = 0, bh = 0, bl = 0;
    auto add = [](float& sh, float& sl, float wh, float wl) {
      const float t = sh + wh, z = t - sh;
      sl += ((sh - (t - z)) + (wh - z)) + wl;
      sh = t;
    };
    each([&](float l, int i, int) {
      if (l < lim_all.t || (l == lim_all.t && first + i > lim_all.i)) return;
      float wh, wl;
      w_pair(l, wh, wl);
      const int at = place(l);
      if (at == 0) add(ah, al, wh, wl);
      else if (at == 1) add(ih, il, wh, wl);
      else add(bh, bl, wh, wl);
    });
    v[0] = (double)ah + al;
    v[1] = (double)ih + il;
    v[2] = v[0] + v[1] + ((double)bh + bl);
    sum3(v);
  }
  __device__ void evaluate_pairs(float f_lo, float f_hi, double (&v)[3]) {
    weigh_pairs(v, [&](float l) { return l >= f_hi ? 0 : l >= f_lo ? 1 : 2; });
  }
  __device__ __forceinline__ void w_exact(float l, double& w) const {
    float h, t;
    w_pair(l, h, t);
    w = (double)h + t;
  }
  __device__ __forceinline__ void w_exact(float l, mass_t& w) const { w = __float2ll_rn(w_of(l) * kUnit); }

  // The lists of all CTAs into this one's, sorted; n tokens in all (at most kList).
  __device__ int collect() {
    // (every rank's list was written before the last cl.sync); token i of all of them
    int n = 0, from[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      from[r] = n;
      n += r < C ? min(cl.map_shared_rank(&S, r)->n_list, kList) : 0;
    }
    n = min(n, kList);
    constexpr int kEach = kList / kThreads;
    uint64_t mine[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = threadIdx.x + j * kThreads;
      int r = 0;
#pragma unroll
      for (int q = 1; q < kMaxCluster; ++q)
        if (q < C && i >= from[q]) r = q;
      int base = 0;
#pragma unroll
      for (int q = 1; q < kMaxCluster; ++q)
        if (q == r) base = from[q];
      if (i < n) mine[j] = cl.map_shared_rank(&S, r)->list[i - base];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (threadIdx.x + j * kThreads < n) S.list[threadIdx.x + j * kThreads] = mine[j];
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreads) S.list[i] = ~0ull;
    __syncthreads();
    // Bitonic.  A warp has 64 places to itself, two to a lane, in registers while the distance is below
    // 64 (through shared memory throughout: three times as long).
    static_assert(kList <= 64 * kWarps, "64 places a warp");
    const int lane = threadIdx.x & 31, base = (threadIdx.x >> 5) * 64;
    const bool part = base < size;
    uint64_t x = 0, y = 0;
    auto within = [&](int k) {  // the distances min(k, 64) / 2 .. 1 of phase k
      const bool up = k < 64 || (base & k) == 0;
      if (k >= 64 && (x > y) == up) {
        const uint64_t t = x;
        x = y;
        y = t;
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        if (d >= k) continue;
        const uint64_t a = __shfl_xor_sync(0xffffffffu, x, d), b = __shfl_xor_sync(0xffffffffu, y, d);
        // places base + lane and base + lane + 32
        const bool low = (lane & d) == 0;
        const bool up_x = k < 64 ? (lane & k) == 0 : up, up_y = k < 64 ? ((lane + 32) & k) == 0 : up;
        x = ((x > a) == (up_x == low)) ? a : x;
        y = ((y > b) == (up_y == low)) ? b : y;
      }
    };
    if (part) {
      x = S.list[base + lane];
      y = S.list[base + lane + 32];
#pragma unroll
      for (int k = 2; k <= 64; k <<= 1) within(k);
      S.list[base + lane] = x;
      S.list[base + lane + 32] = y;
    }
    __syncthreads();
    for (int k = 128; k <= size; k <<= 1) {
      for (int d = k >> 1; d >= 64; d >>= 1) {
        for (int i = threadIdx.x; i < size / 2; i += kThreads) {
          const int a = 2 * i - (i & (d - 1)), b = a + d;
          const uint64_t u = S.list[a], w = S.list[b];
          if ((u > w) == ((a & k) == 0)) {
            S.list[a] = w;
            S.list[b] = u;
          }
        }
        __syncthreads();
      }
      if (part) {
        x = S.list[base + lane];
        y = S.list[base + lane + 32];
        within(k);
        S.list[base + lane] = x;
        S.list[base + lane + 32] = y;
      }
      __syncthreads();
    }
    return n;
  }

  __device__ __forceinline__ float list_l(int i) const {
    return float_of(~(uint32_t)(S.list[i] >> 32));
  }

  // By the first CTA, over its sorted list of n tokens with masses v[0] above them and v[2] in all: the
  // end of the first `k` of them (k >= n: all) and, where use_p, of the part p of the whole, which is
  // v[2] or (list_only) what these k hold.  Sets S.t_cut, S.i_cut, S.z_kept (the mass kept with
  // what is above), and S.again if the sums in fp32 do not decide it.
  template <typename M>
  __device__ void walk(int n, const M (&v)[3], int k, bool list_only, bool use_p, float p) {
    constexpr bool kPairs = sizeof(M) == 8 && M(0.5f) != M(0);
    constexpr int kPer = kList / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    M* const wm = reinterpret_cast<M*>(S.wmass);
    n = min(n, k);
    M w[kPer], ws = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = tid * kPer + j;
      w[j] = 0;
      if (i < n) w_exact(list_l(i), w[j]);
      ws += w[j];
    }
    M wi = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const M d = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += d;
    }
    if (lane == 31) wm[wid] = wi;
    if (tid == 0) {
      S.n_keep = n;
      S.again = 0;
    }
    __syncthreads();
    // (each warp adds the totals before it up, and all of them)
    M t = lane < kWarps ? wm[lane] : M(0), all = t, part = lane < wid ? t : M(0);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      part += __shfl_xor_sync(0xffffffffu, part, o);
    }
    all = v[0] + __shfl_sync(0xffffffffu, all, 0);
    M w0 = v[0] + __shfl_sync(0xffffffffu, part, 0) + (wi - ws);
    if (use_p) {
      const M whole = list_only ? all : v[2], goal = goal_of(p, whole);
      const M near = kPairs ? M(0) : M(near_fixed(p, whole) + slack_of(v[0], v[1]));
      M run = w0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = tid * kPer + j;
        if (i < n) {
          // token i is kept if the mass before it is short of the goal
          if constexpr (!kPairs)
            if (i > 0 && distance(run, goal) <= near) S.again = 1;
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
        S.z_kept = kPairs ? (float)w0 : (float)w0 * (1.f / kUnit);
        S.t_cut = list_l(keep - 1);
        S.i_cut = (int)(uint32_t)S.list[keep - 1];
      }
    }
    __syncthreads();
  }

  // The lowest index among the largest logits.
  __device__ int first_top() {
    int at = kNone;
    each_from<false>(m, [&](float, bool in, int i, int) { at = min(at, in ? first + i : kNone); });
    at = __reduce_min_sync(0xffffffffu, at);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) S.r_idx[threadIdx.x >> 5] = at;
    __syncthreads();
    if (threadIdx.x < C) {
      for (int w = 0; w < kWarps; ++w) at = min(at, S.r_idx[w]);
      cl.map_shared_rank(&S, threadIdx.x)->n_near[rank] = at;
    }
    cl.sync();
    at = kNone;
    for (int r = 0; r < C; ++r) at = min(at, S.n_near[r]);
    return at;
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
      for (int r = 0; r < C; ++r) cl.map_shared_rank(&S, r)->part[set][rank][0] = (unsigned long long)total;
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

  // The end within a bracket whose tokens all CTAs have listed (kList in all at most): by the first
  // CTA, `before` tokens and masses v (d, where `pairs`) above it as in walk.  Sets lim, listed and z,
  // the mass kept; false, and none of them, if v does not tell (the list stays as it is, sorted).
  __device__ bool resolve(const mass_t (&v)[3], const double (&d)[3], bool pairs, unsigned before, int k,
                          bool use_p, float p, float& z) {
    if (rank == 0) {
      if (!pairs || !sorted) {
        const int n = collect();
        if (threadIdx.x == 0) S.n_sorted = n;
        __syncthreads();
      }
      const int n = S.n_sorted, most = k > 0 ? (int)min((unsigned)n, (unsigned)k - before) : n;
      if (pairs) make_table();  // (where the list has it all nothing was weighed in pairs before)
      if (pairs) walk(n, d, most, k > 0, use_p, p);
      else walk(n, v, most, k > 0, use_p, p);
      if (threadIdx.x > 0 && threadIdx.x < C) {
        Shared* o = cl.map_shared_rank(&S, threadIdx.x);
        o->t_cut = S.t_cut;
        o->i_cut = S.i_cut;
        o->z_kept = S.z_kept;
        o->again = S.again;
      }
    }
    cl.sync();
    sorted = S.again && !pairs;
    // (before they are written again the CTAs meet)
    if (sorted) return false;
    lim.t = S.t_cut;
    lim.i = S.i_cut;
    z = S.z_kept;
    whole = -1;
    listed = before == 0;
    return true;
  }

  // A logit below which the filter keeps nothing, from what is known before the row is searched.  The
  // same in all CTAs, as the bracket's ends in `cut` follow from it.
  __device__ float bound(int k, float p) {
    if (k > 0) return fmaxf(k_least, lim.t);
    // n tokens below weigh less than n times that one's w: the part 1 - p of the whole lies above
    const float x = log2f(2.f * n_row / ((1.f - p) * ((float)whole * (1.f / kUnit))));
    return fmaxf(m + fmaxf(x, 0.f) / nc, lim.t);
  }

  // The chunk's probabilities w inv (probs and noise: of the whole row), and the race.
  template <typename P, bool RACE, bool LIMITED>
  __device__ __forceinline__ void distribute(P* probs, const float* noise, float inv, Racer& b) const {
    P* const out = probs + first - shift;              // of slot 0
    const float* const e = noise + first - shift;
    const bool out_wide = (reinterpret_cast<uintptr_t>(out) & (sizeof(P) * V::N - 1) & 15) == 0;
    const bool e_wide = RACE && (reinterpret_cast<uintptr_t>(e) & 15) == 0;
    if (!out_wide) {
      // Rows whose groups lie otherwise in memory than in the logits: token by token, each warp's side
      // by side.
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float l = V::one(data, i + shift);
        const bool is = LIMITED ? left(l, i) : l >= lim.t;
        const float w = is ? w_of(l) : 0.f;
        probs[first + i] = P(w * inv);
        if (RACE && is) {
          const float f = noise[first + i];
          if (w > b.s2 * f) b.take(__fdividef(w, f), l, first + i);
        }
      }
      return;
    }
    const uint4* p = reinterpret_cast<const uint4*>(data);
    for (int q = threadIdx.x; q < groups; q += kThreads) {
      const int s0 = q * V::N;
      float x[V::N], w[V::N];
      V::get(p[q], x);
      bool any = false, keep[V::N];
#pragma unroll
      for (int j = 0; j < V::N; ++j) {
        keep[j] = LIMITED ? left(x[j], s0 + j - shift) : x[j] >= lim.t;
        w[j] = keep[j] ? w_of(x[j]) : 0.f;
        any |= keep[j];
      }
      const bool inside = s0 >= shift && s0 + V::N <= shift + n;
      if (inside) {
        store_group<P>(out + s0, w, inv);
      } else {
#pragma unroll
        for (int j = 0; j < V::N; ++j)
          if (s0 + j >= shift && s0 + j < shift + n) out[s0 + j] = P(w[j] * inv);
      }
      if (RACE && any) {
        float f[V::N];
        load_noise(e, s0, e_wide && inside, x, f);
#pragma unroll
        for (int j = 0; j < V::N; ++j)
          if (keep[j] && w[j] > b.s2 * f[j]) b.take(__fdividef(w[j], f[j]), x[j], first + s0 + j - shift);
      }
    }
  }
  // The race alone.
  template <bool LIMITED>
  __device__ __forceinline__ void run_race(const float* noise, Racer& b) const {
    const float* const e = noise + first - shift;      // of slot 0
    const bool e_wide = (reinterpret_cast<uintptr_t>(e) & 15) == 0;
    if (!e_wide) {
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float l = V::one(data, i + shift);
        if (!(LIMITED ? left(l, i) : l >= lim.t)) continue;
        const float w = w_of(l), f = noise[first + i];
        if (w > b.s2 * f) b.take(__fdividef(w, f), l, first + i);
      }
      return;
    }
    const uint4* p = reinterpret_cast<const uint4*>(data);
    for (int q = threadIdx.x; q < groups; q += kThreads) {
      const int s0 = q * V::N;
      float x[V::N], f[V::N];
      V::get(p[q], x);
      float top = x[0];
#pragma unroll
      for (int j = 1; j < V::N; ++j) top = fmaxf(top, x[j]);
      if (!(top >= lim.t)) continue;
      // (a group's noise is a sector of memory, or half of one: it comes whole)
      load_noise(e, s0, s0 >= shift && s0 + V::N <= shift + n, x, f);
#pragma unroll
      for (int j = 0; j < V::N; ++j) {
        const bool keep = LIMITED ? left(x[j], s0 + j - shift) : x[j] >= lim.t;
        const float w = w_of(x[j]);
        if (keep && w > b.s2 * f[j]) b.take(__fdividef(w, f[j]), x[j], first + s0 + j - shift);
      }
    }
  }
  __device__ __forceinline__ void load_noise(const float* e, int s0, bool wide, const float (&x)[V::N],
                                             float (&f)[V::N]) const {
    if (wide) {
#pragma unroll
      for (int j = 0; j < V::N; j += 4) {
        const uint4 u = ld_stream(reinterpret_cast<const uint4*>(e + s0 + j));
        f[j] = __uint_as_float(u.x);
        f[j + 1] = __uint_as_float(u.y);
        f[j + 2] = __uint_as_float(u.z);
        f[j + 3] = __uint_as_float(u.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V::N; ++j) f[j] = x[j] >= lim.t ? e[s0 + j] : 1.f;
    }
  }
  template <typename P>
  static __device__ __forceinline__ void store_group(P* to, const float (&w)[V::N], float inv) {
    if constexpr (sizeof(P) == 4) {
#pragma unroll
      for (int j = 0; j < V::N; j += 4)
        __stcs(reinterpret_cast<float4*>(to + j),
               make_float4(w[j] * inv, w[j + 1] * inv, w[j + 2] * inv, w[j + 3] * inv));
    } else {
      uint32_t u[V::N / 2];
#pragma unroll
      for (int j = 0; j < V::N / 2; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(w[2 * j] * inv, w[2 * j + 1] * inv);
        u[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if constexpr (V::N == 8) __stcs(reinterpret_cast<uint4*>(to), make_uint4(u[0], u[1], u[2], u[3]));
      else __stcs(reinterpret_cast<uint2*>(to), make_uint2(u[0], u[1]));
    }
  }

  // One filter's end (k > 0: top-k, with top-p at once where the list holds all that top-k keeps;
  // else top-p of what is left).  Sets lim; returns the mass kept; done_p: top-p is applied.
  __device__ float cut(int k, bool use_p, float p, bool& done_p) {
    const bool by_count = k > 0;
    listed = sorted = false;
    lim_all = lim;
    mass_t v[3];    // masses in fixed point from fp32,
    double d[3];    // or, once those have not told, from pairs
    bool pairs = false;
    if (!by_count && whole < 0) weigh();
    // 0: what may be kept at all
    const float least = bound(k, p);
    if (least > lim.t) {
      lim.t = least;
      lim.i = kNone;
    }
    // Of kThreads threads' tokens about kThreads ln(1 / (1 - k / kThreads)) pass k of their maxima;
    // where that is well below the list's size in all CTAs together, it is listed at once (fewer, as the
    // bound is the best of theirs).
    if (by_count && k < kThreads && -kThreads * __logf(1.f - k / (float)kThreads) * C < 0.6f * kList) {
      evaluate(lim.t, INFINITY, true, true, v);
      if (n_listed <= kList) {
        done_p = true;
        float z;
        if (!resolve(v, d, false, 0, k, use_p, p, z)) {
          cl.sync();
          d[0] = d[1] = d[2] = 0;  // (the list has it all)
          resolve(v, d, true, 0, k, use_p, p, z);
        }
        return z;
      }
    }
    // 1: buckets of (m - l) / T
    histogram([&](float l) { return bucket_of(l); });
    // (a bucket's tokens weigh its middle to 1%, many of them far closer)
    locate(!by_count, (unsigned)k, by_count ? 0.f : p * ((float)whole * (1.f / kUnit)), false,
           [](int b) { return ex2(b * (-1.f / kPerOctave)); });
    // 2: the bracket [f_lo, f_hi): `before` tokens above it, `in` in it, of `total`
    unsigned before = S.cum_before, in = S.cum_in;
    const unsigned total = S.total;
    const int b1 = S.b_at, b0 = before + in <= (unsigned)kList ? 0 : b1;
    if (b0 == 0) {  // everything down to it fits the list
      in += before;
      before = 0;
    }
    if (in <= (unsigned)kList) {
      // mostly that is it: the bracket by its buckets, from a logit that lies safely below
      const float near = m - (b1 + 1.5f) / s;
      auto place = [&](float l) {
        const int b = bucket_of(l);
        return b < b0 ? 0 : b <= b1 ? 1 : 2;
      };
      list_by(fmaxf(b1 == kBuckets - 1 ? -FLT_MAX : near - 4e-7f * (fabsf(m) + fabsf(near)), lim.t), true, before == 0, v,
              place);
      lost = (unsigned)n_listed != in;
      if (lost) return 0.f;
      float z;
      done_p = !by_count || before == 0;
      const mass_t goal = by_count ? 0 : goal_of(p, whole), margin = by_count ? 0 : near_fixed(p, whole);
      const mass_t slack = slack_of(v[0], v[1]);
      const bool sure = by_count || (v[0] + slack + margin < goal && v[0] + v[1] - margin > goal);
      if (sure && resolve(v, d, false, before, k, use_p && done_p, p, z)) return z;
      // fp32 does not tell (or has told that the end lies elsewhere)
      if (by_count || (v[0] - slack - margin < goal && v[0] + v[1] + margin > goal)) {
        cl.sync();
        bool holds = true;
        if (by_count) {
          d[0] = d[1] = d[2] = 0;  // (before is 0: the list has it all)
        } else {
          weigh_pairs(d, place);
          const double g = goal_of(p, d[2]);
          holds = (before == 0 || d[0] < g) && !(d[0] + d[1] < g);
        }
        if (holds) {
          resolve(v, d, true, before, k, use_p && done_p, p, z);
          return z;
        }
      }
    }
    float share = 0.f;
    __syncthreads();
    if (threadIdx.x < 32) {
      const float lo = b1 == kBuckets - 1 ? lim.t : fmaxf(edge(b1 + 1), lim.t);
      if (threadIdx.x == 0) S.f_lo = lo;
    } else if (threadIdx.x < 64) {
      const float hi = b0 == 0 ? INFINITY : edge(b0);
      if (threadIdx.x == 32) S.f_hi = hi;
    }
    __syncthreads();
    float f_lo = S.f_lo, f_hi = S.f_hi;
    // the end lies in [out_lo, out_hi), with out_before tokens above and out_below below
    float out_lo = lim.t, out_hi = INFINITY;
    unsigned out_before = 0, out_below = 0;
    // (each round halves the outer range at least once or cuts it into 2048: far fewer are needed)
    for (int round = 0; round < 100; ++round) {
      const bool gather = in <= (unsigned)kList;
      evaluate(f_lo, f_hi, gather, before == 0, v);
      lost = (unsigned)n_listed != in;
      if (lost) return 0.f;
      if (!by_count) {
        // does the bracket hold the end?
        if (!pairs) {
          const mass_t goal = goal_of(p, v[2]), near = near_fixed(p, v[2]);
          pairs = distance(v[0], goal) <= near + slack_of(v[0], v[1]) || distance(v[0] + v[1], goal) <= near;
        }
        bool below_top, reached;
        if (pairs) {
          evaluate_pairs(f_lo, f_hi, d);
          const double goal = goal_of(p, d[2]);
          below_top = d[0] < goal;
          reached = !(d[0] + d[1] < goal);
          share = (float)((goal - d[0]) / d[1]);
        } else {
          const mass_t goal = goal_of(p, v[2]);
          below_top = v[0] < goal;
          reached = !(v[0] + v[1] < goal);
          share = (float)(goal - v[0]) / (float)v[1];
        }
        if (before > out_before && !below_top) {
          out_lo = f_lo = f_hi;
          f_hi = out_hi;
          out_below = total - before;
          in = before - out_before;
          before = out_before;
          continue;
        }
        if (f_lo > out_lo && !reached && before + in + out_below < total) {
          out_hi = f_hi = f_lo;
          f_lo = out_lo;
          out_before = before = before + in;
          in = total - before - out_below;
          continue;
        }
      }
      if (gather) {
        // 3: the list
        done_p = !by_count || before == 0;
        sorted = false;
        float z;
        if (resolve(v, d, pairs, before, k, use_p && done_p, p, z)) return z;
        cl.sync();
        if (by_count) d[0] = d[1] = d[2] = 0;
        else evaluate_pairs(f_lo, f_hi, d);
        resolve(v, d, true, before, k, use_p && done_p, p, z);
        return z;
      }
      const uint32_t ka = code_of(f_lo), kz = f_hi == INFINITY ? code_of(m) : code_of(f_hi) - 1;
      if (kz <= ka) {
        // equal logits: a number of them, the lowest indices first
        const float w1 = w_of(f_lo);
        long long nth = (long long)k - before;
        if (!by_count) {
          // the first so many that bring the mass to the goal (by one division a row: in 64 bits)
          if (!pairs) evaluate_pairs(f_lo, f_hi, d);
          double w;
          w_exact(f_lo, w);
          nth = (long long)ceil((goal_of(p, d[2]) - d[0]) / w);
        }
        nth = max(1ll, min(nth, (long long)in));
        nth_equal(f_lo, nth);
        lim.t = f_lo;
        lim.i = S.i_cut;
        whole = -1;
        done_p = !by_count;
        cl.sync();
        return (float)v[0] * (1.f / kUnit) + nth * w1;
      }
      // 2 again: the bracket is cut by the codes of its logits
      out_lo = f_lo;
      out_hi = f_hi;
      out_before = before;
      out_below = total - before - in;
      int sh = 0;
      while (((kz - ka) >> sh) >= (uint32_t)kBuckets) ++sh;
      histogram([&](float l) { return l >= f_lo && l < f_hi ? (int)((kz - code_of(l)) >> sh) : -1; });
      locate(!by_count, (unsigned)k - before, share, true, [&](int b) {
        const uint32_t off = ((uint32_t)b << sh) + ((1u << sh) >> 1);
        return w_of(float_of(off > kz - ka ? ka : kz - off));
      });
      const uint32_t top = kz - ((uint32_t)S.b_at << sh);
      f_lo = float_of(top - ka < (1u << sh) ? ka : top - (1u << sh) + 1);
      if (top < kz) f_hi = float_of(top + 1);
      before += S.cum_before;
      in = S.cum_in;
    }
    lost = true;
    return 0.f;
  }
};

__device__ __forceinline__ float block_max(Shared& S, float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) S.wmax[threadIdx.x >> 5] = v;
  __syncthreads();
  v = S.wmax[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v = fmaxf(v, S.wmax[w]);
  return v;
}

// A logit that k (1 .. kThreads) of this CTA's tokens reach, from the largest logit of each thread's
// tokens: from there on lie the maxima of so many threads of each warp that they are k.
__device__ __forceinline__ float reached_by(Shared& S, int k, float mx) {
  const int need = (k + kWarps - 1) / kWarps, lane = threadIdx.x & 31;
  const uint32_t mine = code_of(mx);
  int above = 0;
#pragma unroll
  for (int o = 1; o < 32; ++o) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, o);
    above += other > mine || (other == mine && (lane ^ o) < lane);
  }
  const uint32_t at = __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, above == need - 1)) - 1);
  __syncthreads();
  if (lane == 0) S.wcnt[threadIdx.x >> 5] = at;
  __syncthreads();
  uint32_t least = S.wcnt[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) least = min(least, S.wcnt[w]);
  return float_of(least);
}

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

  if (a.n_rows && row >= *a.n_rows) return;
  const int req = a.row_req ? a.row_req[row] : row;
  Row<T> R{cl, S, data};
  R.C = C;
  R.rank = rank;
  R.first = min(a.V, rank * chunk);
  R.n = min(a.V, R.first + chunk) - R.first;
  R.set = 0;
  R.n_row = a.V;
  R.whole = -1;
  R.listed = R.sorted = R.lost = false;
  const T* src = static_cast<const T*>(a.logits) + row * a.stride + R.first;
  R.shift = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  R.groups = (R.n + R.shift + V::N - 1) / V::N;
  if (R.n == 0) R.groups = 0;

  // the chunk into shared memory, and its maximum (of a padding row too: its parameters come later)
  float mx = -INFINITY;
  {
    const uint4* g = reinterpret_cast<const uint4*>(src - R.shift);
    uint4* d = reinterpret_cast<uint4*>(data);
    // four loads of a thread under way
    for (int q0 = tid; q0 < R.groups; q0 += 4 * kThreads) {
      uint4 u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = q0 + k * kThreads, e0 = q * V::N - R.shift;
        if (e0 >= 0 && e0 + V::N <= R.n) {
          u[k] = ld_stream(g + q);
        } else if (q < R.groups) {
          float x[V::N];
#pragma unroll
          for (int j = 0; j < V::N; ++j)
            x[j] = (e0 + j >= 0 && e0 + j < R.n) ? V::one(src, e0 + j) : -INFINITY;
          u[k] = V::put(x);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = q0 + k * kThreads;
        if (q >= R.groups) break;
        float x[V::N];
        V::get(u[k], x);
#pragma unroll
        for (int j = 0; j < V::N; ++j) {
          x[j] = fmaxf(x[j], -INFINITY);  // (NaN counts as -inf)
          mx = fmaxf(mx, x[j]);
        }
        d[q] = V::put(x);
      }
    }
  }
  // the row's parameters (every decision below is the same in all threads of the cluster)
  P* const probs = a.probs ? static_cast<P*>(a.probs) + (long long)row * a.V : nullptr;
  auto none = [&]() {  // no token, no probability
    if (probs)
      for (int i = tid; i < R.n; i += kThreads) probs[R.first + i] = P(0.f);
    if (a.tokens && rank == 0 && tid == 0) a.tokens[row] = -1;
  };
  if (req < 0) {
    if (a.every_row) none();
    return;
  }
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
    if (a.every_row) none();
    return;
  }
  const bool greedy = temp == 0.f;
  if (greedy) temp = p = 1.f, k = 0, mp = 0.f;
  mp = fminf(mp, 1.f);
  if (p <= 0.f) p = 1.f, k = 1;  // the first token alone
  const bool use_k = k > 0 && k < a.V, use_p = p < 1.f;
  cl.barrier_arrive();  // (waited for before the first access to another CTA's memory)
  // (one thread: 64 bits are slow here, and only a border needs them)
  if (mp > 0.f && tid == 0) S.log_min = (double)temp * log((double)mp);
  if (tid == kThreads - 1) {
    // log2(e) = 1.44269502162933349609375 + 1.92596299112661746887e-8
    const float h = 1.44269502162933349609375f, c = h / temp;
    S.c_hi = c;
    S.c_lo = (fmaf(-c, temp, h) + 1.92596299112661746887e-8f) / temp;
  }
  const float mx_cta = block_max(S, mx);
  const float least_cta = use_k && k <= kThreads ? reached_by(S, k, mx) : -INFINITY;
  cl.barrier_wait();
  if (tid < C) {
    Shared* o = cl.map_shared_rank(&S, tid);
    o->cmax[rank] = mx_cta;
    o->cleast[rank] = least_cta;
  }
  cl.sync();
  // (k tokens of one CTA are k of the row: its best bound is any CTA's)
  float m = S.cmax[0], least = S.cleast[0];
  for (int r = 1; r < C; ++r) {
    m = fmaxf(m, S.cmax[r]);
    least = fmaxf(least, S.cleast[r]);
  }
  if (m == INFINITY) {  // +inf counts as the type's largest number
    m = V::kTop;
    least = fminf(least, m);
    uint4* const d = reinterpret_cast<uint4*>(data);
    for (int q = tid; q < R.groups; q += kThreads) {
      float x[V::N];
      V::get(d[q], x);
#pragma unroll
      for (int j = 0; j < V::N; ++j) x[j] = fminf(x[j], m);
      d[q] = V::put(x);
    }
    __syncthreads();
  }
  R.m = m;
  R.k_least = least;
  R.s = S.c_hi * kPerOctave;
  R.nc = -S.c_hi;
  const float* const noise = a.noise ? a.noise + (long long)row * a.V : nullptr;
  if (m == -INFINITY) {  // no token is left to draw from
    none();
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
  float z = -1.f;
  bool done_p = false;
  if (greedy) {
    R.lim.t = m;
    R.lim.i = R.first_top();
    z = 1.f;
  }
  if (use_k) z = R.cut(k, use_p, p, done_p);
  if (use_p && !done_p && !R.lost) z = R.cut(0, true, p, done_p);
  if (R.lost) {
    if (rank == 0 && tid == 0) raise_error(a.err, DSPARK_DEVERR_WORK_OVERFLOW);
    if (a.every_row) none();
    return;
  }
  const bool race = a.tokens != nullptr;
  if (greedy && race && rank == 0 && tid == 0) a.tokens[row] = R.lim.i;
  if (!probs && (greedy || (R.listed && rank != 0))) return;
  if (z < 0.f && probs) {
    R.weigh();
    z = (float)R.whole * (1.f / kUnit);
  }

  // the distribution, and each thread's two best in the race
  Racer b;
  const bool solo = !probs && R.listed;  // the list's tokens alone, by the first CTA
  if (solo) {
    for (int i = tid; i < S.n_keep; i += kThreads) {
      const float l = R.list_l(i);
      const int at = (int)(uint32_t)S.list[i];
      b.take(__fdividef(R.w_of(l), noise[at]), l, at);
    }
  } else if (probs) {
    if (race && !greedy) {
      if (R.lim.i == kNone) R.template distribute<P, true, false>(probs, noise, 1.f / z, b);
      else R.template distribute<P, true, true>(probs, noise, 1.f / z, b);
    } else {
      R.template distribute<P, false, true>(probs, noise, 1.f / z, b);
    }
  } else {
    if (R.lim.i == kNone) R.template run_race<false>(noise, b);
    else R.template run_race<true>(noise, b);
  }
  if (!race || greedy) return;

  // The best in fp32: mostly nothing comes near it.  A score whose logit lies x octaves below the top is
  // off by ln 2 * 3 * 2^-24 x (three roundings of the exponent) + 2^-21 (exponential and division) at
  // most.  With noise between 2^-100 and 2^20 no token more than 120 octaves down wins or comes near:
  // two scores are off by 2^-15 together.
  const float top_cta = block_max(S, b.s1);
  constexpr float kClose = 1.f - 0x1p-14f;
  auto close = [&](float s, int i, float top) { return i != kNone && s >= top * kClose; };
  int n_near = __syncthreads_count(close(b.s1, b.i1, top_cta)) + __syncthreads_count(close(b.s2, b.i2, top_cta));
  float top = top_cta;
  if (!solo) {
    if (tid < C) {
      Shared* o = cl.map_shared_rank(&S, tid);
      o->c_best[rank] = top_cta;
      o->n_near[rank] = n_near;
    }
    cl.sync();
    for (int r = 0; r < C; ++r) top = fmaxf(top, S.c_best[r]);
    n_near = 0;
    for (int r = 0; r < C; ++r) n_near += S.c_best[r] >= top * kClose ? S.n_near[r] : 0;
  }
  if (n_near == 1) {
    if (close(b.s1, b.i1, top)) a.tokens[row] = b.i1;
    return;
  }
  // else in 64 bits, among those that come near
  double rs = -INFINITY;
  int ri = kNone;
  float pl = 0.f, pe = 0.f;  // (equal pairs of logit and noise have equal scores: the first one's counts)
  auto precise = [&](float l, float e, int i) {
    if (ri != kNone && l == pl && e == pe) return;
    better(rs, ri, ((double)l - (double)m) / (double)temp - log((double)e), i);
    pl = l;
    pe = e;
  };
  if (__syncthreads_or(!solo && close(b.s2, b.i2, top))) {
    // a thread whose second comes near may have had a third (not of a list: that is two to a thread)
    for (int i = tid; i < R.n; i += kThreads) {
      const float l = V::one(data, i + R.shift);
      if (!R.left(l, i)) continue;
      const float e = noise[R.first + i];
      if (close(__fdividef(R.w_of(l), e), i, top)) precise(l, e, R.first + i);
    }
  } else {
    if (close(b.s1, b.i1, top)) precise(b.l1, noise[b.i1], b.i1);
    if (close(b.s2, b.i2, top)) precise(b.l2, noise[b.i2], b.i2);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    better(rs, ri, __shfl_xor_sync(0xffffffffu, rs, o), __shfl_xor_sync(0xffffffffu, ri, o));
  __syncthreads();
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
  if (solo) __syncthreads();
  else cl.sync();
  if (rank == 0 && tid == 0) {
    rs = S.cr_best[0];
    ri = S.cr_idx[0];
    for (int r = 1; r < (solo ? 1 : C); ++r) better(rs, ri, S.cr_best[r], S.cr_idx[r]);
    a.tokens[row] = ri == kNone ? -1 : ri;
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
