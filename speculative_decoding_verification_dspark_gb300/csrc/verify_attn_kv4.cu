// Varlen verify attention over a 4-bit paged KV cache (layout: kv4.cuh), GQA head dim 128.
//
// For packed row cu_seqlens[r] + i and query head h of KV group kvh:
//   o = softmax(scale q.K^T) V over the ctx_len[r] committed keys, whose K and V are
//   (code - 8) * scale * g, followed by block rows 0..i (bf16); lse = log-sum-exp.
//
// As in the bf16 cache's kernel, keys lie on the MMA's M side and the few query rows on
// N (NT = 32 or 64 columns), and the key tiles of all groups are cut into equal ranges, one per
// CTA (worklist.cuh):
//   S^T [128 keys x NT] = K [128 x 128] . Q^T        O^T [128 d x NT] += V^T [128 x 128] . P^T
// The left operands are in tensor memory: a lane of K is a key and a lane of V^T a channel,
// so the thread that reads a key's (a channel's) codes expands them and writes its own
// lane.  Through shared memory the expanded tile would cost 64 KB of writes and 64 KB
// of MMA reads per 17 KB of cache, more than the SM's share of HBM time.
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
// Warp roles (one CTA per SM):
//   warp 0       issues S = K Q^T (one lane); owns the TMEM allocation
//   warp 1       query loader: the next item's rows into the other Q buffer
//   warp 2       issues O += V^T P^T.  (Two issuers: an unrolled chain of 8 N = 32 products
//                takes about 46 cycles a piece to issue, so 16 of them from one thread
//                would take as long as the tile's share of HBM time.)
//   warp 3       copies cache tiles into a ring of shared memory: one bulk copy per run of
//                blocks that lie together (a block where pages hold 16 tokens), each
//                from a lane of its own
//   warps 4-7    K: thread = key; codes from the ring, expanded into TMEM
//   warps 8-11   V: warp = group of 32 channels, thread = channel; the same
//   warps 12-15  softmax of columns 0..31, thread = key; epilogue, thread = channel
//   warps 16-19  (64-column tile only) softmax of columns 32..63
// The softmax takes a tile in one pass against the row references of the tiles before; only
// if some key lies 2^8 above its row's maximum then (always in an item's first tile)
// does the tile go through the pass that moves references and rescales O.  Row sums stay in
// the threads (each sums its own keys) until the item ends.
// Every wait on an mbarrier is bounded in time (DSPARK_DEVERR_WAIT_TIMEOUT on expiry); a
// softmax warpgroup's own barriers carry the failure, so its warps leave together.

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

using namespace ptx;
using namespace dspark::kv4;

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kKT = 128;               // keys per tile (MMA M)
constexpr int kStages = 8;             // ring of cache tiles (a power of two)
constexpr int kBlocks = kKT / kBlock;  // blocks of a tile
constexpr int kStageBytes = kBlocks * kBlockBytes;
constexpr int kSmemItems = 32;         // work items of a CTA kept in shared memory
constexpr int kQkWarp = 0, kQWarp = 1, kPvWarp = 2, kCopyWarp = 3, kKWarp0 = 4, kVWarp0 = 8, kSmWarp0 = 12;
constexpr float kRefDrop = 6.f;        // reference = maximum - 6 (log2)
constexpr float kMove = 14.f;          // a key above reference + 14 moves it
constexpr float kNoRef = -1e30f;       // reference of a row that has seen no key (`ref` holds the negatives)

template <int NT_>
struct Cfg {
  static constexpr int NT = NT_;
  static constexpr int WGS = NT / 32;               // softmax warpgroups
  static constexpr int THREADS = (kSmWarp0 + 4 * WGS) * 32;
  static constexpr int Q_CB = NT * 128;             // one 64-wide column block of Q
  static constexpr int Q_BYTES = 2 * Q_CB;
  static constexpr int P_ROW = NT * 2;
  static constexpr int P_BYTES = kKT * P_ROW;
  static constexpr SwizzleMode P_SW = NT == 32 ? SW_64B : SW_128B;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;
  static constexpr int OFF_RING = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_VS = OFF_RING + kStages * kStageBytes; // V scale pairs: [4 warps][512 B]
  static constexpr int OFF_CF = OFF_VS + 4 * 512;                 // float cf[2][NT]: softmax scale per row
  static constexpr int OFF_REF = OFF_CF + 2 * NT * 4;             // float ref[WGS][4][32]
  static constexpr int OFF_AL = OFF_REF + WGS * 512;              // float alpha[WGS][4][32]
  static constexpr int OFF_RED = OFF_AL + WGS * 512;              // float red[WGS][4][32]
  static constexpr int OFF_SUM = OFF_RED + WGS * 512;              // float sum[WGS][4][32]
  static constexpr int OFF_ITEMS = OFF_SUM + WGS * 512;
  static constexpr int OFF_BAR = OFF_ITEMS + kSmemItems * (int)sizeof(AttnItem);
  static constexpr int N_BARS = 18 + 2 * kStages;
  static constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;
  static constexpr int TMEM_S = 0, TMEM_O = 2 * NT, TMEM_K = 4 * NT, TMEM_V = 4 * NT + 128;
  static constexpr int TMEM_COLS = 512;
  static_assert(NT == 32 || NT == 64, "query tile");
  static_assert(TMEM_V + 128 <= TMEM_COLS, "tensor memory");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

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
  float sl2;            // scale * log2(e) * 16 * k_scale
  float k_unit, v_unit; // 1 / (16 k_scale), 1 / (16 v_scale)
  float o_unit;         // 16 v_scale
};

struct Ctx {
  volatile int* abort_flag;
  unsigned int* err;
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Ctx& cx) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
    if (*cx.abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *cx.abort_flag = 1;
      raise_error(cx.err, DSPARK_DEVERR_WAIT_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Ctx& cx) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, cx));
}
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity, unsigned int* err) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      raise_error(err, DSPARK_DEVERR_WAIT_TIMEOUT);
      return;
    }
  }
}

// Barrier of one softmax warpgroup (128 threads) that ors a flag over it.
__device__ __forceinline__ bool group_or(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %2, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t sw128_off(int row, int chunk) {
  return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint32_t sw64_off(int row, int chunk) {
  return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
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
// Two fp32 operations in one instruction.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack(F2 x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return (uint32_t)r.x | ((uint32_t)r.y << 16);
}
// Eight codes of a word -> four pairs (code - 8) s / 16: pair p with s[p], b[p] as the
// head of the file has them for even (low nibbles) and odd (high nibbles) p.
__device__ __forceinline__ void expand(uint32_t w, const uint32_t (&s)[4], const uint32_t (&b)[4],
                                       uint32_t* o) {
  const uint32_t w8 = w >> 8;
  o[0] = hfma2_bits((w & 0x000f000fu) | 0x64006400u, s[0], b[0]);
  o[1] = hfma2_bits((w & 0x00f000f0u) | 0x64006400u, s[1], b[1]);
  o[2] = hfma2_bits((w8 & 0x000f000fu) | 0x64006400u, s[2], b[2]);
  o[3] = hfma2_bits((w8 & 0x00f000f0u) | 0x64006400u, s[3], b[3]);
}
// x in cache units, two of them as fp16, saturating (a NaN stays one).
__device__ __forceinline__ float sat16(float x) {
  return x != x ? x : fminf(fmaxf(x, -65504.f), 65504.f);
}
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return h2_bits(__floats2half2_rn(sat16(a), sat16(b)));
}

// fp16 x fp16 -> fp32 instruction descriptor, A in tensor memory (K-major), B K-major or
// MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Warp transpose-reduction: lane l holds v[0..31]; returns op over all lanes of v[l].
template <bool MAX, int W>
__device__ __forceinline__ void transpose_step(float (&v)[32], int lane) {
  const bool hi = (lane & W) != 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float send = hi ? v[i] : v[i + W];
    const float keep = hi ? v[i + W] : v[i];
    const float got = __shfl_xor_sync(0xffffffffu, send, W);
    v[i] = MAX ? fmaxf(keep, got) : keep + got;
  }
}
template <bool MAX>
__device__ __forceinline__ float transpose_reduce(float (&v)[32], int lane) {
  transpose_step<MAX, 16>(v, lane);
  transpose_step<MAX, 8>(v, lane);
  transpose_step<MAX, 4>(v, lane);
  transpose_step<MAX, 2>(v, lane);
  transpose_step<MAX, 1>(v, lane);
  return v[0];
}

__device__ __forceinline__ AttnItem fetch_item(const AttnItem* s_items, const AttnItem* g_items,
                                               int it, int it_begin) {
  const int k = it - it_begin;
  return k < kSmemItems ? s_items[k] : g_items[it];
}
// Keys of tile t that some query row can see: cache keys below ctx, or block rows below n_r.
__device__ __forceinline__ int visible_keys(int t, int ct, int ctx, int n_r) {
  const int v = t < ct ? ctx - t * kKT : n_r - (t - ct) * kKT;
  return v < kKT ? v : kKT;
}

template <int NT>
__global__ void __launch_bounds__(Cfg<NT>::THREADS, 1) verify_attn_kv4_kernel(const Params prm) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  AttnItem* s_items = reinterpret_cast<AttnItem*>(bp + C::OFF_ITEMS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bp + C::OFF_MISC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bp + C::OFF_MISC + 16);
  const Ctx cx{abort_flag, prm.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + C::OFF_BAR + 8 * i; };
  // Barriers, pairs indexed by tile or item parity.  A tile's QK^T releases its K operand with
  // s_full, its PV its V operand and P with pv_done.
  auto k_full = [&](int b) { return bar(0 + b); };
  auto v_full = [&](int b) { return bar(2 + b); };
  auto s_full = [&](int b) { return bar(4 + b); };
  auto s_free = [&](int b) { return bar(6 + b); };
  auto p_full = [&](int b) { return bar(8 + b); };
  auto pv_done = [&](int b) { return bar(10 + b); };
  auto q_full = [&](int b) { return bar(12 + b); };
  auto q_empty = [&](int b) { return bar(14 + b); };
  auto o_free = [&](int b) { return bar(16 + b); };
  auto c_full = [&](int i) { return bar(18 + i); };             // ring of cache tiles
  auto c_empty = [&](int i) { return bar(18 + kStages + i); };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int b = 0; b < 2; ++b) {
      mbar_init(k_full(b), 4);
      mbar_init(v_full(b), 4);
      mbar_init(s_full(b), 1);
      mbar_init(s_free(b), 4 * C::WGS);
      mbar_init(p_full(b), C::WGS);
      mbar_init(pv_done(b), 1);
      mbar_init(q_full(b), 1);
      mbar_init(q_empty(b), 1 + 4 * C::WGS);
      mbar_init(o_free(b), 4 * C::WGS);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(c_full(i), 1);
      mbar_init(c_empty(i), 8);
    }
    fence_mbar_init();
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_release();
  pdl_wait();  // the work list and the step's inputs come from earlier kernels
  const int it_begin = prm.item_begin[blockIdx.x];
  const int it_end = prm.item_begin[blockIdx.x + 1];
  {
    const int n_s = min(kSmemItems, it_end - it_begin);
    constexpr int kWords = (int)(sizeof(AttnItem) / sizeof(uint4));
    for (int i = threadIdx.x; i < n_s * kWords; i += C::THREADS)
      reinterpret_cast<uint4*>(s_items)[i] = reinterpret_cast<const uint4*>(prm.items + it_begin)[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = prm.Hq / prm.Hkv;

  if (warp == kQkWarp) {
    // ------------------------------------------------------------- S^T = K Q^T
    constexpr uint32_t IDESC = idesc_f16_f32(kKT, NT, 0);
    int g = 0, n_it = 0;
    bool ok = true;
    for (int it = it_begin; it < it_end && ok; ++it, ++n_it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int qb = n_it & 1;
      if (!wait_warp(q_full(qb), (n_it >> 1) & 1, cx)) break;
      const uint64_t bd = smem_desc(base + C::OFF_Q + qb * C::Q_BYTES, 16, 1024, SW_128B);
      for (int t = item.tb; t < item.te; ++t, ++g) {
        const int b = g & 1;
        ok = wait_warp(k_full(b), (g >> 1) & 1, cx);
        if (ok && g >= 2) ok = wait_warp(s_free(b), ((g >> 1) - 1) & 1, cx);
        if (!ok) break;
        if (lane == 0) {
          tc_fence_after();
          const uint32_t a = tmem + C::TMEM_K + b * 64, d = tmem + C::TMEM_S + b * NT;
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk)
            umma_bf16_ts(d, a + kk * 8, bd + ((kk >> 2) * C::Q_CB + (kk & 3) * 32) / 16, IDESC,
                         kk > 0 ? 1u : 0u);
          umma_commit(s_full(b));
          if (t == item.te - 1) umma_commit(q_empty(qb));
        }
        __syncwarp();
      }
    }
    if (lane == 0 && g > 0) drain_bar(s_full((g - 1) & 1), ((g - 1) >> 1) & 1, prm.err);
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------- O^T += V^T P^T
    constexpr uint32_t IDESC = idesc_f16_f32(kD, NT, 1);
    int g = 0, n_it = 0;
    bool ok = true;
    for (int it = it_begin; it < it_end && ok; ++it, ++n_it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ob = n_it & 1, ct = ceil_div(item.ctx, kKT);
      if (n_it >= 2 && !wait_warp(o_free(ob), ((n_it >> 1) - 1) & 1, cx)) break;
      for (int t = item.tb; t < item.te; ++t, ++g) {
        const int b = g & 1;
        ok = wait_warp(v_full(b), (g >> 1) & 1, cx) && wait_warp(p_full(b), (g >> 1) & 1, cx);
        if (!ok) break;
        if (lane == 0) {
          tc_fence_after();
          const uint32_t a = tmem + C::TMEM_V + b * 64, d = tmem + C::TMEM_O + ob * NT;
          const uint64_t bd = smem_desc(base + C::OFF_P + b * C::P_BYTES, kKT * 128, 8 * C::P_ROW, C::P_SW);
          // only the 16-key steps that hold a visible key
          const int nch = ceil_div(visible_keys(t, ct, item.ctx, item.n_r), 16);
#pragma unroll
          for (int kk = 0; kk < kKT / 16; ++kk)
            if (kk < nch)
              umma_bf16_ts(d, a + kk * 8, bd + kk * 16 * C::P_ROW / 16, IDESC,
                           (t > item.tb || kk > 0) ? 1u : 0u);
          umma_commit(pv_done(b));
        }
        __syncwarp();
      }
    }
    if (lane == 0 && g > 0) drain_bar(pv_done((g - 1) & 1), ((g - 1) >> 1) & 1, prm.err);
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------- query loader
    // Tile row n = (block row n / G, head kvh G + n % G); rows past the item's are zero.  A
    // half-warp holds a row, 8 elements per lane.
    bool ok = true;
    int n_it = 0;
    for (int it = it_begin; it < it_end && ok; ++it, ++n_it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int qb = n_it & 1;
      if (n_it >= 2) {
        ok = wait_warp(q_empty(qb), ((n_it >> 1) - 1) & 1, cx);
        if (!ok) break;
      }
      const int nq = item.ni * G, l = lane & 15;
      const long long row0 = item.c0 + item.i0;
      const uint32_t qd = base + C::OFF_Q + qb * C::Q_BYTES;
      float* cf = reinterpret_cast<float*>(bp + C::OFF_CF) + qb * NT;
#pragma unroll 1
      for (int n0 = 0; n0 < NT; n0 += 16) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = n0 + 2 * i + (lane >> 4);
          v[i] = make_uint4(0, 0, 0, 0);
          if (n < nq)
            v[i] = *reinterpret_cast<const uint4*>(
                prm.q + ((row0 + n / G) * prm.Hq + item.kvh * G + n % G) * kD + l * 8);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int n = n0 + 2 * i + (lane >> 4);
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t top = 0;  // largest magnitude, as bits (a NaN is above all)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            top = max(top, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          // the largest element's power of two, no smaller than 2^-100 (fp32 holds 2^114)
          const int e = max((int)(top >> 23), 27);
          const float f = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = h2_bits(__floats2half2_rn(__uint_as_float(w[j] << 16) * f,
                                             __uint_as_float(w[j] & 0xffff0000u) * f));
          st_shared_v4(qd + (l >> 3) * C::Q_CB + sw128_off(n, l & 7), make_uint4(h[0], h[1], h[2], h[3]));
          if (l == 0)  // (never 0: a masked score is -inf times it)
            cf[n] = fmaxf(__uint_as_float((uint32_t)(e - 14) << 23) * prm.sl2, 1.17549435e-38f);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(qb));
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------- cache tiles into the ring
    // Lane j looks up and copies block j % 8 of tile j / 8 of a window of four; `nxt` is its
    // page in the window after.  Blocks that lie together in a page go as one copy.
    const int per = 1 << (prm.log2_page - 4);        // blocks of a page
    const int run = min(per, kBlocks);               // blocks of a copy
    const int lt = lane >> 3, lb = lane & 7;
    auto lookup = [&](int r, int ctx, int t) -> int {
      const int pos = (t + lt) * kKT + lb * kBlock;
      const int slot = pos >> prm.log2_page;
      if (pos >= ctx) return -1;
      return slot < prm.max_pages ? __ldg(prm.page_table + (long long)r * prm.max_pages + slot) : -1;
    };
    int gc = 0, nxt = -1;
    bool ok = true;
    if (it_begin < it_end) {
      const AttnItem x = fetch_item(s_items, prm.items, it_begin, it_begin);
      nxt = lookup(x.r, x.ctx, x.tb);
    }
    for (int it = it_begin; it < it_end && ok; ++it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int te = min(item.te, ceil_div(item.ctx, kKT));  // cache tiles of the item
      for (int t0 = item.tb; t0 < item.te && ok; t0 += 4) {
        int page = nxt;
        if (t0 + 4 < item.te) {
          nxt = lookup(item.r, item.ctx, t0 + 4);
        } else if (it + 1 < it_end) {
          const AttnItem x = fetch_item(s_items, prm.items, it + 1, it_begin);
          nxt = lookup(x.r, x.ctx, x.tb);
        }
        const int pos = (t0 + lt) * kKT + lb * kBlock;
        const bool want = pos < item.ctx && t0 + lt < te;
        const bool valid = want && page >= 0 && page < prm.n_pages;
        if (want && !valid) raise_error(prm.err, DSPARK_DEVERR_BAD_INPUT);
        // this lane's copy: `run` blocks from its own, as far as the context reaches
        const int nb = min(run, ceil_div(item.ctx - pos, kBlock));
        const uint32_t bytes = valid && lb % run == 0 ? (uint32_t)(nb * kBlockBytes) : 0u;
        const uint8_t* src = prm.cache + (((long long)(valid ? page : 0) * prm.Hkv + item.kvh) * per +
                                          ((pos >> 4) & (per - 1))) * kBlockBytes;
        uint32_t total = bytes;                      // of the lane's tile
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        for (int i = 0; i < 4 && t0 + i < te; ++i, ++gc) {
          const int st = gc & (kStages - 1);
          if (gc >= kStages) {
            ok = wait_warp(c_empty(st), ((gc / kStages) - 1) & 1, cx);
            if (!ok) break;
          }
          if (lane == 8 * i) mbar_arrive_expect_tx(c_full(st), total);
          __syncwarp();
          if (lt == i && bytes)
            bulk_load_g2s(base + C::OFF_RING + st * kStageBytes + lb * kBlockBytes, src, bytes, c_full(st));
        }
      }
    }
    // no copy may be in flight when the CTA ends
    for (int x = max(gc - kStages, 0); x < gc; ++x)
      if (lane == 0) drain_bar(c_full(x & (kStages - 1)), (x / kStages) & 1, prm.err);
  } else if (warp >= kKWarp0 && warp < kVWarp0) {
    // ------------------------------------------------------------- K: thread = key
    const int w = warp - kKWarp0, kl = w * 32 + lane;
    // this key's codes and scales within a stage
    const uint32_t ring = base + C::OFF_RING + (2 * w + (lane >> 4)) * kBlockBytes;
    const uint32_t codes = ring + (lane & 15) * 16, scales = ring + kOffKs + (lane & 15) * 4;
    const uint32_t t_k = tmem + (static_cast<uint32_t>(w * 32) << 16) + C::TMEM_K;
    int g = 0, gc = 0;
    bool ok = true;
    for (int it = it_begin; it < it_end && ok; ++it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ct = ceil_div(item.ctx, kKT);
      for (int t = item.tb; t < item.te; ++t, ++g) {
        const int b = g & 1, st = gc & (kStages - 1);
        if (t < ct) ok = wait_warp(c_full(st), (gc / kStages) & 1, cx);
        if (ok && g >= 2) ok = wait_warp(s_full(b), ((g >> 1) - 1) & 1, cx);  // QK^T of tile g - 2 done
        if (!ok) break;
        tc_fence_after();
        if (t < ct) {
          const uint32_t src = codes + st * kStageBytes;
          const uint32_t sc = ld_shared(scales + st * kStageBytes);
          const uint32_t s01 = e4m3x2_to_h2(sc & 0xffffu), s23 = e4m3x2_to_h2(sc >> 16);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            const uint4 v = ld_shared_v4(src + c * 256);
            const uint32_t s = __byte_perm(c < 2 ? s01 : s23, 0, (c & 1) ? 0x3232 : 0x1010);
            const uint32_t sl = hmul2_bits(s, kSixteenth), bl = hmul2_bits(s, kBiasLow);
            const uint32_t sh = hmul2_bits(s, k256th), bh = hmul2_bits(s, kBiasHigh);
            const uint32_t ss[4] = {sl, sh, sl, sh}, bb[4] = {bl, bh, bl, bh};
            uint32_t o[16];
            expand(v.x, ss, bb, o);
            expand(v.y, ss, bb, o + 4);
            expand(v.z, ss, bb, o + 8);
            expand(v.w, ss, bb, o + 12);
            tmem_st16u(t_k + b * 64 + c * 16, o);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(c_empty(st));
          ++gc;
        } else {
          // the request's own rows: bf16 / (16 k_scale)
          const int bi = (t - ct) * kKT + kl;
          const __nv_bfloat16* src = prm.k_new + ((long long)(item.c0 + bi) * prm.Hkv + item.kvh) * kD;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = make_uint4(0, 0, 0, 0);
              if (bi < item.n_r) v[j] = reinterpret_cast<const uint4*>(src)[c * 4 + j];
            }
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                o[4 * j + q] = pack16(__uint_as_float(x[q] << 16) * prm.k_unit,
                                      __uint_as_float(x[q] & 0xffff0000u) * prm.k_unit);
            }
            tmem_st16u(t_k + b * 64 + c * 16, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full(b));
      }
    }
  } else if (warp >= kVWarp0 && warp < kSmWarp0) {
    // ------------------------------------------------------------- V: thread = channel
    const int w = warp - kVWarp0;
    const uint32_t ring = base + C::OFF_RING;
    const uint32_t codes = ring + kOffV + (w * 32 + lane) * 8;
    const uint32_t scales = ring + (lane >> 2) * kBlockBytes + kOffVs + w * kBlock + (lane & 3) * 4;
    const uint32_t vs = base + C::OFF_VS + w * 512;
    const uint32_t t_v = tmem + (static_cast<uint32_t>(w * 32) << 16) + C::TMEM_V;
    int g = 0, gc = 0;
    bool ok = true;
    for (int it = it_begin; it < it_end && ok; ++it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ct = ceil_div(item.ctx, kKT);
      for (int t = item.tb; t < item.te; ++t, ++g) {
        const int b = g & 1, st = gc & (kStages - 1);
        const int vis = visible_keys(t, ct, item.ctx, item.n_r);
        const int np = ceil_div(vis, 32);  // pairs of blocks that hold a visible key
        if (t < ct) {
          ok = wait_warp(c_full(st), (gc / kStages) & 1, cx);
          // scale pairs of the tile's keys 4 lane .. + 3, shared by the warp's channels; keys
          // past the context get scale 0, whatever their page holds
          uint32_t sc = ld_shared(scales + st * kStageBytes);
          const int left = vis - 4 * lane;
          if (left < 4) sc = left <= 0 ? 0u : sc & ((1u << (8 * left)) - 1u);
          const uint32_t s0 = e4m3x2_to_h2(sc & 0xffffu), s1 = e4m3x2_to_h2(sc >> 16);
          const uint32_t at = vs + (lane >> 1) * 32 + (lane & 1) * 8;
          st_shared_v2(at, hmul2_bits(s0, kSixteenth), hmul2_bits(s1, k256th));
          st_shared_v2(at + 16, hmul2_bits(s0, kBiasLow), hmul2_bits(s1, kBiasHigh));
          __syncwarp();
        }
        if (ok && g >= 2) ok = wait_warp(pv_done(b), ((g >> 1) - 1) & 1, cx);  // PV of tile g - 2 done
        if (!ok) break;
        tc_fence_after();
        if (t < ct) {
          const uint32_t src = codes + st * kStageBytes;
#pragma unroll 1
          for (int i = 0; i < np; ++i) {
            uint32_t o[16];
            const uint2 v0 = ld_shared_v2(src + 2 * i * kBlockBytes);
            const uint2 v1 = ld_shared_v2(src + (2 * i + 1) * kBlockBytes);
            const uint32_t word[4] = {v0.x, v0.y, v1.x, v1.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t at = vs + (4 * i + j) * 32;
              const uint4 s = ld_shared_v4(at), c = ld_shared_v4(at + 16);
              const uint32_t ss[4] = {s.x, s.y, s.z, s.w}, bb[4] = {c.x, c.y, c.z, c.w};
              expand(word[j], ss, bb, o + j * 4);
            }
            tmem_st16u(t_v + b * 64 + i * 16, o);
          }
          __syncwarp();  // (also: every lane has read the scale pairs)
          if (lane == 0) mbar_arrive(c_empty(st));
          ++gc;
        } else {
          const int b0 = (t - ct) * kKT;
          const __nv_bfloat16* vn = prm.v_new + ((long long)(item.c0 + b0) * prm.Hkv + item.kvh) * kD +
                                    w * 32 + lane;
#pragma unroll 1
          for (int i = 0; i < np; ++i) {
            const long long step = (long long)prm.Hkv * kD;
            float x[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              x[j] = 32 * i + j < vis ? __bfloat162float(vn[(32 * i + j) * step]) : 0.f;
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pack16(x[2 * j] * prm.v_unit, x[2 * j + 1] * prm.v_unit);
            tmem_st16u(t_v + b * 64 + i * 16, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full(b));
      }
    }
  } else if (warp >= kSmWarp0) {
    // ------------------------------------------------------------- softmax and epilogue
    const int sw = warp & 3, wg = (warp - kSmWarp0) >> 2;
    const int kl = sw * 32 + lane;               // key of a tile, channel of O^T
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(sw * 32) << 16) + wg * 32;
    const int bar_id = 1 + wg;
    float* ref = reinterpret_cast<float*>(bp + C::OFF_REF) + (wg * 4 + sw) * 32;   // this warp's copy
    float* alpha = reinterpret_cast<float*>(bp + C::OFF_AL) + (wg * 4 + sw) * 32;
    float* red = reinterpret_cast<float*>(bp + C::OFF_RED) + wg * 128;             // [4 warps][32]
    float* sums = reinterpret_cast<float*>(bp + C::OFF_SUM) + wg * 128;
    int g = 0, n_it = 0;
    bool bad = false;                            // a wait ran out
    for (int it = it_begin; it < it_end; ++it, ++n_it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ctx = item.ctx, ct = ceil_div(ctx, kKT);
      const int nq = min(max(item.ni * G - wg * 32, 0), 32);  // rows in this group's columns
      const int nc8 = (nq + 7) >> 3;
      const int qb = n_it & 1;
      const float* cf = reinterpret_cast<const float*>(bp + C::OFF_CF) + qb * NT + wg * 32;
      bad |= !wait_warp(q_full(qb), (n_it >> 1) & 1, cx);
      float mref = -INFINITY;                    // reference of row `lane`
      float lacc[32];                            // this thread's part of each row's sum
#pragma unroll
      for (int k = 0; k < 32; ++k) lacc[k] = 0.f;
      for (int t = item.tb; t < item.te; ++t, ++g) {
        const int b = g & 1;
        bad |= !wait_warp(s_full(b), (g >> 1) & 1, cx);
        if (nq == 0) {
          // no row of the item in these columns: P's are left as they are, they only reach
          // columns of O^T that nothing reads
          if (group_or(bar_id, bad)) goto done;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free(b));
          if (sw == 0 && lane == 0) mbar_arrive(p_full(b));
          continue;
        }
        if (g >= 2) bad |= !wait_warp(pv_done(b), ((g >> 1) - 1) & 1, cx);  // P buffer free
        tc_fence_after();
        // row n of these columns sees this key iff n >= nmin
        int nmin = 0;
        if (t < ct) {
          if (t * kKT + kl >= ctx) nmin = 1 << 30;
        } else {
          const int bi = (t - ct) * kKT + kl;
          nmin = bi < item.n_r ? (bi - item.i0) * G - wg * 32 : 1 << 30;
        }
        const uint32_t s_col = t_lane + C::TMEM_S + b * NT;
        const uint32_t prow = base + C::OFF_P + b * C::P_BYTES;
        const bool masked = t >= ct || (t + 1) * kKT > ctx;  // some key is not seen by all rows
        float x[32];
        auto scores = [&]() {
          tmem_ld32(s_col, x);
          tmem_wait_ld32(x);
          if (masked) {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = nmin <= k ? x[k] : -INFINITY;
          }
        };
        bool move = t == item.tb;  // the references have to move first
        for (;;) {
          if (move) {
            // ---- the tile's maximum per row, over the group's warps
            scores();
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] *= cf[k];
            red[sw * 32 + lane] = transpose_reduce<true>(x, lane);
            // O^T holds the products up to tile g - 1 before it is rescaled
            if (t > item.tb) bad |= !wait_warp(pv_done((g - 1) & 1), ((g - 1) >> 1) & 1, cx);
            if (group_or(bar_id, bad)) goto done;
            const float tm = fmaxf(fmaxf(red[lane], red[32 + lane]), fmaxf(red[64 + lane], red[96 + lane]));
            float al = 1.f;
            if (tm - kRefDrop > mref + (kMove - kRefDrop)) {
              al = mref == -INFINITY ? 0.f : fast_exp2(mref - (tm - kRefDrop));
              mref = tm - kRefDrop;
            }
            __syncwarp();
            ref[lane] = mref == -INFINITY ? -kNoRef : -mref;
            alpha[lane] = al;
            __syncwarp();
            if (t > item.tb) {
              tc_fence_after();
              const uint32_t t_o = t_lane + C::TMEM_O + (n_it & 1) * NT;
              tmem_ld32(t_o, x);
              tmem_wait_ld32(x);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                lacc[k] *= alpha[k];
                x[k] *= alpha[k];
              }
              tmem_st32(t_o, x);
              tmem_wait_st();
              tc_fence_before();
            }
          }
          // ---- P of this key against the references
          scores();
          float top = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q >= nc8) break;
            uint32_t pk[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = q * 8 + h * 4;
              const float4 c4 = reinterpret_cast<const float4*>(cf)[q * 2 + h];
              const float4 r4 = reinterpret_cast<const float4*>(ref)[q * 2 + h];
              unpack(fma2(f2(x[k], x[k + 1]), f2(c4.x, c4.y), f2(r4.x, r4.y)), x[k], x[k + 1]);
              unpack(fma2(f2(x[k + 2], x[k + 3]), f2(c4.z, c4.w), f2(r4.z, r4.w)), x[k + 2], x[k + 3]);
              top = fmaxf(top, fmaxf(x[k], x[k + 1]));
              top = fmaxf(top, fmaxf(x[k + 2], x[k + 3]));
#pragma unroll
              for (int j = 0; j < 4; ++j) x[k + j] = fast_exp2(x[k + j]);
              pk[2 * h] = h2_bits(__floats2half2_rn(x[k], x[k + 1]));
              pk[2 * h + 1] = h2_bits(__floats2half2_rn(x[k + 2], x[k + 3]));
            }
            const uint32_t off = NT == 32 ? sw64_off(kl, q) : sw128_off(kl, wg * 4 + q);
            st_shared_v4(prow + off, make_uint4(pk[0], pk[1], pk[2], pk[3]));
          }
          fence_proxy_async_smem();
          // all of P is written when the group passes; a key far above its row's reference
          // sends the tile through once more, after the references have moved
          const bool again = group_or(bar_id, top > kMove || bad);
          if (!again) break;
          if (group_or(bar_id, bad)) goto done;
          if (move) break;
          move = true;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free(b));
        if (sw == 0 && lane == 0) mbar_arrive(p_full(b));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= nc8) break;
#pragma unroll
          for (int k = q * 8; k < q * 8 + 8; k += 2)
            unpack(add2(f2(lacc[k], lacc[k + 1]), f2(x[k], x[k + 1])), lacc[k], lacc[k + 1]);
        }
      }
      if (nq > 0) {
        // ---- epilogue: row sums over the group, O^T / l
        sums[sw * 32 + lane] = transpose_reduce<false>(lacc, lane);
        bad |= !wait_warp(pv_done((g - 1) & 1), ((g - 1) >> 1) & 1, cx);
        if (group_or(bar_id, bad)) goto done;
        const float l = (sums[lane] + sums[32 + lane]) + (sums[64 + lane] + sums[96 + lane]);
        const bool split = item.nsplit > 1;
        alpha[lane] = l == 0.f ? 0.f : prm.o_unit / l;
        const long long row0 = (long long)item.c0 + item.i0;
        const int n_l = wg * 32 + lane;
        if (sw == 0 && lane < nq) {
          const float v = (mref + log2f(l)) * 0.69314718055994530942f;
          if (split)
            prm.ws_lse[(long long)item.slot * kKT + n_l] = v;
          else
            prm.lse[(row0 + n_l / G) * prm.Hq + item.kvh * G + n_l % G] = v;
        }
        __syncwarp();
        tc_fence_after();
        float o[32];
        tmem_ld32(t_lane + C::TMEM_O + (n_it & 1) * NT, o);
        tmem_wait_ld32(o);
        if (split) {
          float* dst = prm.ws_o + ((long long)item.slot * kKT + wg * 32) * kD + kl;
#pragma unroll
          for (int n = 0; n < 32; ++n)
            if (n < nq) dst[n * kD] = o[n] * alpha[n];
        } else {
          int h = (wg * 32) % G;
          __nv_bfloat16* dst = prm.out + ((row0 + wg * 32 / G) * prm.Hq + item.kvh * G + h) * kD + kl;
          const long long next = (long long)(prm.Hq - G) * kD;  // to the next block row's heads
#pragma unroll
          for (int n = 0; n < 32; ++n) {
            if (n < nq) *dst = __float2bfloat16(o[n] * alpha[n]);
            dst += kD;
            if (++h == G) {
              h = 0;
              dst += next;
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(o_free(n_it & 1));
        mbar_arrive(q_empty(qb));
      }
    }
  done:;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc(tmem, C::TMEM_COLS);
}

// ---------------------------------------------------------------- split combine
// Block (c, y): the split group recorded by CTA c, query rows 8y..8y+7, a warp per row:
//   lse = log sum_s e^{lse_s},  o = sum_s e^{lse_s - lse} o_s
__global__ void __launch_bounds__(256)
    combine_kv4_kernel(const int32_t* __restrict__ cu_seqlens, const SplitGroup* __restrict__ groups,
                       int G, int Hq, const float* __restrict__ ws_o,
                       const float* __restrict__ ws_lse, __nv_bfloat16* __restrict__ out,
                       float* __restrict__ lse, int B, int max_rows, unsigned int* __restrict__ err) {
  pdl_release();
  pdl_wait();  // inputs come from the kernels before this one
  // packed rows beyond the call's buffers: the work list ran nothing; say so here too, for
  // the call whose work list was built by the pack call
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && cu_seqlens[B] > max_rows)
    raise_error(err, DSPARK_DEVERR_ROWS_OVERFLOW);
  const int lane = threadIdx.x & 31;
  const SplitGroup sg = groups[blockIdx.x];
  const int ns = sg.nsplit;
  const int n = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (ns <= 1 || n >= sg.ni * G) return;
  int slot = 0;
  float my = -INFINITY;
  if (lane < ns) {
    slot = (lane == 0 && sg.slot0_last) ? 2 * sg.c_first + 1 : 2 * (sg.c_first + lane);
    my = ws_lse[(long long)slot * kKT + n];
  }
  float mx = my;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float wgt = lane < ns ? expf(my - mx) : 0.f;
  float sum = wgt;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = 1.f / sum;
  const long long row = cu_seqlens[sg.r] + sg.i0 + n / G;
  const int head = sg.kvh * G + n % G;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < ns; ++s) {
    const float w = __shfl_sync(0xffffffffu, wgt, s);
    const int sl = __shfl_sync(0xffffffffu, slot, s);
    const float4 v = reinterpret_cast<const float4*>(ws_o + ((long long)sl * kKT + n) * kD)[lane];
    acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(out + (row * Hq + head) * kD)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
  if (lane == 0) lse[row * Hq + head] = mx + logf(sum);
}

// ---------------------------------------------------------------- host side
template <int NT>
static bool configure() {
  static PerDevice<bool> done;
  return once_per_device(done, false, [] {
    return cudaFuncSetAttribute(verify_attn_kv4_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg<NT>::SMEM_BYTES) == cudaSuccess;
  });
}

template <int NT>
static int launch_tile(const Params& p, int ncta, cudaStream_t stream) {
  if (!configure<NT>()) return DSPARK_ECUDA;
  return launch_pdl(verify_attn_kv4_kernel<NT>, dim3(ncta), dim3(Cfg<NT>::THREADS),
                    Cfg<NT>::SMEM_BYTES, stream, p) == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

int launch(const void* q, const void* k_new, const void* v_new, const void* cache, int n_pages,
           const int32_t* page_table, int max_pages, const int32_t* ctx_len,
           const int32_t* cu_seqlens, int B, int max_rows, int Hq, int Hkv, int page_size,
           float scale, float gk, float gv, int max_splits, void* out, float* lse, void* ws,
           const Plan& pl, cudaStream_t stream, bool planned) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  AttnItem* items = reinterpret_cast<AttnItem*>(w + pl.off_items);
  int* item_begin = reinterpret_cast<int*>(w + pl.off_begin);
  SplitGroup* groups = reinterpret_cast<SplitGroup*>(w + pl.off_groups);
  if (!planned) {
    const int rc = launch_worklist(ctx_len, cu_seqlens, B, max_rows, Hkv, max_splits, ws, pl, stream);
    if (rc != DSPARK_OK) return rc;
  }
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.cache = static_cast<const uint8_t*>(cache);
  p.page_table = page_table;
  p.items = items;
  p.item_begin = item_begin;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.ws_o = reinterpret_cast<float*>(w + pl.off_o);
  p.ws_lse = reinterpret_cast<float*>(w + pl.off_lse);
  p.err = device_error_word();
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.log2_page = 0;
  while ((1 << p.log2_page) < page_size) ++p.log2_page;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.sl2 = scale * 1.4426950408889634f * (16.f * gk);
  p.k_unit = 1.f / (16.f * gk);
  p.v_unit = 1.f / (16.f * gv);
  p.o_unit = 16.f * gv;
  const int rc = pl.nt == 32 ? launch_tile<32>(p, pl.ncta, stream) : launch_tile<64>(p, pl.ncta, stream);
  if (rc != DSPARK_OK) return rc;
  return launch_pdl(combine_kv4_kernel, dim3(pl.ncta, pl.nt / 8), dim3(256), 0, stream, cu_seqlens,
                    groups, Hq / Hkv, Hq, p.ws_o, p.ws_lse, p.out, lse, B, max_rows,
                    p.err) == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

}  // namespace kv4a
}  // namespace attn
}  // namespace dspark
