// Verify attention over a paged bf16 cache for trees of drafted tokens, GQA head dim 128.
//
// Packed row cu_seqlens[r] + i, query head h, sees the ctx_len[r] committed keys of its request and
// the block rows j of its segment whose bit j is set in row_mask: o = softmax(scale q.K^T) V,
// lse = log-sum-exp.  A row that sees no key gets o = 0, lse = -inf.
//
// A tree brings many query rows to each key (64 nodes of 4 heads: 256, some 250 FLOP a byte, where
// HBM and the tensor cores balance), so queries lie on the MMA's M side, 128 rows to a tile, and a
// work item has up to two tiles that share the keys:
//   S [128 rows x 128 keys] = Q . K^T         O [128 rows x 128 d] += P . V       (tcgen05)
// with S and O in tensor memory and P, in bf16, in the columns that held S (the product takes 16-bit
// operands; against 64 bits the output is off by 0.0019 to 0.0023 with that, by 0.0017 from its own
// rounding alone).  All 512 columns are taken: two S, two O.  An item of one tile's rows runs as two
// streams of its key tiles, even and odd, each with an S, an O and statistics of its own, joined at the
// item's end: so that one stream's softmax runs beside the other's products whether there are two tiles
// or one.
//
// Warps (one CTA an SM, persistent over its share of the key tiles, see own_items.cuh):
//   0      K and Q, 2  V: TMA (128-byte swizzle), K and V into a ring of five 32 KB slots
//   1, 3   issue the products of one stream each: O += P V of its last tile, then S of its next
// Warp 2 also looks over its V tiles: keys past the visible ones of a chunk of 16 become zero; so do
// NaN and infinities of block rows, since a row that does not see them weighs them 0, and 0 times
// them is NaN: the rows that do see them get them after the epilogue (write_specials).
//   4-7, 8-11  the softmax of the streams, thread = row: maximum, exponentials and sum of 128 keys
//          without a word to another thread; O is rescaled only where a row's maximum grows by 2^8
// Every wait is bounded (DSPARK_DEVERR_WAIT_TIMEOUT on expiry).
//
// What bounds it: with one query tile HBM (256 single tokens over 0.5k to 4k keys 402 us, 357 at the copy
// rate); with two a stream's chain, 3500 cycles a key tile: S to the softmax 150, 128 exponentials a
// thread and P 1300, P to the issuing thread 150, O += P V and the next S 2 x 520, and 250 more each
// time the tensor cores change from the one kind of product to the other (32 requests of 17 to 64
// nodes over 1k to 4k keys 111 us, 52 at the copy rate; 16 of 97 to 256 nodes 295 us).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "common.cuh"
#include "own_items.cuh"
#include "ptx.cuh"

namespace dspark {
namespace attn {
namespace tree {

using namespace ptx;

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kD = 128;
constexpr int kM = 128;                // query rows of a tile
constexpr int kHalf = 128 * 128;       // bytes of 64 columns of a [128 x 128] bf16 tile
constexpr int kTile = 2 * kHalf;
constexpr int kStages = 5;
constexpr int kBoxRows = 16;           // block rows of a TMA box
constexpr int kThreads = 384;
constexpr int kKWarp = 0, kMmaWarp = 1, kVWarp = 2, kSoftmaxWarp = 4;  // 3: the other stream's kMmaWarp
constexpr int kFlags = 8;
// TMEM columns
constexpr int kTmemS = 0, kTmemO = 256;

struct Smem {  // the first 3 KB; then Q (two tiles) and the ring
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2], joined;
  uint32_t tmem;
  int abort;
  // Counts beside the barriers: a barrier shows the parity of a phase only, and not every waiter comes
  // by at every phase.
  uint32_t armed[kStages];             // fills of a slot that were begun
  uint32_t looked[kStages];            // V's last fill of a slot that was looked over, + 1
  uint32_t turns[2];                   // steps that a stream issued of items with two query tiles
  uint32_t epilogues;                  // softmax warps that are done with an item, over all items
  int special[kFlags];                 // by item: block rows held NaN or infinities
  float ml[2][kM][2];                  // (reference, sum) of a stream's rows at an item's end
  AttnItem items[4];
};
constexpr int kHead = 3 * 1024;
static_assert(sizeof(Smem) <= kHead, "head of the shared memory");
constexpr int kSmemBytes = kHead + 2 * kTile + kStages * kTile;
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(sizeof(ItemScratch) <= kStages * kTile, "scratch in the ring");

struct Params {
  const __nv_bfloat16* v_new;
  const int32_t* page_table;
  const int32_t *ctx_len, *cu_seqlens;
  const uint64_t* mask;
  AttnItem* items;
  SplitGroup* groups;
  __nv_bfloat16* out;
  float *lse, *ws_o, *ws_lse;
  unsigned int* err;
  int Hq, Hkv, log2_page, max_pages, n_pages, words;
  int B, max_rows, rows_per_tile, max_splits;
  int tile_rows;        // block rows of one query tile; rows_per_tile is this or twice this
  int slot_rows;
  float sl2;            // scale * log2(e)
};

struct Ctx {
  volatile int* abort;
  unsigned int* err;
};

// Bounded waits of one thread: on a barrier's phase, and until a count has come to `least`.  Bounded by
// their number of polls, in few instructions: the roles' loops and a dozen waits by the clock would not
// fit the instruction cache together.  (A poll of a barrier sleeps up to 20 us, one of a count takes 20
// ns: the limits are some seconds.)
constexpr int kBarrierPolls = 400000, kCountPolls = 100000000;
__device__ __forceinline__ bool wait1(uint64_t& b, uint32_t parity, const Ctx& cx) {
  const uint32_t bar = smem_addr(&b);
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < kBarrierPolls; ++i) {
    if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
    if (*cx.abort) return false;
  }
  *cx.abort = 1;
  return false;
}
__device__ __forceinline__ bool wait_count(uint32_t& count, uint32_t least, const Ctx& cx) {
  const uint32_t at = smem_addr(&count);
#pragma unroll 1
  for (int i = 0; i < kCountPolls; ++i) {
    uint32_t c;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(c) : "r"(at) : "memory");
    if ((int)(c - least) >= 0) return true;
    if ((i & 1023) == 1023 && *cx.abort) return false;
  }
  *cx.abort = 1;
  return false;
}
__device__ __forceinline__ void set_count(uint32_t& count, uint32_t to) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(smem_addr(&count)), "r"(to) : "memory");
}
// Fill g of the ring: its slot is free / its data is there.
__device__ __forceinline__ bool wait_free(Smem& S, int g, const Ctx& cx) {
  const int slot = g % kStages, use = g / kStages;
  return use == 0 || (wait_count(S.armed[slot], use, cx) && wait1(S.empty[slot], (use - 1) & 1, cx));
}
__device__ __forceinline__ bool wait_filled(Smem& S, int g, const Ctx& cx) {
  const int slot = g % kStages, use = g / kStages;
  return wait_count(S.armed[slot], use + 1, cx) && wait1(S.full[slot], use & 1, cx);
}
// wait1 of a warp, its lanes agreeing on the outcome.
__device__ __forceinline__ bool wait(uint64_t& b, uint32_t parity, const Ctx& cx) {
  return __all_sync(0xffffffffu, wait1(b, parity, cx));
}
// The same by one thread, for copies in flight at the end, whatever the abort flag says.
__device__ __forceinline__ void drain(uint64_t& b, uint32_t parity, unsigned int* err) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_sleep(smem_addr(&b), parity, 20000))
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      raise_error(err, DSPARK_DEVERR_WAIT_TIMEOUT);
      return;
    }
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fused multiply-adds, or two additions, in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// A product whose operands' descriptors share their high word: one thread issues all of them, and
// what it computes between two is time the tensor cores wait (descriptors built whole: 150 cycles a
// product, twice what it takes).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// No use of a pending tmem load's registers is scheduled before the wait that this follows.
template <int N>
__device__ __forceinline__ void tie(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ AttnItem fetch(const Smem& S, const AttnItem* more, int it) {
  return it < 4 ? S.items[it] : more[it];
}
__device__ __forceinline__ int visible(int t, int ct, const AttnItem& x) {
  return min(t < ct ? x.ctx - t * kKT : x.n_r - (t - ct) * kKT, kKT);
}
// An item's fills of the ring, in the order in which the products take them, so that no slot is held
// longer than need be: two query tiles take K0 V0 K1 V1 .., two streams K0 K1 V0 K2 V1 .. (a
// stream's P V comes after the other's next S).
__device__ __forceinline__ int fill_of_k(int k, bool two) { return two ? 2 * k : max(2 * k - 1, 0); }
__device__ __forceinline__ int fill_of_v(int k, int nt, bool two) {
  return two ? 2 * k + 1 : k == nt - 1 ? 2 * nt - 1 : 2 * k + 2;
}

// A warp's window on a request's page table: lane j holds the page of slot first + j.
struct Pages {
  int first = -1, page = 0;
  __device__ __forceinline__ void look_up(const Params& p, const AttnItem& x, int t) {
    const int lp = p.log2_page, s0 = (int)(((long long)t * kKT) >> lp), ns = max(kKT >> lp, 1);
    if (first >= 0 && s0 + ns <= first + 32) return;
    first = s0;
    const int slot = first + (threadIdx.x & 31);
    page = 0;
    if (((long long)slot << lp) < x.ctx) {
      page = slot < p.max_pages ? p.page_table[(long long)x.r * p.max_pages + slot] : -1;
      // (a page that no cache holds: its keys read as zero)
      if (page < 0 || page >= p.n_pages) {
        raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
        page = p.n_pages;
      }
    }
  }
  __device__ __forceinline__ int of(int slot) const {
    return __shfl_sync(0xffffffffu, page, (slot - first) & 31);
  }
};

// After the outputs of query row n (block row b) of an item: the NaN and infinities of the values
// that it sees among the block rows of the item's tiles, in channels c0 .. c1 - 1.
__device__ __noinline__ void write_specials(const Params& p, const AttnItem& x, int n, int row,
                                            int c0, int c1) {
  const int ct = ceil_div(x.ctx, kKT), G = p.Hq / p.Hkv;
  const int b0 = max(x.tb - ct, 0) * kKT, b1 = min(min((x.te - ct) * kKT, x.n_r), 64 * p.words);
  const uint64_t* m = p.mask + (long long)row * p.words;
  const __nv_bfloat16* v = p.v_new + ((long long)x.c0 * p.Hkv + x.kvh) * kD;
  const long long step = (long long)p.Hkv * kD;
  for (int c = c0; c < c1; ++c) {
    float add = 0.f;
    for (int j = b0; j < b1; ++j) {
      if (!(m[j >> 6] >> (j & 63) & 1)) continue;
      const float f = __bfloat162float(v[j * step + c]);
      if (!(fabsf(f) <= 3.4e38f)) add += f;
    }
    if (add == 0.f) continue;
    if (x.nsplit > 1) {
      float* o = p.ws_o + ((long long)x.slot * p.slot_rows + n) * kD + c;
      *o += add;
    } else {
      __nv_bfloat16* o = p.out + ((long long)row * p.Hq + x.kvh * G + n % G) * kD + c;
      *o = __float2bfloat16(__bfloat162float(*o) + add);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    verify_attn_tree_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ CUtensorMap tm_kn,
                            const __grid_constant__ CUtensorMap tm_vn, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Smem& S = *reinterpret_cast<Smem*>(smem);
  const uint32_t q_base = smem_addr(smem) + kHead, ring = q_base + 2 * kTile;
  const Ctx cx{&S.abort, p.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    S.abort = 0;
    S.epilogues = S.turns[0] = S.turns[1] = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&S.full[i]), 1);
      mbar_init(smem_addr(&S.empty[i]), 2);  // the products of both streams
      S.armed[i] = S.looked[i] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&S.q_full[i]), 1);
      mbar_init(smem_addr(&S.q_empty[i]), 2);
      mbar_init(smem_addr(&S.s_full[i]), 1);
      mbar_init(smem_addr(&S.p_full[i]), 4);
      mbar_init(smem_addr(&S.pv_done[i]), 1);
    }
    mbar_init(smem_addr(&S.joined), 8);
    fence_mbar_init();
  }
  if (threadIdx.x < kFlags) S.special[threadIdx.x] = 0;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&S.tmem), 512);
    tmem_relinquish();
  }
  pdl_release();
  pdl_wait();  // inputs come from the kernels before this one
  const OwnItems own =
      own_items<kThreads, 4>(p, *reinterpret_cast<ItemScratch*>(smem + kHead + 2 * kTile), S.items);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const int G = p.Hq / p.Hkv;
  // 384 threads of 168 registers: 128 x 104 + 256 x 200
  if (warp < kSoftmaxWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (warp == kKWarp) {
    // ------------------------------------------------------------- K and Q
    const int lp = p.log2_page, rpt = p.tile_rows;
    int g0 = 0;                                  // fills of the items before
    int used0 = 0, used1 = 0, turn = 0;          // Q tiles loaded, the buffer of the next single one
    bool ok = true;
    for (int it = 0; it < own.n && ok; ++it) {
      const AttnItem x = fetch(S, own.more, it);
      const int ct = ceil_div(x.ctx, kKT), nt = x.te - x.tb;
      const bool two = x.ni > rpt;
      auto load_q = [&]() {
        for (int k = 0; k < (two ? 2 : 1) && ok; ++k) {
          const int b = two ? k : turn, u = b ? used1 : used0;
          if (u > 0) ok = wait(S.q_empty[b], (u - 1) & 1, cx);
          if (!ok) break;
          if (elect_one()) {
            const uint32_t bar = smem_addr(&S.q_full[b]);
            mbar_arrive_expect_tx(bar, (uint32_t)rpt * G * 256);
            for (int half = 0; half < 2; ++half)
              tma_load_3d(q_base + b * kTile + half * kHalf, &tm_q, bar, half * 64, x.kvh * G,
                          x.c0 + x.i0 + k * rpt);
          }
          __syncwarp();
          ++(b ? used1 : used0);
        }
        if (!two) turn ^= 1;
      };
      Pages pages;
      if (it == 0) load_q();
      for (int k = 0; k < nt && ok; ++k) {
        // Q's buffer is free once the last item's last S is done, which the third K waits for too
        if (k == min(2, nt - 1) && it > 0) load_q();
        const int g = g0 + fill_of_k(k, two);
        const int slot = g % kStages;
        if (!(ok = __all_sync(0xffffffffu, ok && wait_free(S, g, cx)))) break;
        const int t = x.tb + k;
        const bool cached = t < ct;
        const int lb = cached ? min(lp, 7) : 4;  // log2 of a box's keys
        const int nb = (visible(t, ct, x) + (1 << lb) - 1) >> lb;
        const uint32_t bar = smem_addr(&S.full[slot]), dst = ring + slot * kTile;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, nb * (256 << lb));
          if (!two) mbar_arrive(smem_addr(&S.empty[slot]));  // (for the stream that has no part in it)
          set_count(S.armed[slot], g / kStages + 1);
        }
        __syncwarp();
        if (cached) pages.look_up(p, x, t);
        // lane = (box, column half); at most 16 boxes
        const int bx = lane >> 1, half = lane & 1, at = t * kKT + (bx << lb);
        const int page = cached ? pages.of(at >> lp) : 0;
        if (bx < nb) {
          const uint32_t to = dst + half * kHalf + bx * (128 << lb);
          if (cached)
            tma_load_4d(to, &tm_k, bar, half * 64, x.kvh, at & ((1 << lp) - 1), page);
          else
            tma_load_3d(to, &tm_kn, bar, half * 64, x.kvh, x.c0 + (t - ct) * kKT + bx * kBoxRows);
        }
        __syncwarp();
      }
      g0 += 2 * nt;
    }
    if (elect_one()) {
      if (used0 > 0) drain(S.q_full[0], (used0 - 1) & 1, p.err);
      if (used1 > 0) drain(S.q_full[1], (used1 - 1) & 1, p.err);
    }
  } else if (warp == kVWarp) {
    // ------------------------------------------------------------- V, loaded and looked over
    const int lp = p.log2_page;
    int g0 = 0, g_last = -1;                     // fills of the items before; the fill to look over
    // of that fill: log2 of its boxes' keys, visible keys, whether block rows, its item
    int lb_last = 0, vis_last = 0, it_last = 0;
    bool new_last = false, ok = true;
    auto look = [&]() -> bool {
      if (g_last < 0) return true;
      const int slot = g_last % kStages;
      if (!wait(S.full[slot], (g_last / kStages) & 1, cx)) return false;
      if (new_last || (vis_last & 15)) {
        uint8_t* const v = smem + kHead + 2 * kTile + slot * kTile;
        const int lb = lb_last, vis = vis_last;
        // 16-byte piece o & 7 of key o >> 3 in a column half
        auto piece = [&](int o, int half) {
          const int key = o >> 3;
          return reinterpret_cast<uint4*>(v + ((key >> lb) << (lb + 8)) + (half << (lb + 7)) +
                                          ((key & ((1 << lb) - 1)) << 7) + (o & 7) * 16);
        };
        bool odd = false;
        if (new_last) {
          for (int o = lane; o < vis * 8; o += 32) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint4* const at = piece(o, half);
              const uint4 u = *at;
              // an exponent of ones carries into the bit above it
              const uint32_t ones =
                  (((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
                   ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u)) &
                  0x80008000u;
              if (ones) {
                odd = true;
                auto clear = [](uint32_t w) {
                  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
                  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
                  return w;
                };
                *at = make_uint4(clear(u.x), clear(u.y), clear(u.z), clear(u.w));
              }
            }
          }
        }
        // keys vis .. the end of their chunk of 16
        const int nz = (-vis & 15) * 8;
        for (int o = lane; o < 2 * nz; o += 32) {
          const int half = o >= nz;
          *piece(vis * 8 + o - (half ? nz : 0), half) = make_uint4(0, 0, 0, 0);
        }
        if (odd) S.special[it_last % kFlags] = 1;
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) set_count(S.looked[slot], g_last + 1);
      g_last = -1;
      return true;
    };
    for (int it = 0; it < own.n && ok; ++it) {
      const AttnItem x = fetch(S, own.more, it);
      const int ct = ceil_div(x.ctx, kKT), nt = x.te - x.tb;
      const bool two = x.ni > p.tile_rows;
      Pages pages;
      if (lane == 0) S.special[it % kFlags] = 0;
      __syncwarp();
      for (int k = 0; k < nt && ok; ++k) {
        const int g = g0 + fill_of_v(k, nt, two), slot = g % kStages;
        if (!(ok = __all_sync(0xffffffffu, wait_free(S, g, cx)))) break;
        const int t = x.tb + k, vis = visible(t, ct, x);
        const bool cached = t < ct;
        const int lb = cached ? min(lp, 7) : 4, nb = (vis + (1 << lb) - 1) >> lb;
        const uint32_t bar = smem_addr(&S.full[slot]), dst = ring + slot * kTile;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, nb * (256 << lb));
          if (!two) mbar_arrive(smem_addr(&S.empty[slot]));
          set_count(S.armed[slot], g / kStages + 1);
        }
        __syncwarp();
        if (cached) pages.look_up(p, x, t);
        const int bx = lane, at = t * kKT + (bx << lb);
        const int page = cached ? pages.of(at >> lp) : 0;
        if (bx < nb) {
          const uint32_t to = dst + bx * (256 << lb);
          if (cached)
            tma_load_5d(to, &tm_v, bar, 0, at & ((1 << lp) - 1), 0, x.kvh, page);
          else
            tma_load_4d(to, &tm_vn, bar, 0, x.c0 + (t - ct) * kKT + bx * kBoxRows, 0, x.kvh);
        }
        __syncwarp();
        // the fill before this one; its product comes after the one that made room here
        ok = look();
        g_last = g;
        lb_last = lb;
        vis_last = vis;
        new_last = !cached;
        it_last = it;
      }
      // (an item's last fill at once: its product may be what the next item's fills wait for)
      if (ok) ok = look();
      g0 += 2 * nt;
    }
  } else if (elect_one()) {
    // ------------------------------------------------------------- products
    // One thread for each stream: the two share the tensor cores, and the one waits and computes
    // addresses while the other's products run.
    constexpr uint32_t kQk = idesc_bf16_f32(kM, kKT, 0, 0), kPv = idesc_bf16_f32(kM, kD, 0, 1);
    const int s = warp == kMmaWarp ? 0 : 1;
    // (addresses are the low 14 bits, in 16 bytes, of a descriptor's low word)
    const uint64_t dq = smem_desc(q_base, 16, 1024, SW_128B), dk = smem_desc(ring, 16, 1024, SW_128B),
                   dv = smem_desc(ring, 0, 1024, SW_128B);
    const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32);
    const uint32_t v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);  // (its column halves: p_lb)
    const uint32_t t_s = tmem + kTmemS + s * 128, t_o = tmem + kTmemO + s * 128;
    // the product P V that is still to be issued: its item (-1: none), V's fill, chunks and log2 of
    // its boxes' keys, and whether it is the item's first
    int p_item = -1, p_fill = 0, p_nch = 0, p_lb = 4;
    bool p_first = false;
    int nv = 0, g = 0, used0 = 0, used1 = 0, turn = 0;
    bool ok = true;
    uint32_t at[8];          // of that V, each chunk's descriptor (what is computed between two
                             // products is time that the tensor cores wait)
    // what the product waits for, then the product
    auto p_ready = [&]() -> bool {
      const int slot = p_fill % kStages, lb = p_lb;
      // a box of 2^lb keys lies as its two column halves, one behind the other
      const uint32_t v = v_lo + slot * (kTile >> 4) + (8u << (lb + 16));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t key = 16 * k;
        at[k] = v + ((key >> lb) << (lb + 4)) + ((key & ((1u << lb) - 1)) << 3);
      }
      return (!p_first || wait_count(S.epilogues, 8 * p_item, cx)) &&  // O is free
             wait_count(S.looked[slot], p_fill + 1, cx) && wait1(S.p_full[s], (nv - 1) & 1, cx);
    };
    auto issue_pv = [&]() {
      const uint32_t old = p_first ? 0u : 1u;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < p_nch) mma_ts(t_o, t_s + k * 8, at[k], v_hi, kPv, k ? 1u : old);
      umma_commit(smem_addr(&S.pv_done[s]));
      umma_commit(smem_addr(&S.empty[p_fill % kStages]));
      p_item = -1;
    };
    uint32_t turns = 0;
    // (one round more, for the product that the last item left)
    for (int it = 0; it <= own.n && ok; ++it) {
      const bool end = it == own.n;
      AttnItem x{};
      if (!end) x = fetch(S, own.more, it);
      const int ct = ceil_div(x.ctx, kKT), nt = x.te - x.tb;
      const bool two = x.ni > p.tile_rows;
      const int qb = two ? s : turn, step = two ? 1 : 2;
      const uint32_t q = q_lo + qb * (kTile >> 4);
      const uint32_t q_par = (qb ? used1 : used0) & 1;
      bool first = true;
      for (int k = two ? 0 : s; first || k < nt; k += step, first = false) {
        // (a stream without a tile of the item comes by once, for what the last one left)
        const bool tile = k < nt;
        const int f = g + fill_of_k(k, two), slot = f % kStages;
        // Two query tiles take turns, so that one's softmax runs beside the other's products: left to
        // themselves both fall into step.
        if (tile && two && !(ok = wait_count(S.turns[s ^ 1], turns + s, cx))) break;
        if (p_item >= 0) {
          if (!(ok = p_ready())) break;
          issue_pv();
        }
        if (first && !end) {
          if (!(ok = wait1(S.q_full[qb], q_par, cx))) break;
          // (each stream follows both buffers' phases)
          if (two) {
            if (!(ok = wait1(S.q_full[qb ^ 1], (qb ? used0 : used1) & 1, cx))) break;
            mbar_arrive(smem_addr(&S.q_empty[qb ^ 1]));
          }
          if (!tile) mbar_arrive(smem_addr(&S.q_empty[qb]));
        }
        if (!tile) break;
        if (!(ok = wait_filled(S, f, cx))) break;
        const int vis = visible(x.tb + k, ct, x);
        const uint32_t kb = k_lo + slot * (kTile >> 4);
        tc_fence_after();
#pragma unroll
        for (int d = 0; d < kD / 16; ++d) {
          const uint32_t o = ((d >> 2) * kHalf + (d & 3) * 32) >> 4;
          mma_ss(t_s, q + o, kb + o, k_hi, kQk, d > 0 ? 1u : 0u);
        }
        if (two) set_count(S.turns[s], ++turns);
        umma_commit(smem_addr(&S.s_full[s]));
        umma_commit(smem_addr(&S.empty[slot]));
        if (k + step >= nt) umma_commit(smem_addr(&S.q_empty[qb]));
        ++nv;
        p_item = it;
        p_fill = g + fill_of_v(k, nt, two);
        p_lb = x.tb + k < ct ? min(p.log2_page, 7) : 4;
        p_nch = (vis + 15) >> 4;
        p_first = first;
      }
      if (two) {
        ++used0;
        ++used1;
      } else {
        ++(turn ? used1 : used0);
        turn ^= 1;
      }
      g += 2 * nt;
    }
    // whatever was issued completes before the memory is given back
    if (nv > 0) drain(S.s_full[s], (nv - 1) & 1, p.err);
    const int done = nv - (p_item >= 0 ? 1 : 0);
    if (done > 0) drain(S.pv_done[s], (done - 1) & 1, p.err);
  }
  __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax / epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int sw = warp & 3, s = (warp - kSoftmaxWarp) >> 2;
    const int n = sw * 32 + lane;  // row of the tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(sw * 32) << 16);
    const uint32_t t_s = t_lane + kTmemS + s * 128, t_o = t_lane + kTmemO + s * 128;
    const float sl2 = p.sl2;
    int nv[2] = {0, 0}, joins = 0;
    bool ok = true;
    for (int it = 0; it < own.n && ok; ++it) {
      const AttnItem x = fetch(S, own.more, it);
      const int ct = ceil_div(x.ctx, kKT), nt = x.te - x.tb, rpt = p.tile_rows;
      const bool two = x.ni > rpt;
      const int first_row = two && s ? rpt : 0;                       // of the item's rows
      const int nq = (min(x.ni, first_row + rpt) - first_row) * G;    // rows of this tile
      const bool warp_live = sw * 32 < nq, live = n < nq;
      const int row = x.c0 + x.i0 + first_row + min(n, nq - 1) / G;   // packed row
      const uint32_t* mrow = reinterpret_cast<const uint32_t*>(p.mask + (long long)row * p.words);
      const int mine = two ? nt : (nt + 1 - s) >> 1;                  // key tiles of this stream
      float ref = -INFINITY, sum = 0.f;
      for (int k = 0; k < mine; ++k) {
        const int t = x.tb + (two ? k : 2 * k + s);
        const int c = (s ? nv[1] : nv[0]) + k;
        if (!wait(S.s_full[s], c & 1, cx)) { ok = false; break; }
        if (warp_live) {
          tc_fence_after();
          float v[128];
          {
            float(&v0)[32] = reinterpret_cast<float(&)[32]>(v[0]);
            float(&v1)[32] = reinterpret_cast<float(&)[32]>(v[32]);
            float(&v2)[32] = reinterpret_cast<float(&)[32]>(v[64]);
            float(&v3)[32] = reinterpret_cast<float(&)[32]>(v[96]);
            tmem_ld32(t_s, v0);
            tmem_ld32(t_s + 32, v1);
            tmem_ld32(t_s + 64, v2);
            tmem_ld32(t_s + 96, v3);
            tmem_wait_ld();
            tie(v);
          }
          const int vis = visible(t, ct, x);
          if (t >= ct || vis < kKT) {
            // bits of the tile's 128 keys: visible at all, and of block rows those of the mask
            const int w0 = (t - ct) * 4;
            uint32_t bits[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int left = vis - 32 * w;
              bits[w] = t < ct ? ~0u : w0 + w < 2 * p.words ? mrow[w0 + w] : 0u;
              if (left < 32) bits[w] &= left <= 0 ? 0u : (1u << left) - 1u;
            }
#pragma unroll
            for (int j = 0; j < kKT; ++j) v[j] = (bits[j >> 5] >> (j & 31) & 1) ? v[j] : -INFINITY;
          }
          float m8[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) m8[j] = v[j];
#pragma unroll
          for (int j = 8; j < kKT; j += 16)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              m8[i] = j + 8 + i < kKT ? fmaxf(fmaxf(m8[i], v[j + i]), v[j + 8 + i]) : fmaxf(m8[i], v[j + i]);
          const float top = sl2 * fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                        fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
          const bool move = top > ref + 8.f;  // (from -inf: any key)
          const float alpha = move && ref != -INFINITY ? fast_exp2(ref - top) : 1.f;
          if (move) {
            ref = top;
            sum *= alpha;
          }
          if (k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O has the products up to the last tile once that is done
            if (!wait(S.pv_done[s], (c - 1) & 1, cx)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < kD; d += 16) {
              float o[16];
              tmem_ld16(t_o + d, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= alpha;
              tmem_st16(t_o + d, o);
            }
          }
          const float base = ref == -INFINITY ? 0.f : ref;
          const float2 f = make_float2(sl2, sl2), b = make_float2(-base, -base);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 e = fma2(make_float2(v[32 * q + 2 * j], v[32 * q + 2 * j + 1]), f, b);
              e.x = fast_exp2(e.x);
              e.y = fast_exp2(e.y);
              if (j & 1) acc1 = add2(acc1, e); else acc0 = add2(acc0, e);
              pk[j] = pack_bf16(e.x, e.y);
            }
            tmem_st16u(t_s + 16 * q, pk);
          }
          acc0 = add2(acc0, acc1);
          sum += acc0.x + acc0.y;
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&S.p_full[s]));
      }
      if (!ok) break;
      nv[0] += two ? nt : (nt + 1) >> 1;
      nv[1] += two ? nt : nt >> 1;
      // ---- epilogue: this stream's tile, or half the columns of both streams' sums
      if (two || s == 0 || nt > 1) ok = wait(S.pv_done[s], ((s ? nv[1] : nv[0]) - 1) & 1, cx);
      // (the other stream's phase is the last item's until that is done with)
      if (!two && ok) ok = __all_sync(0xffffffffu, wait_count(S.epilogues, 8 * it, cx));
      if (!two && ok && (s == 1 || nt > 1))
        ok = wait(S.pv_done[s ^ 1], ((s ? nv[0] : nv[1]) - 1) & 1, cx);
      if (!ok) break;
      if (!two) {
        // (the last item's numbers are read: its O was given back before the products waited for)
        S.ml[s][n][0] = ref;
        S.ml[s][n][1] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&S.joined));
        ok = wait(S.joined, joins & 1, cx);
        ++joins;
        if (!ok) break;
      }
      float w0 = 1.f, w1 = 0.f;  // weights of this stream's O and the other's
      if (!two) {
        const float r1 = S.ml[s ^ 1][n][0], s1 = S.ml[s ^ 1][n][1];
        const float r = fmaxf(ref, r1);
        w0 = ref == -INFINITY ? 0.f : fast_exp2(ref - r);
        w1 = r1 == -INFINITY ? 0.f : fast_exp2(r1 - r);
        if (sum != sum || s1 != s1) w0 = w1 = sum + s1;  // (NaN)
        sum = sum * w0 + s1 * w1;
        ref = r;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const bool split = x.nsplit > 1;
      const int nn = first_row * G + n;                                 // row of the item
      const int head = x.kvh * G + n % G;
      if (warp_live) {
        tc_fence_after();
        w0 *= inv;
        w1 *= inv;
        const int d0 = two ? 0 : 64 * s, d1 = two ? kD : d0 + 64;
        const uint32_t t_other = t_lane + kTmemO + (s ^ 1) * 128;
#pragma unroll 1
        for (int d = d0; d < d1; d += 32) {
          float o[32];
          tmem_ld32(t_o + d, o);
          tmem_wait_ld();
          tie(o);
          if (two) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= w0;
          } else {
            float u[32];
            tmem_ld32(t_other + d, u);
            tmem_wait_ld();
            tie(u);
            // (a stream without keys has no sums, whatever its columns hold)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = (w0 == 0.f ? 0.f : o[j] * w0) + (w1 == 0.f ? 0.f : u[j] * w1);
          }
          if (live) {
            if (split) {
              float4* dst = reinterpret_cast<float4*>(p.ws_o + ((long long)x.slot * p.slot_rows + nn) * kD + d);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(p.out + ((long long)row * p.Hq + head) * kD + d);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                dst[j] = make_uint4(pack_bf16(o[8 * j], o[8 * j + 1]), pack_bf16(o[8 * j + 2], o[8 * j + 3]),
                                    pack_bf16(o[8 * j + 4], o[8 * j + 5]), pack_bf16(o[8 * j + 6], o[8 * j + 7]));
            }
          }
        }
        if (live && (two || s == 0)) {
          const float l = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994530942f;
          if (split) p.ws_lse[(long long)x.slot * p.slot_rows + nn] = l;
          else p.lse[(long long)row * p.Hq + head] = l;
        }
        if (live && *(volatile int*)&S.special[it % kFlags]) write_specials(p, x, nn, row, d0, d1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;" ::"r"(smem_addr(&S.epilogues)) : "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && S.abort) raise_error(p.err, DSPARK_DEVERR_WAIT_TIMEOUT);
  if (threadIdx.x < kStages && S.armed[threadIdx.x] > 0)  // no copy is left in flight
    drain(S.full[threadIdx.x], (S.armed[threadIdx.x] - 1) & 1, p.err);
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- split combine
// Block (c, y): the split group recorded by CTA c, query rows 8y .. 8y + 7, a warp per row:
//   lse = log sum_s e^{lse_s},  o = sum_s e^{lse_s - lse} o_s
__global__ void __launch_bounds__(256)
    combine_tree_kernel(const int32_t* __restrict__ cu_seqlens, const SplitGroup* __restrict__ groups,
                        int G, int Hq, int slot_rows, const float* __restrict__ ws_o,
                        const float* __restrict__ ws_lse, __nv_bfloat16* __restrict__ out,
                        float* __restrict__ lse) {
  pdl_release();
  pdl_wait();  // inputs come from the kernels before this one
  const int lane = threadIdx.x & 31;
  const SplitGroup sg = groups[blockIdx.x];
  const int ns = sg.nsplit;
  const int n = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (ns <= 1 || n >= sg.ni * G) return;
  // piece s is in slot 2 (c_first + s), but for a first piece that is not its CTA's first
  auto slot = [&](int s) {
    return (long long)(2 * (sg.c_first + s) + (s == 0 && sg.slot0_last ? 1 : 0)) * slot_rows + n;
  };
  float mx = -INFINITY;
  for (int s = lane; s < ns; s += 32) mx = fmaxf(mx, ws_lse[slot(s)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < ns; s0 += 32) {
    // (a piece in which the row sees no key weighs nothing)
    const float l = s0 + lane < ns ? ws_lse[slot(s0 + lane)] : -INFINITY;
    const float wgt = l == -INFINITY ? 0.f : expf(l - mx);
    sum += wgt;
    const int m = min(32, ns - s0);
#pragma unroll 4
    for (int s = 0; s < m; ++s) {
      const float w = __shfl_sync(0xffffffffu, wgt, s);
      const float4 v = reinterpret_cast<const float4*>(ws_o + slot(s0 + s) * kD)[lane];
      acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const long long row = cu_seqlens[sg.r] + sg.i0 + n / G;
  const int head = sg.kvh * G + n % G;
  reinterpret_cast<uint2*>(out + (row * Hq + head) * kD)[lane] =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (lane == 0) lse[row * Hq + head] = sum == 0.f ? -INFINITY : mx + logf(sum);
}

// ---------------------------------------------------------------- host side
struct TreePlan {
  int tile_rows, rows_per_tile, slot_rows, ncta;
  size_t off_items, off_groups, off_o, off_lse, bytes;
};

TreePlan plan(int B, int max_rows, int Hq, int Hkv, int max_block_rows) {
  TreePlan p{};
  const int G = Hq / Hkv;
  p.tile_rows = kM / G;
  // Two query tiles to an item wherever a segment may need them: they share the keys.
  const int tiles = (max_block_rows > 0 ? max_block_rows : 1) > p.tile_rows ? 2 : 1;
  p.rows_per_tile = tiles * p.tile_rows;
  p.slot_rows = tiles * kM;
  p.ncta = num_sms_cached();
  if (p.ncta > kMaxCtas) p.ncta = kMaxCtas;
  const long long items = (long long)Hkv * ((long long)max_rows / p.rows_per_tile + B) + p.ncta;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~size_t(255);
    return at;
  };
  p.off_items = take(sizeof(AttnItem) * (size_t)items);
  p.off_groups = take(sizeof(SplitGroup) * (size_t)p.ncta);
  p.off_o = take(sizeof(float) * (size_t)2 * p.ncta * p.slot_rows * kD);  // slots 2c, 2c + 1
  p.off_lse = take(sizeof(float) * (size_t)2 * p.ncta * p.slot_rows);
  p.bytes = off;
  return p;
}

}  // namespace

size_t workspace(int B, int max_rows, int Hq, int Hkv, int max_block_rows) {
  return plan(B, max_rows, Hq, Hkv, max_block_rows).bytes;
}

int launch(const void* q, const void* k_new, const void* v_new, const void* k_cache,
           const void* v_cache, int n_pages, const int32_t* page_table, int max_pages,
           const int32_t* ctx_len, const int32_t* cu_seqlens, const uint64_t* mask, int words, int B,
           int max_rows, int Hq, int Hkv, int page_size, float scale, int max_splits,
           int max_block_rows, void* out, float* lse, void* ws, cudaStream_t stream) {
  const TreePlan pl = plan(B, max_rows, Hq, Hkv, max_block_rows);
  const int G = Hq / Hkv;
  uint8_t* w = static_cast<uint8_t*>(ws);
  Params p;
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.page_table = page_table;
  p.ctx_len = ctx_len;
  p.cu_seqlens = cu_seqlens;
  p.mask = mask;
  p.items = reinterpret_cast<AttnItem*>(w + pl.off_items);
  p.groups = reinterpret_cast<SplitGroup*>(w + pl.off_groups);
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
  p.words = words;
  p.B = B;
  p.max_rows = max_rows;
  p.rows_per_tile = pl.rows_per_tile;
  // five times as many pieces as asked for, so that 32 reach every SM with one long group
  p.max_splits = max_splits < 2 ? 2 : 5 * max_splits;
  p.tile_rows = pl.tile_rows;
  p.slot_rows = pl.slot_rows;
  p.sl2 = scale * 1.4426950408889634f;

  CUtensorMap tq, tk, tv, tkn, tvn;
  {
    const uint64_t dims[3] = {kD, (uint64_t)Hq, (uint64_t)max_rows};
    const uint64_t st[2] = {kD * 2, (uint64_t)Hq * kD * 2};
    const uint32_t box[3] = {64, (uint32_t)G, (uint32_t)pl.tile_rows};
    if (!gqa::encode_bf16_map(&tq, q, 3, dims, st, box)) return DSPARK_ECUDA;
  }
  const uint64_t H = (uint64_t)Hkv, P = (uint64_t)page_size, tok = H * kD * 2;
  const uint32_t keys = (uint32_t)(page_size < kKT ? page_size : kKT);
  {
    const uint64_t dims[4] = {kD, H, P, (uint64_t)n_pages}, st[3] = {kD * 2, tok, P * tok};
    const uint32_t box[4] = {64, 1, keys, 1};
    if (!gqa::encode_bf16_map(&tk, k_cache, 4, dims, st, box)) return DSPARK_ECUDA;
  }
  {  // V: a box brings both column halves
    const uint64_t dims[5] = {64, P, 2, H, (uint64_t)n_pages}, st[4] = {tok, 128, kD * 2, P * tok};
    const uint32_t box[5] = {64, keys, 2, 1, 1};
    if (!gqa::encode_bf16_map(&tv, v_cache, 5, dims, st, box)) return DSPARK_ECUDA;
  }
  {
    const uint64_t dims[3] = {kD, H, (uint64_t)max_rows}, st[2] = {kD * 2, tok};
    const uint32_t box[3] = {64, 1, kBoxRows};
    if (!gqa::encode_bf16_map(&tkn, k_new, 3, dims, st, box)) return DSPARK_ECUDA;
  }
  {
    const uint64_t dims[4] = {64, (uint64_t)max_rows, 2, H}, st[3] = {tok, 128, kD * 2};
    const uint32_t box[4] = {64, kBoxRows, 2, 1};
    if (!gqa::encode_bf16_map(&tvn, v_new, 4, dims, st, box)) return DSPARK_ECUDA;
  }
  static PerDevice<bool> done;
  if (!once_per_device(done, false, [] {
        return cudaFuncSetAttribute(verify_attn_tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kSmemBytes) == cudaSuccess;
      }))
    return DSPARK_ECUDA;
  if (launch_pdl(verify_attn_tree_kernel, dim3(pl.ncta), dim3(kThreads), kSmemBytes, stream, tq, tk, tv,
                 tkn, tvn, p) != cudaSuccess)
    return DSPARK_ECUDA;
  return launch_pdl(combine_tree_kernel, dim3(pl.ncta, pl.slot_rows / 8), dim3(256), 0, stream,
                    cu_seqlens, p.groups, G, Hq, pl.slot_rows, p.ws_o, p.ws_lse, p.out,
                    lse) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ECUDA;
}

}  // namespace tree
}  // namespace attn
}  // namespace dspark
