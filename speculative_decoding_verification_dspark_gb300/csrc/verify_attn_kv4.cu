// Varlen verify attention over a 4-bit paged KV cache (layout: kv4.cuh), GQA head dim 128.
//
// For packed row cu_seqlens[r] + i and query head h of KV group kvh:
//   o = softmax(scale q.K^T) V over the ctx_len[r] committed keys, whose K and V are
//   (code - 8) * scale * g, followed by block rows 0..i (bf16); lse = log-sum-exp.
//
// As in the bf16 cache's kernel, keys lie on the MMA's M side and the few query rows on
// N (32 columns), and the key tiles of all groups are cut into equal ranges, one per CTA
// (worklist.cuh):
//   S^T [128 keys x 32] = K [128 x 128] . Q^T        O^T [128 d x 32] += V^T [128 x 128] . P^T
// The left operands are in tensor memory: a lane of K is a key and a lane of V^T a channel,
// and the threads that read codes expand them and write their lanes.  Through shared memory
// the expanded tile would cost 64 KB of writes and 64 KB of MMA reads per 17 KB of cache,
// more than the SM's share of HBM time.
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
// What bounds it is not HBM but instructions: about a thousand per tile and scheduler
// against 850 cycles of HBM time, most of them in chains of one warp, which issues one
// in five or six cycles.  So every role is there twice and the CTA runs two streams, of the
// even and of the odd tiles, each a softmax of its own (references, sums, O^T) that meet
// at the end of an item.
//
// Warp roles (one CTA per SM; stream x = tiles of parity x):
//   warps 0, 1    issue S^T of stream 0, 1 (one lane)
//   warps 2, 3    issue O^T of stream 0, 1
//   warp 4        copies cache tiles into a ring of shared memory: one bulk copy per run
//                 of blocks that lie together (a block where pages hold 16 tokens), each
//                 from a lane of its own; owns the TMEM allocation
//   warp 5        query loader: the next item's rows into the other Q buffer
//   warps 8-15    K of stream 0, 1: thread = key; codes from the ring, expanded into TMEM
//   warps 16-23   V of stream 0, 1: warp = group of 32 channels.  A thread expands four
//                 channels (of every eighth) for a quarter of the tile's keys, so that the
//                 scales it reads (one per key and 32 channels) serve four words of codes.
//                 The products' key order is the one this gives: column pair 8 e + 2 q + i of
//                 V^T holds keys 32 q + 4 e + 2 i, + 1, and P is written in the same order
//   warps 24-31   softmax of stream 0, 1: thread = key; epilogue, thread = channel, 16 of
//                 the columns per stream's warps
// The softmax needs more registers than the launch gives a thread; the others hand theirs over.
// It takes a tile in one pass against its stream's row references; only if some key lies
// 2^8 above its row's maximum then (always in the stream's first tile of an item) does
// the tile go through the pass that moves references and rescales O.  Row sums stay in the
// threads (each sums its own keys) until the item ends.
// Every wait on an mbarrier is bounded in time (DSPARK_DEVERR_WAIT_TIMEOUT on expiry); the
// softmax warps' own barriers carry the failure, so that they leave together.

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
constexpr int kRingRows = 32;          // block rows of a tile that go through the ring
constexpr int kRowBytes = kD * 2;
constexpr int kRingV = kRingRows * kRowBytes;  // their V rows in the stage, after the K rows
constexpr int kSmemItems = 32;         // work items of a CTA kept in shared memory
constexpr int kNT = 32;                // query rows of a tile (MMA N)
constexpr int kPvWarp = 2, kCopyWarp = 4, kQWarp = 5, kKWarp0 = 8, kVWarp0 = 16,
              kSmWarp0 = 24, kThreads = 1024;
// Registers per thread at launch, and after the warpgroups have traded them: issuers, copy
// and query loader, K and V, softmax.
constexpr int kRegs = 65536 / kThreads, kRegsIssue = 40, kRegsLoad = 40, kRegsExpand = 56,
              kRegsSoftmax = 104;
static_assert(kRegsIssue + kRegsLoad + 4 * kRegsExpand + 2 * kRegsSoftmax <= 8 * kRegs, "register split");
constexpr float kRefDrop = 6.f;        // reference = maximum - 6 (log2)
constexpr float kMove = 14.f;          // a key above reference + 14 moves it
constexpr float kNoRef = -1e30f;       // reference of a row that has seen no key (`ref` holds the negatives)

// Shared memory (offsets from a 1024-byte boundary) and tensor memory (columns).
constexpr int kQCb = kNT * 128;                            // one 64-wide column block of Q
constexpr int kQBytes = 2 * kQCb;
constexpr int kPRow = kNT * 2, kPBytes = kKT * kPRow;
constexpr int kOffQ = 0;                                   // two items
constexpr int kOffP = kOffQ + 2 * kQBytes;                 // four tiles
constexpr int kOffRing = kOffP + 4 * kPBytes;
constexpr int kOffScale = kOffRing + kStages * kStageBytes;  // V scale pairs [8 warps][512 B]
constexpr int kOffCf = kOffScale + 8 * 512;                // softmax scale per row [2 items][32]
constexpr int kOffRef = kOffCf + 2 * 128;                  // negative references [8 warps][32]
constexpr int kOffAlpha = kOffRef + 8 * 128;               // factors [8 warps][2][32]
constexpr int kOffMax = kOffAlpha + 8 * 256;               // tile maxima [2 streams][4 warps][32]
constexpr int kOffSum = kOffMax + 2 * 512;                 // row sums [2 items][2 streams][4 warps][32]
constexpr int kOffItemRef = kOffSum + 4 * 512;             // references [2 items][2 streams][32]
constexpr int kOffItems = kOffItemRef + 4 * 128;
constexpr int kOffBar = kOffItems + kSmemItems * (int)sizeof(AttnItem);
constexpr int kBars = 26 + 2 * kStages;
constexpr int kOffMisc = kOffBar + kBars * 8;
constexpr int kSmemBytes = kOffMisc + 32 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");
static_assert(2 * kRingV <= kStageBytes, "block rows in a stage");
constexpr int kTmemS = 0, kTmemO = 4 * kNT, kTmemK = 8 * kNT, kTmemV = 8 * kNT + 128, kTmemCols = 512;
static_assert(kTmemV + 128 <= kTmemCols, "tensor memory");

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

// The barrier suspends the thread for up to 20 us a try; the clock is read only after 64.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Ctx& cx) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
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
// The same without suspending: for the issuers, whose wake-up is on every tile's path.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool spin_bar(uint32_t bar, uint32_t parity, const Ctx& cx) {
#pragma unroll 1
  for (int i = 0; i < 4096; ++i)
    if (mbar_test_wait(bar, parity)) return true;
  return wait_bar(bar, parity, cx);
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

// Barrier of `n` softmax threads that ors a flag over them.
__device__ __forceinline__ bool group_or(int id, int n, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)x)
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
// 16 lanes x 16 columns: thread t holds columns 8 e + 2 (t % 4) + {0, 1} of lane t / 4 in
// r[4 e], r[4 e + 1] and of lane t / 4 + 8 in r[4 e + 2], r[4 e + 3], e = 0, 1.
__device__ __forceinline__ void tmem_st_16x256b_x2(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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

__global__ void __launch_bounds__(kThreads, 1) verify_attn_kv4_kernel(const Params prm) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  AttnItem* s_items = reinterpret_cast<AttnItem*>(bp + kOffItems);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bp + kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bp + kOffMisc + 16);
  const Ctx cx{abort_flag, prm.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) { return base + kOffBar + 8 * i; };
  // Barriers.  Tile g belongs to stream g & 1; its operands K and V are that stream's, its
  // scores and probabilities are in S and P buffer g & 3.  Its QK^T releases the K operand with
  // s_full, its PV the V operand and P with pv_done.
  auto k_full = [&](int x) { return bar(0 + x); };
  auto v_full = [&](int x) { return bar(2 + x); };
  auto s_full = [&](int i) { return bar(4 + i); };
  auto s_free = [&](int i) { return bar(8 + i); };
  auto p_full = [&](int i) { return bar(12 + i); };
  auto pv_done = [&](int i) { return bar(16 + i); };
  auto q_full = [&](int i) { return bar(20 + i); };   // by item parity
  auto q_empty = [&](int i) { return bar(22 + i); };
  auto o_free = [&](int i) { return bar(24 + i); };
  auto c_full = [&](int i) { return bar(26 + i); };   // ring of cache tiles
  auto c_empty = [&](int i) { return bar(26 + kStages + i); };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full(i), 4);
      mbar_init(v_full(i), 4);
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 2 + 8);  // two issuers, eight softmax warps
      mbar_init(o_free(i), 8);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(s_free(i), 4);
      mbar_init(p_full(i), 1);
      mbar_init(pv_done(i), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(c_full(i), 1);
      mbar_init(c_empty(i), 8);  // a K and a V warpgroup
    }
    fence_mbar_init();
  }
  if (warp == kCopyWarp) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  pdl_release();
  pdl_wait();  // the work list and the step's inputs come from earlier kernels
  const int it_begin = prm.item_begin[blockIdx.x];
  const int it_end = prm.item_begin[blockIdx.x + 1];
  {
    const int n_s = min(kSmemItems, it_end - it_begin);
    constexpr int kWords = (int)(sizeof(AttnItem) / sizeof(uint4));
    for (int i = threadIdx.x; i < n_s * kWords; i += kThreads)
      reinterpret_cast<uint4*>(s_items)[i] = reinterpret_cast<const uint4*>(prm.items + it_begin)[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int G = prm.Hq / prm.Hkv;

  if (warp < kCopyWarp) {
    regs_down<kRegsIssue>();
    const int x = warp & 1;
    if (warp < kPvWarp) {
      // ----------------------------------------------------------- S^T = K Q^T
      constexpr uint32_t IDESC = idesc_f16_f32(kKT, kNT, 0);
      if (lane == 0) {
        const uint32_t a = tmem + kTmemK + x * 64;
        int g0 = 0, n_it = 0, last = -1;  // first tile of the item
        bool ok = true;
        for (int it = it_begin; it < it_end && ok; ++it, ++n_it) {
          const int k = it - it_begin;
          const AttnItem* item = k < kSmemItems ? s_items + k : prm.items + it;
          const int g1 = g0 + item->te - item->tb, qb = n_it & 1;
          if (!wait_bar(q_full(qb), (n_it >> 1) & 1, cx)) break;
          const uint64_t bd = smem_desc(base + kOffQ + qb * kQBytes, 16, 1024, SW_128B);
          int g = g0 + ((g0 ^ x) & 1);
          if (g >= g1) mbar_arrive(q_empty(qb));  // no tile of this stream in the item
          for (; g < g1; g += 2) {
            const int i = g & 3;
            ok = wait_bar(k_full(x), (g >> 1) & 1, cx) &&
                 (g < 4 || wait_bar(s_free(i), ((g >> 2) - 1) & 1, cx));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + kTmemS + i * kNT;
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk)
              umma_bf16_ts(d, a + kk * 8, bd + ((kk >> 2) * kQCb + (kk & 3) * 32) / 16, IDESC,
                           kk > 0 ? 1u : 0u);
            umma_commit(s_full(i));
            if (g + 2 >= g1) umma_commit(q_empty(qb));
            last = g;
          }
          g0 = g1;
        }
        if (last >= 0) drain_bar(s_full(last & 3), (last >> 2) & 1, prm.err);
      }
    } else {
      // ----------------------------------------------------------- O^T += V^T P^T
      constexpr uint32_t IDESC = idesc_f16_f32(kD, kNT, 1);
      if (lane == 0) {
        const uint32_t a = tmem + kTmemV + x * 64;
        int g0 = 0, n_it = 0, last = -1;
        bool ok = true;
        for (int it = it_begin; it < it_end && ok; ++it, ++n_it) {
          const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
          const int g1 = g0 + item.te - item.tb, ct = ceil_div(item.ctx, kKT);
          const uint32_t d = tmem + kTmemO + (2 * x + (n_it & 1)) * kNT;
          const int first = g0 + ((g0 ^ x) & 1);
          if (first < g1 && n_it >= 2 && !wait_bar(o_free(n_it & 1), ((n_it >> 1) - 1) & 1, cx)) break;
          for (int g = first; g < g1; g += 2) {
            ok = wait_bar(v_full(x), (g >> 1) & 1, cx) && wait_bar(p_full(g & 3), (g >> 2) & 1, cx);
            if (!ok) break;
            tc_fence_after();
            const uint64_t bd = smem_desc(base + kOffP + (g & 3) * kPBytes, kKT * 128, 8 * kPRow, SW_64B);
            const int t = item.tb + g - g0;
            umma_bf16_ts(d, a, bd, IDESC, g > first ? 1u : 0u);
            if (t < ct) {
#pragma unroll
              for (int kk = 1; kk < kKT / 16; ++kk)
                umma_bf16_ts(d, a + kk * 8, bd + kk * kPRow, IDESC, 1u);
            } else {
              // only the 16-row steps that hold a row
              const int nch = ceil_div(visible_keys(t, ct, item.ctx, item.n_r), 16);
#pragma unroll 1
              for (int kk = 1; kk < nch; ++kk) umma_bf16_ts(d, a + kk * 8, bd + kk * kPRow, IDESC, 1u);
            }
            umma_commit(pv_done(g & 3));
            last = g;
          }
          g0 = g1;
        }
        if (last >= 0) drain_bar(pv_done(last & 3), (last >> 2) & 1, prm.err);
      }
    }
    __syncwarp();
  } else if (warp < kKWarp0) {
    regs_down<kRegsLoad>();
    if (warp == kCopyWarp) {
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
    int g = 0, nxt = -1;
    bool ok = true;
    if (it_begin < it_end) {
      const AttnItem x = fetch_item(s_items, prm.items, it_begin, it_begin);
      nxt = lookup(x.r, x.ctx, x.tb);
    }
    for (int it = it_begin; it < it_end && ok; ++it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ct = ceil_div(item.ctx, kKT);
      for (int t0 = item.tb; t0 < item.te && ok; t0 += 4) {
        const int page = nxt;
        if (t0 + 4 < item.te) {
          nxt = lookup(item.r, item.ctx, t0 + 4);
        } else if (it + 1 < it_end) {
          const AttnItem x = fetch_item(s_items, prm.items, it + 1, it_begin);
          nxt = lookup(x.r, x.ctx, x.tb);
        }
        const int pos = (t0 + lt) * kKT + lb * kBlock;
        const bool want = pos < item.ctx && t0 + lt < item.te;
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
#pragma unroll 1
        for (int i = 0; i < 4 && t0 + i < item.te; ++i, ++g) {
          const int st = g & (kStages - 1);
          if (g >= kStages) {
            ok = wait_warp(c_empty(st), ((g / kStages) - 1) & 1, cx);
            if (!ok) break;
          }
          const uint32_t dst = base + kOffRing + st * kStageBytes;
          if (t0 + i < ct) {
            if (lane == 8 * i) mbar_arrive_expect_tx(c_full(st), total);
            __syncwarp();
            if (lt == i && bytes) bulk_load_g2s(dst + lb * kBlockBytes, src, bytes, c_full(st));
          } else {
            // the first block rows of a tile of them, K then V
            const int b0 = (t0 + i - ct) * kKT, rows = min(item.n_r - b0, kRingRows);
            if (lane == 0) mbar_arrive_expect_tx(c_full(st), (uint32_t)rows * 2 * kRowBytes);
            __syncwarp();
            if (lane < rows) {
              const long long off = ((long long)(item.c0 + b0 + lane) * prm.Hkv + item.kvh) * kD;
              bulk_load_g2s(dst + lane * kRowBytes, prm.k_new + off, kRowBytes, c_full(st));
              bulk_load_g2s(dst + kRingV + lane * kRowBytes, prm.v_new + off, kRowBytes, c_full(st));
            }
          }
        }
      }
    }
    // no copy may be in flight when the CTA ends
    for (int x = max(g - kStages, 0); x < g; ++x)
      if (lane == 0) drain_bar(c_full(x & (kStages - 1)), (x / kStages) & 1, prm.err);
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
      const uint32_t qd = base + kOffQ + qb * kQBytes;
      float* cf = reinterpret_cast<float*>(bp + kOffCf) + qb * kNT;
#pragma unroll 1
      for (int n0 = 0; n0 < kNT; n0 += 8) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + 2 * i + (lane >> 4);
          v[i] = make_uint4(0, 0, 0, 0);
          if (n < nq)
            v[i] = *reinterpret_cast<const uint4*>(
                prm.q + ((row0 + n / G) * prm.Hq + item.kvh * G + n % G) * kD + l * 8);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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
          st_shared_v4(qd + (l >> 3) * kQCb + sw128_off(n, l & 7), make_uint4(h[0], h[1], h[2], h[3]));
          if (l == 0)  // (never 0: a masked score is -inf times it)
            cf[n] = fmaxf(__uint_as_float((uint32_t)(e - 14) << 23) * prm.sl2, 1.17549435e-38f);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(qb));
    }
    }
  } else if (warp < kVWarp0) {
    regs_down<kRegsExpand>();
    // ------------------------------------------------------------- K: thread = key
    const int w = warp & 3, kl = w * 32 + lane;
    const int b = (warp - kKWarp0) >> 2;               // this warpgroup's tiles and operand buffer
    // this key's codes and scales within a stage
    const uint32_t ring = base + kOffRing + (2 * w + (lane >> 4)) * kBlockBytes;
    const uint32_t codes = ring + (lane & 15) * 16, scales = ring + kOffKs + (lane & 15) * 4;
    const uint32_t t_k = tmem + (static_cast<uint32_t>(w * 32) << 16) + kTmemK + b * 64;
    int g = 0;
    bool ok = true;
    for (int it = it_begin; it < it_end && ok; ++it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ct = ceil_div(item.ctx, kKT);
      for (int t = item.tb; t < item.te; ++t, ++g) {
        if ((g & 1) != b) continue;
        const int st = g & (kStages - 1);
        ok = wait_warp(c_full(st), (g / kStages) & 1, cx);
        if (ok && g >= 2) ok = wait_warp(s_full((g - 2) & 3), ((g - 2) >> 2) & 1, cx);  // its QK^T done
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
            tmem_st16u(t_k + c * 16, o);
          }
        } else {
          // the request's own rows: bf16 / (16 k_scale); the first ones from the ring
          const int bi = (t - ct) * kKT + kl;
          const __nv_bfloat16* src = prm.k_new + ((long long)(item.c0 + bi) * prm.Hkv + item.kvh) * kD;
          const uint32_t row = base + kOffRing + st * kStageBytes + kl * kRowBytes;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[j] = make_uint4(0, 0, 0, 0);
              if (bi < item.n_r)
                v[j] = kl < kRingRows ? ld_shared_v4(row + (c * 4 + j) * 16)
                                      : reinterpret_cast<const uint4*>(src)[c * 4 + j];
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
            tmem_st16u(t_k + c * 16, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(c_empty(st));
          mbar_arrive(k_full(b));
        }
      }
    }
  } else if (warp < kSmWarp0) {
    regs_down<kRegsExpand>();
    // ------------------------------------------------------------- V: thread = channel
    const int w = warp & 3;
    const int b = (warp - kVWarp0) >> 2;               // this warpgroup's tiles and operand buffer
    const uint32_t ring = base + kOffRing;
    // quad lane % 4 expands blocks 2 (lane % 4) and + 1, channels lane / 4 + 8 j of the warp's 32
    const uint32_t codes = ring + 2 * (lane & 3) * kBlockBytes + kOffV + (w * 32 + (lane >> 2)) * 8;
    const uint32_t scales = ring + (lane >> 2) * kBlockBytes + kOffVs + w * kBlock + (lane & 3) * 4;
    const uint32_t vs = base + kOffScale + (warp - kVWarp0) * 512;
    const uint32_t t_v = tmem + (static_cast<uint32_t>(w * 32) << 16) + kTmemV + b * 64;
    int g = 0;
    bool ok = true;
    for (int it = it_begin; it < it_end && ok; ++it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ct = ceil_div(item.ctx, kKT);
      for (int t = item.tb; t < item.te; ++t, ++g) {
        if ((g & 1) != b) continue;
        const int st = g & (kStages - 1);
        const int vis = visible_keys(t, ct, item.ctx, item.n_r);
        ok = wait_warp(c_full(st), (g / kStages) & 1, cx);
        if (t < ct) {
          // scale pairs of the tile's keys 4 lane .. + 3, shared by the warp's channels; keys
          // past the context get scale 0, whatever their page holds
          uint32_t sc = ld_shared(scales + st * kStageBytes);
          const int left = vis - 4 * lane;
          if (left < 4) sc = left <= 0 ? 0u : sc & ((1u << (8 * left)) - 1u);
          const uint32_t s0 = e4m3x2_to_h2(sc & 0xffffu), s1 = e4m3x2_to_h2(sc >> 16);
          const uint32_t at = vs + ((lane & 7) >> 1) * 128 + (lane >> 3) * 32 + (lane & 1) * 8;
          st_shared_v2(at, hmul2_bits(s0, kSixteenth), hmul2_bits(s1, k256th));
          st_shared_v2(at + 16, hmul2_bits(s0, kBiasLow), hmul2_bits(s1, kBiasHigh));
          __syncwarp();
        }
        if (ok && g >= 2) ok = wait_warp(pv_done((g - 2) & 3), ((g - 2) >> 2) & 1, cx);  // its PV done
        if (!ok) break;
        tc_fence_after();
        if (t < ct) {
          const uint32_t src = codes + st * kStageBytes;
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {  // the quad's two blocks
            uint2 v[4];                  // channels 8 j + lane / 4
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ld_shared_v2(src + u * kBlockBytes + j * 64);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t at = vs + (2 * u + h) * 128 + (lane & 3) * 32;
              const uint4 s = ld_shared_v4(at), c = ld_shared_v4(at + 16);
              const uint32_t ss[4] = {s.x, s.y, s.z, s.w}, bb[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
              for (int f = 0; f < 2; ++f) {  // lanes 0-15 and 16-31 of the quadrant
                uint32_t lo[4], hi[4];
                expand(h ? v[2 * f].y : v[2 * f].x, ss, bb, lo);
                expand(h ? v[2 * f + 1].y : v[2 * f + 1].x, ss, bb, hi);
                const uint32_t o[8] = {lo[0], lo[1], hi[0], hi[1], lo[2], lo[3], hi[2], hi[3]};
                tmem_st_16x256b_x2(t_v + (static_cast<uint32_t>(f * 16) << 16) + (2 * u + h) * 16, o);
              }
            }
          }
        } else {
          const int b0 = (t - ct) * kKT;
          const long long step = (long long)prm.Hkv * kD;
          const __nv_bfloat16* vn = prm.v_new + ((long long)(item.c0 + b0) * prm.Hkv + item.kvh) * kD +
                                    w * 32 + lane;
          const __nv_bfloat16* vr = reinterpret_cast<const __nv_bfloat16*>(
              bp + kOffRing + st * kStageBytes + kRingV) + w * 32 + lane;
          static_assert(kRingRows == 32, "one pair of V blocks");
#pragma unroll 1
          for (int i = 0; 32 * i < vis; ++i) {
            const __nv_bfloat16* from = i == 0 ? vr : vn + 32 * i * step;
            const long long by = i == 0 ? kD : step;
            float x[32];
#pragma unroll
            for (int j = 0; j < 32; ++j)
              x[j] = 32 * i + j < vis ? __bfloat162float(from[j * by]) : 0.f;
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pack16(x[2 * j] * prm.v_unit, x[2 * j + 1] * prm.v_unit);
            tmem_st16u(t_v + i * 16, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();  // (also: every lane has read its stage and the scale pairs)
        if (lane == 0) {
          mbar_arrive(c_empty(st));
          mbar_arrive(v_full(b));
        }
      }
    }
  } else {
    regs_up<kRegsSoftmax>();
    // ------------------------------------------------------------- softmax and epilogue
    const int sw = warp & 3, x = (warp - kSmWarp0) >> 2;
    const int kl = sw * 32 + lane;               // key of a tile, channel of O^T
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(sw * 32) << 16);
    const int bar_id = 1 + x, kBoth = 3;
    float* ref = reinterpret_cast<float*>(bp + kOffRef) + (warp - kSmWarp0) * 32;  // this warp's copies
    float* alpha = reinterpret_cast<float*>(bp + kOffAlpha) + (warp - kSmWarp0) * 64;
    float* tmax = reinterpret_cast<float*>(bp + kOffMax) + x * 128;                // [4 warps][32]
    // this key's step of the PV product in a cache tile, and in a block tile
    const int row_cache = 16 * (lane >> 2) + 4 * sw + (lane & 3);
    int g0 = 0, n_it = 0, last = -1;
    bool bad = false;                            // a wait ran out
    for (int it = it_begin; it < it_end; ++it, ++n_it) {
      const AttnItem item = fetch_item(s_items, prm.items, it, it_begin);
      const int ctx = item.ctx, ct = ceil_div(ctx, kKT);
      const int nq = item.ni * G;                // rows of the tile
      const int nc8 = (nq + 7) >> 3;
      const int ip = n_it & 1;
      const float* cf = reinterpret_cast<const float*>(bp + kOffCf) + ip * kNT;
      bad |= !wait_warp(q_full(ip), (n_it >> 1) & 1, cx);
      float mref = -INFINITY;                    // reference of row `lane`
      float lacc[32];                            // this thread's part of each row's sum
#pragma unroll
      for (int k = 0; k < 32; ++k) lacc[k] = 0.f;
      const int g1 = g0 + item.te - item.tb, first = g0 + ((g0 ^ x) & 1);
      const uint32_t t_o = t_lane + kTmemO + (2 * x + ip) * kNT;
#pragma unroll 1
      for (int g = first; g < g1; g += 2) {
        const int t = item.tb + g - g0, i = g & 3;
        bad |= !wait_warp(s_full(i), (g >> 2) & 1, cx);
        // the P buffer is free once the PV of tile g - 4 is done; that of g - 2 may still run
        if (g >= 4) bad |= !wait_warp(pv_done(i), ((g >> 2) - 1) & 1, cx);
        tc_fence_after();
        // row n sees this key iff n >= nmin
        const bool cached = t < ct;
        const bool masked = !cached || (t + 1) * kKT > ctx;  // some key is not seen by all rows
        int nmin = 0;
        if (masked) {
          const int bi = (t - ct) * kKT + kl;
          nmin = cached ? (t * kKT + kl < ctx ? 0 : 1 << 30)
                        : (bi < item.n_r ? (bi - item.i0) * G : 1 << 30);
        }
        const uint32_t s_col = t_lane + kTmemS + i * kNT;
        const int pr = cached ? row_cache : kl;
        const uint32_t pbuf = base + kOffP + i * kPBytes;
        float s[32];
        auto scores = [&]() {
          tmem_ld32(s_col, s);
          tmem_wait_ld32(s);
          if (masked) {
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = nmin <= k ? s[k] : -INFINITY;
          }
        };
        bool move = g == first;  // the references have to move first
        for (;;) {
          if (move) {
            // ---- the tile's maximum per row, over the stream's warps
            scores();
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] *= cf[k];
            tmax[sw * 32 + lane] = transpose_reduce<true>(s, lane);
            if (group_or(bar_id, 128, bad)) goto done;
            const float tm =
                fmaxf(fmaxf(tmax[lane], tmax[32 + lane]), fmaxf(tmax[64 + lane], tmax[96 + lane]));
            float al = 1.f;
            if (tm - kRefDrop > mref + (kMove - kRefDrop)) {
              al = mref == -INFINITY ? 0.f : fast_exp2(mref - (tm - kRefDrop));
              mref = tm - kRefDrop;
            }
            __syncwarp();
            ref[lane] = mref == -INFINITY ? -kNoRef : -mref;
            alpha[lane] = al;
            __syncwarp();
            if (g > first) {
              // O^T holds the products up to the stream's last tile before it is rescaled
              bad |= !wait_warp(pv_done((g - 2) & 3), ((g - 2) >> 2) & 1, cx);
              tc_fence_after();
              tmem_ld32(t_o, s);
              tmem_wait_ld32(s);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                lacc[k] *= alpha[k];
                s[k] *= alpha[k];
              }
              tmem_st32(t_o, s);
              tmem_wait_st();
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
              unpack(fma2(f2(s[k], s[k + 1]), f2(c4.x, c4.y), f2(r4.x, r4.y)), s[k], s[k + 1]);
              unpack(fma2(f2(s[k + 2], s[k + 3]), f2(c4.z, c4.w), f2(r4.z, r4.w)), s[k + 2], s[k + 3]);
              top = fmaxf(top, fmaxf(s[k], s[k + 1]));
              top = fmaxf(top, fmaxf(s[k + 2], s[k + 3]));
#pragma unroll
              for (int j = 0; j < 4; ++j) s[k + j] = fast_exp2(s[k + j]);
              pk[2 * h] = h2_bits(__floats2half2_rn(s[k], s[k + 1]));
              pk[2 * h + 1] = h2_bits(__floats2half2_rn(s[k + 2], s[k + 3]));
            }
            st_shared_v4(pbuf + sw64_off(pr, q), make_uint4(pk[0], pk[1], pk[2], pk[3]));
          }
          fence_proxy_async_smem();
          tc_fence_before();
          // all of P is written when the group passes; a key far above its row's reference
          // sends the tile through once more, after the references have moved
          const bool again = group_or(bar_id, 128, top > kMove || bad);
          if (!again) break;
          if (group_or(bar_id, 128, bad)) goto done;
          if (move) break;
          move = true;
        }
        if (lane == 0) mbar_arrive(s_free(i));
        if (sw == 0 && lane == 0) mbar_arrive(p_full(i));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= nc8) break;
#pragma unroll
          for (int k = q * 8; k < q * 8 + 8; k += 2)
            unpack(add2(f2(lacc[k], lacc[k + 1]), f2(s[k], s[k + 1])), lacc[k], lacc[k + 1]);
        }
        last = g;
      }
      // ---- epilogue: the two streams' row sums and references meet; the warps of stream x
      // write columns 16 x .. + 15 of (w0 O0 + w1 O1) / (w0 l0 + w1 l1), w = 2^(ref - max ref)
      {
        float* sums = reinterpret_cast<float*>(bp + kOffSum) + ip * 256;
        float* refs = reinterpret_cast<float*>(bp + kOffItemRef) + ip * 64;
        sums[x * 128 + sw * 32 + lane] = transpose_reduce<false>(lacc, lane);
        if (sw == 0) refs[x * 32 + lane] = mref;
        if (last >= g0) bad |= !wait_warp(pv_done(last & 3), (last >> 2) & 1, cx);  // O^T of this stream whole
        if (group_or(kBoth, 256, bad)) goto done;
        tc_fence_after();
        const float r0 = refs[lane], r1 = refs[32 + lane], m = fmaxf(r0, r1);
        const float w0 = r0 == -INFINITY ? 0.f : fast_exp2(r0 - m);
        const float w1 = r1 == -INFINITY ? 0.f : fast_exp2(r1 - m);
        const float l0 = (sums[lane] + sums[32 + lane]) + (sums[64 + lane] + sums[96 + lane]);
        const float l1 = (sums[128 + lane] + sums[160 + lane]) + (sums[192 + lane] + sums[224 + lane]);
        const float l = w0 * l0 + w1 * l1;
        const float inv = l == 0.f ? 0.f : prm.o_unit / l;
        alpha[lane] = w0 * inv;
        alpha[32 + lane] = w1 * inv;
        const bool split = item.nsplit > 1;
        const long long row0 = (long long)item.c0 + item.i0;
        if (x == 0 && sw == 0 && lane < nq) {
          const float v = (m + log2f(l)) * 0.69314718055994530942f;
          if (split)
            prm.ws_lse[(long long)item.slot * kKT + lane] = v;
          else
            prm.lse[(row0 + lane / G) * prm.Hq + item.kvh * G + lane % G] = v;
        }
        __syncwarp();
        float o[16];
#pragma unroll
        for (int n = 0; n < 16; ++n) o[n] = 0.f;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          if (g0 + ((g0 ^ y) & 1) >= g1) continue;  // that stream had no tile here
          float u[16];
          tmem_ld16(t_lane + kTmemO + (2 * y + ip) * kNT + 16 * x, u);
          tmem_wait_ld16(u);
#pragma unroll
          for (int n = 0; n < 16; ++n) o[n] = fmaf(u[n], alpha[32 * y + 16 * x + n], o[n]);
        }
        if (split) {
          float* dst = prm.ws_o + ((long long)item.slot * kKT + 16 * x) * kD + kl;
#pragma unroll
          for (int n = 0; n < 16; ++n)
            if (16 * x + n < nq) dst[n * kD] = o[n];
        } else {
          int h = (16 * x) % G;
          __nv_bfloat16* dst = prm.out + ((row0 + 16 * x / G) * prm.Hq + item.kvh * G + h) * kD + kl;
          const long long next = (long long)(prm.Hq - G) * kD;  // to the next block row's heads
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            if (16 * x + n < nq) *dst = __float2bfloat16(o[n]);
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
        mbar_arrive(o_free(ip));
        mbar_arrive(q_empty(ip));
      }
      g0 = g1;
    }
  done:;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kCopyWarp) tmem_dealloc(tmem, kTmemCols);
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
static bool configure() {
  static PerDevice<bool> done;
  return once_per_device(done, false, [] {
    return cudaFuncSetAttribute(verify_attn_kv4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemBytes) == cudaSuccess;
  });
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
  if (!configure()) return DSPARK_ECUDA;
  if (launch_pdl(verify_attn_kv4_kernel, dim3(pl.ncta), dim3(kThreads), kSmemBytes, stream, p) !=
      cudaSuccess)
    return DSPARK_ECUDA;
  return launch_pdl(combine_kv4_kernel, dim3(pl.ncta, kNT / 8), dim3(256), 0, stream, cu_seqlens,
                    groups, Hq / Hkv, Hq, p.ws_o, p.ws_lse, p.out, lse, B, max_rows,
                    p.err) == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

}  // namespace kv4a
}  // namespace attn
}  // namespace dspark
