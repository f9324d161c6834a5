// Varlen verify attention over a 4-bit paged KV cache (layout: kv4.cuh), GQA head dim 128.
//
// For packed row cu_seqlens[r] + i and query head h of KV group kvh:
//   o = softmax(scale q.K^T) V over the ctx_len[r] committed keys, whose K and V are
//   (code - 8) * scale * g, followed by block rows 0..i (bf16); lse = log-sum-exp.
//
// For query tiles of 17 to 64 rows.  As in the bf16 cache's kernel, keys lie on the MMA's M
// side and the query rows on N:
//   S^T [128 keys x N] = K [128 x 128] . Q^T        O^T [128 d x N] += V^T [128 x 128] . P^T
// by tcgen05.mma with the left operand in tensor memory, written there by the threads that
// expand the codes.  A CTA, two to an SM, persistent over its share of the key tiles
// (own_items), is nine warps: four expand K (thread = key), a tile ahead; four expand V
// (the warp's 32 channels); then all eight weigh, each half of them N / 2 of the rows
// (thread = key).  One barrier of the eight per tile votes on the references, one hands P(t),
// V(t) and K(t + 1) to the ninth warp, which issues S^T(t + 1) and O^T(t) and refills the ring.
//
// Why so.  Measured with time stamps of the warps: a thread that issues the eight
// instructions of a product is held for 700 to 1700 cycles (they queue behind the other CTA's), so
// no warp that computes may issue; with it, K's and V's operands in columns of their own, and V's
// in halves that go round, so that an expansion hardly waits for a product, a tile of 32 rows
// takes 3200 cycles per CTA (two share an SM), 5800 before (131k contexts 194 us -> 155).
// S^T(t + 1) goes first: K's expansion waits for it and is on the longer path (170 us against
// 175).  Half of K's expansion given to V's warps: 160.  Warps of six different loops (K, V, two
// softmax streams, issuers) needed 2.2 us a tile; teams of four warps that do everything in
// turn, four to an SM, 170 us and no more than 32 rows.  More rows than 64 do not fit: N columns
// of S^T, N of O^T, 64 of K and 64 or more of V in half of the 512.  A ring of two tiles is a
// third slower, one of four no faster.
//
// Bound by the chain of a tile's steps: 0.53 instructions per cycle and scheduler, 950 a tile of
// 32 rows (K 180, V 190, softmax 110, the rest waits, addresses and loops of nine warps), the
// tensor pipe 13% busy; with two of the products' 16 instructions left it is 17% faster, without
// the expansion of K (V) 9% (16%).  131k contexts of 3 requests (428 MB): 154 us, 2.8 TB/s.
// Registers: 96 a thread, the most that two CTAs leave; 44, 152 and 268 bytes are spilled with 32, 48
// and 64 rows.

#include "kv4_attn.cuh"

namespace dspark {
namespace attn {
namespace kv4a {

using namespace ptx;

constexpr int kTeam = 256;             // two warps for each quarter of the lanes that expand and weigh;
constexpr int kThreads = 288;          // a ninth copies and issues the products
constexpr int kStages = 3;

// Shared memory of a tile of up to N query rows (N a multiple of 16; each half of the team has
// N / 2), from a 1024-byte boundary.  Q lies K-major in two column blocks of 64 dims, P with the
// rows along a line of 64 bytes (32 of them) in blocks of 128 keys.
template <int N>
struct WideSmem {
  static constexpr int kHalf = N / 2;
  static constexpr int kQBytes = N * 128, kPBlock = kKT * 64;
  __align__(1024) uint8_t q[2 * kQBytes];
  __align__(1024) uint8_t p[(N + 31) / 32 * kPBlock];
  __align__(128) uint8_t ring[kStages][kStageBytes];
  __align__(16) uint8_t scale[4][512];   // V's scale pairs, per warp of half 1
  __align__(16) float cf[N];             // softmax scale per row
  __align__(16) float ref[8][kHalf];     // negative references, per warp
  __align__(16) float alpha[8][kHalf];   // factors, per warp
  float red[8][kHalf];                   // maxima of a tile, row sums of an item, per warp
  int nan[4];                            // a NaN among the item's values, per warp of half 1
  __align__(16) AttnItem items[kSmemItems];
  __align__(8) uint64_t full[kStages], qk_done, pv_half, pv_done;
  uint32_t tmem;
};
constexpr int kTmemCols = 256;         // S^T and O^T N each, K 64, the rest V's
// V's operand lies in halves of 64 keys (32 columns) that go round as many places as there are.
constexpr int v_places(int N) { return (kTmemCols - 2 * N - 64) / 32; }

__device__ __forceinline__ uint32_t sw128_off(int row, int chunk) {
  return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}
__device__ __forceinline__ uint32_t sw64_off(int row, int chunk) {
  return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
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
// 16 lanes x 16 columns: thread t holds columns 8 e + 2 (t % 4) + {0, 1} of lane t / 4 in
// r[4 e], r[4 e + 1] and of lane t / 4 + 8 in r[4 e + 2], r[4 e + 3], e = 0, 1.
__device__ __forceinline__ void tmem_st_16x256b_x2(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// fp16 x fp16 -> fp32 instruction descriptor, A in tensor memory (K-major), B K-major or
// MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// op over the warp of eight values per lane: lane l returns that of v[l & 7].
template <bool MAX>
__device__ __forceinline__ float reduce8(float (&v)[8], int lane) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + o], o);
      v[i] = op(up ? v[i + o] : v[i], other);
    }
  }
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 8));
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// Barrier of the team, the same that ors a flag over it, and the one that hands operands to the
// ninth warp (the team arrives, that warp waits).
__device__ __forceinline__ void team_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kTeam) : "memory"); }
__device__ __forceinline__ bool team_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %2, 0;\n\t"
      "barrier.cta.red.or.pred p, 1, %1, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "n"(kTeam), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void hand_over() { asm volatile("barrier.cta.arrive 2, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ void take_over() { asm volatile("barrier.cta.sync 2, %0;" ::"n"(kThreads) : "memory"); }

// The cache tiles of a CTA in order, for the warp that copies them into the ring.  Lane j knows
// block j % 8 of tile j / 8 of a window of four tiles; the pages of a window are read while
// the window before it is copied, so that nothing waits for the page table.
struct Copier {
  const Params& p;
  const AttnItem* s_items;
  OwnItems own;
  int it, t, te, r, ctx, kvh;  // the next tile to copy (te: end of the item's cache tiles)
  int window;                  // first tile of the window, -1: none yet
  int block;                   // this lane's block, by its index among all blocks of the cache; -1: none
  int page;                    // and its page in the next window
  bool holds;                  // where that block holds a committed key of the item's tiles
  int stage;
  __device__ __forceinline__ void look(int lane, int t0) {
    const int pos = t0 * kKT + lane * kBlock, slot = pos >> p.log2_page;
    holds = pos < ctx && t0 + (lane >> 3) < te;
    page = holds && slot < p.max_pages ? __ldg(p.page_table + (long long)r * p.max_pages + slot) : -1;
  }
  // The first item from `at` on that has cache tiles, and the pages of its first window.
  __device__ __forceinline__ void start(int lane, int at) {
    for (it = at; it < own.n; ++it) {
      const AttnItem x = fetch_item(s_items, own.more, it);
      t = x.tb; r = x.r; ctx = x.ctx; kvh = x.kvh;
      te = min(x.te, ceil_div(ctx, kKT));
      if (t < te) break;
    }
    window = -1;
    if (it < own.n) look(lane, t);
  }
  // The next tile into its stage.
  __device__ __forceinline__ void copy(int lane, uint32_t ring, uint32_t full) {
    if (it >= own.n) return;
    if (window < 0 || t == window + 4) {
      window = t;
      block = -1;
      if ((unsigned)page < (unsigned)p.n_pages) {
        const int lp = p.log2_page - 4, pos = t * kKT + lane * kBlock;
        block = ((page * p.Hkv + kvh) << lp) + ((pos >> 4) & ((1 << lp) - 1));
      } else if (holds) {
        raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
      }
      if (t + 4 < te) look(lane, t + 4);
    }
    const int first = 8 * (t - window);  // lanes first .. first + 7 hold the tile's blocks
    const bool mine = (lane & ~7) == first && block >= 0;
    const unsigned n = __popc(__ballot_sync(0xffffffffu, mine));
    const uint32_t bar = full + 8 * stage;
    if (lane == 0) mbar_arrive_expect_tx(bar, n * kBlockBytes);
    __syncwarp();
    if (mine)
      bulk_load_g2s(ring + stage * kStageBytes + (lane & 7) * kBlockStride,
                    p.cache + (long long)block * kBlockBytes, kBlockBytes, bar);
    if (++stage == kStages) stage = 0;
    if (++t == te) start(lane, it + 1);
  }
};

template <int N>
__global__ void __launch_bounds__(kThreads, kWideCtasPerSm) verify_attn_kv4_wide_kernel(const Params prm) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  WideSmem<N>& S = *reinterpret_cast<WideSmem<N>*>(smem_raw + (((raw + 1023u) & ~1023u) - raw));
  constexpr int NH = N / 2;
  constexpr int kTmemO = 0, kTmemS = N, kTmemK = 2 * N, kTmemV = 2 * N + 64, kPlaces = v_places(N);
  static_assert(kPlaces >= 2, "tensor memory");
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, wq = w & 3, half = w >> 2;
  const uint32_t ring = smem_addr(S.ring), full = smem_addr(S.full);
  const uint32_t qk_done = smem_addr(&S.qk_done);
  const uint32_t pv_half = smem_addr(&S.pv_half), pv_done = smem_addr(&S.pv_done);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1);
    mbar_init(qk_done, 1);
    mbar_init(pv_half, 1);
    mbar_init(pv_done, 1);
    fence_mbar_init();
  }
  pdl_wait();  // the step's inputs come from earlier kernels (no early release, as there)
  static_assert(sizeof(ItemScratch) <= sizeof(S.ring), "the scratch lies in the ring");
  const OwnItems own = own_items<kThreads>(prm, *reinterpret_cast<ItemScratch*>(S.ring), S.items);
  if (own.n == 0) return;
  if (w == 0) {
    tmem_alloc(smem_addr(&S.tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem;
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
  const int G = prm.Hq / prm.Hkv;
  const int kl = 32 * wq + lane;               // key of a tile, channel of O^T
  uint32_t magic;  // 1024 twice; opaque, so that it stays in a register
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
  if (w == 8) {
    Copier cp{prm, S.items, own};
    cp.stage = 0;
    cp.start(lane, 0);
    for (int i = 0; i < kStages; ++i) cp.copy(lane, ring, full);
    const uint64_t q_desc = smem_desc(smem_addr(S.q), 16, 1024, SW_128B);
    int place = 0;  // of V's next half
    const uint64_t p_desc = smem_desc(smem_addr(S.p), WideSmem<N>::kPBlock, 512, SW_64B);
    for (int it = 0; it < own.n; ++it) {
      const AttnItem item = fetch_item(S.items, own.more, it);
      const int ct = ceil_div(item.ctx, kKT), n_mma = (item.ni * G + 15) & ~15;
      const uint32_t qk_idesc = idesc_f16_f32(kKT, n_mma, 0), pv_idesc = idesc_f16_f32(kD, n_mma, 1);
      for (int t = item.tb - 1; t < item.te; ++t) {
        take_over();  // Q and K of tile tb; P and V of tile t and K of t + 1
        tc_fence_after();
        const bool cached = t < ct;
        if (lane == 0) {
          if (t + 1 < item.te) {
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk)
              umma_bf16_ts(tmem + kTmemS, tmem + kTmemK + kk * 8,
                           q_desc + ((kk >> 2) * WideSmem<N>::kQBytes + (kk & 3) * 32) / 16, qk_idesc,
                           kk > 0 ? 1u : 0u);
            umma_commit(qk_done);
          }
          if (t >= item.tb) {
            // of a block tile only the 16-row steps that hold a row
            const int nch = cached ? kKT / 16 : ceil_div(min(item.n_r - (t - ct) * kKT, kKT), 16);
            const uint32_t acc = t > item.tb ? 1u : 0u;
            const uint32_t v0 = tmem + kTmemV + place * 32;
            const uint32_t v1 = tmem + kTmemV + (place + 1 == kPlaces ? 0 : place + 1) * 32;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < nch)
                umma_bf16_ts(tmem + kTmemO, v0 + kk * 8, p_desc + kk * 64, pv_idesc, kk > 0 ? 1u : acc);
            umma_commit(pv_half);
#pragma unroll
            for (int kk = 4; kk < 8; ++kk)
              if (kk < nch) umma_bf16_ts(tmem + kTmemO, v1 + (kk - 4) * 8, p_desc + kk * 64, pv_idesc, 1u);
            umma_commit(pv_done);
          }
        }
        __syncwarp();
        if (t >= item.tb) place = (place + 2) % kPlaces;
        if (t >= item.tb && cached) cp.copy(lane, ring, full);  // the stage has been read by all
      }
    }
  } else {
    const float* const cf = S.cf + half * NH;
    float* const ref = S.ref[w];
    float* const alpha = S.alpha[w];
    int stage = 0;                 // of the next cache tile, for V
    int k_stage = 0, k_parity = 0;  // and for K, a tile ahead
    int g = 0;                      // tiles
    int place = 0;                  // of V's next half

    // ---- Q: tile row n = (block row n / G, head kvh G + n % G), a half-warp holds a row, 8 dims per
    // lane; read at the end of the item before
    const int G_inv = 65535 / G + 1;             // n / G = n G_inv >> 16 for n < 80, G <= 32
    uint4 qv[N / 16];
    auto load_q = [&](const AttnItem& x) {
      const long long row = (long long)x.c0 + x.i0;
      const int n_q = x.ni * G;
#pragma unroll
      for (int i = 0; i < N / 16; ++i) {
        const int n = 16 * i + 2 * w + (lane >> 4), r = (n * G_inv) >> 16;
        qv[i] = make_uint4(0, 0, 0, 0);
        if (n < n_q)
          qv[i] = *reinterpret_cast<const uint4*>(
              prm.q + ((row + r) * prm.Hq + x.kvh * G + n - r * G) * kD + (lane & 15) * 8);
      }
    };
    load_q(S.items[0]);

    for (int it = 0; it < own.n; ++it) {
      const AttnItem item = fetch_item(S.items, own.more, it);
      const int ctx = item.ctx, ct = ceil_div(ctx, kKT);
      const int nq = item.ni * G;              // rows of the tile
      const long long row0 = (long long)item.c0 + item.i0;
      // ---- Q as fp16 scaled by a power of two per row
      {
        const int l = lane & 15;
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
          const int n = 16 * i + 2 * w + (lane >> 4);
          const uint32_t x[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
          uint32_t top = 0;  // largest magnitude, as bits (a NaN is above all)
#pragma unroll
          for (int j = 0; j < 4; ++j) top = max(top, max((x[j] << 16) & 0x7fffffffu, x[j] & 0x7fff0000u));
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          // the largest element's power of two, no smaller than 2^-100 (fp32 holds 2^114)
          const int e = max((int)(top >> 23), 27);
          const float f = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = h2_bits(__floats2half2_rn(bf_lo(x[j]) * f, bf_hi(x[j]) * f));
          st_shared_v4(smem_addr(S.q) + (l >> 3) * WideSmem<N>::kQBytes + sw128_off(n, l & 7),
                       make_uint4(h[0], h[1], h[2], h[3]));
          if (l == 0)  // (never 0: a masked score is -inf times it)
            S.cf[n] = fmaxf(__uint_as_float((uint32_t)(e - 14) << 23) * prm.sl2, 1.17549435e-38f);
        }
        fence_proxy_async_smem();
      }
      for (int k = lane; k < NH; k += 32) ref[k] = -kNoRef;
      float lacc[NH];                            // this thread's part of each row's sum
#pragma unroll
      for (int k = 0; k < NH; ++k) lacc[k] = 0.f;

      // ---- K of tile t into its operand columns: thread = key (half 0)
      auto expand_k = [&](int t) {
        const bool cached = t < ct;
        const int vis = min(item.n_r - (t - ct) * kKT, kKT);  // (of a block tile)
        if (cached) {
          wait_bar(full + 8 * k_stage, k_parity, prm.err);
          const uint32_t tile = ring + k_stage * kStageBytes;
          if (++k_stage == kStages) {
            k_stage = 0;
            k_parity ^= 1;
          }
          const uint32_t blk = tile + (kl >> 4) * kBlockStride;
          const uint32_t sc = ld_shared(blk + kOffKs + (kl & 15) * 4);
          const uint32_t s01 = e4m3_low(sc), s23 = e4m3_high(sc);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 v = ld_shared_v4(blk + c * 256 + (kl & 15) * 16);
            const uint32_t s = __byte_perm(c < 2 ? s01 : s23, 0, (c & 1) ? 0x3232 : 0x1010);
            const uint32_t sl = hmul2_bits(s, kSixteenth), bl = hmul2_bits(s, kBiasLow);
            const uint32_t sh = hmul2_bits(s, k256th), bh = hmul2_bits(s, kBiasHigh);
            uint32_t o[16], x[4];
            const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              expand(word[q], magic, sl, bl, sh, bh, sl, bl, sh, bh, x);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[4 * q + e] = x[e];
            }
            tmem_st16u(t_lane + kTmemK + c * 16, o);
          }
        } else if (32 * wq < vis) {  // (other keys are masked, whatever the columns hold)
          // the request's own rows: bf16 / (16 k_scale)
          const int bi = (t - ct) * kKT + min(kl, vis - 1);  // (past the last row that row again)
          const uint4* src = reinterpret_cast<const uint4*>(
              prm.k_new + ((long long)(item.c0 + bi) * prm.Hkv + item.kvh) * kD);
#pragma unroll 2
          for (int c = 0; c < 4; ++c) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = src[c * 4 + j];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (kl >= vis) v[j] = make_uint4(0, 0, 0, 0);
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                o[4 * j + q] = pack16(bf_lo(x[q]) * prm.k_unit, bf_hi(x[q]) * prm.k_unit);
            }
            tmem_st16u(t_lane + kTmemK + c * 16, o);
          }
        }
        tmem_wait_st();
      };
      if (half == 0) expand_k(item.tb);
      tc_fence_before();
      hand_over();
      team_sync();  // cf
      if (half == 1) {
        if (lane == 0) S.nan[wq] = 0;   // (the epilogue before has been left by all)
        __syncwarp();
      }

#pragma unroll 1
      for (int t = item.tb; t < item.te; ++t, ++g) {
        const bool cached = t < ct;
        const int vis = cached ? min(ctx - t * kKT, kKT) : min(item.n_r - (t - ct) * kKT, kKT);
        const uint32_t tile = ring + stage * kStageBytes;
        if (half == 1) {
          // ---- V's scale pairs of keys 4 lane .. + 3, shared by the warp's channels; keys past the
          // context get scale 0, whatever their page holds
          const uint32_t vs = smem_addr(S.scale[wq]);
          if (cached) {
            uint32_t sc = ld_shared(tile + (lane >> 2) * kBlockStride + kOffVs + wq * kBlock + (lane & 3) * 4);
            const int left = vis - 4 * lane;
            if (left < 4) sc = left <= 0 ? 0u : sc & ((1u << (8 * left)) - 1u);
            const uint32_t s0 = e4m3_low(sc), s1 = e4m3_high(sc);
            const uint32_t at = vs + ((lane & 7) >> 1) * 128 + (lane >> 3) * 32 + (lane & 1) * 8;
            st_shared_v2(at, hmul2_bits(s0, kSixteenth), hmul2_bits(s1, k256th));
            st_shared_v2(at + 16, hmul2_bits(s0, kBiasLow), hmul2_bits(s1, kBiasHigh));
            __syncwarp();
          }
          // The places of the next two halves.  The products of the tile before last are done (this
          // thread waited for them when it wrote P), so with four places both are free, with three
          // the second half waits for the first half's products of the tile before, with two either
          // half for its own.
          auto place_free = [&](int u) {
            if (g > 0 && kPlaces - u < 3) wait_bar(kPlaces == 2 && u == 1 ? pv_done : pv_half, (g - 1) & 1, prm.err);
            tc_fence_after();
          };
          const uint32_t v_at[2] = {t_lane + kTmemV + place * 32,
                                    t_lane + kTmemV + (place + 1 == kPlaces ? 0 : place + 1) * 32};
          place = (place + 2) % kPlaces;
          // ---- V into the operand columns
          if (cached) {
            uint2 v[4];
            // quad lane % 4 expands blocks 2 (lane % 4) and + 1, channels lane / 4 + 8 j of the warp's 32
            const uint32_t src = tile + 2 * (lane & 3) * kBlockStride + kOffV + (wq * 32 + (lane >> 2)) * 8;
#pragma unroll
            for (int uh = 0; uh < 4; ++uh) {
              const int h = uh & 1;
              if (h == 0) {
                place_free(uh >> 1);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = ld_shared_v2(src + (uh >> 1) * kBlockStride + j * 64);
              }
              const uint32_t at = vs + uh * 128 + (lane & 3) * 32;
              const uint4 s = ld_shared_v4(at), c = ld_shared_v4(at + 16);
#pragma unroll
              for (int f = 0; f < 2; ++f) {  // lanes 0-15 and 16-31 of the quadrant
                uint32_t lo[4], hi[4];
                expand(h ? v[2 * f].y : v[2 * f].x, magic, s.x, c.x, s.y, c.y, s.z, c.z, s.w, c.w, lo);
                expand(h ? v[2 * f + 1].y : v[2 * f + 1].x, magic, s.x, c.x, s.y, c.y, s.z, c.z, s.w, c.w, hi);
                const uint32_t o[8] = {lo[0], lo[1], hi[0], hi[1], lo[2], lo[3], hi[2], hi[3]};
                tmem_st_16x256b_x2(v_at[uh >> 1] + (static_cast<uint32_t>(f * 16) << 16) + h * 16, o);
              }
            }
          } else {
            const long long step = (long long)prm.Hkv * kD;
            const __nv_bfloat16* vn =
                prm.v_new + ((long long)(item.c0 + (t - ct) * kKT) * prm.Hkv + item.kvh) * kD + kl;
            uint32_t nan = 0;
            place_free(0);
            place_free(1);
#pragma unroll 1
            for (int i = 0; 32 * i < vis; ++i) {
              uint32_t o[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const int k = 32 * i + 2 * j;
                // (past the last row that row again: loads in a batch, no branches)
                float x = __bfloat162float(vn[min(k, vis - 1) * step]) * prm.v_unit;
                float y = __bfloat162float(vn[min(k + 1, vis - 1) * step]) * prm.v_unit;
                if (k >= vis) x = 0.f;
                if (k + 1 >= vis) y = 0.f;
                o[j] = pack16_value(x, y, nan);
              }
              tmem_st16u((i < 2 ? v_at[0] : v_at[1]) + (i & 1) * 16, o);
            }
            if (has_nan(nan)) S.nan[wq] = 1;
          }
        } else if (t + 1 < item.te) {
          wait_bar(qk_done, g & 1, prm.err);  // K's columns are free
          tc_fence_after();
          expand_k(t + 1);
        }
        wait_bar(qk_done, g & 1, prm.err);
        if (g > 0) wait_bar(pv_done, (g - 1) & 1, prm.err);  // P is free
        tc_fence_after();
        // ---- softmax of rows half NH .. + NH - 1: row n sees this key iff n >= nmin
        const bool masked = !cached || vis < kKT;
        int nmin = 0;
        if (masked) nmin = (kl >= vis ? 1 << 30 : cached ? 0 : ((t - ct) * kKT + kl - item.i0) * G) - half * NH;
        // this key's step of the PV product: that of V's expansion in a cache tile
        const int pr = cached ? 16 * (lane >> 2) + 4 * wq + (lane & 3) : kl;
        const int nc8 = ceil_div(min(nq - half * NH, NH), 8);  // 8-row pieces that hold rows (may be < 0)
        float s[NH];
        auto scores = [&]() {
#pragma unroll
          for (int q = 0; q < NH / 8; ++q)
            tmem_ld8(t_lane + kTmemS + half * NH + q * 8, *reinterpret_cast<float(*)[8]>(&s[q * 8]));
          tmem_wait_ld();
#pragma unroll
          for (int q = 0; q < NH / 8; ++q)  // (not read before the wait)
            asm volatile("" : "+f"(s[q * 8]), "+f"(s[q * 8 + 1]), "+f"(s[q * 8 + 2]), "+f"(s[q * 8 + 3]),
                              "+f"(s[q * 8 + 4]), "+f"(s[q * 8 + 5]), "+f"(s[q * 8 + 6]), "+f"(s[q * 8 + 7]));
          if (masked) {
#pragma unroll
            for (int k = 0; k < NH; ++k) s[k] = nmin <= k ? s[k] : -INFINITY;
          }
        };
        bool move = t == item.tb;  // the references have to move first
#pragma unroll 1
        for (;;) {
          scores();
          if (move) {
            // ---- the tile's maximum per row, over the four warps of the half
#pragma unroll
            for (int q = 0; q < NH / 8; ++q) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = s[q * 8 + k] * cf[q * 8 + k];
              const float m = reduce8<true>(v, lane);
              if (lane < 8) S.red[w][q * 8 + lane] = m;
            }
            team_sync();
            for (int k = lane; k < NH; k += 32) {
              const float tm = fmaxf(fmaxf(S.red[4 * half][k], S.red[4 * half + 1][k]),
                                     fmaxf(S.red[4 * half + 2][k], S.red[4 * half + 3][k]));
              const float old = -ref[k];
              float al = 1.f;
              if (tm - kRefDrop > old + (kMove - kRefDrop)) {
                al = old == kNoRef ? 0.f : fast_exp2(old - (tm - kRefDrop));
                ref[k] = -(tm - kRefDrop);
              }
              alpha[k] = al;
            }
            __syncwarp();
            if (t > item.tb) {  // (the products of the tiles before are done)
#pragma unroll 1
              for (int q = 0; q < NH / 8; ++q) {
                float o[8];
                tmem_ld8(t_lane + kTmemO + half * NH + q * 8, o);
                tmem_wait_ld8(o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= alpha[q * 8 + k];
                tmem_st8(t_lane + kTmemO + half * NH + q * 8, o);
              }
#pragma unroll
              for (int k = 0; k < NH; ++k) lacc[k] *= alpha[k];
            }
          }
          // ---- P of this key against the references
          float top = -INFINITY;
#pragma unroll
          for (int q = 0; q < NH / 8; ++q) {
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
            const int chunk = half * (NH / 8) + q;
            st_shared_v4(smem_addr(S.p) + (chunk >> 2) * WideSmem<N>::kPBlock + sw64_off(pr, chunk & 3),
                         make_uint4(pk[0], pk[1], pk[2], pk[3]));
          }
          fence_proxy_async_smem();
          tmem_wait_st();
          tc_fence_before();
          // P and V are whole when the team passes; a key far above its row's reference sends the
          // tile through once more, after the references have moved
          const bool again = team_or(top > kMove);
          if (!again || move) break;
          move = true;
        }
        hand_over();
        if (cached) {
          if (++stage == kStages) stage = 0;
        }
#pragma unroll
        for (int q = 0; q < NH / 8; ++q) {
          if (q >= nc8) break;
#pragma unroll
          for (int k = q * 8; k < q * 8 + 8; k += 2)
            unpack(add2(f2(lacc[k], lacc[k + 1]), f2(s[k], s[k + 1])), lacc[k], lacc[k + 1]);
        }
      }

      if (it + 1 < own.n) load_q(fetch_item(S.items, own.more, it + 1));
      // ---- epilogue: row sums over the half's warps, O^T / l; thread = channel
#pragma unroll
      for (int q = 0; q < NH / 8; ++q) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = lacc[q * 8 + k];
        const float l = reduce8<false>(v, lane);
        if (lane < 8) S.red[w][q * 8 + lane] = l;
      }
      team_sync();
      const bool split = item.nsplit > 1;
      const int n_half = min(nq - half * NH, NH);  // rows of this half (may be < 0)
      for (int k = lane; k < NH; k += 32) {
        const float l = (S.red[4 * half][k] + S.red[4 * half + 1][k]) +
                        (S.red[4 * half + 2][k] + S.red[4 * half + 3][k]);
        alpha[k] = l == 0.f ? 0.f : prm.o_unit / l;
        if (wq == 0 && k < n_half) {
          const int n = half * NH + k;
          const float v = l == 0.f ? -INFINITY : (log2f(l) - ref[k]) * 0.69314718055994530942f;
          if (split)
            prm.ws_lse[(long long)item.slot * prm.slot_rows + n] = v;
          else
            prm.lse[(row0 + ((n * G_inv) >> 16)) * prm.Hq + item.kvh * G + n - ((n * G_inv) >> 16) * G] = v;
        }
      }
      __syncwarp();
      wait_bar(pv_done, (g - 1) & 1, prm.err);
      tc_fence_after();
      float* dst_ws = prm.ws_o + ((long long)item.slot * prm.slot_rows + half * NH) * kD + kl;
      int h = half * NH - ((half * NH * G_inv) >> 16) * G;   // head of the group
      __nv_bfloat16* dst = prm.out + ((row0 + ((half * NH * G_inv) >> 16)) * prm.Hq + item.kvh * G + h) * kD + kl;
      const long long next = (long long)(prm.Hq - G) * kD;   // to the next block row's heads
#pragma unroll 1
      for (int q = 0; q * 8 < n_half; ++q) {
        float o[8];
        tmem_ld8(t_lane + kTmemO + half * NH + q * 8, o);
        tmem_wait_ld8(o);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float y = o[k] * alpha[q * 8 + k];
          if (q * 8 + k < n_half) {
            if (split)
              dst_ws[(q * 8 + k) * kD] = y;
            else
              *dst = __float2bfloat16(y);
          }
          dst += kD;
          if (++h == G) {
            h = 0;
            dst += next;
          }
        }
      }
      if (S.nan[wq]) write_nans(prm, item, kl, half * NH, half * NH + n_half);
      // (the next item's Q, cf and references are written behind this barrier's and the products'
      // last reads; `red` next after its first tile's barrier)
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (w == 0) tmem_dealloc(tmem, kTmemCols);
}

template <int N>
static int run(const Params& p, int ncta, cudaStream_t stream) {
  static PerDevice<bool> done;
  constexpr int bytes = (int)sizeof(WideSmem<N>) + 1024;
  static_assert(kWideCtasPerSm * (bytes + 1024) <= 228 * 1024, "shared memory of an SM");
  if (!once_per_device(done, false, [] {
        return cudaFuncSetAttribute(verify_attn_kv4_wide_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    bytes) == cudaSuccess;
      }))
    return DSPARK_ECUDA;
  return launch_pdl(verify_attn_kv4_wide_kernel<N>, dim3(ncta), dim3(kThreads), bytes, stream, p) == cudaSuccess
             ? DSPARK_OK : DSPARK_ECUDA;
}
int launch_wide(const Params& p, int n, int ncta, cudaStream_t stream) {
  return n == 32 ? run<32>(p, ncta, stream) : n == 48 ? run<48>(p, ncta, stream) : run<64>(p, ncta, stream);
}

}  // namespace kv4a
}  // namespace attn
}  // namespace dspark
