// Varlen verify attention over a 4-bit paged KV cache (layout: kv4.cuh), GQA head dim 128.
//
// For packed row cu_seqlens[r] + i and query head h of KV group kvh:
//   o = softmax(scale q.K^T) V over the ctx_len[r] committed keys, whose K and V are
//   (code - 8) * scale * g, followed by block rows 0..i (bf16); lse = log-sum-exp.
//
// Two kernels by the rows of a query tile (G heads x block rows): this one for up to 16, the
// wide one (verify_attn_kv4_wide.cu) for up to 64.  Here a tile's 8 NT rows (NT = 1, 2) meet
// tiles of 128 keys on a team of four warps, with a fifth that copies, a CTA of its own,
// several to an SM, persistent over an equal share of the key tiles (own_items).  Both
// products have the cache on the MMA's M side:
//   S^T [128 keys x 8 NT] = K . Q^T     warp w: keys 32 w .. + 31 (two blocks of the cache)
//   O^T [128 d    x 8 NT] += V^T . P^T  warp w: channels 32 w .. + 31 (one group of V scales)
// so that warp w expands its keys of K and its channels of V and every code once, and the
// left operand goes from the codes in a thread's registers straight into its fragment:
// the product's inner index may run in any order, and here it runs in the order in which a
// thread's 16-byte loads hold it (dims of K: thread t of a quad has group t; keys of V: it
// has block t of each 64 keys), the same order being given to Q and P in shared memory.
//
// Why fragments in registers (mma.sync) for few rows: with tcgen05 the expanded operand goes
// through tensor memory and the team waits for the products; with mma.sync nothing waits but
// at one barrier per tile, a tile of 8 rows being 730 instructions on each scheduler (K 210,
// V 250).  But m16n8k16
// takes 2.05 cycles of an SM (measured) and other instructions hardly issue beside it, so
// each 8 rows more add 260 cycles to a tile for which HBM needs 850.  Measured, this kernel
// against the wide one: 256 decodes of 5 heads 181 : 293 us, 64 x 3 and 4 rows of 4 heads at
// 2048 tokens 58 : 73; with tiles of 24 rows 71 : 62 (32 short windows) and 32 rows 194 : 155
// (131k contexts).
//
// Bound by instruction issue (0.63 per cycle and scheduler, which 18 warps per SM cannot
// raise): 256 decodes read 646 MB in 170 us, 3.8 TB/s.  The copies alone (same blocks, same
// ring) take 96 us.
//
#include "kv4_attn.cuh"

namespace dspark {
namespace attn {
namespace kv4a {

constexpr int kTeam = 128;             // four warps that compute; a fifth copies
constexpr int kThreads = 160;
constexpr int kStages = 2;             // cache tiles in a CTA's ring
// CTAs per SM for a tile of this many rows, by registers (the fragments of O^T and S^T are one
// per row); for more than 16 rows those of the wide kernel.
__host__ __device__ constexpr int ctas_per_sm(int rows) {
  return rows <= 8 ? 4 : rows <= 16 ? 3 : kWideCtasPerSm;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
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
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// Barrier of the team, and the same that ors a flag over it.
__device__ __forceinline__ void team_sync() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kTeam) : "memory");
}
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
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D += A B, m16n8k16, fp16 with fp32 accumulators.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Chunk j (8 query rows, 16 bytes) of row r of P in shared memory, placed so that neither the
// eight rows of a fragment nor the rows {0, 1, 8, 9, 16, 17, 24, 25} + x that a warp writes at
// once share banks: by padding after each eight rows and, with two chunks, by the chunk's place.
template <int NT>
__device__ __forceinline__ uint32_t p_off(int r, int j) {
  static_assert(NT == 1 || NT == 2, "tiles of 8 or 16 rows");
  if (NT == 1) return r * 16 + (r >> 3) * 32;
  return r * 32 + (r >> 3) * 64 + ((j ^ (((r >> 2) ^ (r >> 4)) & 1)) << 4);
}
template <int NT>
constexpr int p_bytes() { return kKT * 16 * NT + 16 * (NT == 1 ? 32 : 64); }
// Row of Q (256 bytes, 16 chunks).
__device__ __forceinline__ uint32_t q_off(int row, int c) { return row * 256 + ((c ^ (row & 7)) << 4); }

template <int NT>
struct Smem {
  __align__(128) uint8_t q[8 * NT * 256];
  __align__(128) uint8_t p[2][p_bytes<NT>()];
  __align__(128) uint8_t ring[kStages][kStageBytes];
  float cf[8 * NT];          // softmax scale per row
  float ref[4][8 * NT];      // references, a copy per warp
  float red[4][8 * NT];      // maxima of a tile per warp
  float sum[4][8 * NT];      // row sums of an item per warp
  int nan[4];                // a warp met a NaN among the item's values
  __align__(16) AttnItem items[kSmemItems];
  __align__(8) uint64_t full[kStages], empty[kStages];
};

// The copying warp: the cache tiles of the CTA in order into the ring.  Lane j knows block
// j % 8 of tile j / 8 of a window of four tiles; the pages of a window are read while the
// window before it is copied, so that nothing waits for the page table.
template <int ST>
__device__ __forceinline__ void copy_tiles(const Params& p, const AttnItem* s_items, const OwnItems& own,
                                           uint32_t ring, uint32_t full, uint32_t empty) {
  const int lane = threadIdx.x & 31;
  int stage = 0, parity = 1, page = -1;
  bool holds = false;
  // whether this lane's block in the window at tile t0 holds a committed key of the item's tiles, and
  // its page (not looked at before the window is copied: nothing waits for the read here)
  auto look = [&](const AttnItem& x, int t0) {
    const int pos = t0 * kKT + lane * kBlock, slot = pos >> p.log2_page;
    holds = pos < x.ctx && t0 + (lane >> 3) < x.te;
    page = holds && slot < p.max_pages ? __ldg(p.page_table + (long long)x.r * p.max_pages + slot) : -1;
  };
  AttnItem x = s_items[0];
  look(x, x.tb);
  const int lp = p.log2_page - 4;
  bool fresh = true;  // the first pass over the ring finds it empty
  for (int it = 0; it < own.n; ++it) {
    AttnItem next = x;
    if (it + 1 < own.n) next = fetch_item(s_items, own.more, it + 1);
    const int te = min(x.te, ceil_div(x.ctx, kKT));
    for (int t0 = x.tb; t0 < x.te; t0 += 4) {
      int block = -1;
      if ((unsigned)page < (unsigned)p.n_pages)
        block = ((page * p.Hkv + x.kvh) << lp) + (((t0 * kKT + lane * kBlock) >> 4) & ((1 << lp) - 1));
      else if (holds)
        raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
      if (t0 + 4 < x.te) look(x, t0 + 4); else look(next, next.tb);
      const uint8_t* src = p.cache + (long long)(block < 0 ? 0 : block) * kBlockBytes;
      const unsigned have = __ballot_sync(0xffffffffu, block >= 0);
      for (int i = 0; i < 4 && t0 + i < te; ++i) {
        if (!fresh) wait_bar(empty + 8 * stage, parity, p.err);
        const uint32_t bar = full + 8 * stage;
        if (lane == 0)
          ptx::mbar_arrive_expect_tx(bar, __popc(have >> (8 * i) & 0xffu) * kBlockBytes);
        __syncwarp();
        if ((lane >> 3) == i && block >= 0)
          ptx::bulk_load_g2s(ring + stage * kStageBytes + (lane & 7) * kBlockStride, src, kBlockBytes, bar);
        if (++stage == ST) {
          stage = 0;
          parity ^= 1;
          fresh = false;
        }
      }
    }
    x = next;
  }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(8 * NT)) verify_attn_kv4_kernel(const Params prm) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<NT>& S = *reinterpret_cast<Smem<NT>*>(smem_raw);
  constexpr int ST = kStages;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  // (no early release: what follows would take the first SMs that fall free, and the next call's
  // persistent CTAs come to lie unevenly: 256 decodes 197 us one call after another, 170 without)
  pdl_wait();  // the step's inputs come from earlier kernels
  const uint32_t ring = smem_u32(S.ring), full = smem_u32(S.full), empty = smem_u32(S.empty);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(full + 8 * i, 1);
      ptx::mbar_init(empty + 8 * i, 4);
    }
    ptx::fence_mbar_init();
    for (int i = 0; i < 4; ++i) S.nan[i] = 0;
  }
  static_assert(sizeof(ItemScratch) <= sizeof(S.ring), "the scratch lies in the ring");
  const OwnItems own = own_items<kThreads>(prm, *reinterpret_cast<ItemScratch*>(S.ring), S.items);
  if (own.n == 0) return;
  if (w == kTeam / 32) {
    copy_tiles<ST>(prm, S.items, own, ring, full, empty);
    return;
  }

  const int G = prm.Hq / prm.Hkv;
  uint32_t magic;  // 1024 twice; opaque, so that it stays in a register
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
  const uint32_t sq = smem_u32(S.q), sp = smem_u32(S.p);
  // Key 16 b + tok of a tile is inner index 64 (b >> 2) + 16 (tok >> 2) + 8 ((tok >> 1) & 1) +
  // 2 (b & 3) + (tok & 1) of the PV product, the order of V's fragments: this thread's first
  // key (b = 2 w, tok = g); block 2 w + i is 2 i further, tok + 8 another 32
  const int p_row = 64 * (w >> 1) + 16 * (g >> 2) + 8 * ((g >> 1) & 1) + 4 * (w & 1) + (g & 1);
  int stage = 0, parity = 0;   // of the next cache tile

  // ---- Q: tile row n = (block row n / G, head kvh G + n % G), a half-warp holds a row, 8 dims per
  // lane; read in the last tile of the item before
  uint4 qv[NT];
  auto load_q = [&](const AttnItem& x) {
    const long long row = (long long)x.c0 + x.i0;
    const int n_q = x.ni * G, h0 = x.kvh * G;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int n = 8 * i + 2 * w + (lane >> 4);
      qv[i] = make_uint4(0, 0, 0, 0);
      if (n < n_q)
        qv[i] = *reinterpret_cast<const uint4*>(
            prm.q + ((row + n / G) * prm.Hq + h0 + n % G) * kD + (lane & 15) * 8);
    }
  };
  load_q(S.items[0]);

  for (int it = 0; it < own.n; ++it) {
    const AttnItem item = fetch_item(S.items, own.more, it);
    const int ctx = item.ctx, ct = ceil_div(ctx, kKT);
    const int nq = item.ni * G;              // rows of the tile
    const long long row0 = (long long)item.c0 + item.i0;
    // ---- Q as fp16 scaled by a power of two, in the order of K's fragments: dim 32 t + 8 v + e
    // (word v of group t) is at inner index 16 s + 2 t + (e & 1) + 8 ((e >> 1) & 1), s = 2 c + (e >> 2),
    // where thread t of a quad takes word v in turn c, its pairs of words swapped for odd t
    {
      const int l = lane & 15;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int n = 8 * i + 2 * w + (lane >> 4);
        const uint32_t x[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
        uint32_t top = 0;  // largest magnitude, as bits (a NaN is above all)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max((x[j] << 16) & 0x7fffffffu, x[j] & 0x7fff0000u));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // the largest element's power of two, no smaller than 2^-100 (fp32 holds 2^114)
        const int e = max((int)(top >> 23), 27);
        const float f = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // dims 8 l + 2 j, + 1
          const int t = l >> 2, c = 2 * ((((l & 3) >> 1) + t) & 1) + (l & 1), s = 2 * c + (j >> 1);
          const int at = 16 * s + 2 * t + 8 * (j & 1);
          st_shared(sq + q_off(n, at >> 3) + (at & 7) * 2,
                    h2_bits(__floats2half2_rn(bf_lo(x[j]) * f, bf_hi(x[j]) * f)));
        }
        if (l == 0)  // (never 0: a masked score is -inf times it)
          S.cf[n] = fmaxf(__uint_as_float((uint32_t)(e - 14) << 23) * prm.sl2, 1.17549435e-38f);
      }
    }
    team_sync();
    // this thread's rows: 8 j + 2 t4 + {0, 1}
    float l[NT][2];
    float o[2][NT][4];      // O^T: channels 32 w + 16 i + 2 g + {0, 1} x rows
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      l[j][0] = l[j][1] = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[0][j][e] = o[1][j][e] = 0.f;
    }
    float* const my_ref = S.ref[w];
    if (lane < 8 * NT) my_ref[lane] = kNoRef;

#pragma unroll 1
    for (int t = item.tb; t < item.te; ++t) {
      const bool cached = t < ct;
      const int vis = cached ? min(ctx - t * kKT, kKT) : min(item.n_r - (t - ct) * kKT, kKT);
      const uint32_t pbuf = sp + ((t - item.tb) & 1) * p_bytes<NT>();
      const uint32_t tile = ring + stage * kStageBytes;
      if (t == item.te - 1 && it + 1 < own.n) load_q(fetch_item(S.items, own.more, it + 1));
      if (cached) wait_bar(full + 8 * stage, parity, prm.err);
      // ---- S^T: two m-tiles of 16 keys
      float s[2][NT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) s[i][j][0] = s[i][j][1] = s[i][j][2] = s[i][j][3] = 0.f;
      // inner steps 2 c and 2 c + 1: Q's fragments, and the products with those of one m-tile from
      // the four pairs of row g's and row g + 8's word
      auto q_frags = [&](int c, uint32_t (&b)[NT][4]) {
#pragma unroll
        for (int j = 0; j < NT; ++j) ldsm4(b[j], sq + q_off(8 * j + (lane & 7), 4 * c + (lane >> 3)));
      };
      auto qk = [&](float (&d)[NT][4], const uint32_t (&b)[NT][4], const uint32_t (&lo)[4],
                    const uint32_t (&hi)[4]) {
        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
        for (int j = 0; j < NT; ++j) mma(d[j], a0, b[j][0], b[j][1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma(d[j], a1, b[j][2], b[j][3]);
      };
      if (cached) {
        // per key (m-tile i, row g + 8 h at 2 i + h): its words in turn, pairs swapped for odd t4 so
        // that a half-warp's reads lie in different banks; its scale
        const uint32_t codes = tile + 2 * w * kBlockStride + t4 * 256 + g * 16;
        uint2 kc[4];
        uint32_t sl[4], sh[4], bl[4], bh[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t sc_at = tile + (2 * w + i) * kBlockStride + kOffKs + g * 4 + t4;
          const uint32_t two = e4m3_low(ld_shared_u8(sc_at) | (ld_shared_u8(sc_at + 32) << 8));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sc = __byte_perm(two, 0, h ? 0x3232 : 0x1010);
            sl[2 * i + h] = hmul2_bits(sc, kSixteenth);
            sh[2 * i + h] = hmul2_bits(sc, k256th);
            bl[2 * i + h] = hmul2_bits(sc, kBiasLow);
            bh[2 * i + h] = hmul2_bits(sc, kBiasHigh);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if ((c & 1) == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              kc[k] = ld_shared_v2(codes + (k >> 1) * kBlockStride + (k & 1) * 128 + (((c >> 1) + t4) & 1) * 8);
          }
          uint32_t b[NT][4];
          q_frags(c, b);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int k = 2 * i + h;
              const uint32_t word = c & 1 ? kc[k].y : kc[k].x;
              expand(word, magic, sl[k], bl[k], sh[k], bh[k], sl[k], bl[k], sh[k], bh[k], x[h]);
            }
            qk(s[i], b, x[0], x[1]);
          }
        }
      } else if (32 * w < vis) {
        // the request's own rows, bf16 / (16 k_scale)
        const uint4* src = reinterpret_cast<const uint4*>(
            prm.k_new + ((long long)(item.c0 + (t - ct) * kKT) * prm.Hkv + item.kvh) * kD + t4 * 32);
        const int row_vecs = prm.Hkv * kD / 8;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)  // (past the last row that row again: loads in a batch, no branches)
            v[k] = src[(long long)(min(32 * w + g + 8 * k, vis - 1) * row_vecs) + 2 * (((c >> 1) + t4) & 1) + (c & 1)];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (32 * w + g + 8 * k >= vis) v[k] = make_uint4(0, 0, 0, 0);
          uint32_t b[NT][4];
          q_frags(c, b);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 u = v[2 * i + h];
              const uint32_t y[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int q = 0; q < 4; ++q)
                x[h][q] = pack16(bf_lo(y[q]) * prm.k_unit, bf_hi(y[q]) * prm.k_unit);
            }
            qk(s[i], b, x[0], x[1]);
          }
        }
      }
      // ---- masks: s[i][j][2 h + e] is key 32 w + 16 i + g + 8 h, row 8 j + 2 t4 + e; a block
      // row b is seen by rows n >= (b - i0) G
      if (!cached || vis < kKT) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = 32 * w + 16 * i + g + 8 * h;
            const int nmin = k >= vis ? 1 << 30 : cached ? 0 : ((t - ct) * kKT + k - item.i0) * G;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (8 * j + 2 * t4 + e < nmin) s[i][j][2 * h + e] = -INFINITY;
          }
      }
      // ---- P against the references; a key far above its row's makes them move first
      bool move = t == item.tb;
#pragma unroll 1
      for (;;) {
        if (move) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = fmaxf(fmaxf(s[0][j][e], s[0][j][2 + e]), fmaxf(s[1][j][e], s[1][j][2 + e]));
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
              if (g == 0) S.red[w][8 * j + 2 * t4 + e] = m * S.cf[8 * j + 2 * t4 + e];
            }
          team_sync();
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int n = 8 * j + 2 * t4 + e;
              const float m = fmaxf(fmaxf(S.red[0][n], S.red[1][n]), fmaxf(S.red[2][n], S.red[3][n]));
              const float old = my_ref[n];
              __syncwarp();
              if (m - kRefDrop > old + (kMove - kRefDrop)) {
                const float al = old == kNoRef ? 0.f : fast_exp2(old - (m - kRefDrop));
                if (g == 0) my_ref[n] = m - kRefDrop;
                l[j][e] *= al;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  o[i][j][e] *= al;
                  o[i][j][2 + e] *= al;
                }
              }
            }
          __syncwarp();
        }
        float2 cf[NT], ref[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          cf[j] = *reinterpret_cast<const float2*>(&S.cf[8 * j + 2 * t4]);
          ref[j] = *reinterpret_cast<const float2*>(&my_ref[8 * j + 2 * t4]);
        }
        float top = -INFINITY;
        float p0[NT][2];    // this thread's part of the tile's row sums
#pragma unroll
        for (int j = 0; j < NT; ++j) p0[j][0] = p0[j][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = p_row + 2 * i + 32 * h;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const float x0 = fmaf(s[i][j][2 * h], cf[j].x, -ref[j].x);
              const float x1 = fmaf(s[i][j][2 * h + 1], cf[j].y, -ref[j].y);
              top = fmaxf(top, fmaxf(x0, x1));
              const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
              p0[j][0] += e0;
              p0[j][1] += e1;
              st_shared(pbuf + p_off<NT>(at, j) + t4 * 4, h2_bits(__floats2half2_rn(e0, e1)));
            }
          }
        // P is whole when the team passes
        const bool again = team_or(top > kMove);
        if (!again || move) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            l[j][0] += p0[j][0];
            l[j][1] += p0[j][1];
          }
          break;
        }
        move = true;
      }
      // ---- O^T: two m-tiles of 16 channels, rows g and g + 8 being channels 2 g and 2 g + 1;
      // inner steps 4 u + 2 h, + 1 from the four key pairs of either channel's word
      auto pv = [&](int u, int h, const uint32_t (&lo)[2][4], const uint32_t (&hi)[2][4]) {
        uint32_t b[NT][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) ldsm4_t(b[j], pbuf + p_off<NT>(64 * u + 32 * h + lane, j));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a0[4] = {lo[i][0], hi[i][0], lo[i][1], hi[i][1]};
          const uint32_t a1[4] = {lo[i][2], hi[i][2], lo[i][3], hi[i][3]};
#pragma unroll
          for (int j = 0; j < NT; ++j) mma(o[i][j], a0, b[j][0], b[j][1]);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma(o[i][j], a1, b[j][2], b[j][3]);
        }
      };
      if (cached) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {    // block t4 + 4 u
          const uint32_t blk = tile + (t4 + 4 * u) * kBlockStride;
          const uint4 vs4 = ld_shared16(blk + kOffVs + w * kBlock);
          uint32_t vsc[4] = {vs4.x, vs4.y, vs4.z, vs4.w};
          uint4 vc[2];                   // channels 2 g (x, y) and 2 g + 1 (z, w) of 16 i
#pragma unroll
          for (int i = 0; i < 2; ++i) vc[i] = ld_shared16(blk + kOffV + (32 * w + 16 * i + 2 * g) * 8);
          if (vis < kKT) {  // masked keys get scale 0, whatever their page holds
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int left = vis - (t4 + 4 * u) * kBlock - 4 * q;
              if (left < 4) vsc[q] = left <= 0 ? 0u : vsc[q] & ((1u << (8 * left)) - 1u);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 8 keys of it
            uint32_t ss[4], bb[4];       // scale pairs of the channels' group
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t x = vsc[2 * h + q];
              const uint32_t s0 = e4m3_low(x), s1 = e4m3_high(x);
              ss[2 * q] = hmul2_bits(s0, kSixteenth);
              bb[2 * q] = hmul2_bits(s0, kBiasLow);
              ss[2 * q + 1] = hmul2_bits(s1, k256th);
              bb[2 * q + 1] = hmul2_bits(s1, kBiasHigh);
            }
            uint32_t lo[2][4], hi[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              expand(h ? vc[i].y : vc[i].x, magic, ss[0], bb[0], ss[1], bb[1], ss[2], bb[2], ss[3], bb[3], lo[i]);
              expand(h ? vc[i].w : vc[i].z, magic, ss[0], bb[0], ss[1], bb[1], ss[2], bb[2], ss[3], bb[3], hi[i]);
            }
            pv(u, h, lo, hi);
          }
        }
      } else {
        const uint32_t* vn = reinterpret_cast<const uint32_t*>(
            prm.v_new + ((long long)(item.c0 + (t - ct) * kKT) * prm.Hkv + item.kvh) * kD) + 16 * w + g;
        const long long step = (long long)prm.Hkv * kD / 2;
        uint32_t nan = 0;
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
          if (64 * (n >> 1) + 8 * (n & 1) >= vis) continue;  // no key of it
          uint32_t lo[2][4], hi[2][4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int k = 16 * (t4 + 4 * (n >> 1)) + 8 * (n & 1) + 2 * p;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t y = vn[min(k, vis - 1) * step + 8 * i], z = vn[min(k + 1, vis - 1) * step + 8 * i];
              if (k >= vis) y = 0;
              if (k + 1 >= vis) z = 0;
              lo[i][p] = pack16_value(bf_lo(y) * prm.v_unit, bf_lo(z) * prm.v_unit, nan);
              hi[i][p] = pack16_value(bf_hi(y) * prm.v_unit, bf_hi(z) * prm.v_unit, nan);
            }
          }
          pv(n >> 1, n & 1, lo, hi);
        }
        if (has_nan(nan)) S.nan[w] = 1;
      }
      if (cached) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(empty + 8 * stage);
        if (++stage == ST) {
          stage = 0;
          parity ^= 1;
        }
      }
    }

    // ---- epilogue: row sums over the team, O^T / l
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], x);
        if (g == 0) S.sum[w][8 * j + 2 * t4 + e] = l[j][e];
      }
    team_sync();
    const bool split = item.nsplit > 1;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 8 * j + 2 * t4 + e;
        if (n >= nq) continue;
        const float sum = (S.sum[0][n] + S.sum[1][n]) + (S.sum[2][n] + S.sum[3][n]);
        const float inv = sum == 0.f ? 0.f : prm.o_unit / sum;
        const float lse = sum == 0.f ? -INFINITY : (my_ref[n] + log2f(sum)) * 0.69314718055994530942f;
        const long long at = (row0 + n / G) * prm.Hq + item.kvh * G + n % G;
        if (split) {
          if (w == 0 && g == 0) prm.ws_lse[(long long)item.slot * prm.slot_rows + n] = lse;
          float2* dst = reinterpret_cast<float2*>(prm.ws_o + ((long long)item.slot * prm.slot_rows + n) * kD + 32 * w) + g;
          dst[0] = make_float2(o[0][j][e] * inv, o[0][j][2 + e] * inv);
          dst[8] = make_float2(o[1][j][e] * inv, o[1][j][2 + e] * inv);
        } else {
          if (w == 0 && g == 0) prm.lse[at] = lse;
          __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(prm.out + at * kD + 32 * w) + g;
          dst[0] = __floats2bfloat162_rn(o[0][j][e] * inv, o[0][j][2 + e] * inv);
          dst[8] = __floats2bfloat162_rn(o[1][j][e] * inv, o[1][j][2 + e] * inv);
        }
      }
    __syncwarp();  // (behind the warp's outputs)
    const int nan = S.nan[w];
    __syncwarp();
    if (nan) {
      write_nans(prm, item, 32 * w + lane, 0, nq);
      if (lane == 0) S.nan[w] = 0;
    }
    // (the next item's barriers stand between these reads of shared memory and its writes: Q
    // and cf were last read before the team's last tile barrier, `sum` is written next after
    // two more)
  }
}

// ---------------------------------------------------------------- split combine
// Block (c, y): the split group recorded by CTA c, query rows 8y..8y+7, a warp per row:
//   lse = log sum_s e^{lse_s},  o = sum_s e^{lse_s - lse} o_s
__global__ void __launch_bounds__(256)
    combine_kv4_kernel(const int32_t* __restrict__ cu_seqlens, const SplitGroup* __restrict__ groups,
                       int G, int Hq, int slot_rows, const float* __restrict__ ws_o,
                       const float* __restrict__ ws_lse, __nv_bfloat16* __restrict__ out,
                       float* __restrict__ lse) {
  pdl_wait();  // inputs come from the kernels before this one
  const int lane = threadIdx.x & 31;
  const SplitGroup sg = groups[blockIdx.x];
  const int ns = sg.nsplit;
  const int n = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (ns <= 1 || n >= sg.ni * G) return;
  // piece s is in slot 2 (c_first + s), but for a first piece that is not its CTA's first
  auto slot = [&](int s) { return (long long)(2 * (sg.c_first + s) + (s == 0 && sg.slot0_last ? 1 : 0)) * slot_rows + n; };
  float mx = -INFINITY;
  for (int s = lane; s < ns; s += 32) mx = fmaxf(mx, ws_lse[slot(s)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < ns; s0 += 32) {
    const float wgt = s0 + lane < ns ? expf(ws_lse[slot(s0 + lane)] - mx) : 0.f;
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
  const float inv = 1.f / sum;
  const long long row = cu_seqlens[sg.r] + sg.i0 + n / G;
  const int head = sg.kvh * G + n % G;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 c = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(out + (row * Hq + head) * kD)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&c));
  if (lane == 0) lse[row * Hq + head] = mx + logf(sum);
}

// ---------------------------------------------------------------- host side
template <int NT>
static int launch_tile(const Params& p, int ncta, cudaStream_t stream) {
  static PerDevice<bool> done;
  const bool ok = once_per_device(done, false, [] {
    return cudaFuncSetAttribute(verify_attn_kv4_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(Smem<NT>)) == cudaSuccess;
  });
  if (!ok) return DSPARK_ECUDA;
  return launch_pdl(verify_attn_kv4_kernel<NT>, dim3(ncta), dim3(kThreads), sizeof(Smem<NT>), stream,
                    p) == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

Plan plan(int B, int max_rows, int Hq, int Hkv, int max_block_rows) {
  Plan p{};
  const int G = Hq / Hkv;
  const long long rows = (long long)G * (max_block_rows > 0 ? max_block_rows : 1);
  p.parts = 1;
  // (64 requests of 16 rows of 4 heads: one tile of 64 rows 117 us, two of 32 141; 12 rows: one of
  // 48 94 us, two of 24 137)
  p.nt = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
  p.rows_per_tile = p.nt / G;
  p.nk = kKT;
  p.d_part = kD;
  p.ncta = num_sms_cached() * ctas_per_sm(p.nt);
  if (p.ncta > kMaxCtas) p.ncta = kMaxCtas;
  p.max_items = (long long)Hkv * ((long long)max_rows / p.rows_per_tile + B) + p.ncta;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~size_t(255);
    return at;
  };
  p.off_items = take(sizeof(AttnItem) * (size_t)p.max_items);
  p.off_groups = take(sizeof(SplitGroup) * (size_t)p.ncta);
  p.off_o = take(sizeof(float) * (size_t)2 * p.ncta * p.nt * kD);  // slots 2c, 2c + 1
  p.off_lse = take(sizeof(float) * (size_t)2 * p.ncta * p.nt);
  p.bytes = off;
  return p;
}

int launch(const void* q, const void* k_new, const void* v_new, const void* cache, int n_pages,
           const int32_t* page_table, int max_pages, const int32_t* ctx_len,
           const int32_t* cu_seqlens, int B, int max_rows, int Hq, int Hkv, int page_size,
           float scale, float gk, float gv, int max_splits, void* out, float* lse, void* ws,
           const Plan& pl, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  Params p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.cache = static_cast<const uint8_t*>(cache);
  p.page_table = page_table;
  p.ctx_len = ctx_len;
  p.cu_seqlens = cu_seqlens;
  p.items = reinterpret_cast<AttnItem*>(w + pl.off_items);
  p.groups = reinterpret_cast<SplitGroup*>(w + pl.off_groups);
  p.B = B;
  p.max_rows = max_rows;
  p.rows_per_tile = pl.rows_per_tile;
  // a CTA of the bf16 kernels is an SM; here several share it, and a group may be cut finer
  p.max_splits = (max_splits < 2 ? 2 : max_splits) * ctas_per_sm(pl.nt);
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
  p.slot_rows = pl.nt;
  p.sl2 = score_factor(scale, gk);
  p.k_unit = 1.f / (16.f * gk);
  p.v_unit = 1.f / (16.f * gv);
  p.o_unit = 16.f * gv;
  const int lc = pl.nt == 8    ? launch_tile<1>(p, pl.ncta, stream)
                 : pl.nt == 16 ? launch_tile<2>(p, pl.ncta, stream)
                               : launch_wide(p, pl.nt, pl.ncta, stream);
  if (lc != DSPARK_OK) return lc;
  return launch_pdl(combine_kv4_kernel, dim3(pl.ncta, pl.nt / 8), dim3(256), 0, stream, cu_seqlens,
                    p.groups, Hq / Hkv, Hq, pl.nt, p.ws_o,
                    p.ws_lse, p.out, lse) == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

}  // namespace kv4a
}  // namespace attn
}  // namespace dspark
