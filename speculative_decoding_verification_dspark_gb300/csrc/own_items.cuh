// Work items of the attention kernels whose CTAs find their own shares.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"

namespace dspark {
namespace attn {

constexpr int kKT = 128;               // keys of a tile
constexpr int kSmemItems = 16;         // work items of a CTA kept in shared memory
// Largest context and segment together.  Each fills tiles of its own, and the lanes of a copying
// warp form positions up to 31 blocks past the start of the last tile, 622 past this end at most.
constexpr long long kMaxEnd = 0x7fffffffll - 6 * kKT;
constexpr int kMaxCtas = 1024;         // (own_items: products of a unit and a CTA in 32 bits)

// ---------------------------------------------------------------- work items
// The key tiles of every (request, row tile, KV head) group are laid end to end (U units) and
// CTA c of n takes units [c U / n, (c + 1) U / n), the same number for each, as the
// causal bf16 kernels do with a list that a kernel of one CTA builds; here each CTA finds its own
// items, which costs it 2 to 3 us in place of that kernel's 5 to 14 (its time grows with the
// groups) and one launch.  A group cut by CTA boundaries becomes pieces, at most max_splits; a
// piece is the first or the last of its CTA and goes to slot 2 c or 2 c + 1; the CTA of a group's
// last piece records the group for the merge.
struct OwnItems {
  int n;                  // items of this CTA
  const AttnItem* more;   // all of them, if n > SMEM_ITEMS
};
struct ItemScratch {
  long long off[DSPARK_MAX_B + 1];  // first unit of request r
  int goff[DSPARK_MAX_B + 1];       // first group
  int tt[DSPARK_MAX_B];             // tiles of a group
  long long w_units[32];
  int w_groups[32], w_tmax[32];
};

// Largest r in [a, b) with off[r] <= x (off non-decreasing, off[a] <= x).
template <typename T>
__device__ __forceinline__ int last_le(const T* off, int a, int b, T x) {
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (off[mid] <= x) a = mid; else b = mid;
  }
  return a;
}

// By the whole CTA of THREADS; ends with a barrier behind which the scratch is free.
// Params has B, max_rows, rows_per_tile, max_splits, Hkv, cu_seqlens, ctx_len, items, groups, err.
template <int THREADS, int SMEM_ITEMS = kSmemItems, class Params>
__device__ __forceinline__ OwnItems own_items(const Params& p, ItemScratch& S, AttnItem* s_items) {
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, c = blockIdx.x;
  const int B = p.B, rpt = p.rows_per_tile;
  // (with the last row no less than 0, as here, and the others no less than 0, as below, n does not
  // pass 32 bits)
  const bool rows_ok = (unsigned)p.cu_seqlens[B] <= (unsigned)p.max_rows;
  // this thread's requests
  const int per = (B + THREADS - 1) / THREADS, r_begin = tid * per, r_end = min(B, r_begin + per);
  long long units = 0;
  int groups = 0, tmax = 0;
  // a length or a first row below zero, or a segment whose end lies past kMaxEnd: no shares can be
  // made of it
  bool bad = false;
  for (int r = r_begin; r < r_end; ++r) {
    const int c0 = p.cu_seqlens[r], n = p.cu_seqlens[r + 1] - c0, ctx = p.ctx_len[r];
    bad |= c0 < 0 || n < 0 || ctx < 0 || (long long)ctx + n > kMaxEnd;
    const int t = ceil_div(ctx, kKT) + ceil_div(n, kKT), ng = ceil_div(n, rpt) * p.Hkv;
    S.tt[r] = t;
    S.goff[r] = ng;
    units += (long long)t * ng;
    groups += ng;
    if (ng > 0) tmax = max(tmax, t);
  }
  long long u_incl = units;
  int g_incl = groups;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, u_incl, o);
    const int g = __shfl_up_sync(0xffffffffu, g_incl, o);
    if (lane >= o) {
      u_incl += u;
      g_incl += g;
    }
    tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, o));
  }
  if (lane == 31) {
    S.w_units[wid] = u_incl;
    S.w_groups[wid] = g_incl;
    S.w_tmax[wid] = tmax;
  }
  bad = __syncthreads_or(bad);
  long long U = 0, u0 = u_incl - units;
  int g0 = g_incl - groups;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < wid) {
      u0 += S.w_units[i];
      g0 += S.w_groups[i];
    }
    U += S.w_units[i];
    tmax = max(tmax, S.w_tmax[i]);
  }
  for (int r = r_begin; r < r_end; ++r) {
    const int ng = S.goff[r];
    S.off[r] = u0;
    S.goff[r] = g0;
    u0 += (long long)S.tt[r] * ng;
    g0 += ng;
  }
  __syncthreads();
  // No group in more than max_splits pieces: every range holds L = floor(U / n) units, and a group
  // of T meets at most ceil((T - 1) / L) + 1 ranges, so L >= ceil((T - 1) / (max_splits - 1)).
  const bool small = U < (1 << 20);  // (with 1024 CTAs all products fit 32 bits)
  const unsigned l_req = max(1u, (unsigned)(tmax - 1 + p.max_splits - 2) / (unsigned)(p.max_splits - 1));
  long long n_max = small ? (unsigned)U / l_req : U / l_req;
  const int n_cta = (int)max(1ll, min(n_max, (long long)gridDim.x));
  auto first_unit = [&](int cc) -> long long {
    return small ? (unsigned)cc * (unsigned)U / (unsigned)n_cta : (long long)cc * U / n_cta;
  };
  OwnItems own{0, nullptr};
  const bool active = rows_ok && !bad && U > 0 && c < n_cta;
  if (c == 0 && tid == 0 && !rows_ok) raise_error(p.err, DSPARK_DEVERR_ROWS_OVERFLOW);
  if (c == 0 && tid == 0 && bad) raise_error(p.err, DSPARK_DEVERR_BAD_INPUT);
  SplitGroup record{};
  if (active) {
    const long long lo = first_unit(c), hi = first_unit(c + 1);
    const int r0 = last_le(S.off, 0, B, lo), r1 = last_le(S.off, r0, B, hi - 1);
    const long long d0 = lo - S.off[r0], d1 = hi - 1 - S.off[r1];
    const int gf = S.goff[r0] + (int)(small ? (unsigned)d0 / (unsigned)S.tt[r0] : d0 / S.tt[r0]);
    const int gl = S.goff[r1] + (int)(small ? (unsigned)d1 / (unsigned)S.tt[r1] : d1 / S.tt[r1]);
    // the CTA of unit x: the largest cc with cc U / n_cta <= x
    auto cta_of = [&](long long x) -> int {
      return small ? (int)(((unsigned)(x + 1) * (unsigned)n_cta - 1) / (unsigned)U)
                   : (int)(((x + 1) * n_cta - 1) / U);
    };
    own.n = gl - gf + 1;
    // (items of earlier CTAs number gf + c at most)
    AttnItem* const list = p.items + gf + c;
    own.more = list;
    for (int i = tid; i < own.n; i += THREADS) {
      const int g = gf + i, r = last_le(S.goff, r0, r1 + 1, g);
      const int lg = g - S.goff[r], t = lg / p.Hkv, t_r = S.tt[r];
      const long long gs = S.off[r] + (long long)lg * t_r, ge = gs + t_r;
      const long long a = max(gs, lo), b = min(ge, hi);
      const int c_first = gs < lo ? cta_of(gs) : c, c_last = ge > hi ? cta_of(ge - 1) : c;
      AttnItem x;
      x.c0 = p.cu_seqlens[r];
      x.n_r = p.cu_seqlens[r + 1] - x.c0;
      x.ctx = p.ctx_len[r];
      x.r = r; x.kvh = lg - t * p.Hkv; x.i0 = t * rpt; x.ni = min(rpt, x.n_r - x.i0);
      x.part = 0; x.split = c - c_first;
      x.tb = (int)(a - gs); x.te = (int)(b - gs);
      x.nsplit = c_last - c_first + 1;
      x.slot = a == lo ? 2 * c : 2 * c + 1;
      x.pad0 = x.pad1 = x.pad2 = 0;
      if (i < SMEM_ITEMS) s_items[i] = x;
      if (own.n > SMEM_ITEMS) list[i] = x;
      if (i == 0 && gs < lo && ge <= hi) {  // a split group that ends here
        record.r = r; record.kvh = x.kvh; record.part = 0; record.i0 = x.i0;
        record.ni = x.ni; record.c_first = c_first; record.nsplit = x.nsplit;
        record.slot0_last = gs != first_unit(c_first);
      }
    }
  }
  if (tid == 0) p.groups[c] = record;  // (nsplit 0: none)
  ptx::fence_proxy_async_smem();  // (bulk copies land where the scratch is)
  __syncthreads();
  return own;
}

__device__ __forceinline__ AttnItem fetch_item(const AttnItem* s_items, const AttnItem* more, int it) {
  return it < kSmemItems ? s_items[it] : more[it];
}

}  // namespace attn
}  // namespace dspark
