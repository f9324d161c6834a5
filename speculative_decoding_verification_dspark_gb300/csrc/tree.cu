// Trees of drafted tokens: what a step needs before and after its forward pass.
//
// A request's packed rows are the nodes of a forest: row i of a segment has the parent
// row_parent (an index in the segment, less than i) or none (-1).  Row 0 is the anchor.
//   tree_pack     mask_i = bit i | mask of its parent (itself and its ancestors),
//                 pos_i  = ctx + the number of ancestors
//   accept_tree   from row 0 down: the lowest child whose token is the one sampled at its
//                 parent, until none has it; that sample is the bonus or correction token.  A row
//                 without a sample (negative) is not passed: nothing could follow it
// The walk keeps the target's distribution: every committed token is the target's own sample
// at its position.
//
// Both are bound by latency (24 bytes a row): one launch each, a CTA (a warp) per request, the
// parents in shared memory.

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

constexpr int kMaxTree = DSPARK_MAX_TREE;
constexpr int kPackThreads = 128;

// The segment of request r: [first, first + n), or n = -1 for one that no buffer holds.
struct Segment {
  int first, n;
};
__device__ __forceinline__ Segment segment(const int32_t* cu, int r, int max_rows) {
  const int a = cu[r], z = cu[r + 1];
  return {a, a < 0 || z < a || z > max_rows ? -1 : z - a};
}

// Each thread takes rows tid, tid + threads, ... and climbs.  Indices fall on the way up, so
// the mask comes out word by word from the row's own down to the first: one word in a register.
__global__ void __launch_bounds__(kPackThreads)
    tree_pack_kernel(const int32_t* __restrict__ parent, const int32_t* __restrict__ cu,
                     const int32_t* __restrict__ ctx_len, int B, int max_rows, int words,
                     uint64_t* __restrict__ mask, int32_t* __restrict__ pos,
                     unsigned int* __restrict__ err) {
  pdl_release();
  pdl_wait();
  __shared__ int16_t up[kMaxTree];
  const int r = blockIdx.x, tid = threadIdx.x;
  if (cu[B] > max_rows) {
    if (r == 0 && tid == 0) raise_error(err, DSPARK_DEVERR_ROWS_OVERFLOW);
    return;
  }
  const Segment s = segment(cu, r, max_rows);
  const int ctx = ctx_len[r];
  if (s.n < 0 || s.n > min(kMaxTree, 64 * words) || ctx < 0 || ctx > 0x7fffffff - kMaxTree) {
    if (tid == 0) raise_error(err, DSPARK_DEVERR_BAD_INPUT);
    return;
  }
  bool bad = false;
  for (int i = tid; i < s.n; i += kPackThreads) {
    int p = parent[s.first + i];
    if (p < -1 || p >= i) {
      bad = true;
      p = -1;
    }
    up[i] = static_cast<int16_t>(p);
  }
  if (bad) raise_error(err, DSPARK_DEVERR_BAD_INPUT);
  __syncthreads();
  for (int i = tid; i < s.n; i += kPackThreads) {
    uint64_t* m = mask + (long long)(s.first + i) * words;
    int depth = -1, at = i;
    for (int w = words - 1; w >= 0; --w) {
      uint64_t bits = 0;
      while (at >= 64 * w) {  // (at = -1 ends every word)
        bits |= 1ull << (at & 63);
        at = up[at];
        ++depth;
      }
      m[w] = bits;
    }
    pos[s.first + i] = ctx + depth;
  }
}

// One warp per request.  A child lies behind its parent, so the search for each goes on from
// where the last one ended: the walk passes the segment once.
__global__ void __launch_bounds__(32)
    accept_tree_kernel(const int32_t* __restrict__ row_tok, const int32_t* __restrict__ parent,
                       const int32_t* __restrict__ row_sample, const int32_t* __restrict__ cu, int B,
                       int gamma, int max_rows, int32_t* __restrict__ path,
                       int32_t* __restrict__ path_tok, int32_t* __restrict__ accept_len,
                       int32_t* __restrict__ out_tok, unsigned int* __restrict__ err) {
  pdl_release();
  pdl_wait();
  __shared__ int s_tok[kMaxTree], s_sample[kMaxTree];
  __shared__ int16_t s_up[kMaxTree];
  const int r = blockIdx.x, lane = threadIdx.x;
  if (cu[B] > max_rows) {
    if (r == 0 && lane == 0) raise_error(err, DSPARK_DEVERR_ROWS_OVERFLOW);
    return;
  }
  Segment s = segment(cu, r, max_rows);
  if (s.n < 0 || s.n > kMaxTree) {
    if (lane == 0) raise_error(err, DSPARK_DEVERR_BAD_INPUT);
    s.n = 0;
  }
  for (int i = lane; i < s.n; i += 32) {
    const int p = parent[s.first + i];
    s_up[i] = static_cast<int16_t>(p < -1 || p >= i ? -1 : p);
    s_tok[i] = row_tok[s.first + i];
    s_sample[i] = row_sample[s.first + i];
  }
  __syncwarp();
  int32_t* const p_out = path + (long long)r * (gamma + 1);
  int32_t* const t_out = path_tok + (long long)r * gamma;
  int len = 0, at = s.n > 0 && s_sample[0] >= 0 ? 0 : -1, say = -1;
  while (at >= 0) {
    if (lane == 0) {
      p_out[len] = at;
      if (len > 0) t_out[len - 1] = s_tok[at];
    }
    say = s_sample[at];
    const int from = at;
    at = -1;
    if (++len <= gamma) {
      for (int j0 = from + 1; j0 < s.n; j0 += 32) {
        const int j = j0 + lane;
        const unsigned hit =
            __ballot_sync(0xffffffffu, j < s.n && s_up[j] == from && s_tok[j] == say);
        if (hit) {
          at = j0 + __ffs(hit) - 1;
          if (s_sample[at] < 0) at = -1;
          break;
        }
      }
    }
  }
  for (int i = len + lane; i <= gamma; i += 32) p_out[i] = -1;
  for (int i = max(len - 1, 0) + lane; i < gamma; i += 32) t_out[i] = -1;
  if (lane == 0) {
    accept_len[r] = len - 1;
    out_tok[r] = say;
  }
}

}  // namespace

int launch_tree_pack(const int32_t* parent, const int32_t* cu, const int32_t* ctx_len, int B,
                     int max_rows, int words, uint64_t* mask, int32_t* pos, cudaStream_t stream) {
  return launch_pdl(tree_pack_kernel, dim3(B), dim3(kPackThreads), 0, stream, parent, cu, ctx_len,
                    B, max_rows, words, mask, pos, device_error_word()) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ECUDA;
}

int launch_accept_tree(const int32_t* row_tok, const int32_t* parent, const int32_t* row_sample,
                       const int32_t* cu, int B, int gamma, int max_rows, int32_t* path,
                       int32_t* path_tok, int32_t* accept_len, int32_t* out_tok,
                       cudaStream_t stream) {
  return launch_pdl(accept_tree_kernel, dim3(B), dim3(32), 0, stream, row_tok, parent, row_sample,
                    cu, B, gamma, max_rows, path, path_tok, accept_len, out_tok,
                    device_error_word()) == cudaSuccess
             ? DSPARK_OK
             : DSPARK_ECUDA;
}

}  // namespace dspark
