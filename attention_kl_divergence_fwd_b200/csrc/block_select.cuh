// block_select.cuh - the key blocks each query reads, from their masses.
//
// Of the n_vis blocks that hold an allowed key of the query: the first n_first, the last
// n_last, and then the heaviest of the rest until topk are taken; equal masses go to the lower
// index, NaN ranks below every number. Written in ascending order, -1 behind the last.
//
// A row's masses become unsigned keys in their order (forced blocks get the largest key) and
// stay in registers. The topk-th largest key is found bit by bit from the top: each step counts
// the keys that reach the candidate and stops early once exactly topk do. The selection is then
// written by ranks in index order, which gives the ascending list and the ties' order without
// a sort. One warp per row up to 1024 blocks, one CTA per row beyond. Bound by reading the
// masses for many rows, by latency for few.
#pragma once

#include "sparse_common.cuh"

namespace skl {

struct SelectArgs {
  const float* mass;  // [B, Hsel, N_Q, NB]
  const int* lens;
  int* idx;           // [B, Hsel, N_Q, topk]
  long long rows;     // B * Hsel * N_Q
  int Hsel, N_Q, N_K, NB, causal, topk, n_first, n_last;
};

// Order-preserving key of a mass: 0 is kept for blocks that cannot be taken, 0xffffffff for
// forced ones; -0 counts as 0 and NaN as the least.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = 0
  const uint32_t k = (u & 0x80000000u) ? ~u : u | 0x80000000u;  // -inf: 0x007fffff
  return k;                                                       // inf: 0xff800000
}

template <int WARPS>
__device__ __forceinline__ int select_sum(int x, int* red, int warp, int lane) {
  x = __reduce_add_sync(0xffffffffu, x);
  if (WARPS == 1) return x;
  if (lane == 0) red[warp] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int k = 0; k < WARPS; ++k) s += red[k];
  __syncthreads();
  return s;
}

// V keys per thread, WARPS warps per row (1: four rows per CTA). Thread t of a row holds the
// blocks (w * V + k) * 32 + lane for warp w, k < V: reads are coalesced and ranks in index
// order follow from ballots.
template <int V, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS)
streamkl_block_select_kernel(const SelectArgs a) {
  __shared__ int red[WARPS == 1 ? 1 : WARPS];
  const int lane = threadIdx.x & 31;
  const int warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const long long row = WARPS == 1 ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.rows) return;
  const long long bh = row / a.N_Q;
  const int i = (int)(row - bh * a.N_Q), b = (int)(bh / a.Hsel);
  const int nk = sp_len(a.lens, b, a.N_K);
  const int last = sp_last(i, nk, a.N_Q, a.causal);
  const int n = last < 0 ? 0 : last / kSpBlock + 1;
  const float* src = a.mass + row * a.NB;
  int* dst = a.idx + row * a.topk;

  uint32_t key[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (warp * V + k) * 32 + lane;
    key[k] = 0u;
    if (c < n) key[k] = c < a.n_first || c >= n - a.n_last ? 0xffffffffu : mass_key(__ldg(src + c));
  }
  // Largest threshold that at least topk keys reach (1 when fewer blocks are visible).
  uint32_t thr = 1u;
  int above = n;  // keys >= thr
  if (n > a.topk) {
    uint32_t t = 0u;
    int reach = n;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = t | (1u << bit);
      int cnt = 0;
#pragma unroll
      for (int k = 0; k < V; ++k) cnt += key[k] >= cand ? 1 : 0;
      cnt = select_sum<WARPS>(cnt, red, warp, lane);
      if (cnt >= a.topk) {
        t = cand;
        reach = cnt;
        if (cnt == a.topk) break;
      }
    }
    thr = t;
    above = reach;
  }
  // Keys above thr are all taken; of those equal to it, the lowest indices fill up.
  int ties = a.topk;  // how many keys equal to thr are taken
  if (above > a.topk) {
    int cnt = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) cnt += key[k] > thr ? 1 : 0;
    ties = a.topk - select_sum<WARPS>(cnt, red, warp, lane);
  }
  // Ranks in index order: this warp's blocks are consecutive, earlier warps come first.
  int eq0 = 0, gt0 = 0;  // equal / greater keys of earlier warps
  if (WARPS > 1) {
    int e = 0, g = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      e += __popc(__ballot_sync(0xffffffffu, key[k] == thr));
      g += __popc(__ballot_sync(0xffffffffu, key[k] > thr));
    }
    if (lane == 0) red[warp] = e;
    __syncthreads();
    for (int w = 0; w < warp; ++w) eq0 += red[w];
    __syncthreads();
    if (lane == 0) red[warp] = g;
    __syncthreads();
    for (int w = 0; w < warp; ++w) gt0 += red[w];
  }
  int at = gt0 + min(eq0, ties);
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const uint32_t eq = __ballot_sync(0xffffffffu, key[k] == thr);
    const bool take = key[k] > thr || (key[k] == thr && eq0 + __popc(eq & below) < ties);
    const uint32_t taken = __ballot_sync(0xffffffffu, take);
    if (take) dst[at + __popc(taken & below)] = (warp * V + k) * 32 + lane;
    at += __popc(taken);
    eq0 += __popc(eq);
  }
  const int have = min(n, a.topk);
  for (int e = have + (WARPS == 1 ? lane : (int)threadIdx.x); e < a.topk;
       e += WARPS == 1 ? 32 : 32 * WARPS)
    dst[e] = -1;
}

}  // namespace skl
