// block_select.cuh - the key blocks each query reads, from their masses.
//
// Of the n_vis blocks that hold an allowed key of the query: the first n_first, the last
// n_last, and then the heaviest of the rest until topk are taken; equal masses go to the lower
// index, NaN ranks below every number. Written in ascending order, -1 behind the last.
//
// A row's masses become unsigned keys in their order (forced blocks get the largest key) and
// stay in registers. A threshold that exactly topk keys reach is found by bisection between the
// least lane maximum (or key) and the largest free key: keys order like the logarithm of the mass, so the bracket
// narrows to the gap behind the topk-th key in a few steps (6 on average for 256 blocks), and the
// search ends with the first threshold in that gap, or, with ties, at the topk-th key itself. The
// selection is then written by ranks in index order, which gives the ascending list and the
// ties' order without a sort. One warp per row when there are many rows, eight when there are few
// or when a row has more than 1024 blocks. Bound by issue slots (89 %) for many rows: 131072 rows of up to 256 blocks
// 62 us (1.2 TB/s of masses), of which the bisection is 8 us and the stores 10; by latency for few:
// 512 rows of 1024 blocks 6.4 us.
#pragma once

#include "sparse_common.cuh"

namespace skl {

struct SelectArgs {
  const float* mass;  // [B, Hsel, N_Q, NB]
  const int* lens;
  int* idx;           // [B, Hsel, N_Q, topk]
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

// Reductions over a row's warps; `red` alternates between two sets so that one barrier per
// reduction suffices.
template <int WARPS, typename Op>
__device__ __forceinline__ uint32_t select_join(uint32_t x, uint32_t (*red)[8], int& turn, int warp,
                                                int lane, Op op) {
  if (WARPS == 1) return x;
  if (lane == 0) red[turn][warp] = x;
  __syncthreads();
  uint32_t r = red[turn][0];
#pragma unroll
  for (int k = 1; k < WARPS; ++k) r = op(r, red[turn][k]);
  turn ^= 1;
  return r;
}

// One row whose n visible blocks fit V keys per thread. Warp w, register k and lane hold block
// (w * V + k) * 32 + lane: reads are coalesced and ranks in index order follow from ballots.
template <int V, int WARPS>
__device__ __forceinline__ void select_row(const SelectArgs& a, long long row, int n,
                                           uint32_t (*red)[8], int warp, int lane) {
  int turn = 0;
  const float* src = a.mass + row * a.NB;
  int* dst = a.idx + row * a.topk;
  const int base = warp * V * 32;
  auto add = [](uint32_t x, uint32_t y) { return x + y; };
  auto lesser = [](uint32_t x, uint32_t y) { return min(x, y); };
  auto larger = [](uint32_t x, uint32_t y) { return max(x, y); };
  float x[V];
  uint32_t key[V];
  bool plain = true;  // masses that are >= 0 (not NaN) need only their sign bit set
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = base + k * 32 + lane;
    x[k] = c < n ? __ldg(src + c) : 0.f;
  }
#pragma unroll
  for (int k = 0; k < V; ++k) plain = plain && x[k] >= 0.f;
  if (__all_sync(0xffffffffu, plain)) {
#pragma unroll
    for (int k = 0; k < V; ++k) key[k] = __float_as_uint(x[k]) | 0x80000000u;  // -0 equals 0
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) key[k] = mass_key(x[k]);
  }
  uint32_t kmax = 0u, lane_max = 0u;  // of the free blocks; of all visible ones of this lane
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c0 = base + k * 32, c = c0 + lane;
    if (c0 + 32 > n && c >= n) key[k] = 0u;
    // Registers without a forced block (most) skip the per-lane tests.
    if (c0 < a.n_first || c0 + 32 > n - a.n_last) {
      const bool force = c < n && (c < a.n_first || c >= n - a.n_last);
      kmax = force ? kmax : max(kmax, key[k]);
      key[k] = force ? 0xffffffffu : key[k];
    } else {
      kmax = max(kmax, key[k]);
    }
    lane_max = max(lane_max, key[k]);
  }
  uint32_t thr = 1u;  // taken: keys above thr, and the first `ties` equal to it
  int ties = a.topk;
  bool exact = true;  // every key that reaches thr is taken
  if (n > a.topk) {
    // count(key >= lo) >= topk > count(key >= hi); forced keys reach every threshold.
    const int forced = a.n_first + a.n_last;  // n > topk >= n_first + n_last: they are distinct
    if (forced == a.topk) {
      thr = 0xfffffffeu;  // no free key is taken (masses' keys end below)
    } else {
      kmax = select_join<WARPS>(__reduce_max_sync(0xffffffffu, kmax), red, turn, warp, lane, larger);
      // The least of the lanes' largest keys is reached by 32 keys per warp that holds 32 visible
      // blocks; else the least key of all.
      uint32_t lo;
      if (a.topk <= 32 && n >= 32) {
        lo = n >= base + 32 ? __reduce_min_sync(0xffffffffu, lane_max) : 0u;
        lo = select_join<WARPS>(lo, red, turn, warp, lane, larger);
      } else {
        uint32_t kmin = 0xffffffffu;
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (base + k * 32 + lane < n) kmin = min(kmin, key[k]);
        lo = select_join<WARPS>(__reduce_min_sync(0xffffffffu, kmin), red, turn, warp, lane, lesser);
      }
      uint32_t hi = kmax + 1u;
      int reach = a.topk + 1;  // keys >= lo: exactly topk once found so, else more (or ties)
      while (hi - lo > 1u && hi > lo) {
        const uint32_t mid = lo + ((hi - lo) >> 1);
        uint32_t cnt = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) cnt += key[k] >= mid ? 1u : 0u;
        cnt = select_join<WARPS>(__reduce_add_sync(0xffffffffu, cnt), red, turn, warp, lane, add);
        if ((int)cnt >= a.topk) {
          lo = mid;
          reach = (int)cnt;
          if (reach == a.topk) break;
        } else {
          hi = mid;
        }
      }
      thr = lo;
      if (reach != a.topk) {
        exact = false;
        uint32_t cnt = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) cnt += key[k] > thr ? 1u : 0u;
        ties = a.topk - (int)select_join<WARPS>(__reduce_add_sync(0xffffffffu, cnt), red, turn, warp,
                                                lane, add);
      }
    }
  }
  // Ranks in index order: this warp's blocks are consecutive, earlier warps come first.
  int eq0 = 0, gt0 = 0;  // equal / greater keys of earlier warps
  if (WARPS > 1) {
    uint32_t e = 0, g = 0;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      e += __popc(__ballot_sync(0xffffffffu, key[k] == thr));
      g += __popc(__ballot_sync(0xffffffffu, key[k] > thr));
    }
    if (lane == 0) red[turn][warp] = e | (g << 16);  // at most 8192 blocks
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
      eq0 += red[turn][w] & 0xffffu;
      gt0 += red[turn][w] >> 16;
    }
  }
  int at = gt0 + min(eq0, ties);
  const uint32_t below = (1u << lane) - 1u;
  if (exact) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const bool take = key[k] >= thr;
      const uint32_t taken = __ballot_sync(0xffffffffu, take);
      if (take) dst[at + __popc(taken & below)] = base + k * 32 + lane;
      at += __popc(taken);
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const uint32_t eq = __ballot_sync(0xffffffffu, key[k] == thr);
      const bool take = key[k] > thr || (key[k] == thr && eq0 + __popc(eq & below) < ties);
      const uint32_t taken = __ballot_sync(0xffffffffu, take);
      if (take) dst[at + __popc(taken & below)] = base + k * 32 + lane;
      at += __popc(taken);
      eq0 += __popc(eq);
    }
  }
  const int have = min(n, a.topk);
  for (int e = have + (WARPS == 1 ? lane : (int)threadIdx.x); e < a.topk;
       e += WARPS == 1 ? 32 : 32 * WARPS)
    dst[e] = -1;
}

// WARPS = 1: four rows per CTA, one warp each, with the fewest registers that hold the row's
// visible blocks (causal rows see half of them on average). WARPS > 1: one row per CTA. The grid is
// (selection heads, rows), so that no row needs a division.
template <int V, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS)
streamkl_block_select_kernel(const SelectArgs a) {
  __shared__ uint32_t red[2][8];
  constexpr int ROWS = WARPS == 1 ? 4 : 1;
  const int lane = threadIdx.x & 31;
  const int warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const int bh = blockIdx.x;
  const int nk = a.lens == nullptr ? a.N_K : sp_len(a.lens, bh / a.Hsel, a.N_K);
  for (int i = blockIdx.y * ROWS + (WARPS == 1 ? threadIdx.x >> 5 : 0); i < a.N_Q;
       i += gridDim.y * ROWS) {
    const long long row = (long long)bh * a.N_Q + i;
    const int last = sp_last(i, nk, a.N_Q, a.causal);
    const int n = last < 0 ? 0 : last / kSpBlock + 1;
    if (WARPS == 1 && V > 2 && n <= 64)
      select_row<2, WARPS>(a, row, n, red, warp, lane);
    else if (WARPS == 1 && V > 4 && n <= 128)
      select_row<4, WARPS>(a, row, n, red, warp, lane);
    else if (WARPS == 1 && V == 8 && n <= 192)
      select_row<6, WARPS>(a, row, n, red, warp, lane);
    else
      select_row<V, WARPS>(a, row, n, red, warp, lane);
    if (WARPS > 1) __syncthreads();  // the next row starts over with the reduction buffers
  }
}

}  // namespace skl
