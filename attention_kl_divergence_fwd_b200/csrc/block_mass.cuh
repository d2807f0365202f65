// block_mass.cuh - probability mass of an attention map on blocks of 64 keys (tcgen05 + TMA).
//
//   mass[i, c] = 1/G sum_{g < G} sum_{j in block c, j allowed} exp(scale <q_gi, k_j> - LSE_gi)
// over the G query heads that share a K head. The map itself is never stored.
//
// CTA = one 128-row tile of packed query heads (sparse_common.cuh) and a range of blocks. K
// streams through a ring in pairs of blocks; per pair one N = 128 product into one of two TMEM
// score buffers; one thread per row reduces each block's 64 scores to one number. The row
// numbers of 32 blocks are staged in shared memory, summed over the heads of the group and
// written as 128 contiguous bytes per query.
// Three forms (MODE):
//   kMassNorm   the rows' LSEs are given (the divergence's forward has them): that is the result;
//   kMassParts  per head the block's base-2 log-sum-exp is written, and a second kernel sums those
//               to the row's LSE and normalises;
//   kMassFused  (QUAD) a cluster shares a tile's blocks, keeps the block log-sum-exps in shared
//               memory, exchanges the rows' sums through distributed shared memory and writes
//               normalised masses: single tokens in one launch without a workspace.
// The scores of a block need no running maximum across blocks, so the keys of one query can be
// spread over as many CTAs as there are pairs of blocks.
// Bound by the exponential unit (one exponential per pair) for many queries, by reading K for
// few. Two CTAs per SM. Measured on a B200: 32 heads, 16384 tokens, d = 64, causal: 1011 us (the
// unit alone would take 923 us; a quarter of the exponentials runs on the FMA pipe, 1196, 1095,
// 1027 and 1117 us with 0, 1, 2 and 3 of 8 pairs); one token of 16 sequences of up to 32768 keys:
// 72 us, K read at 4.8 TB/s.
//
// QUAD: tiles of at most 32 rows, four copies, each row warp 32 of a pair's 128 keys (sp_quad);
// a block's two halves are joined when the staged values are written.
//
// Warps: 0-7 rows (warp w: lane quarter w & 3, block w >> 2 of every pair; QUAD: the pairs of
// parity w >> 2), 8 TMA producer, 9 MMA + TMEM.
#pragma once

#include "fwd_kernel.cuh"
#include "sparse_common.cuh"

namespace skl {

constexpr int kMassNorm = 0, kMassParts = 1, kMassFused = 2;
constexpr int kMassStage = 128 * 33;  // staged values (floats)

struct MassArgs {
  SparseArgs s;         // P = K heads of the map, G = query heads per K head
  int bpc;              // blocks per CTA (a multiple of 2), n_chunks = ceil(NB / bpc)
  int n_chunks;
  const float* row_lse; // [B, H, N_Q] (kMassNorm)
  float* mass;          // [B, P, N_Q, NB]
  float* blse;          // [B, H, N_Q, NB] base-2 log-sum-exp of each visible block (kMassParts)
};

template <int D>
struct MassCfg {
  static constexpr int BM = 128;
  static constexpr int QBYTES = BM * D * 2;
  static constexpr int KBYTES = 128 * D * 2;
  static constexpr int NST = D == 128 ? 2 : 4;
  static constexpr int OFF_K = QBYTES;
  static constexpr int OFF_STG = OFF_K + NST * KBYTES;  // [128 rows][33] floats
  static constexpr int OFF_BAR = OFF_STG + kMassStage * 4;
  static constexpr int SMEM = OFF_BAR + 512;
  static constexpr int TM_COLS = 256;
  static_assert(2 * (SMEM + 1024) <= 233472, "two CTAs per SM");
};

struct MassBars {
  uint64_t q_full;
  uint64_t k_full[4], k_empty[4];
  uint64_t s_full[2], s_free[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  float2 row[32];  // kMassFused: {maximum, sum relative to it} of this CTA's blocks, per row
};
static_assert(sizeof(MassBars) <= 512, "barrier block");

constexpr int kMassThreads = 320;

// Exponentials of a block on the FMA pipe, of every 8 pairs of keys (the rest on the
// exponential unit, which otherwise bounds the kernel).
constexpr int kMassPoly = 2;

// Value of a row over N keys: sum 2^(s c - lse2) (NORM) or log2 sum 2^(s c); keys past lim are
// left out.
template <bool NORM, int N>
__device__ __forceinline__ float mass_block(const uint32_t (&v)[N], float c, float nl, int lim) {
  float bias = nl;
  if (!NORM) {
    float mx = -INFINITY;
    if (lim >= N - 1) {
#pragma unroll
      for (int k = 0; k < N; k += 32) mx = fmaxf(mx, max_tree32<false>(v, k, 31));
    } else {
#pragma unroll
      for (int k = 0; k < N; k += 32) mx = fmaxf(mx, max_tree32<true>(v, k, lim - k));
    }
    if (mx == -INFINITY) return -INFINITY;
    bias = -mx * c;
  }
  float sum;
  if (lim >= N - 1) {
    const uint64_t c2 = f2_pack(c, c), b2 = f2_pack(bias, bias);
    uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const uint64_t x =
          f2_fma(f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, b2);
      uint64_t e;
      if (poly_rank((k >> 1) & 7) < kMassPoly) {
        e = exp2_fma2_low(x);
      } else {
        float x0, x1;
        f2_unpack(x, x0, x1);
        e = f2_pack(ex2_approx(x0), ex2_approx(x1));
      }
      if (k & 2)
        acc1 = f2_add(acc1, e);
      else
        acc0 = f2_add(acc0, e);
    }
    float s0, s1;
    f2_unpack(f2_add(acc0, acc1), s0, s1);
    sum = s0 + s1;
  } else {
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float e = ex2_approx(fmaf(__uint_as_float(v[k]), c, bias));
      sum += k <= lim ? e : 0.f;
    }
  }
  return NORM ? sum : log2f(sum) - bias;
}

template <int D, int MODE, bool QUAD>
__global__ void __launch_bounds__(kMassThreads, 2)
streamkl_block_mass_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k, const MassArgs ma,
                           const uint32_t idesc) {
  using C = MassCfg<D>;
  constexpr bool NORM = MODE == kMassNorm;
  static_assert(MODE != kMassFused || QUAD, "the fused form is for tiles of few rows");
  const SparseArgs& a = ma.s;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_skl_error, 4u);
    return;
  }
  MassBars* bars = reinterpret_cast<MassBars*>(smem + C::OFF_BAR);
  float* stage = reinterpret_cast<float*>(smem + C::OFF_STG);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int chunk = blockIdx.x % ma.n_chunks, unit = blockIdx.x / ma.n_chunks;
  const int bp = unit / a.n_tiles, tile = a.n_tiles - 1 - unit % a.n_tiles;
  const int b = bp / a.P, p = bp - b * a.P;
  const int q0 = tile * a.Qn, h0 = b * a.H + p * a.G;
  const int nk = sp_len(a.lens, b, a.N_K);
  const int c_begin = chunk * ma.bpc, c_end = min(a.NB, c_begin + ma.bpc);
  // Blocks that the tile's last query sees; the rest of the range is only written as 0.
  const int last_tile = sp_last(min(q0 + a.Qn, a.N_Q) - 1, nk, a.N_Q, a.causal);
  const int n_vis = min(c_end, last_tile / kSpBlock + (last_tile >= 0 ? 1 : 0)) - c_begin;
  const int steps = n_vis > 0 ? (n_vis + 1) / 2 : 0;
  if (MODE == kMassParts && steps == 0) return;

  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_k);
      bars->abort_flag = 0;
    }
    constexpr int S_FREE = offsetof(MassBars, s_free) / 8, LAST = offsetof(MassBars, drain) / 8;
    sp_init_barriers(&bars->q_full, LAST + 1, kMassThreads, lane, [](int i) {
      return i == S_FREE || i == S_FREE + 1 ? (QUAD ? 4 : 8) : 1;
    });
  } else {
    if (warp == 9) {
      tmem_alloc(smem_u32(&bars->tmem_base), C::TM_COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    named_bar_sync(15, kMassThreads);
    tc_fence_after();
  }
  const uint32_t tmem = bars->tmem_base;

  if (warp < 8) {
    const int quarter = warp & 3, wg = warp >> 2;
    const int r = QUAD ? lane : quarter * 32 + lane;
    const int g = r / a.Qn, qi = r - g * a.Qn, i = q0 + qi;
    const bool valid = g < a.G && i < a.N_Q;
    const int last = valid ? sp_last(i, nk, a.N_Q, a.causal) : -1;
    const bool warp_live = __any_sync(0xffffffffu, valid);
    const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16);
    const float c = a.c;
    float nl = 0.f;
    bool row_on = valid;
    if (NORM && valid) {
      const float l = __ldg(ma.row_lse + (size_t)(h0 + g) * a.N_Q + i);
      row_on = l != -INFINITY;
      nl = row_on ? -l * 1.4426950408889634f : 0.f;
    }
    const int rows = a.Qn * a.G;
    // Queries of this tile that exist; rows are written for those only.
    const int nq = min(a.Qn, a.N_Q - q0);
    const float inv_g = 1.f / (float)a.G;
    // Writes the staged values of blocks cg .. cg + n - 1.
    auto staged = [&](int row) -> float {
      const float x = stage[row * 33 + lane];
      if (!QUAD) return x;
      const float y = stage[(32 + row) * 33 + lane];  // the block's other half
      if (NORM) return x + y;
      const float m = fmaxf(x, y);
      return m == -INFINITY ? m : m + log2f(exp2f(x - m) + exp2f(y - m));
    };
    auto flush = [&](int cg, int n) {
      named_bar_sync(1, 256);
      if (NORM) {
        float* dst = ma.mass + ((size_t)bp * a.N_Q + q0) * a.NB + cg;
        for (int q = warp; q < nq; q += 8) {
          float s = 0.f;
          for (int h = 0; h < a.G; ++h) s += staged(h * a.Qn + q);
          if (lane < n) dst[(size_t)q * a.NB + lane] = s * inv_g;
        }
      } else {
        float* dst = ma.blse + ((size_t)h0 * a.N_Q + q0) * a.NB + cg;
        for (int h = 0; h < a.G; ++h)
          for (int q = warp; q < nq; q += 8)
            if (lane < n) dst[((size_t)h * a.N_Q + q) * a.NB + lane] = staged(h * a.Qn + q);
      }
      named_bar_sync(1, 256);
    };
    bool ok = true;
    const int n_blocks = c_end - c_begin;
    for (int s = 0; s < steps; ++s) {
      const int cb = 2 * s;  // first block of the pair, from c_begin
      if (!QUAD || (s & 1) == wg) {
        // After a wait that ran out the warp still takes part in every named barrier.
        if (ok && !mbar_wait(smem_u32(&bars->s_full[s & 1]), (s >> 1) & 1)) ok = false;
        tc_fence_after();
        float x = NORM ? 0.f : -INFINITY;
        if constexpr (QUAD) {
          // Keys 32 quarter .. +31 of the pair: half quarter & 1 of block quarter / 2.
          uint32_t v[32];
          tmem_ld_32_wait(ts + (s & 1) * 128 + 32 * quarter, v);
          const int lim =
              row_on ? last - (c_begin + cb) * kSpBlock - 32 * quarter : (valid ? -1 : 31);
          if (__all_sync(0xffffffffu, lim >= 31)) {
            x = mass_block<NORM, 32>(v, c, nl, 31);
          } else if (__any_sync(0xffffffffu, lim >= 0)) {
            const float y = mass_block<NORM, 32>(v, c, nl, min(lim, 30));
            const float z = mass_block<NORM, 32>(v, c, nl, 31);
            x = lim >= 31 ? z : (lim >= 0 ? y : x);
          }
          if constexpr (MODE == kMassFused) {
            if (valid) stage[((quarter & 1) * rows + r) * (ma.bpc + 1) + cb + (quarter >> 1)] = x;
          } else {
            stage[((quarter & 1) * 32 + r) * 33 + ((cb + (quarter >> 1)) & 31)] = x;
          }
        } else {
          if (warp_live) {
            uint32_t v[64];
            tmem_ld_2x32_wait(ts + (s & 1) * 128 + 64 * wg, ts + (s & 1) * 128 + 64 * wg + 32, v);
            // Rows past the tile's end take the common path; their values are not written.
            const int lim = row_on ? last - (c_begin + cb + wg) * kSpBlock : (valid ? -1 : 63);
            if (__all_sync(0xffffffffu, lim >= 63)) {
              x = mass_block<NORM, 64>(v, c, nl, 63);
            } else if (__any_sync(0xffffffffu, lim >= 0)) {
              const float y = mass_block<NORM, 64>(v, c, nl, min(lim, 62));
              const float z = mass_block<NORM, 64>(v, c, nl, 63);
              x = lim >= 63 ? z : (lim >= 0 ? y : x);
            }
          }
          stage[r * 33 + ((cb + wg) & 31)] = x;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->s_free[s & 1]));
      }
      if (MODE != kMassFused && (((cb + 2) & 31) == 0 || s == steps - 1)) {
        const int cg = cb & ~31;
        flush(c_begin + cg, min(cb + 2, n_blocks) - cg);
      }
    }
    if (!ok) {
      atomicOr(&g_skl_error, 1u);
      *abort_flag = 1;
    }
    if constexpr (MODE == kMassFused) {
      // Per row: the two halves of every block joined into the first, and the chunk's sum.
      named_bar_sync(1, 256);
      const int ld = ma.bpc + 1, have = min(2 * steps, max(n_blocks, 0));
      for (int row = warp; row < rows; row += 8) {
        float* x = stage + row * ld;
        const float* y = stage + (rows + row) * ld;
        float m = -INFINITY, sum = 0.f;
        for (int k = lane; k < have; k += 32) {
          const float lo = x[k], hi = y[k], t = fmaxf(lo, hi);
          const float v = t == -INFINITY ? t : t + log2f(exp2f(lo - t) + exp2f(hi - t));
          x[k] = v;
          if (v > m) {
            sum = sum * exp2f(m - v) + 1.f;
            m = v;
          } else if (v > -INFINITY) {
            sum += exp2f(v - m);
          }
        }
        float mx = m;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        sum = m > -INFINITY ? sum * exp2f(m - mx) : 0.f;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (lane == 0) bars->row[row] = make_float2(mx, sum);
      }
    }
    if (NORM) {  // blocks that no query of the tile sees
      const int z0 = c_begin + min(2 * steps, n_blocks);
      float* dst = ma.mass + ((size_t)bp * a.N_Q + q0) * a.NB;
      for (int q = warp; q < nq; q += 8)
        for (int cc = z0 + lane; cc < c_end; cc += 32) dst[(size_t)q * a.NB + cc] = 0.f;
    }
  } else if (warp == 8) {
    if (lane == 0 && steps > 0) {
      // A tile that is the only one of its K head is the only reader of that K.
      const uint64_t keep = a.n_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
      const uint32_t qb = smem_u32(&bars->q_full);
      mbar_arrive_expect_tx(qb, (QUAD ? 4 : 1) * a.Qn * a.G * D * 2);
      for (int blk = 0; blk < D / 64; ++blk)
        for (int copy = 0; copy < (QUAD ? 4 : 1); ++copy)
          tma_load_3d(sb + blk * (C::BM * 128) + copy * (32 * 128), &map_q, qb, blk * 64, q0, h0,
                      keep);
      int issued = 0;
      for (int s = 0; s < steps; ++s) {
        const int st = s % C::NST;
        if (!mbar_wait(smem_u32(&bars->k_empty[st]), ((s / C::NST) & 1) ^ 1)) {
          atomicOr(&g_skl_error, 1u);
          *abort_flag = 1;
          break;
        }
        const uint32_t kf = smem_u32(&bars->k_full[st]);
        mbar_arrive_expect_tx(kf, C::KBYTES);
        for (int blk = 0; blk < D / 64; ++blk)
          tma_load_3d(sb + C::OFF_K + st * C::KBYTES + blk * (128 * 128), &map_k, kf, blk * 64,
                      (c_begin + 2 * s) * kSpBlock, bp, keep);
        issued = s + 1;
      }
      if (*abort_flag) {
        mbar_wait(qb, 0);
        for (int j = max(0, issued - C::NST); j < issued; ++j)
          mbar_wait(smem_u32(&bars->k_full[j % C::NST]), (j / C::NST) & 1);
      }
    }
  } else if (steps > 0 && elect_one()) {
    bool ok = mbar_wait(smem_u32(&bars->q_full), 0);
    for (int s = 0; ok && s < steps; ++s) {
      const int st = s % C::NST;
      ok = mbar_wait(smem_u32(&bars->k_full[st]), (s / C::NST) & 1) &&
           mbar_wait(smem_u32(&bars->s_free[s & 1]), ((s >> 1) & 1) ^ 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sk = sb + C::OFF_K + st * C::KBYTES;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
        umma_bf16_ss(tmem + (s & 1) * 128, sdesc_sw128(sb + off, 16, 1024),
                     sdesc_sw128(sk + off, 16, 1024), idesc, kk > 0);
      }
      umma_commit(smem_u32(&bars->k_empty[st]));
      umma_commit(smem_u32(&bars->s_full[s & 1]));
    }
    umma_commit(smem_u32(&bars->drain));
    if (!ok) {
      atomicOr(&g_skl_error, 1u);
      *abort_flag = 1;
    }
    mbar_wait(smem_u32(&bars->drain), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  if constexpr (MODE == kMassFused) {
    // The rows' log-sum-exps over the whole cluster, then mass = 1/G sum_g 2^(x_g - L_g).
    __syncwarp();
    cluster_sync();
    if (warp < 8) {
      const int rows = a.Qn * a.G, ld = ma.bpc + 1;
      const int have = min(2 * steps, max(c_end - c_begin, 0));
      float big = 0.f;  // lane = row
      if (lane < rows) {
        float2 part[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          part[e] = e < ma.n_chunks ? ld_cluster_f32x2(cluster_map(smem_u32(&bars->row[lane]), e))
                                    : make_float2(-INFINITY, 0.f);
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, part[e].x);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (part[e].x > -INFINITY) sum += part[e].y * exp2f(part[e].x - mx);
        big = sum > 0.f ? mx + log2f(sum) : 0.f;  // a row without keys: every x is -inf
      }
      const float inv_g = 1.f / (float)a.G;
      const int nq = min(a.Qn, a.N_Q - q0);
      float* dst = ma.mass + ((size_t)bp * a.N_Q + q0) * a.NB + c_begin;
      for (int q = 0; q < nq; ++q)
        for (int k0 = warp * 32; k0 < c_end - c_begin; k0 += 256) {
          const int k = k0 + lane;
          float s = 0.f;
          for (int g = 0; g < a.G; ++g) {
            const float l = __shfl_sync(0xffffffffu, big, g * a.Qn + q);
            if (k < have) s += exp2f(stage[(g * a.Qn + q) * ld + k] - l);
          }
          if (k < c_end - c_begin) dst[(size_t)q * a.NB + k] = s * inv_g;
        }
    }
    __syncwarp();
    cluster_sync();  // another CTA may still be reading this one's rows
  }
}

// Second kernel of kMassParts: mass[c] = 1/G sum_g 2^(x_gc - L_g), with
// L_g = log2 sum_c 2^(x_gc) over the row's visible blocks. One CTA per (K head, query): each warp
// takes the sums of every eighth head, then all threads the blocks.
__global__ void __launch_bounds__(256) streamkl_block_norm_kernel(const MassArgs ma) {
  const SparseArgs& a = ma.s;
  __shared__ float row_l[128];
  const int bp = blockIdx.x / a.N_Q, i = blockIdx.x - bp * a.N_Q, b = bp / a.P, p = bp - b * a.P;
  const int nk = sp_len(a.lens, b, a.N_K);
  const int last = sp_last(i, nk, a.N_Q, a.causal);
  const int n = last < 0 ? 0 : last / kSpBlock + 1;
  float* dst = ma.mass + ((size_t)bp * a.N_Q + i) * a.NB;
  const float* x = ma.blse + ((size_t)(b * a.H + p * a.G) * a.N_Q + i) * a.NB;
  const size_t hs = (size_t)a.N_Q * a.NB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < a.G; g += 8) {
    float mx = -INFINITY, sum = 0.f;
    for (int c = lane; c < n; c += 128) {  // four loads in flight
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = c + 32 * k < n ? x[g * hs + c + 32 * k] : -INFINITY;
      const float t = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
      if (t > mx) {
        sum *= exp2f(mx - t);
        mx = t;
      }
      if (mx > -INFINITY) {
#pragma unroll
        for (int k = 0; k < 4; ++k) sum += exp2f(y[k] - mx);
      }
    }
    float all = mx;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, s));
    sum = mx > -INFINITY ? sum * exp2f(mx - all) : 0.f;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
    if (lane == 0) row_l[g] = all + log2f(sum);
  }
  __syncthreads();
  const float inv_g = 1.f / (float)a.G;
  for (int c = threadIdx.x; c < a.NB; c += 256) {
    float y = 0.f;
    if (c < n)
      for (int g = 0; g < a.G; ++g) y += exp2f(x[g * hs + c] - row_l[g]);
    dst[c] = y * inv_g;
  }
}

}  // namespace skl
