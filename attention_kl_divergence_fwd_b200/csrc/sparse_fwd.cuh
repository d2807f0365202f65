// sparse_fwd.cuh - attention over selected key blocks, forward (tcgen05 + TMEM + TMA).
//
//   out[i] = sum_j p_ij v_j,  p_ij = exp(s_ij - LSE_i),  s_ij = scale <q_i, k_j>,
//   LSE_i = log sum_j exp(s_ij),  j over the allowed keys of the blocks that i lists.
//
// CTA = one 128-row tile of packed query heads (sparse_common.cuh). Key tiles are pairs of
// listed blocks (128 keys, gathered into one buffer by two TMA boxes). Per key tile:
//   S = Q K^T into TMEM; two threads per row (one per block of the pair) turn 64 scores each
//   into probabilities against the row's reference m and write them back over the scores as
//   bf16; O += P V with P read from TMEM.
// The two threads share m. They raise it, with a rescale of O in TMEM, only when a score of
// theirs exceeds it by 2^8, so most tiles leave m and O alone; they exchange their maxima
// through shared memory every tile and so decide alike. Each thread keeps its own sum.
// P is rounded to bf16 for the tensor core (relative error at most 2^-8 each, the same as the
// output's own rounding); the row sums, references and O stay in fp32.
// A CTA keeps one score buffer: 256 TMEM columns and 97 KB of shared memory, so two CTAs share
// an SM and one's MMAs run under the other's exponentials.
// `splits` > 1: the tile's list is dealt to the CTAs of a cluster by rank; their normalised
// outputs and log-sum-exps are joined through distributed shared memory, so that a single
// token is one launch and no partial result leaves the chip.
// QUAD: tiles of at most 32 rows, four copies, each warp a quarter of the keys (sp_quad); the
// four quarters are joined like splits.
//
// Warps: 0-7 softmax (warp w: lane quarter w & 3, block w >> 2 of the pair), 8 producer (scans
// the bit matrix, TMA), 9 MMA + TMEM. QUAD: warps 0-3 only, 32 keys each.
#pragma once

#include "sparse_common.cuh"

namespace skl {

constexpr int kSpThreads = 320;

// One key tile as the producer announces it: how many blocks (0 = end), which, and which of
// the tile's queries list them.
struct SpInfo {
  int nb;
  int c[2];
  uint32_t w[2][4];
};

template <int D>
struct SpFwdCfg {
  static constexpr int BM = 128;
  static constexpr int QBYTES = BM * D * 2;
  static constexpr int KVBYTES = 128 * D * 2;         // one pair of K (or V) blocks
  static constexpr int NST = D == 128 ? 1 : 2;        // pair buffers each of K and V
  static constexpr int OFF_K = QBYTES;
  static constexpr int OFF_V = OFF_K + NST * KVBYTES;
  static constexpr int OFF_BAR = OFF_V + NST * KVBYTES;
  static constexpr int BAR_BYTES = 3584;
  static constexpr int SMEM = OFF_BAR + BAR_BYTES;
  static constexpr int TM_S = 0;    // 128 columns of scores, P over the first 64
  static constexpr int TM_O = 128;  // D columns
  static constexpr int TM_COLS = 256;
  static_assert(2 * (SMEM + 1024) <= 233472, "two CTAs per SM");
};

struct SpFwdBars {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t info_full[4];
  uint64_t s_full, p_full, o_full;
  uint64_t pair[4];  // the two warps of a lane quarter
  uint32_t tmem_base;
  int abort_flag;
  SpInfo info[4];
  float l2[128];  // row sums, then base-2 log-sum-exps of the partial rows
  float xch[2][2][128];  // what the two threads of a row exchange: tile parity, thread, row
};
static_assert(sizeof(SpFwdBars) <= SpFwdCfg<128>::BAR_BYTES, "barrier block");

// Sets the rows past nk of a [D/64][128][64] pair buffer's half to zero: with a padded cache
// they hold whatever the cache held, and 0 * NaN would reach the products.
template <int D>
__device__ __forceinline__ void sp_zero_tail(uint8_t* buf, int half, int first, int tid,
                                             int nthreads) {
  const int n = (kSpBlock - first) * 8 * (D / 64);  // 16-byte pieces
  for (int e = tid; e < n; e += nthreads) {
    const int blk = e / ((kSpBlock - first) * 8), r = e % ((kSpBlock - first) * 8);
    *reinterpret_cast<uint4*>(buf + blk * (128 * 128) + (half * 64 + first) * 128 + r * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}

// Producer's walk over the blocks of a tile's union, whole warp: emit(c, w0..w3) for each
// (w in units of the tile's own bits), in ascending order.
template <typename Emit>
__device__ __forceinline__ bool sp_scan(const SparseArgs& a, const SpTile& t, int lane,
                                        Emit&& emit) {
  const uint32_t tmask = a.Qn >= 32 ? 0xffffffffu : ((1u << a.Qn) - 1u) << t.bit0;
  for (int base = 0; base < a.NB; base += 32) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (base + lane < a.NB) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < t.nwords) w[k] = __ldg(t.words + (size_t)k * a.NB + base + lane) & tmask;
    }
    uint32_t nz = __ballot_sync(0xffffffffu, (w[0] | w[1] | w[2] | w[3]) != 0u);
    while (nz) {
      const int pos = __ffs(nz) - 1;
      nz &= nz - 1;
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = __shfl_sync(0xffffffffu, w[k], pos);
      if (!emit(base + pos, u)) return false;
    }
  }
  return true;
}

// Joins the partial rows of this cluster's CTAs (and of the four quarters): every source holds
// rows normalised by its own sum, with stage[slot * (D + 4)] and the base-2 log-sum-exps in l2;
// out = sum_s 2^(l_s - L) o_s, L = log2 sum_s 2^(l_s). Row r is joined by CTA r % splits, one
// warp per row.
template <int D, bool QUAD>
__device__ __forceinline__ void sp_join(const SparseArgs& a, const SpTile& t, uint32_t stage,
                                        uint32_t l2, int split, int warp, int lane) {
  constexpr int NS = QUAD ? 4 : 1;
  const int rows = a.Qn * a.G;
  for (int r = split + warp * a.splits; r < rows; r += 4 * a.splits) {
    const int g = r / a.Qn, i = t.q0 + r - g * a.Qn;
    if (i >= a.N_Q) continue;
    const int srcs = a.splits * NS;
    float mx = -INFINITY;
    for (int s = lane; s < srcs; s += 32)
      mx = fmaxf(mx, ld_cluster_f32(cluster_map(l2 + ((s % NS) * 32 + r) * 4, s / NS)));
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
    float acc[D / 32], tot = 0.f;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) acc[k] = 0.f;
    if (mx > -INFINITY) {
#pragma unroll 4
      for (int s = 0; s < srcs; ++s) {
        const int slot = (s % NS) * 32 + r;
        const float w = ex2_approx(ld_cluster_f32(cluster_map(l2 + slot * 4, s / NS)) - mx);
        tot += w;
        const uint32_t src = cluster_map(stage + slot * (D + 4) * 4, s / NS);
#pragma unroll
        for (int k = 0; k < D / 64; ++k) {
          const float2 o = ld_cluster_f32x2(src + (k * 64 + lane * 2) * 4);
          acc[2 * k] = fmaf(w, o.x, acc[2 * k]);
          acc[2 * k + 1] = fmaf(w, o.y, acc[2 * k + 1]);
        }
      }
    }
    const float inv = tot > 0.f ? 1.f / tot : 0.f;
    const size_t row = (size_t)(t.h0 + g) * a.N_Q + i;
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      *reinterpret_cast<uint32_t*>(a.out + row * D + k * 64 + lane * 2) =
          pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    if (lane == 0)
      a.lse[row] = tot > 0.f ? (mx + log2f(tot)) * 0.69314718055994530942f : -INFINITY;
  }
}

template <int D, bool QUAD>
__global__ void __launch_bounds__(kSpThreads, 2)
streamkl_sparse_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v, const SparseArgs a,
                           const uint32_t idesc_s2, const uint32_t idesc_s1,
                           const uint32_t idesc_o) {
  using C = SpFwdCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_skl_error, 4u);
    return;
  }
  SpFwdBars* bars = reinterpret_cast<SpFwdBars*>(smem + C::OFF_BAR);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Tiles of one pack are neighbours in the grid (they share K and V in L2), last tile first
  // (causal: the longest lists).
  const int split = blockIdx.x % a.splits;
  const int unit = blockIdx.x / a.splits;
  const int bp = unit / a.n_tiles;
  const SpTile t = sp_tile(a, bp, a.n_tiles - 1 - unit % a.n_tiles);

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars->q_full), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars->k_full[s]), 1);
      mbar_init(smem_u32(&bars->k_empty[s]), 1);
      mbar_init(smem_u32(&bars->v_full[s]), 1);
      mbar_init(smem_u32(&bars->v_empty[s]), 1);
    }
    for (int s = 0; s < 4; ++s) mbar_init(smem_u32(&bars->info_full[s]), 1);
    mbar_init(smem_u32(&bars->s_full), 1);
    mbar_init(smem_u32(&bars->p_full), QUAD ? 4 : 8);
    mbar_init(smem_u32(&bars->o_full), 1);
    for (int s = 0; s < 4; ++s) mbar_init(smem_u32(&bars->pair[s]), 2);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&bars->tmem_base), C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp < (QUAD ? 4 : 8)) {
    // ------------------------------------------------------------- softmax rows
    const int quarter = warp & 3, half = warp >> 2;
    const int r = QUAD ? lane : quarter * 32 + lane;
    const int g = r / a.Qn, qi = r - g * a.Qn, i = t.q0 + qi;
    const bool valid = g < a.G && i < a.N_Q;
    const int last = valid ? sp_last(i, t.nk, a.N_Q, a.causal) : -1;
    const int wi = qi >> 5, bi = a.Qn >= 32 ? (qi & 31) : t.bit0 + qi;
    const bool warp_live = __any_sync(0xffffffffu, valid);
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::TM_S, to = tmem + lane_off + C::TM_O;
    const float c = a.c;
    float m = -INFINITY, l = 0.f;
    // O *= f0 (this row; the two threads of a row take half of the columns each). S(n) is
    // complete, so O holds every earlier product.
    auto rescale = [&](float f0) {
      constexpr int DC = QUAD ? D : D / 2;
#pragma unroll
      for (int k = 0; k < DC; k += 8) {  // few registers: the scores are live
        const uint32_t at = to + (QUAD ? 0 : half * DC) + k;
        uint32_t o[8];
        tmem_ld_8_wait(at, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
        tmem_st_8(at, o);
      }
    };
    bool ok = true;
    int n = 0;
    for (;; ++n) {
      if (!mbar_wait(smem_u32(&bars->info_full[n & 3]), (n >> 2) & 1)) { ok = false; break; }
      const SpInfo& f = bars->info[n & 3];
      const int nb = f.nb;
      if (nb == 0) break;
      // This thread's block of the pair (QUAD: its half of one), and the last key of it that
      // the row reads.
      const int hb = QUAD ? quarter >> 1 : half;
      const bool on = hb < nb && ((f.w[hb][wi & 3] >> bi) & 1u);
      const int lim = on ? last - f.c[hb] * kSpBlock : -1;
      if (!mbar_wait(smem_u32(&bars->s_full), n & 1)) { ok = false; break; }
      tc_fence_after();
      // A padded cache's last block: rows past nk of V must not reach the product. S(n) is
      // complete, so the products before it are too and v_full is in this tile's phase.
      const int tail = t.nk & (kSpBlock - 1);
      bool at_end = false;
      if (tail != 0 && t.nk < a.N_K) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h < nb && f.c[h] == t.nk / kSpBlock) {
            const int st = n % C::NST;
            if (!mbar_wait(smem_u32(&bars->v_full[st]), (n / C::NST) & 1)) ok = false;
            sp_zero_tail<D>(smem + C::OFF_V + st * C::KVBYTES, h, tail, threadIdx.x, QUAD ? 128 : 256);
            fence_async_smem();
            at_end = true;
          }
      }
      if (!ok) break;
      if constexpr (QUAD) {
        // Columns 32 warp .. +31 of the key tile: half of block warp / 2.
        const int lq = lim - 32 * (warp & 1);
        uint32_t v[32];
        tmem_ld_32_wait(ts + 32 * warp, v);
        float mx = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if (k > lq) v[k] = 0xff800000u;  // -inf
          mx = fmaxf(mx, __uint_as_float(v[k]));
        }
        const float ms = mx == -INFINITY ? -INFINITY : mx * c;
        const bool raise = ms > m + 8.f || (m == -INFINITY && ms > -INFINITY);
        if (__any_sync(0xffffffffu, raise)) {
          const float f0 = raise ? ex2_approx(m - ms) : 1.f;
          if (raise) m = ms;
          l *= f0;
          if (n > 0) rescale(f0);
        }
        const float bias = m == -INFINITY ? 0.f : -m;
        uint32_t p[16], zero[16];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float e0 = ex2_approx(fmaf(__uint_as_float(v[k]), c, bias));
          const float e1 = ex2_approx(fmaf(__uint_as_float(v[k + 1]), c, bias));
          s0 += e0;
          s1 += e1;
          p[k >> 1] = pack_bf16x2(e0, e1);
          zero[k >> 1] = 0u;
        }
        l += s0 + s1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t at = ts + (q >> 1) * 64 + (q & 1) * 16;
          if (q == warp)
            tmem_st_16(at, p);
          else
            tmem_st_16(at, zero);
        }
        tmem_st_wait();
      } else {
        uint32_t v[64];
        float mx = -INFINITY;
        // A warp without rows, or whose block of the pair is missing, only votes.
        const bool work = warp_live && hb < nb;
        if (work) {
          tmem_ld_2x32_wait(ts + 64 * half, ts + 64 * half + 32, v);
          // Blocks are read whole or not at all except at the causal diagonal and the
          // sequence's end; only those mask single scores (the end's scores may be NaN).
          if (at_end || __any_sync(0xffffffffu, lim >= 0 && lim < 63)) {
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (k > lim) v[k] = 0xff800000u;  // -inf
          }
          mx = fmaxf(max_tree32<false>(v, 0, 31), max_tree32<false>(v, 32, 31));
          if (lim < 0) mx = -INFINITY;
        }
        const float ms = mx == -INFINITY ? -INFINITY : mx * c;
        // Exchange with the row's other thread (slots alternate by tile: the other thread has
        // read tile n - 2's before it arrives for n - 1).
        bars->xch[n & 1][half][quarter * 32 + lane] = ms;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->pair[quarter]));
        if (!mbar_wait(smem_u32(&bars->pair[quarter]), n & 1)) { ok = false; break; }
        const float both = fmaxf(ms, bars->xch[n & 1][half ^ 1][quarter * 32 + lane]);
        const bool raise = both > m + 8.f || (m == -INFINITY && both > -INFINITY);
        if (__any_sync(0xffffffffu, raise)) {
          const float f0 = raise ? ex2_approx(m - both) : 1.f;  // m = -inf: 0
          if (raise) m = both;
          l *= f0;
          if (n > 0) rescale(f0);
        }
        if (work) {
          const float bias = lim < 0 ? -INFINITY : (m == -INFINITY ? 0.f : -m);
          const uint64_t c2 = f2_pack(c, c), b2 = f2_pack(bias, bias);
          uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
          // Over the scores this thread has read, 32 keys at a time.
#pragma unroll
          for (int q = 0; q < 64; q += 32) {
            uint32_t p[16];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[q + k]), __uint_as_float(v[q + k + 1])), c2,
                               b2), x0, x1);
              x0 = ex2_approx(x0);
              x1 = ex2_approx(x1);
              if (k & 2)
                acc1 = f2_add(acc1, f2_pack(x0, x1));
              else
                acc0 = f2_add(acc0, f2_pack(x0, x1));
              p[k >> 1] = pack_bf16x2(x0, x1);
            }
            tmem_st_16(ts + 64 * half + q / 2, p);
          }
          float s0, s1;
          f2_unpack(f2_add(acc0, acc1), s0, s1);
          l += s0 + s1;
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->p_full));
    }
    if (ok && !mbar_wait(smem_u32(&bars->o_full), 0)) ok = false;
    if (!ok) {
      atomicOr(&g_skl_error, 1u);
      *abort_flag = 1;
    }
    tc_fence_after();
    if constexpr (!QUAD) {  // the row's sum over both blocks of every pair
      const int at = quarter * 32 + lane;
      bars->xch[n & 1][half][at] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->pair[quarter]));
      if (ok && !mbar_wait(smem_u32(&bars->pair[quarter]), n & 1)) {
        atomicOr(&g_skl_error, 1u);
        ok = false;
      }
      l = bars->xch[n & 1][0][at] + bars->xch[n & 1][1][at];
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const float l2 = l > 0.f ? m + log2f(l) : -INFINITY;
    const bool some = n > 0;  // else O was never written
    constexpr int DC = QUAD ? D : D / 2;  // columns this thread writes
    if (QUAD || a.splits > 1) {
      // The copies and products of this CTA are done; its buffers take the partial rows.
      if (!mbar_wait(smem_u32(&bars->q_full), 0)) ok = false;
      const int slot = quarter * 32 + lane;
      if (half == 0) bars->l2[slot] = ok && valid ? l2 : -INFINITY;
      float* dst = reinterpret_cast<float*>(smem) + slot * (D + 4);
#pragma unroll
      for (int k0 = 0; k0 < DC; k0 += 32) {
        const int k = half * DC + k0;
        uint32_t o[32];
        if (some) tmem_ld_32_wait(to + k, o);
        if (valid) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = some && l > 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(dst + k + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
    } else if (warp_live && ok) {
      const size_t row = (size_t)(t.h0 + g) * a.N_Q + i;
#pragma unroll
      for (int k0 = 0; k0 < DC; k0 += 32) {
        const int k = half * DC + k0;
        uint32_t o[32];
        if (some) tmem_ld_32_wait(to + k, o);
        if (valid) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = some && l > 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * D + k);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(o[e]), __uint_as_float(o[e + 1]));
            w.y = pack_bf16x2(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
            w.z = pack_bf16x2(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5]));
            w.w = pack_bf16x2(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7]));
            dst[e >> 3] = w;
          }
        }
      }
      if (valid && half == 0) a.lse[row] = l2 * 0.69314718055994530942f;
    }
  } else if (warp == 8) {
    // ---------------------------------------------------- producer (whole warp scans)
    if (lane == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
      const uint32_t qb = smem_u32(&bars->q_full);
      mbar_arrive_expect_tx(qb, (QUAD ? 4 : 1) * a.Qn * a.G * D * 2);
      for (int blk = 0; blk < D / 64; ++blk)
        for (int copy = 0; copy < (QUAD ? 4 : 1); ++copy)
          tma_load_3d(sb + blk * (C::BM * 128) + copy * (32 * 128), &map_q, qb, blk * 64, t.q0,
                      t.h0, l2_policy_evict_first());
    }
    const uint64_t keep = l2_policy_evict_last();
    bool ok = true;
    int n = 0, rank = 0, pend = 0;
    int pc[2] = {0, 0};
    uint32_t pw[2][4] = {};
    // Announces the pending blocks as key tile n and loads them (nb = 0: the end).
    auto push = [&](int nb) -> bool {
      bool fine = true;
      if (lane == 0) {
        SpInfo& f = bars->info[n & 3];
        f.nb = nb;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f.c[h] = pc[h];
#pragma unroll
          for (int k = 0; k < 4; ++k) f.w[h][k] = pw[h][k];
        }
        mbar_arrive(smem_u32(&bars->info_full[n & 3]));
        if (nb > 0) {
          const int st = n % C::NST;
          const uint32_t ph = ((n / C::NST) & 1) ^ 1;
          const uint32_t kf = smem_u32(&bars->k_full[st]), vf = smem_u32(&bars->v_full[st]);
          fine = mbar_wait(smem_u32(&bars->k_empty[st]), ph);
          if (fine) {
            mbar_arrive_expect_tx(kf, nb * 64 * D * 2);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              for (int blk = 0; blk < D / 64 && h < nb; ++blk)
                tma_load_3d(sb + C::OFF_K + st * C::KVBYTES + blk * (128 * 128) + h * (64 * 128),
                            &map_k, kf, blk * 64, pc[h] * kSpBlock, t.kv, keep);
            fine = mbar_wait(smem_u32(&bars->v_empty[st]), ph);
          }
          if (fine) {
            mbar_arrive_expect_tx(vf, nb * 64 * D * 2);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              for (int blk = 0; blk < D / 64 && h < nb; ++blk)
                tma_load_3d(sb + C::OFF_V + st * C::KVBYTES + blk * (128 * 128) + h * (64 * 128),
                            &map_v, vf, blk * 64, pc[h] * kSpBlock, t.kv, keep);
          }
        }
      }
      fine = __shfl_sync(0xffffffffu, fine ? 1 : 0, 0) != 0;
      ++n;
      pend = 0;
      return fine;
    };
    auto emit = [&](int c, const uint32_t (&u)[4]) -> bool {
      if (rank++ % a.splits != split) return true;
      if (pend == 0) {
        pc[0] = c;
#pragma unroll
        for (int k = 0; k < 4; ++k) pw[0][k] = u[k];
        pend = 1;
        return true;
      }
      pc[1] = c;
#pragma unroll
      for (int k = 0; k < 4; ++k) pw[1][k] = u[k];
      return push(2);
    };
    if (a.direct) {
      // One query: its list as a bitmap over the blocks, in the rows 16-31 of the Q buffer that
      // the pack's at most 16 rows leave unused (2 KB: 16384 blocks).
      uint32_t* bits = reinterpret_cast<uint32_t*>(smem + 16 * 128);
      const int sel = t.b * a.Hsel + t.p / (a.P / a.Hsel);
      const int* idx = a.idx + (size_t)sel * a.topk;
      const int lastkey = sp_last(0, t.nk, 1, a.causal);
      for (int w = lane; w < (a.NB + 31) / 32; w += 32) bits[w] = 0u;
      __syncwarp();
      for (int e = lane; e < a.topk; e += 32) {
        const int c = __ldg(idx + e);
        if (lastkey >= 0 && c >= 0 && c <= lastkey / kSpBlock) atomicOr(&bits[c >> 5], 1u << (c & 31));
      }
      __syncwarp();
      const uint32_t one[4] = {1u, 0u, 0u, 0u};
      for (int w0 = 0; ok && w0 < (a.NB + 31) / 32; w0 += 32) {
        const uint32_t mine = w0 + lane < (a.NB + 31) / 32 ? bits[w0 + lane] : 0u;
        uint32_t lanes = __ballot_sync(0xffffffffu, mine != 0u);
        while (ok && lanes) {
          const int src = __ffs(lanes) - 1;
          lanes &= lanes - 1;
          uint32_t w = __shfl_sync(0xffffffffu, mine, src);
          while (ok && w) {
            ok = emit((w0 + src) * 32 + __ffs(w) - 1, one);
            w &= w - 1;
          }
        }
      }
    } else {
      ok = sp_scan(a, t, lane, emit);
    }
    if (ok && pend) ok = push(1);
    const int tiles = n;
    if (ok) ok = push(0);
    if (!ok && lane == 0) {
      atomicOr(&g_skl_error, 1u);
      *abort_flag = 1;
      // Let the copies in flight land before the CTA can exit (each wait is bounded).
      mbar_wait(smem_u32(&bars->q_full), 0);
      for (int j = max(0, tiles - C::NST); j < tiles; ++j) {
        mbar_wait(smem_u32(&bars->k_full[j % C::NST]), (j / C::NST) & 1);
        mbar_wait(smem_u32(&bars->v_full[j % C::NST]), (j / C::NST) & 1);
      }
    }
    // With no key tile nothing else waits for the Q copy.
    if (lane == 0 && tiles == 0) mbar_wait(smem_u32(&bars->q_full), 0);
  } else if (warp == 9 && elect_one()) {
    // ------------------------------------------------------------------ MMA issuer
    bool ok = mbar_wait(smem_u32(&bars->q_full), 0);
    for (int n = 0; ok; ++n) {
      ok = mbar_wait(smem_u32(&bars->info_full[n & 3]), (n >> 2) & 1);
      if (!ok) break;
      const int nb = bars->info[n & 3].nb;
      if (nb == 0) break;
      const int st = n % C::NST;
      const uint32_t ph = (n / C::NST) & 1;
      const uint32_t sk = sb + C::OFF_K + st * C::KVBYTES, sv = sb + C::OFF_V + st * C::KVBYTES;
      if (!(ok = mbar_wait(smem_u32(&bars->k_full[st]), ph))) break;
      tc_fence_after();
      const uint32_t id = nb == 2 ? idesc_s2 : idesc_s1;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
        umma_bf16_ss(tmem + C::TM_S, sdesc_sw128(sb + off, 16, 1024),
                     sdesc_sw128(sk + off, 16, 1024), id, kk > 0);
      }
      umma_commit(smem_u32(&bars->k_empty[st]));
      umma_commit(smem_u32(&bars->s_full));
      if (!(ok = mbar_wait(smem_u32(&bars->v_full[st]), ph))) break;
      if (!(ok = mbar_wait(smem_u32(&bars->p_full), n & 1))) break;
      tc_fence_after();
      // O += P V: A = P from TMEM, B = V [keys][d] MN-major, 16 keys per step.
      for (int kk = 0; kk < 4 * nb; ++kk)
        umma_bf16_ts(tmem + C::TM_O, tmem + C::TM_S + (kk >> 2) * 64 + (kk & 3) * 8,
                     sdesc_sw128(sv + kk * 2048, 128 * 128, 1024), idesc_o,
                     (n > 0 || kk > 0) ? 1u : 0u);
      umma_commit(smem_u32(&bars->v_empty[st]));
    }
    umma_commit(smem_u32(&bars->o_full));
    if (!ok) {
      atomicOr(&g_skl_error, 1u);
      *abort_flag = 1;
    }
    // Every MMA of this thread must be complete before TMEM is released.
    mbar_wait(smem_u32(&bars->o_full), 0);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  __syncwarp();
  if (a.splits > 1) cluster_sync();
  if ((QUAD || a.splits > 1) && warp < 4)
    sp_join<D, QUAD>(a, t, sb, smem_u32(bars->l2), split, warp, lane);
  __syncwarp();
  if (a.splits > 1) cluster_sync();  // another CTA may still be reading this one's rows
}

}  // namespace skl
