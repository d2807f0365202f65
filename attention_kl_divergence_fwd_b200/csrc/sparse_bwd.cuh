// sparse_bwd.cuh - attention over selected key blocks, backward (tcgen05 + TMEM + TMA).
//
// With p_ij = exp(s_ij - LSE_i) recomputed tile by tile, D_i = sum_d out_i dout_i and
//   dP_ij = <dout_i, v_j>,  dS_ij = p_ij (dP_ij - D_i):
//   dV_j = sum_i p_ij dout_i,  dK_j = scale sum_i dS_ij q_i,  dQ_i = scale sum_j dS_ij k_j.
// Two kernels (the second starts in the first one's tail: 1337 tokens 101 -> 91 us, 2 x 4096 tokens
// 420 -> 404), one per direction of the bit matrix, so that every sum has one owner: no
// atomics, the same bits every time, and K heads shared by a group of query heads are summed
// inside one CTA (a tile's rows are the whole group). Recomputing S and dP in both costs 7
// products per tile pair instead of 5; adding dQ parts (or dK and dV parts) through L2 instead
// would move 64 KB of fp32 per (tile, block) pair, more time than the two extra products.
// P and dS are rounded to bf16 for the tensor core; every accumulator is fp32, and each
// gradient is rounded once, to bf16.
#pragma once

#include "sparse_fwd.cuh"

namespace skl {

// Sum of the products of eight bf16 pairs (a bf16 is the upper half of its fp32).
__device__ __forceinline__ float dot8(const uint4& u, const uint4& v, float acc) {
  const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), acc);
    acc = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), acc);
  }
  return acc;
}

// rows[r] = {LSE * log2(e), D_r = sum_d out * dout}: D / 8 lanes per row, 16 bytes each, several
// rows in flight per lane. Bound by reading out and dout once (2 x 16 heads x 4096 rows of 128:
// 67 MB in 10.8 us, 6.2 TB/s). Rows that see one block are left to the kernel below
// (skip_short).
constexpr int kRowsPerGroup = 4;
template <int D>
__global__ void __launch_bounds__(256)
streamkl_sparse_rows_kernel(const SparseArgs a, const __nv_bfloat16* out,
                            const __nv_bfloat16* dout, const float* lse, long long rows,
                            bool skip_short) {
  grid_allow_next();
  constexpr int L = D / 8;                       // lanes per row
  constexpr int GROUPS = 256 / L;                // rows a CTA takes at once
  const int at = threadIdx.x % L;
  const long long row0 = (long long)blockIdx.x * (GROUPS * kRowsPerGroup) + threadIdx.x / L;
  uint4 o[kRowsPerGroup], g[kRowsPerGroup];
#pragma unroll
  for (int k = 0; k < kRowsPerGroup; ++k) {
    const long long row = row0 + k * GROUPS;
    o[k] = g[k] = make_uint4(0u, 0u, 0u, 0u);
    if (row < rows) {
      o[k] = __ldg(reinterpret_cast<const uint4*>(out + row * D) + at);
      g[k] = __ldg(reinterpret_cast<const uint4*>(dout + row * D) + at);
    }
  }
#pragma unroll
  for (int k = 0; k < kRowsPerGroup; ++k) {
    float acc = dot8(o[k], g[k], 0.f);
#pragma unroll
    for (int s = L / 2; s > 0; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    const long long row = row0 + k * GROUPS;
    if (at == 0 && row < rows) {
      if (skip_short) {
        const int bh = (int)(row / a.N_Q);
        const int last = sp_last((int)(row - (long long)bh * a.N_Q),
                                 sp_len(a.lens, bh / a.H, a.N_K), a.N_Q, a.causal);
        if (last >= 0 && last < kSpBlock) continue;
      }
      a.rows[row] = make_float2(__ldg(lse + row) * 1.4426950408889634f, acc);
    }
  }
  grid_end_after_previous();
}

// D_r = sum_j p_rj <dout_r, v_j> in fp32 for the rows that see at most one block. out carries the
// roundings of P and its own, which the sum above passes on to dS: about 2^-8.7 / sqrt(n) of it
// for n keys of like weight, so much as dS's own rounding when n is small (a step over 200 tokens:
// dQ and dK 2.7e-3 off in norm with the sum above, 2.4e-3 with this).
// CTA = 8 queries of one head (one warp each, two keys per lane); K and V of block 0 in shared
// memory. It reads the lists and LSEs itself and writes rows[] for these rows, so that it, the
// kernel above and the one that builds the bit matrix run beside one another (training step of
// 2 x 16 heads x 4096 tokens 402 -> 397 us).
template <int D>
__global__ void __launch_bounds__(256)
streamkl_sparse_short_rows_kernel(const SparseArgs a, const __nv_bfloat16* q,
                                  const __nv_bfloat16* kk, const __nv_bfloat16* v,
                                  const __nv_bfloat16* dout, const float* lse) {
  grid_allow_next();
  constexpr int PITCH = D / 8 + 1;  // 16-byte pieces; the odd pitch spreads a column over banks
  __shared__ uint4 sk[kSpBlock * PITCH], sv[kSpBlock * PITCH];
  const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H;
  const int nk = sp_len(a.lens, b, a.N_K);
  // Rows see more keys as i grows: this CTA has short rows only if its first row is one (or sees
  // none). The grid covers at most 65535 * 8 rows at once.
  if (nk < 1 || sp_last(blockIdx.y * 8, nk, a.N_Q, a.causal) >= kSpBlock) {
    grid_end_after_previous();
    return;
  }
  const size_t kv0 = (size_t)(b * a.Hkv + h / (a.H / a.Hkv)) * a.N_K * D;
  for (int e = threadIdx.x; e < min(nk, kSpBlock) * (D / 8); e += 256) {
    const int j = e / (D / 8), ch = e % (D / 8);
    sk[j * PITCH + ch] = __ldg(reinterpret_cast<const uint4*>(kk + kv0) + e);
    sv[j * PITCH + ch] = __ldg(reinterpret_cast<const uint4*>(v + kv0) + e);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, sel = b * a.Hsel + h / (a.H / a.Hsel);
  const float c = a.scale * 1.4426950408889634f;
  for (long long at = blockIdx.y * 8 + (threadIdx.x >> 5); at < a.N_Q; at += 8ll * gridDim.y) {
    const int i = (int)at, last = sp_last(i, nk, a.N_Q, a.causal);
    if (last >= kSpBlock) break;
    if (last < 0) continue;
    const int* idx = a.idx + ((size_t)sel * a.N_Q + i) * a.topk;
    bool listed = false;
    for (int e = lane; e < a.topk; e += 32) listed |= __ldg(idx + e) == 0;
    listed = __any_sync(0xffffffffu, listed);
    const size_t row = (size_t)blockIdx.x * a.N_Q + i;
    const uint4* qr = reinterpret_cast<const uint4*>(q + row * D);
    const uint4* gr = reinterpret_cast<const uint4*>(dout + row * D);
    // Keys past the row's last are left out below; their index stays within what was loaded.
    const int j0 = min(lane, last) * PITCH, j1 = min(lane + 32, last) * PITCH;
    float s0 = 0.f, s1 = 0.f, d0 = 0.f, d1 = 0.f;
#pragma unroll 4
    for (int ch = 0; ch < D / 8; ++ch) {
      const uint4 x = __ldg(qr + ch), y = __ldg(gr + ch);
      s0 = dot8(x, sk[j0 + ch], s0);
      s1 = dot8(x, sk[j1 + ch], s1);
      d0 = dot8(y, sv[j0 + ch], d0);
      d1 = dot8(y, sv[j1 + ch], d1);
    }
    const float x = __ldg(lse + row) * 1.4426950408889634f, nl = -x;
    float acc = lane <= last ? ex2_approx(fmaf(s0, c, nl)) * d0 : 0.f;
    acc += lane + 32 <= last ? ex2_approx(fmaf(s1, c, nl)) * d1 : 0.f;
#pragma unroll
    for (int e = 16; e > 0; e >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, e);
    if (lane == 0) a.rows[row] = make_float2(x, listed ? acc : 0.f);
  }
  grid_end_after_previous();
}

// ------------------------------------------------------------------ dQ, query-major
//
// CTA = one 128-row tile, as in the forward; key tiles are single blocks. Per block:
// S = Q K^T and dP = dO V^T into TMEM, two threads per row form dS and write it over S as
// bf16, dQ += dS K. 256 TMEM columns and 113 KB: two CTAs per SM. Bound by the chain of a
// step (scores 768 cycles, dS 900, product 256, hand-overs; 2880 per step and CTA, the products'
// operand reads 1024 of 1440 per block and SM; 16 heads over 4, 16384 tokens, 32 blocks per query:
// 456 us). One CTA per SM with Q and dO in TMEM and two score buffers took 460.
// Warps: 0-7 rows (warp w: lane quarter w & 3, keys 32 (w >> 2) .. +31), 8 producer, 9 MMA.
constexpr int kSpDqThreads = 320;
template <int D>
struct SpDqCfg {
  static constexpr int BM = 128;
  static constexpr int QBYTES = BM * D * 2;
  static constexpr int SLOT = 64 * D * 2;
  static constexpr int NK = 2;                      // K slots
  static constexpr int NV = D == 128 ? 1 : 2;       // V slots
  static constexpr int OFF_DO = QBYTES;
  static constexpr int OFF_K = 2 * QBYTES;
  static constexpr int OFF_V = OFF_K + NK * SLOT;
  static constexpr int OFF_BAR = OFF_V + NV * SLOT;
  static constexpr int SMEM = OFF_BAR + 1024;
  static constexpr int TM_S = 0, TM_DP = 64, TM_DQ = 128, TM_COLS = 256;
  static_assert(2 * (SMEM + 1024) <= 233472, "two CTAs per SM");
};

struct SpDqBars {
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t info_full[4];
  uint64_t s_full, ds_full, dq_full;
  uint32_t tmem_base;
  int abort_flag;
  SpBlockInfo info[4];
};
static_assert(sizeof(SpDqBars) <= 1024, "barrier block");

// dS = p (dP - D), and p itself (BOTH), of 32 keys as bf16 pairs, from scores v[0..31] and
// dP v[32..63]; keys past lim give 0.
template <bool BOTH>
__device__ __forceinline__ void sp_ds(const uint32_t (&v)[64], float c, float nl, float nd,
                                      int lim, uint32_t (&ds)[16], uint32_t (&pp)[16]) {
  const uint64_t c2 = f2_pack(c, c), nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
  const bool whole = __all_sync(0xffffffffu, lim >= 31);
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float x0, x1, d0, d1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, nl2), x0, x1);
    const uint64_t e = f2_pack(ex2_approx(x0), ex2_approx(x1));
    const uint64_t t =
        f2_add(f2_pack(__uint_as_float(v[32 + k]), __uint_as_float(v[33 + k])), nd2);
    f2_unpack(f2_mul(e, t), d0, d1);
    float e0, e1;
    f2_unpack(e, e0, e1);
    if (!whole) {
      d0 = k <= lim ? d0 : 0.f;
      d1 = k + 1 <= lim ? d1 : 0.f;
      e0 = k <= lim ? e0 : 0.f;
      e1 = k + 1 <= lim ? e1 : 0.f;
    }
    ds[k >> 1] = pack_bf16x2(d0, d1);
    if (BOTH) pp[k >> 1] = pack_bf16x2(e0, e1);
  }
}

template <int D>
__global__ void __launch_bounds__(kSpDqThreads, 2)
streamkl_sparse_dq_kernel(const __grid_constant__ CUtensorMap map_q,
                          const __grid_constant__ CUtensorMap map_do,
                          const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const SparseArgs a,
                          const uint32_t idesc_s, const uint32_t idesc_dp,
                          const uint32_t idesc_dq) {
  using C = SpDqCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_skl_error, 4u);
    return;
  }
  SpDqBars* bars = reinterpret_cast<SpDqBars*>(smem + C::OFF_BAR);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
  const int bp = unit / a.n_tiles;
  const SpTile t = sp_tile(a, bp, a.n_tiles - 1 - unit % a.n_tiles);

  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_do);
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
      bars->abort_flag = 0;
    }
    constexpr int DS_FULL = offsetof(SpDqBars, ds_full) / 8, LAST = offsetof(SpDqBars, dq_full) / 8;
    sp_init_barriers(&bars->q_full, LAST + 1, kSpDqThreads, lane,
                     [](int i) { return i == DS_FULL ? 8 : 1; });
  } else {
    if (warp == 9) {
      tmem_alloc(smem_u32(&bars->tmem_base), C::TM_COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    named_bar_sync(15, kSpDqThreads);
    tc_fence_after();
  }
  const uint32_t tmem = bars->tmem_base;

  if (warp < 8) {
    const int quarter = warp & 3, half = warp >> 2;
    const int r = quarter * 32 + lane;
    const int g = r / a.Qn, qi = r - g * a.Qn, i = t.q0 + qi;
    const bool valid = g < a.G && i < a.N_Q;
    const int last = valid ? sp_last(i, t.nk, a.N_Q, a.causal) : -1;
    const int wi = qi >> 5, bi = a.Qn >= 32 ? (qi & 31) : t.bit0 + qi;
    const size_t row = (size_t)(t.h0 + g) * a.N_Q + i;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::TM_S, tp = tmem + lane_off + C::TM_DP;
    const uint32_t tq = tmem + lane_off + C::TM_DQ;
    const float2 rv = valid ? __ldg(a.rows + row) : make_float2(0.f, 0.f);
    const float nl = -rv.x, nd = -rv.y, c = a.c;
    bool ok = true;
    int n = 0;
    for (;; ++n) {
      if (!mbar_wait(smem_u32(&bars->info_full[n & 3]), (n >> 2) & 1)) { ok = false; break; }
      const SpBlockInfo& f = bars->info[n & 3];
      if (f.c < 0) break;
      const bool on = (f.w[wi & 3] >> bi) & 1u;
      const int lim = on ? last - f.c * kSpBlock : -1;
      const int tail = t.nk & (kSpBlock - 1);
      const bool at_end = tail != 0 && t.nk < a.N_K && f.c == t.nk / kSpBlock;
      if (!mbar_wait(smem_u32(&bars->s_full), n & 1)) { ok = false; break; }
      tc_fence_after();
      if (at_end) {  // S is complete: K may lose its rows past nk before dQ += dS K
        uint8_t* kb = smem + C::OFF_K + (n % C::NK) * C::SLOT;
        const int per = (kSpBlock - tail) * 8;
        for (int e = threadIdx.x; e < per * (D / 64); e += 256)
          *reinterpret_cast<uint4*>(kb + (e / per) * (64 * 128) + tail * 128 + (e % per) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
      }
      uint32_t v[64], p[16];  // 32 scores, 32 dP
      tmem_ld_2x32_wait(ts + 32 * half, tp + 32 * half, v);
      sp_ds<false>(v, c, nl, nd, lim - 32 * half, p, p);
      tmem_st_16(ts + 32 * half, p);  // over the scores this thread has read
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ds_full));
    }
    if (ok && !mbar_wait(smem_u32(&bars->dq_full), 0)) ok = false;
    if (a.splits > 1 && ok && !mbar_wait(smem_u32(&bars->q_full), 0)) ok = false;
    if (!ok) {
      atomicOr(&g_skl_error, 2u);
      *abort_flag = 1;
    }
    tc_fence_after();
    if (ok) {
#pragma unroll
      for (int k0 = 0; k0 < D / 2; k0 += 32) {
        const int k = half * (D / 2) + k0;
        uint32_t o[32];
        if (n > 0) tmem_ld_32_wait(tq + k, o);
        if (a.splits > 1) {
          // The copies and products of this CTA are done; its buffers take the partial rows.
          float* part = reinterpret_cast<float*>(smem) + r * (D + 4) + k;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(part + e) =
                n > 0 ? make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_uint4(0u, 0u, 0u, 0u);
        } else if (valid) {
          uint4* dst = reinterpret_cast<uint4*>(a.dq + row * D + k);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = n > 0 ? __uint_as_float(o[e + q]) * a.scale : 0.f;
            dst[e >> 3] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                     pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
          }
        }
      }
    }
  } else if (warp == 8) {
    if (lane == 0) {
      const uint32_t qb = smem_u32(&bars->q_full);
      mbar_arrive_expect_tx(qb, 2 * a.Qn * a.G * D * 2);
      for (int blk = 0; blk < D / 64; ++blk) {
        tma_load_3d(sb + blk * (C::BM * 128), &map_q, qb, blk * 64, t.q0, t.h0,
                    l2_policy_evict_first());
        tma_load_3d(sb + C::OFF_DO + blk * (C::BM * 128), &map_do, qb, blk * 64, t.q0, t.h0,
                    l2_policy_evict_first());
      }
    }
    const uint64_t keep = l2_policy_evict_last();
    SpScan scan;
    bool ok = true;
    int n = 0;
    for (;;) {
      uint32_t u[4] = {0u, 0u, 0u, 0u};
      const int c = scan.next(a, t, split, lane, u);
      if (lane == 0) {
        SpBlockInfo& f = bars->info[n & 3];
        f.c = c;
#pragma unroll
        for (int k = 0; k < 4; ++k) f.w[k] = u[k];
        mbar_arrive(smem_u32(&bars->info_full[n & 3]));
        const int ks = n % C::NK, vs = n % C::NV;
        const uint32_t kf = smem_u32(&bars->k_full[ks]), vf = smem_u32(&bars->v_full[vs]);
        ok = mbar_wait(smem_u32(&bars->k_empty[ks]), ((n / C::NK) & 1) ^ 1);
        if (ok && c < 0) {
          mbar_arrive(kf);  // the MMA thread learns of the end from k_full alone
        } else if (ok) {
          mbar_arrive_expect_tx(kf, C::SLOT);
          for (int blk = 0; blk < D / 64; ++blk)
            tma_load_3d(sb + C::OFF_K + ks * C::SLOT + blk * (64 * 128), &map_k, kf, blk * 64,
                        c * kSpBlock, t.kv, keep);
          ok = mbar_wait(smem_u32(&bars->v_empty[vs]), ((n / C::NV) & 1) ^ 1);
          if (ok) {
            mbar_arrive_expect_tx(vf, C::SLOT);
            for (int blk = 0; blk < D / 64; ++blk)
              tma_load_3d(sb + C::OFF_V + vs * C::SLOT + blk * (64 * 128), &map_v, vf, blk * 64,
                          c * kSpBlock, t.kv, keep);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (c < 0 || !ok) break;
      ++n;
    }
    if (!ok && lane == 0) {
      atomicOr(&g_skl_error, 2u);
      *abort_flag = 1;
      mbar_wait(smem_u32(&bars->q_full), 0);
      // Of step n itself K may not have been asked for; then its wait runs out.
      for (int j = max(0, n + 1 - C::NK); j <= n; ++j)
        mbar_wait(smem_u32(&bars->k_full[j % C::NK]), (j / C::NK) & 1);
      for (int j = max(0, n - C::NV); j < n; ++j)
        mbar_wait(smem_u32(&bars->v_full[j % C::NV]), (j / C::NV) & 1);
    }
    if (lane == 0 && n == 0) mbar_wait(smem_u32(&bars->q_full), 0);
  } else if (elect_one()) {
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t lq = sdesc_lo(sb, 16), ldo = sdesc_lo(sb + C::OFF_DO, 16);
    const uint32_t lk0 = sdesc_lo(sb + C::OFF_K, 16), lv0 = sdesc_lo(sb + C::OFF_V, 16);
    const uint32_t lkn0 = sdesc_lo(sb + C::OFF_K, 64 * 128);  // K as [keys][d], MN-major
    bool ok = mbar_wait(smem_u32(&bars->q_full), 0);
    // Waits for K and V of step n: 1, no such step: 0, a wait ran out: -1.
    auto loaded = [&](int n) -> int {  // the entry was written before the arrival on k_full
      if (!mbar_wait(smem_u32(&bars->k_full[n % C::NK]), (n / C::NK) & 1)) return -1;
      if (bars->info[n & 3].c < 0) return 0;
      return mbar_wait(smem_u32(&bars->v_full[n % C::NV]), (n / C::NV) & 1) ? 1 : -1;
    };
    auto scores = [&](int n) {
      const int ks = n % C::NK, vs = n % C::NV;
      const uint32_t lk = lk0 + ks * (C::SLOT >> 4), lv = lv0 + vs * (C::SLOT >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16_ss_lh(tmem + C::TM_S, lq + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                        lk + (((kk >> 2) * (64 * 128) + (kk & 3) * 32) >> 4), hi, idesc_s, kk > 0);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16_ss_lh(tmem + C::TM_DP, ldo + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                        lv + (((kk >> 2) * (64 * 128) + (kk & 3) * 32) >> 4), hi, idesc_dp, kk > 0);
      umma_commit(smem_u32(&bars->s_full));
      umma_commit(smem_u32(&bars->v_empty[vs]));
    };
    int next = ok ? loaded(0) : -1;
    if (next > 0) {
      tc_fence_after();
      scores(0);
    }
    for (int n = 0; next > 0; ++n) {
      // The next step's K and V are awaited before this step's dS, so that once dS is there its
      // product and the next scores go out back to back.
      if ((next = loaded(n + 1)) < 0) break;
      if (!mbar_wait(smem_u32(&bars->ds_full), n & 1)) {
        next = -1;
        break;
      }
      tc_fence_after();
      const uint32_t lkn = lkn0 + (n % C::NK) * (C::SLOT >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_bf16_ts_lh(tmem + C::TM_DQ, tmem + C::TM_S + (kk >> 1) * 32 + (kk & 1) * 8,
                        lkn + kk * (2048 >> 4), hi, idesc_dq, (n > 0 || kk > 0) ? 1u : 0u);
      umma_commit(smem_u32(&bars->k_empty[n % C::NK]));
      if (next > 0) scores(n + 1);
    }
    ok = next >= 0;
    umma_commit(smem_u32(&bars->dq_full));
    if (!ok) {
      atomicOr(&g_skl_error, 2u);
      *abort_flag = 1;
    }
    mbar_wait(smem_u32(&bars->dq_full), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  if (a.splits > 1) {
    // dQ = the sum of the cluster's parts, in rank order; row r is summed by CTA r % splits.
    __syncwarp();
    cluster_sync();
    for (int r = split + warp * a.splits; r < a.Qn * a.G; r += 10 * a.splits) {
      const int g = r / a.Qn, i = t.q0 + r - g * a.Qn;
      if (i >= a.N_Q) continue;
#pragma unroll
      for (int k = lane * 2; k < D; k += 64) {
        float x = 0.f, y = 0.f;
        for (int p = 0; p < a.splits; ++p) {
          const float2 v = ld_cluster_f32x2(cluster_map(sb + (r * (D + 4) + k) * 4, p));
          x += v.x;
          y += v.y;
        }
        *reinterpret_cast<uint32_t*>(a.dq + ((size_t)(t.h0 + g) * a.N_Q + i) * D + k) =
            pack_bf16x2(x * a.scale, y * a.scale);
      }
    }
    __syncwarp();
    cluster_sync();  // another CTA may still be reading this one's rows
  }
  grid_end_after_previous();
}

// ------------------------------------------------------------------ dK, dV, key-major
//
// CTA (or cluster of kv_splits CTAs, which deal the tiles by rank and sum their parts through
// distributed shared memory) = one block of 64 keys of one K head; it walks the tiles (of every pack that reads this
// K head) whose word column lists the block. Per tile: S = Q K^T and dP = dO V^T (rows on the
// lanes, 64 key columns), one thread per row writes P and dS as bf16 into shared memory, then
//   dV^T += dO^T P  and  dK^T += Q^T dS   (d on the lanes, keys on the columns).
// Three Q and two dO buffers: with two {Q, dO} stages the MMA thread waited 1000 of 3250 cycles per
// step for loads; now a step takes about 1950, of them 1536 in 32 MMAs bound by their operand reads
// (16 heads over 4, 16384 tokens, 32 blocks per query: 730 us).
// For d = 64 both products take the stacked operand [dO | Q] (128 lanes) and keep the half
// they need: an M of 64 would run at the same speed.
// Warps: 0-15 rows (warp w: lane quarter w & 3, steps of parity (w >> 2) & 1, keys 32 (w >> 3)
// .. +31), 16 producer, 17 MMA + TMEM.
constexpr int kSpDkvThreads = 576;

template <int D>
struct SpDkvCfg {
  static constexpr int SLOT = 64 * D * 2;
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr int PT = 128 * 128;              // bf16 [128 rows][64 keys]
  // Buffers of Q, dO and {P, dS}. At d = 128 shared memory holds three Q, two dO and one P / dS;
  // at d = 64 {dO, Q} are stacked operands, adjacent in four stages.
  static constexpr int NQ = D == 128 ? 3 : 4;
  static constexpr int ND = D == 128 ? 2 : 4;
  static constexpr int NP = D == 128 ? 1 : 2;
  static constexpr int OFF_V = SLOT;                // K first
  static constexpr int OFF_Q = 2 * SLOT;
  static constexpr int OFF_P = OFF_Q + (NQ + ND) * QBYTES;
  static constexpr int OFF_BAR = OFF_P + NP * 2 * PT;
  static constexpr int SMEM = OFF_BAR + 1024;
  static __device__ __forceinline__ uint32_t off_do(int n) {
    return OFF_Q + (D == 128 ? (n % ND) * QBYTES : (n % ND) * 2 * QBYTES);
  }
  static __device__ __forceinline__ uint32_t off_q(int n) {
    return OFF_Q + (D == 128 ? (ND + n % NQ) * QBYTES : (n % NQ) * 2 * QBYTES + QBYTES);
  }
  static constexpr int TM_S = 0;                    // buffer b: S at 128 b, dP at 128 b + 64
  static constexpr int TM_DV = 256, TM_DK = 320, TM_COLS = 512;
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct SpTileInfo {
  int tile;  // tile of pack p, -1 = end
  int p;
  uint32_t w[4];
};

struct SpDkvBars {
  uint64_t k_full;
  uint64_t q_full[4], q_empty[4], do_full[4], do_empty[4];
  uint64_t info_full[8];
  uint64_t s_full[2], ds_full[2], ds_empty[2];  // ds_empty by P / dS buffer
  uint64_t acc_full;
  uint32_t tmem_base;
  int abort_flag;
  SpTileInfo info[8];
};
static_assert(sizeof(SpDkvBars) <= 1024, "barrier block");

template <int D>
__global__ void __launch_bounds__(kSpDkvThreads, 1)
streamkl_sparse_dkv_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_do,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v, const SparseArgs a,
                           const uint32_t idesc_s, const uint32_t idesc_dp,
                           const uint32_t idesc_acc) {
  using C = SpDkvCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_skl_error, 4u);
    return;
  }
  SpDkvBars* bars = reinterpret_cast<SpDkvBars*>(smem + C::OFF_BAR);
  volatile int* abort_flag = &bars->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_allow_next();
  // Block 0 of every head first: causal maps list the early blocks most.
  const int split = blockIdx.x % a.kv_splits, unit = blockIdx.x / a.kv_splits;
  const int kv = unit % (a.B * a.Hkv), blk0 = unit / (a.B * a.Hkv);
  const int b = kv / a.Hkv;
  const int nk = sp_len(a.lens, b, a.N_K);
  const int ppk = a.P / a.Hkv;               // packs that read this K head
  const int p0 = (kv - b * a.Hkv) * ppk;
  const int rows = a.Qn * a.G;               // rows of a tile that TMA writes

  if (warp == 16) {
    if (lane == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_do);
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
      bars->abort_flag = 0;
    }
    constexpr int DS_FULL = offsetof(SpDkvBars, ds_full) / 8;
    constexpr int LAST = offsetof(SpDkvBars, acc_full) / 8;
    sp_init_barriers(&bars->k_full, LAST + 1, kSpDkvThreads, lane,
                     [](int i) { return i == DS_FULL || i == DS_FULL + 1 ? 8 : 1; });
  } else {
    if (warp == 17) {
      tmem_alloc(smem_u32(&bars->tmem_base), C::TM_COLS);
      tmem_relinquish();
    }
    // Rows of the Q and dO buffers that no copy writes enter the row sums of dV and dK with a
    // factor of 0 and must be finite: zero them once.
    if (rows < 128 && warp < 16) {
      const int per = (128 - rows) * 8;
      for (int e = threadIdx.x; e < per * (C::NQ + C::ND) * (D / 64); e += 512)
        *reinterpret_cast<uint4*>(smem + C::OFF_Q + (e / per) * (128 * 128) + rows * 128 +
                                  (e % per) * 16) = make_uint4(0u, 0u, 0u, 0u);
      fence_async_smem();
    }
    tc_fence_before();
    named_bar_sync(15, kSpDkvThreads);
    tc_fence_after();
  }
  const uint32_t tmem = bars->tmem_base;

  if (warp < 16) {
    const int wg = (warp >> 2) & 1, half = warp >> 3, quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int g = r / a.Qn, qi = r - g * a.Qn;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::TM_S + 128 * wg;
    const uint32_t prow = sb + C::OFF_P + (C::NP == 2 ? wg * 2 * C::PT : 0) + r * 128;
    const float c = a.c;
    bool ok = true;
    int n = 0;
    for (;; ++n) {
      if (!mbar_wait(smem_u32(&bars->info_full[n & 7]), (n >> 3) & 1)) { ok = false; break; }
      const SpTileInfo& f = bars->info[n & 7];
      if (f.tile < 0) break;
      if ((n & 1) != wg) continue;
      const int i = f.tile * a.Qn + qi;
      const bool valid = g < a.G && i < a.N_Q;
      const int bit = a.Qn >= 32 ? (qi & 31) : ((f.tile * a.Qn) & 31) + qi;
      const bool on = valid && ((f.w[(qi >> 5) & 3] >> bit) & 1u);
      const int lim = on ? sp_last(i, nk, a.N_Q, a.causal) - blk0 * kSpBlock : -1;
      const float2 rv =
          on ? __ldg(a.rows + (size_t)(b * a.H + f.p * a.G + g) * a.N_Q + i) : make_float2(0.f, 0.f);
      const float nl = -rv.x, nd = -rv.y;
      const uint32_t ph = (n >> 1) & 1;
      if (!mbar_wait(smem_u32(&bars->s_full[wg]), ph)) { ok = false; break; }
      tc_fence_after();
      uint32_t v[64], p[16], d[16];
      tmem_ld_2x32_wait(ts + 32 * half, ts + 64 + 32 * half, v);
      sp_ds<true>(v, c, nl, nd, lim - 32 * half, d, p);
      // The buffer's last products (step n - NP's) have to be complete. With one buffer the other
      // parity's warps wait on the same barrier; step n - 1's products are at most one phase
      // ahead, since step n + 1's need this step's P and dS.
      if (n >= C::NP &&
          !mbar_wait(smem_u32(&bars->ds_empty[C::NP == 2 ? wg : 0]), ((n / C::NP) - 1) & 1)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        const uint32_t at = prow + (((4 * half + ch) ^ (r & 7)) << 4);
        st_shared_v4(at, p[4 * ch], p[4 * ch + 1], p[4 * ch + 2], p[4 * ch + 3]);
        st_shared_v4(at + C::PT, d[4 * ch], d[4 * ch + 1], d[4 * ch + 2], d[4 * ch + 3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->ds_full[wg]));
    }
    if (ok && !mbar_wait(smem_u32(&bars->acc_full), 0)) ok = false;
    if (!ok) {
      atomicOr(&g_skl_error, 2u);
      *abort_flag = 1;
    }
    tc_fence_after();
    // Parity 0 writes dV, parity 1 dK, each warp 32 keys: lane = d, columns = keys. For d = 64
    // dV is on lanes 0-63 and dK on lanes 64-127 of the stacked products.
    const int col = D == 128 ? r : (wg == 0 ? r : r - 64);
    const bool mine = D == 128 || (wg == 0 ? quarter < 2 : quarter >= 2);
    if (ok && mine) {
      const float f = wg == 0 ? 1.f : a.scale;
      __nv_bfloat16* dst = wg == 0 ? a.dv : a.dk;
      float* part = reinterpret_cast<float*>(smem + C::OFF_Q);
      uint32_t v[32];
      if (n > 0) tmem_ld_32_wait(tmem + lane_off + (wg == 0 ? C::TM_DV : C::TM_DK) + 32 * half, v);
      if (a.kv_splits > 1) {  // fp32 parts [dV, dK][64 keys][D] over the Q and dO buffers
#pragma unroll
        for (int k = 0; k < 32; ++k)
          part[(wg * 64 + 32 * half + k) * D + col] = n > 0 ? __uint_as_float(v[k]) : 0.f;
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int key = blk0 * kSpBlock + 32 * half + k;
          if (key < a.N_K)
            dst[((size_t)kv * a.N_K + key) * D + col] =
                __float2bfloat16_rn(n > 0 ? __uint_as_float(v[k]) * f : 0.f);
        }
      }
    }
  } else if (warp == 16) {
    const uint64_t keep = l2_policy_evict_last();
    if (lane == 0) {
      const uint32_t kf = smem_u32(&bars->k_full);
      mbar_arrive_expect_tx(kf, 2 * C::SLOT);
      for (int blk = 0; blk < D / 64; ++blk) {
        tma_load_3d(sb + blk * (64 * 128), &map_k, kf, blk * 64, blk0 * kSpBlock, kv, keep);
        tma_load_3d(sb + C::OFF_V + blk * (64 * 128), &map_v, kf, blk * 64, blk0 * kSpBlock, kv,
                    keep);
      }
    }
    // The tiles of every pack whose word column lists this block, in turn for a cluster's CTAs; the
    // end is a step without a tile.
    const int iws = (a.N_Q + 31) >> 5;
    bool ok = true;
    int n = 0, turn = 0, p = p0, base = -32;
    uint32_t nz = 0u, w[4] = {0u, 0u, 0u, 0u};
    for (;;) {
      int tile = -1;
      uint32_t u[4] = {0u, 0u, 0u, 0u};
      while (tile < 0) {
        if (nz == 0u) {
          base += 32;
          if (base >= a.n_tiles) {
            base = 0;
            ++p;
          }
          if (p >= p0 + ppk) break;
          const uint32_t* col =
              a.mask + (size_t)(b * a.Hsel + p / (a.P / a.Hsel)) * iws * a.NB + blk0;
          const int q0 = (base + lane) * a.Qn, iw = q0 >> 5;
          const uint32_t tmask = a.Qn >= 32 ? 0xffffffffu : ((1u << a.Qn) - 1u) << (q0 & 31);
          const int nw = base + lane >= a.n_tiles ? 0 : (a.Qn <= 32 ? 1 : min(a.Qn >> 5, iws - iw));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = k < nw ? __ldg(col + (size_t)(iw + k) * a.NB) & tmask : 0u;
          nz = __ballot_sync(0xffffffffu, (w[0] | w[1] | w[2] | w[3]) != 0u);
          continue;
        }
        const int pos = __ffs(nz) - 1;
        nz &= nz - 1;
        const bool mine = turn == split;
        turn = turn + 1 == a.kv_splits ? 0 : turn + 1;
        if (mine) {
          tile = base + pos;
#pragma unroll
          for (int k = 0; k < 4; ++k) u[k] = __shfl_sync(0xffffffffu, w[k], pos);
        }
      }
      if (lane == 0) {
        // Entry n & 7 was last read for step n - 8; loads run at most NQ steps ahead of the
        // products, which wait for the warps of their step.
        SpTileInfo& f = bars->info[n & 7];
        f.tile = tile;
        f.p = p;
#pragma unroll
        for (int k = 0; k < 4; ++k) f.w[k] = u[k];
        mbar_arrive(smem_u32(&bars->info_full[n & 7]));
        const int sq = n % C::NQ, sd = n % C::ND, head = b * a.H + p * a.G;
        const uint32_t qf = smem_u32(&bars->q_full[sq]);
        ok = mbar_wait(smem_u32(&bars->q_empty[sq]), ((n / C::NQ) & 1) ^ 1);
        if (ok && tile < 0) {
          mbar_arrive(qf);  // the MMA thread learns of the end from q_full alone
        } else if (ok) {
          mbar_arrive_expect_tx(qf, rows * D * 2);
          for (int blk = 0; blk < D / 64; ++blk)
            tma_load_3d(sb + C::off_q(n) + blk * (128 * 128), &map_q, qf, blk * 64, tile * a.Qn,
                        head, keep);
          ok = mbar_wait(smem_u32(&bars->do_empty[sd]), ((n / C::ND) & 1) ^ 1);
          if (ok) {
            const uint32_t df = smem_u32(&bars->do_full[sd]);
            mbar_arrive_expect_tx(df, rows * D * 2);
            for (int blk = 0; blk < D / 64; ++blk)
              tma_load_3d(sb + C::off_do(n) + blk * (128 * 128), &map_do, df, blk * 64,
                          tile * a.Qn, head, keep);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (tile < 0 || !ok) break;
      ++n;
    }
    if (lane == 0) mbar_wait(smem_u32(&bars->k_full), 0);
    if (!ok && lane == 0) {
      atomicOr(&g_skl_error, 2u);
      *abort_flag = 1;
      // Of step n itself Q may not have been asked for; then its wait runs out.
      for (int j = max(0, n + 1 - C::NQ); j <= n; ++j)
        mbar_wait(smem_u32(&bars->q_full[j % C::NQ]), (j / C::NQ) & 1);
      for (int j = max(0, n - C::ND); j < n; ++j)
        mbar_wait(smem_u32(&bars->do_full[j % C::ND]), (j / C::ND) & 1);
    }
  } else if (elect_one()) {
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t lk = sdesc_lo(sb, 16), lv = sdesc_lo(sb + C::OFF_V, 16);
    const uint32_t lp0 = sdesc_lo(sb + C::OFF_P, 128 * 128);
    bool ok = mbar_wait(smem_u32(&bars->k_full), 0);
    // S and dP of step n: 1, no such step: 0, a wait ran out: -1. Score buffer n & 1 was last
    // read for step n - 2, whose P and dS this thread has seen.
    auto scores = [&](int n) -> int {
      if (!mbar_wait(smem_u32(&bars->q_full[n % C::NQ]), (n / C::NQ) & 1)) return -1;
      if (bars->info[n & 7].tile < 0) return 0;  // written before the arrival on q_full
      tc_fence_after();
      const uint32_t ds = tmem + C::TM_S + 128 * (n & 1);
      const uint32_t lq = sdesc_lo(sb + C::off_q(n), 16), ldo = sdesc_lo(sb + C::off_do(n), 16);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16_ss_lh(ds, lq + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                        lk + (((kk >> 2) * (64 * 128) + (kk & 3) * 32) >> 4), hi, idesc_s, kk > 0);
      if (!mbar_wait(smem_u32(&bars->do_full[n % C::ND]), (n / C::ND) & 1)) return -1;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16_ss_lh(ds + 64, ldo + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                        lv + (((kk >> 2) * (64 * 128) + (kk & 3) * 32) >> 4), hi, idesc_dp, kk > 0);
      umma_commit(smem_u32(&bars->s_full[n & 1]));
      return 1;
    };
    int ahead = 0;  // steps whose scores have been issued
    bool more = ok;
    auto reach = [&](int n) {
      while (ok && more && ahead <= n) {
        const int got = scores(ahead);
        if (got < 0) ok = false;
        if (got == 0) more = false;
        if (got > 0) ++ahead;
      }
    };
    reach(1);
    for (int n = 0; ok && n < ahead; ++n) {
      if (!(ok = mbar_wait(smem_u32(&bars->ds_full[n & 1]), (n >> 1) & 1))) break;
      tc_fence_after();
      // A = dO (d = 64: the stacked [dO | Q]) and Q, B = P and dS; 16 rows a step, both operands
      // row-contracted (MN-major).
      const uint32_t ldo = sdesc_lo(sb + C::off_do(n), 128 * 128);
      const uint32_t lq = D == 128 ? sdesc_lo(sb + C::off_q(n), 128 * 128) : ldo;
      const uint32_t lp = lp0 + (C::NP == 2 ? (n & 1) * (2 * C::PT >> 4) : 0);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_bf16_ss_lh(tmem + C::TM_DV, ldo + kk * (2048 >> 4), lp + kk * (2048 >> 4), hi,
                        idesc_acc, (n > 0 || kk > 0) ? 1u : 0u);
      if (D == 128) umma_commit(smem_u32(&bars->do_empty[n % C::ND]));
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_bf16_ss_lh(tmem + C::TM_DK, lq + kk * (2048 >> 4),
                        lp + (C::PT >> 4) + kk * (2048 >> 4), hi, idesc_acc,
                        (n > 0 || kk > 0) ? 1u : 0u);
      umma_commit(smem_u32(&bars->ds_empty[C::NP == 2 ? n & 1 : 0]));
      umma_commit(smem_u32(&bars->q_empty[n % C::NQ]));
      if (D != 128) umma_commit(smem_u32(&bars->do_empty[n % C::ND]));
      reach(n + 2);
    }
    umma_commit(smem_u32(&bars->acc_full));
    if (!ok) {
      atomicOr(&g_skl_error, 2u);
      *abort_flag = 1;
    }
    mbar_wait(smem_u32(&bars->acc_full), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
  if (a.kv_splits > 1) {
    // Sums of the cluster's parts in rank order, one row (key of dV or dK) per warp.
    __syncwarp();
    cluster_sync();
    for (int r = split + warp * a.kv_splits; r < 128; r += 18 * a.kv_splits) {
      const int key = blk0 * kSpBlock + (r & 63);
      if (key >= a.N_K) continue;
      const float f = r < 64 ? 1.f : a.scale;
      __nv_bfloat16* dst = (r < 64 ? a.dv : a.dk) + ((size_t)kv * a.N_K + key) * D;
#pragma unroll
      for (int k = lane * 2; k < D; k += 64) {
        float x = 0.f, y = 0.f;
        for (int p = 0; p < a.kv_splits; ++p) {
          const float2 v = ld_cluster_f32x2(cluster_map(sb + C::OFF_Q + (r * D + k) * 4, p));
          x += v.x;
          y += v.y;
        }
        *reinterpret_cast<uint32_t*>(dst + k) = pack_bf16x2(x * f, y * f);
      }
    }
    __syncwarp();
    cluster_sync();  // another CTA may still be reading this one's parts
  }
}

}  // namespace skl
