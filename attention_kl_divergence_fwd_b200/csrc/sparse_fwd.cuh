// sparse_fwd.cuh - attention over selected key blocks, forward (tcgen05 + TMEM + TMA).
//
//   out[i] = sum_j p_ij v_j,  p_ij = exp(s_ij - LSE_i),  s_ij = scale <q_i, k_j>,
//   LSE_i = log sum_j exp(s_ij),  j over the allowed keys of the blocks that i lists.
//
// CTA = one 128-row tile of packed query heads (sparse_common.cuh); it walks the blocks of its
// union. Per block:
//   S = Q K^T into one of two TMEM score buffers; one thread per row turns its 64 scores into
//   probabilities against the row's reference m and writes them back over the scores as bf16;
//   O += P V with P read from TMEM; S of the next but one block follows at once.
// Two groups of four warps take alternate blocks, so one block's exponentials run under the other
// block's products and loads. They share m, handed from block to block through shared memory.
// The sums are exact for any reference, so a block is folded against m as it stands; only a
// row's first block, partial blocks and a block whose sum reaches 2^64 take its maximum first,
// and raise m, with a rescale of O in TMEM, when it exceeds m by 2^8. Each group keeps its own
// part of the row sum.
// P is rounded to bf16 for the tensor core (relative error at most 2^-8 each, the same as the
// output's own rounding); the row sums, references and O stay in fp32.
// A CTA takes 256 TMEM columns and about 100 KB of shared memory: two CTAs share an SM, which
// hides the start and end of one behind the other.
// `splits` > 1: the tile's list is dealt to the CTAs of a cluster by rank; their normalised
// outputs and log-sum-exps are joined through distributed shared memory, so that a single
// token is one launch and no partial result leaves the chip.
// QUAD: tiles of at most 32 rows, four copies, each warp a quarter of the block's keys (sp_quad);
// the four quarters are joined like splits.
//
// Bound by the chain of a block: S (N = 64 with both operands in shared memory: 384 cycles), the
// fold (600 to 900), O += P V (256) and the hand-overs between them, about 2000 cycles per block and
// CTA. No single unit is full (tensor pipe 640 and exponentials 512 of about 1040 cycles per block
// and SM, issue slots 41 %); without exponentials a prompt takes 6 % less, with half of the S products
// 6 %, without loads 2 %.
// Measured on a B200, kernel only: 32 heads over 8, 16384 tokens, 32 blocks per query: 630 us
// (818 TFLOP/s of the queries' own blocks, 1090 of the tiles' unions); one token of 32 sequences,
// 16 blocks: 29.4 us (4.6 TB/s); one token of a 65536-key sequence, 32 blocks: 10.4 us.
//
// Warps: 0-7 softmax (warp w: lane quarter w & 3, blocks of parity w >> 2), 8 producer (scans the
// bit matrix, TMA), 9 MMA + TMEM.
#pragma once

#include "sparse_common.cuh"

namespace skl {

constexpr int kSpThreads = 320;

// One block as the producer announces it: which (-1 = end), and which queries list it.
struct SpBlockInfo {
  int c;
  uint32_t w[4];
};

template <int D>
struct SpFwdCfg {
  static constexpr int BM = 128;
  static constexpr int QBYTES = BM * D * 2;
  static constexpr int SLOT = 64 * D * 2;             // one K (or V) block
  static constexpr int NST = D == 128 ? 2 : 4;        // slots each of K and V
  static constexpr int OFF_K = QBYTES;
  static constexpr int OFF_V = OFF_K + NST * SLOT;
  static constexpr int OFF_BAR = OFF_V + NST * SLOT;
  static constexpr int BAR_BYTES = 4352;
  static constexpr int SMEM = OFF_BAR + BAR_BYTES;
  static constexpr int TM_S = 0;    // two buffers of 64 columns of scores, P over the first 32
  static constexpr int TM_O = 128;  // D columns
  static constexpr int TM_COLS = 256;
  static_assert(2 * (SMEM + 1024) <= 233472, "two CTAs per SM");
};

struct SpFwdBars {
  uint64_t q_full;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t info_full[8];
  uint64_t s_full[2], p_full[2], o_full;
  uint64_t m_pass[4][2];  // per lane quarter: the reference after an even / odd block is there
  uint64_t pair[4];       // the two warps of a lane quarter at the end
  uint32_t tmem_base;
  int abort_flag;
  SpBlockInfo info[8];
  float l2[128];       // base-2 log-sum-exps of the partial rows
  float m[2][128];     // the rows' references after an even / odd block
  float ml[2][2][128];  // the groups' final references and sums
};
static_assert(sizeof(SpFwdBars) <= SpFwdCfg<128>::BAR_BYTES, "barrier block");

// Sets the rows from `first` of a [D/64][64][64] block to zero: with a padded cache the rows
// past nk hold whatever the cache held, and 0 * NaN would reach the products.
template <int D>
__device__ __forceinline__ void sp_zero_tail(uint8_t* buf, int first, int tid, int nthreads) {
  const int per = (kSpBlock - first) * 8;  // 16-byte pieces
  for (int e = tid; e < per * (D / 64); e += nthreads)
    *reinterpret_cast<uint4*>(buf + (e / per) * (64 * 128) + first * 128 + (e % per) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
}

// 2^(v c + bias) of 32 scores as bf16 pairs, and their sum (two packed partial sums). All on the
// exponential unit: the loop is bound by issue slots, and a share of polynomial exponentials as in
// the divergence's forward makes it slower (prompt of 16384 tokens: 660 us without, 686, 718 and
// 737 us with 1, 2 and 3 of 8 pairs).
__device__ __forceinline__ void sp_exp32(const uint32_t (&v)[32], uint64_t c2, uint64_t b2,
                                         uint64_t& acc0, uint64_t& acc1, uint32_t (&p)[16]) {
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    float x0, x1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, b2), x0, x1);
    x0 = ex2_approx(x0);
    x1 = ex2_approx(x1);
    if (k & 2)
      acc1 = f2_add(acc1, f2_pack(x0, x1));
    else
      acc0 = f2_add(acc0, f2_pack(x0, x1));
    p[k >> 1] = pack_bf16x2(x0, x1);
  }
}

// Producer's walk over the blocks of a tile's union, whole warp, in ascending order; of a cluster's
// CTAs each takes every `splits`-th block. next() returns the block (-1 at the end) and its words;
// it is called in one place, so that its state stays in registers. The words are read with ordinary
// loads: the forward starts beside the kernel that writes them, and only its wait for that kernel
// (grid_wait_previous) orders the two. A read through the read-only path (__ldg) would promise
// memory that nothing writes while this kernel runs, and could be moved ahead of the wait.
struct SpScan {
  int base = -32, turn = 0;
  uint32_t nz = 0u, w[4] = {0u, 0u, 0u, 0u};

  __device__ __forceinline__ int next(const SparseArgs& a, const SpTile& t, int split, int lane,
                                      uint32_t (&u)[4]) {
    const uint32_t tmask = a.Qn >= 32 ? 0xffffffffu : ((1u << a.Qn) - 1u) << t.bit0;
    for (;;) {
      while (nz == 0u) {
        base += 32;
        if (base >= a.NB) return -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = 0u;
          if (base + lane < a.NB && k < t.nwords)
            w[k] = ld_global_u32(t.words + (size_t)k * a.NB + base + lane) & tmask;
        }
        nz = __ballot_sync(0xffffffffu, (w[0] | w[1] | w[2] | w[3]) != 0u);
      }
      const int pos = __ffs(nz) - 1;
      nz &= nz - 1;
      const bool mine = turn == split;
      turn = turn + 1 == a.splits ? 0 : turn + 1;
      if (mine) {
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = __shfl_sync(0xffffffffu, w[k], pos);
        return base + pos;
      }
    }
  }
};

// One row from `srcs` partial ones (at most 8), each normalised by its own sum: out =
// sum_s 2^(l_s - L) o_s, L = log2 sum_s 2^(l_s). Source s's row and log-sum-exp are at the shared
// addresses row_at(s) and l2_at(s) (of any CTA of the cluster). One warp; lane holds the columns
// 2 lane, 2 lane + 1 of every 64. All reads are in flight at once.
template <int D, typename RowAt, typename L2At>
__device__ __forceinline__ float sp_join_row(int srcs, int lane, RowAt row_at, L2At l2_at,
                                             float (&acc)[D / 32]) {
  const float mine = lane < srcs ? ld_cluster_f32(l2_at(lane)) : -INFINITY;
  float2 o[8][D / 64];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      if (e < srcs) o[e][k] = ld_cluster_f32x2(row_at(e) + k * 256 + lane * 8);
  }
  float mx = mine;
#pragma unroll
  for (int k = 4; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  mx = __shfl_sync(0xffffffffu, mx, 0);
  float w = mx > -INFINITY ? ex2_approx(mine - mx) : 0.f, tot = w;
#pragma unroll
  for (int k = 4; k > 0; k >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, k);
  tot = __shfl_sync(0xffffffffu, tot, 0);
  w *= tot > 0.f ? 1.f / tot : 0.f;
#pragma unroll
  for (int k = 0; k < D / 32; ++k) acc[k] = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float ws = __shfl_sync(0xffffffffu, w, e);
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      if (e < srcs) {
        acc[2 * k] = fmaf(ws, o[e][k].x, acc[2 * k]);
        acc[2 * k + 1] = fmaf(ws, o[e][k].y, acc[2 * k + 1]);
      }
  }
  return tot > 0.f ? mx + log2f(tot) : -INFINITY;
}

// Joins the partial rows of this CTA's four quarters (QUAD), then those of the cluster's CTAs:
// row r is joined by CTA r % splits. Slot s of a CTA is at stage + s * (D + 4) floats.
template <int D, bool QUAD>
__device__ __forceinline__ void sp_join(const SparseArgs& a, const SpTile& t, uint32_t stage,
                                        float* l2, int split, int warp, int lane) {
  const int rows = a.Qn * a.G;
  const uint32_t l2a = smem_u32(l2);
  float acc[D / 32];
  auto write = [&](int r, float l) {
    const int g = r / a.Qn, i = t.q0 + r - g * a.Qn;
    if (i >= a.N_Q) return;
    const size_t row = (size_t)(t.h0 + g) * a.N_Q + i;
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      *reinterpret_cast<uint32_t*>(a.out + row * D + k * 64 + lane * 2) =
          pack_bf16x2(acc[2 * k], acc[2 * k + 1]);
    if (lane == 0 && a.lse) a.lse[row] = l * 0.69314718055994530942f;
  };
  if (QUAD && warp < 8) {
    for (int r = warp; r < rows; r += 8) {
      const float l = sp_join_row<D>(
          4, lane, [&](int s) { return stage + (s * 32 + r) * (D + 4) * 4; },
          [&](int s) { return l2a + (s * 32 + r) * 4; }, acc);
      if (a.splits == 1) {
        write(r, l);
        continue;
      }
      float* dst = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(l2) + (stage - l2a)) +
                   r * (D + 4);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
        *reinterpret_cast<float2*>(dst + k * 64 + lane * 2) = make_float2(acc[2 * k], acc[2 * k + 1]);
      if (lane == 0) l2[r] = l;
    }
  }
  if (a.splits == 1) return;
  __syncwarp();
  cluster_sync();
  if (warp < 8) {
    for (int r = split + warp * a.splits; r < rows; r += 8 * a.splits) {
      const float l = sp_join_row<D>(
          a.splits, lane, [&](int s) { return cluster_map(stage + r * (D + 4) * 4, s); },
          [&](int s) { return cluster_map(l2a + r * 4, s); }, acc);
      write(r, l);
    }
  }
  __syncwarp();
  cluster_sync();  // another CTA may still be reading this one's rows
}

template <int D, bool QUAD>
__global__ void __launch_bounds__(kSpThreads, 2)
streamkl_sparse_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v, const SparseArgs a,
                           const uint32_t idesc_s, const uint32_t idesc_o) {
  using C = SpFwdCfg<D>;
  constexpr int NST = C::NST;
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

  if (warp == 8) {
    if (lane == 0) {
      tma_prefetch_desc(&map_q);
      tma_prefetch_desc(&map_k);
      tma_prefetch_desc(&map_v);
      bars->abort_flag = 0;
    }
    constexpr int P_FULL = offsetof(SpFwdBars, p_full) / 8, PAIR = offsetof(SpFwdBars, pair) / 8;
    sp_init_barriers(&bars->q_full, PAIR + 4, kSpThreads, lane, [](int i) {
      return i == P_FULL || i == P_FULL + 1 ? 4 : (i >= PAIR ? 2 : 1);
    });
  } else {
    if (warp == 9) {
      tmem_alloc(smem_u32(&bars->tmem_base), C::TM_COLS);
      tmem_relinquish();
    }
    tc_fence_before();
    named_bar_sync(15, kSpThreads);
    tc_fence_after();
  }
  const uint32_t tmem = bars->tmem_base;

  if (warp < 8) {
    // ------------------------------------------------------------- softmax rows
    const int quarter = warp & 3, grp = warp >> 2;
    const int r = QUAD ? lane : quarter * 32 + lane, slot = quarter * 32 + lane;
    const int g = r / a.Qn, qi = r - g * a.Qn, i = t.q0 + qi;
    const bool valid = g < a.G && i < a.N_Q;
    const int last = valid ? sp_last(i, t.nk, a.N_Q, a.causal) : -1;
    const int wi = (qi >> 5) & 3, bi = a.Qn >= 32 ? (qi & 31) : t.bit0 + qi;
    const bool live = __any_sync(0xffffffffu, valid);
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_off + C::TM_S + 64 * grp, to = tmem + lane_off + C::TM_O;
    const float c = a.c;
    // Block that holds the end of a padded sequence (rows of it past nk are not keys), or none.
    const int c_end = (t.nk & (kSpBlock - 1)) != 0 && t.nk < a.N_K ? t.nk / kSpBlock : -1;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int n = 0;
    for (;; ++n) {
      if (!mbar_wait(smem_u32(&bars->info_full[n & 7]), (n >> 3) & 1)) { ok = false; break; }
      const SpBlockInfo& f = bars->info[n & 7];
      const int blk = f.c;
      if (blk < 0) break;
      if ((n & 1) != grp) continue;
      // Last key of the block that this row reads, -1 or less for none.
      const int lim = (f.w[wi] >> bi) & 1u ? last - blk * kSpBlock : -1;
      if (!mbar_wait(smem_u32(&bars->s_full[grp]), (n >> 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const bool at_end = blk == c_end;
      if (at_end) {
        // V's product with this block waits for p_full below, and its copy is the next phase of
        // v_full: the product of block n - NST, which freed the slot, is complete (S(n) is,
        // and products complete in order).
        if (!mbar_wait(smem_u32(&bars->v_full[n % NST]), (n / NST) & 1)) { ok = false; break; }
        sp_zero_tail<D>(smem + C::OFF_V + (n % NST) * C::SLOT, t.nk & (kSpBlock - 1),
                        threadIdx.x & 127, 128);
        fence_async_smem();
      }
      // Fast way: probabilities against the reference at hand, without the block's maximum first.
      // It holds when no row's partial block or first block is among them, the row's sum stays
      // below 2^64 (no score is far above the reference) and the other group has not raised it.
      uint64_t acc0 = f2_pack(0.f, 0.f), acc1 = acc0;
      const uint64_t c2 = f2_pack(c, c);
      float m0 = -INFINITY;  // the reference after block n - 1
      bool have_m0 = n == 0;
      // Slots alternate by block; a slot's next value needs one from the other group in between.
      auto reference = [&]() -> bool {
        if (have_m0) return true;
        have_m0 = true;
        if (!mbar_wait(smem_u32(&bars->m_pass[quarter][(n - 1) & 1]), ((n - 1) >> 1) & 1))
          return false;
        m0 = bars->m[(n - 1) & 1][slot];
        return true;
      };
      auto publish = [&](float m1) {
        bars->m[n & 1][slot] = m1;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->m_pass[quarter][n & 1]));
      };
      bool done = false;
      if constexpr (!QUAD) {
        if (n == 1) {
          if (!reference()) { ok = false; break; }
          m = m0;
        }
        if (live && n > 0 && !at_end &&
            __all_sync(0xffffffffu, lim < 0 || (lim >= 63 && m > -INFINITY))) {
          uint32_t v[32], p0[16], p1[16];  // 32 scores at a time: registers are short
          const uint64_t b2 = f2_pack(-m, -m);
          tmem_ld_32_wait(ts, v);
          sp_exp32(v, c2, b2, acc0, acc1, p0);
          tmem_ld_32_wait(ts + 32, v);
          sp_exp32(v, c2, b2, acc0, acc1, p1);
          float s0, s1;
          f2_unpack(f2_add(acc0, acc1), s0, s1);
          float sum = s0 + s1;
          if (__any_sync(0xffffffffu, lim < 0)) {  // rows that do not list the block
            if (lim < 0) sum = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              p0[k] = lim < 0 ? 0u : p0[k];
              p1[k] = lim < 0 ? 0u : p1[k];
            }
          }
          if (!reference()) { ok = false; break; }
          if (__all_sync(0xffffffffu, m0 == m && sum < 0x1p64f)) {
            publish(m);
            // P goes over the scores this thread has read.
            tmem_st_16(ts, p0);
            tmem_st_16(ts + 16, p1);
            l += sum;
            done = true;
          }
        }
      }
      if (!done) {
        constexpr int NC = QUAD ? 16 : 32;  // scores at a time
        uint32_t v[NC];
        float mx = -INFINITY;
        // Blocks are read whole or not at all except at the causal diagonal and the sequence's
        // end; only those mask single scores (the end's scores may be NaN).
        const bool single = at_end || __any_sync(0xffffffffu, lim >= 0 && lim < 63);
        auto mask = [&](int first) {
#pragma unroll
          for (int k = 0; k < NC; ++k)
            if (first + k > lim) v[k] = 0xff800000u;  // -inf
        };
        if constexpr (QUAD) {
          tmem_ld_16_wait(ts + 16 * quarter, v);
          mask(16 * quarter);
#pragma unroll
          for (int k = 0; k < 16; ++k) mx = fmaxf(mx, __uint_as_float(v[k]));
        } else if (live) {
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            tmem_ld_32_wait(ts + h, v);
            if (single) mask(h);
            mx = fmaxf(mx, max_tree32<false>(v, 0, 31));
          }
          if (lim < 0) mx = -INFINITY;
        }
        const float ms = mx == -INFINITY ? -INFINITY : mx * c;
        if (!reference()) { ok = false; break; }
        const bool raise = ms > m0 + 8.f || (m0 == -INFINITY && ms > -INFINITY);
        const float m1 = raise ? ms : m0;
        publish(m1);
        if (m1 != m) {
          l *= ex2_approx(m - m1);  // m = -inf: l = 0
          m = m1;
        }
        if (n > 0 && __any_sync(0xffffffffu, raise)) {
          // O *= 2^(m0 - m1) once it holds every product before this block's.
          if (!mbar_wait(smem_u32(&bars->v_empty[(n - 1) % NST]), ((n - 1) / NST) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f0 = raise ? ex2_approx(m0 - m1) : 1.f;  // m0 = -inf: 0
#pragma unroll
          for (int k = 0; k < D; k += 8) {  // few registers: the scores are live
            uint32_t o[8];
            tmem_ld_8_wait(to + k, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
            tmem_st_8(to + k, o);
          }
        }
        acc0 = acc1 = f2_pack(0.f, 0.f);
        const float bias = lim < 0 ? -INFINITY : (m == -INFINITY ? 0.f : -m);
        const uint64_t b2 = f2_pack(bias, bias);
        if constexpr (QUAD) {
          uint32_t p[8], zero[8];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, b2), x0,
                      x1);
            x0 = ex2_approx(x0);
            x1 = ex2_approx(x1);
            acc0 = f2_add(acc0, f2_pack(x0, x1));
            p[k >> 1] = pack_bf16x2(x0, x1);
            zero[k >> 1] = 0u;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q == quarter)
              tmem_st_8(ts + 8 * q, p);
            else
              tmem_st_8(ts + 8 * q, zero);
          }
        } else if (live) {
          // P goes over scores that have been read: keys 0-31 over the columns 0-15.
          uint32_t p[16];
#pragma unroll
          for (int h = 0; h < 64; h += 32) {
            tmem_ld_32_wait(ts + h, v);
            if (single) mask(h);
            sp_exp32(v, c2, b2, acc0, acc1, p);
            tmem_st_16(ts + h / 2, p);
          }
        }
        float s0, s1;
        f2_unpack(f2_add(acc0, acc1), s0, s1);
        l += s0 + s1;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[grp]));
    }
    if (ok && !mbar_wait(smem_u32(&bars->o_full), 0)) ok = false;
    tc_fence_after();
    // The two groups' sums, at the later of their references.
    bars->ml[grp][0][slot] = m;
    bars->ml[grp][1][slot] = l;
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&bars->pair[quarter]));
    if (ok && !mbar_wait(smem_u32(&bars->pair[quarter]), 0)) ok = false;
    if (!ok) {
      atomicOr(&g_skl_error, 1u);
      *abort_flag = 1;
    }
    {
      const float ma = bars->ml[0][0][slot], mb = bars->ml[1][0][slot];
      m = fmaxf(ma, mb);
      l = 0.f;
      if (ma > -INFINITY) l = bars->ml[0][1][slot] * ex2_approx(ma - m);
      if (mb > -INFINITY) l += bars->ml[1][1][slot] * ex2_approx(mb - m);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const float l2 = l > 0.f ? m + log2f(l) : -INFINITY;
    const bool some = n > 0;  // else O was never written
    const bool parts = QUAD || a.splits > 1;
    // The copies and products of this CTA are done; its buffers take the partial rows.
    if (parts && !mbar_wait(smem_u32(&bars->q_full), 0)) ok = false;
    if (parts && grp == 0) bars->l2[slot] = ok && valid ? l2 : -INFINITY;
    const size_t row = (size_t)(t.h0 + g) * a.N_Q + i;
    if (live && ok) {
#pragma unroll
      for (int k0 = 0; k0 < D / 2; k0 += 32) {  // half of the columns per group
        const int k = grp * (D / 2) + k0;
        uint32_t o[32];
        if (some) tmem_ld_32_wait(to + k, o);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          o[e] = some && l > 0.f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
        if (!valid) {
          // no row to write
        } else if (parts) {
          float* dst = reinterpret_cast<float*>(smem) + slot * (D + 4) + k;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else {
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
      if (!parts && valid && grp == 0 && a.lse) a.lse[row] = l2 * 0.69314718055994530942f;
    }
  } else if (warp == 8) {
    // ---------------------------------------------------- producer (whole warp scans)
    if (lane == 0) {
      const uint32_t qb = smem_u32(&bars->q_full);
      mbar_arrive_expect_tx(qb, (QUAD ? 4 : 1) * a.Qn * a.G * D * 2);
      for (int blk = 0; blk < D / 64; ++blk)
        for (int copy = 0; copy < (QUAD ? 4 : 1); ++copy)
          tma_load_3d(sb + blk * (C::BM * 128) + copy * (32 * 128), &map_q, qb, blk * 64, t.q0,
                      t.h0, l2_policy_evict_first());
    }
    // K and V of a tile that is the only one of its pack are read once (tokens: 31.0 -> 29.4 us).
    const uint64_t keep = a.n_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
    // One query: its list becomes a bitmap over the blocks (repeats fall away) and that the
    // ascending list of this CTA's share, both in rows of the Q buffer that the copies of the
    // pack's at most 16 rows leave unused: 16-31 (2 KB: 16384 blocks) and 48-63 (512 entries).
    int* list = reinterpret_cast<int*>(smem + 48 * 128);
    int listed = 0;
    if (a.direct) {
      uint32_t* bits = reinterpret_cast<uint32_t*>(smem + 16 * 128);
      const int sel = t.b * a.Hsel + t.p / (a.P / a.Hsel);
      const int* idx = a.idx + (size_t)sel * a.topk;
      const int lastkey = sp_last(0, t.nk, 1, a.causal);
      const int top = lastkey < 0 ? -1 : lastkey / kSpBlock;
      const int words = (a.NB + 31) / 32;
      for (int w = lane; w < words; w += 32) bits[w] = 0u;
      __syncwarp();
      for (int e = lane; e < a.topk; e += 32) {
        const int c = __ldg(idx + e);
        if (c >= 0 && c <= top) atomicOr(&bits[c >> 5], 1u << (c & 31));
      }
      __syncwarp();
      int before = 0;  // blocks of earlier words
      for (int w0 = 0; w0 < words; w0 += 32) {
        uint32_t mine = w0 + lane < words ? bits[w0 + lane] : 0u;
        int upto = __popc(mine);
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, upto, k);
          upto += lane >= k ? x : 0;
        }
        for (int rank = before + upto - __popc(mine); mine != 0u; ++rank, mine &= mine - 1)
          if (rank % a.splits == split) list[rank / a.splits] = (w0 + lane) * 32 + __ffs(mine) - 1;
        before += __shfl_sync(0xffffffffu, upto, 31);
      }
      listed = (before - split + a.splits - 1) / a.splits;  // before >= 0, split < splits
      __syncwarp();
    } else {
      grid_wait_previous();  // launched beside the end of the kernel that builds the bit matrix
    }
    // Step n: announces the next block and loads its K, then V of the step before: K's slot is free
    // as soon as S(n - NST) is done, V's only after the product of step n - 1 - NST, and waiting
    // for that first would hold K back. The end is a step without a block.
    SpScan scan;
    bool ok = true;
    int n = 0, c_prev = -1;
    for (;;) {
      uint32_t u[4] = {0u, 0u, 0u, 0u};
      int c;
      if (a.direct) {
        c = n < listed ? list[n] : -1;
        u[0] = 1u;
      } else {
        c = scan.next(a, t, split, lane, u);
      }
      if (lane == 0) {
        // Entry n & 7 was last read for step n - 8: loads run at most NST + 3 steps ahead of
        // the products, which wait for every softmax warp.
        SpBlockInfo& f = bars->info[n & 7];
        f.c = c;
#pragma unroll
        for (int k = 0; k < 4; ++k) f.w[k] = u[k];
        mbar_arrive(smem_u32(&bars->info_full[n & 7]));
        const uint32_t kf = smem_u32(&bars->k_full[n % NST]);
        ok = mbar_wait(smem_u32(&bars->k_empty[n % NST]), ((n / NST) & 1) ^ 1);
        if (ok && c >= 0) {
          mbar_arrive_expect_tx(kf, C::SLOT);
          for (int blk = 0; blk < D / 64; ++blk)
            tma_load_3d(sb + C::OFF_K + (n % NST) * C::SLOT + blk * (64 * 128), &map_k, kf, blk * 64,
                        c * kSpBlock, t.kv, keep);
        } else if (ok) {
          mbar_arrive(kf);  // the MMA thread learns of the end from k_full alone
        }
        if (ok && n > 0) {
          const int st = (n - 1) % NST;
          const uint32_t vf = smem_u32(&bars->v_full[st]);
          ok = mbar_wait(smem_u32(&bars->v_empty[st]), (((n - 1) / NST) & 1) ^ 1);
          if (ok) {
            mbar_arrive_expect_tx(vf, C::SLOT);
            for (int blk = 0; blk < D / 64; ++blk)
              tma_load_3d(sb + C::OFF_V + st * C::SLOT + blk * (64 * 128), &map_v, vf, blk * 64,
                          c_prev * kSpBlock, t.kv, keep);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (c < 0 || !ok) break;
      c_prev = c;
      ++n;
    }
    if (!ok && lane == 0) {
      atomicOr(&g_skl_error, 1u);
      *abort_flag = 1;
      // Let the copies in flight land before the CTA can exit (each wait is bounded).
      mbar_wait(smem_u32(&bars->q_full), 0);
      // Of step n itself K may not have been asked for; then its wait runs out.
      for (int j = max(0, n + 1 - NST); j <= n; ++j) {
        mbar_wait(smem_u32(&bars->k_full[j % NST]), (j / NST) & 1);
        if (j < n) mbar_wait(smem_u32(&bars->v_full[j % NST]), (j / NST) & 1);
      }
    }
    // With no block nothing else waits for the Q copy.
    if (lane == 0 && n == 0) mbar_wait(smem_u32(&bars->q_full), 0);
  } else if (elect_one()) {
    // ------------------------------------------------------------------ MMA issuer
    // Descriptors are a base per operand plus constants: this thread's instruction stream is on
    // the critical path.
    const uint32_t hi = sdesc_hi(1024);
    const uint32_t lq = sdesc_lo(sb, 16), lk0 = sdesc_lo(sb + C::OFF_K, 16);
    const uint32_t lv0 = sdesc_lo(sb + C::OFF_V, 64 * 128);
    bool ok = mbar_wait(smem_u32(&bars->q_full), 0);
    // Waits for K of step n: 1, no such step: 0, a wait ran out: -1. The entry was written before
    // the producer's arrival on k_full.
    auto keys = [&](int n) -> int {
      if (!mbar_wait(smem_u32(&bars->k_full[n % NST]), (n / NST) & 1)) return -1;
      return bars->info[n & 7].c < 0 ? 0 : 1;
    };
    // S of step n. The buffer's last P has been handed to a product issued before.
    auto scores = [&](int n) {
      const int st = n % NST;
      const uint32_t lk = lk0 + st * (C::SLOT >> 4), ds = tmem + C::TM_S + 64 * (n & 1);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16_ss_lh(ds, lq + (((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4),
                        lk + (((kk >> 2) * (64 * 128) + (kk & 3) * 32) >> 4), hi, idesc_s, kk > 0);
      umma_commit(smem_u32(&bars->s_full[n & 1]));
      umma_commit(smem_u32(&bars->k_empty[st]));
    };
    int ahead = 0;   // steps whose S has been issued
    int next = ok ? 1 : -1;  // whether there is a step `ahead` with its K landed
    for (; ahead < 2 && (next = next < 0 ? next : keys(ahead)) > 0; ++ahead) {
      tc_fence_after();
      scores(ahead);
    }
    for (int n = 0; next >= 0 && n < ahead; ++n) {
      const int st = n % NST;
      // Everything but P is awaited first, so that once P is there the products of this step
      // and S of the next but one go out back to back.
      if (next > 0 && (next = keys(n + 2)) < 0) break;
      if (!mbar_wait(smem_u32(&bars->v_full[st]), (n / NST) & 1) ||
          !mbar_wait(smem_u32(&bars->p_full[n & 1]), (n >> 1) & 1)) {
        next = -1;
        break;
      }
      tc_fence_after();
      // O += P V: A = P from TMEM, B = V [keys][d] MN-major, 16 keys per step.
      const uint32_t lv = lv0 + st * (C::SLOT >> 4), tp = tmem + C::TM_S + 64 * (n & 1);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_bf16_ts_lh(tmem + C::TM_O, tp + kk * 8, lv + kk * (2048 >> 4), hi, idesc_o,
                        (n > 0 || kk > 0) ? 1u : 0u);
      umma_commit(smem_u32(&bars->v_empty[st]));
      if (next > 0) {
        scores(n + 2);
        ++ahead;
      }
    }
    ok = next >= 0;
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
  if (QUAD || a.splits > 1) sp_join<D, QUAD>(a, t, sb, bars->l2, split, warp, lane);
}

}  // namespace skl
