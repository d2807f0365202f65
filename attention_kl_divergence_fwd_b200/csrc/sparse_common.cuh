// sparse_common.cuh - shared pieces of the block-sparse attention kernels: problem view,
// packing of grouped query heads into 128-row tiles, the selection bit matrix.
//
// Keys are cut into blocks of 64. Every query of every selection head lists the blocks it
// reads. The tensor core works on tiles of 128 rows, so rows that share a K head and a
// selection are packed: a tile holds Qn queries (a power of two) of the G query heads of
// one pack, row r = g * Qn + (query - q0). A tile reads the union of its queries' blocks and
// each row drops the blocks that its own query did not list. For neighbouring queries, whose
// lists largely agree, the union is little longer than one list; a gather per query instead
// would move every block through L2 once per query (at 16384 tokens, 8 K heads and 16 blocks
// of 64 x 256 bf16 that is 69 GB), and for unrelated lists the union ends at dense attention.
//
// The lists become a bit matrix first: word (iw, c) of a selection head holds, for queries
// 32 iw .. 32 iw + 31, whether each reads block c. It turns lists in any order, with repeated
// or negative entries, into sets; a tile scans its row of words (consecutive c), the
// key-major backward scans a column.
#pragma once

#include <cstddef>

#include "ptx.cuh"

namespace skl {

constexpr int kSpBlock = 64;  // keys per block

struct SparseArgs {
  int B, H, N_Q, N_K, NB;  // NB = ceil(N_K / 64)
  int P, G;                // packs of query heads per batch entry, heads per pack (H = P * G)
  int Hkv, Hsel;           // K heads, selection heads (both divide P)
  int Qn, n_tiles;         // queries per 128-row tile, tiles per pack
  int causal, topk;
  int splits;              // CTAs (one cluster) that share one tile's list (forward, dQ)
  int kv_splits;           // the same for a block's tiles (dK, dV)
  int direct;              // forward of one query: blocks straight from the list
  float c, scale;          // |scale| * log2(e); signed scale
  const int* idx;          // [B, Hsel, N_Q, topk]
  const int* lens;         // [B] keys of each sequence, or null (N_K)
  const uint32_t* mask;    // [B * Hsel, ceil(N_Q / 32), NB]
  float2* rows;            // backward: {LSE * log2(e), sum_d out * dout} per row
  __nv_bfloat16* out;      // forward
  float* lse;              // may be null
  __nv_bfloat16* dq;       // backward
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
};

// Keys of sequence b. A length outside 0 .. N_K is recorded and read as an empty sequence.
__device__ __forceinline__ int sp_len(const int* lens, int b, int N_K) {
  if (lens == nullptr) return N_K;
  const int n = __ldg(lens + b);
  if (n < 0 || n > N_K) {
    if (threadIdx.x == 0) atomicOr(&g_skl_error, kErrBadOffsets);
    return 0;
  }
  return n;
}

// Last key index that query i may read (bottom-right causal alignment), -1 for none.
__device__ __forceinline__ int sp_last(int i, int nk, int N_Q, int causal) {
  return causal ? max(-1, min(nk - 1, i + nk - N_Q)) : nk - 1;
}

// A tile of one pack: sequence, K head, selection head, first query and first row.
struct SpTile {
  int b, p, q0, nk;
  int kv;        // head coordinate of K and V in the tensor maps
  int h0;        // head coordinate of the pack's first query head
  const uint32_t* words;  // row of the bit matrix that holds query q0
  int bit0;      // bit of query q0 within its word (0 unless Qn < 32)
  int nwords;    // words that cover the tile's queries (1, 2 or 4)
};

__device__ __forceinline__ SpTile sp_tile(const SparseArgs& a, int bp, int tile) {
  SpTile t;
  t.b = bp / a.P;
  t.p = bp - t.b * a.P;
  t.q0 = tile * a.Qn;
  t.nk = sp_len(a.lens, t.b, a.N_K);
  t.kv = t.b * a.Hkv + t.p / (a.P / a.Hkv);
  t.h0 = t.b * a.H + t.p * a.G;
  const int sel = t.b * a.Hsel + t.p / (a.P / a.Hsel);
  const int iws = (a.N_Q + 31) >> 5;
  t.words = a.mask + ((size_t)sel * iws + (t.q0 >> 5)) * a.NB;
  t.bit0 = t.q0 & 31;
  t.nwords = a.Qn <= 32 ? 1 : min(a.Qn >> 5, iws - (t.q0 >> 5));
  return t;
}

// Tiles of at most 32 rows (single tokens of small groups): the tile's rows are loaded four
// times, at lanes 0, 32, 64 and 96, and each of the four row warps takes a quarter of every key
// tile's columns. TMEM lets a warp read only its own 32 lanes, so without the copies one warp
// would do all of the tile's exponentials while three sit idle.
__host__ __device__ inline bool sp_quad(int Qn, int G) { return Qn * G <= 32; }

// Start of a kernel's CTA. The producer warp initialises the barriers (an array of `n` at the start
// of the barrier block, `arrivals(i)` each), announces that and goes on to its first loads; the
// other warps come here after their own preparations and wait for the barriers (and for the TMEM
// address). Named barrier 15 of `threads` threads.
template <typename Arrivals>
__device__ __forceinline__ void sp_init_barriers(uint64_t* bars, int n, int threads, int lane,
                                                 Arrivals arrivals) {
  for (int i = lane; i < n; i += 32) mbar_init(smem_u32(bars + i), arrivals(i));
  fence_mbar_init();
  __syncwarp();
  named_bar_arrive(15, threads);
}

// Programmatic launches. The next kernel of the stream, launched with the overlap attribute, starts
// once every CTA of this one has called grid_allow_next (or ended), and takes the SMs that its last
// CTAs leave free. grid_wait_previous waits for that earlier kernel's end and its writes.
__device__ __forceinline__ void grid_allow_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// At the end of a kernel that runs beside an earlier one without reading what that writes: its last
// CTA waits for the earlier kernel, so that what follows in the stream follows both.
__device__ __forceinline__ void grid_end_after_previous() {
  if (blockIdx.x == gridDim.x - 1) grid_wait_previous();
}

// Builds the bit matrix: one CTA per 32 queries of a selection head. Entries that are
// negative, beyond the last block, or of a block the query may not see set no bit. Bound by the
// latency of its reads (8 heads x 16384 queries x 32 entries: 15 us).
constexpr int kMaskChunk = 8192;  // blocks per pass (32 KB of shared memory at most)
__global__ void __launch_bounds__(256)
streamkl_sparse_mask_kernel(const SparseArgs a, uint32_t* mask) {
  extern __shared__ __align__(1024) uint8_t smem[];
  grid_allow_next();
  uint32_t* sm = reinterpret_cast<uint32_t*>(smem);
  const int iws = (a.N_Q + 31) >> 5;
  const int sel = blockIdx.x / iws, iw = blockIdx.x - sel * iws, b = sel / a.Hsel, i0 = iw * 32;
  const int nk = sp_len(a.lens, b, a.N_K);
  const int nq = min(32, a.N_Q - i0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int* idx = a.idx + ((size_t)sel * a.N_Q + i0) * a.topk;
  uint32_t* dst = mask + ((size_t)sel * iws + iw) * a.NB;
  for (int c0 = 0; c0 < a.NB; c0 += kMaskChunk) {
    const int n = min(kMaskChunk, a.NB - c0);
    // The first entries of the warp's four queries are read while shared memory is cleared.
    int first[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int q = warp + 8 * k;
      first[k] = q < nq && lane < a.topk ? __ldg(idx + (size_t)q * a.topk + lane) : -1;
    }
    for (int c = threadIdx.x; c < n; c += 256) sm[c] = 0u;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int q = warp + 8 * k;
      if (q >= nq) continue;
      const int last = sp_last(i0 + q, nk, a.N_Q, a.causal);
      // Last block the query sees; c <= that keeps c * 64 from being formed for wild entries.
      const int top = last < 0 ? -1 : last / kSpBlock;
      for (int e = lane; e < a.topk; e += 32) {
        const int c = e == lane ? first[k] : __ldg(idx + (size_t)q * a.topk + e);
        if (c >= 0 && c <= top && c >= c0 && c - c0 < n) atomicOr(&sm[c - c0], 1u << q);
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += 256) dst[c0 + c] = sm[c];
    __syncthreads();
  }
  grid_end_after_previous();
}

}  // namespace skl
