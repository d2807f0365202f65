// sparse_api.cuh - argument checks and launch planner of the block-sparse attention entry
// points (include/streamkl.h states the contract). Part of streamkl_api.cu.
#pragma once

namespace {

// Tensor map over [heads, rows, d] bf16 with a box of 64 columns x box_rows x box_heads.
bool make_map_heads(CUtensorMap* m, const void* base, int d, long long rows, long long heads,
                    int box_rows, int box_heads) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)rows, (cuuint64_t)heads};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)rows * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_heads};
  const cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&] {
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (encode()) return true;
  // A driver call wants a current context, which a thread without CUDA work so far does not have;
  // selecting the device that is current anyway makes its context current.
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

// Raises a kernel's dynamic shared-memory limit on the current device once (`done`: one flag
// per device and kernel; threads that race on it set the same value).
template <typename Kern>
bool set_smem_once(Kern k, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_acquire)) return true;
  if (!set_smem(k, bytes)) return false;
  if (dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_release);
  return true;
}

bool misaligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

constexpr int kMaxTopk = 1 << 20;

// Sizes common to every block-sparse entry point, and the packing of rows into tiles.
streamkl_status sparse_problem(skl::SparseArgs& a, const int* lens, int B, int H, int Hkv,
                               int Hsel, int N_Q, int N_K, int d, float scale, int causal) {
  if (B < 1 || H < 1 || N_Q < 1 || N_K < 1 || !std::isfinite(scale))
    return STREAMKL_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return STREAMKL_ERR_UNSUPPORTED;
  if (Hkv < 1 || Hsel < 1 || H % Hkv != 0 || H % Hsel != 0) return STREAMKL_ERR_UNSUPPORTED;
  const int P = Hkv > Hsel ? Hkv : Hsel;
  if (P % Hkv != 0 || P % Hsel != 0 || H / P > 128) return STREAMKL_ERR_UNSUPPORTED;
  const long long bh = (long long)B * H, nmax = N_Q > N_K ? N_Q : N_K;
  if (bh >= (1ll << 24) || bh * nmax >= (1ll << 31)) return STREAMKL_ERR_UNSUPPORTED;
  if (misaligned4(lens)) return STREAMKL_ERR_MISALIGNED;
  a.B = B;
  a.H = H;
  a.N_Q = N_Q;
  a.N_K = N_K;
  a.NB = (N_K + skl::kSpBlock - 1) / skl::kSpBlock;
  a.P = P;
  a.G = H / P;
  a.Hkv = Hkv;
  a.Hsel = Hsel;
  a.Qn = 1;
  while (a.Qn * 2 * a.G <= 128 && a.Qn < N_Q) a.Qn *= 2;
  a.n_tiles = (N_Q + a.Qn - 1) / a.Qn;
  a.causal = causal ? 1 : 0;
  a.splits = 1;
  // A scale of 0 keeps a positive factor (masked scores are -inf, and -inf * 0 is NaN); it is
  // far below what the scores' products with it can show in fp32.
  a.c = scale == 0.f ? 1e-30f : std::fabs(scale) * kLog2e;
  a.scale = scale;
  a.lens = lens;
  return STREAMKL_OK;
}

long long round256(long long n) { return (n + 255) / 256 * 256; }

long long mask_bytes(const skl::SparseArgs& a) {
  return round256(4ll * a.B * a.Hsel * ((a.N_Q + 31) / 32) * a.NB);
}

// CTAs of a cluster that share a tile's list: as many as keep the grid within one wave (two CTAs
// per SM), at most 8 (the portable cluster size), each with at least one block. A
// second wave costs more than longer lists: one token of 32 sequences of 8 K heads (256 tiles of
// 16 blocks) takes 31.5, 41.1, 50.7 and 57.2 us with 1, 2, 3 and 4 CTAs per tile, one sequence of
// 32 blocks (8 tiles) 24.6, 18.2, 16.1 and 15.9 us.
int sparse_splits(const skl::SparseArgs& a) {
  const long long ctas = (long long)a.B * a.P * a.n_tiles;
  long long blocks = (long long)a.Qn * a.topk;
  blocks = blocks < a.NB ? blocks : a.NB;
  long long s = 2ll * sm_count() / ctas;
  if (s > blocks) s = blocks;
  return (int)(s < 1 ? 1 : (s > 8 ? 8 : s));
}

// The same for the tiles of one block (dK, dV; one CTA per SM). A block that every query lists (the
// first one) has n_tiles steps while the average one has its share of the lists, so with few
// heads its CTA alone outlasts the rest of the grid. A CTA of a cluster costs about 17 steps
// (measured: 1024 clusters of two instead of 1024 CTAs take 238 us more at 16384 tokens, 4 K
// heads), so blocks are split only when the longest one dominates. That figure, and the 1.3 lists'
// worth of blocks that a tile is taken to read, come from d = 128 and lists that runs of 128 queries
// share; they are estimates for d = 64 and for unrelated lists, which only the split depends on.
int sparse_kv_splits(const skl::SparseArgs& a) {
  const double longest = (double)a.n_tiles * (a.P / a.Hkv), heads = (double)a.B * a.Hkv;
  const double per_tile = a.NB < 1.3 * a.topk ? a.NB : 1.3 * a.topk;
  int best = 1;
  double best_cost = 0;
  for (int s = 1; s <= 8; s *= 2) {
    const double start = s == 1 ? 2 : 17 * s;
    const double work = heads * (longest * per_tile + a.NB * start) / sm_count();
    const double cost = work > longest / s ? work : longest / s;
    if (s == 1 || cost < 0.9 * best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

bool sparse_direct(const skl::SparseArgs& a) {
  return a.N_Q == 1 && a.G <= 16 && a.NB <= 16384 && a.topk <= 512;
}

long long fwd_ws_bytes(const skl::SparseArgs& a) { return sparse_direct(a) ? 0 : mask_bytes(a); }

long long bwd_ws_bytes(const skl::SparseArgs& a) {
  return mask_bytes(a) + round256(8ll * a.B * a.H * a.N_Q);
}

streamkl_status ok_launch() {
  return cudaGetLastError() == cudaSuccess ? STREAMKL_OK : STREAMKL_ERR_LAUNCH;
}

// Launches a grid, in clusters along x for cluster > 1; overlap: beside the tail of the stream's
// previous kernel (grid_allow_next in sparse_common.cuh).
template <typename... Params, typename... Args>
streamkl_status launch(void (*kern)(Params...), dim3 grid, int cluster, int threads, int smem,
                       bool overlap, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n++].val.clusterDim = {(unsigned)cluster, 1, 1};
  }
  if (overlap) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess) return STREAMKL_OK;
  cudaGetLastError();
  return STREAMKL_ERR_LAUNCH;
}

// units * cluster CTAs (plain CTAs for a cluster of one).
template <typename... Params, typename... Args>
streamkl_status launch_cluster(void (*kern)(Params...), long long units, int cluster, int threads,
                               int smem, bool overlap, cudaStream_t stream, const Args&... args) {
  if (units * cluster >= (1ll << 31)) return STREAMKL_ERR_UNSUPPORTED;
  return launch(kern, dim3((unsigned)(units * cluster)), cluster, threads, smem, overlap, stream,
                args...);
}

streamkl_status launch_mask(skl::SparseArgs& a, void* ws, bool overlap, cudaStream_t stream) {
  const long long grid = (long long)((a.N_Q + 31) / 32) * a.B * a.Hsel;
  uint32_t* mask = static_cast<uint32_t*>(ws);
  const int smem = 4 * (a.NB < skl::kMaskChunk ? a.NB : skl::kMaskChunk);
  const streamkl_status st = launch_cluster(skl::streamkl_sparse_mask_kernel, grid, 1, 256, smem,
                                            overlap, stream, a, mask);
  a.mask = mask;
  return st;
}

template <int D, bool QUAD>
streamkl_status launch_sparse_fwd(const skl::SparseArgs& a, const void* q, const void* k,
                                  const void* v, cudaStream_t stream) {
  using C = skl::SpFwdCfg<D>;
  CUtensorMap mq, mk, mv;
  if (!make_map_heads(&mq, q, D, a.N_Q, (long long)a.B * a.H, a.Qn, a.G) ||
      !make_map_heads(&mk, k, D, a.N_K, (long long)a.B * a.Hkv, 64, 1) ||
      !make_map_heads(&mv, v, D, a.N_K, (long long)a.B * a.Hkv, 64, 1))
    return STREAMKL_ERR_LAUNCH;
  auto kern = skl::streamkl_sparse_fwd_kernel<D, QUAD>;
  static std::atomic<bool> done[64] = {};
  if (!set_smem_once(kern, C::SMEM, done)) return STREAMKL_ERR_LAUNCH;
  const bool neg = a.scale < 0.f;
  return launch_cluster(kern, (long long)a.B * a.P * a.n_tiles, a.splits, skl::kSpThreads, C::SMEM,
                        !a.direct, stream, mq, mk, mv, a,
                        skl::idesc_bf16_f32(128, 64, false, false, neg),
                        skl::idesc_bf16_f32(128, D, false, true));
}

template <int D>
streamkl_status launch_sparse_bwd(skl::SparseArgs& a, const void* q, const void* k,
                                  const void* v, const void* out, const float* lse,
                                  const void* dout, void* ws, cudaStream_t stream) {
  using CQ = skl::SpDqCfg<D>;
  using CK = skl::SpDkvCfg<D>;
  CUtensorMap mq, mdo, mk, mv;
  if (!make_map_heads(&mq, q, D, a.N_Q, (long long)a.B * a.H, a.Qn, a.G) ||
      !make_map_heads(&mdo, dout, D, a.N_Q, (long long)a.B * a.H, a.Qn, a.G) ||
      !make_map_heads(&mk, k, D, a.N_K, (long long)a.B * a.Hkv, 64, 1) ||
      !make_map_heads(&mv, v, D, a.N_K, (long long)a.B * a.Hkv, 64, 1))
    return STREAMKL_ERR_LAUNCH;
  auto kq = skl::streamkl_sparse_dq_kernel<D>;
  auto kk = skl::streamkl_sparse_dkv_kernel<D>;
  static std::atomic<bool> done_q[64] = {}, done_k[64] = {};
  if (!set_smem_once(kq, CQ::SMEM, done_q) || !set_smem_once(kk, CK::SMEM, done_k))
    return STREAMKL_ERR_LAUNCH;
  const bool neg = a.scale < 0.f;
  const uint32_t i_s = skl::idesc_bf16_f32(128, 64, false, false, neg);
  const uint32_t i_dp = skl::idesc_bf16_f32(128, 64, false, false);
  const long long rows = (long long)a.B * a.H * a.N_Q;
  constexpr int per_cta = 8 * 32 / (D / 8) * skl::kRowsPerGroup;
  // Rows that see one block at most: the first ones of a causal sequence, or all rows of a short
  // one. Without padded lengths the host knows whether there are any.
  const bool any_short =
      a.lens || (a.causal ? a.N_K - a.N_Q < skl::kSpBlock : a.N_K <= skl::kSpBlock);
  const auto* o16 = static_cast<const __nv_bfloat16*>(out);
  const auto* do16 = static_cast<const __nv_bfloat16*>(dout);
  streamkl_status st = STREAMKL_OK;
  if (any_short) {
    // Causal without lengths: the last such query is N_Q - N_K + 63.
    long long n = a.N_Q;
    if (!a.lens && a.causal && n > (long long)a.N_Q - a.N_K + 64) n = (long long)a.N_Q - a.N_K + 64;
    const long long y = (n + 7) / 8;
    const dim3 grid((unsigned)(a.B * a.H), (unsigned)(y < 65535 ? y : 65535));
    st = launch(skl::streamkl_sparse_short_rows_kernel<D>, grid, 1, 256, 0, false, stream, a,
                static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
                static_cast<const __nv_bfloat16*>(v), do16, lse);
  }
  if (st == STREAMKL_OK)
    st = launch(skl::streamkl_sparse_rows_kernel<D>, dim3((unsigned)((rows + per_cta - 1) / per_cta)), 1,
                256, 0, any_short, stream, a, o16, do16, lse, rows, any_short);
  if (st == STREAMKL_OK) st = launch_mask(a, ws, true, stream);
  if (st != STREAMKL_OK) return st;
  st = launch_cluster(
      kk, (long long)a.B * a.Hkv * a.NB, a.kv_splits, skl::kSpDkvThreads, CK::SMEM, false, stream, mq,
      mdo, mk, mv, a, i_s, i_dp, skl::idesc_bf16_f32(128, 64, true, true));
  if (st != STREAMKL_OK) return st;
  // Beside dK and dV's tail: neither reads the other's results.
  return launch_cluster(kq, (long long)a.B * a.P * a.n_tiles, a.splits, skl::kSpDqThreads, CQ::SMEM,
                        true, stream, mq, mdo, mk, mv, a, i_s, i_dp,
                        skl::idesc_bf16_f32(128, D, false, true));
}

// CTAs of the cluster that normalises a tile of few rows on chip (kMassFused), 0 for the two-kernel
// form: as many as the portable cluster size allows while every CTA gets a pair of blocks. Only
// while all clusters fit on the chip at once (two CTAs per SM) and a CTA's share of the values
// fits its shared memory: 16 sequences of up to 32768 keys and 8 K heads (1024 CTAs) take 93 us
// in clusters, where CTAs without keys hold their SM until the cluster ends, and 73 us as two
// kernels; one sequence of 4097 keys 7.3 us and one launch instead of 7.2 us and two.
int mass_fused(const skl::SparseArgs& a) {
  if (!skl::sp_quad(a.Qn, a.G)) return 0;
  int s = (a.NB + 1) / 2;
  s = s > 8 ? 8 : s;
  if ((long long)a.B * a.P * a.n_tiles * s > 2ll * sm_count()) return 0;
  const long long bpc = ((a.NB + s - 1) / s + 1) / 2 * 2;
  return 2ll * a.Qn * a.G * (bpc + 1) <= skl::kMassStage ? s : 0;
}

long long mass_ws_bytes(const skl::SparseArgs& a) { return 4ll * a.B * a.H * a.N_Q * a.NB; }

template <int D, int MODE, bool QUAD>
streamkl_status launch_mass(const skl::MassArgs& ma, const void* q, const void* k,
                            cudaStream_t stream) {
  using C = skl::MassCfg<D>;
  const skl::SparseArgs& a = ma.s;
  CUtensorMap mq, mk;
  if (!make_map_heads(&mq, q, D, a.N_Q, (long long)a.B * a.H, a.Qn, a.G) ||
      !make_map_heads(&mk, k, D, a.N_K, (long long)a.B * a.P, 128, 1))
    return STREAMKL_ERR_LAUNCH;
  auto kern = skl::streamkl_block_mass_kernel<D, MODE, QUAD>;
  static std::atomic<bool> done[64] = {};
  if (!set_smem_once(kern, C::SMEM, done)) return STREAMKL_ERR_LAUNCH;
  const streamkl_status st = launch_cluster(
      kern, (long long)a.B * a.P * a.n_tiles * (MODE == skl::kMassFused ? 1 : ma.n_chunks),
      MODE == skl::kMassFused ? ma.n_chunks : 1, skl::kMassThreads, C::SMEM, false, stream, mq, mk, ma,
      skl::idesc_bf16_f32(128, 128, false, false, a.scale < 0.f));
  if (st != STREAMKL_OK || MODE != skl::kMassParts) return st;
  skl::streamkl_block_norm_kernel<<<(unsigned)((long long)a.B * a.P * a.N_Q), 256, 0, stream>>>(ma);
  return ok_launch();
}

}  // namespace

extern "C" {

long long streamkl_sparse_attn_workspace(int B, int H, int H_kv, int H_sel, int N_Q, int N_K,
                                         int d, int topk, int backward) {
  skl::SparseArgs a{};
  if (topk < 1 || topk > kMaxTopk ||
      sparse_problem(a, nullptr, B, H, H_kv, H_sel, N_Q, N_K, d, 1.f, 0) != STREAMKL_OK)
    return -1;
  a.topk = topk;
  return backward ? bwd_ws_bytes(a) : fwd_ws_bytes(a);
}

long long streamkl_block_mass_workspace(int B, int H, int H_kv, int N_Q, int N_K, int d) {
  skl::SparseArgs a{};
  if (sparse_problem(a, nullptr, B, H, H_kv, H_kv, N_Q, N_K, d, 1.f, 0) != STREAMKL_OK) return -1;
  return mass_fused(a) ? 0 : mass_ws_bytes(a);
}

streamkl_status streamkl_sparse_attn_fwd(const void* q, const void* k, const void* v,
                                         const int* block_idx, const int* seqlens_k, int B, int H,
                                         int H_kv, int H_sel, int N_Q, int N_K, int d, int topk,
                                         float scale, int causal, void* workspace,
                                         long long workspace_bytes, void* out, float* lse,
                                         cudaStream_t stream) {
  skl::SparseArgs a{};
  const streamkl_status st =
      sparse_problem(a, seqlens_k, B, H, H_kv, H_sel, N_Q, N_K, d, scale, causal);
  if (st != STREAMKL_OK) return st;
  if (topk < 1 || !q || !k || !v || !block_idx || !out) return STREAMKL_ERR_INVALID_ARG;
  if (topk > kMaxTopk) return STREAMKL_ERR_UNSUPPORTED;
  a.topk = topk;
  const long long need = fwd_ws_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return STREAMKL_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse) ||
      !aligned16(workspace) || misaligned4(block_idx))
    return STREAMKL_ERR_MISALIGNED;
  a.idx = block_idx;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.splits = sparse_splits(a);
  a.direct = sparse_direct(a) ? 1 : 0;
  if (!a.direct) {
    const streamkl_status sm = launch_mask(a, workspace, false, stream);
    if (sm != STREAMKL_OK) return sm;
  }
  if (skl::sp_quad(a.Qn, a.G))
    return d == 128 ? launch_sparse_fwd<128, true>(a, q, k, v, stream)
                    : launch_sparse_fwd<64, true>(a, q, k, v, stream);
  return d == 128 ? launch_sparse_fwd<128, false>(a, q, k, v, stream)
                  : launch_sparse_fwd<64, false>(a, q, k, v, stream);
}

streamkl_status streamkl_sparse_attn_bwd(const void* q, const void* k, const void* v,
                                         const void* out, const float* lse, const void* dout,
                                         const int* block_idx, const int* seqlens_k, int B, int H,
                                         int H_kv, int H_sel, int N_Q, int N_K, int d, int topk,
                                         float scale, int causal, void* workspace,
                                         long long workspace_bytes, void* dq, void* dk, void* dv,
                                         cudaStream_t stream) {
  skl::SparseArgs a{};
  const streamkl_status st =
      sparse_problem(a, seqlens_k, B, H, H_kv, H_sel, N_Q, N_K, d, scale, causal);
  if (st != STREAMKL_OK) return st;
  if (topk < 1 || !q || !k || !v || !out || !lse || !dout || !block_idx || !dq || !dk || !dv)
    return STREAMKL_ERR_INVALID_ARG;
  if (topk > kMaxTopk) return STREAMKL_ERR_UNSUPPORTED;
  a.topk = topk;
  if (!workspace || workspace_bytes < bwd_ws_bytes(a)) return STREAMKL_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse) ||
      !aligned16(dout) || !aligned16(workspace) || !aligned16(dq) || !aligned16(dk) ||
      !aligned16(dv) || misaligned4(block_idx))
    return STREAMKL_ERR_MISALIGNED;
  a.idx = block_idx;
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  char* ws = static_cast<char*>(workspace);
  a.rows = reinterpret_cast<float2*>(ws + mask_bytes(a));
  a.splits = sparse_splits(a);
  a.kv_splits = sparse_kv_splits(a);
  return d == 128 ? launch_sparse_bwd<128>(a, q, k, v, out, lse, dout, ws, stream)
                  : launch_sparse_bwd<64>(a, q, k, v, out, lse, dout, ws, stream);
}

streamkl_status streamkl_block_mass(const void* q, const void* k, const int* seqlens_k, int B,
                                    int H, int H_kv, int N_Q, int N_K, int d, float scale,
                                    int causal, const float* lse, void* workspace,
                                    long long workspace_bytes, float* mass, cudaStream_t stream) {
  skl::MassArgs ma{};
  const streamkl_status st =
      sparse_problem(ma.s, seqlens_k, B, H, H_kv, H_kv, N_Q, N_K, d, scale, causal);
  if (st != STREAMKL_OK) return st;
  const skl::SparseArgs& a = ma.s;
  if (!q || !k || !mass) return STREAMKL_ERR_INVALID_ARG;
  const int fused = lse ? 0 : mass_fused(a);
  if (!lse && !fused && (!workspace || workspace_bytes < mass_ws_bytes(a)))
    return STREAMKL_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(mass) || !aligned16(lse) ||
      !aligned16(workspace))
    return STREAMKL_ERR_MISALIGNED;
  ma.row_lse = lse;
  ma.mass = mass;
  ma.blse = lse || fused ? nullptr : static_cast<float*>(workspace);
  // A tile's blocks are spread over CTAs while there are fewer than about four waves of them
  // (two per SM; the tail of a wave and padded sequences' early ends even out); a CTA takes at
  // least one pair.
  const long long tiles = (long long)a.B * a.P * a.n_tiles, want = 8ll * sm_count();
  const long long chunks = fused ? fused : (want / tiles > 1 ? want / tiles : 1);
  const long long bpc = ((a.NB + chunks - 1) / chunks + 1) / 2 * 2;
  ma.bpc = (int)bpc;
  ma.n_chunks = (int)((a.NB + bpc - 1) / bpc);
  if (fused) ma.n_chunks = fused;  // the cluster's last CTAs may have no block
  const bool quad = skl::sp_quad(a.Qn, a.G);
  auto go = [&](auto dim, auto norm) {
    constexpr int D = decltype(dim)::value;
    constexpr int N = decltype(norm)::value;
    return quad ? launch_mass<D, N, true>(ma, q, k, stream)
                : launch_mass<D, N, false>(ma, q, k, stream);
  };
  auto pick = [&](auto dim) {
    if (lse) return go(dim, std::integral_constant<int, skl::kMassNorm>{});
    if (fused)
      return launch_mass<decltype(dim)::value, skl::kMassFused, true>(ma, q, k, stream);
    return go(dim, std::integral_constant<int, skl::kMassParts>{});
  };
  return d == 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 64>{});
}

streamkl_status streamkl_block_select(const float* mass, const int* seqlens_k, int B, int H_sel,
                                      int N_Q, int N_K, int causal, int topk, int n_first,
                                      int n_last, int* block_idx, cudaStream_t stream) {
  if (!mass || !block_idx || B < 1 || H_sel < 1 || N_Q < 1 || N_K < 1 || topk < 1 ||
      n_first < 0 || n_last < 0 || n_first > topk || n_last > topk - n_first)
    return STREAMKL_ERR_INVALID_ARG;
  const long long rows = (long long)B * H_sel * N_Q;
  const int nb = (N_K + skl::kSpBlock - 1) / skl::kSpBlock;
  if (topk > kMaxTopk || (long long)B * H_sel >= (1ll << 24) || rows >= (1ll << 31) || nb > 8192)
    return STREAMKL_ERR_UNSUPPORTED;
  if (!aligned16(mass) || !aligned16(block_idx) || misaligned4(seqlens_k))
    return STREAMKL_ERR_MISALIGNED;
  const skl::SelectArgs a{mass, seqlens_k, block_idx, H_sel, N_Q, N_K, nb, causal ? 1 : 0, topk,
                          n_first, n_last};
  // (selection heads, rows): y is limited to 65535, beyond that a CTA takes several rows.
  auto grid = [&](int rows_per_cta) {
    const int y = (N_Q + rows_per_cta - 1) / rows_per_cta;
    return dim3((unsigned)(B * H_sel), (unsigned)(y < 65535 ? y : 65535));
  };
  // Few rows leave the SMs idle: then a row's blocks are spread over eight warps (512 rows of 1024
  // blocks: 14.3 us with one warp each, 6.6 us with eight).
  const bool few = rows < 16ll * sm_count();
  if (nb <= 64)
    skl::streamkl_block_select_kernel<2, 1><<<grid(4), 128, 0, stream>>>(a);
  else if (nb <= 256)
    skl::streamkl_block_select_kernel<8, 1><<<grid(4), 128, 0, stream>>>(a);
  else if (nb <= 1024 && few)
    skl::streamkl_block_select_kernel<4, 8><<<grid(1), 256, 0, stream>>>(a);
  else if (nb <= 1024)
    skl::streamkl_block_select_kernel<32, 1><<<grid(4), 128, 0, stream>>>(a);
  else
    skl::streamkl_block_select_kernel<32, 8><<<grid(1), 256, 0, stream>>>(a);
  return ok_launch();
}

}  // extern "C"
