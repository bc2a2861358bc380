// Host side of the balance loss and the 8-bit floating-point operators.
// Part of coli_moe.cu (included there, after the launch helpers).
#pragma once

namespace {

// ---- balance ---------------------------------------------------------------

// Blocks of a balance pass: one cluster up to kBalFused tokens, else a token per
// warp up to kBalMaxBlocks, so that the workspace depends on T and E alone.
inline bool balance_fused(int T) { return T <= kBalFused; }
inline int balance_blocks(int T) {
  return balance_fused(T) ? kBalCluster : std::min((T + kBalWarps - 1) / kBalWarps, kBalMaxBlocks);
}

template <typename... KArgs, typename... Args>
bool launch_balance(void (*kernel)(KArgs...), int grid, bool cluster, int threads, size_t smem, cudaStream_t st,
                    Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kBalCluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  ++t_launches;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...) == cudaSuccess;
}

struct BalWs {
  float* p;      // [blocks][E] column sums
  int32_t* c;    // [blocks][E] pair counts
  int32_t* n;    // [blocks] live tokens
  size_t bytes;
};

BalWs balance_layout(int T, int E, void* base) {
  BalWs w{};
  const size_t nb = static_cast<size_t>(balance_blocks(T));
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t o = 0;
  auto take = [&](size_t bytes) -> void* {
    void* p = b ? b + o : nullptr;
    o += align256(bytes);
    return p;
  };
  w.p = static_cast<float*>(take(nb * E * 4));
  w.c = static_cast<int32_t*>(take(nb * E * 4));
  w.n = static_cast<int32_t*>(take(nb * 4));
  w.bytes = o;
  return w;
}

coli_status check_balance(int T, int E, int k) {
  if (T < 0 || E < 1 || k < 1) return COLI_ERR_INVALID_ARG;
  if (E > 1024 || k > 32 || k > E || static_cast<int64_t>(T) * k > (int64_t(1) << 24)) return COLI_ERR_UNSUPPORTED;
  return COLI_OK;
}

// Rows move as 16-byte loads when every row starts on a 16-byte boundary.
inline bool balance_vec4(int E, const void* a, const void* b, const void* c) {
  return E % 4 == 0 && aligned(a, 16) && aligned(b, 16) && aligned(c, 16);
}

#define COLI_BAL_DISPATCH(E, vec, CALL)                                        \
  switch (route_nv(E)) {                                                       \
    case 1: case 2: case 4:                                                    \
      ok = vec ? CALL(4, 4) : CALL(4, 1); break;                               \
    case 8: ok = vec ? CALL(8, 4) : CALL(8, 1); break;                         \
    case 16: ok = vec ? CALL(16, 4) : CALL(16, 1); break;                      \
    default: ok = vec ? CALL(32, 4) : CALL(32, 1); break;                      \
  }

// ---- 8-bit floating point ----------------------------------------------------

coli_status check_dims_fp8(const coli_moe_dims* d) {
  if (!d) return COLI_ERR_INVALID_ARG;
  if (d->group != kF8Block || d->code_bits != 8) return COLI_ERR_UNSUPPORTED;
  if (d->hidden <= 0 || d->hidden % kF8Block != 0 || d->inter <= 0 || d->inter % kF8Block != 0)
    return COLI_ERR_UNSUPPORTED;
  if (d->n_experts < 1 || d->n_experts > 1024) return COLI_ERR_UNSUPPORTED;
  if (d->top_k < 1 || d->top_k > 32 || d->top_k > d->n_experts) return COLI_ERR_UNSUPPORTED;
  if (d->n_shared < 0 || d->n_shared > 4) return COLI_ERR_UNSUPPORTED;
  const int64_t n = d->n_experts + d->n_shared, r = std::max(d->hidden, d->inter);
  if (n * r > INT32_MAX / 2) return COLI_ERR_UNSUPPORTED;
  return COLI_OK;
}

struct F8Ws {
  uint8_t* xg;    // [P+T][H] codes of x in pair order, then token order (more than 32 tokens)
  float* sg;      // [P+T][H/128]
  uint8_t* hq;    // [P+S*T][I] codes of h
  float* hs;      // [P+S*T][I/128]
  float* y;       // [P+S*T][H]
  size_t bytes;
};

F8Ws fp8_layout(const coli_moe_dims* d, int T, void* base) {
  F8Ws w{};
  const size_t rows = static_cast<size_t>(T) * (d->top_k + d->n_shared), I = d->inter, H = d->hidden;
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t o = 0;
  auto take = [&](size_t bytes) -> void* {
    void* p = b ? b + o : nullptr;
    o += align256(bytes);
    return p;
  };
  const size_t grows = T > kF8Few ? static_cast<size_t>(T) * (d->top_k + 1) : 0;
  w.xg = static_cast<uint8_t*>(take(grows * H));
  w.sg = static_cast<float*>(take(grows * (H / kF8Block) * 4));
  w.hq = static_cast<uint8_t*>(take(rows * I));
  w.hs = static_cast<float*>(take(rows * (I / kF8Block) * 4));
  w.y = static_cast<float*>(take(rows * H * 4));
  w.bytes = o;
  return w;
}

// Tensor maps of one launch: weights (two matrices of the same shape, or one),
// token rows in boxes of 128, 64, 32 and 16 rows, and single rows to gather.
bool fp8_maps(CUtensorMap* m, const uint8_t* w0, const uint8_t* w1, int64_t w_rows, const uint8_t* a, int64_t a_rows,
              int K) {
  auto enc = [&](CUtensorMap* out, const uint8_t* p, int64_t rows, uint32_t box) {
    return encode_2d(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, K, rows, K, kF8Block, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  bool ok = enc(&m[0], w0, w_rows, 128) && enc(&m[1], w1 ? w1 : w0, w_rows, 128);
  for (int j = 0; ok && j < 4; ++j) ok = enc(&m[2 + j], a, a_rows, 128u >> j);
  return ok && enc(&m[6], a, a_rows, 1);
}

// One product over `tiles` tiles (an upper bound for routed batches): persistent
// CTAs, or `split` of them in a cluster for each tile.
template <int NMAT, int NT, bool GU>
bool launch_fp8(const CUtensorMap* m, const F8Args& a, int64_t tiles, int split, int sms, cudaStream_t st) {
  auto kernel = fp8_gemm_kernel<NMAT, NT, GU>;
  using C = F8Cfg<NMAT, NT>;
  if (tiles < 1) return true;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split > 1 ? tiles * split : std::min<int64_t>(tiles, sms)));
  cfg.blockDim = dim3(kF8Threads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  ++t_launches;
  return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], m[4], m[5], m[6], a, split) == cudaSuccess;
}

}  // namespace

extern "C" {

size_t coli_moe_balance_workspace_bytes(int T_max, int E) {
  if (T_max < 0 || E < 1 || E > 1024) return 0;
  return balance_layout(std::max(T_max, 1), E, nullptr).bytes;
}

coli_status coli_moe_balance(const float* logits, const float* bias, const int32_t* topk_ids, const uint8_t* mask,
                             int T, int E, int k, int32_t* counts, int32_t* n_live, float* prob_mean, float* loss,
                             void* ws, size_t ws_bytes, void* stream) {
  const coli_status st = check_balance(T, E, k);
  if (st != COLI_OK) return st;
  if ((T > 0 && (!logits || !topk_ids)) || !counts || !n_live || !prob_mean || !loss || !ws || !aligned(ws, 256))
    return COLI_ERR_INVALID_ARG;
  const BalWs w = balance_layout(std::max(T, 1), E, ws);
  if (ws_bytes < w.bytes) return COLI_ERR_WORKSPACE;
  DevInfo di;
  if (dev_info(&di) != COLI_OK || !kernels_ready(di.dev, g_balance_ready, balance_kernels_ready)) return COLI_ERR_CUDA;
  const cudaStream_t s = as_stream(stream);
  const int blocks = balance_blocks(T);
  const bool fused = balance_fused(T);
  const bool vec = balance_vec4(E, logits, bias, nullptr);
  const size_t smem = static_cast<size_t>(kBalWarps + 1) * E * 4;
  const BalOut out{counts, n_live, prob_mean, loss};
  bool ok;
#define COLI_BAL_FWD(NV, VEC)                                                                                     \
  launch_balance(balance_kernel<NV, VEC>, blocks, fused, kBalWarps * 32, smem, s, logits, bias, topk_ids, mask, T, E, \
                 k, fused ? 1 : 0, w.p, w.c, w.n, out, di.status)
  COLI_BAL_DISPATCH(E, vec, COLI_BAL_FWD)
#undef COLI_BAL_FWD
  if (!ok) return COLI_ERR_CUDA;
  if (!fused && !launch_balance(balance_finish_kernel, kBalCluster, true, 512, 0, s, static_cast<const float*>(w.p),
                                static_cast<const int32_t*>(w.c), static_cast<const int32_t*>(w.n), blocks, E, k, out))
    return COLI_ERR_CUDA;
  return COLI_OK;
}

coli_status coli_moe_balance_backward(const float* logits, const float* bias, const uint8_t* mask,
                                      const int32_t* counts, const int32_t* n_live, const float* grad_loss,
                                      const int32_t* topk_ids, const float* topk_w, const float* d_topk_w, int T,
                                      int E, int k, float* d_logits, float* d_bias, void* ws, size_t ws_bytes,
                                      void* stream) {
  const coli_status st = check_balance(T, E, k);
  if (st != COLI_OK) return st;
  if (!counts || !n_live || (!grad_loss && !d_topk_w) || !ws || !aligned(ws, 256)) return COLI_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !d_logits || (d_topk_w && (!topk_ids || !topk_w)))) return COLI_ERR_INVALID_ARG;
  const BalWs w = balance_layout(std::max(T, 1), E, ws);
  if (ws_bytes < w.bytes) return COLI_ERR_WORKSPACE;
  DevInfo di;
  if (dev_info(&di) != COLI_OK || !kernels_ready(di.dev, g_balance_ready, balance_kernels_ready)) return COLI_ERR_CUDA;
  const cudaStream_t s = as_stream(stream);
  const int blocks = balance_blocks(T);
  const bool fused = balance_fused(T);
  const bool vec = balance_vec4(E, logits, bias, d_logits);
  const size_t smem = static_cast<size_t>(kBalWarps) * E * 4;
  bool ok;
#define COLI_BAL_BWD(NV, VEC)                                                                                    \
  launch_balance(balance_backward_kernel<NV, VEC>, blocks, fused, kBalWarps * 32, smem, s, logits, bias, mask, counts, \
                 n_live, grad_loss, topk_ids, topk_w, d_topk_w, T, E, k, fused ? 1 : 0, d_logits, w.p, d_bias)
  COLI_BAL_DISPATCH(E, vec, COLI_BAL_BWD)
#undef COLI_BAL_BWD
  if (!ok) return COLI_ERR_CUDA;
  if (d_bias && !fused && !launch(balance_bias_kernel, dim3((E + 31) / 32), dim3(512), 0, s,
                                  static_cast<const float*>(w.p), blocks, E, d_bias))
    return COLI_ERR_CUDA;
  return COLI_OK;
}

coli_status coli_add_rmsnorm_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, int T,
                                 int H, uint16_t* sum_out, uint16_t* norm_out, uint8_t* q, float* q_scale,
                                 void* stream) {
  if (T < 0 || H < 1 || !(eps >= 0.f)) return COLI_ERR_INVALID_ARG;
  if (H % kF8Block != 0 || H > 32768 || T > (1 << 24)) return COLI_ERR_UNSUPPORTED;
  if (T == 0) return COLI_OK;
  if (!x || !q || !q_scale) return COLI_ERR_INVALID_ARG;
  const void* ps[6] = {x, residual, weight, sum_out, norm_out, q};
  for (const void* p : ps)
    if (!aligned(p, 16)) return COLI_ERR_INVALID_ARG;
  if (!aligned(q_scale, 4) || norm_out == x || (residual && norm_out == residual) || (norm_out && norm_out == sum_out))
    return COLI_ERR_INVALID_ARG;
  DevInfo di;
  if (dev_info(&di) != COLI_OK) return COLI_ERR_CUDA;
  const cudaStream_t s = as_stream(stream);
  const int nc = (H + 2047) / 2048;
  const NormArgs a{x, residual, weight, eps, H, sum_out, norm_out, q, q_scale, di.status};
  bool ok;
#define COLI_NORM(NC) \
  launch(add_rmsnorm_fp8_kernel<NC>, dim3(T), dim3(256), 0, s, a)
  if (nc <= 1) ok = COLI_NORM(1);
  else if (nc <= 2) ok = COLI_NORM(2);
  else if (nc <= 3) ok = COLI_NORM(3);
  else if (nc <= 4) ok = COLI_NORM(4);
  else if (nc <= 8) ok = COLI_NORM(8);
  else ok = COLI_NORM(16);
#undef COLI_NORM
  return ok ? COLI_OK : COLI_ERR_CUDA;
}

coli_status coli_fp8_matmul(const uint8_t* a, const float* a_scale, const uint8_t* w, const float* w_scale, int M,
                            int N, int K, void* out, uint32_t flags, void* stream) {
  if (M < 0 || N < 1 || K < 1 || (flags & ~COLI_FP8_OUT_F32)) return COLI_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > (1 << 20) || N > (1 << 21) || M > (1 << 24)) return COLI_ERR_UNSUPPORTED;
  if (M == 0) return COLI_OK;
  if (!a || !a_scale || !w || !w_scale || !out) return COLI_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4))
    return COLI_ERR_INVALID_ARG;
  DevInfo di;
  if (dev_info(&di) != COLI_OK || !kernels_ready(di.dev, g_fp8_ready, fp8_kernels_ready)) return COLI_ERR_CUDA;
  const int nk = (K + kF8Block - 1) / kF8Block, nrb = (N + kF8Block - 1) / kF8Block;
  F8Args g{};
  g.a_s = a_scale;
  g.w_s = w_scale;
  g.out = out;
  g.status = di.status;
  g.M = M;
  g.R = N;
  g.nk = nk;
  g.out_f32 = (flags & COLI_FP8_OUT_F32) ? 1 : 0;
  g.wide = N % 8 == 0 && aligned(out, 32);
  CUtensorMap maps[7];
  if (!fp8_maps(maps, w, nullptr, N, a, M, K)) return COLI_ERR_CUDA;
  const cudaStream_t s = as_stream(stream);
  const bool few = M <= kF8Few;
  const int64_t blocks = few ? 1 : (M + kF8Tokens - 1) / kF8Tokens;
  // Two weight blocks a tile where such tiles fill the SMs: 48 KB of copies per K block
  // for twice the products of 32 KB (2048 x 4608 x 6144, 288 tiles of two: 74 us, 84 with
  // single blocks; 32 x 20480 x 6144, where the rule takes single ones in two waves, 41
  // with two and 57 so).  Below, single blocks, and several CTAs per tile where those
  // are fewer than the SMs too (1024 x 2048 x 6144, 128 tiles: 27 us, 39 with two).
  // Between the two, where single-block tiles need a second wave and two-block ones do
  // not, single blocks are 5 to 14 % slower (1024 x 4096 x 6144: 47 against 42 us); just
  // above one wave of two-block tiles they would be 10 % faster (1024 x 5120 x 6144: 64
  // against 72).
  const int64_t tiles1 = blocks * nrb, tiles2 = blocks * ((nrb + 1) / 2);
  bool ok;
  if (tiles2 >= di.sms) {
    ok = few ? launch_fp8<2, kF8Few, false>(maps, g, tiles2, 1, di.sms, s)
             : launch_fp8<2, kF8Tokens, false>(maps, g, tiles2, 1, di.sms, s);
  } else {
    // fewer tiles than SMs: single weight blocks, and several CTAs per tile
    int split = static_cast<int>(std::min<int64_t>({kF8MaxSplit, di.sms / tiles1, nk / 2}));
    if (split < 1) split = 1;
    ok = few ? launch_fp8<1, kF8Few, false>(maps, g, tiles1, split, di.sms, s)
             : launch_fp8<1, kF8Tokens, false>(maps, g, tiles1, split, di.sms, s);
  }
  return ok ? COLI_OK : COLI_ERR_CUDA;
}

size_t coli_moe_fp8_workspace_bytes(const coli_moe_dims* dims, int T_max) {
  if (check_dims_fp8(dims) != COLI_OK || T_max < 0) return 0;
  return fp8_layout(dims, std::max(T_max, 1), nullptr).bytes;
}

coli_status coli_moe_expert_ffn_fp8(const coli_moe_dims* dims, const coli_moe_weights_fp8* w, const uint8_t* x,
                                    const float* x_scale, int T, const int32_t* topk_ids, const float* topk_w,
                                    const int32_t* unique_ids, const int32_t* n_unique, const int32_t* seg_off,
                                    const int32_t* perm, const int32_t* pair_pos, const uint16_t* residual,
                                    uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  const coli_status st = check_dims_fp8(dims);
  if (st != COLI_OK) return st;
  if (T < 0) return COLI_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * (dims->top_k + dims->n_shared) > (int64_t(1) << 24)) return COLI_ERR_UNSUPPORTED;
  if (!w || !w->gate_q || !w->up_q || !w->down_q || !w->gate_s || !w->up_s || !w->down_s) return COLI_ERR_INVALID_ARG;
  if (T == 0) return COLI_OK;
  if (!x || !x_scale || !topk_ids || !topk_w || !unique_ids || !n_unique || !seg_off || !perm || !pair_pos || !out || !ws)
    return COLI_ERR_INVALID_ARG;
  const void* ps[9] = {w->gate_q, w->up_q, w->down_q, w->gate_s, w->up_s, w->down_s, x, out, residual};
  for (const void* p : ps)
    if (!aligned(p, 16)) return COLI_ERR_INVALID_ARG;
  if (!aligned(x_scale, 4) || !aligned(ws, 256)) return COLI_ERR_INVALID_ARG;
  const F8Ws lay = fp8_layout(dims, T, ws);
  if (ws_bytes < lay.bytes) return COLI_ERR_WORKSPACE;
  DevInfo di;
  if (dev_info(&di) != COLI_OK || !kernels_ready(di.dev, g_fp8_ready, fp8_kernels_ready)) return COLI_ERR_CUDA;
  const cudaStream_t s = as_stream(stream);
  const int H = dims->hidden, I = dims->inter, E = dims->n_experts, k = dims->top_k, S = dims->n_shared, P = T * k;
  F8Args g{};
  g.status = di.status;
  g.unique_ids = unique_ids;
  g.n_unique = n_unique;
  g.seg_off = seg_off;
  g.T = T;
  g.k = k;
  g.E = E;
  g.S = S;
  g.P = P;
  // Tiles of 32 tokens with gathered copies, or of 128 in pair order behind a gather
  // launch.  The short ones save that launch: one token of a layer of 64 experts (H 2048,
  // I 1024) 43 against 48 us, of 256 experts (H 6144, I 2048) 92 against 95, cold.  They
  // lose where more pairs come together: 64 tokens of the wide layer over 55 experts 532
  // against 461 us, 512 over 118 1882 against 989.  Between 4 and 32 tokens it depends on
  // the widths: 32 tokens 100 against 99 us in the small layer, 1183 against 1027 in the
  // wide one, where the long tiles would be 3 to 13 % faster.
  const bool few = T <= kF8Few;
  const int nt = few ? kF8Few : kF8Tokens;
  const int64_t blocks_ub = static_cast<int64_t>(std::min(P, E)) + P / nt + static_cast<int64_t>(S) * (T / nt + 1);
  const int64_t rows = static_cast<int64_t>(P) + static_cast<int64_t>(S) * T;
  // gate and up: token rows gathered by pair, h out
  CUtensorMap maps[7];
  if (few) {
    if (!fp8_maps(maps, w->gate_q, w->up_q, static_cast<int64_t>(E + S) * I, x, T, H)) return COLI_ERR_CUDA;
    g.a_s = x_scale;
    g.perm = perm;
    g.shared_row = 0;
  } else {
    const int64_t grows = static_cast<int64_t>(P) + (S ? T : 0);
    if (!launch(f8_gather_kernel, dim3(static_cast<unsigned>(std::min<int64_t>((grows + 7) / 8, 8L * di.sms))), dim3(256),
                0, s, x, x_scale, perm, k, P, S ? T : 0, T, H, lay.xg, lay.sg) ||
        !fp8_maps(maps, w->gate_q, w->up_q, static_cast<int64_t>(E + S) * I, lay.xg, grows, H))
      return COLI_ERR_CUDA;
    g.a_s = lay.sg;
    g.shared_row = P;
  }
  g.w_s = w->gate_s;
  g.w_s1 = w->up_s;
  g.out = lay.hq;
  g.out_s = lay.hs;
  g.R = I;
  g.nk = H / kF8Block;
  const int64_t tiles_gu = blocks_ub * (I / kF8Block);
  if (!(few ? launch_fp8<2, kF8Few, true>(maps, g, tiles_gu, 1, di.sms, s)
            : launch_fp8<2, kF8Tokens, true>(maps, g, tiles_gu, 1, di.sms, s)))
    return COLI_ERR_CUDA;
  // down: h rows in pair order, y out
  if (!fp8_maps(maps, w->down_q, nullptr, static_cast<int64_t>(E + S) * H, lay.hq, rows, I)) return COLI_ERR_CUDA;
  g.a_s = lay.hs;
  g.w_s = w->down_s;
  g.w_s1 = nullptr;
  g.out = lay.y;
  g.out_s = nullptr;
  g.out_f32 = 1;
  g.wide = 1;
  g.perm = nullptr;
  g.shared_row = -1;
  g.early = 1;
  g.R = H;
  g.nk = I / kF8Block;
  const int64_t tiles_dn = blocks_ub * (H / kF8Block);
  if (!(few ? launch_fp8<1, kF8Few, false>(maps, g, tiles_dn, 1, di.sms, s)
            : launch_fp8<2, kF8Tokens, false>(maps, g, (tiles_dn + 1) / 2, 1, di.sms, s)))
    return COLI_ERR_CUDA;
  const long work = static_cast<long>(T) * (H / 4);
  return launch(combine_kernel, dim3(static_cast<unsigned>(std::min<long>((work + 255) / 256, 16L * di.sms))), dim3(256),
                0, s, static_cast<const float*>(lay.y), pair_pos, topk_w, residual, T, k, S, H, out,
                static_cast<const int32_t*>(nullptr), 0, E, static_cast<float*>(nullptr))
             ? COLI_OK
             : COLI_ERR_CUDA;
}

}  // extern "C"
