// Load balance of the router: per-expert counts, the balance loss, and the
// gradient of the loss and of the renormalised weights with respect to the
// router logits.
//
//   l' = l + bias, p = softmax(l') over all E experts, n live tokens (mask != 0)
//   c_e = pairs (t, j) of live tokens with id e,  f_e = c_e / (n k)
//   P_e = sum_t p[t,e] / n,  L = E * sum_e f_e P_e   (1 for a uniform router)
//   dL/dl[t,e] = E/n * p[t,e] * (f_e - sum_i p[t,i] f_i)
//   dw/dl at the selected experts: w_j * (dw_j - sum_i w_i dw_i)
// f_e is piecewise constant and carries no gradient.  In the gradient any
// constant may be taken off every f_e; 1/E is, as (E c_e - n k) / (n k E) with an
// exact integer numerator, so that nearly balanced experts do not cancel.
//
// One warp owns a token's row: E <= 1024 values in registers, read once, the next
// token's row on its way.  Column sums (P, the bias gradient) are summed per warp
// in registers, then over a block's warps, then over the blocks, each in a fixed
// order: no float atomics.  Up to kBalFused tokens one cluster of 8 blocks does
// everything in one launch, adding over the blocks through distributed shared
// memory; larger batches write their blocks' sums to the workspace and a second
// launch adds them.
// The column sums are fp32: up to 4736 warps share the tokens, so that a chain is T /
// 4736 + 51 additions long (65536 x 256: all outputs within 7.3e-8 of the 64-bit ones,
// relative to their norm; a form whose sums are 64-bit is within 5.2e-8).  Sums in 64
// bits would double the registers that hold them.
// Bound by HBM (4 bytes per logit read forward; 4 read and 4 written backward) for
// large batches and by latency for small ones.  65536 x 256, top-8: 68 us for both
// passes with the bias gradient (210 MB), 27 forward and 40 backward; under a profiler,
// each launch alone and cold, 27 + 10 and 40 + 6.  64 x 256: 5.0 and 5.2 us.
#pragma once
#include "common.cuh"

namespace coli {

constexpr int kBalWarps = 16;          // per block
constexpr int kBalCluster = 8;
constexpr int kBalFused = 256;         // tokens: two rows per warp of the cluster
constexpr int kBalMaxBlocks = 296;     // two per SM

__device__ __forceinline__ void bal_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t bal_cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The 32 bits at this block's shared address p in block `rank` of the cluster.
__device__ __forceinline__ uint32_t bal_peer(const void* p, uint32_t rank) {
  uint32_t a, v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Warp-wide sum and maximum, the same value in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  // as integers of the same order: one instruction over the warp
  const uint32_t u = __float_as_uint(v);
  const uint32_t m = __reduce_max_sync(0xffffffffu, (u & 0x80000000u) ? ~u : (u | 0x80000000u));
  return __uint_as_float((m & 0x80000000u) ? (m & 0x7fffffffu) : ~m);
}

// Lane `lane` holds experts e(q) = (q / VEC * 32 + lane) * VEC + q % VEC of a row.
template <int VEC>
__device__ __forceinline__ int bal_expert(int q, int lane) {
  return (q / VEC * 32 + lane) * VEC + q % VEC;
}

// A lane's share of a row of E floats (`fill` past the end).  Plain loads: the
// backward may write its gradient over the logits.
template <int NV, int VEC>
__device__ __forceinline__ void bal_load(const float* row, int E, int lane, float fill, float (&v)[NV]) {
#pragma unroll
  for (int q = 0; q < NV; q += VEC) {
    const int e = bal_expert<VEC>(q, lane);
    if (VEC == 4) {
      const float4 x = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(fill, fill, fill, fill);
      v[q] = x.x;
      v[q + 1 < NV ? q + 1 : q] = x.y;
      v[q + 2 < NV ? q + 2 : q] = x.z;
      v[q + 3 < NV ? q + 3 : q] = x.w;
    } else {
      v[q] = e < E ? row[e] : fill;
    }
  }
}

// Softmax of a token's row in place.  NaN counts as -inf; an expert at +inf
// shares the whole mass with the others at +inf; a row with nothing above -inf
// gets p = 0 everywhere.  Returns whether the row held NaN or +inf.
template <int NV>
__device__ __forceinline__ bool bal_softmax(float (&v)[NV], const float (&b)[NV]) {
  bool bad = false;
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    v[q] += b[q];
    if (isnan(v[q])) {
      bad = true;
      v[q] = -INFINITY;
    }
    m = fmaxf(m, v[q]);
  }
  m = warp_max(m);
  bad |= m == INFINITY;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    v[q] = m == -INFINITY ? 0.f : v[q] == m ? 1.f : expf(v[q] - m);
    s += v[q];
  }
  s = warp_sum(s);
  const float r = s > 0.f ? 1.f / s : 0.f;
#pragma unroll
  for (int q = 0; q < NV; ++q) v[q] *= r;
  return bad;
}

// Adds the kBalWarps warps' column sums in warp order: thread e gets columns e,
// e + blockDim.x ..  `sm` holds E floats per warp; fn(e, sum) takes each.
template <int NV, int VEC, typename F>
__device__ __forceinline__ void bal_block_columns(const float (&acc)[NV], int E, float* sm, F fn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int e = bal_expert<VEC>(q, lane);
    if (e < E) sm[warp * E + e] = acc[q];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBalWarps; ++w) s += sm[w * E + e];
    fn(e, s);
  }
}

// What is left of one expert once its column sum p and count c are known; its term of the loss.
__device__ __forceinline__ double bal_expert_out(float p, int c, int n, int k, int32_t* counts, float* prob_mean) {
  const float mean = n > 0 ? p / static_cast<float>(n) : 0.f;
  *counts = c;
  *prob_mean = mean;
  return n > 0 ? static_cast<double>(c) * mean / (static_cast<double>(n) * k) : 0.0;
}

// Sum of v over a block of NT threads in a fixed order (valid in thread 0); `sm`: NT / 32 doubles.
template <int NT>
__device__ __forceinline__ double bal_block_sum(double v, double* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < NT / 32; ++w) s += sm[w];
  return s;
}

// Adds the cluster's loss terms in rank order and writes the loss.  Ends with a
// cluster barrier: the peers' shared memory is read before it.
__device__ __forceinline__ void bal_cluster_loss(double mine, double* slot, int E, int n, float* loss, int32_t* n_live) {
  if (threadIdx.x == 0) *slot = mine;
  bal_cluster_sync();
  if (bal_cluster_rank() == 0 && threadIdx.x == 0) {
    double s = 0.0;
    for (int r = 0; r < kBalCluster; ++r) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(slot);
      s += __hiloint2double(static_cast<int>(bal_peer(p + 1, r)), static_cast<int>(bal_peer(p, r)));
    }
    *loss = static_cast<float>(E * s);
    *n_live = n;
  }
  bal_cluster_sync();
}

struct BalOut {
  int32_t* counts;
  int32_t* n_live;
  float* prob_mean;
  float* loss;
};

// Forward: each block's sums of p, pair counts and live tokens.  With `fused` the
// grid is one cluster, which goes on to the results; otherwise they are left in
// part_*.  Dynamic shared memory: (kBalWarps + 1) * E words.
template <int NV, int VEC>
__global__ void __launch_bounds__(kBalWarps * 32, NV <= 8 ? 2 : 1)
    balance_kernel(const float* __restrict__ logits, const float* __restrict__ bias, const int32_t* __restrict__ ids,
                   const uint8_t* __restrict__ mask, int T, int E, int k, int fused, float* __restrict__ part_p,
                   int32_t* __restrict__ part_c, int32_t* __restrict__ part_n, BalOut out,
                   uint32_t* __restrict__ status) {
  extern __shared__ float bal_sm[];
  int32_t* hist = reinterpret_cast<int32_t*>(bal_sm + kBalWarps * E);
  __shared__ int live_n;
  __shared__ double loss_sm[kBalWarps + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  if (threadIdx.x == 0) live_n = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  constexpr bool AHEAD = NV < 32;      // registers for the next row
  float b[NV], acc[NV], v[NV], nx[AHEAD ? NV : 1];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    b[q] = 0.f;
    acc[q] = 0.f;
  }
  if (bias) bal_load<NV, VEC>(bias, E, lane, 0.f, b);
  uint32_t flags = 0;
  int live = 0, id = 0, idn = 0;
  bool on = false, onn = false;
  const int step = gridDim.x * kBalWarps;
  auto fetch = [&](int t) {
    onn = t < T && (!mask || mask[t] != 0);
    if (onn) {
      if constexpr (AHEAD) bal_load<NV, VEC>(logits + static_cast<size_t>(t) * E, E, lane, -INFINITY, nx);
      if (lane < k) idn = __ldg(ids + static_cast<size_t>(t) * k + lane);
    }
  };
  const int t0 = blockIdx.x * kBalWarps + warp;
  fetch(t0);
  for (int t = t0; t < T; t += step) {
    on = onn;
    id = idn;
    if constexpr (AHEAD) {
#pragma unroll
      for (int q = 0; q < NV; ++q) v[q] = nx[q];
    } else if (on) {
      bal_load<NV, VEC>(logits + static_cast<size_t>(t) * E, E, lane, -INFINITY, v);
    }
    fetch(t + step);
    if (!on) continue;
    if (lane < k) {
      if (id >= 0 && id < E)
        atomicAdd(hist + id, 1);
      else
        flags |= COLI_FLAG_BAD_ID;
    }
    if (bal_softmax<NV>(v, b)) flags |= COLI_FLAG_NONFINITE;
#pragma unroll
    for (int q = 0; q < NV; ++q) acc[q] += v[q];
    ++live;
  }
  if (lane == 0 && live) atomicAdd(&live_n, live);
  if (flags) atomicOr(status, flags);
  if (!fused) {
    // the barrier inside also covers hist and live_n
    bal_block_columns<NV, VEC>(acc, E, bal_sm, [&](int e, float s) {
      part_p[static_cast<size_t>(blockIdx.x) * E + e] = s;
      part_c[static_cast<size_t>(blockIdx.x) * E + e] = hist[e];
    });
    if (threadIdx.x == 0) part_n[blockIdx.x] = live_n;
    return;
  }
  // block sums over warp 0's row (each thread reads and writes its own columns)
  bal_block_columns<NV, VEC>(acc, E, bal_sm, [&](int e, float s) { bal_sm[e] = s; });
  bal_cluster_sync();
  const uint32_t rank = bal_cluster_rank();
  int n = 0;
  for (int r = 0; r < kBalCluster; ++r) n += static_cast<int>(bal_peer(&live_n, r));
  double term = 0.0;
  for (int e = rank + kBalCluster * threadIdx.x; e < E; e += kBalCluster * blockDim.x) {
    float p = 0.f;
    int c = 0;
    for (int r = 0; r < kBalCluster; ++r) {
      p += __uint_as_float(bal_peer(bal_sm + e, r));
      c += static_cast<int>(bal_peer(hist + e, r));
    }
    term += bal_expert_out(p, c, n, k, out.counts + e, out.prob_mean + e);
  }
  term = bal_block_sum<kBalWarps * 32>(term, loss_sm);
  bal_cluster_loss(term, loss_sm + kBalWarps, E, n, out.loss, out.n_live);
}

constexpr int kBalGroup = 16;          // warps that share a column's rows in the second passes

// Second pass of the forward (one cluster): the blocks' rows added in a fixed
// order, then the results.
__global__ void __launch_bounds__(512)
    balance_finish_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                          const int32_t* __restrict__ part_n, int blocks, int E, int k, BalOut out) {
  __shared__ float ps[kBalGroup][33];
  __shared__ int cs[kBalGroup][33];
  __shared__ double loss_sm[17];
  __shared__ int n_sm;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int n = 0;
    for (int i = lane; i < blocks; i += 32) n += part_n[i];
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) n_sm = n;
  }
  double term = 0.0;
  // 32 neighbouring columns at a time (rows of 128 bytes), a warp per row group
  for (int e0 = 32 * static_cast<int>(bal_cluster_rank()); e0 < E; e0 += 32 * kBalCluster) {
    const int e = e0 + lane;
    float p = 0.f;
    int c = 0;
    if (e < E) {
#pragma unroll 4
      for (int i = warp; i < blocks; i += kBalGroup) {
        p += part_p[static_cast<size_t>(i) * E + e];
        c += part_c[static_cast<size_t>(i) * E + e];
      }
    }
    ps[warp][lane] = p;
    cs[warp][lane] = c;
    __syncthreads();
    if (warp == 0 && e < E) {
      p = 0.f;
      c = 0;
#pragma unroll
      for (int w = 0; w < kBalGroup; ++w) {
        p += ps[w][lane];
        c += cs[w][lane];
      }
      term += bal_expert_out(p, c, n_sm, k, out.counts + e, out.prob_mean + e);
    }
    __syncthreads();
  }
  __syncthreads();
  const int n = n_sm;
  term = bal_block_sum<512>(term, loss_sm);
  bal_cluster_loss(term, loss_sm + 16, E, n, out.loss, out.n_live);
}

// Backward: d_logits, and the column sums when d_bias is not NULL: with `fused`
// (one cluster) added over the blocks here, otherwise left in part_b.  Dynamic
// shared memory: kBalWarps * E floats (a row of the selected experts' terms per
// warp, then the column sums).
template <int NV, int VEC>
__global__ void __launch_bounds__(kBalWarps * 32, NV <= 8 ? 2 : 1)
    balance_backward_kernel(const float* logits, const float* __restrict__ bias, const uint8_t* __restrict__ mask,
                            const int32_t* __restrict__ counts, const int32_t* __restrict__ n_live,
                            const float* __restrict__ grad_loss, const int32_t* __restrict__ ids,
                            const float* __restrict__ w, const float* __restrict__ d_w, int T, int E, int k, int fused,
                            float* d_logits, float* __restrict__ part_b, float* __restrict__ d_bias) {
  extern __shared__ float bal_sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* sel = bal_sm + warp * E;      // zero between tokens
  for (int e = lane; e < E; e += 32) sel[e] = 0.f;
  pdl_wait();
  pdl_trigger();
  __syncwarp();
  const int n = __ldg(n_live);
  const long long nk = static_cast<long long>(n) * k;
  const float coef = grad_loss && n > 0 ? __ldg(grad_loss) * static_cast<float>(E) / static_cast<float>(n) : 0.f;
  const float fscale = n > 0 ? static_cast<float>(1.0 / (static_cast<double>(nk) * E)) : 0.f;
  constexpr bool AHEAD = NV < 32;      // registers for the next row
  float b[NV], f[NV], acc[NV], v[NV], nx[AHEAD ? NV : 1];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int e = bal_expert<VEC>(q, lane);
    b[q] = 0.f;
    acc[q] = 0.f;
    f[q] = e < E ? static_cast<float>(static_cast<long long>(E) * __ldg(counts + e) - nk) * fscale : 0.f;
  }
  if (bias) bal_load<NV, VEC>(bias, E, lane, 0.f, b);
  bool on = false, onn = false;
  int id = -1, idn = -1;
  float wj = 0.f, dj = 0.f, wn = 0.f, dn = 0.f;
  const int step = gridDim.x * kBalWarps;
  auto fetch = [&](int t) {
    onn = t < T && (!mask || mask[t] != 0);
    if (!onn) return;
    if constexpr (AHEAD) {
      if (coef != 0.f) bal_load<NV, VEC>(logits + static_cast<size_t>(t) * E, E, lane, -INFINITY, nx);
    }
    if (d_w && lane < k) {
      const size_t at = static_cast<size_t>(t) * k + lane;
      idn = __ldg(ids + at);
      wn = __ldg(w + at);
      dn = __ldg(d_w + at);
    }
  };
  const int t0 = blockIdx.x * kBalWarps + warp;
  fetch(t0);
  for (int t = t0; t < T; t += step) {
    on = onn;
    id = idn;
    wj = wn;
    dj = dn;
    if constexpr (AHEAD) {
#pragma unroll
      for (int q = 0; q < NV; ++q) v[q] = nx[q];
    } else if (on && coef != 0.f) {
      bal_load<NV, VEC>(logits + static_cast<size_t>(t) * E, E, lane, -INFINITY, v);
    }
    fetch(t + step);
    if (on && coef != 0.f) {
      bal_softmax<NV>(v, b);
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < NV; ++q) s = fmaf(v[q], f[q], s);
      s = warp_sum(s);
#pragma unroll
      for (int q = 0; q < NV; ++q) v[q] = coef * v[q] * (f[q] - s);
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q) v[q] = 0.f;
    }
    if (on && d_w) {
      const float sj = wj * (dj - warp_sum(wj * dj));
      const bool mine = lane < k && static_cast<unsigned>(id) < static_cast<unsigned>(E);
      // the selected experts' terms through a row of shared memory; the same
      // expert twice is added in slot order
      const unsigned same = __match_any_sync(0xffffffffu, mine ? id : -1 - lane);
      if (__any_sync(0xffffffffu, (same & (same - 1)) != 0)) {
        for (int j = 0; j < k; ++j) {
          if (lane == j && mine) sel[id] += sj;
          __syncwarp();
        }
      } else if (mine) {
        sel[id] = sj;
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < NV; q += VEC) {
        const int e = bal_expert<VEC>(q, lane);
        if (e < E) {
          if (VEC == 4) {
            const float4 x = *reinterpret_cast<const float4*>(sel + e);
            v[q] += x.x;
            v[q + 1 < NV ? q + 1 : q] += x.y;
            v[q + 2 < NV ? q + 2 : q] += x.z;
            v[q + 3 < NV ? q + 3 : q] += x.w;
          } else {
            v[q] += sel[e];
          }
        }
      }
      __syncwarp();
      if (mine) sel[id] = 0.f;
      __syncwarp();
    }
#pragma unroll
    for (int q = 0; q < NV; ++q) acc[q] += v[q];
    float* row = d_logits + static_cast<size_t>(t) * E;
#pragma unroll
    for (int q = 0; q < NV; q += VEC) {
      const int e = bal_expert<VEC>(q, lane);
      if (e < E) {
        if (VEC == 4)
          *reinterpret_cast<float4*>(row + e) =
              make_float4(v[q], v[q + 1 < NV ? q + 1 : q], v[q + 2 < NV ? q + 2 : q], v[q + 3 < NV ? q + 3 : q]);
        else
          row[e] = v[q];
      }
    }
  }
  if (!d_bias) return;
  if (!fused) {
    bal_block_columns<NV, VEC>(acc, E, bal_sm,
                               [&](int e, float s) { part_b[static_cast<size_t>(blockIdx.x) * E + e] = s; });
    return;
  }
  bal_block_columns<NV, VEC>(acc, E, bal_sm, [&](int e, float s) { bal_sm[e] = s; });
  bal_cluster_sync();
  for (int e = bal_cluster_rank() + kBalCluster * threadIdx.x; e < E; e += kBalCluster * blockDim.x) {
    float s = 0.f;
    for (int r = 0; r < kBalCluster; ++r) s += __uint_as_float(bal_peer(bal_sm + e, r));
    d_bias[e] = s;
  }
  bal_cluster_sync();
}

// d_bias: the blocks' column sums added in a fixed order, 32 columns a block.
__global__ void __launch_bounds__(512) balance_bias_kernel(const float* __restrict__ part_b, int blocks, int E,
                                                           float* __restrict__ d_bias) {
  __shared__ float ps[kBalGroup][33];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int e = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (e < E) {
#pragma unroll 4
    for (int i = warp; i < blocks; i += kBalGroup) s += part_b[static_cast<size_t>(i) * E + e];
  }
  ps[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && e < E) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kBalGroup; ++w) s += ps[w][lane];
    d_bias[e] = s;
  }
}

}  // namespace coli
