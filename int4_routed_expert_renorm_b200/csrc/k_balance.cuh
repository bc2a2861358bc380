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
// One warp owns a token's row: E <= 1024 values in registers, read once.  The
// kernels are bound by HBM (4 bytes per logit read forward; 4 read and 4
// written backward) for large batches and by launch latency for small ones.
// Column sums (P, the bias gradient) are summed per warp in registers, then over
// a block's warps, then over the blocks, each in a fixed order: no float atomics.
#pragma once
#include "common.cuh"

namespace coli {

constexpr int kBalWarps = 8;

// Warp-wide sum and maximum, the same value in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
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

// Adds the kBalWarps warps' column sums in warp order and writes the block's
// row of `part` ([blocks][E]).  `sm` holds E floats per warp.
template <int NV, int VEC>
__device__ __forceinline__ void bal_block_columns(const float (&acc)[NV], int E, float* sm, float* __restrict__ part) {
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
    part[static_cast<size_t>(blockIdx.x) * E + e] = s;
  }
}

// Forward, first pass: each block's sums of p, pair counts and live tokens.
// Dynamic shared memory: (kBalWarps + 1) * E words.
template <int NV, int VEC>
__global__ void __launch_bounds__(kBalWarps * 32)
    balance_partial_kernel(const float* __restrict__ logits, const float* __restrict__ bias,
                           const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int T, int E, int k,
                           float* __restrict__ part_p, int32_t* __restrict__ part_c, int32_t* __restrict__ part_n,
                           uint32_t* __restrict__ status) {
  extern __shared__ float bal_sm[];
  int32_t* hist = reinterpret_cast<int32_t*>(bal_sm + kBalWarps * E);
  __shared__ int live_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
  if (threadIdx.x == 0) live_n = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  float b[NV], acc[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    b[q] = 0.f;
    acc[q] = 0.f;
  }
  if (bias) bal_load<NV, VEC>(bias, E, lane, 0.f, b);
  uint32_t flags = 0;
  int live = 0;
  for (int t = blockIdx.x * kBalWarps + warp; t < T; t += gridDim.x * kBalWarps) {
    if (mask && mask[t] == 0) continue;
    float v[NV];
    bal_load<NV, VEC>(logits + static_cast<size_t>(t) * E, E, lane, -INFINITY, v);
    if (lane < k) {
      const int id = __ldg(ids + static_cast<size_t>(t) * k + lane);
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
  bal_block_columns<NV, VEC>(acc, E, bal_sm, part_p);   // its barrier also covers hist and live_n
  for (int e = threadIdx.x; e < E; e += blockDim.x) part_c[static_cast<size_t>(blockIdx.x) * E + e] = hist[e];
  if (threadIdx.x == 0) part_n[blockIdx.x] = live_n;
}

// Forward, second pass (one block of 1024 threads): the blocks' rows added in
// block order; counts, mean probabilities, live tokens and the loss.
__global__ void __launch_bounds__(1024)
    balance_finish_kernel(const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                          const int32_t* __restrict__ part_n, int blocks, int E, int k, int32_t* __restrict__ counts,
                          int32_t* __restrict__ n_live, float* __restrict__ prob_mean, float* __restrict__ loss) {
  __shared__ double sm[32];
  __shared__ int n_sm;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < 32) {
    int n = 0;
    for (int i = threadIdx.x; i < blocks; i += 32) n += part_n[i];
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x == 0) n_sm = n;
  }
  __syncthreads();
  const int n = n_sm;
  const int e = threadIdx.x;
  double term = 0.0;
  if (e < E) {
    float p = 0.f;
    int c = 0;
    for (int i = 0; i < blocks; ++i) {
      p += part_p[static_cast<size_t>(i) * E + e];
      c += part_c[static_cast<size_t>(i) * E + e];
    }
    const float mean = n > 0 ? p / static_cast<float>(n) : 0.f;
    counts[e] = c;
    prob_mean[e] = mean;
    term = n > 0 ? static_cast<double>(c) * mean / (static_cast<double>(n) * k) : 0.0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < 32; ++w) s += sm[w];
    *loss = static_cast<float>(E * s);
    *n_live = n;
  }
}

// Backward: d_logits, and each block's column sums when part_b is not NULL.
// Dynamic shared memory: kBalWarps * E floats when part_b is not NULL.
template <int NV, int VEC>
__global__ void __launch_bounds__(kBalWarps * 32)
    balance_backward_kernel(const float* logits, const float* __restrict__ bias,
                            const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
                            const int32_t* __restrict__ n_live, const float* __restrict__ grad_loss,
                            const int32_t* __restrict__ ids, const float* __restrict__ w,
                            const float* __restrict__ d_w, int T, int E, int k, float* d_logits,
                            float* __restrict__ part_b) {
  extern __shared__ float bal_sm[];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = __ldg(n_live);
  const long long nk = static_cast<long long>(n) * k;
  const float coef = grad_loss && n > 0 ? __ldg(grad_loss) * static_cast<float>(E) / static_cast<float>(n) : 0.f;
  const float fscale = n > 0 ? static_cast<float>(1.0 / (static_cast<double>(nk) * E)) : 0.f;
  float b[NV], f[NV], acc[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int e = bal_expert<VEC>(q, lane);
    b[q] = 0.f;
    acc[q] = 0.f;
    f[q] = e < E ? static_cast<float>(static_cast<long long>(E) * __ldg(counts + e) - nk) * fscale : 0.f;
  }
  if (bias) bal_load<NV, VEC>(bias, E, lane, 0.f, b);
  for (int t = blockIdx.x * kBalWarps + warp; t < T; t += gridDim.x * kBalWarps) {
    float v[NV];
    if (mask && mask[t] == 0) {
#pragma unroll
      for (int q = 0; q < NV; ++q) v[q] = 0.f;
    } else {
      if (coef != 0.f) {
        bal_load<NV, VEC>(logits + static_cast<size_t>(t) * E, E, lane, -INFINITY, v);
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
      if (d_w) {
        const size_t at = static_cast<size_t>(t) * k + lane;
        const int id = lane < k ? __ldg(ids + at) : -1;
        const float wj = lane < k ? __ldg(w + at) : 0.f;
        const float dj = lane < k ? __ldg(d_w + at) : 0.f;
        const float sj = wj * (dj - warp_sum(wj * dj));
        for (int j = 0; j < k; ++j) {
          const int ej = __shfl_sync(0xffffffffu, id, j);
          const float gj = __shfl_sync(0xffffffffu, sj, j);
#pragma unroll
          for (int q = 0; q < NV; ++q)
            if (bal_expert<VEC>(q, lane) == ej) v[q] += gj;
        }
      }
#pragma unroll
      for (int q = 0; q < NV; ++q) acc[q] += v[q];
    }
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
  if (part_b) bal_block_columns<NV, VEC>(acc, E, bal_sm, part_b);
}

// d_bias[e] = the blocks' column sums added in block order.
__global__ void __launch_bounds__(256) balance_bias_kernel(const float* __restrict__ part_b, int blocks, int E,
                                                           float* __restrict__ d_bias) {
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= E) return;
  float s = 0.f;
  for (int i = 0; i < blocks; ++i) s += part_b[static_cast<size_t>(i) * E + e];
  d_bias[e] = s;
}

}  // namespace coli
