// Matrix product of e4m3 codes with an fp32 scale for each block of 128, dense
// and over the experts of a routed batch.
//
//   out[m][n] = sum_b sa[m][b] * sw[n / 128][b] * sum_{k in block b} a[m][k] w[n][k]
// a: rows of codes with one scale per row and 128 columns; w: one scale per 128
// rows x 128 columns.  Each block's products are summed in fp32, then scaled and
// added to the fp32 total in block order.
#pragma once
#include "common.cuh"
#include "k_norm_fp8.cuh"

namespace coli {

constexpr int kF8MaxSeg = 1024 + 8;   // unique routed + shared segments

// What a launch multiplies: one dense product (seg_off NULL), or the segments of
// a routed batch: the union's experts over their pairs, then the S shared experts
// over all T tokens.  Weights of expert e start at row e * R of w.
struct F8Gemm {
  const uint8_t* a;        // [rows][K] codes
  const float* a_s;        // [rows][ceil(K / 128)]
  const uint8_t* w;        // [experts * R][K]
  const float* w_s;        // [experts][ceil(R / 128)][ceil(K / 128)]
  void* out;               // [rows][R] bf16 or fp32
  int M, R, K;             // dense rows; output columns of one expert; K
  int out_f32;
  const int32_t* unique_ids;
  const int32_t* n_unique;
  const int32_t* seg_off;
  const int32_t* perm;
  int T, k, E, S, P;
  int gather;              // rows of a: token of the pair (perm / k), else the pair's own row
};

// First version: one block per 64 rows x 64 columns, codes widened to fp32 in
// shared memory, a 4 x 4 register tile per thread.  Right for every case, far
// from any bound.
__global__ void __launch_bounds__(256) fp8_gemm_simple_kernel(F8Gemm g) {
  __shared__ float as[32][65], ws[32][65];
  __shared__ int tile[4];   // expert, first pair row, rows, first a row (or -1: gathered)
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (tid == 0) {
    int blk = blockIdx.x, e = -1, row0 = 0, rows = 0, arow = 0;
    if (!g.seg_off) {
      e = 0;
      row0 = blk * 64;
      rows = min(64, g.M - row0);
      arow = row0;
    } else {
      const int U = *g.n_unique;
      for (int s = 0; s < U + g.S; ++s) {
        const int base = s < U ? g.seg_off[s] : g.P + (s - U) * g.T;
        const int cnt = s < U ? g.seg_off[s + 1] - base : g.T;
        const int nb = (cnt + 63) / 64;
        if (blk < nb) {
          e = s < U ? g.unique_ids[s] : g.E + (s - U);
          row0 = base + blk * 64;
          rows = min(64, cnt - blk * 64);
          arow = g.gather ? (s < U ? -1 : blk * 64) : row0;
          break;
        }
        blk -= nb;
      }
    }
    tile[0] = e;
    tile[1] = row0;
    tile[2] = rows;
    tile[3] = arow;
  }
  __syncthreads();
  const int e = tile[0], row0 = tile[1], rows = tile[2], arow = tile[3];
  if (e < 0) return;
  const int n0 = blockIdx.y * 64;
  const int nkb = (g.K + kF8Block - 1) / kF8Block, nrb = (g.R + kF8Block - 1) / kF8Block;
  const int ty = tid >> 4, tx = tid & 15;
  float acc[4][4] = {};
  auto a_row = [&](int m) -> size_t {
    return arow < 0 ? static_cast<size_t>(g.perm[row0 + m] / g.k) : static_cast<size_t>(arow + m);
  };
  for (int kb = 0; kb < nkb; ++kb) {
    float part[4][4] = {};
    for (int k0 = kb * kF8Block; k0 < min(g.K, (kb + 1) * kF8Block); k0 += 32) {
      for (int i = tid; i < 64 * 32; i += 256) {
        const int m = i >> 5, kk = i & 31;
        float av = 0.f, wv = 0.f;
        if (k0 + kk < g.K) {
          __nv_fp8_e4m3 c;
          if (m < rows) {
            c.__x = g.a[a_row(m) * g.K + k0 + kk];
            av = static_cast<float>(c);
          }
          if (n0 + m < g.R) {
            c.__x = g.w[(static_cast<size_t>(e) * g.R + n0 + m) * g.K + k0 + kk];
            wv = static_cast<float>(c);
          }
        }
        as[kk][m] = av;
        ws[kk][m] = wv;
      }
      __syncthreads();
      for (int kk = 0; kk < 32; ++kk)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(as[kk][ty * 4 + i], ws[kk][tx * 4 + j], part[i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
      const int m = ty * 4 + i;
      const float sa = m < rows ? g.a_s[a_row(m) * nkb + kb] : 0.f;
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n < g.R) acc[i][j] = fmaf(part[i][j], sa * g.w_s[(static_cast<size_t>(e) * nrb + n / kF8Block) * nkb + kb], acc[i][j]);
      }
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= rows || n >= g.R) continue;
      const size_t at = static_cast<size_t>(row0 + m) * g.R + n;
      if (g.out_f32)
        static_cast<float*>(g.out)[at] = acc[i][j];
      else
        static_cast<uint16_t*>(g.out)[at] = float_to_bf16_bits(acc[i][j]);
    }
}

// h = silu(gate) * up of fp32 rows, as e4m3 codes with a scale per 128 columns:
// one warp per (row, block).
__global__ void __launch_bounds__(256) swiglu_fp8_kernel(const float* __restrict__ gate, const float* __restrict__ up,
                                                         long blocks, uint8_t* __restrict__ hq,
                                                         float* __restrict__ hs) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  for (long b = blockIdx.x * 8L + (threadIdx.x >> 5); b < blocks; b += gridDim.x * 8L) {
    const float4 gv = reinterpret_cast<const float4*>(gate)[b * 32 + lane];
    const float4 uv = reinterpret_cast<const float4*>(up)[b * 32 + lane];
    auto h1 = [](float x, float y) { return x / (1.0f + expf(-x)) * y; };
    const float h[4] = {h1(gv.x, uv.x), h1(gv.y, uv.y), h1(gv.z, uv.z), h1(gv.w, uv.w)};
    float m = max_nan(max_nan(fabsf(h[0]), fabsf(h[1])), max_nan(fabsf(h[2]), fabsf(h[3])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    const float sc = f8_scale(m, &inv);
    if (lane == 0) hs[b] = sc;
    reinterpret_cast<uint32_t*>(hq)[b * 32 + lane] = f8x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
  }
}

}  // namespace coli
