// Residual addition, root-mean-square norm and 8-bit rows with block scales.
//
//   s = bf16(x + r)                      (s = x without a residual)
//   n = s * (mean(s^2) + eps)^(-1/2) * g (g = 1 without a weight), in fp32
//   per 128 columns: c = max(max|n| / 448, 2^-126),  q = e4m3(n / c)
// 448 is e4m3's largest value, so the block's largest |n| lands on it.  The
// codes are rounded from the unrounded n, not from its bf16 copy.  The floor 2^-126
// keeps the scale a normal number for blocks of zeros.
// The root cancels in n / c: q = e4m3(s g * (448 / max|s g|)).  s g (two bf16 numbers)
// is exact in fp32, so a code sees two roundings before its own, the block's quotient
// and the product; from n and c it would see six, and a value near a border of the
// codes would land on the wrong side more often.  (A division per value would leave
// one, and costs 176 against 141 us at 16384 x 6144.)
//
// One block of 256 threads per row; a thread holds 8 consecutive values per 2048
// columns (one 16-byte load), so a 128-column block is 16 neighbouring lanes and
// its maximum a 4-step shuffle.  The row is read once and stays in registers.
// Bound by HBM for large batches (9.03 bytes per value with everything written)
// and by latency for single tokens (1 x 6144: 3.6 us).  16384 x 6144 with residual,
// weight and all outputs: 137 us on one set of buffers, 6.6 TB/s, 146 us with others
// from pass to pass (five blocks per SM; with four 3.5 % more).
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace coli {

constexpr int kF8Block = 128;           // columns (and weight rows) per scale
constexpr float kF8Max = 448.0f;        // largest e4m3 value
constexpr float kF8MinScale = 1.17549435e-38f;   // 2^-126

// max(a, b) that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The scale of a block whose largest magnitude is m, and its inverse.
__device__ __forceinline__ float f8_scale(float m, float* inv) {
  const float c = max_nan(m / kF8Max, kF8MinScale);
  *inv = 1.0f / c;
  return c;
}

// Four values as e4m3 bytes (round to nearest even, saturating, NaN kept).
__device__ __forceinline__ uint32_t f8x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  return float_to_bf16_bits(a) | (static_cast<uint32_t>(float_to_bf16_bits(b)) << 16);
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* weight;
  float eps;
  int H;
  uint16_t* sum_out;
  uint16_t* norm_out;
  uint8_t* q;
  float* q_scale;
  uint32_t* status;
};

// The rest of a block's row whose mean of squares plus eps is no normal fp32 number
// (values past 1e19 whose squares overflow, values below 1e-19 with next to no eps, a
// row of zeros with eps = 0, infinities, NaN): sum, root and n in 64 bits, where the
// squares of bf16 numbers neither overflow nor vanish.  n of a row of zeros is 0
// whatever eps.
__device__ __forceinline__ void norm_row_wide(const NormArgs& a) {
  __shared__ double wide_sm[8];
  const int tid = threadIdx.x;
  const size_t row = static_cast<size_t>(blockIdx.x) * a.H;
  auto value = [&](int c) -> double {
    if (a.sum_out) return bf16_bits_to_float(a.sum_out[row + c]);      // this thread wrote it
    const float v = bf16_bits_to_float(a.x[row + c]);
    return a.residual ? bf16_bits_to_float(float_to_bf16_bits(v + bf16_bits_to_float(a.residual[row + c]))) : v;
  };
  double ss = 0.0;
#pragma unroll 1
  for (int c = tid * 8; c < a.H; c += 2048)
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const double v = value(c + k);
      ss += v * v;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((tid & 31) == 0) wide_sm[tid >> 5] = ss;
  __syncthreads();
  ss = 0.0;
#pragma unroll 1
  for (int w = 0; w < 8; ++w) ss += wide_sm[w];
  if (tid == 0 && !(ss < INFINITY)) atomicOr(a.status, COLI_FLAG_NONFINITE);
  const double ms = ss / a.H + static_cast<double>(a.eps);
  const double rs = ms == 0.0 ? 0.0 : 1.0 / sqrt(ms);
  auto n_at = [&](int c) {
    return static_cast<float>(value(c) * rs * (a.weight ? static_cast<double>(bf16_bits_to_float(a.weight[c])) : 1.0));
  };
  // as many rounds for every thread: a block's maximum is over 16 lanes
#pragma unroll 1
  for (int c0 = 0; c0 < a.H; c0 += 2048) {
    const int c = c0 + tid * 8;
    float m = 0.f;
    if (c < a.H)
#pragma unroll 1
      for (int k = 0; k < 8; ++k) m = max_nan(m, fabsf(n_at(c + k)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (c >= a.H) continue;
    float inv;
    const float sc = f8_scale(m, &inv);
    if ((tid & 15) == 0) a.q_scale[(row + c) / kF8Block] = sc;
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      const float z = n_at(c + k);
      a.q[row + c + k] = static_cast<uint8_t>(f8x4(z * inv, 0.f, 0.f, 0.f));
      if (a.norm_out) a.norm_out[row + c + k] = float_to_bf16_bits(z);
    }
  }
}

// NC: 2048-column steps of a row (H <= 2048 * NC).  x, residual and sum_out may
// be the same buffer: a thread reads its values before it writes them.
template <int NC>
__global__ void __launch_bounds__(256, NC <= 1 ? 8 : NC <= 3 ? 5 : 1)
    add_rmsnorm_fp8_kernel(const __grid_constant__ NormArgs a) {
  const uint16_t* x = a.x;
  const uint16_t* residual = a.residual;
  const uint16_t* weight = a.weight;
  uint16_t* sum_out = a.sum_out;
  uint16_t* norm_out = a.norm_out;
  uint8_t* q = a.q;
  float* q_scale = a.q_scale;
  const int H = a.H;
  __shared__ float sm[8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t row = static_cast<size_t>(blockIdx.x) * H;
  uint4 v[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * 256 + tid) * 8;
    v[i] = c < H ? *reinterpret_cast<const uint4*>(x + row + c) : make_uint4(0, 0, 0, 0);
  }
  if (residual) {
    uint4 r[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * 256 + tid) * 8;
      r[i] = c < H ? *reinterpret_cast<const uint4*>(residual + row + c) : make_uint4(0, 0, 0, 0);
    }
    auto add2 = [](uint32_t a, uint32_t b) {
      return bf16x2(__uint_as_float(a << 16) + __uint_as_float(b << 16),
                    __uint_as_float(a & 0xffff0000u) + __uint_as_float(b & 0xffff0000u));
    };
#pragma unroll
    for (int i = 0; i < NC; ++i)
      v[i] = make_uint4(add2(v[i].x, r[i].x), add2(v[i].y, r[i].y), add2(v[i].z, r[i].z), add2(v[i].w, r[i].w));
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * 256 + tid) * 8;
    if (sum_out && c < H) *reinterpret_cast<uint4*>(sum_out + row + c) = v[i];
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = __uint_as_float(w[k] << 16), b = __uint_as_float(w[k] & 0xffff0000u);
      ss = fmaf(a, a, ss);
      ss = fmaf(b, b, ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) sm[warp] = ss;
  __syncthreads();
  ss = ((sm[0] + sm[1]) + (sm[2] + sm[3])) + ((sm[4] + sm[5]) + (sm[6] + sm[7]));
  const float rs = 1.0f / sqrtf(ss / static_cast<float>(H) + a.eps);
  // rs of a mean that is no normal number is 0, NaN or more than 2^63.  (Squares below
  // fp32's normal numbers lose bits: 2^-150 of the mean at most, half a step of any
  // normal one.)
  const bool normal = rs > 0.f && rs <= 9.223372e18f;
  const int nb = H / kF8Block;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * 256 + tid) * 8;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint4 gw = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);   // bf16 ones
    if (weight && c < H) gw = __ldg(reinterpret_cast<const uint4*>(weight + c));
    const uint32_t g[4] = {gw.x, gw.y, gw.z, gw.w};
    float y[8];
    float m = 0.f;            // max|s g|
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      y[2 * k] = __uint_as_float(w[k] << 16) * __uint_as_float(g[k] << 16);
      y[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * __uint_as_float(g[k] & 0xffff0000u);
      m = max_nan(m, max_nan(fabsf(y[2 * k]), fabsf(y[2 * k + 1])));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    float rn = rs, mn = m * rs;      // n = y * rn, max|n|
    // s g at fp32's ends, where it is no longer exact (zeros and NaN among them): y becomes n
    const bool exact = m > 1e-25f && m < 1e35f && normal;
    if (__any_sync(0xffffffffu, !exact)) {
      // every warp of such a row's block comes here; asked here and not on the path of
      // all other rows (65536 x 1024 142 us, 148 us with the call in front of this loop,
      // 139 without it)
      if (!normal) {
        norm_row_wide(a);
        return;
      }
      float z[8];
      float mz = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        z[2 * k] = __uint_as_float(w[k] << 16) * rs * __uint_as_float(g[k] << 16);
        z[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * rs * __uint_as_float(g[k] & 0xffff0000u);
        mz = max_nan(mz, max_nan(fabsf(z[2 * k]), fabsf(z[2 * k + 1])));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mz = max_nan(mz, __shfl_xor_sync(0xffffffffu, mz, o));
      if (!exact) {
        rn = 1.0f;
        mn = mz;
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = z[k];
      }
    }
    if (c < H) {
      float inv;
      const float sc = f8_scale(mn, &inv);
      if ((lane & 15) == 0) q_scale[static_cast<size_t>(blockIdx.x) * nb + c / kF8Block] = sc;
      const float by = exact && sc > kF8MinScale ? kF8Max / m : rn * inv;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = y[k] * by;
      uint2 o;
      o.x = f8x4(v[0], v[1], v[2], v[3]);
      o.y = f8x4(v[4], v[5], v[6], v[7]);
      *reinterpret_cast<uint2*>(q + row + c) = o;
      if (norm_out)
        *reinterpret_cast<uint4*>(norm_out + row + c) =
            make_uint4(bf16x2(y[0] * rn, y[1] * rn), bf16x2(y[2] * rn, y[3] * rn), bf16x2(y[4] * rn, y[5] * rn),
                       bf16x2(y[6] * rn, y[7] * rn));
    }
  }
}

}  // namespace coli
