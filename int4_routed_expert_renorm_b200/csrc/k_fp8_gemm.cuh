// Matrix product of e4m3 codes with an fp32 scale for each block of 128, dense
// and over the experts of a routed batch.
//
//   out[m][n] = sum_b sa[m][b] * sw[n / 128][b] * sum_{k in block b} a[m][k] w[n][k]
// a: rows of codes with one scale per row and 128 columns; w: one scale per 128
// rows x 128 columns.  Each block's products are summed in fp32, then scaled and
// added to the fp32 total in block order.
//
// One tcgen05 kernel does every product.  The tokens are the MMA's A operand (128
// rows of tensor memory, a thread's lane = a token), NMAT blocks of 128 weight
// rows its N side: the scale of a K block is then one number per thread and
// weight block, the token's scale times the block's, kept in a register.  (With
// the weights as A a thread needs a scale per column from shared memory: 849
// against 798 us at 8192 x 12288 x 6144.)  A
// tile is up to NT tokens x NMAT * 128 weight rows: gate and up blocks of the same
// 128 columns of h, or neighbouring blocks of one matrix.  Per 128-wide K block:
//   * warp 0 brings the weight blocks (128 x 128 bytes each) and the token rows
//     into a stage of shared memory by TMA (128B swizzle); in batches of up to 32
//     tokens the rows of a routed segment are gathered four at a time by their
//     token index, larger ones are copied into pair order first;
//   * warp 1 multiplies them (four tcgen05.mma kind::f8f6f4, K = 32 each) into a
//     slot of tensor memory, a fresh accumulator per K block;
//   * warps 4..11 read the slot (tcgen05.ld), multiply-add it into fp32 totals in
//     registers and free the slot.  A thread owns one token and half of the
//     columns, of each weight block or of the pair: 128 totals, hence the register
//     split below;
//   * warps 2 and 3 keep the scales of the next four K blocks in shared memory.
// The gate/up launch ends a tile with h = silu(g) u, the token's maximum over the
// tile's 128 columns (two threads, through shared memory) and e4m3 codes with
// their scale: g and u never leave the SM.
// A operand rows past the tile's tokens are whatever shared memory holds; they
// only reach tensor-memory lanes that nothing reads.
// Measured on one B200, over calls as a program makes them (runs of seconds, where the
// clock settles under the power cap; in brackets tens of passes): 8192 x 12288 x 6144
// in 886 us (748), 1.40 PFLOP/s; 1 x 4096 x 6144 in 11 us; the FFN of a 256-expert layer
// (H 6144, I 2048, top-8, one shared) in 85 us (76) for 1 token, 466 us for 64 tokens
// over about 62 experts (HBM floor 357), 3.44 ms (2.93) for 4096.  A K block of a dense
// tile takes about 1190 cycles, its MMAs 512, its copies alone 1035; the totals wait for
// tensor memory most of the time (FMA pipe 30 % active, issue 0.41 per cycle).
#pragma once
#include <type_traits>

#include "common.cuh"
#include "k_ffn_prefill.cuh"
#include "k_norm_fp8.cuh"

namespace coli {

constexpr int kF8MaxSeg = 1024 + 8;   // unique routed + shared segments
constexpr int kF8Threads = 384;       // warp 0 TMA, warp 1 MMA, warps 4..11 totals
constexpr int kF8MaxSplit = 8;        // CTAs of a cluster that share a tile's K

// What a launch multiplies: one dense product (seg_off NULL), or the segments of
// a routed batch: the union's experts over their pairs, then the S shared experts
// over all T tokens.  Weights of expert e start at row e * R of w.
struct F8Args {
  const float* a_s;        // token scales [rows][nk]
  const float* w_s;        // weight scales [experts][ceil(R / 128)][nk]
  const float* w_s1;       // gate/up launch: the up matrix's (w_s: the gate's)
  void* out;               // [rows][R] bf16 or fp32; gate/up launch: e4m3 codes of h
  float* out_s;            // gate/up launch: scales of h [rows][R / 128]
  uint32_t* status;
  int M, R, nk;            // dense rows; output columns of one expert; K blocks
  int out_f32;
  int wide;                // fp32 rows start on 32-byte boundaries
  const int32_t* unique_ids;
  const int32_t* n_unique;
  const int32_t* seg_off;
  const int32_t* perm;     // rows gathered by the copies: token perm / k of a pair (NULL: the pair's own row)
  int shared_row;          // first token row of every shared expert; -1: each has rows of its own, as out has
  int T, k, E, S, P;
  int early;               // only a and a_s come from the kernel before this one
};

template <int NMAT, int NT>
struct F8Cfg {
  static constexpr int WSTAGE = NMAT * 128 * 128;
  static constexpr int ASTAGE = NT * 128;
  // A slot of tensor memory holds one weight block's product of a K block: four
  // slots, freed one by one, but announced together by one commit per K block (with
  // one per slot and one per stage 1225 cycles a K block, so 1076, operands
  // resident); the barrier that it arrives on frees the stage for the copies and
  // hands the slots to the totals.
  static constexpr int SLOT = 128;
  static constexpr int NSLOT = 4;
  static constexpr int META_INTS = 2 * kF8MaxSeg + 4 + kF8MaxSeg / 2;
  static constexpr int SCG = 4 * NMAT * 128;                        // scales of a group of four K blocks
  static constexpr int FIXED = 2 * SCG * 4 + 4 * 128 * 4 + META_INTS * 4 + 512;
  static constexpr int NST = (232448 - 1024 - FIXED) / (WSTAGE + ASTAGE);
  static constexpr size_t SMEM = 1024 + static_cast<size_t>(NST) * (WSTAGE + ASTAGE) + FIXED;
  static constexpr int TOT_LD = NMAT * 128 + 1;                     // split K: totals [token][TOT_LD]
  static_assert(NT % 32 == 0 && NT <= 128, "a tile's tokens are tensor-memory lanes");
  static_assert(NST >= 3 && 2 * NST + NSLOT + 11 <= 60 && NST > NSLOT / NMAT, "stages");
  // the A operand's descriptor spans 128 rows whatever NT: the weight stages that
  // follow the token stages keep that inside the allocation
  static_assert(NST * WSTAGE >= 128 * 128 && ASTAGE % 1024 == 0, "operand extent");
  static_assert(NT * TOT_LD * 4 <= NST * (WSTAGE + ASTAGE), "split-K totals fit the stages");
};

// ------------------------------------------------------------------ PTX --

// D[128 x N] (+)= A[128 x 32] * B[N x 32]^T of e4m3, both K-major in shared memory,
// issued by the lane whose `on` is not 0 (a predicate instead of a branch keeps
// the descriptors warp-uniform).
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}

// tc_commit by the lane whose `on` is not 0.
__device__ __forceinline__ void tc_commit_on(uint64_t* bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(on)
      : "memory");
}

// Whether the phase with this parity is complete, without waiting; the same answer in every lane.
__device__ __forceinline__ bool warp_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

// True in one lane of a converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Four rows (y0..y3) of a 2-D map whose box is one row, 128 bytes from column x.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int4 y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
      : "memory");
}

// 16 columns of this warp's lane quarter.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// Waits for this thread's tensor-memory loads; the registers pass through, so
// that nothing that uses them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
}

// Two fp32 totals as a register pair: t += d * s in each half.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair2(uint32_t x, uint32_t y) {
  f32x2 t;
  asm("mov.b64 %0, {%1, %2};" : "=l"(t) : "r"(x), "r"(y));
  return t;
}
__device__ __forceinline__ void fma2(f32x2& t, uint32_t d0, uint32_t d1, f32x2 s) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t) : "l"(pair2(d0, d1)), "l"(s));
}
// The two halves of N / 2 pairs.
template <int N>
__device__ __forceinline__ void unpack_pairs(const f32x2* t, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2 * i]), "=f"(v[2 * i + 1]) : "l"(t[i]));
}

// x / (1 + exp(-x)) in four instructions.  The exponent's argument is rounded to
// |x| 2^-24 of the result (a step of the e4m3 codes is 2^-3); the code runs once per
// tile, so its length costs more than its arithmetic (single token, gate/up: 8.6 us
// after the last product with expf and a division, 4.1 so).
__device__ __forceinline__ float silu(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return x * r;
}

// A load that stays where it is written (left to itself the compiler moves a
// prefetch down to its use when registers are short).
__device__ __forceinline__ float ldg_here(const float* p) {
  float v;
  asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ void ldg4_here(const float* p, float (&v)[4]) {
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// One fp32 from the shared memory of CTA `rank` of this cluster, at this CTA's address `addr`.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  uint32_t a;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// ----------------------------------------------------------------- tiles --

struct F8Tile {
  int e;        // expert (dense: 0)
  int rblk;     // tile of NMAT * 128 output columns (gate/up: of 128)
  int ntok;     // tokens
  int npad;     // rows copied: rounded up to 16
  int arow;     // first token row, or first pair of a gathered segment
  int orow;     // first output row
  bool gather;
};

// Tile t: token blocks outermost, so that CTAs running side by side read the same
// tokens and, across the blocks of an expert, the same weights from L2.
template <int NT>
__device__ __forceinline__ F8Tile f8_tile(const F8Args& a, const int32_t* blk_off, const int32_t* seg,
                                          const uint16_t* uniq, int n_seg, int U, int mbk, int t) {
  F8Tile ti;
  const int blk = t / mbk;
  ti.rblk = t - blk * mbk;
  int cnt, j, nb, abase, obase;
  ti.gather = false;
  if (!a.seg_off) {
    ti.e = 0;
    cnt = a.M;
    j = blk;
    nb = (a.M + NT - 1) / NT;
    abase = obase = 0;
  } else {
    int lo = 0, hi = n_seg - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (blk_off[mid] <= blk) lo = mid; else hi = mid - 1;
    }
    j = blk - blk_off[lo];
    nb = blk_off[lo + 1] - blk_off[lo];
    if (lo < U) {
      ti.e = uniq[lo];
      abase = obase = seg[lo];
      cnt = seg[lo + 1] - seg[lo];
      ti.gather = a.perm != nullptr;
    } else {
      ti.e = a.E + (lo - U);
      cnt = a.T;
      obase = a.P + (lo - U) * a.T;
      abase = a.shared_row >= 0 ? a.shared_row : obase;
    }
  }
  const int start = static_cast<int>(static_cast<int64_t>(cnt) * j / nb);
  const int end = static_cast<int>(static_cast<int64_t>(cnt) * (j + 1) / nb);
  ti.ntok = end - start;
  ti.npad = (ti.ntok + 15) & ~15;
  ti.arow = abase + start;
  ti.orow = obase + start;
  return ti;
}

// Row of a's for column n of a tile (columns past the last token repeat it).
__device__ __forceinline__ int f8_row(const F8Args& a, const F8Tile& ti, int n) {
  const int c = n < ti.ntok ? n : ti.ntok - 1;
  return ti.gather ? __ldg(a.perm + ti.arow + c) / a.k : ti.arow + c;
}

// The expert input of a routed batch in pair order: row i < P is the codes and
// scales of token perm[i] / k, the `extra` rows after them the tokens in order (T of
// them for the shared experts, or none).  One warp per row, 16-byte moves.  For more
// than 32 tokens this pays: copies that gather four rows each bring 128 rows in 1800
// cycles, a plain 128-row copy in 1000 (gate/up of 4096 tokens 2.84 against 1.76 ms,
// and this kernel takes 0.07).
__global__ void __launch_bounds__(256) f8_gather_kernel(const uint8_t* __restrict__ x, const float* __restrict__ x_s,
                                                        const int32_t* __restrict__ perm, int k, int P, int extra, int T, int H,
                                                        uint8_t* __restrict__ xg, float* __restrict__ sg) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < P + extra; i += gridDim.x * 8) {
    // a pair whose expert was out of range is in no segment: perm may not name it
    const int t = i < P ? __ldg(perm + i) / k : i - P;
    if (static_cast<unsigned>(t) >= static_cast<unsigned>(T)) continue;
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<size_t>(t) * H);
    uint4* dst = reinterpret_cast<uint4*>(xg + static_cast<size_t>(i) * H);
    for (int c = lane; c < H / 16; c += 32) dst[c] = __ldg(src + c);
    for (int c = lane; c < H / kF8Block; c += 32)
      sg[static_cast<size_t>(i) * (H / kF8Block) + c] = __ldg(x_s + static_cast<size_t>(t) * (H / kF8Block) + c);
  }
}

// Eight fp32 values as one 32-byte store (a whole sector of a row).
__device__ __forceinline__ void st_f32x8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// N values of one output row from column col on, as 16-byte stores where rows and
// columns allow it.
template <int N>
__device__ __forceinline__ void f8_store_row(const F8Args& a, size_t row, int col, const float (&v)[N]) {
  const int left = a.R - col;
  if (a.out_f32) {
    float* o = static_cast<float*>(a.out) + row * a.R + col;
    if (a.wide) {
#pragma unroll
      for (int i = 0; i < N; i += 8)
        if (i < left) st_f32x8(o + i, &v[i]);
    } else if (a.R % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4)
        if (i < left) *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) o[i] = v[i];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(a.out) + row * a.R + col;
    if (a.R % 8 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 8)
        if (i < left)
          *reinterpret_cast<uint4*>(o + i) = make_uint4(bf16x2(v[i], v[i + 1]), bf16x2(v[i + 2], v[i + 3]),
                                                        bf16x2(v[i + 4], v[i + 5]), bf16x2(v[i + 6], v[i + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) o[i] = float_to_bf16_bits(v[i]);
    }
  }
}

// ------------------------------------------------------------ the kernel --

// GU: the gate/up launch (NMAT = 2).  gridDim.x: the tiles' CTAs, or with clusters
// of c CTAs (dense, one tile per cluster) c of them per tile, each taking its share
// of the K blocks; their totals are added in rank order through distributed shared
// memory.
template <int NMAT, int NT, bool GU>
__global__ void __launch_bounds__(kF8Threads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap mw0, const __grid_constant__ CUtensorMap mw1,
                    const __grid_constant__ CUtensorMap mb128, const __grid_constant__ CUtensorMap mb64,
                    const __grid_constant__ CUtensorMap mb32, const __grid_constant__ CUtensorMap mb16,
                    const __grid_constant__ CUtensorMap mgat, F8Args a, int split) {
  using C = F8Cfg<NMAT, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* a_stages = smem;                                              // token rows
  uint8_t* w_stages = smem + C::NST * C::ASTAGE;                         // weight rows
  float* red = reinterpret_cast<float*>(w_stages + C::NST * C::WSTAGE);  // [2 parities][2 halves][128]: maxima
  float* scales = red + 4 * 128;                                         // [2][4][NMAT][128]
  int32_t* blk_off = reinterpret_cast<int32_t*>(scales + 2 * C::SCG);
  int32_t* seg = blk_off + kF8MaxSeg + 2;
  uint16_t* uniq = reinterpret_cast<uint16_t*>(seg + kF8MaxSeg + 2);      // expert ids below 1024
  uint64_t* bars = reinterpret_cast<uint64_t*>(blk_off + C::META_INTS);
  uint64_t* full = bars;
  uint64_t* done = full + C::NST;                 // the stage's MMAs are complete
  uint64_t* slot_empty = done + C::NST;
  uint64_t* first_done = slot_empty + C::NSLOT;    // [2]: a K block's first weight block is multiplied (BYMAT)
  uint64_t* pair_bar = first_done + 2;             // [4]: the two warps of a lane quarter
  uint64_t* sc_full = pair_bar + 4;                // [2]: a group's scales are written
  uint64_t* sc_empty = sc_full + 2;                // and read
  uint64_t* mma_done = sc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  int* scratch = reinterpret_cast<int*>(red);     // 33 ints, before the tiles
  // A dense or down tile of two weight blocks: each block has four warps of totals
  // of its own; otherwise all eight share every block's columns.
  constexpr bool BYMAT = NMAT == 2 && !GU;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int q = 0; q < C::NST; ++q) {
      mbar_init(&full[q], 1);
      mbar_init(&done[q], 1);
    }
    for (int q = 0; q < C::NSLOT; ++q) {
      mbar_init(&slot_empty[q], BYMAT ? 4 : 8);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&pair_bar[q], 2);
    for (int q = 0; q < 2; ++q) {
      mbar_init(&first_done[q], 1);
      mbar_init(&sc_full[q], 2);
      mbar_init(&sc_empty[q], 8);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&mw0);
    if (GU) prefetch_tensormap(&mw1);
    prefetch_tensormap(&mb16);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  // The down launch follows the gate/up one, which passed its own wait before it
  // let this one start: the plan and the weights are there, only h is not.
  if (!a.early) pdl_wait();
  pdl_trigger();
  int n_seg = 0, U = 0, total_blocks;
  if (a.seg_off) {
    // token blocks of every segment, each of near-equal parts of at most NT tokens
    // (the arrays have room for min(E, P) segments: no need to know U to load them)
    const int most = min(a.E, a.P);
    U = __ldg(a.n_unique);
    for (int i = threadIdx.x; i < most; i += blockDim.x) uniq[i] = static_cast<uint16_t>(__ldg(a.unique_ids + i));
    for (int i = threadIdx.x; i <= most; i += blockDim.x) seg[i] = __ldg(a.seg_off + i);
    n_seg = U + a.S;
    __syncthreads();
    int base = 0;
    for (int i0 = 0; i0 < n_seg; i0 += blockDim.x) {
      const int i = i0 + threadIdx.x;
      const int cnt = i < U ? seg[i + 1] - seg[i] : i < n_seg ? a.T : 0;
      int sum = 0;
      const int off = block_exclusive_scan((cnt + NT - 1) / NT, scratch, &sum);
      if (i < n_seg) blk_off[i] = base + off;
      base += sum;
    }
    if (threadIdx.x == 0) blk_off[n_seg] = base;
    total_blocks = base;
  } else {
    total_blocks = (a.M + NT - 1) / NT;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  constexpr int ROWS = GU ? 128 : NMAT * 128;     // output columns of a tile
  const int nrb = (a.R + 127) / 128;              // rows of weight scales of an expert
  const int mbk = (a.R + ROWS - 1) / ROWS;
  const int tiles = total_blocks * mbk;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int kb0 = split > 1 ? a.nk * rank / split : 0;
  const int kb1 = split > 1 ? a.nk * (rank + 1) / split : a.nk;
  const int t_first = blockIdx.x / split, t_step = gridDim.x / split;
  auto tile_at = [&](int t) { return f8_tile<NT>(a, blk_off, seg, uniq, n_seg, U, mbk, t); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      // ----------------------------------------------------- TMA producer
      uint32_t st = 0;
      bool ok = true;
      auto copy_weights = [&](const F8Tile& ti, int kb, int s) {       // one lane
        const int row0 = ti.e * a.R + ti.rblk * ROWS;
        uint8_t* dst = w_stages + s * C::WSTAGE;
        mbar_arrive_expect_tx(&full[s], C::WSTAGE + ti.npad * 128);
        tma_load_2d(dst, &mw0, &full[s], kb * 128, row0);
        if (NMAT == 2) tma_load_2d(dst + 128 * 128, GU ? &mw1 : &mw0, &full[s], kb * 128, GU ? row0 : row0 + 128);
      };
      // gathered rows: lane l takes rows 4l..4l+3
      auto rows_of = [&](const F8Tile& ti) {
        if (!ti.gather || 4 * lane >= ti.npad) return make_int4(0, 0, 0, 0);
        return make_int4(f8_row(a, ti, 4 * lane), f8_row(a, ti, 4 * lane + 1), f8_row(a, ti, 4 * lane + 2),
                         f8_row(a, ti, 4 * lane + 3));
      };
      auto copy_tokens = [&](const F8Tile& ti, int4 y, int kb, int s) {
        uint8_t* d = a_stages + s * C::ASTAGE;
        if (ti.gather) {
          if (4 * lane < ti.npad) tma_gather4(d + lane * 512, &mgat, &full[s], kb * 128, y);
        } else if (lane == 0) {
          int row = ti.arow, rem = ti.npad;
          if (rem >= 128) { tma_load_2d(d, &mb128, &full[s], kb * 128, row); rem = 0; }
          if (rem >= 64) { tma_load_2d(d, &mb64, &full[s], kb * 128, row); rem -= 64; row += 64; d += 64 * 128; }
          if (rem >= 32) { tma_load_2d(d, &mb32, &full[s], kb * 128, row); rem -= 32; row += 32; d += 32 * 128; }
          if (rem >= 16) tma_load_2d(d, &mb16, &full[s], kb * 128, row);
        }
      };
      // the first tile's weights are on their way while the rows are still written
      const int ahead = a.early && t_first < tiles ? min(C::NST, kb1 - kb0) : 0;
      if (ahead) {
        const F8Tile ti = tile_at(t_first);
        if (lane == 0)
          for (int i = 0; i < ahead; ++i) copy_weights(ti, kb0 + i, i);
        __syncwarp();
        if (a.early) pdl_wait();
        // the rows may come from an earlier kernel's plain stores
        asm volatile("fence.proxy.async;" ::: "memory");
        const int4 y = rows_of(ti);
        for (int i = 0; i < ahead; ++i) copy_tokens(ti, y, kb0 + i, i);
        st = ahead;
      } else if (a.early) {
        pdl_wait();
      }
      for (int t = t_first; ok && t < tiles; t += t_step) {
        const F8Tile ti = tile_at(t);
        const int4 y = rows_of(ti);
        for (int kb = kb0 + (t == t_first ? ahead : 0); kb < kb1; ++kb, ++st) {
          const int s = static_cast<int>(st % C::NST);
          if (!(ok = warp_wait(&done[s], ((st / C::NST) & 1u) ^ 1u, abort_flag, a.status))) break;
          if (lane == 0) copy_weights(ti, kb, s);
          __syncwarp();
          copy_tokens(ti, y, kb, s);
        }
      }
      if (!ok && lane == 0) {
        // bounded wait (ignoring the abort flag) for the copies still in flight
        int dummy = 0;
        for (uint32_t q = st > C::NST ? st - C::NST : 0; q < st; ++q)
          mbar_wait(&full[q % C::NST], (q / C::NST) & 1u, reinterpret_cast<volatile int*>(&dummy), a.status);
      }
      __syncwarp();
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issue
      // The whole warp walks the loop, so that addresses and descriptors stay
      // warp-uniform; one elected lane issues.  The barriers of the next product are
      // looked at before the last MMA of this one.
      const uint32_t leader = elect_one();
      int s = 0, q = 0;
      uint32_t sph = 0, qph = 1;              // phases: stage filled, slot freed
      const uint64_t wdesc0 = sw128_kmajor_desc(smem_addr(w_stages));
      const uint64_t adesc0 = sw128_kmajor_desc(smem_addr(a_stages));
      const uint32_t idesc = idesc_f16_m128(128);     // e4m3 has type field 0 too
      bool ok = true, stage_ready = false, slot_ready = false;
      for (int t = t_first; ok && t < tiles; t += t_step) {
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          if (!stage_ready && !(ok = warp_wait(&full[s], sph, abort_flag, a.status))) break;
          const uint64_t wdesc = wdesc0 + static_cast<uint64_t>(s * (C::WSTAGE / 16));
          const uint64_t adesc = adesc0 + static_cast<uint64_t>(s * (C::ASTAGE / 16));
          const int s1 = s + 1 == C::NST ? 0 : s + 1;
          const uint32_t sph1 = s1 ? sph : sph ^ 1u;
#pragma unroll
          for (int m = 0; m < NMAT; ++m) {
            if (!slot_ready && !(ok = warp_wait(&slot_empty[q], qph, abort_flag, a.status))) break;
            tc_fence_after();
            const int q1 = (q + 1) % C::NSLOT;
            const uint32_t qph1 = q1 ? qph : qph ^ 1u;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk == 3) {
                if (m == NMAT - 1) stage_ready = warp_test(&full[s1], sph1);
                slot_ready = warp_test(&slot_empty[q1], qph1);
              }
              mma_f8_ss(tbase + q * C::SLOT, adesc + kk * 2, wdesc + m * 1024 + kk * 2, idesc, kk != 0, leader);
            }
            if (BYMAT && m == 0) tc_commit_on(&first_done[q >> 1], leader);
            q = q1;
            qph = qph1;
          }
          if (!ok) break;
          tc_commit_on(&done[s], leader);
          s = s1;
          sph = sph1;
        }
      }
      // every MMA of this CTA has completed before TMEM is released
      if (leader) {
        int dummy = 0;
        tc_commit(mma_done);
        mbar_wait(mma_done, 0, reinterpret_cast<volatile int*>(&dummy), a.status);
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------------- scales
      // Warps 2 and 3: the tile's scales, token's times weight block's, four K
      // blocks at a time, to shared memory.  A warp's 32 rows are 32 lines, and a
      // line costs the shared-memory pipe as much as 128 bytes of operands: they
      // are read once here (16 bytes a line where rows allow it) rather than by the
      // totals' eight warps.  Warp 2 + w takes tokens 32 w .. and 64 + 32 w ..; the
      // next four K blocks are on their way.
      constexpr int NI = NT > 64 ? 2 : 1;
      const int c0 = lane + 32 * (warp - 2);
      const bool rows4 = a.nk % 4 == 0 && kb0 % 4 == 0 && kb1 % 4 == 0 && (reinterpret_cast<uintptr_t>(a.a_s) & 15) == 0;
      const float* ap[NI];
      const float* wp[NMAT];
      float an[NI][4], wn[NMAT][4];
      auto set_tile = [&](int t) {
        const F8Tile ti = tile_at(t);
#pragma unroll
        for (int i = 0; i < NI; ++i) ap[i] = a.a_s + static_cast<size_t>(f8_row(a, ti, c0 + 64 * i)) * a.nk;
#pragma unroll
        for (int m = 0; m < NMAT; ++m) {
          const int rb = GU ? ti.rblk : min(ti.rblk * NMAT + m, nrb - 1);
          wp[m] = (GU && m ? a.w_s1 : a.w_s) + (static_cast<size_t>(ti.e) * nrb + rb) * a.nk;
        }
      };
      auto load = [&](int g) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (rows4) {
            ldg4_here(ap[i] + g, an[i]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) an[i][c] = ldg_here(ap[i] + min(g + c, kb1 - 1));
          }
        }
#pragma unroll
        for (int m = 0; m < NMAT; ++m)
#pragma unroll
          for (int c = 0; c < 4; ++c) wn[m][c] = ldg_here(wp[m] + min(g + c, kb1 - 1));
      };
      bool ok = true;
      uint32_t gi = 0;
      if (a.early) pdl_wait();
      if (t_first < tiles) {
        set_tile(t_first);
        load(kb0);
      }
      for (int t = t_first; ok && t < tiles; t += t_step) {
        for (int g = kb0; g < kb1; g += 4, ++gi) {
          if (!(ok = warp_wait(&sc_empty[gi & 1u], ((gi >> 1) & 1u) ^ 1u, abort_flag, a.status))) break;
          float* to = scales + (gi & 1u) * C::SCG;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int m = 0; m < NMAT; ++m)
#pragma unroll
              for (int i = 0; i < NI; ++i) to[(c * NMAT + m) * 128 + c0 + 64 * i] = an[i][c] * wn[m][c];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[gi & 1u]);
          if (g + 4 < kb1) {
            load(g + 4);
          } else if (t + t_step < tiles) {
            set_tile(t + t_step);
            load(kb0);
          }
        }
      }
      __syncwarp();
    }
    if (split > 1) {
      cluster_arrive();
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
  } else {
    // ------------------------------------------------------------- totals
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int q4 = warp & 3;                   // TMEM lane quarter
    // BYMAT: warps 4..7 take the first weight block's 128 columns and warps 8..11 the
    // second one's, each as soon as it is multiplied, so that the two warps of a
    // scheduler wait and add in turn (K block of a dense product 1240 -> 1133 cycles;
    // for gate/up it loses: u then has to travel, 1.67 against 1.78 ms).  Otherwise a
    // warp takes half of each block's columns.
    const int half = (warp - 4) >> 2;
    constexpr int MH = BYMAT ? 1 : NMAT, NCOL = BYMAT ? 128 : 64, NB = NCOL / 16;
    const int r = 32 * q4 + lane;              // token of the tile
    const uint32_t tq = tbase + (static_cast<uint32_t>(32 * q4) << 16) + (BYMAT ? 0 : half * 64);
    int q = BYMAT ? half : 0;                  // next slot
    int s = 0;                                 // stage of the next K block
    uint32_t sph = 0, met = 0, gi = 0;         // gi: groups of four K blocks so far
    bool ok = true;
    // Waits for the next K block's products.  The MMAs run at most NSLOT / NMAT K
    // blocks ahead, fewer than the stages: no barrier can be a phase further.
    auto next_block = [&]() -> bool {
      const bool first = BYMAT && half == 0;
      if (!warp_wait(first ? &first_done[s] : &done[s], sph, abort_flag, a.status)) return false;
      if (++s == (first ? 2 : C::NST)) {
        s = 0;
        sph ^= 1u;
      }
      tc_fence_after();
      return true;
    };
    f32x2 acc[MH][NCOL / 2];                   // columns in pairs
    for (int t = t_first; ok && t < tiles; t += t_step) {
      const F8Tile ti = tile_at(t);
      const bool any = 32 * q4 < ti.ntok;      // this warp's lanes hold tokens
#pragma unroll
      for (int m = 0; m < MH; ++m)
#pragma unroll
        for (int i = 0; i < NCOL / 2; ++i) acc[m][i] = 0ull;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&slot_empty[q]);
        q = (q + (BYMAT ? 2 : 1)) % C::NSLOT;
      };
      auto free_scales = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_empty[gi & 1u]);
        ++gi;
      };
      if (!any) {
        for (int kb = kb0; kb < kb1 && (ok = next_block()); ++kb) {
          for (int m = 0; m < MH; ++m) release();
          if ((kb - kb0) % 4 == 3 || kb + 1 == kb1) {
            if (!(ok = warp_wait(&sc_full[gi & 1u], (gi >> 1) & 1u, abort_flag, a.status))) break;
            free_scales();
          }
        }
      } else {
        // 16 columns are on their way from tensor memory while 16 are added, the
        // next K block's first ones too.  The loop over K blocks is not unrolled:
        // then nothing is spilled and the body stays in the instruction cache
        // (layer of 4096 tokens 2.97 against 3.13 ms unrolled by four, one token 76
        // against 82 us).
        uint32_t d[2][16];
        if ((ok = next_block())) tmem_ld16(tq + q * C::SLOT, d[0]);
        for (int g = kb0; ok && g < kb1; g += 4) {
          if (!(ok = warp_wait(&sc_full[gi & 1u], (gi >> 1) & 1u, abort_flag, a.status))) break;
          const float* scp = scales + (gi & 1u) * C::SCG + (BYMAT ? half * 128 : 0) + r;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (g + c >= kb1) break;
            float sm[MH];
#pragma unroll
            for (int m = 0; m < MH; ++m) sm[m] = scp[(c * NMAT + m) * 128];
            if (c == 3 || g + c + 1 == kb1) free_scales();
#pragma unroll
            for (int m = 0; m < MH; ++m) {
              const f32x2 s2 = pair2(__float_as_uint(sm[m]), __float_as_uint(sm[m]));
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                uint32_t(&cur)[16] = d[b & 1];
                uint32_t(&nxt)[16] = d[(b + 1) & 1];
                tmem_wait_ld16(cur);
                if (b + 1 < NB) {
                  tmem_ld16(tq + q * C::SLOT + 16 * (b + 1), nxt);
                } else {
                  release();
                  if (m + 1 < MH) {
                    tmem_ld16(tq + q * C::SLOT, nxt);
                  } else if (g + c + 1 < kb1) {
                    if (!(ok = next_block())) break;
                    tmem_ld16(tq + q * C::SLOT, nxt);
                  }
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) fma2(acc[m][8 * b + x], cur[2 * x], cur[2 * x + 1], s2);
              }
              if (!ok) break;
            }
            if (!ok) break;
          }
        }
      }
      if (!ok) break;
      if constexpr (GU) {
        if (!any) continue;
        // h, the maximum of the token's 128 columns (64 in each of two threads),
        // codes and scale.  A code sees two roundings before its own, of 1 / c and of
        // the product (a division by c would be one, for 64 values a thread): half a
        // step 2^-24 each, less than the sums of g and u are off by.
        float mx = 0.f, h[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float g[32];
          unpack_pairs<32>(&acc[0][16 * c], g);
          unpack_pairs<32>(&acc[MH - 1][16 * c], h[c]);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            h[c][i] *= silu(g[i]);
            mx = max_nan(mx, fabsf(h[c][i]));
          }
        }
        // the two warps of this lane quarter meet; with two sets of maxima a warp
        // writes a set again only after its partner came to the meeting in between
        float* rw = red + (met & 1u) * 256;
        rw[half * 128 + r] = mx;
        __syncwarp();
        if (lane == 0) mbar_arrive(&pair_bar[q4]);
        if (!(ok = warp_wait(&pair_bar[q4], met & 1u, abort_flag, a.status))) break;
        ++met;
        mx = max_nan(mx, rw[(half ^ 1) * 128 + r]);
        if (r < ti.ntok) {
          float inv;
          const float scl = f8_scale(mx, &inv);
          const size_t row = static_cast<size_t>(ti.orow + r);
          if (half == 0) a.out_s[row * nrb + ti.rblk] = scl;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + row * a.R + ti.rblk * 128 + half * 64);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float* e = &h[c][16 * x + 4 * y];
                w[y] = f8x4(e[0] * inv, e[1] * inv, e[2] * inv, e[3] * inv);
              }
              dst[2 * c + x] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
      } else if (split == 1) {
        if (r < ti.ntok) {
#pragma unroll
          for (int c = 0; c < NCOL / 32; ++c) {
            float v[32];
            unpack_pairs<32>(&acc[0][16 * c], v);
            f8_store_row<32>(a, static_cast<size_t>(ti.orow + r), ti.rblk * ROWS + half * NCOL + c * 32, v);
          }
        }
      } else if (r < NT) {
        // split K: totals to shared memory (every copy and MMA of this CTA is done),
        // rows of odd length: no bank twice here, whole 128-byte lines to the peers
        float* tot = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < NCOL / 32; ++c) {
          float v[32];
          unpack_pairs<32>(&acc[0][16 * c], v);
#pragma unroll
          for (int i = 0; i < 32; ++i) tot[r * C::TOT_LD + half * NCOL + c * 32 + i] = v[i];
        }
      }
    }
    if (split > 1) {
      cluster_arrive();
      cluster_wait();
      if (ok && t_first < tiles) {
        // this CTA adds its share of the tokens over the ranks, in rank order
        const F8Tile ti = tile_at(t_first);
        const int x = threadIdx.x - 128;
        constexpr int PER = 256 / (NMAT * 128);           // tokens at a time
        const int c = x % (NMAT * 128);
        const int col = ti.rblk * ROWS + c;
        const uint32_t base = smem_addr(smem);
        constexpr int UN = 4;                              // tokens in flight: up to 32 loads
        for (int n0 = rank * PER + x / (NMAT * 128); n0 < ti.ntok; n0 += UN * split * PER) {
          float v[UN][kF8MaxSplit];
#pragma unroll
          for (int p = 0; p < kF8MaxSplit; ++p)
#pragma unroll
            for (int u = 0; u < UN; ++u) {
              const int n = n0 + u * split * PER;
              if (p < split && n < ti.ntok) v[u][p] = ld_cluster_f32(base + (n * C::TOT_LD + c) * 4, p);
            }
#pragma unroll
          for (int u = 0; u < UN; ++u) {
            const int n = n0 + u * split * PER;
            if (n < ti.ntok && col < a.R) {
              float y = 0.f;
#pragma unroll
              for (int p = 0; p < kF8MaxSplit; ++p)
                if (p < split) y += v[u][p];
              const size_t at = static_cast<size_t>(ti.orow + n) * a.R + col;
              if (a.out_f32)
                static_cast<float*>(a.out)[at] = y;
              else
                static_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(y);
            }
          }
        }
      }
      cluster_arrive();
      cluster_wait();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace coli
