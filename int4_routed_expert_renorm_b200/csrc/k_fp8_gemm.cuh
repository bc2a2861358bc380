// Matrix product of e4m3 codes with an fp32 scale for each block of 128, dense
// and over the experts of a routed batch.
//
//   out[m][n] = sum_b sa[m][b] * sw[n / 128][b] * sum_{k in block b} a[m][k] w[n][k]
// a: rows of codes with one scale per row and 128 columns; w: one scale per 128
// rows x 128 columns.  Each block's products are summed in fp32, then scaled and
// added to the fp32 total in block order.
//
// One tcgen05 kernel does every product.  The weights are the MMA's A operand
// (128 rows = one row of weight scales), the tokens its N side (up to NT of them,
// rounded up to 16), so that a batch of one token costs no more tensor work than
// 16 and an expert's tokens are never padded to 128.  A tile is NMAT blocks of
// 128 weight rows x up to NT tokens: gate and up blocks of the same 128 columns of
// h, or neighbouring blocks of one matrix.  Per 128-wide K block:
//   * warp 0 brings the weight blocks (128 x 128 bytes each) and the token rows
//     into a stage of shared memory by TMA (128B swizzle); rows of a routed segment
//     are gathered four at a time by their token index, so the batch is never
//     copied into pair order;
//   * one thread of warp 1 multiplies each weight block with the tokens (four
//     tcgen05.mma kind::f8f6f4, K = 32 each) into a slot of tensor memory, a fresh
//     accumulator per K block;
//   * warps 2 and 3 write the slot's token scales times its weight scale to shared
//     memory;
//   * warps 4..11 read the slot (tcgen05.ld), multiply-add it into fp32 totals in
//     registers (fma.rn.f32x2: two columns an instruction) and free the slot.
// A thread of warps 4..11 owns one weight row and every other 16-token chunk: 160
// totals for 2 x 160 tokens, hence the register split below.
// The gate/up launch ends a tile with h = silu(g) u, the row block's maximum over
// its 128 columns (one redux per warp and token, four warps through shared
// memory) and e4m3 codes with their scale: g and u never leave the SM.
#pragma once
#include "common.cuh"
#include "k_ffn_prefill.cuh"
#include "k_norm_fp8.cuh"

namespace coli {

constexpr int kF8MaxSeg = 1024 + 8;   // unique routed + shared segments
constexpr int kF8Threads = 384;       // warp 0 TMA, warp 1 MMA, warps 2 and 3 scales, warps 4..11 totals
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
  const int32_t* unique_ids;
  const int32_t* n_unique;
  const int32_t* seg_off;
  const int32_t* perm;     // gathered token rows: perm / k (NULL: the pair's own row)
  int T, k, E, S, P;
};

template <int NMAT, int NT>
struct F8Cfg {
  static constexpr int WSTAGE = NMAT * 128 * 128;
  static constexpr int STAGE = WSTAGE + NT * 128;
  static constexpr int NSLOT = NT > 128 ? 3 : NT > 64 ? 4 : 8;      // accumulators in tensor memory
  static constexpr int CH = 16;                                     // columns of a chunk
  static constexpr int NCH = (NT / CH + 1) / 2;                     // chunks of a thread
  static constexpr int META_INTS = 3 * kF8MaxSeg + 4;
  static constexpr int FIXED = NSLOT * NT * 4 + 4 * NT * 4 + META_INTS * 4 + 512;
  static constexpr int NST = (232448 - 1024 - FIXED) / STAGE;
  static constexpr size_t SMEM = 1024 + static_cast<size_t>(NST) * STAGE + FIXED;
  static_assert(NT % 16 == 0 && NT <= 256 && NSLOT * NT <= 512, "tensor memory budget");
  static_assert(NST >= 3 && 2 * NST + 2 * NSLOT + 1 <= 60, "stages");
  static_assert(STAGE % 1024 == 0, "stage alignment");
  static_assert(NMAT * 128 * NT * 4 <= NST * STAGE, "split-K totals fit the stages");
};

// ------------------------------------------------------------------ PTX --

// D[128 x N] (+)= A[128 x 32] * B[N x 32]^T of e4m3, both K-major in shared memory.
__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four rows (y0..y3) of a 2-D map whose box is one row, 128 bytes from column x.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int4 y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Two fp32 totals as one 64-bit register pair: t = fma(d, s, t) in each half.
using f32x2 = unsigned long long;
__device__ __forceinline__ void fma2(f32x2& t, uint32_t d0, uint32_t d1, f32x2 s) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t) : "l"(d), "l"(s));
}
__device__ __forceinline__ float2 unpack2(f32x2 t) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(t));
  return f;
}
__device__ __forceinline__ void lds_2x64(uint32_t addr, f32x2& a, f32x2& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
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

// Barrier of the four warps of one column half (128 threads), id 1 or 2.
__device__ __forceinline__ void half_barrier(int half) {
  asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory");
}

// ----------------------------------------------------------------- tiles --

struct F8Tile {
  int e;        // expert (dense: 0)
  int rblk;     // tile of NMAT * 128 output columns (gate/up: of 128)
  int ntok;     // tokens
  int npad;     // rounded up to 16
  int arow;     // first token row, or first pair of a gathered segment
  int orow;     // first output row
  bool gather;
};

// Tile t: token blocks outermost, so that CTAs running side by side read the same
// tokens and, across the blocks of an expert, the same weights from L2.
template <int NT>
__device__ __forceinline__ F8Tile f8_tile(const F8Args& a, const int32_t* blk_off, const int32_t* seg,
                                          const int32_t* uniq, int n_seg, int U, int mbk, int t) {
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
      abase = a.perm ? 0 : obase;
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
  float* sc_base = reinterpret_cast<float*>(smem + C::NST * C::STAGE);    // [NSLOT][NT]
  float* red = sc_base + C::NSLOT * NT;                                   // [4][NT]: row-block maxima
  int32_t* blk_off = reinterpret_cast<int32_t*>(red + 4 * NT);
  int32_t* uniq = blk_off + kF8MaxSeg + 2;
  int32_t* seg = uniq + kF8MaxSeg;
  uint64_t* bars = reinterpret_cast<uint64_t*>(red + 4 * NT + C::META_INTS);
  uint64_t* full = bars;
  uint64_t* empty = full + C::NST;
  uint64_t* slot_full = empty + C::NST;
  uint64_t* slot_empty = slot_full + C::NSLOT;
  uint64_t* mma_done = slot_empty + C::NSLOT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* scratch = reinterpret_cast<int*>(red);     // 33 ints, before the tiles

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int q = 0; q < C::NST; ++q) {
      mbar_init(&full[q], 1);
      mbar_init(&empty[q], 1);
    }
    for (int q = 0; q < C::NSLOT; ++q) {
      mbar_init(&slot_full[q], 3);      // the MMAs' commit and the two scale warps
      mbar_init(&slot_empty[q], 8);
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
  pdl_wait();
  pdl_trigger();
  int n_seg = 0, U = 0, total_blocks;
  if (a.seg_off) {
    // token blocks of every segment, each of near-equal parts of at most NT tokens
    U = __ldg(a.n_unique);
    n_seg = U + a.S;
    for (int i = threadIdx.x; i < U; i += blockDim.x) uniq[i] = __ldg(a.unique_ids + i);
    for (int i = threadIdx.x; i <= U; i += blockDim.x) seg[i] = __ldg(a.seg_off + i);
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
      // the rows may come from an earlier kernel's plain stores
      asm volatile("fence.proxy.async;" ::: "memory");
      uint32_t st = 0;
      bool ok = true;
      for (int t = t_first; ok && t < tiles; t += t_step) {
        const F8Tile ti = tile_at(t);
        const int row0 = ti.e * a.R + ti.rblk * ROWS;
        // gathered rows: lane l takes rows 4l..4l+3 and 4(l+32)..: NT <= 256
        int4 y0 = make_int4(0, 0, 0, 0), y1 = y0;
        if (ti.gather) {
          if (4 * lane < ti.npad)
            y0 = make_int4(f8_row(a, ti, 4 * lane), f8_row(a, ti, 4 * lane + 1), f8_row(a, ti, 4 * lane + 2),
                           f8_row(a, ti, 4 * lane + 3));
          if (NT > 128 && 4 * (lane + 32) < ti.npad)
            y1 = make_int4(f8_row(a, ti, 4 * lane + 128), f8_row(a, ti, 4 * lane + 129),
                           f8_row(a, ti, 4 * lane + 130), f8_row(a, ti, 4 * lane + 131));
        }
        for (int kb = kb0; kb < kb1; ++kb, ++st) {
          const int s = static_cast<int>(st % C::NST);
          if (!(ok = warp_wait(&empty[s], ((st / C::NST) & 1u) ^ 1u, abort_flag, a.status))) break;
          uint8_t* dst = smem + s * C::STAGE;
          uint8_t* bdst = dst + C::WSTAGE;
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[s], C::WSTAGE + ti.npad * 128);
            tma_load_2d(dst, &mw0, &full[s], kb * 128, row0);
            if (NMAT == 2) tma_load_2d(dst + 128 * 128, GU ? &mw1 : &mw0, &full[s], kb * 128, GU ? row0 : row0 + 128);
            if (!ti.gather) {
              int row = ti.arow, rem = ti.npad;
              uint8_t* d = bdst;
              for (; rem >= 128; rem -= 128, row += 128, d += 128 * 128) tma_load_2d(d, &mb128, &full[s], kb * 128, row);
              if (rem >= 64) { tma_load_2d(d, &mb64, &full[s], kb * 128, row); rem -= 64; row += 64; d += 64 * 128; }
              if (rem >= 32) { tma_load_2d(d, &mb32, &full[s], kb * 128, row); rem -= 32; row += 32; d += 32 * 128; }
              if (rem >= 16) tma_load_2d(d, &mb16, &full[s], kb * 128, row);
            }
          }
          __syncwarp();
          if (ti.gather) {
            if (4 * lane < ti.npad) tma_gather4(bdst + lane * 512, &mgat, &full[s], kb * 128, y0);
            if (NT > 128 && 4 * (lane + 32) < ti.npad)
              tma_gather4(bdst + (lane + 32) * 512, &mgat, &full[s], kb * 128, y1);
          }
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
      if (lane == 0) {
        uint32_t st = 0, sl = 0;
        bool ok = true;
        for (int t = t_first; ok && t < tiles; t += t_step) {
          const F8Tile ti = tile_at(t);
          const uint32_t idesc = idesc_f16_m128(ti.npad);     // e4m3 has type field 0 too
          for (int kb = kb0; ok && kb < kb1; ++kb, ++st) {
            const int s = static_cast<int>(st % C::NST);
            if (!(ok = mbar_wait(&full[s], (st / C::NST) & 1u, abort_flag, a.status))) break;
            const uint32_t ws = smem_addr(smem + s * C::STAGE), bs = ws + C::WSTAGE;
#pragma unroll
            for (int m = 0; m < NMAT; ++m, ++sl) {
              const int q = static_cast<int>(sl % C::NSLOT);
              if (!(ok = mbar_wait(&slot_empty[q], ((sl / C::NSLOT) & 1u) ^ 1u, abort_flag, a.status))) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f8_ss(tbase + q * NT, sw128_kmajor_desc(ws + m * 128 * 128 + kk * 32),
                          sw128_kmajor_desc(bs + kk * 32), idesc, kk != 0);
              tc_commit(&slot_full[q]);
            }
            if (!ok) break;
            tc_commit(&empty[s]);
          }
        }
        // every MMA of this CTA has completed before TMEM is released
        int dummy = 0;
        tc_commit(mma_done);
        mbar_wait(mma_done, 0, reinterpret_cast<volatile int*>(&dummy), a.status);
      }
      __syncwarp();
    } else {
      // ----------------------------------------------------------- scales
      // Both warps serve every slot, each its 32 of every 64 columns (a warp that
      // skipped slots could run a whole barrier phase ahead of the others).  The
      // next four K blocks' scales, of the next tile at a tile's end, are loaded
      // while four are in use.
      constexpr int NI = (NT + 63) / 64;
      const int c0 = lane + 32 * (warp - 2);
      const float* ap[NI];
      const float* wp[NMAT];
      float av[NI][4], wv[NMAT][4], an[NI][4], wn[NMAT][4];
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
        for (int c = 0; c < 4; ++c) {
          const int kb = min(g + c, kb1 - 1);
#pragma unroll
          for (int i = 0; i < NI; ++i) an[i][c] = __ldg(ap[i] + kb);
#pragma unroll
          for (int m = 0; m < NMAT; ++m) wn[m][c] = __ldg(wp[m] + kb);
        }
      };
      uint32_t sl = 0;
      bool ok = true;
      if (t_first < tiles) {
        set_tile(t_first);
        load(kb0);
      }
      for (int t = t_first; ok && t < tiles; t += t_step) {
        for (int g = kb0; ok && g < kb1; g += 4) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int i = 0; i < NI; ++i) av[i][c] = an[i][c];
#pragma unroll
            for (int m = 0; m < NMAT; ++m) wv[m][c] = wn[m][c];
          }
          if (g + 4 < kb1) {
            load(g + 4);
          } else if (t + t_step < tiles) {
            set_tile(t + t_step);
            load(kb0);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (g + c >= kb1 || !ok) break;
#pragma unroll
            for (int m = 0; m < NMAT; ++m, ++sl) {
              const int q = static_cast<int>(sl % C::NSLOT);
              if (!(ok = warp_wait(&slot_empty[q], ((sl / C::NSLOT) & 1u) ^ 1u, abort_flag, a.status))) break;
#pragma unroll
              for (int i = 0; i < NI; ++i)
                if (c0 + 64 * i < NT) sc_base[q * NT + c0 + 64 * i] = av[i][c] * wv[m][c];
              __syncwarp();
              if (lane == 0) mbar_arrive(&slot_full[q]);
            }
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
    const int half = (warp - 4) >> 2;          // chunks half, half + 2, ...
    const int r = 32 * q4 + lane;              // weight row within a 128-row block
    const uint32_t tq = tbase + (static_cast<uint32_t>(32 * q4) << 16);
    uint32_t sl = 0;
    bool ok = true;
    for (int t = t_first; ok && t < tiles; t += t_step) {
      const F8Tile ti = tile_at(t);
      const int nch = ti.npad >> 4;
      f32x2 acc[NMAT][C::NCH][8];
#pragma unroll
      for (int m = 0; m < NMAT; ++m)
#pragma unroll
        for (int c = 0; c < C::NCH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[m][c][i] = 0ull;
      for (int kb = kb0; ok && kb < kb1; ++kb) {
#pragma unroll
        for (int m = 0; m < NMAT; ++m, ++sl) {
          const int q = static_cast<int>(sl % C::NSLOT);
          if (!(ok = warp_wait(&slot_full[q], (sl / C::NSLOT) & 1u, abort_flag, a.status))) break;
          tc_fence_after();
          const uint32_t sca = smem_addr(sc_base + q * NT);
#pragma unroll
          for (int c = 0; c < C::NCH; ++c) {
            const int ch = 2 * c + half;
            if (ch < nch) {
              uint32_t d[16];
              tmem_ld16(tq + q * NT + ch * 16, d);
              f32x2 s[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) lds_2x64(sca + ch * 64 + i * 16, s[2 * i], s[2 * i + 1]);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) fma2(acc[m][c][i], d[2 * i], d[2 * i + 1], s[i]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&slot_empty[q]);
        }
      }
      if (!ok) break;
      if constexpr (GU) {
        // h, the maximum of its 128 columns per token, codes and scale
        float* rw = red + q4 * NT;
#pragma unroll
        for (int c = 0; c < C::NCH; ++c) {
          const int ch = 2 * c + half;
          if (ch < nch) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 g = unpack2(acc[0][c][i]), u = unpack2(acc[1][c][i]);
              const float h0 = g.x / (1.0f + expf(-g.x)) * u.x, h1 = g.y / (1.0f + expf(-g.y)) * u.y;
              asm("mov.b64 %0, {%1, %2};" : "=l"(acc[0][c][i]) : "f"(h0), "f"(h1));
              // magnitudes compare as unsigned integers, NaN above infinity
              const uint32_t m0 = __reduce_max_sync(0xffffffffu, __float_as_uint(h0) & 0x7fffffffu);
              const uint32_t m1 = __reduce_max_sync(0xffffffffu, __float_as_uint(h1) & 0x7fffffffu);
              if (lane == 0) {
                rw[ch * 16 + 2 * i] = __uint_as_float(m0);
                rw[ch * 16 + 2 * i + 1] = __uint_as_float(m1);
              }
            }
          }
        }
        half_barrier(half);
        uint8_t* hq = static_cast<uint8_t*>(a.out);
#pragma unroll
        for (int c = 0; c < C::NCH; ++c) {
          const int ch = 2 * c + half;
          if (ch < nch) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int n = ch * 16 + i;
              if (n < ti.ntok) {
                const float m = max_nan(max_nan(red[n], red[NT + n]), max_nan(red[2 * NT + n], red[3 * NT + n]));
                float inv;
                const float scl = f8_scale(m, &inv);
                const float2 h = unpack2(acc[0][c][i >> 1]);
                const size_t row = static_cast<size_t>(ti.orow + n);
                hq[row * a.R + ti.rblk * 128 + r] =
                    static_cast<uint8_t>(__nv_cvt_float_to_fp8((i & 1 ? h.y : h.x) * inv, __NV_SATFINITE, __NV_E4M3));
                if (r == 0) a.out_s[row * nrb + ti.rblk] = scl;
              }
            }
          }
        }
        half_barrier(half);      // the maxima have been read
      } else if (split == 1) {
#pragma unroll
        for (int m = 0; m < NMAT; ++m) {
          const int col = ti.rblk * ROWS + m * 128 + r;
          if (col < a.R) {
#pragma unroll
            for (int c = 0; c < C::NCH; ++c) {
              const int ch = 2 * c + half;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int n = ch * 16 + i;
                if (n < ti.ntok) {
                  const float2 v = unpack2(acc[m][c][i >> 1]);
                  const float y = i & 1 ? v.y : v.x;
                  const size_t at = static_cast<size_t>(ti.orow + n) * a.R + col;
                  if (a.out_f32)
                    static_cast<float*>(a.out)[at] = y;
                  else
                    static_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(y);
                }
              }
            }
          }
        }
      } else {
        // split K: totals to shared memory (every copy and MMA of this CTA is done:
        // its last slot was full), [column][NMAT * 128] so that lanes are neighbours
        float* tot = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int m = 0; m < NMAT; ++m)
#pragma unroll
          for (int c = 0; c < C::NCH; ++c) {
            const int ch = 2 * c + half;
            if (ch < nch) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 v = unpack2(acc[m][c][i]);
                tot[(ch * 16 + 2 * i) * (NMAT * 128) + m * 128 + r] = v.x;
                tot[(ch * 16 + 2 * i + 1) * (NMAT * 128) + m * 128 + r] = v.y;
              }
            }
          }
      }
    }
    if (split > 1) {
      cluster_arrive();
      cluster_wait();
      if (ok && t_first < tiles) {
        // this CTA adds its share of the columns over the ranks, in rank order
        const F8Tile ti = tile_at(t_first);
        const int x = threadIdx.x - 128;
        constexpr int PER = 256 / (NMAT * 128);           // columns at a time
        const int row = x % (NMAT * 128);
        const int col = ti.rblk * ROWS + row;
        const uint32_t base = smem_addr(smem);
        for (int n = rank * PER + x / (NMAT * 128); n < ti.ntok; n += split * PER) {
          float y = 0.f;
          for (int c = 0; c < split; ++c) y += ld_cluster_f32(base + (n * (NMAT * 128) + row) * 4, c);
          if (col < a.R) {
            const size_t at = static_cast<size_t>(ti.orow + n) * a.R + col;
            if (a.out_f32)
              static_cast<float*>(a.out)[at] = y;
            else
              static_cast<uint16_t*>(a.out)[at] = float_to_bf16_bits(y);
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
