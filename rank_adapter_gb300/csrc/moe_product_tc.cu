// The experts' products on the tensor cores (bf16 and microscaled 4-bit).
//
// The weights are the MMA's A operand (128 outputs a CTA, 256 a CTA pair) and
// the gathered x rows its B operand, so the side that varies, a segment's
// rows, is the MMA's N: a tile takes as many rows as the segment has, in
// steps of 32, and a ragged or short segment pays for little it does not use.
// The accumulator's transpose costs nothing: a TMEM lane is an output, a
// column a row of y.
//
// A CTA pair (cta_group::2) works on one tile of 256 outputs by up to kTN rows:
// each CTA loads its own 128 weight rows (TMA) and half of the x rows (16-byte
// cp.async into the swizzled operand layout; no copy of x in segment order),
// and the leader's MMAs read both halves. That halves the x traffic of each
// SM. Pairs are persistent and walk the tiles in (segment, outputs, rows)
// order, so that pairs at work on one expert's rows share its weights in L2.
// (TMA gathers of four rows each took about 75 clocks apiece: 1908 us instead
// of 746 us for 32744 rows of 2048 by 7168 outputs in bf16.)
//
// 4-bit operands use the block-scaled MMA: codes go to shared memory like any
// operand, the scale bytes are brought by warps of their own into the layout the
// tensor core wants (32 lanes by one word of four scales for each group of 32
// rows) and copied to TMEM ahead of each stage's MMAs.
#include <cstring>

#include "tcgen05.cuh"

namespace ra {
namespace {

constexpr int kErrProduct = 8;      // bit of the work lists' device error word
constexpr int kStepBytes = 128;     // bytes of a row a stage holds: 64 bf16, 256 codes
constexpr int kRowsA = 128;         // outputs of a CTA
constexpr int kPairA = 2 * kRowsA;  // outputs of a pair
constexpr int kBytesA = kRowsA * kStepBytes;
constexpr int kEpiWarp = 4, kRowWarp = 8, kScaleWarp = 12;  // first of the four epilogue, four x and the scale warps

// Shared-memory layout and TMEM columns of a variant: tiles of up to TN rows,
// ACC accumulators, STAGES pipeline stages, SW warps that bring scales.
template <bool MX, int TN_, int ACC_, int STAGES_, int SW_ = 0>
struct Shape {
  static constexpr bool kMx = MX;
  static constexpr int kTN = TN_, kAcc = ACC_, kStages = STAGES_;
  static constexpr int kScaleWarps = SW_, kThreads = 32 * (kScaleWarp + kScaleWarps);
  // A scale warp fills two stages in a row and skips those of the others. Its
  // wait tells a stage's phases apart only while its last own stage, 2 SW - 1
  // back, lies within one turn of the pipeline.
  static_assert(MX == (kScaleWarps > 0) && STAGES_ >= 2 * SW_ - 1, "scale warps");
  static constexpr int kBytesB = TN_ / 2 * kStepBytes;
  static constexpr int kAtomsB = (TN_ + 127) / 128;             // 512-byte scale atoms of a word of the x rows
  static constexpr int kBytesSf = MX ? 2 * (1 + kAtomsB) * 512 : 0;
  static constexpr int kStageBytes = kBytesA + kBytesB + kBytesSf;
  static constexpr int kSfCols = MX ? 8 + 8 * kAtomsB : 0;       // TMEM columns of a stage's scales
  static constexpr int kSfCol = ACC_ * TN_;
  static constexpr int kUsedCols = kSfCol + STAGES_ * kSfCols;
  static constexpr int kTmemCols = kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static_assert(kUsedCols <= 512, "TMEM");
  static constexpr int kBarriers = 3 * STAGES_ + 2 * ACC_ + 1;
  static size_t smem(int num_slots) {
    return 1024 + (size_t)STAGES_ * kStageBytes + kBarriers * 8 + 16 + (size_t)(num_slots + 1) * 4;
  }
};

struct TcArgs {
  const uint8_t *x, *x_scale, *W_scale;
  int64_t ldx, ld_xs, ld_ws, ldy;  // bytes a row of x and of the scales; elements of y
  void *y;
  const int32_t *work, *sorted_rows;
  int *err;
  int num_slots, K, N, x_div;
};
struct TcMaps {
  CUtensorMap W;  // {row bytes, d_out, experts}, boxes of 128 bytes x 128 rows
};

// ------------------------------------------------------------------ PTX of the CTA pair

__device__ __forceinline__ uint32_t leader_addr(const void *p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
  return r;
}
// (With .release.cluster semantics each arrival took some 1800 clocks, three
// times a decode stage; the rows it vouches for are ordered by the proxy fence
// before it, an accumulator read by tcgen05.wait::ld.)
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void tma_w(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
// One arrival on a barrier of this CTA when the thread's cp.async so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tmem_alloc2(uint32_t *slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               ::"r"(smem_addr(slot)), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// One arrival on the barrier at this offset in both CTAs once every MMA issued so far is complete.
__device__ __forceinline__ void mma_commit2(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\t.reg .b16 m;\n\telect.sync r|e, 0xffffffff;\n\tmov.b16 m, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}"
      ::"r"(smem_addr(bar)) : "memory");
}
// The four MMAs of a stage (32 bytes of each row a step), one elected lane.
__device__ __forceinline__ void mma_stage_bf16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred q, e, t;\n\t.reg .b32 r;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync r|e, 0xffffffff;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, %3, %3;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, t;\n\t}"
      ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(acc) : "memory");
}
// The same on 4-bit operands: 64 elements a step; a word of four scales serves
// two steps, which take its bytes 0-1 and 2-3 (the scale ids in the descriptor).
__device__ __forceinline__ void mma_stage_mx(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id0, uint32_t id2,
                                             uint32_t sa0, uint32_t sa1, uint32_t sb0, uint32_t sb1, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred q, e, t;\n\t.reg .b32 r;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "elect.sync r|e, 0xffffffff;\n\tsetp.ne.b32 q, %9, 0;\n\tsetp.eq.b32 t, %3, %3;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%7], q;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a1, b1, %4, [%5], [%7], t;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a2, b2, %3, [%6], [%8], t;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a3, b3, %4, [%6], [%8], t;\n\t}"
      ::"r"(d), "l"(ad), "l"(bd), "r"(id0), "r"(id2), "r"(sa0), "r"(sa1), "r"(sb0), "r"(sb1), "r"(acc) : "memory");
}
// 32 rows of 16 bytes in shared memory to four TMEM columns, in each quarter of the lanes (one elected lane).
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t sdesc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(sdesc) : "memory");
}
// kind::f16: fp32 accumulator, bf16 A and B, both K-major.
__device__ __forceinline__ uint32_t idesc_bf16_kk(int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kPairA >> 4) << 24);
}
// kind::mxf4: e2m1 A and B, scales 2^(b - 127), scale ids (both operands) `id`.
__device__ __forceinline__ uint32_t idesc_mx(int N, uint32_t id) {
  return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(kPairA >> 4) << 24) | (id << 29);
}

// ------------------------------------------------------------------ tiles

// Row tiles of a segment of `count` pairs: as few as kTN allows, of equal
// size rounded up to 32 (the last one may be shorter, never empty).
template <int TN> __device__ __forceinline__ int row_tiles(int count) { return (count + TN - 1) / TN; }

struct Tile {
  int slot, first, rows, f0;  // first sorted row, rows, first output of the pair
  __device__ __forceinline__ int n_pad() const { return (rows + 31) & ~31; }
};
template <int TN>
__device__ __forceinline__ Tile tile_at(const int32_t *work, int num_slots, const int32_t *cum, int n_list, int F,
                                        int64_t t) {
  int lo = 0, hi = n_list - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)cum[mid] * F <= t) lo = mid;
    else hi = mid - 1;
  }
  const int ntt = cum[lo + 1] - cum[lo];
  const int64_t local = t - (int64_t)cum[lo] * F;
  const int f = (int)(local / ntt), tt = (int)(local - (int64_t)f * ntt);
  const int4 rec = *reinterpret_cast<const int4 *>(work + WorkLists::list(num_slots, kListAll) + lo * WorkLists::kRec);
  const int tr = (((rec.z + ntt - 1) / ntt) + 31) & ~31;
  Tile r;
  r.slot = rec.y;
  r.first = rec.w + tt * tr;
  r.rows = min(tr, rec.z - tt * tr);
  r.f0 = f * kPairA;
  return r;
}

// ------------------------------------------------------------------ kernel

template <class S, typename TY>
__global__ void __launch_bounds__(S::kThreads, 1) moe_product_tc_kernel(const __grid_constant__ TcMaps maps, const TcArgs a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = align1024(smem_raw);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::kStages * S::kStageBytes);  // leader's: a stage of both CTAs is in
  uint64_t *empty = full + S::kStages;  // the stage's MMAs are done
  uint64_t *rows = empty + S::kStages;  // this CTA's x rows (and scales) of a stage are in
  uint64_t *accf = rows + S::kStages;   // an accumulator is complete
  uint64_t *acce = accf + S::kAcc;      // leader's: both CTAs have read it
  uint64_t *fin = acce + S::kAcc;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(fin + 1);
  int32_t *cum = reinterpret_cast<int32_t *>(tslot + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 3);  // the weights' bytes, and each CTA's rows
      mbar_init(&empty[s], 1);
      mbar_init(&rows[s], 128 + (S::kMx ? 1 : 0));
    }
    for (int i = 0; i < S::kAcc; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 8);
    }
    mbar_init(fin, 1);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc2(tslot, S::kTmemCols);
  pdl_wait();
  pdl_trigger();
  const int n_list = a.work[0];
  if (warp == 3) {  // row tiles before each segment
    int base = 0;
    for (int i0 = 0; i0 < n_list; i0 += 32) {
      const int i = i0 + lane;
      const int c = i < n_list ? row_tiles<S::kTN>(a.work[WorkLists::list(a.num_slots, kListAll) + i * WorkLists::kRec + 2]) : 0;
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (i < n_list) cum[i] = base + incl - c;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) cum[n_list] = base;
  }
  tc_before_sync();
  cluster_sync();  // also a CTA barrier: cum, the barriers and the TMEM address are visible
  tc_after_sync();
  const uint32_t tmem = *tslot;
  const int F = (a.N + kPairA - 1) / kPairA;
  const int64_t n_tiles = (int64_t)cum[n_list] * F;
  const int row_bytes = S::kMx ? a.K / 2 : a.K * 2;
  const int nkb = (row_bytes + kStepBytes - 1) / kStepBytes;
  const int64_t t0 = blockIdx.x >> 1, dt = gridDim.x >> 1;
  auto tile = [&](int64_t t) { return tile_at<S::kTN>(a.work, a.num_slots, cum, n_list, F, t); };
  constexpr int kElemsPerStep = S::kMx ? kStepBytes : kStepBytes / 2;  // in units of the tensor maps' elements

  if (warp == 0) {
    // ---- weights
    uint32_t it = 0;
    bool ok = true;
    for (int64_t t = t0; t < n_tiles && ok; t += dt) {
      const Tile ti = tile(t);
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const uint32_t s = it % S::kStages;
        if (!mbar_wait_warp(&empty[s], ((it / S::kStages) & 1) ^ 1, a.err, kErrProduct)) { ok = false; break; }
        if (lane == 0) {
          if (rank == 0) mbar_arrive_tx(&full[s], 2 * kBytesA);
          tma_w(smem_addr(sm + s * S::kStageBytes), &maps.W, kb * kElemsPerStep, ti.f0 + (int)rank * kRowsA,
                ti.slot - 1, leader_addr(&full[s]));
        }
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ---- passes this CTA's rows on to the leader. The rows were written by
    // ordinary stores and cp.async; the fence orders them before the tensor
    // core's reads.
    uint32_t it = 0;
    bool ok = true;
    for (int64_t t = t0; t < n_tiles && ok; t += dt)
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const uint32_t s = it % S::kStages;
        if (!mbar_wait_warp(&rows[s], (it / S::kStages) & 1, a.err, kErrProduct)) { ok = false; break; }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(leader_addr(&full[s]));
      }
  } else if (warp == 2) {
    // ---- MMA issue (leader)
    if (rank == 0) {
      uint32_t it = 0, item = 0;
      bool ok = true;
      for (int64_t t = t0; t < n_tiles && ok; t += dt, ++item) {
        const int n = tile(t).n_pad();
        const uint32_t acc = item % S::kAcc, d = tmem + acc * S::kTN;
        if (!mbar_wait_warp(&acce[acc], ((item / S::kAcc) & 1) ^ 1, a.err, kErrProduct)) break;
        tc_after_sync();
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          const uint32_t s = it % S::kStages;
          if (!mbar_wait_warp(&full[s], (it / S::kStages) & 1, a.err, kErrProduct)) { ok = false; break; }
          tc_after_sync();
          const uint32_t st = smem_addr(sm + s * S::kStageBytes);
          const uint64_t ad = smem_desc(st, 16, 1024, kSw128), bd = smem_desc(st + kBytesA, 16, 1024, kSw128);
          if constexpr (S::kMx) {
            const uint32_t sf = st + kBytesA + S::kBytesB, sa = tmem + S::kSfCol + s * S::kSfCols, sb = sa + 8;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              scales_to_tmem(sa + 4 * w, smem_desc(sf + w * 512, 16, 128, 0));
#pragma unroll
              for (int h = 0; h < S::kAtomsB; ++h)
                scales_to_tmem(sb + 4 * (w * S::kAtomsB + h), smem_desc(sf + 1024 + (w * S::kAtomsB + h) * 512, 16, 128, 0));
            }
            mma_stage_mx(d, ad, bd, idesc_mx(n, 0), idesc_mx(n, 2), sa, sa + 4, sb, sb + 4 * S::kAtomsB, kb > 0);
          } else {
            mma_stage_bf16(d, ad, bd, idesc_bf16_kk(n), kb > 0);
          }
          mma_commit2(&empty[s]);
        }
        if (ok) mma_commit2(&accf[acc]);
      }
      mma_commit2(fin);
      mbar_wait_warp(fin, 0, a.err, kErrProduct);  // every MMA is done before either CTA leaves
    }
  } else if (warp >= kEpiWarp && warp < kEpiWarp + 4) {
    // ---- accumulator -> y: a lane holds an output, a column a row
    const int q = warp & 3;
    TY *y = static_cast<TY *>(a.y);
    uint32_t item = 0;
    for (int64_t t = t0; t < n_tiles; t += dt, ++item) {
      const Tile ti = tile(t);
      const uint32_t acc = item % S::kAcc;
      if (!mbar_wait_warp(&accf[acc], (item / S::kAcc) & 1, a.err, kErrProduct)) break;
      tc_after_sync();
      const int f = ti.f0 + (int)rank * kRowsA + q * 32 + lane;
      for (int c = 0; c < ti.rows; c += 32) {
        const int row = c + lane < ti.rows ? a.sorted_rows[ti.first + c + lane] : 0;
        float v[32];
        tmem_ld32_async(tmem + ((uint32_t)(q * 32) << 16) + acc * S::kTN + c, v);
        tmem_wait_ld();
        const int m = min(32, ti.rows - c);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int64_t rj = __shfl_sync(0xffffffffu, row, j);
          if (j < m && f < a.N) y[rj * a.ldy + f] = Elem<TY>::from_f(v[j]);
        }
      }
      tc_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_addr(&acce[acc]));
    }
  } else if (warp >= kRowWarp && warp < kRowWarp + 4) {
    // ---- x rows: this CTA's half of the tile's rows, a thread the same 16
    // bytes of every 16th row of a stage
    constexpr int kMine = S::kTN / 32;
    const int tid = threadIdx.x - kRowWarp * 32, r0 = tid >> 3, chunk = tid & 7;
    uint32_t it = 0;
    bool ok = true;
    for (int64_t t = t0; t < n_tiles && ok; t += dt) {
      const Tile ti = tile(t);
      const int half = ti.n_pad() / 2;
      const uint8_t *src[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i)  // rows past the segment repeat its last one; their columns are not stored
        src[i] = a.x + (int64_t)(a.sorted_rows[ti.first + min((int)rank * half + r0 + 16 * i, ti.rows - 1)] / a.x_div) * a.ldx + chunk * 16;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const uint32_t s = it % S::kStages;
        if (!mbar_wait_warp(&empty[s], ((it / S::kStages) & 1) ^ 1, a.err, kErrProduct)) { ok = false; break; }
        unsigned char *st = sm + s * S::kStageBytes + kBytesA;
        const int off = kb * kStepBytes;
        const bool in = off + chunk * 16 < row_bytes;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int r = r0 + 16 * i;
          if (r < half) cp_async16_zfill(st + swz128(r, chunk), in ? src[i] + off : a.x, in);
        }
        cp_async_arrive(&rows[s]);
      }
    }
    cp_async_wait_upto(0);
  } else if constexpr (S::kMx) if (warp >= kScaleWarp) {
    // ---- scale bytes. The warps take chunks of 512 elements (16 bytes a
    // row, two stages) in turn; lane l holds rows l, l + 32, ... of the weights
    // and of x. Words land as [row % 32][row / 32 % 4] of a 512-byte atom.
    uint32_t it = 0, chunk = 0;
    const int nb = a.K / LORA_MX_BLOCK;
    bool ok = true;
    for (int64_t t = t0; t < n_tiles && ok; t += dt, it += nkb) {
      const Tile ti = tile(t);
      constexpr int kGb = 4 * S::kAtomsB;
      const uint8_t *pa[4], *pb[kGb];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int f = min(ti.f0 + (int)rank * kRowsA + 32 * g + lane, a.N - 1);
        pa[g] = a.W_scale + ((int64_t)(ti.slot - 1) * a.N + f) * a.ld_ws;
      }
#pragma unroll
      for (int g = 0; g < kGb; ++g)
        pb[g] = a.x_scale + (int64_t)(a.sorted_rows[ti.first + min(32 * g + lane, ti.rows - 1)] / a.x_div) * a.ld_xs;
      for (int kb0 = 0; kb0 < nkb && ok; kb0 += 2, ++chunk) {
        if (chunk % S::kScaleWarps != (uint32_t)(warp - kScaleWarp)) continue;
        uint4 va[4], vb[kGb];
#pragma unroll
        for (int g = 0; g < 4; ++g) va[g] = __ldg(reinterpret_cast<const uint4 *>(pa[g] + kb0 * 8));
#pragma unroll
        for (int g = 0; g < kGb; ++g)
          if (32 * g < ti.rows) vb[g] = __ldg(reinterpret_cast<const uint4 *>(pb[g] + kb0 * 8));
          else vb[g] = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // the chunk's stages
          if (kb0 + h >= nkb) break;
          const uint32_t i = it + kb0 + h, s = i % S::kStages;
          if (!mbar_wait_warp(&empty[s], ((i / S::kStages) & 1) ^ 1, a.err, kErrProduct)) { ok = false; break; }
          unsigned char *sf = sm + s * S::kStageBytes + kBytesA + S::kBytesB;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            // Scales past the row's blocks stand beside codes the loads filled with
            // zeros; any number will do, a NaN would not.
            const int left = nb - ((kb0 + h) * 8 + 4 * w);
            const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            auto word = [&](const uint4 &v) {
              const uint32_t u = h == 0 ? (w == 0 ? v.x : v.y) : (w == 0 ? v.z : v.w);
              return (u & keep) | (0x7f7f7f7fu & ~keep);
            };
            *reinterpret_cast<uint4 *>(sf + w * 512 + lane * 16) = make_uint4(word(va[0]), word(va[1]), word(va[2]), word(va[3]));
#pragma unroll
            for (int b = 0; b < S::kAtomsB; ++b)
              *reinterpret_cast<uint4 *>(sf + 1024 + (w * S::kAtomsB + b) * 512 + lane * 16) =
                  make_uint4(word(vb[4 * b]), word(vb[4 * b + 1]), word(vb[4 * b + 2]), word(vb[4 * b + 3]));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&rows[s]);
        }
      }
    }
  }
  tc_before_sync();
  cluster_sync();  // no barrier of this CTA is signalled after its peer is past here
  if (warp == 2) {
    tc_after_sync();
    tmem_free2(tmem, S::kTmemCols);
  }
}

// ------------------------------------------------------------------ host side

cudaError_t encode(CUtensorMap *m, const void *base, bool mx, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                   const cuuint32_t *box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = enc(m, mx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
                         const_cast<void *>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Pairs of this kernel the device holds at once.
template <class S, typename TY>
cudaError_t resident_pairs(size_t smem, int *out) {
  static std::mutex mu;
  static std::map<std::pair<int, size_t>, int> cache;  // (device, shared memory)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find({dev, smem});
  if (it == cache.end()) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, moe_product_tc_kernel<S, TY>, &cfg);
    if (e != cudaSuccess) return e;
    it = cache.emplace(std::make_pair(dev, smem), std::max(1, n)).first;
  }
  *out = it->second;
  return cudaSuccess;
}

template <class S, typename TY>
cudaError_t launch(const TcMaps &maps, const TcArgs &a, int num_tokens, cudaStream_t st) {
  const size_t smem = S::smem(a.num_slots);
  cudaError_t e = set_max_dynamic_smem((const void *)moe_product_tc_kernel<S, TY>, (int)smem);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  e = resident_pairs<S, TY>(smem, &pairs);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)num_tokens / S::kTN + std::min(a.num_slots - 1, num_tokens)) * ((a.N + kPairA - 1) / kPairA);
  const unsigned grid = 2u * (unsigned)std::min<int64_t>(tiles, pairs);
  return launch_pdl(moe_product_tc_kernel<S, TY>, dim3(grid), dim3(S::kThreads), smem, st, 2u, maps, a);
}

template <class S>
cudaError_t launch(const TcMaps &maps, const TcArgs &a, int num_tokens, int y_dtype, cudaStream_t st) {
  return y_dtype == LORA_BF16 ? launch<S, __nv_bfloat16>(maps, a, num_tokens, st) : launch<S, float>(maps, a, num_tokens, st);
}

using NarrowBf16 = Shape<false, 64, 2, 10>;
using WideBf16 = Shape<false, 256, 2, 6>;
using NarrowMx = Shape<true, 64, 2, 9, 4>;
using WideMx = Shape<true, 192, 2, 5, 2>;

}  // namespace

cudaError_t launch_moe_product_tc(const lora_expert_desc &d, const MetaView &mv, const void *x, int64_t ldx,
                                  const uint8_t *x_scale, int64_t ld_xs, void *y, int64_t ldy, int y_dtype,
                                  cudaStream_t st) {
  const bool mx = d.dtype == LORA_MXFP4;
  const int div = std::max(1, d.x_row_div);
  const cuuint64_t row_bytes = mx ? (cuuint64_t)d.d_in / 2 : (cuuint64_t)d.d_in * 2;
  const cuuint64_t elems = mx ? row_bytes : (cuuint64_t)d.d_in;
  const cuuint32_t step = mx ? kStepBytes : kStepBytes / 2;
  TcMaps maps;
  const cuuint64_t wd[3] = {elems, (cuuint64_t)d.d_out, (cuuint64_t)d.num_experts};
  const cuuint64_t ws[2] = {row_bytes, row_bytes * (cuuint64_t)d.d_out};
  const cuuint32_t wb[3] = {step, kRowsA, 1};
  cudaError_t e = encode(&maps.W, d.W, mx, 3, wd, ws, wb);
  if (e != cudaSuccess) return e;
  TcArgs a;
  a.x = static_cast<const uint8_t *>(x);
  a.ldx = mx ? ldx / 2 : ldx * 2;
  a.x_scale = x_scale;
  a.W_scale = d.W_scale;
  a.ld_xs = ld_xs;
  a.ld_ws = d.ld_scale;
  a.ldy = ldy;
  a.y = y;
  a.work = mv.work;
  a.sorted_rows = mv.sorted_rows;
  a.err = const_cast<int32_t *>(mv.work) + WorkLists::kErrWord;
  a.num_slots = mv.num_slots;
  a.K = d.d_in;
  a.N = d.d_out;
  a.x_div = div;
  const bool narrow = mv.num_tokens <= 64 * (mv.num_slots - 1);
  if (mx) return narrow ? launch<NarrowMx>(maps, a, mv.num_tokens, y_dtype, st) : launch<WideMx>(maps, a, mv.num_tokens, y_dtype, st);
  return narrow ? launch<NarrowBf16>(maps, a, mv.num_tokens, y_dtype, st) : launch<WideBf16>(maps, a, mv.num_tokens, y_dtype, st);
}

}  // namespace ra
