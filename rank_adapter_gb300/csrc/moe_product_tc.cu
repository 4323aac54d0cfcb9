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
//
// What bounds it (w2 prefill: 32744 rows of 16 experts, 2048 by 7168; w13:
// 7168 by 4096): few rows, the weights' bytes (7.0 to 7.5 TB/s); bf16 prefill
// the tensor pipe, 96 % active, and the power cap (w2 in short runs 512 us, 1.88
// PFLOP/s, sustained 598 to 635 us, 1.5 to 1.6 PFLOP/s); 4-bit prefill no single
// unit (tensor pipe 54 % active, shared memory 64 % busy) but the order of scale
// copies and MMAs in the tensor pipe (w13 in short runs 367 us, 5.2 PFLOP/s,
// sustained 381 to 388 us); one or two experts' few tiles the pipeline's round
// trip, about 0.2 us a stage.
#include <atomic>

#include "mx.cuh"
#include "tcgen05.cuh"

namespace ra {
namespace {

constexpr int kErrProduct = 8;      // bit of the work lists' device error word
constexpr int kStepBytes = 128;     // bytes of a row a stage holds: 64 bf16, 256 codes
constexpr int kRowsA = 128;         // outputs of a CTA
constexpr int kPairA = 2 * kRowsA;  // outputs of a pair
constexpr int kBytesA = kRowsA * kStepBytes;

// Warps of a CTA: 0 weights, 1 passes this CTA's rows on to the leader, 2 MMA,
// 3 tiles, then four of the epilogue, eight of the x rows and the scale warps.
constexpr int kRowWarp = 8, kRowWarps = 8, kScaleWarp = kRowWarp + kRowWarps;
constexpr int kRing = 3;            // tiles described ahead

// A tile as its warps read it.
template <int TN>
struct alignas(16) TileInfo {
  int expert, rows, f0, pad;        // rows of the tile, first output of the pair
  int x[TN], y[TN];                 // the rows' x rows (past the tile the last one again) and y rows
  __device__ __forceinline__ int n_pad() const { return (rows + 31) & ~31; }
};

// Shared-memory layout and TMEM columns of a variant: tiles of up to TN rows,
// ACC accumulators, STAGES pipeline stages, SW warps that bring scales.
template <bool MX, int TN_, int ACC_, int STAGES_, int SW_ = 0>
struct Shape {
  static constexpr bool kMx = MX;
  static constexpr int kTN = TN_, kAcc = ACC_, kStages = STAGES_;
  static constexpr int kScaleWarps = SW_, kThreads = 32 * (kScaleWarp + kScaleWarps + (MX ? 1 : 0));
  // A scale warp fills two stages in a row and skips those of the others. Its
  // wait tells a stage's phases apart only while its last own stage, 2 SW - 1
  // back, lies within one turn of the pipeline.
  static_assert(MX == (kScaleWarps > 0) && STAGES_ >= 2 * SW_ - 1, "scale warps");
  static constexpr int kBytesB = TN_ / 2 * kStepBytes;
  static constexpr int kAtomsB = (TN_ + 127) / 128;              // 512-byte scale atoms of a word of the x rows
  static constexpr int kBytesSf = MX ? 2 * (1 + kAtomsB) * 512 : 0;
  static constexpr int kStageBytes = kBytesA + kBytesB + kBytesSf;
  // TMEM: the accumulators, then each stage's scales.
  static constexpr int kSfCols = MX ? 8 + 8 * kAtomsB : 0, kSfCol = ACC_ * TN_;
  static constexpr int kUsedCols = kSfCol + STAGES_ * kSfCols;
  static constexpr int kTmemCols = kUsedCols <= 128 ? 128 : kUsedCols <= 256 ? 256 : 512;
  static_assert(kUsedCols <= 512, "TMEM");
  static constexpr int kBarriers = 4 * STAGES_ + 2 * ACC_ + 2 * kRing + 1;
  static constexpr int kTurnOff = STAGES_ * kStageBytes;         // the epilogue warps' blocks of 32 rows
  static constexpr int kTurnBytes = 32 * (32 + 4) * 4;
  static constexpr int kRingOff = kTurnOff + 4 * kTurnBytes;
  static constexpr int kBarOff = kRingOff + kRing * (int)sizeof(TileInfo<TN_>);
  static constexpr int kCumOff = kBarOff + kBarriers * 8 + 16;
  static constexpr int kSmem = 1024 + kCumOff + LORA_MAX_NUM_SLOTS * 4;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct TcArgs {
  const uint8_t *x, *x_scale;
  int64_t ldx, ld_xs, ldy;         // bytes a row of x and of the scales; elements of y
  void *y;
  const int32_t *work, *sorted_rows;
  int *err;
  int num_slots, K, N, x_div;
};
struct TcMaps {
  CUtensorMap W_scale;  // {256 words, pairs of tiles}, boxes of one pair (4-bit weights)
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
// Waits for all of the thread's cp.async (they are in no commit group).
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void tma_scales(uint32_t dst, const CUtensorMap *map, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(bar) : "memory");
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
// One arrival on the leader's barrier once every tensor-core copy issued so far is complete.
__device__ __forceinline__ void commit2_leader(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
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
// 16 lanes by 32 columns, without waiting: register 4 i + {0, 1} holds row
// lane / 4, columns 8 i + 2 (lane % 4) + {0, 1}, register 4 i + {2, 3} row 8 + lane / 4.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}
// Two fp32 values, rounded to nearest, as bf16 (the first in the low half).
__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Four 8 x 8 blocks of 16-bit elements, transposed; lane l gives the address of row l % 8 of block l / 8.
__device__ __forceinline__ void store_transposed(uint32_t addr, const uint32_t (&p)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
               ::"r"(addr), "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]) : "memory");
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

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// 16-byte cp.async to a shared-memory address, zeros when !valid (nothing is read then).
__device__ __forceinline__ void cp_async16_to(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

// Position in a ring of N: the slot, and the parity of the turn.
template <int N>
struct Stage {
  uint32_t s = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      phase ^= 1;
    }
  }
};

// ------------------------------------------------------------------ kernel

template <class S, typename TY>
__global__ void __launch_bounds__(S::kThreads, 1) moe_product_tc_kernel(const __grid_constant__ TcMaps maps, const TcArgs a) {
  extern __shared__ unsigned char smem_raw[];
  using Info = TileInfo<S::kTN>;
  unsigned char *sm = align1024(smem_raw);
  Info *ring = reinterpret_cast<Info *>(sm + S::kRingOff);
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + S::kBarOff);  // leader's: a stage of both CTAs is in
  uint64_t *empty = full + S::kStages;  // the stage's MMAs are done
  uint64_t *rows = empty + S::kStages;  // this CTA's x rows (and scales) of a stage are in
  uint64_t *sfull = rows + S::kStages;  // leader's: a stage's scales are in TMEM (4-bit)
  uint64_t *accf = sfull + S::kStages;  // an accumulator is complete
  uint64_t *acce = accf + S::kAcc;      // leader's: both CTAs have read it
  uint64_t *tfull = acce + S::kAcc;     // a tile is described
  uint64_t *tempty = tfull + kRing;     // every warp has what it needs of it
  uint64_t *fin = tempty + kRing;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(fin + 1);
  int32_t *lists = reinterpret_cast<int32_t *>(tslot + 1);  // segments, row tiles of them all
  int32_t *cum = reinterpret_cast<int32_t *>(sm + S::kCumOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 3);  // the weights' bytes, and each CTA's rows
      mbar_init(&empty[s], 1);
      mbar_init(&sfull[s], 1);
      mbar_init(&rows[s], 128 + (S::kMx ? 1 : 0));
    }
    for (int i = 0; i < S::kAcc; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 8);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 1 + (rank == 0 ? 1 : 0) + 4 + kRowWarps + S::kScaleWarps);
    }
    mbar_init(fin, 1);
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc2(tslot, S::kTmemCols);
  if (warp == 0 && lane == 0) prefetch_map(&maps.W);
  if (S::kMx && warp == 0 && lane == 1) prefetch_map(&maps.W_scale);
  pdl_wait();
  const int32_t *list = a.work + WorkLists::list(a.num_slots, kListAll);
  // Records of the list: segment, slot, pairs, first sorted row; unused ones hold -1.
  auto record = [&](int i) {
    return i < a.num_slots ? *reinterpret_cast<const int4 *>(list + i * WorkLists::kRec) : make_int4(-1, 0, 0, 0);
  };
  int4 head = make_int4(-1, 0, 0, 0);  // warp 3: record `lane`
  if (warp == 3) {  // row tiles before each segment: as few as kTN allows
    head = record(lane);
    const int n_list = a.work[0];
    int base = 0;
    int4 rec = head;
    for (int i0 = 0; i0 < n_list; i0 += 32) {
      const int i = i0 + lane;
      int incl = rec.z > 0 ? (rec.z + S::kTN - 1) / S::kTN : 0;
      const int mine = incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (i < n_list) cum[i] = base + incl - mine;
      base += __shfl_sync(0xffffffffu, incl, 31);
      if (i0 + 32 < n_list) rec = record(i + 32);
    }
    if (lane == 0) {
      cum[n_list] = base;
      lists[0] = n_list;
      lists[1] = base;
    }
  }
  tc_before_sync();
  cluster_sync();  // also a CTA barrier: cum, the barriers and the TMEM address are visible
  tc_after_sync();
  pdl_trigger();  // only now: a successor that takes TMEM must not start before this CTA has its own
  const uint32_t tmem = *tslot;
  const int F = (a.N + kPairA - 1) / kPairA, n_list = lists[0];
  const int row_bytes = S::kMx ? a.K / 2 : a.K * 2;
  const int nkb = (row_bytes + kStepBytes - 1) / kStepBytes;
  const int64_t n_tiles = (int64_t)lists[1] * F, t0 = blockIdx.x >> 1, dt = gridDim.x >> 1;
  const uint32_t n_items = n_tiles > t0 ? (uint32_t)((n_tiles - t0 + dt - 1) / dt) : 0u;  // tiles of this pair
  constexpr int kElemsPerStep = S::kMx ? kStepBytes : kStepBytes / 2;  // in units of the tensor maps' elements
  // Item `item` of this pair, once it is described (nullptr: the wait ran out), and its release.
  auto tile = [&](uint32_t item) -> const Info * {
    return mbar_wait_warp(&tfull[item % kRing], (item / kRing) & 1, a.err, kErrProduct) ? &ring[item % kRing] : nullptr;
  };
  auto release = [&](uint32_t item) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&tempty[item % kRing]);
  };

  if (warp == 0) {
    // ---- weights
    Stage<S::kStages> st;
    bool ok = true;
    for (uint32_t item = 0; item < n_items && ok; ++item) {
      const Info *ti = tile(item);
      if (ti == nullptr) { ok = false; break; }
      const int f = ti->f0 + (int)rank * kRowsA, e = ti->expert;
      // The first pair of the CTA's scale tiles; outputs past the last tile take that one's (they are not stored).
      const int sf = S::kMx ? (e * mx_tiles_out(a.N) + min(f / kMxTile, mx_tiles_out(a.N) - 1)) * (mx_tiles_in(a.K) / 2) : 0;
      release(item);
      for (int kb = 0; kb < nkb; ++kb, st.next()) {
        if (!mbar_wait_warp(&empty[st.s], st.phase ^ 1, a.err, kErrProduct)) { ok = false; break; }
        if (lane == 0) {
          if (rank == 0) mbar_arrive_tx(&full[st.s], 2 * (kBytesA + (S::kMx ? 2 * kMxTileBytes : 0)));
          tma_w(smem_addr(sm + st.s * S::kStageBytes), &maps.W, kb * kElemsPerStep, f, e, leader_addr(&full[st.s]));
        }
        if (S::kMx && lane == 1)
          tma_scales(smem_addr(sm + st.s * S::kStageBytes + kBytesA + S::kBytesB), &maps.W_scale, sf + kb, leader_addr(&full[st.s]));
        __syncwarp();
      }
    }
    // Every stage's last use, as if to fill it again: its loads have landed and
    // its arrivals on this CTA's barriers are in. (A wait that ran out, here or
    // above, has left the loads issued before it its whole limit to land.)
    for (int i = 0; i < S::kStages && ok; ++i, st.next()) ok = mbar_wait_warp(&empty[st.s], st.phase ^ 1, a.err, kErrProduct);
  } else if (warp == 1) {
    // ---- passes this CTA's rows on to the leader. The rows were written by
    // ordinary stores and cp.async; the fence orders them before the tensor
    // core's reads.
    Stage<S::kStages> st;
    const uint64_t n = (uint64_t)n_items * nkb;
    for (uint64_t i = 0; i < n; ++i, st.next()) {
      if (!mbar_wait_warp(&rows[st.s], st.phase, a.err, kErrProduct)) break;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_addr(&full[st.s]));
    }
  } else if (warp == 2) {
    // ---- MMA issue (leader)
    if (rank == 0) {
      Stage<S::kStages> st;
      bool ok = true;
      for (uint32_t item = 0; item < n_items && ok; ++item) {
        const Info *ti = tile(item);
        if (ti == nullptr) break;
        const int n = ti->n_pad();
        release(item);
        const uint32_t acc = item % S::kAcc, d = tmem + acc * S::kTN;
        if (!mbar_wait_warp(&acce[acc], ((item / S::kAcc) & 1) ^ 1, a.err, kErrProduct)) break;
        tc_after_sync();
        for (int kb = 0; kb < nkb; ++kb, st.next()) {
          if (!mbar_wait_warp(S::kMx ? &sfull[st.s] : &full[st.s], st.phase, a.err, kErrProduct)) { ok = false; break; }
          tc_after_sync();
          const uint32_t at = smem_addr(sm + st.s * S::kStageBytes);
          const uint64_t ad = smem_desc(at, 16, 1024, kSw128), bd = smem_desc(at + kBytesA, 16, 1024, kSw128);
          if constexpr (S::kMx) {
            const uint32_t sa = tmem + S::kSfCol + st.s * S::kSfCols, sb = sa + 8;
            mma_stage_mx(d, ad, bd, idesc_mx(n, 0), idesc_mx(n, 2), sa, sa + 4, sb, sb + 4 * S::kAtomsB, kb > 0);
          } else {
            mma_stage_bf16(d, ad, bd, idesc_bf16_kk(n), kb > 0);
          }
          mma_commit2(&empty[st.s]);
        }
        if (ok) mma_commit2(&accf[acc]);
      }
      mma_commit2(fin);
      mbar_wait_warp(fin, 0, a.err, kErrProduct);  // every MMA is done before either CTA leaves
    }
  } else if (warp == 3) {
    // ---- describes the pair's tiles, kRing ahead of the slowest warp. A
    // segment's row tiles are of equal size rounded up to 32 (the last one may
    // be shorter, never empty); tiles run in (segment, outputs, rows) order.
    for (uint32_t item = 0; item < n_items; ++item) {
      const int64_t t = t0 + (int64_t)item * dt;
      int lo = 0, hi = n_list - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)cum[mid] * F <= t) lo = mid;
        else hi = mid - 1;
      }
      int4 rec;
      if (lo < 32) {
        rec.y = __shfl_sync(0xffffffffu, head.y, lo);
        rec.z = __shfl_sync(0xffffffffu, head.z, lo);
        rec.w = __shfl_sync(0xffffffffu, head.w, lo);
      } else {
        rec = record(lo);
      }
      const int ntt = cum[lo + 1] - cum[lo];
      const int64_t local = t - (int64_t)cum[lo] * F;
      const int f = (int)(local / ntt), tt = (int)(local - (int64_t)f * ntt);
      const int tr = (((rec.z + ntt - 1) / ntt) + 31) & ~31, n = min(tr, rec.z - tt * tr);
      if (!mbar_wait_warp(&tempty[item % kRing], ((item / kRing) & 1) ^ 1, a.err, kErrProduct)) break;
      Info &ti = ring[item % kRing];
      if (lane == 0) {
        ti.expert = rec.y - 1;
        ti.rows = n;
        ti.f0 = f * kPairA;
      }
      int p[S::kTN / 32];
#pragma unroll
      for (int g = 0; g < S::kTN / 32; ++g) p[g] = a.sorted_rows[rec.w + tt * tr + min(32 * g + lane, n - 1)];
#pragma unroll
      for (int g = 0; g < S::kTN / 32; ++g) {
        ti.x[32 * g + lane] = p[g] / a.x_div;
        ti.y[32 * g + lane] = p[g];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&tfull[item % kRing]);
    }
  } else if (warp < kRowWarp) {
    // ---- accumulator -> y, 32 rows of this warp's 32 outputs at a time, turned
    // round in shared memory so that a row leaves in 16-byte pieces (stored from
    // the lanes, two bytes each, the w2 prefill took 669 us instead of 558).
    constexpr int kVec = 16 / sizeof(TY), kPieces = 32 / kVec, kRowsAtOnce = 32 / kPieces;
    constexpr int kPitch = 32 + kVec;  // elements a row of the block: a piece more, which spreads the banks
    const int q = warp & 3;
    TY *y = static_cast<TY *>(a.y), *turn = reinterpret_cast<TY *>(sm + S::kTurnOff + q * S::kTurnBytes);
    const int piece = lane % kPieces, sub = lane / kPieces;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    for (uint32_t item = 0; item < n_items; ++item) {
      const uint32_t acc = item % S::kAcc;
      const Info *ti = tile(item);
      if (ti == nullptr) break;
      const int f = ti->f0 + (int)rank * kRowsA + q * 32 + piece * kVec, n = ti->rows;
      if (!mbar_wait_warp(&accf[acc], (item / S::kAcc) & 1, a.err, kErrProduct)) break;
      tc_after_sync();
      // The block in `turn` to its rows of y.
      auto rows_out = [&](int c) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; j += kRowsAtOnce) {
          const uint4 u = *reinterpret_cast<const uint4 *>(turn + (j + sub) * kPitch + piece * kVec);
          if (c + j + sub < n && f < a.N) *reinterpret_cast<uint4 *>(y + (int64_t)ti->y[c + j + sub] * a.ldy + f) = u;
        }
        __syncwarp();
      };
      if constexpr (sizeof(TY) == 2) {
        // Fragments of 16 outputs by 8 rows, packed to bf16 and stored transposed,
        // four 8 x 8 blocks an instruction. (With a lane an output and 32 two-byte
        // stores the epilogue bound products over a short d_in: about 10000 pairs
        // of 32 experts, 1216 by 7136 in 4 bits, 82 us, now 71 us.)
        uint32_t va[2][16];
        auto request = [&](uint32_t(&v)[2][16], int c) {
          tmem_ld_16x32(lanes + acc * S::kTN + c, v[0]);
          tmem_ld_16x32(lanes + (16u << 16) + acc * S::kTN + c, v[1]);
        };
        const uint32_t at = smem_addr(turn) + (uint32_t)((lane >> 4) * 8 + (lane & 7)) * (kPitch * 2) + ((lane >> 3) & 1) * 16;
        auto put = [&](uint32_t(&v)[2][16], int c) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t p[4];
#pragma unroll
              for (int m = 0; m < 4; ++m) p[m] = pack_bf16(v[h][8 * i + 2 * m], v[h][8 * i + 2 * m + 1]);
              store_transposed(at + (uint32_t)(16 * i * kPitch * 2 + 32 * h), p);
            }
          rows_out(c);
        };
        if constexpr (S::kMx) {  // registers for one block only
          for (int c = 0; c < n; c += 32) {
            request(va, c);
            tmem_wait_ld();
            put(va, c);
          }
        } else {
          uint32_t vb[2][16];
          request(va, 0);
          for (int c = 0; c < n; c += 64) {
            tmem_wait_ld();
            if (c + 32 < n) request(vb, c + 32);
            put(va, c);
            if (c + 32 >= n) break;
            tmem_wait_ld();
            if (c + 64 < n) request(va, c + 64);
            put(vb, c + 32);
          }
        }
      } else {
        for (int c = 0; c < n; c += 32) {
          float v[32];
          tmem_ld32_async(lanes + acc * S::kTN + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) turn[j * kPitch + lane] = v[j];
          rows_out(c);
        }
      }
      release(item);
      tc_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(leader_addr(&acce[acc]));
    }
    mbar_wait_warp(fin, 0, a.err, kErrProduct);  // the leader's last arrival on this CTA, right behind its last accumulator
  } else if (warp < kScaleWarp) {
    // ---- x rows: this CTA's half of the tile's rows. Two groups of four warps
    // take the stages in turn (a group needs about 640 clocks for 128 rows, an
    // MMA stage 512); a thread copies the same 16 bytes of every 16th row.
    constexpr int kMine = S::kTN / 32;
    const int group = (warp - kRowWarp) >> 2, tid = threadIdx.x & 127, r0 = tid >> 3, chunk = tid & 7;
    const uint32_t to = smem_addr(sm + kBytesA) + swz128(r0, chunk);  // 16 rows on: 2048 bytes
    Stage<S::kStages> st;
    bool odd = false, ok = true;
    for (uint32_t item = 0; item < n_items && ok; ++item) {
      const Info *ti = tile(item);
      if (ti == nullptr) break;
      const int half = ti->n_pad() / 2;
      const uint8_t *src[kMine];
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        src[i] = a.x + (int64_t)ti->x[min((int)rank * half + r0 + 16 * i, S::kTN - 1)] * a.ldx + chunk * 16;
      release(item);
      for (int kb = 0; kb < nkb; ++kb, st.next(), odd = !odd) {
        if (odd != (group != 0)) continue;
        if (!mbar_wait_warp(&empty[st.s], st.phase ^ 1, a.err, kErrProduct)) { ok = false; break; }
        const uint32_t dst = to + st.s * S::kStageBytes;
        const int off = kb * kStepBytes;
        const bool in = off + chunk * 16 < row_bytes;
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (r0 + 16 * i < half) cp_async16_to(dst + 2048 * i, in ? src[i] + off : a.x, in);
        cp_async_arrive(&rows[st.s]);
      }
    }
    cp_async_wait_all();
  } else if (S::kMx && warp == kScaleWarp + S::kScaleWarps) {
    // ---- scales of a stage to TMEM (leader). A warp of its own: with these
    // copies in the MMA warp's stream its issue bound the kernel (w13 prefill
    // 421 us, now 377 us).
    if (rank == 0) {
      Stage<S::kStages> st;
      const uint64_t n = (uint64_t)n_items * nkb;
      for (uint64_t i = 0; i < n; ++i, st.next()) {
        if (!mbar_wait_warp(&full[st.s], st.phase, a.err, kErrProduct)) break;
        tc_after_sync();
        const uint32_t sf = smem_addr(sm + st.s * S::kStageBytes) + kBytesA + S::kBytesB;
        const uint32_t sa = tmem + S::kSfCol + st.s * S::kSfCols;
#pragma unroll
        for (int w = 0; w < 2 * (1 + S::kAtomsB); ++w) scales_to_tmem(sa + 4 * w, smem_desc(sf + w * 512, 16, 128, 0));
        commit2_leader(&sfull[st.s]);
      }
    }
  } else if constexpr (S::kMx) {
    // ---- scale bytes of the x rows. The warps take chunks of 512 elements (16
    // bytes a row, two stages) in turn; lane l holds rows l, l + 32, ... Words
    // land as [row % 32][row / 32 % 4] of a 512-byte atom, like the weights'
    // tiles. A chunk is requested before the previous one is stored.
    constexpr int kGb = S::kTN / 32;
    const int nb = a.K / LORA_MX_BLOCK;
    struct Chunk { uint4 b[kGb]; };
    uint32_t it = 0;
    int skip = warp - kScaleWarp;  // chunks of the other warps before this warp's next
    bool ok = true;
    for (uint32_t item = 0; item < n_items && ok; ++item, it += nkb) {
      const Info *ti = tile(item);
      if (ti == nullptr) break;
      const int n = ti->rows;
      int xr[kGb];
#pragma unroll
      for (int g = 0; g < kGb; ++g) xr[g] = ti->x[32 * g + lane];
      release(item);
      auto load = [&](Chunk &v, int kb) {
        if (kb >= nkb) return;
#pragma unroll
        for (int g = 0; g < kGb; ++g)
          if (32 * g < n) v.b[g] = __ldg(reinterpret_cast<const uint4 *>(a.x_scale + (int64_t)xr[g] * a.ld_xs + kb * 8));
      };
      Chunk now{}, then{};
      int kb0 = 2 * skip;
      load(now, kb0);
      for (; kb0 < nkb && ok; kb0 += 2 * S::kScaleWarps) {
        load(then, kb0 + 2 * S::kScaleWarps);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // the chunk's stages
          if (kb0 + h >= nkb) break;
          const uint32_t i = it + kb0 + h, s = i % S::kStages;
          if (!mbar_wait_warp(&empty[s], ((i / S::kStages) & 1) ^ 1, a.err, kErrProduct)) { ok = false; break; }
          unsigned char *sf = sm + s * S::kStageBytes + kBytesA + S::kBytesB + 2 * kMxTileBytes;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            // Scales past the row's blocks stand beside codes the loads filled with
            // zeros; any number will do, a NaN would not.
            const int left = nb - ((kb0 + h) * 8 + 4 * w);
            const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            auto word = [&](int g) {
              if (g >= kGb) return 0x7f7f7f7fu;
              const uint4 &v = now.b[g < kGb ? g : 0];
              const uint32_t u = h == 0 ? (w == 0 ? v.x : v.y) : (w == 0 ? v.z : v.w);
              return (u & keep) | (0x7f7f7f7fu & ~keep);
            };
#pragma unroll
            for (int b = 0; b < S::kAtomsB; ++b)
              *reinterpret_cast<uint4 *>(sf + (w * S::kAtomsB + b) * 512 + lane * 16) =
                  make_uint4(word(4 * b), word(4 * b + 1), word(4 * b + 2), word(4 * b + 3));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&rows[s]);
        }
        now = then;
      }
      skip = (kb0 - (nkb + 1) / 2 * 2) / 2;
    }
  }
  tc_before_sync();
  // No barrier of this CTA is signalled after this: the tensor core's arrivals
  // (empty, accf, fin; both CTAs' barriers) and the loads' have been waited for
  // in the CTA they go to, the threads' own ones come before their cluster barrier.
  cluster_sync();
  if (warp == 2) {
    tc_after_sync();
    tmem_free2(tmem, S::kTmemCols);
  }
}

// ------------------------------------------------------------------ host side

cudaError_t encode(CUtensorMap *m, const void *base, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                   const cuuint32_t *box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = enc(m, type, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Pairs of this kernel the device holds at once, looked up once a device.
template <class S, typename TY>
cudaError_t resident_pairs(int *out) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // zero: not looked up yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kDevices && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 2;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(out, moe_product_tc_kernel<S, TY>, &cfg);
  if (e != cudaSuccess) return e;
  *out = std::max(1, *out);
  if (dev < kDevices) known[dev].store(*out, std::memory_order_relaxed);
  return cudaSuccess;
}

template <class S, typename TY>
cudaError_t launch(const TcMaps &maps, const TcArgs &a, int num_tokens, cudaStream_t st) {
  cudaError_t e = set_max_dynamic_smem((const void *)moe_product_tc_kernel<S, TY>, S::kSmem);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  e = resident_pairs<S, TY>(&pairs);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)num_tokens / S::kTN + std::min(a.num_slots - 1, num_tokens)) * ((a.N + kPairA - 1) / kPairA);
  const unsigned grid = 2u * (unsigned)std::min<int64_t>(tiles, pairs);
  return launch_pdl(moe_product_tc_kernel<S, TY>, dim3(grid), dim3(S::kThreads), S::kSmem, st, 2u, maps, a);
}

template <class S>
cudaError_t launch(const TcMaps &maps, const TcArgs &a, int num_tokens, int y_dtype, cudaStream_t st) {
  return y_dtype == LORA_BF16 ? launch<S, __nv_bfloat16>(maps, a, num_tokens, st) : launch<S, float>(maps, a, num_tokens, st);
}

using NarrowBf16 = Shape<false, 64, 2, 10>;
using WideBf16 = Shape<false, 256, 2, 6>;
using NarrowMx = Shape<true, 64, 2, 9, 2>;
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
  cudaError_t e = encode(&maps.W, d.W, mx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         CU_TENSOR_MAP_SWIZZLE_128B, 3, wd, ws, wb);
  if (e != cudaSuccess) return e;
  if (mx) {
    const cuuint64_t sd[2] = {kMxTileBytes / 2, (cuuint64_t)d.num_experts * mx_tiles_out(d.d_out) * (mx_tiles_in(d.d_in) / 2)};
    const cuuint64_t ss[1] = {2 * kMxTileBytes};
    const cuuint32_t sb[2] = {kMxTileBytes / 2, 1};
    e = encode(&maps.W_scale, d.W_scale, CU_TENSOR_MAP_DATA_TYPE_UINT32, CU_TENSOR_MAP_SWIZZLE_NONE, 2, sd, ss, sb);
    if (e != cudaSuccess) return e;
  } else {
    maps.W_scale = maps.W;  // not used
  }
  TcArgs a;
  a.x = static_cast<const uint8_t *>(x);
  a.ldx = mx ? ldx / 2 : ldx * 2;
  a.x_scale = x_scale;
  a.ld_xs = ld_xs;
  a.ldy = ldy;
  a.y = y;
  a.work = mv.work;
  a.sorted_rows = mv.sorted_rows;
  a.err = const_cast<int32_t *>(mv.work) + WorkLists::kErrWord;
  a.num_slots = mv.num_slots;
  a.K = d.d_in;
  a.N = d.d_out;
  a.x_div = div;
  // Narrow tiles (more stages, less shared memory for rows) while an expert has
  // up to 48 pairs on average. w13 of 32 experts, 7168 by 4096, in bf16 (4-bit):
  // 16 pairs an expert 267 us narrow, 280 wide (79, 86); 48 pairs 285, 285 (86,
  // 89); 64 pairs 305, 287 (95, 90); 128 pairs 428, 314 (140, 104). Pairs of
  // other ranks' experts count as well, the host does not know better; that
  // costs at most the 5 % between the two at few pairs.
  const bool narrow = mv.num_tokens <= (int64_t)48 * (mv.num_slots - 1);
  if (mx) return narrow ? launch<NarrowMx>(maps, a, mv.num_tokens, y_dtype, st) : launch<WideMx>(maps, a, mv.num_tokens, y_dtype, st);
  return narrow ? launch<NarrowBf16>(maps, a, mv.num_tokens, y_dtype, st) : launch<WideBf16>(maps, a, mv.num_tokens, y_dtype, st);
}

}  // namespace ra
