// Attention of few rows on the tensor cores (bf16, heads of 64 and 128): the single tokens
// and short drafts of a decode step, whose time is that of reading the cache, and small
// batches, whose time is that of one pass from end to end.
//
// The keys take the MMA's long side and a unit's N = 16, 32 or 64 rows (token, query head)
// its short one, so that little is computed for rows that are not there, and shared memory
// goes to blocks in flight, 160 to 192 KB of an SM:
//   S^T = K Q^T     128 keys by N, in TMEM, a thread a key
//   P^T = 2^(c S^T - m)    to shared memory, a thread its key's N weights, each as a bf16 and
//                   the bf16 of what that leaves, so that it is off by 2^-16 at most and
//                   outputs are as good as fp32's (256 requests of up to 4000 keys, 32/8
//                   heads of 128: 319 us, 312 with one bf16, which over 100 thousand keys
//                   is off by 0.0020 of the outputs' norm, as much as their own rounding)
//   O^T += V^T P^T  128 elements of the head by N, in TMEM, a thread an element (a head of
//                   64 leaves the other 64 rows to whatever lies behind the block)
// The base m of a row is common to its keys. It need not be their largest score: fp32 and
// bf16 carry a common factor of 2^24 without loss. A unit begins with the score of its
// first key, and the base rises to the largest score so far where the threads agree (one
// barrier a block) that some weight exceeds 2^24. Sums stay with the keys' threads until a
// unit's end. (With the maximum over the keys at each unit's first block, and bases held
// within 2^8, three requests of 110 thousand keys took as long, one of 999 keys 0.8 us more.)
// Scores and products are issued by a warp each. Units of 16 rows leave room for two CTAs
// of an SM with three (heads of 64: six) blocks in flight each, so that one's waits and
// ends of units are the other's time (five requests of 21 thousand keys, 20 heads of 64:
// 123 us with one warp for all MMAs, 119 with two, 89 with two CTAs, 95 with the weights'
// second bf16; 232 requests of a few keys by 8 heads of 128 34, 34, 20 and 22 us).
#include "attn_tc.cuh"

namespace ra {
namespace {

constexpr int kKeys = 128;
constexpr int kScoreWarp = 4, kKWarp = 5, kVWarp = 6, kProductWarp = 7, kThreads = 256;
constexpr float kLazy = 24.f;     // log2 of the factor that a weight may exceed 1 by
constexpr float kLowest = -3e38f; // base of a row without a key so far
constexpr int kFlags = 8;         // units that the loads can be ahead of an epilogue, and more

template <int N_, int D_>
struct FewShape {
  static constexpr int N = N_, D = D_, kHalves = D / 64;
  static constexpr int kHalfBytes = kKeys * 128, kTileBytes = kHalves * kHalfBytes;  // a K or V block, 64 elements at a time
  // CTAs of an SM: two, with half of the blocks in flight each, where that leaves room for enough of them.
  static constexpr int kCtas = N == 16 ? 2 : 1;
  static constexpr uint32_t kK = N == 16 ? (D == 64 ? 3 : 2) : (D == 64 ? 6 : 3), kV = N == 16 ? (D == 64 ? 3 : 1) : D == 64 ? 5 : N == 64 ? 2 : 3;
  static constexpr uint32_t kQ = N == 64 || (N == 16 && D == 128) ? 1 : 2, kP = 1;
  static constexpr int kQHalf = N * 128, kQBytes = kHalves * kQHalf, kPPart = kKeys * N * 2, kPBytes = 2 * kPPart;
  static constexpr uint32_t kPLayout = N == 16 ? kSw32 : N == 32 ? kSw64 : kSw128;
  static constexpr int kKOff = 0, kVOff = kKOff + (int)kK * kTileBytes, kQOff = kVOff + (int)kV * kTileBytes;
  static constexpr int kPOff = kQOff + (int)kQ * kQBytes;
  static constexpr int kRowOff = kPOff + (int)kP * kPBytes;   // of each row: base, factor, keys, and where it goes
  static constexpr int kWarpOff = kRowOff + N * 20 + 16 - N * 20 % 16;  // a value of each row from each warp
  static constexpr int kBarOff = kWarpOff + 4 * N * 4;
  static constexpr int kBarriers = 2 * (int)kK + 2 * (int)kV + 2 * (int)kQ + 4 + 2 * (int)kP + 2;
  static constexpr int kWalkOff = kBarOff + (kBarriers * 8 + 16 + kFlags * 4 + 15) / 16 * 16;
  static constexpr int kEnd = kWalkOff + 32 * (kThreads / 32);
  static constexpr int kSmem = 1024 + (kEnd > kQOff + kHalfBytes ? kEnd : kQOff + kHalfBytes);  // what the MMA reads behind V, too
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "shared memory");
  static constexpr uint32_t kO = 2 * N, kTmemCols = N == 16 ? 64 : N == 32 ? 128 : 256;  // TMEM: two S, then O
};

struct FewMaps {
  CUtensorMap q;     // {D, heads, rows}, boxes of 64 x group x unit tokens
  CUtensorMap k, v;  // pages: {D, keys of a page, heads, pages}, boxes of 64 x keys x 1 x 1; packed rows: {D, heads, rows}, 64 x 1 x 128
};

// Barrier of the four softmax warps; the second one says whether any thread's p holds.
__device__ __forceinline__ void keys_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool keys_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"((uint32_t)p) : "memory");
  return r != 0;
}
// Over a warp's lanes, the maximum or the sum of each of N values: afterwards v[0] (v[0] and v[1] for N = 64) of lane i is
// that of value i / 2, i or 2 i (+ 1).
template <int N, bool MAX, int LEFT = N, int O = 16>
__device__ __forceinline__ void across_lanes(float (&v)[N], int lane) {
  constexpr int n = LEFT > 1 ? LEFT / 2 : 1;
  const bool upper = (lane & O) != 0;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const float send = LEFT > 1 && !upper ? v[i + LEFT - n] : v[i], keep = LEFT > 1 && upper ? v[i + LEFT - n] : v[i];
    const float got = __shfl_xor_sync(0xffffffffu, send, O);
    v[i] = MAX ? fmaxf(keep, got) : keep + got;
  }
  if constexpr (O > 1) across_lanes<N, MAX, n, O / 2>(v, lane);
}
template <int N>
__device__ __forceinline__ void store_across(float *to, const float (&v)[N], int lane) {
  if constexpr (N == 16) {
    if ((lane & 1) == 0) to[lane / 2] = v[0];
  } else if constexpr (N == 32) {
    to[lane] = v[0];
  } else {
    *reinterpret_cast<float2 *>(to + 2 * lane) = make_float2(v[0], v[1]);
  }
}

template <int N, int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, (FewShape<N, D>::kCtas)) attn_few_kernel(const __grid_constant__ FewMaps maps, const AttnArgs a) {
  using S = FewShape<N, D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = align1024(smem_raw);
  uint64_t *kfull = reinterpret_cast<uint64_t *>(sm + S::kBarOff);  // a K block is in
  uint64_t *kfree = kfull + S::kK;       // its scores are done
  uint64_t *vfull = kfree + S::kK;       // a V block is in
  uint64_t *vfree = vfull + S::kV;       // its product is done
  uint64_t *qfull = vfree + S::kV;       // a unit's Q is in
  uint64_t *qfree = qfull + S::kQ;       // its last scores are done
  uint64_t *sfull = qfree + S::kQ;       // a block's S^T is in TMEM
  uint64_t *sread = sfull + 2;           // it has been read
  uint64_t *pfull = sread + 2;           // a block's P^T is in shared memory
  uint64_t *pfree = pfull + S::kP;       // its product is done
  uint64_t *fin = pfree + S::kP;
  uint32_t *tslot = reinterpret_cast<uint32_t *>(fin + 2);
  volatile int32_t *flags = reinterpret_cast<int32_t *>(tslot + 1);  // [item % kFlags]: the last item with values taken out
  int64_t *to_row = reinterpret_cast<int64_t *>(sm + S::kRowOff);    // byte offsets of the rows in the output, -1 for none
  float *base = reinterpret_cast<float *>(to_row + N), *factor = base + N;
  int32_t *sees = reinterpret_cast<int32_t *>(factor + N);
  float *by_warp = reinterpret_cast<float *>(sm + S::kWarpOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < S::kK; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kfree[i], 1);
    }
    for (uint32_t i = 0; i < S::kV; ++i) {
      mbar_init(&vfull[i], 1);
      mbar_init(&vfree[i], 1);
    }
    for (uint32_t i = 0; i < S::kQ; ++i) {
      mbar_init(&qfull[i], 1);
      mbar_init(&qfree[i], 1);
    }
    for (uint32_t i = 0; i < S::kP; ++i) {
      mbar_init(&pfull[i], 4);
      mbar_init(&pfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sread[i], 4);
      mbar_init(&fin[i], 1);
    }
    for (int i = 0; i < kFlags; ++i) flags[i] = -1;
    fence_mbar_init();
  }
  if (warp == kScoreWarp) tmem_alloc(tslot, S::kTmemCols);
  if (warp == kKWarp && lane < 2) prefetch_map(lane == 0 ? &maps.k : &maps.q);
  if (warp == kVWarp && lane == 0) prefetch_map(&maps.v);
  // Rows of Q that no unit has: zeros, which raise no base.
  for (int i = threadIdx.x; i < (int)S::kQ * S::kQBytes / 16; i += kThreads)
    reinterpret_cast<uint4 *>(sm + S::kQOff)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  pdl_wait();
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  pdl_trigger();  // only now: a successor that takes TMEM must not start before this CTA has its own
  const uint32_t tmem = *tslot;
  Walk w(a, sm + S::kWalkOff + 32 * warp);
  Item it;

  if (warp == kScoreWarp) {
    // ---- scores
    constexpr uint32_t id_s = idesc_kk(kKeys, N);
    const uint64_t kd = smem_desc(smem_addr(sm + S::kKOff), 16, 1024, kSw128), qd = smem_desc(smem_addr(sm + S::kQOff), 16, 1024, kSw128);
    uint32_t g = 0, items = 0;  // blocks, and units with any, so far
    bool ok = true;
    while (ok && w.item(it)) {
      if (it.blocks == 0) continue;
      const uint32_t qs = items % S::kQ;
      if (!await(&qfull[qs], items / S::kQ & 1, a.err, kErrAttn)) break;
      ++items;
      for (int b = 0; b < it.blocks; ++b, ++g) {
        const uint32_t slot = g % S::kK;
        if (!(ok = await(&kfull[slot], g / S::kK & 1, a.err, kErrAttn) && await(&sread[g & 1], (g >> 1 & 1) ^ 1, a.err, kErrAttn))) break;
        tc_after_sync();
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h)
          mma_run<4>(tmem + (g & 1) * N, kd + slot * (S::kTileBytes >> 4) + h * (S::kHalfBytes >> 4),
                     qd + qs * (S::kQBytes >> 4) + h * (S::kQHalf >> 4), 2, 2, id_s, h > 0);
        mma_commit_elect(&sfull[g & 1]);
        mma_commit_elect(&kfree[slot]);
      }
      mma_commit_elect(&qfree[qs]);
    }
    mma_commit_elect(&fin[0]);
    await(&fin[0], 0, a.err, kErrAttn);  // every MMA is done before TMEM is freed
  } else if (warp == kKWarp || warp == kVWarp) {
    // ---- loads: one warp Q and K blocks, one V blocks
    const bool keys = warp == kKWarp;
    uint64_t *full = keys ? kfull : vfull, *free = keys ? kfree : vfree;
    const CUtensorMap *map = keys ? &maps.k : &maps.v;
    unsigned char *ring = sm + (keys ? S::kKOff : S::kVOff);
    const int half = lane % S::kHalves, part = lane / S::kHalves, ps = PAGED ? a.kv.page_size : kKeyBlock, rows = min(ps, kKeyBlock);
    const uint32_t n_slots = keys ? S::kK : S::kV;
    uint32_t slot = 0, phase = 0, items = 0;
    bool ok = true;
    while (ok && w.item(it)) {
      if (keys && it.blocks > 0) {
        const uint32_t qs = items % S::kQ;
        if (!await(&qfree[qs], (items / S::kQ & 1) ^ 1, a.err, kErrAttn)) break;
        ++items;
        if (lane == 0) mbar_arrive_tx(&qfull[qs], (uint32_t)(S::kHalves * a.s.unit_tokens * a.s.G * 128));
        __syncwarp();
        if (lane < S::kHalves)
          tma_load_3d(sm + S::kQOff + qs * S::kQBytes + lane * S::kQHalf, &maps.q, lane * 64, it.head * a.s.G, it.u.row0, &qfull[qs]);
      }
      const int32_t *table = a.kv.table + (int64_t)it.u.seq * a.kv.ld_table;
      auto page_at = [&](int b) {  // a lane a page of block b: its id, or one past the cache (which reads zeros)
        const int j = (it.u.kb0 + b) * kKeyBlock + part * rows;
        int page = 0;
        if (!PAGED) return page;
        if (b < it.blocks && part * rows < kKeyBlock && j < it.u.kv_len) {
          page = table[j >> a.kv.log2_page];
          if ((unsigned)page >= (unsigned)a.kv.num_pages) {
            atomicOr(a.err, kErrBadPage);
            page = a.kv.num_pages;
          }
        }
        return page;
      };
      int next = page_at(0);
      for (int b = 0; b < it.blocks; ++b) {
        const int page = next, j0 = (it.u.kb0 + b) * kKeyBlock;
        next = page_at(b + 1);
        const int copies = PAGED ? (min(kKeyBlock, it.u.kv_len - j0) + rows - 1) / rows * S::kHalves : S::kHalves;
        if (!await(&free[slot], phase ^ 1, a.err, kErrAttn)) { ok = false; break; }
        if (lane == 0) mbar_arrive_tx(&full[slot], (uint32_t)(copies * rows * 128));
        __syncwarp();
        if (lane < copies) {
          unsigned char *dst = ring + slot * S::kTileBytes + half * S::kHalfBytes + part * rows * 128;
          if constexpr (PAGED) tma_load_4d(dst, map, half * 64, (j0 + part * rows) & (ps - 1), it.head, page, &full[slot]);
          else tma_load_3d(dst, map, half * 64, it.head, it.u.row0 - it.u.pos0 + j0, &full[slot]);
        }
        if (++slot == n_slots) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == kProductWarp) {
    // ---- products, once the values that not every row sees have been looked at: rows behind the keys are zeroed up to the
    // last MMA's end
    constexpr uint32_t id_o = idesc_bf16(128, N) | (1u << 15);  // both operands as they lie
    // (With one half, the MMA's other 64 rows come from the next block or from Q, and go nowhere.)
    const uint64_t vd = smem_desc(smem_addr(sm + S::kVOff), S::kHalfBytes, 1024, kSw128);
    const uint64_t pd = smem_desc(smem_addr(sm + S::kPOff), 16, 16 * N, S::kPLayout);
    uint32_t g = 0;
    bool ok = true;
    while (ok && w.item(it)) {
      const int seen = common_keys(it.u, a.s.causal);
      for (int b = 0; b < it.blocks; ++b, ++g) {
        const uint32_t slot = g % S::kV, ps = g % S::kP;
        const int j0 = (it.u.kb0 + b) * kKeyBlock, keys = it.u.kv_len - j0;
        if (!(ok = await(&vfull[slot], g / S::kV & 1, a.err, kErrAttn))) break;
        if (j0 + kKeyBlock > seen) {
          if (fix_values<D>(sm + S::kVOff + slot * S::kTileBytes, S::kHalfBytes, max(0, seen - j0), min(kKeyBlock, keys), lane, 32))
            flags[w.index % kFlags] = (int)w.index;
          fence_async_smem();
          __syncwarp();
        }
        if (!(ok = await(&pfull[ps], g / S::kP & 1, a.err, kErrAttn))) break;
        tc_after_sync();
        const uint64_t vs = vd + slot * (S::kTileBytes >> 4), pp = pd + ps * (S::kPBytes >> 4);
        if (keys >= kKeys) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mma_run<4>(tmem + S::kO, vs, pp + i * (S::kPPart >> 4), 128, 2 * N, id_o, b > 0 || i > 0);
            mma_run<4>(tmem + S::kO, vs + 4 * 128, pp + i * (S::kPPart >> 4) + 8 * N, 128, 2 * N, id_o, 1);
          }
        } else {
#pragma unroll 1
          for (int s = 0; s * 16 < keys; ++s) {
            mma_run<1>(tmem + S::kO, vs + s * 128, pp + s * 2 * N, 0, 0, id_o, b > 0 || s > 0);
            mma_run<1>(tmem + S::kO, vs + s * 128, pp + (S::kPPart >> 4) + s * 2 * N, 0, 0, id_o, 1);
          }
        }
        mma_commit_elect(&pfree[ps]);
        mma_commit_elect(&vfree[slot]);
      }
      w.done(it);
    }
    mma_commit_elect(&fin[1]);
    await(&fin[1], 0, a.err, kErrAttn);
  } else {
    // ---- weights: a thread a key; and the outputs: a thread an element of the head
    const int tid = threadIdx.x;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const float c = a.s.scale_log2;
    const int swz = N == 16 ? (tid >> 2 & 1) : N == 32 ? (tid >> 1 & 3) : (tid & 7);
    uint32_t g = 0;
    bool ok = true;
    while (w.item(it)) {
      if (keys_any(!ok)) break;  // all four warps or none; the rows' values are free to be written
      const int rows = it.u.tokens * a.s.G, seen = common_keys(it.u, a.s.causal);
      if (tid < N) {
        const int tok = tid / a.s.G, head = it.head * a.s.G + tid % a.s.G;
        const bool live = tid < rows;
        sees[tid] = live ? visible_keys(it.u.pos0 + tok, it.u.kv_len, a.s.causal) : it.u.kv_len;
        to_row[tid] = !live ? -1
                      : it.u.slot >= 0
                          ? (((int64_t)it.u.slot * a.s.Hkv + it.head) * slot_floats(a.s) + (int64_t)tid * D) * 4
                          : (((int64_t)it.u.row0 + tok) * a.ldo + (int64_t)head * D) * 2;
        base[tid] = live ? kLowest : INFINITY;  // rows of Q behind the unit's, another sequence's: weights 0, and no rise for them
      }
      keys_sync();
      float l[N];
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.f;
      bool failed = false;
      for (int b = 0; b < it.blocks; ++b, ++g) {
        const int j = (it.u.kb0 + b) * kKeyBlock + tid;
        ok = await(&sfull[g & 1], g >> 1 & 1, a.err, kErrAttn) && ok;
        tc_after_sync();
        float s[N];
        if constexpr (N == 16) {
          tmem_ld16(lanes + (g & 1) * N, s);
        } else {
#pragma unroll
          for (int x = 0; x < N; x += 32) tmem_ld32_async(lanes + (g & 1) * N + x, s + x);
          tmem_wait_ld();
        }
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sread[g & 1]);
        if ((it.u.kb0 + b + 1) * kKeyBlock > seen) {
#pragma unroll
          for (int n = 0; n < N; ++n) s[n] = j < sees[n] ? s[n] : -INFINITY;
        }
        if (b == 0) {
          if (tid == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) base[n] = fmaxf(s[n] * c, base[n]);
          }
          keys_sync();
        }
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < N; ++n) top = fmaxf(top, fmaf(s[n], c, -base[n]));
        if (keys_any(!ok || top > kLazy)) {
          // Raise the rows' bases to their largest scores so far.
          if (keys_any(!ok)) { failed = true; break; }
          float v[N];
#pragma unroll
          for (int n = 0; n < N; ++n) v[n] = s[n] * c;
          across_lanes<N, true>(v, lane);
          store_across<N>(by_warp + warp * N, v, lane);
          keys_sync();
          if (tid < N) {
            const float m = fmaxf(fmaxf(fmaxf(by_warp[tid], by_warp[N + tid]), fmaxf(by_warp[2 * N + tid], by_warp[3 * N + tid])), base[tid]);
            factor[tid] = ex2(base[tid] - m);
            base[tid] = m;
          }
          keys_sync();
          if (b > 0) {  // the sums and O so far, whose last product has to be done
            ok = await(&pfree[(g - 1) % S::kP], (g - 1) / S::kP & 1, a.err, kErrAttn) && ok;
            tc_after_sync();
#pragma unroll
            for (int n = 0; n < N; ++n) l[n] *= factor[n];
#pragma unroll 1
            for (int x = 0; x < N; x += 16) {
              float o[16];
              tmem_ld16(lanes + S::kO + x, o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] *= factor[x + y];
              tmem_st16(lanes + S::kO + x, o);
            }
            tmem_wait_st();
          }
        }
        // The weights, in the order in which the MMA takes them: a key's N side by side.
        if (g >= S::kP) ok = await(&pfree[g % S::kP], (g / S::kP & 1) ^ 1, a.err, kErrAttn) && ok;
        unsigned char *row = sm + S::kPOff + (g % S::kP) * S::kPBytes + tid * (2 * N);
#pragma unroll
        for (int x = 0; x < N; x += 8) {
          uint32_t p[4], rest[4];
#pragma unroll
          for (int y = 0; y < 8; y += 2) {
            const float p0 = ex2(fmaf(s[x + y], c, -base[x + y])), p1 = ex2(fmaf(s[x + y + 1], c, -base[x + y + 1]));
            l[x + y] += p0;
            l[x + y + 1] += p1;
            const uint32_t both = pack_bf16(p0, p1);
            p[y / 2] = both;
            rest[y / 2] = pack_bf16(p0 - __uint_as_float(both << 16), p1 - __uint_as_float(both & 0xffff0000u));
          }
          uint4 *to = reinterpret_cast<uint4 *>(row + ((x / 8) ^ swz) * 16);
          to[0] = make_uint4(p[0], p[1], p[2], p[3]);
          to[S::kPPart / 16] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
        }
        fence_async_smem();
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[g % S::kP]);
      }
      if (failed) break;
      // ---- the end of the unit
      across_lanes<N, false>(l, lane);
      store_across<N>(by_warp + warp * N, l, lane);
      keys_sync();
      const bool split = it.u.slot >= 0, some = it.blocks > 0;
      if (tid < N) {
        const float sum = by_warp[tid] + by_warp[N + tid] + by_warp[2 * N + tid] + by_warp[3 * N + tid];
        const float m = base[tid] == kLowest ? -INFINITY : base[tid];
        factor[tid] = split ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        if (to_row[tid] >= 0) {
          if (split)
            *reinterpret_cast<float2 *>(a.ws + ((int64_t)it.u.slot * a.s.Hkv + it.head) * slot_floats(a.s) +
                                        (int64_t)a.s.slot_rows * D + 2 * tid) = make_float2(m, sum);
          else if (a.lse != nullptr)
            a.lse[((int64_t)it.u.row0 + tid / a.s.G) * a.s.Hq + it.head * a.s.G + tid % a.s.G] =
                sum == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(sum));
        }
      }
      if (some) ok = await(&pfree[(g - 1) % S::kP], (g - 1) / S::kP & 1, a.err, kErrAttn) && ok;
      keys_sync();
      tc_after_sync();
      unsigned char *to = split ? reinterpret_cast<unsigned char *>(a.ws) + tid * 4 : static_cast<unsigned char *>(a.out) + tid * 2;
#pragma unroll 1
      for (int x = 0; x < N && x < rows; x += 16) {
        float o[16];
        tmem_ld16(lanes + S::kO + x, o);
#pragma unroll
        for (int y = 0; y < 16; ++y) {
          const int64_t at = to_row[x + y];
          const float v = some ? o[y] * factor[x + y] : 0.f;
          if (at < 0 || tid >= D) continue;
          if (split) *reinterpret_cast<float *>(to + at) = v;
          else *reinterpret_cast<__nv_bfloat16 *>(to + at) = __float2bfloat16_rn(v);
        }
      }
      tc_before_sync();
      if (some && flags[w.index % kFlags] == (int)w.index) {
        // Values that were taken out, for the rows that see them.
        for (int n = 0; n < rows && tid < D; ++n) {
          const float sum = taken_out(a, it.u, it.head, tid, seen, sees[n]);
          if (sum == 0.f) continue;
          if (split) {
            *reinterpret_cast<float *>(to + to_row[n]) += sum;
          } else {
            __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(to + to_row[n]);
            *p = __float2bfloat16_rn(__bfloat162float(*p) + sum);
          }
        }
      }
      w.done(it);
    }
  }
  tc_before_sync();
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_after_sync();
    tmem_free(tmem, S::kTmemCols);
  }
}

template <int N, int D, bool PAGED>
cudaError_t launch(const AttnArgs &a, cudaStream_t st) {
  FewMaps maps;
  cudaError_t e = encode_rows(&maps.q, a.q, D, a.s.Hq, D, a.num_tokens, a.ldq, a.s.G, a.s.unit_tokens);
  if (PAGED) {
    if (e == cudaSuccess) e = encode_pages(&maps.k, a.kv.k, a, a.kv.k_row, a.kv.k_head, a.kv.k_page);
    if (e == cudaSuccess) e = encode_pages(&maps.v, a.kv.v, a, a.kv.v_row, a.kv.v_head, a.kv.v_page);
  } else {
    if (e == cudaSuccess) e = encode_rows(&maps.k, a.kv.k, D, a.s.Hkv, a.kv.k_head, a.num_tokens, a.kv.k_row, 1, kKeys);
    if (e == cudaSuccess) e = encode_rows(&maps.v, a.kv.v, D, a.s.Hkv, a.kv.v_head, a.num_tokens, a.kv.v_row, 1, kKeys);
  }
  if (e == cudaSuccess) e = set_max_dynamic_smem((const void *)attn_few_kernel<N, D, PAGED>, FewShape<N, D>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)a.p.max_units * a.s.Hkv;
  return launch_pdl(attn_few_kernel<N, D, PAGED>, dim3((unsigned)std::min<int64_t>(most, a.s.ctas)), dim3(kThreads),
                    FewShape<N, D>::kSmem, st, 1u, maps, a);
}

template <int D, bool PAGED>
cudaError_t launch(const AttnArgs &a, cudaStream_t st) {
  if (a.s.few == 16) return launch<16, D, PAGED>(a, st);
  if (a.s.few == 32) return launch<32, D, PAGED>(a, st);
  return launch<64, D, PAGED>(a, st);
}

}  // namespace

cudaError_t launch_attn_few(const AttnArgs &a, cudaStream_t st) {
  const bool paged = a.kv.page_size > 0;
  if (a.s.D == 128) return paged ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return paged ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace ra
