// Attention on the tensor cores (bf16, heads of 64 and 128).
//
// Rows of a tile are 128 (token, query head) pairs of one key-value head, so that a
// group of heads shares each key and value that is loaded. A CTA works on two streams of
// (tile, 128 keys) steps at once, each with a softmax warpgroup and a warp that issues its
// MMAs, so that the tensor core multiplies for one stream while the other takes its
// exponentials:
//   S = Q K^T    both operands in shared memory, S in TMEM (fp32)
//   P = 2^(c S - m)    a thread a row, S from TMEM, P back over S as bf16
//   O += P V     P from TMEM, V from shared memory as it lies there; in two halves of the
//                keys, the first while the second's exponentials are taken
// A unit of two tiles gives one to each stream; a unit of one tile deals its blocks of keys
// out to both, and their results are added up. A stream's next scores are issued right
// behind the product that reads its P (MMAs of one thread run in order), over units' ends
// as well. (One warp that issued both streams' MMAs spent 1750 clocks a step on them and on
// its waits, of which the MMAs take 1024.) What bounds it is a block's chain of scores,
// exponentials, weights and product: a pair of blocks takes 3450 clocks, 2048 of them the
// MMAs', and a unit's begin and end 12000 (32 query and 8 key-value heads of 128: 16381
// tokens 1510 to 1545 us, 1.42 to 1.45 PFLOP/s; 16 prompts of 128 to 2048 296 us).
//
// The running maximum of a row rises only when a block exceeds it by more than 2^8 (all
// weights carry the same factor, fp32 and bf16 have the range for it), so that O is
// rescaled in few steps. S of a step is complete only once every MMA that its warp issued
// before is, the last product with V among them: O can be rescaled without a wait.
//
// Values that some row of a unit does not see (behind the keys, of later tokens) are
// looked at by warps of their own before the MMA, since 0 * NaN is NaN: rows behind
// the keys are zeroed, and where a later token's value is not finite it is taken out and
// added to the rows that see it at the end.
#include "attn_tc.cuh"

namespace ra {
namespace {

constexpr int kRows = 128;      // rows of a tile
// Warps: 0-3 and 4-7 the streams' softmax, then their MMAs, the loads, the values that not every row sees.
constexpr int kMmaWarp = 8, kKWarp = 10, kVWarp = 11, kFixWarp = 12, kFixWarps = 4;
constexpr int kThreads = 32 * (kFixWarp + kFixWarps);
// Registers: the softmax warps hold a row of S. 8 * 200 + 8 * 56 = 16 * 128, the launch's own.
constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;
constexpr float kLazy = 8.f;    // log2 of the factor that a weight may exceed 1 by
constexpr int kFlags = 8;       // units that the loads can be ahead of an epilogue, and more

template <int D_>
struct TcShape {
  static constexpr int D = D_, kHalves = D / 64;
  static constexpr int kHalfBytes = kRows * 128;              // 128 rows of 64 elements
  static constexpr int kTileBytes = kHalves * kHalfBytes;     // Q tile, K or V block
  // K and V blocks in flight. Even, so that where the streams take blocks in turn each has
  // slots of its own.
  static constexpr uint32_t kK = D == 128 ? 2 : 4, kV = D == 128 ? 2 : 4;
  static constexpr int kKOff = 2 * kTileBytes, kVOff = kKOff + (int)kK * kTileBytes;
  static constexpr int kTurnOff = kVOff + (int)kV * kTileBytes;   // a softmax warp's 32 rows of 128 bytes on their way out
  static constexpr int kTurnBytes = 32 * 128;
  static constexpr int kStatOff = kTurnOff + 8 * kTurnBytes;  // {m, l} of a merged stream's rows
  static constexpr int kBarOff = kStatOff + kRows * 8;
  static constexpr int kBarriers = 2 * (int)kK + 3 * (int)kV + 18;
  static constexpr int kWalkOff = kBarOff + (kBarriers * 8 + 16 + kFlags * 4 + 8 + 15) / 16 * 16;
  static constexpr int kSmem = 1024 + kWalkOff + 32 * (kThreads / 32 + 2);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // TMEM columns: two streams' S (and P over it), two streams' O.
  static constexpr uint32_t kS = 0, kO = 256, kTmemCols = 512;
};

struct TcMaps {
  CUtensorMap q;     // {D, heads, rows}, boxes of 64 x group x tile tokens
  CUtensorMap k, v;  // packed rows: {D, heads, rows}, boxes of 64 x 1 x 128; pages: {D, keys of a page, heads, pages}, 64 x keys x 1 x 1
};

// ------------------------------------------------------------------ kernel

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ TcMaps maps, const AttnArgs a) {
  using S = TcShape<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = align1024(smem_raw);
  uint64_t *kfull = reinterpret_cast<uint64_t *>(sm + S::kBarOff);  // a K block is in
  uint64_t *kfree = kfull + S::kK;       // both streams' MMAs on it are done
  uint64_t *vfull = kfree + S::kK;       // a V block is in
  uint64_t *vfree = vfull + S::kV;       // both streams' MMAs on it are done
  uint64_t *fixed = vfree + S::kV;       // it has been looked at
  uint64_t *qfull = fixed + S::kV;       // a stream's Q tile is in
  uint64_t *qfree = qfull + 2;           // its last scores are done
  uint64_t *sfull = qfree + 2;           // S of a stream's step is in TMEM
  uint64_t *pfull = sfull + 2;           // [stream][half]: P of it is
  uint64_t *ofull = pfull + 4;           // a stream's last product with V is done
  uint64_t *fin = ofull + 2;             // [stream]
  uint64_t *go = fin + 2;                // [stream]: its turn to issue a step's MMAs
  uint64_t *mfull = go + 2;              // the statistics of the stream to merge are in shared memory
  uint64_t *mfree = mfull + 1;           // its O has been read
  uint32_t *tslot = reinterpret_cast<uint32_t *>(mfree + 1);
  volatile int32_t *flags = reinterpret_cast<int32_t *>(tslot + 1);  // [item % kFlags]: the last item with values taken out
  volatile uint32_t *reached = const_cast<volatile uint32_t *>(reinterpret_cast<volatile uint32_t *>(flags + kFlags));
  float2 *stats = reinterpret_cast<float2 *>(sm + S::kStatOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (uint32_t i = 0; i < S::kK; ++i) {
      mbar_init(&kfull[i], 1);
      mbar_init(&kfree[i], 2);
    }
    for (uint32_t i = 0; i < S::kV; ++i) {
      mbar_init(&vfull[i], 1);
      mbar_init(&vfree[i], 2);
      mbar_init(&fixed[i], kFixWarps);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&qfull[t], 1);
      mbar_init(&qfree[t], 1);
      mbar_init(&sfull[t], 1);
      mbar_init(&pfull[2 * t], 4);
      mbar_init(&pfull[2 * t + 1], 4);
      mbar_init(&ofull[t], 1);
      mbar_init(&fin[t], 1);
      mbar_init(&go[t], 1);
    }
    mbar_init(mfull, 4);
    mbar_init(mfree, 4);
    for (int i = 0; i < kFlags; ++i) flags[i] = -1;
    reached[0] = reached[1] = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc(tslot, S::kTmemCols);
  if (warp == kKWarp && lane < 2) prefetch_map(lane == 0 ? &maps.k : &maps.q);
  if (warp == kVWarp && lane == 0) prefetch_map(&maps.v);
  pdl_wait();
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  pdl_trigger();  // only now: a successor that takes TMEM must not start before this CTA has its own
  const uint32_t tmem = *tslot;
  Walk w(a, sm + S::kWalkOff + 32 * warp);
  Item it;

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kKWarp) {
      // ---- MMAs of stream t
      constexpr uint32_t id_s = idesc_kk(kRows, kKeyBlock), id_o = idesc_bf16(kRows, D);
      const int t = warp - kMmaWarp;
      const uint32_t ts = tmem + S::kS + t * 128, to = tmem + S::kO + t * 128;
      const uint64_t qd = smem_desc(smem_addr(sm + t * S::kTileBytes), 16, 1024, kSw128);
      const uint64_t kd = smem_desc(smem_addr(sm + S::kKOff), 16, 1024, kSw128);
      const uint64_t vd = smem_desc(smem_addr(sm + S::kVOff), S::kHalfBytes, 1024, kSw128);
      Walk ws(a, sm + S::kWalkOff + kThreads + 32 * t);  // of the scores, a step ahead
      Item is{};
      int sb = 0;          // their next block in the item
      uint32_t items = 0, steps = 0, turns = t == 0 ? 1 : 0;
      uint64_t *kfree_next = kfree;
      uint32_t own = ~0u;  // slots whose last K block this stream has used (or none has been in)
      bool more = ws.item(is);
      if (more) sb = ws.first(is, t);
      // The next step's scores, in two parts so that nothing but MMAs stands between a step's products: its operands, and
      // its MMAs.
      uint64_t kd_next = 0;
      auto operands = [&]() -> bool {
        while (more && sb >= is.blocks) {
          if (ws.first(is, t ^ 1) < is.blocks && !is.pair) own &= t == 0 ? 0x55555555u : 0xaaaaaaaau;
          ws.done(is);
          more = ws.item(is);
          if (more) sb = ws.first(is, t);
        }
        const uint32_t pos = more ? ws.pos + sb : ~0u, slot = pos % S::kK;
        if (lane == 0) reached[t] = pos;  // every K block of this stream before it has been in
        if (!more) return true;
        // A barrier's phases are told apart by their parity only. Where the slot's last block was the other stream's alone,
        // that one has to have been in before this stream may wait for the next.
        if ((own >> slot & 1) == 0 && pos >= S::kK &&
            !__all_sync(0xffffffffu, past(&reached[t ^ 1], pos - S::kK, a.err, kErrAttn)))
          return false;
        own |= 1u << slot;
        if (sb < ws.step(is) && !await(&qfull[t], items++ & 1, a.err, kErrAttn)) return false;
        if (!await(&kfull[slot], pos / S::kK & 1, a.err, kErrAttn)) return false;
        kd_next = kd + slot * (S::kTileBytes >> 4);
        kfree_next = &kfree[slot];
        return true;
      };
      auto scores = [&]() {
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h)
          mma_run<4>(ts, qd + h * (S::kHalfBytes >> 4), kd_next + h * (S::kHalfBytes >> 4), 2, 2, id_s, h > 0);
        mma_commit_elect(&sfull[t]);
      };
      auto scores_done = [&]() {  // behind scores(): what its end releases
        mma_commit_elect(kfree_next);
        if (!is.pair) mma_commit_elect(kfree_next);  // for the other stream
        sb += ws.step(is);
        if (sb >= is.blocks) mma_commit_elect(&qfree[t]);
      };
      bool ok = operands();
      tc_after_sync();
      if (ok && more) {
        scores();
        scores_done();
      }
      while (ok && w.item(it)) {
        const int d = w.step(it), b0 = w.first(it, t);
        for (int b = b0; b < it.blocks; b += d, ++steps) {
          const uint32_t pos = w.pos + b, slot = pos % S::kV;
          const uint64_t vd_now = vd + slot * (S::kTileBytes >> 4);
          if (!(ok = operands() && await(&fixed[slot], pos / S::kV & 1, a.err, kErrAttn) &&
                     await(&pfull[2 * t], steps & 1, a.err, kErrAttn)))
            break;
          // Streams of two tiles take turns: left alone they fall into step, and the tensor core idles while both take
          // exponentials.
          if (it.pair && !await(&go[t], turns++ & 1, a.err, kErrAttn)) { ok = false; break; }
          tc_after_sync();
          mma_pv4(to, ts, vd_now, 128, id_o, b != b0);  // 64 keys
          if (!await(&pfull[2 * t + 1], steps & 1, a.err, kErrAttn)) { ok = false; break; }
          tc_after_sync();
          mma_pv4(to, ts + 32, vd_now + (64 * 128 >> 4), 128, id_o, 1);
          if (b + d >= it.blocks) mma_commit_elect(&ofull[t]);
          if (more) scores();
          if (it.pair && lane == 0) mbar_arrive(&go[t ^ 1]);
          mma_commit_elect(&vfree[slot]);
          if (!it.pair) mma_commit_elect(&vfree[slot]);
          if (more) scores_done();
        }
        w.done(it);
      }
      mma_commit_elect(&fin[t]);
      await(&fin[t], 0, a.err, kErrAttn);  // every MMA is done before TMEM is freed
    } else if (warp < kFixWarp) {
      // ---- loads: one warp K blocks and Q tiles, one V blocks
      const bool keys = warp == kKWarp;
      const uint32_t n_slots = keys ? S::kK : S::kV;
      uint64_t *full = keys ? kfull : vfull, *free = keys ? kfree : vfree;
      const CUtensorMap *map = keys ? &maps.k : &maps.v;
      unsigned char *ring = sm + (keys ? S::kKOff : S::kVOff);
      const int half = lane % S::kHalves, part = lane / S::kHalves;
      uint32_t slot = 0, phase = 0, used0 = 0, used1 = 0;
      bool ok = true, alone = false;  // alone: the unit before had one tile
      while (ok && w.item(it)) {
        for (int b = 0; b < it.blocks; ++b) {
          const int j0 = (it.u.kb0 + b) * kKeyBlock;
          int page = 0, copies = S::kHalves, in_page = 0, rows = kKeyBlock;  // copies of a block, rows of each
          if constexpr (PAGED) {
            // A lane a page: its id, or one past the cache (which reads zeros).
            const int ps = a.kv.page_size;
            rows = min(ps, kKeyBlock);
            copies = (min(kKeyBlock, it.u.kv_len - j0) + rows - 1) / rows * S::kHalves;
            const int j = j0 + part * rows;
            in_page = j & (ps - 1);
            if (lane < copies) {
              page = a.kv.table[(int64_t)it.u.seq * a.kv.ld_table + (j >> a.kv.log2_page)];
              if ((unsigned)page >= (unsigned)a.kv.num_pages) {
                atomicOr(a.err, kErrBadPage);
                page = a.kv.num_pages;
              }
            }
          }
          if (!await(&free[slot], phase ^ 1, a.err, kErrAttn)) { ok = false; break; }
          if (lane == 0) mbar_arrive_tx(&full[slot], (uint32_t)(copies * rows * 128));
          __syncwarp();
          unsigned char *dst = ring + slot * S::kTileBytes + half * S::kHalfBytes;
          if (lane < copies) {
            if constexpr (PAGED) tma_load_4d(dst + part * rows * 128, map, half * 64, in_page, it.head, page, &full[slot]);
            else tma_load_3d(dst, map, half * 64, it.head, it.u.row0 - it.u.pos0 + j0, &full[slot]);
          }
          if (++slot == n_slots) {
            slot = 0;
            phase ^= 1;
          }
          if (!keys || b != (alone ? 0 : min(1, it.blocks - 1))) continue;
          // Q tiles, behind the first two K blocks, which need not wait for the previous unit's last scores: a
          // stream's own where there are two, the same for both where there is one. Behind a unit of one tile only behind
          // the first: the second may have to wait for a stream that waits for its turn, which the other gives it
          // once its next unit's Q is in.
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t &used = t == 0 ? used0 : used1;
            if (!ok || w.first(it, t) >= it.blocks) continue;
            if (!await(&qfree[t], (used & 1) ^ 1, a.err, kErrAttn)) { ok = false; continue; }
            ++used;
            if (lane == 0) mbar_arrive_tx(&qfull[t], (uint32_t)(S::kHalves * a.s.tile_tokens * a.s.G * 128));
            __syncwarp();
            if (lane < S::kHalves)
              tma_load_3d(sm + t * S::kTileBytes + lane * S::kHalfBytes, &maps.q, lane * 64, it.head * a.s.G,
                          it.u.row0 + (it.pair ? t * a.s.tile_tokens : 0), &qfull[t]);
          }
          if (!ok) break;
        }
        alone = !it.pair;
        w.done(it);
      }
    } else {
      // ---- values that not every row sees: each warp looks at every kFixWarps-th group of 32 chunks of 16 bytes
      constexpr int kChunks = D / 8;  // of a row
      const int me = (warp - kFixWarp) * 32 + lane;
      uint32_t slot = 0, phase = 0;
      bool ok = true;
      while (ok && w.item(it)) {
        const int seen = common_keys(it.u, a.s.causal);
        for (int b = 0; b < it.blocks; ++b) {
          const int j0 = (it.u.kb0 + b) * kKeyBlock;
          if (!await(&vfull[slot], phase, a.err, kErrAttn)) { ok = false; break; }
          if (j0 + kKeyBlock > seen) {
            unsigned char *base = sm + S::kVOff + slot * S::kTileBytes;
            auto chunk = [&](int i) {
              const int r = i / kChunks, c = i % kChunks;
              return reinterpret_cast<uint4 *>(base + (c / 8) * S::kHalfBytes + swz128(r, c % 8));
            };
            const int i0 = max(0, seen - j0) * kChunks, i1 = min(kKeyBlock, it.u.kv_len - j0) * kChunks;  // looked at; zeroed from i1 on
            uint32_t any = 0;  // an exponent of all ones, plus one, carries into its sign
#pragma unroll 4
            for (int i = i0 + me; i < i1; i += 32 * kFixWarps) {
              const uint4 x = *chunk(i);
              any |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                     ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
            }
            if (any & 0x80008000u) {
              flags[w.index % kFlags] = (int)w.index;
              for (int i = i0 + me; i < i1; i += 32 * kFixWarps) {
                const uint4 x = *chunk(i);
                uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((q[e] & 0x7f80u) == 0x7f80u) q[e] &= 0xffff0000u;
                  if ((q[e] & 0x7f800000u) == 0x7f800000u) q[e] &= 0xffffu;
                }
                *chunk(i) = make_uint4(q[0], q[1], q[2], q[3]);
              }
            }
            for (int i = i1 + me; i < kKeyBlock * kChunks; i += 32 * kFixWarps) *chunk(i) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&fixed[slot]);
          if (++slot == S::kV) {
            slot = 0;
            phase ^= 1;
          }
        }
        w.done(it);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---- softmax of stream t, a thread a row
    const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + S::kS + t * 128, to = tmem + lanes + S::kO + t * 128;
    const uint32_t to_other = tmem + lanes + S::kO + (t ^ 1) * 128;
    unsigned char *turn = sm + S::kTurnOff + warp * S::kTurnBytes;
    const float c = a.s.scale_log2;
    const int tile_rows = a.s.tile_tokens * a.s.G, row_tok = r / a.s.G, row_head = r % a.s.G;
    uint32_t steps = 0, mine_used = 0, other_used = 0, merges = 0;
    bool ok = true;
    while (ok && w.item(it)) {
      const int d = w.step(it), b0 = w.first(it, t);
      const bool mine = b0 < it.blocks, other = w.first(it, t ^ 1) < it.blocks;
      const bool writes = it.pair || b0 == 0;  // the stream whose warpgroup stores the rows
      // The row: its token, and the keys it sees.
      const int tile = it.pair ? t : 0, tok = tile * a.s.tile_tokens + row_tok;
      const bool live = r < tile_rows && tok < it.u.tokens;
      const bool busy = __any_sync(0xffffffffu, live);
      const int lim = live ? visible_keys(it.u.pos0 + tok, it.u.kv_len, a.s.causal) : INT32_MAX / 2;
      float m = -INFINITY, l = 0.f;  // of c * s
      for (int b = b0; b < it.blocks; b += d, ++steps) {
        if (!await(&sfull[t], steps & 1, a.err, kErrAttn)) { ok = false; break; }
        if (!busy) {
          if (lane < 2) mbar_arrive(&pfull[2 * t + lane]);
          continue;
        }
        tc_after_sync();
        float s[128];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32_async(ts + 32 * x, s + 32 * x);
        tmem_wait_ld();
        const int sees = lim - (it.u.kb0 + b) * kKeyBlock;
        if (__any_sync(0xffffffffu, sees < kKeyBlock)) {
#pragma unroll
          for (int x = 0; x < 128; ++x) s[x] = x < sees ? s[x] : -INFINITY;
        }
        float top[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) top[x] = max3(s[x], s[x + 4], s[x + 8]);
#pragma unroll
        for (int x = 12; x < 124; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y) top[y] = max3(top[y], s[x + y], s[x + y + 4]);
        const float mn = max3(max3(top[0], top[1], s[124]), max3(top[2], top[3], s[125]), fmaxf(s[126], s[127])) * c;
        const bool rise = mn > m + kLazy;
        if (__any_sync(0xffffffffu, rise)) {
          const float up = rise ? ex2(m - mn) : 1.f;
          if (rise) m = mn;
          l *= up;
          if (b != b0) {
#pragma unroll 1
            for (int x = 0; x < D; x += 16) {
              float o[16];
              tmem_ld16(to + x, o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] *= up;
              tmem_st16(to + x, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weights = [&](int x0) {  // 32 of the row's weights, to where the MMA takes them from
          uint32_t p[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float2 e = fma2(make_float2(s[x0 + 2 * x], s[x0 + 2 * x + 1]), c2, b2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[x & 1] = add2(sum[x & 1], e);
            p[x] = pack_bf16(e.x, e.y);
          }
          tmem_st16u(ts + x0 / 2, p);
        };
        auto ready = [&](int h) {
          tmem_wait_st();
          tc_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[2 * t + h]);
        };
        weights(0);
        weights(32);
        ready(0);
        weights(64);
        weights(96);
        ready(1);
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
      }
      if (!ok) break;
      // ---- the end of the unit
      const bool merge = !it.pair && other && mine;
      if (!writes) {
        mine_used += mine;
        other_used += other;
        if (merge) {
          stats[r] = make_float2(m, l);
          __syncwarp();
          if (lane == 0) mbar_arrive(mfull);
          if (!await(mfree, merges & 1, a.err, kErrAttn)) { ok = false; break; }
          ++merges;
        }
        w.done(it);
        continue;
      }
      if (mine && !await(&ofull[t], mine_used & 1, a.err, kErrAttn)) { ok = false; break; }
      mine_used += mine;
      float w0 = 1.f, w1 = 0.f;  // weights of this stream's and the other's O
      if (merge) {
        // First the statistics: behind them the other stream has seen its last product of every unit before, so that the parity
        // of its products' barrier stands for this unit's.
        if (!await(mfull, merges & 1, a.err, kErrAttn) || !await(&ofull[t ^ 1], other_used & 1, a.err, kErrAttn)) { ok = false; break; }
        ++merges;
        const float2 o = stats[r];
        const float mm = fmaxf(m, o.x), base = mm == -INFINITY ? 0.f : mm;
        w0 = ex2(m - base);
        w1 = ex2(o.x - base);
        l = l * w0 + o.y * w1;
        m = mm;
      }
      other_used += other;
      tc_after_sync();
      if (busy) {
        const int64_t row = (int64_t)it.u.row0 + tok;
        const int head = it.head * a.s.G + row_head;
        const bool split = it.u.slot >= 0;
        const float inv = split ? 1.f : l == 0.f ? 0.f : 1.f / l;
        w0 *= inv;
        w1 *= inv;
        const bool taken = mine && live && flags[w.index % kFlags] == (int)w.index;
        // The row's address (nothing there for rows that are none), and what a warp turns round at a time: 128 bytes a row.
        unsigned char *dst = nullptr;
        if (live && split) {
          float *part = a.ws + ((int64_t)it.u.slot * a.s.Hkv + it.head) * slot_floats(a.s);
          const int unit_row = tile * tile_rows + r;
          dst = reinterpret_cast<unsigned char *>(part + (int64_t)unit_row * D);
          *reinterpret_cast<float2 *>(part + (int64_t)a.s.slot_rows * D + 2 * unit_row) = make_float2(m, l);
        } else if (live) {
          dst = reinterpret_cast<unsigned char *>(static_cast<__nv_bfloat16 *>(a.out) + row * a.ldo + (int64_t)head * D);
          if (a.lse != nullptr) a.lse[row * a.s.Hq + head] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
        }
        const uint64_t mine_at = reinterpret_cast<uint64_t>(dst);
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
          float o[32];
          if (mine) {
            tmem_ld32_async(to + x, o);
            tmem_wait_ld();
          }
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = mine ? o[y] * w0 : 0.f;
          if (merge) {
            float o1[32];
            tmem_ld32_async(to_other + x, o1);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = fmaf(o1[y], w1, o[y]);
          }
          if (taken) {
            // Values that were taken out, for the rows that see them.
            const int end = min(lim, it.u.kb1 * kKeyBlock);
            for (int j = max(common_keys(it.u, a.s.causal), it.u.kb0 * kKeyBlock); j < end; ++j) {
              int64_t at = -1;
              if constexpr (PAGED) {
                const int page = a.kv.table[(int64_t)it.u.seq * a.kv.ld_table + (j >> a.kv.log2_page)];
                if ((unsigned)page < (unsigned)a.kv.num_pages) at = page * a.kv.v_page + (j & (a.kv.page_size - 1)) * a.kv.v_row;
              } else {
                at = ((int64_t)it.u.row0 - it.u.pos0 + j) * a.kv.v_row;
              }
              if (at < 0) continue;
              const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.kv.v) + at + it.head * a.kv.v_head + x;
#pragma unroll
              for (int y = 0; y < 32; ++y) {
                const float f = __bfloat162float(v[y]);
                if (!isfinite(f)) o[y] += f;
              }
            }
          }
          // To shared memory, 16-byte chunks rotated by the row, and out in whole 128-byte pieces of four rows: after each
          // 32 columns of partial results, after each 64 of a result.
          auto put = [&](int chunk, uint4 v) { *reinterpret_cast<uint4 *>(turn + lane * 128 + ((chunk ^ lane) & 7) * 16) = v; };
          if (split) {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              put(y, make_uint4(__float_as_uint(o[4 * y]), __float_as_uint(o[4 * y + 1]), __float_as_uint(o[4 * y + 2]),
                                __float_as_uint(o[4 * y + 3])));
          } else {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              put((x >> 5 & 1) * 4 + y, make_uint4(pack_bf16(o[8 * y], o[8 * y + 1]), pack_bf16(o[8 * y + 2], o[8 * y + 3]),
                                                   pack_bf16(o[8 * y + 4], o[8 * y + 5]), pack_bf16(o[8 * y + 6], o[8 * y + 7])));
            if ((x & 32) == 0) continue;
          }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int rr = 4 * y + lane / 8, cc = lane & 7;
            const uint64_t at = __shfl_sync(0xffffffffu, mine_at, rr);
            const uint4 v = *reinterpret_cast<const uint4 *>(turn + rr * 128 + ((cc ^ rr) & 7) * 16);
            if (at != 0) *reinterpret_cast<uint4 *>(at + (split ? x * 4 : (x & ~63) * 2) + cc * 16) = v;
          }
          __syncwarp();
        }
      }
      tc_before_sync();
      if (merge) {
        __syncwarp();
        if (lane == 0) mbar_arrive(mfree);
      }
      w.done(it);
    }
  }
  tc_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_after_sync();
    tmem_free(tmem, S::kTmemCols);
  }
}

// ------------------------------------------------------------------ host side

template <int D, bool PAGED>
cudaError_t launch(const AttnArgs &a, cudaStream_t st) {
  TcMaps maps;
  cudaError_t e = encode_rows(&maps.q, a.q, D, a.s.Hq, D, a.num_tokens, a.ldq, a.s.G, a.s.tile_tokens);
  if (PAGED) {
    if (e == cudaSuccess) e = encode_pages(&maps.k, a.kv.k, a, a.kv.k_row, a.kv.k_head, a.kv.k_page);
    if (e == cudaSuccess) e = encode_pages(&maps.v, a.kv.v, a, a.kv.v_row, a.kv.v_head, a.kv.v_page);
  } else {
    if (e == cudaSuccess) e = encode_rows(&maps.k, a.kv.k, D, a.s.Hkv, a.kv.k_head, a.num_tokens, a.kv.k_row, 1, kKeyBlock);
    if (e == cudaSuccess) e = encode_rows(&maps.v, a.kv.v, D, a.s.Hkv, a.kv.v_head, a.num_tokens, a.kv.v_row, 1, kKeyBlock);
  }
  if (e == cudaSuccess) e = set_max_dynamic_smem((const void *)attn_tc_kernel<D, PAGED>, TcShape<D>::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)a.p.max_units * a.s.Hkv;
  return launch_pdl(attn_tc_kernel<D, PAGED>, dim3((unsigned)std::min<int64_t>(most, a.s.ctas)), dim3(kThreads), TcShape<D>::kSmem,
                    st, 1u, maps, a);
}

}  // namespace

bool attn_tc_takes(const AttnShape &s) {
  return s.dtype == LORA_BF16 && (s.D == 64 || s.D == 128) && s.G <= kRows && sgmv_supported();
}

cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t st) {
  const bool paged = a.kv.page_size > 0;
  if (a.s.D == 128) return paged ? launch<128, true>(a, st) : launch<128, false>(a, st);
  return paged ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace ra
