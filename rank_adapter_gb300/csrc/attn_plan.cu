// The plan of a step's attention (lora_prepare_seqs) and the cache write
// (lora_kv_write).
//
// Plan: a sequence's rows are cut into units (up to two 128-row tiles of one
// key-value head's query heads), a unit's cost is its blocks of keys times its
// tiles. Units above a size are cut along their keys; the units are written in the
// order of falling cost, so that CTAs that take every ctas-th one end together. The
// size is the even share of a CTA, total cost x heads / CTAs, where there are many
// units; where there are few, 32 sizes around it are tried, a warp each, and the one
// is taken whose rounds of CTAs end first (three sequences of 110 thousand keys: 168
// pieces of a share on 152 CTAs 299 us, 144 larger ones 213). One CTA does it
// all; it is latency, which a step pays once for all layers: 6.3 us for 256 single tokens,
// 8.3 for 48 drafts, 14 for those three long ones.
//
// Cache write: a warp a row, all of its 16-byte loads in flight before the first
// store; it moves each byte once in and once out (16 prompts of 128 to 2048 tokens, 162
// MB: 27.2 us, 5.96 TB/s; 256 single tokens 2.9 us with the host's call).
#include "attn.cuh"
#include "tcgen05.cuh"

namespace ra {

constexpr int kFewRows = 32;  // rows of a sequence, on average, up to which units are of few rows

AttnShape attn_shape(const lora_seqs &q) {
  AttnShape s{};
  s.dtype = q.dtype;
  s.Hq = q.num_heads;
  s.Hkv = q.num_kv_heads;
  s.G = s.Hq / s.Hkv;
  s.D = q.head_dim;
  s.causal = q.causal != 0;
  s.tc = attn_tc_takes(s);
  s.tile_tokens = s.tc ? 128 / s.G : std::max(1, 32 / s.G);
  s.unit_tokens = s.tc ? 2 * s.tile_tokens : s.tile_tokens;
  s.slot_rows = s.tc ? 256 : std::max(32, s.G);
  // Units of few rows where a sequence has up to kFewRows rows on average, of the least size that takes a token of every
  // sequence, or 1.4 times the average where there are more (48 drafts of 1 to 5 tokens by 7 heads: 24.4 us in units of 32
  // rows, 29.3 in units of 64). (256 requests of a token by 4 heads a group: 306 us, 429 as tiles
  // of 128 rows. A prompt of 500 tokens by 4: 20.9 us in units of 64 rows, 16.0 as tiles.)
  const int64_t rows = (int64_t)q.num_tokens * s.G;
  if (s.tc && s.G <= 64 && rows <= (int64_t)kFewRows * q.num_seqs) {
    const int64_t want = std::max<int64_t>(s.G, q.num_tokens > q.num_seqs ? 7 * rows / 5 / q.num_seqs : 0);
    s.few = want <= 16 ? 16 : want <= 32 ? 32 : 64;
    s.unit_tokens = s.few / s.G;
    s.slot_rows = s.few;
  }
  s.ctas = (s.tc && s.few != 16 ? 1 : 2) * std::max(1, sm_count());
  s.min_cost = 2;
  // In blocks of keys by tiles, as measured: two CTAs of 16 rows take 3 us a block while all read, one alone about 1.1;
  // one of 32 or 64 rows 1.5 and 0.86; one of two tiles 0.85 a tile, whatever the others do.
  s.alone = s.few == 16 ? 0.35f : s.few > 0 ? 0.57f : 1.f;
  s.piece_cost = s.few > 0 ? 1.f : 5.f;
  s.join_cost = s.few == 16 ? 0.8f : s.few > 0 ? 2.5f : 8.f;
  s.max_slots = (s.few > 0 ? 4 : 2) * s.ctas / s.Hkv + 2;
  s.scale_log2 = (float)((double)q.scale * 1.4426950408889634);
  return s;
}

AttnPlan attn_plan(const AttnShape &s, int num_seqs, int num_tokens) {
  AttnPlan p;
  p.max_seqs = std::max(1, num_seqs);
  p.max_units = num_tokens / s.unit_tokens + num_seqs + s.max_slots + 1;
  p.max_groups = s.max_slots;
  return p;
}

// Partial results of a key-value head, however units are cut, and the rows of them all.
int most_slots(const AttnShape &s) { return 8 * std::max(1, sm_count()) / s.Hkv + 2; }

int64_t attn_slot_rows(const lora_seqs &q) {
  const AttnShape s = attn_shape(q);
  if (!s.tc) return (int64_t)s.max_slots * s.slot_rows;
  const int sms = std::max(1, sm_count());
  return std::max({256ll * (2 * sms / s.Hkv + 2), 64ll * (4 * sms / s.Hkv + 2), 16ll * (8 * sms / s.Hkv + 2)});
}

size_t attn_plan_bytes(const lora_seqs &q) {
  AttnShape s = attn_shape(q);
  if (s.tc) s.max_slots = most_slots(s);
  AttnPlan p = attn_plan(s, q.num_seqs, q.num_tokens);
  if (s.tc) {
    // Units of few rows: sequences make one each, and one for each unit_tokens of the batch's tokens, which are less than
    // two a sequence (a unit has room for 1.4 times the average of rows and holds more than half of it, or for a token).
    const int long_tokens = 2 * (128 / s.G);
    p.max_units = (int)std::max<int64_t>(q.num_tokens / long_tokens + q.num_seqs,
                                         std::min<int64_t>((int64_t)q.num_tokens + q.num_seqs, 3ll * q.num_seqs)) + s.max_slots + 1;
  }
  return (size_t)p.words() * sizeof(int32_t);
}

bool attn_may_split(const AttnShape &s, int64_t max_kv) {
  return (max_kv + kKeyBlock - 1) / kKeyBlock * (s.unit_tokens > s.tile_tokens ? 2 : 1) > s.min_cost;
}

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 256;
constexpr int kNear = 1024;  // sequences that are kept in shared memory

struct PlanArgs {
  AttnShape s;
  AttnPlan p;
  const int32_t *q_start, *kv_len;
  int S, T;
  int64_t max_kv;
  int32_t *plan;
};

// What the CTA's warps tell one another in a scan. Calls take its two halves in turn, so that each needs one barrier: a
// warp writes a half again only behind the next call's barrier, which the last readers of it have passed.
struct ScanRoom {
  unsigned long long part[2][kThreads / 32];
  int top[2][kThreads / 32];
};

// Exclusive sum over the CTA's threads; *total gets the sum of all.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long v, ScanRoom &room, uint32_t &turn,
                                                         unsigned long long *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long incl = v, *part = room.part[turn++ & 1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  unsigned long long w = part[lane];  // every warp: the sums up to each warp's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const unsigned long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return incl - v + (warp > 0 ? before : 0ull);
}

// The largest value of the CTA's earlier threads, 0 where there is none above it; *most gets that of all threads.
__device__ __forceinline__ int block_max(int v, ScanRoom &room, uint32_t &turn, int *most) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int *top = room.top[turn++ & 1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = max(v, u);
  }
  if (lane == 31) top[warp] = v;
  const int before = __shfl_up_sync(0xffffffffu, v, 1);
  __syncthreads();
  const int other = top[lane];
  *most = __reduce_max_sync(0xffffffffu, other);
  return max(lane > 0 ? before : 0, __reduce_max_sync(0xffffffffu, lane < warp ? other : 0));
}

struct Cut {  // a unit before it is split
  int seq, row0, tokens, kv_len, pos0, blocks, cost;
};

__device__ __forceinline__ Cut cut_of(const PlanArgs &a, const int32_t *cum, const int4 *seqs, int i) {
  int lo = 0, hi = a.S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  const int4 q = seqs[lo];
  Cut c;
  c.seq = lo;
  const int off = (i - cum[lo]) * a.s.unit_tokens;
  c.row0 = q.x + off;
  c.tokens = min(a.s.unit_tokens, q.y - off);
  c.kv_len = q.z;
  c.pos0 = q.z - q.y + off;
  c.blocks = (visible_keys(c.pos0 + c.tokens - 1, q.z, a.s.causal) + kKeyBlock - 1) / kKeyBlock;
  c.cost = c.blocks * (c.tokens > a.s.tile_tokens ? 2 : 1);
  return c;
}

__global__ void __launch_bounds__(kThreads) prepare_seqs_kernel(const PlanArgs a) {
  __shared__ ScanRoom room;
  __shared__ unsigned long long total_cost;
  __shared__ int bins[kBins], bad, most, groups, sizes[kThreads / 32], costs[kThreads];
  __shared__ float ends[kThreads / 32];
  __shared__ int4 near_seqs[kNear];
  __shared__ int32_t near_cum[kNear];
  const int tid = threadIdx.x;
  uint32_t turn = 0;
  int32_t *const out_cum = a.plan + a.p.cum();
  int4 *const out_seqs = reinterpret_cast<int4 *>(a.plan + a.p.seqs());
  const bool near = a.S <= kNear;
  int32_t *cum = near ? near_cum : out_cum;
  int4 *seqs = near ? near_seqs : out_seqs;
  if (tid == 0) {
    total_cost = 0;
    bad = most = groups = 0;
  }
  if (tid < kBins) bins[tid] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  // The sequences, and the units before each.
  unsigned long long total, base = 0;
  int end = 0;  // where the sequences so far end
  for (int b0 = 0; b0 < a.S; b0 += kThreads) {
    const int b = b0 + tid;
    int u = 0, first = 0, last = 0;
    if (b < a.S) {
      const int r0 = a.q_start[b], r1 = a.q_start[b + 1];
      const int kv = a.kv_len != nullptr ? a.kv_len[b] : r1 - r0;
      const bool good = r0 >= 0 && r1 >= r0 && r1 <= a.T && kv >= 0 && kv <= a.max_kv;
      if (!good) atomicAdd(&bad, 1);
      seqs[b] = good ? make_int4(r0, r1 - r0, kv, 0) : make_int4(0, 0, 0, 0);
      if (near) out_seqs[b] = seqs[b];
      u = good ? (r1 - r0 + a.s.unit_tokens - 1) / a.s.unit_tokens : 0;
      first = good ? r0 : 0;
      last = good ? r1 : 0;
    }
    int most_end;
    first = max(first, max(end, block_max(last, room, turn, &most_end)));  // one treated as empty starts where those before it end
    end = max(end, most_end);
    const unsigned long long before = base + block_scan(u, room, turn, &total);
    if (b < a.S) {
      cum[b] = (int)min(before, (unsigned long long)INT32_MAX);
      a.plan[a.p.start() + b] = first;
    }
    base += total;
  }
  // Sequences that overlap (q_start out of order) can make more units than there is room
  // for: the last of them are dropped.
  const int most_units = a.p.max_units - a.s.max_slots;
  if (tid == 0 && base > (unsigned long long)most_units) atomicAdd(&bad, 1);
  const int n = (int)min(base, (unsigned long long)most_units);
  __syncthreads();
  unsigned long long mine = 0;
  int top = 0;
  Cut own{};  // this thread's unit, where there is at most one
  for (int i = tid; i < n; i += kThreads) {
    own = cut_of(a, cum, seqs, i);
    mine += own.cost;
    top = max(top, own.cost);
  }
  costs[tid] = own.cost;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0 && mine > 0) {
    atomicAdd(&total_cost, mine);
    atomicMax(&most, top);
  }
  __syncthreads();
  const int64_t share = ((int64_t)total_cost * a.s.Hkv + a.s.ctas - 1) / a.s.ctas;
  int64_t chunk = max((int64_t)a.s.min_cost, share) * 5 / 4;  // units above it are cut
  int64_t piece = max((int64_t)a.s.min_cost, share);          // into pieces of about this cost
  if (n <= kThreads && (int64_t)n * a.s.Hkv <= 2 * a.s.ctas) {
    // Sizes from half a share to 2.4 shares, and no cut at all. The last CTA ends with the largest piece, or where the
    // share and the smallest piece on top of it end, or, of even pieces, with a whole round; pieces that are left over
    // run faster where the others' traffic was the limit. A piece's beginning and end and the joining cost blocks' time too.
    const int warp = tid >> 5, lane = tid & 31;
    const int size = warp == 31 ? INT32_MAX / 2 : (int)max((int64_t)a.s.min_cost, share * (8 + warp) / 16 + 1);
    int pieces = 0, largest = 0, smallest = INT32_MAX;
    for (int i = lane; i < n; i += 32) {
      const int p = max(1, (costs[i] + size - 1) / size), each = (costs[i] + p - 1) / p;
      pieces += p;
      largest = max(largest, each);
      smallest = min(smallest, each);
    }
    pieces = __reduce_add_sync(0xffffffffu, pieces);
    largest = __reduce_max_sync(0xffffffffu, largest);
    smallest = __reduce_min_sync(0xffffffffu, smallest);
    if (lane == 0) {
      const int items = pieces * a.s.Hkv, rounds = (items + a.s.ctas - 1) / a.s.ctas, last = items - (rounds - 1) * a.s.ctas;
      const float average = (float)total_cost / (float)max(1, pieces);
      const float even = ((float)(rounds - 1) + a.s.alone + (1.f - a.s.alone) * (float)last / (float)a.s.ctas) * average;
      const float end = fmaxf((float)largest * a.s.alone, fminf(even, (float)share + (float)smallest));
      ends[warp] = pieces - n > a.s.max_slots / 2 ? INFINITY : end + a.s.piece_cost * (float)rounds + (pieces > n ? a.s.join_cost + 0.1f * (float)pieces / (float)n : 0.f);
      sizes[warp] = size;
    }
    __syncthreads();
    int best = 31;
    for (int x = 30; x >= 0; --x)
      if (ends[x] < ends[best]) best = x;
    chunk = piece = sizes[best];
  }
  const int peak = max(1, most);
  auto bin_of = [&](int cost) { return kBins - 1 - (int)((int64_t)cost * (kBins - 1) / peak); };
  // Twice over the units: the pieces of each cost counted, then written in that order.
  for (int pass = 0; pass < 2; ++pass) {
    base = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
      const int i = i0 + tid;
      Cut c{};
      int pieces = 0;
      if (i < n) {
        c = n <= kThreads ? own : cut_of(a, cum, seqs, i);
        pieces = c.cost > chunk ? (int)min((int64_t)c.blocks, (c.cost + piece - 1) / piece) : 1;
      }
      const bool wants = pieces > 1;
      const unsigned long long at = base + block_scan(wants ? (unsigned long long)pieces : 0ull, room, turn, &total);
      base += total;
      const bool split = wants && at + pieces <= (unsigned long long)a.s.max_slots;
      if (i >= n) continue;
      if (!split) pieces = 1;
      const int tiles = c.tokens > a.s.tile_tokens ? 2 : 1;
      for (int j = 0; j < pieces; ++j) {
        const int kb0 = (int)((int64_t)c.blocks * j / pieces), kb1 = (int)((int64_t)c.blocks * (j + 1) / pieces);
        const int bin = bin_of((kb1 - kb0) * tiles);
        const int pos = atomicAdd(&bins[bin], 1);
        if (pass == 1) {
          int4 *u = reinterpret_cast<int4 *>(a.plan + a.p.units() + (int64_t)AttnPlan::kUnit * pos);
          u[0] = make_int4(c.seq, c.row0, c.tokens, kb0);
          u[1] = make_int4(kb1, c.kv_len, c.pos0, split ? (int)at + j : -1);
        }
      }
      if (pass == 1 && split) {
        const int g = atomicAdd(&groups, 1);
        *reinterpret_cast<int4 *>(a.plan + a.p.groups() + (int64_t)AttnPlan::kGroup * g) =
            make_int4(c.row0, c.tokens, (int)at, pieces);
      }
    }
    __syncthreads();
    if (pass == 0) {
      const unsigned long long v = tid < kBins ? (unsigned long long)bins[tid] : 0ull;
      const unsigned long long at = block_scan(v, room, turn, &total);
      if (tid < kBins) bins[tid] = (int)at;
      if (tid == 0) a.plan[AttnPlan::kUnits] = (int)total;
      __syncthreads();
    }
  }
  if (tid == 0) {
    a.plan[AttnPlan::kGroups] = groups;
    a.plan[AttnPlan::kErr] = 0;
    a.plan[AttnPlan::kBad] = bad;
  }
}

// ------------------------------------------------------------------ cache write

struct WriteArgs {
  const int32_t *plan;
  AttnPlan p;
  int *err;
  const uint8_t *k, *v;
  uint8_t *kc, *vc;
  int64_t ldk, ldv, k_page, k_row, k_head, v_page, v_row, v_head, ld_table;  // bytes but for ld_table
  const int32_t *table;
  int S, T, page_size, log2_page, num_pages, max_pages, chunks, head_chunks;  // 16-byte chunks of a row and of a head
};

constexpr int kWriteWarps = 4;

__global__ void __launch_bounds__(32 * kWriteWarps) kv_write_kernel(const WriteArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int4 *seqs = reinterpret_cast<const int4 *>(a.plan + a.p.seqs());
  for (int t = blockIdx.x * kWriteWarps + (threadIdx.x >> 5); t < a.T; t += gridDim.x * kWriteWarps) {
    // The sequence that holds row t: the last one that starts at or before it.
    int lo = 0, hi = a.S;  // the answer is in [lo, hi)
    while (hi - lo > 1) {  // 32 probes a round
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const bool before = at < hi && a.plan[a.p.start() + at] <= t;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, before) | 1u);
      hi = min(hi, lo + (last + 1) * step);
      lo = lo + last * step;
    }
    const int4 q = seqs[lo];
    const int i = t - q.x, p = q.z - q.y + i;
    if (i < 0 || i >= q.y || p < 0) continue;
    const int page = a.table[(int64_t)lo * a.ld_table + (p >> a.log2_page)];
    if ((unsigned)page >= (unsigned)a.num_pages) {
      if (lane == 0) atomicOr(a.err, kErrBadPage);
      continue;
    }
    const int64_t in_page = p & (a.page_size - 1);
    const uint8_t *ks = a.k + (int64_t)t * a.ldk, *vs = a.v + (int64_t)t * a.ldv;
    uint8_t *kd = a.kc + page * a.k_page + in_page * a.k_row, *vd = a.vc + page * a.v_page + in_page * a.v_row;
    for (int c0 = lane; c0 < a.chunks; c0 += 128) {
      uint4 x[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c0 + 32 * j < a.chunks) {
          x[j] = __ldg(reinterpret_cast<const uint4 *>(ks) + c0 + 32 * j);
          y[j] = __ldg(reinterpret_cast<const uint4 *>(vs) + c0 + 32 * j);
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + 32 * j;
        if (c < a.chunks) {
          const int h = c / a.head_chunks;
          const int64_t d = (int64_t)(c - h * a.head_chunks) * 16;
          *reinterpret_cast<uint4 *>(kd + h * a.k_head + d) = x[j];
          *reinterpret_cast<uint4 *>(vd + h * a.v_head + d) = y[j];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_prepare_seqs(const lora_seqs &q, cudaStream_t st) {
  PlanArgs a{};
  a.s = attn_shape(q);
  a.p = attn_plan(a.s, q.num_seqs, q.num_tokens);
  a.q_start = q.q_start;
  a.kv_len = q.kv_len;
  a.S = q.num_seqs;
  a.T = q.num_tokens;
  a.max_kv = q.page_size > 0 ? std::min<int64_t>((int64_t)q.page_size * q.max_pages, LORA_MAX_KV_LEN) : q.num_tokens;
  a.plan = static_cast<int32_t *>(q.plan);
  return launch_pdl(prepare_seqs_kernel, dim3(1), dim3(kThreads), 0, st, 1u, a);
}

cudaError_t launch_kv_write(const lora_seqs &q, const lora_kv_cache &c, const void *k, int64_t ldk, const void *v,
                            int64_t ldv, cudaStream_t st) {
  const AttnShape s = attn_shape(q);
  const int es = q.dtype == LORA_BF16 ? 2 : 4;
  WriteArgs a{};
  a.plan = static_cast<const int32_t *>(q.plan);
  a.p = attn_plan(s, q.num_seqs, q.num_tokens);
  a.err = static_cast<int32_t *>(q.plan) + AttnPlan::kErr;
  a.k = static_cast<const uint8_t *>(k);
  a.v = static_cast<const uint8_t *>(v);
  a.kc = static_cast<uint8_t *>(c.k);
  a.vc = static_cast<uint8_t *>(c.v);
  a.ldk = ldk * es;
  a.ldv = ldv * es;
  a.k_page = c.k_page * es;
  a.k_row = c.k_row * es;
  a.k_head = c.k_head * es;
  a.v_page = c.v_page * es;
  a.v_row = c.v_row * es;
  a.v_head = c.v_head * es;
  a.table = q.block_table;
  a.ld_table = q.ld_table;
  a.S = q.num_seqs;
  a.T = q.num_tokens;
  a.page_size = q.page_size;
  while ((1 << a.log2_page) < q.page_size) ++a.log2_page;
  a.num_pages = c.num_pages;
  a.max_pages = q.max_pages;
  a.head_chunks = s.D * es / 16;
  a.chunks = s.Hkv * a.head_chunks;
  const int ctas = (int)std::min<int64_t>(((int64_t)q.num_tokens + kWriteWarps - 1) / kWriteWarps, 16 * 152);
  return launch_pdl(kv_write_kernel, dim3((unsigned)ctas), dim3(32 * kWriteWarps), 0, st, 1u, a);
}

}  // namespace ra
