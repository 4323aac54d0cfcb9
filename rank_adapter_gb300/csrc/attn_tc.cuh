// Shared pieces of the tensor-core attention kernels: PTX, waits, the walk over a CTA's
// work, tensor maps.
#pragma once

#include "attn.cuh"
#include "tcgen05.cuh"

namespace ra {
namespace {

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Four MMAs of 16 keys each: A (P) in TMEM, 8 columns a step, B (V) in shared memory. Every lane of the warp calls it.
__device__ __forceinline__ void mma_pv4(uint32_t d, uint32_t p, uint64_t bd, uint64_t b_step, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred q, e, t;\n\t.reg .b32 r, a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
      "elect.sync r|e, 0xffffffff;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.eq.b32 t, %3, %3;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
      "add.s64 b1, %2, %5;\n\tadd.s64 b2, b1, %5;\n\tadd.s64 b3, b2, %5;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}"
      ::"r"(d), "r"(p), "l"(bd), "r"(idesc), "r"(acc), "l"(b_step) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}
// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// kind::f16 with fp32 accumulator and both operands K-major.
__host__ __device__ constexpr uint32_t idesc_kk(int M, int N) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// mbar_wait_warp, but for its first look at the clock: reading %globaltimer takes longer than most of these waits.
__device__ __forceinline__ bool await(uint64_t *b, uint32_t parity, int *err, int code) {
  bool ok = mbar_try(b, parity);
  for (int i = 0; !ok && i < 32; ++i) ok = mbar_try(b, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  return mbar_wait_warp(b, parity, err, code);
}

// Waits, for up to kWaitNs, until *at is past pos.
__device__ __forceinline__ bool past(const volatile uint32_t *at, uint32_t pos, int *err, int code) {
  const uint64_t t0 = *at > pos ? 0 : global_ns();
  while (*at <= pos)
    if (global_ns() - t0 > kWaitNs) {
      atomicOr(err, code);
      return false;
    }
  __threadfence_block();
  return true;
}

// ------------------------------------------------------------------ walk over a CTA's items

// Item k of this CTA (a unit of one key-value head): the units lie in order of falling cost; every other round of
// CTAs runs backwards.
struct Item {
  AttnUnit u;
  int head, blocks;
  bool pair;
};

// One warp's walk; every lane calls. The next item's record comes by cp.async into 32 bytes of shared memory of the
// warp's own (in registers, it was waited for and spilled ahead of the current item).
struct Walk {
  const AttnArgs &a;
  int4 *record;
  uint32_t n, at, k = 0;
  uint32_t pos = 0;      // blocks before the current item: block b of one tile belongs to stream (pos + b) & 1
  uint32_t index = 0;    // items with any before it
  __device__ __forceinline__ Walk(const AttnArgs &args, void *slot) : a(args), record(static_cast<int4 *>(slot)), n(~0u) {
    fetch();  // the first record with the number of units, not behind it: the plan has room for a unit of each CTA
    n = (uint32_t)args.plan[AttnPlan::kUnits] * (uint32_t)args.s.Hkv;
  }
  static __device__ __forceinline__ uint32_t at_of(uint32_t k) {
    return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  }
  __device__ __forceinline__ void fetch() {
    at = at_of(k);
    const uint32_t lane = threadIdx.x & 31;
    if (at < n && lane < 2)
      cp_async16(record + lane, a.plan + a.p.units() + (int64_t)AttnPlan::kUnit * (at / (uint32_t)a.s.Hkv) + 4 * lane);
  }
  // False at the end. Call done() after each item.
  __device__ __forceinline__ bool item(Item &it) {
    if (at >= n) return false;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    const int4 r0 = record[0], r1 = record[1];
    __syncwarp();
    it.u = AttnUnit{r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
    it.head = (int)(at % (uint32_t)a.s.Hkv);
    it.blocks = it.u.kb1 - it.u.kb0;
    it.pair = it.u.tokens > a.s.tile_tokens;
    ++k;
    fetch();
    return true;
  }
  __device__ __forceinline__ void done(const Item &it) {
    pos += it.blocks;
    index += it.blocks > 0;
  }
  // Stream t's blocks of the item: from first(t) on, every step(it)-th one.
  __device__ __forceinline__ int first(const Item &it, int t) const { return it.pair ? 0 : (int)((pos ^ (uint32_t)t) & 1u); }
  __device__ __forceinline__ int step(const Item &it) const { return it.pair ? 1 : 2; }
};

// Keys that every row of a unit sees.
__device__ __forceinline__ int common_keys(const AttnUnit &u, int causal) { return visible_keys(u.pos0, u.kv_len, causal); }

// ------------------------------------------------------------------ values that not every row sees

// A V block in shared memory as the tensor core takes it (rows of 128 bytes, swizzled, 64 elements of all rows and then the
// next 64): rows [r0, r1), which some row of the unit does not see, are looked at, and elements that are not finite become
// zeros; rows from r1 to the next multiple of 16, behind the keys, are zeroed. `me` of `of` threads does its share; true
// where it took a value out.
template <int D>
__device__ __forceinline__ bool fix_values(unsigned char *block, int half_bytes, int r0, int r1, int me, int of) {
  constexpr int kChunks = D / 8;  // of a row
  auto chunk = [&](int i) {
    const int r = i / kChunks, c = i % kChunks;
    return reinterpret_cast<uint4 *>(block + (c / 8) * half_bytes + swz128(r, c % 8));
  };
  uint32_t any = 0;  // an exponent of all ones, plus one, carries into its sign
#pragma unroll 4
  for (int i = r0 * kChunks + me; i < r1 * kChunks; i += of) {
    const uint4 x = *chunk(i);
    any |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) | ((x.z & 0x7f807f80u) + 0x00800080u) |
           ((x.w & 0x7f807f80u) + 0x00800080u);
  }
  const bool bad = (any & 0x80008000u) != 0;
  if (bad) {
#pragma unroll 1
    for (int i = r0 * kChunks + me; i < r1 * kChunks; i += of) {
      uint32_t *q = reinterpret_cast<uint32_t *>(chunk(i));
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        uint32_t x = q[e];
        if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
        if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
        q[e] = x;
      }
    }
  }
#pragma unroll 1
  for (int i = r1 * kChunks + me; i < ((r1 + 15) & ~15) * kChunks; i += of) *chunk(i) = make_uint4(0, 0, 0, 0);
  return bad;
}

// What fix_values took out of column d of the unit's values, for a row that sees keys up to `end`: next to it, what is
// finite does not count. Zero where nothing was.
__device__ __forceinline__ float taken_out(const AttnArgs &a, const AttnUnit &u, int head, int d, int seen, int end) {
  float sum = 0.f;
  for (int j = max(seen, u.kb0 * kKeyBlock); j < min(end, u.kb1 * kKeyBlock); ++j) {
    int64_t at;
    if (a.kv.page_size > 0) {
      const int page = a.kv.table[(int64_t)u.seq * a.kv.ld_table + (j >> a.kv.log2_page)];
      if ((unsigned)page >= (unsigned)a.kv.num_pages) continue;
      at = page * a.kv.v_page + (j & (a.kv.page_size - 1)) * a.kv.v_row;
    } else {
      at = ((int64_t)u.row0 - u.pos0 + j) * a.kv.v_row;
    }
    const float f = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.kv.v)[at + head * a.kv.v_head + d]);
    if (!isfinite(f)) sum += f;
  }
  return sum;
}

// ------------------------------------------------------------------ host side

cudaError_t encode(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                   const cuuint32_t *box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows of `heads` heads of D elements, boxes of 64 elements x box_heads x box_rows.
cudaError_t encode_rows(CUtensorMap *m, const void *base, int D, int heads, int64_t head, int64_t rows, int64_t ld, int box_heads,
                        int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  return encode(m, base, 3, dims, strides, box);
}

cudaError_t encode_pages(CUtensorMap *m, const void *base, const AttnArgs &a, int64_t row, int64_t head, int64_t page) {
  const cuuint64_t dims[4] = {(cuuint64_t)a.s.D, (cuuint64_t)a.kv.page_size, (cuuint64_t)a.s.Hkv, (cuuint64_t)a.kv.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)row * 2, (cuuint64_t)head * 2, (cuuint64_t)page * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(a.kv.page_size, kKeyBlock), 1, 1};
  return encode(m, base, 4, dims, strides, box);
}

}  // namespace
}  // namespace ra
