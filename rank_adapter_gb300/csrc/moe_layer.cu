// The parts of a mixture-of-experts layer around its products: the router
// (lora_moe_route), the gated activation between w13 and w2 (lora_moe_act,
// lora_moe_act_mx) and the weighted sum over a token's choices
// (lora_moe_combine). Pairs are token-major, p = t * topk + k.
#include "mx.cuh"

namespace ra {
namespace {

// ------------------------------------------------------------------ router
//
// One warp a token: lane l holds logits l, l + 32, ... in registers. A round
// finds the warp's largest key (redux.sync) and among the lanes that hold it
// the lowest expert; topk rounds choose topk experts, so a row is read once
// and nothing is sorted that is not asked for. Lane k keeps choice k and the
// weights need one or two warp sums. A long batch is bound by the rounds'
// instructions: 16-bit logits carry their expert in the key's low half, so
// that one reduction a round gives both, and lanes with few keys sort them first
// (16381 tokens of 256 experts, top 8: 8.8 us; before that
// unsorted 11.5 us; with separate reductions, as for fp32 logits, 15.1 us).

constexpr int kRouteWarps = 4;

struct RouteArgs {
  const void *logits;
  int64_t ldl;
  int32_t *ids;
  float *w;
  const int32_t *expert_map;
  int32_t *pair_slot;
  int T, E, topk, local;
  int sigmoid, renorm;
  float scale;
};

// Order-preserving key of a logit; 0 is below every key. NaN counts as
// -infinity, +infinity as the largest finite number (so that a row's weights
// stay numbers), -0 as 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (isnan(v)) v = -INFINITY;
  const uint32_t u = __float_as_uint(fminf(v, 3.402823466e38f) + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
// Logits of type T in a lane's registers: the key of expert e, its logit, and
// the warp's largest with its expert (the lowest where logits are equal).
template <typename T, int NV> struct RouteKeys;
template <int NV> struct RouteKeys<float, NV> {
  uint32_t key[NV];
  __device__ __forceinline__ static uint32_t make(float v, int) { return order_key(v); }
  __device__ __forceinline__ static float value(uint32_t k) { return key_value(k); }
  __device__ __forceinline__ static bool numbered(uint32_t k) { return k > order_key(-INFINITY); }
  __device__ __forceinline__ uint32_t take(int lane, int &e) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = max(m, key[i]);
    const uint32_t best = __reduce_max_sync(0xffffffffu, m);
    uint32_t first = 0x7fffffffu;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i)
      if (key[i] == best) first = lane + 32 * i;
    e = (int)__reduce_min_sync(0xffffffffu, first);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (lane + 32 * i == e) key[i] = 0u;
    return best;
  }
};
template <int NV> struct RouteKeys<__nv_bfloat16, NV> {
  uint32_t key[NV];
  static constexpr float kMax = 3.3895314e38f;  // the largest finite bf16
  // A finite bf16 value's key has all bits of the low half equal (0 or 1): the half is free for the expert.
  __device__ __forceinline__ static uint32_t make(float v, int e) {
    return (order_key(v > kMax ? kMax : v) & 0xffff0000u) | (uint32_t)(0xffff - e);
  }
  __device__ __forceinline__ static float value(uint32_t k) {
    return key_value(k >> 31 ? k & 0xffff0000u : k | 0xffffu);
  }
  __device__ __forceinline__ static bool numbered(uint32_t k) { return k >= (order_key(-INFINITY) | 0xffffu) + 1u; }
  // The lane's keys largest first: Batcher's odd-even merge sort.
  __device__ __forceinline__ void sort() {
#pragma unroll
    for (int p = 1; p < NV; p *= 2)
#pragma unroll
      for (int k = p; k >= 1; k /= 2)
#pragma unroll
        for (int j = k % p; j + k < NV; j += 2 * k)
#pragma unroll
          for (int i = 0; i < k; ++i)
            if (i + j + k < NV && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
              const uint32_t x = key[i + j], y = key[i + j + k];
              key[i + j] = max(x, y);
              key[i + j + k] = min(x, y);
            }
  }
  __device__ __forceinline__ uint32_t take_sorted(int, int &e) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, key[0]);
    if (key[0] == best) {
#pragma unroll
      for (int i = 0; i + 1 < NV; ++i) key[i] = key[i + 1];
      key[NV - 1] = 0u;
    }
    e = 0xffff - (int)(best & 0xffffu);
    return best;
  }
  __device__ __forceinline__ uint32_t take(int, int &e) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = max(m, key[i]);
    const uint32_t best = __reduce_max_sync(0xffffffffu, m);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] == best) key[i] = 0u;
    e = 0xffff - (int)(best & 0xffffu);
    return best;
  }
};

template <typename T, int NV>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(RouteArgs a) {
  // The next kernel may read pair_slot before its wait (lora_prepare_meta), so
  // this one releases it only by completing.
  pdl_wait();
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kAll = 0xffffffffu;
  using Keys = RouteKeys<T, NV>;
  // A sorted lane offers its first key and moves up, an unsorted one searches
  // all NV. Eight keys' sort is repaid from three rounds on (7.56 us, unsorted
  // 7.87); sixteen keys' is not with eight (28.2 us, unsorted 21.7).
  constexpr bool kSort = sizeof(T) == 2 && NV > 1 && NV <= 8;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5); t < a.T;
       t += (int64_t)gridDim.x * kRouteWarps) {
    const T *row = static_cast<const T *>(a.logits) + t * a.ldl;
    Keys k;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      k.key[i] = e < a.E ? Keys::make(Elem<T>::to_f(row[e]), e) : 0u;
    }
    float total = 0.f;  // softmax without renormalisation: the sum over all experts
    if (!a.sigmoid && !a.renorm) {
      uint32_t m = k.key[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) m = max(m, k.key[i]);
      m = __reduce_max_sync(kAll, m);
      if (Keys::numbered(m)) {
        const float top = Keys::value(m);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (Keys::numbered(k.key[i])) total += expf(Keys::value(k.key[i]) - top);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    }
    uint32_t mine = 0, first = 0;  // keys of choice `lane` and of the first
    int id = 0;
    auto chose = [&](int c, uint32_t key, int e) {
      if (c == 0) first = key;
      if (lane == c) {
        mine = key;
        id = e;
      }
    };
    int e;
    if (kSort && a.topk >= 3) {
      if constexpr (kSort) {
        k.sort();
        for (int c = 0; c < a.topk; ++c) {
          const uint32_t key = k.take_sorted(lane, e);
          chose(c, key, e);
        }
      }
    } else {
      for (int c = 0; c < a.topk; ++c) {
        const uint32_t key = k.take(lane, e);
        chose(c, key, e);
      }
    }
    const bool chosen = lane < a.topk, live = chosen && Keys::numbered(mine);
    float w = 0.f;
    if (live) {
      // A sigmoid below e^-18 is its exponential (1 + e^v is 1 in fp32), which
      // keeps it a number down to -103. Where the first choice is one, all are:
      // renormalised weights are then a softmax's, whose common factor cancels,
      // however low the logits are.
      const float v = Keys::value(mine);
      if (!a.sigmoid || (a.renorm && first < order_key(-18.f))) w = expf(v - Keys::value(first));
      else if (v < -18.f) w = expf(v);
      else w = 1.f / (1.f + expf(-v));
    }
    if (a.renorm) {
      total = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    }
    if ((a.renorm || !a.sigmoid) && total > 0.f) w /= total;
    if (!chosen) continue;
    const int64_t p = t * a.topk + lane;
    a.ids[p] = id;
    a.w[p] = w * a.scale;
    if (a.pair_slot != nullptr) {
      const int el = a.expert_map != nullptr ? a.expert_map[id] : id;
      a.pair_slot[p] = el >= a.local ? -1 : (el < 0 || !live) ? 0 : 1 + el;
    }
  }
}

template <typename T>
cudaError_t route_launch(const RouteArgs &a, cudaStream_t st) {
  const int nv = (a.E + 31) / 32;
  void (*k)(RouteArgs) = nv <= 1 ? moe_route_kernel<T, 1> : nv <= 2 ? moe_route_kernel<T, 2>
                       : nv <= 4 ? moe_route_kernel<T, 4> : nv <= 8 ? moe_route_kernel<T, 8>
                       : nv <= 16 ? moe_route_kernel<T, 16> : moe_route_kernel<T, 32>;
  const int blocks = (int)std::min<int64_t>(((int64_t)a.T + kRouteWarps - 1) / kRouteWarps, 152 * 64);
  return launch_pdl(k, dim3((unsigned)blocks), dim3(kRouteWarps * 32), 0, st, 1u, a);
}

// ------------------------------------------------------------------ activation
//
// h = silu(gate) * up over rows of [gate | up], eight elements a thread;
// rows of pairs without a local expert are neither read nor written.

constexpr int kThreads = 256;

struct ActArgs {
  const void *y13;
  int64_t ldy;
  const int32_t *pair_slot;
  void *h;         // bf16 / f32 rows, or the codes of the 4-bit form
  int64_t ldh;     // elements; bytes of a row of codes
  uint8_t *scales;
  int64_t lds;
  int P, inter;
};

// silu(g) = g * (g < 0 ? e : 1) / (1 + e), e = exp(-|g|): nothing overflows, so
// that a gate far below -87 still counts beside a large `up` (the quotient
// g / (1 + exp(-g)) would be 0 before the product). For a result that is rounded
// to bf16 the approximate powers of two and reciprocal do, together within
// (10 + |g|) * 2^-23 of the value: exp(-|g| / 2) within 2 ulp and the rounding of
// its exponent, its square, the reciprocal within 1 ulp, three roundings. The
// square reaches the subnormal numbers, so the power need not: no scaling of its
// own (with CUDA's fast exponential and a reciprocal 65.5 us for 32744 rows of
// 2048, as here 59.0). An fp32 result takes the exact ones; for a bf16 one they bound
// the kernel by instructions (88.5 us where CUDA's fast ones took 66.9, at an
// earlier stage).
template <bool kFast> __device__ __forceinline__ float silu(float g) {
  if constexpr (kFast) {
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(fabsf(g) * -0.72134752f));  // -log2(e) / 2
    const float e = h * h;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));  // of 1 to 2
    return g * (g < 0.f ? e * r : r);
  } else {
    const float e = expf(-fabsf(g));
    return (g < 0.f ? g * e : g) / (1.f + e);
  }
}

// The activation of chunk c of kActRows rows, p0 and every blockDim.y on: their
// slots, then all their loads, then row by row the arithmetic and
// put(p, live, v); live: the row is in range and has an expert. At 32744 rows
// of 2048, one row a thread at a time 77.6 us, two 69.7 us, four 63.8 us (with the
// quotient form of silu, which stood here before; now 59.0 us, 6.8 TB/s, the
// measured copy rate).
constexpr int kActRows = 4;

template <bool kFast, typename TY, typename Put>
__device__ __forceinline__ void act_rows(const ActArgs &a, int64_t p0, int c, bool in, Put put) {
  int slot[kActRows];
#pragma unroll
  for (int i = 0; i < kActRows; ++i) slot[i] = 1;
  if (a.pair_slot != nullptr)
#pragma unroll
    for (int i = 0; i < kActRows; ++i)
      slot[i] = __ldg(a.pair_slot + min(p0 + i * (int64_t)blockDim.y, (int64_t)a.P - 1));
  Raw8<TY> g[kActRows], u[kActRows];
#pragma unroll
  for (int i = 0; i < kActRows; ++i) {
    const int64_t p = p0 + i * blockDim.y;
    if (!in || p >= a.P) slot[i] = 0;
    const TY *row = static_cast<const TY *>(a.y13) + p * a.ldy + (int64_t)c * 8;
    g[i] = u[i] = Raw8<TY>{};
    if (slot[i] > 0) {
      g[i] = raw8(row);
      u[i] = raw8(row + a.inter);
    }
  }
#pragma unroll
  for (int i = 0; i < kActRows; ++i) {
    float v[8], w[8];
    widen8(g[i], v);
    widen8(u[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu<kFast>(v[j]) * w[j];
    put(p0 + i * blockDim.y, slot[i] > 0, v);
  }
}

template <typename TY, typename TH>
__global__ void __launch_bounds__(kThreads) moe_act_kernel(ActArgs a) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.inter / 8) return;
  const int64_t step = (int64_t)gridDim.y * blockDim.y * kActRows;
  for (int64_t p0 = (int64_t)blockIdx.y * blockDim.y * kActRows + threadIdx.y; p0 < a.P; p0 += step)
    act_rows<sizeof(TH) == 2, TY>(a, p0, c, true, [&](int64_t p, bool live, const float(&v)[8]) {
      if (live) store8(static_cast<TH *>(a.h) + p * a.ldh + (int64_t)c * 8, v);
    });
}

// The same into the 4-bit format. The activation is rounded to bf16 first, so
// that the result is bitwise that of lora_moe_act into bf16 and
// lora_mx_quantize after it.
template <typename TY>
__global__ void __launch_bounds__(kThreads) moe_act_mx_kernel(ActArgs a) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)gridDim.y * blockDim.y * kActRows;
  for (int64_t b0 = (int64_t)blockIdx.y * blockDim.y * kActRows; b0 < a.P; b0 += step)
    act_rows<true, TY>(a, b0 + threadIdx.y, c, c < a.inter / 8, [&](int64_t p, bool live, const float(&v)[8]) {
      // The four lanes of a block of 32 are in one row and in range together.
      float r[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = __bfloat162float(__float2bfloat16_rn(v[j]));
      uint32_t byte;
      const uint32_t q = mx_quantize8(r, byte);
      if (live) {
        *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.h) + p * a.ldh + (int64_t)c * 4) = q;
        if ((c & 3) == 0) a.scales[p * a.lds + (c >> 2)] = (uint8_t)byte;
      }
    });
}

// ------------------------------------------------------------------ weighted sum
//
// out[t] = (out[t] or 0) + sum_k w[t, k] * y[t * topk + k], in fp32 in the
// order of k and rounded once. A thread owns eight columns of a token; the
// rows of up to kAhead choices are requested before the first is used. With
// tokens enough for every SM a CTA walks all columns of its tokens, so that
// the token's slots and weights come from L1 after the first (32744 rows of
// 7168: 83.8 us, 0.93 of the measured copy rate; with CTAs of 256 threads 85.4
// us, and with one of those for each 2048 columns 94.8 us).
constexpr int kCombineThreads = 128;

struct CombineArgs {
  const void *y;
  int64_t ldy;
  const float *w;
  const int32_t *pair_slot;
  void *out;
  int64_t ldo;
  int T, topk, n;
  int accumulate;
};

template <typename TY, typename TO>
__global__ void __launch_bounds__(kCombineThreads, 8) moe_combine_kernel(CombineArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kAhead = sizeof(TY) == 2 ? 8 : 4;
  const int chunks = a.n / 8;
  for (int64_t t = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; t < a.T; t += (int64_t)gridDim.y * blockDim.y) {
    const float *w = a.w + t * a.topk;
    const int32_t *slot = a.pair_slot != nullptr ? a.pair_slot + t * a.topk : nullptr;
    for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < chunks; c += gridDim.x * blockDim.x) {
      TO *o = static_cast<TO *>(a.out) + t * a.ldo + (int64_t)c * 8;
      float acc[8] = {};
      if (a.accumulate) load8_rw(o, acc);
      const TY *y = static_cast<const TY *>(a.y) + t * a.topk * a.ldy + (int64_t)c * 8;
      for (int k0 = 0; k0 < a.topk; k0 += kAhead) {
        Raw8<TY> raw[kAhead];
        float wk[kAhead];
        int sk[kAhead];
        // Slots and weights first, unconditionally: a load behind a branch on
        // the previous one's value would wait for it.
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int k = min(k0 + i, a.topk - 1);
          wk[i] = __ldg(w + k);
          sk[i] = slot != nullptr ? __ldg(slot + k) : 1;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {  // a choice that does not count adds 0 * 0
          const bool live = k0 + i < a.topk && sk[i] > 0;
          raw[i] = Raw8<TY>{};
          if (live) raw[i] = raw8(y + (k0 + i) * a.ldy);
          wk[i] = live ? wk[i] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          float v[8];
          widen8(raw[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = fmaf(wk[i], v[j], acc[j]);
        }
      }
      store8(o, acc);
    }
  }
}

}  // namespace

cudaError_t launch_moe_route(const void *logits, int64_t ldl, int dtype, int T, int E, int topk, int score, int renorm,
                             float scale, const int32_t *expert_map, int local, int32_t *ids, float *w,
                             int32_t *pair_slot, cudaStream_t st) {
  RouteArgs a{logits, ldl, ids, w, expert_map, pair_slot, T, E, topk, local, score == LORA_SCORE_SIGMOID, renorm, scale};
  return dtype == LORA_BF16 ? route_launch<__nv_bfloat16>(a, st) : route_launch<float>(a, st);
}

cudaError_t launch_moe_act(const void *y13, int64_t ldy, int y_dtype, const int32_t *pair_slot, int P, int inter,
                           void *h, int64_t ldh, int h_dtype, cudaStream_t st) {
  const ActArgs a{y13, ldy, pair_slot, h, ldh, nullptr, 0, P, inter};
  const RowGrid l = RowGrid::of(P, inter / 8, kThreads, kActRows);
  void (*k)(ActArgs) =
      y_dtype == LORA_BF16
          ? (h_dtype == LORA_BF16 ? moe_act_kernel<__nv_bfloat16, __nv_bfloat16> : moe_act_kernel<__nv_bfloat16, float>)
          : (h_dtype == LORA_BF16 ? moe_act_kernel<float, __nv_bfloat16> : moe_act_kernel<float, float>);
  return launch_pdl(k, l.grid, l.block, 0, st, 1u, a);
}

cudaError_t launch_moe_act_mx(const void *y13, int64_t ldy, int y_dtype, const int32_t *pair_slot, int P, int inter,
                              uint8_t *codes, int64_t ldc, uint8_t *scales, int64_t lds, cudaStream_t st) {
  const ActArgs a{y13, ldy, pair_slot, codes, ldc, scales, lds, P, inter};
  const RowGrid l = RowGrid::of(P, inter / 8, kThreads, kActRows);
  return launch_pdl(y_dtype == LORA_BF16 ? moe_act_mx_kernel<__nv_bfloat16> : moe_act_mx_kernel<float>, l.grid, l.block,
                    0, st, 1u, a);
}

cudaError_t launch_moe_combine(const void *y, int64_t ldy, int y_dtype, const float *w, const int32_t *pair_slot, int T,
                               int topk, int n, void *out, int64_t ldo, int out_dtype, int accumulate,
                               cudaStream_t st) {
  const CombineArgs a{y, ldy, w, pair_slot, out, ldo, T, topk, n, accumulate};
  RowGrid l = RowGrid::of(T, n / 8, kCombineThreads, 1);
  if (T >= 152 * 8) l.grid.x = 1;
  void (*k)(CombineArgs) = y_dtype == LORA_BF16
                               ? (out_dtype == LORA_BF16 ? moe_combine_kernel<__nv_bfloat16, __nv_bfloat16>
                                                         : moe_combine_kernel<__nv_bfloat16, float>)
                               : (out_dtype == LORA_BF16 ? moe_combine_kernel<float, __nv_bfloat16>
                                                         : moe_combine_kernel<float, float>);
  return launch_pdl(k, l.grid, l.block, 0, st, 1u, a);
}

}  // namespace ra
