// Attention on the CUDA cores (fp32, and bf16 heads of other sizes than the
// tensor-core kernel takes), and the joining of partial results for both.
//
// A CTA takes a unit of one key-value head: 32 rows at a time, 4 a warp, over
// tiles of 32 keys that all its rows share in shared memory. A lane is a key for
// the scores (rows' maxima and sums by shuffles) and an element of the head for
// the outputs, with the softmax's running maximum and sum in between. What
// bounds it is shared memory, read 16 bytes at a time: a lane's part of a key
// serves 4 rows' products (six fp32 prompts of 1 to 37 tokens 6.9 us, 18.4 with 4-byte
// reads).
#include "attn.cuh"
#include "tcgen05.cuh"

namespace ra {
namespace {

constexpr int kWarps = 8, kWarpRows = 4, kRows = kWarps * kWarpRows, kKeys = 32;

template <typename T, int N>  // N: 32-element steps of a head
struct RowsSmem {
  static constexpr int kD = 32 * N;
  float k[kKeys][kD + 4], v[kKeys][kD], q[kRows][kD], p[kWarps][kKeys][kWarpRows];
};

// Keys [j0, j0 + 32) of the unit's sequence and head to shared memory as fp32; zeros past n keys and past the head.
template <typename T, int N>
__device__ __forceinline__ void load_keys(RowsSmem<T, N> &sm, const AttnArgs &a, const AttnUnit &u, int head, int j0, int n) {
  constexpr int kVec = Elem<T>::kVec, kSteps = 32 * N / kVec;
  const int steps = a.s.D / kVec;
  for (int i = threadIdx.x; i < kKeys * kSteps; i += 32 * kWarps) {
    const int r = i / kSteps, c = i % kSteps, j = j0 + r;
    float k[kVec] = {}, v[kVec] = {};
    if (j < n && c < steps) {
      int64_t ko = -1, vo = -1;
      if (a.kv.page_size > 0) {
        const int page = a.kv.table[(int64_t)u.seq * a.kv.ld_table + (j >> a.kv.log2_page)];
        const int64_t in_page = j & (a.kv.page_size - 1);
        if ((unsigned)page < (unsigned)a.kv.num_pages) {
          ko = page * a.kv.k_page + in_page * a.kv.k_row;
          vo = page * a.kv.v_page + in_page * a.kv.v_row;
        } else {
          atomicOr(a.err, kErrBadPage);
        }
      } else {
        const int64_t row = (int64_t)u.row0 - u.pos0 + j;
        if (row >= 0 && row < a.num_tokens) {
          ko = row * a.kv.k_row;
          vo = row * a.kv.v_row;
        }
      }
      if (ko >= 0) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.kv.k) + ko + head * a.kv.k_head) + c);
        const uint4 y = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.kv.v) + vo + head * a.kv.v_head) + c);
        const T *xt = reinterpret_cast<const T *>(&x), *yt = reinterpret_cast<const T *>(&y);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          k[e] = Elem<T>::to_f(xt[e]);
          v[e] = Elem<T>::to_f(yt[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kVec; e += 4) {
      *reinterpret_cast<float4 *>(&sm.k[r][c * kVec + e]) = make_float4(k[e], k[e + 1], k[e + 2], k[e + 3]);
      *reinterpret_cast<float4 *>(&sm.v[r][c * kVec + e]) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    }
  }
}

template <typename T, int N>
__global__ void __launch_bounds__(32 * kWarps) attn_rows_kernel(const AttnArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  RowsSmem<T, N> &sm = *reinterpret_cast<RowsSmem<T, N> *>(raw);
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t items = (int64_t)a.plan[AttnPlan::kUnits] * a.s.Hkv;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int head = (int)(it % a.s.Hkv);
    AttnUnit u;
    const int4 *up = reinterpret_cast<const int4 *>(a.plan + a.p.units() + AttnPlan::kUnit * (it / a.s.Hkv));
    reinterpret_cast<int4 *>(&u)[0] = up[0];
    reinterpret_cast<int4 *>(&u)[1] = up[1];
    const int rows = u.tokens * a.s.G;
    for (int r0 = 0; r0 < rows; r0 += kRows) {
      __syncthreads();
      for (int i = threadIdx.x; i < kRows * 4 * N; i += 32 * kWarps) {  // eight elements of a row
        const int r = i / (4 * N), d = i % (4 * N) * 8, row = r0 + r;
        float x[8] = {};
        if (row < rows && d < a.s.D)
          load8_f32(static_cast<const T *>(a.q) + (int64_t)(u.row0 + row / a.s.G) * a.ldq +
                        (int64_t)(head * a.s.G + row % a.s.G) * a.s.D + d, x);
        store8(&sm.q[r][d], x);
      }
      float m[kWarpRows], l[kWarpRows], o[kWarpRows][N];
      int lim[kWarpRows], first = INT32_MAX, most = 0;
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) o[r][i] = 0.f;
        const int row = r0 + warp * kWarpRows + r;
        lim[r] = row < rows ? visible_keys(u.pos0 + row / a.s.G, u.kv_len, a.s.causal) : 0;
        first = min(first, lim[r]);
        most = max(most, lim[r]);
      }
      const int last = min(rows, r0 + kRows) - 1;  // the row of this pass that sees most
      const int end = min(u.kb1 * kKeyBlock, visible_keys(u.pos0 + last / a.s.G, u.kv_len, a.s.causal));
      for (int j0 = u.kb0 * kKeyBlock; j0 < end; j0 += kKeys) {
        __syncthreads();
        load_keys<T, N>(sm, a, u, head, j0, u.kv_len);
        __syncthreads();
        if (j0 >= most) continue;
        float s[kWarpRows] = {};
#pragma unroll 4
        for (int d = 0; d < 32 * N; d += 4) {
          const float4 k = *reinterpret_cast<const float4 *>(&sm.k[lane][d]);
#pragma unroll
          for (int r = 0; r < kWarpRows; ++r) {
            const float4 q = *reinterpret_cast<const float4 *>(&sm.q[warp * kWarpRows + r][d]);
            s[r] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, s[r]))));
          }
        }
#pragma unroll
        for (int r = 0; r < kWarpRows; ++r) {
          const bool sees = j0 + lane < lim[r];
          float top = sees ? s[r] : -INFINITY;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float mn = fmaxf(m[r], top), base = mn == -INFINITY ? 0.f : mn * a.s.scale_log2;
          const float old = exp2f(m[r] * a.s.scale_log2 - base);
          const float p = sees ? exp2f(fmaf(s[r], a.s.scale_log2, -base)) : 0.f;
          float sum = p;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          l[r] = l[r] * old + sum;
          m[r] = mn;
          s[r] = p;
#pragma unroll
          for (int i = 0; i < N; ++i) o[r][i] *= old;
        }
        *reinterpret_cast<float4 *>(sm.p[warp][lane]) = make_float4(s[0], s[1], s[2], s[3]);
        __syncwarp();
        // Rows that do not see key j0 + j take nothing of it, whatever its value.
#pragma unroll 4
        for (int j = 0; j < kKeys; ++j) {
          if (j0 + j >= most) break;
          const float4 p4 = *reinterpret_cast<const float4 *>(sm.p[warp][j]);
          const float p[kWarpRows] = {p4.x, p4.y, p4.z, p4.w};
          float v[N];
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] = sm.v[j][32 * i + lane];
          if (j0 + j < first) {
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r) {
#pragma unroll
              for (int i = 0; i < N; ++i) o[r][i] = fmaf(p[r], v[i], o[r][i]);
            }
          } else {
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r) {
              if (j0 + j < lim[r]) {
#pragma unroll
                for (int i = 0; i < N; ++i) o[r][i] = fmaf(p[r], v[i], o[r][i]);
              }
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kWarpRows; ++r) {
        const int row = r0 + warp * kWarpRows + r;
        if (row >= rows) break;
        if (u.slot >= 0) {
          float *part = a.ws + ((int64_t)u.slot * a.s.Hkv + head) * slot_floats(a.s);
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (32 * i + lane < a.s.D) part[(int64_t)row * a.s.D + 32 * i + lane] = o[r][i];
          if (lane < 2) part[(int64_t)a.s.slot_rows * a.s.D + 2 * row + lane] = lane == 0 ? m[r] * a.s.scale_log2 : l[r];
          continue;
        }
        const int64_t t = u.row0 + row / a.s.G;
        const int h = head * a.s.G + row % a.s.G;
        const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
        T *out = static_cast<T *>(a.out) + t * a.ldo + (int64_t)h * a.s.D;
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (32 * i + lane < a.s.D) out[32 * i + lane] = Elem<T>::from_f(o[r][i] * inv);
        if (a.lse != nullptr && lane == 0)
          a.lse[t * a.s.Hq + h] = l[r] == 0.f ? -INFINITY : 0.6931471805599453f * (m[r] * a.s.scale_log2 + log2f(l[r]));
      }
    }
  }
}

// ------------------------------------------------------------------ joining

constexpr int kJoinWarps = 8;

// A warp a row: the pieces' maxima and sums by lanes, then their outputs one after another, in the order of the keys.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_combine_kernel(const AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int steps = (a.s.slot_rows + kJoinWarps - 1) / kJoinWarps;
  const int64_t pitch = slot_floats(a.s) * a.s.Hkv;  // from one piece to the next
  // The first group's record is asked for with the number of groups, a row's first outputs with its statistics: three
  // round trips to memory instead of five.
  auto group_at = [&](int i) {
    return *reinterpret_cast<const int4 *>(a.plan + a.p.groups() +
                                           (int64_t)AttnPlan::kGroup * min(i / steps / a.s.Hkv, a.p.max_groups - 1));
  };
  int4 g = group_at(blockIdx.x);
  const int n = a.plan[AttnPlan::kGroups] * a.s.Hkv * steps;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    if (i != blockIdx.x) g = group_at(i);
    const int step = i % steps, head = i / steps % a.s.Hkv;
    const int row = step * kJoinWarps + warp;
    if (row >= g.y * a.s.G) continue;
    const float *part = a.ws + ((int64_t)g.z * a.s.Hkv + head) * slot_floats(a.s);
    const float *stats = part + (int64_t)a.s.slot_rows * a.s.D + 2 * row;
    const float *first = part + (int64_t)row * a.s.D + lane;
    constexpr int kAhead = 4;  // pieces whose first 128 elements are in flight with the statistics
    float ahead[kAhead][4];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) ahead[k][e] = k < g.w && 32 * e + lane < a.s.D ? first[k * pitch + 32 * e] : 0.f;
    float2 mine = lane < g.w ? *reinterpret_cast<const float2 *>(stats + lane * pitch) : make_float2(-INFINITY, 0.f);
    float m = mine.x;
    for (int j = lane + 32; j < g.w; j += 32) m = fmaxf(m, stats[j * pitch]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float base = m == -INFINITY ? 0.f : m;
    float acc[8] = {}, l = 0.f;
    for (int j0 = 0; j0 < g.w; j0 += 32) {
      const int j = j0 + lane;
      if (j0 > 0) mine = j < g.w ? *reinterpret_cast<const float2 *>(stats + j * pitch) : make_float2(-INFINITY, 0.f);
      const float w = exp2f(mine.x - base);
      float lw = w * mine.y;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, x);
      l += lw;
      const int here = min(32, g.w - j0);
      if (j0 == 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, k);
          if (k < here) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(wk, ahead[k][e], acc[e]);
#pragma unroll
            for (int e = 4; e < 8; ++e)
              if (32 * e + lane < a.s.D) acc[e] = fmaf(wk, first[k * pitch + 32 * e], acc[e]);
          }
        }
      }
#pragma unroll 4
      for (int k = j0 == 0 ? kAhead : 0; k < here; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const float *o = first + (j0 + k) * pitch;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (32 * e + lane < a.s.D) acc[e] = fmaf(wk, o[32 * e], acc[e]);
      }
    }
    const int64_t t = g.x + row / a.s.G;
    const int h = head * a.s.G + row % a.s.G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T *out = static_cast<T *>(a.out) + t * a.ldo + (int64_t)h * a.s.D;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (32 * e + lane < a.s.D) out[32 * e + lane] = Elem<T>::from_f(acc[e] * inv);
    if (a.lse != nullptr && lane == 0)
      a.lse[t * a.s.Hq + h] = l == 0.f ? -INFINITY : 0.6931471805599453f * (base + log2f(l));
  }
}

template <typename T, int N>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t st) {
  constexpr int smem = (int)sizeof(RowsSmem<T, N>);
  const cudaError_t e = set_max_dynamic_smem((const void *)attn_rows_kernel<T, N>, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)a.p.max_units * a.s.Hkv;
  return launch_pdl(attn_rows_kernel<T, N>, dim3((unsigned)std::min<int64_t>(most, a.s.ctas)), dim3(32 * kWarps), smem, st, 1u, a);
}

template <typename T>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t st) {
  if (a.s.D <= 64) return launch_rows<T, 2>(a, st);
  if (a.s.D <= 128) return launch_rows<T, 4>(a, st);
  return launch_rows<T, 8>(a, st);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t st) {
  return a.s.dtype == LORA_BF16 ? launch_rows<__nv_bfloat16>(a, st) : launch_rows<float>(a, st);
}

cudaError_t launch_attn_combine(const AttnArgs &a, cudaStream_t st) {
  const int64_t most = (int64_t)a.s.max_slots / 2 * a.s.Hkv * ((a.s.slot_rows + kJoinWarps - 1) / kJoinWarps);
  const dim3 grid((unsigned)std::min<int64_t>(std::max<int64_t>(1, most), 2 * 152)), block(32 * kJoinWarps);
  return a.s.dtype == LORA_BF16 ? launch_pdl(attn_combine_kernel<__nv_bfloat16>, grid, block, 0, st, 1u, a)
                                : launch_pdl(attn_combine_kernel<float>, grid, block, 0, st, 1u, a);
}

}  // namespace ra
