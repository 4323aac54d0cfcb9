// The experts' own products (lora_moe_product): pairs grouped by local expert
// through the token metadata, y[p] = x[p / x_row_div] . W[slot p - 1]^T.
// fp32 weights (accuracy runs) go to a CUDA-core kernel, bf16 and 4-bit ones
// to the tensor cores (moe_product_tc.cu).
//
// CUDA-core kernel: 64 rows by 64 outputs a CTA, fp32 sums.
#include "common.cuh"

namespace ra {
namespace {

constexpr int kTile = 64;   // rows and outputs of a CTA
constexpr int kStep = 16;   // elements of d_in a step
constexpr int kThreads = 256;

struct ProductArgs {
  const float *x, *W;
  int64_t ldx, ldy;
  float *y;
  const int32_t *work, *sorted_rows;
  int num_slots, K, N, x_div;
};

__global__ void __launch_bounds__(kThreads) moe_product_kernel(ProductArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float xs[kStep][kTile + 4], ws[kStep][kTile + 4];
  __shared__ int rows_s[kTile];
  const int S = a.num_slots, n_list = a.work[0], n_tiles = a.work[3];
  const int32_t *ts = a.work + WorkLists::all_tile_start(S);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int n0 = blockIdx.x * kTile;
  constexpr int kHalves = LORA_SGMV_TILE_M / kTile;
  for (int it = blockIdx.y; it < n_tiles * kHalves; it += gridDim.y) {
    const int tile = it / kHalves;
    int lo = 0, hi = n_list - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (ts[mid] <= tile) lo = mid;
      else hi = mid - 1;
    }
    const int32_t *rec = a.work + WorkLists::list(S, kListAll) + lo * WorkLists::kRec;
    const int first = (tile - ts[lo]) * LORA_SGMV_TILE_M + it % kHalves * kTile;
    const int rows = min(kTile, rec[2] - first);
    if (rows <= 0) continue;
    const int64_t w0 = (int64_t)(rec[1] - 1) * a.N;
    __syncthreads();
    if (threadIdx.x < kTile) rows_s[threadIdx.x] = a.sorted_rows[rec[3] + first + min((int)threadIdx.x, rows - 1)];
    __syncthreads();
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += kStep) {
      for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
        const int r = i / kStep, k = i % kStep;
        const bool in = k0 + k < a.K;
        xs[k][r] = in ? a.x[(int64_t)(rows_s[r] / a.x_div) * a.ldx + k0 + k] : 0.f;
        ws[k][r] = in && n0 + r < a.N ? a.W[(w0 + n0 + r) * a.K + k0 + k] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[k][ty * 4 + i], ws[k][tx * 4 + j], acc[i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= rows) break;
      float *y = a.y + (int64_t)rows_s[r] * a.ldy;
      for (int j = 0; j < 4; ++j)
        if (n0 + tx * 4 + j < a.N) y[n0 + tx * 4 + j] = acc[i][j];
    }
  }
}

}  // namespace

cudaError_t launch_moe_product(const lora_expert_desc &d, const MetaView &mv, const void *x, int64_t ldx,
                               const uint8_t *x_scale, int64_t ld_xs, void *y, int64_t ldy, int y_dtype,
                               cudaStream_t st) {
  const int64_t tiles = (int64_t)mv.num_tokens / LORA_SGMV_TILE_M + std::min(mv.num_slots - 1, mv.num_tokens);
  if (tiles == 0) return cudaSuccess;
  if (d.dtype != LORA_F32) return launch_moe_product_tc(d, mv, x, ldx, x_scale, ld_xs, y, ldy, y_dtype, st);
  const ProductArgs a{static_cast<const float *>(x), static_cast<const float *>(d.W), ldx, ldy, static_cast<float *>(y),
                      mv.work, mv.sorted_rows, mv.num_slots, d.d_in, d.d_out, std::max(1, d.x_row_div)};
  const dim3 grid((unsigned)((d.d_out + kTile - 1) / kTile),
                  (unsigned)std::min<int64_t>(tiles * (LORA_SGMV_TILE_M / kTile), 1024));
  return launch_pdl(moe_product_kernel, grid, dim3(kThreads), 0, st, 1u, a);
}

}  // namespace ra
