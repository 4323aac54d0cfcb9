// Rows to the microscaled 4-bit format and back (lora_mx_quantize,
// lora_mx_dequantize). Both are bound by memory: a bf16 row is read once and
// 17/32 byte an element written, or the reverse. Four neighbouring lanes hold
// one block of 32, eight elements (one or two 16-byte loads) each, so a warp
// reads whole lines and the block's largest magnitude is two shuffles away.
#include "mx.cuh"

namespace ra {
namespace {

constexpr int kThreads = 128;  // 8191 rows of 7168 in bf16, there and back: 53.0 us (256: 58.5, 64: 60.6)
// Rows a thread takes at once: four (their loads are in flight together) once
// that leaves every SM two full sets of threads. The same rows with CTAs of 256
// threads: 58.5 us, with two rows 66.1 us, with one 83.1 us; eight are no gain.
bool four_rows(int64_t rows, int chunks) { return rows * chunks >= (int64_t)152 * 2048 * 2 * 4; }

template <typename T, int R>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const T *x, int64_t ldx, uint8_t *codes, int64_t ldc,
                                                               uint8_t *scales, int64_t lds, int64_t rows, int chunks) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)gridDim.y * blockDim.y * R;
  for (int64_t r0 = (int64_t)blockIdx.y * blockDim.y * R; r0 < rows; r0 += step) {
    // Chunks come in fours (a row is whole blocks), so the four lanes of a
    // block are in range together; the others take part in the shuffles only.
    Raw8<T> raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + i * blockDim.y + threadIdx.y;
      raw[i] = Raw8<T>{};
      if (r < rows && c < chunks) raw[i] = raw8(x + r * ldx + (int64_t)c * 8);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + i * blockDim.y + threadIdx.y;
      float v[8];
      widen8(raw[i], v);
      uint32_t byte;
      const uint32_t q = mx_quantize8(v, byte);
      if (r < rows && c < chunks) {
        *reinterpret_cast<uint32_t *>(codes + r * ldc + (int64_t)c * 4) = q;
        if ((c & 3) == 0) scales[r * lds + (c >> 2)] = (uint8_t)byte;
      }
    }
  }
}

template <typename T, int R>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const uint8_t *codes, int64_t ldc,
                                                                 const uint8_t *scales, int64_t lds, T *y, int64_t ldy,
                                                                 int64_t rows, int chunks) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= chunks) return;
  const int64_t step = (int64_t)gridDim.y * blockDim.y * R;
  for (int64_t r0 = (int64_t)blockIdx.y * blockDim.y * R + threadIdx.y; r0 < rows; r0 += step) {
    uint32_t q[R], b[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = min(r0 + i * (int64_t)blockDim.y, rows - 1);
      q[i] = __ldg(reinterpret_cast<const uint32_t *>(codes + r * ldc + (int64_t)c * 4));
      b[i] = __ldg(scales + r * lds + (c >> 2));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + i * blockDim.y;
      if (r >= rows) break;
      const float s = mx_scale(b[i]);
      float v[8];
      mx_decode8(q[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
      store8(y + r * ldy + (int64_t)c * 8, v);
    }
  }
}

// One thread a word of four scales of a tile.
__global__ void __launch_bounds__(kThreads) mx_tile_scales_kernel(const uint8_t *scales, int64_t lds, int d_out, int nb,
                                                                  int t_out, int t_in, uint32_t *tiles, int64_t words) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += (int64_t)gridDim.x * kThreads) {
    const int in_tile = (int)(i & 127), r = (in_tile >> 2) + 32 * (in_tile & 3);
    const int64_t tile = i >> 7;
    const int ti = (int)(tile % t_in);
    const int64_t eo = tile / t_in, e = eo / t_out;
    const int64_t row = (eo - e * t_out) * kMxTile + r;
    uint32_t w = 0x7f7f7f7fu;
    if (row < d_out) {
      const uint8_t *p = scales + (e * d_out + row) * lds;
      w = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) w |= (uint32_t)(4 * ti + b < nb ? p[4 * ti + b] : 127) << (8 * b);
    }
    tiles[i] = w;
  }
}

template <typename T>
cudaError_t quantize(const void *x, int64_t ldx, int64_t rows, int chunks, uint8_t *codes, int64_t ldc, uint8_t *scales,
                     int64_t lds, cudaStream_t st) {
  const bool four = four_rows(rows, chunks);
  const RowGrid l = RowGrid::of(rows, chunks, kThreads, four ? 4 : 1);
  return launch_pdl(four ? mx_quantize_kernel<T, 4> : mx_quantize_kernel<T, 1>, l.grid, l.block, 0, st, 1u,
                    static_cast<const T *>(x), ldx, codes, ldc, scales, lds, rows, chunks);
}
template <typename T>
cudaError_t dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds, int64_t rows, int chunks,
                       void *y, int64_t ldy, cudaStream_t st) {
  const bool four = four_rows(rows, chunks);
  const RowGrid l = RowGrid::of(rows, chunks, kThreads, four ? 4 : 1);
  return launch_pdl(four ? mx_dequantize_kernel<T, 4> : mx_dequantize_kernel<T, 1>, l.grid, l.block, 0, st, 1u, codes,
                    ldc, scales, lds, static_cast<T *>(y), ldy, rows, chunks);
}

}  // namespace

cudaError_t launch_mx_tile_scales(const uint8_t *scales, int64_t lds, int experts, int d_out, int d_in, uint8_t *tiles,
                                  cudaStream_t st) {
  const int64_t words = (int64_t)experts * mx_tiles_out(d_out) * mx_tiles_in(d_in) * (kMxTileBytes / 4);
  const unsigned grid = (unsigned)std::min<int64_t>((words + kThreads - 1) / kThreads, 152 * 16);
  return launch_pdl(mx_tile_scales_kernel, dim3(grid), dim3(kThreads), 0, st, 1u, scales, lds, d_out, d_in / kMxBlock,
                    mx_tiles_out(d_out), mx_tiles_in(d_in), reinterpret_cast<uint32_t *>(tiles), words);
}

cudaError_t launch_mx_quantize(const void *x, int64_t ldx, int x_dtype, int64_t rows, int cols, uint8_t *codes,
                               int64_t ldc, uint8_t *scales, int64_t lds, cudaStream_t st) {
  return x_dtype == LORA_BF16 ? quantize<__nv_bfloat16>(x, ldx, rows, cols / 8, codes, ldc, scales, lds, st)
                              : quantize<float>(x, ldx, rows, cols / 8, codes, ldc, scales, lds, st);
}

cudaError_t launch_mx_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds, int64_t rows,
                                 int cols, void *y, int64_t ldy, int y_dtype, cudaStream_t st) {
  return y_dtype == LORA_BF16 ? dequantize<__nv_bfloat16>(codes, ldc, scales, lds, rows, cols / 8, y, ldy, st)
                              : dequantize<float>(codes, ldc, scales, lds, rows, cols / 8, y, ldy, st);
}

}  // namespace ra
