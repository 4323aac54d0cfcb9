// Rows to the microscaled 4-bit format and back (lora_mx_quantize,
// lora_mx_dequantize). Both are bound by memory: a bf16 row is read once and
// 17/32 byte an element written, or the reverse. Four neighbouring lanes hold
// one block of 32, eight elements (one or two 16-byte loads) each, so a warp
// reads whole lines and the block's largest magnitude is two shuffles away.
#include "mx.cuh"

namespace ra {
namespace {

constexpr int kThreads = 256;

// Threads along a row (a power of two of at least 4) and rows a CTA, for rows
// of `chunks` eight-element chunks.
struct RowShape {
  int tx, ty;
};
RowShape row_shape(int chunks) {
  int tx = 4;
  while (tx < kThreads && tx < chunks) tx *= 2;
  return {tx, kThreads / tx};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx_quantize_kernel(const T *x, int64_t ldx, uint8_t *codes, int64_t ldc,
                                                               uint8_t *scales, int64_t lds, int64_t rows, int chunks) {
  pdl_wait();
  pdl_trigger();
  const int nx = blockDim.x;
  for (int64_t r0 = (int64_t)blockIdx.y * blockDim.y; r0 < rows; r0 += (int64_t)gridDim.y * blockDim.y) {
    const int64_t r = r0 + threadIdx.y;
    // Chunks come in fours (a row is whole blocks), so the four lanes of a
    // block are in range together; the others take part in the shuffles only.
    const int c = blockIdx.x * nx + threadIdx.x;
    const bool in = r < rows && c < chunks;
    float v[8] = {};
    if (in) load8_f32(x + r * ldx + (int64_t)c * 8, v);
    uint32_t byte;
    const uint32_t q = mx_quantize8(v, byte);
    if (in) {
      *reinterpret_cast<uint32_t *>(codes + r * ldc + (int64_t)c * 4) = q;
      if ((c & 3) == 0) scales[r * lds + (c >> 2)] = (uint8_t)byte;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) mx_dequantize_kernel(const uint8_t *codes, int64_t ldc,
                                                                 const uint8_t *scales, int64_t lds, T *y, int64_t ldy,
                                                                 int64_t rows, int chunks) {
  pdl_wait();
  pdl_trigger();
  const int nx = blockDim.x;
  for (int64_t r = (int64_t)blockIdx.y * blockDim.y + threadIdx.y; r < rows; r += (int64_t)gridDim.y * blockDim.y) {
    const int c = blockIdx.x * nx + threadIdx.x;
    if (c >= chunks) continue;
    const uint32_t q = *reinterpret_cast<const uint32_t *>(codes + r * ldc + (int64_t)c * 4);
    const float s = mx_scale(scales[r * lds + (c >> 2)]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mx_decode(q >> (4 * i) & 15u) * s;
    store8(y + r * ldy + (int64_t)c * 8, v);
  }
}

struct Launch {
  dim3 grid, block;
};
Launch shape_of(int64_t rows, int chunks) {
  const RowShape s = row_shape(chunks);
  const int64_t by = (rows + s.ty - 1) / s.ty;
  return {dim3((unsigned)((chunks + s.tx - 1) / s.tx), (unsigned)std::min<int64_t>(by, 65535)),
          dim3((unsigned)s.tx, (unsigned)s.ty)};
}

}  // namespace

cudaError_t launch_mx_quantize(const void *x, int64_t ldx, int x_dtype, int64_t rows, int cols, uint8_t *codes,
                               int64_t ldc, uint8_t *scales, int64_t lds, cudaStream_t st) {
  const Launch l = shape_of(rows, cols / 8);
  if (x_dtype == LORA_BF16)
    return launch_pdl(mx_quantize_kernel<__nv_bfloat16>, l.grid, l.block, 0, st, 1u,
                      static_cast<const __nv_bfloat16 *>(x), ldx, codes, ldc, scales, lds, rows, cols / 8);
  return launch_pdl(mx_quantize_kernel<float>, l.grid, l.block, 0, st, 1u, static_cast<const float *>(x), ldx, codes,
                    ldc, scales, lds, rows, cols / 8);
}

cudaError_t launch_mx_dequantize(const uint8_t *codes, int64_t ldc, const uint8_t *scales, int64_t lds, int64_t rows,
                                 int cols, void *y, int64_t ldy, int y_dtype, cudaStream_t st) {
  const Launch l = shape_of(rows, cols / 8);
  if (y_dtype == LORA_BF16)
    return launch_pdl(mx_dequantize_kernel<__nv_bfloat16>, l.grid, l.block, 0, st, 1u, codes, ldc, scales, lds,
                      static_cast<__nv_bfloat16 *>(y), ldy, rows, cols / 8);
  return launch_pdl(mx_dequantize_kernel<float>, l.grid, l.block, 0, st, 1u, codes, ldc, scales, lds,
                    static_cast<float *>(y), ldy, rows, cols / 8);
}

}  // namespace ra
