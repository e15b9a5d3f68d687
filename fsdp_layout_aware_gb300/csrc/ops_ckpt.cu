// 8-bit activation checkpoints: store and load (include/tide_ops.h).
//
// Both directions are one pass over the matrix, a few operations per element,
// so they are bound by memory traffic: store reads s bytes and writes 1 + 1/32
// per element, load reads 1 + 1/32 (and s for a gradient) and writes s.

#include "ops_common.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;

// A thread owns eight neighbouring columns, four neighbouring lanes a block of
// 32: the block's largest magnitude takes two shuffles.  Rows start on 16-byte
// boundaries (x) and 8-byte ones (codes).
template <typename T>
__global__ void __launch_bounds__(kThreads) store_vec_kernel(int64_t rows, int64_t cols, const T* __restrict__ x,
                                                             int64_t ldx, uint8_t* __restrict__ codes, int64_t ldc,
                                                             uint8_t* __restrict__ scales, int64_t lds) {
  const int64_t per_row = (cols + kMxBlock - 1) / kMxBlock * 4;  // threads a row
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = i / per_row;
  const int64_t col = (i - row * per_row) * 8;
  float v[8];
  float a = 0.0f;
  const bool here = row < rows && col < cols;
  if (here) {
    load_vec<8>(x + row * ldx + col, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[k] = finite_or_nan(v[k]);
      a = fmaxf(a, fabsf(v[k]));
    }
  }
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
  if (!here) return;
  const int byte = scale_byte(a);
  const float inv = scale_inverse(byte);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k / 2] |= e4m3_pair(clamp_top(v[2 * k] * inv, byte), clamp_top(v[2 * k + 1] * inv, byte)) << (16 * (k % 2));
  *reinterpret_cast<uint2*>(codes + row * ldc + col) = make_uint2(w[0], w[1]);
  if (col % kMxBlock == 0) scales[row * lds + col / kMxBlock] = (uint8_t)byte;
}

// Any alignment: a warp takes a block of 32 columns, one element a lane.
template <typename T>
__global__ void __launch_bounds__(kThreads) store_any_kernel(int64_t rows, int64_t cols, const T* __restrict__ x,
                                                             int64_t ldx, uint8_t* __restrict__ codes, int64_t ldc,
                                                             uint8_t* __restrict__ scales, int64_t lds) {
  const int64_t blocks = (cols + kMxBlock - 1) / kMxBlock;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32;
  const int64_t row = i / blocks;
  if (row >= rows) return;
  const int64_t b = i - row * blocks, col = b * kMxBlock + threadIdx.x % 32;
  float v[1] = {0.0f};
  if (col < cols) load_vec<1>(x + row * ldx + col, v);
  v[0] = finite_or_nan(v[0]);
  // Magnitudes order as their bits do.
  const uint32_t a = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fabsf(v[0]), 0.0f)));
  const int byte = scale_byte(__uint_as_float(a));
  if (col < cols)
    codes[row * ldc + col] = (uint8_t)e4m3_pair(clamp_top(v[0] * scale_inverse(byte), byte), 0.0f);
  if (threadIdx.x % 32 == 0) scales[row * lds + b] = (uint8_t)byte;
}

template <typename T>
__device__ __forceinline__ float loaded(float value, int act, bool has_grad, float grad) {
  constexpr bool fast = sizeof(T) == 2;
  return has_grad ? grad * act_grad<fast>(act, value) : act_value<fast>(act, value);
}

// Eight neighbouring columns a thread; rows on 16-byte (out, grad) and 8-byte
// (codes) boundaries.
template <typename T>
__global__ void __launch_bounds__(kThreads) load_vec_kernel(int64_t rows, int64_t cols,
                                                            const uint8_t* __restrict__ codes, int64_t ldc,
                                                            const uint8_t* __restrict__ scales, int64_t lds, int act,
                                                            const T* grad, int64_t ldg, T* out, int64_t ldo) {
  const int64_t per_row = cols / 8;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = i / per_row;
  if (row >= rows) return;
  const int64_t col = (i - row * per_row) * 8;
  const uint2 c = *reinterpret_cast<const uint2*>(codes + row * ldc + col);
  const float s = scale_value(scales[row * lds + col / kMxBlock]);
  float g[8] = {};
  if (grad) load_vec<8>(grad + row * ldg + col, g);
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = e4m3_values(((k < 2 ? c.x : c.y) >> (16 * (k % 2))) & 0xffffu);
    v[2 * k] = loaded<T>(t.x * s, act, grad != nullptr, g[2 * k]);
    v[2 * k + 1] = loaded<T>(t.y * s, act, grad != nullptr, g[2 * k + 1]);
  }
  store_vec<8>(out + row * ldo + col, v);
}

// Any alignment: neighbouring lanes on neighbouring elements.
template <typename T>
__global__ void __launch_bounds__(kThreads) load_any_kernel(int64_t rows, int64_t cols,
                                                            const uint8_t* __restrict__ codes, int64_t ldc,
                                                            const uint8_t* __restrict__ scales, int64_t lds, int act,
                                                            const T* grad, int64_t ldg, T* out, int64_t ldo) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = i / cols;
  if (row >= rows) return;
  const int64_t col = i - row * cols;
  const float value = e4m3_values(codes[row * ldc + col]).x * scale_value(scales[row * lds + col / kMxBlock]);
  float g[1] = {0.0f};
  if (grad) load_vec<1>(grad + row * ldg + col, g);
  const float v[1] = {loaded<T>(value, act, grad != nullptr, g[0])};
  store_vec<1>(out + row * ldo + col, v);
}

// Blocks for rows * per_row threads; UNIMPLEMENTED past the grid limit (over
// 1.7e10 blocks of 32).
tide_status grid_for(int64_t rows, int64_t per_row, unsigned int* grid) {
  if (rows > (int64_t)INT32_MAX * kThreads / per_row)
    return fail(TIDE_ERR_UNIMPLEMENTED, "matrix has too many elements for one launch");
  *grid = (unsigned int)((rows * per_row + kThreads - 1) / kThreads);
  return TIDE_OK;
}

template <typename T>
tide_status store(int64_t rows, int64_t cols, const void* x, int64_t ldx, uint8_t* codes, int64_t ldc, uint8_t* scales,
                  int64_t lds, cudaStream_t stream) {
  const int64_t blocks = (cols + kMxBlock - 1) / kMxBlock;
  const bool vec = cols % 8 == 0 && rows_aligned(x, ldx, sizeof(T), rows) && (uintptr_t)codes % 8 == 0 &&
                   (rows <= 1 || ldc % 8 == 0);
  unsigned int grid;
  TIDE_TRY(grid_for(rows, blocks * (vec ? 4 : 32), &grid));
  if (vec)
    store_vec_kernel<T><<<grid, kThreads, 0, stream>>>(rows, cols, (const T*)x, ldx, codes, ldc, scales, lds);
  else
    store_any_kernel<T><<<grid, kThreads, 0, stream>>>(rows, cols, (const T*)x, ldx, codes, ldc, scales, lds);
  return cuda_status(cudaGetLastError(), "checkpoint store");
}

template <typename T>
tide_status load(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                 int32_t act, const void* grad, int64_t ldg, void* out, int64_t ldo, cudaStream_t stream) {
  const bool vec = cols % 8 == 0 && rows_aligned(grad, ldg, sizeof(T), rows) &&
                   rows_aligned(out, ldo, sizeof(T), rows) && (uintptr_t)codes % 8 == 0 && (rows <= 1 || ldc % 8 == 0);
  unsigned int grid;
  TIDE_TRY(grid_for(rows, vec ? cols / 8 : cols, &grid));
  if (vec)
    load_vec_kernel<T><<<grid, kThreads, 0, stream>>>(rows, cols, codes, ldc, scales, lds, act, (const T*)grad, ldg,
                                                      (T*)out, ldo);
  else
    load_any_kernel<T><<<grid, kThreads, 0, stream>>>(rows, cols, codes, ldc, scales, lds, act, (const T*)grad, ldg,
                                                      (T*)out, ldo);
  return cuda_status(cudaGetLastError(), "checkpoint load");
}

}  // namespace

tide_status launch_checkpoint_load_bf16(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc,
                                        const uint8_t* scales, int64_t lds, int32_t act, void* out, int64_t ldo,
                                        cudaStream_t stream) {
  return load<bf16>(rows, cols, codes, ldc, scales, lds, act, nullptr, 0, out, ldo, stream);
}

}  // namespace tide

using namespace tide;

extern "C" {

tide_status tide_checkpoint_store(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx, uint8_t* codes,
                                  int64_t ld_codes, uint8_t* scales, int64_t ld_scales, void* stream) {
  clear_error();
  TIDE_TRY(check_sizes(rows, cols, "checkpoint"));
  TIDE_TRY(check_dtype(dtype));
  if (rows == 0 || cols == 0) return TIDE_OK;
  TIDE_TRY(check_matrix(x, rows, cols, ldx, elem_bytes_of(dtype), "x"));
  TIDE_TRY(check_checkpoint(codes, ld_codes, scales, ld_scales, rows, cols));
  return dtype == TIDE_BF16
             ? store<bf16>(rows, cols, x, ldx, codes, ld_codes, scales, ld_scales, (cudaStream_t)stream)
             : store<float>(rows, cols, x, ldx, codes, ld_codes, scales, ld_scales, (cudaStream_t)stream);
}

tide_status tide_checkpoint_load(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ld_codes,
                                 const uint8_t* scales, int64_t ld_scales, int32_t act, int32_t dtype, const void* grad,
                                 int64_t ld_grad, void* out, int64_t ld_out, void* stream) {
  clear_error();
  TIDE_TRY(check_sizes(rows, cols, "checkpoint"));
  TIDE_TRY(check_dtype(dtype));
  TIDE_TRY(check_act(act));
  if (rows == 0 || cols == 0) return TIDE_OK;
  TIDE_TRY(check_checkpoint(codes, ld_codes, scales, ld_scales, rows, cols));
  if (grad) TIDE_TRY(check_matrix(grad, rows, cols, ld_grad, elem_bytes_of(dtype), "grad"));
  TIDE_TRY(check_matrix(out, rows, cols, ld_out, elem_bytes_of(dtype), "out"));
  return dtype == TIDE_BF16 ? load<bf16>(rows, cols, codes, ld_codes, scales, ld_scales, act, grad, ld_grad, out,
                                         ld_out, (cudaStream_t)stream)
                            : load<float>(rows, cols, codes, ld_codes, scales, ld_scales, act, grad, ld_grad, out,
                                          ld_out, (cudaStream_t)stream);
}

}  // extern "C"
