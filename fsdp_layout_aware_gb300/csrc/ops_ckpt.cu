// 8-bit activation checkpoints: store and load (include/tide_ops.h).
//
// Both directions are one pass over the matrix, a few operations per element,
// so they are bound by memory traffic: store reads s bytes and writes 1 + 1/32
// per element, load reads 1 + 1/32 (and s for a gradient) and writes s.
//   8192 x 13824 bf16 (343 MB each way): store 57 us, load 50 us, 6.0 and 6.8 TB/s
// Rows of odd alignment and the costlier activations are bound by issuing
// instructions instead:
//   4093 x 4095 bf16 times a gradient through SiLU' (84 MB): 17 us, 4.8 TB/s; 30
//   instructions a value keep 79% of the issue slots busy, and DRAM 33%
//   8192 x 13824 bf16 through GELU 65 us, its erf form 97 us

#include <algorithm>

#include "ops_common.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;

struct StoreArgs {
  uint32_t items;   // units of work (store_vec: 8 columns, store_any: 256) in this launch
  FastDiv per_row;  // of them in a row
  int64_t cols;
  const void* x;
  int64_t ldx;
  uint8_t* codes;
  int64_t ldc;
  uint8_t* scales;
  int64_t lds;
};

struct LoadArgs {
  uint32_t items;
  FastDiv per_row;
  int64_t cols;
  const uint8_t* codes;
  int64_t ldc;
  const uint8_t* scales;
  int64_t lds;
  const void* grad;
  int64_t ldg;
  void* out;
  int64_t ldo;
};

// Aligned rows: a thread owns eight neighbouring columns, four neighbouring
// lanes a block of 32, whose largest magnitude takes two shuffles.  kItems such
// groups a thread, all loads first, keep enough bytes in flight.  Rows start
// on 16-byte boundaries (x) and 8-byte ones (codes).
constexpr int kItems = 4;

template <typename T>
__global__ void __launch_bounds__(kThreads) store_vec_kernel(const StoreArgs a) {
  float v[kItems][8];
  int64_t row[kItems], col[kItems];
  bool here[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const uint32_t i = (blockIdx.x * kItems + j) * kThreads + threadIdx.x;
    const uint32_t r = a.per_row.quotient(i);
    row[j] = r;
    col[j] = (int64_t)(i - r * a.per_row.d) * 8;
    here[j] = i < a.items && col[j] < a.cols;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] = 0.0f;
    if (here[j]) load_vec<8>((const T*)a.x + row[j] * a.ldx + col[j], v[j]);
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const int byte = scale_byte(block_magnitude<4>(v[j]));
    uint32_t w[2];
    encode(v[j], byte, w);
    if (!here[j]) continue;
    *reinterpret_cast<uint2*>(a.codes + row[j] * a.ldc + col[j]) = make_uint2(w[0], w[1]);
    if (col[j] % kMxBlock == 0) a.scales[row[j] * a.lds + col[j] / kMxBlock] = (uint8_t)byte;
  }
}

// Any alignment: a warp takes 256 columns of a row, a lane eight of them as
// above.
template <typename T>
__global__ void __launch_bounds__(kThreads) store_any_kernel(const StoreArgs a) {
  const uint32_t i = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (i >= a.items) return;
  const int lane = threadIdx.x % 32;
  const int64_t row = a.per_row.quotient(i);
  const int64_t col = (int64_t)(i - (uint32_t)row * a.per_row.d) * 256 + lane * 8;
  const int n = (int)max((int64_t)0, min((int64_t)8, a.cols - col));  // columns that exist
  float v[8];
  load_any8((const T*)a.x + row * a.ldx + col, n, v);
  const int byte = scale_byte(block_magnitude<4>(v));
  uint32_t w[2];
  encode(v, byte, w);
  if (n > 0 && lane % 4 == 0) a.scales[row * a.lds + col / kMxBlock] = (uint8_t)byte;
  store_codes_any(a.codes + row * a.ldc + col, n, w);
}

// f(v), or g * f'(v).  fp32 outputs take the accurate exponential and division.
template <typename T, bool GRAD, int ACT, int N>
__device__ __forceinline__ void loaded(float (&v)[N], const float (&g)[N]) {
  constexpr bool fast = sizeof(T) == 2;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if constexpr (GRAD)
      v[k] = ACT == TIDE_ACT_NONE ? g[k] : g[k] * act_grad<fast>(ACT, v[k]);
    else
      v[k] = act_value<fast>(ACT, v[k]);
  }
}

// Eight neighbouring columns a thread and item; rows on 16-byte (out, grad)
// and 8-byte (codes) boundaries.
// Registers are bounded, to what bf16 asks for: one more than 48 cost a block an SM
// (58 us became 60).  fp32's erf form alone keeps 4 bytes of a thread in memory for it.
template <typename T, bool GRAD, int ACT>
__global__ void __launch_bounds__(kThreads, GRAD ? 3 : 5) load_vec_kernel(const LoadArgs a) {
  uint2 c[kItems];
  uint8_t s[kItems];
  float g[kItems][8];
  int64_t row[kItems], col[kItems];
  bool here[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const uint32_t i = (blockIdx.x * kItems + j) * kThreads + threadIdx.x;
    const uint32_t r = a.per_row.quotient(i);
    row[j] = r;
    here[j] = i < a.items;
    col[j] = (int64_t)(i - r * a.per_row.d) * 8;
    if (here[j]) {
      c[j] = *reinterpret_cast<const uint2*>(a.codes + row[j] * a.ldc + col[j]);
      s[j] = a.scales[row[j] * a.lds + col[j] / kMxBlock];
      if (GRAD) load_vec<8>((const T*)a.grad + row[j] * a.ldg + col[j], g[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    if (!here[j]) continue;
    float v[8];
    decode8(c[j], scale_value(s[j]), v);
    loaded<T, GRAD, ACT>(v, g[j]);
    store_vec<8>((T*)a.out + row[j] * a.ldo + col[j], v);
  }
}

// Any alignment: a thread takes the eight columns of an aligned word of out
// (the row's first and last words may be partial), so that out is stored whole,
// and grad read whole where it lies as out does.  Full occupancy pays: 34 registers
// instead of 32 cost 7% (the SiLU' case above).
template <typename T, bool GRAD, int ACT>
__global__ void __launch_bounds__(kThreads, GRAD && sizeof(T) == 4 ? 6 : 8) load_any_kernel(const LoadArgs a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.items) return;
  const int64_t row = a.per_row.quotient(i);
  T* out = (T*)a.out + row * a.ldo;
  const int phase = (int)((uintptr_t)out % 16 / sizeof(T));
  const int64_t col = (int64_t)(i - (uint32_t)row * a.per_row.d) * 8 - phase;
  if (col >= a.cols) return;
  const uint8_t* codes = a.codes + row * a.ldc;
  const uint8_t* scales = a.scales + row * a.lds;
  const T* grad = GRAD ? (const T*)a.grad + row * a.ldg : nullptr;
  float v[8], g[8] = {};
  if (col >= 0 && col + 8 <= a.cols) {
    const uint2 c = load_any_bytes(codes + col);
    const float s0 = scale_value(scales[col / kMxBlock]), s1 = scale_value(scales[(col + 7) / kMxBlock]);
    const int first = kMxBlock - (int)(col % kMxBlock);  // columns of the first block
    if (GRAD) load_any8(grad + col, 8, g);
    decode8(c, 1.0f, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= k < first ? s0 : s1;
    loaded<T, GRAD, ACT>(v, g);
    store_vec<8>(out + col, v);
  } else {
    for (int64_t k = max(col, (int64_t)0); k < min(col + 8, a.cols); ++k) {
      float t[1] = {e4m3_values(codes[k]).x * scale_value(scales[k / kMxBlock])}, u[1] = {0.0f};
      if (GRAD) load_vec<1>(grad + k, u);
      loaded<T, GRAD, ACT>(t, u);
      store_vec<1>(out + k, t);
    }
  }
}

// Calls launch(first row, rows, items, grid) until every row is done: a launch
// has fewer than 2^31 items (per_row in a row, per_block in a block).
template <typename F>
tide_status in_launches(int64_t rows, int64_t per_row, int per_block, F&& launch) {
  const int64_t most = ((int64_t)1 << 31) - 65536;
  if (per_row > most || rows > ((int64_t)1 << 42) / per_row) return fail(TIDE_ERR_UNIMPLEMENTED, "matrix has more elements than any GPU holds");
  const int64_t step = most / per_row;
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t n = std::min(step, rows - r), items = n * per_row;
    launch(r, (uint32_t)items, (unsigned)((items + per_block - 1) / per_block));
    TIDE_TRY(cuda_status(cudaGetLastError(), "checkpoint"));
  }
  return TIDE_OK;
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <typename T>
tide_status store(int64_t rows, int64_t cols, const void* x, int64_t ldx, uint8_t* codes, int64_t ldc, uint8_t* scales,
                  int64_t lds, cudaStream_t stream) {
  const int64_t blocks = div_up(cols, kMxBlock);
  const bool vec = cols % 8 == 0 && rows_aligned(x, ldx, sizeof(T), rows) && (uintptr_t)codes % 8 == 0 &&
                   (rows <= 1 || ldc % 8 == 0);
  const int64_t per_row = vec ? blocks * 4 : div_up(cols, 256);
  return in_launches(rows, per_row, vec ? kThreads * kItems : kThreads / 32, [&](int64_t r, uint32_t items, unsigned grid) {
    const StoreArgs a{items, FastDiv((uint32_t)per_row), cols, (const T*)x + r * ldx, ldx, codes + r * ldc, ldc,
                      scales + r * lds, lds};
    if (vec)
      store_vec_kernel<T><<<grid, kThreads, 0, stream>>>(a);
    else
      store_any_kernel<T><<<grid, kThreads, 0, stream>>>(a);
  });
}

template <typename T, bool GRAD, int ACT>
tide_status load_act(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                     const void* grad, int64_t ldg, void* out, int64_t ldo, cudaStream_t stream) {
  const bool vec = cols % 8 == 0 && rows_aligned(grad, ldg, sizeof(T), rows) &&
                   rows_aligned(out, ldo, sizeof(T), rows) && (uintptr_t)codes % 8 == 0 && (rows <= 1 || ldc % 8 == 0);
  const int64_t per_row = vec ? cols / 8 : (cols + 14) / 8;  // words that any phase of a row touches
  return in_launches(rows, per_row, vec ? kThreads * kItems : kThreads, [&](int64_t r, uint32_t items, unsigned grid) {
    const LoadArgs a{items, FastDiv((uint32_t)per_row), cols, codes + r * ldc, ldc, scales + r * lds, lds,
                     GRAD ? (const T*)grad + r * ldg : nullptr, ldg, (T*)out + r * ldo, ldo};
    if (vec)
      load_vec_kernel<T, GRAD, ACT><<<grid, kThreads, 0, stream>>>(a);
    else
      load_any_kernel<T, GRAD, ACT><<<grid, kThreads, 0, stream>>>(a);
  });
}

template <typename T>
tide_status load(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                 int32_t act, const void* grad, int64_t ldg, void* out, int64_t ldo, cudaStream_t stream) {
  return with_act(act, [&](auto a) {
    return grad ? load_act<T, true, a.value>(rows, cols, codes, ldc, scales, lds, grad, ldg, out, ldo, stream)
                : load_act<T, false, a.value>(rows, cols, codes, ldc, scales, lds, nullptr, 0, out, ldo, stream);
  });
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
