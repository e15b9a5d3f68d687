// RMS norm with the residual's addition, forward and backward
// (include/tide_ops.h).
//
// Both directions read each input and write each output once, with about ten
// operations per element, so they are bound by memory traffic; a row stays in
// registers between its sum and its outputs.

#include <algorithm>
#include <type_traits>

#include "ops_common.cuh"

namespace tide {
namespace {

constexpr int kMaxCols = 16384;
constexpr int kMinBlock = 256;

struct NormArgs {
  int64_t rows, cols;
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  float eps;
  void* h;
  int64_t ldh;
  void* y;
  int64_t ldy;
  float* rstd;
  uint8_t* codes;
  int64_t ldc;
  uint8_t* scales;
  int64_t lds;
};

struct NormGradArgs {
  int64_t rows, cols;
  const void* dy;
  int64_t lddy;
  const void* h;
  int64_t ldh;
  const uint8_t* codes;
  int64_t ldc;
  const uint8_t* scales;
  int64_t lds;
  const void* weight;
  const float* rstd;
  const void* dres;
  int64_t ldres;
  void* dx;
  int64_t lddx;
  float* partial;  // [groups][cols]: each row group's sum of dy * n; NULL: not wanted
};

// Sum of v over the TPR threads that share a row (TPR a power of two, at least
// 32); `scratch` has a float per warp.  The order is fixed.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (TPR > 32) {
    constexpr int warps = TPR / 32;
    const int warp = threadIdx.x / 32, first = warp / warps * warps;
    __syncthreads();  // the previous row's sums have been read
    if (threadIdx.x % 32 == 0) scratch[warp] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < warps; ++w) v += scratch[first + w];
  }
  return v;
}

// A row takes TPR threads, each NV vectors of V columns; a block holds
// blockDim.x / TPR rows.
template <typename T, int TPR, int V, int NV>
__global__ void __launch_bounds__(TPR < kMinBlock ? kMinBlock : TPR) norm_kernel(const NormArgs a) {
  __shared__ float scratch[32];
  const int lane = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
  const bool here = row < a.rows;
  float s[NV][V];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * V;
#pragma unroll
    for (int k = 0; k < V; ++k) s[i][k] = 0.0f;
    if (here && col < a.cols) {
      load_vec<V>((const T*)a.x + row * a.ldx + col, s[i]);
      if (a.residual) {
        float r[V];
        load_vec<V>((const T*)a.residual + row * a.ldr + col, r);
#pragma unroll
        for (int k = 0; k < V; ++k) s[i][k] += r[k];
      }
    }
#pragma unroll
    for (int k = 0; k < V; ++k) sum = fmaf(s[i][k], s[i][k], sum);
  }
  sum = row_sum<TPR>(sum, scratch);
  const float rstd = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
  if (here && lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * V;
    const bool in = here && col < a.cols;
    float y[V];
    if (in) {
      if (a.h) store_vec<V>((T*)a.h + row * a.ldh + col, s[i]);
      load_vec<V>((const T*)a.weight + col, y);
#pragma unroll
      for (int k = 0; k < V; ++k) y[k] *= s[i][k] * rstd;
      if (a.y) store_vec<V>((T*)a.y + row * a.ldy + col, y);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) y[k] = 0.0f;
    }
    if (a.codes) {
      // 32 / V neighbouring lanes hold a block of 32 columns.
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        y[k] = finite_or_nan(y[k]);
        m = fmaxf(m, fabsf(y[k]));
      }
#pragma unroll
      for (int d = 1; d < kMxBlock / V; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      const int byte = scale_byte(m);
      const float inv = scale_inverse(byte);
      if (in) {
        uint8_t* c = a.codes + row * a.ldc + col;
        if constexpr (V == 8) {
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k / 2] |= e4m3_pair(clamp_top(y[2 * k] * inv, byte), clamp_top(y[2 * k + 1] * inv, byte)) << (16 * (k % 2));
          *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
        } else {
          *c = (uint8_t)e4m3_pair(clamp_top(y[0] * inv, byte), 0.0f);
        }
        if (col % kMxBlock == 0) a.scales[row * a.lds + col / kMxBlock] = (uint8_t)byte;
      }
    }
  }
}

// Row groups (TPR threads each) walk the rows with a fixed stride, so a thread
// keeps its columns and their share of dweight in registers.
template <typename T, int TPR, int V, int NV>
__global__ void __launch_bounds__(TPR < kMinBlock ? kMinBlock : TPR) norm_grad_kernel(const NormGradArgs a) {
  __shared__ float scratch[32];
  const int lane = threadIdx.x % TPR;
  const int64_t group = (int64_t)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR;
  const int64_t groups = (int64_t)gridDim.x * (blockDim.x / TPR);
  float acc[NV][V] = {};
  // Every group of a block makes the same number of turns (row_sum's barriers).
  for (int64_t first = (int64_t)blockIdx.x * (blockDim.x / TPR); first < a.rows; first += groups) {
    const int64_t row = first + threadIdx.x / TPR;
    const bool here = row < a.rows;
    const float rstd = here ? a.rstd[row] : 0.0f;
    float n[NV][V], g[NV][V];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + lane) * V;
#pragma unroll
      for (int k = 0; k < V; ++k) n[i][k] = g[i][k] = 0.0f;
      if (here && col < a.cols) {
        if (a.h) {
          load_vec<V>((const T*)a.h + row * a.ldh + col, n[i]);
        } else {
          const float sc = scale_value(a.scales[row * a.lds + col / kMxBlock]);
          const uint8_t* c = a.codes + row * a.ldc + col;
          if constexpr (V == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 t = e4m3_values(((k < 2 ? u.x : u.y) >> (16 * (k % 2))) & 0xffffu);
              n[i][2 * k] = t.x * sc;
              n[i][2 * k + 1] = t.y * sc;
            }
          } else {
            n[i][0] = e4m3_values(*c).x * sc;
          }
        }
        load_vec<V>((const T*)a.dy + row * a.lddy + col, g[i]);
        float w[V];
        load_vec<V>((const T*)a.weight + col, w);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          n[i][k] *= rstd;
          acc[i][k] = fmaf(g[i][k], n[i][k], acc[i][k]);
          g[i][k] *= w[k];
          sum = fmaf(g[i][k], n[i][k], sum);
        }
      }
    }
    if (!a.dx) continue;
    sum = row_sum<TPR>(sum, scratch);
    const float mean = sum / (float)a.cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * TPR + lane) * V;
      if (here && col < a.cols) {
        float d[V] = {};
        if (a.dres) load_vec<V>((const T*)a.dres + row * a.ldres + col, d);
#pragma unroll
        for (int k = 0; k < V; ++k) d[k] = fmaf(rstd, fmaf(-n[i][k], mean, g[i][k]), d[k]);
        store_vec<V>((T*)a.dx + row * a.lddx + col, d);
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * TPR + lane) * V;
    if (col < a.cols) {
#pragma unroll
      for (int k = 0; k < V; ++k) a.partial[group * a.cols + col + k] = acc[i][k];
    }
  }
}

// dweight: the sum of the groups' partials, in a fixed order.  A block takes
// 32 columns; warp w adds partials w, w + 32, ...
template <typename T>
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float* __restrict__ partial, int64_t groups,
                                                           int64_t cols, T* __restrict__ dweight) {
  __shared__ float s[32][33];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (col < cols)
    for (int64_t g = warp; g < groups; g += 32) v += partial[g * cols + col];
  s[warp][lane] = v;
  __syncthreads();
  v = s[lane][warp];  // lane l of warp w: column w's sum over warp l's groups
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int64_t out = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && out < cols) {
    const float t[1] = {v};
    store_vec<1>(dweight + out, t);
  }
}

// Calls f(TPR, V, NV as constants) for the smallest instance that holds a row.
template <typename F>
void with_shape(bool vec, int64_t cols, F&& f) {
#define TIDE_SHAPE(tpr, v, nv) \
  if (cols <= (int64_t)(tpr) * (v) * (nv)) \
    return f(std::integral_constant<int, tpr>(), std::integral_constant<int, v>(), std::integral_constant<int, nv>())
  if (vec) {
    TIDE_SHAPE(32, 8, 1);
    TIDE_SHAPE(32, 8, 2);
    TIDE_SHAPE(128, 8, 1);
    TIDE_SHAPE(128, 8, 2);
    TIDE_SHAPE(256, 8, 2);
    TIDE_SHAPE(512, 8, 2);
    TIDE_SHAPE(1024, 8, 2);
  } else {
    TIDE_SHAPE(32, 1, 8);
    TIDE_SHAPE(128, 1, 8);
    TIDE_SHAPE(256, 1, 8);
    TIDE_SHAPE(512, 1, 8);
    TIDE_SHAPE(1024, 1, 8);
    TIDE_SHAPE(1024, 1, 16);
  }
#undef TIDE_SHAPE
}

int rows_per_block(int tpr) { return tpr < kMinBlock ? kMinBlock / tpr : 1; }

template <typename T>
tide_status norm(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.x, a.ldx, sizeof(T), a.rows) &&
                   rows_aligned(a.residual, a.ldr, sizeof(T), a.rows) && rows_aligned(a.h, a.ldh, sizeof(T), a.rows) &&
                   rows_aligned(a.y, a.ldy, sizeof(T), a.rows) && (uintptr_t)a.weight % 16 == 0 &&
                   (uintptr_t)a.codes % 8 == 0 && (!a.codes || a.rows <= 1 || a.ldc % 8 == 0);
  tide_status st = TIDE_OK;
  with_shape(vec, a.cols, [&](auto tpr, auto v, auto nv) {
    const int rpb = rows_per_block(tpr);
    const int64_t grid = (a.rows + rpb - 1) / rpb;
    if (grid > INT32_MAX) {
      st = fail(TIDE_ERR_UNIMPLEMENTED, "too many rows for one launch");
      return;
    }
    norm_kernel<T, tpr(), v(), nv()><<<(unsigned)grid, tpr() * rpb, 0, stream>>>(a);
    st = cuda_status(cudaGetLastError(), "rms norm");
  });
  return st;
}

// Row groups of the backward pass: what fills the GPU, at most one a row.
int64_t grad_groups(int64_t rows, int tpr, int sms) {
  const int rpb = rows_per_block(tpr);
  const int64_t blocks = std::min<int64_t>((rows + rpb - 1) / rpb, (int64_t)sms * (2048 / (tpr * rpb)));
  return blocks * rpb;
}

template <typename T>
tide_status norm_grad(NormGradArgs a, void* dweight, cudaStream_t stream) {
  const int sms = ops_num_sms();
  if (sms <= 0) return fail(TIDE_ERR_CUDA, "the current device could not be queried");
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.dy, a.lddy, sizeof(T), a.rows) &&
                   rows_aligned(a.h, a.ldh, sizeof(T), a.rows) && rows_aligned(a.dres, a.ldres, sizeof(T), a.rows) &&
                   rows_aligned(a.dx, a.lddx, sizeof(T), a.rows) && (uintptr_t)a.weight % 16 == 0 &&
                   (uintptr_t)a.codes % 8 == 0 && (a.h || a.rows <= 1 || a.ldc % 8 == 0);
  tide_status st = TIDE_OK;
  int64_t groups = 0;
  if (a.rows > 0)
    with_shape(vec, a.cols, [&](auto tpr, auto v, auto nv) {
      const int rpb = rows_per_block(tpr);
      groups = grad_groups(a.rows, tpr, sms);
      norm_grad_kernel<T, tpr(), v(), nv()><<<(unsigned)(groups / rpb), tpr() * rpb, 0, stream>>>(a);
      st = cuda_status(cudaGetLastError(), "rms norm backward");
    });
  if (st == TIDE_OK && dweight) {
    norm_weight_kernel<T><<<(unsigned)((a.cols + 31) / 32), 1024, 0, stream>>>(a.partial, groups, a.cols, (T*)dweight);
    st = cuda_status(cudaGetLastError(), "rms norm weight gradient");
  }
  return st;
}

tide_status check_cols(int64_t cols) {
  return cols > kMaxCols ? fail(TIDE_ERR_UNIMPLEMENTED, "rms norm: rows longer than 16384") : TIDE_OK;
}

}  // namespace

int ops_num_sms() {
  static int known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 64 && known[dev] > 0) return known[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev] = n;
  return n;
}

}  // namespace tide

using namespace tide;

extern "C" {

tide_status tide_rms_norm(int64_t rows, int64_t cols, int32_t dtype, const void* x, int64_t ldx, const void* residual,
                          int64_t ldr, const void* weight, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                          float* rstd, uint8_t* codes, int64_t ld_codes, uint8_t* scales, int64_t ld_scales,
                          void* stream) {
  clear_error();
  TIDE_TRY(check_sizes(rows, cols, "rms norm"));
  TIDE_TRY(check_dtype(dtype));
  if (rows == 0 || cols == 0) return TIDE_OK;
  TIDE_TRY(check_cols(cols));
  const int64_t e = elem_bytes_of(dtype);
  TIDE_TRY(check_matrix(x, rows, cols, ldx, e, "x"));
  if (residual) TIDE_TRY(check_matrix(residual, rows, cols, ldr, e, "residual"));
  TIDE_TRY(check_matrix(weight, 1, cols, cols, e, "weight"));
  if (h) TIDE_TRY(check_matrix(h, rows, cols, ldh, e, "h"));
  if (y) TIDE_TRY(check_matrix(y, rows, cols, ldy, e, "y"));
  if (rstd) TIDE_TRY(check_matrix(rstd, 1, rows, rows, 4, "rstd"));
  if (codes || scales) TIDE_TRY(check_checkpoint(codes, ld_codes, scales, ld_scales, rows, cols));
  const NormArgs a{rows, cols, x,   ldx,  residual, ldr,      weight, eps,      h,
                   ldh,  y,    ldy, rstd, codes,    ld_codes, scales, ld_scales};
  return dtype == TIDE_BF16 ? norm<bf16>(a, (cudaStream_t)stream) : norm<float>(a, (cudaStream_t)stream);
}

int64_t tide_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
  const int sms = ops_num_sms();
  int64_t most = 0;  // whichever instance the alignment of the call's rows selects
  for (const bool vec : {true, false})
    with_shape(vec, cols, [&](auto tpr, auto, auto) { most = std::max(most, grad_groups(rows, tpr, sms)); });
  return most * cols * 4;
}

tide_status tide_rms_norm_backward(int64_t rows, int64_t cols, int32_t dtype, const void* dy, int64_t lddy,
                                   const void* h, int64_t ldh, const uint8_t* codes, int64_t ld_codes,
                                   const uint8_t* scales, int64_t ld_scales, const void* weight, const float* rstd,
                                   const void* dres, int64_t ld_dres, void* dx, int64_t lddx, void* dweight,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  TIDE_TRY(check_sizes(rows, cols, "rms norm backward"));
  TIDE_TRY(check_dtype(dtype));
  if (cols == 0 || (!dx && !dweight)) return TIDE_OK;
  TIDE_TRY(check_cols(cols));
  const int64_t e = elem_bytes_of(dtype);
  TIDE_TRY(check_matrix(dy, rows, cols, lddy, e, "dy"));
  if (h) {
    if (codes || scales) return fail(TIDE_ERR_INVALID_ARG, "h is given both plain and as a checkpoint");
    TIDE_TRY(check_matrix(h, rows, cols, ldh, e, "h"));
  } else {
    TIDE_TRY(check_checkpoint(codes, ld_codes, scales, ld_scales, rows, cols));
  }
  if (rows > 0) TIDE_TRY(check_matrix(weight, 1, cols, cols, e, "weight"));
  TIDE_TRY(check_matrix(rstd, 1, rows, rows, 4, "rstd"));
  if (dres) TIDE_TRY(check_matrix(dres, rows, cols, ld_dres, e, "dres"));
  if (dx) TIDE_TRY(check_matrix(dx, rows, cols, lddx, e, "dx"));
  if (dweight) {
    TIDE_TRY(check_matrix(dweight, 1, cols, cols, e, "dweight"));
    const int64_t need = tide_rms_norm_backward_workspace(rows, cols);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(TIDE_ERR_INVALID_ARG, "workspace too small: " + std::to_string(need) + " bytes are needed");
    if ((uintptr_t)workspace % 16) return fail(TIDE_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  }
  const NormGradArgs a{rows,   cols, dy,   lddy,    h,  ldh,  codes, ld_codes, scales, ld_scales,
                       weight, rstd, dres, ld_dres, dx, lddx, dweight ? (float*)workspace : nullptr};
  return dtype == TIDE_BF16 ? norm_grad<bf16>(a, dweight, (cudaStream_t)stream)
                            : norm_grad<float>(a, dweight, (cudaStream_t)stream);
}

}  // extern "C"
