// Linear layer: forward with bias, activation and residual, input gradient
// with the previous activation's derivative, weight and bias gradients
// (include/tide_ops.h).

#include "ops_common.cuh"

namespace tide {

tide_status launch_checkpoint_load_bf16(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc,
                                        const uint8_t* scales, int64_t lds, int32_t act, void* out, int64_t ldo,
                                        cudaStream_t stream);

namespace {

// out[m, n] = epilogue(sum over k of A(m, k) * B(n, k)), with element strides.
struct GemmArgs {
  int64_t m, n, k;
  const bf16* a;
  int64_t a_m, a_k;
  const bf16* b;
  int64_t b_n, b_k;
  // Epilogue: v = sum + bias[n]; z and its checkpoint get v; then
  // v = f(v) + residual, or v * f'(kept z), to out.
  const bf16* bias;
  int32_t act;
  bool grad;  // multiply by f'(zin) instead of applying f
  const bf16* residual;
  int64_t ldr;
  bf16* out;
  int64_t ldo;
  bf16* z;
  int64_t ldz;
  uint8_t* codes;
  int64_t ldc;
  uint8_t* scales;
  int64_t lds;
  const bf16* zin;
  int64_t ldzin;
  const uint8_t* cin;
  int64_t ldcin;
  const uint8_t* sin;
  int64_t ldsin;
};

constexpr int kTile = 64, kStep = 16;

__global__ void __launch_bounds__(256) gemm_kernel(const GemmArgs g) {
  __shared__ float sa[kStep][kTile + 4], sb[kStep][kTile + 4];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t tiles_n = (g.n + kTile - 1) / kTile;
  const int64_t m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < g.k; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      // Neighbouring threads follow whichever axis is contiguous.
      const int ma = g.a_k == 1 ? i / kStep : i % kTile, ka = g.a_k == 1 ? i % kStep : i / kTile;
      const int nb = g.b_k == 1 ? i / kStep : i % kTile, kb = g.b_k == 1 ? i % kStep : i / kTile;
      sa[ka][ma] = m0 + ma < g.m && k0 + ka < g.k ? __bfloat162float(g.a[(m0 + ma) * g.a_m + (k0 + ka) * g.a_k]) : 0.0f;
      sb[kb][nb] = n0 + nb < g.n && k0 + kb < g.k ? __bfloat162float(g.b[(n0 + nb) * g.b_n + (k0 + kb) * g.b_k]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    float most = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx * 4 + j;
      if (m < g.m && n < g.n) {
        float v = acc[i][j] + (g.bias ? __bfloat162float(g.bias[n]) : 0.0f);
        acc[i][j] = v;
        if (g.z) g.z[m * g.ldz + n] = __float2bfloat16_rn(v);
        if (g.grad) {
          if (g.act != TIDE_ACT_NONE) {
            const float z = g.zin ? __bfloat162float(g.zin[m * g.ldzin + n])
                                  : e4m3_values(g.cin[m * g.ldcin + n]).x *
                                        scale_value(g.sin[m * g.ldsin + n / kMxBlock]);
            v *= act_grad<true>(g.act, z);
          }
        } else {
          v = act_value<true>(g.act, v);
        }
        if (g.residual) v += __bfloat162float(g.residual[m * g.ldr + n]);
        if (g.out) g.out[m * g.ldo + n] = __float2bfloat16_rn(v);
      } else {
        acc[i][j] = 0.0f;
      }
      acc[i][j] = finite_or_nan(acc[i][j]);
      most = fmaxf(most, fabsf(acc[i][j]));
    }
    if (g.codes) {
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
      const int byte = scale_byte(most);
      const float inv = scale_inverse(byte);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + tx * 4 + j;
        if (m < g.m && n < g.n) {
          g.codes[m * g.ldc + n] = (uint8_t)e4m3_pair(clamp_top(acc[i][j] * inv, byte), 0.0f);
          if (n % kMxBlock == 0) g.scales[m * g.lds + n / kMxBlock] = (uint8_t)byte;
        }
      }
    }
  }
}

tide_status gemm(const GemmArgs& g, cudaStream_t stream) {
  const int64_t tiles_m = (g.m + kTile - 1) / kTile, tiles_n = (g.n + kTile - 1) / kTile;
  if (tiles_m > INT32_MAX / tiles_n) return fail(TIDE_ERR_UNIMPLEMENTED, "product has too many tiles for one launch");
  gemm_kernel<<<(unsigned)(tiles_m * tiles_n), 256, 0, stream>>>(g);
  return cuda_status(cudaGetLastError(), "linear product");
}

// db: a block sums 32 columns over all rows, in a fixed order.
__global__ void __launch_bounds__(1024) column_sum_kernel(int64_t rows, int64_t cols, const bf16* __restrict__ x,
                                                          int64_t ldx, bf16* __restrict__ out) {
  __shared__ float s[32][33];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (col < cols)
    for (int64_t r = warp; r < rows; r += 32) v += __bfloat162float(x[r * ldx + col]);
  s[warp][lane] = v;
  __syncthreads();
  v = s[lane][warp];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int64_t o = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && o < cols) out[o] = __float2bfloat16_rn(v);
}

tide_status check_product(int64_t rows, int64_t inner, int64_t outer) {
  if (rows < 0 || inner < 0 || outer < 0) return fail(TIDE_ERR_INVALID_ARG, "linear: negative size");
  return TIDE_OK;
}

tide_status check_workspace(const void* workspace, int64_t bytes, int64_t need) {
  if (need > 0 && (!workspace || bytes < need))
    return fail(TIDE_ERR_INVALID_ARG, "workspace too small: " + std::to_string(need) + " bytes are needed");
  if ((uintptr_t)workspace % 16) return fail(TIDE_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  return TIDE_OK;
}

int64_t packed_ld(int64_t cols) { return (cols + 7) / 8 * 8; }

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" {

int64_t tide_linear_workspace(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t) { return 0; }

tide_status tide_linear(int64_t rows, int64_t inner, int64_t outer, const void* x, int64_t ldx, const void* w,
                        int64_t ldw, const void* bias, int32_t act, const void* residual, int64_t ldr, void* y,
                        int64_t ldy, void* z, int64_t ldz, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                        int64_t ld_scales, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  TIDE_TRY(check_product(rows, inner, outer));
  TIDE_TRY(check_act(act));
  if (rows == 0 || outer == 0) return TIDE_OK;
  TIDE_TRY(check_matrix(x, rows, inner, ldx, 2, "x"));
  TIDE_TRY(check_matrix(w, outer, inner, ldw, 2, "w"));
  if (bias) TIDE_TRY(check_matrix(bias, 1, outer, outer, 2, "bias"));
  if (residual) TIDE_TRY(check_matrix(residual, rows, outer, ldr, 2, "residual"));
  TIDE_TRY(check_matrix(y, rows, outer, ldy, 2, "y"));
  if (z) TIDE_TRY(check_matrix(z, rows, outer, ldz, 2, "z"));
  if (codes || scales) TIDE_TRY(check_checkpoint(codes, ld_codes, scales, ld_scales, rows, outer));
  TIDE_TRY(check_workspace(workspace, workspace_bytes, tide_linear_workspace(rows, inner, outer, x, ldx, w, ldw)));
  GemmArgs g{};
  g.m = rows, g.n = outer, g.k = inner;
  g.a = (const bf16*)x, g.a_m = ldx, g.a_k = 1;
  g.b = (const bf16*)w, g.b_n = ldw, g.b_k = 1;
  g.bias = (const bf16*)bias, g.act = act;
  g.residual = (const bf16*)residual, g.ldr = ldr;
  g.out = (bf16*)y, g.ldo = ldy, g.z = (bf16*)z, g.ldz = ldz;
  g.codes = codes, g.ldc = ld_codes, g.scales = scales, g.lds = ld_scales;
  return gemm(g, (cudaStream_t)stream);
}

int64_t tide_linear_grad_input_workspace(int64_t, int64_t, int64_t, const void*, int64_t, const void*, int64_t) {
  return 0;
}

tide_status tide_linear_grad_input(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                   const void* w, int64_t ldw, int32_t act, const void* z, int64_t ldz,
                                   const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                                   void* dx, int64_t lddx, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  TIDE_TRY(check_product(rows, inner, outer));
  TIDE_TRY(check_act(act));
  if (rows == 0 || inner == 0) return TIDE_OK;
  TIDE_TRY(check_matrix(dy, rows, outer, lddy, 2, "dy"));
  TIDE_TRY(check_matrix(w, outer, inner, ldw, 2, "w"));
  if (act != TIDE_ACT_NONE) {
    if (z) {
      if (codes || scales) return fail(TIDE_ERR_INVALID_ARG, "z is given both plain and as a checkpoint");
      TIDE_TRY(check_matrix(z, rows, inner, ldz, 2, "z"));
    } else {
      TIDE_TRY(check_checkpoint(codes, ld_codes, scales, ld_scales, rows, inner));
    }
  }
  TIDE_TRY(check_matrix(dx, rows, inner, lddx, 2, "dx"));
  TIDE_TRY(check_workspace(workspace, workspace_bytes,
                           tide_linear_grad_input_workspace(rows, inner, outer, dy, lddy, w, ldw)));
  GemmArgs g{};
  g.m = rows, g.n = inner, g.k = outer;
  g.a = (const bf16*)dy, g.a_m = lddy, g.a_k = 1;
  g.b = (const bf16*)w, g.b_n = 1, g.b_k = ldw;
  g.act = act, g.grad = true;
  g.zin = (const bf16*)z, g.ldzin = ldz;
  g.cin = codes, g.ldcin = ld_codes, g.sin = scales, g.ldsin = ld_scales;
  g.out = (bf16*)dx, g.ldo = lddx;
  return gemm(g, (cudaStream_t)stream);
}

int64_t tide_linear_grad_weight_workspace(int64_t rows, int64_t inner, int64_t outer, const void*, int64_t,
                                          const void* x, int64_t) {
  if (rows <= 0 || inner <= 0 || outer <= 0 || x) return 0;
  return rows * packed_ld(inner) * 2;
}

tide_status tide_linear_grad_weight(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                    const void* x, int64_t ldx, const uint8_t* codes, int64_t ld_codes,
                                    const uint8_t* scales, int64_t ld_scales, int32_t act, void* dw, int64_t lddw,
                                    void* db, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  TIDE_TRY(check_product(rows, inner, outer));
  TIDE_TRY(check_act(act));
  if (outer == 0) return TIDE_OK;
  TIDE_TRY(check_matrix(dy, rows, outer, lddy, 2, "dy"));
  if (x) {
    if (codes || scales) return fail(TIDE_ERR_INVALID_ARG, "x is given both plain and as a checkpoint");
    if (act != TIDE_ACT_NONE) return fail(TIDE_ERR_INVALID_ARG, "an activation goes with a checkpoint, not with x");
    TIDE_TRY(check_matrix(x, rows, inner, ldx, 2, "x"));
  } else {
    TIDE_TRY(check_checkpoint(codes, ld_codes, scales, ld_scales, rows, inner));
  }
  TIDE_TRY(check_matrix(dw, outer, inner, lddw, 2, "dw"));
  if (db) TIDE_TRY(check_matrix(db, 1, outer, outer, 2, "db"));
  TIDE_TRY(check_workspace(workspace, workspace_bytes,
                           tide_linear_grad_weight_workspace(rows, inner, outer, dy, lddy, x, ldx)));
  if (inner > 0) {
    GemmArgs g{};
    g.m = outer, g.n = inner, g.k = rows;
    g.a = (const bf16*)dy, g.a_m = 1, g.a_k = lddy;
    g.b = (const bf16*)x, g.b_n = 1, g.b_k = ldx;
    if (!x && rows > 0) {
      TIDE_TRY(launch_checkpoint_load_bf16(rows, inner, codes, ld_codes, scales, ld_scales, act, workspace,
                                           packed_ld(inner), (cudaStream_t)stream));
      g.b = (const bf16*)workspace, g.b_k = packed_ld(inner);
    }
    g.out = (bf16*)dw, g.ldo = lddw;
    TIDE_TRY(gemm(g, (cudaStream_t)stream));
  }
  if (db) {
    column_sum_kernel<<<(unsigned)((outer + 31) / 32), 1024, 0, (cudaStream_t)stream>>>(
        rows, outer, (const bf16*)dy, lddy, (bf16*)db);
    return cuda_status(cudaGetLastError(), "bias gradient");
  }
  return TIDE_OK;
}

}  // extern "C"
