// Device helpers and host-side argument checks shared by the training-block
// operators (ops_norm.cu, ops_ckpt.cu, ops_linear.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "../../include/tide_ops.h"
#include "tide_internal.h"

namespace tide {

using bf16 = __nv_bfloat16;

// Columns that share one scale of an 8-bit checkpoint.
constexpr int kMxBlock = 32;

// ---------------------------------------------------------------- host side

inline tide_status cuda_status(cudaError_t err, const char* what) {
  return err == cudaSuccess ? TIDE_OK : fail(TIDE_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(err));
}

inline int64_t elem_bytes_of(int32_t dtype) { return dtype == TIDE_BF16 ? 2 : 4; }

inline tide_status check_sizes(int64_t rows, int64_t cols, const char* what) {
  if (rows < 0 || cols < 0) return fail(TIDE_ERR_INVALID_ARG, std::string(what) + ": negative size");
  return TIDE_OK;
}

// One matrix argument: non-null, aligned to its element, rows of at least
// `cols` elements, and byte offsets that fit int64.
inline tide_status check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t elem, const char* what) {
  if (rows == 0 || cols == 0) return TIDE_OK;
  if (!p) return fail(TIDE_ERR_INVALID_ARG, std::string(what) + " is NULL");
  if ((uintptr_t)p % elem) return fail(TIDE_ERR_ALIGNMENT, std::string(what) + " is not aligned to its element size");
  if (rows > 1 && ld < cols) return fail(TIDE_ERR_INVALID_ARG, std::string(what) + ": row stride shorter than a row");
  if (cols > INT64_MAX / elem || (rows > 1 && (ld > INT64_MAX / elem || rows - 1 > (INT64_MAX - cols * elem) / (ld * elem))))
    return fail(TIDE_ERR_OVERFLOW, std::string(what) + " does not fit int64 bytes");
  return TIDE_OK;
}

inline tide_status check_checkpoint(const void* codes, int64_t ld_codes, const void* scales, int64_t ld_scales,
                                    int64_t rows, int64_t cols) {
  tide_status st = check_matrix(codes, rows, cols, ld_codes, 1, "codes");
  if (st == TIDE_OK) st = check_matrix(scales, rows, (cols + kMxBlock - 1) / kMxBlock, ld_scales, 1, "scales");
  return st;
}

inline tide_status check_act(int32_t act) {
  return act < TIDE_ACT_NONE || act > TIDE_ACT_SILU ? fail(TIDE_ERR_INVALID_ARG, "unknown activation") : TIDE_OK;
}

inline tide_status check_dtype(int32_t dtype) {
  return dtype != TIDE_BF16 && dtype != TIDE_F32 ? fail(TIDE_ERR_INVALID_ARG, "unknown element type") : TIDE_OK;
}

// f called with the activation as a constant: kernels are built for each, since one
// for all of them takes the registers and the order of code that the costliest asks
// for (24832 x 64 -> 10301 without any 181 us then, 167 alone; 4093 x 4095 bf16 loaded
// without any 13.0 and 10.9).
template <int ACT>
struct ActTag {
  static constexpr int value = ACT;
};
template <typename F>
auto with_act(int act, F&& f) {
  switch (act) {
    case TIDE_ACT_RELU: return f(ActTag<TIDE_ACT_RELU>());
    case TIDE_ACT_GELU: return f(ActTag<TIDE_ACT_GELU>());
    case TIDE_ACT_GELU_ERF: return f(ActTag<TIDE_ACT_GELU_ERF>());
    case TIDE_ACT_SILU: return f(ActTag<TIDE_ACT_SILU>());
    default: return f(ActTag<TIDE_ACT_NONE>());
  }
}

// Whether rows of a matrix start on 16-byte boundaries (NULL counts: it is
// not touched).
inline bool rows_aligned(const void* p, int64_t ld, int64_t elem, int64_t rows) {
  return !p || ((uintptr_t)p % 16 == 0 && (rows <= 1 || ld * elem % 16 == 0));
}

// out[c] (of `dtype`) = the sum of partial[g][c] over the groups, in a fixed
// order; zero with none.  `after`: the stream's last kernel is this call's.
tide_status launch_sum_groups(const float* partial, int64_t groups, int64_t cols, int32_t dtype, void* out, bool after,
                              cudaStream_t stream);

// The current device's count of waits that ran out (read by tide_ops_check) and the
// bound on every wait.
tide_status ops_timeouts(uint32_t** word);
uint64_t ops_wait_limit_ns();
int64_t ops_test_drop();  // the calling thread's TIDE_OPS_OPT_TEST_DROP_LOAD

// SMs of the current device (asked once per device); 0 if the query failed.
int ops_num_sms();

// Division of 32-bit numbers below 2^31 by a fixed one: a multiplication and a
// shift.  For 2^(s-1) < d <= 2^s, m = ceil(2^(31+s) / d) is below 2^32 and the
// quotient is floor(n * m / 2^(31+s)): the error n * (m d - 2^(31+s)) / (d
// 2^(31+s)) is below n / 2^(31+s) <= 1 / d for n < 2^31.
struct FastDiv {
  uint32_t d = 1, m = 1u << 31, s = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  }
#if defined(__CUDACC__)
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> 31 >> s);
  }
#endif
};

#define TIDE_TRY(expr)                    \
  do {                                    \
    tide_status st_ = (expr);             \
    if (st_ != TIDE_OK) return st_;       \
  } while (0)

// ---------------------------------------------------------------- device side

// V consecutive elements as fp32.  V = 8: 16-byte accesses; V = 1: one element.
template <int V>
__device__ __forceinline__ void load_vec(const bf16* p, float (&v)[V]) {
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __bfloat162float(p[i]);
  }
}

template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[V]) {
  if constexpr (V == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[i];
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

template <int V>
__device__ __forceinline__ void store_vec(bf16* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}

template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[V]) {
  if constexpr (V == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = v[i];
  }
}

// Eight elements at any alignment, as fp32: the widest loads that stay inside
// them.
__device__ __forceinline__ void load_any8(const bf16* p, float (&v)[8]) {
  const uint16_t* x = reinterpret_cast<const uint16_t*>(p);
  uint32_t w[4];
  if ((uintptr_t)x % 4 == 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = reinterpret_cast<const uint32_t*>(x)[j];
  } else {  // an element, three aligned pairs, an element
    const uint32_t first = x[0], last = x[7];
    uint32_t q[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) q[j] = reinterpret_cast<const uint32_t*>(x + 1)[j];
    w[0] = first | q[0] << 16;
    w[1] = __funnelshift_r(q[0], q[1], 16);
    w[2] = __funnelshift_r(q[1], q[2], 16);
    w[3] = q[2] >> 16 | last << 16;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load_any8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = p[j];
}

// The first n of eight elements at any alignment, zeros for the rest.
template <typename T>
__device__ __forceinline__ void load_any8(const T* p, int n, float (&v)[8]) {
  if (n == 8) {
    if ((uintptr_t)p % 16 == 0)
      load_vec<8>(p, v);
    else
      load_any8(p, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? (float)p[k] : 0.0f;
  }
}

// Eight bytes at any alignment.
__device__ __forceinline__ uint2 load_any_bytes(const uint8_t* p) {
  const uint32_t phase = (uint32_t)(uintptr_t)p & 3u;
  if (phase == 0) return make_uint2(reinterpret_cast<const uint32_t*>(p)[0], reinterpret_cast<const uint32_t*>(p)[1]);
  if (phase == 2) {
    const uint32_t a = reinterpret_cast<const uint16_t*>(p)[0], b = *reinterpret_cast<const uint32_t*>(p + 2),
                   c = reinterpret_cast<const uint16_t*>(p)[3];
    return make_uint2(a | b << 16, b >> 16 | c << 16);
  }
  if (phase == 3) {  // 1, 4, 2, 1
    const uint32_t a = p[0], b = *reinterpret_cast<const uint32_t*>(p + 1), c = *reinterpret_cast<const uint16_t*>(p + 5),
                   d = p[7];
    return make_uint2(a | b << 8, b >> 24 | c << 8 | d << 24);
  }
  const uint32_t a = p[0], b = *reinterpret_cast<const uint16_t*>(p + 1), c = *reinterpret_cast<const uint32_t*>(p + 3),
                 d = p[7];  // 1, 2, 4, 1
  return make_uint2(a | b << 8 | c << 24, c >> 8 | d << 24);
}

// ---- 8-bit checkpoints

// Scale byte of a block whose largest finite magnitude is `a`: the smallest
// e >= -127 with a <= 448 * 2^e, plus 127.  With a = 1.m * 2^E and
// 448 = 1.75 * 2^8, e = E - 8 if 1.m <= 1.75, else E - 7.
__device__ __forceinline__ int scale_byte(float a) {
  const uint32_t u = __float_as_uint(a);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b > 0 ? b : 0;
}
// 2^(127 - byte) and 2^(byte - 127); byte is at most 247.
__device__ __forceinline__ float scale_inverse(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
__device__ __forceinline__ float scale_value(int byte) {
  return __uint_as_float(byte > 0 ? (uint32_t)byte << 23 : 0x400000u);
}

// What a checkpoint keeps of a value: infinities become NaN (0 * inf), finite
// values and NaN stay.
__device__ __forceinline__ float finite_or_nan(float v) { return __fmaf_rn(0.0f, v, v); }

// Largest magnitude over the N values of each of LANES neighbouring lanes (a
// power of two) that hold a block; NaN does not count.  Infinities, which are
// rare, are made NaN in v and the finite values looked at again.  With LANES
// above 1 the whole warp calls it.
template <int LANES, int N>
__device__ __forceinline__ float block_magnitude(float (&v)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) m = fmaxf(m, fabsf(v[k]));
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (LANES > 1 ? __any_sync(0xffffffffu, isinf(m)) : isinf(m)) {
    m = 0.0f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = finite_or_nan(v[k]);
      m = fmaxf(m, fabsf(v[k]));
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  return m;
}

// Two codes of values already divided by the scale (lo in the low byte).
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// N values (a multiple of 4) of a block with scale byte `byte` to N / 4 words
// of codes.  The topmost scale's codes stop at 240: the next value, 256 * 2^120,
// is beyond fp32.
template <int N>
__device__ __forceinline__ void encode(float (&v)[N], int byte, uint32_t (&w)[N / 4]) {
  const float inv = scale_inverse(byte);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] *= inv;
  if (byte >= 247) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = fabsf(v[k]) > 240.0f ? copysignf(240.0f, v[k]) : v[k];
  }
#pragma unroll
  for (int k = 0; k < N / 4; ++k)
    w[k] = e4m3_pair(v[4 * k], v[4 * k + 1]) | e4m3_pair(v[4 * k + 2], v[4 * k + 3]) << 16;
}
// One value.
__device__ __forceinline__ uint8_t encode_one(float v, int byte) {
  v *= scale_inverse(byte);
  if (byte >= 247 && fabsf(v) > 240.0f) v = copysignf(240.0f, v);
  return (uint8_t)e4m3_pair(v, 0.0f);
}

// fp32 values of two codes (exact: e4m3 is a subset of fp16).
__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)pair, __NV_E4M3);
  return __half22float2(__half2(h));
}

// A whole warp stores 256 neighbouring codes at any alignment, lane l the first
// n of eight (w) at c; only the last lanes have fewer than eight.  With the
// row's codes `p` bytes past an 8-byte boundary, a lane's aligned word is the
// last p codes of the lane before and its own first 8 - p.
__device__ __forceinline__ void store_codes_any(uint8_t* c, int n, const uint32_t (&w)[2]) {
  const int lane = threadIdx.x % 32;
  const int p = (int)((uintptr_t)c & 7);  // the same for every lane
  const uint64_t cur = (uint64_t)w[1] << 32 | w[0];
  const uint64_t before = __shfl_up_sync(0xffffffffu, cur, 1);
  int n_before = __shfl_up_sync(0xffffffffu, n, 1);
  if (lane == 0) n_before = 0;
  const uint64_t word = p ? cur << (8 * p) | before >> (64 - 8 * p) : cur;
  // Byte j of the word is column j - p; valid from `lo` to below `hi`.
  const int lo = lane == 0 ? p : 0;
  const int hi = n > 0 ? min(8, p + n) : n_before - (8 - p);
  if (lo == 0 && hi == 8) {
    *reinterpret_cast<uint64_t*>(c - p) = word;
  } else {
    for (int j = lo; j < hi; ++j) (c - p)[j] = (uint8_t)(word >> (8 * j));
  }
  if (lane == 31)
    for (int k = 8 - p; k < n; ++k) c[k] = (uint8_t)(cur >> (8 * k));
}

// Eight values from two words of codes.
__device__ __forceinline__ void decode8(uint2 c, float scale, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = e4m3_values(((k < 2 ? c.x : c.y) >> (16 * (k % 2))) & 0xffffu);
    v[2 * k] = t.x * scale;
    v[2 * k + 1] = t.y * scale;
  }
}

// ---- activations

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2/pi)
constexpr float kGeluB = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865475f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// FAST: exp(t) = 2^(t log2 e) and the reciprocal by the approximate instructions
// that flush subnormal numbers (a result below 2^-126 becomes 0), good to a few
// units in the last place of fp32 over the range that matters, for results that
// are then rounded to bf16 or 8 bits.  fp32 results take the accurate functions.
template <bool FAST>
__device__ __forceinline__ float exp_of(float t) {
  if constexpr (!FAST) return expf(t);
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t * 1.4426950408889634f));
  return r;
}

__device__ __forceinline__ float reciprocal_ftz(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

// 1 / (1 + exp(-t)): 0 at -inf (and where the exponential overflows), 1 at
// +inf, NaN at NaN.
template <bool FAST>
__device__ __forceinline__ float sigmoid(float t) {
  const float d = 1.0f + exp_of<FAST>(-t);
  return FAST ? reciprocal_ftz(d) : 1.0f / d;
}

// The normal distribution's p(z), and e = exp(-z^2 / 2).  FAST: for x = |z| and
// t = 1 / (1 + 0.324 x) the ratio p(-x) / e is smooth in t and goes as 1 / x, so it is
// t times a polynomial in t, here the one of degree 7 with the least largest error
// relative to the ratio over all x >= 0 (found by linear programming): 2^-20.6, with
// fp32's roundings below 2^-19.  Relative, because p alone, of z < 0, is what z * p
// is made of: 0.5 + 0.5 erf(z / sqrt(2)) cancels there and has nothing left at -5.6.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  e = exp_of<FAST>(-0.5f * z * z);
  if constexpr (!FAST) return 0.5f * erfcf(-kInvSqrt2 * z);
  const float t = reciprocal_ftz(fmaf(0.324f, fabsf(z), 1.0f));
  float q = fmaf(0.0340613537f, t, -0.11560633f);
  q = fmaf(q, t, 0.0897367969f);
  q = fmaf(q, t, 0.0238828231f);
  q = fmaf(q, t, 0.0942828283f);
  q = fmaf(q, t, 0.115103588f);
  q = fmaf(q, t, 0.129282221f);
  q = fmaf(q, t, 0.129257008f);
  q *= t * e;
  return z < 0.0f ? q : 1.0f - q;
}

// GELU, GELU_ERF and SILU are z * p(z) with p from 0 to 1; where p has come
// down to 0 the product is 0 (not -inf * 0).
template <bool FAST>
__device__ __forceinline__ float act_value(int act, float z) {
  float p, e;
  switch (act) {
    case TIDE_ACT_RELU: return z < 0.0f ? 0.0f : z;
    case TIDE_ACT_GELU: p = sigmoid<FAST>(2.0f * kGeluA * (z + kGeluB * z * z * z)); break;
    case TIDE_ACT_GELU_ERF: p = normal_cdf<FAST>(z, e); break;
    case TIDE_ACT_SILU: p = sigmoid<FAST>(z); break;
    default: return z;
  }
  return p == 0.0f ? 0.0f : z * p;
}

// f' = p + z p'; where p' has come down to 0 it is p (not inf * 0).
template <bool FAST>
__device__ __forceinline__ float act_grad(int act, float z) {
  float p, d;
  switch (act) {
    case TIDE_ACT_RELU: return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    case TIDE_ACT_GELU:
      p = sigmoid<FAST>(2.0f * kGeluA * (z + kGeluB * z * z * z));
      d = p * (1.0f - p);
      return d == 0.0f ? p : p + z * d * (2.0f * kGeluA * (1.0f + 3.0f * kGeluB * z * z));
    case TIDE_ACT_GELU_ERF:
      p = normal_cdf<FAST>(z, d);
      return d == 0.0f ? p : p + z * d * kInvSqrt2Pi;
    case TIDE_ACT_SILU:
      p = sigmoid<FAST>(z);
      d = p * (1.0f - p);
      return d == 0.0f ? p : p + z * d;
    default: return 1.0f;
  }
}

}  // namespace tide
