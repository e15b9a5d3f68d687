// What the operators at the ends of a training step share (ops_embed.cu,
// ops_logprob.cu): token ids, and rows of any alignment walked in vectors of
// eight elements that start on 16-byte boundaries.
#pragma once

#include "ops_common.cuh"

#include "../../include/tide_lm_ops.h"

namespace tide {

inline tide_status check_index(int32_t index) {
  return index != TIDE_I32 && index != TIDE_I64 ? fail(TIDE_ERR_INVALID_ARG, "unknown type of token ids") : TIDE_OK;
}
inline int64_t index_bytes_of(int32_t index) { return index == TIDE_I64 ? 8 : 4; }

// Launches rows in parts whose units of work are counted in 32 bits: f(first row, units,
// blocks), `unit` units of work a block, `per_row` a row.
template <typename F>
tide_status in_row_launches(int64_t rows, int64_t per_row, int64_t unit, const char* what, F&& f) {
  const int64_t most = ((int64_t)INT32_MAX - unit) / per_row;  // rows of a launch
  if (most <= 0) return fail(TIDE_ERR_UNIMPLEMENTED, std::string(what) + ": rows too long");
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most, items = n * per_row;
    f(r, (uint32_t)items, (unsigned)((items + unit - 1) / unit));
    TIDE_TRY(cuda_status(cudaGetLastError(), what));
  }
  return TIDE_OK;
}

#if defined(__CUDACC__)

// The token at place i; outside 0..vocab-1: -1.
__device__ __forceinline__ int token_at(const void* ids, int32_t index, int64_t i, int64_t vocab) {
  const int64_t t = index == TIDE_I64 ? reinterpret_cast<const int64_t*>(ids)[i] : reinterpret_cast<const int32_t*>(ids)[i];
  return t >= 0 && t < vocab ? (int)t : -1;
}

// Elements that a row starts past a 16-byte boundary: vector v of the row holds the columns
// from 8 v - phase on, the first and the last fewer than eight.
template <typename T>
__device__ __forceinline__ int row_phase(const T* row) {
  return (int)((uintptr_t)row & 15) / (int)sizeof(T);
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ float value(int k) const {
    if constexpr (sizeof(T) == 2)
      return __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    else
      return __uint_as_float(w[k]);
  }
  __device__ __forceinline__ void load(const T* p) {  // on a 16-byte boundary
#pragma unroll
    for (int j = 0; j < (int)sizeof(T) / 2; ++j) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[j];
      w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
    }
  }
  // The columns from `col` on of a row of `cols`; -inf where there is none.
  __device__ __forceinline__ void load_some(const T* row, int64_t col, int64_t cols) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) * 2; ++k) w[k] = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (col + k < 0 || col + k >= cols) continue;
      if constexpr (sizeof(T) == 2) {
        const uint32_t x = reinterpret_cast<const uint16_t*>(row)[col + k];
        w[k / 2] = k % 2 ? (w[k / 2] & 0xffffu) | x << 16 : (w[k / 2] & 0xffff0000u) | x;
      } else {
        w[k] = reinterpret_cast<const uint32_t*>(row)[col + k];
      }
    }
  }
};

// Eight elements that begin BYTES past a 16-byte boundary, from the granules that hold them.
template <int BYTES, typename T>
__device__ __forceinline__ void load_shifted(const T* p, float (&v)[8]) {
  constexpr int kGranules = (BYTES + 8 * (int)sizeof(T) + 15) / 16, kWord = BYTES / 4;
  const uint4* g = reinterpret_cast<const uint4*>((uintptr_t)p - BYTES);
  uint32_t w[4 * kGranules];
#pragma unroll
  for (int j = 0; j < kGranules; ++j) {
    const uint4 u = g[j];
    w[4 * j] = u.x, w[4 * j + 1] = u.y, w[4 * j + 2] = u.z, w[4 * j + 3] = u.w;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if constexpr (sizeof(T) == 2) {
      const int e = BYTES / 2 + k;
      v[k] = __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    } else {
      v[k] = __uint_as_float(w[kWord + k]);
    }
  }
}

// The columns col .. col + 7 of a row of `cols` that exist, at any alignment of the row;
// zeros for the rest.  Whole granules inside the row where there are any: narrow loads at a
// stride cost L1 four to eight times as many turns.  A row's vectors all branch alike.
template <typename T>
__device__ __forceinline__ void load_columns(const T* row, int64_t col, int64_t cols, float (&v)[8]) {
  const T* p = row + col;
  const int phase = (int)((uintptr_t)p & 15), before = phase / (int)sizeof(T);
  if (col >= before && col - before + (phase ? 16 / (int)sizeof(T) : 0) + 8 <= cols) {
    switch (phase) {
      case 0: return load_vec<8>(p, v);
      case 4: return load_shifted<4>(p, v);
      case 8: return load_shifted<8>(p, v);
      case 12: return load_shifted<12>(p, v);
    }
    if constexpr (sizeof(T) == 2) {
      switch (phase) {
        case 2: return load_shifted<2>(p, v);
        case 6: return load_shifted<6>(p, v);
        case 10: return load_shifted<10>(p, v);
        default: return load_shifted<14>(p, v);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = col + k >= 0 && col + k < cols ? (float)p[k] : 0.0f;
}
// ... and stored, at a 16-byte boundary where all eight exist.
template <typename T>
__device__ __forceinline__ void store_columns(T* row, int64_t col, int64_t cols, const float (&v)[8]) {
  if (col >= 0 && col + 8 <= cols) {
    store_vec<8>(row + col, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float one[1] = {v[k]};
      if (col + k >= 0 && col + k < cols) store_vec<1>(row + col + k, one);
    }
  }
}

#endif  // __CUDACC__

}  // namespace tide
