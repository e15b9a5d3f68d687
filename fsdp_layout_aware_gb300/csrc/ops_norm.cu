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
  float* partial;  // [row groups][cols]: each one's sum of dy * n; NULL: not wanted
};

// Sum of v over the threads of a row (blockDim.x, a multiple of 32; threadIdx.y
// is the row).  One barrier: `turn` alternates the scratch floats, one per
// warp, so a sum is read before its place is written again.  The order is
// fixed.
__device__ __forceinline__ float row_sum(float v, float (&scratch)[2][32], int& turn) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int warps = blockDim.x / 32;
  if (warps > 1) {
    const int first = threadIdx.y * warps;
    float* s = scratch[turn];
    turn ^= 1;
    if (threadIdx.x % 32 == 0) s[first + threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < warps; ++w) v += s[first + w];
  }
  return v;
}

// A row takes blockDim.x threads, each NV vectors of V columns; a block holds
// blockDim.y rows.
template <typename T, int V, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a) {
  __shared__ float scratch[2][32];
  int turn = 0;
  const int lane = threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool here = row < a.rows;
  float s[NV][V];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * blockDim.x + lane) * V;
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
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) sum = fmaf(s[i][k], s[i][k], sum);
  sum = row_sum(sum, scratch, turn);
  const float rstd = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
  if (here && lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * blockDim.x + lane) * V;
    const bool in = here && col < a.cols;
    float y[V];
#pragma unroll
    for (int k = 0; k < V; ++k) y[k] = 0.0f;
    if (in) {
      if (a.h) store_vec<V>((T*)a.h + row * a.ldh + col, s[i]);
      load_vec<V>((const T*)a.weight + col, y);
#pragma unroll
      for (int k = 0; k < V; ++k) y[k] *= s[i][k] * rstd;
      if (a.y) store_vec<V>((T*)a.y + row * a.ldy + col, y);
    }
    if (a.codes) {
      // 32 / V neighbouring lanes hold a block of 32 columns.
      const int byte = scale_byte(block_magnitude<kMxBlock / V>(y));
      if (in) {
        uint8_t* c = a.codes + row * a.ldc + col;
        if constexpr (V == 8) {
          uint32_t w[2];
          encode(y, byte, w);
          *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
        } else {
          *c = encode_one(y[0], byte);
        }
        if (col % kMxBlock == 0) a.scales[row * a.lds + col / kMxBlock] = (uint8_t)byte;
      }
    }
  }
}

// ---- backward

// dx of one row's columns and their share of dweight, once n = h (still without
// rstd) and g = dy are in registers.
template <typename T, int V, int NV>
__device__ __forceinline__ void grad_row(const NormGradArgs& a, int64_t row, bool here, float rstd, float (&n)[NV][V],
                                         float (&g)[NV][V], const float (&w)[NV][V], float (&acc)[NV][V],
                                         float (&scratch)[2][32], int& turn, const float (&dres)[NV][V]) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      n[i][k] *= rstd;
      acc[i][k] = fmaf(g[i][k], n[i][k], acc[i][k]);
      g[i][k] *= w[i][k];
      sum = fmaf(g[i][k], n[i][k], sum);
    }
  if (!a.dx) return;
  const float mean = row_sum(sum, scratch, turn) / (float)a.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * blockDim.x + threadIdx.x) * V;
    if (here && col < a.cols) {
      float d[V];
#pragma unroll
      for (int k = 0; k < V; ++k) d[k] = fmaf(rstd, fmaf(-n[i][k], mean, g[i][k]), dres[i][k]);
      store_vec<V>((T*)a.dx + row * a.lddx + col, d);
    }
  }
}

template <int V, int NV>
__device__ __forceinline__ void store_partial(const NormGradArgs& a, const float (&acc)[NV][V]) {
  if (!a.partial) return;
  float* p = a.partial + ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * a.cols;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * blockDim.x + threadIdx.x) * V;
    if (col < a.cols) store_vec<V>(p + col, acc[i]);
  }
}

// Row groups (blockDim.x threads) walk the rows with a fixed stride, so a
// thread keeps its columns' weights and their share of dweight in registers.
// Any alignment (V = 1), and rows too long for the ring below.
template <typename T, int V, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_grad_kernel(const NormGradArgs a) {
  __shared__ float scratch[2][32];
  int turn = 0;
  float acc[NV][V] = {}, w[NV][V] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * blockDim.x + threadIdx.x) * V;
    if (col < a.cols) load_vec<V>((const T*)a.weight + col, w[i]);
  }
  // Every group of a block makes the same number of turns (row_sum's barrier).
  for (int64_t first = (int64_t)blockIdx.x * blockDim.y; first < a.rows; first += (int64_t)gridDim.x * blockDim.y) {
    const int64_t row = first + threadIdx.y;
    const bool here = row < a.rows;
    const float rstd = here ? a.rstd[row] : 0.0f;
    float n[NV][V] = {}, g[NV][V] = {}, dres[NV][V] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int col = (i * blockDim.x + threadIdx.x) * V;
      if (here && col < a.cols) {
        if (a.h) {
          load_vec<V>((const T*)a.h + row * a.ldh + col, n[i]);
        } else {
          const float scale = scale_value(a.scales[row * a.lds + col / kMxBlock]);
          const uint8_t* c = a.codes + row * a.ldc + col;
          if constexpr (V == 8)
            decode8(*reinterpret_cast<const uint2*>(c), scale, n[i]);
          else
            n[i][0] = e4m3_values(*c).x * scale;
        }
        load_vec<V>((const T*)a.dy + row * a.lddy + col, g[i]);
        if (a.dres) load_vec<V>((const T*)a.dres + row * a.ldres + col, dres[i]);
      }
    }
    grad_row<T, V, NV>(a, row, here, rstd, n, g, w, acc, scratch, turn, dres);
  }
  store_partial<V, NV>(a, acc);
}

__device__ __forceinline__ void copy_async16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void copy_async8(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem), "l"(gmem) : "memory");
}

// Shared memory a ring slot (one row of the block) takes: for every thread and
// vector, its h (or codes), dy and dres.
inline int ring_slot_bytes(int threads, int nv, int elem, bool kept, bool dres) {
  return threads * nv * ((kept ? 8 : 8 * elem) + 8 * elem * (dres ? 2 : 1));
}

// As above with aligned rows, eight columns a vector, DEPTH rows of a group in
// flight: each thread copies its own columns of the rows to come into a ring in
// shared memory and reads nothing else from it, so the copies need no barrier
// and cost no registers.  What is in flight then is DEPTH - 1 rows a block,
// whatever the one barrier of a row costs.
template <typename T, int NV, int DEPTH, bool KEPT, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_grad_ring_kernel(const NormGradArgs a) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float scratch[2][32];
  constexpr int kWords = sizeof(T) / 2;  // 16-byte words of a vector
  constexpr int kPer = 16 / sizeof(T);   // elements of a word
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const bool has_dres = a.dres != nullptr;
  // Within a slot: dy, dres, h; within each, word by word over the threads, so
  // neighbouring threads use neighbouring banks.
  const uint32_t vec_bytes = (uint32_t)threads * 16;
  const uint32_t off_dres = NV * kWords * vec_bytes, off_h = off_dres * (has_dres ? 2 : 1);
  const uint32_t slot = off_h + NV * (KEPT ? vec_bytes / 2 : kWords * vec_bytes);
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);
  const int apart = blockDim.x * 8;  // columns from one of a thread's vectors to the next
  const int col0 = threadIdx.x * 8;

  int turn = 0;
  float acc[NV][8] = {};
  T w[NV][8];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    in[i] = col0 + i * apart < a.cols;
#pragma unroll
    for (int k = 0; k < 8; ++k) w[i][k] = in[i] ? ((const T*)a.weight)[col0 + i * apart + k] : T(0.0f);
  }
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;

  // The next row to fetch, and where its vectors are.
  int64_t ahead = row;
  const T* dy = (const T*)a.dy + row * a.lddy + col0;
  const T* dres = has_dres ? (const T*)a.dres + row * a.ldres + col0 : nullptr;
  const T* h = KEPT ? nullptr : (const T*)a.h + row * a.ldh + col0;
  const uint8_t* codes = KEPT ? a.codes + row * a.ldc + col0 : nullptr;
  T* dx = (T*)a.dx + row * a.lddx + col0;
  auto fetch = [&](uint32_t at) {
    if (ahead < a.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!in[i]) continue;
#pragma unroll
        for (int q = 0; q < kWords; ++q) {
          const uint32_t o = at + (i * kWords + q) * vec_bytes + tid * 16;
          copy_async16(o, dy + i * apart + q * kPer);
          if (has_dres) copy_async16(o + off_dres, dres + i * apart + q * kPer);
          if constexpr (!KEPT) copy_async16(o + off_h, h + i * apart + q * kPer);
        }
        if constexpr (KEPT) copy_async8(at + off_h + (i * threads + tid) * 8, codes + i * apart);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += step;
    dy += step * a.lddy;
    if (has_dres) dres += step * a.ldres;
    if constexpr (KEPT)
      codes += step * a.ldc;
    else
      h += step * a.ldh;
  };
  auto word = [&](const unsigned char* s, float* v) {  // a 16-byte word of T
    if constexpr (kWords == 1) {
      load_vec<8>(reinterpret_cast<const T*>(s), *reinterpret_cast<float(*)[8]>(v));
    } else {
      const float4 x = *reinterpret_cast<const float4*>(s);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    }
  };
  // rstd and the scales of a row, one row ahead.
  float rstd = 0.0f;
  uint8_t scale[NV] = {};
  auto fetch_small = [&](int64_t r) {
    if (r >= a.rows) return;
    rstd = a.rstd[r];
    if constexpr (KEPT) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i]) scale[i] = a.scales[r * a.lds + (col0 + i * apart) / kMxBlock];
    }
  };

#pragma unroll
  for (int d = 0; d < DEPTH - 1; ++d) fetch(base + d * slot);
  fetch_small(row);
  int at = 0;
  // Every group of a block makes the same number of turns (row_sum's barrier).
  for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < a.rows; r0 += step, row += step, dx += step * a.lddx) {
    const bool here = row < a.rows;
    int next = at + DEPTH - 1;
    if (next >= DEPTH) next -= DEPTH;
    fetch(base + next * slot);
    const float r = here ? rstd : 0.0f;
    float to_n[NV];  // what turns a kept value into n
#pragma unroll
    for (int i = 0; i < NV; ++i) to_n[i] = KEPT ? scale_value(scale[i]) * r : r;
    fetch_small(row + step);
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    const unsigned char* s = ring + at * slot + tid * 16;
    float n[NV][8] = {}, g[NV][8] = {};
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!here || !in[i]) continue;
#pragma unroll
      for (int q = 0; q < kWords; ++q) {
        word(s + (i * kWords + q) * vec_bytes, g[i] + q * kPer);
        if constexpr (!KEPT) word(s + off_h + (i * kWords + q) * vec_bytes, n[i] + q * kPer);
      }
      if constexpr (KEPT) decode8(*reinterpret_cast<const uint2*>(ring + at * slot + off_h + (i * threads + tid) * 8), to_n[i], n[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (!KEPT) n[i][k] *= to_n[i];
        acc[i][k] = fmaf(g[i][k], n[i][k], acc[i][k]);
        g[i][k] *= (float)w[i][k];
        sum = fmaf(g[i][k], n[i][k], sum);
      }
    }
    if (a.dx) {
      const float mean = row_sum(sum, scratch, turn) / (float)a.cols;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!here || !in[i]) continue;
        float d[8] = {};
        if (has_dres) {
#pragma unroll
          for (int q = 0; q < kWords; ++q) word(s + off_dres + (i * kWords + q) * vec_bytes, d + q * kPer);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = fmaf(r, fmaf(-n[i][k], mean, g[i][k]), d[k]);
        store_vec<8>(dx + i * apart, d);
      }
    }
    if (++at == DEPTH) at = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  store_partial<8, NV>(a, acc);
}

// A block takes 32 columns; warp w adds partials w, w + 32, ...
template <typename T>
__global__ void __launch_bounds__(1024) sum_groups_kernel(const float* __restrict__ partial, int64_t groups,
                                                          int64_t cols, T* __restrict__ out) {
  __shared__ float s[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (col < cols) {
    int64_t g = warp;
    for (; g + 7 * 32 < groups; g += 8 * 32) {  // eight loads at a time
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = partial[(g + j * 32) * cols + col];
#pragma unroll
      for (int j = 0; j < 8; ++j) v += t[j];
    }
    for (; g < groups; g += 32) v += partial[g * cols + col];
  }
  s[warp][lane] = v;
  __syncthreads();
  v = s[lane][warp];  // lane l of warp w: column w's sum over warp l's groups
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int64_t o = (int64_t)blockIdx.x * 32 + warp;
  if (lane == 0 && o < cols) {
    const float t[1] = {v};
    store_vec<1>(out + o, t);
  }
}

// How a row is spread: V columns a vector, NV vectors a thread, `threads`
// threads a row, `rows` rows a block.  NV grows with the row so that a block
// stays at 512 threads or fewer where it can (several blocks an SM).
struct RowShape {
  int nv, threads, rows;
};
RowShape row_shape(bool vec, int64_t cols) {
  RowShape s{};
  if (vec)
    s.nv = cols <= 2048 ? 1 : cols <= 8192 ? 2 : 4;
  else
    s.nv = cols <= 1024 ? 4 : cols <= 4096 ? 8 : 16;
  const int64_t each = (int64_t)s.nv * (vec ? 8 : 1);
  s.threads = (int)((cols + each * 32 - 1) / (each * 32) * 32);
  s.rows = std::max(1, 256 / s.threads);
  return s;
}

template <int N>
using Int = std::integral_constant<int, N>;

// f(V, NV, most threads of a block), as constants.
template <typename F>
void with_shape(bool vec, const RowShape& s, F&& f) {
  if (vec)
    s.nv == 1 ? f(Int<8>(), Int<1>(), Int<256>()) : s.nv == 2 ? f(Int<8>(), Int<2>(), Int<512>()) : f(Int<8>(), Int<4>(), Int<512>());
  else
    s.nv == 4 ? f(Int<1>(), Int<4>(), Int<256>()) : s.nv == 8 ? f(Int<1>(), Int<8>(), Int<512>()) : f(Int<1>(), Int<16>(), Int<1024>());
}

template <typename T>
tide_status norm(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.x, a.ldx, sizeof(T), a.rows) &&
                   rows_aligned(a.residual, a.ldr, sizeof(T), a.rows) && rows_aligned(a.h, a.ldh, sizeof(T), a.rows) &&
                   rows_aligned(a.y, a.ldy, sizeof(T), a.rows) && (uintptr_t)a.weight % 16 == 0 &&
                   (uintptr_t)a.codes % 8 == 0 && (!a.codes || a.rows <= 1 || a.ldc % 8 == 0);
  const RowShape s = row_shape(vec, a.cols);
  const int64_t grid = (a.rows + s.rows - 1) / s.rows;
  if (grid > INT32_MAX) return fail(TIDE_ERR_UNIMPLEMENTED, "too many rows for one launch");
  with_shape(vec, s, [&](auto v, auto nv, auto threads) {
    norm_kernel<T, v(), nv(), threads()><<<(unsigned)grid, dim3(s.threads, s.rows), 0, stream>>>(a);
  });
  return cuda_status(cudaGetLastError(), "rms norm");
}

// Blocks of the backward pass: up to `per_sm` an SM, but past 64 row groups at
// least four rows a group, so that the partial sums stay few.
int64_t grad_blocks(int64_t rows, const RowShape& s, int per_sm, int sms) {
  const int64_t most = (rows + s.rows - 1) / s.rows;
  const int64_t few = std::max<int64_t>(64 / s.rows, (rows + 4 * s.rows - 1) / (4 * s.rows));
  return std::min(std::min(most, few), (int64_t)sms * per_sm);
}
int most_per_sm(const RowShape& s) { return std::max(1, 1024 / (s.threads * s.rows)); }

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
  if (a.rows > 0) {
    const RowShape s = row_shape(vec, a.cols);
    const dim3 block(s.threads, s.rows);
    const int slot = ring_slot_bytes(s.threads * s.rows, s.nv, sizeof(T), !a.h, a.dres != nullptr);
    constexpr int kRoom = 200 * 1024;  // shared memory of an SM that rings may take
    const int depth = 4 * slot <= kRoom ? 4 : 2 * slot <= kRoom ? 2 : 0;
    const int per_sm = vec && depth ? std::min(most_per_sm(s), kRoom / (depth * slot)) : most_per_sm(s);
    const int64_t blocks = grad_blocks(a.rows, s, per_sm, sms);
    groups = blocks * s.rows;
    with_shape(vec, s, [&](auto v, auto nv, auto threads) {
      if constexpr (v() == 8) {
        auto ring = [&](auto kernel) {
          const int smem = depth * slot;
          cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
          if (err == cudaSuccess) {
            kernel<<<(unsigned)blocks, block, smem, stream>>>(a);
            err = cudaGetLastError();
          }
          st = cuda_status(err, "rms norm backward");
        };
        // Registers for two blocks an SM where the block is small enough, for
        // one otherwise (with one, 5120 columns took 79 us where two take 57).
        auto pick = [&](auto most, auto min_blocks) {
          constexpr int kT = most(), kB = min_blocks();
          if (depth == 4)
            a.h ? ring(norm_grad_ring_kernel<T, nv(), 4, false, kT, kB>) : ring(norm_grad_ring_kernel<T, nv(), 4, true, kT, kB>);
          else
            a.h ? ring(norm_grad_ring_kernel<T, nv(), 2, false, kT, kB>) : ring(norm_grad_ring_kernel<T, nv(), 2, true, kT, kB>);
        };
        if (depth) {
          if constexpr (nv() == 1) {
            pick(Int<256>(), Int<3>());
          } else if constexpr (nv() == 2) {
            s.threads <= 320 ? pick(Int<320>(), Int<2>()) : pick(Int<512>(), Int<1>());
          } else {
            pick(Int<512>(), Int<1>());
          }
          return;
        }
      }
      norm_grad_kernel<T, v(), nv(), threads()><<<(unsigned)blocks, block, 0, stream>>>(a);
      st = cuda_status(cudaGetLastError(), "rms norm backward");
    });
  }
  if (st == TIDE_OK && dweight)
    st = launch_sum_groups(a.partial, groups, a.cols, sizeof(T) == 2 ? TIDE_BF16 : TIDE_F32, dweight, groups > 0, stream);
  return st;
}

tide_status check_cols(int64_t cols) {
  return cols > kMaxCols ? fail(TIDE_ERR_UNIMPLEMENTED, "rms norm: rows longer than 16384") : TIDE_OK;
}

}  // namespace

tide_status launch_sum_groups(const float* partial, int64_t groups, int64_t cols, int32_t dtype, void* out, bool after,
                              cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((cols + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cuda_status(dtype == TIDE_BF16
                         ? cudaLaunchKernelEx(&cfg, sum_groups_kernel<bf16>, partial, groups, cols, (bf16*)out)
                         : cudaLaunchKernelEx(&cfg, sum_groups_kernel<float>, partial, groups, cols, (float*)out),
                     "joining partial sums");
}

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
  int64_t most = 0;  // whichever the alignment of the call's rows selects
  for (const bool vec : {true, false}) {
    const RowShape s = row_shape(vec, cols);
    most = std::max(most, grad_blocks(rows, s, most_per_sm(s), sms) * s.rows);
  }
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
