// RMS norm with the residual's addition, forward and backward
// (include/tide_ops.h).
//
// Both directions read each input and write each output once, with about ten
// operations per element, so they are bound by memory traffic; a row stays in
// registers (forward) or in shared memory (backward) between its sum and its
// outputs.
//   forward, 16384 x 8192 bf16, residual added, y also in 8 bits (1.21 GB): 175 us,
//   6.9 TB/s
//   backward, 8192 x 5120 bf16 from a checkpoint, dres added (294 MB): 46 us, 6.3
//   TB/s, 49 with dweight's partial sums joined; without dres 4096 x 8192 fp32 67 us,
//   6.0 TB/s, 8192 x 14336 bf16 120 us, 5.9 TB/s
//   4999 x 4095 bf16, rows of odd alignment: forward (82 MB) 31 us, backward (123 MB, 103
//   from a checkpoint) 57 and 56 us, bound by their instructions

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "bulk_ptx.cuh"
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
  int64_t ahead;  // a row's threads ask for the row so many rows on; 0: for none
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
  float* partial;  // [blocks][cols]: each one's sum of dy * n; NULL: not wanted
};

// The threads that share a row: per_row of them (a multiple of 32), this one the
// x-th, of the y-th row of the block; `all` threads work on rows.  Barriers are
// named, so that a warp beside them can do something else.
struct RowThread {
  int per_row, x, y, all;
  __device__ __forceinline__ void sync() const {
    if (per_row > 32)
      asm volatile("bar.sync 1, %0;" ::"r"(all) : "memory");
    else
      __syncwarp();
  }
};
// In a block of (per_row, rows) threads.
__device__ __forceinline__ RowThread row_thread() {
  return {(int)blockDim.x, (int)threadIdx.x, (int)threadIdx.y, (int)(blockDim.x * blockDim.y)};
}

// Sum of v over the threads of a row.  One barrier: `turn` alternates the
// scratch floats, one per warp, so a sum is read before its place is written
// again.  The order is fixed.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}
__device__ __forceinline__ float row_sum(float v, const RowThread& t, float (&scratch)[2][32], int& turn) {
  v = warp_sum(v);
  const int warps = t.per_row / 32;
  if (warps > 1) {
    const int first = t.y * warps, lane = threadIdx.x % 32;
    float* s = scratch[turn];
    turn ^= 1;
    if (lane == 0) s[first + t.x / 32] = v;
    t.sync();
    v = warp_sum(lane < warps ? s[first + lane] : 0.0f);
  }
  return v;
}

// Eight codes of a kept row at any alignment, the first n; the rest as zeros.
__device__ __forceinline__ uint2 load_codes_any(const uint8_t* c, int n) {
  if (n == 8) return (uintptr_t)c % 8 == 0 ? *reinterpret_cast<const uint2*>(c) : load_any_bytes(c);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) w[k / 4] |= (uint32_t)c[k] << (8 * (k % 4));
  return make_uint2(w[0], w[1]);
}

// Rows of any alignment leave through shared memory: threads put their vectors
// down whole, and the row is stored with neighbouring threads on neighbouring
// elements, so in whole sectors.  (Staged at its phase and stored in words of 16
// bytes it was slower: the vectors then go down piece by piece.  So were pairs
// of bf16.)
template <typename T>
__device__ __forceinline__ void store_staged(T* out, const T* staged, int cols, const RowThread& t) {
  for (int c = t.x; c < cols; c += t.per_row) out[c] = staged[c];
}
// Shared memory of a staged row: whole vectors.
__host__ __device__ constexpr int stage_room(int64_t cols, int elem) { return (int)((cols + 7) / 8 * 8 * elem); }

// Asks for a row to be brought to L2.
template <typename T>
__device__ __forceinline__ void prefetch_l2(const T* row, int64_t cols) {
  const uintptr_t from = ((uintptr_t)row + 15) / 16 * 16, end = (uintptr_t)(row + cols) / 16 * 16;
  if (from < end) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"((uint32_t)(end - from)));
}

// A row takes blockDim.x threads, each NV vectors of eight columns; a block
// holds blockDim.y rows.  ANY: rows of any alignment; h and y then leave through shared
// memory.
template <typename T, int NV, bool ANY, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) unsigned char stage[];
  __shared__ float scratch[2][32];
  int turn = 0;
  const RowThread t = row_thread();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + t.y;
  const bool here = row < a.rows;
  const int cols = (int)a.cols;
  T* const h_out = (T*)a.h + row * a.ldh;
  T* const y_out = (T*)a.y + row * a.ldy;
  const int room = stage_room(cols, sizeof(T));
  T* const h_stage = reinterpret_cast<T*>(stage + t.y * 2 * room);
  T* const y_stage = reinterpret_cast<T*>(stage + t.y * 2 * room + room);
  if (a.ahead && t.x == 0 && row < a.rows - a.ahead) {
    prefetch_l2((const T*)a.x + (row + a.ahead) * a.ldx, cols);
    if (a.residual) prefetch_l2((const T*)a.residual + (row + a.ahead) * a.ldr, cols);
  }
  float s[NV][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = ((int)i * (int) blockDim.x + t.x) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) s[i][k] = 0.0f;
    if (here && col < cols) {
      const int n = min(8, cols - col);
      const T* x = (const T*)a.x + row * a.ldx + col;
      if constexpr (ANY)
        load_any8(x, n, s[i]);
      else
        load_vec<8>(x, s[i]);
      if (a.residual) {
        const T* q = (const T*)a.residual + row * a.ldr + col;
        float r[8];
        if constexpr (ANY)
          load_any8(q, n, r);
        else
          load_vec<8>(q, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[i][k] += r[k];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = fmaf(s[i][k], s[i][k], sum);
  sum = row_sum(sum, t, scratch, turn);
  const float rstd = 1.0f / sqrtf(sum / (float)cols + a.eps);
  if (here && t.x == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = ((int)i * (int) blockDim.x + t.x) * 8;
    const int n = here ? max(0, min(8, cols - col)) : 0;
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = 0.0f;
    if (n > 0) {
      const T* w = (const T*)a.weight + col;
      if constexpr (ANY)
        load_any8(w, n, y);
      else
        load_vec<8>(w, y);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= s[i][k] * rstd;
      if constexpr (ANY) {
        store_vec<8>(h_stage + col, s[i]);
        store_vec<8>(y_stage + col, y);
      } else {
        if (a.h) store_vec<8>(h_out + col, s[i]);
        if (a.y) store_vec<8>(y_out + col, y);
      }
    }
    if (a.codes) {
      const int byte = scale_byte(block_magnitude<4>(y));
      uint32_t w[2];
      encode(y, byte, w);
      uint8_t* c = a.codes + row * a.ldc + col;
      if constexpr (ANY)
        store_codes_any(c, n, w);
      else if (n > 0)
        *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
      if (n > 0 && col % kMxBlock == 0) a.scales[row * a.lds + col / kMxBlock] = (uint8_t)byte;
    }
  }
  if constexpr (ANY) {
    t.sync();
    if (!here) return;
    if (a.h) store_staged(h_out, h_stage, cols, t);
    if (a.y) store_staged(y_out, y_stage, cols, t);
  }
}

// ---- backward
//
// Row groups (per_row threads) walk the rows with a fixed stride, so a thread
// keeps its columns' weights and their share of dweight in registers.  Within a
// row each thread has NV vectors of eight columns.

// Eight elements of T as they lie in memory.
template <typename T>
struct Kept8 {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ float value(int k) const {
    if constexpr (sizeof(T) == 2)
      return __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    else
      return __uint_as_float(w[k]);
  }
  // The first n at p, one by one; zeros for the rest.
  __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
    for (int k = 0; k < 2 * (int)sizeof(T); ++k) w[k] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= n) continue;
      if constexpr (sizeof(T) == 2)
        w[k / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[k] << (16 * (k % 2));
      else
        w[k] = reinterpret_cast<const uint32_t*>(p)[k];
    }
  }
};

// The block's share of dweight to its row of `partial`; with several rows a block
// they are joined in `joined`, [rows][cols], first.
template <int NV>
__device__ __forceinline__ void store_partial(const NormGradArgs& a, const RowThread& t, int rows,
                                              const float (&acc)[NV][8], float* joined) {
  if (!a.partial) return;
  const int cols = (int)a.cols;
  float* out = a.partial + (int64_t)blockIdx.x * cols;
  if (rows > 1) asm volatile("bar.sync 1, %0;" ::"r"(t.all) : "memory");  // what was there has been read
  float* p = rows > 1 ? joined + t.y * cols : out;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * t.per_row + t.x) * 8;
    if (cols % 4 == 0 && col + 8 <= cols) {
      store_vec<8>(p + col, acc[i]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < cols) p[col + k] = acc[i][k];
    }
  }
  if (rows == 1) return;
  asm volatile("bar.sync 1, %0;" ::"r"(t.all) : "memory");
  for (int c = t.y * t.per_row + t.x; c < cols; c += t.all) {
    float v = 0.0f;
    for (int y = 0; y < rows; ++y) v += joined[y * cols + c];
    out[c] = v;
  }
}

// Before the row's mean is known: n (from h times to_n), dweight's share,
// g = dy * weight and this thread's part of the sum of g * n.
template <typename T>
__device__ __forceinline__ float grad_vector(float (&n)[8], float (&g)[8], float to_n, const Kept8<T>& w,
                                             float (&acc)[8], float sum) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    n[k] *= to_n;
    acc[k] = fmaf(g[k], n[k], acc[k]);
    g[k] *= w.value(k);
    sum = fmaf(g[k], n[k], sum);
  }
  return sum;
}

// ---- the backward pass through a ring of rows
//
// DEPTH rows of every group lie in shared memory, copied there whole (dy, dres,
// h or its codes and scales, rstd) by bulk copies, so that a row costs the
// threads that compute its one barrier and no memory latency, and no address
// arithmetic.  A warp of its own issues them, lane y for the block's y-th row,
// once every warp has said that it is done with the slot.

// The part of a row of `bytes` at `from` that whole granules of 16 bytes cover:
// `skip` bytes after from's granule, the returned number of bytes.  Granules
// reach up to 15 bytes past the row on either side; one that would begin before
// the matrix's first byte or end after its last is left out.
__device__ __forceinline__ uint32_t row_span(const unsigned char* from, int64_t bytes, const unsigned char* first,
                                             const unsigned char* last, uint32_t& skip) {
  const uintptr_t f = (uintptr_t)from, lo = f & ~(uintptr_t)15, hi = (f + bytes + 15) & ~(uintptr_t)15;
  const uintptr_t l = lo < (uintptr_t)first ? lo + 16 : lo, h = hi > (uintptr_t)last ? hi - 16 : hi;
  skip = (uint32_t)(l - lo);
  return h > l ? (uint32_t)(h - l) : 0u;
}

// Copies a row of a matrix (`at`, of cols * elem bytes) to `to` plus its phase
// within 16 bytes; returns the bytes that will count on `bar`.  What no granule
// covers goes byte by byte.  withheld (tests): the counted bytes never come.
__device__ __forceinline__ uint32_t copy_row(unsigned char* to, const unsigned char* at, const void* base, int64_t rows,
                                             int64_t cols, int64_t ld, int elem, bool withheld, uint64_t* bar) {
  const unsigned char* first = (const unsigned char*)base;
  const unsigned char* end = at + cols * elem;
  uint32_t skip;
  const uint32_t n = row_span(at, cols * elem, first, first + ((rows - 1) * ld + cols) * elem, skip);
  const unsigned char* lo = (const unsigned char*)((uintptr_t)at & ~(uintptr_t)15);
  if (n && !withheld) bulk_load(to + skip, lo + skip, n, bar);
  for (const unsigned char* q = at; q < lo + skip && q < end; ++q) to[q - lo] = *q;
  for (const unsigned char* q = at < lo + skip + n ? lo + skip + n : at; q < end; ++q) to[q - lo] = *q;
  return n;
}

// Copies in flight are waited for so long, however short the limit on waits: a
// millisecond is ample for them.
constexpr uint64_t kDrainNs = 1000000;

struct RingArgs {
  NormGradArgs g;
  int32_t per_row, rows;
  int32_t dres_passes;  // dres is read from where it is
  uint32_t* timeouts;
  uint64_t wait_limit_ns;
  int64_t test_drop;  // turn (counted per block) whose copies are withheld (tests); -1: none
};

// A row in the ring, with room for its phase within 16 bytes.
__host__ __device__ constexpr int ring_room(int64_t cols, int elem) { return (int)((cols * elem + 15) / 16 * 16) + 16; }

// A row's part of a slot: where each of the others lies in it, with its phase
// (five words), then dy, dres, h or codes, scales and rstd.
enum RingPart { AT_DY, AT_DRES, AT_H, AT_SCALES, AT_RSTD };
struct RingRow {
  int dy, dres, h, scales, rstd, bytes;
  __host__ __device__ constexpr RingRow(int64_t cols, int elem, bool kept, bool has_dres)
      : dy(32),
        dres(dy + ring_room(cols, elem)),
        h(dres + (has_dres ? ring_room(cols, elem) : 0)),
        scales(h + ring_room(cols, kept ? 1 : elem)),
        rstd(scales + (kept ? ring_room((cols + kMxBlock - 1) / kMxBlock, 1) : 0)),
        bytes(rstd + 32) {}
};

template <typename T, int NV, int DEPTH, bool KEPT, bool ANY, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) norm_grad_ring_kernel(const RingArgs p) {
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float scratch[2][32];
  __shared__ uint64_t full[DEPTH], empty[DEPTH];
  const NormGradArgs& a = p.g;
  constexpr int kElem = sizeof(T);
  // With so many threads registers are few: the row is read from its slot again when
  // its mean is known (8192 x 14336 bf16 174 us without, 118 with).
  constexpr bool kReload = THREADS > 288;
  // Rows so long that dres may have no room in the ring.
  constexpr bool kMayPass = kReload || (NV == 4 && ANY && !KEPT && kElem == 4);
  const bool has_dres = a.dres != nullptr, ring_dres = has_dres && !(kMayPass && p.dres_passes);
  const int cols = (int)a.cols, rows = p.rows, workers = p.per_row * rows;
  const RingRow part(cols, kElem, KEPT, ring_dres);
  const int slot_bytes = rows * part.bytes;
  const int64_t step = (int64_t)gridDim.x * rows, first_row = (int64_t)blockIdx.x * rows;

  if (threadIdx.x == 0) {
    for (int d = 0; d < DEPTH; ++d) {
      mbar_init(full + d, rows);
      mbar_init(empty + d, workers / 32);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  // Copies the block's y-th row of a turn (`row`) into a slot.
  auto issue = [&](int y, int64_t row, int slot, bool withheld) {
    uint32_t bytes = 0;
    if (row < a.rows) {
      unsigned char* to = ring + slot * slot_bytes + y * part.bytes;
      uint64_t* bar = full + slot;
      fence_proxy_async_smem();
      auto one = [&](RingPart which, const void* base, int64_t n, int64_t ld, int elem, int where) {
        const unsigned char* at = (const unsigned char*)base + row * ld * elem;
        reinterpret_cast<int*>(to)[which] = where + (int)((uintptr_t)at & 15);
        bytes += copy_row(to + where, at, base, a.rows, n, ld, elem, withheld, bar);
      };
      one(AT_DY, a.dy, cols, a.lddy, kElem, part.dy);
      if (ring_dres)
        one(AT_DRES, a.dres, cols, a.ldres, kElem, part.dres);
      else if (has_dres)
        prefetch_l2((const T*)a.dres + row * a.ldres, cols);
      if constexpr (KEPT) {
        one(AT_H, a.codes, cols, a.ldc, 1, part.h);
        one(AT_SCALES, a.scales, (cols + kMxBlock - 1) / kMxBlock, a.lds, 1, part.scales);
      } else {
        one(AT_H, a.h, cols, a.ldh, kElem, part.h);
      }
      one(AT_RSTD, a.rstd, 1, 1, 4, part.rstd);
    }
    // After the bytes moved one by one; the counted ones may land before they
    // are expected.
    mbar_arrive_expect_tx(full + slot, bytes);
  };

  const int turns = (int)((a.rows - first_row + step - 1) / step);
  if ((int)threadIdx.x >= workers) {
    const int y = (int)threadIdx.x - workers;
    if (y >= rows) return;
    bool ok = true;
    int slot = 0, k = 0;
    for (; k < turns; ++k) {
      if (k >= DEPTH && !(ok = mbar_wait_bounded(empty + slot, (uint32_t)(k / DEPTH - 1) & 1, p.wait_limit_ns))) break;
      issue(y, first_row + y + k * step, slot, k == p.test_drop);
      if (++slot == DEPTH) slot = 0;
    }
    if (!ok) atomicAdd(p.timeouts, 1u);
    // What was asked for lands before the block, and its shared memory, is gone: also
    // where the threads that compute have given up and wait for nothing more.
    const uint64_t limit = p.wait_limit_ns > kDrainNs ? p.wait_limit_ns : kDrainNs;
    for (int d = 0; d < DEPTH && d < k; ++d)
      mbar_wait_bounded(full + d, (uint32_t)((k - d + DEPTH - 1) / DEPTH - 1) & 1, limit);
    return;
  }

  const int t_y = (int)threadIdx.x / p.per_row;
  const RowThread t{p.per_row, (int)threadIdx.x - t_y * p.per_row, t_y, workers};
  const int col0 = t.x * 8, apart = p.per_row * 8;
  const float inv_cols = 1.0f / (float)cols;
  float acc[NV][8] = {};
  Kept8<T> w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i].load((const T*)a.weight + col0 + i * apart, min(8, cols - (col0 + i * apart)));
  // Every group of a block makes the same number of turns (the row's barriers);
  // this one has rows in the first `mine`.
  const int mine = (int)((a.rows - (first_row + t.y) + step - 1) / step);
  T* dx = (T*)a.dx + (first_row + t.y) * a.lddx;
  const T* dres = (const T*)a.dres + (first_row + t.y) * a.ldres;
  T* const staged = reinterpret_cast<T*>(ring + DEPTH * slot_bytes + t.y * stage_room(cols, kElem));  // ANY: dx
  int turn = 0, slot = 0;
  uint32_t phase = 0;
  bool late = false;
  for (int k = 0; k < turns; ++k) {
    const unsigned char* from = ring + slot * slot_bytes + t.y * part.bytes;
    const int* at = reinterpret_cast<const int*>(from);
    if (!late && !mbar_wait_bounded(full + slot, phase, p.wait_limit_ns)) late = true;
    const bool here = !late && k < mine;  // nothing of a slot is read that did not come
    float n[kReload ? 1 : NV][8], g[kReload ? 1 : NV][8];
    float sum = 0.0f, rstd = 0.0f;
    if (here) rstd = *reinterpret_cast<const float*>(from + at[AT_RSTD]);
    // h and dy of vector i, and what turns a value of h into n.
    auto fetch = [&](int col, float (&n)[8], float (&g)[8]) {
      const T* dy = reinterpret_cast<const T*>(from + (ANY ? at[AT_DY] : part.dy)) + col;
      const unsigned char* h = from + (ANY || KEPT ? at[AT_H] : part.h) + col * (KEPT ? 1 : kElem);
      float to_n = rstd;
      if constexpr (KEPT) to_n *= scale_value(from[at[AT_SCALES] + col / kMxBlock]);
      if constexpr (ANY) {
        const int m = min(8, cols - col);
        load_any8(dy, m, g);
        if constexpr (KEPT)
          decode8(load_codes_any(h, m), 1.0f, n);
        else
          load_any8(reinterpret_cast<const T*>(h), m, n);
      } else {
        load_vec<8>(dy, g);
        if constexpr (KEPT)
          decode8(*reinterpret_cast<const uint2*>(h), 1.0f, n);
        else
          load_vec<8>(reinterpret_cast<const T*>(h), n);
      }
      return to_n;
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float (&ni)[8] = n[kReload ? 0 : i];
      float (&gi)[8] = g[kReload ? 0 : i];
#pragma unroll
      for (int j = 0; j < 8; ++j) ni[j] = gi[j] = 0.0f;
      const int col = col0 + i * apart;
      if (!here || col >= cols) continue;
      const float to_n = fetch(col, ni, gi);
      sum = grad_vector(ni, gi, to_n, w[i], acc[i], sum);
    }
    const float mean = row_sum(sum, t, scratch, turn) * inv_cols;
    if (a.dx) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = col0 + i * apart;
        if (!here || col >= cols) continue;
        float (&ni)[8] = n[kReload ? 0 : i];
        float (&gi)[8] = g[kReload ? 0 : i];
        if constexpr (kReload) {
          const float to_n = fetch(col, ni, gi);
#pragma unroll
          for (int j = 0; j < 8; ++j) ni[j] *= to_n, gi[j] *= w[i].value(j);
        }
        float d[8] = {};
        if (ring_dres) {
          const T* q = reinterpret_cast<const T*>(from + (ANY ? at[AT_DRES] : part.dres)) + col;
          if constexpr (ANY)
            load_any8(q, min(8, cols - col), d);
          else
            load_vec<8>(q, d);
        } else if (kMayPass && has_dres) {
          const T* q = dres + col;
          if constexpr (ANY)
            load_any8(q, min(8, cols - col), d);
          else
            load_vec<8>(q, d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, fmaf(-ni[j], mean, gi[j]), d[j]);
        if constexpr (ANY)
          store_vec<8>(staged + col, d);
        else
          store_vec<8>(dx + col, d);
      }
    }
    __syncwarp();
    // After a wait that ran out no slot is handed back, so the copies end too.
    if (!late && threadIdx.x % 32 == 0) mbar_arrive(empty + slot);
    if constexpr (ANY) {
      if (a.dx) {
        t.sync();
        if (here) store_staged(dx, staged, cols, t);
        if (p.per_row == 32) __syncwarp();  // row_sum has no barrier then
      }
    }
    dx += step * a.lddx;
    dres += step * a.ldres;
    if (++slot == DEPTH) slot = 0, phase ^= 1;
  }
  if (late) atomicAdd(p.timeouts, 1u);
  store_partial(a, t, rows, acc, reinterpret_cast<float*>(ring));
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

// How a row is spread: NV vectors of eight columns a thread, `threads` threads a
// row, `rows` rows a block, and, in the backward pass, the blocks an SM that its
// registers are bounded to.
struct RowShape {
  int nv, threads, rows, per_sm;
};
constexpr RowShape spread(int64_t cols, int nv) {
  const int64_t each = (int64_t)nv * 8 * 32;
  const int threads = (int)((cols + each - 1) / each * 32);
  return {nv, threads, std::max(1, 256 / threads), 1};
}
// Forward: NV grows with the row so that a block stays at 512 threads or fewer
// (several blocks an SM).
RowShape forward_shape(int64_t cols) { return spread(cols, cols <= 2048 ? 1 : cols <= 8192 ? 2 : 4); }
// Backward: the row's barrier and the latencies around it bind, so few threads
// with much independent work each: four vectors beat two from 2048 columns on
// (8192 x 5120 from a checkpoint 50 us against 63, 8192 x 8192 88 against 96).  More
// than 16 warps, the copying one among them, leave a thread 96 registers, 16 leave it
// 128 (8192 x 10240 bf16 96 us with 10 to 15 working warps, 130 in a kernel bounded
// to 16); hence five vectors for the longest rows.
constexpr RowShape backward_shape(int64_t cols) {
  RowShape s = spread(cols, cols <= 512 ? 1 : cols <= 2048 ? 2 : cols <= 480 * 32 ? 4 : 5);
  if (s.nv >= 4) s.rows = 1;
  s.per_sm = s.nv == 1 ? 3 : s.nv == 2 || (s.nv == 4 && s.threads <= 160) ? 2 : 1;
  return s;
}

// The ring of a call: its depth and the shared memory it takes, dx's staged rows
// included; whether dres is left out of it.
struct Ring {
  int depth, smem;
  bool passes;
};
constexpr int kRingRoom = 208 * 1024;  // shared memory of an SM that rings may take

// Four rows, or two; without dres where two do not fit with it; one of fp32 rows that
// are too long for that (h plain: from 13304 columns, or 10641 if rows are not
// aligned; h from a checkpoint: from 15129 if not aligned).
constexpr Ring ring_of(const RowShape& s, int64_t cols, int elem, bool kept, bool any, bool has_dres) {
  const int beside = any ? s.rows * stage_room(cols, elem) : 0;
  for (int depth = s.threads <= 256 ? 4 : 2; depth > 0; depth /= 2) {
    for (const bool with_dres : {true, false}) {
      if (!with_dres && depth == 4) continue;
      if (with_dres && depth == 1) continue;
      const int smem = depth * s.rows * RingRow(cols, elem, kept, with_dres && has_dres).bytes + beside;
      if (smem * (depth == 4 ? s.per_sm : 1) <= kRingRoom) return {depth, smem, has_dres && !with_dres};
    }
  }
  return {0, 0, false};
}

// Whether some row of NV vectors and more than LEAST, at most MOST threads has a ring
// of so many rows.  For each number of threads: its shortest row takes the deepest,
// its longest the shallowest.
constexpr bool ring_taken(int nv, int least, int most, int elem, bool kept, bool any, int depth) {
  for (int threads = least + 32; threads <= most; threads += 32) {
    const int64_t longest = (int64_t)threads * nv * 8 < kMaxCols ? (int64_t)threads * nv * 8 : kMaxCols;
    const int64_t shortest = (int64_t)(threads - 32) * nv * 8 + (any ? 1 : 8);
    const RowShape s = backward_shape(longest), t = backward_shape(shortest);
    if (s.nv != nv || t.nv != nv || s.threads != threads || t.threads != threads) continue;
    if (ring_of(s, longest, elem, kept, any, true).depth <= depth &&
        depth <= ring_of(t, shortest, elem, kept, any, false).depth)
      return true;
  }
  return false;
}

template <int N>
using Int = std::integral_constant<int, N>;

// f(NV, most threads of a block that work on rows, blocks an SM), as constants.
template <typename F>
void with_forward_shape(const RowShape& s, F&& f) {
  if (s.nv == 1)
    f(Int<1>(), Int<256>());
  else if (s.nv == 2)
    f(Int<2>(), Int<512>());
  else
    f(Int<4>(), Int<512>());
}
// Here also the fewest threads a row, less one warp.
template <typename F>
void with_backward_shape(const RowShape& s, F&& f) {
  if (s.nv == 1)
    f(Int<1>(), Int<0>(), Int<256>(), Int<3>());
  else if (s.nv == 2)
    f(Int<2>(), Int<0>(), Int<256>(), Int<2>());
  else if (s.nv == 5)
    f(Int<5>(), Int<0>(), Int<416>(), Int<1>());
  else if (s.threads <= 160)
    f(Int<4>(), Int<0>(), Int<160>(), Int<2>());
  else if (s.threads <= 256)
    f(Int<4>(), Int<160>(), Int<256>(), Int<1>());
  else
    f(Int<4>(), Int<256>(), Int<480>(), Int<1>());
}

// Raises a kernel's dynamic shared memory limit as far as it goes, once for each
// thread, kernel and device.
tide_status allow_smem(const void* kernel, const char* what) {
  struct Done {
    const void* kernel;
    int dev;
  };
  static thread_local Done done[128];
  static thread_local int count = 0;
  int dev = 0, most = 0;
  TIDE_TRY(cuda_status(cudaGetDevice(&dev), what));
  for (int i = 0; i < count; ++i)
    if (done[i].kernel == kernel && done[i].dev == dev) return TIDE_OK;
  cudaFuncAttributes attr;
  TIDE_TRY(cuda_status(cudaFuncGetAttributes(&attr, kernel), what));
  TIDE_TRY(cuda_status(cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev), what));
  TIDE_TRY(cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            most - (int)attr.sharedSizeBytes), what));
  if (count < 128) done[count++] = {kernel, dev};
  return TIDE_OK;
}

// Launches with `smem` bytes of dynamic shared memory.
template <typename... Params, typename... Args>
tide_status launch(void (*kernel)(Params...), int64_t grid, dim3 threads, int smem, cudaStream_t stream, const char* what,
                   const Args&... args) {
  if (smem > 32 * 1024) TIDE_TRY(allow_smem((const void*)kernel, what));  // 48 KB, static included, need no leave
  kernel<<<(unsigned)grid, threads, smem, stream>>>(args...);
  return cuda_status(cudaGetLastError(), what);
}

template <typename T>
tide_status norm(NormArgs a, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.x, a.ldx, sizeof(T), a.rows) &&
                   rows_aligned(a.residual, a.ldr, sizeof(T), a.rows) && rows_aligned(a.h, a.ldh, sizeof(T), a.rows) &&
                   rows_aligned(a.y, a.ldy, sizeof(T), a.rows) && (uintptr_t)a.weight % 16 == 0 &&
                   (uintptr_t)a.codes % 8 == 0 && (!a.codes || a.rows <= 1 || a.ldc % 8 == 0);
  const RowShape s = forward_shape(a.cols);
  const int64_t grid = (a.rows + s.rows - 1) / s.rows;
  if (grid > INT32_MAX) return fail(TIDE_ERR_UNIMPLEMENTED, "too many rows for one launch");
  const dim3 block(s.threads, s.rows);
  const int stage = s.rows * 2 * stage_room(a.cols, sizeof(T));
  // Rows are asked for kAheadBytes early: registers hold few rows, and those of
  // bf16 are less than DRAM's latency asks for (8192 x 8192 62 us without, 50 with; with
  // the residual and codes 101 and 91).  Where that is no further than the rows at
  // work, or there are few rows, it does not help, and L2 does not hold 20 MB of rows
  // to come beside the outputs (168 us became 185 for fp32 with the residual).
  constexpr int64_t kAheadBytes = 10 << 20;
  const int64_t at_work = (int64_t)ops_num_sms() * std::max(1, 1024 / (s.threads * s.rows)) * s.rows;
  a.ahead = kAheadBytes / (a.cols * (int64_t)sizeof(T) * (a.residual ? 2 : 1));
  if (a.ahead < at_work || a.rows < 4 * a.ahead) a.ahead = 0;
  tide_status st = TIDE_OK;
  with_forward_shape(s, [&](auto nv, auto threads) {
    st = vec ? launch(norm_kernel<T, nv(), false, threads()>, grid, block, 0, stream, "rms norm", a)
             : launch(norm_kernel<T, nv(), true, threads()>, grid, block, stage, stream, "rms norm", a);
  });
  return st;
}

// Blocks of the backward pass: up to `per_sm` an SM, but past 64 at least four
// turns a block, so that the partial sums stay few.
int64_t grad_blocks(int64_t rows, const RowShape& s, int per_sm, int sms) {
  const int64_t most = (rows + s.rows - 1) / s.rows;
  const int64_t few = std::max<int64_t>(64, (rows + 4 * s.rows - 1) / (4 * s.rows));
  return std::min(std::min(most, few), (int64_t)sms * per_sm);
}

template <typename T>
tide_status norm_grad(NormGradArgs a, void* dweight, cudaStream_t stream) {
  const int sms = ops_num_sms();
  if (sms <= 0) return fail(TIDE_ERR_CUDA, "the current device could not be queried");
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.dy, a.lddy, sizeof(T), a.rows) &&
                   rows_aligned(a.h, a.ldh, sizeof(T), a.rows) && rows_aligned(a.dres, a.ldres, sizeof(T), a.rows) &&
                   rows_aligned(a.dx, a.lddx, sizeof(T), a.rows) && (uintptr_t)a.codes % 8 == 0 &&
                   (a.h || a.rows <= 1 || a.ldc % 8 == 0);
  tide_status st = TIDE_OK;
  int64_t groups = 0;
  if (a.rows > 0) {
    const RowShape s = backward_shape(a.cols);
    const char* what = "rms norm backward";
    const bool kept = !a.h;
    const Ring ring = ring_of(s, a.cols, sizeof(T), kept, !vec, a.dres != nullptr);
    const int64_t blocks = grad_blocks(a.rows, s, std::max(1, std::min(s.per_sm, kRingRoom / ring.smem)), sms);
    const int with_copies = s.threads * s.rows + 32;
    groups = blocks;
    RingArgs r{a, s.threads, s.rows, ring.passes, nullptr, ops_wait_limit_ns(), ops_test_drop()};
    TIDE_TRY(ops_timeouts(&r.timeouts));
    bool built = false;
    with_backward_shape(s, [&](auto nv, auto least, auto most, auto per_sm) {
      auto go = [&](auto d, auto k, auto any) {
        if constexpr (ring_taken(nv(), least(), most(), sizeof(T), k(), any(), d())) {
          if (ring.depth != d() || kept != k() || vec == any()) return;
          built = true;
          st = launch(norm_grad_ring_kernel<T, nv(), d(), k(), any(), most() + 32, per_sm()>, blocks, with_copies, ring.smem,
                      stream, what, r);
        }
      };
      auto depths = [&](auto k, auto any) { go(Int<4>(), k, any), go(Int<2>(), k, any), go(Int<1>(), k, any); };
      depths(std::false_type(), std::false_type()), depths(std::false_type(), std::true_type());
      depths(std::true_type(), std::false_type()), depths(std::true_type(), std::true_type());
    });
    if (!built) return fail(TIDE_ERR_UNIMPLEMENTED, "rms norm backward: no kernel for rows of this length");
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
  static std::atomic<int> known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed) > 0) return known[dev].load(std::memory_order_relaxed);
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
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
  const NormArgs a{rows, cols, x,   ldx,  residual, ldr,      weight, eps,       h,
                   ldh,  y,    ldy, rstd, codes,    ld_codes, scales, ld_scales, 0};
  return dtype == TIDE_BF16 ? norm<bf16>(a, (cudaStream_t)stream) : norm<float>(a, (cudaStream_t)stream);
}

int64_t tide_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || cols > kMaxCols) return 0;
  const int sms = ops_num_sms();
  const RowShape s = backward_shape(cols);
  return grad_blocks(rows, s, s.per_sm, sms) * cols * 4;
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
