// Log probabilities of given tokens, entropy and alternatives, and their gradient
// (include/tide_lm_ops.h).
//
// Forward: one pass over a row.  Each thread keeps the largest logit m it has met
// and, over its own logits, S = sum 2^d and E = sum 2^d d with d = (logit - m) scale
// log2(e); when m grows by -D / (scale log2 e), S becomes S 2^D and E becomes 2^D (E + S D).
// The threads' (m, S, E) are joined by the same rule, and
//   lse = scale m + ln S,   entropy = ln S - ln 2 E / S  (no cancellation: E <= 0),
//   logp = scale (logit - m) - ln S.
// Alternatives: each thread also keeps the first vector of eight in which its largest
// logit stood.  The `top` threads with the largest such (logit, vector) pairs are the only ones
// that can hold any of the `top` largest logits: against a logit of another thread there are
// `top` larger ones.  So only those threads' logits, 1 / 25 of a row or less, are read again (L2
// has them), by whole warps that keep a sorted list of 32 in their lanes.
//
// Backward: element by element, one exponential each.

#include <algorithm>
#include <cmath>

#include "cluster_ptx.cuh"
#include "lm_common.cuh"

namespace tide {
namespace {

constexpr int kMaxTop = 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// 2^kLeast is 0 in fp32: exponents are kept from -inf, which times 0 would be NaN.
constexpr float kLeast = -200.0f;
constexpr float kLowest = -3.402823466e38f;

struct LogProbArgs {
  int64_t rows, vocab;
  const void* logits;
  int64_t ldl;
  float scale;
  int32_t index;
  const void* targets;
  float *logp, *lse, *entropy;
  int32_t top;
  float* top_logp;
  int64_t ld_logp;
  int32_t* top_tokens;
  int64_t ld_tokens;
};

__device__ __forceinline__ float exp2_of(float d) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

// What a set of logits leaves: the largest, and the sums over it (none: m is the lowest
// number, S and E are 0).  An infinite or NaN logit makes S NaN.
struct Sums {
  float m = kLowest, s = 0.0f, e = 0.0f;
  __device__ __forceinline__ void raise(float to, float k) {
    const float d = fmaxf((m - to) * k, kLeast), f = exp2_of(d);
    e = f * fmaf(s, d, e);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void join(Sums o, float k) {
    if (o.m > m)
      raise(o.m, k);
    else
      o.raise(m, k);
    s += o.s;
    e += o.e;
  }
};

// ---- alternatives: keys that order logits, larger first, ties by the lower place

__device__ __forceinline__ uint32_t ordered(float v) {
  v = fmaxf(v, -INFINITY) + 0.0f;  // NaN as -inf, -0 as 0
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t place) { return (uint64_t)ordered(v) << 32 | (uint32_t)~place; }

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t smaller(uint64_t a, uint64_t b) { return a < b ? a : b; }

// One exchange of a bitonic network over the warp: lanes j apart, the larger key to the lower
// lane where `down`.
__device__ __forceinline__ uint64_t exchange(uint64_t key, int j, bool down) {
  const uint64_t other = __shfl_xor_sync(0xffffffffu, key, j);
  const bool low = (threadIdx.x & j) == 0;
  return low == down ? larger(key, other) : smaller(key, other);
}
__device__ __forceinline__ uint64_t sort_down(uint64_t key) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) key = exchange(key, j, (threadIdx.x & k) == 0 || k == 32);
  return key;
}
// The 32 largest of two lists sorted downwards over the lanes, the second one given backwards.
__device__ __forceinline__ uint64_t merge_down(uint64_t list, uint64_t backwards) {
  list = larger(list, backwards);
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) list = exchange(list, j, true);
  return list;
}

// The row's list, in its first warp, from one list a warp.
template <int WARPS>
__device__ __forceinline__ uint64_t merge_warps(uint64_t list, uint64_t (&lists)[WARPS][32]) {
  if constexpr (WARPS > 1) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    lists[warp][lane] = list;
    __syncthreads();
#pragma unroll
    for (int step = 1; step < WARPS; step <<= 1) {
      if (warp % (2 * step) == 0 && warp + step < WARPS) {
        list = merge_down(list, lists[warp + step][31 - lane]);
        lists[warp][lane] = list;
      }
      __syncthreads();
    }
  }
  return list;
}

// PER_ROW threads share a row (a warp, or a whole block), or those of a cluster of
// blocks; a block of warps takes eight rows.
template <typename T, int PER_ROW, bool CLUSTER, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(PER_ROW == 32 ? 256 : PER_ROW, PER_ROW == 512 ? 2 : 4)
    log_probs_kernel(const LogProbArgs a) {
  constexpr int WARPS = PER_ROW / 32, kAhead = sizeof(T) == 2 ? 4 : 2;
  __shared__ float stat[3][WARPS];
  __shared__ uint64_t lists[TOP ? WARPS : 1][32];
  __shared__ uint64_t bound;
  const uint32_t blocks = CLUSTER ? cluster_size() : 1, rank = CLUSTER ? cluster_rank() : 0;
  const int64_t row = PER_ROW == 32 ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : (int64_t)(blockIdx.x / blocks);
  if (row >= a.rows) return;  // a whole warp, of rows of one
  const int x = threadIdx.x % PER_ROW, warp = x / 32, lane = x % 32;
  const int64_t vocab = a.vocab;
  const T* const logits = (const T*)a.logits + row * a.ldl;
  const float k = a.scale * kLog2e;
  // Vectors of the row that are whole: from `lo` to below `hi`.
  const int phase = row_phase(logits), count = (int)((vocab + phase + 7) / 8);
  const int lo = phase > 0, hi = (int)((vocab + phase) / 8);
  const int64_t stride = (int64_t)PER_ROW * blocks, first = (int64_t)rank * PER_ROW + x;

  int target = -1;
  float target_logit = 0.0f;
  if (x == 0 && rank == 0 && a.targets) {
    target = token_at(a.targets, a.index, row, vocab);
    if (target >= 0) target_logit = (float)logits[target];
  }

  Sums sums;
  float best = -INFINITY;
  int64_t best_at = first;
  for (int64_t v = first; v < count; v += kAhead * stride) {
    Raw8<T> r[kAhead];
    if (v >= lo && v + (kAhead - 1) * stride < hi) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) r[j].load(logits + (v + j * stride) * 8 - phase);
    } else {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t at = v + j * stride;
        if (at >= lo && at < hi)
          r[j].load(logits + at * 8 - phase);
        else
          r[j].load_some(logits, at * 8 - phase, vocab);
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      float most = r[j].value(0);
#pragma unroll
      for (int i = 1; i < 8; ++i) most = fmaxf(most, r[j].value(i));
      if constexpr (TOP) {
        if (most > best) best = most, best_at = v + j * stride;
      }
      if (most > sums.m) sums.raise(most, k);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = (r[j].value(i) - sums.m) * k, p = exp2_of(d);
        sums.s += p;
        if constexpr (ENTROPY) sums.e = fmaf(p, fmaxf(d, kLeast), sums.e);
      }
    }
  }

#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    Sums o;
    o.m = __shfl_xor_sync(0xffffffffu, sums.m, d);
    o.s = __shfl_xor_sync(0xffffffffu, sums.s, d);
    o.e = __shfl_xor_sync(0xffffffffu, sums.e, d);
    // Both lanes of a pair add the same two in the same order.
    Sums& lower = lane & d ? o : sums;
    Sums& upper = lane & d ? sums : o;
    lower.join(upper, k);
    sums = lower;
  }
  if constexpr (WARPS > 1) {
    if (lane == 0) stat[0][warp] = sums.m, stat[1][warp] = sums.s, stat[2][warp] = sums.e;
  }

  uint64_t key = 0, list = 0;
  if constexpr (TOP) {
    key = first < count ? key_of(best, (uint32_t)best_at) : 0;
    list = merge_warps(sort_down(key), lists);
    if constexpr (CLUSTER) {
      cluster_sync();
      if (warp == 0) {
        for (uint32_t b = 0; b < blocks; ++b)
          if (b != rank) list = merge_down(list, load_peer_u64(peer_smem(&lists[0][31 - lane], b)));
      }
      cluster_sync();  // the lists are written again below
    }
    const uint64_t least = __shfl_sync(0xffffffffu, list, a.top - 1);
    if constexpr (WARPS > 1) {
      if (x == 0) bound = least;
      __syncthreads();
    } else {
      bound = 0;  // not used
    }
    const uint64_t from = WARPS > 1 ? bound : least;
    list = 0;
    for (uint32_t mine = __ballot_sync(0xffffffffu, key != 0 && key >= from); mine; mine &= mine - 1) {
      const int64_t start = first - lane + (__ffs(mine) - 1);  // that thread's first vector
      for (int64_t v = start; v < count; v += 32 * stride) {
        const int64_t at = v + lane * stride;
        Raw8<T> r;
        if (at >= lo && at < hi)
          r.load(logits + at * 8 - phase);
        else
          r.load_some(logits, at * 8 - phase, vocab);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t col = at * 8 - phase + i;
          const float z = r.value(i);
          uint64_t one = col >= 0 && col < vocab ? key_of(z, (uint32_t)col) : 0;
          const uint64_t last = __shfl_sync(0xffffffffu, list, a.top - 1);
          if (key_of(z, (uint32_t)at) < from || one < last) one = 0;
          if (__any_sync(0xffffffffu, one != 0)) {
            one = sort_down(one);
            list = merge_down(list, __shfl_sync(0xffffffffu, one, 31 - lane));
          }
        }
      }
    }
    list = merge_warps(list, lists);
  } else if constexpr (WARPS > 1) {
    __syncthreads();
  }

  // The row's sums, in the first warp.
  if constexpr (WARPS > 1) {
    if (warp == 0) {
      sums = Sums();
      for (int w = 0; w < WARPS; ++w) {
        Sums o;
        o.m = stat[0][w], o.s = stat[1][w], o.e = stat[2][w];
        sums.join(o, k);
      }
    }
  }
  if constexpr (CLUSTER) {
    __syncwarp();  // the first warp has read them
    if (x == 0) stat[0][0] = sums.m, stat[1][0] = sums.s, stat[2][0] = sums.e;
    cluster_sync();
    if (warp == 0 && rank == 0) {
      for (uint32_t b = 1; b < blocks; ++b) {
        Sums o;
        o.m = load_peer_f32(peer_smem(&stat[0][0], b));
        o.s = load_peer_f32(peer_smem(&stat[1][0], b));
        o.e = load_peer_f32(peer_smem(&stat[2][0], b));
        sums.join(o, k);
        if constexpr (TOP) list = merge_down(list, load_peer_u64(peer_smem(&lists[0][31 - lane], b)));
      }
    }
    cluster_sync();  // no block leaves while it is read
  }
  if (warp != 0 || rank != 0) return;
  const bool empty = sums.s == 0.0f;
  const float log_s = logf(sums.s);
  if (x == 0) {
    if (a.lse) a.lse[row] = empty ? -INFINITY : fmaf(sums.m, a.scale, log_s);
    if (ENTROPY) a.entropy[row] = empty ? 0.0f : log_s - kLn2 * (sums.e / sums.s);
    if (a.logp) a.logp[row] = target < 0 ? 0.0f : empty ? -INFINITY : fmaf(target_logit - sums.m, a.scale, -log_s);
  }
  if constexpr (TOP) {
    if (lane < a.top) {
      if (a.top_logp)
        a.top_logp[row * a.ld_logp + lane] =
            empty ? -INFINITY : fmaf(of_ordered((uint32_t)(list >> 32)) - sums.m, a.scale, -log_s);
      if (a.top_tokens) a.top_tokens[row * a.ld_tokens + lane] = (int32_t)~(uint32_t)list;
    }
  }
}

// ---- backward

struct GradArgs {
  uint32_t items;   // vectors of eight columns in this launch
  FastDiv per_row;  // of them in a row
  int64_t row0, vocab;
  const void* logits;
  int64_t ldl;
  float scale;
  const float* lse;
  int32_t index;
  const void* targets;
  const float *dlogp, *entropy, *dentropy;
  void* out;
  int64_t ldd;
};

// A row's gradient: p (a + b ln p), and g more at the target.
struct RowGrad {
  float lse, a, b, g;
  int target;
  __device__ __forceinline__ RowGrad(const GradArgs& p, int64_t row) : g(0.0f), target(-1) {
    lse = p.lse[row];
    const bool empty = lse == -INFINITY;
    if (empty) lse = INFINITY;  // every p is 0
    float h = 0.0f, entropy = 0.0f;
    if (p.dentropy) h = p.dentropy[row], entropy = p.entropy[row];
    if (p.targets) {
      target = token_at(p.targets, p.index, row, p.vocab);
      if (target >= 0 && !empty) g = p.scale * p.dlogp[row];
    }
    b = -p.scale * h;
    a = fmaf(b, entropy, -g);
  }
};

template <typename T, bool ENTROPY>
__device__ __forceinline__ float grad_of(float z, const RowGrad& r, float scale) {
  const float d = fmaf(z, scale, -r.lse);
  const float p = sizeof(T) == 2 ? exp2_of(d * kLog2e) : expf(d);
  if constexpr (ENTROPY) return p * fmaf(r.b, fmaxf(d, kLeast), r.a);
  return p * r.a;
}

constexpr int kThreads = 256, kItems = 4;

// Rows on 16-byte boundaries, of whole vectors.
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kThreads) grad_vec_kernel(const GradArgs a) {
  Raw8<T> r[kItems];
  uint32_t row[kItems], v[kItems];
  bool here[kItems];
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    const uint32_t i = (blockIdx.x * kItems + j) * kThreads + threadIdx.x;
    here[j] = i < a.items;
    row[j] = a.per_row.quotient(i);
    v[j] = i - row[j] * a.per_row.d;
    if (here[j]) r[j].load((const T*)a.logits + (a.row0 + row[j]) * a.ldl + (int64_t)v[j] * 8);
  }
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    if (!here[j]) continue;
    const RowGrad g(a, a.row0 + row[j]);
    float d[8];
    const int at = g.target - (int)(v[j] * 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) d[k] = grad_of<T, ENTROPY>(r[j].value(k), g, a.scale) + (k == at ? g.g : 0.0f);
    store_vec<8>((T*)a.out + (a.row0 + row[j]) * a.ldd + (int64_t)v[j] * 8, d);
  }
}

// Any rows: vectors lie on the output's 16-byte boundaries.
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kThreads) grad_any_kernel(const GradArgs a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.items) return;
  const uint32_t r = a.per_row.quotient(i);
  const int64_t row = a.row0 + r;
  T* const out = (T*)a.out + row * a.ldd;
  const int64_t col = (int64_t)(i - r * a.per_row.d) * 8 - row_phase(out);
  if (col >= a.vocab) return;
  float d[8];
  load_columns((const T*)a.logits + row * a.ldl, col, a.vocab, d);
  const RowGrad g(a, row);
#pragma unroll
  for (int k = 0; k < 8; ++k) d[k] = grad_of<T, ENTROPY>(d[k], g, a.scale) + (g.target >= 0 && col + k == g.target ? g.g : 0.0f);
  store_columns(out, col, a.vocab, d);
}

// ---------------------------------------------------------------- host side

// f with a truth value as a constant.
template <typename F>
void with_bool(bool b, F&& f) {
  if (b)
    f(std::true_type());
  else
    f(std::false_type());
}

template <typename T>
tide_status log_probs(const LogProbArgs& a, cudaStream_t stream) {
  const int sms = ops_num_sms();
  if (sms <= 0) return fail(TIDE_ERR_CUDA, "the current device could not be queried");
  // A warp for short rows, a block for long ones; where they are too few to fill the GPU,
  // up to eight blocks share a row, while each thread has a vector or more.
  const int64_t vectors = a.vocab / 8;
  int cluster = 1;
  if (vectors > 1024)
    while (cluster < 8 && a.rows * cluster * 2 <= 2 * sms && vectors >= (int64_t)cluster * 2 * 512) cluster *= 2;
  cudaError_t err = cudaSuccess;
  with_bool(a.entropy != nullptr, [&](auto entropy) {
    with_bool(a.top > 0, [&](auto top) {
      auto go = [&](auto per_row, auto clusters) {
        constexpr int P = decltype(per_row)::value;
        const int64_t grid = P == 32 ? (a.rows + 7) / 8 : a.rows * cluster;
        const ClusterLaunch l(grid, dim3(P == 32 ? 256 : P), cluster, false, 0, stream);
        err = cudaLaunchKernelEx(&l.cfg, log_probs_kernel<T, P, clusters.value, entropy.value, top.value>, a);
      };
      if (cluster > 1)
        go(std::integral_constant<int, 512>(), std::true_type());
      else if (vectors > 1024)
        go(std::integral_constant<int, 512>(), std::false_type());
      else if (vectors > 128)
        go(std::integral_constant<int, 128>(), std::false_type());
      else
        go(std::integral_constant<int, 32>(), std::false_type());
    });
  });
  return cuda_status(err, "log probabilities");
}

template <typename T>
tide_status log_probs_grad(GradArgs a, int64_t rows, cudaStream_t stream) {
  const bool vec = a.vocab % 8 == 0 && rows_aligned(a.logits, a.ldl, sizeof(T), rows) &&
                   rows_aligned(a.out, a.ldd, sizeof(T), rows);
  const int64_t per_row = vec ? a.vocab / 8 : (a.vocab + 14) / 8;  // vectors that any phase of a row touches
  a.per_row = FastDiv((uint32_t)per_row);
  return in_row_launches(rows, per_row, vec ? kThreads * kItems : kThreads, "log probabilities backward",
                         [&](int64_t r, uint32_t items, unsigned grid) {
                           a.row0 = r, a.items = items;
                           with_bool(a.dentropy != nullptr, [&](auto entropy) {
                             if (vec)
                               grad_vec_kernel<T, entropy.value><<<grid, kThreads, 0, stream>>>(a);
                             else
                               grad_any_kernel<T, entropy.value><<<grid, kThreads, 0, stream>>>(a);
                           });
                         });
}

tide_status check_logits(int64_t rows, int64_t vocab, int32_t dtype, const void* logits, int64_t ldl, float scale) {
  TIDE_TRY(check_sizes(rows, vocab, "log probabilities"));
  TIDE_TRY(check_dtype(dtype));
  if (!(scale > 0.0f) || std::isinf(scale)) return fail(TIDE_ERR_INVALID_ARG, "scale is not positive and finite");
  if (rows > INT32_MAX || vocab > INT32_MAX - 16) return fail(TIDE_ERR_UNIMPLEMENTED, "log probabilities: 2^31 rows or logits a row");
  return check_matrix(logits, rows, vocab, ldl, elem_bytes_of(dtype), "logits");
}

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" {

tide_status tide_log_probs(int64_t rows, int64_t vocab, int32_t dtype, const void* logits, int64_t ldl, float scale,
                           int32_t index, const void* targets, float* logp, float* lse, float* entropy, int32_t top,
                           float* top_logp, int64_t ld_top_logp, int32_t* top_tokens, int64_t ld_top_tokens,
                           void* stream) {
  clear_error();
  TIDE_TRY(check_logits(rows, vocab, dtype, logits, ldl, scale));
  if (top < 0 || top > kMaxTop || top > vocab) return fail(TIDE_ERR_INVALID_ARG, "top is 0 to 32 and at most the vocabulary");
  if (!targets != !logp && rows > 0) return fail(TIDE_ERR_INVALID_ARG, "targets and logp go together");
  if (rows == 0) return TIDE_OK;
  if (targets) {
    TIDE_TRY(check_index(index));
    TIDE_TRY(check_matrix(targets, 1, rows, rows, index_bytes_of(index), "targets"));
    TIDE_TRY(check_matrix(logp, 1, rows, rows, 4, "logp"));
  }
  if (lse) TIDE_TRY(check_matrix(lse, 1, rows, rows, 4, "lse"));
  if (entropy) TIDE_TRY(check_matrix(entropy, 1, rows, rows, 4, "entropy"));
  if (top > 0 && top_logp) TIDE_TRY(check_matrix(top_logp, rows, top, ld_top_logp, 4, "top_logp"));
  if (top > 0 && top_tokens) TIDE_TRY(check_matrix(top_tokens, rows, top, ld_top_tokens, 4, "top_tokens"));
  if (!top_logp && !top_tokens) top = 0;
  if (!logp && !lse && !entropy && top == 0) return TIDE_OK;
  const LogProbArgs a{rows, vocab,   logits, ldl,      scale,       index,      targets, logp,
                      lse,  entropy, top,    top_logp, ld_top_logp, top_tokens, ld_top_tokens};
  return dtype == TIDE_BF16 ? log_probs<bf16>(a, (cudaStream_t)stream) : log_probs<float>(a, (cudaStream_t)stream);
}

tide_status tide_log_probs_backward(int64_t rows, int64_t vocab, int32_t dtype, const void* logits, int64_t ldl,
                                    float scale, const float* lse, int32_t index, const void* targets,
                                    const float* dlogp, const float* entropy, const float* dentropy, void* dlogits,
                                    int64_t ldd, void* stream) {
  clear_error();
  TIDE_TRY(check_logits(rows, vocab, dtype, logits, ldl, scale));
  if (rows == 0 || vocab == 0) return TIDE_OK;
  if (!targets != !dlogp) return fail(TIDE_ERR_INVALID_ARG, "targets and dlogp go together");
  if (!entropy != !dentropy) return fail(TIDE_ERR_INVALID_ARG, "entropy and dentropy go together");
  TIDE_TRY(check_matrix(lse, 1, rows, rows, 4, "lse"));
  if (targets) {
    TIDE_TRY(check_index(index));
    TIDE_TRY(check_matrix(targets, 1, rows, rows, index_bytes_of(index), "targets"));
    TIDE_TRY(check_matrix(dlogp, 1, rows, rows, 4, "dlogp"));
  }
  if (entropy) {
    TIDE_TRY(check_matrix(entropy, 1, rows, rows, 4, "entropy"));
    TIDE_TRY(check_matrix(dentropy, 1, rows, rows, 4, "dentropy"));
  }
  TIDE_TRY(check_matrix(dlogits, rows, vocab, ldd, elem_bytes_of(dtype), "dlogits"));
  const GradArgs a{0,       FastDiv(), 0,     vocab,   logits,   ldl,     scale, lse,
                   index,   targets,   dlogp, entropy, dentropy, dlogits, ldd};
  return dtype == TIDE_BF16 ? log_probs_grad<bf16>(a, rows, (cudaStream_t)stream)
                            : log_probs_grad<float>(a, rows, (cudaStream_t)stream);
}

}  // extern "C"
