// Log probabilities of given tokens, entropy and alternatives, and their gradient
// (include/tide_lm_ops.h).
//
// Forward: one pass over a row.  Each thread keeps the largest logit m it has met
// and, over its own logits, S = sum 2^d and E = sum 2^d d with d = (logit - m) scale
// log2(e); when m grows by -D / (scale log2 e), S becomes S 2^D and E becomes 2^D (E + S D).
// The threads' (m, S, E) are joined by the same rule, and
//   lse = scale m + ln S,   entropy = ln S - ln 2 E / S  (no cancellation: E <= 0),
//   logp = scale (logit - m) - ln S.
// Alternatives: the threads' largest logits, joined by lane, are the largest of 32 disjoint parts of the row,
// and the `top`-th largest of these 32 is one that `top` logits at least reach.  So all alternatives are
// among the logits that reach it: 31 are expected for 20 alternatives of a row in random order, 112 for 32.
// A thread also keeps where its largest stood and the largest of its other vectors: where only the first
// reaches the bound one vector is read again, else all of the thread's (L2 has them), by all of the row's threads.  The
// logits that reach the bound are listed in shared memory, and each finds its rank by counting.
// Where equal logits make the list too long only those above the bound are listed, and the first of the ones at it.
// Where all that fails (more than 512 different logits above a bound, NaN that makes it too high) the alternatives
// are found one after the other.

// Backward: element by element, one exponential each.
//
// Both are bound by memory traffic while rows are long and many: 4096 x 131072 bf16 (1.07 GB) forward 156 to 160 us, 6.7
// to 6.9 TB/s, with entropy 166 to 169, with 20 alternatives too 190 to 194 (an exponential and some ten instructions an
// element, and of its own a row what the joining of its threads costs); backward 308 us, 7.0 TB/s.  Shorter rows pay for
// that joining, and for alternatives' bounds, lists and ranks, more often: 8192 x 32000 bf16 90 us (5.8 TB/s), with 20
// alternatives 114; 16384 x 4999 37 and 72; 16384 x 1000 14 and 33.  Odd rows cost the backward pass a vector a
// thread and edges by elements: 8192 x 131071 bf16 891 us, 4.8 TB/s (131072: 611).

#include <algorithm>
#include <cmath>

#include "cluster_ptx.cuh"
#include "lm_common.cuh"

namespace tide {
namespace {

constexpr int kMaxTop = 32;
constexpr uint32_t kMostBlocks = 8;  // of a cluster
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
  float *logp, *lse, *lse_parts, *entropy;
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

// Two fp32 in one register pair, added and multiplied by one instruction.
struct Pair {
  uint64_t v;
  __device__ __forceinline__ Pair(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ float2 parts() const {
    float2 p;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(p.x), "=f"(p.y) : "l"(v));
    return p;
  }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
  return a;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a.v) : "l"(b.v));
  return a;
}
__device__ __forceinline__ Pair fma_pair(Pair a, Pair b, Pair c) {
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a.v) : "l"(b.v), "l"(c.v));
  return a;
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

// ---- alternatives: keys that order logits, larger first, ties by the lower token

__device__ __forceinline__ uint32_t ordered(float v) {
  v = fmaxf(v, -INFINITY) + 0.0f;  // NaN as -inf, -0 as 0
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_ordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t token) { return (uint64_t)ordered(v) << 32 | (uint32_t)~token; }

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t warp_largest(uint64_t key) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) key = larger(key, __shfl_xor_sync(0xffffffffu, key, d));
  return key;
}

// The top-th largest of the lanes' values, by a bitonic sort.
__device__ __forceinline__ float warp_nth(float v, int top) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      const float o = __shfl_xor_sync(0xffffffffu, v, j);
      const bool low = (threadIdx.x & j) == 0, down = k == 32 || (threadIdx.x & k) == 0;
      v = low == down ? fmaxf(v, o) : fminf(v, o);
    }
  return __shfl_sync(0xffffffffu, v, top - 1);
}

// PER_ROW threads share a row (a warp, or a whole block), or those of a cluster of
// blocks; a block of warps takes eight rows.
template <typename T, int PER_ROW, bool CLUSTER, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(PER_ROW == 32 ? 256 : PER_ROW, 1024 / (PER_ROW == 32 ? 256 : PER_ROW))
    log_probs_kernel(const LogProbArgs a) {
  constexpr int WARPS = PER_ROW / 32, kAhead = sizeof(T) == 2 ? 4 : 2;
  constexpr int kRowsHere = PER_ROW == 32 ? 8 : 1, kRoom = 512;
  __shared__ float stat[3][WARPS];
  __shared__ float largest[TOP ? WARPS : 1][32];
  __shared__ uint64_t listed[TOP ? kRowsHere : 1][TOP ? kRoom : 1];
  __shared__ uint32_t listed_count[kRowsHere];
  __shared__ uint32_t again_count[kRowsHere];
  __shared__ int2 again[TOP ? kRowsHere : 1][TOP ? PER_ROW : 1];
  __shared__ uint64_t found[TOP ? WARPS + 1 : 1];
  const uint32_t blocks = CLUSTER ? cluster_size() : 1, rank = CLUSTER ? cluster_rank() : 0;
  const int64_t row = PER_ROW == 32 ? (int64_t)blockIdx.x * 8 + threadIdx.x / 32 : (int64_t)(blockIdx.x / blocks);
  if (row >= a.rows) return;  // a whole warp, of rows of one
  const int x = threadIdx.x % PER_ROW, warp = x / 32, lane = x % 32, here = PER_ROW == 32 ? threadIdx.x / 32 : 0;
  const int64_t vocab = a.vocab;
  const T* const logits = (const T*)a.logits + row * a.ldl;
  const float k = a.scale * kLog2e;
  // Vectors of the row that are whole: from `lo` to below `hi`.
  const int phase = row_phase(logits), count = (int)((vocab + phase + 7) / 8);
  const int lo = phase > 0, hi = (int)((vocab + phase) / 8);
  const int stride = PER_ROW * (int)blocks, first = (int)rank * PER_ROW + x;  // vectors are fewer than 2^28
  auto sync = [&]() {
    if constexpr (WARPS > 1)
      __syncthreads();
    else
      __syncwarp();
  };

  int target = -1;
  float target_logit = 0.0f;
  if (x == 0 && rank == 0 && a.targets) {
    target = token_at(a.targets, a.index, row, vocab);
    if (target >= 0) target_logit = (float)logits[target];
  }
  if (TOP && x == 0) listed_count[here] = again_count[here] = 0;
  __syncwarp();  // for rows of a warp; others have a barrier below

  Sums sums;
  int best_at = first;   // the vector in which the largest logit stood first
  float second = -INFINITY;  // the largest of the others
  for (int v = first; v < count; v += kAhead * stride) {
    Raw8<T> r[kAhead];
    if (v >= lo && v + (kAhead - 1) * stride < hi) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) r[j].load(logits + (int64_t)(v + j * stride) * 8 - phase);
    } else {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int at = v + j * stride;
        if (at >= lo && at < hi)
          r[j].load(logits + (int64_t)at * 8 - phase);
        else
          r[j].load_some(logits, (int64_t)at * 8 - phase, vocab);
      }
    }
    // Alternatives want each vector's largest logit; else one rise for all of them will do.
    constexpr int kAtOnce = TOP || !ENTROPY ? 1 : kAhead;
#pragma unroll
    for (int j = 0; j < kAhead; j += kAtOnce) {
      auto value = [&](int i) { return r[j + i / 8].value(i % 8); };
      float most = value(0);
#pragma unroll
      for (int i = 1; i < 8 * kAtOnce; ++i) most = fmaxf(most, value(i));
      if (most > sums.m) {
        if constexpr (TOP) second = sums.m, best_at = v + j * stride;
        sums.raise(most, k);
      } else if constexpr (TOP) {
        second = fmaxf(second, most);
      }
      if constexpr (ENTROPY) {
        // In pairs, which take half the issue slots (4096 x 131072 bf16 172 us became 168; without the entropy they
        // were slower, 162 against 156).
        Pair s2(sums.s, 0.0f), e2(sums.e, 0.0f);
        const Pair down(-sums.m, -sums.m), by(k, k);
#pragma unroll
        for (int i = 0; i < 8 * kAtOnce; i += 2) {
          const float2 d = ((Pair(value(i), value(i + 1)) + down) * by).parts();
          const Pair p(exp2_of(d.x), exp2_of(d.y));
          s2 = s2 + p;
          e2 = fma_pair(p, Pair(fmaxf(d.x, kLeast), fmaxf(d.y, kLeast)), e2);
        }
        sums.s = s2.parts().x + s2.parts().y;
        sums.e = e2.parts().x + e2.parts().y;
      } else {
#pragma unroll
        for (int i = 0; i < 8 * kAtOnce; ++i) sums.s += exp2_of((value(i) - sums.m) * k);
      }
    }
  }
  // This thread's largest logit: -inf with none (or no other).
  const float mine = sums.s == 0.0f ? -INFINITY : sums.m;

  auto join_lanes = [&](int lanes) {
    for (int d = lanes / 2; d > 0; d >>= 1) {
      Sums o;
      o.m = __shfl_xor_sync(0xffffffffu, sums.m, d);
      o.s = __shfl_xor_sync(0xffffffffu, sums.s, d);
      if (ENTROPY) o.e = __shfl_xor_sync(0xffffffffu, sums.e, d);
      // Both lanes of a pair add the same two in the same order.
      Sums& lower = lane & d ? o : sums;
      Sums& upper = lane & d ? sums : o;
      lower.join(upper, k);
      sums = lower;
    }
  };
  join_lanes(32);
  float bound = mine;  // the largest of the row's part that goes by this lane
  if constexpr (WARPS > 1) {
    if (lane == 0) stat[0][warp] = sums.m, stat[1][warp] = sums.s, stat[2][warp] = sums.e;
    if constexpr (TOP) largest[warp][lane] = mine;
    __syncthreads();
    if constexpr (TOP) {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) bound = fmaxf(bound, largest[w][lane]);
    }
    // Every warp joins the warps' sums.
    sums = Sums();
    if (lane < WARPS) sums.m = stat[0][lane], sums.s = stat[1][lane], sums.e = stat[2][lane];
    join_lanes(WARPS);
  }
  if constexpr (CLUSTER) {
    // The blocks' in their turn, all of each.
    __syncthreads();
    if (warp == 0) {
      if (lane == 0) stat[0][0] = sums.m, stat[1][0] = sums.s, stat[2][0] = sums.e;
      if constexpr (TOP) largest[0][lane] = bound;
    }
    cluster_sync();
    sums = Sums();
    if ((uint32_t)lane < blocks) {
      sums.m = load_peer_f32(peer_smem(&stat[0][0], lane));
      sums.s = load_peer_f32(peer_smem(&stat[1][0], lane));
      sums.e = load_peer_f32(peer_smem(&stat[2][0], lane));
    }
    if constexpr (TOP) {
      float theirs[kMostBlocks];  // loads at once: each takes the better part of a microsecond
#pragma unroll
      for (uint32_t b = 0; b < kMostBlocks; ++b)
        theirs[b] = b < blocks ? load_peer_f32(peer_smem(&largest[0][lane], b)) : -INFINITY;
#pragma unroll
      for (uint32_t b = 0; b < kMostBlocks; ++b) bound = fmaxf(bound, theirs[b]);
    }
    join_lanes(kMostBlocks);
    sums.m = __shfl_sync(0xffffffffu, sums.m, 0);
    sums.s = __shfl_sync(0xffffffffu, sums.s, 0);
    sums.e = __shfl_sync(0xffffffffu, sums.e, 0);
    if constexpr (!TOP) cluster_sync();  // no block leaves while it is read
  } else if constexpr (WARPS > 1) {
    sums.m = __shfl_sync(0xffffffffu, sums.m, 0);
    sums.s = __shfl_sync(0xffffffffu, sums.s, 0);
    sums.e = __shfl_sync(0xffffffffu, sums.e, 0);
  }

  const bool empty = sums.s == 0.0f;
  const float log_s = logf(sums.s);
  // A logit's log probability.  Of the halves, whose difference is in fp32's range where the logits' is not.
  auto logp_of = [&](float logit) { return fmaf(0.5f * logit - 0.5f * sums.m, 2.0f * a.scale, -log_s); };
  if (x == 0 && rank == 0) {
    if (a.lse) a.lse[row] = empty ? -INFINITY : fmaf(sums.m, a.scale, log_s);
    if (a.lse_parts) a.lse_parts[2 * row] = empty ? -INFINITY : sums.m, a.lse_parts[2 * row + 1] = log_s;
    if (ENTROPY) a.entropy[row] = empty ? 0.0f : log_s - kLn2 * (sums.e / sums.s);
    if (a.logp) a.logp[row] = target < 0 ? 0.0f : empty ? -INFINITY : logp_of(target_logit);
  }
  if constexpr (TOP) {
    const int top = a.top;
    auto put = [&](int at, uint64_t key) {
      if (a.top_logp)
        a.top_logp[row * a.ld_logp + at] =
            empty ? -INFINITY : logp_of(of_ordered((uint32_t)(key >> 32)));
      if (a.top_tokens) a.top_tokens[row * a.ld_tokens + at] = (int32_t)~(uint32_t)key;
    };
    auto load = [&](Raw8<T>& r, int at) {
      if (at >= lo && at < hi)
        r.load(logits + (int64_t)at * 8 - phase);
      else
        r.load_some(logits, (int64_t)at * 8 - phase, vocab);
    };
    // Which of a vector's logits reach a finite limit (what is not there is -inf).
    auto reach = [&](const Raw8<T>& r, float limit) {
      uint32_t hits = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r.value(i) >= limit) hits |= 1u << i;
      return hits;
    };
    auto list = [&](const Raw8<T>& r, int v, uint32_t hits) {
      if (hits == 0) return;
      uint32_t at = atomicAdd(&listed_count[here], (uint32_t)__popc(hits));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (hits >> i & 1) {
          if (at < kRoom) listed[here][at] = key_of(r.value(i), (uint32_t)v * 8 - (uint32_t)(phase - i));
          ++at;
        }
    };
    bound = warp_nth(bound, top);
    // Logits that reach the bound; where too many do (or the bound is that of masked ones), those above
    // it, and of the ones at it as many as it takes, the lowest tokens, below.
    bool strict = bound == -INFINITY;
    uint32_t n = 0, theirs = 0;  // listed, of a cluster also by block `lane`
    for (;;) {
      const float limit = strict ? nextafterf(bound, INFINITY) : bound;  // of +inf itself; NaN rows alone have that
      if (mine >= limit && first < count) {
        Raw8<T> r;
        load(r, best_at);
        list(r, best_at, reach(r, limit));
      }
      // Threads that may have met more: all their other vectors, spread over the row's threads here.
      if (mine >= limit && second >= limit && first < count) {
        const uint32_t at = atomicAdd(&again_count[here], 1u);
        again[here][at] = make_int2(first, best_at);
      }
      sync();
      const uint32_t each = (uint32_t)((count + stride - 1) / stride), all = each * again_count[here];
      for (uint32_t i0 = x; i0 < all; i0 += PER_ROW * kAhead) {
        Raw8<T> r[kAhead];
        int at[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const uint32_t i = i0 + j * PER_ROW, which = i / each;
          at[j] = -1;
          if (i >= all) continue;
          const int2 of = again[here][which];
          at[j] = of.x + (int)(i - which * each) * stride;
          if (at[j] >= count || at[j] == of.y) at[j] = -1;
          if (at[j] >= 0) load(r[j], at[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (at[j] >= 0) list(r[j], at[j], reach(r[j], limit));
      }
      if constexpr (CLUSTER) {
        cluster_sync();
        theirs = (uint32_t)lane < blocks ? min(load_peer_u32(peer_smem(&listed_count[0], lane)), kRoom + 1u) : 0;
        n = theirs;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
        n = min(n, kRoom + 1u);
      } else {
        sync();
        n = listed_count[here];
      }
      if (strict || n <= kRoom) break;
      strict = true;
      if constexpr (CLUSTER)
        cluster_sync();
      else
        sync();
      if (x == 0) listed_count[here] = again_count[here] = 0;
      sync();
    }
    if constexpr (CLUSTER) {
      // The first block brings the others' lists to its own, behind one another.
      if (rank == 0 && n <= kRoom) {
        uint32_t from = 0, i = x;
        bool found = false;
#pragma unroll
        for (int b = 0; b < (int)kMostBlocks; ++b) {
          const uint32_t c = __shfl_sync(0xffffffffu, theirs, b);
          if (!found && i < c) from = b, found = true;
          if (!found) i -= c;
        }
        if (found && from > 0) listed[0][x] = load_peer_u64(peer_smem(&listed[0][i], from));
        __syncthreads();
      }
    }
    // The ones at the bound in order, eight vectors and then 32 at a time, by one warp, until there are enough (of a
    // row of equals eight vectors hold them, and ranks cost their number squared).
    constexpr uint32_t kSweep = 256;
    if (strict && n < (uint32_t)top) {
      // All have read the counts, by which they came here, before a count moves.
      if constexpr (CLUSTER) {
        cluster_sync();
        if (x == 0 && rank == 0) listed_count[0] = n;
        __syncwarp();
      } else {
        sync();
      }
      if (warp == 0 && rank == 0) {
        for (int from = 0, most = 8; from < count; from += most, most = 32) {
          const int v = from + lane;
          if (lane < most && v < count) {
            Raw8<T> r;
            load(r, v);
            uint32_t hits = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int64_t col = (int64_t)v * 8 - phase + i;
              if (fmaxf(r.value(i), -INFINITY) == bound && col >= 0 && col < vocab) hits |= 1u << i;  // NaN as -inf
            }
            list(r, v, hits);
          }
          __syncwarp();
          const uint32_t so_far = *(volatile uint32_t*)&listed_count[here];
          __syncwarp();
          if (so_far >= (uint32_t)top) break;
        }
      }
      if constexpr (CLUSTER) {
        cluster_sync();
        n = load_peer_u32(peer_smem(&listed_count[0], 0));
      } else {
        sync();
        n = listed_count[here];
      }
    }
    static_assert(kMaxTop + kSweep <= kRoom, "fewer than top are listed when a sweep begins");
    if (n >= (uint32_t)top && n <= kRoom) {
      if (rank != 0) n = 0;
      for (uint32_t i = x; i < n; i += PER_ROW) {
        const uint64_t key = listed[here][i];
        int above = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < n; ++j) above += listed[here][j] > key;
        if (above < top) put(above, key);
      }
    } else {
      // One after the other: the largest key below the last one.
      uint64_t last = ~0ull;
      for (int i = 0; i < top; ++i) {
        uint64_t key = 0;
        for (int v = first; v < count; v += stride) {
          Raw8<T> r;
          load(r, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int64_t col = (int64_t)v * 8 - phase + j;
            const uint64_t one = key_of(r.value(j), (uint32_t)col);
            if (col >= 0 && col < vocab && one < last) key = larger(key, one);
          }
        }
        key = warp_largest(key);
        if constexpr (WARPS > 1) {
          if (lane == 0) found[warp] = key;
          __syncthreads();
          key = warp_largest(lane < WARPS ? found[lane] : 0);
          if constexpr (CLUSTER) {
            if (x == 0) found[WARPS] = key;
            cluster_sync();
            for (uint32_t b = 0; b < blocks; ++b) key = larger(key, load_peer_u64(peer_smem(&found[WARPS], b)));
            cluster_sync();
          } else {
            __syncthreads();
          }
        }
        if (x == 0 && rank == 0) put(i, key);
        last = key;
      }
    }
    if constexpr (CLUSTER) cluster_sync();  // no block leaves while its list is read
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
  const float *lse, *lse_parts;
  int32_t index;
  const void* targets;
  const float *dlogp, *entropy, *dentropy;
  void* out;
  int64_t ldd;
};

// A row's gradient: p (a + b ln p), and g more at the target, with ln p = (logit - peak) scale - rest.
struct RowGrad {
  float peak, rest, a, b, g;
  int target;
  __device__ __forceinline__ void load(const GradArgs& p, int64_t row) {
    peak = 0.0f, g = 0.0f, target = -1;
    if (p.lse_parts)
      peak = p.lse_parts[2 * row], rest = p.lse_parts[2 * row + 1];
    else
      rest = p.lse[row];
    const bool empty = rest == -INFINITY;
    if (empty) peak = 0.0f, rest = INFINITY;  // every p is 0
    float h = 0.0f, entropy = 0.0f;
    if (p.dentropy) h = p.dentropy[row], entropy = p.entropy[row];
    if (empty) h = entropy = 0.0f;  // what came back for it may be infinite or NaN, and 0 times that is not 0
    if (p.targets) {
      target = token_at(p.targets, p.index, row, p.vocab);
      if (target >= 0 && !empty) g = p.scale * p.dlogp[row];
    }
    b = -p.scale * h;
    a = fmaf(b, entropy, -g);
  }
};

// The gradient of a vector's logits; at: the target's place in it, if it is there.
template <typename T, bool ENTROPY>
__device__ __forceinline__ void grad_of(float (&z)[8], const RowGrad& r, float scale, int64_t at) {
  const Pair down(-r.peak, -r.peak), by(scale, scale), rest(-r.rest, -r.rest), a(r.a, r.a), b(r.b, r.b),
      to_two(kLog2e, kLog2e);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const Pair d2 = fma_pair(Pair(z[k], z[k + 1]) + down, by, rest);
    const float2 d = d2.parts(), t = (d2 * to_two).parts();
    const Pair p = sizeof(T) == 2 ? Pair(exp2_of(t.x), exp2_of(t.y)) : Pair(expf(d.x), expf(d.y));
    const float2 g = (p * (ENTROPY ? fma_pair(b, Pair(fmaxf(d.x, kLeast), fmaxf(d.y, kLeast)), a) : a)).parts();
    z[k] = g.x, z[k + 1] = g.y;
  }
  if (at >= 0 && at < 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k == at) z[k] += r.g;
  }
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
  RowGrad g;
#pragma unroll
  for (int j = 0; j < kItems; ++j) {
    if (!here[j]) continue;
    if (j == 0 || row[j] != row[j - 1]) g.load(a, a.row0 + row[j]);
    float d[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) d[k] = r[j].value(k);
    grad_of<T, ENTROPY>(d, g, a.scale, g.target < 0 ? -1 : g.target - (int64_t)v[j] * 8);
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
  RowGrad g;
  g.load(a, row);
  grad_of<T, ENTROPY>(d, g, a.scale, g.target < 0 ? -1 : g.target - col);
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
  // The fewest threads a row that still fill the GPU, since what is not a thread's own logits costs each of
  // them alike (16384 x 4999 bf16: 38 us with a warp a row, 80 with 128 threads, 112 with 256; 2048 x
  // 131072: 124, 92 and 92).  800 threads an SM fill it where rows are long, fewer where a row's latency
  // is a launch's (warps against 128 threads: 300 x 4999 6.3 and 5.2 us, 600 x 4999 6.4 and 6.5, 1500 x 16384 18
  // and 16, 4800 x 16384 31 and 34; 128 against 256: 600 x 50001 18 and 16, 1021 x 50001 24 and 26).  Beyond 32768
  // logits a warp is slower however many rows there are (4096 x 65536 99 and 90), and with alternatives beyond 12288,
  // since its lanes hold too much of the row to read again (16384 x 16384 with 20 180 and 154, 16384 x 8192 105 and 114).
  const int64_t vectors = a.vocab / 8, threads = (int64_t)sms * std::min<int64_t>(800, vectors / 5);
  int want = 32;
  for (const int next : {128, 256, 512})
    if (vectors >= next && (a.rows * want < threads || (next == 128 && vectors > (a.top > 0 ? 1536 : 4096)))) want = next;
  // Still too few: up to eight blocks share a row, while each thread has a vector or more.
  int cluster = 1;
  if (vectors > 1024)
    while (cluster < (int)kMostBlocks && a.rows * cluster * 2 <= 2 * sms && vectors >= (int64_t)cluster * 2 * 512) cluster *= 2;
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
      else if (want == 512)
        go(std::integral_constant<int, 512>(), std::false_type());
      else if (want == 256)
        go(std::integral_constant<int, 256>(), std::false_type());
      else if (want == 128)
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
  // A logit whose distance from the largest leaves fp32's range (above) has p = 0: so it must at this scale.
  if (!(scale >= 0x1p-120f && scale <= 0x1p64f)) return fail(TIDE_ERR_INVALID_ARG, "scale is not between 2^-120 and 2^64");
  if (rows > INT32_MAX || vocab > INT32_MAX - 16) return fail(TIDE_ERR_UNIMPLEMENTED, "log probabilities: 2^31 rows or logits a row");
  return check_matrix(logits, rows, vocab, ldl, elem_bytes_of(dtype), "logits");
}

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" {

tide_status tide_log_probs(int64_t rows, int64_t vocab, int32_t dtype, const void* logits, int64_t ldl, float scale,
                           int32_t index, const void* targets, float* logp, float* lse, float* lse_parts,
                           float* entropy, int32_t top, float* top_logp, int64_t ld_top_logp, int32_t* top_tokens, int64_t ld_top_tokens,
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
  if (lse_parts) TIDE_TRY(check_matrix(lse_parts, rows, 2, 2, 4, "lse_parts"));
  if (entropy) TIDE_TRY(check_matrix(entropy, 1, rows, rows, 4, "entropy"));
  if (top > 0 && top_logp) TIDE_TRY(check_matrix(top_logp, rows, top, ld_top_logp, 4, "top_logp"));
  if (top > 0 && top_tokens) TIDE_TRY(check_matrix(top_tokens, rows, top, ld_top_tokens, 4, "top_tokens"));
  if (!top_logp && !top_tokens) top = 0;
  if (!logp && !lse && !lse_parts && !entropy && top == 0) return TIDE_OK;
  const LogProbArgs a{rows,    vocab,   logits, ldl, scale,    index,       targets,    logp,
                      lse,     lse_parts, entropy, top, top_logp, ld_top_logp, top_tokens, ld_top_tokens};
  return dtype == TIDE_BF16 ? log_probs<bf16>(a, (cudaStream_t)stream) : log_probs<float>(a, (cudaStream_t)stream);
}

tide_status tide_log_probs_backward(int64_t rows, int64_t vocab, int32_t dtype, const void* logits, int64_t ldl,
                                    float scale, const float* lse, const float* lse_parts, int32_t index,
                                    const void* targets, const float* dlogp, const float* entropy, const float* dentropy, void* dlogits,
                                    int64_t ldd, void* stream) {
  clear_error();
  TIDE_TRY(check_logits(rows, vocab, dtype, logits, ldl, scale));
  if (rows == 0 || vocab == 0) return TIDE_OK;
  if (!targets != !dlogp) return fail(TIDE_ERR_INVALID_ARG, "targets and dlogp go together");
  if (!entropy != !dentropy) return fail(TIDE_ERR_INVALID_ARG, "entropy and dentropy go together");
  if (lse_parts)
    TIDE_TRY(check_matrix(lse_parts, rows, 2, 2, 4, "lse_parts"));
  else
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
  const GradArgs a{0,     FastDiv(), 0,     vocab, logits,  ldl,      scale,   lse,
                   lse_parts, index,   targets, dlogp, entropy, dentropy, dlogits, ldd};
  return dtype == TIDE_BF16 ? log_probs_grad<bf16>(a, rows, (cudaStream_t)stream)
                            : log_probs_grad<float>(a, rows, (cudaStream_t)stream);
}

}  // extern "C"
