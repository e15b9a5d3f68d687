// Token embedding, and its gradient by sorted tokens (include/tide_lm_ops.h).
//
// Forward: rows of the table are copied, scaled on the way; bound by memory traffic (16384 rows of 8192 bf16, 380 MB
// with the rows read once: 62 us, 6.1 TB/s; rows of 8191 104 us: a vector a thread, cut out of two granules).
//
// Backward, dweight[v] = scale * sum of dy[t] over the t with token v, is dense: every row
// of dweight is written once, the rows of dy are read once, and both dwarf the ids.
//   1. A cluster of blocks sorts the ids, stably, by nine bits at a time (their places
//      with them), so that a token's rows of dy are a run of sorted places, in ascending order: the
//      sum's order is fixed.  A second kernel writes the rows that no id names meanwhile.
//   2. The sorted places are cut into tiles.  A thread takes eight columns and a tile, and
//      sums and stores the runs that begin in it, reading up to a tile beyond its end for the last.
//      Where a run is longer than that, every tile leaves its part of it in the workspace.
//   3. The parts of such runs (padding, separators, articles) are joined, a block at a time.
// 16384 tokens into 131072 x 8192 bf16 (2.4 GB): 370 us, 6.5 TB/s; zeros 298 beside the sort's 18, sums 63, parts 10.
// Small and odd ones wait for memory, not for its bandwidth: 4093 tokens into 4999 x 4095 fp32 (110 MB) 54 us, of which
// 20 are zeros beside the sort's 12, 30 sums and 9 parts, one behind the other.  The sums read at a fifth of DRAM's rate:
// 64 registers a thread leave half of an SM's warps, and 1026 blocks are 1.7 turns of the 608 that run at once.

#include <algorithm>
#include <type_traits>

#include "cluster_ptx.cuh"
#include "lm_common.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxCols = 1 << 24;

// ---------------------------------------------------------------- forward

struct EmbedArgs {
  uint32_t items;   // vectors of eight columns in this launch
  FastDiv per_row;  // of them in a row
  int64_t row0, vocab, cols;
  int32_t index;
  const void* ids;
  const void* weight;
  int64_t ldw;
  float scale;
  void* out;
  int64_t ldo;
};

// Rows on 16-byte boundaries, of whole vectors; ITEMS vectors a thread.
template <typename T, int ITEMS>
__global__ void __launch_bounds__(kThreads) embed_vec_kernel(const EmbedArgs a) {
  Raw8<T> r[ITEMS];
  uint32_t row[ITEMS], col[ITEMS];
  int token[ITEMS];
  bool here[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const uint32_t i = (blockIdx.x * ITEMS + j) * kThreads + threadIdx.x;
    here[j] = i < a.items;
    row[j] = a.per_row.quotient(i);
    col[j] = i - row[j] * a.per_row.d;
    token[j] = here[j] ? token_at(a.ids, a.index, a.row0 + row[j], a.vocab) : -1;
  }
#pragma unroll
  for (int j = 0; j < ITEMS; ++j)
    if (token[j] >= 0) r[j].load((const T*)a.weight + token[j] * a.ldw + (int64_t)col[j] * 8);
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    if (!here[j]) continue;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = token[j] >= 0 ? r[j].value(k) * a.scale : 0.0f;
    store_vec<8>((T*)a.out + (a.row0 + row[j]) * a.ldo + (int64_t)col[j] * 8, v);
  }
}

// Any rows: vectors lie on the output's 16-byte boundaries.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_any_kernel(const EmbedArgs a) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.items) return;
  const uint32_t r = a.per_row.quotient(i);
  const int64_t row = a.row0 + r;
  T* const out = (T*)a.out + row * a.ldo;
  const int64_t col = (int64_t)(i - r * a.per_row.d) * 8 - row_phase(out);
  if (col >= a.cols) return;
  const int token = token_at(a.ids, a.index, row, a.vocab);
  float v[8] = {};
  if (token >= 0) {
    load_columns((const T*)a.weight + token * a.ldw, col, a.cols, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= a.scale;
  }
  store_columns(out, col, a.cols, v);
}

// ---------------------------------------------------------------- sorting

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kSortCluster = 8;
// A digit: 18 bits, a vocabulary of 262,143, take two passes.
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kRounds = 8;  // places a lane has in registers
static_assert(kDigits == kSortThreads, "a thread a digit");

struct SortArgs {
  int64_t tokens, vocab;
  int32_t index;
  const void* ids;
  uint32_t *key, *place;    // out, sorted by key; ids outside the vocabulary have key vocab
  uint32_t *key2, *place2;  // scratch
  int passes;
  int32_t tile;     // places a tile
  uint32_t* longs;  // number of the runs that are joined from parts, and the tiles that they begin in
};

// One cluster: a stable counting sort a digit at a time.  The cluster's warps take consecutive
// parts of the places; a warp walks its part 32 places at a time, and equal digits among
// those are ranked by lane.  16384 ids of 18 bits take 17 us, 4093 of 13 bits 11, nearly all of it
// latency: of the ids, of a pass's counts on their way between blocks, of its keys.
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const SortArgs a) {
  __shared__ uint32_t counts[kSortWarps][kDigits];
  __shared__ uint32_t totals[kDigits];  // the block's
  __shared__ uint32_t scan[kSortWarps];
  let_next_kernel_start();
  const uint32_t blocks = cluster_size(), rank = cluster_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, digit_here = threadIdx.x;
  const uint32_t n = (uint32_t)a.tokens, parts = blocks * kSortWarps;
  const uint32_t part = (uint32_t)(((uint64_t)n + parts * 32 - 1) / (parts * 32) * 32);
  const uint64_t begin = min((uint64_t)(rank * kSortWarps + warp) * part, (uint64_t)n), end = min(begin + part, (uint64_t)n);
  const bool held = part <= kRounds * 32;  // all of a warp's part in registers
  if (rank == 0 && threadIdx.x == 0) a.longs[0] = 0;
  for (int pass = 0; pass < a.passes; ++pass) {
    // The last pass ends in key and place.
    const bool to_first = (a.passes - pass) % 2 == 1;
    const uint32_t *key = to_first ? a.key2 : a.key, *place = to_first ? a.place2 : a.place;
    uint32_t *key_out = to_first ? a.key : a.key2, *place_out = to_first ? a.place : a.place2;
    const int shift = pass * kDigitBits;
    uint32_t k[kRounds], q[kRounds];
    auto load = [&](uint64_t i0) {
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const uint64_t i = i0 + r * 32 + lane;
        k[r] = 0, q[r] = (uint32_t)i;
        if (i >= end) continue;
        if (pass == 0) {
          const int t = token_at(a.ids, a.index, (int64_t)i, a.vocab);
          k[r] = t >= 0 ? (uint32_t)t : (uint32_t)a.vocab;
        } else {
          k[r] = __ldcg(key + i), q[r] = __ldcg(place + i);
        }
      }
    };
    for (int d = lane; d < kDigits; d += 32) counts[warp][d] = 0;
    __syncwarp();
    for (uint64_t i0 = begin; i0 < end; i0 += kRounds * 32) {
      load(i0);
#pragma unroll
      for (int r = 0; r < kRounds; ++r)
        if (i0 + r * 32 + lane < end) atomicAdd(&counts[warp][(k[r] >> shift) % kDigits], 1u);
    }
    __syncthreads();
    // A digit's places in each warp's part begin behind those in the parts before.
    uint32_t in_warp[kSortWarps], sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) in_warp[w] = counts[w][digit_here];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = in_warp[w];
      in_warp[w] = sum;
      sum += c;
    }
    totals[digit_here] = sum;
    cluster_sync();
    uint32_t before = 0, all = 0, peer[kSortCluster];
#pragma unroll
    for (uint32_t b = 0; b < kSortCluster; ++b) peer[b] = b < blocks ? load_peer_u32(peer_smem(&totals[digit_here], b)) : 0;
#pragma unroll
    for (uint32_t b = 0; b < kSortCluster; ++b) {
      if (b < rank) before += peer[b];
      all += peer[b];
    }
    uint32_t up = all;  // ... and behind all of the smaller digits'
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, up, d);
      if (lane >= d) up += o;
    }
    if (lane == 31) scan[warp] = up;
    __syncthreads();
    uint32_t base = before + up - all;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w)
      if (w < warp) base += scan[w];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) counts[w][digit_here] = base + in_warp[w];
    __syncthreads();
    for (uint64_t i0 = begin; i0 < end; i0 += kRounds * 32) {
      if (!held) load(i0);
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        if (i0 + r * 32 >= end) break;  // the same for the warp
        const bool here = i0 + r * 32 + lane < end;
        const uint32_t digit = here ? (k[r] >> shift) % kDigits : kDigits;
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        const uint32_t rank_in = __popc(same & ((1u << lane) - 1));
        const uint32_t at = here ? counts[warp][digit] : 0;
        __syncwarp();
        if (here) {
          if (rank_in == 0) counts[warp][digit] = at + __popc(same);
          key_out[at + rank_in] = k[r];
          place_out[at + rank_in] = q[r];
        }
        __syncwarp();
      }
    }
    cluster_sync();
  }
  // Runs that begin in a tile and go on beyond the next one's end.
  const int64_t tile = a.tile, tiles = (a.tokens + tile - 1) / tile;
  for (int64_t t = rank * kSortThreads + threadIdx.x; t + 2 < tiles; t += blocks * kSortThreads) {
    const uint32_t k = __ldcg(a.key + (t + 1) * tile), last = __ldcg(a.key + (t + 1) * tile - 1),
                   behind = __ldcg(a.key + (t + 2) * tile), before = t > 0 ? __ldcg(a.key + t * tile - 1) : (uint32_t)a.vocab;
    if (k < (uint32_t)a.vocab && last == k && behind == k && before != k) a.longs[1 + atomicAdd(a.longs, 1u)] = (uint32_t)t;
  }
}

// ---------------------------------------------------------------- rows without a token

constexpr int kZeroThreads = 1024, kZeroWords = 8192;
// Bytes of neighbouring rows that a block writes in a row: by single rows of 16 KB 335 us for 131072 x 8192 bf16,
// in chunks of 16 to 64 KB 298, of 1 MB 312.
constexpr int64_t kZeroChunk = 32 << 10;

struct ZeroArgs {
  int64_t tokens, vocab, cols;
  int32_t index;
  const void* ids;
  void* dweight;
  int64_t lddw;
  FastDiv vectors, blocks;
  int32_t shift;
};

// Zeros for the rows of dweight that no id names.  Block b of B takes chunks b, b + B, ... of 2^shift
// rows (named ones lie together), a piece at a time, with a bit for each row that an id names: it looks
// at all ids by itself, so that it need not wait for the sort, which runs beside it.
template <typename T>
__global__ void __launch_bounds__(kZeroThreads, 1) zero_kernel(const ZeroArgs a) {
  __shared__ uint32_t named[kZeroWords];
  let_next_kernel_start();
  const uint32_t step = gridDim.x, in_chunk = (1u << a.shift) - 1;
  const int64_t chunks = (a.vocab + in_chunk) >> a.shift;
  const int64_t all = (chunks - blockIdx.x + step - 1) / step << a.shift;  // rows of this block, some perhaps beyond the last
  const int64_t most = min((int64_t)kZeroWords * 32, (int64_t)(1 << 30) / a.vectors.d);
  for (int64_t first = 0; first < all; first += most) {
    const uint32_t rows = (uint32_t)min(most, all - first);
    for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += kZeroThreads) named[i] = 0;
    __syncthreads();
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < a.tokens; i += kZeroThreads) {
      const int token = token_at(a.ids, a.index, i, a.vocab);
      const uint32_t chunk = token < 0 ? 0 : (uint32_t)token >> a.shift, down = a.blocks.quotient(chunk);
      const int64_t r = ((int64_t)down << a.shift) + (token & in_chunk) - first;
      if (token >= 0 && chunk - down * step == blockIdx.x && r >= 0 && r < rows) atomicOr(named + r / 32, 1u << (r % 32));
    }
    __syncthreads();
    const float zeros[8] = {};
    for (uint32_t i = threadIdx.x; i < rows * a.vectors.d; i += kZeroThreads) {
      const uint32_t r = a.vectors.quotient(i);
      if (named[r / 32] >> (r % 32) & 1) continue;
      const int64_t mine = first + r, row = (((mine >> a.shift) * step + blockIdx.x) << a.shift) + (mine & in_chunk);
      if (row >= a.vocab) continue;
      T* const out = (T*)a.dweight + row * a.lddw;
      const int64_t col = (int64_t)(i - r * a.vectors.d) * 8 - row_phase(out);
      if (col < a.cols) store_columns(out, col, a.cols, zeros);
    }
    __syncthreads();  // the bits are written again
  }
  wait_for_kernel_before();  // so that the next kernel, which waits for this one, has waited for the sort too
}

// ---------------------------------------------------------------- sums

struct SumArgs {
  uint32_t items;    // threads with work in this launch
  FastDiv vectors;   // of a row, at any phase; a thread's is the remainder
  int64_t tile0;     // the launch's first tile
  int64_t tokens, vocab, cols;
  int32_t tile;
  const uint32_t *key, *place, *longs;
  const void* dy;
  int64_t lddy;
  float scale;
  void* dweight;
  int64_t lddw;
  int32_t accumulate;
  float* parts;  // [tiles][2][vectors * 8]: a tile's part of a long run that began before it, and of one that begins in it
};

__device__ __forceinline__ float* part_of(const SumArgs& a, int64_t tile, int which, uint32_t vector) {
  return a.parts + ((tile * 2 + which) * a.vectors.d + vector) * 8;
}

// The column that a vector of a row of dweight starts at.
template <typename T, bool ANY>
__device__ __forceinline__ int64_t column(const SumArgs& a, int64_t row, uint32_t vector) {
  return (int64_t)vector * 8 - (ANY ? row_phase((const T*)a.dweight + row * a.lddw) : 0);
}

template <typename T, bool ANY>
__device__ __forceinline__ void store_sum(const SumArgs& a, int64_t row, uint32_t vector, float (&sum)[8]) {
  T* const out = (T*)a.dweight + row * a.lddw;
  const int64_t col = column<T, ANY>(a, row, vector);
  if (col >= a.cols) return;
  float old[8];
  if (a.accumulate) load_columns(out, col, a.cols, old);
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = a.accumulate ? fmaf(sum[k], a.scale, old[k]) : sum[k] * a.scale;
  if constexpr (ANY)
    store_columns(out, col, a.cols, sum);
  else
    store_vec<8>(out + col, sum);
}

// Rows of dy on their way to a thread, through slots of its own in shared memory by asynchronous
// copies of 16 bytes, which take no registers: with them eight rows ahead, not four, and four blocks
// an SM, not two (16384 rows of 8192 bf16 into 131072: 108 us became 64).  Of rows of any alignment (ANY) the granules
// that hold a vector are copied, one more than a vector fills, and it is cut out when it is added.
// Granules reach up to 31 bytes past a row, but never past the matrix: at its ends elements go one by
// one.
template <typename T, bool ANY, int kAhead>
struct Coming {
  static constexpr int kGranules = (int)sizeof(T) / 2 + ANY;
  static constexpr int kBytes = kAhead * kGranules * 16 * kThreads;
  uint4* mine;  // [kAhead][kGranules][kThreads], this thread's
  uintptr_t first, last;  // the matrix's bytes
  int64_t whole;          // granules that begin less than this behind `first` lie inside

  __device__ __forceinline__ Coming(uint4* ring, const void* dy, int64_t rows, int64_t ld, int64_t cols)
      : mine(ring + threadIdx.x), first((uintptr_t)dy), last((uintptr_t)dy + ((rows - 1) * ld + cols) * sizeof(T)),
        whole((int64_t)(last - first) - 16 * kGranules) {}
  __device__ __forceinline__ void fetch(int slot, const T* p) {
    const uintptr_t from = (uintptr_t)p & ~(uintptr_t)15;
    uint4* const to = mine + slot * kGranules * kThreads;
    const int64_t behind = (int64_t)(from - first);
    if (!ANY || (behind >= 0 && behind <= whole)) {
#pragma unroll
      for (int g = 0; g < kGranules; ++g)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to + g * kThreads)), "l"(from + g * 16)
                     : "memory");
    } else {
      for (int g = 0; g < kGranules; ++g)
        for (int e = 0; e < 16; e += (int)sizeof(T)) {
          const uintptr_t at = from + g * 16 + e;
          if (at >= first && at < last)
            *reinterpret_cast<T*>(reinterpret_cast<unsigned char*>(to + g * kThreads) + e) = *reinterpret_cast<const T*>(at);
        }
    }
  }
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
  template <int BYTES>
  __device__ __forceinline__ void add_shifted(int slot, float (&sum)[8]) {
    uint32_t w[4 * kGranules];
#pragma unroll
    for (int g = 0; g < kGranules; ++g) {
      if (16 * g >= BYTES + 8 * (int)sizeof(T)) continue;  // nothing of it
      const uint4 u = mine[(slot * kGranules + g) * kThreads];
      w[4 * g] = u.x, w[4 * g + 1] = u.y, w[4 * g + 2] = u.z, w[4 * g + 3] = u.w;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int at = BYTES + k * (int)sizeof(T);
      if constexpr (sizeof(T) == 2)
        sum[k] += __uint_as_float(at % 4 ? w[at / 4] & 0xffff0000u : w[at / 4] << 16);
      else
        sum[k] += __uint_as_float(w[at / 4]);
    }
  }
  // phase: bytes by which the vector lies past a granule's start; a row's vectors all have the same.
  __device__ __forceinline__ void add(int slot, int phase, float (&sum)[8]) {
    if constexpr (!ANY) return add_shifted<0>(slot, sum);
    switch (phase) {
      case 0: return add_shifted<0>(slot, sum);
      case 4: return add_shifted<4>(slot, sum);
      case 8: return add_shifted<8>(slot, sum);
      case 12: return add_shifted<12>(slot, sum);
    }
    if constexpr (sizeof(T) == 2) {
      switch (phase) {
        case 2: return add_shifted<2>(slot, sum);
        case 6: return add_shifted<6>(slot, sum);
        case 10: return add_shifted<10>(slot, sum);
        default: return add_shifted<14>(slot, sum);
      }
    }
  }
};

// ANY: rows of any alignment; the vectors of a row of dweight start on its 16-byte boundaries.
// kAhead rows of dy are on their way to a thread, and the place of the one behind them.
template <typename T, bool ANY, int kAhead>
__global__ void __launch_bounds__(kThreads, 4) runs_kernel(const SumArgs a) {
  extern __shared__ __align__(16) uint4 ring[];
  wait_for_kernel_before();
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.items) return;
  const uint32_t down = a.vectors.quotient(i), vector = i - down * a.vectors.d;
  const uint32_t n = (uint32_t)a.tokens, tile = (uint32_t)a.tile, none = (uint32_t)a.vocab;
  const int64_t t = a.tile0 + down;
  const uint32_t begin = (uint32_t)t * tile, end = min(begin + tile, n), next_end = min(end + tile, n);  // below 2^31 + 2^7
  // The keys at the tile's ends, beside it, and beside its neighbours.
  const uint32_t first = a.key[begin], last = a.key[end - 1], before = begin > 0 ? a.key[begin - 1] : none,
                 two_before = begin > tile ? a.key[begin - tile - 1] : none, behind = end < n ? a.key[end] : none,
                 two_behind = next_end < n ? a.key[next_end] : none;
  if (first >= none) return;
  // The run that has begun before: the tile before sums it, if it begins in that one and ends in
  // this; else it is left in parts.
  bool head = before == first;
  const bool skip = head && two_before != first && behind != first;
  // The last run goes on to the end of the next tile at most, if it begins in this one.
  const bool goes_on = behind == last && last < none, further = goes_on && two_behind != last && !(head && first == last);
  const uint32_t stop = further ? next_end : end;
  Coming<T, ANY, kAhead> coming(ring, a.dy, n, a.lddy, a.cols);
  auto source = [&](uint32_t key, uint32_t place) {
    return (const T*)a.dy + (int64_t)place * a.lddy + column<T, ANY>(a, key, vector);
  };
  auto fetch = [&](int slot, uint32_t p, uint32_t key, uint32_t place) {
    if (p < stop && key < none && !(skip && key == first) && (p < end || key == last)) {
      coming.fetch(slot, source(key, place));
    }
    coming.commit();
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const uint32_t p = min(begin + j, n - 1);
    fetch(j, begin + j, a.key[p], a.place[p]);
  }
  uint32_t key = first, here = first, here_place = a.place[begin];
  // Of the place that comes kAhead behind.
  uint32_t far_key = a.key[min(begin + kAhead, n - 1)], far_place = a.place[min(begin + kAhead, n - 1)];
  float sum[8] = {};
  auto flush = [&](bool part) {
    if (part) {
      if (!skip || !head) store_vec<8>(part_of(a, t, head ? 0 : 1, vector), sum);
    } else {
      store_sum<T, ANY>(a, key, vector, sum);
    }
  };
  int slot = 0;
#pragma unroll 1
  for (uint32_t p = begin; p < stop; ++p) {
    const uint32_t next = min(p + 1, n - 1), far = min(p + kAhead + 1, n - 1);
    const uint32_t next_here = a.key[next], next_place = ANY ? a.place[next] : 0, next_far_key = a.key[far], next_far_place = a.place[far];
    if (here != key) {
      flush(head);
      head = false;
      key = here;
      if (key >= none || p >= end) break;
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] = 0.0f;
    }
    coming.wait();
    if (!(skip && key == first)) coming.add(slot, ANY ? (int)((uintptr_t)source(key, here_place) & 15) : 0, sum);
    fetch(slot, p + kAhead, far_key, far_place);
    here = next_here, here_place = next_place, far_key = next_far_key, far_place = next_far_place;
    if (++slot == kAhead) slot = 0;
    if (p + 1 == stop) flush(head || (goes_on && !further));
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

constexpr int kJoinThreads = 512;

// Joins a long run's parts for 32 vectors: a thread of each warp a vector, and their sums in order.
template <typename T, bool ANY>
__global__ void __launch_bounds__(kJoinThreads, 2) join_kernel(const SumArgs a) {
  __shared__ __align__(16) float joined[kJoinThreads / 32][32][8];
  wait_for_kernel_before();
  const uint32_t chunks = (a.vectors.d + 31) / 32;
  const int64_t items = (int64_t)a.longs[0] * chunks;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int64_t t = a.longs[1 + i / chunks];
    const uint32_t vector = (uint32_t)(i % chunks) * 32 + lane, key = a.key[(t + 1) * a.tile];
    // Tiles behind t that begin with the key: the run's other parts.
    int64_t more = 0;
    for (;;) {
      const int64_t p = (t + 1 + more + threadIdx.x) * a.tile;
      const int found = __syncthreads_count(p < a.tokens && a.key[p] == key);
      more += found;
      if (found < kJoinThreads) break;
    }
    float sum[8] = {};
    if (vector < a.vectors.d) {
#pragma unroll 4
      for (int64_t j = warp; j <= more; j += kJoinThreads / 32) {
        float v[8];
        load_vec<8>(part_of(a, t + j, j == 0, vector), v);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] += v[c];
      }
    }
    store_vec<8>(joined[warp][lane], sum);
    __syncthreads();
    if (warp == 0 && vector < a.vectors.d) {
#pragma unroll 8
      for (int w = 1; w < kJoinThreads / 32; ++w) {
        float v[8];
        load_vec<8>(joined[w][lane], v);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] += v[c];
      }
      store_sum<T, ANY>(a, key, vector, sum);
    }
    __syncthreads();  // the sums are written again
  }
}

// ---------------------------------------------------------------- few tokens

// One launch and no workspace, for 512 tokens at most and 2^21 elements of dweight, or 64 and 2^24: 512 into 1000 x 64 bf16
// 4.9 us against 14.4 with the sort, 100 into 300 x 101 6.9 against 14.9; 512 into 32000 x 2048 are
// 36 against 33, and, all of one token, into 1000 x 8192 44 against 16.  A block looks at all ids by itself, lists those of its rows of dweight
// in the rows' order, and writes kFewVectors vectors of each row.  A run of more than kFewLong rows
// is added up by all of the block's warps.
constexpr int kFew = 512, kFewRows = 128, kFewVectors = 128, kFewLong = 16;
constexpr int kVeryFew = 64;
constexpr int64_t kFewElements = 1 << 21, kVeryFewElements = 1 << 24, kFewBytes = 64 << 10;
static_assert(kFew == 2 * kThreads, "two ids a thread");

struct FewArgs {
  int64_t tokens, vocab, cols;
  int32_t index;
  const void* ids;
  const void* dy;
  int64_t lddy;
  float scale;
  void* dweight;
  int64_t lddw;
  int32_t accumulate;
  int32_t rows;        // of dweight a block
  FastDiv slabs;       // blocks beside each other
  FastDiv vectors;     // of a row in a block, the last of them perhaps beyond the row
};

template <typename T, bool ANY>
__global__ void __launch_bounds__(kThreads, 4) few_kernel(const FewArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ uint16_t row_of[kFew], place_of[kFew], place[kFew];  // by place; by row
  __shared__ uint16_t begins[kFewRows + 1];
  __shared__ int warp_count[kWarps];
  __shared__ __align__(16) float joined[kWarps][kFewVectors][8];
  const int x = threadIdx.x, warp = x / 32, lane = x % 32;
  const uint32_t down = a.slabs.quotient(blockIdx.x), slab = blockIdx.x - down * a.slabs.d;
  const int64_t row0 = (int64_t)down * a.rows;
  const int rows = (int)min((int64_t)a.rows, a.vocab - row0);
  int mine[2], count = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = 2 * x + j, token = t < a.tokens ? token_at(a.ids, a.index, t, a.vocab) : -1;
    mine[j] = token >= row0 && token < row0 + rows ? (int)(token - row0) : -1;
    count += mine[j] >= 0;
  }
  int up = count;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, up, d);
    if (lane >= d) up += o;
  }
  if (lane == 31) warp_count[warp] = up;
  __syncthreads();
  int at = up - count, n = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += warp_count[w];
    n += warp_count[w];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (mine[j] >= 0) row_of[at] = (uint16_t)mine[j], place_of[at++] = (uint16_t)(2 * x + j);
  __syncthreads();
  for (int i = x; i < n; i += kThreads) {  // behind those of lower rows, and those before of its own
    const int r = row_of[i];
    int to = 0;
    for (int j = 0; j < n; ++j) to += row_of[j] < r || (row_of[j] == r && j < i);
    place[to] = place_of[i];
  }
  for (int r = x; r <= rows; r += kThreads) {
    int to = 0;
    for (int j = 0; j < n; ++j) to += row_of[j] < r;
    begins[r] = (uint16_t)to;
  }
  __syncthreads();

  auto column_of = [&](int64_t row, uint32_t v) {
    return ((int64_t)slab * kFewVectors + v) * 8 - (ANY ? row_phase((const T*)a.dweight + row * a.lddw) : 0);
  };
  auto add = [&](float (&sum)[8], int p, int64_t col) {
    const T* row = (const T*)a.dy + (int64_t)place[p] * a.lddy;
    float v[8];
    if constexpr (ANY)
      load_columns(row, col, a.cols, v);
    else
      load_vec<8>(row + col, v);
#pragma unroll
    for (int c = 0; c < 8; ++c) sum[c] += v[c];
  };
  // by: the scale, but 0 of a row that no id names: its zeros have a sign, or are NaN, by some scales.
  auto store = [&](float (&sum)[8], int64_t row, int64_t col, float by) {
    T* const out = (T*)a.dweight + row * a.lddw;
    float old[8];
    if (a.accumulate) load_columns(out, col, a.cols, old);
#pragma unroll
    for (int c = 0; c < 8; ++c) sum[c] = a.accumulate ? fmaf(sum[c], by, old[c]) : sum[c] * by;
    if constexpr (ANY)
      store_columns(out, col, a.cols, sum);
    else
      store_vec<8>(out + col, sum);
  };
  for (uint32_t i = x; i < rows * a.vectors.d; i += kThreads) {
    const uint32_t r = a.vectors.quotient(i), v = i - r * a.vectors.d;
    const int begin = begins[r], end = begins[r + 1];
    if (end - begin > kFewLong || (begin == end && a.accumulate)) continue;
    const int64_t row = row0 + r, col = column_of(row, v);
    if (col >= a.cols) continue;
    float sum[8] = {};
#pragma unroll 4
    for (int p = begin; p < end; ++p) add(sum, p, col);
    store(sum, row, col, begin == end ? 0.0f : a.scale);
  }
  if (n <= kFewLong) return;
  for (int r = 0; r < rows; ++r) {
    const int begin = begins[r], end = begins[r + 1];
    if (end - begin <= kFewLong) continue;
    const int64_t row = row0 + r;
    __syncthreads();  // what the last run left has been read
    for (uint32_t v = lane; v < a.vectors.d; v += 32) {
      const int64_t col = column_of(row, v);
      float sum[8] = {};
      if (col < a.cols) {
#pragma unroll 4
        for (int p = begin + warp; p < end; p += kWarps) add(sum, p, col);
      }
      store_vec<8>(joined[warp][v], sum);
    }
    __syncthreads();
    for (uint32_t v = x; v < a.vectors.d; v += kThreads) {
      const int64_t col = column_of(row, v);
      if (col >= a.cols) continue;
      float sum[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        float t[8];
        load_vec<8>(joined[w][v], t);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] += t[c];
      }
      store(sum, row, col, a.scale);
    }
  }
}

// ---------------------------------------------------------------- host side

template <typename T>
tide_status embed(EmbedArgs a, int64_t tokens, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.weight, a.ldw, sizeof(T), a.vocab) &&
                   rows_aligned(a.out, a.ldo, sizeof(T), tokens);
  const int64_t per_row = vec ? a.cols / 8 : (a.cols + 14) / 8;  // vectors that any phase of a row touches
  a.per_row = FastDiv((uint32_t)per_row);
  // Few vectors: one a thread, on more SMs.
  const bool few = tokens * per_row <= (int64_t)ops_num_sms() * 2048;
  return in_row_launches(tokens, per_row, vec && !few ? kThreads * 4 : kThreads, "embedding",
                         [&](int64_t r, uint32_t items, unsigned grid) {
                           a.row0 = r, a.items = items;
                           if (!vec)
                             embed_any_kernel<T><<<grid, kThreads, 0, stream>>>(a);
                           else if (few)
                             embed_vec_kernel<T, 1><<<grid, kThreads, 0, stream>>>(a);
                           else
                             embed_vec_kernel<T, 4><<<grid, kThreads, 0, stream>>>(a);
                         });
}

// Places a tile: few, while that leaves less than two turns of the SMs' threads, since a thread's
// places follow one another; many, since runs of more than a tile or two go through memory.
int tile_of(int64_t tokens, int64_t vectors) {
  const int64_t enough = (int64_t)std::max(ops_num_sms(), 1) * 2048;
  int tile = 64;
  while (tile > 8 && tokens / tile * vectors < enough) tile /= 2;
  return tile;
}

// The workspace: sorted keys and places, twice; the long runs; their parts.  Few tokens need none.
struct GradSpace {
  int64_t list = 0, longs = 0, parts = 0, bytes = 0;
  int tile = 0;
};
bool few(int64_t tokens, int64_t vocab, int64_t cols) {
  return tokens <= kFew && vocab <= (tokens <= kVeryFew ? kVeryFewElements : kFewElements) / cols;
}
GradSpace grad_space(int64_t tokens, int64_t vocab, int64_t cols) {
  GradSpace g;
  if (tokens == 0 || few(tokens, vocab, cols)) return g;
  const int64_t vectors = (cols + 14) / 8;
  g.tile = tile_of(tokens, vectors);
  const int64_t tiles = (tokens + g.tile - 1) / g.tile;
  g.list = (tokens * 4 + 15) / 16 * 16;
  g.longs = (4 + tiles * 4 + 15) / 16 * 16;
  g.parts = tiles > 2 ? tiles * 2 * vectors * 32 : 0;
  g.bytes = 4 * g.list + g.longs + g.parts;
  return g;
}

// Up to 64 KB of dweight a block, less where that would leave the GPU with fewer blocks than it holds.
template <typename T>
tide_status embed_grad_few(FewArgs a, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.dy, a.lddy, sizeof(T), a.tokens) &&
                   rows_aligned(a.dweight, a.lddw, sizeof(T), a.vocab);
  const int64_t vectors = vec ? a.cols / 8 : (a.cols + 14) / 8, slabs = (vectors + kFewVectors - 1) / kFewVectors;
  const int64_t here = std::min<int64_t>(vectors, kFewVectors), most = (int64_t)std::max(ops_num_sms(), 1) * 4;
  a.slabs = FastDiv((uint32_t)slabs), a.vectors = FastDiv((uint32_t)here);
  a.rows = 1;
  while (a.rows < kFewRows && a.rows * here * 8 * (int64_t)sizeof(T) < kFewBytes && a.vocab / (2 * a.rows) * slabs >= most)
    a.rows *= 2;
  const int64_t grid = (a.vocab + a.rows - 1) / a.rows * slabs;
  if (grid > INT32_MAX) return fail(TIDE_ERR_UNIMPLEMENTED, "embedding gradient: too many rows for one launch");
  if (vec)
    few_kernel<T, false><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  else
    few_kernel<T, true><<<(unsigned)grid, kThreads, 0, stream>>>(a);
  return cuda_status(cudaGetLastError(), "embedding gradient");
}

template <typename T>
tide_status embed_grad(SumArgs a, SortArgs s, cudaStream_t stream) {
  const char* const what = "embedding gradient";
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.dy, a.lddy, sizeof(T), a.tokens) &&
                   rows_aligned(a.dweight, a.lddw, sizeof(T), a.vocab);
  const int sms = ops_num_sms();
  if (sms <= 0) return fail(TIDE_ERR_CUDA, "the current device could not be queried");
  const int64_t vectors = vec ? a.cols / 8 : (a.cols + 14) / 8;
  a.vectors = FastDiv((uint32_t)vectors);
  int bits = 1;
  while (a.vocab >> bits) ++bits;  // keys are 0 .. vocab
  s.passes = (bits + kDigitBits - 1) / kDigitBits;
  // Few ids: a block's warps have them all in registers.
  const int cluster = a.tokens > 1024 ? kSortCluster : 1;
  if (a.tokens > 0) {
    const ClusterLaunch l(cluster, dim3(kSortThreads), cluster, false, 0, stream);
    TIDE_TRY(cuda_status(cudaLaunchKernelEx(&l.cfg, sort_kernel, s), what));
  }
  if (!a.accumulate) {
    // The sort's SMs have no room: a block there would be as late as the sort is long.
    const int most = std::max(1, sms - cluster);
    int shift = 0;
    while ((a.vocab >> shift) > 4 * most && (vectors * 8 * (int64_t)sizeof(T) << shift) < kZeroChunk) ++shift;
    const int grid = (int)std::min<int64_t>(most, (a.vocab + (1 << shift) - 1) >> shift);
    const ZeroArgs z{a.tokens, a.vocab, a.cols, s.index, s.ids, a.dweight, a.lddw, a.vectors, FastDiv((uint32_t)grid), shift};
    const ClusterLaunch l(grid, dim3(kZeroThreads), 1, a.tokens > 0, 0, stream);
    TIDE_TRY(cuda_status(cudaLaunchKernelEx(&l.cfg, zero_kernel<T>, z), what));
  }
  if (a.tokens == 0) return TIDE_OK;
  const int64_t tiles = (a.tokens + a.tile - 1) / a.tile;
  cudaError_t err = cudaSuccess;
  TIDE_TRY(in_row_launches(tiles, vectors, kThreads, what, [&](int64_t t, uint32_t items, unsigned blocks) {
    a.tile0 = t, a.items = items;
    // 32 KB of slots a block, or 48.
    constexpr int kAhead = sizeof(T) == 2 ? 8 : 4, kAnyAhead = sizeof(T) == 2 ? 6 : 4;
    const int room = vec ? Coming<T, false, kAhead>::kBytes : Coming<T, true, kAnyAhead>::kBytes;
    const ClusterLaunch l(blocks, dim3(kThreads), 1, true, room, stream);
    if (err == cudaSuccess)
      err = vec ? cudaLaunchKernelEx(&l.cfg, runs_kernel<T, false, kAhead>, a)
                : cudaLaunchKernelEx(&l.cfg, runs_kernel<T, true, kAnyAhead>, a);
  }));
  TIDE_TRY(cuda_status(err, what));
  if (tiles <= 2) return TIDE_OK;  // no run goes on beyond a second tile
  const ClusterLaunch l(sms * 2, dim3(kJoinThreads), 1, true, 0, stream);
  return cuda_status(vec ? cudaLaunchKernelEx(&l.cfg, join_kernel<T, false>, a) : cudaLaunchKernelEx(&l.cfg, join_kernel<T, true>, a),
                     what);
}

tide_status check_embedding(int64_t tokens, int64_t vocab, int64_t cols, int32_t index, int32_t dtype, const void* ids) {
  TIDE_TRY(check_sizes(tokens, cols, "embedding"));
  TIDE_TRY(check_sizes(vocab, 0, "embedding"));
  TIDE_TRY(check_dtype(dtype));
  TIDE_TRY(check_index(index));
  if (tokens > INT32_MAX || vocab >= INT32_MAX) return fail(TIDE_ERR_UNIMPLEMENTED, "embedding: 2^31 tokens or rows");
  if (cols > kMaxCols) return fail(TIDE_ERR_UNIMPLEMENTED, "embedding: rows longer than 2^24");
  return check_matrix(ids, 1, tokens, tokens, index_bytes_of(index), "ids");
}

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" {

tide_status tide_embedding(int64_t tokens, int64_t vocab, int64_t cols, int32_t index, const void* ids, int32_t dtype,
                           const void* weight, int64_t ldw, float scale, void* out, int64_t ldo, void* stream) {
  clear_error();
  TIDE_TRY(check_embedding(tokens, vocab, cols, index, dtype, ids));
  if (tokens == 0 || cols == 0) return TIDE_OK;
  const int64_t e = elem_bytes_of(dtype);
  TIDE_TRY(check_matrix(weight, vocab, cols, ldw, e, "weight"));
  TIDE_TRY(check_matrix(out, tokens, cols, ldo, e, "out"));
  const EmbedArgs a{0, FastDiv(), 0, vocab, cols, index, ids, weight, ldw, scale, out, ldo};
  return dtype == TIDE_BF16 ? embed<bf16>(a, tokens, (cudaStream_t)stream) : embed<float>(a, tokens, (cudaStream_t)stream);
}

int64_t tide_embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t cols) {
  if (tokens <= 0 || vocab <= 0 || cols <= 0 || tokens > INT32_MAX || cols > kMaxCols) return 0;
  return grad_space(tokens, vocab, cols).bytes;
}

tide_status tide_embedding_backward(int64_t tokens, int64_t vocab, int64_t cols, int32_t index, const void* ids,
                                    int32_t dtype, const void* dy, int64_t lddy, float scale, void* dweight,
                                    int64_t lddw, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                    void* stream) {
  clear_error();
  TIDE_TRY(check_embedding(tokens, vocab, cols, index, dtype, ids));
  if (vocab == 0 || cols == 0 || (tokens == 0 && accumulate)) return TIDE_OK;
  const int64_t e = elem_bytes_of(dtype);
  TIDE_TRY(check_matrix(dy, tokens, cols, lddy, e, "dy"));
  TIDE_TRY(check_matrix(dweight, vocab, cols, lddw, e, "dweight"));
  const int64_t need = tide_embedding_backward_workspace(tokens, vocab, cols);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(TIDE_ERR_INVALID_ARG, "workspace too small: " + std::to_string(need) + " bytes are needed");
  if ((uintptr_t)workspace % 16) return fail(TIDE_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  if (few(tokens, vocab, cols)) {
    const FewArgs f{tokens, vocab, cols, index, ids, dy, lddy, scale, dweight, lddw, accumulate, 0, FastDiv(), FastDiv()};
    return dtype == TIDE_BF16 ? embed_grad_few<bf16>(f, (cudaStream_t)stream) : embed_grad_few<float>(f, (cudaStream_t)stream);
  }
  const GradSpace g = grad_space(tokens, vocab, cols);
  uint8_t* const w = (uint8_t*)workspace;
  uint32_t* list[4];
  for (int i = 0; i < 4; ++i) list[i] = (uint32_t*)(w + i * g.list);
  uint32_t* const longs = (uint32_t*)(w + 4 * g.list);
  float* const parts = (float*)(w + 4 * g.list + g.longs);
  const SortArgs s{tokens, vocab, index, ids, list[0], list[1], list[2], list[3], 0, g.tile, longs};
  const SumArgs a{0,  FastDiv(), 0,     tokens,  vocab, cols,       g.tile, list[0], list[1], longs,
                  dy, lddy,      scale, dweight, lddw,  accumulate, parts};
  return dtype == TIDE_BF16 ? embed_grad<bf16>(a, s, (cudaStream_t)stream) : embed_grad<float>(a, s, (cudaStream_t)stream);
}

}  // extern "C"
