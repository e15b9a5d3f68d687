// Token embedding, and its gradient by sorted tokens (include/tide_lm_ops.h).
//
// Forward: rows of the table are copied, scaled on the way; bound by memory traffic.
//
// Backward, dweight[v] = scale * sum of dy[t] over the t with token v, is dense: every row
// of dweight is written once, the rows of dy are read once, and both dwarf the ids.
//   1. A cluster of blocks sorts the ids, stably, by eight bits at a time (their places
//      with them), so that a token's rows of dy are a run of places in ascending order: the sum's order
//      is fixed.
//   2. Tokens that fill whole tiles of kTile sorted places (padding, separators, articles) have
//      these tiles' rows summed, a tile a block, so that no block is left with a run of thousands.
//   3. A block takes kRows rows of dweight by kCols columns, finds its tokens' runs by binary
//      search, and writes zeros or sums.  A run of more than kLong rows is added up by all of the
//      block's warps, with the tiles' sums in the place of their rows.

#include <algorithm>

#include "cluster_ptx.cuh"
#include "lm_common.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
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
  if (token >= 0) load_columns((const T*)a.weight + token * a.ldw, col, a.cols, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= a.scale;
  store_columns(out, col, a.cols, v);
}

// ---------------------------------------------------------------- sorting

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kDigits = 256;
constexpr int kSortCluster = 8;

struct SortArgs {
  int64_t tokens, vocab;
  int32_t index;
  const void* ids;
  uint32_t *key, *place;    // out, sorted by key; ids outside the vocabulary have key vocab
  uint32_t *key2, *place2;  // scratch
  int passes;
};

// A stable counting sort a digit of eight bits.  The cluster's warps take consecutive parts of
// the places; a warp walks its part 32 places at a time, and equal digits among those are
// ranked by lane.
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const SortArgs a) {
  __shared__ uint32_t counts[kSortWarps][kDigits];
  __shared__ uint32_t totals[kDigits];  // the block's
  __shared__ uint32_t scan[kDigits / 32];
  const uint32_t blocks = cluster_size(), rank = cluster_rank();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t n = (uint32_t)a.tokens, parts = blocks * kSortWarps;
  const uint32_t part = (uint32_t)(((uint64_t)n + parts * 32 - 1) / (parts * 32) * 32);
  const uint64_t begin = min((uint64_t)(rank * kSortWarps + warp) * part, (uint64_t)n), end = min(begin + part, (uint64_t)n);
  for (int pass = 0; pass < a.passes; ++pass) {
    // The last pass ends in key and place.
    const bool to_first = (a.passes - pass) % 2 == 1;
    const uint32_t *key = to_first ? a.key2 : a.key, *place = to_first ? a.place2 : a.place;
    uint32_t *key_out = to_first ? a.key : a.key2, *place_out = to_first ? a.place : a.place2;
    const int shift = pass * 8;
    auto key_at = [&](uint64_t i) {
      if (pass == 0) {
        const int t = token_at(a.ids, a.index, (int64_t)i, a.vocab);
        return t >= 0 ? (uint32_t)t : (uint32_t)a.vocab;
      }
      return __ldcg(key + i);
    };
    for (int d = lane; d < kDigits; d += 32) counts[warp][d] = 0;
    __syncwarp();
    for (uint64_t i = begin + lane; i < end; i += 32) atomicAdd(&counts[warp][(key_at(i) >> shift) & 255], 1u);
    __syncthreads();
    uint32_t sum = 0;
    if (threadIdx.x < kDigits) {
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = counts[w][threadIdx.x];
        counts[w][threadIdx.x] = sum;
        sum += c;
      }
      totals[threadIdx.x] = sum;
    }
    cluster_sync();
    if (threadIdx.x < kDigits) {  // where each digit's keys of this block begin
      uint32_t before = 0, all = 0;
      for (uint32_t b = 0; b < blocks; ++b) {
        const uint32_t c = load_peer_u32(peer_smem(&totals[threadIdx.x], b));
        if (b < rank) before += c;
        all += c;
      }
      uint32_t up = all;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += o;
      }
      if (lane == 31) scan[warp] = up;
      sum = before + up - all;
    }
    __syncthreads();
    if (threadIdx.x < kDigits) {
      for (int w = 0; w < warp; ++w) sum += scan[w];
      for (int w = 0; w < kSortWarps; ++w) counts[w][threadIdx.x] += sum;
    }
    __syncthreads();
    for (uint64_t i0 = begin; i0 < end; i0 += 32) {
      const uint64_t i = i0 + lane;
      const bool here = i < end;
      const uint32_t k = here ? key_at(i) : 0;
      const uint32_t digit = here ? (k >> shift) & 255 : kDigits;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      const uint32_t rank_in = __popc(same & ((1u << lane) - 1));
      const uint32_t base = here ? counts[warp][digit] : 0;
      __syncwarp();
      if (here) {
        if (rank_in == 0) counts[warp][digit] = base + __popc(same);
        key_out[base + rank_in] = k;
        place_out[base + rank_in] = pass == 0 ? (uint32_t)i : __ldcg(place + i);
      }
      __syncwarp();
    }
    __threadfence();
    cluster_sync();
  }
}

// ---------------------------------------------------------------- sums

constexpr int kTile = 64;                 // sorted places of a tile
constexpr int kRows = 32;                 // rows of dweight a block
constexpr int kSteps = 4;                 // vectors of a row a lane holds
constexpr int kCols = kSteps * 256;       // columns a block
constexpr int kLong = 64;                 // rows of a run that one warp adds up

struct SumArgs {
  int64_t tokens, vocab, cols;
  const uint32_t *key, *place;
  const void* dy;
  int64_t lddy;
  float scale;
  void* dweight;
  int64_t lddw;
  int32_t accumulate;
  float* tiles;    // [whole tiles][ldt]: sums of the tiles of one token; NULL: none are made
  int64_t ldt;
  FastDiv slabs;   // blocks beside each other
};

// A lane's columns of a block's: kSteps vectors of eight, a warp's width (256) apart.
struct Columns {
  float v[kSteps][8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[s][k] = 0.0f;
  }
};

// Adds row `p` (of `cols`) from column `col` on.
template <bool ANY, typename T>
__device__ __forceinline__ void add_row(Columns& c, const T* p, int64_t col, int64_t cols) {
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t at = col + s * 256;
    if (at >= cols) continue;
    float t[8];
    if constexpr (ANY)
      load_columns(p, at, cols, t);
    else
      load_vec<8>(p + at, t);
#pragma unroll
    for (int k = 0; k < 8; ++k) c.v[s][k] += t[k];
  }
}

// A block: a tile by kCols columns.  Only tiles of one token; warp w adds rows w, w + 8, ...
template <typename T, bool ANY>
__global__ void __launch_bounds__(kThreads) tiles_kernel(const SumArgs a) {
  __shared__ __align__(16) float joined[kWarps][kCols];
  wait_for_kernel_before();
  const int64_t first = (int64_t)blockIdx.x * kTile;
  const uint32_t token = a.key[first];
  if (token >= (uint32_t)a.vocab || a.key[first + kTile - 1] != token) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t col0 = (int64_t)blockIdx.y * kCols, col = col0 + lane * 8;
  Columns c;
  c.zero();
#pragma unroll 2
  for (int i = warp; i < kTile; i += kWarps)
    add_row<ANY>(c, (const T*)a.dy + (int64_t)a.place[first + i] * a.lddy, col, a.cols);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) store_vec<8>(&joined[warp][s * 256 + lane * 8], c.v[s]);
  __syncthreads();
  for (int i = threadIdx.x; i < kCols; i += kThreads) {
    float v = 0.0f;
    for (int w = 0; w < kWarps; ++w) v += joined[w][i];
    if (col0 + i < a.cols) a.tiles[(int64_t)blockIdx.x * a.ldt + col0 + i] = v;
  }
}

// First place whose key is not below `key`.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t n, uint32_t key) {
  uint32_t lo = 0;
  while (n > 0) {
    const uint32_t half = n / 2;
    if (keys[lo + half] < key)
      lo += half + 1, n -= half + 1;
    else
      n = half;
  }
  return lo;
}

template <typename T, bool ANY>
__device__ __forceinline__ void store_row(const SumArgs& a, int64_t row, int64_t col, Columns& c) {
  T* const out = (T*)a.dweight + row * a.lddw;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t at = col + s * 256;
    if (at >= a.cols) continue;
    float old[8];
    if (a.accumulate) {
      if constexpr (ANY)
        load_columns(out, at, a.cols, old);
      else
        load_vec<8>(out + at, old);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) c.v[s][k] = a.accumulate ? fmaf(c.v[s][k], a.scale, old[k]) : c.v[s][k] * a.scale;
    if constexpr (ANY)
      store_columns(out, at, a.cols, c.v[s]);
    else
      store_vec<8>(out + at, c.v[s]);
  }
}

// ANY: rows of any alignment; the vectors of a row of dweight start on its 16-byte boundaries.
template <typename T, bool ANY>
__global__ void __launch_bounds__(kThreads) sum_kernel(const SumArgs a) {
  __shared__ uint32_t begins[kRows + 1];
  __shared__ __align__(16) float joined[kWarps][kCols];
  wait_for_kernel_before();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t down = a.slabs.quotient(blockIdx.x), slab = blockIdx.x - down * a.slabs.d;
  const int64_t row0 = (int64_t)down * kRows;
  const int rows = (int)min((int64_t)kRows, a.vocab - row0);
  if ((int)threadIdx.x <= rows) begins[threadIdx.x] = lower_bound(a.key, (uint32_t)a.tokens, (uint32_t)(row0 + threadIdx.x));
  __syncthreads();
  const int64_t col0 = (int64_t)slab * kCols;
  Columns c;
  bool any_long = false;
  for (int r = warp; r < rows; r += kWarps) {
    const uint32_t begin = begins[r], end = begins[r + 1];
    if (end - begin > kLong) continue;
    if (begin == end && a.accumulate) continue;
    const int64_t row = row0 + r, col = col0 + lane * 8 - (ANY ? row_phase((T*)a.dweight + row * a.lddw) : 0);
    c.zero();
#pragma unroll 2
    for (uint32_t i = begin; i < end; ++i) add_row<ANY>(c, (const T*)a.dy + (int64_t)a.place[i] * a.lddy, col, a.cols);
    store_row<T, ANY>(a, row, col, c);
  }
  for (int r = 0; r < rows; ++r) any_long |= begins[r + 1] - begins[r] > kLong;
  if (!any_long) return;  // the same for every thread
  for (int r = 0; r < rows; ++r) {
    const uint32_t begin = begins[r], end = begins[r + 1];
    if (end - begin <= kLong) continue;
    const int64_t row = row0 + r, col = col0 + lane * 8 - (ANY ? row_phase((T*)a.dweight + row * a.lddw) : 0);
    // Rows before the first whole tile, the whole tiles, rows behind the last.
    uint32_t head = end, tail = end;
    if (a.tiles) {
      head = min(end, (begin + kTile - 1) / kTile * kTile);
      tail = max(head, end / kTile * kTile);
    }
    c.zero();
#pragma unroll 2
    for (uint32_t i = begin + warp; i < head; i += kWarps)
      add_row<ANY>(c, (const T*)a.dy + (int64_t)a.place[i] * a.lddy, col, a.cols);
#pragma unroll 2
    for (uint32_t i = head / kTile + warp; i < tail / kTile; i += kWarps)
      add_row<ANY>(c, a.tiles + (int64_t)i * a.ldt, col, a.cols);
#pragma unroll 2
    for (uint32_t i = tail + warp; i < end; i += kWarps)
      add_row<ANY>(c, (const T*)a.dy + (int64_t)a.place[i] * a.lddy, col, a.cols);
    __syncthreads();  // what the last run left has been read
#pragma unroll
    for (int s = 0; s < kSteps; ++s) store_vec<8>(&joined[warp][s * 256 + lane * 8], c.v[s]);
    __syncthreads();
    if (warp == 0) {
      c.zero();
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          float t[8];
          load_vec<8>(&joined[w][s * 256 + lane * 8], t);
#pragma unroll
          for (int k = 0; k < 8; ++k) c.v[s][k] += t[k];
        }
      store_row<T, ANY>(a, row, col, c);
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

// The workspace: sorted keys and places, twice, and the whole tiles' sums.
struct GradSpace {
  int64_t list, tiles, ldt, bytes;
};
GradSpace grad_space(int64_t tokens, int64_t cols) {
  GradSpace g;
  g.list = (tokens * 4 + 15) / 16 * 16;
  g.tiles = tokens > 4 * kTile ? tokens / kTile : 0;
  g.ldt = (cols + 3) / 4 * 4;
  g.bytes = 4 * g.list + g.tiles * g.ldt * 4;
  return g;
}

template <typename T>
tide_status embed_grad(SumArgs a, SortArgs s, cudaStream_t stream) {
  const bool vec = a.cols % 8 == 0 && rows_aligned(a.dy, a.lddy, sizeof(T), a.tokens) &&
                   rows_aligned(a.dweight, a.lddw, sizeof(T), a.vocab);
  // With a phase a row may touch one vector more.
  const int64_t wide = vec ? a.cols : a.cols + 7;
  a.slabs = FastDiv((uint32_t)((wide + kCols - 1) / kCols));
  const int64_t grid = (a.vocab + kRows - 1) / kRows * a.slabs.d;
  if (grid > INT32_MAX) return fail(TIDE_ERR_UNIMPLEMENTED, "embedding gradient: too many rows for one launch");
  int bits = 1;
  while (a.vocab >> bits) ++bits;  // keys are 0 .. vocab
  s.passes = (bits + 7) / 8;
  // A block sorts 4096 ids about as fast as a cluster, whose barriers cost more.
  const int cluster = a.tokens > 4096 ? kSortCluster : 1;
  const ClusterLaunch sort(cluster, dim3(kSortThreads), cluster, false, 0, stream);
  TIDE_TRY(cuda_status(cudaLaunchKernelEx(&sort.cfg, sort_kernel, s), "sorting token ids"));
  const GradSpace g = grad_space(a.tokens, a.cols);
  if (g.tiles > 0) {
    ClusterLaunch l(1, dim3(kThreads), 1, true, 0, stream);
    l.cfg.gridDim = dim3((unsigned)g.tiles, (unsigned)((a.cols + kCols - 1) / kCols));
    TIDE_TRY(cuda_status(vec ? cudaLaunchKernelEx(&l.cfg, tiles_kernel<T, false>, a)
                             : cudaLaunchKernelEx(&l.cfg, tiles_kernel<T, true>, a),
                         "embedding gradient, frequent tokens"));
  }
  const ClusterLaunch l(grid, dim3(kThreads), 1, true, 0, stream);
  return cuda_status(vec ? cudaLaunchKernelEx(&l.cfg, sum_kernel<T, false>, a)
                         : cudaLaunchKernelEx(&l.cfg, sum_kernel<T, true>, a),
                     "embedding gradient");
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
  return grad_space(tokens, cols).bytes;
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
  const GradSpace g = grad_space(tokens, cols);
  uint32_t* const w = (uint32_t*)workspace;
  const int64_t n = g.list / 4;
  const SortArgs s{tokens, vocab, index, ids, w, w + n, w + 2 * n, w + 3 * n, 0};
  const SumArgs a{tokens, vocab, cols, w, w + n, dy, lddy, scale, dweight, lddw, accumulate,
                  g.tiles > 0 ? (float*)(w + 4 * n) : nullptr, g.ldt, FastDiv()};
  return dtype == TIDE_BF16 ? embed_grad<bf16>(a, s, (cudaStream_t)stream) : embed_grad<float>(a, s, (cudaStream_t)stream);
}

}  // extern "C"
