// Linear layer: forward with bias, activation and residual, input gradient
// with the previous activation's derivative, weight and bias gradients
// (include/tide_ops.h).

#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <utility>

#include "gemm_tc.cuh"

namespace tide {

tide_status launch_checkpoint_load_bf16(int64_t rows, int64_t cols, const uint8_t* codes, int64_t ldc,
                                        const uint8_t* scales, int64_t lds, int32_t act, void* out, int64_t ldo,
                                        cudaStream_t stream);

namespace {

// Raised where an operator's kernel gives up a wait.  It only grows, so that no
// check takes a report from another: each remembers what it saw (tide_ops_check).
__device__ uint32_t g_timeouts;
std::atomic<int64_t> g_wait_limit_ns{2000000000};
thread_local int64_t g_test_drop = -1;

// One operand: `rows` rows of `cols` contiguous elements.
struct Operand {
  const bf16* p;
  int64_t rows, cols, ld;
};

// Whether TMA can read the operand in place: 16-byte aligned base and rows, and
// a row stride that its descriptor holds.
bool readable(const void* p, int64_t rows, int64_t ld) {
  return (uintptr_t)p % 16 == 0 && (rows <= 1 || (ld % 8 == 0 && ld < (int64_t)1 << 38));
}

int64_t packed_ld(int64_t cols) { return (cols + 7) / 8 * 8; }
int64_t packed_bytes(int64_t rows, int64_t cols) { return (rows * packed_ld(cols) * 2 + 255) / 256 * 256; }

// How a product [m, k] x [n, k] runs.
struct Plan {
  TcTile tile = TILE_256x256;
  int32_t tiles_a = 0, tiles_b = 0, k_blocks = 0, split_blocks = 0, splits = 1;
  int64_t ldp = 0;            // columns of a partial sum, whole tiles
  int64_t partial_bytes = 0;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile and the number of splits with the smallest estimated time, in SM
// clocks: what a CTA sets up and winds down, the turns of the busiest CTA times
// the clocks of a turn (or what DRAM takes to deliver the operands), and the
// joining of splits.  Clocks of a block of 64 of the sum, measured with every SM
// at work (alone, the first two run at the tensor cores' rate, 512 and 256):
// 570 on 256 x 256, 340 on 256 x 128, and 275 to 420 on the single CTA's tiles.
// The epilogues' clocks are fitted to the times of 84 products of 1 to 6000 rows,
// each with every tile and up to 16 splits; the plan they lead to took 2% longer
// than the quickest one on average, at worst 19% (16.6 us instead of 14.0).
Plan choose_plan(int64_t m, int64_t n, int64_t k, bool a_mn, bool vec, int sms) {
  Plan best;
  double best_cost = 1e300;
  const int64_t kb = ceil_div(k, kTcK);
  for (const TcTile t : {TILE_256x256, TILE_256x128, TILE_SWAP_128, TILE_SWAP_SMALL}) {
    const TcTileShape ts = tile_shape(t, a_mn);
    if (t == TILE_SWAP_128 && m <= small_b(a_mn)) continue;
    Plan s;
    s.tile = t;
    s.tiles_a = (int32_t)ceil_div(ts.swap ? n : m, ts.a);
    s.tiles_b = (int32_t)ceil_div(ts.swap ? m : n, ts.b);
    s.k_blocks = (int32_t)kb;
    s.ldp = ts.swap ? s.tiles_a * (int64_t)ts.a : s.tiles_b * (int64_t)ts.b;
    const double block = t == TILE_256x256 ? 570 : t == TILE_256x128 ? 340 : 225 + ts.b * 1.5;
    // The epilogue of a tile, which the next tile's blocks hide if they take
    // longer; `vec`: the output's rows take whole vectors.
    // A plain one (the weight gradient's) loads nothing and needs no activation.
    const int64_t rows = std::min<int64_t>(ceil_div(m, 8) * 8, ts.b);  // of a swapped tile
    const double whole = a_mn ? 550 + (ts.swap ? 18.0 * rows : (vec ? 7.0 : 11.0) * ts.b)
                              : 1800 + (ts.swap ? 73.0 * rows : (vec ? 14.5 : 17.0) * ts.b);
    for (int64_t want = 1; want <= 32 && want <= std::max<int64_t>(1, kb / 4); ++want) {
      s.split_blocks = (int32_t)ceil_div(kb, want);
      s.splits = (int32_t)ceil_div(kb, s.split_blocks);
      if (s.splits != want) continue;  // the same split as a smaller number's
      if ((int64_t)s.tiles_a * s.tiles_b * s.splits > INT32_MAX / 2) continue;  // counted in 32 bits
      const double turns = (double)ceil_div((int64_t)s.tiles_a * s.tiles_b * s.splits, sms / ts.ctas);
      const double epilogue = s.splits > 1 ? 5.0 * (ts.swap ? rows : ts.b) : whole;
      const double busy = turns * std::max(s.split_blocks * block + 300.0, epilogue);
      const double dram = (double)(m + n) * k * 2.0 / 3500.0;
      // Neither hides the other altogether; a last turn of few CTAs draws less.
      const double idle = 1.0 - (double)s.tiles_a * s.tiles_b * s.splits / (turns * (sms / ts.ctas));
      double cost = std::max(busy, dram * (1.0 + 0.3 * idle)) + 0.25 * std::min(busy, dram) + epilogue;
      s.partial_bytes = s.splits > 1 ? s.splits * (ts.swap ? m : ceil_div(m, 32) * 32) * s.ldp * 4 : 0;
      if (s.splits > 1) cost += 5000.0 + (double)s.partial_bytes / 2300.0;
      if (cost < best_cost) best = s, best_cost = cost;
    }
  }
  return best;
}

// choose_plan, remembering the sizes a thread asked for last (a pure function of
// them; it costs a microsecond or two, and a call and its workspace query ask
// for the same).
Plan pick_plan(int64_t m, int64_t n, int64_t k, bool a_mn, bool vec, int sms) {
  struct Known {
    int64_t m = -1, n = -1, k = -1;
    int sms = 0;
    bool a_mn = false, vec = false;
    Plan plan;
  };
  static thread_local Known known[64];
  const uint64_t mix = ((uint64_t)m * 0x9E3779B97F4A7C15ull ^ (uint64_t)n * 0xC2B2AE3D27D4EB4Full ^
                        (uint64_t)k * 0x165667B19E3779F9ull ^ (uint64_t)(a_mn * 2 + vec)) *
                       0x9E3779B97F4A7C15ull;
  Known& e = known[mix >> 58];
  if (e.m != m || e.n != n || e.k != k || e.sms != sms || e.a_mn != a_mn || e.vec != vec)
    e = Known{m, n, k, sms, a_mn, vec, choose_plan(m, n, k, a_mn, vec, sms)};
  return e.plan;
}

tide_status check_extent(int64_t m, int64_t n, int64_t k) {
  const int64_t most = INT32_MAX - 1024;
  if (m > most || n > most || k > most || ceil_div(m, 128) * ceil_div(n, 128) > most / 16)
    return fail(TIDE_ERR_UNIMPLEMENTED, "linear: sizes beyond 2^31, or too many tiles");
  return TIDE_OK;
}

// Workspace of a product: packed copies of operands that TMA cannot read (or
// that a checkpoint holds), then the splits' partial sums.
int64_t product_workspace(int64_t m, int64_t n, int64_t k, bool a_mn, bool pack_a, int64_t a_rows, int64_t a_cols, bool pack_b,
                          int64_t b_rows, int64_t b_cols) {
  if (m <= 0 || n <= 0 || k <= 0) return 0;
  const int sms = std::max(2, ops_num_sms());
  return (pack_a ? packed_bytes(a_rows, a_cols) : 0) + (pack_b ? packed_bytes(b_rows, b_cols) : 0) +
         std::max(pick_plan(m, n, k, a_mn, false, sms).partial_bytes, pick_plan(m, n, k, a_mn, true, sms).partial_bytes);
}

// Rows of any alignment to rows of packed_ld(cols), for up to two operands.  (What
// lies between a row's end and the next row is not read by the product.)
struct PackArgs {
  const bf16* x;
  bf16* out;
  int64_t rows, cols, ldx, ldo;
  FastDiv per_row;  // warps a row
};
constexpr int kPackItems = 2;  // blocks of 256 elements a warp

// The 16 bytes at `at` (a multiple of 16), but only those inside [first, last).
__device__ __forceinline__ uint4 load_granule(uintptr_t at, uintptr_t first, uintptr_t last) {
  if (at >= first && at + 16 <= last) return *reinterpret_cast<const uint4*>(at);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uintptr_t q = at + 2 * k;
    if (q >= first && q < last) w[k / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(q) << (16 * (k % 2));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes from byte p (even) of the 32 bytes c, n.
__device__ __forceinline__ uint4 shifted(const uint4& c, const uint4& n, uint32_t p) {
  const uint32_t h = p & 2 ? 16 : 0;
  auto f = [&](uint32_t a, uint32_t b, uint32_t d, uint32_t e, uint32_t g) {
    return make_uint4(__funnelshift_r(a, b, h), __funnelshift_r(b, d, h), __funnelshift_r(d, e, h),
                      __funnelshift_r(e, g, h));
  };
  switch (p >> 2) {
    case 0: return f(c.x, c.y, c.z, c.w, n.x);
    case 1: return f(c.y, c.z, c.w, n.x, n.y);
    case 2: return f(c.z, c.w, n.x, n.y, n.z);
    default: return f(c.w, n.x, n.y, n.z, n.w);
  }
}

// A warp takes kPackItems blocks of 256 elements of a row, a lane eight of each:
// it loads the aligned 16 bytes that hold its first element and has the rest
// from the next lane, so that every byte is read once, in whole sectors.  (Five
// narrow loads a lane took 10 us for 25 MB, bound by the L1 cache.)
__device__ __forceinline__ void pack_warp(const PackArgs& a, uint32_t warp) {
  const int64_t row = a.per_row.quotient(warp);
  if (row >= a.rows) return;
  const int lane = threadIdx.x % 32;
  const int64_t e0 = (int64_t)(warp - (uint32_t)row * a.per_row.d) * (256 * kPackItems) + lane * 8;
  const uintptr_t first = (uintptr_t)a.x, last = (uintptr_t)(a.x + (a.rows - 1) * a.ldx + a.cols);
  const uintptr_t from = (uintptr_t)(a.x + row * a.ldx), end = from + a.cols * 2;
  const uint32_t p = (uint32_t)from & 15;  // the same for every lane: they are 16 bytes apart
  uint4 c[kPackItems], n[kPackItems];
#pragma unroll
  for (int j = 0; j < kPackItems; ++j) {
    const uintptr_t at = from + (e0 + 256 * j) * 2 - p;
    c[j] = at < end ? load_granule(at, first, last) : make_uint4(0, 0, 0, 0);
    n[j] = lane == 31 && p && at + 16 < end ? load_granule(at + 16, first, last) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < kPackItems; ++j) {
    const uint4 next = make_uint4(__shfl_down_sync(0xffffffffu, c[j].x, 1), __shfl_down_sync(0xffffffffu, c[j].y, 1),
                                  __shfl_down_sync(0xffffffffu, c[j].z, 1), __shfl_down_sync(0xffffffffu, c[j].w, 1));
    const int64_t e = e0 + 256 * j;
    if (e < a.cols) *reinterpret_cast<uint4*>(a.out + row * a.ldo + e) = shifted(c[j], lane == 31 ? n[j] : next, p);
  }
}

__global__ void __launch_bounds__(256) pack_kernel(const PackArgs a, const PackArgs b, uint32_t blocks_a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x < blocks_a)
    pack_warp(a, blockIdx.x * 8 + threadIdx.x / 32);
  else
    pack_warp(b, (blockIdx.x - blocks_a) * 8 + threadIdx.x / 32);
}

// A launch that may begin before the stream's last kernel, this call's, ends
// (the kernel waits for it before it reads anything).
struct LaunchAfter {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  LaunchAfter(int64_t grid, int threads, bool after, cudaStream_t stream) {
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
  }
};

// Lays out anew, at *at, those of the operands that TMA cannot read.
tide_status pack(Operand* const (&which)[2], unsigned char** at, bool* after, cudaStream_t stream) {
  PackArgs a[2] = {};
  int64_t blocks[2] = {0, 0};
  int count = 0;
  for (Operand* o : which) {
    if (readable(o->p, o->rows, o->ld)) continue;
    const int64_t ld = packed_ld(o->cols), per_row = ceil_div(o->cols, 256 * kPackItems);
    if (o->rows > ((int64_t)1 << 31) / per_row - 8)
      return fail(TIDE_ERR_UNIMPLEMENTED, "linear: operand too large to lay out anew");
    a[count] = {o->p, (bf16*)*at, o->rows, o->cols, o->ld, ld, FastDiv((uint32_t)per_row)};
    blocks[count++] = ceil_div(o->rows * per_row, 8);
    o->p = (const bf16*)*at;
    o->ld = ld;
    *at += packed_bytes(o->rows, o->cols);
  }
  if (count == 0) return TIDE_OK;
  const LaunchAfter l(blocks[0] + blocks[1], 256, *after, stream);
  *after = true;
  return cuda_status(cudaLaunchKernelEx(&l.cfg, pack_kernel, a[0], a[1], (uint32_t)blocks[0]), "laying out operands");
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeTiled)p;
  }();
  return fn;
}

// A 2-D map with 128-byte swizzle; elements outside the matrix read as zero.
tide_status make_map(CUtensorMap* map, const Operand& o, int box_rows) {
  const EncodeTiled encode = encode_tiled();
  if (!encode) return fail(TIDE_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[2] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(o.rows > 1 ? o.ld : packed_ld(o.cols)) * 2};
  const cuuint32_t box[2] = {kTcK, (cuuint32_t)box_rows}, steps[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<bf16*>(o.p), dims, strides, box, steps,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? TIDE_OK : fail(TIDE_ERR_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
}

using Launch = cudaError_t (*)(const TcArgs&, TcTile, int, bool, cudaStream_t);

// out [m, n] = epilogue(sum over k); a_mn / b_mn: the operand's rows run along
// k (its contiguous axis is m or n).  `after`: the stream's last kernel is this
// call's; `beside`, if not null, is called once the operands are laid out, to
// launch a kernel that the product may overlap.
struct Nothing {
  tide_status operator()() const { return TIDE_OK; }
};
template <int EPI, typename Beside = Nothing>
tide_status product(int64_t m, int64_t n, int64_t k, Operand a, bool a_mn, Operand b, bool b_mn, EpilogueArgs e,
                    Launch launch, unsigned char* workspace, bool after, cudaStream_t stream,
                    const Beside* beside = nullptr) {
  const int sms = ops_num_sms();
  if (sms <= 0) return fail(TIDE_ERR_CUDA, "the current device could not be queried");
  uint32_t* timeouts = nullptr;
  TIDE_TRY(ops_timeouts(&timeouts));
  TIDE_TRY(check_extent(m, n, k));
  e.rows = m, e.cols = n;
  int splits = 0;
  bool swapped = true;
  if (k > 0) {
    const Plan s = pick_plan(m, n, k, a_mn, e.unit == 16, sms);
    const TcTileShape ts = tile_shape(s.tile, a_mn);
    Operand* const both[2] = {&a, &b};
    TIDE_TRY(pack(both, &workspace, &after, stream));
    if (ts.swap) std::swap(a, b), std::swap(a_mn, b_mn);
    TcArgs p{};
    if (beside) {
      TIDE_TRY((*beside)());
      p.beside = after = true;
    }
    TIDE_TRY(make_map(&p.a, a, a_mn ? kTcK : 128));
    TIDE_TRY(make_map(&p.b, b, b_mn ? kTcK : ts.b / ts.ctas));
    if (s.splits > 1) e.partial = (float*)workspace, e.ldp = s.ldp;
    p.e = e;
    p.tiles_a = s.tiles_a, p.tiles_b = s.tiles_b;
    p.k_blocks = s.k_blocks, p.split_blocks = s.split_blocks, p.splits = s.splits;
    p.timeouts = timeouts;
    p.wait_limit_ns = ops_wait_limit_ns();
    p.test_drop = ops_test_drop();
    const int64_t units = (int64_t)s.tiles_a * s.tiles_b * s.splits;
    const int grid = (int)std::min<int64_t>(units * ts.ctas, sms / ts.ctas * ts.ctas);
    TIDE_TRY(cuda_status(launch(p, s.tile, grid, after, stream), "linear product"));
    if (s.splits == 1) return TIDE_OK;
    splits = s.splits;
    swapped = ts.swap;
    after = true;
  }
  const int64_t warps = (swapped ? m : ceil_div(m, 32)) * ceil_div(n, 32), grid = ceil_div(warps * 32, kJoinThreads);
  if (grid > INT32_MAX) return fail(TIDE_ERR_UNIMPLEMENTED, "linear: too many elements for one launch");
  const LaunchAfter l(grid, kJoinThreads, after, stream);
  return cuda_status(with_act(EPI == EPI_PLAIN ? TIDE_ACT_NONE : e.act,
                              [&](auto act) {
                                constexpr int kAct = EPI == EPI_PLAIN ? TIDE_ACT_NONE : act.value;
                                return swapped ? cudaLaunchKernelEx(&l.cfg, join_kernel<EPI, kAct, true>, e, splits)
                                               : cudaLaunchKernelEx(&l.cfg, join_kernel<EPI, kAct, false>, e, splits);
                              }),
                     "linear epilogue");
}

// db: column sums.  A thread sums V neighbouring columns over every other one
// of its block's rows, and the block's two are joined in shared memory; block
// row y gives partial[y], summed by launch_sum_groups.  It runs beside the
// product, which it lets start as soon as its blocks are all there: they are few, and a
// pair tile's CTA leaves 17 KB of shared memory for their 4.  The swapped tiles of 64
// and 128 tokens leave half a KB: such a CTA starts once the sums on its SM are done.
constexpr int kSumLanes = 64;

template <int V>
__global__ void __launch_bounds__(2 * kSumLanes) column_sum_kernel(int64_t rows, int64_t cols,
                                                                   const bf16* __restrict__ x, int64_t ldx,
                                                                   int64_t rows_per_block,
                                                                   float* __restrict__ partial) {
  __shared__ float s[2][kSumLanes * V];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x % kSumLanes, part = threadIdx.x / kSumLanes;
  const int64_t col = ((int64_t)blockIdx.x * kSumLanes + lane) * V;
  const int64_t r0 = blockIdx.y * rows_per_block, r1 = min(rows, r0 + rows_per_block);
  float v[V] = {};
  if (col < cols) {
    int64_t r = r0 + part;
    constexpr int kAhead = V == 8 ? 8 : 16;
    for (; r + 2 * (kAhead - 1) < r1; r += 2 * kAhead) {
      float t[kAhead][V];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) load_vec<V>(x + (r + 2 * j) * ldx + col, t[j]);
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] += t[j][k];
    }
    for (; r < r1; r += 2) {
      float t[V];
      load_vec<V>(x + r * ldx + col, t);
#pragma unroll
      for (int k = 0; k < V; ++k) v[k] += t[k];
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) s[part][lane * V + k] = v[k];
  __syncthreads();
  for (int i = threadIdx.x; i < kSumLanes * V; i += 2 * kSumLanes) {
    const int64_t c = (int64_t)blockIdx.x * kSumLanes * V + i;
    if (c < cols) partial[blockIdx.y * cols + c] = s[0][i] + s[1][i];
  }
}

// Columns a thread sums, and the row groups of the partial sums: two blocks an
// SM in all, groups of at least 32 rows.
int sum_vector(int64_t rows, int64_t cols, const void* x, int64_t ldx) {
  return cols % 8 == 0 && rows_aligned(x, ldx, 2, rows) ? 8 : 1;
}
int64_t sum_groups(int64_t rows, int64_t cols, int v, int sms) {
  const int64_t across = ceil_div(cols, kSumLanes * v);
  const int64_t groups = std::max<int64_t>(1, std::min(ceil_div(rows, 32), ceil_div(2 * sms, across)));
  return ceil_div(rows, ceil_div(rows, groups));  // groups that have rows
}

int64_t sum_bytes(int64_t rows, int64_t cols, int v, int sms) {
  return ceil_div(sum_groups(rows, cols, v, sms) * cols * 4, 256) * 256;
}

tide_status column_sums(int64_t rows, int64_t cols, const bf16* x, int64_t ldx, int v, int64_t groups, float* partial,
                        cudaStream_t stream) {
  const dim3 grid((unsigned)ceil_div(cols, kSumLanes * v), (unsigned)groups);
  const int64_t per = ceil_div(rows, groups);
  if (v == 8)
    column_sum_kernel<8><<<grid, 2 * kSumLanes, 0, stream>>>(rows, cols, x, ldx, per, partial);
  else
    column_sum_kernel<1><<<grid, 2 * kSumLanes, 0, stream>>>(rows, cols, x, ldx, per, partial);
  return cuda_status(cudaGetLastError(), "bias gradient");
}

// EpilogueArgs::unit of bf16 matrices (base, row stride; absent ones null), and
// code_unit of a checkpoint's codes.
struct Rows {
  const void* p;
  int64_t ld;
};
int32_t row_unit(std::initializer_list<Rows> matrices, int64_t rows) {
  uintptr_t bits = 0;
  for (const Rows& x : matrices)
    if (x.p) bits |= (uintptr_t)x.p | (rows > 1 ? (uintptr_t)x.ld * 2 : 0);
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}
int32_t code_unit(const uint8_t* codes, int64_t ld, int64_t rows) {
  const uintptr_t bits = (uintptr_t)codes | (rows > 1 ? (uintptr_t)ld : 0);
  return bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 1;
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

}  // namespace

tide_status ops_timeouts(uint32_t** word) {
  static std::atomic<uint32_t*> known[64];
  int dev = -1;
  TIDE_TRY(cuda_status(cudaGetDevice(&dev), "cudaGetDevice"));
  if (dev < 64 && (*word = known[dev].load(std::memory_order_relaxed))) return TIDE_OK;
  void* p = nullptr;
  TIDE_TRY(cuda_status(cudaGetSymbolAddress(&p, g_timeouts), "cudaGetSymbolAddress"));
  *word = (uint32_t*)p;
  if (dev < 64) known[dev].store(*word, std::memory_order_relaxed);
  return TIDE_OK;
}

uint64_t ops_wait_limit_ns() { return (uint64_t)g_wait_limit_ns.load(std::memory_order_relaxed); }
int64_t ops_test_drop() { return g_test_drop; }

}  // namespace tide

using namespace tide;

extern "C" {

int64_t tide_linear_workspace(int64_t rows, int64_t inner, int64_t outer, const void* x, int64_t ldx, const void* w,
                              int64_t ldw) {
  return product_workspace(rows, outer, inner, false, !readable(x, rows, ldx), rows, inner, !readable(w, outer, ldw), outer,
                           inner);
}

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
  EpilogueArgs e{};
  e.act = act;
  e.bias = (const bf16*)bias;
  e.residual = (const bf16*)residual, e.ldr = ldr;
  e.out = (bf16*)y, e.ldo = ldy;
  e.z = (bf16*)z, e.ldz = ldz;
  e.codes = codes, e.ldc = ld_codes, e.scales = scales, e.lds = ld_scales;
  e.unit = row_unit({{residual, ldr}, {y, ldy}, {z, ldz}}, rows);
  e.code_unit = code_unit(codes, ld_codes, rows);
  return product<EPI_FORWARD>(rows, outer, inner, {(const bf16*)x, rows, inner, ldx}, false,
                              {(const bf16*)w, outer, inner, ldw}, false, e, launch_forward, (unsigned char*)workspace, false,
                              (cudaStream_t)stream);
}

int64_t tide_linear_grad_input_workspace(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                         const void* w, int64_t ldw) {
  return product_workspace(rows, inner, outer, false, !readable(dy, rows, lddy), rows, outer, !readable(w, outer, ldw), outer,
                           inner);
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
  EpilogueArgs e{};
  e.act = act;
  e.zin = (const bf16*)z, e.ldzin = ldz;
  e.cin = codes, e.ldcin = ld_codes, e.sin = scales, e.ldsin = ld_scales;
  e.out = (bf16*)dx, e.ldo = lddx;
  e.unit = row_unit({{dx, lddx}, {act == TIDE_ACT_NONE ? nullptr : z, ldz}}, rows);
  e.code_unit = code_unit(codes, ld_codes, rows);
  return product<EPI_GRAD_INPUT>(rows, inner, outer, {(const bf16*)dy, rows, outer, lddy}, false,
                                 {(const bf16*)w, outer, inner, ldw}, true, e, launch_grad_input,
                                 (unsigned char*)workspace, false, (cudaStream_t)stream);
}

int64_t tide_linear_grad_weight_workspace(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                          const void* x, int64_t ldx, int32_t with_db) {
  const int sms = std::max(2, ops_num_sms());
  if (rows <= 0 || outer <= 0) return 0;
  // The bias gradient's partial sums, then the product's.
  return (with_db ? sum_bytes(rows, outer, sum_vector(rows, outer, dy, lddy), sms) : 0) +
         product_workspace(outer, inner, rows, true, !readable(dy, rows, lddy), rows, outer,
                           !x || !readable(x, rows, ldx), rows, inner);
}

tide_status tide_linear_grad_weight(int64_t rows, int64_t inner, int64_t outer, const void* dy, int64_t lddy,
                                    const void* x, int64_t ldx, const uint8_t* codes, int64_t ld_codes,
                                    const uint8_t* scales, int64_t ld_scales, int32_t act, void* dw, int64_t lddw,
                                    void* db, void* workspace, int64_t workspace_bytes, void* stream_) {
  clear_error();
  const cudaStream_t stream = (cudaStream_t)stream_;
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
                           tide_linear_grad_weight_workspace(rows, inner, outer, dy, lddy, x, ldx, db != nullptr)));
  const int sms = std::max(2, ops_num_sms());
  const int v = sum_vector(rows, outer, dy, lddy);
  const int64_t groups = db && rows > 0 ? sum_groups(rows, outer, v, sms) : 0;
  float* partial = (float*)workspace;
  const auto sums = [&] {
    return column_sums(rows, outer, (const bf16*)dy, lddy, v, groups, partial, stream);
  };
  bool summed = false;
  if (inner > 0) {
    unsigned char* at = (unsigned char*)workspace + (groups > 0 ? sum_bytes(rows, outer, v, sms) : 0);
    Operand b{(const bf16*)x, rows, inner, ldx};
    if (!x && rows > 0) {
      TIDE_TRY(launch_checkpoint_load_bf16(rows, inner, codes, ld_codes, scales, ld_scales, act, at, packed_ld(inner),
                                           stream));
      b.p = (const bf16*)at, b.ld = packed_ld(inner);
      at += packed_bytes(rows, inner);
    }
    EpilogueArgs e{};
    e.out = (bf16*)dw, e.ldo = lddw;
    e.unit = row_unit({{dw, lddw}}, outer);
    summed = groups > 0;
    TIDE_TRY(product<EPI_PLAIN>(outer, inner, rows, {(const bf16*)dy, rows, outer, lddy}, true, b, true, e,
                                launch_grad_weight, at, !x && rows > 0, stream, summed ? &sums : nullptr));
  }
  if (!db) return TIDE_OK;
  if (groups > 0 && !summed) TIDE_TRY(sums());
  return launch_sum_groups(partial, groups, outer, TIDE_BF16, db, groups > 0, stream);
}

tide_status tide_ops_check(void) {
  clear_error();
  static thread_local uint32_t seen[64];
  int dev = 0;
  uint32_t* word = nullptr;
  TIDE_TRY(ops_timeouts(&word));
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceSynchronize();
  uint32_t count = 0;
  if (err == cudaSuccess) err = cudaMemcpy(&count, word, sizeof count, cudaMemcpyDeviceToHost);
  TIDE_TRY(cuda_status(err, "reading the operators' count of timeouts"));
  uint32_t& last = seen[std::min(dev, 63)];
  if (count == last) return TIDE_OK;
  last = count;
  return fail(TIDE_ERR_TIMEOUT, "an operator's kernel gave up a bounded wait; its outputs are undefined");
}

tide_status tide_ops_set_option(int32_t option, int64_t value) {
  clear_error();
  switch (option) {
    case TIDE_OPS_OPT_WAIT_LIMIT_NS:
      if (value <= 0) return fail(TIDE_ERR_INVALID_ARG, "the wait limit must be positive");
      g_wait_limit_ns.store(value);
      return TIDE_OK;
    case TIDE_OPS_OPT_TEST_DROP_LOAD:
      if (value < -1) return fail(TIDE_ERR_INVALID_ARG, "the load to withhold must be -1 or more");
      g_test_drop = value;
      return TIDE_OK;
    default: return fail(TIDE_ERR_INVALID_ARG, "unknown option");
  }
}

}  // extern "C"
