// Tensor-core products of the linear layer, out = epilogue(A B^T).
//
// A and B are bf16, each either with k contiguous (K-major) or with its other
// axis contiguous (MN-major); sums are fp32 in tensor memory.  A tile is 128 *
// CG rows of A by BN rows of B; with CG = 2 two CTAs of a cluster share it, each
// holding 128 rows of A, half of B's rows and its 128 rows of the accumulator,
// so that every byte staged in shared memory feeds twice the arithmetic.
// Normally A's rows are the output's rows.  With SWAP they are its columns (A is
// then the weight): for outputs of few rows, whose tiles would be mostly empty,
// 128 weight rows fill a tile however few tokens there are.
//
// One persistent CTA per SM.  Warp 0 streams 64-deep blocks of A and B into a
// ring of shared-memory stages with TMA; warp 1 (of the first CTA of a pair)
// issues the matrix instructions; warps 4-11 take a finished accumulator out of
// tensor memory and run the epilogue while the next tile accumulates in the
// other half.  Every wait is bounded: a wait that runs out is
// counted, and the CTA drains its copies, frees its tensor memory and returns.
//
// What binds it, measured:
//   8192 x 5120 x 13824 with bias, GELU and an 8-bit z: 600 to 611 us from a cold
//   start, by the GPU (1.9 PFLOP/s, tensor pipe 97% active), 700 us (1.66) in a long
//   loop, where the power limit holds the clock near 1450 MHz; the input gradient 598
//   to 614 and 697 us, 8192 x 28672 x 8192's weight gradient 1.8 to 1.9 and 2.2 ms
//   one token, 8192 -> 28672: 73 us, 6.4 TB/s of weights (DRAM)
//   short sums, by their output: 24832 x 64 -> 10304 in 103 us, 5.0 TB/s (plain, a
//   weight gradient's, 98 us, 5.2); rows of odd alignment 2.2 to 3.6 TB/s
//   a block of 64 of the sum takes a pair 512 clocks on 256 x 256 and 260 on 256 x
//   128 alone, 570 and 340 with all SMs drawing on L2; a single CTA 270 to 420
#pragma once

#include <atomic>

#include "ops_common.cuh"
#include "tc_ptx.cuh"

namespace tide {

enum Epilogue { EPI_FORWARD, EPI_GRAD_INPUT, EPI_PLAIN, EPI_PARTIAL };

// What becomes of a sum v at (row, col):
//   FORWARD      v += bias; z, and its checkpoint, get v; out = f(v) + residual
//   GRAD_INPUT   out = v * f'(kept z), or v with no activation
//   PLAIN        out = v
//   PARTIAL      v in fp32 to partial[split], for join_kernel
struct EpilogueArgs {
  int64_t rows, cols;
  int32_t act;
  // Bytes that every bf16 matrix's (16, 4 or 2) and checkpoint's (8, 4 or 1) rows
  // are aligned to; cols may be odd all the same.
  int32_t unit, code_unit;
  const bf16* bias;
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
  // Sums of the splits: with swapped operands [splits][rows][ldp]; otherwise in
  // blocks of 32 x 32, [splits][blocks of rows][ldp / 32][8][32 rows][4], so that
  // a warp that holds a row a lane writes and reads 512 bytes at a time.
  float* partial;
  int64_t ldp;
};

struct TcArgs {
  CUtensorMap a, b;
  EpilogueArgs e;
  int32_t tiles_a, tiles_b;  // tiles along A's and B's rows
  int32_t k_blocks;        // of 64, over the whole sum
  int32_t split_blocks;    // k blocks of one split (all of them without splitting)
  int32_t splits;
  uint32_t* timeouts;
  uint64_t wait_limit_ns;
  bool beside;             // runs beside the kernel before it, whose results it does not read
  int64_t test_drop;       // k block (counted per CTA) whose loads are withheld (tests); -1: none
};

constexpr int kTcThreads = 384;    // warps 0 to 3 as above, and eight for the epilogue
constexpr int kTcK = 64;           // values of k a stage holds: 128 bytes, one swizzle row
constexpr int kTcGroup = 8;        // tile rows walked together, for reuse of B in L2
constexpr int kTcRoom = 227 * 1024;  // shared memory a CTA may take

// A 32 x 32 block per epilogue warp: bf16 to pass through, or, swapped, fp32 to be
// turned (rows of 33).
template <bool SWAP>
constexpr int kBlockBytes = SWAP ? 32 * 33 * 4 : 32 * 64;

template <int CG, int BN, int EPI, bool SWAP>
struct TcShape {
  static constexpr int a_bytes = 128 * kTcK * 2;
  static constexpr int b_rows = BN / CG;
  static constexpr int b_bytes = b_rows * kTcK * 2;
  static constexpr int stage_bytes = a_bytes + b_bytes;
  static constexpr int transpose_bytes = 8 * kBlockBytes<SWAP>;
  static constexpr int columns = 2 * BN;                   // two accumulators
  static constexpr int fixed_bytes = 1024 + transpose_bytes + 512;
  static constexpr int stages = (kTcRoom - fixed_bytes) / stage_bytes < 12 ? (kTcRoom - fixed_bytes) / stage_bytes : 12;
  static constexpr int smem_bytes = fixed_bytes + stages * stage_bytes;
};

// ---- epilogues

// A warp moves 32 x 32 blocks of a matrix through shared memory (its `block`), so
// that a lane can hold a whole row of the block while global memory sees
// neighbouring lanes on neighbouring words: W bytes a lane, the ROW bytes of a
// block's row by ROW / W lanes.  (A lane storing its own row touches 32 lines an
// instruction: 2235 x 2632 with a sum of 64 took 50 us that way, 19 this way.)  The
// staged rows' 16-byte words are permuted so that both sides are free of bank
// conflicts.  Only the first `rows` rows and `bytes` bytes of each exist.
template <int ROW>
__device__ __forceinline__ int staged(int r, int b) {
  return r * ROW + (b ^ ((r * ROW / 128 % (ROW / 16)) << 4));
}
template <int W>
struct UnitOf;
template <> struct UnitOf<16> { using type = uint4; };
template <> struct UnitOf<8> { using type = uint2; };
template <> struct UnitOf<4> { using type = uint32_t; };
template <> struct UnitOf<2> { using type = uint16_t; };
template <> struct UnitOf<1> { using type = uint8_t; };

template <int ROW, int W>
__device__ __forceinline__ void load_units(const unsigned char* p, int64_t ld, int lane, int rows, int bytes,
                                           unsigned char* block) {
  using Unit = typename UnitOf<W>::type;
  constexpr int kLanes = ROW / W, kBatch = kLanes < 16 ? kLanes : 16;
  const int b = lane % kLanes * W;
#pragma unroll
  for (int j = 0; j < kLanes; j += kBatch) {
    Unit u[kBatch];  // all on their way before the first is waited for
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = (j + i) * (32 / kLanes) + lane / kLanes;
      u[i] = b < bytes && r < rows ? *reinterpret_cast<const Unit*>(p + r * ld + b) : Unit{};
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      *reinterpret_cast<Unit*>(block + staged<ROW>((j + i) * (32 / kLanes) + lane / kLanes, b)) = u[i];
  }
  __syncwarp();
}

template <int ROW, int W>
__device__ __forceinline__ void store_units(unsigned char* p, int64_t ld, int lane, int rows, int bytes,
                                            const unsigned char* block) {
  using Unit = typename UnitOf<W>::type;
  constexpr int kLanes = ROW / W;
  const int b = lane % kLanes * W;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kLanes; ++i) {
    const int r = i * (32 / kLanes) + lane / kLanes;
    const Unit u = *reinterpret_cast<const Unit*>(block + staged<ROW>(r, b));
    if (b < bytes && r < rows) *reinterpret_cast<Unit*>(p + r * ld + b) = u;
  }
  __syncwarp();
}

// A 32 x 32 block of a bf16 matrix whose rows take units of `unit` bytes, `cols` of
// its columns existing; lane l has row l.
__device__ __forceinline__ void load_tile(const bf16* p, int64_t ld, int unit, int lane, int rows, int cols,
                                          unsigned char* block, float (&v)[32]) {
  const unsigned char* x = reinterpret_cast<const unsigned char*>(p);
  if (unit == 16)
    load_units<64, 16>(x, ld * 2, lane, rows, 64, block);
  else if (unit == 4)
    load_units<64, 4>(x, ld * 2, lane, rows, 64, block);
  else
    load_units<64, 2>(x, ld * 2, lane, rows, cols * 2, block);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t[8];
    load_vec<8>(reinterpret_cast<const bf16*>(block + staged<64>(lane, 16 * i)), t);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[8 * i + k] = t[k];
  }
  __syncwarp();
}

__device__ __forceinline__ void store_tile(bf16* p, int64_t ld, int unit, int lane, int rows, int cols,
                                           unsigned char* block, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = v[8 * i + k];
    store_vec<8>(reinterpret_cast<bf16*>(block + staged<64>(lane, 16 * i)), t);
  }
  unsigned char* x = reinterpret_cast<unsigned char*>(p);
  if (unit == 16)
    store_units<64, 16>(x, ld * 2, lane, rows, 64, block);
  else if (unit == 4)
    store_units<64, 4>(x, ld * 2, lane, rows, 64, block);
  else
    store_units<64, 2>(x, ld * 2, lane, rows, cols * 2, block);
}

// The same for codes.
__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t ld, int unit, int lane, int rows, int cols,
                                           unsigned char* block, uint32_t (&w)[8]) {
  if (unit == 8)
    load_units<32, 8>(p, ld, lane, rows, 32, block);
  else if (unit == 4)
    load_units<32, 4>(p, ld, lane, rows, 32, block);
  else
    load_units<32, 1>(p, ld, lane, rows, cols, block);
  const uint4 a = *reinterpret_cast<const uint4*>(block + staged<32>(lane, 0));
  const uint4 b = *reinterpret_cast<const uint4*>(block + staged<32>(lane, 16));
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  __syncwarp();
}

__device__ __forceinline__ void store_codes(uint8_t* p, int64_t ld, int unit, int lane, int rows, int cols,
                                            unsigned char* block, const uint32_t (&w)[8]) {
  *reinterpret_cast<uint4*>(block + staged<32>(lane, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(block + staged<32>(lane, 16)) = make_uint4(w[4], w[5], w[6], w[7]);
  if (unit == 8)
    store_units<32, 8>(p, ld, lane, rows, 32, block);
  else if (unit == 4)
    store_units<32, 4>(p, ld, lane, rows, 32, block);
  else
    store_units<32, 1>(p, ld, lane, rows, cols, block);
}

// The 32 x 32 block of the output at (row, col), lane l holding its l-th row, a
// whole warp; any alignment.
template <int EPI, int ACT>
__device__ __forceinline__ void epilogue_tile(const EpilogueArgs& e, int64_t row, int64_t col, int lane,
                                              unsigned char* block, float (&v)[32]) {
  const int rows = (int)min((int64_t)32, e.rows - row), cols = (int)min((int64_t)32, e.cols - col);
  const int unit = cols == 32 ? e.unit : 2, code_unit = cols == 32 ? e.code_unit : 1;
  float t[32];
  if constexpr (EPI == EPI_FORWARD) {
    if (e.bias) {
      const float mine = lane < cols ? __bfloat162float(e.bias[col + lane]) : 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, mine, i);
    }
    if (e.z) store_tile(e.z + row * e.ldz + col, e.ldz, unit, lane, rows, cols, block, v);
    if (e.codes) {
      // Columns that do not exist are sums of zeros (or NaN, of a row with an
      // infinity): neither counts for the scale.
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = v[i];
      const int byte = scale_byte(block_magnitude<1>(t));
      uint32_t w[8];
      encode(t, byte, w);
      store_codes(e.codes + row * e.ldc + col, e.ldc, code_unit, lane, rows, cols, block, w);
      if (lane < rows) e.scales[(row + lane) * e.lds + col / kMxBlock] = (uint8_t)byte;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_value<true>(ACT, v[i]);
    if (e.residual) {
      load_tile(e.residual + row * e.ldr + col, e.ldr, unit, lane, rows, cols, block, t);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += t[i];
    }
  }
  if constexpr (EPI == EPI_GRAD_INPUT && ACT != TIDE_ACT_NONE) {
    if (e.zin) {
      load_tile(e.zin + row * e.ldzin + col, e.ldzin, unit, lane, rows, cols, block, t);
    } else {
      uint32_t w[8];
      load_codes(e.cin + row * e.ldcin + col, e.ldcin, code_unit, lane, rows, cols, block, w);
      const float s = scale_value(e.sin[(row + min(lane, rows - 1)) * e.ldsin + col / kMxBlock]);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 q = e4m3_values((w[i / 2] >> (16 * (i % 2))) & 0xffffu);
        t[2 * i] = q.x * s;
        t[2 * i + 1] = q.y * s;
      }
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= act_grad<true>(ACT, t[i]);
  }
  store_tile(e.out + row * e.ldo + col, e.ldo, unit, lane, rows, cols, block, v);
}

// Where lane `lane`'s row of the 32 x 32 block at (row, col) keeps its partial
// sums: columns 4 q to 4 q + 3 are the float4 at 32 q.
__device__ __forceinline__ float4* partial_block(const EpilogueArgs& e, int split, int64_t row, int64_t col, int lane) {
  const int64_t block = (split * ((e.rows + 31) / 32) + row / 32) * (e.ldp / 32) + col / 32;
  return reinterpret_cast<float4*>(e.partial) + block * 256 + lane;
}

// N rows from `row` (the first n of them exist), a whole warp on one block of 32
// columns of each, an element a lane; any alignment.  `in`: the column exists.
// The rows' steps are independent, and what they load is loaded whether or not it
// exists (from the nearest place that does): behind a branch each load would be
// waited for by itself.
template <int EPI, int ACT, int N>
__device__ __forceinline__ void epilogue_columns(const EpilogueArgs& e, int64_t row, int n, int64_t col, bool in,
                                                 float (&v)[N], float bias) {
  const int64_t c = in ? col : e.cols - 1;  // where to load from
  if constexpr (EPI == EPI_FORWARD) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += bias;
    if (e.z) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (in && i < n) e.z[(row + i) * e.ldz + col] = __float2bfloat16_rn(v[i]);
    }
    if (e.codes) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float t = finite_or_nan(v[i]);
        const uint32_t m = __reduce_max_sync(0xffffffffu, in ? __float_as_uint(fmaxf(fabsf(t), 0.0f)) : 0u);
        const int byte = scale_byte(__uint_as_float(m));
        if (in && i < n) {
          e.codes[(row + i) * e.ldc + col] = encode_one(t, byte);
          if (col % kMxBlock == 0) e.scales[(row + i) * e.lds + col / kMxBlock] = (uint8_t)byte;
        }
      }
    }
    float r[N] = {};
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = __bfloat162float(e.residual[(row + min(i, n - 1)) * e.ldr + c]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value<true>(ACT, v[i]);
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += r[i];
    }
  }
  if constexpr (EPI == EPI_GRAD_INPUT && ACT != TIDE_ACT_NONE) {
    float z[N] = {};
    if (e.zin) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = __bfloat162float(e.zin[(row + min(i, n - 1)) * e.ldzin + c]);
    } else {
      uint8_t code[N], scale[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        code[i] = e.cin[(row + min(i, n - 1)) * e.ldcin + c];
        scale[i] = e.sin[(row + min(i, n - 1)) * e.ldsin + c / kMxBlock];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = e4m3_values(code[i]).x * scale_value(scale[i]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= act_grad<true>(ACT, z[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (in && i < n) e.out[(row + i) * e.ldo + col] = __float2bfloat16_rn(v[i]);
}

// Brings into L2 what the epilogue of a lane's row (n columns from col) will
// read.
template <int EPI, int ACT>
__device__ __forceinline__ void prefetch_row(const EpilogueArgs& e, int64_t row, int64_t col, int n) {
  if (row >= e.rows) return;
  auto lines = [&](const void* from, int64_t bytes) {
    for (int64_t b = 0; b < bytes; b += 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"((const unsigned char*)from + b));
  };
  const int64_t m = min((int64_t)n, e.cols - col);
  if (EPI == EPI_FORWARD && e.residual) lines(e.residual + row * e.ldr + col, m * 2);
  if (EPI == EPI_GRAD_INPUT && ACT != TIDE_ACT_NONE) {
    if (e.zin)
      lines(e.zin + row * e.ldzin + col, m * 2);
    else
      lines(e.cin + row * e.ldcin + col, m);
  }
}

// ---- the kernel

struct TileAt {
  int a, b;
};
// Tiles in groups of kTcGroup along A, down A's rows first: CTAs at work at
// one time share few rows of A and B.
__device__ __forceinline__ TileAt tile_at(const TcArgs& p, int t) {
  const int per_group = kTcGroup * p.tiles_b;
  const int g = t / per_group, first = g * kTcGroup;
  const int height = min(kTcGroup, p.tiles_a - first);
  const int i = t - g * per_group;
  return {first + i % height, i / height};
}

template <int CG, int BN, bool A_MN, bool B_MN, int EPI, int ACT, bool SWAP>
__global__ void __launch_bounds__(kTcThreads, 1) gemm_tc_kernel(const __grid_constant__ TcArgs p) {
  using Shape = TcShape<CG, BN, EPI, SWAP>;
  constexpr int kStages = Shape::stages;
  static_assert((2 * kStages + 5) * 8 + 4 <= 512, "barriers");
  extern __shared__ unsigned char raw[];
  // 1024-byte aligned: the swizzle pattern follows address bits.
  unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  unsigned char* transpose = smem + kStages * Shape::stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(transpose + Shape::transpose_bytes);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drained = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 8 * CG);
    }
    mbar_init(drained, 1);
    fence_mbar_init_cluster();
    tma_prefetch_map(&p.a);
    tma_prefetch_map(&p.b);
  }
  if (warp == 2) tmem_alloc<CG>(tmem_slot, Shape::columns);
  tc_fence_before();
  if constexpr (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Only now is anything read that an earlier kernel of the call wrote; what
  // follows may be launched while this runs (it waits likewise).
  if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int tiles = p.tiles_a * p.tiles_b;
  const int units = tiles * p.splits;
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  bool ok = true;

  if (warp == 0) {
    // Producer.  The pair's loads all count on the first CTA's barrier.
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    const uint32_t full0 = CG == 2 ? mapped_addr(smem_addr(full), 0) : smem_addr(full);
    for (int u = first; u < units && ok; u += step) {
      const TileAt at = tile_at(p, u % tiles);
      const int split = u / tiles;
      const int kb0 = split * p.split_blocks, kb1 = min(p.k_blocks, kb0 + p.split_blocks);
      const int a0 = (at.a * CG + (int)rank) * 128, b0 = at.b * BN + (int)rank * Shape::b_rows;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = warp_wait_bounded(empty + stage, phase ^ 1, p.wait_limit_ns))) break;
        unsigned char* a = smem + stage * Shape::stage_bytes;
        unsigned char* b = a + Shape::a_bytes;
        const uint32_t bar = full0 + stage * 8;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full + stage, CG * Shape::stage_bytes);
          if (issued != p.test_drop) {
            if constexpr (A_MN) {
              tma_load_2d<CG>(a, &p.a, a0, kb * kTcK, bar);
              tma_load_2d<CG>(a + 8192, &p.a, a0 + 64, kb * kTcK, bar);
            } else {
              tma_load_2d<CG>(a, &p.a, kb * kTcK, a0, bar);
            }
            if constexpr (B_MN) {
#pragma unroll
              for (int i = 0; i < Shape::b_rows / 64; ++i)
                tma_load_2d<CG>(b + 8192 * i, &p.b, b0 + 64 * i, kb * kTcK, bar);
            } else {
              tma_load_2d<CG>(b, &p.b, kb * kTcK, b0, bar);
            }
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
    // Before leaving, every stage is handed back (no commit's arrival is still
    // under way), or, after a wait that ran out, the loads in flight landed.
    for (int s = 0; s < kStages; ++s) {
      const int64_t uses = (issued - s + kStages - 1) / kStages;  // times stage s was filled
      if (uses <= 0) break;
      if (ok) ok = warp_wait_bounded(empty + s, (uint32_t)(uses - 1) & 1, p.wait_limit_ns);
      if (!ok && rank == 0) warp_wait_bounded(full + s, (uint32_t)(uses - 1) & 1, p.wait_limit_ns);
    }
    if (!ok) {  // the pair's other CTA counts on barriers it cannot ask: a millisecond is ample for a load
      const uint64_t t = global_ns();
      while (global_ns() - t < 1000000) __nanosleep(1000);
    }
  } else if (warp == 1 && rank == 0) {
    // Matrix instructions, for both CTAs of a pair.
    constexpr uint32_t idesc = instruction_desc(128 * CG, BN, A_MN, B_MN);
    const uint64_t desc_a0 = operand_desc<A_MN>(smem_addr(smem));
    const uint64_t desc_b0 = operand_desc<B_MN>(smem_addr(smem) + Shape::a_bytes);
    int stage = 0;
    uint32_t phase = 0;
    int turn = 0;
    for (int u = first; u < units && ok; u += step, ++turn) {
      const int split = u / tiles;
      const int kb0 = split * p.split_blocks, kb1 = min(p.k_blocks, kb0 + p.split_blocks);
      const int acc = turn & 1;
      if (!(ok = warp_wait_bounded(acc_empty + acc, ((turn >> 1) & 1) ^ 1, p.wait_limit_ns))) break;
      tc_fence_after();
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = warp_wait_bounded(full + stage, phase, p.wait_limit_ns))) break;
        tc_fence_after();
        const uint64_t da = desc_a0 + stage * (Shape::stage_bytes >> 4), db = desc_b0 + stage * (Shape::stage_bytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTcK / 16; ++k)
            tc_mma<CG>(tmem + acc * BN, da + k * kDescStep<A_MN>, db + k * kDescStep<B_MN>, idesc, kb > kb0 || k > 0);
          tc_commit<CG>(empty + stage);
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
      if (ok && elect_one()) tc_commit<CG>(acc_full + acc);
      __syncwarp();
    }
    if (!ok) {
      if (elect_one()) tc_commit<CG>(drained);
      __syncwarp();
      warp_wait_bounded(drained, 0, p.wait_limit_ns);
    }
  } else if (warp >= 4) {
    // Epilogue: warp w reads lanes 32 (w mod 4) onwards, one row of the tile a
    // lane; warps 4-7 take every other 32 columns, warps 8-11 the rest.
    const int quad = warp % 4, half = warp / 4 - 1;
    unsigned char* block = transpose + (warp - 4) * kBlockBytes<SWAP>;
    int turn = 0;
    for (int u = first; u < units; u += step, ++turn) {
      const TileAt at = tile_at(p, u % tiles);
      const int split = u / tiles;
      const int acc = turn & 1;
      const int64_t a_row = (int64_t)(at.a * CG + (int)rank) * 128 + quad * 32;  // lane 0's row of A
      const EpilogueArgs& e = p.e;
      if constexpr (!SWAP) {
        if (half == 0 && (int64_t)at.b * BN < e.cols) prefetch_row<EPI, ACT>(e, a_row + lane, (int64_t)at.b * BN, BN);
      }
      ok = warp_wait_bounded(acc_full + acc, (turn >> 1) & 1, p.wait_limit_ns);
      if (!ok) break;
      tc_fence_after();
      const uint32_t from = tmem + acc * BN + ((uint32_t)(quad * 32) << 16);
      float lane_bias = 0.0f;
      if (SWAP && EPI == EPI_FORWARD && e.bias && a_row + lane < e.cols) lane_bias = __bfloat162float(e.bias[a_row + lane]);
      auto hand_back = [&] {  // this warp has read its share: the accumulator may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_cluster_relaxed(mapped_addr(smem_addr(acc_empty + acc), 0));
          else
            mbar_arrive(acc_empty + acc);
        }
      };
      if (half * 32 >= BN) hand_back();
#pragma unroll 1
      for (int c = half * 32; c < BN; c += 64) {
        const int64_t b_row = (int64_t)at.b * BN + c;  // the first of 32 rows of B
        float v[32];
        __syncwarp();
        tmem_load32(from + c, v);
        if (c + 64 >= BN) hand_back();
        if constexpr (SWAP) {
          // Lane l has column a_row + l of the output in 32 rows: neighbouring
          // lanes on neighbouring elements.
          if (a_row >= e.cols || b_row >= e.rows) continue;
          float* turned = reinterpret_cast<float*>(block);
#pragma unroll
          for (int i = 0; i < 32; ++i) turned[lane * 33 + i] = v[i];
          __syncwarp();
          const int n = (int)min((int64_t)32, e.rows - b_row);
          const bool in = a_row + lane < e.cols;
          for (int r = 0; r < n; r += 8) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = turned[lane * 33 + r + i];
            if constexpr (EPI == EPI_PARTIAL) {
              float* q = e.partial + (split * e.rows + b_row + r) * e.ldp + a_row + lane;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (r + i < n) q[i * e.ldp] = t[i];
            } else {
              epilogue_columns<EPI, ACT>(e, b_row + r, n - r, a_row + lane, in, t, lane_bias);
            }
          }
        } else {
          if (a_row >= e.rows || (EPI != EPI_PARTIAL && b_row >= e.cols)) continue;
          if constexpr (EPI == EPI_PARTIAL) {
            float4* q = partial_block(e, split, a_row, b_row, lane);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[32 * i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            epilogue_tile<EPI, ACT>(e, a_row, b_row, lane, block, v);
          }
        }
      }
    }
  }
  // This kernel is not done before the one beside it is.
  if (p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!ok && lane == 0) atomicAdd(p.timeouts, 1u);
  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2)
    cluster_sync();
  else
    __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_free<CG>(tmem, Shape::columns);
  }
}

// The sums of the splits, in order, through the epilogue.  Swapped: a warp
// takes 32 columns of a row; without splits (nothing to sum) the sums are zero.
// Otherwise a warp takes a block of 32 x 32.
constexpr int kJoinThreads = 128;

template <int EPI, int ACT, bool SWAP>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const EpilogueArgs e, int splits) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32;
  const int64_t across = (e.cols + 31) / 32;
  const int64_t i = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) / 32;
  if constexpr (SWAP) {
    const int64_t row = i / across;
    if (row >= e.rows) return;
    const int64_t col = (i - row * across) * 32 + lane;
    const bool in = col < e.cols;
    float v[1] = {0.0f};
    const float* q = e.partial + row * e.ldp + col;
    if (in)
      for (int s = 0; s < splits; ++s) v[0] += q[(int64_t)s * e.rows * e.ldp];
    float bias = 0.0f;
    if (EPI == EPI_FORWARD && e.bias && in) bias = __bfloat162float(e.bias[col]);
    epilogue_columns<EPI, ACT>(e, row, 1, col, in, v, bias);
  } else {
    __shared__ __align__(128) unsigned char blocks[kJoinThreads / 32][kBlockBytes<false>];
    const int64_t row = i / across * 32, col = i % across * 32;
    if (row >= e.rows) return;
    float v[32] = {};
    for (int s = 0; s < splits; ++s) {
      const float4* q = partial_block(e, s, row, col, lane);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 t = q[32 * k];
        v[4 * k] += t.x, v[4 * k + 1] += t.y, v[4 * k + 2] += t.z, v[4 * k + 3] += t.w;
      }
    }
    epilogue_tile<EPI, ACT>(e, row, col, lane, blocks[threadIdx.x / 32], v);
  }
}

// The tiles that are built: pairs of CTAs on 256 x 256 and 256 x 128, and, with
// A and B swapped, single CTAs on 128 weight rows by kSmallB or 128 tokens.
enum TcTile { TILE_256x256, TILE_256x128, TILE_SWAP_128, TILE_SWAP_SMALL };
struct TcTileShape {
  int a, b, ctas;  // rows of A and of B in a tile, CTAs on it
  bool swap;
};
// Rows of B in the small swapped tile; an MN-major operand comes in 64s.
constexpr int small_b(bool mn) { return mn ? 64 : 32; }
inline TcTileShape tile_shape(TcTile t, bool b_mn_when_swapped) {
  switch (t) {
    case TILE_256x256: return {256, 256, 2, false};
    case TILE_256x128: return {256, 128, 2, false};
    case TILE_SWAP_128: return {128, 128, 1, true};
    default: return {128, small_b(b_mn_when_swapped), 1, true};
  }
}

// Launches the product kernel of one operand layout (ops_linear_*.cu).  `after`:
// the kernel before it on the stream belongs to the same call.
cudaError_t launch_forward(const TcArgs& p, TcTile t, int grid, bool after, cudaStream_t stream);
cudaError_t launch_grad_input(const TcArgs& p, TcTile t, int grid, bool after, cudaStream_t stream);
cudaError_t launch_grad_weight(const TcArgs& p, TcTile t, int grid, bool after, cudaStream_t stream);

template <int CG, int BN, bool A_MN, bool B_MN, int EPI, int ACT, bool SWAP>
cudaError_t launch_tc(const TcArgs& p, int grid, bool after, cudaStream_t stream) {
  auto kernel = gemm_tc_kernel<CG, BN, A_MN, B_MN, EPI, ACT, SWAP>;
  constexpr int smem = TcShape<CG, BN, EPI, SWAP>::smem_bytes;
  static std::atomic<uint64_t> ready{0};  // devices (bits) whose limit has been raised
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  if (CG == 2) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = CG;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// A tile's kernel, of the call's epilogue or, with several splits, of the one that
// puts their sums to p.e.partial.
template <int CG, int BN, bool A_MN, bool B_MN, int EPI, bool SWAP>
cudaError_t launch_tile(const TcArgs& p, int grid, bool after, cudaStream_t stream) {
  if (p.splits > 1) return launch_tc<CG, BN, A_MN, B_MN, EPI_PARTIAL, TIDE_ACT_NONE, SWAP>(p, grid, after, stream);
  if constexpr (EPI == EPI_PLAIN)
    return launch_tc<CG, BN, A_MN, B_MN, EPI, TIDE_ACT_NONE, SWAP>(p, grid, after, stream);
  else
    return with_act(p.e.act, [&](auto act) {
      return launch_tc<CG, BN, A_MN, B_MN, EPI, act.value, SWAP>(p, grid, after, stream);
    });
}

// A_MN, B_MN: the operands' majors unswapped.
template <bool A_MN, bool B_MN, int EPI>
cudaError_t launch_layout(const TcArgs& p, TcTile t, int grid, bool after, cudaStream_t stream) {
  switch (t) {
    case TILE_256x256: return launch_tile<2, 256, A_MN, B_MN, EPI, false>(p, grid, after, stream);
    case TILE_256x128: return launch_tile<2, 128, A_MN, B_MN, EPI, false>(p, grid, after, stream);
    case TILE_SWAP_128: return launch_tile<1, 128, B_MN, A_MN, EPI, true>(p, grid, after, stream);
    default: return launch_tile<1, small_b(A_MN), B_MN, A_MN, EPI, true>(p, grid, after, stream);
  }
}

}  // namespace tide
