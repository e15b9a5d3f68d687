// The global norm of many tensors, and clipping by it (include/tide_lm_ops.h).
//
// One pass over the tensors for the norm, one more (in and out) for clipping, a
// few operations an element: both are bound by memory traffic.  The list of tensors
// travels in the kernel's arguments (up to 32 KB of them), so a call copies nothing to the device,
// and a captured one keeps its list.
//
//   64 fp32 tensors of 5.5 million elements (1.4 GB): norm 195 to 198 us, 7.1 TB/s; clipping 433 us, 6.5 TB/s of
//   reads and writes; 391 tensors of all sizes and alignments (60 MB) 17 and 23 us
//
// A tensor is walked in chunks of kChunk bytes counted from the 16-byte granule it starts
// in, so that every load but the first and the last granule's is a whole 16 bytes
// whatever the tensor's alignment.

#include <algorithm>
#include <cmath>

#include "cluster_ptx.cuh"
#include "ops_common.cuh"

#include "../../include/tide_lm_ops.h"

namespace tide {
namespace {

constexpr int kThreads = 256;
// Granules of 16 bytes a thread and chunk (with 4, 64 tensors of 22 MB take 205 and 448 us, with 2 215 and 462).
constexpr int kGranules = 8;
constexpr int64_t kChunk = 16 * kThreads * kGranules;    // 32 KB
constexpr int kPerSm = 4;                                // blocks an SM: 128 KB of loads in flight
// The norm asks L2 to keep the last 64 MB of a launch's tensors, from which clipping begins, and to let what
// is before go first (norm and clipping of 200 MB 103 us without, 100 with; of 1.4 GB 654 and 648).  That helps lists
// of one launch: of more tensors than a table holds, launches follow one another from the list's front, in the norm
// and in clipping, so that clipping begins with what left L2 long ago.
constexpr int kKept = (64 << 20) / (int)kChunk;

// Tensors of a launch, by the room that a kernel's 32,764 bytes of arguments leave;
// small lists take small tables, since arguments are copied for every launch.
constexpr int kNormTables[] = {32, 256, 512, 1600}, kClipTables[] = {32, 256, 512, 1150};

template <int CAP>
struct NormTable {
  int32_t count, chunks;
  float per_chunk;    // tensors
  uint64_t at[CAP];   // address; bit 0: fp32
  int64_t bytes[CAP];
  int32_t end[CAP];   // chunks of the tensors up to this one
};
template <int CAP>
struct ClipTable {
  NormTable<CAP> from;
  void* out[CAP];
};

struct ChunkRange {
  const unsigned char* granule;  // the tensor's first granule
  int64_t first, last;           // the tensor's bytes, from there
  int64_t at;                    // the chunk's first byte
  bool fp32;
  int tensor;
  __device__ __forceinline__ bool whole() const { return at >= first && at + kChunk <= last; }
};

template <int CAP>
__device__ __forceinline__ ChunkRange chunk_of(const NormTable<CAP>& t, int chunk) {
  // The first tensor whose chunks end behind this one.  Each look at the table costs half a microsecond while it is
  // not in the SM's constant cache, so the first is at the place where a list of like tensors has it.
  int lo = 0, hi = t.count - 1;
  int mid = min((int)((float)chunk * t.per_chunk), hi);
  while (lo < hi) {
    const int end = t.end[mid], begin = mid > 0 ? t.end[mid - 1] : 0;
    if (begin <= chunk && chunk < end)
      lo = hi = mid;
    else if (chunk < begin)
      hi = mid - 1;
    else
      lo = mid + 1;
    mid = (lo + hi) / 2;
  }
  const uint64_t a = t.at[lo] & ~1ull;
  ChunkRange r;
  r.granule = reinterpret_cast<const unsigned char*>(a & ~15ull);
  r.first = (int64_t)(a & 15);
  r.last = r.first + t.bytes[lo];
  r.at = (int64_t)(chunk - (lo > 0 ? t.end[lo - 1] : 0)) * kChunk;
  r.fp32 = t.at[lo] & 1;
  r.tensor = lo;
  return r;
}

// The 16 bytes at `off` (from the first granule): those of the tensor, zeros for the rest.
__device__ __forceinline__ uint4 load_edge(const ChunkRange& r, int64_t off) {
  uint32_t w[4] = {0, 0, 0, 0};
  const int step = r.fp32 ? 4 : 2;
#pragma unroll
  for (int k = 0; k < 8; ++k) {  // pairs of bytes
    const int64_t b = off + 2 * k;
    if (b < r.first || b >= r.last || (step == 4 && k % 2)) continue;
    if (step == 4)
      w[k / 2] = *reinterpret_cast<const uint32_t*>(r.granule + b);
    else
      w[k / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(r.granule + b) << (16 * (k % 2));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes with an L2 policy.
__device__ __forceinline__ uint4 load_once(const unsigned char* p, uint64_t policy) {
  uint4 v;
  asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p), "l"(policy));
  return v;
}

// The granules of a chunk that are the x-th of kThreads threads'; once: an L2 policy for whole chunks' loads, 0 for none.
__device__ __forceinline__ void load_chunk(const ChunkRange& r, int x, uint4 (&u)[kGranules], uint64_t once = 0) {
  const unsigned char* p = r.granule + r.at + x * 16;
  if (r.whole()) {
#pragma unroll
    for (int j = 0; j < kGranules; ++j) u[j] = once ? load_once(p + j * kThreads * 16, once) : *reinterpret_cast<const uint4*>(p + j * kThreads * 16);
  } else {
#pragma unroll
    for (int j = 0; j < kGranules; ++j) {
      const int64_t off = r.at + (j * kThreads + x) * 16;
      u[j] = make_uint4(0, 0, 0, 0);
      if (off >= r.first && off + 16 <= r.last)
        u[j] = *reinterpret_cast<const uint4*>(r.granule + off);
      else if (off + 16 > r.first && off < r.last)
        u[j] = load_edge(r, off);
    }
  }
}

__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The sum of a thread's squares of a chunk.  fp32 over the 32 or 64 of them, and fp64
// from chunk to chunk (a conversion and an addition a chunk).  Where the fp32 sum is
// so small that squares may have been lost below its range, or so large that they
// left it above, the same values are summed in fp64 instead.
__device__ __forceinline__ double squares(const uint4 (&u)[kGranules], bool fp32) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (fp32) {
#pragma unroll
    for (int j = 0; j < kGranules; ++j) {
      const float x = __uint_as_float(u[j].x), y = __uint_as_float(u[j].y), z = __uint_as_float(u[j].z),
                  w = __uint_as_float(u[j].w);
      s[0] = fmaf(x, x, s[0]), s[1] = fmaf(y, y, s[1]), s[2] = fmaf(z, z, s[2]), s[3] = fmaf(w, w, s[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kGranules; ++j) {
      const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = lo_bf16(w[k]), b = hi_bf16(w[k]);
        s[k] = fmaf(a, a, s[k]);
        s[k] = fmaf(b, b, s[k]);
      }
    }
  }
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  // 64 squares lost below 2^-126 are 2^-30 of 2^-90.
  if (sum >= 0x1p-90f && sum < 0x1p120f) return (double)sum;
  uint32_t any = 0;
#pragma unroll
  for (int j = 0; j < kGranules; ++j) any |= u[j].x | u[j].y | u[j].z | u[j].w;
  if ((any & (fp32 ? 0x7fffffffu : 0x7fff7fffu)) == 0) return 0.0;
  double d = 0.0;
#pragma unroll
  for (int j = 0; j < kGranules; ++j) {
    const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const double a = (double)(fp32 ? __uint_as_float(w[k]) : lo_bf16(w[k]));
      const double b = fp32 ? 0.0 : (double)hi_bf16(w[k]);
      d += a * a + b * b;
    }
  }
  return d;
}

// The block's sum, in a fixed order, in thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warps[32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x < 32) {
    v = threadIdx.x < blockDim.x / 32 ? warps[threadIdx.x] : 0.0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  }
  return v;
}

// JOIN: the grid is one cluster, whose first block joins the others' sums by itself.  Blocks take AT_ONCE chunks at a time.
template <int CAP, bool JOIN, int AT_ONCE>
__global__ void __launch_bounds__(kThreads * AT_ONCE, AT_ONCE == 1 ? kPerSm : 1)
    norm_kernel(const __grid_constant__ NormTable<CAP> t, double* partial, float* norm) {
  if constexpr (!JOIN) let_next_kernel_start();  // the join's block waits beside this: 211 tensors of 400 bytes 5.9 us became 5.2
  const uint64_t policy = policy_evict_first();
  double sum = 0.0;
  for (int c = blockIdx.x * AT_ONCE + threadIdx.x / kThreads; c < t.chunks; c += gridDim.x * AT_ONCE) {
    const ChunkRange r = chunk_of(t, c);
    uint4 u[kGranules];
    load_chunk(r, threadIdx.x % kThreads, u, c < t.chunks - kKept ? policy : 0);
    sum += squares(u, r.fp32);
  }
  sum = block_sum(sum);
  if constexpr (JOIN) {
    __shared__ double mine;
    if (threadIdx.x == 0) mine = sum;
    cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x < 32) {
      sum = threadIdx.x < gridDim.x ? load_peer_f64(peer_smem(&mine, threadIdx.x)) : 0.0;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (threadIdx.x == 0) *norm = (float)sqrt(sum);
    }
    cluster_sync();  // no block leaves while its sum is being read
  } else {
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
  }
}

__global__ void __launch_bounds__(kThreads) norm_join_kernel(const double* partial, int64_t n, float* norm) {
  wait_for_kernel_before();
  double sum = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += partial[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) *norm = (float)sqrt(sum);
}

// The last chunks first: where the list is one launch's, the norm's pass has left them in L2.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kPerSm) clip_kernel(const __grid_constant__ ClipTable<CAP> t, const float* norm,
                                                               float max_norm, float eps) {
  const float n = *norm, q = max_norm / (n + eps);
  const float by = isnan(n) ? n : q < 1.0f ? q : 1.0f;
  for (int c = t.from.chunks - 1 - (int)blockIdx.x; c >= 0; c -= (int)gridDim.x) {
    const ChunkRange r = chunk_of(t.from, c);
    unsigned char* const out = (unsigned char*)t.out[r.tensor];  // byte `first` of the granules
    if (by == 1.0f && out == r.granule + r.first) continue;
    if (((uintptr_t)out & 15) == (uintptr_t)r.first) {
      uint4 u[kGranules];
      load_chunk(r, threadIdx.x, u);
#pragma unroll
      for (int j = 0; j < kGranules; ++j) {
        uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = r.fp32 ? __float_as_uint(__uint_as_float(w[k]) * by) : pack_bf16(lo_bf16(w[k]) * by, hi_bf16(w[k]) * by);
        const int64_t off = r.at + (j * kThreads + (int)threadIdx.x) * 16;
        if (off >= r.first && off + 16 <= r.last) {
          *reinterpret_cast<uint4*>(out - r.first + off) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if (off + 16 > r.first && off < r.last) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int64_t b = off + 2 * k;
            if (b < r.first || b >= r.last || (r.fp32 && k % 2)) continue;
            if (r.fp32)
              *reinterpret_cast<uint32_t*>(out - r.first + b) = w[k / 2];
            else
              *reinterpret_cast<uint16_t*>(out - r.first + b) = (uint16_t)(w[k / 2] >> (16 * (k % 2)));
          }
        }
      }
    } else {  // another phase within 16 bytes: element by element (1.4 GB of fp32 1237 us, against 474 of one phase)
      const int step = r.fp32 ? 4 : 2;
      const int64_t lo = r.at > r.first ? r.at : r.first, hi = r.at + kChunk < r.last ? r.at + kChunk : r.last;
      for (int64_t b = lo + (int64_t)threadIdx.x * step; b < hi; b += kThreads * step) {
        if (r.fp32)
          *reinterpret_cast<float*>(out - r.first + b) = *reinterpret_cast<const float*>(r.granule + b) * by;
        else
          *reinterpret_cast<bf16*>(out - r.first + b) =
              __float2bfloat16_rn(__bfloat162float(*reinterpret_cast<const bf16*>(r.granule + b)) * by);
      }
    }
  }
}

// ---------------------------------------------------------------- host side

tide_status check_list(int32_t count, const void* const* tensors, const int64_t* numels, const int32_t* dtypes) {
  if (count < 0) return fail(TIDE_ERR_INVALID_ARG, "negative number of tensors");
  if (count > 0 && (!tensors || !numels || !dtypes)) return fail(TIDE_ERR_INVALID_ARG, "a list of tensors is NULL");
  for (int32_t i = 0; i < count; ++i) {
    TIDE_TRY(check_dtype(dtypes[i]));
    if (numels[i] < 0) return fail(TIDE_ERR_INVALID_ARG, "tensor " + std::to_string(i) + " has a negative size");
    TIDE_TRY(check_matrix(tensors[i], 1, numels[i], numels[i], elem_bytes_of(dtypes[i]), "a tensor of the list"));
    // Chunks of a launch are counted in 32 bits.
    if (numels[i] > (int64_t)1 << 40) return fail(TIDE_ERR_UNIMPLEMENTED, "a tensor of more than 2^40 elements");
  }
  return TIDE_OK;
}

int64_t list_bytes(int32_t count, const int64_t* numels, const int32_t* dtypes) {
  int64_t n = 0;
  for (int32_t i = 0; i < count; ++i) n += std::min<int64_t>(numels[i], (int64_t)1 << 40) * elem_bytes_of(dtypes[i]);
  return n;
}

int table_size(int64_t count, const int (&sizes)[4]) {
  for (int i = 0; i < 3; ++i)
    if (count <= sizes[i]) return sizes[i];
  return sizes[3];
}

// Fills a table from tensor `i` on, at most CAP tensors and so many chunks that 32 bits
// count them; returns the next.
template <int CAP, typename F>
int32_t fill(NormTable<CAP>& t, int32_t i, int32_t count, const void* const* tensors, const int64_t* numels,
             const int32_t* dtypes, F&& also) {
  t.count = 0;
  int64_t chunks = 0;
  for (; i < count && t.count < CAP; ++i) {
    if (numels[i] == 0) continue;
    const int64_t bytes = numels[i] * elem_bytes_of(dtypes[i]);
    const int64_t more = ((int64_t)((uintptr_t)tensors[i] & 15) + bytes + kChunk - 1) / kChunk;
    if (chunks + more > INT32_MAX / 2) break;  // one tensor's alone are below 2^27 + 1
    chunks += more;
    t.at[t.count] = (uint64_t)(uintptr_t)tensors[i] | (dtypes[i] == TIDE_F32 ? 1u : 0u);
    t.bytes[t.count] = bytes;
    t.end[t.count] = (int32_t)chunks;
    also(t.count, i);
    ++t.count;
  }
  t.chunks = (int32_t)chunks;
  t.per_chunk = chunks > 0 ? (float)t.count / (float)chunks : 0.0f;
  return i;
}

// Up to so many chunks a single cluster of kCluster blocks does alone: no partial sums in memory, for which the
// binding would ask the allocator (7 us), and one launch.  One cluster against two launches, us a call from Python and in a
// graph: 12 tensors of 32 KB 4.4 and 4.4 against 13.6 and 4.6, 60 of 32 KB 7.4 and 7.8 against 14.0 and 5.1, one of 2 MB
// 4.3 and 6.9 against 13.2 and 4.9; 100 of 400 bytes 8.9 and 10.5 against 14.9 and 4.5.  Blocks of kAtOnce chunks at a
// time take a microsecond longer to begin (12 tensors in a graph 5.7 against 4.4), so those are for the longer lists.
constexpr int64_t kAlone = 64;
constexpr int kCluster = 8, kAtOnce = 4;
bool alone(int32_t count, const int64_t* numels, const int32_t* dtypes) {
  int64_t chunks = 0;  // at most, whatever the addresses
  for (int32_t i = 0; i < count && chunks <= kAlone; ++i) {
    const int64_t bytes = std::min<int64_t>(numels[i], (int64_t)1 << 40) * elem_bytes_of(dtypes[i]);
    chunks += bytes > 0 ? (15 + bytes + kChunk - 1) / kChunk : 0;
  }
  return chunks <= kAlone;
}

// Launches of a list of tensors at most: a table full of tensors, or of chunks.
int64_t launches(int32_t count, int64_t bytes, const int (&sizes)[4]) {
  return (count + sizes[3] - 1) / sizes[3] + bytes / ((INT32_MAX / 4) * kChunk);
}

template <int CAP>
tide_status norm_list(int32_t count, const void* const* tensors, const int64_t* numels, const int32_t* dtypes, float* norm,
                      double* partial, int64_t room, cudaStream_t stream) {
  NormTable<CAP> t;
  if (alone(count, numels, dtypes)) {
    fill(t, 0, count, tensors, numels, dtypes, [](int, int32_t) {});
    const bool few = t.chunks <= 3 * kCluster;
    const ClusterLaunch l(kCluster, dim3(few ? kThreads : kThreads * kAtOnce), kCluster, false, 0, stream);
    return cuda_status(few ? cudaLaunchKernelEx(&l.cfg, norm_kernel<CAP, true, 1>, t, (double*)nullptr, norm)
                           : cudaLaunchKernelEx(&l.cfg, norm_kernel<CAP, true, kAtOnce>, t, (double*)nullptr, norm),
                       "gradient norm");
  }
  const int64_t most = (int64_t)ops_num_sms() * kPerSm;
  int64_t sums = 0;
  for (int32_t i = 0; i < count;) {
    i = fill(t, i, count, tensors, numels, dtypes, [](int, int32_t) {});
    if (t.count == 0) continue;
    const int64_t grid = std::min<int64_t>(t.chunks, most);
    if ((sums + grid) * (int64_t)sizeof(double) > room) return fail(TIDE_ERR_INVALID_ARG, "workspace too small");
    norm_kernel<CAP, false, 1><<<(unsigned)grid, kThreads, 0, stream>>>(t, partial + sums, nullptr);
    TIDE_TRY(cuda_status(cudaGetLastError(), "gradient norm"));
    sums += grid;
  }
  const ClusterLaunch l(1, dim3(kThreads), 1, sums > 0, 0, stream);
  return cuda_status(cudaLaunchKernelEx(&l.cfg, norm_join_kernel, (const double*)partial, sums, norm), "joining partial sums");
}

template <int CAP>
tide_status clip_list(int32_t count, const void* const* tensors, void* const* outs, const int64_t* numels,
                      const int32_t* dtypes, const float* norm, float max_norm, float eps, cudaStream_t stream) {
  ClipTable<CAP> t;
  const int64_t most = (int64_t)ops_num_sms() * kPerSm;
  for (int32_t i = 0; i < count;) {
    i = fill(t.from, i, count, tensors, numels, dtypes, [&](int at, int32_t which) { t.out[at] = outs[which]; });
    if (t.from.count == 0) continue;
    clip_kernel<CAP><<<(unsigned)std::min<int64_t>(t.from.chunks, most), kThreads, 0, stream>>>(t, norm, max_norm, eps);
    TIDE_TRY(cuda_status(cudaGetLastError(), "gradient clipping"));
  }
  return TIDE_OK;
}

}  // namespace
}  // namespace tide

using namespace tide;

extern "C" {

int64_t tide_grad_norm_workspace(int32_t count, const int64_t* numels, const int32_t* dtypes) {
  if (count <= 0 || !numels || !dtypes || alone(count, numels, dtypes)) return 0;
  return launches(count, list_bytes(count, numels, dtypes), kNormTables) * ops_num_sms() * kPerSm * (int64_t)sizeof(double);
}

tide_status tide_grad_norm(int32_t count, const void* const* tensors, const int64_t* numels, const int32_t* dtypes,
                           float* norm, void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  TIDE_TRY(check_list(count, tensors, numels, dtypes));
  TIDE_TRY(check_matrix(norm, 1, 1, 1, 4, "norm"));
  const int64_t need = tide_grad_norm_workspace(count, numels, dtypes);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(TIDE_ERR_INVALID_ARG, "workspace too small: " + std::to_string(need) + " bytes are needed");
  if ((uintptr_t)workspace % 16) return fail(TIDE_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  if (ops_num_sms() <= 0) return fail(TIDE_ERR_CUDA, "the current device could not be queried");
  double* const partial = (double*)workspace;
  const cudaStream_t s = (cudaStream_t)stream;
  switch (table_size(count, kNormTables)) {
    case kNormTables[0]: return norm_list<kNormTables[0]>(count, tensors, numels, dtypes, norm, partial, need, s);
    case kNormTables[1]: return norm_list<kNormTables[1]>(count, tensors, numels, dtypes, norm, partial, need, s);
    case kNormTables[2]: return norm_list<kNormTables[2]>(count, tensors, numels, dtypes, norm, partial, need, s);
    default: return norm_list<kNormTables[3]>(count, tensors, numels, dtypes, norm, partial, need, s);
  }
}

tide_status tide_grad_clip(int32_t count, const void* const* tensors, void* const* outs, const int64_t* numels,
                           const int32_t* dtypes, const float* norm, float max_norm, float eps, void* stream) {
  clear_error();
  TIDE_TRY(check_list(count, tensors, numels, dtypes));
  if (!(max_norm >= 0.0f) || !(eps >= 0.0f)) return fail(TIDE_ERR_INVALID_ARG, "max_norm and eps are not negative");
  if (count == 0) return TIDE_OK;
  if (!outs) return fail(TIDE_ERR_INVALID_ARG, "a list of tensors is NULL");
  for (int32_t i = 0; i < count; ++i)
    TIDE_TRY(check_matrix(outs[i], 1, numels[i], numels[i], elem_bytes_of(dtypes[i]), "an output of the list"));
  TIDE_TRY(check_matrix(norm, 1, 1, 1, 4, "norm"));
  if (ops_num_sms() <= 0) return fail(TIDE_ERR_CUDA, "the current device could not be queried");
  const cudaStream_t s = (cudaStream_t)stream;
  switch (table_size(count, kClipTables)) {
    case kClipTables[0]: return clip_list<kClipTables[0]>(count, tensors, outs, numels, dtypes, norm, max_norm, eps, s);
    case kClipTables[1]: return clip_list<kClipTables[1]>(count, tensors, outs, numels, dtypes, norm, max_norm, eps, s);
    case kClipTables[2]: return clip_list<kClipTables[2]>(count, tensors, outs, numels, dtypes, norm, max_norm, eps, s);
    default: return clip_list<kClipTables[3]>(count, tensors, outs, numels, dtypes, norm, max_norm, eps, s);
  }
}

}  // extern "C"
