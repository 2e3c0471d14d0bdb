// smla_step_tables: what the other calls take of a step's geometry, from the requests' lengths.
//
// [AgentX "Hybrid KV cache management"]: sequences hold blocks of one shared pool.  [GLM-5.3 "Config and
// numbers"]: with drafted tokens (MTP3) a step's lengths follow from what the step before accepted, which the GPU
// knows first.  Entry i of the step is the request in row r = rows[i] of the persistent tables:
//   blocks_i = ceil((len_r + new_i) / block_size),  need_i = max(0, blocks_i - held_r)
//   query_start_loc = exclusive sums of new_i,  first_i = free_used + exclusive sum of need_i
//   block j of the sequence: table[r][j] if j < held_r, else free_blocks[first_i + j - held_r]
//   token k of the entry: position len_r + k, slot block * block_size + position % block_size
// In whole numbers throughout: the same call gives the same tables whatever the order of its threads.
//
// One CTA forms both sums and what depends on them alone, while others copy the blocks of cached tokens, which need
// no sum; all others wait for it and then take the new blocks and the tokens.  Only that CTA reads and writes
// held and free_used, which may therefore be updated in place.  Steps of small tables are one launch, a cluster of up to
// eight CTAs that meet at its barrier; large ones are two, the second launched with the first and over all SMs
// (an SM writes 32 bytes a cycle).
// Bound by latency: the chain rows -> lengths -> two sums over 1,024 threads -> plan -> table -> slots, each a round of
// loads, and a launch.  A request 8.3 us replayed as a graph (12 a call), 64 requests of up to 262,144 positions with four
// tokens each 10.3 (13), 1,024 requests of up to 32,768 positions on pages of 16, 512 new tokens at most, 10.3 in two
// launches (15).
#include <algorithm>
#include <climits>

#include "smla_internal.h"

namespace smla {
namespace {

constexpr int kPlanThreads = 1024, kFillThreads = 256, kSegment = 1024;  // kSegment: table entries of a warp's unit
constexpr int kMaxCluster = 8;  // the portable size
// One launch up to here: a call for one request 12.3 us (two launches 14.3), 64 rows of 4,096 blocks, half of these entries,
// 12.9 (15.4).  Beyond, eight CTAs would write the tables at 256 bytes a cycle at most: 8 MB of 1,024 rows take 16 us.
constexpr int64_t kOneLaunchEntries = 1 << 19, kOneLaunchTokens = 1 << 15;
constexpr int kSearchEntries = 4096;  // batches whose query_start_loc is searched in shared memory
constexpr int kMaxContext = INT_MAX - 1023;  // as smla_attend_dense

struct TableArgs {
  int block_size;
  int64_t num_blocks;
  const int32_t *rows, *lens, *new_lens;
  int batch;
  int32_t* table;
  int64_t n_rows;
  int table_stride;
  const int32_t* held;
  int32_t* held_out;
  const int32_t* free_blocks;
  int64_t n_free;
  const int64_t* free_used;
  int64_t* free_used_out;
  int n_tokens;
  int32_t *seq_lens, *qsl;
  int64_t *positions, *slots;
  int32_t* block_table;
  int bt_stride;
  int cap;         // positions that a row holds, kMaxContext at most
  int segments;    // of a row
  bool vec;        // the rows of both tables load and store in 16-byte pieces
  int4* plan;      // [batch]: row (-1: none), held, blocks, len
  int64_t* first;  // [batch]
  unsigned* err;
};

// Row and cached length of entry i, the length cut to what a row holds; row -1: an entry without a request.
__device__ __forceinline__ int entry_row(const TableArgs& A, int i, int& len, bool& bad) {
  int row = A.rows != nullptr ? __ldg(A.rows + i) : i;
  bad = row >= A.n_rows;
  if (row < 0 || bad) {
    len = 0;
    return -1;
  }
  const int n = __ldg(A.lens + row);
  len = min(max(n, 0), A.cap);
  bad = n != len;
  return row;
}

__device__ __forceinline__ int blocks_of(const TableArgs& A, int len) {
  return static_cast<int>((static_cast<unsigned>(len) + A.block_size - 1) / static_cast<unsigned>(A.block_size));
}

// Exclusive sum over the CTA (`sums`: a slot per warp), and the total of all threads.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // the slots of the scan before are read
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t w = sums[lane];  // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return (warp > 0 ? before : 0) + incl - v;
}

// Sums, lengths and offsets of all entries, by one CTA of kPlanThreads.
__device__ __forceinline__ void plan_entries(const TableArgs& A, int64_t* sums) {
  static_assert(kPlanThreads == 32 * 32, "scan takes 32 warps");
  const int64_t used0 = *A.free_used;  // read before the last barrier, written after it: the two may be one word
  const int64_t used = min(max(used0, static_cast<int64_t>(0)), A.n_free);
  bool bad = used0 != used, out_of_blocks = false;
  int64_t tokens = 0, taken = 0;
  for (int i0 = 0; i0 < A.batch; i0 += kPlanThreads) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    int row = -1, len = 0, n = 0, held = 0;
    if (i < A.batch) {
      bool b = false;
      row = entry_row(A, i, len, b);
      bad |= b;
      if (row >= 0) {
        const int want = __ldg(A.new_lens + i);
        n = min(max(want, 0), A.cap - len);
        bad |= n != want;
        held = min(max(A.held[row], blocks_of(A, len)), A.table_stride);
      }
    }
    int64_t all;
    const int64_t q0 = tokens + scan(n, sums, all);
    tokens += all;
    // tokens that the arrays do not hold are not taken
    const int s = static_cast<int>(min(q0, static_cast<int64_t>(A.n_tokens)));
    const int e = static_cast<int>(min(q0 + n, static_cast<int64_t>(A.n_tokens)));
    bad |= e - s != n;
    n = e - s;
    const int blocks = blocks_of(A, len + n);
    const int need = row >= 0 ? max(0, blocks - held) : 0;
    const int64_t first = used + taken + scan(need, sums, all);
    taken += all;
    if (i < A.batch) {
      A.plan[i] = make_int4(row, held, blocks, len);
      A.first[i] = first;
      A.seq_lens[i] = len + n;
      A.qsl[i] = s;
      if (row >= 0) {
        const int64_t there = max(static_cast<int64_t>(0), A.n_free - first);
        out_of_blocks |= there < need;
        A.held_out[row] = held + static_cast<int>(min(static_cast<int64_t>(need), there));
      }
    }
  }
  // the entries' faults are reported together, so that which one is latched does not depend on their threads
  out_of_blocks = __syncthreads_or(out_of_blocks) != 0;
  bad = __syncthreads_or(bad) != 0;
  if (threadIdx.x == 0) {
    A.qsl[A.batch] = static_cast<int>(min(tokens, static_cast<int64_t>(A.n_tokens)));
    *A.free_used_out = min(used + taken, A.n_free);
    if (out_of_blocks) latch_error(A.err, SMLA_ERR_NO_BLOCKS);
    else if (bad) latch_error(A.err, SMLA_ERR_BAD_INDEX);
  }
}

// The blocks of cached tokens, by warp `warp` of `warps`: nothing else of this call writes what is read here.
__device__ __forceinline__ void copy_cached(const TableArgs& A, int64_t warp, int64_t warps) {
  const int lane = threadIdx.x & 31;
  const int64_t units = static_cast<int64_t>(A.batch) * A.segments;
  if (A.block_table != nullptr) {
    for (int64_t u = warp; u < units; u += warps) {
      const int i = static_cast<int>(u / A.segments), j0 = static_cast<int>(u % A.segments) * kSegment;
      int len;
      bool bad;
      const int row = entry_row(A, i, len, bad);
      const int n = min(row < 0 ? 0 : blocks_of(A, len), j0 + kSegment) - j0;
      if (n <= 0) continue;
      const int32_t* src = A.table + row * static_cast<int64_t>(A.table_stride) + j0;
      int32_t* dst = A.block_table + i * static_cast<int64_t>(A.bt_stride) + j0;
      int at = 0;
      if (A.vec) {
        at = n & ~3;
        int4 v[kSegment / 128];
#pragma unroll
        for (int x = 0; x < kSegment / 128; ++x)
          if (128 * x + 4 * lane < at) v[x] = *reinterpret_cast<const int4*>(src + 128 * x + 4 * lane);
#pragma unroll
        for (int x = 0; x < kSegment / 128; ++x)
          if (128 * x + 4 * lane < at) *reinterpret_cast<int4*>(dst + 128 * x + 4 * lane) = v[x];
      }
      for (int j = at + lane; j < n; j += 32) dst[j] = src[j];
    }
  }
}

// What needs the plan (read by ordinary loads: it was written in this launch or the one beside it), by CTA `cta` of `ctas`.
template <int kThreads>
__device__ __forceinline__ void fill(const TableArgs& A, int32_t* loc, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(cta) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t warps = static_cast<int64_t>(ctas) * (kThreads / 32);
  const int64_t units = static_cast<int64_t>(A.batch) * A.segments;
  // ---- blocks behind the cached ones: held ones, then new ones ----
  for (int64_t u = warp; u < units; u += warps) {
    const int i = static_cast<int>(u / A.segments), j0 = static_cast<int>(u % A.segments) * kSegment;
    const int4 p = A.plan[i];  // row, held, blocks, len
    if (p.x < 0) continue;
    const int64_t first = A.first[i];
    int32_t* row = A.table + p.x * static_cast<int64_t>(A.table_stride);
    const int end = min(p.z, j0 + kSegment);
    for (int j = max(j0, blocks_of(A, p.w)) + lane; j < end; j += 32) {
      int id;
      if (j < p.y) {
        id = row[j];
      } else {
        const int64_t k = first + (j - p.y);
        id = k < A.n_free ? __ldg(A.free_blocks + k) : -1;
        row[j] = id;
      }
      if (A.block_table != nullptr) A.block_table[i * static_cast<int64_t>(A.bt_stride) + j] = id;
    }
  }
  // ---- tokens ----
  if (static_cast<int64_t>(cta) * kThreads >= A.n_tokens) return;
  const bool near = A.batch <= kSearchEntries;
  if (near) {
    for (int i = threadIdx.x; i <= A.batch; i += kThreads) loc[i] = A.qsl[i];
    __syncthreads();
  }
  const int32_t* q = near ? loc : A.qsl;
  const int total = q[A.batch];
  for (int64_t t = static_cast<int64_t>(cta) * kThreads + threadIdx.x; t < A.n_tokens; t += static_cast<int64_t>(ctas) * kThreads) {
    int64_t pos = 0, slot = -1;
    if (t < total) {
      int lo = 0, hi = A.batch - 1;  // the last entry that begins at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (q[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int4 p = A.plan[lo];
      const unsigned at = static_cast<unsigned>(p.w + (static_cast<int>(t) - q[lo]));
      const int j = static_cast<int>(at / static_cast<unsigned>(A.block_size));
      const int64_t k = A.first[lo] + (j - p.y);
      const bool none = j >= p.y && k >= A.n_free;
      const int id = none ? -1 : j < p.y ? A.table[p.x * static_cast<int64_t>(A.table_stride) + j] : __ldg(A.free_blocks + k);
      pos = at;
      if (id >= 0 && id < A.num_blocks) slot = static_cast<int64_t>(id) * A.block_size + (at - static_cast<unsigned>(j) * A.block_size);
      else if (!none) latch_error(A.err, SMLA_ERR_BAD_INDEX);
    }
    A.positions[t] = pos;
    A.slots[t] = slot;
  }
}

__global__ void __launch_bounds__(kPlanThreads) step_plan_kernel(const TableArgs A) {
  __shared__ int64_t sums[32];
  cudaTriggerProgrammaticLaunchCompletion();
  plan_entries(A, sums);
}

__global__ void __launch_bounds__(kFillThreads) step_fill_kernel(const TableArgs A) {
  extern __shared__ int32_t loc[];
  copy_cached(A, static_cast<int64_t>(blockIdx.x) * (kFillThreads / 32) + (threadIdx.x >> 5), static_cast<int64_t>(gridDim.x) * (kFillThreads / 32));
  cudaGridDependencySynchronize();  // the plan
  fill<kFillThreads>(A, loc, blockIdx.x, gridDim.x);
}

// The whole call as one cluster (the grid): its first CTA plans, the others copy meanwhile.
__global__ void __launch_bounds__(kPlanThreads) step_tables_kernel(const TableArgs A) {
  extern __shared__ int32_t loc[];
  __shared__ int64_t sums[32];
  const int ctas = gridDim.x, copiers = max(ctas - 1, 1), me = ctas > 1 ? static_cast<int>(blockIdx.x) - 1 : 0;
  if (blockIdx.x == 0) plan_entries(A, sums);
  if (me >= 0) copy_cached(A, static_cast<int64_t>(me) * (kPlanThreads / 32) + (threadIdx.x >> 5), static_cast<int64_t>(copiers) * (kPlanThreads / 32));
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  fill<kPlanThreads>(A, loc, blockIdx.x, ctas);
}

// Whether two ranges of bytes share one.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" size_t smla_step_tables_workspace_size(int batch) {
  return batch > 0 ? static_cast<size_t>(batch) * (sizeof(int4) + sizeof(int64_t)) : 0;
}

extern "C" smla_status_t smla_step_tables(const smla_layout_t* layout, const int32_t* rows, const int32_t* lens,
                                          const int32_t* new_lens, int batch, int32_t* table, int64_t n_rows,
                                          int table_stride, const int32_t* held, int32_t* held_out,
                                          const int32_t* free_blocks, int64_t n_free, const int64_t* free_used,
                                          int64_t* free_used_out, int n_tokens, int32_t* seq_lens,
                                          int32_t* query_start_loc, int64_t* positions, int64_t* slot_mapping,
                                          int32_t* block_table, int bt_stride, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  if (!layout_ok(layout) || batch <= 0 || n_rows <= 0 || table_stride <= 0 || n_free < 0 || n_tokens < 0 || !lens ||
      !new_lens || !table || !held || !held_out || (n_free > 0 && !free_blocks) || !free_used || !free_used_out ||
      !seq_lens || !query_start_loc || (n_tokens > 0 && (!positions || !slot_mapping)))
    return SMLA_ERR_INVALID_ARG;
  // without rows entry i is row i; only then can the persistent table stand in for the batch's
  if ((rows == nullptr && batch > n_rows) || (rows != nullptr && block_table == nullptr) ||
      (block_table != nullptr && (bt_stride <= 0 || overlap(table, 4 * n_rows * table_stride, block_table, 4ll * batch * bt_stride))))
    return SMLA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15) != 0 ||
      workspace_bytes < smla_step_tables_workspace_size(batch))
    return SMLA_ERR_INVALID_ARG;
  // lengths are read while their results are written
  const auto over_lengths = [&](const void* to, int64_t n) {
    return overlap(lens, 4 * n_rows, to, 4 * n) || overlap(new_lens, 4ll * batch, to, 4 * n);
  };
  if (over_lengths(seq_lens, batch) || over_lengths(query_start_loc, batch + 1ll) || over_lengths(held_out, n_rows)) return SMLA_ERR_INVALID_ARG;
  TableArgs A{};
  const smla_status_t st = checked_device(&A.err);
  if (st != SMLA_OK) return st;
  A.block_size = layout->block_size;
  A.num_blocks = layout->num_blocks;
  A.rows = rows;
  A.lens = lens;
  A.new_lens = new_lens;
  A.batch = batch;
  A.table = table;
  A.n_rows = n_rows;
  A.table_stride = table_stride;
  A.held = held;
  A.held_out = held_out;
  A.free_blocks = free_blocks;
  A.n_free = n_free;
  A.free_used = free_used;
  A.free_used_out = free_used_out;
  A.n_tokens = n_tokens;
  A.seq_lens = seq_lens;
  A.qsl = query_start_loc;
  A.positions = positions;
  A.slots = slot_mapping;
  A.block_table = block_table;
  A.bt_stride = bt_stride;
  const int width = block_table != nullptr ? std::min(table_stride, bt_stride) : table_stride;
  A.cap = static_cast<int>(std::min(static_cast<int64_t>(width) * layout->block_size, static_cast<int64_t>(kMaxContext)));
  A.segments = (width - 1) / kSegment + 1;
  A.vec = (reinterpret_cast<uintptr_t>(table) & 15) == 0 && table_stride % 4 == 0 &&
          (reinterpret_cast<uintptr_t>(block_table) & 15) == 0 && bt_stride % 4 == 0;
  A.plan = static_cast<int4*>(workspace);
  A.first = reinterpret_cast<int64_t*>(A.plan + batch);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t units = static_cast<int64_t>(batch) * A.segments;
  cudaLaunchConfig_t cfg{};
  cfg.dynamicSmemBytes = batch <= kSearchEntries ? 4 * (static_cast<size_t>(batch) + 1) : 0;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int64_t entries = block_table != nullptr ? static_cast<int64_t>(batch) * width : 0;
  if (entries <= kOneLaunchEntries && n_tokens <= kOneLaunchTokens) {
    // a CTA for every 32 segments (one a warp) or 4,096 tokens
    const int64_t want = std::max((units + 31) / 32 + (units > 32 ? 1 : 0), (static_cast<int64_t>(n_tokens) + 4095) / 4096);
    int ctas = 1;
    while (ctas < want && ctas < kMaxCluster) ctas *= 2;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    return cudaLaunchKernelEx(&cfg, step_tables_kernel, static_cast<const TableArgs>(A)) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
  }
  step_plan_kernel<<<1, kPlanThreads, 0, s>>>(A);
  if (cudaGetLastError() != cudaSuccess) return SMLA_ERR_CUDA;
  const int64_t per = kFillThreads / 32;
  const int64_t want = std::max((units + per - 1) / per, (static_cast<int64_t>(n_tokens) + kFillThreads - 1) / kFillThreads);
  cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(want, 8 * device_sm_count()))));
  cfg.blockDim = dim3(kFillThreads);
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, step_fill_kernel, static_cast<const TableArgs>(A)) == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}
