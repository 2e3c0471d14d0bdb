// What the tensor-core attention kernels over the full latent shape share: the cut of the work into equal ranges of
// key tiles on the device, the units of a range, and the join of the parts that a cut leaves.
//
// Work is counted in tiles of 128 keys.  A worker (a CTA, or a pair of them) takes the range [p total / n,
// (p + 1) total / n) of all units' tiles and walks over the units in it; a unit that crosses ranges leaves partial
// results, which part_merge_kernel joins by their lse.  The cut needs no host plan, so that a captured step follows
// lengths that change.
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "latent4.cuh"
#include "smla_internal.h"

namespace smla {

struct DenseArgs {
  KernelLayout L;
  int n_heads, layer;
  float scale_log2;  // softmax_scale * log2(e)
  const uint8_t* pool;
  const __nv_bfloat16 *q, *q_pe;
  const int32_t *block_table, *seq_lens, *qsl;
  int bt_stride, batch, n_tokens;
  // Positions of a sequence that are visited at most: those of its block-table row, kMaxContext at most.  In 64 bits:
  // compared in 32, the code around came out 1 % slower on a batch of short units (1,023 us against 1,011).
  int64_t most;
  __nv_bfloat16* out;
  float* lse;  // or nullptr
  unsigned* err;
};

// Units of at most 64 rows over E2M1 records of the full shape (attend4.cu).
smla_status_t launch_attend4_dense(const DenseArgs& D, float softmax_scale, void* workspace, size_t workspace_bytes, cudaStream_t s);

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKeys = 128;                        // of a tile
constexpr int kDL = 512, kDR = 64, kChunks = 9;   // the full latent shape; 64-dim chunks: 8 latent, 1 rope
constexpr int kMaxContext = INT_MAX - 1023;  // a tile's rounding up and a range's start stay below 2^31 from there


// The running maximum moves when a score passes it by 2^8: few tiles rescale O (2^12 was no faster).
constexpr float kRescale = 8.0f;
// P is formed 2^7 times as large, 2^15 at most: fp16's last step, 2^-24, is then 2^-31 of a row's largest weight at
// most.  Without it a long tail 17 nats below one position rounded to zeros in P but not in the sum that divides.
constexpr float kLift = 7.0f;
constexpr uint32_t kHalfEnd = 0x4780;  // bf16 of 65536, the first bf16 value that fp16 does not reach

// Positions that the i-th of n_q query tokens of a sequence of len positions sees: len - n_q + i + 1, at least
// none and at most A.most.
__device__ __forceinline__ int64_t visible(const DenseArgs& A, int len, int i, int n_q) {
  const int64_t n = static_cast<int64_t>(len) - n_q + i + 1;
  return n < 0 ? 0 : n < A.most ? n : A.most;
}

// The unit that begins in a worker's range and goes on in the next workers' (ntok = 0: none): its parts are
// slot 2 p + 1 of this worker and slot 2 r of every worker r > p whose range begins before `end`.
struct PartMeta {
  int64_t end, total;  // one past the unit's last tile; all work, divided evenly over `pairs`
  int pairs, tok0, ntok;  // (workers)
};

// sum_{g < n} floor((a g + b) / m), with a n + b and the sums of the descent below 2^32 (Euclid's algorithm
// on the lattice points below a line).
__device__ __noinline__ int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t s = 0;
  while (n > 0) {
    s += static_cast<int64_t>(n - 1) * n / 2 * (a / m) + static_cast<int64_t>(n) * (b / m);
    a %= m;
    b %= m;
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return s;
}

// A unit is `group` query tokens of a sequence (fewer at its end) with the key tiles its last token sees
// (at least one, so that tokens which see nothing are written too).
template <class Args>
__device__ __forceinline__ int unit_tiles(const Args& A, int len, int g, int n_q) {
  const int last = min((g + 1) * A.group, n_q) - 1;
  return max(1, static_cast<int>((visible(A.D, len, last, n_q) + kKeys - 1) / kKeys));
}

// Work of the first g units of a sequence of len positions and n_q query tokens: their tiles and unit_cost more for
// each (the time between two units, in tiles), or their number where units are not split.
template <class Args>
__device__ int64_t work_before(const Args& A, int len, int g, int n_q) {
  if (A.part_out == nullptr) return g;
  const int units = (n_q + A.group - 1) / A.group;
  if (units == 1) return g == 0 ? 0 : unit_tiles(A, len, 0, n_q) + A.unit_cost;
  if (len >= n_q && len <= A.D.most) {
    const int whole = min(g, units - 1);
    int64_t s = floor_sum(whole, kKeys, A.group, len - n_q + A.group + kKeys - 1);
    if (g == units) s += (len + kKeys - 1) / kKeys;
    return s + static_cast<int64_t>(g) * A.unit_cost;
  }
  int64_t s = 0;
  for (int i = 0; i < g; ++i) s += unit_tiles(A, len, i, n_q);
  return s + static_cast<int64_t>(g) * A.unit_cost;
}

// The units of this worker (a CTA, or a pair of them) in turn.  Positions count work from the start of its range: the
// unit's first tile is at `rel`, behind its cost (below zero if an earlier worker began it), and the range ends at `len`.
// A range that ends within a unit's cost has none of its tiles: the next worker begins it.
struct Walk {
  int b, g, q0, n_q, nvis, rel, len, seq_len;
  template <class Args, class Smem>
  __device__ __forceinline__ void start(const Args& A, const Smem& sm) {
    b = sm.b;
    g = sm.g;
    rel = sm.rel + (A.part_out != nullptr ? A.unit_cost : 0);
    len = sm.len;
    q0 = sm.q0;
    n_q = sm.n_q;
    seq_len = sm.seq_len;
    if (on()) unit(A);
  }
  __device__ __forceinline__ bool on() const { return rel < len; }
  template <class Args>
  __device__ __forceinline__ int tok0(const Args& A) const { return q0 + g * A.group; }
  template <class Args>
  __device__ __forceinline__ int ntok(const Args& A) const { return min(A.group, n_q - g * A.group); }
  // Rows of this CTA: the first half of the unit's rows, or the others.
  template <class Args>
  __device__ __forceinline__ int rows_before(const Args& A, int cta) const { return cta * ((ntok(A) * A.D.n_heads + 1) / 2); }
  template <class Args>
  __device__ __forceinline__ int rows(const Args& A, int cta) const {
    const int all = ntok(A) * A.D.n_heads, first = (all + 1) / 2;
    return cta == 0 ? first : all - first;
  }
  __device__ __forceinline__ int tiles() const { return max(1, (nvis + kKeys - 1) / kKeys); }
  // the worker's tiles [ta, tb) of the unit
  template <class Args>
  __device__ __forceinline__ int ta(const Args& A) const { return A.part_out != nullptr ? max(-rel, 0) : 0; }
  template <class Args>
  __device__ __forceinline__ int tb(const Args& A) const {
    return A.part_out != nullptr ? min(tiles(), len - rel) : tiles();
  }
  template <class Args>
  __device__ __forceinline__ void unit(const Args& A) {
    nvis = static_cast<int>(visible(A.D, seq_len, g * A.group + ntok(A) - 1, n_q));
  }
  template <class Args>
  __device__ __forceinline__ void next(const Args& A) {
    rel += A.part_out != nullptr ? tiles() + A.unit_cost : 1;
    if (!on()) return;
    if (++g * A.group >= n_q) {
      g = 0;
      q0 += n_q;
      int end;
      do end = __ldg(A.D.qsl + ++b + 1);
      while (end == q0);
      n_q = end - q0;
      seq_len = __ldg(A.D.seq_lens + b);
    }
    unit(A);
  }
};

// A walk tile by tile.
template <class W>
struct TileWalkOf {
  W w;
  int tile, tb;
  __device__ __forceinline__ bool on() const { return w.on(); }
  template <class Args>
  __device__ __forceinline__ void enter(const Args& A) {
    tile = w.on() ? w.ta(A) : 0;
    tb = w.on() ? w.tb(A) : 0;
  }
  template <class Args, class Smem>
  __device__ __forceinline__ void start(const Args& A, const Smem& sm) {
    w.start(A, sm);
    enter(A);
  }
  template <class Args>
  __device__ __forceinline__ void next(const Args& A) {
    if (!w.on()) return;
    if (++tile >= tb) {
      w.next(A);
      enter(A);
    }
  }
};
using TileWalk = TileWalkOf<Walk>;

// Non-blocking test of a barrier's phase.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// Requests a record into L2, line by line (kBytes from a multiple of 32 on).
template <int kBytes>
__device__ __forceinline__ void prefetch_record(const uint8_t* p) {
#pragma unroll
  for (int i = 0; i < kBytes - 1; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i) : "memory");
  if (kBytes % 128 != 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + kBytes - 1) : "memory");
}
// f(integral_constant 0) .. f(integral_constant N - 1)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// (a, b) * (c, c) + (d, d) and (a, b) + (c, d) as packed fp32 operations
__device__ __forceinline__ float2 fma2(float2 a, float c, float d) {
  uint64_t r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %3};\n\tmov.b64 z, {%4, %4};\n\t"
      "fma.rn.f32x2 %0, x, y, z;\n\t}"
      : "=l"(r)
      : "f"(a.x), "f"(a.y), "f"(c), "f"(d));
  return make_float2(__uint_as_float(static_cast<uint32_t>(r)), __uint_as_float(static_cast<uint32_t>(r >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %2};\n\tmov.b64 y, {%3, %4};\n\tadd.rn.f32x2 %0, x, y;\n\t}"
      : "=l"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return make_float2(__uint_as_float(static_cast<uint32_t>(r)), __uint_as_float(static_cast<uint32_t>(r >> 32)));
}

// Page of position j: j / block_size by multiplication (Granlund and Montgomery's round-up method).
template <class Args>
__device__ __forceinline__ int page_of(const Args& A, int j) {
  const uint32_t t = __umulhi(static_cast<uint32_t>(j), A.pages.mul);
  return static_cast<int>((t + ((static_cast<uint32_t>(j) - t) >> A.pages.shift1)) >> A.pages.shift2);
}

// Constants of page_of for a block size.
struct PageDiv {
  uint32_t mul, shift1, shift2;
};
inline PageDiv page_div(int block_size) {
  uint32_t log2 = 0;
  while ((1ull << log2) < static_cast<uint64_t>(block_size)) ++log2;
  return {static_cast<uint32_t>((((1ull << log2) - block_size) << 32) / block_size + 1), log2 > 0 ? 1u : 0u, log2 > 0 ? log2 - 1 : 0u};
}

// A worker's range of work (`pair` of n_pairs).  Threads take the sequences in turn and a scan over the CTA finds the total and
// the sequence in which the range begins (again from the start if there are more sequences than
// threads); the first warp then looks for the unit.
template <int kThreads, class Args, class Smem>
__device__ __forceinline__ void plan(const Args& A, Smem& sm, int pair, int n_pairs) {
  int64_t* warp_sum = reinterpret_cast<int64_t*>(sm.red);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int batch = A.D.batch;
  int64_t total = -1, x0 = 0, x1 = 0, carry = 0;
#pragma unroll 1
  for (int c0 = 0;;) {
    const int b = c0 + threadIdx.x;
    int64_t mine = 0;
    int q0 = 0, n_q = 0, len = 0;
    if (b < batch) {
      q0 = __ldg(A.D.qsl + b);
      n_q = __ldg(A.D.qsl + b + 1) - q0;
      len = __ldg(A.D.seq_lens + b);
      if (n_q > 0) mine = work_before(A, len, (n_q + A.group - 1) / A.group, n_q);
      if (blockIdx.x == 0 && n_q > 0 && len > A.D.most)
        latch_error(A.D.err, SMLA_ERR_BAD_INDEX);
    }
    int64_t incl = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int64_t lo = carry + incl - mine;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) lo += warp_sum[w];
      carry += warp_sum[w];
    }
    c0 += kThreads;
    if (total < 0 && c0 >= batch) {  // the total is known: the pair's range, and the first sequences again if need be
      total = carry;
      const int64_t P = max(static_cast<int64_t>(1), min(static_cast<int64_t>(n_pairs), A.part_out != nullptr ? total / A.min_tiles : total));
      x0 = pair < P ? pair * total / P : total;
      x1 = pair < P ? (pair + 1) * total / P : total;
      if (threadIdx.x == 0) {
        sm.x0 = x0;
        sm.len = static_cast<int>(x1 - x0);
        sm.total = total;
        sm.pairs = static_cast<int>(P);
        sm.rel = 0;
      }
      if (batch > kThreads) {
        c0 = 0;
        carry = 0;
        continue;
      }
    }
    if (total >= 0) {
      if (x0 < x1 && mine > 0 && lo <= x0 && x0 < lo + mine) {
        sm.b = b;
        sm.seq_at = lo;
        sm.q0 = q0;
        sm.n_q = n_q;
        sm.seq_len = len;
      }
      if (c0 >= batch) break;
    }
  }
  __syncthreads();
  if (warp == 0 && x0 < x1) {
    const int n_q = sm.n_q, len = sm.seq_len;
    const int64_t at = x0 - sm.seq_at;
    int ga = 0, gb = (n_q + A.group - 1) / A.group - 1;  // the last unit that begins at or before the range is in [ga, gb]
#pragma unroll 1
    while (ga < gb) {
      const int step = (gb - ga + 31) / 32, g = ga + (lane + 1) * step;
      const int past = __popc(__ballot_sync(0xffffffffu, g <= gb && work_before(A, len, g, n_q) <= at));
      ga += past * step;
      gb = min(gb, ga + step - 1);
    }
    if (lane == 0) {
      sm.g = ga;
      sm.rel = -static_cast<int>(at - work_before(A, len, ga, n_q));
    }
  }
}

// A lane's part of a query row: 16 latent and 2 rope dims, as nine pairs.
template <class Args>
__device__ __forceinline__ void load_query(const Args& A, int64_t row, int lane, uint32_t (&v)[9]) {
  const __nv_bfloat16* src = A.D.q + row * kDL + 16 * lane;
  const __nv_bfloat16* pe = A.D.q_pe + row * kDR + 2 * lane;
  if (A.q_vec) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(src)), b = __ldg(reinterpret_cast<const uint4*>(src) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    v[8] = __ldg(reinterpret_cast<const uint32_t*>(pe));
  } else {
    const uint16_t* u = reinterpret_cast<const uint16_t*>(src);
    const uint16_t* w = reinterpret_cast<const uint16_t*>(pe);
#pragma unroll
    for (int x = 0; x < 8; ++x) v[x] = u[2 * x] | (static_cast<uint32_t>(u[2 * x + 1]) << 16);
    v[8] = w[0] | (static_cast<uint32_t>(w[1]) << 16);
  }
}

// Lane i of a group of four holds four items of four words; afterwards item j is what lane j held as item i.
__device__ __forceinline__ void transpose4(uint32_t (&o)[16], bool hi1, bool hi2) {
#pragma unroll
  for (int st = 1; st <= 2; st <<= 1) {
    const bool hi = st == 1 ? hi1 : hi2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if ((j & st) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? o[4 * j + i] : o[4 * (j | st) + i], st);
          if (hi) o[4 * j + i] = got;
          else o[4 * (j | st) + i] = got;
        }
      }
    }
  }
}

// Joins the parts of units that ran on several workers: lse = ln sum e^lse_i, out = sum e^(lse_i - lse) out_i
// in fp32.  A warp takes a row (a lane 16 dims) where a few parts are to be joined; where there are many, as
// for one long sequence, the block's four warps share it (a lane 4 dims, eight parts' loads in flight).
// With the whole call's time: one sequence of 262,143 positions 95 us (117 with a warp per row), 64 sequences of
// four tokens 645 us (655 with a block per row).
constexpr int kMergeThreads = 128, kFewParts = 8;
template <int kMax, int kStep>
__device__ __forceinline__ void merge_row(const PartMeta& M, int p, int parts, int row, int slot_rows, int quarter0, int quarters,
                                          const float* part_lse, const float* part_out, int n_heads, __nv_bfloat16* out, float* lse) {
  const int lane = threadIdx.x & 31;
  const auto slot = [&](int i) -> int64_t { return i == 0 ? 2 * p + 1 : 2 * (p + i); };
  float v[kMax / 32], mx = -INFINITY, z = 0.f;
#pragma unroll
  for (int i = 0; i < kMax / 32; ++i) {
    v[i] = 32 * i + lane < parts ? __ldcg(part_lse + slot(32 * i + lane) * slot_rows + row) : -INFINITY;
    mx = fmaxf(mx, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
  for (int i = 0; i < kMax / 32; ++i) {
    v[i] = expf(v[i] - base);  // NaN stays NaN
    z += v[i];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  const float inv = z == 0.f ? 0.f : 1.f / z;
  const int64_t orow = static_cast<int64_t>(M.tok0) * n_heads + row;
#pragma unroll 1
  for (int q = quarter0; q < quarter0 + quarters; q += kStep == 2 ? 4 : 1) {
    constexpr int kQ = kStep == 2 ? 4 : 1;  // quarters at once
    float4 acc[kQ];
#pragma unroll
    for (int y = 0; y < kQ; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += kStep) {
      float4 a[kStep][kQ];
      float f[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int part = min(i0 + i, parts - 1);
        float w = v[0];
#pragma unroll
        for (int x = 1; x < kMax / 32; ++x) w = part >= 32 * x ? v[x] : w;
        f[i] = __shfl_sync(0xffffffffu, w, part & 31) * inv;
        if (i0 + i >= parts) f[i] = 0.f;
#pragma unroll
        for (int y = 0; y < kQ; ++y)
          a[i][y] = __ldcg(reinterpret_cast<const float4*>(part_out + (slot(part) * slot_rows + row) * kDL + 128 * (q + y)) + lane);
      }
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
#pragma unroll
        for (int y = 0; y < kQ; ++y) {
          acc[y].x += f[i] * a[i][y].x;
          acc[y].y += f[i] * a[i][y].y;
          acc[y].z += f[i] * a[i][y].z;
          acc[y].w += f[i] * a[i][y].w;
        }
      }
    }
#pragma unroll
    for (int y = 0; y < kQ; ++y)
      reinterpret_cast<uint2*>(out + orow * kDL + 128 * (q + y))[lane] =
          make_uint2(pack_bf16x2(acc[y].x, acc[y].y), pack_bf16x2(acc[y].z, acc[y].w));
  }
  if (quarter0 == 0 && lane == 0 && lse != nullptr) lse[orow] = z == 0.f ? -INFINITY : mx + logf(z);
}

// Starts while the workers still write what it reads.  So the reads come after its wait for them, are ordinary ones
// and not of the read-only path, which stands for data that no one writes while the kernel lives, and no pointer
// is marked as free of aliases, so that none of them moves before the wait.
template <int kMax>
__global__ void __launch_bounds__(kMergeThreads) part_merge_kernel(const PartMeta* meta, const float* part_lse,
                                                                   const float* part_out, int n_pairs, int slot_rows, int n_heads,
                                                                   __nv_bfloat16* out, float* lse) {
  constexpr int kPer = (kMax + 31) / 32;  // workers of a lane of the first warp
  __shared__ int cum[32 * kPer + 1];  // rows to join of the workers before p
  const int tid = threadIdx.x, warp = tid >> 5;
  cudaGridDependencySynchronize();
  if (warp == 0) {
    int v[kPer], sum = 0;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      v[x] = kPer * tid + x < n_pairs ? meta[kPer * tid + x].ntok * n_heads : 0;
      sum += v[x];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += y;
    }
    int at = incl - sum;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      cum[kPer * tid + x] = at;
      at += v[x];
    }
    if (tid == 31) cum[32 * kPer] = at;
  }
  __syncthreads();
  const int total = cum[32 * kPer];
  const auto join = [&](int item, bool few) {
    int p = 0, hi = n_pairs - 1;
    while (p < hi) {
      const int mid = (p + hi + 1) / 2;
      if (cum[mid] <= item) p = mid;
      else hi = mid - 1;
    }
    const PartMeta M = meta[p];
    // pairs p + 1 .. carry the rest: range r begins at floor(r total / pairs), before the unit's end for
    // r < end pairs / total
    const int n = static_cast<int>(min((M.end * M.pairs + M.total - 1) / M.total, static_cast<int64_t>(M.pairs))) - p;
    if (few && n <= kFewParts) merge_row<kMax, 2>(M, p, n, item - cum[p], slot_rows, 0, 4, part_lse, part_out, n_heads, out, lse);
    if (!few && n > kFewParts) merge_row<kMax, 8>(M, p, n, item - cum[p], slot_rows, warp, 1, part_lse, part_out, n_heads, out, lse);
  };
#pragma unroll 1
  for (int item = 4 * blockIdx.x + warp; item < total; item += 4 * gridDim.x) join(item, true);
#pragma unroll 1
  for (int item = blockIdx.x; item < total; item += gridDim.x) join(item, false);
}

// Launched while the workers still work (its blocks wait for their results before they read).
template <int kMax>
smla_status_t launch_part_merge(const PartMeta* meta, const float* part_lse, const float* part_out, int workers, int slot_rows,
                                int n_heads, __nv_bfloat16* out, float* lse, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(6 * device_sm_count());
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, part_merge_kernel<kMax>, meta, part_lse, part_out, workers, slot_rows, n_heads, out, lse) == cudaSuccess
             ? SMLA_OK
             : SMLA_ERR_CUDA;
}

}  // namespace
}  // namespace smla
