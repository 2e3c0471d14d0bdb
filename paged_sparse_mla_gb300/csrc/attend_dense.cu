// smla_attend_dense: latent MQA attention of each query token over its whole visible context.
//
// [AgentX "Kimi K3"], [GLM-5.3 "What is new"]: MLA keeps one latent KV shared by all query heads, so
// attention is MQA over the latent; V is the latent.  [GLM-5.3 "How to try"]: a prompt that fits the
// top-k attends over all of its positions; here that holds at any length.
//
//   s_j = softmax_scale (q . K_j + q_pe . kpe_j),  m = max_j s_j,  l = sum_j e^(s_j - m)
//   out = sum_j e^(s_j - m) K_j / l,  lse = m + ln l            over the positions j that the token sees
// in one pass over the keys: m and l are running values, and what is summed so far is multiplied by
// e^(m_old - m_new) when m moves.  Exponentials are powers of two (the scale carries log2 e).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "smla_internal.h"

namespace smla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxHeads = 128;
constexpr int kMaxContext = INT_MAX - 1023;  // a tile's rounding up and a range's start stay below 2^31 from there

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

// Positions that the i-th of n_q query tokens of a sequence of len positions sees: len - n_q + i + 1, at least
// none and at most A.most.
__device__ __forceinline__ int64_t visible(const DenseArgs& A, int len, int i, int n_q) {
  const int64_t n = static_cast<int64_t>(len) - n_q + i + 1;
  return n < 0 ? 0 : n < A.most ? n : A.most;
}

// ---------------------------------------------------------------------------
// Shapes without a tensor-core kernel: fp32 throughout.  One CTA per (query token, 8 heads); keys in
// tiles of 32, dequantised into shared memory; warp h scores head h (a lane per key), then every
// thread accumulates its dims for the 8 heads.  Bound by shared-memory reads, one per multiply-add: on the
// full shape, which has its own kernel, it took 33.6 ms where that takes 0.19 (32 tokens, 64 heads,
// 8,192 to 32,768 positions each).
// ---------------------------------------------------------------------------
constexpr int kSHeads = 8, kSKeys = 32, kSThreads = 256;

__global__ void __launch_bounds__(kSThreads) dense_fp32_kernel(const DenseArgs A) {
  extern __shared__ float dense_smem[];
  const KernelLayout& L = A.L;
  const int DL = L.d_latent, D = DL + L.d_rope, DP = D + 1;  // odd row stride: a lane per key reads without conflicts
  float* q = dense_smem;             // [8][D]
  float* k = q + kSHeads * D;        // [32][DP]
  float* p = k + kSKeys * DP;        // [8][32]
  float* alpha = p + kSHeads * kSKeys;  // [8]
  float* inv_l = alpha + kSHeads;       // [8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x, h0 = blockIdx.y * kSHeads;
  if (t >= __ldg(A.qsl + A.batch)) return;  // behind the last sequence: left as it was
  const int b = seq_of_token(A.qsl, A.batch, t);
  const int q0 = __ldg(A.qsl + b), n_q = __ldg(A.qsl + b + 1) - q0;
  const int64_t n = visible(A, __ldg(A.seq_lens + b), t - q0, n_q);
  if (threadIdx.x == 0 && __ldg(A.seq_lens + b) > A.most)
    latch_error(A.err, SMLA_ERR_BAD_INDEX);
  for (int u = threadIdx.x; u < kSHeads * D; u += kSThreads) {
    const int h = h0 + u / D, d = u % D;
    float v = 0.f;
    if (h < A.n_heads)
      v = __bfloat162float(d < DL ? A.q[(static_cast<int64_t>(t) * A.n_heads + h) * DL + d]
                                  : A.q_pe[(static_cast<int64_t>(t) * A.n_heads + h) * L.d_rope + d - DL]);
    q[u] = v;
  }
  float acc[2][kSHeads] = {};  // dims threadIdx.x and threadIdx.x + 256
  float m = -INFINITY, l = 0.f;  // of head `warp`
  const int32_t* bt = A.block_table + static_cast<int64_t>(b) * A.bt_stride;
  for (int64_t j0 = 0; j0 < n; j0 += kSKeys) {
    __syncthreads();
    for (int i = warp; i < kSKeys; i += kSThreads / 32) {
      const int64_t j = j0 + i;
      const uint8_t* rec = nullptr;
      if (j < n) {
        const int blk = __ldg(bt + j / L.block_size);
        if (blk >= 0 && blk < L.num_blocks)
          rec = A.pool + blk * L.block_stride + static_cast<int64_t>(A.layer) * L.layer_stride + L.rec_off +
                (j % L.block_size) * L.rec_stride;
        else if (lane == 0)
          latch_error(A.err, SMLA_ERR_BAD_INDEX);
      }
      for (int d = lane; d < D; d += 32) {
        float v = 0.f;
        if (rec != nullptr) {
          if (d < DL) {
            const __half_raw hr = __nv_cvt_fp8_to_halfraw(rec[d], __NV_E4M3);
            v = __half2float(*reinterpret_cast<const __half*>(&hr)) *
                reinterpret_cast<const float*>(rec + DL)[d / L.quant_tile];
          } else {
            v = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(rec + DL + 4 * L.n_scales)[d - DL]);
          }
        }
        k[i * DP + d] = v;
      }
    }
    __syncthreads();
    float s = 0.f;
    for (int d = 0; d < D; ++d) s += q[warp * D + d] * k[lane * DP + d];
    s = j0 + lane < n ? s * A.scale_log2 : -INFINITY;
    float mt = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    const float mn = fmaxf(m, mt);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float e = s == -INFINITY ? 0.f : exp2f(s - mn);
    float sum = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * a + sum;
    m = mn;
    p[warp * kSKeys + lane] = e;
    if (lane == 0) alpha[warp] = a;
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int d = threadIdx.x + x * kSThreads;
      if (d < DL) {
#pragma unroll
        for (int h = 0; h < kSHeads; ++h) acc[x][h] *= alpha[h];
        for (int i = 0; i < kSKeys && j0 + i < n; ++i) {
          const float v = k[i * DP + d];
#pragma unroll
          for (int h = 0; h < kSHeads; ++h) acc[x][h] += p[h * kSKeys + i] * v;
        }
      }
    }
  }
  if (lane == 0) {
    inv_l[warp] = l > 0.f || l != l ? 1.f / l : 0.f;  // no visible position: out = 0, lse = -inf
    if (A.lse != nullptr && h0 + warp < A.n_heads)
      A.lse[static_cast<int64_t>(t) * A.n_heads + h0 + warp] = n > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int d = threadIdx.x + x * kSThreads;
    if (d < DL)
#pragma unroll
      for (int h = 0; h < kSHeads; ++h)
        if (h0 + h < A.n_heads)
          A.out[(static_cast<int64_t>(t) * A.n_heads + h0 + h) * DL + d] = __float2bfloat16_rn(acc[x][h] * inv_l[h]);
  }
}

smla_status_t launch_dense_fp32(const DenseArgs& A, cudaStream_t s) {
  const int D = A.L.d_latent + A.L.d_rope;
  const size_t smem = sizeof(float) * (kSHeads * D + kSKeys * (D + 1) + kSHeads * kSKeys + 2 * kSHeads);
  static std::atomic<bool> attr_set[kMaxDeviceSlots] = {};
  const int dev = current_device_index();
  if (dev < 0) return SMLA_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(dense_fp32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024) != cudaSuccess)
      return SMLA_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  dense_fp32_kernel<<<dim3(A.n_tokens, (A.n_heads + kSHeads - 1) / kSHeads), kSThreads, smem, s>>>(A);
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}


// ---------------------------------------------------------------------------
// The full latent shape (512 latent dims in tiles of 128, 64 rope dims) on the tensor cores.
//
// A cluster of two CTAs (a pair) works on 128 rows, a row being one (query token, head) of one
// sequence, and on tiles of 128 keys; each CTA owns 64 of the rows and 64 of the keys:
//   S[128 x 128] = Q[128 x 576] . K^T      two-SM MMAs, M = 128, N = 128: each CTA brings its 64 query
//                                          rows and its 64 keys
//   P = 2^(S f - m + 7), row sums in registers  each CTA for its 64 rows and all 128 keys
//   O[128 x 512] += P[128 x 128] . V        two-SM MMAs, M = 128, N = 256, twice: each CTA brings its 64
//                                          rows of P and all 128 keys of its 256 latent dims
// An M = 128 two-SM accumulator keeps a CTA's 64 rows in 128 lanes: lanes 0-63 hold the first half of
// the columns, lanes 64-127 the second.  So O (64 rows x 512 dims in fp32) takes 256 tensor-memory
// columns of each CTA, which leaves room for two score buffers; with one SM per 128 rows it would
// fill all 512.
//
// K and V are the same latents, but a CTA needs 64 keys x 512 dims of them as K and 128 keys x 256 dims
// as V, and one MMA reads the same addresses in both CTAs.  So a tile buffer holds the CTA's own keys
// in eight 64-dim chunks (and the rope in a ninth), and once S is formed, the half of the chunks that
// the CTA does not need as V makes room for the other CTA's keys: in the first CTA chunks 0-3 are
// already V's keys 0-63 of its dims 0-255 and chunks 4-7 are refilled with keys 64-127 of the same
// dims; in the second, chunks 4-7 are keys 64-127 of dims 256-511 and chunks 0-3 are refilled with
// keys 0-63 of those.  The rope chunk, free then too, takes the first half of P.  That leaves shared
// memory for two tile buffers beside the queries.
//
// Operands are fp16, not bf16: an E4M3 code is exact in it, so that a key carries the rounding of its scale
// and of the product (2^-11 each; bf16 2^-8), P that of 2^-11 (see kLift for its smallest values).  What fp16
// lacks in range is met by a power of two per query row and checked for keys (SMLA_ERR_RANGE).  Sums, maxima
// and O are fp32.
//
// Warps: eight take the softmax of the CTA's rows, its queries and results; eight turn the CTA's keys into K,
// eight the other CTA's into V; one lane of one warp issues all MMAs of the pair, another warp asks for
// keys and queries to come into L2, a third looks for NaN where it would spread.  The grid is one pair
// per two SMs.  All work, counted in key tiles, is cut into as many equal ranges: a pair walks over the
// units (sequence, group of query tokens) of its range, and a unit that crosses ranges leaves partial
// results, which dense_merge_kernel joins by their lse.
//
// Bound by the shared-memory and L1 data path.  A tile moves, per SM, 240 KB of MMA operands, 120 KB of
// stores of converted keys and 59 KB of record loads through it (1.9 us with records from L2), against
// 1.2 us of MMA at full rate.  With loads that always hit L1 (a wrong answer) the cases below took 8 to
// 18 % less, the largest share of any one part.  The second limit is the instruction cache, which five roles
// share: one copy of every part of the loops took 5 to 7 % off.  Measured, 64 heads:
//   2,048 query tokens, 18,432 positions     3.96 ms, 1.25 PFLOP/s (tensor pipe active half of the time)
//   32 decode tokens, 8,192 to 32,768        188 us, 2.3 TB/s (half of a pair's rows are empty, and
//                                            DRAM's latency adds a sixth)
//   64 x 4 drafted tokens, 4,096 to 32,768   646 us, 1.02 PFLOP/s
//   5 ragged chunks on short contexts        1.01 ms, 0.73 PFLOP/s at 128 heads (the cut, see launch_dense_pair)
//   one token at one position                15 us, the chain plan -> queries -> tile -> results -> merge
// ---------------------------------------------------------------------------
constexpr int kRows = 128, kKeys = 128;      // of a pair
constexpr int kCtaRows = 64, kCtaKeys = 64;  // of a CTA
constexpr int kDL = 512, kDR = 64, kChunks = 9;  // 64-dim chunks: 8 latent, 1 rope
constexpr int kSoftmaxWarps = 8, kKWarps = 8, kVWarps = 8;
constexpr int kKeysPerK = kCtaKeys / kKWarps, kKeysPerV = kCtaKeys / kVWarps;  // of a warp, in a tile
constexpr int kFirstK = kSoftmaxWarps, kFirstV = kFirstK + kKWarps, kIssuer = kFirstV + kVWarps;
constexpr int kThreads = 32 * (kIssuer + 4);  // the last four: issuer, L2 requests, check for NaN, none
constexpr int kLaunchRegs = 72, kSoftmaxRegs = 104, kKRegs = 72, kVRegs = 48, kIssuerRegs = 56;
static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kKWarps * kKRegs + kVWarps * kVRegs + 4 * kIssuerRegs) <=
                  kThreads * kLaunchRegs,
              "register split exceeds the launch");
// The running maximum moves when a score passes it by 2^8: few tiles rescale O (2^12 was no faster).
constexpr float kRescale = 8.0f;
// P is formed 2^7 times as large, 2^15 at most: fp16's last step, 2^-24, is then 2^-31 of a row's largest weight at
// most.  Without it a long tail 17 nats below one position rounded to zeros in P but not in the sum that divides.
constexpr float kLift = 7.0f;
// A scale rounds to fp16 before it multiplies: 146.125 is the last value whose product with code 448 stays finite
// (65,464; 146.25 gives 65,520, which rounds to infinity), and from half way between them a scale rounds up.
constexpr float kScaleEnd = 146.1875f;
constexpr uint32_t kHalfEnd = 0x4780;  // bf16 of 65536, the first bf16 value that fp16 does not reach
// Below 2^-13 a scale would lose bits in fp16 (from 2^-14 on).  Such a scale is taken times 2^19, which keeps its
// products (at most 448 x 2^6) in range, and what was stored is multiplied by 2^-19 in a second pass: exact down to
// fp16's smallest normal value, within half its step (2^-25) below.  A second pass over the few tiles that need
// it and not a second form of the loop: the loop's code shares the instruction cache with the other warps'.
constexpr float kSmallScale = 1.220703125e-4f, kSmallUp = 524288.f;
constexpr int kMaxPairs = 128;
constexpr int kRec = kDL + 16 + 2 * kDR;  // bytes of a record: codes, four scales, rope
constexpr int kMinTiles = 2;  // key tiles a pair takes at least (1 to 4: the same)
// Tiles requested into L2 ahead of the loads (1 to 16: the same; none: decode steps 2 % slower, a chunk 1 %).
constexpr int kPrefetchAhead = 4;

struct __align__(1024) PairSmem {
  uint8_t kv[2][kChunks][kCtaKeys * 128];  // tile buffer, chunk: [64 keys][64 dims] fp16, 128-byte swizzle; see above
  uint8_t q[kChunks][kCtaRows * 128];
  uint8_t p1[kCtaRows * 128];              // P [64 rows][64 keys], keys 64-127 of a tile (keys 0-63: its rope chunk)
  float red[4][kCtaRows];
  float row_f[2][kCtaRows];            // per unit (alternating): |softmax_scale| log2(e) / the row's query factor
  uint64_t k_full[2][2], v_full[2], p_full[2], q_full, s_free[2];  // used in the first CTA; both CTAs arrive (K: by halves)
  uint64_t s_full[2], kv_free[2][2];  // completed by the MMAs in both CTAs (tile buffer: chunks 0-3, then all)
  uint64_t final_bar;
  int64_t x0, total, seq_at;           // start of the pair's range of work; all work, over `pairs` pairs; (plan)
  int pairs, b, g, rel, len, q0, n_q, seq_len;  // the range's first unit, its position (see Walk) and sequence
  int abort;
  uint32_t tmem_slot;
  uint32_t k_loaded;                   // tiles whose keys the first K warp has asked for
};
constexpr size_t kPairSmemBytes = sizeof(PairSmem) + 1024;
static_assert(kPairSmemBytes <= 232448, "shared memory");

// The unit that begins in a pair's range and goes on in the next pairs' (ntok = 0: none): its parts are
// slot 2 p + 1 of this pair and slot 2 r of every pair r > p whose range begins before `end`.
struct PairMeta {
  int64_t end, total;  // one past the unit's last tile; all work, divided evenly over `pairs`
  int pairs, tok0, ntok;
};

struct PairArgs {
  DenseArgs D;
  int group;        // query tokens of a unit: as many as fit 128 rows
  float abs_scale;  // |softmax_scale| log2(e)
  float sign;       // of softmax_scale, applied to the queries
  bool q_vec;       // q and q_pe are 16-byte aligned
  float *part_out, *part_lse;  // partial results, slots [2 pairs][128 rows]; nullptr: units are not split
  PairMeta* meta;   // [pairs]
  const uint8_t* records;               // the layer's records in block 0
  uint32_t bs_mul, bs_shift1, bs_shift2;  // division by block_size
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
__device__ __forceinline__ int unit_tiles(const PairArgs& A, int len, int g, int n_q) {
  const int last = min((g + 1) * A.group, n_q) - 1;
  return max(1, static_cast<int>((visible(A.D, len, last, n_q) + kKeys - 1) / kKeys));
}

// Work of the first g units of a sequence of len positions and n_q query tokens: their tiles, or their
// number where units are not split.
__device__ int64_t work_before(const PairArgs& A, int len, int g, int n_q) {
  if (A.part_out == nullptr) return g;
  const int units = (n_q + A.group - 1) / A.group;
  if (units == 1) return g == 0 ? 0 : unit_tiles(A, len, 0, n_q);
  if (len >= n_q && len <= A.D.most) {
    const int whole = min(g, units - 1);
    int64_t s = floor_sum(whole, kKeys, A.group, len - n_q + A.group + kKeys - 1);
    if (g == units) s += (len + kKeys - 1) / kKeys;
    return s;
  }
  int64_t s = 0;
  for (int i = 0; i < g; ++i) s += unit_tiles(A, len, i, n_q);
  return s;
}

// The units of this pair in turn.  Positions count tiles from the start of the pair's range: the unit
// begins at `rel` (below zero if an earlier pair began it) and the range ends at `len`.
struct Walk {
  int b, g, q0, n_q, nvis, rel, len, seq_len;
  __device__ __forceinline__ void start(const PairArgs& A, const PairSmem& sm) {
    b = sm.b;
    g = sm.g;
    rel = sm.rel;
    len = sm.len;
    q0 = sm.q0;
    n_q = sm.n_q;
    seq_len = sm.seq_len;
    if (on()) unit(A);
  }
  __device__ __forceinline__ bool on() const { return rel < len; }
  __device__ __forceinline__ int tok0(const PairArgs& A) const { return q0 + g * A.group; }
  __device__ __forceinline__ int ntok(const PairArgs& A) const { return min(A.group, n_q - g * A.group); }
  // Rows of this CTA: the first half of the unit's rows, or the others.
  __device__ __forceinline__ int rows_before(const PairArgs& A, int cta) const { return cta * ((ntok(A) * A.D.n_heads + 1) / 2); }
  __device__ __forceinline__ int rows(const PairArgs& A, int cta) const {
    const int all = ntok(A) * A.D.n_heads, first = (all + 1) / 2;
    return cta == 0 ? first : all - first;
  }
  __device__ __forceinline__ int tiles() const { return max(1, (nvis + kKeys - 1) / kKeys); }
  // the pair's tiles [ta, tb) of the unit
  __device__ __forceinline__ int ta(const PairArgs& A) const { return A.part_out != nullptr ? max(-rel, 0) : 0; }
  __device__ __forceinline__ int tb(const PairArgs& A) const {
    return A.part_out != nullptr ? min(tiles(), len - rel) : tiles();
  }
  __device__ __forceinline__ void unit(const PairArgs& A) {
    nvis = static_cast<int>(visible(A.D, seq_len, g * A.group + ntok(A) - 1, n_q));
  }
  __device__ __forceinline__ void next(const PairArgs& A) {
    rel += A.part_out != nullptr ? tiles() : 1;
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
struct TileWalk {
  Walk w;
  int tile, tb;
  __device__ __forceinline__ bool on() const { return w.on(); }
  __device__ __forceinline__ void enter(const PairArgs& A) {
    tile = w.on() ? w.ta(A) : 0;
    tb = w.on() ? w.tb(A) : 0;
  }
  __device__ __forceinline__ void start(const PairArgs& A, const PairSmem& sm) {
    w.start(A, sm);
    enter(A);
  }
  __device__ __forceinline__ void next(const PairArgs& A) {
    if (!w.on()) return;
    if (++tile >= tb) {
      w.next(A);
      enter(A);
    }
  }
};

// ---- cluster and two-SM instructions ----
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrive on a barrier of another (or this) CTA of the pair; the address comes from map_cta.  What the
// arrival hands over is this CTA's own shared memory, already made visible to the MMAs by the proxy
// fence before it, or tensor memory that has been read: no thread of the other CTA reads it, so the
// release need not reach past this CTA.  (A release at cluster scope waits for every outstanding load
// of the thread: it took 1,500 to 2,000 cycles of each hand-off.)
__device__ __forceinline__ void arrive_cluster(uint32_t mapped) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(mapped) : "memory");
}
// Ends the work of both CTAs; `timeout`: because a wait gave up.
__device__ __forceinline__ void raise_abort(unsigned* err, int* abort, bool timeout) {
  if (timeout) latch_error(err, SMLA_ERR_TIMEOUT);
  for (uint32_t r = 0; r < 2; ++r)
    asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(map_cta(smem_u32(abort), r)) : "memory");
}
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
// Bounded wait as mbar_wait; a wait that gives up raises the abort flag of both CTAs.
__device__ __forceinline__ bool pair_wait(uint64_t* bar, uint32_t parity, unsigned* err, int* abort) {
  const uint32_t addr = smem_u32(bar);
  volatile int* flag = abort;
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(addr, parity)) return true;
    if ((i & 15u) == 15u) {
      if (*flag) return false;
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > kWaitLimitNs) {
        raise_abort(err, abort, true);
        return false;
      }
    }
  }
}
__device__ __forceinline__ void pair_drain(uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(addr, parity) && globaltimer_ns() - t0 <= kWaitLimitNs) {
  }
}
// D (+)= A . B over both CTAs, issued by the lane whose `elected` is set; the whole warp comes here, so
// that the operands live in uniform registers (issued from a branch of one lane, each instruction moved
// them there again and took about 60 cycles whatever its size).  The operands move by constant byte
// offsets from a descriptor's low word (its address field counts 16 bytes); the loops around are short,
// since this warp shares the instruction cache with 27 others (all 36 products of a tile unrolled were
// issued at 65 cycles each).
template <int kAOff, int kBOff>
__device__ __forceinline__ void mma2_f16(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                         uint32_t idesc, uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "add.u32 x, %1, %7;\n\tadd.u32 y, %3, %8;\n\t"
      "mov.b64 a, {x, %2};\n\tmov.b64 b, {y, %4};\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %9, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "n"(kAOff >> 4), "n"(kBOff >> 4),
      "r"(elected)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// f(integral_constant 0) .. f(integral_constant N - 1)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unrolled<N, I + 1>(f);
  }
}
// Arrive on `bar` of both CTAs when every MMA issued so far by the elected lane has completed.
__device__ __forceinline__ void commit2(uint64_t* bar, uint32_t elected) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3)), "r"(elected)
      : "memory");
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

// Eight E4M3 codes times a scale as fp16.  The codes are exact in fp16; the scale (two halves) rounds to 11
// bits and the product once more (2 x 2^-11 in all).
__device__ __forceinline__ uint4 dequant8(const uint2& codes, uint32_t sc) {
  uint32_t o[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t w = x < 2 ? codes.x : codes.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * (x & 1))), __NV_E4M3);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h), *reinterpret_cast<const __half2*>(&sc));
    o[x] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Eight stored values of a key with a small scale, times 2^-19 (see kSmallScale).
__device__ __forceinline__ void shrink8(uint8_t* p) {
  uint32_t* w = reinterpret_cast<uint32_t*>(p);
  const uint32_t k = 0x00200020u;  // 2^-19 twice
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(w + x), *reinterpret_cast<const __half2*>(&k));
    w[x] = *reinterpret_cast<const uint32_t*>(&y);
  }
}
__device__ __forceinline__ bool small_scale(float s) { return fabsf(s) < kSmallScale && s != 0.f; }

// What unreadable records read as (bad block ids, and nothing left to read): 16 records of zeros.
__device__ uint4 g_zero_records[16 * 41];

// Page of position j: j / block_size by multiplication (Granlund and Montgomery's round-up method).
__device__ __forceinline__ int page_of(const PairArgs& A, int j) {
  const uint32_t t = __umulhi(static_cast<uint32_t>(j), A.bs_mul);
  return static_cast<int>((t + ((static_cast<uint32_t>(j) - t) >> A.bs_shift1)) >> A.bs_shift2);
}

// Record of a page's token `off`, in 64 bits: a page may hold more than 2^31 bytes of records.
__device__ __forceinline__ const uint8_t* record(const PairArgs& A, int blk, int off) {
  return A.records + static_cast<int64_t>(blk) * A.D.L.block_stride + static_cast<int64_t>(off) * kRec;
}

// The records of kN consecutive positions from a multiple of kN on.  kRuns: the block size is a multiple
// of 16, so that they lie one after another in a block and every lane knows them all from the first
// (`n` of them hold visible positions; what follows in the block is read too and zeroed by the caller).
// Otherwise lane i looks up the i-th and the lanes pass the addresses around, two shuffles a record: on blocks of
// 64 that takes 3 % longer in decode steps (194 us against 188) and 5 % in a chunk (4.11 ms against 3.89).
// find() asks for the block id, take() turns it into the address: a tile later, so that nothing waits for
// the block table.
template <bool kRuns, int kN>
struct Records {
  const uint8_t* at;
  int blk, off, n;  // blk = INT_MIN: past the visible positions; off: token of the page
  __device__ __forceinline__ void find(const PairArgs& A, const TileWalk& tw, int key0, int lane) {
    blk = INT_MIN;
    if (!tw.on()) return;
    const int j = tw.tile * kKeys + key0 + (kRuns ? 0 : lane & (kN - 1));
    if (j >= tw.w.nvis) return;
    const int pg = page_of(A, j);
    off = j - pg * A.D.L.block_size;
    n = kRuns ? min(tw.w.nvis - j, kN) : kN;
    blk = max(__ldg(A.D.block_table + static_cast<int64_t>(tw.w.b) * A.D.bt_stride + pg), -1);
  }
  // returns how many of the records hold visible positions
  __device__ __forceinline__ int take(const PairArgs& A) {
    at = reinterpret_cast<const uint8_t*>(g_zero_records);
    if (blk == INT_MIN) return kN;
    if (blk < 0 || blk >= A.D.L.num_blocks) {
      latch_error(A.D.err, SMLA_ERR_BAD_INDEX);
      return kN;
    }
    at = record(A, blk, off);
    return n;
  }
  __device__ __forceinline__ const uint8_t* get(int i) const {
    if constexpr (kRuns) return at + i * kRec;
    return reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(at), i));
  }
};

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

// The pair's range of work.  Threads take the sequences in turn and a scan over the CTA finds the total and
// the sequence in which the range begins (again from the start if there are more sequences than
// threads); the first warp then looks for the unit.
__device__ __forceinline__ void plan(const PairArgs& A, PairSmem& sm, int pair, int n_pairs) {
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
      const int64_t P = max(static_cast<int64_t>(1), min(static_cast<int64_t>(n_pairs), A.part_out != nullptr ? total / kMinTiles : total));
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
__device__ __forceinline__ void load_query(const PairArgs& A, int64_t row, int lane, uint32_t (&v)[9]) {
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

template <bool kRuns>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) dense_pair_kernel(const PairArgs A) {
  extern __shared__ uint8_t smem_raw[];
  PairSmem& sm = *reinterpret_cast<PairSmem*>(
      smem_raw + ((1024u - (static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)) & 1023u)) & 1023u));
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform to the compiler
  const uint32_t cta = cluster_rank();
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  unsigned* err = A.D.err;
  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 2 * kSoftmaxWarps);
    mbar_init(&sm.final_bar, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i][0], 2 * kKWarps);
      mbar_init(&sm.k_full[i][1], 2 * kKWarps);
      mbar_init(&sm.v_full[i], 2 * kVWarps);
      mbar_init(&sm.p_full[i], 2 * kSoftmaxWarps);
      mbar_init(&sm.kv_free[i][0], 1);
      mbar_init(&sm.kv_free[i][1], 1);
      mbar_init(&sm.s_free[i], 2 * kSoftmaxWarps);
      mbar_init(&sm.s_full[i], 1);
    }
    sm.abort = 0;
    sm.k_loaded = 0;
    mbar_fence_init();
  }
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  cudaTriggerProgrammaticLaunchCompletion();  // the merge may be launched; it waits for this grid's end
  plan(A, sm, pair, n_pairs);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either arrives on the other's
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem_slot, 0);
  const uint32_t tmem_o = tmem, tmem_s = tmem + 256;

  if (warp >= kIssuer) {
    // ------------------------------ MMA issuer (one warp of the first CTA) ------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssuerRegs));
    if (warp == kIssuer && cta == 0) {
      const uint32_t elected = elect_one();
      const uint32_t idesc1 = make_idesc(128, kKeys, 0, 0, 0, 0);  // fp16, both K-major
      const uint32_t idesc2 = make_idesc(128, 256, 0, 0, 0, 1);    // fp16, P K-major, V MN-major
      constexpr int kChunk = kCtaKeys * 128, kTileBytes = kChunks * kChunk;
      const uint64_t dq = sw128_desc(smem_u32(sm.q[0]), 16, 1024), dk = sw128_desc(smem_u32(sm.kv[0][0]), 16, 1024);
      const uint64_t dp = sw128_desc(smem_u32(sm.p1), 16, 1024), dv = sw128_desc(smem_u32(sm.kv[0][0]), kChunk, 1024);
      const uint32_t dq_lo = static_cast<uint32_t>(dq), dk_lo = static_cast<uint32_t>(dk), dp_lo = static_cast<uint32_t>(dp), dv_lo = static_cast<uint32_t>(dv);
      const uint32_t dk_hi = static_cast<uint32_t>(dk >> 32), dv_hi = static_cast<uint32_t>(dv >> 32);  // Q and P as K
      uint32_t k1 = 0, k2 = 0, n = 0;  // MMA1s and MMA2s issued, units begun
      const auto ready = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_test(bar, parity));
      };
      // S = Q . K^T of tile k1 into score buffer k1 % 2: its dims 0-255, then the others
      const auto mma1 = [&](int part) {
        const uint32_t buf = k1 & 1;
        const int end = part == 0 ? 4 : kChunks;
        tc_fence_after();
#pragma unroll 1
        for (int c = 4 * part; c < end; ++c)
          unrolled<4>([&](auto x) {
            mma2_f16<x() * 32, x() * 32>(tmem_s + buf * 64, dq_lo + c * (kChunk >> 4), dk_hi,
                                         dk_lo + (buf * kTileBytes + c * kChunk) / 16, dk_hi, idesc1, (c | x()) != 0, elected);
          });
        if (part == 0) return;
        commit2(&sm.s_full[buf], elected);
        ++k1;
      };
      // O (+)= P . V of tile k2
      const auto mma2 = [&](bool first) {
        const uint32_t buf = k2 & 1;
        tc_fence_after();
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // keys 0-63 and 64-127
          const uint32_t p = h == 0 ? dk_lo + (buf * kTileBytes + 8 * kChunk) / 16 : dp_lo;
          unrolled<8>([&](auto i) {
            constexpr int x = i() / 2, j = i() % 2;
            mma2_f16<x * 32, 2 * j * kChunk + x * 2048>(tmem_o + j * 128, p, dk_hi, dv_lo + (buf * kTileBytes + 4 * h * kChunk) / 16,
                                                         dv_hi, idesc2, !(first && (h | x) == 0), elected);
          });
          commit2(&sm.kv_free[buf][h], elected);
        }
        ++k2;
      };
      Walk w;
      bool ok = true;
      for (w.start(A, sm); w.on() && ok; w.next(A), ++n) {
        ok = __all_sync(0xffffffffu, pair_wait(&sm.q_full, n & 1, err, &sm.abort));
        const uint32_t begin = k1, end = begin + w.tb(A) - w.ta(A);
        // Whichever is ready: P . V of the oldest tile with written probabilities (it frees the tile
        // buffer), else the next tile's scores (so that they are formed while the softmax works).
        uint64_t t0 = 0;
        int half = 0;  // of tile k1's scores
        for (uint32_t idle = 0; ok && k2 < end;) {
          if (k2 < k1 && ready(&sm.p_full[k2 & 1], (k2 >> 1) & 1) && ready(&sm.v_full[k2 & 1], (k2 >> 1) & 1)) {
            mma2(k2 == begin);
            idle = 0;
          } else if (k1 < end && ready(&sm.k_full[k1 & 1][half], (k1 >> 1) & 1) &&
                     (half == 1 || ready(&sm.s_free[k1 & 1], ((k1 >> 1) & 1) ^ 1))) {
            mma1(half);
            half ^= 1;
            idle = 0;
          } else if ((++idle & 63u) == 0) {  // as pair_wait: give up after kWaitLimitNs
            const uint64_t t = __shfl_sync(0xffffffffu, globaltimer_ns(), 0);
            if (idle == 64) t0 = t;
            ok = *static_cast<volatile int*>(&sm.abort) == 0 && t - t0 <= kWaitLimitNs;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) raise_abort(err, &sm.abort, t - t0 > kWaitLimitNs);
          }
        }
      }
      if (k1 > 0) {  // nothing may still read or write the pair's memory when it leaves
        commit2(&sm.final_bar, elected);
        pair_drain(&sm.final_bar, 0);
      }
    } else if (warp == kIssuer + 1) {
      // Requests this CTA's keys into L2 a few tiles before the K warps load them.
      TileWalk tw;
      tw.start(A, sm);
      uint64_t last = globaltimer_ns();
      uint32_t seen = 0;
      for (uint32_t kk = 0; tw.on(); ++kk, tw.next(A)) {
        if (kk < *static_cast<volatile uint32_t*>(&sm.k_loaded)) continue;  // too late for this tile
        for (;;) {
          const uint32_t done = *static_cast<volatile uint32_t*>(&sm.k_loaded);
          if (kk + 1 < done + kPrefetchAhead && done > 0) break;  // not before the first tile and the queries are asked for
          const uint64_t now = globaltimer_ns();
          if (done != seen) last = now;
          seen = done;
          if (*static_cast<volatile int*>(&sm.abort) || now - last > kWaitLimitNs) break;  // requests only: nothing waits for them
          __nanosleep(100);
        }
        __syncwarp();
        if (kk > 0 && tw.tile == tw.w.ta(A) && A.q_vec) {
          // a unit's first tile: its queries as well (unasked, they cost the softmax warps 4 % of a batch of short units)
          const int rows = tw.w.rows(A, cta);
          const int64_t first = static_cast<int64_t>(tw.w.tok0(A)) * A.D.n_heads + tw.w.rows_before(A, cta);
          for (int r = lane; r < rows; r += 32) {
            prefetch_l2_bulk(A.D.q + (first + r) * kDL, 2 * kDL);
            prefetch_l2_bulk(A.D.q_pe + (first + r) * kDR, 2 * kDR);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = tw.tile * kKeys + kCtaKeys * static_cast<int>(cta) + 32 * i + lane;
          if (j < tw.w.nvis) {
            const int pg = page_of(A, j);
            const int blk = __ldg(A.D.block_table + static_cast<int64_t>(tw.w.b) * A.D.bt_stride + pg);
            if (blk >= 0 && blk < A.D.L.num_blocks)
              prefetch_l2_bulk(record(A, blk, j - pg * A.D.L.block_size), kRec);
          }
        }
      }
    } else if (warp == kIssuer + 2) {
      // A NaN (code 0x7F of either sign) at a position that only some of a unit's tokens see reaches the others
      // too: their zeros times it.  So those few positions are looked at.  (In the K warps, which hold
      // the codes anyway, the same check cost 5 % of the whole call.)
      bool bad = false;
      Walk w;
      for (w.start(A, sm); w.on(); w.next(A)) {
        const int end = min(w.nvis, w.tb(A) * kKeys);
#pragma unroll 1
        for (int j = max(w.nvis - w.ntok(A) + 1, w.ta(A) * kKeys) + static_cast<int>(cta); j < end; j += 2) {
          const int pg = page_of(A, j);
          const int blk = __ldg(A.D.block_table + static_cast<int64_t>(w.b) * A.D.bt_stride + pg);
          if (blk < 0 || blk >= A.D.L.num_blocks) continue;
          const uint4 c = __ldg(reinterpret_cast<const uint4*>(record(A, blk, j - pg * A.D.L.block_size)) + lane);
          const auto is = [](uint32_t x) { return (x & 0x7F7F7F7Fu) + 0x01010101u; };
          bad |= ((is(c.x) | is(c.y) | is(c.z) | is(c.w)) & 0x80808080u) != 0;
        }
      }
      if (bad) latch_error(err, SMLA_ERR_RANGE);
    }
  } else if (warp >= kFirstV) {
    // ------------------------------ V: the other CTA's 64 keys x this CTA's 256 latent dims ------------------------------
    // Warp vw takes 8 of the keys, two at a time.  A lane loads 16 codes of a key, which become two 16-byte
    // slots of a chunk: a key's 256 codes are read together, and a quarter-warp's stores go to eight
    // different slots (lanes of odd chunks store their second slot first).  (Loads of 64 bytes from each of
    // eight keys need no shuffles, but took 24 passes of the load pipe each; eight codes a lane need
    // no swap, but twice the loads and shuffles.)  Lane 2 i + x keeps scale x of key i.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kVRegs));
    constexpr int kN = kKeysPerV;
    const int vw = warp - kFirstV, other = 1 - static_cast<int>(cta);
    const int key0 = kCtaKeys * other + kN * vw;
    const int sub = lane & 15, odd = (sub >> 2) & 1;
    const int code_off = 256 * static_cast<int>(cta) + 16 * sub, scale_off = kDL + 8 * static_cast<int>(cta) + 4 * (lane & 1);
    // row & 7 of key 2 i + (lane >> 4) is that of key lane >> 4 xor 2 i
    const uint32_t dst = (4 * other + (sub >> 2)) * kCtaKeys * 128 + sw128_off(kN * vw + (lane >> 4), 2 * (sub & 3) + odd);
    const uint32_t full[2] = {map_cta(smem_u32(&sm.v_full[0]), 0), map_cta(smem_u32(&sm.v_full[1]), 0)};
    uint4 codes[kN / 2];
    float sc;
    Records<kRuns, kN> rec;
    const auto load = [&](int i) { codes[i] = __ldg(reinterpret_cast<const uint4*>(rec.get(2 * i + (lane >> 4)) + code_off)); };
    const auto load_scale = [&]() { sc = __ldg(reinterpret_cast<const float*>(rec.get((lane >> 1) & (kN - 1)) + scale_off)); };
    const auto store = [&](uint32_t mine, unsigned small, uint8_t* tile) {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) {
        const uint32_t s = __shfl_sync(0xffffffffu, mine, 2 * (2 * i + (lane >> 4)) + (sub >> 3));
        const uint4 c = codes[i];
        uint8_t* to = tile + 256 * i;
        *reinterpret_cast<uint4*>(to + (dst ^ (i << 5))) = dequant8(odd ? make_uint2(c.z, c.w) : make_uint2(c.x, c.y), s);
        *reinterpret_cast<uint4*>(to + (dst ^ (i << 5) ^ 16)) = dequant8(odd ? make_uint2(c.x, c.y) : make_uint2(c.z, c.w), s);
      }
      if (small != 0) {
#pragma unroll 1
        for (int i = 0; i < kN / 2; ++i)
          if (small >> (2 * (2 * i + (lane >> 4)) + (sub >> 3)) & 1) {
            shrink8(tile + 256 * i + (dst ^ (i << 5)));
            shrink8(tile + 256 * i + (dst ^ (i << 5) ^ 16));
          }
      }
    };
    TileWalk tw;
    tw.start(A, sm);
    rec.find(A, tw, key0, lane);
    int n = 0;  // visible records among the loaded ones
    const auto load_tile = [&]() {
      n = rec.take(A);
      load_scale();
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) load(i);
      tw.next(A);
      rec.find(A, tw, key0, lane);
    };
    for (uint32_t kk = 0;; ++kk) {
      const bool on = tw.on();
      load_tile();  // after the fence, which would wait for loads in flight
      if (!on) break;
      if (n < kN) {  // the end of a context: whatever lies behind it counts as zeros
#pragma unroll
        for (int i = 0; i < kN / 2; ++i)
          if (2 * i + (lane >> 4) >= n) codes[i] = make_uint4(0, 0, 0, 0);
        if (((lane >> 1) & (kN - 1)) >= n) sc = 0.f;
      }
      const unsigned small = __ballot_sync(0xffffffffu, small_scale(sc));
      const float scaled = small_scale(sc) ? sc * kSmallUp : sc;
      const uint32_t mine = pack_half2(scaled, scaled);
      // the tile's scores are formed: the chunks that V does not need are free
      if (!__all_sync(0xffffffffu, pair_wait(&sm.s_full[kk & 1], (kk >> 1) & 1, err, &sm.abort))) break;
      store(mine, small, sm.kv[kk & 1][0]);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_cluster(full[kk & 1]);
    }
  } else if (warp >= kFirstK) {
    // ------------------------------ K: this CTA's 64 keys x 576 dims ------------------------------
    // Warp kw takes keys 8 kw .. + 7.  A lane loads eight codes of a key at a time, so that dims 0-255 of all
    // keys are handed over while the others are still converted.
    // Lane 4 i + x keeps scale x of key i.
    static_assert(kKRegs == kLaunchRegs, "no change of registers");
    constexpr int kN = kKeysPerK;
    const int kw = warp - kFirstK, key0 = kN * kw + kCtaKeys * static_cast<int>(cta);
    const uint32_t dst = (lane >> 3) * kCtaKeys * 128 + sw128_off(kN * kw, lane & 7);
    const uint32_t full = map_cta(smem_u32(&sm.k_full[0][0]), 0);
    uint2 codes[2][kN];
    uint4 rope[2];
    float sc;
    Records<kRuns, kN> rec;
    const auto load = [&](int i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) codes[h][i] = __ldg(reinterpret_cast<const uint2*>(rec.get(i) + 256 * h) + lane);
    };
    const auto load_scale = [&]() { sc = __ldg(reinterpret_cast<const float*>(rec.get(lane >> 2) + kDL + 4 * (lane & 3))); };
    const auto load_rope = [&](int i) {
      rope[i] = __ldg(reinterpret_cast<const uint4*>(rec.get(4 * i + (lane >> 3)) + kDL + 16) + (lane & 7));
    };
    const auto store = [&](auto h, uint32_t mine, unsigned small, uint8_t* tile) {
      uint8_t* to = tile + 4 * kCtaKeys * 128 * h();
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const uint32_t s = __shfl_sync(0xffffffffu, mine, 4 * i + 2 * h() + (lane >> 4));
        *reinterpret_cast<uint4*>(to + 128 * i + (dst ^ (i << 4))) = dequant8(codes[h()][i], s);
      }
      if (small != 0) {
#pragma unroll 1
        for (int i = 0; i < kN; ++i)
          if (small >> (4 * i + 2 * h() + (lane >> 4)) & 1) shrink8(to + 128 * i + (dst ^ (i << 4)));
      }
    };
    TileWalk tw;
    tw.start(A, sm);
    bool bad = false;
    rec.find(A, tw, key0, lane);
    int n = 0;  // visible records among the loaded ones
    const auto load_tile = [&]() {
      n = rec.take(A);
      load_scale();
#pragma unroll
      for (int i = 0; i < kN; ++i) load(i);
      load_rope(0);
      load_rope(1);
      tw.next(A);
      rec.find(A, tw, key0, lane);
    };
    for (uint32_t kk = 0;; ++kk) {
      const bool on = tw.on();
      load_tile();  // after the fence, which would wait for loads in flight
      if (!on) break;
      if (threadIdx.x == 32 * kFirstK) *static_cast<volatile uint32_t*>(&sm.k_loaded) = kk + 1;
      if (n < kN) {  // the end of a context
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (i >= n) codes[0][i] = codes[1][i] = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (4 * i + (lane >> 3) >= n) rope[i] = make_uint4(0, 0, 0, 0);
        if ((lane >> 2) >= n) sc = 0.f;
      }
      bad |= !(fabsf(sc) < kScaleEnd);
      const unsigned small = __ballot_sync(0xffffffffu, small_scale(sc));
      const float scaled = small_scale(sc) ? sc * kSmallUp : sc;
      const uint32_t mine = pack_half2(scaled, scaled);
      if (!__all_sync(0xffffffffu, pair_wait(&sm.kv_free[kk & 1][0], ((kk >> 1) & 1) ^ 1, err, &sm.abort))) break;
      uint8_t* tile = sm.kv[kk & 1][0];
      store(std::integral_constant<int, 0>{}, mine, small, tile);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_cluster(full + 16 * (kk & 1));
      if (!__all_sync(0xffffffffu, pair_wait(&sm.kv_free[kk & 1][1], ((kk >> 1) & 1) ^ 1, err, &sm.abort))) break;
      store(std::integral_constant<int, 1>{}, mine, small, tile);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {rope[i].x, rope[i].y, rope[i].z, rope[i].w};
        uint32_t o[4];
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          top = __vmaxu2(top, w[x] & 0x7FFF7FFFu);
          o[x] = pack_half2(__uint_as_float(w[x] << 16), __uint_as_float(w[x] & 0xFFFF0000u));
        }
        bad |= (top & 0xFFFFu) >= kHalfEnd || (top >> 16) >= kHalfEnd;
        *reinterpret_cast<uint4*>(tile + 8 * kCtaKeys * 128 + sw128_off(kN * kw + 4 * i + (lane >> 3), lane & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_cluster(full + 16 * (kk & 1) + 8);
    }
    if (bad) latch_error(err, SMLA_ERR_RANGE);
  } else {
    // ------------------------------ queries, softmax, epilogue ------------------------------
    // Thread: TMEM lane L = 32 (warp % 4) + lane, which is row L % 64 and half kh = L / 64 of a tile's
    // keys (of O's dims); warps 0-3 take the first 32 columns of the half (the first 128 of O's), warps
    // 4-7 the others.  The four threads of a row agree on its running maximum.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int sp = warp & 3, wg = warp >> 2;
    const int L = 32 * sp + lane, row = L & 63, kh = L >> 6;
    const uint32_t lane_base = static_cast<uint32_t>(sp * 32) << 16;
    // (p_full by the tile's parity: one CTA's warps may be a tile ahead of the other's)
    const uint32_t p_full[2] = {map_cta(smem_u32(&sm.p_full[0]), 0), map_cta(smem_u32(&sm.p_full[1]), 0)}, q_full = map_cta(smem_u32(&sm.q_full), 0);
    const uint32_t s_free[2] = {map_cta(smem_u32(&sm.s_free[0]), 0), map_cta(smem_u32(&sm.s_free[1]), 0)};
    const int H = A.D.n_heads;
    // Queries of a unit: warp w loads rows 8 w .. + 7, a lane 16 latent and 2 rope dims of each.  A row is
    // scaled by a power of two that takes its largest element to [2^8, 2^9): fp16 then holds bf16's
    // eight bits exactly down to 2^-23 of that element.
    // (Short code matters here as much as loads in flight: it runs once a unit, from a cold instruction
    // cache.)
    const auto load_q = [&](const Walk& w, int slot) {
      const int rows = w.rows(A, cta);
      const int64_t first = static_cast<int64_t>(w.tok0(A)) * H + w.rows_before(A, cta);
      uint32_t v[4][9];
      const auto ask = [&](int i, int r) {
#pragma unroll
        for (int x = 0; x < 9; ++x) v[i][x] = 0;
        if (r < rows) load_query(A, first + r, lane, v[i]);
      };
#pragma unroll
      for (int i = 0; i < 4; ++i) ask(i, 8 * warp + i);
#pragma unroll 1
      for (int r0 = 8 * warp; r0 < 8 * warp + 8; r0 += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = r0 + i;
          uint32_t top2 = 0;  // the largest magnitude (bf16 bits of non-negative values order as integers)
#pragma unroll
          for (int x = 0; x < 9; ++x) top2 = __vmaxu2(top2, v[i][x] & 0x7FFF7FFFu);
          const uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xFFFFu, top2 >> 16));
          const int ex = static_cast<int>(top >> 7);  // biased exponent
          const int up = (ex == 0 || ex == 255) ? 0 : min(126, 127 + 8 - ex);  // zeros, infinities and NaN as they are
          const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23) * A.sign;
          uint32_t o[9];
#pragma unroll
          for (int x = 0; x < 9; ++x)
            o[x] = pack_half2(__uint_as_float(v[i][x] << 16) * f, __uint_as_float(v[i][x] & 0xFFFF0000u) * f);
#pragma unroll
          for (int x = 0; x < 9; ++x) v[i][x] = v[i + 2][x];
          const int c = lane >> 2, odd = c & 1, s0 = 2 * (lane & 3);
          const uint4 o0 = make_uint4(o[0], o[1], o[2], o[3]), o1 = make_uint4(o[4], o[5], o[6], o[7]);
          *reinterpret_cast<uint4*>(&sm.q[c][sw128_off(r, s0 + odd)]) = odd ? o1 : o0;
          *reinterpret_cast<uint4*>(&sm.q[c][sw128_off(r, s0 + 1 - odd)]) = odd ? o0 : o1;
          *reinterpret_cast<uint32_t*>(&sm.q[8][sw128_off(r, lane >> 2) + 4 * (lane & 3)]) = o[8];
          if (lane == 0) sm.row_f[slot][r] = A.abs_scale * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        }
        if (r0 < 8 * warp + 4) {
          ask(2, r0 + 4);
          ask(3, r0 + 5);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) arrive_cluster(q_full);
    };

    Walk w;
    w.start(A, sm);
    if (A.meta != nullptr && cta == 0 && threadIdx.x == 0) A.meta[pair].ntok = 0;
    Walk nx = w;  // the unit whose queries come next
    uint32_t kk = 0, n = 0;
    float m = 0.f, l = 0.f;
    bool ok = true;
    // Each turn: the next unit's queries (while the last MMAs run: the last scores are read, Q is free), the
    // results of the unit before, then the unit's tiles.  In this order the loop holds one copy of each
    // part, which matters where its code is met for the first time.
    for (;; ++n) {
      if (nx.on()) load_q(nx, n & 1);
      if (n > 0) {
        // ---- end of unit ----
        const int rows = w.rows(A, cta), grow = w.rows_before(A, cta) + row;  // grow: row of the unit
        const bool real = row < rows, idle = 32 * (sp & 1) >= rows;
        const int ta = w.ta(A), tb = w.tb(A);
        ok = pair_wait(&sm.kv_free[(kk - 1) & 1][1], ((kk - 1) >> 1) & 1, err, &sm.abort) && ok;
        __syncwarp();
        tc_fence_after();
        sm.red[2 * wg + kh][row] = l;
        if (bar_red_or(1, 32 * kSoftmaxWarps, !ok)) break;
        const float lt = (sm.red[0][row] + sm.red[1][row]) + (sm.red[2][row] + sm.red[3][row]);
        const float inv = lt == 0.f ? 0.f : 1.f / lt;  // no visible key: zeros
        const float lse = lt == 0.f ? -INFINITY : (m + log2f(lt)) * kLn2;
        const bool partial = ta > 0 || tb < w.tiles();
        const int64_t slot = 2 * pair + (ta > 0 ? 0 : 1);
        const int64_t orow = static_cast<int64_t>(w.tok0(A)) * H + grow;
        const int d0 = 256 * kh + 128 * wg;
        if (kh == 0 && wg == 0 && real) {
          if (partial) A.part_lse[slot * kRows + grow] = lse;
          else if (A.D.lse != nullptr) A.D.lse[orow] = lse;
        }
        // A lane holds 128 dims of its row and reads them 32 at a time.  The lanes of a group of four exchange them
        // (as bf16 pairs; partial results in fp32, in two halves), so that the group stores 64 consecutive
        // bytes of each of its rows: a lane that stores its own row's dims touches 32 rows in every store, and
        // exchanges in fp32 throughout made a batch of short units 6 % slower.
        const int i4 = lane & 3;
        const bool hi1 = (i4 & 1) != 0, hi2 = (i4 & 2) != 0;
        const uint32_t t_o = tmem_o + lane_base + 128 * wg;
#pragma unroll 1
        for (int x = 0; x < 4 && !idle; ++x) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(t_o + 32 * x, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          uint32_t h[16];
          if (partial) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
              for (int i = 0; i < 16; ++i) h[i] = o[16 * y + i];
              transpose4(h, hi1, hi2);
              float* to = A.part_out + (slot * kRows + grow - i4) * kDL + d0 + 32 * x + 16 * y + 4 * i4;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (row - i4 + j < rows)
                  *reinterpret_cast<uint4*>(to + j * kDL) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) h[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
            transpose4(h, hi1, hi2);
            __nv_bfloat16* to = A.D.out + (orow - i4) * kDL + d0 + 32 * x + 8 * i4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (row - i4 + j < rows)
                *reinterpret_cast<uint4*>(to + j * kDL) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
          }
        }
        tc_fence_before();
        // the unit that goes on in the next pair: what the merge has to join
        if (cta == 0 && threadIdx.x == 0 && ta == 0 && tb < w.tiles())
          A.meta[pair] = {sm.x0 + w.rel + w.tiles(), sm.total, sm.pairs, w.tok0(A), w.ntok(A)};
      }
      named_bar_sync(1, 32 * kSoftmaxWarps);  // red is read, row_f is written
      w = nx;
      if (!w.on()) break;
      nx.next(A);
      const int rows = w.rows(A, cta), grow = w.rows_before(A, cta) + row;  // grow: row of the unit
      const bool real = row < rows;
      const bool idle = 32 * (sp & 1) >= rows;  // no row of this warp is one: it only keeps the others company
      const int vis = real ? static_cast<int>(visible(A.D, w.seq_len, w.g * A.group + grow / H, w.n_q)) : 0;
      const int ta = w.ta(A), tb = w.tb(A);
      // above zero, so that a masked score (-inf) stays one whatever softmax_scale is
      const float f = fmaxf(sm.row_f[n & 1][row], 1.2e-38f);
      m = -INFINITY;
      l = 0.f;
      bool failed = false;
      for (int tile = ta; tile < tb; ++tile, ++kk) {
        const int buf = kk & 1;
        ok = ok && pair_wait(&sm.s_full[buf], (kk >> 1) & 1, err, &sm.abort);
        __syncwarp();
        tc_fence_after();
        uint32_t r[32];
        tmem_ld32(tmem_s + lane_base + buf * 64 + 32 * wg, r);
        tmem_ld_wait(r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(s_free[buf]);
        // visible keys among this thread's 32
        const int vr = vis - (tile * kKeys + 64 * kh + 32 * wg);
        float mx = -INFINITY;
        if (!idle) {
          if (!__all_sync(0xffffffffu, vr >= 32)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= vr) r[i] = 0xFF800000u;  // -inf
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(r[i]));
        }
        // The maximum of a row moves only when a score passes it by 2^8; only then (and on the first
        // tile) the four threads of every row compare notes.  It is kept as the products' value, before the
        // scale: a score's difference from it is exact near it, however large both are, while a product
        // m f would round by many powers of two in probability from 2^28 on.
        const bool first = tile == ta;
        if (bar_red_or(1, 32 * kSoftmaxWarps, first || !ok || (mx - m) * f > kRescale)) {
          sm.red[2 * wg + kh][row] = mx;
          if (bar_red_or(1, 32 * kSoftmaxWarps, !ok)) {
            failed = true;
            break;
          }
          const float mt = fmaxf(fmaxf(sm.red[0][row], sm.red[1][row]), fmaxf(sm.red[2][row], sm.red[3][row]));
          const bool move = first || (mt - m) * f > kRescale;
          const float mn = move ? fmaxf(m, mt) : m;
          const float alpha = move && m != -INFINITY ? exp2f((m - mn) * f) : 1.f;
          l *= alpha;
          m = mn;
          if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
            // O holds the tiles before this one once their last MMA is done; this tile's waits for p_full
            ok = pair_wait(&sm.kv_free[(kk - 1) & 1][1], ((kk - 1) >> 1) & 1, err, &sm.abort) && ok;
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < 4; ++x) {
              uint32_t o[32];
              tmem_ld32(tmem_o + lane_base + 128 * wg + 32 * x, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tmem_o + lane_base + 128 * wg + 32 * x, o);
            }
            tmem_st_wait();
          }
          named_bar_sync(1, 32 * kSoftmaxWarps);  // red is read
        }
        if (idle) {  // the rows' P is whatever it was; their part of O is not read
          if (kh == 1 && kk > 0) ok = pair_wait(&sm.kv_free[(kk - 1) & 1][1], ((kk - 1) >> 1) & 1, err, &sm.abort) && ok;
          __syncwarp();
          if (lane == 0) arrive_cluster(p_full[buf]);
          continue;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        uint32_t pw[16];
        float2 ls = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float2 x = fma2(add2(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), make_float2(-mu, -mu)), f, kLift);
          const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          ls = add2(ls, p);
          pw[i / 2] = pack_half2(p.x, p.y);
        }
        l += ls.x + ls.y;
        // keys 0-63 go to this tile's rope chunk; p1 is free once the last tile's MMAs have read it
        if (kh == 1 && kk > 0) ok = pair_wait(&sm.kv_free[(kk - 1) & 1][1], ((kk - 1) >> 1) & 1, err, &sm.abort) && ok;
        uint8_t* p = kh == 0 ? sm.kv[buf][8] : sm.p1;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          *reinterpret_cast<uint4*>(p + sw128_off(row, 4 * wg + v)) = make_uint4(pw[4 * v], pw[4 * v + 1], pw[4 * v + 2], pw[4 * v + 3]);
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(p_full[buf]);
      }
      if (failed) break;
      m = m * f - kLift;  // for the unit's end: in powers of two
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's arrivals and MMAs no longer touch this one
  if (warp == kIssuer) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Joins the parts of units that ran on several pairs: lse = ln sum e^lse_i, out = sum e^(lse_i - lse) out_i
// in fp32.  A warp takes a row (a lane 16 dims) where a few parts are to be joined; where there are many, as
// for one long sequence, the block's four warps share it (a lane 4 dims, eight parts' loads in flight).
// With the whole call's time: one sequence of 262,143 positions 95 us (117 with a warp per row), 64 sequences of
// four tokens 645 us (655 with a block per row).
constexpr int kMergeThreads = 128, kFewParts = 4;
template <int kStep>
__device__ __forceinline__ void merge_row(const PairMeta& M, int p, int parts, int row, int quarter0, int quarters,
                                          const float* part_lse, const float* part_out, int n_heads, __nv_bfloat16* out, float* lse) {
  const int lane = threadIdx.x & 31;
  const auto slot = [&](int i) -> int64_t { return i == 0 ? 2 * p + 1 : 2 * (p + i); };
  float v[kMaxPairs / 32], mx = -INFINITY, z = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxPairs / 32; ++i) {
    v[i] = 32 * i + lane < parts ? __ldcg(part_lse + slot(32 * i + lane) * kRows + row) : -INFINITY;
    mx = fmaxf(mx, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
  for (int i = 0; i < kMaxPairs / 32; ++i) {
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
        const float w = part < 32 ? v[0] : part < 64 ? v[1] : part < 96 ? v[2] : v[3];
        f[i] = __shfl_sync(0xffffffffu, w, part & 31) * inv;
        if (i0 + i >= parts) f[i] = 0.f;
#pragma unroll
        for (int y = 0; y < kQ; ++y)
          a[i][y] = __ldcg(reinterpret_cast<const float4*>(part_out + (slot(part) * kRows + row) * kDL + 128 * (q + y)) + lane);
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

// Starts while the pairs still write what it reads.  So the reads come after its wait for them, are ordinary ones
// and not of the read-only path, which stands for data that no one writes while the kernel lives, and no pointer
// is marked as free of aliases, so that none of them moves before the wait.
__global__ void __launch_bounds__(kMergeThreads) dense_merge_kernel(const PairMeta* meta, const float* part_lse,
                                                                    const float* part_out, int n_pairs, int n_heads,
                                                                    __nv_bfloat16* out, float* lse) {
  __shared__ int cum[kMaxPairs + 1];  // rows to join of the pairs before p
  static_assert(kMergeThreads == kMaxPairs, "a thread per pair");
  const int tid = threadIdx.x, warp = tid >> 5;
  cudaGridDependencySynchronize();
  cum[tid + 1] = tid < n_pairs ? meta[tid].ntok * n_heads : 0;
  if (tid == 0) cum[0] = 0;
  __syncthreads();
#pragma unroll 1
  for (int o = 1; o < kMaxPairs; o <<= 1) {
    const int v = tid + 1 > o ? cum[tid + 1 - o] : 0;
    __syncthreads();
    cum[tid + 1] += v;
    __syncthreads();
  }
  const int total = cum[kMaxPairs];
  const auto join = [&](int item, bool few) {
    int p = 0, hi = n_pairs - 1;
    while (p < hi) {
      const int mid = (p + hi + 1) / 2;
      if (cum[mid] <= item) p = mid;
      else hi = mid - 1;
    }
    const PairMeta M = meta[p];
    // pairs p + 1 .. carry the rest: range r begins at floor(r total / pairs), before the unit's end for
    // r < end pairs / total
    const int n = static_cast<int>(min((M.end * M.pairs + M.total - 1) / M.total, static_cast<int64_t>(M.pairs))) - p;
    if (few && n <= kFewParts) merge_row<2>(M, p, n, item - cum[p], 0, 4, part_lse, part_out, n_heads, out, lse);
    if (!few && n > kFewParts) merge_row<8>(M, p, n, item - cum[p], warp, 1, part_lse, part_out, n_heads, out, lse);
  };
#pragma unroll 1
  for (int item = 4 * blockIdx.x + warp; item < total; item += 4 * gridDim.x) join(item, true);
#pragma unroll 1
  for (int item = blockIdx.x; item < total; item += gridDim.x) join(item, false);
}

// Layouts of the full latent shape.
bool pair_shape(const KernelLayout& L) { return L.d_latent == kDL && L.quant_tile == 128 && L.d_rope == kDR; }

constexpr size_t kMetaBytes = (kMaxPairs * sizeof(PairMeta) + 255) / 256 * 256;
constexpr size_t kPartLseBytes = 2 * kMaxPairs * kRows * sizeof(float);
constexpr size_t kPartOutBytes = size_t(2) * kMaxPairs * kRows * kDL * sizeof(float);

template <bool kRuns>
smla_status_t resident_pairs(int* out) {
  static std::atomic<int> pairs_of[kMaxDeviceSlots] = {};
  const int dev = current_device_index();
  if (dev < 0) return SMLA_ERR_CUDA;
  int pairs = pairs_of[dev].load(std::memory_order_acquire);
  if (pairs == 0) {
    const auto kernel = dense_pair_kernel<kRuns>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kPairSmemBytes)) != cudaSuccess)
      return SMLA_ERR_CUDA;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return SMLA_ERR_CUDA;
    if (fa.numRegs < kLaunchRegs) return SMLA_ERR_UNSUPPORTED;  // setmaxnreg.inc draws on the launch's registers
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * kMaxPairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kPairSmemBytes;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess || pairs <= 0) return SMLA_ERR_CUDA;
    if (pairs > kMaxPairs) pairs = kMaxPairs;
    pairs_of[dev].store(pairs, std::memory_order_release);
  }
  *out = pairs;
  return SMLA_OK;
}

smla_status_t launch_dense_pair(const DenseArgs& D, float softmax_scale, void* workspace, size_t workspace_bytes,
                                cudaStream_t s) {
  const bool runs = D.L.block_size % 16 == 0;
  int pairs = 0;  // resident at once
  const smla_status_t st = runs ? resident_pairs<true>(&pairs) : resident_pairs<false>(&pairs);
  if (st != SMLA_OK) return st;
  PairArgs A{};
  A.D = D;
  A.group = kRows / D.n_heads;
  A.abs_scale = fabsf(softmax_scale) * kLog2e;
  A.sign = softmax_scale < 0.f ? -1.f : 1.f;
  A.q_vec = (reinterpret_cast<uintptr_t>(D.q) & 15) == 0 && (reinterpret_cast<uintptr_t>(D.q_pe) & 15) == 0;
  A.records = D.pool + static_cast<int64_t>(D.layer) * D.L.layer_stride + D.L.rec_off;
  uint32_t log2 = 0;
  while ((1ull << log2) < static_cast<uint64_t>(D.L.block_size)) ++log2;
  A.bs_mul = static_cast<uint32_t>((((1ull << log2) - D.L.block_size) << 32) / D.L.block_size + 1);
  A.bs_shift1 = log2 > 0 ? 1 : 0;
  A.bs_shift2 = log2 > 0 ? log2 - 1 : 0;
  // Splitting pays wherever units are fewer or more uneven than pairs: 32 decode tokens 188 us (598 without), one
  // long sequence 95 us (4.7 ms), a chunk of 1,024 units 3.89 ms (4.17).  Without a workspace units stay whole.
  // The ranges count tiles only, not the time between units (about four tiles' of each): where short contexts
  // stand beside long ones, the pairs with the short ones' many units end last (8 to 70 units a pair in a ragged
  // batch of contexts from 777 to 5,003).
  const bool split = workspace != nullptr && workspace_bytes >= kMetaBytes + kPartLseBytes + kPartOutBytes;
  if (split) {
    uint8_t* w = static_cast<uint8_t*>(workspace);
    A.meta = reinterpret_cast<PairMeta*>(w);
    A.part_lse = reinterpret_cast<float*>(w + kMetaBytes);
    A.part_out = reinterpret_cast<float*>(w + kMetaBytes + kPartLseBytes);
  }
  if (runs) dense_pair_kernel<true><<<2 * pairs, kThreads, kPairSmemBytes, s>>>(A);
  else dense_pair_kernel<false><<<2 * pairs, kThreads, kPairSmemBytes, s>>>(A);
  if (cudaGetLastError() != cudaSuccess) return SMLA_ERR_CUDA;
  if (split) {
    // launched while the pairs still work (its blocks wait for their results before they read)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(6 * device_sm_count());
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dense_merge_kernel, static_cast<const PairMeta*>(A.meta), static_cast<const float*>(A.part_lse),
                           static_cast<const float*>(A.part_out), pairs, D.n_heads, D.out, D.lse) != cudaSuccess)
      return SMLA_ERR_CUDA;
  }
  return SMLA_OK;
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" size_t smla_attend_dense_workspace_size(const smla_layout_t* layout, const smla_params_t* params,
                                                   int n_tokens) {
  if (!layout_ok(layout) || params == nullptr || n_tokens <= 0 || params->n_heads <= 0) return 0;
  return pair_shape(kernel_layout(*layout)) ? kMetaBytes + kPartLseBytes + kPartOutBytes : 0;
}

extern "C" smla_status_t smla_attend_dense(const smla_layout_t* layout, const smla_params_t* params, const void* pool,
                                           int layer, const void* q, const void* q_pe, const int32_t* block_table,
                                           int bt_stride, const int32_t* seq_lens, const int32_t* query_start_loc,
                                           int batch, int n_tokens, void* out, float* lse, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (!layout_ok(layout) || !params || layer < 0 || layer >= layout->n_layers || batch <= 0 || n_tokens < 0 ||
      params->n_heads <= 0 || (workspace == nullptr && workspace_bytes != 0) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15) != 0)
    return SMLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return SMLA_OK;
  if (!pool || (reinterpret_cast<uintptr_t>(pool) & 15) != 0 || !q || (layout->d_rope > 0 && !q_pe) || !block_table ||
      bt_stride <= 0 || !seq_lens || !query_start_loc || !out || (reinterpret_cast<uintptr_t>(out) & 15) != 0)
    return SMLA_ERR_INVALID_ARG;
  const KernelLayout L = kernel_layout(*layout);
  if (!store_shape_supported(L) || L.d_rope > 64 || params->n_heads > kMaxHeads) return SMLA_ERR_UNSUPPORTED;
  DenseArgs A{};
  const smla_status_t st = checked_device(&A.err);
  if (st != SMLA_OK) return st;
  A.L = L;
  A.n_heads = params->n_heads;
  A.layer = layer;
  A.scale_log2 = params->softmax_scale * kLog2e;
  A.pool = static_cast<const uint8_t*>(pool);
  A.q = static_cast<const __nv_bfloat16*>(q);
  A.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
  A.block_table = block_table;
  A.bt_stride = bt_stride;
  A.most = std::min(static_cast<int64_t>(bt_stride) * L.block_size, static_cast<int64_t>(kMaxContext));
  A.seq_lens = seq_lens;
  A.qsl = query_start_loc;
  A.batch = batch;
  A.n_tokens = n_tokens;
  A.out = static_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pair_shape(L)) return launch_dense_pair(A, params->softmax_scale, workspace, workspace_bytes, s);
  return launch_dense_fp32(A, s);
}
