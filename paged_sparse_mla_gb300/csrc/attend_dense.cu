// smla_attend_dense: latent MQA attention of each query token over its whole visible context.
//
// [AgentX "Kimi K3"], [GLM-5.3 "What is new"]: MLA keeps one latent KV shared by all query heads, so
// attention is MQA over the latent; V is the latent.  [GLM-5.3 "How to try"]: a prompt that fits the
// top-k attends over all of its positions; here that holds at any length.
#include <atomic>

#include "smla_internal.h"

namespace smla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxHeads = 128;

struct DenseArgs {
  KernelLayout L;
  int n_heads, layer;
  float scale_log2;  // softmax_scale * log2(e)
  const uint8_t* pool;
  const __nv_bfloat16 *q, *q_pe;
  const int32_t *block_table, *seq_lens, *qsl;
  int bt_stride, batch, n_tokens;
  __nv_bfloat16* out;
  float* lse;  // or nullptr
  unsigned* err;
};

// Positions that query token t (the i-th of sequence b's n_q) sees: seq_len - n_q + i + 1, at least
// none and at most what the block-table row holds.
__device__ __forceinline__ int64_t visible(const DenseArgs& A, int b, int i, int n_q) {
  const int64_t n = static_cast<int64_t>(__ldg(A.seq_lens + b)) - n_q + i + 1;
  const int64_t most = static_cast<int64_t>(A.bt_stride) * A.L.block_size;
  return n < 0 ? 0 : n < most ? n : most;
}

// ---------------------------------------------------------------------------
// Shapes without a tensor-core kernel: fp32 throughout.  One CTA per (query token, 8 heads); keys in
// tiles of 32, dequantised into shared memory; warp h scores head h (a lane per key), then every
// thread accumulates its dims for the 8 heads.
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
  const int64_t n = visible(A, b, t - q0, n_q);
  if (threadIdx.x == 0 && __ldg(A.seq_lens + b) > static_cast<int64_t>(A.bt_stride) * L.block_size)
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

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" size_t smla_attend_dense_workspace_size(const smla_layout_t* layout, const smla_params_t* params,
                                                   int n_tokens) {
  if (!layout_ok(layout) || params == nullptr || n_tokens <= 0 || params->n_heads <= 0) return 0;
  return 0;
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
  A.seq_lens = seq_lens;
  A.qsl = query_start_loc;
  A.batch = batch;
  A.n_tokens = n_tokens;
  A.out = static_cast<__nv_bfloat16*>(out);
  A.lse = lse;
  return launch_dense_fp32(A, static_cast<cudaStream_t>(stream));
}
