// kvpack_append and smla_query_prep: from a layer's projections to the cache and to the queries.
//
// [GLM-5.3 "How to try", "Config and numbers"]: the KV cache is FP8.  [AgentX "Hybrid KV cache
// management"]: one packed allocation per block holds every cache group.  [AgentX "DeepSeek V4"]: 64
// indexer heads a token.
//
// Norm, position rotation, quantisation and the scatter (or the head weight) are one pass: a row is
// read once as bf16, kept in fp32 registers (in shared memory only where a rotation pairs elements of
// different lanes) and leaves as codes.  The normalised values are not rounded to bf16 before they are
// quantised: that rounding (2^-8) would only add to the code's (2^-4).
#include <cuda_fp4.h>

#include "smla_internal.h"

namespace smla {
namespace {

constexpr int kWarps = 8;             // warps per CTA
constexpr int kMaxIndex = 256;        // largest d_index
constexpr float kTinyAmax = 7.888609052210118e-31f;  // 2^-100: below it 448 / amax would near fp32's end

struct RopeArgs {
  const float* cos_sin;  // nullptr: nothing rotates
  int64_t n_positions;
  const int64_t* positions;
  int d_rope, interleaved, idx_interleaved, idx_rope;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// N consecutive bf16 values; `vec`: the address is a multiple of min(16, 2 N) bytes.
template <int N>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, bool vec, float (&x)[N]) {
  if constexpr (N % 8 == 0) {
    if (vec) {
#pragma unroll
      for (int v = 0; v < N / 8; ++v) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + v);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          x[8 * v + 2 * q] = __uint_as_float(ws[q] << 16);
          x[8 * v + 2 * q + 1] = __uint_as_float(ws[q] & 0xFFFF0000u);
        }
      }
      return;
    }
  } else if constexpr (N == 4) {
    if (vec) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
      x[0] = __uint_as_float(w.x << 16);
      x[1] = __uint_as_float(w.x & 0xFFFF0000u);
      x[2] = __uint_as_float(w.y << 16);
      x[3] = __uint_as_float(w.y & 0xFFFF0000u);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __bfloat162float(p[i]);
}

// amax -> (scale, its reciprocal) for codes of largest magnitude `top` = 1 / rtop.  Each is within two units of
// the last place of the quotient; a scale that is a little small saturates.
__device__ __forceinline__ void quant_scale(float amax, float rtop, float& scale, float& inv) {
  const bool tiny = amax < kTinyAmax;
  scale = tiny ? 1.0f : amax * rtop;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
}
constexpr float kRE4M3 = 1.0f / 448.0f, kRE2M1 = 1.0f / 6.0f;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Element pairs of a rotation: the pair of element i, and whether i is its first one.
__device__ __forceinline__ void rope_pair(int i, int half, int interleaved, int& pair, int& other, bool& first) {
  if (interleaved) {
    pair = i >> 1;
    other = i ^ 1;
    first = (i & 1) == 0;
  } else {
    first = i < half;
    pair = first ? i : i - half;
    other = first ? i + half : i - half;
  }
}

// Rotates the first d_rope of the row's 32 * EK values (lane l holds elements EK l .. EK l + EK - 1)
// through `stage`, a row of floats of this warp.
template <int EK>
__device__ __forceinline__ void rotate_row(float (&z)[EK], const float* cs, int d_rope, int interleaved, float* stage,
                                           int lane) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < EK; ++i) stage[lane * EK + i] = z[i];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < EK; ++i) {
    const int e = lane * EK + i;
    if (e < d_rope) {
      int pair, other;
      bool first;
      rope_pair(e, d_rope / 2, interleaved, pair, other, first);
      const float c = __ldg(cs + pair), s = __ldg(cs + d_rope / 2 + pair), o = stage[other];
      z[i] = first ? z[i] * c - o * s : o * s + z[i] * c;
    }
  }
}

struct AppendArgs {
  KernelLayout L;
  uint8_t* pool;
  int layer;
  const __nv_bfloat16 *latent, *rope_key, *idx_k;
  int64_t latent_stride, rope_stride, idx_stride;
  const float *latent_norm, *idx_norm, *idx_bias;
  float eps;
  RopeArgs rope;
  const int64_t* slots;
  int n_tokens;
  bool vec_latent, vec_idx;
  unsigned* err;
};

// Any shape and alignment: one warp per token, lane l owns latent elements [E l, E l + E) and key elements
// [EK l, EK l + EK).
template <int E, int EK>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendArgs A) {
  __shared__ float stage[kWarps][32 * EK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= A.n_tokens) return;
  const KernelLayout& L = A.L;
  const int64_t slot = __ldg(A.slots + t);
  const int64_t pos = A.rope.cos_sin ? __ldg(A.rope.positions + t) : 0;
  float x[E];
  load_bf16<E>(A.latent + t * A.latent_stride + lane * E, A.vec_latent, x);
  float z[EK];
  if (A.idx_k) load_bf16<EK>(A.idx_k + t * A.idx_stride + lane * EK, A.vec_idx, z);
  const int half = L.d_rope / 2;
  int ra = lane, rb = lane + half;
  if (A.rope.interleaved) {
    ra = 2 * lane;
    rb = 2 * lane + 1;
  }
  float r0 = 0.f, r1 = 0.f;
  if (lane < half) {
    r0 = __bfloat162float(A.rope_key[t * A.rope_stride + ra]);
    r1 = __bfloat162float(A.rope_key[t * A.rope_stride + rb]);
  }
  if (slot < 0) return;
  if (slot >= L.num_blocks * L.block_size || (A.rope.cos_sin && (pos < 0 || pos >= A.rope.n_positions))) {
    if (lane == 0) latch_error(A.err, SMLA_ERR_BAD_INDEX);
    return;
  }
  const int64_t blk = slot / L.block_size;
  const int off = static_cast<int>(slot - blk * L.block_size);
  uint8_t* base = A.pool + blk * L.block_stride + static_cast<int64_t>(A.layer) * L.layer_stride;
  uint8_t* rec = base + L.rec_off + static_cast<int64_t>(off) * L.rec_stride;
  const float* cs = A.rope.cos_sin ? A.rope.cos_sin + pos * L.d_rope : nullptr;

  // ---- rope key ----
  if (lane < half) {
    if (cs) {
      const float c = __ldg(cs + lane), s = __ldg(cs + half + lane);
      const float y0 = r0 * c - r1 * s;
      r1 = r0 * s + r1 * c;
      r0 = y0;
    }
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(rec + L.d_latent + 4 * L.n_scales);
    dst[ra] = __float2bfloat16_rn(r0);
    dst[rb] = __float2bfloat16_rn(r1);
  }

  // ---- latent: norm, per-tile scale, codes ----
  if (A.latent_norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) ss += x[i] * x[i];
    const float rstd = rsqrtf(warp_sum(ss) / static_cast<float>(32 * E) + A.eps);
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = x[i] * rstd * __ldg(A.latent_norm + lane * E + i);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(x[i]));
  const int lanes_per_tile = L.quant_tile / E;
  for (int m = 1; m < lanes_per_tile; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  float scale, inv;
  quant_scale(amax, kRE4M3, scale, inv);
  // the record is 16-byte aligned: a lane's codes leave as one store
  if constexpr (E == 2) {
    reinterpret_cast<uint16_t*>(rec)[lane] = static_cast<uint16_t>(e4m3x2(x[0] * inv, x[1] * inv));
  } else {
    uint32_t w[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i)
      w[i] = e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) | e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16;
    if constexpr (E == 16) reinterpret_cast<uint4*>(rec)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (E == 8) reinterpret_cast<uint2*>(rec)[lane] = make_uint2(w[0], w[1]);
    else reinterpret_cast<uint32_t*>(rec)[lane] = w[0];
  }
  if ((lane * E) % L.quant_tile == 0) reinterpret_cast<float*>(rec + L.d_latent)[(lane * E) / L.quant_tile] = scale;

  // ---- indexer key ----
  if (A.idx_k == nullptr) return;
  constexpr float kN = 32 * EK;
  if (A.idx_norm) {
    float mean = 0.f;
    if (A.idx_bias) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < EK; ++i) sum += z[i];
      mean = warp_sum(sum) / kN;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < EK; ++i) {
      z[i] -= mean;
      ss += z[i] * z[i];
    }
    const float rstd = rsqrtf(warp_sum(ss) / kN + A.eps);
#pragma unroll
    for (int i = 0; i < EK; ++i) {
      z[i] = z[i] * rstd * __ldg(A.idx_norm + lane * EK + i);
      if (A.idx_bias) z[i] += __ldg(A.idx_bias + lane * EK + i);
    }
  }
  if (cs && A.rope.idx_rope) rotate_row<EK>(z, cs, L.d_rope, A.rope.idx_interleaved, stage[warp], lane);
  float kmax = 0.f;
#pragma unroll
  for (int i = 0; i < EK; ++i) kmax = fmaxf(kmax, fabsf(z[i]));
  float kscale, kinv;
  const bool fp4 = L.key_format == SMLA_KEY_E2M1;
  quant_scale(warp_max(kmax), fp4 ? kRE2M1 : kRE4M3, kscale, kinv);
  uint8_t* kdst = base + L.idx_key_off + static_cast<int64_t>(off) * L.key_bytes;
  if (fp4) {
    if constexpr (EK == 1) {
      const float hi = __shfl_down_sync(0xffffffffu, z[0], 1);
      if ((lane & 1) == 0)
        kdst[lane / 2] = __nv_cvt_float2_to_fp4x2(make_float2(z[0] * kinv, hi * kinv), __NV_E2M1, cudaRoundNearest);
    } else {
#pragma unroll
      for (int i = 0; i < EK; i += 2)
        kdst[(lane * EK + i) / 2] =
            __nv_cvt_float2_to_fp4x2(make_float2(z[i] * kinv, z[i + 1] * kinv), __NV_E2M1, cudaRoundNearest);
    }
  } else if constexpr (EK >= 4) {
#pragma unroll
    for (int i = 0; i < EK; i += 4)
      *reinterpret_cast<uint32_t*>(kdst + lane * EK + i) =
          e4m3x2(z[i] * kinv, z[i + 1] * kinv) | e4m3x2(z[i + 2] * kinv, z[i + 3] * kinv) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < EK; ++i)
      kdst[lane * EK + i] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(z[i] * kinv, __NV_SATFINITE, __NV_E4M3));
  }
  if (lane == 0) reinterpret_cast<float*>(base + L.idx_scale_off)[off] = kscale;
}

struct QueryArgs {
  const __nv_bfloat16 *q_pe, *q_idx;
  int64_t pe_token, pe_head, idx_token, idx_head;
  __nv_bfloat16* q_pe_out;
  const float *idx_norm, *w;
  float eps, w_scale;
  uint8_t* codes;
  float* w_out;
  int n_tokens, n_heads, n_idx_heads, d_rope, d_index;
  RopeArgs rope;
  bool vec_idx;
  unsigned* err;
};

// Any shape and alignment, one warp per row: rows [0, n_idx_heads) of a token are its indexer heads, the next
// n_heads its q_pe.
template <int EK>
__global__ void __launch_bounds__(32 * kWarps) query_kernel(const QueryArgs A) {
  __shared__ float stage[kWarps][32 * EK];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hi = A.q_idx ? A.n_idx_heads : 0, rows = hi + (A.q_pe ? A.n_heads : 0);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t t = row / rows;
  const int h = static_cast<int>(row - t * rows);
  if (t >= A.n_tokens) return;
  const float* cs = nullptr;
  if (A.rope.cos_sin) {
    const int64_t pos = __ldg(A.rope.positions + t);
    if (pos < 0 || pos >= A.rope.n_positions) {
      if (lane == 0 && h == 0) latch_error(A.err, SMLA_ERR_BAD_INDEX);
      return;
    }
    cs = A.rope.cos_sin + pos * A.d_rope;
  }
  const int half = A.d_rope / 2;
  if (h >= hi) {
    if (lane >= half) return;
    const int head = h - hi;
    const int a = A.rope.interleaved ? 2 * lane : lane, b = A.rope.interleaved ? 2 * lane + 1 : lane + half;
    const __nv_bfloat16* src = A.q_pe + t * A.pe_token + head * A.pe_head;
    float x0 = __bfloat162float(src[a]), x1 = __bfloat162float(src[b]);
    if (cs) {
      const float c = __ldg(cs + lane), s = __ldg(cs + half + lane);
      const float y0 = x0 * c - x1 * s;
      x1 = x0 * s + x1 * c;
      x0 = y0;
    }
    __nv_bfloat16* dst = A.q_pe_out + (t * A.n_heads + head) * A.d_rope;
    dst[a] = __float2bfloat16_rn(x0);
    dst[b] = __float2bfloat16_rn(x1);
    return;
  }
  float z[EK];
  load_bf16<EK>(A.q_idx + t * A.idx_token + h * A.idx_head + lane * EK, A.vec_idx, z);
  if (A.idx_norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < EK; ++i) ss += z[i] * z[i];
    const float rstd = rsqrtf(warp_sum(ss) / static_cast<float>(32 * EK) + A.eps);
#pragma unroll
    for (int i = 0; i < EK; ++i) z[i] = z[i] * rstd * __ldg(A.idx_norm + lane * EK + i);
  }
  if (cs && A.rope.idx_rope) rotate_row<EK>(z, cs, A.d_rope, A.rope.idx_interleaved, stage[warp], lane);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < EK; ++i) amax = fmaxf(amax, fabsf(z[i]));
  float scale, inv;
  quant_scale(warp_max(amax), kRE4M3, scale, inv);
  uint8_t* dst = A.codes + (t * A.n_idx_heads + h) * A.d_index + lane * EK;
#pragma unroll
  for (int i = 0; i < EK; ++i) dst[i] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(z[i] * inv, __NV_SATFINITE, __NV_E4M3));
  if (lane == 0) A.w_out[t * A.n_idx_heads + h] = __ldg(A.w + t * A.n_idx_heads + h) * A.w_scale * scale;
}

// Eight lanes hold 64 dims, lane j dims 4 j .. + 3 and 32 + 4 j .. + 3: every rotation pair lies in one lane,
// whether it is (i, i + 32) or (2 i, 2 i + 1), and rows load and store in whole sectors.
// Cosines and sines of the lane's four pairs: halves, pairs 4 j .. + 3; interleaved, 2 j, 2 j + 1, 16 + 2 j, 17 + 2 j.
__device__ __forceinline__ void load_angles(const float* cs, int j, bool interleaved, float (&c)[4], float (&sn)[4]) {
  if (interleaved) {
    const float2 a = __ldg(reinterpret_cast<const float2*>(cs) + j), b = __ldg(reinterpret_cast<const float2*>(cs) + 8 + j);
    const float2 d = __ldg(reinterpret_cast<const float2*>(cs) + 16 + j), e = __ldg(reinterpret_cast<const float2*>(cs) + 24 + j);
    c[0] = a.x, c[1] = a.y, c[2] = b.x, c[3] = b.y;
    sn[0] = d.x, sn[1] = d.y, sn[2] = e.x, sn[3] = e.y;
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(cs) + j), d = __ldg(reinterpret_cast<const float4*>(cs) + 8 + j);
    c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
    sn[0] = d.x, sn[1] = d.y, sn[2] = d.z, sn[3] = d.w;
  }
}

__device__ __forceinline__ void rotate8(float (&x)[8], const float (&c)[4], const float (&sn)[4], bool interleaved) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (interleaved) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * sn[i];
      x[2 * i + 1] = a * sn[i] + b * c[i];
    } else {
      const float a = x[i], b = x[i + 4];
      x[i] = a * c[i] - b * sn[i];
      x[i + 4] = a * sn[i] + b * c[i];
    }
  }
}

// The lane's eight bf16 of a row (p: the row's 64 dims) and its eight fp32 of a weight vector.
struct Raw8 {
  uint2 lo, hi;
};
__device__ __forceinline__ Raw8 load_raw8(const __nv_bfloat16* p, int j) {
  return {__ldg(reinterpret_cast<const uint2*>(p) + j), __ldg(reinterpret_cast<const uint2*>(p) + 8 + j)};
}
__device__ __forceinline__ void unpack8(const Raw8& w, float (&x)[8]) {
  const uint32_t ws[4] = {w.lo.x, w.lo.y, w.hi.x, w.hi.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(ws[i] << 16);
    x[2 * i + 1] = __uint_as_float(ws[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, int j, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p) + j), b = __ldg(reinterpret_cast<const float4*>(p) + 8 + j);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store_codes8(uint8_t* p, int j, const float (&x)[8], float inv) {
  reinterpret_cast<uint32_t*>(p)[j] = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
  reinterpret_cast<uint32_t*>(p)[8 + j] = e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16;
}
__device__ __forceinline__ void store_bf16x8(__nv_bfloat16* p, int j, const float (&x)[8]) {
  reinterpret_cast<uint2*>(p)[j] = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  reinterpret_cast<uint2*>(p)[8 + j] = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// sum and maximum over the half-warp
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float half_max8(const float (&x)[8]) {
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v = fmaxf(v, fabsf(x[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// kvpack_append for the full shape (512 latent dims in tiles of 128, 64 rope and 128 indexer dims), 16-byte
// aligned rows: two warps per token, since a token's two parts do not meet and a few tokens are a matter of
// latency.  Warp 0: the latent, 64 dims to eight lanes twice (dims 0-255, then the others), so that a
// quantisation tile is a half-warp.  Warp 1: the indexer key in its first half-warp and the rope key in eight
// lanes of the second.
// 8,192 tokens (20 MB with their records) take 8.0 us with inputs in L2, 2.5 TB/s, launch included (the kernel
// above, a warp per token with byte stores for the key: 15.2), 11.5 us from DRAM, one token 2.7 us (3.7): the
// chain slot -> row -> sums -> codes, a launch and, for the chunk, instructions (68 % of the issue slots), not
// bandwidth.  So as many warps as the SM holds: with 40 registers a thread instead of 32 a chunk from DRAM took
// 1.3 us more, one token 0.2 less (1, 2 or 8 tokens a CTA: the same).
constexpr int kAppendTokens = 4;  // of a CTA
template <bool kFp4>
__global__ void __launch_bounds__(64 * kAppendTokens, 8) append_full_kernel(const AppendArgs A) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kAppendTokens + (warp >> 1);
  if (t >= A.n_tokens) return;
  const KernelLayout& L = A.L;
  const int64_t slot = __ldg(A.slots + t);
  const int64_t pos = A.rope.cos_sin ? __ldg(A.rope.positions + t) : 0;
  const int j = lane & 7, g = lane >> 3;  // the lane's place in its 64 dims, and which 64 dims
  const bool key_part = (warp & 1) != 0, is_key = lane < 16;
  Raw8 v0 = {}, v1 = {};
  if (!key_part) {
    const __nv_bfloat16* src = A.latent + t * A.latent_stride + 64 * g;
    v0 = load_raw8(src, j);
    v1 = load_raw8(src + 256, j);
  } else if (is_key) {
    if (A.idx_k) v0 = load_raw8(A.idx_k + t * A.idx_stride + 64 * g, j);
  } else {
    v0 = load_raw8(A.rope_key + t * A.rope_stride, j);  // lanes 24-31 as 16-23
  }
  if (slot < 0) return;
  if (slot >= L.num_blocks * L.block_size || (A.rope.cos_sin && (pos < 0 || pos >= A.rope.n_positions))) {
    if (lane == 0) latch_error(A.err, SMLA_ERR_BAD_INDEX);
    return;
  }
  const int64_t blk = slot / L.block_size;
  const int off = static_cast<int>(slot - blk * L.block_size);
  uint8_t* base = A.pool + blk * L.block_stride + static_cast<int64_t>(A.layer) * L.layer_stride;
  uint8_t* rec = base + L.rec_off + static_cast<int64_t>(off) * L.rec_stride;
  float x[8], w[8];
  unpack8(v0, x);
  if (!key_part) {
    float y[8];
    unpack8(v1, y);
    if (A.latent_norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
      const float rstd = rsqrtf(warp_sum(ss) / 512.0f + A.eps);
      load8(A.latent_norm + 64 * g, j, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * rstd * w[i];
      load8(A.latent_norm + 256 + 64 * g, j, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * w[i];
    }
    float sx, ix, sy, iy;
    quant_scale(half_max8(x), kRE4M3, sx, ix);
    quant_scale(half_max8(y), kRE4M3, sy, iy);
    store_codes8(rec + 64 * g, j, x, ix);
    store_codes8(rec + 256 + 64 * g, j, y, iy);
    if ((lane & 15) == 0) {
      float* sc = reinterpret_cast<float*>(rec + 512) + (lane >> 4);
      sc[0] = sx;
      sc[2] = sy;
    }
    return;
  }
  const float* cs = A.rope.cos_sin ? A.rope.cos_sin + pos * 64 : nullptr;
  // the norm of the key, in the first half-warp (the sums of the second are not used)
  if (A.idx_k && A.idx_norm) {
    const float mean = A.idx_bias ? half_sum(((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]))) / 128.0f : 0.f;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += (x[i] - mean) * (x[i] - mean);
    const float rstd = rsqrtf(half_sum(ss) / 128.0f + A.eps);
    if (is_key) {
      load8(A.idx_norm + 64 * g, j, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (x[i] - mean) * rstd * w[i];
      if (A.idx_bias) {
        load8(A.idx_bias + 64 * g, j, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += w[i];
      }
    }
  }
  if (cs && (is_key ? g == 0 && A.rope.idx_rope : true)) {
    float c[4], sn[4];
    const bool interleaved = is_key ? A.rope.idx_interleaved : A.rope.interleaved;
    load_angles(cs, j, interleaved, c, sn);
    rotate8(x, c, sn, interleaved);
  }
  __syncwarp();
  const float amax = half_max8(x);
  if (!is_key) {
    if (lane < 24) store_bf16x8(reinterpret_cast<__nv_bfloat16*>(rec + 528), j, x);
    return;
  }
  if (!A.idx_k) return;
  float scale, inv;
  quant_scale(amax, kFp4 ? kRE2M1 : kRE4M3, scale, inv);
  uint8_t* kdst = base + L.idx_key_off + static_cast<int64_t>(off) * L.key_bytes;
  if constexpr (kFp4) {
    const auto four = [&](int i) -> uint16_t {  // elements i .. i + 3
      return static_cast<uint16_t>(__nv_cvt_float2_to_fp4x2(make_float2(x[i] * inv, x[i + 1] * inv), __NV_E2M1, cudaRoundNearest) |
                                   __nv_cvt_float2_to_fp4x2(make_float2(x[i + 2] * inv, x[i + 3] * inv), __NV_E2M1, cudaRoundNearest) << 8);
    };
    uint16_t* q = reinterpret_cast<uint16_t*>(kdst + 32 * g);
    q[j] = four(0);
    q[8 + j] = four(4);
  } else {
    store_codes8(kdst + 64 * g, j, x, inv);
  }
  if (lane == 0) reinterpret_cast<float*>(base + L.idx_scale_off)[off] = scale;
}

// Two floats in a register pair: packed fp32 operations take half the issue slots.
__device__ __forceinline__ uint64_t pair_of(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 of_pair(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)));
  return of_pair(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)), "l"(pair_of(c)));
  return of_pair(r);
}

// The lane's eight values x of 64 dims as pairs (x0, x2), (x1, x3), (x4, x6), (x5, x7): both kinds of
// rotation pairs then meet in packed operations.
__device__ __forceinline__ void unpack_pairs(const Raw8& w, float2* x) {
  x[0] = make_float2(__uint_as_float(w.lo.x << 16), __uint_as_float(w.lo.y << 16));
  x[1] = make_float2(__uint_as_float(w.lo.x & 0xFFFF0000u), __uint_as_float(w.lo.y & 0xFFFF0000u));
  x[2] = make_float2(__uint_as_float(w.hi.x << 16), __uint_as_float(w.hi.y << 16));
  x[3] = make_float2(__uint_as_float(w.hi.x & 0xFFFF0000u), __uint_as_float(w.hi.y & 0xFFFF0000u));
}
struct Turn {
  float2 c[2], s[2], n[2];  // cosines, sines, minus the sines
};
__device__ __forceinline__ void load_turn(const float* cs, int j, bool interleaved, Turn& u) {
  float c[4], s[4];
  load_angles(cs, j, interleaved, c, s);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    u.c[i] = interleaved ? make_float2(c[2 * i], c[2 * i + 1]) : make_float2(c[i], c[i + 2]);
    u.s[i] = interleaved ? make_float2(s[2 * i], s[2 * i + 1]) : make_float2(s[i], s[i + 2]);
    u.n[i] = make_float2(-u.s[i].x, -u.s[i].y);
  }
}
__device__ __forceinline__ void turn2(float2& a, float2& b, float2 c, float2 s, float2 n) {
  const float2 a0 = a;
  a = fma2(b, n, mul2(a, c));
  b = fma2(a0, s, mul2(b, c));
}
__device__ __forceinline__ void rotate_pairs(float2* x, const Turn& u, bool interleaved) {
  if (interleaved) {
    turn2(x[0], x[1], u.c[0], u.s[0], u.n[0]);
    turn2(x[2], x[3], u.c[1], u.s[1], u.n[1]);
  } else {
    turn2(x[0], x[2], u.c[0], u.s[0], u.n[0]);
    turn2(x[1], x[3], u.c[1], u.s[1], u.n[1]);
  }
}

// smla_query_prep for 128 indexer dims and 64 rope dims, everything 16-byte aligned: one CTA per token.  Eight
// lanes hold a head (the lanes' dims: above; an indexer head's dims 64-127 likewise), so that a row's sum
// and maximum are three shuffles each, its rotation none, and the angles, loaded once a token, stay in
// registers for all heads.  A norm's 1 / rms scales the whole row: only the row's scale sees it, its codes
// are those of the row without it.
// Bound by memory: 8,192 tokens of 64 + 64 heads move 342 MB in 58.7 us, 5.8 TB/s (a warp per row, with
// rotations through shared memory and byte stores, the kernel above: 243 us; sixteen lanes a head, unpacked
// fp32 and every warp at both kinds of heads: 70 us, bound by its instructions).
// Three warps a token leave the SM eight tokens at a time and most loads in flight; a step of a few tokens
// is a matter of latency and takes twelve warps, as long as all of its CTAs (two an SM) run at once:
// 1 token 2.3 us against 3.5 with three warps, 256 tokens 3.1 against 4.1, 512 tokens 5.0 against 4.7,
// 8,192 tokens 86 against 58.7.
constexpr int kQWarps = 12;  // of a CTA, at most; a multiple of three
__global__ void __launch_bounds__(32 * kQWarps, 2) query_full_kernel(const QueryArgs A) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int64_t t = blockIdx.x;
  const int sub = lane >> 3, j = lane & 7;  // the lane's head of four, its place in 64 dims
  const int idx_quads = A.q_idx ? (A.n_idx_heads + 3) / 4 : 0, pe_quads = A.q_pe ? (A.n_heads + 3) / 4 : 0;
  // a third of the warps takes q_pe (64 dims a head against 128)
  const int pe_warps = pe_quads == 0 ? 0 : idx_quads == 0 ? warps : warps / 3;
  const float* cs = nullptr;
  int64_t pos = 0;
  if (A.rope.cos_sin) pos = __ldg(A.rope.positions + t);
  const auto angles = [&]() -> bool {
    if (A.rope.cos_sin == nullptr) return true;
    if (pos < 0 || pos >= A.rope.n_positions) {
      if (threadIdx.x == 0) latch_error(A.err, SMLA_ERR_BAD_INDEX);
      return false;
    }
    cs = A.rope.cos_sin + pos * 64;
    return true;
  };
  Turn u;
  if (warp < pe_warps) {  // ---- q_pe ----
    constexpr int kIt = 4;
    Raw8 v[kIt];
    const auto ask = [&](int i, int it) {
      const int h = 4 * it + sub;
      v[i] = Raw8{};
      if (it < pe_quads && h < A.n_heads) v[i] = load_raw8(A.q_pe + t * A.pe_token + h * A.pe_head, j);
    };
    // the first rows are asked for before the position is known to be good
#pragma unroll
    for (int i = 0; i < kIt; ++i) ask(i, warp + pe_warps * i);
    if (!angles()) return;
    if (cs != nullptr) load_turn(cs, j, A.rope.interleaved, u);
#pragma unroll 1
    for (int it0 = warp; it0 < pe_quads; it0 += pe_warps * kIt) {
#pragma unroll
      for (int i = 0; i < kIt; ++i) {
        const int it = it0 + pe_warps * i, h = 4 * it + sub;
        if (it >= pe_quads) break;
        float2 x[4];
        unpack_pairs(v[i], x);
        ask(i, it + pe_warps * kIt);
        if (cs != nullptr) rotate_pairs(x, u, A.rope.interleaved);
        if (h < A.n_heads) {
          uint2* dst = reinterpret_cast<uint2*>(A.q_pe_out + (t * A.n_heads + h) * 64) + j;
          dst[0] = make_uint2(pack_bf16x2(x[0].x, x[1].x), pack_bf16x2(x[0].y, x[1].y));
          dst[8] = make_uint2(pack_bf16x2(x[2].x, x[3].x), pack_bf16x2(x[2].y, x[3].y));
        }
      }
    }
    return;
  }
  // ---- indexer heads ----
  const int step = warps - pe_warps;
  constexpr int kIt = 2;
  Raw8 v[kIt][2];
  float wv[kIt];
  const auto ask = [&](int i, int it) {
    const int h = 4 * it + sub;
    v[i][0] = v[i][1] = Raw8{};
    wv[i] = 0.f;
    if (it < idx_quads && h < A.n_idx_heads) {
      const __nv_bfloat16* src = A.q_idx + t * A.idx_token + h * A.idx_head;
      v[i][0] = load_raw8(src, j);
      v[i][1] = load_raw8(src + 64, j);
      wv[i] = __ldg(A.w + t * A.n_idx_heads + h);
    }
  };
#pragma unroll
  for (int i = 0; i < kIt; ++i) ask(i, warp - pe_warps + step * i);
  if (!angles()) return;
  const bool turn = cs != nullptr && A.rope.idx_rope;
  if (turn) load_turn(cs, j, A.rope.idx_interleaved, u);
#pragma unroll 1
  for (int it0 = warp - pe_warps; it0 < idx_quads; it0 += step * kIt) {
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int it = it0 + step * i, h = 4 * it + sub;
      if (it >= idx_quads) break;
      float2 x[8];
      unpack_pairs(v[i][0], x);
      unpack_pairs(v[i][1], x + 4);
      const float weight = wv[i];
      ask(i, it + step * kIt);
      float rstd = 1.f;
      if (A.idx_norm) {
        float2 ss = mul2(x[0], x[0]), sr = mul2(x[1], x[1]);
#pragma unroll
        for (int e = 2; e < 8; e += 2) {
          ss = fma2(x[e], x[e], ss);
          sr = fma2(x[e + 1], x[e + 1], sr);
        }
        float sum = (ss.x + sr.x) + (ss.y + sr.y);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        rstd = rsqrtf(sum / 128.0f + A.eps);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {  // read again for every head: sixteen registers less are a CTA more
          float4 w;
          asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
                       : "l"(A.idx_norm + 16 * e + 4 * j));
          x[e] = mul2(x[e], make_float2(w.x, w.z));
          x[e + 1] = mul2(x[e + 1], make_float2(w.y, w.w));
        }
      }
      if (turn) rotate_pairs(x, u, A.rope.idx_interleaved);
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      float scale, inv;
      quant_scale(amax * rstd, kRE4M3, scale, inv);
      inv *= rstd;
      if (h < A.n_idx_heads) {
        const int64_t row = t * A.n_idx_heads + h;
        uint32_t* dst = reinterpret_cast<uint32_t*>(A.codes + row * 128) + j;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = mul2(x[e], make_float2(inv, inv));
#pragma unroll
        for (int e = 0; e < 8; e += 2)  // x0 .. x3 and x4 .. x7 of either half
          dst[8 * (e >> 1)] = e4m3x2(x[e].x, x[e + 1].x) | e4m3x2(x[e].y, x[e + 1].y) << 16;
        if (j == 0) A.w_out[row] = weight * A.w_scale * scale;
      }
    }
  }
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// SMLA_ERR_INVALID_ARG for a rotation that cannot be applied to these dims.
smla_status_t check_rope(const smla_rope_t* rope, const int64_t* positions, int d_rope, int d_index, bool indexer) {
  if (rope == nullptr) return SMLA_OK;
  if (!rope->cos_sin || !aligned(rope->cos_sin, 4) || rope->n_positions <= 0 || !positions) return SMLA_ERR_INVALID_ARG;
  if (indexer && rope->idx_rope && d_rope > d_index) return SMLA_ERR_INVALID_ARG;
  return SMLA_OK;
}

RopeArgs rope_args(const smla_rope_t* rope, const int64_t* positions, int d_rope) {
  RopeArgs r{};
  r.d_rope = d_rope;
  if (rope != nullptr && d_rope > 0) {
    r.cos_sin = rope->cos_sin;
    r.n_positions = rope->n_positions;
    r.positions = positions;
    r.interleaved = rope->interleaved != 0;
    r.idx_interleaved = rope->idx_interleaved != 0;
    r.idx_rope = rope->idx_rope != 0;
  }
  return r;
}

bool index_dims_supported(int d_index) { return d_index == 32 || d_index == 64 || d_index == 128 || d_index == kMaxIndex; }

template <int E>
void launch_append(const AppendArgs& A, int d_index, cudaStream_t s) {
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(A.n_tokens) + kWarps - 1) / kWarps);
  switch (d_index) {
    case 32: append_kernel<E, 1><<<blocks, 32 * kWarps, 0, s>>>(A); break;
    case 64: append_kernel<E, 2><<<blocks, 32 * kWarps, 0, s>>>(A); break;
    case 128: append_kernel<E, 4><<<blocks, 32 * kWarps, 0, s>>>(A); break;
    default: append_kernel<E, 8><<<blocks, 32 * kWarps, 0, s>>>(A); break;
  }
}

}  // namespace
}  // namespace smla

using namespace smla;

extern "C" smla_status_t kvpack_append(const smla_layout_t* layout, void* pool, int layer, const void* latent,
                                       int64_t latent_stride, const void* rope_key, int64_t rope_stride,
                                       const void* idx_k, int64_t idx_k_stride, const float* latent_norm,
                                       const float* idx_norm, const float* idx_bias, float eps,
                                       const smla_rope_t* rope, const int64_t* positions, const int64_t* slot_mapping,
                                       int n_tokens, void* stream) {
  if (!layout_ok(layout) || n_tokens < 0 || layer < 0 || layer >= layout->n_layers) return SMLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return SMLA_OK;
  const bool idx = idx_k != nullptr;
  if (!pool || !aligned(pool, 16) || !latent || !slot_mapping || (layout->d_rope > 0 && !rope_key) ||
      latent_stride < 0 || rope_stride < 0 || idx_k_stride < 0 || (idx_bias && !idx_norm) || !(eps >= 0.f))
    return SMLA_ERR_INVALID_ARG;
  smla_status_t st = check_rope(rope, positions, layout->d_rope, layout->d_index, idx);
  if (st != SMLA_OK) return st;
  const KernelLayout L = kernel_layout(*layout);
  if (!store_shape_supported(L) || L.d_rope > 64 || !index_dims_supported(L.d_index)) return SMLA_ERR_UNSUPPORTED;
  AppendArgs A{};
  st = checked_device(&A.err);
  if (st != SMLA_OK) return st;
  A.L = L;
  A.pool = static_cast<uint8_t*>(pool);
  A.layer = layer;
  A.latent = static_cast<const __nv_bfloat16*>(latent);
  A.rope_key = static_cast<const __nv_bfloat16*>(rope_key);
  A.idx_k = static_cast<const __nv_bfloat16*>(idx_k);
  A.latent_stride = latent_stride;
  A.rope_stride = rope_stride;
  A.idx_stride = idx_k_stride;
  A.latent_norm = latent_norm;
  A.idx_norm = idx_norm;
  A.idx_bias = idx_bias;
  A.eps = eps;
  A.rope = rope_args(rope, positions, L.d_rope);
  A.slots = slot_mapping;
  A.n_tokens = n_tokens;
  A.vec_latent = aligned(latent, 16) && latent_stride % 8 == 0;
  A.vec_idx = aligned(idx_k, 16) && idx_k_stride % 8 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // The full shape with rows that load as 16-byte pieces takes the kernel built for it (half the time at 8,192
  // tokens, two thirds at one: see there).
  if (L.d_latent == 512 && L.quant_tile == 128 && L.d_rope == 64 && L.d_index == 128 && A.vec_latent &&
      aligned(rope_key, 16) && rope_stride % 8 == 0 && (!idx || A.vec_idx) && aligned(latent_norm, 16) &&
      aligned(idx_norm, 16) && aligned(idx_bias, 16) && aligned(A.rope.cos_sin, 16)) {
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(n_tokens) + kAppendTokens - 1) / kAppendTokens);
    if (L.key_format == SMLA_KEY_E2M1) append_full_kernel<true><<<blocks, 64 * kAppendTokens, 0, s>>>(A);
    else append_full_kernel<false><<<blocks, 64 * kAppendTokens, 0, s>>>(A);
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
  }
  switch (L.d_latent / 32) {
    case 2: launch_append<2>(A, L.d_index, s); break;
    case 4: launch_append<4>(A, L.d_index, s); break;
    case 8: launch_append<8>(A, L.d_index, s); break;
    default: launch_append<16>(A, L.d_index, s); break;
  }
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}

extern "C" smla_status_t smla_query_prep(const smla_layout_t* layout, const smla_params_t* params,
                                         const smla_rope_t* rope, const int64_t* positions, const void* q_pe,
                                         int64_t q_pe_token_stride, int64_t q_pe_head_stride, void* q_pe_out,
                                         const void* q_idx, int64_t q_idx_token_stride, int64_t q_idx_head_stride,
                                         const float* idx_norm, float eps, const float* w, float w_scale,
                                         uint8_t* q_idx_out, float* w_out, int n_tokens, void* stream) {
  if (!layout_ok(layout) || !params || n_tokens < 0) return SMLA_ERR_INVALID_ARG;
  if (n_tokens == 0) return SMLA_OK;
  const bool pe = q_pe != nullptr, idx = q_idx != nullptr;
  if ((pe && (!q_pe_out || params->n_heads <= 0 || layout->d_rope <= 0 || q_pe_token_stride < 0 || q_pe_head_stride < 0)) ||
      (idx && (!w || !q_idx_out || !w_out || params->n_idx_heads <= 0 || q_idx_token_stride < 0 ||
               q_idx_head_stride < 0)) ||
      !(eps >= 0.f))
    return SMLA_ERR_INVALID_ARG;
  if (!pe && !idx) return SMLA_OK;
  smla_status_t st = check_rope(rope, positions, layout->d_rope, layout->d_index, idx);
  if (st != SMLA_OK) return st;
  if (layout->d_rope > 64 || (idx && !index_dims_supported(layout->d_index))) return SMLA_ERR_UNSUPPORTED;
  QueryArgs A{};
  st = checked_device(&A.err);
  if (st != SMLA_OK) return st;
  A.q_pe = static_cast<const __nv_bfloat16*>(q_pe);
  A.q_idx = static_cast<const __nv_bfloat16*>(q_idx);
  A.pe_token = q_pe_token_stride;
  A.pe_head = q_pe_head_stride;
  A.idx_token = q_idx_token_stride;
  A.idx_head = q_idx_head_stride;
  A.q_pe_out = static_cast<__nv_bfloat16*>(q_pe_out);
  A.idx_norm = idx_norm;
  A.w = w;
  A.eps = eps;
  A.w_scale = w_scale;
  A.codes = q_idx_out;
  A.w_out = w_out;
  A.n_tokens = n_tokens;
  A.n_heads = params->n_heads;
  A.n_idx_heads = params->n_idx_heads;
  A.d_rope = layout->d_rope;
  A.d_index = layout->d_index;
  A.rope = rope_args(rope, positions, layout->d_rope);
  A.vec_idx = aligned(q_idx, 16) && q_idx_token_stride % 8 == 0 && q_idx_head_stride % 8 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Rows that load as 16-byte pieces take the kernel built for them (a quarter of the time at 8,192 tokens: see there).
  if ((!idx || (layout->d_index == 128 && A.vec_idx && aligned(q_idx_out, 8) && aligned(idx_norm, 16))) &&
      (layout->d_rope == 64 || (!pe && !(A.rope.cos_sin && A.rope.idx_rope))) &&
      (!pe || (aligned(q_pe, 16) && q_pe_token_stride % 8 == 0 && q_pe_head_stride % 8 == 0 && aligned(q_pe_out, 16))) &&
      aligned(A.rope.cos_sin, 16)) {
    query_full_kernel<<<n_tokens, 32 * (n_tokens <= 2 * device_sm_count() ? kQWarps : 3), 0, s>>>(A);
    return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
  }
  const int64_t rows = static_cast<int64_t>(n_tokens) * ((pe ? A.n_heads : 0) + (idx ? A.n_idx_heads : 0));
  if ((rows + kWarps - 1) / kWarps > 0x7fffffff) return SMLA_ERR_UNSUPPORTED;
  const unsigned blocks = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
  switch (idx ? layout->d_index : 32) {
    case 32: query_kernel<1><<<blocks, 32 * kWarps, 0, s>>>(A); break;
    case 64: query_kernel<2><<<blocks, 32 * kWarps, 0, s>>>(A); break;
    case 128: query_kernel<4><<<blocks, 32 * kWarps, 0, s>>>(A); break;
    default: query_kernel<8><<<blocks, 32 * kWarps, 0, s>>>(A); break;
  }
  return cudaGetLastError() == cudaSuccess ? SMLA_OK : SMLA_ERR_CUDA;
}
