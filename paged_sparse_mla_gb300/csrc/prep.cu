// kvpack_append and smla_query_prep: from a layer's projections to the cache and to the queries.
//
// [GLM-5.3 "How to try", "Config and numbers"]: the KV cache is FP8.  [AgentX "Hybrid KV cache
// management"]: one packed allocation per block holds every cache group.  [AgentX "DeepSeek V4"]: 64
// indexer heads a token.
//
// Norm, position rotation, quantisation and the scatter (or the head weight) are one pass: a row is
// read once as bf16, kept in fp32 registers (in shared memory only where a rotation pairs elements of
// different lanes) and leaves as codes.  The normalised values are not rounded to bf16 before they are
// quantised: that rounding (2^-9) would only add to the code's (2^-4).
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

// One warp per token: lane l owns latent elements [E l, E l + E) and key elements [EK l, EK l + EK).
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

// One warp per row: rows [0, n_idx_heads) of a token are its indexer heads, the next n_heads its q_pe.
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

// Cosines and sines for the eight consecutive elements that start at element 8 s of a vector whose first 64
// elements rotate: interleaved, those of pairs 4 s .. + 3 (in the first four); halves, those of pairs
// 8 (s % 4) .. + 7 with the sine's sign as the element's place in its pair wants it.  Past the rotated
// elements (s >= 8) the angle is zero.
__device__ __forceinline__ void load_angles(const float* cs, int s, bool interleaved, float (&c)[8], float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    sn[i] = 0.f;
  }
  if (s >= 8) return;
  const float4* p = reinterpret_cast<const float4*>(cs + (interleaved ? 4 * s : 8 * (s & 3)));
  const float4 a = __ldg(p), b = __ldg(p + 8);
  c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
  sn[0] = b.x, sn[1] = b.y, sn[2] = b.z, sn[3] = b.w;
  if (interleaved) return;
  const float4 d = __ldg(p + 1), e = __ldg(p + 9);
  c[4] = d.x, c[5] = d.y, c[6] = d.z, c[7] = d.w;
  sn[4] = e.x, sn[5] = e.y, sn[6] = e.z, sn[7] = e.w;
  if (s < 4) {  // first elements: a c - b s, second: b c + a s
#pragma unroll
    for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
  }
}

// Rotates a lane's eight consecutive elements; halves pair with the lane four away.
__device__ __forceinline__ void rotate8(float (&x)[8], const float (&c)[8], const float (&sn)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * sn[i];
      x[2 * i + 1] = a * sn[i] + b * c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + __shfl_xor_sync(0xffffffffu, x[i], 4) * sn[i];
  }
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(ws[i] << 16);
    x[2 * i + 1] = __uint_as_float(ws[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  return make_uint2(e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16,
                    e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16);
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
// latency.  Warp 0: the latent, a lane dims 8 l .. + 7 and 256 + 8 l .. + 7, so that rows, norm weights and
// codes are coalesced and a quantisation tile is a half-warp.  Warp 1: the indexer key (eight dims a lane of
// the first half-warp) and the rope key (eight lanes of the second).
constexpr int kAppendTokens = 4;  // of a CTA
template <bool kFp4>
__global__ void __launch_bounds__(64 * kAppendTokens) append_full_kernel(const AppendArgs A) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kAppendTokens + (warp >> 1);
  if (t >= A.n_tokens) return;
  const KernelLayout& L = A.L;
  const int64_t slot = __ldg(A.slots + t);
  const int64_t pos = A.rope.cos_sin ? __ldg(A.rope.positions + t) : 0;
  const int sub = lane & 15, s8 = lane & 7;
  const bool key_part = (warp & 1) != 0, is_key = lane < 16;
  uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
  if (!key_part) {
    const uint4* src = reinterpret_cast<const uint4*>(A.latent + t * A.latent_stride);
    v0 = __ldg(src + lane);
    v1 = __ldg(src + 32 + lane);
  } else if (is_key) {
    if (A.idx_k) v0 = __ldg(reinterpret_cast<const uint4*>(A.idx_k + t * A.idx_stride) + sub);
  } else {
    v0 = __ldg(reinterpret_cast<const uint4*>(A.rope_key + t * A.rope_stride) + s8);  // lanes 24-31 as 16-23
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
      load8(A.latent_norm + 8 * lane, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * rstd * w[i];
      load8(A.latent_norm + 256 + 8 * lane, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * rstd * w[i];
    }
    float sx, ix, sy, iy;
    quant_scale(half_max8(x), kRE4M3, sx, ix);
    quant_scale(half_max8(y), kRE4M3, sy, iy);
    reinterpret_cast<uint2*>(rec)[lane] = codes8(x, ix);
    reinterpret_cast<uint2*>(rec)[32 + lane] = codes8(y, iy);
    if (sub == 0) {
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
      load8(A.idx_norm + 8 * sub, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = (x[i] - mean) * rstd * w[i];
      if (A.idx_bias) {
        load8(A.idx_bias + 8 * sub, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += w[i];
      }
    }
  }
  // Key and rope may pair their elements differently: the halves' exchange is done for both and taken where
  // it belongs.
  if (cs) {
    const bool inter = is_key ? A.rope.idx_interleaved : A.rope.interleaved;
    const int s = is_key ? (A.rope.idx_rope ? sub : 8) : s8;
    float c[8], sn[8];
    load_angles(cs, s, inter, c, sn);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __shfl_xor_sync(0xffffffffu, x[i], 4);
    if (inter) {
      rotate8(x, c, sn, true);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + w[i] * sn[i];
    }
  }
  const float amax = half_max8(x);
  if (!is_key) {
    if (lane < 24)
      reinterpret_cast<uint4*>(rec + 528)[s8] =
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    return;
  }
  if (!A.idx_k) return;
  float scale, inv;
  quant_scale(amax, kFp4 ? kRE2M1 : kRE4M3, scale, inv);
  uint8_t* kdst = base + L.idx_key_off + static_cast<int64_t>(off) * L.key_bytes;
  if constexpr (kFp4) {
    uint32_t q = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_E2M1, cudaRoundNearest)) << (8 * i);
    reinterpret_cast<uint32_t*>(kdst)[sub] = q;
  } else {
    reinterpret_cast<uint2*>(kdst)[sub] = codes8(x, inv);
  }
  if (sub == 0) reinterpret_cast<float*>(base + L.idx_scale_off)[off] = scale;
}

// smla_query_prep for 128 indexer dims and 64 rope dims, everything 16-byte aligned: one CTA per token.  Sixteen
// lanes hold an indexer head (eight dims each), eight lanes a q_pe head, so that a row is one coalesced
// 16-byte load a lane, its sums and maxima four shuffles, and the angles, loaded once a token, stay in
// registers for all heads.  Bound by memory: 8,192 tokens of 64 + 64 heads, 342 MB, QUERY_FIGURE (the kernel above, a
// warp per row with rotations through shared memory and byte stores: 254 us).
constexpr int kQWarps = 8;
__global__ void __launch_bounds__(32 * kQWarps) query_full_kernel(const QueryArgs A) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int sub = lane & 15, hi = lane >> 4, s8 = lane & 7;
  const float* cs = nullptr;
  int64_t pos = 0;
  if (A.rope.cos_sin) pos = __ldg(A.rope.positions + t);
  // the first rows are asked for before the position is known to be good
  constexpr int kIt = 4;
  uint4 v[kIt];
  float wv[kIt];
  uint8_t* codes = A.codes + t * A.n_idx_heads * 128;
  const int idx_pairs = A.q_idx ? (A.n_idx_heads + 1) / 2 : 0;
  const auto ask = [&](int i, int it) {
    const int h = 2 * it + hi;
    v[i] = make_uint4(0, 0, 0, 0);
    wv[i] = 0.f;
    if (it < idx_pairs && h < A.n_idx_heads) {
      v[i] = __ldg(reinterpret_cast<const uint4*>(A.q_idx + t * A.idx_token + h * A.idx_head) + sub);
      wv[i] = __ldg(A.w + t * A.n_idx_heads + h);
    }
  };
#pragma unroll
  for (int i = 0; i < kIt; ++i) ask(i, warp + kQWarps * i);
  const int pe_quads = A.q_pe ? (A.n_heads + 3) / 4 : 0;
  constexpr int kPe = 2;
  uint4 pv[kPe];
  const auto ask_pe = [&](int it) -> uint4 {
    const int h = 4 * it + (lane >> 3);
    if (it < pe_quads && h < A.n_heads)
      return __ldg(reinterpret_cast<const uint4*>(A.q_pe + t * A.pe_token + h * A.pe_head) + s8);
    return make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int i = 0; i < kPe; ++i) pv[i] = ask_pe(warp + kQWarps * i);
  float c[8], sn[8], norm[8];
  if (A.rope.cos_sin) {
    if (pos < 0 || pos >= A.rope.n_positions) {
      if (threadIdx.x == 0) latch_error(A.err, SMLA_ERR_BAD_INDEX);
      return;
    }
    cs = A.rope.cos_sin + pos * 64;
  }
  // ---- indexer heads ----
  const bool turn = cs != nullptr && A.rope.idx_rope;
  if (idx_pairs > 0) {
    if (turn) load_angles(cs, sub, A.rope.idx_interleaved, c, sn);
    if (A.idx_norm) load8(A.idx_norm + 8 * sub, norm);
  }
  for (int it0 = warp; it0 < idx_pairs; it0 += kQWarps * kIt) {
#pragma unroll
    for (int i = 0; i < kIt; ++i) {
      const int it = it0 + kQWarps * i, h = 2 * it + hi;
      if (it >= idx_pairs) break;
      float x[8];
      unpack8(v[i], x);
      if (A.idx_norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
        const float rstd = rsqrtf(half_sum(ss) / 128.0f + A.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * norm[e];
      }
      if (turn) rotate8(x, c, sn, A.rope.idx_interleaved);
      float scale, inv;
      quant_scale(half_max8(x), kRE4M3, scale, inv);
      if (h < A.n_idx_heads) {
        reinterpret_cast<uint2*>(codes + h * 128)[sub] = codes8(x, inv);
        if (sub == 0) A.w_out[t * A.n_idx_heads + h] = wv[i] * A.w_scale * scale;
      }
    }
    if (it0 + kQWarps * kIt < idx_pairs) {
#pragma unroll
      for (int i = 0; i < kIt; ++i) ask(i, it0 + kQWarps * (kIt + i));
    }
  }
  // ---- q_pe ----
  if (pe_quads > 0 && cs != nullptr) load_angles(cs, s8, A.rope.interleaved, c, sn);
  for (int it0 = warp; it0 < pe_quads; it0 += kQWarps * kPe) {
#pragma unroll
    for (int i = 0; i < kPe; ++i) {
      const int it = it0 + kQWarps * i, h = 4 * it + (lane >> 3);
      if (it >= pe_quads) break;
      float x[8];
      unpack8(pv[i], x);
      if (cs != nullptr) rotate8(x, c, sn, A.rope.interleaved);
      if (h < A.n_heads)
        reinterpret_cast<uint4*>(A.q_pe_out + (t * A.n_heads + h) * 64)[s8] =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    if (it0 + kQWarps * kPe < pe_quads) {
#pragma unroll
      for (int i = 0; i < kPe; ++i) pv[i] = ask_pe(it0 + kQWarps * (kPe + i));
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
  // The full shape with rows that load as 16-byte pieces takes the kernel built for it.
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
  // Rows that load as 16-byte pieces take the kernel built for them.
  if ((!idx || (layout->d_index == 128 && A.vec_idx && aligned(q_idx_out, 8) && aligned(idx_norm, 16))) &&
      (layout->d_rope == 64 || (!pe && !(A.rope.cos_sin && A.rope.idx_rope))) &&
      (!pe || (aligned(q_pe, 16) && q_pe_token_stride % 8 == 0 && q_pe_head_stride % 8 == 0 && aligned(q_pe_out, 16))) &&
      aligned(A.rope.cos_sin, 16)) {
    query_full_kernel<<<n_tokens, 32 * kQWarps, 0, s>>>(A);
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
