// blocknorm.cu -- the end of one block and the start of the next in one pass
// over the rows: (weighted sum of a token's expert rows,) the norm behind the
// block, gate, scaled residual, the norm before the next block with the folded
// 1/s, and per-token INT8 / FP8 codes.  ("SmoothQuant, in depth" -- "Where the
// scales go in a decoder block": 1/s folds into the norm in front of a Linear;
// "Granularity": per-token scales.)
//
// One CTA per row; a thread keeps its CH chunks of 8 values in fp32 registers
// from the first load to the last store, so each input is read once and each
// output written once.  The row statistics are reduced by warp shuffles and one
// shared-memory exchange each: a barrier per reduction (sum of squares; mean
// then squares around it for LayerNorm; max |y|).  Everything is fp32: a
// row's sum runs over at most 64 values per thread and a tree across threads,
// a relative error of a few 2^-24, below the rounding of its inputs.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "sq_device.cuh"
#include "sq_launch.h"

namespace sq {
namespace {

struct BlockNormParams {
  sq_block_norm_args a;
  int K;
  int fp8;
  int stages;  // reductions before the codes' (for the shared-memory slots)
};

// 8 consecutive values as loaded: 16 bytes of bf16 or 32 bytes of fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* v) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Raw8<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    lo = q[0];
    hi = q[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float* v) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

__device__ __forceinline__ void load_vec8(const float* p, int i, float (&v)[8]) {
  const float4* q = reinterpret_cast<const float4*>(p + i);
  const float4 a = __ldg(q), b = __ldg(q + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Sum over the CTA; `slot` is a 32-entry row of shared memory no other
// reduction of the same row uses.  Every thread gets the same bits.
__device__ __forceinline__ float cta_sum(float v, float* slot, int warps) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slot[warp] = v;
  __syncthreads();
  float t = lane < warps ? slot[lane] : 0.0f;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) t += __shfl_xor_sync(~0u, t, s);
  return t;
}

// Max of |.| bit patterns: NaN's lie above infinity's, so a NaN survives.
__device__ __forceinline__ uint32_t cta_max(uint32_t v, float* slot, int warps) {
  v = __reduce_max_sync(~0u, v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) slot[warp] = __uint_as_float(v);
  __syncthreads();
  return __reduce_max_sync(~0u, lane < warps ? __float_as_uint(slot[lane]) : 0u);
}

// INT8 codes of 8 values: rne(fl32(v / step)).  v * fl32(1 / step) is within
// 2^-22 relative of that quotient, under 4e-5 for |code| <= 127; only a
// product that near a half-integer can round another way and is divided.
__device__ __forceinline__ uint2 codes_i8(const float* v, float step, float inv) {
  float t[8], frac = 0.0f;
  int q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    t[j] = __fmul_rn(v[j], inv);
    const float r = rintf(t[j]);
    frac = fmaxf(frac, fabsf(t[j] - r));
    q[j] = static_cast<int>(r);
  }
  if (!(frac < 0.5f - 4e-5f && step >= FLT_MIN && step <= FLT_MAX)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = quant_code(v[j], step);
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    w[h] = (q[4 * h] & 0xff) | ((q[4 * h + 1] & 0xff) << 8) | ((q[4 * h + 2] & 0xff) << 16) |
           (static_cast<uint32_t>(q[4 * h + 3]) << 24);
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 codes_f8(const float* v, float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(v[4 * h], inv), __fmul_rn(v[4 * h + 1], inv)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fmul_rn(v[4 * h + 2], inv), __fmul_rn(v[4 * h + 3], inv)), __NV_SATFINITE,
        __NV_E4M3);
    w[h] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// v (this thread's chunks) -> norm(v), in place.  Two reductions for
// LayerNorm, one for RMSNorm, none without a norm.
template <int CH>
__device__ __forceinline__ void apply_norm(float (&v)[CH][8], int K, int norm, const float* gamma,
                                           const float* beta, float eps, float (*slots)[32],
                                           int warps) {
  const int chunks = K >> 3;
  float mu = 0.0f, r = 1.0f;
  if (norm == SQ_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[i][j];
    mu = cta_sum(s, slots[0], warps) / static_cast<float>(K);
  }
  if (norm != SQ_NORM_NONE) {
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
      if (c < chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] -= mu;
          s[j & 1] = fmaf(v[i][j], v[i][j], s[j & 1]);
        }
      }
    }
    const float var = cta_sum(s[0] + s[1], slots[1], warps) / static_cast<float>(K);
    r = 1.0f / sqrtf(var + eps);
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
    if (c < chunks) {
      if (norm != SQ_NORM_NONE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= r;
      }
      if (gamma) {
        float g[8];
        load_vec8(gamma, c * 8, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= g[j];
      }
      if (beta && norm == SQ_NORM_LAYER) {
        float b[8];
        load_vec8(beta, c * 8, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += b[j];
      }
    }
  }
}

template <typename T, int CH, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const BlockNormParams p) {
  __shared__ float slots[5][32];
  const sq_block_norm_args& a = p.a;
  const int chunks = p.K >> 3;
  const int warps = static_cast<int>(blockDim.x) >> 5;
  const int64_t m = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  float v[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
  if (a.token_row) {
    for (int k = 0; k < a.top_k; ++k) {
      const int64_t row = a.token_row[m * a.top_k + k];
      if (row < 0 || row >= a.R) continue;
      const float w = a.weights[m * a.top_k + k];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
        if (c < chunks) {
          Raw8<T> raw;
          raw.load(a.x, row * a.ldx + c * 8);
          float t[8];
          raw.get(t);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = fmaf(w, t[j], v[i][j]);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
      if (c < chunks) {
        Raw8<T> raw;
        raw.load(a.x, m * a.ldx + c * 8);
        raw.get(v[i]);
      }
    }
  }
  apply_norm<CH>(v, p.K, a.post_norm, a.post_gamma, a.post_beta, a.post_eps, slots, warps);
  const float tg = a.token_gate ? a.token_gate[m] : 1.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
    if (c < chunks) {
      if (a.gate) {
        float g[8];
        load_vec8(a.gate, c * 8, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= g[j];
      }
      if (a.token_gate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] *= tg;
      }
      if (a.residual) {
        Raw8<T> raw;
        raw.load(a.residual, m * a.ld_res + c * 8);
        float t[8];
        raw.get(t);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = fmaf(a.residual_scale, t[j], v[i][j]);
      }
      if (a.h_out) Raw8<T>::store(a.h_out, m * a.ld_h + c * 8, v[i]);
    }
  }
  if (!a.Xq) return;
  apply_norm<CH>(v, p.K, a.pre_norm, a.pre_gamma, a.pre_beta, a.pre_eps, slots + 2, warps);
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
    if (c < chunks) {
#pragma unroll
      for (int j = 0; j < 8; ++j) am = max(am, __float_as_uint(v[i][j]) & 0x7fffffffu);
    }
  }
  const float amax = __uint_as_float(cta_max(am, slots[4], warps));
  float step = __fdiv_rn(amax, p.fp8 ? 448.0f : 127.0f);
  if (p.fp8 && step < FLT_MIN) step = 0.0f;
  const float inv = step != 0.0f ? __fdiv_rn(1.0f, step) : 0.0f;
  if (threadIdx.x == 0) a.x_scale[m] = step;
  uint8_t* q = static_cast<uint8_t*>(a.Xq) + m * p.K;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = static_cast<int>(threadIdx.x) + i * static_cast<int>(blockDim.x);
    if (c < chunks)
      *reinterpret_cast<uint2*>(q + c * 8) =
          p.fp8 ? codes_f8(v[i], inv) : codes_i8(v[i], step, inv);
  }
}

template <typename T>
cudaError_t launch_block_norm_t(const BlockNormParams& p, cudaStream_t st) {
  const int chunks = p.K >> 3;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.a.M));
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto threads = [&](int ch) { return static_cast<unsigned>(((chunks + ch - 1) / ch + 31) / 32 * 32); };
  if (chunks <= 1024) {
    cfg.blockDim = dim3(threads(1));
    return cudaLaunchKernelEx(&cfg, block_norm_kernel<T, 1, 1024>, p);
  }
  if (chunks <= 2048) {
    cfg.blockDim = dim3(threads(4));
    return cudaLaunchKernelEx(&cfg, block_norm_kernel<T, 4, 512>, p);
  }
  cfg.blockDim = dim3(threads(8));
  return cudaLaunchKernelEx(&cfg, block_norm_kernel<T, 8, 512>, p);
}

}  // namespace

cudaError_t launch_block_norm(const sq_block_norm_args& a, bool fp8, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  BlockNormParams p{};
  p.a = a;
  p.K = static_cast<int>(a.K);
  p.fp8 = fp8 ? 1 : 0;
  return a.dtype == SQ_BF16 ? launch_block_norm_t<__nv_bfloat16>(p, st)
                            : launch_block_norm_t<float>(p, st);
}

}  // namespace sq
