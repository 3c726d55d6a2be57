// grouped.cu -- the 8-bit GEMM of rows grouped by expert, each group with its
// own weights, and the fused dequantising epilogue ("SmoothQuant, in depth" --
// "Granularity": an INT32 accumulator, both scales in the epilogue).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sq_device.cuh"
#include "sq_launch.h"

namespace sq {
namespace {

constexpr int TR = 32, TC = 64, TK = 64;  // rows, columns, K bytes of a step

struct GroupedParams {
  const uint8_t* Xq;
  const uint8_t* Wq;
  const float* x_scale;
  const float* w_scale;
  const int32_t* offsets;
  const int32_t* row_token;
  int64_t X, R, N, K;
  int E, epi;
  void* out;
  int64_t ldo;
};

__device__ __forceinline__ float e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

template <bool kF8>
__global__ void __launch_bounds__(256) grouped_simple_kernel(const GroupedParams p) {
  __shared__ uint32_t xs[TR][TK / 4 + 1], ws[TC][TK / 4 + 1];
  __shared__ int64_t src[TR];
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * TC;
  const int e = blockIdx.y;
  const int64_t begin = min(max(static_cast<int64_t>(p.offsets[e]), int64_t(0)), p.R);
  const int64_t end = min(static_cast<int64_t>(p.offsets[e + 1]), p.R);
  const int tc = threadIdx.x % 32, tr = threadIdx.x / 32;
  for (int64_t r0 = begin; r0 < end; r0 += TR) {
    __syncthreads();
    if (threadIdx.x < TR) {
      const int64_t r = r0 + threadIdx.x;
      int64_t s = -1;
      if (r < end) s = p.row_token ? p.row_token[r] : r;
      src[threadIdx.x] = s >= 0 && s < p.X ? s : -1;
    }
    int ai[TR / 8][2] = {};
    float af[TR / 8][2] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += TK) {
      __syncthreads();
      for (int i = threadIdx.x; i < TR * TK / 4; i += 256) {
        const int r = i / (TK / 4), c = i % (TK / 4);
        uint32_t v = 0;
        if (src[r] >= 0 && k0 + 4 * c < p.K)
          v = *reinterpret_cast<const uint32_t*>(p.Xq + src[r] * p.K + k0 + 4 * c);
        xs[r][c] = v;
      }
      for (int i = threadIdx.x; i < TC * TK / 4; i += 256) {
        const int n = i / (TK / 4), c = i % (TK / 4);
        uint32_t v = 0;
        if (n0 + n < p.N && k0 + 4 * c < p.K)
          v = *reinterpret_cast<const uint32_t*>(p.Wq + (e * p.N + n0 + n) * p.K + k0 + 4 * c);
        ws[n][c] = v;
      }
      __syncthreads();
      for (int c = 0; c < TK / 4; ++c) {
#pragma unroll
        for (int i = 0; i < TR / 8; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t x = xs[tr + 8 * i][c], w = ws[tc + 32 * j][c];
            if constexpr (kF8) {
#pragma unroll
              for (int b = 0; b < 4; ++b)
                af[i][j] = fmaf(e4m3((x >> (8 * b)) & 0xff), e4m3((w >> (8 * b)) & 0xff), af[i][j]);
            } else {
              ai[i][j] = __dp4a(static_cast<int>(x), static_cast<int>(w), ai[i][j]);
            }
          }
      }
    }
#pragma unroll
    for (int i = 0; i < TR / 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t r = r0 + tr + 8 * i, n = n0 + tc + 32 * j;
        if (r >= end || n >= p.N) continue;
        const int64_t o = r * p.ldo + n, s = src[tr + 8 * i];
        if (p.epi == SQ_EPI_I32_RAW) {
          static_cast<int32_t*>(p.out)[o] = ai[i][j];
        } else if (p.epi == SQ_EPI_F32_RAW) {
          static_cast<float*>(p.out)[o] = af[i][j];
        } else {
          const float acc = kF8 ? af[i][j] : __int2float_rn(ai[i][j]);
          float t = __fmul_rn(__fmul_rn(acc, s >= 0 ? p.x_scale[s] : 0.0f), p.w_scale[e * p.N + n]);
          if (p.epi == SQ_EPI_BF16_RELU) t = t > 0.0f ? t : 0.0f;
          static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(t);
        }
      }
  }
}

}  // namespace

cudaError_t launch_gemm_grouped(const void* Xq, int64_t X, const void* Wq, const float* x_scale,
                                const float* w_scale, const int32_t* offsets,
                                const int32_t* row_token, int64_t R, int64_t E, int64_t N,
                                int64_t K, int epi, void* out, int64_t ldo, int path_hint,
                                int64_t wait_polls, int* error_word, bool fp8, cudaStream_t st) {
  GroupedParams p{static_cast<const uint8_t*>(Xq), static_cast<const uint8_t*>(Wq), x_scale, w_scale,
                  offsets, row_token, X, R, N, K, static_cast<int>(E), epi, out, ldo};
  const dim3 grid(static_cast<unsigned>((N + TC - 1) / TC), static_cast<unsigned>(E));
  if (fp8)
    grouped_simple_kernel<true><<<grid, 256, 0, st>>>(p);
  else
    grouped_simple_kernel<false><<<grid, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace sq
