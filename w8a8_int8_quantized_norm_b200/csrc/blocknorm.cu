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
// a relative error of a few 2^-24, below the rounding of its inputs; the few
// rows whose sums leave fp32's range are scaled and summed again.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "sq_device.cuh"
#include "sq_launch.h"

namespace sq {
namespace {

struct BlockNormParams {
  sq_block_norm_args a;
  int K;
  int fp8;
};

// Rows pass through once: they leave L1 to the parameter vectors.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 load_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

// 8 consecutive values as loaded: 16 bytes of bf16 or 32 bytes of fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    w = load_stream(static_cast<const __nv_bfloat16*>(p) + i);
  }
  // 16 bytes a lane: all banks once
  __device__ __forceinline__ void load_shared(uint32_t buf, int c) { w = load_shared16(buf + c * 16); }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float2 (&v)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[j].x, v[j].y);
      u[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Raw8<float> {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float* q = static_cast<const float*>(p) + i;
    lo = load_stream(q);
    hi = load_stream(q + 4);
  }
  __device__ __forceinline__ void load_shared(uint32_t buf, int c) {
    lo = load_shared16(buf + c * 32);
    hi = load_shared16(buf + c * 32 + 16);
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = make_float2(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1]));
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const float2 (&v)[4]) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
};

// 8 parameters of chunk c: from global memory as they are, or from the shared
// copy, whose two halves lie apart (16 bytes a lane: all banks once).
struct GlobalVec {
  const float* p;
  __device__ __forceinline__ void get(int c, float2 (&g)[4]) const {
    const float4* q = reinterpret_cast<const float4*>(p + c * 8);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    g[0] = make_float2(a.x, a.y);
    g[1] = make_float2(a.z, a.w);
    g[2] = make_float2(b.x, b.y);
    g[3] = make_float2(b.z, b.w);
  }
};
struct SharedVec {
  uint32_t addr;  // 0: none
  int half;       // bytes between the halves
  __device__ __forceinline__ explicit operator bool() const { return addr != 0; }
  __device__ __forceinline__ void get(int c, float2 (&g)[4]) const {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(g[0].x), "=f"(g[0].y), "=f"(g[1].x), "=f"(g[1].y)
                 : "r"(addr + c * 16));
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(g[2].x), "=f"(g[2].y), "=f"(g[3].x), "=f"(g[3].y)
                 : "r"(addr + half + c * 16));
  }
};

template <typename V>
__device__ __forceinline__ void mul8(float2 (&v)[4], const V& p, int c) {
  float2 g[4];
  p.get(c, g);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(v[j], g[j]);
}
template <typename V>
__device__ __forceinline__ void add8(float2 (&v)[4], const V& p, int c) {
  float2 b[4];
  p.get(c, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __fadd2_rn(v[j], b[j]);
}
__device__ __forceinline__ void fma8(float2 (&v)[4], float w, const float2 (&t)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __ffma2_rn(make_float2(w, w), t[j], v[j]);
}
__device__ __forceinline__ void scale8(float2 (&v)[4], float w) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(v[j], make_float2(w, w));
}

// The warps that share a row: a whole CTA, or one of its groups.
struct Team {
  int thread, threads, warps, bar;  // bar: named barrier of a group, 0 for the CTA's
  __device__ __forceinline__ void sync() const {
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
  }
};

// Sum over the team; `slot` is a 32-entry row of shared memory no other
// reduction of the same row uses.  Every thread gets the same bits.
__device__ __forceinline__ float team_sum(float v, float* slot, const Team& tm) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(~0u, v, s);
  const int warp = tm.thread >> 5, warps = tm.warps, lane = threadIdx.x & 31;
  if (lane == 0) slot[warp] = v;
  tm.sync();
  float t = lane < warps ? slot[lane] : 0.0f;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) t += __shfl_xor_sync(~0u, t, s);
  return t;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN survives
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Max over the team of values >= 0 (or NaN, whose bits order above infinity's).
__device__ __forceinline__ float team_max(float v, float* slot, const Team& tm) {
  const uint32_t u = __reduce_max_sync(~0u, __float_as_uint(v) & 0x7fffffffu);
  const int warp = tm.thread >> 5, warps = tm.warps, lane = threadIdx.x & 31;
  if (lane == 0) slot[warp] = __uint_as_float(u);
  tm.sync();
  return __uint_as_float(
      __reduce_max_sync(~0u, lane < warps ? __float_as_uint(slot[lane]) : 0u));
}

// INT8 codes of 8 values: rne(fl32(v / step)).  Adding 1.5 2^23 leaves the
// integer in the low byte.  v fl32(inv (1 - 2^-21)) and v fl32(inv (1 + 2^-21)),
// inv = fl32(1 / step), lie on either side of v / step and of its fp32
// rounding (each off by at most 2^-23 relative); when both round to the same
// integer that is the code, else the quotient itself is taken.
__device__ __forceinline__ uint2 codes_i8(const float2 (&v)[4], float step, float inv) {
  const float lo = __fmul_rn(inv, 1.0f - 0x1p-21f), hi = __fmul_rn(inv, 1.0f + 0x1p-21f);
  const float2 magic = make_float2(12582912.0f, 12582912.0f);
  uint32_t q[8], differ = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = __ffma2_rn(v[j], make_float2(lo, lo), magic);
    const float2 b = __ffma2_rn(v[j], make_float2(hi, hi), magic);
    q[2 * j] = __float_as_uint(a.x);
    q[2 * j + 1] = __float_as_uint(a.y);
    differ |= (q[2 * j] ^ __float_as_uint(b.x)) | (q[2 * j + 1] ^ __float_as_uint(b.y));
  }
  // outside this range (zero, subnormal, huge, not finite) inv is no reciprocal
  if (differ != 0 || !(step >= FLT_MIN && step <= 0x1p125f)) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      q[2 * j] = static_cast<uint32_t>(quant_code(v[j].x, step));
      q[2 * j + 1] = static_cast<uint32_t>(quant_code(v[j].y, step));
    }
  }
  return make_uint2(
      __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410),
      __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410));
}

__device__ __forceinline__ uint2 codes_f8(const float2 (&v)[4], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(v[j], make_float2(inv, inv)), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The norm's factor 1 / sqrt(mean square + eps) of a row whose sums overflow or
// vanish in fp32: v (this thread's ch chunks, in local memory) is multiplied by
// a power of two that brings its largest value near 2^50, eps by its square,
// LayerNorm's mean taken off, and the squares summed again.  A function of its
// own on a copy of v: inlined, it took registers from the rows that never need
// it (16384 x 8192: 156 us without, 176 to 213 inlined, 160 like this).
__device__ __noinline__ float rescue(float2* v, int ch, int K, bool layer, float eps, float* slot,
                                     Team tm) {
  const int own = max(0, min(ch, ((K >> 3) - tm.thread + tm.threads - 1) / tm.threads)) * 4;
  float am = 0.0f;
#pragma unroll 1
  for (int i = 0; i < own; ++i) am = max_nan(am, max_nan(fabsf(v[i].x), fabsf(v[i].y)));
  tm.sync();  // `slot` has been read
  am = team_max(am, slot, tm);
  tm.sync();
  if (!(am <= FLT_MAX)) return NAN;  // a NaN or an infinity in the row
  if (am == 0.0f) return rsqrtf(eps);
  // 2^100 at most, so that an eps this is done for (below 2^-100) stays finite
  const float c = __uint_as_float(static_cast<uint32_t>(min(50 - ilogbf(am), 100) + 127) << 23);
  float sum = 0.0f;
#pragma unroll 1
  for (int i = 0; i < own; ++i) {
    v[i] = make_float2(v[i].x * c, v[i].y * c);
    sum += v[i].x + v[i].y;
  }
  float mu = 0.0f;
  if (layer) {
    mu = team_sum(sum, slot, tm) / static_cast<float>(K);
    tm.sync();
  }
  sum = 0.0f;
#pragma unroll 1
  for (int i = 0; i < own; ++i) {
    v[i] = make_float2(v[i].x - mu, v[i].y - mu);
    sum = fmaf(v[i].x, v[i].x, fmaf(v[i].y, v[i].y, sum));
  }
  return rsqrtf(team_sum(sum, slot, tm) / static_cast<float>(K) + eps * c * c);
}

// v (this thread's chunks) -> its norm before gamma and beta, in place.  Two
// reductions for LayerNorm, one for RMSNorm, none without a norm.  Rows with
// values above about 1e19, a mean that could carry the largest values over, or
// an eps of nearly 0 and values below 1e-15 go through rescue(); every thread
// sees the same sums, so all take the same way.
template <int CH, bool kFull>
__device__ __forceinline__ void normalise(float2 (&v)[CH][4], int K, int norm, float eps,
                                          float (*slots)[32], const Team& tm) {
  if (norm == SQ_NORM_NONE) return;
  const float inv_k = __frcp_rn(static_cast<float>(K));
  float2 s[2];
  bool sound = true;
  if (norm == SQ_NORM_LAYER) {
    s[0] = s[1] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j & 1] = __fadd2_rn(s[j & 1], v[i][j]);
    const float mu = team_sum((s[0].x + s[0].y) + (s[1].x + s[1].y), slots[0], tm) * inv_k;
    sound = fabsf(mu) <= 0x1p96f;  // up to there FLT_MAX - mu rounds to FLT_MAX
    const float off = sound ? mu : 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (kFull || tm.thread + i * tm.threads < (K >> 3)) {  // the rest of v stays zero
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = __fadd2_rn(v[i][j], make_float2(-off, -off));
      }
  }
  s[0] = s[1] = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j & 1] = __ffma2_rn(v[i][j], v[i][j], s[j & 1]);
  const float t =
      team_sum((s[0].x + s[0].y) + (s[1].x + s[1].y), slots[1], tm) * inv_k + eps;
  float r;
  if (sound && t >= 0x1p-100f && t <= FLT_MAX) {
    r = rsqrtf(t);  // within 2 units in the last place
  } else {
    float2 copy[CH][4];
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) copy[i][j] = v[i][j];
    r = rescue(&copy[0][0], CH, K, norm == SQ_NORM_LAYER, eps, slots[0], tm);
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = copy[i][j];
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) scale8(v[i], r);
}

// The codes of y and their scale; one reduction.  kFull: every thread has all
// its CH chunks (no test per chunk, so the chunks' work runs together).
template <int CH, bool kFull>
__device__ __forceinline__ void store_codes(const float2 (&v)[CH][4], const BlockNormParams& p,
                                            int64_t m, float* slot, const Team& tm) {
  const int chunks = p.K >> 3;
  float am[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < CH; ++i)
    if (kFull || tm.thread + i * tm.threads < chunks) {  // a row of NaN leaves them past its end too
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        am[0] = max_nan(am[0], fabsf(v[i][j].x));
        am[1] = max_nan(am[1], fabsf(v[i][j].y));
      }
    }
  const float amax = team_max(max_nan(am[0], am[1]), slot, tm);
  float step = __fdiv_rn(amax, p.fp8 ? 448.0f : 127.0f);
  if (p.fp8 && step < FLT_MIN) step = 0.0f;
  const float inv = step != 0.0f ? __fdiv_rn(1.0f, step) : 0.0f;
  if (tm.thread == 0) p.a.x_scale[m] = step;
  uint8_t* q = static_cast<uint8_t*>(p.a.Xq) + m * p.K + tm.thread * 8;
  const int stride = tm.threads * 8;
  if (p.fp8) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (kFull || tm.thread + i * tm.threads < chunks)
        *reinterpret_cast<uint2*>(q + i * stride) = codes_f8(v[i], inv);
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (kFull || tm.thread + i * tm.threads < chunks)
        *reinterpret_cast<uint2*>(q + i * stride) = codes_i8(v[i], step, inv);
  }
}

// One row per CTA, straight from global memory: few rows, and rows whose
// parameters and buffers do not fit the pipeline below.  kFull: every thread has
// all its chunks (2000 x 16384, LayerNorm: 87 us, 99 with a test per chunk).
template <typename T, int CH, int kRegs, bool kFull>
__global__ void __maxnreg__(kRegs) block_norm_kernel(const BlockNormParams p) {
  __shared__ float slots[5][32];
  const sq_block_norm_args& a = p.a;
  const int chunks = p.K >> 3;
  const Team tm{static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x),
                static_cast<int>(blockDim.x) >> 5, 0};
  const int64_t m = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  float2 v[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = make_float2(0.0f, 0.0f);
  if (a.token_row) {
    for (int k = 0; k < a.top_k; ++k) {
      const int64_t row = a.token_row[m * a.top_k + k];
      if (row < 0 || row >= a.R) continue;
      const float w = a.weights[m * a.top_k + k];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = tm.thread + i * tm.threads;
        if (kFull || c < chunks) {
          Raw8<T> raw;
          raw.load(a.x, row * a.ldx + c * 8);
          float2 t[4];
          raw.get(t);
          fma8(v[i], w, t);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tm.thread + i * tm.threads;
      if (kFull || c < chunks) {
        Raw8<T> raw;
        raw.load(a.x, m * a.ldx + c * 8);
        raw.get(v[i]);
      }
    }
  }
  // the residual is on its way through the first norm's reductions
  Raw8<T> res[CH];
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = tm.thread + i * tm.threads;
      if (kFull || c < chunks) res[i].load(a.residual, m * a.ld_res + c * 8);
    }
  }
  const float tg = a.token_gate ? a.token_gate[m] : 1.0f;
  normalise<CH, kFull>(v, p.K, a.post_norm, a.post_eps, slots, tm);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tm.thread + i * tm.threads;
    if (kFull || c < chunks) {
      if (a.post_gamma) mul8(v[i], GlobalVec{a.post_gamma}, c);
      if (a.post_beta && a.post_norm == SQ_NORM_LAYER) add8(v[i], GlobalVec{a.post_beta}, c);
      if (a.gate) mul8(v[i], GlobalVec{a.gate}, c);
      if (a.token_gate) scale8(v[i], tg);
      if (a.residual) {
        float2 t[4];
        res[i].get(t);
        fma8(v[i], a.residual_scale, t);
      }
      if (a.h_out) Raw8<T>::store(a.h_out, m * a.ld_h + c * 8, v[i]);
    }
  }
  if (!a.Xq) return;
  normalise<CH, kFull>(v, p.K, a.pre_norm, a.pre_eps, slots + 2, tm);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = tm.thread + i * tm.threads;
    if (kFull || c < chunks) {
      if (a.pre_gamma) mul8(v[i], GlobalVec{a.pre_gamma}, c);
      if (a.pre_beta && a.pre_norm == SQ_NORM_LAYER) add8(v[i], GlobalVec{a.pre_beta}, c);
    }
  }
  store_codes<CH, kFull>(v, p, m, slots[4], tm);
}

// ---------------------------------------------------------------------------
// Many rows: one persistent CTA per SM, its warps in groups of a row each.  A
// group's inputs arrive by cp.async.bulk into its own shared-memory buffers:
// the next row's x is fetched as soon as this row's is in registers, the next
// residual after this one, so copies are in flight through the reductions and
// stores; with plain loads the kernel waited for them (long-scoreboard stalls
// 8.6 of 15 warps, a third of HBM).  Bound by HBM with the rows of two experts
// (16384 x 8192, RMSNorm twice: 191 us, 6.3 TB/s), close to it without (160 us,
// 5.9 TB/s).  The parameter vectors (post_gamma * gate,
// post_beta * gate, pre_gamma, pre_beta) are put into shared memory once per
// CTA: read per row through L1 they were more bytes than the row itself.
// ---------------------------------------------------------------------------
constexpr int kMaxGroups = 8;
// Expert rows a token sums, at most.  More were not tried here: they take the
// one-row kernel (eight rows, 4096 x 4096: 74 us, 54 at HBM's rate).
constexpr int kPipeMaxSum = 4;
// Chunks of a thread and threads of a CTA.  Without a sum 64 values a thread
// measured best (16384 x 8192: 160 us, 178 us with 32 a thread); with one the
// rows' copies leave room for three groups at 8192 channels, and 32 values a
// thread keep more warps (192 against 221 us).  Below 80 registers a thread the
// same code spills and loses a third.
__host__ __device__ constexpr int pipe_ch(bool sum) { return sum ? 4 : 8; }
constexpr int pipe_max_threads(bool sum) { return sum ? 768 : 512; }

struct PipeShape {
  int groups, threads;         // threads of a group
  int x_rows;                  // buffers of x rows per group
  int vecs;                    // parameter vectors in shared memory
  int vec_at[4];               // slot of A, B, C, D, or -1
  int row_bytes, smem;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// mbarrier.try_wait that may suspend the thread for up to `ns` nanoseconds.
__device__ __forceinline__ bool mbar_try_wait_for(uint32_t bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

// One probe that does not suspend the thread.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

template <typename T>
__device__ __forceinline__ void shared8(uint32_t buf, int c, float2 (&v)[4]) {
  Raw8<T> raw;
  raw.load_shared(buf, c);
  raw.get(v);
}

template <typename T, bool kSum, bool kFull>
__global__ void __launch_bounds__(pipe_max_threads(kSum), 1)
    block_norm_pipe_kernel(const BlockNormParams p, const PipeShape sh, int* error_word,
                           int64_t wait_polls) {
  constexpr int CH = pipe_ch(kSum);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float slots[kMaxGroups][5][32];
  __shared__ uint64_t bars[kMaxGroups][2];
  __shared__ float sum_w[kMaxGroups][2][kPipeMaxSum];  // weights of the row being fetched, by parity
  __shared__ int sum_ok[kMaxGroups][2];                // which of its rows exist, a bit each
  __shared__ int late[kMaxGroups][2];                  // a wait of the row ran out, by parity
  __shared__ int abort_flag;
  const sq_block_norm_args& a = p.a;
  const int chunks = p.K >> 3;
  const int g = static_cast<int>(threadIdx.x) / sh.threads;
  const Team tm{static_cast<int>(threadIdx.x) - g * sh.threads, sh.threads, sh.threads >> 5, 1 + g};
  float* params = reinterpret_cast<float*>(smem);
  const uint32_t xbuf = smem_u32(smem) + sh.vecs * p.K * 4 +
                        g * (sh.x_rows + (a.residual ? 1 : 0)) * sh.row_bytes;
  const uint32_t rbuf = xbuf + sh.x_rows * sh.row_bytes;
  const uint32_t xbar = smem_u32(&bars[g][0]), rbar = smem_u32(&bars[g][1]);
  const int64_t step_rows = static_cast<int64_t>(gridDim.x) * sh.groups;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * sh.groups + g;

  if (threadIdx.x == 0) abort_flag = 0;
  if (tm.thread == 0) {
    late[g][0] = late[g][1] = 0;
    mbar_init(xbar, 1);
    mbar_init(rbar, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The group's first warp fetches.  Lane j < top_k has the j-th expert row and
  // weight of the next row to fetch, read a row ahead (peek).
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const bool fetcher = tm.thread < 32;
  int next_row = -1;
  float next_w = 0.0f;
  auto peek = [&](int64_t m) {
    next_row = -1;
    if (kSum && lane < a.top_k && m < a.M) {
      next_row = a.token_row[m * a.top_k + lane];
      next_w = a.weights[m * a.top_k + lane];
    }
  };
  auto fetch_x = [&](int64_t m, int parity) {
    if constexpr (!kSum) {
      if (lane == 0) {
        mbar_arrive_expect_tx(xbar, sh.row_bytes);
        bulk_load(xbuf, static_cast<const T*>(a.x) + m * a.ldx, sh.row_bytes, xbar);
      }
    } else {
    const bool mine = next_row >= 0 && next_row < a.R;
    const uint32_t ok = __ballot_sync(~0u, mine);
    if (lane < a.top_k) sum_w[g][parity][lane] = next_w;
    if (lane == 0) sum_ok[g][parity] = static_cast<int>(ok);
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(xbar, __popc(ok) * sh.row_bytes);
    __syncwarp();
    if (mine)
      bulk_load(xbuf + lane * sh.row_bytes,
                static_cast<const T*>(a.x) + static_cast<int64_t>(next_row) * a.ldx, sh.row_bytes,
                xbar);
    }
  };
  auto fetch_res = [&](int64_t m) {
    mbar_arrive_expect_tx(rbar, sh.row_bytes);
    bulk_load(rbuf, static_cast<const T*>(a.residual) + m * a.ld_res, sh.row_bytes, rbar);
  };
  if (fetcher && m0 < a.M) {
    peek(m0);
    fetch_x(m0, 0);
    if (a.residual && lane == 0) fetch_res(m0);
    peek(m0 + step_rows);
  }
  // the parameters, the halves of every 8 apart
  for (int i = threadIdx.x; i < p.K; i += blockDim.x) {
    const int at = ((i & 4) ? p.K / 2 : 0) + (i >> 3) * 4 + (i & 3);
    const float g1 = a.gate ? a.gate[i] : 1.0f;
    if (sh.vec_at[0] >= 0)
      params[sh.vec_at[0] * p.K + at] = (a.post_gamma ? a.post_gamma[i] : 1.0f) * g1;
    if (sh.vec_at[1] >= 0) params[sh.vec_at[1] * p.K + at] = a.post_beta[i] * g1;
    if (sh.vec_at[2] >= 0) params[sh.vec_at[2] * p.K + at] = a.pre_gamma[i];
    if (sh.vec_at[3] >= 0) params[sh.vec_at[3] * p.K + at] = a.pre_beta[i];
  }
  SharedVec vec[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    vec[i] = SharedVec{sh.vec_at[i] >= 0 ? smem_u32(params + sh.vec_at[i] * p.K) : 0u, p.K * 2};
  __syncthreads();

  uint32_t phase = 0;
  // The first probe sleeps up to 20 us in hardware: a group that spins takes
  // issue slots from the ones at work.  A wait that runs out is recorded and
  // marks its row late.  The row goes through (the others wait at its barriers),
  // but a barrier whose phase the arming thread gave up on may still be open: it
  // is armed no more and no copy follows, and behind the row the group leaves.
  // The marks are read behind the row's last barrier, and by parity, since a
  // thread may be a row ahead of one that still reads.  (16384 x 8192 behind two
  // experts: 187 us; 191 with a flag in a register joined at that barrier, 191
  // with the marks read before every copy.)  A limit of n polls allows n - 1
  // probes, which do not sleep: 1 always runs out.
  auto wait = [&](uint32_t bar) {
    if (wait_polls > 0) {
      for (int64_t i = 1; i < wait_polls; ++i)
        if (mbar_test_wait(bar, phase)) return true;
    } else if (mbar_try_wait_for(bar, phase, 20000u) || wait_phase(bar, phase, 0, &abort_flag)) {
      return true;
    }
    record_device_error(error_word, SQ_ERR_PIPELINE_TIMEOUT);
    *const_cast<volatile int*>(&late[g][phase]) = 1;
    *const_cast<volatile int*>(&abort_flag) = 1;
    return false;
  };
  auto on_time = [&]() { return *const_cast<volatile int*>(&late[g][phase]) == 0; };
  for (int64_t m = m0; m < a.M; m += step_rows, phase ^= 1u) {
    const bool more = m + step_rows < a.M;
    float2 v[CH][4];
    const float tg = a.token_gate ? __ldg(a.token_gate + m) : 1.0f;
    // one loop over the chunks per step, its condition outside: the chunks'
    // loads then go out together
    auto in = [&](int i) { return kFull || tm.thread + i * tm.threads < chunks; };
    auto at = [&](int i) { return tm.thread + i * tm.threads; };
    bool r_ok = true;
    const bool x_ok = wait(xbar);
    // (a test at run time, although kSum says the same: without it the loads are
    // all moved up and spill, 200 us instead of 162 at 16384 x 8192)
    if (!a.token_row) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (in(i)) {
          shared8<T>(xbuf, at(i), v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = make_float2(0.0f, 0.0f);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = make_float2(0.0f, 0.0f);
      const int ok = sum_ok[g][phase];
      for (int k = 0; k < a.top_k; ++k) {
        if (!((ok >> k) & 1)) continue;
        const float w = sum_w[g][phase][k];
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (in(i)) {
            float2 t[4];
            shared8<T>(xbuf + k * sh.row_bytes, at(i), t);
            fma8(v[i], w, t);
          }
      }
    }
    if (a.post_norm == SQ_NORM_NONE) tm.sync();  // the row is in registers (else: by the sum)
    normalise<CH, kFull>(v, p.K, a.post_norm, a.post_eps, slots[g], tm);
    if (fetcher && more && __all_sync(~0u, x_ok)) {
      fetch_x(m + step_rows, phase ^ 1u);
      peek(m + 2 * step_rows);
    }
    if (vec[0]) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (in(i)) mul8(v[i], vec[0], at(i));
    }
    if (vec[1]) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (in(i)) add8(v[i], vec[1], at(i));
    }
    if (a.token_gate) {
#pragma unroll
      for (int i = 0; i < CH; ++i) scale8(v[i], tg);
    }
    if (a.residual) {
      r_ok = wait(rbar);
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (in(i)) {
          float2 t[4];
          shared8<T>(rbuf, at(i), t);
          fma8(v[i], a.residual_scale, t);
        }
    }
    if (a.h_out) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (in(i)) Raw8<T>::store(a.h_out, m * a.ld_h + at(i) * 8, v[i]);
    }
    if (a.Xq) {
      normalise<CH, kFull>(v, p.K, a.pre_norm, a.pre_eps, slots[g] + 2, tm);
      // (a sum's barrier, or the maximum's below, follows the residual's reads)
      const bool early = a.pre_norm != SQ_NORM_NONE;
      if (a.residual && early && tm.thread == 0 && more && r_ok) fetch_res(m + step_rows);
      if (vec[2]) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (in(i)) mul8(v[i], vec[2], at(i));
      }
      if (vec[3]) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (in(i)) add8(v[i], vec[3], at(i));
      }
      store_codes<CH, kFull>(v, p, m, slots[g][4], tm);
      if (a.residual && !early && tm.thread == 0 && more && r_ok) fetch_res(m + step_rows);
    } else {
      tm.sync();
      if (a.residual && tm.thread == 0 && more && r_ok) fetch_res(m + step_rows);
    }
    if (!on_time()) break;
  }
  if (*const_cast<volatile int*>(&abort_flag)) {
    // about 20 ms: every copy in flight lands before the shared memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < 40000000LL) {
    }
  }
}

// Groups of the pipeline for these arguments, or false if it does not pay:
// fewer than two groups fit (their copies would not overlap a row's
// reductions), or there are too few rows for every group to have two (the
// parameters are then copied for one row each).  16384 x 8192: 160 us, one row
// per CTA 350; 8192 x 4096: 47 against 72.
bool pipe_shape(const sq_block_norm_args& a, int sms, PipeShape& sh) {
  const int K = static_cast<int>(a.K), es = a.dtype == SQ_BF16 ? 2 : 4;
  const bool sum = a.token_row != nullptr;
  if (a.top_k > kPipeMaxSum) return false;
  sh.threads = ((K / 8 + pipe_ch(sum) - 1) / pipe_ch(sum) + 31) / 32 * 32;
  sh.x_rows = sum ? a.top_k : 1;
  sh.row_bytes = K * es;
  const int group = (sh.x_rows + (a.residual ? 1 : 0)) * sh.row_bytes;
  const bool has[4] = {a.post_gamma || a.gate, a.post_beta && a.post_norm == SQ_NORM_LAYER,
                       a.Xq && a.pre_gamma,
                       a.Xq && a.pre_beta && a.pre_norm == SQ_NORM_LAYER};
  sh.vecs = 0;
  for (int i = 0; i < 4; ++i) sh.vec_at[i] = has[i] ? sh.vecs++ : -1;
  int n = (221 * 1024 - sh.vecs * K * 4) / group;
  if (n > pipe_max_threads(sum) / sh.threads) n = pipe_max_threads(sum) / sh.threads;
  if (n > kMaxGroups) n = kMaxGroups;
  if (n < 2 || a.M < static_cast<int64_t>(2) * n * sms) return false;
  sh.groups = n;
  sh.smem = sh.vecs * K * 4 + n * group;
  return true;
}

template <typename T, bool kSum>
cudaError_t launch_pipe(const BlockNormParams& p, const PipeShape& sh, int sms, int* error_word,
                        int64_t wait_polls, cudaLaunchConfig_t cfg) {
  auto kern = (p.K >> 3) == pipe_ch(kSum) * sh.threads ? block_norm_pipe_kernel<T, kSum, true>
                                                       : block_norm_pipe_kernel<T, kSum, false>;
  cudaError_t e = launch_cache().ensure_smem(reinterpret_cast<const void*>(kern), sh.smem);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(sms));
  cfg.blockDim = dim3(static_cast<unsigned>(sh.groups * sh.threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(sh.smem);
  return cudaLaunchKernelEx(&cfg, kern, p, sh, error_word, wait_polls);
}

template <typename T>
cudaError_t launch_block_norm_t(const BlockNormParams& p, int sms, int64_t wait_polls,
                                int* error_word, cudaStream_t st) {
  const int chunks = p.K >> 3;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  PipeShape sh;
  if (pipe_shape(p.a, sms, sh))
    return p.a.token_row ? launch_pipe<T, true>(p, sh, sms, error_word, wait_polls, cfg)
                         : launch_pipe<T, false>(p, sh, sms, error_word, wait_polls, cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(p.a.M));
  // one chunk a thread while 1024 threads cover the row: least latency (1 x 8192
  // 9 us against 17 with four, 37 x 4096 8 against 16); then two (4096 x 9216 in
  // fp32 128 us, with four 140), then eight
  const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 8;
  const int threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
  const bool full = chunks == ch * threads;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  auto kern = ch == 1   ? (full ? block_norm_kernel<T, 1, 32, true> : block_norm_kernel<T, 1, 32, false>)
              : ch == 2 ? (full ? block_norm_kernel<T, 2, 56, true> : block_norm_kernel<T, 2, 56, false>)
                        : (full ? block_norm_kernel<T, 8, 128, true> : block_norm_kernel<T, 8, 128, false>);
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_block_norm(const sq_block_norm_args& a, bool fp8, int num_sms,
                              int64_t wait_polls, int* error_word, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  const int sms = num_sms > 0 ? num_sms : 148;
  BlockNormParams p{};
  p.a = a;
  p.K = static_cast<int>(a.K);
  p.fp8 = fp8 ? 1 : 0;
  return a.dtype == SQ_BF16
             ? launch_block_norm_t<__nv_bfloat16>(p, sms, wait_polls, error_word, st)
             : launch_block_norm_t<float>(p, sms, wait_polls, error_word, st);
}

}  // namespace sq
