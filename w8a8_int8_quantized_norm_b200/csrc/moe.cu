// moe.cu -- the router of a layer of experts: each token's top-k experts with
// their weights, and the (token, expert) rows sorted by expert.
//
// Two passes.  The first ranks: a warp per token holds the token's logits in
// registers (lane l the experts l, l + 32, ...), takes the largest key k
// times with warp-wide integer maxima (keys are the logits' bits mapped to
// order like integers, so a maximum costs one redux), and the lowest index
// among equal keys with a warp-wide minimum; up to 128 experts a warp takes two
// tokens at once, so that one's maxima are in flight behind the other's, and
// sorts each lane's keys first, so that a choice looks at one of them.  A CTA
// walks a contiguous range of tokens in groups of 64; within a group each expert
// keeps a 64-bit mask of the tokens that chose it (a token chooses an expert at
// most once), so a row's rank among the group's rows of that expert is a
// population count -- stable in token order whatever order the mask's atomics
// arrived in.  The
// second pass adds, per expert, the counts of all earlier CTAs and experts and
// scatters.  With one CTA's worth of tokens the first pass scatters itself.
// Bound by latency, neither by its 6 MB (1 us) nor by issue (8.2 M warp
// instructions, 7 us): each choice is a warp-wide maximum and then a minimum
// that waits for it, a CTA's two groups of tokens follow one another between
// barriers, and registers allow one CTA an SM.  16384 tokens, 128 experts, top 8
// take 21 us, 16.5 of them the first pass; every choice searching all of a
// lane's keys, 27 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "sq_device.cuh"
#include "sq_launch.h"

namespace sq {
namespace {

constexpr int kRouteThreads = 1024;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kGroup = 64;      // tokens of one mask
constexpr int kPerWarp = kGroup / kRouteWarps;
constexpr int kMaxBlocks = 148; // CTAs of the first pass: the second reads all their counts
static_assert(kPerWarp == 2, "a warp ranks two tokens of a group");
constexpr int kMaxExperts = SQ_MOE_MAX_EXPERTS;

struct RouteParams {
  const void* logits;
  int64_t T, ld;
  int E, top_k, sigmoid, renorm;
  const float* bias;
  float scale;
  float* weights;
  int32_t* experts;
  int32_t* offsets;
  int32_t* row_token;
  int32_t* token_row;
  int32_t* hist;      // [blocks][E] rows of each expert per CTA of the first pass
  int blocks;
  int64_t per_block;  // tokens per CTA, a multiple of kGroup
};

// Finite floats and +-inf to unsigned integers of the same order.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(~0u, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(~0u, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u;
  return (static_cast<uint64_t>(hi) << 32) | __reduce_max_sync(~0u, lo);
}

// NaN and -inf (never chosen) become -inf, +inf the largest finite value, -0
// becomes +0 (equal keys).
__device__ __forceinline__ float clean_logit(float v) {
  return v >= -FLT_MAX ? fminf(v, FLT_MAX) + 0.0f : -INFINITY;
}

// 1 / (1 + exp(-l)) without an exp that overflows.
__device__ __forceinline__ float sigmoid_f(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// Below it a sigmoid score leaves the normal range of 64 bits and counts as 0.
constexpr float kLowestScore = -708.0f;

// sigmoid(l) / sigmoid(m) up to a factor of m alone, l <= m < 0: exp(l - m) /
// (1 + exp(l)).  The scores themselves leave fp32 below about -88, their ratios
// do not.  l - m is rounded; what it lost is put back to first order.
__device__ __forceinline__ float sigmoid_ratio(float l, float m) {
  const float d = l - m, b = d - l;
  const float lost = (l - (d - b)) - (m + b);
  const float e = expf(d);
  return fmaf(e, lost, e) / (1.0f + expf(l));
}

__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_logit(const float* p) { return *p; }

// The choices of U tokens by one warp: lane j < top_k gets each token's j-th
// expert (-1: none left, or no token) and its weight.  V: experts per lane.
// Key 0 marks an expert that cannot be chosen (every finite value's key is above
// it).  Up to 4 keys a lane are sorted first: 6 exchanges, then a choice costs
// one maximum and a shift (16384 x 128, top 8: 28.6 us against 34.8 searching,
// 7 us of the timing's own in both);
// 8 and 16 keys would need 28 and 120 exchanges, and are searched.
template <typename T, int V, int U, bool kBias>
__device__ __forceinline__ void choose(const RouteParams& p, const int64_t (&t)[U], int64_t t_end,
                                       int lane, int (&my_e)[U], float (&my_w)[U]) {
  using Key = typename std::conditional<kBias, uint64_t, uint32_t>::type;
  constexpr bool kSorted = V <= 4;
  float l[U][V];
  Key key[U][V];
  int ex[U][V];  // the keys' experts
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const T* row = static_cast<const T*>(p.logits) + t[u] * p.ld;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 32 * i;
      l[u][i] = -INFINITY;
      if (t[u] < t_end && e < p.E) l[u][i] = load_logit(row + e);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float v = l[u][i] = clean_logit(l[u][i]);
      ex[u][i] = lane + 32 * i;
      key[u][i] = 0;
      if (v >= -FLT_MAX) {
        if constexpr (kBias) {
          const double s = 1.0 / (1.0 + exp(-static_cast<double>(v))) +
                           static_cast<double>(p.bias[lane + 32 * i]) + 0.0;
          if (s > -INFINITY) key[u][i] = order_key(s);  // false for NaN
        } else {
          key[u][i] = order_key(v);
        }
      }
    }
    if constexpr (kSorted) {  // adjacent exchanges: equal keys keep their order
#pragma unroll
      for (int a = 0; a < V - 1; ++a)
#pragma unroll
        for (int b = 0; b < V - 1 - a; ++b) {
          const bool swap = key[u][b + 1] > key[u][b];
          const Key k = key[u][b];
          const int e = ex[u][b];
          key[u][b] = swap ? key[u][b + 1] : k;
          ex[u][b] = swap ? ex[u][b + 1] : e;
          key[u][b + 1] = swap ? k : key[u][b + 1];
          ex[u][b + 1] = swap ? e : ex[u][b + 1];
        }
    }
    my_e[u] = -1;
  }
  for (int j = 0; j < p.top_k; ++j) {
    Key best[U], top[U];
    int at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      best[u] = key[u][0];
      at[u] = ex[u][0];
      if constexpr (!kSorted) {
#pragma unroll
        for (int i = 1; i < V; ++i)  // ascending index: the first of equal keys stays
          if (key[u][i] > best[u]) {
            best[u] = key[u][i];
            at[u] = ex[u][i];
          }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) top[u] = warp_max(best[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool wins = top[u] != 0 && best[u] == top[u];  // 0: nothing left to choose
      const int e = static_cast<int>(
          __reduce_min_sync(~0u, static_cast<uint32_t>(wins ? at[u] : kMaxExperts)));
      if (lane == j && e < kMaxExperts) my_e[u] = e;
      if constexpr (kSorted) {
        if (wins && at[u] == e) {  // the winner's list moves up
#pragma unroll
          for (int i = 0; i + 1 < V; ++i) {
            key[u][i] = key[u][i + 1];
            ex[u][i] = ex[u][i + 1];
          }
          key[u][V - 1] = 0;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e == ex[u][i]) key[u][i] = 0;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float mine = 0.0f;  // the chosen logit, from L1
    if (my_e[u] >= 0)
      mine = clean_logit(load_logit(static_cast<const T*>(p.logits) + t[u] * p.ld + my_e[u]));
    // the largest chosen logit: the first one, unless a bias decided
    float m = __shfl_sync(~0u, mine, 0);
    if constexpr (kBias) {
      const uint32_t k = warp_max(my_e[u] >= 0 ? order_key(mine) : 0u);
      m = __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
    }
    my_w[u] = 0.0f;
    if (my_e[u] >= 0) {
      if (!p.sigmoid) my_w[u] = expf(mine - m);
      else if (!p.renorm || m >= 0.0f) my_w[u] = sigmoid_f(mine);
      else if (m >= kLowestScore) my_w[u] = sigmoid_ratio(mine, m);
    }
    float total = 1.0f;
    if (p.renorm || !p.sigmoid) {
      total = my_w[u];
      if (!p.renorm) {
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (l[u][i] >= -FLT_MAX) total += expf(l[u][i] - m);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(~0u, total, s);
    }
    my_w[u] = total > 0.0f ? my_w[u] / total * p.scale : 0.0f;
  }
}

// Exclusive prefix sum of counts[0 .. E) into offsets[0 .. E] (shared memory),
// by the first warp.
__device__ __forceinline__ void scan_offsets(const int* counts, int* offsets, int E, int lane) {
  int run = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int v = e0 + lane < E ? counts[e0 + lane] : 0;
    int inc = v;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int u = __shfl_up_sync(~0u, inc, s);
      if (lane >= s) inc += u;
    }
    if (e0 + lane < E) offsets[e0 + lane] = run + inc - v;
    run += __shfl_sync(~0u, inc, 31);
  }
  if (lane == 0) offsets[E] = run;
}

template <typename T, int V, bool kBias>
__global__ void __launch_bounds__(kRouteThreads) moe_route_kernel(const RouteParams p) {
  __shared__ unsigned long long mask[32 * V];
  __shared__ int count[32 * V];
  __shared__ int off[32 * V + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t_begin = static_cast<int64_t>(blockIdx.x) * p.per_block;
  const int64_t t_end = min(p.T, t_begin + p.per_block);
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) count[e] = 0;
  // the second pass may be scheduled now; it waits for this grid before it reads
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t g = t_begin; g < t_end; g += kGroup) {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) mask[e] = 0;
    __syncthreads();
    const int64_t t[kPerWarp] = {g + warp, g + warp + kRouteWarps};
    int my_e[kPerWarp];
    float w[kPerWarp];
    if constexpr (V <= 4) {
      choose<T, V, kPerWarp, kBias>(p, t, t_end, lane, my_e, w);
    } else {  // registers: one token after the other
#pragma unroll
      for (int u = 0; u < kPerWarp; ++u) {
        const int64_t one[1] = {t[u]};
        int e1[1];
        float w1[1];
        choose<T, V, 1, kBias>(p, one, t_end, lane, e1, w1);
        my_e[u] = e1[0];
        w[u] = w1[0];
      }
    }
#pragma unroll
    for (int u = 0; u < kPerWarp; ++u)
      if (t[u] < t_end && lane < p.top_k) {
        p.weights[t[u] * p.top_k + lane] = w[u];
        p.experts[t[u] * p.top_k + lane] = my_e[u];
        if (my_e[u] >= 0) atomicOr(&mask[my_e[u]], 1ull << (warp + u * kRouteWarps));
      }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPerWarp; ++u)
      if (t[u] < t_end && lane < p.top_k) {
        // the row's rank among this CTA's rows of its expert
        const unsigned long long before = (1ull << (warp + u * kRouteWarps)) - 1ull;
        p.token_row[t[u] * p.top_k + lane] =
            my_e[u] < 0 ? -1 : count[my_e[u]] + __popcll(mask[my_e[u]] & before);
      }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) count[e] += __popcll(mask[e]);
  }
  __syncthreads();
  if (p.blocks > 1) {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads)
      p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = count[e];
    return;
  }
  if (warp == 0) scan_offsets(count, off, p.E, lane);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) p.offsets[e] = off[e];
  const int rows = static_cast<int>(p.T) * p.top_k;
  for (int i = threadIdx.x; i < rows; i += kRouteThreads) {
    const int e = p.experts[i];
    if (e >= 0) {
      const int r = off[e] + p.token_row[i];
      p.token_row[i] = r;
      p.row_token[r] = i / p.top_k;
    }
  }
  for (int r = off[p.E] + threadIdx.x; r < rows; r += kRouteThreads) p.row_token[r] = -1;
}

__global__ void __launch_bounds__(kRouteThreads) moe_scatter_kernel(const RouteParams p) {
  __shared__ int before[kMaxExperts];  // rows of the earlier CTAs' tokens
  __shared__ int total[kMaxExperts];
  __shared__ int off[kMaxExperts + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = static_cast<int>(blockIdx.x);
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) before[e] = total[e] = 0;
  __syncthreads();
  // the counts of all CTAs of the first pass, the threads of an expert taking
  // every parts-th of them, eight loads in flight each
  const int parts = max(1, kRouteThreads / p.E);
  for (int i = threadIdx.x; i < parts * p.E; i += kRouteThreads) {
    const int e = i % p.E;
    int s = 0, all = 0;
#pragma unroll 8
    for (int k = i / p.E; k < p.blocks; k += parts) {
      const int c = __ldcg(p.hist + static_cast<int64_t>(k) * p.E + e);
      if (k < b) s += c;
      all += c;
    }
    atomicAdd(&before[e], s);
    atomicAdd(&total[e], all);
  }
  __syncthreads();
  if (threadIdx.x < 32) scan_offsets(total, off, p.E, static_cast<int>(threadIdx.x));
  __syncthreads();
  if (b == 0)
    for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) p.offsets[e] = off[e];
  const int64_t i0 = b * p.per_block * p.top_k;
  const int64_t i1 = min(p.T, (b + 1) * p.per_block) * p.top_k;
  for (int64_t i = i0 + threadIdx.x; i < i1; i += kRouteThreads) {
    const int e = p.experts[i];
    if (e >= 0) {
      const int r = off[e] + before[e] + p.token_row[i];
      p.token_row[i] = r;
      p.row_token[r] = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.top_k));
    }
    if (i >= off[p.E]) p.row_token[i] = -1;  // behind the last expert's rows
  }
}

void route_shape(int64_t T, int& blocks, int64_t& per_block) {
  const int64_t groups = (T + kGroup - 1) / kGroup;
  const int64_t per = (groups + kMaxBlocks - 1) / kMaxBlocks;
  per_block = per * kGroup;
  blocks = static_cast<int>((groups + per - 1) / per);
}

cudaError_t launch_dependent(const void* kernel, int grid, const RouteParams& p, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kRouteThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[1] = {const_cast<RouteParams*>(&p)};
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <typename T, int V>
const void* pick_bias(bool bias) {
  return bias ? reinterpret_cast<const void*>(moe_route_kernel<T, V, true>)
              : reinterpret_cast<const void*>(moe_route_kernel<T, V, false>);
}
template <typename T>
const void* pick_kernel(int E, bool bias) {
  return E <= 32 ? pick_bias<T, 1>(bias) : E <= 64 ? pick_bias<T, 2>(bias)
       : E <= 128 ? pick_bias<T, 4>(bias) : E <= 256 ? pick_bias<T, 8>(bias)
                                                      : pick_bias<T, 16>(bias);
}

}  // namespace

size_t moe_route_workspace(int64_t T, int64_t E) {
  if (T <= 0) return 0;
  int blocks;
  int64_t per;
  route_shape(T, blocks, per);
  return blocks > 1 ? static_cast<size_t>(blocks) * static_cast<size_t>(E) * 4u : 0u;
}

cudaError_t launch_moe_route(const void* logits, bool bf16, int64_t T, int E, int64_t ld, int top_k,
                             bool sigmoid, const float* bias, bool renorm, float scale,
                             float* weights, int32_t* experts, int32_t* offsets,
                             int32_t* row_token, int32_t* token_row, void* workspace,
                             cudaStream_t st) {
  if (T == 0) return cudaMemsetAsync(offsets, 0, static_cast<size_t>(E + 1) * 4u, st);
  RouteParams p{};
  p.logits = logits;
  p.T = T;
  p.ld = ld;
  p.E = E;
  p.top_k = top_k;
  p.sigmoid = sigmoid;
  p.renorm = renorm;
  p.bias = bias;
  p.scale = scale;
  p.weights = weights;
  p.experts = experts;
  p.offsets = offsets;
  p.row_token = row_token;
  p.token_row = token_row;
  p.hist = static_cast<int32_t*>(workspace);
  route_shape(T, p.blocks, p.per_block);
  const void* k = bf16 ? pick_kernel<__nv_bfloat16>(E, bias != nullptr)
                       : pick_kernel<float>(E, bias != nullptr);
  cudaError_t e = launch_dependent(k, p.blocks, p, st);
  if (e == cudaSuccess && p.blocks > 1)
    e = launch_dependent(reinterpret_cast<const void*>(moe_scatter_kernel), p.blocks, p, st);
  return e;
}

}  // namespace sq
