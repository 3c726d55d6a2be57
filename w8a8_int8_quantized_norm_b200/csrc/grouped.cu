// grouped.cu -- the 8-bit GEMM of rows grouped by expert, each group with its
// own weights, and the fused dequantising epilogue, on the sm_100a tensor cores
// (tcgen05 + tensor memory + TMA).  ("SmoothQuant, in depth" -- "Granularity":
// an INT32 accumulator, both scales in the epilogue.)
//
// The group sizes are on the device and ragged, so the weights take the MMA's M
// side -- full blocks of 128 (256 on a CTA pair) weight rows whatever the
// groups are -- and the tokens its N side, whose width is set per tile in the
// instruction descriptor: an expert with c rows runs ceil(c / QT) tiles of
// equal width, rounded up to 16 (pairs: 32) rows, so a small or ragged group
// costs MMA time and token loads for little more than its own rows.
//   pair tiles   (prefill) 256 weight rows x up to 256 tokens on a CTA pair
//                (cta_group::2), two accumulators in tensor memory;
//   decode tiles 128 weight rows x up to 32 tokens per CTA, eight stages in
//                flight (ten measured the same).
// Every CTA first turns the offsets into a table of the non-empty experts and
// their tiles; persistent CTAs then walk the flattened tiles, a weight block's
// token tiles next to each other, so a weight byte comes from HBM once.
// Tokens are gathered by TMA (tile::gather4: four rows at their own row
// coordinates per instruction), so sorting the rows by expert never copies them.
// Measured (int8, 8192 x 4096 weights): 8 groups of 1024 rows 154 to 160 us
// contiguous (3579 to 3436 TOPS), 175 to 182 us gathered, 71 % of the tensor
// pipe's cycles at 4096 tokens spread unevenly; one token's two experts 15 us
// (67 MB, 0.65 of HBM).  Bound by the MMA and the delivery of its operands,
// decode tiles by the weight stream (fp8, 32 tokens over 59 of 64 experts 2048 x
// 4096: 83 us, 500 MB).
// Warp roles as in gemm.cu: 0 producer, 1 MMA issuer, 2-5 epilogue, 6 the
// issuer's scheduler; 7-10 gather tokens.  Every wait is bounded; one that runs
// out records SQ_ERR_PIPELINE_TIMEOUT and the CTAs drain and return.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "sq_device.cuh"
#include "sq_launch.h"

namespace sq {
namespace {

constexpr int BK = 128;      // K bytes per stage = one 128-byte swizzle atom row
constexpr int UMMA_K = 32;   // K of one 8-bit MMA
constexpr int kSchedWarp = 6;
constexpr int kGatherWarp = 7;   // first of the warps that gather tokens
constexpr int kGatherWarps = 4;
constexpr int kThreads = 32 * (kGatherWarp + kGatherWarps);
constexpr int kMaxExperts = SQ_MOE_MAX_EXPERTS;
constexpr int kBand = 16;    // token tiles of a band: their codes stay in L2 while it sweeps N
constexpr int kBoxes = 4;    // token boxes of 128, 64, 32 and 16 contiguous rows

template <bool kPair>
struct Cfg {
  static constexpr int QT = kPair ? 256 : 32;          // tokens of a tile at most
  static constexpr int GRAIN = kPair ? 32 : 16;        // tile widths are multiples of this
  static constexpr int PT = kPair ? 256 : 128;         // weight rows of a tile
  static constexpr int Q_LOCAL = kPair ? QT / 2 : QT;  // token rows a CTA loads at most
  static constexpr int A_BYTES = 128 * BK;
  static constexpr int B_BYTES = Q_LOCAL * BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = kPair ? 6 : 8;
  static constexpr int TMEM_COLS = kPair ? 512 : 64;   // two accumulators
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int OUT_BYTES = kPair ? 32 * 128 * 2 : 0;  // 32 tokens of bf16 outputs, twice
  static constexpr int XS_BYTES = kPair ? QT * 4 : 0;         // a tile's token scales, twice
  static constexpr int OUT = STAGES * STAGE_BYTES;
  static constexpr int XS = OUT + 2 * OUT_BYTES;
  static constexpr int TABLE = XS + 2 * XS_BYTES;
  static constexpr int BARS = TABLE + kMaxExperts * 16;
  static constexpr int SMEM_BYTES = 1024 + BARS + 8 * NUM_BARS + 16;
  static constexpr int GATHER = Q_LOCAL / kGatherWarps;  // rows a gather warp loads at most
  static_assert(GATHER <= 32 && GATHER % 4 == 0, "a lane finds one row's token");
  static_assert((kPair ? GRAIN / 2 : GRAIN) % (4 * kGatherWarps) == 0, "a gather4 per warp");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms need 1024-byte aligned stages");
};

// Token maps: [0] gathers (boxes of one row) or [0 .. kBoxes) contiguous boxes.
struct TokenMaps {
  CUtensorMap m[kBoxes];
};

struct GroupedParams {
  const float* x_scale;
  const float* w_scale;
  const int32_t* offsets;
  const int32_t* row_token;
  void* out;
  int64_t ldo;
  int X, R, E, N, k_blocks, p_blocks, epi;
  int vec_out;          // output rows 16-byte aligned
  int64_t wait_polls;   // > 0: poll budget per wait; 0: ~2 s of SM clock cycles
  int* error_word;
};

// A non-empty expert: its rows are [begin, begin + count), its tiles the
// flattened units up to unit_end.
struct Entry {
  int expert, begin, count, unit_end;
};

template <bool kPair>
__device__ __forceinline__ int tiles_of(int count) {
  return (count + Cfg<kPair>::QT - 1) / Cfg<kPair>::QT;
}

// The table, by one warp; returns the number of entries (in every lane).  The
// offsets count as their running maximum within [0, R]: whatever they hold, no
// two groups share a row and the tiles are no more than the host allowed for.
template <bool kPair>
__device__ int build_table(const GroupedParams& p, Entry* table, int lane) {
  int entries = 0, units = 0, reached = 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane;
    int begin = 0, end = 0;
    if (e < p.E) {
      begin = min(max(__ldg(p.offsets + e), 0), p.R);
      end = min(max(__ldg(p.offsets + e + 1), 0), p.R);
    }
    begin = max(begin, reached);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int u = __shfl_up_sync(~0u, begin, s);
      if (lane >= s) begin = max(begin, u);
    }
    const int count = max(end - begin, 0);
    reached = __shfl_sync(~0u, max(begin, end), 31);
    const int mine = tiles_of<kPair>(count) * p.p_blocks;
    int inc = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int u = __shfl_up_sync(~0u, inc, s);
      if (lane >= s) inc += u;
    }
    const uint32_t active = __ballot_sync(~0u, count > 0);
    if (count > 0)
      table[entries + __popc(active & ((1u << lane) - 1u))] = Entry{e, begin, count, units + inc};
    entries += __popc(active);
    units += __shfl_sync(~0u, inc, 31);
  }
  return entries;
}

struct Tile {
  int expert, pb, row0, rows, width;  // width: rows rounded up to the grain
};

// The tiles of one cluster, in order; every warp role walks the same sequence.
template <bool kPair>
struct Walk {
  const Entry* table;
  int entries, p_blocks, u, step, i, first;
  __device__ __forceinline__ Walk(const GroupedParams& p, const Entry* t, int n, int id, int count)
      : table(t), entries(n), p_blocks(p.p_blocks), u(id), step(count), i(0), first(0) {}
  // Called by whole warps; the shuffles make what is read uniform, so that TMA
  // coordinates stay in uniform registers.
  __device__ __forceinline__ Entry entry(int k) const {
    const Entry e = table[k];
    return Entry{__shfl_sync(~0u, e.expert, 0), __shfl_sync(~0u, e.begin, 0),
                 __shfl_sync(~0u, e.count, 0), __shfl_sync(~0u, e.unit_end, 0)};
  }
  __device__ __forceinline__ bool next(Tile& t) {
    if (i >= entries) return false;
    Entry e = entry(i);
    while (u >= e.unit_end) {
      first = e.unit_end;
      if (++i >= entries) return false;
      e = entry(i);
    }
    const int q_tiles = tiles_of<kPair>(e.count);
    const int grain = Cfg<kPair>::GRAIN;
    const int width = ((e.count + q_tiles - 1) / q_tiles + grain - 1) / grain * grain;
    // bands of token tiles sweep the weight blocks, a block's tiles together
    const int idx = u - first;
    const int band = idx / (kBand * p_blocks);
    const int rem = idx - band * kBand * p_blocks;
    const int size = min(kBand, q_tiles - band * kBand);
    const int qb = band * kBand + rem % size;
    t.expert = e.expert;
    t.pb = rem / size;
    t.row0 = e.begin + qb * width;
    t.rows = min(width, e.count - qb * width);
    t.width = (t.rows + grain - 1) / grain * grain;
    u += step;
    return true;
  }
};

// The four epilogue warps only; true where any of them gave up.
__device__ __forceinline__ bool epilogue_sync(bool stop) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 2, 128, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(stop ? 1u : 0u)
      : "memory");
  return r != 0;
}

// In place of the scale of a row without a token: its outputs are zeros.
constexpr uint32_t kNoToken = 0x80000000u;

template <bool kF8>
__device__ __forceinline__ float acc_value(uint32_t r) {
  if constexpr (kF8) return __uint_as_float(r);
  else return __int2float_rn(static_cast<int>(r));
}

template <bool kPair, bool kF8>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap mapW,
                        const __grid_constant__ TokenMaps mapX, const GroupedParams prm) {
  using C = Cfg<kPair>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw_u32);
  const uint32_t a_base = base;
  const uint32_t b_base = base + STAGES * C::A_BYTES;
  Entry* table = reinterpret_cast<Entry*>(base_ptr + C::TABLE);
  const uint32_t bar_base = base + C::BARS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base_ptr + C::BARS + 8 * C::NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* entries_slot = reinterpret_cast<int*>(tmem_slot + 2);
#define FULL_BAR(s) (bar_base + 8u * static_cast<uint32_t>(s))
#define EMPTY_BAR(s) (bar_base + 8u * static_cast<uint32_t>(STAGES + (s)))
#define TFULL_BAR(a) (bar_base + 8u * static_cast<uint32_t>(2 * STAGES + (a)))
#define TEMPTY_BAR(a) (bar_base + 8u * static_cast<uint32_t>(2 * STAGES + 2 + (a)))
#define DRAIN_BAR (bar_base + 8u * static_cast<uint32_t>(2 * STAGES + 4))

  const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;
  const int rank = kPair ? __shfl_sync(~0u, static_cast<int>(cluster_ctarank()), 0) : 0;
  const bool issues = rank == 0;  // this CTA's warp 1 issues MMAs
  const int id = static_cast<int>(blockIdx.x) / (kPair ? 2 : 1);
  const int workers = static_cast<int>(gridDim.x) / (kPair ? 2 : 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(FULL_BAR(s), 1);
      mbar_init(EMPTY_BAR(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(TFULL_BAR(a), 1);
      mbar_init(TEMPTY_BAR(a), kPair ? 8 : 4);
    }
    mbar_init(DRAIN_BAR, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&mapW);
    tma_prefetch_desc(&mapX.m[0]);
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  // programmatic launch: the next kernel may be scheduled; this one reads and
  // writes global memory only after the previous grid has completed
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 0) {
    const int n = build_table<kPair>(prm, table, lane);
    if (lane == 0) *entries_slot = n;
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync_all();  // every CTA's barriers exist before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(~0u, *tmem_slot, 0);
  const int entries = __shfl_sync(~0u, *entries_slot, 0);
  const int64_t polls = prm.wait_polls;
  Walk<kPair> walk(prm, table, entries, id, workers);
  Tile t;

  // a wait ran out: stop this CTA and its partner
  auto give_up = [&]() {
    fail(prm.error_word, abort_flag);
    if (kPair) st_cluster_u32(map_to_cta(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1), 1u);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && walk.next(t)) {
      const int local = kPair ? t.width >> 1 : t.width;  // token rows this CTA loads
      const int j0 = kPair ? rank * local : 0;
      const int w_row = t.expert * prm.N + t.pb * C::PT + (kPair ? rank * 128 : 0);
      for (int kb = 0; kb < prm.k_blocks; ++kb) {
        if (!__all_sync(~0u, wait_phase(EMPTY_BAR(stage), phase ^ 1u, polls, abort_flag))) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        const uint32_t sa = a_base + stage * C::A_BYTES, sb = b_base + stage * C::B_BYTES;
        // a pair's loads complete on the leader's barrier
        const uint32_t fb = kPair && rank ? map_to_cta(FULL_BAR(stage), 0) : FULL_BAR(stage);
        if (elect_one()) {
          const uint32_t bytes = C::A_BYTES + local * BK;
          if (issues) mbar_arrive_expect_tx(FULL_BAR(stage), kPair ? 2 * bytes : bytes);
          if constexpr (kPair) tma_load_2d_pair(sa, &mapW, fb, kb * BK, w_row);
          else tma_load_2d(sa, &mapW, fb, kb * BK, w_row);
          if (!prm.row_token) {
            // the tile's rows as boxes of falling powers of two
            int j = 0;
#pragma unroll
            for (int i = 0; i < kBoxes; ++i) {
              const int rows = 128 >> i;
              if (j + rows <= local) {
                if constexpr (kPair)
                  tma_load_2d_pair(sb + j * BK, &mapX.m[i], fb, kb * BK, t.row0 + j0 + j);
                else
                  tma_load_2d(sb + j * BK, &mapX.m[i], fb, kb * BK, t.row0 + j0 + j);
                j += rows;
              }
            }
          }
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (issues) {
      int stage = 0;
      int acc = 0;
      bool ok = true;
      while (ok && walk.next(t)) {
        const uint32_t idesc = kF8 ? idesc_f8(C::PT, t.width) : idesc_i8(C::PT, t.width);
        if (sched_sync(false)) break;  // the scheduler saw the accumulator free (or gave up)
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::QT);
        for (int kb = 0; kb < prm.k_blocks; ++kb) {
          if (sched_sync(false)) {  // the scheduler saw this stage land (or gave up)
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = a_base + stage * C::A_BYTES;
            const uint32_t sb = b_base + stage * C::B_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / UMMA_K; ++kk) {
              const uint64_t da = smem_desc_k_sw128(sa + kk * UMMA_K);
              const uint64_t db = smem_desc_k_sw128(sb + kk * UMMA_K);
              const uint32_t add = (kb > 0 || kk > 0) ? 1u : 0u;
              if constexpr (kPair && kF8) mma_f8_pair(d_tmem, da, db, idesc, add);
              else if constexpr (kPair) mma_i8_pair(d_tmem, da, db, idesc, add);
              else if constexpr (kF8) mma_f8(d_tmem, da, db, idesc, add);
              else mma_i8(d_tmem, da, db, idesc, add);
            }
            if constexpr (kPair) {
              mma_commit_pair(EMPTY_BAR(stage));
              mma_commit_pair(map_to_cta(EMPTY_BAR(stage), 1));
            } else {
              mma_commit(EMPTY_BAR(stage));
            }
          }
          __syncwarp();
          if (++stage == STAGES) stage = 0;
        }
        if (!ok) break;
        if (elect_one()) {  // the same lane every time: a commit covers its thread's MMAs
          if constexpr (kPair) {
            mma_commit_pair(TFULL_BAR(acc));
            mma_commit_pair(map_to_cta(TFULL_BAR(acc), 1));
          } else {
            mma_commit(TFULL_BAR(acc));
          }
        }
        __syncwarp();
        acc ^= 1;
      }
      if (elect_one()) {
        // every MMA issued by this thread completes before tensor memory is freed
        if constexpr (kPair) mma_commit_pair(DRAIN_BAR);
        else mma_commit(DRAIN_BAR);
        wait_phase(DRAIN_BAR, 0, 0, nullptr);
      }
      __syncwarp();
    }
  } else if (warp == kSchedWarp) {
    // ------------------------------------------------------------ MMA scheduler
    if (issues) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      while (ok && walk.next(t)) {
        bool w = false;
        if (lane == 0) w = wait_phase(TEMPTY_BAR(acc), acc_phase ^ 1u, polls, abort_flag);
        w = __shfl_sync(~0u, w, 0);
        if (!w && lane == 0) give_up();
        if (sched_sync(!w)) break;
        for (int kb = 0; kb < prm.k_blocks; ++kb) {
          w = false;
          if (lane == 0) w = wait_phase(FULL_BAR(stage), phase, polls, abort_flag);
          w = __shfl_sync(~0u, w, 0);
          if (!w && lane == 0) give_up();
          if (sched_sync(!w)) {
            ok = false;
            break;
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
  } else if (warp >= kGatherWarp) {
    // ------------------------------------------------------------ token gather
    // An elected lane issues: a tile::gather4 takes uniform coordinates, and a
    // warp whose lanes issue one each serialises them (measured 90 cycles
    // apart: 2.3x the time of the whole tile).
    if (prm.row_token) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      // The token of this lane's row, a tile ahead: the load's latency passes
      // while the tile before is copied.  Every warp takes a quarter of a tile
      // (a multiple of 4 rows): each has bytes in every stage, so none falls a
      // phase behind the ring.
      auto find = [&](const Tile& a) {
        const int local = kPair ? a.width >> 1 : a.width;
        const int mine = local / kGatherWarps;
        const int j = (kPair ? rank * local : 0) + (warp - kGatherWarp) * mine + lane;
        return lane < mine && j < a.rows ? __ldg(prm.row_token + a.row0 + j) : 0;
      };
      bool live = walk.next(t);
      int found = live ? find(t) : 0;
      while (ok && live) {
        Tile ahead;
        const bool more = walk.next(ahead);
        const int found_ahead = more ? find(ahead) : 0;
        const int mine = (kPair ? t.width >> 1 : t.width) / kGatherWarps;
        const int g0 = (warp - kGatherWarp) * mine;
        // a row past the tile, or of no token, loads token 0: its column is
        // dropped, or zeroed, by the epilogue
        if (found < 0 || found >= prm.X) found = 0;
        int src[C::GATHER];
#pragma unroll
        for (int i = 0; i < C::GATHER; ++i) src[i] = __shfl_sync(~0u, found, i);
        for (int kb = 0; kb < prm.k_blocks; ++kb) {
          if (!__all_sync(~0u, wait_phase(EMPTY_BAR(stage), phase ^ 1u, polls, abort_flag))) {
            if (lane == 0) give_up();
            ok = false;
            break;
          }
          const uint32_t fb = kPair && rank ? map_to_cta(FULL_BAR(stage), 0) : FULL_BAR(stage);
          const uint32_t sb = b_base + stage * C::B_BYTES + g0 * BK;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < C::GATHER; i += 4) {
              if (i < mine) {
                const int rows[4] = {src[i], src[i + 1], src[i + 2], src[i + 3]};
                if constexpr (kPair) tma_gather4_pair(sb + i * BK, &mapX.m[0], fb, kb * BK, rows);
                else tma_gather4(sb + i * BK, &mapX.m[0], fb, kb * BK, rows);
              }
            }
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        t = ahead;
        live = more;
        found = found_ahead;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;  // tensor-memory lanes this warp may access
    const int p_local = quarter * 32 + lane;
    const bool raw = prm.epi == SQ_EPI_I32_RAW || prm.epi == SQ_EPI_F32_RAW;
    const bool relu = prm.epi == SQ_EPI_BF16_RELU;
    const int et = static_cast<int>(threadIdx.x) - 64;
    float* xs_smem = reinterpret_cast<float*>(base_ptr + C::XS);
    int acc = 0;
    uint32_t acc_phase = 0;
    // What a tile needs from global memory, loaded ahead of it: its rows' tokens
    // two tiles before, their scales and the columns' scale one tile before, so
    // that neither latency falls between two tiles (few K blocks: it was most
    // of the tile's time).  Pair tiles: thread et holds tokens et and et + 128;
    // decode tiles: lane l token l.
    constexpr int NT = kPair ? 2 : 1;
    struct Ahead {
      Tile t;
      bool live;
      int src[NT];
      float xs[NT], ws;
    };
    auto load_rows = [&](Ahead& a) {
      a.live = walk.next(a.t);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int j = kPair ? et + 128 * i : lane;
        a.src[i] = -1;
        if (a.live && j < a.t.rows) {
          a.src[i] = a.t.row0 + j;
          if (prm.row_token) a.src[i] = __ldg(prm.row_token + a.src[i]);
        }
      }
    };
    auto column = [&](const Tile& a) { return a.pb * C::PT + (kPair ? rank * 128 : 0) + p_local; };
    auto load_scales = [&](Ahead& a) {
      if (!a.live) return;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        a.xs[i] = __uint_as_float(kNoToken);
        if (a.src[i] >= 0 && a.src[i] < prm.X)
          a.xs[i] = raw ? 1.0f : __ldg(prm.x_scale + a.src[i]);
      }
      const int n = column(a.t);
      a.ws = !raw && n < prm.N
                 ? __ldg(prm.w_scale + static_cast<int64_t>(a.t.expert) * prm.N + n) : 0.0f;
    };
    Ahead cur, nxt, far;
    load_rows(cur);
    load_rows(nxt);
    load_scales(cur);
    for (; cur.live; cur = nxt, nxt = far) {
      load_rows(far);
      load_scales(nxt);
      t = cur.t;
      const float ws = cur.ws;
      const int n = column(t);  // this thread's output column
      const bool n_in = n < prm.N;
      if constexpr (kPair) {
#pragma unroll
        for (int i = 0; i < NT; ++i) xs_smem[acc * C::QT + et + 128 * i] = cur.xs[i];
      }
      bool w = false;
      if (lane == 0) w = wait_phase(TFULL_BAR(acc), acc_phase, polls, abort_flag);
      w = __shfl_sync(~0u, w, 0);
      if (!w && lane == 0) give_up();
      if constexpr (kPair) {
        // the tile's token scales are in shared memory, and no warp waits for
        // one that gave up: past this point a tile has no way out but its end
        if (epilogue_sync(!w)) break;
      } else {
        if (!w) break;
      }
      tc_fence_after();
      const uint32_t trow = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                            static_cast<uint32_t>(acc * C::QT);
      if constexpr (kPair) {
        const float* xs_tile = xs_smem + acc * C::QT;
#pragma unroll 1
        for (int c = 0; c < t.rows; c += 32) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_32x32b_x32(trow + static_cast<uint32_t>(c), r);
          tmem_wait_ld();
          if (c + 32 >= t.rows) {  // the accumulator is read: free it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (rank) mbar_arrive_cluster(map_to_cta(TEMPTY_BAR(acc), 0));
              else mbar_arrive(TEMPTY_BAR(acc));
            }
          }
          const int64_t row = t.row0 + c;
          if (raw) {
            uint32_t* dst = static_cast<uint32_t*>(prm.out) + row * prm.ldo + n;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (c + j < t.rows && n_in)
                *dst = __float_as_uint(xs_tile[c + j]) == kNoToken ? 0u : r[j];
              dst += prm.ldo;
            }
            continue;
          }
          __nv_bfloat16 v[32];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 x4 = *reinterpret_cast<const float4*>(xs_tile + c + j);
            const float xs[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float f = __fmul_rn(__fmul_rn(acc_value<kF8>(r[j + i]), xs[i]), ws);
              if (__float_as_uint(xs[i]) == kNoToken) f = 0.0f;
              if (relu) f = f > 0.0f ? f : 0.0f;  // -0 (a zero scale) becomes +0
              v[j + i] = __float2bfloat16_rn(f);
            }
          }
          if (!prm.vec_out) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(prm.out) + row * prm.ldo + n;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (c + j < t.rows && n_in) *dst = v[j];
              dst += prm.ldo;
            }
            continue;
          }
          // lanes hold columns, rows are contiguous in memory: through shared
          // memory, 256-byte pieces of the rows leave as 16-byte stores (the
          // 2-byte stores above took 12.6 us of a 256 x 256 tile)
          __nv_bfloat16* out_buf = reinterpret_cast<__nv_bfloat16*>(base_ptr + C::OUT) +
                                   ((c >> 5) & 1) * (C::OUT_BYTES / 2);
#pragma unroll
          for (int j = 0; j < 32; ++j) out_buf[j * 128 + p_local] = v[j];
          epilogue_sync(false);  // two buffers: the next write here is two syncs away
          const int col = t.pb * C::PT + rank * 128 + (et & 15) * 8;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = (et >> 4) + 8 * k;
            if (c + j < t.rows && col < prm.N) {
              const uint4 w4 = *reinterpret_cast<const uint4*>(out_buf + j * 128 + (et & 15) * 8);
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(prm.out) + (row + j) * prm.ldo + col;
              if (col + 8 <= prm.N) {
                *reinterpret_cast<uint4*>(dst) = w4;
              } else {
                const uint32_t u[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (col + i < prm.N)
                    reinterpret_cast<uint16_t*>(dst)[i] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
              }
            }
          }
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
        continue;
      }
      {  // QT = 32: one chunk
        uint32_t r[32];
        __syncwarp();
        tmem_ld_32x32b_x32(trow, r);
        const uint32_t zero = __ballot_sync(~0u, __float_as_uint(cur.xs[0]) == kNoToken);
        tmem_wait_ld();
        if (raw) {
          uint32_t* dst = static_cast<uint32_t*>(prm.out) + static_cast<int64_t>(t.row0) * prm.ldo + n;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (j < t.rows && n_in) *dst = (zero >> j) & 1u ? 0u : r[j];
            dst += prm.ldo;
          }
        } else {
          __nv_bfloat16* dst =
              static_cast<__nv_bfloat16*>(prm.out) + static_cast<int64_t>(t.row0) * prm.ldo + n;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float xs = __shfl_sync(~0u, cur.xs[0], j);
            float v = __fmul_rn(__fmul_rn(acc_value<kF8>(r[j]), xs), ws);
            if ((zero >> j) & 1u) v = 0.0f;
            if (relu) v = v > 0.0f ? v : 0.0f;  // -0 (a zero scale) becomes +0
            if (j < t.rows && n_in) *dst = __float2bfloat16_rn(v);
            dst += prm.ldo;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(TEMPTY_BAR(acc));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  __syncthreads();
  if (kPair) cluster_sync_all();  // no MMA, load signal or remote store is pending
  if (*abort_flag) {
    // after an abort some loads may still be in flight, and the barriers that
    // would tell may never complete: about 20 ms, thousands of times a load's
    // latency, pass before the shared memory is given back
    const long long t0 = clock64();
    while (clock64() - t0 < 40000000LL) {
    }
  }
  __syncthreads();
  if (kPair) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
#undef FULL_BAR
#undef EMPTY_BAR
#undef TFULL_BAR
#undef TEMPTY_BAR
#undef DRAIN_BAR
}

template <bool kPair, bool kF8>
cudaError_t launch(const CUtensorMap& mw, const TokenMaps& mx, const GroupedParams& prm,
                   int64_t max_units, int sms, cudaStream_t st) {
  using C = Cfg<kPair>;
  auto kern = grouped_gemm_kernel<kPair, kF8>;
  cudaError_t e = launch_cache().ensure_smem(reinterpret_cast<const void*>(kern), C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  constexpr int csize = kPair ? 2 : 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(csize);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  int64_t clusters = sms / csize;
  if (kPair) {
    // as many pairs as the device holds at once, asked once per device
    static std::atomic<int> held[64];
    const int dev = LaunchCache::device();
    int n = dev >= 0 && dev < 64 ? held[dev].load() : 0;
    if (n == 0) {
      cfg.gridDim = dim3(static_cast<unsigned>(clusters * csize));
      if ((e = resident_clusters(&n, kern, &cfg)) != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) held[dev].store(n);
    }
    if (n < clusters) clusters = n;
  }
  if (max_units < clusters) clusters = max_units;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * csize));
  return cudaLaunchKernelEx(&cfg, kern, mw, mx, prm);
}

// Decode tiles while an expert has few rows: they keep more weight blocks in
// flight and need no cluster; past 32 rows an expert's weights would be read
// again for every 32.  The sizes are on the device, so the mean has to decide:
// even groups turn between 32 and 48 rows, skewed ones earlier.  Decode / pair in
// us (the timing's own 5 in both), even, and with half of the rows at one expert:
//   rows an expert          16          24          32          48          96
//   64 x 2048 x 4096 fp8  90 / 94     90 / 95     90 / 96    111 / 98   153 / 102
//     skewed              99 / 102   105 / 101   112 / 102   123 / 103  178 / 118
//   16 x 4000 x 1040      21 / 23     22 / 24     22 / 24     27 / 25    35 / 27
//     skewed              23 / 25     23 / 25     23 / 26     26 / 25    37 / 27
//   8 x 8192 x 4096       51 / 55     51 / 55     51 / 55     59 / 57    82 / 58
//     skewed              51 / 55     55 / 55     56 / 56     61 / 56    91 / 58
bool pair_tiles(int64_t R, int64_t E, int path_hint) {
  return path_hint == 1 || (path_hint == 0 && R > 24 * E);
}

}  // namespace

int64_t grouped_tiles(int64_t R, int64_t E, int64_t N, int path_hint) {
  const bool pair = pair_tiles(R, E, path_hint);
  const int64_t pt = pair ? Cfg<true>::PT : Cfg<false>::PT, qt = pair ? Cfg<true>::QT : Cfg<false>::QT;
  return ((R + qt - 1) / qt + (E < R ? E : R)) * ((N + pt - 1) / pt);
}

cudaError_t launch_gemm_grouped(const void* Xq, int64_t X, const void* Wq, const float* x_scale,
                                const float* w_scale, const int32_t* offsets,
                                const int32_t* row_token, int64_t R, int64_t E, int64_t N,
                                int64_t K, int epi, void* out, int64_t ldo, int path_hint,
                                int num_sms, int64_t wait_polls, int* error_word, bool fp8,
                                cudaStream_t st) {
  const int sms = num_sms > 0 ? num_sms : 148;
  const bool pair = pair_tiles(R, E, path_hint);
  GroupedParams p{};
  p.x_scale = x_scale;
  p.w_scale = w_scale;
  p.offsets = offsets;
  p.row_token = row_token;
  p.out = out;
  p.ldo = ldo;
  p.X = static_cast<int>(X);
  p.R = static_cast<int>(R);
  p.E = static_cast<int>(E);
  p.N = static_cast<int>(N);
  p.k_blocks = static_cast<int>((K + BK - 1) / BK);
  const int pt = pair ? Cfg<true>::PT : Cfg<false>::PT;
  p.p_blocks = static_cast<int>((N + pt - 1) / pt);
  p.epi = epi;
  p.vec_out = (reinterpret_cast<uintptr_t>(out) & 15u) == 0 && ldo % 8 == 0;
  p.wait_polls = wait_polls;
  p.error_word = error_word;
  const int64_t max_units = grouped_tiles(R, E, N, path_hint);
  CUtensorMap mw;
  TokenMaps mx;
  bool ok = make_code_map(&mw, Wq, E * N, K, 128);
  if (row_token) {
    ok = ok && make_code_map(&mx.m[0], Xq, X, K, 1);
  } else {
    for (int i = 0; i < kBoxes; ++i) ok = ok && make_code_map(&mx.m[i], Xq, X, K, 128 >> i);
  }
  if (!ok) return cudaErrorInvalidValue;
  if (pair)
    return fp8 ? launch<true, true>(mw, mx, p, max_units, sms, st)
               : launch<true, false>(mw, mx, p, max_units, sms, st);
  return fp8 ? launch<false, true>(mw, mx, p, max_units, sms, st)
             : launch<false, false>(mw, mx, p, max_units, sms, st);
}

}  // namespace sq
