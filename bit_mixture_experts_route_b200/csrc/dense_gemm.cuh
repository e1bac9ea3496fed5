// Dense 16-bit GEMM on the 5th-generation tensor cores, the core of the
// gated feed-forward block (ffn.cu) and of the vocabulary cross entropy
// (linear_ce.cu): D[m, n] = sum_k A[m, k] B[n, k], fp32 sums in tensor memory,
// with the operator's own arithmetic in the epilogue.
//
// Either operand may lie the other way round (its m or n index contiguous
// instead of k): the products of a backward pass read the forward's matrices
// as they are, through the MN-major forms of the shared-memory descriptor, and
// nothing is transposed in memory.
//
// Work split.  A cluster of two CTAs (two SMs) computes a 256 x 256 tile with
// tcgen05.mma.cta_group::2: each CTA loads 128 rows of A and 128 rows of B per
// 64-k stage (32 KB), so a tile reads 64 KB per 256 x 256 x 64 MACs -- half of
// what two separate 128 x 256 tiles would read -- and each CTA's 128 x 256
// accumulator block sits in its own tensor memory.  Two accumulators of 256
// columns fill the 512 columns, so the epilogue of one tile runs under the
// MMAs of the next.  Persistent: every pair walks units u = pair, pair +
// pairs, ... of a list of (tile, k split), tiles ordered in groups of GROUP_M
// row tiles so that the pairs running together share operand tiles in L2.
//
// Warp roles (384 threads): warp 0 loads (TMA), warp 1 issues the MMAs (the
// leader CTA's) and owns the tensor memory, warps 4-11 are the epilogue, two
// per TMEM lane quarter, each taking 128 of the tile's 256 columns.  16-bit
// results go through a 128-byte-swizzled staging block per warp (32 rows x 64
// columns) and leave by TMA, which clips at the matrix's edge; ragged sizes
// read as zeros.  Every wait is bounded: on expiry MOE_DEVERR_TIMEOUT is set
// and the kernel drains its copies and MMAs and returns.
#pragma once

#include "tc_ops.cuh"

namespace moe {
namespace dense {

using namespace moe::tc;

constexpr int CM = 128;              // rows of A (and of B) per CTA and stage
constexpr int TILE = 256;            // rows of the pair's tile; its columns TN: 256 or 128
constexpr int GK = 64;               // k per stage
constexpr int OPERAND = CM * GK * 2; // 16 KB of A
constexpr int stage_bytes(int tn) { return OPERAND + tn / 2 * GK * 2; }  // A then B, per CTA
constexpr int EPI_W0 = 4, EPI_NW = 8;
constexpr int GEMM_THREADS = 32 * (EPI_W0 + EPI_NW);
constexpr int STG = 32 * 128;        // one staging block: 32 rows x 128 bytes
constexpr int GROUP_M = 8;
constexpr int TILE_FLOATS = TILE * TILE;  // a tile of fp32 partial sums, [column][row]
constexpr float kLog2e = 1.4426950408889634f;

// What the epilogue does with the sums.
enum Epilogue {
  E_STORE,       // D0 = 16-bit (sum * *scale + residual)
  E_STORE2,      // E_STORE of two products with the same k, one unit list
  E_PART,        // partial sums to the workspace, [tile][column][row] fp32
  E_SWIGLU,      // columns are gate [0,128) | up [128,256): D0 = h, D1 = gate | up
  E_SWIGLU_BWD,  // sums are dh: D0 = h, D1 = dgate | dup, from gu
  E_STATS,       // per row and 128 columns: max and sum of exponentials
  E_DLOGITS,     // D0 = (exp(sum - lse) - [column is the target]) * row scale
};
constexpr bool is_swiglu(int epi) { return epi == E_SWIGLU || epi == E_SWIGLU_BWD; }
// Epilogue warps per TMEM lane quarter, each with 128 or 64 columns (E_SWIGLU:
// gate columns and as many up columns).
constexpr int halves_of(int epi, int tn) {
  return epi == E_SWIGLU ? tn / 128 : 2;
}
// Bytes of staging per epilogue warp: blocks of 64 columns that the warp's
// stores take in turn, one (E_SWIGLU), two (E_STORE, E_DLOGITS, so that a short
// reduction's tile need not wait for its store's way out) or three of 32 columns
// (E_SWIGLU_BWD).  More would cost an operand stage, and the loads' way from L2
// needs them: at 4096 x 2048 x 8192, 4 stages kept the tensor cores 71 % busy, 5
// stages 87 %.
constexpr int stg_of(int epi) {
  return epi == E_SWIGLU_BWD ? 3 * STG / 2
         : epi == E_SWIGLU   ? STG
         : (epi == E_PART || epi == E_STATS) ? 0 : 2 * STG;
}
constexpr int stg_bytes(int epi, int tn) { return 4 * halves_of(epi, tn) * stg_of(epi); }
// Which of the two blocks the store `turn` of a warp's unit number `unit` is
// staged in, with `turns` stores in a unit (two of 64 columns in a 256-column
// tile, one in a 128-column tile).  The warp waits for all its stores but the
// newest, so a store never takes the block of the one before it, which may still
// be on its way -- over the end of a unit too.
constexpr int staging_block(int unit, int turn, int turns) { return (unit * turns + turn) & 1; }
constexpr bool staging_alternates(int turns) {
  for (int i = 1; i < 4 * turns; ++i)
    if (staging_block(i / turns, i % turns, turns) ==
        staging_block((i - 1) / turns, (i - 1) % turns, turns))
      return false;
  return true;
}
// As many stages as the shared memory holds beside the staging blocks.
constexpr int kSmemBudget = 227 * 1024 - 1024 - 512;
constexpr int stages_of(int epi, int tn) {
  const int n = (kSmemBudget - stg_bytes(epi, tn)) / stage_bytes(tn);
  return n > 10 ? 10 : n;
}

struct GemmArgs {
  int N;                 // columns (E_SWIGLU: of h)
  int m_tiles, n_tiles;  // tiles of 256 rows; of 256 columns (E_SWIGLU: 128)
  int k_stages;          // ceil(K / 64)
  int splits, kps;       // k splits and stages per split
  const int* splits_of;  // E_PART: device word with the splits (at most `splits`), or null
  // *rows (device) replaces the row count (dyn = 1) or the length of the
  // reduction (dyn = 2); a multiple of 256 rows is readable either way
  const int* rows;
  int dyn;
  float* part;           // E_PART: [split][tile][256][256], the tiles of *rows
  int accumulate;        // E_PART: add to what is there
  const float* residual; // E_STORE: fp32 [rows, N] or null
  const float* scale;    // E_STORE: device scalar or null
  int M;
  const void* gu;        // E_SWIGLU_BWD: [M, 2N] gate | up
  int save;              // E_SWIGLU: write D1; E_SWIGLU_BWD: write D0
  int early;             // B is an input of the whole call: load its first stages at once
  int gate_up;           // E_PART: B and the columns as in E_SWIGLU
  float2* stats;         // E_STATS: [2 n_tiles][rows_pad]
  const float* target_sum;  // E_STATS, E_DLOGITS: the target column's sum of each row
  const int* targets;    // E_STATS, E_DLOGITS: column of each row (relative to this matrix)
  const float* lse;      // E_DLOGITS
  const float* row_scale;
  int col0;              // E_DLOGITS: targets minus col0 are this piece's columns
  int rows_pad;
  int32_t* dev_err;
};

// The second product of E_STORE2.
struct alignas(64) SecondProduct {
  CUtensorMap a, b, d;
  int N, M, m_tiles, n_tiles;
};
struct NoProduct {};
template <int EPI>
using SecondFor = typename std::conditional<EPI == E_STORE2, SecondProduct, NoProduct>::type;

template <int NS, int SB, int NW, int NSTG>
struct __align__(8) GemmSmem {
  uint8_t ab[NS][SB];  // 1024-aligned
  uint8_t stg[NW][NSTG > 0 ? NSTG : 16];
  uint64_t full[NS], empty[NS];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
template <int EPI, int TN>
using GemmSmemFor =
    GemmSmem<stages_of(EPI, TN), stage_bytes(TN), 4 * halves_of(EPI, TN), stg_of(EPI)>;
static_assert(sizeof(GemmSmemFor<E_STORE, 256>) + 1024 <= 227 * 1024, "shared memory budget");
static_assert(sizeof(GemmSmemFor<E_STORE, 128>) + 1024 <= 227 * 1024, "shared memory budget");
static_assert(sizeof(GemmSmemFor<E_SWIGLU, 256>) + 1024 <= 227 * 1024, "shared memory budget");
static_assert(sizeof(GemmSmemFor<E_PART, 256>) + 1024 <= 227 * 1024, "shared memory budget");

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + exp(-x)) by the fast exponential and reciprocal, relative error about
// 1e-6, far below a 16-bit rounding.  The ftz forms spend nothing on subnormal
// arguments; where exp(-x) leaves fp32's range the result is 0.
__device__ __forceinline__ float sigmoid_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_approx(-kLog2e * x)));
  return r;
}

// The activation backward of h = silu(g) u for the gradient dh of h, with
// s = sigmoid(g): dg = dh u s (1 + g (1 - s)), du = dh g s; and h again.
struct SwigluGrad {
  float h, dg, du;
};
__device__ __forceinline__ SwigluGrad swiglu_grad(float dh, float g, float u) {
  const float s = sigmoid_fast(g), silu = g * s;
  return {silu * u, dh * u * (s + silu * (1.0f - s)), dh * silu};
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t cluster_bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x,
                                             int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y,
                                             int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Shared-memory descriptor of an operand tile.  K-major: 128 rows of 128
// bytes (64 k), 8-row groups 1024 bytes apart.  MN-major: two blocks of 64
// rows, each 64 k-lines of 128 bytes (64 rows): 8 k-lines are 1024 bytes (the
// stride offset), the blocks 8192 bytes (the leading offset).  A k step of 16
// is 32 bytes further in the first, 16 k-lines = 2048 bytes in the second.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
  uint64_t d = sw128_desc(saddr);
  if (MN) d = (d & ~((uint64_t)0x3FFF << 16)) | ((uint64_t)(8192u >> 4) << 16);
  return d;
}
template <bool MN>
constexpr uint32_t kstep_units() {
  return (MN ? 2048u : 32u) >> 4;
}

// Instruction descriptor: D fp32, A and B of T, M = 256, N = TN.
template <typename T, bool AMN, bool BMN, int TN>
__device__ __forceinline__ constexpr uint32_t gemm_idesc() {
  const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((AMN ? 1u : 0u) << 15) | ((BMN ? 1u : 0u) << 16) |
         ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
}

__device__ __forceinline__ void mma_ss_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Unit u -> its tile and its k stages [k0, k1).  Tiles run down GROUP_M row
// tiles before they step to the next column.
struct Unit {
  int mt, nt, split, k0, k1;
};
__device__ __forceinline__ Unit unit_of(int u, int m_tiles, int n_tiles, int k_stages, int kps) {
  Unit r;
  const int tiles = m_tiles * n_tiles;
  r.split = u / tiles;
  const int t = u - r.split * tiles;
  const int per = GROUP_M * n_tiles;
  const int grp = t / per, first = grp * GROUP_M;
  const int gm = min(GROUP_M, m_tiles - first);
  const int in = t - grp * per;
  r.nt = in / gm;
  r.mt = first + in - r.nt * gm;
  r.k0 = min(k_stages, r.split * kps);
  r.k1 = min(k_stages, r.k0 + kps);
  return r;
}

// Splits of the reduction for `tiles` tiles of `k_stages` stages on `pairs`
// pairs, at most `most` (<= 32): the rounds of units (whole tiles or parts of
// them) that the busiest pair runs, each its stages and about 6 more to fill
// and drain.  A lane of the calling warp looks at one number each.
__device__ inline int even_splits(int tiles, int k_stages, int most, int pairs) {
  const int sp = (threadIdx.x & 31) + 1;
  int cost = INT32_MAX;
  if (sp <= most && sp <= k_stages) {
    const int kps = (k_stages + sp - 1) / sp;
    if ((k_stages + kps - 1) / kps == sp)  // no empty last split
      cost = (tiles * sp + pairs - 1) / pairs * (kps + 6);
  }
  const int least = __reduce_min_sync(0xffffffffu, cost);
  return __ffs(__ballot_sync(0xffffffffu, cost == least));
}

template <typename T, bool AMN, bool BMN, int EPI, int TN>
__global__ void __launch_bounds__(GEMM_THREADS, 1) dense_gemm_kernel(
    const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
    const __grid_constant__ CUtensorMap dmap0, const __grid_constant__ CUtensorMap dmap1,
    const __grid_constant__ GemmArgs p, const __grid_constant__ SecondFor<EPI> second) {
  extern __shared__ uint8_t smem_raw[];
  static_assert(EPI != E_PART || TN == TILE, "partial sums are whole 256 x 256 tiles");
  static_assert(EPI != E_STORE2 || (AMN && BMN), "made for weight gradients");
  constexpr int NS = stages_of(EPI, TN), STAGE = stage_bytes(TN), BROWS = TN / 2;
  constexpr int HALVES = halves_of(EPI, TN);
  using Smem = GemmSmemFor<EPI, TN>;
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    prefetch_map(&amap);
    prefetch_map(&bmap);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.acc_full[a], 1);
      mbar_init(&sm.acc_empty[a], 4 * HALVES * 2);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(2 * TN));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;
  const int u0 = blockIdx.x >> 1, ustep = gridDim.x >> 1;
  constexpr int NCOLS = EPI == E_SWIGLU ? TN / 2 : TN;  // columns of one tile
  const bool gate_up = EPI == E_SWIGLU || (EPI == E_PART && p.gate_up);
  // E_STORE2: units from `units1` on are the second product's
  const int units1 = EPI == E_STORE2 ? p.m_tiles * p.n_tiles : INT32_MAX;
  auto unit_at = [&](int u, int m_tiles, int k_stages, int kps) {
    if constexpr (EPI == E_STORE2)
      if (u >= units1)
        return unit_of(u - units1, second.m_tiles, second.n_tiles, k_stages, kps);
    return unit_of(u, m_tiles, p.n_tiles, k_stages, kps);
  };
  auto load_b = [&](int s, const Unit& w, int k, const CUtensorMap* bmap) {
    uint8_t* b = sm.ab[s] + OPERAND;
    const uint32_t bar = cluster_addr(&sm.full[s], 0);
    const int brow = gate_up ? w.nt * BROWS : w.nt * TN + rank * BROWS;
    if (gate_up) {  // gate rows in the leader, up rows in its peer
      tma_load_3d_pair(b, bmap, bar, k * GK, brow, rank);
    } else if (BMN) {
      tma_load_2d_pair(b, bmap, bar, brow, k * GK);
      if (BROWS > 64) tma_load_2d_pair(b + OPERAND / 2, bmap, bar, brow + 64, k * GK);
    } else {
      tma_load_2d_pair(b, bmap, bar, k * GK, brow);
    }
  };
  // the first unit's first stages: their slots are free from the start, and
  // what the kernel before writes is not B (the host sets early without dyn, and
  // for the first product)
  int early = 0;
  if (p.early && warp == 0 && lane == 0 && u0 < p.m_tiles * p.n_tiles * p.splits) {
    const Unit w = unit_of(u0, p.m_tiles, p.n_tiles, p.k_stages, p.kps);
    early = min(NS, w.k1 - w.k0);
    for (int i = 0; i < early; ++i) {
      if (leader) mbar_arrive_expect_tx(&sm.full[i], 2 * STAGE);
      load_b(i, w, w.k0 + i, &bmap);
    }
  }
  pdl_wait();
  pdl_trigger();

  int m_tiles = p.m_tiles, k_stages = p.k_stages, kps = p.kps, splits = p.splits;
  if (p.dyn) {
    const int rows = *p.rows;
    if (p.dyn == 1) m_tiles = min(m_tiles, (rows + TILE - 1) / TILE);
    if (p.dyn == 2) {
      k_stages = min(k_stages, (rows + GK - 1) / GK);
      kps = max(1, (k_stages + p.splits - 1) / p.splits);
    }
  }
  if (EPI == E_PART && p.splits_of) {
    splits = *p.splits_of;
    kps = (k_stages + splits - 1) / splits;
  }
  int units = m_tiles * p.n_tiles * splits;
  if constexpr (EPI == E_STORE2) units += second.m_tiles * second.n_tiles;

  if (warp == 0) {
    // ---------------- TMA producer
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = u0; u < units && ok; u += ustep) {
        const Unit w = unit_at(u, m_tiles, k_stages, kps);
        const CUtensorMap *am = &amap, *bm = &bmap;
        if constexpr (EPI == E_STORE2)
          if (u >= units1) {
            am = &second.a;
            bm = &second.b;
          }
        const int arow = w.mt * TILE + rank * CM;
        for (int k = w.k0; k < w.k1; ++k) {
          const bool has_b = early > 0;  // B is on its way already
          if (has_b) {
            --early;
          } else {
            if (!(ok = mbar_wait<true>(&sm.empty[s], ph ^ 1, sm, p.dev_err))) break;
            if (leader) mbar_arrive_expect_tx(&sm.full[s], 2 * STAGE);
          }
          const uint32_t bar = cluster_addr(&sm.full[s], 0);
          uint8_t* a = sm.ab[s];
          if (AMN) {
            tma_load_2d_pair(a, am, bar, arow, k * GK);
            tma_load_2d_pair(a + OPERAND / 2, am, bar, arow + 64, k * GK);
          } else {
            tma_load_2d_pair(a, am, bar, k * GK, arow);
          }
          if (!has_b) load_b(s, w, k, bm);
          ++issued;
          if (++s == NS) { s = 0; ph ^= 1; }
        }
      }
      // every copy that this pair requested has landed before it may leave
      // (bounded, and not cut short by an abort)
      if (leader) {
        for (int i = 0; i < min(issued, NS); ++i) {
          if (--s < 0) { s = NS - 1; ph ^= 1; }
          for (uint32_t n = 0; n < kWaitLimit && !mbar_try_wait_suspend_cl(&sm.full[s], ph); ++n) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = gemm_idesc<T, AMN, BMN, TN>();
      const uint64_t ad0 = operand_desc<AMN>(smem_u32(sm.ab[0]));
      const uint64_t bd0 = operand_desc<BMN>(smem_u32(sm.ab[0]) + OPERAND);
      int s = 0, lt = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = u0; u < units && ok; u += ustep, ++lt) {
        const Unit w = unit_at(u, m_tiles, k_stages, kps);
        const int acc = lt & 1;
        if (!(ok = mbar_poll(&sm.acc_empty[acc], ((lt >> 1) & 1) ^ 1, sm, p.dev_err))) break;
        tc_fence_after();
        const uint32_t dcol = tmem_base + acc * TN;
        for (int k = w.k0; k < w.k1; ++k) {
          if (!(ok = mbar_poll(&sm.full[s], ph, sm, p.dev_err))) break;
          tc_fence_after();
          const uint64_t ad = ad0 + (uint64_t)((s * STAGE) >> 4);
          const uint64_t bd = bd0 + (uint64_t)((s * STAGE) >> 4);
#pragma unroll
          for (int kk = 0; kk < GK / 16; ++kk)
            mma_ss_pair(dcol, ad + kk * kstep_units<AMN>(), bd + kk * kstep_units<BMN>(), idesc,
                        (k != w.k0 || kk != 0) ? 1u : 0u);
          mma_commit_pair(&sm.empty[s]);
          if (++s == NS) { s = 0; ph ^= 1; }
        }
        if (ok) mma_commit_pair(&sm.acc_full[acc]);
      }
      // every MMA issued here is done with both CTAs' memory before either leaves
      mma_commit_pair_local(&sm.drain);
      for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait_suspend_cl(&sm.drain, 0); ++i) {
      }
    }
  } else if (warp >= EPI_W0 && warp < EPI_W0 + 4 * HALVES) {
    // ---------------- epilogue: TMEM lanes 32 q .., columns CW hc .. of the tile
    constexpr int CW = NCOLS / HALVES;
    const int ew = warp - EPI_W0, q = warp & 3, hc = ew >> 2;
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    uint8_t* stg = sm.stg[ew];
    int lt = 0;
    bool ovf = false;
    const float scale = (EPI == E_STORE && p.scale) ? *p.scale : 1.0f;
    // 16 bytes (8 columns) of this lane's row into chunk c of the staging block
    uint8_t* stg_now = stg;
    auto stage16 = [&](int c, uint4 v) {
      *reinterpret_cast<uint4*>(stg_now + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
    };
    auto stage32 = [&](int c, const uint32_t (&v)[32]) {  // 32 columns from chunk c on
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 o;
        o.x = pack2<T>(__uint_as_float(v[8 * j]), __uint_as_float(v[8 * j + 1]));
        o.y = pack2<T>(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3]));
        o.z = pack2<T>(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5]));
        o.w = pack2<T>(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7]));
        stage16(c + j, o);
      }
    };
    // the warp's last store has left the staging block
    auto stage_free = [&]() {
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
    };
    // E_SWIGLU_BWD: gate and up of the warp's 32 rows x 32 columns, four lanes
    // a row (a lane per row would touch four times the lines per load): 16 bytes
    // of rows lane / 4 + 8 i
    uint4 gu_next[2][4];
    auto load_gu = [&](int row0, int col) {
      const int r0 = row0 + (lane >> 2), c = col + 8 * (lane & 3);
      const T* gp = reinterpret_cast<const T*>(p.gu) + (size_t)r0 * (2 * (size_t)p.N) + c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = r0 + 8 * i < p.M && c < p.N;  // N is a multiple of 8
        const uint4* g = reinterpret_cast<const uint4*>(gp + (size_t)(16 * i) * p.N);
        const uint4* u = reinterpret_cast<const uint4*>(gp + (size_t)(16 * i + 1) * p.N);
        gu_next[0][i] = in ? ld_stream_u4(g) : make_uint4(0, 0, 0, 0);
        gu_next[1][i] = in ? ld_stream_u4(u) : make_uint4(0, 0, 0, 0);
      }
    };
    // chunk c (16 bytes) of row r in a 64-byte-swizzled block
    auto at64 = [](int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); };
    for (int u = u0; u < units; u += ustep, ++lt) {
      const Unit w = unit_at(u, m_tiles, k_stages, kps);
      const int acc = lt & 1;
      const int row = w.mt * TILE + rank * CM + 32 * q + lane;  // this lane's row of D
      const int row_w = row - lane;                             // the warp's first
      const bool none = w.k0 >= w.k1;  // nothing to sum: the tensor memory holds old values
      if constexpr (EPI == E_SWIGLU_BWD) load_gu(row_w, w.nt * TN + hc * CW);  // under the MMAs
      if (!__all_sync(0xffffffffu,
                      mbar_wait<true>(&sm.acc_full[acc], (lt >> 1) & 1, sm, p.dev_err)))
        break;
      tc_fence_after();
      const uint32_t tacc = tmem_base + lane_addr + acc * TN;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (leader) mbar_arrive(&sm.acc_empty[acc]);
          else mbar_arrive_remote(cluster_addr(&sm.acc_empty[acc], 0));
        }
      };
      auto load32 = [&](int col, uint32_t (&v)[32]) {
        tmem_ld32(tacc + col, v);
        if (none) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
      };

      if constexpr (EPI == E_PART) {
        const int tile = w.mt * p.n_tiles + w.nt;
        float* dst = p.part +
                     ((size_t)w.split * m_tiles * p.n_tiles + tile) * (size_t)TILE_FLOATS +
                     (rank * CM + 32 * q + lane);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int col = hc * CM + 32 * c;
          uint32_t v[32];
          load32(col, v);
          if (c == 3) release();
          float* d = dst + (size_t)col * TILE;
          if (p.accumulate) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              v[i] = __float_as_uint(__uint_as_float(v[i]) + d[(size_t)i * TILE]);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) d[(size_t)i * TILE] = __uint_as_float(v[i]);
        }
      } else if constexpr (EPI == E_STATS) {
        // running maximum m and sum s of exp(l - m) over this warp's columns
        const int tgt = p.targets[row] - w.nt * TN - hc * CW;
        // (the target's sum is given: see linear_ce.cu)
        const float tl = p.target_sum[row];
        float m = -INFINITY, s = 0.0f;
#pragma unroll 1
        for (int c = 0; c < CW / 32; ++c) {
          uint32_t v[32];
          load32(hc * CW + 32 * c, v);
          if (c == CW / 32 - 1) release();
          const int left = p.N - (w.nt * TN + hc * CW + 32 * c);  // real columns here
          if (left <= 0) continue;
          if (left < 32) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i >= left) v[i] = 0xff800000u;  // -inf
          }
          if ((unsigned)(tgt - 32 * c) < 32u) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i == tgt - 32 * c) v[i] = __float_as_uint(tl);
          }
          float cm = __uint_as_float(v[0]);
#pragma unroll
          for (int i = 1; i < 32; ++i) cm = fmaxf(cm, __uint_as_float(v[i]));
          const float mn = fmaxf(m, cm);
          // differences first: a product with log2(e) rounds by 2^-24 of its own
          // size, which for logits of hundreds is too much for the exponent
          float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            s0 += exp2_approx((__uint_as_float(v[i]) - mn) * kLog2e);
            s1 += exp2_approx((__uint_as_float(v[i + 1]) - mn) * kLog2e);
            s2 += exp2_approx((__uint_as_float(v[i + 2]) - mn) * kLog2e);
            s3 += exp2_approx((__uint_as_float(v[i + 3]) - mn) * kLog2e);
          }
          s = s * exp2_approx((m - mn) * kLog2e) + ((s0 + s1) + (s2 + s3));
          m = mn;
        }
        p.stats[(size_t)(HALVES * w.nt + hc) * p.rows_pad + row] = make_float2(m, s);
      } else if constexpr (EPI == E_STORE || EPI == E_STORE2 || EPI == E_DLOGITS) {
        int cols = p.N, rows_end = EPI == E_DLOGITS ? p.rows_pad : p.M;
        const CUtensorMap* dm = &dmap0;
        if constexpr (EPI == E_STORE2)
          if (u >= units1) {
            cols = second.N;
            rows_end = second.M;
            dm = &second.d;
          }
        // p = exp(l - lse) by one FMA on l; what the product lse * log2(e) rounds
        // off is common to the row and goes into its factor rp
        float nlse = 0.f, rp = 0.f, pt = 0.f;
        int tgt = -1;
        if (EPI == E_DLOGITS) {
          const float lse = p.lse[row], rs = p.row_scale[row];
          nlse = -lse * kLog2e;
          rp = rs * exp2_approx(-fmaf(lse, kLog2e, nlse));
          pt = (exp2_approx((p.target_sum[row] - lse) * kLog2e) - 1.0f) * rs;
          tgt = p.targets[row] - p.col0 - w.nt * TN - hc * CW;
        }
#pragma unroll 1
        for (int blk = 0; blk < CW / 64; ++blk) {
          // the store before last has left this block; the last one reads the other
          static_assert(staging_alternates(CW / 64), "a store would be staged over the last one");
          stg_now = stg + staging_block(lt, blk, CW / 64) * STG;
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
          uint32_t w64[2][32];
          tmem_ld64(tacc + hc * CW + 64 * blk, w64[0], w64[1]);
          if (blk == CW / 64 - 1) release();
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const int c = 64 * blk + 32 * h2;  // within this warp's columns
            uint32_t(&v)[32] = w64[h2];
            if (none) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0u;
            }
            if (EPI == E_DLOGITS) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                v[i] = __float_as_uint(exp2_approx(fmaf(__uint_as_float(v[i]), kLog2e, nlse)));
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * rp);
              if ((unsigned)(tgt - c) < 32u) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (i == tgt - c) v[i] = __float_as_uint(pt);
              }
            } else {
              if (p.scale) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  v[i] = __float_as_uint(__uint_as_float(v[i]) * scale);
              }
              if (p.residual && row < p.M) {
                const int col = w.nt * TN + hc * CW + c;
                const float* r = p.residual + (size_t)row * p.N + col;
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                  if (col + i < p.N) {  // N is a multiple of 8
                    const float4 x = *reinterpret_cast<const float4*>(r + i);
                    v[i] = __float_as_uint(__uint_as_float(v[i]) + x.x);
                    v[i + 1] = __float_as_uint(__uint_as_float(v[i + 1]) + x.y);
                    v[i + 2] = __float_as_uint(__uint_as_float(v[i + 2]) + x.z);
                    v[i + 3] = __float_as_uint(__uint_as_float(v[i + 3]) + x.w);
                  }
              }
#pragma unroll
              for (int i = 0; i < 32; ++i) ovf |= overflows_out<T>(__uint_as_float(v[i]));
            }
            stage32(4 * h2, v);
          }
          fence_proxy_async();
          __syncwarp();
          const int col0 = w.nt * TN + hc * CW + 64 * blk;
          if (lane == 0) {
            if (row_w < rows_end && col0 < cols) tma_store_2d(dm, stg_now, col0, row_w);
            bulk_commit();  // a group per turn, stored or not: the wait above counts them
          }
        }
      } else if constexpr (EPI == E_SWIGLU) {
        // this warp's 64 gate columns and the same 64 up columns: h, then, from
        // the tensor memory again, gate and up
        const int c0 = CW * hc, col0 = w.nt * NCOLS + c0;
        stage_free();
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t vg[32], vu[32];
          load32(c0 + 32 * h2, vg);
          load32(TN / 2 + c0 + 32 * h2, vu);
          if (h2 == 1 && !p.save) release();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float g = __uint_as_float(vg[i]), u = __uint_as_float(vu[i]);
            const float h = g * sigmoid_fast(g) * u;
            ovf |= overflows_out<T>(h);
            vg[i] = __float_as_uint(h);
          }
          stage32(4 * h2, vg);
        }
        fence_proxy_async();
        __syncwarp();
        const bool in = row_w < p.M && col0 < p.N;
        if (lane == 0 && in) {
          tma_store_2d(&dmap0, stg, col0, row_w);
          bulk_commit();
        }
        if (p.save) {
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            stage_free();
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              uint32_t v[32];
              load32(part * (TN / 2) + c0 + 32 * h2, v);
              if (part == 1 && h2 == 1) release();
#pragma unroll
              for (int i = 0; i < 32; ++i) ovf |= overflows_out<T>(__uint_as_float(v[i]));
              stage32(4 * h2, v);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && in) {
              tma_store_3d(&dmap1, stg, col0, part, row_w);
              bulk_commit();
            }
          }
        }
      } else {
        // E_SWIGLU_BWD: columns of dh, 32 at a time; the next 32 columns of gu
        // are on their way meanwhile.  Staging: h, gate, up, each 32 rows of 64
        // bytes (64-byte swizzle); the gradients take gate's and up's places
#pragma unroll 1
        for (int c = 0; c < CW; c += 32) {
          const int col0 = w.nt * TN + hc * CW + c;
          stage_free();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = at64((lane >> 2) + 8 * i, lane & 3);
            *reinterpret_cast<uint4*>(stg + STG / 2 + at) = gu_next[0][i];
            *reinterpret_cast<uint4*>(stg + STG + at) = gu_next[1][i];
          }
          if (c + 32 < CW) load_gu(row_w, col0 + 32);
          __syncwarp();
          uint32_t v[32];
          load32(hc * CW + c, v);
          if (c + 32 == CW) release();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint8_t* d = stg + at64(lane, j);
            const uint4 gv = *reinterpret_cast<const uint4*>(d + STG / 2);
            const uint4 uv = *reinterpret_cast<const uint4*>(d + STG);
            const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
            const uint32_t uw[4] = {uv.x, uv.y, uv.z, uv.w};
            uint32_t ho[4], go[4], uo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 g2 = unpack2<T>(gw[i]), u2 = unpack2<T>(uw[i]);
              const SwigluGrad a = swiglu_grad(__uint_as_float(v[8 * j + 2 * i]), g2.x, u2.x);
              const SwigluGrad b = swiglu_grad(__uint_as_float(v[8 * j + 2 * i + 1]), g2.y, u2.y);
              ovf |= overflows_out<T>(a.du) | overflows_out<T>(a.dg);
              ovf |= overflows_out<T>(b.du) | overflows_out<T>(b.dg);
              if (p.save) {
                ovf |= overflows_out<T>(a.h) | overflows_out<T>(b.h);
                ho[i] = pack2<T>(a.h, b.h);
              }
              go[i] = pack2<T>(a.dg, b.dg);
              uo[i] = pack2<T>(a.du, b.du);
            }
            if (p.save) *reinterpret_cast<uint4*>(d) = make_uint4(ho[0], ho[1], ho[2], ho[3]);
            *reinterpret_cast<uint4*>(d + STG / 2) = make_uint4(go[0], go[1], go[2], go[3]);
            *reinterpret_cast<uint4*>(d + STG) = make_uint4(uo[0], uo[1], uo[2], uo[3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0 && row_w < p.M && col0 < p.N) {
            if (p.save) tma_store_2d(&dmap0, stg, col0, row_w);
            tma_store_3d(&dmap1, stg + STG / 2, col0, 0, row_w);
            tma_store_3d(&dmap1, stg + STG, col0, 1, row_w);
            bulk_commit();
          }
        }
      }
    }
    // the stores have read the shared memory; the kernel's end waits for their writes
    if (stg_of(EPI) > 0 && lane == 0) bulk_wait_read<0>();
    __syncwarp();
    // the loop exits are warp-uniform, so every lane takes part
    if (__any_sync(0xffffffffu, ovf) && lane == 0) set_dev_err(p.dev_err, MOE_DEVERR_RANGE);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(2 * TN));
  }
}

// ---------------------------------------------------------------- host side

// Tensor map of a row-major 16-bit matrix [rows, cols] with `ld` elements per
// row; box of 64 columns x box_rows, 128-byte swizzle (or 32 and 64 bytes).
template <typename T>
inline bool map_2d(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld,
                   int box_rows, int box_cols = 64) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return encode_tiled(
             m,
             std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             2, const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <typename T>
inline bool map_3d(CUtensorMap* m, const void* p, const int64_t (&d)[3], const int64_t (&ld)[2],
                   const int (&b)[3]) {
  const cuuint64_t dims[3] = {(cuuint64_t)d[0], (cuuint64_t)d[1], (cuuint64_t)d[2]};
  const cuuint64_t strides[2] = {(cuuint64_t)ld[0] * 2, (cuuint64_t)ld[1] * 2};
  const cuuint32_t box[3] = {(cuuint32_t)b[0], (cuuint32_t)b[1], (cuuint32_t)b[2]},
                   es[3] = {1, 1, 1};
  return encode_tiled(
             m,
             std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             3, const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             b[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand of the GEMM: rows (m or n) x k, either way round.
struct Operand {
  const void* p;
  int64_t rows, k, ld;  // ld: elements between consecutive lines of memory
};
template <typename T, bool MN>
inline bool operand_map(CUtensorMap* m, const Operand& o, int box_rows) {
  return MN ? map_2d<T>(m, o.p, o.k, o.rows, o.ld, GK)
            : map_2d<T>(m, o.p, o.rows, o.k, o.ld, box_rows);
}

// Pairs of CTAs that fit on the device at once (one CTA per SM).
inline int max_pairs(const void* kern, size_t smem) {
  static std::mutex mu;
  static std::unordered_map<uint64_t, int> cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const uint64_t key = (reinterpret_cast<uint64_t>(kern) << 6) ^ (uint64_t)dev;
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) return it->second;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * std::max(1, device_sm_count() / 2));
  cfg.blockDim = dim3(GEMM_THREADS);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = std::max(1, device_sm_count() / 2);
  }
  std::lock_guard<std::mutex> lock(mu);
  cache[key] = n;
  return n;
}

template <typename T, bool AMN, bool BMN, int EPI, int TN>
cudaError_t launch_gemm_maps(const CUtensorMap& am, const CUtensorMap& bm, const CUtensorMap& d0,
                             const CUtensorMap& d1, const GemmArgs& p, cudaStream_t s,
                             const SecondFor<EPI>& second = {}) {
  auto kern = dense_gemm_kernel<T, AMN, BMN, EPI, TN>;
  const void* kp = reinterpret_cast<const void*>(kern);
  const size_t smem = sizeof(GemmSmemFor<EPI, TN>) + 1024;
  cudaError_t err = set_max_dynamic_smem_once(kp, (int)smem);
  if (err != cudaSuccess) return err;
  int64_t units = (int64_t)p.m_tiles * p.n_tiles * p.splits;
  if constexpr (EPI == E_STORE2) units += (int64_t)second.m_tiles * second.n_tiles;
  if (units > INT32_MAX / 2) return cudaErrorInvalidValue;
  const int pairs = (int)std::max<int64_t>(1, std::min<int64_t>(max_pairs(kp, smem), units));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(GEMM_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, am, bm, d0, d1, p, second);
}

// The GEMM on two plain operands; d0 / d1 are the epilogue's output maps.
template <typename T, bool AMN, bool BMN, int EPI, int TN>
cudaError_t launch_gemm(const Operand& a, const Operand& b, const CUtensorMap& d0,
                        const CUtensorMap& d1, const GemmArgs& p, cudaStream_t s) {
  CUtensorMap am, bm;
  if (!operand_map<T, AMN>(&am, a, CM) || !operand_map<T, BMN>(&bm, b, TN / 2))
    return cudaErrorInvalidValue;
  return launch_gemm_maps<T, AMN, BMN, EPI, TN>(am, bm, d0, d1, p, s);
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
inline size_t align1k(size_t b) { return (b + 1023) & ~(size_t)1023; }

// Pairs of CTAs of the current device (two SMs each), as the plans count them.
inline int device_pairs() { return std::max(1, device_sm_count() / 2); }

// Tile width and k splits of one product.
struct Plan {
  int tn, splits;
};
// Modelled time of a product of `rows` x `cols` over `k_stages` stages, in
// microseconds.  A stage costs an SM's way from L2, about 100 GB/s: 0.32 us for
// the 32 KB of a 256-column tile, 0.25 us for the 24 KB of 128 columns; or, where
// few row tiles share a column tile, its operands' way from memory at this
// pair's share of 6.4 TB/s.  A unit costs about 2 us more to fill and `epilogue`
// us per column to drain, which runs under the next unit's stages.  Splits cost
// the joining launch (4 us) and their partial sums' way through L2.
inline Plan plan_product(int64_t rows, int64_t cols, int k_stages, int most_tiles,
                         double epilogue = 0.008) {
  const int pairs = device_pairs(), mt = ceil_div(rows, TILE);
  Plan best = {TILE, 1};
  double best_cost = 1e30;
  for (int tn = TILE; tn >= 128; tn /= 2) {
    const int tiles = mt * ceil_div(cols, tn);
    const double l2 = tn == 256 ? 0.32 : 0.25;
    const double bytes = 128.0 * (std::min<int64_t>(rows, TILE) + tn) / std::min(mt, 4);
    const double stage = std::max(l2, bytes / (6.4e6 / pairs));
    for (int sp = 1; sp <= 16 && sp <= k_stages; ++sp) {
      if (sp > 1 && (tn != TILE || tiles * sp > most_tiles)) break;
      const int kps = ceil_div(k_stages, sp);
      if (ceil_div(k_stages, kps) != sp) continue;  // an empty last split
      const int rounds = ceil_div((int64_t)tiles * sp, pairs);
      const double drain = (sp > 1 ? 0.008 : epilogue) * tn;
      double cost = rounds * kps * stage + 2.0 + drain;
      cost += (rounds - 1) * std::max(0.0, drain - kps * stage);
      // the joining launch, longer where it does a long epilogue's work
      if (sp > 1) cost += 4.0 + 0.015 * tiles * sp + 150.0 * (epilogue - 0.008);
      if (cost < best_cost) {
        best_cost = cost;
        best = {tn, sp};
      }
    }
  }
  return best;
}

// ---------------------------------------------------------------- joining the splits

enum Finish {
  F_PLAIN,       // out = 16-bit (sum * *scale + residual)
  F_SWIGLU,      // partial columns gate | up: out = h, out1 = gate | up (if given)
  F_SWIGLU_BWD,  // sums are dh: out = h, out1 = dgate | dup, from gu
};
struct FinishArgs {
  const float* part;  // [split][tile][256 columns][256 rows]
  int splits, n_tiles;
  const int* splits_of;  // device word with the splits, or null
  size_t split_stride;  // floats; or, with `rows` (device), that of so many rows' tiles
  const int* rows;
  int M, N;             // rows and columns of out
  const float* residual;
  const float* scale;
  const int* row_of;    // F_PLAIN: out row -> row of the sums, -1 for a zero row; or null
  const void* gu;
  void* out;            // F_SWIGLU_BWD: h, or null
  void* out1;
  int32_t* dev_err;
};

// One block joins 32 rows x 64 columns.  Groups of eight warps take every
// G-th split each, all their loads in flight at once, and the groups' sums are
// added in order (so the result does not depend on timing), turned from
// [column][row] to rows through shared memory, and finished.  Bound by the
// partial sums' way out of L2.
template <int FIN>
constexpr int finish_groups() {
  return FIN == F_SWIGLU ? 2 : 4;
}
template <typename T, int FIN>
__global__ void __launch_bounds__(256 * finish_groups<FIN>()) finish_kernel(FinishArgs p) {
  constexpr int G = finish_groups<FIN>();
  __shared__ float t0[G][64][33];
  __shared__ float t1[FIN == F_SWIGLU ? G : 1][FIN == F_SWIGLU ? 64 : 1][33];
  pdl_wait();
  pdl_trigger();
  const int warp = (threadIdx.x >> 5) & 7, grp = threadIdx.x >> 8, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x * 64, row0 = blockIdx.y * 32;
  {
    const int row = row0 + lane;
    int cr = row < p.M ? row : -1;
    const int splits = p.splits_of ? *p.splits_of : p.splits;
    if (p.row_of && cr >= 0) cr = p.row_of[row];
    const int nt = FIN == F_SWIGLU ? c0 / (TILE / 2) : c0 / TILE;
    const int col = FIN == F_SWIGLU ? c0 % (TILE / 2) : c0 % TILE;
    const float* src = p.part + ((size_t)(cr >> 8) * p.n_tiles + nt) * (size_t)TILE_FLOATS +
                       (size_t)(col + warp) * TILE + (cr & 255);
    float a[8] = {}, b[8] = {};
    if (cr >= 0) {
      size_t stride = p.split_stride;
      if (p.rows) stride = (size_t)((*p.rows + TILE - 1) / TILE) * p.n_tiles * TILE_FLOATS;
      src += (size_t)grp * stride;
#pragma unroll 4
      for (int sp = grp; sp < splits; sp += G, src += G * stride) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] += src[(size_t)(8 * i) * TILE];
          if (FIN == F_SWIGLU) b[i] += src[(size_t)(8 * i + TILE / 2) * TILE];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t0[grp][warp + 8 * i][lane] = a[i];
      if (FIN == F_SWIGLU) t1[grp][warp + 8 * i][lane] = b[i];
    }
  }
  __syncthreads();
  if (threadIdx.x >= 256) return;
  const int r = threadIdx.x >> 3, cj = (threadIdx.x & 7) * 8;
  const int row = row0 + r, col = c0 + cj;
  if (row >= p.M || col >= p.N) return;  // N is a multiple of 8
  float v[8], w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] = t0[0][cj + e][r];
    w[e] = FIN == F_SWIGLU ? t1[0][cj + e][r] : 0.0f;
#pragma unroll
    for (int g = 1; g < G; ++g) {
      v[e] += t0[g][cj + e][r];
      if (FIN == F_SWIGLU) w[e] += t1[g][cj + e][r];
    }
  }
  bool ovf = false;
  auto put = [&](void* base, size_t at, const float (&x)[8]) {
    uint4 o;
    o.x = pack2<T>(x[0], x[1]);
    o.y = pack2<T>(x[2], x[3]);
    o.z = pack2<T>(x[4], x[5]);
    o.w = pack2<T>(x[6], x[7]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ovf |= overflows_out<T>(x[e]);
    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(base) + at) = o;
  };
  const size_t at = (size_t)row * p.N + col;
  const size_t at2 = (size_t)row * (2 * (size_t)p.N) + col;  // in a gate | up row
  if (FIN == F_PLAIN) {
    if (p.scale) {
      const float sc = *p.scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= sc;
    }
    if (p.residual) {
      const float4 a = *reinterpret_cast<const float4*>(p.residual + at);
      const float4 b = *reinterpret_cast<const float4*>(p.residual + at + 4);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    }
    put(p.out, at, v);
  } else if (FIN == F_SWIGLU) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = v[e] * sigmoid_fast(v[e]) * w[e];
    put(p.out, at, h);
    if (p.out1) {
      put(p.out1, at2, v);
      put(p.out1, at2 + p.N, w);
    }
  } else {
    const T* gu = reinterpret_cast<const T*>(p.gu);
    float h[8], dg[8], du[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const SwigluGrad r =
          swiglu_grad(v[e], to_f32<T>(gu[at2 + e]), to_f32<T>(gu[at2 + p.N + e]));
      h[e] = r.h;
      dg[e] = r.dg;
      du[e] = r.du;
    }
    if (p.out) put(p.out, at, h);
    put(p.out1, at2, dg);
    put(p.out1, at2 + p.N, du);
  }
  if (ovf) set_dev_err(p.dev_err, MOE_DEVERR_RANGE);
}

template <typename T, int FIN>
cudaError_t launch_finish(const FinishArgs& p, cudaStream_t s) {
  return launch_pdl(finish_kernel<T, FIN>, dim3(ceil_div(p.N, 64), ceil_div(p.M, 32)),
                    dim3(256 * finish_groups<FIN>()), 0, s, p);
}

}  // namespace dense
}  // namespace moe
