// Products of a weight matrix with few tokens (at most 128), on the tensor cores:
//   D[t, n] = sum_k X[t, k] W[n, k],  W either way round,
// the form that the feed-forward block and the vocabulary cross entropy take
// for a decode batch (the block's forward pass of a few tokens and not too large
// weights: ffn_gemv.cuh).  Such a product is bound by reading W once, so the roles
// of the operands are swapped against dense_gemm.cuh: 128 rows of W are the
// MMA's M, the tokens its N (32 to 128 columns), and a stage is 16 KB of W with
// 4 to 16 KB of tokens, where a 256-row tile of mostly absent tokens would
// fill as much shared memory with zeros as with weights.
//
// Work split.  A tile of W is 128 rows.  Where the tiles alone leave SMs idle,
// a cluster of 2, 4 or 8 CTAs shares one tile along k; each CTA leaves its fp32
// sums in its shared memory and joins its share of the tokens from all CTAs of
// the cluster through distributed shared memory, in rank order, so the result
// does not depend on timing and nothing goes through global memory or a second
// launch.  Where even clusters of 8 leave most SMs idle (a short row of W, a long
// k), several clusters take a slice of k each and leave fp32 sums that a second
// launch adds in slice order.  Persistent: a cluster walks tiles, and the tensor
// memory holds two accumulators, so that loads and MMAs of the next tile run
// under the join.
//
// Measured: 201 MB of weights at 32 tokens (4096 x 8192, both products) in 45 us,
// 4.5 TB/s over the whole call (a copy: 6.46).  The two kernels alone, caches cold,
// take 30 us for 134 MB and 20 us for 67 MB: a fixed part of about 10 us each (the
// start, the way to the first operands, the last tile's join, the end) beside
// the stream, of which the chained launch hides some.  A CTA takes all of an SM's
// shared memory, so the next launch's CTAs are set up only where this one's have
// left.
//
// Warp roles (384 threads): warp 0 loads (TMA), warp 1 issues the MMAs and owns
// the tensor memory, warps 4-11 move sums to shared memory (two per TMEM lane
// quarter) and join.  Kernels that follow another of the same call (early) load
// the first weights before they wait for it: nothing in the call writes W.
// Every wait is bounded as in dense_gemm.cuh.
#pragma once

#include "dense_gemm.cuh"

namespace moe {
namespace dense {

constexpr int kSkinnyRows = 128;  // tokens at most
constexpr int kSkinnyStages = 10; // at most

enum SkinnyEpilogue {
  S_STORE,       // out[row_of[t] or t] = 16-bit (sum * *scale + residual)
  S_SWIGLU,      // tile = 64 gate rows, 64 up rows: out = h, out1 = gate | up (if given)
  S_SWIGLU_BWD,  // sums are dh: out = h (if given), out1 = dgate | dup, from gu
  S_STATS,       // per token: loss and lse of the softmax over the columns
  S_DLOGITS,     // out = (exp(sum - lse) - [column is the target]) * row scale
};

struct SkinnyArgs {
  int n;         // tokens, rounded up to 32
  int M;         // tokens
  const int* live;  // device: tokens that count (<= M), or null: M
  int rows;      // columns of the result (S_SWIGLU: of h)
  int tiles, k_stages, stages, early;
  int slices;    // of k, over clusters; S_STORE only
  float* part;   // slices > 1: [slice][M][rows] sums
  const float* residual;
  const float* scale;
  const int* row_of;
  const void* gu;
  void* out;
  void* out1;
  int ld;        // S_DLOGITS: elements per row of out
  // S_STATS: a cluster keeps the running maximum and sum of its tiles and leaves
  // them in stats [M][clusters]; per subset of tokens (that of one warp in every
  // cluster) the last cluster to arrive adds them in order.  arrived: a zeroed
  // word per subset
  float2* stats;
  int* arrived;
  float* loss;
  float* lse_out;
  const float* target_sum;
  const int* targets;
  const float* lse;
  const float* row_scale;
  int32_t* dev_err;
};

struct SkinnyBars {
  uint64_t full[kSkinnyStages], empty[kSkinnyStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t ready, taken;  // the sums of all CTAs stand / have been read by all
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

__host__ __device__ constexpr int skinny_stage(int n) { return CM * GK * 2 + n * GK * 2; }
__host__ __device__ constexpr int skinny_sums(int n) { return n * CM * 4; }
constexpr int kSkinnySmem = 227 * 1024;
inline int skinny_stages(int n) {
  const int room = kSkinnySmem - 1024 - (int)sizeof(SkinnyBars) - skinny_sums(n);
  return std::min(kSkinnyStages, room / skinny_stage(n));
}

__device__ __forceinline__ void mma_ss_one(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ float4 lds_cluster4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a));
  return v;
}

// S_STATS, one warp: leaves its tokens' maximum and sum (lane i's token's m, s);
// the last cluster's warp of this subset joins all clusters' and writes.
__device__ __forceinline__ void stats_join(const SkinnyArgs& p, int tokens, int cluster,
                                           int clusters, int rank, int cs, int ew, int lane,
                                           float m, float s, int row_l, float tsum_l) {
  const int t_l = rank + cs * (ew + EPI_NW * lane);
  if (lane < 16 && t_l < tokens) p.stats[(size_t)t_l * clusters + cluster] = make_float2(m, s);
  __threadfence();
  __syncwarp();
  int before = 0;
  if (lane == 0) before = atomicAdd(&p.arrived[rank * EPI_NW + ew], 1);
  if (__shfl_sync(0xffffffffu, before, 0) != clusters - 1) return;
  __threadfence();
  float top_l = 0.0f, sum_l = 1.0f;  // lane i's token's
  constexpr int G = 4, J = 5;        // tokens and, by 32, clusters whose loads are in flight
  for (int i0 = 0; i0 < 16 && rank + cs * (ew + EPI_NW * i0) < tokens; i0 += G) {
    float mg[G], sg[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      mg[g] = -INFINITY;
      sg[g] = 0.0f;
    }
    for (int c0 = lane; c0 < clusters; c0 += 32 * J) {
      float2 o[G][J];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int t = rank + cs * (ew + EPI_NW * (i0 + g));
#pragma unroll
        for (int j = 0; j < J; ++j)
          o[g][j] = t < tokens && c0 + 32 * j < clusters
                        ? __ldcg(&p.stats[(size_t)t * clusters + c0 + 32 * j])
                        : make_float2(-INFINITY, 0.0f);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float mn = mg[g];
#pragma unroll
        for (int j = 0; j < J; ++j) mn = fmaxf(mn, o[g][j].x);
        sg[g] = sg[g] == 0.0f ? 0.0f : sg[g] * exp2_approx((mg[g] - mn) * kLog2e);
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (o[g][j].y != 0.0f) sg[g] += o[g][j].y * exp2_approx((o[g][j].x - mn) * kLog2e);
        mg[g] = mn;
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float top = warp_max(mg[g]);
      const float sum =
          warp_sum(sg[g] == 0.0f ? 0.0f : sg[g] * exp2_approx((mg[g] - top) * kLog2e));
      if (lane == i0 + g) {
        top_l = top;
        sum_l = sum;
      }
    }
  }
  if (lane < 16 && t_l < tokens) {
    const float ls = logf(sum_l);
    p.loss[row_l] = (top_l - tsum_l) + ls;  // lse - target would lose lse's rounding
    p.lse_out[row_l] = top_l + ls;
  }
}

template <typename T, bool AMN, int EPI>
__global__ void __launch_bounds__(GEMM_THREADS, 1) skinny_gemm_kernel(
    const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
    const __grid_constant__ SkinnyArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int NS = p.stages, STAGE = skinny_stage(p.n), N = p.n;
  float* sums = reinterpret_cast<float*>(ring + NS * STAGE);  // [token][128 rows of W]
  SkinnyBars& sm = *reinterpret_cast<SkinnyBars*>(ring + NS * STAGE + skinny_sums(N));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank(), cs = (int)cluster_size();
  const uint32_t tmem_cols = N <= 32 ? 64u : N <= 64 ? 128u : 256u;  // two accumulators

  if (threadIdx.x == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.acc_full[a], 1);
      mbar_init(&sm.acc_empty[a], EPI_NW);
    }
    mbar_init(&sm.ready, EPI_NW * cs);
    mbar_init(&sm.taken, EPI_NW * cs);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sm.tmem_base)),
                 "r"(tmem_cols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = sm.tmem_base;

  // this CTA's stages of every tile, and the tiles of its cluster: a cluster
  // keeps its slice (the grid is a multiple of the slices' clusters)
  const int slice = (blockIdx.x / cs) % p.slices, share = slice * cs + rank;
  const int k0 = (int)((int64_t)p.k_stages * share / (cs * p.slices));
  const int k1 = (int)((int64_t)p.k_stages * (share + 1) / (cs * p.slices));
  const int t0 = blockIdx.x / cs / p.slices, tstep = gridDim.x / cs / p.slices;

  if (warp == 0) {
    // ---------------- TMA producer
    if (lane == 0) {
      auto load_w = [&](int s, int tile, int k) {
        uint8_t* a = ring + s * STAGE;
        mbar_arrive_expect_tx(&sm.full[s], (uint32_t)STAGE);
        if (EPI == S_SWIGLU) {  // 64 gate rows, 64 up rows
          tma_load_3d(a, &wmap, &sm.full[s], k * GK, tile * 64, 0);
          tma_load_3d(a + OPERAND / 2, &wmap, &sm.full[s], k * GK, tile * 64, 1);
        } else if (AMN) {
          tma_load_2d(a, &wmap, &sm.full[s], tile * CM, k * GK);
          tma_load_2d(a + OPERAND / 2, &wmap, &sm.full[s], tile * CM + 64, k * GK);
        } else {
          tma_load_2d(a, &wmap, &sm.full[s], k * GK, tile * CM);
        }
      };
      auto load_x = [&](int s, int k) {
        tma_load_2d(ring + s * STAGE + OPERAND, &xmap, &sm.full[s], k * GK, 0);
      };
      // the first tile's first stages: their slots are free from the start
      const int early = p.early && t0 < p.tiles ? min(NS, k1 - k0) : 0;
      for (int i = 0; i < early; ++i) load_w(i, t0, k0 + i);
      pdl_wait();
      pdl_trigger();
      const bool some = p.live == nullptr || *p.live > 0;
      int s = 0, issued = 0;
      uint32_t ph = 0;
      for (int i = 0; i < early; ++i) {
        load_x(i, k0 + i);
        ++issued;
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      bool ok = true;
      for (int tile = t0; tile < p.tiles && some && ok; tile += tstep) {
        for (int k = k0 + (tile == t0 ? early : 0); k < k1; ++k) {
          if (!(ok = mbar_wait(&sm.empty[s], ph ^ 1, sm, p.dev_err))) break;
          load_w(s, tile, k);
          load_x(s, k);
          ++issued;
          if (++s == NS) { s = 0; ph ^= 1; }
        }
      }
      // every copy that was requested has landed before the CTA may leave
      for (int i = 0; i < min(issued, NS); ++i) {
        if (--s < 0) { s = NS - 1; ph ^= 1; }
        for (uint32_t n = 0; n < kWaitLimit && !mbar_try_wait_suspend(&sm.full[s], ph); ++n) {
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer
    if (lane == 0) {
      pdl_wait();
      const bool some = p.live == nullptr || *p.live > 0;
      const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
      const uint32_t idesc = (1u << 4) | (f << 7) | (f << 10) | ((AMN ? 1u : 0u) << 15) |
                             ((uint32_t)(N >> 3) << 17) | ((uint32_t)(CM >> 4) << 24);
      const uint64_t ad0 = operand_desc<AMN>(smem_u32(ring));
      const uint64_t bd0 = operand_desc<false>(smem_u32(ring) + OPERAND);
      int s = 0, lt = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = t0; tile < p.tiles && some && ok; tile += tstep, ++lt) {
        const int acc = lt & 1;
        if (!(ok = mbar_poll(&sm.acc_empty[acc], ((lt >> 1) & 1) ^ 1, sm, p.dev_err))) break;
        tc_fence_after();
        const uint32_t dcol = tmem_base + acc * N;
        for (int k = k0; k < k1; ++k) {
          if (!(ok = mbar_poll(&sm.full[s], ph, sm, p.dev_err))) break;
          tc_fence_after();
          const uint64_t ad = ad0 + (uint64_t)((s * STAGE) >> 4);
          const uint64_t bd = bd0 + (uint64_t)((s * STAGE) >> 4);
#pragma unroll
          for (int kk = 0; kk < GK / 16; ++kk)
            mma_ss_one(dcol, ad + kk * kstep_units<AMN>(), bd + kk * kstep_units<false>(), idesc,
                       (k != k0 || kk != 0) ? 1u : 0u);
          mma_commit(&sm.empty[s]);
          if (++s == NS) { s = 0; ph ^= 1; }
        }
        if (ok) mma_commit(&sm.acc_full[acc]);
      }
      // every MMA issued here is done with the shared memory before the CTA leaves
      mma_commit(&sm.drain);
      for (uint32_t i = 0; i < kWaitLimit && !mbar_try_wait_suspend(&sm.drain, 0); ++i) {
      }
    }
  } else if (warp >= EPI_W0) {
    // ---------------- sums to shared memory, join, epilogue
    pdl_wait();
    const int tokens = p.live ? min(*p.live, p.M) : p.M;
    // S_DLOGITS also writes the rows behind the last token, as zeros: dW's reduction reads them
    const int joined = EPI == S_DLOGITS ? N : tokens;
    const int ew = warp - EPI_W0, q = warp & 3, hc = ew >> 2;
    const uint32_t lane_addr = (uint32_t)(32 * q) << 16;
    const float scale = (EPI == S_STORE && p.scale) ? *p.scale : 1.0f;
    bool ovf = false;
    int lt = 0;
    uint32_t bases[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) bases[r] = cluster_addr(sums, r < cs ? r : rank);
    // this warp's tokens are t = rank + cs * (ew + 8 i), i < 16; lane i keeps what
    // the epilogue needs to know of the i-th
    const int t_l = rank + cs * (ew + EPI_NW * lane);
    int tgt_l = -1, row_l = t_l;
    float tsum_l = 0.0f, lse_l = 0.0f, rs_l = 0.0f;
    if (lane < 16 && t_l < joined) {
      if (EPI == S_STATS || EPI == S_DLOGITS) {
        tgt_l = p.targets[t_l];
        tsum_l = p.target_sum[t_l];
      }
      if (EPI == S_DLOGITS) {
        lse_l = p.lse[t_l];
        rs_l = p.row_scale[t_l];
      }
      if ((EPI == S_STORE && p.row_of && p.slices == 1) || (EPI == S_STATS && t_l < tokens))
        row_l = p.row_of[t_l];
    }
    float run_m = -INFINITY, run_s = 0.0f;  // S_STATS: lane i's token's
    bool done = true;
    for (int tile = t0; tile < p.tiles && tokens > 0; tile += tstep, ++lt) {
      const int acc = lt & 1;
      if constexpr (EPI == S_STORE || EPI == S_SWIGLU_BWD) {
        // what the join will read, on its way to L2 under the MMAs
        const int col = tile * CM + 4 * lane;
        if (col < p.rows && (EPI == S_SWIGLU_BWD || (p.residual && p.slices == 1)))
          for (int t = rank + cs * ew; t < tokens; t += cs * EPI_NW) {
            if (EPI == S_STORE) {
              prefetch_l2(p.residual + (size_t)t * p.rows + col);
            } else {
              const T* gu = static_cast<const T*>(p.gu) + (size_t)t * 2 * p.rows + col;
              prefetch_l2(gu);
              prefetch_l2(gu + p.rows);
            }
          }
      }
      done = false;
      if (!__all_sync(0xffffffffu, mbar_wait(&sm.acc_full[acc], (lt >> 1) & 1, sm, p.dev_err)))
        break;
      tc_fence_after();
      // all CTAs have read the tile before
      if (!__all_sync(0xffffffffu, mbar_wait<true>(&sm.taken, (lt & 1) ^ 1, sm, p.dev_err))) break;
      for (int c = hc; 32 * c < joined; c += 2) {
        uint32_t v[32];
        tmem_ld32(tmem_base + lane_addr + acc * N + 32 * c, v);
        float* d = sums + (size_t)(32 * c) * CM + 32 * q + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) d[i * CM] = __uint_as_float(v[i]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_empty[acc]);
      if (cs == 1) {
        if (lane == 0) mbar_arrive(&sm.ready);
      } else if (lane < cs) {
        mbar_arrive_remote(cluster_addr(&sm.ready, lane));
      }
      if (!__all_sync(0xffffffffu, mbar_wait_soon(&sm.ready, lt & 1, sm, p.dev_err))) break;

      // tokens rank + cs * (ew + 8 i) of this tile
      auto sum4 = [&](int t, int row) {  // 4 rows from `row` on
        if (cs == 1) return *reinterpret_cast<const float4*>(sums + t * CM + row);
        const uint32_t at = (uint32_t)(t * CM + row) * 4u;
        float4 b[8];  // all ranks' loads in flight, then the sum in rank order
#pragma unroll
        for (int r = 0; r < 8; ++r)
          b[r] = r < cs ? lds_cluster4(bases[r] + at) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 a = b[0];
#pragma unroll
        for (int r = 1; r < 8; ++r) {
          a.x += b[r].x; a.y += b[r].y; a.z += b[r].z; a.w += b[r].w;
        }
        return a;
      };
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int t = rank + cs * (ew + EPI_NW * i);
        if (t >= joined) break;
        if constexpr (EPI == S_SWIGLU) {
          // lanes 0-15 hold gate columns 4 lane .., lanes 16-31 the same up columns
          const float4 v = sum4(t, 4 * lane);
          const int col = tile * 64 + 4 * (lane & 15);
          const float vs[4] = {v.x, v.y, v.z, v.w};
          float o[4], h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = __shfl_down_sync(0xffffffffu, vs[e], 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[e] = vs[e] * sigmoid_fast(vs[e]) * o[e];
          if (col < p.rows) {  // a multiple of 8
            if (lane < 16) {
              ovf |= overflows_out<T>(h[0]) | overflows_out<T>(h[1]) | overflows_out<T>(h[2]) |
                     overflows_out<T>(h[3]);
              *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (size_t)t * p.rows + col) =
                  make_uint2(pack2<T>(h[0], h[1]), pack2<T>(h[2], h[3]));
            }
            if (p.out1) {
              ovf |= overflows_out<T>(vs[0]) | overflows_out<T>(vs[1]) |
                     overflows_out<T>(vs[2]) | overflows_out<T>(vs[3]);
              *reinterpret_cast<uint2*>(static_cast<T*>(p.out1) + (size_t)t * 2 * p.rows +
                                        (lane < 16 ? 0 : p.rows) + col) =
                  make_uint2(pack2<T>(vs[0], vs[1]), pack2<T>(vs[2], vs[3]));
            }
          }
        } else {
          const int col = tile * CM + 4 * lane;
          const float4 v4 = sum4(t, 4 * lane);
          float v[4] = {v4.x, v4.y, v4.z, v4.w};
          if constexpr (EPI == S_STORE) {
            const int row = __shfl_sync(0xffffffffu, row_l, i);
            if (col < p.rows && p.slices > 1) {
              *reinterpret_cast<float4*>(p.part + ((size_t)slice * p.M + t) * p.rows + col) = v4;
            } else if (col < p.rows) {
              const size_t at = (size_t)row * p.rows + col;
              if (p.scale) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= scale;
              }
              if (p.residual) {
                const float4 r = *reinterpret_cast<const float4*>(p.residual + at);
                v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) ovf |= overflows_out<T>(v[e]);
              *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at) =
                  make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
            }
          } else if constexpr (EPI == S_SWIGLU_BWD) {
            if (col < p.rows) {
              const size_t at = (size_t)t * p.rows + col, at2 = (size_t)t * 2 * p.rows + col;
              const T* gu = static_cast<const T*>(p.gu) + at2;
              const uint2 gw = *reinterpret_cast<const uint2*>(gu);
              const uint2 uw = *reinterpret_cast<const uint2*>(gu + p.rows);
              const float2 ga = unpack2<T>(gw.x), gb = unpack2<T>(gw.y);
              const float2 ua = unpack2<T>(uw.x), ub = unpack2<T>(uw.y);
              const float g[4] = {ga.x, ga.y, gb.x, gb.y}, uu[4] = {ua.x, ua.y, ub.x, ub.y};
              float h[4], dg[4], du[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const SwigluGrad r = swiglu_grad(v[e], g[e], uu[e]);
                h[e] = r.h;
                dg[e] = r.dg;
                du[e] = r.du;
                ovf |= overflows_out<T>(du[e]) | overflows_out<T>(dg[e]);
              }
              T* d = static_cast<T*>(p.out1) + at2;
              if (p.out) {
#pragma unroll
                for (int e = 0; e < 4; ++e) ovf |= overflows_out<T>(h[e]);
                *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at) =
                    make_uint2(pack2<T>(h[0], h[1]), pack2<T>(h[2], h[3]));
              }
              *reinterpret_cast<uint2*>(d) =
                  make_uint2(pack2<T>(dg[0], dg[1]), pack2<T>(dg[2], dg[3]));
              *reinterpret_cast<uint2*>(d + p.rows) =
                  make_uint2(pack2<T>(du[0], du[1]), pack2<T>(du[2], du[3]));
            }
          } else if constexpr (EPI == S_STATS) {
            const int tgt = __shfl_sync(0xffffffffu, tgt_l, i) - col;
            const float tsum = __shfl_sync(0xffffffffu, tsum_l, i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (tgt == e) v[e] = tsum;
              if (col + e >= p.rows) v[e] = -INFINITY;
            }
            const float m = warp_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
            const float s = warp_sum((exp2_approx((v[0] - m) * kLog2e) +
                                      exp2_approx((v[1] - m) * kLog2e)) +
                                     (exp2_approx((v[2] - m) * kLog2e) +
                                      exp2_approx((v[3] - m) * kLog2e)));
            if (lane == i) {
              const float mn = fmaxf(run_m, m);
              run_s =
                  run_s * exp2_approx((run_m - mn) * kLog2e) + s * exp2_approx((m - mn) * kLog2e);
              run_m = mn;
            }
          } else {  // S_DLOGITS
            const float lse = __shfl_sync(0xffffffffu, lse_l, i);
            const float rs = __shfl_sync(0xffffffffu, rs_l, i);
            const float tsum = __shfl_sync(0xffffffffu, tsum_l, i);
            const int tgt = __shfl_sync(0xffffffffu, tgt_l, i) - col;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = exp2_approx((v[e] - lse) * kLog2e);
              if (tgt == e) x = exp2_approx((tsum - lse) * kLog2e) - 1.0f;
              v[e] = x * rs;
            }
            // rows of out are p.ld >= 128 tiles long: the last tile's end is theirs too
            *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (size_t)t * p.ld + col) =
                make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
          }
        }
      }
      done = true;
      if (tile + tstep >= p.tiles) break;  // nobody waits for the last tile's
      __syncwarp();
      if (cs == 1) {
        if (lane == 0) mbar_arrive(&sm.taken);
      } else if (lane < cs) {
        mbar_arrive_remote(cluster_addr(&sm.taken, lane));
      }
    }
    if constexpr (EPI == S_STATS) {
      // (after a wait that ran out, done is false in the whole warp and the error word set)
      if (done && rank + cs * ew < tokens)
        stats_join(p, tokens, t0, tstep, rank, cs, ew, lane, run_m, run_s, row_l, tsum_l);
    }
    __syncwarp();
    if (__any_sync(0xffffffffu, ovf) && lane == 0) set_dev_err(p.dev_err, MOE_DEVERR_RANGE);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nobody leaves while a peer may read its sums or arrive on its barriers
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(tmem_cols));
  }
}

// Clusters of c CTAs that fit on the device at once.
inline int max_clusters(const void* kern, int c) {
  static std::mutex mu;
  static std::unordered_map<uint64_t, int> cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  const uint64_t key =
      (reinterpret_cast<uint64_t>(kern) << 10) ^ (uint64_t)(dev << 4) ^ (uint64_t)c;
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find(key);
    if (it != cache.end()) return it->second;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c * std::max(1, device_sm_count() / c));
  cfg.blockDim = dim3(GEMM_THREADS);
  cfg.dynamicSmemBytes = kSkinnySmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = std::max(1, device_sm_count() / c);
  }
  std::lock_guard<std::mutex> lock(mu);
  cache[key] = n;
  return n;
}

// Adds the slices' sums: a thread takes four columns of a token.
template <typename T>
__global__ void __launch_bounds__(256) skinny_join_kernel(SkinnyArgs p) {
  pdl_wait();
  pdl_trigger();
  const int tokens = p.live ? min(*p.live, p.M) : p.M;
  const int t = blockIdx.y, col = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (t >= tokens || col >= p.rows) return;
  const float* src = p.part + (size_t)t * p.rows + col;
  const size_t step = (size_t)p.M * p.rows;
  float4 a = *reinterpret_cast<const float4*>(src);
#pragma unroll 8
  for (int i = 1; i < p.slices; ++i) {
    const float4 b = *reinterpret_cast<const float4*>(src + i * step);
    a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
  }
  float v[4] = {a.x, a.y, a.z, a.w};
  const size_t at = (size_t)(p.row_of ? p.row_of[t] : t) * p.rows + col;
  if (p.scale) {
    const float scale = *p.scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= scale;
  }
  if (p.residual) {
    const float4 r = *reinterpret_cast<const float4*>(p.residual + at);
    v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
  }
  bool ovf = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) ovf |= overflows_out<T>(v[e]);
  *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at) =
      make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  if (ovf) set_dev_err(p.dev_err, MOE_DEVERR_RANGE);
}

// Slices of k for W of `rows` x `k`: as many clusters of 8 as fill the device,
// where one slice would leave half of it idle for 5 us or more (a CTA reads a
// stage in about 0.3 us) -- the joining launch costs about 4.
inline int skinny_slices(int64_t rows, int64_t k) {
  const int tiles = ceil_div(rows, CM), stages = ceil_div(k, GK);
  const int most = device_sm_count() / (8 * tiles);
  if (most < 2) return 1;
  const int s = std::min(most, stages / 32);  // 4 stages per CTA at least
  return s > 1 && 0.3 * stages / 8 * (1.0 - 1.0 / s) > 5.0 ? s : 1;
}
inline size_t skinny_part_bytes(int M, int64_t rows, int64_t k) {
  const int s = skinny_slices(rows, k);
  return s > 1 ? (size_t)s * M * rows * 4 : 0;
}

inline size_t skinny_stats_bytes(int M, int64_t rows) {
  return (size_t)std::min(ceil_div(rows, CM), device_sm_count()) * M * sizeof(float2);
}

// W: rows x k (S_SWIGLU: [2][rows][k]); X [M, k] with ldx elements per row.
// S_STORE: p.part holds skinny_part_bytes.
template <typename T, bool AMN, int EPI>
cudaError_t launch_skinny(const Operand& w, const void* X, int64_t ldx, int x_rows, SkinnyArgs p,
                          cudaStream_t s) {
  auto kern = skinny_gemm_kernel<T, AMN, EPI>;
  const void* kp = reinterpret_cast<const void*>(kern);
  if (cudaError_t e = set_max_dynamic_smem_once(kp, kSkinnySmem)) return e;
  p.n = (p.M + 31) / 32 * 32;
  p.stages = skinny_stages(p.n);
  p.rows = (int)w.rows;
  p.tiles = ceil_div(w.rows, EPI == S_SWIGLU ? 64 : CM);
  p.k_stages = ceil_div(w.k, GK);
  CUtensorMap wm, xm;
  const bool mapped =
      EPI == S_SWIGLU
          ? map_3d<T>(&wm, w.p, {w.k, w.rows, 2}, {w.ld, w.rows * w.ld}, {GK, 64, 1})
          : operand_map<T, AMN>(&wm, w, CM);
  if (!mapped || !map_2d<T>(&xm, X, x_rows, w.k, ldx, p.n)) return cudaErrorInvalidValue;
  p.slices = EPI == S_STORE ? skinny_slices(w.rows, w.k) : 1;
  int best = p.slices > 1 ? 8 : 1;
  double best_cost = 1e30;
  for (int c = 1; c <= 8 && c <= p.k_stages && p.slices == 1; c *= 2) {
    const int fit = max_clusters(kp, c);
    // rounds of the busiest cluster, each its stages and about `fixed` more
    const double cost = (double)ceil_div(p.tiles, fit) * ((double)ceil_div(p.k_stages, c) + 5.0);
    if (cost < best_cost) {
      best_cost = cost;
      best = c;
    }
  }
  cudaLaunchConfig_t cfg = {};
  // clusters per slice
  const int clusters = std::min(p.tiles, std::max(1, max_clusters(kp, best) / p.slices));
  cfg.gridDim = dim3(best * p.slices * clusters);
  cfg.blockDim = dim3(GEMM_THREADS);
  cfg.dynamicSmemBytes = kSkinnySmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = best;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, wm, xm, p);
  if (e || p.slices == 1) return e;
  return launch_pdl(skinny_join_kernel<T>, dim3(ceil_div(p.rows, 1024), p.M), dim3(256), 0, s, p);
}

}  // namespace dense
}  // namespace moe
