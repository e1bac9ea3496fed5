// The gated feed-forward block for a few tokens (at most 16): both products
// are bound by streaming the weights once, so they run as matrix-vector
// kernels on the warp MMA (m16n8k16, 16 weight rows x 8 tokens), which needs
// no tensor-memory round trip and no second pass over partial sums.
//
// A block owns 16 weight rows (up: 8 gate rows and their 8 up rows, which land
// in the same thread's accumulators; down: 16 output rows) and its eight warps
// take every eighth 64-k chunk of them.  The sum over k does not depend on
// which k sits in which MMA slot, so a thread feeds the 16 consecutive bytes
// that it loads (8 k of its row) to two MMAs as they are and loads the tokens'
// rows in the same pattern: wide loads, no shuffles, no shared memory but for
// the eight warps' sums at the end, which are added in warp order.  Where k is
// long and the blocks are few, a cluster of 2 to 8 blocks shares the rows along
// k and its first block adds the others' sums, in order, through distributed
// shared memory.
#pragma once

#include "dense_gemm.cuh"

namespace moe {
namespace dense {

constexpr int kGemvWarps = 8;
constexpr int kGemvK = 64;      // k of a chunk: a 128-byte line of each of its rows
// Half chunks in flight per warp (UNROLL).  Fewer let more blocks share an SM,
// which streams better; more take a short row in one round of loads.  8 tokens,
// 4 against 2: 2048 x 1024 (13 MB) 7.4 and 8.5 us, 2048 x 4096 (50 MB) 17.3 and
// 14.8 us, 4096 x 4096 (101 MB) 28.6 and 24.4 us.  Two groups of 8 tokens read
// the tokens twice as often; 16 tokens, 4 against 8: 256 x 8192 (13 MB) 11.5 and
// 14.0 us, 2048 x 4096 24 and 19 us.
inline bool gemv_streams(int H, int I) { return (int64_t)6 * H * I > 32 << 20; }
constexpr int kGemvRows = 16;   // tokens at most

// Whether so many tokens take these kernels.  Beyond some size of the weights the
// tensor-core form streams them as fast or faster: 4096 x 8192 (201 MB) in 43 us
// against 53 us for 8 tokens and 65 us for 16; 4096 x 4096 (101 MB) in 28 against
// 24 and 35 us; 2048 x 4096 (50 MB) in 21 against 15 and 19 us.
inline bool use_gemv(int M, int H, int I) {
  const int64_t bytes = (int64_t)6 * H * I;
  return M <= 8 ? bytes <= 128 << 20 : M <= kGemvRows && bytes <= 64 << 20;
}

template <typename T>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  if (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 lds_cluster2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(a)
               : "memory");
  return v;
}

// UP: out = h [M, rows], gu (if given) [M, 2 rows], A = W_gu [2 rows, K].
// Otherwise out [M, rows] (+ residual), A = W_d [rows, K].  NT: groups of 8
// tokens.  K and rows are multiples of 8.  The down form is launched right
// behind the up form, so its weights cannot be anyone's pending output: it
// loads the first of them before it waits for h.  Any input may be what the
// launch before the call has written, so all loads are coherent ones.
template <typename T, int NT, bool UP, int UNROLL>
__global__ void __launch_bounds__(32 * kGemvWarps) ffn_gemv_kernel(
    const T* A, const T* X, int M, int rows, int K, const float* residual, T* __restrict__ out,
    T* __restrict__ gu, int32_t* dev_err) {
  __shared__ float sums[kGemvWarps][NT][32][4];
  __shared__ float2 joined[NT][64];
  const int cs = (int)cluster_size(), rank = (int)cluster_rank();
  const int row_blk = blockIdx.x / cs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (UP) {
    pdl_wait();
    pdl_trigger();
  }
  // this thread's two weight rows (clamped to a real one; the last block of
  // the down form may own 8 rows only) and its tokens' rows
  const int r0 = UP ? row_blk * 8 + g : row_blk * 16 + g;
  const int r1 = UP ? rows + r0 : min(r0 + 8, rows - 1);
  const T* a0p = A + (size_t)r0 * K + 8 * t;
  const T* a1p = A + (size_t)r1 * K + 8 * t;
  const T* xp[NT];
  bool live[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    live[n] = 8 * n + g < M;
    xp[n] = X + (size_t)(live[n] ? 8 * n + g : 0) * K + 8 * t;
  }
  float acc[NT][4] = {};
  const int chunks = (K + kGemvK - 1) / kGemvK;
  const int lo = chunks * rank / cs, hi = chunks * (rank + 1) / cs;  // this block's
  const int kend = min(K, kGemvK * hi);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  bool first = !UP;
  for (int c0 = lo + warp; c0 < hi; c0 += kGemvWarps * UNROLL / 2) {
    uint4 a0[UNROLL], a1[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int k = kGemvK * (c0 + (i >> 1) * kGemvWarps) + 32 * (i & 1);
      const bool in = k + 8 * t < kend;
      a0[i] = in ? ld_stream_u4(a0p + k) : zero;
      a1[i] = in ? ld_stream_u4(a1p + k) : zero;
    }
    if (first) {
      pdl_wait();
      pdl_trigger();
      first = false;
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int k = kGemvK * (c0 + (i >> 1) * kGemvWarps) + 32 * (i & 1);
      if (k >= kend) break;
      const bool in = k + 8 * t < kend;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = in && live[n] ? ld_u4(xp[n] + k) : zero;
        mma_16x8x16<T>(acc[n], a0[i].x, a1[i].x, a0[i].y, a1[i].y, b.x, b.y);
        mma_16x8x16<T>(acc[n], a0[i].z, a1[i].z, a0[i].w, a1[i].w, b.z, b.w);
      }
    }
  }
  if (first) {  // a warp without chunks
    pdl_wait();
    pdl_trigger();
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
    *reinterpret_cast<float4*>(sums[warp][n][lane]) =
        make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  __syncthreads();
  // accumulator e of lane 4 g + t is weight row g (e < 2) or g + 8, token 2 t + (e & 1)
  auto add = [&](int i) {
    const int n = i >> 6, tok_l = (i >> 3) & 7, row = i & 7;
    const int src = 4 * row + (tok_l >> 1), e = tok_l & 1;
    float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kGemvWarps; ++w) {
      v.x += sums[w][n][src][e];
      v.y += sums[w][n][src][2 + e];
    }
    return v;
  };
  if (cs > 1) {
    for (int i = threadIdx.x; i < NT * 64; i += 32 * kGemvWarps) joined[i >> 6][i & 63] = add(i);
    cluster_sync();
  }
  bool ovf = false;
  for (int i = threadIdx.x; i < NT * 64 && rank == 0; i += 32 * kGemvWarps) {
    const int n = i >> 6, tok_l = (i >> 3) & 7, row = i & 7, tok = 8 * n + tok_l;
    if (tok >= M) continue;
    float v0, v1;
    if (cs == 1) {
      const float2 v = add(i);
      v0 = v.x;
      v1 = v.y;
    } else {
      float2 o[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        o[r] = r < cs ? lds_cluster2(cluster_addr(&joined[n][i & 63], r)) : make_float2(0.f, 0.f);
      v0 = v1 = 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        v0 += o[r].x;
        v1 += o[r].y;
      }
    }
    if (UP) {
      const int j = row_blk * 8 + row;
      const float h = v0 * sigmoid_fast(v0) * v1;
      ovf |= overflows_out<T>(h);
      out[(size_t)tok * rows + j] = from_f32<T>(h);
      if (gu) {
        ovf |= overflows_out<T>(v0) | overflows_out<T>(v1);
        gu[(size_t)tok * 2 * rows + j] = from_f32<T>(v0);
        gu[(size_t)tok * 2 * rows + rows + j] = from_f32<T>(v1);
      }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int j = row_blk * 16 + 8 * half + row;
        if (j >= rows) continue;
        float v = half ? v1 : v0;
        if (residual) v += residual[(size_t)tok * rows + j];
        ovf |= overflows_out<T>(v);
        out[(size_t)tok * rows + j] = from_f32<T>(v);
      }
    }
  }
  if (cs > 1) cluster_sync();  // the first block has read the others' sums
  if (ovf) set_dev_err(dev_err, MOE_DEVERR_RANGE);
}

// Blocks per row block: until one round of loads or four blocks per SM is reached.  464 x 7712, 5
// tokens: one block a row block took 15 us.
inline int gemv_cluster(int blocks, int K, int unroll) {
  int c = 1;
  while (c < 8 && K > c * 32 * kGemvWarps * unroll && 2 * c * blocks <= 4 * device_sm_count())
    c *= 2;
  return c;
}

template <typename T, int NT, bool UP, int UNROLL>
cudaError_t launch_gemv(const void* A, const void* X, int M, int rows, int K,
                        const float* residual, void* out, void* gu, int32_t* dev_err,
                        cudaStream_t s) {
  const int blocks = UP ? rows / 8 : ceil_div(rows, 16),
            c = gemv_cluster(blocks, K, UNROLL);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks * c);
  cfg.blockDim = dim3(32 * kGemvWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = c > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, ffn_gemv_kernel<T, NT, UP, UNROLL>, static_cast<const T*>(A),
                            static_cast<const T*>(X), M, rows, K, residual, static_cast<T*>(out),
                            static_cast<T*>(gu), dev_err);
}

template <typename T, int NT, int UNROLL>
cudaError_t launch_both(const void* X, const void* W_gu, const void* W_d, int M, int H, int I,
                        const float* residual, void* Y, void* gu, void* h, int32_t* dev_err,
                        cudaStream_t s) {
  if (cudaError_t e =
          launch_gemv<T, NT, true, UNROLL>(W_gu, X, M, I, H, nullptr, h, gu, dev_err, s))
    return e;
  return launch_gemv<T, NT, false, UNROLL>(W_d, h, M, H, I, residual, Y, nullptr, dev_err, s);
}

template <typename T>
cudaError_t launch_ffn_gemv(const void* X, const void* W_gu, const void* W_d, int M, int H, int I,
                            const float* residual, void* Y, void* gu, void* h, int32_t* dev_err,
                            cudaStream_t s) {
  const bool streams = gemv_streams(H, I);
  if (M > 8)
    return streams
               ? launch_both<T, 2, 8>(X, W_gu, W_d, M, H, I, residual, Y, gu, h, dev_err, s)
               : launch_both<T, 2, 4>(X, W_gu, W_d, M, H, I, residual, Y, gu, h, dev_err, s);
  return streams ? launch_both<T, 1, 2>(X, W_gu, W_d, M, H, I, residual, Y, gu, h, dev_err, s)
                 : launch_both<T, 1, 4>(X, W_gu, W_d, M, H, I, residual, Y, gu, h, dev_err, s);
}

}  // namespace dense
}  // namespace moe
