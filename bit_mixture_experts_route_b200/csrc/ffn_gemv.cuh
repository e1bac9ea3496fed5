// The gated feed-forward block for a few tokens (at most 16): both products
// are bound by streaming the weights once, so they run as matrix-vector
// kernels on the warp MMA (m16n8k16, 16 weight rows x 8 tokens), which needs
// no tensor-memory round trip and no second pass over partial sums.
//
// A block owns 16 weight rows (up: 8 gate rows and their 8 up rows, which land
// in the same thread's accumulators; down: 16 output rows) and its eight warps
// take every eighth 32-k chunk of them.  The sum over k does not depend on
// which k sits in which MMA slot, so a thread feeds the 16 consecutive bytes
// that it loads (8 k of its row) to two MMAs as they are and loads the tokens'
// rows in the same pattern: wide loads, no shuffles, no shared memory but for
// the eight warps' sums at the end, which are added in warp order.
#pragma once

#include "dense_gemm.cuh"

namespace moe {
namespace dense {

constexpr int kGemvWarps = 8;
constexpr int kGemvUnroll = 8;  // 32-k chunks in flight per warp: 16 x 16 bytes a thread
constexpr int kGemvRows = 16;   // tokens at most

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

// UP: out = h [M, rows], gu (if given) [M, 2 rows], A = W_gu [2 rows, K].
// Otherwise out [M, rows] (+ residual), A = W_d [rows, K].  NT: groups of 8
// tokens.  K and rows are multiples of 8.  The down form is launched right
// behind the up form, so its weights cannot be anyone's pending output: it
// loads the first of them before it waits for h.
template <typename T, int NT, bool UP>
__global__ void __launch_bounds__(32 * kGemvWarps) ffn_gemv_kernel(
    const T* __restrict__ A, const T* __restrict__ X, int M, int rows, int K,
    const float* __restrict__ residual, T* __restrict__ out, T* __restrict__ gu,
    int32_t* dev_err) {
  __shared__ float sums[kGemvWarps][NT][32][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (UP) {
    pdl_wait();
    pdl_trigger();
  }
  // this thread's two weight rows (clamped to a real one; the last block of
  // the down form may own 8 rows only) and its tokens' rows
  const int r0 = UP ? blockIdx.x * 8 + g : blockIdx.x * 16 + g;
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
  const int chunks = (K + 31) / 32;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  bool first = !UP;
  for (int c0 = warp; c0 < chunks; c0 += kGemvWarps * kGemvUnroll) {
    uint4 a0[kGemvUnroll], a1[kGemvUnroll];
#pragma unroll
    for (int i = 0; i < kGemvUnroll; ++i) {
      const int k = 32 * (c0 + i * kGemvWarps);
      const bool in = k + 8 * t < K;
      a0[i] = in ? ldg_stream_u4(a0p + k) : zero;
      a1[i] = in ? ldg_stream_u4(a1p + k) : zero;
    }
    if (first) {
      pdl_wait();
      pdl_trigger();
      first = false;
    }
#pragma unroll
    for (int i = 0; i < kGemvUnroll; ++i) {
      const int k = 32 * (c0 + i * kGemvWarps);
      if (k >= K) break;
      const bool in = k + 8 * t < K;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = in && live[n] ? *reinterpret_cast<const uint4*>(xp[n] + k) : zero;
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
  bool ovf = false;
  for (int i = threadIdx.x; i < NT * 64; i += 32 * kGemvWarps) {
    const int n = i >> 6, tok_l = (i >> 3) & 7, row = i & 7;
    const int src = 4 * row + (tok_l >> 1), e = tok_l & 1, tok = 8 * n + tok_l;
    if (tok >= M) continue;
    float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kGemvWarps; ++w) {
      v0 += sums[w][n][src][e];
      v1 += sums[w][n][src][2 + e];
    }
    if (UP) {
      const int j = blockIdx.x * 8 + row;
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
        const int j = blockIdx.x * 16 + 8 * half + row;
        if (j >= rows) continue;
        float v = half ? v1 : v0;
        if (residual) v += residual[(size_t)tok * rows + j];
        ovf |= overflows_out<T>(v);
        out[(size_t)tok * rows + j] = from_f32<T>(v);
      }
    }
  }
  if (ovf) set_dev_err(dev_err, MOE_DEVERR_RANGE);
}

template <typename T, int NT>
cudaError_t launch_ffn_gemv(const void* X, const void* W_gu, const void* W_d, int M, int H, int I,
                            const float* residual, void* Y, void* gu, void* h, int32_t* dev_err,
                            cudaStream_t s) {
  cudaError_t e = launch_pdl(ffn_gemv_kernel<T, NT, true>, dim3(I / 8), dim3(32 * kGemvWarps), 0, s,
                             static_cast<const T*>(W_gu), static_cast<const T*>(X), M, I, H,
                             static_cast<const float*>(nullptr), static_cast<T*>(h),
                             static_cast<T*>(gu), dev_err);
  if (e) return e;
  return launch_pdl(ffn_gemv_kernel<T, NT, false>, dim3(ceil_div(H, 16)), dim3(32 * kGemvWarps), 0,
                    s, static_cast<const T*>(W_d), static_cast<const T*>(h), M, H, I, residual,
                    static_cast<T*>(Y), static_cast<T*>(nullptr), dev_err);
}

}  // namespace dense
}  // namespace moe
