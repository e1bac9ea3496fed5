// Global 2-norm of many gradient tensors and clipping by it:
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c g.
// A few pieces of work are one launch: a cluster of eight blocks takes them all
// and joins its sums through distributed shared memory.  Beyond that, two
// launches: every block sums the squares of its share of the elements and
// leaves one double; every block of the second adds those in the same fixed
// order (so all agree, and a run repeats bit for bit) and scales its share.
// Which elements add up in fp32 first follows from the 16-byte boundaries of
// memory: the same values at another offset may differ in the last bits.
// The tensors' addresses travel in the launch's parameters, up to kMaxTensors
// per launch, so a captured graph holds them and no device table is needed.
// Bound by memory: 1.02e9 bf16 elements in 290 tensors take 969 us, the three
// passes over 2.04 GB (read; read and write) at 6.3 TB/s, 6.6 within the kernels.
#include "tc_ops.cuh"

namespace moe {
namespace {

constexpr int kMaxTensors = 1024;  // per launch: 24 of the 32764 bytes of parameters each
constexpr int kThreads = 256;
constexpr int kChunkBytes = 32768;  // one piece of work, within one tensor
// Blocks, in multiples of a B200's SMs: the squares' are resident all at once
// there (their number is that of the partial sums, so it is fixed: the sum's order
// must not follow from the device); the scaling's are many, which keeps reads and
// writes mixed.
constexpr int kSumBlocks = 148 * 6, kScaleBlocks = 148 * 128;
// elements of a chunk: 16-bit types 16384, fp32 8192
__host__ __device__ constexpr int chunk_of(uint32_t dt) {
  return dt == MOE_DT_F32 ? kChunkBytes / 4 : kChunkBytes / 2;
}

template <int CAP>
struct Table {
  const void* in[CAP];
  void* out[CAP];
  int chunk0[CAP + 1];  // chunks before tensor i
  uint32_t tail[CAP];   // elements of its last chunk | dtype << 30
  int n;
};

// Squares of N values added in fp32, unless they leave its range, then in
// fp64; the running sum is fp64 either way.
template <int N>
__device__ __forceinline__ void add_squares(double& sum, const float (&v)[N]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(v[i], v[i], s);
  // below 1e-20 a square may have lost bits as a subnormal; NaN fails both
  if (s > 1e-20f && s < 1e38f) {
    sum += (double)s;
  } else {
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) d += (double)v[i] * (double)v[i];
    sum += d;
  }
}

// The values of 16 bytes of T.
template <typename T>
constexpr int per16() {
  return 16 / (int)sizeof(T);
}
template <typename T>
__device__ __forceinline__ void unpack16(uint4 r, float (&v)[per16<T>()]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&v)[per16<T>()]) {
  uint4 r;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(v[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  r.x = w[0]; r.y = w[1]; r.z = w[2]; r.w = w[3];
  return r;
}

constexpr int kSumUnroll = 4, kScaleUnroll = 4;  // 16-byte loads in flight per thread

// Elements before the first 16-byte boundary at or after p.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
  const int h = (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T));
  return min(h, n);
}

// (no read-only loads of the gradients: the launch before, a weight gradient or
// an earlier clipping, may still write them when the kernel starts, and in place
// the kernel of few pieces writes them itself)
template <int TH, typename T>
__device__ __forceinline__ double chunk_squares(const T* p, int n) {
  constexpr int P = per16<T>();
  double sum = 0.0;
  const int head = head_of(p, n), vecs = (n - head) / P, tail0 = head + P * vecs;
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kSumUnroll * TH) {
    uint4 r[kSumUnroll];
#pragma unroll
    for (int j = 0; j < kSumUnroll; ++j)
      r[j] = i0 + j * TH < vecs ? q[i0 + j * TH] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < kSumUnroll; ++j) {
      if (i0 + j * TH >= vecs) break;
      float v[P];
      unpack16<T>(r[j], v);
      add_squares(sum, v);
    }
  }
  const int rest = head + (n - tail0);  // fewer than 16 elements
  if ((int)threadIdx.x < rest) {
    const int i = threadIdx.x < head ? threadIdx.x : tail0 + (threadIdx.x - head);
    const double d = (double)to_f32<T>(p[i]);
    sum += d * d;
  }
  return sum;
}

template <int TH, typename T>
__device__ __forceinline__ void chunk_scale(const T* p, T* o, int n, float c) {
  const int head = head_of(o, n);
  if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0) {
    constexpr int P = per16<T>();
    const int vecs = (n - head) / P, tail0 = head + P * vecs;
    const uint4* q = reinterpret_cast<const uint4*>(p + head);
    uint4* w = reinterpret_cast<uint4*>(o + head);
    for (int i0 = threadIdx.x; i0 < vecs; i0 += kScaleUnroll * TH) {
      uint4 r[kScaleUnroll];
#pragma unroll
      for (int j = 0; j < kScaleUnroll; ++j)
        if (i0 + j * TH < vecs) r[j] = q[i0 + j * TH];
#pragma unroll
      for (int j = 0; j < kScaleUnroll; ++j) {
        if (i0 + j * TH >= vecs) break;
        float v[P];
        unpack16<T>(r[j], v);
#pragma unroll
        for (int e = 0; e < P; ++e) v[e] *= c;
        w[i0 + j * TH] = pack16<T>(v);
      }
    }
    const int rest = head + (n - tail0);
    if ((int)threadIdx.x < rest) {
      const int i = threadIdx.x < head ? threadIdx.x : tail0 + (threadIdx.x - head);
      o[i] = from_f32<T>(to_f32<T>(p[i]) * c);
    }
  } else {  // the two lie differently against 16 bytes
    for (int i = threadIdx.x; i < n; i += TH) o[i] = from_f32<T>(to_f32<T>(p[i]) * c);
  }
}

template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& t, int chunk) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.chunk0[mid] <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

template <int TH>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double w[TH / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) w[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < TH / 32; ++i) v += w[i];
  __syncthreads();
  return v;
}

// Squares of piece c of the table.
template <int TH, int CAP>
__device__ __forceinline__ double piece_squares(const Table<CAP>& t, int c) {
  const int i = tensor_of(t, c), k = c - t.chunk0[i];
  const uint32_t dt = t.tail[i] >> 30;
  const int n = c + 1 == t.chunk0[i + 1] ? (int)(t.tail[i] & 0x3fffffffu) : chunk_of(dt);
  const size_t at = (size_t)k * chunk_of(dt);
  if (dt == MOE_DT_F32) return chunk_squares<TH>(static_cast<const float*>(t.in[i]) + at, n);
  if (dt == MOE_DT_BF16)
    return chunk_squares<TH>(static_cast<const __nv_bfloat16*>(t.in[i]) + at, n);
  return chunk_squares<TH>(static_cast<const __half*>(t.in[i]) + at, n);
}
template <int TH, int CAP>
__device__ __forceinline__ void piece_scale(const Table<CAP>& t, int c, float f) {
  const int i = tensor_of(t, c), k = c - t.chunk0[i];
  if (f == 1.0f && t.in[i] == t.out[i]) return;  // in place and nothing to change
  const uint32_t dt = t.tail[i] >> 30;
  const int n = c + 1 == t.chunk0[i + 1] ? (int)(t.tail[i] & 0x3fffffffu) : chunk_of(dt);
  const size_t at = (size_t)k * chunk_of(dt);
  if (dt == MOE_DT_F32)
    chunk_scale<TH>(static_cast<const float*>(t.in[i]) + at, static_cast<float*>(t.out[i]) + at, n,
                    f);
  else if (dt == MOE_DT_BF16)
    chunk_scale<TH>(static_cast<const __nv_bfloat16*>(t.in[i]) + at,
                    static_cast<__nv_bfloat16*>(t.out[i]) + at, n, f);
  else
    chunk_scale<TH>(static_cast<const __half*>(t.in[i]) + at, static_cast<__half*>(t.out[i]) + at,
                    n, f);
}

// The factor for the sum of squares; one thread of the grid (tell) writes the norm.
__device__ __forceinline__ float factor_of(double sum, float max_norm, float* norm_out, bool tell,
                                           int32_t* dev_err) {
  const double norm = sqrt(sum);
  const bool fine = isfinite(norm);
  const double f = (double)max_norm / (norm + 1e-6);
  if (tell) {
    *norm_out = (float)norm;
    if (!fine) set_dev_err(dev_err, MOE_DEVERR_NONFINITE);
  }
  return fine && f < 1.0 ? (float)f : 1.0f;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 6) squares_kernel(const __grid_constant__ Table<CAP> t,
                                                              double* part) {
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  const int chunks = t.chunk0[t.n];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) sum += piece_squares<kThreads>(t, c);
  sum = block_sum<kThreads>(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// (part is no restricted pointer: the launch before may still write it when this
// one starts, so it must not be read by read-only loads)
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4)
    scale_kernel(const __grid_constant__ Table<CAP> t, const double* part, int parts,
                 float max_norm, float* __restrict__ norm_out, int first, int32_t* dev_err) {
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
  sum = block_sum<kThreads>(sum);
  const float f = factor_of(sum, max_norm, norm_out,
                            first && blockIdx.x == 0 && threadIdx.x == 0, dev_err);
  const int chunks = t.chunk0[t.n];
  // from the last chunk down: what the first pass read last is still in L2
  for (int c = chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) piece_scale<kThreads>(t, c, f);
}

// Few pieces: one cluster of kFewBlocks blocks, one launch.
constexpr int kFewBlocks = 8, kFewThreads = 512;
// At most so many: 1.2 MB in 37 pieces took 11 us here and 5 us in two launches, whose host
// side is 3 us longer.
constexpr int kFewPieces = 24;
template <int CAP>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_kernel(const __grid_constant__ Table<CAP> t, float max_norm, float* __restrict__ norm_out,
               int32_t* dev_err) {
  __shared__ double mine;
  pdl_wait();
  pdl_trigger();
  double sum = 0.0;
  const int chunks = t.chunk0[t.n], rank = (int)tc::cluster_rank();
  for (int c = rank; c < chunks; c += kFewBlocks) sum += piece_squares<kFewThreads>(t, c);
  sum = block_sum<kFewThreads>(sum);
  if (threadIdx.x == 0) mine = sum;
  tc::cluster_sync();
  sum = 0.0;
#pragma unroll
  for (int r = 0; r < kFewBlocks; ++r) {  // in rank order: all agree
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(tc::cluster_addr(&mine, r)));
    sum += v;
  }
  const float f =
      factor_of(sum, max_norm, norm_out, rank == 0 && threadIdx.x == 0, dev_err);
  for (int c = rank; c < chunks; c += kFewBlocks) piece_scale<kFewThreads>(t, c, f);
  tc::cluster_sync();  // nobody leaves while a peer may read its sum
}

}  // namespace
}  // namespace moe

namespace moe_launch {
using namespace moe;

size_t grad_norm_clip_workspace(int n) {
  const size_t launches = ((size_t)n + kMaxTensors - 1) / kMaxTensors;
  return std::max<size_t>(launches, 1) * kSumBlocks * sizeof(double);
}

// Fills a table with tensors [i0, i1) of the non-empty ones.
template <int CAP>
static cudaError_t run(const void* const* grads, const int64_t* numel, const moe_dtype_t* dt, int n,
                       float max_norm, void* const* outs, float* norm, double* part,
                       int32_t* dev_err, cudaStream_t s) {
  const int launches = std::max(1, (n + CAP - 1) / CAP);
  auto fill = [&](Table<CAP>& t, int l) {
    t.n = 0;
    int64_t chunks = 0;
    t.chunk0[0] = 0;
    for (int i = l * CAP; i < std::min(n, (l + 1) * CAP); ++i) {
      if (numel[i] == 0) continue;
      const uint32_t per = chunk_of(dt[i]);
      const int64_t c = (int64_t)(((uint64_t)numel[i] + per - 1) / per);
      t.in[t.n] = grads[i];
      t.out[t.n] = outs ? outs[i] : const_cast<void*>(grads[i]);
      t.tail[t.n] = (uint32_t)(numel[i] - (c - 1) * per) | ((uint32_t)dt[i] << 30);
      chunks += c;
      t.chunk0[++t.n] = (int)chunks;
    }
    return chunks;
  };
  auto blocks_of = [](int64_t chunks, int most) {
    return dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(chunks, most)));
  };
  Table<CAP> t;
  int parts = 0;
  int64_t chunks = fill(t, 0);
  if (launches == 1 && chunks <= kFewPieces) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kFewBlocks);
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kFewBlocks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_kernel<CAP>, t, max_norm, norm, dev_err);
  }
  for (int l = 0; l < launches; ++l) {
    if (l > 0) chunks = fill(t, l);
    const dim3 b = blocks_of(chunks, kSumBlocks);
    cudaError_t e = launch_pdl(squares_kernel<CAP>, b, dim3(kThreads), 0, s, t, part + parts);
    if (e) return e;
    parts += (int)b.x;
  }
  for (int l = 0; l < launches; ++l) {
    if (launches > 1) chunks = fill(t, l);
    cudaError_t e = launch_pdl(scale_kernel<CAP>, blocks_of(chunks, kScaleBlocks), dim3(kThreads),
                               0, s, t, static_cast<const double*>(part), parts, max_norm, norm,
                               l == 0 ? 1 : 0, dev_err);
    if (e) return e;
  }
  return cudaSuccess;
}

cudaError_t grad_norm_clip(const void* const* grads, const int64_t* numel, const moe_dtype_t* dt,
                           int n, float max_norm, void* const* outs, float* norm, void* ws,
                           int32_t* dev_err, cudaStream_t s) {
  double* part = static_cast<double*>(ws);
  // parameters cost host time by their size: the smallest table that holds all
  if (n <= 64)
    return run<64>(grads, numel, dt, n, max_norm, outs, norm, part, dev_err, s);
  if (n <= 256)
    return run<256>(grads, numel, dt, n, max_norm, outs, norm, part, dev_err, s);
  if (n <= 512)
    return run<512>(grads, numel, dt, n, max_norm, outs, norm, part, dev_err, s);
  return run<kMaxTensors>(grads, numel, dt, n, max_norm, outs, norm, part, dev_err, s);
}

}  // namespace moe_launch
