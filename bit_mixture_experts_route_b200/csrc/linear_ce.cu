// Softmax cross entropy over a large vocabulary, straight from the hidden rows
// and the head's weights, and its gradient; the logits l = X W^T are never
// kept.
//   lse_t = log sum_v exp l[t, v],  loss_t = lse_t - l[t, y_t]
//   dl[t, v] = (exp(l[t, v] - lse_t) - [v = y_t]) dloss_t,  dX = dl W,  dW = dl^T X
//
// Rows whose target is the ignored index take no part: the rows that count are
// gathered first (X rows, targets, upstream gradients), so nothing of an
// ignored row -- NaN included -- reaches a sum, and the tensor cores spend
// nothing on it.  Their number stays on the device.
//
// Forward: one GEMM over all tiles; each epilogue thread owns one row and 128
// vocabulary columns of a tile and leaves (maximum, sum of exponentials); a
// second kernel joins the pieces of a row in a fixed order.
// Backward: pieces of the vocabulary.  Per piece the logits are computed again
// and turned to dl (16 bits, at most kPieceBytes of workspace), which two more
// GEMMs read: dX accumulates over the pieces in fp32 partial sums, dW's rows of
// the piece are written at once.  dl enters them as (p - [v = y]) * dloss /
// max|dloss| (fp16: times 2^15, so that probabilities down to 2e-9 stay normal
// numbers), and the factor comes back in fp32 at the end.
#include "dense_gemm.cuh"

namespace moe {
namespace {

using namespace dense;

constexpr size_t kPieceBytes = (size_t)256 << 20;  // of dl
constexpr int kPartTiles = 148;

struct Meta {
  int rows;         // that count
  float in_scale;   // dl = (p - onehot) * dloss * in_scale
  float out_scale;  // 1 / in_scale, rounded once
};

// One block: the rows that count, in order.  inv[t] = place of row t among
// them or -1; row_of and target by place; loss and lse of ignored rows are 0.
__global__ void __launch_bounds__(1024) ce_select_kernel(
    const int* __restrict__ targets, int T, int V, int ignore_index,
    const float* __restrict__ dloss, float in_unit, Meta* meta, int* __restrict__ inv,
    int* __restrict__ row_of, float* __restrict__ loss, float* __restrict__ lse,
    int32_t* dev_err) {
  __shared__ int wcount[32];
  __shared__ float wmax[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int base = 0;
  float big = 0.0f;
  bool bad = false;
  for (int t0 = 0; t0 < T; t0 += 1024) {
    const int t = t0 + tid;
    const int y = t < T ? targets[t] : ignore_index;
    const bool real = t < T && y != ignore_index;
    const bool keep = real && y >= 0 && y < V;
    bad |= real && !keep;
    const unsigned m = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) wcount[warp] = __popc(m);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
      before += w < warp ? wcount[w] : 0;
      all += wcount[w];
    }
    __syncthreads();
    const int at = base + before + __popc(m & lanemask_lt());
    if (keep) {
      row_of[at] = t;
      if (dloss) big = fmaxf(big, fabsf(dloss[t]));
    } else if (t < T && loss) {
      loss[t] = 0.0f;
      lse[t] = 0.0f;
    }
    if (t < T) inv[t] = keep ? at : -1;
    base += all;
  }
  if (bad) set_dev_err(dev_err, MOE_DEVERR_BAD_INDEX);
  big = warp_max(big);
  if (lane == 0) wmax[warp] = big;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < 32; ++w) big = fmaxf(big, wmax[w]);
    // no scaling by a zero, infinite or subnormal maximum
    if (!(big >= 1e-30f && big <= 1e30f)) big = 1.0f;
    meta->rows = base;
    meta->in_scale = in_unit / big;
    meta->out_scale = big / in_unit;
  }
}

// One warp per place: the row's X, target and gradient scale; zero rows up to
// the end of the last 256-row tile.
__global__ void __launch_bounds__(256) ce_gather_kernel(
    const uint4* __restrict__ X, int vecs, const int* __restrict__ targets,
    const float* __restrict__ dloss, const float* __restrict__ lse, const Meta* __restrict__ meta,
    const int* __restrict__ row_of, uint4* __restrict__ Xc, int* __restrict__ ctarget,
    float* __restrict__ clse, float* __restrict__ cscale) {
  pdl_wait();
  pdl_trigger();
  const int at = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int rows = meta->rows;
  if (at >= (rows + TILE - 1) / TILE * TILE) return;
  const bool real = at < rows;
  const int t = real ? row_of[at] : 0;
  const uint4* src = X + (size_t)t * vecs;
  uint4* dst = Xc + (size_t)at * vecs;
  for (int i = lane; i < vecs; i += 32) dst[i] = real ? src[i] : make_uint4(0, 0, 0, 0);
  if (lane == 0) {
    ctarget[at] = real ? targets[t] : -1;
    if (dloss) {
      clse[at] = real ? lse[t] : 0.0f;
      cscale[at] = real ? dloss[t] * meta->in_scale : 0.0f;
    }
  }
}

// The (max, sum) pieces of 32 rows: warp w joins pieces w, w + W, ..., then the
// first warp joins the warps in order.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps) ce_join_kernel(
    const float2* __restrict__ stats, int pieces, int rows_pad, const float* __restrict__ tsum,
    const Meta* __restrict__ meta, const int* __restrict__ row_of, float* __restrict__ loss,
    float* __restrict__ lse) {
  __shared__ float2 part[kJoinWarps][32];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int at = blockIdx.x * 32 + lane, rows = meta->rows;
  if (blockIdx.x * 32 >= rows) return;
  float m = -INFINITY, s = 0.0f;
  auto join = [&](float2 o) {
    if (o.y == 0.0f && o.x == -INFINITY) return;  // no columns
    const float mn = fmaxf(m, o.x);
    s = s * exp2f((m - mn) * kLog2e) + o.y * exp2f((o.x - mn) * kLog2e);
    m = mn;
  };
  if (at < rows) {
    int i = warp;
    for (; i + 3 * kJoinWarps < pieces; i += 4 * kJoinWarps) {
      float2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = stats[(size_t)(i + j * kJoinWarps) * rows_pad + at];
#pragma unroll
      for (int j = 0; j < 4; ++j) join(o[j]);
    }
    for (; i < pieces; i += kJoinWarps) join(stats[(size_t)i * rows_pad + at]);
  }
  part[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp == 0 && at < rows) {
    for (int w = 1; w < kJoinWarps; ++w) join(part[w][lane]);
    const float z = m + logf(s);
    const int t = row_of[at];
    loss[t] = z - tsum[at];
    lse[t] = z;
  }
}

size_t align1k(size_t b) { return (b + 1023) & ~(size_t)1023; }

// Layout of both workspaces.
struct Space {
  size_t meta, inv, row_of, ctarget, clse, cscale, xc, stats, tsum, dl, part, total;
  int rows_pad, piece, pieces, splits;
};
// Vocabulary columns of one piece: dl of all rows within kPieceBytes, the
// pieces as even as whole 256-column tiles allow.
Space space_of(int T, int H, int V, bool backward) {
  Space w = {};
  w.rows_pad = ceil_div(T, TILE) * TILE;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align1k(bytes);
    return o;
  };
  w.meta = take(sizeof(Meta));
  w.inv = take((size_t)T * 4);
  w.row_of = take((size_t)T * 4);
  w.ctarget = take((size_t)w.rows_pad * 4);
  w.xc = take((size_t)w.rows_pad * H * 2);
  if (!backward) {
    w.stats = take((size_t)2 * ceil_div(V, TILE) * w.rows_pad * sizeof(float2));
    w.tsum = take((size_t)w.rows_pad * 4);
  } else {
    w.clse = take((size_t)w.rows_pad * 4);
    w.cscale = take((size_t)w.rows_pad * 4);
    const int64_t most = std::max<int64_t>(
        TILE, (int64_t)(kPieceBytes / (2 * (size_t)w.rows_pad)) / TILE * TILE);
    w.pieces = ceil_div(V, most);
    w.piece = ceil_div(ceil_div(V, w.pieces), TILE) * TILE;
    w.pieces = ceil_div(V, w.piece);
    w.dl = take((size_t)w.rows_pad * w.piece * 2);
    const int tiles = w.rows_pad / TILE * ceil_div(H, TILE);
    const int ks = ceil_div(std::min(V, w.piece), GK);
    w.splits = pick_splits(tiles, ks, std::max(1, kPartTiles / tiles), true);
    w.part = take((size_t)w.splits * tiles * TILE_FLOATS * 4);
  }
  w.total = at;
  return w;
}

template <typename T>
cudaError_t select(const Space& w, char* ws, const void* X, const int* targets, int rows, int H,
                   int V, int ignore_index, const float* dloss, const float* lse_in, float* loss,
                   float* lse, int32_t* dev_err, cudaStream_t s) {
  const float unit = std::is_same<T, __half>::value ? 32768.0f : 1.0f;
  Meta* meta = reinterpret_cast<Meta*>(ws + w.meta);
  int* row_of = reinterpret_cast<int*>(ws + w.row_of);
  cudaError_t e = launch_pdl(ce_select_kernel, dim3(1), dim3(1024), 0, s, targets, rows, V,
                             ignore_index, dloss, unit, meta, reinterpret_cast<int*>(ws + w.inv),
                             row_of, loss, lse, dev_err);
  if (e) return e;
  return launch_pdl(ce_gather_kernel, dim3(w.rows_pad / 8), dim3(256), 0, s,
                    static_cast<const uint4*>(X), H / 8, targets, dloss, lse_in,
                    static_cast<const Meta*>(meta), static_cast<const int*>(row_of),
                    reinterpret_cast<uint4*>(ws + w.xc), reinterpret_cast<int*>(ws + w.ctarget),
                    reinterpret_cast<float*>(ws + w.clse),
                    reinterpret_cast<float*>(ws + w.cscale));
}

template <typename T>
cudaError_t forward(const void* X, const void* W, const int* targets, int rows, int H, int V,
                    int ignore_index, float* loss, float* lse, char* ws, int32_t* dev_err,
                    cudaStream_t s) {
  const Space w = space_of(rows, H, V, false);
  cudaError_t e = select<T>(w, ws, X, targets, rows, H, V, ignore_index, nullptr, nullptr, loss,
                            lse, dev_err, s);
  if (e) return e;
  const Meta* meta = reinterpret_cast<const Meta*>(ws + w.meta);
  GemmArgs p = {};
  p.N = V;
  p.M = rows;
  p.m_tiles = w.rows_pad / TILE;
  p.n_tiles = ceil_div(V, TILE);
  p.k_stages = p.kps = ceil_div(H, GK);
  p.splits = 1;
  p.rows = &meta->rows;
  p.dyn = 1;
  p.stats = reinterpret_cast<float2*>(ws + w.stats);
  p.target_sum = reinterpret_cast<float*>(ws + w.tsum);
  p.targets = reinterpret_cast<const int*>(ws + w.ctarget);
  p.rows_pad = w.rows_pad;
  p.dev_err = dev_err;
  CUtensorMap am, bm;
  if (!map_2d<T>(&am, ws + w.xc, w.rows_pad, H, H, CM) || !map_2d<T>(&bm, W, V, H, H, CM))
    return cudaErrorInvalidValue;
  e = launch_gemm_maps<T, false, false, E_STATS>(am, bm, am, am, p, s);
  if (e) return e;
  return launch_pdl(ce_join_kernel, dim3(w.rows_pad / 32), dim3(32 * kJoinWarps), 0, s,
                    static_cast<const float2*>(p.stats), 2 * p.n_tiles, w.rows_pad,
                    static_cast<const float*>(p.target_sum), meta,
                    reinterpret_cast<const int*>(ws + w.row_of), loss, lse);
}

template <typename T>
cudaError_t backward(const float* dloss, const void* X, const void* W, const int* targets,
                     const float* lse, int rows, int H, int V, int ignore_index, void* dX,
                     void* dW, char* ws, int32_t* dev_err, cudaStream_t s) {
  const Space w = space_of(rows, H, V, true);
  cudaError_t e = select<T>(w, ws, X, targets, rows, H, V, ignore_index, dloss, lse, nullptr,
                            nullptr, dev_err, s);
  if (e) return e;
  const Meta* meta = reinterpret_cast<const Meta*>(ws + w.meta);
  const int mt = w.rows_pad / TILE, ht = ceil_div(H, TILE);
  char* dl = ws + w.dl;
  float* part = reinterpret_cast<float*>(ws + w.part);
  int splits = 0;
  for (int i = 0; i < w.pieces; ++i) {
    const int v0 = i * w.piece, vn = std::min(w.piece, V - v0);
    const char* Wi = static_cast<const char*>(W) + (size_t)v0 * H * 2;
    GemmArgs p = {};
    p.N = vn;
    p.M = rows;
    p.m_tiles = mt;
    p.n_tiles = ceil_div(vn, TILE);
    p.k_stages = p.kps = ceil_div(H, GK);
    p.splits = 1;
    p.rows = &meta->rows;
    p.dyn = 1;
    p.targets = reinterpret_cast<const int*>(ws + w.ctarget);
    p.lse = reinterpret_cast<const float*>(ws + w.clse);
    p.row_scale = reinterpret_cast<const float*>(ws + w.cscale);
    p.col0 = v0;
    p.rows_pad = w.rows_pad;
    p.dev_err = dev_err;
    CUtensorMap lm;
    if (!map_2d<T>(&lm, dl, w.rows_pad, vn, w.piece, 32)) return cudaErrorInvalidValue;
    e = launch_gemm<T, false, false, E_DLOGITS>({ws + w.xc, w.rows_pad, H, H}, {Wi, vn, H, H}, lm,
                                                lm, p, s);
    if (e) return e;
    if (dX) {
      GemmArgs q = {};
      q.N = H;
      q.M = rows;
      q.m_tiles = mt;
      q.n_tiles = ht;
      // every piece adds to the same splits' sums: a shorter last piece is cut
      // anew, and a split left without stages adds zeros
      q.k_stages = ceil_div(vn, GK);
      if (i == 0) splits = ceil_div(q.k_stages, ceil_div(q.k_stages, w.splits));
      q.kps = ceil_div(q.k_stages, splits);
      q.splits = splits;
      q.rows = &meta->rows;
      q.dyn = 1;
      q.part = part;
      q.accumulate = i > 0;
      q.dev_err = dev_err;
      e = launch_gemm<T, false, true, E_PART>({dl, w.rows_pad, vn, w.piece}, {Wi, H, vn, H}, lm,
                                              lm, q, s);
      if (e) return e;
    }
    if (dW) {
      GemmArgs q = {};
      q.N = H;
      q.M = vn;
      q.m_tiles = ceil_div(vn, TILE);
      q.n_tiles = ht;
      q.k_stages = q.kps = w.rows_pad / GK;
      q.splits = 1;
      q.rows = &meta->rows;
      q.dyn = 2;
      q.scale = &meta->out_scale;
      q.dev_err = dev_err;
      CUtensorMap om;
      if (!map_2d<T>(&om, static_cast<char*>(dW) + (size_t)v0 * H * 2, vn, H, H, 32))
        return cudaErrorInvalidValue;
      e = launch_gemm<T, true, true, E_STORE>({dl, vn, w.rows_pad, w.piece},
                                              {ws + w.xc, H, w.rows_pad, H}, om, om, q, s);
      if (e) return e;
    }
  }
  if (!dX) return cudaSuccess;
  FinishArgs f = {};
  f.part = part;
  f.splits = splits;
  f.n_tiles = ht;
  f.split_stride = (size_t)mt * ht * TILE_FLOATS;
  f.M = rows;
  f.N = H;
  f.scale = &meta->out_scale;
  f.row_of = reinterpret_cast<const int*>(ws + w.inv);
  f.out = dX;
  f.dev_err = dev_err;
  return launch_finish<T, F_PLAIN>(f, s);
}

}  // namespace
}  // namespace moe

namespace moe_launch {
using namespace moe;

size_t linear_ce_workspace(int T, int H, int V, bool backward) {
  return space_of(T, H, V, backward).total;
}

cudaError_t linear_ce_forward(const void* X, moe_dtype_t dt, const void* W, const int32_t* targets,
                              int T, int H, int V, int ignore_index, float* loss, float* lse,
                              void* ws, int32_t* dev_err, cudaStream_t s) {
  if (dt == MOE_DT_F16)
    return forward<__half>(X, W, targets, T, H, V, ignore_index, loss, lse,
                           static_cast<char*>(ws), dev_err, s);
  return forward<__nv_bfloat16>(X, W, targets, T, H, V, ignore_index, loss, lse,
                                static_cast<char*>(ws), dev_err, s);
}

cudaError_t linear_ce_backward(const float* dloss, const void* X, moe_dtype_t dt, const void* W,
                               const int32_t* targets, const float* lse, int T, int H, int V,
                               int ignore_index, void* dX, void* dW, void* ws, int32_t* dev_err,
                               cudaStream_t s) {
  if (dt == MOE_DT_F16)
    return backward<__half>(dloss, X, W, targets, lse, T, H, V, ignore_index, dX, dW,
                            static_cast<char*>(ws), dev_err, s);
  return backward<__nv_bfloat16>(dloss, X, W, targets, lse, T, H, V, ignore_index, dX, dW,
                                 static_cast<char*>(ws), dev_err, s);
}

}  // namespace moe_launch
