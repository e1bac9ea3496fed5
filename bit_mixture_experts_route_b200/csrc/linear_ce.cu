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
// Measured (bf16, 4096 rows of 2048, 151936 words): forward 1.96 ms = 1.30
// PFLOP/s; backward with a quarter of the rows ignored 4.83 ms = 1.19, under the
// power cap; 40 rows, 50304 words: 47 us, 4.4 TB/s of W over the whole call.
#include "skinny_gemm.cuh"

namespace moe {
namespace {

using namespace dense;

constexpr size_t kPieceBytes = (size_t)256 << 20;  // of dl
// dX's fp32 sums: at most so many tiles of 256 KB for the splits of its
// reduction, unless one copy is more.  Splits are worth their sums where the
// tiles of the rows that count leave a part-filled last round, so their number is
// chosen on the device within this room.
constexpr int kSumTiles = 1024;

struct Meta {
  int rows;         // that count
  int splits;       // of dX's reduction (see even_splits)
  float out_scale;  // of dl's products: max |dloss| / the unit of dl
  int arrived[EPI_NW * 8];  // see SkinnyArgs, 0 from the gathering launch on
};

// What the gathering kernels read and write, by row and by place.
struct GatherArgs {
  const uint4* X;
  const uint4* W;
  int vecs;            // 16-byte vectors of a row
  const int* targets;
  int rows_all, V, ignore_index;
  const float* dloss;  // backward: with lse_in; or null
  const float* lse_in;
  float in_unit;
  Meta* meta;
  // of dX's reduction; most_splits 0: none
  int n_tiles, k_stages, most_splits, part_tiles, pairs;
  int* inv;
  int* row_of;
  uint4* Xc;
  int* ctarget;
  float* ctsum;
  float* clse;
  float* cscale;
  float* loss;         // forward: 0 in the other rows; or null
  float* lse;
  uint4* dX;           // zero rows for the other rows; or null
  int32_t* dev_err;
};

// Gathers the rows that count, in order: place among them = how many before it
// count.  Every block counts for itself (the targets are few next to X), so
// one launch does it all.  Slot t is row t: if it counts, its X, target and
// gradient scale go to its place, with its target's logit in fp32; if not, the
// slot writes a zero row behind the last place, up to the end of that 256-row
// tile.  inv[t] = place or -1; row_of by place; loss and lse (and, where given,
// dX) of the other rows are 0.
//
// The target's logit is computed here, not taken from the tensor cores' sums:
// those round toward zero at every step (about 2e-6 relative at 2048 terms),
// which in loss = lse - l[target] and in p[target] - 1 does not average out.
// It also stands in for the tile's own sum, so that the loss of a confident
// row stays the logarithm of a sum >= 1.
struct Count {
  int all, before;  // rows that count; those before `first`
  float big;        // max |dloss|
};
// By the whole block of 256 threads.
__device__ __forceinline__ Count count_rows(const GatherArgs& p, int first) {
  __shared__ int s_all[8], s_before[8];
  __shared__ float s_big[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int all = 0, before = 0;
  float big = 0.0f;
  bool bad = false;
  auto count = [&](int t, int y) {
    const bool real = y != p.ignore_index;
    const bool keep = real && (unsigned)y < (unsigned)p.V;
    bad |= real && !keep;
    all += keep;
    before += keep && t < first;
    if (keep && p.dloss) big = fmaxf(big, fabsf(p.dloss[t]));
  };
  const int quads = p.rows_all / 4;
#pragma unroll 4
  for (int i = tid; i < quads; i += 256) {
    const int4 y = reinterpret_cast<const int4*>(p.targets)[i];
    count(4 * i, y.x);
    count(4 * i + 1, y.y);
    count(4 * i + 2, y.z);
    count(4 * i + 3, y.w);
  }
  if (4 * quads + tid < p.rows_all) count(4 * quads + tid, p.targets[4 * quads + tid]);
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  big = warp_max(big);
  if (lane == 0) {
    s_all[warp] = all;
    s_before[warp] = before;
    s_big[warp] = big;
  }
  __syncthreads();
  Count c = {0, 0, 0.0f};
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    c.all += s_all[w];
    c.before += s_before[w];
    c.big = fmaxf(c.big, s_big[w]);
  }
  // no scaling by a zero, infinite or tiny maximum
  if (!(c.big >= 1e-30f && c.big <= 1e30f)) c.big = 1.0f;
  if (blockIdx.x == 0 && tid == 0) {
    p.meta->rows = c.all;
    p.meta->out_scale = c.big / p.in_unit;
  }
  if (blockIdx.x == 0 && tid < EPI_NW * 8) p.meta->arrived[tid] = 0;
  if (blockIdx.x == 0 && warp == 1 && p.most_splits > 0) {
    const int tiles = (c.all + TILE - 1) / TILE * p.n_tiles;
    const int most = min(p.most_splits, p.part_tiles / max(tiles, 1));
    const int sp = even_splits(tiles, p.k_stages, most, p.pairs);
    if (lane == 0) p.meta->splits = sp;
  }
  if (blockIdx.x == 0 && bad) set_dev_err(p.dev_err, MOE_DEVERR_BAD_INDEX);
  return c;
}
template <typename T>
__device__ __forceinline__ void dot_add(float (&d)[4], uint4 x, uint4 w) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = unpack2<T>(xs[e]), b = unpack2<T>(ws[e]);
    d[e] = fmaf(a.x, b.x, d[e]);
    d[e] = fmaf(a.y, b.y, d[e]);
  }
}
// The scalars of slot t, by one thread: place `at`, target y (keep) or none.
__device__ __forceinline__ void gather_scalars(const GatherArgs& p, int t, int at, bool keep,
                                               int y, float dot, float big) {
  p.ctarget[at] = keep ? y : -1;
  p.ctsum[at] = dot;
  if (keep) {
    p.inv[t] = at;
    p.row_of[at] = t;
  }
  if (p.dloss) {
    p.clse[at] = keep ? p.lse_in[t] : 0.0f;
    p.cscale[at] = keep ? p.dloss[t] / big * p.in_unit : 0.0f;
  }
}
__device__ __forceinline__ void gather_left_out(const GatherArgs& p, int t) {
  p.inv[t] = -1;
  if (p.loss) {
    p.loss[t] = 0.0f;
    p.lse[t] = 0.0f;
  }
}

// Few rows: a block per slot, so that a row's loads are all in flight at once
// and run under the count.  At 84 of 169 rows of 3432 the warp-per-row form
// took 12 us.
template <typename T>
__global__ void __launch_bounds__(256) ce_gather_few_kernel(const GatherArgs p) {
  __shared__ float s_dot[8];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, t = blockIdx.x;
  const int y = t < p.rows_all ? p.targets[t] : p.ignore_index;
  const bool keep = y != p.ignore_index && (unsigned)y < (unsigned)p.V;
  const uint4* src = p.X + (size_t)t * p.vecs;
  float d[4] = {};
  constexpr int HELD = 2;  // vectors of the row that a thread keeps
  uint4 x[HELD];
  if (keep) {
    const uint4* wr = p.W + (size_t)y * p.vecs;
    uint4 w[HELD];
#pragma unroll
    for (int j = 0; j < HELD; ++j) {
      const bool in = tid + 256 * j < p.vecs;
      x[j] = in ? src[tid + 256 * j] : make_uint4(0, 0, 0, 0);
      w[j] = in ? wr[tid + 256 * j] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < HELD; ++j) dot_add<T>(d, x[j], w[j]);
    for (int i = tid + 256 * HELD; i < p.vecs; i += 256) dot_add<T>(d, src[i], wr[i]);
  }
  const float dot = warp_sum((d[0] + d[1]) + (d[2] + d[3]));
  if ((tid & 31) == 0) s_dot[tid >> 5] = dot;
  const Count c = count_rows(p, t);  // its barrier also stands behind s_dot
  const int at = keep ? c.before : c.all + (t - c.before);
  if (!keep && t < p.rows_all) {
    if (tid == 0) gather_left_out(p, t);
    if (p.dX)
      for (int i = tid; i < p.vecs; i += 256) p.dX[(size_t)t * p.vecs + i] = make_uint4(0, 0, 0, 0);
  }
  if (!keep && at >= (c.all + TILE - 1) / TILE * TILE) return;
  uint4* dst = p.Xc + (size_t)at * p.vecs;
#pragma unroll
  for (int j = 0; j < HELD; ++j)
    if (tid + 256 * j < p.vecs) dst[tid + 256 * j] = keep ? x[j] : make_uint4(0, 0, 0, 0);
  for (int i = tid + 256 * HELD; i < p.vecs; i += 256)
    dst[i] = keep ? src[i] : make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += s_dot[w];
    gather_scalars(p, t, at, keep, y, sum, c.big);
  }
}

// Many rows: a block takes per_block slots, a warp a row at a time.  Every block
// reads all targets, rows^2 / 16 bytes in all beyond 8192 rows: 0.3 GB from L2 for
// 70000, 69 GB for 2^20, which is then a few per cent of the products' time.
template <typename T>
__global__ void __launch_bounds__(256) ce_gather_kernel(const GatherArgs p, int per_block) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x * per_block;
  const Count c = count_rows(p, first);
  int before = c.before;
  const int end = (c.all + TILE - 1) / TILE * TILE;  // of the zero rows
  for (int g = 0; g < per_block; g += 32) {          // 32 slots at a time
    const int t0 = first + g;
    const int y_l =
        t0 + lane < p.rows_all && g + lane < per_block ? p.targets[t0 + lane] : p.ignore_index;
    const unsigned kept =
        __ballot_sync(0xffffffffu, y_l != p.ignore_index && (unsigned)y_l < (unsigned)p.V);
    for (int j = warp; j < 32 && g + j < per_block; j += 8) {
      const int t = t0 + j;
      const int rank = before + __popc(kept & ((1u << j) - 1u));  // rows that count before t
      const bool keep = (kept >> j) & 1u;
      const int y = __shfl_sync(0xffffffffu, y_l, j);
      const int at = keep ? rank : c.all + (t - rank);
      if (!keep && t < p.rows_all) {
        if (lane == 0) gather_left_out(p, t);
        if (p.dX)
          for (int i = lane; i < p.vecs; i += 32)
            p.dX[(size_t)t * p.vecs + i] = make_uint4(0, 0, 0, 0);
      }
      if (!keep && at >= end) continue;
      uint4* dst = p.Xc + (size_t)at * p.vecs;
      float dot = 0.0f;
      if (keep) {
        const uint4* src = p.X + (size_t)t * p.vecs;
        const uint4* wr = p.W + (size_t)y * p.vecs;
        float d[4] = {};
#pragma unroll 4
        for (int i = lane; i < p.vecs; i += 32) {
          const uint4 x = src[i], w = wr[i];
          dst[i] = x;
          dot_add<T>(d, x, w);
        }
        dot = warp_sum((d[0] + d[1]) + (d[2] + d[3]));
      } else {
        for (int i = lane; i < p.vecs; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
      }
      if (lane == 0) gather_scalars(p, t, at, keep, y, dot, c.big);
    }
    before += __popc(kept);
  }
}

// The (max, sum) pieces of 32 rows: warp w joins pieces w, w + W, ..., then the
// first warp joins the warps in order.
constexpr int kJoinWarps = 32;
// (no restricted pointers: the launch before may still write when this one starts)
__global__ void __launch_bounds__(32 * kJoinWarps) ce_join_kernel(
    const float2* stats, int pieces, int rows_pad, const float* tsum, const Meta* meta,
    const int* row_of, float* loss, float* lse) {
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
    for (; i < pieces; i += 8 * kJoinWarps) {
      float2 o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        o[j] = i + j * kJoinWarps < pieces ? stats[(size_t)(i + j * kJoinWarps) * rows_pad + at]
                                           : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int j = 0; j < 8; ++j) join(o[j]);
    }
  }
  part[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp == 0 && at < rows) {
    for (int w = 1; w < kJoinWarps; ++w) join(part[w][lane]);
    const float ls = logf(s);
    const int t = row_of[at];
    loss[t] = (m - tsum[at]) + ls;  // not lse - target: a confident row would lose lse's rounding
    lse[t] = m + ls;
  }
}

// Layout of both workspaces.
struct Space {
  size_t meta, inv, row_of, ctarget, clse, cscale, xc, stats, tsum, dl, part, total;
  int rows_pad, piece, pieces, most_splits, part_tiles;
  bool skinny;  // few rows, one piece: skinny_gemm.cuh
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
  w.tsum = take((size_t)w.rows_pad * 4);
  w.xc = take((size_t)w.rows_pad * H * 2);
  if (!backward) {
    w.skinny = T <= kSkinnyRows;
    w.stats = take(w.skinny ? skinny_stats_bytes(T, V)
                            : (size_t)2 * ceil_div(V, TILE) * w.rows_pad * sizeof(float2));
  } else {
    w.clse = take((size_t)w.rows_pad * 4);
    w.cscale = take((size_t)w.rows_pad * 4);
    const int64_t most = std::max<int64_t>(
        TILE, (int64_t)(kPieceBytes / (2 * (size_t)w.rows_pad)) / TILE * TILE);
    w.pieces = ceil_div(V, most);
    w.piece = ceil_div(ceil_div(V, w.pieces), TILE) * TILE;
    w.pieces = ceil_div(V, w.piece);
    w.dl = take((size_t)w.rows_pad * w.piece * 2);
    w.skinny = T <= kSkinnyRows && w.pieces == 1;
    if (w.skinny) {
      w.part = take(skinny_part_bytes(T, H, V));
    } else {
      const int tiles = w.rows_pad / TILE * ceil_div(H, TILE);
      // few tiles: up to two units per pair of a B200
      w.most_splits = std::min(16, std::max(4, 148 / tiles));
      w.part_tiles = std::min(w.most_splits * tiles, std::max(tiles, kSumTiles));
      w.part = take((size_t)w.part_tiles * TILE_FLOATS * 4);
    }
  }
  w.total = at;
  return w;
}

template <typename T>
cudaError_t gather(const Space& w, char* ws, const void* X, const void* W, const int* targets,
                   int rows, int H, int V, int ignore_index, const float* dloss,
                   const float* lse_in, float* loss, float* lse, void* dX, int32_t* dev_err,
                   cudaStream_t s) {
  GatherArgs g = {};
  g.X = static_cast<const uint4*>(X);
  g.W = static_cast<const uint4*>(W);
  g.vecs = H / 8;
  g.targets = targets;
  g.rows_all = rows;
  g.V = V;
  g.ignore_index = ignore_index;
  g.dloss = dloss;
  g.lse_in = lse_in;
  g.in_unit = std::is_same<T, __half>::value ? 32768.0f : 1.0f;
  g.meta = reinterpret_cast<Meta*>(ws + w.meta);
  g.n_tiles = ceil_div(H, TILE);
  g.k_stages = w.piece / GK;
  g.most_splits = w.most_splits;
  g.part_tiles = w.part_tiles;
  g.pairs = device_pairs();
  g.inv = reinterpret_cast<int*>(ws + w.inv);
  g.row_of = reinterpret_cast<int*>(ws + w.row_of);
  g.Xc = reinterpret_cast<uint4*>(ws + w.xc);
  g.ctarget = reinterpret_cast<int*>(ws + w.ctarget);
  g.ctsum = reinterpret_cast<float*>(ws + w.tsum);
  g.clse = reinterpret_cast<float*>(ws + w.clse);
  g.cscale = reinterpret_cast<float*>(ws + w.cscale);
  g.loss = loss;
  g.lse = lse;
  g.dX = static_cast<uint4*>(dX);
  g.dev_err = dev_err;
  if (rows <= 2048)
    return launch_pdl(ce_gather_few_kernel<T>, dim3(w.rows_pad), dim3(256), 0, s, g);
  // each block reads all targets: more rows per block once the targets are many
  const int per = rows <= 8192 ? 8 : 64;
  return launch_pdl(ce_gather_kernel<T>, dim3(w.rows_pad / per), dim3(256), 0, s, g, per);
}

template <typename T>
cudaError_t forward(const void* X, const void* W, const int* targets, int rows, int H, int V,
                    int ignore_index, float* loss, float* lse, char* ws, int32_t* dev_err,
                    cudaStream_t s) {
  const Space w = space_of(rows, H, V, false);
  cudaError_t e = gather<T>(w, ws, X, W, targets, rows, H, V, ignore_index, nullptr, nullptr,
                            loss, lse, nullptr, dev_err, s);
  if (e) return e;
  Meta* meta = reinterpret_cast<Meta*>(ws + w.meta);
  float2* stats = reinterpret_cast<float2*>(ws + w.stats);
  const float* tsum = reinterpret_cast<const float*>(ws + w.tsum);
  const int* ctarget = reinterpret_cast<const int*>(ws + w.ctarget);
  const int* row_of = reinterpret_cast<const int*>(ws + w.row_of);
  if (w.skinny) {
    SkinnyArgs a = {};
    a.M = rows;
    a.live = &meta->rows;
    a.early = 1;
    a.stats = stats;
    a.arrived = meta->arrived;
    a.target_sum = tsum;
    a.targets = ctarget;
    a.row_of = row_of;
    a.loss = loss;
    a.lse_out = lse;
    a.dev_err = dev_err;
    return launch_skinny<T, false, S_STATS>({W, V, H, H}, ws + w.xc, H, w.rows_pad, a, s);
  }
  GemmArgs p = {};
  p.N = V;
  p.M = rows;
  p.m_tiles = w.rows_pad / TILE;
  p.n_tiles = ceil_div(V, TILE);
  p.k_stages = p.kps = ceil_div(H, GK);
  p.splits = 1;
  p.rows = &meta->rows;
  p.dyn = 1;
  p.stats = stats;
  p.target_sum = tsum;
  p.targets = ctarget;
  p.rows_pad = w.rows_pad;
  p.dev_err = dev_err;
  CUtensorMap am, bm;
  if (!map_2d<T>(&am, ws + w.xc, w.rows_pad, H, H, CM) || !map_2d<T>(&bm, W, V, H, H, CM))
    return cudaErrorInvalidValue;
  e = launch_gemm_maps<T, false, false, E_STATS, 256>(am, bm, am, am, p, s);
  if (e) return e;
  return launch_pdl(ce_join_kernel, dim3(w.rows_pad / 32), dim3(32 * kJoinWarps), 0, s,
                    static_cast<const float2*>(stats), 2 * ceil_div(V, TILE), w.rows_pad, tsum,
                    static_cast<const Meta*>(meta), row_of, loss, lse);
}

// Rows [v0, v0 + vn) of dW = dl^T X, from the first `reach` rows of dl.
template <typename T>
cudaError_t head_gradient(const Space& w, char* ws, int v0, int vn, int reach, int H, void* dW,
                          int32_t* dev_err, cudaStream_t s) {
  const Meta* meta = reinterpret_cast<const Meta*>(ws + w.meta);
  GemmArgs q = {};
  q.N = H;
  q.M = vn;
  q.m_tiles = ceil_div(vn, TILE);
  q.n_tiles = ceil_div(H, TILE);
  q.k_stages = q.kps = ceil_div(reach, GK);
  q.splits = 1;
  q.rows = &meta->rows;
  q.dyn = 2;
  q.scale = &meta->out_scale;
  q.dev_err = dev_err;
  CUtensorMap om;
  if (!map_2d<T>(&om, static_cast<char*>(dW) + (size_t)v0 * H * 2, vn, H, H, 32))
    return cudaErrorInvalidValue;
  return launch_gemm<T, true, true, E_STORE, 256>({ws + w.dl, vn, reach, w.piece},
                                                  {ws + w.xc, H, w.rows_pad, H}, om, om, q, s);
}

template <typename T>
cudaError_t backward(const float* dloss, const void* X, const void* W, const int* targets,
                     const float* lse, int rows, int H, int V, int ignore_index, void* dX,
                     void* dW, char* ws, int32_t* dev_err, cudaStream_t s) {
  const Space w = space_of(rows, H, V, true);
  cudaError_t e = gather<T>(w, ws, X, W, targets, rows, H, V, ignore_index, dloss, lse, nullptr,
                            nullptr, w.skinny ? dX : nullptr, dev_err, s);
  if (e) return e;
  const Meta* meta = reinterpret_cast<const Meta*>(ws + w.meta);
  if (w.skinny) {
    SkinnyArgs a = {};
    a.M = rows;
    a.live = &meta->rows;
    a.early = 1;
    a.dev_err = dev_err;
    a.out = ws + w.dl;
    a.ld = w.piece;
    a.targets = reinterpret_cast<const int*>(ws + w.ctarget);
    a.lse = reinterpret_cast<const float*>(ws + w.clse);
    a.row_scale = reinterpret_cast<const float*>(ws + w.cscale);
    a.target_sum = reinterpret_cast<const float*>(ws + w.tsum);
    e = launch_skinny<T, false, S_DLOGITS>({W, V, H, H}, ws + w.xc, H, w.rows_pad, a, s);
    if (e) return e;
    if (dX) {
      a.out = dX;
      a.scale = &meta->out_scale;
      a.row_of = reinterpret_cast<const int*>(ws + w.row_of);
      a.part = reinterpret_cast<float*>(ws + w.part);
      e = launch_skinny<T, true, S_STORE>({W, H, V, H}, ws + w.dl, w.piece, w.rows_pad, a, s);
      if (e) return e;
    }
    // dl has the rows that the product's tokens fill; behind them nothing is read
    return dW ? head_gradient<T>(w, ws, 0, V, (rows + 31) / 32 * 32, H, dW, dev_err, s)
              : cudaSuccess;
  }
  const int mt = w.rows_pad / TILE, ht = ceil_div(H, TILE);
  char* dl = ws + w.dl;
  float* part = reinterpret_cast<float*>(ws + w.part);
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
    p.target_sum = reinterpret_cast<const float*>(ws + w.tsum);
    p.col0 = v0;
    p.rows_pad = w.rows_pad;
    p.dev_err = dev_err;
    CUtensorMap lm;
    if (!map_2d<T>(&lm, dl, w.rows_pad, vn, w.piece, 32)) return cudaErrorInvalidValue;
    e = launch_gemm<T, false, false, E_DLOGITS, 256>({ws + w.xc, w.rows_pad, H, H},
                                                     {Wi, vn, H, H}, lm, lm, p, s);
    if (e) return e;
    if (dX) {
      GemmArgs q = {};
      q.N = H;
      q.M = rows;
      q.m_tiles = mt;
      q.n_tiles = ht;
      // every piece adds to the same splits' sums, so all run as many stages:
      // a shorter last piece reads zeros behind its end
      q.k_stages = w.piece / GK;
      q.splits = w.most_splits;
      q.splits_of = &meta->splits;
      q.rows = &meta->rows;
      q.dyn = 1;
      q.part = part;
      q.accumulate = i > 0;
      q.dev_err = dev_err;
      e = launch_gemm<T, false, true, E_PART, 256>({dl, w.rows_pad, vn, w.piece},
                                                   {Wi, H, vn, H}, lm, lm, q, s);
      if (e) return e;
    }
    if (dW) {
      e = head_gradient<T>(w, ws, v0, vn, w.rows_pad, H, dW, dev_err, s);
      if (e) return e;
    }
  }
  if (!dX) return cudaSuccess;
  FinishArgs f = {};
  f.part = part;
  f.splits_of = &meta->splits;
  f.n_tiles = ht;
  f.rows = &meta->rows;
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
