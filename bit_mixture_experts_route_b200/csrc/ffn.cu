// Dense gated feed-forward block in 16 bits, the expert that runs beside the
// routed 4-bit ones:
//   g = X Wg^T, u = X Wu^T, h = silu(g) u, Y = h Wd^T (+ residual)
// and its backward pass
//   dh = dY Wd, s = sigmoid(g), dg = dh u s (1 + g (1 - s)), du = dh g s,
//   dX = [dg | du] W_gu, dW_gu = [dg | du]^T X, dW_d = dY^T h.
// Forward: one launch computes both projections, the activation and the
// product (gate rows are one CTA's half of the tile, up rows the other's, so
// column j of both is in the same thread); h is rounded once to 16 bits, as the
// MMA's operand must be, and the down projection is the second launch.
// Backward: three launches, the first fusing the whole activation backward
// (and h again, for dW_d) into the epilogue of dY Wd; both weight gradients are
// one list of tiles.  Where tiles alone leave SMs idle a product is split along k
// and one more launch joins it.
// Measured (bf16, 4096 tokens, 2048 x 8192): forward 343 us = 1.20 PFLOP/s,
// backward 721 us = 1.14, under the power cap; a library GEMM sustains 1.39.
#include "ffn_gemv.cuh"
#include "skinny_gemm.cuh"

namespace moe {
namespace {

using namespace dense;

// At most this many tiles of partial sums (256 KB each) in a workspace.
constexpr int kPartTiles = 148;

Plan plan_of(int64_t rows, int64_t cols, int64_t K) {
  return plan_product(rows, cols, ceil_div(K, GK), kPartTiles);
}
// dY W_d: the activation backward takes about 12 us per 256 columns.
Plan plan_dh(int M, int H, int I) {
  return plan_product(M, I, ceil_div(H, GK), kPartTiles, 0.048);
}
size_t part_bytes(int64_t rows, int64_t cols, const Plan& pl) {
  return pl.splits == 1
             ? 0
             : (size_t)pl.splits * ceil_div(rows, TILE) * ceil_div(cols, TILE) * TILE_FLOATS * 4;
}
size_t part_bytes(int64_t rows, int64_t cols, int64_t K) {
  return part_bytes(rows, cols, plan_of(rows, cols, K));
}

void set_plan(GemmArgs& a, int64_t rows, int64_t cols, int64_t K, Plan pl) {
  a.m_tiles = ceil_div(rows, TILE);
  a.n_tiles = ceil_div(cols, pl.tn);
  a.k_stages = ceil_div(K, GK);
  a.kps = ceil_div(a.k_stages, pl.splits);
  a.splits = pl.splits;
}

FinishArgs finish_of(const GemmArgs& p, int32_t* dev_err) {
  FinishArgs f = {};
  f.part = p.part;
  f.splits = p.splits;
  f.n_tiles = p.n_tiles;
  f.split_stride = (size_t)p.m_tiles * p.n_tiles * TILE_FLOATS;
  f.M = p.M;
  f.N = p.N;
  f.dev_err = dev_err;
  return f;
}

// D [M, N] (16 bits) = A B^T (+ residual); narrower tiles, or splits along k,
// where 256-column tiles alone leave SMs idle.  early: nothing in the call
// writes b.
template <typename T, bool AMN, bool BMN>
cudaError_t product(const Operand& a, const Operand& b, void* d, const float* residual, float* part,
                    bool early, int32_t* dev_err, cudaStream_t s) {
  const Plan pl = plan_of(a.rows, b.rows, a.k);
  GemmArgs p = {};
  p.N = (int)b.rows;
  p.M = (int)a.rows;
  p.early = early;
  p.dev_err = dev_err;
  set_plan(p, a.rows, b.rows, a.k, pl);
  CUtensorMap dm;
  if (!map_2d<T>(&dm, d, a.rows, b.rows, b.rows, 32)) return cudaErrorInvalidValue;
  if (pl.splits == 1) {
    p.residual = residual;
    if (pl.tn == 128) return launch_gemm<T, AMN, BMN, E_STORE, 128>(a, b, dm, dm, p, s);
    return launch_gemm<T, AMN, BMN, E_STORE, 256>(a, b, dm, dm, p, s);
  }
  p.part = part;
  if (cudaError_t e = launch_gemm<T, AMN, BMN, E_PART, 256>(a, b, dm, dm, p, s)) return e;
  FinishArgs f = finish_of(p, dev_err);
  f.residual = residual;
  f.out = d;
  return launch_finish<T, F_PLAIN>(f, s);
}

// Map of [T][2][I] (gate | up rows), boxes of `cols` columns x 1 x 32 rows.
template <typename T>
bool gate_up_map(CUtensorMap* m, const void* p, int64_t rows, int64_t I, int cols) {
  return map_3d<T>(m, p, {I, 2, rows}, {I, 2 * I}, {cols, 1, 32});
}

template <typename T>
cudaError_t forward(const void* X, const void* W_gu, const void* W_d, int M, int H, int I,
                    const float* residual, void* Y, void* gu, void* ws, int32_t* dev_err,
                    cudaStream_t s) {
  void* h = ws;
  if (use_gemv(M, H, I))
    return launch_ffn_gemv<T>(X, W_gu, W_d, M, H, I, residual, Y, gu, h, dev_err, s);
  if (M <= kSkinnyRows) {
    SkinnyArgs a = {};
    a.M = M;
    a.dev_err = dev_err;
    a.out = h;
    a.out1 = gu;
    cudaError_t e = launch_skinny<T, false, S_SWIGLU>({W_gu, I, H, H}, X, H, M, a, s);
    if (e) return e;
    a.early = 1;
    a.out = Y;
    a.residual = residual;
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + align1k((size_t)M * I * 2));
    return launch_skinny<T, false, S_STORE>({W_d, H, I, I}, h, I, M, a, s);
  }
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + align1k((size_t)M * I * 2));
  const Plan pl = plan_of(M, 2 * (int64_t)I, H);
  GemmArgs p = {};
  p.N = I;
  p.M = M;
  p.dev_err = dev_err;
  p.save = gu != nullptr;
  set_plan(p, M, 2 * (int64_t)I, H, pl);
  p.n_tiles = ceil_div(I, pl.tn / 2);
  CUtensorMap am, bm, hm, gm;
  // W_gu as [2][I][H]: box = 64 k x half a tile's rows of gate or of up
  if (!map_2d<T>(&am, X, M, H, H, CM) ||
      !map_3d<T>(&bm, W_gu, {H, I, 2}, {H, (int64_t)I * H}, {64, pl.tn / 2, 1}) ||
      !map_2d<T>(&hm, h, M, I, I, 32))
    return cudaErrorInvalidValue;
  gm = hm;
  if (gu && !gate_up_map<T>(&gm, gu, M, I, 64)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (pl.splits > 1) {
    p.part = part;
    p.gate_up = 1;
    e = launch_gemm_maps<T, false, false, E_PART, 256>(am, bm, hm, hm, p, s);
    if (e) return e;
    FinishArgs f = finish_of(p, dev_err);
    f.out = h;
    f.out1 = gu;
    e = launch_finish<T, F_SWIGLU>(f, s);
  } else if (pl.tn == 128) {
    e = launch_gemm_maps<T, false, false, E_SWIGLU, 128>(am, bm, hm, gm, p, s);
  } else {
    e = launch_gemm_maps<T, false, false, E_SWIGLU, 256>(am, bm, hm, gm, p, s);
  }
  if (e) return e;
  return product<T, false, false>({h, M, I, I}, {W_d, H, I, I}, Y, residual, part, true, dev_err,
                                  s);
}

template <typename T, int TN>
cudaError_t both_gradients(const void* dY, const void* X, const void* h, const void* dgu, int M,
                           int H, int I, void* dW_gu, void* dW_d, int32_t* dev_err,
                           cudaStream_t s) {
  const int64_t I2 = 2 * (int64_t)I;
  GemmArgs p = {};
  p.N = H;
  p.M = (int)I2;
  p.early = 1;
  p.dev_err = dev_err;
  set_plan(p, I2, H, M, {TN, 1});
  SecondProduct q = {};
  q.N = I;
  q.M = H;
  q.m_tiles = ceil_div(H, TILE);
  q.n_tiles = ceil_div(I, TN);
  CUtensorMap am, bm, dm;
  if (!operand_map<T, true>(&am, {dgu, I2, M, I2}, CM) ||
      !operand_map<T, true>(&bm, {X, H, M, H}, CM) || !map_2d<T>(&dm, dW_gu, I2, H, H, 32) ||
      !operand_map<T, true>(&q.a, {dY, H, M, H}, CM) ||
      !operand_map<T, true>(&q.b, {h, I, M, I}, CM) || !map_2d<T>(&q.d, dW_d, H, I, I, 32))
    return cudaErrorInvalidValue;
  return launch_gemm_maps<T, true, true, E_STORE2, TN>(am, bm, dm, dm, p, s, q);
}

// dW_gu = dgu^T X, dW_d = dY^T h; either may be null.
template <typename T>
cudaError_t weight_gradients(const void* dY, const void* X, const void* h, const void* dgu, int M,
                             int H, int I, void* dW_gu, void* dW_d, float* part, int32_t* dev_err,
                             cudaStream_t s) {
  const int64_t I2 = 2 * (int64_t)I;
  cudaError_t e;
  if (dW_gu && dW_d && plan_of(I2, H, M).splits == 1 && plan_of(H, I, M).splits == 1) {
    // both in one launch: their tiles share the rounds, and a launch's start and
    // end cost about 5 us
    auto tiles = [&](int tn) {
      return ceil_div(I2, TILE) * ceil_div(H, tn) + ceil_div(H, TILE) * ceil_div(I, tn);
    };
    // tiles of 128 columns where one round takes them all
    if (tiles(128) <= device_pairs())
      return both_gradients<T, 128>(dY, X, h, dgu, M, H, I, dW_gu, dW_d, dev_err, s);
    return both_gradients<T, 256>(dY, X, h, dgu, M, H, I, dW_gu, dW_d, dev_err, s);
  }
  if (dW_gu) {
    e = product<T, true, true>({dgu, I2, M, I2}, {X, H, M, H}, dW_gu, nullptr, part, true,
                               dev_err, s);
    if (e) return e;
  }
  if (dW_d) {
    e = product<T, true, true>({dY, H, M, H}, {h, I, M, I}, dW_d, nullptr, part, false,
                               dev_err, s);
    if (e) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t backward(const void* dY, const void* X, const void* gu, const void* W_gu,
                     const void* W_d, int M, int H, int I, void* dX, void* dW_gu, void* dW_d,
                     void* ws, int32_t* dev_err, cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  void* h = w;
  void* dgu = w + align1k((size_t)M * I * 2);
  float* part = reinterpret_cast<float*>(static_cast<char*>(dgu) + align1k((size_t)M * 2 * I * 2));
  const int64_t I2 = 2 * (int64_t)I;
  cudaError_t e;
  if (M <= kSkinnyRows) {
    SkinnyArgs a = {};
    a.M = M;
    a.dev_err = dev_err;
    a.gu = gu;
    a.out = dW_d ? h : nullptr;
    a.out1 = dgu;
    e = launch_skinny<T, true, S_SWIGLU_BWD>({W_d, I, H, I}, dY, H, M, a, s);
    if (e) return e;
    if (dX) {
      a.early = 1;
      a.out = dX;
      a.part = part;
      e = launch_skinny<T, true, S_STORE>({W_gu, H, I2, H}, dgu, I2, M, a, s);
      if (e) return e;
    }
    return weight_gradients<T>(dY, X, h, dgu, M, H, I, dW_gu, dW_d, part, dev_err, s);
  }
  const Plan pl = plan_dh(M, H, I);
  GemmArgs p = {};
  p.N = I;
  p.M = M;
  p.dev_err = dev_err;
  p.gu = gu;
  p.save = dW_d != nullptr;  // h is dW_d's operand only
  set_plan(p, M, I, H, pl);
  const Operand a = {dY, M, H, H}, b = {W_d, I, H, I};  // b: column i of W_d [H, I]
  CUtensorMap hm, gm;
  if (!map_2d<T>(&hm, h, M, I, I, 32, 32) || !gate_up_map<T>(&gm, dgu, M, I, 32))
    return cudaErrorInvalidValue;
  if (pl.splits > 1) {
    p.part = part;
    e = launch_gemm<T, false, true, E_PART, 256>(a, b, hm, hm, p, s);
    if (e) return e;
    FinishArgs f = finish_of(p, dev_err);
    f.gu = gu;
    f.out = dW_d ? h : nullptr;
    f.out1 = dgu;
    e = launch_finish<T, F_SWIGLU_BWD>(f, s);
  } else if (pl.tn == 128) {
    e = launch_gemm<T, false, true, E_SWIGLU_BWD, 128>(a, b, hm, gm, p, s);
  } else {
    e = launch_gemm<T, false, true, E_SWIGLU_BWD, 256>(a, b, hm, gm, p, s);
  }
  if (e) return e;
  if (dX) {
    e = product<T, false, true>({dgu, M, I2, I2}, {W_gu, H, I2, H}, dX, nullptr, part, true,
                                dev_err, s);
    if (e) return e;
  }
  return weight_gradients<T>(dY, X, h, dgu, M, H, I, dW_gu, dW_d, part, dev_err, s);
}

}  // namespace
}  // namespace moe

namespace moe_launch {
using namespace moe;

size_t gated_ffn_forward_workspace(int M, int H, int I) {
  const size_t h = align1k((size_t)M * I * 2);
  if (use_gemv(M, H, I)) return h;
  if (M <= kSkinnyRows) return h + skinny_part_bytes(M, H, I);
  return h + std::max(part_bytes(M, 2 * (int64_t)I, H), part_bytes(M, H, I));
}
size_t gated_ffn_backward_workspace(int M, int H, int I) {
  const int64_t I2 = 2 * (int64_t)I;
  const size_t part =
      std::max(std::max(part_bytes(I2, H, M), part_bytes(H, I, M)),
               M <= kSkinnyRows
                   ? skinny_part_bytes(M, H, I2)
                   : std::max(part_bytes(M, I, plan_dh(M, H, I)), part_bytes(M, H, I2)));
  return align1k((size_t)M * I * 2) + align1k((size_t)M * I * 4) + part;
}

cudaError_t gated_ffn_forward(const void* X, moe_dtype_t dt, const void* W_gu, const void* W_d,
                              int M, int H, int I, const float* residual, void* Y, void* gu,
                              void* ws, int32_t* dev_err, cudaStream_t s) {
  if (dt == MOE_DT_F16)
    return forward<__half>(X, W_gu, W_d, M, H, I, residual, Y, gu, ws, dev_err, s);
  return forward<__nv_bfloat16>(X, W_gu, W_d, M, H, I, residual, Y, gu, ws, dev_err, s);
}

cudaError_t gated_ffn_backward(const void* dY, moe_dtype_t dt, const void* X, const void* gu,
                               const void* W_gu, const void* W_d, int M, int H, int I, void* dX,
                               void* dW_gu, void* dW_d, void* ws, int32_t* dev_err,
                               cudaStream_t s) {
  if (dt == MOE_DT_F16)
    return backward<__half>(dY, X, gu, W_gu, W_d, M, H, I, dX, dW_gu, dW_d, ws, dev_err, s);
  return backward<__nv_bfloat16>(dY, X, gu, W_gu, W_d, M, H, I, dX, dW_gu, dW_d, ws, dev_err, s);
}

}  // namespace moe_launch
