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
// Backward: four launches, the first fusing the whole activation backward
// (and h again, for dW_d) into the epilogue of dY Wd.
#include "ffn_gemv.cuh"

namespace moe {
namespace {

using namespace dense;

// At most this many tiles of partial sums (256 KB each) in a workspace.
constexpr int kPartTiles = 148;

int splits_for(int tiles, int64_t K) {
  return pick_splits(tiles, ceil_div(K, GK), std::max(1, kPartTiles / std::max(1, tiles)), false);
}
size_t part_bytes(int tiles, int64_t K) {
  const int sp = splits_for(tiles, K);
  return sp == 1 ? 0 : (size_t)sp * tiles * TILE_FLOATS * 4;
}
size_t align1k(size_t b) { return (b + 1023) & ~(size_t)1023; }

void plan(GemmArgs& a, int m_tiles, int n_tiles, int64_t K, int splits) {
  a.m_tiles = m_tiles;
  a.n_tiles = n_tiles;
  a.k_stages = ceil_div(K, GK);
  a.kps = ceil_div(a.k_stages, splits);
  a.splits = ceil_div(a.k_stages, a.kps);
}

// D [M, N] (16 bits) = A B^T (+ residual), split along k where the tiles alone
// leave SMs idle.
template <typename T, bool AMN, bool BMN>
cudaError_t product(const Operand& a, const Operand& b, void* d, const float* residual, float* part,
                    int32_t* dev_err, cudaStream_t s) {
  const int mt = ceil_div(a.rows, TILE), nt = ceil_div(b.rows, TILE);
  GemmArgs p = {};
  p.N = (int)b.rows;
  p.M = (int)a.rows;
  p.dev_err = dev_err;
  plan(p, mt, nt, a.k, splits_for(mt * nt, a.k));
  CUtensorMap dm;
  if (!map_2d<T>(&dm, d, a.rows, b.rows, b.rows, 32)) return cudaErrorInvalidValue;
  if (p.splits == 1) {
    p.residual = residual;
    return launch_gemm<T, AMN, BMN, E_STORE>(a, b, dm, dm, p, s);
  }
  p.part = part;
  if (cudaError_t e = launch_gemm<T, AMN, BMN, E_PART>(a, b, dm, dm, p, s)) return e;
  FinishArgs f = {};
  f.part = part;
  f.splits = p.splits;
  f.n_tiles = nt;
  f.split_stride = (size_t)mt * nt * TILE_FLOATS;
  f.M = p.M;
  f.N = p.N;
  f.residual = residual;
  f.out = d;
  f.dev_err = dev_err;
  return launch_finish<T, F_PLAIN>(f, s);
}

// Map of [T][2][I] (gate | up rows), boxes of 64 columns x 1 x 32 rows.
template <typename T>
bool gate_up_map(CUtensorMap* m, const void* p, int64_t rows, int64_t I) {
  return map_3d<T>(m, p, {I, 2, rows}, {I, 2 * I}, {64, 1, 32});
}

template <typename T>
cudaError_t forward(const void* X, const void* W_gu, const void* W_d, int M, int H, int I,
                    const float* residual, void* Y, void* gu, void* ws, int32_t* dev_err,
                    cudaStream_t s) {
  void* h = ws;
  if (M <= 8)
    return launch_ffn_gemv<T, 1>(X, W_gu, W_d, M, H, I, residual, Y, gu, h, dev_err, s);
  if (M <= kGemvRows)
    return launch_ffn_gemv<T, 2>(X, W_gu, W_d, M, H, I, residual, Y, gu, h, dev_err, s);
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + align1k((size_t)M * I * 2));
  const int mt = ceil_div(M, TILE), nt = ceil_div(I, TILE / 2);
  GemmArgs p = {};
  p.N = I;
  p.M = M;
  p.dev_err = dev_err;
  p.save = gu != nullptr;
  plan(p, mt, nt, H, splits_for(mt * nt, H));
  CUtensorMap am, bm, hm, gm;
  // W_gu as [2][I][H]: box = 64 k x 128 rows of one half
  if (!map_2d<T>(&am, X, M, H, H, CM) ||
      !map_3d<T>(&bm, W_gu, {H, I, 2}, {H, (int64_t)I * H}, {64, CM, 1}) ||
      !map_2d<T>(&hm, h, M, I, I, 32))
    return cudaErrorInvalidValue;
  gm = hm;
  if (gu && !gate_up_map<T>(&gm, gu, M, I)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (p.splits == 1) {
    e = launch_gemm_maps<T, false, false, E_SWIGLU>(am, bm, hm, gm, p, s);
  } else {
    p.part = part;
    p.gate_up = 1;
    e = launch_gemm_maps<T, false, false, E_PART>(am, bm, hm, hm, p, s);
    if (e) return e;
    FinishArgs f = {};
    f.part = part;
    f.splits = p.splits;
    f.n_tiles = nt;
    f.split_stride = (size_t)mt * nt * TILE_FLOATS;
    f.M = M;
    f.N = I;
    f.out = h;
    f.out1 = gu;
    f.dev_err = dev_err;
    e = launch_finish<T, F_SWIGLU>(f, s);
  }
  if (e) return e;
  return product<T, false, false>({h, M, I, I}, {W_d, H, I, I}, Y, residual, part, dev_err, s);
}

template <typename T>
cudaError_t backward(const void* dY, const void* X, const void* gu, const void* W_gu,
                     const void* W_d, int M, int H, int I, void* dX, void* dW_gu, void* dW_d,
                     void* ws, int32_t* dev_err, cudaStream_t s) {
  char* w = static_cast<char*>(ws);
  void* h = w;
  void* dgu = w + align1k((size_t)M * I * 2);
  float* part = reinterpret_cast<float*>(static_cast<char*>(dgu) + align1k((size_t)M * 2 * I * 2));
  const int mt = ceil_div(M, TILE), nt = ceil_div(I, TILE);
  GemmArgs p = {};
  p.N = I;
  p.M = M;
  p.dev_err = dev_err;
  p.gu = gu;
  plan(p, mt, nt, H, splits_for(mt * nt, H));
  const Operand a = {dY, M, H, H}, b = {W_d, I, H, I};  // b: column i of W_d [H, I]
  CUtensorMap hm, gm;
  if (!map_2d<T>(&hm, h, M, I, I, 32) || !gate_up_map<T>(&gm, dgu, M, I))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if (p.splits == 1) {
    e = launch_gemm<T, false, true, E_SWIGLU_BWD>(a, b, hm, gm, p, s);
  } else {
    p.part = part;
    e = launch_gemm<T, false, true, E_PART>(a, b, hm, hm, p, s);
    if (e) return e;
    FinishArgs f = {};
    f.part = part;
    f.splits = p.splits;
    f.n_tiles = nt;
    f.split_stride = (size_t)mt * nt * TILE_FLOATS;
    f.M = M;
    f.N = I;
    f.gu = gu;
    f.out = h;
    f.out1 = dgu;
    f.dev_err = dev_err;
    e = launch_finish<T, F_SWIGLU_BWD>(f, s);
  }
  if (e) return e;
  const int64_t I2 = 2 * (int64_t)I;
  if (dX) {
    e = product<T, false, true>({dgu, M, I2, I2}, {W_gu, H, I2, H}, dX, nullptr, part, dev_err, s);
    if (e) return e;
  }
  if (dW_gu) {
    e = product<T, true, true>({dgu, I2, M, I2}, {X, H, M, H}, dW_gu, nullptr, part, dev_err, s);
    if (e) return e;
  }
  if (dW_d) {
    e = product<T, true, true>({dY, H, M, H}, {h, I, M, I}, dW_d, nullptr, part, dev_err, s);
    if (e) return e;
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace moe

namespace moe_launch {
using namespace moe;

size_t gated_ffn_forward_workspace(int M, int H, int I) {
  const int mt = ceil_div(M, TILE);
  if (M <= kGemvRows) return align1k((size_t)M * I * 2);
  return align1k((size_t)M * I * 2) + std::max(part_bytes(mt * ceil_div(I, TILE / 2), H),
                                               part_bytes(mt * ceil_div(H, TILE), I));
}
size_t gated_ffn_backward_workspace(int M, int H, int I) {
  const int mt = ceil_div(M, TILE), ht = ceil_div(H, TILE), it = ceil_div(I, TILE);
  const int64_t I2 = 2 * (int64_t)I;
  const size_t part = std::max(std::max(part_bytes(mt * it, H), part_bytes(mt * ht, I2)),
                               std::max(part_bytes(ceil_div(I2, TILE) * ht, M),
                                        part_bytes(ht * it, M)));
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
