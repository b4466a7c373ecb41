// The gradient of the root-mean-square norm of rows.  With u = dy gamma and
// n = h rstd,
//   dres = dh + rstd (u - n mean(u n)),   dx = dropout's gradient of dres,
//   dgamma = sum over the rows of dy n.
// A CTA goes over many rows and keeps its columns' share of dgamma in registers, so
// the rows are read once; the CTAs' shares go to the workspace and a second small
// kernel adds them in a fixed order.
#include "rmsnorm.cuh"

namespace fr {
namespace {

template <bool F32>
__device__ __forceinline__ const char *row_of(const void *p, int64_t row, int64_t ld) {
  return static_cast<const char *>(p) + row * ld * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ char *row_of(void *p, int64_t row, int64_t ld) {
  return static_cast<char *>(p) + row * ld * (F32 ? 4 : 2);
}

// The gradients of a lane's elements of a chunk and their share of dgamma, given
// the row's mean(u n); n and u are formed again from h and dy.
template <bool F32, bool VEC>
__device__ __forceinline__ void chunk_grad(const NormBackward &a, const Mask &mask, int64_t row,
                                           int c, int lane, const Lane8<F32> &dy,
                                           const Lane8<F32> &h, const Lane8<F32> &dh,
                                           const float (&g)[8], float rstd, float mean,
                                           float (&acc)[8]) {
  const int cols = static_cast<int>(a.cols);
  float d[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float n = h.at(j) * rstd;
    acc[j] = fmaf(dy.at(j), n, acc[j]);
    d[j] = rstd * fmaf(-n, mean, dy.at(j) * g[j]);
    if (a.dh != nullptr) d[j] += dh.at(j);
  }
  Lane8<F32> out;
  if (a.drop.rng != nullptr) {
    if (a.dres != nullptr) {
      out.set(d);
      store8<F32, VEC>(row_of<F32>(a.dres, row, a.ld_dres), c, lane, cols, out);
    }
    drop8<VEC>(d, mask, static_cast<uint32_t>(row), c, lane);
  }
  out.set(d);
  store8<F32, VEC>(row_of<F32>(a.dx, row, a.ld_dx), c, lane, cols, out);
}

template <bool F32>
__device__ __forceinline__ float chunk_dot(const Lane8<F32> &dy, const Lane8<F32> &h,
                                           const float (&g)[8]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(dy.at(j) * g[j], h.at(j), s);
  return s;
}

template <bool VEC>
__device__ __forceinline__ void store_cols8(float *p, int c, int lane, int cols,
                                            const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int col = lane_col<VEC>(c, lane, j);
    if (col < cols) p[col] = v[j];
  }
}

// Persistent form: blockDim = (32 W, R), R rows at a time, W warps a row, NU chunks a
// warp; a CTA takes every gridDim.x-th group of R rows.
template <bool F32, bool VEC, int NU>
__global__ void __launch_bounds__(512) rmsnorm_grad_held(NormBackward a) {
  pdl_enter();
  __shared__ float red[2][16];
  extern __shared__ float sums[];  // R > 1: the CTA's share of dgamma
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int R = blockDim.y;
  const int cols = static_cast<int>(a.cols);
  const float over = 1.0f / static_cast<float>(cols);
  Mask mask{};
  if (a.drop.rng != nullptr) mask = mask_of(a.drop);
  float acc[NU][8];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * R; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * R, turn ^= 1) {
    const int64_t row = base + threadIdx.y;
    const bool live = row < a.rows;
    const char *dhr = row_of<F32>(a.dh, row, a.ld_dh);
    // dh is loaded ahead where there are registers for it
    constexpr bool EARLY = VEC && NU <= 2;
    Lane8<F32> dy[NU], h[NU], dh[EARLY ? NU : 1];
    float rstd = 0.0f, dot = 0.0f;
    if (live) {
      const char *dyr = row_of<F32>(a.dy, row, a.ld_dy), *hr = row_of<F32>(a.h, row, a.ld_h);
#pragma unroll
      for (int i = 0; i < NU; ++i) dy[i] = load8<F32, VEC>(dyr, i * W + warp, lane, cols);
#pragma unroll
      for (int i = 0; i < NU; ++i) h[i] = load8<F32, VEC>(hr, i * W + warp, lane, cols);
      if (EARLY && a.dh != nullptr) {
#pragma unroll
        for (int i = 0; i < NU; ++i) dh[i] = load8<F32, VEC>(dhr, i * W + warp, lane, cols);
      }
      rstd = ld_keep_f32(a.rstd + row);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float g[8];
        load_cols8<VEC>(g, a.gamma, i * W + warp, lane, cols);
        dot += chunk_dot<F32>(dy[i], h[i], g);
      }
    }
    dot = warp_sum(dot);
    if (W > 1) {  // the two halves of red in turn: one barrier a row
      if (lane == 0) red[turn][threadIdx.y * W + warp] = dot;
      __syncthreads();
      dot = warp_sum(lane < W ? red[turn][threadIdx.y * W + lane] : 0.0f);
    }
    if (!live) continue;
    const float mean = dot * over * rstd;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int c = i * W + warp;
      if (c * kChunk >= cols) continue;
      float g[8];
      load_cols8<VEC>(g, a.gamma, c, lane, cols);
      if (!EARLY && a.dh != nullptr) dh[0] = load8<F32, VEC>(dhr, c, lane, cols);
      chunk_grad<F32, VEC>(a, mask, row, c, lane, dy[i], h[i], dh[EARLY ? i : 0], g, rstd, mean,
                           acc[i]);
    }
  }
  if (a.dgamma == nullptr) return;
  float *part = static_cast<float *>(a.workspace) + static_cast<int64_t>(blockIdx.x) * cols;
  if (R == 1) {
#pragma unroll
    for (int i = 0; i < NU; ++i) store_cols8<VEC>(part, i * W + warp, lane, cols, acc[i]);
    return;
  }
  for (int y = 0; y < R; ++y) {
    __syncthreads();
    if (static_cast<int>(threadIdx.y) != y) continue;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = lane_col<VEC>(i * W + warp, lane, j);
        if (col < cols) sums[col] = y == 0 ? acc[i][j] : sums[col] + acc[i][j];
      }
    }
  }
  __syncthreads();
  for (int col = threadIdx.y * blockDim.x + threadIdx.x; col < cols; col += blockDim.x * R)
    part[col] = sums[col];
}

// Looped form, first kernel: sum(u h) of each row, a CTA a row.
constexpr int kLoopThreads = 512;
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kLoopThreads) rmsnorm_grad_dots(NormBackward a, float *dots) {
  pdl_enter();
  __shared__ float red[2][kLoopThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int W = kLoopThreads / 32;
  const int cols = static_cast<int>(a.cols);
  const int chunks = static_cast<int>((a.cols + kChunk - 1) / kChunk);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const char *dyr = row_of<F32>(a.dy, row, a.ld_dy), *hr = row_of<F32>(a.h, row, a.ld_h);
    float dot = 0.0f;
    for (int c = warp; c < chunks; c += W) {
      const Lane8<F32> dy = load8<F32, VEC, true>(dyr, c, lane, cols);
      const Lane8<F32> h = load8<F32, VEC, true>(hr, c, lane, cols);
      float g[8];
      load_cols8<VEC>(g, a.gamma, c, lane, cols);
      dot += chunk_dot<F32>(dy, h, g);
    }
    dot = warp_sum(dot);
    if (lane == 0) red[turn][warp] = dot;
    __syncthreads();
    if (warp == 0) {
      dot = warp_sum(lane < W ? red[turn][lane] : 0.0f);
      if (lane == 0) dots[row] = dot;
    }
  }
}

// Looped form, second kernel: a warp keeps a chunk of columns and goes over every
// gridDim.y-th row.
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) rmsnorm_grad_cols(NormBackward a, const float *dots,
                                                         float *partial) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int cols = static_cast<int>(a.cols);
  const int chunks = static_cast<int>((a.cols + kChunk - 1) / kChunk);
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (c >= chunks) return;
  const float over = 1.0f / static_cast<float>(cols);
  Mask mask{};
  if (a.drop.rng != nullptr) mask = mask_of(a.drop);
  float g[8], acc[8];
  load_cols8<VEC>(g, a.gamma, c, lane, cols);
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const Lane8<F32> dy = load8<F32, VEC>(row_of<F32>(a.dy, row, a.ld_dy), c, lane, cols);
    const Lane8<F32> h = load8<F32, VEC>(row_of<F32>(a.h, row, a.ld_h), c, lane, cols);
    Lane8<F32> dh{};
    if (a.dh != nullptr) dh = load8<F32, VEC>(row_of<F32>(a.dh, row, a.ld_dh), c, lane, cols);
    const float rstd = ld_keep_f32(a.rstd + row);
    const float mean = ld_keep_f32(dots + row) * over * rstd;
    chunk_grad<F32, VEC>(a, mask, row, c, lane, dy, h, dh, g, rstd, mean, acc);
  }
  if (a.dgamma != nullptr)
    store_cols8<VEC>(partial + static_cast<int64_t>(blockIdx.y) * cols, c, lane, cols, acc);
}

// dgamma: the sum of P shares of each column.  32 columns a CTA, 32 runs of shares.
__global__ void __launch_bounds__(1024) rmsnorm_grad_join(const float *partial, float *dgamma,
                                                          int P, int64_t cols) {
  pdl_enter();
  __shared__ float red[32][33];
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.0f;
  if (col < cols)
    for (int p = threadIdx.y; p < P; p += 32) s += ld_keep_f32(partial + p * cols + col);
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < cols) dgamma[out] = s;
}

// Shapes of the launches, which the workspace follows.
struct GradShape {
  int units, W, R;  // persistent
  int64_t grid;     // CTAs, or the looped form's runs of rows
};

GradShape held_shape(int64_t rows, int64_t cols, bool f32, int sm_count) {
  const int chunks = static_cast<int>((cols + kChunk - 1) / kChunk);
  GradShape g{};
  g.units = chunks <= 2 ? 1 : (chunks <= 32 || f32) ? 2 : 4;
  g.W = (chunks + g.units - 1) / g.units;
  g.R = g.W >= 8 ? 1 : 8 / g.W;
  const int64_t per = g.W * g.R >= 16 ? 1 : 2;
  const int64_t groups = (rows + g.R - 1) / g.R;
  g.grid = groups < sm_count * per ? groups : sm_count * per;
  return g;
}

GradShape looped_shape(int64_t rows, int64_t cols, int sm_count) {
  const int64_t blocks = ((cols + kChunk - 1) / kChunk + 7) / 8;
  GradShape g{};
  int64_t runs = (4 * static_cast<int64_t>(sm_count) + blocks - 1) / blocks;
  g.grid = rows < runs ? rows : runs;
  return g;
}

int64_t dots_bytes(int64_t rows) { return (rows * 4 + 15) / 16 * 16; }

template <bool F32, bool VEC>
cudaError_t launch_grad(const NormBackward &a, bool held, int sm_count, cudaStream_t s) {
  cudaError_t e;
  const float *partial = static_cast<const float *>(a.workspace);
  int64_t P;
  if (held) {
    const GradShape g = held_shape(a.rows, a.cols, F32, sm_count);
    const dim3 grid(static_cast<unsigned>(g.grid)), block(32 * g.W, g.R);
    const size_t smem = g.R > 1 ? a.cols * 4 : 0;
    if (g.units == 1) e = launch_k(rmsnorm_grad_held<F32, VEC, 1>, grid, block, smem, s, 0, a);
    else if (F32 || !VEC || g.units == 2) e = launch_k(rmsnorm_grad_held<F32, VEC, 2>, grid, block, smem, s, 0, a);
    else e = launch_k(rmsnorm_grad_held<false, true, 4>, grid, block, smem, s, 0, a);
    P = g.grid;
  } else {
    float *dots = static_cast<float *>(a.workspace);
    float *shares = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + dots_bytes(a.rows));
    const int64_t most = static_cast<int64_t>(sm_count) * 4;
    e = launch_k(rmsnorm_grad_dots<F32, VEC>, dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                 dim3(kLoopThreads), 0, s, 0, a, dots);
    if (e != cudaSuccess) return e;
    const GradShape g = looped_shape(a.rows, a.cols, sm_count);
    const unsigned blocks = static_cast<unsigned>(((a.cols + kChunk - 1) / kChunk + 7) / 8);
    e = launch_k(rmsnorm_grad_cols<F32, VEC>, dim3(blocks, static_cast<unsigned>(g.grid)), dim3(256), 0, s, 0,
                 a, dots, shares);
    partial = shares;
    P = g.grid;
  }
  if (e != cudaSuccess || a.dgamma == nullptr) return e;
  return launch_k(rmsnorm_grad_join, dim3(static_cast<unsigned>((a.cols + 31) / 32)), dim3(32, 32), 0, s, 0,
                  partial, a.dgamma, static_cast<int>(P), a.cols);
}

}  // namespace

bool rmsnorm_grad_held_ok(int64_t cols, bool f32, bool vec) {
  return cols <= kChunk * 16 * (!f32 && vec ? 4 : 2);
}

size_t rmsnorm_grad_workspace(int64_t rows, int64_t cols, bool f32, bool held, int sm_count) {
  if (held) return static_cast<size_t>(held_shape(rows, cols, f32, sm_count).grid * cols * 4);
  return static_cast<size_t>(dots_bytes(rows) + looped_shape(rows, cols, sm_count).grid * cols * 4);
}

cudaError_t launch_rmsnorm_backward(const NormBackward &a, bool f32, bool vec, bool held,
                                    int sm_count, cudaStream_t s) {
  if (f32) return vec ? launch_grad<true, true>(a, held, sm_count, s) : launch_grad<true, false>(a, held, sm_count, s);
  return vec ? launch_grad<false, true>(a, held, sm_count, s) : launch_grad<false, false>(a, held, sm_count, s);
}

}  // namespace fr
