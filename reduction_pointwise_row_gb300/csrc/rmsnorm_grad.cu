// The gradient of the root-mean-square norm of rows.  With u = dy gamma and
// n = h rstd,
//   dres = dh + rstd (u - n mean(u n)),   dx = dropout's gradient of dres,
//   dgamma = sum over the rows of dy n.
// A CTA goes over many rows and keeps its columns' share of dgamma in registers, so
// the rows are read once; the CTAs' shares go to the workspace and a second small
// kernel adds them in a fixed order.
#include <algorithm>

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

// The sum of u n over a lane's elements.
template <bool F32>
__device__ __forceinline__ float chunk_dot(const Lane8<F32> &dy, const Lane8<F32> &h,
                                           const float (&g)[8], float rstd) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(dy.at(j) * g[j], h.at(j) * rstd, s);
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

// Rows that the ring below does not take (out of phase, or with edges and long): element
// accesses.  blockDim = (32 W, R), R rows at a time, W warps a row, NU chunks a warp; a CTA
// takes every gridDim.x-th group of R rows.  dh is loaded when its turn comes: there are no
// registers for it before.
template <bool F32, int NU>
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
    Lane8<F32> dy[NU], h[NU];
    float rstd = 0.0f, dot = 0.0f;
    if (live) {
      const char *dyr = row_of<F32>(a.dy, row, a.ld_dy), *hr = row_of<F32>(a.h, row, a.ld_h);
#pragma unroll
      for (int i = 0; i < NU; ++i) dy[i] = load8<F32, false>(dyr, i * W + warp, lane, cols);
#pragma unroll
      for (int i = 0; i < NU; ++i) h[i] = load8<F32, false>(hr, i * W + warp, lane, cols);
      rstd = ld_keep_f32(a.rstd + row);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        float g[8];
        load_cols8<false>(g, a.gamma, i * W + warp, lane, cols);
        dot += chunk_dot<F32>(dy[i], h[i], g, rstd);
      }
    }
    dot = warp_sum(dot);
    if (W > 1) {  // the two halves of red in turn: one barrier a row
      if (lane == 0) red[turn][threadIdx.y * W + warp] = dot;
      __syncthreads();
      dot = warp_sum(lane < W ? red[turn][threadIdx.y * W + lane] : 0.0f);
    }
    if (!live) continue;
    const float mean = dot * over;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int c = i * W + warp;
      if (c * kChunk >= cols) continue;
      float g[8];
      load_cols8<false>(g, a.gamma, c, lane, cols);
      Lane8<F32> dh{};
      if (a.dh != nullptr) dh = load8<F32, false>(dhr, c, lane, cols);
      chunk_grad<F32, false>(a, mask, row, c, lane, dy[i], h[i], dh, g, rstd, mean, acc[i]);
    }
  }
  if (a.dgamma == nullptr) return;
  float *part = static_cast<float *>(a.workspace) + static_cast<int64_t>(blockIdx.x) * cols;
  if (R == 1) {
#pragma unroll
    for (int i = 0; i < NU; ++i) store_cols8<false>(part, i * W + warp, lane, cols, acc[i]);
    return;
  }
  for (int y = 0; y < R; ++y) {
    __syncthreads();
    if (static_cast<int>(threadIdx.y) != y) continue;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = lane_col<false>(i * W + warp, lane, j);
        if (col < cols) sums[col] = y == 0 ? acc[i][j] : sums[col] + acc[i][j];
      }
    }
  }
  __syncthreads();
  for (int col = threadIdx.y * blockDim.x + threadIdx.x; col < cols; col += blockDim.x * R)
    part[col] = sums[col];
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Rows in phase (every matrix's row starts at the same element of a 16-byte unit; base
// addresses at its first): the rows' units come through a ring of `stages` stages of
// RP rows in shared memory by asynchronous 16-byte copies.  A thread reads only what it
// copied, so the ring needs no barrier, and the copies of the next rows are in flight
// while a row is reduced and written.  blockDim = (32 W, R), R groups of RP rows at a time,
// NU units a lane; short rows (1 << lg < 32 lanes a row, W = NU = 1) several a warp.  Paired
// fp32 arithmetic; n is formed before it meets mean(u n) or dy, as rstd^2 mean(u n) and rstd dy
// may be past fp32, or below its normal values, where the gradients are not.
//
// kExact: aligned rows of 32 NU W units.  kWhole: aligned rows of whole units, fewer than
// that (or short ones), no element of a unit masked: bf16 [4096, 11008] 65.7 us (149 element
// by element), fp32 [4096, 5000] 53.5 (61.8 as rows with edges).  kEdges: a row may start
// within a unit and end within one: a CTA takes rows that start at one such place (phase),
// so that its threads' columns stay the same.  The first and last unit of such a row hold
// elements of its neighbours (or nothing, which the copy leaves out past the matrix's end);
// they count as 0 and are not written.
enum Rows { kExact, kWhole, kEdges };

// Warps of a CTA, at most: 128 registers a thread, or 170 where NU units of rows with edges
// need them, or 80 where one aligned unit takes no more ([65536, 1024] 78.5 us, 81.3 with 16
// warps; [32768, 768] 27.7, 29.7).
template <Rows HOW, int NU>
constexpr int kRingWarps = HOW != kEdges && NU == 1 ? 24 : HOW != kEdges || NU <= 2 ? 16 : 12;

template <bool F32, Rows HOW, int NU, int RP>
__global__ void __launch_bounds__(kRingWarps<HOW, NU> * 32, 1)
rmsnorm_grad_ring(NormBackward a, int stages, int classes, int lg) {
  pdl_enter();
  constexpr bool EDGES = HOW == kEdges;
  constexpr int E = Unit<F32>::E, ES = 16 / E, kUnits = 32 * E;  // columns of a warp's unit
  __shared__ float red[2][16][RP][16];  // [round & 1][row group][row][warp]
  extern __shared__ __align__(16) unsigned char ring[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5, R = blockDim.y;
  const int at = lane & ((1 << lg) - 1), sub = lane >> lg, per = 32 >> lg;
  const int T = blockDim.x * R, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int cols = static_cast<int>(a.cols);
  const uint32_t rows = static_cast<uint32_t>(a.rows);
  const bool up = a.dh != nullptr, drop = RP == 1 && a.drop.rng != nullptr;
  // rows cls, cls + classes, ...: of these, runs of per R, every step-th run, RP of them a round
  // (runs of RP adjacent ones leave some CTAs RP rows more than others: [4096, 8192] 46.1 us, 45.7 so)
  const uint32_t cls = blockIdx.x % classes;
  const uint32_t next = classes * per * R * (gridDim.x / classes);  // from a group's row to its next
  const uint32_t hop = next * RP;
  const uint32_t begin = cls + classes * per * R * (blockIdx.x / classes);
  uint32_t row = begin + classes * (threadIdx.y * per + sub);
  const int rounds = begin < rows ? static_cast<int>((rows - begin - 1) / hop + 1) : 0;
  const int phase = !EDGES ? 0 : static_cast<int>((cls * a.ld_h) & (E - 1));
  // a lane's first unit, and columns from one to the next (rows with edges: a warp's chunks
  // follow one another, as their mask goes on from each to the next)
  const int chunk0 = EDGES ? warp * NU : warp, chunk_step = EDGES ? 1 : W;
  const int col0 = chunk0 * kUnits + at * E - phase, unit_cols = chunk_step * kUnits;

  const int row_bytes = NU * T * 16, input_bytes = RP * row_bytes;
  const int stage_bytes = (up ? 3 : 2) * input_bytes;
  uint32_t ahead = row;  // the next row to copy, and where to
  const uint32_t base = smem_addr(ring) + tid * 16, end = base + stages * stage_bytes;
  uint32_t into = base;
  const auto copy_row = [&](const void *m, int64_t ld, uint32_t r, uint32_t dst) {
    const char *src = static_cast<const char *>(m) + (r * ld + col0) * ES;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int left = cols - (col0 + i * unit_cols);
      if (HOW == kExact || (HOW == kWhole ? left > 0 : left >= E)) {
        cp_async_16(dst + i * (T * 16), src + i * ES * unit_cols);
      } else if (EDGES && left > 0) {
        cp_async_16_part(dst + i * (T * 16), src + i * ES * unit_cols, ES * left);
      }
    }
  };
  const auto issue = [&] {
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      const uint32_t r = ahead + p * next;
      if (r >= rows) break;
      copy_row(a.dy, a.ld_dy, r, into + p * row_bytes);
      copy_row(a.h, a.ld_h, r, into + input_bytes + p * row_bytes);
      if (up) copy_row(a.dh, a.ld_dh, r, into + 2 * input_bytes + p * row_bytes);
    }
    cp_async_commit();
    ahead += hop;  // rows <= INT32_MAX and hops of under 2^22: no wrap
    into += stage_bytes;
    if (into == end) into = base;
  };
  uint32_t slot = base;
  // a lane's unit i of row p of input n of the stage at `slot`
  const auto unit = [&](int n, int p, int i) {
    const uint4 u = lds_u4(slot + n * input_bytes + p * row_bytes + i * (T * 16));
    Unit<F32> v;
    v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    const int col = col0 + i * unit_cols;
    if constexpr (EDGES) {
      if (col < 0 || col + E > cols) v.clip(-col, cols - col);
    } else if (HOW == kWhole && col >= cols) {
      v.w[0] = v.w[1] = v.w[2] = v.w[3] = 0;
    }
    return v;
  };

  for (int k = 0; k < stages - 1; ++k) issue();
  uint64_t g[NU][E / 2], acc[NU][E / 2];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const int col = col0 + i * unit_cols + 2 * j;
      g[i][j] = pack_f32x2(col >= 0 && col < cols ? ld_keep_f32(a.gamma + col) : 0.0f,
                           col >= -1 && col + 1 < cols ? ld_keep_f32(a.gamma + col + 1) : 0.0f);
      acc[i][j] = 0;
    }
  for (int i = tid; i < 2 * 16 * RP * 16; i += T) (&red[0][0][0][0])[i] = 0.0f;
  __syncthreads();
  const float over = 1.0f / static_cast<float>(cols);
  Mask mask{};
  if (drop) mask = mask_of(a.drop);
  float scale[RP];  // rstd of the next round's rows
#pragma unroll
  for (int p = 0; p < RP; ++p) scale[p] = row + p * next < rows ? ld_keep_f32(a.rstd + row + p * next) : 0.0f;
  for (int k = 0; k < rounds; ++k) {
    issue();
    if (stages == 3) cp_async_wait<2>();
    else cp_async_wait<1>();
    float dot[RP], rstd[RP];
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      rstd[p] = scale[p];
      const uint32_t r = row + hop + p * next;
      if (r < rows) scale[p] = ld_keep_f32(a.rstd + r);
      uint64_t s = 0;
      if (row + p * next < rows) {
        const uint64_t rstd2 = pack_f32x2(rstd[p], rstd[p]);
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const Unit<F32> dy = unit(0, p, i), h = unit(1, p, i);
#pragma unroll
          for (int j = 0; j < E / 2; ++j)
            s = fma_f32x2(mul_f32x2(dy.pair(j), g[i][j]), mul_f32x2(h.pair(j), rstd2), s);
        }
      }
      dot[p] = f32x2_lo(s) + f32x2_hi(s);
    }
    if (lg < 5) {
#pragma unroll
      for (int p = 0; p < RP; ++p)
        for (int o = 1 << lg >> 1; o > 0; o >>= 1) dot[p] += __shfl_xor_sync(0xffffffffu, dot[p], o);
    } else {
      // two rows: each half of the warp adds up one of them
      float v = dot[0];
      if (RP == 2) {
        const float other = lane < 16 ? dot[RP - 1] : dot[0];
        v = (lane < 16 ? dot[0] : dot[RP - 1]) + __shfl_xor_sync(0xffffffffu, other, 16);
      } else {
        v += __shfl_xor_sync(0xffffffffu, v, 16);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (W > 1) {  // the two halves of red in turn: one barrier a round
        float *r = red[k & 1][threadIdx.y][RP == 2 ? lane >> 4 : 0];
        if ((lane & (RP == 2 ? 15 : 31)) == 0) r[warp] = v;
        group_barrier(1 + threadIdx.y, blockDim.x);
        v = r[lane & 15];
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      }
      dot[0] = v;
      if (RP == 2) {
        dot[0] = __shfl_sync(0xffffffffu, v, 0);
        dot[RP - 1] = __shfl_sync(0xffffffffu, v, 16);
      }
    }
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      const uint32_t r = row + p * next;
      if (r >= rows) break;
      const float less = -dot[p] * over;
      const uint64_t rstd2 = pack_f32x2(rstd[p], rstd[p]), less2 = pack_f32x2(less, less);
      uint32_t before = 0;
      if (EDGES && drop && chunk0 > 0) before = kept_group<E>(mask, r, chunk0 * 32 - 1);
      char *const out_x = row_of<F32>(a.dx, r, a.ld_dx), *const out_r = row_of<F32>(a.dres, r, a.ld_dres);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const int c = chunk0 + i * chunk_step, col = col0 + i * unit_cols;
        if (HOW != kExact && c * kUnits - phase >= cols) continue;
        const Unit<F32> dy = unit(0, p, i), h = unit(1, p, i);
        Unit<F32> dh{};
        if (up) dh = unit(2, p, i);
        float d[E];
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const uint64_t n = mul_f32x2(h.pair(j), rstd2);
          acc[i][j] = fma_f32x2(dy.pair(j), n, acc[i][j]);
          const uint64_t t = fma_f32x2(n, less2, mul_f32x2(dy.pair(j), g[i][j]));
          const uint64_t v = up ? fma_f32x2(t, rstd2, dh.pair(j)) : mul_f32x2(t, rstd2);
          d[2 * j] = f32x2_lo(v);
          d[2 * j + 1] = f32x2_hi(v);
        }
        Unit<F32> out;
        const int bound = HOW == kExact ? INT32_MAX : cols;
        if (drop) {
          if (a.dres != nullptr) {
            out.set(d);
            out.template store<!EDGES>(out_r, col, bound);
          }
          if constexpr (EDGES) drop_unit_phase<E>(d, mask, r, c * 32 + lane, lane, phase, before);
          else drop_unit<E>(d, mask, r, c * 32 + at);
        }
        out.set(d);
        out.template store<!EDGES>(out_x, col, bound);
      }
    }
    row += hop;
    slot += stage_bytes;
    if (slot == end) slot = base;
  }
  if (a.dgamma == nullptr) return;
  // a warp's rows, then the row groups in their order, in the ring's memory (a group's
  // columns are at most half of its units there).  [262144, 128] 35.0 us, 42.3 with the
  // groups one after the other.
  float *part = static_cast<float *>(a.workspace) + static_cast<int64_t>(blockIdx.x) * cols;
  float *const sums = reinterpret_cast<float *>(ring), *const mine = sums + threadIdx.y * cols;
  for (int o = 16; o >= 1 << lg; o >>= 1)
#pragma unroll
    for (int j = 0; j < E / 2; ++j)  // short rows: NU = 1
      acc[0][j] = add_f32x2(acc[0][j], __shfl_xor_sync(0xffffffffu, acc[0][j], o));
  cp_async_wait<0>();
  __syncthreads();
  // 16-byte pieces where columns allow: a float an access cost 3 us at 8192 columns
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int col = col0 + i * unit_cols;
    if constexpr (!EDGES) {
      if (sub != 0 || col >= cols) continue;
      float *const to = (R == 1 ? part : mine) + col;
#pragma unroll
      for (int q = 0; q < E / 4; ++q)
        reinterpret_cast<float4 *>(to)[q] =
            make_float4(f32x2_lo(acc[i][2 * q]), f32x2_hi(acc[i][2 * q]), f32x2_lo(acc[i][2 * q + 1]),
                        f32x2_hi(acc[i][2 * q + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (col + j >= 0 && col + j < cols) mine[col + j] = j & 1 ? f32x2_hi(acc[i][j >> 1]) : f32x2_lo(acc[i][j >> 1]);
    }
  }
  if (!EDGES && R == 1) return;
  __syncthreads();
  constexpr int kStep = EDGES ? 1 : 4;
  for (int col = tid * kStep; col < cols; col += T * kStep) {
    if constexpr (EDGES) {
      float v = sums[col];
      for (int y = 1; y < R; ++y) v += sums[y * cols + col];
      part[col] = v;
    } else {
      float4 v = *reinterpret_cast<const float4 *>(sums + col);
      for (int y = 1; y < R; ++y) v = add4(v, *reinterpret_cast<const float4 *>(sums + y * cols + col));
      *reinterpret_cast<float4 *>(part + col) = v;
    }
  }
}

// Looped form, first kernel: sum(u n) of each row, a CTA a row.
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
    const float rstd = ld_keep_f32(a.rstd + row);
    float dot = 0.0f;
    for (int c = warp; c < chunks; c += W) {
      const Lane8<F32> dy = load8<F32, VEC, true>(dyr, c, lane, cols);
      const Lane8<F32> h = load8<F32, VEC, true>(hr, c, lane, cols);
      float g[8];
      load_cols8<VEC>(g, a.gamma, c, lane, cols);
      dot += chunk_dot<F32>(dy, h, g, rstd);
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
    const float mean = ld_keep_f32(dots + row) * over;
    chunk_grad<F32, VEC>(a, mask, row, c, lane, dy, h, dh, g, rstd, mean, acc);
  }
  if (a.dgamma != nullptr)
    store_cols8<VEC>(partial + static_cast<int64_t>(blockIdx.y) * cols, c, lane, cols, acc);
}

// dgamma: the sum of P shares of each column.  32 columns a CTA, 32 runs of shares; a
// thread's loads are in flight together (one after the other: 4 us more with 152 shares).
__global__ void __launch_bounds__(1024) rmsnorm_grad_join(const float *partial, float *dgamma,
                                                          int P, int64_t cols) {
  pdl_enter();
  __shared__ float red[32][33];
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.0f;
  for (int p = threadIdx.y; p < P; p += 32 * 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = col < cols && p + 32 * i < P ? ld_keep_f32(partial + (p + 32 * i) * cols + col) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[i];
  }
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < cols) dgamma[out] = s;
}

// The ring's launch; W = 0: the row does not fit.
struct RingShape {
  int units, W, R, rp, lg, stages, classes;
  Rows how;
  int64_t grid;
  size_t smem;
};

template <bool F32>
RingShape ring_shape(const NormBackward &a, int sm_count, int smem_max) {
  constexpr int E = Unit<F32>::E, kUnits = 32 * E;
  RingShape g{};
  const int64_t rem = a.rows == 1 ? 0 : a.ld_h & (E - 1);
  g.classes = rem == 0 ? 1 : rem & 1 ? E : rem & 2 ? E / 2 : 2;
  const int chunks = static_cast<int>((a.cols + (g.classes > 1 ? E - 1 : 0) + kUnits - 1) / kUnits);
  const bool whole = g.classes == 1 && a.cols % E == 0;
  g.lg = 5;
  if (whole)
    while (g.lg > 0 && (E << g.lg >> 1) >= a.cols) --g.lg;
  // Two rows at a time, one with dropout (with two its generator's code, twice, costs more
  // than they gain: bf16 [16384, 4096] 121 us against 105) or where two do not fit.  Without:
  // [8192, 8192] 64.2 us against 77.7.
  g.rp = a.drop.rng != nullptr || chunks > 32 ? 1 : 2;
  // Aligned rows of 33 to 48 chunks: three units a lane and up to 16 warps, not four and up
  // to 12 ([4096, 11008] 65.7 us, 73.2 with four).
  g.units = chunks <= 4 ? 1 : chunks <= 32 ? 2 : whole && chunks <= 48 ? 3 : 4;
  int warps = 16;
  const auto fit = [&](int units) {
    g.units = units;
    g.W = (chunks + units - 1) / units;
    g.how = !whole ? kEdges : a.cols == static_cast<int64_t>(kUnits) * units * g.W ? kExact : kWhole;
    warps = whole && units == 1 ? 24 : whole || units <= 2 ? 16 : 12;
    return warps / g.W * g.W;
  };
  // Rows of 9 to 11 warps leave the others idle: three units a lane instead.  [8192, 4097] 88 us,
  // 62 so; one aligned row a round (dropout, [8192, 5120]) 79.4, 77.7 so.  Two of them
  // a round do not gain: [6000, 5120] 42.2, 47.6 so.
  if (fit(g.units) < 12 && g.units == 2 && (!whole || g.rp == 1)) fit(3);
  if (g.W > warps || (!F32 && g.units == 4 && !whole)) return RingShape{};
  const int64_t rows = (a.rows + g.classes - 1) / g.classes, ctas = std::max(1, sm_count / g.classes);
  const int64_t per = (32 >> g.lg) * g.rp, groups = (rows + per - 1) / per;
  g.R = static_cast<int>(std::min<int64_t>(g.W > 1 ? std::min(15, warps / g.W) : warps, (groups + ctas - 1) / ctas));
  g.grid = std::min<int64_t>((groups + g.R - 1) / g.R, ctas) * g.classes;
  const size_t stage = static_cast<size_t>(a.dh ? 3 : 2) * g.units * 32 * g.W * g.R * 16 * g.rp;
  // (a fourth stage, or a third of two rows, gains nothing: 43.6 us at [262144, 128], 44.5)
  g.stages = static_cast<int>(std::min<size_t>(g.rp == 2 ? 2 : 3, (smem_max - 5120) / stage));
  if (g.stages < 2) return RingShape{};
  g.smem = g.stages * stage;
  return g;
}

template <bool F32, Rows HOW, int NU, int RP>
cudaError_t launch_ring_of(const NormBackward &a, const RingShape &g, cudaStream_t s) {
  const auto kern = rmsnorm_grad_ring<F32, HOW, NU, RP>;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kern), g.smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(static_cast<unsigned>(g.grid)), dim3(32 * g.W, g.R), g.smem, s, 0, a, g.stages,
                  g.classes, g.lg);
}

template <bool F32, Rows HOW>
cudaError_t launch_ring_how(const NormBackward &a, const RingShape &g, cudaStream_t s) {
  if (g.units == 1) return g.rp == 1 ? launch_ring_of<F32, HOW, 1, 1>(a, g, s) : launch_ring_of<F32, HOW, 1, 2>(a, g, s);
  if (g.units == 2) return g.rp == 1 ? launch_ring_of<F32, HOW, 2, 1>(a, g, s) : launch_ring_of<F32, HOW, 2, 2>(a, g, s);
  if constexpr (HOW == kEdges)
    if (g.units == 3 && g.rp == 2) return launch_ring_of<F32, HOW, 3, 2>(a, g, s);
  if (g.units == 3) return launch_ring_of<F32, HOW, 3, 1>(a, g, s);
  if constexpr (HOW != kEdges || F32) return launch_ring_of<F32, HOW, 4, 1>(a, g, s);
  return cudaErrorInvalidValue;  // ring_shape gives no such shape
}

template <bool F32>
cudaError_t launch_ring(const NormBackward &a, const RingShape &g, cudaStream_t s) {
  return g.how == kExact   ? launch_ring_how<F32, kExact>(a, g, s)
         : g.how == kWhole ? launch_ring_how<F32, kWhole>(a, g, s)
                           : launch_ring_how<F32, kEdges>(a, g, s);
}

// Shapes of the other launches, which the workspace follows.
struct GradShape {
  int units, W, R;  // persistent
  int64_t grid;     // CTAs, or the looped form's runs of rows
};

GradShape held_shape(int64_t rows, int64_t cols, int sm_count) {
  const int chunks = static_cast<int>((cols + kChunk - 1) / kChunk);
  GradShape g{};
  g.units = chunks <= 2 ? 1 : 2;
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
cudaError_t launch_grad(const NormBackward &a, bool held, bool phase, int sm_count, int smem_max, cudaStream_t s) {
  cudaError_t e;
  const float *partial = static_cast<const float *>(a.workspace);
  int64_t P;
  RingShape rs{};
  if (held && phase) rs = ring_shape<F32>(a, sm_count, smem_max);
  if (rs.W > 0) {
    e = launch_ring<F32>(a, rs, s);
    P = rs.grid;
  } else if (held) {
    const GradShape g = held_shape(a.rows, a.cols, sm_count);
    const dim3 grid(static_cast<unsigned>(g.grid)), block(32 * g.W, g.R);
    const size_t smem = g.R > 1 ? a.cols * 4 : 0;
    e = g.units == 1 ? launch_k(rmsnorm_grad_held<F32, 1>, grid, block, smem, s, 0, a)
                     : launch_k(rmsnorm_grad_held<F32, 2>, grid, block, smem, s, 0, a);
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

bool rmsnorm_grad_held_ok(int64_t cols, bool f32, bool whole) {
  return cols <= kChunk * 16 * (!f32 && whole ? 4 : 2);
}

size_t rmsnorm_grad_workspace(int64_t rows, int64_t cols, bool held, int sm_count) {
  // a share a CTA: at most two an SM, and at most a CTA a row, or in the ring a row of the
  // longest of 8 classes for each of them
  if (held) return static_cast<size_t>(std::min<int64_t>((rows + 7) / 8 * 8, std::max(8, 2 * sm_count)) * cols * 4);
  return static_cast<size_t>(dots_bytes(rows) + looped_shape(rows, cols, sm_count).grid * cols * 4);
}

cudaError_t launch_rmsnorm_backward(const NormBackward &a, bool f32, bool vec, bool phase, bool held,
                                    int sm_count, int smem_max, cudaStream_t s) {
  if (f32)
    return vec ? launch_grad<true, true>(a, held, phase, sm_count, smem_max, s)
               : launch_grad<true, false>(a, held, phase, sm_count, smem_max, s);
  return vec ? launch_grad<false, true>(a, held, phase, sm_count, smem_max, s)
             : launch_grad<false, false>(a, held, phase, sm_count, smem_max, s);
}

}  // namespace fr
