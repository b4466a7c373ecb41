// Dropout and the root-mean-square norm of rows, with the residual's addition
// before it and an output of the matrices' type or in 8 bits (e4m3) with scales:
//   h = residual + dropout(x)            rounded to the type, what the residual's path keeps
//   rstd = 1 / sqrt(mean(h^2) + eps)     of the rounded h, so that a backward pass that
//   y = h rstd gamma                     reads h sees the norm that was taken
// One pass: the row is held in registers from its load to its store, so the bytes
// are those of the inputs and outputs, and memory bounds every size but the smallest.
#include <algorithm>

#include "rmsnorm.cuh"

namespace fr {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr int kGroup = FR_SCALE_COLS;  // columns of a scale in groups

// v = h k gamma for a lane's 8 elements.
template <bool F32>
__device__ __forceinline__ void normed8(float (&v)[8], const Lane8<F32> &h, float k, const float (&g)[8]) {
  const uint64_t k2 = pack_f32x2(k, k);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = mul_f32x2(mul_f32x2(pack_f32x2(h.at(2 * i), h.at(2 * i + 1)), k2),
                                 pack_f32x2(g[2 * i], g[2 * i + 1]));
    v[2 * i] = f32x2_lo(x);
    v[2 * i + 1] = f32x2_hi(x);
  }
}

// s + the squares of a lane's 8 elements, the even and the odd ones apart.
template <bool F32>
__device__ __forceinline__ uint64_t squares8(const Lane8<F32> &h, uint64_t s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t x = pack_f32x2(h.at(2 * i), h.at(2 * i + 1));
    s = fma_f32x2(x, x, s);
  }
  return s;
}

// Two values to e4m3, to nearest even, past the largest to it; lo in the low byte.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// 8 values to e4m3, the first four times inv[0], the others times inv[1]: reciprocals of
// the scales.  Divided by the scales, [8192, 8192] took 56.6 us (36.2 so), and no fewer values
// differed from 64 bits' (those near halfway between two of e4m3: some 10 of 21 million).
__device__ __forceinline__ void e4m3_8(uint32_t (&w)[2], const float (&v)[8], const float (&inv)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t k = pack_f32x2(inv[i], inv[i]);
    const uint64_t a = mul_f32x2(pack_f32x2(v[4 * i], v[4 * i + 1]), k);
    const uint64_t b = mul_f32x2(pack_f32x2(v[4 * i + 2], v[4 * i + 3]), k);
    w[i] = pack_e4m3x2(f32x2_lo(a), f32x2_hi(a)) |
           static_cast<uint32_t>(pack_e4m3x2(f32x2_lo(b), f32x2_hi(b))) << 16;
  }
}

// A lane's 8 values times inv, in 8 bits.
template <bool VEC>
__device__ __forceinline__ void store8_e4m3(void *row, int c, int lane, int cols,
                                            const float (&v)[8], const float (&inv)[2]) {
  uint32_t w[2];
  e4m3_8(w, v, inv);
  if constexpr (VEC) {
    const int col = c * kChunk + lane * 8;
    if (col < cols)
      asm volatile("st.global.cs.v2.b32 [%0], {%1, %2};" ::"l"(static_cast<char *>(row) + col),
                   "r"(w[0]), "r"(w[1])
                   : "memory");
  } else {
    const int first = lane_col<false>(c, lane, 0), left = cols - first;
    char *p = static_cast<char *>(row) + first;
    const auto st = [&](int j) {
      asm volatile("st.global.cs.u8 [%0], %1;" ::"l"(p + 32 * j), "r"(w[j >> 2] >> (8 * (j & 3)))
                   : "memory");
    };
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * j < left) st(j);
  }
}

// The same for a unit of a row in phase, from column `col` on.
__device__ __forceinline__ void store_unit_e4m3(char *row, int col, int cols, const float (&v)[8],
                                                const float (&inv)[2]) {
  uint32_t w[2];
  e4m3_8(w, v, inv);
  if (col >= 0 && col + 8 <= cols) {
    asm volatile("st.global.cs.v2.b32 [%0], {%1, %2};" ::"l"(row + col), "r"(w[0]), "r"(w[1]) : "memory");
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (col + j >= 0 && col + j < cols)
      asm volatile("st.global.cs.u8 [%0], %1;" ::"l"(row + col + j), "r"(w[j >> 2] >> (8 * (j & 3))) : "memory");
}

// The largest magnitude of three (NaN if one is).
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// The scale for values whose largest magnitude is `most` (NaN stays): never below
// the smallest normal, so that its reciprocal is finite and rows of zeros give zeros.
__device__ __forceinline__ float scale_for(float most) {
  return max_nan(most * (1.0f / kE4m3Max), 1.17549435e-38f);
}

// The scale that the caller gives: no smaller than a written one, for the same reasons.
__device__ __forceinline__ float scale_given(const float *scale) {
  return max_nan(ld_keep_f32(scale), 1.17549435e-38f);
}

// A chunk of y in 8 bits with a scale per 128 columns: two scales a chunk.  Aligned
// rows: the halves of the warp hold one group each; others: a lane's first and last
// four elements belong to one each.
template <bool VEC>
__device__ __forceinline__ void store_groups(const NormForward &a, int64_t row, void *yrow, int c,
                                             int lane, const float (&y)[8]) {
  const int cols = static_cast<int>(a.cols);
  float m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    m[i] = max_nan(max_nan(fabsf(y[4 * i]), fabsf(y[4 * i + 1])),
                   max_nan(fabsf(y[4 * i + 2]), fabsf(y[4 * i + 3])));
  float inv[2];
  if constexpr (VEC) {
    float v = max_nan(m[0], m[1]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    const float s = scale_for(v);
    inv[0] = inv[1] = 1.0f / s;
    const int g = 2 * c + (lane >> 4);
    if ((lane & 15) == 0 && g * kGroup < cols) a.scale[row * a.scale_row + g * a.scale_col] = s;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float s = scale_for(warp_max(m[i]));
      inv[i] = 1.0f / s;
      const int g = 2 * c + i;
      if (lane == i && g * kGroup < cols) a.scale[row * a.scale_row + g * a.scale_col] = s;
    }
  }
  store8_e4m3<VEC>(yrow, c, lane, cols, y, inv);
}

// h of a chunk: residual + dropout(x), rounded; x becomes it.
template <bool F32, bool VEC>
__device__ __forceinline__ void block_sum(const NormForward &a, const Mask &mask, uint32_t row,
                                          int c, int lane, Lane8<F32> &x, const Lane8<F32> &res) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = x.at(j);
  if (a.drop.rng != nullptr) drop8<VEC>(v, mask, row, c, lane);
  if (a.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += res.at(j);
  }
  x.set(v);
}

// The same for a chunk of a row in phase.
__device__ __forceinline__ void block_sum_phase(const NormForward &a, const Mask &mask, uint32_t row,
                                                int c, int lane, int phase, uint32_t &before,
                                                Lane8<false> &x, const Lane8<false> &res) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = x.at(j);
  if (a.drop.rng != nullptr) drop8_phase(v, mask, row, c, lane, phase, before);
  if (a.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += res.at(j);
  }
  x.set(v);
}

template <bool F32>
__device__ __forceinline__ const char *row_of(const void *p, int64_t row, int64_t ld) {
  return static_cast<const char *>(p) + row * ld * (F32 ? 4 : 2);
}
template <bool F32>
__device__ __forceinline__ char *row_of(void *p, int64_t row, int64_t ld) {
  return static_cast<char *>(p) + row * ld * (F32 ? 4 : 2);
}

// The largest h rstd gamma of a thread's share of a row of h, read again by its row group, an
// element an access.  It is seldom called, and apart: of what is still held, within the
// kernel, 8 bits took up to 3 % more time, from fp32 13 % (registers).
template <bool F32>
__device__ __noinline__ float most_again(const void *h, const float *gamma, uint32_t cols, float rstd) {
  __syncwarp();  // h as the row group has stored it
  float most = 0.0f;
#pragma unroll 1
  for (uint32_t c = threadIdx.x; c < cols; c += blockDim.x) {
    float v;
    if constexpr (F32) v = ld_keep_f32(static_cast<const float *>(h) + c);
    else v = bf16_lo(ld_stream_u16(static_cast<const char *>(h) + static_cast<size_t>(c) * 2));
    most = max_nan(most, fabsf(v * rstd * ld_keep_f32(gamma + c)));
  }
  return most;
}

// The largest magnitude of a row's h rstd gamma.  While the row is read the largest h gamma is
// found, `most`; times rstd it is that, unless the product of two is infinite, or short of bits
// that count beside the smallest scale, though the product of three is neither.  `red` is one
// pass's own.
template <bool F32>
__device__ __forceinline__ float row_most(const NormForward &a, int64_t row, float most, float rstd,
                                          int W, float (&red)[32]) {
  if (most < __int_as_float(0x7f800000) && (most >= 1.17549435e-38f || rstd <= 4096.0f)) return most * rstd;
  const void *h = a.h != nullptr ? row_of<F32>(static_cast<const void *>(a.h), row, a.ldh)
                                 : row_of<F32>(a.x, row, a.ldx);
  most = warp_max(most_again<F32>(h, a.gamma, static_cast<uint32_t>(a.cols), rstd));
  if (W == 1) return most;
  const int lane = threadIdx.x & 31, first = threadIdx.y * W;
  if (lane == 0) red[first + (threadIdx.x >> 5)] = most;
  // (two row groups at most; a computed barrier would take all 16, and fewer CTAs fit an SM:
  // [8192, 8192] 47.6 us, 36.3 so)
  if (threadIdx.y == 0) asm volatile("bar.sync 1, %0;" ::"r"(32 * W) : "memory");
  else asm volatile("bar.sync 2, %0;" ::"r"(32 * W) : "memory");
  return warp_max(lane < W ? red[first + lane] : 0.0f);
}

// The sum of a row's squares (and its largest magnitude) over the W warps that hold
// it: every thread gets them.  `red` is one pass's own.
__device__ __forceinline__ void row_reduce(float &ss, float &most, bool with_max, int W,
                                           float (&red)[2][32]) {
  ss = warp_sum(ss);
  if (with_max) most = warp_max(most);
  if (W == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = threadIdx.y * W;  // of this row's warps
  if (lane == 0) {
    red[0][first + warp] = ss;
    if (with_max) red[1][first + warp] = most;
  }
  __syncthreads();
  ss = warp_sum(lane < W ? red[0][first + lane] : 0.0f);
  if (with_max) most = warp_max(lane < W ? red[1][first + lane] : 0.0f);
}

// Threads of a CTA that holds NU chunks a warp, at most; an SM holds 1024 of them.
template <int NU>
constexpr int kHeldThreads = NU <= 2 ? 1024 : NU <= 4 ? 512 : 256;

// Persistent form: blockDim = (32 W, R), R rows a CTA, W warps a row, NU chunks a warp.
// T: threads of a CTA at most (8 bits from fp32 rows of up to 4096 columns: 256, of which an SM
// holds five within 48 registers; [8192, 4096] 30.9 us, with 56 registers and four of them 35.0).
// EXACT: rows of NU W whole chunks, without a comparison an access (to e4m3 without a residual,
// which instructions bound, bf16 [8192, 8192] 36.3 us, 39.1 with; given scale [2048, 10240] 12.5,
// 13.8; bf16 out and a residual's sum within 1 %).
template <bool F32, bool VEC, int NU, bool SUM, bool QUANT, bool EXACT, int T = kHeldThreads<NU>>
__global__ void __launch_bounds__(T, NU == 2 && T == 256 ? 5 : 1024 / T)
rmsnorm_held(NormForward a) {
  pdl_enter();
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int cols = EXACT ? INT32_MAX : static_cast<int>(a.cols);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = row < a.rows;
  const bool with_max = QUANT && a.scale_mode == FR_SCALE_ROW;
  float ss = 0.0f, most = 0.0f;
  uint64_t squares = 0;
  Lane8<F32> h[NU];
  if (live) {
    const char *xr = row_of<F32>(a.x, row, a.ldx);
#pragma unroll
    for (int i = 0; i < NU; ++i) h[i] = load8<F32, VEC>(xr, i * W + warp, lane, cols);
    if constexpr (SUM) {
      Lane8<F32> res[NU];
      const char *rr = row_of<F32>(a.residual, row, a.ldr);
      if (a.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < NU; ++i) res[i] = load8<F32, VEC>(rr, i * W + warp, lane, cols);
      }
      Mask mask{};
      if (a.drop.rng != nullptr) mask = mask_of(a.drop);
      char *hr = row_of<F32>(a.h, row, a.ldh);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        block_sum<F32, VEC>(a, mask, static_cast<uint32_t>(row), i * W + warp, lane, h[i], res[i]);
        store8<F32, VEC>(hr, i * W + warp, lane, cols, h[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float g[8];
      if (with_max) load_cols8<VEC>(g, a.gamma, i * W + warp, lane, cols);
      if constexpr (NU < 8) {
        squares = squares8(h[i], squares);  // 0 past the row
      } else {  // (a register fewer: 64 suffice)
        // runs of 4: of a lane's 64 squares, added one by one, the last ones lose bits
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          float part = h[i].at(j) * h[i].at(j);
#pragma unroll
          for (int k = 1; k < 4; ++k) part = fmaf(h[i].at(j + k), h[i].at(j + k), part);
          ss += part;
        }
      }
      if (with_max) {
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(h[i].at(j) * g[j]));
      }
    }
  }
  if constexpr (NU < 8) ss = f32x2_lo(squares) + f32x2_hi(squares);
  row_reduce(ss, most, with_max, W, red);
  if (!live) return;
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
  float inv[2] = {1.0f, 1.0f};
  if (QUANT && a.scale_mode != FR_SCALE_GROUP) {
    __shared__ float again[32];
    const float s = with_max ? scale_for(row_most<F32>(a, row, most, rstd, W, again)) : scale_given(a.scale);
    if (with_max && threadIdx.x == 0) a.scale[row * a.scale_row] = s;
    inv[0] = inv[1] = 1.0f / s;
  }
  char *yr = QUANT ? static_cast<char *>(a.y) + row * a.ldy : row_of<F32>(a.y, row, a.ldy);
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int c = i * W + warp;
    if (c * kChunk >= cols) continue;
    float v[8], g[8];
    load_cols8<VEC>(g, a.gamma, c, lane, cols);
    normed8(v, h[i], rstd, g);
    if constexpr (QUANT) {
      if (a.scale_mode == FR_SCALE_GROUP) store_groups<VEC>(a, row, yr, c, lane, v);
      else store8_e4m3<VEC>(yr, c, lane, cols, v, inv);
    } else {
      Lane8<F32> y;
      y.set(v);
      store8<F32, VEC>(yr, c, lane, cols, y);
    }
  }
}

// Looped form, rows of any length: a CTA goes over its row twice, the second time
// over h, which its own threads stored (or x), from L2.
constexpr int kLoopThreads = 512;
template <bool F32, bool VEC, bool QUANT>
__global__ void __launch_bounds__(kLoopThreads) rmsnorm_looped(NormForward a) {
  pdl_enter();
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int W = kLoopThreads / 32;
  const int cols = static_cast<int>(a.cols);
  const int chunks = static_cast<int>((a.cols + kChunk - 1) / kChunk);
  Mask mask{};
  if (a.drop.rng != nullptr) mask = mask_of(a.drop);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const char *xr = row_of<F32>(a.x, row, a.ldx);
    const char *rr = row_of<F32>(a.residual, row, a.ldr);
    char *hr = row_of<F32>(a.h, row, a.ldh);
    float ss = 0.0f, most = 0.0f;
    for (int c = warp; c < chunks; c += W) {
      Lane8<F32> x = load8<F32, VEC>(xr, c, lane, cols), res{};
      if (a.residual != nullptr) res = load8<F32, VEC>(rr, c, lane, cols);
      if (a.h != nullptr) {
        block_sum<F32, VEC>(a, mask, static_cast<uint32_t>(row), c, lane, x, res);
        store8<F32, VEC>(hr, c, lane, cols, x);
      }
      // a short run of its own: long rows add chunk sums, not elements
      const uint64_t part = squares8(x, 0);
      ss += f32x2_lo(part) + f32x2_hi(part);
      if (QUANT && a.scale_mode == FR_SCALE_ROW) {
        float g[8];
        load_cols8<VEC>(g, a.gamma, c, lane, cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(x.at(j) * g[j]));
      }
    }
    row_reduce(ss, most, QUANT && a.scale_mode == FR_SCALE_ROW, W, red);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(cols) + a.eps);
    if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
    float inv[2] = {1.0f, 1.0f};
    if (QUANT && a.scale_mode != FR_SCALE_GROUP) {
      __shared__ float again[32];
      const float s = a.scale_mode == FR_SCALE_ROW ? scale_for(row_most<F32>(a, row, most, rstd, W, again))
                                                   : scale_given(a.scale);
      if (a.scale_mode == FR_SCALE_ROW && threadIdx.x == 0) a.scale[row * a.scale_row] = s;
      inv[0] = inv[1] = 1.0f / s;
    }
    const char *again = a.h != nullptr ? hr : xr;
    char *yr = QUANT ? static_cast<char *>(a.y) + row * a.ldy : row_of<F32>(a.y, row, a.ldy);
    for (int c = warp; c < chunks; c += W) {
      const Lane8<F32> x = load8<F32, VEC, true>(again, c, lane, cols);
      float v[8], g[8];
      load_cols8<VEC>(g, a.gamma, c, lane, cols);
      normed8(v, x, rstd, g);
      if constexpr (QUANT) {
        if (a.scale_mode == FR_SCALE_GROUP) store_groups<VEC>(a, row, yr, c, lane, v);
        else store8_e4m3<VEC>(yr, c, lane, cols, v, inv);
      } else {
        Lane8<F32> y;
        y.set(v);
        store8<F32, VEC>(yr, c, lane, cols, y);
      }
    }
    __syncthreads();  // `red` is free for the next row
  }
}

// bf16 rows in phase that are not aligned (odd row lengths): a lane's units are aligned ones
// that begin up to 7 elements before their columns.  One 16-byte access instead of 8 of an
// element: bf16 [16384, 4097] with residual 85.8 us, 108 so.
template <int NU, bool SUM, bool QUANT>
__global__ void __launch_bounds__(kHeldThreads<NU>, 1024 / kHeldThreads<NU>)
rmsnorm_phase(NormForward a) {
  pdl_enter();
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int cols = static_cast<int>(a.cols);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = row < a.rows;
  const bool with_max = QUANT && a.scale_mode == FR_SCALE_ROW;
  const int phase = static_cast<int>(row * a.ldx & 7);
  const int col0 = warp * NU * kChunk + lane * 8 - phase;  // a warp's chunks follow one another
  float most = 0.0f;
  uint64_t squares = 0;
  Lane8<false> h[NU];
  if (live) {
    const char *xr = row_of<false>(a.x, row, a.ldx);
    const int x_left = elements_left(a.rows, row, a.ldx, cols);
#pragma unroll
    for (int i = 0; i < NU; ++i) h[i] = load_unit<false>(xr, col0 + i * kChunk, cols, x_left);
    if constexpr (SUM) {
      Lane8<false> res[NU];
      const char *rr = row_of<false>(a.residual, row, a.ldr);
      if (a.residual != nullptr) {
        const int r_left = elements_left(a.rows, row, a.ldr, cols);
#pragma unroll
        for (int i = 0; i < NU; ++i) res[i] = load_unit<false>(rr, col0 + i * kChunk, cols, r_left);
      }
      Mask mask{};
      uint32_t before = 0;
      if (a.drop.rng != nullptr) {
        mask = mask_of(a.drop);
        before = kept_before(mask, static_cast<uint32_t>(row), warp * NU);
      }
      char *hr = row_of<false>(a.h, row, a.ldh);
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        block_sum_phase(a, mask, static_cast<uint32_t>(row), warp * NU + i, lane, phase, before, h[i],
                        res[i]);
        store_unit<false, true>(hr, col0 + i * kChunk, cols, h[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int col = col0 + i * kChunk;
      if (col < 0 || col + 8 > cols) h[i].clip(-col, cols - col);
      float g[8];
      if (with_max) load_cols_unit(g, a.gamma, col, cols);
      squares = squares8(h[i], squares);
      if (with_max) {
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(h[i].at(j) * g[j]));
      }
    }
  }
  float ss = f32x2_lo(squares) + f32x2_hi(squares);
  row_reduce(ss, most, with_max, W, red);
  if (!live) return;
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(cols) + a.eps);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[row] = rstd;
  float inv[2] = {1.0f, 1.0f};
  if (QUANT) {
    __shared__ float again[32];
    const float s = with_max ? scale_for(row_most<false>(a, row, most, rstd, W, again)) : scale_given(a.scale);
    if (with_max && threadIdx.x == 0) a.scale[row * a.scale_row] = s;
    inv[0] = inv[1] = 1.0f / s;
  }
  char *yr = QUANT ? static_cast<char *>(a.y) + row * a.ldy : row_of<false>(a.y, row, a.ldy);
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int col = col0 + i * kChunk;
    if (col >= cols) continue;
    float v[8], g[8];
    load_cols_unit(g, a.gamma, col, cols);
    normed8(v, h[i], rstd, g);
    if constexpr (QUANT) {
      store_unit_e4m3(yr, col, cols, v, inv);
    } else {
      Lane8<false> y;
      y.set(v);
      store_unit<false, true>(yr, col, cols, y);
    }
  }
}

// Rows of at most a chunk, aligned: 1 << lg lanes hold a row, a warp U times 32 >> lg
// rows at a time, with one reading of gamma; no barrier.  Instructions bound it (e4m3 out,
// [524288, 128]: 43.2 us, a copy 30): the rows' steps of a reduction stand side by side, and
// the root and the reciprocals are the approximate ones, off by 2 units in the last place and
// by 1 (exact reciprocals 45.3), which is less than a sum of 256 columns may be off by.
template <bool F32, int U, bool SUM, bool QUANT>
__global__ void __launch_bounds__(256) rmsnorm_short(NormForward a, int lg) {
  pdl_enter();
  const int lane = threadIdx.x & 31, at = lane & ((1 << lg) - 1), sub = lane >> lg, per = 32 >> lg;
  const int cols = static_cast<int>(a.cols);
  const int64_t first =
      (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (U * per) + sub;
  const auto at_row = [&](const void *m, int64_t ld, int es) {
    return static_cast<char *>(const_cast<void *>(m)) + first * ld * es;
  };
  constexpr int ES = F32 ? 4 : 2;
  const char *const xr = at_row(a.x, a.ldx, ES);
  const int64_t xs = per * a.ldx * ES;
  Lane8<F32> h[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = first + u * per;
    if (row < a.rows) h[u] = load8<F32, true>(xr + u * xs, 0, at, cols);
    else h[u].zero();
  }
  if constexpr (SUM) {
    Lane8<F32> res[U];
    if (a.residual != nullptr) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = first + u * per;
        if (row < a.rows) res[u] = load8<F32, true>(row_of<F32>(a.residual, row, a.ldr), 0, at, cols);
      }
    }
    Mask mask{};
    if (a.drop.rng != nullptr) mask = mask_of(a.drop);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = first + u * per;
      if (row >= a.rows) continue;
      block_sum<F32, true>(a, mask, static_cast<uint32_t>(row), 0, at, h[u], res[u]);
      store8<F32, true>(row_of<F32>(a.h, row, a.ldh), 0, at, cols, h[u]);
    }
  }
  float g[8];
  load_cols8<true>(g, a.gamma, 0, at, cols);
  const float over = 1.0f / static_cast<float>(cols);
  float ss[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t squares = squares8(h[u], 0);
    ss[u] = f32x2_lo(squares) + f32x2_hi(squares);
  }
#pragma unroll
  for (int k = 4; k >= 0; --k)
    if (k < lg)
#pragma unroll
      for (int u = 0; u < U; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], 1 << k);
  if constexpr (!QUANT) {
    char *const yr = at_row(a.y, a.ldy, ES);
    const int64_t ys = per * a.ldy * ES;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = first + u * per;
      if (row >= a.rows) break;
      const float rstd = rsqrtf(fmaf(ss[u], over, a.eps));
      float v[8];
      normed8(v, h[u], rstd, g);
      if (a.rstd != nullptr && at == 0) a.rstd[row] = rstd;
      Lane8<F32> y;
      y.set(v);
      store8<F32, true>(yr + u * ys, 0, at, cols, y);
    }
  } else {
    float v[U][8], s[U];
    const bool row_scale = a.scale_mode == FR_SCALE_ROW;
    const int lanes_lg = !row_scale && lg > 4 ? 4 : lg;  // groups of 128 columns are 16 lanes
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ss[u] = rsqrtf(fmaf(ss[u], over, a.eps));
      normed8(v[u], h[u], ss[u], g);
      s[u] = max_nan(max_abs(max_abs(v[u][0], v[u][1], v[u][2]), v[u][3], v[u][4]),
                     max_abs(v[u][5], v[u][6], v[u][7]));
    }
    if (a.scale_mode == FR_SCALE_GIVEN) {
      const float given = scale_given(a.scale);
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = given;
    } else {
#pragma unroll
      for (int k = 4; k >= 0; --k)
        if (k < lanes_lg)
#pragma unroll
          for (int u = 0; u < U; ++u) s[u] = max_nan(s[u], __shfl_xor_sync(0xffffffffu, s[u], 1 << k));
    }
    const int group = row_scale ? 0 : at >> 4;
    const bool writes = a.scale_mode != FR_SCALE_GIVEN && (at & ((1 << lanes_lg) - 1)) == 0 && group * kGroup < cols;
    char *const yr = at_row(a.y, a.ldy, 1);
    const int64_t ys = per * a.ldy;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = first + u * per;
      if (row >= a.rows) break;
      if (a.rstd != nullptr && at == 0) a.rstd[row] = ss[u];
      if (a.scale_mode != FR_SCALE_GIVEN) s[u] = scale_for(s[u]);
      if (writes) a.scale[row * a.scale_row + (row_scale ? 0 : group * a.scale_col)] = s[u];
      float k;
      asm("rcp.approx.f32 %0, %1;" : "=f"(k) : "f"(s[u]));
      const float inv[2] = {k, k};
      store8_e4m3<true>(yr + u * ys, 0, at, cols, v[u], inv);
    }
  }
}

// Dropout alone, of aligned rows or element by element.  A warp has NU chunks of a row, one
// after the other (a CTA's 8 warps a run of 8 NU of them, or R = 8 / W rows), or for short
// rows (SHORT) the same chunk of NU rows; 1 << lg lanes hold an aligned row of at most a
// chunk (32 of others).
template <bool F32, bool VEC, int NU, bool SHORT, bool RES>
__global__ void __launch_bounds__(256, VEC && RES ? 3 : 4) dropout_chunks(NormForward a, unsigned runs, int lg) {
  pdl_enter();
  const int lane = threadIdx.x & 31, at = lane & ((1 << lg) - 1), W = blockDim.x >> 5;
  const int cols = static_cast<int>(a.cols);
  const unsigned group = SHORT ? blockIdx.x : blockIdx.x / runs;
  const int first = SHORT ? threadIdx.x >> 5
                          : (static_cast<int>(blockIdx.x - group * runs) * W + static_cast<int>(threadIdx.x >> 5)) * NU;
  const int64_t row0 = ((static_cast<int64_t>(group) * ((SHORT ? NU : 1) * blockDim.y) + threadIdx.y) << (5 - lg)) +
                       (lane >> lg);
  const auto row_at = [&](int i) { return SHORT ? row0 + (static_cast<int64_t>(i * blockDim.y) << (5 - lg)) : row0; };
  const auto chunk_at = [&](int i) { return SHORT ? first : first + i; };
  const auto has = [&](int i) {  // a warp's lanes agree but for short aligned rows
    return row_at(i) < a.rows && chunk_at(i) <= (cols - 1) / kChunk;
  };
  Mask mask{};
  if (a.drop.rng != nullptr) mask = mask_of(a.drop);
  Lane8<F32> x[NU], res[RES ? NU : 1];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (!has(i)) continue;
    const int64_t row = row_at(i);
    const char *xr = row_of<F32>(a.x, row, a.ldx), *rr = row_of<F32>(a.residual, row, a.ldr);
    x[i] = load8<F32, VEC>(xr, chunk_at(i), at, cols);
    if constexpr (RES) res[i] = load8<F32, VEC>(rr, chunk_at(i), at, cols);
  }
  // The generator's work is done while the loads are on their way: bf16 [16384, 4096] 43.7
  // us, 47.2 with each chunk's done when its turn comes.
  uint4 words[NU];
  if constexpr (VEC) {
    if (a.drop.rng != nullptr) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        words[i] = block_of(mask, static_cast<uint32_t>(row_at(i)), chunk_at(i), at);
        asm volatile("" : "+r"(words[i].x), "+r"(words[i].y), "+r"(words[i].z), "+r"(words[i].w));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (!has(i)) continue;
    const int64_t row = row_at(i);
    const int c = chunk_at(i);
    char *yr = row_of<F32>(a.h, row, a.ldh);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = x[i].at(j);
    if (a.drop.rng != nullptr) {
      if constexpr (VEC) drop8_by<true>(v, mask, words[i], at);
      else drop8<false>(v, mask, static_cast<uint32_t>(row), c, lane);
    }
    if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += res[i].at(j);
    }
    x[i].set(v);
    store8<F32, VEC>(yr, c, at, cols, x[i]);
  }
}

// Dropout of rows in phase.  The units of all rows, `units` a row, follow one another over
// the lanes, so that no length leaves lanes idle: a warp has NU spans of 31 units, one after
// the other.  A unit's elements lie in two blocks of the mask, its own and the one before,
// which the lane before has drawn; lane 0 only draws the block before its span.  bf16
// [1000000, 63] 72 us (a warp a row 309), [16384, 4097] 57.1 (element by element 87.5; the
// mask's bits, packed and moved, bound it: a copy takes 39.6), fp32 [500000, 63] 45.4 (129.6).
template <bool F32, int NU, bool RES>
__global__ void __launch_bounds__(256, 4) dropout_units(NormForward a, int units) {
  pdl_enter();
  const int lane = threadIdx.x & 31, cols = static_cast<int>(a.cols);
  const int64_t begin = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * (NU * 31);
  uint32_t row0;
  int at0;  // of the unit of lane 1 in the first span
  if (begin <= UINT32_MAX) {
    row0 = static_cast<uint32_t>(begin) / static_cast<uint32_t>(units);
    at0 = static_cast<int>(static_cast<uint32_t>(begin) - row0 * static_cast<uint32_t>(units));
  } else {
    row0 = static_cast<uint32_t>(begin / units);
    at0 = static_cast<int>(begin - static_cast<int64_t>(row0) * units);
  }
  // n / units for n < units + 31 NU
  const uint32_t over = units > 1 && units < 31 * NU ? 0xFFFFFFFFu / units + 1 : 0;
  const auto rows_on = [&](int n) {
    if (units >= 31 * NU) return n >= units ? 1 : 0;
    return units == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), over));
  };
  Mask mask{};
  if (a.drop.rng != nullptr) mask = mask_of(a.drop);
  Lane8<F32> x[NU], res[RES ? NU : 1];
  const uint32_t rows = static_cast<uint32_t>(a.rows), ld8 = static_cast<uint32_t>(a.ldx) & 7;
  uint32_t row[NU];
  int col[NU];  // cols: nothing of the row
  uint32_t own[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int n = at0 + 31 * i + lane - 1, on = n < 0 ? 0 : rows_on(n), at = n - on * units;
    row[i] = row0 + on;
    col[i] = lane == 0 || row[i] >= rows ? cols : at * 8 - static_cast<int>(row[i] * ld8 & 7);
    x[i].zero();
    if (col[i] < cols) {
      const auto left = [&](int64_t ld) {  // rows before the last 8 end 8 elements before the matrix, or more
        return row[i] + 8 < rows ? INT32_MAX : elements_left(a.rows, row[i], ld, cols);
      };
      x[i] = load_unit<F32>(row_of<F32>(a.x, row[i], a.ldx), col[i], cols, left(a.ldx));
      if constexpr (RES) res[i] = load_unit<F32>(row_of<F32>(a.residual, row[i], a.ldr), col[i], cols, left(a.ldr));
    }
    own[i] = static_cast<uint32_t>(at);
  }
  if (a.drop.rng != nullptr) {  // while the loads are on their way
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t bits = kept_bits(mask, row[i], own[i]);
      own[i] = (__shfl_up_sync(0xffffffffu, bits, 1) | bits << 8) >> (8 - (row[i] * ld8 & 7));
      asm volatile("" : "+r"(own[i]));
    }
  }
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (col[i] >= cols) continue;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = x[i].at(j);
    if (a.drop.rng != nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = own[i] >> j & 1u ? v[j] * mask.factor : 0.0f;
    }
    if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += res[i].at(j);
    }
    x[i].set(v);
    store_unit<F32, true>(row_of<F32>(a.h, row[i], a.ldh), col[i], cols, x[i]);
  }
}

constexpr int kHeldChunks = 64;  // of a row, at most: 32 warps with 2 each

template <bool F32, int U, bool SUM, bool QUANT>
cudaError_t launch_short_of(const NormForward &a, int lg, cudaStream_t s) {
  const int64_t per = 8 * U * static_cast<int64_t>(32 >> lg);
  return launch_k(rmsnorm_short<F32, U, SUM, QUANT>, dim3(static_cast<unsigned>((a.rows + per - 1) / per)),
                  dim3(256), 0, s, 0, a, lg);
}

// Rows a lane: one while more would leave fewer than two CTAs an SM (us with 1, 2, 4: bf16
// [2048, 128] 1.4, 1.6, 1.7; [8192, 128] 2.0, 2.5, 2.7; e4m3 out [16384, 128] 2.9, 3.0, 3.6),
// else four, which share the fixed work (bf16 [32768, 128] 3.3, 3.4, 3.0; [524288, 128]
// 44.8, 41.6, 40.3; e4m3 out 62.0, 50.0, 43.2, with eight 53.1; bf16 with a residual to e4m3,
// [262144, 128], 43.8, 37.8, 37.2), or two where a residual's sum leaves less room (bf16 with
// dropout 43.5, 41.1, 42.0; fp32 to e4m3 64.4, 64.5, 66.2).
template <bool F32, bool SUM, bool QUANT>
cudaError_t launch_short(const NormForward &a, int sm_count, cudaStream_t s) {
  int lg = 5;
  while (lg > 0 && (8 << lg >> 1) >= a.cols) --lg;
  constexpr int MANY = SUM && !(QUANT && !F32) ? 2 : 4;
  if (a.rows < 2 * 8 * MANY * static_cast<int64_t>(32 >> lg) * sm_count)
    return launch_short_of<F32, 1, SUM, QUANT>(a, lg, s);
  return launch_short_of<F32, MANY, SUM, QUANT>(a, lg, s);
}

// How many chunks a warp holds: few warps a row make the row's reduction cheap and the
// loads in flight of each many, as long as 64 registers suffice (1024 threads an SM).
// Measured (us with 1, 2, 3, 4, 6, 8): bf16 with residual, [16384, 4096] with dropout 90,
// 84.8, -, 78.7, 80, -; [32768, 768] without, 3 chunks, -, 27, 14.7, 15.4, 16.2, -; [8192,
// 16384] without -, 146, 143, 94.7, -, 80.1; fp32 [8192, 4096] with 83, 78.6, 79.1, -, -, -.
// e4m3 out with 4, 8: [8192, 8192] 44.1, 39.1; [32768, 2048] 42.0, 36.2; or 7, 6 or 5 if they
// divide the row ([12000, 5120] 34.4, 38.7 with 8; [22000, 2560] 31.5, 39.2).  Fewer rows than
// about a wave and a half of CTAs: 4 ([512, 4096] to e4m3 4.0, 5.8; bf16 [200, 16384] 3.8, 4.7).
template <bool F32, bool VEC, bool QUANT, bool SUM>
cudaError_t launch_held(const NormForward &a, int sm_count, cudaStream_t s) {
  const int chunks = static_cast<int>((a.cols + kChunk - 1) / kChunk);
  const bool many = a.rows * chunks >= 384 * static_cast<int64_t>(sm_count);
  int units = F32 ? 2 : !VEC ? (QUANT ? 2 : 3) : SUM || chunks <= (QUANT ? 7 : 40) || !many ? 4 : 8;
  if (QUANT && units == 8 && a.cols % kChunk == 0)
    for (int u = 8; u >= 5; --u)
      if (chunks % u == 0 && chunks / u <= 8) {
        units = u;
        break;
      }
  if (units == 3 && chunks > 3 * kHeldThreads<3> / 32) units = 2;
  if (chunks < units) units = chunks;
  if (a.rows < sm_count && chunks <= 32) units = 1;  // few rows: latency
  const int W = (chunks + units - 1) / units, R = W >= 4 ? 1 : 4 / W;
  const dim3 grid(static_cast<unsigned>((a.rows + R - 1) / R)), block(32 * W, R);
  if (units == 1) return launch_k(rmsnorm_held<F32, VEC, 1, SUM, QUANT, false>, grid, block, 0, s, 0, a);
  if constexpr (!F32) {
    if constexpr (VEC || !QUANT)
      if (units == 3) return launch_k(rmsnorm_held<F32, VEC, 3, SUM, QUANT, false>, grid, block, 0, s, 0, a);
    if constexpr (VEC) {
      const bool exact = a.cols == static_cast<int64_t>(kChunk) * units * W;
      if (units == 4)
        return exact ? launch_k(rmsnorm_held<F32, VEC, 4, SUM, QUANT, true>, grid, block, 0, s, 0, a)
                     : launch_k(rmsnorm_held<F32, VEC, 4, SUM, QUANT, false>, grid, block, 0, s, 0, a);
      if constexpr (!SUM && QUANT) {
        if (units == 7 && exact) return launch_k(rmsnorm_held<F32, VEC, 7, SUM, QUANT, true>, grid, block, 0, s, 0, a);
        if (units == 6 && exact) return launch_k(rmsnorm_held<F32, VEC, 6, SUM, QUANT, true>, grid, block, 0, s, 0, a);
        if (units == 5 && exact) return launch_k(rmsnorm_held<F32, VEC, 5, SUM, QUANT, true>, grid, block, 0, s, 0, a);
      }
      if constexpr (!SUM)
        if (units == 8)
          return exact ? launch_k(rmsnorm_held<F32, VEC, 8, SUM, QUANT, true>, grid, block, 0, s, 0, a)
                       : launch_k(rmsnorm_held<F32, VEC, 8, SUM, QUANT, false>, grid, block, 0, s, 0, a);
    }
  }
  if constexpr (F32 && VEC && QUANT && !SUM)
    if (W <= 8) return launch_k(rmsnorm_held<F32, VEC, 2, SUM, QUANT, false, 256>, grid, block, 0, s, 0, a);
  return launch_k(rmsnorm_held<F32, VEC, 2, SUM, QUANT, false>, grid, block, 0, s, 0, a);
}

// Chunks a warp holds (us with 1, 2, 3, 4: [16384, 4097] with residual 134, 108, 89.1, 87.7;
// [32768, 769] without 34.8, 27.6, 31.7, 23.8; [65536, 255] 57.9, 45.6, -, 61.7).
template <bool QUANT, bool SUM>
cudaError_t launch_phase(const NormForward &a, int sm_count, cudaStream_t s) {
  const int chunks = static_cast<int>((a.cols + 7 + kChunk - 1) / kChunk);
  const int units = a.rows < sm_count && chunks <= 32 ? 1 : chunks <= 2 ? 2 : 4;  // few rows: latency
  const int W = (chunks + units - 1) / units, R = W >= 4 ? 1 : 4 / W;
  const dim3 grid(static_cast<unsigned>((a.rows + R - 1) / R)), block(32 * W, R);
  if (units == 1) return launch_k(rmsnorm_phase<1, SUM, QUANT>, grid, block, 0, s, 0, a);
  if (units == 2) return launch_k(rmsnorm_phase<2, SUM, QUANT>, grid, block, 0, s, 0, a);
  return launch_k(rmsnorm_phase<4, SUM, QUANT>, grid, block, 0, s, 0, a);
}

template <bool F32, bool VEC, bool QUANT>
cudaError_t launch_looped(const NormForward &a, int sm_count, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(sm_count) * 4;
  return launch_k(rmsnorm_looped<F32, VEC, QUANT>, dim3(static_cast<unsigned>(a.rows < most ? a.rows : most)),
                  dim3(kLoopThreads), 0, s, 0, a);
}

template <bool F32, bool VEC, bool QUANT>
cudaError_t launch_form(const NormForward &a, bool phase, bool held, int sm_count, cudaStream_t s) {
  if (!held) return launch_looped<F32, VEC, QUANT>(a, sm_count, s);
  const bool sum = a.h != nullptr;
  if constexpr (VEC)
    if (a.cols <= kChunk)
      return sum ? launch_short<F32, true, QUANT>(a, sm_count, s) : launch_short<F32, false, QUANT>(a, sm_count, s);
  if constexpr (!F32 && !VEC)
    if (phase && !(QUANT && a.scale_mode == FR_SCALE_GROUP) && a.cols + 7 <= kChunk * kHeldChunks)
      return sum ? launch_phase<QUANT, true>(a, sm_count, s) : launch_phase<QUANT, false>(a, sm_count, s);
  return sum ? launch_held<F32, VEC, QUANT, true>(a, sm_count, s)
             : launch_held<F32, VEC, QUANT, false>(a, sm_count, s);
}

template <bool F32, bool VEC>
cudaError_t launch_norm(const NormForward &a, bool phase, bool quant, bool held, int sm_count,
                        cudaStream_t s) {
  return quant ? launch_form<F32, VEC, true>(a, phase, held, sm_count, s)
               : launch_form<F32, VEC, false>(a, phase, held, sm_count, s);
}

template <bool F32, bool VEC, bool RES>
cudaError_t launch_drop_chunks(const NormForward &a, int sm_count, cudaStream_t s) {
  const int64_t chunks = (a.cols + kChunk - 1) / kChunk;
  int lg = 5;
  if (VEC)
    while (lg > 0 && (8 << lg >> 1) >= a.cols) --lg;
  // several chunks a warp: their loads are in flight together (us with 1, 2, 4: bf16
  // [16384, 4096] 57.0, 49.8, 47.0); few in all, or fp32 (39.8, 40.1, 40.3 at [8192, 4096]): one
  const int units = !F32 && a.rows * chunks >= 64 * static_cast<int64_t>(sm_count) ? 4 : 1;
  const bool rows4 = units == 4 && chunks <= 2;
  const int W = static_cast<int>(rows4 ? chunks : std::min<int64_t>(8, (chunks + units - 1) / units)), R = 8 / W;
  const int64_t runs = (chunks + W * units - 1) / (W * units);
  const int64_t per = (static_cast<int64_t>(R) << (5 - lg)) * (rows4 ? units : 1);
  const dim3 grid(static_cast<unsigned>((a.rows + per - 1) / per * runs)), block(32 * W, R);
  const unsigned n = static_cast<unsigned>(runs);
  if constexpr (!F32) {
    if (rows4) return launch_k(dropout_chunks<F32, VEC, 4, true, RES>, grid, block, 0, s, 0, a, n, lg);
    if (units == 4) return launch_k(dropout_chunks<F32, VEC, 4, false, RES>, grid, block, 0, s, 0, a, n, lg);
  }
  return launch_k(dropout_chunks<F32, VEC, 1, false, RES>, grid, block, 0, s, 0, a, n, lg);
}

template <bool F32, int NU, bool RES>
cudaError_t launch_drop_units_of(const NormForward &a, int64_t units, cudaStream_t s) {
  const int64_t per = 8 * NU * 31;
  return launch_k(dropout_units<F32, NU, RES>, dim3(static_cast<unsigned>((a.rows * units + per - 1) / per)), dim3(256),
                  0, s, 0, a, static_cast<int>(units));
}

template <bool F32, bool RES>
cudaError_t launch_drop_units(const NormForward &a, int sm_count, cudaStream_t s) {
  // the furthest into a unit that a row starts
  const int64_t ld = a.ldx, most = a.rows == 1 || ld % 8 == 0 ? 0 : ld % 4 == 0 ? 4 : ld % 2 == 0 ? 6 : 7;
  const int64_t units = (a.cols - 1 + most) / 8 + 1;
  // spans a warp, us with 1, 2, 4: fp32 [8192, 4097] 40.4, 47.5, -; bf16 with a residual [16384,
  // 4097] -, 72.6, 68.9 (63.6 now); few in all: one
  if constexpr (!F32)
    if (a.rows * units >= 64 * 31 * static_cast<int64_t>(sm_count)) return launch_drop_units_of<F32, 4, RES>(a, units, s);
  return launch_drop_units_of<F32, 1, RES>(a, units, s);
}

template <bool F32, bool RES>
cudaError_t launch_drop(const NormForward &a, bool vec, bool phase, int sm_count, cudaStream_t s) {
  if (vec) return launch_drop_chunks<F32, true, RES>(a, sm_count, s);
  if (phase && a.cols <= (INT64_C(1) << 30))  // 32-bit columns, up to 7 past the row
    return launch_drop_units<F32, RES>(a, sm_count, s);
  return launch_drop_chunks<F32, false, RES>(a, sm_count, s);
}

}  // namespace

bool rmsnorm_held_ok(int64_t cols) { return cols <= kChunk * kHeldChunks; }

cudaError_t launch_rmsnorm(const NormForward &a, bool f32, bool vec, bool phase, bool quant, bool held,
                           int sm_count, cudaStream_t s) {
  if (f32)
    return vec ? launch_norm<true, true>(a, phase, quant, held, sm_count, s)
               : launch_norm<true, false>(a, phase, quant, held, sm_count, s);
  return vec ? launch_norm<false, true>(a, phase, quant, held, sm_count, s)
             : launch_norm<false, false>(a, phase, quant, held, sm_count, s);
}

cudaError_t launch_dropout(const NormForward &a, bool f32, bool vec, bool phase, int sm_count,
                           cudaStream_t s) {
  if (a.residual != nullptr)
    return f32 ? launch_drop<true, true>(a, vec, phase, sm_count, s) : launch_drop<false, true>(a, vec, phase, sm_count, s);
  return f32 ? launch_drop<true, false>(a, vec, phase, sm_count, s) : launch_drop<false, false>(a, vec, phase, sm_count, s);
}

}  // namespace fr
