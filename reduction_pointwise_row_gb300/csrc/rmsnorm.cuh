// Pieces shared by the kernels of a residual block's row operators (dropout, the
// root-mean-square norm and its gradient): rows read and written in chunks of
// 256 columns a warp, and the dropout mask.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace fr {

// ---- rows in chunks of 256 columns a warp --------------------------------------
// A lane holds 8 elements of a chunk.  Aligned rows (VEC): the 8 consecutive ones
// from 8 lane on, one 16-byte (bf16) or 32-byte (fp32) access.  Other rows: columns
// lane, 32 + lane, ... 224 + lane, an element an access, which needs no alignment and
// keeps a warp's accesses adjacent.
constexpr int kChunk = 256;

template <bool F32>
struct Lane8 {
  static constexpr int NW = F32 ? 8 : 4;
  uint32_t w[NW];  // fp32 values, or bf16 pairs (element 2i in the low half of w[i])
  __device__ __forceinline__ float at(int j) const {
    if constexpr (F32) return __uint_as_float(w[j]);
    else return (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
  }
  // rounds v to the type (nearest even)
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      if constexpr (F32) w[i] = __float_as_uint(v[i]);
      else w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
  // elements before `lo` and from `hi` on become 0
  __device__ __forceinline__ void clip(int lo, int hi) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= lo && j < hi) continue;
      if constexpr (F32) w[j] = 0;
      else w[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = 0;
  }
};

// Column (within the row) of a lane's element j of chunk c.
template <bool VEC>
__device__ __forceinline__ int lane_col(int c, int lane, int j) {
  return c * kChunk + (VEC ? lane * 8 + j : j * 32 + lane);
}

// A lane's elements of chunk c of the row at `row`; 0 past the row's end.
// KEEP: the row is read again soon (ordinary caching), else once.
template <bool F32, bool VEC, bool KEEP = false>
__device__ __forceinline__ Lane8<F32> load8(const void *row, int c, int lane, int cols) {
  constexpr int ES = F32 ? 4 : 2;
  Lane8<F32> v;
  if constexpr (VEC) {
    const int col = c * kChunk + lane * 8;
    const char *p = static_cast<const char *>(row) + static_cast<int64_t>(col) * ES;
    if (col >= cols) {
      v.zero();
    } else if constexpr (F32) {
      const V8 u = KEEP ? ld_keep_v8(p) : ld_stream_v8(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v.w[i] = u.w[i];
    } else {
      const uint4 u = KEEP ? ld_keep_u4(p) : ld_once_u4(p);
      v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    }
  } else {
    const int first = lane_col<false>(c, lane, 0), left = cols - first;
    const char *p = static_cast<const char *>(row) + static_cast<int64_t>(first) * ES;
    const auto ld = [&](int j) -> uint32_t {
      if constexpr (F32) return __float_as_uint(ld_stream_f32(reinterpret_cast<const float *>(p + 32 * j * ES)));
      else return ld_stream_u16(p + 32 * j * ES);
    };
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = 32 * j < left ? ld(j) : 0;
#pragma unroll
    for (int i = 0; i < Lane8<F32>::NW; ++i) v.w[i] = F32 ? e[i] : (e[2 * i] | (e[2 * i + 1] << 16));
  }
  return v;
}

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void *row, int c, int lane, int cols, const Lane8<F32> &v) {
  constexpr int ES = F32 ? 4 : 2;
  if constexpr (VEC) {
    const int col = c * kChunk + lane * 8;
    if (col >= cols) return;
    char *p = static_cast<char *>(row) + static_cast<int64_t>(col) * ES;
    if constexpr (F32) {
      V8 u;
#pragma unroll
      for (int i = 0; i < 8; ++i) u.w[i] = v.w[i];
      st_stream_v8(p, u);
    } else {
      st_stream_u4(p, make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]));
    }
  } else {
    const int first = lane_col<false>(c, lane, 0), left = cols - first;
    char *p = static_cast<char *>(row) + static_cast<int64_t>(first) * ES;
    const auto st = [&](int j) {
      if constexpr (F32) st_stream_f32(reinterpret_cast<float *>(p + 32 * j * ES), __uint_as_float(v.w[j]));
      else st_stream_u16(p + 32 * j * ES, static_cast<uint16_t>((j & 1) ? v.w[j >> 1] >> 16 : v.w[j >> 1]));
    };
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * j < left) st(j);
  }
}

// A lane's 8 values of a vector over the columns (gamma), 0 past its end.
template <bool VEC>
__device__ __forceinline__ void load_cols8(float (&g)[8], const float *p, int c, int lane,
                                           int cols) {
  if constexpr (VEC) {
    const int col = c * kChunk + lane * 8;
    if (col < cols) {
      const V8 u = ld_keep_v8(p + col);  // (two 16-byte loads would each touch every sector)
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __uint_as_float(u.w[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 0.0f;
    }
  } else {
    const int first = lane_col<false>(c, lane, 0), left = cols - first;
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 32 * j < left ? ld_keep_f32(p + first + 32 * j) : 0.0f;
  }
}

// ---- the dropout mask -----------------------------------------------------------
// Element (r, c) has the 16-bit half c mod 8 of the Philox4x32 block (7 rounds: the
// fewest that pass every test of BigCrush; Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011) of counter (c / 8, r, offset low,
// offset high) and key seed; it is dropped where that half is below 65536 p.  A lane
// of an aligned chunk needs one block for its 8 elements.  16 bits and 7 rounds
// because the rounds' wide products, not memory, bound dropout alone: bf16 [32768,
// 4096], 86 us; with 32 bits an element 100, with 10 rounds 100, with both 121 (a
// copy of the same size: 80).
struct Mask {
  uint32_t k0, k1, o0, o1;  // key and offset
  uint32_t limit;           // (t << 16) - 1 for threshold t in 1 .. 65536
  float factor;             // 65536 / (65536 - t) for the elements that stay
};

__device__ __forceinline__ Mask mask_of(const DropSpec &d) {
  int64_t seed, offset;
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(seed) : "l"(d.rng) : "memory");
  asm volatile("ld.global.b64 %0, [%1];" : "=l"(offset) : "l"(d.rng + 1) : "memory");
  const uint64_t s = static_cast<uint64_t>(seed);
  const uint64_t o = static_cast<uint64_t>(offset) + static_cast<uint64_t>(d.site);
  return Mask{static_cast<uint32_t>(s), static_cast<uint32_t>(s >> 32), static_cast<uint32_t>(o),
              static_cast<uint32_t>(o >> 32), d.limit, d.factor};
}

// The four words of a block.
__device__ __forceinline__ uint4 philox7(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                         uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ (k0 + i * 0x9E3779B9u);
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ (k1 + i * 0xBB67AE85u);
    c3 = static_cast<uint32_t>(a);
  }
  return make_uint4(c0, c1, c2, c3);
}

// The block of a lane's aligned chunk c of a row.
__device__ __forceinline__ uint4 block_of(const Mask &m, uint32_t row, int c, int lane) {
  return philox7(static_cast<uint32_t>(c * 32 + lane), row, m.o0, m.o1, m.k0, m.k1);
}

// v[j] = kept ? v[j] * factor : 0 for a lane's elements of a chunk, given its block b.
// Every lane of the warp takes part.  A dropped element is 0 whatever it holds.
template <bool VEC>
__device__ __forceinline__ void drop8_by(float (&v)[8], const Mask &m, const uint4 &b, int lane) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a half above the limit in the upper 16 bits: kept
      v[2 * i] = (w[i] << 16) > m.limit ? v[2 * i] * m.factor : 0.0f;
      v[2 * i + 1] = w[i] > m.limit ? v[2 * i + 1] * m.factor : 0.0f;
    }
  } else {
    // element j is column 32 j + lane: half lane % 8 of the block of lane 4 j + lane / 8
    uint32_t mine = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = (e & 1) ? w[e >> 1] : w[e >> 1] << 16;
      const uint32_t kept = __ballot_sync(0xffffffffu, h > m.limit);
      if ((lane & 7) == e) mine = kept;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = (mine >> (4 * j + (lane >> 3))) & 1u ? v[j] * m.factor : 0.0f;
  }
}

template <bool VEC>
__device__ __forceinline__ void drop8(float (&v)[8], const Mask &m, uint32_t row, int c, int lane) {
  drop8_by<VEC>(v, m, block_of(m, row, c, lane), lane);
}

// ---- rows in phase ------------------------------------------------------------------
// Rows that start at element `phase` (0 .. 7) of an aligned 8-element unit: lane l of
// chunk c holds the columns from 256 c + 8 l - phase on, one aligned unit; the first and
// the last unit of a row lie partly outside it.

// Elements from the start of row `row` to the end of its matrix (or more than a row has).
__device__ __forceinline__ int elements_left(int64_t rows, int64_t row, int64_t ld, int cols) {
  const int64_t n = (rows - 1 - row) * ld;
  return n >= 8 ? INT32_MAX : static_cast<int>(n) + cols;
}

// The unit from column `col` on of the row at `row`, as it lies in memory: elements
// outside the row are its neighbours', to be clipped.  A matrix's first row has no head
// (its base is aligned); what lies past the matrix's end, `left` elements on, is not read.
template <bool F32>
__device__ __forceinline__ Lane8<F32> load_unit(const char *row, int col, int cols, int left) {
  constexpr int ES = F32 ? 4 : 2;
  Lane8<F32> v;
  v.zero();
  const char *p = row + static_cast<int64_t>(col) * ES;
  if (col < cols && col <= left - 8) {
    if constexpr (F32) {
      const V8 u = ld_stream_v8(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) v.w[i] = u.w[i];
    } else {
      const uint4 u = ld_once_u4(p);
      v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    }
  } else if (col < cols) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (col + j >= cols) continue;
      if constexpr (F32) v.w[j] = __float_as_uint(ld_stream_f32(reinterpret_cast<const float *>(p) + j));
      else v.w[j >> 1] |= static_cast<uint32_t>(ld_stream_u16(p + 2 * j)) << (16 * (j & 1));
    }
  }
  return v;
}

template <int T>
__device__ __forceinline__ void cut8(float (&g)[8], const V8 &a, const V8 &b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] = __uint_as_float(j + T < 8 ? a.w[(j + T) & 7] : b.w[(j + T) & 7]);
}

// The 8 values from column `col` on of a 32-byte aligned vector over the columns, 0
// outside it: the two aligned 32-byte pieces that hold them, cut at the same place in
// every lane (rows start at one phase), instead of 8 scattered values a lane.
__device__ __forceinline__ void load_cols_unit(float (&g)[8], const float *p, int col, int cols) {
  const int t = col & 7, first = col - t;
  if (first >= 0 && first + 16 <= cols) {
    const V8 a = ld_keep_v8(p + first), b = ld_keep_v8(p + first + 8);
    switch (t) {
      case 0: cut8<0>(g, a, b); break;
      case 1: cut8<1>(g, a, b); break;
      case 2: cut8<2>(g, a, b); break;
      case 3: cut8<3>(g, a, b); break;
      case 4: cut8<4>(g, a, b); break;
      case 5: cut8<5>(g, a, b); break;
      case 6: cut8<6>(g, a, b); break;
      default: cut8<7>(g, a, b); break;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      g[j] = col + j >= 0 && col + j < cols ? ld_keep_f32(p + col + j) : 0.0f;
  }
}

// Writes the elements of a unit from column `col` on that are within the row.
template <bool F32, bool PH>
__device__ __forceinline__ void store_unit(char *row, int col, int cols, const Lane8<F32> &v) {
  constexpr int ES = F32 ? 4 : 2;
  if (col >= cols) return;
  char *p = row + static_cast<int64_t>(col) * ES;
  if (!PH || (col >= 0 && col + 8 <= cols)) {
    if constexpr (F32) {
      V8 u;
#pragma unroll
      for (int i = 0; i < 8; ++i) u.w[i] = v.w[i];
      st_stream_v8(p, u);
    } else {
      st_stream_u4(p, make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (col + j < 0 || col + j >= cols) continue;
    if constexpr (F32) st_stream_f32(reinterpret_cast<float *>(p) + j, __uint_as_float(v.w[j]));
    else st_stream_u16(p + 2 * j, static_cast<uint16_t>((j & 1) ? v.w[j >> 1] >> 16 : v.w[j >> 1]));
  }
}

// Which elements of block `b` of a row stay: bit e of element e.  A half in the upper 16 bits
// is above the limit where it carries over 32 bits with the limit's complement, and the
// carry is shifted in (dropout of bf16 [16384, 4097] 57.1 us, with comparisons 60.7).
__device__ __forceinline__ uint32_t kept_bits(const Mask &m, uint32_t row, uint32_t b) {
  const uint4 r = philox7(b, row, m.o0, m.o1, m.k0, m.k1);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    uint32_t sum;
    asm("add.cc.u32 %1, %2, %4;\n\taddc.u32 %0, %0, %0;\n\t"
        "add.cc.u32 %1, %3, %4;\n\taddc.u32 %0, %0, %0;"
        : "+r"(bits), "=&r"(sum)
        : "r"(w[i]), "r"(w[i] << 16), "r"(~m.limit));
  }
  return bits;
}

// The kept bits of the block before a row's chunk c (none before its first).
__device__ __forceinline__ uint32_t kept_before(const Mask &m, uint32_t row, int c) {
  return c > 0 ? kept_bits(m, row, static_cast<uint32_t>(c * 32 - 1)) : 0;
}

// drop8 for a lane's unit of a row in phase: its first `phase` elements belong to the
// block before its lane's, lane 0's to the one with the kept bits `before`, which become
// those before the next chunk.
__device__ __forceinline__ void drop8_phase(float (&v)[8], const Mask &m, uint32_t row, int c,
                                            int lane, int phase, uint32_t &before) {
  const uint32_t own = kept_bits(m, row, static_cast<uint32_t>(c * 32 + lane));
  uint32_t prev = __shfl_up_sync(0xffffffffu, own, 1);
  if (lane == 0) prev = before;
  before = __shfl_sync(0xffffffffu, own, 31);
  const uint32_t bits = (prev | own << 8) >> (8 - phase);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = bits >> j & 1u ? v[j] * m.factor : 0.0f;
}

// ---- 16-byte units ------------------------------------------------------------------
// A lane's 16 bytes of a row: E = 8 elements of bf16, 4 of fp32.
template <bool F32>
struct Unit {
  static constexpr int E = F32 ? 4 : 8;
  uint32_t w[4];
  __device__ __forceinline__ uint64_t pair(int k) const {  // elements 2 k and 2 k + 1
    if constexpr (F32) return pack_u32x2(w[2 * k], w[2 * k + 1]);
    else return pack_f32x2(bf16_lo(w[k]), bf16_hi(w[k]));
  }
  __device__ __forceinline__ void set(const float (&v)[E]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) w[i] = __float_as_uint(v[i]);
      else w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
  // elements before `lo` and from `hi` on become 0
  __device__ __forceinline__ void clip(int lo, int hi) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (j >= lo && j < hi) continue;
      if constexpr (F32) w[j] = 0;
      else w[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    }
  }
  // writes the elements from column `col` of `row` on that are within it; WHOLE: all are
  // or none
  template <bool WHOLE>
  __device__ __forceinline__ void store(char *row, int col, int cols) const {
    constexpr int ES = 16 / E;
    if (col >= cols) return;
    char *p = row + static_cast<int64_t>(col) * ES;
    if (WHOLE || (col >= 0 && col + E <= cols)) {
      st_stream_u4(p, make_uint4(w[0], w[1], w[2], w[3]));
      return;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (col + j < 0 || col + j >= cols) continue;
      if constexpr (F32) st_stream_f32(reinterpret_cast<float *>(p) + j, __uint_as_float(w[j]));
      else st_stream_u16(p + 2 * j, static_cast<uint16_t>((j & 1) ? w[j >> 1] >> 16 : w[j >> 1]));
    }
  }
};

// Which of a row's elements E k .. E k + E - 1 stay, bit by bit.
template <int E>
__device__ __forceinline__ uint32_t kept_group(const Mask &m, uint32_t row, int k) {
  if constexpr (E == 8) return kept_bits(m, row, static_cast<uint32_t>(k));
  return kept_bits(m, row, static_cast<uint32_t>(k >> 1)) >> (4 * (k & 1)) & 15u;
}

// Dropout of a lane's unit of aligned rows, group k of its row.
template <int E>
__device__ __forceinline__ void drop_unit(float (&v)[E], const Mask &m, uint32_t row, int k) {
  if constexpr (E == 8) {
    drop8<true>(v, m, row, k >> 5, k & 31);
  } else {
    const uint32_t bits = kept_group<E>(m, row, k);
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = bits >> j & 1u ? v[j] * m.factor : 0.0f;
  }
}

// The same for rows in phase, the lanes of a warp holding groups k after one another: a
// lane's first `phase` elements belong to the group before its own, lane 0's to the one
// with the kept bits `before`, which become those of lane 31's.
template <int E>
__device__ __forceinline__ void drop_unit_phase(float (&v)[E], const Mask &m, uint32_t row, int k,
                                                int lane, int phase, uint32_t &before) {
  const uint32_t own = kept_group<E>(m, row, k);
  uint32_t prev = __shfl_up_sync(0xffffffffu, own, 1);
  if (lane == 0) prev = before;
  before = __shfl_sync(0xffffffffu, own, 31);
  const uint32_t bits = (prev | own << E) >> (E - phase);
#pragma unroll
  for (int j = 0; j < E; ++j) v[j] = bits >> j & 1u ? v[j] * m.factor : 0.0f;
}

}  // namespace fr
