// Pieces shared by the kernels over rows of logits (log probabilities,
// distillation, their gradients and cross entropy's): a row's softmax
// statistics with the entropy's sum, order-preserving keys of logits, and the
// teacher's entries of a row.
#pragma once

#include "common.cuh"

namespace fr {

// Statistics of the elements seen so far, at a scale c = log2(e) / T:
//   m = max x,  l = sum exp((x - m) / T),  s = sum exp((x - m) / T) (x - m).
// LSE(x / T) = m / T + log l; at T = 1 the entropy of the softmax is
// log l - s / l and the mean logit under it m + s / l.
struct RowStat {
  float m, l, s;
};

// Differences below this have exp = 0; s takes max(x - m, kFarBelow), so an
// element of -inf adds 0 * kFarBelow = 0 to it and not 0 * -inf = NaN.
constexpr float kFarBelow = -1e30f;

__device__ __forceinline__ RowStat stat_empty() { return RowStat{-INFINITY, 0.0f, 0.0f}; }

__device__ __forceinline__ RowStat stat_merge(RowStat a, RowStat b, float c) {
  const float M = max_nan(a.m, b.m);
  if (M == -INFINITY) return stat_empty();
  const float da = a.m - M, db = b.m - M;
  const float fa = ex2(da * c), fb = ex2(db * c);
  const float sa = fmaf(a.l, fmaxf(da, kFarBelow), a.s);
  const float sb = fmaf(b.l, fmaxf(db, kFarBelow), b.s);
  return RowStat{M, __fadd_rn(__fmul_rn(a.l, fa), __fmul_rn(b.l, fb)),
                 __fadd_rn(__fmul_rn(fa, sa), __fmul_rn(fb, sb))};
}

// The maximum of a warp's values (NaN if there is one), in every lane.
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// Every lane gets the merge of the warp's statistics: the common maximum first,
// then one rescaling a lane and two sums.
__device__ __forceinline__ RowStat warp_stat(RowStat v, float c) {
  const float M = warp_max(v.m);
  if (M == -INFINITY) return stat_empty();
  const float d = v.m - M, f = ex2(d * c);
  return RowStat{M, warp_sum(v.l * f), warp_sum(f * fmaf(v.l, fmaxf(d, kFarBelow), v.s))};
}

// Every thread of a T-thread CTA gets the merge of all threads' statistics.
// `red` is used until the next barrier after the call.
template <int T>
__device__ __forceinline__ RowStat block_stat(RowStat v, float c, RowStat (&red)[T / 32]) {
  v = warp_stat(v, c);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_stat(lane < T / 32 ? red[lane] : stat_empty(), c);
}

// A vector of logits: element j (0 .. EPV - 1) as fp32, and the filler whose
// elements are all -inf.
template <bool F32>
struct Logits {
  static constexpr int ES = F32 ? 4 : 2;    // bytes per logit
  static constexpr int EPV = kVecBytes / ES;  // logits per 32-byte vector
  static constexpr uint32_t kNegInf = F32 ? 0xFF800000u : 0xFF80FF80u;
  __device__ static __forceinline__ float at(const V8 &v, int j) {
    if constexpr (F32) return __uint_as_float(v.w[j]);
    else return (j & 1) ? bf16_hi(v.w[j >> 1]) : bf16_lo(v.w[j >> 1]);
  }
  __device__ static __forceinline__ V8 filler() {
    V8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.w[j] = kNegInf;
    return v;
  }
  // the largest element (NaN if there is one)
  template <int N>
  __device__ static __forceinline__ float max(const V8 (&v)[N]) {
    if constexpr (F32) {
      float m = __uint_as_float(v[0].w[0]);
#pragma unroll
      for (int i = 1; i < 8 * N; ++i) m = max_nan(m, __uint_as_float(v[i / 8].w[i % 8]));
      return m;
    } else {
      uint32_t m = v[0].w[0];
#pragma unroll
      for (int i = 1; i < 8 * N; ++i) m = max_nan_bf16x2(m, v[i / 8].w[i % 8]);
      return max_nan(bf16_lo(m), bf16_hi(m));
    }
  }
  __device__ static __forceinline__ float max(const V8 &v) {
    const V8 one[1] = {v};
    return max(one);
  }
  // logit i of a row by an ordinary load
  __device__ static __forceinline__ float load(const void *row, int64_t i) {
    if constexpr (F32) return static_cast<const float *>(row)[i];
    else return bf16_to_f32(static_cast<const uint16_t *>(row)[i]);
  }
  __device__ static __forceinline__ void store(void *row, int64_t i, float v) {
    if constexpr (F32) static_cast<float *>(row)[i] = v;
    else static_cast<uint16_t *>(row)[i] = to_bf16(v);
  }
};

// Where |m c| is at most this, |m c rounded - m c| is at most 1/2: 2^rest stays close to
// 1 (from |m c| = 2^31 on it may leave the range of fp32) and costs s no digits.
constexpr float kFusedRange = 16777216.0f;

// Folds NV vectors with largest element cm into a thread's statistics; the
// entropy's sum (at T = 1) only with ENT.  Two partial sums of pairs per call are
// added to the running fp32 sums once, so a thread's chains of additions stay
// short.
//
// t = x c - m c takes one fused multiply-add per pair of logits: with mc the
// rounded product and rest = m c - mc exactly (one more fused multiply-add),
// x c - mc is rounded once, at its own size, and every exponential is too large
// by the same 2^rest, which is taken out of the sums.  Where that does not
// serve -- m c past kFusedRange, or an element at t = -inf, whose exp * t = 0 * -inf
// -- the sums are taken again from x - m with the far differences cut off.
// (Measured with the alternatives of a row off, bf16 [2432, 50257]: 7.0
// instructions a logit with x - m and the cut for every logit.)
template <bool F32, bool ENT, int NV>
__device__ __forceinline__ void stat_fold(RowStat &st, const V8 (&v)[NV], float cm, float c) {
  using L = Logits<F32>;
  if (!(cm <= st.m)) {
    const float M = max_nan(st.m, cm);
    const float dm = st.m - M, f = ex2(dm * c);
    if constexpr (ENT) st.s = f * fmaf(st.l, fmaxf(dm, kFarBelow), st.s);
    st.l *= f;
    st.m = M;
  }
  if (st.m == -INFINITY) {  // nothing but -inf so far
    st.l = st.s = 0.0f;
    return;
  }
  const uint64_t c2 = pack_f32x2(c, c);
  const float mc = st.m * c;
  if (fabsf(mc) <= kFusedRange) {
    const uint64_t nmc2 = pack_f32x2(-mc, -mc);
    uint64_t al[2] = {0, 0}, as[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int j = 0; j < L::EPV / 2; ++j) {
        const uint64_t t =
            fma_f32x2(pack_f32x2(L::at(v[k], 2 * j), L::at(v[k], 2 * j + 1)), c2, nmc2);
        const uint64_t e = pack_f32x2(ex2(f32x2_lo(t)), ex2(f32x2_hi(t)));
        al[j & 1] = add_f32x2(al[j & 1], e);
        if constexpr (ENT) as[j & 1] = fma_f32x2(e, t, as[j & 1]);
      }
    const float rest = fmaf(st.m, c, -mc), f = ex2(-rest);
    const uint64_t l2 = add_f32x2(al[0], al[1]);
    const float l = f32x2_lo(l2) + f32x2_hi(l2);
    if constexpr (ENT) {
      const uint64_t s2 = add_f32x2(as[0], as[1]);
      const float s = f32x2_lo(s2) + f32x2_hi(s2);
      if (s == s || l != l) {
        st.l = fmaf(f, l, st.l);
        st.s = fmaf(f * kLn2, fmaf(-rest, l, s), st.s);  // 1 / c = ln 2
        return;
      }
    } else {
      st.l = fmaf(f, l, st.l);
      return;
    }
  }
  const uint64_t m2 = pack_f32x2(st.m, st.m);
  uint64_t al = 0, as = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = 0; j < L::EPV / 2; ++j) {
      const uint64_t d = sub_f32x2(pack_f32x2(L::at(v[k], 2 * j), L::at(v[k], 2 * j + 1)), m2);
      const uint64_t t = mul_f32x2(d, c2);
      const uint64_t e = pack_f32x2(ex2(f32x2_lo(t)), ex2(f32x2_hi(t)));
      al = add_f32x2(al, e);
      if constexpr (ENT)
        as = fma_f32x2(e, pack_f32x2(fmaxf(f32x2_lo(d), kFarBelow),
                                     fmaxf(f32x2_hi(d), kFarBelow)), as);
    }
  st.l += f32x2_lo(al) + f32x2_hi(al);
  if constexpr (ENT) st.s += f32x2_lo(as) + f32x2_hi(as);
}

// ---- order-preserving keys ---------------------------------------------------

// a < b as numbers <=> key(a) < key(b); both zeros share a key; every NaN has
// the largest key.  0 is below the key of -inf.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);  // key of NaN: a NaN
}
// A logit with its place: larger logits first, equal ones by lower index.
__device__ __forceinline__ uint64_t place_key(uint32_t key, uint32_t index) {
  return (static_cast<uint64_t>(key) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ uint32_t place_index(uint64_t p) {
  return 0xFFFFFFFFu - static_cast<uint32_t>(p);
}

// ---- a row's teacher entries ---------------------------------------------------

constexpr int kTopPerLane = FR_TOP_MAX / 32;
static_assert(FR_TOP_MAX % 32 == 0, "a warp holds a row's entries, the same number a lane");

// Entries lane, lane + 32, ... of a row in the lanes of one warp: q = softmax of
// the live entries' z / T, and the student's logit at each.  An entry is live
// when its index is not negative.
struct Teacher {
  int64_t idx[kTopPerLane];  // -1: not live
  float q[kTopPerLane], logq[kTopPerLane], x[kTopPerLane];
  bool any;  // some live entry has weight (z not all -inf); the same in every lane
  bool bad;  // some index is past the row; the same in every lane
};

// The entries of a row as they are in memory, and the student's logits at them:
// two steps of loads, so that a caller can have others in flight between.
struct TeacherRaw {
  int64_t idx[kTopPerLane];
  float z[kTopPerLane], x[kTopPerLane];
};

__device__ __forceinline__ void teacher_fetch(TeacherRaw &t, const int64_t *index, const float *z,
                                              int k) {
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i) {
    const int e = (threadIdx.x & 31) + 32 * i;
    t.idx[i] = e < k ? index[e] : -1;
    t.z[i] = e < k ? z[e] : 0.0f;
  }
}

template <bool F32>
__device__ __forceinline__ void teacher_gather(TeacherRaw &t, const void *row, int64_t cols) {
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i)
    t.x[i] = t.idx[i] >= 0 && t.idx[i] < cols ? Logits<F32>::load(row, t.idx[i]) : 0.0f;
}

__device__ __forceinline__ Teacher teacher_finish(const TeacherRaw &raw, int64_t cols,
                                                  float temperature) {
  Teacher t;
  float zv[kTopPerLane], zm = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i) {
    t.idx[i] = raw.idx[i];
    t.x[i] = raw.x[i];
    zv[i] = t.idx[i] >= 0 ? raw.z[i] : -INFINITY;
    bad |= t.idx[i] >= cols;
    zm = max_nan(zm, zv[i]);
  }
  zm = warp_max(zm);
  t.bad = __any_sync(0xffffffffu, bad);
  t.any = zm != -INFINITY;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i) {
    const bool live = t.idx[i] >= 0;
    t.logq[i] = live && t.any ? (zv[i] - zm) / temperature : -INFINITY;
    t.q[i] = live && t.any ? expf(t.logq[i]) : 0.0f;
    sum += t.q[i];
  }
  sum = warp_sum(sum);
  const float logsum = logf(sum);
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i)
    if (t.idx[i] >= 0 && t.any) {
      t.q[i] /= sum;
      t.logq[i] -= logsum;
    }
  return t;
}

template <bool F32>
__device__ __forceinline__ Teacher teacher_load(const int64_t *index, const float *z, int k,
                                                const void *row, int64_t cols, float temperature) {
  TeacherRaw raw;
  teacher_fetch(raw, index, z, k);
  teacher_gather<F32>(raw, row, cols);
  return teacher_finish(raw, cols, temperature);
}

// T^2 sum q (log q - log p) with log p = (x - m) / T - log l, as sum q T (T (log q +
// log l) - (x - m)): x - m may be the type's lowest value, which 1 / T, or a sum without
// the weights or T, would take out of range.  Entries without weight add nothing,
// whatever the student gives them.
__device__ __forceinline__ float teacher_loss(const Teacher &t, const RowStat &st,
                                              float temperature) {
  const float logl = logf(st.l);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i)
    if (t.q[i] != 0.0f)
      sum += t.q[i] * temperature * (temperature * (t.logq[i] + logl) - (t.x[i] - st.m));
  sum = warp_sum(sum);
  if (t.bad) return __int_as_float(0x7fc00000);
  return t.any ? sum : 0.0f;
}

}  // namespace fr
