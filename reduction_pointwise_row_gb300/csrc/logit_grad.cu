// Gradients with respect to rows of logits, statistics and gradient in one
// call: of the log probability and the entropy of given tokens, of cross
// entropy, and of distillation from a teacher's top logits.
//
// With d_j = x_j - m, e_j = exp(d_j / T), p_j = e_j / l (logits.cuh):
//   token:    dx_j = g (delta_jt - p_j) - h p_j (d_j - s / l)
//             (g: the log probability's gradient, h: the entropy's; m + s / l
//             is the mean logit, and log p_j + H = x_j - that mean).  Cross
//             entropy is this with g = -dloss and no h.
//   distill:  dx_j = dloss T (p_j - Q_j), Q_j the teacher's weight on j (all
//             entries that name j added up).
// Every element is a row scalar times e_j, and a few elements a row (the token,
// the teacher's entries) differ: the row is written without them first, and
// after a barrier those elements are written again with their term, each from
// the logit read before the row was written (dlogits may be the logits).
//
// What bounds these kernels is the row's bytes, read once and written once.  The
// staged form keeps the row in shared memory between the two passes (the ring
// of bulk copies of "Stax (4)", section 9.8, with whole rows as its stages); the
// looped form streams it twice and relies on L2 for the second time, which
// misses for about half of it (bf16 [2048, 50257]: 411 MB of DRAM traffic, with
// 60 MB of the output still in L2, for 412 algorithmic).
#include "launch.h"
#include "logits.cuh"

namespace fr {
namespace {

constexpr int kT = 512;  // threads per CTA of the looped form
constexpr int kNV = 2;   // 32-byte vectors a thread folds at once

// An ordinary (coherent) 32-byte load: the row may be written by this kernel.
__device__ __forceinline__ V8 ld_v8(const void *p) {
  V8 v;
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]),
                 "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
               : "l"(p)
               : "memory");
  return v;
}

// What the elements of a row are computed from: with t = (x - m) c,
//   dx = 2^t (a + b max(t, kFar)).
// 2^t is 0 from kFar down, and the bound keeps b t finite where x is -inf.  Where
// |m c| <= kFusedRange, t is one fused multiply-add, x c - mc, larger than (x - m) c by
// rest = m c - mc (see stat_fold), which a and b take in.
constexpr float kFar = -200.0f;

template <bool B>
struct Flag {
  static constexpr bool value = B;
};

struct RowCoef {
  float m, c, mc, a, b;
  bool fused;
};

// From the row's statistics: dx = e (a + b (x - m) c) before the correction.
__device__ __forceinline__ RowCoef row_coef(const RowStat &st, float c, float a, float b) {
  RowCoef r{st.m, c, st.m * c, a, b, false};
  r.fused = fabsf(r.mc) <= kFusedRange;
  if (r.fused) {
    const float rest = fmaf(st.m, c, -r.mc), f = ex2(-rest);
    r.a = fmaf(-b, rest, a) * f;
    r.b = b * f;
  }
  return r;
}

// The coefficients of a row with the token's gradient g and the entropy's h.
__device__ __forceinline__ RowCoef token_coef(const RowStat &st, float c, float g, float h,
                                              bool has_h) {
  const float inv = 1.0f / st.l;
  if (!has_h) return row_coef(st, c, -g * inv, 0.0f);
  return row_coef(st, c, (h * (st.s * inv) - g) * inv, -h * inv * kLn2);  // c = log2(e) here
}

template <bool HAS_B>
__device__ __forceinline__ float grad_scalar(float x, const RowCoef &r) {
  const float t = r.fused ? fmaf(x, r.c, -r.mc) : (x - r.m) * r.c;
  return ex2(t) * (HAS_B ? fmaf(r.b, fmaxf(t, kFar), r.a) : r.a);
}

// FUSED is r.fused, a branch around the caller's loop.
template <bool F32, bool HAS_B, bool FUSED>
__device__ __forceinline__ V8 grad_vector(const V8 &x, const RowCoef &r) {
  using L = Logits<F32>;
  const uint64_t c2 = pack_f32x2(r.c, r.c), a2 = pack_f32x2(r.a, r.a), b2 = pack_f32x2(r.b, r.b);
  const uint64_t nmc2 = pack_f32x2(-r.mc, -r.mc), m2 = pack_f32x2(r.m, r.m);
  V8 o;
#pragma unroll
  for (int j = 0; j < L::EPV / 2; ++j) {
    const uint64_t v = pack_f32x2(L::at(x, 2 * j), L::at(x, 2 * j + 1));
    const uint64_t t = FUSED ? fma_f32x2(v, c2, nmc2) : mul_f32x2(sub_f32x2(v, m2), c2);
    const uint64_t e = pack_f32x2(ex2(f32x2_lo(t)), ex2(f32x2_hi(t)));
    uint64_t f = a2;
    if constexpr (HAS_B)
      f = fma_f32x2(b2, pack_f32x2(fmaxf(f32x2_lo(t), kFar), fmaxf(f32x2_hi(t), kFar)), a2);
    const uint64_t y = mul_f32x2(e, f);
    if constexpr (F32) {
      o.w[2 * j] = __float_as_uint(f32x2_lo(y));
      o.w[2 * j + 1] = __float_as_uint(f32x2_hi(y));
    } else {
      o.w[j] = pack_bf16x2(f32x2_lo(y), f32x2_hi(y));
    }
  }
  return o;
}

// A row's gradient is all zeros (an ignored row, a row without teacher) or all
// NaN (a target past the row) before anything is read of it.
enum RowKind { kRowGrad = 0, kRowZero = 1, kRowNan = 2, kNoRow = 3 };

// What a token makes of its row.  An ignored one leaves the entropy's gradient (HAS_B).
template <bool HAS_B>
__device__ __forceinline__ int token_kind(const LogitsBackward &a, int64_t token) {
  if (!a.token) return kRowGrad;
  if (token == a.ignore_index) return HAS_B ? kRowGrad : kRowZero;
  return token < 0 || token >= a.cols ? kRowNan : kRowGrad;
}

// A row's teacher entries in shared memory, by one warp.
struct TeacherShared {
  int32_t idx[FR_TOP_MAX];  // -1: no weight
  float q[FR_TOP_MAX], logq[FR_TOP_MAX], x[FR_TOP_MAX];
  float sum[FR_TOP_MAX];  // the weights of all entries that name idx
};
using EntryTable = uint16_t[256];

// Whether two of the warp's entries name the same element.  Each puts its number
// in the table at a hash of its index and looks who is there: an entry with the
// same index, or another index with the same hash, which is met by another
// round of those that lost.
__device__ __forceinline__ bool teacher_repeats(const TeacherShared &sh, int top,
                                                EntryTable &table) {
  const int lane = threadIdx.x & 31;
  uint32_t open = 0;
  bool repeats = false;
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i)
    if (lane + 32 * i < top && sh.idx[lane + 32 * i] >= 0) open |= 1u << i;
  while (__any_sync(0xffffffffu, open != 0)) {
#pragma unroll
    for (int i = 0; i < kTopPerLane; ++i)
      if ((open >> i) & 1) {
        const int32_t j = sh.idx[lane + 32 * i];
        table[(j ^ (j >> 8)) & 255] = static_cast<uint16_t>(lane + 32 * i);
      }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kTopPerLane; ++i)
      if ((open >> i) & 1) {
        const int32_t j = sh.idx[lane + 32 * i];
        const int e = table[(j ^ (j >> 8)) & 255];
        if (sh.idx[e] == j) {
          open &= ~(1u << i);
          repeats |= e != lane + 32 * i;
        }
      }
    __syncwarp();
  }
  return __any_sync(0xffffffffu, repeats);
}

__device__ __forceinline__ void teacher_share(const Teacher &t, int top, TeacherShared &sh,
                                              EntryTable &table) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kTopPerLane; ++i) {
    const int e = lane + 32 * i;
    sh.idx[e] = t.q[i] != 0.0f ? static_cast<int32_t>(t.idx[i]) : -1;
    sh.q[e] = sh.sum[e] = t.q[i];
    sh.logq[e] = t.logq[i];
    sh.x[e] = t.x[i];
  }
  __syncwarp();
  if (teacher_repeats(sh, top, table))
    for (int e = lane; e < top; e += 32) {
      const int32_t j = sh.idx[e];
      float sum = 0.0f;  // in the entries' order
      for (int n = 0; n < top; ++n) sum += sh.idx[n] == j ? sh.q[n] : 0.0f;
      sh.sum[e] = sum;
    }
  __syncwarp();
}

// The row's loss from its shared entries, in every lane of one warp (as the other
// teacher_loss, for its range).
__device__ __forceinline__ float teacher_loss(const TeacherShared &sh, int top, const RowStat &st,
                                              float temperature) {
  const float logl = logf(st.l);
  float sum = 0.0f;
  for (int e = threadIdx.x & 31; e < top; e += 32)
    if (sh.idx[e] >= 0)
      sum += sh.q[e] * temperature * (temperature * (sh.logq[e] + logl) - (sh.x[e] - st.m));
  return warp_sum(sum);
}

// Entry e's element: g (p - sum of its weights).
__device__ __forceinline__ float teacher_element(const TeacherShared &sh, int e, const RowStat &st,
                                                 float c, float g) {
  return g * (ex2((sh.x[e] - st.m) * c) * (1.0f / st.l) - sh.sum[e]);
}

// ---- held: a warp per row, the row in registers ----------------------------------------
//
// Rows of at most 8 KiB, 1 to 8 32-byte vectors a lane.  The staged form has a few
// us to do once a row, which such a row's bytes do not cover (us held / staged, bf16:
// 30000 x 1000 22.1 / 62.0; 30000 x 2048 38.9 / 80; 16000 x 4096 41.9 / 53.1, with 20
// teacher entries 58.8 / 72.5).  For longer rows a CTA holding the row in its registers
// was no faster than the staged form (8192 x 8192 47.4 / 45.2, 4096 x 30000 107 / 83).

constexpr int kRowWarps = 4;  // rows per CTA
constexpr int64_t kHeldVectors = 256;

template <bool F32, bool DISTILL, bool HAS_B, int NV, bool VEC>
__global__ void __launch_bounds__(32 * kRowWarps, NV > 4 ? 4 : NV > 2 ? 5 : NV > 1 ? 7 : 8)
logit_grad_held(LogitsBackward a) {
  pdl_enter();
  using L = Logits<F32>;
  __shared__ TeacherShared teachers[DISTILL ? kRowWarps : 1];
  __shared__ EntryTable tables[DISTILL ? kRowWarps : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp;
  if (row >= a.rows) return;
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  const float nan = __int_as_float(0x7fc00000);
  const unsigned char *pr = static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
  unsigned char *po = static_cast<unsigned char *>(a.dlogits) + row * a.ldd * L::ES;
  const RowSplit sp = row_split(pr, a.cols, L::ES);
  const int nvec = static_cast<int>(sp.nvec), v0 = sp.head * L::ES;
  // everything that the row is computed from, before any of it is overwritten
  const int64_t token = !DISTILL && a.token ? a.token[row] : -1;
  V8 v[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u)
    v[u] = lane + 32 * u < nvec ? ld_v8(pr + v0 + (lane + 32 * u) * kVecBytes) : L::filler();
  int si = -1;
  if (lane < sp.head) si = lane;
  else if (lane < sp.head + sp.tail) si = sp.head + nvec * L::EPV + (lane - sp.head);
  const float sx = si >= 0 ? L::load(pr, si) : -INFINITY;
  float g = 0.0f, h = 0.0f, xt = 0.0f;
  int kind = kRowGrad, own = -1;
  if constexpr (DISTILL) {
    g = a.dloss[row * a.dloss_stride] * a.temperature;
    const Teacher t = teacher_load<F32>(a.index + row * a.ldt, a.teacher + row * a.ldt, a.top, pr,
                                        a.cols, a.temperature);
    kind = t.bad ? kRowNan : t.any ? kRowGrad : kRowZero;
    teacher_share(t, a.top, teachers[warp], tables[warp]);
  } else {
    kind = token_kind<HAS_B>(a, token);
    if (kind == kRowGrad && a.token && token != a.ignore_index) {
      own = static_cast<int>(token);
      xt = L::load(pr, own);
      g = a.dloss[row * a.dloss_stride] * a.dloss_sign;
    }
    if constexpr (HAS_B) h = a.dentropy[row * a.dentropy_stride];
  }

  RowStat st = stat_empty();
  stat_fold<F32, HAS_B, NV>(st, v, L::max(v), c);
  if (sx != -INFINITY) st = stat_merge(st, RowStat{sx, 1.0f, 0.0f}, c);
  st = warp_stat(st, c);
  __syncwarp();  // every lane has read its part of the row
  if (kind == kRowNan && lane == 0) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
  const RowCoef r =
      DISTILL ? row_coef(st, c, g * (1.0f / st.l), 0.0f) : token_coef(st, c, g, h, HAS_B);
  const float fill = kind == kRowNan ? nan : 0.0f;
  const uint32_t fill_w = kind == kRowNan ? (F32 ? 0x7FC00000u : 0x7FC07FC0u) : 0;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    if (lane + 32 * u >= nvec) continue;
    V8 y;
    if (kind != kRowGrad) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y.w[j] = fill_w;
    } else if (r.fused) {
      y = grad_vector<F32, HAS_B, true>(v[u], r);
    } else {
      y = grad_vector<F32, HAS_B, false>(v[u], r);
    }
    if constexpr (VEC) {
      st_stream_v8(po + v0 + (lane + 32 * u) * kVecBytes, y);
    } else {
#pragma unroll
      for (int j = 0; j < L::EPV; ++j)
        L::store(po, sp.head + (lane + 32 * u) * L::EPV + j, L::at(y, j));
    }
  }
  if (si >= 0) L::store(po, si, kind == kRowGrad ? grad_scalar<HAS_B>(sx, r) : fill);
  // the elements with a term of their own come after the rest
  __syncwarp();
  float loss = fill;
  if (kind == kRowGrad) {
    if constexpr (DISTILL) {
      const TeacherShared &t = teachers[warp];
      for (int e = lane; e < a.top; e += 32)
        if (t.idx[e] >= 0) L::store(po, t.idx[e], teacher_element(t, e, st, c, g));
      if (a.loss) loss = teacher_loss(t, a.top, st, a.temperature);
    } else if (own >= 0) {
      if (lane == 0) L::store(po, own, grad_scalar<HAS_B>(xt, r) + g);
      loss = logf(st.l) - (xt - st.m);
    }
  }
  if (a.loss && lane == 0) a.loss[row] = loss;
}

template <bool F32, bool DISTILL, bool HAS_B, int NV>
cudaError_t launch_held(const LogitsBackward &a, bool vec, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.rows + kRowWarps - 1) / kRowWarps));
  const dim3 block(32 * kRowWarps);
  return vec ? launch_k(logit_grad_held<F32, DISTILL, HAS_B, NV, true>, grid, block, 0, s, 0, a)
             : launch_k(logit_grad_held<F32, DISTILL, HAS_B, NV, false>, grid, block, 0, s, 0, a);
}

// ---- looped: a CTA per row, the row streamed twice ---------------------------------

template <bool F32, bool DISTILL, bool HAS_B, bool VEC>
__global__ void __launch_bounds__(kT, 2) logit_grad_looped(LogitsBackward a) {
  pdl_enter();
  using L = Logits<F32>;
  __shared__ RowStat red[kT / 32];
  __shared__ TeacherShared sh[1];
  __shared__ EntryTable table;
  __shared__ int kind_s;
  const int tid = threadIdx.x;
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  const float nan = __int_as_float(0x7fc00000);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const unsigned char *pr = static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
    unsigned char *po = static_cast<unsigned char *>(a.dlogits) + row * a.ldd * L::ES;
    const RowSplit sp = row_split(pr, a.cols, L::ES);
    const int64_t vo = static_cast<int64_t>(sp.head) * L::ES;

    int64_t token = -1;
    float xt = 0.0f, g = 0.0f, h = 0.0f;
    if constexpr (DISTILL) {
      if (tid < 32) {
        const Teacher t = teacher_load<F32>(a.index + row * a.ldt, a.teacher + row * a.ldt, a.top,
                                            pr, a.cols, a.temperature);
        teacher_share(t, a.top, sh[0], table);
        if (tid == 0) {
          kind_s = t.bad ? kRowNan : t.any ? kRowGrad : kRowZero;
          if (t.bad) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
        }
      }
      g = a.dloss[row * a.dloss_stride] * a.temperature;
      __syncthreads();
    } else {
      if (a.token) token = a.token[row];
      if (tid == 0) kind_s = token_kind<HAS_B>(a, token);
      __syncthreads();
      if (a.token && (kind_s != kRowGrad || token == a.ignore_index)) {
        if (kind_s == kRowNan && tid == 0) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
        token = -1;
      }
      if (token >= 0) {
        xt = L::load(pr, token);
        g = a.dloss[row * a.dloss_stride] * a.dloss_sign;
      }
      if constexpr (HAS_B) h = a.dentropy[row * a.dentropy_stride];
    }
    const int kind = kind_s;

    if (kind != kRowGrad) {
      for (int64_t j = tid; j < a.cols; j += kT) L::store(po, j, kind == kRowNan ? nan : 0.0f);
      if (a.loss && tid == 0) a.loss[row] = kind == kRowNan ? nan : 0.0f;
      __syncthreads();
      continue;
    }

    int64_t si = -1;
    if (tid < sp.head) si = tid;
    else if (tid < sp.head + sp.tail) si = sp.head + sp.nvec * L::EPV + (tid - sp.head);
    RowStat st = stat_empty();
    if (si >= 0) {
      const float x = L::load(pr, si);
      if (x != -INFINITY) st = RowStat{x, 1.0f, 0.0f};
    }
    for (int64_t b = tid; b < sp.nvec; b += kT * kNV) {
      V8 v[kNV];
#pragma unroll
      for (int k = 0; k < kNV; ++k)
        v[k] = b + k * kT < sp.nvec ? ld_v8(pr + vo + (b + k * kT) * kVecBytes) : L::filler();
      stat_fold<F32, HAS_B, kNV>(st, v, L::max(v), c);
    }
    st = block_stat<kT>(st, c, red);

    const RowCoef r =
        DISTILL ? row_coef(st, c, g * (1.0f / st.l), 0.0f) : token_coef(st, c, g, h, HAS_B);
    if constexpr (DISTILL) {
      if (a.loss && tid < 32) {
        const float loss = teacher_loss(sh[0], a.top, st, a.temperature);
        if (tid == 0) a.loss[row] = loss;
      }
    } else if (a.loss && tid == 0) {
      a.loss[row] = logf(st.l) - (xt - st.m);
    }
    // in place, every element is read by the thread that writes it
    if constexpr (VEC) {
      if (si >= 0) L::store(po, si, grad_scalar<HAS_B>(L::load(pr, si), r));
      auto write = [&](auto fused) {
        for (int64_t b = tid; b < sp.nvec; b += kT) {
          const V8 x = ld_v8(pr + vo + b * kVecBytes);
          st_stream_v8(po + vo + b * kVecBytes, grad_vector<F32, HAS_B, fused.value>(x, r));
        }
      };
      if (r.fused) write(Flag<true>());
      else write(Flag<false>());
    } else {
      for (int64_t j = tid; j < a.cols; j += kT)
        L::store(po, j, grad_scalar<HAS_B>(L::load(pr, j), r));
    }
    __syncthreads();
    if constexpr (DISTILL) {
      if (tid < a.top && sh[0].idx[tid] >= 0)
        L::store(po, sh[0].idx[tid], teacher_element(sh[0], tid, st, c, g));
    } else if (tid == 0 && token >= 0) {
      L::store(po, token, grad_scalar<HAS_B>(xt, r) + g);
    }
    __syncthreads();
  }
}

// ---- staged: rows (or a cluster's runs of them) in a ring of bulk copies --------------
//
// The grid has a cluster of C CTAs for every row, and those that run take the rows of
// those not yet launched, one at a time, by cluster launch control.  With rows
// dealt out in advance the SMs that the memory system serves better were done 20-30 us
// before the last (xent_backward bf16 [4096, 50257]: 132-140 us).  CTA q of C holds the
// row's 16-byte units [n q / C, n (q + 1) / C) in one of the
// `nbuf` buffers of its ring.  All warps but the last few (the workers) fold the
// run's units into the statistics and, after the CTA's and the cluster's merge,
// write the gradient from shared memory; a worker goes on to the next row when its
// own part of a row is written, so one row's writing overlaps the next one's
// folding.  The last warps (the helpers) keep them supplied, each with every H-th
// row: a helper reads a row's token, upstream gradients, ragged ends and teacher
// entries H rows ahead, and when a row's workers are done it refills their buffer
// and writes the loss and the elements with a term of their own.  A helper's
// row takes 6-7 us with teacher entries (dependent loads and one warp's
// arithmetic), so one of them would be the bound: bf16 [4096, 50257] with 64
// entries, H = 1: 187 us.  Every wait is on an mbarrier and bounded; the cluster's
// statistics travel by st.async, which does not wait for the row's stores as a
// cluster barrier's release does.

constexpr int kMaxBufs = 4;
constexpr int kMaxThreads = 832;  // 72 registers a thread
constexpr int kMaxCluster = 8;
constexpr long long kWaitBudget = 1LL << 31;  // SM clocks, about one second
// A test-only build (-DFR_TEST_GRAD_WAIT_RUNS_OUT, =2: in the first CTA of a cluster alone)
// gives the wait for a CTA's first row no budget: it runs out whether or not the copy has
// landed.
#ifndef FR_TEST_GRAD_WAIT_RUNS_OUT
#define FR_TEST_GRAD_WAIT_RUNS_OUT 0
#endif
__device__ __forceinline__ long long row_budget(uint32_t k, uint32_t q) {
  constexpr int in = FR_TEST_GRAD_WAIT_RUNS_OUT;
  return in != 0 && k == 0 && (in == 1 || q == 0) ? 0 : kWaitBudget;
}

struct RowParams {
  int kind;
  int n;               // this CTA's units
  unsigned char *out;  // where the gradient of the first one goes
  int ends;            // this CTA's scalars of the row's head and tail: bits
  int token;           // of which the gradient has a term here, or -1
  float g, h, xt;      // upstream gradients, the token's logit
  float end[32];       // the head's and then the tail's logits
};

// Helper warps, and rows that they prepare ahead; a last warp finds the rows.
template <bool DISTILL>
constexpr int kHelpers = DISTILL ? 4 : 2;
constexpr int kRowRing = 32;  // rows whose numbers are kept
// Answers that are kept: a CTA asks for row j when its row j - 2 has landed, so its row
// j - 2 - nbuf is written and its peers sent their statistics of that one, which
// they had named: they have read all answers but the last nbuf + 2.
constexpr int kAnswers = 8;
static_assert(kMaxBufs + 2 < kAnswers, "no answer is overwritten before it is read");

template <bool DISTILL>
struct StagedShared {
  static constexpr int H = kHelpers<DISTILL>;
  uint64_t full[kMaxBufs];  // a buffer's copy has landed (or none was needed)
  uint64_t ready[H];        // a row's parameters are there
  uint64_t done[H];         // a row's workers have written it
  uint64_t merged[2];       // the cluster's statistics are there
  RowStat red[2][kMaxThreads / 32];
  float4 part[2][kMaxCluster];
  RowStat stat[H];  // the row's, for its helper
  RowParams par[H];
  TeacherShared teacher[DISTILL ? H : 1];
  EntryTable table[DISTILL ? H : 1];
  // the CTA's (cluster's) rows in turn, -1 past the last
  uint64_t named[kRowRing];  // row k's number is there
  int64_t row[kRowRing];
  // answers to the requests for another row, to all CTAs of the cluster
  uint4 answer[kAnswers];
  uint64_t answered[kAnswers];
  int gave_up;  // a wait ran out
};

struct UnitGeom {
  int head, tail;  // scalars before and after the units
  int u0, u1;      // this CTA's 16-byte units
  int64_t first;   // the first unit's byte offset in the row
};

// C = 1 << lg CTAs.
template <int ES>
__device__ __forceinline__ UnitGeom unit_geom(const unsigned char *pr, int64_t cols, uint32_t q,
                                              int lg) {
  const uint64_t s0 = reinterpret_cast<uint64_t>(pr), s1 = s0 + cols * ES;
  const uint64_t a0 = (s0 + 15) & ~uint64_t{15}, a1 = s1 & ~uint64_t{15};
  UnitGeom g;
  if (a1 <= a0) {  // fewer than 32 bytes: all scalars
    g.head = static_cast<int>(cols);
    g.tail = g.u0 = g.u1 = 0;
    g.first = 0;
    return g;
  }
  const uint64_t n = (a1 - a0) / 16;
  g.head = static_cast<int>((a0 - s0) / ES);
  g.tail = static_cast<int>((s1 - a1) / ES);
  g.first = static_cast<int64_t>(a0 - s0);
  g.u0 = static_cast<int>((n * q) >> lg);
  g.u1 = static_cast<int>((n * (q + 1)) >> lg);
  return g;
}

// Units i and i + step of the n at `buf` as one vector; CHECKED: -inf past the end.
template <bool F32, bool CHECKED>
__device__ __forceinline__ V8 lds_units(const unsigned char *buf, int i, int step, int n) {
  V8 v = Logits<F32>::filler();
  if (!CHECKED || i < n) {
    const uint4 x = lds_u4(buf + 16 * i);
    v.w[0] = x.x, v.w[1] = x.y, v.w[2] = x.z, v.w[3] = x.w;
  }
  if (!CHECKED || i + step < n) {
    const uint4 x = lds_u4(buf + 16 * (i + step));
    v.w[4] = x.x, v.w[5] = x.y, v.w[6] = x.z, v.w[7] = x.w;
  }
  return v;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A barrier of the workers; whether `any` holds in one of them, in all of them.
__device__ __forceinline__ bool worker_barrier(int workers, bool any) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.or.pred q, 1, %1, p;\n"
      " selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(workers), "r"(static_cast<uint32_t>(any))
      : "memory");
  return r != 0;
}

// A wait of at most `budget` SM clocks (0: it runs out at once), shorter where another
// of the CTA's waits ran out.  After that its thread waits for nothing any more, the
// CTA's helpers copy nothing more, and its workers stop.
__device__ __forceinline__ void wait_for(uint64_t *bar, uint32_t parity, bool &ok, int *gave_up,
                                         int *err, long long budget = kWaitBudget) {
  if (!ok) return;
  const long long t0 = clock64();
  while (budget == 0 || !mbar_try_wait(bar, parity)) {
    if (*reinterpret_cast<volatile int *>(gave_up) == 0) {
      if (budget > 0 && clock64() - t0 <= budget) continue;
      *reinterpret_cast<volatile int *>(gave_up) = 1;
      atomicCAS(err, 0, FR_DEVERR_TIMEOUT);
    }
    ok = false;
    return;
  }
}

// The same by a whole warp, whose lanes keep one `ok`.
__device__ __forceinline__ void warp_wait(uint64_t *bar, uint32_t parity, bool &ok, int *gave_up,
                                          int *err, long long budget = kWaitBudget) {
  wait_for(bar, parity, ok, gave_up, err, budget);
  ok = __all_sync(0xffffffffu, ok);
}

// Asks for a cluster of this grid that has not been launched, to be taken over by
// this one; the answer arrives in the shared memory of all its CTAs (at the same
// place), counted on their `bar`.  Not to be asked again once the answer was no.
// (multicast::cluster here is the answer's 16 bytes to the CTAs of the cluster; nothing is
// loaded from memory by it.)
__device__ __forceinline__ void request_cluster(uint4 *answer, uint64_t *bar, bool peers) {
  if (peers)
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".multicast::cluster::all.b128 [%0], [%1];" ::"r"(smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
  else
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes"
        ".b128 [%0], [%1];" ::"r"(smem_addr(answer)),
        "r"(smem_addr(bar))
        : "memory");
}
// The first CTA's x index of the cluster that was taken over, -1: none was left.
__device__ __forceinline__ int64_t requested_cluster(const uint4 *answer) {
  uint32_t taken, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 a;\n ld.shared.b128 a, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n selp.u32 %0, 1, 0, p;\n"
      " mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n}"
      : "=r"(taken), "=r"(x)
      : "r"(smem_addr(answer))
      : "memory");
  return taken ? static_cast<int64_t>(x) : -1;
}

template <bool F32, bool DISTILL, bool HAS_B, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, 1)
logit_grad_staged(LogitsBackward a, uint32_t buf_bytes, int nbuf, int lg) {
  pdl_enter();
  using L = Logits<F32>;
  constexpr int EPU = 16 / L::ES;  // logits per unit
  extern __shared__ __align__(128) unsigned char bufs[];  // [nbuf][buf_bytes]
  __shared__ StagedShared<DISTILL> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int H = kHelpers<DISTILL>;
  static_assert(2 * (H + kMaxBufs + 2) <= kRowRing, "no number is needed when its place is reused");
  const int workers = static_cast<int>(blockDim.x) - 32 * (H + 1), worker_warps = workers >> 5;
  const uint32_t C = 1u << lg;
  const uint32_t q = cluster_ctarank();
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  const float nan = __int_as_float(0x7fc00000);
  const unsigned char *logits = static_cast<const unsigned char *>(a.logits);
  if (tid == 0) {
    for (int b = 0; b < nbuf; ++b) mbar_init(&sh.full[b], 1);
    for (int i = 0; i < H; ++i) {
      mbar_init(&sh.ready[i], 1);
      mbar_init(&sh.done[i], worker_warps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sh.merged[i], 1);
    for (int i = 0; i < kRowRing; ++i) mbar_init(&sh.named[i], 1);
    for (int i = 0; i < kAnswers; ++i) mbar_init(&sh.answered[i], 1);
    sh.gave_up = 0;
    mbar_init_fence();
  }
  if (C > 1) {  // the peers' barriers are initialised before anything is sent
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  bool ok = true;

  if (warp == worker_warps + H) {
    if (lane == 0) {
      // names the rows: each when the row two before has landed, so that no CTA
      // takes many at the start (the row before, with one buffer: the row named
      // last must not land in the same one before this looks)
      const int back = nbuf > 1 ? 2 : 1;
      int64_t row = cluster_id_x();
      auto name = [&](int k) {
        sh.row[k % kRowRing] = row;
        mbar_arrive(&sh.named[k % kRowRing]);
      };
      int k = 0;
      while (row >= 0) {
        name(k++);
        if (k >= back)
          wait_for(&sh.full[(k - back) % nbuf], ((k - back) / nbuf) & 1, ok, &sh.gave_up, a.err);
        if (!ok && q == 0) {
          row = -1;  // no more requests
        } else {     // the others wait for what the first may still have asked for
          const int i = (k - 1) % kAnswers;
          fence_proxy_async_smem();  // the answer that was here before is read
          mbar_arrive_expect_tx(&sh.answered[i], 16);
          if (q == 0) request_cluster(&sh.answer[i], &sh.answered[i], C > 1);
          // to the end of its own budget, whoever else gave up: the answer is on its way
          ok = mbar_wait_bounded(&sh.answered[i], ((k - 1) / kAnswers) & 1, kWaitBudget);
          if (!ok) atomicCAS(a.err, 0, FR_DEVERR_TIMEOUT);
          row = ok ? requested_cluster(&sh.answer[i]) : -1;
          if (row > 0) row >>= lg;
        }
      }
      for (int i = 0; i < H + kMaxBufs + 1; ++i) name(k++);
    }
  } else if (warp >= worker_warps) {
    const int slot = warp - worker_warps;  // of the rows k = slot, slot + H, ... of the cluster
    const uint64_t policy = l2_evict_first_policy();
    int last_k = -1;  // the last row that this helper copied
    auto row_of = [&](int k) -> int64_t {
      warp_wait(&sh.named[k % kRowRing], (k / kRowRing) & 1, ok, &sh.gave_up, a.err);
      return ok ? sh.row[k % kRowRing] : -1;
    };
    // A copy of row k of the cluster into its buffer; no bytes: nothing is needed.
    struct Copy {
      const unsigned char *src;
      uint32_t bytes;
      int b;
    };
    auto copy_of = [&](int64_t row, int k, bool wanted) {
      if (row < 0) return Copy{nullptr, 0, k % nbuf};
      const unsigned char *pr = logits + row * a.ld * L::ES;
      const UnitGeom g = unit_geom<L::ES>(pr, a.cols, q, lg);
      return Copy{pr + g.first + 16 * static_cast<int64_t>(g.u0),
                  wanted ? 16u * static_cast<uint32_t>(g.u1 - g.u0) : 0, k % nbuf};
    };
    auto issue = [&](const Copy &c, int k) {
      if (lane != 0) return;
      if (c.bytes == 0) {
        mbar_arrive(&sh.full[c.b]);
        return;
      }
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&sh.full[c.b], c.bytes);
      bulk_copy_g2s(bufs + static_cast<size_t>(c.b) * buf_bytes, c.src, c.bytes, &sh.full[c.b],
                    policy);
      last_k = k;
    };
    auto token_of = [&](int64_t row) -> int64_t {
      return !DISTILL && a.token && row >= 0 ? a.token[row] : -1;
    };
    auto wanted = [&](int64_t token) {
      return DISTILL || token_kind<HAS_B>(a, token) == kRowGrad;
    };
    // A row's parameters are fetched (loads in flight) and, later, published.
    struct Fetched {
      TeacherRaw teacher;
      int64_t token;
      float g, h, xt, end;
    } f;
    auto fetch = [&](int64_t row, int64_t token) {
      if (row < 0) return;
      const unsigned char *pr = logits + row * a.ld * L::ES;
      const UnitGeom g = unit_geom<L::ES>(pr, a.cols, q, lg);
      f.token = token;
      f.g = f.h = f.xt = f.end = 0.0f;
      if constexpr (DISTILL)
        teacher_fetch(f.teacher, a.index + row * a.ldt, a.teacher + row * a.ldt, a.top);
      if (lane < g.head) f.end = L::load(pr, lane);
      else if (lane < g.head + g.tail) f.end = L::load(pr, a.cols - g.tail + lane - g.head);
      if constexpr (DISTILL) {
        f.g = a.dloss[row * a.dloss_stride];
        teacher_gather<F32>(f.teacher, pr, a.cols);
      } else {
        if (token >= 0 && token < a.cols && token != a.ignore_index) {
          f.xt = L::load(pr, token);
          f.g = a.dloss[row * a.dloss_stride];
        }
        if constexpr (HAS_B) f.h = a.dentropy[row * a.dentropy_stride];
      }
    };
    auto publish = [&](int64_t row) {
      RowParams &p = sh.par[slot];
      if (row < 0) {
        if (lane == 0) {
          p.kind = kNoRow;
          mbar_arrive(&sh.ready[slot]);
        }
        return;
      }
      const unsigned char *pr = logits + row * a.ld * L::ES;
      const UnitGeom g = unit_geom<L::ES>(pr, a.cols, q, lg);
      int kind, token = -1;
      if constexpr (DISTILL) {
        const Teacher t = teacher_finish(f.teacher, a.cols, a.temperature);
        kind = t.bad ? kRowNan : t.any ? kRowGrad : kRowZero;
        teacher_share(t, a.top, sh.teacher[slot], sh.table[slot]);
      } else {
        kind = token_kind<HAS_B>(a, f.token);
        if (kind == kRowGrad && a.token && f.token != a.ignore_index)
          token = static_cast<int>(f.token);
      }
      p.end[lane] = f.end;
      const bool end = lane < g.head ? q == 0 : lane < g.head + g.tail && q + 1 == C;
      const uint32_t ends = __ballot_sync(0xffffffffu, end);
      if (lane == 0) {
        p.kind = kind;
        p.n = g.u1 - g.u0;
        p.out = static_cast<unsigned char *>(a.dlogits) + row * a.ldd * L::ES + g.first +
                16 * static_cast<int64_t>(g.u0);
        p.ends = static_cast<int>(ends);
        p.token = token;
        p.g = f.g * (DISTILL ? a.temperature : a.dloss_sign);
        p.h = f.h;
        p.xt = f.xt;
        if (kind == kRowNan) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.ready[slot]);
    };
    auto first_copy = [&](int64_t row, int k) {
      if (row >= 0) issue(copy_of(row, k, wanted(token_of(row))), k);
    };
    int k = slot;  // of this helper's rows in turn
    int64_t row = row_of(k);
    if (k < nbuf) first_copy(row, k);
    fetch(row, token_of(row));
    publish(row);
    for (int i = k + H; i < nbuf; i += H) first_copy(row_of(i), i);
    for (uint32_t turn = 0; row >= 0; ++turn) {
      const int64_t refill = row_of(k + nbuf);
      const Copy next = copy_of(refill, k + nbuf, wanted(token_of(refill)));
      warp_wait(&sh.done[slot], turn & 1, ok, &sh.gave_up, a.err);
      // after a timeout nothing: the buffer's barrier may still count row k's copy, and
      // takes no second arrival until that has landed
      if (refill >= 0 && *reinterpret_cast<volatile int *>(&sh.gave_up) == 0) issue(next, k + nbuf);
      const RowParams &p = sh.par[slot];
      const RowStat st = sh.stat[slot];
      const unsigned char *pr = logits + row * a.ld * L::ES;
      unsigned char *po = static_cast<unsigned char *>(a.dlogits) + row * a.ldd * L::ES;
      const UnitGeom g = unit_geom<L::ES>(pr, a.cols, q, lg);
      // element j is written here if it is this CTA's: the first has the head (all of
      // a row without units), the last the tail
      int64_t lo = q == 0 ? 0 : (g.first + 16 * static_cast<int64_t>(g.u0)) / L::ES;
      int64_t hi = q + 1 == C ? a.cols : (g.first + 16 * static_cast<int64_t>(g.u1)) / L::ES;
      if (g.head == a.cols) {
        lo = q == 0 ? 0 : a.cols;
        hi = a.cols;
      }
      const bool grad = p.kind == kRowGrad;
      float loss = p.kind == kRowNan ? nan : 0.0f;
      RowCoef r{};
      if (grad)
        r = DISTILL ? row_coef(st, c, p.g * (1.0f / st.l), 0.0f)
                    : token_coef(st, c, p.g, p.h, HAS_B);
      if ((p.ends >> lane) & 1)
        L::store(po, lane < g.head ? lane : a.cols - g.tail + lane - g.head,
                 grad ? grad_scalar<HAS_B>(p.end[lane], r) : p.kind == kRowNan ? nan : 0.0f);
      __syncwarp();  // an end may be written again below
      if (grad) {
        if constexpr (DISTILL) {
          const TeacherShared &t = sh.teacher[slot];
          for (int e = lane; e < a.top; e += 32)
            if (t.idx[e] >= lo && t.idx[e] < hi)
              L::store(po, t.idx[e], teacher_element(t, e, st, c, p.g));
          if (a.loss && q == 0) loss = teacher_loss(t, a.top, st, a.temperature);
        } else if (p.token >= 0) {
          if (lane == 0 && p.token >= lo && p.token < hi)
            L::store(po, p.token, grad_scalar<HAS_B>(p.xt, r) + p.g);
          loss = logf(st.l) - (p.xt - st.m);
        }
      }
      if (a.loss && q == 0 && lane == 0) a.loss[row] = loss;
      k += H;
      row = row_of(k);
      fetch(row, token_of(row));
      __syncwarp();
      publish(row);
    }
    // Every copy was waited for by the workers, unless one gave up: then this
    // helper waits (bounded) for those it issued last, as none may outlive the CTA.
    if (*reinterpret_cast<volatile int *>(&sh.gave_up) != 0)
      for (int i = 0; last_k >= 0 && i < kMaxBufs; last_k -= H, ++i)
        mbar_wait_bounded(&sh.full[last_k % nbuf], (last_k / nbuf) & 1, kWaitBudget);
  } else {
    int b = 0, slot = 0;
    uint32_t lap = 0, turn = 0, k = 0;  // times through the buffers, the slots
    for (;; ++k) {
      const unsigned char *buf = bufs + static_cast<size_t>(b) * buf_bytes;
      const RowParams &par = sh.par[slot];
      auto ready = [&] {
        warp_wait(&sh.ready[slot], turn & 1, ok, &sh.gave_up, a.err);
        return ok ? par.kind : kNoRow;
      };
      // A row with a teacher is copied whatever its entries are: the first one, whose
      // entries have been looked at no earlier than its copy landed, is folded before
      // (bf16 [2048, 50257], 64 entries: 73.6 us, 72.7 so; every row so: 71.5, but in
      // clusters [1022, 65537] 59.8, 61.3).  Every row with a teacher adds its ragged
      // ends after its units: which rows are a CTA's first differs from run to run, and
      // the sums' order must not.
      const bool early = DISTILL && k == 0;
      int kind = kRowGrad, n = 0;
      if (early) {
        const UnitGeom g = unit_geom<L::ES>(
            logits + static_cast<int64_t>(cluster_id_x()) * a.ld * L::ES, a.cols, q, lg);
        n = g.u1 - g.u0;
      } else {
        kind = ready();
        if (kind != kNoRow) n = par.n;
      }
      if (kind != kNoRow)
        warp_wait(&sh.full[b], lap & 1, ok, &sh.gave_up, a.err, row_budget(k, q));
      if (!ok) kind = kNoRow;
      RowCoef r{};
      auto end_stat = [&](int kind) {  // this lane's scalar of the row's ends
        const bool has = warp == 0 && kind == kRowGrad && ((par.ends >> lane) & 1);
        const float x = has ? par.end[lane] : -INFINITY;
        return x != -INFINITY ? RowStat{x, 1.0f, 0.0f} : stat_empty();
      };
      RowStat st = DISTILL ? stat_empty() : end_stat(kind);
      if (kind == kRowGrad) {
        int i = tid;
        for (; i + 3 * workers < n; i += 4 * workers) {
          const V8 v[2] = {lds_units<F32, false>(buf, i, workers, n),
                           lds_units<F32, false>(buf, i + 2 * workers, workers, n)};
          stat_fold<F32, HAS_B, 2>(st, v, L::max(v), c);
        }
        for (; i < n; i += 2 * workers) {
          const V8 v[1] = {lds_units<F32, true>(buf, i, workers, n)};
          stat_fold<F32, HAS_B, 1>(st, v, L::max(v), c);
        }
        if (early) kind = ready();
        if constexpr (DISTILL) {
          const RowStat end = end_stat(kind);
          if (end.l != 0.0f) st = stat_merge(st, end, c);
        }
        st = warp_stat(st, c);
        if (lane == 0) sh.red[k & 1][warp] = st;
      }
      // every worker comes here whatever it saw, and all of them stop together
      if (worker_barrier(workers, !ok) || kind == kNoRow) break;
      if (kind == kRowGrad)
        st = warp_stat(lane < worker_warps ? sh.red[k & 1][lane] : stat_empty(), c);
      if (C > 1) {  // for every row, so that no CTA gets far ahead of its peers
        const int i = k & 1;
        if (warp == 0) {
          if (lane == 0) mbar_arrive_expect_tx(&sh.merged[i], 16u * C);
          __syncwarp();
          if (lane < C)
            st_async_f4(&sh.part[i][q], &sh.merged[i], lane,
                        make_float4(st.m, st.l, st.s, 0.0f));
        }
        // to the end of its own budget, whoever else gave up: a CTA comes to its end only
        // when what it sent has long landed, in a peer that may wait for it no more
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&sh.merged[i], (k >> 1) & 1, kWaitBudget));
        if (!ok) {
          *reinterpret_cast<volatile int *>(&sh.gave_up) = 1;
          atomicCAS(a.err, 0, FR_DEVERR_TIMEOUT);
        }
        const float4 o = lane < C ? sh.part[i][lane] : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
        if (kind == kRowGrad) st = warp_stat(RowStat{o.x, o.y, o.z}, c);
      }
      if (kind == kRowGrad) {
        if (tid == 0) sh.stat[slot] = st;
        r = DISTILL ? row_coef(st, c, par.g * (1.0f / st.l), 0.0f)
                    : token_coef(st, c, par.g, par.h, HAS_B);
      }
      unsigned char *out = par.out;
      if (kind == kRowGrad && VEC) {
        auto write = [&](auto fused) {
          int i = tid;
          for (; i + workers < n; i += 2 * workers) {
            const V8 y = grad_vector<F32, HAS_B, fused.value>(
                lds_units<F32, false>(buf, i, workers, n), r);
            st_stream_u4(out + 16 * i, make_uint4(y.w[0], y.w[1], y.w[2], y.w[3]));
            st_stream_u4(out + 16 * (i + workers), make_uint4(y.w[4], y.w[5], y.w[6], y.w[7]));
          }
          if (i < n) {
            const V8 y = grad_vector<F32, HAS_B, fused.value>(
                lds_units<F32, true>(buf, i, workers, n), r);
            st_stream_u4(out + 16 * i, make_uint4(y.w[0], y.w[1], y.w[2], y.w[3]));
          }
        };
        if (r.fused) write(Flag<true>());
        else write(Flag<false>());
      } else if (VEC) {
        const uint32_t w = kind == kRowNan ? (F32 ? 0x7FC00000u : 0x7FC07FC0u) : 0;
        for (int i = tid; i < n; i += workers) st_stream_u4(out + 16 * i, make_uint4(w, w, w, w));
      } else {
        for (int j = tid; j < n * EPU; j += workers)
          L::store(out, j, kind == kRowGrad ? grad_scalar<HAS_B>(L::load(buf, j), r)
                                            : kind == kRowNan ? nan : 0.0f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.done[slot]);
      if (++b == nbuf) b = 0, ++lap;
      if (++slot == H) slot = 0, ++turn;
    }
  }
  if (C > 1) {  // no CTA goes while a peer may still send to it
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
}

// Bytes of a CTA's run of a row, for any offset of the row.
int64_t staged_buf_bytes(int64_t cols, int es, int cluster) {
  const int64_t units = cols * es / 16;
  return ((units + cluster - 1) / cluster * 16 + 127) / 128 * 128;
}

// Shared memory left for the ring of one CTA.
int64_t staged_smem(bool distill, int max_smem_optin) {
  return max_smem_optin -
         static_cast<int64_t>(distill ? sizeof(StagedShared<true>) : sizeof(StagedShared<false>));
}

struct StagedShape {
  int threads, nbuf;
  uint32_t buf_bytes;
};

// As many CTAs an SM as two buffers each and their registers leave room for, with 64
// workers or more: a row is a chain of dependent steps for its CTA, so rows in flight
// matter more than workers a row.  (us, CTAs an SM of the rule / with workers for 8
// units each first: logprobs_backward bf16 [6000, 24001] 97.7 / 128.2, [16000, 8200]
// 94.6 / 113.0; distill_backward with 64 entries [16000, 8200] 110.3 / 156.5, [10000,
// 12000] 96.4 / 115.8.)  Four at most, five where that takes all rows at once
// (logprobs_backward [16000, 8200] 94.6 with four, 100.1 with five; [700, 8200] 10.1,
// 8.3), and two buffers, not one, for each ([2048, 50257] 70.3 in one CTA with two, 75.7
// in two with one).  Then workers for 8 units (64 bf16 logits) each, or 10 where
// that is over 576 of them, as far as there is room: fewer units leave more of the time
// to what every thread does once a row, more of them too few warps to cover the
// latencies (6283 units, bf16 [4096, 50257]: 320 workers 128.8, 512 126.1, 640 126.0,
// 800 131.0; 4096 units, bf16 [1022, 65537] in clusters of two: 416 54.9, 512 53.3, 576
// 57.8).  Up to four buffers where the room is there.
StagedShape staged_shape(int64_t rows, int64_t cols, int es, int cluster, bool distill,
                         const DevInfo &info) {
  StagedShape sh;
  sh.buf_bytes = static_cast<uint32_t>(staged_buf_bytes(cols, es, cluster));
  const int64_t units = sh.buf_bytes / 16;
  const int helpers = 32 * ((distill ? kHelpers<true> : kHelpers<false>) + 1);
  const int64_t sm_threads = kMaxThreads + 64;  // at 72 registers a thread
  const int64_t sm_smem = info.max_smem_optin + 1024;
  const int64_t other = sm_smem - staged_smem(distill, info.max_smem_optin);
  const int64_t wanted = (rows * cluster + info.sm_count - 1) / info.sm_count;
  int64_t ctas = 1, room = kMaxThreads - helpers;
  for (int64_t n = 2; n <= (wanted <= 5 ? wanted : 4); ++n) {
    const int64_t left = sm_threads / n / 32 * 32 - helpers;
    if (left < 64 || n * (2 * sh.buf_bytes + other) > sm_smem) break;
    ctas = n;
    room = left;
  }
  int64_t workers = (units / 8 + 31) / 32 * 32;
  if (workers > 576) workers = (units / 10 + 31) / 32 * 32;
  workers = workers < 64 ? 64 : workers > room ? room : workers;
  sh.threads = static_cast<int>(workers) + helpers;
  const int64_t nbuf = (sm_smem / ctas - other) / (sh.buf_bytes > 0 ? sh.buf_bytes : 1);
  sh.nbuf = static_cast<int>(nbuf < 1 ? 1 : nbuf > kMaxBufs ? kMaxBufs : nbuf);
  return sh;
}

template <bool F32, bool DISTILL, bool HAS_B>
cudaError_t launch_form(const LogitsBackward &a, int cluster, bool vec32, bool vec16,
                        const DevInfo &info, cudaStream_t s) {
  if (cluster == 0) {
    const int64_t grid = a.rows < (INT64_C(1) << 30) ? a.rows : (INT64_C(1) << 30);
    const dim3 g(static_cast<unsigned>(grid)), b(kT);
    return vec32 ? launch_k(logit_grad_looped<F32, DISTILL, HAS_B, true>, g, b, 0, s, 0, a)
                 : launch_k(logit_grad_looped<F32, DISTILL, HAS_B, false>, g, b, 0, s, 0, a);
  }
  const int64_t vectors = a.cols * (F32 ? 4 : 2) / kVecBytes;
  if (cluster == 1 && vectors <= kHeldVectors) {
    if (vectors <= 32) return launch_held<F32, DISTILL, HAS_B, 1>(a, vec32, s);
    if (vectors <= 64) return launch_held<F32, DISTILL, HAS_B, 2>(a, vec32, s);
    if (vectors <= 128) return launch_held<F32, DISTILL, HAS_B, 4>(a, vec32, s);
    return launch_held<F32, DISTILL, HAS_B, 8>(a, vec32, s);
  }
  auto *kern = vec16 ? &logit_grad_staged<F32, DISTILL, HAS_B, true>
                     : &logit_grad_staged<F32, DISTILL, HAS_B, false>;
  const StagedShape sh = staged_shape(a.rows, a.cols, F32 ? 4 : 2, cluster, DISTILL, info);
  const size_t smem = static_cast<size_t>(sh.buf_bytes) * sh.nbuf;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void *>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_k(kern, dim3(static_cast<unsigned>(a.rows * cluster)), dim3(sh.threads), smem,
                  s, cluster, a, sh.buf_bytes, sh.nbuf, __builtin_ctz(cluster));
}

}  // namespace

bool logit_grad_staged_ok(int64_t cols, int es, int cluster, bool distill, int max_smem_optin) {
  return staged_buf_bytes(cols, es, cluster) <= staged_smem(distill, max_smem_optin);
}

cudaError_t launch_logits_backward(const LogitsBackward &a, bool f32, bool distill, int cluster,
                                   bool vec32, bool vec16, const DevInfo &info, cudaStream_t s) {
  if (distill)
    return f32 ? launch_form<true, true, false>(a, cluster, vec32, vec16, info, s)
               : launch_form<false, true, false>(a, cluster, vec32, vec16, info, s);
  if (a.dentropy)
    return f32 ? launch_form<true, false, true>(a, cluster, vec32, vec16, info, s)
               : launch_form<false, false, true>(a, cluster, vec32, vec16, info, s);
  return f32 ? launch_form<true, false, false>(a, cluster, vec32, vec16, info, s)
             : launch_form<false, false, false>(a, cluster, vec32, vec16, info, s);
}

}  // namespace fr
