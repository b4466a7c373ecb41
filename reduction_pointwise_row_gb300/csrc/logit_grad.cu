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
#include "launch.h"
#include "logits.cuh"

namespace fr {
namespace {

constexpr int kT = 512;  // threads per CTA
constexpr int kNV = 2;   // 32-byte vectors a thread loads at once

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

// What the row's elements are computed from: dx = e (a + b (x - m)).
struct RowCoef {
  float m, a, b;
};

struct GradShared {
  int64_t idx[FR_TOP_MAX];  // elements written again (-1: none)
  float val[FR_TOP_MAX];    // what they get
  float q[FR_TOP_MAX];
};

template <bool F32, bool HAS_B>
__device__ __forceinline__ V8 grad_vector(const V8 &x, const RowCoef &r, float c) {
  using L = Logits<F32>;
  const uint64_t m2 = pack_f32x2(r.m, r.m), c2 = pack_f32x2(c, c), a2 = pack_f32x2(r.a, r.a);
  V8 o;
#pragma unroll
  for (int j = 0; j < L::EPV / 2; ++j) {
    const uint64_t d = sub_f32x2(pack_f32x2(L::at(x, 2 * j), L::at(x, 2 * j + 1)), m2);
    const uint64_t t = mul_f32x2(d, c2);
    const uint64_t e = pack_f32x2(ex2(f32x2_lo(t)), ex2(f32x2_hi(t)));
    uint64_t f = a2;
    if constexpr (HAS_B)
      f = fma_f32x2(pack_f32x2(r.b, r.b), pack_f32x2(fmaxf(f32x2_lo(d), kFarBelow),
                                                     fmaxf(f32x2_hi(d), kFarBelow)), a2);
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

template <bool HAS_B>
__device__ __forceinline__ float grad_scalar(float x, const RowCoef &r, float c) {
  const float d = x - r.m;
  return ex2(d * c) * (HAS_B ? fmaf(r.b, fmaxf(d, kFarBelow), r.a) : r.a);
}

// A row's gradient is all zeros (an ignored row, a row without teacher) or all
// NaN (a target past the row) before anything is read of it.
enum RowKind { kRowGrad = 0, kRowZero = 1, kRowNan = 2 };

template <bool F32, bool DISTILL, bool HAS_B, bool VEC>
__global__ void __launch_bounds__(kT) logit_grad_looped(LogitsBackward a) {
  pdl_enter();
  using L = Logits<F32>;
  __shared__ RowStat red[kT / 32];
  __shared__ GradShared sh;
  __shared__ int kind_s;
  const int tid = threadIdx.x;
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  const float nan = __int_as_float(0x7fc00000);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const unsigned char *pr = static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
    unsigned char *po = static_cast<unsigned char *>(a.dlogits) + row * a.ldd * L::ES;
    const RowSplit sp = row_split(pr, a.cols, L::ES);
    const int64_t vo = static_cast<int64_t>(sp.head) * L::ES;

    Teacher t;
    int64_t token = -1;
    float xt = 0.0f, g = 0.0f, h = 0.0f;
    bool ignored = false;
    if constexpr (DISTILL) {
      if (tid < 32) {
        t = teacher_load<F32>(a.index + row * a.ldt, a.teacher + row * a.ldt, a.top, pr, a.cols,
                              a.temperature);
        if (tid == 0) {
          kind_s = t.bad ? kRowNan : t.any ? kRowGrad : kRowZero;
          if (t.bad) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
        }
      }
      g = a.dloss[row * a.dloss_stride] * a.temperature;
    } else {
      if (a.token) {
        token = a.token[row];
        ignored = token == a.ignore_index;
        const bool bad = !ignored && (token < 0 || token >= a.cols);
        if (tid == 0) {
          kind_s = bad ? kRowNan : ignored && !HAS_B ? kRowZero : kRowGrad;
          if (bad) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
        }
        if (!ignored && !bad) {
          xt = L::load(pr, token);
          g = a.dloss[row * a.dloss_stride] * a.dloss_sign;
        } else {
          token = -1;
        }
      } else if (tid == 0) {
        kind_s = kRowGrad;
      }
      if constexpr (HAS_B) h = a.dentropy[row * a.dentropy_stride];
    }
    __syncthreads();
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

    RowCoef r;
    r.m = st.m;
    r.b = HAS_B ? -h / st.l : 0.0f;
    if constexpr (DISTILL) r.a = g / st.l;
    else r.a = HAS_B ? (h * (st.s / st.l) - g) / st.l : -g / st.l;

    // the elements with a term of their own, before the row is overwritten
    if constexpr (DISTILL) {
      if (tid < 32) {
#pragma unroll
        for (int i = 0; i < kTopPerLane; ++i) {
          sh.idx[tid + 32 * i] = t.q[i] != 0.0f ? t.idx[i] : -1;
          sh.q[tid + 32 * i] = t.q[i];
        }
        __syncwarp();
        const float loss = teacher_loss(t, st, a.temperature);
        if (a.loss && tid == 0) a.loss[row] = loss;
#pragma unroll
        for (int i = 0; i < kTopPerLane; ++i) {
          const int64_t j = sh.idx[tid + 32 * i];
          if (j < 0) continue;
          float q = 0.0f;  // entries that name j, in their order
          for (int n = 0; n < a.top; ++n)
            if (sh.idx[n] == j) q += sh.q[n];
          sh.val[tid + 32 * i] = g * (ex2((t.x[i] - st.m) * c) / st.l - q);
        }
      }
    } else if (a.loss && tid == 0) {
      a.loss[row] = logf(st.l) - (xt - st.m);
    }
    // in place, every element is read by the thread that writes it
    if constexpr (VEC) {
      if (si >= 0) L::store(po, si, grad_scalar<HAS_B>(L::load(pr, si), r, c));
      for (int64_t b = tid; b < sp.nvec; b += kT) {
        const V8 x = ld_v8(pr + vo + b * kVecBytes);
        st_stream_v8(po + vo + b * kVecBytes, grad_vector<F32, HAS_B>(x, r, c));
      }
    } else {
      for (int64_t j = tid; j < a.cols; j += kT)
        L::store(po, j, grad_scalar<HAS_B>(L::load(pr, j), r, c));
    }
    __syncthreads();
    if constexpr (DISTILL) {
      if (tid < a.top && sh.idx[tid] >= 0) L::store(po, sh.idx[tid], sh.val[tid]);
    } else if (tid == 0 && token >= 0) {
      L::store(po, token, grad_scalar<HAS_B>(xt, r, c) + g);
    }
    __syncthreads();
  }
}

template <bool F32, bool DISTILL, bool HAS_B>
cudaError_t launch_looped(const LogitsBackward &a, bool vec, cudaStream_t s) {
  const int64_t grid = a.rows < (INT64_C(1) << 30) ? a.rows : (INT64_C(1) << 30);
  const dim3 g(static_cast<unsigned>(grid)), b(kT);
  return vec ? launch_k(logit_grad_looped<F32, DISTILL, HAS_B, true>, g, b, 0, s, 0, a)
             : launch_k(logit_grad_looped<F32, DISTILL, HAS_B, false>, g, b, 0, s, 0, a);
}

}  // namespace

cudaError_t launch_logits_backward(const LogitsBackward &a, bool f32, bool distill, bool vec,
                                   cudaStream_t s) {
  if (distill)
    return f32 ? launch_looped<true, true, false>(a, vec, s)
               : launch_looped<false, true, false>(a, vec, s);
  if (a.dentropy)
    return f32 ? launch_looped<true, false, true>(a, vec, s)
               : launch_looped<false, false, true>(a, vec, s);
  return f32 ? launch_looped<true, false, false>(a, vec, s)
             : launch_looped<false, false, false>(a, vec, s);
}

}  // namespace fr
