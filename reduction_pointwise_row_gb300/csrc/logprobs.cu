// Log probabilities of given tokens with the entropy and the top alternatives
// of their rows, and the forward pass of distillation from a teacher's top
// logits: one pass over each row of logits.
//
// Each thread keeps the statistics (m, l, s) of logits.cuh over its vectors,
// folding every group of vectors in with the online-softmax merge of "Stax
// (4): GPU Codegen and Dynamic Shapes", section 9.5; lanes, warps and CTAs merge
// theirs the same way (Proposition 9.1).  Then, at T = 1,
//   log p_t = (x_t - m) - log l,   H = log l - s / l,   LSE = m + log l,
// the differences from m taken first, so that a large common offset of a row's
// logits costs no digits.
//
// Top alternatives.  The order is larger logits first, equal ones by index, every
// NaN largest; what matters is to sort few candidates.  Every form finds a floor that at least k
// logits reach: the k-th largest of the maxima of at least k disjoint groups of
// the row's logits.  With g groups about g log(g / (g - k)) logits reach it, some
// more than k.  Only vectors that reach it are read again, for their logits.
//   looped  the pass over the row writes the maximum of every 128 bytes of logits
//           to the workspace, 1/64 of a row, and a
//           second kernel, a warp per row with little state and so many warps an
//           SM, does the rest: the groups are every eighth of a lane's maxima; the
//           vectors under the maxima that reach the floor are read again.  (In
//           one kernel the list's 5-7 us a row of dependent steps held up the loads:
//           bf16 [8192, 50257] top 20 took 173 us by each warp after its row and 192
//           by a helper warp, 152 so.)  A list that still grows
//           (equal logits, an order that puts the largest together)
//           is cut to its k largest, whose least is the next floor.
//   held    (rows in registers) the groups are places of the lanes' vectors; the
//           candidates are listed as in the looped form.
//   split   the groups are the threads' vectors, floors of a cluster's CTAs for
//           k / CTAs each, the least of them the row's; candidates that do not
//           fit are replaced by an exact bisection over the keys of the row, up to 33
//           passes of one CTA.  That is where a row goes whose alternatives lie
//           unevenly over the CTAs' runs, or which has few values (us, an ordinary
//           row / only its first 2000 columns unmasked / rising with the index /
//           constant; bf16 [1, 50257] top 20: 8.3 / 169 / 223 / 31, fp32 [61, 65537]
//           top 5: 10.1 / 490 / 603 / 86; a CTA per row, bf16 [300, 50257] top 20:
//           19.1 / 13.8 / 24.2 / 100).
// Candidates are compared with their indexes, so no result depends on the order
// in which they were found.
#include "launch.h"
#include "logits.cuh"

namespace fr {
namespace {

constexpr int kWarps = 8;  // warps per CTA
constexpr int kT = 32 * kWarps;

// The row's results from its statistics, its token and the token's logit.
__device__ __forceinline__ void write_stats(const LogitsForward &a, int64_t row, int64_t token,
                                            float xt, const RowStat &st, float logl) {
  if (a.logprob) {
    float lp = (xt - st.m) - logl;
    if (token == a.ignore_index) {
      lp = 0.0f;
    } else if (token < 0 || token >= a.cols) {
      lp = __int_as_float(0x7fc00000);
      atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
    }
    a.logprob[row] = lp;
  }
  if (a.entropy) a.entropy[row] = logl - st.s / st.l;
  if (a.lse) a.lse[row] = st.m + logl;
}

__device__ __forceinline__ void write_alternative(const LogitsForward &a, int64_t row, int place,
                                                  uint64_t e, const RowStat &st, float logl) {
  a.top_index[row * a.top + place] = place_index(e);
  a.top_logprob[row * a.top + place] =
      (key_logit(static_cast<uint32_t>(e >> 32)) - st.m) - logl;
}

// Candidates list[0, n), n <= 32 R, to their places among the first k by one
// warp: a bitonic sort, entry R lane + i in a lane's register i.
template <int R>
__device__ __forceinline__ void sort_top(const LogitsForward &a, int64_t row, const uint64_t *list,
                                         int n, const RowStat &st, float logl) {
  const int lane = threadIdx.x & 31;
  uint64_t e[R];
#pragma unroll
  for (int i = 0; i < R; ++i) e[i] = R * lane + i < n ? list[R * lane + i] : 0;
#pragma unroll
  for (int size = 2; size <= 32 * R; size *= 2) {
#pragma unroll
    for (int stride = size / 2; stride > 0; stride /= 2) {
      if (stride >= R) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const uint64_t o = __shfl_xor_sync(0xffffffffu, e[i], stride / R);
          const bool down = ((R * lane + i) & size) == 0;  // larger ones to the front
          const bool low = (lane & (stride / R)) == 0;
          e[i] = (low == down) == (e[i] > o) ? e[i] : o;
        }
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if ((i & stride) == 0) {
            const bool down = ((R * lane + i) & size) == 0;
            const uint64_t x = e[i], y = e[i | stride];
            const bool swap = (x < y) == down;
            e[i] = swap ? y : x;
            e[i | stride] = swap ? x : y;
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (R * lane + i < a.top) write_alternative(a, row, R * lane + i, e[i], st, logl);
}

__device__ __forceinline__ void write_distill(const LogitsForward &a, int64_t row,
                                              const Teacher &t, const RowStat &st) {
  const float loss = teacher_loss(t, st, a.temperature);
  if ((threadIdx.x & 31) != 0) return;
  a.loss[row] = loss;
  if (t.bad) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
}

// ---- looped: a warp per row ----------------------------------------------------

constexpr int kNV = 8;           // 32-byte vectors a lane loads at once
constexpr int kStep = 32 * kNV;  // vectors a warp loads at once
static_assert(kNV == 8, "two maxima of four vectors a step");

// Workspace of a call with alternatives: (m, log l) of each row, then the maxima
// of its steps, [rows][steps][32 lanes] pairs of bf16 rounded down.
__host__ __device__ constexpr int64_t maxima_steps(int64_t cols, int es) {
  return (cols * es / kVecBytes + kStep - 1) / kStep;
}

constexpr int kTopWarps = 4;            // warps per CTA of the second kernel
constexpr int kSegment = 16;            // steps that it takes together
constexpr int kCutAt = 2 * FR_TOP_MAX;  // a longer list is cut before more is listed

// A warp's workspace in the second kernel: 6.25 KiB.
struct WarpTop {
  uint16_t hot[kSegment * 64];     // first vectors of the maxima that reach the floor
  uint16_t vec[128];               // vectors (in the segment) that do
  uint64_t list[kCutAt + 32 * 8];  // room for half the logits of 32 bf16 vectors
};

// Cuts list[0, n), n > k, to its k largest entries (in any order); returns a
// bound that those reach and the others do not.  Entries differ (each has its
// index).  One warp.
__device__ __noinline__ uint64_t cut_list(uint64_t *list, int n, int k) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  uint32_t kmin = 0xFFFFFFFFu, kmax = 0;
  for (int i = lane; i < n; i += 32) {
    const uint32_t key = static_cast<uint32_t>(list[i] >> 32);
    kmin = min(kmin, key);
    kmax = max(kmax, key);
  }
  uint32_t lo = __reduce_min_sync(0xffffffffu, kmin);  // count(>= lo) >= k
  uint32_t hi = __reduce_max_sync(0xffffffffu, kmax);  // count(> hi) < k
  int reach = n;
  while (lo < hi && reach != k) {
    const uint32_t mid = hi - (hi - lo) / 2;  // lo < mid <= hi
    int c = 0;
    for (int i = lane; i < n; i += 32) c += static_cast<uint32_t>(list[i] >> 32) >= mid;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= k) {
      lo = mid;
      reach = c;
    } else {
      hi = mid - 1;
    }
  }
  uint64_t least = static_cast<uint64_t>(lo) << 32;
  if (reach != k) {  // equal logits: the same bisection over their indexes
    uint32_t a = 0, b = 0xFFFFFFFFu;
    while (a < b) {
      const uint32_t mid = b - (b - a) / 2;
      int c = 0;
      for (int i = lane; i < n; i += 32) c += list[i] >= (least | mid);
      c = __reduce_add_sync(0xffffffffu, c);
      if (c >= k) a = mid;
      else b = mid - 1;
      if (c == k) break;
    }
    least |= a;
  }
  int out = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const uint64_t e = i0 + lane < n ? list[i0 + lane] : 0;
    const bool keep = i0 + lane < n && e >= least;
    const uint32_t kept = __ballot_sync(0xffffffffu, keep);
    if (keep) list[out + __popc(kept & ((1u << lane) - 1))] = e;  // at or before i0 + lane
    out += __popc(kept);
    __syncwarp();
  }
  return least;
}

// The key of a floor that at least k of the G * 32 keys in a warp's lanes reach,
// and not many more: a bisection that stops early.
template <int G>
__device__ __forceinline__ uint32_t group_floor(const uint32_t (&key)[G], int k) {
  uint32_t lo = key[0], hi = key[0];
#pragma unroll
  for (int g = 1; g < G; ++g) {
    lo = min(lo, key[g]);
    hi = max(hi, key[g]);
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  int reach = 32 * G;
  while (lo < hi && reach > k + k / 4 + 4) {
    const uint32_t mid = hi - (hi - lo) / 2;  // lo < mid <= hi
    int c = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) c += key[g] >= mid;
    c = __reduce_add_sync(0xffffffffu, c);
    if (c >= k) {
      lo = mid;
      reach = c;
    } else {
      hi = mid - 1;
    }
  }
  return lo;
}

// What a logit has to pass to be listed: `v` (a NaN passes any v), and after a
// cut also to precede `bound` among the place keys.
struct Floor {
  float v;
  uint64_t bound;  // 0: no cut yet
  __device__ __forceinline__ bool passed(float x) const { return !(x < v); }
  __device__ __forceinline__ void raise(uint32_t key) {
    const float f = key_logit(key);
    v = f != f ? INFINITY : f;  // all NaN: the bound decides
  }
};

// The sum of n over the lanes before this one; `total` over all.
__device__ __forceinline__ int lanes_before(int n, int &total) {
  int s = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) >= o) s += t;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  return s - n;
}

__device__ __forceinline__ void cut_if_long(WarpTop &w, int k, int most, int &n, Floor &floor) {
  if (n <= most) return;
  floor.bound = cut_list(w.list, n, k);
  floor.raise(static_cast<uint32_t>(floor.bound >> 32));
  n = k;
}

// Lists the logits of each lane's vector (where it has one) that pass; `index` is
// the first one's place in the row.
template <bool F32>
__device__ __forceinline__ void list_vector(WarpTop &w, const V8 &v, bool have, uint32_t index,
                                            int k, int &n, Floor &floor) {
  using L = Logits<F32>;
#pragma unroll
  for (int j0 = 0; j0 < L::EPV; j0 += 8) {
    cut_if_long(w, k, kCutAt, n, floor);
    uint32_t pass = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) pass |= have && floor.passed(L::at(v, j0 + j)) ? 1u << j : 0;
    if (floor.bound != 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (place_key(logit_key(L::at(v, j0 + j)), index + j0 + j) < floor.bound)
          pass &= ~(1u << j);
    }
    if (!__any_sync(0xffffffffu, pass != 0)) continue;
    int more;
    int to = n + lanes_before(__popc(pass), more);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((pass >> j) & 1) w.list[to++] = place_key(logit_key(L::at(v, j0 + j)), index + j0 + j);
    n += more;
    __syncwarp();
  }
}

// The same of the row's vectors b0 + vec[0, count), count <= 32.
template <bool F32>
__device__ __forceinline__ void list_vectors(const unsigned char *pv, int head, WarpTop &w, int b0,
                                             const uint16_t *vec, int count, int k, int &n,
                                             Floor &floor) {
  const int lane = threadIdx.x & 31;
  const bool have = lane < count;
  const int vi = b0 + (have ? vec[lane] : 0);
  const V8 v =
      have ? ld_keep_v8(pv + static_cast<int64_t>(vi) * kVecBytes) : Logits<F32>::filler();
  list_vector<F32>(w, v, have, static_cast<uint32_t>(head + vi * Logits<F32>::EPV), k, n, floor);
}

// The listed candidates to their places (one warp).
__device__ __forceinline__ void sort_list(const LogitsForward &a, int64_t row, WarpTop &w, int n,
                                          Floor &floor, const RowStat &st, float logl) {
  if (n <= 32) sort_top<1>(a, row, w.list, n, st, logl);
  else if (n <= 64) sort_top<2>(a, row, w.list, n, st, logl);
  else if (n <= 128) sort_top<4>(a, row, w.list, n, st, logl);
  else {
    cut_if_long(w, a.top, kCutAt, n, floor);
    sort_top<8>(a, row, w.list, n, st, logl);
  }
}

// Lists one logit a lane (`take`), if it passes.
__device__ __forceinline__ void list_scalars(WarpTop &w, bool take, float x, int index, int &n,
                                             const Floor &floor) {
  const uint64_t place = place_key(logit_key(x), static_cast<uint32_t>(index));
  const bool hit = take && floor.passed(x) && place >= floor.bound;
  const uint32_t hits = __ballot_sync(0xffffffffu, hit);
  if (hit) w.list[n + __popc(hits & ((1u << (threadIdx.x & 31)) - 1))] = place;
  n += __popc(hits);
  __syncwarp();
}

// The largest bf16 that is not above v (v itself where it is one), NaN for NaN.
__device__ __forceinline__ uint32_t bf16_below(float v) {
  const uint32_t u = __float_as_uint(v);
  if (v != v) return 0x7FFFu;
  return (u >> 16) + ((u & 0x80000000u) && (u & 0xFFFFu) ? 1 : 0);  // towards -inf
}

// Writes the maxima of a step's lines (128 bytes of logits: one vector of each of
// four lanes), rounded down to bf16, as lane 4 g + w's word for vectors 2 w and
// 2 w + 1 of lanes 4 g .. 4 g + 3; returns the lane's own maximum.  The four lanes
// exchange in two halving steps, each keeping the half it will write.
template <bool F32>
__device__ __forceinline__ float step_maxima(const V8 (&v)[kNV], uint32_t *out) {
  using L = Logits<F32>;
  const bool hi2 = threadIdx.x & 2, hi1 = threadIdx.x & 1;
  if constexpr (F32) {
    float m[kNV];
#pragma unroll
    for (int u = 0; u < kNV; ++u) m[u] = L::max(v[u]);
    float own = m[0], h[4];
#pragma unroll
    for (int u = 1; u < kNV; ++u) own = max_nan(own, m[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = max_nan(hi2 ? m[4 + i] : m[i],
                     __shfl_xor_sync(0xffffffffu, hi2 ? m[i] : m[4 + i], 2));
    float q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      q[i] = max_nan(hi1 ? h[2 + i] : h[i],
                     __shfl_xor_sync(0xffffffffu, hi1 ? h[i] : h[2 + i], 1));
    *out = bf16_below(q[0]) | bf16_below(q[1]) << 16;
    return own;
  } else {
    uint32_t m[4];  // (vector 2 w, vector 2 w + 1), exact: they are bf16
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a = v[2 * w].w[0], b = v[2 * w + 1].w[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        a = max_nan_bf16x2(a, v[2 * w].w[j]);
        b = max_nan_bf16x2(b, v[2 * w + 1].w[j]);
      }
      m[w] = max_nan_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
    const uint32_t own = max_nan_bf16x2(max_nan_bf16x2(m[0], m[1]), max_nan_bf16x2(m[2], m[3]));
    uint32_t h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      h[i] = max_nan_bf16x2(hi2 ? m[2 + i] : m[i],
                            __shfl_xor_sync(0xffffffffu, hi2 ? m[i] : m[2 + i], 2));
    *out = max_nan_bf16x2(hi1 ? h[1] : h[0],
                          __shfl_xor_sync(0xffffffffu, hi1 ? h[0] : h[1], 1));
    return max_nan(bf16_lo(own), bf16_hi(own));
  }
}

template <bool F32, bool DISTILL, bool TOP>
__global__ void __launch_bounds__(kT, 2) logit_rows_warp(LogitsForward a) {
  pdl_enter();
  using L = Logits<F32>;
  const int lane = threadIdx.x & 31;
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  const int64_t nw = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); row < a.rows;
       row += nw) {
    const unsigned char *pr = static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
    const RowSplit sp = row_split(pr, a.cols, L::ES);
    const unsigned char *pv = pr + static_cast<int64_t>(sp.head) * L::ES;
    const int nvec = static_cast<int>(sp.nvec);  // cols < 2^31, so at most 2^28
    uint32_t *maxima = nullptr;
    if constexpr (TOP)
      maxima = reinterpret_cast<uint32_t *>(static_cast<float2 *>(a.workspace) + a.rows) +
               row * maxima_steps(a.cols, L::ES) * 32 + lane;
    // loads that nothing waits for before the row's end
    const float head = lane < sp.head ? L::load(pr, lane) : -INFINITY;
    const float tail = lane < sp.tail ? L::load(pr, a.cols - sp.tail + lane) : -INFINITY;
    const int64_t token = !DISTILL && a.logprob ? a.token[row] : -1;
    float xt = 0.0f;
    TeacherRaw teacher;
    if constexpr (DISTILL)
      teacher_fetch(teacher, a.index + row * a.ldt, a.teacher + row * a.ldt, a.top);
    RowStat st = stat_empty();
    for (int b = 0; b < nvec; b += kStep) {
      V8 v[kNV];
#pragma unroll
      for (int u = 0; u < kNV; ++u) {
        const int vi = b + lane + 32 * u;
        v[u] = vi < nvec ? ld_stream_v8(pv + static_cast<int64_t>(vi) * kVecBytes) : L::filler();
      }
      // the teacher's entries with the row's first loads: bf16 [8192, 50257] 133.3 us with
      // them after the row, 125.7 so
      if constexpr (DISTILL) {
        if (b == 0) teacher_gather<F32>(teacher, pr, a.cols);
      }
      float cm = -INFINITY;
      if constexpr (TOP) cm = step_maxima<F32>(v, maxima), maxima += 32;
      if (b + kStep <= nvec) {
        if constexpr (!TOP) cm = L::max(v);
        stat_fold<F32, !DISTILL, kNV>(st, v, cm, c);
      } else {
        // the last step, as far as there are vectors (us, all of it / so: bf16 [30000,
        // 4200] 82.6 / 57.3, [8192, 50257] 129.3 / 125.9)
#pragma unroll
        for (int u = 0; u < kNV; u += 2) {
          if (b + 32 * u >= nvec) break;
          const V8 w[2] = {v[u], v[u + 1]};
          stat_fold<F32, !DISTILL, 2>(st, w, L::max(w), c);
        }
      }
    }
    if (!DISTILL && token >= 0 && token < a.cols) xt = L::load(pr, token);
    if constexpr (DISTILL) {
      if (nvec == 0) teacher_gather<F32>(teacher, pr, a.cols);
    }
    if (head != -INFINITY) st = stat_merge(st, RowStat{head, 1.0f, 0.0f}, c);
    if (tail != -INFINITY) st = stat_merge(st, RowStat{tail, 1.0f, 0.0f}, c);
    st = warp_stat(st, c);
    if constexpr (DISTILL) {
      write_distill(a, row, teacher_finish(teacher, a.cols, a.temperature), st);
    } else if (lane == 0) {
      const float logl = logf(st.l);
      write_stats(a, row, token, xt, st, logl);
      if constexpr (TOP) static_cast<float2 *>(a.workspace)[row] = make_float2(st.m, logl);
    }
    __syncwarp();
  }
}

// The alternatives of the rows whose maxima the kernel above wrote: a warp per row.
template <bool F32>
__global__ void __launch_bounds__(32 * kTopWarps, 8) logit_top_rows(LogitsForward a) {
  pdl_enter();
  using L = Logits<F32>;
  __shared__ WarpTop tops[kTopWarps];
  WarpTop &w = tops[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTopWarps + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const unsigned char *pr = static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
  const RowSplit sp = row_split(pr, a.cols, L::ES);
  const unsigned char *pv = pr + static_cast<int64_t>(sp.head) * L::ES;
  const int nvec = static_cast<int>(sp.nvec), steps = (nvec + kStep - 1) / kStep;
  const float2 stat = static_cast<const float2 *>(a.workspace)[row];
  const uint32_t *maxima =
      reinterpret_cast<const uint32_t *>(static_cast<const float2 *>(a.workspace) + a.rows) +
      row * maxima_steps(a.cols, L::ES) * 32 + lane;
  const float head = lane < sp.head ? L::load(pr, lane) : -INFINITY;
  const float tail = lane < sp.tail ? L::load(pr, a.cols - sp.tail + lane) : -INFINITY;
  const int k = a.top;

  uint32_t sub[4] = {0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};  // 8 groups a lane
  for (int step = 0; step < steps; step += kSegment) {
    uint32_t m[kSegment];  // a segment's loads at once
#pragma unroll
    for (int i = 0; i < kSegment; ++i)
      m[i] = step + i < steps ? maxima[(step + i) * 32] : 0xFF80FF80u;
#pragma unroll
    for (int i = 0; i < kSegment; ++i) sub[i % 4] = max_nan_bf16x2(sub[i % 4], m[i]);
  }
  uint32_t key[8];  // of bf16 values: 16 bits order them
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    key[2 * g] = logit_key(bf16_lo(sub[g])) >> 16;
    key[2 * g + 1] = logit_key(bf16_hi(sub[g])) >> 16;
  }
  Floor floor{-INFINITY, 0};
  const uint32_t fkey = group_floor(key, k);
  floor.raise(fkey << 16 | (fkey & 0x8000u ? 0 : 0xFFFFu));

  int n = 0, pending = 0;
  if (sp.head > 0) list_scalars(w, lane < sp.head, head, lane, n, floor);
  if (sp.tail > 0)
    list_scalars(w, lane < sp.tail, tail, static_cast<int>(a.cols) - sp.tail + lane, n, floor);
  for (int s0 = 0; s0 < steps; s0 += kSegment) {
    const int b0 = s0 * kStep;  // the segment's first vector
    // the maxima are rounded down, so the floor is too: max >= v makes both >= v's
    const float low = bf16_lo(bf16_below(floor.v));
    uint32_t mask = 0;  // bit 2 s + h: half h of this lane's word of step s0 + s passes
#pragma unroll
    for (int s = 0; s < kSegment; ++s) {
      const uint32_t m = s0 + s < steps ? maxima[(s0 + s) * 32] : 0xFF80FF80u;
      mask |= (bf16_lo(m) < low ? 0 : 1u) << (2 * s) | (bf16_hi(m) < low ? 0 : 2u) << (2 * s);
    }
    if (s0 + kSegment > steps) mask &= (1u << (2 * (steps - s0))) - 1;
    int total;
    int at = lanes_before(__popc(mask), total);
    while (mask != 0) {
      const int bit = __ffs(static_cast<int>(mask)) - 1;
      mask &= mask - 1;
      // vector 2 (lane % 4) + h of lanes 4 (lane / 4) .. + 3 of the step
      w.hot[at++] = static_cast<uint16_t>((bit >> 1) * kStep + 32 * (2 * (lane & 3) + (bit & 1)) +
                                          (lane & ~3));
    }
    __syncwarp();
    // a lane reads one vector, four lanes a listed line; kAhead loads at once
    constexpr int kAhead = 4;
    for (int i0 = 0; i0 < 4 * total; i0 += 32 * kAhead) {
      V8 v[kAhead];
      int vec[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + 32 * u + lane;
        vec[u] = i < 4 * total ? w.hot[i / 4] + i % 4 : nvec;
        v[u] = b0 + vec[u] < nvec
                   ? ld_keep_v8(pv + static_cast<int64_t>(b0 + vec[u]) * kVecBytes)
                   : L::filler();
      }
      uint32_t hits[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        hits[u] = __ballot_sync(0xffffffffu, b0 + vec[u] < nvec && floor.passed(L::max(v[u])));
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (hits[u] == 0) continue;
        if ((hits[u] >> lane) & 1)
          w.vec[pending + __popc(hits[u] & ((1u << lane) - 1))] = static_cast<uint16_t>(vec[u]);
        pending += __popc(hits[u]);
        __syncwarp();
      }
      for (int done = 0; done < pending; done += 32)
        list_vectors<F32>(pv, sp.head, w, b0, w.vec + done, min(32, pending - done), k, n, floor);
      pending = 0;
    }
  }
  sort_list(a, row, w, n, floor, RowStat{stat.x, 0.0f, 0.0f}, stat.y);
}

// ---- held: a warp per row, the row in registers ------------------------------------
//
// Rows of at most 4 KiB, NV vectors a lane.  The groups of the alternatives' floor
// are the lanes' 32-bit words at one place of their vectors, 8 a lane.

constexpr int64_t kHeldVectors = 128;

template <bool F32, bool DISTILL, bool TOP, int NV>
__global__ void __launch_bounds__(32 * kTopWarps, 5)
logit_rows_held(LogitsForward a) {
  pdl_enter();
  using L = Logits<F32>;
  __shared__ WarpTop tops[TOP ? kTopWarps : 1];
  WarpTop &w = tops[TOP ? threadIdx.x >> 5 : 0];
  const int lane = threadIdx.x & 31;
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTopWarps + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const unsigned char *pr = static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
  const RowSplit sp = row_split(pr, a.cols, L::ES);
  const unsigned char *pv = pr + static_cast<int64_t>(sp.head) * L::ES;
  const int nvec = static_cast<int>(sp.nvec), tail0 = static_cast<int>(a.cols) - sp.tail;
  const int64_t token = !DISTILL && a.logprob ? a.token[row] : -1;
  V8 v[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u)
    v[u] = lane + 32 * u < nvec ? ld_stream_v8(pv + (lane + 32 * u) * kVecBytes) : L::filler();
  const float head = lane < sp.head ? L::load(pr, lane) : -INFINITY;
  const float tail = lane < sp.tail ? L::load(pr, tail0 + lane) : -INFINITY;
  const float xt = token >= 0 && token < a.cols ? L::load(pr, token) : 0.0f;
  RowStat st = stat_empty();
  stat_fold<F32, !DISTILL, NV>(st, v, L::max(v), c);
  if (head != -INFINITY) st = stat_merge(st, RowStat{head, 1.0f, 0.0f}, c);
  if (tail != -INFINITY) st = stat_merge(st, RowStat{tail, 1.0f, 0.0f}, c);
  st = warp_stat(st, c);
  if constexpr (DISTILL) {
    write_distill(a, row, teacher_load<F32>(a.index + row * a.ldt, a.teacher + row * a.ldt, a.top,
                                            pr, a.cols, a.temperature), st);
  } else {
    const float logl = logf(st.l);
    if (lane == 0) write_stats(a, row, token, xt, st, logl);
    if constexpr (TOP) {
      uint32_t key[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = v[0].w[j];
        if constexpr (F32) {
#pragma unroll
          for (int u = 1; u < NV; ++u)
            m = __float_as_uint(max_nan(__uint_as_float(m), __uint_as_float(v[u].w[j])));
          key[j] = logit_key(__uint_as_float(m));
        } else {
#pragma unroll
          for (int u = 1; u < NV; ++u) m = max_nan_bf16x2(m, v[u].w[j]);
          key[j] = logit_key(max_nan(bf16_lo(m), bf16_hi(m)));
        }
      }
      Floor floor{-INFINITY, 0};
      floor.raise(group_floor(key, a.top));
      int n = 0;
      list_scalars(w, lane < sp.head, head, lane, n, floor);
      list_scalars(w, lane < sp.tail, tail, tail0 + lane, n, floor);
#pragma unroll
      for (int u = 0; u < NV; ++u)
        if (32 * u < nvec)
          list_vector<F32>(w, v[u], lane + 32 * u < nvec,
                           static_cast<uint32_t>(sp.head + (lane + 32 * u) * L::EPV), a.top, n,
                           floor);
      sort_list(a, row, w, n, floor, st, logl);
    }
  }
}

// ---- split: a cluster of CTAs per row ---------------------------------------------

constexpr int kSplitNV = 4;        // 32-byte vectors a thread loads at once
constexpr int kStepMaxima = 16;
constexpr int kCandidates = 1024;  // candidates of a row that its first CTA holds

// 8 bytes from the shared memory of CTA `rank` of this cluster, at the offset
// that `local` has here.
__device__ __forceinline__ uint64_t ld_dsmem_u64(const void *local, uint32_t rank) {
  uint32_t remote;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote) : "memory");
  return v;
}

struct SplitShared {
  float4 part;  // this CTA's m, l, s and (as bits) the key of its floor
  RowStat red[kWarps];
  uint32_t key[kT];  // the threads' maxima
  int warp_n[2][kWarps];
  uint64_t count;  // candidates found (may pass kCandidates)
  uint64_t cand[kCandidates];
  V8 vec[kT];  // a vector of each thread
  float step_max[kStepMaxima][kT];  // the maxima of the threads' steps (the last: of the rest)
};

// The sum of n over the CTA, in every thread.  `buf` alternates between the
// two sets so that one barrier a call is enough.
__device__ __forceinline__ int block_count(SplitShared &sh, int n, int &buf) {
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) sh.warp_n[buf][threadIdx.x >> 5] = n;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) sum += sh.warp_n[buf][i];
  buf ^= 1;
  return sum;
}

__device__ __forceinline__ void add_candidate(SplitShared &sh, float x, int64_t index) {
  const uint32_t at = atomicAdd(reinterpret_cast<uint32_t *>(&sh.count), 1u);  // its low half
  if (at < kCandidates) sh.cand[at] = place_key(logit_key(x), static_cast<uint32_t>(index));
}

// Keys of the row's logits at or above `key`, counted over the CTA.
template <bool F32>
__device__ int count_from(SplitShared &sh, const unsigned char *pr, int64_t cols, uint32_t key,
                          int &buf) {
  int n = 0;
  for (int64_t i = threadIdx.x; i < cols; i += kT) n += logit_key(Logits<F32>::load(pr, i)) >= key;
  return block_count(sh, n, buf);
}

// The row's k candidates by its exact k-th largest key, given a key that at
// least k logits reach: leaves exactly k of them in sh.cand.  One CTA.
template <bool F32>
__device__ __noinline__ void exact_candidates(SplitShared &sh, const unsigned char *pr,
                                              int64_t cols, int k, uint32_t reached) {
  int buf = 0;
  uint32_t lo = reached;
  if (lo != 0xFFFFFFFFu && count_from<F32>(sh, pr, cols, lo + 1, buf) >= k) {
    uint64_t a = lo + 1ull, b = 1ull << 32;  // count(>= a) >= k > count(>= b) = 0
    while (b - a > 1) {
      const uint64_t mid = (a + b) / 2;
      if (count_from<F32>(sh, pr, cols, static_cast<uint32_t>(mid), buf) >= k) a = mid;
      else b = mid;
    }
    lo = static_cast<uint32_t>(a);
  }
  // everything above lo (fewer than k), then the first logits equal to it
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < cols; i += kT) {
    const float x = Logits<F32>::load(pr, i);
    if (logit_key(x) > lo) add_candidate(sh, x, i);
  }
  __syncthreads();
  int have = static_cast<int>(sh.count);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int64_t i0 = 0; i0 < cols && have < k; i0 += kT) {
    const int64_t i = i0 + threadIdx.x;
    const bool hit = i < cols && logit_key(Logits<F32>::load(pr, i)) == lo;
    const uint32_t hits = __ballot_sync(0xffffffffu, hit);
    const int total = block_count(sh, hit ? 1 : 0, buf);  // buf ^ 1 holds the warps' counts
    int at = have + __popc(hits & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += sh.warp_n[buf ^ 1][w];
    if (hit && at < k) sh.cand[at] = place_key(lo, static_cast<uint32_t>(i));
    have += total;
  }
  __syncthreads();
}

template <bool F32, bool DISTILL, bool TOP>
__global__ void __launch_bounds__(kT, TOP ? 3 : 4) logit_rows_split(LogitsForward a) {
  pdl_enter();
  using L = Logits<F32>;
  __shared__ SplitShared sh;
  __shared__ Teacher entries[DISTILL ? 32 : 1];
  // The last warp works on the teacher's entries (two loads that wait for each other,
  // then a softmax) while the others read the row: after the row they cost 1-2 us (bf16
  // [1024, 50257], 64 entries: 23.8 us, 22.3 so; fp32 [300, 65537]: 19.7, 15.9).
  constexpr int W = DISTILL ? kT - 32 : kT;
  const int tid = threadIdx.x, lane = tid & 31;
  const int C = static_cast<int>(cluster_nctarank()), q = static_cast<int>(cluster_ctarank());
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  for (int64_t row = cluster_id_x(); row < a.rows; row += ncluster_x()) {
    const unsigned char *pr = static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
    const RowSplit sp = row_split(pr, a.cols, L::ES);
    const unsigned char *pv = pr + static_cast<int64_t>(sp.head) * L::ES;
    // a row of fewer vectors than threads goes logit by logit, so that every
    // thread has some: at least k groups for any k
    const bool scalar = sp.nvec < kT && C == 1;
    const int v0 = scalar ? 0 : static_cast<int>(sp.nvec * q / C);
    const int v1 = scalar ? 0 : static_cast<int>(sp.nvec * (q + 1) / C);
    // this thread's scalars: i0, i0 + kT, ... below i1
    int i0 = tid, i1 = 0;
    if (scalar) i1 = static_cast<int>(a.cols);
    else if (q == 0 && tid < sp.head) i1 = sp.head;
    const int tail0 = static_cast<int>(a.cols) - sp.tail;
    if (!scalar && q == C - 1 && tid >= 32 && tid < 32 + sp.tail) {
      i0 = tail0 + tid - 32;
      i1 = i0 + 1;
    }
    const int64_t token = !DISTILL && a.logprob ? a.token[row] : -1;
    if constexpr (DISTILL) {
      if (q == 0 && tid >= W)
        entries[lane] = teacher_load<F32>(a.index + row * a.ldt, a.teacher + row * a.ldt, a.top,
                                          pr, a.cols, a.temperature);
    }
    RowStat st = stat_empty();
    for (int i = i0; i < i1; i += kT) {
      const float x = L::load(pr, i);
      if (x != -INFINITY) st = stat_merge(st, RowStat{x, 1.0f, 0.0f}, c);
    }
    for (int b = v0 + (tid < W ? tid : v1), step = 0; b < v1; b += W * kSplitNV, ++step) {
      V8 v[kSplitNV];
#pragma unroll
      for (int u = 0; u < kSplitNV; ++u)
        v[u] = b + u * W < v1 ? ld_keep_v8(pv + static_cast<int64_t>(b + u * W) * kVecBytes)
                              : L::filler();
      const float cm = L::max(v);
      if constexpr (TOP) {
        float &m = sh.step_max[step < kStepMaxima ? step : kStepMaxima - 1][tid];
        m = step < kStepMaxima ? cm : max_nan(m, cm);
      }
      stat_fold<F32, !DISTILL, kSplitNV>(st, v, cm, c);
    }
    const float xt = token >= 0 && token < a.cols ? L::load(pr, token) : 0.0f;
    const float mine = st.m;  // the largest of this thread's logits
    const uint32_t mykey = i0 < i1 || v0 + tid < v1 ? logit_key(mine) : 0;
    if constexpr (TOP) {
      sh.key[tid] = mykey;
      if (tid == 0) sh.count = 0;
    }
    st = block_stat<kT>(st, c, sh.red);
    uint32_t fkey = 0;
    if constexpr (TOP) {
      // this CTA's floor, for its share of k (every warp computes it)
      uint32_t key[kWarps];
#pragma unroll
      for (int g = 0; g < kWarps; ++g) key[g] = sh.key[g * 32 + lane];
      fkey = group_floor(key, (a.top + C - 1) / C);
      if (tid == 0) sh.part.w = __uint_as_float(fkey);
    }
    if (tid == 0) {
      sh.part.x = st.m;
      sh.part.y = st.l;
      sh.part.z = st.s;
    }
    if (C > 1) {
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      const float4 o = lane < C ? ld_dsmem_f4(&sh.part, lane)
                                : make_float4(-INFINITY, 0, 0, __uint_as_float(0xFFFFFFFFu));
      st = warp_stat(RowStat{o.x, o.y, o.z}, c);
      if constexpr (TOP) fkey = __reduce_min_sync(0xffffffffu, __float_as_uint(o.w));
    }
    if constexpr (DISTILL) {
      if (q == 0 && tid >= W) write_distill(a, row, entries[lane], st);
    } else {
      const float logl = logf(st.l);
      if (q == 0 && tid == 0) write_stats(a, row, token, xt, st, logl);
      if constexpr (TOP) {
        if (mykey != 0 && mykey >= fkey) {
          for (int i = i0; i < i1; i += kT) {
            const float x = L::load(pr, i);
            if (logit_key(x) >= fkey) add_candidate(sh, x, i);
          }
          // a NaN passes any floor; a floor of NaN is left to the candidates' keys
          const float fl = fkey == 0 ? -INFINITY : key_logit(fkey);
          const float floor = fl != fl ? INFINITY : fl;
          for (int b = v0 + tid, step = 0; b < v1; b += kT * kSplitNV, ++step) {
            if (sh.step_max[step < kStepMaxima ? step : kStepMaxima - 1][tid] < floor) continue;
            V8 v[kSplitNV];
#pragma unroll
            for (int u = 0; u < kSplitNV; ++u)
              v[u] = b + u * kT < v1 ? ld_keep_v8(pv + static_cast<int64_t>(b + u * kT) * kVecBytes)
                                     : L::filler();
#pragma unroll
            for (int u = 0; u < kSplitNV; ++u) {
              if (b + u * kT >= v1 || L::max(v[u]) < floor) continue;
              // the vector by its elements, which a loop cannot pick from registers
              sh.vec[tid] = v[u];
              const int64_t index = sp.head + int64_t{b + u * kT} * L::EPV;
#pragma unroll 4
              for (int j = 0; j < L::EPV; ++j) {
                const float x = L::load(&sh.vec[tid], j);
                if (!(x < floor)) add_candidate(sh, x, index + j);
              }
            }
          }
        }
        if (C > 1) {
          __syncwarp();
          cluster_arrive();
          cluster_wait();
        } else {
          __syncthreads();
        }
        if (q == 0) {
          int n = static_cast<int>(sh.count);
          if (C > 1) {  // warp r takes CTA r's candidates (C is at most kWarps)
            const int r = tid >> 5;
            const int mine = lane < C ? static_cast<int>(ld_dsmem_u64(&sh.count, lane)) : 0;
            const int at = __shfl_sync(0xffffffffu, lanes_before(mine, n), r);
            const int count = __shfl_sync(0xffffffffu, mine, r);
            if (n <= kCandidates && r > 0)
              for (int i = lane; i < count; i += 32) sh.cand[at + i] = ld_dsmem_u64(&sh.cand[i], r);
            __syncthreads();
          }
          if (n > kCandidates) {
            exact_candidates<F32>(sh, pr, a.cols, a.top, fkey);
            n = a.top;
          }
          // a candidate's place: the number of candidates before it
          for (int i = tid; i < n; i += kT) {
            const uint64_t mine = sh.cand[i];
            int before = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) before += sh.cand[j] > mine;
            if (before < a.top) write_alternative(a, row, before, mine, st, logl);
          }
        }
      }
    }
    if (C > 1) {  // no CTA's shared memory is written again, or given up, while it is read
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  }
}

template <bool F32, bool DISTILL, bool TOP>
cudaError_t launch_held(const LogitsForward &a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.rows + kTopWarps - 1) / kTopWarps));
  const dim3 block(32 * kTopWarps);
  const int64_t vectors = a.cols * (F32 ? 4 : 2) / kVecBytes;
  return vectors <= 32 ? launch_k(logit_rows_held<F32, DISTILL, TOP, 1>, grid, block, 0, s, 0, a)
         : vectors <= 64
             ? launch_k(logit_rows_held<F32, DISTILL, TOP, 2>, grid, block, 0, s, 0, a)
             : launch_k(logit_rows_held<F32, DISTILL, TOP, 4>, grid, block, 0, s, 0, a);
}

template <bool F32, bool DISTILL, bool TOP>
cudaError_t launch_forward(const LogitsForward &a, int split, int sm_count, cudaStream_t s) {
  if (split < 0) return launch_held<F32, DISTILL, TOP>(a, s);
  const dim3 block(kT);
  if (split == 0) {
    // a persistent grid of two CTAs an SM, shrunk so that every warp takes the
    // same number of rows
    const int64_t warps = static_cast<int64_t>(sm_count) * 2 * kWarps;
    const int64_t per_warp = (a.rows + warps - 1) / warps;
    const int64_t grid = (a.rows + per_warp * kWarps - 1) / (per_warp * kWarps);
    const dim3 g(static_cast<unsigned>(grid));
    if constexpr (!TOP) {
      return launch_k(logit_rows_warp<F32, DISTILL, TOP>, g, block, 0, s, 0, a);
    } else {
      // An ordinary launch: placed while the second kernel of the call before is
      // ending, its CTAs fill the SMs that free up first (bf16 [8192, 50257]: 173
      // us a call with one alternative, 144 so).
      logit_rows_warp<F32, DISTILL, TOP><<<g, block, 0, s>>>(a);
      cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      return launch_k(logit_top_rows<F32>,
                      dim3(static_cast<unsigned>((a.rows + kTopWarps - 1) / kTopWarps)),
                      dim3(32 * kTopWarps), 0, s, 0, a);
    }
  }

  const int64_t most = (INT64_C(1) << 30) / split;
  const int64_t clusters = a.rows < most ? a.rows : most;
  return launch_k(logit_rows_split<F32, DISTILL, TOP>,
                  dim3(static_cast<unsigned>(clusters * split)), block, 0, s, split, a);
}

}  // namespace

bool logits_held_ok(int64_t cols, int es) { return cols * es / kVecBytes <= kHeldVectors; }

bool logits_grid_ok(int64_t rows) { return rows <= int64_t{INT32_MAX} * kTopWarps; }

size_t logprobs_workspace(int64_t rows, int64_t cols, int es) {
  return static_cast<size_t>(rows) * (8 + 128 * static_cast<size_t>(maxima_steps(cols, es)));
}

cudaError_t launch_logits_forward(const LogitsForward &a, bool f32, bool distill, int split,
                                  int sm_count, cudaStream_t s) {
  if (distill)
    return f32 ? launch_forward<true, true, false>(a, split, sm_count, s)
               : launch_forward<false, true, false>(a, split, sm_count, s);
  if (a.top > 0)
    return f32 ? launch_forward<true, false, true>(a, split, sm_count, s)
               : launch_forward<false, false, true>(a, split, sm_count, s);
  return f32 ? launch_forward<true, false, false>(a, split, sm_count, s)
             : launch_forward<false, false, false>(a, split, sm_count, s);
}

}  // namespace fr
