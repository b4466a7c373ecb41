// Log probabilities of given tokens with the entropy and the top alternatives
// of their rows, and the forward pass of distillation from a teacher's top
// logits: one pass over each row of logits.
//
// Each thread keeps the statistics (m, l, s) of logits.cuh over its vectors,
// folding every group of vectors in with the online-softmax merge of "Stax
// (4): GPU Codegen and Dynamic Shapes", section 9.5; the CTA merges them
// (Proposition 9.1).  Then, at T = 1,
//   log p_t = (x_t - m) - log l,   H = log l - s / l,   LSE = m + log l,
// the differences from m taken first, so that a large common offset of a row's
// logits costs no digits.
//
// Top alternatives.  The pass keeps the largest logit of every group of
// vectors (a chunk) in shared memory.  The k-th largest of the chunk maxima is
// a lower bound of the row's k-th largest logit (k chunks hold one each that
// large), so only chunks whose maximum reaches a threshold at or below it are
// read again -- about k of them -- and their logits at or above the threshold
// are the candidates.  Each candidate's place in the order (larger first, equal
// ones by index, every NaN largest) is the number of candidates before it.
// A row whose candidates do not fit (many equal logits, or a row of fewer
// chunks than k) takes its exact k-th largest logit by bisection over the
// keys, counting in the row itself.
#include "launch.h"
#include "logits.cuh"

namespace fr {
namespace {

constexpr int kT = 256;           // threads per CTA
constexpr int kNV = 4;            // 32-byte vectors a thread loads at once
constexpr int kChunkSlots = 8;    // chunk maxima a thread keeps
constexpr int kCandidates = 1024; // candidates a CTA holds

struct TopShared {
  uint32_t chunk[kChunkSlots * kT];  // keys of the chunk maxima (0: no such chunk)
  uint64_t cand[kCandidates];
  int count;                         // candidates found (may pass kCandidates)
  int warp_n[2][kT / 32];
};

// The sum of n over the CTA, in every thread.  `buf` alternates between the
// two sets so that one barrier a call is enough.
__device__ __forceinline__ int block_count(TopShared &sh, int n, int &buf) {
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) sh.warp_n[buf][threadIdx.x >> 5] = n;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kT / 32; ++i) sum += sh.warp_n[buf][i];
  buf ^= 1;
  return sum;
}

__device__ __forceinline__ void add_candidate(TopShared &sh, uint32_t key, int64_t index) {
  const int at = atomicAdd(&sh.count, 1);
  if (at < kCandidates) sh.cand[at] = place_key(key, static_cast<uint32_t>(index));
}

// Keys of the row's logits at or above `key`, counted over the CTA.
template <bool F32>
__device__ int count_from(TopShared &sh, const unsigned char *pr, int64_t cols, uint32_t key,
                          int &buf) {
  int n = 0;
  for (int64_t i = threadIdx.x; i < cols; i += kT) n += logit_key(Logits<F32>::load(pr, i)) >= key;
  return block_count(sh, n, buf);
}

// The row's k candidates by its exact k-th largest key, given a key that at
// least k logits reach.  Leaves exactly k of them in sh.cand.
template <bool F32>
__device__ void exact_candidates(TopShared &sh, const unsigned char *pr, int64_t cols, int k,
                                 uint32_t reached, int &buf) {
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
    const uint32_t key = logit_key(Logits<F32>::load(pr, i));
    if (key > lo) add_candidate(sh, key, i);
  }
  __syncthreads();
  int have = sh.count;
  __syncthreads();
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
  if (threadIdx.x == 0) sh.count = k;
  __syncthreads();
}

template <bool F32, bool DISTILL>
__global__ void __launch_bounds__(kT) logit_rows(LogitsForward a) {
  pdl_enter();
  using L = Logits<F32>;
  __shared__ RowStat red[kT / 32];
  __shared__ TopShared sh;
  const int tid = threadIdx.x;
  const float c = DISTILL ? kLog2e / a.temperature : kLog2e;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const unsigned char *pr =
        static_cast<const unsigned char *>(a.logits) + row * a.ld * L::ES;
    const RowSplit sp = row_split(pr, a.cols, L::ES);
    const unsigned char *pv = pr + static_cast<int64_t>(sp.head) * L::ES;
    const int64_t steps = (sp.nvec + kT * kNV - 1) / (kT * kNV);
    const int64_t per_slot = (steps + kChunkSlots - 1) / kChunkSlots;  // steps of one chunk
    // the scalar this thread takes, if any
    int64_t si = -1;
    if (tid < sp.head) si = tid;
    else if (tid < sp.head + sp.tail) si = sp.head + sp.nvec * L::EPV + (tid - sp.head);
    const float sv = si >= 0 ? L::load(pr, si) : -INFINITY;
    RowStat st{sv, si >= 0 ? 1.0f : 0.0f, 0.0f};
    if (sv == -INFINITY) st = stat_empty();

    float chunk = -INFINITY;
    int slot = 0;
    bool chunk_any = false;
    for (int64_t step = 0; step < steps; ++step) {
      V8 v[kNV];
      const int64_t b = step * (kT * kNV) + tid;
#pragma unroll
      for (int k = 0; k < kNV; ++k)
        v[k] = b + k * kT < sp.nvec ? ld_stream_v8(pv + (b + k * kT) * kVecBytes) : L::filler();
      float cm = L::max(v[0]);
#pragma unroll
      for (int k = 1; k < kNV; ++k) cm = max_nan(cm, L::max(v[k]));
      stat_fold<F32, !DISTILL, kNV>(st, v, cm, c);
      if (!DISTILL && a.top > 0) {
        chunk = max_nan(chunk, cm);
        chunk_any |= b < sp.nvec;
        if ((step + 1) % per_slot == 0 || step + 1 == steps) {
          sh.chunk[slot * kT + tid] = chunk_any ? logit_key(chunk) : 0;
          ++slot;
          chunk = -INFINITY;
          chunk_any = false;
        }
      }
    }
    st = block_stat<kT>(st, c, red);

    if constexpr (DISTILL) {
      if (tid < 32) {
        const Teacher t = teacher_load<F32>(a.index + row * a.ldt, a.teacher + row * a.ldt, a.top,
                                            pr, a.cols, a.temperature);
        const float loss = teacher_loss(t, st, a.temperature);
        if (tid == 0) {
          a.loss[row] = loss;
          if (t.bad) atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
        }
      }
    } else {
      const float logl = logf(st.l);
      if (tid == 0) {
        if (a.logprob) {
          const int64_t t = a.token[row];
          float lp = 0.0f;
          if (t != a.ignore_index) {
            if (t < 0 || t >= a.cols) {
              lp = __int_as_float(0x7fc00000);
              atomicCAS(a.err, 0, FR_DEVERR_BAD_TARGET);
            } else {
              lp = (L::load(pr, t) - st.m) - logl;
            }
          }
          a.logprob[row] = lp;
        }
        if (a.entropy) a.entropy[row] = logl - st.s / st.l;
        if (a.lse) a.lse[row] = st.m + logl;
      }
      if (a.top > 0) {
        const int k = a.top;
        int buf = 0;
        if (tid == 0) sh.count = 0;
        // A threshold that at least k chunks reach and not many more: bisection
        // over the keys, down from the row's maximum.  With fewer chunks than k
        // (the head's and tail's scalars count as one each) every logit passes.
        const uint32_t skey = si >= 0 ? logit_key(sv) : 0;
        auto reaching = [&](uint32_t key) {
          int n = skey >= key;
          for (int i = 0; i < slot; ++i) n += sh.chunk[i * kT + tid] >= key;
          return block_count(sh, n, buf);
        };
        uint32_t lo = 0;
        if (reaching(1) >= k) {
          uint64_t x0 = 1, x1 = static_cast<uint64_t>(logit_key(st.m)) + 1;
          while (x1 - x0 > 1) {
            const uint64_t mid = (x0 + x1) / 2;
            const int n = reaching(static_cast<uint32_t>(mid));
            if (n >= k) x0 = mid;
            else x1 = mid;
            if (n >= k && n <= k + k / 2 + 8) break;
          }
          lo = static_cast<uint32_t>(x0);
        }
        __syncthreads();
        if (skey != 0 && skey >= lo) add_candidate(sh, skey, si);
        for (int i = 0; i < slot; ++i) {
          if (sh.chunk[i * kT + tid] == 0 || sh.chunk[i * kT + tid] < lo) continue;
          const int64_t s1 = (i + 1) * per_slot < steps ? (i + 1) * per_slot : steps;
          for (int64_t step = i * per_slot; step < s1; ++step)
            for (int q = 0; q < kNV; ++q) {
              const int64_t vi = step * (kT * kNV) + q * kT + tid;
              if (vi >= sp.nvec) break;
              const V8 v = ld_stream_v8(pv + vi * kVecBytes);
              if (logit_key(L::max(v)) < lo) continue;
#pragma unroll
              for (int j = 0; j < L::EPV; ++j) {
                const uint32_t key = logit_key(L::at(v, j));
                if (key >= lo) add_candidate(sh, key, sp.head + vi * L::EPV + j);
              }
            }
        }
        __syncthreads();
        if (sh.count > kCandidates) exact_candidates<F32>(sh, pr, a.cols, k, lo, buf);
        const int n = sh.count;
        for (int i = tid; i < n; i += kT) {
          const uint64_t mine = sh.cand[i];
          int before = 0;
          for (int j = 0; j < n; ++j) before += sh.cand[j] > mine;
          if (before < k) {
            const int64_t o = row * k + before;
            a.top_index[o] = place_index(mine);
            a.top_logprob[o] = (key_logit(static_cast<uint32_t>(mine >> 32)) - st.m) - logl;
          }
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_logits_forward(const LogitsForward &a, bool f32, bool distill,
                                  cudaStream_t s) {
  const int64_t grid = a.rows < (INT64_C(1) << 30) ? a.rows : (INT64_C(1) << 30);
  const dim3 g(static_cast<unsigned>(grid)), b(kT);
  if (distill)
    return f32 ? launch_k(logit_rows<true, true>, g, b, 0, s, 0, a)
               : launch_k(logit_rows<false, true>, g, b, 0, s, 0, a);
  return f32 ? launch_k(logit_rows<true, false>, g, b, 0, s, 0, a)
             : launch_k(logit_rows<false, false>, g, b, 0, s, 0, a);
}

}  // namespace fr
