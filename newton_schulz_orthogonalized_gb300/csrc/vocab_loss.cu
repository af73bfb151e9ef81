// Losses over a vocabulary: log probabilities of given tokens (with entropy and top
// alternatives) and distillation from a teacher's top logits, forward and backward.
//
//   k_logprobs   y = x / t, lse = log sum exp(y), logprob = y_token - lse,
//                entropy = -sum q log q, the k largest logits; gradient of
//                a logprob + b entropy: (a (1[v = token] - q_v) - b q_v (log q_v + entropy)) / t
//   k_distill    loss = sum_j p_j (log p_j - log q_{i_j}) [+ p_r (log p_r - log q_r)] over the
//                teacher's entries S = {i_j} and, with the tail, the rest of the row as one
//                bucket (q_r = sum of q outside S); gradient g/t times
//                q_v (1 + excess) - p_v in S and q_v (1 + excess) - p_r q_v / q_r outside,
//                where 1 + excess = sum p + p_r
//
// One block per row: a pass over the row's 16-byte vectors with a running sum of
// exponentials relative to a running reference, then (for the gradient) a second pass.
// Sums and statistics are fp32, a gradient is rounded once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "launch.cuh"
#include "nsm_internal.h"

namespace nsm {
namespace {

constexpr int kVocabThreads = 256;
constexpr int kVocabWarps = kVocabThreads / 32;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
// A thread's reference moves only when a logit exceeds it by this many binary orders:
// sums then stay below 2^16 elements' worth of their largest term, far from overflow.
constexpr float kRefSlack = 16.f;
// log2 q below this is a q of 0 in fp32: it bounds 0 * -inf in entropy terms
constexpr float kLog2Floor = -200.f;
constexpr int kTopCandidates = 1024;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr int kKeyLowBit = 0;  // lowest bit in which two values' keys can differ
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float from_float(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static constexpr int kKeyLowBit = 16;
  static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static constexpr int kKeyLowBit = 13;
  static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One row of logits (or gradients) as 16-byte vectors on the address grid: vector i holds
// elements i kVec - lead ... + kVec, of which those in [0, vocab) exist.
template <typename T>
struct Row {
  static constexpr int kVec = Elem<T>::kVec;
  T* p;
  int vocab, lead, nvec;
  __device__ __forceinline__ Row(T* base, int vocab_) : p(base), vocab(vocab_) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
    nvec = (vocab + lead + kVec - 1) / kVec;
  }
  __device__ __forceinline__ int first(int i) const { return i * kVec - lead; }
  __device__ __forceinline__ bool whole(int i) const { return first(i) >= 0 && first(i) + kVec <= vocab; }
  // elements outside the row read as -inf
  __device__ __forceinline__ void load(int i, float (&f)[kVec], int* status, int kernel) const {
    const int e0 = first(i);
    if (whole(i)) {
      if (!bounds_ok(i >= 0 && (reinterpret_cast<uintptr_t>(p + e0) & 15) == 0, status, kernel, 0, NSM_SITE_LOGITS)) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) f[e] = kNegInf;
        return;
      }
      const uint4 raw = *reinterpret_cast<const uint4*>(p + e0);
      const T* h = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int e = 0; e < kVec; ++e) f[e] = Elem<T>::to_float(h[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int v = e0 + e;
        f[e] = v >= 0 && v < vocab ? Elem<T>::to_float(p[v]) : kNegInf;
      }
    }
  }
};

// Writes kVec gradients whose first element is e0 of a row, as one 16-byte store where the
// vector is whole and the gradient's row is aligned like the logits'.
template <typename T>
__device__ __forceinline__ void store_vec(T* row, int vocab, int e0, const float (&g)[Elem<T>::kVec], int* status,
                                          int kernel) {
  constexpr int kVec = Elem<T>::kVec;
  const bool whole = e0 >= 0 && e0 + kVec <= vocab;
  if (whole && (reinterpret_cast<uintptr_t>(row + e0) & 15) == 0) {
    uint4 raw;
    T* h = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int e = 0; e < kVec; ++e) h[e] = Elem<T>::from_float(g[e]);
    *reinterpret_cast<uint4*>(row + e0) = raw;
  } else {
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int v = e0 + e;
      if (v >= 0 && v < vocab) row[v] = Elem<T>::from_float(g[e]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void zero_row(T* row, int vocab, int* status, int kernel) {
  const Row<T> out(row, vocab);
  float g[Elem<T>::kVec] = {};
  for (int i = threadIdx.x; i < out.nvec; i += kVocabThreads) store_vec<T>(row, vocab, out.first(i), g, status, kernel);
}

// A sum of exponentials s = sum 2^((x - ref) c) with its sum of y 2^y (y the exponent), the
// largest x and where this thread met it first.
struct Sums {
  float ref = 0.f, limit = kNegInf;  // no reference yet: every finite logit exceeds the limit
  float s = 0.f, sy = 0.f;
  float max = kNegInf;
  int max_vec = -1;
};

template <int N, bool ENT>
__device__ __forceinline__ void add_vec(Sums& a, const float (&f)[N], int i, float c) {
  float m = f[0];
#pragma unroll
  for (int e = 1; e < N; ++e) m = fmaxf(m, f[e]);
  if (m > a.max) {
    a.max = m;
    a.max_vec = i;
  }
  if (m > a.limit) {
    if (a.limit != kNegInf) {  // move what is there to the new reference
      const float d = (a.ref - m) * c, r = ex2(d);
      if (ENT) a.sy = r > 0.f ? r * (a.sy + d * a.s) : 0.f;
      a.s *= r;
    }
    a.ref = m;
    a.limit = m + kRefSlack / c;
  }
  float s = 0.f, sy = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float y = (f[e] - a.ref) * c;
    const float x = ex2(y);
    s += x;
    if (ENT) sy += x * fmaxf(y, kLog2Floor);
  }
  a.s += s;
  if (ENT) a.sy += sy;
}

// Two sums relative to the larger of their maxima (max is then the reference).
__device__ __forceinline__ void rebase(float& s, float& sy, float ref, float max, float c) {
  const float d = (ref - max) * c;
  const float r = max == kNegInf ? 0.f : ex2(d);  // nothing there: s is 0 (or a NaN, which stays)
  sy = r > 0.f ? r * (sy + d * s) : r * s;
  s *= r;
}

struct Totals {
  float max, s, sy;
};

__device__ __forceinline__ Totals merge(const Totals& a, const Totals& b, float c) {
  Totals t;
  t.max = fmaxf(a.max, b.max);
  float as = a.s, asy = a.sy, bs = b.s, bsy = b.sy;
  if (a.max != t.max) rebase(as, asy, a.max, a.max == kNegInf ? kNegInf : t.max, c);
  if (b.max != t.max) rebase(bs, bsy, b.max, b.max == kNegInf ? kNegInf : t.max, c);
  t.s = as + bs;
  t.sy = asy + bsy;
  return t;
}

// The block's sums relative to its largest logit, the same in every thread (fixed order).
__device__ __forceinline__ Totals block_totals(const Sums& a, float c, Totals* parts) {
  Totals t{a.max, a.s, a.sy};
  if (a.max != kNegInf) rebase(t.s, t.sy, a.ref, a.max, c);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const Totals other{__shfl_xor_sync(~0u, t.max, o), __shfl_xor_sync(~0u, t.s, o), __shfl_xor_sync(~0u, t.sy, o)};
    // the same operand order in both lanes of a pair
    t = (threadIdx.x & o) ? merge(other, t, c) : merge(t, other, c);
  }
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = t;
  __syncthreads();
  t = parts[0];
#pragma unroll
  for (int w = 1; w < kVocabWarps; ++w) t = merge(t, parts[w], c);
  __syncthreads();
  return t;
}

__device__ __forceinline__ int64_t load_index(const void* p, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

// ---------------------------------------------------------------- the k largest

// Order of floats as unsigned integers; -0 and +0 are the same value.
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;

struct TopShared {
  uint32_t key[kVocabThreads];
  int32_t vec[kVocabThreads];
  int32_t list[kVocabThreads];
  uint64_t cand[kTopCandidates];
  uint64_t best[kVocabWarps];
  uint32_t bound_key, bound_tie_top;
  int32_t bound_vec, nlist, ncand;
};

__device__ __forceinline__ uint64_t full_key(float f, int v) {
  return (static_cast<uint64_t>(order_key(f)) << 32) | (0xffffffffu - static_cast<uint32_t>(v));
}

// The first warp finds a bound that at least k threads' largest logits reach: the k-th
// largest of them (bits below kKeyLowBit do not tell two values apart), and where more than
// k reach it, the vector number up to which the ones equal to it are needed.
template <typename T>
__device__ __forceinline__ void top_bound(TopShared& sh, int k) {
  constexpr int kLow = Elem<T>::kKeyLowBit;
  constexpr int kPer = kVocabThreads / 32;
  const int lane = threadIdx.x;
  uint32_t key[kPer];
  int vec[kPer];
  int valid = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    key[j] = sh.key[j * 32 + lane];
    vec[j] = sh.vec[j * 32 + lane];
    valid += key[j] > kKeyNegInf;
  }
  valid = __reduce_add_sync(~0u, valid);
  uint32_t bound = kKeyNegInf + 1, tie_top = kKeyNegInf;
  int bound_vec = 0x7fffffff;
  if (valid > k) {
    bound = 0;
    int reach = valid;
    for (int b = 31; b >= kLow && reach != k; --b) {
      const uint32_t test = bound | (1u << b);
      int n = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) n += key[j] >= test;
      n = __reduce_add_sync(~0u, n);
      if (n >= k) {
        bound = test;
        reach = n;
      }
    }
    if (bound <= kKeyNegInf) bound = kKeyNegInf + 1;
    if (reach > k) {  // every bit is fixed: the threads that tie differ below kLow at most
      tie_top = bound | ((1u << kLow) - 1u);
      int above = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) above += key[j] > tie_top;
      above = __reduce_add_sync(~0u, above);
      bound_vec = 0;
      for (int b = 30; b >= 0; --b) {
        const int test = bound_vec | ((1 << b) - 1);
        int n = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) n += key[j] >= bound && key[j] <= tie_top && vec[j] <= test;
        if (__reduce_add_sync(~0u, n) < k - above) bound_vec |= 1 << b;
      }
    }
  }
  if (lane == 0) {
    sh.bound_key = bound;
    sh.bound_tie_top = tie_top;
    sh.bound_vec = bound_vec;
    sh.nlist = 0;
    sh.ncand = 0;
  }
}

// The row's k largest logits, from every thread's largest one and where it met it.
template <typename T>
__device__ __forceinline__ void row_top(const Row<T>& row, const Sums& a, int k, float max, float inv_t, float log_s,
                                        float* out_value, int32_t* out_index, TopShared& sh, int* status) {
  constexpr int kVec = Elem<T>::kVec;
  const int tid = threadIdx.x;
  sh.key[tid] = order_key(a.max);
  sh.vec[tid] = a.max_vec;
  __syncthreads();
  if (tid < 32) top_bound<T>(sh, k);
  __syncthreads();
  const uint32_t bound = sh.bound_key, tie_top = sh.bound_tie_top;
  const int bound_vec = sh.bound_vec;
  const uint32_t key = sh.key[tid];
  if (key >= bound && (key > tie_top || a.max_vec <= bound_vec)) sh.list[atomicAdd(&sh.nlist, 1)] = tid;
  __syncthreads();
  const int nlist = sh.nlist, lane = tid & 31;
  for (int q = tid >> 5; q < nlist; q += kVocabWarps) {
    for (int i = sh.list[q] + lane * kVocabThreads; i < row.nvec; i += 32 * kVocabThreads) {
      float f[kVec];
      row.load(i, f, status, NSM_KERNEL_LOGPROBS);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const uint32_t ek = order_key(f[e]);
        if (ek >= bound && (ek > tie_top || i <= bound_vec)) {
          const int at = atomicAdd(&sh.ncand, 1);
          if (at < kTopCandidates) sh.cand[at] = full_key(f[e], row.first(i) + e);
        }
      }
    }
  }
  __syncthreads();
  const int ncand = sh.ncand;
  if (ncand <= kTopCandidates) {
    // keys are distinct: a candidate's place is the number of larger ones
    for (int j = tid; j < ncand; j += kVocabThreads) {
      const uint64_t mine = sh.cand[j];
      int place = 0;
      for (int o = 0; o < ncand; ++o) place += sh.cand[o] > mine;
      if (place < k) {
        const int v = static_cast<int>(0xffffffffu - static_cast<uint32_t>(mine));
        out_index[place] = v;
        out_value[place] = (Elem<T>::to_float(row.p[v]) - max) * inv_t - log_s;
      }
    }
    for (int j = ncand + tid; j < k; j += kVocabThreads) {
      out_index[j] = -1;
      out_value[j] = kNegInf;
    }
  } else {
    // so many logits above the bound sit in few threads: one block-wide maximum per place
    uint64_t last = ~0ull;
    for (int j = 0; j < k; ++j) {
      uint64_t best = 0;
      for (int i = tid; i < row.nvec; i += kVocabThreads) {
        float f[kVec];
        row.load(i, f, status, NSM_KERNEL_LOGPROBS);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const uint64_t fk = full_key(f[e], row.first(i) + e);
          if (fk < last && fk > best && order_key(f[e]) > kKeyNegInf) best = fk;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t other = __shfl_xor_sync(~0u, best, o);
        best = other > best ? other : best;
      }
      if (lane == 0) sh.best[tid >> 5] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kVocabWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
      __syncthreads();
      last = best;  // more than kTopCandidates >= k logits are there
      if (tid == 0) {
        const int v = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
        out_index[j] = v;
        out_value[j] = (Elem<T>::to_float(row.p[v]) - max) * inv_t - log_s;
      }
    }
  }
}

// ---------------------------------------------------------------- log probabilities

template <typename T, bool FWD, bool GRAD>
__global__ void __launch_bounds__(kVocabThreads) k_logprobs(const LogprobArgs g, int* status) {
  constexpr int kVec = Elem<T>::kVec;
  __shared__ Totals parts[kVocabWarps];
  __shared__ TopShared top;
  grid_dependency_sync();
  release_dependents();
  const int64_t r = blockIdx.x;
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab);
  int64_t token = g.tokens ? load_index(g.tokens, g.tokens_wide, r) : -1;
  if (token < 0 || token >= vocab) token = -1;
  float ref, log_s, log2_s, entropy = 0.f;
  bool empty;
  const float x_token = token >= 0 ? Elem<T>::to_float(row.p[token]) : 0.f;
  if (FWD) {
    Sums a;
    for (int i = threadIdx.x; i < row.nvec; i += kVocabThreads) {
      float f[kVec];
      row.load(i, f, status, NSM_KERNEL_LOGPROBS);
      add_vec<kVec, true>(a, f, i, c);
    }
    const Totals t = block_totals(a, c, parts);
    empty = t.max == kNegInf && t.s == 0.f;  // a row of NaN has a NaN sum
    ref = empty ? 0.f : t.max;
    log2_s = empty ? 0.f : log2f(t.s);
    log_s = empty ? 0.f : logf(t.s);
    if (!empty) {
      entropy = log_s - kLn2 * (t.sy / t.s);
      if (entropy < 0.f) entropy = 0.f;
    }
    if (threadIdx.x == 0) {
      if (g.lse) g.lse[r] = empty ? kNegInf : ref * inv_t + log_s;
      if (g.entropy) g.entropy[r] = entropy;
      if (g.logprob) g.logprob[r] = token < 0 ? 0.f : (empty ? kNegInf : (x_token - ref) * inv_t - log_s);
    }
    if (g.k > 0) {
      float* value = g.top_logprob + r * g.k;
      int32_t* index = g.top_index + r * g.k;
      if (log_s != log_s) {  // NaN or +inf in the row
        for (int j = threadIdx.x; j < g.k; j += kVocabThreads) {
          value[j] = log_s;
          index[j] = -1;
        }
      } else {
        row_top<T>(row, a, g.k, ref, inv_t, log_s, value, index, top, status);
      }
    }
  } else {
    const float lse = g.in_lse[r];
    empty = lse == kNegInf;
    ref = empty ? 0.f : lse * g.v.t;
    log2_s = log_s = 0.f;
    if (g.d_entropy) entropy = g.in_entropy[r];
  }
  if (GRAD) {
    T* out = static_cast<T*>(g.v.d_logits) + r * g.v.ldd;
    const float w = g.d_logprob && token >= 0 ? g.d_logprob[r] : 0.f;
    const float h = g.d_entropy ? g.d_entropy[r] : 0.f;
    if (empty || (w == 0.f && h == 0.f)) {
      zero_row<T>(out, vocab, status, NSM_KERNEL_LOGPROBS);
      return;
    }
    // -q (w + h (log q + entropy)) / t = q (ca + cb log2 q)
    const float ca = -(w + h * entropy) * inv_t, cb = -h * kLn2 * inv_t;
    float g_token = 0.f;
    const float log_q = (x_token - ref) * inv_t - log_s;
    if (log_q != kNegInf) {  // at the token 1 - q without cancellation; 0 where it is masked
      g_token = -(w * expm1f(log_q) + h * expf(log_q) * (log_q + entropy)) * inv_t;
    }
    for (int i = threadIdx.x; i < row.nvec; i += kVocabThreads) {
      float f[kVec];
      row.load(i, f, status, NSM_KERNEL_LOGPROBS);
      const int e0 = row.first(i);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const float y = (f[e] - ref) * c - log2_s;
        f[e] = ex2(y) * (ca + cb * fmaxf(y, kLog2Floor));
      }
      if (token >= e0 && token < e0 + kVec) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (e0 + e == token) f[e] = g_token;
      }
      store_vec<T>(out, vocab, e0, f, status, NSM_KERNEL_LOGPROBS);
    }
  }
}

// ---------------------------------------------------------------- distillation

struct DistillShared {
  int32_t index[kDistillMaxK];   // -1: the entry does not count
  float x[kDistillMaxK];         // the student's logit there
  float log_p[kDistillMaxK];
  Totals parts[kVocabWarps];
  float sum[kVocabWarps];
  double dsum[kVocabWarps];
};

__device__ __forceinline__ float block_sum(float v, float* parts) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = v;
  __syncthreads();
  v = parts[0];
#pragma unroll
  for (int w = 1; w < kVocabWarps; ++w) v += parts[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ double block_sum(double v, double* parts) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = v;
  __syncthreads();
  v = parts[0];
#pragma unroll
  for (int w = 1; w < kVocabWarps; ++w) v += parts[w];
  __syncthreads();
  return v;
}

__device__ __forceinline__ float block_max(float v, float* parts) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = v;
  __syncthreads();
  v = parts[0];
#pragma unroll
  for (int w = 1; w < kVocabWarps; ++w) v = fmaxf(v, parts[w]);
  __syncthreads();
  return v;
}

__device__ __forceinline__ float load_number(const void* p, int dtype, int64_t i) {
  if (dtype == NSM_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == NSM_FP16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

template <typename T, bool FWD, bool GRAD>
__global__ void __launch_bounds__(kVocabThreads) k_distill(const DistillArgs g, int* status) {
  constexpr int kVec = Elem<T>::kVec;
  extern __shared__ __align__(16) uint8_t members[];  // FWD: a bit per element of vector i in byte i
  __shared__ DistillShared sh;
  static_assert(kDistillMaxK <= kVocabThreads, "one thread per entry");
  grid_dependency_sync();
  release_dependents();
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, k = g.k, vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab);

  // the teacher's entries: of equal indexes the first counts
  float z = kNegInf;
  if (tid < k) {
    const int64_t v = load_index(g.index, g.index_wide, r * g.ldi + tid);
    const bool in = v >= 0 && v < vocab;
    sh.index[tid] = in ? static_cast<int32_t>(v) : -1;
    sh.x[tid] = in ? Elem<T>::to_float(row.p[v]) : 0.f;
    z = load_number(g.teacher, g.teacher_dtype, r * g.ldt + tid);
  }
  if (FWD) {
    for (int i = tid; i < (row.nvec + 3) / 4; i += kVocabThreads) reinterpret_cast<uint32_t*>(members)[i] = 0;
  }
  __syncthreads();
  int mine = tid < k ? sh.index[tid] : -1;
  for (int j = 0; j < tid && mine >= 0; ++j)
    if (sh.index[j] == mine) mine = -1;
  __syncthreads();
  if (tid < k) sh.index[tid] = mine;
  if (FWD && mine >= 0) {
    const int at = mine + row.lead, i = at / kVec;
    atomicOr(reinterpret_cast<uint32_t*>(members) + i / 4, 1u << (8 * (i & 3) + at % kVec));
  }
  const bool counts = mine >= 0;
  float log_p = kNegInf;
  float p_rest = 0.f, lacking = 0.f;
  bool any;
  if (g.tail) {
    if (counts) log_p = z;
    // 1 - sum p: the teacher's rest is often a small difference, so in 64 bits
    const double sum = block_sum(counts ? exp(static_cast<double>(log_p)) : 0.0, sh.dsum);
    lacking = static_cast<float>(1.0 - sum);
    p_rest = lacking > 0.f ? lacking : (lacking != lacking ? lacking : 0.f);
    any = __syncthreads_or(counts);
  } else {
    const float y = counts ? z * inv_t : kNegInf;
    const float m = block_max(y, sh.sum);
    // a NaN entry makes the sum, and with it every p, a NaN
    const float total = block_sum(!counts ? 0.f : (m != kNegInf ? expf(y - m) : (y != y ? y : 0.f)), sh.sum);
    if (counts && !(y == kNegInf)) log_p = (y - m) - logf(total);
    any = m != kNegInf || total != total;
  }
  if (tid < k) sh.log_p[tid] = log_p;
  const float p = expf(log_p);
  const float x_mine = counts ? sh.x[tid] : kNegInf;

  // the student: the row outside S first, then S
  float rest_ref = 0.f, rest_log2 = 0.f;  // q_v / q_r = 2^((x_v - rest_ref) c - rest_log2)
  float lse_ref = 0.f, lse_log = 0.f;     // log q_v = (x_v - lse_ref) / t - lse_log
  float rest;                             // log q_r
  bool empty;
  if (FWD) {
    Sums a;
    for (int i = tid; i < row.nvec; i += kVocabThreads) {
      float f[kVec];
      row.load(i, f, status, NSM_KERNEL_DISTILL);
      const uint32_t bits = members[i];
      if (bits) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          if (bits >> e & 1) f[e] = kNegInf;
      }
      add_vec<kVec, false>(a, f, i, c);
    }
    const Totals out = block_totals(a, c, sh.parts);
    Sums b;
    if (counts) {
      const float f[1] = {x_mine};
      add_vec<1, false>(b, f, 0, c);
    }
    const Totals all = merge(out, block_totals(b, c, sh.parts), c);
    empty = all.max == kNegInf && all.s == 0.f;
    lse_ref = empty ? 0.f : all.max;
    lse_log = empty ? 0.f : logf(all.s);
    const bool no_rest = out.max == kNegInf && out.s == 0.f;
    rest_ref = no_rest ? 0.f : out.max;
    rest_log2 = no_rest ? 0.f : log2f(out.s);
    rest = no_rest ? kNegInf : (out.max - lse_ref) * inv_t + (logf(out.s) - lse_log);
    const float log_q = (x_mine - lse_ref) * inv_t - lse_log;
    if (rest == kNegInf) p_rest = 0.f;
    float term = p > 0.f || p != p ? p * (log_p - log_q) : 0.f;
    float loss = block_sum(term, sh.sum);
    if (p_rest > 0.f || p_rest != p_rest) loss += p_rest * (logf(p_rest) - rest);
    if (tid == 0) {
      if (g.loss) g.loss[r] = any ? loss : 0.f;
      if (g.lse) g.lse[r] = empty ? kNegInf : lse_ref * inv_t + lse_log;
      if (g.rest) g.rest[r] = rest;
    }
  } else {
    const float lse = g.in_lse[r];
    empty = lse == kNegInf;
    lse_ref = empty ? 0.f : lse * g.v.t;
    rest = g.tail ? g.in_rest[r] : 0.f;
    rest_ref = empty || rest == kNegInf ? 0.f : (lse + rest) * g.v.t;
    if (rest == kNegInf) p_rest = 0.f;
  }
  if (GRAD) {
    T* out = static_cast<T*>(g.v.d_logits) + r * g.v.ldd;
    const float w = g.d_loss ? g.d_loss[r] : 1.f;
    if (empty || !any || w == 0.f) {
      zero_row<T>(out, vocab, status, NSM_KERNEL_DISTILL);
      return;
    }
    const float excess = g.tail ? p_rest - lacking : 0.f;  // sum p + p_rest - 1
    const float scale = w * inv_t;
    // outside S, with the tail: q (1 + excess) - p_rest q / q_r = (q / q_r) (q_r (1 + excess) - p_rest)
    float ref, log2_s, coef;
    if (g.tail) {
      ref = rest_ref;
      log2_s = rest_log2;
      coef = rest == kNegInf ? 0.f : scale * (expf(rest) * (1.f + excess) - p_rest);
    } else {
      ref = lse_ref;
      log2_s = lse_log * (1.f / kLn2);
      coef = scale;
    }
    float g_mine = 0.f;  // in S: q (1 + excess) - p, q - p without cancellation
    const float log_q = (x_mine - lse_ref) * inv_t - lse_log;
    if (counts && log_q != kNegInf) {
      const float q = expf(log_q);
      g_mine = scale * ((p > 0.f || p != p ? p * expm1f(log_q - log_p) : q) + q * excess);
    }
    for (int i = tid; i < row.nvec; i += kVocabThreads) {
      float f[kVec];
      row.load(i, f, status, NSM_KERNEL_DISTILL);
#pragma unroll
      for (int e = 0; e < kVec; ++e) f[e] = ex2((f[e] - ref) * c - log2_s) * coef;
      store_vec<T>(out, vocab, row.first(i), f, status, NSM_KERNEL_DISTILL);
    }
    __syncthreads();  // the entries' own values go over what the pass wrote there
    if (counts) out[mine] = Elem<T>::from_float(g_mine);
  }
}

template <typename K, typename A>
cudaError_t launch_rows(K* kernel, const A& args, size_t smem, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  if (const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(args.v.rows)), dim3(kVocabThreads), smem, stream, args, status))
    return e;
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_logprobs_t(const LogprobArgs& a, cudaStream_t stream) {
  if (a.in_lse) return launch_rows(k_logprobs<T, false, true>, a, 0, stream);
  if (a.v.d_logits) return launch_rows(k_logprobs<T, true, true>, a, 0, stream);
  return launch_rows(k_logprobs<T, true, false>, a, 0, stream);
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs& a, cudaStream_t stream) {
  const size_t nvec = (static_cast<size_t>(a.v.vocab) + 2 * Elem<T>::kVec) / Elem<T>::kVec;
  const size_t smem = (nvec + 15) / 16 * 16;
  if (a.in_lse) return launch_rows(k_distill<T, false, true>, a, 0, stream);
  if (a.v.d_logits) return launch_rows(k_distill<T, true, true>, a, smem, stream);
  return launch_rows(k_distill<T, true, false>, a, smem, stream);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  if (a.v.dtype == NSM_BF16) return launch_logprobs_t<__nv_bfloat16>(a, stream);
  if (a.v.dtype == NSM_FP16) return launch_logprobs_t<__half>(a, stream);
  return launch_logprobs_t<float>(a, stream);
}

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
  if (a.v.dtype == NSM_BF16) return launch_distill_t<__nv_bfloat16>(a, stream);
  if (a.v.dtype == NSM_FP16) return launch_distill_t<__half>(a, stream);
  return launch_distill_t<float>(a, stream);
}

}  // namespace nsm
