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
// A cluster of blocks per row (one block where rows are many): a pass over the row's 16-byte
// vectors with a running sum of exponentials relative to a running reference, then (for the
// gradient) a second pass.  Sums and statistics are fp32, a gradient is rounded once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "launch.cuh"
#include "nsm_internal.h"
#include "ptx.cuh"

namespace nsm {
namespace {

constexpr int kMaxWarps = 8;  // of the blocks below: NT = 32, 64, ..., 256 threads
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
// A thread's reference moves only when a logit exceeds it by this many binary orders:
// sums then stay below 2^16 elements' worth of their largest term, far from overflow.
constexpr float kRefSlack = 16.f;
// log2 q below this is a q of 0 in fp32: it bounds 0 * -inf in entropy terms
constexpr float kLog2Floor = -200.f;
constexpr int kTopCandidates = 1024;
constexpr int kMaxCluster = 8;
constexpr uint64_t kWaitNs = 2000000000ull;  // a wait's limit

// Two fp32 values in one 64-bit register: add, multiply and fused multiply-add of both are
// one instruction each.
using Pair = uint64_t;
__device__ __forceinline__ Pair make_pair(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split_pair(Pair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair pair_mul(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair pair_fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A 16-byte vector of one of the logits' types.
template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr int kKeyLowBit = 0;  // lowest bit in which two values' keys can differ
  static constexpr uint32_t kNegInfBits = 0xff800000u;
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float from_float(float v) { return v; }
  static __device__ __forceinline__ void unpack(const uint4& r, Pair (&x)[2]) {
    x[0] = (static_cast<Pair>(r.y) << 32) | r.x;
    x[1] = (static_cast<Pair>(r.w) << 32) | r.z;
  }
  static __device__ __forceinline__ uint4 pack(const Pair (&x)[2]) {
    return make_uint4(static_cast<uint32_t>(x[0]), static_cast<uint32_t>(x[0] >> 32), static_cast<uint32_t>(x[1]),
                      static_cast<uint32_t>(x[1] >> 32));
  }
  static __device__ __forceinline__ float largest(const uint4& r) {  // NaNs aside
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static constexpr int kKeyLowBit = 16;
  static constexpr uint32_t kNegInfBits = 0xff80u;
  static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ Pair widen(uint32_t w) {
    return (static_cast<Pair>(w & 0xffff0000u) << 32) | (w << 16);
  }
  static __device__ __forceinline__ uint32_t narrow(Pair p) {
    float lo, hi;
    split_pair(p, lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, Pair (&x)[4]) {
    x[0] = widen(r.x);
    x[1] = widen(r.y);
    x[2] = widen(r.z);
    x[3] = widen(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const Pair (&x)[4]) {
    return make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
  }
  static __device__ __forceinline__ float largest(const uint4& r) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
    const float2 m = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
    return fmaxf(m.x, m.y);
  }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  static constexpr int kKeyLowBit = 13;
  static constexpr uint32_t kNegInfBits = 0xfc00u;
  static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ Pair widen(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_pair(f.x, f.y);
  }
  static __device__ __forceinline__ uint32_t narrow(Pair p) {
    float lo, hi;
    split_pair(p, lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  static __device__ __forceinline__ void unpack(const uint4& r, Pair (&x)[4]) {
    x[0] = widen(r.x);
    x[1] = widen(r.y);
    x[2] = widen(r.z);
    x[3] = widen(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const Pair (&x)[4]) {
    return make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
  }
  static __device__ __forceinline__ float largest(const uint4& r) {
    const __half2* h = reinterpret_cast<const __half2*>(&r);
    const float2 m = __half22float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
    return fmaxf(m.x, m.y);
  }
};

// Element e of a vector, and the vector with element e replaced (e may vary at run time).
template <typename T>
__device__ __forceinline__ float vec_get(const uint4& r, int e) {
  return Elem<T>::to_float(reinterpret_cast<const T*>(&r)[e]);
}
template <typename T>
__device__ __forceinline__ void vec_mask(uint4& r, uint32_t bits) {  // -inf where a bit is set
  uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (sizeof(T) == 4) {
      if (bits >> j & 1) w[j] = Elem<T>::kNegInfBits;
    } else {
      if (bits >> (2 * j) & 1) w[j] = (w[j] & 0xffff0000u) | Elem<T>::kNegInfBits;
      if (bits >> (2 * j + 1) & 1) w[j] = (w[j] & 0x0000ffffu) | (Elem<T>::kNegInfBits << 16);
    }
  }
}
template <typename T>
__device__ __forceinline__ void vec_set(uint4& r, int e, float v) {
  reinterpret_cast<T*>(&r)[e] = Elem<T>::from_float(v);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A vector that begins at element e0 of a row, element by element, for the ragged ends of rows.
// Out of line: rare, and long beside the loops of the forward kernels (in line where a call would
// take registers from a kernel that has few: the top alternatives').
template <typename T>
__device__ __forceinline__ uint4 load_elements_here(const T* p, int vocab, int e0) {
  uint4 raw = make_uint4(0, 0, 0, 0);
  T* h = reinterpret_cast<T*>(&raw);
  uint32_t none = 0;  // -inf outside the row
#pragma unroll
  for (int e = 0; e < Elem<T>::kVec; ++e) {
    const int v = e0 + e;
    if (v >= 0 && v < vocab) h[e] = p[v]; else none |= 1u << e;
  }
  vec_mask<T>(raw, none);
  return raw;
}
template <typename T>
__device__ __noinline__ uint4 load_elements(const T* p, int vocab, int e0) {
  return load_elements_here<T>(p, vocab, e0);
}

// One row of logits (or gradients) as 16-byte vectors on the address grid: vector i holds
// elements i kVec - lead ... + kVec, of which those in [0, vocab) exist.
template <typename T>
struct Row {
  static constexpr int kVec = Elem<T>::kVec;
  T* p;
  int vocab, lead, nvec;
  int* status;
  int kernel;
  __device__ __forceinline__ Row(T* base, int vocab_, int* status_, int kernel_)
      : p(base), vocab(vocab_), status(status_), kernel(kernel_) {
    lead = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15) / sizeof(T));
    nvec = (vocab + lead + kVec - 1) / kVec;
  }
  __device__ __forceinline__ int first(int i) const { return i * kVec - lead; }
  __device__ __forceinline__ bool whole(int i) const { return first(i) >= 0 && first(i) + kVec <= vocab; }
  __device__ __forceinline__ uint4 load_whole(int i) const {
    if (!bounds_ok(i >= 0 && whole(i) && (reinterpret_cast<uintptr_t>(p + first(i)) & 15) == 0, status, kernel, 0,
                   NSM_SITE_LOGITS))
      return make_uint4(0, 0, 0, 0);
    return *reinterpret_cast<const uint4*>(p + first(i));
  }
  // vector i of the row, with -inf outside it
  __device__ __forceinline__ uint4 load(int i) const {
    const int e0 = first(i);
    return whole(i) ? load_whole(i) : load_elements<T>(p, vocab, e0);
  }
  __device__ __forceinline__ uint4 load_here(int i) const {
    return whole(i) ? load_whole(i) : load_elements_here<T>(p, vocab, first(i));
  }
  // writes vector i, which is whole
  __device__ __forceinline__ void store_whole(int i, const uint4& raw) const {
    if (!bounds_ok(whole(i) && (reinterpret_cast<uintptr_t>(p + first(i)) & 15) == 0, status, kernel, 0, NSM_SITE_GRADIENT)) return;
    *reinterpret_cast<uint4*>(p + first(i)) = raw;
  }
  // writes kVec gradients whose first element is e0 of the row, as one 16-byte store where
  // the vector is whole and aligned
  __device__ __forceinline__ void store(int e0, const uint4& raw) const {
    if (!bounds_ok(e0 > -kVec && e0 < vocab, status, kernel, 0, NSM_SITE_GRADIENT)) return;
    if (e0 >= 0 && e0 + kVec <= vocab && (reinterpret_cast<uintptr_t>(p + e0) & 15) == 0) {
      *reinterpret_cast<uint4*>(p + e0) = raw;
    } else {
      const T* h = reinterpret_cast<const T*>(&raw);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int v = e0 + e;
        if (v >= 0 && v < vocab) p[v] = h[e];
      }
    }
  }
};

// The part of a row's vectors that one block takes: whole vectors [begin, end), of which
// thread t of NT has every NT-th from begin + t on, and the row's ragged first and last
// vector (-1: not here), which threads kHeadThread and kTailThread have as well.
constexpr int kHeadThread = 0, kTailThread = 32;
struct Part {
  int begin, end, head, tail;
};

template <typename T>
__device__ __forceinline__ Part part_of(const Row<T>& row, int piece, int pieces) {
  const int whole_begin = row.lead > 0 ? 1 : 0;
  const int whole_end = max(whole_begin, (row.vocab + row.lead) / Elem<T>::kVec);
  const int count = whole_end - whole_begin, each = (count + pieces - 1) / pieces;
  Part part;
  part.begin = whole_begin + min(count, piece * each);
  part.end = whole_begin + min(count, (piece + 1) * each);
  part.head = row.lead > 0 && piece == 0 ? 0 : -1;
  part.tail = whole_end < row.nvec && piece == pieces - 1 ? whole_end : -1;
  return part;
}

// use(i, vector, whole) for every vector of the part that this thread has, four loads in flight;
// done(n) after the n-th four of them (the ragged ones come last and are not counted).
template <int NT, bool HERE, typename T, typename F, typename D>
__device__ __forceinline__ void for_batches(const Row<T>& row, const Part& part, F&& use, D&& done) {
  int i = part.begin + static_cast<int>(threadIdx.x), n = 0;
  for (; i + 3 * NT < part.end; i += 4 * NT, ++n) {
    uint4 raw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = row.load_whole(i + u * NT);
#pragma unroll
    for (int u = 0; u < 4; ++u) use(i + u * NT, raw[u], true);
    done(n);
  }
  if (i < part.end) {  // three at most, their loads together too
    uint4 raw[3];
#pragma unroll
    for (int u = 0; u < 3; ++u)
      if (i + u * NT < part.end) raw[u] = row.load_whole(i + u * NT);
#pragma unroll
    for (int u = 0; u < 3; ++u)
      if (i + u * NT < part.end) use(i + u * NT, raw[u], true);
    done(n);
  }
  if (part.head >= 0 && threadIdx.x == kHeadThread) use(part.head, HERE ? row.load_here(part.head) : row.load(part.head), false);
  if (part.tail >= 0 && threadIdx.x == kTailThread) use(part.tail, HERE ? row.load_here(part.tail) : row.load(part.tail), false);
}

// A thread's first four vectors of a part, loaded ahead of what their use waits for.
template <int NT, typename T>
struct FirstFour {
  uint4 raw[4];
  __device__ __forceinline__ void load(const Row<T>& row, const Part& part) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = part.begin + static_cast<int>(threadIdx.x) + u * NT;
      if (i < part.end) raw[u] = row.load_whole(i);
    }
  }
  // use(i, vector, whole) for those, and what follows them in the part
  template <typename F>
  __device__ __forceinline__ void use_all(const Row<T>& row, Part part, F&& use) const;
};

template <int NT, bool HERE = false, typename T, typename F>
__device__ __forceinline__ void for_vectors(const Row<T>& row, const Part& part, F&& use) {
  for_batches<NT, HERE>(row, part, use, [](int) {});
}

template <int NT, typename T>
template <typename F>
__device__ __forceinline__ void FirstFour<NT, T>::use_all(const Row<T>& row, Part part, F&& use) const {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = part.begin + static_cast<int>(threadIdx.x) + u * NT;
    if (i < part.end) use(i, raw[u], true);
  }
  part.begin = min(part.end, part.begin + 4 * NT);
  for_vectors<NT>(row, part, use);
}

template <int NT, typename T>
__device__ __forceinline__ void zero_part(const Row<T>& out, int piece, int pieces) {
  const Part part = part_of(out, piece, pieces);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int i = part.begin + static_cast<int>(threadIdx.x); i < part.end; i += NT) out.store(out.first(i), zero);
  if (part.head >= 0 && threadIdx.x == kHeadThread) out.store(out.first(part.head), zero);
  if (part.tail >= 0 && threadIdx.x == kTailThread) out.store(out.first(part.tail), zero);
}

// A sum of exponentials s = sum 2^y, y = (x - ref) c, with sum y 2^y (both in two halves, one
// per element of a pair), and the largest x.  (x - ref) c and not x c - ref c in one fused step:
// the latter needs a correction for its rounding and a second way for the types' lowest values,
// which cost more than the step saves (8192 x 8000 bf16, loss and gradient: 75 us for 62).
struct Sums {
  float ref = 0.f, limit = kNegInf;  // no reference yet: every finite logit exceeds the limit
  Pair s = 0, sy = 0;
  float max = kNegInf;
};

// Adds a vector; its largest element.
template <typename T, bool ENT>
__device__ __forceinline__ float add_vec(Sums& a, const uint4& raw, float c) {
  constexpr int kPairs = Elem<T>::kVec / 2;
  const float m = Elem<T>::largest(raw);
  a.max = fmaxf(a.max, m);
  if (m > a.limit) {
    if (a.limit != kNegInf) {  // move what is there to the new reference
      const float d = (a.ref - m) * c, r = ex2(d);
      if (ENT) a.sy = r > 0.f ? pair_mul(make_pair(r, r), pair_fma(make_pair(d, d), a.s, a.sy)) : 0;
      a.s = pair_mul(a.s, make_pair(r, r));
    }
    a.ref = m;
    a.limit = m + kRefSlack / c;
  }
  Pair x[kPairs];
  Elem<T>::unpack(raw, x);
  const Pair minus_ref = make_pair(-a.ref, -a.ref), cc = make_pair(c, c);
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const Pair y = pair_mul(pair_add(x[j], minus_ref), cc);
    float y0, y1;
    split_pair(y, y0, y1);
    const Pair e = make_pair(ex2(y0), ex2(y1));
    a.s = pair_add(a.s, e);
    if (ENT) a.sy = pair_fma(e, make_pair(fmaxf(y0, kLog2Floor), fmaxf(y1, kLog2Floor)), a.sy);
  }
  return m;
}

struct Totals {
  float max, s, sy;
};

// Moves sums from their reference to `max` (>= ref); what has no reference is 0, or a NaN.
template <bool ENT>
__device__ __forceinline__ void rebase(float& s, float& sy, float ref, float max, float c) {
  const float d = (ref - max) * c;
  const float r = ref == kNegInf ? 0.f : ex2(d);
  if (ENT) sy = r > 0.f ? r * (sy + d * s) : r * s;
  s *= r;
}

// Totals of a group of `N` (a power of two) lanes, the same in every lane, in a fixed order.
template <bool ENT, int N>
__device__ __forceinline__ Totals group_totals(float ref, float max, float s, float sy, float c) {
  Totals t{max, s, sy};
#pragma unroll
  for (int o = N / 2; o; o >>= 1) t.max = fmaxf(t.max, __shfl_xor_sync(~0u, t.max, o));
  rebase<ENT>(t.s, t.sy, ref, t.max, c);
#pragma unroll
  for (int o = N / 2; o; o >>= 1) {
    t.s += __shfl_xor_sync(~0u, t.s, o);
    if (ENT) t.sy += __shfl_xor_sync(~0u, t.sy, o);
  }
  return t;
}

template <bool ENT>
__device__ __forceinline__ Totals warp_totals(const Sums& a, float c) {
  float s0, s1, y0 = 0.f, y1 = 0.f;
  split_pair(a.s, s0, s1);
  if (ENT) split_pair(a.sy, y0, y1);
  return group_totals<ENT, 32>(a.limit == kNegInf ? kNegInf : a.ref, a.max, s0 + s1, y0 + y1, c);
}

// The totals of every CTA's threads of a cluster relative to the row's largest logit, the
// same in every thread: warps, then CTAs, in a fixed order.  Every thread of the block calls
// this, the sums of the first NT count; the next use of `sh` needs a barrier.  The CTAs
// exchange theirs through a barrier in shared memory that counts one arrival from each: only
// the threads that send wait for their stores, not the whole block.  With more than one CTA,
// start_totals comes first.
struct TotalsShared {
  Totals warp[kMaxWarps];
  Totals cta[kMaxCluster];
  uint64_t joined;
  int abort;
};
__device__ __forceinline__ void start_totals(TotalsShared& sh, int ctas) {
  if (ctas == 1) return;
  if (threadIdx.x == 0) {
    ptx::mbar_init(ptx::smem_u32(&sh.joined), ctas);
    sh.abort = 0;
    ptx::fence_mbarrier_init();
  }
  __syncwarp();
  ptx::cluster_arrive();  // the wait is in row_totals: by then every CTA runs
}
template <bool ENT, int NT>
__device__ __forceinline__ Totals row_totals(const Sums& a, float c, TotalsShared& sh, int ctas, int* status, int kernel) {
  const Totals w = warp_totals<ENT>(a, c);
  if ((threadIdx.x & 31) == 0 && threadIdx.x < NT) sh.warp[threadIdx.x >> 5] = w;
  if (ctas > 1) ptx::cluster_wait();
  __syncthreads();
  const Totals v = sh.warp[threadIdx.x & (NT / 32 - 1)];
  const Totals mine = group_totals<ENT, NT / 32>(v.max, v.max, v.s, v.sy, c);
  if (ctas == 1) return mine;
  if (static_cast<int>(threadIdx.x) < ctas) {
    const uint32_t to = ptx::mapa_shared(ptx::smem_u32(&sh.cta[ptx::cluster_ctarank()]), threadIdx.x);
    ptx::st_cluster_f32(to, mine.max);
    ptx::st_cluster_f32(to + 4, mine.s);
    ptx::st_cluster_f32(to + 8, mine.sy);
    ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_u32(&sh.joined), threadIdx.x));
  }
  if (!ptx::mbar_wait_bounded_cluster(ptx::smem_u32(&sh.joined), 0, &sh.abort, kWaitNs)) {
    record_timeout(status, kernel, NSM_ROLE_EPILOGUE, NSM_SITE_ACC_FULL);
    *static_cast<volatile int*>(&sh.abort) = 1;
  }
  Totals t{kNegInf, 0.f, 0.f};
  for (int r = 0; r < ctas; ++r) t.max = fmaxf(t.max, sh.cta[r].max);
  for (int r = 0; r < ctas; ++r) {
    Totals o = sh.cta[r];
    rebase<ENT>(o.s, o.sy, o.max, t.max, c);
    t.s += o.s;
    t.sy += o.sy;
  }
  return t;
}

// One vector of gradients q (ca + cb log2 q), q = 2^((x - ref) c - log2_s).
template <typename T, bool ENT>
__device__ __forceinline__ uint4 gradient_vec(const uint4& raw, float ref, float c, float log2_s, float ca, float cb) {
  constexpr int kPairs = Elem<T>::kVec / 2;
  Pair x[kPairs];
  Elem<T>::unpack(raw, x);
  const Pair minus_ref = make_pair(-ref, -ref), cc = make_pair(c, c), minus_log = make_pair(-log2_s, -log2_s);
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const Pair y = pair_fma(pair_add(x[j], minus_ref), cc, minus_log);
    float y0, y1;
    split_pair(y, y0, y1);
    const Pair q = make_pair(ex2(y0), ex2(y1));
    const Pair f = ENT ? pair_fma(make_pair(fmaxf(y0, kLog2Floor), fmaxf(y1, kLog2Floor)), make_pair(cb, cb), make_pair(ca, ca))
                       : make_pair(ca, ca);
    x[j] = pair_mul(q, f);
  }
  return Elem<T>::pack(x);
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
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;
static_assert(kTopCandidates >= kMaxCluster * kTopMaxK, "every CTA's k largest fit");

// What one of the k largest logits reaches: keys from `key` on, and of those up to tie_top only
// in vectors up to `vec`.
struct TopBound {
  uint32_t key, tie_top;
  int vec;
};

constexpr int kTopThreads = 256, kTopWarps = kTopThreads / 32;
constexpr int kTopGroups = 32;   // groups of batches per thread at most
constexpr int kTopList = 1024;
struct TopShared {
  uint32_t key[kTopThreads];
  int32_t vec[kTopThreads];
  uint32_t list[kTopList];                    // group * kTopThreads + thread
  uint64_t cand[kTopCandidates];
  uint64_t best[kTopWarps];
  TopBound bound;
  int32_t nlist, ncand;
  uint32_t taken[kMaxCluster];                // how many keys each CTA gave
};

// A thread's largest logit and the vector where it met it first.
template <typename T>
struct TopMax {
  float max = kNegInf;
  int max_vec = -1;
  __device__ __forceinline__ void see(float m, int i) {
    if (m > max) {
      max = m;
      max_vec = i;
    }
  }
};

// The largest logit of every group of a thread's batches: which groups can hold one of the
// row's k largest, without reading the row again.  A 16-bit key where that tells two values
// of the type apart.
template <typename T>
struct TopGroups {
  using Key = typename std::conditional<Elem<T>::kKeyLowBit == 16, uint16_t, uint32_t>::type;
  Key* top;       // [group][thread], in shared memory; a thread reads what it wrote itself
  int shift;      // batches per group: 1 << shift
  float running;
  __device__ __forceinline__ void batch(int n) {
    const uint32_t key = order_key(running);
    top[(n >> shift) * kTopThreads + threadIdx.x] = static_cast<Key>(sizeof(Key) == 2 ? key >> 16 : key);
    if ((n + 1) >> shift != n >> shift) running = kNegInf;
  }
  // the largest key that the group can hold
  __device__ __forceinline__ uint32_t largest(int group) const {
    const uint32_t key = top[group * kTopThreads + threadIdx.x];
    return sizeof(Key) == 2 ? key << 16 | 0xffffu : key;
  }
};

__device__ __forceinline__ uint64_t full_key(float f, int v) {
  return (static_cast<uint64_t>(order_key(f)) << 32) | (0xffffffffu - static_cast<uint32_t>(v));
}

// From the largest logits of groups of vectors (PER keys of each lane of a warp, with the vector
// where each was met first): a bound that at least k groups reach and at most `enough` do.  The
// k-th largest key, bit by bit until that holds (bits below kKeyLowBit do not tell two values
// apart), and where too many are equal to it, the vector number up to which they are needed.
template <typename T, int PER>
__device__ __forceinline__ TopBound top_bound(const uint32_t (&key)[PER], const int (&vec)[PER], int k, int enough) {
  constexpr int kLow = Elem<T>::kKeyLowBit;
  static_assert(32 * PER < 1 << 10, "ten bits hold a count");
  int valid = 0;
  uint32_t high = 0, low = ~0u;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    valid += key[j] > kKeyNegInf;
    high = max(high, key[j]);
    low = min(low, key[j]);
  }
  valid = __reduce_add_sync(~0u, valid);
  TopBound t{kKeyNegInf + 1, kKeyNegInf, 0x7fffffff};
  if (valid <= k) return t;
  high = __reduce_max_sync(~0u, high);
  low = __reduce_min_sync(~0u, low);
  // bits above the first in which the keys differ are common to all
  int b = high == low ? kLow - 1 : 31 - __clz(high ^ low);
  uint32_t bound = b < kLow ? high >> kLow << kLow : (b >= 31 ? 0 : high >> (b + 1) << (b + 1));
  int reach = 32 * PER;
  // two bits at a time: the counts of three thresholds side by side in one sum
  for (; b >= kLow && reach > enough; b -= 2) {
    const uint32_t half = b > kLow ? 1u << (b - 1) : 0u, one = 1u << b;  // the last bit alone: half 0
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      n += (key[j] >= (bound | half) ? 1u : 0u) + (key[j] >= (bound | one) ? 1u << 10 : 0u) +
           (key[j] >= (bound | one | half) ? 1u << 20 : 0u);
    n = __reduce_add_sync(~0u, n);
    const int n1 = n & 1023, n2 = n >> 10 & 1023, n3 = n >> 20;
    if (n3 >= k) {
      bound |= one | half;
      reach = n3;
    } else if (n2 >= k) {
      bound |= one;
      reach = n2;
    } else if (n1 >= k) {
      bound |= half;
      reach = n1;
    }
  }
  t.key = max(bound, kKeyNegInf + 1);
  if (reach > enough) {  // every bit is fixed: the groups that tie differ below kLow at most
    t.tie_top = bound | ((1u << kLow) - 1u);
    int above = 0, most = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      above += key[j] > t.tie_top;
      most = max(most, vec[j]);
    }
    above = __reduce_add_sync(~0u, above);
    most = __reduce_max_sync(~0u, most);
    t.vec = 0;
    for (int c = 31 - __clz(most | 1); c >= 0; --c) {
      const int test = t.vec | ((1 << c) - 1);
      int n = 0;
#pragma unroll
      for (int j = 0; j < PER; ++j) n += key[j] >= t.key && key[j] <= t.tie_top && vec[j] <= test;
      if (__reduce_add_sync(~0u, n) < k - above) t.vec |= 1 << c;
    }
  }
  return t;
}

// Places `n` distinct keys in descending order: put(place, key) for the first k.
template <typename F>
__device__ __forceinline__ void place_keys(const uint64_t* keys, int n, int k, F&& put) {
  for (int j = threadIdx.x; j < n; j += kTopThreads) {
    const uint64_t mine = keys[j];
    int place = 0;
#pragma unroll 8
    for (int o = 0; o < n; ++o) place += keys[o] > mine;
    if (place < k) put(place, mine);
  }
}

// The k largest logits of the block's part of a row, from every thread's largest one and
// where it met it: put(place, key), and the number of places that were filled.
template <typename T, typename F>
__device__ __forceinline__ int part_top(const Row<T>& row, const Part& part, const TopMax<T>& a, const TopGroups<T>& groups, int k,
                                        TopShared& sh, F&& put) {
  constexpr int kVec = Elem<T>::kVec;
  const int tid = threadIdx.x, lane = tid & 31;
  sh.key[tid] = order_key(a.max);
  sh.vec[tid] = a.max_vec;
  __syncthreads();
  if (tid < 32) {
    uint32_t key[kTopThreads / 32];
    int vec[kTopThreads / 32];
#pragma unroll
    for (int j = 0; j < kTopThreads / 32; ++j) {
      key[j] = sh.key[j * 32 + tid];
      vec[j] = sh.vec[j * 32 + tid];
    }
    // a few more threads than k cost less than the steps that would tell them apart
    const TopBound t = top_bound<T>(key, vec, k, 2 * k + 8);
    if (tid == 0) {
      sh.bound = t;
      sh.nlist = sh.ncand = 0;
    }
  }
  __syncthreads();
  const uint32_t bound = sh.bound.key, tie_top = sh.bound.tie_top;
  const int bound_vec = sh.bound.vec;
  const int per = 4 << groups.shift;  // vectors of a group
  if (sh.key[tid] >= bound) {
    for (int j = 0; part.begin + tid + j * per * kTopThreads < part.end; ++j) {
      const uint32_t largest = groups.largest(j);
      if (largest >= bound && (largest > tie_top || part.begin + tid + j * per * kTopThreads <= bound_vec)) {
        const int at = atomicAdd(&sh.nlist, 1);
        if (at < kTopList) sh.list[at] = j * kTopThreads + tid;
      }
    }
  }
  __syncthreads();
  const int nlist = sh.nlist;
  auto offer = [&](int i) {
    const uint4 raw = row.load_here(i);
    uint32_t hits = 0;  // a bit per element that reaches the bound
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const uint32_t key = order_key(vec_get<T>(raw, e));
      if (key >= bound && (key > tie_top || i <= bound_vec)) hits |= 1u << e;
    }
    if (hits == 0) return;
    int at = atomicAdd(&sh.ncand, __popc(hits));
    for (; hits; hits &= hits - 1, ++at) {
      const int e = __ffs(hits) - 1;
      if (at < kTopCandidates) sh.cand[at] = full_key(Elem<T>::to_float(row.p[row.first(i) + e]), row.first(i) + e);
    }
  };
  if (nlist <= kTopList) {
    for (int q = tid; q < nlist * per; q += kTopThreads) {
      const int item = static_cast<int>(sh.list[q / per]), j = item / kTopThreads, owner = item % kTopThreads;
      const int i = part.begin + owner + (j * per + q % per) * kTopThreads;
      if (i < part.end) offer(i);
    }
    if (part.head >= 0 && tid == kHeadThread) offer(part.head);
    if (part.tail >= 0 && tid == kTailThread) offer(part.tail);
  }
  __syncthreads();
  const int ncand = sh.ncand;
  if (nlist <= kTopList && ncand <= kTopCandidates) {
    place_keys(sh.cand, ncand, k, put);
    return min(ncand, k);
  }
  // many logits above the bound sit in few threads: one block-wide maximum per place
  uint64_t last = ~0ull;
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0;
    for_vectors<kTopThreads, true>(row, part, [&](int i, const uint4& raw, bool) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const uint64_t fk = full_key(vec_get<T>(raw, e), row.first(i) + e);
        if (fk < last && fk > best && static_cast<uint32_t>(fk >> 32) > kKeyNegInf) best = fk;
      }
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(~0u, best, o);
      best = other > best ? other : best;
    }
    if (lane == 0) sh.best[tid >> 5] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTopWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
    __syncthreads();
    if (best == 0) return j;  // nothing above -inf is left
    last = best;
    if (tid == 0) put(j, best);
  }
  return k;
}

// The row's k largest logits: of the block's part, or gathered from the cluster's parts.
template <typename T>
__device__ __forceinline__ void row_top(const Row<T>& row, const Part& part, const TopMax<T>& a, const TopGroups<T>& groups, int k,
                                        float max, float inv_t, float log_s, float* out_value, int32_t* out_index, TopShared& sh,
                                        uint64_t* gathered, int ctas) {
  auto write = [&](int place, uint64_t key) {
    const int v = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
    out_index[place] = v;
    out_value[place] = (key_value(static_cast<uint32_t>(key >> 32)) - max) * inv_t - log_s;
  };
  int found;
  if (ctas == 1) {
    found = part_top<T>(row, part, a, groups, k, sh, write);
  } else {
    const uint32_t rank = ptx::cluster_ctarank();
    const uint32_t to = ptx::mapa_shared(ptx::smem_u32(gathered + rank * k), 0);
    const int mine = part_top<T>(row, part, a, groups, k, sh, [&](int place, uint64_t key) { ptx::st_cluster_u64(to + place * 8, key); });
    if (threadIdx.x == 0) ptx::st_cluster_u32(ptx::mapa_shared(ptx::smem_u32(&sh.taken[rank]), 0), mine);
    ptx::cluster_sync();
    if (rank != 0) return;
    // closed up, in kTopCandidates = kMaxCluster kTopMaxK places
    int total = 0;
    for (int r = 0; r < ctas; ++r) {
      const int n = static_cast<int>(sh.taken[r]);
      for (int j = threadIdx.x; j < n; j += kTopThreads) sh.cand[total + j] = gathered[r * k + j];
      total += n;
    }
    __syncthreads();
    place_keys(sh.cand, total, k, write);
    found = min(total, k);
  }
  for (int j = found + threadIdx.x; j < k; j += kTopThreads) {
    out_index[j] = -1;
    out_value[j] = kNegInf;
  }
}

// ---------------------------------------------------------------- rows kept on chip

// A block's part of a row in shared memory: vector i at v[i - base].  The whole vectors come
// by bulk copies in chunks, each with a barrier of its own, so that the pass over the first
// runs while the others arrive; the ragged ones by plain loads of the threads that have them.
constexpr int kSlabChunks = 4;
struct SlabShared {
  uint64_t full[kSlabChunks];
  int abort;
};

template <typename T, int NT>
struct Slab {
  uint4* v;
  SlabShared* sh;
  Part part;
  int base, each;  // vectors per chunk
  int* status;
  int kernel;

  __device__ __forceinline__ void start(const Row<T>& row, const Part& part_, uint4* shared, SlabShared* sh_) {
    v = shared;
    sh = sh_;
    part = part_;
    status = row.status;
    kernel = row.kernel;
    base = part.head >= 0 ? part.head : part.begin;
    each = max(2, (part.end - part.begin + kSlabChunks * NT - 1) / (kSlabChunks * NT)) * NT;
    if (threadIdx.x == 0) {
#pragma unroll
      for (int q = 0; q < kSlabChunks; ++q) ptx::mbar_init(ptx::smem_u32(&sh->full[q]), 1);
      sh->abort = 0;
      ptx::fence_mbarrier_init();
#pragma unroll
      for (int q = 0; q < kSlabChunks; ++q) {
        const int b = min(part.end, part.begin + q * each), e = min(part.end, b + each);
        const uint32_t bar = ptx::smem_u32(&sh->full[q]);
        bool load = e > b;
        if (load)
          load = bounds_ok(row.whole(b) && row.whole(e - 1) && (reinterpret_cast<uintptr_t>(row.p + row.first(b)) & 15) == 0,
                           status, kernel, NSM_ROLE_PRODUCER, NSM_SITE_LOGITS);
        ptx::mbar_arrive_expect_tx(bar, load ? (e - b) * 16 : 0);
        if (load) ptx::bulk_load(ptx::smem_u32(v + (b - base)), row.p + row.first(b), (e - b) * 16, bar);
      }
    }
    if (part.head >= 0 && threadIdx.x == kHeadThread) v[part.head - base] = row.load(part.head);
    if (part.tail >= 0 && threadIdx.x == kTailThread) v[part.tail - base] = row.load(part.tail);
    __syncthreads();  // the barriers are there
  }
  __device__ __forceinline__ void wait(int q) const { wait_on(&sh->full[q]); }
  // Until a barrier's first phase is over.  After a wait that ran out (recorded) the block goes on with
  // what is there, so that every barrier is still met; drain() then waits once more.
  __device__ __forceinline__ void wait_on(uint64_t* bar) const {
    if (!ptx::mbar_wait_bounded(ptx::smem_u32(bar), 0, &sh->abort, kWaitNs)) {
      record_timeout(status, kernel, NSM_ROLE_PRODUCER, NSM_SITE_STAGE_FULL);
      sh->abort = 1;
    }
  }
  // use(i, vector) for this thread's vectors of chunk q.
  template <typename F>
  __device__ __forceinline__ void chunk(int q, F&& use) const {
    const int b = min(part.end, part.begin + q * each), e = min(part.end, b + each);
#pragma unroll 2
    for (int i = b + static_cast<int>(threadIdx.x); i < e; i += NT) use(i, v[i - base], true);
  }
  template <typename F>
  __device__ __forceinline__ void ragged(F&& use) const {
    if (part.head >= 0 && threadIdx.x == kHeadThread) use(part.head, v[part.head - base], false);
    if (part.tail >= 0 && threadIdx.x == kTailThread) use(part.tail, v[part.tail - base], false);
  }
  template <typename F>
  __device__ __forceinline__ void all(F&& use) const {
#pragma unroll 2
    for (int i = part.begin + static_cast<int>(threadIdx.x); i < part.end; i += NT) use(i, v[i - base], true);
    ragged(use);
  }
  // Before the block ends: no copy into its shared memory may be in flight.
  __device__ __forceinline__ void drain() const {
    if (*static_cast<volatile int*>(&sh->abort) == 0) return;
    int never = 0;
    if (threadIdx.x == 0) {
      for (int q = 0; q < kSlabChunks; ++q)
        if (!ptx::mbar_wait_bounded(ptx::smem_u32(&sh->full[q]), 0, &never, kWaitNs)) break;
    }
    __syncthreads();
  }
};

// ---------------------------------------------------------------- log probabilities

// A row's statistics from its totals: log q_v = (x_v - ref) / t - log_s.
struct RowLogprob {
  float ref, log_s, log2_s, entropy;
  bool empty;
};

template <bool ENT>
__device__ __forceinline__ RowLogprob row_logprob(const Totals& t, float inv_t) {
  RowLogprob s;
  s.empty = t.max == kNegInf && t.s == 0.f;  // a row of NaN has a NaN sum
  s.ref = s.empty ? 0.f : t.max;
  s.log_s = s.empty ? 0.f : logf(t.s);
  s.log2_s = s.empty ? 0.f : log2f(t.s);
  s.entropy = 0.f;
  if (ENT && !s.empty) {
    s.entropy = s.log_s - kLn2 * (t.sy / t.s);
    if (s.entropy < 0.f) s.entropy = 0.f;
  }
  return s;
}

// One thread writes the row's numbers.
template <bool ENT>
__device__ __forceinline__ void write_logprob(const LogprobArgs& g, int64_t r, const RowLogprob& s, int token, float x_token,
                                              float inv_t) {
  if (g.lse) g.lse[r] = s.empty ? kNegInf : s.ref * inv_t + s.log_s;
  if (ENT && g.entropy) g.entropy[r] = s.entropy;
  if (g.logprob) g.logprob[r] = token < 0 ? 0.f : (s.empty ? kNegInf : (x_token - s.ref) * inv_t - s.log_s);
}

// What the gradient pass of a row needs: q (ca + cb log2 q), and the token's own value.
struct TokenGradient {
  float ref, log2_s, ca, cb;
  bool zero;
};

// w logprob + h entropy: d/dx = (w (1[token] - q) - h q (log q + entropy)) / t.  low: what the
// reference lost to rounding.
__device__ __forceinline__ TokenGradient token_gradient(float w, float h, const RowLogprob& s, float low, float c, float inv_t) {
  TokenGradient k;
  k.zero = s.empty || (w == 0.f && h == 0.f);
  k.ref = s.ref;
  k.log2_s = fmaf(low, c, s.log2_s);
  k.ca = -(w + h * s.entropy) * inv_t;
  k.cb = -h * kLn2 * inv_t;
  return k;
}

// The gradient at the token itself: 1 - q without cancellation; 0 where it is masked.
__device__ __forceinline__ float gradient_at_token(float w, float h, const RowLogprob& s, float low, float x_token, float inv_t) {
  const float log_q = ((x_token - s.ref) - low) * inv_t - s.log_s;
  if (log_q == kNegInf) return 0.f;
  return -(w * expm1f(log_q) + (h == 0.f ? 0.f : h * expf(log_q) * (log_q + s.entropy))) * inv_t;
}

// The gradients of the vectors that each(use) gives this thread, and then the token's own over
// what was written there (at_token()), by the thread that wrote it (`mine`).  same: gradient and logits are
// aligned alike, so that whole vectors are whole 16-byte stores.
template <typename T, bool ENT, typename E, typename F>
__device__ __forceinline__ void store_token_gradients(const Row<T>& row, const Row<T>& out, const Part& part, const TokenGradient& k,
                                                      int token, bool mine, float c, E&& each, F&& at_token) {
  const bool same = row.lead == out.lead;
  each([&](int i, const uint4& raw, bool whole) {
    const uint4 grad = gradient_vec<T, ENT>(raw, k.ref, c, k.log2_s, k.ca, k.cb);
    if (whole && same) out.store_whole(i, grad);
    else out.store(row.first(i), grad);
  });
  if (mine && bounds_ok(token >= 0 && token < out.vocab, out.status, out.kernel, 0, NSM_SITE_GRADIENT))
    out.p[token] = Elem<T>::from_float(at_token());
}

// Whether thread `tid` of NT has the vector that holds element v (v < 0: no).
template <int NT, typename T>
__device__ __forceinline__ bool owns(const Row<T>& row, const Part& part, int v) {
  if (v < 0) return false;
  const int at = (v + row.lead) / Elem<T>::kVec, tid = threadIdx.x;
  if (at == part.head) return tid == kHeadThread;
  if (at == part.tail) return tid == kTailThread;
  return at >= part.begin && at < part.end && (at - part.begin) % NT == tid;
}

// A cluster of CTAs per row (one CTA where there are rows enough).  TOP: dynamic shared
// memory holds rank 0's gathered keys (ctas k of them where ctas > 1), then the groups' tops.
template <typename T, bool ENT, bool TOP, bool GRAD, int NT>
__global__ void __launch_bounds__(NT, TOP ? 6 : 1280 / NT) k_logprobs(const LogprobArgs g, int group_shift, int* status) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ TotalsShared totals;
  __shared__ typename std::conditional<TOP, TopShared, int>::type top;
  grid_dependency_sync();
  release_dependents();
  const int ctas = static_cast<int>(ptx::cluster_nctarank()), rank = static_cast<int>(ptx::cluster_ctarank());
  start_totals(totals, ctas);
  const int64_t r = blockIdx.x / ctas;
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_LOGPROBS);
  const Part part = part_of(row, rank, ctas);
  int64_t token64 = g.tokens ? load_index(g.tokens, g.tokens_wide, r) : -1;
  const int token = token64 < 0 || token64 >= vocab ? -1 : static_cast<int>(token64);
  const float x_token = token >= 0 ? Elem<T>::to_float(row.p[token]) : kNegInf;
  uint64_t* gathered = reinterpret_cast<uint64_t*>(dynamic);
  TopGroups<T> groups{reinterpret_cast<typename TopGroups<T>::Key*>(gathered + (ctas > 1 ? ctas * g.k : 0)), group_shift, kNegInf};
  Sums a;
  TopMax<T> seen;
  for_batches<NT, TOP>(row, part,
              [&](int i, const uint4& raw, bool) {
                const float m = add_vec<T, ENT>(a, raw, c);
                if (TOP) {
                  seen.see(m, i);
                  groups.running = fmaxf(groups.running, m);
                }
              },
              [&](int n) {
                if (TOP) groups.batch(n);
              });
  const Totals t = row_totals<ENT, NT>(a, c, totals, ctas, status, NSM_KERNEL_LOGPROBS);
  const RowLogprob s = row_logprob<ENT>(t, inv_t);
  if (rank == 0 && threadIdx.x == 0) write_logprob<ENT>(g, r, s, token, x_token, inv_t);
  if constexpr (GRAD) {
    const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_LOGPROBS);
    const float w = g.d_logprob && token >= 0 ? g.d_logprob[r] : 0.f;
    const float h = ENT && g.d_entropy ? g.d_entropy[r] : 0.f;
    const TokenGradient k = token_gradient(w, h, s, 0.f, c, inv_t);
    if (k.zero) {
      zero_part<NT>(out, rank, ctas);
    } else {
      store_token_gradients<T, ENT>(row, out, part, k, token, owns<NT>(row, part, token), c,
                                    [&](auto&& use) { for_vectors<NT>(row, part, use); },
                                    [&] { return gradient_at_token(w, h, s, 0.f, x_token, inv_t); });
    }
  }
  if constexpr (TOP) {
    float* value = g.top_logprob + r * g.k;
    int32_t* index = g.top_index + r * g.k;
    if (s.log_s != s.log_s) {  // NaN or +inf in the row
      if (rank == 0) {
        for (int j = threadIdx.x; j < g.k; j += NT) {
          value[j] = s.log_s;
          index[j] = -1;
        }
      }
    } else {
      row_top<T>(row, part, seen, groups, g.k, s.ref, inv_t, s.log_s, value, index, top, gathered, ctas);
    }
  }
}

// Forward and backward in one pass over memory: the row stays in the shared memory of the
// cluster's blocks between its sums and its gradient.
template <typename T, bool ENT, int NT>
__global__ void __launch_bounds__(NT) k_logprobs_resident(const LogprobArgs g, int* status) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ TotalsShared totals;
  __shared__ SlabShared slab_shared;
  grid_dependency_sync();
  release_dependents();
  const int ctas = static_cast<int>(ptx::cluster_nctarank()), rank = static_cast<int>(ptx::cluster_ctarank());
  start_totals(totals, ctas);
  const int64_t r = blockIdx.x / ctas;
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_LOGPROBS);
  const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_LOGPROBS);
  Slab<T, NT> slab;
  slab.start(row, part_of(row, rank, ctas), reinterpret_cast<uint4*>(dynamic), &slab_shared);
  const int64_t token64 = g.tokens ? load_index(g.tokens, g.tokens_wide, r) : -1;
  const int token = token64 < 0 || token64 >= vocab ? -1 : static_cast<int>(token64);
  const float x_token = token >= 0 ? Elem<T>::to_float(row.p[token]) : kNegInf;
  const float w = g.d_logprob && token >= 0 ? g.d_logprob[r] : 0.f;
  const float h = ENT && g.d_entropy ? g.d_entropy[r] : 0.f;
  Sums a;
  auto add = [&](int, const uint4& raw, bool) { add_vec<T, ENT>(a, raw, c); };
  slab.ragged(add);
#pragma unroll 1
  for (int q = 0; q < kSlabChunks; ++q) {
    slab.wait(q);
    slab.chunk(q, add);
  }
  const Totals t = row_totals<ENT, NT>(a, c, totals, ctas, status, NSM_KERNEL_LOGPROBS);
  const RowLogprob s = row_logprob<ENT>(t, inv_t);
  if (rank == 0 && threadIdx.x == 0) write_logprob<ENT>(g, r, s, token, x_token, inv_t);
  const TokenGradient k = token_gradient(w, h, s, 0.f, c, inv_t);
  if (k.zero) {
    zero_part<NT>(out, rank, ctas);
  } else {
    store_token_gradients<T, ENT>(row, out, slab.part, k, token, owns<NT>(row, slab.part, token), c, [&](auto&& use) { slab.all(use); },
                                  [&] { return gradient_at_token(w, h, s, 0.f, x_token, inv_t); });
  }
  slab.drain();
}

// The backward pass alone: pieces of rows, every element on its own.
template <typename T, bool ENT, int NT>
__global__ void __launch_bounds__(NT, 1536 / NT) k_logprobs_backward(const LogprobArgs g, int pieces, int* status) {
  grid_dependency_sync();
  release_dependents();
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const int64_t total = g.v.rows * pieces;
  for (int64_t work = blockIdx.x; work < total; work += gridDim.x) {
    const int64_t r = work / pieces;
    const int piece = static_cast<int>(work - r * pieces);
    const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_LOGPROBS);
    const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_LOGPROBS);
    const int64_t token64 = g.tokens ? load_index(g.tokens, g.tokens_wide, r) : -1;
    const int token = token64 < 0 || token64 >= vocab ? -1 : static_cast<int>(token64);
    const float w = g.d_logprob && token >= 0 ? g.d_logprob[r] : 0.f;
    const float h = ENT && g.d_entropy ? g.d_entropy[r] : 0.f;
    const float lse = g.in_lse[r];
    const float ref = lse * g.v.t, low = fmaf(lse, g.v.t, -ref);
    const RowLogprob s{ref, 0.f, 0.f, ENT && g.d_entropy ? g.in_entropy[r] : 0.f, lse == kNegInf};
    if (s.empty || (w == 0.f && h == 0.f)) {
      zero_part<NT>(out, piece, pieces);
      continue;
    }
    // in place, another block may have written the token's own gradient already: only the
    // thread that has the token's vector reads its logit, before it writes there
    const Part part = part_of(row, piece, pieces);
    const bool mine = owns<NT>(row, part, token);
    const float x_token = mine ? Elem<T>::to_float(row.p[token]) : kNegInf;
    const TokenGradient k = token_gradient(w, h, s, low, c, inv_t);
    store_token_gradients<T, ENT>(row, out, part, k, token, mine, c, [&](auto&& use) { for_vectors<NT>(row, part, use); },
                                  [&] { return gradient_at_token(w, h, s, low, x_token, inv_t); });
  }
}

// ---------------------------------------------------------------- distillation

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// The teacher of a row lives in one warp (a warp of its own beside the ones that sum the row,
// so that its many small steps cost them no time): lane l has entries l, l + 32, ...
constexpr int kLaneEntries = kDistillMaxK / 32;
struct Entries {
  int v[kLaneEntries];  // its token, -1 where it does not count
  float log_p[kLaneEntries], p[kLaneEntries], x[kLaneEntries];  // x: the student's logit
};
// What the row's other threads need of it.
struct TeacherStats {
  Totals inside;          // the student's sum over the entries
  float p_rest, lacking;  // the tail's 1 - sum p, as at least 0 and as it is
  int any;                // there is a target
};

template <typename V>
__device__ __forceinline__ V load_if(bool p, const void* from, int64_t i, V otherwise) {
  return p ? static_cast<const V*>(from)[i] : otherwise;
}

// The entries' tokens and scores (in log_p); equal tokens are still there.  Every load is on its
// way before the first is looked at: under load each takes microseconds.
__device__ __forceinline__ void load_entries(Entries& e, const DistillArgs& g, int64_t r) {
  const int lane = threadIdx.x & 31;
  const int64_t at_index = r * g.ldi + lane, at_score = r * g.ldt + lane;
  int64_t v[kLaneEntries];
  if (g.index_wide) {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) v[u] = load_if<int64_t>(lane + 32 * u < g.k, g.index, at_index + 32 * u, -1);
  } else {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) v[u] = load_if<int32_t>(lane + 32 * u < g.k, g.index, at_index + 32 * u, -1);
  }
  if (g.teacher_dtype == NSM_FP32) {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) e.log_p[u] = load_if<float>(lane + 32 * u < g.k, g.teacher, at_score + 32 * u, kNegInf);
  } else {
    const bool bf16 = g.teacher_dtype == NSM_BF16;
    uint16_t h[kLaneEntries];
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) h[u] = load_if<uint16_t>(lane + 32 * u < g.k, g.teacher, at_score + 32 * u, 0);
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u)
      e.log_p[u] = bf16 ? __bfloat162float(__ushort_as_bfloat16(h[u])) : __half2float(__ushort_as_half(h[u]));
  }
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u) {
    e.v[u] = v[u] >= 0 && v[u] < g.v.vocab ? static_cast<int>(v[u]) : -1;
    e.x[u] = kNegInf;
  }
}

// The student's logits at the entries' tokens, read from the row.
template <typename T>
__device__ __forceinline__ void load_logits(Entries& e, const Row<T>& row) {
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u)
    if (e.v[u] >= 0) e.x[u] = Elem<T>::to_float(row.p[e.v[u]]);
}

// Of equal tokens the first counts; then the teacher's probabilities (the student is not asked
// yet: while its row is on the way).
__device__ __forceinline__ TeacherStats teacher_stats(Entries& e, const DistillArgs& g) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = kLaneEntries - 1; u >= 0; --u) {  // later groups first: earlier ones are whole
    if (32 * u >= g.k) continue;
    int v = e.v[u];
    const uint32_t same = __match_any_sync(~0u, v >= 0 ? v : -1 - lane);
    if (same & ((1u << lane) - 1u)) v = -1;
#pragma unroll
    for (int w = 0; w < u; ++w)
#pragma unroll 8
      for (int l = 0; l < 32; ++l)
        if (__shfl_sync(~0u, e.v[w], l) == v) v = -1;
    e.v[u] = v;
  }
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u)
    if (e.v[u] < 0) e.log_p[u] = kNegInf;
  TeacherStats t;
  t.p_rest = t.lacking = 0.f;
  if (g.tail) {
    // 1 - sum p as (1 - largest p) - the others: the teacher's rest is often a small part of
    // what its first entry leaves (64-bit sums are too slow here: they cost half the row's time)
    float m = kNegInf, others = 0.f;
    bool some = false;
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) {
      m = fmaxf(m, e.log_p[u]);
      some |= e.v[u] >= 0;
    }
    const float largest = warp_max(m);
    bool taken = false;
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) {
      if (32 * u >= g.k) continue;
      const uint32_t at = __ballot_sync(~0u, !taken && e.log_p[u] == largest);  // its first holder
      const bool is_largest = at && (at & -at) == 1u << lane && !taken;
      if (!is_largest && !(e.log_p[u] == kNegInf)) others += expf(e.log_p[u]);
      taken |= at != 0;
    }
    t.lacking = (largest == kNegInf ? 1.f : -expm1f(largest)) - warp_sum(others);
    t.p_rest = t.lacking < 0.f ? 0.f : t.lacking;
    t.any = __any_sync(~0u, some);
  } else {
    float m = kNegInf, total = 0.f;
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) {
      if (e.v[u] >= 0) e.log_p[u] *= g.v.inv_t;
      m = fmaxf(m, e.log_p[u]);
    }
    m = warp_max(m);
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u)  // a NaN entry makes the sum, and with it every p, a NaN
      if (e.v[u] >= 0 && !(e.log_p[u] == kNegInf)) total += m == kNegInf ? e.log_p[u] : expf(e.log_p[u] - m);
    total = warp_sum(total);
    const float log_total = logf(total);
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u)
      if (!(e.log_p[u] == kNegInf)) e.log_p[u] = (e.log_p[u] - m) - log_total;
    t.any = m != kNegInf || total != total;
  }
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u) e.p[u] = expf(e.log_p[u]);
  t.inside = Totals{kNegInf, 0.f, 0.f};
  return t;
}

// The student's sum over the entries that count.
__device__ __forceinline__ Totals inside_totals(const Entries& e, float c) {
  float max = kNegInf, s = 0.f;
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u)
    if (e.v[u] >= 0) max = fmaxf(max, e.x[u]);
  max = warp_max(max);
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u)
    if (e.v[u] >= 0 && !(e.x[u] == kNegInf)) s += max == kNegInf ? e.x[u] : ex2((e.x[u] - max) * c);  // a NaN stays one
  return Totals{max, warp_sum(s), 0.f};
}

// The student's row: log q_v = (x_v - lse_ref) / t - lse_log,
// rest = log q_rest, with rest_ref where the sum outside the entries stands.
// *_low: what the references lost to rounding.
struct Student {
  float lse_ref, lse_log, rest_ref, rest;
  bool empty;
  float lse_low, rest_low;
};

__device__ __forceinline__ Student student_of(const TeacherStats& t, const Totals& outside, float c, float inv_t) {
  Totals all{fmaxf(outside.max, t.inside.max), outside.s, 0.f};
  float inside_s = t.inside.s, none = 0.f;
  rebase<false>(all.s, none, outside.max, all.max, c);
  rebase<false>(inside_s, none, t.inside.max, all.max, c);
  all.s += inside_s;
  Student st;
  st.lse_low = st.rest_low = 0.f;
  st.empty = all.max == kNegInf && all.s == 0.f;
  const bool no_rest = outside.max == kNegInf && outside.s == 0.f;
  st.lse_ref = st.empty ? 0.f : all.max;
  st.lse_log = st.empty ? 0.f : logf(all.s);
  st.rest_ref = no_rest ? 0.f : outside.max;
  st.rest = no_rest ? kNegInf : (outside.max - st.lse_ref) * inv_t + (logf(outside.s) - st.lse_log);
  return st;
}

// The same from the lse and rest that the forward pass left.
__device__ __forceinline__ Student student_from(const DistillArgs& g, int64_t r) {
  const float lse = g.in_lse[r], rest = g.tail ? g.in_rest[r] : 0.f, t = g.v.t;
  Student st{lse * t, 0.f, 0.f, rest, lse == kNegInf, 0.f, 0.f};
  st.lse_low = fmaf(lse, t, -st.lse_ref);
  if (rest != kNegInf) {
    const float sum = lse + rest, b = sum - lse;  // and the sum's rounding, exactly
    st.rest_ref = sum * t;
    st.rest_low = fmaf(sum, t, -st.rest_ref) + ((lse - (sum - b)) + (rest - b)) * t;
  }
  return st;
}

// The teacher's warp writes the row's loss, lse and rest.
__device__ __forceinline__ void write_loss(const DistillArgs& g, int64_t r, const Entries& e, const TeacherStats& t,
                                           const Student& st) {
  const float inv_t = g.v.inv_t, p_rest = st.rest == kNegInf ? 0.f : t.p_rest;
  float loss = 0.f;
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u)
    if (e.p[u] > 0.f || e.p[u] != e.p[u]) loss += e.p[u] * (e.log_p[u] - ((e.x[u] - st.lse_ref) * inv_t - st.lse_log));
  loss = warp_sum(loss);
  if (p_rest > 0.f || p_rest != p_rest) loss += p_rest * (logf(p_rest) - st.rest);
  if ((threadIdx.x & 31) == 0) {
    if (g.loss) g.loss[r] = t.any ? loss : 0.f;
    if (g.lse) g.lse[r] = st.empty ? kNegInf : st.lse_ref * inv_t + st.lse_log;
    if (g.rest) g.rest[r] = st.rest;
  }
}

// w loss: d/dx = w / t (q (1 + excess) - p) at the entries, and outside them, with the tail,
// q (1 + excess) - p_rest q / q_rest = (q / q_rest) (q_rest (1 + excess) - p_rest), as
// scale 2^((x - ref) c - log2_s).  excess = sum p + p_rest - 1.
struct EntryGradient {
  float ref, log2_s, scale, unit, excess;
  bool zero;
};

// From the sums outside the entries; what the threads of the dense pass need.
__device__ __forceinline__ EntryGradient entry_gradient(const TeacherStats& t, const Totals& outside, float w, int tail, float c,
                                                        float inv_t) {
  float all_max = fmaxf(outside.max, t.inside.max), out_s = outside.s, in_s = t.inside.s, none = 0.f;
  rebase<false>(out_s, none, outside.max, all_max, c);
  rebase<false>(in_s, none, t.inside.max, all_max, c);
  const float all_s = out_s + in_s;
  const bool empty = all_max == kNegInf && all_s == 0.f, no_rest = outside.max == kNegInf && outside.s == 0.f;
  EntryGradient k;
  k.zero = empty || !t.any || w == 0.f;
  const float p_rest = no_rest ? 0.f : t.p_rest;
  k.excess = tail ? p_rest - t.lacking : 0.f;
  k.unit = w * inv_t;
  k.ref = tail ? outside.max : all_max;
  k.log2_s = log2f(tail ? outside.s : all_s);
  k.scale = tail ? k.unit * (out_s / all_s * (1.f + k.excess) - p_rest) : k.unit;
  if (tail && no_rest) k.ref = k.log2_s = k.scale = 0.f;  // nothing is there
  return k;
}
// From the statistics that the forward pass left.
__device__ __forceinline__ EntryGradient entry_gradient(const TeacherStats& t, const Student& s, float w, int tail, float c,
                                                        float inv_t) {
  EntryGradient k;
  k.zero = s.empty || !t.any || w == 0.f;
  const float p_rest = s.rest == kNegInf ? 0.f : t.p_rest;
  k.excess = tail ? p_rest - t.lacking : 0.f;
  k.unit = w * inv_t;
  k.ref = tail ? s.rest_ref : s.lse_ref;
  k.log2_s = (tail ? s.rest_low : s.lse_low) * c;
  k.scale = !tail ? k.unit : s.rest == kNegInf ? 0.f : k.unit * (expf(s.rest) * (1.f + k.excess) - p_rest);
  return k;
}

template <typename T>
__device__ __forceinline__ bool in_part(const Row<T>& row, const Part& part, int v) {
  const int at = (v + row.lead) / Elem<T>::kVec;
  return (at >= part.begin && at < part.end) || at == part.head || at == part.tail;
}

template <typename T>
__device__ __forceinline__ void store_dense(const Row<T>& row, const Row<T>& out, int i, const uint4& raw, bool whole,
                                            const EntryGradient& k, float c) {
  const uint4 grad = gradient_vec<T, false>(raw, k.ref, c, k.log2_s, k.scale, 0.f);
  if (whole && row.lead == out.lead) out.store_whole(i, grad);
  else out.store(row.first(i), grad);
}

// The teacher's warp writes the gradients at the entries of the block's part, over what the
// pass over the row wrote there.
template <typename T>
__device__ __forceinline__ void store_entries(const Row<T>& row, const Row<T>& out, const Part& part, const Entries& e,
                                              const Student& s, const EntryGradient& k, float inv_t) {
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u) {
    if (e.v[u] < 0 || !in_part(row, part, e.v[u])) continue;
    const float log_q = ((e.x[u] - s.lse_ref) - s.lse_low) * inv_t - s.lse_log, p = e.p[u];
    float grad = 0.f;
    if (log_q != kNegInf) {  // q - p without cancellation
      const float q = expf(log_q);
      grad = k.unit * ((p > 0.f || p != p ? p * expm1f(log_q - e.log_p[u]) : q) + q * k.excess);
    }
    if (bounds_ok(e.v[u] < out.vocab, out.status, out.kernel, 0, NSM_SITE_GRADIENT)) out.p[e.v[u]] = Elem<T>::from_float(grad);
  }
}

// NT threads sum the row (a cluster of blocks per row where rows are few), a warp more has the
// teacher.  GRAD: rows too long to stay in shared memory, read a second time.
template <typename T, bool GRAD, int NT>
__global__ void __launch_bounds__(NT + 32) k_distill(const DistillArgs g, int* status) {
  constexpr int kVec = Elem<T>::kVec;
  extern __shared__ __align__(16) uint8_t members[];  // a bit per element of vector i in byte i - part's first
  __shared__ TotalsShared totals;
  __shared__ TeacherStats shared_stats;
  grid_dependency_sync();
  release_dependents();
  const int ctas = static_cast<int>(ptx::cluster_nctarank()), rank = static_cast<int>(ptx::cluster_ctarank());
  start_totals(totals, ctas);
  const int64_t r = blockIdx.x / ctas;
  const int tid = threadIdx.x, vocab = g.v.vocab;
  const bool teacher = tid >= NT;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_DISTILL);
  const Part part = part_of(row, rank, ctas);
  // head is vector begin - 1 and tail vector end: the part's vectors from `base` on
  const int base = part.head >= 0 ? part.head : part.begin;
  const int bytes = (part.tail >= 0 ? part.tail + 1 : part.end) - base;
  Entries e;
  Sums a;
  if (teacher) load_entries(e, g, r);
  else
    for (int i = tid; i < (bytes + 15) / 16; i += NT) reinterpret_cast<uint4*>(members)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (teacher) {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) {
      if (e.v[u] >= 0 && in_part(row, part, e.v[u])) {
        const int at = e.v[u] + row.lead, i = at / kVec - base;
        atomicOr(reinterpret_cast<uint32_t*>(members) + i / 4, 1u << (8 * (i & 3) + at % kVec));
      }
    }
  }
  __syncthreads();
  if (teacher) {
    TeacherStats t = teacher_stats(e, g);
    load_logits(e, row);
    t.inside = inside_totals(e, c);
    if (tid == NT) shared_stats = t;
  } else {  // the student outside the entries
    for_vectors<NT>(row, part, [&](int i, const uint4& raw, bool) {
      const uint32_t bits = members[i - base];
      uint4 v = raw;
      if (bits) vec_mask<T>(v, bits);
      add_vec<T, false>(a, v, c);
    });
  }
  const Totals outside = row_totals<false, NT>(a, c, totals, ctas, status, NSM_KERNEL_DISTILL);
  const TeacherStats t = shared_stats;
  Student st;
  if (teacher) {
    st = student_of(t, outside, c, inv_t);
    if (rank == 0) write_loss(g, r, e, t, st);
  }
  if constexpr (GRAD) {
    const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_DISTILL);
    const EntryGradient k = entry_gradient(t, outside, g.d_loss ? g.d_loss[r] : 1.f, g.tail, c, inv_t);
    if (!teacher) {
      if (k.zero) zero_part<NT>(out, rank, ctas);
      else
        for_vectors<NT>(row, part, [&](int i, const uint4& raw, bool whole) {
          store_dense(row, out, i, raw, whole, k, c);
        });
    }
    __syncthreads();
    if (teacher && !k.zero) store_entries(row, out, part, e, st, k, inv_t);
  }
}

// Forward and backward in one pass over memory, as k_logprobs_resident.
template <typename T, int NT>
__global__ void __launch_bounds__(NT + 32) k_distill_resident(const DistillArgs g, int* status) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  __shared__ TotalsShared totals;
  __shared__ TeacherStats shared_stats;
  __shared__ SlabShared slab_shared;
  __shared__ uint64_t ready[kSlabChunks];
  grid_dependency_sync();
  release_dependents();
  const int ctas = static_cast<int>(ptx::cluster_nctarank()), rank = static_cast<int>(ptx::cluster_ctarank());
  start_totals(totals, ctas);
  const int64_t r = blockIdx.x / ctas;
  const int tid = threadIdx.x, vocab = g.v.vocab;
  const bool teacher = tid >= NT;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_DISTILL);
  const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_DISTILL);
  const Part part = part_of(row, rank, ctas);
  if (tid < kSlabChunks) ptx::mbar_init(ptx::smem_u32(&ready[tid]), 1);
  Slab<T, NT> slab;
  slab.start(row, part, reinterpret_cast<uint4*>(dynamic), &slab_shared);  // ends with a barrier
  const float w = g.d_loss ? g.d_loss[r] : 1.f;
  Entries e;
  Sums a;
  if (teacher) {
    load_entries(e, g, r);
    // What other blocks of the cluster hold of the row comes from memory; of the rest, the chunk
    // it comes with and its place there.
    T elsewhere[kLaneEntries];
    int chunk_of[kLaneEntries];
    T* place[kLaneEntries];
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) {
      const int at = (e.v[u] + row.lead) / Elem<T>::kVec, from = at - part.begin;
      chunk_of[u] = -1;
      place[u] = reinterpret_cast<T*>(slab.v) + (e.v[u] + row.lead - slab.base * Elem<T>::kVec);
      if (e.v[u] < 0) continue;
      if (at >= part.begin && at < part.end) chunk_of[u] = (from >= slab.each) + (from >= 2 * slab.each) + (from >= 3 * slab.each);
      else if (at == part.head || at == part.tail) chunk_of[u] = 0;
      else elsewhere[u] = row.p[e.v[u]];
    }
    // The entries leave the sums outside them: chunk by chunk as it arrives, their logits are
    // taken and -inf goes in their place.
    static_assert(kSlabChunks == 4, "three comparisons find the chunk");
#pragma unroll 1
    for (int q = 0; q < kSlabChunks; ++q) {
      slab.wait(q);
#pragma unroll
      for (int u = 0; u < kLaneEntries; ++u)
        if (chunk_of[u] == q) e.x[u] = Elem<T>::to_float(*place[u]);
      __syncwarp();  // equal tokens have all read
#pragma unroll
      for (int u = 0; u < kLaneEntries; ++u)
        if (chunk_of[u] == q) *place[u] = Elem<T>::from_float(kNegInf);
      __syncwarp();
      if (tid == NT) ptx::mbar_arrive(ptx::smem_u32(&ready[q]));
    }
    TeacherStats t = teacher_stats(e, g);  // while the other warps are in the row
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u)
      if (e.v[u] >= 0 && chunk_of[u] < 0) e.x[u] = Elem<T>::to_float(elsewhere[u]);
    t.inside = inside_totals(e, c);
    if (tid == NT) shared_stats = t;
  } else {
    auto add = [&](int, const uint4& raw, bool) { add_vec<T, false>(a, raw, c); };
#pragma unroll 1
    for (int q = 0; q < kSlabChunks; ++q) {
      slab.wait(q);
      slab.wait_on(&ready[q]);
      slab.chunk(q, add);
      if (q == 0) slab.ragged(add);
    }
  }
  const Totals outside = row_totals<false, NT>(a, c, totals, ctas, status, NSM_KERNEL_DISTILL);
  const TeacherStats t = shared_stats;
  const EntryGradient k = entry_gradient(t, outside, w, g.tail, c, inv_t);
  Student st;
  if (teacher) {
    st = student_of(t, outside, c, inv_t);
    if (rank == 0) write_loss(g, r, e, t, st);
  } else if (k.zero) {
    zero_part<NT>(out, rank, ctas);
  } else {
    slab.all([&](int i, const uint4& raw, bool whole) { store_dense(row, out, i, raw, whole, k, c);
    });
  }
  __syncthreads();
  if (teacher && !k.zero) store_entries(row, out, part, e, st, k, inv_t);
  slab.drain();
}

// The backward pass alone, in pieces of rows.
template <typename T, int NT>
__global__ void __launch_bounds__(NT + 32, 1280 / (NT + 32)) k_distill_backward(const DistillArgs g, int pieces, int* status) {
  __shared__ TeacherStats shared_stats;
  grid_dependency_sync();
  release_dependents();
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  const bool teacher = threadIdx.x >= NT;
  const int64_t total = g.v.rows * pieces;
  for (int64_t work = blockIdx.x; work < total; work += gridDim.x) {
    const int64_t r = work / pieces;
    const int piece = static_cast<int>(work - r * pieces);
    const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_DISTILL);
    const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_DISTILL);
    const Part part = part_of(row, piece, pieces);
    const float w = g.d_loss ? g.d_loss[r] : 1.f;
    if (w == 0.f || g.in_lse[r] == kNegInf) {
      if (!teacher) zero_part<NT>(out, piece, pieces);
      continue;
    }
    const Student st = student_from(g, r);
    Entries e;
    if (teacher) {
      load_entries(e, g, r);
      const TeacherStats t = teacher_stats(e, g);
      load_logits(e, row);  // of entries that count, in time for store_entries
      if (threadIdx.x == NT) shared_stats = t;
    }
    FirstFour<NT, T> first;
    if (!teacher) first.load(row, part);
    __syncthreads();
    const TeacherStats t = shared_stats;
    const EntryGradient k = entry_gradient(t, st, w, g.tail, c, inv_t);
    if (!teacher) {
      if (k.zero) zero_part<NT>(out, piece, pieces);
      else first.use_all(row, part, [&](int i, const uint4& raw, bool whole) { store_dense(row, out, i, raw, whole, k, c); });
    }
    __syncthreads();  // and shared_stats is free again
    if (teacher && !k.zero) store_entries(row, out, part, e, st, k, inv_t);
  }
}

// ---------------------------------------------------------------- short rows

// A warp per row, the row in its registers: N vectors per lane at most.  Forward, forward and
// backward, or the backward pass alone; for rows so short that a block's barriers and its
// threads' own fixed work would cost more than the row.
constexpr int kShortWarps = 4;
enum ShortMode { kShortForward, kShortTop, kShortBoth, kShortBackward };  // kShortTop: forward with alternatives

// The k largest logits of a row that a warp has in its registers.
template <typename T, int N>
__device__ __forceinline__ void short_top(const Row<T>& row, const uint4 (&raw)[N], int k, const RowLogprob& s, float inv_t,
                                          float* value, int32_t* index, uint64_t* cand, int* count) {
  constexpr int kVec = Elem<T>::kVec;
  const int lane = threadIdx.x & 31;
  if (s.log_s != s.log_s) {  // NaN or +inf in the row
    for (int j = lane; j < k; j += 32) {
      value[j] = s.log_s;
      index[j] = -1;
    }
    return;
  }
  uint32_t key[N];
  int vec[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    vec[u] = lane + 32 * u;
    key[u] = order_key(Elem<T>::largest(raw[u]));
  }
  // at most max(k, 128) vectors reach the bound: their elements fit the candidates
  const TopBound t = top_bound<T>(key, vec, k, max(k, min(2 * k + 8, kTopMaxK)));
  if (lane == 0) *count = 0;
  __syncwarp();
#pragma unroll
  for (int u = 0; u < N; ++u) {
    if (key[u] < t.key || (key[u] <= t.tie_top && vec[u] > t.vec)) continue;
    uint32_t hits = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const uint32_t ek = order_key(vec_get<T>(raw[u], e));
      if (ek >= t.key && (ek > t.tie_top || vec[u] <= t.vec)) hits |= 1u << e;
    }
    int at = atomicAdd(count, __popc(hits));
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      if (hits >> e & 1) cand[at++] = full_key(vec_get<T>(raw[u], e), row.first(vec[u]) + e);
  }
  __syncwarp();
  const int n = *count;
  for (int j = lane; j < n; j += 32) {
    const uint64_t mine = cand[j];
    int place = 0;
#pragma unroll 8
    for (int o = 0; o < n; ++o) place += cand[o] > mine;
    if (place < k) {
      index[place] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(mine));
      value[place] = (key_value(static_cast<uint32_t>(mine >> 32)) - s.ref) * inv_t - s.log_s;
    }
  }
  for (int j = n + lane; j < k; j += 32) {
    index[j] = -1;
    value[j] = kNegInf;
  }
  __syncwarp();
}

template <typename T, typename Args, bool ENT, int MODE, int N>
__global__ void __launch_bounds__(32 * kShortWarps) k_short(const Args g, int* status) {
  constexpr bool DISTILL = std::is_same<Args, DistillArgs>::value;
  constexpr int kVec = Elem<T>::kVec;
  constexpr int kKernel = DISTILL ? NSM_KERNEL_DISTILL : NSM_KERNEL_LOGPROBS;
  __shared__ uint32_t members[kShortWarps][DISTILL ? 32 * N / 4 : 1];  // a byte per vector, a bit per element
  __shared__ uint64_t cand[kShortWarps][MODE == kShortTop ? kTopCandidates : 1];
  __shared__ int ncand[kShortWarps];
  grid_dependency_sync();
  release_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kShortWarps + warp; r < g.v.rows;
       r += static_cast<int64_t>(gridDim.x) * kShortWarps) {
    const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, kKernel);
    const Part part = part_of(row, 0, 1);
    uint4 raw[N];
    uint4 none = make_uint4(0, 0, 0, 0);
    vec_mask<T>(none, 0xffu);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = lane + 32 * u;
      raw[u] = i >= part.begin && i < part.end ? row.load_whole(i) : none;
    }
    if (part.head == 0 && lane == 0) raw[0] = row.load(0);
    if (part.tail >= 0 && (part.tail & 31) == lane) {
      const uint4 tail = row.load(part.tail);
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (part.tail == lane + 32 * u) raw[u] = tail;
    }
    auto store = [&](bool zero, auto&& value) {  // the lane's vectors of the gradient
      const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, kKernel);
      const bool same = row.lead == out.lead;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int i = lane + 32 * u;
        if (i >= row.nvec) continue;
        uint4 grad = make_uint4(0, 0, 0, 0);
        if (!zero) grad = value(raw[u]);
        if (same && i >= part.begin && i < part.end) out.store_whole(i, grad);
        else out.store(row.first(i), grad);
      }
    };
    if constexpr (DISTILL) {
      Entries e;
      load_entries(e, g, r);
      load_logits(e, row);
      TeacherStats t = teacher_stats(e, g);
      t.inside = inside_totals(e, c);
      const float w = MODE == kShortForward || !g.d_loss ? 1.f : g.d_loss[r];
      EntryGradient k;
      Student st;
      if constexpr (MODE == kShortBackward) {
        st = student_from(g, r);
        k = entry_gradient(t, st, w, g.tail, c, inv_t);
      } else {
        // the row outside the entries
#pragma unroll
        for (int j = 0; j < N / 4; ++j) members[warp][lane + 32 * j] = 0;
        if (N < 4 && lane < 32 * N / 4) members[warp][lane] = 0;
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kLaneEntries; ++u) {
          const int at = e.v[u] + row.lead, i = at / kVec;
          if (e.v[u] >= 0) atomicOr(&members[warp][i / 4], 1u << (8 * (i & 3) + at % kVec));
        }
        __syncwarp();
        Sums a;
#pragma unroll
        for (int u = 0; u < N; ++u) {
          if (32 * u >= row.nvec) continue;
          uint4 v = raw[u];
          const uint32_t bits = reinterpret_cast<const uint8_t*>(members[warp])[lane + 32 * u];
          if (bits) vec_mask<T>(v, bits);
          add_vec<T, false>(a, v, c);
        }
        const Totals outside = warp_totals<false>(a, c);
        st = student_of(t, outside, c, inv_t);
        write_loss(g, r, e, t, st);
        k = entry_gradient(t, outside, w, g.tail, c, inv_t);
      }
      if constexpr (MODE != kShortForward) {  // kShortTop is not distillation's
        store(k.zero, [&](const uint4& v) { return gradient_vec<T, false>(v, k.ref, c, k.log2_s, k.scale, 0.f); });
        __syncwarp();  // the entries' own values go over what was written there
        if (!k.zero) {
          const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, kKernel);
          store_entries(row, out, part, e, st, k, inv_t);
        }
      }
    } else {
      const int64_t token64 = g.tokens ? load_index(g.tokens, g.tokens_wide, r) : -1;
      const int token = token64 < 0 || token64 >= vocab ? -1 : static_cast<int>(token64);
      const float x_token = token >= 0 ? Elem<T>::to_float(row.p[token]) : kNegInf;
      RowLogprob s;
      float low = 0.f;
      if constexpr (MODE == kShortBackward) {
        const float lse = g.in_lse[r];
        s = RowLogprob{lse * g.v.t, 0.f, 0.f, ENT && g.d_entropy ? g.in_entropy[r] : 0.f, lse == kNegInf};
        low = fmaf(lse, g.v.t, -s.ref);
      } else {
        Sums a;
#pragma unroll
        for (int u = 0; u < N; ++u)
          if (32 * u < row.nvec) add_vec<T, ENT>(a, raw[u], c);
        s = row_logprob<ENT>(warp_totals<ENT>(a, c), inv_t);
        if (lane == 0) write_logprob<ENT>(g, r, s, token, x_token, inv_t);
        if constexpr (MODE == kShortTop)
          short_top<T, N>(row, raw, g.k, s, inv_t, g.top_logprob + r * g.k, g.top_index + r * g.k, cand[warp], &ncand[warp]);
      }
      if constexpr (MODE == kShortBoth || MODE == kShortBackward) {
        const float w = g.d_logprob && token >= 0 ? g.d_logprob[r] : 0.f;
        const float h = ENT && g.d_entropy ? g.d_entropy[r] : 0.f;
        const TokenGradient k = token_gradient(w, h, s, low, c, inv_t);
        __syncwarp();  // in place: every lane has read the token's logit
        store(k.zero, [&](const uint4& v) { return gradient_vec<T, ENT>(v, k.ref, c, k.log2_s, k.ca, k.cb); });
        if (!k.zero && token >= 0 && ((token + row.lead) / kVec & 31) == lane) {
          const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, kKernel);
          if (bounds_ok(token < vocab, status, kKernel, 0, NSM_SITE_GRADIENT))
            out.p[token] = Elem<T>::from_float(gradient_at_token(w, h, s, low, x_token, inv_t));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- launches

// CTAs per row: where there are fewer rows than the GPU takes blocks at a time, a cluster
// shares each row, down to two vectors of a thread.
int cluster_for(int64_t rows, int nvec, int NT) {
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas * NT < 1024 * 152 && nvec >= ctas * 4 * NT) ctas *= 2;
  return ctas;
}

// Threads per row of a forward pass, and per piece of a row of a backward pass.  Measured on a
// GB300: 16384 x 4000 bf16 forward 29 us with 64 threads, 43 with 128; 8192 x 131072 302 with 128,
// 354 with 512; 16384 x 2100 backward 37 us with 64 and 58 with 256, 8192 x 131072 677 with 256.
int forward_threads(int nvec) { return nvec <= 1024 ? 64 : 128; }
int backward_threads(int nvec) { return nvec <= 1024 ? 64 : 256; }

// Pieces per row of a backward pass: `most` vectors each, less where rows are few.
int pieces_for(int64_t rows, int nvec, int most, int least) {
  int each = most;
  while (each > least && rows * ((nvec + each - 1) / each) < 8 * 152) each /= 2;
  return (nvec + each - 1) / each;
}

constexpr size_t kSlabBytes = 76 << 10, kSlabAlone = 112 << 10, kSlabMost = 216 << 10;
constexpr size_t kMembersMost = 160 << 10;  // of k_distill's bits per block

size_t slab_bytes(int nvec, int ctas) { return (static_cast<size_t>((nvec + ctas - 1) / ctas) + 2) * 16; }

// Threads and CTAs per row that keep it in shared memory; ctas 0 where it does not fit.
struct Resident {
  int threads, ctas;
};
// Measured on a GB300, loss and gradient in bf16: slabs of 64 KB, three blocks a SM, 32768
// columns 162 us for 8192 rows (98% of the copy rate); the same row over two blocks of a cluster
// 208 us, so a row stays in one block up to 112 KB (50257 columns 281 us in one, 302 in two) where
// rows are many; beyond, clusters of 76 KB slabs (131072 columns 777 us in four, 822 in eight).
// Eight vectors a thread: 8000 columns 47 us with 128 threads, 62 with 256.
Resident resident_for(int64_t rows, int nvec) {
  Resident r{256, 1};
  if (rows < 2048 || slab_bytes(nvec, 1) > kSlabAlone)
    while (r.ctas < kMaxCluster && slab_bytes(nvec, r.ctas) > kSlabBytes) r.ctas *= 2;
  if (slab_bytes(nvec, r.ctas) > kSlabMost) return Resident{0, 0};
  while (r.threads > 64 && nvec < r.threads * 8) r.threads /= 2;
  while (r.ctas < kMaxCluster && rows * r.ctas * r.threads < 1024 * 152 && nvec >= r.ctas * 4 * r.threads) r.ctas *= 2;
  return r;
}

template <typename T>
int vectors_of(int vocab) {
  return (vocab + 2 * Elem<T>::kVec - 2) / Elem<T>::kVec;  // at any alignment
}

template <typename... K, typename... A>
cudaError_t launch_clusters(void (*kernel)(K...), int threads, int64_t grid, int ctas, size_t smem, cudaStream_t stream, A... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (ctas > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<K>(args)...);
}

// Vectors per lane of a warp per row, 0 where rows are too long for that.  Measured on a GB300
// against blocks of 64 to 256 threads per row, 16384 rows: 259 columns bf16, distillation's loss
// and gradient 23 us for 60, log probabilities 10 for 24; 2000 columns 45 for 64 and 14 for 30; for
// 8 rows the two are alike.
int short_for(int nvec) {
  if (nvec > 32 * 8) return 0;
  return nvec <= 64 ? 2 : nvec <= 128 ? 4 : 8;
}

template <typename T, typename Args, bool ENT, int MODE>
cudaError_t launch_short(int n, const Args& a, int* status, cudaStream_t stream) {
  auto* kernel = n == 2 ? k_short<T, Args, ENT, MODE, 2> : n == 4 ? k_short<T, Args, ENT, MODE, 4> : k_short<T, Args, ENT, MODE, 8>;
  const int64_t blocks = std::min<int64_t>((a.v.rows + kShortWarps - 1) / kShortWarps, 1 << 16);
  return launch_clusters(kernel, 32 * kShortWarps, blocks, 1, 0, stream, a, status);
}

template <typename T>
cudaError_t launch_logprobs_t(const LogprobArgs& a, int* status, cudaStream_t stream) {
  const int nvec = vectors_of<T>(a.v.vocab), n = short_for(nvec);
  if (n > 0) {
    const bool ent = a.d_entropy || a.entropy;
    if (a.in_lse)
      return ent ? launch_short<T, LogprobArgs, true, kShortBackward>(n, a, status, stream)
                 : launch_short<T, LogprobArgs, false, kShortBackward>(n, a, status, stream);
    if (a.v.d_logits)
      return ent ? launch_short<T, LogprobArgs, true, kShortBoth>(n, a, status, stream)
                 : launch_short<T, LogprobArgs, false, kShortBoth>(n, a, status, stream);
    if (a.k > 0)
      return ent ? launch_short<T, LogprobArgs, true, kShortTop>(n, a, status, stream)
                 : launch_short<T, LogprobArgs, false, kShortTop>(n, a, status, stream);
    return ent ? launch_short<T, LogprobArgs, true, kShortForward>(n, a, status, stream)
               : launch_short<T, LogprobArgs, false, kShortForward>(n, a, status, stream);
  }
  if (a.in_lse) {
    const int threads = backward_threads(nvec), pieces = pieces_for(a.v.rows, nvec, 4 * threads, threads);
    auto* kernel = threads == 64 ? (a.d_entropy ? k_logprobs_backward<T, true, 64> : k_logprobs_backward<T, false, 64>)
                                 : (a.d_entropy ? k_logprobs_backward<T, true, 256> : k_logprobs_backward<T, false, 256>);
    return launch_clusters(kernel, threads, std::min<int64_t>(a.v.rows * pieces, 1 << 30), 1, 0, stream, a, pieces, status);
  }
  if (a.v.d_logits) {
    const Resident r = resident_for(a.v.rows, nvec);
    if (r.ctas) {
      const bool ent = a.d_entropy || a.entropy;
      auto* kernel = r.threads == 64    ? (ent ? k_logprobs_resident<T, true, 64> : k_logprobs_resident<T, false, 64>)
                     : r.threads == 128 ? (ent ? k_logprobs_resident<T, true, 128> : k_logprobs_resident<T, false, 128>)
                                        : (ent ? k_logprobs_resident<T, true, 256> : k_logprobs_resident<T, false, 256>);
      return launch_clusters(kernel, r.threads, a.v.rows * r.ctas, r.ctas, slab_bytes(nvec, r.ctas), stream, a, status);
    }
  }
  const int threads = a.v.d_logits || a.k > 0 ? 256 : forward_threads(nvec);
  const int ctas = cluster_for(a.v.rows, nvec, threads);
  const int64_t grid = a.v.rows * ctas;
  if (a.v.d_logits)
    return launch_clusters(a.d_entropy || a.entropy ? k_logprobs<T, true, false, true, 256> : k_logprobs<T, false, false, true, 256>,
                           threads, grid, ctas, 0, stream, a, 0, status);
  if (a.k == 0) {
    auto* kernel = threads == 64 ? (a.entropy ? k_logprobs<T, true, false, false, 64> : k_logprobs<T, false, false, false, 64>)
                                 : (a.entropy ? k_logprobs<T, true, false, false, 128> : k_logprobs<T, false, false, false, 128>);
    return launch_clusters(kernel, threads, grid, ctas, 0, stream, a, 0, status);
  }
  const int batches = ((nvec + ctas - 1) / ctas + 4 * kTopThreads - 1) / (4 * kTopThreads);
  int shift = 0;
  while (((batches + (1 << shift) - 1) >> shift) > kTopGroups) ++shift;
  const size_t smem = (ctas > 1 ? size_t(ctas) * a.k * 8 : 0) +
                      size_t((batches + (1 << shift) - 1) >> shift) * kTopThreads * sizeof(typename TopGroups<T>::Key);
  return launch_clusters(a.entropy ? k_logprobs<T, true, true, false, kTopThreads> : k_logprobs<T, false, true, false, kTopThreads>, threads, grid, ctas,
                         smem, stream, a, shift, status);
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs& a, int* status, cudaStream_t stream) {
  const int nvec = vectors_of<T>(a.v.vocab);
  if (const int n = short_for(nvec)) {
    if (a.in_lse) return launch_short<T, DistillArgs, false, kShortBackward>(n, a, status, stream);
    if (a.v.d_logits) return launch_short<T, DistillArgs, false, kShortBoth>(n, a, status, stream);
    return launch_short<T, DistillArgs, false, kShortForward>(n, a, status, stream);
  }
  if (a.in_lse) {
    const int threads = backward_threads(nvec), pieces = pieces_for(a.v.rows, nvec, 16 * threads, threads);
    auto* kernel = threads == 64 ? k_distill_backward<T, 64> : k_distill_backward<T, 256>;
    return launch_clusters(kernel, threads + 32, std::min<int64_t>(a.v.rows * pieces, 1 << 30), 1, 0, stream, a, pieces, status);
  }
  if (a.v.d_logits) {
    const Resident r = resident_for(a.v.rows, nvec);
    if (r.ctas) {
      auto* kernel = r.threads == 64    ? k_distill_resident<T, 64>
                     : r.threads == 128 ? k_distill_resident<T, 128>
                                        : k_distill_resident<T, 256>;
      return launch_clusters(kernel, r.threads + 32, a.v.rows * r.ctas, r.ctas, slab_bytes(nvec, r.ctas), stream, a, status);
    }
  }
  const int threads = a.v.d_logits ? 256 : forward_threads(nvec);
  int ctas = cluster_for(a.v.rows, nvec, threads);
  auto members = [&] { return (static_cast<size_t>((nvec + ctas - 1) / ctas) + 2 + 15) / 16 * 16; };
  while (members() > kMembersMost && ctas < kMaxCluster) ctas *= 2;
  auto* kernel = a.v.d_logits ? k_distill<T, true, 256> : threads == 64 ? k_distill<T, false, 64> : k_distill<T, false, 128>;
  return launch_clusters(kernel, threads + 32, a.v.rows * ctas, ctas, members(), stream, a, status);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  if (a.v.dtype == NSM_BF16) return launch_logprobs_t<__nv_bfloat16>(a, status, stream);
  if (a.v.dtype == NSM_FP16) return launch_logprobs_t<__half>(a, status, stream);
  return launch_logprobs_t<float>(a, status, stream);
}

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  if (a.v.dtype == NSM_BF16) return launch_distill_t<__nv_bfloat16>(a, status, stream);
  if (a.v.dtype == NSM_FP16) return launch_distill_t<__half>(a, status, stream);
  return launch_distill_t<float>(a, status, stream);
}

}  // namespace nsm
