// What the losses over a vocabulary share: rows of logits as 16-byte vectors, sums of
// exponentials joined over warps, blocks and clusters, rows kept in shared memory or in a
// warp's registers, and the rules that choose between them.
//
// A pass over a row keeps, per thread, a sum of exponentials relative to a reference that
// moves only when a logit exceeds it by 16 binary orders; statistics and sums are fp32, a
// gradient is rounded once.  The passes are bound by memory: 2 or 4 bytes per logit read and,
// for a gradient, as many written, against some 6 instructions per logit for the sums and 6 for
// the gradient.
#pragma once

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
  // element v of the row
  __device__ __forceinline__ T at(int v) const {
    return bounds_ok(v >= 0 && v < vocab, status, kernel, 0, NSM_SITE_LOGITS) ? p[v] : Elem<T>::from_float(0.f);
  }
  __device__ __forceinline__ void put(int v, T value) const {
    if (bounds_ok(v >= 0 && v < vocab, status, kernel, 0, NSM_SITE_GRADIENT)) p[v] = value;
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
// which cost more than the step saves (8192 x 8000 bf16, loss and gradient with 256 threads a row:
// 75 us for 62).
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
// this, the sums of the first NT count; the next use of `sh` needs a barrier.  With more than
// one CTA, start_totals comes first.
// Each CTA stores its totals in the others' shared memory, counted as bytes on a barrier there:
// one way over the cluster and no wait for it.  With plain stores and a remote arrival behind
// them, which waits until they are done, loss and gradient of 8192 x 131072 bf16 took 7%
// longer, and with a message per warp in place of one per CTA 2000 x 151936 fp32 20% longer over
// eight CTAs (distillation; over four it saves 1%).
// `read` is what the thread has read of the row and still needs: it goes along, so that its load
// is over before another CTA can write a gradient there.
struct TotalsShared {
  Totals warp[kMaxWarps];
  float4 cta[kMaxCluster];
  uint64_t joined;
  int abort;
};
__device__ __forceinline__ void start_totals(TotalsShared& sh, int ctas) {
  if (ctas == 1) return;
  if (threadIdx.x == 32) {  // the first warp starts the row's copies
    const uint32_t bar = ptx::smem_u32(&sh.joined);
    ptx::mbar_init(bar, 1);
    sh.abort = 0;
    ptx::fence_mbarrier_init();
    ptx::mbar_arrive_expect_tx(bar, ctas * sizeof(float4));
  }
  __syncwarp();
  ptx::cluster_arrive();  // the wait is in row_totals: by then every CTA runs
}
template <bool ENT, int NT>
__device__ __forceinline__ Totals row_totals(const Sums& a, float c, TotalsShared& sh, int ctas, int* status, int kernel, float read) {
  const Totals w = warp_totals<ENT>(a, c);
  if ((threadIdx.x & 31) == 0 && threadIdx.x < NT) sh.warp[threadIdx.x >> 5] = w;
  if (ctas > 1) ptx::cluster_wait();
  __syncthreads();
  const Totals v = sh.warp[threadIdx.x & (NT / 32 - 1)];
  const Totals mine = group_totals<ENT, NT / 32>(v.max, v.max, v.s, v.sy, c);
  if (ctas == 1) return mine;
  const uint32_t bar = ptx::smem_u32(&sh.joined);
  if (static_cast<int>(threadIdx.x) < ctas)
    ptx::st_async_f32x4(ptx::mapa_shared(ptx::smem_u32(&sh.cta[ptx::cluster_ctarank()]), threadIdx.x), mine.max, mine.s, mine.sy, read,
                        ptx::mapa_shared(bar, threadIdx.x));
  if (!ptx::mbar_wait_bounded_cluster(bar, 0, &sh.abort, kWaitNs)) {
    record_timeout(status, kernel, NSM_ROLE_EPILOGUE, NSM_SITE_ACC_FULL);
    *static_cast<volatile int*>(&sh.abort) = 1;
  }
  const int from = threadIdx.x & (kMaxCluster - 1);
  const float4 t = from < ctas ? sh.cta[from] : make_float4(kNegInf, 0.f, 0.f, 0.f);
  return group_totals<ENT, kMaxCluster>(t.x, t.x, t.y, t.z, c);
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
    // The ragged vectors count as copies of the first chunk: two threads of the second warp load
    // them and say when they are there.
    const int ragged = threadIdx.x == 32 ? part.head : threadIdx.x == 33 ? part.tail : -1;
    uint4 ragged_vec;
    if (ragged >= 0) ragged_vec = row.load(ragged);
    if (threadIdx.x < kSlabChunks) {  // a thread per chunk
      const int q = threadIdx.x;
      const int b = min(part.end, part.begin + q * each), e = min(part.end, b + each);
      const uint32_t bar = ptx::smem_u32(&sh->full[q]);
      ptx::mbar_init(bar, 1 + (q == 0 ? (part.head >= 0) + (part.tail >= 0) : 0));
      if (q == 0) sh->abort = 0;
      ptx::fence_mbarrier_init();
      bool load = e > b;
      if (load)
        load = bounds_ok(row.whole(b) && row.whole(e - 1) && (reinterpret_cast<uintptr_t>(row.p + row.first(b)) & 15) == 0,
                         status, kernel, NSM_ROLE_PRODUCER, NSM_SITE_LOGITS);
      ptx::mbar_arrive_expect_tx(bar, load ? (e - b) * 16 : 0);
      if (load) ptx::bulk_load(ptx::smem_u32(v + (b - base)), row.p + row.first(b), (e - b) * 16, bar);
    }
    __syncthreads();  // the barriers are there
    if (ragged >= 0) {
      v[ragged - base] = ragged_vec;
      ptx::mbar_arrive(ptx::smem_u32(&sh->full[0]));
    }
  }
  // Asks for a later row's part in L2.
  __device__ __forceinline__ void prefetch(const Row<T>& later, int piece, int pieces) const {
    const Part p = part_of(later, piece, pieces);
    if (p.end > p.begin && bounds_ok(later.whole(p.begin) && later.whole(p.end - 1), status, kernel, NSM_ROLE_PRODUCER, NSM_SITE_LOGITS))
      ptx::bulk_prefetch_l2(later.p + later.first(p.begin), (p.end - p.begin) * 16);
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
  // The same for the ragged vectors, which come with the first chunk.
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

// ---------------------------------------------------------------- short rows

// A warp per row, the row in its registers: N vectors per lane at most.  Forward, forward and
// backward, or the backward pass alone; for rows so short that a block's barriers and its
// threads' own fixed work would cost more than the row.
constexpr int kShortWarps = 4;
enum ShortMode { kShortForward, kShortTop, kShortBoth, kShortBackward };  // kShortTop: forward with alternatives

template <typename T, int N>
struct ShortRow {
  uint4 raw[N];  // vector lane + 32 u of the row, -inf outside it
  __device__ __forceinline__ void load(const Row<T>& row, const Part& part) {
    const int lane = threadIdx.x & 31;
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
  }
  // value(vector), or zeros, to the lane's vectors of the gradient
  template <typename F>
  __device__ __forceinline__ void store(const Row<T>& row, const Row<T>& out, const Part& part, bool zero, F&& value) const {
    const bool same = row.lead == out.lead;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = static_cast<int>(threadIdx.x & 31) + 32 * u;
      if (i >= row.nvec) continue;
      uint4 grad = make_uint4(0, 0, 0, 0);
      if (!zero) grad = value(raw[u]);
      if (same && i >= part.begin && i < part.end) out.store_whole(i, grad);
      else out.store(row.first(i), grad);
    }
  }
};

// ---------------------------------------------------------------- launches

// CTAs per row: where there are fewer rows than the GPU takes blocks at a time, a cluster
// shares each row, down to two vectors of a thread, until 256 threads a SM are there.  Measured on
// a GB300 with 256, 512 and 160 a SM: 600 x 32000 bf16 6.8, 8.2 and 8.0 us, 300 x 131072 19.7, 21.4
// and 28.8, 64 x 50257 with 20 alternatives 8.6, 13.4 and 8.8.
inline int cluster_for(int64_t rows, int nvec, int NT) {
  int ctas = 1;
  while (ctas < kMaxCluster && rows * ctas * NT < 256 * 152 && nvec >= ctas * 4 * NT) ctas *= 2;
  return ctas;
}

// Threads per row of a forward pass, and per piece of a row of a backward pass.  Measured on a
// GB300: 16384 x 4000 bf16 forward 30 us with 64 threads, 38 with 128; 8192 x 131072 297 with 128,
// a sixth more with 512; 16384 x 2100 backward 37 us with 64 and 57 with 256, 8192 x 131072 677
// with 256.
inline int forward_threads(int nvec) { return nvec <= 1024 ? 64 : 128; }
inline int backward_threads(int nvec) { return nvec <= 1024 ? 64 : 256; }

// Pieces per row of a backward pass: `most` vectors each, less where rows are few.
inline int pieces_for(int64_t rows, int nvec, int most, int least) {
  int each = most;
  while (each > least && rows * ((nvec + each - 1) / each) < 8 * 152) each /= 2;
  return (nvec + each - 1) / each;
}

constexpr size_t kSlabBytes = 76 << 10, kSlabMost = 216 << 10;

inline size_t slab_bytes(int nvec, int ctas) { return (static_cast<size_t>((nvec + ctas - 1) / ctas) + 2) * 16; }

// A block keeps memory busy only while its own row is on the way, not in its passes.  So each
// asks for a part of a later row in L2 when it has asked for its own: of a row half as far on as
// there are rows on the GPU, whose block starts about when the copy is there.  Measured on a
// GB300, loss and gradient of 8192 x 131072 bf16: 645 us without, 627 at half as far (and at a
// quarter), 803 as far as the rows on the GPU, 879 at twice that; 2000 x 151936 fp32 346 without and
// with, 390 and 496 further on.  The passes that only read, or read and write in pieces, were much
// slower with it: 8192 x 131072 with 64 alternatives by half, distillation's backward pass by 45%.
inline int rows_ahead(size_t slab, int threads, int ctas) {
  const int blocks = static_cast<int>(std::min<size_t>((227 << 10) / (slab + 2048), 2048 / threads));
  return std::max(1, 152 * blocks / 2 / ctas);
}

// Threads and CTAs per row that keep it in shared memory; ctas 0 where it does not fit.
struct Resident {
  int threads, ctas;
};
// Measured on a GB300, loss and gradient in bf16: slabs of 64 KB, three blocks a SM, 8192 x 32768
// 158 us (the rate of a copy), the same row over two blocks of a cluster 170.  Beyond 76 KB a row is
// shared by a cluster, with 56 KB as the limit 8192 x 131072 takes 680 us for 627; `alone`, the
// most that a row keeps in one block where rows are many, is 76 KB as well for log probabilities
// (8192 x 50257 244 us over two blocks, 266 in one of 112 KB) and 112 KB for distillation, whose
// blocks each wait for the row's entries (287 us over two, 281 in one).
// Eight vectors a thread: 8000 columns 44 us with 128 threads, 62 with 256.
// Where rows are few, clusters grow until 1024 threads a SM are there: 257 x 32003 fp32 16.4 us,
// 17.5 with half or twice as many.
inline Resident resident_for(int64_t rows, int nvec, size_t alone) {
  Resident r{256, 1};
  if (rows < 2048 || slab_bytes(nvec, 1) > alone)
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

// A kernel's launches: clusters of `ctas` blocks with `smem` bytes of dynamic shared memory each, of
// which no launch of that kernel asks for more than `most`.
template <auto KERNEL>
struct Launch;
template <typename... K, void (*KERNEL)(K...)>
struct Launch<KERNEL> {
  static cudaError_t run(int threads, int64_t grid, int ctas, size_t smem, size_t most, cudaStream_t stream, K... args) {
    if (most > 0) {
      static std::atomic<uint64_t> done{0};
      const cudaError_t e = set_smem_once(KERNEL, most, done);
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
    return cudaLaunchKernelEx(&cfg, KERNEL, args...);
  }
};

// Vectors per lane of a warp per row, 0 where rows are too long for that.  Measured on a GB300
// against blocks of 64 to 256 threads per row, 16384 rows: 259 columns bf16, distillation's loss
// and gradient 25 us for 57, log probabilities 10 for 17; 2000 columns 44 for 62 and 15 for 22; for
// 8 rows the two are alike.
inline int short_for(int nvec) {
  if (nvec > 32 * 8) return 0;
  return nvec <= 64 ? 2 : nvec <= 128 ? 4 : 8;
}

inline int64_t short_blocks(int64_t rows) { return std::min<int64_t>((rows + kShortWarps - 1) / kShortWarps, 1 << 16); }

}  // namespace
}  // namespace nsm
