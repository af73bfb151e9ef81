// Distillation from a teacher's top logits, and its gradient.
//
//   loss = sum_j p_j (log p_j - log q_{i_j}) [+ p_r (log p_r - log q_r)] over the teacher's
//   entries S = {i_j} and, with the tail, the rest of the row as one bucket (q_r = sum of q
//   outside S, summed without S and not as a difference); gradient w/t times
//   q_v (1 + excess) - p_v in S and q_v (1 + excess) - p_r q_v / q_r outside, where
//   1 + excess = sum p + p_r.
//
//   k_distill            forward: as k_logprobs, S taken out by a bit per element.
//                        8192 x 131072 bf16, 64 entries and the tail 325 us (6.6 TB/s), 1024 x
//                        50257, 32 entries 22.
//   k_distill_resident   forward and backward in one pass, the row in shared memory, the
//                        teacher in a warp of its own: 8192 x 32768 bf16, 64 entries 169 us (6.4
//                        TB/s), 8192 x 131072 (four blocks a row) 704.  Bound by the latency of the
//                        entries' loads before the sums and by the cluster's slowest block.
//   k_distill_backward   pieces of rows from saved statistics: 8192 x 131072, 64 entries and the tail
//                        762 us (5.6 TB/s).
//   k_distill_short      a warp per row of at most 256 vectors: 16384 x 259, loss and gradient 25 us.
#include "vocab_rows.cuh"

namespace nsm {
namespace {

constexpr size_t kMembersMost = 160 << 10;  // of k_distill's bits per block

// ---------------------------------------------------------------- distillation

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {  // NaNs aside
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
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

// The entries as they are in memory.  Every load is on its way before the first is looked at:
// under load each takes microseconds.
struct RawEntries {
  int64_t v[kLaneEntries];
  uint32_t score[kLaneEntries];
};
__device__ __forceinline__ void load_raw(RawEntries& raw, const DistillArgs& g, int64_t r) {
  const int lane = threadIdx.x & 31;
  const int64_t at_index = r * g.ldi + lane, at_score = r * g.ldt + lane;
  int64_t* v = raw.v;
  if (g.index_wide) {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) v[u] = load_if<int64_t>(lane + 32 * u < g.k, g.index, at_index + 32 * u, -1);
  } else {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) v[u] = load_if<int32_t>(lane + 32 * u < g.k, g.index, at_index + 32 * u, -1);
  }
  if (g.teacher_dtype == NSM_FP32) {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) raw.score[u] = load_if<uint32_t>(lane + 32 * u < g.k, g.teacher, at_score + 32 * u, 0);
  } else {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) raw.score[u] = load_if<uint16_t>(lane + 32 * u < g.k, g.teacher, at_score + 32 * u, 0);
  }
}

// The entries' tokens and scores (in log_p); equal tokens are still there.
__device__ __forceinline__ void entries_of(Entries& e, const RawEntries& raw, const DistillArgs& g) {
  if (g.teacher_dtype == NSM_FP32) {
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) e.log_p[u] = __uint_as_float(raw.score[u]);
  } else {
    const bool bf16 = g.teacher_dtype == NSM_BF16;
#pragma unroll
    for (int u = 0; u < kLaneEntries; ++u) {
      const uint16_t h = static_cast<uint16_t>(raw.score[u]);
      e.log_p[u] = bf16 ? __bfloat162float(__ushort_as_bfloat16(h)) : __half2float(__ushort_as_half(h));
    }
  }
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u) {
    e.v[u] = raw.v[u] >= 0 && raw.v[u] < g.v.vocab ? static_cast<int>(raw.v[u]) : -1;
    e.x[u] = kNegInf;
  }
}
__device__ __forceinline__ void load_entries(Entries& e, const DistillArgs& g, int64_t r) {
  RawEntries raw;
  load_raw(raw, g, r);
  entries_of(e, raw, g);
}

// Asks for a later row's entries in L2, sector by sector.
__device__ __forceinline__ void prefetch_entries(const DistillArgs& g, int64_t r) {
  const int lane = threadIdx.x & 31, index_size = g.index_wide ? 8 : 4, score_size = g.teacher_dtype == NSM_FP32 ? 4 : 2;
  if (lane * 32 < g.k * index_size) ptx::prefetch_l2(static_cast<const char*>(g.index) + r * g.ldi * index_size + lane * 32);
  if (lane * 32 < g.k * score_size) ptx::prefetch_l2(static_cast<const char*>(g.teacher) + r * g.ldt * score_size + lane * 32);
}

// The student's logits at the entries' tokens, read from the row.
template <typename T>
__device__ __forceinline__ void load_logits(Entries& e, const Row<T>& row) {
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u)
    if (e.v[u] >= 0) e.x[u] = Elem<T>::to_float(row.at(e.v[u]));
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
  // where the entries have the smaller part: log (1 - q of the entries), which a difference of
  // two logs would lose
  st.rest = no_rest                   ? kNegInf
            : inside_s < 0.5f * all.s ? log1pf(-inside_s / all.s)
                                      : (outside.max - st.lse_ref) * inv_t + (logf(outside.s) - st.lse_log);
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

// The gradients at the entries, and their way into the block's part over what the pass over the
// row wrote there: the teacher's warp has the first done when that pass ends.
template <typename T>
__device__ __forceinline__ void entry_gradients(T (&grads)[kLaneEntries], const Entries& e, const Student& s, const EntryGradient& k,
                                                float inv_t) {
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u) {
    if (e.v[u] < 0) continue;
    const float log_q = ((e.x[u] - s.lse_ref) - s.lse_low) * inv_t - s.lse_log, p = e.p[u];
    float grad = 0.f;
    if (log_q != kNegInf) {
      // q - p without cancellation where they are near.  Where q is far larger, p may be a subnormal
      // number with few digits, or 0, and expm1 of the distance infinite: there the difference itself.
      const float q = expf(log_q), apart = log_q - e.log_p[u];
      grad = k.unit * ((apart < 1.f ? p * expm1f(apart) : q - p) + q * k.excess);
    }
    grads[u] = Elem<T>::from_float(grad);
  }
}
template <typename T>
__device__ __forceinline__ void store_entries(const T (&grads)[kLaneEntries], const Row<T>& row, const Row<T>& out, const Part& part,
                                              const Entries& e) {
#pragma unroll
  for (int u = 0; u < kLaneEntries; ++u)
    if (e.v[u] >= 0 && in_part(row, part, e.v[u])) out.put(e.v[u], grads[u]);
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
  FirstFour<NT, T> first;
  if (!teacher) first.load(row, part);
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
    first.use_all(row, part, [&](int i, const uint4& raw, bool) {
      const uint32_t bits = members[i - base];
      uint4 v = raw;
      if (bits) vec_mask<T>(v, bits);
      add_vec<T, false>(a, v, c);
    });
  }
  const Totals outside = row_totals<false, NT>(a, c, totals, ctas, status, NSM_KERNEL_DISTILL, 0.f);
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
    T grads[kLaneEntries];
    if (teacher) entry_gradients(grads, e, st, k, inv_t);
    __syncthreads();
    if (teacher && !k.zero) store_entries(grads, row, out, part, e);
  }
}

// Forward and backward in one pass over memory, as k_logprobs_resident.
template <typename T, int NT>
__global__ void __launch_bounds__(NT + 32) k_distill_resident(const DistillArgs g, int ahead, int* status) {
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
  RawEntries raw;
  if (teacher) load_raw(raw, g, r);
  Slab<T, NT> slab;
  slab.start(row, part, reinterpret_cast<uint4*>(dynamic), &slab_shared);  // ends with a barrier
  const float w = g.d_loss ? g.d_loss[r] : 1.f;
  if (threadIdx.x == 0 && r + ahead < g.v.rows)
    slab.prefetch(Row<T>(static_cast<T*>(const_cast<void*>(g.v.logits)) + (r + ahead) * g.v.ld, vocab, status, NSM_KERNEL_DISTILL), rank, ctas);
  Entries e;
  Sums a;
  if (teacher) {
    entries_of(e, raw, g);
    if (rank == 0 && r + ahead < g.v.rows) prefetch_entries(g, r + ahead);
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
      else elsewhere[u] = row.at(e.v[u]);
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
    }
    slab.ragged(add);
  }
  const Totals outside = row_totals<false, NT>(a, c, totals, ctas, status, NSM_KERNEL_DISTILL, 0.f);
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
  T grads[kLaneEntries];
  if (teacher) entry_gradients(grads, e, st, k, inv_t);
  __syncthreads();
  if (teacher && !k.zero) store_entries(grads, row, out, part, e);
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
    T grads[kLaneEntries];
    if (teacher) entry_gradients(grads, e, st, k, inv_t);
    __syncthreads();  // and shared_stats is free again
    if (teacher && !k.zero) store_entries(grads, row, out, part, e);
  }
}

// ---------------------------------------------------------------- short rows

template <typename T, int MODE, int N>
__global__ void __launch_bounds__(32 * kShortWarps) k_distill_short(const DistillArgs g, int* status) {
  constexpr int kVec = Elem<T>::kVec;
  __shared__ uint32_t members[kShortWarps][32 * N / 4];  // a byte per vector, a bit per element
  grid_dependency_sync();
  release_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kShortWarps + warp; r < g.v.rows;
       r += static_cast<int64_t>(gridDim.x) * kShortWarps) {
    const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_DISTILL);
    const Part part = part_of(row, 0, 1);
    ShortRow<T, N> x;
    x.load(row, part);
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
      for (int j = 0; j < (N + 3) / 4; ++j)
        if (lane + 32 * j < 32 * N / 4) members[warp][lane + 32 * j] = 0;
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
        uint4 v = x.raw[u];
        const uint32_t bits = reinterpret_cast<const uint8_t*>(members[warp])[lane + 32 * u];
        if (bits) vec_mask<T>(v, bits);
        add_vec<T, false>(a, v, c);
      }
      __syncwarp();  // members is free again
      const Totals outside = warp_totals<false>(a, c);
      st = student_of(t, outside, c, inv_t);
      write_loss(g, r, e, t, st);
      k = entry_gradient(t, outside, w, g.tail, c, inv_t);
    }
    if constexpr (MODE != kShortForward) {
      const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_DISTILL);
      __syncwarp();  // in place: every lane has read its entries' logits
      x.store(row, out, part, k.zero,
              [&](const uint4& v) { return gradient_vec<T, false>(v, k.ref, c, k.log2_s, k.scale, 0.f); });
      __syncwarp();  // the entries' own values go over what was written there
      if (!k.zero) {
        T grads[kLaneEntries];
        entry_gradients(grads, e, st, k, inv_t);
        store_entries(grads, row, out, part, e);
      }
    }
  }
}

// ---------------------------------------------------------------- launches

template <typename T, int MODE>
cudaError_t launch_distill_short(int n, const DistillArgs& a, int* status, cudaStream_t stream) {
  auto* launch = n == 2   ? Launch<k_distill_short<T, MODE, 2>>::run
                 : n == 4 ? Launch<k_distill_short<T, MODE, 4>>::run
                          : Launch<k_distill_short<T, MODE, 8>>::run;
  return launch(32 * kShortWarps, short_blocks(a.v.rows), 1, 0, 0, stream, a, status);
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs& a, int* status, cudaStream_t stream) {
  const int nvec = vectors_of<T>(a.v.vocab);
  if (const int n = short_for(nvec)) {
    if (a.in_lse) return launch_distill_short<T, kShortBackward>(n, a, status, stream);
    if (a.v.d_logits) return launch_distill_short<T, kShortBoth>(n, a, status, stream);
    return launch_distill_short<T, kShortForward>(n, a, status, stream);
  }
  if (a.in_lse) {
    const int threads = backward_threads(nvec), pieces = pieces_for(a.v.rows, nvec, 16 * threads, threads);
    auto* launch = threads == 64 ? Launch<k_distill_backward<T, 64>>::run : Launch<k_distill_backward<T, 256>>::run;
    return launch(threads + 32, std::min<int64_t>(a.v.rows * pieces, 1 << 30), 1, 0, 0, stream, a, pieces, status);
  }
  if (a.v.d_logits) {
    const Resident r = resident_for(a.v.rows, nvec, 112 << 10);
    if (r.ctas) {
      auto* launch = r.threads == 64    ? Launch<k_distill_resident<T, 64>>::run
                     : r.threads == 128 ? Launch<k_distill_resident<T, 128>>::run
                                        : Launch<k_distill_resident<T, 256>>::run;
      const size_t slab = slab_bytes(nvec, r.ctas);
      return launch(r.threads + 32, a.v.rows * r.ctas, r.ctas, slab, kSlabMost, stream, a, rows_ahead(slab, r.threads, r.ctas), status);
    }
  }
  const int threads = a.v.d_logits ? 256 : forward_threads(nvec);
  int ctas = cluster_for(a.v.rows, nvec, threads);
  auto members = [&] { return (static_cast<size_t>((nvec + ctas - 1) / ctas) + 2 + 15) / 16 * 16; };
  while (members() > kMembersMost && ctas < kMaxCluster) ctas *= 2;
  auto* launch = a.v.d_logits   ? Launch<k_distill<T, true, 256>>::run
                 : threads == 64 ? Launch<k_distill<T, false, 64>>::run
                                 : Launch<k_distill<T, false, 128>>::run;
  return launch(threads + 32, a.v.rows * ctas, ctas, members(), kMembersMost, stream, a, status);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  if (a.v.dtype == NSM_BF16) return launch_distill_t<__nv_bfloat16>(a, status, stream);
  if (a.v.dtype == NSM_FP16) return launch_distill_t<__half>(a, status, stream);
  return launch_distill_t<float>(a, status, stream);
}

}  // namespace nsm
