// The norm of many gradients together, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out = g min(1, max_norm / norm)
//
//   k_grad_squares  every block takes a run of chunks of kGradChunk elements: of each tensor that it
//                   meets the sum of squares, and of all of them.  A thread adds a chunk's
//                   squares in fp32, and its chunks in two numbers of fp32.
//   k_grad_exact    where fp32 overflows, or a sum is so small that squares were lost below its
//                   range, takes the tensor's chunks again in 64 bits.
//   k_grad_small    for few chunks, all of it by one cluster of blocks.
//   k_grad_norms    one block adds the blocks' sums, and the parts of each tensor.
//   k_grad_clip     every block adds the blocks' sums for itself, in the same order, and scales a run
//                   of chunks, the last ones first: those are what L2 still holds of it.
// The table of tensors travels as the kernel's argument, so nothing is copied to the device and a
// captured call keeps its own.  All sums run in a fixed order.
//
// Bound by memory: the norm of 1.4G fp32 gradients takes 772 us (7.3 TB/s), clipping them into bf16 slots
// 1240 more (6.8 TB/s read and written); 147 tensors of 163M bf16 elements take 58 and 166 us together.
#include "elem.cuh"
#include "launch.cuh"
#include "nsm_internal.h"
#include "ptx.cuh"

#include <algorithm>
#include <type_traits>

namespace nsm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 4;  // resident on an SM
constexpr int kClipBlocks = 8;  // of k_grad_clip; 6 took 5% longer
constexpr int kSmallBlocks = 8, kSmallThreads = 512, kSmallWarps = kSmallThreads / 32;  // of k_grad_small's cluster
// A thread's sum of a chunk's squares is taken as it is between these.  Below, it may lack squares that
// fp32 cannot hold: 2^7 of them at most, each under 2^-126, are less than 2^-38 of the least one.
// Above, sums of some more of them would leave fp32's range.
constexpr float kLeastSum = 0x1p-80f, kMostSum = 0x1p100f;

template <int kMost>
struct Table {
  GradTensor t[kMost];
  int n;
};

// The tensor that chunk c belongs to.
template <int kMost>
__device__ __forceinline__ int index_of(const Table<kMost>& table, int c) {
  int low = 0, high = table.n - 1;
  while (low < high) {
    const int mid = (low + high + 1) >> 1;
    if (table.t[mid].chunk_begin <= c) low = mid; else high = mid - 1;
  }
  return low;
}

// Block b of `blocks` takes the chunks from here to the next one's.
__device__ __forceinline__ int first_chunk(int b, int blocks, int chunks) { return static_cast<int>(int64_t(b) * chunks / blocks); }
// The block that takes chunk c.
__device__ __forceinline__ int block_of(int c, int blocks, int chunks) {
  return static_cast<int>((int64_t(c + 1) * blocks + chunks - 1) / chunks) - 1;
}

// Vectors of eight under way per thread: 64 bytes of either size of type.
template <typename T>
constexpr int kAhead = 8 / sizeof(T);

// Every element of a chunk once: whole vectors of eight on the 16-byte grid, several under way
// together, and what lies beside them one by one.
template <int NT, typename T, typename F8, typename F1>
__device__ __forceinline__ void for_chunk(const T* p, int n, int* status, F8 eight, F1 one) {
  constexpr int kPer = 16 / sizeof(T);
  const int head = min((kPer - lead_of(p)) % kPer, n);
  const int vecs = (n - head) / 8;
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kAhead<T> * NT) {
    Eight<T> r[kAhead<T>];
#pragma unroll
    for (int k = 0; k < kAhead<T>; ++k) {
      const int i = head + (i0 + k * NT) * 8;
      if (i0 + k * NT < vecs && bounds_ok(i >= 0 && i + 8 <= n && on_16_bytes(p + i), status, NSM_KERNEL_GRADS, 0, NSM_SITE_GRADS))
        r[k].load_written(p + i);
    }
#pragma unroll
    for (int k = 0; k < kAhead<T>; ++k)
      if (i0 + k * NT < vecs) eight(r[k]);
  }
  if (static_cast<int>(threadIdx.x) < head) one(p[threadIdx.x]);
  const int rest = head + vecs * 8 + threadIdx.x;
  if (rest < n) one(p[rest]);
}

// A warp's sum.  64-bit additions take this GPU 16 cycles a warp, and all of an SM's warps in turn: a
// block leaves them to one warp.
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// sqrt(sum) = m 2^k with m in [1, 2), or sum itself in m where it is zero or no number: the root in
// fp32, the range that of 64 bits.
struct Root {
  float m;
  int k;
  bool finite;
  __device__ __forceinline__ explicit Root(double sum) : m(static_cast<float>(sum)), k(0), finite(sum <= 1.7976931348623157e308) {
    if (!(sum > 0.) || !finite) return;
    const int64_t bits = __double_as_longlong(sum);
    const int e = static_cast<int>(bits >> 52) - 1023;  // sums of squares are normal numbers
    k = e >> 1;
    m = sqrtf(static_cast<float>(__longlong_as_double((bits & 0xfffffffffffffll) | int64_t(1023 + (e & 1)) << 52)));
  }
  __device__ __forceinline__ float value() const { return scalbnf(m, k); }
};

// The thread's part of a chunk's squares in fp32; -1 where that does not hold it.
template <int NT, typename T>
__device__ __forceinline__ float squares(const T* p, int n, int* status) {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  uint32_t bits = 0;  // of all elements: none but signs where they are zeros
  for_chunk<NT>(
      p, n, status,
      [&](const Eight<T>& r) {
        float f[8];
        r.get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = fmaf(f[e], f[e], s[e]);
#pragma unroll
        for (int i = 0; i < Eight<T>::kWords; ++i) bits |= r.w[i].x | r.w[i].y | r.w[i].z | r.w[i].w;
      },
      [&](T v) {
        const float f = Elem<T>::to_float(v);
        s[0] = fmaf(f, f, s[0]);
        if (f != 0.f) bits |= 1;
      });
  const float sum = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  const bool zeros = (bits & (sizeof(T) == 2 ? 0x7fff7fffu : 0x7fffffffu)) == 0;
  return (sum >= kLeastSum && sum <= kMostSum) || zeros ? sum : -1.f;
}

__device__ __forceinline__ int chunk_of(const GradTensor& t, int c, int64_t* first) {
  *first = int64_t(c - t.chunk_begin) * kGradChunk;
  return static_cast<int>(min(t.numel - *first, int64_t(kGradChunk)));
}

template <int NT>
struct BlockSum {
  float2 part[NT / 32];
  double result;
};

// A block's sum over many chunks of a tensor: two fp32 numbers a thread, what the addition to the first one
// loses going to the second.
template <int NT>
struct Sum {
  float high = 0.f, low = 0.f;
  bool lost = false;  // fp32 did not hold some chunk's
  template <typename T>
  __device__ __forceinline__ void add(const T* p, int n, int* status) {
    const float s = squares<NT>(p, n, status);
    lost |= s < 0.f;
    const float t = high + s, back = t - high;
    low += (high - (t - back)) + (s - back);
    high = t;
  }
  template <typename T>
  __device__ __forceinline__ void add_chunks(const GradTensor& t, int begin, int end, int* status) {
#pragma unroll 1
    for (int c = begin; c < end; ++c) {
      int64_t first;
      const int n = chunk_of(t, c, &first);
      add(static_cast<const T*>(t.in) + first, n, status);
    }
  }
};

// The same in 64 bits, for tensors that fp32 does not hold.
template <int NT, typename T>
__device__ __forceinline__ double add_exactly(const GradTensor& t, int begin, int end, int* status) {
  double sum = 0.;
  const auto add = [&](float f) {
    if (f != 0.f) sum += static_cast<double>(f) * f;
  };
#pragma unroll 1
  for (int c = begin; c < end; ++c) {
    int64_t first;
    const int n = chunk_of(t, c, &first);
    for_chunk<NT>(
        static_cast<const T*>(t.in) + first, n, status,
        [&](const Eight<T>& r) {
          float f[8];
          r.get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) add(f[e]);
        },
        [&](T v) { add(Elem<T>::to_float(v)); });
  }
  return sum;
}
template <int NT>
__device__ __forceinline__ double squares_exactly(const GradTensor& t, int begin, int end, int* status) {
  __shared__ double shared[NT];
  shared[threadIdx.x] = t.in_dtype == NSM_BF16   ? add_exactly<NT, __nv_bfloat16>(t, begin, end, status)
                        : t.in_dtype == NSM_FP16 ? add_exactly<NT, __half>(t, begin, end, status)
                                                 : add_exactly<NT, float>(t, begin, end, status);
  __syncthreads();
  double sum = 0.;
  for (int i = threadIdx.x & 31; i < NT; i += 32) sum += shared[i];
  __syncthreads();
  return warp_sum(sum);
}

// The squares of a tensor's chunks, by every thread of a block; -1 where fp32 does not hold some.  T: the
// type of all of a launch's tensors, or void where they are of several.
template <int NT, typename T>
__device__ __forceinline__ double squares_of(const GradTensor& t, int begin, int end, BlockSum<NT>& block, int* status) {
  Sum<NT> sum;
  if constexpr (!std::is_same<T, void>::value) sum.template add_chunks<T>(t, begin, end, status);
  else if (t.in_dtype == NSM_BF16) sum.template add_chunks<__nv_bfloat16>(t, begin, end, status);
  else if (t.in_dtype == NSM_FP16) sum.template add_chunks<__half>(t, begin, end, status);
  else sum.template add_chunks<float>(t, begin, end, status);
  const int lane = threadIdx.x & 31;
  const float h = warp_sum(sum.high), l = warp_sum(sum.low);
  if (lane == 0) block.part[threadIdx.x / 32] = make_float2(h, l);
  if (__syncthreads_or(sum.lost)) return -1.;
  if (threadIdx.x < 32) {
    double all = 0.;
    if (lane < NT / 32) all = static_cast<double>(block.part[lane].x) + block.part[lane].y;
    all = warp_sum(all);
    if (lane == 0) block.result = all;
  }
  __syncthreads();
  return block.result;
}

// totals: a sum per block.  parts[b + i]: block b's of tensor i (no two pairs that meet have the same
// place: along the chunks neither falls).
// Calls f(i, begin, end) for the chunks of each tensor that the block meets.
template <int kMost, typename F>
__device__ __forceinline__ void for_tensors(const Table<kMost>& table, int chunks, F f) {
  const int end = first_chunk(blockIdx.x + 1, gridDim.x, chunks);
  int c = first_chunk(blockIdx.x, gridDim.x, chunks);
  for (int i = index_of(table, c); c < end; ++i) {
    const int last = min(end, i + 1 < table.n ? table.t[i + 1].chunk_begin : chunks);
    if (last <= c) continue;  // an empty tensor
    f(i, c, last);
    c = last;
  }
}

// One type alone takes 57 registers a thread (fp16 59), several together 96; and the 64-bit sums in the same
// kernel made its loop spill (5.7 GB of fp32 3070 us for 810), so they have one of their own.
template <int kMost, typename T>
__global__ void __launch_bounds__(kThreads, std::is_same<T, void>::value ? 2 : kBlocks)
    k_grad_squares(const __grid_constant__ Table<kMost> table, int chunks, double* totals, double* parts, int* status) {
  __shared__ BlockSum<kThreads> block;
  grid_dependency_sync();
  release_dependents();
  double total = 0.;
  for_tensors(table, chunks, [&](int i, int begin, int end) {
    const double sum = squares_of<kThreads, T>(table.t[i], begin, end, block, status);
    if (threadIdx.x == 0) {
      parts[blockIdx.x + i] = sum;
      total = sum < 0. || total < 0. ? -1. : total + sum;
    }
  });
  if (threadIdx.x == 0) totals[blockIdx.x] = total;
}

// The sums that k_grad_squares left at -1.
template <int kMost>
__global__ void __launch_bounds__(kThreads)
    k_grad_exact(const __grid_constant__ Table<kMost> table, int chunks, double* totals, double* parts, int* status) {
  grid_dependency_sync();
  release_dependents();
  if (!(totals[blockIdx.x] < 0.)) return;
  double total = 0.;
  for_tensors(table, chunks, [&](int i, int begin, int end) {
    double sum = parts[blockIdx.x + i];
    if (sum < 0.) sum = squares_exactly<kThreads>(table.t[i], begin, end, status);
    __syncthreads();  // every thread has read the part
    if (threadIdx.x == 0) parts[blockIdx.x + i] = sum;
    total += sum;
  });
  __syncthreads();
  if (threadIdx.x == 0) totals[blockIdx.x] = total;
}

// The sum of n numbers, by every warp that calls it.
__device__ __forceinline__ double all_sum(const double* totals, int n) {
  double sum = 0.;
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < n; i += 32) sum += totals[i];
  return warp_sum(sum);
}

// The norms of a launch's tensors from their parts, a warp per tensor: tensors `first`, first +
// step, ...
template <int kMost>
__device__ __forceinline__ void tensor_norms(const Table<kMost>& table, int chunks, int blocks, const double* parts, float* norms,
                                             int first, int step) {
  const int lane = threadIdx.x & 31;
  for (int i = first; i < table.n; i += step) {
    const int begin = table.t[i].chunk_begin, end = i + 1 < table.n ? table.t[i + 1].chunk_begin : chunks;
    double sum = 0.;
    if (begin < end) {
      const int last = block_of(end - 1, blocks, chunks);
      for (int b = block_of(begin, blocks, chunks) + lane; b <= last; b += 32) sum += parts[b + i];
    }
    sum = warp_sum(sum);
    if (lane == 0) norms[i] = Root(sum).value();
  }
}

// The norms of one launch's tensors and, with `norm`, that of all.
template <int kMost>
__global__ void __launch_bounds__(kThreads)
    k_grad_norms(const __grid_constant__ Table<kMost> table, int chunks, int blocks, const double* parts, float* norms,
                 const double* totals, int n_totals, float* norm) {
  grid_dependency_sync();
  release_dependents();
  if (norm && blockIdx.x == gridDim.x - 1 && threadIdx.x < 32) {
    const double sum = all_sum(totals, n_totals);
    if (threadIdx.x == 0) *norm = Root(sum).value();
  }
  if (norms) tensor_norms(table, chunks, blocks, parts, norms, blockIdx.x * kWarps + threadIdx.x / 32, gridDim.x * kWarps);
}

__global__ void __launch_bounds__(32) k_grad_total(const double* totals, int n, double* total) {
  grid_dependency_sync();
  release_dependents();
  const double sum = all_sum(totals, n);
  if (threadIdx.x == 0) *total = sum;
}

constexpr int kBatch = 1;  // vectors under way per thread of k_grad_clip; 2 took 2750 us where 1 takes 2012

// A chunk's elements, in units of eight on the 16-byte grid of where they go.  Around it the tensor
// goes on for `before` and `after` elements.
template <int NT, typename T, typename O>
__device__ __noinline__ void scale_chunk(const T* p, O* out, int n, int before, int after, float factor, float more, int* status) {
  if constexpr (std::is_same<T, O>::value)  // in place a factor of 1 writes nothing: the product would give NaNs other bits
    if (p == out && factor * more == 1.f) return;
  const int lead = lead_of(out), units = (n + lead + 7) / 8;
  const auto put = [&](int u, const Eight<T>& r) {
    float f[8];
    r.get(f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] * factor * more;
    store8(out, 0, n, u * 8 - lead, f, status, NSM_KERNEL_GRADS, NSM_SITE_GRADS);
  };
  const auto one = [&](int u) {
    Eight<T> r;
    load8(p, -before, n + after, u * 8 - lead, r, status, NSM_KERNEL_GRADS, NSM_SITE_GRADS);
    put(u, r);
  };
  if (lead_of(p - lead) != 0) {  // the two are not aligned alike: vectors are put together of two
#pragma unroll 1
    for (int u = threadIdx.x; u < units; u += NT) one(u);
    return;
  }
  // whole units, then the first and the last one.  Where one of the types is fp32 a thread takes half
  // a unit: 16 bytes of it, so that a warp's accesses lie side by side.
  const int low = lead ? 1 : 0, high = (n + lead) / 8;
  constexpr int kPer = sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4;
  const int from = low * 8 - lead, count = (high - low) * (8 / kPer);
#pragma unroll 1
  for (int v0 = threadIdx.x; v0 < count; v0 += kBatch * NT) {
    Side<T, kPer> r[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int v = v0 + k * NT;
      if (v < count && bounds_ok(from >= 0 && from + v * kPer + kPer <= n, status, NSM_KERNEL_GRADS, 0, NSM_SITE_GRADS))
        r[k].load(p + from + v * kPer);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int v = v0 + k * NT;
      if (v < count) {
        float f[kPer];
        r[k].get(f);
#pragma unroll
        for (int e = 0; e < kPer; ++e) f[e] = f[e] * factor * more;
        Side<O, kPer> w;
        w.set(f);
        w.store(out + from + v * kPer);
      }
    }
  }
  if (threadIdx.x == 0 && low > 0) one(0);
  if (threadIdx.x == 32 && high < units && high >= low) one(high);
}

template <int NT, typename T>
__device__ __forceinline__ void scale_chunk_to(const GradTensor& t, int64_t first, int n, float factor, float more, int* status) {
  const T* p = static_cast<const T*>(t.in) + first;
  const int before = static_cast<int>(min(first, int64_t(8))), after = static_cast<int>(min(t.numel - first - n, int64_t(8)));
  if (t.out_dtype == NSM_BF16) scale_chunk<NT>(p, static_cast<__nv_bfloat16*>(t.out) + first, n, before, after, factor, more, status);
  else if (t.out_dtype == NSM_FP16) scale_chunk<NT>(p, static_cast<__half*>(t.out) + first, n, before, after, factor, more, status);
  else scale_chunk<NT>(p, static_cast<float*>(t.out) + first, n, before, after, factor, more, status);
}

// What the gradients are multiplied by, in two steps where one is below fp32's normal range.  A norm
// that is no number leaves them as they are.
struct Factor {
  bool clip;
  float first, more;
};
__device__ __forceinline__ Factor factor_of(const Root& norm, float max_norm) {
  const bool clip = norm.finite && norm.value() > max_norm;
  if (!clip) return {false, 1.f, 1.f};
  const float f = max_norm / norm.m;  // times 2^-k, which is at most 1
  const float factor = scalbnf(f, -norm.k);
  if (factor >= 0x1p-60f) return {true, factor, 1.f};
  return {true, scalbnf(f, 60 - norm.k), 0x1p-60f};
}

template <int NT>
__device__ __forceinline__ void scale_chunk_of(const GradTensor& t, int c, const Factor& f, int* status) {
  int64_t first;
  const int n = chunk_of(t, c, &first);
  if (t.in_dtype == NSM_BF16) scale_chunk_to<NT, __nv_bfloat16>(t, first, n, f.first, f.more, status);
  else if (t.in_dtype == NSM_FP16) scale_chunk_to<NT, __half>(t, first, n, f.first, f.more, status);
  else scale_chunk_to<NT, float>(t, first, n, f.first, f.more, status);
}

template <int kMost>
__global__ void __launch_bounds__(kThreads, kClipBlocks)
    k_grad_clip(const __grid_constant__ Table<kMost> table, int chunks, int blocks, const double* parts, float* norms, const double* totals,
                int n_totals, float max_norm, float* norm, int in_place, int* status) {
  __shared__ Factor factor;
  grid_dependency_sync();
  release_dependents();
  if (norms) tensor_norms(table, chunks, blocks, parts, norms, blockIdx.x * kWarps + threadIdx.x / 32, gridDim.x * kWarps);
  if (threadIdx.x < 32) {
    const Root total(all_sum(totals, n_totals));
    if (threadIdx.x == 0) {
      factor = factor_of(total, max_norm);
      if (norm && blockIdx.x == 0) *norm = total.value();
    }
  }
  __syncthreads();
  const Factor f = factor;
  if (!f.clip && in_place) return;
  for (int c = chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= static_cast<int>(gridDim.x))
    scale_chunk_of<kThreads>(table.t[index_of(table, c)], c, f, status);
}

// Both passes over few chunks by one cluster, whose blocks send each other their chunks' sums: one
// launch.  The norms of four 128 x 256 matrices and a vector take 5.8 us, clipping them 7.7; of 25
// chunks in fp32 the kernels above clip in 11.5.
template <int kMost>
__global__ void __cluster_dims__(kSmallBlocks, 1, 1) __launch_bounds__(kSmallThreads)
    k_grad_small(const __grid_constant__ Table<kMost> table, int chunks, int clip, float max_norm, float* norm, float* norms,
                 int in_place, int* status) {
  __shared__ BlockSum<kSmallThreads> block;
  __shared__ __align__(8) double sums[kGradSmall];
  __shared__ Factor factor;
  ptx::cluster_arrive();
  const int rank = blockIdx.x, lane = threadIdx.x & 31;
  grid_dependency_sync();
  release_dependents();
  ptx::cluster_wait();  // every block of the cluster has begun
  for (int c = rank; c < chunks; c += kSmallBlocks) {
    const GradTensor& t = table.t[index_of(table, c)];
    double sum = squares_of<kSmallThreads, void>(t, c, c + 1, block, status);
    if (sum < 0.) sum = squares_exactly<kSmallThreads>(t, c, c + 1, status);
    if (threadIdx.x < kSmallBlocks)
      ptx::st_cluster_u64(ptx::mapa_shared(ptx::smem_u32(&sums[c]), threadIdx.x), static_cast<uint64_t>(__double_as_longlong(sum)));
  }
  ptx::cluster_sync();
  const auto sum_of = [&](int begin, int end) {  // of chunks, by a warp
    return warp_sum(begin + lane < end ? sums[begin + lane] : 0.);
  };
  static_assert(kGradSmall <= 32, "a lane per chunk");
  if (threadIdx.x < 32) {
    const Root total(sum_of(0, chunks));
    if (threadIdx.x == 0) {
      factor = factor_of(total, max_norm);
      if (norm && rank == 0) *norm = total.value();
    }
  }
  if (norms) {
    for (int i = rank * kSmallWarps + threadIdx.x / 32; i < table.n; i += kSmallBlocks * kSmallWarps) {
      const double s = sum_of(table.t[i].chunk_begin, i + 1 < table.n ? table.t[i + 1].chunk_begin : chunks);
      if (lane == 0) norms[i] = Root(s).value();
    }
  }
  if (!clip) return;
  __syncthreads();
  const Factor f = factor;
  if (!f.clip && in_place) return;
  for (int c = rank; c < chunks; c += kSmallBlocks) scale_chunk_of<kSmallThreads>(table.t[index_of(table, c)], c, f, status);
}

// f with the smallest of the argument's sizes that holds the table
template <typename F>
cudaError_t with_table(const GradTensor* tensors, int n, F f) {
  const auto fill = [&](auto& table) {
    std::copy(tensors, tensors + n, table.t);
    table.n = n;
    return f(table);
  };
  if (n <= 16) {
    Table<16> t{};
    return fill(t);
  }
  if (n <= 128) {
    Table<128> t{};
    return fill(t);
  }
  Table<kGradTable> t{};
  return fill(t);
}

}  // namespace

int grad_blocks(int chunks) { return std::min(chunks, kGradBlocks); }

// The kernel for the type that all tensors have, or for several, and what it leaves.
template <int kMost>
cudaError_t launch_squares(const Table<kMost>& t, int chunks, double* totals, double* parts, int* status, cudaStream_t stream) {
  bool same = true;
  for (int i = 1; i < t.n; ++i) same &= t.t[i].in_dtype == t.t[0].in_dtype;
  const int dtype = same ? t.t[0].in_dtype : -1;
  const auto kernel = dtype == NSM_BF16   ? k_grad_squares<kMost, __nv_bfloat16>
                      : dtype == NSM_FP16 ? k_grad_squares<kMost, __half>
                      : dtype == NSM_FP32 ? k_grad_squares<kMost, float>
                                          : k_grad_squares<kMost, void>;
  const cudaError_t e = launch_pdl(kernel, dim3(grad_blocks(chunks)), dim3(kThreads), 0, stream, t, chunks, totals, parts, status);
  if (e != cudaSuccess) return e;
  return launch_pdl(k_grad_exact<kMost>, dim3(grad_blocks(chunks)), dim3(kThreads), 0, stream, t, chunks, totals, parts, status);
}

cudaError_t launch_grad_squares(const GradTensor* tensors, int n, int chunks, double* totals, double* parts, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  return with_table(tensors, n, [&](const auto& t) { return launch_squares(t, chunks, totals, parts, status, stream); });
}

cudaError_t launch_grad_norms(const GradTensor* tensors, int n, int chunks, const double* parts, float* norms, const double* totals,
                              int n_totals, float* norm, cudaStream_t stream) {
  return with_table(tensors, n, [&](const auto& t) {
    return launch_pdl(k_grad_norms<sizeof(t.t) / sizeof(t.t[0])>, dim3(norms ? (n + kWarps - 1) / kWarps : 1), dim3(kThreads), 0, stream, t,
                      chunks, grad_blocks(chunks), parts, norms, totals, n_totals, norm);
  });
}

cudaError_t launch_grad_total(const double* totals, int n, double* total, cudaStream_t stream) {
  return launch_pdl(k_grad_total, dim3(1), dim3(32), 0, stream, totals, n, total);
}

cudaError_t launch_grad_clip(const GradTensor* tensors, int n, int chunks, const double* parts, float* norms, const double* totals,
                             int n_totals, float max_norm, float* norm, int in_place, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  return with_table(tensors, n, [&](const auto& t) {
    return launch_pdl(k_grad_clip<sizeof(t.t) / sizeof(t.t[0])>, dim3(std::min(chunks, kGradSms * kClipBlocks)), dim3(kThreads), 0, stream, t, chunks, grad_blocks(chunks),
                      parts, norms, totals, n_totals, max_norm, norm, in_place, status);
  });
}

cudaError_t launch_grad_small(const GradTensor* tensors, int n, int chunks, int clip, float max_norm, float* norm, float* norms,
                              int in_place, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  return with_table(tensors, n, [&](const auto& t) {
    return launch_pdl(k_grad_small<sizeof(t.t) / sizeof(t.t[0])>, dim3(kSmallBlocks), dim3(kSmallThreads), 0, stream, t, chunks, clip,
                      max_norm, norm, norms, in_place, status);
  });
}

}  // namespace nsm
