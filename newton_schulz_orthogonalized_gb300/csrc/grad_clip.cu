// The norm of many gradients together, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out = g min(1, max_norm / norm)
//
//   k_grad_chunks  a block per chunk of kGradChunk elements: its sum of squares, as a 64-bit
//                  number.  The sum is taken in fp32; where that overflows, or is so small
//                  that squares were lost below fp32's range, the chunk is read again (from L2) and
//                  its elements are scaled by a power of two first.
//   k_grad_sums    a block per tensor adds its chunks' sums and writes the tensor's norm.
//   k_grad_total   one block adds the tensors' sums.
//   k_grad_clip    every block adds the tensors' sums for itself, in the same order, and scales
//                  chunks, the last ones first: those are what L2 still holds.
// The table of tensors travels as the kernel's argument, so nothing is copied to the device and a
// captured call keeps its own.  All sums run in a fixed order.
#include "elem.cuh"
#include "launch.cuh"
#include "nsm_internal.h"

#include <algorithm>

namespace nsm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kFltMax = 3.40282347e38f;
// Below this a chunk's sum may lack squares that fp32 cannot hold: 2^14 of them at most, each
// under 2^-126, are less than 2^-32 of it.
constexpr float kLeastSum = 0x1p-80f;

template <int kMost>
struct Table {
  GradTensor t[kMost];
  int n;
};

// The tensor that chunk c belongs to.
template <int kMost>
__device__ __forceinline__ const GradTensor& tensor_of(const Table<kMost>& table, int c) {
  int low = 0, high = table.n - 1;
  while (low < high) {
    const int mid = (low + high + 1) >> 1;
    if (table.t[mid].chunk_begin <= c) low = mid; else high = mid - 1;
  }
  return table.t[low];
}

constexpr int kAhead = 4;  // vectors of eight under way per thread

// Every element of a chunk once: whole vectors of eight on the 16-byte grid, several under way
// together, and what lies beside them one by one.
template <typename T, typename F8, typename F1>
__device__ __forceinline__ void for_chunk(const T* p, int n, int* status, F8 eight, F1 one) {
  const int head = min((16 / static_cast<int>(sizeof(T)) - lead_of(p)) % (16 / static_cast<int>(sizeof(T))), n);
  const int vecs = (n - head) / 8;
  for (int i0 = threadIdx.x; i0 < vecs; i0 += kAhead * kThreads) {
    Eight<T> r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = head + (i0 + k * kThreads) * 8;
      if (i0 + k * kThreads < vecs && bounds_ok(i >= 0 && i + 8 <= n && on_16_bytes(p + i), status, NSM_KERNEL_GRADS, 0, NSM_SITE_GRADS))
        r[k].load_written(p + i);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i0 + k * kThreads < vecs) eight(r[k]);
  }
  if (static_cast<int>(threadIdx.x) < head) one(p[threadIdx.x]);
  const int rest = head + vecs * 8 + threadIdx.x;
  if (rest < n) one(p[rest]);
}

__device__ __forceinline__ float block_sum(float v, float* shared) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // what the call before left there has been read
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x / 32] = v;
  __syncthreads();
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += shared[w];
  return sum;
}
__device__ __forceinline__ double block_sum(double v, double* shared) {
#pragma unroll
  for (int o = 16; o; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x / 32] = v;
  __syncthreads();
  double sum = 0.;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += shared[w];
  return sum;
}
__device__ __forceinline__ float block_max(float v, float* shared) {  // NaN if any is
#pragma unroll
  for (int o = 16; o; o /= 2) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = v != v || w != w ? v + w : fmaxf(v, w);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x / 32] = v;
  __syncthreads();
  float most = shared[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) most = most != most || shared[w] != shared[w] ? most + shared[w] : fmaxf(most, shared[w]);
  return most;
}

template <typename T>
__device__ double chunk_sum(const T* p, int n, int* status) {
  __shared__ float shared[kWarps];
  const auto sum_scaled = [&](float scale) {
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for_chunk(
        p, n, status,
        [&](const Eight<T>& r) {
          float f[8];
          r.get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = fmaf(f[e] * scale, f[e] * scale, s[e]);
        },
        [&](T v) {
          const float f = Elem<T>::to_float(v) * scale;
          s[0] = fmaf(f, f, s[0]);
        });
    return block_sum(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])), shared);
  };
  const float sum = sum_scaled(1.f);
  if (sum >= kLeastSum && sum <= kFltMax) return sum;
  float most = 0.f;
  const auto take = [&](float f) { most = f != f || most != most ? most + f : fmaxf(most, fabsf(f)); };
  for_chunk(
      p, n, status,
      [&](const Eight<T>& r) {
        float f[8];
        r.get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) take(f[e]);
      },
      [&](T v) { take(Elem<T>::to_float(v)); });
  most = block_max(most, shared);
  if (!(most > 0.f) || most > kFltMax) return most;  // nothing but zeros; an infinity or NaN
  // the largest element to [1, 2) (a subnormal one no further than fp32's exponents reach)
  int k = 127 - static_cast<int>(__float_as_uint(most) >> 23);
  if (k > 126) k = 126;
  const float scale = k >= -126 ? __uint_as_float(static_cast<uint32_t>(k + 127) << 23) : 0x1p-127f;
  const double back = 1.0 / scale;
  return static_cast<double>(sum_scaled(scale)) * back * back;
}

template <int kMost>
__global__ void __launch_bounds__(kThreads)
    k_grad_chunks(const __grid_constant__ Table<kMost> table, double* partials, int* status) {
  grid_dependency_sync();
  release_dependents();
  const GradTensor& t = tensor_of(table, blockIdx.x);
  const int64_t first = int64_t(static_cast<int>(blockIdx.x) - t.chunk_begin) * kGradChunk;
  const int n = static_cast<int>(min(t.numel - first, int64_t(kGradChunk)));
  double sum;
  if (t.in_dtype == NSM_BF16) sum = chunk_sum(static_cast<const __nv_bfloat16*>(t.in) + first, n, status);
  else if (t.in_dtype == NSM_FP16) sum = chunk_sum(static_cast<const __half*>(t.in) + first, n, status);
  else sum = chunk_sum(static_cast<const float*>(t.in) + first, n, status);
  if (threadIdx.x == 0) partials[blockIdx.x] = sum;
}

template <int kMost>
__global__ void __launch_bounds__(kThreads)
    k_grad_sums(const __grid_constant__ Table<kMost> table, int total_chunks, const double* partials, double* sums, float* norms) {
  __shared__ double shared[kWarps];
  grid_dependency_sync();
  release_dependents();
  const int i = blockIdx.x;
  const int end = i + 1 < table.n ? table.t[i + 1].chunk_begin : total_chunks;
  double sum = 0.;
  for (int c = table.t[i].chunk_begin + threadIdx.x; c < end; c += kThreads) sum += partials[c];
  sum = block_sum(sum, shared);
  if (threadIdx.x == 0) {
    sums[i] = sum;
    if (norms) norms[i] = static_cast<float>(sqrt(sum));
  }
}

__device__ __forceinline__ double all_sum(const double* sums, int n, double* shared) {
  double sum = 0.;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += sums[i];
  return block_sum(sum, shared);
}

__global__ void __launch_bounds__(kThreads) k_grad_total(const double* sums, int n, float* norm) {
  __shared__ double shared[kWarps];
  grid_dependency_sync();
  release_dependents();
  const double sum = all_sum(sums, n, shared);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

// A chunk's elements, in units of eight on the 16-byte grid of where they go.  Around it the tensor
// goes on for `before` and `after` elements.
template <typename T, typename O>
__device__ void scale_chunk(const T* p, O* out, int n, int before, int after, float factor, float more, int* status) {
  const int lead = lead_of(out), units = (n + lead + 7) / 8;
  for (int u0 = threadIdx.x; u0 < units; u0 += kAhead * kThreads) {
    Eight<T> r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int u = u0 + k * kThreads;
      if (u < units) load8(p, -before, n + after, u * 8 - lead, r[k], status, NSM_KERNEL_GRADS, NSM_SITE_GRADS);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int u = u0 + k * kThreads;
      if (u >= units) break;
      float f[8];
      r[k].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] * factor * more;
      store8(out, 0, n, u * 8 - lead, f, status, NSM_KERNEL_GRADS, NSM_SITE_GRADS);
    }
  }
}

template <typename T>
__device__ __forceinline__ void scale_chunk_to(const GradTensor& t, int64_t first, int n, float factor, float more, int* status) {
  const T* p = static_cast<const T*>(t.in) + first;
  const int before = static_cast<int>(min(first, int64_t(8))), after = static_cast<int>(min(t.numel - first - n, int64_t(8)));
  if (t.out_dtype == NSM_BF16) scale_chunk(p, static_cast<__nv_bfloat16*>(t.out) + first, n, before, after, factor, more, status);
  else if (t.out_dtype == NSM_FP16) scale_chunk(p, static_cast<__half*>(t.out) + first, n, before, after, factor, more, status);
  else scale_chunk(p, static_cast<float*>(t.out) + first, n, before, after, factor, more, status);
}

template <int kMost>
__global__ void __launch_bounds__(kThreads)
    k_grad_clip(const __grid_constant__ Table<kMost> table, int total_chunks, const double* sums, int n_sums, float max_norm,
                float* norm, int in_place, int* status) {
  __shared__ double shared[kWarps];
  grid_dependency_sync();
  release_dependents();
  const double total = sqrt(all_sum(sums, n_sums, shared));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  // a norm that is no number leaves the gradients as they are
  const bool clip = total > max_norm && total < __longlong_as_double(0x7ff0000000000000ll);
  if (!clip && in_place) return;
  // a factor below fp32's normal range is applied in two steps
  const double factor = clip ? max_norm / total : 1.;
  const bool tiny = factor < 0x1p-60;
  const float first_factor = static_cast<float>(tiny ? factor * 0x1p60 : factor), more = tiny ? 0x1p-60f : 1.f;
  for (int c = total_chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const GradTensor& t = tensor_of(table, c);
    const int64_t first = int64_t(c - t.chunk_begin) * kGradChunk;
    const int n = static_cast<int>(min(t.numel - first, int64_t(kGradChunk)));
    if (t.in_dtype == NSM_BF16) scale_chunk_to<__nv_bfloat16>(t, first, n, first_factor, more, status);
    else if (t.in_dtype == NSM_FP16) scale_chunk_to<__half>(t, first, n, first_factor, more, status);
    else scale_chunk_to<float>(t, first, n, first_factor, more, status);
  }
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

cudaError_t launch_grad_chunks(const GradTensor* tensors, int n, int total_chunks, double* partials, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  return with_table(tensors, n, [&](const auto& t) {
    return launch_pdl(k_grad_chunks<sizeof(t.t) / sizeof(t.t[0])>, dim3(total_chunks), dim3(kThreads), 0, stream, t, partials, status);
  });
}

cudaError_t launch_grad_sums(const GradTensor* tensors, int n, int total_chunks, const double* partials, double* sums,
                             float* norms, cudaStream_t stream) {
  return with_table(tensors, n, [&](const auto& t) {
    return launch_pdl(k_grad_sums<sizeof(t.t) / sizeof(t.t[0])>, dim3(n), dim3(kThreads), 0, stream, t, total_chunks, partials, sums, norms);
  });
}

cudaError_t launch_grad_total(const double* sums, int n, float* norm, cudaStream_t stream) {
  return launch_pdl(k_grad_total, dim3(1), dim3(kThreads), 0, stream, sums, n, norm);
}

cudaError_t launch_grad_clip(const GradTensor* tensors, int n, int total_chunks, const double* all_sums, int all_n,
                             float max_norm, float* norm, int in_place, int num_sms, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  return with_table(tensors, n, [&](const auto& t) {
    return launch_pdl(k_grad_clip<sizeof(t.t) / sizeof(t.t[0])>, dim3(std::min(total_chunks, 8 * num_sms)), dim3(kThreads), 0,
                      stream, t, total_chunks, all_sums, all_n, max_norm, norm, in_place, status);
  });
}

}  // namespace nsm
