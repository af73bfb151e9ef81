// Penalties for repeated tokens, biases and grammar masks on rows of logits, and their backward
// pass.
//
//   c_v = how often token v occurs in the row's history
//   a_v = x_v / repetition (x_v > 0) or x_v repetition where c_v > 0, else x_v
//   out_v = a_v - (frequency c_v + presence [c_v > 0]) + sum of the biases at v; -inf where banned
//   d x_v = d out_v (d a_v / d x_v); 0 where banned
//
// A block takes 8192 logits of a row.  It counts the history's tokens among them in shared memory
// (whole numbers: their order does not matter), while its logits are on their way to
// registers.  Every slice of a row reads the row's history again, from L2: 4 or 8 bytes per token
// against 16 KB of logits and as many written.
#include "elem.cuh"
#include "launch.cuh"
#include "nsm_internal.h"

namespace nsm {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                        // of eight logits, per thread
constexpr int kSlice = kThreads * kUnits * 8;    // logits of a block
constexpr uint32_t kHasBias = 0x80000000u;       // in a count: some bias is for this token

struct Rows {  // of one matrix: where row r begins
  template <typename T>
  static __device__ __forceinline__ T* at(T* p, int64_t r, int64_t ld) {
    return p + r * ld;
  }
};

__device__ __forceinline__ int64_t index_at(const void* p, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

// The eight bits of a row's mask from element e0 on (bit set: allowed); what lies outside is 0.
__device__ __forceinline__ uint32_t mask_bits(const int32_t* words, int nwords, int e0, int* status) {
  const int w = e0 >> 5, bit = e0 & 31;
  const auto word = [&](int i) {
    return i >= 0 && i < nwords && bounds_ok(i < nwords, status, NSM_KERNEL_ADJUST, 0, NSM_SITE_SIDE)
               ? static_cast<uint32_t>(__ldg(words + i)) : 0u;
  };
  return __funnelshift_r(word(w), bit > 24 ? word(w + 1) : 0u, bit) & 0xffu;
}

// A: type of what is read, B: of what is written.
template <typename A, typename B, bool kBackward>
__global__ void __launch_bounds__(kThreads)
    k_adjust(const AdjustArgs a, int slices, int* status) {
  extern __shared__ __align__(16) uint32_t shared[];
  uint32_t* count = shared;                                        // kSlice
  float* bias = reinterpret_cast<float*>(shared + kSlice);         // a.k
  int32_t* bias_index = reinterpret_cast<int32_t*>(bias + a.k);    // a.k
  grid_dependency_sync();
  release_dependents();
  const int tid = threadIdx.x, vocab = a.vocab;
  const int nwords = (vocab + 31) / 32;
  const int64_t items = a.rows * slices;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t row = item / slices;
    const A* in = Rows::at(static_cast<const A*>(a.in), row, a.ld_in);
    B* out = Rows::at(static_cast<B*>(a.out), row, a.ld_out);
    // units of eight on the 16-byte grid of what is read: unit u begins at element 8 u - lead
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(in) & 15) / sizeof(A));
    const int v0 = static_cast<int>(item % slices) * kSlice - lead;
    if (v0 >= vocab) continue;
    const int v1 = min(v0 + kSlice, vocab);

    const int32_t* mask = nullptr;
    if (a.mask) {
      const int64_t m = a.mask_row ? a.mask_row[row] : row;
      if (m >= 0 && m < a.mask_rows) mask = a.mask + m * a.ldm;
    }
    int64_t tokens = 0, line = 0;
    if (a.history) {
      line = a.history_row ? a.history_row[row] : row;
      tokens = a.length ? a.length[row] : a.history_len;
      tokens = line >= 0 && line < a.history_rows ? min(max(tokens, int64_t(0)), a.history_len) : 0;
    }

    // what the mask allows of each unit, of the elements that exist
    uint32_t exists[kUnits], allowed[kUnits];
    Eight<A> raw[kUnits];
    const auto load = [&](int i, int e0) {
      if (exists[i] == 0xffu) {
        if (bounds_ok(e0 >= 0 && e0 + 8 <= vocab && on_16_bytes(in + e0), status, NSM_KERNEL_ADJUST, 0, NSM_SITE_LOGITS))
          raw[i].load_written(in + e0);
      } else {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = exists[i] >> e & 1 ? Elem<A>::to_float(in[e0 + e]) : 0.f;
        raw[i].set(f);
      }
    };
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int e0 = v0 + (tid + i * kThreads) * 8;
      const uint32_t low = e0 < 0 ? 0xffu << -e0 : 0xffu;
      const uint32_t high = e0 + 8 <= vocab ? 0xffu : e0 < vocab ? 0xffu >> (e0 + 8 - vocab) : 0u;
      exists[i] = low & high & 0xffu;
      allowed[i] = mask && exists[i] ? mask_bits(mask, nwords, e0, status) & exists[i] : exists[i];
#pragma unroll
      for (int w = 0; w < Eight<A>::kWords; ++w) raw[i].w[w] = make_uint4(0, 0, 0, 0);
    }
    if (!a.in_place) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        if (allowed[i]) load(i, v0 + (tid + i * kThreads) * 8);
    }

    const bool counted = tokens > 0 || a.k > 0;
    if (counted) {
#pragma unroll
      for (int i = 0; i < kSlice / 4 / kThreads; ++i)
        reinterpret_cast<uint4*>(count)[tid + i * kThreads] = make_uint4(0, 0, 0, 0);
      for (int j = tid; j < a.k; j += kThreads) {
        const int64_t v = index_at(a.bias_index, a.bias_wide, row * a.ldbi + j);
        bias_index[j] = v >= v0 && v < v1 && v >= 0 ? static_cast<int32_t>(v) : -1;
        bias[j] = a.bias[row * a.ldb + j];
      }
      __syncthreads();
      for (int64_t j = tid; j < tokens; j += kThreads) {
        if (!bounds_ok(line >= 0 && line < a.history_rows && j < a.history_len, status, NSM_KERNEL_ADJUST, 0, NSM_SITE_SIDE)) break;
        const int64_t v = index_at(a.history, a.history_wide, line * a.ldh + j);
        if (v >= v0 && v < v1 && v >= 0) atomicAdd(&count[v - v0], 1u);
      }
      for (int j = tid; j < a.k; j += kThreads)
        if (bias_index[j] >= 0) atomicOr(&count[bias_index[j] - v0], kHasBias);
      __syncthreads();
    }
    const float theta = a.repetition ? a.repetition[row] : 1.f;
    const float frequency = a.frequency ? a.frequency[row] : 0.f;
    const float presence = a.presence ? a.presence[row] : 0.f;
    const B* logits = kBackward && a.logits ? Rows::at(static_cast<const B*>(a.logits), row, a.ld_logits) : nullptr;
    const bool aligned_out = on_16_bytes(out + v0);

#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int u = tid + i * kThreads;
      const int e0 = v0 + u * 8;
      if (!exists[i]) continue;
      uint32_t c[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      uint32_t any = 0;
      if (counted) {
        *reinterpret_cast<uint4*>(c) = reinterpret_cast<const uint4*>(count)[2 * u];
        *reinterpret_cast<uint4*>(c + 4) = reinterpret_cast<const uint4*>(count)[2 * u + 1];
        any = c[0] | c[1] | c[2] | c[3] | c[4] | c[5] | c[6] | c[7];
      }
      if (a.in_place) {
        if (!any && allowed[i] == exists[i]) continue;  // stays as it is
        if (allowed[i]) load(i, e0);
      }
      float f[8];
      raw[i].get(f);
      if (any) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t n = c[e] & ~kHasBias;
          if (!c[e] || !(allowed[i] >> e & 1)) continue;
          if (n && a.repetition) {
            const float sign = kBackward ? Elem<B>::to_float(logits[e0 + e]) : f[e];
            f[e] = sign > 0.f ? f[e] / theta : f[e] * theta;
          }
          if (!kBackward) {
            if (n) f[e] -= fmaf(frequency, static_cast<float>(n), presence);
            if (c[e] & kHasBias)
              for (int j = 0; j < a.k; ++j)
                if (bias_index[j] == e0 + e) f[e] += bias[j];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(allowed[i] >> e & 1)) f[e] = kBackward ? 0.f : -__builtin_huge_valf();
      if (exists[i] == 0xffu && aligned_out) {
        Eight<B> r;
        r.set(f);
        if (bounds_ok(e0 >= 0 && e0 + 8 <= vocab && on_16_bytes(out + e0), status, NSM_KERNEL_ADJUST, 0, NSM_SITE_GRADIENT))
          r.store(out + e0);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (exists[i] >> e & 1) out[e0 + e] = Elem<B>::from_float(f[e]);
      }
    }
    if (item + gridDim.x < items) __syncthreads();  // the counts have been read
  }
}

template <typename A, typename B, bool kBackward>
cudaError_t launch_as(const AdjustArgs& a, int* status, cudaStream_t stream) {
  const int units = (a.vocab + 7 + 7) / 8;  // the lead is at most seven
  const int slices = (units + kSlice / 8 - 1) / (kSlice / 8);
  const bool counted = a.history || a.k;
  const size_t smem = counted ? size_t(kSlice) * 4 + size_t(a.k) * 8 : 0;
  const int64_t items = a.rows * slices;
  const int grid = static_cast<int>(std::min<int64_t>(items, INT32_MAX));
  return launch_pdl(k_adjust<A, B, kBackward>, dim3(grid), dim3(kThreads), smem, stream, a, slices, status);
}

template <typename T>
cudaError_t launch_forward(const AdjustArgs& a, int* status, cudaStream_t stream) {
  return a.out_dtype == NSM_FP32 ? launch_as<T, float, false>(a, status, stream) : launch_as<T, T, false>(a, status, stream);
}
template <typename T>
cudaError_t launch_backward(const AdjustArgs& a, int* status, cudaStream_t stream) {
  return a.in_dtype == NSM_FP32 ? launch_as<float, T, true>(a, status, stream) : launch_as<T, T, true>(a, status, stream);
}

}  // namespace

cudaError_t launch_adjust(const AdjustArgs& a, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  const int dtype = a.backward ? a.out_dtype : a.in_dtype;
  if (dtype == NSM_BF16)
    return a.backward ? launch_backward<__nv_bfloat16>(a, status, stream) : launch_forward<__nv_bfloat16>(a, status, stream);
  if (dtype == NSM_FP16)
    return a.backward ? launch_backward<__half>(a, status, stream) : launch_forward<__half>(a, status, stream);
  return a.backward ? launch_backward<float>(a, status, stream) : launch_forward<float>(a, status, stream);
}

}  // namespace nsm
