// Penalties for repeated tokens, biases and grammar masks on rows of logits, and their backward
// pass.
//
//   c_v = how often token v occurs in the row's history
//   a_v = x_v / repetition (x_v > 0) or x_v repetition where c_v > 0, else x_v
//   out_v = a_v - (frequency c_v + presence [c_v > 0]) + sum of the biases at v; -inf where banned
//   d x_v = d out_v (d a_v / d x_v); 0 where banned
//
// A block takes a slice of 4096 (fp32: 2048) logits of one row after another.  It counts the history's
// tokens among them in shared memory (whole numbers: their order does not matter), writes the
// slice as it was read, with the mask applied, and then settles the tokens that a penalty or a
// bias is for, one thread each.  Rows that share a history, as the positions of one sequence
// do, follow one another in a block, which counts only the tokens that a row has more.  The next
// slice's logits are asked for before a slice is settled, and which history it has a row earlier.
//
// Without penalties bound by memory (8192 x 50257 bf16 256 us, 6.4 TB/s read and written); with them by
// the two barriers of a slice and the accesses to single tokens between them: 281 us with a sequence's
// growing history of 1024 tokens, 256 x 131072 to fp32 with 4096 tokens and masks 55 us.
#include "elem.cuh"
#include "launch.cuh"
#include "nsm_internal.h"

#include <algorithm>
#include <type_traits>

namespace nsm {
namespace {

constexpr int kThreads = 128;
constexpr uint32_t kHasBias = 0x80000000u;       // in a count: some bias is for this token

__device__ __forceinline__ bool on_bytes(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

__device__ __forceinline__ int64_t index_at(const void* p, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

// The bits of a row's mask for the unit of kE elements from e0 on (bit set: allowed); all of them exist.
template <int kE>
__device__ __forceinline__ uint32_t mask_bits(const int32_t* words, int nwords, int e0, int* status) {
  const int w = e0 >> 5, bit = e0 & 31;
  if (!bounds_ok(w >= 0 && (e0 + kE - 1) >> 5 < nwords, status, NSM_KERNEL_ADJUST, 0, NSM_SITE_SIDE)) return 0;
  const uint32_t low = static_cast<uint32_t>(__ldg(words + w));
  return __funnelshift_r(low, bit > 32 - kE ? static_cast<uint32_t>(__ldg(words + w + 1)) : 0u, bit) & ((1u << kE) - 1);
}

// A unit with -inf (0 in the backward pass) where a bit of `allowed` is clear.
template <typename T, int kE, bool kBackward>
__device__ __forceinline__ void ban(Side<T, kE>& r, uint32_t allowed) {
  constexpr uint32_t kGone = kBackward ? 0u : Elem<T>::kNegInfBits;
  uint32_t* w = reinterpret_cast<uint32_t*>(&r.w);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (!(allowed >> e & 1)) w[e] = kGone;
  } else {
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      const uint32_t keep = (allowed >> (2 * i) & 1) * 0xffffu | (allowed >> (2 * i + 1) & 1) * 0xffff0000u;
      w[i] = (w[i] & keep) | (~keep & (kGone * 0x10001u));
    }
  }
}

template <typename A, typename B, int kE>
__device__ __forceinline__ void convert(const Side<A, kE>& from, Side<B, kE>& to) {
  if constexpr (std::is_same<A, B>::value) {
    to.w = from.w;
  } else {
    float f[kE];
    from.get(f);
    to.set(f);
  }
}

// Logits of a unit: 16 bytes of what is read, so that a warp's loads lie side by side (fp32 in units of
// eight, 32 bytes apart: 2049 x 65537 copied in 212 us for 177).  Units per thread, and logits of a
// block: 8 KB.
template <typename A>
constexpr int kUnitOf = 16 / sizeof(A);
template <typename A>
constexpr int kSliceOf = kThreads * (sizeof(A) == 4 ? 16 : 32);
// Resident blocks of an SM.  8192 x 50257 bf16 with histories takes 281 us with 7, 341 with 8 (whose 64
// registers a thread are too few) and 295 with 6, 256 x 131072 bf16 to fp32 55, 59 and 60; 2049 x 65537 fp32 203 with 8,
// 380 with 9, 214 with 7.
template <typename A>
constexpr int kBlocks = sizeof(A) == 4 ? 8 : 7;

// Rows at most whose slices a block takes after one another: the two cases above take 302 and 227 us with
// 16, 281 and 203 with 4, 288 and 203 with 2.
constexpr int kRun = 4;

// Calls f with every token of a row's history, in no order.
template <typename I, typename F>
__device__ __forceinline__ void for_history(const I* p, int tokens, F f) {
  constexpr int kPer = 16 / sizeof(I);
  const int head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) % 16 / sizeof(I)), tokens);
  const int vecs = (tokens - head) / kPer;
  const int4* v = reinterpret_cast<const int4*>(p + head);
  const auto all = [&](const int4& q) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) f(static_cast<int64_t>(reinterpret_cast<const I*>(&q)[e]));
  };
  for (int i = threadIdx.x; i < vecs; i += 2 * kThreads) {
    const bool two = i + kThreads < vecs;
    const int4 q = v[i];
    const int4 r = two ? v[i + kThreads] : q;
    all(q);
    if (two) all(r);
  }
  const int rest = head + vecs * kPer + threadIdx.x;
  if (static_cast<int>(threadIdx.x) < head) f(static_cast<int64_t>(p[threadIdx.x]));
  if (rest < tokens) f(static_cast<int64_t>(p[rest]));
}

// A: type of what is read, B: of what is written.
template <typename A, typename B, bool kBackward>
__global__ void __launch_bounds__(kThreads, kBlocks<A>) k_adjust(const AdjustArgs a, int slices, int run, int* status) {
  constexpr int kE = kUnitOf<A>, kSlice = kSliceOf<A>, kUnits = kSlice / kThreads / kE, kPlaces = kSlice + 8;
  constexpr uint32_t kAll = (1u << kE) - 1;
  constexpr size_t kStore = kE * sizeof(B) < 16 ? kE * sizeof(B) : 16;  // what a unit's stores are aligned to
  static_assert(kUnits * kE <= 32, "a bit per element");
  extern __shared__ __align__(16) uint32_t shared[];
  uint32_t* count = shared;                                              // kPlaces
  uint16_t* list = reinterpret_cast<uint16_t*>(shared + kPlaces);        // kPlaces: those with a count
  float* bias = reinterpret_cast<float*>(list + kPlaces);                // a.k
  int32_t* bias_index = reinterpret_cast<int32_t*>(bias + a.k);          // a.k
  __shared__ int listed[2];
  const int tid = threadIdx.x, vocab = a.vocab;
  const bool counts = a.history || a.k;
  if (counts) {  // once: every count goes back to 0 with the last row that wants it
    for (int i = tid; i < kPlaces / 4; i += kThreads) reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
    if (tid < 2) listed[tid] = 0;
    __syncthreads();
  }
  grid_dependency_sync();
  release_dependents();
  const int nwords = (vocab + 31) / 32;
  const uint32_t rows = static_cast<uint32_t>(a.rows);
  // A block takes one slice of `run` rows after one another, then of other rows.
  const int run_step = gridDim.x / slices, slice_step = gridDim.x % slices;

  // One slice of a row: units on the grid that their loads want, unit u from element v0 + kE u on.  v0 may lie before the row, by less than a vector.
  struct Place {
    uint32_t row;
    int line, slice, v0, tokens;
    const A* in;
    const int32_t* mask;
  };
  const auto place = [&](Place& p) {
    p.in = static_cast<const A*>(a.in) + int64_t(p.row) * a.ld_in;
    p.v0 = p.slice * kSlice - static_cast<int>((reinterpret_cast<uintptr_t>(p.in) & (kE * sizeof(A) - 1)) / sizeof(A));
    p.mask = nullptr;
    if (a.mask) {
      const int m = a.mask_row ? a.mask_row[p.row] : static_cast<int>(p.row);
      if (m >= 0 && m < a.mask_rows) p.mask = a.mask + m * a.ldm;
    }
  };
  // Which history a row has, as the tables hold it: asked for a row ahead, looked at when its turn comes.
  struct Held {
    int line, length;
  };
  const auto look = [&](uint32_t row) {
    Held h{0, 0};
    if (a.history && row < rows) {
      h.line = a.history_row ? a.history_row[row] : static_cast<int>(row);
      h.length = a.length ? a.length[row] : static_cast<int>(a.history_len);
    }
    return h;
  };
  const auto take = [&](Place& p, const Held& h) {
    p.line = h.line;
    p.tokens = h.line >= 0 && h.line < a.history_rows ? min(max(h.length, 0), static_cast<int>(a.history_len)) : 0;
  };
  // Most slices lie inside their row with all their units.
  const auto inside = [&](int v0) { return v0 >= 0 && v0 + kSlice <= vocab; };
  const auto whole = [&](int e0) { return e0 >= 0 && e0 + kE <= vocab; };
  uint32_t allowed = 0;  // with a mask, kE bits per unit: the elements that it allows
  Side<A, kE> raw[kUnits];
  // What a row has before its first whole unit and behind its last one: threads 0 to 7 and 8 to
  // 15 of the block that has them take an element each.
  A edge = Elem<A>::from_float(0.f);
  const auto edge_at = [&](int v0) {  // -1: none
    if (tid >= 16) return -1;
    const int tail = v0 + (vocab - v0) / kE * kE;
    const int e = tid < 8 ? v0 + tid : tail + tid - 8;
    const bool mine = (tid & 7) < kE && (tid < 8 ? v0 < 0 : tail < v0 + kSlice && !(v0 < 0 && tail == v0));
    return mine && e >= 0 && e < vocab ? e : -1;
  };
  const auto load = [&](const A* from, int i) {
    if (bounds_ok(on_bytes(from + i * kThreads * kE, kE * sizeof(A)), status, NSM_KERNEL_ADJUST, 0, NSM_SITE_LOGITS)) raw[i].load(from + i * kThreads * kE);
  };
  const auto fetch_units = [&](const Place& p, auto all) {
    const int first = p.v0 + tid * kE;
    const A* from = p.in + first;
    if (!p.mask) {
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
        if (decltype(all)::value || whole(first + i * kThreads * kE)) load(from, i);
      return;
    }
    allowed = 0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const int e0 = first + i * kThreads * kE;
      if (decltype(all)::value || whole(e0)) allowed |= mask_bits<kE>(p.mask, nwords, e0, status) << (kE * i);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t may = allowed >> (kE * i) & kAll;
      if (may && !(a.in_place && may == kAll)) load(from, i);
    }
  };
  const auto fetch = [&](const Place& p) {
    if (a.in_place && !p.mask) return;
    if (inside(p.v0)) {
      fetch_units(p, std::true_type());
    } else {
      fetch_units(p, std::false_type());
      const int e = edge_at(p.v0);
      if (e >= 0) {
        edge = p.in[e];
        if (p.mask && !(static_cast<uint32_t>(p.mask[e >> 5]) >> (e & 31) & 1)) edge = Elem<A>::from_float(kBackward ? 0.f : -__builtin_huge_valf());
      }
    }
  };

  Place now{};
  uint32_t first = blockIdx.x / slices * run;  // of the rows that it takes after one another
  now.row = first;
  now.slice = blockIdx.x % slices;
  if (now.row >= rows) return;
  place(now);
  fetch(now);
  take(now, look(now.row));
  // the row and slice after one
  const auto advance = [&](uint32_t& row, int& slice, uint32_t& of_run) {
    if (++row >= min(of_run + run, rows)) {
      const int carry = slice + slice_step >= slices;
      of_run += (run_step + carry) * run;
      row = of_run;
      slice += slice_step - (carry ? slices : 0);
    }
  };
  uint32_t next_row = now.row;
  int next_slice = now.slice;
  advance(next_row, next_slice, first);
  Held next_held = look(next_row);
  int parity = 0, held = 0;  // tokens of this row's history that are counted already
  for (;;) {
    // counts are kept of all tokens that may be in this slice of some row, whatever its v0
    const int v0 = now.v0, base = now.slice * kSlice - 7;
    const int low = max(base, 0), span = min(base + 7 + kSlice, vocab) - low;  // span <= 0: nothing is left
    if (now.tokens > held && span > 0) {
      const auto bump = [&](int64_t v) {
        if (static_cast<uint64_t>(v - low) >= static_cast<uint64_t>(span)) return;
        if (atomicAdd(&count[v - base], 1u) == 0) list[atomicAdd(&listed[parity], 1)] = static_cast<uint16_t>(v - base);
      };
      if (a.history_wide) for_history(static_cast<const int64_t*>(a.history) + int64_t(now.line) * a.ldh + held, now.tokens - held, bump);
      else for_history(static_cast<const int32_t*>(a.history) + int64_t(now.line) * a.ldh + held, now.tokens - held, bump);
    }
    for (int j = tid; j < a.k; j += kThreads) {
      const int64_t v = index_at(a.bias_index, a.bias_wide, int64_t(now.row) * a.ldbi + j);
      const bool here = span > 0 && static_cast<uint64_t>(v - low) < static_cast<uint64_t>(span);
      bias_index[j] = here ? static_cast<int32_t>(v) : -1;
      bias[j] = a.bias[int64_t(now.row) * a.ldb + j];
      if (here && atomicOr(&count[v - base], kHasBias) == 0) list[atomicAdd(&listed[parity], 1)] = static_cast<uint16_t>(v - base);
    }

    B* out = static_cast<B*>(a.out) + int64_t(now.row) * a.ld_out;
    const bool aligned_out = on_bytes(out + v0, kStore);
    const auto store_units = [&](auto all) {
      const int first_unit = v0 + tid * kE;
      B* to = out + first_unit;
#pragma unroll
      for (int i = 0; i < kUnits; ++i) {
        const uint32_t may = now.mask ? allowed >> (kE * i) & kAll : kAll;
        if (!(decltype(all)::value || whole(first_unit + i * kThreads * kE)) || (a.in_place && may == kAll)) continue;
        Side<B, kE> r;
        convert(raw[i], r);
        if (may != kAll) ban<B, kE, kBackward>(r, may);
        if (aligned_out) {
          if (bounds_ok(on_bytes(to + i * kThreads * kE, kStore), status, NSM_KERNEL_ADJUST, 0, NSM_SITE_GRADIENT)) r.store(to + i * kThreads * kE);
        } else {
#pragma unroll
          for (int e = 0; e < kE; ++e) to[i * kThreads * kE + e] = reinterpret_cast<const B*>(&r.w)[e];
        }
      }
    };
    if (!a.in_place || now.mask) {
      if (inside(v0)) {
        store_units(std::true_type());
      } else {
        store_units(std::false_type());
        const int e = edge_at(v0);
        if (e >= 0) out[e] = Elem<B>::from_float(Elem<A>::to_float(edge));
      }
    }

    // the next slice's logits are asked for before this one's tokens are settled
    const Place last = now;
    const float theta = a.repetition ? a.repetition[last.row] : 1.f;
    const float frequency = a.frequency ? a.frequency[last.row] : 0.f;
    const float presence = a.presence ? a.presence[last.row] : 0.f;
    now.row = next_row;
    now.slice = next_slice;
    const bool more = now.row < rows;
    if (more) {
      place(now);
      fetch(now);
      take(now, next_held);
      advance(next_row, next_slice, first);
      next_held = look(next_row);
    }

    // what a penalty or a bias is for, one token at a time, over what was just written
    held = 0;
    if (last.tokens > 0 || a.k > 0) {
      // positions of one sequence: the next row's history is this one's and some tokens more
      const bool keep = more && a.k == 0 && now.slice == last.slice && now.line == last.line && now.tokens >= last.tokens;
      if (keep) held = last.tokens;
      __syncthreads();
      const int n_listed = listed[parity];
      if (tid == 0) listed[parity ^ 1] = 0;
      for (int i = tid; i < n_listed; i += kThreads) {
        const int at = list[i], v = base + at;
        const uint32_t c = count[at], n = c & ~kHasBias;
        if (!keep) count[at] = 0;
        if (v < v0 || v >= v0 + kSlice) continue;  // another slice's of this row
        if (last.mask && !(static_cast<uint32_t>(last.mask[v >> 5]) >> (v & 31) & 1)) continue;
        if (!bounds_ok(v >= 0 && v < vocab, status, NSM_KERNEL_ADJUST, 0, NSM_SITE_LOGITS)) continue;
        float f = Elem<A>::to_float(last.in[v]);
        if (n && a.repetition) {
          const float sign = kBackward ? Elem<B>::to_float(static_cast<const B*>(a.logits)[int64_t(last.row) * a.ld_logits + v]) : f;
          f = sign > 0.f ? f / theta : f * theta;
        }
        if (!kBackward) {
          if (n) f -= fmaf(frequency, static_cast<float>(n), presence);
          if (c & kHasBias)
            for (int j = 0; j < a.k; ++j)
              if (bias_index[j] == v) f += bias[j];
        }
        out[v] = Elem<B>::from_float(f);
      }
      __syncthreads();  // the next row counts in the same places
      if (!keep) parity ^= 1;
    }
    if (!more) return;
  }
}

template <typename A, typename B, bool kBackward>
cudaError_t launch_as(const AdjustArgs& a, int* status, cudaStream_t stream) {
  constexpr int kSlice = kSliceOf<A>;
  const int slices = (a.vocab + 7 + kSlice - 1) / kSlice;  // the lead is at most seven
  const bool counts = a.history || a.k;
  const size_t places = kSlice + 8, smem = counts ? places * 6 + size_t(a.k) * 8 : 0;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = set_smem_once(k_adjust<A, B, kBackward>, places * 6 + size_t(kBiasMaxK) * 8, done);
  if (e != cudaSuccess) return e;
  // Rows that share histories are taken in runs, so that a history is counted once per run; a
  // block still gets four of them, of different slices.
  const int64_t resident = int64_t(a.num_sms) * kBlocks<A>;
  const int run = a.history_row ? static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kRun, a.rows * slices / (4 * resident)))) : 1;
  const int64_t items = (a.rows + run - 1) / run * slices;
  const int grid = static_cast<int>(std::min<int64_t>(items, resident));
  return launch_pdl(k_adjust<A, B, kBackward>, dim3(grid), dim3(kThreads), smem, stream, a, slices, run, status);
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
