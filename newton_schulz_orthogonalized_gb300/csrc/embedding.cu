// The embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out_r = scale weight[token_r]                       (0 without a token)
//   d_weight[v] (+)= scale sum_{r: token_r = v} d_out_r
//
//   k_embed        a group of lanes per row: reads and writes, nothing else.
//   k_sort_count, k_sort_place
//                  one pass of a stable radix sort of (token, row) by a digit of the token: a
//                  block per tile counts its digits; every block then adds up the counts of
//                  the tiles before its own and places its pairs in order.  Rows without a token
//                  sort behind the others.
//   k_embed_sums   pieces of kPiece sorted entries: a group of lanes adds the rows of equal
//                  tokens in ascending order and writes each sum; the sums of a token that lies
//                  in several pieces go to the workspace.  Blocks behind those clear the rows
//                  of the gradient that no token asks for.
//   k_embed_join   adds up such tokens' sums, piece after piece.
// No atomic adds a floating-point number: the order of every sum is that of the rows.
#include "elem.cuh"
#include "launch.cuh"
#include "nsm_internal.h"

#include <algorithm>

namespace nsm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnits = 4;      // of eight columns, per lane of k_embed
constexpr int kMaxBits = 10;   // of a sorting pass's digit
constexpr int kMaxTiles = 64;
constexpr int kPiece = 32;     // sorted entries of a group of lanes
constexpr int kClear = 64;     // rows of the gradient that a block looks at

__device__ __forceinline__ int64_t token_at(const EmbeddingArgs& a, int64_t r) {
  return a.tokens_wide ? static_cast<const int64_t*>(a.tokens)[r] : static_cast<const int32_t*>(a.tokens)[r];
}
// The token as a key: those that are none are `vocab`, behind all others.
__device__ __forceinline__ uint32_t key_at(const EmbeddingArgs& a, int64_t r) {
  const int64_t t = token_at(a, r);
  return static_cast<uint32_t>(t >= 0 && t < a.vocab ? t : a.vocab);
}

__device__ __forceinline__ bool row_ok(bool ok, int* status, int site) {
  return bounds_ok(ok, status, NSM_KERNEL_EMBEDDING, 0, site);
}

// Eight columns from c0 on: the next eight where kVec (16-byte accesses), else every lanes-th.
template <bool kVec>
__device__ __forceinline__ int64_t column(int64_t slice, int lanes, int lane, int e) {
  return kVec ? (slice * lanes + lane) * 8 + e : slice * lanes * 8 + lane + int64_t(e) * lanes;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load_columns(const T* row, int64_t cols, int64_t slice, int lanes, int lane, Eight<T>& r,
                                             int* status, int site) {
  const int64_t c0 = column<kVec>(slice, lanes, lane, 0);
  if (kVec && c0 + 8 <= cols) {
    if (row_ok(on_16_bytes(row + c0), status, site)) r.load(row + c0);
    return;
  }
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t c = column<kVec>(slice, lanes, lane, e);
    f[e] = c < cols ? Elem<T>::to_float(row[c]) : 0.f;
  }
  r.set(f);
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_columns(T* row, int64_t cols, int64_t slice, int lanes, int lane, const float (&f)[8],
                                              int* status, int site) {
  const int64_t c0 = column<kVec>(slice, lanes, lane, 0);
  if (kVec && c0 + 8 <= cols && on_16_bytes(row + c0)) {
    Eight<T> r;
    r.set(f);
    r.store(row + c0);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t c = column<kVec>(slice, lanes, lane, e);
    if (c < cols) row[c] = Elem<T>::from_float(f[e]);
  }
}

// ---------------------------------------------------------------- lookup

template <typename W, typename O, bool kVec>
__global__ void __launch_bounds__(kThreads) k_embed(const EmbeddingArgs a, int lanes, int chunks, int* status) {
  grid_dependency_sync();
  release_dependents();
  const int lane = threadIdx.x & (lanes - 1), groups = kThreads / lanes;
  const int64_t items = a.rows * chunks;
  const int64_t slices = (a.cols + lanes * 8 - 1) / (lanes * 8);
  for (int64_t item = int64_t(blockIdx.x) * groups + threadIdx.x / lanes; item < items; item += int64_t(gridDim.x) * groups) {
    const int64_t row = item / chunks, first = item % chunks * kUnits;
    const int64_t token = token_at(a, row);
    const bool has = token >= 0 && token < a.vocab;
    const W* from = static_cast<const W*>(a.weight) + (has ? token : 0) * a.ld_weight;
    O* to = static_cast<O*>(a.rows_out) + row * a.ld_rows;
    Eight<W> raw[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
      if (has && first + i < slices)
        load_columns<W, kVec>(from, a.cols, first + i, lanes, lane, raw[i], status, NSM_SITE_EMBEDDING);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (first + i >= slices) break;
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (has) {
        raw[i].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= a.scale;
      }
      store_columns<O, kVec>(to, a.cols, first + i, lanes, lane, f, status, NSM_SITE_EMBEDDING);
    }
  }
}

// ---------------------------------------------------------------- sorting tokens

// The pair of entry i: from the tokens in the first pass, from the pass before later on.
__device__ __forceinline__ uint2 pair_at(const EmbeddingArgs& a, const uint2* pairs, int64_t i) {
  return pairs ? pairs[i] : make_uint2(key_at(a, i), static_cast<uint32_t>(i));
}

__global__ void __launch_bounds__(kThreads)
    k_sort_count(const EmbeddingArgs a, const EmbeddingPlan p, const uint2* pairs, int shift, uint32_t* counts,
                 int32_t* last, int* status) {
  __shared__ uint32_t hist[1 << kMaxBits];
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += kThreads) hist[b] = 0;
  __syncthreads();
  grid_dependency_sync();
  release_dependents();
  const int64_t first = int64_t(blockIdx.x) * p.tile, end = min(first + p.tile, a.rows);
  for (int64_t i = first + threadIdx.x; i < end; i += kThreads) {
    if (!row_ok(i < a.rows, status, NSM_SITE_WORKSPACE)) break;
    const uint32_t key = pair_at(a, pairs, i).x;
    atomicAdd(&hist[key >> shift & (bins - 1)], 1u);
    // some row that asks for this token, whichever thread comes last: see k_embed_sums
    if (last && key < a.vocab) asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(last + key), "r"(static_cast<int32_t>(i)) : "memory");
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kThreads) counts[int64_t(blockIdx.x) * bins + b] = hist[b];
}

__global__ void __launch_bounds__(kThreads)
    k_sort_place(const EmbeddingArgs a, const EmbeddingPlan p, const uint2* pairs, int shift, const uint32_t* counts,
                 uint2* placed, int* status) {
  __shared__ uint32_t place[kWarps][1 << kMaxBits];  // of each warp's next pair with a digit
  __shared__ uint32_t warp_total[kWarps];
  const int bins = 1 << p.bits, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int w = 0; w < kWarps; ++w)
    for (int b = threadIdx.x; b < bins; b += kThreads) place[w][b] = 0;
  __syncthreads();
  grid_dependency_sync();
  release_dependents();
  const int64_t tile0 = int64_t(blockIdx.x) * p.tile, tile1 = min(tile0 + p.tile, a.rows);
  const int64_t part = p.tile / kWarps;  // whole groups of 32
  const int64_t first = min(tile0 + warp * part, tile1), end = min(first + part, tile1);
  for (int64_t i = first + lane; i < end; i += 32) atomicAdd(&place[warp][pair_at(a, pairs, i).x >> shift & (bins - 1)], 1u);

  // digits 4 tid ... 4 tid + 3: all pairs with a digit, and those of the tiles before this one
  uint32_t all[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
  const int b0 = threadIdx.x * 4;
  for (int t = 0; t < p.tiles; ++t) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (b0 + d >= bins) break;
      const uint32_t n = counts[int64_t(t) * bins + b0 + d];
      all[d] += n;
      if (t < blockIdx.x) before[d] += n;
    }
  }
  const uint32_t own = all[0] + all[1] + all[2] + all[3];
  uint32_t scan = own;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t n = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += n;
  }
  if (lane == 31) warp_total[warp] = scan;
  __syncthreads();
  uint32_t base = scan - own;
  for (int w = 0; w < warp; ++w) base += warp_total[w];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if (b0 + d >= bins) break;
    uint32_t at = base + before[d];
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t n = place[w][b0 + d];
      place[w][b0 + d] = at;
      at += n;
    }
    base += all[d];
  }
  __syncthreads();
  for (int64_t i0 = first; i0 < end; i0 += 32) {
    const int64_t i = i0 + lane;
    const uint32_t live = __ballot_sync(0xffffffffu, i < end);
    if (i < end) {
      const uint2 pair = pair_at(a, pairs, i);
      const uint32_t digit = pair.x >> shift & (bins - 1);
      const uint32_t same = __match_any_sync(live, digit);
      const uint32_t rank = __popc(same & ((1u << lane) - 1));
      const uint32_t at = place[warp][digit] + rank;
      __syncwarp(live);
      if (rank == 0) place[warp][digit] += __popc(same);
      __syncwarp(live);
      if (row_ok(at < a.rows, status, NSM_SITE_WORKSPACE)) placed[at] = pair;
    }
  }
}

// ---------------------------------------------------------------- sums

// Whether some row asks for token v: last[v], which nothing ever clears, is then one of them.
__device__ __forceinline__ bool asked_for(const EmbeddingArgs& a, const int32_t* last, int64_t v) {
  const int64_t r = last[v];
  return r >= 0 && r < a.rows && token_at(a, r) == v;
}

template <typename W>
__device__ __forceinline__ void clear_row(W* row, int64_t cols, int lane, int* status) {
  constexpr int kVecElems = 16 / sizeof(W);
  const int64_t head = min(static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / sizeof(W)), cols);
  const int64_t vecs = (cols - head) / kVecElems;
  if (lane < head) row[lane] = Elem<W>::from_float(0.f);
  for (int64_t i = lane; i < vecs; i += 32)
    if (row_ok(on_16_bytes(row + head + i * kVecElems), status, NSM_SITE_EMBEDDING))
      reinterpret_cast<uint4*>(row + head)[i] = make_uint4(0, 0, 0, 0);
  const int64_t c = head + vecs * kVecElems + lane;
  if (c < cols) row[c] = Elem<W>::from_float(0.f);
}

template <typename W, bool kVec>
__device__ __forceinline__ void write_sum(const EmbeddingArgs& a, uint32_t token, int64_t slice, int lanes, int lane,
                                          const float (&sum)[8], int* status) {
  if (!row_ok(token < a.vocab, status, NSM_SITE_EMBEDDING)) return;
  W* row = static_cast<W*>(a.d_weight) + int64_t(token) * a.ld_weight;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = a.scale * sum[e];
  if (a.accumulate) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = column<kVec>(slice, lanes, lane, e);
      if (c < a.cols) f[e] += Elem<W>::to_float(row[c]);
    }
  }
  store_columns<W, kVec>(row, a.cols, slice, lanes, lane, f, status, NSM_SITE_EMBEDDING);
}

// A piece's two sums in the workspace: of a token that began in an earlier piece and ends in
// this one, and of one that goes on in the next.
__device__ __forceinline__ float* piece_sum(const EmbeddingPlan& p, float* sums, int64_t piece, int which) {
  return sums + (piece * 2 + which) * p.cols;
}

// G: type of the rows' gradients, W: of the weight's.
template <typename G, typename W, bool kVec>
__global__ void __launch_bounds__(kThreads)
    k_embed_sums(const EmbeddingArgs a, const EmbeddingPlan p, const uint2* pairs, const int32_t* last, float* sums,
                 int lanes, int slices, int64_t sum_blocks, int* status) {
  grid_dependency_sync();
  release_dependents();
  if (blockIdx.x >= sum_blocks) {  // rows of the gradient that no token asks for
    const int64_t v0 = (blockIdx.x - sum_blocks) * kClear + threadIdx.x / 32 * (kClear / kWarps);
    const int lane = threadIdx.x & 31;
    const int64_t v = v0 + lane;
    const bool none = lane < kClear / kWarps && v < a.vocab && !asked_for(a, last, v);
    uint32_t rows = __ballot_sync(0xffffffffu, none);
    for (; rows; rows &= rows - 1)
      clear_row(static_cast<W*>(a.d_weight) + (v0 + __ffs(rows) - 1) * a.ld_weight, a.cols, lane, status);
    return;
  }
  const int lane = threadIdx.x & (lanes - 1), groups = kThreads / lanes;
  const int64_t item = blockIdx.x * int64_t(groups) + threadIdx.x / lanes;
  const int64_t piece = item % p.units, slice = item / p.units;
  if (slice >= slices) return;
  const int64_t first = piece * kPiece, end = min(first + kPiece, a.rows);
  uint32_t token = pairs[first].x;
  if (token >= a.vocab) return;
  bool joined = first > 0 && pairs[first - 1].x == token;  // the token began in an earlier piece
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const auto keep = [&](int which) {
    float* to = piece_sum(p, sums, piece, which);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = column<kVec>(slice, lanes, lane, e);
      if (c < p.cols) to[c] = sum[e];
    }
  };
  const auto finish = [&]() {
    if (joined) keep(0); else write_sum<W, kVec>(a, token, slice, lanes, lane, sum, status);
  };
  constexpr int kAhead = 4;
  for (int64_t j0 = first; j0 < end; j0 += kAhead) {
    uint2 pair[kAhead];
    Eight<G> raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) pair[i] = j0 + i < end ? pairs[j0 + i] : make_uint2(static_cast<uint32_t>(a.vocab), 0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (pair[i].x < a.vocab && row_ok(pair[i].y < a.rows, status, NSM_SITE_EMBEDDING))
        load_columns<G, kVec>(static_cast<const G*>(a.rows_in) + int64_t(pair[i].y) * a.ld_rows, a.cols, slice, lanes, lane,
                              raw[i], status, NSM_SITE_EMBEDDING);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (pair[i].x >= a.vocab) break;
      if (pair[i].x != token) {
        finish();
        token = pair[i].x;
        joined = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = 0.f;
      }
      float f[8];
      raw[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += f[e];
    }
  }
  if (end < a.rows && pairs[end].x == token) keep(1); else finish();
}

// For every piece in which a token of earlier pieces ends: their sums in order.
template <typename W, bool kVec>
__global__ void __launch_bounds__(kThreads)
    k_embed_join(const EmbeddingArgs a, const EmbeddingPlan p, const uint2* pairs, const float* sums, int lanes, int slices,
                 int* status) {
  grid_dependency_sync();
  release_dependents();
  const int lane = threadIdx.x & (lanes - 1), groups = kThreads / lanes;
  const int64_t item = blockIdx.x * int64_t(groups) + threadIdx.x / lanes;
  const int64_t piece = item % p.units, slice = item / p.units;
  if (slice >= slices || piece == 0) return;
  const int64_t first = piece * kPiece, end = min(first + kPiece, a.rows);
  const uint32_t token = pairs[first].x;
  if (token >= a.vocab || pairs[first - 1].x != token) return;
  if (end < a.rows && pairs[end].x == token) return;  // goes on
  int64_t low = 0, high = first - 1;  // where the token's entries begin
  while (low < high) {
    const int64_t mid = (low + high) / 2;
    if (pairs[mid].x < token) low = mid + 1; else high = mid;
  }
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t w = low / kPiece; w <= piece; ++w) {
    const float* from = piece_sum(p, const_cast<float*>(sums), w, w < piece ? 1 : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = column<kVec>(slice, lanes, lane, e);
      if (c < p.cols) sum[e] += from[c];
    }
  }
  write_sum<W, kVec>(a, token, slice, lanes, lane, sum, status);
}

// Lanes that share a row: as many as its eights of columns ask for, a power of two, a warp at most.
int lanes_for(int64_t cols) {
  int lanes = 1;
  while (lanes < 32 && lanes * 8 < cols) lanes *= 2;
  return lanes;
}

bool rows_aligned(const void* p, int64_t ld, int dtype) {
  const int64_t size = dtype == NSM_FP32 ? 4 : 2;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

int blocks(int64_t n) { return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 1), INT32_MAX)); }

template <typename W, typename O>
cudaError_t launch_embed(const EmbeddingArgs& a, int* status, cudaStream_t stream) {
  const int lanes = lanes_for(a.cols);
  const int64_t slices = (a.cols + lanes * 8 - 1) / (lanes * 8);
  const int chunks = static_cast<int>((slices + kUnits - 1) / kUnits);
  const dim3 grid(blocks((a.rows * chunks + kThreads / lanes - 1) / (kThreads / lanes)));
  const bool vec = rows_aligned(a.weight, a.ld_weight, a.weight_dtype) && rows_aligned(a.rows_out, a.ld_rows, a.rows_dtype);
  return launch_pdl(vec ? k_embed<W, O, true> : k_embed<W, O, false>, grid, dim3(kThreads), 0, stream, a, lanes, chunks, status);
}

template <typename G, typename W, bool kVec>
cudaError_t launch_sums(const EmbeddingArgs& a, const EmbeddingPlan& p, const uint2* pairs, const int32_t* last, float* sums,
                        int* launches, int* status, cudaStream_t stream) {
  const int lanes = lanes_for(a.cols);
  const int64_t slices = (a.cols + lanes * 8 - 1) / (lanes * 8);
  const int64_t groups = kThreads / lanes, sum_blocks = (p.units * slices + groups - 1) / groups;
  const int64_t clear = a.accumulate ? 0 : (a.vocab + kClear - 1) / kClear;
  cudaError_t e = launch_pdl(k_embed_sums<G, W, kVec>, dim3(blocks(sum_blocks + clear)), dim3(kThreads), 0, stream, a, p, pairs,
                             last, sums, lanes, static_cast<int>(slices), sum_blocks, status);
  ++*launches;
  if (e != cudaSuccess || p.units <= 1) return e;
  ++*launches;
  return launch_pdl(k_embed_join<W, kVec>, dim3(blocks(sum_blocks)), dim3(kThreads), 0, stream, a, p, pairs,
                    static_cast<const float*>(sums), lanes, static_cast<int>(slices), status);
}

template <typename G, typename W>
cudaError_t launch_gradient(const EmbeddingArgs& a, const EmbeddingPlan& p, const uint2* pairs, const int32_t* last,
                            float* sums, int* launches, int* status, cudaStream_t stream) {
  return rows_aligned(a.rows_in, a.ld_rows, a.rows_dtype)
             ? launch_sums<G, W, true>(a, p, pairs, last, sums, launches, status, stream)
             : launch_sums<G, W, false>(a, p, pairs, last, sums, launches, status, stream);
}

// f with a value of each of the two types
template <typename F>
cudaError_t for_types(int first, int second, F f) {
  const auto with = [&](auto x) {
    if (second == NSM_BF16) return f(x, __nv_bfloat16());
    if (second == NSM_FP16) return f(x, __half());
    return f(x, float());
  };
  if (first == NSM_BF16) return with(__nv_bfloat16());
  if (first == NSM_FP16) return with(__half());
  return with(float());
}

}  // namespace

EmbeddingPlan embedding_plan(int64_t rows, int64_t vocab, int64_t cols) {
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  EmbeddingPlan p{};
  int bits = 1;
  while (bits < 62 && vocab >> bits) ++bits;  // keys 0 ... vocab
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  const int64_t step = 32 * kWarps;
  p.tile = static_cast<int32_t>(std::max<int64_t>(1024, ((rows + kMaxTiles - 1) / kMaxTiles + step - 1) / step * step));
  p.tiles = static_cast<int32_t>((rows + p.tile - 1) / p.tile);
  p.units = static_cast<int32_t>((rows + kPiece - 1) / kPiece);
  p.cols = (cols + 7) / 8 * 8;
  p.off_pairs[0] = 0;
  p.off_pairs[1] = p.off_pairs[0] + up(size_t(rows) * 8);
  p.off_counts = p.off_pairs[1] + up(p.passes > 1 ? size_t(rows) * 8 : 0);
  p.off_last = p.off_counts + up(size_t(p.tiles) * 4 << p.bits);
  p.off_sums = p.off_last + up(size_t(vocab) * 4);
  p.bytes = p.off_sums + up(size_t(p.units) * 2 * size_t(p.cols) * 4);
  return p;
}

cudaError_t launch_embedding(const EmbeddingArgs& a, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  return for_types(a.weight_dtype, a.rows_dtype,
                   [&](auto w, auto o) { return launch_embed<decltype(w), decltype(o)>(a, status, stream); });
}

cudaError_t launch_embedding_backward(const EmbeddingArgs& a, void* workspace, int num_sms, int* launches, cudaStream_t stream) {
  (void)num_sms;
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  const EmbeddingPlan p = embedding_plan(a.rows, a.vocab, a.cols);
  char* ws = static_cast<char*>(workspace);
  uint2* pairs[2] = {reinterpret_cast<uint2*>(ws + p.off_pairs[0]), reinterpret_cast<uint2*>(ws + p.off_pairs[1])};
  uint32_t* counts = reinterpret_cast<uint32_t*>(ws + p.off_counts);
  int32_t* last = reinterpret_cast<int32_t*>(ws + p.off_last);
  const uint2* sorted = nullptr;
  *launches = 0;
  for (int pass = 0; pass < p.passes && a.rows > 0; ++pass) {
    const int shift = pass * p.bits;
    cudaError_t e = launch_pdl(k_sort_count, dim3(p.tiles), dim3(kThreads), 0, stream, a, p, sorted, shift, counts,
                               pass == 0 && !a.accumulate ? last : static_cast<int32_t*>(nullptr), status);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_sort_place, dim3(p.tiles), dim3(kThreads), 0, stream, a, p, sorted, shift,
                   static_cast<const uint32_t*>(counts), pairs[pass & 1], status);
    if (e != cudaSuccess) return e;
    *launches += 2;
    sorted = pairs[pass & 1];
  }
  return for_types(a.rows_dtype, a.weight_dtype, [&](auto g, auto w) {
    return launch_gradient<decltype(g), decltype(w)>(a, p, sorted, last, reinterpret_cast<float*>(ws + p.off_sums), launches,
                                                     status, stream);
  });
}

}  // namespace nsm
