// The embedding lookup with scaling, and its gradient by sorted tokens.
//
//   out_r = scale weight[token_r]                       (0 without a token)
//   d_weight[v] (+)= scale sum_{r: token_r = v} d_out_r
//
//   k_embed        a group of lanes per row: reads and writes, nothing else.
//   k_sort_count, k_sort_place
//                  a stable radix sort of (token, row) by digits of the token: a block per tile
//                  counts its first digits; in each pass every block adds up the counts of
//                  the tiles before its own, places its pairs in order, and counts where their next
//                  digits come to lie.  Rows without a token sort behind the others.
//   k_sort_block   the same for few rows, by one block in shared memory.
//   k_embed_sums   pieces of the sorted entries: a group of lanes adds the rows of equal tokens
//                  in ascending order and writes each sum.  It goes on into the next piece for a
//                  token that ends there; of one that reaches further every piece leaves its
//                  sum in the workspace.  Blocks behind those clear the rows of the gradient that no token
//                  asks for.
//   k_embed_join   adds up such tokens' sums.
// No atomic adds a floating-point number: the order of every sum is set by the sizes and the tokens.
//
// Bound by memory where rows are many (the gradient of 65536 x 4096 bf16 rows into 131072: 274 us, of
// which sums and clearing 235 at 6.7 TB/s; the lookup of 65536 x 2048 from 100003: 79 us), and by
// its kernels' latencies where they are few (16384 x 768 into 50257: 37 us; 257 x 769 added to
// 32003 fp32 rows: 12.5 us).
#include "elem.cuh"
#include "launch.cuh"
#include "nsm_internal.h"

#include <algorithm>

namespace nsm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnits = 4;      // of eight columns, per lane of k_embed
constexpr int kMaxBits = 9;    // of a sorting pass's digit
constexpr int kMaxBins = 1 << kMaxBits;
static_assert(kMaxBins == 4 * 128, "scan_bins gives four digits to each of 128 threads");
constexpr int kMaxTiles = 64;
constexpr int kPlaceThreads = 512;
constexpr int kPlaceWarps = kPlaceThreads / 32;
constexpr int kBlockThreads = 1024;  // of k_sort_block
constexpr int kBlockRows = 4096;     // that it takes at most
// Sorted entries of a piece: the most that still make so many warps, 16 for each SM.  Pieces of 32
// whatever the sizes took 53 us for 257 x 769 in place of 13.
constexpr int kMaxPiece = 32, kMinPiece = 4;
// 152 is a GB300's SMs, as a constant: the workspace's size and the order of the sums follow from it.
constexpr int kWantedWarps = 152 * 16;
// Blocks of k_embed at most.  Three are resident on an SM: 65536 rows of 2048 take 79 us with 16 for each and 72
// with 3, of 256 columns 15.7 and 12.6.
constexpr int kEmbedBlocks = 152 * 16;
constexpr int kJoinThreads = 256;
constexpr int kJoinPieces = 8;  // that a block of k_embed_join looks at
// Bytes of rows without a token that a sorting pass clears on the side: about what its time leaves
// room for (12 and 40 MB take as long).
constexpr int64_t kClearBytes = 24 << 20;
constexpr int kClearBlocks = 150;  // that clear beside k_sort_block's first
constexpr int kClear = 8;      // rows of the gradient that a warp looks at

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

// Rows are cut into units of eight columns on the 16-byte grid of where results go: unit u holds
// columns 8 u - lead ... + 8, of which those in [0, cols) exist.
template <typename T>
__device__ __forceinline__ void load_unit(const T* row, int cols, int c0, Eight<T>& r, int* status) {
  load8(row, 0, cols, c0, r, status, NSM_KERNEL_EMBEDDING, NSM_SITE_EMBEDDING);
}
template <typename T>
__device__ __forceinline__ void store_unit(T* row, int cols, int c0, const float (&f)[8], int* status) {
  store8(row, 0, cols, c0, f, status, NSM_KERNEL_EMBEDDING, NSM_SITE_EMBEDDING);
}

// ---------------------------------------------------------------- lookup

// Units of eight columns per lane, one row's after the other's: a group takes kUnits of them at a
// time, and asks for the tokens of its next ones before.
template <typename W, typename O>
__global__ void __launch_bounds__(kThreads) k_embed(const EmbeddingArgs a, int lanes, int slices, int* status) {
  grid_dependency_sync();
  release_dependents();
  const int lane = threadIdx.x & (lanes - 1), groups = kThreads / lanes, cols = static_cast<int>(a.cols);
  const int64_t units = a.rows * slices, step = int64_t(gridDim.x) * groups * kUnits;
  int64_t unit = (int64_t(blockIdx.x) * groups + threadIdx.x / lanes) * kUnits;
  // the row and slice of `unit`, and how far they move with a step
  int row = static_cast<int>(unit / slices), slice = static_cast<int>(unit % slices);
  const int64_t row_step = step / slices;
  const int slice_step = static_cast<int>(step % slices), rows = static_cast<int>(a.rows);
  const auto tokens_of = [&](int r, int s, int (&t)[kUnits]) {  // -1: none
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      t[i] = -1;
      if (r < rows) {
        const int64_t v = token_at(a, r);
        if (v >= 0 && v < a.vocab) t[i] = static_cast<int>(v);
      }
      if (++s == slices) {
        s = 0;
        ++r;
      }
    }
  };
  int token[kUnits];
  if (unit < units) tokens_of(row, slice, token);
  while (unit < units) {
    Eight<W> raw[kUnits];
    int r = row, s = slice;
    uint32_t has = 0;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      O* to = static_cast<O*>(a.rows_out) + r * a.ld_rows;
      if (r < rows && token[i] >= 0) {
        has |= 1u << i;
        load_unit(static_cast<const W*>(a.weight) + token[i] * a.ld_weight, cols, (s * lanes + lane) * 8 - lead_of(to), raw[i], status);
      }
      if (++s == slices) {
        s = 0;
        ++r;
      }
    }
    r = row;
    s = slice;
    unit += step;
    if (unit < units) {
      row += static_cast<int>(row_step);
      slice += slice_step;
      if (slice >= slices) {
        slice -= slices;
        ++row;
      }
      tokens_of(row, slice, token);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (r < rows) {
        O* to = static_cast<O*>(a.rows_out) + r * a.ld_rows;
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (has >> i & 1) {
          raw[i].get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= a.scale;
        }
        store_unit(to, cols, (s * lanes + lane) * 8 - lead_of(to), f, status);
      }
      if (++s == slices) {
        s = 0;
        ++r;
      }
    }
  }
}

// ---------------------------------------------------------------- rows without a token

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

// Clears those of the rows from v0 on, kClear per warp, that no token asks for.
template <typename W>
__device__ __forceinline__ void clear_rows(const EmbeddingArgs& a, const int32_t* last, int64_t v0, int64_t end, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t first = v0 + threadIdx.x / 32 * kClear, v = first + lane;
  const bool none = lane < kClear && v < end && !asked_for(a, last, v);
  for (uint32_t rows = __ballot_sync(0xffffffffu, none); rows; rows &= rows - 1)
    clear_row(static_cast<W*>(a.d_weight) + (first + __ffs(rows) - 1) * a.ld_weight, a.cols, lane, status);
}

// ---------------------------------------------------------------- sorting tokens

// The pair of entry i: from the tokens in the first pass, from the pass before later on.
__device__ __forceinline__ uint2 pair_at(const EmbeddingArgs& a, const uint2* pairs, int64_t i) {
  return pairs ? pairs[i] : make_uint2(key_at(a, i), static_cast<uint32_t>(i));
}

// Notes some row that asks for the token, whichever comes last: see asked_for.
__device__ __forceinline__ void note_row(const EmbeddingArgs& a, int32_t* last, uint32_t key, int64_t row) {
  if (key < a.vocab)
    asm volatile("st.relaxed.gpu.global.s32 [%0], %1;" ::"l"(last + key), "r"(static_cast<int32_t>(row)) : "memory");
}

// counts: of every pass one after the other, tiles x bins each.
__global__ void __launch_bounds__(kThreads)
    k_sort_count(const EmbeddingArgs a, const EmbeddingPlan p, uint32_t* counts, int32_t* last, int* status) {
  __shared__ uint32_t hist[kMaxBins];
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += kThreads) hist[b] = 0;
  __syncthreads();
  grid_dependency_sync();
  release_dependents();
  const int64_t first = int64_t(blockIdx.x) * p.tile, end = min(first + p.tile, a.rows);
  for (int64_t i = first + threadIdx.x; i < end; i += kThreads) {
    if (!row_ok(i < a.rows, status, NSM_SITE_WORKSPACE)) break;
    const uint32_t key = key_at(a, i);
    atomicAdd(&hist[key & (bins - 1)], 1u);
    if (last) note_row(a, last, key, i);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kThreads) {
    counts[int64_t(blockIdx.x) * bins + b] = hist[b];
    for (int pass = 1; pass < p.passes; ++pass) counts[(int64_t(pass) * p.tiles + blockIdx.x) * bins + b] = 0;
  }
}

// Exclusive sums over kMaxBins numbers, four to each of the first 128 threads of a block.
__device__ __forceinline__ void scan_bins(uint32_t (&n)[4], uint32_t* warp_total) {
  const uint32_t own = n[0] + n[1] + n[2] + n[3];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  uint32_t scan = own;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t m = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += m;
  }
  if (lane == 31 && warp < 4) warp_total[warp] = scan;
  __syncthreads();
  uint32_t base = scan - own;
  for (int w = 0; w < min(warp, 4); ++w) base += warp_total[w];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t m = n[d];
    n[d] = base;
    base += m;
  }
}

// The lanes of `live` whose digit is this lane's: a vote per bit (with a match instruction one block
// sorted 16384 rows in 46 us, with votes in 34).
__device__ __forceinline__ uint32_t same_digit(uint32_t live, uint32_t digit, int bits) {
  uint32_t same = live;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(live, digit >> b & 1);
    same &= digit >> b & 1 ? set : ~set;
  }
  return same;
}

// Hands out places in order: each warp's entries [first, end) one group of 32 after the other,
// from next[digit] on.
template <typename Get, typename Put>
__device__ __forceinline__ void place_in_order(uint32_t* next, int first, int end, int shift, int bits, Get get, Put put) {
  const int lane = threadIdx.x & 31;
  for (int i0 = first; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t live = __ballot_sync(0xffffffffu, i < end);
    if (i < end) {
      const uint2 pair = get(i);
      const uint32_t digit = pair.x >> shift & ((1u << bits) - 1);
      const uint32_t same = same_digit(live, digit, bits);
      const uint32_t rank = __popc(same & ((1u << lane) - 1));
      const uint32_t at = next[digit] + rank;
      __syncwarp(live);
      if (rank == 0) next[digit] += __popc(same);
      __syncwarp(live);
      put(at, pair);
    }
  }
}

// Blocks behind the tiles' clear a part of the rows that no token asks for, on the SMs that the
// sort leaves idle.  W: type of the weight's gradient.
template <typename W>
__global__ void __launch_bounds__(kPlaceThreads)
    k_sort_place(const EmbeddingArgs a, const EmbeddingPlan p, const uint2* pairs, int pass, uint32_t* counts, uint2* placed,
                 const int32_t* last, int* status) {
  __shared__ uint32_t next[kPlaceWarps][kMaxBins];  // each warp's next place for a digit
  __shared__ __align__(16) uint32_t part[4][kMaxBins];
  __shared__ uint32_t warp_total[4];
  const int bins = 1 << p.bits, shift = pass * p.bits, tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
  for (int b = tid; b < kPlaceWarps * kMaxBins; b += kPlaceThreads) next[0][b] = 0;
  __syncthreads();
  grid_dependency_sync();
  release_dependents();
  if (blockIdx.x >= p.tiles) {
    clear_rows<W>(a, last, p.clear_first + int64_t(blockIdx.x - p.tiles) * kPlaceWarps * kClear, p.clear_end, status);
    return;
  }
  // the counts of all tiles and of those before this one: four digits and every fourth tile per thread
  const int b0 = (tid & 127) * 4, group = tid / 128;
  const uint32_t* of_pass = counts + int64_t(pass) * p.tiles * bins;
  uint4 all = make_uint4(0, 0, 0, 0), before = all;
  if (b0 < bins) {
#pragma unroll 8
    for (int t = group; t < p.tiles; t += 4) {
      const uint4 n = *reinterpret_cast<const uint4*>(of_pass + int64_t(t) * bins + b0);
      all = make_uint4(all.x + n.x, all.y + n.y, all.z + n.z, all.w + n.w);
      if (t < static_cast<int>(blockIdx.x)) before = make_uint4(before.x + n.x, before.y + n.y, before.z + n.z, before.w + n.w);
    }
  }
  const int64_t tile0 = int64_t(blockIdx.x) * p.tile, tile1 = min(tile0 + p.tile, a.rows);
  const int64_t per_warp = p.tile / kPlaceWarps;  // whole groups of 32
  const int64_t first = min(tile0 + warp * per_warp, tile1), end = min(first + per_warp, tile1);
  for (int64_t i = first + lane; i < end; i += 32) atomicAdd(&next[warp][pair_at(a, pairs, i).x >> shift & (bins - 1)], 1u);
  *reinterpret_cast<uint4*>(&part[group][b0]) = all;
  __syncthreads();
  uint32_t base[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) base[d] = part[0][b0 + d] + part[1][b0 + d] + part[2][b0 + d] + part[3][b0 + d];
  scan_bins(base, warp_total);
  __syncthreads();  // the parts have been read
  *reinterpret_cast<uint4*>(&part[group][b0]) = before;
  __syncthreads();
#pragma unroll
  for (int d = 0; d < 4; ++d) base[d] += part[0][b0 + d] + part[1][b0 + d] + part[2][b0 + d] + part[3][b0 + d];
  __syncthreads();
  if (group == 0) *reinterpret_cast<uint4*>(&part[0][b0]) = make_uint4(base[0], base[1], base[2], base[3]);
  __syncthreads();
  if (tid < bins) {  // a digit per thread: where each warp's own begin
    uint32_t at = part[0][tid];
    for (int w = 0; w < kPlaceWarps; ++w) {
      const uint32_t n = next[w][tid];
      next[w][tid] = at;
      at += n;
    }
  }
  __syncthreads();
  uint32_t* of_next = pass + 1 < p.passes ? counts + int64_t(pass + 1) * p.tiles * bins : nullptr;
  place_in_order(
      next[warp], static_cast<int>(first), static_cast<int>(end), shift, p.bits, [&](int i) { return pair_at(a, pairs, i); },
      [&](uint32_t at, const uint2& pair) {
        if (!row_ok(at < a.rows, status, NSM_SITE_WORKSPACE)) return;
        placed[at] = pair;
        if (of_next) atomicAdd(&of_next[int64_t(at / p.tile) * bins + (pair.x >> (shift + p.bits) & (bins - 1))], 1u);
      });
}

constexpr size_t kBlockSmem = size_t(kBlockRows) * 8 + size_t(kBlockThreads / 32) * kMaxBins * 4;

// All passes for at most kBlockRows rows (one block's instructions bound it: the whole gradient of
// 4096 x 768 takes 27 us with it and 29 with the kernels above, of 16384 x 768 49 and 36), whose token and row fit 32 bits together, by the first
// block.  The others (none where the sums are added to the gradient) note the rows and clear those
// of the gradient from p.clear_end on, asked for or not: k_embed_sums writes later.
template <typename W>
__global__ void __launch_bounds__(kBlockThreads)
    k_sort_block(const EmbeddingArgs a, const EmbeddingPlan p, uint2* sorted, int32_t* last, int* status) {
  extern __shared__ __align__(16) uint32_t block_pairs[];  // two times kBlockRows, then the warps' counts
  uint32_t* from = block_pairs;
  uint32_t* to = block_pairs + kBlockRows;
  constexpr int kAllWarps = kBlockThreads / 32;
  uint32_t* next = block_pairs + 2 * kBlockRows;
  __shared__ __align__(16) uint32_t total[kMaxBins];
  __shared__ uint32_t warp_total[4];
  const int bins = 1 << p.bits, tid = threadIdx.x, warp = tid / 32, lane = tid & 31, rows = static_cast<int>(a.rows);
  grid_dependency_sync();
  release_dependents();
  if (blockIdx.x > 0) {
    for (int i = (blockIdx.x - 1) * kBlockThreads + tid; i < rows; i += (gridDim.x - 1) * kBlockThreads) note_row(a, last, key_at(a, i), i);
    for (int64_t v = p.clear_end + int64_t(blockIdx.x - 1) * kAllWarps + warp; v < a.vocab; v += int64_t(gridDim.x - 1) * kAllWarps)
      clear_row(static_cast<W*>(a.d_weight) + v * a.ld_weight, a.cols, lane, status);
    return;
  }
  const int row_bits = p.row_bits;
  const uint32_t row_mask = (1u << row_bits) - 1;
  for (int i = tid; i < rows; i += kBlockThreads) {
    from[i] = key_at(a, i) << row_bits | i;
  }
  const int warps = min((rows + 31) / 32, kAllWarps);  // that have entries
  const int per_warp = (rows + warps * 32 - 1) / (warps * 32) * 32;
  const int first = min(warp * per_warp, rows), end = min(first + per_warp, rows);
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits + row_bits;
    for (int i = tid; i < warps * kMaxBins; i += kBlockThreads) next[i] = 0;
    __syncthreads();
    for (int i = first + lane; i < end; i += 32) atomicAdd(&next[warp * kMaxBins + (from[i] >> shift & (bins - 1))], 1u);
    __syncthreads();
    if (tid < kMaxBins) {  // a digit per thread: what the warps before each have of it
      uint32_t at = 0;
      for (int w = 0; w < warps; ++w) {
        const uint32_t n = next[w * kMaxBins + tid];
        next[w * kMaxBins + tid] = at;
        at += n;
      }
      total[tid] = at;
    }
    __syncthreads();
    uint32_t n[4] = {0, 0, 0, 0};
    if (tid < kMaxBins / 4) *reinterpret_cast<uint4*>(n) = reinterpret_cast<const uint4*>(total)[tid];
    scan_bins(n, warp_total);
    if (tid < kMaxBins / 4) reinterpret_cast<uint4*>(total)[tid] = make_uint4(n[0], n[1], n[2], n[3]);
    __syncthreads();
    place_in_order(
        next + warp * kMaxBins, first, end, shift, p.bits, [&](int i) { return make_uint2(from[i], 0); },
        [&](uint32_t at, const uint2& pair) {
          at += total[pair.x >> shift & (bins - 1)];
          if (!row_ok(at < a.rows, status, NSM_SITE_WORKSPACE)) return;
          to[at] = pair.x;
        });
    __syncthreads();
    uint32_t* other = from;
    from = to;
    to = other;
  }
  for (int i = tid; i < rows; i += kBlockThreads) sorted[i] = make_uint2(from[i] >> row_bits, from[i] & row_mask);
}

// ---------------------------------------------------------------- sums

template <typename W>
__device__ __forceinline__ W* weight_row(const EmbeddingArgs& a, uint32_t token) {
  return static_cast<W*>(a.d_weight) + int64_t(token) * a.ld_weight;
}

// Unit u of a token's row: its first column.
template <typename W>
__device__ __forceinline__ int unit_column(const EmbeddingArgs& a, uint32_t token, int u) {
  return u * 8 - lead_of(weight_row<W>(a, token));
}

// The columns that the gradient holds already, where the sums are added to them.
template <typename W>
__device__ __forceinline__ void load_old(const EmbeddingArgs& a, uint32_t token, int u, Eight<W>& old, int* status) {
  if (row_ok(token < a.vocab, status, NSM_SITE_EMBEDDING))
    load_unit(static_cast<const W*>(weight_row<W>(a, token)), static_cast<int>(a.cols), unit_column<W>(a, token, u), old, status);
}

template <typename W, bool kAccumulate>
__device__ __forceinline__ void write_sum(const EmbeddingArgs& a, uint32_t token, int u, const float (&sum)[8], const Eight<W>& old,
                                          int* status) {
  if (!row_ok(token < a.vocab, status, NSM_SITE_EMBEDDING)) return;
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = a.scale * sum[e];
  if (kAccumulate) {
    float g[8];
    old.get(g);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += g[e];
  }
  store_unit(weight_row<W>(a, token), static_cast<int>(a.cols), unit_column<W>(a, token, u), f, status);
}

// A piece's two sums in the workspace, unit after unit, of tokens in more than two pieces: of the
// one that ends here, and of the one that goes on behind this piece.
__device__ __forceinline__ float* piece_sum(const EmbeddingPlan& p, float* sums, int64_t piece, int which) {
  return sums + (piece * 2 + which) * p.cols;
}

__device__ __forceinline__ void keep_sum(float* sums, int u, const float (&sum)[8], int* status) {
  Eight<float> r;
  r.set(sum);
  if (row_ok(on_16_bytes(sums), status, NSM_SITE_WORKSPACE)) r.store(sums + u * 8);
}

__device__ __forceinline__ bool token_is(const uint2* pairs, int64_t i, int64_t rows, uint32_t token) {
  return i >= 0 && i < rows && pairs[i].x == token;
}

// G: type of the rows' gradients, W: of the weight's.  The block's groups take pieces that follow
// one another, of one slice of the columns; their pairs, with those of a piece and an entry more on
// either side, are read to shared memory first.
template <typename G, typename W, bool kAccumulate>
__global__ void __launch_bounds__(kThreads, !kAccumulate && sizeof(G) == 2 ? 4 : 2)
    k_embed_sums(const EmbeddingArgs a, const EmbeddingPlan p, const uint2* pairs, const int32_t* last, float* sums,
                 int lanes, int64_t sum_blocks, int blocks_per_slice, int* status) {
  extern __shared__ __align__(16) uint2 near[];
  grid_dependency_sync();
  release_dependents();
  if (blockIdx.x >= sum_blocks) {
    clear_rows<W>(a, last, p.clear_first + (blockIdx.x - sum_blocks) * kWarps * kClear, p.clear_end, status);
    return;
  }
  const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = kThreads / lanes;
  const int64_t piece0 = int64_t(blockIdx.x % blocks_per_slice) * groups;
  const int u = static_cast<int>(blockIdx.x / blocks_per_slice) * lanes + lane;
  const int halo = p.piece + 1, total = groups * p.piece + 2 * halo;
  const int64_t near0 = piece0 * p.piece - halo;
  const uint32_t none = static_cast<uint32_t>(a.vocab);
  for (int i = threadIdx.x; i < total; i += kThreads) {
    const int64_t j = near0 + i;
    near[i] = j >= 0 && j < a.rows ? pairs[j] : make_uint2(none, 0);
  }
  __syncthreads();
  const int64_t piece = piece0 + group;
  const int first = halo + group * p.piece, end = first + p.piece;
  const uint32_t first_token = near[first].x, last_token = near[end - 1].x;
  if (first_token >= none) return;
  // a token of the piece before that ends here is that piece's, unless it began further back
  const bool from_before = near[first - 1].x == first_token;
  const bool joined = from_before && (near[first - halo].x == first_token || near[end].x == first_token);
  int j = first;
  if (from_before && !joined)
    while (j < end && near[j].x == first_token) ++j;
  // a token that begins here and ends in the next piece is added up whole
  int until = end;
  const bool goes_on = last_token < none && near[end].x == last_token;
  const bool whole = goes_on && !(from_before && last_token == first_token) && near[end + p.piece].x != last_token;
  if (whole)
    while (near[until].x == last_token) ++until;

  constexpr int kAhead = kAccumulate || sizeof(G) == 4 ? 4 : 8;
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool of_before = joined;  // the sum is of a token that began before this piece
  for (; j < until; j += kAhead) {
    if (near[j].x >= none) break;
    Eight<G> raw[kAhead];
    Eight<W> old[kAccumulate ? kAhead : 1];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint2 pair = near[min(j + i, until - 1)];
      if (j + i >= until || pair.x >= none || !row_ok(pair.y < a.rows, status, NSM_SITE_EMBEDDING)) continue;
      load_unit(static_cast<const G*>(a.rows_in) + int64_t(pair.y) * a.ld_rows, static_cast<int>(a.cols), unit_column<W>(a, pair.x, u), raw[i], status);
      if (kAccumulate && near[j + i + 1].x != pair.x) load_old<W>(a, pair.x, u, old[i], status);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (j + i >= until) break;
      const uint32_t token = near[j + i].x;
      if (token >= none) break;
      float f[8];
      raw[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += f[e];
      if (near[j + i + 1].x == token) continue;
      if (of_before) keep_sum(piece_sum(p, sums, piece, 0), u, sum, status);
      else write_sum<W, kAccumulate>(a, token, u, sum, old[kAccumulate ? i : 0], status);
      of_before = false;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0.f;
    }
  }
  if (goes_on && !whole) keep_sum(piece_sum(p, sums, piece, 1), u, sum, status);
}

// Tokens of more than two pieces that begin in one of the block's: their sums, the block's groups
// a part of the pieces each, then the groups' in order.  A block looks at every `blocks`-th piece, so
// that the pieces of frequent tokens, which follow one another, are different blocks'.
template <typename W, bool kAccumulate>
__global__ void __launch_bounds__(kJoinThreads)
    k_embed_join(const EmbeddingArgs a, const EmbeddingPlan p, const uint2* pairs, float* sums, int lanes, int slices,
                 int blocks, int* status) {
  __shared__ __align__(16) float part[kJoinThreads * 8], total[256];
  grid_dependency_sync();
  release_dependents();
  const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x / lanes, groups = kJoinThreads / lanes;
  const int64_t piece0 = blockIdx.x / slices;
  const int u = static_cast<int>(blockIdx.x % slices) * lanes + lane;
  const int64_t rows = a.rows;
  // every warp finds the same ones
  const int64_t mine = piece0 + int64_t(threadIdx.x & 31) * blocks, end = (mine + 1) * p.piece;
  bool begins = false;
  if ((threadIdx.x & 31) < kJoinPieces && end + p.piece < rows) {
    const uint32_t token = pairs[end - 1].x, next = pairs[end].x, far = pairs[end + p.piece].x;
    const uint32_t back = mine > 0 ? pairs[end - p.piece - 1].x : static_cast<uint32_t>(a.vocab);
    begins = (token < a.vocab) & (next == token) & (far == token) & (back != token);
  }
  for (uint32_t some = __ballot_sync(0xffffffffu, begins); some; some &= some - 1) {
    const int64_t begin = piece0 + int64_t(__ffs(some) - 1) * blocks;
    const uint32_t token = pairs[(begin + 1) * p.piece - 1].x;
    // it fills whole pieces from begin + 1 on, and ends in the one behind them
    int64_t last = begin + 1;
    for (int full = kJoinThreads; full == kJoinThreads; last += full)
      full = __syncthreads_count(token_is(pairs, (last + 1 + threadIdx.x) * p.piece, rows, token));
    const int64_t count = last + 1 - begin;
    const int64_t from = begin + count * group / groups, to = begin + count * (group + 1) / groups;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    constexpr int kAhead = 4;
    for (int64_t w0 = from; w0 < to; w0 += kAhead) {
      Eight<float> f[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (w0 + i < to && row_ok(u * 8 + 8 <= p.cols, status, NSM_SITE_WORKSPACE)) f[i].load_written(piece_sum(p, sums, w0 + i, w0 + i < last ? 1 : 0) + u * 8);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (w0 + i >= to) break;
        float g[8];
        f[i].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += g[e];
      }
    }
    // a column per thread over the groups
    float* own = part + (group * lanes + lane) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) own[e] = sum[e];
    __syncthreads();
    if (threadIdx.x < lanes * 8) {
      float s = 0.f;
      for (int g = 0; g < groups; ++g) s += part[g * lanes * 8 + threadIdx.x];
      total[threadIdx.x] = s;
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = total[lane * 8 + e];
      Eight<W> old;
      if (kAccumulate) load_old<W>(a, token, u, old, status);
      write_sum<W, kAccumulate>(a, token, u, sum, old, status);
    }
    __syncthreads();
  }
}

// How a row of `cols` columns is cut: lanes that share it, a power of two up to a warp, each with a
// unit at a time, and slices of so many units.  Rows that do not begin on 16-byte boundaries have up
// to seven columns' room more.
struct Cut {
  int lanes, slices;
};
Cut cut_rows(int64_t cols, bool aligned) {
  const int64_t room = cols + (aligned ? 0 : 7);
  int lanes = 1;
  while (lanes < 32 && lanes * 8 < room) lanes *= 2;
  return {lanes, static_cast<int>((room + lanes * 8 - 1) / (lanes * 8))};
}

bool rows_aligned(const void* p, int64_t ld, int dtype) {
  const int64_t size = dtype == NSM_FP32 ? 4 : 2;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * size % 16 == 0;
}

int blocks(int64_t n) { return static_cast<int>(std::min<int64_t>(std::max<int64_t>(n, 1), INT32_MAX)); }

template <typename W, typename O>
cudaError_t launch_embed(const EmbeddingArgs& a, int* status, cudaStream_t stream) {
  const Cut cut = cut_rows(a.cols, rows_aligned(a.rows_out, a.ld_rows, a.rows_dtype));
  const int64_t per_block = int64_t(kThreads / cut.lanes) * kUnits;
  const dim3 grid(blocks(std::min<int64_t>((a.rows * cut.slices + per_block - 1) / per_block, kEmbedBlocks)));
  return launch_pdl(k_embed<W, O>, grid, dim3(kThreads), 0, stream, a, cut.lanes, cut.slices, status);
}

template <typename G, typename W, bool kAccumulate>
cudaError_t launch_sums(const EmbeddingArgs& a, const EmbeddingPlan& p, const uint2* pairs, const int32_t* last, float* sums,
                        int* launches, int* status, cudaStream_t stream) {
  const Cut cut = cut_rows(a.cols, rows_aligned(a.d_weight, a.ld_weight, a.weight_dtype));
  const int groups = kThreads / cut.lanes;
  const int per_slice = (p.units + groups - 1) / groups;
  const int64_t sum_blocks = int64_t(per_slice) * cut.slices;
  const int64_t left = kAccumulate ? 0 : std::max<int64_t>(p.clear_end - p.clear_first, 0);
  const int64_t clear = (left + kWarps * kClear - 1) / (kWarps * kClear);
  const size_t smem = size_t(groups * p.piece + 2 * (p.piece + 1)) * sizeof(uint2);
  if (sum_blocks + clear > 0) {
    const cudaError_t e = launch_pdl(k_embed_sums<G, W, kAccumulate>, dim3(blocks(sum_blocks + clear)), dim3(kThreads), smem,
                                     stream, a, p, pairs, last, sums, cut.lanes, sum_blocks, per_slice, status);
    ++*launches;
    if (e != cudaSuccess) return e;
  }
  if (p.units <= 2) return cudaSuccess;
  ++*launches;
  const int join = (p.units + kJoinPieces - 1) / kJoinPieces;
  return launch_pdl(k_embed_join<W, kAccumulate>, dim3(blocks(int64_t(join) * cut.slices)), dim3(kJoinThreads), 0, stream, a, p, pairs,
                    sums, cut.lanes, cut.slices, join, status);
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
  int bits = 2;
  while (bits < 62 && vocab >> bits) ++bits;  // keys 0 ... vocab
  p.passes = (bits + kMaxBits - 1) / kMaxBits;
  p.bits = (bits + p.passes - 1) / p.passes;
  const int64_t step = 32 * kPlaceWarps;
  p.tile = static_cast<int32_t>(std::max<int64_t>(1024, ((rows + kMaxTiles - 1) / kMaxTiles + step - 1) / step * step));
  p.tiles = static_cast<int32_t>((rows + p.tile - 1) / p.tile);
  // the longest pieces that still make some 16 warps for each SM
  const Cut cut = cut_rows(cols, true), wide = cut_rows(cols, false);
  const int32_t longest = std::min(kMaxPiece, 8 * cut.lanes);  // a block's pairs are 16 KB and little more at most
  p.piece = longest;
  while (p.piece > kMinPiece && (rows + p.piece - 1) / p.piece * cut.slices * cut.lanes < int64_t(kWantedWarps) * 32) p.piece /= 2;
  p.units = static_cast<int32_t>((rows + p.piece - 1) / p.piece);
  p.cols = std::max(int64_t(cut.lanes) * cut.slices, int64_t(wide.lanes) * wide.slices) * 8;
  p.off_pairs[0] = 0;
  p.off_pairs[1] = p.off_pairs[0] + up(size_t(rows) * 8);
  p.off_counts = p.off_pairs[1] + up(p.passes > 1 ? size_t(rows) * 8 : 0);
  // Room for the most tiles and pieces that any smaller number of rows has, where their lengths grow there are
  // fewer: the bytes never fall as rows grow, and a workspace for the largest batch serves all.  A length below
  // the longest is taken only while pieces of twice that length are too few, `few` at most.
  const int64_t tiles = std::min<int64_t>(kMaxTiles, (rows + 1023) / 1024);
  const int64_t few = (int64_t(kWantedWarps) * 32 - 1) / (int64_t(cut.slices) * cut.lanes);
  const int64_t units = std::max(std::min((rows + kMinPiece - 1) / kMinPiece, 2 * few), (rows + longest - 1) / longest);
  p.off_last = p.off_counts + up(size_t(p.passes) * size_t(tiles) * 4 << p.bits);
  p.off_sums = p.off_last + up(size_t(vocab) * 4);
  p.bytes = p.off_sums + up(size_t(units) * 2 * size_t(p.cols) * 4);
  return p;
}

cudaError_t launch_embedding(const EmbeddingArgs& a, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  return for_types(a.weight_dtype, a.rows_dtype,
                   [&](auto w, auto o) { return launch_embed<decltype(w), decltype(o)>(a, status, stream); });
}

cudaError_t launch_embedding_backward(const EmbeddingArgs& a, void* workspace, int* launches, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  EmbeddingPlan p = embedding_plan(a.rows, a.vocab, a.cols);
  char* ws = static_cast<char*>(workspace);
  uint2* pairs[2] = {reinterpret_cast<uint2*>(ws + p.off_pairs[0]), reinterpret_cast<uint2*>(ws + p.off_pairs[1])};
  uint32_t* counts = reinterpret_cast<uint32_t*>(ws + p.off_counts);
  int32_t* last = reinterpret_cast<int32_t*>(ws + p.off_last);
  const uint2* sorted = nullptr;
  *launches = 0;
  int32_t* noted = a.accumulate ? nullptr : last;
  // rows of the gradient whose writing takes about as long as one of the sort's kernels
  const int64_t aside = a.accumulate ? 0 : std::min<int64_t>(kClearBytes / (a.cols * (a.weight_dtype == NSM_FP32 ? 4 : 2)) + 1, a.vocab);
  p.clear_first = 0;
  p.clear_end = a.vocab;
  int key_bits = 1;
  while (a.vocab >> key_bits) ++key_bits;
  p.row_bits = std::min(32 - key_bits, 12);
  static_assert(kBlockRows == 1 << 12, "row_bits");
  cudaError_t e = cudaSuccess;
  if (a.rows > 0 && a.rows <= int64_t(1) << p.row_bits) {
    p.clear_end = a.vocab - aside;
    const int clear = static_cast<int>(std::min<int64_t>((aside + kBlockThreads / 32 - 1) / (kBlockThreads / 32), kClearBlocks));
    e = for_types(a.weight_dtype, NSM_FP32, [&](auto w, auto) {
      static std::atomic<uint64_t> done{0};
      const cudaError_t set = set_smem_once(k_sort_block<decltype(w)>, kBlockSmem, done);
      if (set != cudaSuccess) return set;
      return launch_pdl(k_sort_block<decltype(w)>, dim3(1 + clear), dim3(kBlockThreads), kBlockSmem, stream, a, p, pairs[0], noted, status);
    });
    *launches = 1;
    sorted = pairs[0];
  } else if (a.rows > 0) {
    e = launch_pdl(k_sort_count, dim3(p.tiles), dim3(kThreads), 0, stream, a, p, counts, noted, status);
    for (int pass = 0; pass < p.passes && e == cudaSuccess; ++pass) {
      p.clear_end = std::min(p.clear_first + aside, a.vocab);
      const int64_t clear = p.clear_end - p.clear_first;
      const dim3 grid(p.tiles + static_cast<int>((clear + kPlaceWarps * kClear - 1) / (kPlaceWarps * kClear)));
      e = for_types(a.weight_dtype, NSM_FP32, [&](auto w, auto) {
        return launch_pdl(k_sort_place<decltype(w)>, grid, dim3(kPlaceThreads), 0, stream, a, p, sorted, pass, counts, pairs[pass & 1],
                          static_cast<const int32_t*>(last), status);
      });
      sorted = pairs[pass & 1];
      p.clear_first = p.clear_end;
    }
    p.clear_end = a.vocab;
    *launches = 1 + p.passes;
  }
  if (e != cudaSuccess) return e;
  return for_types(a.rows_dtype, a.weight_dtype, [&](auto g, auto w) {
    float* sums = reinterpret_cast<float*>(ws + p.off_sums);
    return a.accumulate ? launch_sums<decltype(g), decltype(w), true>(a, p, sorted, last, sums, launches, status, stream)
                        : launch_sums<decltype(g), decltype(w), false>(a, p, sorted, last, sums, launches, status, stream);
  });
}

}  // namespace nsm
