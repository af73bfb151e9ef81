// Log probabilities of given tokens, with entropy and top alternatives, and their gradient.
//
//   y = x / t, lse = log sum exp(y), q = exp(y - lse), logprob = y_token - lse,
//   entropy = -sum q log q, the k largest logits; gradient of w logprob + h entropy:
//   (w (1[v = token] - q_v) - h q_v (log q_v + entropy)) / t
//
//   k_logprobs           forward: a block per row, a cluster of blocks where rows are few; one
//                        pass, alternatives from groups that can hold one.  Bound by the read:
//                        8192 x 131072 bf16 297 us (7.2 TB/s), with 64 alternatives 360, with 128
//                        420.
//   k_logprobs_resident  forward and backward in one pass over memory, the row in shared memory:
//                        8192 x 32768 bf16 158 us, 8192 x 50257 244, 8192 x 131072 (four blocks
//                        a row) 627: the rate of a copy, 6.8 TB/s read and written.
//   k_logprobs_backward  pieces of rows from saved statistics: 8192 x 131072 677 us (6.3 TB/s).
//   k_logprobs_short     a warp per row of at most 256 vectors, every direction: 16384 x 1000
//                        forward 8.6 us, forward and backward 19.
#include "vocab_rows.cuh"

namespace nsm {
namespace {

// Places for candidates: 128 vectors of eight and a row's ragged first and last one, which two
// threads have beside the whole vectors that they begin with.
constexpr int kTopCandidates = 1024 + 16;

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
  int32_t count[2][kTopWarps];
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

// Leaves of the candidates the k largest and at most 32 more: a bound on whole keys, which are
// distinct, by those of their bits that differ at all.  Every thread calls it, behind a barrier, with
// n > k + 32; the number left.
__device__ __forceinline__ int cut_candidates(TopShared& sh, int n, int k) {
  constexpr int kOwn = (kTopCandidates + kTopThreads - 1) / kTopThreads;
  const int tid = threadIdx.x;
  const uint64_t one = sh.cand[0];
  uint64_t mine[kOwn], differ = 0;  // 0 is no candidate's key
#pragma unroll
  for (int u = 0; u < kOwn; ++u) {
    mine[u] = tid + u * kTopThreads < n ? sh.cand[tid + u * kTopThreads] : 0;
    if (mine[u] != 0) differ |= mine[u] ^ one;
  }
  differ = static_cast<uint64_t>(__reduce_or_sync(~0u, static_cast<uint32_t>(differ >> 32))) << 32 |
           __reduce_or_sync(~0u, static_cast<uint32_t>(differ));
  if ((tid & 31) == 0) sh.best[tid >> 5] = differ;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTopWarps; ++w) differ |= sh.best[w];
  uint64_t bound = one & ~differ;
#pragma unroll 1
  for (int reach = n, step = 0; reach > k + 32 && differ != 0; step ^= 1) {
    const uint64_t bit = 1ull << (63 - __clzll(differ)), test = bound | bit;
    differ ^= bit;
    int c = 0;
#pragma unroll
    for (int u = 0; u < kOwn; ++u) c += mine[u] >= test;
    c = __reduce_add_sync(~0u, c);
    if ((tid & 31) == 0) sh.count[step][tid >> 5] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int w = 0; w < kTopWarps; ++w) c += sh.count[step][w];
    if (c >= k) {
      bound = test;
      reach = c;
    }
  }
  if (tid == 0) sh.ncand = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kOwn; ++u)
    if (mine[u] != 0 && mine[u] >= bound) sh.cand[atomicAdd(&sh.ncand, 1)] = mine[u];
  __syncthreads();
  return sh.ncand;
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
    // A few more threads than k cost less than the steps that would tell them apart, and up to 32
    // more less than their logits among the candidates (2048 x 50257 bf16, 64 alternatives: 57 us,
    // 61 with k + 8 more).  But three quarters of the threads at most: a bound that all reach is
    // none, and one that nearly all reach has more logits above it than the candidates' places (512
    // x 131072 bf16, 128 alternatives: 6.9 ms where rows were read once per place, 0.04 with this).
    // And no more threads than the places hold whole vectors of, as where the logits fall from the
    // first token on (the same rows falling, 100 alternatives: 5.4 ms and 0.04).
    constexpr int kVectors = kTopCandidates / kVec - 2, kThreads = 3 * kTopThreads / 4;
    constexpr int kMost = kVectors < kThreads ? kVectors : kThreads;
    static_assert(kMost >= kTopMaxK, "k threads may reach the bound");
    const TopBound t = top_bound<T>(key, vec, k, min(min(2 * k + 8, k + 32), kMost));
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
      if (at < kTopCandidates) sh.cand[at] = full_key(Elem<T>::to_float(row.at(row.first(i) + e)), row.first(i) + e);
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
  int ncand = sh.ncand;
  if (nlist <= kTopList && ncand <= kTopCandidates) {
    // Placing takes n^2 comparisons.  Rows of noise have some 2 k candidates; rows that fall from
    // token to token have whole vectors of them (608 x 9001 bf16, 128 alternatives: 20 us of noise,
    // falling 122 without this and 24 with it).
    if (ncand > 3 * k + 64) ncand = cut_candidates(sh, ncand, k);
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
    // closed up, in kTopCandidates >= kMaxCluster kTopMaxK places
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
  if (mine) out.put(token, Elem<T>::from_float(at_token()));
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
  const float x_token = token >= 0 ? Elem<T>::to_float(row.at(token)) : kNegInf;
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
  const Totals t = row_totals<ENT, NT>(a, c, totals, ctas, status, NSM_KERNEL_LOGPROBS, x_token);
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
__global__ void __launch_bounds__(NT) k_logprobs_resident(const LogprobArgs g, int ahead, int* status) {
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
  if (threadIdx.x == 0 && r + ahead < g.v.rows)
    slab.prefetch(Row<T>(static_cast<T*>(const_cast<void*>(g.v.logits)) + (r + ahead) * g.v.ld, vocab, status, NSM_KERNEL_LOGPROBS), rank, ctas);
  const int64_t token64 = g.tokens ? load_index(g.tokens, g.tokens_wide, r) : -1;
  const int token = token64 < 0 || token64 >= vocab ? -1 : static_cast<int>(token64);
  const float x_token = token >= 0 ? Elem<T>::to_float(row.at(token)) : kNegInf;
  const float w = g.d_logprob && token >= 0 ? g.d_logprob[r] : 0.f;
  const float h = ENT && g.d_entropy ? g.d_entropy[r] : 0.f;
  Sums a;
  auto add = [&](int, const uint4& raw, bool) { add_vec<T, ENT>(a, raw, c); };
#pragma unroll 1
  for (int q = 0; q < kSlabChunks; ++q) {
    slab.wait(q);
    slab.chunk(q, add);
  }
  slab.ragged(add);  // in the loop this costs the first passes more than it is (254 us for 244)
  const Totals t = row_totals<ENT, NT>(a, c, totals, ctas, status, NSM_KERNEL_LOGPROBS, x_token);
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
    const float x_token = mine ? Elem<T>::to_float(row.at(token)) : kNegInf;
    const TokenGradient k = token_gradient(w, h, s, low, c, inv_t);
    store_token_gradients<T, ENT>(row, out, part, k, token, mine, c, [&](auto&& use) { for_vectors<NT>(row, part, use); },
                                  [&] { return gradient_at_token(w, h, s, low, x_token, inv_t); });
  }
}

// ---------------------------------------------------------------- short rows

// Leaves of a warp's n candidates the k largest and at most 32 more: a bound on whole keys, which
// are distinct, by those of their bits that differ at all.  The number left.
__device__ __forceinline__ int short_cut(uint64_t* cand, int n, int k) {
  const int lane = threadIdx.x & 31;
  const uint64_t one = cand[0];
  uint64_t differ = 0;
#pragma unroll 4
  for (int j = lane; j < n; j += 32) differ |= cand[j] ^ one;
  differ = static_cast<uint64_t>(__reduce_or_sync(~0u, static_cast<uint32_t>(differ >> 32))) << 32 |
           __reduce_or_sync(~0u, static_cast<uint32_t>(differ));
  uint64_t bound = one & ~differ;
#pragma unroll 1
  for (int reach = n; reach > k + 32 && differ != 0;) {
    const uint64_t bit = 1ull << (63 - __clzll(differ)), test = bound | bit;
    differ ^= bit;
    int c = 0;
#pragma unroll 4
    for (int j = lane; j < n; j += 32) c += cand[j] >= test;
    c = __reduce_add_sync(~0u, c);
    if (c >= k) {
      bound = test;
      reach = c;
    }
  }
  int left = 0;  // a candidate moves to the front, over ones that have been read
#pragma unroll 1
  for (int from = 0; from < n; from += 32) {
    const uint64_t mine = from + lane < n ? cand[from + lane] : 0;
    const uint32_t stay = __ballot_sync(~0u, from + lane < n && mine >= bound);
    __syncwarp();
    if (stay >> lane & 1) cand[left + __popc(stay & ((1u << lane) - 1u))] = mine;
    left += __popc(stay);
    __syncwarp();
  }
  return left;
}

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
  int n = *count;
  // Placing takes n^2 comparisons.  A row of little more vectors than alternatives has all its
  // logits here, and one of whole vectors of its largest logits hundreds: 2000 x 1000 bf16 with 64
  // alternatives took 506 us without this, 29 with it.
  if (n > k + 64) n = short_cut(cand, n, k);
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

// With alternatives five blocks a SM: left to itself the compiler takes 80 registers for N = 8, and
// 2000 x 2000 bf16 with 20 alternatives 12.1 us, 10.8 with up to 102.
template <typename T, bool ENT, int MODE, int N>
__global__ void __launch_bounds__(32 * kShortWarps, MODE == kShortTop ? 5 : 0) k_logprobs_short(const LogprobArgs g, int* status) {
  __shared__ uint64_t cand[kShortWarps][MODE == kShortTop ? kTopCandidates : 1];
  __shared__ int ncand[kShortWarps];
  grid_dependency_sync();
  release_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vocab = g.v.vocab;
  const float c = g.v.c, inv_t = g.v.inv_t;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kShortWarps + warp; r < g.v.rows;
       r += static_cast<int64_t>(gridDim.x) * kShortWarps) {
    const Row<T> row(static_cast<T*>(const_cast<void*>(g.v.logits)) + r * g.v.ld, vocab, status, NSM_KERNEL_LOGPROBS);
    const Part part = part_of(row, 0, 1);
    ShortRow<T, N> x;
    x.load(row, part);
    const int64_t token64 = g.tokens ? load_index(g.tokens, g.tokens_wide, r) : -1;
    const int token = token64 < 0 || token64 >= vocab ? -1 : static_cast<int>(token64);
    const float x_token = token >= 0 ? Elem<T>::to_float(row.at(token)) : kNegInf;
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
        if (32 * u < row.nvec) add_vec<T, ENT>(a, x.raw[u], c);
      s = row_logprob<ENT>(warp_totals<ENT>(a, c), inv_t);
      if (lane == 0) write_logprob<ENT>(g, r, s, token, x_token, inv_t);
      if constexpr (MODE == kShortTop)
        short_top<T, N>(row, x.raw, g.k, s, inv_t, g.top_logprob + r * g.k, g.top_index + r * g.k, cand[warp], &ncand[warp]);
    }
    if constexpr (MODE == kShortBoth || MODE == kShortBackward) {
      const Row<T> out(static_cast<T*>(g.v.d_logits) + r * g.v.ldd, vocab, status, NSM_KERNEL_LOGPROBS);
      const float w = g.d_logprob && token >= 0 ? g.d_logprob[r] : 0.f;
      const float h = ENT && g.d_entropy ? g.d_entropy[r] : 0.f;
      const TokenGradient k = token_gradient(w, h, s, low, c, inv_t);
      __syncwarp();  // in place: every lane has read the token's logit
      x.store(row, out, part, k.zero, [&](const uint4& v) { return gradient_vec<T, ENT>(v, k.ref, c, k.log2_s, k.ca, k.cb); });
      if (!k.zero && token >= 0 && ((token + row.lead) / Elem<T>::kVec & 31) == lane)
        out.put(token, Elem<T>::from_float(gradient_at_token(w, h, s, low, x_token, inv_t)));
    }
  }
}

// ---------------------------------------------------------------- launches

template <typename T, bool ENT, int MODE>
cudaError_t launch_logprobs_short(int n, const LogprobArgs& a, int* status, cudaStream_t stream) {
  auto* launch = n == 2   ? Launch<k_logprobs_short<T, ENT, MODE, 2>>::run
                 : n == 4 ? Launch<k_logprobs_short<T, ENT, MODE, 4>>::run
                          : Launch<k_logprobs_short<T, ENT, MODE, 8>>::run;
  return launch(32 * kShortWarps, short_blocks(a.v.rows), 1, 0, 0, stream, a, status);
}

template <typename T>
cudaError_t launch_logprobs_t(const LogprobArgs& a, int* status, cudaStream_t stream) {
  const int nvec = vectors_of<T>(a.v.vocab), n = short_for(nvec);
  if (n > 0) {
    const bool ent = a.d_entropy || a.entropy;
    if (a.in_lse)
      return ent ? launch_logprobs_short<T, true, kShortBackward>(n, a, status, stream)
                 : launch_logprobs_short<T, false, kShortBackward>(n, a, status, stream);
    if (a.v.d_logits)
      return ent ? launch_logprobs_short<T, true, kShortBoth>(n, a, status, stream)
                 : launch_logprobs_short<T, false, kShortBoth>(n, a, status, stream);
    if (a.k > 0)
      return ent ? launch_logprobs_short<T, true, kShortTop>(n, a, status, stream)
                 : launch_logprobs_short<T, false, kShortTop>(n, a, status, stream);
    return ent ? launch_logprobs_short<T, true, kShortForward>(n, a, status, stream)
               : launch_logprobs_short<T, false, kShortForward>(n, a, status, stream);
  }
  if (a.in_lse) {
    const int threads = backward_threads(nvec), pieces = pieces_for(a.v.rows, nvec, 4 * threads, threads);
    auto* launch = threads == 64
                       ? (a.d_entropy ? Launch<k_logprobs_backward<T, true, 64>>::run : Launch<k_logprobs_backward<T, false, 64>>::run)
                       : (a.d_entropy ? Launch<k_logprobs_backward<T, true, 256>>::run : Launch<k_logprobs_backward<T, false, 256>>::run);
    return launch(threads, std::min<int64_t>(a.v.rows * pieces, 1 << 30), 1, 0, 0, stream, a, pieces, status);
  }
  if (a.v.d_logits) {
    const Resident r = resident_for(a.v.rows, nvec, 76 << 10);
    if (r.ctas) {
      const bool ent = a.d_entropy || a.entropy;
      auto* launch =
          r.threads == 64    ? (ent ? Launch<k_logprobs_resident<T, true, 64>>::run : Launch<k_logprobs_resident<T, false, 64>>::run)
          : r.threads == 128 ? (ent ? Launch<k_logprobs_resident<T, true, 128>>::run : Launch<k_logprobs_resident<T, false, 128>>::run)
                             : (ent ? Launch<k_logprobs_resident<T, true, 256>>::run : Launch<k_logprobs_resident<T, false, 256>>::run);
      const size_t slab = slab_bytes(nvec, r.ctas);
      return launch(r.threads, a.v.rows * r.ctas, r.ctas, slab, kSlabMost, stream, a, rows_ahead(slab, r.threads, r.ctas), status);
    }
  }
  const int threads = a.v.d_logits || a.k > 0 ? 256 : forward_threads(nvec);
  const int ctas = cluster_for(a.v.rows, nvec, threads);
  const int64_t grid = a.v.rows * ctas;
  if (a.v.d_logits) {
    auto* launch = a.d_entropy || a.entropy ? Launch<k_logprobs<T, true, false, true, 256>>::run
                                            : Launch<k_logprobs<T, false, false, true, 256>>::run;
    return launch(threads, grid, ctas, 0, 0, stream, a, 0, status);
  }
  if (a.k == 0) {
    auto* launch =
        threads == 64 ? (a.entropy ? Launch<k_logprobs<T, true, false, false, 64>>::run : Launch<k_logprobs<T, false, false, false, 64>>::run)
                      : (a.entropy ? Launch<k_logprobs<T, true, false, false, 128>>::run : Launch<k_logprobs<T, false, false, false, 128>>::run);
    return launch(threads, grid, ctas, 0, 0, stream, a, 0, status);
  }
  const int batches = ((nvec + ctas - 1) / ctas + 4 * kTopThreads - 1) / (4 * kTopThreads);
  int shift = 0;
  while (((batches + (1 << shift) - 1) >> shift) > kTopGroups) ++shift;
  const size_t smem = (ctas > 1 ? size_t(ctas) * a.k * 8 : 0) +
                      size_t((batches + (1 << shift) - 1) >> shift) * kTopThreads * sizeof(typename TopGroups<T>::Key);
  constexpr size_t kMost = size_t(kMaxCluster) * kTopMaxK * 8 + size_t(kTopGroups) * kTopThreads * sizeof(typename TopGroups<T>::Key);
  auto* launch = a.entropy ? Launch<k_logprobs<T, true, true, false, kTopThreads>>::run
                           : Launch<k_logprobs<T, false, true, false, kTopThreads>>::run;
  return launch(threads, grid, ctas, smem, kMost, stream, a, shift, status);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream) {
  int* status = device_status_ptr();
  if (!status) return cudaErrorInvalidSymbol;
  if (a.v.dtype == NSM_BF16) return launch_logprobs_t<__nv_bfloat16>(a, status, stream);
  if (a.v.dtype == NSM_FP16) return launch_logprobs_t<__half>(a, status, stream);
  return launch_logprobs_t<float>(a, status, stream);
}

}  // namespace nsm
