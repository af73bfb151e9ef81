// 16-byte vectors of bf16, fp16 and fp32 elements, and pairs of fp32 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "nsm_internal.h"

namespace nsm {
namespace {

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

// A 16-byte vector of elements of one type.
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

// Eight elements: one 16-byte vector of a 16-bit type, two of fp32.
template <typename T>
struct Eight {
  static constexpr int kWords = sizeof(T) / 2;
  uint4 w[kWords];
  // p on a 16-byte boundary
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  // what this kernel itself may write goes past the read-only path
  __device__ __forceinline__ void load_written(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  }
  // what is not read again soon
  __device__ __forceinline__ void store_streaming(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) __stcs(reinterpret_cast<uint4*>(p) + i, w[i]);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      Pair x[8 / kWords / 2];
      Elem<T>::unpack(w[i], x);
#pragma unroll
      for (int j = 0; j < 8 / kWords / 2; ++j) split_pair(x[j], f[i * (8 / kWords) + 2 * j], f[i * (8 / kWords) + 2 * j + 1]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      Pair x[8 / kWords / 2];
#pragma unroll
      for (int j = 0; j < 8 / kWords / 2; ++j) x[j] = make_pair(f[i * (8 / kWords) + 2 * j], f[i * (8 / kWords) + 2 * j + 1]);
      w[i] = Elem<T>::pack(x);
    }
  }
};

__device__ __forceinline__ bool on_16_bytes(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Bytes32 {
  uint4 low, high;
};

// kPer elements side by side: 8, 16 or 32 bytes.
template <typename T, int kPer>
struct Side {
  static constexpr int kBytes = kPer * sizeof(T);
  using Word = typename std::conditional<kBytes == 32, Bytes32, typename std::conditional<kBytes == 16, uint4, uint2>::type>::type;
  Word w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Word*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Word*>(p) = w; }
  __device__ __forceinline__ void get(float (&f)[kPer]) const {
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < kPer; ++i) f[i] = Elem<T>::to_float(e[i]);
  }
  __device__ __forceinline__ void set(const float (&f)[kPer]) {
    T* e = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = Elem<T>::from_float(f[i]);
  }
};

// How many elements past a 16-byte boundary.
template <typename T>
__device__ __forceinline__ int lead_of(const T* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}

// The elements c0 ... c0 + 7 of a row that has [low, high), zeros outside it, whatever their
// alignment: whole vectors around them, shifted into place, where those lie within the row.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int low, int high, int c0, Eight<T>& r, int* status, int kernel, int site) {
  constexpr int kPer = 16 / sizeof(T);
  const T* at = row + c0;
  const int s = lead_of(at);
  if (s == 0 && c0 >= low && c0 + 8 <= high) {
    if (bounds_ok(on_16_bytes(at), status, kernel, 0, site)) r.load_written(at);
    return;
  }
  if (c0 - s >= low && c0 - s + 8 + kPer <= high) {
    uint32_t w[4 * (Eight<T>::kWords + 1)];
    const uint4* from = reinterpret_cast<const uint4*>(at - s);
    if (!bounds_ok(on_16_bytes(from), status, kernel, 0, site)) return;
#pragma unroll
    for (int i = 0; i <= Eight<T>::kWords; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = from[i];
    constexpr int kNeed = 4 * Eight<T>::kWords;  // words that are wanted
    const int words = sizeof(T) == 4 ? s : s >> 1;
    if (words & 2) {
#pragma unroll
      for (int i = 0; i < kNeed + 2; ++i) w[i] = w[i + 2];
    }
    if (words & 1) {
#pragma unroll
      for (int i = 0; i < kNeed + 1; ++i) w[i] = w[i + 1];
    }
    if (sizeof(T) == 2 && (s & 1)) {
#pragma unroll
      for (int i = 0; i < kNeed; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
#pragma unroll
    for (int i = 0; i < Eight<T>::kWords; ++i) r.w[i] = *reinterpret_cast<const uint4*>(w + 4 * i);
    return;
  }
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = c0 + i >= low && c0 + i < high ? at[i] : Elem<T>::from_float(0.f);
#pragma unroll
  for (int i = 0; i < Eight<T>::kWords; ++i) r.w[i] = reinterpret_cast<const uint4*>(e)[i];
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int low, int high, int c0, const float (&f)[8], int* status, int kernel, int site) {
  T* at = row + c0;
  Eight<T> r;
  r.set(f);
  if (c0 >= low && c0 + 8 <= high && on_16_bytes(at)) {
    if (bounds_ok(on_16_bytes(at), status, kernel, 0, site)) r.store(at);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c0 + i >= low && c0 + i < high) at[i] = reinterpret_cast<const T*>(r.w)[i];
}

}  // namespace
}  // namespace nsm
