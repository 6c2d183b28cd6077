// Rows read and written in chunks of 16 bytes, and sums and maxima over the lanes
// and waves that share one: the norms' common parts.
#pragma once

#include "fh_device.hpp"

namespace fh {

// Elements of T as they are stored, eight of bfloat16 or four of float32 (16
// bytes), at any alignment of the element: rows of odd widths are read and
// written 16 bytes at a time too, only a row's last chunk may be partial.
template <typename T>
struct Elems;
template <>
struct Elems<float> {
  static constexpr int N = 4;
  typedef float V __attribute__((ext_vector_type(4), aligned(4)));
  __device__ static float get(float v) { return v; }
  __device__ static float put(float v) { return v; }
};
template <>
struct Elems<uint16_t> {
  static constexpr int N = 8;
  typedef uint16_t V __attribute__((ext_vector_type(8), aligned(2)));
  __device__ static float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  __device__ static uint16_t put(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);  // round to nearest even
  }
};

// Elements at .. at + N - 1 of a row of d, zero past it.
template <typename T>
__device__ __forceinline__ void load_chunk(const T* p, int64_t at, int64_t d, float (&v)[Elems<T>::N]) {
  constexpr int N = Elems<T>::N;
  if (at + N <= d) {
    const typename Elems<T>::V x = *reinterpret_cast<const typename Elems<T>::V*>(p + at);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Elems<T>::get(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = at + i < d ? Elems<T>::get(p[at + i]) : 0.f;
  }
}

// PAST: by the caches.
template <typename T, bool PAST = false>
__device__ __forceinline__ void store_chunk(T* p, int64_t at, int64_t d, const float (&v)[Elems<T>::N]) {
  constexpr int N = Elems<T>::N;
  if (at + N <= d) {
    typename Elems<T>::V x;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Elems<T>::put(v[i]);
    if constexpr (PAST)
      __builtin_nontemporal_store(x, reinterpret_cast<typename Elems<T>::V*>(p + at));
    else
      *reinterpret_cast<typename Elems<T>::V*>(p + at) = x;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at + i < d) p[at + i] = Elems<T>::put(v[i]);
  }
}

// Largest |y| as its bit pattern: NaN's is above infinity's, so a maximum of
// patterns keeps it.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Sum and maximum over the L lanes that share a row.
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
  if constexpr (L == 64) return wave_sum(v);
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lane_umax(uint32_t v) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}

// Sum (or maximum) over the W waves that share a row; W = 1 needs no LDS.
template <int W, typename V, typename Op>
__device__ __forceinline__ V across(V v, V* sh, Op op) {
  if constexpr (W == 1) return v;
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sh[0];
#pragma unroll
  for (int w = 1; w < W; ++w) v = op(v, sh[w]);
  return v;
}

}  // namespace fh
