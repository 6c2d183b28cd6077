// What the 8-bit products share: how results leave, the choice of a token over a
// tile of logits, a barrier that lets loads pass, reads of a weight's rows.
#pragma once

#include "fh_choice.hpp"

namespace fh {

// N results of one token from channel j up, those below n, in 16 (or 8) bytes.
// STREAM: past the caches, which the operands need (64 x 151936 float results
// beside 389 MB of weights: 95 -> 85 us; 4096 x 10240 bf16: 144 -> 132 us).
template <typename T, int N, bool STREAM>
__device__ __forceinline__ void store_run(T* o, int64_t j, int64_t n, const T* v) {
  typedef T V __attribute__((ext_vector_type(N), aligned(sizeof(T))));
  if (j + N <= n) {
    V x;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v[i];
    if (STREAM)
      __builtin_nontemporal_store(x, reinterpret_cast<V*>(o + j));
    else
      *reinterpret_cast<V*>(o + j) = x;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (j + i < n) o[j + i] = v[i];
  }
}

template <bool BF16>
struct Out {
  typedef float T;
  __device__ static float of(float z) { return z; }
};
template <>
struct Out<true> {
  typedef uint16_t T;
  __device__ static uint16_t of(float z) { return __builtin_bit_cast(uint16_t, (__bf16)z); }
};

// A lane's 4 FN logits z[m][i] of row q, tokens 16 (t0 + m) + 4 g + i, as a Part.
template <int FN, typename Args>
__device__ __forceinline__ Part choose_tile(const Args& a, const float (&z)[FN][4], int64_t q, int64_t t0, int g) {
  float v[4 * FN];
  int32_t id[4 * FN];
  uint32_t word[4 * FN];
#pragma unroll
  for (int m = 0; m < FN; ++m) {
    const int64_t j = 16 * (t0 + m) + 4 * g;
    U4 words{0u, 0u, 0u, 0u};
    if (a.token_sample) words = token_words(a.seed, (uint32_t)q, (uint32_t)(j >> 2));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[4 * m + i] = j + i < a.n ? z[m][i] : -INFINITY;
      id[4 * m + i] = (int32_t)(j + i);
      word[4 * m + i] = u4_word(words, i);
    }
  }
  return choose<4 * FN, true>(v, id, a.token_sample != 0, a.inverse_t, word);
}

// Orders this workgroup's LDS accesses around a barrier; loads from memory stay
// in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// N consecutive elements of W from i on as floats, in 16-byte loads at any
// alignment of the element (one by one the layout of 128256 x 2048 bfloat16 took
// 525 us and its scales 273, with them 147 and 108).
template <typename T, int N>
__device__ __forceinline__ void w_run(const void* W, int64_t i, float (&v)[N]) {
  constexpr int kPer = 16 / (int)sizeof(T);
  typedef T V __attribute__((ext_vector_type(kPer), aligned(sizeof(T))));
#pragma unroll
  for (int e = 0; e < N; e += kPer) {
    const V x = *reinterpret_cast<const V*>(static_cast<const T*>(W) + i + e);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if constexpr (sizeof(T) == 2)
        v[e + u] = __uint_as_float((uint32_t)x[u] << 16);
      else
        v[e + u] = x[u];
    }
  }
}
template <typename T>
__device__ __forceinline__ float w_elem(const void* W, int64_t i) {
  if constexpr (sizeof(T) == 2)
    return __uint_as_float((uint32_t)static_cast<const T*>(W)[i] << 16);
  else
    return static_cast<const T*>(W)[i];
}

}  // namespace fh
