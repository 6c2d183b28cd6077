// The choice of a token over logits that may hold infinities, NaN and rows
// with nothing left: Part folds and merges that keep their meaning there.
//
// A Part holds the best (key, id) with its logit z, and (m, s) with m = max x,
// s = sum exp(x - m), x = z / T'.  exp_from(x, m) is 1 where x = m, so m = +inf
// counts its own terms (s >= 1, LSE +inf) and a row of -inf alone has
// m = -inf (LSE -inf, whatever s); a NaN x leaves m and makes s NaN (LSE NaN).
// A NaN key compares false and is never taken; a best key of -inf means that
// nothing is left.
#pragma once

#include "fh_device.hpp"

namespace fh {

__device__ __forceinline__ float exp_from(float x, float m) {
  return x == m ? 1.f : __expf(x - m);
}

// z / T', held at the largest finite value where a finite z leaves the range (a
// mask of the type's lowest value at a small T stays above -inf).
__device__ __forceinline__ float scaled_logit(float z, float tprime) {
  const float x = z / tprime;
  return fabsf(x) == INFINITY && fabsf(z) < INFINITY ? copysignf(FLT_MAX, z) : x;
}

__device__ __forceinline__ void choice_key(Part& p, float key, float z, int32_t id) {
  if (better(key, id, p.key, p.id)) {
    p.key = key;
    p.z = z;
    p.id = id;
  }
}

__device__ __forceinline__ void choice_lse(Part& p, float m, float s) {
  const float hm = fmaxf(p.m, m);
  p.s = p.s * exp_from(p.m, hm) + s * exp_from(m, hm);
  p.m = hm;
}

__device__ __forceinline__ Part choice_merge(Part a, const Part& b) {
  choice_key(a, b.key, b.z, b.id);
  choice_lse(a, b.m, b.s);
  return a;
}

__device__ __forceinline__ Part shfl_part(const Part& p, int mask) {
  return Part{__shfl_xor(p.key, mask), __shfl_xor(p.z, mask), __shfl_xor(p.m, mask),
              __shfl_xor(p.s, mask), __shfl_xor(p.id, mask)};
}

// Merge the lanes of a wave whose numbers differ in the bits from LO up.
template <int LO = 1>
__device__ __forceinline__ Part wave_choice(Part p) {
#pragma unroll
  for (int mask = LO; mask < 64; mask <<= 1) p = choice_merge(p, shfl_part(p, mask));
  return p;
}

__device__ __forceinline__ void write_choice(const Part& r, int64_t q, int32_t* out_token,
                                             float* out_logit, float* out_lse) {
  const bool none = !(r.key > -INFINITY);
  if (out_token) out_token[q] = none ? -1 : r.id;
  if (out_logit) out_logit[q] = none ? -INFINITY : r.z;
  if (out_lse) out_lse[q] = r.m + logf(r.s);
}

}  // namespace fh
