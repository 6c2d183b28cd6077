// The choice of a token over logits that may hold infinities, NaN and rows
// with nothing left: Part folds and merges that keep their meaning there.
//
// A Part holds the best (key, id) with its logit z, and (m, s) with m = max x,
// s = sum exp(x - m), x = z / T'.  A row of -inf alone has m = -inf (LSE -inf,
// whatever s), one with +inf m = s = +inf (LSE +inf); exp_from(x, m) is 1 where
// x = m, so merges keep both.  A NaN x leaves m and makes s NaN (LSE NaN).
// A NaN key compares false and is never taken; a best key of -inf means that
// nothing is left.
#pragma once

#include "fh_device.hpp"

namespace fh {

__device__ __forceinline__ float exp_from(float x, float m) {
  return x == m ? 1.f : __expf(x - m);
}

// z / T' as z times 1 / T', held within the finite values where a finite z leaves
// them (a mask of the type's lowest value at a small T stays above -inf).
__device__ __forceinline__ float scaled_logit(float z, float inverse) {
  const bool finite = fabsf(z) < INFINITY;  // false for NaN
  return finite ? fminf(fmaxf(z * inverse, -FLT_MAX), FLT_MAX) : z;
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

__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);  // the truth table of a ^ b ^ c
}

// Philox4x32-10 of philox_block's counter for token draws (stage 1), both halves
// of each 32 x 32 product from one instruction.
__device__ __forceinline__ U4 token_words(uint64_t seed, uint32_t row, uint32_t blk) {
  uint32_t x = blk, y = row, z = 1u, w = 0u, k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * x, c = (uint64_t)0xCD9E8D57u * z;
    x = xor3((uint32_t)(c >> 32), y, k0);
    y = (uint32_t)c;
    z = xor3((uint32_t)(a >> 32), w, k1);
    w = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return U4{x, y, z, w};
}

// -log2 u of a word's uniform u (gumbel_from_word is -ln of it times ln 2); u is
// exact and never below 2^-24, so the instruction needs no help.
__device__ __forceinline__ float exponential_from_word(uint32_t w) {
  return -__builtin_amdgcn_logf(fmaf((float)(w >> 9), 1.1920928955078125e-07f, 5.9604644775390625e-08f));
}

// A lane's N logits as a Part; what does not count is -inf.  word: Philox words
// of the draws (sampling).  The largest x = z / T' comes first, then the
// exponentials e = exp(x - m) that the LSE sums.  The draw is the same race in
// another form: the largest x - ln(-ln u) is the largest e / (-ln u), so it needs
// one logarithm more per logit and no division (e l' > e' l); the key itself is
// formed for the winner alone, to be compared between lanes.  ORDERED: the ids
// ascend, so a tie stays with the earlier one; else the ids are compared.
//
// The exponent's shift is m within the finite values: beside x = +inf every finite
// e is then at most 1 and the infinite e wins the race (a shift of 0 would let any
// x above 88 overflow to the same +inf); m = -inf leaves e = 0.
template <int N, bool ORDERED>
__device__ __forceinline__ Part choose(const float (&z)[N], const int32_t (&id)[N], bool sample, float inverse,
                                       const uint32_t (&word)[N]) {
  Part p = part_empty();
  if (sample) {
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = scaled_logit(z[i], inverse);
      p.m = fmaxf(p.m, x[i]);
    }
    const float shift = __builtin_amdgcn_fmed3f(p.m, -FLT_MAX, FLT_MAX);
    float be = 0.f, bl = 1.f;
    uint32_t bw = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = __expf(x[i] - shift), l = exponential_from_word(word[i]);
      p.s += e;
      const float mine = e * bl, best = be * l;
      if (mine > best || (!ORDERED && mine == best && mine > 0.f && id[i] < p.id)) {
        be = e;
        bl = l;
        bw = word[i];
        p.z = z[i];
        p.id = id[i];
      }
    }
    if (be > 0.f) p.key = scaled_logit(p.z, inverse) + gumbel_from_word(bw);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (z[i] > p.key || (!ORDERED && z[i] == p.key && z[i] > -INFINITY && id[i] < p.id)) {
        p.key = z[i];
        p.id = id[i];
      }
    }
    p.z = p.key;
    p.m = p.key;  // -inf or the largest; a NaN is neither
    const float shift = __builtin_amdgcn_fmed3f(p.m, -FLT_MAX, FLT_MAX);
#pragma unroll
    for (int i = 0; i < N; ++i) p.s += __expf(z[i] - shift);
  }
  return p;
}

// The two values that lanes l and l ^ SPAN hold (SPAN 16 or 32), in one
// instruction and in one order for both lanes.
template <int SPAN>
__device__ __forceinline__ void pair(uint32_t x, uint32_t* lo, uint32_t* hi) {
  static_assert(SPAN == 16 || SPAN == 32, "rows or halves of a wave");
  if constexpr (SPAN == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    *lo = r[0];
    *hi = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    *lo = r[0];
    *hi = r[1];
  }
}

template <int SPAN>
__device__ __forceinline__ Part merge_pair(const Part& p) {
  uint32_t lo[5], hi[5];
  const uint32_t v[5] = {__float_as_uint(p.key), __float_as_uint(p.z), __float_as_uint(p.m),
                         __float_as_uint(p.s), (uint32_t)p.id};
#pragma unroll
  for (int i = 0; i < 5; ++i) pair<SPAN>(v[i], &lo[i], &hi[i]);
  return choice_merge(
      Part{__uint_as_float(lo[0]), __uint_as_float(lo[1]), __uint_as_float(lo[2]), __uint_as_float(lo[3]), (int32_t)lo[4]},
      Part{__uint_as_float(hi[0]), __uint_as_float(hi[1]), __uint_as_float(hi[2]), __uint_as_float(hi[3]), (int32_t)hi[4]});
}

// The four lanes l % 16 of a wave merged; every one gets the result.
__device__ __forceinline__ Part column_choice(const Part& p) { return merge_pair<32>(merge_pair<16>(p)); }

// All lanes of a wave merged, uniform: the largest m, then one exponential per
// lane; the largest key, then the lane that holds it.
__device__ __forceinline__ Part wave_choice(const Part& p) {
  Part r = part_empty();
  r.m = wave_max(p.m);
  r.s = wave_sum(p.s * exp_from(p.m, r.m));
  const float key = wave_max(p.key);
  if (key == -INFINITY) return r;
  uint64_t who = __ballot(p.key == key);
  if (who & (who - 1)) {  // a tie: the smallest id of those lanes
    int32_t id = p.key == key ? p.id : 0x7FFFFFFF;
    id = min(id, dpp_i<0xB1>(id));
    id = min(id, dpp_i<0x4E>(id));
    id = min(id, dpp_i<0x141>(id));
    id = min(id, dpp_i<0x140>(id));
    id = min(min(__builtin_amdgcn_readlane(id, 0), __builtin_amdgcn_readlane(id, 16)),
             min(__builtin_amdgcn_readlane(id, 32), __builtin_amdgcn_readlane(id, 48)));
    who = __ballot(p.key == key && p.id == id);
  }
  const int lane = __ffsll((unsigned long long)who) - 1;
  r.key = key;
  r.z = readlane_f(p.z, lane);
  r.id = __builtin_amdgcn_readlane(p.id, lane);
  return r;
}

__device__ __forceinline__ void write_choice(const Part& r, int64_t q, int32_t* out_token,
                                             float* out_logit, float* out_lse) {
  const bool none = !(r.key > -INFINITY);
  if (out_token) out_token[q] = none ? -1 : r.id;
  if (out_logit) out_logit[q] = none ? -INFINITY : r.z;
  if (out_lse) out_lse[q] = r.m + logf(r.s);
}

}  // namespace fh
