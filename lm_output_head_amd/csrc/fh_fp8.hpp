// OCP E4M3 codes of values under a scale, and the interface between the C ABI
// (fh_fp8_api.cpp) and the launchers of the fp8 operators.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fh_internal.hpp"

namespace fh {

#ifdef __HIP_DEVICE_COMPILE__
// Four codes, rounded to nearest even; |t| <= 448 but for a rounding of the
// quotient, which still rounds to 448.
__device__ __forceinline__ uint32_t e4m3_of(float t0, float t1, float t2, float t3) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t2, t3, __builtin_amdgcn_cvt_pk_fp8_f32(t0, t1, 0, false), true);
}
#else
__device__ uint32_t e4m3_of(float, float, float, float);
#endif

// What makes codes round(y / scale), scale = max |y| / 448, the division rounded
// once to float32: with r = 1 / scale rounded once, t = y r is within two units of
// the quotient's last place; a correction by the exact remainder y - t scale leaves
// a neighbour of the quotient and a second one the rounded quotient itself
// (Markstein 1990).  A remainder can underflow only where the quotient is far below
// half of the smallest code.
struct E4M3Scale {
  static constexpr float kSmall = 0x1p-100f, kUp = 0x1p64f;
  float scale, by, r;
  uint32_t sign;
  bool small;
  __device__ __forceinline__ explicit E4M3Scale(float s) {
    scale = s;
    small = scale < kSmall;
    by = small ? scale * kUp : scale;
    r = by > 0.f ? 1.f / by : 0.f;
    sign = by > 0.f ? 0x80000000u : 0u;
  }
  // Values near the subnormals are brought up; their scale has few bits, so what
  // the quotient's bounds leave is cut here.
  template <int N>
  __device__ __forceinline__ void raise(float (&y)[N]) const {
    if (!small) return;
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __builtin_amdgcn_fmed3f(y[i], -448.f * scale, 448.f * scale) * kUp;
  }
  __device__ __forceinline__ float of(float y) const {
    float t = y * r;
    t = fmaf(fmaf(-t, by, y), r, t);
    t = fmaf(fmaf(-t, by, y), r, t);
    // the corrections make +0 of a quotient of -0
    return __uint_as_float((__float_as_uint(y) & sign) | (__float_as_uint(t) & ~sign));
  }
};

// Hidden states in fp8 (fh_fp8_quant.hip): fh_rmsnorm_fp8's and fh_fp8_quant's
// arguments as checked.
struct FP8QuantArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;    // or null
  void* out;             // or null, as the next two
  void* out_residual;
  uint8_t* out_q;
  float* out_scale;      // [B x ld_scale]
  int64_t ld_x, ld_residual, ld_out, ld_out_residual, ld_q, ld_scale;
  int64_t d;
  float eps, offset;
};
hipError_t launch_rmsnorm_fp8(const FP8QuantArgs& a, bool bf16, int64_t B, hipStream_t st);
hipError_t launch_fp8_quant(const FP8QuantArgs& a, bool bf16, int64_t B, hipStream_t st);

// The fp8 product and the dense head on it (fh_fp8.hip).  Weights lie in the int8
// product's fragment order (fh_serve.hpp), codes as they are.
struct FP8Args {
  const void* W;         // [ceil(n / 16)][2 ceil(k / 128)][64] 16-byte chunks
  const float* ws;       // [ceil(n / 128)][ceil(k / 128)]
  int64_t n;
  int k;
  const uint8_t* q;      // [B x ld_q], 16-byte aligned rows of ceil(k / 16) 16 readable bytes
  int64_t ld_q;
  const float* qs;       // [B x ld_qs]
  int64_t ld_qs;
  int B;
  void* out;             // float or bf16 [B x ld_out], or null (head)
  int64_t ld_out;
  // head
  int token_sample;
  float inverse_t;       // 1 / T'
  uint64_t seed;
  Part* parts;           // [B x fp8_parts]
};
hipError_t launch_fp8_scales(const void* W, bool bf16, int64_t n, int64_t k, float* scales, int* bad, hipStream_t st);
hipError_t launch_fp8_pack(const void* W, bool bf16, const float* scales, int64_t n, int64_t k, void* packed,
                           hipStream_t st);
int64_t fp8_parts(int64_t n, int64_t k, int64_t B);  // partials per row of the head
bool fp8_fits(int64_t n, int64_t k, int64_t B);  // a launch holds fewer than 2^32 threads
// What a launch gives: results, in the matrix cores' own fp8 where that is asked
// for, or a head's float32 logits (or none) and partials.
enum class FP8Out { kF32, kBf16, kBf16Native, kHead };
hipError_t launch_fp8(const FP8Args& a, FP8Out out, hipStream_t st);

}  // namespace fh
