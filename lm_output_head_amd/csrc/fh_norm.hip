// Root-mean-square norm of rows with the residual's addition and an int8 output
// with a scale per row: s = x + residual, y = s / sqrt(mean(s^2) + eps) *
// (offset + weight), q = rint(y / (max |y| / 127)), all in float32 with one
// rounding per output.  Bound by the bytes of its rows.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fh_device.hpp"
#include "fh_internal.hpp"

namespace fh {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);  // round to nearest even
}

// Largest |y| as its bit pattern: NaN's is above infinity's, so a maximum of
// patterns keeps it.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ int quant8(float y, float scale) {
  return scale > 0.f ? (int)fminf(fmaxf(rintf(y / scale), -127.f), 127.f) : 0;
}

template <typename T>
__global__ __launch_bounds__(256) void k_rmsnorm(NormArgs a, int64_t B) {
  __shared__ float red[4];
  __shared__ uint32_t redu[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t d = a.d;
  for (int64_t b = blockIdx.x; b < B; b += gridDim.x) {
  const T* x = static_cast<const T*>(a.x) + b * a.ld_x;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + b * a.ld_residual : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  auto sum_at = [&](int64_t i) { return r ? to_f32<T>(x[i]) + to_f32<T>(r[i]) : to_f32<T>(x[i]); };
  float ss = 0.f;
  for (int64_t i = tid; i < d; i += 256) {
    const float s = sum_at(i);
    ss = fmaf(s, s, ss);
  }
  ss = wave_sum(ss);
  if (lane == 0) red[wave] = ss;
  __syncthreads();
  const float inv = 1.f / sqrtf(((red[0] + red[1]) + (red[2] + red[3])) / (float)d + a.eps);
  auto norm_at = [&](int64_t i, float s) {
    const float y = s * inv;
    return w ? y * (a.offset + to_f32<T>(w[i])) : y;
  };
  float scale = 0.f;
  if (a.out_q) {
    uint32_t top = 0u;
    for (int64_t i = tid; i < d; i += 256) top = max(top, abs_bits(norm_at(i, sum_at(i))));
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if (lane == 0) redu[wave] = top;
    __syncthreads();
    scale = __uint_as_float(max(max(redu[0], redu[1]), max(redu[2], redu[3]))) / 127.f;
    if (tid == 0) a.out_scale[b] = scale;
  }
  // each element is read and written by one thread, x and residual before the
  // outputs that may be their own storage
  for (int64_t i = tid; i < d; i += 256) {
    const float s = sum_at(i), y = norm_at(i, s);
    if (a.out) static_cast<T*>(a.out)[b * a.ld_out + i] = from_f32<T>(y);
    if (a.out_residual) static_cast<T*>(a.out_residual)[b * a.ld_out_residual + i] = from_f32<T>(s);
    if (a.out_q) a.out_q[b * a.ld_q + i] = (int8_t)quant8(y, scale);
  }
  __syncthreads();  // red and redu are free for the next row
  }
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, bool bf16, int64_t B, hipStream_t stream) {
  const dim3 grid((unsigned)std::min<int64_t>(B, 1 << 20)), block(256);
  if (bf16)
    hipLaunchKernelGGL((k_rmsnorm<uint16_t>), grid, block, 0, stream, a, B);
  else
    hipLaunchKernelGGL((k_rmsnorm<float>), grid, block, 0, stream, a, B);
  return hipGetLastError();
}

}  // namespace fh
