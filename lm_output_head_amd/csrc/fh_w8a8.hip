// The int8 matrix product with a scale per row of both operands (W8A8),
// out[b, j] = (sum_i q[b, i] w[j, i]) (qs[b] ws[j]), and the dense head on it.
//
// v_mfma_i32_16x16x64_i8 multiplies 16 rows of W with 16 tokens over 64
// elements of k, exact in int32: lane l holds W's row l % 16 and token l % 16
// at elements 16 (l / 16) .. + 15, and the result's token l % 16 at W's rows
// 4 (l / 16) .. + 3.  W is kept in that order (fragment order), so one
// instruction's operand is one contiguous 1 KB.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fh_choice.hpp"
#include "fh_internal.hpp"

namespace fh {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ i32x4 mfma_i8(const uint4& a, const uint4& b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Four results of one token at channels j .. j + 3, those below n.
__device__ __forceinline__ void store4(const W8A8Args& a, bool bf16, int64_t q, int64_t j, const float (&z)[4]) {
  if (bf16) {
    uint16_t* o = static_cast<uint16_t*>(a.out) + q * a.ld_out + j;
    if (j + 3 < a.n)
      *reinterpret_cast<u16x4u*>(o) = u16x4u{bf16_bits(z[0]), bf16_bits(z[1]), bf16_bits(z[2]), bf16_bits(z[3])};
    else
      for (int i = 0; i < 4 && j + i < a.n; ++i) o[i] = bf16_bits(z[i]);
  } else {
    float* o = static_cast<float*>(a.out) + q * a.ld_out + j;
    if (j + 3 < a.n)
      *reinterpret_cast<f32x4u*>(o) = f32x4u{z[0], z[1], z[2], z[3]};
    else
      for (int i = 0; i < 4 && j + i < a.n; ++i) o[i] = z[i];
  }
}

constexpr int kWaves = 4;

// NT token tiles and MT row tiles of 16 per wave.
template <int NT, int MT, bool BF16, bool HEAD>
__global__ __launch_bounds__(64 * kWaves) void k_w8a8(W8A8Args a) {
  __shared__ Part sh[HEAD ? kWaves : 1][HEAD ? 16 * NT : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, col = lane & 15;
  const int64_t tiles = (a.n + 15) / 16;
  const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wave) * MT;
  const int q0 = blockIdx.y * 16 * NT;
  const int steps = (a.k + 63) / 64, chunks = (a.k + 15) / 16;

  const uint4* wp[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) wp[m] = a.W + min(t0 + m, tiles - 1) * steps * 64 + lane;
  const int8_t* qp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) qp[t] = a.q + (int64_t)min(q0 + 16 * t + col, a.B - 1) * a.ld_q;

  i32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = i32x4{0, 0, 0, 0};
  for (int s = 0; s < steps; ++s) {
    // a 16-byte chunk past the row stands in as its first: W is zero there
    const int ch = 4 * s + g < chunks ? 4 * s + g : 0;
    uint4 wf[MT], qf[NT];
#pragma unroll
    for (int m = 0; m < MT; ++m) wf[m] = wp[m][s * 64];
#pragma unroll
    for (int t = 0; t < NT; ++t) qf[t] = *reinterpret_cast<const uint4*>(qp[t] + 16 * ch);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[m][t] = mfma_i8(wf[m], qf[t], acc[m][t]);
  }

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t q = q0 + 16 * t + col;
    const float qs = q < a.B ? a.qs[q] : 0.f;
    Part p = part_empty();
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t j = 16 * (t0 + m) + 4 * g;
      float z[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[i] = j + i < a.n ? (float)acc[m][t][i] * (qs * a.ws[j + i]) : 0.f;
        if (HEAD && j + i < a.n) {
          const float x = scaled_logit(z[i], a.tprime);
          const int32_t id = (int32_t)(j + i);
          choice_key(p, a.token_sample ? x + gumbel_at(a.seed, (uint32_t)q, (uint32_t)id, 1u) : z[i], z[i], id);
          choice_lse(p, x, 1.f);
        }
      }
      if (a.out && q < a.B && j < a.n) store4(a, BF16, q, j, z);
    }
    if (HEAD) {
      p = wave_choice<16>(p);
      if (g == 0) sh[wave][16 * t + col] = p;
    }
  }
  if (HEAD) {
    __syncthreads();
    const int i = threadIdx.x;
    if (i < 16 * NT && q0 + i < a.B) {
      Part p = sh[0][i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) p = choice_merge(p, sh[w][i]);
      a.parts[(int64_t)(q0 + i) * gridDim.x + blockIdx.x] = p;
    }
  }
}

// scale[j] = max |W[j]| / 127; *bad is set where a row is not finite.
template <typename T>
__device__ __forceinline__ float w_elem(const void* W, int64_t i);
template <>
__device__ __forceinline__ float w_elem<float>(const void* W, int64_t i) { return static_cast<const float*>(W)[i]; }
template <>
__device__ __forceinline__ float w_elem<uint16_t>(const void* W, int64_t i) {
  return __uint_as_float((uint32_t)static_cast<const uint16_t*>(W)[i] << 16);
}

template <typename T>
__global__ __launch_bounds__(256) void k_w8a8_scales(const void* W, int64_t n, int64_t k, float* scales, int* bad) {
  for (int64_t j = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); j < n; j += (int64_t)gridDim.x * 4) {
    uint32_t top = 0u;  // |W| as bits: NaN's and infinity's are above every finite value's
    for (int64_t i = threadIdx.x & 63; i < k; i += 64)
      top = max(top, __float_as_uint(w_elem<T>(W, j * k + i)) & 0x7FFFFFFFu);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if ((threadIdx.x & 63) == 0) {
      scales[j] = __uint_as_float(top) / 127.f;
      if (top >= 0x7F800000u) atomicOr(bad, 1);
    }
  }
}

// One thread per 16-byte chunk of the fragment order.
template <typename T>
__global__ __launch_bounds__(256) void k_w8a8_pack(const int8_t* codes, const void* W, const float* scales, int64_t n,
                                                   int64_t k, int64_t chunks, uint4* out) {
  const int64_t steps = (k + 63) / 64;
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks; c += (int64_t)gridDim.x * 256) {
    const int lane = (int)(c & 63);
    const int64_t s = (c >> 6) % steps, j = (c >> 6) / steps * 16 + (lane & 15), i0 = s * 64 + (lane >> 4) * 16;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (j < n) {
      const float sc = codes ? 0.f : scales[j];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (i0 + e >= k) break;
        int v = 0;
        if (codes)
          v = codes[j * k + i0 + e];
        else if (sc > 0.f)
          v = (int)fminf(fmaxf(rintf(w_elem<T>(W, j * k + i0 + e) / sc), -127.f), 127.f);
        w[e >> 2] |= ((uint32_t)v & 0xFFu) << (8 * (e & 3));
      }
    }
    out[c] = uint4{w[0], w[1], w[2], w[3]};
  }
}

__global__ __launch_bounds__(256) void k_w8a8_unpack(const int8_t* packed, int64_t n, int64_t k, int8_t* codes) {
  const int64_t steps = (k + 63) / 64;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * k; i += (int64_t)gridDim.x * 256) {
    const int64_t j = i / k, e = i % k;
    const int64_t lane = (j & 15) + 16 * ((e & 63) >> 4);
    codes[i] = packed[(((j >> 4) * steps + (e >> 6)) * 64 + lane) * 16 + (e & 15)];
  }
}

__global__ __launch_bounds__(256) void k_w8a8_align(const int8_t* q, int64_t ld_q, int64_t B, int64_t k, int8_t* out,
                                                    int64_t ld) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < B * ld; i += (int64_t)gridDim.x * 256) {
    const int64_t b = i / ld, e = i % ld;
    out[i] = e < k ? q[b * ld_q + e] : (int8_t)0;
  }
}

__global__ __launch_bounds__(64) void k_choice(const Part* parts, int64_t nparts, int32_t* out_token, float* out_logit,
                                               float* out_lse) {
  const int64_t q = blockIdx.x;
  Part p = part_empty();
  for (int64_t i = threadIdx.x; i < nparts; i += 64) p = choice_merge(p, parts[q * nparts + i]);
  p = wave_choice(p);
  if (threadIdx.x == 0) write_choice(p, q, out_token, out_logit, out_lse);
}

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20); }

int token_tiles(int64_t B) { return B <= 16 ? 1 : B <= 32 ? 2 : 4; }
constexpr int kMT = 2;

template <int NT>
hipError_t launch_nt(const W8A8Args& a, bool out_bf16, bool head, hipStream_t st) {
  const dim3 grid((unsigned)w8a8_parts(a.n, a.B), (unsigned)((a.B + 16 * NT - 1) / (16 * NT))), block(64 * kWaves);
  if (head)
    hipLaunchKernelGGL((k_w8a8<NT, kMT, false, true>), grid, block, 0, st, a);
  else if (out_bf16)
    hipLaunchKernelGGL((k_w8a8<NT, kMT, true, false>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_w8a8<NT, kMT, false, false>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

int64_t w8a8_packed_bytes(int64_t n, int64_t k) { return (n + 15) / 16 * ((k + 63) / 64) * 1024; }

int64_t w8a8_parts(int64_t n, int64_t) { return (n + 16 * kMT * kWaves - 1) / (16 * kMT * kWaves); }

hipError_t launch_w8a8(const W8A8Args& a, bool out_bf16, bool head, hipStream_t st) {
  switch (token_tiles(a.B)) {
    case 1: return launch_nt<1>(a, out_bf16, head, st);
    case 2: return launch_nt<2>(a, out_bf16, head, st);
    default: return launch_nt<4>(a, out_bf16, head, st);
  }
}

hipError_t launch_w8a8_scales(const void* W, bool bf16, int64_t n, int64_t k, float* scales, int* bad, hipStream_t st) {
  const dim3 grid((unsigned)std::min<int64_t>((n + 3) / 4, 1 << 20));
  if (bf16)
    hipLaunchKernelGGL((k_w8a8_scales<uint16_t>), grid, dim3(256), 0, st, W, n, k, scales, bad);
  else
    hipLaunchKernelGGL((k_w8a8_scales<float>), grid, dim3(256), 0, st, W, n, k, scales, bad);
  return hipGetLastError();
}

hipError_t launch_w8a8_pack(const int8_t* codes, const void* W, bool bf16, const float* scales, int64_t n, int64_t k,
                            void* packed, hipStream_t st) {
  const int64_t chunks = w8a8_packed_bytes(n, k) / 16;
  const dim3 grid(grid_of(chunks));
  uint4* out = static_cast<uint4*>(packed);
  if (bf16)
    hipLaunchKernelGGL((k_w8a8_pack<uint16_t>), grid, dim3(256), 0, st, codes, W, scales, n, k, chunks, out);
  else
    hipLaunchKernelGGL((k_w8a8_pack<float>), grid, dim3(256), 0, st, codes, W, scales, n, k, chunks, out);
  return hipGetLastError();
}

hipError_t launch_w8a8_unpack(const void* packed, int64_t n, int64_t k, int8_t* codes, hipStream_t st) {
  hipLaunchKernelGGL(k_w8a8_unpack, dim3(grid_of(n * k)), dim3(256), 0, st, static_cast<const int8_t*>(packed), n, k,
                     codes);
  return hipGetLastError();
}

hipError_t launch_w8a8_align(const int8_t* q, int64_t ld_q, int64_t B, int64_t k, int8_t* out, int64_t ld,
                             hipStream_t st) {
  hipLaunchKernelGGL(k_w8a8_align, dim3(grid_of(B * ld)), dim3(256), 0, st, q, ld_q, B, k, out, ld);
  return hipGetLastError();
}

hipError_t launch_choice(const Part* parts, int64_t B, int64_t nparts, int32_t* out_token, float* out_logit,
                         float* out_lse, hipStream_t st) {
  hipLaunchKernelGGL(k_choice, dim3((unsigned)B), dim3(64), 0, st, parts, nparts, out_token, out_logit, out_lse);
  return hipGetLastError();
}

}  // namespace fh
