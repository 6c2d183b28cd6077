// Hidden states in 8-bit floating point (OCP E4M3) with a scale per 128 elements
// of a row, as they are or after the final norm with the residual's addition:
// s = x + residual, y = s / sqrt(mean(s^2) + eps) * (offset + weight), and of each
// 128 scale = max |y| / 448, code = round(y / scale), in float32 with one rounding
// per output.
//
// A row is read once, 16 bytes a lane, and stays in registers for the norm; the 128
// elements of a scale lie in 16 lanes (32 of float32), whose maximum takes
// exchanges within a row of lanes alone, so the codes cost no LDS and no second
// pass.  What bounds it is memory: 16384 x 2560 bfloat16 with a residual and both
// outputs, 295 MB, takes 63 us (the fastest 61), 4.7 TB/s, nearly the rate of a copy.
// One row takes 2.5 us.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fh_fp8.hpp"
#include "fh_rows.hpp"

namespace fh {
namespace {

// The largest of the L lanes (8, 16, 32 or 64) that this one is in, as bits.
template <int L>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
  v = max(v, (uint32_t)dpp_i<0xB1>((int)v));   // quads
  v = max(v, (uint32_t)dpp_i<0x4E>((int)v));
  v = max(v, (uint32_t)dpp_i<0x141>((int)v));  // eight
  if constexpr (L >= 16) v = max(v, (uint32_t)dpp_i<0x140>((int)v));
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(r[0], r[1]);
  }
  return v;
}

// The scale and codes of one chunk at `at` of row b; its 128 elements lie in
// min(L, 128 / N) lanes.
template <typename T, int L>
__device__ __forceinline__ void store_fp8(const FP8QuantArgs& a, int64_t b, int64_t at, float (&y)[Elems<T>::N]) {
  constexpr int N = Elems<T>::N, kLanes = L < 128 / N ? L : 128 / N;
  uint32_t top = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at + i < a.d) top = max(top, abs_bits(y[i]));
  top = group_umax<kLanes>(top);
  const E4M3Scale sc(__uint_as_float(top) / 448.f);
  if (at % 128 == 0 && at < a.d) a.out_scale[b * a.ld_scale + at / 128] = sc.scale;
  sc.raise<N>(y);
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j)
    w[j] = e4m3_of(sc.of(y[4 * j]), sc.of(y[4 * j + 1]), sc.of(y[4 * j + 2]), sc.of(y[4 * j + 3]));
  uint8_t* p = a.out_q + b * a.ld_q;
  if (at + N <= a.d) {
    typedef uint32_t W __attribute__((ext_vector_type(N / 4), aligned(1)));
    W x;
#pragma unroll
    for (int j = 0; j < N / 4; ++j) x[j] = w[j];
    *reinterpret_cast<W*>(p + at) = x;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at + i < a.d) p[at + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// W waves (or, W = 1, L of a wave's lanes) per row, C chunks per lane: the row
// stays in registers between its one read and the writes.  A workgroup is
// max(4, W) waves.  PAST: out and out_residual pass the caches by.
template <typename T, int L, int W, int C, bool PAST>
__global__ __launch_bounds__(W <= 4 ? 256 : 64 * W) void k_rmsnorm_fp8(FP8QuantArgs a, int64_t B) {
  static_assert(W == 1 || L == 64, "waves that share a row do so with all lanes");
  constexpr int N = Elems<T>::N, kRows = W == 1 ? 256 / L : 1, kLanes = L * W;
  __shared__ float sum_sh[W];
  const int64_t b = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes, d = a.d;
  if (b >= B) return;
  const int lane = threadIdx.x % kLanes;
  const T* x = static_cast<const T*>(a.x) + b * a.ld_x;
  const T* r = a.residual ? static_cast<const T*>(a.residual) + b * a.ld_residual : nullptr;
  const T* w = static_cast<const T*>(a.weight);
  float y[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c) load_chunk<T>(x, (int64_t)N * (lane + kLanes * c), d, y[c]);
  if (r) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float v[N];
      load_chunk<T>(r, (int64_t)N * (lane + kLanes * c), d, v);
#pragma unroll
      for (int i = 0; i < N; ++i) y[c][i] += v[i];
    }
  }
  // the sum leaves here: out_residual may be x or residual, whose chunk this
  // lane has read
  if (a.out_residual) {
    T* o = static_cast<T*>(a.out_residual) + b * a.ld_out_residual;
#pragma unroll
    for (int c = 0; c < C; ++c) store_chunk<T, PAST>(o, (int64_t)N * (lane + kLanes * c), d, y[c]);
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(y[c][i], y[c][i], ss);
  ss = across<W>(lane_sum<L>(ss), sum_sh, [](float p, float q) { return p + q; });
  const float inv = 1.f / sqrtf(ss / (float)d + a.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t at = (int64_t)N * (lane + kLanes * c);
    float v[N];
    if (w) load_chunk<T>(w, at, d, v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      y[c][i] *= inv;
      if (w) y[c][i] *= a.offset + v[i];
    }
    if (a.out) store_chunk<T, PAST>(static_cast<T*>(a.out) + b * a.ld_out, at, d, y[c]);
    store_fp8<T, L>(a, b, at, y[c]);
  }
}

// Rows too long for the registers: two passes over the row, the second from the
// caches.
template <typename T>
__global__ __launch_bounds__(1024) void k_rmsnorm_fp8_long(FP8QuantArgs a, int64_t B) {
  constexpr int W = 16, N = Elems<T>::N;
  __shared__ float sum_sh[W];
  const int64_t d = a.d, first = (int64_t)N * threadIdx.x, step = (int64_t)N * 64 * W;
  const T* w = static_cast<const T*>(a.weight);
  for (int64_t b = blockIdx.x; b < B; b += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + b * a.ld_x;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + b * a.ld_residual : nullptr;
    auto load_sum = [&](int64_t at, float (&s)[N]) {
      load_chunk<T>(x, at, d, s);
      if (r) {
        float v[N];
        load_chunk<T>(r, at, d, v);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] += v[i];
      }
    };
    float ss = 0.f;
    for (int64_t at = first; at < d; at += step) {
      float s[N];
      load_sum(at, s);
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(s[i], s[i], ss);
    }
    ss = across<W>(wave_sum(ss), sum_sh, [](float p, float q) { return p + q; });
    const float inv = 1.f / sqrtf(ss / (float)d + a.eps);
    // a chunk is read and written by one thread, x and residual before the
    // outputs that may be their own storage; every lane stays for the 128's maximum
    for (int64_t at0 = 0; at0 < d; at0 += step) {
      const int64_t at = at0 + first;
      float s[N], y[N], v[N];
      load_sum(at, s);
      if (w) load_chunk<T>(w, at, d, v);
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = w ? s[i] * inv * (a.offset + v[i]) : s[i] * inv;
      if (a.out) store_chunk<T>(static_cast<T*>(a.out) + b * a.ld_out, at, d, y);
      if (a.out_residual) store_chunk<T>(static_cast<T*>(a.out_residual) + b * a.ld_out_residual, at, d, s);
      store_fp8<T, 64>(a, b, at, y);
    }
    __syncthreads();  // sum_sh is free for the next row
  }
}

// Rows as they are: 128 / N lanes per 128 elements, over all of them in a row.
// 16384 x 2560 bfloat16, 127 MB, takes 28 us, 4.5 TB/s; 4096 x 8192 float32, 168 MB, 35
// us, 4.8; rows of 2563, whose 16 bytes are not aligned, 33 us; 1 x 2048 2.1 us.
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_quant(FP8QuantArgs a, int64_t groups, int64_t per_row) {
  constexpr int N = Elems<T>::N, L = 128 / N;
  for (int64_t i = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; i < groups; i += (int64_t)gridDim.x * (256 / L)) {
    const int64_t b = i / per_row, at = i % per_row * 128 + threadIdx.x % L * N;
    float y[N];
    load_chunk<T>(static_cast<const T*>(a.x) + b * a.ld_x, at, a.d, y);
    store_fp8<T, L>(a, b, at, y);
  }
}

// Chunks per lane that rows of these lanes and waves come to.
template <int L, int W>
constexpr int kMost = L < 64 ? 1 : W == 1 ? 6 : W == 16 ? 6 : 2;

template <typename T, int L, int W>
bool launch_w(const FP8QuantArgs& a, int64_t B, bool past, hipStream_t st) {
  const int64_t chunks = (a.d + Elems<T>::N - 1) / Elems<T>::N, c = (chunks + L * W - 1) / (L * W);
  const int64_t rows = W == 1 ? 256 / L : 1, groups = (B + rows - 1) / rows;
  const dim3 grid((unsigned)groups), block(W <= 4 ? 256 : 64 * W);
  if (groups * block.x >= int64_t(1) << 32) return false;  // more threads than a launch holds
  switch (c) {
#define FH_CASE(CC)                                                                     \
  case CC:                                                                              \
    if constexpr (CC <= kMost<L, W>) {                                                  \
      if constexpr (sizeof(T) == 2 && L == 64)                                          \
        if (past) {                                                                     \
          hipLaunchKernelGGL((k_rmsnorm_fp8<T, L, W, CC, true>), grid, block, 0, st, a, B); \
          return true;                                                                  \
        }                                                                               \
      hipLaunchKernelGGL((k_rmsnorm_fp8<T, L, W, CC, false>), grid, block, 0, st, a, B); \
      return true;                                                                      \
    }                                                                                   \
    return false;
    FH_CASE(1) FH_CASE(2) FH_CASE(3) FH_CASE(4) FH_CASE(5) FH_CASE(6)
#undef FH_CASE
    default: return false;
  }
}

// Lanes and waves per row, by its chunks of 16 bytes: the int8 norm's rule, but
// that many rows take a wave each up to six chunks a lane, as nothing waits for
// other waves behind the sum (us a call: 16384 x 2560 bfloat16 with a residual 62.2,
// in four waves 64.9; 4000 x 1152 float32 9.6 and 11.1; 8192 x 4096 in eight chunks
// 74, in four waves 52).  bfloat16 outputs of more than 64 MB pass the caches by (62.2
// -> 60.3; float32 ones lose, 3000 x 6000 50.0 -> 51.1).
template <typename T>
void launch_norm(const FP8QuantArgs& a, int64_t B, hipStream_t st) {
  const bool past = B * a.d * (int64_t)sizeof(T) > int64_t(64) << 20;
  const int64_t chunks = (a.d + Elems<T>::N - 1) / Elems<T>::N;
  const bool done = chunks <= 8                      ? launch_w<T, 8, 1>(a, B, past, st)
                    : chunks <= 16                   ? launch_w<T, 16, 1>(a, B, past, st)
                    : chunks <= 32                   ? launch_w<T, 32, 1>(a, B, past, st)
                    : chunks <= (B < 2048 ? 64 : 384) ? launch_w<T, 64, 1>(a, B, past, st)
                    : chunks <= (B < 1024 ? 256 : 384) ? launch_w<T, 64, 4>(a, B, past, st)
                    : chunks <= (B < 512 ? 512 : 1024) ? launch_w<T, 64, 8>(a, B, past, st)
                                                     : launch_w<T, 64, 16>(a, B, past, st);
  if (!done)
    hipLaunchKernelGGL((k_rmsnorm_fp8_long<T>), dim3((unsigned)std::min<int64_t>(B, 1 << 20)), dim3(1024), 0, st, a, B);
}

template <typename T>
void launch_plain(const FP8QuantArgs& a, int64_t B, hipStream_t st) {
  constexpr int kGroups = 256 / (128 / Elems<T>::N);
  const int64_t per_row = (a.d + 127) / 128, groups = B * per_row;
  const dim3 grid((unsigned)std::min<int64_t>((groups + kGroups - 1) / kGroups, 1 << 20));
  hipLaunchKernelGGL((k_fp8_quant<T>), grid, dim3(256), 0, st, a, groups, per_row);
}

}  // namespace

hipError_t launch_rmsnorm_fp8(const FP8QuantArgs& a, bool bf16, int64_t B, hipStream_t st) {
  if (bf16)
    launch_norm<uint16_t>(a, B, st);
  else
    launch_norm<float>(a, B, st);
  return hipGetLastError();
}

hipError_t launch_fp8_quant(const FP8QuantArgs& a, bool bf16, int64_t B, hipStream_t st) {
  if (bf16)
    launch_plain<uint16_t>(a, B, st);
  else
    launch_plain<float>(a, B, st);
  return hipGetLastError();
}

}  // namespace fh
