// Root-mean-square norm of rows with the residual's addition and an int8 output
// with a scale per row: s = x + residual, y = s / sqrt(mean(s^2) + eps) *
// (offset + weight), q = rint(y / (max |y| / 127)), all in float32 with one
// rounding per output.  Bound by the bytes of its rows: 16384 x 2560 bfloat16
// with a residual and every output (378 MB) in 74.5 us, 5.07 TB/s (a copy reaches
// 4.8 to 4.9; 266 us when each pass read the row again).  One row of 2048 takes
// 3.2 us: a load, two reductions and a store on end.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fh_device.hpp"
#include "fh_serve.hpp"

namespace fh {
namespace {

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

template <typename T>
__device__ __forceinline__ void store_chunk(T* p, int64_t at, int64_t d, const float (&v)[Elems<T>::N]) {
  constexpr int N = Elems<T>::N;
  if (at + N <= d) {
    typename Elems<T>::V x;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Elems<T>::put(v[i]);
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

// rint(t), |t| <= 127.01, as a byte: adding 1.5 2^23 leaves the integer, rounded
// to nearest even, in the low bits of the sum.
__device__ __forceinline__ uint32_t byte_of(float t) { return __float_as_uint(t + 12582912.f) & 0xFFu; }

// A row's scale, from its largest |y| in bits, and what makes its codes
// rint(y / scale), the division rounded once.  With r = 1 / scale rounded once,
// t = y r is within two units of the quotient's last place; a correction by the
// exact remainder y - t scale leaves a neighbour of the quotient and a second one
// the rounded quotient itself (Markstein 1990).  A remainder can underflow only
// where the quotient is far below a half.  16384 x 2560, all outputs: 79.0 us; 76.6
// with one product by 127 / max |y|, which misses halves, 85.4 with the division.
struct CodeScale {
  static constexpr float kSmall = 0x1p-100f, kUp = 0x1p64f;
  float scale, by, r;
  bool small;
  __device__ explicit CodeScale(uint32_t top) {
    scale = __uint_as_float(top) / 127.f;
    small = scale < kSmall;
    by = small ? scale * kUp : scale;
    r = by > 0.f ? 1.f / by : 0.f;
  }
  // A row near the subnormals is brought up for the codes; its scale has few bits,
  // so what the quotient's bounds leave is cut here.
  template <int N>
  __device__ __forceinline__ void raise(float (&y)[N]) const {
    if (!small) return;
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __builtin_amdgcn_fmed3f(y[i], -127.f * scale, 127.f * scale) * kUp;
  }
  __device__ float of(float y) const {
    float t = y * r;
    t = fmaf(fmaf(-t, by, y), r, t);
    return fmaf(fmaf(-t, by, y), r, t);
  }
};

// Codes of one chunk.
template <int N>
__device__ __forceinline__ void store_codes(int8_t* p, int64_t at, int64_t d, float (&y)[N], const CodeScale& c) {
  c.raise<N>(y);
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j)
    w[j] = byte_of(c.of(y[4 * j])) | byte_of(c.of(y[4 * j + 1])) << 8 | byte_of(c.of(y[4 * j + 2])) << 16 |
           byte_of(c.of(y[4 * j + 3])) << 24;
  if (at + N <= d) {
    typedef uint32_t W __attribute__((ext_vector_type(N / 4), aligned(1)));
    W x;
#pragma unroll
    for (int j = 0; j < N / 4; ++j) x[j] = w[j];
    *reinterpret_cast<W*>(p + at) = x;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at + i < d) p[at + i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

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

// W waves (or, W = 1, L of a wave's lanes) per row, C chunks per lane: the row
// stays in registers between its one read and the writes.  A workgroup is
// max(4, W) waves.
template <typename T, int L, int W, int C>
__global__ __launch_bounds__(W <= 4 ? 256 : 64 * W) void k_rmsnorm(NormArgs a, int64_t B) {
  static_assert(W == 1 || L == 64, "waves that share a row do so with all lanes");
  constexpr int N = Elems<T>::N, kRows = W == 1 ? 256 / L : 1, kLanes = L * W;
  static_assert(kRows == 1 || W == 1, "waves that share a row make up the workgroup");
  __shared__ float sum_sh[W];
  __shared__ uint32_t top_sh[W];
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
    for (int c = 0; c < C; ++c) store_chunk<T>(o, (int64_t)N * (lane + kLanes * c), d, y[c]);
    if (!a.out && !a.out_q) return;
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < N; ++i) ss = fmaf(y[c][i], y[c][i], ss);
  ss = across<W>(lane_sum<L>(ss), sum_sh, [](float p, float q) { return p + q; });
  const float inv = 1.f / sqrtf(ss / (float)d + a.eps);
  uint32_t top = 0u;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t at = (int64_t)N * (lane + kLanes * c);
    float v[N];
    if (w) load_chunk<T>(w, at, d, v);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      y[c][i] *= inv;
      if (w) y[c][i] *= a.offset + v[i];
      if (at + i < d) top = max(top, abs_bits(y[c][i]));
    }
    if (a.out) store_chunk<T>(static_cast<T*>(a.out) + b * a.ld_out, at, d, y[c]);
  }
  if (!a.out_q) return;
  top = across<W>(lane_umax<L>(top), top_sh, [](uint32_t p, uint32_t q) { return max(p, q); });
  const CodeScale cs(top);
  if (lane == 0) a.out_scale[b] = cs.scale;
#pragma unroll
  for (int c = 0; c < C; ++c)
    store_codes<N>(a.out_q + b * a.ld_q, (int64_t)N * (lane + kLanes * c), d, y[c], cs);
}

// Rows too long for the registers: three passes over the row, the later two from
// the caches.
template <typename T>
__global__ __launch_bounds__(1024) void k_rmsnorm_long(NormArgs a, int64_t B) {
  constexpr int W = 16, N = Elems<T>::N;
  __shared__ float sum_sh[W];
  __shared__ uint32_t top_sh[W];
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
    auto norm = [&](int64_t at, const float (&s)[N], float (&y)[N]) {
      float v[N];
      if (w) load_chunk<T>(w, at, d, v);
#pragma unroll
      for (int i = 0; i < N; ++i) y[i] = w ? s[i] * inv * (a.offset + v[i]) : s[i] * inv;
    };
    uint32_t top = 0u;
    if (a.out_q) {
      for (int64_t at = first; at < d; at += step) {
        float s[N], y[N];
        load_sum(at, s);
        norm(at, s, y);
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (at + i < d) top = max(top, abs_bits(y[i]));
      }
      top = across<W>(lane_umax<64>(top), top_sh, [](uint32_t p, uint32_t q) { return max(p, q); });
    }
    const CodeScale cs(top);
    if (a.out_q && threadIdx.x == 0) a.out_scale[b] = cs.scale;
    // a chunk is read and written by one thread, x and residual before the
    // outputs that may be their own storage
    for (int64_t at = first; at < d; at += step) {
      float s[N], y[N];
      load_sum(at, s);
      norm(at, s, y);
      if (a.out) store_chunk<T>(static_cast<T*>(a.out) + b * a.ld_out, at, d, y);
      if (a.out_residual) store_chunk<T>(static_cast<T*>(a.out_residual) + b * a.ld_out_residual, at, d, s);
      if (a.out_q) store_codes<N>(a.out_q + b * a.ld_q, at, d, y, cs);
    }
    __syncthreads();  // sum_sh and top_sh are free for the next row
  }
}

// Chunks per lane that rows of these lanes and waves come to.
template <int L, int W>
constexpr int kMost = L < 64 ? 1 : W == 1 ? 3 : W == 16 ? 6 : 2;

template <typename T, int L, int W>
bool launch_w(const NormArgs& a, int64_t B, hipStream_t st) {
  const int64_t chunks = (a.d + Elems<T>::N - 1) / Elems<T>::N, c = (chunks + L * W - 1) / (L * W);
  const int64_t rows = W == 1 ? 256 / L : 1, groups = (B + rows - 1) / rows;
  const dim3 grid((unsigned)groups), block(W <= 4 ? 256 : 64 * W);
  if (groups * block.x >= int64_t(1) << 32) return false;  // more threads than a launch holds
  switch (c) {
#define FH_CASE(CC)                                                                                     \
  case CC:                                                                                              \
    if constexpr (CC <= kMost<L, W>) {                                                                  \
      hipLaunchKernelGGL((k_rmsnorm<T, L, W, CC>), grid, block, 0, st, a, B);                           \
      return true;                                                                                      \
    }                                                                                                   \
    return false;
    FH_CASE(1) FH_CASE(2) FH_CASE(3) FH_CASE(4) FH_CASE(5) FH_CASE(6)
#undef FH_CASE
    default: return false;
  }
}

// Lanes and waves per row, by its chunks of 16 bytes (us a launch, bfloat16 with a
// residual and all outputs, three sets of buffers in turn): the fewest that keep a
// lane's chunks to one or two, more where rows are few (64 x 2560: 4.5 with 8
// waves, 5.5 with 4 or 16; 16384 x 2560: 85.7 with 4, 88.8 with 8; 16384 x 4096 110
// with 8, 111 with 4; 4096 x 16384 116 with 16, and 7 and 45% longer with the four
// or eight chunks that 8 or 4 waves would hold; 16384 x 1152 41 with one wave, 48
// with 4).
template <typename T>
void launch(const NormArgs& a, int64_t B, hipStream_t st) {
  const int64_t chunks = (a.d + Elems<T>::N - 1) / Elems<T>::N;
  const bool done = chunks <= 8                      ? launch_w<T, 8, 1>(a, B, st)
                    : chunks <= 16                   ? launch_w<T, 16, 1>(a, B, st)
                    : chunks <= 32                   ? launch_w<T, 32, 1>(a, B, st)
                    : chunks <= (B < 2048 ? 64 : 192) ? launch_w<T, 64, 1>(a, B, st)
                    : chunks <= (B < 1024 ? 256 : 384) ? launch_w<T, 64, 4>(a, B, st)
                    : chunks <= (B < 512 ? 512 : 1024) ? launch_w<T, 64, 8>(a, B, st)
                                                     : launch_w<T, 64, 16>(a, B, st);
  if (!done)
    hipLaunchKernelGGL((k_rmsnorm_long<T>), dim3((unsigned)std::min<int64_t>(B, 1 << 20)), dim3(1024), 0, st, a, B);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, bool bf16, int64_t B, hipStream_t stream) {
  if (bf16)
    launch<uint16_t>(a, B, stream);
  else
    launch<float>(a, B, stream);
  return hipGetLastError();
}

}  // namespace fh
