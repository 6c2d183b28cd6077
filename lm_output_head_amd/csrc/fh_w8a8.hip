// The int8 matrix product with a scale per row of both operands (W8A8),
// out[b, j] = (sum_i q[b, i] w[j, i]) (qs[b] ws[j]), and the dense head on it.
//
// v_mfma_i32_16x16x64_i8 multiplies 16 rows of W with 16 tokens over 64
// elements of k, exact in int32: lane l holds W's row l % 16 and token l % 16
// at elements 16 (l / 16) .. + 15, and the result's token l % 16 at W's rows
// 4 (l / 16) .. + 3.  W is kept in that order (fragment order), so one
// instruction's operand is one contiguous 1 KB.
//
// Few tokens are bound by the bytes of W: 1 x 128256 x 2048 in 37.8 us, 6.97 TB/s
// (a read through the caches reaches 6.3); 64 x 151936 x 2560 with float results in 84 us,
// 5.1 TB/s.  Many by how well the matrix cores are fed: 4096 x 10240 x 2560 in 114
// to 120 us, 1.8 to 1.9 POP/s (the library's product reaches 2.06 at 8192^3), where
// they are busy 47% of the cycles, at a clock that falls to 1.8 to 1.9 GHz.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fh_choice.hpp"
#include "fh_serve.hpp"

namespace fh {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Steps of 64 elements in a row of W: a multiple of kStepPad, zero past k.
constexpr int kStepPad = 2;
__host__ __device__ constexpr int w_steps(int64_t k) {
  return (int)((k + 64 * kStepPad - 1) / (64 * kStepPad) * kStepPad);
}

__device__ __forceinline__ i32x4 mfma_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

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

// The scales of a lane's rows 16 (t0 + m) + 4 g + i, zero past n.
template <int FN>
__device__ __forceinline__ void load_scales(const W8A8Args& a, int64_t t0, int g, float (&ws)[FN][4]) {
#pragma unroll
  for (int m = 0; m < FN; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t j = 16 * (t0 + m) + 4 * g + i;
      ws[m][i] = j < a.n ? a.ws[j] : 0.f;
    }
}

// A lane's 4 FN logits z[m][i] of row q, tokens 16 (t0 + m) + 4 g + i, as a Part.
template <int FN>
__device__ __forceinline__ Part choose_tile(const W8A8Args& a, const float (&z)[FN][4], int64_t q, int64_t t0, int g) {
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

// Few tokens, or too few rows for a tile per CU: 16 FN rows of W are streamed by
// KW waves, each a run of the steps of k, that take their 16 FT tokens from the
// caches and add up their sums in LDS (exact, so in any order).  A workgroup is
// G such groups.  One wave per 32 rows left loads of one step in flight: 1 x
// 128256 x 2048 45.7 -> 42.0 us, 1 x 4096 x 4096 20.8 -> 5.8, 1 x 1000 x 8192
// 41.7 -> 5.2.  PAST: the rows pass the caches by (42.0 -> 37.7).
template <int FT, int FN, int KW, int G, bool PAST, bool BF16, bool HEAD>
__global__ __launch_bounds__(64 * KW * G) void k_w8a8_few(W8A8Args a) {
  constexpr int kAhead = FN == 1 ? 4 : 2;  // steps whose loads go out together
  typedef typename Out<BF16>::T T;
  __shared__ i32x4 sums[G][KW * FN * FT * 64];
  __shared__ Part sP[HEAD ? G : 1][HEAD ? 16 * FT : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, kw = wave % KW, group = wave / KW;
  const int g = lane >> 4, col = lane & 15;
  const int64_t tiles = (a.n + 15) / 16;
  const int64_t t0 = ((int64_t)blockIdx.x * G + group) * FN;
  const int q0 = blockIdx.y * 16 * FT;
  const int steps = w_steps(a.k), chunks = (a.k + 15) / 16;

  const i32x4* wp[FN];
#pragma unroll
  for (int m = 0; m < FN; ++m) wp[m] = static_cast<const i32x4*>(a.W) + min(t0 + m, tiles - 1) * steps * 64 + lane;
  const int8_t* qp[FT];
#pragma unroll
  for (int t = 0; t < FT; ++t) qp[t] = a.q + (int64_t)min(q0 + 16 * t + col, a.B - 1) * a.ld_q;
  i32x4 acc[FN][FT];
#pragma unroll
  for (int m = 0; m < FN; ++m)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[m][t] = i32x4{0, 0, 0, 0};
  // N steps from s: their loads together, then their products.  A 16-byte chunk
  // past the row stands in as its first: W is zero there.
  auto advance = [&](auto count, int s) {
    constexpr int N = decltype(count)::value;
    i32x4 wf[N][FN], qf[N][FT];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int ch = 4 * (s + u) + g < chunks ? 4 * (s + u) + g : 0;
#pragma unroll
      for (int m = 0; m < FN; ++m) {
        const i32x4* p = wp[m] + (s + u) * 64;
        wf[u][m] = PAST ? __builtin_nontemporal_load(p) : *p;
      }
#pragma unroll
      for (int t = 0; t < FT; ++t) qf[u][t] = *reinterpret_cast<const i32x4*>(qp[t] + 16 * ch);
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int m = 0; m < FN; ++m)
#pragma unroll
        for (int t = 0; t < FT; ++t) acc[m][t] = mfma_i8(wf[u][m], qf[u][t], acc[m][t]);
  };
  const int end = (int)((int64_t)steps * (kw + 1) / KW);
  int s = (int)((int64_t)steps * kw / KW);
  for (; s + kAhead <= end; s += kAhead) advance(std::integral_constant<int, kAhead>(), s);
  for (; s < end; ++s) advance(std::integral_constant<int, 1>(), s);
#pragma unroll
  for (int m = 0; m < FN; ++m)
#pragma unroll
    for (int t = 0; t < FT; ++t) sums[group][((kw * FT + t) * FN + m) * 64 + lane] = acc[m][t];
  __syncthreads();
  float ws[FN][4];
  load_scales<FN>(a, t0, g, ws);
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    if (t % KW != kw) continue;  // the group's waves finish its token tiles in turn
    const int64_t q = q0 + 16 * t + col;
    const float qs = q < a.B ? a.qs[q] : 0.f;
    float z[FN][4];
#pragma unroll
    for (int m = 0; m < FN; ++m) {
      i32x4 v = sums[group][(t * FN + m) * 64 + lane];
#pragma unroll
      for (int w = 1; w < KW; ++w) v += sums[group][((w * FT + t) * FN + m) * 64 + lane];
      T o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[m][i] = (float)v[i] * (qs * ws[m][i]);
        o[i] = Out<BF16>::of(z[m][i]);
      }
      if (a.out && q < a.B) store_run<T, 4, false>(static_cast<T*>(a.out) + q * a.ld_out, 16 * (t0 + m) + 4 * g, a.n, o);
    }
    if (HEAD) {
      const Part p = column_choice(choose_tile<FN>(a, z, q, t0, g));
      if (g == 0) sP[group][16 * t + col] = p;
    }
  }
  if (HEAD) {
    __syncthreads();
    const int i = threadIdx.x;
    if (i < 16 * FT && q0 + i < a.B) {
      Part p = sP[0][i];
#pragma unroll
      for (int w = 1; w < G; ++w) p = choice_merge(p, sP[w][i]);
      a.parts[(int64_t)(q0 + i) * gridDim.x + blockIdx.x] = p;
    }
  }
}

// Orders this workgroup's LDS accesses around a barrier; loads from memory stay
// in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// More tokens: a workgroup of WN waves covers 16 FN WN rows by 16 FT tokens.  The
// tokens' block of kStage steps of k is staged in LDS in fragment order (a
// fragment is read as one contiguous 1 KB), double buffered and loaded one block
// ahead; each wave's rows of W go straight to registers (fragment
// order, one contiguous 1 KB per load), two blocks ahead.  PAST: the rows pass
// the caches by (64 x 151936 x 2560: 87.5 -> 83.8 us).
//
// Tiles of eight waves are held to 128 registers, two workgroups per CU: one's
// results overlap the other's products (a head of 128 x 128256 sampled went from
// 102 to 88 us by it, and later changes took it to 75; with the 250 registers of a
// 256 x 256 tile, one per CU, 4096 x 10240 x 2560 took 137 us, not 119).
//
// KW groups of WN waves share the tile: each takes a run of the blocks of k, with
// buffers of its own, and the first adds up the sums.
template <int FT, int FN, int WN, int KW, bool PAST, bool BF16, bool HEAD>
__global__ __launch_bounds__(64 * WN * KW) __attribute__((amdgpu_waves_per_eu(WN * KW == 8 ? 4 : 1))) void k_w8a8_tile(W8A8Args a, int n_tiles, int q_tiles) {
  constexpr int kStage = kStepPad, kFrags = FT * kStage;  // fragments of a token block
  constexpr int kOwn = (kFrags + WN - 1) / WN;       // of them, this wave's to stage
  constexpr int kBlock = kFrags * 64;
  typedef typename Out<BF16>::T T;
  // results of 16 tokens on their way out, two buffers
  constexpr int kRow = 16 * FN * WN + 16 / (int)sizeof(T), kTurn = 16 * kRow;
  constexpr int kShared = 2 * kBlock * 16 * KW, kStaged = 2 * kTurn * (int)sizeof(T);
  constexpr int kSums = (KW - 1) * WN * FN * FT * 64 * 16;
  __shared__ __attribute__((aligned(16))) char smem[std::max(kShared, std::max(kStaged, kSums))];
  __shared__ Part sP[HEAD ? WN : 1][HEAD ? 16 * FT : 1];

  // workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles, token
  // tiles fastest, so that its L2 keeps the rows of W that they share
  const int total = n_tiles * q_tiles, per = (total + 7) / 8;
  const int tile = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || tile >= total) return;
  const int nt = tile / q_tiles, qt = tile % q_tiles;

  const int tid = threadIdx.x, lane = tid & 63, wave = KW == 1 ? tid >> 6 : (tid >> 6) % WN, group = KW == 1 ? 0 : (tid >> 6) / WN;
  const int g = lane >> 4, col = lane & 15;
  i32x4* sQ = reinterpret_cast<i32x4*>(smem) + group * 2 * kBlock;
  const int64_t rows = (a.n + 15) / 16;
  const int64_t t0 = ((int64_t)nt * WN + wave) * FN;
  const int q0 = qt * 16 * FT;
  const int steps = w_steps(a.k), chunks = (a.k + 15) / 16;
  const int blocks = (steps / kStage + KW - 1) / KW, first = group * blocks;  // the last group's may end past the row

  const i32x4* wp[FN];
#pragma unroll
  for (int m = 0; m < FN; ++m) wp[m] = static_cast<const i32x4*>(a.W) + min(t0 + m, rows - 1) * steps * 64 + lane;
  // this wave's fragments of a block: f = step * FT + token tile
  const int8_t* qp[kOwn];
  int qs[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int f = min(wave + i * WN, kFrags - 1);
    // a token past the last stands in as the last, its results are dropped
    qp[i] = a.q + (int64_t)min(q0 + 16 * (f % FT) + col, a.B - 1) * a.ld_q;
    qs[i] = f / FT;
  }
  i32x4 qr[kOwn];
  auto load_q = [&](int blk) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      // a 16-byte chunk past the row stands in as its first: W is zero there
      const int c = 4 * (kStage * (first + blk) + qs[i]) + g;
      qr[i] = *reinterpret_cast<const i32x4*>(qp[i] + 16 * (c < chunks ? c : 0));
    }
  };
  auto store_q = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      if (kFrags % WN == 0 || wave + i * WN < kFrags) sQ[buf * kBlock + (wave + i * WN) * 64 + lane] = qr[i];
  };
  i32x4 wf[2][kStage][FN];
  auto load_w = [&](int blk, i32x4 (&dst)[kStage][FN]) {
#pragma unroll
    for (int s = 0; s < kStage; ++s)
#pragma unroll
      for (int m = 0; m < FN; ++m) {
        const i32x4* p = wp[m] + (int64_t)min(kStage * (first + blk) + s, steps - 1) * 64;
        dst[s][m] = PAST ? __builtin_nontemporal_load(p) : *p;
      }
  };
  i32x4 acc[FN][FT];
#pragma unroll
  for (int m = 0; m < FN; ++m)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[m][t] = i32x4{0, 0, 0, 0};
  auto multiply = [&](int blk, int buf, const i32x4 (&w)[kStage][FN]) {
    if (KW > 1 && kStage * (first + blk) >= steps) return;
#pragma unroll
    for (int s = 0; s < kStage; ++s) {
      i32x4 qf[FT];
#pragma unroll
      for (int t = 0; t < FT; ++t) qf[t] = sQ[buf * kBlock + (s * FT + t) * 64 + lane];
#pragma unroll
      for (int t = 0; t < FT; ++t)
#pragma unroll
        for (int m = 0; m < FN; ++m) acc[m][t] = mfma_i8(w[s][m], qf[t], acc[m][t]);
    }
  };

  // The compiler would move the loads down to the stores that take them.
  auto stay = []() { __builtin_amdgcn_sched_barrier(0); };
  // Block blk is multiplied from buffer blk % 2 while block blk + 1 travels to
  // registers; it is stored into the other buffer, which every wave has left
  // since the barrier before.  Loads past the last block repeat its last step.
  load_q(0);
  load_w(0, wf[0]);
  load_w(1, wf[1]);
  store_q(0);
  lds_barrier();
  for (int blk = 0; blk < blocks; blk += 2) {
    load_q(blk + 1);
    stay();
    multiply(blk, 0, wf[0]);
    stay();
    load_w(blk + 2, wf[0]);
    stay();
    store_q(1);
    lds_barrier();
    if (blk + 1 < blocks) {
      load_q(blk + 2);
      stay();
      multiply(blk + 1, 1, wf[1]);
      stay();
      load_w(blk + 3, wf[1]);
      stay();
      store_q(0);
      lds_barrier();
    }
  }

  // Every wave is past its last read of the blocks.  16 tokens at a time the
  // results go through LDS, so that a wave writes runs of whole rows (64 bytes
  // per token straight from the accumulators cost 22 us of 96 at 64 x 151936 and
  // 49 us of 187 at 4096 x 10240).
  if constexpr (KW > 1) {
    i32x4* sums = reinterpret_cast<i32x4*>(smem);
    if (group > 0) {
#pragma unroll
      for (int m = 0; m < FN; ++m)
#pragma unroll
        for (int t = 0; t < FT; ++t) sums[((((group - 1) * WN + wave) * FN + m) * FT + t) * 64 + lane] = acc[m][t];
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int w = 0; w < KW - 1; ++w)
#pragma unroll
        for (int m = 0; m < FN; ++m)
#pragma unroll
          for (int t = 0; t < FT; ++t) acc[m][t] += sums[(((w * WN + wave) * FN + m) * FT + t) * 64 + lane];
    }
    __syncthreads();
  }
  float ws[FN][4];
  load_scales<FN>(a, t0, g, ws);
  T* turn = reinterpret_cast<T*>(smem);
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    if (group == 0) {
      const int64_t q = q0 + 16 * t + col;
      const float qsc = q < a.B ? a.qs[q] : 0.f;
      T* row = turn + (t & 1) * kTurn + col * kRow + 16 * FN * wave + 4 * g;
      float z[FN][4];
#pragma unroll
      for (int m = 0; m < FN; ++m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) z[m][i] = (float)acc[m][t][i] * (qsc * ws[m][i]);
        typedef T V __attribute__((ext_vector_type(4)));
        V o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = Out<BF16>::of(z[m][i]);
        if (a.out) *reinterpret_cast<V*>(row + 16 * m) = o;
      }
      if (HEAD) {
        const Part p = column_choice(choose_tile<FN>(a, z, q, t0, g));
        if (g == 0) sP[wave][16 * t + col] = p;
      }
    }
    if (a.out) {
      lds_barrier();  // the other buffer is read until the barrier after this one
      constexpr int kPer = 16 / (int)sizeof(T), kRuns = 16 * FN * WN / kPer;  // 16-byte runs of a token
#pragma unroll
      for (int c = tid; c < 16 * kRuns; c += 64 * WN * KW) {
        const int tok = c / kRuns, at = c % kRuns * kPer;
        const int64_t b = q0 + 16 * t + tok;
        if (b < a.B)
          store_run<T, kPer, true>(static_cast<T*>(a.out) + b * a.ld_out, (int64_t)nt * (16 * FN * WN) + at, a.n,
                             turn + (t & 1) * kTurn + tok * kRow + at);
      }
    }
  }
  if (HEAD) {
    __syncthreads();
    for (int i = tid; i < 16 * FT && q0 + i < a.B; i += 64 * WN * KW) {
      Part p = sP[0][i];
#pragma unroll
      for (int w = 1; w < WN; ++w) p = choice_merge(p, sP[w][i]);
      a.parts[(int64_t)(q0 + i) * n_tiles + nt] = p;
    }
  }
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

// scale[j] = max |W[j]| / 127; *bad is set where a row is not finite.
template <typename T>
__global__ __launch_bounds__(256) void k_w8a8_scales(const void* W, int64_t n, int64_t k, float* scales, int* bad) {
  constexpr int N = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 63;
  for (int64_t j = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); j < n; j += (int64_t)gridDim.x * 4) {
    uint32_t top = 0u;  // |W| as bits: NaN's and infinity's are above every finite value's
    auto take = [&](float v) { top = max(top, __float_as_uint(v) & 0x7FFFFFFFu); };
    const int64_t whole = k / N * N;
    for (int64_t i = (int64_t)N * lane; i < whole; i += 64 * N) {
      float v[N];
      w_run<T, N>(W, j * k + i, v);
#pragma unroll
      for (int e = 0; e < N; ++e) take(v[e]);
    }
    if (whole + lane < k) take(w_elem<T>(W, j * k + whole + lane));
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if (lane == 0) {
      scales[j] = __uint_as_float(top) / 127.f;
      if (top >= 0x7F800000u) atomicOr(bad, 1);
    }
  }
}

// One thread per 16-byte chunk of the fragment order.
template <typename T>
__global__ __launch_bounds__(256) void k_w8a8_pack(const int8_t* codes, const void* W, const float* scales, int64_t n,
                                                   int64_t k, int64_t chunks, uint4* out) {
  const int64_t steps = w_steps(k);
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks; c += (int64_t)gridDim.x * 256) {
    const int lane = (int)(c & 63);
    const int64_t s = (c >> 6) % steps, j = (c >> 6) / steps * 16 + (lane & 15), i0 = s * 64 + (lane >> 4) * 16;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (j < n) {
      const bool whole = i0 + 16 <= k;
      if (codes && whole) {  // 16 codes as they are, at any alignment
        typedef uint32_t V __attribute__((ext_vector_type(4), aligned(1)));
        const V x = *reinterpret_cast<const V*>(codes + j * k + i0);
        out[c] = uint4{x[0], x[1], x[2], x[3]};
        continue;
      }
      const float sc = codes ? 0.f : scales[j];
      float v[16];
      if (!codes && whole) {
        w_run<T, 16>(W, j * k + i0, v);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          v[e] = i0 + e < k ? codes ? (float)codes[j * k + i0 + e] : w_elem<T>(W, j * k + i0 + e) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        int q = 0;
        if (codes)
          q = (int)v[e];
        else if (sc > 0.f)
          q = (int)fminf(fmaxf(rintf(v[e] / sc), -127.f), 127.f);
        w[e >> 2] |= ((uint32_t)q & 0xFFu) << (8 * (e & 3));
      }
    }
    out[c] = uint4{w[0], w[1], w[2], w[3]};
  }
}

__global__ __launch_bounds__(256) void k_w8a8_unpack(const int8_t* packed, int64_t n, int64_t k, int8_t* codes) {
  const int64_t steps = w_steps(k);
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

// The choice over a row's parts, 8 per thread at a time: their loads together,
// the largest m first, then every part's sum relative to it.
constexpr int kChoiceN = 8;
template <int TH>
__global__ __launch_bounds__(TH) void k_choice(const Part* parts, int64_t nparts, int32_t* out_token,
                                                    float* out_logit, float* out_lse) {
  __shared__ Part sh[TH / 64];
  const int64_t q = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Part* row = parts + q * nparts;
  Part p = part_empty();
  for (int64_t i0 = threadIdx.x; i0 < nparts; i0 += TH * kChoiceN) {
    Part v[kChoiceN];
#pragma unroll
    for (int i = 0; i < kChoiceN; ++i) v[i] = row[min(i0 + i * TH, nparts - 1)];
    float m = p.m, s = 0.f;
#pragma unroll
    for (int i = 0; i < kChoiceN; ++i) {
      if (i0 + i * TH >= nparts) v[i] = part_empty();
      choice_key(p, v[i].key, v[i].z, v[i].id);
      m = fmaxf(m, v[i].m);
    }
#pragma unroll
    for (int i = 0; i < kChoiceN; ++i) s += v[i].s * exp_from(v[i].m, m);
    p.s = p.s * exp_from(p.m, m) + s;
    p.m = m;
  }
  p = wave_choice(p);
  if (lane == 0) sh[wave] = p;
  __syncthreads();
  if (wave == 0) {
    p = wave_choice(lane < TH / 64 ? sh[lane] : part_empty());
    if (lane == 0) write_choice(p, q, out_token, out_logit, out_lse);
  }
}

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20); }

// How a call is cut up: a tile of k_w8a8_tile (named by its tokens), or a shape
// of k_w8a8_few.  x2, x4: groups that share a tile's k.
enum Kind { kFew16Rows8, kFew16Rows4, kFew16Rows2, kTokens32Rows8, kTokens32Rows4, k16, k32, k32x2, k32x4, k64, k64x2, k128 };
struct Plan {
  Kind kind;
  int rows, tokens;  // of a workgroup
  int64_t row_tiles(int64_t n) const { return (n + rows - 1) / rows; }
  int64_t token_tiles(int64_t B) const { return (B + tokens - 1) / tokens; }
  int64_t tiles(int64_t n, int64_t B) const { return row_tiles(n) * token_tiles(B); }
};
// What decides is how many waves have loads in flight: the larger a tile, the
// seldomer W and the tokens are read again, but a CU wants some eight waves of it,
// so a call takes the largest shape whose workgroups still reach most CUs (180 of
// 256 count as most), and where tiles are few the waves come from sharing k, which
// pays once each has about eight steps of it to cover its start and the joining.
//
// us a launch, weights of 400 MB together in turn, so that none is still cached
// (256 x 4096 x 8192 below takes 24.0 where three are):
// Up to 4 tokens: waves of some 8 steps of k each (1 token: 128256 x 2048 in 38.2,
// 41.6 and 41.2 us with 4, 2 and 8 waves, 262144 x 1152 in 43.9, 44.2 and 57.8,
// 40000 x 4096 in 26.9, 27.6 and 25.6); the fewer rows, the more waves (1000 x 8192
// with 8 waves 5.3 us, with 4 7.6).
// Up to 16: a wave reads its tokens once per KB of W, so they are staged in LDS
// where rows are many (16 tokens, 151936 x 2560: 69.5 us, with two waves on 32 rows
// 81.1; 128256 x 2048 46.4 and 52.3; 30001 x 6144 32.7 and 39.0).
// More: the largest tile that about fills the CUs and leaves less than half its
// tokens empty (4096 x 10240 x 2560: 114 us with 256 rows x 128 tokens, 143 with
// 256 x 64, 245 with 128 x 32).  Where that is none, tiles of 128 x 32 while k is
// short, else groups that share a tile's k, so that larger tiles still keep a CU's
// eight waves (tiles of 128 x 32, the same in two groups, 128 x 64 in two, 64 x 32
// in four; 512 x 4096 x 8192 42.8, 42.1, 36.5 and 56.7 us; 512 x 4096 x 2048 12.1,
// 13.0, 12.5 and 19.2; 256 x 4096 x 8192 38.7, 26.9, 35.4 and 30.8; 128 x 4096 x
// 8192 37.7, 26.1, 34.8 and 19.8).  Fewer tiles still: waves sharing k on 32 rows
// (128 x 4096 x 2048 7.9, 64 x 32 in four groups 8.0; 64 x 4096 x 4096 9.1 and
// 11.1) or on 16 (64 x 1000 x 8192 11.4, on 32 14.4; 32 x 6000 x 4096 12.6 and
// 10.7; 17 x 8192 x 8192, little of whose second 16 tokens is read, 17.5 and 20.8).
Plan plan_of(int64_t n, int64_t k, int64_t B) {
  constexpr int kFull = 180;  // workgroups that about fill the 256 CUs
  const int64_t tiles = (n + 15) / 16, steps = w_steps(k);
  if (B <= 16) {
    if (tiles < 512 || (B <= 4 && steps >= 44)) return Plan{kFew16Rows8, 16, 16};
    if (tiles < 2048 || (B <= 4 && steps >= 24)) return Plan{kFew16Rows4, 16, 16};
    return B <= 4 ? Plan{kFew16Rows2, 32, 16} : Plan{k16, 128, 16};
  }
  for (const Plan& p : {Plan{k128, 256, 128}, Plan{k64, 256, 64}})
    if (2 * B > p.tokens && p.tiles(n, B) >= kFull) return p;
  const Plan p{k32, 128, 32};
  const int64_t t = p.tiles(n, B);
  if (t >= 2 * kFull) return steps >= 48 && B > 32 ? Plan{k64x2, 128, 64} : p;
  if (t >= 150 && t <= 256 && steps >= 24) return Plan{k32x2, 128, 32};
  if (t >= kFull) return p;
  if (t >= 100 && steps >= 64) return Plan{k32x4, 64, 32};
  const bool narrow = B <= 24 || (t < 40 && (B <= 32 || steps >= 64));
  return narrow ? Plan{kTokens32Rows8, 16, 32} : Plan{kTokens32Rows4, 32, 32};
}

// Whether W passes the caches by: its rows are read by one workgroup alone, and
// too many to be there still at the next call, at least once other work has run.
// The more tokens, the more of the time is other than W's, and the larger the W
// that gains.  us with several weights in turn, then (one weight again and again):
//   waves sharing k: 1 x 4096 x 4096 5.3 -> 5.5 (4.4 -> 4.6), 1 x 128256 x 1024,
//     131 MB, 21.7 -> 19.8 (19.8 -> 19.0);
//   up to 32 tokens: 32 x 65536 x 1024, 67 MB, 16.1 -> 16.0 (13.7 -> 14.9), 32 x
//     128256 x 2048, 263 MB, 51.8 -> 50.3 (45.5 -> 49.2);
//   more: 64 x 65536 x 2048, 134 MB, 29.1 -> 29.9 (24.8 -> 28.5), 128 x 128256 x
//     2048 67.7 -> 71.0 (67.0 -> 69.7), 64 x 151936 x 2560, 389 MB, 87.5 -> 83.8.
bool past_caches(const Plan& p, int64_t n, int64_t k, int64_t B) {
  const int64_t from = (int64_t)(p.kind < k16 ? 64 : p.kind < k64 ? 128 : 256) << 20;
  return p.token_tiles(B) == 1 && w8a8_packed_bytes(n, k) > from;
}

template <int FT, int FN, int KW, int G, bool PAST, bool BF16, bool HEAD>
void launch_few(const W8A8Args& a, hipStream_t st) {
  constexpr int kRows = 16 * FN * G, kTokens = 16 * FT;
  const dim3 grid((unsigned)((a.n + kRows - 1) / kRows), (unsigned)((a.B + kTokens - 1) / kTokens));
  hipLaunchKernelGGL((k_w8a8_few<FT, FN, KW, G, PAST, BF16, HEAD>), grid, dim3(64 * KW * G), 0, st, a);
}

template <int FT, int FN, int WN, int KW, bool PAST, bool BF16, bool HEAD>
void launch_tile(const W8A8Args& a, hipStream_t st) {
  constexpr int kRows = 16 * FN * WN, kTokens = 16 * FT;
  const int nt = (int)((a.n + kRows - 1) / kRows), qt = (a.B + kTokens - 1) / kTokens;
  const dim3 grid((unsigned)(((int64_t)nt * qt + 7) / 8 * 8));
  hipLaunchKernelGGL((k_w8a8_tile<FT, FN, WN, KW, PAST, BF16, HEAD>), grid, dim3(64 * WN * KW), 0, st, a, nt, qt);
}

template <bool PAST, bool BF16, bool HEAD>
void launch_kind(const W8A8Args& a, Kind kind, hipStream_t st) {
  switch (kind) {
    case kFew16Rows8: return launch_few<1, 1, 8, 1, PAST, BF16, HEAD>(a, st);
    case kFew16Rows4: return launch_few<1, 1, 4, 1, PAST, BF16, HEAD>(a, st);
    case kFew16Rows2: return launch_few<1, 1, 2, 2, PAST, BF16, HEAD>(a, st);
    case kTokens32Rows8: return launch_few<2, 1, 8, 1, PAST, BF16, HEAD>(a, st);
    case kTokens32Rows4: return launch_few<2, 2, 4, 1, PAST, BF16, HEAD>(a, st);
    case k16: return launch_tile<1, 2, 4, 1, PAST, BF16, HEAD>(a, st);
    case k32: return launch_tile<2, 2, 4, 1, PAST, BF16, HEAD>(a, st);
    case k32x2: return launch_tile<2, 2, 4, 2, PAST, BF16, HEAD>(a, st);
    case k32x4: return launch_tile<2, 2, 2, 4, PAST, BF16, HEAD>(a, st);
    case k64: return launch_tile<4, 2, 8, 1, PAST, BF16, HEAD>(a, st);
    case k64x2: return launch_tile<4, 2, 4, 2, PAST, BF16, HEAD>(a, st);
    case k128: return launch_tile<8, 2, 8, 1, PAST, BF16, HEAD>(a, st);
  }
}

template <bool BF16, bool HEAD>
void launch_product(const W8A8Args& a, hipStream_t st) {
  const Plan p = plan_of(a.n, a.k, a.B);
  if (past_caches(p, a.n, a.k, a.B))
    launch_kind<true, BF16, HEAD>(a, p.kind, st);
  else
    launch_kind<false, BF16, HEAD>(a, p.kind, st);
}

}  // namespace

int64_t w8a8_packed_bytes(int64_t n, int64_t k) { return (n + 15) / 16 * w_steps(k) * 1024; }

int64_t w8a8_parts(int64_t n, int64_t k, int64_t B) { return plan_of(n, k, B).row_tiles(n); }

bool w8a8_fits(int64_t n, int64_t k, int64_t B) {
  // tiles of 512 threads; the few-token kernels' grids have the tokens in y
  const Plan p = plan_of(n, k, B);
  return p.kind < k16 || p.tiles(n, B) < (int64_t(1) << 23);
}

hipError_t launch_w8a8(const W8A8Args& a, bool out_bf16, bool head, hipStream_t st) {
  if (head)
    launch_product<false, true>(a, st);
  else if (out_bf16)
    launch_product<true, false>(a, st);
  else
    launch_product<false, false>(a, st);
  return hipGetLastError();
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
  if (nparts > 256 * kChoiceN)  // the head of 1 x 128256 x 2048, 8016 parts: 44.9 us with 1024 threads, 46.9 with 256
    hipLaunchKernelGGL(k_choice<1024>, dim3((unsigned)B), dim3(1024), 0, st, parts, nparts, out_token, out_logit, out_lse);
  else
    hipLaunchKernelGGL(k_choice<256>, dim3((unsigned)B), dim3(256), 0, st, parts, nparts, out_token, out_logit, out_lse);
  return hipGetLastError();
}

}  // namespace fh
