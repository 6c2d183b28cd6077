// The product of operands in 8-bit floating point (OCP E4M3) with a scale per 128
// of k of each token and per block of 128 x 128 of the weight,
//   out[b, j] = sum_g (sum_{i in g} q[b, i] w[j, i]) (qs[b, g] ws[j / 128, g]),
// and the dense head on it.
//
// Two instructions can do it.  Products are formed in half precision
// (v_mfma_f32_16x16x32_f16), which every code converts to exactly: exact products,
// summed in float32 (1e-8 of normally distributed results, 2-norm).  The matrix
// cores' own fp8 product (v_mfma_f32_16x16x128_f8f6f4, at twice the rate; the one
// over 32 elements rounds alike) adds up eight neighbouring products before
// anything is float32 and drops what lies 13 binades below the largest, whose power of
// two it takes from the sum of the codes' exponent fields (a subnormal code, 2^-9 say,
// has that of 2^-6, which leaves 10 binades below; 0 has none): 1.5e-5 of normally
// distributed results, 5e-5 of codes of all sizes, and all of a result
// whose large products cancel.  One bfloat16 result in ninety comes out another
// value for it.  So only a call that asks for it (fh_fp8_matmul_native, bfloat16
// results) takes it, where the matrix cores are the bound.  Either way the sum
// over one g is scaled and added to the running sum in float32, a fused
// multiply-add per result.
//
// W lies in the int8 product's order: of 16 rows and 64 elements of k one contiguous
// 1 KB, lane l's 16 bytes row l % 16 and elements 16 (l / 16) .. + 15 (any order
// of the elements will do that both operands share); the result of lane l is token
// l % 16 at W's rows 4 (l / 16) .. + 3.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fh_fp8.hpp"
#include "fh_product.hpp"
#include "fh_serve.hpp"

namespace fh {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__host__ __device__ constexpr int k_blocks(int64_t k) { return (int)((k + 127) / 128); }

__device__ __forceinline__ i32x8 both(i32x4 lo, i32x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The sum over 128 elements; scale operands of 0 select the plain instruction.
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// Eight codes in half precision, each exactly.
__device__ __forceinline__ f16x8 half_of(int lo, int hi) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// A lane's 32 codes of 128 elements as four operands.
struct Halves {
  f16x8 v[4];
  __device__ __forceinline__ Halves() {}
  __device__ __forceinline__ Halves(i32x4 lo, i32x4 hi)
      : v{half_of(lo[0], lo[1]), half_of(lo[2], lo[3]), half_of(hi[0], hi[1]), half_of(hi[2], hi[3])} {}
};
__device__ __forceinline__ f32x4 mfma_half(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ void add_scaled(f32x4& acc, f32x4 part, float scale) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = fmaf(part[i], scale, acc[i]);
}

// Few tokens, or too few rows for a tile per CU: 16 FN rows of W are streamed by
// KW waves, each a run of the blocks of k, that take their 16 FT tokens from the
// caches and add up their sums in LDS, in one order.  A workgroup is G such
// groups.  PAST: the rows pass the caches by.
// One token is a read of W: 128256 x 2048 takes 37.5 us, 7.0 TB/s, so half precision
// and its conversions cost nothing that shows; two blocks' loads go out
// together (one at a time 1.5 us more).
template <int FT, int FN, int KW, int G, bool PAST, bool BF16, bool HEAD>
__global__ __launch_bounds__(64 * KW * G) void k_fp8_few(FP8Args a) {
  constexpr int kAhead = FN == 1 ? 2 : 1;  // blocks whose loads go out together
  typedef typename Out<BF16>::T T;
  __shared__ f32x4 sums[G][KW * FN * FT * 64];
  __shared__ Part sP[HEAD ? G : 1][HEAD ? 16 * FT : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave % KW, group = wave / KW;
  const int g = lane >> 4, col = lane & 15;
  const int64_t tiles = (a.n + 15) / 16;
  const int64_t t0 = ((int64_t)blockIdx.x * G + group) * FN;
  const int q0 = blockIdx.y * 16 * FT;
  const int blocks = k_blocks(a.k), chunks = (a.k + 15) / 16;

  const i32x4* wp[FN];
  const float* sp[FN];
#pragma unroll
  for (int m = 0; m < FN; ++m) {
    const int64_t tile = min(t0 + m, tiles - 1);
    wp[m] = static_cast<const i32x4*>(a.W) + tile * blocks * 128 + lane;
    sp[m] = a.ws + tile / 8 * blocks;
  }
  const uint8_t* qp[FT];
  const float* qsp[FT];
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    const int64_t q = min(q0 + 16 * t + col, a.B - 1);
    qp[t] = a.q + q * a.ld_q;
    qsp[t] = a.qs + q * a.ld_qs;
  }
  f32x4 acc[FN][FT];
#pragma unroll
  for (int m = 0; m < FN; ++m)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // N blocks from s: their loads together, then their products.  A 16-byte chunk
  // past the row stands in as its first: W is zero there, and a NaN in that chunk
  // is in the row's every result anyway.
  auto advance = [&](auto count, int s) {
    constexpr int N = decltype(count)::value;
    i32x4 wf[N][FN][2], qf[N][FT][2];
    float qs[N][FT], ws[N][FN];
#pragma unroll
    for (int u = 0; u < N; ++u) {
#pragma unroll
      for (int m = 0; m < FN; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const i32x4* p = wp[m] + (s + u) * 128 + 64 * h;
          wf[u][m][h] = PAST ? __builtin_nontemporal_load(p) : *p;
        }
        ws[u][m] = sp[m][s + u];
      }
#pragma unroll
      for (int t = 0; t < FT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ch = 8 * (s + u) + 4 * h + g;
          qf[u][t][h] = *reinterpret_cast<const i32x4*>(qp[t] + 16 * (ch < chunks ? ch : 0));
        }
        qs[u][t] = qsp[t][s + u];
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      Halves w[FN];
#pragma unroll
      for (int m = 0; m < FN; ++m) w[m] = Halves(wf[u][m][0], wf[u][m][1]);
#pragma unroll
      for (int t = 0; t < FT; ++t) {
        const Halves q(qf[u][t][0], qf[u][t][1]);
#pragma unroll
        for (int m = 0; m < FN; ++m) {
          f32x4 part{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 4; ++h) part = mfma_half(w[m].v[h], q.v[h], part);
          add_scaled(acc[m][t], part, qs[u][t] * ws[u][m]);
        }
      }
    }
  };
  const int end = (int)((int64_t)blocks * (kw + 1) / KW);
  int s = (int)((int64_t)blocks * kw / KW);
  for (; s + kAhead <= end; s += kAhead) advance(std::integral_constant<int, kAhead>(), s);
  for (; s < end; ++s) advance(std::integral_constant<int, 1>(), s);
#pragma unroll
  for (int m = 0; m < FN; ++m)
#pragma unroll
    for (int t = 0; t < FT; ++t) sums[group][((kw * FT + t) * FN + m) * 64 + lane] = acc[m][t];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    if (t % KW != kw) continue;  // the group's waves finish its token tiles in turn
    const int64_t q = q0 + 16 * t + col;
    float z[FN][4];
#pragma unroll
    for (int m = 0; m < FN; ++m) {
      f32x4 v = sums[group][(t * FN + m) * 64 + lane];
#pragma unroll
      for (int w = 1; w < KW; ++w) v += sums[group][((w * FT + t) * FN + m) * 64 + lane];
      T o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[m][i] = v[i];
        o[i] = Out<BF16>::of(v[i]);
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

// More tokens: a workgroup of WN waves covers 16 FN WN rows by 16 FT tokens.  A
// block of 128 of k of the tokens is staged in LDS in fragment order with its
// scales, double buffered and loaded one block ahead; each wave's rows of W go
// straight to registers, one or two blocks ahead.  KW groups of WN waves share the
// tile: each takes a run of the blocks of k, with buffers of its own, and the first
// adds up the sums.  HALF: in half precision, which the tokens are staged in and
// each wave's rows of W are converted to as they are used.
//
// 64 rows of a wave (FN = 4) halve what it reads of LDS for a product; their sums
// take half the registers, so two waves share a SIMD, and W has room for one block
// alone: a row's registers are loaded again right behind their last use, and the
// other wave covers the wait.
// Native (128 tokens) 4096 x 10240 x 2560 in us: 132 with 32 rows of eight waves; 118 with 64 of four; 109 with tokens read in
// whole lines (16 rows of 64 bytes a load before) and eight neighbouring row tiles
// of a panel at once; 102 with those loads spread over the products and sums three
// products behind (2.1 PFLOP/s; the library's fp8 product without scales per block
// takes 122).  Without any load it would take 82, without the multiply-adds of
// the scales too 67: the matrix cores are busy 63% of the cycles, at 1.75 GHz.
// In half precision (64 tokens) 4096 x 10240 x 2560 takes 190 us, 1.13 PFLOP/s: the
// matrix cores are busy 51% of the cycles.  300 x 100000 x 1024 takes 80 us, 0.77 PFLOP/s, and 82
// with W's 64 rows converted at once and two blocks of them.  128 x 262144 x 1152 with
// neither results nor draws takes 98: 86 with W from the caches, and some 5 less each
// without the tokens' loads, the multiply-adds or the conversions; 66 with products
// alone.  Work between each two products by hand gave nothing.
// 32 rows of eight waves, whose next W is on its way before the products: 64 x 151936
// x 2560 84 us, 88 with its loads behind them, the rate of a copy.
template <int FT, int FN, int WN, int KW, bool HALF, bool PAST, bool BF16, bool HEAD>
__global__ __launch_bounds__(64 * WN * KW) __attribute__((amdgpu_waves_per_eu(FN == 4 || WN * KW == 8 ? 2 : 1))) void k_fp8_tile(FP8Args a, int n_tiles, int q_tiles) {
  constexpr int kFrags = 2 * FT;                // 1 KB of codes each, of a token block
  constexpr int kBlock = kFrags * 64 * (HALF ? 2 : 1);
  constexpr int kDepth = FN == 4 ? 1 : 2;  // blocks of W in registers
  // a row's next load goes out as soon as its registers are free, not behind the
  // block's products
  constexpr bool kEarly = FN * WN == 16;
  static_assert(kEarly ? KW == 1 : kDepth == 2, "a block that is not multiplied loads nothing");
  static_assert(FT * 16 <= 64 * WN, "a thread of a group per token scale");
  static_assert(8 % FN == 0, "a wave's rows lie in one block of 128");
  typedef typename Out<BF16>::T T;
  // results of 16 tokens on their way out, two buffers
  constexpr int kRow = 16 * FN * WN + 16 / (int)sizeof(T), kTurn = 16 * kRow;
  constexpr int kShared = 2 * kBlock * 16 * KW, kStaged = 2 * kTurn * (int)sizeof(T);
  constexpr int kSums = (KW - 1) * WN * FN * FT * 64 * 16;
  __shared__ __attribute__((aligned(16))) char smem[std::max(kShared, std::max(kStaged, kSums))];
  __shared__ float sScale[KW][2][16 * FT];
  __shared__ Part sP[HEAD ? WN : 1][HEAD ? 16 * FT : 1];

  // workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles, by panels of
  // eight row tiles, so that its L2 keeps what neighbours share
  const int total = n_tiles * q_tiles, per = (total + 7) / 8;
  const int tile = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || tile >= total) return;
  constexpr int kPanel = 8;
  const int panel = tile / (kPanel * q_tiles), in = tile % (kPanel * q_tiles);
  const int wide = min(kPanel, n_tiles - panel * kPanel);
  const int nt = panel * kPanel + in % wide, qt = in / wide;

  const int tid = threadIdx.x, lane = tid & 63, all = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = all % WN, group = all / WN;
  const int g = lane >> 4, col = lane & 15;
  i32x4* sQ = reinterpret_cast<i32x4*>(smem) + group * 2 * kBlock;
  const int64_t rows = (a.n + 15) / 16;
  const int64_t t0 = ((int64_t)nt * WN + wave) * FN;
  const int q0 = qt * 16 * FT;
  const int steps = k_blocks(a.k), chunks = (a.k + 15) / 16;
  const int blocks = (steps + KW - 1) / KW, first = group * blocks;  // the last group's may end past the row

  const i32x4* wp[FN];
#pragma unroll
  for (int m = 0; m < FN; ++m) wp[m] = static_cast<const i32x4*>(a.W) + min(t0 + m, rows - 1) * steps * 128 + lane;
  const float* sp = a.ws + min(t0, rows - 1) / 8 * steps;
  // A block's chunks of 16 codes go to the group's threads in the order of the
  // tokens' rows, so that eight lanes read 128 bytes of one; in LDS chunk g of half h
  // of token `col` stands at 16 g + (col ^ (g + 4 h)) of its fragment, which spreads
  // those eight over the banks.
  const int mine = tid - group * 64 * WN;  // this thread in its group
  constexpr int kOwn = (128 * FT + 64 * WN - 1) / (64 * WN);
  constexpr bool kAllOwn = 128 * FT % (64 * WN) == 0;  // else some threads stage nothing
  const uint8_t* qp[kOwn];
  int qs_at[kOwn];
  const int qc = mine & 7;  // its chunk of the 128
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int row = min(i * 8 * WN + (mine >> 3), 16 * FT - 1);
    // a token past the last stands in as the last, its results are dropped
    qp[i] = a.q + (int64_t)min(q0 + row, a.B - 1) * a.ld_q;
    qs_at[i] = ((HALF ? 2 : 1) * (qc >> 2) * FT + row / 16) * 64 + 16 * (qc & 3) + ((row & 15) ^ qc);
  }
  int at_half[2];  // where this lane's chunk stands in a fragment of either half
#pragma unroll
  for (int h = 0; h < 2; ++h) at_half[h] = 16 * g + (col ^ (g + 4 * h));
  const float* qsp = a.qs + (int64_t)min(q0 + min(mine, 16 * FT - 1), a.B - 1) * a.ld_qs;
  i32x4 qr[kOwn];
  float sr;
  auto load_own = [&](int blk, int i) {
    // a 16-byte chunk past the row stands in as its first (see k_fp8_few)
    const int c = 8 * (first + blk) + qc;
    qr[i] = *reinterpret_cast<const i32x4*>(qp[i] + 16 * (c < chunks ? c : 0));
    if (i == 0) sr = qsp[min(first + blk, steps - 1)];
  };
  auto load_q = [&](int blk) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) load_own(blk, i);
  };
  auto store_q = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      if (!kAllOwn && i * 8 * WN + (mine >> 3) >= 16 * FT) continue;
      i32x4* at = sQ + buf * kBlock + qs_at[i];
      if constexpr (HALF) {
        *reinterpret_cast<f16x8*>(at) = half_of(qr[i][0], qr[i][1]);
        *reinterpret_cast<f16x8*>(at + FT * 64) = half_of(qr[i][2], qr[i][3]);
      } else {
        *at = qr[i];
      }
    }
    if (mine < 16 * FT) sScale[group][buf][mine] = sr;
  };
  i32x4 wf[kDepth][FN][2];
  float wsc[2];
  auto load_frag = [&](int blk, int m, i32x4 (&dst)[2]) {
    const int at = min(first + blk, steps - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const i32x4* p = wp[m] + (int64_t)at * 128 + 64 * h;
      dst[h] = PAST ? __builtin_nontemporal_load(p) : *p;
    }
  };
  auto load_w = [&](int blk, i32x4 (&dst)[FN][2], float& s) {
#pragma unroll
    for (int m = 0; m < FN; ++m) load_frag(blk, m, dst[m]);
    s = sp[min(first + blk, steps - 1)];
  };
  f32x4 acc[FN][FT];
#pragma unroll
  for (int m = 0; m < FN; ++m)
#pragma unroll
    for (int t = 0; t < FT; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Block blk from buffer `buf`; where kEarly, its registers and scale are then
  // block blk + kDepth's.
  auto multiply = [&](int blk, int buf, i32x4 (&w)[FN][2], float& scale) {
    if (KW > 1 && first + blk >= steps) return;
    const float ws = scale;
    if constexpr (kEarly) scale = sp[min(first + blk + kDepth, steps - 1)];
    if constexpr (HALF && FN == 4) {
      // the tokens stay in registers, and W is converted 16 rows at a time
      const f16x8* q = reinterpret_cast<const f16x8*>(sQ + buf * kBlock);
      f16x8 qf[FT][4];
      float sc[FT];
#pragma unroll
      for (int t = 0; t < FT; ++t) {
#pragma unroll
        for (int h = 0; h < 4; ++h) qf[t][h] = q[(h * FT + t) * 64 + at_half[h >> 1]];
        sc[t] = sScale[group][buf][16 * t + col] * ws;
      }
#pragma unroll
      for (int m = 0; m < FN; ++m) {
        const Halves wh(w[m][0], w[m][1]);
        load_frag(blk + kDepth, m, w[m]);
        f32x4 part[FT];
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int t = 0; t < FT; ++t)
            part[t] = mfma_half(wh.v[h], qf[t][h], h == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : part[t]);
#pragma unroll
        for (int t = 0; t < FT; ++t) add_scaled(acc[m][t], part[t], sc[t]);
      }
    } else if constexpr (HALF) {
      Halves wh[FN];
#pragma unroll
      for (int m = 0; m < FN; ++m) {
        wh[m] = Halves(w[m][0], w[m][1]);
        if constexpr (kEarly) {
          __builtin_amdgcn_sched_barrier(0);
          load_frag(blk + kDepth, m, w[m]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int t = 0; t < FT; ++t) {
        const float sc = sScale[group][buf][16 * t + col] * ws;
        const f16x8* q = reinterpret_cast<const f16x8*>(sQ + buf * kBlock) + t * 64;
        f32x4 part[FN];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const f16x8 qf = q[h * FT * 64 + at_half[h >> 1]];
#pragma unroll
          for (int m = 0; m < FN; ++m)
            part[m] = mfma_half(wh[m].v[h], qf, h == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : part[m]);
        }
#pragma unroll
        for (int m = 0; m < FN; ++m) add_scaled(acc[m][t], part[m], sc);
      }
    } else {
      // the next tokens are read while these are multiplied, and a product is added
      // up three products later; with one block of W, so are the loads for the next
      static_assert(kDepth == 2 || 4 * kOwn <= FN * FT, "the loads fit between the products");
      constexpr int kBehind = 3;
      i32x8 qf[2];
      float sc[4];  // of three tokens in use, while a fourth comes
      f32x4 part[kBehind + 1];
      auto load = [&](int t) {
        qf[t & 1] = both(sQ[buf * kBlock + t * 64 + at_half[0]], sQ[buf * kBlock + (FT + t) * 64 + at_half[1]]);
        sc[t % 4] = sScale[group][buf][16 * t + col];
      };
      load(0);
#pragma unroll
      for (int i = 0; i < FN * FT + kBehind; ++i) {
        if (i % FN == 0 && i / FN + 1 < FT) load(i / FN + 1);
        if (i < FN * FT) part[i % (kBehind + 1)] = mfma_fp8(both(w[i % FN][0], w[i % FN][1]), qf[i / FN & 1]);
        if (kDepth == 1 && i % 4 == 2 && i / 4 < kOwn) load_own(blk + 1, i / 4);
        if (kEarly && i >= FN * (FT - 1) && i < FN * FT) load_frag(blk + kDepth, i % FN, w[i % FN]);
        if (i >= kBehind) {
          const int b = i - kBehind;
          if (b % FN == 0) sc[b / FN % 4] *= ws;
          add_scaled(acc[b % FN][b / FN], part[b % (kBehind + 1)], sc[b / FN % 4]);
          asm volatile("" : "+v"(acc[b % FN][b / FN]));  // here, not behind the next barrier
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // The compiler would move the loads down to the stores that take them.
  auto stay = []() { __builtin_amdgcn_sched_barrier(0); };
  // Block blk is multiplied from buffer blk % 2 while block blk + 1 travels to
  // registers; it is stored into the other buffer, which every wave has left
  // since the barrier before.  Loads past the last block repeat it.
  load_q(0);
  load_w(0, wf[0], wsc[0]);
  if constexpr (kDepth == 1) {
    store_q(0);
    lds_barrier();
    for (int blk = 0; blk < blocks; ++blk) {
      if constexpr (HALF) load_q(blk + 1);
      stay();
      multiply(blk, blk & 1, wf[0], wsc[0]);
      stay();
      store_q((blk + 1) & 1);
      lds_barrier();
    }
  } else {
    load_w(1, wf[kDepth - 1], wsc[1]);
    store_q(0);
    lds_barrier();
    for (int blk = 0; blk < blocks; blk += 2) {
      load_q(blk + 1);
      stay();
      multiply(blk, 0, wf[0], wsc[0]);
      stay();
      if constexpr (!kEarly) load_w(blk + 2, wf[0], wsc[0]);
      stay();
      store_q(1);
      lds_barrier();
      if (blk + 1 < blocks) {
        load_q(blk + 2);
        stay();
        multiply(blk + 1, 1, wf[kDepth - 1], wsc[1]);
        stay();
        if constexpr (!kEarly) load_w(blk + 3, wf[kDepth - 1], wsc[1]);
        stay();
        store_q(0);
        lds_barrier();
      }
    }
  }

  // Every wave is past its last read of the blocks.
  if constexpr (KW > 1) {
    f32x4* sums = reinterpret_cast<f32x4*>(smem);
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
  // 16 tokens at a time the results go through LDS, so that a wave writes runs of
  // whole rows.
  T* turn = reinterpret_cast<T*>(smem);
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    if (group == 0) {
      const int64_t q = q0 + 16 * t + col;
      T* row = turn + (t & 1) * kTurn + col * kRow + 16 * FN * wave + 4 * g;
      float z[FN][4];
#pragma unroll
      for (int m = 0; m < FN; ++m) {
        typedef T V __attribute__((ext_vector_type(4)));
        V o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[m][i] = acc[m][t][i];
          o[i] = Out<BF16>::of(z[m][i]);
        }
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

// scale of each block of 128 x 128: max |W| / 448; *bad is set where a block is
// not finite.  128256 x 2048 bfloat16, 525 MB, takes 118 us, 4.4 TB/s; its codes (below),
// 788 MB, 134 us, 5.9 TB/s.  A weight is made once.
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_scales(const void* W, int64_t n, int64_t k, float* scales, int* bad) {
  __shared__ uint32_t sh[4];
  const int64_t G = (k + 127) / 128, total = (n + 127) / 128 * G;
  const int tid = threadIdx.x;
  for (int64_t blk = blockIdx.x; blk < total; blk += gridDim.x) {
    const int64_t j0 = blk / G * 128, i0 = blk % G * 128;
    const int64_t j1 = min(j0 + 128, n), i1 = min(i0 + 128, k);
    uint32_t top = 0u;  // |W| as bits: NaN's and infinity's are above every finite value's
    constexpr int N = 16 / (int)sizeof(T), kLanes = 128 / N;
    const int64_t i = i0 + tid % kLanes * N;
    for (int64_t j = j0 + tid / kLanes; j < j1; j += 256 / kLanes) {
      if (i + N <= i1) {
        float v[N];
        w_run<T, N>(W, j * k + i, v);
#pragma unroll
        for (int e = 0; e < N; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
      } else {
        for (int64_t e = i; e < i1; ++e) top = max(top, __float_as_uint(w_elem<T>(W, j * k + e)) & 0x7FFFFFFFu);
      }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if ((tid & 63) == 0) sh[tid >> 6] = top;
    __syncthreads();
    if (tid == 0) {
      top = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
      scales[blk] = __uint_as_float(top) / 448.f;
      if (top >= 0x7F800000u) atomicOr(bad, 1);
    }
    __syncthreads();  // sh is free for the next block
  }
}

// One thread per 16-byte chunk of the fragment order: codes of W under scales.
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_pack(const void* W, const float* scales, int64_t n, int64_t k,
                                                  int64_t chunks, uint4* out) {
  const int64_t G = (k + 127) / 128;
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks; c += (int64_t)gridDim.x * 256) {
    const int lane = (int)(c & 63);
    const int64_t s = (c >> 6) % (2 * G), j = (c >> 6) / (2 * G) * 16 + (lane & 15), i0 = s * 64 + (lane >> 4) * 16;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (j < n && i0 < k) {
      float v[16];
      if (i0 + 16 <= k) {
        w_run<T, 16>(W, j * k + i0, v);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = i0 + e < k ? w_elem<T>(W, j * k + i0 + e) : 0.f;
      }
      const E4M3Scale sc(scales[j / 128 * G + i0 / 128]);
      sc.raise<16>(v);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = e4m3_of(sc.of(v[4 * e]), sc.of(v[4 * e + 1]), sc.of(v[4 * e + 2]), sc.of(v[4 * e + 3]));
    }
    out[c] = uint4{w[0], w[1], w[2], w[3]};
  }
}

// How a call is cut up: a tile of k_fp8_tile (named by its tokens), or a shape of
// k_fp8_few.  x2, x4: groups that share a tile's k.  Native: in the matrix cores'
// own fp8.
enum Kind {
  kFew16Rows8, kFew16Rows4, kFew16Rows2, kTokens32Rows8, kTokens32Rows4,
  k16, k32, k32x2, k32x4, k64, k64x2, kWide64, k64Native, k64x2Native, k128Native
};
struct Plan {
  Kind kind;
  int rows, tokens;  // of a workgroup
  int64_t row_tiles(int64_t n) const { return (n + rows - 1) / rows; }
  int64_t token_tiles(int64_t B) const { return (B + tokens - 1) / tokens; }
  int64_t tiles(int64_t n, int64_t B) const { return row_tiles(n) * token_tiles(B); }
};
// As for the int8 product the larger a tile, the seldomer W and the tokens are read
// again, but a CU wants some eight waves with loads in flight, so a call takes the
// largest shape whose workgroups still reach most CUs (180 of 256 count as most).
//
// us a call, back to back, weights of 500 MB together in turn (calls below some 8 us
// are the host's time):
// Up to 8 tokens: waves that share k, some 8 blocks of 64 each (1 token: 128256 x
// 2048 37.5 with 4 waves, 40.8 and 42.5 with 2 and 8; 262144 x 1152 43.6 with 2, 44.2
// and 56.0 with 4 and 8).  Up to 16 tokens staged in LDS where rows are many (16
// tokens, 128256 x 2048: 47.7, with two waves on 16 rows 54.7; 8 tokens 46.3 and 42.1).
// More: 256 x 64, by four waves of 64 rows where many tokens fill the CUs (float32
// results: 300 x 100000 x 1024 80, by eight of 32 rows 93 and with 128 tokens 97; 1000 x
// 12000 x 2048 52.9 and 59.7; 500 x 8000 x 1024 15.4 and 12.9; bfloat16 ones: 4096 x
// 10240 x 2560 190 and 222, 2048 x 4096 x 2048 32.7 and 37.9, 1000 x 4096 x 2048 22.2
// and 19.5), by eight of 32 else (64 x 151936 x 2560 84, by four 89).
// Smaller calls as the int8 product's, whose borders hold here within some 10%, us in a
// graph by the shape that is taken and by the nearest other: 1 x 10000 x 2048 6.4 (R4) and
// 7.0 (R8); 16 x 6000 x 2048 7.0 (R8) and 6.1 (R4); 40000 x 2048 by 1 token 14.0 (R2) and
// 13.6 (R4); 4 x 60000 x 2944 29.2 (R8) and 26.9 (R4); 12 x 128256 x 2048 45.4 (16 tokens)
// and 47.6 (R2); 64 x 10000 x 2048 11.4 (32x2) and 13.6 (32); 64 x 12000 x 1024 9.0 (32)
// and 8.3 (32x2); 64 x 25000 x 4096 27.3 (64x2) and 32.1 (32); 64 x 7000 x 4096 13.4
// (32x4) and 17.9 (32x2); 30 x 5000 x 2048 7.6 (32 rows, T4) and 8.1 (T8).  Another shape
// would be faster by more where k is just too short for the groups that share it: 48 x
// 24000 x 2944 24.8 (32) and 20.4 (64x2), 60 x 2000 x 2048 6.3 (T4) and 5.2 (T8), 64 x 7000
// x 2048 10.6 (T4) and 9.4 (32x4).
// Native: 256 rows x 128 tokens (4096 x 10240 x 2560 102, 2048 x 4096 x 2048
// 21.9, with 256 x 64 23.1; 80 x 262144 x 1152 62.6 and 75.7; of two blocks of k alone,
// 500 x 14260 x 256, 12.6 and 8.3); 256 x 64 (1000 x 4096 x 2048 14.2, with 128 x 64
// in two groups 17.9); where those are few, groups that share the k of 128 x 64 (333 x
// 5003 x 1152 8.8, with 256 x 64 10.1, with 128 x 32 11.9; 64 x 20000 x 4096 24.0, 33.0
// and 30.1), down to some 100 of them (128 x 4096 x 8192 23.7, 17.4 with 64 x 32 in
// four groups); else as the others.
Plan plan_of(int64_t n, int64_t k, int64_t B, bool native) {
  constexpr int kFull = 180;  // workgroups that about fill the 256 CUs
  const int64_t tiles = (n + 15) / 16, blocks = k_blocks(k), steps = 2 * blocks;
  if (B <= 16) {
    if (tiles < 512 || (B <= 8 && steps >= 44)) return Plan{kFew16Rows8, 16, 16};
    if (tiles < 2048 || (B <= 8 && steps >= 24)) return Plan{kFew16Rows4, 16, 16};
    return B <= 8 ? Plan{kFew16Rows2, 32, 16} : Plan{k16, 128, 16};
  }
  const Plan big{k128Native, 256, 128}, mid{native ? k64Native : k64, 256, 64}, shared{k64x2Native, 128, 64};
  if (native && B > 64 && blocks >= 4 && big.tiles(n, B) >= kFull) return big;
  if (!native && B > 64 && mid.tiles(n, B) >= 400) return Plan{kWide64, 256, 64};
  if (B > 32 && mid.tiles(n, B) >= kFull) return mid;
  if (native && B > 32 && blocks >= 4 && shared.tiles(n, B) >= 100) return shared;
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
// too many to be there still at the next call (the int8 product's borders, between
// calls on other data).  One weight again and again, with nothing between, us past the
// caches and by them: one token 64 MB 9.8 and 10.9, 256 MB 35.4 and 35.7, 400 MB 55 and
// 64; 8 tokens 100 MB 17.2 and 16.3, 256 MB 41.6 and 37.2, 400 MB 71 and 77; 64 tokens 256
// MB 52.4 and 48.3, 400 MB 82.1 and 83.7.
bool past_caches(const Plan& p, int64_t n, int64_t k, int64_t B) {
  const int64_t from = (int64_t)(p.kind < k16 ? 64 : p.kind < k64 ? 128 : 256) << 20;
  return p.token_tiles(B) == 1 && w8a8_packed_bytes(n, k) > from;
}

template <int FT, int FN, int KW, int G, bool PAST, bool BF16, bool HEAD>
void launch_few(const FP8Args& a, hipStream_t st) {
  constexpr int kRows = 16 * FN * G, kTokens = 16 * FT;
  const dim3 grid((unsigned)((a.n + kRows - 1) / kRows), (unsigned)((a.B + kTokens - 1) / kTokens));
  hipLaunchKernelGGL((k_fp8_few<FT, FN, KW, G, PAST, BF16, HEAD>), grid, dim3(64 * KW * G), 0, st, a);
}

template <int FT, int FN, int WN, int KW, bool HALF, bool PAST, bool BF16, bool HEAD>
void launch_tile(const FP8Args& a, hipStream_t st) {
  constexpr int kRows = 16 * FN * WN, kTokens = 16 * FT;
  const int nt = (int)((a.n + kRows - 1) / kRows), qt = (a.B + kTokens - 1) / kTokens;
  const dim3 grid((unsigned)(((int64_t)nt * qt + 7) / 8 * 8));
  hipLaunchKernelGGL((k_fp8_tile<FT, FN, WN, KW, HALF, PAST, BF16, HEAD>), grid, dim3(64 * WN * KW), 0, st, a, nt, qt);
}

template <bool PAST, bool BF16, bool HEAD>
void launch_kind(const FP8Args& a, Kind kind, hipStream_t st) {
  switch (kind) {
    case kFew16Rows8: return launch_few<1, 1, 8, 1, PAST, BF16, HEAD>(a, st);
    case kFew16Rows4: return launch_few<1, 1, 4, 1, PAST, BF16, HEAD>(a, st);
    case kFew16Rows2: return launch_few<1, 1, 2, 2, PAST, BF16, HEAD>(a, st);
    case kTokens32Rows8: return launch_few<2, 1, 8, 1, PAST, BF16, HEAD>(a, st);
    case kTokens32Rows4: return launch_few<2, 2, 4, 1, PAST, BF16, HEAD>(a, st);
    case k16: return launch_tile<1, 2, 4, 1, true, PAST, BF16, HEAD>(a, st);
    case k32: return launch_tile<2, 2, 4, 1, true, PAST, BF16, HEAD>(a, st);
    case k32x2: return launch_tile<2, 2, 4, 2, true, PAST, BF16, HEAD>(a, st);
    case k32x4: return launch_tile<2, 2, 2, 4, true, PAST, BF16, HEAD>(a, st);
    case k64: return launch_tile<4, 2, 8, 1, true, PAST, BF16, HEAD>(a, st);
    case k64x2: return launch_tile<4, 2, 4, 2, true, PAST, BF16, HEAD>(a, st);
    case kWide64: return launch_tile<4, 4, 4, 1, true, PAST, BF16, HEAD>(a, st);
    default: break;
  }
  if constexpr (BF16) switch (kind) {
    case k64Native: return launch_tile<4, 2, 8, 1, false, PAST, BF16, HEAD>(a, st);
    case k64x2Native: return launch_tile<4, 2, 4, 2, false, PAST, BF16, HEAD>(a, st);
    case k128Native: return launch_tile<8, 4, 4, 1, false, PAST, BF16, HEAD>(a, st);
    default: break;
  }
}

template <bool BF16, bool HEAD>
void launch_product(const FP8Args& a, bool native, hipStream_t st) {
  const Plan p = plan_of(a.n, a.k, a.B, native);
  if (past_caches(p, a.n, a.k, a.B))
    launch_kind<true, BF16, HEAD>(a, p.kind, st);
  else
    launch_kind<false, BF16, HEAD>(a, p.kind, st);
}

}  // namespace

int64_t fp8_parts(int64_t n, int64_t k, int64_t B) { return plan_of(n, k, B, false).row_tiles(n); }

bool fp8_fits(int64_t n, int64_t k, int64_t B) {
  // tiles of 512 threads; the few-token kernels' grids have the tokens in y
  for (bool native : {false, true}) {
    const Plan p = plan_of(n, k, B, native);
    if (p.kind >= k16 && p.tiles(n, B) >= int64_t(1) << 23) return false;
  }
  return true;
}

hipError_t launch_fp8(const FP8Args& a, FP8Out out, hipStream_t st) {
  if (out == FP8Out::kHead)
    launch_product<false, true>(a, false, st);
  else if (out == FP8Out::kF32)
    launch_product<false, false>(a, false, st);
  else
    launch_product<true, false>(a, out == FP8Out::kBf16Native, st);
  return hipGetLastError();
}

hipError_t launch_fp8_scales(const void* W, bool bf16, int64_t n, int64_t k, float* scales, int* bad, hipStream_t st) {
  const dim3 grid((unsigned)std::min<int64_t>((n + 127) / 128 * k_blocks(k), 1 << 20));
  if (bf16)
    hipLaunchKernelGGL((k_fp8_scales<uint16_t>), grid, dim3(256), 0, st, W, n, k, scales, bad);
  else
    hipLaunchKernelGGL((k_fp8_scales<float>), grid, dim3(256), 0, st, W, n, k, scales, bad);
  return hipGetLastError();
}

hipError_t launch_fp8_pack(const void* W, bool bf16, const float* scales, int64_t n, int64_t k, void* packed,
                           hipStream_t st) {
  const int64_t chunks = w8a8_packed_bytes(n, k) / 16;
  const dim3 grid((unsigned)std::min<int64_t>((chunks + 255) / 256, 1 << 20));
  uint4* out = static_cast<uint4*>(packed);
  if (bf16)
    hipLaunchKernelGGL((k_fp8_pack<uint16_t>), grid, dim3(256), 0, st, W, scales, n, k, chunks, out);
  else
    hipLaunchKernelGGL((k_fp8_pack<float>), grid, dim3(256), 0, st, W, scales, n, k, chunks, out);
  return hipGetLastError();
}

}  // namespace fh
