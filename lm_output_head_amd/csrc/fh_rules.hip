// What a server lays on logits before it chooses a token: penalties for
// repeated tokens, biases, grammar masks; then the choice (argmax or a
// Gumbel-max draw, log-sum-exp) over the row.
//
// A workgroup owns one tile of one row and keeps a table of its tokens in LDS: a
// word with the token's count in the output and, in bit 31, whether it is in the
// prompt.  The tile's logits travel to registers while the workgroup walks the
// row's whole history and adds what falls into its tile; biases are added up in a
// second turn of the table.  Dense rows index the table by token; rows of listed
// candidates through a hash of their ids.  Counts are integer sums, and one
// thread adds all biases of a token in the list's order, so results do not
// depend on the order of execution.
//
// us of the GPU's time, sampled, 8192 of history unless said: 64 rows of 151936 with
// masks and 64 biases take 27.1 us and 3.4 more with the choice's launch.  Without
// masks and biases it is 26.6 in all, and 42.4 for 128 rows: 64 rows more cost 15.8
// us, 4.9 TB/s, a copy's rate, but the first 64 go through load, history, choice
// and draw together, so that their stream and their arithmetic overlap little.
// Few rows are bound by latency: the chain of history, table and reductions, 7 us
// in two launches at 1 x 128256, greedy, with 1000 of history.

#include <hip/hip_runtime.h>

#include <type_traits>

#include "fh_choice.hpp"
#include "fh_serve.hpp"

namespace fh {
namespace {

constexpr uint32_t kPrompt = 0x80000000u;
constexpr int32_t kFree = -1;
constexpr int kAhead = 2;  // groups of four history ids that a thread loads at once

typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t i32x4a __attribute__((ext_vector_type(4)));

// W (1 or 4) consecutive elements at i, those below n; `other` past it.  ALL: n
// reaches past them.
template <int W, bool ALL, typename V, typename T>
__device__ __forceinline__ void load_run(const T* p, int i, int n, T other, T (&v)[W]) {
  if constexpr (W == 4) {
    if (ALL || i + 4 <= n) {
      const V x = *reinterpret_cast<const V*>(p + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x[e];
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < W; ++e) v[e] = ALL || i + e < n ? p[i + e] : other;
}

// DENSE: a word per token of the tile, its count and later its bias.  Else a
// hash of twice the tile's size, so that at most half of its slots are taken and
// every search ends, behind a bitmap of the ids' low bits that turns most of the
// history away at its first read.
template <bool DENSE, int TILE, int TH>
struct Tables {
  static constexpr int kSize = DENSE ? TILE : 2 * TILE;
  static constexpr int kBits = TILE > 4096 ? 65536 : 32768;
  alignas(16) uint32_t count[kSize];  // then the sums of the biases
  alignas(16) int32_t key[DENSE ? 4 : kSize];
  alignas(16) uint32_t maybe[DENSE ? 4 : kBits / 32];
  // a list's entries that fall into the tile, by wave, in order
  int listed[TH / 64];
  int list_at[TH];
  float list_add[TH];
  Part parts[TH / 64];

  __device__ void clear(int tid) {
    const i32x4a zero{0, 0, 0, 0};
    for (int i = 4 * tid; i < kSize; i += 4 * TH) {
      *reinterpret_cast<i32x4a*>(&count[i]) = zero;
      if constexpr (!DENSE) *reinterpret_cast<i32x4a*>(&key[i]) = i32x4a{kFree, kFree, kFree, kFree};
    }
    if constexpr (!DENSE)
      for (int i = 4 * tid; i < kBits / 32; i += 4 * TH) *reinterpret_cast<i32x4a*>(&maybe[i]) = zero;
  }
  __device__ static uint32_t hash(int32_t id) { return ((uint32_t)id * 0x9E3779B1u) >> 16 & (kSize - 1); }
  // whether the token may be in the tile: what most of a history fails
  __device__ bool may_hold(int32_t t, int base, int width, int v) const {
    if constexpr (DENSE) {
      return (uint32_t)t - (uint32_t)base < (uint32_t)width;  // past width too where t is below base
    } else {
      return (uint32_t)t < (uint32_t)v && (maybe[(t & (kBits - 1)) >> 5] >> (t & 31) & 1u);
    }
  }
  // the place of a token that may be in the tile, or -1
  __device__ int find(int32_t t, int base) const {
    if constexpr (DENSE) {
      return (int)((uint32_t)t - (uint32_t)base);
    } else {
      for (uint32_t s = hash(t);; s = (s + 1) & (kSize - 1)) {
        const int32_t k = key[s];
        if (k == t) return (int)s;
        if (k == kFree) return -1;
      }
    }
  }
  // the place of a token of the tile, taken if it has none yet
  __device__ int take(int32_t t) {
    atomicOr(&maybe[(t & (kBits - 1)) >> 5], 1u << (t & 31));
    for (uint32_t s = hash(t);; s = (s + 1) & (kSize - 1)) {
      const int32_t k = atomicCAS(&key[s], kFree, t);
      if (k == kFree || k == t) return (int)s;
    }
  }
};

// G runs of W consecutive logits per thread: a tile is TH W G.  Held to the
// registers of six waves per SIMD (64 x 151936 sampled, the whole call: 30.8 us at
// five, 30.5 at six, 31.6 at seven); workgroups of sixteen waves to four.
template <bool DENSE, int TH, int W, int G>
__global__ __launch_bounds__(TH) __attribute__((amdgpu_waves_per_eu(TH == 1024 ? 4 : 6))) void k_rules(RulesArgs a) {
  constexpr int kTile = TH * W * G, N = W * G, kBatch = 4 * TH * kAhead;  // ids of the history at once
  typedef Tables<DENSE, kTile, TH> Table;
  static_assert(DENSE || ((Table::kSize & (Table::kSize - 1)) == 0 && Table::kSize <= 65536), "the hash masks 16 bits");
  static_assert(!DENSE || W == 4, "a Philox block and a mask word serve four tokens of a dense row");
  __shared__ Table sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.y;
  const int base = (int)blockIdx.x * kTile, v = a.v;
  const int width = min(kTile, a.n - base);
  const bool full = width == kTile;

  // this thread's logits W (tid + TH j) .. + W - 1 of the tile and their ids;
  // what is past the tile or no token is -inf from here on
  float z[N];
  int32_t id[N];
  bool open[N];
  const float* zb = a.z + b * a.ld_z + base;
  auto load_tile = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int at = W * (tid + TH * j);
      float x[W];
      int32_t t[W];
      load_run<W, ALL, f32x4>(zb, at, width, -INFINITY, x);
      if constexpr (!DENSE) load_run<W, ALL, i32x4>(a.ids + b * a.ld_ids + base, at, width, (int32_t)-1, t);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const int i = W * j + e;
        z[i] = x[e];
        id[i] = DENSE ? base + at + e : t[e];
        open[i] = DENSE ? ALL || at + e < width : (uint32_t)t[e] < (uint32_t)v;
      }
    }
  };
  if (full)
    load_tile(std::true_type());
  else
    load_tile(std::false_type());

  // the row's mask, a word for four consecutive tokens of a dense row
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int r = a.mask_row ? a.mask_row[b] : (int)b;
    if (r >= 0 && r < a.mask_rows) mask = a.mask + r * a.ld_mask;
  }
  uint32_t allow[DENSE ? G : N];
#pragma unroll
  for (int i = 0; i < (DENSE ? G : N); ++i) {
    const int e = DENSE ? W * i : i;
    allow[i] = mask ? mask[open[e] ? id[e] >> 5 : 0] >> (id[e] & 31) : 0xFFFFFFFFu;
  }

  // the first of the history and of the biases, on their way as well, to the
  // row's capacity: the loads need not wait for its length
  const int32_t* h = a.history ? a.history + b * a.ld_history : nullptr;
  int32_t seen[kAhead][4];
  auto load_history = [&](int i0) {
    if (i0 + kBatch <= a.history_len) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        load_run<4, true, i32x4>(h, i0 + 4 * (tid + TH * u), 0, (int32_t)-1, seen[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        load_run<4, false, i32x4>(h, i0 + 4 * (tid + TH * u), a.history_len, (int32_t)-1, seen[u]);
    }
  };
  if (a.history) load_history(0);
  int32_t bias_id = -1;
  float bias_add = 0.f;
  auto load_bias = [&](int i) {
    bias_id = -1;
    if (i < a.bias_len) {
      bias_id = a.bias_ids[b * a.ld_bias + i];
      bias_add = a.bias[b * a.ld_bias + i];
    }
  };
  int nh = 0, np = 0, nb = 0;
  if (a.history) {
    nh = min(max(a.n_history ? a.n_history[b] : a.history_len, 0), a.history_len);
    np = a.n_prompt ? min(max(a.n_prompt[b], 0), nh) : 0;
  }
  if (a.bias_ids) {
    load_bias(tid);
    nb = min(max(a.n_bias ? a.n_bias[b] : a.bias_len, 0), a.bias_len);
  }

  int place[N];
#pragma unroll
  for (int i = 0; i < N; ++i) place[i] = DENSE ? W * (tid + TH * (i / W)) + i % W : 0;
  if (a.history || (!DENSE && a.bias_ids)) {
    sh.clear(tid);
    __syncthreads();
    if constexpr (!DENSE) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (open[i]) place[i] = sh.take(id[i]);
      __syncthreads();
    }
  }
  if (a.history) {
    // a batch: what may be in the tile is found out for all before any is looked
    // for.  Most batches are all prompt or all output and wholly inside nh.
    auto count_batch = [&](int i0, auto inside, auto prompt, auto output) {
      bool may[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          may[u][e] = sh.may_hold(seen[u][e], base, width, v) &&
                      (decltype(inside)::value || i0 + 4 * (tid + TH * u) + e < nh);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (!may[u][e]) continue;
          const int p = sh.find(seen[u][e], base);
          if (!DENSE && p < 0) continue;
          if (decltype(output)::value || (!decltype(prompt)::value && i0 + 4 * (tid + TH * u) + e >= np))
            atomicAdd(&sh.count[p], 1u);
          else
            atomicOr(&sh.count[p], kPrompt);
        }
    };
    const std::true_type yes;
    const std::false_type no;
    for (int i0 = 0; i0 < nh; i0 += kBatch) {
      if (i0 + kBatch <= np)
        count_batch(i0, yes, yes, no);
      else if (i0 >= np && i0 + kBatch <= nh)
        count_batch(i0, yes, no, yes);
      else
        count_batch(i0, no, no, no);
      if (i0 + kBatch < nh) load_history(i0 + kBatch);
    }
    __syncthreads();
    // a positive logit is multiplied by 1 / rep, itself rounded once per row (a
    // division per logit rounds once less and cost 1.5 us at 64 x 151936 with 8192
    // of history, where nearly every wave has a repeated token at each of its places)
    const float rep = a.repetition ? a.repetition[b] : 1.f, per = 1.f / rep;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t c = sh.count[place[i]];
      if (c && open[i]) {
        const uint32_t made = c & ~kPrompt;
        z[i] = fmaf(-freq, (float)made, z[i] * (z[i] > 0.f ? per : rep));
        z[i] -= made ? pres : 0.f;
      }
    }
  }
  if (a.bias_ids) {
    // the counts make room for the sums, -0 at first, which adds nothing to any
    // logit; a dense row's words have been read by their own thread alone
    float* sums = reinterpret_cast<float*>(sh.count);
    if (!DENSE && a.history) __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (DENSE || open[i]) sums[place[i]] = -0.f;
    for (int i0 = 0; i0 < nb; i0 += TH) {
      if (i0 > 0) load_bias(i0 + tid);
      __syncthreads();  // the sums are there, the list before is done with
      const int mine = i0 + tid < nb && sh.may_hold(bias_id, base, width, v) ? sh.find(bias_id, base) : -1;
      const uint64_t in = __ballot(mine >= 0);
      const int at = 64 * wave + __popcll(in & ((1ull << lane) - 1));
      if (mine >= 0) {
        sh.list_at[at] = mine;
        sh.list_add[at] = bias_add;
      }
      if (lane == 0) sh.listed[wave] = __popcll(in);
      __syncthreads();
      if (mine >= 0) {
        // the first entry of a place goes on with the place's sum, in order; what
        // the others read is not used
        float sum = sums[mine];
        int first = at;
        for (int w = 0; w < TH / 64; ++w) {
          const int m = sh.listed[w];
          for (int e = 64 * w; e < 64 * w + m; ++e)
            if (sh.list_at[e] == mine) {
              first = min(first, e);
              sum += sh.list_add[e];
            }
        }
        if (first == at) sums[mine] = sum;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (DENSE || open[i]) z[i] += sums[place[i]];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    open[i] = open[i] && (DENSE ? allow[i / W] >> (i % W) : allow[DENSE ? 0 : i]) & 1u;
    if (!open[i]) z[i] = -INFINITY;
  }
  if (a.out) {
    float* out = a.out + b * a.ld_out + base;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int at = W * (tid + TH * j);
      if (W == 4 && (full || at + 4 <= width))
        // past the caches: the logits are looked at seldom, once the token is chosen
        __builtin_nontemporal_store(f32x4{z[W * j], z[W * j + 1 % W], z[W * j + 2 % W], z[W * j + 3 % W]},
                                    reinterpret_cast<f32x4*>(out + at));
      else
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (at + e < width) out[at + e] = z[W * j + e];
    }
  }
  if (a.choice) {
    uint32_t word[N] = {};
    if (a.token_sample) {
#pragma unroll
      for (int i = 0; i < N; i += DENSE ? 4 : 1) {
        const U4 w = token_words(a.seed, (uint32_t)b, (uint32_t)id[i] >> 2);
        if constexpr (DENSE) {
#pragma unroll
          for (int e = 0; e < 4; ++e) word[i + e] = u4_word(w, e);
        } else {
          word[i] = u4_word(w, id[i] & 3);
        }
      }
    }
    Part part = wave_choice(choose<N, DENSE>(z, id, a.token_sample != 0, a.inverse_t, word));
    if (lane == 0) sh.parts[wave] = part;
    __syncthreads();
    if (wave == 0) {
      part = wave_choice(lane < TH / 64 ? sh.parts[lane] : part_empty());
      if (lane == 0) {
        if (gridDim.x == 1)
          write_choice(part, b, a.out_token, a.out_token_logit, a.out_lse);
        else
          a.parts[b * gridDim.x + blockIdx.x] = part;
      }
    }
  }
}

// The tile of a call.  A row of one tile writes its choice itself: no second
// launch, 3 us of the host's time and as much of the GPU's.
struct Shape {
  int tile, threads;
  void (*kernel)(RulesArgs);
};

// Dense rows (us of the GPU's time with the choice's launch, sampled, a mask, 1000
// tokens of history, 2000 at 151936).  One tile up to 8192 tokens (64 x 4000: 6.7
// with one of 1024 threads, 8.7 with four of 256; 1024 threads hold few rows of a
// CU, so many rows take 256; 256 x 6000: 9.6 with 8192 to a tile, 11.6 with 1024, 1
// x 6000 8.7 and 7.8, but a launch less for the host).  Beyond, small tiles spread
// few rows over the CUs, large ones walk the history less often; the large one
// where it leaves two workgroups per CU (64 x 151936: 26.6 with tiles of 4096, 32.8
// with 1024, 26.6 with 8192, 35.0 with 16384; 1 x 151936: 10.4, 7.9, 11.5 and 13.4).
Shape dense_shape(int64_t B, int64_t n) {
  const Shape small{1024, 256, k_rules<true, 256, 4, 1>}, large{4096, 256, k_rules<true, 256, 4, 4>};
  if (n <= 1024) return small;
  if (n <= 4096 && B < 512) return Shape{4096, 1024, k_rules<true, 1024, 4, 1>};
  if (n > 4096 && n <= 8192) return Shape{8192, 512, k_rules<true, 512, 4, 4>};
  return B * ((n + large.tile - 1) / large.tile) >= 512 ? large : small;
}

// Listed tokens: each tile searches for the whole history, so a tile has a thread
// per token or few, and a CU at most one tile where that can be (as above, 1000 of
// history: 8 x 8192 11.8 with tiles of 512, 17.4 with 4096; 64 x 8192 18.2 with
// 512, 15.8 with 2048, 19.4 with 8192; 256 x 8192 45.5 with 512, 42.5 with 2048,
// 21.0 with 8192).  Up to 4096 tokens one tile (64 x 1000 8.2, 11.9 in two; 64 x
// 3000 11.9, 13.1 in six; 1 x 4096 12.0, 10.5 in eight, but a launch less for the
// host).
Shape list_shape(int64_t B, int64_t n) {
  const Shape shapes[] = {{512, 512, k_rules<false, 512, 1, 1>},
                          {1024, 512, k_rules<false, 512, 1, 2>},
                          {2048, 1024, k_rules<false, 1024, 1, 2>},
                          {4096, 1024, k_rules<false, 1024, 1, 4>},
                          {8192, 1024, k_rules<false, 1024, 1, 8>}};
  if (n <= 512) return shapes[0];
  if (n <= 4096) return shapes[n <= 1024 ? 2 : 3];
  for (const Shape& s : shapes)
    if (B * ((n + s.tile - 1) / s.tile) <= 256) return s;
  return shapes[4];
}

Shape shape_of(int64_t B, int64_t n, bool dense) { return dense ? dense_shape(B, n) : list_shape(B, n); }

}  // namespace

int64_t rules_parts(int64_t B, int64_t n, bool dense) {
  const int tile = shape_of(B, n, dense).tile;
  return (n + tile - 1) / tile;
}

hipError_t launch_rules(const RulesArgs& a, int64_t B, hipStream_t st) {
  const Shape s = shape_of(B, a.n, !a.ids);
  hipLaunchKernelGGL(s.kernel, dim3((unsigned)((a.n + s.tile - 1) / s.tile), (unsigned)B), dim3(s.threads), 0, st, a);
  return hipGetLastError();
}

}  // namespace fh
