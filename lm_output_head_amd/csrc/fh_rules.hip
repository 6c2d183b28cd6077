// What a server lays on logits before it chooses a token: penalties for
// repeated tokens, biases, grammar masks; then the choice (argmax or a
// Gumbel-max draw, log-sum-exp) over the row.
//
// A workgroup owns one tile of one row and keeps a table of its tokens in LDS:
// a word with the token's count in the output and, in bit 31, whether it is in
// the prompt, and the sum of its biases.  The tile's logits travel to registers
// while the workgroup walks the row's whole history and bias list and adds what
// falls into its tile.  Dense rows index the table by token; rows of listed
// candidates through a hash of their ids.  Counts are integer sums, and one
// thread adds all biases of a token in the list's order, so results do not
// depend on the order of execution.

#include <hip/hip_runtime.h>

#include "fh_choice.hpp"
#include "fh_internal.hpp"

namespace fh {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kPrompt = 0x80000000u;
constexpr int32_t kFree = -1;

typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));

// Four consecutive elements at i, those below n; `other` in the places past it.
template <typename V, typename T>
__device__ __forceinline__ void load4(const T* p, int64_t i, int64_t n, T other, T (&v)[4]) {
  if (i + 4 <= n) {
    const V x = *reinterpret_cast<const V*>(p + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? p[i + e] : other;
  }
}

// DENSE: a table word per token of the tile.  Else a hash of twice the tile's
// size, so that at most half of its slots are taken and every search ends.
template <bool DENSE, int TILE>
struct Tables {
  static constexpr int kSize = DENSE ? TILE : 2 * TILE;
  uint32_t count[kSize];
  float bias[kSize];
  int32_t key[DENSE ? 1 : kSize];
  int list_at[kThreads];
  float list_add[kThreads];
  Part parts[kThreads / 64];

  __device__ static uint32_t hash(int32_t id) { return ((uint32_t)id * 0x9E3779B1u) >> 16 & (kSize - 1); }
  // the token's place, or -1
  __device__ int find(int32_t t, int64_t base, int64_t width, int64_t v) const {
    if constexpr (DENSE) {
      const int64_t u = (int64_t)t - base;
      return u >= 0 && u < width ? (int)u : -1;
    } else {
      if (t < 0 || (int64_t)t >= v) return -1;
      for (uint32_t s = hash(t);; s = (s + 1) & (kSize - 1)) {
        const int32_t k = key[s];
        if (k == t) return (int)s;
        if (k == kFree) return -1;
      }
    }
  }
  // the place of a token of the tile, taken if it has none yet
  __device__ int take(int32_t t) {
    for (uint32_t s = hash(t);; s = (s + 1) & (kSize - 1)) {
      const int32_t k = atomicCAS(&key[s], kFree, t);
      if (k == kFree || k == t) return (int)s;
    }
  }
};

// G groups of 4 logits per thread: a tile is 1024 G.
template <bool DENSE, int G>
__global__ __launch_bounds__(kThreads) void k_rules(RulesArgs a) {
  constexpr int kTile = 4 * G * kThreads, N = 4 * G;
  typedef Tables<DENSE, kTile> Table;
  static_assert((Table::kSize & (Table::kSize - 1)) == 0 && Table::kSize <= 65536, "the hash masks 16 bits");
  __shared__ Table sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.y, base = (int64_t)blockIdx.x * kTile;
  const int64_t width = min((int64_t)kTile, a.n - base);

  // this thread's logits 4 (tid + 256 j) .. + 3 of the tile and their ids
  float z[N];
  int32_t id[N];
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const int64_t at = 4 * (tid + (int64_t)kThreads * j);
    float v[4];
    int32_t t[4];
    load4<f32x4>(a.z + b * a.ld_z + base, at, width, -INFINITY, v);
    if constexpr (!DENSE) load4<i32x4>(a.ids + b * a.ld_ids + base, at, width, (int32_t)-1, t);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[4 * j + e] = v[e];
      id[4 * j + e] = DENSE ? (int32_t)(base + at + e) : t[e];
    }
  }
  bool open[N];
#pragma unroll
  for (int i = 0; i < N; ++i) open[i] = DENSE ? id[i] < a.n : id[i] >= 0 && (int64_t)id[i] < a.v;

  // the row's mask, a word for four consecutive tokens of a dense row
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int64_t r = a.mask_row ? (int64_t)a.mask_row[b] : b;
    if (r >= 0 && r < a.mask_rows) mask = a.mask + r * a.ld_mask;
  }
  uint32_t allow[DENSE ? G : N];
#pragma unroll
  for (int i = 0; i < (DENSE ? G : N); ++i) {
    const int e = DENSE ? 4 * i : i;
    allow[i] = mask && open[e] ? mask[id[e] >> 5] >> (id[e] & 31) : 0xFFFFFFFFu;
  }

  int place[DENSE ? 1 : N];
  if (a.history || a.bias_ids) {
    for (int i = tid; i < Table::kSize; i += kThreads) {
      sh.count[i] = 0u;
      sh.bias[i] = 0.f;
      if (!DENSE) sh.key[i] = kFree;
    }
    __syncthreads();
    if constexpr (!DENSE) {
#pragma unroll
      for (int i = 0; i < N; ++i) place[i] = open[i] ? sh.take(id[i]) : 0;
      __syncthreads();
    }
  }
  if (a.history) {
    int64_t nh = a.n_history ? (int64_t)a.n_history[b] : a.history_len;
    nh = min(max(nh, (int64_t)0), a.history_len);
    const int64_t np = a.n_prompt ? min(max((int64_t)a.n_prompt[b], (int64_t)0), nh) : 0;
    const int32_t* h = a.history + b * a.ld_history;
    for (int64_t i = 4 * tid; i < nh; i += 4 * kThreads) {
      int32_t t[4];
      load4<i32x4>(h, i, nh, (int32_t)-1, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = sh.find(t[e], base, width, a.v);
        if (p >= 0) {
          if (i + e < np)
            atomicOr(&sh.count[p], kPrompt);
          else
            atomicAdd(&sh.count[p], 1u);
        }
      }
    }
  }
  if (a.bias_ids) {
    int64_t nb = a.n_bias ? (int64_t)a.n_bias[b] : a.bias_len;
    nb = min(max(nb, (int64_t)0), a.bias_len);
    for (int64_t i0 = 0; i0 < nb; i0 += kThreads) {
      const int64_t i = i0 + tid;
      const int m = (int)min((int64_t)kThreads, nb - i0);
      const int mine = i < nb ? sh.find(a.bias_ids[b * a.ld_bias + i], base, width, a.v) : -1;
      __syncthreads();  // the list before is done with
      sh.list_at[tid] = mine;
      sh.list_add[tid] = i < nb ? a.bias[b * a.ld_bias + i] : 0.f;
      __syncthreads();
      if (mine >= 0) {
        // the first entry of a place adds up the place's entries, in order
        float sum = sh.bias[mine];
        int first = tid;
#pragma unroll 8
        for (int e = 0; e < m; ++e) {
          if (sh.list_at[e] == mine) {
            first = min(first, e);
            sum += sh.list_add[e];
          }
        }
        if (first == tid) sh.bias[mine] = sum;
      }
    }
  }
  __syncthreads();

  if (a.history || a.bias_ids) {
    const float rep = a.repetition ? a.repetition[b] : 1.f;
    const float freq = a.frequency ? a.frequency[b] : 0.f;
    const float pres = a.presence ? a.presence[b] : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = DENSE ? 4 * (tid + kThreads * (i / 4)) + i % 4 : place[DENSE ? 0 : i];
      const uint32_t c = sh.count[p];
      if (c) {
        z[i] = z[i] > 0.f ? z[i] / rep : z[i] * rep;
        const uint32_t made = c & ~kPrompt;
        z[i] -= freq * (float)made;
        if (made) z[i] -= pres;
      }
      z[i] += sh.bias[p];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    open[i] = open[i] && (DENSE ? allow[i / 4] >> (i % 4) : allow[i]) & 1u;
    if (!open[i]) z[i] = -INFINITY;
  }
  if (a.out) {
    float* out = a.out + b * a.ld_out + base;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const int64_t at = 4 * (tid + (int64_t)kThreads * j);
      if (at + 4 <= width)
        *reinterpret_cast<f32x4*>(out + at) = f32x4{z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]};
      else
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at + e < width) out[at + e] = z[4 * j + e];
    }
  }
  if (a.parts) {
    uint32_t word[N] = {};
    if (a.token_sample) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if constexpr (DENSE) {
          const U4 w = token_words(a.seed, (uint32_t)b, (uint32_t)id[4 * j] >> 2);
#pragma unroll
          for (int e = 0; e < 4; ++e) word[4 * j + e] = u4_word(w, e);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const U4 w = token_words(a.seed, (uint32_t)b, (uint32_t)id[4 * j + e] >> 2);
            word[4 * j + e] = u4_word(w, id[4 * j + e] & 3);
          }
        }
      }
    }
    Part part = wave_choice(choose<N>(z, id, open, a.token_sample != 0, a.tprime, word));
    if (lane == 0) sh.parts[wave] = part;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int w = 1; w < kThreads / 64; ++w) part = choice_merge(part, sh.parts[w]);
      a.parts[b * gridDim.x + blockIdx.x] = part;
    }
  }
}

// Groups per thread: four where that still leaves two workgroups per CU.
int groups_of(int64_t B, int64_t n) { return B * ((n + 4095) / 4096) >= 512 ? 4 : 1; }

template <bool DENSE>
void launch(const RulesArgs& a, int64_t B, hipStream_t st) {
  const dim3 grid((unsigned)rules_parts(B, a.n), (unsigned)B), block(kThreads);
  if (groups_of(B, a.n) == 4)
    hipLaunchKernelGGL((k_rules<DENSE, 4>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_rules<DENSE, 1>), grid, block, 0, st, a);
}

}  // namespace

int64_t rules_parts(int64_t B, int64_t n) {
  const int tile = 4 * kThreads * groups_of(B, n);
  return (n + tile - 1) / tile;
}

hipError_t launch_rules(const RulesArgs& a, int64_t B, hipStream_t st) {
  if (a.ids)
    launch<false>(a, B, st);
  else
    launch<true>(a, B, st);
  return hipGetLastError();
}

}  // namespace fh
