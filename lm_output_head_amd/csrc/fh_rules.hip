// What a server lays on logits before it chooses a token: penalties for
// repeated tokens, biases, grammar masks; then the choice (argmax or a
// Gumbel-max draw, log-sum-exp) over the row.
//
// A workgroup owns one tile of one row and keeps a table of its tokens in LDS:
// a word with the token's count in the output and, in bit 31, whether it is in
// the prompt, and the sum of its biases.  It walks the row's whole history and
// bias list once, adds what falls into its tile, and then streams the tile's
// logits.  Dense rows index the table by token; rows of listed candidates
// through a hash of their ids.  Counts are integer sums, and one thread adds
// all biases of a token in the list's order, so results do not depend on the
// order of execution.

#include <hip/hip_runtime.h>

#include "fh_choice.hpp"
#include "fh_internal.hpp"

namespace fh {
namespace {

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

constexpr int kThreads = 256;
constexpr int kTileDense = 4096;   // tokens of a dense tile: 32 KB of tables
constexpr int kTileIds = 1024;     // candidates of a tile
constexpr int kSlots = 2048;       // hash slots: at most half of them in use
constexpr uint32_t kPrompt = 0x80000000u;
constexpr int32_t kFree = -1;

template <bool DENSE>
struct Tables {
  static constexpr int kSize = DENSE ? kTileDense : kSlots;
  uint32_t count[kSize];
  float bias[kSize];
  int32_t key[DENSE ? 1 : kSize];
  int list_at[kThreads];
  float list_add[kThreads];
  Part parts[kThreads / 64];
};

__device__ __forceinline__ uint32_t hash_id(int32_t id) { return ((uint32_t)id * 0x9E3779B1u) >> 21; }
static_assert(kSlots == 1 << (32 - 21), "the hash gives a slot");

// The table's place of token t, or -1.
template <bool DENSE>
__device__ __forceinline__ int place_of(const Tables<DENSE>& sh, int32_t t, int64_t base, int64_t width, int64_t v) {
  if constexpr (DENSE) {
    const int64_t u = (int64_t)t - base;
    return u >= 0 && u < width ? (int)u : -1;
  } else {
    if (t < 0 || (int64_t)t >= v) return -1;
    uint32_t s = hash_id(t);
    while (true) {  // ends at the token or at a free slot: half of the slots are free
      const int32_t k = sh.key[s];
      if (k == t) return (int)s;
      if (k == kFree) return -1;
      s = (s + 1) & (kSlots - 1);
    }
  }
}

template <bool DENSE>
__global__ __launch_bounds__(kThreads) void k_rules(RulesArgs a) {
  __shared__ Tables<DENSE> sh;
  constexpr int kTile = DENSE ? kTileDense : kTileIds;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t b = blockIdx.y, base = (int64_t)blockIdx.x * kTile;
  const int64_t width = min((int64_t)kTile, a.n - base);
  const int32_t* ids = DENSE ? nullptr : a.ids + b * a.ld_ids + base;

  for (int i = tid; i < Tables<DENSE>::kSize; i += kThreads) {
    sh.count[i] = 0u;
    sh.bias[i] = 0.f;
    if (!DENSE) sh.key[i] = kFree;
  }
  __syncthreads();
  if constexpr (!DENSE) {
    for (int64_t i = tid; i < width; i += kThreads) {
      const int32_t t = ids[i];
      if (t < 0 || (int64_t)t >= a.v) continue;
      uint32_t s = hash_id(t);
      while (true) {  // at most kTileIds of the kSlots slots are taken
        const int32_t k = atomicCAS(&sh.key[s], kFree, t);
        if (k == kFree || k == t) break;
        s = (s + 1) & (kSlots - 1);
      }
    }
    __syncthreads();
  }
  if (a.history) {
    int64_t nh = a.n_history ? (int64_t)a.n_history[b] : a.history_len;
    nh = min(max(nh, (int64_t)0), a.history_len);
    const int64_t np = a.n_prompt ? min(max((int64_t)a.n_prompt[b], (int64_t)0), nh) : 0;
    const int32_t* h = a.history + b * a.ld_history;
    for (int64_t i = tid; i < nh; i += kThreads) {
      const int p = place_of<DENSE>(sh, h[i], base, width, a.v);
      if (p < 0) continue;
      if (i < np)
        atomicOr(&sh.count[p], kPrompt);
      else
        atomicAdd(&sh.count[p], 1u);
    }
  }
  if (a.bias_ids) {
    int64_t nb = a.n_bias ? (int64_t)a.n_bias[b] : a.bias_len;
    nb = min(max(nb, (int64_t)0), a.bias_len);
    for (int64_t i0 = 0; i0 < nb; i0 += kThreads) {
      const int64_t i = i0 + tid;
      const int m = (int)min((int64_t)kThreads, nb - i0);
      __syncthreads();
      sh.list_at[tid] = i < nb ? place_of<DENSE>(sh, a.bias_ids[b * a.ld_bias + i], base, width, a.v) : -1;
      sh.list_add[tid] = i < nb ? a.bias[b * a.ld_bias + i] : 0.f;
      __syncthreads();
      for (int e = 0; e < m; ++e)
        if (sh.list_at[e] >= 0 && (sh.list_at[e] & (kThreads - 1)) == tid) sh.bias[sh.list_at[e]] += sh.list_add[e];
    }
  }
  __syncthreads();

  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int64_t r = a.mask_row ? (int64_t)a.mask_row[b] : b;
    if (r >= 0 && r < a.mask_rows) mask = a.mask + r * a.ld_mask;
  }
  const float* z = a.z + b * a.ld_z + base;
  float* out = a.out ? a.out + b * a.ld_out + base : nullptr;
  Part part = part_empty();
  for (int64_t i0 = 4 * tid; i0 < width; i0 += 4 * kThreads) {
    const int m = (int)min((int64_t)4, width - i0);
    float x[4];
    int32_t id[4];
    if (m == 4) {
      const f32x4u v = *reinterpret_cast<const f32x4u*>(z + i0);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = e < m ? z[i0 + e] : -INFINITY;
    }
    U4 words{0u, 0u, 0u, 0u};
    if (DENSE && a.token_sample) words = philox_block(a.seed, (uint32_t)b, (uint32_t)((base + i0) >> 2), 1u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= m) break;
      id[e] = DENSE ? (int32_t)(base + i0 + e) : ids[i0 + e];
      bool open = DENSE || (id[e] >= 0 && (int64_t)id[e] < a.v);
      if (open) {
        const int p = DENSE ? (int)i0 + e : place_of<DENSE>(sh, id[e], base, width, a.v);
        const uint32_t c = sh.count[p];
        if (c) {
          x[e] = x[e] > 0.f ? x[e] / rep : x[e] * rep;
          const uint32_t made = c & ~kPrompt;
          x[e] -= freq * (float)made;
          if (made) x[e] -= pres;
        }
        x[e] += sh.bias[p];
        if (mask) open = (mask[id[e] >> 5] >> (id[e] & 31)) & 1u;
      }
      if (!open) {
        x[e] = -INFINITY;
        id[e] = 0x7FFFFFFF;
      }
      if (a.parts) {
        const float y = scaled_logit(x[e], a.tprime);
        float key = x[e];
        if (a.token_sample && open)
          key = y + (DENSE ? gumbel_from_word(u4_word(words, e)) : gumbel_at(a.seed, (uint32_t)b, (uint32_t)id[e], 1u));
        choice_key(part, key, x[e], id[e]);
        choice_lse(part, y, 1.f);
      }
    }
    if (out) {
      if (m == 4)
        *reinterpret_cast<f32x4u*>(out + i0) = f32x4u{x[0], x[1], x[2], x[3]};
      else
        for (int e = 0; e < m; ++e) out[i0 + e] = x[e];
    }
  }
  if (a.parts) {
    part = wave_choice(part);
    if (lane == 0) sh.parts[wave] = part;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kThreads / 64; ++w) part = choice_merge(part, sh.parts[w]);
      a.parts[b * gridDim.x + blockIdx.x] = part;
    }
  }
}

}  // namespace

int64_t rules_parts(int64_t, int64_t n, bool dense) {
  const int tile = dense ? kTileDense : kTileIds;
  return (n + tile - 1) / tile;
}

hipError_t launch_rules(const RulesArgs& a, int64_t B, hipStream_t st) {
  const dim3 grid((unsigned)rules_parts(B, a.n, !a.ids), (unsigned)B), block(kThreads);
  if (a.ids)
    hipLaunchKernelGGL((k_rules<false>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((k_rules<true>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace fh
