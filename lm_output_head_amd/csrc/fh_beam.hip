// Decoding by beams: the best continuations of each sequence over its beams and
// all tokens, and the reordering of states by the beams that they continue.
//
// The total of a continuation is t = score + (z - lse), in float64 (logits and
// scores are float32; neighbours of different beams are told apart by the exact
// difference of their logits).  In a row t grows with z, so what one pass over the
// logits leaves is enough: the largest z of each 256 places (a chunk) and sums of
// exponentials of each 1024 for the row's lse.
// The `keep` best of a sequence lie in the `keep` best chunks, by their largest t
// and, of equal ones, by their order: a chunk outside of them is beaten by one
// element of each.  So a second pass looks at those few chunks alone.

#include <hip/hip_runtime.h>

#include <algorithm>

#include "fh_beam.hpp"
#include "fh_choice.hpp"

namespace fh {
namespace {

constexpr int kChunk = 256, kPart = 1024;
constexpr int kMaxBeams = 64, kMaxKeep = 64;

typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4a __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));

// Four logits of a row from place i, -inf where there is no token.
__device__ __forceinline__ void load_logits(const BeamArgs& a, const float* z, const int32_t* ids, int i, float (&v)[4]) {
  if (i + 4 <= a.n) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(z + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < a.n ? z[i + e] : -INFINITY;
  }
  if (ids) {
    if (i + 4 <= a.n) {
      const i32x4 t = *reinterpret_cast<const i32x4*>(ids + i);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((uint32_t)t[e] >= (uint32_t)a.v) v[e] = -INFINITY;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < a.n && (uint32_t)ids[i + e] >= (uint32_t)a.v) v[e] = -INFINITY;
    }
  }
}

// A wave per 1024 logits.
__global__ __launch_bounds__(256) void k_beam_scan(BeamArgs a, int chunks) {
  const int lane = threadIdx.x & 63, part = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6);
  const int64_t row = blockIdx.y;
  // a beam that is finished or has no total yet offers none of its logits
  if (part * 4 >= chunks || (a.finished && a.finished[row]) || !(a.scores[row] > -INFINITY)) return;
  const float* z = a.z + row * a.ld_z;
  const int32_t* ids = a.ids ? a.ids + row * a.ld_ids : nullptr;
  float v[4][4], top[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) load_logits(a, z, ids, part * kPart + c * kChunk + 4 * lane, v[c]);
#pragma unroll
  for (int c = 0; c < 4; ++c) top[c] = wave_max(fmaxf(fmaxf(v[c][0], v[c][1]), fmaxf(v[c][2], v[c][3])));
  float sum = 0.f;
  if (!a.lse) {
    const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const float shift = m == -INFINITY ? 0.f : m;  // +inf leaves NaN, as a NaN does
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += __expf(v[c][e] - shift);
    sum = wave_sum(sum);
  }
  if (lane == 0) {
    *reinterpret_cast<f32x4a*>(a.top + row * chunks + part * 4) = f32x4a{top[0], top[1], top[2], top[3]};
    if (!a.lse) a.sum[row * (chunks / 4) + part] = sum;
  }
}

struct Cand {
  double t;
  int64_t at;  // beam << 32 | place
};
__device__ __forceinline__ bool beats(const Cand& a, const Cand& b) { return a.t > b.t || (a.t == b.t && a.at < b.at); }
__device__ __forceinline__ Cand worst() { return Cand{-INFINITY, INT64_MAX}; }

template <typename V>
__device__ __forceinline__ V lane_xor(V v, int m) {
  static_assert(sizeof(V) == 8, "two words");
  const int64_t x = __builtin_bit_cast(int64_t, v);
  const uint32_t lo = (uint32_t)__shfl_xor((int)x, m), hi = (uint32_t)__shfl_xor((int)(x >> 32), m);
  return __builtin_bit_cast(V, (int64_t)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ Cand lane_xor(const Cand& c, int m) { return Cand{lane_xor(c.t, m), lane_xor(c.at, m)}; }

// The better of lanes l and l ^ m goes to the one whose bit m is `low`.
__device__ __forceinline__ void exchange(Cand& c, int m, bool keep_better) {
  const Cand o = lane_xor(c, m);
  if (beats(o, c) == keep_better) c = o;
}

// A wave's 64 candidates, best first (bitonic); and two such lists' best 64.
__device__ __forceinline__ void sort64(Cand& c, int lane) {
  for (int size = 2; size <= 64; size <<= 1)
    for (int m = size >> 1; m > 0; m >>= 1) exchange(c, m, ((lane & m) == 0) == ((lane & size) == 0 || size == 64));
}
__device__ __forceinline__ void merge64(Cand& c, const Cand& reversed, int lane) {
  if (beats(reversed, c)) c = reversed;
  for (int m = 32; m > 0; m >>= 1) exchange(c, m, (lane & m) == 0);
}
__device__ __forceinline__ Cand reverse64(const Cand& c) { return lane_xor(c, 63); }

// Where a total stands below the best one: eight steps per octave of the distance,
// 2^-6 to 2^25.
constexpr int kBins = 256;
__device__ __forceinline__ int bin_of(double best, double t) {
  const float d = t == best ? 0.f : (float)(best - t);
  return min(max((int)(__float_as_uint(d) >> 20) - 967, 0), kBins - 1);
}

// A workgroup per sequence.
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMaxChunks = 512, kMaxCands = 1024, kAllChunks = 64;
static_assert(kMaxCands == kWaves * 64, "every wave's list has a place");

struct BeamShared {
  double score[kMaxBeams], lse[kMaxBeams], best[kMaxBeams];
  int32_t done[kMaxBeams];
  Cand cand[kMaxCands];
  int rank[kMaxCands];
  int list[kMaxChunks];
  int hist[kBins];
  int border, chunks, cands;
};

__global__ __launch_bounds__(kThreads) void k_beam_choose(BeamArgs a, int chunks) {
  __shared__ BeamShared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t s = blockIdx.x, row0 = s * a.beams;
  const int W = a.beams, M = a.keep, all = W * chunks;

  // the beams' log-sum-exps and best totals
  for (int w = wave; w < W; w += kWaves) {
    const float score = a.scores[row0 + w];
    const bool done = (a.finished && a.finished[row0 + w]) || !(score > -INFINITY);
    double lse = 0., best = score;
    if (!done) {
      const f32x4a* top = reinterpret_cast<const f32x4a*>(a.top + (row0 + w) * chunks);
      const float* sum = a.sum + (row0 + w) * (chunks / 4);
      float m = -INFINITY;
      for (int i = lane; i < chunks / 4; i += 64) {
        const f32x4a x = top[i];
        m = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
      }
      m = wave_max(m);
      if (a.lse) {
        lse = a.lse[row0 + w];
      } else {
        double acc = 0.;
        for (int i = lane; i < chunks / 4; i += 64) {
          const f32x4a x = top[i];
          acc += (double)(sum[i] * exp_from(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), m));
        }
        for (int k = 1; k < 64; k <<= 1) acc += lane_xor(acc, k);
        lse = m + log(acc);
      }
      best = score + ((double)m - lse);
    }
    if (lane == 0) {
      sh.score[w] = score;
      sh.lse[w] = lse;
      sh.best[w] = best;
      sh.done[w] = done;
    }
  }
  if (tid < kBins) sh.hist[tid] = 0;
  if (tid == 0) sh.chunks = sh.cands = 0;
  __syncthreads();
  double best = -INFINITY;
  for (int w = 0; w < W; ++w) best = sh.best[w] > best ? sh.best[w] : best;  // NaN is no total

  auto total = [&](int w, float z) { return sh.score[w] + ((double)z - sh.lse[w]); };
  // every chunk: f(beam, chunk, its largest total)
  auto each_chunk = [&](auto f) {
    for (int i = tid; i < all; i += kThreads) {
      const int w = i / chunks, c = i % chunks;
      if (!sh.done[w]) f(w, c, total(w, a.top[(row0 + w) * chunks + c]));
    }
  };
  // the listed chunks' places, a wave per chunk, and the finished beams:
  // f(total, beam << 32 | place)
  auto each_place = [&](int listed, bool every, auto f) {
    for (int i = wave; i < listed; i += kWaves) {
      const int at = every ? i : sh.list[i], w = at / chunks, c = at % chunks;
      if (sh.done[w]) continue;
      float z[4];
      const int place = c * kChunk + 4 * lane;
      load_logits(a, a.z + (row0 + w) * a.ld_z, a.ids ? a.ids + (row0 + w) * a.ld_ids : nullptr, place, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) f(total(w, z[e]), (int64_t)w << 32 | (place + e));
    }
    if (tid < W && sh.done[tid]) f(sh.score[tid], (int64_t)tid << 32);
  };
  auto count = [&](double t) {
    if (t > -INFINITY) atomicAdd(&sh.hist[bin_of(best, t)], 1);
  };
  // the first bin that, with those before it, holds `keep` totals
  auto find_border = [&]() {
    __syncthreads();
    if (wave == 0) {
      int border = kBins - 1, before = 0;
      for (int b = 0; b < kBins; b += 64) {
        const int upto = before + wave_inclusive_scan(sh.hist[b + lane], lane);
        const uint64_t hit = __ballot(upto >= M);
        if (hit) {
          border = b + __ffsll((unsigned long long)hit) - 1;
          break;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
      }
      if (lane == 0) sh.border = border;
    }
    __syncthreads();
    return sh.border;
  };

  const bool every = all <= kAllChunks;
  int border, listed = all;
  if (every) {
    each_place(all, true, [&](double t, int64_t) { count(t); });
    border = find_border();
  } else {
    each_chunk([&](int, int, double t) { count(t); });
    if (tid < W && sh.done[tid]) count(sh.score[tid]);
    border = find_border();
    each_chunk([&](int w, int c, double t) {
      if (t > -INFINITY && bin_of(best, t) <= border) {
        const int i = atomicAdd(&sh.chunks, 1);
        if (i < kMaxChunks) sh.list[i] = w * chunks + c;
      }
    });
    __syncthreads();
    listed = sh.chunks;
  }
  int cands = kMaxCands + 1;
  if (every || listed <= kMaxChunks) {
    each_place(listed, every, [&](double t, int64_t at) {
      if (t > -INFINITY && bin_of(best, t) <= border) {
        const int i = atomicAdd(&sh.cands, 1);
        if (i < kMaxCands) sh.cand[i] = Cand{t, at};
      }
    });
    __syncthreads();
    cands = sh.cands;
  }

  auto write = [&](int r, const Cand& c) {
    const bool live = c.t > -INFINITY;
    const int w = (int)(c.at >> 32), place = (int)c.at;
    int32_t token = -1;
    if (live) token = sh.done[w] ? a.eos : a.ids ? a.ids[(row0 + w) * a.ld_ids + place] : place;
    a.out_score[s * M + r] = live ? (float)c.t : -INFINITY;
    a.out_token[s * M + r] = token;
    a.out_parent[s * M + r] = live ? w : -1;
    if (a.out_finished) a.out_finished[s * M + r] = live && token == a.eos;
  };
  if (cands <= kMaxCands) {
    // each candidate's place among them, counted by a group of threads
    int per = kThreads;  // threads of a candidate
    while (per * cands > kThreads) per >>= 1;
    const int i = tid / per;
    if (tid < cands) sh.rank[tid] = 0;
    __syncthreads();
    if (i < cands) {
      const Cand mine = sh.cand[i];
      int above = 0;
      for (int j = tid % per; j < cands; j += per) above += beats(sh.cand[j], mine);
      if (above) atomicAdd(&sh.rank[i], above);
    }
    __syncthreads();
    if (tid < cands && sh.rank[tid] < M) write(sh.rank[tid], sh.cand[tid]);
    if (tid >= cands && tid < M) write(tid, worst());
    return;
  }

  // Many totals on one step (rows of equal logits, say): every wave keeps the best
  // 64 of its chunks in order, and the waves' lists are merged.
  Cand mine = worst();
  auto offer = [&](const Cand& c) {
    const Cand last{__builtin_bit_cast(double, (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(__builtin_bit_cast(int64_t, mine.t) >> 32), M - 1) << 32 |
                                                         (uint32_t)__builtin_amdgcn_readlane((int)__builtin_bit_cast(int64_t, mine.t), M - 1))),
                    (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine.at >> 32), M - 1) << 32 |
                              (uint32_t)__builtin_amdgcn_readlane((int)mine.at, M - 1))};
    if (!__ballot(beats(c, last))) return;
    Cand x = c;
    sort64(x, lane);
    merge64(mine, reverse64(x), lane);
  };
  for (int i = wave; i < all; i += kWaves) {
    const int w = i / chunks, c = i % chunks;
    if (sh.done[w]) continue;
    const double top = total(w, a.top[(row0 + w) * chunks + c]);
    if (!(top > -INFINITY) || bin_of(best, top) > border) continue;
    const float* z = a.z + (row0 + w) * a.ld_z;
    const int32_t* ids = a.ids ? a.ids + (row0 + w) * a.ld_ids : nullptr;
    for (int e = 0; e < kChunk; e += 64) {
      const int place = c * kChunk + e + lane;
      double t = -INFINITY;
      if (place < a.n && (!ids || (uint32_t)ids[place] < (uint32_t)a.v)) t = total(w, z[place]);
      offer(t > -INFINITY ? Cand{t, (int64_t)w << 32 | place} : worst());
    }
  }
  if (wave == 0)
    offer(lane < W && sh.done[lane] && sh.score[lane] > -INFINITY ? Cand{sh.score[lane], (int64_t)lane << 32} : worst());
  for (int half = kWaves / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) sh.cand[wave * 64 + 63 - lane] = mine;
    __syncthreads();
    if (wave < half) merge64(mine, sh.cand[(wave + half) * 64 + lane], lane);
  }
  if (wave == 0 && lane < M) write(lane, mine);
}

// ------------------------------------------------------------- reordering

// Rows [sequences x beams] of states are permuted in place within each sequence: a
// thread owns a column, the same bytes of all beams of a sequence, reads what the
// beams continue and then writes those that continue another.  WMAX: registers for
// that many beams, V bytes each.
template <int WMAX, typename V>
__global__ __launch_bounds__(256) void k_beam_reorder(BeamReorderArgs a, int64_t run, int64_t positions, int64_t slabs,
                                                      int64_t items) {
  constexpr int N = (int)sizeof(V);
  const int W = a.beams;
  const bool dense = positions == 1;  // all positions of a row are one run
  const int64_t per = (run + N - 1) / N, columns = per * positions;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t slab = item % slabs, rest = item / slabs;
    const int64_t s = rest % a.sequences, seg = rest / a.sequences;
    const int64_t mid = seg % a.mid, outer = seg / a.mid % a.outer, st = seg / a.mid / a.outer;
    const int64_t col = slab * 256 + threadIdx.x;
    if (col >= columns) continue;
    const int64_t p = dense ? 0 : col / per, o = (dense ? col : col % per) * N;
    char* base = static_cast<char*>(a.state[st]) + outer * a.ld_outer + s * W * a.ld_row + mid * a.ld_mid +
                 p * a.ld_position + o;
    const int32_t* parent = a.parent + s * W;
    // bytes of the column that beam m takes: N, fewer at a row's end, or none
    auto wanted = [&](int m, int* src) -> int {
      *src = m < W ? parent[m] : -1;
      if ((uint32_t)*src >= (uint32_t)W || *src == m) return 0;
      int64_t count = a.positions;
      if (a.lengths) count = min(max((int64_t)a.lengths[s * W + *src], (int64_t)0), a.positions);
      if (!dense) return p < count ? (int)min(run - o, (int64_t)N) : 0;
      return (int)min(max(count * a.run - o, (int64_t)0), (int64_t)N);
    };
    if (o + N <= run) {
      V v[WMAX];
#pragma unroll
      for (int m = 0; m < WMAX; ++m) {
        int src;
        if (wanted(m, &src)) __builtin_memcpy(&v[m], base + src * a.ld_row, N);
      }
#pragma unroll
      for (int m = 0; m < WMAX; ++m) {
        int src;
        const int n = wanted(m, &src);
        if (n == N) {
          __builtin_memcpy(base + m * a.ld_row, &v[m], N);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (i < n) base[m * a.ld_row + i] = reinterpret_cast<const char*>(&v[m])[i];
        }
      }
    } else {  // the row's last bytes, one by one
      for (int i = 0; o + i < run; ++i) {
        char v[WMAX];
#pragma unroll
        for (int m = 0; m < WMAX; ++m) {
          int src;
          if (wanted(m, &src) > i) v[m] = base[src * a.ld_row + i];
        }
#pragma unroll
        for (int m = 0; m < WMAX; ++m) {
          int src;
          if (wanted(m, &src) > i) base[m * a.ld_row + i] = v[m];
        }
      }
    }
  }
}

template <int WMAX, typename V>
void launch_reorder(const BeamReorderArgs& a, hipStream_t st) {
  const bool dense = a.ld_position == a.run || a.positions == 1;
  const int64_t run = dense ? a.run * a.positions : a.run, positions = dense ? 1 : a.positions;
  const int64_t columns = (run + (int64_t)sizeof(V) - 1) / (int64_t)sizeof(V) * positions, slabs = (columns + 255) / 256;
  const int64_t items = slabs * a.sequences * a.mid * a.outer * a.count;
  hipLaunchKernelGGL((k_beam_reorder<WMAX, V>), dim3((unsigned)std::min<int64_t>(items, 1 << 22)), dim3(256), 0, st, a,
                     run, positions, slabs, items);
}

}  // namespace

int64_t beam_chunks(int64_t n) { return (n + kPart - 1) / kPart * (kPart / kChunk); }

hipError_t launch_beam_select(const BeamArgs& a, int64_t sequences, hipStream_t st) {
  const int chunks = (int)beam_chunks(a.n);
  hipLaunchKernelGGL(k_beam_scan, dim3((unsigned)((chunks + 15) / 16), (unsigned)(sequences * a.beams)), dim3(256), 0, st,
                     a, chunks);
  hipLaunchKernelGGL(k_beam_choose, dim3((unsigned)sequences), dim3(kThreads), 0, st, a, chunks);
  return hipGetLastError();
}

hipError_t launch_beam_reorder(const BeamReorderArgs& a, hipStream_t st) {
  if (a.beams <= 4)
    launch_reorder<4, uint4>(a, st);
  else if (a.beams <= 8)
    launch_reorder<8, uint4>(a, st);
  else if (a.beams <= 16)
    launch_reorder<16, uint4>(a, st);
  else if (a.beams <= 32)
    launch_reorder<32, uint32_t>(a, st);
  else
    launch_reorder<64, uint32_t>(a, st);
  return hipGetLastError();
}

}  // namespace fh
