// Decoding by beams: the best continuations of each sequence over its beams and
// all tokens, and the reordering of states by the beams that they continue.
//
// The total of a continuation is t = score + (z - lse), in float64 from there on
// (logits, scores and an lse that is given are float32).  In a row t grows with z, so
// what one pass over the logits leaves is enough: the largest z of each 256 places (a
// chunk) and sums of exponentials of each 1024 for the row's lse.  Those
// exponentials and sums are float32, the hardware's exponential with its argument
// rounded: what an lse is off by, at most (42 + 8 ln n) 2^-24, is common to its beam
// and decides the order only between beams, and only there where their totals are
// nearer than that.  Totals of 64 to 300000 logits were off by 5e-7 at most, their
// rounding to float32 included.  In float64 the 16 million exponentials of 16 x 8 x
// 151936 are, by count, some 8 us of instructions beside a scan of 13.
// The `keep` best of a sequence lie in the `keep` best chunks, by their largest t
// and, of equal ones, by their order: a chunk outside of them is beaten by one
// element of each.  So a second pass looks at those few chunks alone.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fh_beam.hpp"
#include "fh_choice.hpp"

namespace fh {
namespace {

constexpr int kChunk = 256, kPart = 1024;
constexpr int kMaxBeams = 64, kMaxKeep = 64;

typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4a __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

// Four logits of a row from place i and their tokens, -inf where there is none.
__device__ __forceinline__ void load_logits(const BeamArgs& a, const float* z, const int32_t* ids, int i, float (&v)[4],
                                            int32_t (&id)[4]) {
  const bool whole = i + 4 <= a.n;
  if (whole) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(z + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < a.n ? z[i + e] : -INFINITY;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) id[e] = i + e;
  if (ids) {
    if (whole) {
      const i32x4 t = *reinterpret_cast<const i32x4*>(ids + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) id[e] = t[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) id[e] = i + e < a.n ? ids[i + e] : -1;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((uint32_t)id[e] >= (uint32_t)a.v) v[e] = -INFINITY;
  }
}

// A wave's 1024 logits of a row; their chunks' largest, and the sum of exponentials
// from the largest of all.
__device__ __forceinline__ void load_part(const BeamArgs& a, int64_t row, int part, int lane, float (&v)[4][4]) {
  const float* z = a.z + row * a.ld_z;
  const int32_t* ids = a.ids ? a.ids + row * a.ld_ids : nullptr;
  int32_t id[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) load_logits(a, z, ids, part * kPart + c * kChunk + 4 * lane, v[c], id);
}
__device__ __forceinline__ f32x4a reduce_part(const float (&v)[4][4], bool want_sum, float* sum) {
  f32x4a top;
#pragma unroll
  for (int c = 0; c < 4; ++c) top[c] = wave_max(fmaxf(fmaxf(v[c][0], v[c][1]), fmaxf(v[c][2], v[c][3])));
  *sum = 0.f;
  if (want_sum) {
    const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const float shift = m == -INFINITY ? 0.f : m;  // +inf leaves NaN, as a NaN does
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) *sum += __expf(v[c][e] - shift);
    *sum = wave_sum(*sum);
  }
  return top;
}

// A wave per 1024 logits, all on their way before the first is used; the largest
// come out of exchanges between lanes, the exponentials' sum in float32 (1024
// terms of at most 1, in one order).  16 x 8 beams x 151936, of which 62 MB count,
// take 13.0 us (a copy's rate would be 12.7; a read's, 9); two or four of these parts a
// wave 0.9 and 3.4 us more, a workgroup of 1024 threads 1.3.  Four beams of 128256 take
// 3.5.
__global__ __launch_bounds__(256) void k_beam_scan(BeamArgs a, int chunks) {
  const int lane = threadIdx.x & 63, part = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6);
  const int64_t row = blockIdx.y;
  // a finished beam offers none of its logits
  if (part * 4 >= chunks || (a.finished && a.finished[row])) return;
  float v[4][4], sum;
  load_part(a, row, part, lane, v);
  // nor does one without a total yet, whose logits do not wait for that
  if (!(a.scores[row] > -INFINITY)) return;
  const f32x4a top = reduce_part(v, !a.lse, &sum);
  if (lane == 0) {
    *reinterpret_cast<f32x4a*>(a.top + row * chunks + part * 4) = top;
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
#pragma unroll 1
  for (int size = 2; size <= 64; size <<= 1)
#pragma unroll 1
    for (int m = size >> 1; m > 0; m >>= 1) exchange(c, m, ((lane & m) == 0) == ((lane & size) == 0 || size == 64));
}
__device__ __forceinline__ void merge64(Cand& c, const Cand& reversed, int lane) {
  if (beats(reversed, c)) c = reversed;
#pragma unroll 1
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

// A workgroup per sequence: it needs all rows' sums first, then lists the chunks that
// a histogram of totals leaves in question (some `keep` of them), then their places
// in the same bins, and ranks those.  Nothing is sorted unless more than 1024 places
// are left.  It is bound by the chain of its dependent steps and by instructions that
// no cache holds yet, not by data: 6.1 us for one sequence of four beams of 128256, 8.6
// for sixteen of eight of 151936; 256 or 512 threads a workgroup change neither.
//
// SPLIT waves share a row and ROWS rows a wave; of rows of at most 1024 chunks their
// largest logits stay in registers.  ROWS = 0: a wave per row, which reads them again
// wherever it looks at them.  ALONE: nothing has been scanned yet: its waves do that
// first, up to kParts parts of a row each.
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kMaxChunks = 512, kMaxCands = 1024;
constexpr int kQuads = 4;  // four chunks each, of a lane of a wave that has a row to itself
constexpr int kParts = 2;  // of a wave that scans them itself
static_assert(kMaxCands == kWaves * 64 && kThreads == 1 << 10, "every wave's list has a place");

struct BeamShared {
  double score[kMaxBeams], lse[kMaxBeams], best[kMaxBeams];
  double part_sum[kMaxBeams];  // of a row's waves, one after another
  float part_top[kMaxBeams];
  int32_t done[kMaxBeams];
  Cand cand[kMaxCands];
  int32_t token[kMaxCands];
  int rank[kMaxCands];
  int list[kMaxChunks];
  int hist[kBins];
  int border, chunks, cands;
};

__device__ __forceinline__ float most4(const f32x4a& x) { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])); }

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const int64_t x = __builtin_bit_cast(int64_t, v);
  const uint32_t lo = (uint32_t)dpp_i<CTRL>((int)x), hi = (uint32_t)dpp_i<CTRL>((int)(x >> 32));
  return __builtin_bit_cast(double, (int64_t)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ int64_t readlane_l(int64_t x, int l) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)x, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), l);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double readlane_d(double v, int l) {
  return __builtin_bit_cast(double, readlane_l(__builtin_bit_cast(int64_t, v), l));
}
// wave_sum's order in float64
__device__ __forceinline__ double wave_sum_d(double x) {
  x += dpp_d<0xB1>(x);
  x += dpp_d<0x4E>(x);
  x += dpp_d<0x141>(x);
  x += dpp_d<0x140>(x);
  return (readlane_d(x, 0) + readlane_d(x, 16)) + (readlane_d(x, 32) + readlane_d(x, 48));
}

__device__ __forceinline__ double wave_max_d(double x) {
  x = fmax(x, dpp_d<0xB1>(x));
  x = fmax(x, dpp_d<0x4E>(x));
  x = fmax(x, dpp_d<0x141>(x));
  x = fmax(x, dpp_d<0x140>(x));
  return fmax(fmax(readlane_d(x, 0), readlane_d(x, 16)), fmax(readlane_d(x, 32), readlane_d(x, 48)));
}

// ln s of a sum s >= 0 (-inf of 0, NaN of NaN) to some 1e-14: s = f 2^e with f in
// [0.75, 1.5), ln f = 2 artanh((f - 1) / (f + 1)) by its series.
__device__ __forceinline__ double log_of(double s) {
  if (!(s > 0.) || s == INFINITY) return s == 0. ? -INFINITY : s;
  const int64_t b = __builtin_bit_cast(int64_t, s);
  const int64_t up = (b >> 51) & 1;  // f >= 1.5 is halved
  const double f = __builtin_bit_cast(double, (b & 0x000FFFFFFFFFFFFFll) | (1023 - up) << 52);
  const double u = (f - 1.) / (f + 1.), v = u * u;
  double p = 1. / 19.;
#pragma unroll
  for (int k = 17; k > 0; k -= 2) p = fma(p, v, 1. / k);
  return fma((double)((b >> 52) - 1023 + up), 0.693147180559945309417, 2. * u * p);
}

// Places on a list for the lanes that are set in m, in one addition.
__device__ __forceinline__ int take(int* length, uint64_t m, int lane) {
  int first = 0;
  if (lane == 0) first = atomicAdd(length, __popcll(m));
  return __builtin_amdgcn_readfirstlane(first) + __popcll(m & ((1ull << lane) - 1));
}

template <int ROWS, int SPLIT, bool ALONE>
__global__ __launch_bounds__(kThreads) void k_beam_choose(BeamArgs a, int chunks) {
  static_assert(ROWS <= 1 || SPLIT == 1, "waves share rows, or rows a wave");
  static_assert(!ALONE || ROWS == 1, "a wave's parts are of one row");
  constexpr int kRows = ROWS > 0 ? ROWS : 1, kOwn = ALONE ? 1 : kQuads / SPLIT, kTeams = kWaves / SPLIT;
  __shared__ BeamShared sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int team = wave / SPLIT, member = wave % SPLIT;
  const int64_t s = blockIdx.x, row0 = s * a.beams;
  const int W = a.beams, M = a.keep, all = W * chunks, quads = chunks / 4;

  if (tid < kBins) sh.hist[tid] = 0;
  if (tid == 0) sh.chunks = sh.cands = 0;
  // four chunks from 4 i up of row w; a finished row has none written
  auto load_top = [&](int w, int i) {
    return *reinterpret_cast<const f32x4a*>(a.top + (row0 + w) * chunks + 4 * i);
  };
  auto place_of = [&](int q) { return ALONE ? lane * SPLIT + member : lane + 64 * (member + SPLIT * q); };
  const f32x4a none{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  // the beams' scores, and everything that the scan has left of them, on its way
  // together
  float beam_score = 0.f, beam_lse = 0.f;
  int32_t beam_fin = 0;
  if (tid < W) {
    beam_score = a.scores[row0 + tid];
    beam_fin = a.finished ? a.finished[row0 + tid] : 0;
    beam_lse = a.lse ? a.lse[row0 + tid] : 0.f;
  }
  f32x4a top[kRows][kOwn];
  float sum[kRows][kOwn];
  if constexpr (ROWS > 0 && !ALONE) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int w = team + r * kTeams;
      if (w >= W) break;
#pragma unroll
      for (int q = 0; q < kOwn; ++q) {
        const int i = place_of(q);
        top[r][q] = i < quads ? load_top(w, i) : none;
        sum[r][q] = i < quads && !a.lse ? a.sum[(row0 + w) * quads + i] : 0.f;
      }
    }
  }
  if constexpr (ALONE) {
    top[0][0] = none;
    sum[0][0] = 0.f;
    const bool live = team < W && !(a.finished && a.finished[row0 + team]);
    const float score = team < W ? a.scores[row0 + team] : 0.f;
    float v[kParts][4][4];
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      if (live && member + i * SPLIT < quads) load_part(a, row0 + team, member + i * SPLIT, lane, v[i]);
    if (live && score > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int p = member + i * SPLIT;
        if (p >= quads) break;
        float total;
        const f32x4a most = reduce_part(v[i], !a.lse, &total);
        if (lane == i) {
          top[0][0] = most;
          sum[0][0] = total;
          *reinterpret_cast<f32x4a*>(a.top + (row0 + team) * chunks + 4 * p) = most;
        }
      }
    }
  }
  // the rows' largest logits m and sums of exp(z - m); what a finished row holds
  // here is not looked at
  auto leave = [&](int at, float m, double acc) {
    if (lane == 0) {
      sh.part_top[at] = m;
      sh.part_sum[at] = acc;
    }
  };
  if constexpr (ROWS > 0) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int w = team + r * kTeams;
      if (w >= W) break;
      float m = -INFINITY;
      double acc = 0.;
#pragma unroll
      for (int q = 0; q < kOwn; ++q) m = fmaxf(m, most4(top[r][q]));
      m = wave_max(m);
#pragma unroll
      for (int q = 0; q < kOwn; ++q) acc += (double)(sum[r][q] * exp_from(most4(top[r][q]), m));
      leave(w * SPLIT + member, m, wave_sum_d(acc));
    }
  } else {
    for (int w = wave; w < W; w += kWaves) {
      float m = -INFINITY;
      double acc = 0.;
      for (int i = lane; i < quads; i += 64) m = fmaxf(m, most4(load_top(w, i)));
      m = wave_max(m);
      if (!a.lse)
        for (int i = lane; i < quads; i += 64)
          acc += (double)(a.sum[(row0 + w) * quads + i] * exp_from(most4(load_top(w, i)), m));
      leave(w, m, wave_sum_d(acc));
    }
  }
  __syncthreads();
  // the log-sum-exps and best totals, a lane per row
  if (tid < W) {
    const bool done = beam_fin || !(beam_score > -INFINITY);
    double lse = 0., best = beam_score;
    if (!done) {
      float m = sh.part_top[tid * SPLIT];
#pragma unroll
      for (int i = 1; i < SPLIT; ++i) m = fmaxf(m, sh.part_top[tid * SPLIT + i]);
      double acc = sh.part_sum[tid * SPLIT];
      if constexpr (SPLIT > 1) {
        acc = 0.;
#pragma unroll
        for (int i = 0; i < SPLIT; ++i) acc += sh.part_sum[tid * SPLIT + i] * (double)exp_from(sh.part_top[tid * SPLIT + i], m);
      }
      lse = a.lse ? (double)beam_lse : m + log_of(acc);
      best = beam_score + ((double)m - lse);
    }
    sh.score[tid] = beam_score;
    sh.lse[tid] = lse;
    sh.best[tid] = best;
    sh.done[tid] = done;
  }
  __syncthreads();
  const double best = wave_max_d(lane < W ? sh.best[lane] : -INFINITY);  // NaN is no total

  auto total = [&](int w, float z) { return sh.score[w] + ((double)z - sh.lse[w]); };
  auto count = [&](int bin) {
    if (bin < kBins) atomicAdd(&sh.hist[bin], 1);
  };
  auto bin_at = [&](double t) { return t > -INFINITY ? bin_of(best, t) : kBins; };
  // the first bin that, with those before it, holds `keep` totals
  auto find_border = [&]() {
    __syncthreads();
    if (wave == 0) {
      int border = kBins - 1, before = 0;
#pragma unroll 1
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
  // the listed chunks' places, a wave per chunk and two at a time, and the finished
  // beams: f(which lanes' eight and what they are), what they are being given by the
  // bit's number
  auto each_place = [&](int listed, bool every, auto f) {
#pragma unroll 1
    for (int i0 = wave; i0 < listed; i0 += 2 * kWaves) {
      // as vectors: a choice between elements of an array would send it to memory
      f32x8 z;
      i32x8 id;
      auto load = [&](int i, int* w, int* place, auto half) {
        constexpr int H = decltype(half)::value;
        const int at = i < listed ? every ? i : sh.list[i] : 0;
        *w = at / chunks;
        *place = at % chunks * kChunk + 4 * lane;
        float v[4];
        int32_t k[4];
        if (i < listed && !sh.done[*w]) {
          load_logits(a, a.z + (row0 + *w) * a.ld_z, a.ids ? a.ids + (row0 + *w) * a.ld_ids : nullptr, *place, v, k);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = -INFINITY, k[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) z[4 * H + e] = v[e], id[4 * H + e] = k[e];
      };
      int w0, w1, place0, place1;
      load(i0, &w0, &place0, std::integral_constant<int, 0>());
      load(i0 + kWaves, &w1, &place1, std::integral_constant<int, 1>());
      int bin[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) bin[b] = bin_at(total(b < 4 ? w0 : w1, z[b]));
      f(bin, [&](int b, double* t, int64_t* at, int32_t* token) {
        float x = z[0];
        int32_t k = id[0];
#pragma unroll
        for (int c = 1; c < 8; ++c) {
          x = b == c ? z[c] : x;
          k = b == c ? id[c] : k;
        }
        const int row = b < 4 ? w0 : w1;
        *t = total(row, x);
        *at = (int64_t)row << 32 | ((b < 4 ? place0 : place1) + (b & 3));
        *token = k;
      });
    }
    if (wave == 0) {
      const bool mine = lane < W && sh.done[lane];
      int bin[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) bin[b] = b == 0 && mine ? bin_at(sh.score[lane]) : kBins;
      f(bin, [&](int, double* t, int64_t* at, int32_t* token) {
        *t = sh.score[lane < W ? lane : 0];
        *at = (int64_t)lane << 32;
        *token = a.eos;
      });
    }
  };

  // No more chunks than `keep` would all be listed, so their places are counted at
  // once; of more, the chunks' largest say enough (8 x 2048 candidates, keep 8, 9.9 us;
  // counting all of the places 15.5).
  const bool every = all <= M;
  int border = 0, listed = all;
  if (!every) {
    if (wave == 0 && lane < W && sh.done[lane]) count(bin_at(sh.score[lane]));
    auto list = [&](uint32_t hits, auto chunk_of) {
      for (uint64_t m; (m = __ballot(hits != 0)); hits &= hits - 1) {
        const int i = take(&sh.chunks, m, lane);
        if (hits && i < kMaxChunks) sh.list[i] = chunk_of(__ffs(hits) - 1);
      }
    };
    if constexpr (ROWS > 0) {
      constexpr int kMine = kRows * kOwn * 4;
      static_assert(kMine <= 32, "a bit per chunk of a lane");
      int bin[kMine];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int w = team + r * kTeams;
        const bool use = w < W && !sh.done[w];
        const double sc = use ? sh.score[w] : 0., lse = use ? sh.lse[w] : 0.;
#pragma unroll
        for (int q = 0; q < kOwn; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            int& b = bin[(r * kOwn + q) * 4 + e];
            b = use && place_of(q) < quads ? bin_at(sc + ((double)top[r][q][e] - lse)) : kBins;
            count(b);
          }
      }
      border = find_border();
      uint32_t hits = 0;
#pragma unroll
      for (int b = 0; b < kMine; ++b) hits |= (uint32_t)(bin[b] <= border) << b;
      list(hits, [&](int b) {
        return (team + b / (4 * kOwn) * kTeams) * chunks + 4 * place_of(b / 4 % kOwn) + (b & 3);
      });
    } else {
      auto each_quad = [&](auto f) {
        for (int w = wave; w < W; w += kWaves) {
          if (sh.done[w]) continue;
          for (int i0 = 0; i0 < quads; i0 += 64) {
            const int i = i0 + lane;
            const f32x4a x = i < quads ? load_top(w, i) : none;
            int bin[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) bin[e] = bin_at(total(w, x[e]));
            f(w * chunks + 4 * i, bin);
          }
        }
      };
      each_quad([&](int, const int (&bin)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) count(bin[e]);
      });
      border = find_border();
      each_quad([&](int at, const int (&bin)[4]) {
        uint32_t hits = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) hits |= (uint32_t)(bin[e] <= border) << e;
        list(hits, [&](int b) { return at + b; });
      });
    }
    __syncthreads();
    listed = sh.chunks;
  }
  int cands = kMaxCands + 1;
  if (listed <= kMaxChunks) {
    // too many places where most of the chunks are listed (a few beams not finished,
    // say): then by a border among the places themselves (4 x 32 beams of 1000, keep 64,
    // 20 of each 32 finished: 26 us a call; by the sort below 105)
    for (bool counted = every;; counted = true) {
      if (counted) {
        each_place(listed, every, [&](const int (&bin)[8], auto) {
#pragma unroll
          for (int b = 0; b < 8; ++b) count(bin[b]);
        });
        border = find_border();
      }
      each_place(listed, every, [&](const int (&bin)[8], auto what) {
        uint32_t hits = 0;
#pragma unroll
        for (int b = 0; b < 8; ++b) hits |= (uint32_t)(bin[b] <= border) << b;
        for (uint64_t m; (m = __ballot(hits != 0)); hits &= hits - 1) {
          const int i = take(&sh.cands, m, lane);
          if (hits && i < kMaxCands) what(__ffs(hits) - 1, &sh.cand[i].t, &sh.cand[i].at, &sh.token[i]);
        }
      });
      __syncthreads();
      cands = sh.cands;
      if (cands <= kMaxCands || counted) break;
      __syncthreads();
      if (tid < kBins) sh.hist[tid] = 0;
      if (tid == 0) sh.cands = 0;
      __syncthreads();
    }
  }

  auto write = [&](int r, const Cand& c, int32_t token) {
    const bool live = c.t > -INFINITY;
    a.out_score[s * M + r] = live ? (float)c.t : -INFINITY;
    a.out_token[s * M + r] = live ? token : -1;
    a.out_parent[s * M + r] = live ? (int)(c.at >> 32) : -1;
    if (a.out_finished) a.out_finished[s * M + r] = live && token == a.eos;
  };
  if (cands <= kMaxCands) {
    // each candidate's place among them, counted by a group of threads
    int bits = 10;  // threads of a candidate, of all 2^10
    while (cands << bits > kThreads) --bits;
    const int i = tid >> bits;
    if (tid < cands) sh.rank[tid] = 0;
    __syncthreads();
    if (i < cands) {
      const Cand mine = sh.cand[i];
      int above = 0;
      for (int j = tid & ((1 << bits) - 1); j < cands; j += 1 << bits) above += beats(sh.cand[j], mine);
      if (above) atomicAdd(&sh.rank[i], above);
    }
    __syncthreads();
    if (tid < cands && sh.rank[tid] < M) write(sh.rank[tid], sh.cand[tid], sh.token[tid]);
    if (tid >= cands && tid < M) write(tid, worst(), -1);
    return;
  }

  // Many totals on one step: every wave keeps the best 64 of its chunks in order, and
  // the waves' lists are merged.  Rows of equal logits come here (16 x 9 beams of
  // 151936, keep 16, 223 us; one sequence of four 305), and totals far below the best
  // one, whose steps are wide there (a finished beam 40 above the eight live ones of
  // each of those 16 sequences 368 us; among them 24).
  Cand mine = worst();
  auto offer = [&](const Cand& c) {
    const Cand last{readlane_d(mine.t, M - 1), readlane_l(mine.at, M - 1)};
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
  if (wave == 0 && lane < M) {
    int32_t token = -1;
    if (mine.t > -INFINITY) {
      const int w = (int)(mine.at >> 32), place = (int)mine.at;
      token = sh.done[w] ? a.eos : a.ids ? a.ids[(row0 + w) * a.ld_ids + place] : place;
    }
    write(lane, mine, token);
  }
}

// ------------------------------------------------------------- reordering

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The first n < sizeof(V) bytes at p, and n of v to p.
template <typename V>
__device__ __forceinline__ V load_bytes(const char* p, int n) {
  uint64_t lo = 0, hi = 0;
  for (int i = 0; i < n; ++i) {
    const uint64_t b = (uint8_t)p[i];
    if (i < 8)
      lo |= b << (8 * i);
    else
      hi |= b << (8 * i - 64);
  }
  if constexpr (sizeof(V) == 4)
    return (uint32_t)lo;
  else
    return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}
__device__ __forceinline__ void store_bytes(char* p, const u32x4& v, int n) {
  uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  for (int i = 0; i < n; ++i) {
    p[i] = (char)lo;
    lo = lo >> 8 | hi << 56;
    hi >>= 8;
  }
}
__device__ __forceinline__ void store_bytes(char* p, uint32_t v, int n) {
  for (int i = 0; i < n; ++i) p[i] = (char)(v >> (8 * i));
}

// Rows [sequences x beams] of states are permuted in place within each sequence: a
// thread owns columns, the same bytes of all beams of a sequence, reads what the
// beams continue and then writes those that continue another.  A workgroup's
// columns lie in one part of a row (state, layer, sequence, head), kSlab of them;
// lane m of each wave looks up what beam m takes.  WMAX: registers for that many
// beams, V bytes each.  DENSE: the positions of a part are one run.
//
// In place, so what moves is read once and written once, and nothing else is
// touched: no second cache, and beams that continue themselves cost nothing.  Bound by
// memory: 16 states of 8 x 8 beams x 8 heads x 2000 x 64 bfloat16, 2.33 GB read and
// written, take 435 us, 5.3 TB/s, a little above a copy's rate.  Steps there: 1228 us
// with the parents looked up by every thread, 564 by a lane each, 480 with one slab of
// 4 KB a workgroup, 470 with stores past the caches, 448 with the loads past them as
// well (PAST).  Three gigabytes by more beams: 4 x 16 4.7 TB/s, 2 x 32 5.2, 1 x 64 4.8;
// with positions that are not one run (64 of 128 bfloat16 each) 8 x 8 5.0, 4 x 16 4.7,
// 2 x 32 and 1 x 64, whose columns are four bytes, 4.2.
constexpr int kSlab = 256;

template <int WMAX, typename V, bool DENSE, bool PAST>
__global__ __launch_bounds__(256) void k_beam_reorder(BeamReorderArgs a, int64_t run, uint32_t slabs, uint32_t items) {
  constexpr int N = (int)sizeof(V);
  const int W = a.beams, lane = threadIdx.x & 63;
  const uint32_t per = (uint32_t)((run + N - 1) / N);  // columns of a position, unless DENSE
  for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint32_t slab = item % slabs, rest = item / slabs;
    const uint32_t s = rest % (uint32_t)a.sequences, seg = rest / (uint32_t)a.sequences;
    const uint32_t mid = seg % (uint32_t)a.mid, layer = seg / (uint32_t)a.mid;
    const uint32_t outer = layer % (uint32_t)a.outer, st = layer / (uint32_t)a.outer;
    const int64_t col0 = (int64_t)slab * kSlab;
    // what beam `lane` takes: its parent, and the bytes (positions) of it that this
    // workgroup moves
    int src = lane < W ? a.parent[(int64_t)s * W + lane] : -1, moves = 0;
    if ((uint32_t)src < (uint32_t)W && src != lane) {
      int64_t count = a.positions;
      if (a.lengths) count = min(max((int64_t)a.lengths[(int64_t)s * W + src], (int64_t)0), a.positions);
      moves = DENSE ? (int)min(max(count * a.run - col0 * N, (int64_t)0), (int64_t)kSlab * N) : (int)count;
    }
    if (!__ballot(moves > 0)) continue;
    char* base = static_cast<char*>(a.state[st]) + outer * a.ld_outer + (int64_t)s * W * a.ld_row + mid * a.ld_mid +
                 (DENSE ? col0 * N : 0);
    const int64_t left = DENSE ? run - col0 * N : run;  // bytes of the run from `base` on
    // the column's place from `base`, the run's bytes from it on, and its position
    // or (DENSE) its byte of the slab
    typename std::conditional<DENSE, uint32_t, int64_t>::type at;
    int behind, p;
    if (DENSE) {
      p = ((int)threadIdx.x) * N;
      at = p;
      behind = (int)min(left - p, (int64_t)N);
    } else {
      const int64_t col = col0 + threadIdx.x;
      const uint32_t q = (uint32_t)((uint64_t)col / per), o = (uint32_t)((uint64_t)col % per) * N;
      p = (int)q;
      at = q * a.ld_position + o;
      behind = (int64_t)q < a.positions ? (int)min(left - o, (int64_t)N) : 0;
    }
    // bytes (of N) that beam m takes here, its count being `moves` of lane m
    auto wanted = [&](int count) { return min(DENSE ? count - p : p < count ? N : 0, behind); };
    typedef V U __attribute__((aligned(1)));
    V v[WMAX];
#pragma unroll
    for (int m = 0; m < WMAX; ++m) {
      const int count = __builtin_amdgcn_readlane(moves, m), from = __builtin_amdgcn_readlane(src, m);
      const char* row = base + from * a.ld_row;
      if (count > 0 && wanted(count) > 0) {
        if (behind == N)
          v[m] = PAST ? __builtin_nontemporal_load(reinterpret_cast<const U*>(row + at))
                      : *reinterpret_cast<const U*>(row + at);
        else  // a run's last bytes
          v[m] = load_bytes<V>(row + at, behind);
      }
    }
#pragma unroll
    for (int m = 0; m < WMAX; ++m) {
      const int count = __builtin_amdgcn_readlane(moves, m);
      char* row = base + m * a.ld_row;
      if (count > 0) {
        const int n = wanted(count);
        if (n == N)
          __builtin_nontemporal_store(v[m], reinterpret_cast<U*>(row + at));
        else if (n > 0)
          store_bytes(row + at, v[m], n);
      }
    }
  }
}

// How a call is cut up: bytes of a column, of a run, and workgroups' pieces.
struct Cut {
  bool dense, past;
  int64_t run, slabs, items;
  Cut(const BeamReorderArgs& a, int bytes) {
    dense = a.ld_position == a.run || a.positions == 1;
    run = dense ? a.run * a.positions : a.run;
    slabs = ((run + bytes - 1) / bytes * (dense ? 1 : a.positions) + kSlab - 1) / kSlab;
    items = slabs * a.sequences * a.mid * a.outer * a.count;
    // loads past the caches where the states are more than those hold (2.1 GB 448
    // against 471 us, 524 MB 118 and 125); fewer may be there still (131 MB 34 and 28)
    past = items * kSlab * bytes * a.beams > int64_t(256) << 20;
  }
};
// Registers for 32 or 64 beams are four bytes each.
int column_bytes(int beams) { return beams <= 16 ? 16 : 4; }

template <int WMAX, typename V, bool DENSE>
void launch_reorder(const BeamReorderArgs& a, const Cut& c, hipStream_t st) {
  const dim3 grid((unsigned)std::min<int64_t>(c.items, 1 << 20));
  hipLaunchKernelGGL(c.past ? (k_beam_reorder<WMAX, V, DENSE, true>) : (k_beam_reorder<WMAX, V, DENSE, false>), grid,
                     dim3(256), 0, st, a, c.run, (uint32_t)c.slabs, (uint32_t)c.items);
}
template <int WMAX, typename V>
void launch_reorder(const BeamReorderArgs& a, hipStream_t st) {
  const Cut c(a, (int)sizeof(V));
  if (c.dense)
    launch_reorder<WMAX, V, true>(a, c, st);
  else
    launch_reorder<WMAX, V, false>(a, c, st);
}

}  // namespace

int64_t beam_chunks(int64_t n) { return (n + kPart - 1) / kPart * (kPart / kChunk); }

hipError_t launch_beam_select(const BeamArgs& a, int64_t sequences, hipStream_t st) {
  const int chunks = (int)beam_chunks(a.n), W = a.beams;
  void (*choose)(BeamArgs, int);
  // Short rows are scanned by the sequence's one workgroup.  us a call from the host
  // and in a graph, against two launches: 4 x 4096 10.8 and 8.2, 13.5 and 9.0; 8 x 4096
  // candidates 11.6 and 10.1, 14.2 and 9.8; with four parts a wave, 2 x 16384, 10.8 and
  // 9.6, 13.7 and 7.9, with eight 11.9 and 11.7, 13.7 and 7.6.
  const int split = W > 8 ? 1 : W > 4 ? 2 : 4;
  if (W <= 16 && chunks / 4 <= kParts * split) {
    choose = W > 8 ? k_beam_choose<1, 1, true> : W > 4 ? k_beam_choose<1, 2, true> : k_beam_choose<1, 4, true>;
  } else {
    hipLaunchKernelGGL(k_beam_scan, dim3((unsigned)((chunks + 15) / 16), (unsigned)(sequences * W)), dim3(256), 0, st, a,
                       chunks);
    choose = chunks > 256 * kQuads || W > 32 ? k_beam_choose<0, 1, false>
             : W > 16                       ? k_beam_choose<2, 1, false>
             : W > 8                        ? k_beam_choose<1, 1, false>
             : W > 4                        ? k_beam_choose<1, 2, false>
                                            : k_beam_choose<1, 4, false>;
  }
  hipLaunchKernelGGL(choose, dim3((unsigned)sequences), dim3(kThreads), 0, st, a, chunks);
  return hipGetLastError();
}

bool beam_reorder_fits(const BeamReorderArgs& a) {
  const int64_t most = (int64_t(1) << 31) - 1;
  const Cut c(a, column_bytes(a.beams));
  int64_t items = c.slabs;
  if (items > most || (!c.dense && (a.positions > most || a.run > most))) return false;
  for (int64_t n : {a.sequences, a.mid, a.outer, (int64_t)a.count}) {
    if (n > most / items) return false;
    items *= n;
  }
  return true;
}

hipError_t launch_beam_reorder(const BeamReorderArgs& a, hipStream_t st) {
  if (a.beams <= 4)
    launch_reorder<4, u32x4>(a, st);
  else if (a.beams <= 8)
    launch_reorder<8, u32x4>(a, st);
  else if (a.beams <= 16)
    launch_reorder<16, u32x4>(a, st);
  else if (a.beams <= 32)
    launch_reorder<32, uint32_t>(a, st);
  else
    launch_reorder<64, uint32_t>(a, st);
  return hipGetLastError();
}

}  // namespace fh
