// C ABI of decoding by beams: the choice of the best continuations and the
// reordering of states.  Argument checking and launches; the kernels are in
// fh_beam.hip.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <utility>
#include <vector>

#include "fh_beam.hpp"
#include "fh_serve_host.hpp"
#include "flashhead.h"

namespace {

using fh::aligned_to;
using fh::check_ld;
using fh::check_workspace;
using fh::fail;
using fh::guarded;
using fh::hip_fail;

constexpr int64_t kMaxRows = 65535;
constexpr int64_t kMaxWidth = int64_t(1) << 30;  // places of a row in 32 bits, grids below 2^32 threads
constexpr int64_t kMaxBeams = 64, kMaxKeep = 64;
constexpr int64_t kMaxBytes = int64_t(1) << 60;

fh_status check_beams(int64_t sequences, int64_t beams) {
  if (beams < 1 || beams > kMaxBeams) return fail(FH_EINVAL, "beams outside [1, 64]");
  if (sequences < 1 || sequences > kMaxRows / beams) return fail(FH_EINVAL, "sequences * beams outside [1, 65535]");
  return FH_OK;
}

// The largest logit of each 256 and the sum of each 1024.
int64_t need_bytes(int64_t rows, int64_t n) {
  return (int64_t)sizeof(float) * rows * (fh::beam_chunks(n) + fh::beam_chunks(n) / 4);
}

// A call's arguments checked, and as the launcher takes them (but for the states);
// `any` is false where there is nothing to move.
fh_status check_reorder(void* const* states, int64_t count, const fh_beam_layout* layout, int64_t sequences,
                        int64_t beams, const int32_t* parent, const int32_t* lengths, fh::BeamReorderArgs* a,
                        bool* any) {
  *any = false;
  if (count < 0 || count > (int64_t(1) << 20)) return fail(FH_EINVAL, "count outside [0, 2^20]");
  if (!layout || !parent || (count > 0 && !states))
    return fail(FH_EINVAL, "states, layout and parent must not be NULL");
  const fh_status s = check_beams(sequences, beams);
  if (s != FH_OK) return s;
  if (!aligned_to(parent, 4) || !aligned_to(lengths, 4))
    return fail(FH_EINVAL, "parent and lengths must be aligned to 4 bytes");
  const fh_beam_layout& l = *layout;
  if (l.outer < 0 || l.mid < 0 || l.positions < 0 || l.run < 0) return fail(FH_EINVAL, "a size is negative");
  if (l.outer == 0 || l.mid == 0 || l.positions == 0 || l.run == 0) return FH_OK;
  if (l.positions > kMaxBytes / l.run) return fail(FH_EINVAL, "the state is too large");
  // from the smallest stride up, each steps over what the ones before it span:
  // no byte belongs to two places
  std::pair<int64_t, int64_t> dims[] = {
      {l.ld_outer, l.outer}, {l.ld_row, sequences * beams}, {l.ld_mid, l.mid}, {l.ld_position, l.positions}};
  std::sort(dims, dims + 4);
  int64_t span = l.run;
  for (const auto& d : dims) {
    if (d.second == 1) continue;
    if (d.first < span) return fail(FH_EINVAL, "the layout's strides overlap");
    if (d.first > (kMaxBytes - span) / d.second) return fail(FH_EINVAL, "the state is too large");
    span += (d.second - 1) * d.first;
  }
  const uintptr_t list = sizeof(int32_t) * (uintptr_t)(sequences * beams);  // bytes of parent, of lengths
  const auto meets = [&](const void* p, const void* state) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(state);
    return p && a < b + (uintptr_t)span && b < a + list;
  };
  for (int64_t i = 0; i < count; ++i) {
    if (!states[i]) return fail(FH_EINVAL, "a state is NULL");
    if (meets(parent, states[i]) || meets(lengths, states[i]))
      return fail(FH_EINVAL, "parent and lengths must not lie in a state");
  }
  std::vector<void*> sorted(states, states + count);
  std::sort(sorted.begin(), sorted.end());
  if (std::adjacent_find(sorted.begin(), sorted.end()) != sorted.end())
    return fail(FH_EINVAL, "a state is listed twice");
  a->parent = parent;
  a->lengths = lengths;
  a->beams = (int)beams;
  a->sequences = sequences;
  a->outer = l.outer;
  a->mid = l.mid;
  a->positions = l.positions;
  a->run = l.run;
  a->ld_outer = l.ld_outer;
  a->ld_row = l.ld_row;
  a->ld_mid = l.ld_mid;
  a->ld_position = l.ld_position;
  a->count = (int)std::min<int64_t>(count, fh::kReorderStates);  // of the largest launch
  if (count > 0 && !fh::beam_reorder_fits(*a)) return fail(FH_EINVAL, "the states are too large for one call");
  *any = count > 0;
  return FH_OK;
}

}  // namespace

extern "C" {

int64_t fh_beam_workspace(int64_t sequences, int64_t beams, int64_t n) {
  return guarded<int64_t>(FH_ENOMEM, [&]() -> int64_t {
    const fh_status s = check_beams(sequences, beams);
    if (s != FH_OK) return s;
    if (n < 1 || n > kMaxWidth) return fail(FH_EINVAL, "n outside [1, 2^30]");
    return need_bytes(sequences * beams, n);
  });
}

fh_status fh_beam_select(const float* logits, int64_t ld_logits, const int32_t* ids, int64_t ld_ids, int64_t sequences,
                         int64_t beams, int64_t n, int64_t v, const float* lse, const float* scores,
                         const int32_t* finished, int32_t eos, int64_t keep, float* out_score, int32_t* out_token,
                         int32_t* out_parent, int32_t* out_finished, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!logits || !scores) return fail(FH_EINVAL, "logits and scores must not be NULL");
    if (!out_score || !out_token || !out_parent)
      return fail(FH_EINVAL, "out_score, out_token and out_parent must not be NULL");
    fh_status s = check_beams(sequences, beams);
    if (s != FH_OK) return s;
    if (n < 1 || n > kMaxWidth || v < 1 || v > kMaxWidth) return fail(FH_EINVAL, "n and v outside [1, 2^30]");
    if (!ids && n != v) return fail(FH_EINVAL, "logits of all tokens need n = v (ids is NULL)");
    if (keep < 1 || keep > kMaxKeep) return fail(FH_EINVAL, "keep outside [1, 64]");
    if (eos < -1 || eos >= v) return fail(FH_EINVAL, "eos outside [-1, v)");
    if (finished && eos < 0) return fail(FH_EINVAL, "finished beams need an eos token");
    const int64_t rows = sequences * beams;
    s = check_ld("ld_logits", ld_logits, n, rows);
    if (s == FH_OK && ids) s = check_ld("ld_ids", ld_ids, n, rows);
    if (s != FH_OK) return s;
    for (const void* p : {(const void*)logits, (const void*)ids, (const void*)lse, (const void*)scores,
                          (const void*)finished, (const void*)out_score, (const void*)out_token,
                          (const void*)out_parent, (const void*)out_finished})
      if (!aligned_to(p, 4)) return fail(FH_EINVAL, "inputs and outputs must be aligned to 4 bytes");
    if (keep != beams && (out_score == scores || (finished && out_finished == finished)))
      return fail(FH_EINVAL, "outputs on their inputs' storage need keep = beams");
    s = check_workspace(workspace, workspace_bytes, need_bytes(rows, n));
    if (s != FH_OK) return s;
    fh::BeamArgs a{};
    a.z = logits;
    a.ld_z = ld_logits;
    a.ids = ids;
    a.ld_ids = ld_ids;
    a.n = (int)n;
    a.v = (int)v;
    a.beams = (int)beams;
    a.keep = (int)keep;
    a.lse = lse;
    a.scores = scores;
    a.finished = finished;
    a.eos = eos;
    a.out_score = out_score;
    a.out_token = out_token;
    a.out_parent = out_parent;
    a.out_finished = out_finished;
    a.top = static_cast<float*>(workspace);
    a.sum = a.top + rows * fh::beam_chunks(n);
    const hipError_t r = fh::launch_beam_select(a, sequences, static_cast<hipStream_t>(stream));
    return r == hipSuccess ? FH_OK : hip_fail(r, "beam choice launch");
  });
}

fh_status fh_beam_reorder(void* const* states, int64_t count, const fh_beam_layout* layout, int64_t sequences,
                          int64_t beams, const int32_t* parent, const int32_t* lengths, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    fh::BeamReorderArgs a{};
    bool any;
    const fh_status s = check_reorder(states, count, layout, sequences, beams, parent, lengths, &a, &any);
    if (s != FH_OK || !any) return s;
    for (int64_t i = 0; i < count; i += fh::kReorderStates) {
      a.count = (int)std::min<int64_t>(count - i, fh::kReorderStates);
      std::copy(states + i, states + i + a.count, a.state);
      const hipError_t r = fh::launch_beam_reorder(a, static_cast<hipStream_t>(stream));
      if (r != hipSuccess) return hip_fail(r, "reordering launch");
    }
    return FH_OK;
  });
}

fh_status fh_beam_reorder_check(void* const* states, int64_t count, const fh_beam_layout* layout, int64_t sequences,
                                int64_t beams, const int32_t* parent, const int32_t* lengths) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    fh::BeamReorderArgs a{};
    bool any;
    return check_reorder(states, count, layout, sequences, beams, parent, lengths, &a, &any);
  });
}

}  // extern "C"
