// Interface between the C ABI (fh_beam_api.cpp) and the launchers of decoding by beams.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fh {

// The choice of the best continuations (fh_beam.hip): fh_beam_select's arguments
// as checked.
struct BeamArgs {
  const float* z;
  int64_t ld_z;
  const int32_t* ids;       // or null
  int64_t ld_ids;
  int n, v;
  int beams, keep;
  const float* lse;         // or null
  const float* scores;      // [sequences x beams]
  const int32_t* finished;  // or null
  int32_t eos;
  float* out_score;         // [sequences x keep], as the next three
  int32_t* out_token;
  int32_t* out_parent;
  int32_t* out_finished;    // or null
  float* top;               // [rows x beam_chunks]: the largest logit of each 256
  float* sum;               // [rows x beam_chunks / 4]: sum of exp(z - largest) of each 1024
};
int64_t beam_chunks(int64_t n);  // a multiple of 4
hipError_t launch_beam_select(const BeamArgs& a, int64_t sequences, hipStream_t st);

// The reordering of states in place: fh_beam_reorder's arguments as checked, sizes
// and strides in bytes.
constexpr int kReorderStates = 64;  // of a launch
struct BeamReorderArgs {
  void* state[kReorderStates];
  int count;
  const int32_t* parent;   // [sequences x beams]
  const int32_t* lengths;  // [sequences x beams], or null
  int beams;
  int64_t sequences, outer, mid, positions, run;
  int64_t ld_outer, ld_row, ld_mid, ld_position;
};
bool beam_reorder_fits(const BeamReorderArgs& a);  // a launch's pieces are counted in 32 bits
hipError_t launch_beam_reorder(const BeamReorderArgs& a, hipStream_t st);

}  // namespace fh
