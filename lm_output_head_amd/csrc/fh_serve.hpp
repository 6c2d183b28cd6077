// Internal interface between the C ABI (fh_serve.cpp) and the launchers of the
// operators around the dense head.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fh_internal.hpp"

namespace fh {

// The final norm (fh_norm.hip): fh_rmsnorm's arguments as checked.
struct NormArgs {
  const void* x;
  const void* residual;  // or null
  const void* weight;    // or null
  void* out;             // or null, as the next two
  void* out_residual;
  int8_t* out_q;
  float* out_scale;
  int64_t ld_x, ld_residual, ld_out, ld_out_residual, ld_q;
  int64_t d;
  float eps, offset;
};
hipError_t launch_rmsnorm(const NormArgs& a, bool bf16, int64_t B, hipStream_t stream);

// The int8 product and the dense head on it (fh_w8a8.hip).  Weights are kept
// in fragment order: 16 rows x 64 elements of k are 1 KB, lane l's 16 bytes
// row l % 16 and elements 16 (l / 16) .. + 15, tiles of a row group by
// ascending k; rows and elements past n and k are zero.
struct W8A8Args {
  const void* W;         // [ceil(n / 16)][2 ceil(k / 128)][64]
  const float* ws;       // [n]
  int64_t n;
  int k;                 // elements of a row
  const int8_t* q;       // [B x ld_q], 16-byte aligned rows of ceil(k / 16) 16 readable bytes
  int64_t ld_q;
  const float* qs;
  int B;
  void* out;             // float or bf16 [B x ld_out], or null (head)
  int64_t ld_out;
  // head
  int token_sample;
  float inverse_t;       // 1 / T'
  uint64_t seed;
  Part* parts;           // [B x w8a8_parts]
};
int64_t w8a8_packed_bytes(int64_t n, int64_t k);
hipError_t launch_w8a8_scales(const void* W, bool bf16, int64_t n, int64_t k, float* scales, int* bad,
                              hipStream_t st);
// codes as given, or (codes null) of W under scales, into fragment order
hipError_t launch_w8a8_pack(const int8_t* codes, const void* W, bool bf16, const float* scales,
                            int64_t n, int64_t k, void* packed, hipStream_t st);
hipError_t launch_w8a8_unpack(const void* packed, int64_t n, int64_t k, int8_t* codes, hipStream_t st);
// rows of k bytes at any alignment -> rows of ld bytes (a multiple of 16), zero past k
hipError_t launch_w8a8_align(const int8_t* q, int64_t ld_q, int64_t B, int64_t k, int8_t* out,
                             int64_t ld, hipStream_t st);
int64_t w8a8_parts(int64_t n, int64_t k, int64_t B);  // partials per row of the head
bool w8a8_fits(int64_t n, int64_t k, int64_t B);  // a launch holds fewer than 2^32 threads
hipError_t launch_w8a8(const W8A8Args& a, bool out_bf16, bool head, hipStream_t st);

// The rules on logits (fh_rules.hip): fh_logits_apply's arguments as checked.
struct RulesArgs {
  const float* z;
  int64_t ld_z;
  const int32_t* ids;    // or null
  int64_t ld_ids;
  int n, v;
  const int32_t* history;  // or null
  int64_t ld_history;
  int history_len;
  const int32_t* n_prompt;
  const int32_t* n_history;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;  // or null
  const float* bias;
  int64_t ld_bias;
  int bias_len;
  const int32_t* n_bias;
  const uint32_t* mask;  // or null
  int64_t ld_mask;
  int mask_rows;
  const int32_t* mask_row;
  int token_sample;
  float inverse_t;       // 1 / T'
  uint64_t seed;
  float* out;            // or null
  int64_t ld_out;
  int choice;            // whether a token is chosen:
  int32_t* out_token;    // a row of one part writes it here (or null),
  float* out_token_logit;
  float* out_lse;
  Part* parts;           // others their partials [B x rules_parts]
};
int64_t rules_parts(int64_t B, int64_t n, bool dense);  // partials per row; one is its choice
hipError_t launch_rules(const RulesArgs& a, int64_t B, hipStream_t st);
// the choice over each row's parts (w8a8 head, rules)
hipError_t launch_choice(const Part* parts, int64_t B, int64_t nparts, int32_t* out_token,
                         float* out_logit, float* out_lse, hipStream_t st);

}  // namespace fh
