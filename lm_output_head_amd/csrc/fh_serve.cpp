// C ABI of the operators around the dense head: the final norm, the int8
// product and the dense head on it, the rules on logits.  Argument checking,
// ownership and launches; the kernels are in fh_norm.hip, fh_w8a8.hip and
// fh_rules.hip.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <exception>
#include <limits>
#include <new>
#include <string>

#include "fh_host.hpp"
#include "fh_serve.hpp"
#include "flashhead.h"

struct fh_w8a8 {
  int device = 0;
  int64_t n = 0, k = 0;
  void* packed = nullptr;  // fragment order
  float* scales = nullptr;
};

namespace {

using fh::DeviceGuard;
using fh::aligned16;
using fh::fail;
using fh::hip_fail;

// No exception leaves a C entry (building an error text can throw).
template <typename R, typename F>
R guarded(R failed, F&& body) noexcept {
  try {
    fh::g_err.clear();
    return body();
  } catch (const std::exception&) {
    return failed;
  }
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxWidth = int64_t(1) << 30;    // n and v: grids stay below 2^32 threads,
constexpr int64_t kMaxChannels = int64_t(1) << 27;  // and the product's, a wave or more per 16 channels
constexpr int64_t kMaxList = int64_t(1) << 30;     // places of a history or list, in 32 bits with a batch past them
constexpr int64_t kMaxK = (int64_t(1) << 17) - 1;  // 128^2 k < 2^31
constexpr int64_t kMaxElems = int64_t(1) << 60;    // rows * stride stays far inside int64

// The stride of `rows` rows of `width` elements, or an error text.
fh_status check_ld(const char* name, int64_t ld, int64_t width, int64_t rows) {
  if (ld < width)
    return fail(FH_EINVAL, std::string(name) + "=" + std::to_string(ld) + " below the row's " +
                               std::to_string(width) + " elements");
  if (ld > kMaxElems / rows) return fail(FH_EINVAL, std::string(name) + " too large");
  return FH_OK;
}

fh_status check_choice(int mode, float temperature) {
  if (mode != FH_TOKEN_ARGMAX && mode != FH_TOKEN_SAMPLE)
    return fail(FH_EINVAL, "mode must be FH_TOKEN_ARGMAX or FH_TOKEN_SAMPLE");
  if (mode == FH_TOKEN_SAMPLE && !(temperature > 0.f && std::isfinite(temperature)))
    return fail(FH_EINVAL, "sampling needs a finite temperature > 0");
  return FH_OK;
}

float inverse_of(float temperature) {
  return (float)std::min(1.0 / (double)temperature, (double)std::numeric_limits<float>::max());
}

fh_status check_workspace(const void* workspace, int64_t bytes, int64_t need) {
  if (need == 0) return FH_OK;
  if (!workspace || bytes < need)
    return fail(FH_EINVAL, "this call needs " + std::to_string(need) + " bytes of workspace");
  if (!aligned16(workspace)) return fail(FH_EINVAL, "workspace must be 16-byte aligned");
  return FH_OK;
}

void free_w8a8(fh_w8a8* w) {
  if (!w) return;
  (void)hipFree(w->packed);
  (void)hipFree(w->scales);
  delete w;
}

fh_status create_w8a8(const int8_t* codes, const float* scales, const void* W, fh_dtype dtype, int64_t n, int64_t k,
                      hipStream_t st, fh_w8a8** out) {
  if (!out) return fail(FH_EINVAL, "out is NULL");
  if (n < 1 || n > kMaxChannels) return fail(FH_EINVAL, "n outside [1, 2^27]");
  if (k < 1 || k > kMaxK) return fail(FH_EINVAL, "k outside [1, 131071]");
  fh_w8a8* w = new (std::nothrow) fh_w8a8();
  if (!w) return fail(FH_ENOMEM, "host allocation failed");
  w->n = n;
  w->k = k;
  int* bad = nullptr;
  int hbad = 0;
  const bool bf16 = dtype == FH_BF16;
  hipError_t r = hipGetDevice(&w->device);
  if (r == hipSuccess) r = hipMalloc(&w->packed, (size_t)fh::w8a8_packed_bytes(n, k));
  if (r == hipSuccess) r = hipMalloc((void**)&w->scales, sizeof(float) * (size_t)n);
  if (r == hipSuccess) {
    if (codes) {
      r = hipMemcpyAsync(w->scales, scales, sizeof(float) * (size_t)n, hipMemcpyDeviceToDevice, st);
    } else {
      r = hipMalloc((void**)&bad, sizeof(int));
      if (r == hipSuccess) r = hipMemsetAsync(bad, 0, sizeof(int), st);
      if (r == hipSuccess) r = fh::launch_w8a8_scales(W, bf16, n, k, w->scales, bad, st);
      if (r == hipSuccess) r = hipMemcpyAsync(&hbad, bad, sizeof(int), hipMemcpyDeviceToHost, st);
    }
  }
  if (r == hipSuccess) r = fh::launch_w8a8_pack(codes, W, bf16, w->scales, n, k, w->packed, st);
  const hipError_t waited = hipStreamSynchronize(st);  // also before freeing after a failure
  if (r == hipSuccess) r = waited;
  (void)hipFree(bad);
  if (r != hipSuccess) {
    free_w8a8(w);
    return hip_fail(r, "int8 weight");
  }
  if (hbad) {
    free_w8a8(w);
    return fail(FH_EINVAL, "W holds an infinity or NaN");
  }
  *out = w;
  return FH_OK;
}

bool rows_aligned(const fh_w8a8* w, const int8_t* q, int64_t ld_q, int64_t B) {
  return aligned16(q) && w->k % 16 == 0 && (ld_q % 16 == 0 || B == 1);
}

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

// Workspace: the aligned copy of q's rows where they need one, then the head's partials.
int64_t copy_bytes(const fh_w8a8* w, const int8_t* q, int64_t ld_q, int64_t B) {
  return rows_aligned(w, q, ld_q, B) ? 0 : round16(w->k) * B;
}
int64_t need_bytes(const fh_w8a8* w, const int8_t* q, int64_t ld_q, int64_t B, bool forward) {
  const int64_t parts = forward ? (int64_t)sizeof(fh::Part) * B * fh::w8a8_parts(w->n, w->k, B) : 0;
  return copy_bytes(w, q, ld_q, B) + parts;
}

fh_status check_rows(const fh_w8a8* w, int64_t ld_q, int64_t B) {
  if (!w) return fail(FH_EINVAL, "w is NULL");
  if (B < 1 || B > 65535) return fail(FH_EINVAL, "B outside [1, 65535]");
  if (!fh::w8a8_fits(w->n, w->k, B)) return fail(FH_EINVAL, "n and B together too large for one call");
  return check_ld("ld_q", ld_q, w->k, B);
}

fh_status check_product(const fh_w8a8* w, const int8_t* q, int64_t ld_q, const float* q_scale, int64_t B) {
  const fh_status s = check_rows(w, ld_q, B);
  if (s == FH_OK && (!q || !q_scale)) return fail(FH_EINVAL, "q and q_scale must not be NULL");
  return s;
}

// The rules' partials; a row of one part needs none.
int64_t rules_bytes(int64_t B, int64_t n, bool dense) {
  const int64_t parts = fh::rules_parts(B, n, dense);
  return parts > 1 ? (int64_t)sizeof(fh::Part) * B * parts : 0;
}

// q's rows where the kernel can read them, in fields q and ld_q of a.
hipError_t take_rows(const fh_w8a8* w, const int8_t* q, int64_t ld_q, int64_t B, void* workspace, hipStream_t st,
                     fh::W8A8Args* a) {
  a->W = w->packed;
  a->ws = w->scales;
  a->n = w->n;
  a->k = (int)w->k;
  a->B = (int)B;
  a->q = q;
  a->ld_q = ld_q;
  if (rows_aligned(w, q, ld_q, B)) return hipSuccess;
  a->q = static_cast<const int8_t*>(workspace);
  a->ld_q = round16(w->k);
  return fh::launch_w8a8_align(q, ld_q, B, w->k, static_cast<int8_t*>(workspace), a->ld_q, st);
}

}  // namespace

extern "C" {

fh_status fh_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight,
                     fh_dtype dtype, int64_t B, int64_t d, float eps, float weight_offset, void* out, int64_t ld_out,
                     void* out_residual, int64_t ld_out_residual, int8_t* out_q, int64_t ld_q, float* out_scale,
                     void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!x) return fail(FH_EINVAL, "x is NULL");
    if (dtype != FH_F32 && dtype != FH_BF16) return fail(FH_EINVAL, "unknown dtype");
    if (!out && !out_residual && !out_q) return fail(FH_EINVAL, "no output is asked for");
    if (!out_q != !out_scale) return fail(FH_EINVAL, "out_q and out_scale go together");
    if (B < 1 || B > kMaxRows) return fail(FH_EINVAL, "B outside [1, 2^31 - 1]");
    if (d < 1 || d > kMaxRows) return fail(FH_EINVAL, "d outside [1, 2^31 - 1]");
    if (!(eps >= 0.f && std::isfinite(eps))) return fail(FH_EINVAL, "eps must be finite and >= 0");
    if (!std::isfinite(weight_offset)) return fail(FH_EINVAL, "weight_offset must be finite");
    const struct Rows { const char* name; const void* p; int64_t ld; bool elems; } rows[] = {
        {"ld_x", x, ld_x, true}, {"ld_residual", residual, ld_residual, true}, {"ld_out", out, ld_out, true},
        {"ld_out_residual", out_residual, ld_out_residual, true}, {"ld_q", out_q, ld_q, false}};
    const size_t elem = dtype == FH_BF16 ? 2 : 4;
    for (const auto& t : rows) {
      if (!t.p) continue;
      const fh_status s = check_ld(t.name, t.ld, d, B);
      if (s != FH_OK) return s;
      if (t.elems && !aligned_to(t.p, elem)) return fail(FH_EINVAL, "rows must be aligned to their elements");
    }
    if ((weight && !aligned_to(weight, elem)) || (out_scale && !aligned_to(out_scale, 4)))
      return fail(FH_EINVAL, "weight and out_scale must be aligned to their elements");
    if (out && out == out_residual) return fail(FH_EINVAL, "out and out_residual are the same storage");
    for (const auto& o : {rows[2], rows[3]})
      for (const auto& i : {rows[0], rows[1]})
        if (B > 1 && o.p && o.p == i.p && o.ld != i.ld)
          return fail(FH_EINVAL, std::string(o.name) + " and " + i.name + " differ on the same storage");
    fh::NormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.out = out;
    a.out_residual = out_residual;
    a.out_q = out_q;
    a.out_scale = out_scale;
    a.ld_x = ld_x;
    a.ld_residual = ld_residual;
    a.ld_out = ld_out;
    a.ld_out_residual = ld_out_residual;
    a.ld_q = ld_q;
    a.d = d;
    a.eps = eps;
    a.offset = weight_offset;
    const hipError_t r = fh::launch_rmsnorm(a, dtype == FH_BF16, B, static_cast<hipStream_t>(stream));
    return r == hipSuccess ? FH_OK : hip_fail(r, "norm launch");
  });
}

fh_status fh_w8a8_create(const void* W, fh_dtype dtype, int64_t n, int64_t k, void* stream, fh_w8a8** out) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!W) return fail(FH_EINVAL, "W is NULL");
    if (dtype != FH_F32 && dtype != FH_BF16) return fail(FH_EINVAL, "unknown dtype");
    if (!aligned_to(W, dtype == FH_BF16 ? 2 : 4)) return fail(FH_EINVAL, "W must be aligned to its elements");
    return create_w8a8(nullptr, nullptr, W, dtype, n, k, static_cast<hipStream_t>(stream), out);
  });
}

fh_status fh_w8a8_create_codes(const int8_t* codes, const float* scales, int64_t n, int64_t k, void* stream,
                               fh_w8a8** out) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!codes || !scales) return fail(FH_EINVAL, "codes and scales must not be NULL");
    if (!aligned_to(scales, 4)) return fail(FH_EINVAL, "scales must be aligned to 4 bytes");
    return create_w8a8(codes, scales, nullptr, FH_F32, n, k, static_cast<hipStream_t>(stream), out);
  });
}

void fh_w8a8_destroy(fh_w8a8* w) {
  if (!w) return;
  DeviceGuard g(w->device);
  (void)hipDeviceSynchronize();
  free_w8a8(w);
}

fh_status fh_w8a8_get(const fh_w8a8* w, int8_t* codes, float* scales, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!w) return fail(FH_EINVAL, "w is NULL");
    if (!codes || !scales) return fail(FH_EINVAL, "codes and scales must not be NULL");
    DeviceGuard g(w->device);
    if (!g.ok) return fail(FH_EHIP, "cannot select the weight's device");
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t r = fh::launch_w8a8_unpack(w->packed, w->n, w->k, codes, st);
    if (r == hipSuccess)
      r = hipMemcpyAsync(scales, w->scales, sizeof(float) * (size_t)w->n, hipMemcpyDeviceToDevice, st);
    return r == hipSuccess ? FH_OK : hip_fail(r, "copy int8 weight");
  });
}

int64_t fh_w8a8_workspace(const fh_w8a8* w, const int8_t* q, int64_t ld_q, int64_t B, int forward) {
  return guarded<int64_t>(FH_ENOMEM, [&]() -> int64_t {
    const fh_status s = check_rows(w, ld_q, B);
    return s != FH_OK ? (int64_t)s : need_bytes(w, q, ld_q, B, forward != 0);
  });
}

fh_status fh_w8a8_matmul(const fh_w8a8* w, const int8_t* q, int64_t ld_q, const float* q_scale, int64_t B, void* out,
                         int64_t ld_out, fh_dtype out_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    fh_status s = check_product(w, q, ld_q, q_scale, B);
    if (s != FH_OK) return s;
    if (!out) return fail(FH_EINVAL, "out is NULL");
    if (out_dtype != FH_F32 && out_dtype != FH_BF16) return fail(FH_EINVAL, "unknown out_dtype");
    if (!aligned_to(out, out_dtype == FH_BF16 ? 2 : 4) || !aligned_to(q_scale, 4))
      return fail(FH_EINVAL, "out and q_scale must be aligned to their elements");
    s = check_ld("ld_out", ld_out, w->n, B);
    if (s == FH_OK) s = check_workspace(workspace, workspace_bytes, need_bytes(w, q, ld_q, B, false));
    if (s != FH_OK) return s;
    DeviceGuard g(w->device);
    if (!g.ok) return fail(FH_EHIP, "cannot select the weight's device");
    hipStream_t st = static_cast<hipStream_t>(stream);
    fh::W8A8Args a{};
    hipError_t r = take_rows(w, q, ld_q, B, workspace, st, &a);
    a.qs = q_scale;
    a.out = out;
    a.ld_out = ld_out;
    if (r == hipSuccess) r = fh::launch_w8a8(a, out_dtype == FH_BF16, false, st);
    return r == hipSuccess ? FH_OK : hip_fail(r, "int8 product launch");
  });
}

fh_status fh_w8a8_forward(const fh_w8a8* w, const int8_t* q, int64_t ld_q, const float* q_scale, int64_t B, int mode,
                          float temperature, uint64_t seed, int32_t* out_token, float* out_token_logit, float* out_lse,
                          float* out_logits, int64_t ld_logits, void* workspace, int64_t workspace_bytes,
                          void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    fh_status s = check_product(w, q, ld_q, q_scale, B);
    if (s == FH_OK) s = check_choice(mode, temperature);
    if (s != FH_OK) return s;
    if (!out_token) return fail(FH_EINVAL, "out_token is NULL");
    for (const void* p : {(const void*)q_scale, (const void*)out_token, (const void*)out_token_logit,
                          (const void*)out_lse, (const void*)out_logits})
      if (!aligned_to(p, 4)) return fail(FH_EINVAL, "q_scale and outputs must be aligned to 4 bytes");
    if (out_logits) s = check_ld("ld_logits", ld_logits, w->n, B);
    if (s == FH_OK) s = check_workspace(workspace, workspace_bytes, need_bytes(w, q, ld_q, B, true));
    if (s != FH_OK) return s;
    DeviceGuard g(w->device);
    if (!g.ok) return fail(FH_EHIP, "cannot select the weight's device");
    hipStream_t st = static_cast<hipStream_t>(stream);
    fh::W8A8Args a{};
    hipError_t r = take_rows(w, q, ld_q, B, workspace, st, &a);
    a.qs = q_scale;
    a.out = out_logits;
    a.ld_out = ld_logits;
    a.token_sample = mode == FH_TOKEN_SAMPLE;
    a.inverse_t = a.token_sample ? inverse_of(temperature) : 1.f;
    a.seed = seed;
    a.parts = reinterpret_cast<fh::Part*>(static_cast<char*>(workspace) + copy_bytes(w, q, ld_q, B));
    if (r == hipSuccess) r = fh::launch_w8a8(a, false, true, st);
    if (r == hipSuccess)
      r = fh::launch_choice(a.parts, B, fh::w8a8_parts(w->n, w->k, B), out_token, out_token_logit, out_lse, st);
    return r == hipSuccess ? FH_OK : hip_fail(r, "int8 head launch");
  });
}

int64_t fh_logits_workspace(int64_t B, int64_t n) {
  return guarded<int64_t>(FH_ENOMEM, [&]() -> int64_t {
    if (B < 1 || B > 65535) return fail(FH_EINVAL, "B outside [1, 65535]");
    if (n < 1 || n > kMaxWidth) return fail(FH_EINVAL, "n outside [1, 2^30]");
    return std::max(rules_bytes(B, n, true), rules_bytes(B, n, false));
  });
}

fh_status fh_logits_apply(const float* logits, int64_t ld_logits, const int32_t* ids, int64_t ld_ids, int64_t B,
                          int64_t n, int64_t v, const fh_logit_rules* rules, int mode, float temperature,
                          uint64_t seed, float* out_logits, int64_t ld_out, int32_t* out_token,
                          float* out_token_logit, float* out_lse, void* workspace, int64_t workspace_bytes,
                          void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!logits) return fail(FH_EINVAL, "logits is NULL");
    if (B < 1 || B > 65535) return fail(FH_EINVAL, "B outside [1, 65535]");
    if (n < 1 || n > kMaxWidth || v < 1 || v > kMaxWidth) return fail(FH_EINVAL, "n and v outside [1, 2^30]");
    if (!ids && n != v) return fail(FH_EINVAL, "logits of all tokens need n = v (ids is NULL)");
    const bool choice = out_token || out_token_logit || out_lse;
    if (!choice && !out_logits) return fail(FH_EINVAL, "no output is asked for");
    fh_status s = check_choice(mode, temperature);
    if (s == FH_OK) s = check_ld("ld_logits", ld_logits, n, B);
    if (s == FH_OK && ids) s = check_ld("ld_ids", ld_ids, n, B);
    if (s == FH_OK && out_logits) s = check_ld("ld_out", ld_out, n, B);
    if (s != FH_OK) return s;
    if (out_logits == logits && ld_out != ld_logits && B > 1)
      return fail(FH_EINVAL, "ld_out and ld_logits differ on the same storage");
    fh::RulesArgs a{};
    const fh_logit_rules none{};
    const fh_logit_rules& l = rules ? *rules : none;
    for (const void* p : {(const void*)logits, (const void*)ids, (const void*)out_logits, (const void*)out_token,
                          (const void*)out_token_logit, (const void*)out_lse, (const void*)l.history,
                          (const void*)l.n_prompt, (const void*)l.n_history, (const void*)l.repetition,
                          (const void*)l.frequency, (const void*)l.presence, (const void*)l.bias_ids,
                          (const void*)l.bias, (const void*)l.n_bias, (const void*)l.mask, (const void*)l.mask_row})
      if (!aligned_to(p, 4)) return fail(FH_EINVAL, "logits, rules and outputs must be aligned to 4 bytes");
    if (l.history) {
      if (l.history_len < 0 || l.history_len > kMaxList) return fail(FH_EINVAL, "history_len outside [0, 2^30]");
      s = check_ld("ld_history", l.ld_history, l.history_len, B);
    } else if (l.n_history || l.n_prompt) {
      return fail(FH_EINVAL, "n_history and n_prompt need a history");
    }
    if (s != FH_OK) return s;
    if (!l.bias_ids != !l.bias) return fail(FH_EINVAL, "bias_ids and bias go together");
    if (l.bias_ids) {
      if (l.bias_len < 0 || l.bias_len > kMaxList) return fail(FH_EINVAL, "bias_len outside [0, 2^30]");
      s = check_ld("ld_bias", l.ld_bias, l.bias_len, B);
    } else if (l.n_bias) {
      return fail(FH_EINVAL, "n_bias needs a list of biases");
    }
    if (s != FH_OK) return s;
    if (l.mask) {
      if (l.mask_rows < 1 || l.mask_rows > kMaxRows) return fail(FH_EINVAL, "mask_rows outside [1, 2^31 - 1]");
      if (!l.mask_row && l.mask_rows < B) return fail(FH_EINVAL, "the mask has fewer rows than the logits");
      s = check_ld("ld_mask", l.ld_mask, (v + 31) / 32, l.mask_rows);
    } else if (l.mask_row) {
      return fail(FH_EINVAL, "mask_row needs a mask");
    }
    if (s == FH_OK && choice) s = check_workspace(workspace, workspace_bytes, rules_bytes(B, n, !ids));
    if (s != FH_OK) return s;
    a.z = logits;
    a.ld_z = ld_logits;
    a.ids = ids;
    a.ld_ids = ld_ids;
    a.n = (int)n;
    a.v = (int)v;
    a.history = l.history_len > 0 ? l.history : nullptr;
    a.ld_history = l.ld_history;
    a.history_len = (int)l.history_len;
    a.n_prompt = l.n_prompt;
    a.n_history = l.n_history;
    a.repetition = l.repetition;
    a.frequency = l.frequency;
    a.presence = l.presence;
    a.bias_ids = l.bias_len > 0 ? l.bias_ids : nullptr;
    a.bias = l.bias;
    a.ld_bias = l.ld_bias;
    a.bias_len = (int)l.bias_len;
    a.n_bias = l.n_bias;
    a.mask = l.mask;
    a.ld_mask = l.ld_mask;
    a.mask_rows = (int)l.mask_rows;
    a.mask_row = l.mask_row;
    a.token_sample = mode == FH_TOKEN_SAMPLE;
    a.inverse_t = a.token_sample ? inverse_of(temperature) : 1.f;
    a.seed = seed;
    a.out = out_logits;
    a.ld_out = ld_out;
    a.choice = choice;
    a.out_token = out_token;
    a.out_token_logit = out_token_logit;
    a.out_lse = out_lse;
    a.parts = static_cast<fh::Part*>(workspace);
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t r = fh::launch_rules(a, B, st);
    const int64_t parts = fh::rules_parts(B, n, !ids);
    if (r == hipSuccess && choice && parts > 1)
      r = fh::launch_choice(a.parts, B, parts, out_token, out_token_logit, out_lse, st);
    return r == hipSuccess ? FH_OK : hip_fail(r, "logit rules launch");
  });
}

}  // extern "C"
