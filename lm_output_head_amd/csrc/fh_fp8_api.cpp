// C ABI of the fp8 operators: hidden states in fp8, the fp8 product and the dense
// head on it.  Argument checking, ownership and launches; the kernels are in
// fh_fp8_quant.hip and fh_fp8.hip.

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>
#include <string>

#include "fh_fp8.hpp"
#include "fh_serve.hpp"
#include "fh_serve_host.hpp"
#include "flashhead.h"

struct fh_fp8 {
  int device = 0;
  int64_t n = 0, k = 0;
  void* packed = nullptr;  // the int8 product's fragment order
  float* scales = nullptr;
};

namespace {

using fh::DeviceGuard;
using fh::aligned16;
using fh::aligned_to;
using fh::check_choice;
using fh::check_ld;
using fh::check_workspace;
using fh::fail;
using fh::guarded;
using fh::hip_fail;
using fh::inverse_of;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxChannels = int64_t(1) << 27;  // grids stay below 2^32 threads, a wave or more per 16 channels
constexpr int64_t kMaxK = (int64_t(1) << 17) - 1;   // places of a row in 32 bits

int64_t groups_of(int64_t x) { return (x + 127) / 128; }
int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

struct Rows {
  const char* name;
  const void* p;
  int64_t ld, width;
  size_t elem;
};

// Strides and alignment of the matrices that a call was given.
template <size_t N>
fh_status check_rows_of(const Rows (&rows)[N], int64_t B) {
  for (const Rows& t : rows) {
    if (!t.p) continue;
    const fh_status s = check_ld(t.name, t.ld, t.width, B);
    if (s != FH_OK) return s;
    if (!aligned_to(t.p, t.elem)) return fail(FH_EINVAL, "rows must be aligned to their elements");
  }
  return FH_OK;
}

fh_status check_states(const void* x, fh_dtype dtype, int64_t B, int64_t d, const void* out_q, const void* out_scale) {
  if (!x) return fail(FH_EINVAL, "x is NULL");
  if (dtype != FH_F32 && dtype != FH_BF16) return fail(FH_EINVAL, "unknown dtype");
  if (!out_q || !out_scale) return fail(FH_EINVAL, "out_q and out_scale must not be NULL");
  if (B < 1 || B > kMaxRows) return fail(FH_EINVAL, "B outside [1, 2^31 - 1]");
  if (d < 1 || d > kMaxRows) return fail(FH_EINVAL, "d outside [1, 2^31 - 1]");
  return FH_OK;
}

void free_fp8(fh_fp8* w) {
  if (!w) return;
  (void)hipFree(w->packed);
  (void)hipFree(w->scales);
  delete w;
}

fh_status create_fp8(const uint8_t* codes, const float* scales, const void* W, fh_dtype dtype, int64_t n, int64_t k,
                     hipStream_t st, fh_fp8** out) {
  if (!out) return fail(FH_EINVAL, "out is NULL");
  if (n < 1 || n > kMaxChannels) return fail(FH_EINVAL, "n outside [1, 2^27]");
  if (k < 1 || k > kMaxK) return fail(FH_EINVAL, "k outside [1, 131071]");
  fh_fp8* w = new (std::nothrow) fh_fp8();
  if (!w) return fail(FH_ENOMEM, "host allocation failed");
  w->n = n;
  w->k = k;
  int* bad = nullptr;
  int hbad = 0;
  const bool bf16 = dtype == FH_BF16;
  const size_t scale_bytes = sizeof(float) * (size_t)(groups_of(n) * groups_of(k));
  hipError_t r = hipGetDevice(&w->device);
  if (r == hipSuccess) r = hipMalloc(&w->packed, (size_t)fh::w8a8_packed_bytes(n, k));
  if (r == hipSuccess) r = hipMalloc((void**)&w->scales, scale_bytes);
  if (r == hipSuccess) {
    if (codes) {
      r = hipMemcpyAsync(w->scales, scales, scale_bytes, hipMemcpyDeviceToDevice, st);
      if (r == hipSuccess)
        r = fh::launch_w8a8_pack(reinterpret_cast<const int8_t*>(codes), nullptr, false, nullptr, n, k, w->packed, st);
    } else {
      r = hipMalloc((void**)&bad, sizeof(int));
      if (r == hipSuccess) r = hipMemsetAsync(bad, 0, sizeof(int), st);
      if (r == hipSuccess) r = fh::launch_fp8_scales(W, bf16, n, k, w->scales, bad, st);
      if (r == hipSuccess) r = hipMemcpyAsync(&hbad, bad, sizeof(int), hipMemcpyDeviceToHost, st);
      if (r == hipSuccess) r = fh::launch_fp8_pack(W, bf16, w->scales, n, k, w->packed, st);
    }
  }
  const hipError_t waited = hipStreamSynchronize(st);  // also before freeing after a failure
  if (r == hipSuccess) r = waited;
  (void)hipFree(bad);
  if (r != hipSuccess) {
    free_fp8(w);
    return hip_fail(r, "fp8 weight");
  }
  if (hbad) {
    free_fp8(w);
    return fail(FH_EINVAL, "W holds an infinity or NaN");
  }
  *out = w;
  return FH_OK;
}

bool rows_aligned(const fh_fp8* w, const uint8_t* q, int64_t ld_q, int64_t B) {
  return aligned16(q) && w->k % 16 == 0 && (ld_q % 16 == 0 || B == 1);
}

// Workspace: the aligned copy of q's rows where they need one, then the head's partials.
int64_t copy_bytes(const fh_fp8* w, const uint8_t* q, int64_t ld_q, int64_t B) {
  return rows_aligned(w, q, ld_q, B) ? 0 : round16(w->k) * B;
}
int64_t need_bytes(const fh_fp8* w, const uint8_t* q, int64_t ld_q, int64_t B, bool forward) {
  const int64_t parts = forward ? (int64_t)sizeof(fh::Part) * B * fh::fp8_parts(w->n, w->k, B) : 0;
  return copy_bytes(w, q, ld_q, B) + parts;
}

fh_status check_rows(const fh_fp8* w, int64_t ld_q, int64_t B) {
  if (!w) return fail(FH_EINVAL, "w is NULL");
  if (B < 1 || B > 65535) return fail(FH_EINVAL, "B outside [1, 65535]");
  if (!fh::fp8_fits(w->n, w->k, B)) return fail(FH_EINVAL, "n and B together too large for one call");
  return check_ld("ld_q", ld_q, w->k, B);
}

fh_status check_product(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale, int64_t ld_scale,
                        int64_t B) {
  fh_status s = check_rows(w, ld_q, B);
  if (s != FH_OK) return s;
  if (!q || !q_scale) return fail(FH_EINVAL, "q and q_scale must not be NULL");
  if (!aligned_to(q_scale, 4)) return fail(FH_EINVAL, "q_scale must be aligned to 4 bytes");
  return check_ld("ld_scale", ld_scale, groups_of(w->k), B);
}

// q's rows where the kernel can read them, and what else a product reads.
hipError_t take_rows(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale, int64_t ld_scale, int64_t B,
                     void* workspace, hipStream_t st, fh::FP8Args* a) {
  a->W = w->packed;
  a->ws = w->scales;
  a->n = w->n;
  a->k = (int)w->k;
  a->B = (int)B;
  a->q = q;
  a->ld_q = ld_q;
  a->qs = q_scale;
  a->ld_qs = ld_scale;
  if (rows_aligned(w, q, ld_q, B)) return hipSuccess;
  a->q = static_cast<const uint8_t*>(workspace);
  a->ld_q = round16(w->k);
  return fh::launch_w8a8_align(reinterpret_cast<const int8_t*>(q), ld_q, B, w->k, static_cast<int8_t*>(workspace),
                               a->ld_q, st);
}

fh_status matmul(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale, int64_t ld_scale, int64_t B,
                 void* out, int64_t ld_out, fh::FP8Out kind, void* workspace, int64_t workspace_bytes,
                 hipStream_t st) {
  fh_status s = check_product(w, q, ld_q, q_scale, ld_scale, B);
  if (s != FH_OK) return s;
  if (!out) return fail(FH_EINVAL, "out is NULL");
  if (!aligned_to(out, kind == fh::FP8Out::kF32 ? 4 : 2)) return fail(FH_EINVAL, "out must be aligned to its elements");
  s = check_ld("ld_out", ld_out, w->n, B);
  if (s == FH_OK) s = check_workspace(workspace, workspace_bytes, need_bytes(w, q, ld_q, B, false));
  if (s != FH_OK) return s;
  DeviceGuard g(w->device);
  if (!g.ok) return fail(FH_EHIP, "cannot select the weight's device");
  fh::FP8Args a{};
  hipError_t r = take_rows(w, q, ld_q, q_scale, ld_scale, B, workspace, st, &a);
  a.out = out;
  a.ld_out = ld_out;
  if (r == hipSuccess) r = fh::launch_fp8(a, kind, st);
  return r == hipSuccess ? FH_OK : hip_fail(r, "fp8 product launch");
}

}  // namespace

extern "C" {

fh_status fh_rmsnorm_fp8(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, const void* weight,
                         fh_dtype dtype, int64_t B, int64_t d, float eps, float weight_offset, void* out,
                         int64_t ld_out, void* out_residual, int64_t ld_out_residual, uint8_t* out_q, int64_t ld_q,
                         float* out_scale, int64_t ld_scale, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    fh_status s = check_states(x, dtype, B, d, out_q, out_scale);
    if (s != FH_OK) return s;
    if (!(eps >= 0.f && std::isfinite(eps))) return fail(FH_EINVAL, "eps must be finite and >= 0");
    if (!std::isfinite(weight_offset)) return fail(FH_EINVAL, "weight_offset must be finite");
    const size_t elem = dtype == FH_BF16 ? 2 : 4;
    const Rows rows[] = {{"ld_x", x, ld_x, d, elem},
                         {"ld_residual", residual, ld_residual, d, elem},
                         {"ld_out", out, ld_out, d, elem},
                         {"ld_out_residual", out_residual, ld_out_residual, d, elem},
                         {"ld_q", out_q, ld_q, d, 1},
                         {"ld_scale", out_scale, ld_scale, groups_of(d), 4}};
    s = check_rows_of(rows, B);
    if (s != FH_OK) return s;
    if (weight && !aligned_to(weight, elem)) return fail(FH_EINVAL, "weight must be aligned to its elements");
    if (out && out == out_residual) return fail(FH_EINVAL, "out and out_residual are the same storage");
    for (const Rows& o : {rows[2], rows[3]})
      for (const Rows& i : {rows[0], rows[1]})
        if (B > 1 && o.p && o.p == i.p && o.ld != i.ld)
          return fail(FH_EINVAL, std::string(o.name) + " and " + i.name + " differ on the same storage");
    fh::FP8QuantArgs a{x,    residual,    weight, out,    out_residual,    out_q, out_scale, ld_x,
                       ld_residual, ld_out, ld_out_residual, ld_q, ld_scale, d,     eps,       weight_offset};
    const hipError_t r = fh::launch_rmsnorm_fp8(a, dtype == FH_BF16, B, static_cast<hipStream_t>(stream));
    return r == hipSuccess ? FH_OK : hip_fail(r, "fp8 norm launch");
  });
}

fh_status fh_fp8_quant(const void* x, int64_t ld_x, fh_dtype dtype, int64_t B, int64_t d, uint8_t* out_q, int64_t ld_q,
                       float* out_scale, int64_t ld_scale, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    fh_status s = check_states(x, dtype, B, d, out_q, out_scale);
    if (s != FH_OK) return s;
    const Rows rows[] = {{"ld_x", x, ld_x, d, dtype == FH_BF16 ? size_t(2) : size_t(4)},
                         {"ld_q", out_q, ld_q, d, 1},
                         {"ld_scale", out_scale, ld_scale, groups_of(d), 4}};
    s = check_rows_of(rows, B);
    if (s != FH_OK) return s;
    fh::FP8QuantArgs a{};
    a.x = x;
    a.ld_x = ld_x;
    a.out_q = out_q;
    a.ld_q = ld_q;
    a.out_scale = out_scale;
    a.ld_scale = ld_scale;
    a.d = d;
    const hipError_t r = fh::launch_fp8_quant(a, dtype == FH_BF16, B, static_cast<hipStream_t>(stream));
    return r == hipSuccess ? FH_OK : hip_fail(r, "fp8 quantisation launch");
  });
}

fh_status fh_fp8_create(const void* W, fh_dtype dtype, int64_t n, int64_t k, void* stream, fh_fp8** out) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!W) return fail(FH_EINVAL, "W is NULL");
    if (dtype != FH_F32 && dtype != FH_BF16) return fail(FH_EINVAL, "unknown dtype");
    if (!aligned_to(W, dtype == FH_BF16 ? 2 : 4)) return fail(FH_EINVAL, "W must be aligned to its elements");
    return create_fp8(nullptr, nullptr, W, dtype, n, k, static_cast<hipStream_t>(stream), out);
  });
}

fh_status fh_fp8_create_codes(const uint8_t* codes, const float* scales, int64_t n, int64_t k, void* stream,
                              fh_fp8** out) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!codes || !scales) return fail(FH_EINVAL, "codes and scales must not be NULL");
    if (!aligned_to(scales, 4)) return fail(FH_EINVAL, "scales must be aligned to 4 bytes");
    return create_fp8(codes, scales, nullptr, FH_F32, n, k, static_cast<hipStream_t>(stream), out);
  });
}

void fh_fp8_destroy(fh_fp8* w) {
  if (!w) return;
  DeviceGuard g(w->device);
  (void)hipDeviceSynchronize();
  free_fp8(w);
}

fh_status fh_fp8_get(const fh_fp8* w, uint8_t* codes, float* scales, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (!w) return fail(FH_EINVAL, "w is NULL");
    if (!codes || !scales) return fail(FH_EINVAL, "codes and scales must not be NULL");
    DeviceGuard g(w->device);
    if (!g.ok) return fail(FH_EHIP, "cannot select the weight's device");
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t r = fh::launch_w8a8_unpack(w->packed, w->n, w->k, reinterpret_cast<int8_t*>(codes), st);
    if (r == hipSuccess)
      r = hipMemcpyAsync(scales, w->scales, sizeof(float) * (size_t)(groups_of(w->n) * groups_of(w->k)),
                         hipMemcpyDeviceToDevice, st);
    return r == hipSuccess ? FH_OK : hip_fail(r, "copy fp8 weight");
  });
}

int64_t fh_fp8_workspace(const fh_fp8* w, const uint8_t* q, int64_t ld_q, int64_t B, int forward) {
  return guarded<int64_t>(FH_ENOMEM, [&]() -> int64_t {
    const fh_status s = check_rows(w, ld_q, B);
    return s != FH_OK ? (int64_t)s : need_bytes(w, q, ld_q, B, forward != 0);
  });
}

fh_status fh_fp8_matmul(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale, int64_t ld_scale,
                        int64_t B, void* out, int64_t ld_out, fh_dtype out_dtype, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    if (out_dtype != FH_F32 && out_dtype != FH_BF16) return fail(FH_EINVAL, "unknown out_dtype");
    return matmul(w, q, ld_q, q_scale, ld_scale, B, out, ld_out,
                  out_dtype == FH_BF16 ? fh::FP8Out::kBf16 : fh::FP8Out::kF32, workspace, workspace_bytes,
                  static_cast<hipStream_t>(stream));
  });
}

fh_status fh_fp8_matmul_native(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale,
                               int64_t ld_scale, int64_t B, void* out, int64_t ld_out, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    return matmul(w, q, ld_q, q_scale, ld_scale, B, out, ld_out, fh::FP8Out::kBf16Native, workspace, workspace_bytes,
                  static_cast<hipStream_t>(stream));
  });
}

fh_status fh_fp8_forward(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale, int64_t ld_scale,
                         int64_t B, int mode, float temperature, uint64_t seed, int32_t* out_token,
                         float* out_token_logit, float* out_lse, float* out_logits, int64_t ld_logits, void* workspace,
                         int64_t workspace_bytes, void* stream) {
  return guarded(FH_ENOMEM, [&]() -> fh_status {
    fh_status s = check_product(w, q, ld_q, q_scale, ld_scale, B);
    if (s == FH_OK) s = check_choice(mode, temperature);
    if (s != FH_OK) return s;
    if (!out_token) return fail(FH_EINVAL, "out_token is NULL");
    for (const void* p : {(const void*)out_token, (const void*)out_token_logit, (const void*)out_lse,
                          (const void*)out_logits})
      if (!aligned_to(p, 4)) return fail(FH_EINVAL, "outputs must be aligned to 4 bytes");
    if (out_logits) s = check_ld("ld_logits", ld_logits, w->n, B);
    if (s == FH_OK) s = check_workspace(workspace, workspace_bytes, need_bytes(w, q, ld_q, B, true));
    if (s != FH_OK) return s;
    DeviceGuard g(w->device);
    if (!g.ok) return fail(FH_EHIP, "cannot select the weight's device");
    hipStream_t st = static_cast<hipStream_t>(stream);
    fh::FP8Args a{};
    hipError_t r = take_rows(w, q, ld_q, q_scale, ld_scale, B, workspace, st, &a);
    a.out = out_logits;
    a.ld_out = ld_logits;
    a.token_sample = mode == FH_TOKEN_SAMPLE;
    a.inverse_t = a.token_sample ? inverse_of(temperature) : 1.f;
    a.seed = seed;
    a.parts = reinterpret_cast<fh::Part*>(static_cast<char*>(workspace) + copy_bytes(w, q, ld_q, B));
    if (r == hipSuccess) r = fh::launch_fp8(a, fh::FP8Out::kHead, st);
    if (r == hipSuccess)
      r = fh::launch_choice(a.parts, B, fh::fp8_parts(w->n, w->k, B), out_token, out_token_logit, out_lse, st);
    return r == hipSuccess ? FH_OK : hip_fail(r, "fp8 head launch");
  });
}

}  // extern "C"
