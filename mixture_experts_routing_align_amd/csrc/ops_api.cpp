// C ABI of the operators around the layer (include/moe_mi355x_ops.h): argument
// checks and launches.  As in api.cpp, every host argument is checked before the
// HIP runtime is touched, and nothing allocates, synchronises or reads device
// memory.
#include <math.h>

#include <algorithm>

#include "moe_internal.h"
#include "moe_mi355x_ops.h"
#include "ops_internal.h"

namespace {

using moe::fail_status;

constexpr int64_t kInt32Limit = (int64_t)1 << 31;

int hip_status(const char* fn, hipError_t e) {
  return e == hipSuccess ? MOE_OK : fail_status(MOE_ERR_HIP, "%s: %s", fn, hipGetErrorString(e));
}

int null_arg(const char* fn, const char* what) { return fail_status(MOE_ERR_NULL, "%s: %s is NULL", fn, what); }

int check_aligned16(const char* fn, const char* what, const void* p) {
  if (reinterpret_cast<uintptr_t>(p) % 16) return fail_status(MOE_ERR_SHAPE, "%s: %s is not 16-byte aligned", fn, what);
  return MOE_OK;
}

int check_rows(const char* fn, const char* what, int64_t rows) {
  if (rows < 0) return fail_status(MOE_ERR_SHAPE, "%s: %s=%lld is negative", fn, what, (long long)rows);
  if (rows >= kInt32Limit) return fail_status(MOE_ERR_LIMIT, "%s: %s=%lld reaches 2^31", fn, what, (long long)rows);
  return MOE_OK;
}

int check_norm_shape(const char* fn, int64_t M, int32_t H) {
  if (int rc = check_rows(fn, "M", M)) return rc;
  if (H < 1) return fail_status(MOE_ERR_SHAPE, "%s: H=%d must be >= 1", fn, H);
  if (H > MOE_NORM_MAX_H) return fail_status(MOE_ERR_LIMIT, "%s: H=%d exceeds %d columns", fn, H, MOE_NORM_MAX_H);
  return MOE_OK;
}

int check_stream_type(const char* fn, moe_dtype t) {
  if (t != MOE_DT_BF16 && t != MOE_DT_F32) return fail_status(MOE_ERR_SHAPE, "%s: type %d is neither bf16 nor float32", fn, (int)t);
  return MOE_OK;
}

// Shape rules of the calls that map slots to rows.
int check_slots(const char* fn, int64_t M, int32_t top_k, int32_t H, int64_t rows) {
  if (int rc = check_rows(fn, "M", M)) return rc;
  if (int rc = check_rows(fn, "rows", rows)) return rc;
  if (top_k < 1) return fail_status(MOE_ERR_SHAPE, "%s: top_k=%d must be >= 1", fn, top_k);
  if (H < 1) return fail_status(MOE_ERR_SHAPE, "%s: H=%d must be >= 1", fn, H);
  if (H >= (1 << 29)) return fail_status(MOE_ERR_LIMIT, "%s: H=%d: a row reaches 2^30 bytes", fn, H);
  if (M >= kInt32Limit / top_k) return fail_status(MOE_ERR_LIMIT, "%s: M*top_k = %lld*%d slots reach 2^31", fn, (long long)M, top_k);
  return MOE_OK;
}

// Shape rules of the products; `unit` the multiple K and N come in, `item` the
// bytes of an element.
int check_product(const char* fn, int64_t rows, int32_t E, int32_t N, int32_t K, int32_t parts, int unit, int item,
                  const int32_t* offsets, const int32_t* counts) {
  if (int rc = check_rows(fn, "rows", rows)) return rc;
  if (E < 1) return fail_status(MOE_ERR_SHAPE, "%s: E=%d must be >= 1", fn, E);
  if (E > MOE_MAX_EXPERTS) return fail_status(MOE_ERR_LIMIT, "%s: E=%d exceeds %d experts", fn, E, MOE_MAX_EXPERTS);
  if (N < 1 || K < 1 || N % unit || K % unit)
    return fail_status(MOE_ERR_SHAPE, "%s: N=%d, K=%d must be positive multiples of %d", fn, N, K, unit);
  if ((offsets == nullptr) != (counts == nullptr))
    return fail_status(MOE_ERR_NULL, "%s: expert_offsets and expert_counts go together", fn);
  if (offsets == nullptr && E != 1)
    return fail_status(MOE_ERR_NULL, "%s: expert_offsets is NULL (a dense product needs E = 1)", fn);
  // the kernels address one expert's weights, and the rows of one tile, with 31-bit byte offsets
  if ((int64_t)N * K * item >= kInt32Limit)
    return fail_status(MOE_ERR_LIMIT, "%s: one expert's weights, %d x %d, reach 2^31 bytes", fn, N, K);
  if ((int64_t)std::max(K, N * (int64_t)parts > INT32_MAX ? INT32_MAX : N * parts) * item * 256 >= kInt32Limit)
    return fail_status(MOE_ERR_LIMIT, "%s: 256 rows of %d or %d x %d elements reach 2^31 bytes", fn, K, parts, N);
  // the smallest tiles there are, 16 rows by 16 columns, counted in 31 bits, as are the
  // workgroups up to a whole second grid dimension (at most 2^21 more)
  const int64_t tiles = (rows / 16 + std::min<int64_t>(E, rows)) * ((std::max(N, K) + 15) / 16);
  if (tiles >= kInt32Limit - ((int64_t)1 << 22)) return fail_status(MOE_ERR_LIMIT, "%s: %lld tiles reach 2^31", fn, (long long)tiles);
  return MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_ops_abi_version(void) { return 1; }

int moe_add_rms_norm(const void* x, int64_t ldx, const void* residual, moe_dtype rdt, void* residual_out,
                     const void* weight, float eps, void* out, moe_dtype odt, float* out_scale, float* rstd, int64_t M,
                     int32_t H, hipStream_t stream) {
  const char* fn = "moe_add_rms_norm";
  if (int rc = check_norm_shape(fn, M, H)) return rc;
  if (ldx < H) return fail_status(MOE_ERR_SHAPE, "%s: ldx=%lld is less than H=%d", fn, (long long)ldx, H);
  if (!(eps >= 0.f) || isinf(eps)) return fail_status(MOE_ERR_SHAPE, "%s: eps must be finite and not negative", fn);
  if (residual != nullptr) {
    if (int rc = check_stream_type(fn, rdt)) return rc;
  } else if (residual_out != nullptr) {
    return fail_status(MOE_ERR_SHAPE, "%s: residual_out without residual", fn);
  }
  if (odt == MOE_DT_E4M3) {
    if (H % 128) return fail_status(MOE_ERR_SHAPE, "%s: 8-bit rows need H=%d in whole 128-column blocks", fn, H);
  } else if (odt != MOE_DT_BF16) {
    return fail_status(MOE_ERR_SHAPE, "%s: output type %d is neither bf16 nor e4m3", fn, (int)odt);
  }
  if (M == 0) return MOE_OK;
  if (x == nullptr) return null_arg(fn, "x");
  if (weight == nullptr) return null_arg(fn, "weight");
  if (out == nullptr) return null_arg(fn, "out");
  if (odt == MOE_DT_E4M3 && out_scale == nullptr) return null_arg(fn, "out_scale");
  moe::NormArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.res = residual;
  a.zout = residual_out;
  a.w = weight;
  a.eps = eps;
  a.out = out;
  a.scale = odt == MOE_DT_E4M3 ? out_scale : nullptr;
  a.rstd = rstd;
  a.M = M;
  a.H = H;
  return hip_status(fn, moe::launch_norm(a, rdt == MOE_DT_F32, stream));
}

size_t moe_add_rms_norm_backward_workspace_bytes(int64_t M, int32_t H) {
  if (check_norm_shape("moe_add_rms_norm_backward_workspace_bytes", M, H) || M == 0) return 0;
  return moe::norm_backward_workspace(M, H);
}

int moe_add_rms_norm_backward(const void* dy, const void* z, moe_dtype zdt, const void* weight, const float* rstd,
                              const void* dz, void* dx, float* dweight, int64_t M, int32_t H, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "moe_add_rms_norm_backward";
  if (int rc = check_norm_shape(fn, M, H)) return rc;
  if (int rc = check_stream_type(fn, zdt)) return rc;
  if (M > 0) {
    if (dy == nullptr) return null_arg(fn, "dy");
    if (z == nullptr) return null_arg(fn, "z");
    if (weight == nullptr) return null_arg(fn, "weight");
    if (rstd == nullptr) return null_arg(fn, "rstd");
    if (dx == nullptr) return null_arg(fn, "dx");
    const size_t need = dweight != nullptr ? moe::norm_backward_workspace(M, H) : 0;
    if (need && workspace == nullptr) return null_arg(fn, "workspace");
    if (workspace_bytes < need)
      return fail_status(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, needs %zu", fn, workspace_bytes, need);
    if (need)
      if (int rc = check_aligned16(fn, "workspace", workspace)) return rc;
  } else if (dweight == nullptr) {
    return MOE_OK;
  }
  moe::NormBackwardArgs a{};
  a.dy = dy;
  a.z = z;
  a.w = weight;
  a.rstd = rstd;
  a.dz = dz;
  a.dx = dx;
  a.M = M;
  a.H = H;
  return hip_status(fn, moe::launch_norm_backward(a, zdt == MOE_DT_F32, dweight, static_cast<float*>(workspace), stream));
}

int moe_permute(const void* x, moe_dtype dt, const float* x_scale, const int32_t* token_to_perm, int64_t M, int32_t top_k,
                int32_t H, void* out, float* out_scale, int64_t rows, hipStream_t stream) {
  const char* fn = "moe_permute";
  if (int rc = check_slots(fn, M, top_k, H, rows)) return rc;
  if (dt != MOE_DT_BF16 && dt != MOE_DT_E4M3) return fail_status(MOE_ERR_SHAPE, "%s: type %d is neither bf16 nor e4m3", fn, (int)dt);
  if (dt == MOE_DT_E4M3 && H % 128) return fail_status(MOE_ERR_SHAPE, "%s: 8-bit rows need H=%d in whole 128-column blocks", fn, H);
  if (M == 0 || rows == 0) return MOE_OK;
  if (x == nullptr) return null_arg(fn, "x");
  if (token_to_perm == nullptr) return null_arg(fn, "token_to_perm");
  if (out == nullptr) return null_arg(fn, "out");
  if (dt == MOE_DT_E4M3 && (x_scale == nullptr || out_scale == nullptr)) return null_arg(fn, "a scale array of the 8-bit rows");
  moe::PermuteArgs a{};
  a.x = x;
  a.x_scale = x_scale;
  a.perm = token_to_perm;
  a.out = out;
  a.out_scale = out_scale;
  a.M = M;
  a.rows = rows;
  a.top_k = top_k;
  a.row_bytes = dt == MOE_DT_E4M3 ? H : 2 * H;
  a.scales = dt == MOE_DT_E4M3 ? H / 128 : 0;
  return hip_status(fn, moe::launch_permute(a, stream));
}

int moe_unpermute(const void* y, const int32_t* token_to_perm, const float* topk_weights, int64_t M, int32_t top_k,
                  int32_t H, void* out, int64_t rows, hipStream_t stream) {
  const char* fn = "moe_unpermute";
  if (int rc = check_slots(fn, M, top_k, H, rows)) return rc;
  if (M == 0) return MOE_OK;
  if (y == nullptr && rows > 0) return null_arg(fn, "y");
  if (token_to_perm == nullptr) return null_arg(fn, "token_to_perm");
  if (out == nullptr) return null_arg(fn, "out");
  moe::UnpermuteArgs a{static_cast<const uint16_t*>(y), token_to_perm, topk_weights, static_cast<uint16_t*>(out), M, rows, top_k, H};
  return hip_status(fn, moe::launch_unpermute(a, stream));
}

int moe_unpermute_backward(const void* dout, const void* y, const int32_t* token_to_perm, const float* topk_weights,
                           int64_t M, int32_t top_k, int32_t H, void* dy, float* dweights, int64_t rows,
                           hipStream_t stream) {
  const char* fn = "moe_unpermute_backward";
  if (int rc = check_slots(fn, M, top_k, H, rows)) return rc;
  if (M == 0) return MOE_OK;
  if (dout == nullptr) return null_arg(fn, "dout");
  if (rows > 0 && (y == nullptr || dy == nullptr)) return null_arg(fn, "y or dy");
  if (token_to_perm == nullptr) return null_arg(fn, "token_to_perm");
  if (topk_weights == nullptr) return null_arg(fn, "topk_weights");
  if (dweights == nullptr) return null_arg(fn, "dweights");
  moe::UnpermuteBackwardArgs a{static_cast<const uint16_t*>(dout), static_cast<const uint16_t*>(y), token_to_perm, topk_weights,
                               static_cast<uint16_t*>(dy), dweights, M, rows, top_k, H};
  return hip_status(fn, moe::launch_unpermute_backward(a, stream));
}

int moe_grouped_linear(const moe_linear_desc* d, hipStream_t stream) {
  const char* fn = "moe_grouped_linear";
  if (d == nullptr) return null_arg(fn, "descriptor");
  if (d->wdt != MOE_W_BF16 && d->wdt != MOE_W_FP8_E4M3)
    return fail_status(MOE_ERR_SHAPE, "%s: weight dtype %d is neither row-major bf16 nor block-scaled e4m3", fn, (int)d->wdt);
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SWIGLU) return fail_status(MOE_ERR_SHAPE, "%s: unknown activation %d", fn, (int)d->act);
  if (d->ydt != MOE_DT_BF16 && d->ydt != MOE_DT_E4M3)
    return fail_status(MOE_ERR_SHAPE, "%s: output type %d is neither bf16 nor e4m3", fn, (int)d->ydt);
  const bool fp8 = d->wdt == MOE_W_FP8_E4M3, gated = d->act == MOE_ACT_SWIGLU;
  if (int rc = check_product(fn, d->rows, d->E, d->N, d->K, gated ? 2 : 1, fp8 ? 128 : 8, fp8 ? 1 : 2, d->expert_offsets,
                             d->expert_counts))
    return rc;
  if (d->ydt == MOE_DT_E4M3 && d->N % 128)
    return fail_status(MOE_ERR_SHAPE, "%s: 8-bit rows need N=%d in whole 128-column blocks", fn, d->N);
  if (!gated && (d->up.w != nullptr || d->up_bias != nullptr))
    return fail_status(MOE_ERR_SHAPE, "%s: up weights or bias without the SwiGLU activation", fn);
  if (d->rows == 0) return MOE_OK;
  if (d->x == nullptr) return null_arg(fn, "x");
  if (d->w.w == nullptr) return null_arg(fn, "w");
  if (gated && d->up.w == nullptr) return null_arg(fn, "up");
  if (fp8 && (d->x_scale == nullptr || d->w.scale == nullptr || (gated && d->up.scale == nullptr)))
    return null_arg(fn, "a scale array of the 8-bit rows or weights");
  if (d->y == nullptr) return null_arg(fn, "y");
  if (d->ydt == MOE_DT_E4M3 && d->y_scale == nullptr) return null_arg(fn, "y_scale");
  const struct {
    const char* name;
    const void* p;
  } ptrs[] = {{"x", d->x},       {"w", d->w.w},       {"up", d->up.w},   {"bias", d->bias}, {"up_bias", d->up_bias},
              {"residual", d->residual}, {"y", d->y}, {"preact", d->preact}};
  for (const auto& p : ptrs)
    if (int rc = check_aligned16(fn, p.name, p.p)) return rc;
  // bf16 rows replace the residual's element by element; a row of codes would lie over
  // another row's residual
  const char* y0 = static_cast<const char*>(d->y);
  const char* r0 = static_cast<const char*>(d->residual);
  const int64_t cells = d->rows * d->N;
  if (d->ydt == MOE_DT_E4M3 && r0 != nullptr && y0 < r0 + 2 * cells && r0 < y0 + cells)
    return fail_status(MOE_ERR_SHAPE, "%s: 8-bit y overlaps residual", fn);
  moe::LinearArgs a{};
  a.offsets = d->expert_offsets;
  a.counts = d->expert_counts;
  a.rows = (int)d->rows;
  a.E = d->E;
  a.N = d->N;
  a.K = d->K;
  a.x = d->x;
  a.x_scale = d->x_scale;
  a.w[0] = d->w.w;
  a.w[1] = d->up.w;
  a.ws[0] = static_cast<const float*>(d->w.scale);
  a.ws[1] = static_cast<const float*>(d->up.scale);
  a.bias[0] = static_cast<const uint16_t*>(d->bias);
  a.bias[1] = static_cast<const uint16_t*>(d->up_bias);
  a.residual = static_cast<const uint16_t*>(d->residual);
  a.y = d->y;
  a.y_scale = d->ydt == MOE_DT_E4M3 ? d->y_scale : nullptr;
  a.preact = static_cast<uint16_t*>(d->preact);
  a.act = d->act;
  a.parts = gated ? 2 : 1;
  return hip_status(fn, moe::launch_linear(a, fp8, stream));
}

int moe_grouped_act_backward(const void* dy, const void* preact, moe_act act, const int32_t* expert_offsets,
                             const int32_t* expert_counts, int64_t rows, int32_t E, int32_t N, void* dz, hipStream_t stream) {
  const char* fn = "moe_grouped_act_backward";
  if (act <= MOE_ACT_NONE || act > MOE_ACT_SWIGLU)
    return fail_status(MOE_ERR_SHAPE, "%s: activation %d has no gradient kernel", fn, (int)act);
  const int parts = act == MOE_ACT_SWIGLU ? 2 : 1;
  if (int rc = check_product(fn, rows, E, N, 8, parts, 8, 2, expert_offsets, expert_counts)) return rc;
  if (rows == 0) return MOE_OK;
  if (dy == nullptr) return null_arg(fn, "dy");
  if (preact == nullptr) return null_arg(fn, "preact");
  if (dz == nullptr) return null_arg(fn, "dz");
  if (int rc = check_aligned16(fn, "dy", dy)) return rc;
  if (int rc = check_aligned16(fn, "preact", preact)) return rc;
  if (int rc = check_aligned16(fn, "dz", dz)) return rc;
  moe::LinearArgs a{};
  a.offsets = expert_offsets;
  a.counts = expert_counts;
  a.rows = (int)rows;
  a.E = E;
  a.N = N;
  a.act = act;
  a.parts = parts;
  return hip_status(fn, moe::launch_act_backward(a, static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(preact),
                                                 static_cast<uint16_t*>(dz), stream));
}

int moe_grouped_linear_backward_x(const void* dz, const void* w, const void* up, const int32_t* expert_offsets,
                                  const int32_t* expert_counts, int64_t rows, int32_t E, int32_t N, int32_t K, void* dx,
                                  hipStream_t stream) {
  const char* fn = "moe_grouped_linear_backward_x";
  const int parts = up != nullptr ? 2 : 1;
  if (int rc = check_product(fn, rows, E, N, K, parts, 8, 2, expert_offsets, expert_counts)) return rc;
  if (rows == 0) return MOE_OK;
  if (dz == nullptr) return null_arg(fn, "dz");
  if (w == nullptr) return null_arg(fn, "w");
  if (dx == nullptr) return null_arg(fn, "dx");
  if (int rc = check_aligned16(fn, "dz", dz)) return rc;
  if (int rc = check_aligned16(fn, "w", w)) return rc;
  if (int rc = check_aligned16(fn, "up", up)) return rc;
  if (int rc = check_aligned16(fn, "dx", dx)) return rc;
  moe::LinearArgs a{};
  a.offsets = expert_offsets;
  a.counts = expert_counts;
  a.rows = (int)rows;
  a.E = E;
  a.N = N;
  a.K = K;
  a.dz = dz;
  a.w[0] = w;
  a.w[1] = up;
  a.y = dx;
  a.parts = parts;
  return hip_status(fn, moe::launch_linear_backward_x(a, stream));
}

size_t moe_grouped_linear_backward_w_workspace_bytes(int64_t rows, int32_t E, int32_t N, int32_t K, int32_t gated, int32_t bias) {
  const int parts = gated ? 2 : 1;
  // the row runs do not matter for the size: any non-NULL tables stand for them
  static const int32_t some = 0;
  if (check_product("moe_grouped_linear_backward_w_workspace_bytes", rows, E, N, K, parts, 8, 2, &some, &some)) return 0;
  const int splits = moe::backward_w_splits(rows, E, N, K, parts);
  return splits == 1 ? 0 : (size_t)splits * parts * E * N * ((size_t)K + (bias ? 1 : 0)) * 4;
}

int moe_grouped_linear_backward_w(const void* dz, const void* x, int32_t gated, const int32_t* expert_offsets,
                                  const int32_t* expert_counts, int64_t rows, int32_t E, int32_t N, int32_t K,
                                  moe_dtype wdt, void* dw, void* dup, float* db, float* dup_b, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream) {
  const char* fn = "moe_grouped_linear_backward_w";
  const int parts = gated ? 2 : 1;
  if (int rc = check_product(fn, rows, E, N, K, parts, 8, 2, expert_offsets, expert_counts)) return rc;
  if (int rc = check_stream_type(fn, wdt)) return rc;
  if (rows > 0 && dz == nullptr) return null_arg(fn, "dz");
  if (rows > 0 && x == nullptr) return null_arg(fn, "x");
  if (dw == nullptr) return null_arg(fn, "dw");
  if (gated && dup == nullptr) return null_arg(fn, "dup");
  if (!gated && (dup != nullptr || dup_b != nullptr)) return fail_status(MOE_ERR_SHAPE, "%s: dup or dup_b without gated", fn);
  if (gated && (db == nullptr) != (dup_b == nullptr)) return fail_status(MOE_ERR_NULL, "%s: db and dup_b go together", fn);
  if (int rc = check_aligned16(fn, "dz", dz)) return rc;
  if (int rc = check_aligned16(fn, "x", x)) return rc;
  if (int rc = check_aligned16(fn, "dw", dw)) return rc;
  if (int rc = check_aligned16(fn, "dup", dup)) return rc;
  const size_t need = moe_grouped_linear_backward_w_workspace_bytes(rows, E, N, K, gated, db != nullptr);
  if (need && workspace == nullptr) return null_arg(fn, "workspace");
  if (workspace_bytes < need)
    return fail_status(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, needs %zu", fn, workspace_bytes, need);
  if (need)
    if (int rc = check_aligned16(fn, "workspace", workspace)) return rc;
  moe::LinearArgs a{};
  a.offsets = expert_offsets;
  a.counts = expert_counts;
  a.rows = (int)rows;
  a.E = E;
  a.N = N;
  a.K = K;
  a.dz = dz;
  a.x = x;
  a.parts = parts;
  a.dw[0] = dw;
  a.dw[1] = dup;
  a.dw_f32 = wdt == MOE_DT_F32;
  a.db[0] = db;
  a.db[1] = dup_b;
  a.part = static_cast<float*>(workspace);
  a.splits = moe::backward_w_splits(rows, E, N, K, parts);
  return hip_status(fn, moe::launch_linear_backward_w(a, stream));
}

}  // extern "C"
